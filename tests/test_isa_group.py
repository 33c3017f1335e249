"""Waits and registers of the products with group-scaled weights, read from their gfx950 assembly
like tests/test_isa_waits.py does for others: where X goes straight to LDS, a stage's
reads stand behind a wait that leaves at most the other stage's loads and the next block's codes
in flight (what is asked for after the stage itself); every such load has landed when the
stages become the place of the partial sums; kernels do not spill, but for the largest tile's
odd kinds.  No GPU needed."""

import re

import pytest

from tests.test_isa_ext import _asm


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    return _asm(tmp_path_factory, "group_linear")


def _kernels(asm, name):
    for m in re.finditer(r"^(_Z\S*" + name + r"I(\S*?)EEEv\S*):.*?^\.Lfunc_end", asm, re.S | re.M):
        yield [int(v) for v in re.findall(r"L[ib](\d+)E", m.group(2) + "E")], m.group(0)


def test_direct_loads_have_landed(asm):
    seen = 0
    for (xr, nt, *_), body in _kernels(asm, "group_many_kernel"):
        seen += 1
        after = xr // 8 + nt   # loads of a half block of X, loads of a block of codes
        landed, reads, barriers = True, 0, 0
        for line in (ln.strip() for ln in body.splitlines()):
            if line.startswith("buffer_load") and line.endswith(" lds"):
                landed = False
            elif m := re.match(r"s_waitcnt vmcnt\((\d+)\)", line):
                landed = landed or int(m.group(1)) <= after
                drained = int(m.group(1)) == 0
            elif line.startswith("buffer_load"):
                drained = False
            elif line.startswith("ds_read_b128") and not barriers:
                reads += 1
                assert landed, (xr, nt, line)
            elif line.startswith("s_barrier"):
                barriers += 1
                assert barriers > 1 or drained, (xr, nt)
        assert reads >= 2 * 8 and barriers == 2, (xr, nt, reads, barriers)
    assert seen == 7 * 8


def test_no_spills(asm):
    meta = re.findall(r"\.name:\s+(_Z\S+)\n(?:(?!\.name:).)*?\.vgpr_spill_count:\s+(\d+)", asm, re.S)
    assert len(meta) == 7 * 8 + 6 * 8
    spills = {n: int(c) for n, c in meta if "group_" in n and int(c)}
    # 64 tokens x 48 rows hold 252 registers; groups of less than a block want a few more
    assert all("group_many_kernelILi64ELi3E" in n and c <= 24 for n, c in spills.items()), spills
