"""Where the kernels of group-scaled products and of norms with rotation keep values in scratch memory,
read from their gfx950 assembly: only outside the loops over the weight, the tokens and the
heads.  Most kinds of the largest product tile (64 tokens x 48 rows) put addresses of the second
computation away before the first one's loop and take them back behind it; the backward of
norms in fp32 its thread's index.  No GPU needed."""

import re

import pytest

from tests.test_isa_ext import _asm


def _scratch(body):
    """(store or load, in a loop or not, number of loops before it) of each scratch access: the compiler
    notes at the head of each block which loop it belongs to."""
    found, inside, loops = [], False, 0
    lines = [ln.strip() for ln in body.splitlines()]
    for i, ln in enumerate(lines):
        if re.match(r"\.LBB\w+:|; %bb\.", ln):
            note = ln
            for t in lines[i + 1:]:
                if not t.startswith(";"):
                    break
                note += t
            inside = " Loop" in note
            loops += "Loop Header: Depth=1" in note
        elif ln.startswith("scratch_"):
            found.append((ln.split("_")[1], inside, loops))
    return found, loops


def _kernels(asm, name):
    for m in re.finditer(r"^(_Z\S*" + name + r"I\S*):.*?^\.Lfunc_end", asm, re.S | re.M):
        yield m.group(1), m.group(0)


@pytest.mark.parametrize("source,name,count", [("group_linear", "group_many_kernel", 56),
                                               ("group_linear", "group_few_kernel", 48), ("qk", "qk_fwd_kernel", 20),
                                               ("qk", "qk_bwd_kernel", 18)])
def test_no_scratch_in_a_loop(source, name, count, tmp_path_factory, request):
    cache = request.config.__dict__.setdefault("_asm_of", {})
    if source not in cache:
        cache[source] = _asm(tmp_path_factory, source)
    seen = 0
    for kernel, body in _kernels(cache[source], name):
        seen += 1
        found, loops = _scratch(body)
        assert loops >= 1 and not any(inside for _, inside, _ in found), (kernel, found)
        if "group_many" in name:  # before the first computation's loop, and between it and the second's
            assert all(n == (0 if what == "store" else 1) for what, _, n in found), (kernel, found)
    assert seen == count
