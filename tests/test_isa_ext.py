"""Waits and registers of the kernels with dropout and of the gated projections, read from their gfx950 assembly like
tests/test_isa_waits.py does for the others: in the masked staging loops the wait ahead of a
step's masking must retire that step's loads (vmcnt(N) with N <= loads before the loop minus
loads per step, and no other vector memory operation inside the loop); at every barrier of
the extended dX kernel each direct-to-LDS load issued before it must be retired; at each
barrier of the gated forward's pipeline only loads issued after the published tile's may be
in flight; the small-M path's per-wave X stages are read only after their loads' wait; no
kernel spills.  No GPU needed."""

import os
import re
import subprocess

import pytest

from bit_quantized_lora_nf4_amd import build as libbuild
from tests.test_isa_waits import _BR, _VMEM, _all_retired, _barrier_waits, _cfg, _dma, _events, HIPCC


def _asm(tmp_path_factory, name):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("isa") / (name + ".s")
    flags = [f for f in libbuild.FLAGS if f != "-fPIC"]
    cmd = [HIPCC] + flags + ["--cuda-device-only", "-S", os.path.join(libbuild.CSRC, name + ".hip"), "-o", str(out)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    return out.read_text()


@pytest.fixture(scope="module")
def lora_asm(tmp_path_factory):
    return _asm(tmp_path_factory, "lora")


@pytest.fixture(scope="module")
def gemm_asm(tmp_path_factory):
    return _asm(tmp_path_factory, "gemm")


def test_masked_staging_waits(lora_asm):
    kernels = re.findall(r"^(_Z\S*drop_(?:down|reduce)_kernel\S*):", lora_asm, re.M)
    assert len(kernels) == 16, kernels
    for name in kernels:
        body = re.search(r"^" + re.escape(name) + r":.*?^\.Lfunc_end", lora_asm, re.S | re.M).group(0)
        blocks = _cfg(body)
        found = 0
        for h, hb in enumerate(blocks):
            if not re.match(r"; =>This Inner Loop Header: Depth=1", hb["note"]):
                continue
            hid = hb["label"][2:]
            members = {i for i, b in enumerate(blocks) if i == h or f"Header={hid} " in b["note"] + " "}
            lines = [ln for i in sorted(members) for ln in blocks[i]["lines"]]
            if not any(ln.startswith("s_barrier") for ln in lines):
                continue
            assert not [ln for ln in lines if _VMEM.match(ln) and not ln.endswith(" lds")], name
            waits = [int(m.group(1)) for ln in lines if (m := re.match(r"s_waitcnt vmcnt\((\d+)\)", ln))]
            per_step = _dma(lines)
            # the masking reads the step's own chunks right after the one wait
            assert len(waits) == 1, (name, waits)
            pro = sum(_dma(blocks[i]["lines"]) for i in range(len(blocks)) if i not in members)
            # the loads before the loop sit in straight-line blocks: NB - 1 steps of them
            assert pro % per_step == 0 and pro >= per_step, (name, pro, per_step)
            assert waits[0] <= pro - per_step, (name, waits, pro, per_step)
            # the wait precedes the masking reads, which precede the barrier
            order = [("W" if ln.startswith("s_waitcnt vmcnt") else "R" if ln.startswith("ds_read_b128") else
                      "S" if ln.startswith("ds_write_b128") else "B" if ln.startswith("s_barrier") else "")
                     for i in [h] + sorted(members - {h}) for ln in blocks[i]["lines"]]
            order = "".join(order)
            assert re.match(r"^W(RRSS|RSRS)B", order), (name, order[:20])
            found += 1
        assert found == 1, (name, found)


@pytest.mark.parametrize("kernel", ["gemm_dx_ext", "gemm_dx_split"])
@pytest.mark.parametrize("ct", [0, 1, 2])
def test_ext_dx_barrier_waits(gemm_asm, ct, kernel):
    name = re.search(r"^(_Z\S*%s_kernelILi%d\S*):" % (kernel, ct), gemm_asm, re.M).group(1)
    # the whole function: an early exit's s_endpgm may come first in the text
    body = re.search(r"^" + re.escape(name) + r":.*?^\.Lfunc_end", gemm_asm, re.S | re.M).group(0)
    ev = _events(body.replace("s_endpgm", "") + "\ns_endpgm", name)
    waits = _barrier_waits(ev)
    assert len(waits) >= 4
    for i, n in waits:
        j = i - 1
        while j >= 0 and ev[j][0] != "D":
            j -= 1
        if j < 0:
            continue
        after = sum(1 for x in ev[j + 1:i] if x[0] == "R")
        assert n <= after, f"barrier wait vmcnt({n}) with only {after} register loads after the last dY load"


@pytest.mark.parametrize("ct", [0, 1, 2])
def test_gated_barrier_waits(gemm_asm, ct):
    name = re.search(r"^(_Z\S*gemm_gated_kernelILi%d\S*):" % ct, gemm_asm, re.M).group(1)
    ev = _events(gemm_asm, name)
    waits = _barrier_waits(ev)
    assert len(waits) >= 4
    checked = 0
    for i, n in waits:
        j = i - 1
        while j >= 0 and ev[j][0] != "B":
            j -= 1
        if j < 0 or _all_retired(ev, j):
            continue  # a prologue barrier: everything issued before it was retired
        k, seen = j + 1, 0
        while k < i and seen < 4:
            seen += ev[k][0] in ("D", "R")
            k += 1
        after = sum(1 for x in ev[k:i] if x[0] in ("D", "R"))
        assert n <= after, f"barrier wait vmcnt({n}) leaves {n - after} loads of the published tile in flight"
        checked += 1
    assert checked >= 3


def test_mid_barrier_waits(tmp_path_factory):
    """The smaller forward tiles: in the main loop, which alternates barriers that publish two
    X tiles each, the wait at a barrier may leave in flight only the codes issued after those
    tiles' loads; no kernel spills."""
    asm = _asm(tmp_path_factory, "gemm_mid")
    # gemm_mid_kernel<constant type, gated, tile height, split, last tile's height or 0>
    found = re.findall(r"^(_Z\S*gemm_mid_kernelILi\dELb\dELi(\d)ELb\dELi(\d)E\S*):", asm, re.M)
    assert len(found) == 72, len(found)
    for name, ni in [(k, h) for k, *heights in found for h in heights if h != "0"]:
        body = re.search(r"^" + re.escape(name) + r":.*?^\.Lfunc_end", asm, re.S | re.M).group(0)
        lines = [ln.strip() for ln in body.splitlines()]
        labels = {m.group(1): i for i, ln in enumerate(lines) if (m := re.match(r"^(\.LBB\S+):", ln))}
        loops = [lines[labels[m.group(2)]:i + 1] for i, ln in enumerate(lines)
                 if (m := _BR.search(ln)) and m.group(2) in labels and labels[m.group(2)] < i]
        loop = max((x for x in loops if _dma(x) == 8 * int(ni)), key=len)
        # twice around: every wait has the loads of the iteration before it behind it
        pending, seen = [], 0
        for ln in loop + loop:
            if _VMEM.match(ln):
                pending.append("D" if ln.endswith(" lds") else "R")
            elif m := re.match(r"s_waitcnt vmcnt\((\d+)\) lgkmcnt\(0\)$", ln):
                n = int(m.group(1))
                left = pending[len(pending) - n:] if n else []
                assert "D" not in left, (name, n, left)
                pending, seen = left, seen + 1
        assert seen == 8, (name, seen)
    sizes = re.findall(r"\.name:\s+(\S*gemm_mid_\S*kernel\S*)\s.*?\.private_segment_fixed_size:\s+(\d+)", asm, re.S)
    assert len(sizes) == 78 and all(int(n) <= 16 for _, n in sizes), sizes


def test_dx_mid_barrier_waits(tmp_path_factory):
    """dX on smaller tiles: in the main loop of three steps, a step's wait may leave in flight
    only what was loaded behind its dY tile, one later step's tile and codes; no other wait
    makes it wait for its own step's loads; no kernel spills."""
    asm = _asm(tmp_path_factory, "dx_mid")
    kernels = re.findall(r"^(_Z\S*dx_mid_kernelILi(\d)ELi(\d)ELb\d\S*):", asm, re.M)
    assert len(kernels) == 18, len(kernels)
    for name, ct, ni in kernels:
        per_step = int(ni) + (3 if ct == "2" else 5)
        body = re.search(r"^" + re.escape(name) + r":.*?^\.Lfunc_end", asm, re.S | re.M).group(0)
        lines = [ln.strip() for ln in body.splitlines()]
        labels = {m.group(1): i for i, ln in enumerate(lines) if (m := re.match(r"^(\.LBB\S+):", ln))}
        loops = [lines[labels[m.group(2)]:i + 1] for i, ln in enumerate(lines)
                 if (m := _BR.search(ln)) and m.group(2) in labels and labels[m.group(2)] < i]
        loop = max((x for x in loops if _dma(x) == 3 * int(ni)), key=len)
        # twice around, counting the loads issued since the last barrier
        seen, since = 0, 0
        for i, ln in enumerate(loop + loop):
            if _VMEM.match(ln):
                since += 1
            elif m := re.match(r"s_waitcnt (?:.*\s)?vmcnt\((\d+)\)", ln):
                n = int(m.group(1))
                nxt = (loop + loop)[i + 1] if i + 1 < 2 * len(loop) else ""
                if nxt.startswith("s_barrier"):
                    # one whole later step in flight: its tile, then its codes
                    assert n == per_step, (name, n)
                    seen, since = seen + 1, 0
                else:
                    assert n >= since, (name, n, since)
        assert seen == 6, (name, seen)
    sizes = re.findall(r"\.name:\s+(\S*dx_mid_\S*kernel\S*)\s.*?\.private_segment_fixed_size:\s+(\d+)", asm, re.S)
    assert len(sizes) == 21 and all(int(n) == 0 for _, n in sizes), sizes


def test_gemv_ext_x_stage_waits(tmp_path_factory):
    asm = _asm(tmp_path_factory, "gemv")
    # gemv_ext_kernel<CT, XLDS = false, MULTI, DIRECT, XDMA = true>
    kernels = re.findall(r"^(_Z\S*gemv_ext_kernelILi\dELb0ELb\dELb\dELb1E\S*):", asm, re.M)
    assert len(kernels) == 12, kernels
    for name in kernels:
        body = re.search(r"^" + re.escape(name) + r":.*?^\.Lfunc_end", asm, re.S | re.M).group(0)
        lines = [ln.strip() for ln in body.splitlines()]
        labels = {m.group(1): i for i, ln in enumerate(lines) if (m := re.match(r"^(\.LBB\S+):", ln))}
        loops = [(labels[m.group(2)], i) for i, ln in enumerate(lines)
                 if (m := _BR.search(ln)) and m.group(2) in labels and labels[m.group(2)] < i]
        loops = [lines[a:b + 1] for a, b in loops]
        loop = max((x for x in loops if _dma(x) == 16), key=len)  # the main loop: two steps of eight stage loads
        vmem = sum(1 for ln in loop if _VMEM.match(ln))
        assert vmem % 2 == 0, (name, vmem)
        waits, last, seen = [], None, True
        for ln in loop:
            if m := re.match(r"s_waitcnt vmcnt\((\d+)\)", ln):
                last = int(m.group(1))
            elif _VMEM.match(ln):
                seen, last = True, None
            elif ln.startswith("ds_read") and seen:
                waits.append(last)
                seen = False
        assert len(waits) == 2 and all(n is not None and n <= vmem // 2 for n in waits), (name, waits, vmem)
    sizes = re.findall(r"\.name:\s+(\S*gemv_ext\S*)\s.*?\.private_segment_fixed_size:\s+(\d+)", asm, re.S)
    assert len(sizes) == 36 and all(int(n) <= 16 for _, n in sizes), sizes


def test_no_register_spills(gemm_asm, lora_asm):
    for asm, pat in ((gemm_asm, "gemm_dx_ext"), (gemm_asm, "gemm_dx_split"), (gemm_asm, "gemm_gated"), (lora_asm, "drop_")):
        sizes = dict(re.findall(r"\.name:\s+(\S*" + pat + r"\S*kernel\S*)\s.*?\.private_segment_fixed_size:\s+(\d+)",
                                asm, re.S))
        assert len(sizes) >= 3, sizes
        for name, size in sizes.items():
            assert int(size) <= 16, f"{name}: {size} bytes of scratch"
