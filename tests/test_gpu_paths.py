"""Every kernel that the operators with dropout and the gated projections choose between,
against the float64 definition within the derived bounds (tests/drop_cases.py).  Which kernel a
call takes is a cost model's choice, so each case names the kernels it is there for, and the
test reads from the profiler which ones ran."""

import re

import numpy as np
import pytest

from tests import drop_cases as dc
from tests import gpu_cases as gc
from tests.test_gpu_gated import check_all, inputs, run

pytestmark = pytest.mark.gpu
ALPHA = 16.0
NF4, FP4 = 0, 1
INT8, FP8, F32 = 0, 1, 2


@pytest.fixture(scope="module")
def q():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_lora_nf4_amd as lib
    return lib


def traced(fn):
    """fn's result and the names of the library's kernels that it ran, template arguments
    included, in order."""
    import torch
    from torch.profiler import ProfilerActivity, profile
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA]) as prof:
        out = fn()
        torch.cuda.synchronize()
    found = [re.search(r"qlora::\(anonymous namespace\)::(\w+(?:<[^>]*>)?)\(", e.name) for e in prof.events()]
    return out, [m.group(1) for m in found if m]


def took(names, *patterns):
    print("  " + (", ".join(names) or "no kernel names from the profiler: only values are checked"), flush=True)
    if not names:
        return
    for p in patterns:
        assert any(re.match(p + r"(?![\w])", n) for n in names), (p, names)


def quantized(q, W, quant, const):
    """The weight on the device and its W' (from the stored arrays through the oracle, or, for
    the other number types, as the dequantization, tested for itself, gives it)."""
    qw = q.quantize(W, quant_type=quant, const_type=const)
    if (quant, const) == (NF4, INT8):
        return qw, dc.weight64(qw)
    return qw, gc.host_f32_from_bf16(q.dequantize(qw))


# (M, K, P, r, act, p, level table, constants, the forward's kernel)
GATED = [
    # 256 x 256 tiles: ranks through LDS, from memory (past 64), none; odd heights; both
    # activations; every constant type
    (700, 512, 5632, 64, "silu", 0.1, NF4, INT8, "gemm_gated_kernel<0>"),
    (700, 320, 5637, 12, "gelu_tanh", 0.25, FP4, F32, "gemm_gated_kernel<2>"),
    (700, 512, 5632, 72, "gelu_tanh", 0.0, NF4, FP8, "gemm_gated_kernel<1>"),
    (1100, 192, 3001, 20, "silu", 0.1, FP4, INT8, "gemm_gated_kernel<0>"),
    (300, 64, 4097, 0, "gelu_tanh", 0.0, FP4, F32, "gemm_gated_kernel<2>"),
    # smaller tiles, split and whole, with the other constants
    (64, 2048, 520, 16, "silu", 0.1, NF4, FP8, "gemm_mid_kernel<1, true, \\d, true, \\d>"),
    (140, 2112, 501, 24, "gelu_tanh", 0.0, FP4, F32, "gemm_mid_kernel<2, true, \\d, true, \\d>"),
    (520, 256, 3000, 16, "silu", 0.0, NF4, F32, "gemm_mid_kernel<2, true, \\d, false, \\d>"),
    (400, 320, 2501, 40, "silu", 0.1, NF4, FP8, "gemm_mid_kernel<1, true, \\d, false, \\d>"),
]


@pytest.mark.parametrize("M,K,P,r,act,p,quant,const,kernel", GATED)
def test_gated(q, M, K, P, r, act, p, quant, const, kernel):
    import torch
    print(f"gated M={M} K={K} P={P} r={r} {act} p={p} types {quant} {const}", flush=True)
    h = inputs(M, K, P, r, seed=M + K + P)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw, Wd = quantized(q, dev["W"], quant, const)
    d = q.Dropout(p, seed=31 * M + P, offset=P) if p else None
    out, names = traced(lambda: run(q, qw, dev, r, act, d))
    took(names, kernel)
    for a, b in zip(out, run(q, qw, dev, r, act, d)):
        assert (a is None and b is None) or torch.equal(a, b), "not deterministic"
    check_all(q, qw, Wd, h, dev, M, K, P, r, act, p, d, out)


# (M, K, rows of one part, r, parts, p, level table, constants, the forward's kernel, dX's)
LINEAR = [
    # the forward's smaller tiles with the contraction split: every height, one part and several
    (20, 4096, 512, 8, 2, 0.1, NF4, INT8, "gemm_mid_kernel<0, false, 1, true, \\d>", "dx_mid_kernel"),
    (64, 4096, 4096, 16, 1, 0.1, NF4, FP8, "gemm_mid_kernel<1, false, 1, true, \\d>", "dx_mid_kernel<1, 1, true>"),
    (260, 4096, 1000, 8, 1, 0.25, FP4, F32, "gemm_mid_kernel<2, false, 2, true, \\d>", "dx_mid_kernel<2, \\d, false>"),
    (140, 4096, 2000, 72, 1, 0.1, NF4, F32, "gemm_mid_kernel<2, false, 4, true, \\d>", "dx_mid_kernel<2, \\d, true>"),
    (100, 4096, 768, 12, 3, 0.1, FP4, FP8, "gemm_mid_kernel<1, false, \\d, true, \\d>", "dx_mid_kernel<1, \\d, true>"),
    # whole, with two blocks of 32 tokens a tile
    (600, 1024, 512, 16, 1, 0.5, NF4, FP8, "gemm_mid_kernel<1, false, \\d, false, \\d>", "dx_mid_kernel<1, \\d, false>"),
    # dX's smaller tiles split, with the other constants
    (300, 512, 3001, 20, 1, 0.1, NF4, FP8, "gemm_mid_kernel<1, false", "dx_mid_kernel<1, \\d, true>"),
    (150, 2048, 4096, 16, 1, 0.1, FP4, F32, "gemm_mid_kernel<2, false", "dx_mid_kernel<2, \\d, true>"),
    # dX's large tiles split, every constant type
    (80, 512, 12000, 16, 1, 0.1, NF4, INT8, "gemm_mid_kernel<0, false", "gemm_dx_split_kernel<0>"),
    (80, 512, 2560, 16, 4, 0.1, NF4, FP8, "gemm_mid_kernel<1, false", "gemm_dx_split_kernel<1>"),
    (40, 768, 8001, 80, 1, 0.25, FP4, F32, "gemm_mid_kernel<2, false", "gemm_dx_split_kernel<2>"),
    # and whole, several column tiles
    (6000, 2048, 2000, 16, 1, 0.1, NF4, INT8, "gemm_fwd_kernel<0>", "gemm_dx_ext_kernel<0>"),
    (6000, 2048, 2003, 72, 1, 0.1, NF4, FP8, "gemm_fwd_kernel<1>", "gemm_dx_ext_kernel<1>"),
    (6000, 2048, 2000, 12, 1, 0.25, FP4, F32, "gemm_fwd_kernel<2>", "gemm_dx_ext_kernel<2>"),
]


@pytest.mark.parametrize("M,K,Np,r,parts,p,quant,const,fwd,dx", LINEAR)
def test_linear(q, M, K, Np, r, parts, p, quant, const, fwd, dx):
    import torch
    print(f"linear M={M} K={K} Np={Np} r={r} parts={parts} p={p} types {quant} {const}", flush=True)
    h = dc.linear_inputs(M, K, Np, r, parts, seed=M + K + r)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw, Wd = quantized(q, dev["W"], quant, const)
    d = q.Dropout(p, seed=991 * M + 1, offset=r)

    def call():
        Y, U = q.linear_fwd_fused(qw, parts, dev["X"], dev["A"], dev["B"], ALPHA, dropout=d)
        return (Y, U) + q.linear_bwd_fused(qw, parts, dev["dY"], dev["X"], dev["A"], dev["B"], ALPHA, U, dropout=d)

    (Y, U, dX, dA, dB), names = traced(call)
    took(names, fwd, dx)
    for a, b in zip((Y, U, dX, dA, dB), call()):
        assert torch.equal(a, b), "not deterministic"
    X, A, B, dY = dc.f64(h, "X", "A", "B", "dY")
    m, c = dc.mask(M, K, p, d.seed, d.offset)
    rY, eY, rU, eU = dc.forward(X, Wd, A, B, ALPHA, r, parts, m, c)
    dc.check("Y", dc.bits(Y), rY, eY + dc.H * (np.abs(rY) + eY))
    dc.check("U", dc.bits(U), rU, eU)
    want = dc.backward(dY, np.zeros_like(dY), X, Wd, A, B, ALPHA, r, parts, m, c, dc.bits(U))
    for name, got in (("dX", dX), ("dA", dA), ("dB", dB)):
        dc.check(name, dc.bits(got), *want[name])


# (M, K, P, r, p, constants, kernel): the one-launch kernel <constants, X staged, several pieces a
# workgroup, counter hand-over, X staged a wave>
SMALL = [
    (16, 320, 5504, 64, 0.1, INT8, "gemv_ext_kernel<0, true, false, false, false>"),
    (16, 320, 11008, 128, 0.1, INT8, "gemv_ext_kernel<0, false, false, false, false>"),
    (16, 320, 11008, 128, 0.1, FP8, "gemv_ext_kernel<1, false, false, false, false>"),
    (8, 2048, 8200, 1, 0.25, INT8, "gemv_ext_kernel<0, false, false, true, false>"),
    (8, 2048, 8200, 8, 0.25, F32, "gemv_ext_kernel<2, false, false, true, false>"),
    (16, 8192, 40, 0, 0.0, INT8, "gemv_ext_kernel<0, false, false, false, true>"),
    (16, 8192, 40, 0, 0.0, F32, "gemv_ext_kernel<2, false, false, false, true>"),
    (8, 8192, 2050, 128, 0.1, INT8, "gemv_ext_kernel<0, false, true, false, false>"),
    (8, 8192, 2050, 128, 0.1, FP8, "gemv_ext_kernel<1, false, true, false, false>"),
    (16, 8192, 136, 8, 0.1, FP8, "gemv_ext_kernel<1, false, true, false, true>"),
    (16, 8192, 136, 8, 0.1, F32, "gemv_ext_kernel<2, false, true, false, true>"),
    (9, 2048, 515, 128, 0.1, F32, "gemv_ext_kernel<2, true, true, false, false>"),
    (5, 1024, 77, 4, 0.1, FP8, "gemv_ext_kernel<1, true, true, true, false>"),
]


@pytest.mark.parametrize("M,K,P,r,p,const,kernel", SMALL)
def test_gated_small_m(q, M, K, P, r, p, const, kernel):
    import torch
    print(f"gated M={M} K={K} P={P} r={r} p={p} constants {const}", flush=True)
    h = inputs(M, K, P, r, seed=M + K + P)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw, Wd = quantized(q, dev["W"], NF4, const)
    d = q.Dropout(p, seed=31 * M + P, offset=P) if p else None
    out, names = traced(lambda: run(q, qw, dev, r, "silu", d))
    took(names, kernel)
    for a, b in zip(out, run(q, qw, dev, r, "silu", d)):
        assert (a is None and b is None) or torch.equal(a, b), "not deterministic"
    check_all(q, qw, Wd, h, dev, M, K, P, r, "silu", p, d, out)
