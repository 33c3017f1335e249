"""Forward and backward at the largest weights that the header admits: the code array of almost
2^32 bytes, whose height padded to a multiple of 8 would pass that limit."""

import numpy as np
import pytest

import synth
from oracle import gated as og
from oracle import nf4
from tests import drop_cases as dc
from tests import gpu_cases as gc
from tests.test_gpu_gated import ALPHA, grad_bound, q  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("parts,N", [(1, 1048575), (2, 1048574)])
def test_code_arrays_near_four_gib(q, parts, N):  # noqa: F811
    import torch
    print(f"code array of {N} x 8192 / 2 bytes, {parts} parts", flush=True)
    M, K, r, p = 4, 8192, 8, 0.5
    gen = torch.Generator(device="cuda").manual_seed(4)
    blocks = N * K // 64
    groups = -(-blocks // 256)
    codes = torch.randint(0, 256, (N * K // 2,), dtype=torch.uint8, device="cuda", generator=gen)
    cq = torch.randint(-127, 128, (blocks,), dtype=torch.int8, device="cuda", generator=gen)
    scale = torch.rand(groups, device="cuda", generator=gen) * 1e-4
    offset = torch.full((groups,), 0.03, device="cuda")
    qw = q.NF4Weight(codes, cq, scale, offset, N, K)
    rng = np.random.default_rng(9)
    P = N // parts
    cols = np.array([0, 1, 8190, P // 2, P - 2, P - 1])
    rows = np.concatenate([cols + s * P for s in range(parts)])  # the weight rows that take part
    X = gc.dev_bf16(synth.to_bf16_bits(rng.standard_normal((M, K)).astype(np.float32)))
    A = gc.dev_bf16(synth.to_bf16_bits((rng.standard_normal((parts * r, K)) / 8).astype(np.float32)))
    B = (torch.randn(N, r, device="cuda", generator=gen) * 0.1).bfloat16()
    U = (torch.randn(M, parts * r, device="cuda", generator=gen)).bfloat16()
    at = torch.from_numpy(cols).cuda()
    g = torch.zeros(M, P, dtype=torch.bfloat16, device="cuda")
    g[:, at] = torch.randn(M, len(cols), device="cuda", generator=gen).bfloat16()
    d = q.Dropout(p, seed=5)
    at_rows = torch.from_numpy(rows).cuda()
    gs = gc.host_f32_from_bf16(g[:, at])
    if parts == 1:
        fY, fU = q.linear_fwd(qw, X, A, B, ALPHA, dropout=d)
        dX, dA, dB = q.linear_bwd(qw, g, X, A, B, ALPHA, U, dropout=d)
        dY, eY = gs, np.zeros_like(gs)
    else:
        _, fY, fU = q.gated_fwd(qw, X, A, B, ALPHA, dropout=d)
        Y = torch.randn(M, N, device="cuda", generator=gen).bfloat16()
        dX, dA, dB = q.gated_bwd(qw, g, Y, X, A, B, ALPHA, U, dropout=d)
        Ys = gc.host_f32_from_bf16(Y[:, at_rows])
        dY = og.backward(gs, Ys, "silu")
        eY = grad_bound("silu", gs, Ys, dY)
    torch.cuda.synchronize()
    # W' of those rows: every group of 256 constants is two rows of 128
    Wd = np.empty((len(rows), K))
    for j, n in enumerate(rows):
        lo = n - n % 2
        k = min(2, N - lo)
        b, e = lo * 128, (lo + k) * 128
        stored = {"shape": (k, K), "codes": codes[b * 32:e * 32].cpu().numpy(), "absmax_q": cq[b:e].cpu().numpy(),
                  "dq_scale": scale[lo // 2:lo // 2 + 1].cpu().numpy(),
                  "dq_offset": offset[lo // 2:lo // 2 + 1].cpu().numpy()}
        Wd[j] = nf4.dequantize_bf16(stored).astype(np.float64)[n - lo]
    m, c = dc.mask(M, K, p, 5, 0)
    f = gc.host_f32_from_bf16
    rY, reY, rU, reU = dc.forward(f(X), Wd, f(A), f(B[at_rows]), ALPHA, r, parts, m, c)
    dc.check("Y", dc.bits(fY[:, at_rows]), rY, reY + dc.H * (np.abs(rY) + reY))
    dc.check("U", dc.bits(fU), rU, reU)
    want = dc.backward(dY, eY, f(X), Wd, f(A), f(B[at_rows]), ALPHA, r, parts, m, c, f(U))
    dc.check("dX", dc.bits(dX), *want["dX"])
    dc.check("dA", dc.bits(dA), *want["dA"])
    dc.check("dB", dc.bits(dB[at_rows]), *want["dB"])
    dB[at_rows] = 0
    assert int(dB.count_nonzero()) == 0


def _random_weight(q, N, K, gen):
    import torch
    blocks = N * K // 64
    groups = -(-blocks // 256)
    return q.NF4Weight(torch.randint(0, 256, (N * K // 2,), dtype=torch.uint8, device="cuda", generator=gen),
                       torch.randint(-127, 128, (blocks,), dtype=torch.int8, device="cuda", generator=gen),
                       torch.rand(groups, device="cuda", generator=gen) * 1e-4,
                       torch.rand(groups, device="cuda", generator=gen) * 0.02 + 0.02, N, K)


def test_more_slices_than_workgroups_at_once(q):  # noqa: F811
    """One token of 65536 columns at rank 256: 4096 rank x column slices, more than the card
    holds of the workgroups that wait for them."""
    import torch
    M, K, N, r = 1, 65536, 65536, 256
    print(f"small M: {M} x {K} -> {N}, rank {r}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(6)
    qw = _random_weight(q, N, K, gen)
    X = torch.randn(M, K, device="cuda", generator=gen).bfloat16()
    A = (torch.randn(r, K, device="cuda", generator=gen) / 8).bfloat16()
    B = (torch.randn(N, r, device="cuda", generator=gen) * 0.1).bfloat16()
    _, U = q.linear_fwd(qw, X, A, B, ALPHA)
    torch.cuda.synchronize()
    f = gc.host_f32_from_bf16
    want, e = dc.down(f(X), f(A), ALPHA, r, np.ones((M, K)), 1.0)
    dc.check("U", dc.bits(U), want, e)


@pytest.mark.parametrize("N,K,r", [(32768, 25600, 8), (28672, 25600, 0), (28672, 40960, 0), (16384, 34816, 8)])
@pytest.mark.parametrize("M", [1, 4])
def test_rows_of_many_groups_of_constants(q, N, K, r, M):  # noqa: F811
    """Rows long enough that a wave's part of them touches three groups of 256 block constants.
    One element of X a token, so that each output is one weight (and the adapter's zero)."""
    import torch
    print(f"small M: {M} x {K} -> {N}, rank {r}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(7)
    qw = _random_weight(q, N, K, gen)
    cols = [int(K // 64 * f) * 64 + 7 for f in (0.3, 0.1, 0.6, 0.9)[:M]]
    X = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    X[torch.arange(M, device="cuda"), torch.tensor(cols, device="cuda")] = 1.0
    A = torch.zeros(r, K, dtype=torch.bfloat16, device="cuda") if r else None
    B = torch.ones(N, r, dtype=torch.bfloat16, device="cuda") if r else None
    Y, _ = q.linear_fwd(qw, X, A, B, ALPHA)
    assert torch.equal(Y, q.dequantize(qw)[:, cols].t())
