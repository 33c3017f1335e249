"""Norms of query / key heads with the rotation on the GPU, where single values decide: a zero eps with
head counts that leave a wave's round partly filled; elements past the rotated ones beside
infinities, NaN and signed zeros; sines and cosines to half a step; the weights' gradients
summed in 64 bits."""

import numpy as np
import pytest

from oracle import rotation as orot
from tests import gpu_cases as gc
from tests import test_gpu_qk as tq
from tests.test_gpu_qk import Case, q  # noqa: F401  (q: the module's fixture)

pytestmark = pytest.mark.gpu


# ---- eps = 0 ---------------------------------------------------------------------------

@pytest.mark.parametrize("nq,nk", [(1, 1), (3, 1), (4, 4), (15, 5), (7, 2)])
@pytest.mark.parametrize("d,rot", [(128, 128), (80, 32), (64, 64), (256, 64), (12, 4)])
@pytest.mark.parametrize("bf16", [False, True])
def test_zero_eps(q, monkeypatch, nq, nk, d, rot, bf16):  # noqa: F811
    """Rows that are not zero need no eps, whether or not the heads fill a wave's rounds."""
    import torch
    monkeypatch.setattr(tq, "EPS", 0.0)
    c = Case(9, nq, nk, d, rot, True, False, bf16)
    got = c.fwd(q)
    torch.cuda.synchronize()
    c.check_fwd(got)
    got = c.bwd(q)
    torch.cuda.synchronize()
    c.check_bwd(got)


# ---- elements that pass ----------------------------------------------------------------

PASS = [(80, 32), (64, 16), (128, 64), (96, 48), (12, 4), (100, 36), (128, 0), (252, 64), (256, 128)]


def _bits(t):
    import torch
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def _bad_values(bf16):
    """Infinities, quiet and signalling NaN of both signs and a negative zero, as bits."""
    if bf16:
        return np.array([0x7F80, 0xFF80, 0x7FC0, 0xFFC0, 0x7F81, 0xFF93, 0x8000], np.uint16).view(np.int16)
    return np.array([0x7F800000, 0xFF800000, 0x7FC00000, 0xFFC12345, 0x7F800001, 0xFF800101, 0x80000000],
                    np.uint32).view(np.int32)


def _spread(t, rot, bf16, seed):
    """t [M, heads, d] with one bad value in each head, at an element past rot."""
    import torch
    t = t.clone()
    M, H, d = t.shape
    bad = torch.from_numpy(_bad_values(bf16)).cuda()
    rng = np.random.default_rng([seed, d, rot])
    at = torch.from_numpy(rng.integers(rot, d, (M, H))).cuda()[..., None]
    which = torch.arange(M * H, device="cuda").view(M, H, 1) % len(bad)
    _bits(t).scatter_(2, at, bad[which])
    return t


@pytest.mark.parametrize("d,rot", PASS)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
def test_elements_past_rot_pass_bit_for_bit(q, d, rot, inter, bf16):  # noqa: F811
    """Without a norm: what stands past rot comes out with its bits, and leaves the others alone."""
    import torch
    M, nq, nk = 5, 5, 3
    c = Case(M, nq, nk, d, rot, False, inter, bf16)
    Q0, K0 = c.fwd(q)
    dY0 = c.bwd(q)[0].view(M, -1, d)
    rows = c.dY.view(M, nq + 2 * nk, d)
    rows = torch.cat([_spread(rows[:, :nq + nk], rot, bf16, 1), rows[:, nq + nk:]], 1)
    c.dY = rows.reshape(M, -1)
    Q, K = c.fwd(q)
    for got, clean, given in ((Q, Q0, rows[:, :nq]), (K, K0, rows[:, nq:nq + nk])):
        assert torch.equal(_bits(got[..., :rot]), _bits(clean[..., :rot]))
        assert torch.equal(_bits(got[..., rot:]), _bits(given[..., rot:]))
    c.g = [(a, _spread(t, rot, bf16, 2 + i)) for i, (a, t) in enumerate(c.g)]
    dY = c.bwd(q)[0].view(M, -1, d)
    up = torch.cat([t for _, t in c.g], 1)
    assert torch.equal(_bits(dY[..., :rot]), _bits(torch.cat([dY0[:, :nq + nk, :rot], up[:, nq + nk:, :rot]], 1)))
    assert torch.equal(_bits(dY[..., rot:]), _bits(up[..., rot:]))


@pytest.mark.parametrize("d,rot", PASS)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
def test_normed_elements_past_rot(q, d, rot, inter, bf16):  # noqa: F811
    """With a norm a head with an infinity is x * 0: NaN at the infinity, zeros elsewhere, and a
    passed negative zero stays one.  In the backward an infinite gradient of a passed element
    reaches that element of the weight's gradient alone."""
    import torch
    M, nq, nk = 4, 3, 2
    c = Case(M, nq, nk, d, rot, True, inter, bf16)
    rows = c.dY.view(M, -1, d)
    rng = np.random.default_rng(d)
    at = rng.integers(rot, d, (M, nq))
    zero = (at - rot + 1) % (d - rot) + rot        # another element that passes
    for m in range(M):
        for h in range(nq):
            rows[m, h, at[m, h]] = float("inf") if h % 2 else -0.0
            rows[m, h, zero[m, h]] = -0.0
    Q = c.fwd(q)[0]
    for m in range(M):
        for h in range(nq):
            if h % 2:
                hit = torch.zeros(d, dtype=torch.bool, device="cuda")
                hit[at[m, h]] = True
                assert torch.equal(Q[m, h].isnan(), hit) and not bool(Q[m, h][~hit].any())
            else:
                assert bool(Q[m, h].isfinite().all())
            for e in {int(zero[m, h])} - {int(at[m, h])}:
                assert float(Q[m, h, e]) == 0 and bool(torch.signbit(Q[m, h, e]))
    c = Case(M, nq, nk, d, rot, True, inter, bf16)
    want = c.bwd(q)[1:]
    e = [int(v) for v in rng.integers(rot, d, 2)]
    c.g[0][1][1, 2, e[0]] = float("inf")
    c.g[1][1][3, 0, e[1]] = float("-inf")
    for got, clean, j in zip(c.bwd(q)[1:], want, e):
        rest = torch.arange(d, device="cuda") != j
        assert bool(got[j].isinf()) and torch.equal(got[rest], clean[rest])


# ---- angles ----------------------------------------------------------------------------

@pytest.mark.parametrize("far,base", [(4096, 10000.0), (131072, 500000.0), (1 << 24, 10000.0)])
@pytest.mark.parametrize("inter", [False, True])
def test_sines_and_cosines(q, far, base, inter):  # noqa: F811
    """Pairs (1, 0) come out as (cos t, sin t), and backward as (cos t, -sin t): within half a step
    of fp32, 2^-24 of the value, and the error of 64 bits (three roundings of t; 2^-36 for
    sine and cosine on the reduced angle)."""
    import torch
    M, d = 777, 128
    rng = np.random.default_rng(far)
    pos = rng.integers(-far, far, M)
    f = (base ** -(np.arange(d // 2) / (d // 2))).astype(np.float32)
    i, j = orot.pairs(d, inter)
    x = np.zeros((M, 3, d), np.float32)
    x[..., i] = 1.0
    Y, dpos, df = gc.dev_f32(x.reshape(M, -1)), torch.from_numpy(pos).cuda(), gc.dev_f32(f)
    Y = Y.view(M, -1)
    t = pos.astype(np.longdouble)[:, None] * f.astype(np.longdouble)[None]
    co, si = np.cos(t).astype(np.float64), np.sin(t).astype(np.float64)
    slack = 2.0 ** -36 + 4 * 2.0 ** -53 * np.abs(t).astype(np.float64)
    Q, K = q.qk_norm_rope_fwd(Y, dpos, df, 1, 1, interleaved=inter)
    R = Y.view(M, 3, d)
    dY = q.qk_norm_rope_bwd(*(R[:, k:k + 1].contiguous() for k in range(3)), dpos, df, interleaved=inter)[0].view(M, 3, d)
    for z, sign in ((Q[:, 0], 1), (K[:, 0], 1), (dY[:, 0], -1), (dY[:, 1], -1)):
        z = z.cpu().numpy().astype(np.float64)
        for got, want in ((z[:, i], co), (z[:, j], sign * si)):
            tol = 2.0 ** -24 * np.abs(want) + slack
            assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) / tol))


# ---- sums of the weights' gradients ------------------------------------------------------

@pytest.mark.parametrize("M,nq,nk,d", [(333, 15, 5, 64), (1000, 8, 2, 128), (20011, 2, 1, 32), (37, 3, 1, 256)])
def test_weight_gradients_are_summed_in_64_bits(q, M, nq, nk, d):  # noqa: F811
    """Rows of +-1 have the root mean square 1 exactly, so a term is dn x, exact, times 1 / rms (within
    one step, 2^-23, the same for all).  The sum then is the definition's to that, half a step
    of fp32, and one rounding of 64 bits a term."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(M)
    Y = torch.randint(0, 2, (M, (nq + 2 * nk) * d), device="cuda", generator=gen).float() * 2 - 1
    g = [torch.randn((M, n, d), device="cuda", generator=gen) for n in (nq, nk, nk)]
    w = torch.ones(d, device="cuda")
    pos, f = torch.zeros(M, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    got = q.qk_norm_rope_bwd(*g, pos, f, Y, w, w, eps=0.0)[1:]
    x = Y.double().cpu().numpy().reshape(M, -1, d)
    for z, dz, first, n in ((got[0], g[0], 0, nq), (got[1], g[1], nq, nk)):
        term = dz.double().cpu().numpy() * x[:, first:first + n]
        want, mag = term.sum((0, 1)), np.abs(term).sum((0, 1))
        err = np.abs(z.double().cpu().numpy() - want)
        tol = (2.0 ** -24 + 2.0 ** -23) * np.abs(want) + (M * n + 64) * 2.0 ** -53 * mag
        assert np.all(err <= tol), float(np.max(err / tol))


@pytest.mark.parametrize("M,nq,nk,d", [(1, 1, 1, 4), (100, 4, 2, 128), (700, 4, 4, 96), (4097, 8, 2, 256)])
def test_tickets_are_left_zero_and_the_sums_repeat(q, M, nq, nk, d):  # noqa: F811
    """One workgroup, one group of them, a part of the groups and all: every call leaves the workspace's
    header zero and gives the same bits, whatever the partial sums' place held."""
    import torch
    c = Case(M, nq, nk, d, d, True, False, False)
    need = q.qlora_workspace_bytes_qk(q._lib.qlora_qk_shape(M, nq, nk, d, d, 0, 0, tq.EPS), 1)
    want = None
    for fill in (0, 255, 1):
        ws = torch.full((need + 64,), fill, dtype=torch.uint8, device="cuda")
        ws[:q._lib.QLORA_WORKSPACE_HEADER_BYTES].zero_()
        for _ in range(3):
            got = c.bwd(q, ws=ws[:need])
            want = want or got
            for a, b in zip(got, want):
                assert torch.equal(a, b)
        assert not bool(ws[:q._lib.QLORA_WORKSPACE_HEADER_BYTES].any()) and bool((ws[need:] == fill).all())
    c.check_bwd(want)
