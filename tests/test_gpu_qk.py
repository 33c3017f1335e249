"""Norms of query and key heads with the position rotation on the GPU, forward and backward,
against float64 within the bounds derived here: head sizes, partial and interleaved
rotations, shared key heads, one token and many, far and negative positions, bf16 and fp32;
guards, streams, captured graphs; and the run of projection, norms and rotation and back.

Bounds.  h is half a step of the output's type relative to the value, u = 2^-24.  Forward: the
sum of squares has positive terms and fewer than 40 roundings, halved by the root, and a few
more of the root, the quotient and the products; the angle is reduced in 64 bits and rounded
to a fraction of a turn of at most 1/2 (pi 2^-25 in the worst case), its sine and cosine are
good to a few u: both together below 64 u of (|a| + |b|), the magnitudes of a pair.  Backward
the same with the sum's own terms for the part that the norm takes off; a weight's gradient
is a sum over tokens and heads whose additions each lane, wave and workgroup counts: at most
their number plus 64 of u times the terms' magnitudes."""

import numpy as np
import pytest

import synth
from oracle import rotation as orot
from tests import gpu_cases as gc

pytestmark = pytest.mark.gpu
EPS, U = 1e-6, 2.0 ** -24


@pytest.fixture(scope="module")
def q():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_lora_nf4_amd as lib
    return lib


class Case:
    def __init__(self, M, nq, nk, d, rot, norm, inter, bf16, far=5000, seed=0, scale=1.5):
        import torch
        print(f"qk M={M} heads={nq},{nk} d={d} rot={rot} norm={norm} inter={inter} bf16={bf16}", flush=True)
        rng = np.random.default_rng([seed, M, nq, nk, d, rot])
        self.M, self.nq, self.nk, self.d, self.rot, self.inter = M, nq, nk, d, rot, inter
        self.h = 2.0 ** -8 if bf16 else U
        self.dtype = torch.bfloat16 if bf16 else torch.float32

        def tensor(*shape, std=1.0, mean=0.0):
            a = (mean + std * rng.standard_normal(shape)).astype(np.float32)
            if bf16:
                b = synth.to_bf16_bits(a)
                return synth.bf16_bits_to_f32(b).reshape(shape).astype(np.float64), gc.dev_bf16(b).view(shape)
            return a.astype(np.float64), gc.dev_f32(a).view(shape)

        self.Y, self.dY = tensor(M, (nq + 2 * nk) * d, std=scale)
        self.pos = rng.integers(-far, far, M)
        self.dpos = torch.from_numpy(self.pos).cuda()
        self.f = (10000.0 ** -(np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)
        self.df = gc.dev_f32(self.f)
        self.w = [tensor(d, std=0.2, mean=1.0) for _ in range(2)] if norm else [(None, None)] * 2
        self.g = [tensor(M, n, d) for n in (nq, nk, nk)]

    def split(self, a):
        """q and k heads of rows."""
        r = a.reshape(self.M, self.nq + 2 * self.nk, self.d)
        return r[:, :self.nq], r[:, self.nq:self.nq + self.nk]

    def fwd(self, q, **kw):
        return q.qk_norm_rope_fwd(self.dY, self.dpos, self.df, self.nq, self.nk, self.w[0][1], self.w[1][1], eps=EPS,
                                  interleaved=self.inter, **kw)

    def bwd(self, q, **kw):
        return q.qk_norm_rope_bwd(self.g[0][1], self.g[1][1], self.g[2][1], self.dpos, self.df, self.dY, self.w[0][1],
                                  self.w[1][1], eps=EPS, interleaved=self.inter, **kw)

    def paired(self, a):
        """|a| + |its partner| of each element, that which a rotation's value is made of."""
        i, j = orot.pairs(self.rot, self.inter)
        m = np.abs(a).copy()
        m[..., i] = m[..., j] = np.abs(a[..., i]) + np.abs(a[..., j])
        return m

    def check_fwd(self, got):
        for x, (w, _), z in zip(self.split(self.Y), self.w, got):
            want = orot.forward(x, w, self.pos, self.f, EPS, self.inter)
            n = x if w is None else x * orot.inverse_rms(x, EPS) * w
            err = np.abs(z.float().cpu().numpy() - want)
            tol = self.h * np.abs(want) + 64 * U * self.paired(n)
            assert np.all(err <= tol), float(np.max(err / np.maximum(tol, 1e-300)))

    def check_bwd(self, got):
        import torch
        dY, dqw, dkw = got
        rows = dY.float().cpu().numpy().astype(np.float64)
        parts = self.split(rows)
        assert torch.equal(dY.view(self.M, -1, self.d)[:, self.nq + self.nk:], self.g[2][1])
        for x, (w, _), (dz, _), dx, dw in zip(self.split(self.Y), self.w, self.g, parts, (dqw, dkw)):
            want, want_w = orot.backward(dz, x, w, self.pos, self.f, EPS, self.inter)
            up = self.paired(dz)
            if w is None:
                tol = self.h * np.abs(want) + 64 * U * up
            else:
                r = orot.inverse_rms(x, EPS)
                g = up * np.abs(w)
                tol = self.h * np.abs(want) + 128 * U * r * (g + np.abs(x) * r * r * np.mean(g * np.abs(x), -1, keepdims=True))
                mag = np.sum(up * np.abs(x) * r, axis=(0, 1))
                err = np.abs(dw.float().cpu().numpy() - want_w)
                tol_w = self.h * np.abs(want_w) + (self.M * x.shape[1] + 128) * U * mag
                assert np.all(err <= tol_w), float(np.max(err / tol_w))
            err = np.abs(dx - want)
            assert np.all(err <= tol), float(np.max(err / np.maximum(tol, 1e-300)))
        if self.w[0][0] is None:
            assert dqw is None and dkw is None


def _both(q, *a, **kw):
    import torch
    c = Case(*a, **kw)
    got = c.fwd(q)
    torch.cuda.synchronize()
    c.check_fwd(got)
    got = c.bwd(q)
    torch.cuda.synchronize()
    c.check_bwd(got)
    return c


@pytest.mark.parametrize("d,rot", [(4, 4), (8, 8), (12, 4), (20, 20), (32, 32), (40, 16), (64, 64), (64, 16), (72, 72),
                                   (80, 32), (80, 20), (96, 96), (96, 48), (100, 36), (128, 128), (128, 64), (160, 160),
                                   (192, 64), (252, 252), (256, 256), (256, 64), (128, 0), (64, 4)])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
def test_heads(q, d, rot, norm, inter, bf16):
    _both(q, 5, 3, 2, d, rot, norm, inter, bf16)


@pytest.mark.parametrize("nq,nk", [(1, 1), (2, 1), (7, 1), (8, 8), (9, 3), (32, 8), (64, 64), (71, 1)])
@pytest.mark.parametrize("M", [1, 2, 37])
def test_head_counts(q, nq, nk, M):
    _both(q, M, nq, nk, 64, 64, True, False, True)


@pytest.mark.parametrize("M", [1, 3, 64, 333, 1000, 4097])
@pytest.mark.parametrize("bf16", [False, True])
def test_tokens(q, M, bf16):
    _both(q, M, 4, 2, 128, 128, True, False, bf16)


def test_more_tokens_than_workgroups_take_at_once(q):
    _both(q, 20011, 2, 1, 32, 32, True, True, True)


@pytest.mark.parametrize("far", [1, 131072, 1 << 24, 1 << 31])
def test_positions(q, far):
    """The angle of a far position, reduced in 64 bits, is as good as that of a near one."""
    _both(q, 50, 2, 2, 64, 64, False, False, False, far=far)


def test_large_small_and_zero_rows(q):
    """Rows of zeros (the root of eps alone), tiny and large rows."""
    import torch
    for scale in (0.0, 1e-12, 1e4):
        _both(q, 6, 3, 1, 64, 32, True, False, False, scale=scale)


def test_one_bad_row_stays_alone(q):
    import torch
    c = Case(6, 3, 2, 64, 64, True, False, True)
    want, back = c.fwd(q), c.bwd(q)
    c.dY[2, 10] = float("nan")      # query head 0 of token 2
    c.dY[4, 3 * 64 + 1] = float("inf")  # key head 0 of token 4
    Q, K = c.fwd(q)
    same = torch.ones(6, 3, dtype=torch.bool, device="cuda")
    same[2, 0] = False
    assert torch.equal(Q[same], want[0][same]) and bool(Q[2, 0].isnan().all())
    same = torch.ones(6, 2, dtype=torch.bool, device="cuda")
    same[4, 0] = False
    assert torch.equal(K[same], want[1][same])
    dY = c.bwd(q)[0].view(6, -1, 64)
    ref = back[0].view(6, -1, 64)
    hit = torch.zeros(6, 7, dtype=torch.bool, device="cuda")
    hit[2, 0] = hit[4, 3] = True
    assert torch.equal(dY[~hit], ref[~hit])


def test_outputs_given_workspace_of_any_content_and_guards(q):
    import torch
    c = Case(11, 5, 2, 80, 32, True, True, True)
    Q0, K0 = c.fwd(q)
    back = c.bwd(q)
    n = c.dY.numel()

    def guarded(shape):
        k = int(np.prod(shape))
        buf = torch.full((k + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
        return buf, buf[32:32 + k].view(shape)

    bq, Q = guarded(Q0.shape)
    bk, K = guarded(K0.shape)
    got = c.fwd(q, Q=Q, K=K)
    assert got[0] is Q and got[1] is K and torch.equal(Q, Q0) and torch.equal(K, K0)
    by, dY = guarded((11, n // 11))
    bw, dqw = guarded((80,))
    bv, dkw = guarded((80,))
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")
    ws[:65792].zero_()
    got = c.bwd(q, dY=dY, dqw=dqw, dkw=dkw, ws=ws)
    for a, b in zip(got, back):
        assert torch.equal(a, b)
    assert not bool(ws[:65792].any())
    for buf in (bq, bk, by, bw, bv):
        assert bool((buf[:32] == 7).all()) and bool((buf[-32:] == 7).all())


def test_no_tokens(q):
    import torch
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    pos, f, w = torch.empty(0, dtype=torch.int64, device="cuda"), torch.ones(16, device="cuda"), torch.ones(
        32, dtype=torch.bfloat16, device="cuda")
    Q, K = q.qk_norm_rope_fwd(e(0, 8 * 32), pos, f, 4, 2, w, w)
    assert Q.shape == (0, 4, 32) and K.shape == (0, 2, 32)
    dY, dqw, dkw = q.qk_norm_rope_bwd(e(0, 4, 32), e(0, 2, 32), e(0, 2, 32), pos, f, e(0, 256), w, w)
    assert dY.shape == (0, 256) and not bool(dqw.any()) and not bool(dkw.any())
    assert q.qk_norm_rope_bwd(e(0, 4, 32), e(0, 2, 32), e(0, 2, 32), pos, f)[1:] == (None, None)


def test_rows_past_four_gib(q):
    """The last tokens of rows that pass element 2^31 and byte 2^32, both directions."""
    import torch
    nq, nk, d = 64, 64, 128
    N = (nq + 2 * nk) * d
    M = (1 << 32) // (2 * N) + 60
    gen = torch.Generator(device="cuda").manual_seed(1)
    Y = torch.randn((M, N), device="cuda", generator=gen, dtype=torch.bfloat16)
    pos = torch.arange(M, device="cuda")
    f = torch.rand(d // 2, device="cuda", generator=gen)
    w = torch.rand(d, device="cuda", generator=gen).bfloat16()
    Q, K = q.qk_norm_rope_fwd(Y, pos, f, nq, nk, w, w)
    t = slice(M - 50, M)
    Qt, Kt = q.qk_norm_rope_fwd(Y[t], pos[t], f, nq, nk, w, w)
    assert torch.equal(Q[t], Qt) and torch.equal(K[t], Kt)
    dY, _, _ = q.qk_norm_rope_bwd(Q, K, K, pos, f, Y, w, w)
    dYt, _, _ = q.qk_norm_rope_bwd(Qt, Kt, Kt, pos[t], f, Y[t], w, w)
    assert torch.equal(dY[t], dYt)


def test_repeatable_streams_and_captured_graphs(q):
    """Gradients of the weights are summed in a fixed order; two streams with a workspace each;
    one captured graph of both directions replayed on new rows between eager calls."""
    import torch
    c = Case(300, 4, 2, 128, 128, True, False, True)
    other = torch.randn_like(c.dY)
    rows = [c.dY.clone(), other]
    want = []
    for r in rows:
        c.dY = r
        want.append((*c.fwd(q), *c.bwd(q)))
    torch.cuda.synchronize()
    for r, w in zip(rows, want):
        c.dY = r
        for a, b in zip((*c.fwd(q), *c.bwd(q)), w):
            assert torch.equal(a, b)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for k in range(6):
        with torch.cuda.stream(streams[k % 2]):
            c.dY = rows[k % 2]
            got.append((k % 2, (*c.fwd(q), *c.bwd(q))))
    torch.cuda.synchronize()
    for k, g in got:
        for a, b in zip(g, want[k]):
            assert torch.equal(a, b)
    static = rows[0].clone()
    c.dY = static
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    out = [torch.empty_like(t) for t in want[0]]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.fwd(q, Q=out[0], K=out[1])
        c.bwd(q, dY=out[2], dqw=out[3], dkw=out[4], ws=ws)
    for k in range(4):
        static.copy_(rows[k % 2])
        g.replay()
        c.dY = rows[k % 2]
        eager = (*c.fwd(q), *c.bwd(q))
        torch.cuda.synchronize()
        for a, b, e in zip(out, want[k % 2], eager):
            assert torch.equal(a, b) and torch.equal(e, b)
        c.dY = static


def test_projection_norm_rotation_and_back(q):
    """Fused NF4 q/k/v projection, norms and rotation, and the gradients back into the
    adapters: each operator on the one before's output, the last against float64."""
    import torch
    M, H, d, K, r = 24, 4, 64, 256, 8
    gen = torch.Generator(device="cuda").manual_seed(0)
    n = lambda *s, std=1.0: (torch.randn(s, device="cuda", generator=gen) * std).bfloat16()  # noqa: E731
    qw = q.quantize(n(3 * H * d, K, std=0.05))
    X, A, B = n(M, K), n(3 * r, K, std=0.2), n(3 * H * d, r, std=0.05)
    Y, Us = q.linear_fwd_fused(qw, 3, X, A, B, 16.0)
    pos = torch.arange(M, device="cuda")
    f = (10000.0 ** (-torch.arange(0, d, 2, device="cuda") / d)).float()
    wq, wk = n(d, std=0.1) + 1, n(d, std=0.1) + 1
    Q, Kh = q.qk_norm_rope_fwd(Y, pos, f, H, H, wq, wk, eps=EPS)
    dQ, dK, dV = n(M, H, d), n(M, H, d), n(M, H, d)
    dY, dqw, dkw = q.qk_norm_rope_bwd(dQ, dK, dV, pos, f, Y, wq, wk, eps=EPS)
    dX, dA, dB = q.linear_bwd_fused(qw, 3, dY, X, A, B, 16.0, Us)
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    p, fr, y = pos.cpu().numpy(), f.cpu().numpy(), f64(Y).reshape(M, 3 * H, d)
    back = []
    for k, (w, z, dz) in enumerate(((wq, Q, dQ), (wk, Kh, dK))):
        x = y[:, k * H:(k + 1) * H]
        want = orot.forward(x, f64(w), p, fr, EPS, False)
        assert np.max(np.abs(f64(z) - want)) <= 2.0 ** -8 * np.max(np.abs(want)) + 1e-5
        back.append(orot.backward(f64(dz), x, f64(w), p, fr, EPS, False)[0])
    back = np.concatenate([*back, f64(dV)], axis=1).reshape(M, -1)
    W = f64(q.dequantize(qw))
    P = H * d
    dYr, Br, Xr, Ar = f64(dY), f64(B), f64(X), f64(A)
    assert np.max(np.abs(dYr - back)) <= 2.0 ** -8 * np.max(np.abs(back)) + 1e-4
    V = np.concatenate([2.0 * dYr[:, k * P:(k + 1) * P] @ Br[k * P:(k + 1) * P] for k in range(3)], axis=1)
    for got, want in ((dX, dYr @ W + V @ Ar), (dA, V.T @ Xr)):
        assert np.max(np.abs(f64(got) - want)) <= 2e-2 * np.max(np.abs(want))


def test_serving_run(q):
    """One decode step of a served layer: group-scaled projection, then norms and rotation."""
    import torch
    M, nq, nk, d, K = 3, 8, 2, 64, 256
    N = (nq + 2 * nk) * d
    gw = q.group_quantize(torch.randn(N, K, device="cuda") * 0.05, 64, zeros=True)
    X = torch.randn(M, K, device="cuda").bfloat16()
    pos = torch.tensor([5, 100000, 0], device="cuda")
    f = (500000.0 ** (-torch.arange(0, d, 2, device="cuda") / d)).float()
    w = (torch.rand(d, device="cuda") + 0.5).bfloat16()
    Y = q.group_linear_fwd(gw, X)
    Q, Kh = q.qk_norm_rope_fwd(Y, pos, f, nq, nk, w, w, eps=EPS)
    want = X.double().cpu() @ q.group_dequantize(gw, torch.float32).double().cpu().t()
    assert float((Y.double().cpu() - want).abs().max()) <= 2.0 ** -8 * float(want.abs().max()) + 1e-4
    y = Y.double().cpu().numpy().reshape(M, -1, d)
    for x, z in ((y[:, :nq], Q), (y[:, nq:nq + nk], Kh)):
        ref = orot.forward(x, w.double().cpu().numpy(), pos.cpu().numpy(), f.cpu().numpy(), EPS, False)
        assert np.max(np.abs(z.double().cpu().numpy() - ref)) <= 2.0 ** -8 * np.max(np.abs(ref)) + 1e-5
