"""Grouped heads (fewer key heads than query heads) in training without a copy: one QLoRA linear over the
stacked query, key and value rows writes the rows that the norms with rotation read, and its
backward reads the rows that theirs writes.

Bounds.  h = 2^-8 is half a step of bf16 relative to the value; n u, u = 2^-24, are the roundings of fp32
sums of n terms, counted twice.  The base product and the adapter's are of exact bf16 products;
V (the backward's down-projection) is rounded to bf16 before it is multiplied on."""

import numpy as np
import pytest

from oracle import rotation as orot

pytestmark = pytest.mark.gpu
H, U, EPS = 2.0 ** -8, 2.0 ** -24, 1e-6


@pytest.mark.parametrize("M,nq,nk,d,rot,inter", [(24, 4, 2, 64, 64, False), (67, 6, 1, 32, 16, True), (300, 8, 2, 128, 128, False)])
def test_stacked_projection_norm_rotation_and_back(M, nq, nk, d, rot, inter):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_lora_nf4_amd as q
    K, r, alpha = 256, 8, 16.0
    N = (nq + 2 * nk) * d
    gen = torch.Generator(device="cuda").manual_seed(M)
    n = lambda *s, std=1.0: (torch.randn(s, device="cuda", generator=gen) * std).bfloat16()  # noqa: E731
    qw = q.quantize(n(N, K, std=0.05))
    X, A, B = n(M, K), n(r, K, std=0.2), n(N, r, std=0.05)
    Y, Us = q.linear_fwd(qw, X, A, B, alpha)
    pos = torch.arange(M, device="cuda") * 7
    f = (10000.0 ** (-torch.arange(0, rot, 2, device="cuda") / rot)).float()
    wq, wk = n(d, std=0.1) + 1, n(d, std=0.1) + 1
    Q, Kh = q.qk_norm_rope_fwd(Y, pos, f, nq, nk, wq, wk, eps=EPS, interleaved=inter)
    dQ, dK, dV = n(M, nq, d), n(M, nk, d), n(M, nk, d)
    dY, dqw, dkw = q.qk_norm_rope_bwd(dQ, dK, dV, pos, f, Y, wq, wk, eps=EPS, interleaved=inter)
    dX, dA, dB = q.linear_bwd(qw, dY, X, A, B, alpha, Us)
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    p, fr, y = pos.cpu().numpy(), f.cpu().numpy(), f64(Y).reshape(M, -1, d)
    got = f64(dY).reshape(M, -1, d)
    for first, last, w, z, dz, dw in ((0, nq, wq, Q, dQ, dqw), (nq, nq + nk, wk, Kh, dK, dkw)):
        x = y[:, first:last]
        want = orot.forward(x, f64(w), p, fr, EPS, inter)
        head = np.abs(want).max(-1, keepdims=True)    # (a pair's magnitudes are at most twice it)
        assert np.all(np.abs(f64(z) - want) <= H * np.abs(want) + 256 * U * head)
        want, want_w = orot.backward(f64(dz), x, f64(w), p, fr, EPS, inter)
        size = orot.inverse_rms(x, EPS) * 2 * np.abs(f64(dz)).max(-1, keepdims=True) * np.abs(f64(w)).max()
        far = 1 + np.abs(x).max(-1, keepdims=True) * orot.inverse_rms(x, EPS)
        assert np.all(np.abs(got[:, first:last] - want) <= H * np.abs(want) + 128 * U * size * far ** 2)
        terms = M * (last - first) * 2 * np.abs(f64(dz)).max() * far.max()
        assert np.all(np.abs(f64(dw) - want_w) <= H * np.abs(want_w) + 128 * U * terms)
    assert torch.equal(dY.view(M, -1, d)[:, nq + nk:], dV)
    W, g, a, b, xs, us = f64(q.dequantize(qw)), f64(dY), f64(A), f64(B), f64(X), f64(Us)
    V = (alpha / r) * (g @ b)
    Vsum = (alpha / r) * (np.abs(g) @ np.abs(b))
    Vtol = H * np.abs(V) + 2 * N * U * Vsum
    for name, got, want, tol in (
            ("dX", dX, g @ W + V @ a, Vtol @ np.abs(a) + 2 * (N + r) * U * (np.abs(g) @ np.abs(W) + Vsum @ np.abs(a))),
            ("dA", dA, V.T @ xs, Vtol.T @ np.abs(xs) + 2 * M * U * (Vsum.T @ np.abs(xs))),
            ("dB", dB, g.T @ us, 2 * M * U * (np.abs(g).T @ np.abs(us)))):
        err = np.abs(f64(got) - want)
        tol = tol + H * (np.abs(want) + tol)
        assert np.all(err <= tol), (name, float(np.max(err / tol)))
