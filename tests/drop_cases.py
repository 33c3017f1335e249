"""Inputs and derived error bounds shared by the tests of the operators with dropout and of
the gated projections.  The bounds count, element by element, what the operators' documented
roundings allow:

* a bf16 result is off by at most half a step, 2^-8 of its value (``H``), and so is each bf16
  intermediate (U, V, the gradient of [G | L]), whose error then passes through the products;
* an fp32 sum of n products is off by at most n 2^-24 of the sum of magnitudes; ``S`` doubles
  that for the matrix unit's internal additions, and the callers add a few terms for the
  scalings.
"""

import numpy as np

import synth
from oracle import dropout as od
from oracle import nf4
from tests import gpu_cases as gc

H = 2.0 ** -8
S = 2.0 ** -23


def check(name, got, want, tol):
    got = np.asarray(got, np.float64)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert np.all(np.isfinite(got)), f"{name}: not finite"
    # 2^-133 is the spacing of the smallest bf16 values
    over = np.abs(got - want) - (tol + 2.0 ** -133)
    i = np.unravel_index(np.argmax(over), over.shape)
    print(f"  {name}: worst error {np.max(np.abs(got - want)):.3e}, largest share of its bound "
          f"{np.max(np.abs(got - want) / (tol + 2.0 ** -133)):.3f}", flush=True)
    assert over[i] <= 0, f"{name}{list(i)}: {got[i]} vs {want[i]}, bound {tol[i]}"


def bits(t):
    return gc.host_f32_from_bf16(t)


def linear_inputs(M, K, Np, r, parts, seed):
    """Device inputs and their float64 values: quantized stacked weight, X, A, B, dY."""
    d = synth.case(M, K, Np * parts, r, seed=seed, b_std=0.1)
    g = np.random.default_rng(seed + 1)
    A = synth.to_bf16_bits((g.standard_normal((parts * r, K)) / 8).astype(np.float32))
    return {"W": d["W"], "X": d["X"], "A": A, "B": d["B"], "dY": d["dY"]}


def f64(d, *names):
    return tuple(gc.f64(d[n]) for n in names)


def weight64(qw):
    """W' of a quantized weight on the device, from its stored arrays, through the oracle."""
    arr = lambda t: t.cpu().numpy()  # noqa: E731
    stored = {"shape": qw.shape, "codes": arr(qw.codes), "absmax_q": arr(qw.absmax_q),
              "dq_scale": arr(qw.dq_scale), "dq_offset": arr(qw.dq_offset)}
    return nf4.dequantize_bf16(stored).astype(np.float64)


def down(X, A, alpha, r, m, c):
    """U and its bound."""
    k = c * alpha / r
    U = k * ((m * X) @ A.T)
    return U, H * np.abs(U) + (X.shape[1] + 8) * S * abs(k) * (np.abs(m * X) @ np.abs(A).T)


def forward(X, Wd, A, B, alpha, r, parts, m, c):
    """(Y, its bound before the final rounding, U, its bound)."""
    M, K = X.shape
    N = Wd.shape[0]
    Y, mag = X @ Wd.T, np.abs(X) @ np.abs(Wd).T
    if r == 0:
        return Y, (K + 8) * S * mag, None, None
    U, eU = down(X, A, alpha, r, m, c)
    e = np.zeros_like(Y)
    n = N // parts
    for q in range(parts):
        o, k = slice(q * n, (q + 1) * n), slice(q * r, (q + 1) * r)
        Y[:, o] += U[:, k] @ B[o].T
        mag[:, o] += np.abs(U[:, k]) @ np.abs(B[o]).T
        e[:, o] = eU[:, k] @ np.abs(B[o]).T
    return Y, e + (K + r + 8) * S * mag, U, eU


def backward(dY, edY, X, Wd, A, B, alpha, r, parts, m, c, U):
    """{name: (value, bound)} of dX, dA, dB for dY known up to edY and the saved U."""
    M, K = X.shape
    N = Wd.shape[0]
    dX = dY @ Wd
    eX = edY @ np.abs(Wd) + (N + r + 8) * S * (np.abs(dY) @ np.abs(Wd))
    if r == 0:
        return {"dX": (dX, eX + H * (np.abs(dX) + eX))}
    n, k = N // parts, c * alpha / r
    V, eV = np.empty((M, parts * r)), np.empty((M, parts * r))
    dB, eB = np.empty((N, r)), np.empty((N, r))
    for q in range(parts):
        o, j = slice(q * n, (q + 1) * n), slice(q * r, (q + 1) * r)
        V[:, j] = k * (dY[:, o] @ B[o])
        eV[:, j] = abs(k) * (edY[:, o] @ np.abs(B[o]) + (n + 8) * S * (np.abs(dY[:, o]) @ np.abs(B[o])))
        dB[o] = dY[:, o].T @ U[:, j]
        eB[o] = edY[:, o].T @ np.abs(U[:, j]) + (M + 8) * S * (np.abs(dY[:, o]).T @ np.abs(U[:, j]))
    # dA multiplies V and what its rounding took off, itself rounded: 2^-8 of 2^-8
    eV2 = eV + H * H * (np.abs(V) + eV)
    eV = eV + H * (np.abs(V) + eV)
    low = m * (V @ A)
    dX = dX + low
    eX = eX + m * (eV @ np.abs(A) + (N + r + 8) * S * (np.abs(V) @ np.abs(A)))
    mX = m * X
    dA = V.T @ mX
    eA = eV2.T @ np.abs(mX) + 2 * (M + 8) * S * (np.abs(V).T @ np.abs(mX))
    fin = lambda v, e: (v, e + H * (np.abs(v) + e))  # noqa: E731
    return {"dX": fin(dX, eX), "dA": fin(dA, eA), "dB": fin(dB, eB)}


def mask(M, K, p, seed, offset):
    if p == 0.0:
        return np.ones((M, K)), 1.0
    return od.keep((M, K), p, seed, offset).astype(np.float64), od.scale(p)
