"""Infinities and NaN where they have to stay apart: what is dropped for the adapter, what lies
past a lane's own blocks, the other projection's ranks.  A zero that a kernel puts in by
itself must never meet an infinity (their product is NaN, where the definition has none)."""

import numpy as np
import pytest

from tests import drop_cases as dc
from tests import gpu_cases as gc

pytestmark = pytest.mark.gpu
ALPHA = 16.0


@pytest.fixture(scope="module")
def q():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_lora_nf4_amd as lib
    return lib


def same_kind(got, want):
    """Infinities of the same sign and NaN in the same places, finite elsewhere."""
    for f in (np.isposinf, np.isneginf, np.isnan):
        bad = np.argwhere(f(got) != f(want))
        assert bad.size == 0, (f.__name__, bad[:4].tolist(), got[tuple(bad[0])], want[tuple(bad[0])])


@pytest.mark.parametrize("M", [1, 5, 16, 40])
@pytest.mark.parametrize("K", [64, 192, 256, 1024])
def test_dropped_nan_in_any_block_stays_out_of_u(q, M, K):
    """Row i has NaN at a dropped element of block i (rows past the last block again from the
    first): the adapter does not see it, whichever lane holds the block."""
    import torch
    N, r = 64, 8
    h = dc.linear_inputs(M, K, N, r, 1, seed=3)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"])
    d = q.Dropout(0.5, seed=21)
    m, _ = dc.mask(M, K, 0.5, 21, 0)
    X = dev["X"].clone()
    for i in range(M):
        b = 64 * (i % (K // 64))
        X[i, b + int(np.flatnonzero(m[i, b:b + 64] == 0)[0])] = float("nan")
    _, U = q.linear_fwd(qw, dev["X"], dev["A"], dev["B"], ALPHA, dropout=d)
    _, U2 = q.linear_fwd(qw, X, dev["A"], dev["B"], ALPHA, dropout=d)
    assert torch.equal(U, U2)


@pytest.mark.parametrize("dropout", [False, True])
@pytest.mark.parametrize("K", [64, 192, 256, 1024])
def test_infinite_input_of_the_adapter(q, K, dropout):
    """One infinite (kept) element in block i of row i: U is infinite with the sign that the
    definition gives, for one token to 16 and for tiles."""
    N, r, M = 64, 8, 16
    h = dc.linear_inputs(40, K, N, r, 1, seed=5)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"])
    d = q.Dropout(0.5, seed=22) if dropout else None
    m = dc.mask(40, K, 0.5, 22, 0)[0] if dropout else np.ones((40, K))
    X, col = dev["X"].clone(), []
    for i in range(40):
        b = 64 * (i % (K // 64))
        col.append(b + int(np.flatnonzero(m[i, b:b + 64])[3]))
        X[i, col[-1]] = float("inf")
    want = np.inf * gc.f64(h["A"])[:, col].T
    for rows in (1, 3, M, 40):
        _, U = q.linear_fwd(qw, X[:rows].contiguous(), dev["A"], dev["B"], ALPHA, dropout=d)
        same_kind(dc.bits(U), want[:rows])


@pytest.mark.parametrize("M", [1, 7, 16, 40, 300])
@pytest.mark.parametrize("K", [64, 192, 256, 320, 448, 1088])
def test_infinite_input_in_any_block(q, M, K):
    """Row i has an infinity in its block i (rows past the last block again from the first),
    dropped for the adapter: the base product is infinite, or NaN where the weight is zero,
    whichever lane or step holds the block."""
    N, r = 256, 8
    h = dc.linear_inputs(M, K, N, r, 1, seed=6)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"])
    Wd = dc.weight64(qw)
    d = q.Dropout(0.5, seed=23)
    m, _ = dc.mask(M, K, 0.5, 23, 0)
    X, col = dev["X"].clone(), []
    for i in range(M):
        b = 64 * (i % (K // 64))
        col.append(b + int(np.flatnonzero(m[i, b:b + 64] == 0)[1]))
        X[i, col[-1]] = float("inf") if i % 2 else float("-inf")
    sign = np.where(np.arange(M) % 2, np.inf, -np.inf)
    with np.errstate(invalid="ignore"):
        want = sign[:, None] * Wd[:, col].T
    if m[0].any():
        Y, _ = q.linear_fwd(qw, X, dev["A"], dev["B"], ALPHA, dropout=d)
        same_kind(dc.bits(Y), want)
    Y, _ = q.linear_fwd(qw, X)
    same_kind(dc.bits(Y), want)
    _, Y, _ = q.gated_fwd(qw, X)
    same_kind(dc.bits(Y), want)


@pytest.mark.parametrize("M,K,P,r", [
    (1, 256, 72, 8), (3, 256, 71, 12), (16, 512, 264, 64), (16, 8192, 136, 8),  # one launch
    (40, 256, 72, 8), (40, 448, 65, 40), (130, 256, 136, 72), (70, 512, 136, 128), (777, 512, 3000, 16),
    (18, 64, 2200, 8), (300, 64, 4097, 20), (700, 64, 5637, 72),
])
@pytest.mark.parametrize("part", [0, 1])
def test_non_finite_ranks_stay_in_their_projection(q, M, K, P, r, part):
    """Infinite and NaN ranks of one projection's adapter leave the other projection alone."""
    import torch
    h = dc.linear_inputs(M, K, P, r, 2, seed=7)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"])
    _, Y, U = q.gated_fwd(qw, dev["X"], dev["A"], dev["B"], ALPHA)
    A = dev["A"].clone()
    A[part * r, K // 2] = float("inf")
    A[part * r + r - 1, 0] = float("nan")
    _, Y2, U2 = q.gated_fwd(qw, dev["X"], A, dev["B"], ALPHA)
    own, other = slice(part * P, (part + 1) * P), slice((1 - part) * P, (2 - part) * P)
    assert torch.equal(U2[:, (1 - part) * r:(2 - part) * r], U[:, (1 - part) * r:(2 - part) * r])
    assert not bool(torch.isfinite(Y2[:, own]).any())
    assert torch.equal(Y2[:, other], Y[:, other])


@pytest.mark.parametrize("M", [20, 300])
def test_infinite_v_gives_infinite_da(q, M):
    """V = (alpha / r) dY B past the largest bf16 value: dA's rows are infinite with the signs of
    the definition (what V's rounding took off is not a number there and must not be added)."""
    import torch
    K, P, r = 128, 64, 8
    h = dc.linear_inputs(M, K, P, r, 2, seed=8)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"])
    g = np.random.default_rng(1)
    sign = g.choice([-1.0, 1.0], r)
    i, c = M // 2, 5
    Y = torch.zeros(M, 2 * P, dtype=torch.bfloat16, device="cuda")
    Y[:, :P] = 1.0  # act(1) = 0.73
    dH = torch.zeros(M, P, dtype=torch.bfloat16, device="cuda")
    dH[i, c] = 1e37
    B = dev["B"].clone()
    B[P + c] = torch.tensor(sign * 1e3, device="cuda").bfloat16()
    X = dev["X"].clone()
    X[X == 0] = 1.0
    U = torch.zeros(M, 2 * r, dtype=torch.bfloat16, device="cuda")
    _, dA, _ = q.gated_bwd(qw, dH, Y, X, dev["A"], B, ALPHA, U)
    want = np.zeros((2 * r, K))
    want[r:] = sign[:, None] * np.inf * dc.bits(X)[i][None, :]
    same_kind(dc.bits(dA), want)
    assert np.all(dc.bits(dA)[:r] == 0.0)


def ieee(a, b):
    """a b with every product and sum of the contraction carried out (a library's may not)."""
    out = a @ b
    for i in np.flatnonzero(~np.isfinite(a).all(1)):
        out[i] = (a[i][:, None] * b).sum(0)
    return out


@pytest.mark.parametrize("r", [1, 4, 8, 12, 20])
@pytest.mark.parametrize("M,K,N", [(7, 256, 64), (40, 192, 130), (300, 64, 4100), (700, 320, 72)])
def test_infinities_with_ranks_of_any_size(q, M, K, N, r):
    """An infinity in X (kept) and one in dY: U, Y, V's part of dX, dA and dB are infinite, NaN and
    finite where the definition is, also where the rank is padded to a multiple of 8."""
    h = dc.linear_inputs(M, K, N, r, 1, seed=9)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"])
    Wd = dc.weight64(qw)
    d = q.Dropout(0.5, seed=24)
    m, c = dc.mask(M, K, 0.5, 24, 0)
    A, B = dc.f64(h, "A", "B")
    X, dY = dev["X"].clone(), dev["dY"].clone()
    i, j = M // 2, M - 1
    X[i, int(np.flatnonzero(m[i])[-1])] = float("inf")
    dY[j, N // 3] = float("-inf")
    Xf, dYf = dc.bits(X), dc.bits(dY)
    with np.errstate(invalid="ignore"):
        Y, U = q.linear_fwd(qw, X, dev["A"], dev["B"], ALPHA, dropout=d)
        Uf = dc.bits(U)
        same_kind(Uf, ieee(np.where(m != 0, Xf, 0.0), A.T))
        same_kind(dc.bits(Y), ieee(Xf, Wd.T) + ieee(Uf, B.T))
        U = dev["X"][:, :r].contiguous()  # any finite U
        dX, dA, dB = q.linear_bwd(qw, dY, dev["X"], dev["A"], dev["B"], ALPHA, U, dropout=d)
        V = ieee(dYf, B)
        same_kind(dc.bits(dX), ieee(dYf, Wd) + np.where(m != 0, ieee(V, A), 0.0))
        same_kind(dc.bits(dA), ieee(V.T, np.where(m != 0, dc.bits(dev["X"]), 0.0)))
        same_kind(dc.bits(dB), ieee(dYf.T, dc.bits(U)))
