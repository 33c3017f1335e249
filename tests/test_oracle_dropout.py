"""The dropout oracle: known answers of the generator, the mask's rate and scale, and the
gradients against differences.  Also the binding's and the C ABI's refusals (no GPU)."""

import numpy as np
import pytest
import torch

import bit_quantized_lora_nf4_amd as q
from bit_quantized_lora_nf4_amd import _lib
from oracle import dropout as od

FAKE = 0x10000  # 16-byte aligned, never dereferenced (validation fails first)
F = 0xFFFFFFFF


# the generator's published known answers (counter, key, rounds -> block)
@pytest.mark.parametrize("c,k,rounds,want", [
    (0, 0, 7, (0x5F6FB709, 0x0D893F64, 0x4F121F81, 0x4F730A48)),
    (F, F, 7, (0x5207DDC2, 0x45165E59, 0x4D8EE751, 0x8C52F662)),
    (0, 0, 10, (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    (F, F, 10, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
])
def test_philox_known_answers(c, k, rounds, want):
    got = od.philox4x32([np.array([c])] * 4, (k, k), rounds)
    assert tuple(int(x[0]) for x in got) == want


@pytest.mark.parametrize("p", [0.05, 0.1, 0.5, 0.9])
def test_keep_rate(p):
    n = 1 << 20
    t = od.threshold(p)
    m = od.keep((n,), p, seed=12345678901234567, offset=3)
    # the count of a binomial of n draws is within 6 standard deviations
    q1 = 1 - t / 65536
    assert abs(m.sum() - n * q1) <= 6 * np.sqrt(n * q1 * (1 - q1))
    assert od.scale(p) * q1 == pytest.approx(1.0, abs=1e-15)


def test_keep_is_a_function_of_the_index():
    whole = od.keep((1000,), 0.3, 7, 9)
    assert np.array_equal(whole[13:500], od.keep((487,), 0.3, 7, 9, first=13))
    assert not np.array_equal(whole, od.keep((1000,), 0.3, 7, 10))
    assert not np.array_equal(whole, od.keep((1000,), 0.3, 8, 9))
    # groups past 32 bits use the counter's second word
    far = od.keep((64,), 0.5, 7, 9, first=8 << 32)
    assert not np.array_equal(far, od.keep((64,), 0.5, 7, 9))


def test_gradients_against_differences():
    rng = np.random.default_rng(0)
    M, K, N, r, alpha = 3, 16, 5, 2, 4.0
    X, W, A, B, dY = (rng.standard_normal(s) for s in ((M, K), (N, K), (r, K), (N, r), (M, N)))
    m, c = od.keep((M, K), 0.4, 5, 6), od.scale(0.4)
    f = lambda X, A, B: np.sum(dY * od.forward(X, W, A, B, alpha, r, m, c)[0])  # noqa: E731
    _, U = od.forward(X, W, A, B, alpha, r, m, c)
    dX, dA, dB, _ = od.backward(dY, X, W, A, B, alpha, r, m, c, U)
    h = 1e-6  # f is a polynomial of degree at most 2 in each: the central difference is exact to rounding
    for T, dT, g in ((X, dX, lambda T: f(T, A, B)), (A, dA, lambda T: f(X, T, B)), (B, dB, lambda T: f(X, A, T))):
        for i in np.ndindex(T.shape):
            up, dn = T.copy(), T.copy()
            up[i] += h
            dn[i] -= h
            assert (g(up) - g(dn)) / (2 * h) == pytest.approx(dT[i], rel=1e-6, abs=1e-6)


# ---- refusals ------------------------------------------------------------------------

N, K, M, R = 256, 128, 8, 4


def _qw():
    return q.NF4Weight(torch.zeros(N * K // 2, dtype=torch.uint8), torch.zeros(N * K // 64, dtype=torch.int8),
                       torch.zeros(2, dtype=torch.float32), torch.zeros(2, dtype=torch.float32), N, K)


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_binding_rejects():
    with pytest.raises(TypeError, match="CUDA"):
        q.linear_fwd(_qw(), bf(M, K), bf(R, K), bf(N, R), dropout=q.Dropout(0.1))
    with pytest.raises(ValueError):
        q.linear_fwd(_qw(), bf(M, K + 64), bf(R, K), bf(N, R), dropout=q.Dropout(0.1))
    for p in (-0.1, 1.0, 1.5, float("nan")):
        with pytest.raises(ValueError, match="probability"):
            q.linear_fwd(_qw(), bf(M, K), bf(R, K), bf(N, R), dropout=q.Dropout(p))
        with pytest.raises(ValueError, match="probability"):
            q.linear_bwd(_qw(), bf(M, N), bf(M, K), bf(R, K), bf(N, R), dropout=q.Dropout(p))
    for kw in (dict(seed=-1), dict(seed=1 << 64), dict(offset=-5)):
        with pytest.raises(ValueError, match="64-bit"):
            q.linear_fwd(_qw(), bf(M, K), bf(R, K), bf(N, R), dropout=q.Dropout(0.1, **kw))
    with pytest.raises(TypeError):  # a counter must be int64
        q.linear_fwd(_qw(), bf(M, K), bf(R, K), bf(N, R), dropout=q.Dropout(0.1, counter=torch.zeros(1)))
    with pytest.raises(TypeError):
        q.dropout(torch.zeros(8, dtype=torch.float16), q.Dropout(0.1))
    with pytest.raises(ValueError):
        q.dropout(bf(8, 8).t()[1:], q.Dropout(0.1))
    with pytest.raises(ValueError):
        q.linear_fwd(_qw(), bf(M, K), bf(R, K), bf(N, R), ws=torch.zeros(16, dtype=torch.uint8),
                     dropout=q.Dropout(0.1))


def test_abi_rejects():
    w = _lib.qlora_nf4_weight(FAKE, FAKE, FAKE, FAKE, N, K)
    d = lambda p=0.1, counter=None: _lib.qlora_drop(p, 1, 2, counter)  # noqa: E731
    fwd = lambda drop, r=R, parts=1, ws=FAKE, X=FAKE, n=1 << 40: _lib.qlora_linear_fwd_dropout(  # noqa: E731
        w, parts, X, M, FAKE, FAKE, r, 16.0, drop, FAKE, None, ws, n, None)
    for p in (-0.5, 1.0, float("nan"), float("inf"), 1 - 2.0 ** -18):
        assert fwd(d(p)) == _lib.QLORA_ERR_VALUE, p
    assert fwd(d(counter=FAKE + 4)) == _lib.QLORA_ERR_ALIGN
    assert fwd(d(), X=None) == _lib.QLORA_ERR_NULL
    assert fwd(d(), X=FAKE + 2) == _lib.QLORA_ERR_ALIGN
    assert fwd(d(), r=257) == _lib.QLORA_ERR_RANK
    assert fwd(d(), parts=2) == _lib.QLORA_ERR_SHAPE          # parts of 128 rows
    assert fwd(d(), ws=None) == _lib.QLORA_ERR_WORKSPACE
    assert fwd(d(), n=100) == _lib.QLORA_ERR_WORKSPACE
    # three parts of rank 85 stack to 255 ranks, but to 264 when each is padded to 88
    w3 = _lib.qlora_nf4_weight(FAKE, FAKE, FAKE, FAKE, 768, K)
    assert _lib.qlora_linear_fwd_dropout(w3, 3, FAKE, M, FAKE, FAKE, 85, 16.0, d(), FAKE, None, FAKE, 1 << 40,
                                         None) == _lib.QLORA_ERR_RANK
    bwd = lambda drop, dA=FAKE, n=1 << 40, M=M: _lib.qlora_linear_bwd_dropout(  # noqa: E731
        w, 1, FAKE, FAKE, M, FAKE, FAKE, R, 16.0, drop, None, FAKE, dA, FAKE, FAKE, n, None)
    assert bwd(d(2.0)) == _lib.QLORA_ERR_VALUE
    assert bwd(d(), dA=None) == _lib.QLORA_ERR_NULL
    assert bwd(d(), n=64) == _lib.QLORA_ERR_WORKSPACE
    assert bwd(d(), M=1 << 26) in (_lib.QLORA_ERR_SHAPE, _lib.QLORA_ERR_WORKSPACE)
    e = _lib.qlora_dropout
    assert e(None, 1, 8, d(), FAKE, None) == _lib.QLORA_ERR_NULL
    assert e(FAKE, 1, 8, None, FAKE, None) == _lib.QLORA_ERR_NULL
    assert e(FAKE, 3, 8, d(), FAKE, None) == _lib.QLORA_ERR_DTYPE
    assert e(FAKE, 1, 0, d(), FAKE, None) == _lib.QLORA_ERR_SHAPE
    assert e(FAKE + 8, 1, 8, d(), FAKE, None) == _lib.QLORA_ERR_ALIGN
    assert e(FAKE, 1, 8, d(1.0), FAKE, None) == _lib.QLORA_ERR_VALUE


def test_workspace_bytes():
    f = _lib.qlora_workspace_bytes_dropout
    for op in (0, 1):
        for args in ((300, 512, 320, 16, 1), (300, 512, 768, 12, 3), (5, 512, 320, 7, 1), (300, 512, 320, 0, 1)):
            assert f(op, *args) >= _lib.qlora_workspace_bytes_fused(op, *args)
    assert f(0, 300, 512, 320, 257, 1) == 0
    assert f(2, 300, 512, 320, 16, 1) == 0
