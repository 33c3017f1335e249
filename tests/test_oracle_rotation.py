"""The oracle of query / key norms with the position rotation against complex products and
differences, and the refusals of the binding and the C ABI (no GPU)."""

import numpy as np
import pytest
import torch

import bit_quantized_lora_nf4_amd as q
from bit_quantized_lora_nf4_amd import _lib
from oracle import rotation as orot

FAKE = 0x10000
EPS = 1e-5


def _case(seed=0, M=3, heads=2, d=12, rot=8):
    rng = np.random.default_rng(seed)
    return (rng.standard_normal((M, heads, d)), 1 + 0.1 * rng.standard_normal(d), rng.integers(-50, 100, M),
            (100.0 ** -(np.arange(rot // 2) / (rot // 2))).astype(np.float32), rng.standard_normal((M, heads, d)))


@pytest.mark.parametrize("interleaved", [False, True])
def test_turn_is_a_complex_product(interleaved):
    x, _, pos, f, _ = _case()
    z = orot.turn(x, pos, f, interleaved)
    a, b = orot.pairs(8, interleaved)
    want = (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos[:, None] * f.astype(np.float64))[:, None]
    assert np.max(np.abs(z[..., a] + 1j * z[..., b] - want)) < 1e-13
    assert np.array_equal(z[..., 8:], x[..., 8:])
    back = orot.turn(z, pos, f, interleaved, -1.0)
    assert np.max(np.abs(back - x)) < 1e-13


def test_products_depend_on_the_distance_alone():
    """The property the rotation is made for."""
    x, _, _, f, y = _case(1)
    dots = []
    for shift in (0, 1000):
        a = orot.turn(x, np.array([5, 9, 30]) + shift, f, False)
        b = orot.turn(y, np.array([2, 7, 11]) + shift, f, False)
        dots.append(np.sum(a * b, axis=-1))
    assert np.max(np.abs(dots[0] - dots[1])) < 1e-11


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_gradients_against_differences(interleaved, norm):
    x, w, pos, f, dz = _case(2)
    w = w if norm else None
    dx, dw = orot.backward(dz, x, w, pos, f, EPS, interleaved)

    def loss(x, w):
        return np.sum(dz * orot.forward(x, w, pos, f, EPS, interleaved))
    h = 1e-6
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        # rounding of the two sums (about 1e-15 of values near 10) over 2 h, and h^2 times the
        # third derivative
        assert (loss(x + e, w) - loss(x - e, w)) / (2 * h) == pytest.approx(dx[i], abs=1e-7)
    if norm:
        for i in range(len(w)):
            e = np.zeros_like(w)
            e[i] = h
            assert (loss(x, w + e) - loss(x, w - e)) / (2 * h) == pytest.approx(dw[i], abs=1e-7)


M, NQ, NK, D = 5, 4, 2, 32


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def _fwd(**kw):
    a = dict(Y=bf(M, (NQ + 2 * NK) * D), positions=torch.zeros(M, dtype=torch.int64), inv_freq=torch.ones(D // 2),
             n_heads=NQ, n_kv_heads=NK, q_weight=bf(D), k_weight=bf(D))
    a.update(kw)
    return q.qk_norm_rope_fwd(**a)


def _bwd(**kw):
    a = dict(dQ=bf(M, NQ, D), dK=bf(M, NK, D), dV=bf(M, NK, D), positions=torch.zeros(M, dtype=torch.int64),
             inv_freq=torch.ones(D // 2), Y=bf(M, (NQ + 2 * NK) * D), q_weight=bf(D), k_weight=bf(D))
    a.update(kw)
    return q.qk_norm_rope_bwd(**a)


SHARED = [dict(positions=torch.zeros(M + 1, dtype=torch.int64)), dict(positions=torch.zeros(M, 1, dtype=torch.int64)),
          dict(inv_freq=torch.ones(D // 2 + 2)), dict(inv_freq=torch.ones(3)), dict(inv_freq=torch.ones(2, 8)),
          dict(q_weight=None), dict(k_weight=None), dict(q_weight=bf(D - 1)), dict(k_weight=bf(2 * D)),
          dict(inv_freq=torch.ones(2 * D)[::4])]


@pytest.mark.parametrize("kw", SHARED + [dict(n_heads=3), dict(n_heads=0), dict(n_kv_heads=0), dict(Y=bf(M, 8, D)),
                                         dict(Y=bf((NQ + 2 * NK) * D, M).t()), dict(Q=bf(M, NQ, D + 4)),
                                         dict(K=bf(M, NQ, D)), dict(Y=bf(M, 8 * 6), q_weight=bf(6), k_weight=bf(6)),
                                         dict(Y=bf(M, 8 * 260), q_weight=bf(260), k_weight=bf(260))])
def test_forward_rejects(kw):
    with pytest.raises(ValueError):
        _fwd(**kw)


@pytest.mark.parametrize("kw", SHARED + [dict(dK=bf(M + 1, NK, D)), dict(dK=bf(M, NK, D - 4)), dict(dV=bf(M, NK + 1, D)),
                                         dict(dQ=bf(M, NQ * D)), dict(dK=bf(M, NK * D)), dict(Y=bf(M, 6 * D)),
                                         dict(Y=None), dict(dY=bf(M, 7 * D)), dict(dqw=bf(D + 1)),
                                         dict(dkw=bf(1, D)), dict(ws=torch.zeros(64, dtype=torch.uint8)),
                                         dict(dQ=bf(M, 0, D)), dict(dK=bf(M, 0, D), dV=bf(M, 0, D)),
                                         dict(dQ=bf(NQ, M, D).transpose(0, 1))])
def test_backward_rejects(kw):
    with pytest.raises(ValueError):
        _bwd(**kw)


@pytest.mark.parametrize("kw", [dict(positions=torch.zeros(M, dtype=torch.int32)),
                                dict(inv_freq=torch.ones(D // 2, dtype=torch.float64)), dict(q_weight=torch.ones(D)),
                                dict(k_weight=None, q_weight=None), {}])
def test_types_and_device(kw):
    for call in (_fwd, _bwd):
        with pytest.raises(TypeError):
            call(**kw)
    for call, name in ((_fwd, "Y"), (_bwd, "dQ")):
        with pytest.raises(TypeError):
            call(**{name: None})
        with pytest.raises(TypeError):
            call(**{name: torch.zeros(M, NQ, D, dtype=torch.float16)})


def _shape(**kw):
    a = dict(M=M, nq=NQ, nk=NK, d=D, rot=D, dtype=1, interleaved=0, eps=1e-6)
    a.update(kw)
    return _lib.qlora_qk_shape(*a.values())


def test_abi_refusals():
    """Fake addresses: every call stops at its arguments."""
    S, D_, V_ = _lib.QLORA_ERR_SHAPE, _lib.QLORA_ERR_DTYPE, _lib.QLORA_ERR_VALUE
    for kw, status in [(dict(M=0), S), (dict(nq=0), S), (dict(nk=-1), S), (dict(d=30), S), (dict(d=260), S),
                       (dict(d=0), S), (dict(rot=36), S), (dict(rot=-4), S), (dict(rot=6), S), (dict(dtype=2), D_),
                       (dict(M=1 << 40), S), (dict(nq=(1 << 20) + 1), S), (dict(interleaved=2), V_),
                       (dict(eps=float("nan")), V_), (dict(eps=-1.0), V_), (dict(eps=float("inf")), V_)]:
        assert _lib.qlora_qk_fwd(_shape(**kw), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None) == status, kw
        assert _lib.qlora_qk_bwd(_shape(**kw), *[FAKE] * 11, FAKE, 1 << 30, None) == status, kw
        assert _lib.qlora_workspace_bytes_qk(_shape(**kw), 1) == 0, kw
    ok = [FAKE] * 7
    for i, status in [(0, _lib.QLORA_ERR_NULL), (1, _lib.QLORA_ERR_NULL), (2, _lib.QLORA_ERR_NULL),
                      (3, _lib.QLORA_ERR_NULL), (4, _lib.QLORA_ERR_NULL), (5, _lib.QLORA_ERR_NULL),
                      (6, _lib.QLORA_ERR_NULL)]:
        a = list(ok)
        a[i] = None
        assert _lib.qlora_qk_fwd(_shape(), *a, None) == status, i
        a[i] = FAKE + 2
        assert _lib.qlora_qk_fwd(_shape(), *a, None) == _lib.QLORA_ERR_ALIGN, i
    ws = _lib.qlora_workspace_bytes_qk(_shape(), 1)
    assert ws > _lib.QLORA_WORKSPACE_HEADER_BYTES and _lib.qlora_workspace_bytes_qk(_shape(), 0) == 0
    ok = [FAKE] * 11  # dQ dK dV Y positions inv_freq qw kw dY dqw dkw
    for i in range(11):
        a = list(ok)
        a[i] = None
        assert _lib.qlora_qk_bwd(_shape(), *a, FAKE, ws, None) == _lib.QLORA_ERR_NULL, i
        a[i] = FAKE + 2
        assert _lib.qlora_qk_bwd(_shape(), *a, FAKE, ws, None) == _lib.QLORA_ERR_ALIGN, i
    assert _lib.qlora_qk_bwd(_shape(), *ok, FAKE, ws - 1, None) == _lib.QLORA_ERR_WORKSPACE
    assert _lib.qlora_qk_bwd(_shape(), *ok, None, ws, None) == _lib.QLORA_ERR_WORKSPACE
    assert _lib.qlora_qk_bwd(_shape(), *ok, FAKE + 8, ws, None) == _lib.QLORA_ERR_ALIGN
