"""The oracle of 4-bit integers with group scales (facts of arithmetic), and the refusals of
the binding and the C ABI (no GPU)."""

import numpy as np
import pytest
import torch

import bit_quantized_lora_nf4_amd as q
from bit_quantized_lora_nf4_amd import _lib
from oracle import groups as og

FAKE = 0x10000


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
def test_values_are_within_half_a_step(zeros, bf16):
    W = np.random.default_rng(0).standard_normal((5, 256)).astype(np.float32)
    codes, s, z = og.quantize(W, 64, zeros, bf16)
    step = np.repeat(s, 64, axis=1)
    # rounding the scale (by at most 2^-8) can leave the largest values 15 * 2^-8 steps past
    # the last code; without it they are a rounding error past it
    slack = 15 * 2.0 ** -8 if bf16 else 1e-5
    assert np.all(np.abs(og.values(codes, s, z, 64) - W) <= (0.5 + slack) * step)
    assert codes.max() == 15 and codes.min() == (0 if zeros else 1)


def test_exact_multiples_come_back():
    ints = np.random.default_rng(1).integers(-7, 8, (3, 128)).astype(np.float32)
    ints[:, ::32] = 7
    for step in (1.0, 2.0 ** -20, 0.375):
        codes, s, z = og.quantize(ints * np.float32(step) , 32, False, True)
        # max / 7 is rounded twice; where it is the step itself, every value is
        same = s == np.float32(step)
        assert np.array_equal(og.values(codes, s, z, 32)[np.repeat(same, 32, 1)], (ints * step)[np.repeat(same, 32, 1)])
    assert same.all()


def test_zero_and_subnormal_groups_stand_for_zeros():
    W = np.zeros((2, 64), np.float32)
    W[1, :32] = 2.0 ** -140
    for zeros in (False, True):
        codes, s, z = og.quantize(W, 32, zeros, True)
        assert not og.values(codes, s, z, 32).any() and not s.any()


def test_one_sided_groups_keep_zero():
    """A group of one sign is quantized over a range that includes zero."""
    W = np.full((1, 32), 3.0, np.float32)
    W[0, 0] = 0.0
    codes, s, z = og.quantize(W, 32, True, False)
    assert z[0, 0] == 0 and codes[0, 0] == 0 and codes[0, 1] == 15
    codes, s, z = og.quantize(-W, 32, True, False)
    assert z[0, 0] == 15 and codes[0, 0] == 15 and codes[0, 1] == 0


def test_pack():
    codes = np.arange(64, dtype=np.uint8).reshape(2, 32) % 16
    p = og.pack(codes)
    assert p[0] == 0x10 and p[7] == 0xFE
    assert np.array_equal(og.unpack(p, 2, 32), codes)


N, K, G = 24, 128, 32


def _gw(**kw):
    a = dict(codes=torch.zeros(N * K // 2, dtype=torch.uint8), scales=torch.zeros(N, K // G), zeros=None, n_rows=N,
             n_cols=K, group=G)
    a.update(kw)
    return q.GroupWeight(**a)


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("kw", [
    dict(group=48), dict(group=0), dict(group=-32), dict(group=256), dict(n_rows=0), dict(n_cols=96),
    dict(codes=torch.zeros(N * K // 2 - 1, dtype=torch.uint8)), dict(scales=torch.zeros(N, K // G + 1)),
    dict(scales=torch.zeros(N * K // G)), dict(scales=torch.zeros(K // G, N).t()),
    dict(zeros=torch.zeros(N, K // G - 1, dtype=torch.uint8))])
def test_weight_arrays_are_checked(kw):
    for call in (lambda w: q.group_linear_fwd(w, bf(3, w.n_cols)), lambda w: q.group_dequantize(w)):
        with pytest.raises(ValueError):
            call(_gw(**kw))


@pytest.mark.parametrize("kw", [
    dict(codes=torch.zeros(N * K // 2, dtype=torch.int8)), dict(scales=torch.zeros(N, K // G, dtype=torch.float16)),
    dict(zeros=torch.zeros(N, K // G))])
def test_weight_types_are_checked(kw):
    with pytest.raises(TypeError):
        q.group_linear_fwd(_gw(**kw), bf(3, K))
    with pytest.raises(TypeError):
        q.group_dequantize(_gw(**kw))


def test_binding_rejects():
    with pytest.raises(TypeError, match="CUDA"):
        q.group_linear_fwd(_gw(), bf(3, K))
    with pytest.raises(TypeError, match="bfloat16"):
        q.group_linear_fwd(_gw(), torch.zeros(3, K))
    for X in (bf(K), bf(3, K + 32), bf(1, 3, K), bf(K, 3).t()):
        with pytest.raises(ValueError):
            q.group_linear_fwd(_gw(), X)
    for Y in (bf(3, N + 1), bf(2, N), bf(N, 3).t()):
        with pytest.raises(ValueError):
            q.group_linear_fwd(_gw(), bf(3, K), Y=Y)
    with pytest.raises(TypeError):
        q.group_dequantize(_gw(), torch.float16)
    with pytest.raises(ValueError):
        q.group_dequantize(_gw(), out=bf(N, K + 32))
    with pytest.raises(TypeError):
        q.group_dequantize(_gw(), out=torch.zeros(N, K))
    with pytest.raises(TypeError, match="CUDA"):
        q.group_quantize(bf(N, K), G)
    with pytest.raises(TypeError):
        q.group_quantize(torch.zeros(N, K, dtype=torch.float16), G)
    with pytest.raises(TypeError):
        q.group_quantize(bf(N, K), G, scale_dtype=torch.float16)
    with pytest.raises(TypeError):
        q.group_quantize([[0.0] * K], G)
    for W, g in ((bf(N, K), 48), (bf(N, K), 256), (bf(N, K), 0), (bf(0, K), G), (bf(N, 0), G), (bf(N * K), G),
                 (bf(K, N).t(), G)):
        with pytest.raises(ValueError):
            q.group_quantize(W, g)


def _w(**kw):
    a = dict(codes=FAKE, scales=FAKE, zeros=None, n_rows=N, n_cols=K, group=G, scale_type=0)
    a.update(kw)
    return _lib.qlora_group_weight(*a.values())


def test_abi_refusals():
    """Fake addresses: every call stops at its arguments."""
    bad = [(dict(n_rows=0), _lib.QLORA_ERR_SHAPE), (dict(group=33), _lib.QLORA_ERR_SHAPE),
           (dict(n_cols=100), _lib.QLORA_ERR_SHAPE), (dict(group=0), _lib.QLORA_ERR_SHAPE),
           (dict(n_cols=_lib.QLORA_GROUP_MAX_COLS + 32), _lib.QLORA_ERR_SHAPE),
           (dict(n_rows=1 << 40), _lib.QLORA_ERR_SHAPE), (dict(scale_type=2), _lib.QLORA_ERR_DTYPE),
           (dict(codes=None), _lib.QLORA_ERR_NULL), (dict(scales=None), _lib.QLORA_ERR_NULL),
           (dict(codes=FAKE + 8), _lib.QLORA_ERR_ALIGN), (dict(scales=FAKE + 2), _lib.QLORA_ERR_ALIGN)]
    for kw, status in bad:
        assert _lib.qlora_group_linear_fwd(_w(**kw), FAKE, 1, FAKE, None) == status, kw
        assert _lib.qlora_group_dequantize(_w(**kw), FAKE, 1, None) == status, kw
    f = _lib.qlora_group_linear_fwd
    assert f(_w(), FAKE, 0, FAKE, None) == _lib.QLORA_ERR_SHAPE
    assert f(_w(), FAKE, (1 << 20) + 1, FAKE, None) == _lib.QLORA_ERR_SHAPE
    assert f(_w(n_rows=(1 << 31) + 1, n_cols=32), FAKE, 1, FAKE, None) == _lib.QLORA_ERR_SHAPE
    assert f(_w(), None, 1, FAKE, None) == _lib.QLORA_ERR_NULL
    assert f(_w(), FAKE, 1, None, None) == _lib.QLORA_ERR_NULL
    assert f(_w(), FAKE + 8, 1, FAKE, None) == _lib.QLORA_ERR_ALIGN
    d = _lib.qlora_group_dequantize
    assert d(_w(), None, 1, None) == _lib.QLORA_ERR_NULL
    assert d(_w(), FAKE, 2, None) == _lib.QLORA_ERR_DTYPE
    assert d(_w(), FAKE + 4, 1, None) == _lib.QLORA_ERR_ALIGN
    g = _lib.qlora_group_quantize
    assert g(FAKE, 1, N, K, 40, 0, FAKE, FAKE, None, None) == _lib.QLORA_ERR_SHAPE
    assert g(FAKE, 1, N, K, G, 3, FAKE, FAKE, None, None) == _lib.QLORA_ERR_DTYPE
    assert g(FAKE, 3, N, K, G, 0, FAKE, FAKE, None, None) == _lib.QLORA_ERR_DTYPE
    assert g(None, 1, N, K, G, 0, FAKE, FAKE, None, None) == _lib.QLORA_ERR_NULL
    assert g(FAKE, 1, N, K, G, 0, None, FAKE, None, None) == _lib.QLORA_ERR_NULL
    assert g(FAKE, 1, N, K, G, 0, FAKE, None, FAKE, None) == _lib.QLORA_ERR_NULL
    assert g(FAKE + 4, 1, N, K, G, 0, FAKE, FAKE, None, None) == _lib.QLORA_ERR_ALIGN
    assert g(FAKE, 1, N, K, G, 0, FAKE + 4, FAKE, None, None) == _lib.QLORA_ERR_ALIGN
    assert g(FAKE, 1, N, K, G, 0, FAKE, FAKE + 2, None, None) == _lib.QLORA_ERR_ALIGN


@pytest.mark.parametrize("zeros", [False, True])
def test_a_group_with_a_bad_value_is_nan(zeros):
    W = np.ones((3, 64), np.float32)
    W[0, 3], W[1, 40], W[2, 7] = np.inf, np.nan, -np.inf
    with np.errstate(over="ignore", invalid="ignore"):
        codes, s, z = og.quantize(W, 32, zeros, False)
    assert np.isnan(s).tolist() == [[True, False], [False, True], [True, False]]
    v = og.values(codes, s, z, 32).reshape(3, 2, 32)
    assert np.all(np.isnan(v[np.isnan(s)])) and np.allclose(v[~np.isnan(s)], 1.0, atol=1e-6)
