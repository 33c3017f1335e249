"""The gated oracle: activations against their textbook forms and differences; refusals of
the binding and the C ABI (no GPU)."""

import math

import numpy as np
import pytest
import torch

import bit_quantized_lora_nf4_amd as q
from bit_quantized_lora_nf4_amd import _lib
from oracle import gated as og

FAKE = 0x10000


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
def test_activation(name):
    x = np.linspace(-12, 12, 2001)
    f, df = og.act(name, x)
    if name == "silu":
        want = x / (1 + np.exp(-x))
    else:
        want = 0.5 * x * (1 + np.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))
    assert np.max(np.abs(f - want)) < 1e-12
    h = 1e-5
    num = (og.act(name, x + h)[0] - og.act(name, x - h)[0]) / (2 * h)
    assert np.max(np.abs(num - df)) < 1e-8  # h^2 times the third derivative (below 2), and rounding / h


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
def test_gradient_against_differences(name):
    rng = np.random.default_rng(1)
    Y, dH = rng.standard_normal((3, 10)), rng.standard_normal((3, 5))
    dY = og.backward(dH, Y, name)
    h = 1e-5
    for i in np.ndindex(Y.shape):
        up, dn = Y.copy(), Y.copy()
        up[i] += h
        dn[i] -= h
        num = np.sum(dH * (og.forward(up, name) - og.forward(dn, name))) / (2 * h)
        assert num == pytest.approx(dY[i], abs=1e-7)


P, K, M, R = 192, 128, 20, 4


def _qw(rows=2 * P):
    return q.NF4Weight(torch.zeros(rows * K // 2, dtype=torch.uint8), torch.zeros(rows * K // 64, dtype=torch.int8),
                       torch.zeros(2, dtype=torch.float32), torch.zeros(2, dtype=torch.float32), rows, K)


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_binding_rejects():
    with pytest.raises(TypeError, match="CUDA"):
        q.gated_fwd(_qw(), bf(M, K), bf(2 * R, K), bf(2 * P, R))
    with pytest.raises(TypeError, match="CUDA"):
        q.gated_bwd(_qw(), bf(M, P), bf(M, 2 * P), bf(M, K), bf(2 * R, K), bf(2 * P, R))
    with pytest.raises(TypeError, match="CUDA"):
        q.gated_bwd(_qw(), bf(M, P), bf(M, 2 * P))
    bad = [dict(X=bf(M, K + 64)), dict(act="relu"), dict(A=bf(2 * R + 1, K)), dict(B=bf(2 * P, 2 * R)),
           dict(H=bf(M, 2 * P)), dict(Y=bf(M, P)), dict(U=bf(M, R)), dict(qw=_qw(2 * P + 1)),
           dict(ws=torch.zeros(8, dtype=torch.uint8)), dict(X=bf(M * K)), dict(dropout=q.Dropout(1.0))]
    for kw in bad:
        a = dict(qw=_qw(), X=bf(M, K), A=bf(2 * R, K), B=bf(2 * P, R))
        a.update(kw)
        with pytest.raises(ValueError):
            q.gated_fwd(**a)
    bad = [dict(dH=bf(M, 2 * P)), dict(Y=bf(M, P)), dict(X=None), dict(U=bf(M, R)), dict(dX=bf(M, P)),
           dict(dA=bf(R, K)), dict(dB=bf(P, R)), dict(act="gelu"), dict(dH=bf(M + 1, P)), dict(Y=bf(2 * P, M).t())]
    for kw in bad:
        a = dict(qw=_qw(), dH=bf(M, P), Y=bf(M, 2 * P), X=bf(M, K), A=bf(2 * R, K), B=bf(2 * P, R))
        a.update(kw)
        with pytest.raises(ValueError):
            q.gated_bwd(**a)


def test_abi_rejects():
    w = _lib.qlora_nf4_weight(FAKE, FAKE, FAKE, FAKE, 2 * P, K)
    big = 1 << 40
    fwd = lambda w=w, X=FAKE, M=M, A=FAKE, r=R, act=0, drop=None, H=FAKE, ws=FAKE, n=big: _lib.qlora_gated_fwd(  # noqa: E731
        w, X, M, A, FAKE, r, 16.0, act, drop, H, None, None, ws, n, None)
    odd = _lib.qlora_nf4_weight(FAKE, FAKE, FAKE, FAKE, 2 * P + 1, K)
    assert fwd(w=odd) == _lib.QLORA_ERR_SHAPE
    assert fwd(M=0) == _lib.QLORA_ERR_SHAPE
    assert fwd(act=2) == _lib.QLORA_ERR_VALUE
    assert fwd(r=129) == _lib.QLORA_ERR_RANK       # 2 x 136 ranks
    assert fwd(X=None) == _lib.QLORA_ERR_NULL
    assert fwd(H=None) == _lib.QLORA_ERR_NULL
    assert fwd(A=None) == _lib.QLORA_ERR_NULL
    assert fwd(X=FAKE + 8) == _lib.QLORA_ERR_ALIGN
    assert fwd(ws=None) == _lib.QLORA_ERR_WORKSPACE
    assert fwd(n=_lib.qlora_workspace_bytes_gated(0, M, K, P, R) - 1) == _lib.QLORA_ERR_WORKSPACE
    assert fwd(drop=_lib.qlora_drop(1.0, 0, 0, None)) == _lib.QLORA_ERR_VALUE
    assert fwd(M=1 << 25) == _lib.QLORA_ERR_SHAPE  # X past 4 GiB
    bwd = lambda dH=FAKE, Y=FAKE, X=FAKE, r=R, act=0, dX=FAKE, dA=FAKE, n=big, M=M: _lib.qlora_gated_bwd(  # noqa: E731
        w, dH, Y, X, M, FAKE, FAKE, r, 16.0, act, None, None, dX, dA, FAKE, FAKE, n, None)
    assert bwd(dH=None) == _lib.QLORA_ERR_NULL
    assert bwd(Y=None) == _lib.QLORA_ERR_NULL
    assert bwd(X=None) == _lib.QLORA_ERR_NULL
    assert bwd(dA=None) == _lib.QLORA_ERR_NULL
    assert bwd(r=0, dX=None) == _lib.QLORA_ERR_NULL
    assert bwd(act=-1) == _lib.QLORA_ERR_VALUE
    assert bwd(Y=FAKE + 4) == _lib.QLORA_ERR_ALIGN
    assert bwd(n=100) == _lib.QLORA_ERR_WORKSPACE
    assert bwd(M=1 << 25) == _lib.QLORA_ERR_SHAPE
    assert bwd(r=200) == _lib.QLORA_ERR_RANK


def test_workspace_bytes():
    f = _lib.qlora_workspace_bytes_gated
    H = _lib.QLORA_WORKSPACE_HEADER_BYTES
    assert f(0, 4096, 4096, 11008, 0) == 0          # no adapter, nothing to keep
    assert f(0, 1, 4096, 11008, 0) == H             # the small-M path's counters
    assert f(0, 1, 64, 32768, 0) == H
    assert f(0, 1, 64, 32769, 0) == 0               # past the small-M path
    assert f(0, 300, 512, 100, 16) >= H + 300 * 32 * 2
    assert f(1, 300, 512, 101, 0) >= H + 300 * 2 * 104 * 2   # the padded [dG | dL]
    assert f(2, 300, 512, 100, 16) == 0
    assert f(0, 300, 512, 100, 129) == 0
    assert f(0, 300, 500, 100, 8) == 0
