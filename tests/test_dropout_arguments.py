"""The ``dropout`` argument is checked by every call that takes one, also where nothing is
dropped (no adapter): a value of another type, or a Dropout out of range, is refused before
anything else happens.  No GPU needed."""

import pytest
import torch

import bit_quantized_lora_nf4_amd as q

N, K, M, r = 256, 128, 8, 4


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def _qw():
    return q.NF4Weight(torch.zeros(N * K // 2, dtype=torch.uint8), torch.zeros(N * K // 64, dtype=torch.int8),
                       torch.zeros(2, dtype=torch.float32), torch.zeros(2, dtype=torch.float32), N, K)


CALLS = {
    "linear_fwd": lambda d, a: q.linear_fwd(_qw(), bf(M, K), *a(r, r), dropout=d),
    "linear_fwd_fused": lambda d, a: q.linear_fwd_fused(_qw(), 1, bf(M, K), *a(r, r), dropout=d),
    "linear_bwd": lambda d, a: q.linear_bwd(_qw(), bf(M, N), bf(M, K), *a(r, r), dropout=d),
    "linear_bwd_fused": lambda d, a: q.linear_bwd_fused(_qw(), 1, bf(M, N), bf(M, K), *a(r, r), dropout=d),
    "gated_fwd": lambda d, a: q.gated_fwd(_qw(), bf(M, K), *a(2 * r, r), dropout=d),
    "gated_bwd": lambda d, a: q.gated_bwd(_qw(), bf(M, N // 2), bf(M, N), bf(M, K), *a(2 * r, r), dropout=d),
    "dropout": lambda d, a: q.dropout(torch.zeros(8), d),
}
ADAPTERS = {"adapter": lambda R, r: (bf(R, K), bf(N, r)), "none": lambda R, r: (None, None)}


@pytest.mark.parametrize("adapter", ADAPTERS)
@pytest.mark.parametrize("call", CALLS)
def test_refused(call, adapter):
    for bad in (0.1, "0.1", (0.1, 1, 2)):
        with pytest.raises(TypeError, match="Dropout"):
            CALLS[call](bad, ADAPTERS[adapter])
    for p in (-0.1, 1.0, float("nan")):
        with pytest.raises(ValueError, match="probability"):
            CALLS[call](q.Dropout(p), ADAPTERS[adapter])
    with pytest.raises(ValueError, match="64-bit"):
        CALLS[call](q.Dropout(0.1, seed=-1), ADAPTERS[adapter])


@pytest.mark.parametrize("call", CALLS)
def test_taken(call):
    """A good one passes on to the check of the devices."""
    with pytest.raises(TypeError, match="CUDA"):
        CALLS[call](q.Dropout(0.1), ADAPTERS["adapter"])


def test_dropout_by_itself_needs_one():
    with pytest.raises(TypeError, match="Dropout"):
        q.dropout(torch.zeros(8), None)
