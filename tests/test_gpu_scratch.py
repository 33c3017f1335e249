"""The workspaces that the binding makes by itself, and what a workspace holds before a call."""

import pytest

from bit_quantized_lora_nf4_amd import _lib
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


@pytest.mark.parametrize("parts", [1, 3])
def test_large_workspaces_are_not_cleared_whole(q, parts, monkeypatch):
    """A call without a workspace clears the header of a large one and leaves the rest, which
    may be tens of megabytes of partial sums, as it is."""
    import torch
    M, K, N, r = 600, 4096, 2304, 64
    h = dc.linear_inputs(M, K, N // parts, r, parts, seed=3)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"])
    d = q.Dropout(0.25, seed=4)
    assert all(q.qlora_workspace_bytes_dropout(op, M, K, N, r, parts) > 4 << 20 for op in (0, 1))
    filled, real = [], torch.zeros
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: filled.append(real(*a, **k)) or filled[-1])
    Y, U = q.linear_fwd_fused(qw, parts, dev["X"], dev["A"], dev["B"], ALPHA, dropout=d)
    q.linear_bwd_fused(qw, parts, dev["dY"], dev["X"], dev["A"], dev["B"], ALPHA, U, dropout=d)
    torch.cuda.synchronize()
    assert sum(t.numel() * t.element_size() for t in filled) == 0


@pytest.mark.parametrize("M,K,N,r,parts", [(5, 256, 72, 8, 1), (40, 256, 101, 12, 1), (300, 512, 512, 16, 2),
                                           (64, 4096, 4096, 64, 1)])
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_workspace_contents_do_not_matter(q, M, K, N, r, parts, p):
    """A workspace of NaN patterns behind its header gives what a zeroed one gives, with
    dropout and without."""
    import torch
    h = dc.linear_inputs(M, K, N // parts, r, parts, seed=25)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"])
    d = q.Dropout(p, seed=6) if p else None
    size = q.qlora_workspace_bytes_dropout if p else q.qlora_workspace_bytes_fused
    outs = []
    for fill in (0, 0xFF):
        ws = [torch.full((size(op, M, K, N, r, parts),), fill, dtype=torch.uint8, device="cuda") for op in (0, 1)]
        for w in ws:
            w[:_lib.QLORA_WORKSPACE_HEADER_BYTES] = 0
        Y, U = q.linear_fwd_fused(qw, parts, dev["X"], dev["A"], dev["B"], ALPHA, dropout=d, ws=ws[0])
        outs.append((Y, U) + q.linear_bwd_fused(qw, parts, dev["dY"], dev["X"], dev["A"], dev["B"], ALPHA, U, dropout=d,
                                                ws=ws[1]))
    for a, b in zip(*outs):
        assert torch.equal(a, b) and bool(torch.isfinite(a).all())
