"""Norms of query / key heads with the rotation on the GPU, where single values decide: a zero eps with
head counts that leave a wave's round partly filled."""

import pytest

from tests import test_gpu_qk as tq
from tests.test_gpu_qk import Case, q  # noqa: F401  (q: the module's fixture)

pytestmark = pytest.mark.gpu


# ---- eps = 0 ---------------------------------------------------------------------------

@pytest.mark.parametrize("nq,nk", [(1, 1), (3, 1), (4, 4), (15, 5), (7, 2)])
@pytest.mark.parametrize("d,rot", [(128, 128), (80, 32), (64, 64), (256, 64), (12, 4)])
@pytest.mark.parametrize("bf16", [False, True])
def test_zero_eps(q, monkeypatch, nq, nk, d, rot, bf16):  # noqa: F811
    """Rows that are not zero need no eps, whether or not the heads fill a wave's rounds."""
    import torch
    monkeypatch.setattr(tq, "EPS", 0.0)
    c = Case(9, nq, nk, d, rot, True, False, bf16)
    got = c.fwd(q)
    torch.cuda.synchronize()
    c.check_fwd(got)
    got = c.bwd(q)
    torch.cuda.synchronize()
    c.check_bwd(got)
