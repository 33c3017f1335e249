"""Products with group-scaled weights of inputs so large that the integer sums of a group pass fp32's
range while scaled they do not: the bounds of tests/test_gpu_group.py hold there too, for the
tokens beside as well."""

import numpy as np
import pytest

import synth
from oracle import groups as og
from tests import gpu_cases as gc
from tests.test_gpu_group import _bound, _weight, q  # noqa: F401  (q: the module's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N", [(1, 70), (3, 70), (7, 16400), (12, 6000), (40, 70), (64, 4096), (64, 8200)])
@pytest.mark.parametrize("group,zeros,bf16", [(32, True, False), (64, False, True), (128, True, True), (512, False, False)])
def test_large_inputs_with_small_scales(q, M, N, group, zeros, bf16):  # noqa: F811
    """Token 0 near the largest bf16 in every column, scales of 2^-40 to 2^-20 (in a few rows 2^60: infinite
    there, as sums in fp32 are); another token with values of 2^-60; zeros up to 255."""
    print(f"large M={M} N={N} group={group} zeros={zeros} bf16={bf16}", flush=True)
    K = 1024
    rng = np.random.default_rng([M, N, group])
    s = np.exp2(rng.uniform(-40, -20, (N, K // group))).astype(np.float32)
    wide = np.zeros(N, bool)
    wide[3::17] = True
    s[wide] = np.float32(2.0 ** 60)
    z = np.full((N, K // group), 8, np.uint8)
    if zeros:
        z = rng.integers(0, 16, z.shape).astype(np.uint8)
        z[5::11] = 255
    codes, s, z, gw = _weight(q, N, K, group, zeros, bf16, s=s, z=z)
    x = rng.standard_normal((M, K)).astype(np.float32)
    # one sign for the first half: its sums pass the range; both signs after it
    x[0] = 3.3e38 * np.where(np.arange(K) < K // 2, 1, rng.choice([-1, 1], K))
    if M > 2:
        x[2] *= np.float32(2.0 ** -60)
    xb = synth.to_bf16_bits(x)
    with np.errstate(over="ignore"):
        want, mag = og.product(gc.f64(xb), codes, s, z, group)
    Y = gc.host_f32_from_bf16(q.group_linear_fwd(gw, gc.dev_bf16(xb))).reshape(M, N)
    tol = _bound(want, mag, K, group)
    past = np.abs(want) > 1e39
    assert past.any() and not past[1:].any() and not past[:, ~wide].any()
    assert not np.isfinite(Y[past]).any()
    sure = ~wide[None] | (np.arange(M) > 0)[:, None]   # (the others are sums of infinities)
    err = np.abs(Y - want)
    assert np.all(np.isfinite(Y[sure])) and np.all(err[sure] <= tol[sure]), float(np.max((err / tol)[sure]))


@pytest.mark.parametrize("M", [2, 40])
def test_scales_beyond_the_range_of_a_scaled_one(q, M):  # noqa: F811
    """Scales of up to 2^126 with inputs of 2^-110 beside a token that is not finite: neither a scale nor
    a group's sum may leave the range where their product does not."""
    N, K, group = 40, 256, 64
    rng = np.random.default_rng(M)
    s = np.exp2(rng.uniform(80, 126, (N, K // group))).astype(np.float32)
    codes, s, z, gw = _weight(q, N, K, group, True, False, s=s)
    x = rng.standard_normal((M, K)).astype(np.float32) * np.float32(2.0 ** -110)
    x[0, 9] = np.inf
    xb = (x.view(np.uint32) >> 16).astype(np.uint16)
    with np.errstate(invalid="ignore"):
        want, mag = og.product(gc.f64(xb), codes, s, z, group)
    Y = gc.host_f32_from_bf16(q.group_linear_fwd(gw, gc.dev_bf16(xb))).reshape(M, N)
    assert not np.isfinite(Y[0]).any()
    assert np.all(np.abs(Y[1:] - want[1:]) <= _bound(want, mag, K, group)[1:])


def test_launches_of_too_many_threads_are_refused(q):  # noqa: F811
    """Sizes whose launch would pass 2^32 threads along an axis stop on the host (the addresses are not
    used), and the next call runs."""
    import torch
    fake = 0x10000
    lib = q._lib
    assert lib.qlora_group_quantize(fake, 1, 1 << 19, 1 << 18, 128, 1, fake, fake, None, None) == lib.QLORA_ERR_LAUNCH
    w = lib.qlora_group_weight(fake, fake, None, 1 << 31, 32, 32, 1)
    assert lib.qlora_group_linear_fwd(w, fake, 1, fake, None) == lib.QLORA_ERR_LAUNCH
    _, _, _, gw = _weight(q, 8, 64, 32, False, True)
    assert q.group_linear_fwd(gw, torch.ones((1, 64), dtype=torch.bfloat16, device="cuda")).isfinite().all()
