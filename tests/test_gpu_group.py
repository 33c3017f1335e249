"""4-bit integers with group scales on the GPU: the quantizer and its inverse bit for bit, the
product with few tokens against float64 within bounds derived below, over sizes that tiles
and waves do not divide, group sizes, scale types and zeros; inputs that are not finite,
sums that overflow, guards around the outputs, strides of Python views, streams, captured
graphs, offsets past 2^32.

Bound of the product: bf16 rounding of the result, half a step, 2^-8 of it; and fp32 sums.  A
result is a sum of terms s (16 + code) x and s (16 + zero) x (each product of a code and x is
exact), each of which passes through fewer than 32 additions inside a matrix instruction,
group / 32 from one to the next, the difference, the product with s, and one addition for
each block of columns and each of at most 8 waves: fewer than 64 + group / 32 + K / 32
roundings of 2^-24, counted twice since nothing is documented about how a matrix instruction
rounds inside."""

import numpy as np
import pytest

import synth
from oracle import groups as og
from tests import gpu_cases as gc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_quantized_lora_nf4_amd as lib
    return lib


def _scales_dev(s, bf16):
    return gc.dev_bf16(synth.to_bf16_bits(s)).view(s.shape) if bf16 else gc.dev_f32(s)


def _weight(q, N, K, group, zeros, bf16, seed=0, codes=None, s=None, z=None):
    """A weight of random codes, its oracle arrays and its GroupWeight."""
    import torch
    rng = np.random.default_rng([seed, N, K, group])
    G = K // group
    codes = rng.integers(0, 16, (N, K)).astype(np.uint8) if codes is None else codes
    s = (rng.uniform(0.5, 2.0, (N, G)) * 0.01 * rng.choice([-1, 1], (N, G))).astype(np.float32) if s is None else s
    if bf16:
        s = synth.bf16_bits_to_f32(synth.to_bf16_bits(s)).reshape(N, G)
    z = (rng.integers(0, 16, (N, G)) if zeros else np.full((N, G), 8)).astype(np.uint8) if z is None else z
    gw = q.GroupWeight(torch.from_numpy(og.pack(codes)).cuda(), _scales_dev(s, bf16),
                       torch.from_numpy(z).cuda() if zeros else None, N, K, group)
    return codes, s, z, gw


def _bound(want, mag, K, group):
    return np.abs(want) * 2.0 ** -8 + 2 * (64 + group / 32 + K / 32) * 2.0 ** -24 * mag


def _check(q, M, N, K, group, zeros, bf16, seed=0):
    import torch
    print(f"group linear M={M} N={N} K={K} group={group} zeros={zeros} bf16={bf16}", flush=True)
    codes, s, z, gw = _weight(q, N, K, group, zeros, bf16, seed)
    rng = np.random.default_rng([seed, M, K])
    xb = synth.to_bf16_bits(rng.standard_normal((M, K)).astype(np.float32))
    Y = q.group_linear_fwd(gw, gc.dev_bf16(xb))
    torch.cuda.synchronize()
    assert Y.shape == (M, N) and Y.dtype == torch.bfloat16
    want, mag = og.product(gc.f64(xb), codes, s, z, group)
    err = np.abs(gc.host_f32_from_bf16(Y).reshape(M, N) - want)
    assert np.all(err <= _bound(want, mag, K, group)), float(np.max(err / _bound(want, mag, K, group)))
    return gw, xb, Y


# ---- quantizer and inverse, bit for bit -----------------------------------------------

QUANT = [(1, 32, 32), (3, 64, 32), (5, 128, 64), (7, 256, 128), (2, 512, 256), (3, 1024, 512), (2, 2048, 1024),
         (4, 96, 96), (3, 1376, 1376), (2, 1376, 32), (33, 4096, 128), (1001, 320, 64), (1, 11008, 11008)]


@pytest.mark.parametrize("N,K,group", QUANT)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("w16,s16", [(True, True), (True, False), (False, True), (False, False)])
def test_quantize_bits(q, N, K, group, zeros, w16, s16):
    import torch
    print(f"quantize {N}x{K} group={group} zeros={zeros} w16={w16} s16={s16}", flush=True)
    rng = np.random.default_rng([N, K, group])
    W = (rng.standard_normal((N, K)) * np.exp(2 * rng.standard_normal((N, 1)))).astype(np.float32)
    # ties of the rounding: multiples of half a step; groups of zeros, of one sign, subnormal
    W.reshape(-1, group)[::5] = rng.integers(-14, 15, W.reshape(-1, group)[::5].shape) * 0.25
    W.reshape(-1, group)[1::7] = 0.0
    W.reshape(-1, group)[2::7] = np.abs(W.reshape(-1, group)[2::7])
    W.reshape(-1, group)[3::11] *= np.float32(2.0 ** -135)
    if w16:
        bits = synth.to_bf16_bits(W)
        W, dev = synth.bf16_bits_to_f32(bits).reshape(N, K), gc.dev_bf16(bits)
    else:
        dev = gc.dev_f32(W)
    gw = q.group_quantize(dev, group, zeros=zeros, scale_dtype=torch.bfloat16 if s16 else torch.float32)
    codes, s, z = og.quantize(W, group, zeros, s16)
    assert np.array_equal(gw.scales.float().cpu().numpy().view(np.uint32), s.view(np.uint32))
    if zeros:
        assert np.array_equal(gw.zeros.cpu().numpy(), z)
    else:
        assert gw.zeros is None
    assert np.array_equal(gw.codes.cpu().numpy(), og.pack(codes))
    # the inverse: one rounding of a product that fp32 holds to 24 bits
    w32 = ((codes.astype(np.float32) - np.repeat(z, group, 1).astype(np.float32)) * np.repeat(s, group, 1))
    assert np.array_equal(q.group_dequantize(gw, torch.float32).cpu().numpy(), w32)
    assert np.array_equal(gc.host_f32_from_bf16(q.group_dequantize(gw)),
                          synth.bf16_bits_to_f32(synth.to_bf16_bits(w32)).reshape(N, K).astype(np.float64))


@pytest.mark.parametrize("group", [32, 128, 512, 96, 1536])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("w16", [True, False])
def test_quantize_not_finite(q, group, zeros, w16):
    """An infinity or a NaN anywhere in a group makes that group NaN, and no other; so does a range
    that fp32 does not hold."""
    import torch
    N, K = 12, 1536
    W = np.random.default_rng(group).standard_normal((N, K)).astype(np.float32)
    for k, bad in enumerate((np.inf, -np.inf, np.nan, -np.nan)):
        W[2 * k + 1, (0, K // 2 + 5, K - 1, K // 3)[k]] = bad
    if zeros:
        W[9, 0], W[9, 1] = 3e38, -3e38
    if w16:
        bits = synth.to_bf16_bits(W)
        W, dev = synth.bf16_bits_to_f32(bits).reshape(N, K), gc.dev_bf16(bits)
    else:
        dev = gc.dev_f32(W)
    with np.errstate(over="ignore", invalid="ignore"):
        codes, s, z = og.quantize(W, group, zeros, True)
    bad = np.isnan(s)
    assert bad.sum() == 4 + zeros
    gw = q.group_quantize(dev, group, zeros=zeros)
    assert np.array_equal(np.isnan(gw.scales.float().cpu().numpy()), bad)
    got = q.group_dequantize(gw, torch.float32).cpu().numpy().reshape(N, K // group, group)
    assert np.all(np.isnan(got[bad]))
    want = og.values(codes, s, z, group).reshape(got.shape)
    assert np.array_equal(got[~bad], want[~bad].astype(np.float32))
    Y = q.group_linear_fwd(gw, torch.ones((3, K), dtype=torch.bfloat16, device="cuda")).float().cpu().numpy()
    assert np.array_equal(np.isnan(Y), np.repeat(bad.any(1)[None], 3, 0))


def test_dequantize_any_zero_byte_and_out(q):
    import torch
    z = np.random.default_rng(0).integers(0, 256, (9, 5)).astype(np.uint8)
    codes, s, z, gw = _weight(q, 9, 160, 32, True, False, z=z)
    out = torch.full((9, 160), 7.0, device="cuda")
    assert q.group_dequantize(gw, torch.float32, out=out) is out
    want = (codes.astype(np.float32) - np.repeat(z, 32, 1)) * np.repeat(s, 32, 1)
    assert np.array_equal(out.cpu().numpy(), want)


# ---- the product ----------------------------------------------------------------------

@pytest.mark.parametrize("M", [1, 2, 4, 5, 15, 16, 17, 31, 32, 33, 48, 49, 63, 64, 65, 130])
def test_tokens(q, M):
    _check(q, M, 100, 512, 128, True, True)


@pytest.mark.parametrize("N", [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 257, 1001])
@pytest.mark.parametrize("M", [1, 20])
def test_rows(q, M, N):
    _check(q, M, N, 384, 64, False, False)


@pytest.mark.parametrize("K,group", [(32, 32), (64, 32), (64, 64), (96, 32), (96, 96), (128, 128), (160, 32), (160, 160),
                                     (192, 64), (320, 64), (384, 384), (512, 256), (1152, 128), (1376, 32),
                                     (1376, 1376), (2048, 2048), (2176, 128), (4096, 32), (11008, 64), (11008, 11008),
                                     (22016, 128)])
@pytest.mark.parametrize("M", [1, 7, 40])
@pytest.mark.parametrize("zeros,bf16", [(False, True), (True, False)])
def test_columns_and_groups(q, M, K, group, zeros, bf16):
    _check(q, M, 50, K, group, zeros, bf16)


@pytest.mark.parametrize("M,N,K,group", [(1, 11008, 4096, 128), (1, 4096, 11008, 64), (16, 12288, 4096, 128),
                                         (64, 11008, 4096, 32), (3, 1001, 1376, 32), (8, 256, 8192, 128)])
def test_layers(q, M, N, K, group):
    _check(q, M, N, K, group, True, group != 32)


# one shape for each height and width of tile that the launcher chooses (by M and N alone), and two
# lengths of rows: of whole blocks, and with a part of one
@pytest.mark.parametrize("M,N", [(1, 16400), (3, 16400), (7, 16400), (8, 500), (12, 6000), (16, 12288), (64, 4096),
                                 (32, 11008), (64, 8192), (64, 11008), (130, 4100), (1000, 250)])
@pytest.mark.parametrize("K,group,zeros,bf16", [(640, 128, True, True), (640, 64, False, False), (1280, 32, True, False),
                                                (1120, 32, True, True)])
def test_every_tile(q, M, N, K, group, zeros, bf16):
    _check(q, M, N, K, group, zeros, bf16)


def test_longest_rows(q):
    _check(q, 2, 17, 262144, 128, True, True)
    _check(q, 1, 3, 262144, 32, False, True)


def test_no_tokens(q):
    import torch
    _, _, _, gw = _weight(q, 8, 64, 32, False, True)
    assert q.group_linear_fwd(gw, torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")).shape == (0, 8)


def test_a_token_does_not_depend_on_its_batch(q):
    """Rows of a batch on the same tiles are bitwise those of the tokens alone."""
    import torch
    gw, xb, Y = _check(q, 16, 300, 1376, 32, True, True)
    X = gc.dev_bf16(xb)
    for m in range(16):
        assert torch.equal(q.group_linear_fwd(gw, X[m:m + 1])[0], Y[m])


@pytest.mark.parametrize("M,N", [(3, 70), (3, 16400), (12, 6000), (40, 70), (64, 4096), (64, 8200)])
def test_infinite_and_nan_inputs(q, M, N):
    """As the definition: only the token concerned, infinite or NaN where its products are."""
    import torch
    K, group = 512, 64
    codes, s, z, gw = _weight(q, N, K, group, True, True, seed=3)
    codes[5, 100] = z[5, 100 // group]          # a weight of zero meets the infinity
    gw.codes = torch.from_numpy(og.pack(codes)).cuda()
    rng = np.random.default_rng(1)
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[0, 100] = np.inf
    x[1, 7], x[1, 300] = np.inf, -np.inf
    x[2, 511] = np.nan
    xb = (x.view(np.uint32) >> 16).astype(np.uint16)  # truncation keeps infinities and NaN
    Y = gc.host_f32_from_bf16(q.group_linear_fwd(gw, gc.dev_bf16(xb))).reshape(M, N)
    xf = gc.f64(xb)
    with np.errstate(invalid="ignore"):
        want = xf @ og.values(codes, s, z, group).T
    assert np.isnan(want[0, 5]) and np.isinf(want[0]).sum() >= N // 2
    assert np.array_equal(np.isnan(Y), np.isnan(want))
    inf = np.isinf(want)
    assert np.array_equal(Y[inf], want[inf])
    fine = np.isfinite(want)
    _, mag = og.product(np.where(np.isfinite(xf), xf, 0), codes, s, z, group)
    assert np.all(np.abs(Y - np.where(fine, want, 0))[fine] <= _bound(want, mag, K, group)[fine])


def test_sums_that_overflow_only_with_the_offset(q):
    """31 x overflows, (code - 8) x does not: the result is finite and right."""
    import torch
    N, K, group = 40, 256, 128
    codes, s, z, gw = _weight(q, N, K, group, False, False, seed=5, s=np.full((40, 2), 2.0 ** -100, np.float32))
    x = np.random.default_rng(2).standard_normal((2, K)).astype(np.float32)
    x[1, 17] = 3.0e37
    xb = synth.to_bf16_bits(x)
    Y = gc.host_f32_from_bf16(q.group_linear_fwd(gw, gc.dev_bf16(xb))).reshape(2, N)
    want, mag = og.product(gc.f64(xb), codes, s, z, group)
    assert np.all(np.isfinite(Y)) and np.all(np.abs(Y - want) <= _bound(want, mag, K, group))


def test_scales_of_zero_infinity_and_nan(q):
    N, K, group = 20, 256, 64
    s = np.full((N, 4), 0.01, np.float32)
    s[3, 1], s[4, 2], s[5, 0] = 0.0, np.inf, np.nan
    codes, s, z, gw = _weight(q, N, K, group, True, False, s=s)
    xb = synth.to_bf16_bits(np.random.default_rng(2).standard_normal((2, K)).astype(np.float32))
    Y = gc.host_f32_from_bf16(q.group_linear_fwd(gw, gc.dev_bf16(xb))).reshape(2, N)
    bad = np.zeros(N, bool)
    bad[[4, 5]] = True
    assert not np.isfinite(Y[:, bad]).any()
    s2 = np.where(np.isfinite(s), s, 0)
    want, mag = og.product(gc.f64(xb), codes, s2, z, group)
    assert np.all(np.abs(Y - want)[:, ~bad] <= _bound(want, mag, K, group)[:, ~bad])


def test_output_guards_and_unaligned_scales(q):
    """Nothing outside Y is written; scales may start at any of their elements, zeros at any
    byte."""
    import torch
    N, K, group, M = 37, 160, 32, 5
    codes, s, z, gw = _weight(q, N, K, group, True, True)
    xb = synth.to_bf16_bits(np.random.default_rng(2).standard_normal((M, K)).astype(np.float32))
    X = gc.dev_bf16(xb)
    want = q.group_linear_fwd(gw, X)
    n = N * K // group
    for off in (1, 3):
        hold = torch.empty(n + off, dtype=torch.bfloat16, device="cuda")
        hold[off:] = gw.scales.view(-1)
        zhold = torch.empty(n + off, dtype=torch.uint8, device="cuda")
        zhold[off:] = gw.zeros.view(-1)
        moved = q.GroupWeight(gw.codes, hold[off:].view(N, -1), zhold[off:].view(N, -1), N, K, group)
        buf = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
        Y = buf[32:32 + M * N].view(M, N)
        assert q.group_linear_fwd(moved, X, Y=Y) is Y
        assert torch.equal(Y, want) and bool((buf[:32] == 7).all()) and bool((buf[32 + M * N:] == 7).all())
        assert torch.equal(q.group_dequantize(moved), q.group_dequantize(gw))
    with pytest.raises(q.QloraError) as e:   # X off 16 bytes is refused
        q.group_linear_fwd(gw, torch.zeros(M * K + 1, dtype=torch.bfloat16, device="cuda")[1:].view(M, K))
    assert e.value.status == -6


def test_codes_past_four_gib(q):
    """The last rows of a weight whose codes pass byte 2^32, and of its dequantized copy."""
    import torch
    K, group = 8192, 128
    N = (1 << 32) // (K // 2) + 24
    gen = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 256, (N * K // 2,), dtype=torch.uint8, device="cuda", generator=gen)
    scales = torch.rand((N, K // group), device="cuda", generator=gen).bfloat16()
    gw = q.GroupWeight(codes, scales, None, N, K, group)
    X = torch.randn((2, K), device="cuda", generator=gen).bfloat16()
    Y = q.group_linear_fwd(gw, X)
    for first in (0, N - 40):
        n = 40
        sub = q.GroupWeight(codes[first * K // 2:(first + n) * K // 2], scales[first:first + n], None, n, K, group)
        assert torch.equal(q.group_linear_fwd(sub, X), Y[:, first:first + n])
    out = q.group_dequantize(gw)
    assert torch.equal(out[N - 40:], q.group_dequantize(sub))
    again = q.group_quantize(out, group)
    tail = q.group_quantize(out[N - 40:].clone(), group)
    assert torch.equal(again.codes[-20 * K:], tail.codes[-20 * K:]) and torch.equal(again.scales[-40:], tail.scales)


def test_streams_and_captured_graphs(q):
    """Two streams at once; a captured graph replayed on new inputs between eager calls."""
    import torch
    codes, s, z, gw = _weight(q, 500, 1376, 32, True, True)
    X = torch.randn(8, 1376, device="cuda").bfloat16()
    X2 = torch.randn(8, 1376, device="cuda").bfloat16()
    want, want2 = q.group_linear_fwd(gw, X), q.group_linear_fwd(gw, X2)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for k in range(6):
        with torch.cuda.stream(streams[k % 2]):
            got.append((k % 2, q.group_linear_fwd(gw, (X, X2)[k % 2])))
    torch.cuda.synchronize()
    for k, y in got:
        assert torch.equal(y, (want, want2)[k])
    static = X.clone()
    Y = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.group_linear_fwd(gw, static, Y=Y)
    for k in range(4):
        static.copy_((X, X2)[k % 2])
        g.replay()
        eager = q.group_linear_fwd(gw, (X, X2)[k % 2])
        torch.cuda.synchronize()
        assert torch.equal(Y, eager) and torch.equal(eager, (want, want2)[k % 2])


def test_merged_weight_served(q):
    """A tuned NF4 layer merged, quantized with group scales and served: each step against
    the oracle's on the step's own input."""
    import torch
    N, K, r = 96, 256, 8
    W = torch.randn(N, K, device="cuda") * 0.02
    A, B = torch.randn(r, K, device="cuda").bfloat16() * 0.3, torch.randn(N, r, device="cuda").bfloat16() * 0.01
    Wm = q.lora_merge(q.quantize(W), A, B, 16.0)
    gw = q.group_quantize(Wm, 64, zeros=True)
    codes, s, z = og.quantize(gc.host_f32_from_bf16(Wm).astype(np.float32).reshape(N, K), 64, True, True)
    assert np.array_equal(gw.codes.cpu().numpy(), og.pack(codes))
    xb = synth.to_bf16_bits(np.random.default_rng(2).standard_normal((4, K)).astype(np.float32))
    want, mag = og.product(gc.f64(xb), codes, s, z, 64)
    got = gc.host_f32_from_bf16(q.group_linear_fwd(gw, gc.dev_bf16(xb))).reshape(4, N)
    assert np.all(np.abs(got - want) <= _bound(want, mag, K, 64))
