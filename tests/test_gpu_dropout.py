"""Dropout on the GPU: the elementwise operator bit for bit, and the QLoRA linear with
dropout on the adapter's input against the float64 definition within derived bounds
(tests/drop_cases.py), forward and backward, over aligned and odd shapes, ranks, parts and
number types; the counter on the device, captured graphs, streams, determinism."""

import numpy as np
import pytest

import synth
from oracle import dropout as od
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


# ---- the operator by itself -----------------------------------------------------------

@pytest.mark.parametrize("n", [1, 7, 8, 9, 64, 1003, 70001])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1 - 2.0 ** -16])
def test_dropout_bits(q, n, p):
    import torch
    print(f"dropout n={n} p={p}", flush=True)
    rng = np.random.default_rng(n)
    x = rng.standard_normal(n).astype(np.float32)
    d = q.Dropout(p, seed=0x123456789ABCDEF0 + n, offset=(1 << 40) + 5)
    m, c = od.keep((n,), p, d.seed, d.offset), np.float32(od.scale(p))
    got = q.dropout(torch.from_numpy(x).cuda(), d).cpu().numpy()
    want = np.where(m, x * c, np.float32(0.0)).astype(np.float32)
    assert np.array_equal(got.view(np.uint32) & 0x7FFFFFFF if p == 0 else got.view(np.uint32),
                          want.view(np.uint32) & 0x7FFFFFFF if p == 0 else want.view(np.uint32))
    b = synth.to_bf16_bits(x)
    xb = gc.dev_bf16(b)
    want_b = np.where(m, synth.to_bf16_bits(synth.bf16_bits_to_f32(b) * c), np.uint16(0))
    assert np.array_equal(gc.host_bits(q.dropout(xb, d)), want_b)
    q.dropout(xb, d, out=xb)  # in place
    assert np.array_equal(gc.host_bits(xb), want_b)


def test_dropout_empty_and_special_values(q):
    import torch
    d = q.Dropout(0.5, seed=3)
    assert q.dropout(torch.empty(0, 8, device="cuda"), d).shape == (0, 8)
    x = torch.full((4096,), float("nan"), device="cuda")
    y = q.dropout(x, d).cpu().numpy()
    m = od.keep((4096,), 0.5, 3, 0)
    assert np.all(y[~m] == 0.0) and np.all(np.isnan(y[m]))


def test_dropout_past_four_gib(q):
    """A bf16 tensor of more than 4 GiB, in place: the mask around byte 2^32 and at the end."""
    import torch
    n = (1 << 31) + 12345
    d = q.Dropout(0.5, seed=3, offset=8)
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    q.dropout(x, d, out=x)
    for first in (0, (1 << 31) - 4096, n - 9000):
        k = min(8192, n - first)
        m = od.keep((k,), 0.5, 3, 8, first=first)
        assert np.array_equal(x[first:first + k].float().cpu().numpy(), np.where(m, 2.0, 0.0))


def test_counter_is_added_on_the_device(q):
    import torch
    x = torch.ones(1000, device="cuda")
    for v, off in ((0, 7), (5, 7), (-1, 7), (2 ** 62, 2 ** 63 + 2 ** 62)):
        d = q.Dropout(0.5, seed=11, offset=off, counter=torch.tensor([v], device="cuda"))
        m = od.keep((1000,), 0.5, 11, (off + v) % (1 << 64))
        assert np.array_equal(q.dropout(x, d).cpu().numpy() != 0, m)


# ---- the linear ------------------------------------------------------------------------

def _run(q, qw, dev, parts, d, U=None, need_dx=True):
    A, B = dev["A"], dev["B"]
    if parts > 1:
        Y, U1 = q.linear_fwd_fused(qw, parts, dev["X"], A, B, ALPHA, dropout=d)
        g = q.linear_bwd_fused(qw, parts, dev["dY"], dev["X"], A, B, ALPHA, U1 if U is None else None,
                               need_dx=need_dx, dropout=d)
    else:
        Y, U1 = q.linear_fwd(qw, dev["X"], A, B, ALPHA, dropout=d)
        g = q.linear_bwd(qw, dev["dY"], dev["X"], A, B, ALPHA, U1 if U is None else None, need_dx=need_dx, dropout=d)
    return (Y, U1) + g


# (M, K, rows of one part, r, parts, p)
CASES = [
    (1, 64, 64, 8, 1, 0.1), (1, 512, 320, 16, 1, 0.5), (16, 256, 256, 4, 1, 0.25), (17, 128, 40, 8, 1, 0.1),
    (64, 192, 256, 64, 1, 0.05), (300, 512, 320, 16, 1, 0.1), (257, 1024, 520, 32, 1, 0.1),
    (333, 320, 264, 12, 1, 0.25),     # rank padded to 16
    (200, 256, 72, 1, 1, 0.3),        # rank 1
    (130, 256, 101, 20, 1, 0.1),      # odd height: dY padded; rank padded to 24
    (90, 256, 100, 80, 1, 0.1),       # rank steps from memory (past 64 ranks), padded dY
    (70, 512, 136, 256, 1, 0.1),      # the largest rank
    (300, 320, 256, 16, 3, 0.1), (65, 256, 256, 12, 2, 0.5), (33, 192, 256, 8, 4, 0.1), (5, 256, 512, 64, 2, 0.1),
    (530, 2048, 776, 64, 1, 0.1),     # several workgroups of every kind
    (20, 64, 1000, 8, 1, 0.1), (40, 704, 130, 40, 1, 0.1), (100, 320, 513, 72, 1, 0.1),
    (50, 448, 512, 72, 3, 0.1),       # parts of stacked ranks that straddle 64-rank tiles
    # dX on tiles of 128 tokens, whole and split; on the large tiles, split
    (8200, 512, 520, 16, 1, 0.1), (4000, 320, 2000, 72, 1, 0.2), (520, 64, 8195, 20, 1, 0.1), (300, 64, 2048, 72, 2, 0.1),
]


@pytest.mark.parametrize("M,K,Np,r,parts,p", CASES)
def test_linear_dropout(q, M, K, Np, r, parts, p):
    import torch
    print(f"linear dropout M={M} K={K} Np={Np} r={r} parts={parts} p={p}", flush=True)
    h = dc.linear_inputs(M, K, Np, r, parts, seed=M + K + r)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"])
    d = q.Dropout(p, seed=991 * M + 1, offset=r)
    before = {k: v.clone() for k, v in dev.items()}
    Y, U, dX, dA, dB = _run(q, qw, dev, parts, d)
    again = _run(q, qw, dev, parts, d)
    _, U2, dX2, dA2, dB2 = _run(q, qw, dev, parts, d, U="recompute")
    torch.cuda.synchronize()
    for a, b in zip((Y, U, dX, dA, dB), again):
        assert torch.equal(a, b), "not deterministic"
    for a, b in ((U, U2), (dX, dX2), (dA, dA2), (dB, dB2)):
        assert torch.equal(a, b), "recomputing U changed the result"
    for k in dev:
        assert torch.equal(dev[k], before[k]), f"input {k} was changed"
    X, A, B, dY = dc.f64(h, "X", "A", "B", "dY")
    Wd = dc.weight64(qw)
    m, c = dc.mask(M, K, p, d.seed, d.offset)
    rY, eY, rU, eU = dc.forward(X, Wd, A, B, ALPHA, r, parts, m, c)
    dc.check("Y", dc.bits(Y), rY, eY + dc.H * (np.abs(rY) + eY))
    dc.check("U", dc.bits(U), rU, eU)
    want = dc.backward(dY, np.zeros_like(dY), X, Wd, A, B, ALPHA, r, parts, m, c, dc.bits(U))
    for name, got in (("dX", dX), ("dA", dA), ("dB", dB)):
        dc.check(name, dc.bits(got), *want[name])


@pytest.mark.parametrize("quant,const", [(0, 1), (0, 2), (1, 0), (1, 2)])
@pytest.mark.parametrize("M", [6, 150])
def test_linear_dropout_number_types(q, M, quant, const):
    """Other level tables and block constants: against the same operator on the same stored
    weight, the dequantized weight as the reference's W'."""
    K, N, r, p = 320, 200, 16, 0.2
    print(f"types {quant} {const}", flush=True)
    h = dc.linear_inputs(M, K, N, r, 1, seed=5 + quant + const)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"], quant_type=quant, const_type=const)
    Wd = gc.host_f32_from_bf16(q.dequantize(qw))
    d = q.Dropout(p, seed=77)
    Y, U, dX, dA, dB = _run(q, qw, dev, 1, d)
    X, A, B, dY = dc.f64(h, "X", "A", "B", "dY")
    m, c = dc.mask(M, K, p, d.seed, d.offset)
    rY, eY, _, _ = dc.forward(X, Wd, A, B, ALPHA, r, 1, m, c)
    dc.check("Y", dc.bits(Y), rY, eY + dc.H * (np.abs(rY) + eY))
    want = dc.backward(dY, np.zeros_like(dY), X, Wd, A, B, ALPHA, r, 1, m, c, dc.bits(U))
    for name, got in (("dX", dX), ("dA", dA), ("dB", dB)):
        dc.check(name, dc.bits(got), *want[name])


def test_no_dropout_is_the_plain_call(q):
    """p = 0 and no adapter give the calls without dropout bit for bit."""
    import torch
    h = dc.linear_inputs(100, 256, 320, 16, 1, seed=3)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"])
    a = _run(q, qw, dev, 1, q.Dropout(0.0, seed=5))
    b = _run(q, qw, dev, 1, None)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    Y, U = q.linear_fwd(qw, dev["X"], dropout=q.Dropout(0.5))
    assert U is None and torch.equal(Y, q.linear_fwd(qw, dev["X"])[0])


def test_without_dx(q):
    import torch
    h = dc.linear_inputs(100, 256, 320, 12, 1, seed=4)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"])
    d = q.Dropout(0.3, seed=5)
    _, _, _, dA, dB = _run(q, qw, dev, 1, d)
    _, _, none, dA2, dB2 = _run(q, qw, dev, 1, d, need_dx=False)
    assert none is None and torch.equal(dA, dA2) and torch.equal(dB, dB2)


def test_row_invariance(q):
    """A row's results depend on its own index alone: the first rows of a longer batch give
    the shorter batch's U (the sums over K are split by the batch, so within rounding)."""
    h = dc.linear_inputs(300, 512, 256, 16, 1, seed=8)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"])
    d = q.Dropout(0.5, seed=9)
    _, U = q.linear_fwd(qw, dev["X"], dev["A"], dev["B"], ALPHA, dropout=d)
    _, u = q.linear_fwd(qw, dev["X"][:70].contiguous(), dev["A"], dev["B"], ALPHA, dropout=d)
    X, A = dc.f64(h, "X", "A")
    m, c = dc.mask(300, 512, 0.5, 9, 0)
    _, eU = dc.down(X, A, ALPHA, 16, m, c)
    assert np.all(np.abs(dc.bits(U)[:70] - dc.bits(u)) <= 2 * eU[:70])


def test_captured_graph_draws_new_masks(q):
    """A training call captured once and replayed with an advancing device counter equals the
    eager call of the same counter value on every replay, on a side stream, with eager work
    and synchronizations in between."""
    import torch
    M, K, N, r = 200, 512, 320, 16
    h = dc.linear_inputs(M, K, N, r, 1, seed=21)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"])
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")
    d = q.Dropout(0.25, seed=4, offset=100, counter=counter)
    ws = [torch.zeros(q.qlora_workspace_bytes_dropout(op, M, K, N, r, 1), dtype=torch.uint8, device="cuda")
          for op in (0, 1)]
    out = {"Y": torch.empty(M, N, dtype=torch.bfloat16, device="cuda"),
           "U": torch.empty(M, r, dtype=torch.bfloat16, device="cuda"), "dX": torch.empty_like(dev["X"]),
           "dA": torch.empty_like(dev["A"]), "dB": torch.empty_like(dev["B"])}

    def step(drop, o, w):
        q.linear_fwd(qw, dev["X"], dev["A"], dev["B"], ALPHA, Y=o["Y"], U=o["U"], ws=w[0], dropout=drop)
        q.linear_bwd(qw, dev["dY"], dev["X"], dev["A"], dev["B"], ALPHA, o["U"], dX=o["dX"], dA=o["dA"], dB=o["dB"],
                     ws=w[1], dropout=drop)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(d, out, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step(d, out, ws)
            counter.add_(1)
    torch.cuda.synchronize()
    counter.zero_()
    seen = []
    for i in range(4):
        for t in out.values():
            t.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in out.items()}
        want = {k: torch.empty_like(v) for k, v in out.items()}
        step(q.Dropout(0.25, seed=4, offset=100 + i), want, [w.clone() for w in ws])
        torch.cuda.synchronize()
        for k in out:
            assert torch.equal(got[k], want[k]), (i, k)
        seen.append(got["U"])
    assert not torch.equal(seen[0], seen[1])
    assert int(counter.item()) == 4


def test_nothing_outside_the_outputs_is_written(q):
    """Rows behind every output's last one, and the bytes behind a workspace of exactly the
    documented size, stay as they were (aligned and padded rank and height)."""
    import torch
    for M, K, N, r, parts in ((5, 256, 72, 8, 1), (70, 256, 101, 12, 1), (300, 512, 512, 16, 2)):
        h = dc.linear_inputs(M, K, N // parts, r, parts, seed=15)
        dev = {k: gc.dev_bf16(v) for k, v in h.items()}
        qw = q.quantize(dev["W"])
        d = q.Dropout(0.2, seed=5)
        rows = dict(Y=M, U=M, dX=M, dA=parts * r, dB=N)
        cols = dict(Y=N, U=parts * r, dX=K, dA=K, dB=r)
        whole = {k: torch.full((rows[k] + 5, cols[k]), 9.0, dtype=torch.bfloat16, device="cuda") for k in rows}
        o = {k: whole[k][:rows[k]] for k in whole}
        sizes = [q.qlora_workspace_bytes_dropout(op, M, K, N, r, parts) for op in (0, 1)]
        bufs = [torch.zeros(n + 4096, dtype=torch.uint8, device="cuda") for n in sizes]
        for b, n in zip(bufs, sizes):
            b[n:] = 0xA5
        q.linear_fwd_fused(qw, parts, dev["X"], dev["A"], dev["B"], ALPHA, Y=o["Y"], U=o["U"],
                           ws=bufs[0][:sizes[0]], dropout=d)
        q.linear_bwd_fused(qw, parts, dev["dY"], dev["X"], dev["A"], dev["B"], ALPHA, o["U"], dX=o["dX"], dA=o["dA"],
                           dB=o["dB"], ws=bufs[1][:sizes[1]], dropout=d)
        torch.cuda.synchronize()
        for k, t in whole.items():
            assert bool((t[rows[k]:] == 9.0).all()), (M, k)
            assert bool(torch.isfinite(t[:rows[k]]).all()), (M, k)
        for b, n in zip(bufs, sizes):
            assert bool((b[n:] == 0xA5).all()), M


def test_tensors_near_four_gib(q):
    """X and dX of almost 4 GiB: mask indexes and byte offsets past 31 bits.  The first and
    the last rows against the definition."""
    import torch
    K, N, r, parts, p = 8192, 256, 8, 1, 0.25
    M = 262128  # 16 rows short of 2^32 bytes
    h = dc.linear_inputs(16, K, N, r, parts, seed=78)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"])
    X = dev["X"].repeat(M // 16, 1)
    dY = dev["dY"].repeat(M // 16, 1)
    d = q.Dropout(p, seed=4)
    Y, U = q.linear_fwd(qw, X, dev["A"], dev["B"], ALPHA, dropout=d)
    dX, dA, dB = q.linear_bwd(qw, dY, X, dev["A"], dev["B"], ALPHA, U, dropout=d)
    torch.cuda.synchronize()
    Wd = dc.weight64(qw)
    Xf, A, B, dYf = dc.f64(h, "X", "A", "B", "dY")
    c = od.scale(p)
    for first in (0, M - 16):
        m = od.keep((16, K), p, 4, 0, first=first * K).astype(np.float64)
        rY, eY, rU, eU = dc.forward(Xf, Wd, A, B, ALPHA, r, parts, m, c)
        sl = slice(first, first + 16)
        dc.check("Y", dc.bits(Y[sl]), rY, eY + dc.H * (np.abs(rY) + eY))
        dc.check("U", dc.bits(U[sl]), rU, eU)
        want = dc.backward(dYf, np.zeros_like(dYf), Xf, Wd, A, B, ALPHA, r, parts, m, c, dc.bits(U[sl]))
        dc.check("dX", dc.bits(dX[sl]), *want["dX"])
    assert bool(torch.isfinite(dA).all()) and bool(torch.isfinite(dB).all())
    # one row more than 2^32 - 16 bytes hold is refused before anything runs
    big = torch.empty((1 << 18, K), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(Exception, match="32-bit"):
        q.linear_fwd(qw, big, dev["A"], dev["B"], ALPHA, dropout=d)


def test_two_streams(q):
    """Two calls at once on two streams with a workspace each."""
    import torch
    M, K, N, r = 500, 1024, 512, 32
    h = dc.linear_inputs(M, K, N, r, 1, seed=31)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"])
    ds = [q.Dropout(0.1, seed=1), q.Dropout(0.4, seed=2)]
    want = [_run(q, qw, dev, 1, d) for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    got = [None, None]
    for _ in range(3):
        for i, (s, d) in enumerate(zip(streams, ds)):
            with torch.cuda.stream(s):
                got[i] = _run(q, qw, dev, 1, d)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
