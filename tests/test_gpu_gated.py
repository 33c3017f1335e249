"""The gated projections on the GPU, forward and backward, against the float64 definition
within derived bounds (tests/drop_cases.py): the small-M path and the tiled one, odd heights
and ranks, both activations, dropout, number types; and one run of the feed-forward block
as it is trained."""

import numpy as np
import pytest

from oracle import gated as og
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


def act_error(name, x):
    """Relative error allowed to the fp32 logistic: a few 2^-24, and |z| 2^-24 through the
    exponent's product."""
    z, dz = og.argument(name, x)
    return 2.0 ** -20 * (1 + np.abs(z)), dz


def h_bound(name, Y, eY):
    """Bound of H before its rounding for [G | L] known up to eY: |act'| <= 1.13."""
    G, L = np.split(Y, 2, axis=1)
    eG, eL = np.split(eY, 2, axis=1)
    f, _ = og.act(name, G)
    rel, _ = act_error(name, np.abs(G) + eG)
    return 1.13 * eG * (np.abs(L) + eL) + np.abs(f) * eL + rel * (np.abs(f) + 1.13 * eG) * (np.abs(L) + eL)


def grad_bound(name, dH, Y, dY):
    """Bound of the bf16 [dG | dL] of the saved, exactly known [G | L]."""
    G, L = np.split(Y, 2, axis=1)
    f, _ = og.act(name, G)
    rel, dz = act_error(name, G)
    e = np.concatenate([np.abs(dH * L) * rel * (1 + np.abs(f) * dz), np.abs(dH * f) * rel], axis=1)
    return e + dc.H * (np.abs(dY) + e)


def inputs(M, K, P, r, seed):
    h = dc.linear_inputs(M, K, P, max(r, 1), 2, seed)
    h["dH"] = h.pop("dY")[:, :P].copy()
    # a weight of std 0.02 on K inputs of std 1: G reaches where the activations bend
    return h


def run(q, qw, dev, r, act, d, U=None, save=True):
    A, B = (dev["A"], dev["B"]) if r else (None, None)
    H, Y, U1 = q.gated_fwd(qw, dev["X"], A, B, ALPHA, act=act, dropout=d)
    g = q.gated_bwd(qw, dev["dH"], Y, dev["X"] if r else None, A, B, ALPHA, U1 if U is None else None, act=act,
                    dropout=d)
    return (H, Y, U1) + g


def check_all(q, qw, Wd, h, dev, M, K, P, r, act, p, d, out):
    H, Y, U, dX, dA, dB = out
    X, A, B, dH = dc.f64(h, "X", "A", "B", "dH")
    m, c = dc.mask(M, K, p, d.seed, d.offset) if d else (np.ones((M, K)), 1.0)
    rY, eY, rU, eU = dc.forward(X, Wd, A, B, ALPHA, r, 2, m, c)
    dc.check("Y", dc.bits(Y), rY, eY + dc.H * (np.abs(rY) + eY))
    if r:
        dc.check("U", dc.bits(U), rU, eU)
    rH = og.forward(rY, act)
    eH = h_bound(act, rY, eY)
    dc.check("H", dc.bits(H), rH, eH + dc.H * (np.abs(rH) + eH))
    Yd = dc.bits(Y)
    dY = og.backward(dH, Yd, act)
    want = dc.backward(dY, grad_bound(act, dH, Yd, dY), X, Wd, A, B, ALPHA, r, 2, m, c, dc.bits(U) if r else None)
    dc.check("dX", dc.bits(dX), *want["dX"])
    if r:
        dc.check("dA", dc.bits(dA), *want["dA"])
        dc.check("dB", dc.bits(dB), *want["dB"])
    else:
        assert U is None and dA is None and dB is None


# (M, K, P, r, act, p)
CASES = [
    # small-M path: one to 16 tokens, heights inside and across 8-column tiles
    (1, 64, 1, 0, "silu", 0.0), (1, 64, 8, 8, "silu", 0.0), (1, 512, 320, 16, "silu", 0.1),
    (3, 256, 101, 12, "gelu_tanh", 0.25), (5, 1024, 77, 4, "silu", 0.0), (16, 256, 256, 64, "gelu_tanh", 0.0),
    (16, 4096, 2050, 8, "silu", 0.0), (9, 2048, 515, 128, "silu", 0.1), (2, 4096, 40, 16, "silu", 0.3),
    (16, 8192, 136, 1, "silu", 0.0), (16, 8192, 136, 8, "silu", 0.1), (2, 8192, 4100, 24, "gelu_tanh", 0.1),
    # tiled path
    (17, 64, 1, 1, "silu", 0.0), (17, 128, 7, 8, "silu", 0.1), (64, 192, 128, 64, "gelu_tanh", 0.05),
    (300, 512, 320, 16, "silu", 0.1), (257, 320, 129, 0, "gelu_tanh", 0.0), (333, 320, 501, 12, "gelu_tanh", 0.25),
    (200, 256, 72, 1, "silu", 0.0), (130, 256, 136, 80, "silu", 0.1), (70, 512, 136, 128, "silu", 0.0),
    (65, 256, 1000, 20, "silu", 0.5), (530, 1024, 776, 64, "silu", 0.1),
    # every remainder of the contraction's four-step groups, with and without splits; one to
    # three blocks of 32 tokens; both parts' ranks in one and in several 64-rank tiles
    (18, 64, 2200, 8, "silu", 0.0), (31, 320, 70, 32, "silu", 0.0), (40, 448, 65, 40, "gelu_tanh", 0.0),
    (64, 704, 3000, 16, "silu", 0.0), (96, 576, 130, 96, "silu", 0.1), (129, 2112, 40, 8, "silu", 0.0),
    (20, 17408, 33, 8, "silu", 0.0),  # more than 256 steps: always split
    # forward tiles of 128 and 64 tokens whose last one has up to 32 or 64, whole and split
    (777, 512, 3000, 16, "silu", 0.1), (820, 640, 3001, 8, "silu", 0.0), (80, 512, 6000, 16, "gelu_tanh", 0.1),
    (260, 2048, 600, 8, "silu", 0.0), (140, 4096, 1000, 8, "silu", 0.1), (560, 4096, 300, 72, "silu", 0.0),
    # dX on tiles of 64 and 128 tokens, split; on the large tiles, split, with padded blocks
    (1500, 512, 1501, 12, "silu", 0.1), (4000, 320, 1001, 12, "gelu_tanh", 0.1), (300, 64, 4097, 20, "silu", 0.25),
    (100, 256, 4100, 80, "silu", 0.1),
]


@pytest.mark.parametrize("M,K,P,r,act,p", CASES)
def test_gated(q, M, K, P, r, act, p):
    import torch
    print(f"gated M={M} K={K} P={P} r={r} {act} p={p}", flush=True)
    h = inputs(M, K, P, r, seed=M + K + P)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"])
    d = q.Dropout(p, seed=31 * M + P, offset=P) if p else None
    before = {k: v.clone() for k, v in dev.items()}
    out = run(q, qw, dev, r, act, d)
    again = run(q, qw, dev, r, act, d)
    H2, none_y, none_u = q.gated_fwd(qw, dev["X"], dev["A"] if r else None, dev["B"] if r else None, ALPHA, act=act,
                                     save=False, dropout=d)
    torch.cuda.synchronize()
    assert none_y is None and none_u is None and torch.equal(H2, out[0])
    for a, b in zip(out, again):
        assert (a is None and b is None) or torch.equal(a, b), "not deterministic"
    for k in dev:
        assert torch.equal(dev[k], before[k]), f"input {k} was changed"
    check_all(q, qw, dc.weight64(qw), h, dev, M, K, P, r, act, p, d, out)


@pytest.mark.parametrize("quant,const", [(0, 1), (0, 2), (1, 0), (1, 2)])
@pytest.mark.parametrize("M", [4, 140])
def test_gated_number_types(q, M, quant, const):
    K, P, r, p = 320, 200, 16, 0.2  # five blocks a row: no row starts on a dword of constants
    h = inputs(M, K, P, r, seed=9 + quant + const)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"], quant_type=quant, const_type=const)
    d = q.Dropout(p, seed=77)
    out = run(q, qw, dev, r, "silu", d)
    check_all(q, qw, gc.host_f32_from_bf16(q.dequantize(qw)), h, dev, M, K, P, r, "silu", p, d, out)


def test_saved_y_is_the_fused_linear(q):
    """On the tiles that the horizontally fused linear runs on, [G | L] is bit for bit what it
    gives for the same weight (smaller calls take other tiles, which sum in another order)."""
    import torch
    M, K, P, r = 700, 2048, 5632, 16
    h = inputs(M, K, P, r, seed=2)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"])
    _, Y, U = q.gated_fwd(qw, dev["X"], dev["A"], dev["B"], ALPHA)
    Yf, Uf = q.linear_fwd_fused(qw, 2, dev["X"], dev["A"], dev["B"], ALPHA)
    assert torch.equal(Y, Yf) and torch.equal(U, Uf)


def test_recomputed_u_and_given_outputs(q):
    import torch
    M, K, P, r = 150, 256, 104, 8
    h = inputs(M, K, P, r, seed=6)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"])
    d = q.Dropout(0.2, seed=6)
    H, Y, U, dX, dA, dB = run(q, qw, dev, r, "silu", d)
    _, _, _, dX2, dA2, dB2 = run(q, qw, dev, r, "silu", d, U="recompute")
    assert all(torch.equal(a, b) for a, b in ((dX, dX2), (dA, dA2), (dB, dB2)))
    o = {n: torch.full_like(t, 5.0) for n, t in dict(H=H, Y=Y, U=U).items()}
    ws = [torch.zeros(q.qlora_workspace_bytes_gated(op, M, K, P, r), dtype=torch.uint8, device="cuda")
          for op in (0, 1)]
    q.gated_fwd(qw, dev["X"], dev["A"], dev["B"], ALPHA, ws=ws[0], dropout=d, **o)
    g = {n: torch.full_like(t, 5.0) for n, t in dict(dX=dX, dA=dA, dB=dB).items()}
    q.gated_bwd(qw, dev["dH"], o["Y"], dev["X"], dev["A"], dev["B"], ALPHA, o["U"], ws=ws[1], dropout=d, **g)
    for a, b in zip((o["H"], o["Y"], o["U"], g["dX"], g["dA"], g["dB"]), (H, Y, U, dX, dA, dB)):
        assert torch.equal(a, b)
    _, dA3, dB3 = q.gated_bwd(qw, dev["dH"], Y, dev["X"], dev["A"], dev["B"], ALPHA, U, need_dx=False, dropout=d)
    assert torch.equal(dA, dA3) and torch.equal(dB, dB3)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_extreme_gates(q, act):
    """Saved gates from the smallest to the largest bf16 values, zeros and both signs: the
    gradients stay finite and within their bounds (no 0 * inf in the activations)."""
    K, P, M = 64, 64, 20
    rng = np.random.default_rng(0)
    mags = np.array([0.0, 1e-38, 1e-20, 1e-3, 0.5, 1.0, 5.0, 20.0, 89.0, 200.0, 1e4, 1e10, 1e19, 1e25, 1e30])
    G = rng.choice(mags, (M, P)) * rng.choice([-1.0, 1.0], (M, P))
    Yh = np.concatenate([G, rng.standard_normal((M, P))], axis=1).astype(np.float32)
    # dH small enough that dH L act' stays in range
    dHh = (rng.standard_normal((M, P)) * 1e-3).astype(np.float32)
    import synth
    h = inputs(M, K, P, 0, seed=1)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    Yb, dHb = synth.to_bf16_bits(Yh), synth.to_bf16_bits(dHh)
    qw = q.quantize(dev["W"])
    dX, _, _ = q.gated_bwd(qw, gc.dev_bf16(dHb), gc.dev_bf16(Yb), act=act)
    Yd, dH = gc.f64(Yb), gc.f64(dHb)
    with np.errstate(over="ignore", invalid="ignore"):
        dY = og.backward(dH, Yd, act)
        f, df = og.act(act, Yd[:, :P])
    # where the float64 oracle itself overflows (x^3 past 1e308 does not occur here)
    assert np.all(np.isfinite(dY))
    e = grad_bound(act, dH, Yd, dY)
    e = np.where(np.isfinite(e), e, dc.H * np.abs(dY))  # past |z| = 2^20 the logistic is 0 or 1 exactly
    big = np.abs(Yd[:, :P]) > 1e4
    e[:, :P][big] = dc.H * np.abs(dY[:, :P][big]) + 1e-30
    e[:, P:][big] = dc.H * np.abs(dY[:, P:][big]) * 2 + 1e-30
    Wd = dc.weight64(qw)
    want = dc.backward(dY, e, np.zeros((M, K)), Wd, None, None, ALPHA, 0, 2, np.ones((M, K)), 1.0, None)["dX"]
    dc.check("dX", dc.bits(dX), *want)


@pytest.mark.parametrize("M", [7, 200])
def test_captured_graph(q, M):
    """Forward and backward captured once, replayed with new masks and new inputs between
    eager work, against the eager calls."""
    import torch
    K, P, r = 512, 320, 16
    h = inputs(M, K, P, r, seed=12)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"])
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")
    d = q.Dropout(0.25, seed=4, offset=100, counter=counter)
    ws = [torch.zeros(q.qlora_workspace_bytes_gated(op, M, K, P, r), dtype=torch.uint8, device="cuda")
          for op in (0, 1)]
    mk = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    o = dict(H=mk(M, P), Y=mk(M, 2 * P), U=mk(M, 2 * r))
    g = dict(dX=mk(M, K), dA=mk(2 * r, K), dB=mk(2 * P, r))

    def step(drop, o, g, w):
        q.gated_fwd(qw, dev["X"], dev["A"], dev["B"], ALPHA, ws=w[0], dropout=drop, **o)
        q.gated_bwd(qw, dev["dH"], o["Y"], dev["X"], dev["A"], dev["B"], ALPHA, o["U"], ws=w[1], dropout=drop, **g)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(d, o, g, ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(d, o, g, ws)
            counter.add_(1)
    torch.cuda.synchronize()
    counter.zero_()
    for i in range(4):
        dev["X"].copy_(gc.dev_bf16(inputs(M, K, P, r, seed=40 + i)["X"]))
        for t in list(o.values()) + list(g.values()):
            t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        o2, g2 = ({k: torch.empty_like(v) for k, v in x.items()} for x in (o, g))
        step(q.Dropout(0.25, seed=4, offset=100 + i), o2, g2, [torch.zeros_like(w) for w in ws])
        torch.cuda.synchronize()
        for a, b in ((o, o2), (g, g2)):
            for k in a:
                assert torch.equal(a[k], b[k]), (i, k)


def test_small_m_workspace_is_left_ready(q):
    """The small-M path leaves the counters at zero: calls of other shapes and of the other
    operators share one workspace, and nothing behind the outputs' rows is touched."""
    import torch
    K, P, r = 512, 264, 8
    h = inputs(16, K, P, r, seed=3)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"])
    n = max(q.qlora_workspace_bytes_gated(0, m, K, P, r) for m in (1, 5, 16))
    n = max(n, q.qlora_workspace_bytes_fused(0, 16, K, 2 * P, r, 1), q.qlora_workspace_bytes_dropout(0, 16, K, 2 * P, r, 1))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    want = {}
    d = q.Dropout(0.3, seed=1)
    for rep in range(3):
        for m in (1, 5, 16):
            X = dev["X"][:m].contiguous()
            big = torch.full((m + 3, P), 9.0, dtype=torch.bfloat16, device="cuda")
            H, Y, U = q.gated_fwd(qw, X, dev["A"], dev["B"], ALPHA, ws=ws, H=big[:m], dropout=d if rep == 1 else None)
            L, _ = q.linear_fwd(qw, X, dev["A"][:r].contiguous(), dev["B"], ALPHA, ws=ws, dropout=d)
            torch.cuda.synchronize()
            assert bool((big[m:] == 9.0).all())
            assert int(ws[:65792].count_nonzero()) == 0
            key = (m, rep == 1)
            if key in want:
                assert all(torch.equal(a, b) for a, b in zip(want[key], (H, Y, U, L)))
            want[key] = tuple(t.clone() for t in (H, Y, U, L))


@pytest.mark.parametrize("M", [3, 40, 300])
def test_constants_at_any_address(q, M):
    """The 8-bit block constants need no alignment: the same results from every start."""
    import torch
    K, P, r = 320, 72, 8
    h = inputs(M, K, P, r, seed=5)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"])
    d = q.Dropout(0.2, seed=5)
    want = run(q, qw, dev, r, "silu", d)
    n = qw.absmax_q.numel()
    for off in (1, 2, 3):
        buf = torch.full((n + 8,), -77, dtype=torch.int8, device="cuda")
        buf[off:off + n] = qw.absmax_q
        q2 = q.NF4Weight(qw.codes, buf[off:off + n], qw.dq_scale, qw.dq_offset, qw.n_rows, qw.n_cols)
        for a, b in zip(want, run(q, q2, dev, r, "silu", d)):
            assert torch.equal(a, b), off


@pytest.mark.parametrize("M,K,P,r", [(5, 256, 72, 8), (40, 256, 71, 12), (300, 512, 129, 16)])
def test_nothing_outside_the_outputs_is_written(q, M, K, P, r):
    """Rows behind the last one of every output, and the bytes behind a workspace of exactly
    the documented size, stay as they were."""
    import torch
    h = inputs(M, K, P, r, seed=15)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"])
    d = q.Dropout(0.2, seed=5)
    mk = lambda rows, cols: torch.full((rows + 5, cols), 9.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    whole = dict(H=mk(M, P), Y=mk(M, 2 * P), U=mk(M, 2 * r), dX=mk(M, K), dA=mk(2 * r, K), dB=mk(2 * P, r))
    rows = dict(H=M, Y=M, U=M, dX=M, dA=2 * r, dB=2 * P)
    o = {k: whole[k][:rows[k]] for k in whole}
    sizes = [q.qlora_workspace_bytes_gated(op, M, K, P, r) for op in (0, 1)]
    bufs = [torch.zeros(n + 4096, dtype=torch.uint8, device="cuda") for n in sizes]
    for b, n in zip(bufs, sizes):
        b[n:] = 0xA5
    q.gated_fwd(qw, dev["X"], dev["A"], dev["B"], ALPHA, dropout=d, ws=bufs[0][:sizes[0]], H=o["H"], Y=o["Y"], U=o["U"])
    q.gated_bwd(qw, dev["dH"], o["Y"], dev["X"], dev["A"], dev["B"], ALPHA, o["U"], dropout=d, ws=bufs[1][:sizes[1]],
                dX=o["dX"], dA=o["dA"], dB=o["dB"])
    torch.cuda.synchronize()
    for k, t in whole.items():
        assert bool((t[rows[k]:] == 9.0).all()), k
        assert bool(torch.isfinite(t[:rows[k]]).all()), k
    for b, n in zip(bufs, sizes):
        assert bool((b[n:] == 0xA5).all())


SHAPES = [(5, 256, 72, 8), (40, 256, 71, 12), (300, 512, 129, 16), (700, 512, 5632, 16)]


@pytest.mark.parametrize("M,K,P,r", SHAPES)
def test_workspace_contents_do_not_matter(q, M, K, P, r):
    """A workspace of NaN patterns behind its header gives what a zeroed one gives."""
    import torch
    h = inputs(M, K, P, r, seed=25)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"])
    d = q.Dropout(0.2, seed=6)
    outs = []
    for fill in (0, 0xFF):
        ws = [torch.full((q.qlora_workspace_bytes_gated(op, M, K, P, r),), fill, dtype=torch.uint8, device="cuda")
              for op in (0, 1)]
        for w in ws:
            w[:65792] = 0
        H, Y, U = q.gated_fwd(qw, dev["X"], dev["A"], dev["B"], ALPHA, dropout=d, ws=ws[0])
        outs.append((H, Y, U) + q.gated_bwd(qw, dev["dH"], Y, dev["X"], dev["A"], dev["B"], ALPHA, U, dropout=d,
                                            ws=ws[1]))
    for a, b in zip(*outs):
        assert torch.equal(a, b) and bool(torch.isfinite(a).all())


@pytest.mark.parametrize("M,K,P,r", SHAPES)
def test_nan_stays_in_its_row_and_out_of_dropped_places(q, M, K, P, r):
    import torch
    h = inputs(M, K, P, r, seed=26)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"])
    d = q.Dropout(0.3, seed=8)
    H, Y, U, dX, dA, dB = run(q, qw, dev, r, "silu", d)
    m, _ = dc.mask(M, K, 0.3, 8, 0)
    i, j = M // 2, M - 1
    rest = [n for n in range(M) if n not in (i, j)]
    kept, dropped = int(np.flatnonzero(m[i])[0]), int(np.flatnonzero(m[j] == 0)[-1])
    X = dev["X"].clone()
    X[j, dropped] = float("nan")
    # the adapter does not see a dropped element, whatever it is
    H2, Y2, U2 = q.gated_fwd(qw, X, dev["A"], dev["B"], ALPHA, dropout=d)
    assert torch.equal(U2, U) and torch.equal(H2[:j], H[:j]) and torch.equal(Y2[:j], Y[:j])
    assert bool(torch.isnan(Y2[j]).all())
    for a, b in zip(q.gated_bwd(qw, dev["dH"], Y, X, dev["A"], dev["B"], ALPHA, U, dropout=d), (dX, dA, dB)):
        assert torch.equal(a, b)
    X[i, kept] = float("inf")
    H2, Y2, U2 = q.gated_fwd(qw, X, dev["A"], dev["B"], ALPHA, dropout=d)
    for a, b in ((H2, H), (Y2, Y), (U2, U)):
        assert torch.equal(a[rest], b[rest])
    assert not bool(torch.isfinite(U2[i]).any())
    dH = dev["dH"].clone()
    dH[i, P // 2] = float("nan")
    dX2, _, _ = q.gated_bwd(qw, dH, Y, dev["X"], dev["A"], dev["B"], ALPHA, U, dropout=d)
    rest = [n for n in range(M) if n != i]
    assert torch.equal(dX2[rest], dX[rest]) and bool(torch.isnan(dX2[i]).all())


def test_tensors_near_four_gib(q):
    """[G | L] and its gradient of almost 4 GiB: byte offsets past 31 bits.  The first and the
    last rows against the definition."""
    import torch
    M, K, P, r = 48000, 64, 22016, 8
    h = inputs(16, K, P, r, seed=77)
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    qw = q.quantize(dev["W"])
    X = dev["X"].repeat(M // 16, 1)
    dH = dev["dH"].repeat(M // 16, 1)
    d = q.Dropout(0.25, seed=3)
    H, Y, U = q.gated_fwd(qw, X, dev["A"], dev["B"], ALPHA, dropout=d)
    dX, dA, dB = q.gated_bwd(qw, dH, Y, X, dev["A"], dev["B"], ALPHA, U, dropout=d)
    torch.cuda.synchronize()
    Wd = dc.weight64(qw)
    Xf, A, B, dHf = dc.f64(h, "X", "A", "B", "dH")
    from oracle import dropout as od
    for first in (0, M - 16):
        m = od.keep((16, K), 0.25, 3, 0, first=first * K).astype(np.float64)
        c = od.scale(0.25)
        rY, eY, rU, eU = dc.forward(Xf, Wd, A, B, ALPHA, r, 2, m, c)
        sl = slice(first, first + 16)
        dc.check("Y", dc.bits(Y[sl]), rY, eY + dc.H * (np.abs(rY) + eY))
        rH = og.forward(rY, "silu")
        eH = h_bound("silu", rY, eY)
        dc.check("H", dc.bits(H[sl]), rH, eH + dc.H * (np.abs(rH) + eH))
        Yd = dc.bits(Y[sl])
        dY = og.backward(dHf, Yd, "silu")
        want = dc.backward(dY, grad_bound("silu", dHf, Yd, dY), Xf, Wd, A, B, ALPHA, r, 2, m, c, dc.bits(U[sl]))
        dc.check("dX", dc.bits(dX[sl]), *want["dX"])
    assert bool(torch.isfinite(dA).all()) and bool(torch.isfinite(dB).all())


def test_feed_forward_block_training_step(q):
    """The block as it is trained: gated projections and the down linear, both with dropout,
    forward, backward and the optimizer, against the float64 chain on the same masks; every
    bf16 tensor handed on is taken from the device, so that each call's own bound applies."""
    import torch
    M, K, P, r, p = 180, 256, 192, 16, 0.1
    h = inputs(M, K, P, r, seed=50)
    hd = dc.linear_inputs(M, P, K, r, 1, seed=51)  # down: P -> K
    dev = {k: gc.dev_bf16(v) for k, v in h.items()}
    dd = {k: gc.dev_bf16(v) for k, v in hd.items()}
    qg, qd = q.quantize(dev["W"]), q.quantize(dd["W"])
    d1, d2 = q.Dropout(p, seed=8, offset=0), q.Dropout(p, seed=8, offset=1)
    H, Y, U = q.gated_fwd(qg, dev["X"], dev["A"], dev["B"], ALPHA, dropout=d1)
    Z, Ud = q.linear_fwd(qd, H, dd["A"], dd["B"], ALPHA, dropout=d2)
    dH, dAd, dBd = q.linear_bwd(qd, dd["dY"], H, dd["A"], dd["B"], ALPHA, Ud, dropout=d2)
    dX, dA, dB = q.gated_bwd(qg, dH, Y, dev["X"], dev["A"], dev["B"], ALPHA, U, dropout=d1)
    params = []
    for t, g in ((dev["A"], dA), (dev["B"], dB), (dd["A"], dAd), (dd["B"], dBd)):
        w, m, v = t.float(), torch.zeros_like(t, dtype=torch.float32), torch.zeros_like(t, dtype=torch.float32)
        q.adamw_step(w, g, m, v, 1, 1e-3, param_bf16=t)
        params.append((w, g))
    torch.cuda.synchronize()
    check_all(q, qg, dc.weight64(qg), {**h, "dH": gc.host_bits(dH)}, dev, M, K, P, r, "silu", p, d1,
              (H, Y, U, dX, dA, dB))
    Xd = dc.bits(H)
    A, B, dY = dc.f64(hd, "A", "B", "dY")
    Wd = dc.weight64(qd)
    m, c = dc.mask(M, P, p, 8, 1)
    rZ, eZ, rU, eU = dc.forward(Xd, Wd, A, B, ALPHA, r, 1, m, c)
    dc.check("Z", dc.bits(Z), rZ, eZ + dc.H * (np.abs(rZ) + eZ))
    want = dc.backward(dY, np.zeros_like(dY), Xd, Wd, A, B, ALPHA, r, 1, m, c, dc.bits(Ud))
    for name, got in (("dX", dH), ("dA", dAd), ("dB", dBd)):
        dc.check("down " + name, dc.bits(got), *want[name])
    for w, g in params:  # Adam's first step moves every parameter of nonzero gradient by lr
        assert torch.isfinite(w).all() and torch.isfinite(g).all()
