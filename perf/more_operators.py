"""Measured cases of what stands around a layer's query, key and value projections when a
tuned model is served and trained on: weights in 4 bits with one scale for each group of
consecutive elements of a row (made from a bf16 or fp32 weight, multiplied with few
tokens), and the norm of each query and key head with the position rotation in the same
pass, forward and backward.

``run`` computes a case in plain torch operations where ``own`` is false and through the
package's public calls where it is true; ``exact`` evaluates the definitions in 64 bits.

Definitions
    group     g consecutive elements of a row share a scale s (and a zero z); RN rounds to
              fp32, ST to the scales' type
              without zeros: s = ST(RN(max |w| RN(1 / 7))), z = 8
              with zeros:    lo = min(w, 0), hi = max(w, 0), s = ST(RN(RN(hi - lo) RN(1 / 15))),
                             z = clamp(rint(RN(-lo RN(1 / s))), 0, 15)
              code = clamp(rint(RN(w RN(1 / s))) + z, 0, 15); s below 2^-126 counts as 0 and
              1 / s as 0 then; a code stands for (code - z) s
    matvec    Y = X W^T with W's codes as above
    qk        rows of q heads, k heads and v heads, each of d elements; for q and k heads
              x = row's head, n = x / sqrt(mean x^2 + eps) * w (without a norm: n = x), and
              pair (a, b) of the first `rot` elements turns by t = position * inv_freq[i]:
              (a cos t - b sin t, b cos t + a sin t); pair i is (i, i + rot / 2), or
              interleaved (2 i, 2 i + 1)
    its grad  the gradients of the rows and of both w; the v heads' gradient is passed on
"""

import math

import torch

own = False

EPS = 1e-6
TINY = 2.0 ** -126
PER_7, PER_15 = (float(torch.tensor(1.0) / n) for n in (7, 15))  # in fp32
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---- cases ---------------------------------------------------------------------------

def _named(name, c):
    return {"name": name, **c} if name else c


def _matvec(name, M, K, N, group, zeros, scale="bf16"):
    return _named(name, {"op": "matvec", "M": M, "K": K, "N": N, "group": group, "zeros": zeros, "scale": scale})


def _round4(name, N, K, group, zeros, scale="bf16", dtype="bf16"):
    return _named(name, {"op": "round4", "N": N, "K": K, "group": group, "zeros": zeros, "scale": scale, "dtype": dtype})


def _qk(name, op, M, heads, kv, dim, rot, norm, interleaved=False, dtype="bf16", far=4096):
    return _named(name, {"op": op, "M": M, "heads": heads, "kv": kv, "dim": dim, "rot": rot, "norm": norm,
                         "interleaved": interleaved, "dtype": dtype, "far": far})


def listed():
    return [
        # one token through the gate projection while text is generated
        _matvec("matvec_1_up", 1, 4096, 11008, 128, False),
        # the same token through the down projection, finer groups with zeros
        _matvec("matvec_1_down", 1, 11008, 4096, 64, True),
        # query, key and value stacked, four sequences
        _matvec("matvec_4_qkv", 4, 4096, 12288, 128, True),
        # sixteen sequences on the wide layer
        _matvec("matvec_16_wide", 16, 8192, 22016, 128, False),
        # a batch of 64 with the finest groups and fp32 scales
        _matvec("matvec_64", 64, 4096, 11008, 32, True, "fp32"),
        # a small experiment: odd height, few tokens, a length that no tile divides
        _matvec("matvec_odd", 3, 1376, 1001, 32, True, "fp32"),
        # a merged bf16 weight on its way to serving, and what it stands for afterwards
        _round4("round4_gate", 11008, 4096, 128, True),
        # the wide layer's weight from fp32: the largest case
        _round4("round4_wide", 22016, 8192, 64, False, "fp32", "fp32"),
        # eight sequences, a token each, rotation alone, at far positions
        _qk("qk_decode_8", "qk_fwd", 8, 32, 32, 128, 128, False, far=131072),
        # a training batch of the wide layer with norms, both directions
        _qk("qk_fwd_wide", "qk_fwd", 2048, 64, 64, 128, 128, True),
        _qk("qk_bwd_wide", "qk_bwd", 2048, 64, 64, 128, 128, True),
        # a ragged batch with shared key heads, a partial interleaved rotation, fp32
        _qk("qk_bwd_odd", "qk_bwd", 333, 15, 5, 80, 32, True, True, "fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["matvec", "matvec", "matvec", "round4", "qk_fwd", "qk_fwd", "qk_bwd", "qk_bwd"])
    if op in ("matvec", "round4"):
        group = rng.choice([32, 64, 128, 128, 256])
        K = group * _log(rng, max(1, 512 // group), 11008 // group)
        N = _log(rng, 256, 11008) if rng.random() < 0.5 else 16 * _log(rng, 16, 688)
        scale, zeros = rng.choice(["bf16", "bf16", "fp32"]), rng.random() < 0.5
        if op == "matvec":
            return _matvec(None, _log(rng, 1, 64), K, N, group, zeros, scale)
        return _round4(None, N, K, group, zeros, scale, rng.choice(["bf16", "bf16", "fp32"]))
    heads = _log(rng, 4, 64)
    kv = rng.choice([heads, 1, max(1, heads // 4), max(1, heads // 8)])
    dim = rng.choice([64, 80, 96, 128, 128, 128, 256])
    rot = rng.choice([dim, dim, dim, dim // 2])
    M = min(_log(rng, 1, 4096), (1 << 25) // ((heads + 2 * kv) * dim))
    return _qk(None, op, max(1, M), heads, kv, dim, rot, rng.random() < 0.6, rng.random() < 0.3,
               rng.choice(["bf16", "bf16", "bf16", "fp32"]), rng.choice([4096, 32768, 131072]))


def work(case):
    op = case["op"]
    if op.startswith("qk"):
        M, d, heads = case["M"], case["dim"], case["heads"] + case["kv"]
        size = 2 if case["dtype"] == "bf16" else 4
        small = M * 8 + case["rot"] * 2 + (2 * d * size if case["norm"] else 0)
        if op == "qk_fwd":
            return {"bytes": 2 * M * heads * d * size + small, "flops": M * heads * (7 * d if case["norm"] else 3 * d)}
        # the rows are needed for the norm's gradient alone; the v heads' gradient is passed on
        rows = 3 if case["norm"] else 2
        return {"bytes": M * d * size * (rows * heads + 2 * case["kv"]) + small * (2 if case["norm"] else 1),
                "flops": M * heads * (16 * d if case["norm"] else 3 * d)}
    N, K = case["N"], case["K"]
    weight = N * K // 2 + N * (K // case["group"]) * ((2 if case["scale"] == "bf16" else 4) + (1 if case["zeros"] else 0))
    if op == "matvec":
        return {"bytes": weight + 2 * case["M"] * (K + N), "flops": 2 * case["M"] * N * K}
    # the weight is read, codes and scales are written and read, the values are written
    return {"bytes": 2 * N * K * (2 if case["dtype"] == "bf16" else 4) + 2 * weight, "flops": 6 * N * K}


# ---- inputs --------------------------------------------------------------------------

def _quantized(W, case):
    """Codes (0 to 15, one a byte) [N, K / g, g], scales and zeros [N, K / g] of a weight."""
    w = W.float().view(W.shape[0], -1, case["group"])
    if case["zeros"]:
        lo, hi = w.amin(2).clamp_max(0.0), w.amax(2).clamp_min(0.0)
        s = (hi - lo) * PER_15
    else:
        s = w.abs().amax(2) * PER_7
    s = s.to(TYPES[case["scale"]]).float()
    none = s < TINY
    s = s.masked_fill(none, 0.0)
    inv = (1.0 / s).masked_fill(none, 0.0)
    z = (-lo * inv).round().clamp(0.0, 15.0) if case["zeros"] else torch.full_like(s, 8.0)
    codes = ((w * inv[:, :, None]).round() + z[:, :, None]).clamp(0.0, 15.0)
    return codes, s, z


def _packed(W, case):
    codes, s, z = _quantized(W, case)
    flat = codes.to(torch.uint8).view(-1)
    return {"codes": flat[0::2] | (flat[1::2] << 4), "scales": s.to(TYPES[case["scale"]]),
            "zeros": z.to(torch.uint8) if case["zeros"] else None}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=gen, device=dev) * std).to(dtype)

    op = case["op"]
    s = {"case": dict(case)}
    if op in ("matvec", "round4"):
        N, K = case["N"], case["K"]
        # a weight as it stands after training, rows and columns of unlike size
        W = normal(N, K, std=0.02, dtype=torch.float32)
        W *= torch.exp(0.3 * torch.randn((N, 1), generator=gen, device=dev))
        W += normal(N, 1, std=0.002, dtype=torch.float32)
        if op == "round4":
            s["W"] = W.to(TYPES[case["dtype"]])
            return s
        s.update(_packed(W, case))
        # a few channels of activations are much larger than the others
        s["X"] = torch.randn((case["M"], K), generator=gen, device=dev)
        s["X"][:, torch.randint(0, K, (8,), generator=gen, device=dev)] *= 20.0
        s["X"] = s["X"].bfloat16()
        return s
    M, d, heads, kv, dtype = case["M"], case["dim"], case["heads"], case["kv"], TYPES[case["dtype"]]
    s["Y"] = normal(M, (heads + 2 * kv) * d, std=1.5, dtype=dtype)
    # tokens of several sequences one after another, each from a position of its own
    start = torch.randint(0, case["far"], (M,), generator=gen, device=dev)
    run_of = torch.arange(M, device=dev) // 100
    s["positions"] = start[run_of] + torch.arange(M, device=dev) % 100
    base = 10000.0 if case["far"] <= 4096 else 500000.0
    at = torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float64) / case["rot"]
    s["inv_freq"] = (base ** -at).float()
    s["qw"] = s["kw"] = None
    if case["norm"]:
        s["qw"], s["kw"] = (1.0 + normal(d, std=0.2, dtype=torch.float32)).to(dtype), (
            1.0 + normal(d, std=0.2, dtype=torch.float32)).to(dtype)
    if op == "qk_bwd":
        s["dQ"], s["dK"], s["dV"] = normal(M, heads, d, dtype=dtype), normal(M, kv, d, dtype=dtype), normal(M, kv, d, dtype=dtype)
        # the partial sums of the norms' gradients, kept from call to call
        s["ws"] = torch.zeros((16 << 20) + 65792, dtype=torch.uint8, device=dev)
    return s


# ---- plain form ----------------------------------------------------------------------

def _turn(x, cos, sin, rot, interleaved):
    """x [M, heads, d] with the pairs of its first rot elements turned; cos, sin [M, 1, rot / 2]."""
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _plain_qk(s):
    c = s["case"]
    M, d, heads, kv = c["M"], c["dim"], c["heads"], c["kv"]
    Y = s["Y"].view(M, heads + 2 * kv, d)
    dtype = Y.dtype
    x = Y[:, :heads + kv].float()
    angle = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    if c["norm"]:
        w = torch.cat([s["qw"].float().expand(heads, d), s["kw"].float().expand(kv, d)])
        r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    if c["op"] == "qk_fwd":
        n = x * r * w if c["norm"] else x
        z = _turn(n, cos, sin, c["rot"], c["interleaved"]).to(dtype)
        return {"Q": z[:, :heads].contiguous(), "K": z[:, heads:].contiguous()}
    dz = torch.cat([s["dQ"], s["dK"]], dim=1).float()
    dn = _turn(dz, cos, -sin, c["rot"], c["interleaved"])
    out = {}
    if c["norm"]:
        xh = x * r
        dw = (dn * xh).double()  # summed over all tokens
        out["dqw"], out["dkw"] = dw[:, :heads].sum((0, 1)).to(dtype), dw[:, heads:].sum((0, 1)).to(dtype)
        dxh = dn * w
        dn = r * (dxh - xh * (dxh * xh).mean(-1, keepdim=True))
    out["dY"] = torch.cat([dn.to(dtype), s["dV"]], dim=1).view(M, -1)
    return out


def _plain(s):
    c = s["case"]
    if c["op"].startswith("qk"):
        return _plain_qk(s)
    if c["op"] == "round4":
        codes, scale, z = _quantized(s["W"], c)
        out = {"W": ((codes - z[:, :, None]) * scale[:, :, None]).to(s["W"].dtype).view(c["N"], c["K"]),
               "scales": scale.to(TYPES[c["scale"]])}
        if c["zeros"]:
            out["zeros"] = z.to(torch.uint8)
        return out
    codes = torch.stack([s["codes"] & 15, s["codes"] >> 4], dim=1).view(c["N"], -1, c["group"]).float()
    z = 8.0 if s["zeros"] is None else s["zeros"].float()[:, :, None]
    W = ((codes - z) * s["scales"].float()[:, :, None]).view(c["N"], c["K"])
    return {"Y": (s["X"].float() @ W.t()).bfloat16()}


# ---- the framework's calls -----------------------------------------------------------

def _own(s):
    import bit_quantized_lora_nf4_amd as q
    c = s["case"]
    if c["op"] == "matvec":
        gw = q.GroupWeight(s["codes"], s["scales"], s["zeros"], c["N"], c["K"], c["group"])
        return {"Y": q.group_linear_fwd(gw, s["X"])}
    if c["op"] == "round4":
        gw = q.group_quantize(s["W"], c["group"], zeros=c["zeros"], scale_dtype=TYPES[c["scale"]])
        out = {"W": q.group_dequantize(gw, s["W"].dtype), "scales": gw.scales}
        if c["zeros"]:
            out["zeros"] = gw.zeros
        return out
    if c["op"] == "qk_fwd":
        Q, K = q.qk_norm_rope_fwd(s["Y"], s["positions"], s["inv_freq"], c["heads"], c["kv"], s["qw"], s["kw"],
                                  eps=EPS, interleaved=c["interleaved"])
        return {"Q": Q, "K": K}
    dY, dqw, dkw = q.qk_norm_rope_bwd(s["dQ"], s["dK"], s["dV"], s["positions"], s["inv_freq"], s["Y"], s["qw"],
                                      s["kw"], eps=EPS, interleaved=c["interleaved"], ws=s["ws"])
    return {"dY": dY, "dqw": dqw, "dkw": dkw} if c["norm"] else {"dY": dY}


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ---- the definitions in 64 bits ------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "matvec":
        g = case["group"]
        scale = s["scales"].double().repeat_interleave(g, dim=1)
        W = torch.empty((case["N"], case["K"]), dtype=torch.float64, device=scale.device)
        pairs = s["codes"].view(case["N"], -1).long()
        W[:, 0::2], W[:, 1::2] = pairs % 16, pairs // 16
        W -= 8 if s["zeros"] is None else s["zeros"].double().repeat_interleave(g, dim=1)
        return {"Y": s["X"].double() @ (W * scale).t()}
    if op == "round4":
        # the definition's fp32 roundings, each of a value that 64 bits hold (nearly) exactly
        def rn(v):
            return v.float().double()
        w = s["W"].double().unflatten(1, (-1, case["group"]))
        top, bottom = w.amax(2), w.amin(2)
        if case["zeros"]:
            top, bottom = torch.clamp(top, min=0), torch.clamp(bottom, max=0)
            step = rn(rn(top - bottom) * rn(torch.tensor(1 / 15)))
        else:
            step = rn(torch.maximum(top, -bottom) * rn(torch.tensor(1 / 7)))
        step = step.to(TYPES[case["scale"]]).double()
        step = torch.where(step < TINY, torch.zeros_like(step), step)
        per = torch.where(step == 0, torch.zeros_like(step), rn(1 / step))
        zero = torch.round(rn(-bottom * per)).clamp(0, 15) if case["zeros"] else torch.full_like(step, 8)
        code = (torch.round(rn(w * per.unsqueeze(2))) + zero.unsqueeze(2)).clamp(0, 15)
        out = {"W": ((code - zero.unsqueeze(2)) * step.unsqueeze(2)).flatten(1), "scales": step}
        return {**out, "zeros": None} if case["zeros"] else out
    # the rotation as a product of complex numbers
    M, d, heads, kv, rot = case["M"], case["dim"], case["heads"], case["kv"], case["rot"]
    x = s["Y"].double().view(M, heads + 2 * kv, d)[:, :heads + kv]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                       torch.outer(s["positions"].double(), s["inv_freq"].double()))[:, None, :]
    at = torch.arange(rot, device=x.device)
    first = at[0::2] if case["interleaved"] else at[:rot // 2]
    second = at[1::2] if case["interleaved"] else at[rot // 2:]

    def turned(v, by):
        v = v.clone()
        p = torch.complex(v[..., first], v[..., second]) * by
        v[..., first], v[..., second] = p.real, p.imag
        return v

    w = torch.ones((heads + kv, d), dtype=torch.float64, device=x.device)
    length = torch.ones((M, heads + kv, 1), dtype=torch.float64, device=x.device)
    if case["norm"]:
        w[:heads], w[heads:] = s["qw"].double(), s["kw"].double()
        length = torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS)
    if op == "qk_fwd":
        z = turned(x / length * w, turn)
        return {"Q": z[:, :heads], "K": z[:, heads:]}
    up = turned(torch.cat([s["dQ"], s["dK"]], dim=1).double(), turn.conj())
    out = {}
    if case["norm"]:
        per = (up * x / length).sum(0)
        out["dqw"], out["dkw"] = per[:heads].sum(0), per[heads:].sum(0)
        up = up * w
        up = up / length - x * (up * x).sum(-1, keepdim=True) / (d * length ** 3)
    out["dY"] = torch.cat([up, s["dV"].double()], dim=1).view(M, -1)
    return out
