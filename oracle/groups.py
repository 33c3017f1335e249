"""4-bit integers with group scales, in numpy (test infrastructure only).

The quantizer is defined by single roundings to fp32 (and of the scale to its own type), so
the oracle takes the same steps in float32, one IEEE operation each; what the codes stand
for and the product are computed in float64.  [Repro] "官方代码阅读路线" folds the adapter
into the weight for inference; this is a form the folded weight can be served in.
"""

import numpy as np

from . import fp

TINY = np.float32(2.0 ** -126)


def quantize(W, group, zeros, scale_bf16):
    """codes [N, K] (0..15), scales [N, G] fp32 values, zeros [N, G] of W (float32 values).  A group
    whose scale is not finite gets the scale NaN (its codes mean nothing)."""
    W = np.asarray(W, np.float32)
    N, K = W.shape
    w = W.reshape(N, K // group, group)
    if zeros:
        lo, hi = np.minimum(w.min(2), np.float32(0)), np.maximum(w.max(2), np.float32(0))
        s = (hi - lo) * (np.float32(1) / np.float32(15))
    else:
        s = np.abs(w).max(2) * (np.float32(1) / np.float32(7))
    if scale_bf16:
        s = fp.bf16_to_f32(fp.bf16_bits(s)).reshape(s.shape)
    s = np.where(s < TINY, np.float32(0), np.where(np.isfinite(s), s, np.float32(np.nan))).astype(np.float32)
    none = ~(s > 0)
    inv = np.where(none, np.float32(0), np.float32(1) / np.where(none, np.float32(1), s)).astype(np.float32)
    w, lo = (np.where(np.isfinite(v), v, np.float32(0)) for v in (w, lo if zeros else s))
    z = np.clip(np.rint(-lo * inv), 0, 15) if zeros else np.full(s.shape, 8, np.float32)
    codes = np.clip(np.rint(w * inv[:, :, None]) + z[:, :, None], 0, 15)
    return codes.reshape(N, K).astype(np.uint8), s, z.astype(np.uint8)


def pack(codes):
    flat = codes.reshape(-1)
    return (flat[0::2] | (flat[1::2] << 4)).astype(np.uint8)


def unpack(packed, N, K):
    out = np.empty((packed.size, 2), np.uint8)
    out[:, 0], out[:, 1] = packed & 15, packed >> 4
    return out.reshape(N, K)


def values(codes, scales, zeros, group):
    """What the codes stand for, float64 [N, K]."""
    step = np.repeat(np.asarray(scales, np.float64), group, axis=1)
    return (codes.astype(np.float64) - np.repeat(np.asarray(zeros, np.float64), group, axis=1)) * step


def product(X, codes, scales, zeros, group):
    """Y = X W^T in float64 and, for bounds on fp32 sums, the sum of the magnitudes that are
    added: |x| s (16 + code) and |x| s (16 + zero)."""
    X = np.asarray(X, np.float64)
    s = np.abs(np.repeat(np.asarray(scales, np.float64), group, axis=1))
    z = np.repeat(np.asarray(zeros, np.float64), group, axis=1)
    mag = np.abs(X) @ (s * (32 + codes + z)).T
    return X @ values(codes, scales, zeros, group).T, mag
