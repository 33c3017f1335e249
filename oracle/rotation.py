"""Query and key heads normed and turned by their positions, in float64 (test infrastructure
only).  The formulas are the usual ones: a head over its root mean square times a weight,
then rotations of pairs of its elements by angles linear in the position; both are linear
or smooth, and the gradients are pinned by differences in ``tests/test_oracle_rotation.py``.
"""

import numpy as np


def pairs(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def turn(x, positions, inv_freq, interleaved, sign=1.0):
    """x [M, heads, d]: its pairs turned by sign * position * inv_freq."""
    t = sign * np.asarray(positions, np.longdouble)[:, None] * np.asarray(inv_freq, np.longdouble)[None]
    co, si = np.cos(t).astype(np.float64)[:, None], np.sin(t).astype(np.float64)[:, None]
    a, b = pairs(2 * len(inv_freq), interleaved)
    y = x.copy()
    y[..., a] = x[..., a] * co - x[..., b] * si
    y[..., b] = x[..., b] * co + x[..., a] * si
    return y


def inverse_rms(x, eps):
    return 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)


def forward(x, w, positions, inv_freq, eps, interleaved):
    """x [M, heads, d]; w [d] or None."""
    n = x if w is None else x * inverse_rms(x, eps) * w
    return turn(n, positions, inv_freq, interleaved)


def backward(dz, x, w, positions, inv_freq, eps, interleaved):
    """(dx, dw or None)."""
    dn = turn(dz, positions, inv_freq, interleaved, -1.0)
    if w is None:
        return dn, None
    r = inverse_rms(x, eps)
    g = dn * w
    dx = r * (g - x * r * r * np.mean(g * x, axis=-1, keepdims=True))
    return dx, np.sum(dn * x * r, axis=(0, 1))
