"""Dropout from a counter-based generator, and the QLoRA linear with dropout on the
adapter's input, in float64 (test infrastructure only; page names in ``oracle/__init__.py``).

[Repro] "官方代码阅读路线" lists ``lora_dropout`` among the adapter's settings: the adapter
reads a dropped copy D(X) of the linear's input while the frozen path reads X itself.  The
pages fix no generator; the reading here needs no state and stores no mask:

* Philox4x32 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3",
  2011): a block of four 32-bit words from a 128-bit counter and a 64-bit key.  Seven rounds.
* Element e of a row-major tensor takes 16 bits h of the block of counter (e // 8, offset)
  (two 64-bit words, low halves first) under the key seed: word (e % 8) // 2, the low half
  for even e.  It is kept iff h >= t, t = floor(65536 p + 1/2), and scaled by
  c = 65536 / (65536 - t), so that the expectation is the identity exactly.

With V = c (alpha/r) dY B and U = c (alpha/r) (m X) A^T:
    Y = X W'^T + U B^T,  dX = dY W' + m (V A),  dB = dY^T U,  dA = V^T (m X)
"""

import numpy as np

M0, M1 = 0xD2511F53, 0xCD9E8D57
W0, W1 = 0x9E3779B9, 0xBB67AE85
MASK32 = 0xFFFFFFFF


def philox4x32(counter, key, rounds):
    """Blocks of Philox4x32 for counter words (four arrays of 32-bit values) and one key."""
    x = [np.asarray(c, np.uint64) for c in counter]
    k0, k1 = key
    s32, low = np.uint64(32), np.uint64(MASK32)
    for _ in range(rounds):
        a, b = x[0] * np.uint64(M0), x[2] * np.uint64(M1)  # 32 x 32 bits: exact in 64
        x = [(b >> s32) ^ x[1] ^ np.uint64(k0), b & low, (a >> s32) ^ x[3] ^ np.uint64(k1), a & low]
        k0, k1 = (k0 + W0) & MASK32, (k1 + W1) & MASK32
    return x


def threshold(p):
    t = int(np.floor(p * 65536.0 + 0.5))
    if not 0.0 <= p < 1.0 or t > 65535:
        raise ValueError("drop probability outside [0, 1)")
    return t


def scale(p):
    return 65536.0 / (65536 - threshold(p))


def keep(shape, p, seed, offset, first=0):
    """Boolean mask of the kept elements ``first`` .. of a row-major tensor."""
    n = int(np.prod(shape))
    e = np.arange(first, first + n, dtype=np.uint64)
    g0 = first // 8
    g = np.arange(g0, (first + n + 7) // 8, dtype=np.uint64)
    o = offset % (1 << 64)
    words = philox4x32([g & np.uint64(MASK32), g >> np.uint64(32), np.full_like(g, o & MASK32),
                        np.full_like(g, o >> 32)], (seed & MASK32, seed >> 32), 7)
    w = np.stack(words)                                       # [4, groups]
    word = w[((e % np.uint64(8)) // np.uint64(2)).astype(np.int64), (e // np.uint64(8)).astype(np.int64) - g0]
    h = np.where(e % np.uint64(2) == 0, word & np.uint64(0xFFFF), word >> np.uint64(16))
    return (h >= np.uint64(threshold(p))).reshape(shape)


def forward(X, Wd, A, B, alpha, r, m, c):
    """(Y, U) of the linear with mask m [M, K] and scale c."""
    U = c * (alpha / r) * ((m * X) @ A.T)
    return X @ Wd.T + U @ B.T, U


def backward(dY, X, Wd, A, B, alpha, r, m, c, U):
    """(dX, dA, dB, V); U is the saved [M, r] down-projection that the operator uses."""
    V = c * (alpha / r) * (dY @ B)
    return dY @ Wd + m * (V @ A), V.T @ (m * X), dY.T @ U, V
