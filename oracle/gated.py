"""Float64 reference of the gated feed-forward blocks with their gradient, and of dropout
from a counter-based generator.

Readings: with W13 = [Wg; Wu] of a row's expert, g = x Wg^T, u = x Wu^T,
h = drop(act(g) u), y = h W2^T; rows of expert e are offsets[e] .. offsets[e + 1] - 1, rows
behind the last expert's stay as they were (zeros here).  A dropped element is zero, and so are
its gradients, whatever its g and u are (infinities and NaN).  Dropout keeps element (r, c) where
its 16-bit number of Philox-4x32-10 is at least round(p 2^16) and scales it by 1 / (1 - p)
at that rounded p.
(ExactMoE, page "Every Expert Counts: ExactMoE for Memory-Efficient W4A16 Inference",
Abstract: every selected expert runs through fused grouped kernels; it names no activation and
no training.)
"""
import math

import numpy as np

MASK32 = 0xFFFFFFFF


def philox(counter, key):
    """Ten rounds of Philox-4x32 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
    easy as 1, 2, 3", 2011) on one counter of four 32-bit words, in Python integers."""
    c, k = list(counter), list(key)
    for r in range(10):
        if r:
            k = [(k[0] + 0x9E3779B9) & MASK32, (k[1] + 0xBB67AE85) & MASK32]
        p0, p1 = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & MASK32, (p0 >> 32) ^ c[3] ^ k[1], p0 & MASK32]
    return c


def philox_words(c0, c1, c2, c3, seed):
    """The same on arrays of counters (uint64 holding 32-bit words): four arrays."""
    u = np.uint64
    c = [np.asarray(v, dtype=u) for v in np.broadcast_arrays(c0, c1, c2, c3)]
    k = [seed & MASK32, (seed >> 32) & MASK32]
    for _ in range(10):
        p0, p1 = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(p1 >> u(32)) ^ c[1] ^ u(k[0]), p1 & u(MASK32), (p0 >> u(32)) ^ c[3] ^ u(k[1]), p0 & u(MASK32)]
        k = [(k[0] + 0x9E3779B9) & MASK32, (k[1] + 0xBB67AE85) & MASK32]
    return c


def threshold(p):
    return int(math.floor(p * 65536 + 0.5))


def drop_factor(p, seed, step, site, rows, cols, first_row=0):
    """[rows, cols] of 0 (dropped) and 1 / (1 - p) (kept), for rows first_row and up."""
    t = threshold(p)
    if t == 0:
        return np.ones((rows, cols))
    n = -(-cols // 8)
    step &= (1 << 64) - 1
    words = philox_words(np.arange(n, dtype=np.uint64)[None, :] | np.uint64(site << 21),
                         np.arange(first_row, first_row + rows, dtype=np.uint64)[:, None],
                         np.uint64(step & MASK32), np.uint64(step >> 32), seed & ((1 << 64) - 1))
    numbers = np.empty((rows, n, 8), dtype=np.int64)
    for w, v in enumerate(words):
        numbers[:, :, 2 * w] = v & np.uint64(0xFFFF)
        numbers[:, :, 2 * w + 1] = v >> np.uint64(16)
    keep = numbers.reshape(rows, -1)[:, :cols] >= t
    return keep * (65536.0 / (65536 - t) if t < 65536 else 0.0)


def dropout(x, factor, residual=None):
    out = np.where(factor > 0, np.asarray(x, dtype=np.float64) * factor, 0.0)
    return out if residual is None else out + np.asarray(residual, dtype=np.float64)


def activation(name, g):
    """The activation and its derivative."""
    g = np.asarray(g, dtype=np.float64)
    if name == "silu":
        p = 1.0 / (1.0 + np.exp(-g))
        return g * p, p + g * p * (1 - p)
    c = math.sqrt(2 / math.pi)
    th = np.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th ** 2) * c * (1 + 3 * 0.044715 * g ** 2)


def _experts(offsets, num_rows, E):
    if offsets is None:
        return [(0, 0, num_rows)]
    return [(e, int(offsets[e]), int(offsets[e + 1])) for e in range(E)]


def _times(values, factor, a, b):
    """Rows a .. b - 1 of a mask on their values; what is dropped is zero, not times zero."""
    return values if factor is None else np.where(factor[a:b] > 0, values * factor[a:b], 0.0)


def gated_ffn(rows, w13, w2, offsets=None, act="silu", factor=None):
    """(y, h, gu); weights [E, 2I, d] and [E, d, I]."""
    rows = np.asarray(rows, dtype=np.float64)
    (R, d), (E, twoI, _) = rows.shape, w13.shape
    I = twoI // 2
    y, h, gu = np.zeros((R, d)), np.zeros((R, I)), np.zeros((R, twoI))
    for e, a, b in _experts(offsets, R, E):
        gu[a:b] = rows[a:b] @ w13[e].T
        h[a:b] = _times(activation(act, gu[a:b, :I])[0] * gu[a:b, I:], factor, a, b)
        y[a:b] = h[a:b] @ w2[e].T
    return y, h, gu


def gated_ffn_backward(dy, rows, w13, w2, gu, h, offsets=None, act="silu", factor=None):
    """(drows, dw13, dw2, dgu) at the given gu and h."""
    dy, rows = np.asarray(dy, dtype=np.float64), np.asarray(rows, dtype=np.float64)
    R, (E, twoI, d) = rows.shape[0], w13.shape
    I = twoI // 2
    drows, dgu = np.zeros((R, d)), np.zeros((R, twoI))
    dw13, dw2 = np.zeros((E, twoI, d)), np.zeros((E, d, I))
    for e, a, b in _experts(offsets, R, E):
        dh = dy[a:b] @ w2[e]
        value, slope = activation(act, gu[a:b, :I])
        dgu[a:b, :I] = _times(dh * gu[a:b, I:] * slope, factor, a, b)
        dgu[a:b, I:] = _times(dh * value, factor, a, b)
        drows[a:b] = dgu[a:b] @ w13[e]
        dw13[e] = dgu[a:b].T @ rows[a:b]
        dw2[e] = dy[a:b].T @ h[a:b]
    return drows, dw13, dw2, dgu
