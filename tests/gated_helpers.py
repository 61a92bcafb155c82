"""Inputs and error bounds of the gated blocks' tests.

Arithmetic of the kernels: products of 16-bit values are exact in float32; a matrix
instruction adds its 32 products to the running sum, where every eight terms meet at most
one rounding or truncation of the sum of absolute terms so far (2^-23); activation and its
slope by hardware exp and reciprocal; one rounding to the type per stored value."""
import numpy as np
import torch

from oracle import gated
from rows_helpers import TYPES, f64, half_step

DEV = "cuda"
SEED, STEP = 0x1234567890ABCDE, (3 << 32) + 17


def sums(K, absolute):
    """Bound of a float32 sum of K products whose absolute values add up to `absolute`."""
    return (K / 8 + 16) * 2.0 ** -23 * absolute


def activation_error(g):
    """Of act(g) / (1 + |g|) and of act'(g): the logistic function's argument is off by a few
    2^-24 of up to |g| (gelu: of 4 |g| where it is not saturated), its exp and reciprocal by
    two units each."""
    return 2.0 ** -19 * (1 + np.abs(g))


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def inputs(R, E, d, I, dtype, seed=0, device=DEV):
    g = torch.Generator().manual_seed(seed)

    def rand(*shape, std=1.0):
        return (torch.randn(*shape, generator=g) * std).to(TYPES[dtype]).to(device)

    return dict(rows=rand(R, d), w13=rand(E, 2 * I, d, std=d ** -0.5), w2=rand(E, d, I, std=I ** -0.5),
                dy=rand(R, d, std=0.5))


def forward_bounds(x, off, act, factor, dtype):
    """References (y, h, gu) and their bounds."""
    rows, w13, w2 = f64(x["rows"]), f64(x["w13"]), f64(x["w2"])
    (R, d), I, E = rows.shape, w2.shape[2], w2.shape[0]
    y, h, gu = gated.gated_ffn(rows, w13, w2, off, act, factor)
    t = TYPES[dtype]
    by, bh, bgu = np.zeros_like(y), np.zeros_like(h), np.zeros_like(gu)
    for e, a, b in gated._experts(off, R, E):
        raw = sums(d, np.abs(rows[a:b]) @ np.abs(w13[e]).T)
        bgu[a:b] = raw + half_step(t, gu[a:b])
        g, u = gu[a:b, :I], gu[a:b, I:]
        eg, eu = raw[:, :I], raw[:, I:]
        value = gated.activation(act, g)[0]
        ea = 1.2 * eg + activation_error(g) * (1 + np.abs(g))  # |act'| < 1.2
        bh[a:b] = (ea * np.abs(u) + np.abs(value) * eu + ea * eu + 2.0 ** -22 * np.abs(value * u))
        if factor is not None:
            bh[a:b] *= factor[a:b]
        bh[a:b] += half_step(t, h[a:b])
        by[a:b] = sums(I, np.abs(h[a:b]) @ np.abs(w2[e]).T) + bh[a:b] @ np.abs(w2[e]).T + half_step(t, y[a:b])
    return (y, h, gu), (by, bh, bgu)


def backward_bounds(x, gu, h, off, act, factor, dtype):
    """References (drows, dw13, dw2) at the given gu and h, and their bounds."""
    rows, w13, w2, dy = (f64(x[q]) for q in ("rows", "w13", "w2", "dy"))
    (R, d), I, E = rows.shape, w2.shape[2], w2.shape[0]
    drows, dw13, dw2, dgu = gated.gated_ffn_backward(dy, rows, w13, w2, gu, h, off, act, factor)
    t = TYPES[dtype]
    b_rows, b_13, b_2 = np.zeros_like(drows), np.zeros_like(dw13), np.zeros_like(dw2)
    for e, a, b in gated._experts(off, R, E):
        n = b - a
        f = 1.0 if factor is None else factor[a:b]
        dh, edh = dy[a:b] @ w2[e] * f, sums(d, np.abs(dy[a:b]) @ np.abs(w2[e])) * f
        g, u = gu[a:b, :I], gu[a:b, I:]
        value, slope = gated.activation(act, g)
        es = activation_error(g)
        eg = edh * np.abs(u * slope) + np.abs(dh * u) * es + 2.0 ** -22 * np.abs(dgu[a:b, :I])
        eu = edh * np.abs(value) + np.abs(dh) * es * (1 + np.abs(g)) + 2.0 ** -22 * np.abs(dgu[a:b, I:])
        edgu = np.concatenate([eg, eu], axis=1) + half_step(t, dgu[a:b])
        mag = np.abs(dgu[a:b])
        b_rows[a:b] = sums(2 * I, mag @ np.abs(w13[e])) + edgu @ np.abs(w13[e]) + half_step(t, drows[a:b])
        b_13[e] = sums(n, mag.T @ np.abs(rows[a:b])) + edgu.T @ np.abs(rows[a:b]) + half_step(t, dw13[e])
        b_2[e] = sums(n, np.abs(dy[a:b]).T @ np.abs(h[a:b])) + half_step(t, dw2[e])
    return (drows, dw13, dw2), (b_rows, b_13, b_2)
