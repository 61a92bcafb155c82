"""Gated blocks whose outputs are single elements: one-hot rows and weights hand the projections to
the activation, and dg, du or h to the outputs, each by one product with one and zeros besides.
With the elements' references and bounds, over projections of every size.

Arithmetic of an activation (u = 2^-24): s is g (silu) or 2 sqrt(2 / pi) (g + 0.044715 g^3) by six
roundings (gelu, |g| up to 30; the logistic function is 0 or 1 beyond).  e = exp(-s) by one product,
one constant and the hardware's base-two exponential (two u): off by (2 |s| + 3) u, for gelu by
another 6 |s| u.  p = 1 / (1 + e): one sum, one reciprocal of two u.  So p is off by
p ((1 - p) delta + 3 u).  Where e is below u / 2 the sum is one and so is its reciprocal: p is one.
Where s is below -89 e is infinite and p is zero; just above that p may lie below the smallest
normal number and be flushed."""
import numpy as np
import torch

from rows_helpers import TYPES, half_step

U = 2.0 ** -24
TINY = 2.0 ** -126
STEPS = [0.0, 1e-30, 1e-3, 0.25, 0.5, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 12, 14, 16, 17, 17.5, 18, 20, 24, 30, 31, 40, 60, 80,
         86, 87, 87.5, 88, 88.5, 89, 90, 104, 110, 300, 3e4]
LARGE = {"bf16": [1e6, 1e9, 1e20, 1e30], "fp16": [65504.0]}


def values(dtype):
    v = torch.tensor(STEPS + LARGE[dtype], dtype=torch.float64)
    return torch.cat([v, -v]).to(TYPES[dtype])


def logistic(kind, g):
    """s, its slope, p and 1 - p in float64, without cancellation."""
    c = np.clip(g, -1e3, 1e3)
    if kind == "silu":
        s, ds = c, np.ones_like(c)
    else:
        k = 2 * np.sqrt(2 / np.pi)
        s, ds = k * (c + 0.044715 * c ** 3), k * (1 + 3 * 0.044715 * c ** 2)
    with np.errstate(over="ignore"):
        return s, ds, 1 / (1 + np.exp(-s)), 1 / (1 + np.exp(s))


def activation(kind, g):
    """act(g), act'(g) and their bounds."""
    s, ds, p, q = logistic(kind, g)
    tail = p * q  # p (1 - p), zero where the logistic is saturated
    act, slope = np.where(p > 0, g * p, 0.0), p + np.where(tail > 0, g * tail, 0.0) * ds
    delta = ((2 if kind == "silu" else 8) * np.abs(s) + 3) * U
    ep = p * (q * delta + 3 * U) + TINY
    ep = np.where(s > 18, q, np.where(s < -89, p, ep))
    eq = np.where(s > 18, q, ep + U * q)
    some = (ep > 0) | (eq > 0)
    mag = np.where(some, np.abs(g), 0.0)
    e_act = mag * ep + U * np.abs(act)
    e_slope = ep + ds * (mag * (q * ep + p * eq) + 8 * U * np.where(tail > 0, np.abs(g) * tail, 0.0)) + 2 * U * np.abs(slope)
    return act, slope, e_act, e_slope


def elements(dtype, R, I, seed=0):
    """g, u and dh of every element: all values of g, u and dh within a factor of two of one fourth
    and one (their products stay in range)."""
    v = values(dtype)
    gen = torch.Generator().manual_seed(seed)
    g = v[torch.arange(R * I) % len(v)].reshape(R, I)
    assert R * I >= len(v)
    sign = torch.randint(0, 2, (R, I), generator=gen) * 2.0 - 1
    u = (sign * (0.25 + 0.25 * torch.rand(R, I, generator=gen))).to(TYPES[dtype])
    dh = (0.5 + 0.5 * torch.rand(R, I, generator=gen)).to(TYPES[dtype])
    return g, u, dh


def expected(kind, dtype, g, u, dh):
    """h, dg and du with their bounds: {name: (reference, bound)}."""
    t = TYPES[dtype]
    g, u, dh = (x.double().numpy() for x in (g, u, dh))
    act, slope, e_act, e_slope = activation(kind, g)
    out = {}
    for name, ref, err in (("h", act * u, e_act * np.abs(u)), ("dg", dh * u * slope, np.abs(dh * u) * e_slope),
                           ("du", dh * act, np.abs(dh) * e_act)):
        err = err + 3 * U * np.abs(ref) + TINY
        out[name] = (ref, err + half_step(t, np.abs(ref) + err))
    return out


def one_hot_call(dtype, g, u, dh, device="cpu"):
    """Tensors of a forward and of a backward call on those elements.  Forward: row r is one at
    column r, weight rows hold the column's g and u, w2 is one at (c, c): gu = [g, u], y = h.
    Backward: w2 and rows the same, w13 is one at (j, j): drows = [dg, du], dw13 its transpose."""
    R, I = g.shape
    d = -(-max(R, 2 * I) // 8) * 8
    t = TYPES[dtype]
    rows = torch.eye(R, d, dtype=t)
    w13 = torch.zeros(2 * I, d, dtype=t)
    w13[:I, :R], w13[I:, :R] = g.t(), u.t()
    dy = torch.zeros(R, d, dtype=t)
    dy[:, :I] = dh
    x = dict(rows=rows, w13=w13, w2=torch.eye(d, I, dtype=t), back_w13=torch.eye(2 * I, d, dtype=t), dy=dy,
             gu=torch.cat([g, u], dim=1))
    return {k: v.to(device) for k, v in x.items()}
