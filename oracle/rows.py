"""Float64 reference of the row operators around the experts: rows sorted by expert and
back, the router's gradient, and the norms around a block, each with its gradient.

Readings: pair p = t*k + j; a position outside [0, num_rows) drops its pair; weights of
None are ones; rms(v) = v / sqrt(mean(v^2) + eps) over a row.
(ExactMoE, page "Every Expert Counts: ExactMoE for Memory-Efficient W4A16 Inference",
Abstract: top-k routing to grouped experts; router and normalization layers in BF16.)
"""
import numpy as np


def _pairs(pair_pos, k, num_rows, weights):
    pos = np.asarray(pair_pos, dtype=np.int64).reshape(-1, k)
    kept = (pos >= 0) & (pos < num_rows)
    w = np.ones(pos.shape) if weights is None else np.asarray(weights, dtype=np.float64)
    return pos, kept, w


def permute(x, pair_pos, k, num_rows, weights=None, rows=None):
    """rows[pos] = w x[t]; `rows` (default zeros) gives the rows that no pair names."""
    x = np.asarray(x, dtype=np.float64)
    out = np.zeros((num_rows, x.shape[1])) if rows is None else np.array(rows, dtype=np.float64)
    pos, kept, w = _pairs(pair_pos, k, num_rows, weights)
    for t, j in zip(*np.nonzero(kept)):
        out[pos[t, j]] = w[t, j] * x[t]
    return out


def unpermute(rows, pair_pos, k, weights=None):
    """out[t] = sum_j w rows[pos]."""
    rows = np.asarray(rows, dtype=np.float64)
    pos, kept, w = _pairs(pair_pos, k, rows.shape[0], weights)
    out = np.zeros((pos.shape[0], rows.shape[1]))
    for t, j in zip(*np.nonzero(kept)):
        out[t] += w[t, j] * rows[pos[t, j]]
    return out


def pair_products(token_rows, sorted_rows, pair_pos, k):
    """<token_rows[t], sorted_rows[pos]> per pair, 0 for dropped ones: the gradient of the
    weights of both directions."""
    a, b = np.asarray(token_rows, dtype=np.float64), np.asarray(sorted_rows, dtype=np.float64)
    pos, kept, _ = _pairs(pair_pos, k, b.shape[0], None)
    out = np.zeros(pos.shape)
    for t, j in zip(*np.nonzero(kept)):
        out[t, j] = a[t] @ b[pos[t, j]]
    return out


def softmax(logits):
    e = np.exp(logits - logits.max(axis=1, keepdims=True))
    return e / e.sum(axis=1, keepdims=True)


def route_weights(logits, ids, renormalize):
    """The routing weights of given selections (differentiable part of the router)."""
    logits = np.asarray(logits, dtype=np.float64)
    if renormalize:
        return softmax(np.take_along_axis(logits, ids, axis=1))
    return np.take_along_axis(softmax(logits), ids, axis=1)


def route_dlogits(logits, ids, weights, dweights, renormalize, dlogits=None):
    """Gradient of the logits from that of the weights (ids outside [0, E) ignored)."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    ids = np.asarray(ids, dtype=np.int64)
    ok = (ids >= 0) & (ids < E)
    w = np.where(ok, np.asarray(weights, dtype=np.float64), 0.0)
    dw = np.where(ok, np.asarray(dweights, dtype=np.float64), 0.0)
    s = (w * dw).sum(axis=1, keepdims=True)
    g = np.zeros((T, E)) if renormalize else -softmax(logits) * s
    for t, j in zip(*np.nonzero(ok)):
        g[t, ids[t, j]] = w[t, j] * (dw[t, j] - s[t, 0])
    return g if dlogits is None else g + np.asarray(dlogits, dtype=np.float64)


def route_backward(x, w_router, logits, ids, weights, dweights, renormalize, dlogits=None, dx_add=None):
    """(dx, dw_router)."""
    g = route_dlogits(logits, ids, weights, dweights, renormalize, dlogits)
    dx = g @ np.asarray(w_router, dtype=np.float64)
    if dx_add is not None:
        dx = dx + np.asarray(dx_add, dtype=np.float64)
    return dx, g.T @ np.asarray(x, dtype=np.float64)


def _f64(v):
    return None if v is None else np.asarray(v, dtype=np.float64)


def rstd(v, eps):
    return 1.0 / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)


def block_norm(x, y=None, norm_in=None, norm_out=None, gate=None, residual_scale=1.0, eps=1e-6):
    """(h, n): h = a x + g z with z = rms(y) norm_out, n = rms(h) norm_in (None without)."""
    x, y, v_in, v_out, g = (_f64(v) for v in (x, y, norm_in, norm_out, gate))
    h = residual_scale * x
    if y is not None:
        z = y if v_out is None else y * rstd(y, eps) * v_out
        h = h + (z if g is None else g * z)
    return h, None if v_in is None else h * rstd(h, eps) * v_in


def block_norm_backward(x, y=None, norm_in=None, norm_out=None, gate=None, residual_scale=1.0, eps=1e-6, dh=None,
                        dn=None):
    """Gradients of block_norm as a dict: dx, dy, dgate, dnorm_out, dnorm_in."""
    x, y, v_in, v_out, g, dh, dn = (_f64(v) for v in (x, y, norm_in, norm_out, gate, dh, dn))
    h, _ = block_norm(x, y, norm_in, norm_out, gate, residual_scale, eps)
    D = np.zeros_like(x) if dh is None else dh
    out = {}
    if v_in is not None:
        dn = np.zeros_like(x) if dn is None else dn
        r = rstd(h, eps)
        hn, u = h * r, dn * v_in
        out["dnorm_in"] = (dn * hn).sum(axis=0)
        D = D + r * (u - hn * (u * hn).mean(axis=1, keepdims=True))
    out["dx"] = residual_scale * D
    if y is not None:
        ry = 1.0 if v_out is None else rstd(y, eps)
        yn = y * ry
        z = yn if v_out is None else yn * v_out
        if g is not None:
            dg = D * z
            out["dgate"] = dg.sum(axis=0) if g.ndim == 1 else dg.sum(axis=1, keepdims=True) if g.shape[1] == 1 else dg
        q = D if g is None else D * g
        if v_out is None:
            out["dy"] = q
        else:
            out["dnorm_out"] = (q * yn).sum(axis=0)
            u = q * v_out
            out["dy"] = ry * (u - yn * (u * yn).mean(axis=1, keepdims=True))
    return out
