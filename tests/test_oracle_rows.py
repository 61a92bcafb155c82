"""The float64 reference of the row operators: values pinned by hand, and every gradient
against central differences of its forward form."""
import numpy as np
import pytest

from oracle import rows as orow


def differences(f, v, dout, step=1e-6):
    """Gradient of sum(f(v) * dout) by central differences."""
    g = np.zeros_like(v)
    for i in np.ndindex(*v.shape):
        a, b = v.copy(), v.copy()
        a[i] += step
        b[i] -= step
        g[i] = ((f(a) - f(b)) * dout).sum() / (2 * step)
    return g


# central differences with step s of functions of order 1: truncation s^2 = 1e-12 and
# rounding 2^-53 / s = 1e-10, each times factors of order 10
TOL = 1e-7


def test_permute_by_hand():
    x = np.array([[1.0, 2.0], [3.0, 4.0]])
    pos = [2, 0, -1, 1]  # token 1 has one pair dropped
    w = np.array([[0.5, 2.0], [9.0, 1.0]])
    assert orow.permute(x, pos, 2, 3).tolist() == [[1, 2], [3, 4], [1, 2]]
    assert orow.permute(x, pos, 2, 3, w).tolist() == [[2, 4], [3, 4], [0.5, 1]]
    assert orow.permute(x, pos, 2, 2, w).tolist() == [[2, 4], [3, 4]]  # position 2 is past the last row
    rows = np.array([[1.0, 1.0], [2.0, 0.0], [0.0, 4.0]])
    assert orow.unpermute(rows, pos, 2, w).tolist() == [[2.0, 4.0], [2.0, 0.0]]
    assert orow.unpermute(rows, [-1, 5, 7, -3], 2).tolist() == [[0, 0], [0, 0]]
    assert orow.pair_products(x, rows, pos, 2).tolist() == [[8.0, 3.0], [0.0, 6.0]]


def test_permute_gradients_by_differences():
    rng = np.random.default_rng(1)
    T, d, k = 3, 4, 2
    pos, R = np.array([4, 0, 1, -1, 3, 2]), 5
    x, w, rows = rng.normal(size=(T, d)), rng.normal(size=(T, k)), rng.normal(size=(R, d))
    drows, dout = rng.normal(size=(R, d)), rng.normal(size=(T, d))
    assert np.abs(differences(lambda v: orow.permute(v, pos, k, R, w), x, drows)
                  - orow.unpermute(drows, pos, k, w)).max() < TOL
    assert np.abs(differences(lambda v: orow.permute(x, pos, k, R, v), w, drows)
                  - orow.pair_products(x, drows, pos, k)).max() < TOL
    assert np.abs(differences(lambda v: orow.unpermute(v, pos, k, w), rows, dout)
                  - orow.permute(dout, pos, k, R, w)).max() < TOL
    assert np.abs(differences(lambda v: orow.unpermute(rows, pos, k, v), w, dout)
                  - orow.pair_products(dout, rows, pos, k)).max() < TOL


@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient_by_differences(renormalize):
    rng = np.random.default_rng(2)
    T, d, E, k = 3, 4, 5, 2
    x, w = rng.normal(size=(T, d)), rng.normal(size=(E, d))
    ids = np.array([[0, 3], [4, 1], [2, 0]])
    dweights, dlog = rng.normal(size=(T, k)), rng.normal(size=(T, E))

    def loss_terms(x, w):
        l = x @ w.T
        return np.concatenate([orow.route_weights(l, ids, renormalize), l], axis=1)

    both = np.concatenate([dweights, dlog], axis=1)
    logits = x @ w.T
    weights = orow.route_weights(logits, ids, renormalize)
    dx, dw = orow.route_backward(x, w, logits, ids, weights, dweights, renormalize, dlog)
    assert np.abs(differences(lambda v: loss_terms(v, w), x, both) - dx).max() < TOL
    assert np.abs(differences(lambda v: loss_terms(x, v), w, both) - dw).max() < TOL
    dx1, _ = orow.route_backward(x, w, logits, ids, weights, dweights, renormalize, dlog, dx_add=x)
    assert np.allclose(dx1, dx + x, rtol=0, atol=1e-15)


def test_block_norm_by_hand():
    x = np.array([[3.0, 4.0]])
    h, n = orow.block_norm(x, norm_in=np.array([1.0, 2.0]), eps=0.0)
    assert h.tolist() == [[3, 4]] and np.allclose(n, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]])
    h, n = orow.block_norm(x, np.array([[1.0, -1.0]]), norm_out=np.array([2.0, 3.0]), gate=np.array([[0.5]]),
                           residual_scale=2.0, eps=0.0)
    assert np.allclose(h, [[7.0, 6.5]]) and n is None


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("norm_out", [True, False])
@pytest.mark.parametrize("norm_in", [True, False])
def test_block_norm_gradients_by_differences(gate, norm_out, norm_in):
    rng = np.random.default_rng(3)
    T, d = 2, 5
    p = dict(x=rng.normal(size=(T, d)), y=rng.normal(size=(T, d)),
             norm_in=rng.normal(size=d) if norm_in else None, norm_out=rng.normal(size=d) if norm_out else None,
             gate={"none": None, "channel": rng.normal(size=d), "token": rng.normal(size=(T, 1)),
                   "full": rng.normal(size=(T, d))}[gate])
    dh, dn = rng.normal(size=(T, d)), rng.normal(size=(T, d)) if norm_in else None
    got = orow.block_norm_backward(**p, residual_scale=0.7, dh=dh, dn=dn)

    def f(**q):
        h, n = orow.block_norm(**{**p, **q}, residual_scale=0.7)
        return h if n is None else np.concatenate([h, n])

    both = dh if dn is None else np.concatenate([dh, dn])
    names = dict(x="dx", y="dy", norm_in="dnorm_in", norm_out="dnorm_out", gate="dgate")
    for q, grad in names.items():
        if p[q] is None:
            assert grad not in got
            continue
        assert np.abs(differences(lambda v: f(**{q: v}), p[q], both) - got[grad]).max() < TOL, grad
