"""The bounds of the saturated activations' GPU test tell right from wrong: they hold for the
kernel's formulas in float32, and mistakes at every size of projection exceed them."""
import numpy as np
import pytest
import torch

from oracle import gated

from saturation_helpers import activation, elements, expected, one_hot_call, values

CASES = [("silu", "bf16"), ("silu", "fp16"), ("gelu", "bf16"), ("gelu", "fp16")]


def stored(kind, dtype, g, u, dh, act=None, slope=None):
    """What float32 arithmetic with one rounding stores, from the exact activation or another."""
    g64 = g.double().numpy()
    a, s, _, _ = activation(kind, g64)
    a, s = (a if act is None else act(g64, a)), (s if slope is None else slope(g64, s))
    u, dh = u.double().numpy(), dh.double().numpy()
    return {n: torch.from_numpy(v).to(g.dtype).double().numpy()
            for n, v in (("h", a * u), ("dg", dh * u * s), ("du", dh * a))}


def outside(got, want, name):
    ref, bound = want[name]
    return np.abs(got[name] - ref) > bound


@pytest.mark.parametrize("kind,dtype", CASES)
def test_reference_is_the_formula(kind, dtype):
    """The reference without cancellation against the textbook forms, where those have no
    cancellation, and the slope against differences."""
    g = np.linspace(-4, 30, 400)
    act, slope, _, _ = activation(kind, g)
    a, s = gated.activation(kind, g)
    assert np.allclose(act, a, rtol=1e-11, atol=1e-13) and np.allclose(slope, s, rtol=1e-11, atol=1e-13)
    g = np.linspace(-80, 80, 321)
    eps = 1e-6
    diff = (activation(kind, g + eps)[0] - activation(kind, g - eps)[0]) / (2 * eps)
    assert np.allclose(activation(kind, g)[1], diff, rtol=1e-7, atol=1e-8)


@pytest.mark.parametrize("kind,dtype", CASES)
def test_bounds_hold_and_reject(kind, dtype):
    g, u, dh = elements(dtype, 16, 40)
    want = expected(kind, dtype, g, u, dh)
    right = stored(kind, dtype, g, u, dh)
    for name in want:
        assert np.isfinite(want[name][1]).all() and not outside(right, want, name).any()
    # slopes and activations that are wrong beyond some size, for each sign and size beyond
    size, positive = np.abs(g.double().numpy()), g.double().numpy() > 0
    for least in (2, 20, 90, 3e4, float(values(dtype).abs().max())):
        for sign in (positive, ~positive):
            at = (size >= least * 0.99) & sign
            for mistake in (0.0, 7.0, -1.0, 1.01, 0.25):
                bad = stored(kind, dtype, g, u, dh, slope=lambda x, s: np.where(at, mistake, s))
                true = activation(kind, g.double().numpy())[1]
                # a slope's mistake is seen in every element where it is one
                wrong = at & (np.abs(true - mistake) > 0.005)
                assert outside(bad, want, "dg")[wrong].all()
        # dropping the activation of positive projections, keeping that of negative ones
        bad = stored(kind, dtype, g, u, dh, act=lambda x, a: np.where(size >= least * 0.99, x - a, a))
        for name in ("h", "du"):
            assert outside(bad, want, name)[size >= least * 0.99].all()


@pytest.mark.parametrize("kind,dtype", CASES)
def test_one_hot_calls(kind, dtype):
    """The calls compute single elements: the float64 reference on them gives the references."""
    g, u, dh = elements(dtype, 16, 40)
    x = {k: v.double().numpy() for k, v in one_hot_call(dtype, g, u, dh).items()}
    want = expected(kind, dtype, g, u, dh)
    with np.errstate(over="ignore"):
        y, h, gu = gated.gated_ffn(x["rows"], x["w13"][None], x["w2"][None], None, kind)
        drows, dw13, _, _ = gated.gated_ffn_backward(x["dy"], x["rows"], x["back_w13"][None], x["w2"][None], gu, h, None, kind)
    assert np.array_equal(gu, x["gu"])
    near = dict(rtol=1e-3, atol=1e-13)  # (the reference's textbook forms cancel far down the negative side)
    for got, name in ((h, "h"), (y[:, :40], "h"), (drows[:, :40], "dg"), (drows[:, 40:80], "du"),
                      (dw13[0, :40, :16].T, "dg"), (dw13[0, 40:, :16].T, "du")):
        assert np.allclose(got, want[name][0], **near)
    assert not y[:, 40:].any() and not drows[:, 80:].any() and not dw13[0, :, 16:].any()
