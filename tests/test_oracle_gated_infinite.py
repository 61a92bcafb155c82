"""Infinities and NaN in the dropped places of the float64 reference of a gated block."""
import numpy as np

from oracle import gated

P, SEED, STEP, SITE = 0.4, 11, 12, 3


def test_forward():
    factor = gated.drop_factor(P, SEED, STEP, SITE, 2, 8)
    assert 0 < (factor == 0).sum() < 16
    w13, w2 = np.ones((1, 16, 4)), np.ones((1, 4, 8))
    with np.errstate(all="ignore"):
        _, h, _ = gated.gated_ffn(np.full((2, 4), np.inf), w13, w2, None, "silu", factor)
    assert np.array_equal(h == 0, factor == 0)


def test_gradient():
    factor = gated.drop_factor(P, SEED, STEP, SITE, 6, 8)
    rng = np.random.default_rng(1)
    rows, dy = rng.standard_normal((6, 4)), rng.standard_normal((6, 4))
    w13, w2 = rng.standard_normal((1, 16, 4)), rng.standard_normal((1, 4, 8))
    _, h, gu = gated.gated_ffn(rows, w13, w2, None, "silu", factor)
    want = gated.gated_ffn_backward(dy, rows, w13, w2, gu, h, None, "silu", factor)
    for value in (np.inf, -np.inf, np.nan):
        bad = np.where(np.concatenate([factor, factor], axis=1) == 0, value, gu)
        with np.errstate(all="ignore"):
            got = gated.gated_ffn_backward(dy, rows, w13, w2, bad, h, None, "silu", factor)
        for a, b in zip(got, want):
            assert np.array_equal(a, b)
