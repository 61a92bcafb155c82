"""The float64 reference of the gated blocks and of dropout: known answers of the generator,
gradients against differences."""
import numpy as np
import pytest

from oracle import gated

# published known answers of Philox-4x32-10: counter, key, result
KNOWN = [((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
         ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
         ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
          (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))]


@pytest.mark.parametrize("counter,key,result", KNOWN)
def test_generator_known_answers(counter, key, result):
    assert tuple(gated.philox(counter, key)) == result
    words = gated.philox_words(*[np.uint64(c) for c in counter], key[0] | key[1] << 32)
    assert tuple(int(w) for w in words) == result


def test_mask_by_element():
    seed, step, site, p = 0x0123456789ABCDEF, 5 + (7 << 32), 9, 0.3
    f = gated.drop_factor(p, seed, step, site, 5, 21)
    t = gated.threshold(p)
    for r in range(5):
        for c in range(21):
            w = gated.philox((c // 8 + (site << 21), r, 5, 7), (seed & 0xFFFFFFFF, seed >> 32))[(c % 8) // 2]
            number = w >> 16 if c % 2 else w & 0xFFFF
            assert f[r, c] == (65536 / (65536 - t) if number >= t else 0)
    # rows further down are the same mask's
    assert np.array_equal(gated.drop_factor(p, seed, step, site, 2, 21, first_row=3), f[3:])


def test_mask_expectation_and_independence():
    p = 0.25
    f = gated.drop_factor(p, 42, 1, 0, 400, 1000)
    n = f.size
    # a mean of n draws of variance p (1 - p): six deviations
    assert abs((f > 0).mean() - (1 - p)) < 6 * (p * (1 - p) / n) ** 0.5
    for other in (gated.drop_factor(p, 43, 1, 0, 400, 1000), gated.drop_factor(p, 42, 2, 0, 400, 1000),
                  gated.drop_factor(p, 42, 1, 1, 400, 1000)):
        both = ((f > 0) & (other > 0)).mean()
        q = (1 - p) ** 2
        assert abs(both - q) < 6 * (q * (1 - q) / n) ** 0.5


def test_mask_extremes():
    assert np.array_equal(gated.drop_factor(0.0, 1, 1, 0, 3, 5), np.ones((3, 5)))
    assert np.array_equal(gated.drop_factor(1.0, 1, 1, 0, 3, 5), np.zeros((3, 5)))
    x = np.array([[np.inf, np.nan, 1.0]])
    assert np.array_equal(gated.dropout(x, np.zeros((1, 3)), np.ones((1, 3))), np.ones((1, 3)))


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("p", [0.0, 0.4])
def test_gradient_against_differences(act, p):
    rng = np.random.default_rng(5)
    R, d, I, E = 7, 6, 5, 3
    offsets = np.array([0, 3, 3, 6])       # an expert without rows, and a row behind the last one
    rows, dy = rng.standard_normal((R, d)), rng.standard_normal((R, d))
    w13, w2 = rng.standard_normal((E, 2 * I, d)), rng.standard_normal((E, d, I))
    factor = gated.drop_factor(p, 3, 4, 5, R, I)

    def loss(rows, w13, w2):
        return (gated.gated_ffn(rows, w13, w2, offsets, act, factor)[0] * dy).sum()

    _, h, gu = gated.gated_ffn(rows, w13, w2, offsets, act, factor)
    drows, dw13, dw2, _ = gated.gated_ffn_backward(dy, rows, w13, w2, gu, h, offsets, act, factor)
    eps = 1e-6
    for name, leaf, grad in (("rows", rows, drows), ("w13", w13, dw13), ("w2", w2, dw2)):
        for at in np.ndindex(leaf.shape):
            args = dict(rows=rows, w13=w13, w2=w2)
            hi, lo = leaf.copy(), leaf.copy()
            hi[at] += eps
            lo[at] -= eps
            diff = (loss(**{**args, name: hi}) - loss(**{**args, name: lo})) / (2 * eps)
            # third derivatives times eps^2, and cancellation of values below 1e3 over 2 eps
            assert abs(diff - grad[at]) < 1e-6, (name, at)
    assert not drows[6].any() and not dw13[1].any() and not dw2[1].any()
