"""Infinite and NaN elements at the end of a row, where a lane's eight elements may overlap
those of the lane before: they count once, in the results that the formulas give them to."""
import numpy as np
import pytest
import torch

import w4a16_grouped_expert_amd as moe
from oracle import rows as orow

from gpu_helpers import say
from rows_helpers import TYPES, f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF = float("inf")


def same(got, ref):
    np.testing.assert_array_equal(f64(got), ref)


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("k", [2, 3, 9])
@pytest.mark.parametrize("d", [9, 40, 250, 520, 1111, 2600])
def test_products_of_the_last_columns(d, k, type_):
    """The weights' gradients of both directions: one infinite or NaN element in the last
    column, or the first of the last eight, of a token's row or of a sorted row."""
    say(f"products with infinite last columns d={d} k={k} {type_}")
    T, dt = 7, TYPES[type_]
    g = torch.Generator().manual_seed(d * 31 + k)
    pos = torch.randperm(T * k, generator=g).to(torch.int32)
    # small integers: every sum is exact in any order
    x = torch.randint(1, 4, (T, d), generator=g).to(dt)
    r = torch.randint(1, 4, (T * k, d), generator=g).to(dt)
    r[pos[0], d - 1] = INF
    r[pos[k], d - 1] = -INF
    r[pos[2 * k + 1], d - 8] = INF
    r[pos[3 * k], d - 1] = float("nan")
    x[4, d - 1] = INF
    x[5, d - 8] = -INF
    p, xn, rn = pos.numpy(), f64(x), f64(r)
    ref = orow.pair_products(xn, rn, p, k)
    assert np.isposinf(ref[0, 0]) and np.isneginf(ref[1, 0]) and np.isposinf(ref[2, 1]) and np.isnan(ref[3, 0])
    pos, x, r = pos.to(DEV), x.to(DEV), r.to(DEV)
    dw, rows, dx = torch.full((T, k), 7.0, device=DEV), torch.empty_like(r), torch.empty_like(x)
    moe.moe_unpermute_backward_into(x, pos, k, rows, None, r, dw)
    same(dw, ref)
    same(rows, orow.permute(xn, p, k, T * k))
    dw.fill_(7.0)
    moe.moe_permute_backward_into(r, pos, k, dx, None, x, dw)
    same(dw, ref)
    same(dx, orow.unpermute(rn, p, k))
