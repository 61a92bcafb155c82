"""The gradient of moe_block_norm with infinite and NaN elements: each reaches what the
formulas give it to and nothing else."""
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
# rows by parts of a wavefront, by one and by several, whose last pieces overlap
WIDTHS = [9, 40, 520, 1111, 2600, 4104]


def make(T, d, dtype, gate, norm_out, norm_in, seed=0):
    g = torch.Generator().manual_seed(seed + 31 * T + d)

    def rand(*shape):
        # one to two in size, of either sign: no zeros, so that an infinite factor shows
        v = 1 + torch.rand(*shape, generator=g)
        return (v * (1 - 2 * torch.randint(0, 2, shape, generator=g))).to(dtype).to(DEV)

    shape = {"none": None, "channel": (d,), "token": (T, 1), "full": (T, d)}[gate]
    norm = moe.BlockNorm(norm_in=rand(d) if norm_in else None, norm_out=rand(d) if norm_out else None,
                         gate=None if shape is None else rand(*shape), residual_scale=0.5, eps=1e-5)
    return norm, rand(T, d), rand(T, d), rand(T, d), rand(T, d)


def reference(norm, x, y, dh, dn):
    """Without dn: the gradient of h alone, as if there were no norm before the next block
    (zeros in its place would meet the infinite statistics of an infinite h)."""
    v_in = None if dn is None else f64(norm.norm_in)
    with np.errstate(invalid="ignore"):
        return orow.block_norm_backward(f64(x), f64(y), v_in, f64(norm.norm_out), f64(norm.gate), norm.residual_scale,
                                        norm.eps, f64(dh), f64(dn))


def same_kind(name, got, ref):
    """Both finite, or the same infinity, or both NaN."""
    got = f64(got)
    for kind in (np.isfinite, np.isposinf, np.isneginf, np.isnan):
        np.testing.assert_array_equal(kind(got), kind(ref), err_msg=f"{name} {kind.__name__}")


def same_bits(name, a, b, but=None):
    """Equal but for the entries that `but` (a boolean tensor) names."""
    keep = torch.ones_like(a, dtype=torch.bool) if but is None else ~but
    assert torch.equal(a[keep], b[keep]), name


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("gate", ["channel", "token", "full"])
@pytest.mark.parametrize("d", WIDTHS)
def test_infinite_gradient_in_the_last_column(d, gate, type_):
    say(f"block norm gradient, infinite dh in the last columns, d={d} {gate} {type_}")
    T = 5
    for norm_out in (True, False):
        norm, x, y, dh, _ = make(T, d, TYPES[type_], gate, norm_out, False)
        plain = moe.moe_block_norm_backward(norm, x, y, dh)
        bad = dh.clone()
        bad[1, d - 1], bad[3, d - 8] = INF, -INF
        got = moe.moe_block_norm_backward(norm, x, y, bad)
        ref = reference(norm, x, y, bad, None)
        for q, r in ref.items():
            same_kind(f"{q} norm_out={norm_out}", getattr(got, q), r)
        rows = torch.zeros(T, d, dtype=torch.bool, device=DEV)
        at = rows.clone()
        rows[1], rows[3] = True, True
        at[1, d - 1], at[3, d - 8] = True, True
        same_bits("dx", got.dx, plain.dx, at)
        same_bits("dy", got.dy, plain.dy, rows if norm_out else at)


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("d", WIDTHS)
def test_infinite_gradient_of_the_next_norm(d, type_):
    say(f"block norm gradient, infinite dn in the last columns, d={d} {type_}")
    T = 4
    norm, x, y, dh, dn = make(T, d, TYPES[type_], "channel", True, True)
    plain = moe.moe_block_norm_backward(norm, x, y, dh, dn)
    bad = dn.clone()
    bad[0, d - 1], bad[2, d - 8] = INF, -INF
    got = moe.moe_block_norm_backward(norm, x, y, dh, bad)
    ref = reference(norm, x, y, dh, bad)
    same_kind("dx", got.dx, ref["dx"])
    same_kind("dnorm_in", got.dnorm_in, ref["dnorm_in"])
    rows = torch.zeros(T, d, dtype=torch.bool, device=DEV)
    rows[0], rows[2] = True, True
    same_bits("dx", got.dx, plain.dx, rows)
    same_bits("dy", got.dy, plain.dy, rows)


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("d", WIDTHS)
def test_infinite_weights_in_the_last_column(d, type_):
    """An infinite weight of the norm behind the block, of the next norm, or of the gate."""
    say(f"block norm gradient, infinite weights in the last columns, d={d} {type_}")
    for which in ("norm_out", "norm_in", "gate"):
        norm, x, y, dh, dn = make(3, d, TYPES[type_], "channel", True, True)
        getattr(norm, which)[d - 1] = INF
        if which == "norm_in":
            got, ref = moe.moe_block_norm_backward(norm, x, y, dh, dn), reference(norm, x, y, dh, dn)
            same_kind("norm_in dx", got.dx, ref["dx"])
            same_kind("norm_in dnorm_in", got.dnorm_in, ref["dnorm_in"])
        else:  # h is infinite, and without dn not used
            got, ref = moe.moe_block_norm_backward(norm, x, y, dh), reference(norm, x, y, dh, None)
            same_kind(f"{which} dy", got.dy, ref["dy"])
            # A column of dgate is the sum of D yn over the rows times norm_out, one of dnorm_out
            # the same times the gate: an infinite factor times the sum is infinite where the sum of
            # infinite terms of either sign is NaN, so the kind in that column is left open.
            for q in ("dgate", "dnorm_out"):
                np.testing.assert_array_equal(np.isfinite(f64(getattr(got, q))), np.isfinite(ref[q]), err_msg=q)


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("d", WIDTHS + [64, 2048])
def test_infinite_block_output_without_dn(d, gate, type_):
    """Without dn the statistics of h are not used, and without norm_out dy does not depend
    on y: an infinite or NaN element of y reaches the gate's gradient alone."""
    say(f"block norm gradient, infinite y without dn, d={d} {gate} {type_}")
    T = 6
    for norm_in in (False, True):
        norm, x, y, dh, _ = make(T, d, TYPES[type_], gate, False, norm_in)
        plain = moe.moe_block_norm_backward(norm, x, y, dh)
        bad = y.clone()
        bad[1, d // 2], bad[2, d - 1], bad[4, 0] = INF, -INF, float("nan")
        got = moe.moe_block_norm_backward(norm, x, bad, dh)
        same_bits("dx", got.dx, plain.dx)
        same_bits("dy", got.dy, plain.dy)
        if norm_in:
            assert not got.dnorm_in.any()
        if gate != "none":
            ref = reference(norm, x, bad, dh, None)["dgate"]
            same_kind("dgate", got.dgate, ref)
            same_bits("dgate", got.dgate, plain.dgate, torch.from_numpy(~np.isfinite(ref)).to(DEV))


@pytest.mark.parametrize("d", WIDTHS)
def test_block_output_not_a_number_behind_a_norm(d):
    """Without dn, dx is residual_scale dh whatever the block's output holds."""
    say(f"block norm gradient, NaN in y behind a norm, d={d}")
    norm, x, y, dh, _ = make(4, d, torch.float32, "channel", True, True)
    plain = moe.moe_block_norm_backward(norm, x, y, dh)
    y[2, d - 1] = float("nan")
    got = moe.moe_block_norm_backward(norm, x, y, dh)
    same_bits("dx", got.dx, plain.dx)
    rows = torch.zeros(4, d, dtype=torch.bool, device=DEV)
    rows[2] = True
    same_bits("dy", got.dy, plain.dy, rows)
    assert torch.isnan(got.dy[2]).all() and not got.dnorm_in.any()
