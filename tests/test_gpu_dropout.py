"""Dropout with the residual's addition on the GPU against the float64 reference: the mask
exactly, the values within two float32 roundings and one to the type."""
import numpy as np
import pytest
import torch

import w4a16_grouped_expert_amd as moe
from oracle import gated

from gated_helpers import DEV, SEED, STEP
from gpu_helpers import say
from rows_helpers import TYPES, U32, assert_near, f64, half_step, wide

pytestmark = pytest.mark.gpu


def state_of(seed=SEED, step=STEP):
    return torch.tensor([seed, step], device=DEV)


def check(got, x, factor, residual, dtype):
    ref = gated.dropout(f64(x), factor, None if residual is None else f64(residual))
    mag = np.abs(f64(x) * factor) + (0 if residual is None else np.abs(f64(residual)))
    # the scale, the product and the sum: three float32 roundings at most
    assert_near("out", got, ref, 3 * U32 * mag + half_step(TYPES[dtype], ref))


@pytest.mark.parametrize("T,d", [(1, 1), (3, 5), (1, 8), (2, 9), (7, 16), (5, 100), (33, 1111), (1, 4099), (4097, 24),
                                 (260, 2048), (2, 70000)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("p,residual", [(0.1, True), (0.5, False), (0.0, True), (1.0, False)])
def test_values(T, d, dtype, p, residual):
    say(f"dropout T={T} d={d} {dtype} p={p} residual={residual}")
    g = torch.Generator().manual_seed(T * 7 + d)
    x = torch.randn(T, d, generator=g).to(TYPES[dtype]).to(DEV)
    r = torch.randn(T, d, generator=g).to(TYPES[dtype]).to(DEV) if residual else None
    drop = moe.Dropout(p, state_of() if p else None, site=2047)
    out = moe.moe_dropout(x, drop, r)
    factor = gated.drop_factor(p, SEED, STEP, 2047, T, d)
    check(out, x, factor, r, dtype)
    # in place, over x and over the residual
    y = x.clone()
    assert moe.moe_dropout_into(y, drop, y, r) is y and torch.equal(y, out)
    if residual:
        s = r.clone()
        moe.moe_dropout_into(x, drop, s, s)
        assert torch.equal(s, out)
    # rows with another stride, off every alignment
    o = wide(torch.zeros_like(x), 1, 2)
    moe.moe_dropout_into(wide(x, 3, 2), drop, o, None if r is None else wide(r, 1, 4))
    assert torch.equal(o, out)


@pytest.mark.parametrize("seed,step,site", [(0, 0, 0), (-1, -1, 2047), (1 << 62, 1, 1), (7, 1 << 40, 100)])
def test_states(seed, step, site):
    say(f"dropout seed={seed} step={step} site={site}")
    x = torch.ones(50, 300, device=DEV)
    out = moe.moe_dropout(x, moe.Dropout(0.3, state_of(seed, step), site))
    factor = gated.drop_factor(0.3, seed, step, site, 50, 300)
    assert np.array_equal(f64(out), factor.astype(np.float32).astype(np.float64))


def test_dropped_elements_reach_nothing():
    say("dropout of infinities and NaN")
    factor = gated.drop_factor(0.5, SEED, STEP, 0, 20, 333)
    for dtype in TYPES:
        x = torch.from_numpy(np.where(factor > 0, 1.0, np.nan)).to(TYPES[dtype]).to(DEV)
        x[::2][torch.isnan(x[::2])] = float("inf")
        r = torch.full_like(x, 0.25)
        out = moe.moe_dropout(x, moe.Dropout(0.5, state_of()), r)
        assert np.array_equal(f64(out), np.where(factor > 0, 2.25, 0.25))
        # (and kept ones do)
        y = torch.full_like(x, float("inf"))
        assert np.array_equal(np.isinf(f64(moe.moe_dropout(y, moe.Dropout(0.5, state_of()), r))), factor > 0)


def test_gradient_is_the_same_mask():
    say("dropout gradient")
    T, d = 65, 520
    dout = torch.randn(T, d, device=DEV)
    drop = moe.Dropout(0.2, state_of(), 4)
    dx = moe.moe_dropout(dout, drop)
    keep = moe.moe_dropout(torch.ones(T, d, device=DEV), drop)
    # one product's rounding
    assert_near("dx", dx, f64(dout) * f64(keep), U32 * np.abs(f64(dout) * f64(keep)))


def test_broadcast_rows_and_many_elements():
    """One row for all by a stride of zero; element offsets past 2^31."""
    say("dropout of a broadcast row, long tensor")
    row = torch.randn(1, 24, device=DEV).bfloat16()
    x = row.expand(1000, 24)
    out = moe.moe_dropout(x, moe.Dropout(0.3, state_of(), 1))
    check(out, x, gated.drop_factor(0.3, SEED, STEP, 1, 1000, 24), None, "bf16")
    T, d = (1 << 20) + 3, 2200    # 2.3e9 elements
    big = torch.ones(1, d, dtype=torch.bfloat16, device=DEV).expand(T, d)
    out = moe.moe_dropout(big, moe.Dropout(0.3, state_of(), 1))
    for r0 in (0, 976128, T - 5):  # 976128 * 2200 is just below 2^31
        factor = gated.drop_factor(0.3, SEED, STEP, 1, 5, d, first_row=r0)
        check(out[r0:r0 + 5], big[r0:r0 + 5], factor, None, "bf16")


def test_graph_follows_the_step():
    say("dropout in a graph")
    x, state = torch.randn(100, 264, device=DEV).half(), state_of()
    out = torch.empty_like(x)
    drop = moe.Dropout(0.3, state, 1)
    moe.moe_dropout_into(x, drop, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_dropout_into(x, drop, out)
    for s in (0, 5, 1, 0):
        state[1] = STEP + s
        graph.replay()
        torch.cuda.synchronize()
        check(out, x, gated.drop_factor(0.3, SEED, STEP + s, 1, 100, 264), None, "fp16")
        assert torch.equal(moe.moe_dropout(x, drop), out)


def test_streams():
    say("dropout on two streams")
    x = torch.randn(512, 2048, device=DEV)
    drops = [moe.Dropout(0.3, state_of(step=s), 1) for s in range(2)]
    want = [moe.moe_dropout(x, d) for d in drops]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [moe.moe_dropout(x, d, stream=s) for d, s in zip(drops, streams) for _ in range(3)]
    torch.cuda.synchronize()
    for i, t in enumerate(got):
        assert torch.equal(t, want[i // 3])
