"""Gated feed-forward blocks and their gradient on the GPU against the float64 reference."""
import numpy as np
import pytest
import torch

import w4a16_grouped_expert_amd as moe
from oracle import gated

from gated_helpers import DEV, SEED, STEP, backward_bounds, forward_bounds, inputs, offsets_of
from gpu_helpers import say
from rows_helpers import TYPES, assert_near, f64, wide

pytestmark = pytest.mark.gpu
ACTS = {"silu": moe.ACT_SILU, "gelu": moe.ACT_GELU}


def dropout_of(p, site=2):
    state = torch.tensor([SEED, STEP], device=DEV)
    return moe.Dropout(p, state, site) if p else None


def factor_of(p, R, I, site=2):
    return gated.drop_factor(p, SEED, STEP, site, R, I) if p else None


def check_forward(x, off, act, p, dtype, save=True):
    R, I = x["rows"].shape[0], x["w2"].shape[2]
    dev_off = None if off is None else torch.from_numpy(off).to(DEV)
    y, h, gu = moe.moe_gated_ffn(x["rows"], x["w13"], x["w2"], dev_off, ACTS[act], dropout_of(p), save=True)
    ref, bound = forward_bounds(x, off, act, factor_of(p, R, I), dtype)
    for name, got, r, b in zip(("y", "h", "gu"), (y, h, gu), ref, bound):
        assert_near(name, got, r, b)
    if p:
        assert np.array_equal(f64(h)[factor_of(p, R, I) == 0], np.zeros((factor_of(p, R, I) == 0).sum()))
    if not p:
        assert torch.equal(moe.moe_gated_ffn(x["rows"], x["w13"], x["w2"], dev_off, ACTS[act]), y)
    return y, h, gu


def check_backward(x, gu, h, off, act, p, dtype):
    R, I = x["rows"].shape[0], x["w2"].shape[2]
    dev_off = None if off is None else torch.from_numpy(off).to(DEV)
    g = moe.moe_gated_ffn_backward(x["dy"], x["rows"], x["w13"], x["w2"], gu, h, dev_off, ACTS[act], dropout_of(p))
    ref, bound = backward_bounds(x, f64(gu), f64(h), off, act, factor_of(p, R, I), dtype)
    for name, r, b in zip(("drows", "dw13", "dw2"), ref, bound):
        assert_near(name, getattr(g, name), r, b)
    return g


# rows per expert (None: one dense block of that many rows), d, I
SHAPES = [
    (1, 8, 8), (1, 64, 64), (3, 256, 128), (16, 128, 264), (17, 1000, 712), (129, 72, 136), (300, 264, 1032),
    ([1], 64, 72), ([0, 5, 0], 128, 64), ([16, 1, 0, 31, 17], 192, 200), ([128, 127, 129, 1, 0, 255, 257], 136, 264),
    ([600, 3, 900], 72, 80), ([1] * 70, 64, 64), ([0] * 99 + [40] + [0] * 50, 64, 128), ([2048, 2048], 64, 72),
]


@pytest.mark.parametrize("shape", SHAPES, ids=[str(s)[:40] for s in SHAPES])
@pytest.mark.parametrize("dtype,act,p", [("bf16", "silu", 0.0), ("fp16", "gelu", 0.3)])
def test_forward_and_backward(shape, dtype, act, p):
    counts, d, I = shape
    say(f"gated ffn counts={str(counts)[:60]} d={d} I={I} {dtype} {act} p={p}")
    dense = isinstance(counts, int)
    off = None if dense else offsets_of(counts)
    R, E = (counts, 1) if dense else (sum(counts), len(counts))
    x = inputs(R, E, d, I, dtype)
    _, h, gu = check_forward(x, off, act, p, dtype)
    check_backward(x, gu, h, off, act, p, dtype)


@pytest.mark.parametrize("dtype,act,p", [("bf16", "gelu", 0.5), ("fp16", "silu", 0.0)])
def test_long_sums(dtype, act, p):
    """Thousands of channels and rows in every sum."""
    say(f"gated ffn long sums {dtype} {act}")
    counts = [4000, 33]
    x = inputs(sum(counts), 2, 2056, 264, dtype, seed=4)
    _, h, gu = check_forward(x, offsets_of(counts), act, p, dtype)
    check_backward(x, gu, h, offsets_of(counts), act, p, dtype)
    x = inputs(9, 1, 264, 4104, dtype, seed=5)
    _, h, gu = check_forward(x, None, act, p, dtype)
    check_backward(x, gu, h, None, act, p, dtype)


def strided(t, pad):
    """The same values as rows of a wider tensor, 16-byte aligned, NaN beside them."""
    R, n = t.shape
    big = torch.full((R, n + pad), float("nan"), dtype=t.dtype, device=t.device)
    big[:, :n].copy_(t)
    return big[:, :n]


@pytest.mark.parametrize("counts", [[5, 0, 12], [140, 260]])
def test_strides_and_rows_behind(counts):
    """Strided tensors with NaN between the rows; rows behind the last expert's are neither
    read (NaN there) nor written."""
    say(f"gated ffn strides {counts}")
    d, I, behind = 72, 136, 20
    used = sum(counts)
    R, E = used + behind, len(counts)
    off = offsets_of(counts)
    x = inputs(R, E, d, I, "bf16", seed=7)
    x["rows"][used:] = float("nan")
    x["dy"][used:] = float("nan")
    rows, dy = strided(x["rows"], 24), strided(x["dy"], 8)
    dev_off = torch.from_numpy(off).to(DEV)
    out = {q: strided(torch.full((R, n), 7.0, dtype=torch.bfloat16, device=DEV), pad)
           for q, n, pad in (("y", d, 8), ("h", I, 16), ("gu", 2 * I, 40), ("drows", d, 32))}
    moe.moe_gated_ffn_into(rows, x["w13"], x["w2"], out["y"], out["h"], dev_off, out["gu"])
    grads = moe.GatedFfnGrads(out["drows"], torch.full_like(x["w13"], 7.0), torch.full_like(x["w2"], 7.0))
    ws = moe.alloc_gated_ffn_workspace(R, d, I, E, DEV)
    ws.fill_(255)   # NaN where it is not written
    gu_in, h_in = strided(out["gu"].clone(), 40), strided(out["h"].clone(), 16)
    gu_in[used:] = float("nan")
    h_in[used:] = float("nan")
    moe.moe_gated_ffn_backward_into(dy, rows, x["w13"], x["w2"], gu_in, h_in, grads, ws, dev_off)
    small = {q: x[q][:used] if q in ("rows", "dy") else x[q] for q in x}
    ref, bound = forward_bounds(small, off, "silu", None, "bf16")
    for q, r, b in zip(("y", "h", "gu"), ref, bound):
        assert_near(q, out[q][:used], r, b)
        assert bool((out[q][used:] == 7.0).all())
    ref, bound = backward_bounds(small, f64(out["gu"][:used]), f64(out["h"][:used]), off, "silu", None, "bf16")
    for q, got, r, b in zip(("drows", "dw13", "dw2"), (out["drows"][:used], grads.dw13, grads.dw2), ref, bound):
        assert_near(q, got, r, b)
    assert bool((out["drows"][used:] == 7.0).all())


def test_no_rows():
    say("gated ffn without rows")
    x = inputs(0, 3, 64, 72, "bf16")
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    y, h, gu = moe.moe_gated_ffn(x["rows"], x["w13"], x["w2"], off, save=True)
    assert y.shape == (0, 64) and h.shape == (0, 72) and gu.shape == (0, 144)
    g = moe.moe_gated_ffn_backward(x["dy"], x["rows"], x["w13"], x["w2"], gu, h, off)
    assert not g.dw13.any() and not g.dw2.any() and g.drows.shape == (0, 64)


def test_parts_of_a_gradient():
    """Each gradient alone, with the inputs it needs, has the bits of the whole call's."""
    say("gated ffn parts of a gradient")
    counts = [40, 7, 90]
    off = torch.from_numpy(offsets_of(counts)).to(DEV)
    x = inputs(sum(counts), 3, 136, 72, "fp16", seed=8)
    _, h, gu = moe.moe_gated_ffn(x["rows"], x["w13"], x["w2"], off, save=True)
    all_ = moe.moe_gated_ffn_backward(x["dy"], x["rows"], x["w13"], x["w2"], gu, h, off)
    ws = moe.alloc_gated_ffn_workspace(sum(counts), 136, 72, 3, DEV)
    for name in ("drows", "dw13", "dw2"):
        g = moe.GatedFfnGrads(**{name: torch.empty_like(getattr(all_, name))})
        moe.moe_gated_ffn_backward_into(x["dy"], x["rows"], x["w13"], x["w2"], None if name == "dw2" else gu,
                                        h if name == "dw2" else None, g, None if name == "dw2" else ws, off)
        assert torch.equal(getattr(g, name), getattr(all_, name)), name
    # h alone
    only = torch.empty_like(h)
    moe.moe_gated_ffn_into(x["rows"], x["w13"], None, None, only, off)
    assert torch.equal(only, h)


def test_offsets_out_of_range_stay_inside():
    """Offsets that are no partition of the rows: nothing outside the tensors is touched and
    the rows that no expert names keep their contents."""
    say("gated ffn offsets out of range")
    x = inputs(40, 3, 64, 72, "bf16", seed=9)
    off = torch.tensor([-5, 10, 8, 1000], dtype=torch.int32, device=DEV)  # rows 0..9, none, 8..39
    y, h, gu = moe.moe_gated_ffn(x["rows"], x["w13"], x["w2"], off, save=True)
    ref, bound = forward_bounds(x, np.array([0, 10, 10, 40]), "silu", None, "bf16")
    keep = np.r_[0:8, 10:40]  # rows 8 and 9 belong to two experts
    assert_near("y", y[keep], ref[0][keep], bound[0][keep])


def test_graph_streams_and_determinism():
    """A step captured and replayed between eager calls; the masks follow the state's step."""
    say("gated ffn in a graph")
    counts = [100, 0, 31, 260]
    R, E, d, I, p = sum(counts), 4, 136, 200, 0.25
    off = torch.from_numpy(offsets_of(counts)).to(DEV)
    x = inputs(R, E, d, I, "bf16", seed=10)
    state = torch.tensor([SEED, STEP], device=DEV)
    drop = moe.Dropout(p, state, 2)
    y, h, gu = (torch.empty(R, n, dtype=torch.bfloat16, device=DEV) for n in (d, I, 2 * I))
    grads = moe.GatedFfnGrads(torch.empty_like(x["rows"]), torch.empty_like(x["w13"]), torch.empty_like(x["w2"]))
    ws = moe.alloc_gated_ffn_workspace(R, d, I, E, DEV)

    def step():
        moe.moe_gated_ffn_into(x["rows"], x["w13"], x["w2"], y, h, off, gu, dropout=drop)
        moe.moe_gated_ffn_backward_into(x["dy"], x["rows"], x["w13"], x["w2"], gu, h, grads, ws, off, dropout=drop)

    outputs = (y, h, gu, grads.drows, grads.dw13, grads.dw2)
    expect = []
    for s in range(3):
        state[1] = STEP + s
        step()
        torch.cuda.synchronize()
        expect.append([t.clone() for t in outputs])
    assert not torch.equal(expect[0][1], expect[1][1])
    state[1] = STEP
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for s in (0, 1, 2, 0):
        for t in outputs:
            t.fill_(3.0)
        state[1] = STEP + s
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(outputs, expect[s]):
            assert torch.equal(got, want), s
        step()
        torch.cuda.synchronize()
        for got, want in zip(outputs, expect[s]):
            assert torch.equal(got, want), s
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = moe.moe_gated_ffn_backward(x["dy"], x["rows"], x["w13"], x["w2"], gu, h, off, dropout=drop, stream=side)
    side.synchronize()
    assert torch.equal(other.drows, expect[0][3]) and torch.equal(other.dw13, expect[0][4])


def test_mask_is_dropouts():
    """The mask on h is the one that moe_dropout draws for a tensor of h's shape."""
    say("gated ffn mask")
    R, d, I = 70, 64, 200
    x = inputs(R, 1, d, I, "bf16", seed=11)
    drop = dropout_of(0.4, site=5)
    h = torch.empty(R, I, dtype=torch.bfloat16, device=DEV)
    moe.moe_gated_ffn_into(x["rows"], x["w13"][0], None, None, h, dropout=drop)
    mask = moe.moe_dropout(torch.ones_like(h), drop)
    assert torch.equal(h == 0, mask == 0)


def test_binding_refusals():
    say("gated ffn refusals of the binding")
    x = inputs(8, 2, 64, 72, "bf16")
    off = torch.tensor([0, 3, 8], dtype=torch.int32, device=DEV)
    call = moe.moe_gated_ffn
    call(x["rows"], x["w13"], x["w2"], off)
    with pytest.raises(TypeError):
        call(x["rows"].half(), x["w13"], x["w2"], off)
    with pytest.raises(TypeError):
        call(x["rows"], x["w13"], x["w2"], off.long())
    with pytest.raises(ValueError):
        call(x["rows"], x["w13"], x["w2"], off[:2])
    with pytest.raises(ValueError):
        call(x["rows"], x["w13"][:, :, :32], x["w2"], off)
    with pytest.raises(ValueError):
        call(x["rows"], x["w13"], x["w2"][:1], off)
    with pytest.raises(moe.MoeError, match="expert_offsets"):
        call(x["rows"], x["w13"], x["w2"])
    with pytest.raises(moe.MoeError, match="bad dtype"):
        call(x["rows"].float(), x["w13"].float(), x["w2"].float(), off)
    with pytest.raises(moe.MoeError, match="aligned"):
        call(wide(x["rows"], 1, 7), x["w13"], x["w2"], off)
    with pytest.raises(ValueError):
        call(x["rows"], x["w13"], x["w2"], off.cpu())
    with pytest.raises(moe.MoeError, match="state"):
        call(x["rows"], x["w13"], x["w2"], off, dropout=moe.Dropout(0.5))
