"""Gated feed-forward blocks at sizes that take each tile shape in each product: 256 x 256,
128 x 256, 128 x 128 and 64 x 256 tiles, and the products of few rows."""
import numpy as np
import pytest

from gated_helpers import inputs, offsets_of
from gpu_helpers import say
from test_gpu_gated_ffn import check_backward, check_forward

import torch

pytestmark = pytest.mark.gpu


def uneven(R, E):
    """R rows on E experts, some with none, the first ones with the most."""
    rng = np.random.default_rng(R + E)
    p = 1.0 / np.sqrt(np.arange(1, E + 1))
    p[rng.permutation(E)[:E // 5]] = 0
    return rng.multinomial(R, p / p.sum()).tolist()


@pytest.mark.parametrize("R,E,d,I", [(9000, 4, 1032, 1544), (12000, 5, 264, 2056), (2000, 40, 264, 520),
                                     (40, 13, 264, 8200), (4096, 1, 512, 2048), (32, 40, 56, 1032),
                                     (3860, 40, 1336, 32), (36, 3, 32, 32)])
@pytest.mark.parametrize("dtype,act,p", [("bf16", "silu", 0.2), ("fp16", "gelu", 0.0)])
def test_tile_shapes(R, E, d, I, dtype, act, p):
    say(f"gated ffn R={R} E={E} d={d} I={I} {dtype}")
    off = None if E == 1 else offsets_of(uneven(R, E))
    x = inputs(R, E, d, I, dtype, seed=R)
    _, h, gu = check_forward(x, off, act, p, dtype)
    check_backward(x, gu, h, off, act, p, dtype)


@pytest.mark.parametrize("counts", [[300] + [0] * 39, [0] * 39 + [300], [1] * 20 + [0] * 19 + [280],
                                    [17, 16, 15, 33, 0, 1]])
def test_few_rows_on_average_many_on_one(counts):
    """The products of few rows where one expert has more than sixteen."""
    say(f"gated ffn counts={str(counts)[:40]}")
    x = inputs(sum(counts), len(counts), 72, 40, "bf16", seed=21)
    _, h, gu = check_forward(x, offsets_of(counts), "silu", 0.3, "bf16")
    check_backward(x, gu, h, offsets_of(counts), "silu", 0.3, "bf16")


def test_same_bits_every_time():
    """Twenty calls at sizes with every kind of wait between tiles, the same bits each time."""
    import w4a16_grouped_expert_amd as moe
    say("gated ffn repeated")
    counts = [700, 0, 260, 1, 999, 40]
    off = torch.from_numpy(offsets_of(counts)).cuda()
    x = inputs(sum(counts), 6, 520, 264, "bf16", seed=22)
    first = None
    for _ in range(20):
        y, h, gu = moe.moe_gated_ffn(x["rows"], x["w13"], x["w2"], off, save=True)
        g = moe.moe_gated_ffn_backward(x["dy"], x["rows"], x["w13"], x["w2"], gu, h, off)
        now = [y, h, gu, g.drows, g.dw13, g.dw2]
        first = first or now
        for a, b in zip(first, now):
            assert torch.equal(a, b)


def test_rows_far_apart():
    """Rows at the largest stride, 2^20 elements: offsets past 2^32 bytes in every row tensor."""
    import w4a16_grouped_expert_amd as moe
    from gated_helpers import backward_bounds, forward_bounds
    from rows_helpers import assert_near, f64
    counts, d, I = [1500, 0, 900], 72, 40
    say("gated ffn rows far apart")
    R, off = sum(counts), offsets_of(counts)
    x = inputs(R, 3, d, I, "bf16", seed=23)

    def far(n, values=None):
        t = torch.empty((R, 1 << 20), dtype=torch.bfloat16, device="cuda")[:, :n]
        if values is not None:
            t.copy_(values)
        return t

    rows, dy = far(d, x["rows"]), far(d, x["dy"])
    y, h, gu, drows = far(d), far(I), far(2 * I), far(d)
    dev_off = torch.from_numpy(off).cuda()
    moe.moe_gated_ffn_into(rows, x["w13"], x["w2"], y, h, dev_off, gu)
    grads = moe.GatedFfnGrads(drows, torch.empty_like(x["w13"]), torch.empty_like(x["w2"]))
    ws = moe.alloc_gated_ffn_workspace(R, d, I, 3, "cuda")
    moe.moe_gated_ffn_backward_into(dy, rows, x["w13"], x["w2"], gu, h, grads, ws, dev_off)
    ref, bound = forward_bounds(x, off, "silu", None, "bf16")
    for name, got, r, b in zip(("y", "h", "gu"), (y, h, gu), ref, bound):
        assert_near(name, got, r, b)
    ref, bound = backward_bounds(x, f64(gu), f64(h), off, "silu", None, "bf16")
    for name, r, b in zip(("drows", "dw13", "dw2"), ref, bound):
        assert_near(name, getattr(grads, name), r, b)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_saturated_activations(act):
    """Projections where the activation and its slope are 0, 1 or the projection itself."""
    say(f"gated ffn saturated {act}")
    x = inputs(40, 1, 64, 72, "bf16", seed=24)
    _, h, gu = check_forward(x, None, act, 0.0, "bf16")
    values = torch.tensor([-1e30, -1e9, -3e4, -90.0, -20.0, -4.0, -0.5, 0.0, 1e-30, 0.5, 4.0, 20.0, 90.0, 3e4, 1e9, 1e20],
                          device="cuda").bfloat16()
    gu[:, :72] = values.repeat(180)[:2880].reshape(40, 72)
    gu[:, 72:] = 0.25
    x["dy"] = x["dy"] * 2.0 ** -60  # (gradients of u up to 1e20 times it stay in range)
    check_backward(x, gu, h, None, act, 0.0, "bf16")


def test_two_streams_at_once():
    """Forward and backward calls on two streams at the same time, each with its own buffers."""
    import w4a16_grouped_expert_amd as moe
    say("gated ffn on two streams")
    counts = [[300, 0, 900], [17, 640, 1]]
    cases = []
    for i, c in enumerate(counts):
        x = inputs(sum(c), 3, 264, 520, "bf16", seed=30 + i)
        off = torch.from_numpy(offsets_of(c)).cuda()
        drop = moe.Dropout(0.2, torch.tensor([5 + i, 7], device="cuda"), i)
        y, h, gu = moe.moe_gated_ffn(x["rows"], x["w13"], x["w2"], off, dropout=drop, save=True)
        g = moe.moe_gated_ffn_backward(x["dy"], x["rows"], x["w13"], x["w2"], gu, h, off, dropout=drop)
        cases.append((x, off, drop, (y, h, gu), (g.drows, g.dw13, g.dw2)))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, (x, off, drop, fwd, _) in enumerate(cases):
            out = moe.moe_gated_ffn(x["rows"], x["w13"], x["w2"], off, dropout=drop, save=True, stream=streams[i])
            g = moe.moe_gated_ffn_backward(x["dy"], x["rows"], x["w13"], x["w2"], fwd[2], fwd[1], off, dropout=drop,
                                           stream=streams[i])
            got[i].append((*out, g.drows, g.dw13, g.dw2))
    torch.cuda.synchronize()
    for i, case in enumerate(cases):
        for outputs in got[i]:
            for a, b in zip(outputs, (*case[3], *case[4])):
                assert torch.equal(a, b)


@pytest.mark.parametrize("R,E", [(20, 3), (100, 1), (5000, 2)])
def test_rows_that_no_expert_has(R, E):
    """Offsets of zeros: nothing is written but the weights' gradients, which are zero."""
    import w4a16_grouped_expert_amd as moe
    say(f"gated ffn R={R} without an expert")
    x = inputs(R, E, 136, 72, "bf16", seed=40)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    out = [torch.full((R, n), 5.0, dtype=torch.bfloat16, device="cuda") for n in (136, 72, 144, 136)]
    moe.moe_gated_ffn_into(x["rows"], x["w13"], x["w2"], out[0], out[1], off, out[2])
    grads = moe.GatedFfnGrads(out[3], torch.full_like(x["w13"], 5.0), torch.full_like(x["w2"], 5.0))
    ws = moe.alloc_gated_ffn_workspace(R, 136, 72, E, "cuda")
    moe.moe_gated_ffn_backward_into(x["dy"], x["rows"], x["w13"], x["w2"], out[2], out[1], grads, ws, off)
    assert all(bool((t == 5.0).all()) for t in out)
    assert not grads.dw13.any() and not grads.dw2.any()
