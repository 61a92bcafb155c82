"""Infinities and NaN in the dropped places of a gated block: neither the output nor a gradient
sees them."""
import numpy as np
import pytest
import torch

import w4a16_grouped_expert_amd as moe
from oracle import gated

from gated_helpers import DEV, SEED, STEP, inputs, offsets_of
from gpu_helpers import say
from rows_helpers import f64

pytestmark = pytest.mark.gpu
P, SITE = 0.4, 3
# few rows, one tile, tiles of several experts, an expert without rows
COUNTS = [[9], [150], [70, 0, 300, 1], [2000, 2100]]


def dropout():
    return moe.Dropout(P, torch.tensor([SEED, STEP], device=DEV), SITE)


@pytest.mark.parametrize("counts", COUNTS, ids=[str(c) for c in COUNTS])
@pytest.mark.parametrize("dtype,act", [("bf16", "silu"), ("fp16", "gelu")])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_gradient(counts, dtype, act, value):
    """Stored g and u of dropped elements replaced: the gradients keep their bits."""
    say(f"gated ffn gradient with {value} in dropped places, counts={counts} {dtype} {act}")
    R, E, d, I = sum(counts), len(counts), 72, 136
    x = inputs(R, E, d, I, dtype, seed=50)
    off = torch.from_numpy(offsets_of(counts)).to(DEV)
    kind = moe.ACT_SILU if act == "silu" else moe.ACT_GELU
    _, h, gu = moe.moe_gated_ffn(x["rows"], x["w13"], x["w2"], off, kind, dropout(), save=True)
    want = moe.moe_gated_ffn_backward(x["dy"], x["rows"], x["w13"], x["w2"], gu, h, off, kind, dropout())
    dropped = torch.from_numpy(gated.drop_factor(P, SEED, STEP, SITE, R, I) == 0).to(DEV)
    assert 0.3 < dropped.float().mean() < 0.5
    for places in (torch.cat([dropped, dropped & False], dim=1), torch.cat([dropped & False, dropped], dim=1),
                   torch.cat([dropped, dropped], dim=1)):
        bad = gu.masked_fill(places, value)
        got = moe.moe_gated_ffn_backward(x["dy"], x["rows"], x["w13"], x["w2"], bad, h, off, kind, dropout())
        for name in ("drows", "dw13", "dw2"):
            assert torch.equal(getattr(got, name), getattr(want, name)), name


@pytest.mark.parametrize("counts", [[9], [150]])
def test_forward(counts):
    """A row whose projections are all infinite: its dropped elements are zeros."""
    say(f"gated ffn with infinite projections, counts={counts}")
    R, d, I = sum(counts), 72, 136
    x = inputs(R, 1, d, I, "bf16", seed=51)
    x["rows"][3] = float("inf")
    _, h, _ = moe.moe_gated_ffn(x["rows"], x["w13"][0], x["w2"][0], dropout=dropout(), save=True)
    kept = gated.drop_factor(P, SEED, STEP, SITE, R, I) > 0
    assert np.array_equal(np.isfinite(f64(h[3])), ~kept[3]) and not f64(h[3])[~kept[3]].any()
    assert np.isfinite(f64(h)[np.arange(R) != 3]).all()
