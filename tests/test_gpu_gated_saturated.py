"""Gated blocks where the activation and its slope are 0, 1 or the projection itself, and on the
way there: each output depends on one element, so that a large one hides no other."""
import pytest
import torch

import w4a16_grouped_expert_amd as moe

from gpu_helpers import say
from rows_helpers import assert_near, f64
from saturation_helpers import elements, expected, one_hot_call

pytestmark = pytest.mark.gpu
ACTS = {"silu": moe.ACT_SILU, "gelu": moe.ACT_GELU}


# few rows, then tiles of each shape
@pytest.mark.parametrize("R,I", [(3, 72), (16, 40), (120, 200), (600, 264), (4096, 2048)])
@pytest.mark.parametrize("kind,dtype", [("silu", "bf16"), ("silu", "fp16"), ("gelu", "bf16"), ("gelu", "fp16")])
def test_single_elements(R, I, kind, dtype):
    say(f"gated ffn single elements R={R} I={I} {kind} {dtype}")
    g, u, dh = elements(dtype, R, I, seed=R)
    x = one_hot_call(dtype, g, u, dh, "cuda")
    want = expected(kind, dtype, g, u, dh)
    y, h, gu = moe.moe_gated_ffn(x["rows"], x["w13"], x["w2"], activation=ACTS[kind], save=True)
    assert torch.equal(gu, x["gu"])
    assert_near("h", h, *want["h"])
    assert torch.equal(y[:, :I], h) and not y[:, I:].any()
    out = moe.moe_gated_ffn_backward(x["dy"], x["rows"], x["back_w13"], x["w2"], x["gu"], h, activation=ACTS[kind])
    dgu, sums = f64(out.drows), f64(out.dw13)
    for i, name in enumerate(("dg", "du")):
        assert_near(f"drows, {name}", dgu[:, i * I:(i + 1) * I], *want[name])
        assert_near(f"dw13, {name}", sums[i * I:(i + 1) * I, :R].T, *want[name])
    assert not dgu[:, 2 * I:].any() and not sums[:, R:].any()
