"""The range of fp16 in a gated block: h forward, dg and du backward are held in the tensors' type.
Beyond it an element is infinite, and only its own rows of the results see it; small ones keep
the bits that fp16 has for them."""
import pytest
import torch

import w4a16_grouped_expert_amd as moe

from gpu_helpers import say
from saturation_helpers import one_hot_call

pytestmark = pytest.mark.gpu
AT = (2, 5)  # row and column of the element


@pytest.mark.parametrize("R", [12, 100])
def test_beyond_the_range(R):
    say(f"gated ffn fp16 range, R={R}")
    I = 40
    g, u, dh = (torch.full((R, I), v).half() for v in (64.0, 2.0, 3.0))   # h = 128, dg = 6, du = 192
    fine = one_hot_call("fp16", g, u, dh, "cuda")
    big_u, big_dh = u.clone(), dh.clone()
    big_u[AT], big_dh[AT] = 2048.0, 1100.0                                # h = 131072; dg = 2200, du = 70400
    big = one_hot_call("fp16", g, big_u, dh, "cuda")
    y, h, gu = moe.moe_gated_ffn(big["rows"], big["w13"], big["w2"], save=True)
    want, want_h, fine_gu = moe.moe_gated_ffn(fine["rows"], fine["w13"], fine["w2"], save=True)
    others = [r for r in range(R) if r != AT[0]]
    assert torch.equal(gu, big["gu"]) and bool(torch.isinf(h[AT]))
    assert torch.equal(y[others], want[others]) and not torch.isfinite(y[AT]).item()
    args = (fine["rows"], fine["back_w13"], fine["w2"], fine_gu, want_h)
    got = moe.moe_gated_ffn_backward(one_hot_call("fp16", g, u, big_dh, "cuda")["dy"], *args)
    want = moe.moe_gated_ffn_backward(fine["dy"], *args)
    assert float(want.drows[AT[0], I + AT[1]]) == 192.0
    assert not torch.isfinite(got.drows[AT[0], I + AT[1]]).item()
    assert torch.equal(got.drows[others], want.drows[others])
    columns = [j for j in range(2 * I) if j != I + AT[1]]
    assert not torch.isfinite(got.dw13[I + AT[1], AT[0]]).item()
    assert torch.equal(got.dw13[columns][:, others], want.dw13[columns][:, others])
    # (dg of that element is in range, and its row is right)
    assert float(got.dw13[AT[1], AT[0]]) == 2200.0


@pytest.mark.parametrize("R", [12, 100])
def test_small_values(R):
    """du = 2^-24 times whole numbers is exact; below half a step of it nothing is left."""
    say(f"gated ffn fp16 small values, R={R}")
    I = 40
    g, u = torch.full((R, I), 64.0).half(), torch.zeros(R, I).half()
    du = (torch.arange(R * I).reshape(R, I) % 9).double() * 2.0 ** -24
    du[0, :4] = torch.tensor([0.25, 0.75, 1.25, 1.75]).double() * 2.0 ** -24
    dh = (du / 64 * 2.0 ** 16).half()                                     # scaled dy: exact
    x = one_hot_call("fp16", g, u, dh, "cuda")
    gu = x["gu"].clone()
    gu[:, :I] = 64.0
    h = torch.zeros(R, I, dtype=torch.float16, device="cuda")
    w2 = (x["w2"].double() * 2.0 ** -16).half()                           # 2^-16: a subnormal, exact
    got = moe.moe_gated_ffn_backward(x["dy"], x["rows"], x["back_w13"], w2, gu, h).drows[:, I:2 * I].double().cpu()
    want = du.clone()
    want[0, :4] = torch.tensor([0.0, 1.0, 1.0, 2.0]).double() * 2.0 ** -24
    assert torch.equal(got, want)
