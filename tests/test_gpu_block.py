"""The row operators together, as they are used: quantised layers in a chain of blocks
(MoELayer.block), and one training step of a block with the caller's own experts."""
import numpy as np
import pytest
import torch

import synth
import w4a16_grouped_expert_amd as moe
from oracle import ffn as offn
from oracle import rows as orow

from gpu_helpers import check_layer_out, oracle_bank, say
from rows_helpers import f64

pytestmark = pytest.mark.gpu
DEV = "cuda"


def to_bits(a):
    """float64 -> bf16 bit patterns (nearest even)."""
    return torch.from_numpy(a).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


@pytest.mark.parametrize("T", [1, 16, 150])
def test_chain_of_quantised_blocks(T):
    say(f"two blocks of quantised experts T={T}")
    wl = synth.TINY
    s = wl.shape
    g = torch.Generator().manual_seed(3)

    def vec(mean, std):
        return (mean + std * torch.randn(s.d, generator=g)).bfloat16().to(DEV)

    before = [vec(1.0, 0.1) for _ in range(2)]
    after = [moe.BlockNorm(norm_in=before[1], norm_out=vec(1.0, 0.1), gate=vec(0.5, 0.1)),
             moe.BlockNorm(norm_out=vec(1.0, 0.1), residual_scale=0.5)]
    layers, banks, wrs = [], [], []
    for l in range(2):
        w13, w2 = synth.expert_weights(wl, l)
        bank, _ = moe.pack_experts(w13.to(DEV), w2.to(DEV))
        wr = synth.router_weight(wl, l)
        layers.append(moe.MoELayer(wr.to(DEV), bank, s.I, s.k, T, norm_before=before[l], after=after[l]))
        banks.append(oracle_bank(w13, w2))
        wrs.append(wr.contiguous().view(torch.int16).numpy().view(np.uint16))
    x = synth.activations(wl, T, 0).to(DEV)

    def step():
        h, n = layers[0].block(x)
        return layers[1].block(h, n)[0]

    out = step()
    torch.cuda.synchronize()
    # each block against the reference on the inputs that this block saw
    h0, n0 = f64(layers[0].h[:T]), f64(layers[0].n_next[:T])
    n_first = f64(layers[0].n[:T])
    _, ref_n = orow.block_norm(f64(x), norm_in=f64(before[0]))
    check_layer_out("norm before", n_first, ref_n)
    y0 = offn.moe_layer(to_bits(n_first), wrs[0], banks[0], s.k)["out"]
    check_layer_out("layer", f64(layers[0].out[:T]), y0)
    p = dict(norm_in=f64(after[0].norm_in), norm_out=f64(after[0].norm_out), gate=f64(after[0].gate))
    ref_h, ref_n = orow.block_norm(f64(x), f64(layers[0].out[:T]), **p)
    check_layer_out("block h", h0, ref_h)
    check_layer_out("block n", n0, ref_n)
    y1 = offn.moe_layer(to_bits(n0), wrs[1], banks[1], s.k)["out"]
    ref, _ = orow.block_norm(h0, y1, norm_out=f64(after[1].norm_out), residual_scale=0.5)
    check_layer_out("second block", f64(out), ref)
    # the second block from its own norm before: that norm reads h rounded to bf16, the
    # fused one h itself, so its n may be a bf16 step off and select other experts near a
    # tie; the reference takes the n that this call computed
    own, _ = layers[1].block(layers[0].h[:T])
    n_own = f64(layers[1].n[:T])
    _, ref_n = orow.block_norm(h0, norm_in=f64(before[1]))
    check_layer_out("own norm", n_own, ref_n)
    y1 = offn.moe_layer(to_bits(n_own), wrs[1], banks[1], s.k)["out"]
    ref, _ = orow.block_norm(h0, y1, norm_out=f64(after[1].norm_out), residual_scale=0.5)
    check_layer_out("second block, own norm", f64(own), ref)

    step()
    torch.cuda.synchronize()
    keep = layers[1].h[:T].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(3):
        layers[1].h.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(layers[1].h[:T], keep), f"replay {i}"
        assert torch.equal(step(), keep)


def test_block_refusals():
    say("block refusals")
    wl = synth.TINY
    s = wl.shape
    w13, w2 = synth.expert_weights(wl, 0)
    bank, _ = moe.pack_experts(w13.to(DEV), w2.to(DEV))
    wr = synth.router_weight(wl, 0).to(DEV)
    x = synth.activations(wl, 4, 0).to(DEV)
    with pytest.raises(ValueError):
        moe.MoELayer(wr, bank, s.I, s.k, 4).block(x)
    layer = moe.MoELayer(wr, bank, s.I, s.k, 2, after=moe.BlockNorm())
    with pytest.raises(ValueError):
        layer.block(x)                   # more than T_max tokens
    with pytest.raises(ValueError):
        layer.block(x[:2])               # neither n nor norm_before
    h, n = layer.block(x[:2], x[:2])     # no norms at all: x + y
    assert n is None and torch.equal(h, (x[:2].float() + layer.out[:2].float()).bfloat16())


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("gate", ["channel", "token"])
def test_training_step(renormalize, gate):
    """norm -> route -> align -> permute -> the caller's experts -> unpermute -> norm,
    gate, residual and next norm, and back, against float64 autograd of the same block
    with the selection held fixed."""
    say(f"training step renormalize={renormalize} gate={gate}")
    T, d, E, k = 203, 136, 6, 3
    g = torch.Generator().manual_seed(11)

    def rand(*shape, std=1.0, mean=0.0):
        return (mean + std * torch.randn(*shape, generator=g)).bfloat16().to(DEV)

    x, wr, experts = rand(T, d), rand(E, d, std=d ** -0.5), rand(E, d, d, std=d ** -0.5)
    v0, v1, v2 = rand(d, std=0.1, mean=1.0), rand(d, std=0.1, mean=1.0), rand(d, std=0.1, mean=1.0)
    gt = rand(d, std=0.3, mean=1.0) if gate == "channel" else rand(T, 1, std=0.3, mean=1.0)
    dh, dn = rand(T, d, std=0.1), rand(T, d, std=0.1)
    before = moe.BlockNorm(norm_in=v0)
    after = moe.BlockNorm(norm_in=v2, norm_out=v1, gate=gt, residual_scale=0.9)

    _, n0 = moe.moe_block_norm(before, x)
    route = moe.moe_route(n0, wr, k, renormalize)
    al = moe.moe_align(route.ids, E)
    off = al.offsets.tolist()
    rows = moe.moe_permute(n0, al.pair_pos, k)
    mid = torch.empty_like(rows)
    for e in range(E):
        mid[off[e]:off[e + 1]] = (rows[off[e]:off[e + 1]].float() @ experts[e].float()).bfloat16()
    y = moe.moe_unpermute(mid, al.pair_pos, k, T, route.weights)
    h, n = moe.moe_block_norm(after, x, y)

    ga = moe.moe_block_norm_backward(after, x, y, dh, dn)
    dmid = torch.empty_like(mid)
    dweights = torch.empty(T, k, device=DEV)
    moe.moe_unpermute_backward_into(ga.dy, al.pair_pos, k, dmid, route.weights, mid, dweights)
    drows = torch.empty_like(rows)
    dexperts = torch.empty(E, d, d, device=DEV)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        dexperts[e] = rows[r].float().t() @ dmid[r].float()
        drows[r] = (dmid[r].float() @ experts[e].float().t()).bfloat16()
    dn0 = torch.empty_like(n0)
    moe.moe_permute_backward_into(drows, al.pair_pos, k, dn0)
    dn0, dwr = moe.moe_route_backward(n0, wr, route, dweights, renormalize, dx_add=dn0)
    gb = moe.moe_block_norm_backward(before, x, dn=dn0)
    dx = ga.dx.float() + gb.dx.float()
    torch.cuda.synchronize()

    ids = route.ids.cpu().long()
    leaf = {q: t.double().cpu().requires_grad_() for q, t in
            dict(x=x, wr=wr, experts=experts, v0=v0, v1=v1, v2=v2, gt=gt).items()}

    def rms(z):
        return z / torch.sqrt((z * z).mean(1, keepdim=True) + 1e-6)

    rn0 = rms(leaf["x"]) * leaf["v0"]
    logits = rn0 @ leaf["wr"].t()
    w = torch.softmax(logits.gather(1, ids), 1) if renormalize else torch.softmax(logits, 1).gather(1, ids)
    ry = (w[:, :, None] * torch.einsum("td,tkdf->tkf", rn0, leaf["experts"][ids])).sum(1)
    rh = 0.9 * leaf["x"] + leaf["gt"] * (rms(ry) * leaf["v1"])
    rn = rms(rh) * leaf["v2"]
    ((rh * dh.double().cpu()).sum() + (rn * dn.double().cpu()).sum()).backward()

    # at most ten bf16 roundings lie between a leaf and its gradient (n0, rows, experts'
    # rows, y, then dy, dmid, drows, dn0 and the two parts of dx), each 2^-8 of a value
    # that the next steps carry on; in the 2-norm of a tensor their errors add at most
    tol = 10 * 2.0 ** -8
    got = dict(x=dx, wr=dwr, experts=dexperts, v0=gb.dnorm_in, v1=ga.dnorm_out, v2=ga.dnorm_in, gt=ga.dgate)
    for q, t in got.items():
        ref = leaf[q].grad.numpy()
        err = np.linalg.norm(f64(t) - ref) / np.linalg.norm(ref)
        say(f"  d{q}: {err:.2e}")
        assert err <= tol, (q, err)
    for name, a, b in (("h", h, rh), ("n", n, rn)):
        err = np.linalg.norm(f64(a) - b.detach().numpy()) / np.linalg.norm(b.detach().numpy())
        assert err <= tol, (name, err)
