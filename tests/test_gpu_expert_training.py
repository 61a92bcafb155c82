"""The operators of an expert block in training together, as they are used: norm, router,
rows by expert, gated experts with dropout, rows back, dropout with the residual's addition,
and back, against float64 autograd of the same block with the selection held fixed."""
import numpy as np
import pytest
import torch

import w4a16_grouped_expert_amd as moe
from oracle import gated

from gated_helpers import DEV, SEED, STEP
from gpu_helpers import say
from rows_helpers import f64

pytestmark = pytest.mark.gpu
T, d, I, E, k, P = 203, 136, 72, 6, 3, 0.2


def step(x, wr, v0, w13, w2, dout, state):
    """Output and gradients of one step through the package's calls."""
    before = moe.BlockNorm(norm_in=v0)
    inner, outer = moe.Dropout(P, state, 1), moe.Dropout(P, state, 2)
    _, n0 = moe.moe_block_norm(before, x)
    route = moe.moe_route(n0, wr, k)
    al = moe.moe_align(route.ids, E)
    rows = moe.moe_permute(n0, al.pair_pos, k)
    mid, h, gu = moe.moe_gated_ffn(rows, w13, w2, al.offsets, dropout=inner, save=True)
    y = moe.moe_unpermute(mid, al.pair_pos, k, T, route.weights)
    out = moe.moe_dropout(y, outer, residual=x)

    dy = moe.moe_dropout(dout, outer)
    dmid = torch.empty_like(mid)
    dweights = torch.empty(T, k, device=DEV)
    moe.moe_unpermute_backward_into(dy, al.pair_pos, k, dmid, route.weights, mid, dweights)
    g = moe.moe_gated_ffn_backward(dmid, rows, w13, w2, gu, h, al.offsets, dropout=inner)
    dn0 = torch.empty_like(n0)
    moe.moe_permute_backward_into(g.drows, al.pair_pos, k, dn0)
    dn0, dwr = moe.moe_route_backward(n0, wr, route, dweights, dx_add=dn0)
    gb = moe.moe_block_norm_backward(before, x, dn=dn0)
    dx = dout.float() + gb.dx.float()
    return dict(out=out, x=dx, wr=dwr, v0=gb.dnorm_in, w13=g.dw13, w2=g.dw2), route, al


def test_training_step():
    say("training step of an expert block")
    gen = torch.Generator().manual_seed(12)

    def rand(*shape, std=1.0, mean=0.0):
        return (mean + std * torch.randn(*shape, generator=gen)).bfloat16().to(DEV)

    x, wr, v0 = rand(T, d), rand(E, d, std=d ** -0.5), rand(d, std=0.1, mean=1.0)
    w13, w2, dout = rand(E, 2 * I, d, std=d ** -0.5), rand(E, d, I, std=I ** -0.5), rand(T, d, std=0.1)
    state = torch.tensor([SEED, STEP], device=DEV)
    got, route, al = step(x, wr, v0, w13, w2, dout, state)
    torch.cuda.synchronize()

    ids, pos = route.ids.cpu().long(), al.pair_pos.cpu().long().reshape(T, k)
    leaf = {q: t.double().cpu().requires_grad_() for q, t in dict(x=x, wr=wr, v0=v0, w13=w13, w2=w2).items()}
    inner = torch.from_numpy(gated.drop_factor(P, SEED, STEP, 1, T * k, I))
    outer = torch.from_numpy(gated.drop_factor(P, SEED, STEP, 2, T, d))
    n0 = leaf["x"] / torch.sqrt((leaf["x"] ** 2).mean(1, keepdim=True) + 1e-6) * leaf["v0"]
    w = torch.softmax((n0 @ leaf["wr"].t()).gather(1, ids), 1)
    out = torch.zeros(T, d, dtype=torch.float64)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        gu = n0[t] @ leaf["w13"][e].t()
        h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:] * inner[pos[t, j]]
        out = out.index_add(0, t, w[t, j, None] * (h @ leaf["w2"][e].t()))
    out = leaf["x"] + out * outer
    (out * dout.double().cpu()).sum().backward()

    # at most twelve bf16 roundings lie between a leaf and its gradient (n0, rows, gu, h, mid, y,
    # then dy, dmid, dg and du, drows, dn0, dx), each 2^-8 of a value that the next steps carry
    # on; in the 2-norm of a tensor their errors add at most
    tol = 12 * 2.0 ** -8
    for q, t in got.items():
        ref = out.detach().numpy() if q == "out" else leaf[q].grad.numpy()
        err = np.linalg.norm(f64(t) - ref) / np.linalg.norm(ref)
        say(f"  {q}: {err:.2e}")
        assert err <= tol, (q, err)


def test_trained_experts_are_packed_as_they_are():
    """The weights' layouts are those of pack_experts: the quantised layer takes them, and comes
    out near the 16-bit experts (four bits per weight: within a tenth in the 2-norm per output)."""
    say("trained experts quantised")
    d, I, E, k, T = 256, 128, 4, 2, 32
    gen = torch.Generator().manual_seed(3)

    def rand(*shape, std=1.0):
        return (std * torch.randn(*shape, generator=gen)).bfloat16().to(DEV)

    x, wr, w13, w2 = rand(T, d), rand(E, d, std=0.1), rand(E, 2 * I, d, std=0.05), rand(E, d, I, std=0.05)
    # weights that four bits hold exactly: multiples of their group's largest over seven
    def grid(w):
        g = w.float().reshape(*w.shape[:-1], -1, 128)
        s = (g.abs().amax(-1, keepdim=True) / 7).bfloat16().float()
        return (torch.round(g / s).clamp(-7, 7) * s).reshape(w.shape).bfloat16()

    w13, w2 = grid(w13), grid(w2)
    route = moe.moe_route(x, wr, k)
    al = moe.moe_align(route.ids, E)
    y = moe.moe_gated_ffn(moe.moe_permute(x, al.pair_pos, k), w13, w2, al.offsets)
    ours = f64(moe.moe_unpermute(y, al.pair_pos, k, T, route.weights))
    bank, _ = moe.pack_experts(w13, w2)
    quantised = f64(moe.moe_w4a16_grouped_ffn(x, route, al, bank, I))
    # a group's scale may be requantised one bf16 step off (2^-8) and its codes by half a step of
    # one seventh at worst in a rounding tie: far below a tenth of the output
    assert np.linalg.norm(ours - quantised) <= 0.1 * np.linalg.norm(ours)


def test_two_graphs_on_one_workspace():
    """Two captured backward calls that share a workspace, replayed in turn on one stream."""
    say("gated ffn two graphs")
    gen = torch.Generator().manual_seed(4)

    def rand(*shape, std=1.0):
        return (std * torch.randn(*shape, generator=gen)).bfloat16().to(DEV)

    R, d, I = 150, 136, 72
    w13, w2 = rand(2 * I, d, std=0.1), rand(d, I, std=0.1)
    ws = moe.alloc_gated_ffn_workspace(R, d, I, 1, DEV)
    runs = []
    for _ in range(2):
        rows, dy = rand(R, d), rand(R, d)
        _, h, gu = moe.moe_gated_ffn(rows, w13, w2, save=True)
        want = moe.moe_gated_ffn_backward(dy, rows, w13, w2, gu, h)
        grads = moe.GatedFfnGrads(*(torch.empty_like(t) for t in (want.drows, want.dw13, want.dw2)))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.moe_gated_ffn_backward_into(dy, rows, w13, w2, gu, h, grads, ws)
        runs.append((graph, grads, want, (rows, dy, h, gu)))
    for i in (0, 1, 1, 0, 1):
        graph, grads, want, _ = runs[i]
        for t in (grads.drows, grads.dw13, grads.dw2):
            t.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        for name in ("drows", "dw13", "dw2"):
            assert torch.equal(getattr(grads, name), getattr(want, name)), (i, name)
