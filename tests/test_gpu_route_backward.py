"""moe_route_backward against the float64 reference."""
import numpy as np
import pytest
import torch

import w4a16_grouped_expert_amd as moe
from oracle import rows as orow

from gpu_helpers import say
from rows_helpers import U32, assert_near, f64, half_step

pytestmark = pytest.mark.gpu
DEV = "cuda"
# T, d, E, k: single tokens, sizes off every tile, one to many expert tiles, the limits
SHAPES = [(1, 8, 1, 1), (1, 2048, 64, 8), (3, 136, 5, 2), (31, 264, 16, 4), (33, 128, 17, 3), (64, 520, 33, 6),
          (100, 72, 64, 8), (257, 1112, 100, 16), (40, 256, 1024, 16), (1000, 2048, 64, 8), (4100, 328, 8, 2)]


def make(T, d, E, k, renormalize, seed=0):
    g = torch.Generator().manual_seed(seed + T + 7 * d + 13 * E)
    x = torch.randn(T, d, generator=g).bfloat16().to(DEV)
    w = (torch.randn(E, d, generator=g) * d ** -0.5).bfloat16().to(DEV)
    route = moe.moe_route(x, w, k, renormalize)
    dweights = torch.randn(T, k, generator=g).to(DEV)
    dlogits = (0.1 * torch.randn(T, E, generator=g)).to(DEV)
    add = torch.randn(T, d, generator=g).bfloat16().to(DEV)
    return x, w, route, dweights, dlogits, add


def check(name, x, w, route, dweights, renormalize, dlogits, add, dx, dw):
    args = [f64(x), f64(w), f64(route.logits), route.ids.cpu().numpy(), f64(route.weights), f64(dweights), renormalize,
            f64(dlogits)]
    rdx, rdw = orow.route_backward(*args, dx_add=f64(add))
    T, E = args[2].shape
    k = args[3].shape[1]
    # the gradient of the logits: each element is a product of a weight (softmax over E in
    # float32: E additions and expf's few roundings) and a difference of terms of size
    # |dw| + |s|, then one addition
    ids = args[3].astype(np.int64)
    ok = (ids >= 0) & (ids < E)
    wt, dwt = np.where(ok, args[4], 0), np.abs(np.where(ok, args[5], 0))
    s = (wt * dwt).sum(axis=1, keepdims=True)
    size = np.zeros((T, E)) if renormalize else orow.softmax(args[2]) * s
    for t, j in zip(*np.nonzero(ok)):
        size[t, ids[t, j]] += wt[t, j] * (dwt[t, j] + s[t, 0])
    size = size + (0 if dlogits is None else np.abs(args[7]))
    eg = (k + (0 if renormalize else E / 8) + 16) * U32 * size
    # its bf16 parts (2^-18 with two, 2^-27 with three), then E or T float32 additions
    g = np.abs(orow.route_dlogits(*args[2:])) + eg
    if dx is not None:
        e = (eg + (2.0 ** -18 + (2 * E + 8) * U32) * g) @ np.abs(f64(w))
        e = e + (0 if add is None else U32 * (np.abs(rdx) + np.abs(f64(add))))
        assert_near(name + " dx", dx, rdx, half_step(torch.bfloat16, np.abs(rdx) + e) + e)
    if dw is not None:
        e = (eg + (2.0 ** -27 + (3 * T + 8) * U32) * g).T @ np.abs(f64(x))
        assert_near(name + " dw", dw, rdw, e + 1e-45)


@pytest.mark.parametrize("T,d,E,k", SHAPES)
@pytest.mark.parametrize("renormalize", [True, False])
def test_against_reference(T, d, E, k, renormalize):
    say(f"route backward T={T} d={d} E={E} k={k} renormalize={renormalize}")
    x, w, route, dweights, dlogits, add = make(T, d, E, k, renormalize)
    for aux, plus in ((None, None), (dlogits, add)):
        dx, dw = moe.moe_route_backward(x, w, route, dweights, renormalize, aux, plus)
        torch.cuda.synchronize()
        check(f"aux={aux is not None}", x, w, route, dweights, renormalize, aux, plus, dx, dw)


@pytest.mark.parametrize("T,d,E,k", [(129, 200, 65, 2), (300, 136, 129, 3), (520, 264, 257, 6), (70, 128, 513, 9),
                                     (2100, 1024, 128, 8), (300, 136, 63, 16)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_ways_to_the_logits_gradient(T, d, E, k, renormalize):
    """Sizes around those where another kernel computes it, each output alone too."""
    say(f"route backward T={T} d={d} E={E} k={k} renormalize={renormalize}, parts")
    x, w, route, dweights, _, add = make(T, d, E, k, renormalize)
    dx, dw = moe.moe_route_backward(x, w, route, dweights, renormalize, None, add)
    torch.cuda.synchronize()
    check("both", x, w, route, dweights, renormalize, None, add, dx, dw)
    ws = moe.alloc_route_backward_workspace(T, d, E, k, DEV)
    only_x, only_w = torch.empty_like(dx), torch.empty_like(dw)
    moe.moe_route_backward_into(x, w, route, dweights, only_x, None, ws, renormalize, None, add)
    moe.moe_route_backward_into(x, w, route, dweights, None, only_w, ws, renormalize)
    assert torch.equal(only_x, dx) and torch.equal(only_w, dw)


def test_parts_and_accumulation_in_place():
    say("route backward: one output alone, dx added in place")
    T, d, E, k = 200, 264, 40, 5
    x, w, route, dweights, dlogits, add = make(T, d, E, k, True)
    dx, dw = moe.moe_route_backward(x, w, route, dweights, True, dlogits, add)
    ws = moe.alloc_route_backward_workspace(T, d, E, k, DEV)
    only = torch.empty_like(dx)
    moe.moe_route_backward_into(x, w, route, dweights, only, None, ws, True, dlogits, add)
    assert torch.equal(only, dx)
    only = torch.empty_like(dw)
    moe.moe_route_backward_into(x, w, route, dweights, None, only, ws, True, dlogits)
    assert torch.equal(only, dw)
    acc = add.clone()
    moe.moe_route_backward_into(x, w, route, dweights, acc, None, ws, True, dlogits, acc)
    assert torch.equal(acc, dx)


@pytest.mark.parametrize("renormalize", [True, False])
def test_ignored_ids_and_one_expert(renormalize):
    say("route backward with ids outside the experts, and k = E = 1")
    T, d, E, k = 50, 64, 12, 3
    x, w, route, dweights, _, _ = make(T, d, E, k, renormalize)
    route.ids[3] = -1
    route.ids[4, 1] = E
    route.ids[5, 0] = 2 ** 31 - 1
    dx, dw = moe.moe_route_backward(x, w, route, dweights, renormalize)
    torch.cuda.synchronize()
    check("ids", x, w, route, dweights, renormalize, None, None, dx, dw)
    x, w, route, dweights, _, _ = make(70, 64, 1, 1, renormalize)
    dx, dw = moe.moe_route_backward(x, w, route, dweights, renormalize)
    # one expert has the weight 1 whatever its logit
    assert torch.count_nonzero(dx) == 0 and torch.count_nonzero(dw) == 0


def test_large_logits():
    say("route backward with logits of +-1e4")
    T, d, E, k = 64, 128, 20, 4
    x, w, _, dweights, _, _ = make(T, d, E, k, False)
    route = moe.moe_route((x * 100).contiguous(), (w * 100).contiguous(), k, False)
    dx, dw = moe.moe_route_backward(x, w, route, dweights, False)
    torch.cuda.synchronize()
    check("large", x, w, route, dweights, False, None, None, dx, dw)


def test_no_tokens():
    say("route backward T = 0")
    x, w, _, _, _, _ = make(1, 64, 4, 2, True)
    route = moe.alloc_route(0, 4, 2, DEV)
    dx, dw = moe.moe_route_backward(x[:0], w, route, torch.empty(0, 2, device=DEV))
    torch.cuda.synchronize()
    assert dx.shape == (0, 64) and torch.equal(dw, torch.zeros(4, 64, device=DEV))


def test_graph_side_stream_and_determinism():
    say("route backward captured, replayed and on another stream")
    T, d, E, k = 900, 520, 64, 8
    x, w, route, dweights, dlogits, add = make(T, d, E, k, False)
    dx, dw = torch.empty_like(x), torch.empty(E, d, device=DEV)
    ws = moe.alloc_route_backward_workspace(T, d, E, k, DEV)

    def step():
        moe.moe_route_backward_into(x, w, route, dweights, dx, dw, ws, False, dlogits, add)

    step()
    torch.cuda.synchronize()
    ref = dx.clone(), dw.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(3):
        dx.zero_(), dw.zero_(), ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(dx, ref[0]) and torch.equal(dw, ref[1]), f"replay {i}"
        step()
        torch.cuda.synchronize()
        assert torch.equal(dx, ref[0]) and torch.equal(dw, ref[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.moe_route_backward(x, w, route, dweights, False, dlogits, add, stream=side)
    side.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_two_graphs_share_a_workspace_and_two_streams():
    say("route backward: two graphs on one workspace, two streams on two")
    calls = []
    for T, d, E, k, renormalize in ((300, 520, 64, 8, True), (200, 264, 130, 4, False)):
        x, w, route, dweights, _, add = make(T, d, E, k, renormalize)
        dx, dw = torch.empty_like(x), torch.empty(E, d, device=DEV)
        calls.append((x, w, route, dweights, renormalize, add, dx, dw))
    size = max(moe.route_backward_workspace_bytes(c[0].shape[0], c[0].shape[1], c[1].shape[0], c[2].ids.shape[1])
               for c in calls)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)

    def step(c, ws, stream=None):
        x, w, route, dweights, renormalize, add, dx, dw = c
        moe.moe_route_backward_into(x, w, route, dweights, dx, dw, ws, renormalize, None, add, stream)

    refs, graphs = [], []
    for c in calls:
        step(c, ws)
        torch.cuda.synchronize()
        refs.append((c[6].clone(), c[7].clone()))
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(c, ws)
        graphs.append(g)
    for _ in range(3):
        for g, c, ref in zip(graphs, calls, refs):
            c[6].zero_(), c[7].zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(c[6], ref[0]) and torch.equal(c[7], ref[1])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [ws, torch.empty_like(ws)]
    for c in calls:
        c[6].zero_(), c[7].zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for c, space, st in zip(calls, spaces, streams):
            step(c, space, st)
    torch.cuda.synchronize()
    for c, ref in zip(calls, refs):
        assert torch.equal(c[6], ref[0]) and torch.equal(c[7], ref[1])


def test_binding_refusals():
    say("route backward refusals")
    x, w, route, dweights, dlogits, add = make(4, 64, 8, 2, True)
    with pytest.raises(TypeError):
        moe.moe_route_backward(x.float(), w, route, dweights)
    with pytest.raises(TypeError):
        moe.moe_route_backward(x, w, route, dweights.bfloat16())
    with pytest.raises(ValueError):
        moe.moe_route_backward(x, w, route, dweights[:, :1])
    with pytest.raises(ValueError):
        moe.moe_route_backward(x, w, route, dweights, dx_add=add[:2])
    with pytest.raises(moe.MoeError):
        moe.moe_route_backward_into(x, w, route, dweights, torch.empty_like(x), None,
                                    torch.empty(64, dtype=torch.uint8, device=DEV))
