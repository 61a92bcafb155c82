"""Host-side argument checks of the row operators (no GPU: every call below fails its
checks, or is a documented no-op, before anything is enqueued)."""
import ctypes

import pytest
import torch

import w4a16_grouped_expert_amd as moe
from w4a16_grouped_expert_amd import _lib

INVALID, SHAPE, WORKSPACE = 1, 2, 3
P = 256  # a pointer that is never dereferenced


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


# the four calls on good arguments by name, as (function, list of [name, value])
def calls(L):
    common = dict(dtype=0, T=4, d=64, k=2)
    return {
        "permute": (L.moe_permute, dict(x=P, xs=64, **common, pos=P, w=P, rows=P, rs=64, R=8, s=None)),
        "unpermute": (L.moe_unpermute, dict(rows=P, rs=64, R=8, **common, pos=P, w=P, out=P, os=64, s=None)),
        "permute_backward": (L.moe_permute_backward, dict(drows=P, rs=64, R=8, x=P, xs=64, **common, pos=P, w=P, dx=P,
                                                          os=64, dw=P, s=None)),
        "unpermute_backward": (L.moe_unpermute_backward, dict(dout=P, xs=64, rows=P, rs=64, **common, pos=P, w=P,
                                                              drows=P, os=64, R=8, dw=P, s=None)),
    }


@pytest.mark.parametrize("name", ["permute", "unpermute", "permute_backward", "unpermute_backward"])
def test_permute_refusals(L, name):
    fn, good = calls(L)[name]

    def refused(status, **change):
        args = {**good, **change}
        assert set(args) == set(good)
        assert fn(*args.values()) == status, change
        assert name.encode() in L.moe_last_error()

    for bad in (-1, 3):
        refused(INVALID, dtype=bad)
    refused(INVALID, T=-1)
    refused(INVALID, d=0)
    refused(INVALID, k=0)
    refused(INVALID, R=-1)
    refused(SHAPE, k=17)
    refused(SHAPE, T=1 << 24)
    refused(SHAPE, d=(1 << 24) + 1)
    refused(SHAPE, T=1 << 15, d=(1 << 19) + 1)  # more elements than a launch has lanes for
    refused(INVALID, pos=None)
    refused(INVALID, pos=P + 2)
    refused(INVALID, w=P + 1)
    for row in ("x", "rows", "out", "drows", "dx", "dout"):
        if row in good:
            refused(INVALID, **{row: None})
            refused(INVALID, **{row: P + 1})       # off the type's alignment
            refused(INVALID, **{row: P + 2, "dtype": 2})
    for stride in ("xs", "rs", "os"):
        if stride in good:
            refused(INVALID, **{stride: -1})
    written = {"permute": "rs", "unpermute": "os", "permute_backward": "os", "unpermute_backward": "os"}[name]
    refused(INVALID, **{written: 63})
    nothing = {q: None for q in good if q in ("x", "rows", "out", "drows", "dx", "dout", "pos", "w", "dw")}
    assert fn(*{**good, **nothing, "T": 0}.values()) == 0  # no tokens: a no-op


def route_args(**change):
    a = _lib.RouteBackwardArgs()
    a.T, a.d, a.E, a.k, a.renormalize = 4, 64, 8, 2, 1
    for f in ("x", "w_router", "logits", "topk_ids", "topk_weights", "dweights", "dlogits", "dx_add", "dx",
              "dw_router", "workspace"):
        setattr(a, f, P)
    a.workspace_bytes = 1 << 30
    for f, v in change.items():
        setattr(a, f, v)
    return ctypes.byref(a)


def test_route_backward_refusals(L):
    fn = L.moe_route_backward
    assert fn(None, None) == INVALID
    for change in (dict(T=-1), dict(d=0), dict(E=0), dict(k=0), dict(topk_ids=None), dict(topk_weights=None),
                   dict(dweights=None), dict(logits=None, renormalize=0), dict(dx=None, dw_router=None),
                   dict(w_router=None), dict(x=None), dict(x=P + 8), dict(w_router=P + 2), dict(dx=P + 8),
                   dict(dx_add=P + 4), dict(dw_router=P + 4), dict(dweights=P + 2), dict(topk_ids=P + 1),
                   dict(dlogits=P + 2)):
        assert fn(route_args(**change), None) == INVALID, change
    for change in (dict(d=60), dict(E=1025), dict(k=17, E=64), dict(k=9), dict(d=(1 << 20) + 8), dict(T=(1 << 24) + 1)):
        assert fn(route_args(**change), None) == SHAPE, change
    need = L.moe_route_backward_workspace_bytes(4, 64, 8, 2)
    assert need > 0 and need % 256 == 0
    for change in (dict(workspace=None), dict(workspace=P + 16), dict(workspace_bytes=need - 1)):
        assert fn(route_args(**change), None) == WORKSPACE, change
    assert L.moe_route_backward_workspace_bytes(-1, 64, 8, 2) == -1
    for sizes in ((2 ** 31 - 1, 64, 8, 2), (4, 2 ** 31 - 8, 8, 2), (4, 64, 2 ** 31 - 1, 2)):
        assert L.moe_route_backward_workspace_bytes(*sizes) == -1
    assert L.moe_route_backward_workspace_bytes(0, 64, 8, 2) >= 0
    assert fn(route_args(T=0, dw_router=None), None) == 0


def norm_args(**change):
    a = _lib.BlockNormArgs()
    a.dtype, a.T, a.d, a.gate_kind = 0, 4, 64, moe.GATE_CHANNEL
    a.x = a.y = a.norm_out = a.norm_in = a.gate = P
    a.x_stride = a.y_stride = a.gate_stride = 64
    a.residual_scale, a.eps = 1.0, 1e-6
    for f, v in change.items():
        setattr(a, f, v)
    return ctypes.byref(a)


def grad_args(**change):
    g = _lib.BlockNormGradArgs()
    for f in ("dh", "dn", "dx", "dy"):
        setattr(g, f, P)
        setattr(g, f + "_stride", 64)
    g.dgate = g.dnorm_out = g.dnorm_in = g.workspace = P
    g.dgate_stride, g.workspace_bytes = 64, 1 << 30
    for f, v in change.items():
        setattr(g, f, v)
    return ctypes.byref(g)


BAD_NORM = [dict(dtype=3), dict(T=-1), dict(d=0), dict(gate_kind=4), dict(gate_kind=-1), dict(eps=0.0),
            dict(eps=1e-40), dict(eps=float("nan")), dict(eps=float("inf")), dict(residual_scale=float("inf")),
            dict(x=None), dict(x=P + 1), dict(y=P + 1), dict(norm_in=P + 1), dict(gate=P + 1, gate_kind=3),
            dict(y=None), dict(y=None, norm_out=None), dict(gate=None), dict(gate_kind=0), dict(x_stride=-1),
            dict(y_stride=-1), dict(gate_kind=2, gate_stride=-1)]


def test_block_norm_refusals(L):
    fn = L.moe_block_norm
    assert fn(None, P, 64, P, 64, None) == INVALID
    for change in BAD_NORM:
        assert fn(norm_args(**change), P, 64, P, 64, None) == INVALID, change
    for change in (dict(d=16385), dict(T=(1 << 24) + 1), dict(T=1 << 21, d=8193)):
        assert fn(norm_args(**change), P, 1 << 20, P, 1 << 20, None) == SHAPE, change
    assert fn(norm_args(), None, 0, None, 0, None) == INVALID      # nothing wanted
    assert fn(norm_args(), P, 64, None, 0, None) == INVALID        # norm_in without n
    assert fn(norm_args(norm_in=None), P, 64, P, 64, None) == INVALID
    assert fn(norm_args(), P, 63, P, 64, None) == INVALID
    assert fn(norm_args(), P, 64, P + 1, 64, None) == INVALID
    none = dict(x=None, y=None, gate=None, norm_in=None, norm_out=None)
    assert fn(norm_args(T=0, **none), None, 0, None, 0, None) == 0


def test_block_norm_backward_refusals(L):
    fn = L.moe_block_norm_backward
    assert fn(None, grad_args(), None) == INVALID
    assert fn(norm_args(), None, None) == INVALID
    for change in BAD_NORM:
        assert fn(norm_args(**change), grad_args(), None) == INVALID, change
    for change in (dict(dh=None, dn=None), dict(dh_stride=-1), dict(dn_stride=-1), dict(dx_stride=63),
                   dict(dy_stride=63), dict(dx=P + 1), dict(dgate=P + 2), dict(dnorm_in=P + 2),
                   dict(dnorm_out=P + 1)):
        assert fn(norm_args(), grad_args(**change), None) == INVALID, change
    assert fn(norm_args(gate_kind=3), grad_args(dgate_stride=63), None) == INVALID
    plain = dict(gate=None, gate_kind=0)
    assert fn(norm_args(**plain), grad_args(), None) == INVALID                          # dgate without gate
    assert fn(norm_args(norm_in=None), grad_args(), None) == INVALID                     # dn without norm_in
    assert fn(norm_args(norm_in=None), grad_args(dn=None), None) == INVALID              # dnorm_in without it
    assert fn(norm_args(norm_out=None), grad_args(), None) == INVALID
    assert fn(norm_args(y=None, norm_out=None, **plain), grad_args(dgate=None, dnorm_out=None), None) == INVALID
    need = L.moe_block_norm_backward_workspace_bytes(4, 64)
    assert need > 0
    for change in (dict(workspace=None), dict(workspace=P + 128), dict(workspace_bytes=need - 1)):
        assert fn(norm_args(), grad_args(**change), None) == WORKSPACE, change
    assert L.moe_block_norm_backward_workspace_bytes(-1, 64) == -1
    no_vectors = dict(dgate=None, dnorm_out=None, dnorm_in=None, workspace=None)
    assert fn(norm_args(T=0), grad_args(**no_vectors), None) == 0
    # a gate of the channels is there without rows too
    assert fn(norm_args(T=0, gate=None), grad_args(), None) == INVALID


def test_binding_refuses_host_tensors():
    x, pos = torch.zeros(4, 8), torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.moe_permute(x, pos, 2)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.moe_unpermute(x, pos, 2, 2)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.moe_block_norm(moe.BlockNorm(norm_in=torch.ones(8)), x)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.moe_block_norm_backward(moe.BlockNorm(norm_in=torch.ones(8)), x, dn=x)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.moe_route_backward(x, x, None, x)
    with pytest.raises(TypeError):
        moe.moe_permute(x.double(), pos, 2)
    with pytest.raises(TypeError):
        moe.moe_permute([1.0], pos, 2)
