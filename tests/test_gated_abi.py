"""Host-side argument checks of the gated blocks and of dropout (no GPU: every call below
fails its checks, or is a documented no-op, before anything is enqueued)."""
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


def test_dropout_refusals(L):
    good = dict(x=P, xs=64, r=P, rs=64, dtype=0, T=4, d=64, p=0.5, state=P, site=0, out=P, os=64, s=None)

    def status(**change):
        args = {**good, **change}
        assert set(args) == set(good)
        return L.moe_dropout(*args.values())

    for change in (dict(dtype=-1), dict(dtype=3), dict(T=-1), dict(d=0), dict(p=-0.1), dict(p=1.1),
                   dict(p=float("nan")), dict(state=None), dict(state=P + 4), dict(site=-1), dict(site=2048),
                   dict(x=None), dict(out=None), dict(x=P + 1), dict(out=P + 1), dict(r=P + 1),
                   dict(x=P + 2, dtype=2), dict(xs=-1), dict(rs=-1), dict(os=63)):
        assert status(**change) == INVALID, change
        assert b"moe_dropout" in L.moe_last_error()
    for change in (dict(d=(1 << 24) + 1), dict(T=1 << 28, d=64), dict(T=2 ** 31 - 1, d=1),
                   dict(T=1 << 27, d=64, dtype=2)):
        assert status(**change) == SHAPE, change
    assert status(T=0, x=None, r=None, out=None) == 0
    assert status(T=0, x=None, r=None, out=None, p=0.0, state=None) == 0


def ffn_args(**change):
    a = _lib.GatedFfnArgs()
    a.dtype, a.num_rows, a.d, a.I, a.E, a.activation = 0, 4, 64, 72, 2, 0
    a.rows = a.expert_offsets = a.w13 = a.w2 = a.drop_state = P
    a.rows_stride, a.drop_p, a.drop_site = 64, 0.5, 1
    for f, v in change.items():
        setattr(a, f, v)
    return ctypes.byref(a)


def grad_args(**change):
    g = _lib.GatedFfnGradArgs()
    for f, n in (("dy", 64), ("gu", 144), ("h", 72), ("drows", 64)):
        setattr(g, f, P)
        setattr(g, f + "_stride", n)
    g.dw13 = g.dw2 = g.workspace = P
    g.workspace_bytes = 1 << 30
    for f, v in change.items():
        setattr(g, f, v)
    return ctypes.byref(g)


BAD = [dict(dtype=2), dict(dtype=-1), dict(num_rows=-1), dict(d=0), dict(I=0), dict(E=0), dict(activation=2),
       dict(activation=-1), dict(rows=None), dict(rows=P + 8), dict(rows_stride=56), dict(rows_stride=68),
       dict(w13=None), dict(w13=P + 2), dict(w2=None), dict(expert_offsets=None), dict(expert_offsets=P + 2),
       dict(drop_p=-1.0), dict(drop_p=2.0), dict(drop_p=float("nan")), dict(drop_state=None),
       dict(drop_state=P + 1), dict(drop_site=2048), dict(drop_site=-1)]
BAD_SHAPE = [dict(d=60), dict(I=70), dict(d=65544), dict(I=65544), dict(E=1025), dict(num_rows=(1 << 24) + 1),
             dict(rows_stride=(1 << 20) + 8)]


def test_gated_ffn_refusals(L):
    def status(a, gu=P, gs=144, h=P, hs=72, y=P, ys=64):
        return L.moe_gated_ffn(a, gu, gs, h, hs, y, ys, None)

    assert status(None) == INVALID
    for change in BAD:
        assert status(ffn_args(**change)) == INVALID, change
    for change in BAD_SHAPE:
        assert status(ffn_args(**change)) == SHAPE, change
    for change in (dict(gs=136), dict(gs=145), dict(gu=P + 8), dict(h=None), dict(hs=64), dict(h=P + 2), dict(ys=56),
                   dict(y=P + 8)):
        assert status(ffn_args(), **change) == INVALID, change
    none = dict(rows=None, w13=None, w2=None, drop_state=P)
    assert status(ffn_args(num_rows=0, **none), None, 0, None, 0, None, 0) == 0


def test_gated_ffn_backward_refusals(L):
    fn = L.moe_gated_ffn_backward
    assert fn(None, grad_args(), None) == INVALID
    assert fn(ffn_args(), None, None) == INVALID
    for change in BAD:
        assert fn(ffn_args(**change), grad_args(), None) == INVALID, change
    for change in BAD_SHAPE:
        assert fn(ffn_args(**change), grad_args(), None) == SHAPE, change
    for change in (dict(drows=None, dw13=None, dw2=None), dict(dy=None), dict(dy=P + 8), dict(dy_stride=56),
                   dict(gu=None), dict(gu_stride=136), dict(h=None), dict(h_stride=64), dict(drows=P + 4),
                   dict(drows_stride=60), dict(dw13=P + 8), dict(dw2=P + 8)):
        assert fn(ffn_args(), grad_args(**change), None) == INVALID, change
    query = L.moe_gated_ffn_backward_workspace_bytes
    need = query(4, 64, 72, 2)
    assert need >= 4 * 144 * 2
    for change in (dict(workspace=None), dict(workspace=P + 16), dict(workspace_bytes=need - 1)):
        assert fn(ffn_args(), grad_args(**change), None) == WORKSPACE, change
    for bad in ((-1, 64, 72, 2), (4, 60, 72, 2), (4, 64, 0, 2), (4, 64, 72, 1025), (4, 65544, 72, 2),
                ((1 << 24) + 1, 64, 72, 2)):
        assert query(*bad) == -1
    assert query(0, 64, 72, 2) == 0
    nothing = dict(dw13=None, dw2=None, dy=None, drows=None)
    assert fn(ffn_args(num_rows=0), grad_args(**nothing), None) == 0


def test_binding_refuses_host_tensors():
    x, w13, w2 = torch.zeros(4, 8).bfloat16(), torch.zeros(16, 8).bfloat16(), torch.zeros(8, 8).bfloat16()
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.moe_dropout(x, moe.Dropout(0.0))
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.moe_gated_ffn(x, w13, w2)
    with pytest.raises(ValueError, match="GPU tensor"):
        moe.moe_gated_ffn_backward(x, x, w13, w2, None, None)
    with pytest.raises(TypeError):
        moe.moe_dropout(x.double(), moe.Dropout(0.0))
    with pytest.raises(TypeError):
        moe.moe_gated_ffn([1.0], w13, w2)
