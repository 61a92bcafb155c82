"""moe_block_norm and its gradient against the float64 reference."""
import numpy as np
import pytest
import torch

import w4a16_grouped_expert_amd as moe
from oracle import rows as orow

from gpu_helpers import say
from rows_helpers import TYPES, U32, assert_near, f64, half_step, row_sum_ops, wide

pytestmark = pytest.mark.gpu
DEV = "cuda"
GATES = ["none", "channel", "token", "full"]
SHAPES = [(1, 1), (1, 2048), (2, 7), (5, 64), (3, 513), (16, 2048), (33, 1111), (4, 4096), (3, 8200), (2, 16384),
          (1100, 72), (2500, 264), (1300, 2048)]


def make(T, d, dtype, gate="channel", y=True, norm_out=True, norm_in=True, seed=0):
    g = torch.Generator().manual_seed(seed + T * 31 + d)

    def rand(*shape, std=1.0, mean=0.0):
        return (mean + std * torch.randn(*shape, generator=g)).to(dtype).to(DEV)

    shape = {"none": None, "channel": (d,), "token": (T, 1), "full": (T, d)}[gate]
    norm = moe.BlockNorm(norm_in=rand(d, std=0.2, mean=1.0) if norm_in else None,
                         norm_out=rand(d, std=0.2, mean=1.0) if norm_out else None,
                         gate=None if shape is None else rand(*shape, std=0.5), residual_scale=0.75, eps=1e-5)
    return norm, rand(T, d), rand(T, d, std=0.4) if y else None, rand(T, d, std=0.3), rand(T, d, std=0.3)


def params(norm):
    return dict(norm_in=f64(norm.norm_in), norm_out=f64(norm.norm_out), gate=f64(norm.gate),
                residual_scale=float(np.float32(norm.residual_scale)), eps=float(np.float32(norm.eps)))


def stats_error(norm, x, y, d):
    """First-order float32 errors: of h per element, and relative of both 1 / rms."""
    p = params(norm)
    c = row_sum_ops(d) / 2 + 8
    ax = np.abs(p["residual_scale"] * f64(x))
    gz = np.zeros_like(ax)
    if y is not None:
        h0, _ = orow.block_norm(f64(x), f64(y), norm_out=p["norm_out"], gate=p["gate"], residual_scale=0.0,
                                eps=p["eps"])
        gz = np.abs(h0)
    eh = U32 * (2 * ax + c * gz)
    h, _ = orow.block_norm(f64(x), f64(y), **p)
    rel = c * U32 + np.sqrt((eh * eh).mean(axis=1, keepdims=True)
                            / ((h * h).mean(axis=1, keepdims=True) + p["eps"]))
    return h, eh, rel, ax + gz


def check_forward(name, norm, x, y, lay=lambda t: t):
    T, d = x.shape
    h = lay(torch.full((T, d), 7.0, dtype=x.dtype, device=DEV))
    n = lay(torch.full((T, d), 7.0, dtype=x.dtype, device=DEV)) if norm.norm_in is not None else None
    moe.moe_block_norm_into(norm, lay(x), None if y is None else lay(y), h, n)
    torch.cuda.synchronize()
    p = params(norm)
    rh, rn = orow.block_norm(f64(x), f64(y), **p)
    _, eh, rel, _ = stats_error(norm, x, y, d)
    assert_near(name + " h", h, rh, half_step(x.dtype, np.abs(rh) + eh) + eh)
    if n is not None:
        en = np.abs(rn) * (rel + 4 * U32) + np.abs(p["norm_in"]) * orow.rstd(rh, p["eps"]) * eh
        assert_near(name + " n", n, rn, half_step(x.dtype, np.abs(rn) + en) + en)


def check_backward(name, norm, x, y, dh, dn, lay=lambda t: t):
    T, d = x.shape
    dt = x.dtype
    p = params(norm)
    ref = orow.block_norm_backward(f64(x), f64(y), **p, dh=f64(dh), dn=f64(dn))
    # the same formulas with every term's absolute value: what float32 roundings scale with
    h, _, rel, parts = stats_error(norm, x, y, d)
    D = np.zeros((T, d)) if dh is None else np.abs(f64(dh))
    amount = {}
    if norm.norm_in is not None:
        r = orow.rstd(h, p["eps"])
        # h = a x + g z comes with an error of a few 2^-24 of |a x| + |g z|, however far the
        # two cancel in h itself: that sum, not |h|, is what the errors of hn scale with
        a, hn = np.abs(np.zeros((T, d)) if dn is None else f64(dn)), parts * r
        u = a * np.abs(p["norm_in"])
        amount["dnorm_in"] = a * hn
        D = D + r * (u + hn * (u * hn).mean(axis=1, keepdims=True))
    amount["dx"] = p["residual_scale"] * D
    if y is not None:
        ry = 1.0 if norm.norm_out is None else orow.rstd(f64(y), p["eps"])
        yn = np.abs(f64(y)) * ry
        z = yn if norm.norm_out is None else yn * np.abs(p["norm_out"])
        g = 1.0 if p["gate"] is None else np.abs(p["gate"])
        amount["dgate"], amount["dnorm_out"] = D * z, D * g * yn
        q = D * g * (1.0 if norm.norm_out is None else np.abs(p["norm_out"]))
        amount["dy"] = q if norm.norm_out is None else ry * (q + yn * (q * yn).mean(axis=1, keepdims=True))
    # each term carries a few statistics (relative errors rel), row sums and products
    c = (3 * row_sum_ops(d) + 40) * U32 + 4 * rel
    grads = moe.moe_block_norm_backward(norm, lay(x), None if y is None else lay(y),
                                        None if dh is None else lay(dh), None if dn is None else lay(dn))
    torch.cuda.synchronize()
    vec = (T + 300) * U32  # a column sum: each term passes through at most T + 300 additions
    for q, r in ref.items():
        got = getattr(grads, q)
        e = c * amount[q]
        if q in ("dnorm_in", "dnorm_out") or (q == "dgate" and r.ndim == 1):
            e = e.sum(axis=0) + vec * amount[q].sum(axis=0)
            assert_near(f"{name} {q}", got, r, e)
        elif q == "dgate" and r.shape[1] == 1 and d > 1:
            assert_near(f"{name} {q}", got, r, e.sum(axis=1, keepdims=True)
                        + row_sum_ops(d) * U32 * amount[q].sum(axis=1, keepdims=True))
        else:
            assert_near(f"{name} {q}", got, r, half_step(got.dtype, np.abs(r) + e) + e)
    for q in ("dy", "dgate", "dnorm_in", "dnorm_out"):
        assert (getattr(grads, q) is None) == (q not in ref)


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("T,d", SHAPES)
def test_against_reference(T, d, type_):
    say(f"block norm T={T} d={d} {type_}")
    norm, x, y, dh, dn = make(T, d, TYPES[type_], GATES[(T + d) % 4])
    check_forward("fused", norm, x, y)
    check_backward("fused", norm, x, y, dh, dn)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("norm_out", [True, False])
@pytest.mark.parametrize("norm_in", [True, False])
def test_every_part(gate, norm_out, norm_in):
    say(f"block norm gate={gate} norm_out={norm_out} norm_in={norm_in}")
    for type_, (T, d) in (("fp32", (23, 100)), ("bf16", (9, 2056))):
        norm, x, y, dh, dn = make(T, d, TYPES[type_], gate, True, norm_out, norm_in)
        check_forward(type_, norm, x, y)
        check_backward(type_, norm, x, y, dh, dn if norm_in else None)
        if norm_in:
            check_backward(type_ + " dn alone", norm, x, y, None, dn)
            check_backward(type_ + " dh alone", norm, x, y, dh, None)


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("T,d", [(1, 1100), (2, 4096), (8, 2048), (9, 2048), (40, 64), (300, 1100), (300, 2304), (260, 5120),
                                 (70, 6144), (40, 12288)])
def test_ways_to_share_rows(T, d, type_):
    """One workgroup for all rows and several, rows of one wavefront and of many."""
    say(f"block norm gradient T={T} d={d} {type_}")
    for gate in ("channel", "full"):
        norm, x, y, dh, dn = make(T, d, TYPES[type_], gate)
        check_backward(gate, norm, x, y, dh, dn)


def test_many_long_rows_without_norm_out():
    """Rows of several wavefronts, several rows per workgroup, one round of sums each."""
    say("block norm T=1500 d=4104 without norm_out")
    norm, x, y, dh, dn = make(1500, 4104, torch.bfloat16, "token", norm_out=False)
    check_backward("no norm_out", norm, x, y, dh, dn)


def test_norm_alone():
    say("block norm without a block output")
    norm, x, _, dh, dn = make(40, 328, torch.bfloat16, "none", y=False, norm_out=False)
    check_forward("no y", norm, x, None)
    check_backward("no y", norm, x, None, dh, dn)
    check_backward("no y, dn", norm, x, None, None, dn)
    norm.residual_scale = 1.0
    h, n = moe.moe_block_norm(norm, x)
    assert h is None and n.shape == x.shape


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("offset,pad", [(1, 2), (8, 8)])
def test_strided_and_unaligned_rows(type_, offset, pad):
    say(f"block norm strided {type_} offset={offset}")
    for gate in ("token", "full"):
        norm, x, y, dh, dn = make(10, 300, TYPES[type_], gate)
        norm.gate = wide(norm.gate, offset, pad)
        check_forward("strided", norm, x, y, lambda t: wide(t, offset, pad))
        check_backward("strided", norm, x, y, dh, dn, lambda t: wide(t, offset, pad))


def test_extreme_rows():
    """Rows of zeros, of large and of tiny values: eps keeps the statistics finite."""
    say("block norm of extreme rows")
    norm, x, y, dh, dn = make(6, 96, torch.float32, "channel")
    x[0], y[0] = 0.0, 0.0
    y[1] = 0.0
    x[2], y[2] = x[2] * 1e15, y[2] * 1e15
    x[3], y[3] = x[3] * 1e-20, y[3] * 1e-20
    x[4] = 0.0
    check_forward("extreme", norm, x, y)
    check_backward("extreme", norm, x, y, dh, dn)


def test_in_place_outputs():
    say("block norm in place")
    for T, d in ((17, 520), (700, 2048)):
        norm, x, y, dh, dn = make(T, d, torch.bfloat16, "full")
        h0, n0 = moe.moe_block_norm(norm, x, y)
        h, n = x.clone(), y.clone()
        moe.moe_block_norm_into(norm, h, n, h, n)
        assert torch.equal(h, h0) and torch.equal(n, n0)
        ref = moe.moe_block_norm_backward(norm, x, y, dh, dn)
        ws = moe.alloc_block_norm_workspace(T, d, DEV)
        for dy_is in ("y", "dn"):
            dx, yy, dd = dh.clone(), y.clone(), dn.clone()
            out = moe.BlockNormGrads(dx=dx, dy=yy if dy_is == "y" else dd, dgate=torch.empty_like(x),
                                     dnorm_out=torch.empty(d, device=DEV), dnorm_in=torch.empty(d, device=DEV))
            moe.moe_block_norm_backward_into(norm, x, yy, out, ws, dx, dd)
            for q in ("dx", "dy", "dgate", "dnorm_out", "dnorm_in"):
                assert torch.equal(getattr(out, q), getattr(ref, q)), (dy_is, q)


@pytest.mark.parametrize("d", [2052, 4104, 8201])
def test_in_place_without_norms(d):
    """Rows of several wavefronts whose last pieces overlap, h in place of x or y, dx in
    place of dh: no norm, so no row sum orders loads and stores."""
    say(f"block norm in place, no norms, d={d}")
    T = 600
    norm, x, y, dh, _ = make(T, d, torch.bfloat16, "channel", norm_out=False, norm_in=False)
    ref, _ = moe.moe_block_norm(norm, x, y)
    for _ in range(5):
        h = x.clone()
        moe.moe_block_norm_into(norm, h, y, h)
        assert torch.equal(h, ref)
        h = y.clone()
        moe.moe_block_norm_into(norm, x, h, h)
        assert torch.equal(h, ref)
    only = moe.BlockNorm(residual_scale=0.5)
    ref = moe.moe_block_norm_backward(only, x, None, dh).dx
    for _ in range(5):
        dx = dh.clone()
        moe.moe_block_norm_backward_into(only, x, None, moe.BlockNormGrads(dx=dx), None, dx)
        assert torch.equal(dx, ref)


def test_broadcast_inputs():
    """One row for every token as residual stream, block output, gate or gradient."""
    say("block norm of expanded rows")
    T, d = 9, 520
    norm, x, y, dh, dn = make(T, d, torch.float32, "full")
    norm.gate = norm.gate[:1].expand(T, d)
    x, y, dh, dn = (t[:1].expand(T, d) for t in (x, y, dh, dn))
    check_forward("expanded", norm, x, y)
    check_backward("expanded", norm, x, y, dh, dn)
    norm.gate = norm.gate[:1, :1].expand(T, 1)
    check_forward("expanded token gate", norm, x, y)
    check_backward("expanded token gate", norm, x, y, dh, dn)


def test_long_rows_captured():
    """Rows whose vectors need more than 64 KiB of LDS, in a captured graph."""
    say("block norm d=16384 captured")
    T, d = 300, 16384
    norm, x, y, dh, dn = make(T, d, torch.bfloat16, "channel")
    ws = moe.alloc_block_norm_workspace(T, d, DEV)
    f = dict(dtype=torch.float32, device=DEV)
    grads = moe.BlockNormGrads(torch.empty_like(x), torch.empty_like(x), torch.empty(d, **f), torch.empty(d, **f),
                               torch.empty(d, **f))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_block_norm_backward_into(norm, x, y, grads, ws, dh, dn)
    ref = moe.moe_block_norm_backward(norm, x, y, dh, dn)
    for i in range(3):
        grads.dx.zero_(), grads.dnorm_in.zero_()
        g.replay()
        torch.cuda.synchronize()
        for q in ("dx", "dy", "dgate", "dnorm_out", "dnorm_in"):
            assert torch.equal(getattr(grads, q), getattr(ref, q)), (i, q)


def test_two_streams_at_once():
    say("block norm gradient on two streams, each with its workspace")
    jobs = []
    for T, d, gate in ((700, 1100, "channel"), (6, 2048, "token")):
        norm, x, y, dh, dn = make(T, d, torch.bfloat16, gate)
        ref = moe.moe_block_norm_backward(norm, x, y, dh, dn)
        out = moe.BlockNormGrads(*(torch.zeros_like(getattr(ref, q))
                                   for q in ("dx", "dy", "dgate", "dnorm_out", "dnorm_in")))
        jobs.append((norm, x, y, dh, dn, ref, out, moe.alloc_block_norm_workspace(T, d, DEV), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for norm, x, y, dh, dn, _ref, out, ws, stream in jobs:
            moe.moe_block_norm_backward_into(norm, x, y, out, ws, dh, dn, stream)
    torch.cuda.synchronize()
    for *_, ref, out, _ws, _stream in jobs:
        for q in ("dx", "dy", "dgate", "dnorm_out", "dnorm_in"):
            assert torch.equal(getattr(out, q), getattr(ref, q)), q


def test_no_rows():
    say("block norm T = 0")
    norm, x, y, dh, dn = make(1, 48, torch.bfloat16, "channel")
    e = x[:0]
    h, n = moe.moe_block_norm(norm, e, e)
    assert h.shape == (0, 48) and n.shape == (0, 48)
    g = moe.moe_block_norm_backward(norm, e, e, e, e)
    torch.cuda.synchronize()
    for v in (g.dnorm_in, g.dnorm_out, g.dgate):
        assert torch.equal(v, torch.zeros(48, device=DEV))


def test_no_rows_of_infinite_weights():
    """Sums over no rows are zero, whatever they would be multiplied with."""
    say("block norm T = 0 with infinite weights")
    norm, x, y, dh, dn = make(1, 48, torch.float32, "channel")
    norm.norm_out[3], norm.gate[5] = float("inf"), float("nan")
    e = x[:0]
    g = moe.moe_block_norm_backward(norm, e, e, e, e)
    torch.cuda.synchronize()
    for v in (g.dnorm_in, g.dnorm_out, g.dgate):
        assert torch.equal(v, torch.zeros(48, device=DEV))


@pytest.mark.parametrize("d", [40, 2048])
def test_large_rows_without_dn(d):
    """Without dn the statistics of h are not used: squares past float32 change nothing."""
    say(f"block norm gradient of large rows without dn, d={d}")
    norm, x, y, dh, _ = make(3, d, torch.float32, "token", norm_out=False)
    norm.gate[1] = 1.0
    g = moe.moe_block_norm_backward(norm, x, y * 1e25, dh, None)
    ref = (f64(dh) * f64(y * 1e25)).sum(axis=1, keepdims=True)
    size = (np.abs(f64(dh)) * np.abs(f64(y * 1e25))).sum(axis=1, keepdims=True)
    assert_near("dgate", g.dgate, ref, row_sum_ops(d) * U32 * size)
    dx = f64(dh) * 0.75
    assert_near("dx", g.dx, dx, U32 * np.abs(dx))
    assert not g.dnorm_in.any()


def test_some_gradients_only():
    """Gradients that are not wanted change nothing about the others."""
    say("block norm with some gradients")
    T, d = 600, 200
    norm, x, y, dh, dn = make(T, d, torch.float32, "channel")
    ref = moe.moe_block_norm_backward(norm, x, y, dh, dn)
    ws = moe.alloc_block_norm_workspace(T, d, DEV)
    for q in ("dx", "dy", "dgate", "dnorm_out", "dnorm_in"):
        out = moe.BlockNormGrads(**{q: torch.full_like(getattr(ref, q), 7.0)})
        moe.moe_block_norm_backward_into(norm, x, y, out, ws if q[1] in "gn" else None, dh, dn)
        assert torch.equal(getattr(out, q), getattr(ref, q)), q


def test_graph_side_stream_and_determinism():
    say("block norm captured, replayed and on another stream")
    T, d = 1500, 328
    norm, x, y, dh, dn = make(T, d, torch.bfloat16, "channel")
    h, n = torch.empty_like(x), torch.empty_like(x)
    grads = moe.BlockNormGrads(torch.empty_like(x), torch.empty_like(x), torch.empty(d, device=DEV),
                               torch.empty(d, device=DEV), torch.empty(d, device=DEV))
    ws = moe.alloc_block_norm_workspace(T, d, DEV)
    outs = (h, n, grads.dx, grads.dy, grads.dgate, grads.dnorm_out, grads.dnorm_in)

    def step():
        moe.moe_block_norm_into(norm, x, y, h, n)
        moe.moe_block_norm_backward_into(norm, x, y, grads, ws, h, n)

    step()
    torch.cuda.synchronize()
    ref = [t.clone() for t in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(3):
        for t in outs:
            t.zero_()
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        for t, q in zip(outs, ref):
            assert torch.equal(t, q), f"replay {i}"
        step()
        torch.cuda.synchronize()
        for t, q in zip(outs, ref):
            assert torch.equal(t, q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.moe_block_norm_backward(norm, x, y, ref[0], ref[1], stream=side)
    side.synchronize()
    assert torch.equal(got.dx, ref[2]) and torch.equal(got.dnorm_in, ref[6])


def test_binding_refusals():
    say("block norm refusals")
    norm, x, y, dh, dn = make(4, 16, torch.bfloat16, "channel")
    with pytest.raises(TypeError):
        moe.moe_block_norm(norm, x.double(), y)
    with pytest.raises(TypeError):
        moe.moe_block_norm(norm, x.half(), y.half())          # parameters of another type
    with pytest.raises(ValueError):
        moe.moe_block_norm(norm, x, y[:, :8])
    with pytest.raises(ValueError):
        moe.moe_block_norm(moe.BlockNorm(norm_in=norm.norm_in[:8]), x)
    with pytest.raises(ValueError):
        moe.moe_block_norm(moe.BlockNorm(norm_in=norm.norm_in, gate=torch.ones(3, 16, device=DEV).bfloat16()), x, y)
    with pytest.raises(moe.MoeError):
        moe.moe_block_norm(norm, x)                            # norm_out and gate without y
    with pytest.raises(moe.MoeError):
        moe.moe_block_norm(moe.BlockNorm(norm_in=norm.norm_in, eps=0.0), x)
    with pytest.raises(moe.MoeError):
        moe.moe_block_norm(moe.BlockNorm(norm_in=torch.ones(16392, device=DEV)), torch.ones(1, 16392, device=DEV))
    with pytest.raises(moe.MoeError):
        moe.moe_block_norm_into(norm, x, y, torch.empty_like(x), None)   # norm_in without n
    with pytest.raises(moe.MoeError):
        moe.moe_block_norm_backward(norm, x, y)                # neither dh nor dn
    g = moe.BlockNormGrads(dnorm_in=torch.empty(16, device=DEV))
    with pytest.raises(moe.MoeError):
        moe.moe_block_norm_backward_into(norm, x, y, g, None, dh, dn)
