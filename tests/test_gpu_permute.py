"""moe_permute, moe_unpermute and their gradients against the float64 reference."""
import numpy as np
import pytest
import torch

import w4a16_grouped_expert_amd as moe
from oracle import rows as orow

from gpu_helpers import say
from rows_helpers import TYPES, U32, assert_near, f64, half_step, row_sum_ops, wide

pytestmark = pytest.mark.gpu
DEV = "cuda"

# tokens, width, slots: single tokens and long batches, widths of one element, below and
# past a wavefront's pieces, odd ones, every slot count class
SHAPES = [(1, 1, 1), (1, 4096, 2), (3, 7, 2), (5, 64, 3), (16, 2048, 8), (33, 1111, 16), (130, 520, 8), (65, 8, 5),
          (257, 96, 1), (40, 4104, 6), (700, 2048, 8), (9, 12345, 4)]


def make(T, d, k, dtype, weighted, dropped, seed=0):
    g = torch.Generator().manual_seed(seed * 1000 + T * 7 + d * 3 + k)
    P = T * k
    order = torch.randperm(P, generator=g)
    keep = torch.rand(P, generator=g) >= dropped
    if dropped and T > 2:
        keep[k:2 * k] = False  # one token loses every pair
    pos = torch.full((P,), -1, dtype=torch.int32)
    pos[order[keep[order]]] = torch.arange(int(keep.sum()), dtype=torch.int32)
    w = torch.rand(T, k, generator=g) if weighted else None
    x = torch.randn(T, d, generator=g).to(dtype)
    r = torch.randn(P, d, generator=g).to(dtype)
    return (pos.to(DEV), None if w is None else w.to(DEV), x.to(DEV), r.to(DEV), int(keep.sum()))


def check_all(name, pos, w, x, r, k, num_rows=None, lay=lambda t: t):
    """The four calls on inputs x [T, d] (token rows) and r [P, d] (sorted rows)."""
    T, d = x.shape
    R = r.shape[0] if num_rows is None else num_rows
    r = r[:R]
    dt = x.dtype
    p, wn, xn, rn = pos.cpu().numpy(), f64(w), f64(x), f64(r)
    xl, rl = lay(x), lay(r)
    mark = 7.0
    named = np.zeros(R, dtype=bool)
    named[p[(p >= 0) & (p < R)]] = True

    def sorted_out(call, ref_of):
        out = lay(torch.full((R, d), mark, dtype=dt, device=DEV))
        call(out)
        torch.cuda.synchronize()
        ref = ref_of(np.full((R, d), mark))
        # one product in float32, one rounding; without weights the bits are copied
        bound = np.zeros_like(ref) if w is None else half_step(dt, ref) * (1 + 2 * U32) + np.abs(ref) * U32
        bound[~named] = 0.0  # rows that no pair names are left as they were
        assert_near(name, out, ref, bound)

    def token_out(call):
        out = lay(torch.full((T, d), mark, dtype=dt, device=DEV))
        call(out)
        torch.cuda.synchronize()
        ref = orow.unpermute(rn, p, k, wn)
        size = orow.unpermute(np.abs(rn), p, k, None if wn is None else np.abs(wn))
        e = (k + 1) * U32 * size  # k fused multiply-adds
        assert_near(name, out, ref, half_step(dt, np.abs(ref) + e) + e)

    def products(got):
        ref = orow.pair_products(xn, rn, p, k)
        size = orow.pair_products(np.abs(xn), np.abs(rn), p, k)
        assert_near(name + " dweights", got, ref, row_sum_ops(d) * U32 * size)

    sorted_out(lambda o: moe.moe_permute_into(xl, pos, k, o, w), lambda m: orow.permute(xn, p, k, R, wn, m))
    token_out(lambda o: moe.moe_unpermute_into(rl, pos, k, o, w))
    sorted_out(lambda o: moe.moe_unpermute_backward_into(xl, pos, k, o, w),
               lambda m: orow.permute(xn, p, k, R, wn, m))
    token_out(lambda o: moe.moe_permute_backward_into(rl, pos, k, o, w))
    dw = torch.full((T, k), float("nan"), device=DEV)
    sorted_out(lambda o: moe.moe_unpermute_backward_into(xl, pos, k, o, w, rl, dw),
               lambda m: orow.permute(xn, p, k, R, wn, m))
    products(dw)
    dw.fill_(float("nan"))
    token_out(lambda o: moe.moe_permute_backward_into(rl, pos, k, o, w, xl, dw))
    products(dw)


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("T,d,k", SHAPES)
def test_against_reference(T, d, k, type_):
    say(f"permute T={T} d={d} k={k} {type_}")
    for weighted in (False, True):
        for dropped in (0.0, 0.3):
            pos, w, x, r, _ = make(T, d, k, TYPES[type_], weighted, dropped)
            check_all(f"weighted={weighted} dropped={dropped}", pos, w, x, r, k)


@pytest.mark.parametrize("type_", list(TYPES))
@pytest.mark.parametrize("offset,pad", [(1, 2), (8, 8), (3, 0)])
def test_strided_and_unaligned_rows(type_, offset, pad):
    say(f"permute strided {type_} offset={offset}")
    for T, d, k in ((20, 264, 4), (7, 77, 3)):
        pos, w, x, r, _ = make(T, d, k, TYPES[type_], True, 0.2)
        check_all("strided", pos, w, x, r, k, lay=lambda t: wide(t, offset, pad))


def test_positions_past_the_last_row_and_rows_behind():
    say("permute with positions outside the rows")
    T, d, k = 50, 160, 4
    pos, w, x, r, placed = make(T, d, k, torch.bfloat16, True, 0.2)
    assert placed < T * k
    check_all("fewer rows", pos, w, x, r, k, num_rows=placed // 2)
    check_all("no rows", pos, w, x, r, k, num_rows=0)
    far = pos.clone()
    far[pos == 3] = 2 ** 31 - 1
    far[pos == 4] = -2 ** 31
    check_all("extreme positions", far, w, x, r, k)
    # NaN in rows that no pair names reaches nothing
    r2 = r.clone()
    r2[placed:] = float("nan")
    out = moe.moe_unpermute(r2, pos, k, T, w)
    dw = torch.empty(T, k, device=DEV)
    moe.moe_unpermute_backward_into(x, pos, k, torch.empty_like(r), w, r2, dw)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all() and torch.isfinite(dw).all()


@pytest.mark.parametrize("d", [40, 520, 2048])
@pytest.mark.parametrize("k", [3, 9])
def test_infinities_beside_dropped_pairs(d, k):
    """Infinite and NaN weights and elements reach what the kept pairs make of them only."""
    say(f"permute with infinities d={d} k={k}")
    T = 5
    pos = torch.arange(T * k, dtype=torch.int32).reshape(T, k)
    pos[0, 1] = -1         # dropped, its weight NaN
    pos[1, 0] = T * k      # dropped, its weight infinite
    pos[3] = -1            # a token without pairs, its element infinite
    x = torch.randint(1, 4, (T, d), generator=torch.Generator().manual_seed(d)).to(torch.float32)
    r = torch.randint(1, 4, (T * k, d), generator=torch.Generator().manual_seed(k)).to(torch.float32)
    w = torch.ones(T, k)
    w[0, 1], w[1, 0], w[2, k - 1] = float("nan"), float("inf"), float("inf")
    x[3, 5], x[1, 2], r[4 * k, 7] = float("inf"), float("nan"), float("inf")
    p, wn, xn, rn = pos.numpy().ravel(), f64(w), f64(x), f64(r)
    pos, w, x, r = pos.to(DEV), w.to(DEV), x.to(DEV), r.to(DEV)

    def same(got, ref):  # small integers: sums are exact
        np.testing.assert_array_equal(got.cpu().numpy(), ref.astype(np.float32))

    same(moe.moe_unpermute(r, pos, k, T, w), orow.unpermute(rn, p, k, wn))
    rows, drows, dx = torch.zeros_like(r), torch.zeros_like(r), torch.empty_like(x)
    same(moe.moe_permute_into(x, pos, k, rows, w), orow.permute(xn, p, k, T * k, wn))
    dw = torch.full((T, k), 7.0, device=DEV)
    same(moe.moe_unpermute_backward_into(x, pos, k, drows, w, r, dw), orow.permute(xn, p, k, T * k, wn))
    same(dw, orow.pair_products(xn, rn, p, k))
    dw.fill_(7.0)
    same(moe.moe_permute_backward_into(r, pos, k, dx, w, x, dw), orow.unpermute(rn, p, k, wn))
    same(dw, orow.pair_products(xn, rn, p, k))


def test_no_pair_left_and_no_token():
    say("permute with every pair dropped, and T = 0")
    T, d, k = 6, 40, 3
    pos, w, x, r, _ = make(T, d, k, torch.float16, True, 0.0)
    check_all("none left", torch.full_like(pos, -1), w, x, r, k)
    e = torch.empty(0, d, dtype=torch.float16, device=DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    rows = r.clone()
    moe.moe_permute_into(e, none, k, rows)
    moe.moe_unpermute_into(rows, none, k, e)
    torch.cuda.synchronize()
    assert torch.equal(rows, r)


def test_one_row_for_every_token():
    say("permute of an expanded row")
    T, d, k = 12, 72, 2
    pos, w, x, r, _ = make(T, d, k, torch.float32, True, 0.0)
    one = x[:1].expand(T, d)
    rows = torch.empty_like(r)
    moe.moe_permute_into(one, pos, k, rows, w)
    assert torch.equal(rows, moe.moe_permute(one.contiguous(), pos, k, w))


def test_weights_bits_and_determinism():
    """Copies keep the bits (NaN payloads, -0, subnormals); equal calls give equal bits."""
    say("permute bits")
    T, d, k = 8, 256, 2
    pos, w, _, r, _ = make(T, d, k, torch.bfloat16, True, 0.0)
    raw = torch.randint(-32768, 32768, (T, d), dtype=torch.int16, device=DEV)
    rows = moe.moe_permute(raw.view(torch.bfloat16), pos, k)
    for j in range(k):
        assert torch.equal(rows.view(torch.int16)[pos.view(T, k)[:, j].long()], raw)
    x = torch.randn(T, d, device=DEV).bfloat16()
    outs = []
    for _ in range(2):
        dw = torch.empty(T, k, device=DEV)
        dr = torch.empty_like(r)
        moe.moe_unpermute_backward_into(x, pos, k, dr, w, r, dw)
        outs.append((dr, dw, moe.moe_unpermute(r, pos, k, T, w)))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    """Calls that share their inputs run on two streams at a time."""
    say("permute on two streams at once")
    T, d, k = 2000, 1032, 4
    pos, w, x, r, _ = make(T, d, k, torch.bfloat16, True, 0.1)
    ref = moe.moe_unpermute(r, pos, k, T, w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(x) for _ in range(8)] for _ in streams]
    for i in range(8):
        for s, o in zip(streams, outs):
            moe.moe_unpermute_into(r, pos, k, o[i], w, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        for t in o:
            assert torch.equal(t, ref)


def test_timing_hooks():
    say("timing of the row operators")
    T, d, k = 64, 256, 2
    pos, w, x, r, _ = make(T, d, k, torch.bfloat16, True, 0.0)
    moe.timing_reset()
    moe.timing_enable(True)
    moe.moe_permute(x, pos, k)
    moe.moe_unpermute(r, pos, k, T, w)
    moe.moe_unpermute(r, pos, k, T, w)
    moe.timing_enable(False)
    ms, n = moe.timing_read("permute")
    assert n == 1 and ms > 0
    assert moe.timing_read("unpermute")[1] == 2
    moe.timing_reset()


def test_offsets_past_32_bits():
    T, d, k = 1 << 17, 2304, 8  # 2.4e9 elements of sorted rows
    say(f"permute with {T * k * d} elements")
    pos = torch.randperm(T * k, device=DEV).to(torch.int32)
    x = torch.randn(T, d, device=DEV).bfloat16()
    w = torch.rand(T, k, device=DEV)
    rows = moe.moe_permute(x, pos, k)
    p = pos.view(T, k).long()
    for t in (0, 1, T // 2, T - 1):
        assert torch.equal(rows[p[t]], x[t].expand(k, d))
    last = int(torch.argmax(pos))
    assert torch.equal(rows[T * k - 1], x[last // k])
    out = moe.moe_unpermute(rows, pos, k, T, w)
    for t in (0, T // 2, T - 1):
        ref = f64(x[t]) * f64(w[t]).sum()
        assert_near("out", out[t], ref, half_step(torch.bfloat16, ref) * 1.001 + (k + 1) * U32 * np.abs(ref))
    del rows, out
    torch.cuda.empty_cache()


def test_after_moe_align():
    """Positions from the library's own routing and alignment."""
    say("permute after moe_route + moe_align")
    T, d, E, k = 300, 128, 16, 4
    x = torch.randn(T, d, device=DEV).bfloat16()
    wr = torch.randn(E, d, device=DEV).bfloat16()
    route = moe.moe_route(x, wr, k)
    al = moe.moe_align(route.ids, E)
    rows = moe.moe_permute(x, al.pair_pos, k)
    assert torch.equal(rows, x[(al.sorted_pairs // k).long()])
    out = moe.moe_unpermute(rows, al.pair_pos, k, T)
    ref = f64(x) * k
    assert_near("k times x", out, ref, half_step(torch.bfloat16, ref) * 1.001 + (k + 1) * U32 * np.abs(ref))


def test_graph_and_side_stream():
    say("permute captured, replayed and on another stream")
    T, d, k = 37, 328, 5
    pos, w, x, r, _ = make(T, d, k, torch.bfloat16, True, 0.1)
    rows, out = torch.zeros_like(r), torch.empty_like(x)
    drows, dx = torch.zeros_like(r), torch.empty_like(x)
    dw1, dw2 = torch.empty(T, k, device=DEV), torch.empty(T, k, device=DEV)
    outs = (rows, out, drows, dx, dw1, dw2)

    def step():
        moe.moe_permute_into(x, pos, k, rows, w)
        moe.moe_unpermute_into(rows, pos, k, out, w)
        moe.moe_unpermute_backward_into(out, pos, k, drows, w, rows, dw1)
        moe.moe_permute_backward_into(drows, pos, k, dx, w, x, dw2)

    step()
    torch.cuda.synchronize()
    ref = [t.clone() for t in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(3):
        for t in outs:
            t.zero_()
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
    got = moe.moe_unpermute(ref[0], pos, k, T, w, stream=side)
    side.synchronize()
    assert torch.equal(got, ref[1])


def test_binding_refusals():
    say("permute refusals")
    T, d, k = 4, 16, 2
    pos, w, x, r, _ = make(T, d, k, torch.bfloat16, True, 0.0)
    with pytest.raises(TypeError):
        moe.moe_permute(x.double(), pos, k)
    with pytest.raises(TypeError):
        moe.moe_permute_into(x, pos, k, r.half())
    with pytest.raises(TypeError):
        moe.moe_permute(x, pos.long(), k)
    with pytest.raises(TypeError):
        moe.moe_permute(x, pos, k, w.bfloat16())
    with pytest.raises(ValueError):
        moe.moe_permute(x, pos[:-1], k)
    with pytest.raises(ValueError):
        moe.moe_permute(x.t(), pos, k)
    with pytest.raises(ValueError):
        moe.moe_permute(x, pos, k, w[:, :1])
    with pytest.raises(ValueError):
        moe.moe_permute(x, pos.cpu(), k)
    with pytest.raises(ValueError):
        moe.moe_permute_into(x, pos, k, r[:1].expand(8, d))
    with pytest.raises(ValueError):
        moe.moe_unpermute_backward_into(x, pos, k, r, w, rows=r)
    with pytest.raises(moe.MoeError):
        moe.moe_permute(x, torch.zeros(T * 17, dtype=torch.int32, device=DEV), 17)
