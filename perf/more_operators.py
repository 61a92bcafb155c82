"""Measured cases of the experts in training and of dropout.

Two groups of operators:

- ``ffn`` / ``ffn_grad``: gated feed-forward blocks with 16-bit weights, over rows sorted by
  expert or over all rows with one set of weights.  For a row x of expert e
  g = Wg_e x, u = Wu_e x, h = drop(act(g) * u), y = Wd_e h, with act = silu or gelu (tanh form).
  The gradient is taken at the g, u and h that the forward call stored:
  dh = drop(dy Wd), dg = dh u act'(g), du = dh act(g), dx = dg Wg + du Wu,
  dW13 = [dg, du]^T x, dWd = dy^T h.
- ``dropout``: out = residual + x * keep / (1 - p), where keep comes from a counter-based
  generator, so that its gradient is the same call on the gradient and no mask is stored.

keep of element (r, c): Philox-4x32 with ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel
random numbers: as easy as 1, 2, 3", 2011) of the counter
(c / 8 + site * 2^21, r, step mod 2^32, step / 2^32) under the key (seed mod 2^32,
seed / 2^32); its four words are eight 16-bit numbers, low halves first, and the element is
kept where number c mod 8 is at least round(p * 2^16).  The p in 1 / (1 - p) is that number
over 2^16.

``run`` computes them in elementary torch operations, or, where ``own`` is true, through the
package's entry points.  ``exact`` computes the same in float64.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token through a dense block, as a shared expert sees it in decode: bound by launches
        dict(name="ffn one", op="ffn", T=1, k=1, E=1, d=2048, I=1024, type="bf16", act="silu", p=0.0, save=False),
        # a decode step of 16 requests: 128 rows on 64 experts, bound by the weights' bytes
        dict(name="ffn decode", op="ffn", T=16, k=8, E=64, d=2048, I=1024, type="bf16", act="silu", p=0.0, save=False),
        # a prefill batch over the same experts
        dict(name="ffn prefill", op="ffn", T=4096, k=8, E=64, d=2048, I=1024, type="bf16", act="silu", p=0.0,
             save=False),
        # few wide experts
        dict(name="ffn wide", op="ffn", T=1024, k=2, E=8, d=4096, I=14336, type="bf16", act="silu", p=0.0, save=False),
        # forward pass of a training step with odd sizes, the other activation, dropout and stored projections
        dict(name="ffn odd", op="ffn", T=777, k=3, E=13, d=1000, I=712, type="fp16", act="gelu", p=0.1, save=True),
        # training step at the prefill batch's size: every gradient, dropout drawn again
        dict(name="ffn grad train", op="ffn_grad", T=4096, k=8, E=64, d=2048, I=1024, type="bf16", act="silu", p=0.1),
        # one dense block of a training step
        dict(name="ffn grad dense", op="ffn_grad", T=4096, k=1, E=1, d=2048, I=8192, type="bf16", act="silu", p=0.0),
        # the odd sizes backward
        dict(name="ffn grad odd", op="ffn_grad", T=777, k=3, E=13, d=1000, I=712, type="fp16", act="gelu", p=0.1),
        # a short batch: few rows per expert, the weights and their gradients are most of the bytes
        dict(name="ffn grad short", op="ffn_grad", T=16, k=8, E=64, d=2048, I=1024, type="bf16", act="silu", p=0.0),
        # dropout of a short batch: bound by its launch
        dict(name="dropout short", op="dropout", T=16, d=2048, type="bf16", p=0.1, residual=True),
        # dropout before the residual's addition in a long training batch
        dict(name="dropout long", op="dropout", T=16384, d=2048, type="bf16", p=0.1, residual=True),
        # an odd width in float32, as the gradient sees it
        dict(name="dropout odd", op="dropout", T=3001, d=1111, type="fp32", p=0.5, residual=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "ffn_grad", "ffn_grad", "dropout"])
    if op == "dropout":
        kind = rng.choice(["bf16", "fp16", "fp32"])
        d = _log(rng, 1, 16384)
        T = _log(rng, 1, max(1, 16384 * 2048 // (d * (2 if kind == "fp32" else 1))))
        return dict(op=op, T=T, d=d, type=kind, p=rng.choice([0.0, 0.1, 0.25, 0.5, 0.9]),
                    residual=rng.random() < 0.6)
    E = 1 if rng.random() < 0.3 else _log(rng, 2, 256)
    k = rng.randint(1, min(E, 8))
    d, I = 8 * _log(rng, 8, 512), 8 * _log(rng, 8, 1792)
    # no more weights and no more products than the largest listed cases have
    while 3 * E * d * I > 64 * 3 * 2048 * 1024 * 2:
        E = max(1, E // 2)
        k = min(k, E)
        if E == 1:
            break
    most = 32768 * 2048 * 1024 // (d * I)
    T = _log(rng, 1, max(1, min(32768, most) // k))
    s = dict(op=op, T=T, k=k, E=E, d=d, I=I, type=rng.choice(["bf16", "bf16", "fp16"]),
             act=rng.choice(["silu", "silu", "gelu"]), p=rng.choice([0.0, 0.0, 0.1, 0.5]))
    if op == "ffn":
        s["save"] = rng.random() < 0.5
        s["p"] = s["p"] if s["save"] else 0.0
    return s


# ---------------------------------------------------------------- inputs

def _popularity(E):
    w = [1.0 / math.sqrt(e + 1) for e in range(E)]
    total = sum(w)
    return [v / total for v in w]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    s = dict(case)
    t, T, d = TYPES[s["type"]], s["T"], s["d"]
    s["state"] = torch.tensor([seed * 0x9E3779B97F4A7C15 % 2 ** 63, 1000003 * seed % 2 ** 40], device="cuda")
    if s["op"] == "dropout":
        s["site"] = 3
        s["x"] = normal(T, d, dtype=t)
        s["r"] = normal(T, d, dtype=t) if s["residual"] else None
        s["out"] = torch.empty(T, d, dtype=t, device="cuda")
        return s
    E, k, I = s["E"], s["k"], s["I"]
    R = T * k
    s["site"] = 1
    # rows sorted by expert: unequally popular experts, as the routing of T tokens to k of E has them
    if E > 1:
        u = torch.rand(T, E, generator=g, device="cuda").clamp(1e-6, 1 - 1e-6)
        logits = torch.tensor(_popularity(E), device="cuda").log() - torch.log(-torch.log(u))
        counts = torch.bincount(torch.topk(logits, k, dim=1)[1].reshape(-1), minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["bounds"] = s["offsets"].tolist()
    else:
        s["offsets"], s["bounds"] = None, [0, R]
    s["x"] = normal(R, d, dtype=t)
    s["w13"] = torch.empty(E, 2 * I, d, dtype=t, device="cuda")
    s["w2"] = torch.empty(E, d, I, dtype=t, device="cuda")
    for e in range(E):
        s["w13"][e] = normal(2 * I, d, std=d ** -0.5)
        s["w2"][e] = normal(d, I, std=I ** -0.5)
    grad = s["op"] == "ffn_grad"
    s["gu"] = torch.empty(R, 2 * I, dtype=t, device="cuda") if grad or s["save"] else None
    s["h"] = torch.empty(R, I, dtype=t, device="cuda")
    if not grad:
        s["y"] = torch.empty(R, d, dtype=t, device="cuda")
        return s
    # what the forward call of the step stored
    keep = _keep(s, R, I) if s["p"] else None
    for e, (a, b) in _experts(s):
        gu = s["x"][a:b].float() @ s["w13"][e].float().t()
        h = _act(s["act"], gu[:, :I])[0] * gu[:, I:]
        s["gu"][a:b] = gu
        s["h"][a:b] = h if keep is None else torch.where(keep[a:b], h * _scale(s), 0.0)
    s["dy"] = normal(R, d, std=0.1, dtype=t)
    s["dx"] = torch.empty_like(s["x"])
    s["dw13"], s["dw2"] = torch.empty_like(s["w13"]), torch.empty_like(s["w2"])
    return s


# ---------------------------------------------------------------- plain forms

def _experts(s):
    b = s["bounds"]
    return [(e, (b[e], b[e + 1])) for e in range(s["E"]) if b[e + 1] > b[e]]


def _act(name, g):
    """The activation and its derivative."""
    if name == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        return g * p, p * (1.0 + g * (1.0 - p))
    c = math.sqrt(2.0 / math.pi)
    th = torch.tanh(c * (g + 0.044715 * g * g * g))
    return (0.5 * g * (1.0 + th),
            0.5 * (1.0 + th) + 0.5 * g * (1.0 - th * th) * c * (1.0 + 3.0 * 0.044715 * g * g))


def _threshold(s):
    return int(math.floor(s["p"] * 65536 + 0.5))


def _scale(s):
    return 65536.0 / (65536 - _threshold(s)) if _threshold(s) < 65536 else 0.0


def _keep(s, rows, cols):
    """keep [rows, cols]: ten rounds on 32-bit words held in int64."""
    low = 0xFFFFFFFF
    seed, step = s["state"][0], s["state"][1]
    c0 = (torch.arange((cols + 7) // 8, device="cuda") + s["site"] * 2 ** 21)[None, :]
    c1 = torch.arange(rows, device="cuda")[:, None]
    c2, c3 = step & low, (step >> 32) & low
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.broadcast_tensors(c0, c1, c2, c3)
    halves = torch.stack([v for w in words for v in (w & 0xFFFF, w >> 16)], dim=2)
    return halves.reshape(rows, -1)[:, :cols] >= _threshold(s)


def _plain(s):
    if s["op"] == "dropout":
        x = s["x"].float()
        out = torch.where(_keep(s, s["T"], s["d"]), x * _scale(s), 0.0)
        return (out if s["r"] is None else out + s["r"].float()).to(s["x"].dtype)
    t, I = s["x"].dtype, s["I"]
    keep = _keep(s, s["x"].shape[0], I) if s["p"] else None
    if s["op"] == "ffn":
        y = torch.empty_like(s["y"])
        h_all, gu_all = (torch.empty_like(s["h"]), torch.empty_like(s["gu"])) if s["save"] else (None, None)
        for e, (a, b) in _experts(s):
            gu = s["x"][a:b].float() @ s["w13"][e].float().t()
            h = _act(s["act"], gu[:, :I])[0] * gu[:, I:]
            h = h if keep is None else torch.where(keep[a:b], h * _scale(s), 0.0)
            y[a:b] = h @ s["w2"][e].float().t()
            if s["save"]:
                h_all[a:b], gu_all[a:b] = h, gu
        return {"y": y, "h": h_all, "gu": gu_all} if s["save"] else y
    dx, dw13, dw2 = torch.empty_like(s["x"]), torch.zeros_like(s["w13"]), torch.zeros_like(s["w2"])
    for e, (a, b) in _experts(s):
        x, dy, gu = s["x"][a:b].float(), s["dy"][a:b].float(), s["gu"][a:b].float()
        dh = dy @ s["w2"][e].float()
        dh = dh if keep is None else torch.where(keep[a:b], dh * _scale(s), 0.0)
        act, slope = _act(s["act"], gu[:, :I])
        dgu = torch.cat([dh * gu[:, I:] * slope, dh * act], dim=1)
        dx[a:b] = dgu @ s["w13"][e].float()
        dw13[e] = dgu.t() @ x
        dw2[e] = dy.t() @ s["h"][a:b].float()
    return {"dx": dx.to(t), "dw13": dw13, "dw2": dw2}


# ---------------------------------------------------------------- the package's calls

def _own(s):
    import w4a16_grouped_expert_amd as moe
    drop = moe.Dropout(s["p"], s["state"], s["site"]) if s["p"] or s["op"] == "dropout" else None
    if s["op"] == "dropout":
        return moe.moe_dropout_into(s["x"], drop, s["out"], residual=s["r"])
    act = moe.ACT_SILU if s["act"] == "silu" else moe.ACT_GELU
    if s["op"] == "ffn":
        moe.moe_gated_ffn_into(s["x"], s["w13"], s["w2"], s["y"], s["h"], offsets=s["offsets"], gu=s["gu"],
                               activation=act, dropout=drop)
        return {"y": s["y"], "h": s["h"], "gu": s["gu"]} if s["save"] else s["y"]
    if "ws" not in s:
        s["ws"] = moe.alloc_gated_ffn_workspace(s["x"].shape[0], s["d"], s["I"], s["E"], s["x"].device)
    grads = moe.GatedFfnGrads(drows=s["dx"], dw13=s["dw13"], dw2=s["dw2"])
    moe.moe_gated_ffn_backward_into(s["dy"], s["x"], s["w13"], s["w2"], s["gu"], s["h"], grads, s["ws"],
                                    offsets=s["offsets"], activation=act, dropout=drop)
    return {"dx": s["dx"], "dw13": s["dw13"], "dw2": s["dw2"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    s = case
    T, d, b = s["T"], s["d"], TYPES[s["type"]].itemsize
    if s["op"] == "dropout":
        return {"bytes": T * d * b * (3 if s["residual"] else 2), "flops": 3 * T * d}
    R, I, E = T * s["k"], s["I"], s["E"]
    used = sum(1 - (1 - p) ** R for p in _popularity(E))  # experts with a row at all
    weights = 3 * d * I * b
    if s["op"] == "ffn":  # rows in, y (and h, g, u) out
        return {"bytes": used * weights + R * b * (2 * d + (3 * I if s["save"] else 0)), "flops": 6 * R * d * I}
    # rows, dy, h, g, u in and dx out; every weight's gradient out
    return {"bytes": (used + E) * weights + R * b * (3 * d + 3 * I), "flops": 12 * R * d * I}


# ---------------------------------------------------------------- in 64 bits

def _kept(s, rows, cols):
    """keep [rows, cols] by numpy's unsigned words, a block of rows at a time."""
    u64 = np.uint64
    half, low = u64(32), u64(0xFFFFFFFF)
    seed, step = (int(v) for v in s["state"].cpu())
    out = np.empty((rows, cols), dtype=bool)
    n = -(-cols // 8)
    for r0 in range(0, rows, 4096):
        m = min(4096, rows - r0)
        ctr = [np.broadcast_to(np.arange(n, dtype=u64) + u64(s["site"] << 21), (m, n)),
               np.broadcast_to(np.arange(r0, r0 + m, dtype=u64)[:, None], (m, n)),
               np.full((m, n), step & 0xFFFFFFFF, dtype=u64), np.full((m, n), step >> 32, dtype=u64)]
        key = [seed & 0xFFFFFFFF, seed >> 32]
        for _ in range(10):
            left, right = u64(0xD2511F53) * ctr[0], u64(0xCD9E8D57) * ctr[2]
            ctr = [(right >> half) ^ ctr[1] ^ u64(key[0]), right & low, (left >> half) ^ ctr[3] ^ u64(key[1]),
                   left & low]
            key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
        numbers = np.stack(ctr, axis=2).astype("<u4").view("<u2").reshape(m, 8 * n)
        out[r0:r0 + m] = numbers[:, :cols] >= _threshold(s)
    return torch.from_numpy(out).cuda()


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    factor = None
    if s["op"] == "dropout" or s["p"]:
        shape = (s["T"], s["d"]) if s["op"] == "dropout" else (s["x"].shape[0], s["I"])
        factor = torch.zeros(shape, dtype=f64, device="cuda")
        factor[_kept(s, *shape)] = _scale(s)
    if s["op"] == "dropout":
        out = s["x"].double() * factor
        return out if s["r"] is None else s["r"].double() + out
    I, R = s["I"], s["x"].shape[0]

    def gated(gu, rows):
        g, u = gu[:, :I], gu[:, I:]
        if s["act"] == "silu":
            z = u * g * torch.sigmoid(g)
        else:
            z = u * g / 2 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
        return z if factor is None else z * factor[rows]

    if s["op"] == "ffn":
        out = {"y": torch.empty(R, s["d"], dtype=f64, device="cuda")}
        if s["save"]:
            out["h"] = torch.empty(R, I, dtype=f64, device="cuda")
            out["gu"] = torch.empty(R, 2 * I, dtype=f64, device="cuda")
        for e in range(s["E"]):
            rows = slice(s["bounds"][e], s["bounds"][e + 1])
            gu = torch.mm(s["x"][rows].double(), s["w13"][e].double().t())
            h = gated(gu, rows)
            out["y"][rows] = torch.mm(h, s["w2"][e].double().t())
            if s["save"]:
                out["h"][rows], out["gu"][rows] = h, gu
        return out if s["save"] else out["y"]
    out = {"dx": torch.empty(R, s["d"], dtype=f64, device="cuda"),
           "dw13": torch.zeros(s["w13"].shape, dtype=f64, device="cuda"),
           "dw2": torch.zeros(s["w2"].shape, dtype=f64, device="cuda")}
    for e in range(s["E"]):
        rows = slice(s["bounds"][e], s["bounds"][e + 1])
        dy = s["dy"][rows].double()
        # the block's own gradient by differentiating its definition at the stored projections
        gu = s["gu"][rows].double().requires_grad_(True)
        (gated(gu, rows) * torch.mm(dy, s["w2"][e].double())).sum().backward()
        out["dx"][rows] = torch.mm(gu.grad, s["w13"][e].double())
        out["dw13"][e] = torch.mm(gu.grad.t(), s["x"][rows].double())
        out["dw2"][e] = torch.mm(dy.t(), s["h"][rows].double())
    return out
