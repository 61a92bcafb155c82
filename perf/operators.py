"""Measured cases of the operators around the routed experts of one MoE block.

Three groups of operators, each with its gradient:

- ``permute`` / ``permute_grad`` / ``unpermute`` / ``unpermute_grad``: token rows sorted by
  expert and back, with the routing weights applied on the way.  With pos[t, j] the sorted
  position of pair (t, j), negative for a dropped pair:
  rows[pos[t, j]] = w[t, j] x[t] and out[t] = sum_j w[t, j] rows[pos[t, j]].
- ``norm`` / ``norm_grad``: h = a x + g * (rms(y) * v_out), n = rms(h) * v_in with
  rms(z) = z / sqrt(mean(z^2) + eps): the norm behind a block, its gate, the scaled residual
  and the norm before the next block.
- ``route_grad``: from the gradient of the routing weights to those of the logits, of the
  router's input and of its weight.

``run`` computes them in elementary torch operations, or, where ``own`` is true, through the
package's entry points.  ``exact`` computes the same in float64.
"""
import math

import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of 16 requests: the smallest call, bound by its launch
        dict(name="permute decode", op="permute", T=16, d=2048, E=64, k=8, type="bf16", weighted=False, dropped=0.0),
        # a prefill batch laid out by expert for the grouped products
        dict(name="permute prefill", op="permute", T=4096, d=2048, E=64, k=8, type="bf16", weighted=False, dropped=0.0),
        # its gradient in a training step with an odd width, weights on the inputs and pairs that were dropped
        dict(name="permute grad odd", op="permute_grad", T=777, d=1111, E=13, k=3, type="fp16", weighted=True,
             dropped=0.1),
        # one token of a wide layer in float32, back from its two experts
        dict(name="unpermute one", op="unpermute", T=1, d=4096, E=8, k=2, type="fp32", weighted=True, dropped=0.0),
        # the combine of a prefill batch or of a training step's forward pass
        dict(name="unpermute prefill", op="unpermute", T=4096, d=2048, E=64, k=8, type="bf16", weighted=True,
             dropped=0.0),
        # its gradient: the rows' and the routing weights'
        dict(name="unpermute grad prefill", op="unpermute_grad", T=4096, d=2048, E=64, k=8, type="bf16", weighted=True,
             dropped=0.0),
        # between two blocks of a decode step: norm, gate, residual and the next norm in one go
        dict(name="norm decode", op="norm", T=16, d=2048, type="bf16", y=True, norm_out=True, gate="channel",
             norm_in=True, scale=1.0),
        # the same for the largest prefill batch
        dict(name="norm prefill", op="norm", T=16384, d=2048, type="bf16", y=True, norm_out=True, gate="channel",
             norm_in=True, scale=1.0),
        # the gradient in a training step: inputs', both norm weights' and the gate's
        dict(name="norm grad prefill", op="norm_grad", T=8192, d=2048, type="bf16", y=True, norm_out=True,
             gate="channel", norm_in=True, scale=1.0),
        # float32 training of an odd width with a gate per token and a scaled residual
        dict(name="norm grad odd", op="norm_grad", T=1001, d=1111, type="fp32", y=True, norm_out=True, gate="token",
             norm_in=True, scale=0.5),
        # the router's gradient in a training step, weights renormalised over the selected experts
        dict(name="route grad", op="route_grad", T=4096, d=2048, E=64, k=8, renormalize=True, aux=False),
        # many experts, softmax over all of them, and a loss on the logits beside
        dict(name="route grad many", op="route_grad", T=1021, d=4096, E=257, k=6, renormalize=False, aux=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["permute", "permute_grad", "unpermute", "unpermute_grad", "norm", "norm_grad", "route_grad"])
    if op == "route_grad":
        E = _log(rng, 2, 512)
        d = 8 * _log(rng, 8, 1024)
        T = _log(rng, 1, max(1, min(8192, (4096 * 2048 * 64) // (d * max(E, 64)))))
        return dict(op=op, T=T, d=d, E=E, k=rng.randint(1, min(E, 16)), renormalize=rng.random() < 0.7,
                    aux=rng.random() < 0.4)
    kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    width = rng.random()
    d = _log(rng, 64, 8192)
    if width < 0.6:
        d = max(64, d // 64 * 64)
    size = 2 if kind == "fp32" else 1
    if op in ("norm", "norm_grad"):
        y = rng.random() < 0.8
        norm_in = not y or rng.random() < 0.7
        T = _log(rng, 1, max(1, min(16384, 8192 * 2048 // (d * size))))
        return dict(op=op, T=T, d=d, type=kind, y=y, norm_out=y and rng.random() < 0.7,
                    gate=rng.choice(["none", "channel", "token", "full"]) if y else "none", norm_in=norm_in,
                    scale=rng.choice([1.0, 1.0, 0.5, 1.25]))
    E = _log(rng, 2, 512)
    k = rng.randint(1, min(E, 16))
    T = _log(rng, 1, max(1, min(16384, 4096 * 2048 * 8 // (d * k * size))))
    return dict(op=op, T=T, d=d, E=E, k=k, type=kind, weighted=rng.random() < 0.7,
                dropped=rng.choice([0.0, 0.0, 0.1]))


# ---------------------------------------------------------------- inputs

def _maker(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    return normal, uniform


def _routed(s, uniform):
    """Routing of T tokens to k of E unequally popular experts: logits, ids, weights, positions."""
    T, E, k = s["T"], s["E"], s["k"]
    gumbel = -torch.log(-torch.log(uniform(T, E).clamp(1e-6, 1 - 1e-6)))
    logits = gumbel - 0.5 * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    top, ids = torch.topk(logits, k, dim=1)
    weights = torch.softmax(top, dim=1)
    return logits, ids.to(torch.int32), weights


def _positions(ids, E, dropped, uniform):
    """Positions of the pairs in a stable sort by expert; -1 for those that are dropped."""
    flat = ids.reshape(-1).long()
    if dropped:
        flat = torch.where(uniform(flat.numel()) < dropped, torch.full_like(flat, E), flat)
    order = torch.sort(flat, stable=True)[1]
    pos = torch.empty_like(flat)
    pos[order] = torch.arange(flat.numel(), device="cuda")
    return torch.where(flat < E, pos, torch.full_like(pos, -1)).to(torch.int32)


def prepare(case, seed):
    normal, uniform = _maker(seed)
    s = dict(case)
    op, T, d = s["op"], s["T"], s["d"]
    if op == "route_grad":
        E, k = s["E"], s["k"]
        s["x"] = normal(T, d, dtype=torch.bfloat16)
        s["w"] = normal(E, d, std=0.02, dtype=torch.bfloat16)
        s["logits"] = (s["x"].double() @ s["w"].double().t()).float()
        top, ids = torch.topk(s["logits"], k, dim=1)
        s["ids"] = ids.to(torch.int32)
        s["weights"] = torch.softmax(top, dim=1) if s["renormalize"] else torch.softmax(s["logits"], 1).gather(1, ids)
        s["dweights"] = normal(T, k, std=0.1)
        s["dlogits"] = normal(T, E, std=1e-3) if s["aux"] else None
        s["dx_add"] = normal(T, d, std=0.01, dtype=torch.bfloat16)
        s["dx"] = torch.empty_like(s["x"])
        s["dw"] = torch.empty(E, d, device="cuda")
        return s
    t = TYPES[s["type"]]
    if op in ("norm", "norm_grad"):
        s["x"] = normal(T, d, dtype=t)
        s["y"] = normal(T, d, std=0.3, dtype=t) if s["y"] else None
        s["v_out"] = (1 + normal(d, std=0.1)).to(t) if s["norm_out"] else None
        s["v_in"] = (1 + normal(d, std=0.1)).to(t) if s["norm_in"] else None
        shape = {"none": None, "channel": (d,), "token": (T, 1), "full": (T, d)}[s["gate"]]
        s["g"] = None if shape is None else normal(*shape, std=0.5, dtype=t)
        if op == "norm":
            s["h"] = torch.empty(T, d, dtype=t, device="cuda") if s["y"] is not None else None
            s["n"] = torch.empty(T, d, dtype=t, device="cuda") if s["norm_in"] else None
        else:
            s["dh"] = normal(T, d, std=0.1, dtype=t)
            s["dn"] = normal(T, d, std=0.1, dtype=t) if s["norm_in"] else None
            s["dx"] = torch.empty_like(s["x"])
            s["dy"] = None if s["y"] is None else torch.empty_like(s["y"])
            s["dg"] = None if shape is None else torch.empty(shape, dtype=t if s["gate"] == "full" else torch.float32,
                                                             device="cuda")
            s["dv_out"] = torch.empty(d, device="cuda") if s["norm_out"] else None
            s["dv_in"] = torch.empty(d, device="cuda") if s["norm_in"] else None
        return s
    E, k = s["E"], s["k"]
    P = T * k
    _, ids, weights = _routed(s, uniform)
    s["pos"] = _positions(ids, E, s["dropped"], uniform)
    s["weights"] = weights if s["weighted"] else None
    if op in ("permute", "permute_grad"):
        s["x"] = normal(T, d, dtype=t)
    if op == "unpermute_grad":
        s["dout"] = normal(T, d, std=0.1, dtype=t)
    if op in ("unpermute", "unpermute_grad"):
        s["rows"] = normal(P, d, dtype=t)
    if op == "permute_grad":
        s["drows"] = normal(P, d, std=0.1, dtype=t)
    # where the results go; sorted rows that no pair has stay zero
    if op == "permute":
        s["to"] = torch.zeros(P, d, dtype=t, device="cuda")
    elif op == "unpermute_grad":
        s["to"] = torch.zeros(P, d, dtype=t, device="cuda")
    else:
        s["to"] = torch.empty(T, d, dtype=t, device="cuda")
    s["dweights"] = torch.empty(T, k, device="cuda") if s["weighted"] and op in ("permute_grad", "unpermute_grad") else None
    return s


# ---------------------------------------------------------------- plain forms

def _place(vals, pos, P, dtype):
    """vals [T, k, d] to the sorted rows [P, d]; dropped pairs go to a row behind, which is cut off."""
    rows = torch.zeros(P + 1, vals.shape[-1], dtype=dtype, device=vals.device)
    rows.index_copy_(0, torch.where(pos < 0, P, pos).long(), vals.reshape(P, -1).to(dtype))
    return rows[:P]


def _fetch(rows, pos, T, k):
    """The sorted rows of each token, [T, k, d] in float32, zero for dropped pairs."""
    got = rows.float().index_select(0, pos.clamp(min=0).long())
    return torch.where((pos < 0)[:, None], 0.0, got).reshape(T, k, -1)


def _rms(z):
    return torch.rsqrt((z * z).mean(1, keepdim=True) + EPS)


def _plain(s):
    op, T, d = s["op"], s["T"], s["d"]
    if op == "permute":
        k = s["k"]
        x = s["x"].float()[:, None, :].expand(T, k, d)
        vals = x if s["weights"] is None else x * s["weights"][:, :, None]
        return _place(vals, s["pos"], T * k, s["x"].dtype)
    if op == "unpermute":
        got = _fetch(s["rows"], s["pos"], T, s["k"])
        got = got if s["weights"] is None else got * s["weights"][:, :, None]
        return got.sum(1).to(s["rows"].dtype)
    if op == "permute_grad":
        got = _fetch(s["drows"], s["pos"], T, s["k"])
        if s["weights"] is None:
            return {"dx": got.sum(1).to(s["drows"].dtype)}
        return {"dx": (got * s["weights"][:, :, None]).sum(1).to(s["drows"].dtype),
                "dweights": (got * s["x"].float()[:, None, :]).sum(2)}
    if op == "unpermute_grad":
        k = s["k"]
        dout = s["dout"].float()[:, None, :].expand(T, k, d)
        if s["weights"] is None:
            return {"drows": _place(dout, s["pos"], T * k, s["dout"].dtype)}
        return {"drows": _place(dout * s["weights"][:, :, None], s["pos"], T * k, s["dout"].dtype),
                "dweights": (dout * _fetch(s["rows"], s["pos"], T, k)).sum(2)}
    if op == "route_grad":
        ids, w, dw = s["ids"].long(), s["weights"], s["dweights"]
        mean = (w * dw).sum(1, keepdim=True)
        if s["renormalize"]:
            dl = torch.zeros_like(s["logits"]).scatter_(1, ids, w * (dw - mean))
        else:
            dl = torch.softmax(s["logits"], 1) * (torch.zeros_like(s["logits"]).scatter_(1, ids, dw) - mean)
        dl = dl if s["dlogits"] is None else dl + s["dlogits"]
        return {"dx": (dl @ s["w"].float() + s["dx_add"].float()).to(torch.bfloat16), "dw": dl.t() @ s["x"].float()}
    # norm and its gradient
    t = s["x"].dtype
    x = s["x"].float()
    h = s["scale"] * x
    g = None if s["g"] is None else s["g"].float()
    if s["y"] is not None:
        y = s["y"].float()
        yn = y if s["v_out"] is None else y * _rms(y)
        z = yn if s["v_out"] is None else yn * s["v_out"].float()
        h = h + (z if g is None else g * z)
    if op == "norm":
        out = {} if s["y"] is None else {"h": h.to(t)}
        if s["v_in"] is not None:
            out["n"] = (h * _rms(h) * s["v_in"].float()).to(t)
        return out
    out = {}
    dh = s["dh"].float()
    if s["v_in"] is not None:
        r = _rms(h)
        hn, dn = h * r, s["dn"].float()
        out["dv_in"] = (dn * hn).sum(0)
        u = dn * s["v_in"].float()
        dh = dh + r * (u - hn * (u * hn).mean(1, keepdim=True))
    out["dx"] = (s["scale"] * dh).to(t)
    if s["y"] is not None:
        if g is not None:
            dg = dh * z
            out["dg"] = {"channel": dg.sum(0) if s["gate"] == "channel" else None,
                         "token": dg.sum(1, keepdim=True) if s["gate"] == "token" else None,
                         "full": dg.to(t) if s["gate"] == "full" else None}[s["gate"]]
        dz = dh if g is None else dh * g
        if s["v_out"] is None:
            out["dy"] = dz.to(t)
        else:
            out["dv_out"] = (dz * yn).sum(0)
            u = dz * s["v_out"].float()
            out["dy"] = (_rms(y) * (u - yn * (u * yn).mean(1, keepdim=True))).to(t)
    return out


# ---------------------------------------------------------------- the package's calls

def _own(s):
    import w4a16_grouped_expert_amd as moe
    op = s["op"]
    if op == "permute":
        return moe.moe_permute_into(s["x"], s["pos"], s["k"], s["to"], weights=s["weights"])
    if op == "unpermute":
        return moe.moe_unpermute_into(s["rows"], s["pos"], s["k"], s["to"], weights=s["weights"])
    if op == "permute_grad":
        if s["weights"] is None:
            return {"dx": moe.moe_permute_backward_into(s["drows"], s["pos"], s["k"], s["to"])}
        moe.moe_permute_backward_into(s["drows"], s["pos"], s["k"], s["to"], weights=s["weights"], x=s["x"],
                                      dweights=s["dweights"])
        return {"dx": s["to"], "dweights": s["dweights"]}
    if op == "unpermute_grad":
        if s["weights"] is None:
            return {"drows": moe.moe_unpermute_backward_into(s["dout"], s["pos"], s["k"], s["to"])}
        moe.moe_unpermute_backward_into(s["dout"], s["pos"], s["k"], s["to"], weights=s["weights"], rows=s["rows"],
                                        dweights=s["dweights"])
        return {"drows": s["to"], "dweights": s["dweights"]}
    if op == "route_grad":
        if "ws" not in s:
            s["ws"] = moe.alloc_route_backward_workspace(s["T"], s["d"], s["E"], s["k"], s["x"].device)
        route = moe.RouteOut(s["logits"], s["ids"], s["weights"])
        moe.moe_route_backward_into(s["x"], s["w"], route, s["dweights"], s["dx"], s["dw"], s["ws"],
                                    renormalize=s["renormalize"], dlogits=s["dlogits"], dx_add=s["dx_add"])
        return {"dx": s["dx"], "dw": s["dw"]}
    norm = moe.BlockNorm(norm_in=s["v_in"], norm_out=s["v_out"], gate=s["g"], residual_scale=s["scale"], eps=EPS)
    if op == "norm":
        moe.moe_block_norm_into(norm, s["x"], s["y"], h=s["h"], n=s["n"])
        return {q: s[q] for q in ("h", "n") if s[q] is not None}
    if "ws" not in s:
        s["ws"] = moe.alloc_block_norm_workspace(s["T"], s["d"], s["x"].device)
    grads = moe.BlockNormGrads(dx=s["dx"], dy=s["dy"], dgate=s["dg"], dnorm_out=s["dv_out"], dnorm_in=s["dv_in"])
    moe.moe_block_norm_backward_into(norm, s["x"], s["y"], grads, s["ws"], dh=s["dh"], dn=s["dn"])
    return {q: s[q] for q in ("dx", "dy", "dg", "dv_out", "dv_in") if s[q] is not None}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    s = case
    T, d = s["T"], s["d"]
    if s["op"] == "route_grad":
        E, k = s["E"], s["k"]
        logits = 0 if s["renormalize"] else T * E * 4
        aux = T * E * 4 if s["aux"] else 0
        # x, dx_add in and dx out; the weight in, its gradient out; the routing's own values
        return {"bytes": 3 * T * d * 2 + E * d * 6 + logits + aux + T * k * 12, "flops": 4 * T * E * d}
    b = TYPES[s["type"]].itemsize
    if s["op"] in ("norm", "norm_grad"):
        full = T * d * b
        gate = {"none": 0, "channel": d * b, "token": T * b, "full": full}[s["gate"]]
        dgate = {"none": 0, "channel": d * 4, "token": T * 4, "full": full}[s["gate"]]
        vectors = s["norm_out"] + s["norm_in"]
        if s["op"] == "norm":  # x, y in; h, n out
            return {"bytes": full * (1 + 2 * s["y"] + s["norm_in"]) + gate + vectors * d * b, "flops": 12 * T * d}
        # x, y, dh, dn in; dx, dy out
        return {"bytes": full * (3 + 2 * s["y"] + s["norm_in"]) + gate + dgate + vectors * d * (b + 4),
                "flops": 30 * T * d}
    kept = T * s["k"] * (1 - s["dropped"])
    index = T * s["k"] * 4 * (1 + s["weighted"])
    grad = s["op"].endswith("_grad") and s["weighted"]
    if s["op"] == "unpermute_grad":  # dout (and rows) in, drows out
        n = T + kept * (2 if grad else 1)
    else:
        n = T + kept + (T if grad else 0)
    return {"bytes": n * d * b + index + (T * s["k"] * 4 if grad else 0),
            "flops": (4 if grad else 2) * kept * d}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op, T, d = s["op"], s["T"], s["d"]
    if op in ("permute", "unpermute", "permute_grad", "unpermute_grad"):
        k, P = s["k"], s["T"] * s["k"]
        pos = s["pos"].long().reshape(T, k)
        w = torch.ones(T, k, dtype=torch.float64, device="cuda") if s["weights"] is None else s["weights"].double()
        w = torch.where(pos < 0, torch.zeros_like(w), w)
        rows_of = {"unpermute": "rows", "permute_grad": "drows", "unpermute_grad": "rows"}
        to = torch.zeros(T if op in ("unpermute", "permute_grad") else P, d, dtype=torch.float64, device="cuda")
        dweights = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            there = torch.nonzero(pos[:, j] >= 0)[:, 0]
            at = pos[there, j]
            if op in rows_of:
                mine = s[rows_of[op]][at].double()
                other = s["x"] if op == "permute_grad" else s["dout"] if op == "unpermute_grad" else None
                if other is not None:
                    dweights[there, j] = (mine * other[there].double()).sum(1)
            if op in ("unpermute", "permute_grad"):
                to[there] += w[there, j, None] * mine
            else:
                to[at] = w[there, j, None] * (s["x"] if op == "permute" else s["dout"])[there].double()
        if op in ("permute", "unpermute"):
            return to
        name = "dx" if op == "permute_grad" else "drows"
        return {name: to, "dweights": dweights} if s["weighted"] else {name: to}
    if op == "route_grad":
        ids, dw = s["ids"].long(), s["dweights"].double()
        logits = s["logits"].double()
        chosen = torch.zeros_like(logits).scatter(1, ids, 1.0)
        e = torch.exp(logits - logits.max(1, keepdim=True)[0])
        e = e * chosen if s["renormalize"] else e
        # the package's weights are given in float32: the gradient is taken at these
        given = torch.zeros_like(logits).scatter(1, ids, s["weights"].double())
        p = given if s["renormalize"] else e / e.sum(1, keepdim=True)
        back = torch.zeros_like(logits).scatter(1, ids, dw)
        dl = p * (back - (given * back).sum(1, keepdim=True))
        if s["dlogits"] is not None:
            dl = dl + s["dlogits"].double()
        return {"dx": torch.mm(dl, s["w"].double()) + s["dx_add"].double(), "dw": torch.mm(dl.t(), s["x"].double())}
    # norm: the gradient by differentiating the definition
    grad = op == "norm_grad"

    def leaf(v):
        return None if v is None else v.double().requires_grad_(grad)

    x, y, v_out, v_in, g = (leaf(s[q]) for q in ("x", "y", "v_out", "v_in", "g"))
    h = x * s["scale"]
    if y is not None:
        z = y
        if v_out is not None:
            z = v_out * z / torch.sqrt(z.square().sum(1, keepdim=True) / d + EPS)
        h = h + (z * g if g is not None else z)
    n = None if v_in is None else v_in * h / torch.sqrt(h.square().sum(1, keepdim=True) / d + EPS)
    if not grad:
        out = {} if y is None else {"h": h}
        return out if n is None else {**out, "n": n}
    loss = (h * s["dh"].double()).sum() + (0 if n is None else (n * s["dn"].double()).sum())
    loss.backward()
    leaves = dict(dx=x, dy=y, dg=g, dv_out=v_out, dv_in=v_in)
    return {q: v.grad for q, v in leaves.items() if v is not None}
