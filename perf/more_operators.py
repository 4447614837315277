"""The cases that the router and the experts' bf16 products are measured on.

Five operators around the layout, dispatch and combine of this library, in the
order a training step of a mixture-of-experts layer runs them:

  route           the router's choice: scores of the logits (softmax or
                  sigmoid), a bias for balance that counts for the choice
                  only, groups of experts, top-k, weights
  route_backward  the gradient of those weights to the logits
  linear          each expert's rows times its weight in bf16, with bias,
                  activation and residual; without offsets one weight for all
                  rows (the router's own product, a shared expert)
  dgrad           the gradient of such a product to its rows, through the
                  activation that made them
  wgrad           its gradient to the weights, and the bias's

A case is a dict of sizes: T tokens, E experts, top-k, K and N the weights'
sides (N rows of K values for each expert; swiglu: gate rows, then up rows),
`skew` the spread of the router's logits (0.25: a balanced router; larger: some
experts get several times the mean), `drop` the share of (token, slot) entries
that no expert takes, as a capacity limit leaves them.  E = 0 is one weight for
all T rows.

`own` selects what run() does: the library's calls, or the same mathematics in
plain torch operations in 32 bits (in 64 where scores are compared).
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step of a served batch: latency
        {"name": "route_decode", "op": "route", "T": 128, "E": 256, "k": 8, "type": "f32", "score": "sigmoid",
         "bias": True, "groups": 8, "top_groups": 4, "best": 2, "renorm": True, "scale": 2.5},
        # a prefill batch on a plain softmax router whose logits come out of a bf16 product (equal logits are common)
        {"name": "route_prefill_bf16", "op": "route", "T": 16384, "E": 64, "k": 6, "type": "bf16", "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "best": 1, "renorm": False, "scale": 1.0},
        # a large batch on a balanced sigmoid router with groups: the most work a token can be
        {"name": "route_groups", "op": "route", "T": 16384, "E": 256, "k": 8, "type": "f32", "score": "sigmoid",
         "bias": True, "groups": 8, "top_groups": 4, "best": 2, "renorm": True, "scale": 2.5},
        # a training micro-batch, gradient in bf16 for the products that follow
        {"name": "route_bwd_train", "op": "route_backward", "T": 4096, "E": 256, "k": 8, "type": "f32",
         "out": "bf16", "score": "sigmoid", "renorm": True, "scale": 2.5},
        # softmax over all experts: every logit has a gradient; odd sizes
        {"name": "route_bwd_odd", "op": "route_backward", "T": 8191, "E": 60, "k": 5, "type": "f32", "out": "f32",
         "score": "softmax", "renorm": False, "scale": 1.0},
        # the router's own product for a decode batch: few rows, few outputs, a long sum
        {"name": "linear_router", "op": "linear", "T": 128, "E": 0, "k": 1, "K": 7168, "N": 256, "act": "none",
         "bias": False, "res": False, "pre": False, "out": "f32", "skew": 0.0, "drop": 0.0},
        # one decode step of a served batch, down product: weight reading
        {"name": "linear_decode", "op": "linear", "T": 128, "E": 256, "k": 8, "K": 2048, "N": 7168, "act": "none",
         "bias": True, "res": False, "pre": False, "out": "bf16", "skew": 0.5, "drop": 0.0},
        # gate and up product of a training batch, the values before the activation kept for the way back
        {"name": "linear_train", "op": "linear", "T": 8192, "E": 64, "k": 6, "K": 7168, "N": 4096, "act": "swiglu",
         "bias": False, "res": False, "pre": True, "out": "bf16", "skew": 0.25, "drop": 0.0},
        # sizes that no tile divides, dropped entries, an activation with one input
        {"name": "dgrad_odd", "op": "dgrad", "T": 1500, "E": 37, "k": 3, "K": 1000, "N": 1496, "act": "gelu",
         "skew": 0.5, "drop": 0.1},
        # the way back through down product and SwiGLU of the training batch
        {"name": "dgrad_train", "op": "dgrad", "T": 8192, "E": 64, "k": 6, "K": 2048, "N": 7168, "act": "swiglu",
         "skew": 0.25, "drop": 0.0},
        # the router's weight gradient of a training batch: few outputs, a sum over all tokens
        {"name": "wgrad_router", "op": "wgrad", "T": 4096, "E": 0, "k": 1, "K": 7168, "N": 256, "out": "f32",
         "bias": True, "skew": 0.0, "drop": 0.0},
        # the down product's weight gradient of the training batch
        {"name": "wgrad_train", "op": "wgrad", "T": 8192, "E": 64, "k": 6, "K": 2048, "N": 7168, "out": "bf16",
         "bias": True, "skew": 0.25, "drop": 0.0},
    ]


def _log(rng, lo, hi, step=1):
    v = int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))
    return max(lo, min(hi, v // step * step))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50.0)


def draw(rng):
    op = rng.choice(["route", "route_backward", "linear", "dgrad", "wgrad"])
    largest = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        c = {"op": op, "T": _log(rng, 1, 16384)}
        if op in ("route", "route_backward"):
            c["type"], c["score"] = rng.choice(["f32", "f32", "bf16"]), rng.choice(["softmax", "sigmoid"])
            c["renorm"], c["scale"] = rng.random() < 0.6, rng.choice([1.0, 2.5])
            if op == "route":
                c["groups"] = rng.choice([1, 1, 2, 4, 7, 8])
                per = _log(rng, 4, 512 // c["groups"])
                c["E"] = c["groups"] * per
                c["top_groups"] = rng.randint(1, c["groups"])
                c["best"] = rng.choice([1, 2]) if c["groups"] > 1 else 1
                c["k"] = rng.randint(1, min(16, per * c["top_groups"]))
                c["bias"] = rng.random() < 0.5
            else:
                c["E"] = _log(rng, 4, 512)
                c["k"] = rng.randint(2 if c["renorm"] else 1, min(16, c["E"]))  # (one renormalised weight has no gradient)
                c["out"] = rng.choice(["f32", "bf16"])
        else:
            c["E"] = 0 if rng.random() < 0.25 else _log(rng, 4, 256)
            c["k"] = rng.randint(1, min(8, c["E"])) if c["E"] else 1
            c["K"], c["N"] = _log(rng, 64, 8192, 8), _log(rng, 64, 8192, 8)
            c["skew"] = rng.choice([0.0, 0.25, 0.5])
            c["drop"] = rng.choice([0.0, 0.0, 0.1]) if c["E"] else 0.0
            if op != "wgrad":
                c["act"] = rng.choice(["none", "silu", "gelu", "swiglu"])
            if op == "linear":
                c["N"] = c["N"] // 16 * 16
                c["bias"], c["res"], c["pre"] = rng.random() < 0.5, rng.random() < 0.3, c["act"] != "none" and rng.random() < 0.5
            if op != "dgrad":
                c["out"] = rng.choice(["bf16", "bf16", "f32"])
            if op == "wgrad":
                c["bias"] = rng.random() < 0.5
            if max(1, c["E"]) * c["N"] * c["K"] > 2e9 or c["T"] * c["k"] * max(c["N"], 2 * c["K"]) > 8e8:
                continue
        if _cost(c) <= largest:
            return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _logits(T, E, g):
    """Router logits: a spread of 1.5, some experts favoured."""
    return torch.randn(T, E, generator=g, device=DEV) * 1.5 + torch.randn(E, generator=g, device=DEV) * 0.3


def _routing(case, g):
    """The layout of the entries by expert (what ep_layout returns as offsets)
    of a router's choices, by plain counting; for one weight, all rows."""
    T, E, k = case["T"], case["E"], case["k"]
    if not E:
        return None, torch.tensor([T], device=DEV), T
    favour = torch.randn(E, generator=g, device=DEV) * case["skew"]
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device=DEV, dtype=torch.float64)))
    ids = torch.topk(favour.double() + noise, k, dim=1).indices
    ids[torch.rand(T, k, generator=g, device=DEV) < case["drop"]] = E
    counts = torch.bincount(ids.reshape(-1), minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(counts, 0).to(torch.int32)
    return offsets, counts, int(counts.sum())


def _rows(rows, n, g):
    """Hidden rows: unit scale, a spread between tokens, a few loud channels."""
    x = torch.randn(rows, n, generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device=DEV))
    x[:, torch.randint(0, n, (max(1, n // 512),), generator=g, device=DEV)] *= 12.0
    return x.to(torch.bfloat16)


def _weights(E, N, K, g):
    w = torch.empty(E, N, K, dtype=torch.bfloat16, device=DEV)
    step = max(1, (1 << 28) // (N * K))
    for e in range(0, E, step):
        n = min(step, E - e)
        w[e : e + n] = torch.randn(n, N, K, generator=g, device=DEV) * (1.0 / math.sqrt(K))
    return w


def _width(case):
    """Values of a row on the activation's input side: linear's product, dgrad's result."""
    return case["K"] * (2 if case["act"] == "swiglu" else 1)


def prepare(case, seed):
    g = _gen(seed)
    op, T, E, k = case["op"], case["T"], case["E"], case["k"]
    st = dict(case)
    if op in ("route", "route_backward"):
        st["logits"] = _logits(T, E, g).to(TYPES[case["type"]])
        st["idx"] = torch.zeros(T, k, dtype=torch.int32, device=DEV)
        st["w"] = torch.zeros(T, k, device=DEV)
        if op == "route":
            # steps of a thousandth up or down, as balancing updates leave them
            st["b"] = torch.randint(-30, 31, (E,), generator=g, device=DEV) * 0.001 if case["bias"] else None
        else:
            st["idx"].copy_(torch.sort(st["logits"].float(), dim=1, descending=True, stable=True).indices[:, :k])
            st["dw"] = torch.randn(T, k, generator=g, device=DEV)
            st["dl"] = torch.zeros(T, E, dtype=TYPES[case["out"]], device=DEV)
        return st
    offsets, counts, total = _routing(case, g)
    rows, K, N, held = T * k, case["K"], case["N"], counts.numel()
    st.update(offsets=offsets, total=total)
    if op == "linear":
        outs = N // 2 if case["act"] == "swiglu" else N
        st["a"], st["b"] = _rows(rows, K, g), _weights(held, N, K, g)
        st["bv"] = torch.randn(held, N, generator=g, device=DEV) * 0.1 if case["bias"] else None
        st["r"] = torch.randn(rows, outs, generator=g, device=DEV).to(torch.bfloat16) if case["res"] else None
        st["z"] = torch.zeros(rows, N, dtype=torch.bfloat16, device=DEV) if case["pre"] else None
        st["y"] = torch.zeros(rows, outs, dtype=TYPES[case["out"]], device=DEV)
    elif op == "dgrad":
        st["dy"], st["b"] = _rows(rows, N, g), _weights(held, N, K, g)
        wide = _width(case)
        st["z"] = _rows(rows, wide, g) if case["act"] != "none" else None
        st["dx"] = torch.zeros(rows, wide, dtype=torch.bfloat16, device=DEV)
    else:
        st["a"], st["dy"] = _rows(rows, K, g), _rows(rows, N, g)
        st["db"] = torch.zeros(held, N, K, dtype=TYPES[case["out"]], device=DEV)
        st["dbv"] = torch.zeros(held, N, device=DEV) if case["bias"] else None
    # the experts that hold rows, and where each row goes in a padded batch of them (the plain form's plan)
    off = torch.zeros(held + 1, dtype=torch.long, device=DEV)
    off[1:] = torch.cumsum(counts, 0)
    active = torch.nonzero(counts > 0).reshape(-1)
    most = int(counts.max())
    slot = off[active].unsqueeze(1) + torch.arange(most, device=DEV).unsqueeze(0)
    row = torch.arange(total, device=DEV)
    nth = torch.searchsorted(off[active + 1].contiguous(), row, right=True)
    st.update(active=active, most=most, slot_row=torch.minimum(slot, (off[active + 1] - 1).unsqueeze(1)).reshape(-1),
              slot_held=(slot < off[active + 1].unsqueeze(1)).reshape(-1, 1),
              row_slot=nth * most + row - off[active][nth] if total else row, row_expert=active[nth] if total else row)
    return st


# ------------------------------------------------------------------ the plain forms
def _score(kind, l):
    if kind == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _first(v, k):
    """The k largest of each row, ties to the lowest index."""
    return torch.sort(v, dim=1, descending=True, stable=True).indices[:, :k]


def _plain_route(s):
    T, E = s["logits"].shape
    l = s["logits"].float()
    score = _score(s["score"], l)
    choice = _score(s["score"], l.double())
    if s["b"] is not None:
        choice = choice + s["b"].double()
    order = choice if s["b"] is not None else l
    if s["groups"] > 1:
        per = E // s["groups"]
        of_group = torch.sort(choice.view(T, s["groups"], per), dim=2, descending=True).values[:, :, : s["best"]].sum(2)
        kept = torch.zeros(T, s["groups"], dtype=torch.bool, device=l.device)
        kept.scatter_(1, _first(of_group, s["top_groups"]), True)
        order = torch.where(kept.repeat_interleave(per, 1), order, -math.inf)
    idx = _first(order, s["k"])
    w = torch.gather(score, 1, idx)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    s["idx"].copy_(idx)
    s["w"].copy_(w * s["scale"])
    return {"idx": s["idx"], "w": s["w"]}


def _plain_route_backward(s):
    l, idx = s["logits"].float(), s["idx"].long()
    score = _score(s["score"], l)
    chosen = torch.gather(score, 1, idx)
    ds = s["dw"] * s["scale"]
    if s["renorm"]:
        total = chosen.sum(1, keepdim=True)
        ds = (ds - (ds * chosen).sum(1, keepdim=True) / total) / total
    if s["score"] == "sigmoid":
        dl = torch.zeros_like(l).scatter_(1, idx, ds * chosen * (1.0 - chosen))
    else:
        full = torch.zeros_like(l).scatter_(1, idx, ds)
        dl = score * (full - (ds * chosen).sum(1, keepdim=True))
    s["dl"].copy_(dl)
    return {"dlogits": s["dl"]}


def _batched(s, x):
    """The rows of x in a padded batch of the experts that hold any, in 32 bits; padding holds zeros."""
    x = torch.where(s["slot_held"], x[s["slot_row"]].float(), 0.0)
    return x.view(s["active"].numel(), s["most"], x.shape[1])


def _unbatched(s, y):
    return y.reshape(-1, y.shape[2])[s["row_slot"]]


def _activate(act, z):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "swiglu":
        gate, up = z.chunk(2, dim=1)
        return gate / (1.0 + torch.exp(-gate)) * up
    return z


def _activate_back(act, z, d):
    """The gradient at z of _activate(act, z) under d."""
    if act == "none":
        return d
    if act == "gelu":
        return d * (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi))
    gate, up = z.chunk(2, dim=1) if act == "swiglu" else (z, None)
    sig = 1.0 / (1.0 + torch.exp(-gate))
    slope = sig * (1.0 + gate * (1.0 - sig))
    return torch.cat([d * up * slope, d * gate * sig], 1) if act == "swiglu" else d * slope


def _plain_linear(s):
    n = s["total"]
    w = s["b"][s["active"]].float()
    z = _unbatched(s, torch.bmm(_batched(s, s["a"]), w.transpose(1, 2)))
    if s["bv"] is not None:
        z = z + s["bv"][s["row_expert"]]
    y = _activate(s["act"], z)
    if s["r"] is not None:
        y = y + s["r"][:n].float()
    s["y"][:n] = y.to(s["y"].dtype)
    if s["z"] is None:
        return {"y": s["y"]}
    s["z"][:n] = z.to(torch.bfloat16)
    return {"y": s["y"], "pre": s["z"]}


def _plain_dgrad(s):
    n = s["total"]
    d = _unbatched(s, torch.bmm(_batched(s, s["dy"]), s["b"][s["active"]].float()))
    s["dx"][:n] = _activate_back(s["act"], s["z"][:n].float() if s["z"] is not None else None, d).to(torch.bfloat16)
    return {"dx": s["dx"]}


def _plain_wgrad(s):
    dy = _batched(s, s["dy"])
    s["db"].zero_()
    s["db"][s["active"]] = torch.bmm(dy.transpose(1, 2), _batched(s, s["a"])).to(s["db"].dtype)
    if s["dbv"] is None:
        return {"db": s["db"]}
    s["dbv"].zero_()
    s["dbv"][s["active"]] = dy.sum(1)
    return {"db": s["db"], "dbias": s["dbv"]}


_PLAIN = {"route": _plain_route, "route_backward": _plain_route_backward, "linear": _plain_linear,
          "dgrad": _plain_dgrad, "wgrad": _plain_wgrad}


# ------------------------------------------------------------------ the library's calls
def _own(s):
    import bulk_async_tensor_amd as ep

    op = s["op"]
    if op == "route":
        ep.ep_route(s["logits"], s["idx"], s["w"], score=s["score"], bias=s["b"], groups=s["groups"],
                    top_groups=s["top_groups"], group_best=s["best"], renormalize=s["renorm"], scale=s["scale"])
        return {"idx": s["idx"], "w": s["w"]}
    if op == "route_backward":
        return {"dlogits": ep.ep_route_backward(s["logits"], s["idx"], s["dw"], s["dl"], score=s["score"],
                                                renormalize=s["renorm"], scale=s["scale"])}
    if op == "linear":
        ep.ep_grouped_linear(s["a"], s["offsets"], s["b"], s["y"], bias=s["bv"], act=s["act"], residual=s["r"],
                             pre=s["z"])
        return {"y": s["y"]} if s["z"] is None else {"y": s["y"], "pre": s["z"]}
    if op == "dgrad":
        return {"dx": ep.ep_grouped_linear_dgrad(s["dy"], s["offsets"], s["b"], s["dx"], act=s["act"], pre=s["z"])}
    ep.ep_grouped_linear_wgrad(s["dy"], s["a"], s["offsets"], s["db"], dbias=s["dbv"])
    return {"db": s["db"]} if s["dbv"] is None else {"db": s["db"], "dbias": s["dbv"]}


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, T, E, k = case["op"], case["T"], case["E"], case["k"]
    size = {"bf16": 2.0, "f32": 4.0}
    if op == "route":
        # logits in, ids and weights out; a score of each logit and k comparisons of it
        return {"bytes": T * E * size[case["type"]] + 8.0 * T * k + (4.0 * E if case["bias"] else 0.0),
                "flops": T * E * (4.0 + k)}
    if op == "route_backward":
        return {"bytes": T * E * (size[case["type"]] + size[case["out"]]) + 8.0 * T * k, "flops": 4.0 * T * E}
    rows = T * k * (1.0 - case["drop"])
    held = E * (1.0 - (1.0 - k * (1.0 - case["drop"]) / E) ** T) if E else 1  # experts that hold a row
    K, N = case["K"], case["N"]
    flops = 2.0 * rows * N * K
    if op == "linear":
        outs = N // 2 if case["act"] == "swiglu" else N
        row = 2.0 * K + outs * (size[case["out"]] + (2.0 if case["res"] else 0.0)) + (2.0 * N if case["pre"] else 0.0)
        return {"bytes": rows * row + held * N * (2.0 * K + (4.0 if case["bias"] else 0.0)) + 4.0 * (E + 1), "flops": flops}
    if op == "dgrad":
        wide = _width(case)
        return {"bytes": rows * (2.0 * N + 2.0 * wide * (1 if case["act"] == "none" else 2)) + 2.0 * held * N * K,
                "flops": flops}
    return {"bytes": 2.0 * rows * (N + K) + max(1, E) * N * (K * size[case["out"]] + (4.0 if case["bias"] else 0.0)),
            "flops": flops}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return {"idx": None, "w": _exact_route(s)}
    if op == "route_backward":
        return {"dlogits": _exact_route_backward(s)}
    off = [0, case["T"]] if s["offsets"] is None else s["offsets"].tolist()
    spans = [(e, slice(off[e], off[e + 1])) for e in range(len(off) - 1) if off[e + 1] > off[e]]
    if op == "linear":
        out = {"y": s["y"].double()}
        if s["z"] is not None:
            out["pre"] = s["z"].double()
        for e, rows in spans:
            z = s["a"][rows].double() @ s["b"][e].double().t()
            if s["bv"] is not None:
                z += s["bv"][e].double()
            if s["z"] is not None:
                out["pre"][rows] = z
            y = _exact_act(case["act"], z)
            out["y"][rows] = y if s["r"] is None else y + s["r"][rows].double()
        return out
    if op == "dgrad":
        dx = s["dx"].double()
        for e, rows in spans:
            d = s["dy"][rows].double() @ s["b"][e].double()
            if s["z"] is None:
                dx[rows] = d
            else:
                # the derivative as torch's own differentiation gives it
                z = s["z"][rows].double().requires_grad_()
                dx[rows] = torch.autograd.grad(_exact_act(case["act"], z), z, d)[0]
        return {"dx": dx}
    out = {"db": s["db"].double()}
    if s["dbv"] is not None:
        out["dbias"] = s["dbv"].double()
    for e, rows in spans:
        dy = s["dy"][rows].double()
        out["db"][e] = dy.t() @ s["a"][rows].double()
        if s["dbv"] is not None:
            out["dbias"][e] = dy.sum(0)
    return out


def _exact_act(act, z):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    if act == "swiglu":
        half = z.shape[1] // 2
        return z[:, :half] * torch.sigmoid(z[:, :half]) * z[:, half:]
    return z


def _exact_route(s):
    """The weights, by one choice after another: the best that is left, the lowest of equals."""
    l = s["logits"].double()
    T, E = l.shape
    score = torch.sigmoid(l) if s["score"] == "sigmoid" else torch.softmax(l, 1)
    c = score if s["b"] is None else score + s["b"].double()
    left = l.clone() if s["b"] is None else c.clone()
    per = E // s["groups"]
    if s["groups"] > 1:
        rank = torch.stack([torch.topk(c[:, i * per : (i + 1) * per], s["best"], dim=1).values.sum(1)
                            for i in range(s["groups"])], 1)
        closed = torch.ones(T, s["groups"], dtype=torch.bool, device=l.device)
        for _ in range(s["top_groups"]):
            best = _lowest_best(rank)
            rank.scatter_(1, best, -math.inf)
            closed.scatter_(1, best, False)
        for i in range(s["groups"]):
            left[:, i * per : (i + 1) * per].masked_fill_(closed[:, i : i + 1], -math.inf)
    w = torch.empty(T, s["k"], dtype=torch.float64, device=l.device)
    for j in range(s["k"]):
        best = _lowest_best(left)
        w[:, j : j + 1] = torch.gather(score, 1, best)
        left.scatter_(1, best, -math.inf)
    if s["renorm"]:
        w /= w.sum(1, keepdim=True)
    return w * s["scale"]


def _lowest_best(v):
    at = torch.arange(v.shape[1], device=v.device).expand_as(v)
    return torch.where(v == v.amax(1, keepdim=True), at, v.shape[1]).amin(1, keepdim=True)


def _exact_route_backward(s):
    """By torch's own differentiation of the weights."""
    l = s["logits"].double().requires_grad_()
    score = torch.sigmoid(l) if s["score"] == "sigmoid" else torch.softmax(l, 1)
    w = torch.gather(score, 1, s["idx"].long())
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return torch.autograd.grad((w * s["scale"] * s["dw"].double()).sum(), l)[0].detach()
