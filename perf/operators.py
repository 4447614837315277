"""The cases that the expert-side operators are measured on.

Five operators next to the layout, dispatch and combine of this library, in
the order a mixture-of-experts layer runs them:

  dispatch_fp8      rows go to their experts in 8 bits: one e4m3 row and one
                    float32 scale for each block of 128 values
  swiglu            the experts' gate and up products on those rows, 8 bits
                    with block scales on both sides, SiLU(gate) * up and the
                    quantisation of the result for the next product
  gemm              the experts' product in 8 bits with block scales, bf16 out
  combine_backward  the gradient of ep_combine to the expert rows and weights
  dispatch_backward the gradient of ep_dispatch to the token rows

A case is a dict of sizes: T tokens, H (or K) row elements, E experts, top-k,
`skew` the spread of the router's logits (0.25: a balanced router; larger:
some experts get several times the mean), `drop` the share of (token, slot)
entries that no expert takes (id -1, as a capacity limit leaves them).

`own` selects what run() does: the library's calls, or the same mathematics in
plain torch operations in 32 bits.
"""

import math

import torch

own = False

BLOCK = 128          # values that share a scale
E4M3_MAX = 448.0     # largest finite e4m3 value
AMAX_FLOOR = 2.0 ** -100  # block maxima below this are taken as this: scales stay normal numbers
DEV = "cuda"


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the gradient step of a small layer: launch latency
        {"name": "combine_bwd_tiny", "op": "combine_backward", "T": 128, "H": 1024, "E": 8, "k": 2, "skew": 0.25,
         "drop": 0.0},
        # a training micro-batch
        {"name": "combine_bwd_train", "op": "combine_backward", "T": 4096, "H": 7168, "E": 256, "k": 8,
         "skew": 0.25, "drop": 0.0},
        # odd row length and k, and a capacity limit that dropped entries
        {"name": "dispatch_bwd_odd", "op": "dispatch_backward", "T": 777, "H": 1144, "E": 41, "k": 5, "skew": 0.5,
         "drop": 0.1},
        # the same training micro-batch on the way back through dispatch
        {"name": "dispatch_bwd_train", "op": "dispatch_backward", "T": 4096, "H": 7168, "E": 256, "k": 8,
         "skew": 0.25, "drop": 0.0},
        # one decode step of a served batch: latency
        {"name": "dispatch_fp8_decode", "op": "dispatch_fp8", "T": 128, "H": 7168, "E": 256, "k": 8, "skew": 0.5,
         "drop": 0.0},
        # a prefill batch
        {"name": "dispatch_fp8_prefill", "op": "dispatch_fp8", "T": 16384, "H": 7168, "E": 64, "k": 6, "skew": 0.25,
         "drop": 0.0},
        # a single token: k experts, one row each; weight reading
        {"name": "swiglu_one_token", "op": "swiglu", "T": 1, "K": 7168, "I": 2048, "E": 64, "k": 8, "skew": 0.5,
         "drop": 0.0},
        # many experts with about 128 rows each: weight reading and products are close
        {"name": "swiglu_train", "op": "swiglu", "T": 4096, "K": 7168, "I": 2048, "E": 256, "k": 8, "skew": 0.25,
         "drop": 0.0},
        # a prefill batch: products
        {"name": "swiglu_prefill", "op": "swiglu", "T": 16384, "K": 7168, "I": 2048, "E": 64, "k": 6, "skew": 0.25,
         "drop": 0.0},
        # one decode step of a served batch, down projection: weight reading
        {"name": "gemm_decode", "op": "gemm", "T": 128, "K": 2048, "N": 7168, "E": 256, "k": 8, "skew": 0.5,
         "drop": 0.0},
        # sizes that no tile divides, a last block of 80 values, dropped entries
        {"name": "gemm_odd", "op": "gemm", "T": 1500, "K": 1488, "N": 1000, "E": 37, "k": 3, "skew": 0.5,
         "drop": 0.1},
        # a prefill batch, down projection: products
        {"name": "gemm_prefill", "op": "gemm", "T": 16384, "K": 2048, "N": 7168, "E": 64, "k": 6, "skew": 0.25,
         "drop": 0.0},
    ]


def _log(rng, lo, hi, step=1):
    v = int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))
    return max(lo, min(hi, v // step * step))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50.0)


def draw(rng):
    op = rng.choice(["combine_backward", "dispatch_backward", "dispatch_fp8", "swiglu", "gemm"])
    largest = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        E = _log(rng, 4, 256)
        c = {"op": op, "T": _log(rng, 1, 16384), "E": E, "k": rng.randint(1, min(8, E)),
             "skew": rng.choice([0.0, 0.25, 0.5]), "drop": rng.choice([0.0, 0.0, 0.1])}
        if op in ("combine_backward", "dispatch_backward"):
            c["H"] = _log(rng, 256, 8192, 8)
        elif op == "dispatch_fp8":
            c["H"] = _log(rng, 256, 8192, 16)
        elif op == "swiglu":
            c["K"], c["I"] = _log(rng, 256, 8192, 16), _log(rng, 128, 4096, 64)
        else:
            c["K"], c["N"] = _log(rng, 256, 8192, 16), _log(rng, 256, 8192, 8)
        w = c.get("N", 2 * c.get("I", 0)) * c.get("K", 0)
        if _cost(c) <= largest and E * w <= 8e9 and c["T"] * c["k"] * max(c.get("N", 0), c.get("K", 0)) <= 8e8:
            return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _blocks(n):
    return -(-n // BLOCK)


def _routing(case, g):
    """Expert ids as a router picks them, the gate weights, and the layout of
    the entries by expert (what ep_layout returns), by plain sorting."""
    T, E, k = case["T"], case["E"], case["k"]
    favour = torch.randn(E, generator=g, device=DEV) * case["skew"]
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device=DEV, dtype=torch.float64)))
    logits, ids = torch.topk(favour.double() + noise, k, dim=1)
    w = torch.softmax(torch.randn(T, k, generator=g, device=DEV), dim=1)
    ids = ids.to(torch.int32)
    ids[torch.rand(T, k, generator=g, device=DEV) < case["drop"]] = -1
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, E, flat)
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=E + 1)[:E]
    total = int(counts.sum())
    dest = torch.full((T * k,), -1, dtype=torch.int32, device=DEV)
    dest[order[:total]] = torch.arange(total, dtype=torch.int32, device=DEV)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(counts, 0).to(torch.int32)
    entry = torch.nonzero(dest >= 0).reshape(-1)  # the entries that an expert took, and the row of each
    return {"dest_row": dest.view(T, k), "topk_w": w, "offsets": offsets, "counts": counts, "total": total,
            "entry": entry, "entry_row": dest[entry].long()}


def _activations(rows, n, g):
    """Hidden rows: unit scale, a spread between tokens, a few loud channels."""
    x = torch.randn(rows, n, generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device=DEV))
    x[:, torch.randint(0, n, (max(1, n // 512),), generator=g, device=DEV)] *= 12.0
    return x.to(torch.bfloat16)


def _quantise(x):
    """Rows in 8 bits with a scale for each block of 128, as a program holds
    them that got them from an earlier step."""
    rows, n = x.shape
    nb = _blocks(n)
    p = torch.nn.functional.pad(x.float(), (0, nb * BLOCK - n)).view(rows, nb, BLOCK)
    s = p.abs().amax(2).clamp_min(AMAX_FLOOR) / E4M3_MAX
    q = (p / s.unsqueeze(2)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(rows, nb * BLOCK)[:, :n]
    return q.contiguous(), s


def _expert_weights(E, N, K, g):
    """Weights of E experts in 8 bits with a scale for each 128 x 128 block, as
    a checkpoint holds them."""
    q = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device=DEV)
    step = max(1, (1 << 28) // (N * K))
    for e in range(0, E, step):
        n = min(step, E - e)
        q[e : e + n] = (torch.randn(n, N, K, generator=g, device=DEV) * 100.0).clamp_(-E4M3_MAX, E4M3_MAX).to(q.dtype)
    s = torch.exp(0.25 * torch.randn(E, _blocks(N), _blocks(K), generator=g, device=DEV)) / (100.0 * math.sqrt(K))
    return q, s


def prepare(case, seed):
    g = _gen(seed)
    r = _routing(case, g)
    op, rows = case["op"], case["T"] * case["k"]
    st = {"op": op, **r}
    if op == "combine_backward":
        T, H = case["T"], case["H"]
        st["dout"] = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
        st["y"] = _activations(rows, H, g)
        st["dy"] = torch.zeros(rows, H, dtype=torch.bfloat16, device=DEV)
        st["dw"] = torch.zeros(T, case["k"], device=DEV)
    elif op == "dispatch_backward":
        st["drecv"] = torch.randn(rows, case["H"], generator=g, device=DEV).to(torch.bfloat16)
        st["dx"] = torch.zeros(case["T"], case["H"], dtype=torch.bfloat16, device=DEV)
    elif op == "dispatch_fp8":
        H = case["H"]
        st["x"] = _activations(case["T"], H, g)
        st["recv_q"] = torch.zeros(rows, H, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
        st["recv_scale"] = torch.zeros(rows, _blocks(H), device=DEV)
    else:
        K = case["K"]
        N = 2 * case["I"] if op == "swiglu" else case["N"]
        st["a"], st["a_scale"] = _quantise(_activations(rows, K, g))
        st["b"], st["b_scale"] = _expert_weights(case["E"], N, K, g)
        # the experts that hold rows, and where each row goes in a padded batch of them (the plain form's plan)
        active = torch.nonzero(r["counts"] > 0).reshape(-1)
        most = int(r["counts"].max())
        off = r["offsets"].long()
        slot = off[active].unsqueeze(1) + torch.arange(most, device=DEV).unsqueeze(0)
        st["active"] = active
        st["slot_row"] = torch.minimum(slot, (off[active + 1] - 1).unsqueeze(1)).reshape(-1)
        st["most"] = most
        row = torch.arange(r["total"], device=DEV)
        nth = torch.searchsorted(off[active + 1].contiguous(), row, right=True)
        st["row_slot"] = nth * most + row - off[active][nth] if r["total"] else row
        if op == "swiglu":
            st["out_q"] = torch.zeros(rows, case["I"], dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
            st["out_scale"] = torch.zeros(rows, _blocks(case["I"]), device=DEV)
        else:
            st["out"] = torch.zeros(rows, N, dtype=torch.bfloat16, device=DEV)
    return st


# ------------------------------------------------------------------ the plain forms
def _plain_combine_backward(s):
    k = s["dest_row"].shape[1]
    g = s["dout"].float()[s["entry"] // k]
    s["dw"].zero_()
    s["dw"].view(-1)[s["entry"]] = (s["y"][s["entry_row"]].float() * g).sum(1)
    s["dy"][s["entry_row"]] = g.mul_(s["topk_w"].view(-1)[s["entry"]].unsqueeze(1)).to(torch.bfloat16)
    return {"dy": s["dy"], "dw": s["dw"]}


def _plain_dispatch_backward(s):
    ok = s["dest_row"] >= 0
    rows = s["drecv"][s["dest_row"].long().clamp_min(0)].float()
    s["dx"].copy_(torch.where(ok.unsqueeze(2), rows, 0.0).sum(1))
    return {"dx": s["dx"]}


def _plain_quantise(v):
    rows, n = v.shape
    nb = _blocks(n)
    p = torch.nn.functional.pad(v, (0, nb * BLOCK - n)).view(rows, nb, BLOCK)
    amax = p.abs().amax(2).clamp_min(AMAX_FLOOR)
    q = (p * (E4M3_MAX / amax).unsqueeze(2)).to(torch.float8_e4m3fn).view(rows, nb * BLOCK)[:, :n]
    return q, amax / E4M3_MAX


def _plain_dispatch_fp8(s):
    q, scale = _plain_quantise(s["x"].float())
    k = s["dest_row"].shape[1]
    token = s["entry"] // k
    s["recv_q"].view(torch.uint8)[s["entry_row"]] = q.contiguous().view(torch.uint8)[token]
    s["recv_scale"][s["entry_row"]] = scale[token]
    return {"q": s["recv_q"], "scale": s["recv_scale"]}


def _plain_product(s):
    """a @ b[expert]^T of the rows that experts hold, in 32 bits: the active
    experts' weights and their rows, padded to the longest expert, as one
    batched product."""
    K, N = s["a"].shape[1], s["b"].shape[1]
    w = s["b"].view(torch.uint8)[s["active"]].view(torch.float8_e4m3fn).float()
    ws = s["b_scale"][s["active"]]
    w.mul_(ws.repeat_interleave(BLOCK, 1)[:, :N].repeat_interleave(BLOCK, 2)[:, :, :K])
    a = s["a"].float().mul_(s["a_scale"].repeat_interleave(BLOCK, 1)[:, :K])
    a = a[s["slot_row"]].view(w.shape[0], s["most"], K)
    return torch.bmm(a, w.transpose(1, 2)).view(w.shape[0] * s["most"], N)[s["row_slot"]]


def _plain_gemm(s):
    s["out"][: s["total"]] = _plain_product(s).to(torch.bfloat16)
    return {"y": s["out"]}


def _plain_swiglu(s):
    gate, up = _plain_product(s).chunk(2, dim=1)
    q, scale = _plain_quantise(gate / (1.0 + torch.exp(-gate)) * up)
    s["out_q"][: s["total"]] = q
    s["out_scale"][: s["total"]] = scale
    return {"q": s["out_q"], "scale": s["out_scale"]}


_PLAIN = {"combine_backward": _plain_combine_backward, "dispatch_backward": _plain_dispatch_backward,
          "dispatch_fp8": _plain_dispatch_fp8, "swiglu": _plain_swiglu, "gemm": _plain_gemm}


# ------------------------------------------------------------------ the library's calls
def _own(s):
    import bulk_async_tensor_amd as ep

    op = s["op"]
    if op == "combine_backward":
        ep.ep_combine_backward(s["dout"], s["y"], s["dest_row"], s["topk_w"], s["dy"], s["dw"])
        return {"dy": s["dy"], "dw": s["dw"]}
    if op == "dispatch_backward":
        return {"dx": ep.ep_dispatch_backward(s["drecv"], s["dest_row"], s["dx"])}
    if op == "dispatch_fp8":
        ep.ep_dispatch_fp8(s["x"], s["dest_row"], s["recv_q"], s["recv_scale"])
        return {"q": s["recv_q"], "scale": s["recv_scale"]}
    if op == "swiglu":
        ep.ep_grouped_swiglu_fp8(s["a"], s["a_scale"], s["offsets"], s["b"], s["b_scale"], s["out_q"], s["out_scale"])
        return {"q": s["out_q"], "scale": s["out_scale"]}
    return {"y": ep.ep_grouped_gemm_fp8(s["a"], s["a_scale"], s["offsets"], s["b"], s["b_scale"], s["out"])}


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    T, E, k = case["T"], case["E"], case["k"]
    rows = T * k * (1.0 - case["drop"])
    route = 4.0 * T * k
    op = case["op"]
    if op == "combine_backward":
        H = case["H"]
        # dout, y and the weights in; dy and dw out; a scaling and a dot product of each row
        return {"bytes": 2.0 * H * (T + 2 * rows) + 3 * route, "flops": 3.0 * rows * H}
    if op == "dispatch_backward":
        H = case["H"]
        return {"bytes": 2.0 * H * (T + rows) + route, "flops": 1.0 * rows * H}
    if op == "dispatch_fp8":
        H = case["H"]
        return {"bytes": 2.0 * H * T + rows * (H + 4.0 * _blocks(H)) + route, "flops": 2.0 * T * H}
    K = case["K"]
    N = 2 * case["I"] if op == "swiglu" else case["N"]
    held = E * (1.0 - (1.0 - k * (1.0 - case["drop"]) / E) ** T)  # experts that hold a row
    out = case["I"] + 4.0 * _blocks(case["I"]) if op == "swiglu" else 2.0 * N
    weights = held * (N * K + 4.0 * _blocks(N) * _blocks(K))
    return {"bytes": rows * (K + 4.0 * _blocks(K) + out) + weights + 4.0 * (E + 1), "flops": 2.0 * rows * N * K}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op, T, k = case["op"], case["T"], case["k"]
    if op == "combine_backward":
        dy, dw = s["dy"].double(), s["dw"].double()
        for j in range(k):
            t = torch.nonzero(s["dest_row"][:, j] >= 0).reshape(-1)
            r = s["dest_row"][t, j].long()
            d = s["dout"][t].double()
            dy[r] = s["topk_w"][t, j].double()[:, None] * d
            dw[t, j] = (d * s["y"][r].double()).sum(1)
        return {"dy": dy, "dw": dw}
    if op == "dispatch_backward":
        dx = s["dx"].double()
        for j in range(k):
            t = torch.nonzero(s["dest_row"][:, j] >= 0).reshape(-1)
            dx[t] += s["drecv"][s["dest_row"][t, j].long()].double()
        return {"dx": dx}
    if op == "dispatch_fp8":
        q, scale = s["recv_q"].double(), s["recv_scale"].double()
        xq, xs = _exact_scaled(s["x"].double())
        for j in range(k):
            t = torch.nonzero(s["dest_row"][:, j] >= 0).reshape(-1)
            r = s["dest_row"][t, j].long()
            q[r], scale[r] = xq[t], xs[t]
        return {"q": q, "scale": scale}
    off = s["offsets"].tolist()
    if op == "gemm":
        y = s["out"].double()
        for e in range(case["E"]):
            if off[e + 1] > off[e]:
                y[off[e] : off[e + 1]] = _exact_rows(s, e, off)
        return {"y": y}
    q, scale = s["out_q"].double(), s["out_scale"].double()
    for e in range(case["E"]):
        if off[e + 1] > off[e]:
            h = _exact_rows(s, e, off)
            gate, up = h[:, : case["I"]], h[:, case["I"] :]
            q[off[e] : off[e + 1]], scale[off[e] : off[e + 1]] = _exact_scaled(torch.sigmoid(gate) * gate * up)
    return {"q": q, "scale": scale}


def _exact_scaled(v):
    """The values that 8-bit rows stand for before their rounding (value over
    scale, exact) and the scales."""
    q, scales = torch.empty_like(v), []
    for b in range(0, v.shape[1], BLOCK):
        part = v[:, b : b + BLOCK]
        s = part.abs().max(1).values.clamp_min(AMAX_FLOOR) / E4M3_MAX
        q[:, b : b + BLOCK] = part / s[:, None]
        scales.append(s)
    return q, torch.stack(scales, 1)


def _exact_rows(s, e, off):
    """One expert's product in 64 bits, block of 128 by block."""
    K = s["a"].shape[1]
    a, w = s["a"][off[e] : off[e + 1]].double(), s["b"][e].double()
    for c in range(_blocks(K)):
        cols = slice(c * BLOCK, min(K, (c + 1) * BLOCK))
        a[:, cols] *= s["a_scale"][off[e] : off[e + 1], c].double()[:, None]
        w[:, cols] *= torch.repeat_interleave(s["b_scale"][e, :, c].double(), BLOCK)[: w.shape[0], None]
    return a @ w.t()
