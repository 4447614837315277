"""Plain implementations in 64 bits of the router and of the experts' bf16
products, with bounds on what float32 sums and the roundings of the results may
add to them."""

import math

import torch

U32 = 2.0 ** -24   # half a step of float32, relative
UBF16 = 2.0 ** -8  # of bf16
UNIT = {torch.float32: U32, torch.bfloat16: UBF16}


# Rows, experts, K, N at which the products' rule takes tiles of 64, 128 and 256 rows, whole sums and cut ones, for
# each product.
HEIGHTS = [(1106, 1, 64, 64), (224, 20, 64, 1632), (5354, 5, 64, 2560), (5881, 9, 264, 2384), (2971, 1, 144, 3360),
           (3834, 1, 2072, 64), (5589, 3, 264, 2656), (5492, 3, 2344, 288), (2696, 5, 3016, 144), (5493, 9, 3328, 272),
           (5968, 3, 328, 1872), (3939, 1, 136, 1664), (5823, 3, 3608, 144), (110, 1, 1240, 64), (118, 1, 80, 1184),
           (5470, 5, 296, 2864), (4481, 2, 280, 3040)]


def routing(T, E, k, seed, drop=0.0, device="cpu"):
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand(T, E, generator=g).argsort(1)[:, :k].to(torch.int32)
    ids[torch.rand(T, k, generator=g) < drop] = -1
    return ids.to(device)


def rows(n, width, seed, device, scale=1.0):
    g = torch.Generator(device=device).manual_seed(seed)
    return (torch.randn(n, width, generator=g, device=device) * scale).to(torch.bfloat16)


def weights(E, N, K, seed, device):
    g = torch.Generator(device=device).manual_seed(seed)
    return (torch.randn(E, N, K, generator=g, device=device) / math.sqrt(K)).to(torch.bfloat16)


def spans(offsets, n):
    off = [0, n] if offsets is None else offsets.tolist()
    return [(e, slice(off[e], off[e + 1])) for e in range(len(off) - 1)]


# ------------------------------------------------------------------ router
def scores(kind, l):
    """In 64 bits; a row of -infinity alone has scores 0."""
    l = l.double()
    if kind == "sigmoid":
        return torch.sigmoid(l)
    s = torch.softmax(l, 1)
    return torch.where((l == -math.inf).all(1, keepdim=True), 0.0, s)


def best_first(v):
    """Indices by descending value, NaN first, equal ones in their order."""
    key = torch.where(torch.isnan(v), math.inf, v)
    first = torch.sort(key, dim=1, descending=True, stable=True).indices
    nan = torch.gather(torch.isnan(v), 1, first)
    again = torch.sort(nan.to(torch.int8), dim=1, descending=True, stable=True).indices
    return torch.gather(first, 1, again)


def route(logits, k, kind, bias=None, groups=1, top_groups=1, group_best=1, renorm=True, scale=1.0):
    """(ids, weights) in 64 bits on the CPU."""
    l = logits.cpu().double()
    T, E = l.shape
    s = scores(kind, l)
    c = s if bias is None else s + bias.cpu().double()
    order = best_first(l if bias is None else c)
    if groups > 1:
        per = E // groups
        parts = c.view(T * groups, per)
        ranked = torch.gather(parts, 1, best_first(parts))[:, :group_best].sum(1).view(T, groups)
        kept = torch.zeros(T, groups, dtype=torch.bool).scatter_(1, best_first(ranked)[:, :top_groups], True)
        inside = torch.gather(kept.repeat_interleave(per, 1), 1, order)
        order = torch.gather(order, 1, torch.sort(inside.to(torch.int8), dim=1, descending=True, stable=True).indices)
    ids = order[:, :k]
    w = torch.gather(s, 1, ids)
    if renorm:
        chosen = torch.gather(l, 1, ids)
        shift = chosen.amax(1, keepdim=True)
        if kind == "sigmoid":
            shift = shift.clamp(max=0.0)
            w = torch.exp(chosen.clamp(max=0.0) - shift) / (1.0 + torch.exp(-chosen.abs()))
        elif not torch.isnan(s).any():
            w = torch.exp(chosen - shift)
        w = torch.where((chosen == -math.inf).all(1, keepdim=True), 0.0, w / w.sum(1, keepdim=True))
    return ids.to(torch.int32), w * scale


def route_backward(logits, ids, dw, kind, renorm=True, scale=1.0):
    """The header's formulas, entry by entry of ids (any outside [0, E) left out)."""
    l, dw = logits.cpu().double(), dw.cpu().double()
    T, E = l.shape
    ids = ids.cpu().long()
    ok = (ids >= 0) & (ids < E)
    at = ids.clamp(0, E - 1)
    s = scores(kind, l)
    p = torch.where(ok, torch.gather(s, 1, at), 0.0)
    sj = p.clone()
    if renorm:
        p = p / p.sum(1, keepdim=True)
    dw = torch.where(ok, dw, 0.0)
    D = (p * dw).sum(1, keepdim=True)
    if kind == "sigmoid":
        g = p * (1 - sj) * (dw - D if renorm else dw)
    else:
        g = p * (dw - D) if renorm else p * dw
    out = torch.zeros_like(l)
    if kind == "softmax" and not renorm:
        out -= s * D
    for j in range(ids.shape[1]):
        out.scatter_add_(1, at[:, j : j + 1], torch.where(ok, g, 0.0)[:, j : j + 1])
    return out * scale


# ------------------------------------------------------------------ products
def act(kind, z):
    if kind in ("silu", "swiglu"):
        return z * torch.sigmoid(z)
    if kind == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2.0))
    return z


def slope(kind, z):
    if kind in ("silu", "swiglu"):
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if kind == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def of_sum(deep, magnitude):
    """What float32 sums of `deep` exact products may be off by, in any order
    and with each addition cut rather than rounded (a step of 2^-23): the sum of
    the terms' magnitudes times one step an addition."""
    return (deep + 2) * 2 * U32 * magnitude


def of_act(z):
    """Relative error of an activation's own float32 arithmetic at z: the
    argument's rounding moves exp by |z| and erfc by z^2 half steps, and no more
    than 16 are added by the functions and products."""
    return (z * z + z.abs() + 16) * U32


def product(x, offsets, w, across):
    """x[r] times its expert's weight (across: the weight's columns), and the sums of the terms' magnitudes, 64 bits."""
    width = w.shape[2] if across else w.shape[1]
    z = torch.full((x.shape[0], width), math.nan, dtype=torch.float64, device=x.device)
    mag = z.clone()
    for e, r in spans(offsets, x.shape[0]):
        m = w[e].double() if across else w[e].double().t()
        z[r] = x[r].double() @ m
        mag[r] = x[r].double().abs() @ m.abs()
    return z, mag


def linear(a, offsets, b, bias, kind, residual, dtype):
    """y, its bound, pre, its bound."""
    z, mag = product(a, offsets, b, False)
    if bias is not None:
        for e, r in spans(offsets, a.shape[0]):
            z[r] += bias.view(b.shape[0], -1)[e].double()
            mag[r] += bias.view(b.shape[0], -1)[e].double().abs()
    ez = of_sum(a.shape[1], mag)
    if kind == "swiglu":
        g, u = z.chunk(2, 1)
        eg, eu = ez.chunk(2, 1)
        s = act(kind, g)
        y = s * u
        es = 1.13 * eg + of_act(g) * s.abs()
        ey = es * (u.abs() + eu) + s.abs() * eu + U32 * y.abs()
    else:
        y = act(kind, z)
        ey = ez if kind == "none" else 1.13 * ez + of_act(z) * y.abs()
    if residual is not None:
        y = y + residual.double()
        ey = ey + U32 * y.abs()
    return y, UNIT[dtype] * (y.abs() + ey) + ey, z, UBF16 * (z.abs() + ez) + ez


def dgrad(dy, offsets, b, kind, pre):
    """dx and its bound."""
    d, mag = product(dy, offsets, b, True)
    ed = of_sum(dy.shape[1], mag)
    if kind == "none":
        return d, UBF16 * (d.abs() + ed) + ed
    z = pre.double()
    g, u = z.chunk(2, 1) if kind == "swiglu" else (z, None)
    p = slope(kind, g)
    # the slope's terms, each of magnitude 1 + |z| at most, may cancel
    ep = of_act(g) * (torch.exp(-g * g / 4) + torch.sigmoid(g)) * (1 + g.abs())
    if kind == "swiglu":
        s = act(kind, g)
        x = torch.cat([p * u * d, s * d], 1)
        ex = torch.cat([u.abs() * (p.abs() * ed + ep * (d.abs() + ed)), s.abs() * (ed + of_act(g) * (d.abs() + ed))], 1)
    else:
        x = p * d
        ex = p.abs() * ed + ep * (d.abs() + ed)
    ex = ex + 2 * U32 * x.abs()
    return x, UBF16 * (x.abs() + ex) + ex


def wgrad(dy, a, offsets, E, dtype):
    """db, its bound, dbias, its bound."""
    N, K = dy.shape[1], a.shape[1]
    db = torch.zeros(E, N, K, dtype=torch.float64, device=dy.device)
    eb = db.clone()
    dbias = torch.zeros(E, N, dtype=torch.float64, device=dy.device)
    ebias = dbias.clone()
    for e, r in spans(offsets, dy.shape[0]):
        n = r.stop - r.start
        if n <= 0:
            continue
        d, x = dy[r].double(), a[r].double()
        db[e] = d.t() @ x
        eb[e] = of_sum(n, d.abs().t() @ x.abs())
        dbias[e] = d.sum(0)
        ebias[e] = of_sum(n, d.abs().sum(0))
    return db, UNIT[dtype] * (db.abs() + eb) + eb, dbias, ebias + U32 * dbias.abs()
