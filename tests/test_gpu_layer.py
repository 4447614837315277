"""The router and the experts' bf16 products on the GPU (include/ep_layer.h)
against plain implementations in 64 bits (layer_ref.py, whose bounds the
tolerances are), and a layer's forward and backward pass through the library."""

import math

import pytest
import torch

import bulk_async_tensor_amd as ep

import layer_ref as ref
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def same(a, b):
    assert a.shape == b.shape and torch.equal(bits(a), bits(b)), f"{int((bits(a) != bits(b)).sum())} values differ"


# ------------------------------------------------------------------ route
def logits_of(T, E, seed, dtype=F32, scale=1.5):
    return (torch.randn(T, E, generator=gen(seed), device=DEV) * scale).to(dtype)


def call_route(l, k, kind, **over):
    T = l.shape[0]
    idx = torch.full((T, k), -9, dtype=torch.int32, device=DEV)
    w = torch.full((T, k), -9.0, device=DEV)
    got = ep.ep_route(l, idx, w, score=kind, **over)
    assert got[0] is idx and got[1] is w
    return idx, w


def check_weights(w, want, l):
    """float32: a score's exp moves by half a step for each unit of its argument
    (the row's spread; beyond 105 exp is below float32's least number), and the
    exp, the sums and quotients add no more than 80."""
    l = l.double().cpu()
    fin = torch.where(torch.isfinite(l), l, 0.0)
    spread = (fin.amax(1) - fin.amin(1) + fin.abs().amax(1)).clamp(max=210).unsqueeze(1)
    w = w.cpu().double()
    assert torch.equal(torch.isnan(w), torch.isnan(want))
    keep = ~torch.isnan(want)
    err = ((w - want).abs() <= (80 + 2 * spread) * ref.U32 * want.abs() + 2.0 ** -140)
    assert bool(err[keep].all()), float(((w - want).abs() / want.abs())[keep].max())


def check_route(l, k, kind, **over):
    idx, w = call_route(l, k, kind, **over)
    names = dict(renormalize="renorm")
    want, ww = ref.route(l, k, kind, **{names.get(n, n): v for n, v in over.items()})
    wrong = (idx.cpu() != want).any(1)
    assert not bool(wrong.any()), f"{int(wrong.sum())} rows, first {int(wrong.nonzero()[0])}"
    check_weights(w, ww, l)
    return idx, w


ROUTES = [  # T, E, k, groups, top_groups, best
    (1, 1, 1, 1, 1, 1), (1, 256, 8, 8, 4, 2), (3, 8, 2, 1, 1, 1), (7, 5, 5, 1, 1, 1), (65, 64, 6, 1, 1, 1),
    (33, 60, 4, 4, 2, 1), (129, 128, 8, 8, 3, 2), (17, 257, 15, 1, 1, 1), (50, 300, 16, 3, 2, 2),
    (40, 512, 8, 64, 5, 1), (20, 1024, 32, 1, 1, 1), (9, 1000, 31, 8, 4, 2), (500, 96, 8, 2, 1, 2), (64, 64, 3, 64, 3, 1),
    (200, 72, 10, 6, 6, 2), (31, 33, 32, 1, 1, 1), (1000, 16, 2, 4, 1, 2), (6, 130, 17, 2, 2, 1),
]


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T, E, k, groups, top, best", ROUTES)
def test_route(T, E, k, groups, top, best, dtype, kind):
    l = logits_of(T, E, T + E, dtype)
    bias = torch.randint(-30, 31, (E,), generator=gen(E), device=DEV) * 0.001
    more = dict(groups=groups, top_groups=top, group_best=best)
    check_route(l, k, kind, renormalize=True, scale=2.5, bias=bias, **more)
    check_route(l, k, kind, renormalize=False, **more)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_close_scores(kind):
    """Scores that float32 cannot tell apart, and equal ones, are ordered as in 64 bits."""
    T, E, k = 300, 256, 8
    l = 2.0 + logits_of(T, E, 5) * 1e-6
    bias = torch.randn(E, generator=gen(6), device=DEV) * 1e-7
    check_route(l, k, kind, bias=bias)
    check_route(l, k, kind, bias=bias, groups=8, top_groups=3, group_best=2)
    check_route(l, k, kind)
    # a few values only: most comparisons are ties
    l = torch.randint(0, 4, (T, E), generator=gen(7), device=DEV).float()
    steps = torch.randint(0, 2, (E,), generator=gen(8), device=DEV) * 0.125
    for bias in (None, steps):
        check_route(l, k, kind, bias=bias)
        check_route(l.to(BF16), k, kind, bias=bias, groups=4, top_groups=2, group_best=2)
    # a router before its first step
    check_route(torch.zeros(T, E, device=DEV), k, kind)
    # saturated scores: the logits still decide
    check_route(logits_of(T, E, 9, scale=40.0), k, kind, renormalize=False)


@pytest.mark.parametrize("T", [1, 130])
def test_route_one_pair_decides(T):
    """One pair at the edge of the choice, apart by less than float32 holds, in either order of the indices."""
    E, k = 256, 8
    l = logits_of(T, E, 3).clamp_(max=2.0)
    l[:, 10:17] = 4.0 + torch.arange(7, device=DEV)
    l[:, 100], l[:, 200] = 3.0, 3.0
    bias = torch.zeros(E, device=DEV)
    for low, high in ((100, 200), (200, 100)):
        # scores of 0.95: a step of float64 there is 2^-53, so 2^-60 leaves them equal and 2^-50 does not
        for apart, first in ((2.0 ** -60, 100), (2.0 ** -50, high)):
            bias.zero_()
            bias[high] = apart
            idx, _ = check_route(l, k, "sigmoid", bias=bias)
            assert bool((idx[:, 7] == first).all())


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_masks_and_nan(kind, renorm):
    inf, nan = math.inf, math.nan
    T, E, k = 12, 40, 4
    l = logits_of(T, E, 11)
    l[0] = -inf                      # a row whose mask leaves nothing
    l[1, 1:] = -inf                  # one expert
    l[2, ::2] = -inf
    l[3] = torch.finfo(F32).min      # masks of the type's lowest value
    l[4, 3:] = torch.finfo(F32).min
    l[5, 7] = nan
    l[6, 0], l[6, 39] = inf, nan
    l[7, 5], l[7, 6] = inf, inf
    l[8] = nan
    l[9] = -200.0 - torch.arange(E, device=DEV) * 0.01
    l[10] = 0.0
    l[10, 1::2] = -0.0
    for over in (dict(), dict(groups=4, top_groups=2, group_best=2)):
        idx, _ = check_route(l, k, kind, renormalize=renorm, **over)
        assert all(len(set(r)) == k for r in idx.tolist())
    bias = torch.zeros(E, device=DEV)
    bias[5], bias[6], bias[7] = -inf, torch.finfo(F32).min, nan
    check_route(l, k, kind, renormalize=renorm, bias=bias)
    check_route(l, k, kind, renormalize=renorm, bias=bias, groups=8, top_groups=3, group_best=2)


def test_route_unaligned_rows():
    """Tensors aligned to their elements only."""
    for dtype in (F32, BF16):
        big = logits_of(1, 50 * 37 + 3, 21, dtype).view(-1)
        l = big[3:].view(50, 37)
        idx = torch.zeros(50 * 5 + 1, dtype=torch.int32, device=DEV)[1:].view(50, 5)
        w = torch.zeros(50 * 5 + 1, device=DEV)[1:].view(50, 5)
        bias = (torch.arange(38, device=DEV) * 0.003)[1:]
        ep.ep_route(l, idx, w, score="sigmoid", bias=bias)
        want, ww = ref.route(l, 5, "sigmoid", bias=bias)
        assert torch.equal(idx.cpu(), want)
        check_weights(w, ww, l)
        dl = torch.zeros(50 * 37 + 3, dtype=dtype, device=DEV)[3:].view(50, 37)
        check_route_backward(l, idx, "softmax", False, dl)


# ------------------------------------------------------------------ route, backward
def check_route_backward(l, idx, kind, renorm, dl=None, out=F32, seed=1):
    T, E = l.shape
    dw = torch.randn(idx.shape, generator=gen(seed), device=DEV)
    if dl is None:
        dl = torch.full((T, E), 7.0, dtype=out, device=DEV)
    assert ep.ep_route_backward(l, idx, dw, dl, score=kind, renormalize=renorm, scale=2.5) is dl
    want = ref.route_backward(l, idx, dw, kind, renorm, 2.5)
    # float32 as for the weights; the terms are dw's and their mean's size
    spread = float(l.float().max() - l.float().min()) + float(l.float().abs().max())
    size = 2.5 * torch.where(want != 0, dw.abs().amax(1, keepdim=True).cpu().double(), 0.0)
    s = ref.scores(kind, l.cpu())
    if renorm:
        s = s / torch.gather(s, 1, idx.cpu().long().clamp(0, E - 1)).sum(1, keepdim=True)
    tol = (100 + 2 * spread) * ref.U32 * s * size * idx.shape[1] ** 0.5
    got = dl.cpu().double()
    assert bool(((got - want).abs() <= ref.UNIT[dl.dtype] * (want.abs() + tol) + tol + 2.0 ** -133).all())


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T, E, k", [(1, 1, 1), (1, 256, 8), (3, 8, 2), (7, 5, 5), (65, 64, 6), (129, 60, 5),
                                     (40, 256, 8), (20, 1000, 32), (300, 33, 17), (2, 300, 3)])
def test_route_backward(T, E, k, renorm, kind):
    for dtype, out in ((F32, F32), (BF16, BF16), (F32, BF16)):
        l = logits_of(T, E, T + E, dtype)
        idx, _ = call_route(l, k, kind)
        check_route_backward(l, idx, kind, renorm, out=out)


def test_route_backward_odd_choices():
    """Entries of no expert, and an expert listed twice."""
    l = logits_of(30, 24, 1)
    idx, _ = call_route(l, 6, "softmax")
    idx[3, 2], idx[4, 0], idx[5] = -1, 24, -1
    idx[6, 1] = idx[6, 0]
    dw = torch.randn(30, 6, generator=gen(2), device=DEV)
    for kind in ("softmax", "sigmoid"):
        for renorm in (False, True):
            dl = torch.full((30, 24), 7.0, device=DEV)
            ep.ep_route_backward(l, idx, dw, dl, score=kind, renormalize=renorm)
            want = ref.route_backward(l, idx, dw, kind, renorm)
            want[5] = torch.where(torch.isnan(want[5]), 0.0, want[5])  # (no entry: nothing over an empty sum)
            assert bool(((dl.cpu().double() - want).abs() <= 400 * ref.U32 * dw.abs().max().item()).all())


def test_route_backward_masked_rows():
    l = logits_of(4, 16, 1)
    l[0] = -math.inf
    l[1, 2:] = -math.inf
    idx, _ = call_route(l, 4, "softmax")
    dw = torch.ones(4, 4, device=DEV)
    for kind in ("softmax", "sigmoid"):
        for renorm in (False, True):
            dl = torch.full((4, 16), 7.0, device=DEV)
            ep.ep_route_backward(l, idx, dw, dl, score=kind, renormalize=renorm)
            assert bool((dl[0] == 0).all()) and bool(torch.isfinite(dl).all()) and bool((dl[1, 2:] == 0).all())


# ------------------------------------------------------------------ products
def lay(T, E, k, seed, drop):
    if E == 0:
        return None
    return ep.ep_layout(ref.routing(T, E, k, seed, drop, DEV), E)["offsets"]


def within(got, want, bound, what):
    err = (got.double() - want).abs()
    bad = ~(err <= bound + 2.0 ** -130)
    assert not bool(bad.any()), (what, int(bad.sum()), float((err / bound)[bad].max()), bad.nonzero()[0].tolist())


def rms_within(got, want, deep, what):
    """The error's norm: half a step of the type spread evenly (its rms is 1 /
    sqrt 3 of that), and one step of 2^-23 of a sum for each 32 of its terms and 32 more."""
    if want.numel() < 4000:
        return
    limit = ref.UNIT[got.dtype] / math.sqrt(3) * 1.05 + (deep / 32 + 32) * 2 * ref.U32
    off, size = float((got.double() - want).norm()), float(want.norm())
    assert off <= limit * size, (what, off, size, limit)


def check_linear(a, offsets, b, act="none", dtype=BF16, bias=None, residual=None, pre=None, **call):
    rows, N = a.shape[0], b.shape[1]
    outs = N // 2 if act == "swiglu" else N
    y = torch.full((rows, outs), 77.0, dtype=dtype, device=DEV)
    if pre:
        pre = torch.full((rows, N), 55.0, dtype=BF16, device=DEV)
    assert ep.ep_grouped_linear(a, offsets, b, y, bias=bias, act=act, residual=residual, pre=pre, **call) is y
    lo, hi = (0, rows) if offsets is None else (int(offsets[0]), int(offsets[-1]))
    want, ey, z, ez = ref.linear(a, offsets, b, bias, act, residual, dtype)
    within(y[lo:hi], want[lo:hi], ey[lo:hi], "y")
    if act == "none" and residual is None:
        rms_within(y[lo:hi], want[lo:hi], a.shape[1], "y")
    assert bool((y[:lo] == 77).all()) and bool((y[hi:] == 77).all())
    if pre is not None:
        within(pre[lo:hi], z[lo:hi], ez[lo:hi], "pre")
        assert bool((pre[:lo] == 55).all()) and bool((pre[hi:] == 55).all())
    return y


def check_dgrad(dy, offsets, b, act="none", pre=None, **call):
    rows, K = dy.shape[0], b.shape[2]
    wide = 2 * K if act == "swiglu" else K
    dx = torch.full((rows, wide), 77.0, dtype=BF16, device=DEV)
    assert ep.ep_grouped_linear_dgrad(dy, offsets, b, dx, act=act, pre=pre, **call) is dx
    lo, hi = (0, rows) if offsets is None else (int(offsets[0]), int(offsets[-1]))
    want, e = ref.dgrad(dy, offsets, b, act, pre)
    within(dx[lo:hi], want[lo:hi], e[lo:hi], "dx")
    if act == "none":
        rms_within(dx[lo:hi], want[lo:hi], dy.shape[1], "dx")
    assert bool((dx[:lo] == 77).all()) and bool((dx[hi:] == 77).all())
    return dx


def check_wgrad(dy, a, offsets, E, dtype=F32, bias=True, **call):
    db = torch.full((E, dy.shape[1], a.shape[1]), 77.0, dtype=dtype, device=DEV)
    dbias = torch.full((E, dy.shape[1]), 77.0, device=DEV) if bias else None
    ep.ep_grouped_linear_wgrad(dy, a, offsets, db, dbias=dbias, **call)
    want, e, wb, eb = ref.wgrad(dy, a, offsets, E, dtype)
    within(db, want, e, "db")
    rms_within(db, want, dy.shape[0] / E, "db")
    if bias:
        within(dbias, wb, eb, "dbias")
    return db, dbias


SIZES = [  # T, E, k, K, N, drop (E = 0: one weight without offsets)
    (1, 0, 1, 8, 8, 0), (1, 8, 8, 16, 16, 0), (1, 64, 1, 1024, 64, 0), (2, 3, 3, 104, 80, 0), (5, 300, 2, 264, 48, 0.3),
    (16, 4, 1, 136, 272, 0), (63, 0, 1, 64, 256, 0), (64, 0, 1, 256, 64, 0), (65, 2, 1, 2056, 528, 0.1),
    (130, 5, 2, 640, 144, 0), (300, 7, 3, 1480, 1008, 0.1), (700, 3, 2, 384, 640, 0), (1024, 4, 4, 896, 256, 0),
    (3000, 2, 1, 392, 512, 0), (2500, 5, 2, 1152, 336, 0.05), (40, 1024, 8, 128, 32, 0), (128, 0, 1, 7168, 256, 0),
    (4099, 0, 1, 72, 1040, 0), (257, 1, 1, 512, 2064, 0.5), (33, 0, 1, 4096, 16, 0), (1, 0, 1, 7168, 4096, 0),
]
ACTS = ["none", "silu", "gelu", "swiglu"]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T, E, k, K, N, drop", SIZES)
def test_linear(T, E, k, K, N, drop, act):
    offsets, rows, held = lay(T, E, k, T + K, drop), T * k, max(E, 1)
    a, b = ref.rows(rows, K, 1, DEV), ref.weights(held, N, K, 2, DEV)
    bias = torch.randn(held, N, generator=gen(3), device=DEV)
    outs = N // 2 if act == "swiglu" else N
    if act == "swiglu" and N % 16:
        with pytest.raises(ep.EpError, match="multiple of 16"):
            check_linear(a, offsets, b, act)
        return
    check_linear(a, offsets, b, act)
    check_linear(a, offsets, b, act, F32, bias=bias, residual=ref.rows(rows, outs, 4, DEV), pre=True)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T, E, k, K, N, drop", SIZES)
def test_dgrad(T, E, k, K, N, drop, act):
    offsets, rows, held = lay(T, E, k, T + K, drop), T * k, max(E, 1)
    dy, b = ref.rows(rows, K, 1, DEV), ref.weights(held, K, N, 2, DEV)  # (N outputs, a sum over K)
    pre = None if act == "none" else ref.rows(rows, 2 * N if act == "swiglu" else N, 5, DEV, 2.0)
    check_dgrad(dy, offsets, b, act, pre)


@pytest.mark.parametrize("T, E, k, K, N, drop", SIZES + [(20000, 0, 1, 256, 64, 0), (9000, 2, 1, 520, 264, 0.1)])
def test_wgrad(T, E, k, K, N, drop):
    offsets, rows = lay(T, E, k, T + K, drop), T * k
    dy, a = ref.rows(rows, N, 1, DEV), ref.rows(rows, K, 2, DEV)
    check_wgrad(dy, a, offsets, max(E, 1))
    check_wgrad(dy, a, offsets, max(E, 1), BF16, bias=False)


# rows of each expert: none at either end, single rows, one expert with nearly all, edges of the row tiles
COUNTS = [[0, 0, 0], [0, 1, 0, 0, 1], [700, 0, 1, 2], [0, 0, 513], [16, 17, 15, 0, 31, 32, 33, 64, 63, 65],
          [128, 127, 129, 255, 256, 257], [1, 0, 2000, 0, 3]]


@pytest.mark.parametrize("counts", COUNTS)
def test_products_of_uneven_experts(counts):
    rows, E = sum(counts) + 5, len(counts)
    offsets = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    a, d = ref.rows(rows, 528, 3, DEV), ref.rows(rows, 272, 4, DEV)
    b = ref.weights(E, 272, 528, 5, DEV)
    pre = ref.rows(rows, 1056, 6, DEV)
    # rows that no expert holds may be anything
    for t in (a, d, pre):
        t[sum(counts):] = math.nan
    check_linear(a, offsets, b, "swiglu", pre=True)
    check_dgrad(d, offsets, b, "swiglu", pre)
    check_wgrad(d, a, offsets, E)


def test_values_stay_in_their_places():
    """A NaN or infinity reaches the results of its row and weight, and no others;
    past the ends of rows and segments lie NaN of the neighbours."""
    counts = [70, 3, 130]
    offsets = torch.tensor([0, 70, 73, 203], dtype=torch.int32, device=DEV)
    K, N = 136, 200
    a, d, b = ref.rows(203, K, 1, DEV), ref.rows(203, N, 2, DEV), ref.weights(3, N, K, 3, DEV)
    a[70:73] = math.nan   # the middle expert's rows
    d[70:73] = math.nan
    b[1] = math.nan
    a[5, 7], d[5, 9] = math.inf, math.inf
    y = torch.zeros(203, N, dtype=BF16, device=DEV)
    ep.ep_grouped_linear(a, offsets, b, y)
    dx = torch.zeros(203, K, dtype=BF16, device=DEV)
    ep.ep_grouped_linear_dgrad(d, offsets, b, dx)
    db = torch.zeros(3, N, K, device=DEV)
    dbias = torch.zeros(3, N, device=DEV)
    ep.ep_grouped_linear_wgrad(d, a, offsets, db, dbias)
    for t in (y, dx):
        assert bool(torch.isnan(t[70:73]).all())
        ok = torch.isfinite(t).all(1)
        ok[70:73] = True
        assert not bool(ok[5]) and int((~ok).sum()) == 1
    assert bool(torch.isnan(db[1]).all()) and bool(torch.isfinite(db[2]).all())
    bad = ~torch.isfinite(db[0])
    bad[9, :] = False
    bad[:, 7] = False
    assert not bool(bad.any())
    assert not bool(torch.isfinite(dbias[0, 9])) and bool(torch.isfinite(dbias[2]).all())
    assert counts[1] == 3


def test_offsets_out_of_range_are_clamped():
    """Offsets that do not ascend or leave the buffer reach nothing outside it."""
    rows, K, N = 300, 264, 272
    a, d, b = ref.rows(rows, K, 1, DEV), ref.rows(rows, N, 2, DEV), ref.weights(3, N, K, 3, DEV)
    offsets = torch.tensor([-5, 100, 40, 1 << 30], dtype=torch.int32, device=DEV)
    as_taken = [(0, 0, 100), (2, 40, 300)]  # (the second expert's segment ends before it starts)
    y = torch.full((rows, N), 77.0, dtype=BF16, device=DEV)
    ep.ep_grouped_linear(a, offsets, b, y)
    db = torch.full((3, N, K), 77.0, device=DEV)
    ep.ep_grouped_linear_wgrad(d, a, offsets, db)
    dx = torch.full((rows, K), 77.0, dtype=BF16, device=DEV)
    ep.ep_grouped_linear_dgrad(d, offsets, b, dx)
    assert bool((db[1] == 0).all())
    for e, lo, hi in as_taken:
        want, err, _, _ = ref.wgrad(d[lo:hi], a[lo:hi], None, 1, F32)
        within(db[e], want[0], err[0], "db")
    want, err, _, _ = ref.linear(a, None, b[2:], None, "none", None, BF16)
    within(y[100:], want[100:], err[100:], "y")  # rows of one expert alone
    want, err, _, _ = ref.linear(a, None, b[:1], None, "none", None, BF16)
    within(y[:40], want[:40], err[:40], "y")
    assert not bool((dx == 77).all(1).any())


def test_no_rows():
    b = ref.weights(2, 64, 32, 1, DEV)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    empty = torch.zeros(0, 32, dtype=BF16, device=DEV)
    out = torch.zeros(0, 64, dtype=BF16, device=DEV)
    ep.ep_grouped_linear(empty, off, b, out)
    ep.ep_grouped_linear_dgrad(out, off, b, empty)
    db, dbias = torch.full((2, 64, 32), 7.0, device=DEV), torch.full((2, 64), 7.0, device=DEV)
    ep.ep_grouped_linear_wgrad(out, empty, off, db, dbias)
    assert bool((db == 0).all()) and bool((dbias == 0).all())
    idx = torch.zeros(0, 4, dtype=torch.int32, device=DEV)
    w = torch.zeros(0, 4, device=DEV)
    ep.ep_route(torch.zeros(0, 8, device=DEV), idx, w)
    ep.ep_route_backward(torch.zeros(0, 8, device=DEV), idx, w, torch.zeros(0, 8, device=DEV))


def test_one_weight_is_one_expert():
    """Without offsets: the same bits as with one expert that holds every row, weight [N, K] or [1, N, K]."""
    for rows, K, N in ((300, 264, 528), (20, 2048, 64)):
        a, d = ref.rows(rows, K, 1, DEV), ref.rows(rows, N, 2, DEV)
        b = ref.weights(1, N, K, 3, DEV)
        off = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
        out = []
        for w, o in ((b, off), (b, None), (b[0], None)):
            y, dx = torch.zeros(rows, N, dtype=BF16, device=DEV), torch.zeros(rows, K, dtype=BF16, device=DEV)
            db = torch.zeros(w.shape, device=DEV)
            ep.ep_grouped_linear(a, o, w, y)
            ep.ep_grouped_linear_dgrad(d, o, w, dx)
            ep.ep_grouped_linear_wgrad(d, a, o, db)
            out.append((y, dx, db.view(1, N, K)))
        for other in out[1:]:
            for p, q in zip(out[0], other):
                same(p, q)


def test_refusals_of_the_binding():
    a, b = ref.rows(4, 64, 1, DEV), ref.weights(2, 32, 64, 2, DEV)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    y = torch.zeros(4, 32, dtype=BF16, device=DEV)
    l, idx, w = torch.zeros(4, 8, device=DEV), torch.zeros(4, 2, dtype=torch.int32, device=DEV), torch.zeros(4, 2, device=DEV)
    calls = [
        (lambda: ep.ep_grouped_linear(a, None, b, y), ValueError), (lambda: ep.ep_grouped_linear(a, off[:2], b, y), ValueError),
        (lambda: ep.ep_grouped_linear(a, off, b, y[:3]), ValueError), (lambda: ep.ep_grouped_linear(y, off, b, y), ValueError),
        (lambda: ep.ep_grouped_linear(a, off, b, y, act="tanh"), ValueError),
        (lambda: ep.ep_grouped_linear(a, off, b, y, act=1), ValueError),
        (lambda: ep.ep_grouped_linear(a, off, b, y, act="swiglu"), ValueError),
        (lambda: ep.ep_grouped_linear(a, off, b, y, bias=torch.zeros(32, device=DEV)), ValueError),
        (lambda: ep.ep_grouped_linear(a, off, b, y, residual=a), ValueError),
        (lambda: ep.ep_grouped_linear(a, off, b, y, pre=a), ValueError),
        (lambda: ep.ep_grouped_linear(a.half(), off, b, y), TypeError),
        (lambda: ep.ep_grouped_linear(a, off, b, y.half()), TypeError),
        (lambda: ep.ep_grouped_linear(a, off.long(), b, y), TypeError),
        (lambda: ep.ep_grouped_linear(a.t(), off, b, y), ValueError),
        (lambda: ep.ep_grouped_linear(a, off, b, y, workspace=y.cpu()), ValueError),
        (lambda: ep.ep_grouped_linear_dgrad(y, off, b, a, act="silu"), ValueError),
        (lambda: ep.ep_grouped_linear_dgrad(y, off, b, y), ValueError),
        (lambda: ep.ep_grouped_linear_dgrad(y, off, b, a, act="swiglu", pre=a), ValueError),
        (lambda: ep.ep_grouped_linear_wgrad(y, a, off, b.half()), TypeError),
        (lambda: ep.ep_grouped_linear_wgrad(a, y, off, b), ValueError),
        (lambda: ep.ep_grouped_linear_wgrad(y, a[:3], off, b), ValueError),
        (lambda: ep.ep_route(l, idx, w, score="relu"), ValueError), (lambda: ep.ep_route(l, idx, w[:3]), ValueError),
        (lambda: ep.ep_route(l, idx, w, bias=w[0]), ValueError), (lambda: ep.ep_route(l.half(), idx, w), TypeError),
        (lambda: ep.ep_route(l, idx, w, groups=3), ep.EpError), (lambda: ep.ep_route(l, idx, w, scale=math.nan), ep.EpError),
        (lambda: ep.ep_route_backward(l, idx, w, l[:3]), ValueError),
        (lambda: ep.ep_route_backward(l, idx.long(), w, l), TypeError),
    ]
    for call, error in calls:
        with pytest.raises(error):
            call()


# ------------------------------------------------------------------ streams and graphs
def a_pass(s):
    """Every entry point once, on the tensors of s."""
    ep.ep_grouped_linear(s["x"], None, s["wg"], s["logits"])
    ep.ep_route(s["logits"], s["idx"], s["w"], score="sigmoid", bias=s["bias"], groups=4, top_groups=2, group_best=2)
    ep.ep_grouped_linear(s["a"], s["off"], s["b"], s["h"], act="swiglu", pre=s["pre"])
    ep.ep_grouped_linear_dgrad(s["a"], s["off"], s["bt"], s["dpre"], act="swiglu", pre=s["pre"])
    ep.ep_grouped_linear_wgrad(s["dpre"], s["a"], s["off"], s["db"], s["dbias"])
    ep.ep_grouped_linear_wgrad(s["logits16"], s["x"], None, s["dwg"])
    ep.ep_route_backward(s["logits"], s["idx"], s["w"], s["dl"], score="sigmoid")


OUT = ("logits", "idx", "w", "h", "pre", "dpre", "db", "dbias", "dwg", "dl")


def state(seed, T=96, E=16, k=2, H=512, I=128):
    s = {"x": ref.rows(T, H, seed, DEV), "wg": ref.weights(1, E, H, seed + 1, DEV)[0],
         "logits": torch.zeros(T, E, device=DEV), "logits16": ref.rows(T, E, seed + 2, DEV),
         "idx": torch.zeros(T, k, dtype=torch.int32, device=DEV), "w": torch.zeros(T, k, device=DEV),
         "bias": torch.randn(E, generator=gen(seed), device=DEV) * 0.01, "off": lay(T, E, k, seed, 0.1),
         "a": ref.rows(T * k, H, seed + 3, DEV), "b": ref.weights(E, 2 * I, H, seed + 4, DEV),
         "bt": ref.weights(E, H, I, seed + 5, DEV), "dbias": torch.zeros(E, 2 * I, device=DEV),
         "db": torch.zeros(E, 2 * I, H, device=DEV), "dwg": torch.zeros(E, H, device=DEV),
         "dl": torch.zeros(T, E, device=DEV)}
    s.update(h=torch.zeros(T * k, I, dtype=BF16, device=DEV), pre=torch.zeros(T * k, 2 * I, dtype=BF16, device=DEV),
             dpre=torch.zeros(T * k, 2 * I, dtype=BF16, device=DEV))
    return s


def test_captured_graph():
    """A captured pass, replayed on new inputs with the program's own work between the replays."""
    s = state(1)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a_pass(s)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            a_pass(s)
    for seed in (2, 3, 4):
        new, want = state(seed), state(seed)
        for n, t in s.items():
            t.copy_(new[n])
        a_pass(want)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in OUT:
            same(s[n], want[n])
        a_pass(state(seed + 10))


def test_two_streams_at_once():
    states, wants = [state(i) for i in (5, 6)], [state(i) for i in (5, 6)]
    for w in wants:
        a_pass(w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for st, s in zip(streams, states):
            with torch.cuda.stream(st):
                a_pass(s)
    torch.cuda.synchronize()
    for s, w in zip(states, wants):
        for n in OUT:
            same(s[n], w[n])


def test_stream_argument_and_masked_stream():
    s, want = state(7), state(7)
    a_pass(want)
    torch.cuda.synchronize()
    masked = ep.ep_stream_create_cu_masked(ep.cu_mask_words(range(32)))
    try:
        for st in (torch.cuda.Stream(), masked):
            for n in OUT:
                s[n].zero_()
            torch.cuda.synchronize()
            ep.ep_grouped_linear(s["x"], None, s["wg"], s["logits"], stream=st)
            ep.ep_route(s["logits"], s["idx"], s["w"], score="sigmoid", bias=s["bias"], groups=4, top_groups=2,
                        group_best=2, stream=st)
            ep.ep_grouped_linear(s["a"], s["off"], s["b"], s["h"], act="swiglu", pre=s["pre"], stream=st)
            ep.ep_grouped_linear_dgrad(s["a"], s["off"], s["bt"], s["dpre"], act="swiglu", pre=s["pre"], stream=st)
            ep.ep_grouped_linear_wgrad(s["dpre"], s["a"], s["off"], s["db"], s["dbias"], stream=st)
            ep.ep_grouped_linear_wgrad(s["logits16"], s["x"], None, s["dwg"], stream=st)
            ep.ep_route_backward(s["logits"], s["idx"], s["w"], s["dl"], score="sigmoid", stream=st)
            st.synchronize()
            for n in OUT:
                same(s[n], want[n])
    finally:
        torch.cuda.synchronize()
        ep.ep_stream_destroy(masked)


# ------------------------------------------------------------------ a layer
@pytest.mark.parametrize("kind, T, H, I, E, k", [("softmax", 100, 256, 128, 8, 2), ("sigmoid", 333, 512, 192, 16, 4),
                                                 ("sigmoid", 1, 128, 64, 8, 3)])
def test_layer_forward_and_backward(kind, T, H, I, E, k):
    """Router, dispatch, experts, combine and a shared expert, and all their
    gradients, against torch's differentiation of the same layer in 64 bits on
    the same choice.  Every tensor between is rounded to bf16 once; a result
    passes at most 6 such roundings of half a step each, which add as norms, and
    a row's few terms can cancel to a half: 6 * 2^-8 * 2."""
    x = ref.rows(T, H, 1, DEV)
    wg = ref.weights(1, E, H, 2, DEV)
    w1, w2 = ref.weights(E, 2 * I, H, 3, DEV), ref.weights(E, H, I, 4, DEV)
    ws1, ws2 = ref.weights(1, 2 * I, H, 5, DEV), ref.weights(1, H, I, 6, DEV)
    dout = ref.rows(T, H, 7, DEV)
    z = dict(device=DEV)
    logits, idx, w = torch.zeros(T, E, **z), torch.zeros(T, k, dtype=torch.int32, **z), torch.zeros(T, k, **z)
    R = T * k

    def b16(*shape):
        return torch.zeros(*shape, dtype=BF16, device=DEV)

    # forward
    ep.ep_grouped_linear(x, None, wg, logits)
    ep.ep_route(logits, idx, w, score=kind, scale=1.5)
    lay_ = ep.ep_layout(idx, E)
    off, dest = lay_["offsets"], lay_["dest_row"]
    recv, h, pre, y, routed = b16(R, H), b16(R, I), b16(R, 2 * I), b16(R, H), b16(T, H)
    ep.ep_dispatch(x, dest, recv)
    ep.ep_grouped_linear(recv, off, w1, h, act="swiglu", pre=pre)
    ep.ep_grouped_linear(h, off, w2, y)
    ep.ep_combine(y, dest, w, routed)
    hs, pres, out = b16(T, I), b16(T, 2 * I), b16(T, H)
    ep.ep_grouped_linear(x, None, ws1, hs, act="swiglu", pre=pres)
    ep.ep_grouped_linear(hs, None, ws2, out, residual=routed)
    # backward
    dy, dw = b16(R, H), torch.zeros(T, k, **z)
    ep.ep_combine_backward(dout, y, dest, w, dy, dw)
    dw2, dw1 = torch.zeros(E, H, I, **z), torch.zeros(E, 2 * I, H, **z)
    dpre, drecv, dx = b16(R, 2 * I), b16(R, H), b16(T, H)
    ep.ep_grouped_linear_wgrad(dy, h, off, dw2)
    ep.ep_grouped_linear_dgrad(dy, off, w2, dpre, act="swiglu", pre=pre)
    ep.ep_grouped_linear_wgrad(dpre, recv, off, dw1)
    ep.ep_grouped_linear_dgrad(dpre, off, w1, drecv)
    ep.ep_dispatch_backward(drecv, dest, dx)
    dpres, dxs, dws2, dws1 = b16(T, 2 * I), b16(T, H), torch.zeros(1, H, I, **z), torch.zeros(1, 2 * I, H, **z)
    ep.ep_grouped_linear_wgrad(dout, hs, None, dws2)
    ep.ep_grouped_linear_dgrad(dout, None, ws2, dpres, act="swiglu", pre=pres)
    ep.ep_grouped_linear_wgrad(dpres, x, None, dws1)
    ep.ep_grouped_linear_dgrad(dpres, None, ws1, dxs)
    dlogits, dwg, dxg = b16(T, E), torch.zeros(1, E, H, **z), b16(T, H)
    ep.ep_route_backward(logits, idx, dw, dlogits, score=kind, scale=1.5)
    ep.ep_grouped_linear_wgrad(dlogits, x, None, dwg)
    ep.ep_grouped_linear_dgrad(dlogits, None, wg, dxg)
    # the same in 64 bits
    leaves = [t.double().cpu().requires_grad_() for t in (x, wg, w1, w2, ws1, ws2)]
    X, WG, W1, W2, S1, S2 = leaves
    lg = X @ WG[0].t()
    s = torch.sigmoid(lg) if kind == "sigmoid" else torch.softmax(lg, 1)
    ids = idx.cpu().long()
    g = torch.gather(s, 1, ids)
    g = 1.5 * g / g.sum(1, keepdim=True)

    def mlp(v, a, b):
        q = v @ a.t()
        return (torch.nn.functional.silu(q[:, :I]) * q[:, I:]) @ b.t()

    total = mlp(X, S1[0], S2[0])
    for j in range(k):
        total = total + g[:, j : j + 1] * torch.cat([mlp(X[t : t + 1], W1[ids[t, j]], W2[ids[t, j]]) for t in range(T)])
    grads = torch.autograd.grad((total * dout.double().cpu()).sum(), leaves)
    limit = 6 * ref.UBF16 * 2
    for name, got, want in (("out", out, total), ("dx", dx.double() + dxs.double() + dxg.double(), grads[0]),
                            ("dwg", dwg, grads[1]), ("dw1", dw1, grads[2]), ("dw2", dw2, grads[3]),
                            ("dws1", dws1, grads[4]), ("dws2", dws2, grads[5])):
        rel = float((got.double().cpu() - want.detach()).norm() / want.detach().norm())
        print(name, rel)
        assert rel <= limit, (name, rel)
