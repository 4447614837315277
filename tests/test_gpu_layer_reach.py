"""The router and the bf16 products at the ends of their ranges: workgroups that
go through many tiles, sums of few steps, buffers past 4 GiB, launches in more
than one piece, and workspaces of the caller's."""

import math

import pytest
import torch

import bulk_async_tensor_amd as ep

import layer_ref as ref
from gpu_helpers import DEV
from test_gpu_layer import (BF16, F32, check_dgrad, check_linear, check_route, check_wgrad, gen, logits_of, same,
                            within)

pytestmark = pytest.mark.gpu


def offsets_of(counts):
    return torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device=DEV)


@pytest.fixture(scope="module")
def eight_cus():
    stream = ep.ep_stream_create_cu_masked(ep.cu_mask_words(range(8)))
    yield stream
    torch.cuda.synchronize()
    ep.ep_stream_destroy(stream)


# Sums of one to six steps (three copies or two in LDS, one step more in a tile at least), tiles of 64, 128 and 256
# rows, and items that eight workgroups share in many rounds: rows of each expert, K, N.
STREAMS = [([500, 0, 130, 257, 64, 1], 64, 600), ([300, 700], 72, 2056), ([129] * 9, 128, 520), ([256] * 5, 200, 1000),
           ([4000, 5000], 64, 1288), ([3000] * 4, 192, 1040), ([2000, 0, 2500, 1], 264, 1544), ([9000], 384, 776),
           ([4000, 5000], 1288, 64), ([3000] * 4, 1040, 192), ([500, 0, 700, 10], 1032, 4104)]


@pytest.mark.parametrize("counts, K, N", STREAMS)
def test_streams_of_tiles(counts, K, N, eight_cus):
    """On a stream of eight compute units each workgroup goes through many tiles: the same bits as on all."""
    offsets, rows, E = offsets_of(counts), sum(counts), len(counts)
    a, d, b = ref.rows(rows, K, 1, DEV), ref.rows(rows, N, 2, DEV), ref.weights(E, N, K, 3, DEV)
    pre, bias = ref.rows(rows, 2 * K, 4, DEV), torch.randn(E, N, generator=gen(5), device=DEV)
    want = (check_linear(a, offsets, b, "gelu", bias=bias), check_dgrad(d, offsets, b, "swiglu", pre),
            *check_wgrad(d, a, offsets, E))
    torch.cuda.synchronize()
    y = torch.full((rows, N), 77.0, dtype=BF16, device=DEV)
    dx = torch.full((rows, 2 * K), 77.0, dtype=BF16, device=DEV)
    db, dbias = torch.full((E, N, K), 77.0, device=DEV), torch.full((E, N), 77.0, device=DEV)
    torch.cuda.synchronize()
    ep.ep_grouped_linear(a, offsets, b, y, bias=bias, act="gelu", stream=eight_cus)
    ep.ep_grouped_linear_dgrad(d, offsets, b, dx, act="swiglu", pre=pre, stream=eight_cus)
    ep.ep_grouped_linear_wgrad(d, a, offsets, db, dbias, stream=eight_cus)
    eight_cus.synchronize()
    for got, w in zip((y, dx, db, dbias), want):
        same(got, w)


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("rows, E, K, N", ref.HEIGHTS)
def test_every_height(rows, E, K, N, act):
    """Tiles of 64, 128 and 256 rows, whole sums and cut ones, of each product."""
    offsets = None if E == 1 else ep.ep_layout(ref.routing(rows, E, 1, 7, 0.02, DEV), E)["offsets"]
    a, d, b = ref.rows(rows, K, 1, DEV), ref.rows(rows, N, 2, DEV), ref.weights(E, N, K, 3, DEV)
    bias, swiglu = torch.randn(E, N, generator=gen(4), device=DEV), act == "swiglu"
    check_linear(a, offsets, b, act, bias=bias, residual=ref.rows(rows, N // 2 if swiglu else N, 5, DEV), pre=True)
    check_linear(a, offsets, b, act, F32)
    check_dgrad(d, offsets, b, act, None if act == "none" else ref.rows(rows, 2 * K if swiglu else K, 6, DEV, 2.0))
    if act == "none":
        check_wgrad(d, a, offsets, E)
        check_wgrad(d, a, offsets, E, BF16, bias=False)


def test_rows_past_4_gib():
    """Token rows and results whose byte offsets pass 32 bits; the last expert holds the last rows."""
    rows, wide = 300000, 8192
    tail = 777
    offsets = torch.tensor([0, 5, 5, rows - tail, rows], dtype=torch.int32, device=DEV)
    a = torch.zeros(rows, wide, dtype=BF16, device=DEV)
    a[:5] = ref.rows(5, wide, 1, DEV)
    a[-tail:] = ref.rows(tail, wide, 2, DEV)
    narrow = ref.rows(rows, 64, 3, DEV)
    b = ref.weights(4, 64, wide, 4, DEV)
    y = torch.zeros(rows, 64, dtype=BF16, device=DEV)
    ep.ep_grouped_linear(a, offsets, b, y)
    for e, lo in ((0, 0), (3, rows - tail)):
        hi = lo + (5 if e == 0 else tail)
        want, err, _, _ = ref.linear(a[lo:hi], None, b[e : e + 1], None, "none", None, BF16)
        within(y[lo:hi], want, err, "y")
    db = torch.full((4, 64, wide), 7.0, device=DEV)
    ep.ep_grouped_linear_wgrad(narrow, a, offsets, db)
    want, err, _, _ = ref.wgrad(narrow[-tail:], a[-tail:], None, 1, F32)
    within(db[3], want[0], err[0], "db")
    assert bool((db[1] == 0).all())
    dx = torch.empty(rows, wide, dtype=BF16, device=DEV)
    ep.ep_grouped_linear_dgrad(narrow, offsets, b, dx)
    want, err = ref.dgrad(narrow[-tail:], None, b[3:], "none", None)
    within(dx[-tail:], want, err, "dx")
    want, err = ref.dgrad(narrow[5:50], None, b[2:3], "none", None)
    within(dx[5:50], want, err, "dx")


def test_weights_past_4_gib():
    """A weight and a float32 gradient of 5 GB, experts at both ends."""
    E, N, K = 300, 2048, 2048
    rows = 200
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:-1] = 90
    offsets[-1] = rows
    big = torch.zeros(E + 350, N, K, dtype=BF16, device=DEV)
    b = big[350:]
    b[0], b[-1] = ref.weights(1, N, K, 1, DEV)[0], ref.weights(1, N, K, 2, DEV)[0]
    a, d = ref.rows(rows, K, 3, DEV), ref.rows(rows, N, 4, DEV)
    y, dx = torch.zeros(rows, N, dtype=BF16, device=DEV), torch.zeros(rows, K, dtype=BF16, device=DEV)
    # all experts of the larger tensor: the last one lies past 4 GiB
    off_big = torch.zeros(E + 351, dtype=torch.int32, device=DEV)
    off_big[351:-1] = 90
    off_big[-1] = rows
    ep.ep_grouped_linear(a, off_big, big, y)
    ep.ep_grouped_linear_dgrad(d, off_big, big, dx)
    for e, r in ((0, slice(0, 90)), (-1, slice(90, rows))):
        w = b[e].unsqueeze(0)
        want, err, _, _ = ref.linear(a[r], None, w, None, "none", None, BF16)
        within(y[r], want, err, "y")
        want, err = ref.dgrad(d[r], None, w, "none", None)
        within(dx[r], want, err, "dx")
    del big, b
    db = torch.full((E, N, K), 7.0, device=DEV)
    ep.ep_grouped_linear_wgrad(d, a, offsets, db)
    for e, r in ((0, slice(0, 90)), (-1, slice(90, rows))):
        want, err, _, _ = ref.wgrad(d[r], a[r], None, 1, F32)
        within(db[e], want[0], err[0], "db")
    assert float(db[1:-1].abs().max()) == 0.0


def test_longest_sides():
    """A weight's sides at their limit, and sums over very many places."""
    side = 1 << 20
    a, b = ref.rows(3, side, 1, DEV), ref.weights(1, 8, side, 2, DEV)
    check_linear(a, None, b, dtype=F32)
    d = ref.rows(3, 8, 3, DEV)
    check_dgrad(d, None, b)
    check_wgrad(d, a, None, 1)
    w = ref.weights(1, side, 16, 4, DEV)
    x = ref.rows(2, 16, 5, DEV)
    check_linear(x, None, w, "swiglu")
    check_dgrad(ref.rows(2, side, 6, DEV), None, w)


@pytest.mark.parametrize("op", ["linear", "dgrad", "wgrad"])
def test_workspace_of_the_caller(op):
    """What a workspace holds does not matter; one that is too small is refused; a larger one may be any size."""
    rows, K, N = 200, 4096, 264
    a, d, b = ref.rows(rows, K, 1, DEV), ref.rows(rows, N, 2, DEV), ref.weights(1, N, K, 3, DEV)
    if op == "wgrad":
        rows = 8192
        a, d = ref.rows(rows, 264, 1, DEV), ref.rows(rows, 128, 2, DEV)
        need = ep.ep_grouped_linear_wgrad_workspace_bytes(rows, 264, 1, 128)
    elif op == "dgrad":
        d, b = ref.rows(rows, K, 2, DEV), ref.weights(1, K, N, 3, DEV)
        need = ep.ep_grouped_linear_dgrad_workspace_bytes(rows, N, 1, K)
    else:
        need = ep.ep_grouped_linear_workspace_bytes(rows, K, 1, N)
    assert need > 0

    def call(workspace):
        if op == "linear":
            return check_linear(a, None, b, workspace=workspace)
        if op == "dgrad":
            return check_dgrad(d, None, b, workspace=workspace)
        return check_wgrad(d, a, None, 1, workspace=workspace)[0]

    want = call(None)
    for size in (need, need + 4096):
        ws = torch.full((size // 4,), math.nan, device=DEV)
        same(call(ws), want)
        same(call(ws), want)
    with pytest.raises(ep.EpError, match="workspace"):
        call(torch.zeros(need - 16, dtype=torch.uint8, device=DEV))


def test_graphs_that_share_a_workspace():
    """Two captured calls on one workspace, replayed one after the other on a stream."""
    need = ep.ep_grouped_linear_workspace_bytes(64, 4096, 1, 128)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    xs = [ref.rows(64, 4096, i, DEV) for i in (1, 2)]
    b = ref.weights(1, 128, 4096, 3, DEV)
    ys = [torch.zeros(64, 128, device=DEV) for _ in xs]
    side = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(side):
        for x, y in zip(xs, ys):
            ep.ep_grouped_linear(x, None, b, y, workspace=ws)
            side.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                ep.ep_grouped_linear(x, None, b, y, workspace=ws)
            graphs.append(g)
    for seed in (5, 6, 7):
        for i, x in enumerate(xs):
            x.copy_(ref.rows(64, 4096, seed + 10 * i, DEV))
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for x, y in zip(xs, ys):
            want, err, _, _ = ref.linear(x, None, b, None, "none", None, F32)
            within(y, want, err, "y")


def test_route_of_very_many_tokens():
    """More tokens than one launch takes, and logits past 4 GiB."""
    T, E = (1 << 26) + 1000, 4
    l = torch.randint(-8, 8, (T, E), generator=gen(1), device=DEV, dtype=torch.int8).float()
    idx, w = torch.full((T, 1), -9, dtype=torch.int32, device=DEV), torch.full((T, 1), -9.0, device=DEV)
    ep.ep_route(l, idx, w, score="sigmoid", renormalize=False)
    assert torch.equal(idx[:, 0].long(), l.argmax(1))  # (of equal ones the lowest: torch's on these sizes too)
    want = torch.sigmoid(l.double().amax(1))
    assert float(((w[:, 0].double() - want) / want).abs().max()) < 8 * ref.U32 * 8
    del l, idx, w, want
    T, E = 5_000_000, 256
    l = torch.randn(T, E, generator=gen(2), device=DEV)
    idx, w = torch.full((T, 2), -9, dtype=torch.int32, device=DEV), torch.full((T, 2), -9.0, device=DEV)
    ep.ep_route(l, idx, w, score="softmax")
    for r in (slice(0, 500), slice(T - 500, T)):
        assert torch.equal(idx[r].cpu(), ref.route(l[r], 2, "softmax")[0])
    dl = torch.full((T, E), 7.0, dtype=BF16, device=DEV)
    ep.ep_route_backward(l, idx, w, dl)
    r = slice(T - 500, T)
    want = ref.route_backward(l[r], idx[r], w[r], "softmax")
    assert float((dl[r].cpu().double() - want).abs().max()) <= ref.UBF16
    assert bool((w.sum(1) - 1).abs().max() < 4 * ref.U32)


# ------------------------------------------------------------------ enough tokens for 16 lanes each
MANY = 2100  # (2048 and fewer take 64 lanes on 256 compute units)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("E, k, groups, top, best", [(128, 8, 32, 9, 2), (100, 15, 1, 1, 1), (256, 8, 8, 4, 2),
                                                     (255, 6, 5, 2, 2), (512, 8, 64, 5, 1), (300, 15, 3, 2, 2),
                                                     (257, 1, 1, 1, 1), (500, 4, 50, 50, 2)])
def test_route_many_tokens(E, k, groups, top, best, dtype, kind):
    l = logits_of(MANY, E, E, dtype)
    bias = torch.randint(-30, 31, (E,), generator=gen(E), device=DEV) * 0.001
    more = dict(groups=groups, top_groups=top, group_best=best)
    check_route(l, k, kind, renormalize=True, scale=2.5, bias=bias, **more)
    check_route(l, k, kind, renormalize=False, **more)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [128, 256, 512])
def test_route_many_tokens_close(E, kind):
    """Near ties, ties, masks and NaN beside ordinary tokens in one wave."""
    k, inf, nan = 8, math.inf, math.nan
    l = logits_of(MANY, E, 1)
    some = torch.arange(0, MANY, 3, device=DEV)
    l[some] = 2.0 + l[some] * 1e-6
    l[1::7] = torch.randint(0, 4, (len(range(1, MANY, 7)), E), generator=gen(2), device=DEV).float()
    l[5], l[50, 1:], l[51, ::2], l[52] = -inf, -inf, -inf, torch.finfo(F32).min
    l[100, 3:], l[101, 7], l[102, 0], l[102, E - 1], l[103] = torch.finfo(F32).min, nan, inf, nan, nan
    l[104] = -200.0 - torch.arange(E, device=DEV) * 0.01
    l[105, 5], l[105, 6] = inf, inf
    near = torch.randn(E, generator=gen(3), device=DEV) * 1e-7
    odd = near.clone()
    odd[5], odd[6], odd[7] = -inf, torch.finfo(F32).min, nan
    for over in (dict(), dict(bias=near), dict(bias=odd), dict(groups=8, top_groups=3, group_best=2),
                 dict(bias=near, groups=8, top_groups=3, group_best=2),
                 dict(bias=odd, groups=4, top_groups=2, group_best=2)):
        for renorm in (False, True):
            idx, _ = check_route(l, k, kind, renormalize=renorm, **over)
            assert bool((idx.sort(1).values.diff(dim=1) > 0).all()) and bool((idx >= 0).all()) and bool((idx < E).all())


# ------------------------------------------------------------------ what follows a product
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows, E, K, N", [(300, 3, 128, 400), (40, 2, 2048, 272), (2000, 2, 1536, 1040),
                                           (900, 2, 4096, 1040), (3000, 3, 128, 2704), (5493, 9, 3328, 272)])
def test_every_epilogue(rows, E, K, N, dtype, act):
    """Bias, residual and pre in all combinations, on whole sums and on cut ones."""
    first = rows // E + 1
    offsets = offsets_of([first] + [0] * (E - 2) + [rows - first])
    a, b = ref.rows(rows, K, 1, DEV), ref.weights(E, N, K, 2, DEV)
    bias = torch.randn(E, N, generator=gen(3), device=DEV)
    res = ref.rows(rows, N // 2 if act == "swiglu" else N, 4, DEV)
    for use in range(8):
        check_linear(a, offsets, b, act, dtype, bias=bias if use & 1 else None, residual=res if use & 2 else None,
                     pre=bool(use & 4) or None)


@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu"])
def test_activations_over_their_range(act):
    """Values and slopes from far below zero to far above, relative to the value.

    The sum is zero, so z is the bias itself.  The argument's rounding moves exp
    by |z| and erfc by z^2 half steps at most; the fit, its ten additions, the
    exponential, the reciprocal and the products add no more than 18, and 24 are
    allowed.  Below -88.7 the exponential overflows and the result is 0, where it
    is 88.8 e^-88.8 = 2e-37 < 2^-120 in magnitude (times the up product)."""
    n = 4096
    z = torch.linspace(-120, 120, n, device=DEV)
    z[:1000] = torch.linspace(-6, 6, 1000, device=DEV)
    g, u = z.double(), torch.ones(n, dtype=torch.float64, device=DEV)
    if act == "swiglu":
        z = torch.cat([z, z.flip(0)])
        g, u = z.double().chunk(2)
    a, b = torch.zeros(3, 8, dtype=BF16, device=DEV), torch.zeros(1, len(z), 8, dtype=BF16, device=DEV)
    y = torch.full((3, n), 77.0, device=DEV)
    ep.ep_grouped_linear(a, None, b, y, bias=z.view(1, -1), act=act)
    want = ref.act(act, g) * u
    bound = (g * g + g.abs() + 24) * ref.U32 * want.abs() + 2.0 ** -120 * u.abs()
    within(y, want.expand(3, n), bound.expand(3, n), "y")
    pre, dy = z.to(BF16).expand(3, -1).contiguous(), ref.rows(3, 8, 5, DEV)
    ones = torch.ones(1, 8, n, dtype=BF16, device=DEV)
    dx = torch.full(pre.shape, 77.0, dtype=BF16, device=DEV)
    ep.ep_grouped_linear_dgrad(dy, None, ones, dx, act=act, pre=pre)
    want, e = ref.dgrad(dy, None, ones, act, pre)
    within(dx, want, e + 2.0 ** -120 * 128 * 64, "dx")  # (|u| <= 120, |d| <= 64)


def test_rows_before_the_first_segment():
    """Offsets that start past zero: the rows before them are not touched either, whole sums or cut ones."""
    offsets = torch.tensor([5, 20, 20, 33], dtype=torch.int32, device=DEV)
    for K, N in ((64, 264), (4096, 136)):
        a, d, b = ref.rows(40, K, 1, DEV), ref.rows(40, N, 2, DEV), ref.weights(3, N, K, 3, DEV)
        for t in (a, d):
            t[:5], t[33:] = math.nan, math.nan
        check_linear(a, offsets, b, "silu", pre=True, bias=torch.randn(3, N, generator=gen(4), device=DEV))
        check_dgrad(d, offsets, b)
        check_dgrad(a, offsets, b.transpose(1, 2).contiguous())
        check_wgrad(d, a, offsets, 3)
