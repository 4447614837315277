"""The expert side on the GPU: the 8-bit dispatch, the experts' 8-bit products
and the gradients of combine and dispatch against plain implementations in 64
bits (expert_ref.py, whose bounds the tolerances are), and runs of them
together."""

import pytest
import torch

import bulk_async_tensor_amd as ep

import expert_ref as ref
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

F8, BF16 = torch.float8_e4m3fn, torch.bfloat16
NAN8 = 0x7F


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def bf16_rows(rows, n, seed):
    return (torch.randn(rows, n, generator=gen(seed), device=DEV) * 2).to(BF16)


def bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def same(a, b):
    assert a.shape == b.shape and torch.equal(bits(a), bits(b)), f"{int((bits(a) != bits(b)).sum())} values differ"


def lay(T, E, k, seed, drop=0.0):
    ids = ref.routing(T, E, k, seed, drop, DEV)
    out = ep.ep_layout(ids, E)
    return out["offsets"], out["dest_row"]


# ------------------------------------------------------------------ 8-bit dispatch
@pytest.mark.parametrize("T, H, E, k, drop", [
    (1, 16, 4, 1, 0), (1, 7168, 8, 8, 0), (3, 112, 4, 2, 0.3), (7, 128, 8, 3, 0), (65, 1040, 16, 5, 0.2),
    (128, 2048, 32, 8, 0), (33, 4112, 9, 9, 0), (257, 7168, 64, 6, 0.1), (40, 8208, 8, 4, 0), (6, 20480, 40, 32, 0),
    (2100, 512, 16, 2, 0), (1000, 7168, 64, 8, 0.05), (4099, 1024, 8, 1, 0), (2050, 3584, 16, 7, 0),
])
def test_dispatch_fp8(T, H, E, k, drop):
    _, dest = lay(T, E, k, T + H, drop)
    x = bf16_rows(T, H, H)
    x[0, :] = 0
    rows = T * k
    q = torch.full((rows, H), 0x11, dtype=torch.uint8, device=DEV).view(F8)
    s = torch.full((rows, ref.blocks(H)), -7.0, device=DEV)
    ep.ep_dispatch_fp8(x, dest, q, s)
    xq, xs = ref.quantise(x)
    eq, es = torch.full((rows, H), 0x11, dtype=torch.uint8, device=DEV).view(F8), torch.full_like(s, -7.0)
    t, _, r = ref._valid(dest, rows)
    bits(eq)[r] = bits(xq)[t]
    es[r] = xs[t]
    same(q, eq)
    same(s, es)


def test_dispatch_fp8_special_values():
    """Tiny blocks, the largest values, infinities and NaN."""
    H = 128 * 7
    x = torch.zeros(2, H, device=DEV)
    x[0, 128:256] = 2.0 ** -120
    x[0, 256:384] = torch.linspace(-1, 1, 128, device=DEV) * 3.38e38
    x[0, 400] = float("nan")
    x[0, 401] = 3.0
    x[0, 600], x[0, 601] = float("inf"), 1.0
    x[0, 700] = float("-inf")
    x[0, 800:820] = float("nan")
    x[1] = torch.randn(H, generator=gen(1), device=DEV) * 1e-30
    x = x.to(BF16)
    dest = torch.tensor([[1], [0]], dtype=torch.int32, device=DEV)
    q = torch.zeros(2, H, dtype=torch.uint8, device=DEV).view(F8)
    s = torch.zeros(2, 7, device=DEV)
    ep.ep_dispatch_fp8(x, dest, q, s)
    xq, xs = ref.quantise(x)
    assert torch.equal(torch.isnan(q.float()), torch.isnan(xq.float()[[1, 0]]))
    keep = ~torch.isnan(q.float())
    assert torch.equal(q.float()[keep], xq.float()[[1, 0]][keep])
    same(s, xs[[1, 0]].contiguous())
    back = q.float() * s.repeat_interleave(128, 1)
    assert torch.isfinite(back[0]).all() and torch.isfinite(back[1, :400]).all()
    assert torch.isnan(back[1, 400]) and float(back[1, 401]) == 3.0
    assert torch.isnan(back[1, 512:768]).all()  # the blocks that hold an infinity


# ------------------------------------------------------------------ expert products
def operands(T, E, k, K, N, drop, seed):
    offsets, dest = lay(T, E, k, seed, drop)
    a, sa = ref.random_rows(T * k, K, seed + 1, DEV)
    b, sb = ref.random_weights(E, N, K, seed + 2, DEV)
    return offsets, dest, a, sa, b, sb


def held(offsets):
    return int(offsets[0]), int(offsets[-1])


def check_gemm(offsets, a, sa, b, sb):
    rows, N = a.shape[0], b.shape[1]
    p, bound = ref.product(a, sa, offsets, b, sb, eight_bit=True)
    y = torch.full((rows, N), 77.0, dtype=BF16, device=DEV)
    assert ep.ep_grouped_gemm_fp8(a, sa, offsets, b, sb, y) is y
    lo, hi = held(offsets)
    err = (y[lo:hi].double() - p[lo:hi]).abs()
    limit = ref.UBF16 * p[lo:hi].abs() + 1.01 * bound[lo:hi]
    assert bool((err <= limit).all()), f"off by up to {float((err / limit).max()):.3f} of the bound"
    if err.numel() > 4000:  # enough for a mean
        assert float(err.norm() / p[lo:hi].norm()) <= ref.RMS_BF16
    assert bool((y[:lo] == 77).all()) and bool((y[hi:] == 77).all())
    return y


def check_swiglu(offsets, a, sa, b, sb):
    rows, I = a.shape[0], b.shape[1] // 2
    h, bound = ref.swiglu(*ref.product(a, sa, offsets, b, sb))
    q = torch.full((rows, I), 0x33, dtype=torch.uint8, device=DEV).view(F8)
    s = torch.full((rows, ref.blocks(I)), -7.0, device=DEV)
    ep.ep_grouped_swiglu_fp8(a, sa, offsets, b, sb, q, s)
    lo, hi = held(offsets)
    for c in range(ref.blocks(I)):
        cols = slice(c * 128, min(I, (c + 1) * 128))
        e, tol = h[lo:hi, cols], bound[lo:hi, cols]
        es = e.abs().amax(1).clamp_min(ref.AMAX_FLOOR) / 448 if hi > lo else e.sum(1)
        got = s[lo:hi, c].double()
        assert bool(((got - es).abs() <= tol.amax(1) / 448 + 2 * ref.U32 * es).all()) if hi > lo else True
        back = q[lo:hi, cols].double() * got[:, None]
        limit = ref.UE4M3 * e.abs() + ref.E4M3_SUB * got[:, None] + 1.1 * tol
        assert bool(((back - e).abs() <= limit).all()), c
    assert bool((bits(q)[:lo] == 0x33).all()) and bool((bits(q)[hi:] == 0x33).all())
    assert bool((s[:lo] == -7).all()) and bool((s[hi:] == -7).all())
    return q, s


SIZES = [  # T, E, k, K, drop: rows per expert from one to thousands, blocks of 16 to 128 at the end
    (1, 8, 8, 16, 0), (1, 64, 1, 1024, 0), (2, 3, 3, 112, 0), (5, 300, 2, 272, 0.3), (16, 4, 1, 144, 0),
    (63, 1, 1, 128, 0), (64, 1, 1, 256, 0), (65, 2, 1, 2064, 0.1), (130, 5, 2, 640, 0), (300, 7, 3, 1488, 0.1),
    (700, 3, 2, 384, 0), (1024, 4, 4, 896, 0), (3000, 2, 1, 400, 0), (2500, 5, 2, 1152, 0.05),
    (40, 1024, 8, 128, 0), (2048, 128, 8, 256, 0),
]


@pytest.mark.parametrize("N", [8, 328, 1024])
@pytest.mark.parametrize("T, E, k, K, drop", SIZES)
def test_grouped_gemm(T, E, k, K, drop, N):
    offsets, _, a, sa, b, sb = operands(T, E, k, K, N, drop, T + K)
    check_gemm(offsets, a, sa, b, sb)


@pytest.mark.parametrize("I", [64, 320, 512])
@pytest.mark.parametrize("T, E, k, K, drop", SIZES)
def test_grouped_swiglu(T, E, k, K, drop, I):
    offsets, _, a, sa, b, sb = operands(T, E, k, K, 2 * I, drop, T + K)
    check_swiglu(offsets, a, sa, b, sb)


# rows of each expert: none at either end, single rows, one expert with nearly all, edges of the row tiles
COUNTS = [[0, 0, 0], [0, 1, 0, 0, 1], [700, 0, 1, 2], [0, 0, 513], [16, 17, 15, 0, 31, 32, 33, 64, 63, 65],
          [128, 127, 129, 255, 256, 257], [1, 0, 2000, 0, 3]]


@pytest.mark.parametrize("counts", COUNTS)
def test_products_of_uneven_experts(counts):
    rows = sum(counts) + 5
    offsets = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    a, sa = ref.random_rows(rows, 528, 3, DEV)
    b, sb = ref.random_weights(len(counts), 640, 528, 4, DEV)
    # rows that no expert holds may be anything
    bits(a)[sum(counts):] = NAN8
    sa[sum(counts):] = float("nan")
    check_gemm(offsets, a, sa, b, sb)
    check_swiglu(offsets, a, sa, b, sb)


# Calls whose workgroups go through several tiles each, at every tile height and at few, odd and many steps a tile:
# T, E, k, K, N (swiglu: about N / 4 outputs, half a tile past whole ones).
STREAMS = [(1500, 512, 4, 256, 2304), (1500, 512, 4, 528, 2304), (1500, 512, 4, 1168, 2304), (1500, 150, 4, 272, 2304),
           (1500, 150, 4, 640, 2304), (1500, 150, 4, 1280, 2304), (4096, 4, 4, 272, 2304), (4096, 4, 4, 384, 2304),
           (4096, 4, 4, 1040, 2304), (2100, 12, 4, 400, 4352), (2100, 12, 4, 1152, 4352), (4096, 4, 4, 256, 2304),
           (2100, 12, 4, 208, 4352), (3000, 8, 2, 144, 4352)]


@pytest.mark.parametrize("T, E, k, K, N", STREAMS)
def test_streams_of_tiles(T, E, k, K, N):
    offsets, _, a, sa, b, sb = operands(T, E, k, K, N, 0.05, T + K)
    check_gemm(offsets, a, sa, b, sb)
    I = N // 4 // 128 * 128 + 64
    check_swiglu(offsets, a, sa, b[:, : 2 * I].contiguous(), sb[:, : ref.blocks(2 * I)].contiguous())


# A few rows against a few experts: T, E, k, K, N, with a step more, less and exactly the blocks that are read ahead.
FEW = [(1, 8, 8, 272, 8), (1, 64, 8, 1024, 328), (1, 64, 8, 1040, 1024), (2, 16, 4, 7168, 2048), (3, 9, 5, 896, 40),
       (1, 1, 1, 2048, 4096), (20, 16, 2, 2064, 1000), (40, 16, 2, 1152, 1024), (1, 64, 8, 16384, 520),
       (128, 64, 4, 640, 264), (5, 1024, 8, 912, 72)]


@pytest.mark.parametrize("T, E, k, K, N", FEW)
def test_few_rows(T, E, k, K, N):
    offsets, _, a, sa, b, sb = operands(T, E, k, K, N, 0, T + K)
    check_gemm(offsets, a, sa, b, sb)
    if T * k > 2:  # a NaN in a row's last value, one in a scale and one in a weight reach no other result
        bits(a)[0, K - 1] = NAN8
        sa[1, 0] = float("nan")
        bits(b)[:, 3, K - 16] = NAN8
        y = torch.zeros(T * k, N, dtype=BF16, device=DEV)
        ep.ep_grouped_gemm_fp8(a, sa, offsets, b, sb, y)
        want = torch.zeros(T * k, N, dtype=torch.bool, device=DEV)
        want[:2] = True
        want[:, 3] = True
        assert torch.equal(torch.isnan(y), want)


def test_few_rows_of_one_expert():
    """Many tiles of 16 rows for one of many experts, and none for the others."""
    rows, E, K, N = 100, 20, 1296, 520
    a, sa = ref.random_rows(rows + 4, K, 1, DEV)
    b, sb = ref.random_weights(E, N, K, 2, DEV)
    offsets = torch.tensor([0] * 7 + [rows] * 14, dtype=torch.int32, device=DEV)
    check_gemm(offsets, a, sa, b, sb)


@pytest.mark.parametrize("K", [16384, 16400, 20000])
def test_long_rows(K):
    offsets, _, a, sa, b, sb = operands(70, 3, 2, K, 384, 0, K)
    check_gemm(offsets, a, sa, b, sb)
    check_swiglu(offsets, a, sa, b, sb)


def test_equal_calls_give_equal_bits():
    offsets, _, a, sa, b, sb = operands(500, 6, 3, 912, 1280, 0, 1)
    first = check_gemm(offsets, a, sa, b, sb), *check_swiglu(offsets, a, sa, b, sb)
    for _ in range(3):
        again = check_gemm(offsets, a, sa, b, sb), *check_swiglu(offsets, a, sa, b, sb)
        for u, v in zip(first, again):
            same(u, v)


@pytest.mark.parametrize("K", [208, 912, 1024])
def test_bits_do_not_depend_on_the_buffer(K):
    """The kernel is chosen by the rows of the buffer; each takes the same sums
    in the same order, so the rows that are held keep their bits."""
    E, N, held_rows = 16, 384, 40
    a, sa = ref.random_rows(6000, K, 1, DEV)
    b, sb = ref.random_weights(E, N, K, 2, DEV)
    ends = torch.arange(E + 1, device=DEV) * held_rows // E
    out = []
    for rows in (held_rows, 300, 1000, 6000):
        y = torch.zeros(rows, N, dtype=BF16, device=DEV)
        q, s = torch.zeros(rows, N // 2, dtype=torch.uint8, device=DEV).view(F8), torch.zeros(rows, 2, device=DEV)
        off = ends.to(torch.int32)
        ep.ep_grouped_gemm_fp8(a[:rows], sa[:rows], off, b, sb, y)
        ep.ep_grouped_swiglu_fp8(a[:rows], sa[:rows], off, b, sb, q, s)
        out.append((y[:held_rows], q[:held_rows], s[:held_rows]))
    for other in out[1:]:
        for u, v in zip(out[0], other):
            same(u, v)


@pytest.mark.parametrize("K, E, counts", [(112, 3, [70, 1, 329]), (272, 3, [70, 1, 329]), (656, 3, [70, 1, 329]),
                                          (656, 9, [20, 30, 50, 1, 0, 70, 40, 60, 80]),
                                          (656, 20, [11, 1, 28] + [10] * 17)])
def test_swiglu_does_not_mix_rows_or_experts(K, E, counts):
    """As below; a NaN of h leaves the rest of its block of 128 as it is."""
    rows, I = sum(counts), 192
    offsets = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    a, sa = ref.random_rows(rows, K, 5, DEV)
    b, sb = ref.random_weights(E, 2 * I, K, 6, DEV)

    def run():
        q, s = torch.zeros(rows, I, dtype=torch.uint8, device=DEV).view(F8), torch.zeros(rows, 2, device=DEV)
        return ep.ep_grouped_swiglu_fp8(a, sa, offsets, b, sb, q, s)

    q, s = run()
    assert not bool(torch.isnan(q.float()).any())
    bits(a)[10, K - 1] = NAN8
    sa[rows - 2, 0] = float("nan")
    bits(b)[2, 100, 0] = NAN8          # gate of output 100
    bits(b)[2, I + 150, K - 16] = NAN8  # up of output 150
    nq, ns = run()
    bad = torch.isnan(nq.float())
    want = torch.zeros_like(bad)
    lo, hi = int(offsets[2]), int(offsets[3])
    want[10] = want[rows - 2] = True
    want[lo:hi, 100] = want[lo:hi, 150] = True
    assert torch.equal(bad, want)
    touched = torch.zeros(rows, 2, dtype=torch.bool, device=DEV)
    touched[10] = touched[rows - 2] = True
    touched[lo:hi] = True
    assert torch.equal(bits(ns)[~touched], bits(s)[~touched])
    rest = ~touched.repeat_interleave(128, 1)[:, :I]
    assert torch.equal(bits(nq)[rest], bits(q)[rest])


def test_products_do_not_mix_rows_or_experts():
    """A NaN in a row reaches that row only, a NaN in a weight row that output
    only, and a NaN scale its blocks."""
    offsets = torch.tensor([0, 70, 71, 400], dtype=torch.int32, device=DEV)
    a, sa = ref.random_rows(400, 272, 5, DEV)
    b, sb = ref.random_weights(3, 384, 272, 6, DEV)
    bits(a)[10, 271] = NAN8
    sa[300, 1] = float("inf")
    sa[300, 0] = float("nan")
    bits(b)[2, 100, 0] = NAN8
    y = torch.zeros(400, 384, dtype=BF16, device=DEV)
    ep.ep_grouped_gemm_fp8(a, sa, offsets, b, sb, y)
    bad = torch.isnan(y)
    want = torch.zeros_like(bad)
    want[10] = True
    want[300] = True
    want[71:, 100] = True
    assert torch.equal(bad, want)


def test_offsets_are_clamped():
    """Offsets outside [0, rows] or decreasing reach no other memory: rows
    outside stay as they are, rows inside are computed or left."""
    a, sa = ref.random_rows(90, 256, 7, DEV)
    b, sb = ref.random_weights(3, 128, 256, 8, DEV)
    for off in ([-50, 20, 60, 4000], [30, 10, 2000000000, -2000000000]):
        offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
        guard = torch.full((94, 128), 5.0, dtype=BF16, device=DEV)
        ep.ep_grouped_gemm_fp8(a, sa, offsets, b, sb, guard[2:92])
        q = torch.full((94, 64), 0x22, dtype=torch.uint8, device=DEV)
        s = torch.full((94, 1), 5.0, device=DEV)
        ep.ep_grouped_swiglu_fp8(a, sa, offsets, b, sb, q[2:92].view(F8), s[2:92])
        torch.cuda.synchronize()
        for t, v in ((guard, 5), (q, 0x22), (s, 5)):
            assert bool((t[:2] == v).all()) and bool((t[92:] == v).all())
    whole = torch.tensor([-50, 20, 60, 4000], dtype=torch.int32, device=DEV)
    y = torch.zeros(90, 128, dtype=BF16, device=DEV)
    z = torch.zeros(90, 128, dtype=BF16, device=DEV)
    ep.ep_grouped_gemm_fp8(a, sa, whole, b, sb, y)
    ep.ep_grouped_gemm_fp8(a, sa, torch.tensor([0, 20, 60, 90], dtype=torch.int32, device=DEV), b, sb, z)
    same(y, z)


def test_products_past_four_gigabytes():
    """Weights and rows whose byte offsets pass 32 bits."""
    K, N, E = 16384, 4096, 72  # 64 MiB an expert, 4.5 GiB
    b = torch.zeros(E, N, K, dtype=torch.uint8, device=DEV).view(F8)
    b[70] = (torch.randn(N, K, generator=gen(1), device=DEV) * 100).clamp(-448, 448).to(F8)
    sb = torch.full((E, N // 128, K // 128), 1e-3, device=DEV)
    rows = 280000  # 4.3 GiB
    a = torch.zeros(rows, K, dtype=torch.uint8, device=DEV).view(F8)
    sa = torch.full((rows, K // 128), 0.01, device=DEV)
    a[-40:] = (torch.randn(40, K, generator=gen(2), device=DEV) * 100).clamp(-448, 448).to(F8)
    offsets = torch.full((E + 1,), rows - 40, dtype=torch.int32, device=DEV)
    offsets[71:] = rows - 3
    y = torch.full((rows, N), 9.0, dtype=BF16, device=DEV)
    ep.ep_grouped_gemm_fp8(a, sa, offsets, b, sb, y)
    lo = rows - 40
    p, bound = ref.product(a[lo:], sa[lo:], (offsets - lo)[70:72].contiguous(), b[70:71], sb[70:71], eight_bit=True)
    err = (y[lo : rows - 3].double() - p[:37]).abs()
    assert bool((err <= ref.UBF16 * p[:37].abs() + 1.01 * bound[:37]).all())
    assert bool((y[:lo] == 9).all()) and bool((y[rows - 3 :] == 9).all())


# ------------------------------------------------------------------ gradients
GRADS = [  # T, H, E, k, drop
    (1, 8, 4, 1, 0), (1, 7168, 8, 8, 0), (3, 520, 4, 2, 0.4), (17, 1024, 8, 3, 0), (128, 1024, 8, 2, 0),
    (65, 1144, 41, 5, 0.1), (40, 4096, 16, 4, 0), (200, 7168, 64, 6, 0.1), (64, 8192, 16, 8, 0), (9, 16392, 16, 7, 0),
    (5, 30000, 64, 32, 0.1), (2049, 512, 16, 8, 0), (1500, 7168, 32, 8, 0.02), (3001, 2888, 61, 3, 0.1),
    (4100, 2048, 8, 1, 0.5), (2000, 5000, 32, 12, 0),
]


@pytest.mark.parametrize("T, H, E, k, drop", GRADS)
def test_combine_backward(T, H, E, k, drop):
    _, dest = lay(T, E, k, T + H, drop)
    rows = T * k + 3
    dout, y = bf16_rows(T, H, 1), bf16_rows(rows, H, 2)
    w = torch.randn(T, k, generator=gen(3), device=DEV)
    dy = torch.full((rows, H), 55.0, dtype=BF16, device=DEV)
    dw = torch.full((T, k), 55.0, device=DEV)
    ep.ep_combine_backward(dout, y, dest, w, dy, dw)
    t, j, r = ref._valid(dest, rows)
    want = torch.full_like(dy, 55.0)
    want[r] = (w[t, j][:, None] * dout[t].float()).to(BF16)  # one float32 product, one rounding: exact
    same(dy, want)
    _, edw = ref.combine_backward(dout, y, dest, w)
    mag = torch.zeros_like(edw)
    mag[t, j] = (dout[t].double() * y[r].double()).abs().sum(1)
    # products of bf16 are exact in float32; the longest chain is a lane's share and the joining of 64 lanes
    assert bool(((dw.double() - edw).abs() <= (-(-H // 64) + 72) * ref.U32 * mag).all())
    # either gradient alone is the same one
    dy1, dw1 = torch.full_like(dy, 55.0), torch.full_like(dw, 55.0)
    ep.ep_combine_backward(dout, None, dest, w, dy1, None)
    ep.ep_combine_backward(dout, y, dest, None, None, dw1)
    same(dy1, dy)
    same(dw1, dw)


@pytest.mark.parametrize("T, H, E, k, drop", GRADS)
def test_dispatch_backward(T, H, E, k, drop):
    _, dest = lay(T, E, k, T + H, drop)
    rows = T * k
    drecv = bf16_rows(rows, H, 2)
    t, _, r = ref._valid(dest, rows)
    unused = torch.ones(rows, dtype=torch.bool, device=DEV)
    unused[r] = False
    drecv[unused] = float("nan")  # rows of dropped entries are not read
    dx = torch.full((T, H), 55.0, dtype=BF16, device=DEV)
    assert ep.ep_dispatch_backward(drecv, dest, dx) is dx
    exact = ref.dispatch_backward(torch.where(unused[:, None], 0.0, drecv.double()), dest)
    mag = ref.dispatch_backward(torch.where(unused[:, None], 0.0, drecv.double().abs()), dest)
    assert bool(((dx.double() - exact).abs() <= ref.UBF16 * exact.abs() + 1.01 * k * ref.U32 * mag).all())
    out = torch.empty_like(dx)
    same(ep.ep_combine(drecv, dest, torch.ones(T, k, device=DEV), out), dx)


def test_gradients_of_nothing():
    """No receive rows, and destinations outside the buffer."""
    dest = torch.tensor([[0, 9], [-1, 1 << 30]], dtype=torch.int32, device=DEV)
    none = torch.zeros(0, 64, dtype=BF16, device=DEV)
    dout, w = bf16_rows(2, 64, 1), torch.ones(2, 2, device=DEV)
    dw = torch.full((2, 2), 5.0, device=DEV)
    dx = torch.full((2, 64), 5.0, dtype=BF16, device=DEV)
    ep.ep_combine_backward(dout, none, dest, w, none, dw)
    ep.ep_dispatch_backward(none, dest, dx)
    assert bool((dw == 0).all()) and bool((dx == 0).all())
    y = bf16_rows(3, 64, 2)
    dy = torch.full_like(y, 5.0)
    ep.ep_combine_backward(dout, y, dest, w, dy, dw)
    assert bool((dw[0, 1] == 0) & (dw[1] == 0).all()) and bool((dy[1:] == 5).all())
    same(dy[:1], dout[:1])


def test_gradients_of_infinite_rows():
    dest = torch.tensor([[0, 1]], dtype=torch.int32, device=DEV)
    dout, y = bf16_rows(1, 256, 1), bf16_rows(2, 256, 2)
    y[1, 7] = float("inf")
    dout[0, 9] = float("nan")
    dy, dw = torch.zeros_like(y), torch.zeros(1, 2, device=DEV)
    ep.ep_combine_backward(dout, y, dest, torch.ones(1, 2, device=DEV), dy, dw)
    assert bool(torch.isnan(dw).all()) and int(torch.isnan(dy).sum()) == 2
    dx = torch.zeros_like(dout)
    ep.ep_dispatch_backward(y, dest, dx)
    assert bool(torch.isinf(dx[0, 7])) and int(torch.isfinite(dx).sum()) == 255


# ------------------------------------------------------------------ together
def serve(x, ids, w, E, b1, s1, b2, s2, bufs):
    """One expert layer as a serving program runs it."""
    T, k = ids.shape
    lo = ep.ep_layout(ids, E, **bufs["lay"])
    ep.ep_dispatch_fp8(x, lo["dest_row"], bufs["q"], bufs["s"])
    ep.ep_grouped_swiglu_fp8(bufs["q"], bufs["s"], lo["offsets"], b1, s1, bufs["hq"], bufs["hs"])
    ep.ep_grouped_gemm_fp8(bufs["hq"], bufs["hs"], lo["offsets"], b2, s2, bufs["y"])
    return ep.ep_combine(bufs["y"], lo["dest_row"], w, bufs["out"])


def serve_bufs(T, k, E, H, I):
    i32 = dict(dtype=torch.int32, device=DEV)
    R = T * k
    return {"lay": {"counts": torch.zeros(E, **i32), "offsets": torch.zeros(E + 1, **i32),
                    "dest_row": torch.zeros((T, k), **i32), "src_token": torch.zeros(R, **i32),
                    "status": torch.zeros(1, **i32),
                    "workspace": torch.zeros(max(16, ep.ep_layout_workspace_bytes(T, k, E)), dtype=torch.uint8,
                                             device=DEV)},
            "q": torch.zeros(R, H, dtype=torch.uint8, device=DEV).view(F8),
            "s": torch.zeros(R, ref.blocks(H), device=DEV),
            "hq": torch.zeros(R, I, dtype=torch.uint8, device=DEV).view(F8),
            "hs": torch.zeros(R, ref.blocks(I), device=DEV),
            "y": torch.zeros(R, H, dtype=BF16, device=DEV), "out": torch.zeros(T, H, dtype=BF16, device=DEV)}


def serve_exact(x, ids, w, E, b1, s1, b2, s2):
    """The same layer in 64 bits; the two roundings to 8 bits are its own."""
    offsets, dest = ref.layout(ids, E)
    rows = ids.numel()
    q, s = ref.quantise(x)
    t, _, r = ref._valid(dest, rows)
    aq, as_ = torch.zeros(rows, x.shape[1], dtype=torch.uint8, device=DEV), torch.zeros(rows, s.shape[1], device=DEV)
    aq[r] = bits(q)[t]
    as_[r] = s[t]
    h, _ = ref.swiglu(*ref.product(aq.view(F8), as_, offsets, b1, s1))
    hq, hs = ref.quantise(torch.nan_to_num(h))
    y = torch.nan_to_num(ref.product(hq, hs, offsets, b2, s2)[0])
    # A value of h next to a rounding border may take the neighbouring 8-bit value: a whole step, 2 UE4M3 of the value
    # or 2 E4M3_SUB of its scale.  y sums I such values, so it moves by up to that share of the sum of its terms'
    # MAGNITUDES (which cancel in y itself); it is then rounded to bf16, weighted, summed and rounded once more.
    ones = torch.ones(hq.shape, device=DEV).to(F8)
    moved = (2 * ref.UE4M3 * ref.magnitude(hq, hs, offsets, b2, s2)
             + 2 * ref.E4M3_SUB * ref.magnitude(ones, hs, offsets, b2, s2) + ref.UBF16 * y.abs())
    out = ref.combine(y, dest, w)
    return out, 1.01 * (ref.combine(moved, dest, w) + ref.UBF16 * out.abs())


@pytest.mark.parametrize("T, H, I, E, k, drop", [(1, 1024, 256, 8, 2, 0), (33, 512, 320, 16, 4, 0.1),
                                                 (600, 1024, 512, 4, 2, 0)])
def test_serving_layer(T, H, I, E, k, drop):
    ids = ref.routing(T, E, k, 3, drop, DEV)
    x = bf16_rows(T, H, 4)
    w = torch.rand(T, k, generator=gen(5), device=DEV)
    b1, s1 = ref.random_weights(E, 2 * I, H, 6, DEV)
    b2, s2 = ref.random_weights(E, H, I, 7, DEV)
    out = serve(x, ids, w, E, b1, s1, b2, s2, serve_bufs(T, k, E, H, I))
    exact, limit = serve_exact(x, ids, w, E, b1, s1, b2, s2)
    # few values do move: the whole is as near as the two roundings to bf16 leave it
    assert float((out.double() - exact).norm() / exact.norm()) <= 4 * ref.UBF16
    assert bool(((out.double() - exact).abs() <= limit).all())


def test_serving_layer_in_a_graph():
    """Captured once, replayed on new rows and new routing, between eager runs
    of other buffers; every replay against the eager result."""
    T, H, I, E, k = 48, 1024, 256, 16, 4
    x, ids = bf16_rows(T, H, 1), ref.routing(T, E, k, 1, 0, DEV)
    w = torch.rand(T, k, generator=gen(5), device=DEV)
    weights = ref.random_weights(E, 2 * I, H, 6, DEV) + ref.random_weights(E, H, I, 7, DEV)
    bufs, eager = serve_bufs(T, k, E, H, I), serve_bufs(T, k, E, H, I)
    dy, dw = torch.zeros(T * k, H, dtype=BF16, device=DEV), torch.zeros(T, k, device=DEV)
    dx = torch.zeros(T, H, dtype=BF16, device=DEV)

    def step(b, gy, gw, gx):
        out = serve(x, ids, w, E, *weights, b)
        ep.ep_combine_backward(out, b["y"], b["lay"]["dest_row"], w, gy, gw)
        return ep.ep_dispatch_backward(gy, b["lay"]["dest_row"], gx)

    step(bufs, dy, dw, dx)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(bufs, dy, dw, dx)
    for seed in range(4):
        x.copy_(bf16_rows(T, H, seed + 10))
        ids.copy_(ref.routing(T, E, k, seed + 10, 0.1 * (seed % 2), DEV))
        graph.replay()
        torch.cuda.synchronize()
        ey, ew, ex = torch.zeros_like(dy), torch.zeros_like(dw), torch.zeros_like(dx)
        step(eager, ey, ew, ex)
        torch.cuda.synchronize()
        total = int(eager["lay"]["offsets"][-1])
        same(bufs["out"], eager["out"])
        same(dy[:total], ey[:total])
        same(dw, ew)
        same(dx, ex)


def test_training_step_gradients():
    """dispatch, a linear expert and combine forward, and the gradients back:
    against the formulas and against differences of the step in 64 bits."""
    T, H, E, k = 96, 264, 8, 3
    ids = ref.routing(T, E, k, 1, 0.1, DEV)
    lo = ep.ep_layout(ids, E)
    dest, rows = lo["dest_row"], T * k
    x, dout = bf16_rows(T, H, 2), bf16_rows(T, H, 3)
    w = torch.rand(T, k, generator=gen(4), device=DEV)
    scale = 2.0 ** torch.randint(-2, 3, (rows, 1), generator=gen(5), device=DEV)  # exact in bf16
    recv = torch.zeros(rows, H, dtype=BF16, device=DEV)
    ep.ep_dispatch(x, dest, recv)
    y = recv * scale.to(BF16)
    out = torch.empty(T, H, dtype=BF16, device=DEV)
    ep.ep_combine(y, dest, w, out)
    dy, dw = torch.zeros_like(y), torch.zeros_like(w)
    ep.ep_combine_backward(dout, y, dest, w, dy, dw)
    dx = torch.empty_like(x)
    ep.ep_dispatch_backward(dy * scale.to(BF16), dest, dx)

    def loss(xx, ww):
        return (ref.combine(ref.dispatch(xx, dest, rows) * scale.double(), dest, ww) * dout.double()).sum()

    vx = torch.randn(T, H, generator=gen(6), device=DEV, dtype=torch.float64)
    vw = torch.randn(T, k, generator=gen(7), device=DEV, dtype=torch.float64)
    h = 1e-3  # the loss is bilinear: central differences are exact but for rounding
    along_x = float((loss(x.double() + h * vx, w.double()) - loss(x.double() - h * vx, w.double())) / (2 * h))
    along_w = float((loss(x.double(), w.double() + h * vw) - loss(x.double(), w.double() - h * vw)) / (2 * h))
    # dy is rounded to bf16 once and dx once more; dw is a float32 sum
    sx = ref.dispatch_backward(ref.combine_backward(dout, y, dest, w)[0].abs() * scale.double(), dest)
    assert abs(float((dx.double() * vx).sum()) - along_x) <= 2.01 * ref.UBF16 * float((sx * vx.abs()).sum())
    mag = ref.combine_backward(dout.abs(), y.abs(), dest, w)[1]
    assert abs(float((dw.double() * vw).sum()) - along_w) <= 100 * ref.U32 * float((mag * vw.abs()).sum()) + 1e-6


def test_two_streams_at_once():
    """Calls on two streams share nothing."""
    sides = []
    for n in range(2):
        offsets, dest, a, sa, b, sb = operands(300, 8, 2, 512, 512, 0, 10 * n + 1)
        x = bf16_rows(300, 512, n)
        sides.append((offsets, dest, a, sa, b, sb, x, torch.cuda.Stream()))

    def run(side, stream=None):
        offsets, dest, a, sa, b, sb, x, _ = side
        y = torch.zeros(600, 512, dtype=BF16, device=DEV)
        q, s = torch.zeros(600, 256, dtype=torch.uint8, device=DEV).view(F8), torch.zeros(600, 2, device=DEV)
        xq, xs = torch.zeros(600, 512, dtype=torch.uint8, device=DEV).view(F8), torch.zeros(600, 4, device=DEV)
        dy, dw = torch.zeros(600, 512, dtype=BF16, device=DEV), torch.zeros(300, 2, device=DEV)
        dx = torch.zeros(300, 512, dtype=BF16, device=DEV)
        torch.cuda.synchronize()
        return lambda: (ep.ep_grouped_gemm_fp8(a, sa, offsets, b, sb, y, stream=stream),
                        *ep.ep_grouped_swiglu_fp8(a, sa, offsets, b, sb, q, s, stream=stream),
                        *ep.ep_dispatch_fp8(x, dest, xq, xs, stream=stream),
                        *ep.ep_combine_backward(x, y, dest, sa[:300, :2].contiguous(), dy, dw, stream=stream),
                        ep.ep_dispatch_backward(dy, dest, dx, stream=stream))

    alone = [run(s)() for s in sides]
    torch.cuda.synchronize()
    calls = [run(s, s[-1]) for s in sides]
    for _ in range(3):
        both = [c() for c in calls]
    torch.cuda.synchronize()
    for one, two in zip(alone, both):
        for u, v in zip(one, two):
            same(u, v)


@pytest.mark.parametrize("cus", [1, 24, 256])
def test_budget_and_masked_stream(cus):
    """The row movers under a compute-unit budget and on a masked stream."""
    T, H, E, k = 300, 1040, 16, 4
    _, dest = lay(T, E, k, 1, 0.1)
    x, y = bf16_rows(T, H, 1), bf16_rows(T * k, H, 2)
    w = torch.rand(T, k, generator=gen(3), device=DEV)

    def run(stream=None):
        q, s = torch.zeros(T * k, H, dtype=torch.uint8, device=DEV).view(F8), torch.zeros(T * k, 9, device=DEV)
        dy, dw, dx = torch.zeros_like(y), torch.zeros_like(w), torch.zeros_like(x)
        torch.cuda.synchronize()
        ep.ep_dispatch_fp8(x, dest, q, s, stream=stream)
        ep.ep_combine_backward(x, y, dest, w, dy, dw, stream=stream)
        ep.ep_dispatch_backward(y, dest, dx, stream=stream)
        torch.cuda.synchronize()
        return q, s, dy, dw, dx

    want = run()
    try:
        ep.ep_set_num_cus(cus)
        for u, v in zip(run(), want):
            same(u, v)
    finally:
        ep.ep_set_num_cus(0)
    if cus >= 8:
        stream = ep.ep_stream_create_cu_masked(ep.cu_mask_words(range(cus)))
        try:
            for u, v in zip(run(stream), want):
                same(u, v)
            offsets, _, a, sa, b, sb = operands(200, 8, 2, 256, 256, 0, 1)
            y1, y2 = (torch.zeros(400, 256, dtype=BF16, device=DEV) for _ in range(2))
            ep.ep_grouped_gemm_fp8(a, sa, offsets, b, sb, y1)
            torch.cuda.synchronize()
            ep.ep_grouped_gemm_fp8(a, sa, offsets, b, sb, y2, stream=stream)
            torch.cuda.synchronize()
            same(y1, y2)
        finally:
            ep.ep_stream_destroy(stream)


# ------------------------------------------------------------------ refusals of the binding
def test_binding_refusals():
    offsets, dest, a, sa, b, sb = operands(8, 4, 2, 256, 128, 0, 1)
    x, w = bf16_rows(8, 256, 1), torch.ones(8, 2, device=DEV)
    y = torch.zeros(16, 128, dtype=BF16, device=DEV)
    q, s = torch.zeros(16, 64, dtype=torch.uint8, device=DEV).view(F8), torch.zeros(16, 1, device=DEV)
    g = ep.ep_grouped_gemm_fp8
    for call, err in [
        (lambda: g(a.float(), sa, offsets, b, sb, y), TypeError),
        (lambda: g(a, sa.double(), offsets, b, sb, y), TypeError),
        (lambda: g(a, sa, offsets.long(), b, sb, y), TypeError),
        (lambda: g(a, sa, offsets, b, sb, y.float()), TypeError),
        (lambda: g(a.view(torch.uint8).view(torch.float8_e5m2), sa, offsets, b, sb, y), TypeError),
        (lambda: g(a[:, :128], sa, offsets, b, sb, y), ValueError),
        (lambda: g(a, sa[:, :1].contiguous(), offsets, b, sb, y), ValueError),
        (lambda: g(a, sa.t().contiguous().t(), offsets, b, sb, y), ValueError),
        (lambda: g(a, sa, offsets[:4], b, sb, y), ValueError),
        (lambda: g(a, sa, offsets, b[:, :, :128].contiguous(), sb, y), ValueError),
        (lambda: g(a, sa, offsets, b, sb[:, :, :1].contiguous(), y), ValueError),
        (lambda: g(a, sa, offsets, b, sb, y[:15]), ValueError),
        (lambda: ep.ep_grouped_swiglu_fp8(a, sa, offsets, b, sb, q[:, :32].contiguous(), s), ValueError),
        (lambda: ep.ep_grouped_swiglu_fp8(a, sa, offsets, b, sb, q, s[:8]), ValueError),
        (lambda: ep.ep_dispatch_fp8(x.float(), dest, a, sa), TypeError),
        (lambda: ep.ep_dispatch_fp8(x, dest[:4], a, sa), ValueError),
        (lambda: ep.ep_dispatch_fp8(x, dest, a, sa[:, :1].contiguous()), ValueError),
        (lambda: ep.ep_dispatch_backward(x, dest, x[:4]), ValueError),
        (lambda: ep.ep_dispatch_backward(x[:, :128].contiguous(), dest, x), ValueError),
        (lambda: ep.ep_combine_backward(x, x, dest, w, x[:4], None), ValueError),
        (lambda: ep.ep_combine_backward(x, None, dest, w, None, w), ValueError),
        (lambda: ep.ep_combine_backward(x, x, dest, None, x, None), ep.EpError),
        (lambda: ep.ep_combine_backward(x, None, dest, w, x, w), ep.EpError),
        (lambda: ep.ep_combine_backward(x, x, dest, w, None, None), ep.EpError),
        (lambda: g(a.view(torch.uint8).view(-1)[: 4096 - 256].view(-1, 8)[:16].contiguous().view(F8), s, offsets,
                   b.view(torch.uint8)[:, :, :8].contiguous().view(F8), s[:4].view(4, 1, 1).contiguous(), y),
         ep.EpError),
    ]:
        with pytest.raises(err):
            call()


@pytest.mark.parametrize("rows", [9, 100, 127, 300])
def test_one_expert_and_one_tile_of_columns(rows):
    a, sa = ref.random_rows(rows, 656, rows, DEV)
    b, sb = ref.random_weights(1, 248, 656, 2, DEV)
    check_gemm(torch.tensor([0, rows], dtype=torch.int32, device=DEV), a, sa, b, sb)


@pytest.mark.parametrize("K", [144, 272, 384, 400])
@pytest.mark.parametrize("rows, E", [(900, 300), (6000, 150), (1600, 20)])
def test_swiglu_of_short_rows(K, rows, E):
    """Rows of two to four blocks at every tile height, workgroups with several
    tiles, and the same bits from a buffer that takes the tallest tiles."""
    g = torch.Generator().manual_seed(rows + K)
    ends = torch.cat([torch.zeros(1, dtype=torch.int64), torch.randint(0, rows - 3, (E,), generator=g).sort().values])
    offsets = ends.to(torch.int32).to(DEV)
    tall = 90 * E
    a, sa = ref.random_rows(tall, K, 1, DEV)
    b, sb = ref.random_weights(E, 2 * 448, K, 2, DEV)
    q, s = check_swiglu(offsets, a[:rows], sa[:rows], b, sb)
    tq, ts = check_swiglu(offsets, a, sa, b, sb)
    held_rows = int(ends[-1])
    same(tq[:held_rows], q[:held_rows])
    same(ts[:held_rows], s[:held_rows])


@pytest.mark.parametrize("K", [144, 272, 384])
@pytest.mark.parametrize("E, counts", [(9, [20, 30, 50, 1, 0, 70, 40, 60, 80]), (20, [11, 1, 28] + [10] * 17)])
def test_swiglu_of_short_rows_does_not_mix(K, E, counts):
    """A NaN in the last value of a row that ends inside a block, and in weights, at the lower tile heights."""
    test_swiglu_does_not_mix_rows_or_experts(K, E, counts)
