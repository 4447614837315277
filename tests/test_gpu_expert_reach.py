"""The expert side where its other tests do not reach: buffers whose offsets pass
32 bits in every operator and kernel, the same bits from the plain product's two
tile heights, a CU-masked stream under the fused product, and the gradient of
the rows as a product with transposed weights."""

import pytest
import torch

import bulk_async_tensor_amd as ep

import expert_ref as ref
from gpu_helpers import DEV
from test_gpu_expert import bits, check_gemm, check_swiglu, gen, operands, same

pytestmark = pytest.mark.gpu

F8, BF16 = torch.float8_e4m3fn, torch.bfloat16


def zeros8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8, device=DEV).view(F8)


# ------------------------------------------------------------------ past 4 GiB
# With 72 experts of 64 MiB, rows of expert 70.  Plain: the few-row kernel, tiles of 128, and (K past 16384) the kernel
# for long rows; fused: tiles of 32, of 64 and of 128.
@pytest.mark.parametrize("rows, K", [(8, 16384), (40, 16384), (40, 16400), (1200, 16384), (6000, 16384)])
def test_weights_past_four_gigabytes(rows, K):
    N, E = 4096, 72
    b = zeros8(E, N, K)
    b[70] = (torch.randn(N, K, generator=gen(1), device=DEV) * 100).clamp(-448, 448).to(F8)
    sb = torch.full((E, N // 128, ref.blocks(K)), 1e-3, device=DEV)
    a, sa = ref.random_rows(rows, K, 2, DEV)
    sa *= 1e-2
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[71:] = rows - 1
    check_gemm(offsets, a, sa, b, sb)
    check_swiglu(offsets, a, sa, b, sb)


@pytest.mark.parametrize("K, I", [(16384, 512), (256, 16384)])
def test_fused_product_past_four_gigabytes(K, I):
    """Rows (4.6 GB) and outputs (4.6 GB) whose byte offsets pass 32 bits."""
    rows, last = 280000, 40
    lo = rows - last
    a, sa = zeros8(rows, K), torch.full((rows, ref.blocks(K)), 1e-2, device=DEV)
    a[lo:], sa[lo:] = ref.random_rows(last, K, 2, DEV)
    b, sb = ref.random_weights(2, 2 * I, K, 3, DEV)
    offsets = torch.tensor([lo, lo + 17, rows - 3], dtype=torch.int32, device=DEV)
    q = torch.full((rows, I), 0x33, dtype=torch.uint8, device=DEV).view(F8)
    s = torch.full((rows, ref.blocks(I)), -7.0, device=DEV)
    ep.ep_grouped_swiglu_fp8(a, sa, offsets, b, sb, q, s)
    wq, ws = check_swiglu(offsets - lo, a[lo:], sa[lo:], b, sb)
    same(q[lo:], wq)
    same(s[lo:], ws)
    assert bool((bits(q)[:lo] == 0x33).all()) and bool((s[:lo] == -7).all())


def test_row_movers_past_four_gigabytes():
    """The 8-bit dispatch and both gradients on 4.9 GB of rows: the first and the
    last tokens, whose destinations are the last and the first rows."""
    T, H, k, n = 300000, 8192, 2, 64
    ends = torch.cat([torch.arange(n), torch.arange(T - n, T)]).to(DEV)
    dest = torch.arange(T * k, dtype=torch.int32, device=DEV).flip(0).view(T, k).contiguous()
    x = torch.zeros(T, H, dtype=BF16, device=DEV)
    x[ends] = torch.randn(2 * n, H, generator=gen(1), device=DEV).to(BF16)
    q, s = zeros8(T * k, H), torch.zeros(T * k, H // 128, device=DEV)
    ep.ep_dispatch_fp8(x, dest, q, s)
    xq, xs = ref.quantise(x[ends])
    at = dest[ends].long()
    for j in range(k):
        same(q.view(torch.uint8)[at[:, j]], xq.view(torch.uint8))
        same(s[at[:, j]], xs)
    del q, s, xq

    w = torch.rand(T, k, generator=gen(2), device=DEV)
    y = torch.zeros(T * k, H, dtype=BF16, device=DEV)  # 9.8 GB
    y[at.view(-1)] = torch.randn(2 * n * k, H, generator=gen(3), device=DEV).to(BF16)
    dx = torch.zeros_like(x)
    ep.ep_dispatch_backward(y, dest, dx)
    few = torch.arange(2 * n * k, dtype=torch.int32, device=DEV).view(2 * n, k)
    want = torch.zeros(2 * n, H, dtype=BF16, device=DEV)
    rows = y[at.view(-1)]
    same(ep.ep_dispatch_backward(rows, few, want), dx[ends])
    exact = ref.dispatch_backward(rows, few)
    mag = ref.dispatch_backward(rows.abs(), few)
    assert bool(((want.double() - exact).abs() <= ref.UBF16 * exact.abs() + 1.01 * k * ref.U32 * mag).all())
    assert int(dx.count_nonzero()) == int(want.count_nonzero())
    del dx
    dy, dw = torch.zeros_like(y), torch.full_like(w, 5.0)
    ep.ep_combine_backward(x, y, dest, w, dy, dw)
    same(dy[at.view(-1)], (w[ends][:, :, None] * x[ends].float()[:, None, :]).to(BF16).view(-1, H))
    _, edw = ref.combine_backward(x[ends], rows, few, w[ends])
    dots = (x[ends].double().abs()[:, None, :] * rows.double().abs().view(2 * n, k, H)).sum(2)
    assert bool(((dw[ends].double() - edw).abs() <= (H // 64 + 72) * ref.U32 * dots).all())
    assert int(dw.count_nonzero()) == int(dw[ends].count_nonzero())


# ------------------------------------------------------------------ bits
@pytest.mark.parametrize("K", [912, 1024, 1040])
def test_bits_do_not_depend_on_the_tile_height(K):
    """1500 rows take tiles of 128 (one round either way), 16384 rows tiles of
    256: the first 1500 rows have the same bits, odd segments and a last block
    that is not full among them."""
    E, N = 4, 2304
    a, sa = ref.random_rows(16384, K, 1, DEV)
    b, sb = ref.random_weights(E, N, K, 2, DEV)
    offsets = torch.tensor([3, 200, 201, 900, 1500], dtype=torch.int32, device=DEV)
    y, z = torch.zeros(1500, N, dtype=BF16, device=DEV), torch.zeros(16384, N, dtype=BF16, device=DEV)
    ep.ep_grouped_gemm_fp8(a[:1500], sa[:1500], offsets, b, sb, y)
    ep.ep_grouped_gemm_fp8(a, sa, offsets, b, sb, z)
    same(z[:1500], y)
    assert not bool(z[1500:].any()) and not bool(y[:3].any())


# ------------------------------------------------------------------ streams
@pytest.mark.parametrize("cus", [8, 24, 200])
def test_products_on_a_masked_stream(cus):
    offsets, _, a, sa, b, sb = operands(700, 12, 3, 656, 1280, 0.1, 1)
    want = check_gemm(offsets, a, sa, b, sb), *check_swiglu(offsets, a, sa, b, sb)
    rows = a.shape[0]
    y = torch.full((rows, 1280), 77.0, dtype=BF16, device=DEV)
    q = torch.full((rows, 640), 0x33, dtype=torch.uint8, device=DEV).view(F8)
    s = torch.full((rows, 5), -7.0, device=DEV)
    torch.cuda.synchronize()
    stream = ep.ep_stream_create_cu_masked(ep.cu_mask_words(range(cus)))
    try:
        ep.ep_grouped_gemm_fp8(a, sa, offsets, b, sb, y, stream=stream)
        ep.ep_grouped_swiglu_fp8(a, sa, offsets, b, sb, q, s, stream=stream)
        torch.cuda.synchronize()
    finally:
        ep.ep_stream_destroy(stream)
    for u, v in zip((y, q, s), want):
        same(u, v)


# ------------------------------------------------------------------ the gradient of the rows
def test_gradient_of_the_rows_by_transposed_weights():
    """<y, g> changes along a direction of `a` as the product of g with the
    weights stored transposed says."""
    T, E, k, K, N = 60, 5, 2, 272, 400
    offsets, _, a, sa, b, sb = operands(T, E, k, K, N, 0.1, 3)
    rows, total = T * k, int(offsets[-1])
    g, sg = ref.random_rows(rows, N, 7, DEV)
    bt = b.view(torch.uint8).transpose(1, 2).contiguous().view(F8)
    sbt = sb.transpose(1, 2).contiguous()
    da = torch.zeros(rows, K, dtype=BF16, device=DEV)
    ep.ep_grouped_gemm_fp8(g, sg, offsets, bt, sbt, da)

    whole = lambda q, s: q.double() * s.double().repeat_interleave(128, 1)[:, : q.shape[1]]  # noqa: E731
    w = b.double() * sb.double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    expert = torch.searchsorted(offsets[1:].contiguous(), torch.arange(total, dtype=torch.int32, device=DEV), right=True)
    gd = whole(g, sg)[:total]

    def value(rows64):  # <y, g> of float64 rows
        out = torch.stack([w[int(e)] @ rows64[r] for r, e in enumerate(expert)])
        return (out * gd).sum()

    x = whole(a, sa)[:total]
    v = torch.randn(total, K, generator=gen(9), device=DEV, dtype=torch.float64)
    slope = float((value(x + v) - value(x - v)) / 2)  # linear in the rows: exact but for rounding
    mag = torch.stack([w[int(e)].abs().t() @ gd[r].abs() for r, e in enumerate(expert)])
    exact = torch.stack([w[int(e)].t() @ gd[r] for r, e in enumerate(expert)])
    # each value is rounded to bf16 and its sums lose at most 7 * 2^-10 of their terms (see the 8-bit instruction's rule)
    limit = ((ref.UBF16 * exact.abs() + 1.01 * (7 * 2.0 ** -10 + (ref.blocks(N) + 3) * ref.U32) * mag) * v.abs()).sum()
    assert abs(float((da[:total].double() * v).sum()) - slope) <= float(limit)
    err = (da[:total].double() - exact).norm() / exact.norm()
    assert float(err) <= ref.RMS_BF16
