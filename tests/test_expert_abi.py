"""The expert side's C ABI without a GPU: every entry point that
include/ep_expert.h declares is exported and bound, and bad arguments are
rejected on the host before any HIP call."""

import os
import re

import pytest
import torch

import bulk_async_tensor_amd as ep

import expert_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ep_expert.h")

# fake device addresses: only their alignment matters, none is dereferenced
A16 = 0x7F0000000000
A4 = A16 + 4
ODD = A16 + 1


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ep.LIB_PATH):
        pytest.fail("libep.so is not built (run __graft_entry__.build())")
    return ep.lib()


def test_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(ep_\w+)\s*\(", text)))
    assert names == ["ep_combine_backward", "ep_dispatch_backward", "ep_dispatch_fp8", "ep_grouped_gemm_fp8",
                     "ep_grouped_swiglu_fp8"]
    for n in names:
        assert hasattr(lib, n) and n in ep._SIGNATURES and n in ep.__all__, n


def change(args, **over):
    return [over.get(n, v) for n, v in args]


FP8 = [("x", A16), ("T", 4), ("H", 256), ("dest", A4), ("k", 2), ("q", A16), ("s", A4), ("rows", 8), ("stream", None)]


@pytest.mark.parametrize("over, code", [
    (dict(T=-1), -1), (dict(k=0), -1), (dict(k=33), -1), (dict(H=0), -1), (dict(H=-16), -1), (dict(H=264), -1),
    (dict(H=8), -1), (dict(rows=-1), -1), (dict(rows=1 << 31), -1), (dict(T=1 << 30, k=4), -1), (dict(x=None), -1),
    (dict(dest=None), -1), (dict(q=None), -1), (dict(s=None), -1), (dict(x=A16 + 8), -2), (dict(q=A16 + 8), -2),
    (dict(dest=ODD), -2), (dict(s=ODD), -2), (dict(T=0), 0), (dict(rows=0, q=None, s=None), 0),
])
def test_dispatch_fp8_arguments(lib, over, code):
    assert lib.ep_dispatch_fp8(*change(FP8, **over)) == code
    if code:
        assert "ep_dispatch_fp8" in lib.ep_last_error().decode()


GEMM = [("a", A16), ("sa", A4), ("rows", 8), ("K", 256), ("off", A4), ("E", 4), ("b", A16), ("sb", A4), ("N", 64),
        ("y", A16), ("stream", None)]


@pytest.mark.parametrize("over, code", [
    (dict(rows=-1), -1), (dict(rows=1 << 31), -1), (dict(K=0), -1), (dict(K=8), -1), (dict(K=260), -1),
    (dict(N=0), -1), (dict(N=12), -1), (dict(E=0), -1), (dict(E=1025), -1), (dict(N=1 << 16, K=1 << 15), -1),
    (dict(a=None), -1), (dict(sa=None), -1), (dict(off=None), -1), (dict(b=None), -1), (dict(sb=None), -1),
    (dict(y=None), -1), (dict(a=A16 + 8), -2), (dict(b=A16 + 8), -2), (dict(y=A16 + 8), -2), (dict(sa=ODD), -2),
    (dict(sb=ODD), -2), (dict(off=ODD), -2), (dict(rows=0, a=None, sa=None, b=None, sb=None, y=None), 0),
    (dict(rows=0, off=None), -1),
])
def test_grouped_gemm_arguments(lib, over, code):
    assert lib.ep_grouped_gemm_fp8(*change(GEMM, **over)) == code
    if code:
        assert "ep_grouped_gemm_fp8" in lib.ep_last_error().decode()


SWIGLU = [("a", A16), ("sa", A4), ("rows", 8), ("K", 256), ("off", A4), ("E", 4), ("b", A16), ("sb", A4), ("I", 64),
          ("q", A16), ("s", A4), ("stream", None)]


@pytest.mark.parametrize("over, code", [
    (dict(I=0), -1), (dict(I=32), -1), (dict(I=96), -1), (dict(I=-64), -1), (dict(I=(1 << 31) - 64), -1),
    (dict(I=1 << 15, K=1 << 15), -1), (dict(K=24), -1), (dict(E=0), -1), (dict(rows=-1), -1), (dict(q=None), -1),
    (dict(s=None), -1), (dict(q=A16 + 8), -2), (dict(s=ODD), -2), (dict(rows=0, q=None, s=None), 0),
])
def test_grouped_swiglu_arguments(lib, over, code):
    assert lib.ep_grouped_swiglu_fp8(*change(SWIGLU, **over)) == code
    if code:
        assert "ep_grouped_swiglu_fp8" in lib.ep_last_error().decode()


CBWD = [("dout", A16), ("y", A16), ("rows", 8), ("H", 64), ("dest", A4), ("w", A4), ("T", 4), ("k", 2), ("dy", A16),
        ("dw", A4), ("stream", None)]


@pytest.mark.parametrize("over, code", [
    (dict(T=-1), -1), (dict(k=0), -1), (dict(k=33), -1), (dict(H=4), -1), (dict(H=0), -1), (dict(rows=-1), -1),
    (dict(dy=None, dw=None), -1), (dict(dout=None), -1), (dict(dest=None), -1), (dict(w=None), -1),
    (dict(y=None), -1), (dict(dout=A16 + 8), -2), (dict(y=A16 + 8), -2), (dict(dy=A16 + 8), -2),
    (dict(dest=ODD), -2), (dict(w=ODD), -2), (dict(dw=ODD), -2), (dict(T=0), 0), (dict(rows=0, dw=None, y=None), 0),
])
def test_combine_backward_arguments(lib, over, code):
    assert lib.ep_combine_backward(*change(CBWD, **over)) == code
    if code:
        assert "ep_combine_backward" in lib.ep_last_error().decode()


DBWD = [("drecv", A16), ("rows", 8), ("H", 64), ("dest", A4), ("T", 4), ("k", 2), ("dx", A16), ("stream", None)]


@pytest.mark.parametrize("over, code", [
    (dict(T=-1), -1), (dict(k=0), -1), (dict(H=12), -1), (dict(rows=-1), -1), (dict(drecv=None), -1),
    (dict(dest=None), -1), (dict(dx=None), -1), (dict(drecv=A16 + 8), -2), (dict(dx=A4), -2), (dict(dest=ODD), -2),
    (dict(T=0), 0), (dict(T=0, rows=0, drecv=None), 0),
])
def test_dispatch_backward_arguments(lib, over, code):
    assert lib.ep_dispatch_backward(*change(DBWD, **over)) == code
    if code:
        assert "ep_dispatch_backward" in lib.ep_last_error().decode()


def test_binding_refuses_host_tensors():
    """The binding has no fallback: tensors that are not on a GPU are refused."""
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    i = torch.zeros(2, 1, dtype=torch.int32)
    q, s = ref.quantise(x)
    off = torch.tensor([0, 2], dtype=torch.int32)
    for call in (lambda: ep.ep_dispatch_fp8(x, i, q, s), lambda: ep.ep_dispatch_backward(x, i, x),
                 lambda: ep.ep_combine_backward(x, x, i, s, x, s),
                 lambda: ep.ep_grouped_gemm_fp8(q, s, off, q.view(1, 2, 128), s.view(1, 2, 1), x),
                 lambda: ep.ep_grouped_swiglu_fp8(q, s, off, q.view(1, 2, 128), s.view(1, 2, 1), q, s)):
        with pytest.raises(ValueError, match="device"):
            call()


def test_plain_forms_agree_with_each_other():
    """The 64-bit product against a loop over single values, and the gradients'
    formulas against differences of the forward in 64 bits."""
    ids = ref.routing(5, 3, 2, 1, drop=0.2)
    offsets, dest = ref.layout(ids, 3)
    a, sa = ref.random_rows(10, 144, 2, "cpu")
    b, sb = ref.random_weights(3, 24, 144, 3, "cpu")
    p, _ = ref.product(a, sa, offsets, b, sb)
    for e in range(3):
        for r in range(int(offsets[e]), int(offsets[e + 1])):
            for n in (0, 23):
                v = sum(float(a[r, i]) * float(sa[r, i // 128]) * float(b[e, n, i]) * float(sb[e, 0, i // 128])
                        for i in range(144))
                assert abs(v - float(p[r, n])) <= 1e-9 * max(1.0, abs(v))
    assert torch.isnan(p[int(offsets[-1]):]).all()

    g = torch.Generator().manual_seed(4)
    y = torch.randn(10, 16, generator=g, dtype=torch.float64)
    w = torch.randn(5, 2, generator=g, dtype=torch.float64)
    dout = torch.randn(5, 16, generator=g, dtype=torch.float64)
    dy, dw = ref.combine_backward(dout, y, dest, w)
    vy, vw = torch.randn(y.shape, generator=g, dtype=torch.float64), torch.randn(w.shape, generator=g, dtype=torch.float64)
    f = lambda h: float((ref.combine(y + h * vy, dest, w + h * vw) * dout).sum())  # noqa: E731
    slope = (f(1e-4) - f(-1e-4)) / 2e-4  # exact but for rounding: f is quadratic
    assert abs(slope - float((dy * vy).sum() + (dw * vw).sum())) <= 1e-8
    x, vx = torch.randn(5, 16, generator=g, dtype=torch.float64), torch.randn(10, 16, generator=g, dtype=torch.float64)
    dx = ref.dispatch_backward(vx, dest)
    assert abs(float((dx * x).sum()) - float((ref.dispatch(x, dest, 10) * vx).sum())) <= 1e-9


def test_binding_refuses_sizes_past_32_bits(monkeypatch):
    """The C calls take sizes as int: a larger one would arrive cut to its low 32
    bits (2^32 + 4 tokens as 4).  Shapes only, without memory."""
    monkeypatch.setattr(ep, "_operand", lambda t, name, dtype: 0)
    monkeypatch.setattr(ep, "_call_on", lambda *args: pytest.fail("the call went through"))
    f8, bf16, f32, i32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int32

    def t(dtype, *shape):
        return torch.empty(*shape, dtype=dtype, device="meta")

    big = (1 << 32) + 128
    nb = big // 128
    w = t(f32, 4, 2)
    for call in (
        lambda: ep.ep_dispatch_fp8(t(bf16, big, 128), t(i32, big, 2), t(f8, 8, 128), t(f32, 8, 1)),
        lambda: ep.ep_dispatch_fp8(t(bf16, 4, big), t(i32, 4, 2), t(f8, 8, big), t(f32, 8, nb)),
        lambda: ep.ep_dispatch_fp8(t(bf16, 4, 128), t(i32, 4, big), t(f8, 8, 128), t(f32, 8, 1)),
        lambda: ep.ep_grouped_gemm_fp8(t(f8, 8, big), t(f32, 8, nb), t(i32, 3), t(f8, 2, 128, big), t(f32, 2, 1, nb),
                                       t(bf16, 8, 128)),
        lambda: ep.ep_grouped_gemm_fp8(t(f8, 8, 128), t(f32, 8, 1), t(i32, 3), t(f8, 2, big, 128), t(f32, 2, nb, 1),
                                       t(bf16, 8, big)),
        lambda: ep.ep_grouped_gemm_fp8(t(f8, 8, 128), t(f32, 8, 1), t(i32, big + 1), t(f8, big, 128, 128),
                                       t(f32, big, 1, 1), t(bf16, 8, 128)),
        lambda: ep.ep_grouped_swiglu_fp8(t(f8, 8, 128), t(f32, 8, 1), t(i32, 3), t(f8, 2, 2 * big, 128),
                                         t(f32, 2, 2 * nb, 1), t(f8, 8, big), t(f32, 8, nb)),
        lambda: ep.ep_combine_backward(t(bf16, big, 64), t(bf16, 8, 64), t(i32, big, 2), t(f32, big, 2),
                                       t(bf16, 8, 64), t(f32, big, 2)),
        lambda: ep.ep_combine_backward(t(bf16, 4, big), t(bf16, 8, big), t(i32, 4, 2), w, t(bf16, 8, big), w),
        lambda: ep.ep_dispatch_backward(t(bf16, 8, 64), t(i32, big, 2), t(bf16, big, 64)),
        lambda: ep.ep_dispatch_backward(t(bf16, 8, big), t(i32, 4, 2), t(bf16, 4, big)),
        lambda: ep.ep_dispatch_backward(t(bf16, 8, 64), t(i32, 4, big), t(bf16, 4, 64)),
    ):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


def test_binding_refuses_wrong_ranks(monkeypatch):
    """Every operand of another rank is a ValueError, not an IndexError of the check."""
    monkeypatch.setattr(ep, "_operand", lambda t, name, dtype: 0)
    monkeypatch.setattr(ep, "_call_on", lambda *args: pytest.fail("the call went through"))
    bf16, f32, i32, f8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn

    def t(dtype, *shape):
        return torch.empty(shape, dtype=dtype, device="meta")

    good = {
        ep.ep_dispatch_fp8: [t(bf16, 4, 128), t(i32, 4, 2), t(f8, 8, 128), t(f32, 8, 1)],
        ep.ep_grouped_gemm_fp8: [t(f8, 8, 128), t(f32, 8, 1), t(i32, 3), t(f8, 2, 128, 128), t(f32, 2, 1, 1),
                                 t(bf16, 8, 128)],
        ep.ep_grouped_swiglu_fp8: [t(f8, 8, 128), t(f32, 8, 1), t(i32, 3), t(f8, 2, 128, 128), t(f32, 2, 1, 1),
                                   t(f8, 8, 64), t(f32, 8, 1)],
        ep.ep_combine_backward: [t(bf16, 4, 64), t(bf16, 8, 64), t(i32, 4, 2), t(f32, 4, 2), t(bf16, 8, 64),
                                 t(f32, 4, 2)],
        ep.ep_dispatch_backward: [t(bf16, 8, 64), t(i32, 4, 2), t(bf16, 4, 64)],
    }
    for fn, args in good.items():
        for i, a in enumerate(args):
            for shape in ((), (a.numel(),), (*a.shape, 1)):
                if shape != tuple(a.shape):
                    with pytest.raises(ValueError):
                        fn(*args[:i], t(a.dtype, *shape), *args[i + 1 :])
    y_less = good[ep.ep_combine_backward]
    with pytest.raises(ValueError):  # dy alone gives the rows
        ep.ep_combine_backward(y_less[0], None, y_less[2], y_less[3], t(bf16), None)
