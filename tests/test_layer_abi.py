"""The C ABI of include/ep_layer.h without a GPU: every entry point is exported
and bound, bad arguments are rejected on the host before any HIP call, and the
plain forms that the GPU tests compare with agree with differences."""

import math
import os
import re

import pytest
import torch

import bulk_async_tensor_amd as ep

import layer_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ep_layer.h")

# fake device addresses: only their alignment matters, none is dereferenced
A16 = 0x7F0000000000
A4 = A16 + 4
A2 = A16 + 2
ODD = A16 + 1


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ep.LIB_PATH):
        pytest.fail("libep.so is not built (run __graft_entry__.build())")
    return ep.lib()


def test_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(ep_\w+)\s*\(", text)))
    assert names == ["ep_grouped_linear", "ep_grouped_linear_dgrad", "ep_grouped_linear_dgrad_workspace_bytes",
                     "ep_grouped_linear_wgrad", "ep_grouped_linear_wgrad_workspace_bytes",
                     "ep_grouped_linear_workspace_bytes", "ep_route", "ep_route_backward"]
    for n in names:
        assert hasattr(lib, n) and n in ep._SIGNATURES and n in ep.__all__, n
    consts = dict(re.findall(r"\b(EP_(?:ACT|SCORE|BF16|F32)\w*) = (\d+)", text))
    assert len(consts) == 8
    for n, v in consts.items():
        assert getattr(ep, n) == int(v)


def change(args, **over):
    assert set(over) <= {n for n, _ in args}
    return [over.get(n, v) for n, v in args]


def refused(lib, name, args, over, code):
    assert getattr(lib, name)(*change(args, **over)) == code
    if code:
        assert name in lib.ep_last_error().decode()


ROUTE = [("l", A16), ("type", 1), ("T", 4), ("E", 64), ("score", 1), ("bias", A4), ("groups", 8), ("top", 4),
         ("best", 2), ("k", 6), ("renorm", 1), ("scale", 1.0), ("idx", A4), ("w", A4), ("stream", None)]


@pytest.mark.parametrize("over, code", [
    (dict(type=2), -1), (dict(type=-1), -1), (dict(T=-1), -1), (dict(E=0), -1), (dict(E=1032), -1), (dict(score=2), -1),
    (dict(groups=0), -1), (dict(groups=7), -1), (dict(E=1024, groups=128, best=1), -1), (dict(top=0), -1),
    (dict(top=9), -1), (dict(best=0), -1), (dict(best=3), -1), (dict(groups=64, best=2), -1), (dict(k=0), -1),
    (dict(k=33), -1), (dict(top=1, k=9), -1), (dict(E=4, groups=1, top=1, k=5), -1), (dict(scale=math.inf), -1),
    (dict(scale=math.nan), -1), (dict(T=1 << 30, E=64), -1), (dict(l=None), -1), (dict(idx=None), -1),
    (dict(w=None), -1), (dict(l=A2), -2), (dict(l=ODD, type=0), -2), (dict(bias=ODD), -2), (dict(idx=A2), -2),
    (dict(w=A2), -2), (dict(T=0), 0), (dict(T=0, l=None, idx=None, w=None, bias=None), 0),
])
def test_route_arguments(lib, over, code):
    refused(lib, "ep_route", ROUTE, over, code)


RBWD = [("l", A16), ("type", 1), ("T", 4), ("E", 64), ("score", 0), ("idx", A4), ("k", 6), ("renorm", 0),
        ("scale", 2.5), ("dw", A4), ("dl", A16), ("dtype", 0), ("stream", None)]


@pytest.mark.parametrize("over, code", [
    (dict(type=3), -1), (dict(dtype=2), -1), (dict(T=-1), -1), (dict(E=0), -1), (dict(E=1025), -1),
    (dict(score=-1), -1), (dict(k=0), -1), (dict(k=33), -1), (dict(E=4, k=5), -1), (dict(scale=-math.inf), -1),
    (dict(T=1 << 30), -1), (dict(l=None), -1), (dict(idx=None), -1), (dict(dw=None), -1), (dict(dl=None), -1),
    (dict(l=A2), -2), (dict(idx=ODD), -2), (dict(dw=A2), -2), (dict(dl=ODD), -2), (dict(dl=A2, dtype=1), -2),
    (dict(T=0), 0),
])
def test_route_backward_arguments(lib, over, code):
    refused(lib, "ep_route_backward", RBWD, over, code)


SIZES = [
    (dict(rows=-1), -1), (dict(rows=1 << 31), -1), (dict(K=0), -1), (dict(K=12), -1), (dict(K=(1 << 20) + 8), -1),
    (dict(N=0), -1), (dict(N=-8), -1), (dict(N=20), -1), (dict(N=(1 << 20) + 8), -1), (dict(N=1 << 15, K=1 << 15), -1),
    (dict(E=0), -1), (dict(E=1025), -1), (dict(off=None), -1), (dict(off=A2), -2),
]
LINEAR = [("a", A16), ("rows", 4096), ("K", 256), ("off", A4), ("E", 4), ("b", A16), ("bias", A4), ("N", 4096),
          ("act", 0), ("res", A16), ("y", A16), ("type", 0), ("pre", A16), ("ws", A16), ("bytes", 1 << 40),
          ("stream", None)]


@pytest.mark.parametrize("over, code", SIZES + [
    (dict(act=4), -1), (dict(act=-1), -1), (dict(act=3, N=24), -1), (dict(type=2), -1), (dict(a=None), -1),
    (dict(b=None), -1), (dict(y=None), -1), (dict(a=A16 + 8), -2), (dict(b=A16 + 8), -2), (dict(y=A16 + 8), -2),
    (dict(res=A16 + 8), -2), (dict(pre=A4), -2), (dict(bias=A2), -2), (dict(rows=0), 0),
    (dict(rows=0, a=None, b=None, y=None, bias=None, res=None, pre=None, ws=None, bytes=0), 0),
    (dict(rows=2143289343, E=1, N=1 << 20, K=1000), -1),
])
def test_linear_arguments(lib, over, code):
    refused(lib, "ep_grouped_linear", LINEAR, over, code)


DGRAD = [("dy", A16), ("rows", 4096), ("N", 256), ("off", A4), ("E", 4), ("b", A16), ("K", 4096), ("act", 3),
         ("pre", A16), ("dx", A16), ("ws", A16), ("bytes", 1 << 40), ("stream", None)]


@pytest.mark.parametrize("over, code", SIZES + [
    (dict(act=4), -1), (dict(dy=None), -1), (dict(b=None), -1), (dict(dx=None), -1), (dict(pre=None), -1),
    (dict(dy=A4), -2), (dict(b=A4), -2), (dict(dx=A4), -2), (dict(pre=A4), -2), (dict(rows=0), 0),
    (dict(rows=0, pre=None, dy=None), 0),
])
def test_dgrad_arguments(lib, over, code):
    refused(lib, "ep_grouped_linear_dgrad", DGRAD, over, code)


WGRAD = [("dy", A16), ("a", A16), ("rows", 4096), ("N", 1024), ("K", 1024), ("off", A4), ("E", 4), ("db", A16),
         ("type", 1), ("dbias", A4), ("ws", A16), ("bytes", 1 << 40), ("stream", None)]


@pytest.mark.parametrize("over, code", SIZES + [
    (dict(type=2), -1), (dict(dy=None), -1), (dict(a=None), -1), (dict(db=None), -1), (dict(rows=0, db=None), -1),
    (dict(dy=A4), -2), (dict(a=A4), -2), (dict(db=A4), -2), (dict(dbias=A2), -2),
])
def test_wgrad_arguments(lib, over, code):
    refused(lib, "ep_grouped_linear_wgrad", WGRAD, over, code)


def test_workspace_is_checked(lib):
    """Wherever a call needs a workspace, it is refused without one, with one that is too small, and unaligned."""
    cases = [("ep_grouped_linear", LINEAR, lib.ep_grouped_linear_workspace_bytes(128, 7168, 1, 256)),
             ("ep_grouped_linear_dgrad", DGRAD, lib.ep_grouped_linear_dgrad_workspace_bytes(128, 256, 1, 7168)),
             ("ep_grouped_linear_wgrad", WGRAD, lib.ep_grouped_linear_wgrad_workspace_bytes(8192, 1024, 1, 256))]
    sizes = {"ep_grouped_linear": dict(rows=128, K=7168, E=1, off=None, N=256),
             "ep_grouped_linear_dgrad": dict(rows=128, K=256, E=1, off=None, N=7168),
             "ep_grouped_linear_wgrad": dict(rows=8192, K=1024, E=1, off=None, N=256)}
    for name, args, need in cases:
        assert 0 < need <= (64 << 20) + (1 << 20) and need % 16 == 0
        for over, code in ((dict(ws=None, bytes=0), -4), (dict(ws=None), -4), (dict(bytes=need - 1), -4),
                           (dict(ws=A4, bytes=need), -2)):
            refused(lib, name, args, {**sizes[name], **over}, code)
    assert lib.ep_grouped_linear_workspace_bytes(-1, 64, 1, 64) == 0
    assert lib.ep_grouped_linear_dgrad_workspace_bytes(8, 0, 1, 64) == 0
    assert lib.ep_grouped_linear_wgrad_workspace_bytes(8, 64, 0, 64) == 0


def test_binding_refuses_host_tensors():
    """The binding has no fallback: tensors that are not on a GPU are refused."""
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, 2, dtype=torch.int32)
    w = torch.zeros(2, 2)
    b = torch.zeros(1, 64, 64, dtype=torch.bfloat16)
    for call in (lambda: ep.ep_route(x, i, w), lambda: ep.ep_route_backward(x, i, w, x),
                 lambda: ep.ep_grouped_linear(x, None, b, x), lambda: ep.ep_grouped_linear_dgrad(x, None, b, x),
                 lambda: ep.ep_grouped_linear_wgrad(x, x, None, b)):
        with pytest.raises(ValueError, match="device"):
            call()
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        ep._either(ep._torch_objects(), _Half(), "logits")


class _Half:
    """What a float16 device tensor looks like to the binding's checks."""
    dtype, is_cuda = torch.float16, True

    def is_contiguous(self):
        return True


# ------------------------------------------------------------------ the plain forms against differences
def test_route_reference():
    """Ties, masks and NaN by hand."""
    inf, nan = math.inf, math.nan
    l = torch.tensor([[1.0, 3.0, 3.0, 0.0], [-inf, -inf, -inf, -inf], [nan, 1.0, 5.0, nan], [-inf, 2.0, -inf, -inf]])
    ids, w = ref.route(l, 2, "softmax")
    assert ids.tolist() == [[1, 2], [0, 1], [0, 3], [1, 0]]
    assert w[0].tolist() == [0.5, 0.5] and w[1].tolist() == [0, 0] and torch.isnan(w[2]).all()
    assert w[3].tolist() == [1, 0]
    ids, _ = ref.route(torch.tensor([[5.0, 0.0, 3.0, 3.0]]), 1, "sigmoid", groups=2, top_groups=1, group_best=2)
    assert ids.tolist() == [[2]]


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_is_the_difference(kind, renorm):
    g = torch.Generator().manual_seed(1)
    l = torch.randn(3, 9, generator=g).double()
    dw = torch.randn(3, 4, generator=g).double()
    ids, _ = ref.route(l, 4, kind, renorm=renorm)
    got = ref.route_backward(l, ids, dw, kind, renorm, 2.5)

    def loss(x):
        s = torch.gather(ref.scores(kind, x), 1, ids.long())
        return float((2.5 * dw * (s / s.sum(1, keepdim=True) if renorm else s)).sum())

    for t in range(3):
        for e in range(9):
            h = torch.zeros_like(l)
            h[t, e] = 1e-6
            assert abs((loss(l + h) - loss(l - h)) / 2e-6 - float(got[t, e])) < 1e-8


@pytest.mark.parametrize("kind", ["none", "silu", "gelu", "swiglu"])
def test_product_gradients_are_the_differences(kind):
    """A step along a random direction changes the loss as the gradients say."""
    g = torch.Generator().manual_seed(2)
    offsets = torch.tensor([0, 3, 3, 7])
    x0 = torch.randn(7, 8, generator=g).double()
    w1 = torch.randn(3, 12, 8, generator=g).double() * 0.5
    width = 6 if kind == "swiglu" else 12
    w2 = torch.randn(3, 5, width, generator=g).double() * 0.5
    dy = torch.randn(7, 5, generator=g).double()

    def loss(x, w1, w2):
        z, _ = ref.product(x, offsets, w1, False)
        h = ref.act(kind, z[:, :6]) * z[:, 6:] if kind == "swiglu" else ref.act(kind, z)
        return (ref.product(h, offsets, w2, False)[0] * dy).sum(), z, h

    _, z, h = loss(x0, w1, w2)
    dz, _ = ref.dgrad(dy, offsets, w2, kind, z)
    dx, _ = ref.dgrad(dz, offsets, w1, "none", None)
    dw2 = ref.wgrad(dy, h, offsets, 3, torch.float32)[0]
    dw1 = ref.wgrad(dz, x0, offsets, 3, torch.float32)[0]
    assert float(dw1[1].abs().max()) == 0.0
    for which, grad in ((0, dx), (1, dw1), (2, dw2)):
        v = torch.randn(grad.shape, generator=g).double()
        ends = []
        for sign in (1e-6, -1e-6):
            args = [x0, w1, w2]
            args[which] = args[which] + sign * v
            ends.append(float(loss(*args)[0]))
        assert abs((ends[0] - ends[1]) / 2e-6 - float((grad * v).sum())) < 1e-6 * max(1.0, float((grad * v).abs().sum()))
