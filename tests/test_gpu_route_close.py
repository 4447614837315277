"""ep_route where scores or group ranks are closer than float32 holds, and
ep_route_backward where a sigmoid is nearly one, against 64 bits (layer_ref.py)."""

import math

import pytest
import torch

import bulk_async_tensor_amd as ep

import layer_ref as ref
from gpu_helpers import DEV
from test_gpu_layer import BF16, F32, call_route, check_route, gen, logits_of

pytestmark = pytest.mark.gpu

MANY = 2100  # tokens from which, with 512 experts or fewer and k up to 15, 16 lanes take a token


@pytest.mark.parametrize("T", [3, MANY])
def test_saturated_scores_of_a_group(T):
    """Without a bias the logits are compared, also where their sigmoids are equal in float64."""
    l = torch.tensor([40.0, 41.0, -1.0, -2.0, -9.0, -9.0, -9.0, -9.0], device=DEV).repeat(T, 1)
    for dtype in (F32, BF16):
        idx, _ = check_route(l.to(dtype), 1, "sigmoid", groups=2)
        assert bool((idx == 1).all())
    l = torch.zeros(T, 16, device=DEV)
    l[:, 0], l[:, 5] = 40.0, 50.0
    idx, _ = check_route(l, 1, "sigmoid", groups=2)
    assert bool((idx == 5).all())


@pytest.mark.parametrize("T", [40, MANY])  # 64 and 16 lanes a token
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("start", [24.0, 30.0, 40.0, 800.0])
def test_saturated_scores_of_several_groups(T, dtype, start):
    """A few neighbouring logits far above zero in the groups that stay, in ascending and in mixed order."""
    E, k = 128, 5
    step = torch.finfo(dtype).eps * 2.0 ** math.floor(math.log2(start))
    for many in range(2, k + 4):
        l = logits_of(T, E, many).clamp_(max=4.0)
        at = torch.randperm(32, generator=torch.Generator().manual_seed(many))[:many].sort().values.to(DEV)
        up = start + step * torch.arange(1, many + 1, device=DEV)
        l[::2, at] = up
        l[1::2, at] = up[torch.randperm(many, generator=torch.Generator().manual_seed(9)).to(DEV)]
        l = l.to(dtype)
        check_route(l, k, "sigmoid", groups=8, top_groups=2, group_best=2)
        check_route(l, k, "sigmoid", renormalize=False, groups=4, top_groups=1, group_best=1)


def decided(l, kind, bias, groups, top):
    """Rows whose group ranks, sums of two, 64 bits tell apart at the edge of the groups that stay.  A score there is off
    by 4 half steps of 1, a bias added to it by half a step of the sum, twice, and their sum by half a step of at most
    both sizes: two ranks differ for certain from 16 half steps of (1 + the two sizes) on."""
    c = (ref.scores(kind, l.cpu()) + bias.cpu().double()).view(l.shape[0], groups, -1)
    two = c.topk(2, dim=2).values
    rank, order = two.sum(2).sort(1, descending=True)
    size = torch.gather(1.0 + two.abs().sum(2), 1, order)
    return rank[:, top - 1] - rank[:, top] > 16 * 2.0 ** -53 * (size[:, top - 1] + size[:, top])


@pytest.mark.parametrize("T", [500, MANY])
@pytest.mark.parametrize("size", [10.0, 64.0, 1024.0])
def test_group_ranks_whose_biases_cancel(T, size):
    """A group's two best scores with biases of opposite sign: their sum is close to another group's, and each of
    them is rounded at its own size."""
    E, groups = 128, 8
    l = logits_of(T, E, 1)
    apart = torch.randn(T, generator=gen(2), device=DEV).sign() * 10.0 ** (-7.5 + 4 * torch.rand(T, generator=gen(3), device=DEV))
    l[:, 16] = l[:, 0] + apart
    l[:, 17] = l[:, 1]
    bias = torch.full((E,), -4.0 * size, device=DEV)
    bias[0], bias[1], bias[16], bias[17] = size, -size, 0.0, 0.0
    for kind in ("sigmoid", "softmax"):
        for b, top in ((bias, 1), (bias.flip(0).contiguous(), 7)):
            sure = decided(l, kind, b, groups, top)
            assert int(sure.sum()) >= 0.8 * T  # (float32 loses what is below 10^-6.9: 0.6 of the 4 decades)
            check_route(l[sure.to(DEV)], 2, kind, bias=b, groups=groups, top_groups=top, group_best=2)


def test_group_ranks_at_the_ends():
    """Biases of infinite size and sums past float32's range."""
    T, E = 200, 64
    l = logits_of(T, E, 1)
    inf = math.inf
    for a, b in ((-inf, 0.0), (inf, 0.0), (inf, -inf), (3e38, 3e38), (-3e38, 3e38), (-3e38, -3e38), (inf, inf)):
        bias = torch.zeros(E, device=DEV)
        bias[3], bias[4], bias[20] = a, b, a
        for top in (1, 2, 3):
            check_route(l, 4, "sigmoid", bias=bias, groups=8, top_groups=top, group_best=2)
    bias = torch.full((E,), -inf, device=DEV)  # (experts left out by their bias, whole groups of them)
    bias[8:20] = 0.01
    check_route(l, 4, "sigmoid", bias=bias, groups=8, top_groups=2, group_best=2)


def subnormal(steps):
    """Float32 values of so many steps of 2^-149."""
    size = steps.abs().to(torch.int32)
    return torch.where(steps < 0, size | torch.iinfo(torch.int32).min, size).view(torch.float32).to(DEV)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T, E, k", [(1, 4, 1), (300, 64, 4), (300, 256, 8), (MANY, 256, 8), (MANY, 512, 8)])
def test_subnormal_logits(T, E, k, kind):
    """Logits of a few steps of 2^-149: a key's cell there is as wide as the values themselves."""
    l = subnormal(torch.tensor([3, 1, 5, 0])).repeat(T, 1)
    idx, _ = call_route(l, 1, kind)
    assert bool((idx == 2).all())
    g = torch.Generator().manual_seed(E)
    for most in (2, 8, 1 << 10, 1 << 22):
        check_route(subnormal(torch.randint(-most, most + 1, (T, E), generator=g)), k, kind)
        few = torch.where(torch.rand(T, E, generator=g) < 0.02, torch.randint(1, most + 1, (T, E), generator=g), 0)
        check_route(subnormal(few), k, kind)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("out", [F32, BF16])
def test_gradient_of_a_sigmoid_near_one(out, renorm):
    """dl = scale p (1 - s) (dw - D) relative to its own size.  In half steps of float32: exp costs 2, the sum and the
    quotient after it 2, so s and 1 - s are 4 off; p, divided by a sum over k = 4, 12; D, a sum of p dw, 16; the
    difference is 1 + 16 off relative to |dw| + |D|, and four products add 4: 12 + 4 + 17 + 4 = 37."""
    T, E, k = 400, 32, 4
    l = torch.rand(T, E, generator=gen(1), device=DEV) * 75.0 + 5.0
    l[: T // 2] = torch.rand(T // 2, 1, generator=gen(2), device=DEV) * 25.0 + 5.0 + l[: T // 2] * 0.01
    l[-20:] = -l[-20:]
    idx, _ = call_route(l, k, "sigmoid")
    dw = torch.randn(T, k, generator=gen(3), device=DEV)
    dl = torch.full((T, E), 7.0, dtype=out, device=DEV)
    ep.ep_route_backward(l, idx, dw, dl, score="sigmoid", renormalize=renorm, scale=2.5)
    l, at, dw = l.cpu().double(), idx.cpu().long(), dw.cpu().double()
    lj = torch.gather(l, 1, at)
    s, rest = torch.sigmoid(lj), 1.0 / (1.0 + torch.exp(lj))
    p = s / s.sum(1, keepdim=True) if renorm else s
    D = (p * dw).sum(1, keepdim=True) if renorm else torch.zeros(T, 1, dtype=torch.float64)
    want = torch.zeros(T, E, dtype=torch.float64).scatter_(1, at, 2.5 * p * rest * (dw - D))
    size = torch.zeros(T, E, dtype=torch.float64).scatter_(1, at, 2.5 * p * rest * (dw.abs() + D.abs()))
    err = (dl.cpu().double() - want).abs()
    tol = 37 * ref.U32 * size
    tol = tol + ref.UNIT[out] * (want.abs() + tol) + 2.0 ** -133
    assert bool((err <= tol).all()), float((err / tol.clamp_min(1e-300)).max())
