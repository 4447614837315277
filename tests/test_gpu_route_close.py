"""ep_route where scores are closer than float32 or float64 holds, against 64 bits
(layer_ref.py)."""

import math

import pytest
import torch

from gpu_helpers import DEV
from test_gpu_layer import BF16, F32, check_route, logits_of

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
