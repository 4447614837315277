"""Equal calls of the bf16 products give equal bits (include/ep_layer.h), with
other calls between them that nothing waits for."""

import pytest
import torch

import bulk_async_tensor_amd as ep

import layer_ref as ref
from gpu_helpers import DEV
from test_gpu_layer import BF16, F32, same

pytestmark = pytest.mark.gpu


# rows, experts, K, N: tiles of 64, 128 and 256 rows with whole sums and cut ones, and several rounds of tall tiles
@pytest.mark.parametrize("rows, E, K, N", ref.HEIGHTS[::3] + [(12288, 16, 2048, 4096), (128, 1, 7168, 256)])
def test_equal_calls_give_equal_bits(rows, E, K, N):
    off = ep.ep_layout(ref.routing(rows, E, 1, 1, 0, DEV), E)["offsets"]

    def state(seed):
        return (ref.rows(rows, K, seed, DEV), ref.rows(rows, N, seed + 1, DEV), ref.weights(E, N, K, seed + 2, DEV),
                ref.rows(rows, 2 * K, seed + 3, DEV))

    def run(a, dy, b, pre):
        y, dx = torch.empty(rows, N // 2, dtype=BF16, device=DEV), torch.empty(rows, 2 * K, dtype=BF16, device=DEV)
        z = torch.empty(rows, N, dtype=BF16, device=DEV)
        db, dbias = torch.empty(E, N, K, dtype=F32, device=DEV), torch.empty(E, N, device=DEV)
        ep.ep_grouped_linear(a, off, b, y, act="swiglu", pre=z)
        ep.ep_grouped_linear_dgrad(dy, off, b, dx, act="swiglu", pre=pre)
        ep.ep_grouped_linear_wgrad(dy, a, off, db, dbias=dbias)
        return y, z, dx, db, dbias

    one, other = state(1), state(11)
    first = run(*one)
    for _ in range(8):
        run(*other)
        for got, want in zip(run(*one), first):
            same(got, want)
