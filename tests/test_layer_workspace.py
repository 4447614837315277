"""The workspace sizes of ep_layer.h: at most 64 MiB whatever the sizes, and what
a cut sum stores (checked on the host)."""

import random

import pytest

import bulk_async_tensor_amd as ep

LIMIT = 64 << 20
# rows, K, E, N: short rows of a long weight, where a cut sum's bias sums are an eighth of its other results
LONG = [(100_000_000, 8, 1, 66224), (65536, 8, 1, 252688), (131072, 256, 1, 1024), (1 << 30, 8, 1, 1 << 20),
        (300_000, 8, 4, 40000), (1 << 20, 16, 16, 8192), (1 << 22, 8, 1, 8)]


def sizes():
    rng = random.Random(4)

    def log(most):
        return max(1, int(most ** rng.random()))

    short = [(log(1 << 30), 8 * rng.randint(1, 4), rng.choice([1, 1, 2, 5, 64]), 8 * log(1 << 17)) for _ in range(3000)]
    return short + [(log(1 << 24), 8 * log(4096), rng.choice([1, 1, 3, 64, 1024]), 8 * log(4096)) for _ in range(3000)]


@pytest.mark.parametrize("what", ["ep_grouped_linear", "ep_grouped_linear_dgrad", "ep_grouped_linear_wgrad"])
def test_workspaces_stay_within_the_limit(what):
    ask = getattr(ep, what + "_workspace_bytes")
    cut = 0
    for rows, K, E, N in LONG + sizes():
        need = ask(rows, K, E, N)
        assert need <= LIMIT, (rows, K, E, N, need)
        one = {"ep_grouped_linear": rows * N, "ep_grouped_linear_dgrad": rows * K,
               "ep_grouped_linear_wgrad": E * N * (K + 1)}[what] * 4  # float32 results of a run, bias sums included
        assert need % one == 0 and (need == 0 or need // one >= 2), (rows, K, E, N, need)
        cut += need > 0
    assert cut > 100
