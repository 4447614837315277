"""Counts of row tiles stay within 32-bit integers (checked on the host): the
wave that counts them adds 64 experts' tiles to at most 2^29 before them, and
offsets that do not ascend can make every expert hold every row."""

import random

from bulk_async_tensor_amd import EP_LINEAR_MAX_SIDE, EP_LINEAR_MAX_WEIGHT, EP_MAX_ENTRIES, EP_MAX_EXPERTS
from test_layer_shapes import shapes  # noqa: F401  (the fixture)


def test_tiles_of_many_rows_are_tall(shapes):  # noqa: F811
    rng = random.Random(7)
    asked = []
    while len(asked) < 20000:
        rows = min(EP_MAX_ENTRIES, int(2 ** rng.uniform(22, 31)) + 1)
        E = rng.choice([1, 2, 64, int(EP_MAX_EXPERTS ** rng.random()), EP_MAX_EXPERTS])
        cols, deep = (8 * int((EP_LINEAR_MAX_SIDE // 8) ** rng.random()) for _ in range(2))
        if cols * deep <= EP_LINEAR_MAX_WEIGHT:
            asked.append((rows, E, cols, deep))
    for size, (bm, _, _) in zip(asked, shapes(["linear %d %d %d %d" % s for s in asked])):
        assert bm >= 128, size
        assert 64 * -(-size[0] // bm) + (1 << 29) < 1 << 31
    # few rows, tiles of 64: the counts are small by themselves
    assert 64 * ((1 << 22) // 64) + (1 << 29) < 1 << 31
