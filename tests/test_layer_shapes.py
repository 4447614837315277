"""How the router's and the bf16 products' launches cut their work
(csrc/linear_shapes.hpp, csrc/route_shapes.hpp), checked on the host: the
headers are plain C++ and are compiled here."""

import os
import random
import re
import subprocess

import pytest

import layer_ref as ref
from bulk_async_tensor_amd import LIB_PATH

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def shapes(tmp_path_factory):
    """A function from lines of arguments to the rows of numbers chosen for them."""
    exe = str(tmp_path_factory.mktemp("shapes") / "layer_shapes")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "bulk_async_tensor_amd", "csrc"),
                    os.path.join(ROOT, "tests", "layer_shapes.cpp"), "-o", exe], check=True)

    def ask(lines):
        res = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True)
        rows = [tuple(int(v) for v in line.split()) for line in res.stdout.splitlines()]
        assert len(rows) == len(lines)
        return rows

    return ask


def sizes(seed, n=3000):
    rng = random.Random(seed)

    def log(most):
        return max(1, int(most ** rng.random()))

    return [(log(300000), rng.choice([1, 1, 2, 3, 8, 64, 256, 1024]), 8 * log(2048), 8 * log(2048)) for _ in range(n)]


WIDE = {64: 128, 128: 256, 256: 256}  # columns of a tile, by its rows


def test_linear_items_hold_every_tile(shapes):
    """However the rows fall on the experts, there are no more tiles than items
    are counted; a cut sum's results stay within 64 MiB, and no run is empty."""
    asked = sizes(1)
    rng = random.Random(2)
    for (rows, E, cols, deep), (bm, splits, items) in zip(asked, shapes(["linear %d %d %d %d" % s for s in asked])):
        units = -(-cols // WIDE[bm])
        assert 1 <= splits <= max(1, -(-deep // 64))
        assert splits == 1 or splits * rows * cols * 4 <= 64 << 20
        cuts = sorted(rng.choices(range(rows + 1), k=E - 1))
        counts = [b - a for a, b in zip([0] + cuts, cuts + [rows])]
        assert sum(-(-c // bm) for c in counts) * units * splits <= items
        assert (rows // bm + min(E, rows)) * units * splits >= items or E == 1


def test_wgrad_items_are_its_tiles(shapes):
    asked = sizes(3)
    for (rows, E, N, K), (bm, splits, items) in zip(asked, shapes(["wgrad %d %d %d %d" % s for s in asked])):
        assert items == E * -(-N // bm) * -(-K // WIDE[bm]) * splits
        assert splits == 1 or splits * E * N * K * 4 <= 64 << 20
        assert splits <= max(1, -(-(rows // E) // 64))


def test_sizes_of_every_height(shapes):
    for line in ("linear {0} {1} {3} {2}", "linear {0} {1} {2} {3}", "wgrad {0} {1} {3} {2}"):
        got = {(bm, splits > 1) for bm, splits, _ in shapes([line.format(*s) for s in ref.HEIGHTS])}
        assert got == {(bm, cut) for bm in (64, 128, 256) for cut in (False, True)}, line


def test_one_round_of_whole_sums_is_not_cut(shapes):
    """Where tiles of 128 rows fill the compute units exactly, nothing is gained by cutting."""
    for deep in (64, 640, 7168):
        assert shapes(["linear %d 1 256 %d" % (256 * 128, deep)])[0][1] == 1


def test_route_lanes_hold_the_token(shapes):
    asked = [(T, E, k, cus) for T in (1, 128, 2048, 2049, 100000) for E in (1, 5, 16, 64, 65, 128, 256, 257, 512, 513, 1024)
             for k in (1, 8, 15, 16, 32) for cus in (8, 256) if k <= E]
    for (T, E, k, _), (lanes, each) in zip(asked, shapes(["route %d %d %d %d" % s for s in asked])):
        assert lanes * each >= E and lanes > k, (T, E, k)
        assert (lanes, each) in {(16, 4), (16, 8), (16, 16), (16, 32), (64, 4), (64, 8), (64, 16)}


def test_kernels_are_those_that_are_reached(shapes):
    """The library holds the kernels that some call reaches, and no other."""
    names = subprocess.run(["nm", "-C", LIB_PATH], capture_output=True, text=True, check=True).stdout
    built = {(int(a), int(b), t == "true") for a, b, t in re.findall(r"__device_stub__route_kernel<(\d+), (\d+), (\w+)>", names)}
    asked = ["route %d %d %d 256" % (T, E, k) for T in (1, 100000) for E in (4, 64, 128, 256, 512, 1024) for k in (1, 20)
             if k <= E]
    assert built == {(*r, t) for r in shapes(asked) for t in (False, True)}
    # forward and dgrad with every activation, wgrad without, each with three tile heights
    wide = set(re.findall(r"__device_stub__linear_wide_kernel<\S*?(\d), (\d), (\d+), \d>", names))
    if not wide:
        wide = set(re.findall(r"__device_stub__linear_wide_kernel<\(.*?\)(\d), (\d), (\d+), \d>", names))
    assert wide == {(p, a, bm) for bm in ("64", "128", "256") for p, a in [(p, a) for p in "01" for a in "0123"] + [("2", "0")]}
    picked = shapes([f"{what} {sizes}" for what in ("linear", "wgrad")
                     for sizes in ("100 1 256 64", "900 2 1040 4096" if what == "linear" else "512 1 2048 4096",
                                   "65536 1 4096 4096")])
    assert [p[0] for p in picked] == [64, 128, 256] * 2
