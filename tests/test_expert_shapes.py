"""How the expert side's launches cut their work (csrc/expert_shapes.hpp),
checked on the host: the header is plain C++ and is compiled here."""

import os
import re
import subprocess

import pytest

from bulk_async_tensor_amd import LIB_PATH

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# T, vectors per lane of a row, k, compute units
BACKWARD = [(T, nv, k, cus) for T in (1, 2, 31, 128, 400, 777, 2000, 4096, 100000) for nv in range(1, 41)
            for k in (1, 2, 3, 4, 5, 8, 9, 32) for cus in (1, 24, 256)]


@pytest.fixture(scope="module")
def shapes(tmp_path_factory):
    """A function from lines of arguments to the rows of numbers chosen for them."""
    exe = str(tmp_path_factory.mktemp("shapes") / "expert_shapes")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "bulk_async_tensor_amd", "csrc"),
                    os.path.join(ROOT, "tests", "expert_shapes.cpp"), "-o", exe], check=True)

    def ask(lines):
        res = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True)
        rows = [tuple(int(v) for v in line.split()) for line in res.stdout.splitlines()]
        assert len(rows) == len(lines)
        return rows

    return ask


def test_dispatch_backward_segments(shapes):
    """The segments cover the row, and none of them starts past its end; the
    steps are among those that kernels are compiled for."""
    for size, (vs, nseg, steps) in zip(BACKWARD, shapes(["dispatch_backward %d %d %d %d" % s for s in BACKWARD])):
        nv, k = size[1], size[2]
        assert nseg >= 1 and steps >= 1, size
        assert nseg * steps * vs >= nv, f"{size}: the row's end is left out"
        assert (nseg - 1) * steps * vs < nv, f"{size}: a segment holds nothing of the row"
        assert (vs, steps) in ({(4, 1), (2, 1)} if k <= 2 else {(2, 1), (2, 2)} if k <= 4
                               else {(1, n) for n in range(1, 9)}), size


def test_dispatch_backward_kernels_are_all_reached(shapes):
    """The library holds the kernels that some call reaches, and no other."""
    names = subprocess.run(["nm", "-C", LIB_PATH], capture_output=True, text=True, check=True).stdout
    # rows at a time, vectors, steps, whether k is at most the rows at a time (and the load policy: both)
    built = {m for m in re.findall(r"__device_stub__dispatch_backward_kernel<(\d+), (\d+), (\d+), (\w+), true>", names)}
    reached = set()
    for (_, _, k, _), (vs, _, steps) in zip(BACKWARD, shapes(["dispatch_backward %d %d %d %d" % s for s in BACKWARD])):
        reached.add((str(k if k <= 2 else 4 if k <= 4 else 8), str(vs), str(steps), "true" if k <= 8 else "false"))
    assert built == reached


def test_wide_rows_follow_the_rounds(shapes):
    """A tile of 256 rows, 1.6 times the work of one of 128, only where it saves
    rounds: never where the tiles of 128 make a single round."""
    sizes = [(cus, rows, E, N) for cus in (8, 64, 256) for rows in (1, 9, 100, 127, 128, 129, 200, 255, 300, 4096, 100000)
             for E in (1, 2, 7, 64) for N in (8, 256, 264, 2048)]
    for (cus, rows, E, N), (bm,) in zip(sizes, shapes(["wide_rows %d %d %d %d" % s for s in sizes])):
        assert bm in (128, 256)
        # even if every expert's segment ended in a tile of its own
        if -(-N // 256) * (rows // 128 + min(E, rows)) <= cus:
            assert bm == 128, (cus, rows, E, N)


def test_swiglu_tiles_fit_the_rows(shapes):
    """An expert's few rows never take a tile of 128, whatever K; a tile has as
    many blocks as there are steps on the way, and each shape has its kernel."""
    names = subprocess.run(["nm", "-C", LIB_PATH], capture_output=True, text=True, check=True).stdout
    built = {(int(t), int(d)) for t, d in re.findall(r"__device_stub__grouped_swiglu_kernel<(\d+), (\d+)>", names)}
    sizes = [(each * E + E // 2, E, blocks) for each in (0, 1, 15, 16, 40, 64, 65, 80, 81, 128, 5000)
             for E in (1, 8, 256, 1024) for blocks in (2, 3, 4, 5, 56) if each * E + E // 2 > 0]
    reached = set()
    for (rows, E, blocks), (tokens, depth) in zip(sizes, shapes(["swiglu %d %d %d" % s for s in sizes])):
        each = rows // E
        assert depth <= blocks, "a tile is shorter than the steps on the way"
        assert tokens == (32 if each < 16 else 64) if each <= 64 else tokens in (64, 128), (rows, E, blocks)
        # the scan of 64 experts' tile counts is 32 bits wide
        assert 64 * (rows // tokens + 1) < 1 << 31
        reached.add((tokens, depth))
    assert built == reached


def test_wide_rows_at_the_edge_of_a_round(shapes):
    """14 experts of about 722 rows, 3 columns of tiles: 252 tiles of 128 in one
    round of 256 compute units, where half a tile too many would count as two."""
    assert shapes(["wide_rows 256 10107 14 608"]) == [(128,)]
