// How the expert side's launches cut their work, from sizes alone: plain C++
// without HIP, so that the rules can be checked on any host.
#pragma once

#include <stdint.h>

namespace ep {

// ep_dispatch_backward: a token's row of nv vectors per lane in nseg segments
// (one wave each) of `steps` steps of vs vectors.
struct GatherShape {
  int vs, nseg, steps;
};

// Segments of up to 8 KiB, of 4 KiB for k <= 4 (T = 8192, H = 4096: k = 4 57
// against 61 us, k = 2 35 against 36; k = 8, H = 7168 keeps 8: 88 against 93
// at T = 4096), shorter where a batch would leave CUs without 8 waves.  A step
// gathers 4, 2 or 1 vectors at k <= 2, k <= 4 and above, and never more than a
// segment holds: every segment starts inside the row.  Segments of 2 vectors
// against segments of 4 at k = 2: T = 128, H = 7168 2.33 / 2.55 us, T = 1000,
// H = 1024 2.34 / 2.56, T = 2000 2.76 / 3.02; k = 1 gains half of that.
inline GatherShape dispatch_backward_shape(int64_t T, int nv, int k, int cus) {
  int most = k <= 4 ? 4 : 8;
  while (most > 2 && T * ((nv + most - 1) / most) < 8LL * cus) most /= 2;
  GatherShape s;
  s.vs = k <= 2 ? most : k <= 4 ? 2 : 1;
  const int nsteps = (nv + s.vs - 1) / s.vs;
  s.nseg = (nsteps * s.vs + most - 1) / most;
  s.steps = (nsteps + s.nseg - 1) / s.nseg;
  return s;
}

// ep_grouped_gemm_fp8: token rows per workgroup of the wide kernel.  A tile of
// 256 takes 1.6 times as long as one of 128 where the products bound it, so
// the choice goes by the rounds of tiles that the compute units make (every
// expert's last tile is taken as half full, and a lone half-full tile is a
// round).  Measured, 128 against 256: 32 experts, K = N = 4096, 128 rows
// each 148 / 163 us, 512 each 374 / 348, 2048 each 1365 / 1204; one expert of
// 100 rows, K = 2048, N = 256 20.7 / 23.4.
inline int wide_rows(int cus, int64_t rows, int E, int N) {
  const int64_t units_n = (N + 255) / 256, held = E < rows ? E : rows;
  auto rounds = [&](int bm) {
    const int64_t tiles = units_n * (2 * rows / bm + held) / 2;
    return tiles > cus ? (tiles + cus - 1) / cus : 1;
  };
  return 8 * rounds(256) <= 5 * rounds(128) ? 256 : 128;
}

// ep_grouped_swiglu_fp8: token rows of a tile, and the steps (blocks along K)
// whose rows are in registers or on the way; a tile has at least that many
// (a shorter one would be two tiles ahead of its results).
struct SwigluShape {
  int tokens, depth;
};

// The token rows go by the rows that there are for each expert, us with 32 / 64
// / 128.  K 7168, I 2048, 256 experts: 4 rows each 1200 / 1280 / 1684, 16 each
// 1332 / 1324 / 1738, 32 each 1684 / 1436 / 1811, 64 each 2492 / 1908 / 1995,
// 128 each 4430 / 2884 / 2580.  K 2048, I 1024, 16 experts: 8 rows each 24 /
// 25 / 33, 64 each 41 / 27 / 34, 128 each 58 / 45 / 35.  Rows of 2 or 3 blocks
// take the same tiles with 2 steps on the way, I 1024, 256 experts: K 256, 4
// rows each 35 (32) / 75 (128), 64 each 65 (64) / 76 (128), 72 each 79.5 (64) /
// 76.5 (128); K 384, 64 each 76 (64) / 87 (128).
inline SwigluShape swiglu_shape(int64_t rows, int E, int blocks) {
  const int64_t each = rows / E;
  SwigluShape s;
  s.tokens = each < 16 ? 32 : each <= (blocks >= 4 ? 80 : 64) ? 64 : 128;
  s.depth = s.tokens < 128 && blocks >= 4 ? 4 : 2;
  return s;
}
constexpr int kSwigluLeastBlocks = 2;

}  // namespace ep
