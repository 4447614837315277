// How the bf16 products' launches cut their work, from sizes alone: plain C++
// without HIP, so that the rules can be checked on any host.
#pragma once

#include <stdint.h>

namespace ep {

constexpr int kLinearCols = 256, kLinearDeep = 64;  // a tile's columns, and places along the sum in a step
constexpr int kLinearCus = 256;                     // compute units that a call's work is cut for
constexpr int kLinearMostItems = 1 << 30;           // items of a call
constexpr int kLinearMostSplits = 64;
constexpr int64_t kLinearMostPartial = (int64_t)64 << 20;  // bytes of results of cut sums

// Steps whose tiles are in LDS or on the way.
constexpr int linear_copies(int rows) { return rows == 256 ? 2 : 3; }

// Rows of a tile, runs that a sum is cut into, and the items (tiles times
// runs) there can be.
struct LinearShape {
  int rows, splits;
  int64_t items;
};

// The shape is the one whose estimated time is least.  A tile's step takes
// 0.75 us with 128 rows and 1.15 with 256 where half of the CUs or fewer work,
// 0.95 and 1.65 where all do (wgrad, both sides turned, 0.95 and 1.2 with 128), and a
// tile 2.5 or 4 us beside its steps.  The CUs make whole rounds of items.  A
// cut sum costs a second kernel, 5 us, and its results their way to memory and
// back, 2.9 bytes a picosecond.  Measured, us, by rows / runs (the rule's
// choice first):
//   128 rows, K 7168, N 256 (a router)      128/28 16.5  128/1 90.5  128/8 21.8
//   4096 rows of it                         128/8 34.0   128/1 92.6  256/8 41.7
//   97 rows, K 1200, N 336                  128/6 12.7   128/1 19.1  128/16 13.7
//   2 rows, 5 experts, K 576, N 320         128/1 11.0   128/2 12.2
//   416 rows, 34 experts, K 6456, N 816     128/3 101.8  128/1 130.9 128/28 116.3
//   4096 rows, K = N = 4096                 256/1 110.8  128/1 132.1 256/2 177.2
//   1024 rows, K = N = 4096                 128/2 52.5   128/1 55.8  256/4 57.1
//   12078 rows, 7 experts, K 1448, N 368    128/1 28.4   256/1 40.2  128/2 59.2
//   wgrad, 4096 rows, N 256, K 7168         128/4 36.8   128/1 65.8  128/8 49.0
//   wgrad, 56934 rows, 9 experts, 848 x 568 256/2 122.1  128/1 141.8 256/8 157.7
//   wgrad, 3944 rows, 2872 x 4864           256/1 101.5  128/1 130.5 256/2 154.5
struct LinearWork {
  int64_t tiles[2];   // tiles there may be expected to be with 128 and with 256 rows,
  int64_t most[2];    // and at most
  int64_t steps;      // of a tile's sum
  int64_t results;    // float32 values of a run's results
  bool wgrad;
};

inline int64_t linear_cost_ns(const LinearWork& w, int tall, int64_t splits) {
  const int64_t items = w.tiles[tall] * splits;
  const int64_t rounds = (items + kLinearCus - 1) / kLinearCus;
  int64_t steps = (w.steps + splits - 1) / splits;
  const int64_t least = linear_copies(tall ? 256 : 128) + 1;
  if (steps < least) steps = least;
  const bool all = 2 * items > kLinearCus;
  const int64_t step = tall ? (all ? 1650 : 1150) : all ? (w.wgrad ? 1200 : 950) : w.wgrad ? 950 : 750;
  const int64_t join = splits > 1 ? 5000 + splits * w.results * 4 / 2900 : 0;
  return rounds * (steps * step + (tall ? 4000 : 2500)) + join;
}

inline LinearShape linear_best(const LinearWork& w) {
  LinearShape best = {128, 1, w.most[0]};
  int64_t cost = -1;
  for (int tall = 0; tall < 2; ++tall)
    for (int s = 1; s <= kLinearMostSplits && s <= w.steps; ++s) {
      if (s > 1 && s * w.results * 4 > kLinearMostPartial) break;
      const int64_t c = linear_cost_ns(w, tall, s);
      if (cost >= 0 && c >= cost) continue;
      cost = c;
      best.rows = tall ? 256 : 128;
      best.splits = s;
      best.items = w.most[tall] * s;
    }
  return best;
}

// Forward and dgrad: `cols` results a row, sums of `deep`.  `one`: one weight
// for all rows, whose tiles the host can count.  (An expert's last tile counts
// as half; one that holds fewer rows than a tile has one.)
inline LinearShape linear_shape(int64_t rows, int E, int cols, int deep, int64_t results) {
  const int64_t units = (cols + kLinearCols - 1) / kLinearCols, held = E < rows ? E : rows;
  LinearWork w = {};
  for (int tall = 0; tall < 2; ++tall) {
    const int64_t bm = tall ? 256 : 128, half = (2 * rows / bm + held) / 2;
    w.tiles[tall] = units * (E == 1 ? (rows + bm - 1) / bm : half > held ? half : held);
    w.most[tall] = units * (E == 1 ? (rows + bm - 1) / bm : rows / bm + held);
  }
  w.steps = (deep + kLinearDeep - 1) / kLinearDeep;
  w.results = results;
  return linear_best(w);
}

// wgrad: N x K results for each expert, sums over its rows.
inline LinearShape wgrad_shape(int64_t rows, int E, int N, int K) {
  const int64_t units = (K + kLinearCols - 1) / kLinearCols;
  LinearWork w = {};
  for (int tall = 0; tall < 2; ++tall) {
    const int64_t bm = tall ? 256 : 128;
    w.tiles[tall] = w.most[tall] = E * ((N + bm - 1) / bm) * units;
  }
  w.steps = (rows / E + kLinearDeep - 1) / kLinearDeep;
  w.results = (int64_t)E * N * K;
  w.wgrad = true;
  return linear_best(w);
}

}  // namespace ep
