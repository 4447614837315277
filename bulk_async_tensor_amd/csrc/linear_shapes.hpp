// How the bf16 products' launches cut their work, from sizes alone: plain C++
// without HIP, so that the rules can be checked on any host.
#pragma once

#include <stdint.h>

namespace ep {

constexpr int kLinearDeep = 64;            // places along the sum in a step
constexpr int kLinearCus = 256;            // compute units that a call's work is cut for
constexpr int kLinearMostItems = 1 << 30;  // items of a call
constexpr int kLinearMostSplits = 64;
constexpr int64_t kLinearMostPartial = (int64_t)64 << 20;  // bytes that cut sums store

// A tile's columns, by its rows.
constexpr int linear_cols(int rows) { return rows == 64 ? 128 : 256; }
// Steps whose tiles are in LDS or on the way.  (64 rows with four or five: a
// router's product 13.5 or 14.1 us for 13.7, wgrad of 4096 rows, N 256, K 7168
// 41.6 or 42.2 for 38.1.)
constexpr int linear_copies(int rows) { return rows == 256 ? 2 : 3; }

// Rows of a tile, runs that a sum is cut into, and the items (tiles times
// runs) there can be.
struct LinearShape {
  int rows, splits;
  int64_t items;
};

// The shape is the one whose estimated time is least: the CUs make whole rounds
// of items, a tile takes its steps and some time beside them, and a cut sum
// costs a second kernel, 6 us, and its results their way to memory and back, 2.6
// bytes a picosecond.  The times are set so that over 1474 random sizes (1 to
// 8000 rows, 1 to 64 experts, sides of 64 to 8192) the rule's choice takes 1.2 %
// longer than the best of those tried (heights, 1 to 16 runs) on average, and
// 4 % of the sizes more than 10 % longer.
// Measured, us, by rows / runs (the rule's choice first):
//   128 rows, K 7168, N 256 (a router)      64/28 13.4   64/14 13.9   128/28 17.3
//   512 rows of it                          64/16 16.0   64/4 19.7    128/8 24.0
//   32768 rows of it                        128/1 137.0  256/2 157.2  64/1 211.8
//   64 rows, K 8192, N 4096                 64/8 22.8    64/1 59.7    128/4 36.4
//   64 rows, K 1024, N 16384                64/1 14.3    128/1 20.6   64/2 18.3
//   16 rows, K 4096, N 7168                 64/4 18.0    64/8 18.9    128/4 23.0
//   1024 rows, K = N = 1024                 64/1 12.5    128/1 21.3   64/2 16.6
//   512 rows, K = N = 8192                  256/4 84.9   128/2 86.0   64/1 114.6
//   4096 rows, K = N = 4096                 256/1 114.6  128/1 137.8  64/1 227.5
//   1024 rows, 256 experts, K 2048, N 7168  64/1 1230    128/1 1270   256/1 1330
//   416 rows, 34 experts, K 6456, N 816     64/1 83.9    64/2 89.5    128/8 107.3
//   12078 rows, 7 experts, K 1448, N 368    128/1 30.8   64/1 40.4    256/1 43.7
//   wgrad, 1024 rows, N 256, K 8192         64/1 16.0    128/1 24.1   64/2 27.0
//   wgrad, 8192 rows, N 64, K 4096          64/8 21.2    64/4 25.4    64/1 64.4
//   wgrad, 512 rows, N 2048, K 4096         128/1 19.2   64/1 30.3    128/2 50.3
//   wgrad, 56934 rows, 9 experts, 848 x 568 256/2 105.6  128/1 117.2  64/1 179.6
//   wgrad, 3944 rows, 2872 x 4864           256/1 108.0  128/1 140.8  64/1 261.6
constexpr int kLinearHeights[] = {64, 128, 256};

struct LinearWork {
  int64_t tiles[3];   // tiles there may be expected to be with 64, 128 and 256 rows,
  int64_t most[3];    // and at most
  int64_t steps;      // of a tile's sum
  int64_t results;    // float32 values of a run's results,
  int64_t stored;     // and with the bias's sums, which wgrad keeps beside them
  bool wgrad;
};

// By height, in ns: a tile beside its steps, and a step where half of the CUs
// or fewer work, where all do, and both for wgrad.
constexpr int kLinearCosts[][5] = {
    {2000, 430, 440, 460, 550}, {2500, 850, 1050, 950, 1200}, {4000, 1250, 1600, 1400, 1650}};

// `steps` is that of the longest of the runs.
inline int64_t linear_cost_ns(const LinearWork& w, int h, int splits, int steps) {
  const int64_t items = w.tiles[h] * splits;
  const int64_t rounds = (items + kLinearCus - 1) / kLinearCus;
  const int64_t step = kLinearCosts[h][1 + (2 * items > kLinearCus) + 2 * w.wgrad];
  const int64_t join = splits > 1 ? 6000 + splits * w.results * 4 / 2600 : 0;
  return rounds * (steps * step + kLinearCosts[h][0]) + join;
}

inline LinearShape linear_best(const LinearWork& w) {
  LinearShape best = {};
  int64_t cost = -1;
  const uint32_t all = w.steps > 1 ? (uint32_t)w.steps : 1;
  for (int h = 0; h < 3; ++h) {
    const uint32_t least = linear_copies(kLinearHeights[h]) + 1;
    // of the numbers of runs that leave the longest the same steps the smallest
    // costs least, and a run has `least` steps however few it is given
    for (uint32_t s = 1; s <= kLinearMostSplits;) {
      if (s > 1 && s * w.stored * 4 > kLinearMostPartial) break;
      const uint32_t steps = (all + s - 1) / s;
      const int64_t c = linear_cost_ns(w, h, s, steps > least ? steps : least);
      if (cost < 0 || c < cost) {
        cost = c;
        best = {kLinearHeights[h], (int)s, w.most[h] * s};
      }
      if (steps <= least) break;
      s = (all + steps - 2) / (steps - 1);
    }
  }
  return best;
}

// Forward and dgrad: `cols` results a row, sums of `deep`.  `one`: one weight
// for all rows, whose tiles the host can count.  (An expert's last tile counts
// as half; one that holds fewer rows than a tile has one.)
inline LinearShape linear_shape(int64_t rows, int E, int cols, int deep, int64_t results) {
  const int64_t held = E < rows ? E : rows;
  LinearWork w = {};
  for (int h = 0; h < 3; ++h) {
    const int64_t bm = kLinearHeights[h], bn = linear_cols((int)bm), units = (cols + bn - 1) / bn;
    const int64_t half = (2 * rows / bm + held) / 2;
    w.tiles[h] = units * (E == 1 ? (rows + bm - 1) / bm : half > held ? half : held);
    w.most[h] = units * (E == 1 ? (rows + bm - 1) / bm : rows / bm + held);
  }
  w.steps = (deep + kLinearDeep - 1) / kLinearDeep;
  w.results = w.stored = results;
  return linear_best(w);
}

// wgrad: N x K results for each expert, sums over its rows.
inline LinearShape wgrad_shape(int64_t rows, int E, int N, int K) {
  LinearWork w = {};
  for (int h = 0; h < 3; ++h) {
    const int64_t bm = kLinearHeights[h], bn = linear_cols((int)bm);
    w.tiles[h] = w.most[h] = E * ((N + bm - 1) / bm) * ((K + bn - 1) / bn);
  }
  w.steps = (rows / E + kLinearDeep - 1) / kLinearDeep;
  w.results = (int64_t)E * N * K;
  w.stored = (int64_t)E * N * (K + 1LL);
  w.wgrad = true;
  return linear_best(w);
}

}  // namespace ep
