// How the bf16 products' launches cut their work, from sizes alone: plain C++
// without HIP, so that the rules can be checked on any host.
#pragma once

#include <stdint.h>

namespace ep {

constexpr int kLinearCols = 256, kLinearDeep = 64;  // a tile's columns, and places along the sum in a step
constexpr int kLinearCus = 256;                     // compute units that a call's work is cut for

// Steps whose tiles are in LDS or on the way.
constexpr int linear_copies(int rows) { return rows == 256 ? 2 : 3; }

// Rows of a tile, runs that a sum is cut into, and the items (tiles times
// runs) there can be.
struct LinearShape {
  int rows, splits;
  int64_t items;
};

// Rounds of tiles that the compute units make: every expert's last tile is
// taken as half full, and a lone half-full tile is a round.
inline int64_t linear_rounds(int64_t rows, int E, int64_t units, int bm) {
  const int64_t held = E < rows ? E : rows;
  const int64_t tiles = units * (2 * rows / bm + held) / 2;
  return tiles > kLinearCus ? (tiles + kLinearCus - 1) / kLinearCus : 1;
}

// Runs for `tiles` tiles of `steps` steps: enough for every compute unit, of
// at least 4 steps each.
inline int linear_splits(int64_t tiles, int64_t steps) {
  int64_t s = kLinearCus / (tiles > 0 ? tiles : 1);
  if (s > steps / 4) s = steps / 4;
  return s > 1 ? (int)s : 1;
}

// Forward and dgrad: `cols` results a row, sums of `deep`.
inline LinearShape linear_shape(int64_t rows, int E, int cols, int deep) {
  const int64_t units = (cols + kLinearCols - 1) / kLinearCols, held = E < rows ? E : rows;
  LinearShape s;
  s.rows = 8 * linear_rounds(rows, E, units, 256) <= 5 * linear_rounds(rows, E, units, 128) ? 256 : 128;
  const int64_t tiles = (rows / s.rows + held) * units;
  s.splits = linear_splits(tiles, (deep + kLinearDeep - 1) / kLinearDeep);
  s.items = tiles * s.splits;
  return s;
}

// wgrad: N x K results for each expert, sums over its rows.
inline LinearShape wgrad_shape(int64_t rows, int E, int N, int K) {
  const int64_t units = (K + kLinearCols - 1) / kLinearCols;
  auto tiles_of = [&](int bm) { return (int64_t)E * ((N + bm - 1) / bm) * units; };
  auto rounds = [&](int bm) { return (tiles_of(bm) + kLinearCus - 1) / kLinearCus; };
  LinearShape s;
  s.rows = 8 * rounds(256) <= 5 * rounds(128) ? 256 : 128;
  const int64_t tiles = tiles_of(s.rows);
  s.splits = linear_splits(tiles, rows / E / kLinearDeep);
  s.items = tiles * s.splits;
  return s;
}

}  // namespace ep
