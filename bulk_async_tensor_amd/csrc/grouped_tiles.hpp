// Which rows a workgroup of the experts' products takes: the experts' segments
// cut into tiles of BM rows, found from the offsets on the device (the host
// does not know the counts).  Offsets are clamped to [0, rows] and a segment's
// end to its start, so no offset reaches outside the buffers.
#pragma once

#include "ep.h"
#include "ep_device.hpp"
#include "expert_internal.hpp"

namespace ep {

constexpr int kXcds = 8;             // workgroup i of a grid runs on XCD i % 8
constexpr int kWideMaxBlocks = 128;  // scale blocks along K that the wide kernel holds (K <= 16384)

// Tiles there can be: every expert that holds a row may end inside one.
inline int64_t wide_tiles_most(int64_t rows, int E, int bm) { return rows / bm + (E < rows ? E : rows); }

// Workgroups that stay and share `tiles` tiles: one per CU, the same number on
// each XCD.
inline int stay_grid(const Budget& b, int64_t tiles) {
  int64_t grid = b.device_cus / kXcds * kXcds;
  if (grid > tiles) grid = (tiles + kXcds - 1) / kXcds * kXcds;
  return (int)(grid < kXcds ? kXcds : grid);
}

struct Segment {
  int lo, hi;
};
__device__ __forceinline__ Segment segment_of(const int32_t* __restrict__ offsets, int rows, int e) {
  Segment s;
  s.lo = min(max(offsets[e], 0), rows);
  s.hi = min(max(offsets[e + 1], s.lo), rows);
  return s;
}

// Offsets that ascend give at most rows / BM + E tiles; where they do not, the
// segments overlap and their tiles are counted up to this many.
constexpr int kTilesCap = 1 << 29;

// first[e] = tiles before expert e, first[E] = all of them.  One wave.  (64
// experts' tiles fit 30 bits: BM is 128 or more where there are more than 80
// rows for each expert, 81920 with EP_MAX_EXPERTS of them.)
template <int BM>
__device__ __forceinline__ void first_tiles(const int32_t* __restrict__ offsets, int E, int rows, int lane,
                                            int32_t* first) {
  int before = 0;
  for (int e0 = 0; e0 < E; e0 += kWave) {
    const int e = e0 + lane;
    int n = 0;
    if (e < E) {
      const Segment s = segment_of(offsets, rows, e);
      n = (int)(((int64_t)s.hi - s.lo + BM - 1) / BM);
    }
    const int incl = wave_incl_scan(n, lane);
    if (e < E) first[e] = min(before + incl - n, kTilesCap);
    before = min(before + __builtin_amdgcn_readlane(incl, kWave - 1), kTilesCap);
  }
  if (lane == 0) first[E] = before;
}

// A workgroup's rows: expert e, receive rows [r0, r1), and its tile along the
// weight rows.
struct WideTile {
  int e, n;
  int64_t r0, r1;
};

// Tile number id (below first[E] * units_n), expert by expert and row tile
// fastest: neighbours share an expert's weights, and then its rows.  Two
// rounds of 64 and 16 comparisons find the expert (E <= 1024).  Every lane of
// the wave takes part.
template <int BM>
__device__ __forceinline__ void find_tile_of(const int32_t* __restrict__ offsets, const int32_t* first, int E,
                                             int rows, int units_n, int64_t id, int lane, WideTile* out) {
  static_assert(EP_MAX_EXPERTS <= kWave * 16, "the two rounds cover every expert");
  const int q = (int)(id / units_n);
  const int base = 16 * __builtin_popcountll(ballot(first[min((lane + 1) * 16, E)] <= q));
  const int e = base + __builtin_popcountll(ballot(lane < 16 && first[min(base + lane + 1, E)] <= q));
  const int before = __builtin_amdgcn_readfirstlane(first[e]);
  const int tiles = __builtin_amdgcn_readfirstlane(first[e + 1]) - before;
  const int local = (int)(id - (int64_t)before * units_n);
  // (scalar loads: a vector load would wait for every load in flight)
  typedef const __attribute__((address_space(4))) int32_t* scalar_i32;
  const scalar_i32 at = (scalar_i32)(uintptr_t)(offsets + e);
  const int lo = min(max(at[0], 0), rows), hi = min(max(at[1], lo), rows);
  out->e = e;
  out->n = local / tiles;
  out->r0 = (int64_t)lo + (int64_t)(local - out->n * tiles) * BM;
  out->r1 = out->r0 + BM < hi ? out->r0 + BM : hi;
}

}  // namespace ep
