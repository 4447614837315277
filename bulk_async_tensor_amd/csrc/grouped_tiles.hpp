// Which rows a workgroup of the experts' products takes: the experts' segments
// cut into tiles of BM rows, found from the offsets on the device (the host
// does not know the counts).  Offsets are clamped to [0, rows] and a segment's
// end to its start, so no offset reaches outside the buffers.
#pragma once

#include "ep_device.hpp"
#include "expert_internal.hpp"

namespace ep {

constexpr int kXcds = 8;              // workgroup i of a grid runs on XCD i % 8
constexpr int kWideMaxBlocks = 512;   // scale blocks along K that the wide kernel holds (K <= 65536)
constexpr int64_t kWideMaxGrid = 1 << 22;  // workgroups of one launch (2^31 threads)

// Tiles there can be: every expert that holds a row may end inside one.
inline int64_t wide_tiles_most(int64_t rows, int E, int bm) { return rows / bm + (E < rows ? E : rows); }

struct Segment {
  int lo, hi;
};
__device__ __forceinline__ Segment segment_of(const int32_t* __restrict__ offsets, int E, int rows, int e) {
  Segment s = {0, 0};
  if (e < E) {
    s.lo = min(max(offsets[e], 0), rows);
    s.hi = min(max(offsets[e + 1], s.lo), rows);
  }
  return s;
}

// A workgroup's rows: expert e, receive rows [r0, r1), and its tile along the
// weight rows.
struct WideTile {
  int e, n;
  int64_t r0, r1;
};

// The tiles, expert by expert and row tile fastest, are cut into 8 runs of
// equal length, one for each XCD: the workgroups that run together on an XCD
// then share an expert's weights and rows in its L2.  Every lane of the wave
// takes part; false for a workgroup past the last tile.
template <int BM>
__device__ __forceinline__ bool find_wide_tile(const int32_t* __restrict__ offsets, int E, int64_t rows, int units_n,
                                               int lane, WideTile* out) {
  int mine = 0;
  for (int e = lane; e < E; e += kWave) {
    const Segment s = segment_of(offsets, E, (int)rows, e);
    mine += (s.hi - s.lo + BM - 1) / BM;
  }
#pragma unroll
  for (int d = kWave / 2; d > 0; d >>= 1) mine += __shfl_xor(mine, d, kWave);
  const int64_t total = (int64_t)__builtin_amdgcn_readfirstlane(mine) * units_n;
  const int64_t run = (total + kXcds - 1) / kXcds;
  const int64_t slot = blockIdx.x / kXcds;
  const int64_t id = (blockIdx.x % kXcds) * run + slot;
  if (slot >= run || id >= total) return false;
  const int want = (int)(id / units_n);  // row tiles before this one's expert are at most this many
  int before = 0;
  for (int e0 = 0; e0 < E; e0 += kWave) {
    const Segment s = segment_of(offsets, E, (int)rows, e0 + lane);
    const int n = (s.hi - s.lo + BM - 1) / BM;
    const int incl = wave_incl_scan(n, lane);
    const uint64_t past = ballot(before + incl > want);
    if (past) {
      const int l = __builtin_ctzll(past);
      const int tiles = __builtin_amdgcn_readlane(n, l);
      const int first = before + __builtin_amdgcn_readlane(incl, l) - tiles;
      const int local = (int)(id - (int64_t)first * units_n);
      out->e = e0 + l;
      out->n = local / tiles;
      const int lo = __builtin_amdgcn_readlane(s.lo, l), hi = __builtin_amdgcn_readlane(s.hi, l);
      out->r0 = (int64_t)lo + (int64_t)(local - out->n * tiles) * BM;
      out->r1 = out->r0 + BM < hi ? out->r0 + BM : hi;
      return true;
    }
    before += __builtin_amdgcn_readlane(incl, kWave - 1);
  }
  return false;
}

}  // namespace ep
