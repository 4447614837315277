// ep_grouped_linear and its gradients: a workgroup of 8 waves computes 256
// columns x 128 or 256 rows at a time, one of 4 waves 128 x 64 where there is
// little to do, from tiles that both sides' loads bring straight into LDS.  (The
// column side is the one along which results lie in memory: b's rows n in the
// forward product, b's columns in dgrad, a's columns in wgrad; the row side the
// token rows, and in wgrad dy's columns n.)
//
// One step is 64 places along the sum: 64 products of 16 x 16 x 32 for each
// of a wave's 128 x 64 results (256 rows), 32 for 64 x 64, 16 for 64 x 32.  The
// workgroups stay (one per CU; its LDS is full, or half full) and run through
// their tiles as one stream of steps, so that the next tile's loads are under
// way while a tile's last steps and its results are done.  A step's tiles lie in one of two or three copies
// in LDS, and each part of a copy is loaded anew as soon as every wave has read
// it (see the two barriers of a step below).  The stream goes on loading past
// its end (the last tile again), so that the waits can count the loads.
//
// What bounds it (kernel times; clock and counters with the profiler beside).
// 49152 rows, 64 experts, K 7168, I 2048, with SwiGLU and the values before it
// kept: 2.62 ms, 1.10 PFLOP/s, 69 % of what a bf16 library product of 16384^3
// reaches (1.59).  The clock is down to 1.88 GHz under this load, and the matrix
// cores are busy 56 % of its cycles: a step takes 2500 to 2900 for 2048 of
// products, and a tile's results and first step 9000 to 13000 and 4000 more.
// 35 % of the L2 requests miss and bring 8.3 GB; experts of equal rows, where
// 27 % do and bring 5.4 GB, take 2.30 ms.  The down product's gradient 1.52 ms,
// 0.95 PFLOP/s (its tiles read and write 512 KiB beside the product, at the same
// time on all CUs: results and first step 22000 to 28000 cycles and 11000 to
// 15000 more, of a tile's 340000); its weights' gradient 1.59 ms, 0.91 PFLOP/s
// (steps of 3300 to 4400 cycles, both sides turned, and 9000 of a tile's 57000
// on its results and its first step).  A decode batch's down product reads its
// weights at 6.4 TB/s: 64 rows with 128 columns 1165 us, 128 with 256 1217.
//
// A side that lies along the sum in memory (its rows are the tile's rows) has
// LDS rows of 128 bytes, 8 chunks of 16; row r keeps chunk c at place
// c ^ (r & 7).  A side that lies across it has one LDS row for each of the 64
// places (the column side one for each half of the columns), chunks of 32
// bytes: the 16 columns of one product tile.  Row r keeps chunk c at place
// c ^ (r % 4 + 4 * (r / 8 % 4)), or the low bits of that where a row has 8
// chunks, and ds_read_b64_tr_b16 turns four rows of 16 columns into four places
// along the sum for each lane: the 16 rows that one such read touches spread
// over all banks.  The loads write LDS in lane order, so both exchanges are
// made in the address each lane loads from.
//
// A sum's end inside a step: lanes whose places lie past it load from past the
// buffer, which brings zeros.  The same holds for steps that only fill a tile
// up to the number of copies and one.
//
// Few tiles: the sum is cut into `splits` runs of steps, each an item of its
// own whose float32 results go to the workspace; join_kernel adds them in a
// fixed order and does what follows the product.
#include "ep.h"
#include "ep_device.hpp"
#include "fp8_device.hpp"
#include "grouped_tiles.hpp"
#include "linear_epilogue.hpp"
#include "linear_shapes.hpp"

namespace ep {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

enum Product { kForward, kDgrad, kWgrad };

constexpr int kDeep = kLinearDeep;  // places along the sum in a step
constexpr int kStepBytes = 2 * kDeep;
constexpr uint32_t kNowhere = 0x80000000u;  // past every buffer
constexpr int kMostItems = kLinearMostItems;

template <int BM>
struct Wide {
  static constexpr int kCols = linear_cols(BM);  // columns per workgroup
  static constexpr int kHalf = kCols / 2;        // the first and the second of them (swiglu: gate and up)
  static constexpr int kWaves = BM == 64 ? 4 : 8;
  static constexpr int WN = BM == 128 ? 4 : 2;   // waves along the columns
  static constexpr int WM = kWaves / WN;         // waves along the rows
  static constexpr int HT = kHalf / 16 / WN;     // column tiles of a wave in each half
  static constexpr int NT = 2 * HT;
  static constexpr int MT = BM / 16 / WM;  // row tiles of a wave
  static constexpr int kT = BM * kStepBytes, kStage = kT + kCols * kStepBytes;  // rows, then columns
  static constexpr int S = linear_copies(BM);  // copies: steps whose tiles are in LDS or on the way
  static constexpr int kLeast = S + 1;         // steps of a tile: the loads are S steps and one tile ahead at most
  static constexpr int LT = BM / 8 / kWaves;     // load instructions of a wave a step: rows,
  static constexpr int LW = kCols / 8 / kWaves;  // and columns
};

// A raw buffer of `bytes` at p: loads past its end bring zeros, stores go nowhere.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes > 0x7FFFFFFF ? 0x7FFFFFFF : (int)bytes,
                                           0x00020000);
}

// Buffer loads straight to LDS: every lane's 16 bytes from its own offset land
// at lds + 16 * lane, those of the second load of a pair kNext bytes further.
// Written as instructions because the compiler, which cannot tell the copies of
// an array apart, would wait for all of them before any LDS read; the barriers
// below wait for the ones that are due.  They have no result registers, and the
// next instruction may change the address registers.  The s_nop covers M0 and
// buffer registers that a vector instruction has just written (5 wait states).
template <int kNext>
__device__ __forceinline__ void load16_pair_to_lds(const u32x4& buf, uint32_t lds, uint32_t offset0, uint32_t offset1,
                                                   uint32_t base) {
  asm volatile(
      "s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %3, %4 offen lds\n\t"
      "s_add_u32 m0, %0, %5\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, %4 offen lds" ::"s"(lds),
      "v"(offset0), "v"(offset1), "s"(buf), "s"(base), "i"(kNext)
      : "memory", "scc");
}

// Every wave's LDS accesses are done, and the loads that it has waited for are
// there for all (wait_vmcnt<N>: all but its newest N; vmcnt retires in issue
// order).
__device__ __forceinline__ void step_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// An item of a workgroup's stream: expert, first column, rows [r0, r1) and
// steps [k0, k0 + steps) of run `split` of its sum.
struct Item {
  int e, c0, split;
  int r0, r1;
  int lo, hi;  // wgrad: the expert's token rows
  int k0, steps;
};

__device__ __forceinline__ Segment linear_segment(const LinearArgs& g, int e) {
  return g.offsets ? segment_of(g.offsets, (int)g.rows, e) : Segment{0, (int)g.rows};
}

// The sum of eight bf16 values, added to v pair by pair in float32.
__device__ __forceinline__ float add_places(bf16x8 f, float v) {
  const bf16x2 one = {(__bf16)1.0f, (__bf16)1.0f};
#pragma unroll
  for (int i = 0; i < 8; i += 2) v = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{f[i], f[i + 1]}, one, v, false);
  return v;
}

// Rows of each of the n tiles that r rows are cut into: as even as 16 allows, so
// that workgroups beside each other take the same time and find each other's
// operands in their XCD's L2 (49152 rows of 64 experts, 700 to 840 each, gate
// and up product 2680 us for 3050 with tiles of 256 rows and a rest).
__device__ __forceinline__ int even_rows(int r, int n) {
  return (int)(((uint32_t)r + (uint32_t)n * 16 - 1) / ((uint32_t)n * 16) * 16);
}

// Whether step k of an item is the sum's last, and not full.
__device__ __forceinline__ bool late_step(const Item& t, int k, int deep) {
  return k < t.steps && (t.k0 + k + 1) * kDeep > deep;
}

struct Frag {  // 64 places of 16 rows (columns): those of chunk `quad` and of chunk quad + 4
  bf16x8 lo, hi;
};

template <Product P, int ACT, int BM>
__device__ __forceinline__ void linear_wide(const LinearArgs& g, const LinearShape& shape) {
  using W = Wide<BM>;
  constexpr int HT = W::HT, NT = W::NT, MT = W::MT;
  constexpr int kWaves = W::kWaves, kCols = W::kCols, kHalf = W::kHalf;
  constexpr bool kRowsAcross = P == kWgrad, kColsAcross = P != kForward;
  __shared__ __attribute__((aligned(1024))) uint8_t s_rows[W::S * W::kStage];
  __shared__ int32_t s_first[P == kWgrad ? 1 : kMaxExperts + 1];
  __shared__ Segment s_seg[kMaxExperts];
  const int lane = lane_id(), wave = wave_in_group();
  const int col = lane & 15, quad = lane >> 4;
  const int wn = wave % W::WN, wm = wave / W::WN;
  constexpr bool pair = P == kForward && ACT == EP_ACT_SWIGLU;
  const int outs = P == kForward ? (pair ? g.N / 2 : g.N) : g.K;  // columns there are
  const int per_unit = pair ? kHalf : kCols;
  const int units = (outs + per_unit - 1) / per_unit;
  const int rld = P == kForward ? g.K : g.N, cld = g.K;  // values of a row in memory

  // ---- the items of this workgroup
  const int un = (g.N + BM - 1) / BM;  // wgrad: tiles along the weight rows
  int tiles;
  for (int e = threadIdx.x; e < g.E; e += kWaves * kWave) s_seg[e] = linear_segment(g, e);
  if constexpr (P != kWgrad) {
    if (wave == 0) {
      if (g.offsets) first_tiles<BM>(g.offsets, g.E, (int)g.rows, lane, s_first);
      else if (lane < 2) s_first[lane] = lane ? (int32_t)((g.rows + BM - 1) / BM) : 0;
    }
  }
  __syncthreads();
  if constexpr (P == kWgrad) tiles = g.E * un;
  else tiles = __builtin_amdgcn_readfirstlane(s_first[g.E]);
  // (as many as the host counts where offsets ascend; no more where they do not)
  const int products = min(tiles, kMostItems / (units * shape.splits)) * units, total = products * shape.splits;
  const int slots = gridDim.x / kXcds;
  const int xcd = blockIdx.x % kXcds;
  const int slot = blockIdx.x / kXcds;
  int round = 0;
  // Tiles of 256 rows: every XCD takes as many items as it has workgroups in
  // turn, so that what neighbouring items share passes by all of them within a
  // round (and wgrad's items, whose cost goes by their expert's rows, are spread
  // evenly).  Lower tiles, which mostly read weights: a run of items for each XCD.
  // us, in turn / runs: gate and up product of 49152 rows 2615 / 2695, the down
  // product's gradient 1500 / 1535, a decode batch's down product (64) 1190 /
  // 1165, (128) 1244 / 1222.
  const int run = (total + kXcds - 1) / kXcds;
  auto item_no = [&](int r) {
    if constexpr (P == kWgrad || BM == 256) return (r * kXcds + xcd) * slots + slot;
    const int i = slot + r * slots;
    return i < run ? xcd * run + i : total;
  };
  int id = item_no(0);
  if (id >= total) return;

  // ---- the loads of the stream
  u32x4 rb = {}, cb = {};
  Item nxt;
  int lk = 0;  // the step of nxt that loads next
  // A lane's place in a load: of 8 rows along the sum, or of 1 KiB of rows across it.
  const int chunk = (lane & 7) ^ (lane >> 3);
  constexpr int kRowUnits = BM / 8, kColUnits = kHalf / 8;  // 16-byte units in an LDS row across the sum
  auto across = [&](int units16, int ld, int i) -> uint32_t {  // offset of load i of a side across the sum
    const int ri = kWave / units16;  // rows of a load
    const int r = wave * (kDeep / kWaves) + i * ri + lane / units16, u = lane % units16;
    const int f = ((r & 3) | (r >> 3 & 3) << 2) & (units16 / 2 - 1);
    return (uint32_t)(r * ld * 2) + (((u >> 1) ^ f) * 2 + (u & 1)) * 16;
  };
  uint32_t r_at[W::LT], c_at[W::LW];
#pragma unroll
  for (int i = 0; i < W::LT; ++i)
    r_at[i] = kRowsAcross ? across(kRowUnits, rld, i)
                          : (uint32_t)((wave * (BM / kWaves) + i * 8 + (lane >> 3)) * rld * 2) + chunk * 16;
  // from the first half of the columns to the second
  const uint32_t half = kColsAcross ? kHalf * 2 : (uint32_t)((pair ? outs : kHalf) * cld * 2);
#pragma unroll
  for (int j = 0; j < W::LW; ++j)
    c_at[j] = (kColsAcross ? across(kColUnits, cld, j % 2)
                           : (uint32_t)((wave * (kHalf / kWaves) + j % 2 * 8 + (lane >> 3)) * cld * 2) + chunk * 16) +
              j / 2 * half;
  const int deep = P == kForward ? g.K : g.N;  // (not wgrad)
  // lanes past the end of the sum's last step
  const uint32_t late = chunk * 8 >= deep % kDeep ? kNowhere : 0u;
  bool cut = false;          // the offsets are those of that step
  uint32_t base = 0;         // sides along the sum: of step lk
  uint32_t r_size = 0, c_size = 0;
  uint64_t r_from = 0, c_from = 0;  // sides across the sum: the step's first row,
  int left = 0;                     // and the places that are left
  auto set_buffer = [&](u32x4& b, uint64_t from, uint32_t size) {
    b[0] = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)from);
    b[1] = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(from >> 32));
    b[2] = (uint32_t)__builtin_amdgcn_readfirstlane((int)size);
    b[3] = 0x00020000u;
  };
  // The buffers of step lk, once the item or the step has changed.
  auto set_step = [&]() {
    if constexpr (!kRowsAcross) {
      // a step past the item's end: buffers of no size (and a base of zero, which the range check takes from the size)
      const bool in = lk < nxt.steps;
      base = (uint32_t)__builtin_amdgcn_readfirstlane(in ? (nxt.k0 + lk) * kStepBytes : 0);
      rb[2] = (uint32_t)__builtin_amdgcn_readfirstlane(in ? (int)r_size : 0);
      if constexpr (!kColsAcross) cb[2] = (uint32_t)__builtin_amdgcn_readfirstlane(in ? (int)c_size : 0);
      if (late_step(nxt, lk, deep)) {
        cut = true;
#pragma unroll
        for (int i = 0; i < W::LT; ++i) r_at[i] |= late;
        if constexpr (!kColsAcross)
#pragma unroll
          for (int j = 0; j < W::LW; ++j) c_at[j] |= late;
      }
    }
    if constexpr (kColsAcross) {
      // the rows (places) of this step that there are; past its row's end a
      // last row has other values, whose results are not stored, or the end
      const int rows = max(min(left, kDeep), 0);
      set_buffer(cb, c_from, (uint32_t)max(rows * cld * 2 - nxt.c0 * 2, 0));
      if constexpr (kRowsAcross) set_buffer(rb, r_from, (uint32_t)max(rows * rld * 2 - nxt.r0 * 2, 0));
    }
  };
  auto aim = [&]() {
    nxt.split = shape.splits > 1 ? (int)((uint32_t)id / (uint32_t)products) : 0;
    const uint32_t p = id - nxt.split * products;
    int all;  // steps of the whole sum
    if constexpr (P == kWgrad) {
      const uint32_t tile = p / (uint32_t)units;
      nxt.c0 = (int)(p - tile * units) * kCols;
      nxt.e = (int)(tile / (uint32_t)un);
      const int per = even_rows(g.N, un);
      nxt.r0 = (int)(tile - nxt.e * un) * per;
      nxt.r1 = min(nxt.r0 + per, g.N);
      nxt.lo = __builtin_amdgcn_readfirstlane(s_seg[nxt.e].lo);
      nxt.hi = __builtin_amdgcn_readfirstlane(s_seg[nxt.e].hi);
      all = (nxt.hi - nxt.lo + kDeep - 1) / kDeep;
    } else {
      // two rounds of 64 and 16 comparisons find the expert
      const int q = (int)(p / (uint32_t)units);
      const int base16 = 16 * __builtin_popcountll(ballot(s_first[min((lane + 1) * 16, g.E)] <= q));
      const int e = base16 + __builtin_popcountll(ballot(lane < 16 && s_first[min(base16 + lane + 1, g.E)] <= q));
      const int before = __builtin_amdgcn_readfirstlane(s_first[e]);
      const int mine = __builtin_amdgcn_readfirstlane(s_first[e + 1]) - before;
      const uint32_t local = p - (uint32_t)before * units, unit = local / (uint32_t)mine;
      const int lo = __builtin_amdgcn_readfirstlane(s_seg[e].lo), hi = __builtin_amdgcn_readfirstlane(s_seg[e].hi);
      nxt.e = e;
      nxt.c0 = (int)unit * per_unit;
      // (never more than a tile holds, were the count of tiles cut short)
      const int per = min(even_rows(hi - lo, mine), BM);
      nxt.r0 = lo + (int)(local - unit * mine) * per;
      nxt.r1 = min(nxt.r0 + per, hi);
      all = (deep + kDeep - 1) / kDeep;
    }
    nxt.k0 = 0, nxt.steps = all;
    if (shape.splits > 1) {
      nxt.k0 = (int)((uint32_t)all * (uint32_t)nxt.split / (uint32_t)shape.splits);
      nxt.steps = (int)((uint32_t)all * (uint32_t)(nxt.split + 1) / (uint32_t)shape.splits) - nxt.k0;
    }
    if (cut) {
      cut = false;
#pragma unroll
      for (int i = 0; i < W::LT; ++i) r_at[i] &= kNowhere - 1;
      if constexpr (!kColsAcross)
#pragma unroll
        for (int j = 0; j < W::LW; ++j) c_at[j] &= kNowhere - 1;
    }
    const uint64_t rows_in = (uint64_t)(uintptr_t)g.rows_in, cols_in = (uint64_t)(uintptr_t)g.cols_in;
    const int64_t weight = (int64_t)nxt.e * g.N * g.K;
    if constexpr (P == kWgrad) {
      const int row = nxt.lo + nxt.k0 * kDeep;
      left = min(nxt.hi - row, nxt.steps * kDeep);
      r_from = rows_in + ((int64_t)row * rld + nxt.r0) * 2;
      c_from = cols_in + ((int64_t)row * cld + nxt.c0) * 2;
    } else {
      // rows past the segment's end are past the buffer: they bring zeros, and their results are never stored
      r_size = (uint32_t)((nxt.r1 - nxt.r0) * rld * 2);
      set_buffer(rb, rows_in + (int64_t)nxt.r0 * rld * 2, r_size);
      if constexpr (P == kForward) {
        c_size = (uint32_t)((g.N - nxt.c0) * cld * 2);
        set_buffer(cb, cols_in + (weight + (int64_t)nxt.c0 * cld) * 2, c_size);
      } else {
        left = min(deep - nxt.k0 * kDeep, nxt.steps * kDeep);
        c_from = cols_in + (weight + (int64_t)nxt.k0 * kDeep * cld + nxt.c0) * 2;
      }
    }
  };
  bool more = true;
  auto advance = [&]() {  // to the next step, or the next item's first
    ++lk;
    if constexpr (kColsAcross) {
      c_from += (int64_t)kDeep * cld * 2;
      if constexpr (kRowsAcross) r_from += (int64_t)kDeep * rld * 2;
      left -= kDeep;
    }
    if (lk >= nxt.steps && lk >= W::kLeast) {
      lk = 0;
      const int then = item_no(round + 1);
      more = then < total;
      if (more) {  // (else the stream loads its last tile again)
        ++round;
        id = then;
      }
      aim();
    }
    set_step();
  };
  constexpr int kLoads = W::LT + W::LW;
  constexpr int kRowBytes = W::kT / kWaves, kColBytes = kHalf * kStepBytes / kWaves;  // of a wave's loads
  auto load_rows = [&](uint32_t stage, int i) {  // loads i and i + 1 of the rows
    load16_pair_to_lds<1024>(rb, stage + wave * kRowBytes + i * 1024, r_at[i], r_at[i + 1], kRowsAcross ? 0 : base);
  };
  auto load_cols = [&](uint32_t stage, int h) {  // the loads of half h of the columns
    load16_pair_to_lds<1024>(cb, stage + W::kT + h * kHalf * kStepBytes + wave * kColBytes, c_at[2 * h], c_at[2 * h + 1],
                             kColsAcross ? 0 : base);
  };
  auto load_step = [&](uint32_t stage) {
#pragma unroll
    for (int i = 0; i < W::LT; i += 2) load_rows(stage, i);
    load_cols(stage, 0);
    load_cols(stage, 1);
  };

  // ---- the products
  f32x4 acc[NT][MT] = {};
  float bacc[P == kWgrad ? MT : 1] = {};  // wgrad: the sums of dy alone, this lane's places
  // Addresses of a lane in a step's copy.  Along the sum: chunk quad, and chunk
  // quad + 4, of row col of a wave's first tile.  Across: for each of a wave's
  // tiles (their chunks differ in the bits that are exchanged).
  typedef __attribute__((address_space(3))) bf16x8 lds_bf16x8;
  auto along_at = [&](int h) { return col * kStepBytes + (((quad + 4 * h) ^ (col & 7)) * 16); };
  auto across_at = [&](int width, int t) {
    const int f = ((col >> 2) | quad << 2) & (width / 16 - 1);
    return (quad * 8 + (col >> 2)) * width * 2 + ((t ^ f) * 32) + (col & 3) * 8;
  };
  uint32_t r_lds[kRowsAcross ? MT : 2], c_lds[kColsAcross ? HT : 2];
  if constexpr (kRowsAcross) {
#pragma unroll
    for (int m = 0; m < MT; ++m) r_lds[m] = across_at(BM, m * W::WM + wm);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) r_lds[h] = along_at(h) + wm * 16 * kStepBytes;
  }
  if constexpr (kColsAcross) {
#pragma unroll
    for (int n = 0; n < HT; ++n) c_lds[n] = W::kT + across_at(kHalf, wn * HT + n);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) c_lds[h] = W::kT + along_at(h) + wn * HT * 16 * kStepBytes;
  }
  auto across_frag = [&](uint32_t at, int width) {
    s16x4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_s16x4*)(uintptr_t)(at + ((i >> 1) * 32 + (i & 1) * 4) * width * 2));
    Frag r;
    r.lo = __builtin_bit_cast(bf16x8, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
    r.hi = __builtin_bit_cast(bf16x8, __builtin_shufflevector(v[2], v[3], 0, 1, 2, 3, 4, 5, 6, 7));
    return r;
  };
  auto along_frag = [&](uint32_t lo, uint32_t hi) {
    Frag f;
    f.lo = *(lds_bf16x8*)(uintptr_t)lo;
    f.hi = *(lds_bf16x8*)(uintptr_t)hi;
    return f;
  };
  auto col_frag = [&](uint32_t stage, int n) {
    const uint32_t h = n / HT * kHalf * kStepBytes;
    if constexpr (kColsAcross) return across_frag(stage + c_lds[n % HT] + h, kHalf);
    else return along_frag(stage + c_lds[0] + (h + n % HT * 16 * kStepBytes), stage + c_lds[1] + (h + n % HT * 16 * kStepBytes));
  };
  auto row_frag = [&](uint32_t stage, int m) {
    if constexpr (kRowsAcross) return across_frag(stage + r_lds[m], BM);
    else return along_frag(stage + r_lds[0] + m * W::WM * 16 * kStepBytes, stage + r_lds[1] + m * W::WM * 16 * kStepBytes);
  };

  Item cur;
  bool sums = false;
  Frag t[MT], w[4];
  // A step has two barriers.  Before the first, ahead of column tile kOpen,
  // every wave has read the step's rows and the first half of its columns: the
  // loads of the step S ahead into those places start behind it (X).  Before
  // the second, ahead of tile NT - 2, the second half is read too, and its
  // loads follow (Y).  Each load has S - 1/2 steps until it is waited for: X of
  // the next step at the second barrier, Y of this step at the first, with
  // (S - 1) * kLoads newer loads on the way.
  constexpr int kOpen = HT - 2;
  // The products of column tiles n and n + 1.  The fragments of the two tiles
  // after them are read meanwhile, those of the next step from its copy.  The
  // row tiles go one after another through both column tiles, so that in a
  // step's last pair each can be read anew for the next step as soon as its
  // four products have started.  What else the step has to do (`more_work`, the
  // loads) stands between the products, or the matrix cores would wait for it.
  // `held` row tiles of the wave's MT have rows.
  int held = 0;
  auto multiply = [&](uint32_t stage, uint32_t next, int n, auto more_work) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[(n + 2 + i) & 3] = n + 2 < NT ? col_frag(stage, n + 2 + i) : col_frag(next, n + 2 + i - NT);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (m < held) {
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[n + i][m] = mfma_bf16(w[(n + i) & 3].lo, t[m].lo, acc[n + i][m]);
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[n + i][m] = mfma_bf16(w[(n + i) & 3].hi, t[m].hi, acc[n + i][m]);
        if (n == NT - 2) {
          if constexpr (P == kWgrad)
            if (sums) {
              bacc[m] = add_places(t[m].lo, bacc[m]);
              bacc[m] = add_places(t[m].hi, bacc[m]);
            }
          t[m] = row_frag(next, m);
        }
      }
      more_work(m);
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto nothing = [](int) {};
  constexpr int kXLoads = W::LT / 2 + 1;  // pairs of loads of X: rows, first half of the columns
  auto load_x = [&](uint32_t stage, int i) {
    if (i < W::LT / 2) load_rows(stage, 2 * i);
    else if (i < kXLoads) load_cols(stage, 0);
  };
  // The fewest stores that finish() issues.  They are younger than the loads
  // that a tile's first S steps wait for, which need not wait for them too.
  constexpr int kStores = P == kForward && ACT == EP_ACT_SWIGLU ? NT * MT / 4 : NT * MT / 2;
  constexpr int kNewer = (W::S - 1) * kLoads;
  static_assert(kNewer + kStores <= 63, "vmcnt is a 6-bit field");
  bool stored = false;  // the tile before left results
  // Step kb of the current tile in copy `stage`, the next one in `next`.
  auto step = [&](uint32_t stage, uint32_t next, int kb) {
    if constexpr (kOpen > 0) multiply(stage, next, 0, nothing);
    if (stored && kb < W::S) wait_vmcnt<kNewer + kStores>();
    else wait_vmcnt<kNewer>();
    step_barrier();
    constexpr int kPairs = (NT - 2 - kOpen) / 2, kEach = (kXLoads + kPairs - 1) / kPairs;
#pragma unroll
    for (int q = 0; q < kPairs; ++q)
      multiply(stage, next, kOpen + 2 * q, [&](int m) {
        if (m < kEach) load_x(stage, q * kEach + m);
      });
    if (stored && kb < W::S - 1) wait_vmcnt<kNewer + kStores>();
    else wait_vmcnt<kNewer>();
    step_barrier();
    multiply(stage, next, NT - 2, [&](int m) {
      if (m == 0) load_cols(stage, 1);
      if (m == 1) advance();
    });
  };

  // A tile's results.  Lane (col, quad) holds columns 4 quad .. + 3 of each
  // column tile of row col of each row tile; of two neighbouring tiles in bf16
  // the lanes exchange halves, so that each moves 8 adjacent values.  Rows past
  // the tile's end are past the buffers, columns past the row's get an offset
  // that is.
  // The call's pointers are read from the arguments anew: held through the
  // steps they would take more scalar registers than there are.
  typedef const __attribute__((address_space(4))) LinearArgs* ConstArgs;
  auto finish = [&]() {
    ConstArgs f = (ConstArgs)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(f));
    const int64_t held = cur.r1 - cur.r0;
    const int lr = wm * 16 + col;
    auto rows_of = [&](const void* p, int64_t row, int ld, int size) {
      return buffer_at(static_cast<const uint8_t*>(p) + row * ld * size, held * ld * size);
    };
    // column of the first of a lane's 4 (8) results of column tile n (and n + 1)
    auto column4 = [&](int n) { return (wn * HT + n % HT) * 16 + 4 * quad; };
    auto column8 = [&](int n) { return (wn * HT + n % HT) * 16 + 16 * (quad & 1) + 8 * (quad >> 1); };
    auto offset = [&](int m, int ld, int c, int end, int size) {
      return (uint32_t)(((lr + m * (W::WM * 16)) * ld + c) * size) | (c < end ? 0u : kNowhere);
    };
    auto put8 = [&](__amdgpu_buffer_rsrc_t to, uint32_t at, f32x4 a, f32x4 b) {
      const u32x2 x = narrow4(a), y = narrow4(b);
      const u32x2 d0 = swap_rows16(x[0], y[0]), d1 = swap_rows16(x[1], y[1]);
      __builtin_amdgcn_raw_buffer_store_b128(u32x4{d0[0], d1[0], d0[1], d1[1]}, to, at, 0, 0);
    };
    auto get8 = [&](u32x4 v, f32x4& a, f32x4& b) {
      const u32x2 d0 = swap_rows16(v[0], v[2]), d1 = swap_rows16(v[1], v[3]);
      a = widen4(d0[0], d1[0]);
      b = widen4(d0[1], d1[1]);
    };
    auto put4 = [&](__amdgpu_buffer_rsrc_t to, uint32_t at, f32x4 v) {
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), to, at, 0, 0);
    };
    if constexpr (P == kWgrad) {
      if (sums) {
        float* to = shape.splits > 1 ? f->partial + (int64_t)shape.splits * f->E * f->N * f->K +
                                           (int64_t)cur.split * f->E * f->N
                                     : f->dbias;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          bacc[m] += __shfl_xor(bacc[m], 16, kWave);
          bacc[m] += __shfl_xor(bacc[m], 32, kWave);
          if (wn == 0 && quad == 0 && lr + m * (W::WM * 16) < held)
            to[(int64_t)cur.e * f->N + cur.r0 + lr + m * (W::WM * 16)] = bacc[m];
        }
      }
    }
    if (shape.splits > 1) {
      // float32 [split][row][weight row or column]
      const int wide = P == kForward ? f->N : f->K;
      const int64_t row = P == kWgrad ? (int64_t)cur.e * f->N + cur.r0 : cur.r0;
      const int64_t many = P == kWgrad ? (int64_t)f->E * f->N : f->rows;
      const auto to = rows_of(f->partial, cur.split * many + row, wide, 4);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        int c = cur.c0 + column4(n), end = outs;
        if (n >= HT) c += pair ? outs : kHalf, end = pair ? wide : outs;
        if (pair && cur.c0 + column4(n) >= outs) end = 0;
#pragma unroll
        for (int m = 0; m < MT; ++m) put4(to, offset(m, wide, c, end, 4), acc[n][m]);
      }
      return;
    }
    if constexpr (P == kForward) {
      const auto to = rows_of(f->out, cur.r0, outs, f->out_f32 ? 4 : 2);
      const auto res = rows_of(f->residual, cur.r0, outs, 2);
      const auto pre = rows_of(f->pre_out, cur.r0, f->N, 2);
      const auto bias = buffer_at(f->bias + (int64_t)cur.e * f->N, f->bias ? (int64_t)f->N * 4 : 0);
      auto bias4 = [&](int c) {
        return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(bias, c * 4, 0, 0));
      };
      constexpr int kLast = pair ? HT : NT;
      const f32x4 none = {0.0f, 0.0f, 0.0f, 0.0f};
      // (a pair's values are asked for before the results of the pair before it
      // are stored: what is loaded behind stores waits for them)
      u32x4 v[2][MT];
      auto ask = [&](int n) {
        const int c8 = cur.c0 + (n < HT ? 0 : kHalf) + column8(n);
#pragma unroll
        for (int m = 0; m < MT; ++m)
          v[n / 2 % 2][m] = f->residual ? __builtin_amdgcn_raw_buffer_load_b128(res, offset(m, outs, c8, outs, 2), 0, 0)
                                        : u32x4{0u, 0u, 0u, 0u};
      };
      ask(0);
#pragma unroll
      for (int n = 0; n < kLast; n += 2) {
        const int c = cur.c0 + (n < HT ? 0 : kHalf), c4 = c + column4(n), c8 = c + column8(n);
        f32x4 add[2] = {none, none}, add_up[2] = {none, none};
        if (f->bias) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            add[i] = bias4(c4 + i * 16);
            if constexpr (pair) add_up[i] = bias4(c4 + i * 16 + outs);
          }
        }
        if (n + 2 < kLast) ask(n + 2);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          f32x4 z[2], up[2], r[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            z[i] = acc[n + i][m] + add[i];
            if constexpr (pair) up[i] = acc[HT + n + i][m] + add_up[i];
          }
          if (f->pre_out) {
            const uint32_t at = offset(m, f->N, c8, outs, 2);
            put8(pre, at, z[0], z[1]);
            if constexpr (pair) put8(pre, at + outs * 2, up[0], up[1]);
          }
          get8(v[n / 2 % 2][m], r[0], r[1]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            z[i] = activate4<ACT>(z[i]);
            if constexpr (pair) z[i] *= up[i];
            z[i] += r[i];
          }
          if (f->out_f32) {
            put4(to, offset(m, outs, c4, outs, 4), z[0]);
            put4(to, offset(m, outs, c4 + 16, outs, 4), z[1]);
          } else {
            put8(to, offset(m, outs, c8, outs, 2), z[0], z[1]);
          }
        }
      }
    }
    if constexpr (P == kDgrad) {
      const int wide = ACT == EP_ACT_SWIGLU ? 2 * outs : outs;
      const auto to = rows_of(f->out, cur.r0, wide, 2);
      const auto pre = rows_of(f->pre_in, cur.r0, wide, 2);
      // (a pair's values are asked for before the results of the pair before it
      // are stored: what is loaded behind stores waits for them)
      u32x4 v[2][MT], u[2][MT];
      auto ask = [&](int n) {
        const int c8 = cur.c0 + (n < HT ? 0 : kHalf) + column8(n);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const uint32_t at = offset(m, wide, c8, outs, 2);
          v[n / 2 % 2][m] = __builtin_amdgcn_raw_buffer_load_b128(pre, at, 0, 0);
          if constexpr (ACT == EP_ACT_SWIGLU) u[n / 2 % 2][m] = __builtin_amdgcn_raw_buffer_load_b128(pre, at + outs * 2, 0, 0);
        }
      };
      if constexpr (ACT != EP_ACT_NONE) ask(0);
#pragma unroll
      for (int n = 0; n < NT; n += 2) {
        const int c8 = cur.c0 + (n < HT ? 0 : kHalf) + column8(n);
        if constexpr (ACT != EP_ACT_NONE)
          if (n + 2 < NT) ask(n + 2);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const uint32_t at = offset(m, wide, c8, outs, 2);
          f32x4 z[2], up[2];
          if constexpr (ACT != EP_ACT_NONE) get8(v[n / 2 % 2][m], z[0], z[1]);
          if constexpr (ACT == EP_ACT_SWIGLU) {
            get8(u[n / 2 % 2][m], up[0], up[1]);
            put8(to, at, slope4<ACT>(z[0]) * up[0] * acc[n][m], slope4<ACT>(z[1]) * up[1] * acc[n + 1][m]);
            put8(to, at + outs * 2, activate4<ACT>(z[0]) * acc[n][m], activate4<ACT>(z[1]) * acc[n + 1][m]);
          } else if constexpr (ACT != EP_ACT_NONE) {
            put8(to, at, slope4<ACT>(z[0]) * acc[n][m], slope4<ACT>(z[1]) * acc[n + 1][m]);
          } else {
            put8(to, at, acc[n][m], acc[n + 1][m]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if constexpr (P == kWgrad) {
      const auto to = rows_of(f->out, (int64_t)cur.e * f->N + cur.r0, outs, f->out_f32 ? 4 : 2);
#pragma unroll
      for (int n = 0; n < NT; n += 2) {
        const int c = cur.c0 + (n < HT ? 0 : kHalf), c4 = c + column4(n), c8 = c + column8(n);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          if (f->out_f32) {
            put4(to, offset(m, outs, c4, outs, 4), acc[n][m]);
            put4(to, offset(m, outs, c4 + 16, outs, 4), acc[n + 1][m]);
          } else {
            put8(to, offset(m, outs, c8, outs, 2), acc[n][m], acc[n + 1][m]);
          }
        }
      }
    }
  };

  const uint32_t rows0 = lds_addr_of(s_rows), rows_end = rows0 + W::S * W::kStage;
  aim();
  set_step();
  cur = nxt;
  for (int i = 0; i < W::S; ++i) {
    load_step(rows0 + i * W::kStage);
    advance();
  }
  wait_vmcnt<0>();
  step_barrier();
  uint32_t stage = rows0;
  auto after = [&](uint32_t copy) { return copy + W::kStage == rows_end ? rows0 : copy + W::kStage; };
  for (;;) {
    // of the tile's row tiles, every WM-th is the wave's
    held = min(max(((cur.r1 - cur.r0 + 15) / 16 - wm + W::WM - 1) / W::WM, 0), MT);
    if constexpr (P == kWgrad) sums = g.dbias && cur.c0 == 0;
#pragma unroll
    for (int m = 0; m < MT; ++m) t[m] = row_frag(stage, m);
    w[0] = col_frag(stage, 0);
    w[1] = col_frag(stage, 1);
    const int steps = max(cur.steps, W::kLeast);
    for (int kb = 0; kb < steps; ++kb) {
      const uint32_t next = after(stage);
      step(stage, next, kb);
      stage = next;
    }
    if (held > 0) finish();
    stored = held > 0;
    if (!more) break;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[n][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (P == kWgrad)
#pragma unroll
      for (int m = 0; m < MT; ++m) bacc[m] = 0.0f;
    cur = nxt;
  }
  wait_vmcnt<0>();  // no load may write this workgroup's LDS after its end
}

// One workgroup a CU: of 128 and 256 rows it takes 156 and 140 KiB of LDS and
// puts two waves on a SIMD, of 256 registers each; of 64 rows 84 KiB and one
// wave, which may have 512 registers and uses 110 to 150.
template <Product P, int ACT, int BM, int PER_SIMD = Wide<BM>::kWaves / 4>
__global__ __launch_bounds__(Wide<BM>::kWaves * kWave) __attribute__((amdgpu_waves_per_eu(PER_SIMD, PER_SIMD))) void
linear_wide_kernel(LinearArgs g, LinearShape shape) {
  linear_wide<P, ACT, BM>(g, shape);
}

// ---- the runs of a cut sum, added, and what follows the product: a workgroup
// takes 256 columns of a row, a wave every fourth run, eight loads at a time,
// and the waves' sums are added in their order.
constexpr int kJoinWaves = 4, kJoinCols = 4 * kWave;

__device__ __forceinline__ f32x4 join4(const float* p, int64_t stride, int first, int splits) {
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
  for (int s = first; s < splits; s += kJoinWaves) v += *reinterpret_cast<const f32x4*>(p + s * stride);
  return v;
}

template <Product P, int ACT>
__global__ __launch_bounds__(kJoinWaves * kWave) void join_kernel(LinearArgs g, int splits) {
  __shared__ f32x4 s_sum[2][kJoinWaves][kWave];
  const int lane = lane_id(), wave = wave_in_group();
  constexpr bool pair = P == kForward && ACT == EP_ACT_SWIGLU;
  const int wide = P == kForward ? g.N : g.K, outs = pair ? wide / 2 : wide;
  const int units = (outs + kJoinCols - 1) / kJoinCols;
  const int64_t many = P == kWgrad ? (int64_t)g.E * g.N : g.rows;
  const int64_t stride = many * wide;
  for (int64_t u = blockIdx.x; u < many * units; u += gridDim.x) {
    const int64_t r = u / units;
    const int c = (int)(u % units) * kJoinCols + lane * 4;
    int e = 0;
    if (P != kWgrad && g.offsets) {
      if (r < linear_segment(g, 0).lo || r >= linear_segment(g, g.E - 1).hi) continue;  // rows that no expert holds
      // the expert of the row: the offsets after the first that are at most r
      for (int e0 = 0; e0 < g.E; e0 += kWave)
        e += __builtin_popcountll(ballot(e0 + lane < g.E && g.offsets[e0 + lane + 1] <= r));
      e = min(e, g.E - 1);
    }
    const float* p = g.partial + r * wide + c;
    if (c < outs) {
      s_sum[0][wave][lane] = join4(p, stride, wave, splits);
      if constexpr (pair) s_sum[1][wave][lane] = join4(p + outs, stride, wave, splits);
    }
    __syncthreads();
    if (wave == 0 && c < outs) {
      f32x4 v[2];
#pragma unroll
      for (int h = 0; h < (pair ? 2 : 1); ++h) {
        v[h] = s_sum[h][0][lane];
#pragma unroll
        for (int w = 1; w < kJoinWaves; ++w) v[h] += s_sum[h][w][lane];
      }
      if constexpr (pair) finish_swiglu(g, e, r, c, v[0], v[1]);
      else if constexpr (P == kForward) finish_linear<ACT>(g, e, r, c, v[0]);
      else if constexpr (P == kDgrad) finish_dgrad<ACT>(g, r, c, v[0]);
      else finish_wgrad(g, r * wide + c, v[0]);
    }
    if (P == kWgrad && wave == 1 && g.dbias && u % units == 0 && lane == 0) {
      const float* q = g.partial + splits * stride + r;
      float v = q[0];
      for (int s = 1; s < splits; ++s) v += q[s * many];
      g.dbias[r] = v;
    }
    __syncthreads();
  }
}

template <Product P, int ACT>
hipError_t launch(const Budget& b, const LinearArgs& g, const LinearShape& s, hipStream_t stream) {
  const int grid = stay_grid(b, s.items);
  if (s.rows == 256)
    hipLaunchKernelGGL((linear_wide_kernel<P, ACT, 256>), dim3(grid), dim3(Wide<256>::kWaves * kWave), 0, stream, g, s);
  else if (s.rows == 128)
    hipLaunchKernelGGL((linear_wide_kernel<P, ACT, 128>), dim3(grid), dim3(Wide<128>::kWaves * kWave), 0, stream, g, s);
  else
    hipLaunchKernelGGL((linear_wide_kernel<P, ACT, 64>), dim3(grid), dim3(Wide<64>::kWaves * kWave), 0, stream, g, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || s.splits == 1) return e;
  const int wide = P == kForward ? (ACT == EP_ACT_SWIGLU ? g.N / 2 : g.N) : g.K;
  const int64_t units = (P == kWgrad ? (int64_t)g.E * g.N : g.rows) * ((wide + kJoinCols - 1) / kJoinCols);
  const int64_t most = 8LL * b.device_cus;
  hipLaunchKernelGGL((join_kernel<P, ACT>), dim3((uint32_t)(units < most ? units : most)), dim3(kJoinWaves * kWave), 0,
                     stream, g, s.splits);
  return hipGetLastError();
}

template <Product P>
hipError_t launch_act(const Budget& b, const LinearArgs& g, const LinearShape& s, hipStream_t stream) {
  switch (g.act) {
    case EP_ACT_SILU: return launch<P, EP_ACT_SILU>(b, g, s, stream);
    case EP_ACT_GELU: return launch<P, EP_ACT_GELU>(b, g, s, stream);
    case EP_ACT_SWIGLU: return launch<P, EP_ACT_SWIGLU>(b, g, s, stream);
    default: return launch<P, EP_ACT_NONE>(b, g, s, stream);
  }
}

}  // namespace

LinearNeeds linear_needs(int64_t rows, int K, int E, int N) {
  const LinearShape s = linear_shape(rows, E, N, K, rows * N);
  return {s.splits > 1 ? (size_t)s.splits * rows * N * 4 : 0, s.items <= kMostItems};
}
LinearNeeds dgrad_needs(int64_t rows, int K, int E, int N) {
  const LinearShape s = linear_shape(rows, E, K, N, rows * K);
  return {s.splits > 1 ? (size_t)s.splits * rows * K * 4 : 0, s.items <= kMostItems};
}
LinearNeeds wgrad_needs(int64_t rows, int K, int E, int N) {
  const LinearShape s = wgrad_shape(rows, E, N, K);
  return {s.splits > 1 ? (size_t)s.splits * E * N * (K + 1LL) * 4 : 0, s.items <= kMostItems};
}

hipError_t launch_linear(const Budget& b, const LinearArgs& g, hipStream_t stream) {
  return launch_act<kForward>(b, g, linear_shape(g.rows, g.E, g.N, g.K, g.rows * g.N), stream);
}
hipError_t launch_dgrad(const Budget& b, const LinearArgs& g, hipStream_t stream) {
  return launch_act<kDgrad>(b, g, linear_shape(g.rows, g.E, g.K, g.N, g.rows * g.K), stream);
}
hipError_t launch_wgrad(const Budget& b, const LinearArgs& g, hipStream_t stream) {
  return launch<kWgrad, EP_ACT_NONE>(b, g, wgrad_shape(g.rows, g.E, g.N, g.K), stream);
}

}  // namespace ep
