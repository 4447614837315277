// ep_grouped_linear and its gradients: a workgroup of 8 waves computes 256
// columns x BM rows at a time from tiles that both sides' loads bring straight
// into LDS.  (The column side is the one along which results lie in memory:
// b's rows n in the forward product, b's columns in dgrad, a's columns in
// wgrad; the row side the token rows, and in wgrad dy's columns n.)
//
// One step is 64 places along the sum: 32 products of 16 x 16 x 32 for each
// of a wave's 128 x 64 (BM = 256) or 64 x 64 results.  The workgroups stay (one
// per CU; its LDS is full) and run through their tiles as one stream of steps,
// so that the next tile's loads are under way while a tile's last steps and
// its results are done.  A step's tiles lie in one of two or three copies in
// LDS; its one barrier stands where every wave has its last fragments of the
// step in registers and two column tiles' products still to issue: past it the
// copy is free for the loads of the step after next, and the next step's
// fragments are read while those products run.  The stream goes on loading
// past its end (the last tile again), so that the waits can count the loads.
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
// up to the number of copies (a shorter one would be two tiles ahead of its
// results).
//
// Few tiles: the sum is cut into `splits` runs of steps, each an item of its
// own whose float32 results go to the workspace; join_kernel adds them in
// ascending order and does what follows the product.
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

constexpr int kWaves = 8;
constexpr int kCols = kLinearCols;  // columns per workgroup
constexpr int kHalf = kCols / 2;    // the first and the second of them (swiglu: gate and up)
constexpr int kDeep = kLinearDeep;  // places along the sum in a step
constexpr int kStepBytes = 2 * kDeep;
constexpr uint32_t kNowhere = 0x80000000u;  // past every buffer
constexpr int kMostItems = 1 << 30;         // items of a call

template <int BM>
struct Wide {
  static constexpr int WN = BM == 256 ? 2 : 4;  // waves along the columns
  static constexpr int WM = kWaves / WN;        // waves along the rows
  static constexpr int HT = kHalf / 16 / WN;    // column tiles of a wave in each half
  static constexpr int NT = 2 * HT;
  static constexpr int MT = BM / 16 / WM;  // row tiles of a wave
  static constexpr int kT = BM * kStepBytes, kStage = kT + kCols * kStepBytes;  // rows, then columns
  static constexpr int S = linear_copies(BM);  // copies: steps whose tiles are in LDS or on the way
  static constexpr int LT = BM / 64;           // load instructions of a wave a step: rows,
  static constexpr int LW = kCols / 64;        // and columns
};

// A raw buffer of `bytes` at p: loads past its end bring zeros.
__device__ __forceinline__ u32x4 buffer_of(const void* p, int64_t bytes) {
  const uint64_t at = (uint64_t)(uintptr_t)p;
  const uint32_t size = bytes < 0 ? 0u : bytes > 0x7FFFFFFF ? 0x7FFFFFFFu : (uint32_t)bytes;
  u32x4 r = {(uint32_t)at, (uint32_t)(at >> 32) & 0xFFFFu, size, 0x00020000u};
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = (uint32_t)__builtin_amdgcn_readfirstlane((int)r[i]);
  return r;
}

// Buffer load straight to LDS: every lane's 16 bytes from its own offset land at
// lds + 16 * lane.  Written as an instruction because the compiler, which
// cannot tell the copies of an array apart, would wait for all of them before
// any LDS read; the barriers below wait for the ones that are due.  It has no
// result registers, and the next instruction may change the address registers.
// The s_nop covers M0 and buffer registers that a vector instruction has just
// written (5 wait states).
__device__ __forceinline__ void load16_to_lds(const u32x4& buf, uint32_t lds, uint32_t offset, uint32_t base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds), "v"(offset),
               "s"(buf), "s"(base)
               : "memory");
}

// Every wave's loads but its newest N have landed, and its LDS accesses are
// done.  vmcnt retires in issue order.
template <int N>
__device__ __forceinline__ void step_barrier() {
  constexpr int imm = (N & 0xF) | (0x7 << 4) | ((N >> 4) << 14);  // vmcnt(N), lgkmcnt(0)
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(imm);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// An item of a workgroup's stream: expert, first column, rows [r0, r1) and
// steps [k0, k0 + steps) of run `split` of its sum.
struct Item {
  int e, c0, split;
  int64_t r0, r1;
  int64_t lo, hi;  // wgrad: the expert's token rows
  int k0, steps;
};

__device__ __forceinline__ Segment linear_segment(const LinearArgs& g, int e) {
  if (!g.offsets) return Segment{0, (int)g.rows};
  // (scalar loads: a vector load would wait for every load in flight)
  typedef const __attribute__((address_space(4))) int32_t* scalar_i32;
  const scalar_i32 at = (scalar_i32)(uintptr_t)(g.offsets + e);
  Segment s;
  s.lo = min(max(at[0], 0), (int)g.rows);
  s.hi = min(max(at[1], s.lo), (int)g.rows);
  return s;
}

// The sum of eight bf16 values, added to v pair by pair in float32.
__device__ __forceinline__ float add_places(bf16x8 f, float v) {
  const bf16x2 one = {(__bf16)1.0f, (__bf16)1.0f};
#pragma unroll
  for (int i = 0; i < 8; i += 2) v = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{f[i], f[i + 1]}, one, v, false);
  return v;
}

struct Frag {  // 64 places of 16 rows (columns): those of chunk `quad` and of chunk quad + 4
  bf16x8 lo, hi;
};

template <Product P, int ACT, int BM>
__device__ __forceinline__ void linear_wide(const LinearArgs& g, const LinearShape& shape) {
  using W = Wide<BM>;
  constexpr int HT = W::HT, NT = W::NT, MT = W::MT;
  constexpr bool kRowsAcross = P == kWgrad, kColsAcross = P != kForward;
  __shared__ __attribute__((aligned(1024))) uint8_t s_rows[W::S * W::kStage];
  __shared__ int32_t s_first[kMaxExperts + 1];
  const int lane = lane_id(), wave = wave_in_group();
  const int col = lane & 15, quad = lane >> 4;
  const int wn = wave % W::WN, wm = wave / W::WN;
  constexpr bool pair = P == kForward && ACT == EP_ACT_SWIGLU;
  const int outs = P == kForward ? (pair ? g.N / 2 : g.N) : g.K;  // columns there are
  const int per_unit = pair ? kHalf : kCols;
  const int units = (outs + per_unit - 1) / per_unit;
  const int64_t rld = P == kForward ? g.K : g.N, cld = g.K;  // values of a row in memory

  // ---- the items of this workgroup
  const int un = (g.N + BM - 1) / BM;  // wgrad: tiles along the weight rows
  int tiles;
  if constexpr (P == kWgrad) {
    tiles = g.E * un;
  } else {
    if (wave == 0) {
      if (g.offsets) first_tiles<BM>(g.offsets, g.E, (int)g.rows, lane, s_first);
      else if (lane < 2) s_first[lane] = lane ? (int32_t)((g.rows + BM - 1) / BM) : 0;
    }
    __syncthreads();
    tiles = __builtin_amdgcn_readfirstlane(s_first[g.E]);
  }
  // (as many as the host counts where offsets ascend; no more where they do not)
  const int products = min(tiles, kMostItems / (units * shape.splits)) * units, total = products * shape.splits;
  const int slots = gridDim.x / kXcds;
  const int xcd = blockIdx.x % kXcds;
  int turn_no = blockIdx.x / kXcds;
  // Forward and dgrad: a run of items for each XCD, whose tiles share weights.
  // wgrad, where an item's cost goes by its expert's rows: runs of 32 in turn.
  const int run = (total + kXcds - 1) / kXcds;
  auto item_no = [&](int i) {
    if constexpr (P == kWgrad) return ((i >> 5) * kXcds + xcd) * 32 + (i & 31);
    return i < run ? xcd * run + i : total;
  };
  int id = item_no(turn_no);
  if (id >= total) return;

  // ---- the loads of the stream
  u32x4 rb, cb;
  Item nxt;
  int lk = 0;  // the step of nxt that loads next
  // A lane's place in a load: of 8 rows along the sum, or of 1 KiB of rows across it.
  const int chunk = (lane & 7) ^ (lane >> 3);
  constexpr int kRowUnits = BM / 8, kColUnits = kHalf / 8;  // 16-byte units in an LDS row across the sum
  auto across = [&](int units16, int64_t ld, int i) -> uint32_t {  // offset of load i of a side across the sum
    const int ri = kWave / units16;  // rows of a load
    const int r = wave * 8 + i * ri + lane / units16, u = lane % units16;
    const int f = ((r & 3) | (wave & 3) << 2) & (units16 / 2 - 1);
    return (uint32_t)(r * ld * 2) + (((u >> 1) ^ f) * 2 + (u & 1)) * 16;
  };
  uint32_t r_at[kRowsAcross ? W::LT : 1], c_at[kColsAcross ? W::LW : 1];
  if constexpr (kRowsAcross) {
#pragma unroll
    for (int i = 0; i < W::LT; ++i) r_at[i] = across(kRowUnits, rld, i);
  } else {
    r_at[0] = (uint32_t)((lane >> 3) * rld * 2) + chunk * 16;
  }
  if constexpr (kColsAcross) {
#pragma unroll
    for (int j = 0; j < W::LW; ++j) c_at[j] = across(kColUnits, cld, j % (W::LW / 2)) + j / (W::LW / 2) * kHalf * 2;
  } else {
    c_at[0] = (uint32_t)((lane >> 3) * cld * 2) + chunk * 16;
  }
  const int64_t deep = P == kForward ? g.K : g.N;  // (not wgrad)
  // lanes past the end of the sum's last step
  const uint32_t late = chunk * 8 >= (int)(deep % kDeep) ? kNowhere : 0u;
  int half1 = 0;  // forward: weight row of the second half's first
  const uint8_t *rbase, *cbase;
  int64_t rleft, cleft;
  auto aim = [&]() {
    nxt.split = shape.splits > 1 ? (int)((uint32_t)id / (uint32_t)products) : 0;
    const uint32_t p = id - nxt.split * products;
    int all;  // steps of the whole sum
    if constexpr (P == kWgrad) {
      const uint32_t tile = p / (uint32_t)units;
      nxt.c0 = (int)(p - tile * units) * kCols;
      nxt.e = (int)(tile / (uint32_t)un);
      nxt.r0 = (int)(tile - nxt.e * un) * BM;
      nxt.r1 = nxt.r0 + BM < g.N ? nxt.r0 + BM : g.N;
      const Segment s = linear_segment(g, nxt.e);
      nxt.lo = s.lo, nxt.hi = s.hi;
      all = (int)((nxt.hi - nxt.lo + kDeep - 1) / kDeep);
    } else {
      // two rounds of 64 and 16 comparisons find the expert
      const int q = (int)(p / (uint32_t)units);
      const int base = 16 * __builtin_popcountll(ballot(s_first[min((lane + 1) * 16, g.E)] <= q));
      const int e = base + __builtin_popcountll(ballot(lane < 16 && s_first[min(base + lane + 1, g.E)] <= q));
      const int before = __builtin_amdgcn_readfirstlane(s_first[e]);
      const int mine = __builtin_amdgcn_readfirstlane(s_first[e + 1]) - before;
      const uint32_t local = p - (uint32_t)before * units, unit = local / (uint32_t)mine;
      const Segment s = linear_segment(g, e);
      nxt.e = e;
      nxt.c0 = (int)unit * per_unit;
      nxt.r0 = s.lo + (int64_t)(local - unit * mine) * BM;
      nxt.r1 = nxt.r0 + BM < s.hi ? nxt.r0 + BM : s.hi;
      all = (int)((deep + kDeep - 1) / kDeep);
    }
    nxt.k0 = 0, nxt.steps = all;
    if (shape.splits > 1) {
      nxt.k0 = (int)((uint32_t)all * (uint32_t)nxt.split / (uint32_t)shape.splits);
      nxt.steps = (int)((uint32_t)all * (uint32_t)(nxt.split + 1) / (uint32_t)shape.splits) - nxt.k0;
    }
    if constexpr (P == kWgrad) {
      // every step its own buffers: the token rows that are left
      rbase = static_cast<const uint8_t*>(g.rows_in) + ((nxt.lo + (int64_t)nxt.k0 * kDeep) * rld + nxt.r0) * 2;
      cbase = static_cast<const uint8_t*>(g.cols_in) + ((nxt.lo + (int64_t)nxt.k0 * kDeep) * cld + nxt.c0) * 2;
      const int64_t rows_left = min(nxt.hi, nxt.lo + (int64_t)(nxt.k0 + nxt.steps) * kDeep) - nxt.lo - (int64_t)nxt.k0 * kDeep;
      rleft = (rows_left * rld - nxt.r0) * 2;
      cleft = (rows_left * cld - nxt.c0) * 2;
    } else {
      // rows past the segment's end are past the buffer: they bring zeros, and their results are never stored
      rb = buffer_of(static_cast<const uint8_t*>(g.rows_in) + nxt.r0 * rld * 2, (nxt.r1 - nxt.r0) * rld * 2);
      cbase = static_cast<const uint8_t*>(g.cols_in) + (int64_t)nxt.e * g.N * g.K * 2;
      if constexpr (P == kForward) {
        cb = buffer_of(cbase, (int64_t)g.N * g.K * 2);
        half1 = pair ? outs + nxt.c0 : nxt.c0 + kHalf;
      } else {
        cleft = ((int64_t)g.N * g.K - (int64_t)nxt.k0 * kDeep * cld - nxt.c0) * 2;
        cbase += ((int64_t)nxt.k0 * kDeep * cld + nxt.c0) * 2;
      }
    }
  };
  uint32_t mask = 0, base_k = 0;
  // What the loads of step lk share.  Sides across the sum: the buffer moves along.
  auto begin_step = [&]() {
    const int k = nxt.k0 + lk;
    if constexpr (!kRowsAcross) {
      mask = lk >= nxt.steps ? kNowhere : (int64_t)(k + 1) * kDeep > deep ? late : 0u;
      base_k = (uint32_t)__builtin_amdgcn_readfirstlane(k * kStepBytes);
    } else {
      rb = buffer_of(rbase, rleft);
      rbase += kDeep * rld * 2;
      rleft -= kDeep * rld * 2;
    }
    if constexpr (kColsAcross) {
      cb = buffer_of(cbase, lk >= nxt.steps ? 0 : cleft);
      cbase += kDeep * cld * 2;
      cleft -= kDeep * cld * 2;
    }
  };
  const uint32_t rows0 = lds_addr_of(s_rows);
  constexpr int kLoads = W::LT + W::LW;
  auto load = [&](int copy, int i0, int i1) {  // loads [i0, i1) of step lk
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if (i < i0 || i >= i1) continue;
      const uint32_t stage = rows0 + copy * W::kStage;
      if (i < W::LT) {
        const uint32_t lds = stage + wave * (W::kT / kWaves) + i * 1024;
        if constexpr (kRowsAcross) load16_to_lds(rb, lds, r_at[i], 0);
        else load16_to_lds(rb, lds, (r_at[0] + (uint32_t)((wave * (BM / kWaves) + i * 8) * rld * 2)) | mask, base_k);
      } else {
        const int j = i - W::LT, h = j / (W::LW / 2);
        if constexpr (kColsAcross) {
          load16_to_lds(cb, stage + W::kT + h * kHalf * kStepBytes + wave * (kHalf * kStepBytes / kWaves) +
                                j % (W::LW / 2) * 1024,
                        c_at[j], 0);
        } else {
          const int r = wave * (kHalf / kWaves) + j % (W::LW / 2) * 8;
          const int row = (h ? half1 : nxt.c0) + r;
          load16_to_lds(cb, stage + W::kT + (h * kHalf + r) * kStepBytes, (c_at[0] + (uint32_t)(row * cld * 2)) | mask,
                        base_k);
        }
      }
    }
  };

  // ---- the products
  f32x4 acc[NT][MT] = {};
  float bacc[P == kWgrad ? MT : 1] = {};  // wgrad: the sums of dy alone, this lane's places
  const uint32_t off0 = col * kStepBytes + ((quad ^ (col & 7)) * 16);
  const uint32_t off1 = col * kStepBytes + (((quad + 4) ^ (col & 7)) * 16);
  auto along_frag = [&](uint32_t rows) {
    typedef __attribute__((address_space(3))) bf16x8 lds_bf16x8;
    Frag f;
    f.lo = *(lds_bf16x8*)(uintptr_t)(rows + off0);
    f.hi = *(lds_bf16x8*)(uintptr_t)(rows + off1);
    return f;
  };
  // tile `t` of 16 columns of a side across the sum, `width` columns wide
  auto across_frag = [&](uint32_t side, int width, int t) {
    const int f = ((col >> 2) | quad << 2) & (width / 16 - 1);
    const uint32_t at = side + (quad * 8 + (col >> 2)) * width * 2 + ((t ^ f) * 32) + (col & 3) * 8;
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
  auto col_frag = [&](uint32_t stage, int n) {
    const uint32_t half = stage + W::kT + n / HT * kHalf * kStepBytes;
    const int t = wn * HT + n % HT;
    if constexpr (kColsAcross) return across_frag(half, kHalf, t);
    else return along_frag(half + t * 16 * kStepBytes);
  };
  auto row_frag = [&](uint32_t stage, int m) {
    if constexpr (kRowsAcross) return across_frag(stage, BM, wm * MT + m);
    else return along_frag(stage + (wm * MT + m) * 16 * kStepBytes);
  };

  Item cur;
  int kb = 0;
  bool more = true, sums = false;
  Frag t[MT], w[4];
  // A step has two barriers.  Before the first, ahead of column tile kOpen,
  // every wave has read the step's rows and the first half of its columns: the
  // loads of the step S ahead into those places start behind it (X), two with
  // each column tile's products.  Before the second, ahead of tile NT - 2, the
  // second half is read too, and its loads follow (Y).  Each load has S - 1/2
  // steps until it is waited for: X of the next step at the second barrier, Y
  // of this step at the first, with (S - 1) * kLoads newer loads on the way.
  constexpr int kX = W::LT + W::LW / 2, kOpen = HT - 2;
  static_assert(2 * (NT - 2 - kOpen) >= kX && W::LW / 2 <= 4, "the loads are out before the next barrier");
  // The products of column tiles [N0, N1) of the step in `stage`, and loads
  // [i0, i1) into it.  The fragments of the tile two ahead are read meanwhile,
  // those of the next step from its copy; and each row tile's of the next step
  // once its last product has started.  The scheduling barriers keep this order.
  auto multiply = [&](uint32_t stage, uint32_t next, int N0, int N1, int copy, int i0, int i1) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (n < N0 || n >= N1) continue;
      __builtin_amdgcn_sched_barrier(0);
      load(copy, i0 + 2 * (n - N0), i0 + 2 * (n - N0) + 2 < i1 ? i0 + 2 * (n - N0) + 2 : i1);
      w[(n + 2) & 3] = n + 2 < NT ? col_frag(stage, n + 2) : col_frag(next, n + 2 - NT);
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[n][m] = mfma_bf16(w[n & 3].lo, t[m].lo, acc[n][m]);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        acc[n][m] = mfma_bf16(w[n & 3].hi, t[m].hi, acc[n][m]);
        if (n == NT - 1) {
          if constexpr (P == kWgrad)
            if (sums) {
              bacc[m] = add_places(t[m].lo, bacc[m]);
              bacc[m] = add_places(t[m].hi, bacc[m]);
            }
          t[m] = row_frag(next, m);
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  // Lane (col, quad) holds columns 4 quad .. + 3 of each column tile of row col
  // of each row tile.
  auto finish = [&]() {
    const int held = (int)(cur.r1 - cur.r0);
    if constexpr (P == kWgrad)
      if (sums)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          bacc[m] += __shfl_xor(bacc[m], 16, kWave);
          bacc[m] += __shfl_xor(bacc[m], 32, kWave);
        }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int lr = (wm * MT + m) * 16 + col;
      if (lr >= held) continue;
      const int64_t r = cur.r0 + lr;
      if (P == kWgrad && sums && wn == 0) {
        float* to = shape.splits > 1 ? g.partial + (int64_t)shape.splits * g.E * g.N * g.K +
                                           (int64_t)cur.split * g.E * g.N
                                     : g.dbias;
        if (quad == 0) to[(int64_t)cur.e * g.N + r] = bacc[m];
      }
      if (shape.splits > 1) {
        // [split][row][weight row or column]
        const int64_t wide = P == kForward ? g.N : g.K;
        const int64_t row = P == kWgrad ? (int64_t)cur.e * g.N + r : r;
        const int64_t many = P == kWgrad ? (int64_t)g.E * g.N : g.rows;
        float* to = g.partial + (cur.split * many + row) * wide;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int i = (n < HT ? 0 : kHalf) + (wn * HT + n % HT) * 16 + 4 * quad;
          const int c = pair ? (n < HT ? cur.c0 + i : outs + cur.c0 + i - kHalf) : cur.c0 + i;
          const bool in = pair ? cur.c0 + (wn * HT + n % HT) * 16 + 4 * quad < outs : c < outs;
          if (in) *reinterpret_cast<f32x4*>(to + c) = acc[n][m];
        }
        continue;
      }
      if (pair) {
#pragma unroll
        for (int n = 0; n < HT; ++n) {
          const int c = cur.c0 + (wn * HT + n) * 16 + 4 * quad;
          if (c < outs) finish_swiglu(g, cur.e, r, c, acc[n][m], acc[HT + n][m]);
        }
        continue;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int c = cur.c0 + (n < HT ? 0 : kHalf) + (wn * HT + n % HT) * 16 + 4 * quad;
        if (c >= outs) continue;
        if constexpr (P == kForward) finish_linear<ACT>(g, cur.e, r, c, acc[n][m]);
        if constexpr (P == kDgrad) finish_dgrad<ACT>(g, r, c, acc[n][m]);
        if constexpr (P == kWgrad) finish_wgrad(g, ((int64_t)cur.e * g.N + r) * g.K + c, acc[n][m]);
      }
    }
  };

  aim();
  cur = nxt;
  for (; lk < W::S; ++lk) {
    begin_step();
    load(lk, 0, kLoads);
  }
  step_barrier<0>();
  bool fresh = true;  // the current step is a tile's first
  bool live = false;  // waves past the tile's last row only load
  for (int copy = 0;; copy = copy + 1 == W::S ? 0 : copy + 1) {
    // step kb of the current tile
    const uint32_t stage = rows0 + copy * W::kStage;
    const uint32_t next = rows0 + (copy + 1 == W::S ? 0 : copy + 1) * W::kStage;
    if (fresh) {
      live = wm * MT * 16 < (int)(cur.r1 - cur.r0);
      if constexpr (P == kWgrad) sums = g.dbias && cur.c0 == 0;
      // (every wave: fragments held past a tile's results would cost their registers there)
#pragma unroll
      for (int m = 0; m < MT; ++m) t[m] = row_frag(stage, m);
      w[0] = col_frag(stage, 0);
      w[1] = col_frag(stage, 1);
    }
    if (live) multiply(stage, next, 0, kOpen, copy, 0, 0);
    // A tile's first step finds its loads landed (below), and the results of
    // the tile before still on their way out.
    if (fresh) step_barrier<63>();
    else step_barrier<(W::S - 1) * kLoads>();
    if (lk >= nxt.steps && lk >= W::S) {
      lk = 0;
      const int then = item_no(turn_no + slots);
      more = then < total;
      if (more) {  // (else the stream loads its last tile again)
        turn_no += slots;
        id = then;
      }
      aim();
    }
    begin_step();
    if (live) multiply(stage, next, kOpen, NT - 2, copy, 0, kX);
    else load(copy, 0, kX);
    if (fresh) step_barrier<63>();
    else step_barrier<(W::S - 1) * kLoads>();
    if (live) multiply(stage, next, NT - 2, NT, copy, kX, kLoads);
    else load(copy, kX, kLoads);
    ++lk;
    ++kb;
    fresh = kb >= cur.steps && kb >= W::S;
    if (fresh) {
      wait_vmcnt<0>();  // before the stores: the next tile's first step waits for none of them
      if (live) finish();
      if (!more) break;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[n][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if constexpr (P == kWgrad)
#pragma unroll
        for (int m = 0; m < MT; ++m) bacc[m] = 0.0f;
      cur = nxt;
      kb = 0;
    }
  }
  wait_vmcnt<0>();  // no load may write this workgroup's LDS after its end
}

// One workgroup fills a CU's LDS: two waves per SIMD, 256 registers each.
template <Product P, int ACT, int BM>
__global__ __launch_bounds__(kWaves * kWave) __attribute__((amdgpu_waves_per_eu(2, 2))) void linear_wide_kernel(
    LinearArgs g, LinearShape shape) {
  linear_wide<P, ACT, BM>(g, shape);
}

// ---- the runs of a cut sum, added in order, and what follows the product
constexpr int kJoinWaves = 4, kJoinCols = 4 * kWave;  // a wave takes 256 columns of a row

__device__ __forceinline__ f32x4 join4(const float* p, int64_t stride, int splits) {
  f32x4 v = *reinterpret_cast<const f32x4*>(p);
  for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const f32x4*>(p + s * stride);
  return v;
}

template <Product P, int ACT>
__global__ __launch_bounds__(kJoinWaves * kWave) void join_kernel(LinearArgs g, int splits) {
  const int lane = lane_id();
  constexpr bool pair = P == kForward && ACT == EP_ACT_SWIGLU;
  const int wide = P == kForward ? g.N : g.K, outs = pair ? wide / 2 : wide;
  const int units = (outs + kJoinCols - 1) / kJoinCols;
  const int64_t many = P == kWgrad ? (int64_t)g.E * g.N : g.rows;
  const int64_t stride = many * wide;
  for (int64_t u = (int64_t)blockIdx.x * kJoinWaves + wave_in_group(); u < many * units;
       u += (int64_t)gridDim.x * kJoinWaves) {
    const int64_t r = u / units;
    const int c = (int)(u % units) * kJoinCols + lane * 4;
    if (P == kWgrad && g.dbias && u % units == 0 && lane == 0) {
      const float* p = g.partial + splits * stride + r;
      float v = p[0];
      for (int s = 1; s < splits; ++s) v += p[s * many];
      g.dbias[r] = v;
    }
    int e = 0;
    if (P != kWgrad && g.offsets) {
      if (r < linear_segment(g, 0).lo || r >= linear_segment(g, g.E - 1).hi) continue;  // rows that no expert holds
      // the expert of the row: the offsets after the first that are at most r
      for (int e0 = 0; e0 < g.E; e0 += kWave)
        e += __builtin_popcountll(ballot(e0 + lane < g.E && g.offsets[e0 + lane + 1] <= r));
      e = min(e, g.E - 1);
    }
    if (c >= outs) continue;
    const float* p = g.partial + r * wide + c;
    const f32x4 v = join4(p, stride, splits);
    if constexpr (P == kForward) {
      if constexpr (pair) finish_swiglu(g, e, r, c, v, join4(p + outs, stride, splits));
      else finish_linear<ACT>(g, e, r, c, v);
    } else if constexpr (P == kDgrad) {
      finish_dgrad<ACT>(g, r, c, v);
    } else {
      finish_wgrad(g, r * wide + c, v);
    }
  }
}

template <Product P, int ACT>
hipError_t launch(const Budget& b, const LinearArgs& g, const LinearShape& s, hipStream_t stream) {
  if (s.items > kMostItems) return hipErrorInvalidValue;
  const int grid = stay_grid(b, s.items);
  if (s.rows == 256)
    hipLaunchKernelGGL((linear_wide_kernel<P, ACT, 256>), dim3(grid), dim3(kWaves * kWave), 0, stream, g, s);
  else
    hipLaunchKernelGGL((linear_wide_kernel<P, ACT, 128>), dim3(grid), dim3(kWaves * kWave), 0, stream, g, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || s.splits == 1) return e;
  const int wide = P == kForward ? (ACT == EP_ACT_SWIGLU ? g.N / 2 : g.N) : g.K;
  const int64_t units = (P == kWgrad ? (int64_t)g.E * g.N : g.rows) * ((wide + kJoinCols - 1) / kJoinCols);
  const int64_t most = 8LL * b.device_cus, groups = (units + kJoinWaves - 1) / kJoinWaves;
  hipLaunchKernelGGL((join_kernel<P, ACT>), dim3((uint32_t)(groups < most ? groups : most)), dim3(kJoinWaves * kWave), 0,
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

size_t linear_workspace(int64_t rows, int K, int E, int N, int) {
  const LinearShape s = linear_shape(rows, E, N, K);
  return s.splits > 1 ? (size_t)s.splits * rows * N * 4 : 0;
}
size_t dgrad_workspace(int64_t rows, int K, int E, int N) {
  const LinearShape s = linear_shape(rows, E, K, N);
  return s.splits > 1 ? (size_t)s.splits * rows * K * 4 : 0;
}
size_t wgrad_workspace(int64_t rows, int K, int E, int N) {
  const LinearShape s = wgrad_shape(rows, E, N, K);
  return s.splits > 1 ? (size_t)s.splits * E * N * (K + 1LL) * 4 : 0;
}

hipError_t launch_linear(const Budget& b, const LinearArgs& g, hipStream_t stream) {
  return launch_act<kForward>(b, g, linear_shape(g.rows, g.E, g.N, g.K), stream);
}
hipError_t launch_dgrad(const Budget& b, const LinearArgs& g, hipStream_t stream) {
  return launch_act<kDgrad>(b, g, linear_shape(g.rows, g.E, g.K, g.N), stream);
}
hipError_t launch_wgrad(const Budget& b, const LinearArgs& g, hipStream_t stream) {
  return launch<kWgrad, EP_ACT_NONE>(b, g, wgrad_shape(g.rows, g.E, g.N, g.K), stream);
}

}  // namespace ep
