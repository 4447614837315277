// ep_grouped_gemm_fp8: a workgroup of 8 waves computes 256 weight rows x BM
// token rows at a time from tiles that both sides' loads bring straight into
// LDS.
//
// One step is one block of 128 values, so a step's matrix-core results are
// whole inner sums: each is multiplied by its two scales and added to the
// running sum in float32 on the vector units, beside the matrix cores.
//
// The workgroups stay (one per CU; its LDS is full) and run through their
// tiles as one stream of steps, so that the next tile's loads are under way
// while a tile's last steps and its results are done.  A step's tiles
// lie in one of two or three copies in LDS.  A step has one barrier,
// placed where every wave has its last rows of the step in registers and two
// weight tiles' products still to issue: past it the copy is free and the
// loads of the step after next start, and the next step's tiles, whose loads
// started a step ago, are read while those products run.  (With the barrier at
// the step's end the matrix cores wait for 80 KiB of LDS reads each step.)
// With BM = 128, where the weights' bytes bound the kernel, there are three
// copies and two steps' loads on the way.  The stream goes on loading past its
// end (the last tile again), so that the waits can count the loads.
//
// 98304 rows, K 2048, N 7168, 64 experts: 1.52 ms, 1.90 PFLOP/s, 59 % of what
// an 8-bit library product of 16384^3 reaches, with the matrix cores busy 45 %
// of the cycles at 1.8 GHz.  What is done once a tile (its results, the next
// tile's first rows) takes 180 to 240 us of it: the same number of products
// takes 1738 us at K 1024, 1499 at 2048, 1411 at 4096.  4 rows to each of 256
// experts: 591 us, 6.3 TB/s of weights.
//
// LDS rows are 128 bytes, 8 chunks of 16; row r keeps chunk c at place
// c ^ (r & 7), so the 16 rows that one instruction reads at one chunk fall on
// different banks.  The loads write LDS in lane order, so the exchange is made
// in the address each lane loads from.
#include "expert_internal.hpp"
#include "fp8_device.hpp"
#include "grouped_tiles.hpp"

namespace ep {

namespace {

constexpr int kWideWaves = 8;
constexpr int kWideCols = 256;   // weight rows per workgroup
constexpr int kHalf = 128;       // the first and the second weight rows
constexpr int kStepBytes = 128;  // one block of a row

template <int BM>
struct Wide {
  static constexpr int WN = BM == 256 ? 2 : 4;  // waves along the weight rows
  static constexpr int WM = kWideWaves / WN;    // waves along the token rows
  static constexpr int HT = kHalf / 16 / WN;    // weight tiles of a wave in each half
  static constexpr int MT = BM / 16 / WM;       // token tiles of a wave
  static constexpr int kT = BM * kStepBytes, kStage = kT + kWideCols * kStepBytes;  // token rows, then weight rows
  static constexpr int S = BM == 256 ? 2 : 3;   // copies: steps whose tiles are in LDS or on the way
  static constexpr int SS = BM == 256 ? 8 : 4;  // blocks whose token scales are loaded together
  static constexpr int LS = BM / kWideWaves * SS / kWave;  // load instructions of a wave for them
  static constexpr int LT = BM / kWideWaves / 8;     // load instructions of a wave: token rows,
  static constexpr int LW = kHalf / kWideWaves / 8;  // and weight rows of one half
};

// A raw buffer of `bytes` at p: loads past its end bring zeros.
__device__ __forceinline__ u32x4 buffer_of(const void* p, int64_t bytes) {
  const uint64_t at = (uint64_t)(uintptr_t)p;
  u32x4 r = {(uint32_t)at, (uint32_t)(at >> 32) & 0xFFFFu, (uint32_t)bytes, 0x00020000u};
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = (uint32_t)__builtin_amdgcn_readfirstlane((int)r[i]);
  return r;
}

// Buffer loads straight to LDS: every lane's 16 (or 4) bytes from its own
// offset land at lds + 16 (or 4) * lane.  They are written as instructions
// because the compiler, which cannot tell the copies of an array apart, would
// wait for all of them before any LDS read; the barriers below wait for the
// ones that are due.  They have no result registers, and the next instruction
// may change the address registers.  The s_nop covers M0 and buffer registers
// that a vector instruction has just written (5 wait states).
__device__ __forceinline__ void load16_to_lds(const u32x4& buf, uint32_t lds, uint32_t offset, int base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds), "v"(offset),
               "s"(buf), "s"(base)
               : "memory", "m0");
}
__device__ __forceinline__ void load4_to_lds(const u32x4& buf, uint32_t lds, uint32_t offset, int base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"s"(lds), "v"(offset),
               "s"(buf), "s"(base)
               : "memory", "m0");
}

// Every wave's loads but its newest N have landed (N = 63: any may be on the
// way), and its LDS accesses are done.  vmcnt retires in issue order.
template <int N>
__device__ __forceinline__ void wide_barrier() {
  constexpr int imm = (N & 0xF) | (0x7 << 4) | ((N >> 4) << 14);  // vmcnt(N), lgkmcnt(0)
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(imm);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <int BM>
__device__ __forceinline__ void grouped_wide(const GroupedArgs& g, int units_n) {
  using W = Wide<BM>;
  constexpr int HT = W::HT, MT = W::MT, NT = 2 * HT;
  static_assert(MT == 4, "a wave holds four token tiles");
  __shared__ __attribute__((aligned(1024))) uint8_t s_rows[W::S * W::kStage];
  __shared__ float s_sa[W::S][BM * W::SS];
  __shared__ float s_sb[2][2][kWideMaxBlocks];
  __shared__ int32_t s_first[EP_MAX_EXPERTS + 1];
  const int lane = lane_id();
  const int wave = wave_in_group();
  const int col = lane & 15, quad = lane >> 4;
  const int K = g.K, N = g.N, KB = scale_blocks(K), NB = scale_blocks(N);
  const int wn = wave % W::WN, wm = wave / W::WN;

  // ---- the tiles of this workgroup: a run of them for each XCD
  if (wave == 0) first_tiles<BM>(g.offsets, g.E, (int)g.rows, lane, s_first);
  __syncthreads();
  const int64_t total = (int64_t)__builtin_amdgcn_readfirstlane(s_first[g.E]) * units_n;
  const int64_t run = (total + kXcds - 1) / kXcds;
  const int64_t begin = (blockIdx.x % kXcds) * run;
  const int64_t end = begin + run < total ? begin + run : total;
  const int stride = gridDim.x / kXcds;
  int64_t id = begin + blockIdx.x / kXcds;
  if (id >= end) return;

  // ---- the loads of the stream
  u32x4 ra, rb, rs, rw;
  WideTile nxt;
  int lk = 0, lgroup = 0, ltile = 0;  // the step, scale set and tile parity that loads next
  // A lane's place in a load of 8 rows.  Rows past the segment's or the
  // weight's end are past the buffer's: they bring zeros, and their results
  // are never stored.
  const uint32_t at_row = (uint32_t)(lane >> 3) * K + ((lane & 7) ^ (lane >> 3)) * 16;
  auto first_col = [&](const WideTile& t) { return t.n * kWideCols; };
  auto aim = [&]() {
    find_tile_of<BM>(g.offsets, s_first, g.E, (int)g.rows, units_n, id, lane, &nxt);
    const int64_t held = nxt.r1 - nxt.r0;
    ra = buffer_of(static_cast<const uint8_t*>(g.a) + nxt.r0 * K, held * K);
    rb = buffer_of(static_cast<const uint8_t*>(g.b) + (int64_t)nxt.e * N * K, (int64_t)N * K);
    rs = buffer_of(g.a_scale + nxt.r0 * KB, held * KB * 4);
    rw = buffer_of(g.b_scale + (int64_t)nxt.e * NB * KB, (int64_t)NB * KB * 4);
    // The weight scales of all steps, 64 an instruction, of both halves.
    // (Blocks past the last one bring a neighbour's scale, or zero past the
    // buffer; no step uses them.)
    for (int i = wave; i < 2 * ((KB + 63) / 64); i += kWideWaves) {
      const int which = i % 2, k0 = i / 2 * 64;
      int nb = 2 * nxt.n + which;
      if (nb >= NB) nb = NB - 1;
      load4_to_lds(rw, lds_addr_of(&s_sb[ltile][which][k0]), (k0 + lane) * 4, nb * KB * 4);
    }
  };
  const uint32_t rows0 = lds_addr_of(s_rows);
  auto load_scales = [&]() {  // of steps lk .. lk + SS - 1
    // a lane takes one block's scale of one token: 32 or 16 contiguous bytes a
    // token (one block of 64 tokens at a time would touch a line for each value)
#pragma unroll
    for (int j = 0; j < W::LS; ++j) {
      const int r = wave * (BM / kWideWaves) + j * (kWave / W::SS);
      load4_to_lds(rs, lds_addr_of(&s_sa[lgroup][r * W::SS]),
                   (uint32_t)((r + lane / W::SS) * KB + lane % W::SS) * 4, lk * 4);
    }
    lgroup = lgroup + 1 == W::S ? 0 : lgroup + 1;
  };
  constexpr int kLoads = W::LT + 2 * W::LW;
  auto load = [&](int copy, int i0, int i1) {  // loads [i0, i1) of step lk
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if (i < i0 || i >= i1) continue;
      if (i < W::LT) {
        const int r = wave * (BM / kWideWaves) + i * 8;
        load16_to_lds(ra, rows0 + copy * W::kStage + r * kStepBytes, at_row + (uint32_t)r * K, lk * kStepBytes);
      } else {
        const int h = (i - W::LT) / W::LW, j = (i - W::LT) % W::LW;
        const int r = wave * (kHalf / kWideWaves) + j * 8;
        load16_to_lds(rb, rows0 + copy * W::kStage + W::kT + (h * kHalf + r) * kStepBytes,
                      at_row + (uint32_t)(first_col(nxt) + h * kHalf + r) * K,
                      lk * kStepBytes);
      }
    }
  };

  // ---- the products
  f32x4 acc[NT][MT] = {};
  const int off0 = col * kStepBytes + ((quad ^ (col & 7)) * 16);
  const int off1 = col * kStepBytes + (((quad + 4) ^ (col & 7)) * 16);
  auto frag = [&](const uint8_t* rows) {  // 32 values of a row's block
    const u32x4 lo = *reinterpret_cast<const u32x4*>(rows + off0);
    const u32x4 hi = *reinterpret_cast<const u32x4*>(rows + off1);
    i32x8 f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f[q] = (int)lo[q];
      f[4 + q] = (int)hi[q];
    }
    return f;
  };
  // A last block that is not full: its rows hold other bytes past their end
  // (the next row's, or zeros past the buffer), which become zeros here.
  const int full = K / kStepBytes;
  auto clear_tail = [&](uint8_t* rows, int n) {
    const int first = (K - full * kStepBytes) / 16;
    for (int i = threadIdx.x; i < n * 8; i += kWideWaves * kWave) {
      const int r = i >> 3, c = i & 7;
      if (c >= first) *reinterpret_cast<u32x4*>(rows + r * kStepBytes + ((c ^ (r & 7)) * 16)) = u32x4{0u, 0u, 0u, 0u};
    }
  };

  WideTile cur;
  int kb = 0, cgroup = 0, ctile = 0;
  bool more = true;

  i32x8 t[MT], w[4];
  f32x4 p[4] = {};
  float s0[MT] = {}, s1[MT] = {}, v[MT], v0, v1;
  auto add = [&](int n, int m, f32x4 v) {
    const float sc = n < HT ? s0[m] : s1[m];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][m][i] = fmaf(v[i], sc, acc[n][m][i]);
  };
  auto new_scales = [&]() {
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      s0[i] = v[i] * v0;
      s1[i] = v[i] * v1;
    }
  };
  auto weight_rows = [&](const uint8_t* stage, int n) {
    return stage + W::kT + (wn * HT * 16 + (n < HT ? n * 16 : kHalf + (n - HT) * 16)) * kStepBytes;
  };
  auto token_rows = [&](const uint8_t* stage, int m) { return stage + (wm * MT + m) * 16 * kStepBytes; };
  auto read_scales = [&](int tile, int group, int k) {
    v0 = s_sb[tile][0][k];
    v1 = s_sb[tile][1][k];
#pragma unroll
    for (int m = 0; m < MT; ++m) v[m] = s_sa[group][((wm * MT + m) * 16 + col) * W::SS + k % W::SS];
  };
  // The loads of a step are issued two with each weight tile's products: all
  // at once they would hold the waves up until the memory pipeline has taken
  // 64 KiB, a third of a step, with the matrix cores idle.
  constexpr int kPairs = (kLoads + 1) / 2, kEarly = 2 * 2;  // the first two pairs before the step's end
  static_assert(kPairs <= NT, "the loads are out before the next barrier");
  // The products of weight tiles [N0, N1) of the step in `stage`.  The rows of
  // the weight tile two ahead are read meanwhile, those of the next step from
  // its copy; and each token tile's of the next step once its last product has
  // started.  The scheduling barriers keep this order (left alone, the
  // compiler reads all tiles first and spills).
  //
  // Product number q of a step (weight tile q / 4, token tile q % 4) is scaled
  // and added three products after it started, when the matrix core has
  // finished it: the last three of a step in the next step.
  constexpr int kLag = 3;
  auto products = [&](const uint8_t* stage, const uint8_t* next, int N0, int N1, int copy, bool loads) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (n < N0 || n >= N1) continue;
      __builtin_amdgcn_sched_barrier(0);
      const int pair = n >= NT - 2 ? n - (NT - 2) : n + 2;
      if (pair < kPairs && loads) load(copy, 2 * pair, 2 * pair + 2);
      w[(n + 2) & 3] = n + 2 < NT ? frag(weight_rows(stage, n + 2)) : frag(weight_rows(next, n + 2 - NT));
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int q = n * MT + m, b = (q + NT * MT - kLag) % (NT * MT);
        if (q == kLag) new_scales();  // the last products of the step before are added
        p[q & 3] = mfma_e4m3(w[n & 3], t[m]);
        if (n == NT - 1) t[m] = frag(token_rows(next, m));
        add(b / MT, b % MT, p[b & 3]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto drain = [&]() {  // the products that are not added yet
#pragma unroll
    for (int q = NT * MT - kLag; q < NT * MT; ++q) add(q / MT, q % MT, p[q & 3]);
  };

  auto finish = [&]() {  // the tile's results
    const int n0 = first_col(cur), held = (int)(cur.r1 - cur.r0);
    // lane (col, quad) holds rows 4 quad .. + 3 of each weight tile, token col of each token tile
    uint16_t* y = static_cast<uint16_t*>(g.y);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int r = (wm * MT + m) * 16 + col;
#pragma unroll
      for (int n = 0; n < NT; n += 2) {
        // two neighbouring tiles: lanes exchange so that each holds 8 adjacent
        // outputs.  (Cached stores: a row's 128-byte lines are filled by two
        // of them, and streamed ones wrote 2.06 GB for 1.41, 1644 / 1597 us.)
        const u32x2 d0 = swap_rows16(pack_bf16x2(acc[n][m][0], acc[n][m][1]),
                                     pack_bf16x2(acc[n + 1][m][0], acc[n + 1][m][1]));
        const u32x2 d1 = swap_rows16(pack_bf16x2(acc[n][m][2], acc[n][m][3]),
                                     pack_bf16x2(acc[n + 1][m][2], acc[n + 1][m][3]));
        const int tile = n + (quad & 1);
        const int c = n0 + (n < HT ? 0 : kHalf - HT * 16) + (wn * HT + tile) * 16 + 8 * (quad >> 1);
        if (r < held && c < N)
          *reinterpret_cast<u32x4*>(y + (cur.r0 + r) * N + c) = u32x4{d0[0], d1[0], d0[1], d1[1]};
      }
    }
  };

  aim();
  cur = nxt;
  for (; lk < W::S; ++lk) {
    if (lk % W::SS == 0) load_scales();
    load(lk, 0, kLoads);
  }
  wide_barrier<0>();
  bool fresh = true;  // the current step is a tile's first
  bool live = false;  // waves past the tile's last row only load
  for (int copy = 0, prev = W::S - 1;; prev = copy, copy = copy + 1 == W::S ? 0 : copy + 1) {
    // step kb of the current tile
    uint8_t* const stage = s_rows + copy * W::kStage;
    uint8_t* const next = s_rows + (copy + 1 == W::S ? 0 : copy + 1) * W::kStage;
    if (fresh) {
      live = wm * MT * 16 < (int)(cur.r1 - cur.r0);
      if (live) {
#pragma unroll
        for (int m = 0; m < MT; ++m) t[m] = frag(token_rows(stage, m));
        w[0] = frag(weight_rows(stage, 0));
        w[1] = frag(weight_rows(stage, 1));
        read_scales(ctile, cgroup, kb);
      }
    }
    bool last = false;
    auto turn = [&]() {  // the barrier of the step
      if (!fresh) ++lk;  // the loads that the step before began are all out
      wide_barrier<(W::S - 2) * kLoads>();  // the next step's tiles are here; those after may be on the way
      if (kb + 1 == full && full < KB) {
        clear_tail(next, BM + kWideCols);
        wide_barrier<63>();
      }
      if (lk == KB) {
        lk = 0;
        ltile ^= 1;
        id += stride;
        more = id < end;
        if (!more) id -= stride;  // the stream loads its last tile again
        aim();
      }
      if (lk % W::SS == 0) load_scales();
      ++kb;
      last = kb == KB;
      if (last || kb % W::SS == 0) cgroup = cgroup + 1 == W::S ? 0 : cgroup + 1;
    };
    auto first = [&]() { products(stage, next, 0, NT - 2, prev, !fresh); };
    auto second = [&]() {
      if (!last) read_scales(ctile, cgroup, kb);  // the next step's
      products(stage, next, NT - 2, NT, copy, true);
    };
    auto first_loads = [&]() {
      if (!fresh) load(prev, kEarly, kLoads);
    };
    auto second_loads = [&]() { load(copy, 0, kEarly); };
    if (live) first();
    else first_loads();
    turn();
    if (live) second();
    else second_loads();
    fresh = last;
    if (last) {
      load(copy, kEarly, kLoads);
      ++lk;
      drain();
      finish();
      if (!more) break;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[n][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // nothing is left to add in the next step
        p[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        s1[i] = 0.0f;
      }
      cur = nxt;
      kb = 0;
      ctile ^= 1;
    }
  }
  wait_vmcnt<0>();  // no load may write this workgroup's LDS after its end
}

// One workgroup fills a CU's LDS: two waves per SIMD, 256 registers each.
template <int BM>
__global__ __launch_bounds__(kWideWaves * kWave) __attribute__((amdgpu_waves_per_eu(2, 2))) void grouped_wide_kernel(
    GroupedArgs g, int units_n) {
  grouped_wide<BM>(g, units_n);
}

template <int BM>
hipError_t launch(const Budget& b, const GroupedArgs& g, hipStream_t stream) {
  const int units_n = (g.N + kWideCols - 1) / kWideCols;
  const int grid = stay_grid(b, wide_tiles_most(g.rows, g.E, BM) * units_n);
  hipLaunchKernelGGL(grouped_wide_kernel<BM>, dim3(grid), dim3(kWideWaves * kWave), 0, stream, g, units_n);
  return hipGetLastError();
}

}  // namespace

bool grouped_wide_fits(const GroupedArgs& g, int bm) {
  // (a tile shorter than the copies would be two tiles ahead of its results)
  const int blocks = scale_blocks(g.K);
  return blocks >= (bm == 256 ? Wide<256>::S : Wide<128>::S) && blocks <= kWideMaxBlocks;
}

hipError_t launch_grouped_wide(const Budget& b, const GroupedArgs& g, int bm, hipStream_t stream) {
  return bm == 256 ? launch<256>(b, g, stream) : launch<128>(b, g, stream);
}

}  // namespace ep
