// ep_grouped_swiglu_fp8: gate and up products of each expert's rows, SiLU(gate)
// * up, and the rounding to 8 bits with a scale for each 128 outputs.
//
// The results are float32 (the scales) and 8-bit values of float32, so the
// sums are float32 throughout: both sides are widened to bf16, where e4m3
// values and their products are exact (the 8-bit matrix instruction's own sums
// are not, see mfma_e4m3).  Widening is vector work, two values an
// instruction, beside a matrix core that hides about two vector instructions
// behind each of its own; so what is widened is shared and reused:
//   - a workgroup of 8 waves takes 128 outputs (128 gate and 128 up rows) x
//     TOKENS token rows; a wave 16 gate and 16 up rows x all token rows.  Its
//     weight rows are its own: they come from memory straight into its
//     registers, two or four steps ahead, and are widened once a step;
//   - the token rows are widened once a workgroup, an eighth by each wave, into
//     LDS (two copies: the next step's are written while this step's are read).
// One step is one block of 128 values; its sums are scaled by token and weight
// scale and added in float32.  A step has one barrier, before its last token
// rows' products: by then every wave has read the step's copy and written its
// share of the other, and the first rows of the next step are read behind
// those products.
//
// The workgroups stay and run through their tiles as one stream of steps, so
// that the next tile's rows are on the way while a tile's last steps and its
// results are done.
//
// 98304 rows, K 7168, I 2048, 64 experts: 5.2 ms, 1.11 PFLOP/s, two thirds of
// what a bf16 library product of 16384^3 reaches (1.6): the matrix cores are
// busy 56 % of the cycles at 1.9 GHz, with 2.4 vector instructions to a matrix
// instruction.  Each wave widening what it uses took 6.4 ms; 32 x 32 products
// 5.6; a check for token tiles past the segment's end in each step 6.1 (the
// branches keep the vector work from running beside the products), so a
// segment's last tile is computed whole.  A tile of one token takes 61 us at
// that K, alone or beside 127 others: 56 steps of 1.1 us, a pace whose cause is
// not known.
//
// LDS rows hold 128 bf16 in 16 chunks of 16 bytes; row r keeps chunk c at place
// c ^ (r & 15), so the 16 rows read together at one chunk cover all banks.
#include "expert_internal.hpp"
#include "expert_shapes.hpp"
#include "fp8_device.hpp"
#include "grouped_tiles.hpp"

namespace ep {

namespace {

constexpr int kWaves = 8;
constexpr int kOuts = 128;      // outputs of a tile: one scale block
constexpr int kRowBytes = 256;  // of a widened row in LDS

template <int TOKENS, int DEPTH>
struct Shape {
  static constexpr int kTiles = TOKENS / 16;
  static constexpr int kLanes = 512 / TOKENS;           // lanes that widen a token row,
  static constexpr int kParts = TOKENS / 32;            // 8 values at a time
  static constexpr int kTokenLoads = (kParts + 1) / 2;  // of 16 values (or of all 8)
  static constexpr int kLoads = 4 + 3 + kTokenLoads;
  static constexpr int kDepth = DEPTH;  // steps whose rows are in registers or on the way: 2 or 4
};

// The bytes a lane brings for a step: 32 of a gate row, 32 of an up row, its
// share of a token row; and the scales of the token, the gate and the up rows.
struct Raw {
  u32x4 w[2][2];
  u32x4 t[2];
  float s, sb[2];
};

// A raw buffer of `bytes` at p: loads past its end bring zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}

__device__ __forceinline__ bf16x8 widen_half(u32x4 f, int h) { return widen8(f[2 * h], f[2 * h + 1]); }

// v in a register of its own.  (Left to share the load's register, the next
// load into it would go to another one and be moved at the loop's end, which
// waits for it there.)
__device__ __forceinline__ float own_copy(float v) {
  float r;
  asm("v_mov_b32 %0, %1" : "=&v"(r) : "v"(v));
  return r;
}

template <int TOKENS, int DEPTH>
__device__ __forceinline__ void swiglu_body(const GroupedArgs& g, int units_n) {
  using S = Shape<TOKENS, DEPTH>;
  constexpr int kTiles = S::kTiles;
  __shared__ __attribute__((aligned(16))) uint8_t s_t[2][TOKENS * kRowBytes];
  __shared__ float s_sa[2][TOKENS];
  __shared__ float s_max[kWaves][TOKENS];
  __shared__ int32_t s_first[EP_MAX_EXPERTS + 1];
  const int lane = lane_id();
  const int wave = wave_in_group();
  const int col = lane & 15, quad = lane >> 4;
  const int K = g.K, KB = scale_blocks(K), N = g.N, NB = scale_blocks(N), outs = N / 2;

  if (wave == 0) first_tiles<TOKENS>(g.offsets, g.E, (int)g.rows, lane, s_first);
  __syncthreads();
  const int64_t total = (int64_t)__builtin_amdgcn_readfirstlane(s_first[g.E]) * units_n;
  const int64_t run = (total + kXcds - 1) / kXcds;
  const int64_t begin = (blockIdx.x % kXcds) * run;
  const int64_t end = begin + run < total ? begin + run : total;
  const int stride = gridDim.x / kXcds;
  int64_t id = begin + blockIdx.x / kXcds;
  if (id >= end) return;

  // the token row that the lane widens a share of
  const int trow = wave * (TOKENS / kWaves) + lane / S::kLanes, tpart = lane % S::kLanes * (8 * S::kParts);
  const uint32_t at_token = (uint32_t)trow * K + tpart;
  const uint32_t at_scale = (uint32_t)trow * KB * 4;
  uint32_t to_lds[S::kParts];
#pragma unroll
  for (int p = 0; p < S::kParts; ++p) to_lds[p] = trow * kRowBytes + (((tpart / 8 + p) ^ (trow & 15)) * 16);
  WideTile cur, nxt;
  __amdgpu_buffer_rsrc_t ra, rb, rs, rw;
  uint32_t at_w[2], at_sb[2];
  int kb = 0, lk = 0;  // the step computed, and the step of nxt that loads next
  bool more = true, done = false;
  auto aim = [&]() {
    find_tile_of<TOKENS>(g.offsets, s_first, g.E, (int)g.rows, units_n, id, lane, &nxt);
    // Rows past the segment's or the weight's end are past the buffers: they
    // bring zeros, and their results are never stored.
    const int64_t held = nxt.r1 - nxt.r0;
    ra = buffer_at(static_cast<const uint8_t*>(g.a) + nxt.r0 * K, held * K);
    rs = buffer_at(g.a_scale + nxt.r0 * KB, held * KB * 4);
    rb = buffer_at(static_cast<const uint8_t*>(g.b) + (int64_t)nxt.e * N * K, (int64_t)N * K);
    rw = buffer_at(g.b_scale + (int64_t)nxt.e * NB * KB, (int64_t)NB * KB * 4);
    const int n = nxt.n * kOuts + wave * 16;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      at_w[h] = (uint32_t)(h * outs + n + col) * K + quad * 16;
      at_sb[h] = (uint32_t)((h * outs + n) / kScaleBlock) * KB * 4;
    }
  };
  auto load_t = [&](Raw& raw, int i) {
    if constexpr (S::kParts > 1) {
      raw.t[i] = __builtin_amdgcn_raw_buffer_load_b128(ra, at_token + i * 16, lk * kScaleBlock, 0);
    } else {
      const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(ra, at_token, lk * kScaleBlock, 0);
      raw.t[0] = u32x4{v[0], v[1], 0u, 0u};
    }
  };
  // Load i of step lk, in the order in which the step before it needs them:
  // where latency bounds the kernel, that is faster than the weights first (one
  // token 68 / 72 us, 4 rows to each of 256 experts 1195 / 1266, 32 rows 1436 /
  // 1523).  Tiles of 128 token rows, which power bounds, are slower with it
  // (128 rows to each expert 2840 / 2580 us, 1536 rows 5455 / 5320).
  auto load = [&](Raw& raw, int i) {
    // 0-3 weights, 4 and 5 tokens, 6 token scale, 7 and 8 weight scales
    constexpr int kWeightsFirst[] = {0, 1, 2, 3, 6, 7, 8, 4, 5}, kAsNeeded[] = {4, 6, 0, 1, 2, 3, 7, 8};
    static_assert(TOKENS == 128 || S::kTokenLoads == 1);
    const int what = TOKENS == 128 ? kWeightsFirst[i] : kAsNeeded[i & 7];
    if (what < 4)
      raw.w[what >> 1][what & 1] =
          __builtin_amdgcn_raw_buffer_load_b128(rb, at_w[what >> 1] + (what & 1) * 64, lk * kScaleBlock, 0);
    else if (what < 6)
      load_t(raw, what - 4);
    else if (what == 6)
      raw.s = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, at_scale, lk * 4, 0));
    else
      raw.sb[what - 7] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rw, at_sb[what - 7], lk * 4, 0));
  };
  // A last block that is not full: the lanes hold other bytes past the row's
  // end (the next row's, or zeros past the buffer), which become zeros here.
  const int full = K / kScaleBlock;
  auto clear_tail = [&](Raw& raw) {
    const int rest = K - full * kScaleBlock;
    const u32x4 none = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      if ((quad + 4 * p) * 16 >= rest) raw.w[0][p] = raw.w[1][p] = none;
      if (p < S::kTokenLoads && tpart + 16 * p >= rest) raw.t[p] = none;
    }
  };
  // 8 values of the lane's share of a token row, into LDS copy `to`.
  auto widen_token = [&](const Raw& raw, int p, int to) {
    *reinterpret_cast<bf16x8*>(s_t[to] + to_lds[p]) = widen_half(raw.t[p >> 1], p & 1);
    if (p == 0) s_sa[to][trow] = raw.s;  // (the row's lanes hold the same)
  };

  // part s of a token row's block: the same values as part s of a weight row's
  uint32_t from_lds[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) from_lds[s] = col * kRowBytes + (((s >> 1) * 8 + quad * 2 + (s & 1)) ^ col) * 16;
  auto token_frag = [&](int from, int m) {
    Bf16Frag f;
#pragma unroll
    for (int s = 0; s < 4; ++s)
      f.part[s] = *reinterpret_cast<const bf16x8*>(s_t[from] + m * 16 * kRowBytes + from_lds[s]);
    return f;
  };

  f32x4 acc[2][kTiles] = {};

  auto finish = [&]() {
    uint8_t* q = static_cast<uint8_t*>(g.y);
    const int held = (int)(cur.r1 - cur.r0);
    const int n = cur.n * kOuts + wave * 16;  // outs % 64 == 0: a wave is inside or outside as a whole
#pragma unroll
    for (int m = 0; m < kTiles; ++m) {
      float top = kAmaxFloor;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v = silu_mul(acc[0][m][i], acc[1][m][i]);
        acc[0][m][i] = v;
        top = fmaxf(top, n < outs ? fabsf(v) : 0.0f);
      }
      top = fmaxf(top, __shfl_xor(top, 16, kWave));
      top = fmaxf(top, __shfl_xor(top, 32, kWave));
      if (quad == 0) s_max[wave][m * 16 + col] = top;
    }
    lds_barrier();
#pragma unroll
    for (int m = 0; m < kTiles; m += 4) {
      uint32_t d[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (m + j >= kTiles) {
          d[j] = 0u;
          continue;
        }
        const int r = (m + j) * 16 + col;
        float top = s_max[0][r];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) top = fmaxf(top, s_max[w][r]);
        const float inv = block_inverse(top);
        const f32x4 v = acc[0][m + j];
        d[j] = pack_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
        if (wave == 0 && quad == 0 && r < held)
          g.y_scale[(cur.r0 + r) * scale_blocks(outs) + cur.n] = block_scale(top);
      }
      // four token tiles: after two exchanges lane quad j holds its token of tile j, all 16 outputs
      const u32x2 e0 = swap_rows32(d[0], d[2]), e1 = swap_rows32(d[1], d[3]);
      const u32x2 f0 = swap_rows16(e0[0], e1[0]), f1 = swap_rows16(e0[1], e1[1]);
      const int r = (m + quad) * 16 + col;
      if (m + quad < kTiles && r < held && n < outs)
        *reinterpret_cast<u32x4*>(q + (cur.r0 + r) * outs + n) = u32x4{f0[0], f0[1], f1[0], f1[1]};
    }
  };

  Bf16Frag t;  // the first token rows of the step
  float sa;
  float sb[2];  // the step's weight scales
  // Step kb of the current tile, from w and LDS copy `here`; `mine` is free,
  // `other` holds the next step's rows, which become wo and the other copy.
  auto step = [&](Raw& mine, Raw& other, Bf16Frag (&w)[2], Bf16Frag (&wo)[2], int here) {
    const bool last = kb + 1 == KB;
    const float sb0 = sb[0], sb1 = sb[1];
    if (!last && kb + 1 == full) clear_tail(other);
    if (lk == KB) {
      lk = 0;
      id += stride;
      more = id < end;
      if (!more) id -= stride;  // the stream loads its last tile again
      aim();
    }
    f32x4 p0, p1;
    float s0, s1;
#pragma unroll
    for (int m = 0; m < kTiles; ++m) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < S::kLoads; ++i)
        if (i * kTiles / S::kLoads == m) load(mine, i);
      const Bf16Frag now = t;
      const float sn = sa;
      if (m == kTiles - 1) lds_barrier();  // the other copy is written, and this one read
      t = token_frag(m + 1 < kTiles ? here : here ^ 1, (m + 1) % kTiles);
      sa = s_sa[m + 1 < kTiles ? here : here ^ 1][(m + 1) % kTiles * 16 + col];
      f32x4 c0 = {0.0f, 0.0f, 0.0f, 0.0f}, c1 = c0;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        c0 = mfma_bf16(w[0].part[s], now.part[s], c0);
        c1 = mfma_bf16(w[1].part[s], now.part[s], c1);
      }
      if (m < S::kParts) widen_token(other, m, here ^ 1);
      if (m == kTiles - 1) {
        sb[0] = own_copy(other.sb[0]);
        sb[1] = own_copy(other.sb[1]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e * kTiles / 8 == m) wo[e >> 2].part[e & 3] = widen_half(other.w[e >> 2][(e >> 1) & 1], e & 1);
      if (m > 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[0][m - 1][i] = fmaf(p0[i], s0, acc[0][m - 1][i]);
          acc[1][m - 1][i] = fmaf(p1[i], s1, acc[1][m - 1][i]);
        }
      }
      __builtin_amdgcn_sched_group_barrier(0x100, 5, 0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
      }
      p0 = c0;
      p1 = c1;
      s0 = sn * sb0;
      s1 = sn * sb1;
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[0][kTiles - 1][i] = fmaf(p0[i], s0, acc[0][kTiles - 1][i]);
      acc[1][kTiles - 1][i] = fmaf(p1[i], s1, acc[1][kTiles - 1][i]);
    }
    ++lk;
    ++kb;
    if (last) {
      finish();
      done = !more;
#pragma unroll
      for (int m = 0; m < kTiles; ++m) acc[0][m] = acc[1][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      cur = nxt;
      kb = 0;
    }
  };

  Raw raw[S::kDepth];
  Bf16Frag w[2][2];
  aim();
  cur = nxt;
#pragma unroll
  for (int d = 0; d < S::kDepth; ++d) {
    __builtin_amdgcn_sched_barrier(0);  // (in order: the waits count them)
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) load(raw[d], i);
    ++lk;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) w[0][e >> 2].part[e & 3] = widen_half(raw[0].w[e >> 2][(e >> 1) & 1], e & 1);
#pragma unroll
  for (int p = 0; p < S::kParts; ++p) widen_token(raw[0], p, 0);
  sb[0] = raw[0].sb[0];
  sb[1] = raw[0].sb[1];
  lds_barrier();
  t = token_frag(0, 0);
  sa = s_sa[0][col];
  // One way out: with one after each step, the loads on the way would differ at
  // the place where they meet, and the compiler's waits go by the fewest.  The
  // up to kDepth - 1 steps past the end redo the last tile's first ones and
  // store nothing (a tile has more steps than that).
  do {
    step(raw[0], raw[1], w[0], w[1], 0);
    if constexpr (S::kDepth == 2) {
      step(raw[1], raw[0], w[1], w[0], 1);
    } else {
      step(raw[1], raw[2], w[1], w[0], 1);
      step(raw[2], raw[3], w[0], w[1], 0);
      step(raw[3], raw[0], w[1], w[0], 1);
    }
  } while (!done);
}

// Two waves per SIMD, 256 registers each.
template <int TOKENS, int DEPTH>
__global__ __launch_bounds__(kWaves * kWave) __attribute__((amdgpu_waves_per_eu(2, 2))) void grouped_swiglu_kernel(
    GroupedArgs g, int units_n) {
  swiglu_body<TOKENS, DEPTH>(g, units_n);
}

template <int TOKENS, int DEPTH>
hipError_t launch(const Budget& b, const GroupedArgs& g, hipStream_t stream) {
  const int units_n = (g.N / 2 + kOuts - 1) / kOuts;
  const int grid = stay_grid(b, wide_tiles_most(g.rows, g.E, TOKENS) * units_n);
  hipLaunchKernelGGL((grouped_swiglu_kernel<TOKENS, DEPTH>), dim3(grid), dim3(kWaves * kWave), 0, stream, g, units_n);
  return hipGetLastError();
}

}  // namespace

bool grouped_swiglu_fits(const GroupedArgs& g) { return scale_blocks(g.K) >= kSwigluLeastBlocks; }

hipError_t launch_grouped_swiglu(const Budget& b, const GroupedArgs& g, hipStream_t stream) {
  const SwigluShape s = swiglu_shape(g.rows, g.E, scale_blocks(g.K));
  switch (s.tokens) {
    case 32: return s.depth == 4 ? launch<32, 4>(b, g, stream) : launch<32, 2>(b, g, stream);
    case 64: return s.depth == 4 ? launch<64, 4>(b, g, stream) : launch<64, 2>(b, g, stream);
    default: return launch<128, 2>(b, g, stream);
  }
}

}  // namespace ep
