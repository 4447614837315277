// The experts' 8-bit products for experts with many rows: a workgroup of 8
// waves computes 256 weight rows x BM token rows (swiglu: 128 gate and the 128
// up rows of the same outputs) from tiles that both sides' loads bring
// straight into LDS.
//
// One step is one block of 128 values, so a step's matrix-core results are
// whole inner sums: each is multiplied by its two scales and added to the
// running sum in float32 on the vector units, which work beside the matrix
// cores.  Two stages: the next step's tiles (64 KiB at BM = 256) load while
// the current ones are multiplied.
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

typedef __attribute__((address_space(3))) uint8_t lds_byte_t;

constexpr int kWideWaves = 8;
constexpr int kWideCols = 256;   // weight rows per workgroup
constexpr int kStepBytes = 128;  // one block of a row

template <int BM, bool SWIGLU>
struct Wide {
  static constexpr int WN = BM == 256 ? 2 : 4;   // waves along the weight rows
  static constexpr int WM = kWideWaves / WN;     // waves along the token rows
  static constexpr int NT = kWideCols / 16 / WN; // weight tiles of a wave
  static constexpr int MT = BM / 16 / WM;        // token tiles of a wave
  static constexpr int kB = kWideCols * kStepBytes;
  static constexpr int kStage = kB + BM * kStepBytes;
  static_assert(MT == 4, "a wave's token scales are one per lane");
  // first LDS weight row of the wave's tile i
  static __device__ __forceinline__ int row_of(int wn, int i) {
    if (!SWIGLU) return (wn * NT + i) * 16;
    return i < NT / 2 ? (wn * (NT / 2) + i) * 16 : 128 + (wn * (NT / 2) + i - NT / 2) * 16;
  }
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}

template <int BM, bool SWIGLU>
__device__ __forceinline__ void grouped_wide(const GroupedArgs& g, int units_n) {
  using W = Wide<BM, SWIGLU>;
  constexpr int NT = W::NT, MT = W::MT;
  __shared__ __attribute__((aligned(1024))) uint8_t s_stage0[W::kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t s_stage1[W::kStage];
  __shared__ float s_sa0[kWideWaves][kWave], s_sa1[kWideWaves][kWave];
  __shared__ float s_sb[3][kWideMaxBlocks];
  __shared__ float s_max[W::WN][BM];
  const int lane = lane_id();
  const int wave = wave_in_group();
  const int col = lane & 15, quad = lane >> 4;
  const int K = g.K, N = g.N, KB = scale_blocks(K), NB = scale_blocks(N);
  const int outs = SWIGLU ? N / 2 : N;

  WideTile tile;
  if (!find_wide_tile<BM>(g.offsets, g.E, g.rows, units_n, lane, &tile)) return;
  const int n0 = tile.n * (SWIGLU ? kWideCols / 2 : kWideCols);
  const int held = (int)(tile.r1 - tile.r0);
  const int wn = wave % W::WN, wm = wave / W::WN;

  // ---- the loads: each wave brings 32 weight rows and BM / 8 token rows a step, 8 rows an instruction
  const uint8_t* a = static_cast<const uint8_t*>(g.a) + tile.r0 * K;
  const uint8_t* b = static_cast<const uint8_t*>(g.b) + (int64_t)tile.e * N * K;
  const __amdgpu_buffer_rsrc_t ra = buffer_of(a, (int64_t)held * K);
  const __amdgpu_buffer_rsrc_t rb = buffer_of(b, (int64_t)N * K);
  const __amdgpu_buffer_rsrc_t rs = buffer_of(g.a_scale + tile.r0 * KB, (int64_t)held * KB * 4);
  constexpr int LB = kWideCols / kWideWaves / 8, LA = BM / kWideWaves / 8;
  const int chunk = ((lane & 7) ^ (lane >> 3)) * 16;
  uint32_t vb[LB], va[LA], vs;
#pragma unroll
  for (int j = 0; j < LB; ++j) {
    const int r = wave * (kWideCols / kWideWaves) + j * 8 + (lane >> 3);
    int n = SWIGLU ? (r < 128 ? n0 + r : outs + n0 + r - 128) : n0 + r;
    if (n >= N) n = N - 1;  // rows past the end: computed on the last row, never stored
    vb[j] = (uint32_t)n * K + chunk;
  }
#pragma unroll
  for (int j = 0; j < LA; ++j) {
    int r = wave * (BM / kWideWaves) + j * 8 + (lane >> 3);
    if (r >= held) r = held - 1;
    va[j] = (uint32_t)r * K + chunk;
  }
  {
    int r = wm * (MT * 16) + lane;
    if (r >= held) r = held - 1;
    vs = (uint32_t)r * KB * 4;
  }

  // ---- the weight scales of all steps: block rows n0 / 128 and the next; swiglu: one gate and two up rows
  for (int i = threadIdx.x; i < 3 * KB; i += kWideWaves * kWave) {
    const int which = i / KB, kb = i - which * KB;
    int nb = SWIGLU ? (which == 0 ? n0 / kScaleBlock : (outs + n0) / kScaleBlock + which - 1) : n0 / kScaleBlock + which;
    if (nb >= NB) nb = NB - 1;
    s_sb[which][kb] = g.b_scale[((int64_t)tile.e * NB + nb) * KB + kb];
  }
  // the block row of the wave's tiles: plain, its half; swiglu, gate and up
  const int sb0 = SWIGLU ? 0 : wn * NT * 16 / kScaleBlock;
  const int sb1 = SWIGLU ? 1 + ((outs + n0 + wn * (NT / 2) * 16) / kScaleBlock - (outs + n0) / kScaleBlock) : sb0;

  f32x4 acc[NT][MT] = {};
  const int off0 = col * kStepBytes + ((quad ^ (col & 7)) * 16);
  const int off1 = col * kStepBytes + (((quad + 4) ^ (col & 7)) * 16);

  auto load = [&](uint8_t* stage, float* sa, int kb) {
#pragma unroll
    for (int j = 0; j < LB; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rb, (lds_void_t*)(stage + (wave * (kWideCols / kWideWaves) + j * 8) * kStepBytes), 16, vb[j],
          kb * kStepBytes, 0, 0);
#pragma unroll
    for (int j = 0; j < LA; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          ra, (lds_void_t*)(stage + W::kB + (wave * (BM / kWideWaves) + j * 8) * kStepBytes), 16, va[j],
          kb * kStepBytes, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)sa, 4, vs, kb * 4, 0, 0);
  };

  // A fragment: 32 values of a row's block.
  auto frag = [&](const uint8_t* rows) {
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

  // One block: for each weight tile its four products, while the vector units
  // scale and add those of the tile before and the next tile's rows are read.
  // The scheduling barriers keep that order (left alone, the compiler reads
  // all tiles first and spills).
  auto step = [&](const uint8_t* stage, const float* sa, int kb) {
    i32x8 t[MT], w[2];
    float s0[MT], s1[MT];
    f32x4 p[2][MT];
    const uint8_t* wrows = stage + W::row_of(wn, 0) * kStepBytes;
    const uint8_t* trows = stage + W::kB + wm * MT * 16 * kStepBytes;
#pragma unroll
    for (int m = 0; m < MT; ++m) t[m] = frag(trows + m * 16 * kStepBytes);
    w[0] = frag(wrows);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const float v = sa[m * 16 + col];
      s0[m] = v * s_sb[sb0][kb];
      s1[m] = SWIGLU ? v * s_sb[sb1][kb] : s0[m];
    }
#pragma unroll
    for (int n = 0; n <= NT; ++n) {
      __builtin_amdgcn_sched_barrier(0);
      if (n + 1 < NT) w[(n + 1) & 1] = frag(wrows + (W::row_of(0, n + 1) - W::row_of(0, 0)) * kStepBytes);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (n < NT) p[n & 1][m] = mfma_e4m3(w[n & 1], t[m]);
        if (n > 0) {
          const float sc = n - 1 < NT / 2 ? s0[m] : s1[m];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[n - 1][m][i] = fmaf(p[(n - 1) & 1][m][i], sc, acc[n - 1][m][i]);
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  // A last block that is not full: its tiles hold other bytes past the row's
  // end (the next row's, or zeros past the buffer), which become zeros here.
  const int full = K / kStepBytes;
  auto clear_tail = [&](uint8_t* stage) {
    const int first = (K - full * kStepBytes) / 16;
    for (int i = threadIdx.x; i < (kWideCols + BM) * 8; i += kWideWaves * kWave) {
      const int r = i >> 3, c = i & 7;
      if (c >= first) *reinterpret_cast<u32x4*>(stage + r * kStepBytes + ((c ^ (r & 7)) * 16)) = u32x4{0u, 0u, 0u, 0u};
    }
    __syncthreads();
  };

  const bool live = wm * MT * 16 < held;  // waves past the last row only load
  load(s_stage0, s_sa0[wave], 0);
  for (int kb = 0; kb < KB; kb += 2) {
    __syncthreads();
    if (kb + 1 < KB) load(s_stage1, s_sa1[wave], kb + 1);
    if (kb == full) clear_tail(s_stage0);
    if (live) step(s_stage0, s_sa0[wave], kb);
    if (kb + 1 < KB) {
      __syncthreads();
      if (kb + 2 < KB) load(s_stage0, s_sa0[wave], kb + 2);
      if (kb + 1 == full) clear_tail(s_stage1);
      if (live) step(s_stage1, s_sa1[wave], kb + 1);
    }
  }

  // ---- results: lane (col, quad) holds rows 4 quad .. + 3 of each weight tile, token col of each token tile
  if constexpr (!SWIGLU) {
    uint16_t* y = static_cast<uint16_t*>(g.y);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int r = (wm * MT + m) * 16 + col;
      if (r < held) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int c = n0 + W::row_of(wn, n) + 4 * quad;
          if (c < N) {
            const u32x2 o = {pack_bf16x2(acc[n][m][0], acc[n][m][1]), pack_bf16x2(acc[n][m][2], acc[n][m][3])};
            *reinterpret_cast<u32x2*>(y + (tile.r0 + r) * N + c) = o;
          }
        }
      }
    }
  } else {
    uint8_t* y = static_cast<uint8_t*>(g.y);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float top = kAmaxFloor;
#pragma unroll
      for (int n = 0; n < NT / 2; ++n) {
        const bool in = n0 + W::row_of(wn, n) < outs;  // outs % 64 == 0: a tile is inside or outside as a whole
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float v = silu_mul(acc[n][m][i], acc[n + NT / 2][m][i]);
          acc[n][m][i] = v;
          top = fmaxf(top, in ? fabsf(v) : 0.0f);
        }
      }
      top = fmaxf(top, __shfl_xor(top, 16, kWave));
      top = fmaxf(top, __shfl_xor(top, 32, kWave));
      if (quad == 0) s_max[wn][(wm * MT + m) * 16 + col] = top;
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int r = (wm * MT + m) * 16 + col;
      float top = s_max[0][r];
#pragma unroll
      for (int w = 1; w < W::WN; ++w) top = fmaxf(top, s_max[w][r]);
      if (r < held) {
        const float inv = block_inverse(top);
#pragma unroll
        for (int n = 0; n < NT / 2; ++n) {
          const int c = n0 + W::row_of(wn, n) + 4 * quad;
          if (c < outs)
            *reinterpret_cast<uint32_t*>(y + (tile.r0 + r) * outs + c) =
                pack_e4m3x4(acc[n][m][0] * inv, acc[n][m][1] * inv, acc[n][m][2] * inv, acc[n][m][3] * inv);
        }
        if (wn == 0 && quad == 0) g.y_scale[(tile.r0 + r) * scale_blocks(outs) + tile.n] = block_scale(top);
      }
    }
  }
}

// One workgroup fills a CU's LDS: two waves per SIMD, 256 registers each.
template <int BM, bool SWIGLU>
__global__ __launch_bounds__(kWideWaves * kWave) __attribute__((amdgpu_waves_per_eu(2, 2))) void grouped_wide_kernel(
    GroupedArgs g, int units_n) {
  grouped_wide<BM, SWIGLU>(g, units_n);
}

template <int BM, bool SWIGLU>
hipError_t launch(const GroupedArgs& g, hipStream_t stream) {
  const int outs = SWIGLU ? g.N / 2 : g.N, per = SWIGLU ? kWideCols / 2 : kWideCols;
  const int units_n = (outs + per - 1) / per;
  const int64_t want = wide_tiles_most(g.rows, g.E, BM) * units_n;
  const int64_t grid = (want + kXcds - 1) / kXcds * kXcds;
  if (grid > kWideMaxGrid) return hipErrorInvalidValue;
  hipLaunchKernelGGL((grouped_wide_kernel<BM, SWIGLU>), dim3((unsigned)grid), dim3(kWideWaves * kWave), 0, stream, g,
                     units_n);
  return hipGetLastError();
}

}  // namespace

bool grouped_wide_fits(const GroupedArgs& g, bool swiglu, int bm) {
  const int outs = swiglu ? g.N / 2 : g.N, per = swiglu ? kWideCols / 2 : kWideCols;
  return scale_blocks(g.K) <= kWideMaxBlocks &&
         wide_tiles_most(g.rows, g.E, bm) * ((outs + per - 1) / per) <= kWideMaxGrid - kXcds;
}

hipError_t launch_grouped_wide(const GroupedArgs& g, bool swiglu, int bm, hipStream_t stream) {
  if (bm == 256) return swiglu ? launch<256, true>(g, stream) : launch<256, false>(g, stream);
  return swiglu ? launch<128, true>(g, stream) : launch<128, false>(g, stream);
}

}  // namespace ep
