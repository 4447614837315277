// The experts' 8-bit products with block scales (ep_grouped_gemm_fp8 and
// ep_grouped_swiglu_fp8):
//
//   p[r, n] = sum_b sa[r, b] sb[e, n / 128, b] sum_{i in block b} a[r, i] w[e, n, i]
//
// for the rows r that the layout gives expert e, in ascending blocks b.  The
// matrix cores give the inner sum of one whole block for 16 weight rows and 16
// token rows; it is multiplied by the two scales and added in float32.
// grouped_wide.hip holds the plain kernel and grouped_swiglu.hip the fused one;
// here are the choice, the plain kernel for a few rows and the one for the K
// that those do not take.  Weights are the A operand and tokens the B
// operand: a lane's results then belong to ONE token (its column) and four
// adjacent weight rows, so the lane needs one token scale, and the block's
// weight scale is the same for the whole tile.
#include "expert_internal.hpp"
#include "expert_shapes.hpp"
#include "fp8_device.hpp"

#include <type_traits>

namespace ep {

namespace {

// A workgroup's rows: expert e, receive rows [r0, r1).
struct RowTile {
  int e;
  int64_t r0, r1;
};

// Finds tile number `idx` of the experts' rows cut into tiles of BM (expert by
// expert; an expert's last tile may be shorter).  False past the last one.
// Every lane of the wave takes part.  Offsets are clamped to [0, rows].
template <int BM>
__device__ __forceinline__ bool find_tile(const int32_t* __restrict__ offsets, int E, int64_t rows, int64_t idx,
                                          int lane, RowTile* out) {
  int64_t before = 0;
  for (int e0 = 0; e0 < E; e0 += kWave) {
    const int e = e0 + lane;
    int64_t lo = 0, hi = 0;
    if (e < E) {
      lo = offsets[e];
      hi = offsets[e + 1];
      lo = lo < 0 ? 0 : lo > rows ? rows : lo;
      hi = hi < lo ? lo : hi > rows ? rows : hi;
    }
    const int n = (int)((hi - lo + BM - 1) / BM);
    const int incl = wave_incl_scan(n, lane);
    const uint64_t past = ballot(before + incl > idx);
    if (past) {
      const int l = __builtin_ctzll(past);
      const int first = __builtin_amdgcn_readlane(incl - n, l);
      out->e = e0 + l;
      out->r0 = (int64_t)__builtin_amdgcn_readlane((int)lo, l) + (idx - before - first) * BM;
      const int64_t end = __builtin_amdgcn_readlane((int)hi, l);
      out->r1 = out->r0 + BM < end ? out->r0 + BM : end;
      return true;
    }
    before += __builtin_amdgcn_readlane(incl, kWave - 1);
  }
  return false;
}

constexpr int kFewWaves = 4;  // of 16 weight rows each
constexpr int kFewCols = 16 * kFewWaves;
constexpr int kFewRows = 16;
constexpr int kFewDepth = 8;  // blocks on the way

// A few rows against a few experts, plain: too few tiles of the wide kernel to
// reach every CU (64 of them read 39 GB/s of weights each).  Each wave streams
// its 16 weight rows into registers, 8 blocks ahead, against 16 token rows that
// it reads itself (the caches hold them); the waves share nothing, so 64 weight
// rows are a workgroup.  One token, K 7168, N 2048, 8 of 64 experts: 22.5 us,
// 5.2 TB/s.
struct FewRaw {
  u32x4 w[2], t[2];
  float s, sb;
};

__global__ __launch_bounds__(kFewWaves * kWave) void grouped_few_kernel(GroupedArgs g, int units_n) {
  constexpr int D = kFewDepth;
  const int lane = lane_id();
  const int col = lane & 15, quad = lane >> 4;
  const int K = g.K, N = g.N, KB = scale_blocks(K), NB = scale_blocks(N), full = K / kScaleBlock;
  uint16_t* y = static_cast<uint16_t*>(g.y);
  for (int64_t u = blockIdx.x;; u += gridDim.x) {
    RowTile tile;
    if (!find_tile<kFewRows>(g.offsets, g.E, g.rows, u / units_n, lane, &tile)) break;
    const int n0 = (int)(u % units_n) * kFewCols + wave_in_group() * 16;
    if (n0 >= N) continue;
    // rows past the end: computed on the last row, never stored
    const uint8_t* wrow = static_cast<const uint8_t*>(g.b) + ((int64_t)tile.e * N + min(n0 + col, N - 1)) * K;
    const float* wscale = g.b_scale + ((int64_t)tile.e * NB + n0 / kScaleBlock) * KB;
    const int64_t r = tile.r0 + col, token = r < tile.r1 ? r : tile.r1 - 1;
    const uint8_t* trow = static_cast<const uint8_t*>(g.a) + token * K;
    const float* tscale = g.a_scale + token * KB;
    FewRaw raw[D];
    // Block kb (past the last one: the last one again; chunks past the row's end: its last one).
    auto load = [&](FewRaw& f, int kb) {
      kb = min(kb, KB - 1);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int c = min(kb * kScaleBlock + (quad + 4 * p) * 16, K - 16);
        f.w[p] = *reinterpret_cast<const u32x4*>(wrow + c);
        f.t[p] = *reinterpret_cast<const u32x4*>(trow + c);
      }
      f.sb = wscale[kb];
      f.s = tscale[kb];
    };
    auto whole = [](const u32x4 (&v)[2], bool in0, bool in1) {
      i32x8 f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f[q] = in0 ? (int)v[0][q] : 0;
        f[4 + q] = in1 ? (int)v[1][q] : 0;
      }
      return f;
    };
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    // D blocks from kb on; last: those past the row's end add zeros.
    auto group = [&](int kb, auto is_last) {
      constexpr bool kLast = decltype(is_last)::value;
#pragma unroll
      for (int d = 0; d < D; ++d) {
        __builtin_amdgcn_sched_barrier(0);  // (the loads stay in their order: the waits count them)
        const int c = (kb + d) * kScaleBlock + quad * 16;
        const bool in0 = !kLast || c < K, in1 = !kLast || c + 64 < K, in = !kLast || kb + d < KB;
        const f32x4 p = mfma_e4m3(whole(raw[d].w, in0, in1), whole(raw[d].t, in0, in1));
        const float s = in ? raw[d].s * raw[d].sb : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = fmaf(p[i], s, acc[i]);
        if (!kLast) load(raw[d], kb + D + d);
      }
    };
#pragma unroll
    for (int d = 0; d < D; ++d) {
      __builtin_amdgcn_sched_barrier(0);
      load(raw[d], d);
    }
    int kb = 0;
    for (; kb + D <= full; kb += D) group(kb, std::false_type());
    group(kb, std::true_type());
    const int n = n0 + 4 * quad;
    if (r < tile.r1 && n < N)
      *reinterpret_cast<u32x2*>(y + r * N + n) = u32x2{pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3])};
  }
}

constexpr int kNarrowWaves = 8;
constexpr int kNarrowTiles = 4;               // token tiles of 16 per workgroup
constexpr int kNarrowRows = 16 * kNarrowTiles;
constexpr int kNarrowCols = 128;              // swiglu: output columns per workgroup (256 weight rows)

// For the K that the other kernels do not take (swiglu: one scale block; plain:
// one, two with a few rows, or more than the 128 whose weight scales fit in
// LDS): each wave streams two tiles of 16 weight rows from memory straight into
// the matrix cores against up to 64 token rows.  swiglu: the two tiles are the
// gate and the up rows of the same 16 outputs.  Nothing is loaded ahead, which
// long rows pay for, K 16384 (wide, few) against 16400 (this one), N 2048, 8
// experts: one token 42 / 104 us, 32 rows each 101 / 303, 256 each 132 / 648.
template <bool SWIGLU>
__global__ __launch_bounds__(kNarrowWaves * kWave) void grouped_narrow_kernel(GroupedArgs g, int units_n) {
  __shared__ float s_max[kNarrowWaves][kNarrowRows];
  const int lane = lane_id();
  const int wave = wave_in_group();
  const int col = lane & 15, quad = lane >> 4;
  const int K = g.K, N = g.N, KB = scale_blocks(K);
  const int outs = SWIGLU ? N / 2 : N;
  const uint8_t* a = static_cast<const uint8_t*>(g.a);
  const uint8_t* b = static_cast<const uint8_t*>(g.b);
  for (int64_t u = blockIdx.x;; u += gridDim.x) {
    RowTile tile;
    if (!find_tile<kNarrowRows>(g.offsets, g.E, g.rows, u / units_n, lane, &tile)) break;
    const int n0 = (int)(u % units_n) * (SWIGLU ? kNarrowCols : 2 * kNarrowCols) + wave * 16;
    const int nt = (int)((tile.r1 - tile.r0 + 15) / 16);
    int base[2];  // first weight row of each tile
    base[0] = n0;
    base[1] = SWIGLU ? outs + n0 : n0 + kNarrowCols;
    f32x4 acc[2][kNarrowTiles] = {};
    const uint8_t* wrow[2];
    const float* wscale[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      int n = base[h] + col;
      if (n >= N) n = N - 1;  // rows past the end: computed on the last row, never stored
      wrow[h] = b + ((int64_t)tile.e * N + n) * K;
      int nb = base[h] / kScaleBlock;
      if (nb >= scale_blocks(N)) nb = scale_blocks(N) - 1;
      wscale[h] = g.b_scale + ((int64_t)tile.e * scale_blocks(N) + nb) * KB;
    }
    const uint8_t* arow[kNarrowTiles];
    const float* ascale[kNarrowTiles];
#pragma unroll
    for (int m = 0; m < kNarrowTiles; ++m) {
      int64_t r = tile.r0 + m * 16 + col;
      if (r >= tile.r1) r = tile.r1 - 1;
      arow[m] = a + r * K;
      ascale[m] = g.a_scale + r * KB;
    }
    for (int kb = 0; kb < KB; ++kb) {
      i32x8 wv[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int c = kb * kScaleBlock + (quad + 4 * p) * 16;
          u32x4 v = {0u, 0u, 0u, 0u};
          if (c < K) v = *reinterpret_cast<const u32x4*>(wrow[h] + c);
#pragma unroll
          for (int q = 0; q < 4; ++q) wv[h][4 * p + q] = (int)v[q];
        }
#pragma unroll
      for (int m = 0; m < kNarrowTiles; ++m) {
        if (m < nt) {
          i32x8 av;
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const int c = kb * kScaleBlock + (quad + 4 * p) * 16;
            u32x4 v = {0u, 0u, 0u, 0u};
            if (c < K) v = *reinterpret_cast<const u32x4*>(arow[m] + c);
#pragma unroll
            for (int q = 0; q < 4; ++q) av[4 * p + q] = (int)v[q];
          }
          const float sa = ascale[m][kb];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            f32x4 p = {0.0f, 0.0f, 0.0f, 0.0f};
            if constexpr (SWIGLU) {  // float32 sums for float32 results
#pragma unroll
              for (int s = 0; s < 4; ++s)
                p = mfma_bf16(widen8(wv[h][2 * s], wv[h][2 * s + 1]), widen8(av[2 * s], av[2 * s + 1]), p);
            } else {
              p = mfma_e4m3(wv[h], av);
            }
            const float s = sa * wscale[h][kb];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[h][m][i] = fmaf(p[i], s, acc[h][m][i]);
          }
        }
      }
    }
    if constexpr (!SWIGLU) {
      uint16_t* y = static_cast<uint16_t*>(g.y);
#pragma unroll
      for (int m = 0; m < kNarrowTiles; ++m) {
        const int64_t r = tile.r0 + m * 16 + col;
        if (r < tile.r1) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int n = base[h] + 4 * quad;
            if (n < N) {
              const u32x2 o = {pack_bf16x2(acc[h][m][0], acc[h][m][1]), pack_bf16x2(acc[h][m][2], acc[h][m][3])};
              *reinterpret_cast<u32x2*>(y + r * N + n) = o;
            }
          }
        }
      }
    } else {
      uint8_t* y = static_cast<uint8_t*>(g.y);
      const bool in = n0 + 4 * quad < outs;  // outs % 64 == 0: a tile is inside or outside as a whole
#pragma unroll
      for (int m = 0; m < kNarrowTiles; ++m) {
        float top = kAmaxFloor;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float v = silu_mul(acc[0][m][i], acc[1][m][i]);
          acc[0][m][i] = v;
          top = fmaxf(top, in ? fabsf(v) : 0.0f);
        }
        top = fmaxf(top, __shfl_xor(top, 16, kWave));
        top = fmaxf(top, __shfl_xor(top, 32, kWave));
        if (quad == 0) s_max[wave][m * 16 + col] = top;
      }
      __syncthreads();
#pragma unroll
      for (int m = 0; m < kNarrowTiles; ++m) {
        float top = s_max[0][m * 16 + col];
#pragma unroll
        for (int w = 1; w < kNarrowWaves; ++w) top = fmaxf(top, s_max[w][m * 16 + col]);
        const int64_t r = tile.r0 + m * 16 + col;
        if (r < tile.r1 && in) {
          const float inv = block_inverse(top);
          *reinterpret_cast<uint32_t*>(y + r * outs + n0 + 4 * quad) =
              pack_e4m3x4(acc[0][m][0] * inv, acc[0][m][1] * inv, acc[0][m][2] * inv, acc[0][m][3] * inv);
          if (wave == 0 && quad == 0) g.y_scale[r * scale_blocks(outs) + n0 / kScaleBlock] = block_scale(top);
        }
      }
      __syncthreads();
    }
  }
}

}  // namespace

// Whether the wide kernel's tiles leave half of the CUs without one, with a
// tile of 16 rows enough for most experts.  Measured, wide against few: 8 rows
// to 8 of 64 experts, K 7168, N 2048 (64 tiles) 47 / 23 us, K 2048, N 4096 (128)
// 17.9 / 18.4, K 2048, N 7168 (224) 22 / 32; 5 rows to each of 16, K = N = 1024
// (64) 11.2 / 11.1, 10 rows each 11.2 / 19.5.
static bool few_rows(const Budget& b, const GroupedArgs& g) {
  const int64_t units_n = (g.N + 255) / 256, held = g.E < g.rows ? g.E : g.rows;
  return 2 * units_n * held <= b.device_cus && g.rows <= 8 * (int64_t)g.E;
}

// One workgroup for each tile there can be: every expert may end inside one.
static int grid_of(const GroupedArgs& g, int rows, int64_t units_n) {
  const int64_t tiles = g.rows / rows + (g.E < g.rows ? g.E : g.rows), most = 1 << 22;
  return (int)(tiles * units_n < most ? tiles * units_n : most);
}

static hipError_t launch_few(const GroupedArgs& g, hipStream_t stream) {
  const int units_n = (g.N + kFewCols - 1) / kFewCols;
  hipLaunchKernelGGL(grouped_few_kernel, dim3(grid_of(g, kFewRows, units_n)), dim3(kFewWaves * kWave), 0, stream, g,
                     units_n);
  return hipGetLastError();
}

template <bool SWIGLU>
static hipError_t launch_narrow(const GroupedArgs& g, hipStream_t stream) {
  const int outs = SWIGLU ? g.N / 2 : g.N, per = SWIGLU ? kNarrowCols : 2 * kNarrowCols;
  const int units_n = (outs + per - 1) / per;
  hipLaunchKernelGGL(grouped_narrow_kernel<SWIGLU>, dim3(grid_of(g, kNarrowRows, units_n)),
                     dim3(kNarrowWaves * kWave), 0, stream, g, units_n);
  return hipGetLastError();
}

hipError_t launch_grouped_fp8(const Budget& b, const GroupedArgs& g, bool swiglu, hipStream_t stream) {
  if (swiglu) return grouped_swiglu_fits(g) ? launch_grouped_swiglu(b, g, stream) : launch_narrow<true>(g, stream);
  // Two blocks (K <= 256) fit the wide kernel's tiles of 256 rows only.  N 4096,
  // 16 experts, narrow against wide, us: 8 rows each 7.6 / 10.0, 32 each 12.6 /
  // 10.6, 512 each 78 / 32.
  const int bm = scale_blocks(g.K) == 2 ? 256 : wide_rows(b.device_cus, g.rows, g.E, g.N);
  if (!grouped_wide_fits(g, bm) || (scale_blocks(g.K) == 2 && g.rows < 16 * (int64_t)g.E))
    return launch_narrow<false>(g, stream);
  return few_rows(b, g) ? launch_few(g, stream) : launch_grouped_wide(b, g, bm, stream);
}

}  // namespace ep
