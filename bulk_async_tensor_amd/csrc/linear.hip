// ep_grouped_linear and its gradients: bf16 products of each expert's rows.
//
// One workgroup of 4 waves computes 64 x 64 results in steps of 32 along the
// sum, both sides' tiles staged through registers into LDS rows of 32 values
// that lie along the sum; a side that lies across it is turned on the way.
#include "ep.h"
#include "ep_device.hpp"
#include "grouped_tiles.hpp"
#include "linear_epilogue.hpp"

namespace ep {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));

enum Product { kForward, kDgrad, kWgrad };

constexpr int kSide = 64, kDeep = 32, kPitch = kDeep + 8;

// 8 values of a side's tile: its row `row` at places at .. at + 7 along the
// sum (Along), or its 8 rows from `row` at one place (turned).
template <bool ALONG>
__device__ __forceinline__ u32x4 fetch(const uint16_t* base, int64_t ld, int row, int rows_end, int64_t at,
                                       int64_t at_end) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (row < rows_end && at < at_end)
    v = *reinterpret_cast<const u32x4*>(ALONG ? base + row * ld + at : base + at * ld + row);
  return v;
}
template <bool ALONG>
__device__ __forceinline__ void put(uint16_t* lds, int tid, u32x4 v) {
  const u16x8 h = __builtin_bit_cast(u16x8, v);
  if (ALONG) {
    *reinterpret_cast<u32x4*>(lds + (tid >> 2) * kPitch + (tid & 3) * 8) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) lds[((tid & 7) * 8 + i) * kPitch + (tid >> 3)] = h[i];
  }
}

template <Product P>
__global__ __launch_bounds__(256) void linear_kernel(LinearArgs g, int units_n) {
  __shared__ __attribute__((aligned(16))) uint16_t s_r[kSide * kPitch], s_c[kSide * kPitch];
  __shared__ int32_t s_first[kMaxExperts + 1];
  const int lane = lane_id(), wave = wave_in_group(), tid = threadIdx.x;
  const int col = lane & 15, quad = lane >> 4;
  int e, n0;
  int64_t r0, r1;
  int row_limit;  // rows of the row side
  int64_t deep;   // places along the sum
  const uint16_t *rp, *cp;
  int64_t rld, cld;
  if constexpr (P != kWgrad) {
    if (g.offsets) {
      if (wave == 0) first_tiles<kSide>(g.offsets, g.E, (int)g.rows, lane, s_first);
      __syncthreads();
      if ((int64_t)blockIdx.x >= (int64_t)s_first[g.E] * units_n) return;
      WideTile t;
      find_tile_of<kSide>(g.offsets, s_first, g.E, (int)g.rows, units_n, blockIdx.x, lane, &t);
      e = t.e, n0 = t.n, r0 = t.r0, r1 = t.r1;
    } else {
      const int64_t m = (g.rows + kSide - 1) / kSide;
      e = 0, n0 = (int)(blockIdx.x / m), r0 = (int64_t)(blockIdx.x % m) * kSide;
      r1 = r0 + kSide < g.rows ? r0 + kSide : g.rows;
    }
    row_limit = (int)(r1 - r0);
    deep = P == kForward ? g.K : g.N;
    rld = deep, cld = g.K;
    rp = static_cast<const uint16_t*>(g.rows_in) + r0 * rld;
    cp = static_cast<const uint16_t*>(g.cols_in) + (int64_t)e * g.N * g.K;
  } else {
    const int un = (g.N + kSide - 1) / kSide;
    e = blockIdx.x / (un * units_n);
    const int left = blockIdx.x % (un * units_n);
    n0 = left / un;
    const int m0 = left % un * kSide;
    int64_t lo = 0, hi = g.rows;
    if (g.offsets) {
      const Segment s = segment_of(g.offsets, (int)g.rows, e);
      lo = s.lo, hi = s.hi;
    }
    r0 = m0, r1 = hi;
    row_limit = g.N - m0;
    deep = hi - lo;
    rld = g.N, cld = g.K;
    rp = static_cast<const uint16_t*>(g.rows_in) + lo * rld + m0;
    cp = static_cast<const uint16_t*>(g.cols_in) + lo * cld;
  }
  // the tile's columns: two halves of 32, with swiglu gate and up rows
  const bool pair = P == kForward && g.act == EP_ACT_SWIGLU;
  const int outs = P == kForward ? (pair ? g.N / 2 : g.N) : g.K;
  const int c0 = n0 * (pair ? kSide / 2 : kSide);
  const int half1 = pair ? g.N / 2 + c0 : c0 + kSide / 2;  // first weight row of the second half
  f32x4 acc[2][2] = {};
  float sum_dy = 0.0f;
  const int wr = wave >> 1, wc = wave & 1;
  constexpr bool kRowsAlong = P != kWgrad, kColsAlong = P == kForward;
  for (int64_t at = 0; at < deep; at += kDeep) {
    u32x4 vr, vc;
    if (kRowsAlong) vr = fetch<true>(rp, rld, tid >> 2, row_limit, at + (tid & 3) * 8, deep);
    else vr = fetch<false>(rp, rld, (tid & 7) * 8, row_limit, at + (tid >> 3), deep);
    if (kColsAlong) {
      const int c = tid >> 2;
      const int row = c < kSide / 2 ? c0 + c : half1 + c - kSide / 2;
      const int end = pair && c < kSide / 2 ? outs : g.N;
      vc = fetch<true>(cp, cld, row, end, at + (tid & 3) * 8, deep);
    } else {
      vc = fetch<false>(cp, cld, c0 + (tid & 7) * 8, outs, at + (tid >> 3), deep);
    }
    __syncthreads();
    put<kRowsAlong>(s_r, tid, vr);
    put<kColsAlong>(s_c, tid, vc);
    __syncthreads();
    bf16x8 fr[2], fc[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      fr[i] = *reinterpret_cast<const bf16x8*>(s_r + (wr * 32 + i * 16 + col) * kPitch + quad * 8);
      fc[i] = *reinterpret_cast<const bf16x8*>(s_c + (i * 32 + wc * 16 + col) * kPitch + quad * 8);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i) acc[h][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fc[h], fr[i], acc[h][i], 0, 0, 0);
    if (P == kWgrad && g.dbias && n0 == 0 && tid < kSide)
      for (int i = 0; i < kDeep; ++i) sum_dy += __uint_as_float((uint32_t)s_r[tid * kPitch + i] << 16);
  }
  // lane (col, quad): row col of each row tile, columns 4 quad .. + 3 of each column tile
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int lr = wr * 32 + i * 16 + col;
    if (lr >= row_limit) continue;
    if (pair) {
      const int n = c0 + wc * 16 + quad * 4;
      if (n < outs) finish_swiglu(g, e, r0 + lr, n, acc[0][i], acc[1][i]);
      continue;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int n = c0 + h * 32 + wc * 16 + quad * 4;
      if (n >= outs) continue;
      if constexpr (P == kForward) finish_linear(g, g.act, e, r0 + lr, n, acc[h][i]);
      if constexpr (P == kDgrad) finish_dgrad(g, g.act, r0 + lr, n, acc[h][i]);
      if constexpr (P == kWgrad) {
        const int64_t o = ((int64_t)e * g.N + r0 + lr) * g.K + n;
        if (g.out_f32) *reinterpret_cast<f32x4*>(static_cast<float*>(g.out) + o) = acc[h][i];
        else store4_bf16(g.out, o, acc[h][i]);
      }
    }
  }
  if (P == kWgrad && g.dbias && n0 == 0 && tid < kSide && tid < row_limit) g.dbias[(int64_t)e * g.N + r0 + tid] = sum_dy;
}

}  // namespace

size_t linear_workspace(int64_t, int, int, int, int) { return 0; }
size_t dgrad_workspace(int64_t, int, int, int) { return 0; }
size_t wgrad_workspace(int64_t, int, int, int) { return 0; }

hipError_t launch_linear(const Budget&, const LinearArgs& g, hipStream_t stream) {
  const int outs = g.act == EP_ACT_SWIGLU ? g.N / 2 : g.N, wide = g.act == EP_ACT_SWIGLU ? kSide / 2 : kSide;
  const int units = (outs + wide - 1) / wide;
  const int64_t grid = g.offsets ? wide_tiles_most(g.rows, g.E, kSide) * units : (g.rows + kSide - 1) / kSide * units;
  hipLaunchKernelGGL(linear_kernel<kForward>, dim3((uint32_t)grid), dim3(256), 0, stream, g, units);
  return hipGetLastError();
}
hipError_t launch_dgrad(const Budget&, const LinearArgs& g, hipStream_t stream) {
  const int units = (g.K + kSide - 1) / kSide;
  const int64_t grid = g.offsets ? wide_tiles_most(g.rows, g.E, kSide) * units : (g.rows + kSide - 1) / kSide * units;
  hipLaunchKernelGGL(linear_kernel<kDgrad>, dim3((uint32_t)grid), dim3(256), 0, stream, g, units);
  return hipGetLastError();
}
hipError_t launch_wgrad(const Budget&, const LinearArgs& g, hipStream_t stream) {
  const int units = (g.K + kSide - 1) / kSide;
  const int64_t grid = (int64_t)g.E * ((g.N + kSide - 1) / kSide) * units;
  hipLaunchKernelGGL(linear_kernel<kWgrad>, dim3((uint32_t)grid), dim3(256), 0, stream, g, units);
  return hipGetLastError();
}

}  // namespace ep
