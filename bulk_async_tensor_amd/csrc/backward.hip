// The gradients of combine and dispatch.
//
//   ep_combine_backward   dy[dest_row[t, j], :] = bf16(w[t, j] * dout[t, :])
//                         dw[t, j] = <dout[t, :], y[dest_row[t, j], :]>
//   ep_dispatch_backward  dx[t, :] = bf16(sum_j drecv[dest_row[t, j], :])
//
// Both are bound by the rows they move.  combine_backward: a wave takes one
// entry (t, j), reads both rows once, keeps the dot product in registers and
// joins its 64 parts by exchanges, so nothing is added in memory and the order
// of the sum is fixed.  dout[t] is read by the k waves of its token, which are
// neighbours, and comes from HBM once.  dispatch_backward: a wave takes a slab
// of a token and gathers its k rows.
#include "ep_device.hpp"
#include "expert_internal.hpp"
#include "row_io.hpp"

namespace ep {

namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = kWave / 2; d > 0; d >>= 1) v += __shfl_xor(v, d, kWave);
  return v;
}

template <bool DY, bool DW>
__global__ __launch_bounds__(256) void combine_backward_kernel(const u32x4* __restrict__ dout,
                                                               const u32x4* __restrict__ y, u32x4* __restrict__ dy,
                                                               float* __restrict__ dw,
                                                               const int32_t* __restrict__ dest_row,
                                                               const float* __restrict__ w, int64_t recv_rows,
                                                               int row_vec, int k, int64_t entries) {
  const int lane = lane_id();
  const int wpg = blockDim.x >> 6;
  const int64_t stride = (int64_t)gridDim.x * wpg;
  for (int64_t u = (int64_t)blockIdx.x * wpg + wave_in_group(); u < entries; u += stride) {
    const int64_t d = dest_row[u];
    if ((uint64_t)d >= (uint64_t)recv_rows) {
      if (DW && lane == 0) dw[u] = 0.0f;
      continue;
    }
    const u32x4* g = dout + (u / k) * row_vec;
    const float wt = DY ? w[u] : 0.0f;
    float acc = 0.0f;
    for (int c = lane; c < row_vec; c += kWave) {
      const u32x4 gv = ld16<false>(g + c);
      if (DW) {
        const u32x4 yv = ld16<true>(y + d * row_vec + c);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc = fmaf(bf16_lo(gv[e]), bf16_lo(yv[e]), acc);
          acc = fmaf(bf16_hi(gv[e]), bf16_hi(yv[e]), acc);
        }
      }
      if (DY) {
        u32x4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = pack_bf16x2(wt * bf16_lo(gv[e]), wt * bf16_hi(gv[e]));
        st16<true>(dy + d * row_vec + c, o);
      }
    }
    if (DW) {
      acc = wave_sum(acc);
      if (lane == 0) dw[u] = acc;
    }
  }
}

__global__ __launch_bounds__(256) void dispatch_backward_kernel(const u32x4* __restrict__ drecv,
                                                                u32x4* __restrict__ dx,
                                                                const int32_t* __restrict__ dest_row,
                                                                int64_t recv_rows, int row_vec, int nslab, int k,
                                                                int units) {
  constexpr int KB = 8;  // rows whose loads are in flight together
  const int lane = lane_id();
  const int wpg = blockDim.x >> 6;
  const int stride = gridDim.x * wpg;
  for (int u = blockIdx.x * wpg + wave_in_group(); u < units; u += stride) {
    const int t = u / nslab;
    const int c = (u - t * nslab) * kWave + lane;
    const int32_t* dr = dest_row + (int64_t)t * k;
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += KB) {
      u32x4 v[KB];
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        const int64_t d = j0 + j < k ? dr[j0 + j] : -1;
        v[j] = u32x4{0u, 0u, 0u, 0u};
        if ((uint64_t)d < (uint64_t)recv_rows && c < row_vec) v[j] = ld16<true>(drecv + d * row_vec + c);
      }
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        // (a slot that is out of range adds +0, which leaves every sum that
        // starts from +0 as it is)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[2 * e] += bf16_lo(v[j][e]);
          acc[2 * e + 1] += bf16_hi(v[j][e]);
        }
      }
    }
    if (c < row_vec) {
      u32x4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = pack_bf16x2(acc[2 * e], acc[2 * e + 1]);
      st16<true>(dx + (int64_t)t * row_vec + c, o);
    }
  }
}

// Grid and LDS of a launch of `units` waves' work: the whole device, or the
// budget's persistent grid of one workgroup per CU.
hipError_t place(const Budget& b, const void* kernel, int64_t units, int wpg, int* grid, size_t* lds) {
  *lds = 0;
  if (b.num_cus > 0) {
    *grid = b.num_cus < b.device_cus ? b.num_cus : b.device_cus;
    *lds = kExclusiveLds;
    return allow_dynamic_lds(kernel, *lds);
  }
  const int64_t want = (units + wpg - 1) / wpg, most = (int64_t)b.device_cus * 8;
  *grid = (int)(want < most ? want : most);
  return hipSuccess;
}

}  // namespace

hipError_t launch_combine_backward(const Budget& b, const void* dout, const void* y, int64_t recv_rows, int H,
                                   const int32_t* dest_row, const float* w, int T, int k, void* dy, float* dw,
                                   hipStream_t stream) {
  const auto fn = !dw ? combine_backward_kernel<true, false>
                  : !dy ? combine_backward_kernel<false, true> : combine_backward_kernel<true, true>;
  const int64_t entries = (int64_t)T * k;
  int grid;
  size_t lds;
  hipError_t e = place(b, (const void*)fn, entries, 4, &grid, &lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(fn, dim3(grid), dim3(256), lds, stream, static_cast<const u32x4*>(dout),
                     static_cast<const u32x4*>(y), static_cast<u32x4*>(dy), dw, dest_row, w, recv_rows, H / 8, k,
                     entries);
  return hipGetLastError();
}

hipError_t launch_dispatch_backward(const Budget& b, const void* drecv, int64_t recv_rows, int H,
                                    const int32_t* dest_row, int T, int k, void* dx, hipStream_t stream) {
  const int row_vec = H / 8, nslab = (row_vec + kWave - 1) / kWave;
  const int units = T * nslab;  // at most EP_MAX_ENTRIES (checked by the ABI)
  int grid;
  size_t lds;
  hipError_t e = place(b, (const void*)dispatch_backward_kernel, units, 4, &grid, &lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(dispatch_backward_kernel, dim3(grid), dim3(256), lds, stream, static_cast<const u32x4*>(drecv),
                     static_cast<u32x4*>(dx), dest_row, recv_rows, row_vec, nslab, k, units);
  return hipGetLastError();
}

}  // namespace ep
