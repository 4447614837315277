// ep_dispatch_fp8: recv_q[dest_row[t, j], :] = e4m3(x[t, :] * (448 / amax)), one
// amax (and scale amax / 448) for each 128 values.
//
// A wave takes a token: a lane's 16-byte load holds 8 values, so a block is 16
// lanes, its maximum four exchanges inside them.  The row is read and rounded
// once and stored k times.
#include "expert_internal.hpp"
#include "fp8_device.hpp"

namespace ep {

namespace {

__global__ __launch_bounds__(256) void dispatch_fp8_kernel(const u32x4* __restrict__ x, u32x2* __restrict__ q,
                                                           float* __restrict__ scale,
                                                           const int32_t* __restrict__ dest_row, int64_t recv_rows,
                                                           int row_vec, int blocks, int k, int T) {
  const int lane = lane_id();
  const int wpg = blockDim.x >> 6;
  const int64_t stride = (int64_t)gridDim.x * wpg;
  for (int64_t t = (int64_t)blockIdx.x * wpg + wave_in_group(); t < T; t += stride) {
    const int32_t* dr = dest_row + t * k;
    for (int c0 = 0; c0 < row_vec; c0 += kWave) {
      const int c = c0 + lane;
      const bool in = c < row_vec;
      u32x4 v = {0u, 0u, 0u, 0u};
      if (in) v = ld16<true>(x + t * row_vec + c);
      float f[8], m = kAmaxFloor;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[2 * e] = bf16_lo(v[e]);
        f[2 * e + 1] = bf16_hi(v[e]);
        m = fmaxf(m, fmaxf(fabsf(f[2 * e]), fabsf(f[2 * e + 1])));
      }
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, kWave));
      const float inv = block_inverse(m);
      const u32x2 o = {pack_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                       pack_e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv)};
      const float s = block_scale(m);
      for (int j = 0; j < k; ++j) {
        const int64_t d = dr[j];
        if ((uint64_t)d >= (uint64_t)recv_rows) continue;
        if (in) {
          q[d * row_vec + c] = o;
          if ((lane & 15) == 0) scale[d * blocks + c / 16] = s;
        }
      }
    }
  }
}

}  // namespace

hipError_t launch_dispatch_fp8(const Budget& b, const void* x, int T, int H, const int32_t* dest_row, int k,
                               void* recv_q, float* recv_scale, int64_t recv_rows, hipStream_t stream) {
  int grid = (T + 3) / 4;
  size_t lds = 0;
  if (b.num_cus > 0) {
    grid = b.num_cus < b.device_cus ? b.num_cus : b.device_cus;
    lds = kExclusiveLds;
    hipError_t e = allow_dynamic_lds((const void*)dispatch_fp8_kernel, lds);
    if (e != hipSuccess) return e;
  } else if (grid > 8 * b.device_cus) {
    grid = 8 * b.device_cus;
  }
  hipLaunchKernelGGL(dispatch_fp8_kernel, dim3(grid), dim3(256), lds, stream, static_cast<const u32x4*>(x),
                     static_cast<u32x2*>(recv_q), recv_scale, dest_row, recv_rows, H / 8, scale_blocks(H), k, T);
  return hipGetLastError();
}

}  // namespace ep
