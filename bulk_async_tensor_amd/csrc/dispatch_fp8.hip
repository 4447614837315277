// ep_dispatch_fp8: recv_q[dest_row[t, j], :] = e4m3(x[t, :] * (448 / amax)), one
// amax (and scale amax / 448) for each 128 values.
//
// A unit is (token, slab): a wave reads VPL 16-byte vectors per lane of a row,
// all in flight together, rounds them once and stores the slab k times.  A
// lane's vector holds 8 values, so a block is 16 lanes and its maximum four
// exchanges inside them.  The slab's scales are gathered through LDS into
// neighbouring lanes, so that a copy's scales are one store.
//
// The kernel is bound by the bytes it moves, three quarters of them writes at
// k = 6: T = 16384, H = 7168 188 us, 5.1 TB/s (a 4 GiB copy reaches 4.8).  128
// such rows at k = 8 take 6.0 us, 5.0 of them in the kernel.
#include "expert_internal.hpp"
#include "fp8_device.hpp"

namespace ep {

namespace {

constexpr int kMaxVpl = 16;
constexpr int kWaves = 4;                // waves per workgroup
constexpr int64_t kMaxGrid = 1 << 22;  // workgroups of one launch

template <int VPL, bool NT>
__global__ __launch_bounds__(kWaves * kWave) void dispatch_fp8_kernel(const u32x4* __restrict__ x,
                                                                      u32x2* __restrict__ q,
                                                                      float* __restrict__ scale,
                                                                      const int32_t* __restrict__ dest_row,
                                                                      int64_t recv_rows, int row_vec, int blocks,
                                                                      int k, int nslab, int units) {
  __shared__ float s_scale[kWaves][4 * VPL];
  const int lane = lane_id();
  const int wave = wave_in_group();
  const int stride = gridDim.x * kWaves;
  for (int64_t u = (int64_t)blockIdx.x * kWaves + wave; u < units; u += stride) {
    const int t = (int)u / nslab;
    const int c0 = ((int)u - t * nslab) * (VPL * kWave);
    const u32x4* src = x + (int64_t)t * row_vec;
    u32x4 v[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int c = c0 + i * kWave + lane;
      v[i] = ld16<NT>(src + (c < row_vec ? c : row_vec - 1));
    }
    u32x2 o[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const bool in = c0 + i * kWave + lane < row_vec;
      float f[8], m = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[2 * e] = bf16_lo(v[i][e]);
        f[2 * e + 1] = bf16_hi(v[i][e]);
        m = fmaxf(m, fmaxf(fabsf(f[2 * e]), fabsf(f[2 * e + 1])));
      }
      m = in ? fmaxf(m, kAmaxFloor) : kAmaxFloor;  // lanes past the row's end hold its last values again
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, kWave));
      const float inv = block_inverse(m);
      o[i] = u32x2{pack_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                   pack_e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv)};
      if ((lane & 15) == 0) s_scale[wave][4 * i + (lane >> 4)] = block_scale(m);
    }
    // (the wave's own LDS accesses keep their order; this keeps the compiler's)
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int b0 = c0 / 16;
    const bool holds = lane < 4 * VPL && b0 + lane < blocks;
    const float s = lane < 4 * VPL ? s_scale[wave][lane] : 0.0f;
    const int32_t* dr = dest_row + (int64_t)t * k;
    for (int j = 0; j < k; ++j) {
      const int64_t d = dr[j];
      if ((uint64_t)d >= (uint64_t)recv_rows) continue;
      u32x2* out = q + d * row_vec;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int c = c0 + i * kWave + lane;
        if (c < row_vec) __builtin_nontemporal_store(o[i], out + c);
      }
      if (holds) scale[d * blocks + b0 + lane] = s;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

using Fn = void (*)(const u32x4*, u32x2*, float*, const int32_t*, int64_t, int, int, int, int, int);

template <bool NT>
Fn pick(int vpl) {
  switch (vpl) {
    case 1: return dispatch_fp8_kernel<1, NT>;
    case 2: return dispatch_fp8_kernel<2, NT>;
    case 3: return dispatch_fp8_kernel<3, NT>;
    case 4: return dispatch_fp8_kernel<4, NT>;
    case 5: return dispatch_fp8_kernel<5, NT>;
    case 6: return dispatch_fp8_kernel<6, NT>;
    case 7: return dispatch_fp8_kernel<7, NT>;
    case 8: return dispatch_fp8_kernel<8, NT>;
    case 9: return dispatch_fp8_kernel<9, NT>;
    case 10: return dispatch_fp8_kernel<10, NT>;
    case 11: return dispatch_fp8_kernel<11, NT>;
    case 12: return dispatch_fp8_kernel<12, NT>;
    case 13: return dispatch_fp8_kernel<13, NT>;
    case 14: return dispatch_fp8_kernel<14, NT>;
    case 15: return dispatch_fp8_kernel<15, NT>;
    default: return dispatch_fp8_kernel<16, NT>;
  }
}

}  // namespace

hipError_t launch_dispatch_fp8(const Budget& b, const void* x, int T, int H, const int32_t* dest_row, int k,
                               void* recv_q, float* recv_scale, int64_t recv_rows, hipStream_t stream) {
  const int row_vec = H / 8, nv = (row_vec + kWave - 1) / kWave;
  const bool budget = b.num_cus > 0;
  const int cus = budget && b.num_cus < b.device_cus ? b.num_cus : b.device_cus;
  // Whole rows up to 16 KiB; a small batch takes shorter slabs, down to 1 KiB,
  // until every CU has 8 waves of them.
  int64_t want = (int64_t)T * nv / (8 * cus);
  if (want < 1) want = 1;
  int nslab = (nv + kMaxVpl - 1) / kMaxVpl;
  if (want < (nv + nslab - 1) / nslab) nslab = (nv + (int)want - 1) / (int)want;
  const int vpl = (nv + nslab - 1) / nslab;
  nslab = (nv + vpl - 1) / vpl;
  const int units = T * nslab;  // at most EP_MAX_ENTRIES (checked by the ABI)
  Fn fn = stream_rows((int64_t)T * H * 2) ? pick<true>(vpl) : pick<false>(vpl);
  int64_t grid = ((int64_t)units + kWaves - 1) / kWaves;
  size_t lds = 0;
  if (budget) {
    grid = cus;
    lds = kExclusiveLds;
    hipError_t e = allow_dynamic_lds((const void*)fn, lds);
    if (e != hipSuccess) return e;
  } else if (grid > kMaxGrid) {
    grid = kMaxGrid;
  }
  hipLaunchKernelGGL(fn, dim3((unsigned)grid), dim3(kWaves * kWave), lds, stream, static_cast<const u32x4*>(x),
                     static_cast<u32x2*>(recv_q), recv_scale, dest_row, recv_rows, row_vec, scale_blocks(H), k, nslab,
                     units);
  return hipGetLastError();
}

}  // namespace ep
