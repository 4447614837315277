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
// neighbours, and comes from HBM once.  dispatch_backward: a wave takes a
// segment of a token's row, gathers it from the k rows step by step and holds
// the finished vectors; the waves of a workgroup meet between their loads and
// their stores, so that a CU's loads do not queue behind its own stores.
// T = 4096, H = 7168, k = 8: combine_backward 183 us, 5.4 TB/s;
// dispatch_backward 86.4 us, 6.1 TB/s (a 4 GiB copy reaches 4.8).
#include "ep_device.hpp"
#include "expert_internal.hpp"
#include "expert_shapes.hpp"
#include "row_io.hpp"

namespace ep {

namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = kWave / 2; d > 0; d >>= 1) v += __shfl_xor(v, d, kWave);
  return v;
}

constexpr int kMaxVpl = 16;

// VPL vectors per lane of both rows in flight together; rows of more than 16
// KiB in nslab slabs.
template <int VPL, bool NT, bool DY, bool DW>
__global__ __launch_bounds__(512) void combine_backward_kernel(const u32x4* __restrict__ dout,
                                                               const u32x4* __restrict__ y, u32x4* __restrict__ dy,
                                                               float* __restrict__ dw,
                                                               const int32_t* __restrict__ dest_row,
                                                               const float* __restrict__ w, int64_t recv_rows,
                                                               int row_vec, int k, int nslab, int64_t entries) {
  const int lane = lane_id();
  const int wpg = blockDim.x >> 6;
  const int64_t stride = (int64_t)gridDim.x * wpg;
  for (int64_t e = (int64_t)blockIdx.x * wpg + wave_in_group(); e < entries; e += stride) {
    const int64_t d = dest_row[e];
    const bool ok = (uint64_t)d < (uint64_t)recv_rows;
    const u32x4* g = dout + (e / k) * row_vec;
    // an entry without a row reads its token's row instead and stores nothing
    const u32x4* yr = DW && ok ? y + d * row_vec : g;
    const float wt = DY ? w[e] : 0.0f;
    float acc = 0.0f;
    for (int s = 0; s < nslab; ++s) {
      const int c0 = s * VPL * kWave + lane;
      u32x4 gv[VPL], yv[VPL];
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int c = c0 + i * kWave;
        gv[i] = ld16<false>(g + (c < row_vec ? c : row_vec - 1));
      }
      if (DW) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const int c = c0 + i * kWave;
          yv[i] = ld16<NT>(yr + (c < row_vec ? c : row_vec - 1));
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const bool in = c0 + i * kWave < row_vec;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float a0 = fmaf(bf16_lo(gv[i][q]), bf16_lo(yv[i][q]), acc);
            const float a1 = fmaf(bf16_hi(gv[i][q]), bf16_hi(yv[i][q]), a0);
            acc = in ? a1 : acc;
          }
        }
      }
      if (DY) {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) gv[i][q] = pack_bf16x2(wt * bf16_lo(gv[i][q]), wt * bf16_hi(gv[i][q]));
        if (ok) {
#pragma unroll
          for (int i = 0; i < VPL; ++i) {
            const int c = c0 + i * kWave;
            if (c < row_vec) st16<true>(dy + d * row_vec + c, gv[i]);
          }
        }
      }
    }
    if (DW) {
      acc = wave_sum(acc);
      if (lane == 0) dw[e] = ok ? acc : 0.0f;
    }
  }
}

// A unit is one of nseg segments of STEPS * VS vectors per lane of a token's
// row.  A step gathers VS vectors from KS rows at a time (8 loads in flight,
// and the next step's where registers allow); ONE: k is at most KS.
template <int KS, int VS, int STEPS, bool ONE, bool NT>
__global__ __launch_bounds__(256) void dispatch_backward_kernel(const u32x4* __restrict__ drecv,
                                                                u32x4* __restrict__ dx,
                                                                const int32_t* __restrict__ dest_row,
                                                                int64_t recv_rows, int row_vec, int nseg, int k,
                                                                int units, int trips) {
  const int lane = lane_id();
  const int wpg = blockDim.x >> 6;
  const int stride = gridDim.x * wpg;
  for (int trip = 0; trip < trips; ++trip) {
    const int u_raw = blockIdx.x * wpg + wave_in_group() + trip * stride;
    const bool live = u_raw < units;
    const int u = live ? u_raw : 0;
    const int t = u / nseg;
    const int c0 = (u - t * nseg) * (STEPS * VS * kWave) + lane;
    const int32_t* dr = dest_row + (int64_t)t * k;
    u32x4 held[STEPS * VS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      float acc[VS][8] = {};
      for (int j0 = 0; j0 < (ONE ? 1 : k); j0 += KS) {
        u32x4 v[KS][VS];
        uint32_t keep[KS];
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          const int64_t d = j0 + j < k ? dr[j0 + j] : -1;
          const bool ok = (uint64_t)d < (uint64_t)recv_rows;
          keep[j] = ok ? ~0u : 0u;
          // (a slot without a row reads row 0, and adds +0: that leaves every sum that starts from +0 as it is)
          const u32x4* src = drecv + (ok ? d : 0) * row_vec;
#pragma unroll
          for (int i = 0; i < VS; ++i) {
            const int c = c0 + (s * VS + i) * kWave;
            v[j][i] = ld16<NT>(src + (c < row_vec ? c : row_vec - 1));
          }
        }
#pragma unroll
        for (int j = 0; j < KS; ++j)
#pragma unroll
          for (int i = 0; i < VS; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              acc[i][2 * e] += bf16_lo(v[j][i][e] & keep[j]);
              acc[i][2 * e + 1] += bf16_hi(v[j][i][e] & keep[j]);
            }
      }
#pragma unroll
      for (int i = 0; i < VS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) held[s * VS + i][e] = pack_bf16x2(acc[i][2 * e], acc[i][2 * e + 1]);
    }
#pragma unroll
    for (int i = 0; i < STEPS * VS; ++i) asm volatile("" : "+v"(held[i]));
    wait_vmcnt<0>();
    __builtin_amdgcn_s_barrier();
    if (live) {
#pragma unroll
      for (int i = 0; i < STEPS * VS; ++i) {
        const int c = c0 + i * kWave;
        if (c < row_vec) st16<true>(dx + (int64_t)t * row_vec + c, held[i]);
      }
    }
  }
}

// Grid and LDS of a launch of `units` waves' work: a workgroup for all of it
// (a grid of 8 workgroups per CU that loops lost 3% at T = 16384, H = 7168, k
// = 6), or the budget's persistent grid of one workgroup per CU.
hipError_t place(const Budget& b, const void* kernel, int64_t units, int wpg, int* grid, size_t* lds) {
  *lds = 0;
  if (b.num_cus > 0) {
    *grid = b.num_cus < b.device_cus ? b.num_cus : b.device_cus;
    *lds = kExclusiveLds;
    return allow_dynamic_lds(kernel, *lds);
  }
  const int64_t want = (units + wpg - 1) / wpg, most = 1 << 22;
  *grid = (int)(want < most ? want : most);
  return hipSuccess;
}

using CombineFn = void (*)(const u32x4*, const u32x4*, u32x4*, float*, const int32_t*, const float*, int64_t, int, int,
                           int, int64_t);

template <int VPL>
CombineFn pick_outputs(bool nt, bool dy, bool dw) {
  if (!dw) return combine_backward_kernel<VPL, false, true, false>;  // reads no y
  if (!dy) return nt ? combine_backward_kernel<VPL, true, false, true> : combine_backward_kernel<VPL, false, false, true>;
  return nt ? combine_backward_kernel<VPL, true, true, true> : combine_backward_kernel<VPL, false, true, true>;
}

CombineFn pick_combine(int vpl, bool nt, bool dy, bool dw) {
  switch (vpl) {
    case 1: return pick_outputs<1>(nt, dy, dw);
    case 2: return pick_outputs<2>(nt, dy, dw);
    case 3: return pick_outputs<3>(nt, dy, dw);
    case 4: return pick_outputs<4>(nt, dy, dw);
    case 5: return pick_outputs<5>(nt, dy, dw);
    case 6: return pick_outputs<6>(nt, dy, dw);
    case 7: return pick_outputs<7>(nt, dy, dw);
    case 8: return pick_outputs<8>(nt, dy, dw);
    case 9:
    case 10: return pick_outputs<10>(nt, dy, dw);
    case 11:
    case 12: return pick_outputs<12>(nt, dy, dw);
    case 13:
    case 14: return pick_outputs<14>(nt, dy, dw);
    default: return pick_outputs<16>(nt, dy, dw);
  }
}

using DispatchFn = void (*)(const u32x4*, u32x4*, const int32_t*, int64_t, int, int, int, int, int);

// The kernel of 1 .. MOST steps (a last step may be partly past the row's end).
template <int KS, int VS, int MOST, bool ONE, bool NT>
DispatchFn pick_steps(int steps) {
  if (steps == MOST) return dispatch_backward_kernel<KS, VS, MOST, ONE, NT>;
  if constexpr (MOST > 1) return pick_steps<KS, VS, MOST - 1, ONE, NT>(steps);
  return nullptr;
}

// The shapes that dispatch_backward_shape gives: 4 vectors a segment for k <= 4, 8 above.
template <bool NT>
DispatchFn pick_dispatch(int k, const GatherShape& s) {
  return k == 1   ? (s.vs == 4 ? pick_steps<1, 4, 1, true, NT>(s.steps) : pick_steps<1, 2, 1, true, NT>(s.steps))
         : k == 2 ? (s.vs == 4 ? pick_steps<2, 4, 1, true, NT>(s.steps) : pick_steps<2, 2, 1, true, NT>(s.steps))
         : k <= 4 ? pick_steps<4, 2, 2, true, NT>(s.steps)
         : k <= 8 ? pick_steps<8, 1, 8, true, NT>(s.steps)
                  : pick_steps<8, 1, 8, false, NT>(s.steps);
}

}  // namespace

hipError_t launch_combine_backward(const Budget& b, const void* dout, const void* y, int64_t recv_rows, int H,
                                   const int32_t* dest_row, const float* w, int T, int k, void* dy, float* dw,
                                   hipStream_t stream) {
  const int row_vec = H / 8, nv = (row_vec + kWave - 1) / kWave;
  const int nslab = (nv + kMaxVpl - 1) / kMaxVpl;
  const int vpl = nslab == 1 ? nv : kMaxVpl;
  const CombineFn fn = pick_combine(vpl, stream_rows((int64_t)T * k * H * 2), dy != nullptr, dw != nullptr);
  const int64_t entries = (int64_t)T * k;
  // a workgroup is one token, so that its row comes from HBM once (two at k = 2 and 3, four at 1)
  const int wpg = k <= 2 ? 4 : k == 3 ? 6 : k > 8 ? 8 : k;
  int grid;
  size_t lds;
  hipError_t e = place(b, (const void*)fn, entries, wpg, &grid, &lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(fn, dim3(grid), dim3(wpg * kWave), lds, stream, static_cast<const u32x4*>(dout),
                     static_cast<const u32x4*>(y), static_cast<u32x4*>(dy), dw, dest_row, w, recv_rows, row_vec, k,
                     nslab, entries);
  return hipGetLastError();
}

hipError_t launch_dispatch_backward(const Budget& b, const void* drecv, int64_t recv_rows, int H,
                                    const int32_t* dest_row, int T, int k, void* dx, hipStream_t stream) {
  const int row_vec = H / 8, nv = (row_vec + kWave - 1) / kWave;
  // an empty buffer: every slot is out of range, and dx stands in for the row that such slots read
  if (recv_rows == 0) drecv = dx;
  const int cus = b.num_cus > 0 && b.num_cus < b.device_cus ? b.num_cus : b.device_cus;
  const GatherShape shape = dispatch_backward_shape(T, nv, k, cus);
  const int nseg = shape.nseg;
  const DispatchFn fn = stream_rows((int64_t)T * k * H * 2) ? pick_dispatch<true>(k, shape) : pick_dispatch<false>(k, shape);
  if (!fn) return hipErrorInvalidValue;
  const int units = T * nseg;  // at most EP_MAX_ENTRIES (checked by the ABI)
  constexpr int kWaves = 4;
  int grid;
  size_t lds;
  hipError_t e = place(b, (const void*)fn, units, kWaves, &grid, &lds);
  if (e != hipSuccess) return e;
  const int64_t per_trip = (int64_t)grid * kWaves;
  hipLaunchKernelGGL(fn, dim3(grid), dim3(kWaves * kWave), lds, stream, static_cast<const u32x4*>(drecv),
                     static_cast<u32x4*>(dx), dest_row, recv_rows, row_vec, nseg, k, units,
                     (int)((units + per_trip - 1) / per_trip));
  return hipGetLastError();
}

}  // namespace ep
