// Host-side interfaces between the expert side's C ABI (expert_api.hip) and
// its kernel files.
#pragma once

#include "ep_internal.hpp"

namespace ep {

constexpr int kScaleBlock = 128;  // values that share a scale (the ABI's EP_FP8_BLOCK)
inline __host__ __device__ int scale_blocks(int n) { return (n + kScaleBlock - 1) / kScaleBlock; }

// Whether the row movers stream their source rows (non-temporal loads) or load
// them through the caches: the step before has just written them, so a source
// that the 256 MB Infinity Cache holds is mostly still there.  Streamed
// against cached, us: 8-bit dispatch of 59 MB (T = 4096, H = 7168, k = 8) 59 /
// 52, of 235 MB 187 / 192; combine_backward with 34 MB of y 16 / 13, 67 MB 28
// / 26, 470 MB 187 / 199; dispatch_backward of 67 MB 17 / 16, 470 MB 89 / 99.
inline bool stream_rows(int64_t bytes) { return bytes > (int64_t)128 << 20; }

// ---- dispatch_fp8.hip
hipError_t launch_dispatch_fp8(const Budget& b, const void* x, int T, int H, const int32_t* dest_row, int k,
                               void* recv_q, float* recv_scale, int64_t recv_rows, hipStream_t stream);

// ---- grouped_fp8.hip: swiglu = false: N weight rows, y is bf16 [rows, N];
// swiglu = true: N = 2 I weight rows, y is e4m3 [rows, I] and y_scale its scales.
struct GroupedArgs {
  const void* a;
  const float* a_scale;
  int64_t rows;
  int K;
  const int32_t* offsets;
  int E;
  const void* b;
  const float* b_scale;
  int N;
  void* y;
  float* y_scale;
};
hipError_t launch_grouped_fp8(const Budget& b, const GroupedArgs& g, bool swiglu, hipStream_t stream);

// ---- grouped_wide.hip: the plain product, bm = 128 or 256 token rows at a time
bool grouped_wide_fits(const GroupedArgs& g, int bm);  // whether it takes this K
hipError_t launch_grouped_wide(const Budget& b, const GroupedArgs& g, int bm, hipStream_t stream);

// ---- grouped_swiglu.hip
bool grouped_swiglu_fits(const GroupedArgs& g);  // whether it takes this K
hipError_t launch_grouped_swiglu(const Budget& b, const GroupedArgs& g, hipStream_t stream);

// ---- backward.hip
hipError_t launch_combine_backward(const Budget& b, const void* dout, const void* y, int64_t recv_rows, int H,
                                   const int32_t* dest_row, const float* w, int T, int k, void* dy, float* dw,
                                   hipStream_t stream);
hipError_t launch_dispatch_backward(const Budget& b, const void* drecv, int64_t recv_rows, int H,
                                    const int32_t* dest_row, int T, int k, void* dx, hipStream_t stream);

}  // namespace ep
