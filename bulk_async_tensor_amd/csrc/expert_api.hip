// C ABI of the expert side (ep_expert.h): argument checks and launches on the
// caller's stream.  As in ep_api.hip, every host-detectable error is reported
// before any HIP call is made.
#include "ep_expert.h"
#include "ep_host.hpp"
#include "expert_internal.hpp"

using ep::aligned;
using ep::fail;

static_assert(EP_FP8_BLOCK == ep::kScaleBlock, "the kernels' scale block is the ABI's");

namespace {

int check_grouped(const ep::GroupedArgs& g, const char* what, const char* n_name, int n, int n_multiple) {
  if (g.rows < 0 || g.rows > EP_MAX_ENTRIES)
    return fail(EP_ERR_INVALID_ARG, "%s: rows = %lld outside [0, EP_MAX_ENTRIES]", what, (long long)g.rows);
  if (g.K <= 0 || g.K % 16 != 0)
    return fail(EP_ERR_INVALID_ARG, "%s: K = %d must be a positive multiple of 16", what, g.K);
  if (n <= 0 || n % n_multiple != 0)
    return fail(EP_ERR_INVALID_ARG, "%s: %s = %d must be a positive multiple of %d", what, n_name, n, n_multiple);
  if (g.E < 1 || g.E > EP_MAX_EXPERTS)
    return fail(EP_ERR_INVALID_ARG, "%s: E = %d outside [1, %d]", what, g.E, EP_MAX_EXPERTS);
  if ((int64_t)g.N * g.K > INT32_MAX)
    return fail(EP_ERR_INVALID_ARG, "%s: a weight of %lld values exceeds 2^31 - 1", what, (long long)g.N * g.K);
  if (!g.offsets || (g.rows > 0 && (!g.a || !g.a_scale || !g.b || !g.b_scale || !g.y)))
    return fail(EP_ERR_INVALID_ARG, "%s: null pointer", what);
  if (!aligned(g.a, 16) || !aligned(g.b, 16) || !aligned(g.y, 16))
    return fail(EP_ERR_ALIGNMENT, "%s: a row tensor not 16-byte aligned", what);
  if (!aligned(g.a_scale, 4) || !aligned(g.b_scale, 4) || !aligned(g.offsets, 4) || !aligned(g.y_scale, 4))
    return fail(EP_ERR_ALIGNMENT, "%s: a scale or offset tensor not 4-byte aligned", what);
  return EP_OK;
}

int run_grouped(const ep::GroupedArgs& g, bool swiglu, void* stream, const char* what) {
  if (g.rows == 0) return EP_OK;
  ep::Budget b;
  int rc = ep::current_device(&b, stream);
  if (rc) return rc;
  hipError_t e = ep::launch_grouped_fp8(b, g, swiglu, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return ep::hip_fail(e, what);
  return EP_OK;
}

}  // namespace

extern "C" {

int ep_dispatch_fp8(const void* x, int T, int H, const int32_t* dest_row, int k, void* recv_q, float* recv_scale,
                    int64_t recv_rows, void* stream) {
  int rc = ep::check_common(T, k, H, "ep_dispatch_fp8");
  if (rc) return rc;
  rc = ep::check_rows(H, recv_rows, T, "ep_dispatch_fp8");
  if (rc) return rc;
  if (H % 16 != 0) return fail(EP_ERR_INVALID_ARG, "ep_dispatch_fp8: H = %d must be a multiple of 16", H);
  if (T > 0 && (!x || !dest_row || (recv_rows > 0 && (!recv_q || !recv_scale))))
    return fail(EP_ERR_INVALID_ARG, "ep_dispatch_fp8: null x/dest_row/recv_q/recv_scale");
  if (!aligned(x, 16) || !aligned(recv_q, 16))
    return fail(EP_ERR_ALIGNMENT, "ep_dispatch_fp8: a row tensor not 16-byte aligned");
  if (!aligned(dest_row, 4) || !aligned(recv_scale, 4))
    return fail(EP_ERR_ALIGNMENT, "ep_dispatch_fp8: dest_row/recv_scale not 4-byte aligned");
  if (T == 0 || recv_rows == 0) return EP_OK;
  ep::Budget b;
  rc = ep::current_device(&b, stream);
  if (rc) return rc;
  hipError_t e = ep::launch_dispatch_fp8(b, x, T, H, dest_row, k, recv_q, recv_scale, recv_rows,
                                         static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return ep::hip_fail(e, "ep_dispatch_fp8 launch");
  return EP_OK;
}

int ep_grouped_gemm_fp8(const void* a, const float* a_scale, int64_t rows, int K, const int32_t* offsets, int E,
                        const void* b, const float* b_scale, int N, void* y, void* stream) {
  const ep::GroupedArgs g = {a, a_scale, rows, K, offsets, E, b, b_scale, N, y, nullptr};
  int rc = check_grouped(g, "ep_grouped_gemm_fp8", "N", N, 8);
  if (rc) return rc;
  return run_grouped(g, false, stream, "ep_grouped_gemm_fp8 launch");
}

int ep_grouped_swiglu_fp8(const void* a, const float* a_scale, int64_t rows, int K, const int32_t* offsets, int E,
                          const void* b, const float* b_scale, int I, void* out_q, float* out_scale, void* stream) {
  if (I > INT32_MAX / 2) return fail(EP_ERR_INVALID_ARG, "ep_grouped_swiglu_fp8: I = %d too large", I);
  const ep::GroupedArgs g = {a, a_scale, rows, K, offsets, E, b, b_scale, 2 * I, out_q, out_scale};
  int rc = check_grouped(g, "ep_grouped_swiglu_fp8", "I", I, 64);
  if (rc) return rc;
  if (rows > 0 && !out_scale) return fail(EP_ERR_INVALID_ARG, "ep_grouped_swiglu_fp8: null out_scale");
  return run_grouped(g, true, stream, "ep_grouped_swiglu_fp8 launch");
}

int ep_combine_backward(const void* dout, const void* y, int64_t recv_rows, int H, const int32_t* dest_row,
                        const float* topk_w, int T, int k, void* dy, float* dw, void* stream) {
  int rc = ep::check_common(T, k, H, "ep_combine_backward");
  if (rc) return rc;
  rc = ep::check_rows(H, recv_rows, T, "ep_combine_backward");
  if (rc) return rc;
  if (!dy && !dw) return fail(EP_ERR_INVALID_ARG, "ep_combine_backward: neither dy nor dw is wanted");
  if (T > 0 && (!dout || !dest_row || (dy && !topk_w) || (dw && !y && recv_rows > 0)))
    return fail(EP_ERR_INVALID_ARG, "ep_combine_backward: null dout/y/dest_row/topk_w");
  if (!aligned(dout, 16) || !aligned(y, 16) || !aligned(dy, 16))
    return fail(EP_ERR_ALIGNMENT, "ep_combine_backward: bf16 tensor not 16-byte aligned");
  if (!aligned(dest_row, 4) || !aligned(topk_w, 4) || !aligned(dw, 4))
    return fail(EP_ERR_ALIGNMENT, "ep_combine_backward: dest_row/topk_w/dw not 4-byte aligned");
  if (T == 0 || (recv_rows == 0 && !dw)) return EP_OK;
  ep::Budget b;
  rc = ep::current_device(&b, stream);
  if (rc) return rc;
  hipError_t e = ep::launch_combine_backward(b, dout, y, recv_rows, H, dest_row, topk_w, T, k, dy, dw,
                                             static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return ep::hip_fail(e, "ep_combine_backward launch");
  return EP_OK;
}

int ep_dispatch_backward(const void* drecv, int64_t recv_rows, int H, const int32_t* dest_row, int T, int k, void* dx,
                         void* stream) {
  int rc = ep::check_common(T, k, H, "ep_dispatch_backward");
  if (rc) return rc;
  rc = ep::check_rows(H, recv_rows, T, "ep_dispatch_backward");
  if (rc) return rc;
  if (T > 0 && (!dest_row || !dx || (!drecv && recv_rows > 0)))
    return fail(EP_ERR_INVALID_ARG, "ep_dispatch_backward: null drecv/dest_row/dx");
  if (!aligned(drecv, 16) || !aligned(dx, 16))
    return fail(EP_ERR_ALIGNMENT, "ep_dispatch_backward: bf16 tensor not 16-byte aligned");
  if (!aligned(dest_row, 4)) return fail(EP_ERR_ALIGNMENT, "ep_dispatch_backward: dest_row not 4-byte aligned");
  if (T == 0) return EP_OK;
  ep::Budget b;
  rc = ep::current_device(&b, stream);
  if (rc) return rc;
  hipError_t e = ep::launch_dispatch_backward(b, drecv, recv_rows, H, dest_row, T, k, dx,
                                              static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return ep::hip_fail(e, "ep_dispatch_backward launch");
  return EP_OK;
}

}  // extern "C"
