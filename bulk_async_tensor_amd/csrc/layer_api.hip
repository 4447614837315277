// C ABI of ep_layer.h: argument checks and launches on the caller's stream.
// As in ep_api.hip, every host-detectable error is reported before any HIP
// call is made.
#include <math.h>

#include "ep_host.hpp"
#include "ep_layer.h"
#include "layer_internal.hpp"

using ep::aligned;
using ep::fail;

static_assert(EP_MAX_GROUPS == ep::kMaxGroups && EP_MAX_EXPERTS == ep::kMaxExperts, "the kernels' limits are the ABI's");

namespace {

bool is_type(int type) { return type == EP_BF16 || type == EP_F32; }
size_t size_of(int type) { return type == EP_BF16 ? 2 : 4; }

int check_router(const char* what, int type, int T, int E, int score, int k, float scale) {
  if (!is_type(type)) return fail(EP_ERR_INVALID_ARG, "%s: logits_type = %d", what, type);
  if (score != EP_SCORE_SOFTMAX && score != EP_SCORE_SIGMOID)
    return fail(EP_ERR_INVALID_ARG, "%s: score = %d", what, score);
  int rc = ep::check_common(T, k, E, what);
  if (rc) return rc;
  if (E < 1 || E > EP_MAX_EXPERTS)
    return fail(EP_ERR_INVALID_ARG, "%s: E = %d outside [1, %d]", what, E, EP_MAX_EXPERTS);
  if (k > E) return fail(EP_ERR_INVALID_ARG, "%s: k = %d exceeds E = %d", what, k, E);
  if ((int64_t)T * E > EP_MAX_ENTRIES)
    return fail(EP_ERR_INVALID_ARG, "%s: T * E = %lld exceeds EP_MAX_ENTRIES", what, (long long)T * E);
  if (!isfinite(scale)) return fail(EP_ERR_INVALID_ARG, "%s: scale is not finite", what);
  return EP_OK;
}

int check_product(const char* what, int64_t rows, int N, int K, int E, const void* offsets, int act) {
  if (rows < 0 || rows > EP_MAX_ENTRIES)
    return fail(EP_ERR_INVALID_ARG, "%s: rows = %lld outside [0, EP_MAX_ENTRIES]", what, (long long)rows);
  if (N <= 0 || N % 8 != 0 || N > EP_LINEAR_MAX_SIDE)
    return fail(EP_ERR_INVALID_ARG, "%s: N = %d must be a positive multiple of 8 up to %d", what, N,
                EP_LINEAR_MAX_SIDE);
  if (K <= 0 || K % 8 != 0 || K > EP_LINEAR_MAX_SIDE)
    return fail(EP_ERR_INVALID_ARG, "%s: K = %d must be a positive multiple of 8 up to %d", what, K,
                EP_LINEAR_MAX_SIDE);
  if ((int64_t)N * K > EP_LINEAR_MAX_WEIGHT)
    return fail(EP_ERR_INVALID_ARG, "%s: a weight of %lld values exceeds 2^30 - 1", what, (long long)N * K);
  if (E < 1 || E > EP_MAX_EXPERTS)
    return fail(EP_ERR_INVALID_ARG, "%s: E = %d outside [1, %d]", what, E, EP_MAX_EXPERTS);
  if (!offsets && E != 1) return fail(EP_ERR_INVALID_ARG, "%s: null offsets with E = %d", what, E);
  if (!aligned(offsets, 4)) return fail(EP_ERR_ALIGNMENT, "%s: offsets not 4-byte aligned", what);
  if (act < EP_ACT_NONE || act > EP_ACT_SWIGLU) return fail(EP_ERR_INVALID_ARG, "%s: act = %d", what, act);
  return EP_OK;
}

int check_needs(const char* what, const ep::LinearNeeds& needs, const void* workspace, size_t bytes) {
  if (!needs.fits) return fail(EP_ERR_INVALID_ARG, "%s: more than 2^30 tiles of results", what);
  const size_t need = needs.workspace;
  if (need == 0) return EP_OK;
  if (!workspace || bytes < need)
    return fail(EP_ERR_WORKSPACE, "%s: a workspace of %zu bytes is needed, %zu given", what, need,
                workspace ? bytes : (size_t)0);
  if (!aligned(workspace, 16)) return fail(EP_ERR_ALIGNMENT, "%s: workspace not 16-byte aligned", what);
  return EP_OK;
}

bool sizes_fit(int64_t rows, int K, int E, int N) {
  return rows >= 0 && rows <= EP_MAX_ENTRIES && K > 0 && N > 0 && K <= EP_LINEAR_MAX_SIDE && N <= EP_LINEAR_MAX_SIDE &&
         E >= 1 && E <= EP_MAX_EXPERTS;
}

template <class Args, class Launch>
int run(const char* what, const Args& a, Launch launch, void* stream) {
  ep::Budget b;
  int rc = ep::current_device(&b, stream);
  if (rc) return rc;
  hipError_t e = launch(b, a, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return ep::hip_fail(e, what);
  return EP_OK;
}

}  // namespace

extern "C" {

int ep_route(const void* logits, int logits_type, int T, int E, int score, const float* bias, int groups,
             int top_groups, int group_best, int k, int renormalize, float scale, int32_t* topk_idx, float* topk_w,
             void* stream) {
  int rc = check_router("ep_route", logits_type, T, E, score, k, scale);
  if (rc) return rc;
  if (groups < 1 || groups > EP_MAX_GROUPS || E % groups != 0)
    return fail(EP_ERR_INVALID_ARG, "ep_route: groups = %d must divide E = %d and be at most %d", groups, E,
                EP_MAX_GROUPS);
  if (top_groups < 1 || top_groups > groups)
    return fail(EP_ERR_INVALID_ARG, "ep_route: top_groups = %d outside [1, %d]", top_groups, groups);
  if (group_best < 1 || group_best > 2 || group_best > E / groups)
    return fail(EP_ERR_INVALID_ARG, "ep_route: group_best = %d must be 1 or 2 and at most E / groups", group_best);
  if (k > top_groups * (E / groups))
    return fail(EP_ERR_INVALID_ARG, "ep_route: k = %d exceeds the %d experts of the best groups", k,
                top_groups * (E / groups));
  if (T > 0 && (!logits || !topk_idx || !topk_w))
    return fail(EP_ERR_INVALID_ARG, "ep_route: null logits/topk_idx/topk_w");
  if (!aligned(logits, size_of(logits_type)) || !aligned(bias, 4) || !aligned(topk_idx, 4) || !aligned(topk_w, 4))
    return fail(EP_ERR_ALIGNMENT, "ep_route: a tensor not aligned to its element");
  if (T == 0) return EP_OK;
  const ep::RouteArgs a = {logits, logits_type == EP_BF16, T,          E,     score == EP_SCORE_SIGMOID,
                           bias,   groups,                 top_groups, group_best, k,
                           renormalize != 0, scale, topk_idx, topk_w};
  return run("ep_route launch", a, ep::launch_route, stream);
}

int ep_route_backward(const void* logits, int logits_type, int T, int E, int score, const int32_t* topk_idx, int k,
                      int renormalize, float scale, const float* dw, void* dlogits, int dlogits_type, void* stream) {
  int rc = check_router("ep_route_backward", logits_type, T, E, score, k, scale);
  if (rc) return rc;
  if (!is_type(dlogits_type)) return fail(EP_ERR_INVALID_ARG, "ep_route_backward: dlogits_type = %d", dlogits_type);
  if (T > 0 && (!logits || !topk_idx || !dw || !dlogits))
    return fail(EP_ERR_INVALID_ARG, "ep_route_backward: null logits/topk_idx/dw/dlogits");
  if (!aligned(logits, size_of(logits_type)) || !aligned(dlogits, size_of(dlogits_type)) || !aligned(topk_idx, 4) ||
      !aligned(dw, 4))
    return fail(EP_ERR_ALIGNMENT, "ep_route_backward: a tensor not aligned to its element");
  if (T == 0) return EP_OK;
  const ep::RouteBackwardArgs a = {logits, logits_type == EP_BF16, T, E, score == EP_SCORE_SIGMOID, topk_idx, k,
                                   renormalize != 0, scale, dw, dlogits, dlogits_type == EP_BF16};
  return run("ep_route_backward launch", a, ep::launch_route_backward, stream);
}

size_t ep_grouped_linear_workspace_bytes(int64_t rows, int K, int E, int N) {
  return sizes_fit(rows, K, E, N) ? ep::linear_needs(rows, K, E, N).workspace : 0;
}
size_t ep_grouped_linear_dgrad_workspace_bytes(int64_t rows, int K, int E, int N) {
  return sizes_fit(rows, K, E, N) ? ep::dgrad_needs(rows, K, E, N).workspace : 0;
}
size_t ep_grouped_linear_wgrad_workspace_bytes(int64_t rows, int K, int E, int N) {
  return sizes_fit(rows, K, E, N) ? ep::wgrad_needs(rows, K, E, N).workspace : 0;
}

int ep_grouped_linear(const void* a, int64_t rows, int K, const int32_t* offsets, int E, const void* b,
                      const float* bias, int N, int act, const void* residual, void* y, int y_type, void* pre,
                      void* workspace, size_t workspace_bytes, void* stream) {
  const char* what = "ep_grouped_linear";
  int rc = check_product(what, rows, N, K, E, offsets, act);
  if (rc) return rc;
  if (act == EP_ACT_SWIGLU && N % 16 != 0)
    return fail(EP_ERR_INVALID_ARG, "%s: N = %d must be a multiple of 16 with swiglu", what, N);
  if (!is_type(y_type)) return fail(EP_ERR_INVALID_ARG, "%s: y_type = %d", what, y_type);
  if (rows > 0 && (!a || !b || !y)) return fail(EP_ERR_INVALID_ARG, "%s: null a/b/y", what);
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(residual, 16) || !aligned(y, 16) || !aligned(pre, 16))
    return fail(EP_ERR_ALIGNMENT, "%s: a tensor not 16-byte aligned", what);
  if (!aligned(bias, 4)) return fail(EP_ERR_ALIGNMENT, "%s: bias not 4-byte aligned", what);
  if (rows == 0) return EP_OK;
  rc = check_needs(what, ep::linear_needs(rows, K, E, N), workspace, workspace_bytes);
  if (rc) return rc;
  ep::LinearArgs g = {};
  g.rows_in = a, g.cols_in = b, g.rows = rows, g.N = N, g.K = K, g.offsets = offsets, g.E = E, g.act = act;
  g.bias = bias, g.residual = residual, g.pre_out = pre, g.out = y, g.out_f32 = y_type == EP_F32;
  g.partial = static_cast<float*>(workspace);
  return run("ep_grouped_linear launch", g, ep::launch_linear, stream);
}

int ep_grouped_linear_dgrad(const void* dy, int64_t rows, int N, const int32_t* offsets, int E, const void* b, int K,
                            int act, const void* pre, void* dx, void* workspace, size_t workspace_bytes,
                            void* stream) {
  const char* what = "ep_grouped_linear_dgrad";
  int rc = check_product(what, rows, N, K, E, offsets, act);
  if (rc) return rc;
  if (rows > 0 && (!dy || !b || !dx)) return fail(EP_ERR_INVALID_ARG, "%s: null dy/b/dx", what);
  if (rows > 0 && act != EP_ACT_NONE && !pre)
    return fail(EP_ERR_INVALID_ARG, "%s: an activation's gradient needs pre", what);
  if (!aligned(dy, 16) || !aligned(b, 16) || !aligned(pre, 16) || !aligned(dx, 16))
    return fail(EP_ERR_ALIGNMENT, "%s: a tensor not 16-byte aligned", what);
  if (rows == 0) return EP_OK;
  rc = check_needs(what, ep::dgrad_needs(rows, K, E, N), workspace, workspace_bytes);
  if (rc) return rc;
  ep::LinearArgs g = {};
  g.rows_in = dy, g.cols_in = b, g.rows = rows, g.N = N, g.K = K, g.offsets = offsets, g.E = E, g.act = act;
  g.pre_in = pre, g.out = dx, g.partial = static_cast<float*>(workspace);
  return run("ep_grouped_linear_dgrad launch", g, ep::launch_dgrad, stream);
}

int ep_grouped_linear_wgrad(const void* dy, const void* a, int64_t rows, int N, int K, const int32_t* offsets, int E,
                            void* db, int db_type, float* dbias, void* workspace, size_t workspace_bytes,
                            void* stream) {
  const char* what = "ep_grouped_linear_wgrad";
  int rc = check_product(what, rows, N, K, E, offsets, EP_ACT_NONE);
  if (rc) return rc;
  if (!is_type(db_type)) return fail(EP_ERR_INVALID_ARG, "%s: db_type = %d", what, db_type);
  if (!db || (rows > 0 && (!dy || !a))) return fail(EP_ERR_INVALID_ARG, "%s: null dy/a/db", what);
  if (!aligned(dy, 16) || !aligned(a, 16) || !aligned(db, 16))
    return fail(EP_ERR_ALIGNMENT, "%s: a tensor not 16-byte aligned", what);
  if (!aligned(dbias, 4)) return fail(EP_ERR_ALIGNMENT, "%s: dbias not 4-byte aligned", what);
  rc = check_needs(what, ep::wgrad_needs(rows, K, E, N), workspace, workspace_bytes);
  if (rc) return rc;
  ep::LinearArgs g = {};
  g.rows_in = dy, g.cols_in = a, g.rows = rows, g.N = N, g.K = K, g.offsets = offsets, g.E = E;
  g.out = db, g.out_f32 = db_type == EP_F32, g.dbias = dbias, g.partial = static_cast<float*>(workspace);
  return run("ep_grouped_linear_wgrad launch", g, ep::launch_wgrad, stream);
}

}  // extern "C"
