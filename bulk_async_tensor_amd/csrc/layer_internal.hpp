// Host-side interfaces between the C ABI of ep_layer.h (layer_api.hip) and its
// kernel files.
#pragma once

#include "ep_internal.hpp"

namespace ep {

constexpr int kMaxGroups = 64;    // the ABI's EP_MAX_GROUPS
constexpr int kMaxExperts = 1024;  // the ABI's EP_MAX_EXPERTS

// ---- route.hip
struct RouteArgs {
  const void* logits;
  int bf16, T, E, sigmoid;
  const float* bias;
  int groups, top_groups, group_best, k, renorm;
  float scale;
  int32_t* idx;
  float* w;
};
hipError_t launch_route(const Budget& b, const RouteArgs& a, hipStream_t stream);

struct RouteBackwardArgs {
  const void* logits;
  int bf16, T, E, sigmoid;
  const int32_t* idx;
  int k, renorm;
  float scale;
  const float* dw;
  void* dlogits;
  int out_bf16;
};
hipError_t launch_route_backward(const Budget& b, const RouteBackwardArgs& a, hipStream_t stream);

// ---- linear_wide.hip: one product of the three
struct LinearArgs {
  const void* rows_in;  // a or dy, [rows, ...]
  const void* cols_in;  // b, or wgrad's a
  int64_t rows;
  int N, K;  // a weight's sides
  const int32_t* offsets;
  int E;
  int act;
  const float* bias;
  const void* residual;
  const void* pre_in;  // dgrad
  void* pre_out;       // linear
  void* out;
  int out_f32;
  float* dbias;
  float* partial;  // the workspace
};
struct LinearNeeds {
  size_t workspace;
  bool fits;  // no more tiles than a launch counts
};
LinearNeeds linear_needs(int64_t rows, int K, int E, int N);
LinearNeeds dgrad_needs(int64_t rows, int K, int E, int N);
LinearNeeds wgrad_needs(int64_t rows, int K, int E, int N);
hipError_t launch_linear(const Budget& b, const LinearArgs& g, hipStream_t stream);
hipError_t launch_dgrad(const Budget& b, const LinearArgs& g, hipStream_t stream);
hipError_t launch_wgrad(const Budget& b, const LinearArgs& g, hipStream_t stream);

}  // namespace ep
