// ep_route and ep_route_backward: the router's choice of experts for each
// token, its weights, and the weights' gradient to the logits.
#include <math.h>

#include "ep.h"
#include "ep_device.hpp"
#include "layer_internal.hpp"

namespace ep {

namespace {

constexpr int kRouteWaves = 4;
constexpr int kPerLane = kMaxExperts / kWave;

__device__ __forceinline__ float logit_at(const void* logits, int bf16, int64_t i) {
  return bf16 ? __uint_as_float((uint32_t) static_cast<const uint16_t*>(logits)[i] << 16)
              : static_cast<const float*>(logits)[i];
}

// An integer that orders as v does, NaN above everything, -0 as +0; kGone is
// below all of them.
constexpr int64_t kGone = INT64_MIN;
__device__ __forceinline__ int64_t order_of(double v) {
  if (v != v) return INT64_MAX;
  const int64_t b = __double_as_longlong(v + 0.0);
  return b < 0 ? b ^ INT64_MAX : b;
}

// The larger key of two lanes, of equal ones the lower index: over the wave.
__device__ __forceinline__ void wave_best(int64_t& key, int& at) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int64_t k = __shfl_xor(key, d, kWave);
    const int i = __shfl_xor(at, d, kWave);
    if (k > key || (k == key && i < at)) {
      key = k;
      at = i;
    }
  }
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d, kWave);
  return v;
}

__device__ __forceinline__ double sigmoid64(double l) {
  const double e = exp(-fabs(l));
  return (l < 0.0 ? e : 1.0) / (1.0 + e);
}

// One token by one wave, scores in float64.  s_c: E doubles of LDS.
__device__ void route_exact(const RouteArgs& a, int64_t t, int lane, double* s_c) {
  const int E = a.E;
  double l[kPerLane], c[kPerLane];
  double top = -INFINITY, total = 0.0;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int e = i * kWave + lane;
    l[i] = e < E ? (double)logit_at(a.logits, a.bf16, t * E + e) : -INFINITY;
    top = l[i] > top || l[i] != l[i] ? l[i] : top;
  }
  if (!a.sigmoid) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const double o = __shfl_xor(top, d, kWave);
      top = o > top || o != o ? o : top;
    }
  }
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    c[i] = 0.0;
    if (i * kWave >= E) continue;
    if (a.sigmoid) c[i] = sigmoid64(l[i]);
    else if (top != -INFINITY) c[i] = exp(l[i] - top);
    if (i * kWave + lane >= E) c[i] = 0.0;
    total += c[i];
  }
  if (a.sigmoid) total = 1.0;
  else total = wave_sum(total);
  // (a row of -infinity alone: scores 0)
  const bool none = !a.sigmoid && top == -INFINITY;
  int64_t key[kPerLane];
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int e = i * kWave + lane;
    key[i] = kGone;
    if (e >= E) continue;
    c[i] = none ? 0.0 : c[i] / total;
    if (a.bias) c[i] += (double)a.bias[e];
    key[i] = order_of(a.bias ? c[i] : l[i]);
    if (a.groups > 1) s_c[e] = c[i];
  }
  if (a.groups > 1) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int per = E / a.groups;
    int64_t rank = kGone;
    if (lane < a.groups) {
      int64_t k1 = kGone, k2 = kGone;
      double v1 = 0.0, v2 = 0.0;
      for (int i = 0; i < per; ++i) {
        const double v = s_c[lane * per + i];
        const int64_t k = order_of(v);
        if (k > k1) {
          k2 = k1, v2 = v1;
          k1 = k, v1 = v;
        } else if (k > k2) {
          k2 = k, v2 = v;
        }
      }
      rank = order_of(a.group_best == 2 ? v1 + v2 : v1);
    }
    uint64_t kept = 0;
    for (int i = 0; i < a.top_groups; ++i) {
      int64_t best = rank;
      int at = lane;
      wave_best(best, at);
      kept |= 1ull << at;
      if (lane == at) rank = kGone;
    }
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int e = i * kWave + lane;
      if (e < E && !(kept >> (e / per) & 1)) key[i] = kGone;
    }
  }
  int mine = 0;        // lane j: the expert of slot j
  double logit = 0.0;  // and its logit
  for (int j = 0; j < a.k; ++j) {
    int64_t best = kGone;
    int at = INT32_MAX;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i * kWave + lane;
      }
    wave_best(best, at);
    double v = 0.0;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      if (i * kWave + lane == at) {
        key[i] = kGone;
        v = l[i];
      }
    v = __shfl(v, at & (kWave - 1), kWave);
    if (lane == j) {
      mine = at;
      logit = v;
    }
  }
  // ---- the weights
  const bool here = lane < a.k;
  double w;
  if (a.renorm) {
    // sigmoid: both the score and the sum times exp(-shift), shift the largest
    // chosen logit where that is negative
    double shift = here ? logit : -INFINITY;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const double o = __shfl_xor(shift, d, kWave);
      shift = o > shift || o != o ? o : shift;
    }
    const bool empty = shift == -INFINITY;
    if (a.sigmoid) {
      if (shift > 0.0) shift = 0.0;
      w = logit > 0.0 ? 1.0 / (1.0 + exp(-logit)) * exp(-shift) : exp(logit - shift) / (1.0 + exp(logit));
    } else {
      w = exp(logit - shift);
    }
    if (!here || empty) w = 0.0;
    const double sum = wave_sum(w);
    w = empty ? 0.0 : w / sum;
    if (total != total) w = total;
  } else {
    w = a.sigmoid ? sigmoid64(logit) : none ? 0.0 : exp(logit - top) / total;
  }
  if (here) {
    a.idx[t * a.k + lane] = mine;
    a.w[t * a.k + lane] = (float)w * a.scale;
  }
}

__global__ __launch_bounds__(kRouteWaves * kWave) void route_kernel(RouteArgs a) {
  __shared__ double s_c[kRouteWaves][kMaxExperts];
  const int wave = wave_in_group();
  const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
  if (t < a.T) route_exact(a, t, lane_id(), s_c[wave]);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d, kWave);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v = fmaxf(v, __shfl_xor(v, d, kWave));
  return v;
}

__global__ __launch_bounds__(kRouteWaves * kWave) void route_backward_kernel(RouteBackwardArgs a) {
  const int lane = lane_id();
  const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave_in_group();
  if (t >= a.T) return;
  const int E = a.E;
  // lane j: slot j
  const int e = lane < a.k ? a.idx[t * a.k + lane] : -1;
  const bool here = e >= 0 && e < E;
  const float dw = here ? a.dw[t * a.k + lane] : 0.0f;
  const float l = here ? logit_at(a.logits, a.bf16, t * E + e) : -INFINITY;
  const bool dense = !a.sigmoid && !a.renorm;
  float top = 0.0f, total = 1.0f;
  if (dense) {
    top = -INFINITY;
    bool nan = false;
    for (int i = lane; i < E; i += kWave) {
      const float v = logit_at(a.logits, a.bf16, t * E + i);
      nan |= v != v;
      top = fmaxf(top, v);
    }
    top = wave_max(top);
    total = 0.0f;
    for (int i = lane; i < E; i += kWave) total += expf(logit_at(a.logits, a.bf16, t * E + i) - top);
    total = wave_sum(total);
    if (top == -INFINITY) total = 1.0f, top = 0.0f;
    if (ballot(nan)) total = NAN;
  }
  float p = 0.0f;  // the slot's share
  float sig = 1.0f / (1.0f + expf(-l));
  if (a.renorm) {
    float shift = wave_max(l);
    if (ballot(here && l != l)) shift = NAN;
    const bool empty = shift == -INFINITY;
    if (a.sigmoid) {
      shift = shift > 0.0f ? 0.0f : shift;
      p = l > 0.0f ? sig * expf(-shift) : expf(l - shift) / (1.0f + expf(l));
    } else {
      p = expf(l - shift);
    }
    if (!here || empty) p = 0.0f;
    const float sum = wave_sum(p);
    if (!empty) p /= sum;
  } else if (here) {
    p = a.sigmoid ? sig : expf(l - top) / total;
  }
  const float D = a.renorm || !a.sigmoid ? wave_sum(p * dw) : 0.0f;
  // the slot's own part (dense: without the part that every expert has)
  float g = dense ? p * dw : p * (dw - D);
  if (a.sigmoid) g *= 1.0f - sig;
  if (!here) g = 0.0f;
  for (int base = 0; base < E; base += kWave) {
    const int i = base + lane;
    float v = 0.0f;
    if (dense && i < E) v = -D * (expf(logit_at(a.logits, a.bf16, t * E + i) - top) / total);
    for (int j = 0; j < a.k; ++j) {
      const int ej = __shfl(e, j, kWave);
      const float gj = __shfl(g, j, kWave);
      if (ej == i) v += gj;
    }
    v *= a.scale;
    if (i < E) {
      if (a.out_bf16) static_cast<uint16_t*>(a.dlogits)[t * E + i] = (uint16_t)pack_bf16x2(v, v);
      else static_cast<float*>(a.dlogits)[t * E + i] = v;
    }
  }
}

}  // namespace

hipError_t launch_route(const Budget& b, const RouteArgs& a, hipStream_t stream) {
  (void)b;
  hipLaunchKernelGGL(route_kernel, dim3((a.T + kRouteWaves - 1) / kRouteWaves), dim3(kRouteWaves * kWave), 0, stream,
                     a);
  return hipGetLastError();
}

hipError_t launch_route_backward(const Budget& b, const RouteBackwardArgs& a, hipStream_t stream) {
  (void)b;
  hipLaunchKernelGGL(route_backward_kernel, dim3((a.T + kRouteWaves - 1) / kRouteWaves), dim3(kRouteWaves * kWave), 0,
                     stream, a);
  return hipGetLastError();
}

}  // namespace ep
