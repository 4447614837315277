// What follows the experts' bf16 products: bias, activation and residual, and
// the activation's derivative on the way back, for four neighbouring results
// of a row.
#pragma once

#include "ep_device.hpp"
#include "ep_layer.h"
#include "layer_internal.hpp"

namespace ep {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

// four float32 at a float's alignment
typedef f32x4 f32x4_at4 __attribute__((aligned(4)));
__device__ __forceinline__ f32x4 load4_f32(const float* p, int64_t at) {
  return *reinterpret_cast<const f32x4_at4*>(p + at);
}
__device__ __forceinline__ f32x4 load4_bf16(const void* p, int64_t at) {
  const u32x2 v = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(p) + at);
  return f32x4{bf16_lo(v[0]), bf16_hi(v[0]), bf16_lo(v[1]), bf16_hi(v[1])};
}
__device__ __forceinline__ void store4_bf16(void* p, int64_t at, f32x4 v) {
  *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p) + at) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

// 1 / (1 + exp(-z)): exp overflows below -88.7, where the quotient is 0.
__device__ __forceinline__ float sigmoid_of(float z) { return 1.0f / (1.0f + expf(-z)); }
// (1 + erf(z / sqrt 2)) / 2 by the complement, which keeps its places far below zero
__device__ __forceinline__ float normal_cdf(float z) { return 0.5f * erfcf(z * -0.70710678f); }

__device__ __forceinline__ float activate(int act, float z) {
  if (act == EP_ACT_SILU || act == EP_ACT_SWIGLU) return z / (1.0f + expf(-z));
  if (act == EP_ACT_GELU) return z * normal_cdf(z);
  return z;
}
// The derivative of activate().
__device__ __forceinline__ float activate_slope(int act, float z) {
  if (act == EP_ACT_SILU || act == EP_ACT_SWIGLU) {
    const float s = sigmoid_of(z);
    return s * (1.0f + z * (1.0f - s));
  }
  if (act == EP_ACT_GELU) return normal_cdf(z) + z * (0.39894228f * expf(-0.5f * z * z));
  return 1.0f;
}

// Results n .. n + 3 of row r of expert e, act not EP_ACT_SWIGLU.
__device__ __forceinline__ void finish_linear(const LinearArgs& g, int act, int e, int64_t r, int n, f32x4 z) {
  if (g.bias) z += load4_f32(g.bias, (int64_t)e * g.N + n);
  if (g.pre_out) store4_bf16(g.pre_out, r * g.N + n, z);
#pragma unroll
  for (int i = 0; i < 4; ++i) z[i] = activate(act, z[i]);
  if (g.residual) z += load4_bf16(g.residual, r * g.N + n);
  if (g.out_f32) *reinterpret_cast<f32x4*>(static_cast<float*>(g.out) + r * g.N + n) = z;
  else store4_bf16(g.out, r * g.N + n, z);
}
// EP_ACT_SWIGLU: gate and up products n .. n + 3.
__device__ __forceinline__ void finish_swiglu(const LinearArgs& g, int e, int64_t r, int n, f32x4 gate, f32x4 up) {
  const int outs = g.N / 2;
  if (g.bias) {
    gate += load4_f32(g.bias, (int64_t)e * g.N + n);
    up += load4_f32(g.bias, (int64_t)e * g.N + outs + n);
  }
  if (g.pre_out) {
    store4_bf16(g.pre_out, r * g.N + n, gate);
    store4_bf16(g.pre_out, r * g.N + outs + n, up);
  }
  f32x4 z;
#pragma unroll
  for (int i = 0; i < 4; ++i) z[i] = activate(EP_ACT_SILU, gate[i]) * up[i];
  if (g.residual) z += load4_bf16(g.residual, r * outs + n);
  if (g.out_f32) *reinterpret_cast<f32x4*>(static_cast<float*>(g.out) + r * outs + n) = z;
  else store4_bf16(g.out, r * outs + n, z);
}
// The gradient of row r at i .. i + 3 through the activation that made it.
__device__ __forceinline__ void finish_dgrad(const LinearArgs& g, int act, int64_t r, int i, f32x4 d) {
  if (act == EP_ACT_SWIGLU) {
    const int64_t at = r * 2 * g.K + i;
    const f32x4 gate = load4_bf16(g.pre_in, at), up = load4_bf16(g.pre_in, at + g.K);
    f32x4 dg, du;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      dg[j] = activate_slope(EP_ACT_SILU, gate[j]) * up[j] * d[j];
      du[j] = activate(EP_ACT_SILU, gate[j]) * d[j];
    }
    store4_bf16(g.out, at, dg);
    store4_bf16(g.out, at + g.K, du);
    return;
  }
  const int64_t at = r * g.K + i;
  if (act != EP_ACT_NONE) {
    const f32x4 z = load4_bf16(g.pre_in, at);
#pragma unroll
    for (int j = 0; j < 4; ++j) d[j] *= activate_slope(act, z[j]);
  }
  store4_bf16(g.out, at, d);
}

}  // namespace ep
