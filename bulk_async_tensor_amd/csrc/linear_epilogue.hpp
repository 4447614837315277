// What follows the experts' bf16 products: bias, activation and residual, and
// the activation's derivative on the way back.
#pragma once

#include "ep_device.hpp"
#include "ep_layer.h"
#include "fp8_device.hpp"
#include "layer_internal.hpp"

namespace ep {

// four float32 at a float's alignment
typedef f32x4 f32x4_at4 __attribute__((aligned(4)));
__device__ __forceinline__ f32x4 load4_f32(const float* p, int64_t at) {
  return *reinterpret_cast<const f32x4_at4*>(p + at);
}
__device__ __forceinline__ f32x4 widen4(uint32_t lo, uint32_t hi) {
  return f32x4{bf16_lo(lo), bf16_hi(lo), bf16_lo(hi), bf16_hi(hi)};
}
__device__ __forceinline__ u32x2 narrow4(f32x4 v) { return u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])}; }
__device__ __forceinline__ f32x4 load4_bf16(const void* p, int64_t at) {
  const u32x2 v = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(p) + at);
  return widen4(v[0], v[1]);
}
__device__ __forceinline__ void store4_bf16(void* p, int64_t at, f32x4 v) {
  *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p) + at) = narrow4(v);
}

// exp(z) by the hardware's 2^x: the argument's rounding costs 1.5 |z| steps of
// float32 at most, the instruction one.
__device__ __forceinline__ float exp_of(float z) { return __builtin_amdgcn_exp2f(z * 1.44269504f); }
// 1 / (1 + exp(-z)): exp overflows below -88.7, where the quotient is 0.  (The
// hardware's reciprocal, one step off, for the 10 instructions of a division.)
__device__ __forceinline__ float sigmoid_of(float z) { return __builtin_amdgcn_rcpf(1.0f + exp_of(-z)); }

// (1 + erf(z / sqrt 2)) / 2.  With x = |z| / sqrt 2 and t = 1 / (1 + x / 3),
//   erfc(x) = t exp(-x^2 + p(t)),
// p of degree 9 fitted to log(erfc(x) exp(x^2) / t) over x in [0, 10], where it
// is 1.5e-8 off.  22 instructions for the library function's 100.  Far below
// zero the rounding of the argument shows, of which exp makes z^2 / 2 half
// steps and more: relative to its value it is 4 steps of float32 off at -1, 9 at
// -5, 33 at -10 and 63 at -13, a five-hundredth of a bf16 rounding.
__device__ __forceinline__ float normal_cdf(float z) {
  const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(z), 0.23570226f, 1.0f));
  float p = fmaf(-0.311686669f, t, 1.56484535f);
  p = fmaf(p, t, -3.07433251f);
  p = fmaf(p, t, 3.0791728f);
  p = fmaf(p, t, -1.98103654f);
  p = fmaf(p, t, 0.914975638f);
  p = fmaf(p, t, 0.000799481463f);
  p = fmaf(p, t, 0.481627367f);
  p = fmaf(p, t, 0.99646812f);
  p = fmaf(p, t, -1.67083306f);
  const float tail = 0.5f * t * expf(fmaf(-0.5f, z * z, p));
  return z > 0.0f ? 1.0f - tail : tail;
}

template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if constexpr (ACT == EP_ACT_SILU || ACT == EP_ACT_SWIGLU) return z * sigmoid_of(z);
  if constexpr (ACT == EP_ACT_GELU) return z * normal_cdf(z);
  return z;
}
// The derivative of activate().
template <int ACT>
__device__ __forceinline__ float activate_slope(float z) {
  if constexpr (ACT == EP_ACT_SILU || ACT == EP_ACT_SWIGLU) {
    const float s = sigmoid_of(z);
    return s * fmaf(z, 1.0f - s, 1.0f);
  }
  if constexpr (ACT == EP_ACT_GELU) return fmaf(z, 0.39894228f * expf(-0.5f * z * z), normal_cdf(z));
  return 1.0f;
}

template <int ACT>
__device__ __forceinline__ f32x4 activate4(f32x4 z) {
#pragma unroll
  for (int i = 0; i < 4; ++i) z[i] = activate<ACT>(z[i]);
  return z;
}
template <int ACT>
__device__ __forceinline__ f32x4 slope4(f32x4 z) {
#pragma unroll
  for (int i = 0; i < 4; ++i) z[i] = activate_slope<ACT>(z[i]);
  return z;
}

// ---- four neighbouring results of a row, from and to plain pointers (the join
// of a cut sum)

// Results n .. n + 3 of row r of expert e, not EP_ACT_SWIGLU.
template <int ACT>
__device__ __forceinline__ void finish_linear(const LinearArgs& g, int e, int64_t r, int n, f32x4 z) {
  if (g.bias) z += load4_f32(g.bias, (int64_t)e * g.N + n);
  if (g.pre_out) store4_bf16(g.pre_out, r * g.N + n, z);
  z = activate4<ACT>(z);
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
  f32x4 z = activate4<EP_ACT_SILU>(gate) * up;
  if (g.residual) z += load4_bf16(g.residual, r * outs + n);
  if (g.out_f32) *reinterpret_cast<f32x4*>(static_cast<float*>(g.out) + r * outs + n) = z;
  else store4_bf16(g.out, r * outs + n, z);
}
// The gradient of row r at i .. i + 3 through the activation that made it.
template <int ACT>
__device__ __forceinline__ void finish_dgrad(const LinearArgs& g, int64_t r, int i, f32x4 d) {
  if constexpr (ACT == EP_ACT_SWIGLU) {
    const int64_t at = r * 2 * g.K + i;
    const f32x4 gate = load4_bf16(g.pre_in, at), up = load4_bf16(g.pre_in, at + g.K);
    store4_bf16(g.out, at, slope4<EP_ACT_SILU>(gate) * up * d);
    store4_bf16(g.out, at + g.K, activate4<EP_ACT_SILU>(gate) * d);
  } else {
    const int64_t at = r * g.K + i;
    if constexpr (ACT != EP_ACT_NONE) d *= slope4<ACT>(load4_bf16(g.pre_in, at));
    store4_bf16(g.out, at, d);
  }
}
// Four neighbouring values of a weight's gradient.
__device__ __forceinline__ void finish_wgrad(const LinearArgs& g, int64_t at, f32x4 v) {
  if (g.out_f32) *reinterpret_cast<f32x4*>(static_cast<float*>(g.out) + at) = v;
  else store4_bf16(g.out, at, v);
}

}  // namespace ep
