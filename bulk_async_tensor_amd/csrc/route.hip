// ep_route and ep_route_backward: the router's choice of experts for each
// token, its weights, and the weights' gradient to the logits.
//
// ep_route.  The choice has to be that of exact scores, but float32 is enough
// to make nearly all of it: a token's experts are ranked by float32 keys.  Where
// two neighbours of the choice are closer than the keys can be wrong, and not
// equal by having the same logit and bias, a few more experts are taken, up to a
// certain gap, and what lies before it is ranked in float64.  Where that does
// not do either (groups as close at the edge, softmax scores with a bias, a NaN,
// no gap near), the token is done again in float64 by the whole wave
// (route_exact).
//
// 16 lanes take a token (64 where there are more than 512 experts, more than
// 15 are chosen, or few tokens are there), a lane NV neighbouring experts.  A
// key is the 31 high bits of an integer that orders as the score does, its
// lowest bits replaced by the expert's place in the lane, so that keys differ
// within a lane and the largest names its expert.  Choosing one: each lane
// finds its largest key below the last one it gave (key - last wraps to the top
// of the unsigned range exactly for smaller keys, so that is one subtraction
// and half a maximum a key); four exchanges give the token's largest value, a
// ballot the first lane that holds it (of equal values the lowest expert).
//
// us, kernel alone: 128 tokens of 256 experts in 8 groups, k 8 6.7; 16384 of
// them 17.8 (without groups 10.6), 17.8 MB or 1.0 TB/s: 12 are the scores,
// groups and nine rounds of choosing, the rest a token or two that float64
// decides, one load and one exchange after another; 16384 tokens of 64 experts
// in bf16, k 6, 5.6.  The gradient: 4096 tokens of 256 experts 7.6, 8191 of 60
// 6.9: load latency, and for each 64 experts 2 k exchanges and a store of 2 or 4
// bytes a lane.
#include <math.h>

#include "ep.h"
#include "ep_device.hpp"
#include "layer_internal.hpp"
#include "route_shapes.hpp"

namespace ep {

namespace {

constexpr int kRouteWaves = 4;
constexpr int64_t kRouteGroups = 1 << 22;  // workgroups of a launch: a grid has fewer than 2^32 lanes

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

// The exchange of step d within 16 lanes, after which each lane has the value
// of another that held a different half (d = 0, 1: lanes 1 and 2 away; 2, 3:
// the mirrored lane of 8 and of 16).
template <int D>
__device__ __forceinline__ int exchange16(int v) {
  constexpr int ctrl = D == 0 ? 0xB1 : D == 1 ? 0x4E : D == 2 ? 0x141 : 0x140;
  return __builtin_amdgcn_mov_dpp(v, ctrl, 0xF, 0xF, true);
}
template <int L, class Op>
__device__ __forceinline__ int all_lanes(int v, Op op) {
  v = op(v, exchange16<0>(v));
  v = op(v, exchange16<1>(v));
  v = op(v, exchange16<2>(v));
  v = op(v, exchange16<3>(v));
  if constexpr (L == 64) {
    const int a = op(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16));
    const int b = op(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48));
    v = op(a, b);
  }
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  return (uint32_t)all_lanes<L>((int)v, [](int a, int b) { return (int)max((uint32_t)a, (uint32_t)b); });
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
  return __int_as_float(
      all_lanes<L>(__float_as_int(v), [](int a, int b) { return __float_as_int(fmaxf(__int_as_float(a), __int_as_float(b))); }));
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  return __int_as_float(
      all_lanes<L>(__float_as_int(v), [](int a, int b) { return __float_as_int(__int_as_float(a) + __int_as_float(b)); }));
}
// The bits of a ballot that belong to the caller's token, its first lane lowest.
template <int L>
__device__ __forceinline__ uint64_t token_bits(uint64_t ballot_bits, int lane) {
  return L == 64 ? ballot_bits : (ballot_bits >> (lane & ~(L - 1))) & ((1ull << (L & 63)) - 1);
}

// The wave's largest key, and of lanes that hold it the lowest index.
__device__ __forceinline__ void wave_best(int64_t& key, int& at) {
  const int hi = all_lanes<kWave>((int)(key >> 32), [](int a, int b) { return max(a, b); });
  const uint32_t low = (int)(key >> 32) == hi ? (uint32_t)key : 0u;
  const uint32_t lo = lanes_max<kWave>(low);
  const bool mine = (int)(key >> 32) == hi && (uint32_t)key == lo;
  at = all_lanes<kWave>(mine ? at : INT32_MAX, [](int a, int b) { return min(a, b); });
  key = (int64_t)(((uint64_t)(uint32_t)hi << 32) | lo);
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d, kWave);
  return v;
}
// The largest, a NaN above all.
__device__ __forceinline__ double wave_top(double v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const double o = __shfl_xor(v, d, kWave);
    v = o > v || o != o ? o : v;
  }
  return v;
}

__device__ __forceinline__ double sigmoid64(double l) {
  const double e = exp(-fabs(l));
  return (l < 0.0 ? e : 1.0) / (1.0 + e);
}

// One token by one wave, scores in float64.  s_bits: 8 E bytes of LDS, the
// lane's experts e = lane, lane + 64, ...: held there and not in registers,
// which the path that nearly every token takes would lack.  First a score's
// bits, then the key that orders as it does: one type, so that the compiler
// keeps the stores of one before those of the other.
__device__ __forceinline__ void route_exact(const RouteArgs& a, int64_t t, int lane, int64_t* s_bits) {
  const int E = a.E;
  const int64_t row = t * E;
  double top = -INFINITY, total = 0.0;
  if (!a.sigmoid) {
#pragma unroll 4
    for (int e = lane; e < E; e += kWave) {
      const double l = (double)logit_at(a.logits, a.bf16, row + e);
      top = l > top || l != l ? l : top;
    }
    top = wave_top(top);
  }
  // (a softmax's row of -infinity alone: scores 0)
  const bool none = !a.sigmoid && top == -INFINITY;
#pragma unroll 4
  for (int e = lane; e < E; e += kWave) {
    const double l = (double)logit_at(a.logits, a.bf16, row + e);
    const double x = a.sigmoid ? sigmoid64(l) : none ? 0.0 : exp(l - top);
    s_bits[e] = __double_as_longlong(x);
    total += x;
  }
  total = a.sigmoid || none ? 1.0 : wave_sum(total);
#pragma unroll 4
  for (int e = lane; e < E; e += kWave)
    s_bits[e] = __double_as_longlong(__longlong_as_double(s_bits[e]) / total + (a.bias ? (double)a.bias[e] : 0.0));
  uint64_t kept = ~0ull;
  const int per = E / a.groups;
  if (a.groups > 1) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    int64_t rank = kGone;
    if (lane < a.groups) {
      int64_t k1 = kGone, k2 = kGone;
      double v1 = 0.0, v2 = 0.0;
      for (int i = 0; i < per; ++i) {
        const double v = __longlong_as_double(s_bits[lane * per + i]);
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
    kept = 0;
    for (int i = 0; i < a.top_groups; ++i) {
      int64_t best = rank;
      int at = lane;
      wave_best(best, at);
      kept |= 1ull << at;
      if (lane == at) rank = kGone;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
#pragma unroll 4
  for (int e = lane; e < E; e += kWave)
    s_bits[e] = kept >> (a.groups > 1 ? e / per : 0) & 1
                    ? order_of(a.bias ? __longlong_as_double(s_bits[e]) : (double)logit_at(a.logits, a.bf16, row + e))
                    : kGone;
  int mine = 0;  // lane j: the expert of slot j
  for (int j = 0; j < a.k; ++j) {
    int64_t best = kGone;
    int at = INT32_MAX;
#pragma unroll 4
    for (int e = lane; e < E; e += kWave) {
      const int64_t k = s_bits[e];
      if (k > best) {
        best = k;
        at = e;
      }
    }
    wave_best(best, at);
    if (lane == (at & (kWave - 1))) s_bits[at] = kGone;
    if (lane == j) mine = at;
  }
  // ---- the weights
  const bool here = lane < a.k;
  const double logit = here ? (double)logit_at(a.logits, a.bf16, row + mine) : 0.0;
  double w;
  if (a.renorm) {
    // sigmoid: both the score and the sum times exp(-shift), shift the largest
    // chosen logit where that is negative
    double shift = wave_top(here ? logit : -INFINITY);
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

// ---- float32

// 31 bits that order as v does; zero is below all of them.  No NaN, no -0.
__device__ __forceinline__ uint32_t key_of(float v) {
  const int b = __float_as_int(v);
  return ((uint32_t)b ^ ((uint32_t)(b >> 31) | 0x80000000u)) >> 1;
}
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }

template <int L, int NV, bool BF16>
struct RouteShape {
  static constexpr int kTokens = kWave / L;             // of a wave
  static constexpr int kScores = L * NV + kMaxGroups;   // floats of LDS for a token: scores, a place between groups
  static constexpr int kFloats = kTokens * (kScores + kMaxGroups);
  static constexpr int kLds = kFloats * 4 > L * NV * 8 ? kFloats * 4 : L * NV * 8;  // (and the exact path's scores)
};

template <int L, int NV, bool BF16>
__global__ __launch_bounds__(kRouteWaves * kWave) void route_kernel(RouteArgs a, int first) {
  using S = RouteShape<L, NV, BF16>;
  __shared__ __attribute__((aligned(16))) uint8_t s_all[kRouteWaves][S::kLds];
  const int lane = lane_id(), wave = wave_in_group();
  const int sub = lane & (L - 1), token = lane / L;
  const int E = a.E;
  const bool scores = a.bias || a.groups > 1;  // compared by score; else by logit
  const bool vectors = E % (BF16 ? 8 : 4) == 0 && ((uintptr_t)a.logits & 15) == 0;
  const bool sums = !a.sigmoid && (scores || !a.renorm);  // the softmax's sum is needed
  float* const s_c = reinterpret_cast<float*>(s_all[wave]) + token * (S::kScores + kMaxGroups);
  float* const s_rank = s_c + S::kScores;

  const int64_t t0 = first + ((int64_t)blockIdx.x * kRouteWaves + wave) * S::kTokens;
  if (t0 >= a.T) return;
  const int64_t t = t0 + token;
  const bool held = t < a.T;
  const int64_t row = (held ? t : t0) * E;
  // ---- the lane's logits; an absent one counts as -infinity
  float l[NV];
  const int e0 = sub * NV;
  if (vectors) {
    constexpr int kPer = BF16 ? 8 : 4;
#pragma unroll
    for (int i = 0; i < NV; i += kPer) {
      u32x4 v = {0u, 0u, 0u, 0u};
      const bool in = e0 + i < E;
      if (NV < kPer) {
        // (four bf16 values a lane)
        uint2 h = make_uint2(0u, 0u);
        if (in) h = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.logits) + row + e0 + i);
        v[0] = h.x, v[1] = h.y;
      } else if (in) {
        v = *reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(a.logits) + (row + e0 + i) * (BF16 ? 2 : 4));
      }
#pragma unroll
      for (int q = 0; q < (NV < kPer ? NV : kPer); ++q) {
        const float x = BF16 ? (q & 1 ? bf16_hi(v[q / 2]) : bf16_lo(v[q / 2])) : __uint_as_float(v[q & 3]);
        l[i + q] = in ? x : -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] = e0 + i < E ? logit_at(a.logits, BF16, row + e0 + i) : -INFINITY;
  }
  // ---- scores and keys
  bool again = false;  // float32 does not decide this token
  float top = 0.0f, inv = 0.0f;
  if (sums) {
    top = l[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) top = fmaxf(top, l[i]);
    top = lanes_max<L>(top);
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) total += exp_fast(l[i] - top);  // (a NaN, +infinity, or nothing else than -infinity: NaN)
    total = lanes_sum<L>(total);
    again = total != total;
    inv = 1.0f / total;
  }
  // What the scores may be off by, twice.  Sigmoid, in half steps of 1: exp's
  // argument loses 1.22 |l|, exp itself 2, of which the sigmoid's slope leaves
  // 0.27 and 0.5, and the sum and the reciprocal add 3: 3.8, twice 2^-21.
  // Softmax: relative to scores of at most 1 / total, NV and a few half steps by
  // the sum's roundings and by what exp's arguments lose, 2.2 of their own size
  // (2^-22 covers the rest of it; rows of one large logit and many equal ones
  // come to two thirds of this bound).
  const float score_error = !scores ? 0.0f : a.sigmoid ? 0x1p-21f : inv * (NV + 10) * 0x1p-23f + 0x1p-22f;
  uint32_t key[NV];
  float probe = 0.0f;  // NaN if any is
  float c[NV];
  if (scores) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      c[i] = a.sigmoid ? __builtin_amdgcn_rcpf(1.0f + exp_fast(-l[i])) : exp_fast(l[i] - top) * inv;
    }
    if (a.bias) {
      if (E % 4 == 0 && ((uintptr_t)a.bias & 15) == 0) {
#pragma unroll
        for (int i = 0; i < NV; i += 4) {
          float4 b = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (e0 + i < E) b = *reinterpret_cast<const float4*>(a.bias + e0 + i);
          c[i] += b.x, c[i + 1] += b.y, c[i + 2] += b.z, c[i + 3] += b.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (e0 + i < E) c[i] += a.bias[e0 + i];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) c[i] = l[i] + 0.0f;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (e0 + i < E) probe += c[i];
    key[i] = e0 + i < E ? (key_of(c[i]) & ~(uint32_t)(NV - 1)) | (uint32_t)(NV - 1 - i) : 0u;
  }
  probe = lanes_sum<L>(probe);
  again |= probe != probe;
  // ---- the best groups
  if (a.groups > 1) {
    const int per = E / a.groups;
    const uint32_t over = ((1u << 20) + per - 1) / per;  // e / per = e * over >> 20 for e < 1024
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t e = e0 + i;
      if ((int)e < E) s_c[e + (e * over >> 20)] = c[i];  // (a place between the groups: other banks)
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    for (int g = sub; g < a.groups; g += L) {
      float v1 = -INFINITY, v2 = -INFINITY;
      float* p = s_c + g * (per + 1);
      for (int i = 0; i < per; ++i) {
        const float v = p[i];
        v2 = fmaxf(v2, fminf(v1, v));
        v1 = fmaxf(v1, v);
      }
      const bool two = a.group_best == 2;
      s_rank[g] = two ? v1 + v2 : v1;
      // What the rank may be off by, in the place of the group's first score,
      // which is not read again: the scores' errors (half of score_error each),
      // half a step for a bias added to each at its own size, which may be far
      // above the sum's, half a step for the sum and half a step for the sums
      // with this bound below (3 of 2^-24, 3.125 with what this line rounds).
      p[0] = two ? score_error + (fabsf(v1) + fabsf(v2)) * 0x1.9p-23f : 0.5f * score_error + fabsf(v1) * 0x1.1p-23f;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    uint64_t kept = 0;
    // The least that a kept group's rank can be, and the most that another's
    // can.  (Of a kept +infinity and of another's -infinity that is NaN, which
    // fminf and fmaxf pass over: nothing is above the one or below the other.)
    float worst = INFINITY, next = -INFINITY;
    for (int g0 = 0; g0 < a.groups; g0 += L) {
      const int g = g0 + sub;
      const float mine = g < a.groups ? s_rank[g] : -INFINITY;
      int before = g < a.groups ? 0 : kMaxGroups;
      for (int o = 0; o < a.groups; ++o) {
        const float r = s_rank[o];
        before += r > mine || (r == mine && o < g);
      }
      const bool keep = before < a.top_groups;
      const float off = g < a.groups ? s_c[g * (per + 1)] : 0.0f;
      if (keep) worst = fminf(worst, mine - off);
      else next = fmaxf(next, mine + off);
      kept |= token_bits<L>(ballot(keep), lane) << g0;
    }
    worst = -lanes_max<L>(-worst);
    next = lanes_max<L>(next);
    again |= a.top_groups < a.groups && !(worst > next);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t e = e0 + i;
      if (!(kept >> (e * over >> 20 & 63) & 1)) key[i] = 0u;
    }
  }
  // ---- the choice: slot j in lane j, and the best that is left in lane k
  uint32_t last = 1u << 31;
  int32_t* const s_slot = reinterpret_cast<int32_t*>(s_rank);
  auto choose = [&](int j0, int j1) {
    for (int j = j0; j < j1; ++j) {
      uint32_t most = key[0] - last;
#pragma unroll
      for (int i = 1; i < NV; ++i) most = max(most, key[i] - last);
      const uint32_t best = most >> 31 ? most + last : 0u;  // (none left: zero)
      const uint32_t value = best & ~(uint32_t)(NV - 1), all = lanes_max<L>(value);
      const uint64_t who = token_bits<L>(ballot(value == all), lane);
      if (sub == (L == 64 ? __builtin_ctzll(who) : __builtin_ctz((uint32_t)who))) {
        last = best;
        s_slot[j] = all != 0u ? e0 + (NV - 1) - (int)(best & (NV - 1)) : -1;
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  };
  int mine = -1;
  float lj = -INFINITY, bj = 0.0f;
  // The lane's slot of `slots`; bit j: slot j is certainly before slot j + 1,
  // and, from the choice's last slot on, before all that follow.  (Equal ones
  // are in their order, but what follows them may lie in their cell above them.)
  auto certain = [&](int slots) -> uint64_t {
    mine = sub < slots ? s_slot[sub] : -1;
    lj = mine >= 0 ? logit_at(a.logits, BF16, row + mine) : -INFINITY;
    bj = mine >= 0 && a.bias ? a.bias[mine] : 0.0f;
    float cj = lj;
    if (scores) {
      cj = a.sigmoid ? __builtin_amdgcn_rcpf(1.0f + exp_fast(-lj)) : exp_fast(lj - top) * inv;
      cj += bj;
    }
    const int up = sub + 1 < L ? lane + 1 : lane;
    const float cn = __shfl(cj, up, kWave), ln = __shfl(lj, up, kWave), bn = __shfl(bj, up, kWave);
    const int en = __shfl(mine, up, kWave);
    // a key's cell is 2 NV steps of float32 (below its least normal number of
    // 2^-149 each), the sums' roundings two
    const float margin = fmaxf(fmaxf(fabsf(cj), fabsf(cn)), 0x1p-126f) * (2.0f * NV + 2.0f) * 0x1p-23f + score_error;
    const bool clear = en < 0 || (sub < a.k - 1 && lj == ln && bj == bn) || (cn == -INFINITY && cj > cn) || cj - cn > margin;
    return token_bits<L>(ballot(clear), lane);
  };
  choose(0, a.k + 1);
  const uint64_t inside = (1ull << a.k) - 1;
  uint64_t sure = certain(a.k + 1);
  int place = sub;  // of the lane's slot in the choice
  // (the keys hold a bf16 logit whole: their order is the choice)
  if (BF16 && !scores) sure = inside;
  again |= (scores && !a.sigmoid) && (sure & inside) != inside;
  if (ballot((sure & inside) != inside && !again)) {
    // A few more, up to a certain gap: what lies before it holds the choice, and is ranked in float64.
    const int slots = min(L, a.k + 1 + 4);
    choose(a.k + 1, slots);
    sure = certain(slots) >> (a.k - 1);
    const int before = a.k + (sure ? __builtin_ctzll(sure) : L);
    again |= before >= slots;
    // (Without a bias by the logits: from about 24 on the sigmoids of neighbouring ones are equal in float64.)
    const double x = a.bias ? sigmoid64((double)lj) + (double)bj : (double)lj;
    const bool in = sub < before;
    place = in ? 0 : L;
    for (int i = 0; i < slots; ++i) {
      const double o = __shfl(x, (lane & ~(L - 1)) + i, kWave);
      const int e = __shfl(mine, (lane & ~(L - 1)) + i, kWave);
      if (in && i < before) place += o > x || (o == x && e < mine);
    }
  }
  // ---- its weights
  const bool here = place < a.k;
  const float most = lanes_max<L>(here ? lj : -INFINITY);
  again |= !(fabsf(most) < INFINITY);
  float sj;
  if (a.renorm) {
    if (a.sigmoid) {
      const float shift = fminf(most, 0.0f);
      sj = lj > 0.0f ? expf(-shift) / (1.0f + expf(-lj)) : expf(lj - shift) / (1.0f + expf(lj));
    } else {
      sj = expf(lj - most);
    }
    if (!here) sj = 0.0f;
    sj /= lanes_sum<L>(sj);
  } else if (a.sigmoid) {
    const float x = expf(-fabsf(lj));
    sj = (lj < 0.0f ? x : 1.0f) / (1.0f + x);
  } else {
    sj = expf(lj - top) * inv;
  }
  if (held && here && !again) {
    a.idx[t * a.k + place] = mine;
    a.w[t * a.k + place] = sj * a.scale;
  }
  // ---- the tokens that are left
  uint64_t left = ballot(held && sub == 0 && again);
  while (left) {
    const int at = __builtin_ctzll(left);
    left &= left - 1;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    route_exact(a, t0 + at / L, lane, reinterpret_cast<int64_t*>(s_all[wave]));
  }
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

__device__ __forceinline__ void route_back(const RouteBackwardArgs& a, int64_t t, int lane) {
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
  // (1 - s in a form that keeps its digits where s is nearly 1)
  if (a.sigmoid) g *= 1.0f / (1.0f + expf(l));
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

__global__ __launch_bounds__(kRouteWaves * kWave) void route_backward_kernel(RouteBackwardArgs a) {
  const int64_t step = (int64_t)gridDim.x * kRouteWaves;
  for (int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave_in_group(); t < a.T; t += step) route_back(a, t, lane_id());
}

}  // namespace

namespace {

template <int L, int NV>
hipError_t launch_shape(const RouteArgs& a, hipStream_t stream) {
  constexpr int kEach = kRouteWaves * (kWave / L);  // tokens of a workgroup
  for (int64_t first = 0; first < a.T; first += kRouteGroups * kEach) {
    const int64_t groups = (a.T - first + kEach - 1) / kEach;
    const dim3 grid((uint32_t)(groups < kRouteGroups ? groups : kRouteGroups)), block(kRouteWaves * kWave);
    if (a.bf16) hipLaunchKernelGGL((route_kernel<L, NV, true>), grid, block, 0, stream, a, (int)first);
    else hipLaunchKernelGGL((route_kernel<L, NV, false>), grid, block, 0, stream, a, (int)first);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_route(const Budget& b, const RouteArgs& a, hipStream_t stream) {
  const RouteLanes r = route_lanes(a.T, a.E, a.k, b.device_cus);
  if (r.lanes == 16) {
    switch (r.each) {
      case 4: return launch_shape<16, 4>(a, stream);
      case 8: return launch_shape<16, 8>(a, stream);
      case 16: return launch_shape<16, 16>(a, stream);
      default: return launch_shape<16, 32>(a, stream);
    }
  }
  switch (r.each) {
    case 4: return launch_shape<64, 4>(a, stream);
    case 8: return launch_shape<64, 8>(a, stream);
    default: return launch_shape<64, 16>(a, stream);
  }
}

hipError_t launch_route_backward(const Budget&, const RouteBackwardArgs& a, hipStream_t stream) {
  const int64_t groups = ((int64_t)a.T + kRouteWaves - 1) / kRouteWaves;
  hipLaunchKernelGGL(route_backward_kernel, dim3((uint32_t)(groups < kRouteGroups ? groups : kRouteGroups)),
                     dim3(kRouteWaves * kWave), 0, stream, a);
  return hipGetLastError();
}

}  // namespace ep
