// Router scores to the top-k experts of each token and their weights.
//
//   s   = softmax(l) or sigmoid(l)
//   key = l without a bias and groups (both scores rise with l, so the order
//         is the logits' own, with no rounding), else s + bias in 64 bits
//         (scores next to each other are told apart as their logits are)
//   groups: each of n_group groups scores the sum of its two largest keys;
//         the topk_group best groups (ties: the lower) keep their experts
//   ids = the k largest keys in descending order (ties: the lower id)
//   weights = s[ids] (divided by their sum: renorm) * scale
//
// One wave per token: lane i holds the experts i, i + 64, ...; each of the k
// rounds takes the wave's largest (key, lowest id).  Bound by latency (one
// round of loads, k wave reductions) until some thousands of tokens.
#include "bsfp8_internal.h"

namespace bsfp8 {
namespace detail {

typedef unsigned long long u64;

constexpr int kRouteWaves = 4;
constexpr u64 kNever = 0;            // the key of an expert that is never chosen

// order-preserving maps to unsigned; every number maps above 0 (kNever)
__device__ __forceinline__ uint32_t ordered32(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);           // -0 and +0 are equal
  return (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ u64 ordered64(double d) {
  const u64 u = (u64)__double_as_longlong(d + 0.0);
  return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}
__device__ __forceinline__ double unordered64(u64 k) {
  return __longlong_as_double((long long)((k >> 63) ? k & 0x7fffffffffffffffull : ~k));
}

__device__ __forceinline__ u64 wave_max(u64 v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const u64 t = __shfl_xor(v, o, 64);
    v = t > v ? t : v;
  }
  return v;
}

template <bool BF16, bool K64, int NE>
__global__ __launch_bounds__(64 * kRouteWaves) void route_topk_kernel(RouteArgs a) {
  extern __shared__ u64 gkeys[];       // K64 with groups: E keys per wave
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
  if (t >= a.T) return;                // whole waves; no workgroup barrier below
  const int E = a.E;
  const float ninf = -__builtin_inff();
  float l[NE];
  float top = ninf;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = lane + 64 * i;
    l[i] = ninf;
    if (e < E) {
      const int64_t at = t * a.ldl + e;
      const float v = BF16 ? __uint_as_float((uint32_t)((const uint16_t*)a.logits)[at] << 16)
                           : ((const float*)a.logits)[at];
      if (v > ninf) l[i] = v;          // NaN and -inf: never chosen
    }
    top = fmaxf(top, l[i]);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));

  // softmax denominators: needed for the scores as such, not where the
  // chosen ones are divided by their own sum
  double Z = 1.0;
  const bool soft = a.score == 0;
  auto expo = [&](float v) -> double {   // e^(v - top); 1 at the top, +inf included
    return v == top ? 1.0 : exp((double)v - (double)top);
  };
  // in 64 bits: scores that fp32 cannot hold still have a ratio
  auto score = [&](float v) -> double { return soft ? expo(v) / Z : 1.0 / (1.0 + exp(-(double)v)); };
  if (soft && (K64 || !a.renorm)) {
    Z = 0.0;
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (l[i] > ninf) Z += K64 ? expo(l[i]) : l[i] == top ? 1.0 : (double)expf(l[i] - top);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) Z += __shfl_xor(Z, o, 64);
  }

  u64 key[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    key[i] = kNever;
    const int e = lane + 64 * i;
    if (l[i] > ninf) {
      if constexpr (K64) {
        const double v = score(l[i]) + (a.bias ? (double)a.bias[e] : 0.0);
        if (v > -(double)__builtin_inff()) key[i] = ordered64(v);
      } else {
        key[i] = ((u64)ordered32(l[i]) << 32) | (uint32_t)~e;
      }
    }
  }
  if constexpr (K64) {
    if (a.n_group > 1) {
      u64* gk = gkeys + (int64_t)wave * E;
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (lane + 64 * i < E) gk[lane + 64 * i] = key[i];
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      const int gs = E / a.n_group;
      u64 gscore = kNever;
      if (lane < a.n_group) {
        u64 b0 = kNever, b1 = kNever;   // the group's two largest keys
        for (int j = 0; j < gs; ++j) {
          const u64 v = gk[lane * gs + j];
          if (v > b0) { b1 = b0; b0 = v; } else if (v > b1) { b1 = v; }
        }
        if (b0 != kNever)
          gscore = ordered64(unordered64(b0) + (b1 != kNever ? unordered64(b1) : 0.0));
      }
      int better = 0;
      for (int g = 0; g < a.n_group; ++g) {
        const u64 v = __shfl(gscore, g, 64);
        better += (v > gscore || (v == gscore && g < lane)) ? 1 : 0;
      }
      const u64 kept = __ballot(lane < a.n_group && better < a.topk_group);
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int e = lane + 64 * i;
        if (e < E && !((kept >> (e / gs)) & 1)) key[i] = kNever;
      }
    }
  }

  // k rounds; lane j keeps the j-th choice
  int mine = -1;
  for (int j = 0; j < a.k; ++j) {
    u64 best = kNever;
    int at = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (key[i] > best) { best = key[i]; at = lane + 64 * i; }
    const u64 all = wave_max(best);
    if (all == kNever) break;
    int e;
    if constexpr (K64) {
      e = best == all ? at : 0x7fffffff;
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) e = min(e, __shfl_xor(e, o, 64));
    } else {
      e = (int)~(uint32_t)all;
    }
    if (lane == j) mine = e;
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (lane + 64 * i == e) key[i] = kNever;
  }
  // the chosen experts' logits, from their lanes
  float lv = ninf;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const float v = __shfl(l[i], mine & 63, 64);
    if (mine >= 0 && (mine >> 6) == i) lv = v;
  }
  double w = mine >= 0 ? score(lv) : 0.0;
  if (a.renorm) {
    double sum = w;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
    w = sum > 0.0 ? w / sum : 0.0;
  }
  if (lane < a.k) {
    a.ids[t * a.k + lane] = mine;
    a.weights[t * a.k + lane] = (float)(w * (double)a.scale);
  }
}

template <bool BF16, bool K64>
hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.T + kRouteWaves - 1) / kRouteWaves)), block(64 * kRouteWaves);
  const size_t lds = K64 && a.n_group > 1 ? (size_t)kRouteWaves * a.E * 8 : 0;
#define BSFP8_ROUTE(NE)                                                                       \
  hipLaunchKernelGGL((route_topk_kernel<BF16, K64, NE>), grid, block, lds, s, a)
  if (a.E <= 64) BSFP8_ROUTE(1);
  else if (a.E <= 128) BSFP8_ROUTE(2);
  else if (a.E <= 256) BSFP8_ROUTE(4);
  else if (a.E <= 512) BSFP8_ROUTE(8);
  else BSFP8_ROUTE(16);
#undef BSFP8_ROUTE
  return hipGetLastError();
}

}  // namespace detail
using namespace detail;

hipError_t launch_route_topk(const RouteArgs& a, hipStream_t s) {
  const bool k64 = a.bias || a.n_group > 1;
  if (a.bf16) return k64 ? launch_route<true, true>(a, s) : launch_route<true, false>(a, s);
  return k64 ? launch_route<false, true>(a, s) : launch_route<false, false>(a, s);
}

}  // namespace bsfp8
