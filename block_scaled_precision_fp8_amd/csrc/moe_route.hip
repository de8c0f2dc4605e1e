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
// rounds takes the wave's largest (key, lowest id).  Bound by latency for a
// token (one round of loads, k wave reductions), by vector issue for a prompt:
// with 256 experts in 8 groups, sigmoid, top 8, a token takes 958 vector
// instructions, and the four waves that 4096 tokens give each SIMD issue for
// 15.3 thousand of the 18.3 thousand cycles that a wave lives.
// Measured: those 256 experts, 1 token 5.1 us, 4096 tokens 10.8; 60 experts, top
// 4, 333 tokens 3.3.
#include "bsfp8_layer.h"

namespace bsfp8 {
namespace detail {

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

// Wave maxima, as wave_sum.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, dpp<kXor1>(v));
  v = max(v, dpp<kXor2>(v));
  v = max(v, dpp<kMirror8>(v));
  v = max(v, dpp<kMirror16>(v));
  return max(max(lane_u32(v, 0), lane_u32(v, 16)), max(lane_u32(v, 32), lane_u32(v, 48)));
}
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, __uint_as_float(dpp<kXor1>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp<kXor2>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp<kMirror8>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp<kMirror16>(__float_as_uint(v))));
  const uint32_t u = __float_as_uint(v);
  return fmaxf(fmaxf(__uint_as_float(lane_u32(u, 0)), __uint_as_float(lane_u32(u, 16))),
               fmaxf(__uint_as_float(lane_u32(u, 32)), __uint_as_float(lane_u32(u, 48))));
}
// The two largest of two such pairs.
__device__ __forceinline__ void merge2(u64& a0, u64& a1, u64 b0, u64 b1) {
  const u64 lo = a0 < b0 ? a0 : b0, hi = a0 < b0 ? b0 : a0;
  const u64 m = a1 < b1 ? b1 : a1;
  a0 = hi;
  a1 = lo < m ? m : lo;
}

// SOFT: softmax scores, else sigmoid.  Keys are held as two words; with K64
// false the low one is not there.
template <bool BF16, bool SOFT, bool K64, int NE>
__global__ __launch_bounds__(64 * kRouteWaves) void route_topk_kernel(RouteArgs a) {
  extern __shared__ u64 gkeys[];       // with groups: E keys per wave
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = grid_row() * kRouteWaves + wave;
  if (t >= a.T) return;                // whole waves; no workgroup barrier below
  const int E = a.E;
  const float ninf = -__builtin_inff();
  float l[NE], bias[NE];
  float top = ninf;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = min(lane + 64 * i, E - 1);
    const int64_t at = t * a.ldl + e;
    const float v = BF16 ? __uint_as_float((uint32_t)((const uint16_t*)a.logits)[at] << 16)
                         : ((const float*)a.logits)[at];
    if (K64) bias[i] = a.bias ? a.bias[e] : 0.0f;
    l[i] = lane + 64 * i < E && v > ninf ? v : ninf;       // NaN and -inf: never chosen
    top = fmaxf(top, l[i]);
  }
  if (SOFT) top = wave_max(top);

  // Scores in 64 bits: those that fp32 cannot hold still have a ratio.  At
  // the top 1, +inf included; -inf gives 0
  auto expo = [&](float v) -> double { return v == top ? 1.0 : exp((double)v - (double)top); };
  // Softmax denominators: needed for the scores as such, not where the
  // chosen ones are divided by their own sum.  Where they do not enter the
  // keys their terms e^d, d = v - top, are fp32 values (d rounded: |d| 2^-24 of
  // the term, the exponential 2^-22), summed in 64 bits: off by the terms'
  // average |d| + 4, times 2^-24, of the weight, which is rounded to fp32
  // itself.  64-bit exponentials of all experts are left to keys that need them
  double Z = 1.0;
  if (SOFT && (K64 || !a.renorm)) {
    Z = 0.0;
#pragma unroll
    for (int i = 0; i < NE; ++i)
      Z += l[i] == ninf ? 0.0 : K64 ? expo(l[i]) : l[i] == top ? 1.0 : (double)expf(l[i] - top);
    Z = wave_sum(Z);
  }
  auto score = [&](float v) -> double { return SOFT ? expo(v) / Z : 1.0 / (1.0 + exp(-(double)v)); };

  uint32_t hi[NE], lo[K64 ? NE : 1];   // 0, 0: never chosen
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    if constexpr (K64) {
      const double v = score(l[i]) + (double)bias[i];
      const u64 k = l[i] > ninf && v > -(double)__builtin_inff() ? ordered64(v) : kNever;
      hi[i] = (uint32_t)(k >> 32);
      lo[i] = (uint32_t)k;
    } else {
      hi[i] = l[i] > ninf ? ordered32(l[i]) : 0u;
    }
  }
  if constexpr (K64) {
    if (a.n_group > 1) {
      u64* gk = gkeys + (int64_t)wave * E;
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (lane + 64 * i < E) gk[lane + 64 * i] = (u64)hi[i] << 32 | lo[i];
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      // L lanes (a power of two) scan each group, lanes g L .. + L - 1 group g
      const int gs = E / a.n_group, L = a.group_lanes;
      const int g = lane / L;
      u64 b0 = kNever, b1 = kNever;    // the group's two largest keys
      if (g < a.n_group)
        for (int j = lane & (L - 1); j < gs; j += L) merge2(b0, b1, gk[g * gs + j], kNever);
      if (L > 1) merge2(b0, b1, dpp64<kXor1>(b0), dpp64<kXor1>(b1));
      if (L > 2) merge2(b0, b1, dpp64<kXor2>(b0), dpp64<kXor2>(b1));
      if (L > 4) merge2(b0, b1, dpp64<kMirror8>(b0), dpp64<kMirror8>(b1));
      if (L > 8) merge2(b0, b1, dpp64<kMirror16>(b0), dpp64<kMirror16>(b1));
      if (L > 16) merge2(b0, b1, __shfl_xor(b0, 16, 64), __shfl_xor(b1, 16, 64));
      u64 gscore = kNever;
      if (b0 != kNever)
        gscore = ordered64(unordered64(b0) + (b1 != kNever ? unordered64(b1) : 0.0));
      int better = 0;
      for (int o = 0; o < a.n_group; ++o) {
        const u64 v = (u64)lane_u32((uint32_t)(gscore >> 32), o * L) << 32 | lane_u32((uint32_t)gscore, o * L);
        better += (v > gscore || (v == gscore && o < g)) ? 1 : 0;
      }
      const u64 kept = __ballot(g < a.n_group && better < a.topk_group);
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        // e / gs by its reciprocal: exact below e gs = 2^20
        const uint32_t e = lane + 64 * i;
        const bool in = kept >> ((e * a.group_rcp >> 20) * L & 63) & 1;
        hi[i] = in ? hi[i] : 0u;
        lo[i] = in ? lo[i] : 0u;
      }
    }
  }

  // k rounds; lane j keeps the j-th choice
  int mine = -1;
  for (int j = 0; j < a.k; ++j) {
    uint32_t best = hi[0];
#pragma unroll
    for (int i = 1; i < NE; ++i) best = max(best, hi[i]);
    best = wave_max(best);
    if (best == 0) break;
    // the experts with that high word; of several (rare) those with the
    // largest low word; of these the lowest
    u64 has[NE];
    int n = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      has[i] = __ballot(hi[i] == best);
      n += __popcll(has[i]);
    }
    if constexpr (K64) {
      if (n > 1) {
        uint32_t low = 0;
#pragma unroll
        for (int i = 0; i < NE; ++i) low = max(low, hi[i] == best ? lo[i] : 0u);
        low = wave_max(low);
#pragma unroll
        for (int i = 0; i < NE; ++i) has[i] = __ballot(hi[i] == best && lo[i] == low);
      }
    }
    int e = 0;
#pragma unroll
    for (int i = NE - 1; i >= 0; --i)
      if (has[i]) e = 64 * i + __builtin_ctzll(has[i]);
    if (lane == j) mine = e;
#pragma unroll
    for (int i = 0; i < NE; ++i) hi[i] = lane + 64 * i == e ? 0u : hi[i];
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
    const double sum = wave_sum(w);
    w = sum > 0.0 ? w / sum : 0.0;
  }
  if (lane < a.k) {
    a.ids[t * a.k + lane] = mine;
    a.weights[t * a.k + lane] = (float)(w * (double)a.scale);
  }
}

template <bool BF16, bool SOFT, bool K64>
hipError_t launch_route(RouteArgs a, hipStream_t s) {
  a.group_lanes = 1;
  while (a.group_lanes * 2 * a.n_group <= 64) a.group_lanes *= 2;
  a.group_rcp = ((1u << 20) + a.E / a.n_group - 1) / (a.E / a.n_group);
  const dim3 grid = row_grid((a.T + kRouteWaves - 1) / kRouteWaves), block(64 * kRouteWaves);
  const size_t lds = K64 && a.n_group > 1 ? (size_t)kRouteWaves * a.E * 8 : 0;
#define BSFP8_ROUTE(NE)                                                                       \
  hipLaunchKernelGGL((route_topk_kernel<BF16, SOFT, K64, NE>), grid, block, lds, s, a)
  if (a.E <= 64) BSFP8_ROUTE(1);
  else if (a.E <= 128) BSFP8_ROUTE(2);
  else if (a.E <= 256) BSFP8_ROUTE(4);
  else if (a.E <= 512) BSFP8_ROUTE(8);
  else BSFP8_ROUTE(16);
#undef BSFP8_ROUTE
  return hipGetLastError();
}

template <bool BF16, bool SOFT>
hipError_t launch_route_key(const RouteArgs& a, hipStream_t s) {
  if (a.bias || a.n_group > 1) return launch_route<BF16, SOFT, true>(a, s);
  return launch_route<BF16, SOFT, false>(a, s);
}

}  // namespace detail
using namespace detail;

hipError_t launch_route_topk(const RouteArgs& a, hipStream_t s) {
  if (a.bf16) return a.score == 0 ? launch_route_key<true, true>(a, s) : launch_route_key<true, false>(a, s);
  return a.score == 0 ? launch_route_key<false, true>(a, s) : launch_route_key<false, false>(a, s);
}

}  // namespace bsfp8
