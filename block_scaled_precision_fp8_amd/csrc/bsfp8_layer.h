// Declarations shared by the operators around the linears (norm, router, MoE
// layer for few tokens) and the activation quantizer: eight-value encoders,
// wave reductions, launchers.  Apart from bsfp8_internal.h, which the GEMM
// sources' recorded measurements are tied to.
#pragma once

#include "bsfp8_internal.h"

namespace bsfp8 {

// ---------------------------------------------------------------- device

__device__ __forceinline__ int64_t grid_row() {
  return (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
}

namespace detail {

struct Unpacked { float f[8]; };

__device__ __forceinline__ Unpacked unpack8(uint4 v) {
  Unpacked u;
  u.f[0] = bf16_lo(v.x); u.f[1] = bf16_hi(v.x);
  u.f[2] = bf16_lo(v.y); u.f[3] = bf16_hi(v.y);
  u.f[4] = bf16_lo(v.z); u.f[5] = bf16_hi(v.z);
  u.f[6] = bf16_lo(v.w); u.f[7] = bf16_hi(v.w);
  return u;
}

__device__ __forceinline__ float amax8(const Unpacked& u) {
  float a = fabsf(u.f[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) a = fmaxf(a, fabsf(u.f[i]));
  return a;
}

// Encode eight values of one group with the group's scale.  Returns the
// codes packed little-endian; writes the stored scale representation.
// fp32 scales divide by the correctly rounded reciprocal with one exact
// correction (div_by_rcp: the same E4M3 codes as IEEE x / s for a normal s,
// at four operations per value instead of an IEEE division each); a
// subnormal scale divides directly.
template <int FMT>
__device__ __forceinline__ uint2 encode8(const Unpacked& u, float amax, float* s_f32, int* s_exp) {
  const float s = FMT == 0 ? act_scale_f32(amax) : 0.0f;
  const int e = FMT == 0 ? 0 : ue8m0_exp(amax);
  *s_f32 = s;
  *s_exp = e;
  uint2 r;
  if (FMT == 0 && s >= kMinNormal) {
    const RcpDiv dv = rcp_div(s);
    r.x = act_encode4_rcp<FMT>(u.f[0], u.f[1], u.f[2], u.f[3], dv, e);
    r.y = act_encode4_rcp<FMT>(u.f[4], u.f[5], u.f[6], u.f[7], dv, e);
  } else {
    r.x = act_encode4<FMT>(u.f[0], u.f[1], u.f[2], u.f[3], s, e);
    r.y = act_encode4<FMT>(u.f[4], u.f[5], u.f[6], u.f[7], s, e);
  }
  return r;
}

__device__ __forceinline__ float e8m0_f32(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b << 23);   // 2^(b - 127)
}

typedef unsigned long long u64;

// Exchanges between the lanes of a wave on the vector ALU: inside rows of 16
// lanes (lane ^ 1, lane ^ 2, mirrored in eight and in sixteen), then the four
// rows' results one by one.  An exchange through LDS takes ten times as long
// and was a third of a short row's time.
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140;
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xf, 0xf, false);
}
template <int CTRL>
__device__ __forceinline__ u64 dpp64(u64 v) {
  return (u64)dpp<CTRL>((uint32_t)(v >> 32)) << 32 | dpp<CTRL>((uint32_t)v);
}
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  return __longlong_as_double((long long)dpp64<CTRL>((u64)__double_as_longlong(v)));
}
__device__ __forceinline__ uint32_t lane_u32(uint32_t v, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}
__device__ __forceinline__ double lane_f64(double v, int lane) {
  const u64 u = (u64)__double_as_longlong(v);
  return __longlong_as_double((long long)((u64)lane_u32((uint32_t)(u >> 32), lane) << 32 |
                                          lane_u32((uint32_t)u, lane)));
}
__device__ __forceinline__ double row16_sum(double v) {
  v += dpp_f64<kXor1>(v);
  v += dpp_f64<kXor2>(v);
  v += dpp_f64<kMirror8>(v);
  v += dpp_f64<kMirror16>(v);
  return v;
}
// The sum over the wave, in every lane.
__device__ __forceinline__ double wave_sum(double v) {
  v = row16_sum(v);
  return (lane_f64(v, 0) + lane_f64(v, 16)) + (lane_f64(v, 32) + lane_f64(v, 48));
}

}  // namespace detail

// ---------------------------------------------------------------- host

// A grid of n workgroups that may exceed what one dimension's lanes can count
// (2^32): rows of 2^20 workgroups; a kernel's number is grid_row().
inline dim3 row_grid(int64_t n) {
  const int64_t x = n < (1 << 20) ? n : 1 << 20;
  return dim3((unsigned)x, (unsigned)((n + x - 1) / x));
}

struct NormArgs {
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* res;       // null: h = x
  uint16_t* res_out;         // row stride ldr, like res
  int64_t ldr;
  const uint16_t* w;         // [K]
  uint16_t* y;               // bf16 [M][K] or null
  uint8_t* xq;               // [M][K], or null: no quantized output
  void* xs;
  const void* xstat;         // the static scheme's scale, or null
  float eps;
  double inv_k;              // 1 / K
  int64_t M, K;
  int fmt, group_k;
};

struct RouteArgs {
  const void* logits;        // [T][ldl] fp32 or bf16
  int64_t ldl;
  bool bf16;
  const float* bias;         // [E] or null
  int64_t T;
  int E, k, score, renorm;
  float scale;
  int n_group, topk_group;
  int group_lanes;           // set by the launcher: lanes that scan a group,
  uint32_t group_rcp;        // 2^20 / (experts of a group), rounded up
  int32_t* ids;              // [T][k]
  float* weights;            // [T][k]
};

constexpr int kMoeMaxTokens = 128;   // tokens of one moe_decode call
constexpr int kMoeMaxChoices = 16;   // experts per token
constexpr int64_t kMoeMaxRowBytes = int64_t(1) << 30;   // codes of h (T k I)
struct MoeArgs {
  const uint8_t* xq;         // [T][H] and its scales
  const void* xs;
  const int32_t* ids;        // [T][k]
  const float* wt;           // [T][k]
  const uint8_t* w13;        // [E][2I][H] codes (w4: [E][2I][H/2])
  const void* s13;
  const uint8_t* w2;         // [E][H][I] codes (w4: [E][H][I/2])
  const void* s2;
  const uint16_t* addend;    // bf16 [T][H] or null
  uint16_t* y;               // bf16 [T][H]
  int T, k, E;
  int64_t H, I;
  int fmt;
  bool w4;
  void* workspace;
};

hipError_t launch_add_rmsnorm_quant(const NormArgs& a, hipStream_t s);
hipError_t launch_route_topk(const RouteArgs& a, hipStream_t s);
hipError_t launch_moe_decode(const MoeArgs& a, hipStream_t s);
size_t moe_decode_workspace_bytes(int64_t slots, int64_t I);

}  // namespace bsfp8
