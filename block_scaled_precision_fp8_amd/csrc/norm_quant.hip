// Residual addition, RMS norm and FP8 quantization in one pass.
//
//   h  = bf16(x + residual)                 (h = x without a residual)
//   rs = 1 / sqrt(sum_k h^2 / K + eps)
//   y  = fl32(h w rs)
//   codes, scales = the activation codec of fp8_quant_act on the fp32 y
//
// Bound by HBM: per element 2 bytes of x, 2 of the residual and 2 of h, 1
// byte of codes (and 2 of the optional bf16 y).  Measured, launches in the
// profiler: 8192 x 4096 46 to 49 us (235 MB, 4.8 to 5.1 TB/s; a large copy runs
// at 5.1), 1031 x 5136 without a residual 11.8 (16 MB), 64 x 4096 4.4, 1 x 7168
// 4.7.  Rows of two chunks a lane (520 to 1024 values, 8200 to 16384) load the
// second one after the first, and rows of 4104 to 8192 values leave up to half
// of 1024 lanes idle: 8192 x 1024 16.4 us where its 59 MB copy in 11.6, 1031 x
// 5136 with its residual 14.2 (37 MB: 7.3).
//
// The sum of squares is held in 64 bits (a square of a bf16 value is exact
// there, and the vector ALU has the time: one conversion and one FMA per
// element under the loads): it errs by at most K 2^-53 of itself, rs by half
// of that.  h w is exact in fp32 (8 + 8 significant bits; products below
// 2^-126 aside), rs is a sum of two fp32 values (2^-48 of it lost) and its
// small part's product is rounded before the sum (as much again): y is h w rs
// rounded once, to within 1/2 + (K + 140) 2^-30 units in the last place, where
// no small part runs out of exponents (root mean squares below 2^100, y above
// 2^-100).  Only values that near a border between two fp32 numbers can depend
// on how a row is dealt to lanes.  y is not rounded to bf16 before it is
// quantized: the codes then carry one rounding, and a group's scale does not
// jump by a bf16 step.
#include "bsfp8_layer.h"

namespace bsfp8 {
namespace detail {

enum { kNormPlain = 0, kNormG128 = 1, kNormG32 = 2, kNormStatic = 3 };

__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  return f32_to_bf16(bf16_lo(a) + bf16_lo(b)) | (f32_to_bf16(bf16_hi(a) + bf16_hi(b)) << 16);
}
__device__ __forceinline__ uint4 add_bf16x8(uint4 a, uint4 b) {
  return make_uint4(add_bf16x2(a.x, b.x), add_bf16x2(a.y, b.y), add_bf16x2(a.z, b.z),
                    add_bf16x2(a.w, b.w));
}

__device__ __forceinline__ double square_sum8(uint4 v, double s) {
  const Unpacked u = unpack8(v);
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fma((double)u.f[i], (double)u.f[i], s);
  return s;
}

struct RowScale { float hi, lo; };   // rs = hi + lo

// Streaming stores, like the loads: 8192 x 4096 rows 59 us without the hint
// on either store, 49 with it on the codes, 47 on both.
__device__ __forceinline__ void st_stream16(void* p, uint4 v) {
  __builtin_nontemporal_store(u32x4{v.x, v.y, v.z, v.w}, (u32x4*)p);
}
__device__ __forceinline__ void st_stream8(void* p, uint2 v) {
  __builtin_nontemporal_store((uint64_t)v.x | (uint64_t)v.y << 32, (uint64_t*)p);
}

// Eight values of a row: y, its codes and scale, the stores.  Called by all
// lanes of the group together (lanes past the row pass valid = false).
template <int FMT, int MODE>
__device__ __forceinline__ void norm_out8(uint4 hv, uint4 wv, RowScale rs, bool valid, int c,
                                          const void* xstat, uint16_t* y, uint8_t* xq, void* xs,
                                          int64_t m, int64_t K) {
  const Unpacked h = unpack8(hv), w = unpack8(wv);
  Unpacked v;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float p = h.f[i] * w.f[i];
    // the sign is p's: two zeros of unlike signs would add to +0
    v.f[i] = valid ? copysignf(fmaf(p, rs.hi, p * rs.lo), p) : 0.0f;
  }
  const int64_t k0 = (int64_t)c * 8;
  if (y && valid) {
    uint4 o;
    o.x = f32_to_bf16(v.f[0]) | (f32_to_bf16(v.f[1]) << 16);
    o.y = f32_to_bf16(v.f[2]) | (f32_to_bf16(v.f[3]) << 16);
    o.z = f32_to_bf16(v.f[4]) | (f32_to_bf16(v.f[5]) << 16);
    o.w = f32_to_bf16(v.f[6]) | (f32_to_bf16(v.f[7]) << 16);
    *(uint4*)(y + m * K + k0) = o;
  }
  if constexpr (MODE != kNormPlain) {
    constexpr int GK = MODE == kNormG32 ? 32 : 128;
    constexpr int LPG = GK / 8;
    float sf = 0.0f;
    int se = 0;
    uint2 codes;
    if constexpr (MODE == kNormStatic) {
      if (FMT == 0) sf = *(const float*)xstat;
      else se = (int)*(const uint8_t*)xstat - 127;
      codes.x = act_encode4<FMT>(v.f[0], v.f[1], v.f[2], v.f[3], sf, se);
      codes.y = act_encode4<FMT>(v.f[4], v.f[5], v.f[6], v.f[7], sf, se);
    } else {
      float amax = amax8(v);
#pragma unroll
      for (int o = 1; o < LPG; o <<= 1) amax = fmaxf(amax, __shfl_xor(amax, o, 16));
      codes = encode8<FMT>(v, amax, &sf, &se);
    }
    if (valid) {
      st_stream8(xq + m * K + k0, codes);
      if ((c & (LPG - 1)) == 0) {
        const int64_t gi = m * ((K + GK - 1) / GK) + k0 / GK;
        if (FMT == 0) ((float*)xs)[gi] = sf;
        else ((uint8_t*)xs)[gi] = (uint8_t)(se + 127);
      }
    }
  }
}

// TPR lanes per row, NC chunks of eight values per lane held in registers;
// NC = 0: rows of any length, h read a second time.
template <int FMT, int MODE, int TPR, int NC>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_quant_kernel(NormArgs a) {
  constexpr int RPW = TPR < 256 ? 256 / TPR : 1;   // rows per workgroup
  constexpr int WPR = TPR / 64;                    // waves per row
  __shared__ double red[WPR > 1 ? WPR : 1];
  const int tr = threadIdx.x % TPR;
  const int64_t m = grid_row() * RPW + threadIdx.x / TPR;
  if (m >= a.M) return;                            // whole waves: RPW > 1 has one wave per row
  const int C = (int)(a.K / 8);
  const uint16_t* xr = a.x + m * a.ldx;
  const uint16_t* rr = a.res ? a.res + m * a.ldr : nullptr;
  uint16_t* ro = a.res ? a.res_out + m * a.ldr : nullptr;
  double ss = 0.0;
  uint4 hv[NC > 0 ? NC : 1], wv[NC > 0 ? NC : 1];
  const uint4 zero = make_uint4(0, 0, 0, 0);
  if constexpr (NC > 0) {
    uint4 rv[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = tr + i * TPR;
      hv[i] = c < C ? ld_stream16(xr + (int64_t)c * 8) : zero;
      rv[i] = (rr && c < C) ? ld_stream16(rr + (int64_t)c * 8) : zero;
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = tr + i * TPR;
      wv[i] = c < C ? *(const uint4*)(a.w + (int64_t)c * 8) : zero;
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = tr + i * TPR;
      if (rr) {
        hv[i] = add_bf16x8(hv[i], rv[i]);
        if (c < C) st_stream16(ro + (int64_t)c * 8, hv[i]);
      }
      ss = square_sum8(hv[i], ss);
    }
  } else {
    for (int c = tr; c < C; c += TPR) {
      uint4 v = *(const uint4*)(xr + (int64_t)c * 8);
      if (rr) {
        v = add_bf16x8(v, *(const uint4*)(rr + (int64_t)c * 8));
        *(uint4*)(ro + (int64_t)c * 8) = v;
      }
      ss = square_sum8(v, ss);
    }
  }
  ss = wave_sum(ss);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = ss;
    __syncthreads();
    // the waves' sums (at most sixteen) in the lanes of each row of 16
    ss = row16_sum((int)(threadIdx.x & 15) < WPR ? red[threadIdx.x & 15] : 0.0);
  }
  const double r = rsqrt(ss * a.inv_k + (double)a.eps);
  RowScale rs;
  rs.hi = (float)r;
  rs.lo = (float)(r - (double)rs.hi);
  if constexpr (NC > 0) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = tr + i * TPR;
      norm_out8<FMT, MODE>(hv[i], wv[i], rs, c < C, c, a.xstat, a.y, a.xq, a.xs, m, a.K);
    }
  } else {
    // the lane reads back what it wrote itself (or x again)
    const uint16_t* hr = ro ? ro : xr;
    for (int c0 = 0; c0 < C; c0 += TPR) {
      const int c = c0 + tr;
      const uint4 h = c < C ? *(const uint4*)(hr + (int64_t)c * 8) : zero;
      const uint4 w = c < C ? *(const uint4*)(a.w + (int64_t)c * 8) : zero;
      norm_out8<FMT, MODE>(h, w, rs, c < C, c, a.xstat, a.y, a.xq, a.xs, m, a.K);
    }
  }
}

template <int FMT, int MODE>
hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
#define BSFP8_NORM(TPR, NC)                                                     \
  hipLaunchKernelGGL((norm_quant_kernel<FMT, MODE, TPR, NC>),                   \
                     row_grid(TPR < 256 ? (a.M + 256 / TPR - 1) / (256 / TPR) : a.M), \
                     dim3(TPR < 256 ? 256 : TPR), 0, s, a)
  // One chunk per lane where a workgroup has the lanes: the fewest registers
  // and the most rows in flight (8192 x 4096: 512 lanes 47.1 us, 256 lanes of
  // two chunks 46.1, one wave of eight 65).  Up to 1024 values a whole
  // workgroup per row costs more in barriers than it spreads (8192 x 1024: one
  // wave of two chunks 16.4 us, 256 lanes 20.5).
  const int64_t C = a.K / 8;
  if (C <= 64) BSFP8_NORM(64, 1);
  else if (C <= 128) BSFP8_NORM(64, 2);
  else if (C <= 256) BSFP8_NORM(256, 1);
  else if (C <= 512) BSFP8_NORM(512, 1);
  else if (C <= 1024) BSFP8_NORM(1024, 1);
  else if (C <= 2048) BSFP8_NORM(1024, 2);
  else BSFP8_NORM(1024, 0);
#undef BSFP8_NORM
  return hipGetLastError();
}

}  // namespace detail
using namespace detail;

hipError_t launch_add_rmsnorm_quant(const NormArgs& a, hipStream_t s) {
  if (!a.xq) return launch_norm<0, kNormPlain>(a, s);
  if (a.xstat) return a.fmt == 0 ? launch_norm<0, kNormStatic>(a, s) : launch_norm<1, kNormStatic>(a, s);
  if (a.group_k == 32) return a.fmt == 0 ? launch_norm<0, kNormG32>(a, s) : launch_norm<1, kNormG32>(a, s);
  return a.fmt == 0 ? launch_norm<0, kNormG128>(a, s) : launch_norm<1, kNormG128>(a, s);
}

}  // namespace bsfp8
