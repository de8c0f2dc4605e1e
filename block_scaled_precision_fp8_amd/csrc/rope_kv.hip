// Rotary positions, and keys and values into a paged cache, in one pass.
//
//   t = pos inv_freq[i];  a' = m (a cos t - b sin t),  b' = m (b cos t + a sin t)
//
// for the pairs (i, i + rot/2) or (2i, 2i + 1) of the first rot values of a
// head; a cached row is the activation codec of fp8_quant_act over the head
// (one scale per token and head), or bf16.
//
// The angle is a product of a whole number and an fp32 one, taken in 64 bits
// (exact for positions below 2^29); whole turns leave it there, and what is left
// (at most half a turn) goes to fp32.  The rotated key is quantized from fp32, not rounded to bf16 between.
//
// Bound by HBM for a prompt (8192 tokens of 32 + 8 + 8 heads of 128, FP8 cache:
// 185 MB in 34.7 us, 5.3 TB/s; a large copy runs at 5.1), by the launch for a
// token (3.2 us).  A wave has one token, so that its sines and cosines are
// taken once for all its heads; no barrier.
#include "bsfp8_attn.h"

namespace bsfp8 {
namespace detail {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2 r = __builtin_convertvector((f32x2{a, b}), bf16x2);
  return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ uint4 pack8(const Unpacked& u) {
  return make_uint4(pack_bf16(u.f[0], u.f[1]), pack_bf16(u.f[2], u.f[3]),
                    pack_bf16(u.f[4], u.f[5]), pack_bf16(u.f[6], u.f[7]));
}

// The largest value over the LPH lanes that share a head (4, 8 or 16).
template <int LPH>
__device__ __forceinline__ float head_max(float v) {
  v = fmaxf(v, __uint_as_float(dpp<kXor1>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp<kXor2>(__float_as_uint(v))));
  if (LPH >= 8) v = fmaxf(v, __uint_as_float(dpp<kMirror8>(__float_as_uint(v))));
  if (LPH >= 16) v = fmaxf(v, __uint_as_float(dpp<kMirror16>(__float_as_uint(v))));
  return v;
}

// A wave has one token.  LPH lanes share a head, sixteen values each in two
// pieces of eight whose pairs the lane holds itself.  PER_WAVE: a wave takes
// all of its token's heads; otherwise only those of one pass, and the grid's
// second dimension has the rest.
template <int D, int KV, bool PER_WAVE>
__global__ __launch_bounds__(256) void rope_kv_kernel(RopeKvArgs a) {
  constexpr int LPH = D / 16, RPP = 64 / LPH;      // lanes of a head, heads of a pass
  __shared__ float2 turn[4][D / 2];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t t = PER_WAVE ? grid_row() * 4 + wave : (int64_t)blockIdx.x;
  if (t >= a.T) return;                            // whole waves, and no barrier below
  const int nq = a.q ? a.Hq : 0, nkv = a.k ? a.Hkv : 0;
  const int rows = nq + 2 * nkv;
  const int first = PER_WAVE ? 0 : ((int)blockIdx.y * 4 + wave) * RPP;
  const int end = PER_WAVE ? rows : (first + RPP < rows ? first + RPP : rows);
  if (first >= end) return;
  const int p = lane % LPH, half = a.rot / 2;
  const bool turned = 16 * p < a.rot;
  int c0 = 16 * p, c1 = 16 * p + 8;                // the lane's pieces of a head
  if (turned && !a.interleaved) { c0 = 8 * p; c1 = 8 * p + half; }

  int64_t slot = -1;
  if (nkv) {
    slot = a.slots[t];
    if (slot >= a.num_slots) slot = -1;
  }
  const int64_t page = slot >> a.log2_page;
  const int64_t at = slot & ((int64_t(1) << a.log2_page) - 1);

  const double pos = half ? (double)a.positions[t] : 0.0;   // without a rotation there may be none
  for (int i = lane; i < half; i += 64) {
    const double turns = pos * (double)a.inv_freq[i] * 0.15915494309189533577;   // 1 / (2 pi)
    float s, c;
    sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
    turn[wave][i] = make_float2(c * a.mscale, s * a.mscale);
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  float cs[8], sn[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 v = turned ? turn[wave][8 * p + j] : make_float2(1.0f, 0.0f);
    cs[j] = v.x;
    sn[j] = v.y;
  }

  // PER_WAVE: the next head's values are under way while one is computed, and
  // read once, past the caches (tokens of 32 + 8 + 8 heads, with the hint and without:
  // from memory 4096 20 us, 24; 8192 36, 42; where the launch before has just
  // written them 2048 12.8, 11.1; 4096 18.7, 17.7; 8192 36.8, 39.4)
  auto ld = [](const uint16_t* p) { return PER_WAVE ? ld_stream16(p) : *(const uint4*)p; };
  auto source = [&](int r) {
    const uint16_t* p = r < nq ? a.q + t * a.ldq + (int64_t)r * D
                        : r < nq + nkv ? a.k + t * a.ldk + (int64_t)(r - nq) * D
                                       : a.v + t * a.ldv + (int64_t)(r - nq - nkv) * D;
    return p;
  };
  const int stop = slot < 0 && end > nq ? nq : end;   // nothing is cached
  int r = first + lane / LPH;
  uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
  if (r < stop) {
    const uint16_t* src = source(r);
    v0 = ld(src + c0);
    v1 = ld(src + c1);
  }
  for (; r < stop; r += RPP) {
    const bool isq = r < nq, isk = !isq && r < nq + nkv;
    const int h = isq ? r : (isk ? r - nq : r - nq - nkv);
    Unpacked x = unpack8(v0), z = unpack8(v1);
    if (PER_WAVE && r + RPP < stop) {
      const uint16_t* src = source(r + RPP);
      v0 = ld(src + c0);
      v1 = ld(src + c1);
    }
    if (turned && (isq || isk)) {
      if (a.interleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float u0 = x.f[2 * j], u1 = x.f[2 * j + 1], w0 = z.f[2 * j], w1 = z.f[2 * j + 1];
          x.f[2 * j] = u0 * cs[j] - u1 * sn[j];
          x.f[2 * j + 1] = u1 * cs[j] + u0 * sn[j];
          z.f[2 * j] = w0 * cs[4 + j] - w1 * sn[4 + j];
          z.f[2 * j + 1] = w1 * cs[4 + j] + w0 * sn[4 + j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float u = x.f[j], w = z.f[j];
          x.f[j] = u * cs[j] - w * sn[j];
          z.f[j] = w * cs[j] + u * sn[j];
        }
      }
    }
    if (isq) {
      uint16_t* o = a.q_out + t * a.ldqo + (int64_t)h * D;
      *(uint4*)(o + c0) = pack8(x);
      *(uint4*)(o + c1) = pack8(z);
      continue;
    }
    const int64_t row = ((page * a.Hkv + h) << a.log2_page) + at;
    void* cache = isk ? a.k_cache : a.v_cache;
    if constexpr (KV == kKvBf16) {
      uint16_t* o = (uint16_t*)cache + row * D;
      *(uint4*)(o + c0) = pack8(x);
      *(uint4*)(o + c1) = pack8(z);
    } else {
      const float amax = head_max<LPH>(fmaxf(amax8(x), amax8(z)));
      float sf;
      int se;
      uint8_t* o = (uint8_t*)cache + row * D;
      *(uint2*)(o + c0) = encode8<KV>(x, amax, &sf, &se);
      *(uint2*)(o + c1) = encode8<KV>(z, amax, &sf, &se);
      if (p == 0) {
        void* scale = isk ? a.k_scale : a.v_scale;
        if (KV == kKvFloat) ((float*)scale)[row] = sf;
        else ((uint8_t*)scale)[row] = (uint8_t)(se + 127);
      }
    }
  }
}

template <int D>
hipError_t launch_rope_kv(const RopeKvArgs& a, hipStream_t s) {
  const int64_t rows = (a.q ? a.Hq : 0) + 2 * (a.k ? a.Hkv : 0), pass = 4 * (64 / (D / 16));
  // a wave per token, or workgroups: 512 tokens 7.4 us
  // and 5.7, 1024 8.0 and 7.9, 2048 11.3 and 12.2
  const bool per_wave = a.T >= 1024;
  const dim3 grid = per_wave ? row_grid((a.T + 3) / 4)
                             : dim3((unsigned)a.T, (unsigned)((rows + pass - 1) / pass));
#define BSFP8_ROPE(KV)                                                                       \
  do {                                                                                       \
    if (per_wave) hipLaunchKernelGGL((rope_kv_kernel<D, KV, true>), grid, dim3(256), 0, s, a);  \
    else hipLaunchKernelGGL((rope_kv_kernel<D, KV, false>), grid, dim3(256), 0, s, a);       \
  } while (0)
  if (a.fmt == kKvFloat) BSFP8_ROPE(kKvFloat);
  else if (a.fmt == kKvUe8m0) BSFP8_ROPE(kKvUe8m0);
  else BSFP8_ROPE(kKvBf16);
#undef BSFP8_ROPE
  return hipGetLastError();
}

// theta_i = base^(-2i / rot).  By parts: theta turns r = orig_len theta / 2 pi
// times within the original context; from `high` turns on it stays, up to
// `low` it is divided by the factor, between the two linearly mixed.
__global__ void inv_freq_kernel(int scaling, int rot, double base, double factor, double low,
                                double high, double orig_len, float* out) {
  for (int i = threadIdx.x; i < rot / 2; i += blockDim.x) {
    const double f = pow(base, -2.0 * i / rot);
    double keep = scaling == 0 ? 1.0 : 0.0;
    if (scaling == 2) {
      const double r = orig_len * f * 0.15915494309189533577;
      keep = fmin(fmax((r - low) / (high - low), 0.0), 1.0);
    }
    // a factor that nothing is divided by may be anything
    out[i] = (float)(keep == 1.0 ? f : f * keep + f / factor * (1.0 - keep));
  }
}

}  // namespace detail
using namespace detail;

hipError_t launch_rope_inv_freq(int scaling, int rot, double base, double factor, double low,
                                double high, double orig_len, float* out, hipStream_t s) {
  hipLaunchKernelGGL(inv_freq_kernel, dim3(1), dim3(128), 0, s, scaling, rot, base, factor, low,
                     high, orig_len, out);
  return hipGetLastError();
}

hipError_t launch_rope_kv_append(const RopeKvArgs& a, hipStream_t s) {
  if (a.D == 64) return launch_rope_kv<64>(a, s);
  if (a.D == 128) return launch_rope_kv<128>(a, s);
  return launch_rope_kv<256>(a, s);
}

}  // namespace bsfp8
