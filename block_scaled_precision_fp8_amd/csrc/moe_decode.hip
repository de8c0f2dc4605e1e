// A whole MoE layer for a few tokens (at most kMoeMaxTokens).
//
//   slot s = (token t, choice j): expert e = ids[t][j], skipped outside [0, E)
//   g, u = x_t W13_e^T (rows [0, I) gate, [I, 2I) up)
//   h    = bf16(silu(g) u), quantized in 1 x 128 groups (fp8_quant_act)
//   y_t  = bf16(addend_t + sum_j wt[t][j] (h_q W2_e^T)),  summed in fp32
//
// Bound by HBM: every expert that a token chose is read once, 3 H I bytes
// (half with MXFP4 weights); the tokens' own data is small and stays in L2.
//
//   moe_gate_up_kernel  one workgroup per (expert, 16 gate rows and the 16 up
//                       rows beside them): its waves deal the K blocks, each
//                       weight byte is read once for up to 64 of the expert's
//                       slots, and the waves' partial tiles meet in LDS.
//                       Also writes the slots sorted by expert.
//   quant_act_kernel    h to codes and scales
//   moe_down_kernel     one workgroup per 16 output features: its waves deal
//                       the K blocks of all experts' rows, each adds its
//                       weighted products to its own fp32 sums per token in
//                       LDS, which are joined in a fixed order: no atomics,
//                       the same bits on every run.
#include <algorithm>

#include "bsfp8.h"
#include "bsfp8_internal.h"

namespace bsfp8 {
namespace detail {

constexpr int kMoeWaves = 8;
constexpr int kMoeThreads = 64 * kMoeWaves;
constexpr int kMoeMaxSlots = kMoeMaxTokens * kMoeMaxChoices;

// The slots in expert order, left by the gate/up launch for the down launch.
struct MoePlan {
  int32_t total;                       // slots with an expert here
  int32_t pad[3];
  int32_t expert[kMoeMaxSlots];        // [total]
  int32_t slot[kMoeMaxSlots];
};

// One K block's operands of a 16-row weight tile: 32 codes per lane (MXFP4:
// 16 bytes and their scale byte).
struct WFrag {
  uint4 a, b;
  int s;
};

__device__ __forceinline__ uint4 ld_buf16(__amdgpu_buffer_rsrc_t r, uint32_t o) {
  const u32x4 t = __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 0);
  return make_uint4(t.x, t.y, t.z, t.w);
}
// weights are read once: non-temporal
__device__ __forceinline__ uint4 ld_buf16_nt(__amdgpu_buffer_rsrc_t r, uint32_t o) {
  const u32x4 t = __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 2);
  return make_uint4(t.x, t.y, t.z, t.w);
}

// 16 rows of one expert's weight (rows `row0`..) as buffers: codes, and with
// MXFP4 their scale bytes.  Offsets past the tile's end read zeros.
template <bool W4>
struct WTile {
  __amdgpu_buffer_rsrc_t codes, scales;
  uint32_t lo, slo;
  int64_t K;
  __device__ __forceinline__ WTile(const uint8_t* w, const void* sc, int64_t row0, int rows,
                                   int64_t K_, int l16)
      : K(K_) {
    const int64_t KW = W4 ? K / 2 : K;
    codes = make_rsrc(w + row0 * KW, rows * KW);
    lo = (uint32_t)(l16 * KW);
    if (W4) {
      scales = make_rsrc((const uint8_t*)sc + row0 * (K / 32), rows * (K / 32));
      slo = (uint32_t)(l16 * (K / 32));
    }
  }
  __device__ __forceinline__ WFrag load(int kb, int g4) const {
    WFrag f;
    if constexpr (W4) {
      const int64_t k = (int64_t)kb * 64 + g4 * 16;
      const bool in = k < K / 2;
      f.a = ld_buf16_nt(codes, in ? lo + (uint32_t)k : kOOB);
      f.b = make_uint4(0, 0, 0, 0);
      f.s = __builtin_amdgcn_raw_buffer_load_b8(scales, in ? slo + (uint32_t)(kb * 4 + g4) : kOOB, 0, 0);
    } else {
      const int64_t k = (int64_t)kb * 128 + g4 * 32;
      f.a = ld_buf16_nt(codes, k < K ? lo + (uint32_t)k : kOOB);
      f.b = ld_buf16_nt(codes, k + 16 < K ? lo + (uint32_t)k + 16 : kOOB);
      f.s = 0;
    }
    return f;
  }
};

// One K block of a row operand: 32 codes per lane and the group's scale
// (fp32, or the E8M0 byte).
struct XFrag {
  uint4 a, b;
  float s;
};
template <int FMT>
struct XRows {
  __amdgpu_buffer_rsrc_t codes, scales;
  int64_t K;
  int KB;
  __device__ __forceinline__ XRows(const uint8_t* x, const void* sc, int64_t rows, int64_t K_)
      : K(K_), KB((int)((K_ + 127) / 128)) {
    codes = make_rsrc(x, rows * K);
    scales = make_rsrc(sc, rows * KB * (FMT == 0 ? 4 : 1));
  }
  // row < 0: no row, zeros
  template <bool W4>
  __device__ __forceinline__ XFrag load(int row, int kb, int g4) const {
    XFrag f;
    const int64_t k0 = (int64_t)kb * 128 + (W4 ? 16 * g4 : 32 * g4);
    const int64_t k1 = k0 + (W4 ? 64 : 16);
    const uint32_t o = (uint32_t)((int64_t)row * K);
    f.a = ld_buf16(codes, row >= 0 && k0 < K ? o + (uint32_t)k0 : kOOB);
    f.b = ld_buf16(codes, row >= 0 && k1 < K ? o + (uint32_t)k1 : kOOB);
    const uint32_t so = row >= 0 ? (uint32_t)(row * KB + kb) * (FMT == 0 ? 4 : 1) : kOOB;
    if (FMT == 0) f.s = __int_as_float(__builtin_amdgcn_raw_buffer_load_b32(scales, so, 0, 0));
    else f.s = __int_as_float((int)__builtin_amdgcn_raw_buffer_load_b8(scales, so, 0, 0));
    return f;
  }
};

// sw: the weight block's scale (fp32, or the E8M0 byte; not used with MXFP4)
template <int FMT, bool W4>
__device__ __forceinline__ v4f moe_step(v4f acc, const WFrag& w, const XFrag& x, float sw) {
  if constexpr (W4) return mfma_step_w4<FMT>(acc, join(w.a, w.b), join(x.a, x.b), x.s, w.s);
  else return mfma_step<FMT>(acc, join(w.a, w.b), join(x.a, x.b), x.s, sw);
}

// ------------------------------------------------------------------------
// RT: subtiles of 16 slots served by one reading of the weights; an expert
// with more slots reads its rows again (from L2).
template <int FMT, bool W4, int RT>
__global__ __launch_bounds__(kMoeThreads) void moe_gate_up_kernel(MoeArgs a, uint16_t* h,
                                                                  MoePlan* plan, int by_slot) {
  constexpr int DEPTH = 2;
  __shared__ int list[kMoeMaxSlots];
  __shared__ int head[2];              // slots of this expert, slots of lower experts
  __shared__ v4f red[kMoeWaves][2 * RT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g4 = lane >> 4;
  const int S = a.T * a.k;
  const int e = by_slot ? __builtin_amdgcn_readfirstlane(a.ids[blockIdx.y]) : (int)blockIdx.y;
  const bool first = blockIdx.x == 0 && blockIdx.y == 0;
  const bool here = e >= 0 && e < a.E;
  if (!here && !first) return;
  // this expert's slots in slot order (wave 0), and how many lie before them
  if (wave == 0) {
    int n = 0, lower = 0, total = 0;
    for (int s0 = 0; s0 < S; s0 += 64) {
      const int s = s0 + lane;
      const int v = s < S ? a.ids[s] : -1;
      const bool ok = v >= 0 && v < a.E;
      const unsigned long long mine = __ballot(ok && v == e);
      if (ok && v == e) list[n + __popcll(mine & ((1ull << lane) - 1))] = s;
      n += __popcll(mine);
      lower += __popcll(__ballot(ok && v < e));
      total += __popcll(__ballot(ok));
    }
    if (lane == 0) {
      head[0] = here ? n : 0;
      head[1] = lower;
      if (first) plan->total = total;
    }
  }
  __syncthreads();
  const int n = __builtin_amdgcn_readfirstlane(head[0]);
  if (n == 0 || (by_slot && list[0] != (int)blockIdx.y)) return;   // not the expert's first slot
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < n; i += kMoeThreads) {
      plan->expert[head[1] + i] = e;
      plan->slot[head[1] + i] = list[i];
    }
  }

  const int64_t K = a.H, I = a.I, n0 = (int64_t)blockIdx.x * 16;
  const int KB = (int)((K + 127) / 128);
  const WTile<W4> wg(a.w13, a.s13, (int64_t)e * 2 * I + n0, 16, K, l16);
  const WTile<W4> wu(a.w13, a.s13, (int64_t)e * 2 * I + I + n0, 16, K, l16);
  const int64_t sg = ((int64_t)e * 2 * I + n0) / 128 * KB, su = sg + I / 128 * KB;
  const XRows<FMT> xr(a.xq, a.xs, a.T, K);

  for (int r0 = 0; r0 < n; r0 += 16 * RT) {
    int row[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int i = r0 + 16 * r + l16;
      row[r] = i < n ? list[i] / a.k : -1;
    }
    v4f ag[RT], au[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) ag[r] = au[r] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int kb0 = wave; kb0 < KB; kb0 += kMoeWaves * DEPTH) {
      WFrag fg[DEPTH], fu[DEPTH];
      XFrag fx[DEPTH][RT];
      float cg[DEPTH], cu[DEPTH];
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        const int kb = kb0 + d * kMoeWaves;
        const int kc = min(kb, KB - 1);          // past the end: multiplied by zeros
        fg[d] = wg.load(kb, g4);
        fu[d] = wu.load(kb, g4);
        cg[d] = W4 ? 0.f : load_scale<FMT>(a.s13, sg + kc);
        cu[d] = W4 ? 0.f : load_scale<FMT>(a.s13, su + kc);
#pragma unroll
        for (int r = 0; r < RT; ++r)
          fx[d][r] = xr.template load<W4>(kb < KB ? row[r] : -1, kb, g4);
      }
#pragma unroll
      for (int d = 0; d < DEPTH; ++d)
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          ag[r] = moe_step<FMT, W4>(ag[r], fg[d], fx[d][r], cg[d]);
          au[r] = moe_step<FMT, W4>(au[r], fu[d], fx[d][r], cu[d]);
        }
    }
    if (r0 > 0) __syncthreads();                  // the last pass's sums were read
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      red[wave][2 * r][lane] = ag[r];
      red[wave][2 * r + 1][lane] = au[r];
    }
    __syncthreads();
    for (int r = wave; r < RT; r += kMoeWaves) {
      v4f g = red[0][2 * r][lane], u = red[0][2 * r + 1][lane];
#pragma unroll
      for (int w = 1; w < kMoeWaves; ++w) {
        g += red[w][2 * r][lane];
        u += red[w][2 * r + 1][lane];
      }
      // lane: columns n0 + 4 g4 .. + 3 of slot l16
      const int i = r0 + 16 * r + l16;
      if (i < n) {
        uint32_t b[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) b[q] = f32_to_bf16(g[q] / (1.0f + expf(-g[q])) * u[q]);
        *(uint2*)(h + (int64_t)list[i] * I + n0 + 4 * g4) =
            make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
      }
    }
  }
}

// ------------------------------------------------------------------------
template <int FMT, bool W4, int RT>
__global__ __launch_bounds__(kMoeThreads) void moe_down_kernel(MoeArgs a, const uint8_t* hq,
                                                               const void* hs,
                                                               const MoePlan* plan) {
  constexpr int DEPTH = 4;
  extern __shared__ float sums[];      // [kMoeWaves][T][16]
  __shared__ int eid[kMoeMaxSlots];    // the sorted slots' experts
  __shared__ int sl[kMoeMaxSlots];     // slot | which of the token's rows in the run << 16
  __shared__ int run[1024 + 1];        // first row of every expert's run
  __shared__ int nruns;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g4 = lane >> 4;
  const int T = a.T, k = a.k;
  const int64_t N = a.H, K = a.I, n0 = (int64_t)blockIdx.x * 16;
  const int KB = (int)(K / 128);
  const int total = __builtin_amdgcn_readfirstlane(plan->total);
  float* mine = sums + (int64_t)wave * T * 16;
  for (int i = lane * 4; i < T * 16; i += 256) *(float4*)(mine + i) = make_float4(0, 0, 0, 0);
  for (int i = threadIdx.x; i < total; i += kMoeThreads) {
    eid[i] = plan->expert[i];
    sl[i] = plan->slot[i];
  }
  __syncthreads();
  if (wave == 0) {
    int n = 0;
    for (int i0 = 0; i0 < total; i0 += 64) {
      const int i = i0 + lane;
      const bool start = i < total && (i == 0 || eid[i] != eid[i - 1]);
      const unsigned long long b = __ballot(start);
      if (start) run[n + __popcll(b & ((1ull << lane) - 1))] = i;
      n += __popcll(b);
    }
    if (lane == 0) {
      run[n] = total;
      nruns = n;
    }
  } else if (wave == 1) {
    // a token that names an expert twice has neighbouring rows in its run:
    // number them, so that they add to the token's sum one after the other
    for (int i = lane; i < total; i += 64) {
      int nth = 0;
      while (nth < i && nth < k && eid[i - nth - 1] == eid[i] &&
             (sl[i - nth - 1] & 0xffff) / k == (sl[i] & 0xffff) / k)
        ++nth;
      if (nth) atomicOr(&sl[i], nth << 16);
    }
  }
  __syncthreads();

  // (run, K block) pairs dealt to the waves in equal contiguous shares
  const int64_t items = (int64_t)__builtin_amdgcn_readfirstlane(nruns) * KB;
  int64_t it = items * wave / kMoeWaves;
  const int64_t it1 = items * (wave + 1) / kMoeWaves;
  const int rows = (int)min((int64_t)16, N - n0);
  const XRows<FMT> xr(hq, hs, (int64_t)T * k, K);
  const int NB = (int)((N + 127) / 128);
  while (it < it1) {
    const int ri = (int)(it / KB), kb0 = (int)(it - (int64_t)ri * KB);
    const int kb1 = (int)min((int64_t)KB, kb0 + (it1 - it));
    it += kb1 - kb0;
    const int r0 = __builtin_amdgcn_readfirstlane(run[ri]);
    const int r1 = __builtin_amdgcn_readfirstlane(run[ri + 1]);
    const int e = __builtin_amdgcn_readfirstlane(eid[r0]);
    const WTile<W4> wt(a.w2, a.s2, (int64_t)e * N + n0, rows, K, l16);
    const int64_t sb = ((int64_t)e * NB + n0 / 128) * KB;
    for (int rb = r0; rb < r1; rb += 16 * RT) {
      int row[RT], nth[RT];
      float c[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const int i = rb + 16 * r + l16;
        const int v = i < r1 ? sl[i] : -1;
        row[r] = v < 0 ? -1 : v & 0xffff;
        nth[r] = v < 0 ? -1 : v >> 16;
        c[r] = v < 0 ? 0.f : a.wt[row[r]];
      }
      v4f acc[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[r] = v4f{0.f, 0.f, 0.f, 0.f};
      for (int kb = kb0; kb < kb1; kb += DEPTH) {
        WFrag fw[DEPTH];
        XFrag fx[DEPTH][RT];
        float sw[DEPTH];
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
          const bool in = kb + d < kb1;
          fw[d] = wt.load(in ? kb + d : KB, g4);        // KB: past the rows, zeros
          sw[d] = W4 ? 0.f : load_scale<FMT>(a.s2, sb + min(kb + d, KB - 1));
#pragma unroll
          for (int r = 0; r < RT; ++r)
            fx[d][r] = xr.template load<W4>(in ? row[r] : -1, kb + d, g4);
        }
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
#pragma unroll
          for (int r = 0; r < RT; ++r)
            acc[r] = moe_step<FMT, W4>(acc[r], fw[d], fx[d][r], sw[d]);
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        // lane: outputs n0 + 4 g4 .. + 3 of row l16
        float4* to = (float4*)(mine + (row[r] < 0 ? 0 : row[r] / k) * 16 + 4 * g4);
        for (int p = 0; __ballot(nth[r] >= p) != 0; ++p) {
          if (nth[r] == p) {
            float4 v = *to;
            v.x = fmaf(c[r], acc[r][0], v.x);
            v.y = fmaf(c[r], acc[r][1], v.y);
            v.z = fmaf(c[r], acc[r][2], v.z);
            v.w = fmaf(c[r], acc[r][3], v.w);
            *to = v;
          }
          __builtin_amdgcn_wave_barrier();
        }
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < T * 4; i += kMoeThreads) {
    const int t = i >> 2;
    const int64_t n = n0 + 4 * (i & 3);
    if (n >= N) continue;
    v4f v = *(const v4f*)(sums + t * 16 + 4 * (i & 3));
#pragma unroll
    for (int w = 1; w < kMoeWaves; ++w)
      v += *(const v4f*)(sums + ((int64_t)w * T + t) * 16 + 4 * (i & 3));
    const int64_t o = (int64_t)t * N + n;
    if (a.addend) {
      const uint2 d = *(const uint2*)(a.addend + o);
      v[0] += bf16_lo(d.x); v[1] += bf16_hi(d.x);
      v[2] += bf16_lo(d.y); v[3] += bf16_hi(d.y);
    }
    *(uint2*)(a.y + o) = make_uint2(f32_to_bf16(v[0]) | (f32_to_bf16(v[1]) << 16),
                                    f32_to_bf16(v[2]) | (f32_to_bf16(v[3]) << 16));
  }
}

// workspace: [plan][h bf16 S x I][codes S x I][scales S x I/128 x 4]
struct MoeWorkspace {
  size_t plan, h, hq, hs, bytes;
};
inline MoeWorkspace moe_layout(int64_t S, int64_t I) {
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  MoeWorkspace w;
  w.plan = 0;
  w.h = up(sizeof(MoePlan));
  w.hq = w.h + up((size_t)S * I * 2);
  w.hs = w.hq + up((size_t)S * I);
  w.bytes = w.hs + up((size_t)S * ((I + 127) / 128) * 4);
  return w;
}

template <int FMT, bool W4, int RT>
hipError_t launch_moe(const MoeArgs& a, hipStream_t s) {
  const int S = a.T * a.k;
  const MoeWorkspace w = moe_layout(S, a.I);
  uint8_t* ws = (uint8_t*)a.workspace;
  MoePlan* plan = (MoePlan*)(ws + w.plan);
  uint16_t* h = (uint16_t*)(ws + w.h);
  // one row of workgroups per expert, or per slot where those are fewer (a
  // slot whose expert came before leaves at once)
  const int by_slot = S < a.E;
  hipLaunchKernelGGL((moe_gate_up_kernel<FMT, W4, RT>),
                     dim3((unsigned)(a.I / 16), (unsigned)(by_slot ? S : a.E)), dim3(kMoeThreads),
                     0, s, a, h, plan, by_slot);
  hipError_t r = hipGetLastError();
  if (r != hipSuccess) return r;
  r = launch_quant_act(h, S, a.I, a.I, FMT, ws + w.hq, ws + w.hs, s);
  if (r != hipSuccess) return r;
  hipLaunchKernelGGL((moe_down_kernel<FMT, W4, RT>), dim3((unsigned)((a.H + 15) / 16)),
                     dim3(kMoeThreads), (size_t)kMoeWaves * a.T * 64, s, a, ws + w.hq, ws + w.hs,
                     plan);
  return hipGetLastError();
}

template <int FMT, bool W4>
hipError_t launch_moe_rt(const MoeArgs& a, hipStream_t s) {
  // the most slots one expert can expect: T tokens (each names it once)
  if (a.T <= 16) return launch_moe<FMT, W4, 1>(a, s);
  return launch_moe<FMT, W4, 2>(a, s);
}

}  // namespace detail
using namespace detail;

size_t moe_decode_workspace_bytes(int64_t S, int64_t I) { return moe_layout(S, I).bytes; }

hipError_t launch_moe_decode(const MoeArgs& a, hipStream_t s) {
  if (a.w4) return a.fmt == 0 ? launch_moe_rt<0, true>(a, s) : launch_moe_rt<1, true>(a, s);
  return a.fmt == 0 ? launch_moe_rt<0, false>(a, s) : launch_moe_rt<1, false>(a, s);
}

}  // namespace bsfp8
