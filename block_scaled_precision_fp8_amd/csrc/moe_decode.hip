// A whole MoE layer for a few tokens (at most kMoeMaxTokens).
//
//   slot s = (token t, choice j): expert e = ids[t][j], skipped outside [0, E)
//   g, u = x_t W13_e^T (rows [0, I) gate, [I, 2I) up)
//   h    = bf16(silu(g) u), quantized in 1 x 128 groups (fp8_quant_act)
//   y_t  = bf16(addend_t + sum_j wt[t][j] (h_q W2_e^T)),  summed in fp32
//
// Bound by HBM: an expert that a token chose is read once for every segment
// of 16, 32 or 64 of its slots (see subtiles), once where it has no more: 3 H I
// bytes (half with MXFP4 weights); the tokens' own data is small and stays in
// L2.
//
//   moe_gate_up_kernel  one workgroup per CU; its tasks are (segment of an
//                       expert's slots, 16 columns of h), dealt in equal
//                       contiguous shares.  Writes h in bf16, and the slots
//                       sorted by expert for the next launch.
//   quant_act_kernel    h to codes and scales, where the down launch does not
//                       do that itself
//   moe_down_kernel     one workgroup per R (8 to 32) output features; its tasks
//                       are the segments.  Each wave adds its weighted products
//                       to its own fp32 sums per token in LDS, which are
//                       joined in a fixed order.
//
// In both a workgroup's waves take equal contiguous shares of its (task, K
// block) pairs and stream the weights through a ring of registers across
// tasks, with no barrier until the end.  No sum depends on an order that
// varies (the one atomic counts slots, in LDS): the same bits on every run.
//
// Measured (gate/up + down, TB/s of the weights read): 1 token x 8 of 256 FP8
// experts (7168, 2048) 47.5 + 25.0 us (4.9, 4.7), 16 tokens 542 + 255 us (5.5,
// 5.9); 64 tokens on 32 of them 174 + 76 us (4.7, 5.3); 33 x 2 of 8 MXFP4
// experts (4096, 14336) 121 + 73 us (4.1, 3.4); 5 x 6 of 64 (2064, 1408) 40.6 +
// 30.2 us (3.4, 2.3); boxes differ by 3%.  128 tokens: 2 of 8 FP8 experts (4096,
// 14336) 273 + 189 us, MXFP4 236 + 152; 8 of 64 (7168, 2048) 498 + 285; one of
// those 64 for all 128 tokens and the others for one each 436 + 204.  A plain
// read of 235 MB runs at 5.6 to 5.9.  The MXFP4 stream has
// half the bytes for the same conversions and exchanges, and its ring drains
// in part wherever a scale chunk is taken up.  Tried without gain: deeper and
// shallower rings, 16 waves per workgroup, the waves of a workgroup kept in
// step by barriers, non-temporal weight loads (10% slower), a second LDS buffer
// for the tokens' rows, encoding h under the first weights.
#include "bsfp8.h"
#include "bsfp8_layer.h"

namespace bsfp8 {
namespace detail {

constexpr int kMoeWaves = 8;
constexpr int kMoeThreads = 64 * kMoeWaves;
constexpr int kMoeMaxSlots = kMoeMaxTokens * kMoeMaxChoices;

// A sorted slot as one word: slot, its token, and (down launch) which of its
// token's rows in the expert's run it is.
static_assert(kMoeMaxSlots <= 1 << 11 && kMoeMaxTokens <= 1 << 7, "slot word");
__device__ __forceinline__ int slot_word(int slot, int k) { return slot | (slot / k) << 11; }
__device__ __forceinline__ int slot_of(int w) { return w & 0x7ff; }
__device__ __forceinline__ int token_of(int w) { return w >> 11 & 0x7f; }
__device__ __forceinline__ int nth_of(int w) { return w >> 18; }      // -1 for w = -1

// The sorted slots and their segments, left by the gate/up launch for the
// down launch (which loads all arrays before it knows the counts).
struct MoePlan {
  int32_t nsegs, subtiles, pad[2];
  uint16_t seg[kMoeMaxSlots + 8];      // first row of every segment, and total
  int32_t expert[kMoeMaxSlots];
  int32_t slot[kMoeMaxSlots];          // slot words
  float weight[kMoeMaxSlots];
};

// A value that all lanes hold, into a scalar register.  64-bit divisions and
// comparisons leave theirs in vector registers, and a buffer that depends on
// one gets a loop over the lanes around each of its loads.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// ---- operands ----------------------------------------------------------
// The products run on the bf16 MFMA: every E4M3 and E2M1 value is a bf16
// value, and the instruction keeps 24 bits below a group's largest product.
// The FP8 MFMAs keep 13 (measured: 2^-16 of sum |a b| off for normal data,
// 2^-13 with 50-fold outlier channels, against 2^-24 here), which moves
// codes of h.  The conversions are free under the weight stream.
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
struct BFrag { bf8 v[4]; };            // 32 values of one row

__device__ __forceinline__ uint4 ld_buf16(__amdgpu_buffer_rsrc_t r, uint32_t o) {
  const u32x4 t = __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 0);
  return make_uint4(t.x, t.y, t.z, t.w);
}

__device__ __forceinline__ bf8 cvt_e4m3x8(uint32_t a, uint32_t b) {
  const bf2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
  const bf2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
  const bf2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
  const bf2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
  return bf8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}
__device__ __forceinline__ bf8 cvt_e2m1x8(uint32_t a, float s) {
  const bf2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, s, 0);
  const bf2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, s, 1);
  const bf2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, s, 2);
  const bf2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a, s, 3);
  return bf8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// The buffers here have less than 2^31 bytes: no clamp.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, uniform((int)bytes), 0x00020000);
}

// A stored scale, as loaded: the fp32 value, or the E8M0 byte.
template <int FMT>
__device__ __forceinline__ float scale_value(uint32_t s) {
  return FMT == 0 ? __uint_as_float(s) : e8m0_f32(s);
}

// One K block of a 16-row weight tile: a lane's 32 codes of row l16, with
// MXFP4 the scales as loaded.  FP8: K 16 g4 .. + 15 and 64 + 16 g4 .. + 15 (the
// order within a block is free while rows and weights agree; four lanes then
// read 64 bytes in a piece).  MXFP4: the group K 32 g4 .. + 31.
template <bool W4>
struct WFrag {
  uint4 c[W4 ? 1 : 2];
  uint32_t s[W4 ? 1 : 0];              // with BYTES, below
};
// A value per row of a 16-row operand: loaded by the lanes of g4 = 0 only (a
// load costs its lanes' addresses, not its bytes), spread to all four groups.
__device__ __forceinline__ uint32_t spread16(uint32_t v, int l16) {
  return (uint32_t)__builtin_amdgcn_ds_bpermute(l16 * 4, (int)v);
}

// Up to 16 rows of one expert's weight.  MXFP4 scales reach a weight lane
// through LDS, 32 blocks of 16 rows at a time (ScaleChunk), or (BYTES: rows of
// scales that do not begin at a dword) as a byte per lane and block.  A row's
// scales for 32 blocks share one cache line, which has left the L1 before the
// next block: loaded block by block it is fetched again for every one, as
// many bytes as four times the weights.
//
// In a row's last, partial K block a
// lane reads on into the next row: finite values, which meet zeros of the
// tokens' rows.  Blocks from KB on give zeros and no traffic.
template <bool W4, bool BYTES>
struct WTile {
  __amdgpu_buffer_rsrc_t codes, scales;
  uint32_t lo, slo, K;
  int KB, g4;
  __device__ __forceinline__ void init(int64_t K_, int lane) {
    K = (uint32_t)K_;
    KB = (int)((K_ + 127) / 128);
    g4 = lane >> 4;
    lo = (uint32_t)((lane & 15) * (W4 ? K_ / 2 : K_)) + g4 * 16;
    slo = (uint32_t)((lane & 15) * (K_ / 32)) + g4;
  }
  // n <= 16 rows from row0 on; the others give zeros
  __device__ __forceinline__ void aim(const uint8_t* w, const void* sc, int64_t row0, int n) {
    const uint32_t KW = W4 ? K / 2 : K;
    codes = row_rsrc(w + row0 * KW, n * KW);
    if (W4 && BYTES)
      scales = row_rsrc((const uint8_t*)sc + row0 * (K / 32), n * (K / 32));
  }
  __device__ __forceinline__ WFrag<W4> load(int kb) const {
    WFrag<W4> f;
    const uint32_t o = lo + (kb < KB ? (uint32_t)kb * (W4 ? 64 : 128) : kOOB);
    f.c[0] = ld_buf16(codes, o);
    if constexpr (W4) {
      if constexpr (BYTES) {
        // the group itself may lie past the row: its scale is another row's
        const bool in = (uint32_t)kb * 128 + g4 * 32 < K;
        f.s[0] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(scales, in ? slo + (uint32_t)kb * 4 : kOOB, 0, 0);
      }
    } else {
      f.c[1] = ld_buf16(codes, o + 64);
    }
    return f;
  }
  // the codes as bf16, with MXFP4 times their group's scale; chunk: the
  // block's column of this row's dwords in LDS
  __device__ __forceinline__ BFrag bf16(const WFrag<W4>& w, const uint32_t* chunk) const {
    BFrag f;
    if constexpr (W4) {
      const uint32_t b = BYTES ? w.s[0] : *chunk >> (8 * g4) & 0xff;
      const float sc = __uint_as_float(b << 23);     // the conversion reads the exponent field
      f.v[0] = cvt_e2m1x8(w.c[0].x, sc); f.v[1] = cvt_e2m1x8(w.c[0].y, sc);
      f.v[2] = cvt_e2m1x8(w.c[0].z, sc); f.v[3] = cvt_e2m1x8(w.c[0].w, sc);
    } else {
      f.v[0] = cvt_e4m3x8(w.c[0].x, w.c[0].y); f.v[1] = cvt_e4m3x8(w.c[0].z, w.c[0].w);
      f.v[2] = cvt_e4m3x8(w.c[1].x, w.c[1].y); f.v[3] = cvt_e4m3x8(w.c[1].z, w.c[1].w);
    }
    return f;
  }
};

// The scale dwords (four groups, one K block) of 16 rows and 32 blocks:
// loaded into registers a chunk ahead, then kept in the wave's own LDS.
constexpr int kChunk = 32, kChunkRow = kChunk + 1;         // + 1: rows in different banks
constexpr int kChunkDwords = 16 * kChunkRow;
struct ScaleChunk {
  uint32_t v[8];
  // K % 128 == 0
  __device__ __forceinline__ void load(const void* sc, int64_t row0, int n, int64_t K, int kb0,
                                       int lane) {
    const uint32_t row = (uint32_t)(K / 32), kb = kb0 + (lane & 31);
    const __amdgpu_buffer_rsrc_t r = row_rsrc((const uint8_t*)sc + row0 * row, n * row);
    // one choice for all eight: a choice at each load becomes a branch around
    // it, and every such branch waits for all loads in flight
    const uint32_t o = (lane >> 5) * row + (kb * 4 < row ? kb * 4 : kOOB);
#pragma unroll
    for (int q = 0; q < 8; ++q)
      v[q] = __builtin_amdgcn_raw_buffer_load_b32(r, o + 2 * q * row, 0, 0);
  }
  __device__ __forceinline__ void store(uint32_t* lds, int lane) const {
#pragma unroll
    for (int q = 0; q < 8; ++q) lds[(2 * q + (lane >> 5)) * kChunkRow + (lane & 31)] = v[q];
  }
};

// One K block of 16 token (or h) rows.  Loaded eight lanes to a row, whole
// 128-byte pieces, and turned into the MFMA's layout through 2 KB of the
// wave's own LDS: read in that layout (a lane per row) the rows would take
// as many address cycles as the weights.
struct XFrag {
  uint4 c[2];                          // rows lane / 8 and 8 + lane / 8
};
__device__ __forceinline__ int xpiece(int row, int piece) {      // LDS offset, banks spread
  return row * 128 + ((piece ^ (row >> 1 & 7)) * 16);
}
__device__ __forceinline__ void x_to_lds(uint8_t* lds, const XFrag& x, int lane) {
  *(uint4*)(lds + xpiece(lane >> 3, lane & 7)) = x.c[0];
  *(uint4*)(lds + xpiece(8 + (lane >> 3), lane & 7)) = x.c[1];
}
__device__ __forceinline__ BFrag x_bf16(uint4 a, uint4 b) {
  BFrag f;
  f.v[0] = cvt_e4m3x8(a.x, a.y); f.v[1] = cvt_e4m3x8(a.z, a.w);
  f.v[2] = cvt_e4m3x8(b.x, b.y); f.v[3] = cvt_e4m3x8(b.z, b.w);
  return f;
}
// the 32 codes that meet a weight lane's: pieces g4 and 4 + g4, with MXFP4
// 2 g4 and 2 g4 + 1
template <bool W4>
__device__ __forceinline__ BFrag x_from_lds(const uint8_t* lds, int lane) {
  const int l16 = lane & 15, g4 = lane >> 4;
  return x_bf16(*(const uint4*)(lds + xpiece(l16, W4 ? 2 * g4 : g4)),
                *(const uint4*)(lds + xpiece(l16, W4 ? 2 * g4 + 1 : 4 + g4)));
}

// acc += (W X^T of one K block) * scale: output rows n (registers), slots m
// (lanes).  c: the row group's scale, times the weight block's (FP8).
__device__ __forceinline__ v4f moe_step(v4f acc, const BFrag& w, const BFrag& x, float c) {
  v4f t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[i], x.v[i], t, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = fmaf(t[i], c, acc[i]);
  return acc;
}

// ------------------------------------------------------------------------
// The slots sorted by expert (in slot order within one), in LDS, and their
// segments: at most ROWS rows of one expert.
struct SortedSlots {
  int eid[kMoeMaxSlots];
  int sl[kMoeMaxSlots];                // slot words
  uint16_t seg[kMoeMaxSlots + 1];      // first row of every segment
  int nsegs, total, rt;                // rt: subtiles of a segment
};

// Subtiles of 16 rows per segment, by the average run of an expert's slots: a
// run of more rows reads its weights again, a subtile costs registers and a
// shorter ring.  The average says little where one expert has most slots.
// Measured, gate/up + down us with 1 / 2 / 4: FP8, runs of 8 (7168, 2048, 64
// experts) 390 + 169 / 392 + 177 / 456 + 225, of 16 (4096, 14336, 8 experts)
// 291 + 160 / 219 + 140 / 239 + 152, of 32 469 + 270 / 344 + 217 / 272 + 192.
// MXFP4, where 4 leave no room for two blocks an item: runs of 32 280 + 168 /
// 228 + 147 / 243 + 173, of 64 - / 370 + 245 / 393 + 266, of 128 - / 516 + 383
// / 519 + 393.
template <bool W4>
__device__ __forceinline__ int subtiles(int total, int runs) {
  return total <= 10 * runs ? 1 : W4 || total <= 20 * runs ? 2 : 4;
}

// By one wave, after eid.  MANY: a run can have more than 16 rows.
template <bool W4, bool MANY>
__device__ __forceinline__ void find_segments(SortedSlots& p, int total, int lane) {
  auto starts_run = [&](int i) { return i < total && (i == 0 || p.eid[i] != p.eid[i - 1]); };
  int rt = 1;
  if (MANY) {
    int runs = 0;
    for (int i0 = 0; i0 < total; i0 += 64) runs += __popcll(__ballot(starts_run(i0 + lane)));
    rt = subtiles<W4>(total, runs);
  }
  // a row starts a segment when its place in its run is a multiple of 16 rt
  int n = 0, start = 0;
  for (int i0 = 0; i0 < total; i0 += 64) {
    const int i = i0 + lane;
    const unsigned long long b = __ballot(starts_run(i)) & (~0ull >> (63 - lane));
    const int mine = b ? i0 + 63 - __clzll(b) : start;     // this row's run's start
    const bool st = i < total && ((i - mine) & (16 * rt - 1)) == 0;
    const unsigned long long sb = __ballot(st);
    if (st) p.seg[n + __popcll(sb & ((1ull << lane) - 1))] = (uint16_t)i;
    n += __popcll(sb);
    start = __shfl(mine, 63);
  }
  if (lane == 0) {
    p.seg[n] = (uint16_t)total;
    p.nsegs = n;
    p.total = total;
    p.rt = rt;
  }
}

// The sort and the segments, by the whole workgroup: a slot's place is the
// number of slots of lower experts and of earlier slots of its own.  key:
// kMoeMaxSlots words.
template <bool W4, bool MANY>
__device__ __forceinline__ void sort_slots(SortedSlots& p, int* key, const int32_t* ids, int S,
                                           int k, int E, int lane, int wave) {
  constexpr int kSkip = 0x7fffffff;                        // behind all others
  if (S <= 64) {
    // one wave, in registers
    if (wave == 0) {
      int e = lane < S ? ids[lane] : -1;
      if (e < 0 || e >= E) e = kSkip;
      int at = 0;
      for (int j = 0; j < S; ++j) {
        const int o = __builtin_amdgcn_readlane(e, j);
        at += o < e || (o == e && j < lane);
      }
      if (e != kSkip) {
        p.eid[at] = e;
        p.sl[at] = slot_word(lane, k);
      }
      find_segments<W4, MANY>(p, __popcll(__ballot(e != kSkip)), lane);
    }
    __syncthreads();
    return;
  }
  const int S4 = (S + 3) & ~3;
  for (int i = threadIdx.x; i < S4; i += kMoeThreads) {
    const int e = i < S ? ids[i] : -1;
    key[i] = e >= 0 && e < E ? e : kSkip;
  }
  if (threadIdx.x == 0) p.total = 0;
  __syncthreads();
  int valid = 0;
  for (int i = threadIdx.x; i < S; i += kMoeThreads) {
    const int e = key[i];
    if (e == kSkip) continue;
    int at = 0;
    for (int j = 0; j < S4; j += 4) {
      const int4 o = *(const int4*)(key + j);
      at += (o.x < e || (o.x == e && j < i)) + (o.y < e || (o.y == e && j + 1 < i)) +
            (o.z < e || (o.z == e && j + 2 < i)) + (o.w < e || (o.w == e && j + 3 < i));
    }
    p.eid[at] = e;
    p.sl[at] = slot_word(i, k);
    ++valid;
  }
  if (valid) atomicAdd(&p.total, valid);
  __syncthreads();
  if (wave == 0) find_segments<W4, MANY>(p, __builtin_amdgcn_readfirstlane(p.total), lane);
  __syncthreads();
}

// ------------------------------------------------------------------------
template <int FMT, bool W4, bool RAGGED, int RT>
__device__ __forceinline__ void gate_up(const MoeArgs& a, uint16_t* h, const SortedSlots& p,
                                        v4f* part, int lane, int wave) {
  constexpr bool CHUNK = W4 && !RAGGED;
  // an item: U K blocks, 128 bytes of a weight row (MXFP4: both halves of a
  // cache line in one go)
  constexpr int U = W4 ? 2 : 1;
  constexpr int D = W4 ? (RT == 1 ? 4 : 2) : (RT == 1 ? 5 : RT == 2 ? 4 : 2);
  constexpr int SB = FMT == 0 ? 4 : 1;
  const int l16 = lane & 15, g4 = lane >> 4;
  const int64_t K = a.H, I = a.I;
  const int KB = (int)((K + 127) / 128), KI = (KB + U - 1) / U, CT = (int)(I / 16);
  const int64_t tasks = (int64_t)uniform(p.nsegs) * CT;
  const int64_t t0 = tasks * blockIdx.x / gridDim.x, t1 = tasks * (blockIdx.x + 1) / gridDim.x;
  const int64_t items = (t1 - t0) * KI;
  auto share = [&](int w) { return items * w / kMoeWaves; };
  const int64_t it0 = share(wave);
  const int cnt = uniform((int)(share(wave + 1) - it0));

  // partial products of tasks that begin or end inside a wave's share: 0
  // begun by an earlier wave, 1 begun here and left to the next
  auto piece = [&](int w, int which, int i) -> v4f& {
    return part[((w * 2 + which) * 2 * RT + i) * 64 + lane];
  };
  // h of one task from its products: lane (l16, g4) has columns 4 g4 .. + 3
  // of row l16
  auto finish = [&](const v4f (&g)[RT], const v4f (&u)[RT], int seg, int ct) {
    const int r0 = p.seg[seg], r1 = p.seg[seg + 1];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int i = r0 + 16 * r + l16;
      uint32_t b[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        b[q] = f32_to_bf16(g[r][q] / (1.0f + expf(-g[r][q])) * u[r][q]);
      if (i < r1)
        *(uint2*)(h + (int64_t)slot_of(p.sl[i]) * I + ct * 16 + 4 * g4) =
            make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
    }
  };

  if (cnt > 0) {
    uint8_t* xbuf = (uint8_t*)&part[(wave * 2 + 1) * 2 * RT * 64];   // free until the last task
    uint32_t* chunks = (uint32_t*)&part[kMoeWaves * 4 * RT * 64] + wave * 2 * kChunkDwords;
    const __amdgpu_buffer_rsrc_t rows = row_rsrc(a.xq, (uint32_t)(a.T * K));
    const __amdgpu_buffer_rsrc_t rscales = row_rsrc(a.xs, (uint32_t)(a.T * KB * SB));
    // two cursors over the wave's items: loads, and products behind them
    const int64_t task = t0 + it0 / KI;
    int lseg = uniform((int)(task / CT)), lct = uniform((int)(task - (int64_t)lseg * CT));
    int lki = uniform((int)(it0 - it0 / KI * KI)), left = cnt;
    int pseg = lseg, pct = lct, pki = lki, begun = lki;
    const uint32_t xk = (lane & 7) * 16;
    uint32_t xo[2 * RT], so[RT];       // the segment's rows; no row: past the buffers
    int e = 0;
    WTile<W4, RAGGED> wg, wu;
    __amdgpu_buffer_rsrc_t sg, su;
    wg.init(K, lane);
    wu.init(K, lane);
    auto aim_rows = [&]() {
      const int r0 = uniform(p.seg[lseg]), r1 = uniform(p.seg[lseg + 1]);
      e = uniform(p.eid[r0]);
#pragma unroll
      for (int r = 0; r < 2 * RT; ++r) {
        const int i = r0 + 8 * r + (lane >> 3);
        xo[r] = i < r1 ? token_of(p.sl[i]) * (uint32_t)K + xk : kOOB;
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const int i = r0 + 16 * r + l16;
        so[r] = g4 == 0 && i < r1 ? token_of(p.sl[i]) * (uint32_t)KB * SB : kOOB;
      }
    };
    auto aim = [&]() {
      const int64_t row = (int64_t)e * 2 * I + lct * 16;
      wg.aim(a.w13, a.s13, row, 16);
      wu.aim(a.w13, a.s13, row + I, 16);
      if (!W4) {
        sg = row_rsrc((const uint8_t*)a.s13 + row / 128 * KB * SB, KB * SB);
        su = row_rsrc((const uint8_t*)a.s13 + (row + I) / 128 * KB * SB, KB * SB);
      }
    };
    struct Item {
      WFrag<W4> g[U], u[U];
      XFrag x[U][RT];
      uint32_t sx[U][RT], sg, su;
    } ring[D];
    auto next = [&](Item& f) {
      const bool in = left > 0;        // past the share: zeros, no traffic
      const int kb = in ? lki * U : KB;
#pragma unroll
      for (int q = 0; q < U; ++q) f.g[q] = wg.load(kb + q);
#pragma unroll
      for (int q = 0; q < U; ++q) f.u[q] = wu.load(kb + q);
      const uint32_t sk = in ? (uint32_t)kb * SB : 0x40000000u;
#pragma unroll
      for (int q = 0; q < U; ++q) {
        const uint32_t k = (uint32_t)(kb + q) * 128;
        const uint32_t sq = kb + q < KB ? (uint32_t)(kb + q) * SB : 0x40000000u;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          f.x[q][r].c[0] = ld_buf16(rows, k + xk < (uint32_t)K ? xo[2 * r] + k : kOOB);
          f.x[q][r].c[1] = ld_buf16(rows, k + xk < (uint32_t)K ? xo[2 * r + 1] + k : kOOB);
          if (FMT == 0) f.sx[q][r] = __builtin_amdgcn_raw_buffer_load_b32(rscales, so[r] + sq, 0, 0);
          else f.sx[q][r] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(rscales, so[r] + sq, 0, 0);
        }
      }
      if constexpr (!W4) {
        if (FMT == 0) {
          f.sg = __builtin_amdgcn_raw_buffer_load_b32(sg, sk, 0, 0);
          f.su = __builtin_amdgcn_raw_buffer_load_b32(su, sk, 0, 0);
        } else {
          f.sg = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(sg, sk, 0, 0);
          f.su = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(su, sk, 0, 0);
        }
      }
      if (--left > 0 && ++lki == KI) {
        lki = 0;
        if (++lct == CT) {
          lct = 0;
          ++lseg;
          aim_rows();
        }
        aim();
      }
    };
    // scale chunks: loaded one ahead of the products
    ScaleChunk cg4, cu4;
    int cseg = pseg, cct = pct, ckb = pki * U & ~(kChunk - 1), cleft = (cnt + pki) * U - ckb;
    auto next_chunk = [&]() {
      if (cleft <= 0) return;
      const int64_t row = (int64_t)uniform(p.eid[uniform(p.seg[cseg])]) * 2 * I + cct * 16;
      cg4.load(a.s13, row, 16, K, ckb, lane);
      cu4.load(a.s13, row + I, 16, K, ckb, lane);
      cleft -= min(kChunk, KI * U - ckb);
      ckb += kChunk;
      if (ckb >= KB) {
        ckb = 0;
        if (++cct == CT) {
          cct = 0;
          ++cseg;
        }
      }
    };
    if (CHUNK) next_chunk();
    aim_rows();
    aim();
#pragma unroll
    for (int d = 0; d < D; ++d) next(ring[d]);
    bool fresh = true;                 // the products enter a chunk
    v4f ag[RT], au[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) ag[r] = au[r] = v4f{0.f, 0.f, 0.f, 0.f};
    int prows = uniform(p.seg[pseg + 1] - p.seg[pseg]);
    for (int i0 = 0; i0 < cnt; i0 += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (i0 + d < cnt) {
          if (CHUNK && fresh) {
            cg4.store(chunks, lane);
            cu4.store(chunks + kChunkDwords, lane);
            next_chunk();
          }
          const float cg = W4 ? 1.f : scale_value<FMT>(ring[d].sg);
          const float cu = W4 ? 1.f : scale_value<FMT>(ring[d].su);
#pragma unroll
          for (int q = 0; q < U; ++q) {
#pragma unroll
            for (int r = 0; r < RT; ++r) x_to_lds(xbuf + r * 2048, ring[d].x[q][r], lane);
            const uint32_t* ch = chunks + l16 * kChunkRow + (pki * U & (kChunk - 1)) + q;
            const BFrag bg = wg.bf16(ring[d].g[q], ch);
            const BFrag bu = wu.bf16(ring[d].u[q], ch + kChunkDwords);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
              if (r > 0 && prows <= 16 * r) break;
              const BFrag bx = x_from_lds<W4>(xbuf + r * 2048, lane);
              const float sx = scale_value<FMT>(spread16(ring[d].sx[q][r], l16));
              ag[r] = moe_step(ag[r], bg, bx, sx * cg);
              au[r] = moe_step(au[r], bu, bx, sx * cu);
            }
          }
        }
        next(ring[d]);
        const bool last = i0 + d + 1 == cnt;
        if (i0 + d < cnt && (++pki == KI || last)) {         // the task's end, here
          if (pki == KI && begun == 0) {
            finish(ag, au, pseg, pct);
          } else {
#pragma unroll
            for (int r = 0; r < RT; ++r) {
              piece(wave, begun == 0, 2 * r) = ag[r];
              piece(wave, begun == 0, 2 * r + 1) = au[r];
            }
          }
#pragma unroll
          for (int r = 0; r < RT; ++r) ag[r] = au[r] = v4f{0.f, 0.f, 0.f, 0.f};
          if (!last) {
            begun = pki = 0;
            if (++pct == CT) {
              pct = 0;
              ++pseg;
              prows = uniform(p.seg[pseg + 1] - p.seg[pseg]);
            }
          }
        }
        fresh = (pki * U & (kChunk - 1)) == 0;
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    left = begun == 0 && pki < KI;     // the last task: begun here, not ended
    lseg = pseg;
    lct = pct;
    __syncthreads();
    if (left) {
      v4f g[RT], u[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        g[r] = piece(wave, 1, 2 * r);
        u[r] = piece(wave, 1, 2 * r + 1);
      }
      const int64_t end = (share(wave + 1) / KI + 1) * KI;
      for (int w = wave + 1; w < kMoeWaves; ++w) {
        if (share(w) == share(w + 1)) continue;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          g[r] += piece(w, 0, 2 * r);
          u[r] += piece(w, 0, 2 * r + 1);
        }
        if (share(w + 1) >= end) break;
      }
      finish(g, u, lseg, lct);
    }
  } else {
    __syncthreads();
  }
}

// MANY: more than 16 tokens, so that an expert can have more than 16 slots.
template <int FMT, bool W4, bool RAGGED, bool MANY>
__global__ __launch_bounds__(kMoeThreads) void moe_gate_up_kernel(MoeArgs a, uint16_t* h,
                                                                  MoePlan* plan) {
  __shared__ SortedSlots p;
  // partial products of 1, 2 or 4 (MXFP4: 2) subtiles, the scale chunks behind
  constexpr int kPart = kMoeWaves * 4 * 64, kChunks = W4 ? kMoeWaves * 2 * kChunkDwords / 4 : 0;
  __shared__ v4f part[(MANY ? (W4 ? 2 : 4) : 1) * kPart + kChunks];
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  sort_slots<W4, MANY>(p, (int*)part, a.ids, a.T * a.k, a.k, a.E, lane, wave);
  const int rt = MANY ? uniform(p.rt) : 1;
  if (rt == 1) gate_up<FMT, W4, RAGGED, 1>(a, h, p, part, lane, wave);
  if constexpr (MANY) {
    if (rt == 2) gate_up<FMT, W4, RAGGED, 2>(a, h, p, part, lane, wave);
    if constexpr (!W4)
      if (rt == 4) gate_up<FMT, W4, RAGGED, 4>(a, h, p, part, lane, wave);
  }
  if (blockIdx.x == 0) {
    const int total = uniform(p.total), nsegs = uniform(p.nsegs);
    if (threadIdx.x == 0) {
      plan->nsegs = nsegs;
      plan->subtiles = rt;
    }
    for (int i = threadIdx.x; i <= nsegs; i += kMoeThreads) plan->seg[i] = p.seg[i];
    for (int i = threadIdx.x; i < total; i += kMoeThreads) {
      const int e = p.eid[i], w = p.sl[i];
      // a token that names an expert twice has neighbouring rows in its run:
      // numbered, so that they add to the token's sum one after the other
      int nth = 0;
      while (nth < i && p.eid[i - nth - 1] == e && token_of(p.sl[i - nth - 1]) == token_of(w)) ++nth;
      plan->expert[i] = e;
      plan->slot[i] = w | nth << 18;
      plan->weight[i] = a.wt[slot_of(w)];
    }
  }
}

// ------------------------------------------------------------------------
// QUANT: h comes as bf16 and is quantized here, all rows into LDS, by every
// workgroup (launches with few rows; skipped slots' rows, never written, are
// not read back); else as codes and scales.
constexpr int kAhead = 4;

// NT: 16-row weight tiles that make up the workgroup's R output features (R a
// multiple of 4, the last tile partly empty), so that H / R workgroups can
// match the CUs.
template <int FMT, bool W4, int RT, bool QUANT, int NT>
__device__ __forceinline__ void down(const MoeArgs& a, const uint16_t* h, const uint8_t* hq,
                                     const void* hs, const SortedSlots& p, const float* swt,
                                     float* mine, uint8_t* xl, const uint4* hv, int R, int lane,
                                     int wave) {
  constexpr int U = W4 ? 2 : 1;        // K blocks of an item, as above
  constexpr int D = QUANT ? (NT == 2 ? 3 : 6) : RT == 1 ? 4 : RT == 2 && !W4 ? 3 : 2;
  constexpr int SB = FMT == 0 ? 4 : 1;
  const int l16 = lane & 15, g4 = lane >> 4;
  const int T = a.T;
  const int64_t N = a.H, K = a.I, n0 = (int64_t)blockIdx.x * R;
  const int KB = (int)(K / 128), KI = (KB + U - 1) / U;
  constexpr bool CHUNK = W4;           // K is a multiple of 128
  // scale chunks; QUANT: codes of the sorted rows, then their scales; else 2
  // KB RT a wave
  uint32_t* chunks = (uint32_t*)xl + wave * NT * kChunkDwords;
  if (CHUNK) xl += kMoeWaves * NT * kChunkDwords * 4;
  const int stride = (int)K + 16;      // 16: rows start in different banks
  float* xs = (float*)(xl + (QUANT ? (int64_t)T * a.k * stride : 0));
  uint8_t* xbuf = xl + wave * 2048 * RT;

  const int64_t items = (int64_t)uniform(p.nsegs) * KI;
  const int64_t it0 = items * wave / kMoeWaves;
  const int cnt = uniform((int)(items * (wave + 1) / kMoeWaves - it0));
  const int NB = (int)((N + 127) / 128), nrows = uniform((int)min((int64_t)R, N - n0));
  const __amdgpu_buffer_rsrc_t rows = row_rsrc(hq, (uint32_t)(T * a.k * K));
  const __amdgpu_buffer_rsrc_t rscales = row_rsrc(hs, (uint32_t)(T * a.k * KB * SB));
  // two cursors over the wave's items: loads, and products behind them
  int lseg = uniform((int)(it0 / KI)), lki = uniform((int)(it0 - (int64_t)lseg * KI)), left = cnt;
  int pseg = lseg, pki = lki;
  uint32_t xo[2 * RT], so[RT];         // the segment's rows; no row: past the buffers
  WTile<W4, false> wt[NT];
  __amdgpu_buffer_rsrc_t sw;
  uint32_t swo[NT];                    // this lane's four outputs' row of block scales
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    wt[j].init(K, lane);
    swo[j] = (uint32_t)(((n0 + 16 * j + 4 * g4) / 128 - n0 / 128) * KB) * SB;
  }
  auto aim = [&]() {
    const int r0 = uniform(p.seg[lseg]), r1 = uniform(p.seg[lseg + 1]);
    const int e = uniform(p.eid[r0]);
#pragma unroll
    for (int j = 0; j < NT; ++j)
      wt[j].aim(a.w2, a.s2, (int64_t)e * N + n0 + 16 * j, max(0, min(16, nrows - 16 * j)));
    if (!W4)
      sw = row_rsrc((const uint8_t*)a.s2 + ((int64_t)e * NB + n0 / 128) * KB * SB,
                    min(2, NB - (int)(n0 / 128)) * KB * SB);
    if (!QUANT) {
#pragma unroll
      for (int r = 0; r < 2 * RT; ++r) {
        const int i = r0 + 8 * r + (lane >> 3);
        xo[r] = i < r1 ? slot_of(p.sl[i]) * (uint32_t)K + (lane & 7) * 16 : kOOB;
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const int i = r0 + 16 * r + l16;
        so[r] = g4 == 0 && i < r1 ? slot_of(p.sl[i]) * (uint32_t)KB * SB : kOOB;
      }
    }
  };
  struct Item {
    WFrag<W4> w[NT][U];
    XFrag x[QUANT ? 1 : U][QUANT ? 1 : RT];
    uint32_t sx[U][RT], sw[NT];
  } ring[D];
  auto next = [&](Item& f) {
    // past the share, or the row: nothing (2^30 is past every buffer of rows)
    const bool in = left > 0;
    const int kb = in ? lki * U : KB;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int q = 0; q < U; ++q) f.w[j][q] = wt[j].load(kb + q);
    if constexpr (!QUANT) {
#pragma unroll
      for (int q = 0; q < U; ++q) {
        const uint32_t k = kb + q < KB ? (uint32_t)(kb + q) * 128 : 0x40000000u;
        const uint32_t sq = kb + q < KB ? (uint32_t)(kb + q) * SB : 0x40000000u;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          f.x[q][r].c[0] = ld_buf16(rows, xo[2 * r] + k);
          f.x[q][r].c[1] = ld_buf16(rows, xo[2 * r + 1] + k);
          if (FMT == 0) f.sx[q][r] = __builtin_amdgcn_raw_buffer_load_b32(rscales, so[r] + sq, 0, 0);
          else f.sx[q][r] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(rscales, so[r] + sq, 0, 0);
        }
      }
    }
    if constexpr (!W4) {
      const uint32_t sk = in ? (uint32_t)kb * SB : 0x40000000u;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (FMT == 0) f.sw[j] = __builtin_amdgcn_raw_buffer_load_b32(sw, swo[j] + sk, 0, 0);
        else f.sw[j] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(sw, swo[j] + sk, 0, 0);
      }
    }
    if (--left > 0 && ++lki == KI) {
      lki = 0;
      ++lseg;
      aim();
    }
  };
  // scale chunks: loaded one ahead of the products
  ScaleChunk c4[NT];
  int cseg = pseg, ckb = pki * U & ~(kChunk - 1), cleft = (cnt + pki) * U - ckb;
  auto next_chunk = [&]() {
    if (cleft <= 0) return;
    const int64_t row = (int64_t)uniform(p.eid[uniform(p.seg[cseg])]) * N + n0;
#pragma unroll
    for (int j = 0; j < NT; ++j)
      c4[j].load(a.s2, row + 16 * j, max(0, min(16, nrows - 16 * j)), K, ckb, lane);
    cleft -= min(kChunk, KI * U - ckb);
    ckb += kChunk;
    if (ckb >= KB) {
      ckb = 0;
      ++cseg;
    }
  };
  if (cnt > 0) {
    if (CHUNK) next_chunk();
    aim();
#pragma unroll
    for (int d = 0; d < D; ++d) next(ring[d]);
  }
  if constexpr (QUANT) {
    // sixteen lanes hold a group, eight values each
    const int C = KB * 16, all = T * a.k * C;    // 8-value chunks of all slots' rows
    for (int q0 = threadIdx.x, u = 0; q0 - (int)threadIdx.x < all; q0 += kMoeThreads, ++u) {
      const int i = q0 / C, c = q0 - i * C;
      const bool ok = q0 < all;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (u < kAhead) v = u == 0 ? hv[0] : u == 1 ? hv[1] : u == 2 ? hv[2] : hv[3];
      else if (ok) v = *(const uint4*)(h + (int64_t)q0 * 8);
      const Unpacked f = unpack8(v);
      float amax = amax8(f);
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor(amax, o, 16));
      float s = 0.f;
      int x = 0;
      const uint2 codes = encode8<FMT>(f, amax, &s, &x);
      if (ok) {
        *(uint2*)(xl + i * stride + c * 8) = codes;
        if ((c & 15) == 0) xs[i * KB + c / 16] = FMT == 0 ? s : e8m0_f32((uint32_t)(x + 127));
      }
    }
    wait_vmcnt<0>();                   // nothing new: these loads came after the weights
    __syncthreads();
  }
  if (cnt > 0) {
    const uint8_t* px[RT];             // QUANT: the segment's rows in LDS
    const float* ps[RT];
    auto aim_products = [&]() {
      const int r0 = p.seg[pseg], r1 = p.seg[pseg + 1];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const int i = slot_of(p.sl[min(r0 + 16 * r + l16, r1 - 1)]);   // past the rows: not added
        px[r] = xl + i * stride;
        ps[r] = xs + i * KB;
      }
    };
    if (QUANT) aim_products();
    v4f acc[RT][NT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[r][j] = v4f{0.f, 0.f, 0.f, 0.f};
    int prows = uniform(p.seg[pseg + 1] - p.seg[pseg]);
    bool fresh = true;                 // the products enter a chunk
    for (int i0 = 0; i0 < cnt; i0 += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (i0 + d < cnt) {
          if (CHUNK && fresh) {
#pragma unroll
            for (int j = 0; j < NT; ++j) c4[j].store(chunks + j * kChunkDwords, lane);
            next_chunk();
          }
          float cw[NT];
#pragma unroll
          for (int j = 0; j < NT; ++j) cw[j] = W4 ? 1.f : scale_value<FMT>(ring[d].sw[j]);
#pragma unroll
          for (int q = 0; q < U; ++q) {
            if constexpr (!QUANT) {
#pragma unroll
              for (int r = 0; r < RT; ++r) x_to_lds(xbuf + r * 2048, ring[d].x[q][r], lane);
            }
            const uint32_t* ch = chunks + l16 * kChunkRow + (pki * U & (kChunk - 1)) + q;
            BFrag bw[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) bw[j] = wt[j].bf16(ring[d].w[j][q], ch + j * kChunkDwords);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
              if (r > 0 && prows <= 16 * r) break;
              BFrag bx;
              float sx;
              if constexpr (QUANT) {
                const int kb = min(pki * U + q, KB - 1);     // past the row: times zeros
                const uint8_t* x = px[r] + kb * 128;
                bx = x_bf16(*(const uint4*)(x + (W4 ? 32 * g4 : 16 * g4)),
                            *(const uint4*)(x + (W4 ? 32 * g4 + 16 : 64 + 16 * g4)));
                sx = ps[r][kb];
              } else {
                bx = x_from_lds<W4>(xbuf + r * 2048, lane);
                sx = scale_value<FMT>(spread16(ring[d].sx[q][r], l16));
              }
#pragma unroll
              for (int j = 0; j < NT; ++j) acc[r][j] = moe_step(acc[r][j], bw[j], bx, sx * cw[j]);
            }
          }
        }
        next(ring[d]);
        const bool last = i0 + d + 1 == cnt;
        if (i0 + d < cnt && (++pki == KI || last)) {         // the segment's end, here
          const int r0 = p.seg[pseg], r1 = p.seg[pseg + 1];
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            // lane: outputs n0 + 16 j + 4 g4 .. + 3 of row l16
            const int at = r0 + 16 * r + l16;
            const int v = at < r1 ? p.sl[at] : -1;
            const float c = at < r1 ? swt[at] : 0.f;
            const int nth = nth_of(v);
            float* to = mine + (v < 0 ? 0 : token_of(v)) * R + 4 * g4;
            for (int q = 0; __ballot(nth >= q) != 0; ++q) {
#pragma unroll
              for (int j = 0; j < NT; ++j) {
                if (nth == q && 16 * j + 4 * g4 < R) {
                  v4f o = *(v4f*)(to + 16 * j);
#pragma unroll
                  for (int x = 0; x < 4; ++x) o[x] = fmaf(c, acc[r][j][x], o[x]);
                  *(v4f*)(to + 16 * j) = o;
                }
              }
              __builtin_amdgcn_wave_barrier();
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[r][j] = v4f{0.f, 0.f, 0.f, 0.f};
          }
          if (!last) {
            pki = 0;
            ++pseg;
            prows = uniform(p.seg[pseg + 1] - p.seg[pseg]);
            if (QUANT) aim_products();
          }
        }
        fresh = (pki * U & (kChunk - 1)) == 0;
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
}

template <int FMT, bool W4, bool QUANT, int NT, bool MANY>
__global__ __launch_bounds__(kMoeThreads) void moe_down_kernel(MoeArgs a, const uint16_t* h,
                                                               const uint8_t* hq, const void* hs,
                                                               const MoePlan* plan, int R) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];   // sums, then the rows of h
  __shared__ SortedSlots p;
  __shared__ float swt[kMoeMaxSlots];  // the sorted slots' weights
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int T = a.T;
  const int64_t N = a.H, n0 = (int64_t)blockIdx.x * R;
  float* sums = (float*)lds;           // [waves][T][R]
  uint8_t* xl = lds + kMoeWaves * T * R * 4;

  // everything that does not wait for the counts goes out at once
  const int S = T * a.k;
  uint4 hv[kAhead];                    // QUANT: this lane's first chunks of h
  if constexpr (QUANT) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t q = threadIdx.x + u * kMoeThreads;
      hv[u] = q < S * (a.I / 8) ? *(const uint4*)(h + q * 8) : make_uint4(0, 0, 0, 0);
    }
  }
  const int nsegs = plan->nsegs, subs = plan->subtiles;
  float* mine = sums + wave * T * R;
  for (int i = lane * 4; i < T * R; i += 256) *(float4*)(mine + i) = make_float4(0, 0, 0, 0);
  for (int i = threadIdx.x; i < S; i += kMoeThreads) {
    const int e = plan->expert[i], w = plan->slot[i];
    const float c = plan->weight[i];
    const uint16_t g = plan->seg[i];
    p.eid[i] = e;
    p.sl[i] = w;
    swt[i] = c;
    p.seg[i] = g;
  }
  if (threadIdx.x == 0) {
    p.seg[S] = plan->seg[S];
    p.nsegs = nsegs;
    p.rt = subs;
  }
  __syncthreads();
  const int rt = MANY ? uniform(p.rt) : 1;
  if (rt == 1) down<FMT, W4, 1, QUANT, NT>(a, h, hq, hs, p, swt, mine, xl, hv, R, lane, wave);
  if constexpr (MANY) {
    if (rt == 2) down<FMT, W4, 2, QUANT, NT>(a, h, hq, hs, p, swt, mine, xl, hv, R, lane, wave);
    if constexpr (!W4)
      if (rt == 4) down<FMT, W4, 4, QUANT, NT>(a, h, hq, hs, p, swt, mine, xl, hv, R, lane, wave);
  }
  __syncthreads();
  const int Q = R / 4;
  for (int i = threadIdx.x; i < T * Q; i += kMoeThreads) {
    const int t = i / Q, c = 4 * (i - t * Q);
    if (n0 + c >= N) continue;
    v4f v = *(const v4f*)(sums + t * R + c);
#pragma unroll
    for (int w = 1; w < kMoeWaves; ++w) v += *(const v4f*)(sums + (w * T + t) * R + c);
    const int64_t o = (int64_t)t * N + n0 + c;
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
  size_t h, hq, hs, bytes;
};
inline MoeWorkspace moe_layout(int64_t S, int64_t I) {
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  MoeWorkspace w;
  w.h = up(sizeof(MoePlan));
  w.hq = w.h + up((size_t)S * I * 2);
  w.hs = w.hq + up((size_t)S * I);
  w.bytes = w.hs + up((size_t)S * ((I + 127) / 128) * 4);
  return w;
}

constexpr int kMoeGateUpGroups = 256;      // one workgroup per CU
// h in LDS, quantized by the down launch up to here: its encoding, once per
// workgroup, costs less than a launch (1 x 8 of 7168, 2048: 27.1 us against
// 4.6 + 24.1; 43 KB at 5 x 6 of 2064, 1408: 29.0 against 4.8 + 25.0; above it
// 51 KB at 3 x 8 of 7168, 2048: 58.8 against 4.8 + 52.2; 68 KB at 4 x 8: 96
// against 4.8 + 70.8)
constexpr int64_t kMoeQuantBytes = 49152;
constexpr size_t kMoeDownBytes = 163840 - sizeof(SortedSlots) - kMoeMaxSlots * 4;

// Output features of a down workgroup: a multiple of 4 from 8 to 32 (to 16
// where the sums of more would not fit the LDS) with the least to do on the
// busiest of 256 CUs, the larger where that is equal (7168 wide: 28 against
// 16, 16 tokens x 8 of 256 256 us against 317; 8 and 12 read partly empty
// tiles: 435).
inline int moe_down_rows(int64_t H, int T) {
  int best = 0;
  int64_t least = 0;
  for (int r = T > 64 ? 16 : 32; r >= 8; r -= 4) {
    const int64_t groups = (H + r - 1) / r, cost = (groups + 255) / 256 * r;
    if (best == 0 || cost < least) {
      best = r;
      least = cost;
    }
  }
  return best;
}

// LDS of a down workgroup: the sums, and the scale chunks of MXFP4 weights
inline size_t moe_sums_bytes(const MoeArgs& a, int R) { return (size_t)kMoeWaves * a.T * R * 4; }
inline size_t moe_chunk_bytes(const MoeArgs& a, int R) {
  return a.w4 ? (size_t)kMoeWaves * (R > 16 ? 2 : 1) * kChunkDwords * 4 : 0;
}

// lds: bytes beside the sums
template <int FMT, bool W4, bool QUANT, bool MANY>
hipError_t launch_moe_down(const MoeArgs& a, const uint16_t* h, const uint8_t* hq, const void* hs,
                           const MoePlan* plan, int R, size_t lds, hipStream_t s) {
  const dim3 grid((unsigned)((a.H + R - 1) / R));
  lds += moe_sums_bytes(a, R);
  if (R <= 16)
    hipLaunchKernelGGL((moe_down_kernel<FMT, W4, QUANT, 1, MANY>), grid, dim3(kMoeThreads), lds, s,
                       a, h, hq, hs, plan, R);
  else
    hipLaunchKernelGGL((moe_down_kernel<FMT, W4, QUANT, 2, MANY>), grid, dim3(kMoeThreads), lds, s,
                       a, h, hq, hs, plan, R);
  return hipGetLastError();
}

template <int FMT, bool W4, bool MANY>
hipError_t launch_moe(const MoeArgs& a, hipStream_t s) {
  const int64_t S = (int64_t)a.T * a.k;
  const MoeWorkspace w = moe_layout(S, a.I);
  uint8_t* ws = (uint8_t*)a.workspace;
  MoePlan* plan = (MoePlan*)ws;
  uint16_t* h = (uint16_t*)(ws + w.h);
  if (W4 && a.H % 128 != 0)
    hipLaunchKernelGGL((moe_gate_up_kernel<FMT, W4, W4, MANY>), dim3(kMoeGateUpGroups),
                       dim3(kMoeThreads), 0, s, a, h, plan);
  else
    hipLaunchKernelGGL((moe_gate_up_kernel<FMT, W4, false, MANY>), dim3(kMoeGateUpGroups),
                       dim3(kMoeThreads), 0, s, a, h, plan);
  hipError_t r = hipGetLastError();
  if (r != hipSuccess) return r;
  const int64_t codes = S * (a.I + 16 + a.I / 128 * 4);
  const int R = moe_down_rows(a.H, a.T);
  const size_t chunks = moe_chunk_bytes(a, R);
  if (codes <= kMoeQuantBytes && (size_t)codes + chunks + moe_sums_bytes(a, R) <= kMoeDownBytes) {
    // FP8, up to 16 tokens: one row tile instead of two nearly full ones while
    // all workgroups are resident, two to a CU: one's encoding of h runs beside
    // the other's stream (1 token x 8, widths 7168 / 8192 27.1 / 31 us against
    // 25.2 / 28, 16 tokens of one expert each 34.3 against 34.2; alike at 6144,
    // R = 24, and slower at 5120, R = 20, 18 against 19, and with MXFP4, 7168 /
    // 8192 19.2 / 20.8 against 22.0 / 22.6).  The kernel for more tokens has
    // registers for one workgroup per CU: at 7168 two rounds of R = 16 take
    // 56.3 us for 20 tokens and 61.9 for 32, one round of R = 28 44.9 and 48.7
    const int RQ = !W4 && !MANY && R > 24 && a.H <= 512 * 16 ? 16 : R;
    return launch_moe_down<FMT, W4, true, MANY>(a, h, nullptr, nullptr, plan, RQ, codes + chunks, s);
  }
  r = launch_quant_act(h, S, a.I, a.I, FMT, ws + w.hq, ws + w.hs, s);
  if (r != hipSuccess) return r;
  return launch_moe_down<FMT, W4, false, MANY>(a, h, ws + w.hq, ws + w.hs, plan, R,
                                               // the waves' subtiles: 1, 2 or 4 (MXFP4: 2)
                                               chunks + kMoeWaves * 2048 * (MANY ? (W4 ? 2 : 4) : 1), s);
}

template <int FMT, bool W4>
hipError_t launch_moe_many(const MoeArgs& a, hipStream_t s) {
  return a.T > 16 ? launch_moe<FMT, W4, true>(a, s) : launch_moe<FMT, W4, false>(a, s);
}

}  // namespace detail
using namespace detail;

size_t moe_decode_workspace_bytes(int64_t S, int64_t I) { return moe_layout(S, I).bytes; }

hipError_t launch_moe_decode(const MoeArgs& a, hipStream_t s) {
  if (a.w4) return a.fmt == 0 ? launch_moe_many<0, true>(a, s) : launch_moe_many<1, true>(a, s);
  return a.fmt == 0 ? launch_moe_many<0, false>(a, s) : launch_moe_many<1, false>(a, s);
}

}  // namespace bsfp8
