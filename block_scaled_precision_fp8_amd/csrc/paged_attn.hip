// Attention of new tokens over a paged cache of keys and values.
//
//   y = sum_j e^(s_j) v_j / sum_j e^(s_j),   s_j = scale q . k_j
//
// over the keys that a row (a token's query head) sees; 0 where it sees none.
//
// Arithmetic.  One pass over the keys in tiles of 32 with a reference
// exponent r per row: p_j = 2^(s_j log2 e - r), w_j = p_j (v's scale), sums of
// p_j in fp32, and sums of w_j (v's codes) on the matrix cores.  r is raised to
// the row's largest score only when some p_j passes 2^10, which the first tile
// does and few others: the sums are rescaled then, and not at every tile.  It
// goes by the scores alone: with the values' scales in it, sums of p_j over keys
// whose scales differ by more than fp32's range would be lost, and a scale of 0
// has no exponent.
// E4M3 codes, keys' and values', are exact in bf16.  w_j is the sum of two bf16
// numbers (2^-16 of it lost, whatever its size), and the second product is
// taken for both: one bf16 number would lose as much as rounding the output
// does, one of fp16 every weight that is small beside a heavier key's, which an
// element to which that key's value adds nothing consists of (a value row of
// zeros has the scale 1).  The second half of the products costs few rows
// nothing (64 x 8192 112 us, 113 with it), many rows a quarter (2 x 2048 over
// 6000 keys 387 us, 473).
//
// Layout.  The score tile is computed transposed, keys x rows: a lane then
// holds 8 keys of one row, which is what the second product wants of it as an
// operand once the values' order of summation is that same order, and a row's
// statistics are exchanged between four lanes.
// The values' transposition is a byte permutation of what a lane itself loads
// (8 keys x D/16 values).  Few rows (attn_split_kernel): nothing goes through
// LDS on the way from memory to the matrix cores, bound by HBM: 64 sequences
// of up to 8192 keys (32 / 8 heads of 128, E4M3) 575 MB in 100 to 117 us, 4.9 to
// 5.8 TB/s; 131072 keys of one 277 MB in 51.5 us, 5.4; a large copy runs at
// 5.1.  Many rows (attn_rows_kernel): conversions and transpositions are shared
// through LDS, bound by issue: 2 x 2048 tokens over 6000 keys 334 GFLOP (one and a
// half times that on the matrix cores) in 473 us, 706 TFLOP/s, where launches
// follow each other, 557 us alone; a large bf16 product runs at 1415.
#include <type_traits>

#include "bsfp8_attn.h"

namespace bsfp8 {
namespace detail {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kTile = 32;              // keys of a wave's step
constexpr int kUnit = 4 * kTile;       // keys of a step of four waves that split them
constexpr float kLowest = -3.4028234663852886e38f;
constexpr float kMostP = 1024.0f;      // a larger p raises the reference exponent
constexpr float kMostSum = 8192.0f;    // the same of the sum of 8 of them
constexpr float kMostRef = 4096.0f;    // beyond: scores are rounded before the difference

__device__ __forceinline__ int clampi(int v, int lo, int hi) {
  return v < lo ? lo : (v > hi ? hi : v);
}
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// 2^(s k - ref).  One fused operation where the reference is at most kMostRef
// in size.  From there on the score is rounded first, as the reference was: of
// scores from 2^30 on the last place is a whole power of two of the weight, and
// 2^x of what the rounding took off passes fp32's range.  Rounded everywhere it
// costs 3% (2 x 2048 over 6000 keys 470 us, 483), so that such rows take the
// rare path that raises the reference at every tile instead.
template <bool ROUNDED>
__device__ __forceinline__ float weight(float s, float k, float ref) {
#pragma clang fp contract(off)
  if (!ROUNDED) return __builtin_amdgcn_exp2f(fmaf(s, k, -ref));
  const float e = s * k;
  return __builtin_amdgcn_exp2f(e - ref);
}
// What `most` may be before the raising path is taken, for a row's reference.
__device__ __forceinline__ float limit_of(float ref, float most) {
  return fabsf(ref) > kMostRef && ref != kLowest ? -1.0f : most;
}

// The maximum over the four lanes that share lane % 16.
__device__ __forceinline__ float group_max(float v) {
  u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(
      __float_as_uint(v), __float_as_uint(v), false, false));
  v = fmaxf(__uint_as_float(a.x), __uint_as_float(a.y));
  a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(
      __float_as_uint(v), __float_as_uint(v), false, false));
  return fmaxf(__uint_as_float(a.x), __uint_as_float(a.y));
}
__device__ __forceinline__ float group_sum(float v) {
  u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(
      __float_as_uint(v), __float_as_uint(v), false, false));
  v = __uint_as_float(a.x) + __uint_as_float(a.y);
  a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(
      __float_as_uint(v), __float_as_uint(v), false, false));
  return __uint_as_float(a.x) + __uint_as_float(a.y);
}
// The maximum over the 16 lanes of a row of lanes (any sign).
__device__ __forceinline__ int row16_max(int v) {
  v = max(v, (int)dpp<kXor1>((uint32_t)v));
  v = max(v, (int)dpp<kXor2>((uint32_t)v));
  v = max(v, (int)dpp<kMirror8>((uint32_t)v));
  return max(v, (int)dpp<kMirror16>((uint32_t)v));
}

// ------------------------------------------------- sequences, rows, blocks

struct Seq { int q0, n, len; };        // first token, tokens, own cached tokens

__device__ __forceinline__ int len_of(const AttnArgs& a, int b) {
  const int64_t room = (int64_t)a.max_pages << a.log2_page;
  const int len = a.kv_len[b];
  return len < 0 ? 0 : (len > room ? (int)room : len);
}
__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int b, int len) {
  Seq s;
  s.q0 = b;
  s.n = 1;
  if (a.q_start) {
    s.q0 = clampi(a.q_start[b], 0, a.T);
    s.n = clampi(a.q_start[b + 1], s.q0, a.T) - s.q0;
  }
  s.len = len;
  return s;
}
__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int b) { return seq_of(a, b, len_of(a, b)); }

// Own keys that the sequence's first and last token bound: [first, len).
__device__ __forceinline__ int first_key(const AttnArgs& a, const Seq& s) {
  if (!a.window) return 0;
  const int64_t lo = (int64_t)s.len - s.n - a.window + 1;
  return lo > 0 ? (int)lo : 0;
}
__device__ __forceinline__ int units_of(const AttnArgs& a, const Seq& s) {
  if (s.n == 0 || s.len == 0) return 0;
  return (s.len + kUnit - 1) / kUnit - first_key(a, s) / kUnit;
}
// Number of a sequence's first block among all, with gaps: a bound of what
// the sequences before it have.
__device__ __forceinline__ int block_base(const AttnArgs& a, int b, int q0, int rows) {
  return (int)((int64_t)q0 * a.G / rows) + b;
}

// The sequence of a token, -1 for none.  One lane's search.
__device__ __forceinline__ int seq_of_token(const AttnArgs& a, int t) {
  if (!a.q_start) return t;
  int lo = 0, hi = a.B;                // q_start[lo] <= t < q_start[hi], if in any
  if (t < a.q_start[0] || t >= a.q_start[a.B]) return -1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.q_start[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// What a row block works on: rows row0 .. row0 + rows of the sequence (or,
// of the prefix, of all tokens), key head h, keys of a table.
struct Block {
  int q0;                    // token of row 0
  int row0, rows;
  int h;
  const int32_t* table;
  int keys;                  // of the table
  int pre;                   // 1: the prefix's keys
  int n, len;                // the sequence's (own blocks)
};

// The keys [lo, hi) of the block's table that its row r sees.
__device__ __forceinline__ void row_range(const AttnArgs& a, const Block& b, int r, int* lo, int* hi) {
  const int i = (b.row0 + r) / a.G;
  *lo = *hi = 0;
  if (!b.pre) {
    const int pos = b.len - b.n + i;               // among the own keys
    *hi = clampi(pos + 1, 0, b.keys);
    if (a.window) *lo = (int)max((int64_t)pos - a.window + 1, (int64_t)0);
  } else {
    const int s = seq_of_token(a, i);
    if (s < 0) return;
    const Seq sq = seq_of(a, s);
    const int64_t pos = (int64_t)a.prefix_len + sq.len - sq.n + (i - sq.q0);
    *hi = (int)min(max(pos + 1, (int64_t)0), (int64_t)b.keys);
    if (a.window) *lo = (int)min(max(pos - a.window + 1, (int64_t)0), (int64_t)b.keys);
  }
}

// ----------------------------------------------------------- a wave's rows

template <int KV, int D, bool STREAM = false>
struct Wave {
  static constexpr bool F8 = KV != kKvBf16;
  static constexpr int ES = F8 ? 1 : 2;            // bytes of a cached value
  static constexpr int KQ = D * 16 * ES / 1024;    // 16-byte pieces of a lane's 16-key part
  static constexpr int DPL = D / 16;               // values of a key that a lane holds
  static constexpr int VW = DPL * ES / 4;          // dwords of them
  static constexpr int AUX = STREAM ? 2 : 0;       // non-temporal

  struct Raw {
    uint4 k[2][KQ];
    uint32_t v[8][VW];
    float ks[8], vs[8];
    uint32_t ks8[2], vs8[2]; // E8M0 bytes of four keys each
    int id[2];               // page ids, -1: none
  };

  const AttnArgs& a;
  bf16x8 q[D / 32];
  v4f o[DPL];
  float ref, sum;
  float most_p;              // a larger p, and the reference is looked at
  int lo, hi;                // the lane's row's visible keys
  int lo_most, lo_least, hi_least, hi_most;        // over the wave's rows
  int lane, n, g;

  __device__ __forceinline__ explicit Wave(const AttnArgs& args) : a(args) {
    lane = threadIdx.x & 63;
    n = lane & 15;
    g = lane >> 4;
  }

  // Query and visible keys of row n of the block.
  __device__ __forceinline__ void begin(const Block& b) {
    const bool live = n < b.rows;
    const int i = live ? (b.row0 + n) / a.G : 0;
    const int head = b.h * a.G + (b.row0 + n - i * a.G);
    lo = hi = 0;
    if (live) row_range(a, b, n, &lo, &hi);
    const uint16_t* src = a.q + (int64_t)(b.q0 + i) * a.ldq + (int64_t)head * D;
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
      const int d = F8 ? 64 * (s / 2) + 16 * g + 8 * (s % 2) : 32 * s + 8 * g;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (live) v = *(const uint4*)(src + d);
      q[s] = __builtin_bit_cast(bf16x8, v);
    }
#pragma unroll
    for (int t = 0; t < DPL; ++t) o[t] = v4f{0, 0, 0, 0};
    ref = kLowest;
    sum = 0.0f;
    most_p = kMostP;
    lo_most = uniform(row16_max(lo));
    lo_least = -uniform(row16_max(live ? -lo : -0x7fffffff));
    hi_least = -uniform(row16_max(live ? -hi : -0x7fffffff));
    hi_most = uniform(row16_max(hi));
  }

  // Page ids of the 32 tiles tile0, tile0 + step, ..: lane 2 i + s has that
  // of keys 16 s .. of the i-th one.
  __device__ __forceinline__ int page_ids(const Block& b, int tile0, int step) const {
    const int64_t key = ((int64_t)tile0 + (int64_t)(lane >> 1) * step) * kTile + 16 * (lane & 1);
    int id = -1;
    if (key < b.keys) {
      id = b.table[key >> a.log2_page];
      if (id < 0 || id >= a.num_pages) id = -1;
    }
    return id;
  }

  __device__ __forceinline__ void load(const Block& b, int tile, int id0, int id1, Raw& x) const {
    const int in_page = (1 << a.log2_page) - 1;
    int64_t row[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int id = s ? id1 : id0;
      x.id[s] = id;
      // keys without a page: those of page 0 are loaded and not used
      row[s] = (((int64_t)(id < 0 ? 0 : id) * a.Hkv + b.h) << a.log2_page) +
               ((tile * kTile + 16 * s) & in_page);
      const auto kr = make_rsrc(a.kc + row[s] * (D * ES), 16 * D * ES);
#pragma unroll
      for (int i = 0; i < KQ; ++i)
        x.k[s][i] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
            kr, n * (D * ES) + 16 * g + 64 * i, 0, AUX));
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if constexpr (KV == kKvFloat) {
        const float4 e = __builtin_bit_cast(float4, __builtin_amdgcn_raw_buffer_load_b128(
            make_rsrc(a.ks + 4 * row[s], 64), 16 * g, 0, 0));
        const float4 f = __builtin_bit_cast(float4, __builtin_amdgcn_raw_buffer_load_b128(
            make_rsrc(a.vs + 4 * row[s], 64), 16 * g, 0, 0));
        x.ks[4 * s] = e.x; x.ks[4 * s + 1] = e.y; x.ks[4 * s + 2] = e.z; x.ks[4 * s + 3] = e.w;
        x.vs[4 * s] = f.x; x.vs[4 * s + 1] = f.y; x.vs[4 * s + 2] = f.z; x.vs[4 * s + 3] = f.w;
      } else if constexpr (KV == kKvUe8m0) {
        x.ks8[s] = __builtin_amdgcn_raw_buffer_load_b32(make_rsrc(a.ks + row[s], 16), 4 * g, 0, 0);
        x.vs8[s] = __builtin_amdgcn_raw_buffer_load_b32(make_rsrc(a.vs + row[s], 16), 4 * g, 0, 0);
      }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const auto vr = make_rsrc(a.vc + row[s] * (D * ES), 16 * D * ES);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = (4 * g + j) * (D * ES) + n * (DPL * ES);
        uint32_t* v = x.v[4 * s + j];
        if constexpr (VW == 1) {
          v[0] = __builtin_amdgcn_raw_buffer_load_b32(vr, p, 0, AUX);
        } else if constexpr (VW == 2) {
          const u32x2 w = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(vr, p, 0, AUX));
          v[0] = w.x;
          v[1] = w.y;
        } else {
#pragma unroll
          for (int i = 0; i < VW; i += 4) {
            const uint4 w = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(vr, p + 4 * i, 0, AUX));
            v[i] = w.x;
            v[i + 1] = w.y;
            v[i + 2] = w.z;
            v[i + 3] = w.w;
          }
        }
      }
    }
  }

  // The bf16 numbers of a dword's lower or upper two codes.
  template <bool UPPER>
  __device__ __forceinline__ static uint32_t two_codes(uint32_t c) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, UPPER));
  }
  __device__ __forceinline__ static bf16x8 key_operand(uint2 c) {
    return __builtin_bit_cast(bf16x8, u32x4{two_codes<false>(c.x), two_codes<true>(c.x),
                                            two_codes<false>(c.y), two_codes<true>(c.y)});
  }

  // A code or value that is not finite: its mark in each byte or half.
  __device__ __forceinline__ static uint32_t odd_marks(uint32_t v) {
    if (F8) return ((v & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
    return ((v & 0x7fff7fffu) + 0x00800080u) & 0x80008000u;
  }

  // Values that are not finite in a tile that some rows see only part of:
  // they are taken out of the tile (0 w would not be 0) and added, one by one,
  // to the rows that see them.
  __device__ __forceinline__ void odd_values(const Block& b, int tile, Raw& x,
                                             const float (&w)[8], uint32_t seen) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        const uint32_t m = odd_marks(x.v[j][i]);
        x.v[j][i] &= ~((m >> (F8 ? 7 : 15)) * (F8 ? 0xffu : 0xffffu));
      }
    int g = this->g, n = this->n;      // not to be prepared before it is known that they are needed
    asm volatile("" : "+v"(g), "+v"(n));
    const int in_page = (1 << a.log2_page) - 1;
    for (int k = 0; k < kTile; ++k) {
      const int s = k >> 4, j = (k & 3) + 4 * s, from = ((k >> 2) & 3) * 16 + n;
      const int id = s ? x.id[1] : x.id[0];
      if (id < 0) continue;
      const int64_t row = (((int64_t)id * a.Hkv + b.h) << a.log2_page) + ((tile * kTile + k) & in_page);
      float mine = w[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) mine = i == j ? w[i] : mine;
      const float wk = __shfl(mine, from);
      const bool sees = (__shfl((int)seen, from) >> j) & 1;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < DPL; ++t) {
          const int64_t at = row * D + DPL * (4 * g + i) + t;
          float val = 0.0f;
          bool odd;
          if (F8) {
            odd = (a.vc[at] & 0x7fu) == 0x7fu;
            if (odd) val = __uint_as_float(0x7fc00000u);
          } else {
            const uint32_t bits = ((const uint16_t*)a.vc)[at];
            odd = (bits & 0x7f80u) == 0x7f80u;
            val = __uint_as_float(bits << 16);
          }
          if (sees && odd) o[t][i] += wk * val;
        }
    }
  }

  __device__ __forceinline__ void tile(const Block& b, int tile, Raw& x) {
    const int key0 = tile * kTile;
    const bool whole = uniform(x.id[0] >= 0 && x.id[1] >= 0 && key0 >= lo_most && key0 + kTile <= hi_least);

    v4f s[2] = {v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}};
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        bf16x8 k;
        if constexpr (F8) {
          const uint4 c = x.k[h][i / 2];
          k = key_operand(i % 2 ? make_uint2(c.z, c.w) : make_uint2(c.x, c.y));
        } else {
          k = __builtin_bit_cast(bf16x8, x.k[h][i]);
        }
        s[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[i], s[h], 0, 0, 0);
      }

    if constexpr (KV == kKvUe8m0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x.ks[j] = e8m0_f32((x.ks8[j >> 2] >> (8 * (j & 3))) & 255u);
        x.vs[j] = e8m0_f32((x.vs8[j >> 2] >> (8 * (j & 3))) & 255u);
      }
    }
    float ksl[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) ksl[j] = F8 ? x.ks[j] * a.scale_log2 : a.scale_log2;

    uint32_t seen = 0xffu;
    if (!whole) {
      int g = this->g;                 // as above
      asm volatile("" : "+v"(g));
      seen = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int key = key0 + 16 * (j >> 2) + 4 * g + (j & 3);
        const bool ok = x.id[j >> 2] >= 0 && key >= lo && key < hi;
        seen |= (uint32_t)ok << j;
      }
    }
    float p[8];
    auto weigh = [&](auto rounded) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        p[j] = weight<decltype(rounded)::value>(s[j >> 2][j & 3], ksl[j], ref);
      if (!whole) {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = (seen >> j) & 1 ? p[j] : 0.0f;
      }
    };
    weigh(std::false_type());
    float most = p[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) most = fmaxf(most, p[j]);
    if (__any(!(most <= most_p))) {
      float top = kLowest;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float e = s[j >> 2][j & 3] * ksl[j];
        if ((seen >> j) & 1) top = fmaxf(top, e);
      }
      top = fmaxf(ref, group_max(top));
      const float down = __builtin_amdgcn_exp2f(ref - top);
      ref = top;
      sum *= down;
#pragma unroll
      for (int t = 0; t < DPL; ++t) o[t] *= down;
      most_p = limit_of(top, kMostP);
      weigh(std::true_type());
    }
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += p[j];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = F8 ? p[j] * x.vs[j] : p[j];
    // a scale that the row does not use may hold anything
    if (F8 && !whole) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = (seen >> j) & 1 ? w[j] : 0.0f;
    }

    if (!whole) {
      // keys that no row sees may hold anything
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int key = key0 + 16 * (j >> 2) + 4 * g + (j & 3);
        const bool ok = x.id[j >> 2] >= 0 && key >= lo_least && key < hi_most;
#pragma unroll
        for (int i = 0; i < VW; ++i) x.v[j][i] = ok ? x.v[j][i] : 0;
      }
      if (lo_least != lo_most || hi_least != hi_most) {
        uint32_t marks = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int i = 0; i < VW; ++i) marks |= odd_marks(x.v[j][i]);
        if (__any(marks != 0)) odd_values(b, tile, x, w, seen);
      }
    }

    bf16x8 wh, wl;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const bf16x2 c = __builtin_convertvector((f32x2{w[j], w[j + 1]}), bf16x2);
      const bf16x2 d = __builtin_convertvector((f32x2{w[j] - (float)c[0], w[j + 1] - (float)c[1]}), bf16x2);
      wh[j] = c[0];
      wh[j + 1] = c[1];
      wl[j] = d[0];
      wl[j + 1] = d[1];
    }
    // two values of a lane's eight keys, as the first and second operand's rows
    auto add_values = [&](const uint32_t (&c)[8], int t) {
      u32x4 e, f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        e[j] = __builtin_amdgcn_perm(c[2 * j + 1], c[2 * j], 0x05040100u);
        f[j] = __builtin_amdgcn_perm(c[2 * j + 1], c[2 * j], 0x07060302u);
      }
      v4f& u = o[t];
      v4f& v = o[t + 1];
      u = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, e), wh, u, 0, 0, 0);
      v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, f), wh, v, 0, 0, 0);
      u = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, e), wl, u, 0, 0, 0);
      v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, f), wl, v, 0, 0, 0);
    };
#pragma unroll
    for (int i = 0; i < VW; ++i) {
      uint32_t c[8];
      if constexpr (F8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = two_codes<false>(x.v[j][i]);
        add_values(c, 4 * i);
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = two_codes<true>(x.v[j][i]);
        add_values(c, 4 * i + 2);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = x.v[j][i];
        add_values(c, 2 * i);
      }
    }
  }

  // Tiles first, first + step, .. below end.  What hides a tile's loads is the
  // other waves: a second tile in registers costs every third wave, and code
  // that is twice as long (64 x 8192 ragged 121 us with it, 115 without; 1 x
  // 700 8.5 and 7.8).
  __device__ __forceinline__ void walk(const Block& b, int first, int end, int step) {
    // those that some row sees
    end = min(end, (hi_most + kTile - 1) / kTile);
    if (lo_least >= (first + 1) * kTile) first += (lo_least / kTile - first + step - 1) / step * step;
    if (first >= end) return;
    const int count = (end - first + step - 1) / step;
    Raw x;
    int ids = 0;
    for (int i = 0; i < count; ++i) {
      if (i % 32 == 0) ids = page_ids(b, first + i * step, step);
      const int at = 2 * (i % 32);
      load(b, first + i * step, __builtin_amdgcn_readlane(ids, at),
           __builtin_amdgcn_readlane(ids, at + 1), x);
      tile(b, first + i * step, x);
    }
    sum = group_sum(sum);
  }

  // The lane's 4 DPL values of a row: y, or a partial result.
  __device__ __forceinline__ void out_row(const Block& b, int64_t slot, bool direct) const {
    if (n >= b.rows) return;
    if (direct) {
      const int i = (b.row0 + n) / a.G;
      const int head = b.h * a.G + (b.row0 + n - i * a.G);
      const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
      uint16_t* y = a.y + ((int64_t)(b.q0 + i) * a.Hq + head) * D + 4 * DPL * g;
#pragma unroll
      for (int i4 = 0; i4 < 4; ++i4) {
        uint32_t c[DPL / 2];
#pragma unroll
        for (int t = 0; t < DPL; t += 2)
          c[t / 2] = __builtin_bit_cast(uint32_t, __builtin_convertvector(
              (f32x2{o[t][i4] * f, o[t + 1][i4] * f}), bf16x2));
        uint16_t* p = y + DPL * i4;
        if constexpr (DPL == 4) *(uint2*)p = make_uint2(c[0], c[1]);
        else
#pragma unroll
          for (int t = 0; t < DPL / 2; t += 4) *(uint4*)(p + 2 * t) = make_uint4(c[t], c[t + 1], c[t + 2], c[t + 3]);
      }
    } else {
      const int64_t at = slot * 16 + n;
      if (g == 0) a.ml[at] = make_float2(ref, sum);
      float* p = a.part + at * D + 4 * DPL * g;
#pragma unroll
      for (int i4 = 0; i4 < 4; ++i4)
#pragma unroll
        for (int t = 0; t < DPL; t += 4)
          *(float4*)(p + DPL * i4 + t) = make_float4(o[t][i4], o[t + 1][i4], o[t + 2][i4], o[t + 3][i4]);
    }
  }
};

// ------------------------------------------ few rows: four waves split keys

// All (sequence, block of 16 rows, key head) in a row, each its units of 128
// keys; every workgroup takes as many consecutive units as the others.  The
// lengths are read from the device, so that one launch shape (and one graph)
// serves them all.  The prefix, where its rows are few too, comes last, as a
// sequence of its own whose rows are all tokens'.  Lengths that differ cost
// nothing this way: 64 sequences of 130 to 8192 keys run at the rate of one of
// 131072.  A partial result's place is the workgroup's number plus the block's:
// both only grow along the units, so no two share one.
constexpr int split_resident(int kv, int D) {      // workgroups that a CU's registers hold
  return D == 256 ? (kv == kKvBf16 ? 1 : 2) : (kv == kKvBf16 && D == 128 ? 2 : 3);
}
template <int KV, int D, bool STREAM>
__global__ __launch_bounds__(256, split_resident(KV, D)) void attn_split_kernel(AttnArgs a) {
  constexpr int DPL = D / 16;
  __shared__ int before[kAttnMaxSeqs + 2], lens[kAttnMaxSeqs + 1];
  __shared__ int wave_total[4];
  __shared__ float merge[2][16][D + 4];
  __shared__ float2 merge_ml[2][16];
  const int tid = threadIdx.x, wave = uniform(tid >> 6), lane = tid & 63;
  const bool pre = a.prefix_len > 0 && !a.plan.pre_wide;
  const int items = a.B + (pre ? 1 : 0);
  const int pre_blocks = (int)(((int64_t)a.T * a.G + 15) / 16);
  const int pre_units = (a.prefix_len + kUnit - 1) / kUnit;

  int total = 0;
  for (int base = 0; base < items; base += 256) {
    const int b = base + tid;
    int v = 0, len = 0;
    if (b < a.B) {
      len = len_of(a, b);
      const Seq s = seq_of(a, b, len);
      v = units_of(a, s) * ((s.n * a.G + 15) / 16) * a.Hkv;
    } else if (b < items) {
      v = pre_units * pre_blocks * a.Hkv;
    }
    int incl = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int u = __shfl_up(incl, d);
      if (lane >= d) incl += u;
    }
    if (lane == 63) wave_total[wave] = incl;
    // sequences in another order would count rows twice, past what has a place
    if (a.q_start) {
      if (__syncthreads_or(b < a.B && a.q_start[b + 1] < a.q_start[b])) return;
    } else {
      __syncthreads();
    }
    int add = total;
    for (int i = 0; i < wave; ++i) add += wave_total[i];
    if (b < items) before[b] = add + incl - v;
    if (b < a.B) lens[b] = len;
    total += wave_total[0] + wave_total[1] + wave_total[2] + wave_total[3];
    __syncthreads();
  }
  if (tid == 0) before[items] = total;
  __syncthreads();
  total = uniform(total);

  const int groups = a.plan.own_groups;
  const int per = total / groups + (total % groups ? 1 : 0);
  if (per <= 0) return;
  int x = (int)min((int64_t)blockIdx.x * per, (int64_t)total);
  const int xe = (int)min((int64_t)x + per, (int64_t)total);
  if (x >= xe) return;
  int b = 0;
  {
    int hi = items;                      // before[b] <= x < before[hi]
    while (hi - b > 1) {
      const int mid = (b + hi) >> 1;
      if (before[mid] <= x) b = mid;
      else hi = mid;
    }
    b = uniform(b);
  }

  Wave<KV, D, STREAM> w(a);
  while (x < xe) {
    while (b + 1 < items && uniform(before[b + 1]) <= x) ++b;
    Block k;
    int unit0, units, id;
    const int rel = x - uniform(before[b]);
    int part;
    if (b < a.B) {
      Seq s = seq_of(a, b, uniform(lens[b]));
      s.q0 = uniform(s.q0);
      s.n = uniform(s.n);
      units = units_of(a, s);
      unit0 = first_key(a, s) / kUnit;
      part = rel / units;
      const int j = part / a.Hkv;
      k.q0 = s.q0;
      k.row0 = 16 * j;
      k.rows = min(16, s.n * a.G - 16 * j);
      k.h = part - j * a.Hkv;
      k.table = a.table + (int64_t)b * a.max_pages;
      k.keys = s.len;
      k.pre = 0;
      k.n = s.n;
      k.len = s.len;
      id = (block_base(a, b, s.q0, 16) + j) * a.Hkv + k.h;
    } else {
      units = pre_units;
      unit0 = 0;
      part = rel / units;
      const int j = part / a.Hkv;
      k.q0 = 0;
      k.row0 = 16 * j;
      k.rows = (int)min((int64_t)16, (int64_t)a.T * a.G - 16 * j);
      k.h = part - j * a.Hkv;
      k.table = a.prefix_table;
      k.keys = a.prefix_len;
      k.pre = 1;
      k.n = k.len = 0;
      id = (a.plan.own_blocks + j) * a.Hkv + k.h;
    }
    const int u = rel - part * units;
    const int ue = min(units, u + (xe - x));
    const int w0 = (x - u) / per, w1 = (x - u + units - 1) / per;
    const bool direct = w0 == w1 && a.prefix_len == 0;
    const int64_t slot = (int64_t)blockIdx.x + id;
    if (u == 0 && tid == 0) a.meta[id] = make_int2(w0 + id, direct ? -1 : w1 - w0 + 1);

    w.begin(k);
    w.walk(k, (unit0 + u) * 4 + wave, (unit0 + ue) * 4, 4);

    // the waves' sums in two steps: 2 and 3 to 0 and 1, then 1 to 0
#pragma unroll
    for (int step = 2; step; step >>= 1) {
      if (wave >= step && wave < 2 * step) {
        float* m = merge[wave - step][w.n];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int t = 0; t < DPL; t += 4)
            *(float4*)(m + DPL * (4 * w.g + i) + t) =
                make_float4(w.o[t][i], w.o[t + 1][i], w.o[t + 2][i], w.o[t + 3][i]);
        if (w.g == 0) merge_ml[wave - step][w.n] = make_float2(w.ref, w.sum);
      }
      __syncthreads();
      if (wave < step) {
        const float* m = merge[wave][w.n];
        const float2 e = merge_ml[wave][w.n];
        const float top = fmaxf(w.ref, e.x);
        const float f0 = __builtin_amdgcn_exp2f(w.ref - top), f1 = __builtin_amdgcn_exp2f(e.x - top);
        w.ref = top;
        w.sum = w.sum * f0 + e.y * f1;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int t = 0; t < DPL; t += 4) {
            const float4 c = *(const float4*)(m + DPL * (4 * w.g + i) + t);
            w.o[t][i] = w.o[t][i] * f0 + c.x * f1;
            w.o[t + 1][i] = w.o[t + 1][i] * f0 + c.y * f1;
            w.o[t + 2][i] = w.o[t + 2][i] * f0 + c.z * f1;
            w.o[t + 3][i] = w.o[t + 3][i] * f0 + c.w * f1;
          }
      }
      __syncthreads();
    }
    if (wave == 0) w.out_row(k, slot, direct);
    x += ue - u;
  }
}

// --------------------------------------------- many rows: a wave has its own

// Keys and values of KT = 2048 W / D keys at a time go through LDS, converted
// once for the workgroup's 16 W RT rows, each 16-byte piece where a lane of the
// matrix product reads it: lanes read and write consecutive pieces.  While a
// tile is computed the next but one is on its way in registers and the next
// one in the other half of LDS; one barrier per tile.
template <int KV, int D, int RT, int W>
struct Rows {
  static constexpr bool F8 = KV != kKvBf16;
  static constexpr int ES = F8 ? 1 : 2;
  static constexpr int KT = 2048 * W / D;          // keys of a tile
  static constexpr int SUBS = KT / 16, NS = KT / 32;
  static constexpr int COLS = D / 64;              // 64-value columns
  static constexpr int KP = 2 * ES;                // 16-byte pieces of keys of a thread
  static constexpr int NO = D / 16;                // output registers of four
  static constexpr int kIdTiles = 64 / SUBS;       // tiles that one load of page ids covers

  struct Shared {
    uint4 k[2][SUBS * (D / 32) * 64];
    uint4 v[2][NS * NO * 64];
    float ks[2][KT], vs[2][KT];
    int odd[2][W];           // values that are not finite were taken out
    int range[W][4];
  };
  struct Raw {
    uint4 k[KP];
    u32x2 v[8];              // E4M3: the first dword
    uint32_t ks, vs;
  };

  const AttnArgs& a;
  Shared& sh;
  bf16x8 q[RT][D / 32];
  v4f o[RT][NO];             // o[4 i + t][r]: value 64 i + 16 g + 4 r + t
  float ref[RT], sum[RT];
  float most_sum[RT];        // a larger sum of p, and the reference is looked at
  int lo[RT], hi[RT];
  int lo_most, lo_least, hi_least, hi_most;        // of the workgroup's rows
  int wave, lane, n, g;

  __device__ __forceinline__ Rows(const AttnArgs& args, Shared& shared) : a(args), sh(shared) {
    wave = uniform(threadIdx.x >> 6);
    lane = threadIdx.x & 63;
    n = lane & 15;
    g = lane >> 4;
  }

  __device__ __forceinline__ void begin(const Block& b, int row0) {
    int lom = 0, lol = 0x7fffffff, hil = 0x7fffffff, him = 0;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int r = row0 + 16 * rt + n;
      const bool live = r < b.rows;
      const int i = live ? (b.row0 + r) / a.G : 0;
      const int head = b.h * a.G + (b.row0 + r - i * a.G);
      lo[rt] = hi[rt] = 0;
      if (live) {
        row_range(a, b, r, &lo[rt], &hi[rt]);
        lom = max(lom, lo[rt]);
        lol = min(lol, lo[rt]);
        hil = min(hil, hi[rt]);
        him = max(him, hi[rt]);
      }
      const uint16_t* src = a.q + (int64_t)(b.q0 + i) * a.ldq + (int64_t)head * D + 8 * g;
#pragma unroll
      for (int s = 0; s < D / 32; ++s) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (live) v = *(const uint4*)(src + 32 * s);
        q[rt][s] = __builtin_bit_cast(bf16x8, v);
      }
#pragma unroll
      for (int t = 0; t < NO; ++t) o[rt][t] = v4f{0, 0, 0, 0};
      ref[rt] = kLowest;
      sum[rt] = 0.0f;
      most_sum[rt] = kMostSum;
    }
    lom = row16_max(lom);
    lol = -row16_max(-lol);
    hil = -row16_max(-hil);
    him = row16_max(him);
    if (lane == 0) {
      sh.range[wave][0] = lom;
      sh.range[wave][1] = lol;
      sh.range[wave][2] = hil;
      sh.range[wave][3] = him;
    }
    __syncthreads();
    lo_most = sh.range[0][0];
    lo_least = sh.range[0][1];
    hi_least = sh.range[0][2];
    hi_most = sh.range[0][3];
#pragma unroll
    for (int i = 1; i < W; ++i) {
      lo_most = max(lo_most, sh.range[i][0]);
      lo_least = min(lo_least, sh.range[i][1]);
      hi_least = min(hi_least, sh.range[i][2]);
      hi_most = max(hi_most, sh.range[i][3]);
    }
    lo_most = uniform(lo_most);
    lo_least = uniform(lo_least);
    hi_least = uniform(hi_least);
    hi_most = uniform(hi_most);
  }

  // Page ids of 64 times 16 keys from tile on.
  __device__ __forceinline__ int page_ids(const Block& b, int tile) const {
    const int64_t key = (int64_t)tile * KT + 16 * lane;
    int id = -1;
    if (key < b.keys) {
      id = b.table[key >> a.log2_page];
      if (id < 0 || id >= a.num_pages) id = -1;
    }
    return id;
  }
  __device__ __forceinline__ static uint32_t pages_there(int ids, int first_id) {
    return (uint32_t)(__ballot(ids >= 0) >> first_id) & ((1u << SUBS) - 1);
  }
  // The first row (of keys, in the cache) of 16 keys.
  __device__ __forceinline__ int64_t first_row(const Block& b, int id, int key) const {
    return (((int64_t)(id < 0 ? 0 : id) * a.Hkv + b.h) << a.log2_page) + (key & ((1 << a.log2_page) - 1));
  }

  __device__ __forceinline__ void load(const Block& b, int tile, int ids, int first_id, Raw& x) const {
#pragma unroll
    for (int p = 0; p < KP; ++p) {
      const int at = wave * KP + p;
      const int per = F8 ? COLS : 2 * COLS;        // pieces of 64 bytes in a key
      const int s = at / per, col = at % per;
      const int id = __builtin_amdgcn_readlane(ids, first_id + s);
      const auto r = make_rsrc(a.kc + first_row(b, id, tile * KT + 16 * s) * (D * ES), 16 * D * ES);
      x.k[p] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
          r, n * (D * ES) + 64 * col + 16 * g, 0, 0));
    }
    const int s32 = wave / COLS, col = wave % COLS;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int id = __builtin_amdgcn_readlane(ids, first_id + 2 * s32 + h);
      const auto r = make_rsrc(a.vc + first_row(b, id, tile * KT + 32 * s32 + 16 * h) * (D * ES), 16 * D * ES);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = (4 * g + j) * (D * ES) + (64 * col + 4 * n) * ES;
        if constexpr (F8) x.v[4 * h + j].x = __builtin_amdgcn_raw_buffer_load_b32(r, p, 0, 0);
        else x.v[4 * h + j] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, p, 0, 0));
      }
    }
    const int s = (threadIdx.x >> 4) % SUBS;
    const int id = __shfl(ids, first_id + s);
    if (threadIdx.x < KT) {
      const int64_t row = first_row(b, id, tile * KT + 16 * s) + n;
      if constexpr (KV == kKvFloat) {
        x.ks = *(const uint32_t*)(a.ks + 4 * row);
        x.vs = *(const uint32_t*)(a.vs + 4 * row);
      } else if constexpr (KV == kKvUe8m0) {
        x.ks = a.ks[row];
        x.vs = a.vs[row];
      }
    }
  }

  // A tile's values from registers to LDS.
  __device__ __forceinline__ void stage(int tile, int buf, int ids, int first_id, Raw& x) const {
#pragma unroll
    for (int p = 0; p < KP; ++p) {
      const int at = wave * KP + p;
      if constexpr (F8) {
        const int s = at / COLS, col = at % COLS;
        uint4* to = sh.k[buf] + (s * (D / 32) + 2 * col + (g >> 1)) * 64 + 32 * (g & 1) + n;
        to[0] = __builtin_bit_cast(uint4, Wave<KV, D>::key_operand(make_uint2(x.k[p].x, x.k[p].y)));
        to[16] = __builtin_bit_cast(uint4, Wave<KV, D>::key_operand(make_uint2(x.k[p].z, x.k[p].w)));
      } else {
        sh.k[buf][at * 64 + lane] = x.k[p];
      }
    }
    const int s32 = wave / COLS, col = wave % COLS;
    const int key0 = tile * KT + 32 * s32;
    const int id0 = __builtin_amdgcn_readlane(ids, first_id + 2 * s32);
    const int id1 = __builtin_amdgcn_readlane(ids, first_id + 2 * s32 + 1);
    const bool whole = uniform(id0 >= 0 && id1 >= 0 && key0 >= lo_most && key0 + 32 <= hi_least);
    uint32_t marks = 0;
    if (!whole) {
      // keys that no row of the workgroup sees may hold anything; what is
      // not finite elsewhere reaches only the rows that see it
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int key = key0 + 16 * (j >> 2) + 4 * g + (j & 3);
        const bool ok = ((j >> 2) ? id1 : id0) >= 0 && key >= lo_least && key < hi_most;
#pragma unroll
        for (int i = 0; i < ES; ++i) {
          uint32_t v = ok ? x.v[j][i] : 0;
          const uint32_t m = Wave<KV, D>::odd_marks(v);
          marks |= m;
          x.v[j][i] = v & ~((m >> (F8 ? 7 : 15)) * (F8 ? 0xffu : 0xffffu));
        }
      }
    }
    const bool odd = __any(marks != 0);
    if (lane == 0) sh.odd[buf][wave] = odd;
    uint4* to = sh.v[buf] + (s32 * NO + 4 * col) * 64 + lane;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t c[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (F8) c[j] = h ? Wave<KV, D>::template two_codes<true>(x.v[j].x)
                                   : Wave<KV, D>::template two_codes<false>(x.v[j].x);
        else c[j] = x.v[j][h];
      }
      u32x4 e, f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        e[j] = __builtin_amdgcn_perm(c[2 * j + 1], c[2 * j], 0x05040100u);
        f[j] = __builtin_amdgcn_perm(c[2 * j + 1], c[2 * j], 0x07060302u);
      }
      to[(2 * h) * 64] = __builtin_bit_cast(uint4, e);
      to[(2 * h + 1) * 64] = __builtin_bit_cast(uint4, f);
    }
    if (threadIdx.x < KT) {
      if constexpr (F8) {
        const float ks = KV == kKvFloat ? __uint_as_float(x.ks) : e8m0_f32(x.ks);
        const float vs = KV == kKvFloat ? __uint_as_float(x.vs) : e8m0_f32(x.vs);
        sh.ks[buf][threadIdx.x] = ks * a.scale_log2;
        sh.vs[buf][threadIdx.x] = vs;
      }
    }
  }

  __device__ __forceinline__ void odd_values(const Block& b, int key0, const float (&w)[RT][8],
                                             const uint32_t (&seen)[RT]) {
    int g = this->g, n = this->n;      // not to be prepared before it is known that they are needed
    asm volatile("" : "+v"(g), "+v"(n));
    for (int k = 0; k < 32; ++k) {
      const int id = page_of(b, key0 + k);
      if (id < 0) continue;
      const int j = 4 * (k >> 4) + (k & 3), from = ((k >> 2) & 3) * 16 + n;
      const int64_t row = first_row(b, id, key0 + k);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float mine = w[rt][0];
#pragma unroll
        for (int i = 1; i < 8; ++i) mine = i == j ? w[rt][i] : mine;
        const float wk = __shfl(mine, from);
        const bool sees = (__shfl((int)seen[rt], from) >> j) & 1;
#pragma unroll
        for (int t = 0; t < NO; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int64_t at = row * D + 64 * (t >> 2) + 16 * g + 4 * r + (t & 3);
            float val = 0.0f;
            bool odd;
            if (F8) {
              odd = (a.vc[at] & 0x7fu) == 0x7fu;
              if (odd) val = __uint_as_float(0x7fc00000u);
            } else {
              const uint32_t bits = ((const uint16_t*)a.vc)[at];
              odd = (bits & 0x7f80u) == 0x7f80u;
              val = __uint_as_float(bits << 16);
            }
            if (sees && odd) o[rt][t][r] += wk * val;
          }
      }
    }
  }
  __device__ __forceinline__ int page_of(const Block& b, int key) const {
    if (key >= b.keys) return -1;
    const int id = b.table[key >> a.log2_page];
    return id < 0 || id >= a.num_pages ? -1 : id;
  }

  // 32 keys of a tile.  EDGE: some of them may be hidden from some row;
  // `there`: bit h, whether the 16 keys 16 h .. have a page.
  __device__ __forceinline__ void compute(const Block& b, int key0, int buf, int u, uint32_t there, const bool EDGE) {
    uint4 f[2][D / 32];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < D / 32; ++i) f[h][i] = sh.k[buf][((2 * u + h) * (D / 32) + i) * 64 + lane];
    __builtin_amdgcn_sched_barrier(0);
    float ksl[8], vs[8];
    if constexpr (F8) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 c = *(const float4*)(sh.ks[buf] + 32 * u + 16 * h + 4 * g);
        const float4 d = *(const float4*)(sh.vs[buf] + 32 * u + 16 * h + 4 * g);
        ksl[4 * h] = c.x; ksl[4 * h + 1] = c.y; ksl[4 * h + 2] = c.z; ksl[4 * h + 3] = c.w;
        vs[4 * h] = d.x; vs[4 * h + 1] = d.y; vs[4 * h + 2] = d.z; vs[4 * h + 3] = d.w;
      }
    }
    v4f s[RT][2];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) s[rt][0] = s[rt][1] = v4f{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          s[rt][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, f[h][i]), q[rt][i],
                                                             s[rt][h], 0, 0, 0);
    uint4 v[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) v[t] = sh.v[buf][(u * NO + t) * 64 + lane];
    uint32_t seen[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      seen[rt] = 0xffu;
      if (EDGE) {
        int g = this->g;               // as above
        asm volatile("" : "+v"(g));
        seen[rt] = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int key = key0 + 16 * (j >> 2) + 4 * g + (j & 3);
          const bool ok = ((there >> (j >> 2)) & 1) && key >= lo[rt] && key < hi[rt];
          seen[rt] |= (uint32_t)ok << j;
        }
      }
    }
    float w[RT][8];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float add;
      auto weigh = [&](auto rounded) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          w[rt][j] = weight<decltype(rounded)::value>(s[rt][j >> 2][j & 3], F8 ? ksl[j] : a.scale_log2, ref[rt]);
        if (EDGE) {
#pragma unroll
          for (int j = 0; j < 8; ++j) w[rt][j] = (seen[rt] >> j) & 1 ? w[rt][j] : 0.0f;
        }
        add = ((w[rt][0] + w[rt][1]) + (w[rt][2] + w[rt][3])) + ((w[rt][4] + w[rt][5]) + (w[rt][6] + w[rt][7]));
      };
      weigh(std::false_type());
      // the sum of p bounds every p
      if (__builtin_expect(__any(!(add <= most_sum[rt])), 0)) {
        float top = kLowest;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float e = s[rt][j >> 2][j & 3] * (F8 ? ksl[j] : a.scale_log2);
          if ((seen[rt] >> j) & 1) top = fmaxf(top, e);
        }
        top = fmaxf(ref[rt], group_max(top));
        const float down = __builtin_amdgcn_exp2f(ref[rt] - top);
        ref[rt] = top;
        sum[rt] *= down;
#pragma unroll
        for (int t = 0; t < NO; ++t) o[rt][t] *= down;
        most_sum[rt] = limit_of(top, kMostSum);
        weigh(std::true_type());
      }
      sum[rt] += add;
      if constexpr (F8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[rt][j] *= vs[j];
        if (EDGE) {
#pragma unroll
          for (int j = 0; j < 8; ++j) w[rt][j] = (seen[rt] >> j) & 1 ? w[rt][j] : 0.0f;
        }
      }
    }
    if (EDGE) {
      int odd = 0;
#pragma unroll
      for (int i = 0; i < W; ++i) odd |= sh.odd[buf][i];
      if (uniform(odd)) odd_values(b, key0, w, seen);
    }

    u32x4 wh[RT], wl[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const f32x2 p{w[rt][j], w[rt][j + 1]};
        const bf16x2 c = __builtin_convertvector(p, bf16x2);
        wh[rt][j / 2] = __builtin_bit_cast(uint32_t, c);
        wl[rt][j / 2] = __builtin_bit_cast(uint32_t, __builtin_convertvector(
            (f32x2{p.x - (float)c[0], p.y - (float)c[1]}), bf16x2));
      }
    // four registers of sums, the weights' upper parts before the lower ones
    auto add_values = [&](const uint4 (&x)[4], int t0) {
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
            o[rt][t0 + t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8, x[t]), __builtin_bit_cast(bf16x8, part ? wl[rt] : wh[rt]),
                o[rt][t0 + t], 0, 0, 0);
    };
#pragma unroll
    for (int c = 0; c < COLS; ++c) {
      uint4 z[4];
      if (c + 1 < COLS) {
#pragma unroll
        for (int t = 0; t < 4; ++t) z[t] = sh.v[buf][(u * NO + 4 * c + 4 + t) * 64 + lane];
      }
      add_values(v, 4 * c);
#pragma unroll
      for (int t = 0; t < 4; ++t) v[t] = z[t];
    }
  }

  // Tiles first .. end of the block's keys, all waves together.
  __device__ __forceinline__ void walk(const Block& b, int first, int end) {
    end = min(end, (hi_most + KT - 1) / KT);
    first = max(first, lo_least / KT);
    if (first < end) {
      Raw x;
      int ids = page_ids(b, first), next = page_ids(b, first + kIdTiles);
      load(b, first, ids, 0, x);
      stage(first, 0, ids, 0, x);
      int at = 0;                                  // of the tile in x among the ids' tiles
      uint32_t there = pages_there(ids, 0), there_next = 0;
      // x has tile i + 1 while tile i is computed
      auto fetch = [&](int tile) {
        if (tile >= end) return;
        if (++at == kIdTiles) at = 0;
        if (at == 0) {
          ids = next;
          next = page_ids(b, tile + kIdTiles);
        }
        load(b, tile, ids, at * SUBS, x);
      };
      fetch(first + 1);
      __syncthreads();
      for (int i = first; i < end; ++i) {
        const int buf = (i - first) & 1;
        if (i + 1 < end) {
          stage(i + 1, buf ^ 1, ids, at * SUBS, x);
          there_next = pages_there(ids, at * SUBS);
          fetch(i + 2);
        }
        constexpr uint32_t kAll = (1u << SUBS) - 1;
        const bool edge = !(there == kAll && i * KT >= lo_most && i * KT + KT <= hi_least);
#pragma unroll
        for (int u = 0; u < NS; ++u) compute(b, i * KT + 32 * u, buf, u, there >> (2 * u), edge);
        there = there_next;
        __syncthreads();
      }
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) sum[rt] = group_sum(sum[rt]);
  }

  __device__ __forceinline__ void out_row(const Block& b, int row0, int rt, int64_t slot, int block_rows,
                                          bool direct) const {
    const int r = row0 + 16 * rt + n;
    if (r >= b.rows) return;
    if (direct) {
      const int i = (b.row0 + r) / a.G;
      const int head = b.h * a.G + (b.row0 + r - i * a.G);
      const float f = sum[rt] == 0.0f ? 0.0f : 1.0f / sum[rt];
      uint16_t* y = a.y + ((int64_t)(b.q0 + i) * a.Hq + head) * D + 16 * g;
#pragma unroll
      for (int c = 0; c < COLS; ++c) {
        uint32_t p[8];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int t = 0; t < 4; t += 2)
            p[2 * m + t / 2] = __builtin_bit_cast(uint32_t, __builtin_convertvector(
                (f32x2{o[rt][4 * c + t][m] * f, o[rt][4 * c + t + 1][m] * f}), bf16x2));
        *(uint4*)(y + 64 * c) = make_uint4(p[0], p[1], p[2], p[3]);
        *(uint4*)(y + 64 * c + 8) = make_uint4(p[4], p[5], p[6], p[7]);
      }
    } else {
      const int64_t at = slot * block_rows + r;
      if (g == 0) a.ml[at] = make_float2(ref[rt], sum[rt]);
      float* p = a.part + at * D + 16 * g;
#pragma unroll
      for (int c = 0; c < COLS; ++c)
#pragma unroll
        for (int m = 0; m < 4; ++m)
          *(float4*)(p + 64 * c + 4 * m) =
              make_float4(o[rt][4 * c][m], o[rt][4 * c + 1][m], o[rt][4 * c + 2][m], o[rt][4 * c + 3][m]);
    }
  }
};

// A workgroup takes 16 W RT rows of a block and key head; every wave walks all of
// its split of the keys.  pre: the blocks are of all tokens, the keys the
// prefix's.  Eight waves a CU (132 KB of LDS, 256 registers), in one workgroup
// or two: one wave's products run beside another's weights.  Eight waves a
// workgroup at 2 x 2048 over 6000 keys: matrix cores busy 45% of the time,
// vector issue 61%, LDS 30%; waves wait on issue 31% of theirs, on loads, LDS and
// barriers 29%.  Four convert and store a tile for half the rows (522 us against
// 476).  32 rows a wave share an operand read from LDS (16 would double LDS's
// share to where it bounds; 64 leave one wave a SIMD: 689 us against 516, both with
// one product of the weights and four waves).
template <int KV, int D, int RT, int W>
__global__ __launch_bounds__(64 * W, 8 / W) void attn_rows_kernel(AttnArgs a, const int pre) {
  constexpr int ROWS = 16 * W * RT;
  using R = Rows<KV, D, RT, W>;
  constexpr int KT = R::KT;
  __shared__ typename R::Shared sh;
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int splits = pre ? a.plan.pre_splits : a.plan.own_splits;
  const int blocks = pre ? a.plan.pre_blocks : a.plan.own_blocks;
  const int64_t wg = grid_row();
  if (wg >= (int64_t)blocks * splits * a.Hkv) return;
  Block k;
  k.h = (int)(wg % a.Hkv);
  const int64_t rest = wg / a.Hkv;
  const int split = (int)(rest % splits);
  const int blk = blocks - 1 - (int)(rest / splits);   // a sequence's last block has the most keys
  int first = 0, end;
  if (pre) {
    k.q0 = 0;
    k.row0 = blk * ROWS;
    k.rows = (int)min((int64_t)ROWS, (int64_t)a.T * a.G - k.row0);
    k.table = a.prefix_table;
    k.keys = a.prefix_len;
    k.pre = 1;
    k.n = k.len = 0;
    end = (k.keys + KT - 1) / KT;
  } else {
    int count = 0;                     // sequences whose blocks begin at or before this one
    bool falls = false;
    for (int b = threadIdx.x; b < a.B; b += 64 * W) {
      const int q0 = a.q_start ? clampi(a.q_start[b], 0, a.T) : b;
      count += block_base(a, b, q0, ROWS) <= blk;
      falls |= a.q_start && a.q_start[b + 1] < a.q_start[b];
    }
    if (__syncthreads_or(falls)) return;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) count += __shfl_xor(count, d);
    if (lane == 0) sh.range[wave][0] = count;
    __syncthreads();
    count = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) count += sh.range[i][0];
    const int b = uniform(count) - 1;
    __syncthreads();
    if (b < 0) return;
    Seq s = seq_of(a, b);
    s.q0 = uniform(s.q0);
    s.n = uniform(s.n);
    s.len = uniform(s.len);
    const int j = blk - block_base(a, b, s.q0, ROWS);
    if (j < 0 || (int64_t)j * ROWS >= (int64_t)s.n * a.G) return;
    k.q0 = s.q0;
    k.row0 = j * ROWS;
    k.rows = min(ROWS, s.n * a.G - k.row0);
    k.table = a.table + (int64_t)b * a.max_pages;
    k.keys = s.len;
    k.pre = 0;
    k.n = s.n;
    k.len = s.len;
    const int pos0 = s.len - s.n + k.row0 / a.G, pos1 = s.len - s.n + (k.row0 + k.rows - 1) / a.G;
    end = (clampi(pos1 + 1, 0, s.len) + KT - 1) / KT;
    if (a.window) first = (int)(max((int64_t)pos0 - a.window + 1, (int64_t)0) / KT);
  }
  const int tiles = max(end - first, 0);
  const int per = (tiles + splits - 1) / splits;
  const int parts = per ? (tiles + per - 1) / per : 0;
  const int id = (pre ? a.plan.own_blocks + blk : blk) * a.Hkv + k.h;
  const int64_t slot = ((int64_t)blk * a.Hkv + k.h) * splits + split + (pre ? a.plan.own_slots * a.plan.own_rows / ROWS : 0);
  const bool direct = !pre && parts <= 1 && a.prefix_len == 0;
  if (split == 0 && threadIdx.x == 0)
    a.meta[id] = make_int2((int)slot, direct ? -1 : parts);
  if (split >= parts && !(direct && split == 0)) return;
  const int row0 = wave * 16 * RT;
  R w(a, sh);
  w.begin(k, row0);
  w.walk(k, first + split * per, min(first + (split + 1) * per, end));
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) w.out_row(k, row0, rt, slot, ROWS, direct);
}

// ------------------------------------------------------------ joined results

// A row's partial results (of its own keys, of the prefix) to y.  WPR waves
// per row.
template <int D, int WPR>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  constexpr int LPR = D / 4, SUB = 64 / LPR;       // lanes of a partial row, rows at once
  constexpr int RPB = 4 / WPR;
  __shared__ float4 acc[4][64];
  __shared__ float accl[4][64], acct[4];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t row = grid_row() * RPB + wave / WPR;
  if (row >= (int64_t)a.T * a.Hq) return;          // WPR = 4: the whole workgroup
  const int t = uniform((int)(row / a.Hq)), head = uniform((int)(row - (int64_t)t * a.Hq));
  const int h = head / a.G, gq = head - h * a.G;
  int b = t;
  if (a.q_start) {
    int count = 0;                     // sequences that end at or before the token
    bool falls = false;
    for (int i = lane; i < a.B; i += 64) {
      const int next = a.q_start[i + 1];
      count += next <= t;
      falls |= next < a.q_start[i];
    }
    if (__any(falls)) return;          // nothing was computed
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) count += __shfl_xor(count, d);
    b = uniform(count);
    if (b >= a.B || t < a.q_start[b]) return;
  }
  const Seq s = seq_of(a, b);
  if (t >= s.q0 + s.n) return;
  const int local = (t - s.q0) * a.G + gq;
  const int orows = a.plan.own_rows, prows = a.plan.pre_rows;
  // what is of no use (no keys: nobody wrote it) is loaded all the same, not
  // behind the lengths
  const int2 m0 = a.meta[(block_base(a, b, s.q0, orows) + local / orows) * a.Hkv + h];
  int c0 = 0, c1 = 0;
  int64_t f0 = 0, f1 = 0;              // the first partial's rows
  if (a.prefix_len > 0) {
    const int64_t all = (int64_t)t * a.G + gq;
    const int2 m1 = a.meta[(a.plan.own_blocks + (int)(all / prows)) * a.Hkv + h];
    c1 = uniform(m1.y);
    f1 = (int64_t)uniform(m1.x) * prows + all % prows;
  }
  if (uniform(s.len) > 0) {
    if (uniform(m0.y) < 0) return;     // written already
    c0 = uniform(m0.y);
    f0 = (int64_t)uniform(m0.x) * orows + local % orows;
  }
  const int count = c0 + c1;
  auto place = [&](int i) { return i < c0 ? f0 + (int64_t)i * orows : f1 + (int64_t)(i - c0) * prows; };
  const int sub = lane / LPR + SUB * (wave % WPR), d4 = lane % LPR;
  constexpr int STEP = SUB * WPR, NL = 4;          // rows at once, loads under way
  float4 o = make_float4(0, 0, 0, 0);
  float l = 0.0f, top = kLowest;
  for (int i0 = sub; i0 < count; i0 += NL * STEP) {
    float2 e[NL];
    float4 c[NL];
#pragma unroll
    for (int u = 0; u < NL; ++u) {
      const int i = i0 + u * STEP;
      e[u] = make_float2(kLowest, 0.0f);
      c[u] = make_float4(0, 0, 0, 0);
      if (i < count) {
        const int64_t at = place(i);
        e[u] = a.ml[at];
        c[u] = *(const float4*)(a.part + at * D + 4 * d4);
      }
    }
    float high = top;
#pragma unroll
    for (int u = 0; u < NL; ++u) high = fmaxf(high, e[u].x);
    const float down = __builtin_amdgcn_exp2f(top - high);
    top = high;
    l *= down;
    o.x *= down;
    o.y *= down;
    o.z *= down;
    o.w *= down;
#pragma unroll
    for (int u = 0; u < NL; ++u) {
      const float f = __builtin_amdgcn_exp2f(e[u].x - top);
      l += e[u].y * f;
      o.x += c[u].x * f;
      o.y += c[u].y * f;
      o.z += c[u].z * f;
      o.w += c[u].w * f;
    }
  }
  // the lanes' sums, each to its own reference
  float all = top;
#pragma unroll
  for (int d = LPR; d < 64; d <<= 1) all = fmaxf(all, __shfl_xor(all, d));
  if constexpr (WPR > 1) {
    if (lane == 0) acct[wave] = all;
    __syncthreads();
    all = fmaxf(fmaxf(acct[0], acct[1]), fmaxf(acct[2], acct[3]));
  }
  {
    const float down = __builtin_amdgcn_exp2f(top - all);
    l *= down;
    o.x *= down;
    o.y *= down;
    o.z *= down;
    o.w *= down;
  }
#pragma unroll
  for (int d = LPR; d < 64; d <<= 1) {
    l += __shfl_xor(l, d);
    o.x += __shfl_xor(o.x, d);
    o.y += __shfl_xor(o.y, d);
    o.z += __shfl_xor(o.z, d);
    o.w += __shfl_xor(o.w, d);
  }
  if constexpr (WPR > 1) {
    acc[wave][lane] = o;
    accl[wave][lane] = l;
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int i = 1; i < WPR; ++i) {
      const float4 c = acc[i][lane];
      l += accl[i][lane];
      o.x += c.x;
      o.y += c.y;
      o.z += c.z;
      o.w += c.w;
    }
  }
  if (lane >= LPR) return;
  const float f = l == 0.0f ? 0.0f : 1.0f / l;
  const bf16x2 lo = __builtin_convertvector((f32x2{o.x * f, o.y * f}), bf16x2);
  const bf16x2 hi = __builtin_convertvector((f32x2{o.z * f, o.w * f}), bf16x2);
  *(uint2*)(a.y + row * D + 4 * d4) = make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
}

template <int KV, int D>
hipError_t launch_attn(AttnArgs a, hipStream_t s) {
  constexpr int RT = attn_row_tiles(D);
  AttnPlan& p = a.plan;
  // all at once, so that equal shares end together
  if (p.own_groups > 256 * split_resident(KV, D)) p.own_groups = 256 * split_resident(KV, D);
  // What a call may read is left in the last-level cache where it fits there (256
  // MiB), and passes it by where it does not: 64 sequences of up to 8192 keys 118 us
  // with the cache, 106 past it.  It goes by what the tables have room for (the
  // lengths are on the device): shorter sequences in such tables, which the cache
  // might hold from call to call, are read past it too (64 of up to 2000 keys 37 us
  // with it, 40 past it; of up to 600 the same).
  const int64_t room = (int64_t)a.max_pages << a.log2_page;
  const int64_t keys = a.window && a.window < room ? a.window : room;
  const bool stream = keys * a.B * a.Hkv * 2 * (KV == kKvBf16 ? 2 * D : D + 4) > (int64_t(1) << 28);
  auto rows_launch = [&](int waves, int64_t workgroups, int pre) {
    if (waves == 8)
      hipLaunchKernelGGL((attn_rows_kernel<KV, D, RT, 8>), row_grid(workgroups), dim3(512), 0, s, a, pre);
    else
      hipLaunchKernelGGL((attn_rows_kernel<KV, D, RT, 4>), row_grid(workgroups), dim3(256), 0, s, a, pre);
  };
  if (p.pre_wide) rows_launch(p.pre_waves, (int64_t)p.pre_blocks * p.pre_splits * a.Hkv, 1);
  if (p.own_wide) rows_launch(p.own_waves, (int64_t)p.own_blocks * p.own_splits * a.Hkv, 0);
  else if (stream)
    hipLaunchKernelGGL((attn_split_kernel<KV, D, true>), dim3(p.own_groups), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((attn_split_kernel<KV, D, false>), dim3(p.own_groups), dim3(256), 0, s, a);
  if (p.complete) return hipGetLastError();
  const int64_t rows = (int64_t)a.T * a.Hq;
  // four waves a row, or one: 256 rows of 4096 keys 25.0 us and 25.6, one row in
  // a hundred partial results 32.6 and 37.3; 2048 rows 34.7 and 33.2, 16384 85 and 74
  if (rows <= 1024)
    hipLaunchKernelGGL((attn_join_kernel<D, 4>), row_grid(rows), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((attn_join_kernel<D, 1>), row_grid((rows + 3) / 4), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int KV>
hipError_t launch_attn_d(const AttnArgs& a, hipStream_t s) {
  if (a.D == 64) return launch_attn<KV, 64>(a, s);
  if (a.D == 128) return launch_attn<KV, 128>(a, s);
  return launch_attn<KV, 256>(a, s);
}

}  // namespace detail
using namespace detail;

AttnPlan attn_plan(int64_t T, int64_t B, int Hq, int Hkv, int D, int64_t keys, int64_t prefix_len) {
  AttnPlan p{};
  const int64_t G = Hq / Hkv, rows = T * G;
  const int wide = 16 * attn_row_tiles(D);           // of a wave
  auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  auto splits = [&](int64_t blocks, int waves, int64_t most) {
    const int64_t want = up(2048 / waves, blocks * Hkv), tiles = up(most, 8 * kTile);
    return (int)(want < tiles ? want : (tiles > 1 ? tiles : 1));
  };
  // Few rows: four waves share a block's keys, a step of 128 keys is a unit, and
  // every block reads the keys anew.  Many: a wave has its own rows, and a
  // workgroup 128 of a sequence or more, of which few are there where sequences
  // bring few.  Heads of 128, 8 key heads, us, many-row launch and the other,
  // behind 4096 keys:
  //   1 sequence,  128 rows of it (2048 units)  27.6  26.3;  256 (4096)  27.1  33.5
  //   8 sequences,  64 rows of each (8192)  52.6  55.7;  16 (16384)  87.8  94.4;  32  134  219
  //   8 sequences,  48 rows of each (6144)  51.2  35.1;  16 (12288)  84.9  55.5;  32  131  121
  //   16 sequences, 32 rows of each (8192)  68.5  55.6;  32 (16384)  126  117;  128  457  412
  // Behind few keys it is the blocks that count, each with its own latencies; 64
  // rows of each behind 256 keys:  8 sequences (256 blocks and key heads)  17.6  16.5;
  // 16 (512)  17.9  17.2;  32 (1024)  22.5  31.3;  64 (2048)  36.2  44.2;  behind 64 keys 10.3
  // 12.0,  10.6  14.4,  12.9  21.7,  20.1  33.4.  32 rows of each behind 1024 keys:  32
  // sequences (512)  45.8  38.4;  64 (1024)  66.0  61.9;  128 (2048)  128  140;  behind 256 keys
  // 22.3  17.0,  26.7  31.7,  46.0  46.5;  behind 64 keys 11.9  14.0,  15.3  21.8,  25.8  34.1.
  const int64_t blocks = up(rows, 16) * Hkv;
  if (rows > 48 * B) p.own_wide = blocks > 512 || up(keys, kUnit) * blocks > 6144;
  else p.own_wide = rows > 16 * B && blocks > 512 && keys <= 256;
  // The same for the prefix, many-row launch and with the sequences': 64 rows on
  // 4096 keys (1024 units) 29.0  19.5, on 16384 (4096) 39.2  37.8; 256 rows on 4096 (4096)
  // 36.3  35.6, on 16384 (16384) 61  115; 512 rows on 4096 (8192) 51  60; 1024 rows on 1024
  // (4096) 48.5  46.3.
  p.pre_wide = prefix_len > 0 && (p.own_wide || up(prefix_len, kUnit) * up(rows, 16) * Hkv > 4096);
  // Workgroups of eight waves where their 256 rows are mostly there.  Behind 4096
  // keys, four waves and eight, us: 1 sequence of 512 rows 36.0  39.5, of 1024 50.4  52.4,
  // of 2048 76.2  75.5; 2 of 1024 78.5  75.7; 4 of 512 79.3  86.9; 8 of 256 96  117, of 512
  // 135  127, of 1024 215  194; 16 of 512 222  374; 2 of 8192 over 6000 keys 522  476.  The
  // prefix launch's: 512 rows on 4096 keys 51.4  53.1, on 16384 93  88; 1024 on 4096 72.2
  // 70.8, on 16384 151  138.
  p.own_waves = rows >= 1024 * B ? 8 : 4;
  p.pre_waves = rows >= 1024 ? 8 : 4;
  p.own_rows = p.own_wide ? wide * p.own_waves : 16;
  p.pre_rows = p.pre_wide ? wide * p.pre_waves : 16;
  p.own_blocks = (int)(rows / p.own_rows + B);
  p.pre_blocks = prefix_len > 0 ? (int)up(rows, p.pre_rows) : 0;
  if (p.own_wide) {
    p.own_splits = splits(p.own_blocks, p.own_waves, keys);
    p.complete = p.own_splits == 1 && prefix_len == 0;   // rows in one piece, and nothing to join them with
    p.own_slots = (int64_t)p.own_blocks * Hkv * p.own_splits;
  } else {
    const int64_t own = up(keys, kUnit) * (rows / 16 + B) * Hkv;
    const int64_t pre = p.pre_wide ? 0 : up(prefix_len, kUnit) * p.pre_blocks * Hkv;
    const int64_t most = own + pre > 0 ? own + pre : 1;
    p.own_groups = (int)(most < 768 ? most : 768);
    p.own_slots = p.own_groups + (int64_t)(p.own_blocks + (p.pre_wide ? 0 : p.pre_blocks)) * Hkv;
  }
  if (p.pre_wide) {
    p.pre_splits = splits(p.pre_blocks, p.pre_waves, prefix_len);
    p.pre_slots = (int64_t)p.pre_blocks * Hkv * p.pre_splits;
    // the prefix's partials begin at a whole block of theirs
    p.own_slots = up(p.own_slots * p.own_rows, p.pre_rows) * p.pre_rows / p.own_rows;
  }
  auto aligned = [](size_t v) { return (v + 255) & ~size_t(255); };
  const int64_t prow = p.own_slots * p.own_rows + p.pre_slots * p.pre_rows;
  p.off_ml = aligned((size_t)(p.own_blocks + p.pre_blocks) * Hkv * sizeof(int2));
  p.off_part = p.off_ml + aligned((size_t)prow * sizeof(float2));
  // complete rows leave no partial sums (1.1 GB for 32768 tokens of 64 heads of 128)
  p.bytes = p.off_part + (p.complete ? 0 : (size_t)prow * D * sizeof(float));
  return p;
}

hipError_t launch_paged_attn(const AttnArgs& a, hipStream_t s) {
  if (a.fmt == kKvFloat) return launch_attn_d<kKvFloat>(a, s);
  if (a.fmt == kKvUe8m0) return launch_attn_d<kKvUe8m0>(a, s);
  return launch_attn_d<kKvBf16>(a, s);
}

}  // namespace bsfp8
