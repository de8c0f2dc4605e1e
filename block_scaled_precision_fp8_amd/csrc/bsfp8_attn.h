// Declarations of the operators between the QKV and the output linear: rotary
// positions, the paged key/value cache, attention over it.
#pragma once

#include "bsfp8_layer.h"

namespace bsfp8 {

enum { kKvFloat = 0, kKvUe8m0 = 1, kKvBf16 = 2 };   // bsfp8_kv_fmt

struct RopeKvArgs {
  const uint16_t* q;         // bf16 [T][Hq][D], row stride ldq; or null
  int64_t ldq;
  uint16_t* q_out;           // row stride ldqo
  int64_t ldqo;
  const uint16_t* k;         // bf16 [T][Hkv][D], row stride ldk; or null
  int64_t ldk;
  const uint16_t* v;
  int64_t ldv;
  const int32_t* positions;  // [T]
  const float* inv_freq;     // [rot / 2]
  int rot, interleaved;
  float mscale;
  const int64_t* slots;      // [T]
  int64_t T;
  int Hq, Hkv, D, fmt, log2_page;
  int64_t num_slots;         // pages * page size
  void* k_cache;             // [pages][Hkv][page][D] codes or bf16
  void* v_cache;
  void* k_scale;             // [pages][Hkv][page] fp32 or E8M0, null for bf16
  void* v_scale;
};

// The partial sums' place in the workspace and who works on what; host-made
// from sizes alone.
struct AttnPlan {
  int own_rows, pre_rows;    // rows of a block: of one sequence, of the prefix launch
  bool own_wide, pre_wide;   // which launch computes them (pre_wide false: with the sequences)
  int own_blocks, pre_blocks;            // bounds of their numbers (own: also ids between)
  int own_waves, pre_waves;              // of a wide launch's workgroups
  int own_splits, pre_splits;            // of a wide block's keys
  int own_groups;                        // workgroups of the launch that splits keys evenly
  int64_t own_slots, pre_slots;          // partial results
  bool complete;             // the one launch writes all of y, and no partial result
  size_t off_ml, off_part, bytes;
};

struct AttnArgs {
  const uint16_t* q;         // bf16 [T][Hq][D], row stride ldq
  int64_t ldq;
  const int32_t* q_start;    // [B + 1], or null: a token per sequence
  const int32_t* kv_len;     // [B]
  const int32_t* table;      // [B][max_pages]
  int max_pages;
  const int32_t* prefix_table;
  int prefix_len;
  const uint8_t* kc;
  const uint8_t* vc;
  const uint8_t* ks;
  const uint8_t* vs;
  int fmt, log2_page, num_pages;
  int T, B, Hq, Hkv, D, G;
  float scale_log2;          // the scores' scale times log2(e)
  int window;
  uint16_t* y;               // bf16 [T][Hq][D]
  int2* meta;                // per block and key head: first partial, how many
  float2* ml;                // per partial row: reference exponent, sum
  float* part;               // per partial row: D sums
  AttnPlan plan;
};

// Tiles of 16 rows that a wave of the many-row launches has.
constexpr int attn_row_tiles(int D) { return D == 256 ? 1 : 2; }
constexpr int kAttnMaxSeqs = 4096;
constexpr int64_t kAttnMaxKeys = int64_t(1) << 30;

hipError_t launch_rope_inv_freq(int scaling, int rot, double base, double factor, double low,
                                double high, double orig_len, float* out, hipStream_t s);
hipError_t launch_rope_kv_append(const RopeKvArgs& a, hipStream_t s);
AttnPlan attn_plan(int64_t T, int64_t B, int Hq, int Hkv, int D, int64_t keys, int64_t prefix_len);
hipError_t launch_paged_attn(const AttnArgs& a, hipStream_t s);

}  // namespace bsfp8
