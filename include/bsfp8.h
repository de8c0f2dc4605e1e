/*
 * bsfp8.h -- C-ABI of libbsfp8.so: block-scaled FP8 and NVFP4-style linear
 * layers on AMD MI355X (gfx950).
 *
 * Page citations use the page titles:
 *   [FG-FP8] "Transformers 中的细粒度 FP8 量化：配置、DeepGEMM 加速路径与
 *            UE8M0 缩放格式完全指南", sections 一 .. 九
 *   [HF-PT]  "FP8 de granularidade fina" (Transformers docs)
 *   [NVFP4]  "混合精度策略解析：NVIDIA Mistral-Medium-3.5-128B-NVFP4中FP8与
 *            NVFP4的协同工作", sections on NVFP4 and on the config files
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Every tensor pointer is a DEVICE pointer on the current HIP device,
 *   except where a parameter says "host".  The caller allocates and owns all
 *   memory; the library allocates nothing, keeps no state between calls
 *   (apart from a per-device architecture check done once), never
 *   synchronises the device and never prints.
 * - `stream` is a hipStream_t passed as void*; NULL means the default
 *   stream.  Every call only enqueues work on that stream.
 * - Matrices are row-major and dense unless a leading dimension is given.
 *   bf16 tensors are raw 16-bit patterns (uint16_t); FP8 tensors are OCP
 *   E4M3FN bytes; UE8M0 scales are E8M0 bytes (value 2^(b-127)); fp32
 *   scales are IEEE binary32.
 * - All argument checks run on the host before any HIP call, so the error
 *   returns below are reachable without a GPU.  A zero-sized problem
 *   (M, T or R == 0) returns BSFP8_OK without launching anything.
 * - Return value: a bsfp8_status; BSFP8_EHIP means a HIP call or a kernel
 *   launch failed (the HIP error is not cleared and can be read with
 *   hipGetLastError / hipPeekAtLastError).
 * - Pointers must be 16-byte aligned and leading dimensions must keep every
 *   row 16-byte aligned (EINVAL otherwise).
 */
#ifndef BSFP8_H
#define BSFP8_H

#include <stddef.h>
#include <stdint.h>

#ifndef BSFP8_API
#define BSFP8_API __attribute__((visibility("default")))
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  BSFP8_OK = 0,
  BSFP8_EINVAL = 1,   /* bad argument: enum, size, null pointer, alignment  */
  BSFP8_ENOTSUP = 2,  /* legal on the pages but not provided here, or a     */
                      /* device that is not gfx950, or a stream that       */
                      /* belongs to another device                         */
  BSFP8_ENOSPC = 3,   /* workspace smaller than bsfp8_workspace_size()      */
  BSFP8_EHIP = 4      /* HIP runtime / launch error                         */
} bsfp8_status;

/* scale_fmt: [FG-FP8] §四 allows "float" or "ue8m0"; §七 stores UE8M0 scales
   as float8_e8m0fnu bytes. */
typedef enum { BSFP8_SCALE_FLOAT = 0, BSFP8_SCALE_UE8M0 = 1 } bsfp8_scale_fmt;

/* activation_scheme: [FG-FP8] §四 allows "dynamic" or "static" (the pages
   keep static on a separate kernel path, §6.1, §6.3, and give no formula).
   Static here is one calibrated per-tensor scale supplied by the caller:
   fp8_quant_act (in x_scale[0]) and fp8_linear (through act_scale) take it
   with 128 x 128 blocks; the other entry points consume quantized operands
   and do not depend on the scheme. */
typedef enum { BSFP8_ACT_DYNAMIC = 0, BSFP8_ACT_STATIC = 1 } bsfp8_act_scheme;

/* Scores of moe_route_topk. */
typedef enum { BSFP8_SCORE_SOFTMAX = 0, BSFP8_SCORE_SIGMOID = 1 } bsfp8_score;

/* Formats of a paged key/value cache: E4M3 codes with one scale per token and
   head, of a scale_fmt, or bf16 values. */
typedef enum {
  BSFP8_KV_FP8_FLOAT = 0,
  BSFP8_KV_FP8_UE8M0 = 1,
  BSFP8_KV_BF16 = 2
} bsfp8_kv_fmt;

/* Angle tables of rope_inv_freq. */
typedef enum {
  BSFP8_ROPE_PLAIN = 0,
  BSFP8_ROPE_LINEAR = 1,
  BSFP8_ROPE_BY_PARTS = 2
} bsfp8_rope_scaling;

/* Operation ids for bsfp8_workspace_size. */
typedef enum {
  BSFP8_OP_BLOCK_GEMM = 0,
  BSFP8_OP_LINEAR = 1,
  BSFP8_OP_GROUPED_GEMM = 2,
  BSFP8_OP_FP4_QUANT = 3,
  BSFP8_OP_FP4_GEMM = 4,
  BSFP8_OP_FP8_FP4_GEMM = 5,
  BSFP8_OP_LINEAR_B32 = 6,     /* fp8_linear with (32, 32) weight blocks */
  BSFP8_OP_MOE_DECODE = 7      /* fp8_moe_decode and fp8_fp4_moe_decode  */
} bsfp8_op;

/* Kernels fp8_block_gemm / fp8_linear choose between (bsfp8_gemm_kernel). */
typedef enum {
  BSFP8_GEMM_NONE = 0,          /* empty problem: nothing is launched          */
  BSFP8_GEMM_RESERVED = 1,      /* not returned                                */
  BSFP8_GEMM_TILE_128x256 = 2,  /* LDS-staged MFMA kernel, 128 x 256 tiles     */
  BSFP8_GEMM_TILE_256x256 = 3,  /* LDS-staged MFMA kernel, 256 x 256 tiles     */
  BSFP8_GEMM_DECODE = 4         /* M <= 16: one-launch weight-streaming kernel */
} bsfp8_gemm_kind;

/* Library version (major * 10000 + minor * 100 + patch). */
BSFP8_API int32_t bsfp8_version(void);

/* Static, NUL-terminated description of a status code (never NULL). */
BSFP8_API const char* bsfp8_status_string(int32_t status);

/*
 * fp8_quant_act -- activation quantization in 1 x group_k groups: per-token
 * dynamic scales ([FG-FP8] §一, second bullet; [HF-PT] opening list) or one
 * static calibrated scale ([FG-FP8] §四: activation_scheme "static").
 *
 *   x        bf16 [M][ldx], read-only; only the first K columns are used.
 *   M, K     rows (tokens) and columns (input channels); K % 16 == 0.
 *   ldx      row stride of x in elements, ldx >= K, ldx % 8 == 0.
 *   group_k  group width; must equal the weight block's K size: 128, or
 *            32 for (32, 32) weight blocks ([FG-FP8] §一: the groups line
 *            up with the weight blocks; §九: (32, 32) is a tested
 *            non-default block).  STATIC takes 128 only.
 *   act_scheme  BSFP8_ACT_DYNAMIC: the scales below, per group.
 *               BSFP8_ACT_STATIC: x_scale[0] holds the calibrated
 *               per-tensor scale on entry (fp32 s > 0, or the E8M0 byte
 *               b, s = 2^(b-127)); codes = E4M3(fl32(x/s)) or
 *               E4M3(x * 2^-(b-127)), and every entry of x_scale is set to
 *               that scale, so fp8_block_gemm takes the result unchanged.
 *   scale_fmt   FLOAT: s = fl32(amax/448), codes = E4M3(fl32(x/s)).
 *               UE8M0: s = 2^e, e = ceil(log2(amax/448)) clamped to
 *               [-127,127] ([FG-FP8] §七 note: fp32 scales round *up* to
 *               UE8M0), stored as byte e+127; codes = E4M3(x * 2^-e).
 *               amax = 0 gives s = 1.  E4M3 rounding is to nearest even,
 *               saturating at +-448, sign of zero kept.
 *   xq       out, E4M3 [M][K] (dense).
 *   x_scale  out, [M][ceil(K/group_k)] fp32 (FLOAT) or uint8 (UE8M0); the
 *            dequantization multiplier of each group.
 * Errors: EINVAL (null pointers, M or K < 0, K % 16, ldx < K, ldx % 8,
 * group_k <= 0, bad enum, misalignment); ENOTSUP (group_k other than 128 or
 * 32, or 32 with STATIC).
 */
BSFP8_API int32_t fp8_quant_act(const void* x, int64_t M, int64_t K, int64_t ldx,
                      int32_t group_k, int32_t act_scheme, int32_t scale_fmt,
                      void* xq, void* x_scale, void* stream);

/*
 * fp8_add_rmsnorm_quant -- the step before a layer's linears: the residual's
 * addition, RMS norm and the activation quantization, in one pass.
 *
 *   h  = bf16(x + residual)          (h = x when residual is NULL)
 *   y  = fl32(h * weight / sqrt(mean_k(h^2) + eps))
 *   codes, scales = those of fp8_quant_act's codec (per group_k group, or
 *   the static scale) applied to the fp32 row y, which is not rounded to
 *   bf16 in between.
 * The mean is held in 64 bits and y is the product rounded once, to within
 * 1/2 + (K + 140) 2^-30 units in the last place (rows of a root mean square
 * below 2^100, |y| above 2^-100).
 *
 *   x            bf16 [M][ldx], read-only; K % 16 == 0, ldx >= K, ldx % 8 == 0.
 *   residual     bf16 [M][ldr] or NULL; residual_out bf16 [M][ldr], out: h.
 *                Both or neither; residual_out may be residual itself (the
 *                row is updated in place).  ldr is ignored when NULL.
 *   weight       bf16 [K].
 *   eps          finite, > 0.
 *   group_k, act_scheme, scale_fmt   as for fp8_quant_act.
 *   act_scale    STATIC: the calibrated scale (device; fp32 s > 0, 4-byte
 *                aligned, or the E8M0 byte); every entry of x_scale is set
 *                to it.  DYNAMIC: ignored, may be NULL.
 *   y            out, bf16 [M][K] (the norm rounded to bf16, e.g. for a
 *                router), or NULL.
 *   xq, x_scale  out, as fp8_quant_act; both NULL for the norm alone (then
 *                y is required and the quantization arguments are only
 *                checked).
 * Outputs must not overlap inputs or each other, except residual_out =
 * residual.  NaN and Inf are outside the contract, as for fp8_quant_act, and
 * so are rows in which x + residual, h * weight or y passes the range of its
 * type.
 * Errors: EINVAL (null pointers, sizes, strides, eps, enums, misalignment);
 * ENOTSUP (group_k other than 128 or 32, or 32 with STATIC).
 */
BSFP8_API int32_t fp8_add_rmsnorm_quant(const void* x, int64_t ldx, const void* residual,
                                        void* residual_out, int64_t ldr, const void* weight,
                                        float eps, int64_t M, int64_t K, int32_t group_k,
                                        int32_t act_scheme, int32_t scale_fmt,
                                        const void* act_scale, void* y, void* xq,
                                        void* x_scale, void* stream);

/*
 * moe_route_topk -- a router's scores to each token's k experts and weights,
 * as fp8_moe_decode reads them.  For every row l of the logits:
 *
 *   s   = softmax(l)  or  sigmoid(l)
 *   key = l when bias is NULL and n_group == 1 (both scores rise with l),
 *         else s + bias (bias 0 when NULL), held in 64 bits
 *   n_group > 1: the E experts form n_group groups of E / n_group
 *         neighbours; a group's score is the sum of its two largest keys,
 *         and only the topk_group best groups keep their experts
 *   ids = the k experts with the largest keys, in descending order
 *   weights = s[ids], divided by their sum when renorm is 1, times scale
 * Ties go to the lower expert or group.  An expert whose logit is NaN or
 * -inf, or whose key is, is never chosen (NaN and -inf logits count as
 * score 0); a slot with no expert left gets id -1 and weight 0.  Scores
 * below what 64 bits hold are 0 (sigmoid of logits under about -745, softmax
 * of logits that far below the row's largest), and so are all weights of a
 * token whose chosen scores are.
 *
 *   logits       [T][ldl], fp32 or (logits_bf16 = 1) bf16, ldl >= E, any
 *                ldl; aligned to its type only.
 *   bias         fp32 [E] or NULL: enters the choice, not the weights.
 *   E, k         1 <= k <= E <= 1024, k <= 64.
 *   n_group      divides E, <= 64; 1 <= topk_group <= n_group.
 *   ids          out, int32 [T][k];  weights out, fp32 [T][k].
 * Errors: EINVAL (sizes, null pointers, enums, alignment); ENOTSUP (k > 64,
 * n_group > 64).
 */
BSFP8_API int32_t moe_route_topk(const void* logits, int64_t ldl, int32_t logits_bf16,
                                 const float* bias, int64_t T, int32_t E, int32_t k,
                                 int32_t score, int32_t renorm, float scale, int32_t n_group,
                                 int32_t topk_group, int32_t* ids, float* weights,
                                 void* stream);

/*
 * fp8_quant_weight -- per 2D block weight quantization
 * (weight_block_size = (block_n, block_k), [FG-FP8] §一 first bullet; the
 * scale tensor weight_scale_inv has shape (ceil(N/bn), ceil(K/bk)),
 * [FG-FP8] §一 third paragraph).
 *
 *   w        bf16 [N][ldw] in nn.Linear orientation (out, in); read-only.
 *   N, K     output and input features; K % 16 == 0.
 *   ldw      row stride in elements, ldw >= K, ldw % 8 == 0.
 *   block_n, block_k   (128, 128) or (32, 32) ([FG-FP8] §九); other
 *            positive sizes -> ENOTSUP.
 *   scale_fmt  as for fp8_quant_act, with the amax over the whole block.
 *   wq       out, E4M3 [N][K].
 *   w_scale_inv  out, [ceil(N/bn)][ceil(K/bk)] fp32 or uint8 E8M0.
 * A partial edge block takes its amax over its in-range elements only.
 */
BSFP8_API int32_t fp8_quant_weight(const void* w, int64_t N, int64_t K, int64_t ldw,
                         int32_t block_n, int32_t block_k, int32_t scale_fmt,
                         void* wq, void* w_scale_inv, void* stream);

/*
 * fp8_block_gemm -- the block-scaled FP8 GEMM ([FG-FP8] §一: aligned act
 * groups and weight blocks let the matmul run block by block):
 *
 *   Y[m][n] = bf16_rne( sum_kb S_a[m][kb] * S_w[n/B][kb]
 *                          * sum_{k in kb} Xq[m][k] * Wq[n][k]  + bias[n] )
 *
 * with B the block edge (128, or 32), exact FP8 products, fp32
 * accumulation, the combined scale applied to the fp32 partial sum once per
 * B-wide K block, and the unquantized bias ([FG-FP8] §三: bias is not
 * quantized) added in fp32.
 *
 *   xq, x_scale       as written by fp8_quant_act (M rows).
 *   wq, w_scale_inv   as written by fp8_quant_weight (N rows).
 *   bias              bf16 [N] or NULL.
 *   y                 out, bf16 [M][N].
 *   block_n, block_k  (128, 128), or (32, 32) with 1 x 32 act groups
 *                     (a separate kernel, no workspace).
 *   workspace         device buffer of at least
 *                     bsfp8_workspace_size(BSFP8_OP_BLOCK_GEMM, M, N, K, 0)
 *                     bytes (may be NULL when that size is 0); contents on
 *                     entry are ignored, on exit undefined.
 * Errors: EINVAL (dims < 0, K % 16, N % 8, null required pointers, bad
 * enum, misalignment); ENOTSUP (other block sizes, K > 2^22); ENOSPC.
 * fp8_linear shares these limits (with (32, 32) blocks its workspace is
 * bsfp8_workspace_size(BSFP8_OP_LINEAR_B32, ...)); fp8_grouped_gemm takes
 * (128, 128) and (32, 32) blocks, fp8_grouped_gemm_silu_mul_quant
 * (128, 128) only.
 */
BSFP8_API int32_t fp8_block_gemm(const void* xq, const void* x_scale, const void* wq,
                       const void* w_scale_inv, const void* bias, void* y,
                       int64_t M, int64_t N, int64_t K, int32_t block_n,
                       int32_t block_k, int32_t scale_fmt, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * fp8_linear -- one FP8 linear layer on bf16 activations: fp8_quant_act
 * followed by fp8_block_gemm, i.e. the forward of the pages' FP8Linear
 * ([FG-FP8] §八 step 6).  Results are identical to calling the two entry
 * points in sequence.  For small M the quantization runs inside the GEMM
 * launch; otherwise the quantized activations are staged in `workspace`.
 *
 *   x          bf16 [M][ldx];  other arguments as above.
 *   act_scheme BSFP8_ACT_DYNAMIC (act_scale ignored, may be NULL) or
 *              BSFP8_ACT_STATIC: act_scale is a DEVICE pointer to the
 *              calibrated per-tensor scale (fp32 s > 0, 4-byte aligned, or
 *              the E8M0 byte), read-only; the result equals fp8_quant_act
 *              with the static scheme and that scale, then fp8_block_gemm.
 *              STATIC takes 128 x 128 blocks only (ENOTSUP otherwise);
 *              a NULL act_scale is EINVAL.
 *   workspace  >= bsfp8_workspace_size(BSFP8_OP_LINEAR, M, N, K, 0) bytes
 *              (the same for both schemes).
 */
BSFP8_API int32_t fp8_linear(const void* x, int64_t ldx, const void* wq,
                   const void* w_scale_inv, const void* bias, void* y,
                   int64_t M, int64_t N, int64_t K, int32_t block_n,
                   int32_t block_k, int32_t act_scheme, int32_t scale_fmt,
                   const void* act_scale, void* workspace, size_t workspace_bytes,
                   void* stream);

/* Bytes of the device array that fp8_linear_noalloc takes as its workspace
   (one array per GPU the library runs on, held until the process ends). */
#define BSFP8_NOALLOC_SCRATCH_BYTES (32u << 20)

/*
 * fp8_linear_noalloc -- fp8_linear for callers that cannot allocate device
 * memory: code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc.  Same arguments and results as fp8_linear, without the
 * workspace: the library uses a device array of BSFP8_NOALLOC_SCRATCH_BYTES
 * of its own (looked up once per device), and calls no allocating routine.
 *   - Every call on one GPU shares that GPU's array, which keeps the last
 *     call's contents; calls that overlap on one GPU (different streams
 *     without ordering) race and give undefined results.
 *   - Errors: those of fp8_linear, and ENOSPC when
 *     bsfp8_workspace_size(BSFP8_OP_LINEAR or BSFP8_OP_LINEAR_B32, M, N, K, 0)
 *     exceeds BSFP8_NOALLOC_SCRATCH_BYTES (use fp8_linear then).
 */
BSFP8_API int32_t fp8_linear_noalloc(const void* x, int64_t ldx, const void* wq,
                                     const void* w_scale_inv, const void* bias, void* y,
                                     int64_t M, int64_t N, int64_t K, int32_t block_n,
                                     int32_t block_k, int32_t act_scheme, int32_t scale_fmt,
                                     const void* act_scale, void* stream);

/*
 * fp8_grouped_gemm -- MoE expert GEMM over contiguous per-expert row
 * segments ([FG-FP8] §一 FP8Experts; §6.4 and §七 expert backends).  For
 * every expert e, rows [off[e], off[e+1]) of Y are the fp8_block_gemm of the
 * same rows of (xq, x_scale) with expert e's (wq[e], w_scale_inv[e]).
 *
 *   xq           E4M3 [T][K];  x_scale [T][ceil(K/B)] (fp32 | UE8M0).
 *   wq           E4M3 [E][N][K];  w_scale_inv [E][ceil(N/B)][ceil(K/B)].
 *   block_n, block_k  (B, B) = (128, 128), or (32, 32) with 1 x 32 act
 *                groups ([FG-FP8] §九); other sizes ENOTSUP.
 *   seg_offsets  DEVICE int32 [E+1]: off[0] = 0, nondecreasing, off[E] = T.
 *                This is a precondition and is not checked (checking would
 *                need a device synchronisation).
 *   E            number of experts, 1 <= E <= 1024.
 *   y            out, bf16 [T][N]; rows of empty segments do not exist.
 *   workspace    >= bsfp8_workspace_size(BSFP8_OP_GROUPED_GEMM, T, N, K, E).
 */
BSFP8_API int32_t fp8_grouped_gemm(const void* xq, const void* x_scale, const void* wq,
                         const void* w_scale_inv, const int32_t* seg_offsets,
                         int32_t E, void* y, int64_t T, int64_t N, int64_t K,
                         int32_t block_n, int32_t block_k, int32_t scale_fmt,
                         void* workspace, size_t workspace_bytes, void* stream);

/*
 * fp8_grouped_gemm_silu_mul_quant -- an MoE expert MLP's gate/up GEMM with
 * the step to the down GEMM fused into its epilogue: the gate/up/down MLP
 * of [NVFP4] (layer-wise quantization section) run as FP8 experts
 * ([FG-FP8] §一 FP8Experts, §6.4), the down projection's input quantized
 * per token in 1 x 128 groups like any activation ([FG-FP8] §一).
 * For every expert e and row t in [off[e], off[e+1]):
 *   g = (X W_e[0:I]^T)[t],  u = (X W_e[I:2I]^T)[t]   (fp32 accumulation),
 *   h = bf16(silu(g) * u),  silu(g) = g / (1 + e^-g),
 *   (hq, h_scale) = the 1 x 128 activation quantization of h (the codes
 *   and scales fp8_quant_act writes for that bf16 row), in scale_fmt.
 * The result feeds fp8_grouped_gemm (the down projection) unchanged.
 *
 *   xq, x_scale  as fp8_grouped_gemm (K input channels, 1 x 128 groups).
 *   wq           E4M3 [E][2I][K]: rows [0, I) gate, rows [I, 2I) up;
 *                w_scale_inv [E][2I/128][ceil(K/128)] (fp32 | UE8M0).
 *   seg_offsets  DEVICE int32 [E+1], the same precondition as
 *                fp8_grouped_gemm.
 *   hq           out, E4M3 [T][I] (16-byte aligned);  h_scale out,
 *                [T][I/128] fp32 | UE8M0.
 *   h_bf16       out, bf16 [T][I] (the rounded h), or NULL.
 *   I            intermediate size, a positive multiple of 128.
 * No workspace.  Errors: those of fp8_grouped_gemm with N = 2I; EINVAL for
 * I <= 0 or I % 128 != 0, a null or misaligned h_scale (4 bytes) or a
 * misaligned h_bf16 (16 bytes); ENOTSUP when one expert's weight (2 I K
 * bytes) exceeds 2^31 - 1 bytes.
 */
BSFP8_API int32_t fp8_grouped_gemm_silu_mul_quant(const void* xq, const void* x_scale,
                                        const void* wq, const void* w_scale_inv,
                                        const int32_t* seg_offsets, int32_t E, void* hq,
                                        void* h_scale, void* h_bf16, int64_t T, int64_t I,
                                        int64_t K, int32_t scale_fmt, void* stream);

/*
 * fp8_moe_decode -- a whole MoE layer for a few tokens, straight from the
 * tokens' expert ids (no sorting, no segment offsets):
 *
 *   slot (t, j) with e = ids[t][j] in [0, E):
 *     g = (X W13_e[0:I]^T)[t],  u = (X W13_e[I:2I]^T)[t]
 *     (hq, hs) = the 1 x 128 activation quantization of bf16(silu(g) * u)
 *     d(t, j)  = hq W2_e^T                                  (fp32)
 *   y[t] = bf16_rne( addend[t] + sum_j weights[t][j] * d(t, j) )
 *
 * that is fp8_grouped_gemm_silu_mul_quant, fp8_grouped_gemm and the
 * weighted sum, without rounding d to bf16.  An expert that some token
 * names is read once for every 16 of its slots (32, FP8 also 64, where
 * experts have more than 10, 20 slots each on average).  From some 8 (experts
 * of 7168 x 2048) to 32 (4096 x 14336) slots an expert on average on, the
 * sorted path's two GEMMs take less time.
 * Deterministic: the same call gives the same bits.
 *
 *   xq, x_scale  as written by fp8_quant_act or fp8_add_rmsnorm_quant
 *                (T rows of H, 1 x 128 groups).
 *   ids          DEVICE int32 [T][k];  weights DEVICE fp32 [T][k].  A slot
 *                whose id is outside [0, E) is skipped and its weight not
 *                used: padding tokens, or experts that live on another
 *                device.  A token may name an expert more than once.
 *   w13          E4M3 [E][2I][H], gate rows then up rows; w13_scale
 *                [E][2I/128][ceil(H/128)] (fp32 | UE8M0).
 *   w2           E4M3 [E][H][I]; w2_scale [E][ceil(H/128)][I/128].
 *   addend       bf16 [T][H] (a shared expert's output, or the residual)
 *                or NULL; may be y itself.
 *   y            out, bf16 [T][H]; a token with no slot left gets its
 *                addend, or 0.
 *   T <= 128, k <= 16 (ENOTSUP beyond: sort the rows and use
 *   fp8_grouped_gemm); H % 16 == 0, I % 128 == 0, 1 <= E <= 1024.
 *   workspace    >= bsfp8_workspace_size(BSFP8_OP_MOE_DECODE, T * k, H, I, 0);
 *                nothing in it is kept from one call to the next.  Calls that
 *                may overlap need one each.
 * y must not overlap an input other than addend, nor the workspace.
 * Errors: EINVAL (sizes, null pointers, enums, misalignment); ENOTSUP (T, k,
 * H or I > 2^22, T k I > 2^30); ENOSPC.
 */
BSFP8_API int32_t fp8_moe_decode(const void* xq, const void* x_scale, const int32_t* ids,
                                 const float* weights, const void* w13, const void* w13_scale,
                                 const void* w2, const void* w2_scale, const void* addend,
                                 void* y, int64_t T, int32_t k, int64_t H, int64_t I, int32_t E,
                                 int32_t scale_fmt, void* workspace, size_t workspace_bytes,
                                 void* stream);

/*
 * fp8_fp4_moe_decode -- fp8_moe_decode with MXFP4 expert weights (those of
 * fp8_fp4_grouped_gemm):
 *   w13          uint8 [E][2I][H/2], w13_scale E8M0 bytes [E][2I][H/32];
 *   w2           uint8 [E][H][I/2],  w2_scale  E8M0 bytes [E][H][I/32]
 * as mxfp4_quant_weight writes them per expert; H % 32 == 0.  scale_fmt is
 * that of x_scale and of h's scales.  The rest as fp8_moe_decode.
 */
BSFP8_API int32_t fp8_fp4_moe_decode(const void* xq, const void* x_scale, const int32_t* ids,
                                     const float* weights, const void* w13,
                                     const void* w13_scale, const void* w2,
                                     const void* w2_scale, const void* addend, void* y,
                                     int64_t T, int32_t k, int64_t H, int64_t I, int32_t E,
                                     int32_t scale_fmt, void* workspace, size_t workspace_bytes,
                                     void* stream);

/*
 * rope_inv_freq -- the table of rotary angles per position:
 *
 *   theta_i = base^(-2 i / rot_dim),  i < rot_dim / 2
 *   PLAIN     theta_i
 *   LINEAR    theta_i / factor  (positions interpolated)
 *   BY_PARTS  theta_i g + theta_i / factor (1 - g), with
 *             g = clamp((orig_len theta_i / (2 pi) - low) / (high - low), 0, 1):
 *             what turns `high` times or more within the original context
 *             keeps its angle, what turns `low` times or less is interpolated
 *             (YaRN's "NTK-by-parts", arXiv 2309.00071)
 *
 * in 64 bits, rounded once to fp32.
 *
 *   rot_dim   rot_dim % 16 == 0, <= 256.  base >= 1.
 *   factor    > 0, for LINEAR and BY_PARTS;  0 <= low < high and orig_len > 0
 *             for BY_PARTS.  What a scaling does not use is not looked at.
 *   inv_freq  out, fp32 [rot_dim / 2].
 * Errors: EINVAL; ENOTSUP (rot_dim > 256).
 */
BSFP8_API int32_t rope_inv_freq(int32_t scaling, int64_t rot_dim, double base, double factor,
                                double low, double high, double orig_len, float* inv_freq,
                                void* stream);

/*
 * rope_kv_append -- rotary positions for queries and keys, and keys and
 * values into a paged cache:
 *
 *   t = positions[row] inv_freq[i]
 *   a' = mscale (a cos t - b sin t),  b' = mscale (b cos t + a sin t)
 *
 * for the pairs (a, b) = (x[i], x[i + rot_dim/2]) or, interleaved,
 * (x[2i], x[2i+1]) of each head's first rot_dim values; the others stay.
 *   q_out  = bf16_rne(q')
 *   cache: KV_BF16  bf16_rne(k'), v
 *          KV_FP8_* per token and head the codes and the scale that
 *          fp8_quant_act gives a group of the D values of k' (in fp32, not
 *          rounded to bf16 before) or v, in scale_fmt FLOAT or UE8M0
 *
 *   q, q_out   bf16 [T][Hq][D], row strides ldq and ldqo; q_out may be q, or
 *              lie apart from it.  Both NULL: no queries.
 *   k, v       bf16 [T][Hkv][D], row strides ldk and ldv.  Both NULL: no
 *              cache (slots and the caches are not looked at).
 *   positions  DEVICE int32 [T];  inv_freq DEVICE fp32 [rot_dim / 2].  The
 *              angle is taken in 64 bits (exact for positions below 2^29).
 *              rot_dim 0: neither is looked at.
 *   slots      DEVICE int64 [T]: page * page_size + place in the page; a token
 *              whose slot is negative or >= num_pages * page_size is not
 *              cached (padding), its query is rotated.  Slots of one call
 *              must differ: of two tokens with the same one, parts of either
 *              may stay.
 *   k_cache, v_cache   [num_pages][Hkv][page_size][D] E4M3 bytes or bf16.
 *   k_scale, v_scale   [num_pages][Hkv][page_size] fp32 or E8M0 bytes; not
 *              looked at for KV_BF16.
 *   D 64, 128 or 256 (else ENOTSUP); rot_dim % 16 == 0, <= D; Hq, Hkv <= 1024;
 *   page_size a power of two from 16 on (else ENOTSUP); row strides % 8 == 0.
 * Values that are not finite are outside the contract of KV_FP8_*, as for
 * fp8_quant_act, and reach their own token's heads only.
 * Errors: EINVAL; ENOTSUP.
 */
BSFP8_API int32_t rope_kv_append(const void* q, int64_t ldq, void* q_out, int64_t ldqo,
                                 const void* k, int64_t ldk, const void* v, int64_t ldv,
                                 const int32_t* positions, const float* inv_freq, int64_t rot_dim,
                                 int32_t interleaved, float mscale, const int64_t* slots,
                                 int64_t T, int32_t Hq, int32_t Hkv, int32_t D, int32_t kv_fmt,
                                 int64_t num_pages, int32_t page_size, void* k_cache,
                                 void* v_cache, void* k_scale, void* v_scale, void* stream);

/*
 * paged_attn -- causal attention of each sequence's newest tokens over the
 * paged cache (which holds their own keys and values too):
 *
 *   y[t][h] = bf16_rne( sum_j e^(s_j) v_j / sum_j e^(s_j) ),
 *   s_j = scale q[t][h] . k_j      (key head h / (Hq / Hkv))
 *
 * Sequence b has the tokens [q_start[b], q_start[b+1]) and sees prefix_len
 * keys that all sequences share, then kv_len[b] of its own; its last token
 * stands at position prefix_len + kv_len[b] - 1, the others before it.  A
 * token sees the keys at its own position and before, with a window only the
 * last `window` of these (itself among them).  No key seen: y = 0.  The
 * prefix's keys and values are read once per 16 to 256 query rows of the batch
 * (tokens times query heads of a key head), not once per sequence.  Deterministic: the same call gives the same bits.
 *
 *   q           bf16 [T][Hq][D], row stride ldq (ldq % 8 == 0).
 *   q_start     DEVICE int32 [B+1], not decreasing (else y stays as it is),
 *               or NULL: one token per sequence (T == B).  Rows of y before
 *               q_start[0] and from q_start[B] on stay as they are; what is
 *               outside [0, T] counts as its nearer end.
 *   kv_len      DEVICE int32 [B]; negative counts as 0, more than
 *               max_pages * page_size as that.
 *   page_table  DEVICE int32 [B][max_pages]: pages of the own keys in order.
 *               Entries that no key needs are not used.  Keys of a page
 *               outside [0, num_pages) count as not seen.
 *   prefix_table  DEVICE int32 [ceil(prefix_len / page_size)], the same for
 *               the prefix; own keys begin on a page of their own.  Not
 *               looked at for prefix_len 0.
 *   k_cache .. kv_fmt, num_pages, page_size   as rope_kv_append writes them;
 *               value scales beyond 2^75 and bf16 values beyond 2^83 are
 *               outside the contract (sums of e^(s_j) v_j are fp32), scales
 *               below 2^-85 lose precision; 0 is a value of zeros.  A key
 *               whose e^(s_j) is below 2^-126 of the largest adds nothing.
 *               What they hold behind a sequence's or the prefix's last key,
 *               or before the window, reaches no result, NaN and infinities
 *               included; a key or value that a row sees and that is not finite
 *               leaves the row, or its elements, infinite or NaN.
 *   scale       > 0; scores beyond fp32's range are outside the contract.
 *   window      0: none.
 *   y           out, bf16 [T][Hq][D] (dense); must not overlap an input.
 *   workspace   >= paged_attn_workspace_size(...) bytes, 16-byte aligned;
 *               nothing in it is kept from one call to the next.  Calls that
 *               may overlap need one each.
 *   D 64, 128 or 256; page_size a power of two from 16 on; B <= 4096;
 *   max_pages * page_size and prefix_len <= 2^30 (ENOTSUP beyond);
 *   Hq % Hkv == 0, Hq <= 1024.
 * The launches depend on the sizes above alone, not on what kv_len, q_start
 * and the tables hold: a captured call serves other lengths.
 * Errors: EINVAL; ENOTSUP (also sizes whose partial results cannot be counted
 * in 32 bits); ENOSPC.
 */
BSFP8_API int32_t paged_attn(const void* q, int64_t ldq, const int32_t* q_start,
                             const int32_t* kv_len, const int32_t* page_table, int64_t max_pages,
                             const int32_t* prefix_table, int64_t prefix_len, const void* k_cache,
                             const void* v_cache, const void* k_scale, const void* v_scale,
                             int32_t kv_fmt, int64_t num_pages, int32_t page_size, int64_t T,
                             int64_t B, int32_t Hq, int32_t Hkv, int32_t D, float scale,
                             int64_t window, void* y, void* workspace, size_t workspace_bytes,
                             void* stream);

/* Bytes of workspace of paged_attn; (size_t)-1 for sizes that it refuses. */
BSFP8_API size_t paged_attn_workspace_size(int64_t T, int64_t B, int32_t Hq, int32_t Hkv,
                                           int32_t D, int64_t max_pages, int32_t page_size,
                                           int64_t prefix_len);

/*
 * fp4_quant -- NVFP4-style quantization ([NVFP4]: 4-bit float weights and
 * input activations in 16-element groups, group_size 16): E2M1 codes with
 * an E4M3 scale per 16-element group and one fp32 scale per tensor.
 *
 *   g   = fl32(amax_tensor / 2688)  (1.0 for an all-zero tensor)
 *   sg  = E4M3(fl32(amax_group / fl32(6 g)))
 *   eff = fl32(dec(sg) * g);  codes = E2M1(fl32(x / eff)), 0 when eff == 0
 *
 *   x          bf16 [R][K], K % 32 == 0.
 *   dynamic_tscale  1: compute g from x and write it to *tscale;
 *                   0: read g from *tscale (must be > 0, finite).
 *   q4         out, uint8 [R][K/2]; element 2i in the low nibble of byte i.
 *   gscale     out, E4M3 [R][K/16].
 *   tscale     DEVICE float[1], out (dynamic) or in (static).
 *   workspace  >= bsfp8_workspace_size(BSFP8_OP_FP4_QUANT, R, 0, K, 0).
 */
BSFP8_API int32_t fp4_quant(const void* x, int64_t R, int64_t K, int32_t dynamic_tscale,
                  void* q4, void* gscale, float* tscale, void* workspace,
                  size_t workspace_bytes, void* stream);

/*
 * fp4_group_gemm -- GEMM of two NVFP4-style operands (the MLP projections of
 * [NVFP4]):
 *
 *   Y[m][n] = bf16_rne( g_a g_w sum_k dec(qa[m][k]) dec(sa[m][k/16])
 *                                    * dec(qw[n][k]) dec(sw[n][k/16]) )
 *
 *   xq4, x_gscale, x_tscale   as written by fp4_quant for X (M rows).
 *   wq4, w_gscale, w_tscale   as written by fp4_quant for W (N rows).
 *   y                          out, bf16 [M][N].  K % 32 == 0.
 *   workspace  >= bsfp8_workspace_size(BSFP8_OP_FP4_GEMM, M, N, K, 0).
 * Errors: EINVAL (sizes, null pointers, misalignment), ENOTSUP (K > 2^22,
 * the bound of the FP8 GEMMs), ENOSPC (workspace).
 */
BSFP8_API int32_t fp4_group_gemm(const void* xq4, const void* x_gscale,
                       const float* x_tscale, const void* wq4,
                       const void* w_gscale, const float* w_tscale, void* y,
                       int64_t M, int64_t N, int64_t K, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * mxfp4_quant_weight -- FP4-packed weights with UE8M0 block scales, the
 * V4-style expert weights the pages' FP8-activation x FP4-weight linear
 * consumes ([FG-FP8] §一 FP4-packed experts, §6.1 deepgemm_fp8_fp4_linear;
 * UE8M0 scales §七).  Per 1 x 32 group along K of each row:
 *   e = ceil(log2(amax/6)) clamped to [-127,127] (0 for amax = 0), stored
 *   as the byte e+127;  codes = E2M1(w * 2^-e), round to nearest even.
 *
 *   w        bf16 [N][ldw], K % 32 == 0, ldw >= K, ldw % 8 == 0.
 *   wq4      out, uint8 [N][K/2]: element 2i in the low nibble of byte i.
 *   w_scale  out, E8M0 bytes [N][K/32].
 * Errors: EINVAL (sizes, null pointers, misalignment).
 */
BSFP8_API int32_t mxfp4_quant_weight(const void* w, int64_t N, int64_t K, int64_t ldw,
                                     void* wq4, void* w_scale, void* stream);

/*
 * fp8_fp4_gemm -- FP8 activations x MXFP4 weights ([FG-FP8] §6.1, the
 * FP8 x FP4 linear), on gfx950's scaled MFMA with the weights as its FP4
 * operand and their E8M0 group scales as its block scales:
 *
 *   Y[m][n] = bf16( sum_k E4M3(xq[m][k]) S_a[m][k/128]
 *                         * E2M1(wq4[n][k]) 2^(w_scale[n][k/32]-127) + bias[n] )
 *
 *   xq, x_scale  as written by fp8_quant_act (1 x 128 groups; scale_fmt
 *                FLOAT or UE8M0).
 *   wq4, w_scale as written by mxfp4_quant_weight (N rows).
 *   bias         bf16 [N] or NULL;  y out, bf16 [M][N].
 *   K % 32 == 0, N % 8 == 0, K <= 2^22.
 *   workspace    >= bsfp8_workspace_size(BSFP8_OP_FP8_FP4_GEMM, M, N, K, 0).
 * M <= 16 streams the weights in one launch (half the bytes of FP8);
 * larger M runs the LDS MFMA kernel on 128 x 256 tiles, K split as for
 * fp8_block_gemm.  Errors as fp8_block_gemm (block sizes are fixed here).
 */
BSFP8_API int32_t fp8_fp4_gemm(const void* xq, const void* x_scale, const void* wq4,
                               const void* w_scale, const void* bias, void* y, int64_t M,
                               int64_t N, int64_t K, int32_t scale_fmt, void* workspace,
                               size_t workspace_bytes, void* stream);

/*
 * fp8_fp4_grouped_gemm -- MoE expert GEMM with FP4-packed expert weights
 * ([FG-FP8] §一: FP8Experts can take V4-style FP4-packed expert weights;
 * §6.1 and §6.4: the FP8 x FP4 linear and the grouped expert GEMMs of the
 * fast backend).  For every expert e, rows [off[e], off[e+1]) of Y are the
 * fp8_fp4_gemm of the same rows of (xq, x_scale) with expert e's MXFP4
 * weights (wq4[e], w_scale[e]):
 *
 *   Y[t][n] = bf16( sum_k E4M3(xq[t][k]) S_a[t][k/128]
 *                         * E2M1(wq4[e][n][k]) 2^(w_scale[e][n][k/32]-127) )
 *
 *   xq, x_scale  as written by fp8_quant_act (T rows; FLOAT or UE8M0).
 *   wq4          uint8 [E][N][K/2] (mxfp4_quant_weight per expert);
 *   w_scale      E8M0 bytes [E][N][K/32].
 *   seg_offsets  DEVICE int32 [E+1], the precondition of fp8_grouped_gemm.
 *   E            1 <= E <= 1024;  y out, bf16 [T][N].
 *   K % 32 == 0, N % 8 == 0, K <= 2^22.  No workspace.
 * Errors as fp8_grouped_gemm (block sizes are fixed here).
 */
BSFP8_API int32_t fp8_fp4_grouped_gemm(const void* xq, const void* x_scale, const void* wq4,
                                       const void* w_scale, const int32_t* seg_offsets,
                                       int32_t E, void* y, int64_t T, int64_t N, int64_t K,
                                       int32_t scale_fmt, void* stream);

/*
 * fp8_dequant_weight -- fold the block scales back into the weights, the
 * dequantize-on-load step for pre-quantized checkpoints ([FG-FP8] §五,
 * Fp8Dequantize):  W[n][k] = bf16_rne(fl32(E4M3(wq[n][k]) * S_w[n/B][k/B]))
 * for (B, B) blocks, B = 128 or 32.
 *
 *   wq           E4M3 [N][K], K % 16 == 0.
 *   w_scale_inv  [ceil(N/B)][ceil(K/B)] fp32 or UE8M0 bytes.
 *   w            out, bf16 [N][K].
 * Codes 0x7F / 0xFF (E4M3 NaN) and the E8M0 byte 0xFF are outside the
 * contract.  Errors: EINVAL (sizes, null pointers, misalignment, bad enum);
 * ENOTSUP (block sizes other than (128, 128) and (32, 32)).
 */
BSFP8_API int32_t fp8_dequant_weight(const void* wq, int64_t N, int64_t K, int32_t block_n,
                                     int32_t block_k, int32_t scale_fmt,
                                     const void* w_scale_inv, void* w, void* stream);

/*
 * fp8_scale_to_ue8m0 -- power-of-two scales stored in float32 containers to
 * the one-byte UE8M0 form the kernels read, exactly ([FG-FP8] §七: such
 * checkpoints are converted on load).  scale[i] = 2^k with -127 <= k <= 127
 * becomes the byte k + 127; any other value (not a power of two, <= 0,
 * outside that range, Inf, NaN) becomes 0xFF, the E8M0 NaN encoding, which
 * callers can test for.
 *
 *   scale  device fp32 [n];  out  device uint8 [n].
 */
BSFP8_API int32_t fp8_scale_to_ue8m0(const float* scale, int64_t n, void* out, void* stream);

/*
 * Bytes of device workspace the given operation needs for this problem
 * (0 if none).  `op` is a bsfp8_op; M is T for the grouped GEMM, R for
 * fp4_quant and T * k for the MoE layer (N = H, K = I); E is used by the
 * grouped GEMM only.  Returns (size_t)-1 for an
 * unknown op or negative sizes.
 */
BSFP8_API size_t bsfp8_workspace_size(int32_t op, int64_t M, int64_t N, int64_t K,
                            int32_t E);

/*
 * Which kernel (a bsfp8_gemm_kind) fp8_block_gemm and fp8_linear launch for
 * an M x N x K problem with 128 x 128 blocks (fp8_fp4_gemm follows the same
 * choice; (32, 32) blocks run their own kernel, the decode kernel up to
 * M = 16), and into how many K splits it cuts K (*splits, may
 * be NULL; 1 when K is not split: splits above 1 write fp32 partial sums to
 * the workspace and add one reduction launch).  The grouped GEMM does not
 * split K: experts with more than 128 rows run on 256 x 256 tiles and the
 * others on 64 x 256 tiles, in two launches.  Host-only, touches no device.
 * Returns -1 for negative sizes.
 */
BSFP8_API int32_t bsfp8_gemm_kernel(int64_t M, int64_t N, int64_t K, int32_t* splits);

#ifdef __cplusplus
}
#endif

#endif /* BSFP8_H */
