/*
 * qa.h -- C ABI of libqa, quantized linear layers for AMD Instinct MI355X
 * (gfx950, CDNA4).
 *
 * Quantized linear layers of LLM inference:
 *   - LLM.int8() mixed precision: feature columns whose activation magnitude
 *     exceeds a threshold stay in fp16, all other columns are quantized to
 *     int8 with vector-wise absmax scales (per token for X, per output
 *     channel for W), multiplied with int32 accumulation, dequantized by the
 *     outer product of the scales and summed with the fp16 outlier product.
 *   - FlatQuant's Kronecker transform (P = P1 (x) P2) fused with int4
 *     quantization, feeding the same W4A4 GEMM.
 *   - W4A4 group Hadamard: each G-wide block of the K dimension is rotated by
 *     the normalized Hadamard matrix, quantized to int4 (dynamic per-token
 *     scales for X, per-row-per-group scales for W), packed eight per 32-bit
 *     word, multiplied with int32 accumulation per group and dequantized.
 *   - SmoothQuant W8A8: activation columns are divided by per-channel
 *     migration factors and the weight's input channels multiplied by them,
 *     so both quantize to int8 with plain absmax scales (per token or per
 *     tensor for X, per output channel for W) and no fp16 branch.
 *   - Around them: the norm that makes a linear's codes, routing to experts,
 *     the experts' gated feed-forward on int8 codes, an int8 projection
 *     with the low-rank adapters of many requests, an int8 linear with bias,
 *     activation and residual, and a paged cache of keys and values in int8 or
 *     int4 codes with the attention of single tokens over it.
 *
 * Sources, cited by page title and section:
 *   [AIInfra-Q01]  Infrasys-AI "AIInfra" notes, page 05Quantization01 (模型量化):
 *                  the LLM.int8() method -- outlier detection, "a. 向量级量化",
 *                  "b. INT8 矩阵乘法与反量化", merge of the two parts.
 *                  Its advice for training: decompose the largest-magnitude
 *                  1-2% of feature dimensions instead of about 0.1% (top-k).
 *                  Its FlatQuant section: the apply stage reshapes each token
 *                  to X~ [n1 x n2] and computes X~ x1 P1^T x2 P2 with
 *                  P = P1 (x) P2, fused with dynamic int4 quantization; the
 *                  sizes minimize n1 + n2 (8192 -> 64 x 128).
 *   [Scholia-IQ]   "模型推理量化" (Inference Quantization notes): §4 Scale,
 *                  §5 Outlier, §6 Zero-point (§6.2 affine clip), §7 Granularity.
 *   [GroupRot]     "低比特量化加速：分组旋转方法从W8A8到W4A4的实践与展望":
 *                  §二 normalized Hadamard, §5.1 weight transform and storage,
 *                  §5.2 online activation transform fused with quantization,
 *                  §5.4 packing and int32 accumulation.
 *   [QE2]          "Quantization explained, part 2" (tanjunchen.github.io),
 *                  §1.2: threshold 6.0 on a channel's activation magnitude;
 *                  §4.2: SmoothQuant, the per-input-channel migration
 *                  X W = (X diag(s)^-1)(diag(s) W), s_j = max|X_j|^alpha /
 *                  max|W_j|^(1-alpha); §4.4: factors fixed offline.
 *
 * Conventions shared by every entry point:
 *   - All array arguments are DEVICE pointers allocated and owned by the
 *     caller; the library allocates nothing and keeps no per-call state.
 *   - Matrices are row-major.  X is [M x K] (tokens x in-features), W is
 *     [N x K] (out-features x in-features), the output is [M x N].
 *   - fp16 / bf16 arrays are passed as `const void*` holding IEEE binary16 /
 *     bfloat16 bit patterns.
 *   - `stream` is a hipStream_t (NULL: the default stream).  Every call is
 *     asynchronous and stream-ordered; nothing synchronizes the host.
 *   - Every argument check runs before any HIP call.  On error nothing is
 *     launched and outputs are untouched.  Device faults surface at the
 *     caller's next synchronization.
 *   - Sizes and scalar arguments are checked first.  M == 0 or N == 0 (an
 *     empty batch or layer; rows == 0 for the quantizers) is then a valid
 *     no-op, and the pointers of empty arrays may be NULL.
 *   - Inputs must be finite (NaN / Inf are not checked on the hot path).
 *   - Rounding: scales are fl32(absmax / q_max) with IEEE correctly rounded
 *     division (1.0 when absmax is 0, [Scholia-IQ §4]); codes are
 *     clip(rint(fl32(x / s)) + z, q_min, q_max) with ties to even.
 */
#ifndef QA_H
#define QA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    QA_OK = 0,
    QA_ERR_NULL = 1,        /* a required pointer is NULL */
    QA_ERR_SHAPE = 2,       /* negative size, K not a multiple of the required step, bad G */
    QA_ERR_ALIGN = 3,       /* a pointer is not 16-byte aligned */
    QA_ERR_VALUE = 4,       /* q_min > q_max, range outside the code type, NaN threshold, ... */
    QA_ERR_WORKSPACE = 5,   /* workspace smaller than the matching *_workspace() size */
    QA_ERR_UNSUPPORTED = 6, /* a valid request that this library has no kernel for */
    QA_ERR_DEVICE = 7       /* a HIP launch failed; see qa_last_error() */
} qa_status;

typedef enum { QA_F32 = 0, QA_F16 = 1, QA_BF16 = 2 } qa_dtype;

typedef enum { QA_SCALE_PER_ROW = 0, QA_SCALE_PER_GROUP = 1, QA_SCALE_PER_TENSOR = 2 } qa_scale_mode;

/* SmoothQuant side: activations are divided by the factors, weights multiplied. */
typedef enum { QA_SMOOTH_DIVIDE = 0, QA_SMOOTH_MULTIPLY = 1 } qa_smooth_op;

/* Human-readable name of a status code (static string). */
const char* qa_status_string(qa_status s);

/* Detail of the last error raised on the calling thread ("" if none). */
const char* qa_last_error(void);

/* ---------------------------------------------------------------------------
 * Outlier feature columns  [AIInfra-Q01, LLM.int8() detection step; QE2 §1.2]
 *
 * colmax[j] = max_i |X[i][j]| (fp16 widened exactly to fp32).  Column j is an
 * outlier when colmax[j] > threshold (strict; threshold compared in fp32).
 *   X       fp16 [M x K]
 *   mask    u8 [K]: 1 for an outlier column, else 0
 *   idx     i32 [K]: the outlier columns in ascending order in idx[0..count)
 *           (entries from count on are unspecified)
 *   count   i32 [1]: number of outlier columns
 *   colmax  f32 [K] or NULL
 *   scratch device buffer of qa_outlier_cols_workspace(K) bytes (any content)
 * Errors: NULL pointers, M < 0, K <= 0, K > 2^22, K % 8 != 0, X not 16-byte
 * aligned, NaN threshold, small scratch.
 * ------------------------------------------------------------------------- */
size_t qa_outlier_cols_workspace(int64_t K);
qa_status qa_outlier_cols(const void* X_f16, int64_t M, int64_t K, float threshold,
                          uint8_t* mask, int32_t* idx, int32_t* count, float* colmax_or_null,
                          void* scratch, size_t scratch_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Top-k outlier columns  [AIInfra-Q01: decompose the largest-magnitude 1-2%
 * of feature dimensions]
 *
 * Same outputs as qa_outlier_cols, but the set is the k columns with the
 * largest colmax[j] = max_i |X[i][j]|; equal maxima are taken in ascending
 * column order, so exactly k columns are chosen.  k = ceil(p K) decomposes
 * the share p of the dimensions.
 *   scratch qa_outlier_cols_workspace(K) bytes (any content)
 * Errors: as qa_outlier_cols, plus K > 32768 (QA_ERR_SHAPE), k < 0 or
 * k > K (QA_ERR_VALUE).
 * ------------------------------------------------------------------------- */
qa_status qa_outlier_topk(const void* X_f16, int64_t M, int64_t K, int64_t k, uint8_t* mask, int32_t* idx,
                          int32_t* count, float* colmax_or_null, void* scratch, size_t scratch_bytes,
                          void* stream);

/* ---------------------------------------------------------------------------
 * Row-wise int8 quantization  [AIInfra-Q01 "a. 向量级量化"; Scholia-IQ §4,
 * §6.2]
 *
 * One scale per row of X [rows x K] (per token for activations, per output
 * channel for a weight [N x K]).
 *   Dynamic (s_in == NULL): s[r] = absmax over the unmasked columns of row r
 *     divided by q_max (1.0 if that absmax is 0), z = 0, written to s_out[r].
 *     Requires q_max > 0 and z_in == NULL.
 *   Static (s_in != NULL): s = s_in[r] (> 0, finite: not checked),
 *     z = z_in ? z_in[r] : 0; s_out is ignored.
 *   Xq[r][j] = clip(rint(x / s) + z, q_min, q_max); a masked column j
 *     (mask[j] != 0) is skipped by the absmax and receives clip(z).
 *   X       fp16 [rows x K]; mask u8 [K] or NULL; Xq i8 [rows x K]
 * Errors: NULL X / Xq (or s_out in dynamic mode), rows < 0, K <= 0,
 * K > 2^26, K % 8 != 0, X or Xq not 16-byte aligned, q_min > q_max, range outside
 * [-128, 127], dynamic mode with q_max <= 0 or z_in != NULL.
 * ------------------------------------------------------------------------- */
qa_status qa_quantize_rowwise_int8(const void* X_f16, int64_t rows, int64_t K,
                                   const uint8_t* mask_or_null, int32_t q_min, int32_t q_max,
                                   const float* s_in_or_null, const int32_t* z_in_or_null,
                                   int8_t* Xq, float* s_out_or_null, void* stream);

/* ---------------------------------------------------------------------------
 * LLM.int8() mixed-precision linear  [AIInfra-Q01: detection, "a. 向量级量化",
 * "b. INT8 矩阵乘法与反量化", merge; QE2 §1.2]
 *
 *   O       = { j : max_i |X[i][j]| > threshold }            (all M rows)
 *   s_x[m]  = max_{j not in O} |X[m][j]| / 127               (1.0 if 0)
 *   Xq[m][j]= clip(rint(X[m][j] / s_x[m]), -127, 127), 0 for j in O
 *   C[m][n] = sum_k Xq[m][k] * Wq[n][k]                      (int32)
 *   out     = C * s_x[m] * s_w[n] + sum_{h in O} X[m][h] * w~[n][h]
 * with fp16 outlier operands and fp32 accumulation; w~ = W_f16[n][h] when
 * W_f16 is given, else fp16(fl32(s_w[n] * Wq[n][h])).
 *   X       fp16 [M x K]
 *   Wq, s_w the weight quantized per output channel (qa_quantize_rowwise_int8
 *           on W [N x K], q range [-127, 127]): i8 [N x K], f32 [N]
 *   W_f16   fp16 [N x K] or NULL
 *   out     [M x N] of out_dtype (fp32, fp16 or bf16, round to nearest even)
 *   workspace  qa_qlinear_int8_mixed_workspace(M, K) bytes (any content);
 *           holds the outlier mask / list / count, s_x and Xq
 * threshold = +inf gives plain vector-wise W8A8; a negative threshold sends
 * every column through the fp16 product.
 * Errors: NULL pointers, M < 0, N < 0, K <= 0, K % 16 != 0, misaligned
 * pointers, NaN threshold, bad out_dtype, small workspace.
 * ------------------------------------------------------------------------- */
size_t qa_qlinear_int8_mixed_workspace(int64_t M, int64_t K);
qa_status qa_qlinear_int8_mixed(const void* X_f16, int64_t M, int64_t K,
                                const int8_t* Wq, const float* s_w, const void* W_f16_or_null,
                                int64_t N, float threshold, void* out, qa_dtype out_dtype,
                                void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Where the integer stages of an LLM.int8() call sit in its workspace
 * [AIInfra-Q01: detection and "a. 向量级量化"]
 *
 * After qa_qlinear_int8_mixed or qa_qlinear_int8_topk with M, N > 0 has
 * completed on its stream, its workspace holds, at these byte offsets:
 *   offsets[0]  idx    i32 [count]: the outlier columns O, ascending
 *   offsets[1]  count  i32 [1]:     |O|
 *   offsets[2]  s_x    f32 [M]:     the per-token scales
 *   offsets[3]  Xq     i8 [M x K]:  the int8 codes the GEMM consumed
 *                                   (0 in the columns of O)
 * i.e. exactly the values qa_outlier_cols (or qa_outlier_topk) and
 * qa_quantize_rowwise_int8 with that mask produce for the same X.  The
 * offsets depend only on M and K.  offsets: a HOST array of 4 entries.
 * Errors: M <= 0, K <= 0 (QA_ERR_SHAPE), offsets NULL (QA_ERR_NULL).
 * ------------------------------------------------------------------------- */
qa_status qa_qlinear_int8_mixed_offsets(int64_t M, int64_t K, size_t* offsets);

/* ---------------------------------------------------------------------------
 * LLM.int8() mixed linear without a workspace  -- for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc.
 *
 * Same arguments, kernels and results as qa_qlinear_int8_mixed, minus the
 * workspace: the call's scratch lives in a static device array of
 * QA_NOALLOC_SCRATCH_BYTES (40 MiB) that every GPU the library runs on holds
 * until the process ends.  The call allocates nothing (no hipMalloc, hipFree
 * or allocating library routine); the caller still provides X, Wq, s_w,
 * W_f16 and out.  Nothing in the scratch needs clearing: every slot a call
 * reads was written earlier in the same call.  All calls on one GPU share
 * that one array, so calls that overlap on one GPU (on different streams,
 * without ordering between them) race and give undefined results; calls on
 * one stream, or otherwise ordered, are safe.  After the call the scratch
 * holds the integer stages at the offsets of qa_qlinear_int8_mixed_offsets
 * (until the next call on that GPU).
 * Errors: as qa_qlinear_int8_mixed, and QA_ERR_WORKSPACE when
 * qa_qlinear_int8_mixed_workspace(M, K) > QA_NOALLOC_SCRATCH_BYTES (e.g.
 * M x K above about 33.5 million); QA_ERR_DEVICE if the scratch's device
 * address cannot be looked up.
 * ------------------------------------------------------------------------- */
#define QA_NOALLOC_SCRATCH_BYTES ((size_t)40 << 20)
qa_status qa_qlinear_int8_mixed_noalloc(const void* X_f16, int64_t M, int64_t K, const int8_t* Wq,
                                        const float* s_w, const void* W_f16_or_null, int64_t N, float threshold,
                                        void* out, qa_dtype out_dtype, void* stream);

/* ---------------------------------------------------------------------------
 * LLM.int8() linear with top-k decomposition  [AIInfra-Q01: decomposition
 * share raised to the top 1-2% of feature dimensions]
 *
 * qa_qlinear_int8_mixed with O = the k columns of qa_outlier_topk instead of
 * the threshold set; everything else (scales, codes, GEMM, fp16 outlier
 * product) is identical.  k = 0 is plain vector-wise W8A8; k = K sends every
 * column through the fp16 product.
 *   workspace  qa_qlinear_int8_topk_workspace(M, K) bytes (any content)
 * Errors: as qa_qlinear_int8_mixed (no threshold), plus K > 32768
 * (QA_ERR_SHAPE), k < 0 or k > K (QA_ERR_VALUE).
 * ------------------------------------------------------------------------- */
size_t qa_qlinear_int8_topk_workspace(int64_t M, int64_t K);
qa_status qa_qlinear_int8_topk(const void* X_f16, int64_t M, int64_t K, int64_t k, const int8_t* Wq,
                               const float* s_w, const void* W_f16_or_null, int64_t N, void* out,
                               qa_dtype out_dtype, void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Block Hadamard rotation fused with int4 quantization and packing
 * [GroupRot §二, §5.1, §5.2, §5.4; Scholia-IQ §7.3]
 *
 *   X'[r][b*G + j] = fl32( fl64(1/sqrt(G)) * sum_i X[r][b*G + i] * H[i][j] ),
 *   H[i][j] = (-1)^popcount(i & j) (Sylvester order); the +-1 sum is exact.
 *   PER_ROW:   s[r]    = absmax(X'[r][:]) / q_max                (s: [rows])
 *   PER_GROUP: s[r][b] = absmax(X'[r][bG:(b+1)G]) / q_max        (s: [rows x K/G])
 *   code = clip(rint(X' / s), q_min, q_max); element 8w+i of a row is the
 *   two's-complement nibble in bits [4i+3:4i] of packed[r][w].
 *   G = 1 is the identity rotation.
 *   X       fp16 [rows x K]; packed u32 [rows x K/8]; s f32 as above
 * Errors: NULL pointers, rows < 0, K <= 0, K % 8 != 0, K % G != 0, G not a
 * power of two in [1, 256], PER_GROUP with G < 8, q range outside [-8, 7],
 * q_max <= 0, q_min > q_max, misaligned X / packed.
 * ------------------------------------------------------------------------- */
qa_status qa_hadamard_quant_int4(const void* X_f16, int64_t rows, int64_t K, int32_t G,
                                 qa_scale_mode mode, int32_t q_min, int32_t q_max,
                                 uint32_t* packed, float* s, void* stream);

/* ---------------------------------------------------------------------------
 * W4A4 group-Hadamard linear  [GroupRot §5.2, §5.4]
 *
 *   (Xp, s_x) = qa_hadamard_quant_int4(X, G, PER_ROW, -7, 7)  (on device)
 *   acc_g[m][n] = sum_{k in group g} qx[m][k] * qw[n][k]     (int32)
 *   out[m][n]   = s_x[m] * sum_g s_w[n][g] * acc_g[m][n]
 *   X       fp16 [M x K]
 *   Wp, s_w the offline weight: qa_hadamard_quant_int4(W, G, PER_GROUP, ...)
 *           u32 [N x K/8], f32 [N x K/G]
 *   out     [M x N] of out_dtype
 *   workspace  qa_qlinear_w4a4_workspace(M, K) bytes (any content)
 * Errors: NULL pointers, M < 0, N < 0, K <= 0, G not a power of two in [8, 256],
 * K % G != 0, misaligned pointers, bad out_dtype, small workspace.
 * ------------------------------------------------------------------------- */
size_t qa_qlinear_w4a4_workspace(int64_t M, int64_t K);
qa_status qa_qlinear_w4a4(const void* X_f16, int64_t M, int64_t K, const uint32_t* Wp,
                          const float* s_w, int64_t N, int32_t G, void* out, qa_dtype out_dtype,
                          void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Hadamard rotation + per-row int8 codes  [GroupRot §二, §5.2: the rotation
 * fused with dynamic per-token quantization; Scholia-IQ §2.2: 8-bit
 * activations of W4A8]
 *
 *   X'[r] = X[r] * blockdiag(H_G) / sqrt(G)   (as qa_hadamard_quant_int4)
 *   s[r]  = fl32(max_j |X'[r][j]| / q_max)     (1.0 for an all-zero row)
 *   q[r][j] = clip(rint(fl32(X'[r][j] / s[r])), q_min, q_max)
 *   X fp16 [rows x K]; q i8 [rows x K]; s f32 [rows]
 * Errors: NULL pointers, rows < 0, K <= 0, K % 8 != 0, G not a power of two
 * in [1, 256], K % G != 0, q_min > q_max, q_min < -128, q_max > 127,
 * q_max <= 0, misaligned X (16 bytes) / q (8 bytes) / s.
 * ------------------------------------------------------------------------- */
qa_status qa_hadamard_quant_int8(const void* X_f16, int64_t rows, int64_t K, int32_t G, int32_t q_min,
                                 int32_t q_max, int8_t* q, float* s, void* stream);

/* ---------------------------------------------------------------------------
 * W4A8 group-Hadamard linear  [Scholia-IQ §2.1-§2.2: 4-bit weights, 8-bit
 * activations; "从离群值到平坦线" §4: a transform fitted for W4A4 serves W4A8
 * unchanged; GroupRot §5.2, §5.4]
 *
 *   (Xq, s_x) = qa_hadamard_quant_int8(X, G, -127, 127)   (on device)
 *   acc_g[m][n] = sum_{k in group g} Xq[m][k] * qw[n][k]   (int32)
 *   out[m][n]   = s_x[m] * sum_g s_w[n][g] * acc_g[m][n]
 *   Wp, s_w  the offline W4A4 weight: qa_hadamard_quant_int4(W, G, PER_GROUP,
 *            -7, 7): u32 [N x K/8], f32 [N x K/G]
 *   out      [M x N] of out_dtype
 *   workspace  qa_qlinear_w4a8_workspace(M, K) bytes (any content)
 * Errors: NULL pointers, M < 0, N < 0, K <= 0, G not a power of two in [8, 256],
 * K % G != 0, misaligned pointers, bad out_dtype, small workspace.
 * ------------------------------------------------------------------------- */
size_t qa_qlinear_w4a8_workspace(int64_t M, int64_t K);
qa_status qa_qlinear_w4a8(const void* X_f16, int64_t M, int64_t K, const uint32_t* Wp,
                          const float* s_w, int64_t N, int32_t G, void* out, qa_dtype out_dtype,
                          void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Hadamard rotation + zero-point int4 codes per row  [GroupRot §二, §5.2;
 * Scholia-IQ §6 (q = round(x/s) + z, x^ = s (q - z)), §6.2 (the grid on the
 * data's range, clip to [q_min, q_max])]
 *
 *   X'[r] = X[r] * blockdiag(H_G) / sqrt(G)       (as qa_hadamard_quant_int4)
 *   [lo, hi] = [min(min X'[r], 0), max(max X'[r], 0)]
 *   s[r] = fl32(fl32(hi - lo) / 15)   (1.0 when hi == lo)
 *   z[r] = clip(-rint(fl32(lo / s[r])), 0, 15)
 *   q = clip(rint(fl32(X'[r][j] / s[r])) + z[r], 0, 15), packed eight per
 *   word as the two's complement nibble q - 8 (element 8w+i in bits
 *   [4i+3:4i] of word w)
 *   X fp16 [rows x K]; packed u32 [rows x K/8]; s f32, z i32 [rows]
 * Errors: NULL pointers, rows < 0, K <= 0, K % 8 != 0, G not a power of two
 * in [1, 256], K % G != 0, misaligned pointers.
 * ------------------------------------------------------------------------- */
qa_status qa_hadamard_quant_int4_asym(const void* X_f16, int64_t rows, int64_t K, int32_t G, uint32_t* packed,
                                      float* s, int32_t* z, void* stream);

/* Column terms of a per-group int4 weight (offline, with the weight):
 *   c[n] = fl32(sum_g s_w[n][g] * sum_{k in group g} qw[n][k])   (fp64, g ascending)
 *   Wp u32 [N x K/8], s_w f32 [N x K/G]; c f32 [N]
 * Errors: NULL pointers, N < 0, K <= 0, G not a power of two in [8, 256],
 * K % G != 0, misaligned pointers. */
qa_status qa_w4_column_terms(const uint32_t* Wp, const float* s_w, int64_t N, int64_t K, int32_t G, float* c,
                             void* stream);

/* ---------------------------------------------------------------------------
 * W4A4 linear with zero-point activations  [Scholia-IQ §6, §6.2, §7.3;
 * GroupRot §5.2, §5.4]
 *
 *   (Xp, s_x, z_x) = qa_hadamard_quant_int4_asym(X, G)   (on device)
 *   out[m][n] = s_x[m] * sum_g s_w[n][g] * sum_{k in g} (q[m][k] - z_x[m]) qw[n][k]
 *             = s_x[m] * (sum_g s_w[n][g] sum_{k in g} (q - 8) qw - (z_x[m] - 8) c_w[n])
 *   Wp, s_w  the offline W4A4 weight (qa_hadamard_quant_int4, PER_GROUP)
 *   c_w      qa_w4_column_terms(Wp, s_w, G): f32 [N]
 *   out      [M x N] of out_dtype
 *   workspace  qa_qlinear_w4a4_asym_workspace(M, K) bytes (any content)
 * Errors: NULL pointers, M < 0, N < 0, K <= 0, G not a power of two in [8, 256],
 * K % G != 0, misaligned pointers, bad out_dtype, small workspace.
 * ------------------------------------------------------------------------- */
size_t qa_qlinear_w4a4_asym_workspace(int64_t M, int64_t K);
qa_status qa_qlinear_w4a4_asym(const void* X_f16, int64_t M, int64_t K, const uint32_t* Wp, const float* s_w,
                               const float* c_w, int64_t N, int32_t G, void* out, qa_dtype out_dtype,
                               void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Asymmetric (zero-point) row quantization  [Scholia-IQ §6: q = round(x/s) +
 * z, x^ = s (q - z), z the integer that stands for real 0; §6.2: the grid
 * shifted onto the data's range, q clipped to [q_min, q_max]]
 *
 * Per row r (the pages leave the choice of s and z open; min-max is taken):
 *   lo = min(min_j X[r][j], 0), hi = max(max_j X[r][j], 0)
 *   s  = fl32(fl32(hi - lo) / (q_max - q_min))      (1.0 when hi == lo)
 *   z  = clip(q_min - rint(fl32(lo / s)), q_min, q_max)
 *   q[r][j]   = clip(rint(fl32(X[r][j] / s)) + z, q_min, q_max)
 *   rowsum[r] = sum_j q[r][j]                          (if rowsum != NULL)
 *   X fp16 [rows x K]; q i8 [rows x K]; s_out f32, z_out i32, rowsum i32 [rows]
 * Errors: NULL pointers, rows < 0, K <= 0, K > 2^26, K % 8 != 0, X or q not
 * 16-byte aligned, q_min >= q_max or outside [-128, 127].
 * ------------------------------------------------------------------------- */
qa_status qa_quantize_rowwise_int8_asym(const void* X_f16, int64_t rows, int64_t K, int32_t q_min, int32_t q_max,
                                        int8_t* q, float* s_out, int32_t* z_out, int32_t* rowsum_or_null,
                                        void* stream);

/* Row sums of int8 rows: sums[r] = sum_j A[r][j] (the weight term of the
 * zero-point correction below for a weight quantized without zero-point).
 * Errors: NULL pointers, rows < 0, K <= 0, K > 2^26, K % 16 != 0, A not
 * 16-byte aligned. */
qa_status qa_int8_row_sums(const int8_t* A, int64_t rows, int64_t K, int32_t* sums, void* stream);

/* ---------------------------------------------------------------------------
 * W8A8 linear with zero-point activations  [Scholia-IQ §6, §6.2;
 * AIInfra-Q01 "b. INT8 矩阵乘法与反量化"]
 *
 *   (Xq, s_x, z_x) = qa_quantize_rowwise_int8_asym(X, -128, 127)  (per token,
 *                    on device)
 *   out[m][n] = s_x[m] s_w[n] sum_k (Xq[m][k] - z_x[m]) (Wq[n][k] - z_w[n])
 * evaluated as C - z_x a[n] - z_w[n] r_x[m] with C the int32 GEMM,
 * a[n] = w_rowsum[n] - K z_w[n] and r_x the activation code sums (exact).
 *   Wq i8 [N x K], s_w f32 [N]: the weight (symmetric from
 *           qa_quantize_rowwise_int8, or asymmetric from
 *           qa_quantize_rowwise_int8_asym with z_w = its z_out)
 *   z_w     i32 [N] or NULL (zero-point 0)
 *   w_rowsum  i32 [N]: sum_k Wq[n][k] (rowsum_out of the asymmetric
 *           quantizer, or qa_int8_row_sums)
 *   out     [M x N] of out_dtype
 *   workspace  qa_qlinear_int8_asym_workspace(M, K) bytes (any content)
 * Errors: NULL pointers, M < 0, N < 0, K <= 0, K % 16 != 0, K > 32768 (the
 * integer sum must fit int32), misaligned pointers, bad out_dtype, small
 * workspace.
 * ------------------------------------------------------------------------- */
size_t qa_qlinear_int8_asym_workspace(int64_t M, int64_t K);
qa_status qa_qlinear_int8_asym(const void* X_f16, int64_t M, int64_t K, const int8_t* Wq, const float* s_w,
                               const int32_t* z_w_or_null, const int32_t* w_rowsum, int64_t N, void* out,
                               qa_dtype out_dtype, void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Column absolute maxima  [QE2 §4.2: max|X_j| and max|W_j| per input channel]
 *
 *   colmax[j] = max_r |A[r][j]|  (accumulate == 0)
 *   colmax[j] = max(colmax[j], max_r |A[r][j]|)  (accumulate != 0: a running
 *               maximum over calibration batches; colmax must then hold
 *               non-negative finite values, e.g. from an earlier call)
 * For activations A = X [M x K]; for the weight A = W [N x K] gives the
 * maximum over output channels of each input channel.  Exact (fp16 widened).
 *   A       fp16 [rows x K]; colmax f32 [K]
 *   scratch device buffer of qa_col_absmax_workspace(K) bytes (any content)
 * rows == 0 is a no-op.
 * Errors: NULL pointers, rows < 0, K <= 0, K > 2^22, K % 8 != 0, A not
 * 16-byte aligned, small scratch.
 * ------------------------------------------------------------------------- */
size_t qa_col_absmax_workspace(int64_t K);
qa_status qa_col_absmax(const void* A_f16, int64_t rows, int64_t K, float* colmax, int accumulate,
                        void* scratch, size_t scratch_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * SmoothQuant migration factors  [QE2 §4.2]
 *
 *   s[j] = fl32( pow(act_absmax[j], alpha) / pow(w_absmax[j], 1 - alpha) )
 * evaluated in fp64 (alpha widened exactly from fp32); s[j] = 1 when either
 * maximum is 0.  alpha = 0.5 splits the range evenly; alpha = 1 gives
 * s = act_absmax (activation columns scaled to magnitude 1); alpha = 0 gives
 * s = 1 / w_absmax.  The fp64 pow of the device math library may differ from
 * another implementation's by one rounding, so s can differ in the last fp32
 * bit; the smoothing below takes s as given.
 *   act_absmax, w_absmax  f32 [K], non-negative finite
 *   s       f32 [K]
 * Errors: NULL pointers, K < 0, alpha NaN or outside [0, 1].  K == 0 is a
 * no-op.
 * ------------------------------------------------------------------------- */
qa_status qa_smooth_factors(const float* act_absmax, const float* w_absmax, int64_t K, float alpha, float* s,
                            void* stream);

/* ---------------------------------------------------------------------------
 * Smoothing fused with int8 quantization  [QE2 §4.2; Scholia-IQ §4, §7]
 *
 *   a^[r][j] = fl32(A[r][j] / s[j])   (QA_SMOOTH_DIVIDE: activations)
 *   a^[r][j] = fl32(A[r][j] * s[j])   (QA_SMOOTH_MULTIPLY: the weight W [N x K],
 *                                      offline)
 *   QA_SCALE_PER_ROW:    s_out[r] = fl32(max_j |a^[r][j]| / 127)
 *   QA_SCALE_PER_TENSOR: s_out[r] = fl32(max_{r,j} |a^[r][j]| / 127) for every r
 *   (1.0 for an all-zero row / tensor)
 *   q[r][j]  = clip(rint(a^[r][j] / s_out[r]), -127, 127)
 *   A       fp16 [rows x K]; s f32 [K], positive finite; q i8 [rows x K];
 *   s_out   f32 [rows]
 * Errors: NULL pointers, rows < 0, K <= 0, K > 2^26, K % 8 != 0, A or q not
 * 16-byte aligned, bad op, mode not PER_ROW / PER_TENSOR.  rows == 0 is a
 * no-op.
 * ------------------------------------------------------------------------- */
qa_status qa_quantize_smooth_int8(const void* A_f16, int64_t rows, int64_t K, const float* s, qa_smooth_op op,
                                  qa_scale_mode mode, int8_t* q, float* s_out, void* stream);

/* ---------------------------------------------------------------------------
 * SmoothQuant W8A8 linear  [QE2 §4.2, §4.4; AIInfra-Q01 "b. INT8 矩阵乘法与反量化"]
 *
 *   (Xq, s_x) = qa_quantize_smooth_int8(X, s, QA_SMOOTH_DIVIDE, mode)  (on device)
 *   C[m][n]   = sum_k Xq[m][k] * Wq[n][k]                              (int32)
 *   out       = C * s_x[m] * s_w[n]
 *   X       fp16 [M x K]; s f32 [K] (qa_smooth_factors)
 *   Wq, s_w the smoothed weight: qa_quantize_smooth_int8(W, s,
 *           QA_SMOOTH_MULTIPLY, QA_SCALE_PER_ROW): i8 [N x K], f32 [N]
 *   mode    QA_SCALE_PER_ROW (per token) or QA_SCALE_PER_TENSOR for X
 *   out     [M x N] of out_dtype
 *   workspace  qa_qlinear_int8_smooth_workspace(M, K) bytes (any content);
 *           after the call it holds s_x and Xq
 * Decode shapes (K % 256 == 0 with M <= 8 at K <= 4096 or M <= 4 at
 * K <= 8192) run as one kernel that smooths, quantizes and multiplies; the
 * results are the same bits.
 * Errors: NULL pointers, M < 0, N < 0, K <= 0, K % 16 != 0, K > 131072,
 * misaligned pointers, bad mode or out_dtype, small workspace.
 * ------------------------------------------------------------------------- */
size_t qa_qlinear_int8_smooth_workspace(int64_t M, int64_t K);
qa_status qa_qlinear_int8_smooth(const void* X_f16, int64_t M, int64_t K, const float* s, qa_scale_mode mode,
                                 const int8_t* Wq, const float* s_w, int64_t N, void* out, qa_dtype out_dtype,
                                 void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Kronecker affine transform fused with int4 quantization  [AIInfra-Q01,
 * FlatQuant section: X~ x1 P1^T x2 P2, P = P1 (x) P2, dynamic int4 codes in one
 * kernel]
 *
 * Each row x (K = n1 n2) is read as X~[i][j] = x[i n2 + j] and transformed to
 * X' = P1^T X~ P2 (= x (P1 (x) P2)), mode 1 first, every output one fp32 chain
 * of fused multiply-adds over the contraction index in ascending order:
 *   Y[a][j]  = sum_i P1[i][a] X~[i][j],   X'[a][b] = sum_j Y[a][j] P2[j][b].
 * Then int4 codes of X' as qa_hadamard_quant_int4 makes them (PER_ROW: one
 * scale per row; PER_GROUP: per G-wide group), packed eight per word.
 * Activations take the learned P1, P2; the offline weight takes P1^-T, P2^-T
 * (the same matrices when they are orthogonal), so X' W'^T = X W^T.
 *   X       fp16 [rows x K]; P1 f32 [n1 x n1], P2 f32 [n2 x n2] row-major
 *   packed  u32 [rows x K/8]; s f32 [rows] or [rows x K/G]
 * Sizes with a kernel: (n1, n2) in {(8,8), (8,16), (16,16), (16,32), (32,32),
 * (32,64), (64,64), (64,128)} -- the minimal-sum splits of 64 .. 8192; per
 * group, G a multiple of 8 with a group inside one wave's chunks.
 * Errors: NULL pointers, rows < 0, n1 n2 != K (QA_ERR_SHAPE), no kernel for
 * the sizes (QA_ERR_UNSUPPORTED), bad mode / q range, misaligned pointers.
 * ------------------------------------------------------------------------- */
qa_status qa_kron_quant_int4(const void* X_f16, int64_t rows, int64_t K, int64_t n1, int64_t n2, const float* P1,
                             const float* P2, qa_scale_mode mode, int32_t G, int32_t q_min, int32_t q_max,
                             uint32_t* packed, float* s, void* stream);

/* ---------------------------------------------------------------------------
 * Kronecker factor sizes  [AIInfra-Q01, FlatQuant section (the split of P
 * into P1 (x) P2 minimizes n1 + n2 under n1 n2 = n, n1 <= n2; n = 8192 gives
 * 64 x 128); 从离群值到平坦线：FlatQuant 如何重塑 LLM 的 4-bit 量化格局, §2
 * (4096 as 64 x 64)]
 *
 *   n1 = the largest divisor of n not above sqrt(n), n2 = n / n1: the pair
 *   with n1 n2 = n, n1 <= n2 and the smallest n1 + n2.  Host arithmetic, no
 *   device work.
 *   n           transform width (K), > 0
 *   n1, n2      host int64 outputs
 *   has_kernel  host int32 output, may be NULL: 1 when qa_kron_quant_int4 and
 *               qa_qlinear_kron_w4a4 have a kernel for (n1, n2), else 0
 * Errors: NULL n1 or n2 (QA_ERR_NULL), n <= 0 (QA_ERR_SHAPE); the outputs
 * are untouched on error.
 * ------------------------------------------------------------------------- */
qa_status qa_kron_sizes(int64_t n, int64_t* n1, int64_t* n2, int32_t* has_kernel);

/* ---------------------------------------------------------------------------
 * W4A4 linear with the Kronecker transform  [AIInfra-Q01, FlatQuant section:
 * transform + dynamic int4 of X in one kernel, int4 GEMM with the
 * pre-transformed int4 weight]
 *
 *   (Xp, s_x) = qa_kron_quant_int4(X, n1, n2, P1, P2, PER_ROW, -7, 7)
 *   out[m][n] = s_x[m] sum_g s_w[n][g] sum_{k in g} qx[m][k] qw[n][k]
 *   Wp, s_w  the offline weight: qa_kron_quant_int4(W, n1, n2, P1^-T, P2^-T,
 *            PER_GROUP, G, -7, 7): u32 [N x K/8], f32 [N x K/G]
 *   out      [M x N] of out_dtype
 *   workspace  qa_qlinear_kron_w4a4_workspace(M, K) bytes (any content)
 * Errors: NULL pointers, M < 0, N < 0, G not a power of two in [8, 256], K % G != 0,
 * n1 n2 != K, unsupported sizes, misaligned pointers, bad out_dtype, small
 * workspace.
 * ------------------------------------------------------------------------- */
size_t qa_qlinear_kron_w4a4_workspace(int64_t M, int64_t K);
qa_status qa_qlinear_kron_w4a4(const void* X_f16, int64_t M, int64_t K, int64_t n1, int64_t n2, const float* P1,
                               const float* P2, const uint32_t* Wp, const float* s_w, int64_t N, int32_t G, void* out,
                               qa_dtype out_dtype, void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Parity entry points: the integer accumulators of the two GEMMs, stored.
 *
 * qa_gemm_i8_i32  [AIInfra-Q01 "b. INT8 矩阵乘法与反量化"]
 *   C[m][n] = sum_k A[m][k] * B[n][k]; A i8 [M x K], B i8 [N x K],
 *   C i32 [M x N].  The caller keeps |C| < 2^31 (K * 128^2 < 2^31 suffices).
 *   Errors: NULL, M < 0, N < 0, K <= 0, K % 16 != 0, misaligned pointers.
 *
 * qa_gemm_w4a4_group_acc  [GroupRot §5.4]
 *   acc[m][n][g] = sum_{k in group g} qx[m][k] * qw[n][k] from packed int4
 *   Xp u32 [M x K/8], Wp u32 [N x K/8]; acc i32 [M x N x K/G].
 *   Errors: NULL, M < 0, N < 0, K <= 0, G not a power of two in [8, 256],
 *   K % G != 0, misaligned pointers.
 *
 * qa_gemm_w4a8_group_acc  [GroupRot §5.4; Scholia-IQ §2.2]
 *   acc[m][n][g] = sum_{k in group g} Xq[m][k] * qw[n][k] from int8 codes
 *   Xq i8 [M x K] and packed int4 Wp u32 [N x K/8]; acc i32 [M x N x K/G].
 *   Errors as qa_gemm_w4a4_group_acc (Xq 16-byte aligned).
 * ------------------------------------------------------------------------- */
qa_status qa_gemm_i8_i32(const int8_t* A, const int8_t* B, int64_t M, int64_t K, int64_t N,
                         int32_t* C, void* stream);
qa_status qa_gemm_w4a4_group_acc(const uint32_t* Xp, const uint32_t* Wp, int64_t M, int64_t K,
                                 int64_t N, int32_t G, int32_t* acc, void* stream);
qa_status qa_gemm_w4a8_group_acc(const int8_t* Xq, const uint32_t* Wp, int64_t M, int64_t K,
                                 int64_t N, int32_t G, int32_t* acc, void* stream);

/* ---------------------------------------------------------------------------
 * Residual addition, root-mean-square norm and int8 codes in one pass: the
 * operator in front of an int8 linear that takes codes
 *
 *   h = X + residual                    (fp32; residual NULL: h = X)
 *   y = h g / sqrt(mean_j h_j^2 + eps)  (fp32)
 *   s[m] = max_j |y_j| / 127 (1.0 where that is 0), Xq = rint(y / s)
 *   X, residual, g, sum, y   arrays of `dtype` (fp32, fp16 or bf16)
 *   ldx, ldr, lds   row strides of X, residual and sum, in elements
 *   sum     [rows x K] or NULL: h rounded to dtype; may be X or residual itself
 *           (same pointer and stride), no other overlap of outputs is allowed
 *   y       [rows x K] contiguous or NULL: the norm rounded to dtype
 *   Xq, s   i8 [rows x K] contiguous, f32 [rows]
 * Any K >= 1; rows whose arrays all start at 16-byte boundaries (K, strides)
 * are read and written in whole 16-byte pieces.
 * A row that holds an infinity or NaN, or whose sum of squares passes fp32,
 * gets s = NaN and codes 0 (so a linear's output row is NaN) and a y of NaNs and
 * zeros; other rows are unaffected.  g must be finite.
 * Errors: rows < 0, rows > 2^31 - 1, K <= 0, K > 2^26, a stride below K, bad
 * dtype, eps not positive and finite, NULL X / g / Xq / s, X / g / residual /
 * sum / y not aligned to their elements, s not 4-byte aligned.
 * ------------------------------------------------------------------------- */
qa_status qa_rmsnorm_int8(const void* X, int64_t ldx, const void* residual_or_null, int64_t ldr, const void* g,
                          qa_dtype dtype, int64_t rows, int64_t K, float eps, int8_t* Xq, float* s,
                          void* sum_or_null, int64_t lds, void* y_or_null, void* stream);

/* ---------------------------------------------------------------------------
 * Routing of tokens to experts
 *
 *   score_e  = softmax(logits)_e or 1 / (1 + exp(-logit_e))
 *   choice_e = score_e + bias_e
 *   With n_groups > 1 the E experts form n_groups equal ranges; a group's value
 *   is its largest choice (group_top 1) or the sum of its two largest
 *   (group_top 2), and only the top_groups groups of largest value keep their
 *   experts.  The k experts of largest choice are taken in descending order.
 *   Ties, of groups and of experts, go to the lower index.
 *   weight_j = score (without the bias) of the j-th expert; with renorm divided
 *   by the sum of the token's k (where that is not 0); times scale.
 *   logits  [T x E] of dtype, row stride ld elements; bias f32 [E] or NULL
 *   ids     i32 [T x k]; weights f32 [T x k]
 *   order   i32 [T k]: the pairs t k + j grouped by expert, ascending within
 *           an expert; places past the last pair hold -1
 *   offsets i32 [E + 1]: expert e's pairs are order[offsets[e] .. offsets[e+1])
 * Without a bias (and with groups valued by their largest expert) the choice
 * goes by the logits themselves, which have the scores' order; otherwise by
 * scores in fp32, where those of different logits may be equal (sigmoid is 1
 * above 17, softmax 0 far below the row's largest): such ties go to the lower index.
 * A logit (or bias) of -infinity or NaN masks its expert; a logit of +infinity
 * counts as the largest finite value.  Where fewer than k experts are left, the last slots
 * are expert -1 with weight 0 and are in no expert's range.
 *   workspace  qa_route_experts_workspace(T, E, k) bytes (any content)
 * The result does not depend on the order in which blocks run.  T == 0 writes
 * offsets alone (zeros).
 * Errors (QA_ERR_SHAPE): T outside 0..2^23, E outside 1..1024, ld < E, k
 * outside 1..min(32, E), n_groups outside 1..32 or not dividing E,
 * top_groups outside 1..n_groups, k > top_groups E / n_groups; (QA_ERR_VALUE)
 * bad dtype, score or group_top, scale not finite; NULL pointers, alignment to
 * the elements, small workspace.
 * ------------------------------------------------------------------------- */
typedef enum { QA_SCORE_SOFTMAX = 0, QA_SCORE_SIGMOID = 1 } qa_score;
size_t qa_route_experts_workspace(int64_t T, int64_t E, int32_t k);
qa_status qa_route_experts(const void* logits, qa_dtype dtype, int64_t T, int64_t E, int64_t ld,
                           const float* bias_or_null, qa_score score, int32_t n_groups, int32_t top_groups,
                           int32_t group_top, int32_t k, int32_t renorm, float scale, int32_t* ids, float* weights,
                           int32_t* order, int32_t* offsets, void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Gated feed-forward of the experts on int8 codes
 *
 * For every pair p = t k + j in expert e's range of `order`:
 *   g = s_x[t] s13[e][f] sum_c Xq[t][c] W13[e][f][c]          f = 0 .. F-1
 *   u = the same with row F + f
 *   h = g / (1 + exp(-g)) u           (fp32)
 *   s_h = max_f |h| / 127 (1.0 where that is 0), hq = rint(h / s_h)
 *   y = s_h s2[e][c] sum_f hq[f] W2[e][c][f]                  c = 0 .. K-1
 * and out[t] = sum_j weights[t][j] y (j ascending, fp32), rounded once.  Pairs
 * that are in no range add nothing; a token with none gets a row of zeros.
 *   Xq, s_x  i8 [T x K], f32 [T] (qa_rmsnorm_int8 or qa_quantize_rowwise_int8)
 *   weights, order, offsets   of qa_route_experts: f32 [T x k], i32 [T k],
 *            i32 [E + 1], ranges ascending and disjoint, each pair at most once
 *            (others give unspecified values; no access leaves the arrays).
 *            E may be a part of the experts that were routed to: their weights
 *            and their E + 1 starts out of the whole offsets, with all of order
 *   W13, s13 i8 [E x 2F x K] (gate rows, then up rows), f32 [E x 2F]
 *   W2, s2   i8 [E x K x F], f32 [E x K]; scales per output channel
 *   out      [T x K] of out_dtype
 *   workspace  qa_experts_int8_workspace(T, K, k, E, F) bytes (any content)
 * Errors (QA_ERR_SHAPE): T < 0, E outside 1..1024, k outside 1..32, K or F not
 * a positive multiple of 16 up to 131072, T K or 2 F K >= 2^31, T k > 2^23,
 * (T k / 64 + E) (max(2 F, K) / 128 + 1) >= 2^23; bad out_dtype; NULL
 * pointers; Xq, W13, W2, s13, s2, out not 16-byte, others not 4-byte,
 * workspace not 256-byte aligned; small workspace.
 * ------------------------------------------------------------------------- */
size_t qa_experts_int8_workspace(int64_t T, int64_t K, int32_t k, int64_t E, int64_t F);
qa_status qa_experts_int8(const int8_t* Xq, const float* s_x, int64_t T, int64_t K, const float* weights,
                          const int32_t* order, const int32_t* offsets, int64_t E, int32_t k, const int8_t* W13,
                          const float* s13, int64_t F, const int8_t* W2, const float* s2, void* out,
                          qa_dtype out_dtype, void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * A shared int8 projection with the low-rank adapters of many requests
 *
 *   out[m][n] = s_x[m] s_w[n] sum_k Xq[m][k] Wq[n][k]
 *             + alpha[a] sum_j (sum_k X[m][k] A[a][j][k]) B[a][n][j]
 * with a the adapter of the request that holds token m; tokens of requests
 * with adapter -1, and tokens of no request, take the first line alone.  The
 * sum is formed in fp32 and rounded once.  For many tokens the inner products
 * over k enter the second product with a relative step of at most 2^-17 (dtype
 * bf16, 16-bit out) or 2^-23 (otherwise) of the largest of 32 ranks; for few, and
 * for bf16 with fp32 out, in fp32.  One that is infinite or NaN makes its token's
 * outputs infinite or NaN.
 *   Xq, s_x  i8 [M x K], f32 [M]: the tokens' codes (qa_rmsnorm_int8)
 *   X        [M x K] of dtype (fp16 or bf16): the values the adapters see (its y)
 *   Wq, s_w  i8 [N x K], f32 [N]
 *   A, B     [L x r x K], [L x N x r] of dtype; alpha f32 [L]
 *   seg      i32 [R + 1]: request i holds the tokens seg[i] .. seg[i + 1]
 *            (not descending; empty requests are allowed; starts that fall
 *            give unspecified values, no access leaves the arrays)
 *   which    i32 [R]: adapter of a request; outside 0 .. L-1: none
 *   out      [M x N] of out_dtype
 *   workspace  qa_qlinear_int8_lora_workspace(M, K, r) bytes (any content)
 * With R == 0 or L == 0 X, A, B, alpha, seg and which are not read and may be
 * NULL.
 * Errors (QA_ERR_SHAPE): M, N, L or R negative, M > 2^23, N, L or R past
 * 2^31 - 1, ceil(M / 64) ceil(N / 128) >= 2^23, K not a positive multiple of
 * 16 up to 131072, r not a multiple of 8 in 8..256; (QA_ERR_VALUE) dtype not
 * fp16 / bf16, bad out_dtype; NULL pointers; Xq, X, Wq, A, B not 16-byte, others
 * not 4-byte, workspace not 256-byte aligned; small workspace.
 * ------------------------------------------------------------------------- */
size_t qa_qlinear_int8_lora_workspace(int64_t M, int64_t K, int32_t r);
qa_status qa_qlinear_int8_lora(const int8_t* Xq, const float* s_x, const void* X, qa_dtype dtype, int64_t M,
                               int64_t K, const int8_t* Wq, const float* s_w, int64_t N, const void* A, const void* B,
                               const float* alpha, int32_t r, int64_t L, const int32_t* seg, const int32_t* which,
                               int64_t R, void* out, qa_dtype out_dtype, void* workspace, size_t workspace_bytes,
                               void* stream);

/* ---------------------------------------------------------------------------
 * A paged cache of keys and values in int8 or int4 codes
 *
 * The cache is four arrays: for keys and for values, codes and scales.
 *   codes   bits 8: i8 [pages x heads x page x D]
 *           bits 4: u32 [pages x heads x page x D/8], element 8w+i of a row in
 *           bits [4i+3:4i] of its word w, two's complement
 *   scales  f32 [pages x heads x page]
 * A row (one token, one head) x is stored as
 *   s = fl32(max_d |x_d| / q_max) (1.0 where that is 0), q_max = 127 or 7
 *   q_d = clip(rint(fl32(x_d / s)), -q_max, q_max)
 * A row that holds an infinity or NaN gets s = NaN and codes 0; other rows are
 * unaffected.  slots name tokens' places: slot = page index * page + place in
 * the page.
 *
 * qa_kv_write: K, V [T x heads x D] of dtype (fp32, fp16 or bf16), token strides
 *   ldk, ldv in elements (a token's heads are contiguous), into the places
 *   slots i64 [T].  A slot outside 0 .. pages page - 1 (-1 for padding) writes
 *   nothing; places that no slot names are left as they were.  A place named
 *   twice holds unspecified codes and scales (no access leaves the arrays).
 * qa_kv_read: x_d = fl32(q_d s), rounded to dtype, for the places slots i64 [T]
 *   in any order, into K, V [T x heads x D] contiguous of dtype; a slot outside the
 *   cache gives a row of zeros.
 * Errors: (QA_ERR_SHAPE) T outside 0..2^23, heads outside 1..65535, D not a
 * multiple of 16 in 16..256, page not a power of two in 16..1024, pages < 0 or
 * pages > 2^31 - 1, a token stride below heads D or not a multiple of 16
 * bytes; (QA_ERR_VALUE) bad dtype, bits not 8 or 4; NULL pointers; K, V, codes
 * and scales not 16-byte, slots not 8-byte aligned.  T == 0 is a no-op; a cache
 * of no pages may have NULL pointers (and is one that no slot lies in).
 * ------------------------------------------------------------------------- */
qa_status qa_kv_write(const void* K, int64_t ldk, const void* V, int64_t ldv, qa_dtype dtype, int64_t T,
                      const int64_t* slots, int32_t bits, int64_t pages, int32_t heads, int32_t page, int32_t D,
                      void* k_codes, float* k_scales, void* v_codes, float* v_scales, void* stream);
qa_status qa_kv_read(const int64_t* slots, int64_t T, int32_t bits, int64_t pages, int32_t heads, int32_t page,
                     int32_t D, const void* k_codes, const float* k_scales, const void* v_codes, const float* v_scales,
                     void* K, void* V, qa_dtype dtype, void* stream);

/* ---------------------------------------------------------------------------
 * Attention of one new token per sequence over such a cache
 *
 *   n = min(max(lengths[b], 0), max_len);  t runs over max(0, n - window) .. n - 1
 *   (window 0: over 0 .. n - 1), token t at place t % page of page
 *   table[b][t / page]; an entry outside 0 .. pages - 1 masks its tokens
 *   x_t = scale sum_d q[b][h][d] k_t[d]        (k, v of key head h heads / H)
 *   out[b][h][d] = sum_t exp(x_t) v_t[d] / sum_t exp(x_t)
 *   lse[b][h] = log sum_t exp(x_t)
 * A sequence without a token to see (length 0, every page masked) gets a row of
 * zeros and lse = -infinity.  Scores are off by a few roundings of fp32 and by
 * what the queries are rounded to, 2^-30 (fp32) or 2^-22 (fp16, bf16) of the
 * head's largest; weights by 2^-21 of themselves and 2^-37 of the largest, and
 * exp(x_t) below 2^-126 of the largest may count as 0; sums are fp32, and the
 * output is rounded once.  Scales may have either sign.  A NaN scale among the
 * tokens that are seen, or an infinity or NaN in the query, makes the head's
 * outputs NaN; infinite scales and scores past fp32 give infinities or NaNs.
 *   q        [B x H x D] of q_dtype (fp32, fp16 or bf16), token stride ldq
 *            elements
 *   table    i32 [B x width], row stride ldt: the pages of each sequence.  Entries
 *            past the last token's may hold anything
 *   lengths  i32 [B]: tokens in the cache, the new one's included
 *   max_len  an upper bound of the lengths that the host knows: sequences are
 *            split over the card by it.  Longer ones count as max_len
 *   out      [B x H x D] contiguous of out_dtype; lse f32 [B x H] or NULL
 *   workspace  qa_attn_decode_workspace(...) bytes (any content; 0 where a
 *            sequence is not split, workspace may then be NULL)
 * Errors: (QA_ERR_SHAPE) B outside 0..2^20, heads outside 1..65535, H not a
 * multiple of heads, H > 65535, B H > 2^23, D, page, pages as qa_kv_write, width
 * or max_len negative, width page > 2^30, max_len > width page, ldt < width,
 * ldq < H D or not a multiple of 16 bytes, window < 0; (QA_ERR_VALUE) bad dtypes
 * or bits, scale not finite; NULL pointers; q, codes, scales and out not 16-byte,
 * table, lengths and lse not 4-byte, workspace not 256-byte aligned; small
 * workspace.  B == 0 is a no-op.
 * ------------------------------------------------------------------------- */
size_t qa_attn_decode_workspace(int64_t B, int32_t H, int32_t heads, int32_t D, int64_t max_len, int32_t window);
qa_status qa_attn_decode(const void* q, int64_t ldq, qa_dtype q_dtype, int64_t B, int32_t H, int32_t bits,
                         int64_t pages, int32_t heads, int32_t page, int32_t D, const void* k_codes,
                         const float* k_scales, const void* v_codes, const float* v_scales, const int32_t* table,
                         int64_t ldt, int64_t width, const int32_t* lengths, int64_t max_len, int32_t window,
                         float scale, void* out, qa_dtype out_dtype, float* lse_or_null, void* workspace,
                         size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * int8 linear on codes with bias, activation and residual
 *
 *   out[m][n] = act(s_x[m] s_w[n] sum_k Xq[m][k] Wq[n][k] + bias[n]) + residual[m][n]
 * formed in fp32 from the exact integer sum and rounded once.
 *   QA_ACT_NONE x; QA_ACT_RELU max(x, 0); QA_ACT_GELU x Phi(x);
 *   QA_ACT_GELU_TANH x (1 + tanh(sqrt(2 / pi) (x + 0.044715 x^3))) / 2;
 *   QA_ACT_SILU x / (1 + exp(-x))
 *   Xq, s_x  i8 [M x K], f32 [M] (qa_rmsnorm_int8 or qa_quantize_rowwise_int8)
 *   Wq, s_w  i8 [N x K], f32 [N]
 *   bias     f32 [N] or NULL
 *   residual [M x N] of dtype, row stride ldr elements, or NULL
 *   out      [M x N] of dtype, row stride ldo; may be residual itself (same
 *            pointer and stride), no other overlap with the inputs is allowed
 * A row whose scale is NaN (of a token without a finite norm) gives NaNs.
 * Errors: (QA_ERR_SHAPE) M outside 0..2^23, N outside 0..2^31 - 1,
 * ceil(M / 64) ceil(N / 64) >= 2^23, K not a positive multiple of 16 up to
 * 131072, ldo or ldr below N; (QA_ERR_VALUE) bad dtype or act; NULL pointers;
 * Xq and Wq not 16-byte, scales and bias not 4-byte, out and residual not
 * aligned to their elements.  M == 0 or N == 0 is a no-op.
 * ------------------------------------------------------------------------- */
typedef enum { QA_ACT_NONE = 0, QA_ACT_RELU = 1, QA_ACT_GELU = 2, QA_ACT_GELU_TANH = 3, QA_ACT_SILU = 4 } qa_act;
qa_status qa_qlinear_int8_act(const int8_t* Xq, const float* s_x, int64_t M, int64_t K, const int8_t* Wq,
                              const float* s_w, int64_t N, const float* bias_or_null, qa_act act,
                              const void* residual_or_null, int64_t ldr, void* out, int64_t ldo, qa_dtype dtype,
                              void* stream);

/* ---------------------------------------------------------------------------
 * Measurement helper, not part of the method: the single-launch HBM read
 * floor that the decode kernel (one launch streaming the whole int8 weight)
 * is compared with.
 *
 * qa_probe_stream_read
 *   Reads src[0 .. bytes) once with wgs workgroups of 512 threads, each a
 *   contiguous slice; every load instruction moves lane_bytes bytes per lane
 *   (64 * lane_bytes contiguous bytes per wave instruction) and `unroll`
 *   loads per lane are in flight before any is used.  The data are folded
 *   into a value stored to sink[wg * 512 + thread] only if it equals a fixed
 *   constant (so sink is normally left untouched; it must hold wgs * 512
 *   u32).  bytes == 0 launches the same grid with nothing to read (the cost
 *   of the launch itself).
 *   src: device, 16-byte aligned; sink: device u32 [wgs * 512].
 *   Errors: NULL pointers, wgs not in [1, 65536], lane_bytes not 4, 8 or 16,
 *   unroll not 1, 2, 4 or 8, misaligned src.
 * ------------------------------------------------------------------------- */
qa_status qa_probe_stream_read(const void* src, size_t bytes, int32_t wgs, int32_t lane_bytes, int32_t unroll,
                               uint32_t* sink, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QA_H */
