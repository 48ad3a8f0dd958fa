/*
 * fp8blk.h -- FP8 quantization with fine-grained scaling and block-scaled FP8
 * GEMM for AMD Instinct MI355X (gfx950).  C ABI.
 *
 * What the library computes (each entry point cites the passage that defines
 * it):
 *   quantize    x_fp8 = clip(round(x / s), -Vmax, Vmax) with s = amax / Vmax
 *               taken over each scale group of the current tensor
 *   dequantize  x_hat = x_fp8 * s
 *   GEMM        Out = (X_fp8 * s_X) @ (W_fp8 * s_W)^T = s_X * s_W * (X_fp8 @ W_fp8^T),
 *               accumulated in fp32, with per-128-K scale promotion for tile/block
 *               scales and power-of-two microscales for MX blocks.
 * Sources: "The FP8 Family" (sections "The two shapes", "Scaling is what makes
 * FP8 usable", "The scaling granularity ladder", the DeepSeek-V3 callout);
 * "FP8 Mixed-Precision Serving" (sections "The Mathematics of FP8" and
 * "Quantization Granularity and Scaling Topologies"); "Illustrated GPU kernels,
 * Part 8" (the qdq listing and its comments, the NVIDIA scaling taxonomy, the
 * OCP MX paragraph, and the promotion paragraph).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Memory:     every tensor pointer is DEVICE memory owned by the caller.  The
 *             library allocates nothing and keeps no per-call state.
 * Streams:    work is enqueued on `stream` (0 = the null stream) and the call
 *             returns without synchronizing; outputs are valid once the stream
 *             reaches that point.
 * Layouts:    row-major.  An operand is [rows, cols] with cols (= K) contiguous.
 *             FP8 codes are one byte per element, element i at byte i.
 *             bf16 values are stored as 16-bit patterns.
 * Errors:     arguments are checked on the host before any HIP call; a bad
 *             argument returns an FP8_ERR_* code and enqueues nothing.  A failed
 *             launch returns FP8_ERR_HIP.  Nothing is thrown across the ABI.
 * Alignment:  tensor pointers (x, q, y, a, b, out) must be 16-byte aligned;
 *             fp32 scale arrays 4-byte aligned; the GEMM reads UE8M0 scale
 *             arrays as 4-byte words, so there they are 4-byte aligned too
 *             (FP8_ERR_ALIGN otherwise).
 * Inputs:     quantize inputs must be finite; the result for NaN/Inf input is
 *             unspecified (fp8_cast defines it).
 * Empty:      rows == 0 or cols == 0 (M == 0 or N == 0) is valid and does no work,
 *             except that a per-tensor quantize still writes its scale (1.0).
 */
#ifndef FP8BLK_H
#define FP8BLK_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FP8BLK_ABI_VERSION 1

/* FP8 code formats ("The FP8 Family", format table and bit layout; "FP8
 * Mixed-Precision Serving", "The Mathematics of FP8"):
 *   E4M3: bias 7, max 448, min normal 2^-6, subnormals 2^-6*M/8, no Inf, NaN = S.1111.111
 *   E5M2: bias 15, max 57344, min normal 2^-14, IEEE Inf/NaN (0x7C/0xFC = +-Inf) */
typedef enum { FP8_E4M3 = 0, FP8_E5M2 = 1 } fp8_format_t;

/* Scale granularity of one [rows, K] operand and the layout of its scale array
 * ("The FP8 Family", granularity table and DeepSeek-V3 callout; "Part 8",
 * taxonomy list and OCP MX paragraph):
 *   FP8_GRAN_TENSOR         float[1]                          one scale per tensor
 *   FP8_GRAN_ROW            float[rows]                       per token (X) / per output channel (W)
 *   FP8_GRAN_TILE_1x128     float[rows][K/128]  row-major     1 x 128 tiles
 *   FP8_GRAN_BLOCK_128x128  float[rows/128][K/128] row-major  128 x 128 blocks (rows % 128 == 0)
 *   FP8_GRAN_MX32           uint8[rows][K/32]   row-major     UE8M0 byte e+127 per 32 elements
 * fp32 scales are s = RN32(amax / Vmax) (1.0 when that is 0).  The UE8M0
 * exponent e is the smallest integer with amax <= Vmax * 2^e, clamped to
 * [-127, 127] (-127 for an all-zero block); byte 255 is never written and
 * decodes to NaN. */
typedef enum {
  FP8_GRAN_TENSOR = 0,
  FP8_GRAN_ROW = 1,
  FP8_GRAN_TILE_1x128 = 2,
  FP8_GRAN_BLOCK_128x128 = 3,
  FP8_GRAN_MX32 = 4
} fp8_granularity_t;

/* High-precision carriers: fp32, and bf16 (16-bit patterns; conversion to bf16
 * rounds to nearest even). */
typedef enum { FP8_DT_F32 = 0, FP8_DT_BF16 = 1 } fp8_dtype_t;

/* Kernel choice for the GEMM.  AUTO picks the skinny (weight-streaming) kernel
 * for M <= 64 and the tiled MFMA kernel otherwise. */
typedef enum { FP8_GEMM_AUTO = 0, FP8_GEMM_TILED = 1, FP8_GEMM_SKINNY = 2 } fp8_gemm_algo_t;

/* Accumulation of the FP8 products in the GEMM.
 *   FP8_ACCUM_FP32    (default) the products of the decoded values are formed
 *                     exactly and summed in fp32: the codes are expanded exactly
 *                     to bf16 in registers and multiplied on the bf16 matrix
 *                     cores.  Meets |out - exact| <= 1e-4 * sum_k |x_k w_k|.
 *   FP8_ACCUM_NATIVE  the FP8 matrix-core instructions' own accumulation, at
 *                     twice their peak rate.  On gfx950 these add each group of
 *                     8 products in a fixed-point window 14 bits below the
 *                     largest of the 8, truncating smaller products, before the
 *                     fp32 sum; the error of one group can reach 7 * 2^-13 of its
 *                     largest product.  ("Illustrated GPU kernels, Part 8", the
 *                     promotion paragraph and the first of its five rules, note
 *                     the same kind of internal limit for Hopper's FP8 MMA.) */
typedef enum { FP8_ACCUM_FP32 = 0, FP8_ACCUM_NATIVE = 1 } fp8_accum_t;

typedef enum {
  FP8_OK = 0,
  FP8_ERR_NULL = 1,        /* a required pointer is NULL                          */
  FP8_ERR_ENUM = 2,        /* a format / granularity / dtype / algo value is invalid */
  FP8_ERR_SHAPE = 3,       /* negative size, K % 128 != 0, rows % 128 != 0 for     */
                           /* 128x128 blocks, M or N % 16 != 0 or K > 2^22 for the  */
                           /* GEMM, KV head_dim % 16 != 0 or ld_x < heads*head_dim  */
  FP8_ERR_UNSUPPORTED = 4, /* a valid but unsupported combination                 */
  FP8_ERR_WORKSPACE = 5,   /* workspace missing or smaller than required          */
  FP8_ERR_HIP = 6,         /* a HIP launch failed                                  */
  FP8_ERR_ALIGN = 7        /* a pointer is not aligned as documented above        */
} fp8_status_t;

/* Short description of a status code (static string, never NULL). */
const char* fp8_status_string(fp8_status_t status);

/* FP8BLK_ABI_VERSION of the built library. */
int fp8_abi_version(void);

/* Device workspace fp8_quantize needs for this shape and granularity, in
 * bytes.  Non-zero only for FP8_GRAN_TENSOR (per-workgroup partial maxima of
 * the amax pass, at most 32 KiB).  Returns 0 for invalid arguments. */
size_t fp8_quantize_workspace_bytes(int64_t rows, int64_t cols, fp8_granularity_t g);

/* Quantize a [rows, cols] operand with current (just-in-time) scaling.
 *   x      : input, fp32 or bf16 per x_dt, [rows, cols] row-major
 *   fmt    : output code format
 *   g      : scale granularity (layout of `scales` as listed above)
 *   q      : output codes, uint8 [rows, cols]
 *   scales : output scales, float[...] or uint8[...] (MX32) as listed above
 *   workspace, ws_bytes : device scratch of fp8_quantize_workspace_bytes() bytes
 *            (may be NULL when that is 0)
 * Per group: amax = max|x|; s = RN32(amax / Vmax); each element becomes
 * code(RN32(x / s)) where code() rounds to nearest even and saturates finite
 * overflow to +-Vmax, keeping the sign of zero (MX32: code(x * 2^-e)).
 * ("The FP8 Family", "Scaling is what makes FP8 usable", quantize formula;
 * "FP8 Mixed-Precision Serving", scale formula and block-wise formula;
 * "Part 8", qdq listing comments on amax/448, round-to-nearest-even and
 * saturation.)
 * Shapes: cols % 128 == 0; rows % 128 == 0 for FP8_GRAN_BLOCK_128x128. */
fp8_status_t fp8_quantize(const void* x, fp8_dtype_t x_dt, int64_t rows, int64_t cols,
                          fp8_format_t fmt, fp8_granularity_t g,
                          uint8_t* q, void* scales, void* workspace, size_t ws_bytes,
                          hipStream_t stream);

/* fp8_quantize for callers that cannot allocate device memory: code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc.  Same
 * arguments and results as fp8_quantize without the workspace: the one
 * granularity that needs scratch (FP8_GRAN_TENSOR: per-workgroup amax partials)
 * uses a static 32 KiB device array of the library instead, which covers every
 * tensor size (FP8_ERR_WORKSPACE would report a need beyond it).  Each GPU holds
 * its own copy of that array until the process ends; its device address is
 * looked up on the first call on a device (that call alone makes HIP runtime
 * queries besides the launches; none allocates).  Every call on a GPU shares
 * the array, so per-tensor calls that overlap on one GPU (concurrent streams or
 * threads) race and give undefined results; calls ordered on one stream are
 * safe.  Nothing in the array needs clearing between calls. */
fp8_status_t fp8_quantize_noalloc(const void* x, fp8_dtype_t x_dt, int64_t rows, int64_t cols,
                                  fp8_format_t fmt, fp8_granularity_t g, uint8_t* q, void* scales,
                                  hipStream_t stream);

/* Quantize a whole [rows, cols] tensor with delayed scaling ("FP8
 * Mixed-Precision Serving", section "Quantization Granularity and Scaling
 * Topologies", delayed scaling): the scale comes from a history of the amax
 * of earlier iterations instead of from this tensor, saving the reduction
 * pass before the encode.
 *   history   device fp32 [hist_len], caller-owned ring of amax values
 *             (zero-initialized; NaN entries are ignored)
 *   scale     device fp32 [1]: written with s = RN32(max(history) * 2^margin /
 *             Vmax), 1 when that is 0 (the inverse of the page's
 *             rho = FP8max / (2^m max(H)))
 *   q         codes under s; values beyond s * Vmax saturate to +-Vmax
 *   then history[hist_pos] = max |x| of this tensor (the caller advances
 *   hist_pos, modulo hist_len, between iterations).
 * 0 <= hist_pos < hist_len, 1 <= hist_len <= 2^30, 0 <= margin <= 31; cols as
 * for fp8_quantize.  The workspace is as for FP8_GRAN_TENSOR
 * (fp8_quantize_workspace_bytes(rows, cols, FP8_GRAN_TENSOR)).  Everything
 * runs on the stream: no host synchronization. */
fp8_status_t fp8_quantize_delayed(const void* x, fp8_dtype_t x_dt, int64_t rows, int64_t cols,
                                  fp8_format_t fmt, float* history, int64_t hist_len, int64_t hist_pos,
                                  int margin, uint8_t* q, float* scale, void* workspace, size_t ws_bytes,
                                  hipStream_t stream);

/* Dequantize codes back to fp32 or bf16: y = RN32(decode(q) * s) (MX32:
 * decode(q) * 2^e), then rounded to bf16 if y_dt is FP8_DT_BF16.
 * ("The FP8 Family", dequant formula; "Part 8", the dequantization multiply
 * in the qdq listing.)  NaN codes give NaN; E5M2 Inf codes give +-Inf.
 * Arguments mirror fp8_quantize; y is [rows, cols] of y_dt. */
fp8_status_t fp8_dequantize(const uint8_t* q, const void* scales, int64_t rows, int64_t cols,
                            fp8_format_t fmt, fp8_granularity_t g,
                            void* y, fp8_dtype_t y_dt, hipStream_t stream);

/* Unscaled saturating cast of n values (s = 1): code = round-to-nearest-even
 * of x with finite overflow clamped to +-Vmax and the sign of zero kept
 * ("Part 8", qdq listing comments).  Defined for every input: NaN -> 0x7F/0xFF
 * by sign; +-Inf -> +-448 (E4M3, which has no Inf) or +-Inf (E5M2).
 * n % 8 == 0. */
fp8_status_t fp8_cast(const void* x, fp8_dtype_t x_dt, int64_t n, fp8_format_t fmt,
                      uint8_t* q, hipStream_t stream);

/* Block-scaled FP8 GEMM:
 *   out[m, n] = sum_k decode(a[m,k]) * sA(m,k) * decode(b[n,k]) * sB(n,k)
 * with a = X codes [M, K], b = W codes [N, K] (both K-contiguous), out [M, N]
 * row-major in out_dt; products formed exactly and accumulated in fp32.
 * ("The FP8 Family", the MMA identity under "Scaling is what makes FP8 usable"
 * and the accumulator-promotion bullet of the DeepSeek-V3 callout; "Part 8",
 * the promotion paragraph and the OCP MX paragraph.)
 * Supported (a_g, b_g) pairs:
 *   TENSOR/ROW x TENSOR/ROW   scales applied once in the epilogue
 *   TILE_1x128 x BLOCK_128x128 each 128-K partial product is scaled by
 *                              sA[m,kb] * sB[n/128,kb] and added to an fp32
 *                              accumulator (promotion every 128 K)
 *   MX32 x MX32                power-of-two scales 2^(eA + eB) applied per
 *                              32-K block: folded exactly into the operands'
 *                              expansion while every code times 2^e stays in
 *                              bf16's normal range (e in [-117, 119] for E4M3,
 *                              [-110, 112] for E5M2), else applied to each
 *                              block's fp32 sum; the native accumulation gives
 *                              the bytes to the scaled matrix-core instruction
 * Any other pair returns FP8_ERR_UNSUPPORTED.  Formats may differ per operand.
 * Accuracy (FP8_ACCUM_FP32): |out - exact| <= 1e-4 * sum_k |x_k w_k| holds for
 * every code and every UE8M0 exponent, including operands whose decoded values
 * alone lie outside fp32's range (a code times 2^e up to 2^128 or down to
 * 2^-136), as long as every scaled product x_k w_k, every partial sum and the
 * result lie in fp32's normal range [2^-126, 2^128).  A result outside that
 * range cannot be represented to that accuracy in fp32 (it under- or
 * overflows); a bf16 output adds its own rounding, half a bf16 ulp.
 * Shapes: M % 16 == 0, N % 16 == 0, K % 128 == 0, K <= 2^22 (the kernels
 * address up to 256 operand rows through 32-bit buffer offsets); N % 128 == 0
 * for a BLOCK_128x128 b.  K == 0 writes zeros. */
fp8_status_t fp8_gemm_blockscaled(const uint8_t* a, fp8_format_t a_fmt, fp8_granularity_t a_g,
                                  const void* a_scales,
                                  const uint8_t* b, fp8_format_t b_fmt, fp8_granularity_t b_g,
                                  const void* b_scales,
                                  int64_t M, int64_t N, int64_t K,
                                  void* out, fp8_dtype_t out_dt, hipStream_t stream);

/* Same as fp8_gemm_blockscaled (which is AUTO with FP8_ACCUM_FP32) with an
 * explicit kernel and accumulation choice.  The skinny kernel accepts M <= 64
 * only (FP8_ERR_UNSUPPORTED otherwise). */
fp8_status_t fp8_gemm_blockscaled_ex(const uint8_t* a, fp8_format_t a_fmt, fp8_granularity_t a_g,
                                     const void* a_scales,
                                     const uint8_t* b, fp8_format_t b_fmt, fp8_granularity_t b_g,
                                     const void* b_scales,
                                     int64_t M, int64_t N, int64_t K,
                                     void* out, fp8_dtype_t out_dt, fp8_gemm_algo_t algo,
                                     fp8_accum_t accum, hipStream_t stream);

/* Block-scaled FP8 GEMM whose result leaves the kernel already quantized for
 * the next layer ("Illustrated GPU kernels, Part 8", the fourth of its five
 * closing rules: quantize in the epilogue of the kernel that produces the
 * tensor, where the per-block amax is a reduction over values already in
 * registers; "The FP8 Family", DeepSeek-V3 callout: 1x128 activation tiles).
 * Operands, scale pairs, shapes and accum are as for fp8_gemm_blockscaled_ex.
 * The fp32 result (bit for bit the values an FP8_DT_F32 call with the same
 * accum writes) is quantized per row and 128 output columns to out_fmt exactly
 * as fp8_quantize does with FP8_GRAN_TILE_1x128:
 *   out_codes   uint8 [M, N]      one code per element
 *   out_scales  fp32 [M, N/128]   s = RN32(amax / Vmax) of each row tile
 * so (out_codes, out_scales) can be the next GEMM's a / a_scales directly.
 * Requires N % 128 == 0 (FP8_ERR_SHAPE otherwise); out_codes 16-byte and
 * out_scales 4-byte aligned.  K == 0 writes zero codes and scales of 1.
 * Always runs the tiled kernel. */
fp8_status_t fp8_gemm_blockscaled_quant(const uint8_t* a, fp8_format_t a_fmt, fp8_granularity_t a_g,
                                        const void* a_scales,
                                        const uint8_t* b, fp8_format_t b_fmt, fp8_granularity_t b_g,
                                        const void* b_scales,
                                        int64_t M, int64_t N, int64_t K,
                                        fp8_format_t out_fmt, uint8_t* out_codes, float* out_scales,
                                        fp8_accum_t accum, hipStream_t stream);

/* ---- FP8 KV cache ----------------------------------------------------------
 * Key and value states stored as FP8 codes, one byte per element ("FP8
 * Mixed-Precision Serving", section "FP8 KV Cache Architecture and Serving
 * Latency": Memory_KV = 2 * B * L * N_heads * D_head * bytes, halved from bf16;
 * "FP8 Serving", quality table and "Things to try": per-tensor or per-channel
 * scales, E5M2 as the wider-range format).
 * The cache is a pool of num_slots slots; a slot holds one token's
 * [heads, head_dim] codes (uint8 [num_slots, heads, head_dim], row-major).  A
 * paged cache with blocks of b tokens is the same pool with slot =
 * block * b + offset.  Keys and values are two caches and two calls.
 * Scales are static (calibrated by the caller) fp32 values, positive and not
 * NaN (+Inf allowed: codes become signed zeros):
 *   FP8_KV_SCALE_TENSOR   float[1]
 *   FP8_KV_SCALE_HEAD     float[heads]
 *   FP8_KV_SCALE_CHANNEL  float[heads * head_dim]   (head-major)
 * Shapes: head_dim % 16 == 0; heads * head_dim <= 2^24.  Empty calls (no
 * tokens / rows, or heads * head_dim == 0) are valid and do nothing.
 * Duplicate append slots in one call race (one of the rows lands). */
typedef enum {
  FP8_KV_SCALE_TENSOR = 0,
  FP8_KV_SCALE_HEAD = 1,
  FP8_KV_SCALE_CHANNEL = 2
} fp8_kv_scale_t;

/* Quantize on append: for t in [0, tokens) with 0 <= slots[t] < num_slots,
 * cache[slots[t]] = code(RN32(x[t] / s)) elementwise, where code() rounds to
 * nearest even and saturates to +-Vmax (also when the quotient leaves the
 * fp32 range); tokens whose slot is outside the pool are skipped (padding).
 *   x      fp32 or bf16 [tokens, ld_x] with row t's [heads, head_dim] values
 *          in its first heads * head_dim elements; ld_x >= heads * head_dim and
 *          rows 16-byte aligned (ld_x % 4 == 0 for fp32, % 8 for bf16;
 *          FP8_ERR_ALIGN otherwise), so x may be a slice of a fused QKV output
 *   slots  int64 [tokens], device, 8-byte aligned
 *   cache  uint8 [num_slots, heads, head_dim], 16-byte aligned
 * x must be finite. */
fp8_status_t fp8_kv_append(const void* x, fp8_dtype_t x_dt, int64_t tokens, int64_t heads, int64_t head_dim,
                           int64_t ld_x, const int64_t* slots, fp8_format_t fmt, fp8_kv_scale_t scale_kind,
                           const float* scales, uint8_t* cache, int64_t num_slots, hipStream_t stream);

/* Dequantize on read: out[i] = RN32(decode(cache[slots[i]]) * s) elementwise,
 * rounded to bf16 (nearest even) when out_dt is FP8_DT_BF16; a row whose slot
 * is outside [0, num_slots) is written as zeros.
 *   slots  int64 [n], device, 8-byte aligned
 *   out    [n, heads, head_dim] contiguous, 16-byte aligned */
fp8_status_t fp8_kv_gather(const uint8_t* cache, int64_t num_slots, int64_t heads, int64_t head_dim,
                           const int64_t* slots, int64_t n, fp8_format_t fmt, fp8_kv_scale_t scale_kind,
                           const float* scales, void* out, fp8_dtype_t out_dt, hipStream_t stream);

/* ---- Attention over the FP8 KV cache -----------------------------------------
 * What the cache is for ("FP8 Mixed-Precision Serving", section "FP8 KV Cache
 * Architecture and Serving Latency": every decode step reads the whole cache,
 * whose codes are half the bytes of bf16): softmax attention of new tokens
 * over the codes where they lie, with no dequantized copy.
 *
 * Pages: position j of sequence b is slot
 *   block_table[b, j / block_size] * block_size + j % block_size
 * of both caches (the pools of fp8_kv_append); block_size 1 makes the table a
 * slot list.  A position whose slot lies outside [0, num_slots) is left out,
 * so a page can be dropped by writing -1 into the table.  Sequences may share
 * pages.
 *
 * fp8_kv_attention: query tokens q_starts[b] .. q_starts[b+1]-1 are the newest
 * q_len tokens of sequence b, whose kv_lens[b] positions (the new tokens' own
 * among them, appended before) are in the cache.  With kh = h / (heads / kv_heads),
 * khat = decode(k code) * k_scale and vhat alike, token i of the sequence sees
 * the positions j < kv_lens[b] - q_len + i + 1 whose slot is in the pool:
 *   s_j = softmax_scale * sum_c q[i, h, c] khat[j, kh, c]
 *   out[i, h] = sum_j p_j vhat[j, kh],  p = softmax(s)
 *   lse[i, h] = log sum_j exp(s_j)   (natural logarithm; lse may be NULL)
 * A token that sees nothing gets zeros and an lse of -Inf.  What a token does
 * not see (later tokens, stale or NaN codes behind a sequence's last position)
 * has no influence on it; a NaN or Inf code that it sees is its result.
 * weights_out (may be NULL; then weights_in is ignored): the attention weight
 * that each position has received,
 *   weights_out[b, kh, j] = weights_in[b, kh, j] + sum of p_j over the
 *                           sequence's query tokens and the heads of kh,
 * for j < kv_lens[b]; weights_in NULL counts as zeros, and it may be
 * weights_out itself.  Entries behind kv_lens[b] are left as they are.  The
 * sums are formed in a fixed order: equal calls give equal bits.
 *   q            fp32 or bf16 [q_tokens, ld_q], a row's [heads, head_dim]
 *                values in its first heads * head_dim elements; ld_q and
 *                alignment as for fp8_kv_append's x, so q may be a slice of a
 *                fused QKV output
 *   k_cache, v_cache  uint8 [num_slots, kv_heads, head_dim], 16-byte aligned
 *   block_table  int64 [batch, max_blocks];  q_starts  int64 [batch + 1],
 *                ascending;  kv_lens  int64 [batch]; device, 8-byte aligned
 *   max_q        at least every q_len;  max_kv  at least every kv_len, and at
 *                most max_blocks * block_size.  They size the launch: tokens
 *                past max_q are left unwritten, positions past max_kv unread
 *   k_scales, v_scales  as for fp8_kv_append (finite)
 *   out          [q_tokens, heads, head_dim] of out_dt, 16-byte aligned;
 *                lse fp32 [q_tokens, heads].  Rows of tokens that belong to
 *                no sequence are left as they are; neither overlaps an input
 *   weights_in, weights_out  fp32 [batch, kv_heads, ld_w], ld_w >= max_kv
 *   workspace    fp8_kv_attention_workspace_bytes(...) bytes, 16-byte aligned;
 *                calls that may overlap need one each
 * heads % kv_heads == 0; head_dim 64, 128 or 256 (else FP8_ERR_UNSUPPORTED);
 * softmax_scale positive and finite (else FP8_ERR_UNSUPPORTED); num_slots <
 * 2^31; max_kv <= 2^30; q finite.  Accuracy: codes enter the matrix cores as
 * exact fp16, a row of q (times the key scales where they differ by channel)
 * as one fp16 where that is exact (bf16 q, scales per tensor or head) and else
 * as two (22 bits), p as one fp16 (11 bits) for a bf16 out and as two for an
 * fp32 out.  Sums are fp32. */
size_t fp8_kv_attention_workspace_bytes(int64_t q_tokens, int64_t heads, int64_t kv_heads, int64_t head_dim,
                                        int64_t batch, int64_t max_q, int64_t max_kv, int with_weights);
fp8_status_t fp8_kv_attention(const void* q, fp8_dtype_t q_dt, int64_t q_tokens, int64_t heads, int64_t kv_heads,
                              int64_t head_dim, int64_t ld_q, const uint8_t* k_cache, const uint8_t* v_cache,
                              int64_t num_slots, const int64_t* block_table, int64_t max_blocks, int64_t block_size,
                              int64_t batch, const int64_t* q_starts, const int64_t* kv_lens, int64_t max_q,
                              int64_t max_kv, fp8_format_t fmt, fp8_kv_scale_t scale_kind, const float* k_scales,
                              const float* v_scales, float softmax_scale, void* out, fp8_dtype_t out_dt, float* lse,
                              const float* weights_in, float* weights_out, int64_t ld_w, void* workspace,
                              size_t ws_bytes, hipStream_t stream);

/* Which positions of a full cache to keep, by the attention weight they have
 * received.  For sequence b with n = clamp(kv_lens[b], 0, max_kv) positions:
 *   score[j] = RN32(sum over kv heads of weights[b, kh, j])
 * (summed in 64 bits; NaN counts as the lowest score).  All n positions are
 * kept when n <= keep.  Else the first `first` and the last `recent` positions
 * are kept, and of the others those with the largest scores, ties to the
 * lowest position, until `keep` are.
 *   kept       int64 [batch, keep], the positions ascending, -1 behind the last
 *   kept_lens  int64 [batch], their number
 *   weights    fp32 [batch, kv_heads, ld_w], ld_w >= max_kv
 *   workspace  fp8_kv_evict_select_workspace_bytes(batch, max_kv) bytes,
 *              16-byte aligned
 * first + recent <= keep (FP8_ERR_SHAPE otherwise); max_kv <= 2^30. */
size_t fp8_kv_evict_select_workspace_bytes(int64_t batch, int64_t max_kv);
fp8_status_t fp8_kv_evict_select(const float* weights, int64_t ld_w, int64_t batch, int64_t kv_heads,
                                 const int64_t* kv_lens, int64_t max_kv, int64_t keep, int64_t first, int64_t recent,
                                 int64_t* kept, int64_t* kept_lens, void* workspace, size_t ws_bytes,
                                 hipStream_t stream);

/* Move the kept positions of every sequence together, in both caches and in
 * the weights: for i < min(kept_lens[b], keep) with j = kept[b, i],
 *   cache row of position i under dst_table[b]  =  row of position j under src_table[b]
 *   weights_out[b, :, i] = weights_in[b, :, j]   (both may be NULL)
 * dst_table may be src_table (compaction in place; the pages behind the last
 * kept position are then free).  A table of its own names pages that the call's
 * sources do not touch, or the page that src_table[b] has in the same place
 * (pages shared with another sequence must not be written in place); one
 * address with two row lengths is refused for batch > 1 (FP8_ERR_SHAPE).
 * In the same way weights_out may be weights_in with ld_out == ld_in.  Each
 * row of kept ascends strictly (as fp8_kv_evict_select writes it).  A position
 * outside its table or a slot outside the pool, on either side, leaves the
 * destination as it was.
 *   src_table  int64 [batch, src_blocks], dst_table int64 [batch, dst_blocks]
 *   kept int64 [batch, keep];  kept_lens int64 [batch]
 *   weights_in fp32 [batch, kv_heads, ld_in], weights_out [.., ld_out]: an
 *   entry j >= ld_in is not read, i >= ld_out not written
 * head_dim % 16 == 0; num_slots < 2^31. */
fp8_status_t fp8_kv_compact(uint8_t* k_cache, uint8_t* v_cache, int64_t num_slots, int64_t kv_heads,
                            int64_t head_dim, const int64_t* src_table, int64_t src_blocks,
                            const int64_t* dst_table, int64_t dst_blocks, int64_t block_size, int64_t batch,
                            const int64_t* kept, const int64_t* kept_lens, int64_t keep, const float* weights_in,
                            int64_t ld_in, float* weights_out, int64_t ld_out, hipStream_t stream);

/* Causal attention of whole prompts packed one behind the other, over the
 * states before they are quantized into the cache: sequence b is the tokens
 * seq_starts[b] .. seq_starts[b+1]-1, and token i of it sees its tokens 0..i.
 * Formulas, lse and shared heads as for fp8_kv_attention, with k and v in
 * place of khat and vhat; what a token does not see has no influence on it,
 * also where it is NaN or Inf.
 *   q  bf16 [tokens, ld_q] ([heads, head_dim] in front), k, v bf16
 *      [tokens, ld_k], [tokens, ld_v] ([kv_heads, head_dim] in front): all three
 *      may be slices of a fused QKV output; 16-byte aligned, ld % 8 == 0
 *   seq_starts  int64 [batch + 1], ascending, device;  max_len at least every
 *      sequence's length: tokens past it are left unwritten
 *   out  bf16 [tokens, heads, head_dim];  lse fp32 [tokens, heads] or NULL.
 *      Rows of tokens of no sequence are left as they are; neither overlaps
 *      an input
 *   workspace  fp8_prompt_attention_workspace_bytes(...) bytes (0 unless there
 *      are few rows), 16-byte aligned; calls that may overlap need one each
 * heads % kv_heads == 0; head_dim 64, 128 or 256; tokens < 2^30;
 * softmax_scale positive and finite.  p is rounded to bf16 for the second
 * product; sums are fp32. */
size_t fp8_prompt_attention_workspace_bytes(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_dim,
                                            int64_t batch, int64_t max_len);
fp8_status_t fp8_prompt_attention(const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v,
                                  int64_t ld_v, int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_dim,
                                  int64_t batch, const int64_t* seq_starts, int64_t max_len, float softmax_scale,
                                  void* out, float* lse, void* workspace, size_t ws_bytes, hipStream_t stream);

/* ---- FP4 (E2M1) with two-level microscaling ---------------------------------
 * ("Illustrated GPU kernels, Part 8", section "Low precision: FP8, FP4, and
 * microscaling": the OCP MX block of 32 elements with one UE8M0 scale, and
 * NVFP4's blocks of 16 with an E4M3 microscale plus one FP32 scale per tensor
 * that keeps the microscales inside E4M3's range.)
 * E2M1: 1 sign, 2 exponent, 1 mantissa bit, bias 1; magnitudes 0, 0.5, 1,
 * 1.5, 2, 3, 4, 6; no Inf or NaN.  Codes are packed two per byte, element 2i
 * in the low nibble: a [rows, cols] operand is uint8 [rows, cols/2].
 *   FP4_SCALE_MX  block_scales uint8 [rows, cols/32]: byte e + 127, e the
 *                 smallest integer with amax <= 6 * 2^e (clamped to
 *                 [-127, 127]); codes = cast(x * 2^-e).  No tensor scale.
 *   FP4_SCALE_NV  block_scales uint8 [rows, cols/16]: E4M3 microscale codes;
 *                 tensor_scale float[1].  s_t = RN32(amax / 2688) (1 when 0);
 *                 per block u = RN32(amax_b / RN32(6 s_t)), m = E4M3(u) (RNE,
 *                 saturating), S = RN32(m * s_t); codes = cast(RN32(x / S)),
 *                 signed zeros when S == 0.
 * cast() rounds to nearest even, saturates to +-6 and keeps the sign of zero. */
typedef enum { FP4_SCALE_MX = 0, FP4_SCALE_NV = 1 } fp4_scaling_t;

/* Device workspace fp4_quantize needs (NV: partial maxima of the tensor amax,
 * at most 32 KiB; MX: 0).  Returns 0 for invalid arguments. */
size_t fp4_quantize_workspace_bytes(int64_t rows, int64_t cols, fp4_scaling_t kind);

/* Quantize x [rows, cols] (fp32 or bf16, finite) to packed E2M1 codes q with
 * the block scales (and, for NV, the tensor scale) above.  cols % 128 == 0;
 * x and q 16-byte aligned, tensor_scale 4-byte aligned.  An empty NV tensor
 * writes the tensor scale 1. */
fp8_status_t fp4_quantize(const void* x, fp8_dtype_t x_dt, int64_t rows, int64_t cols, fp4_scaling_t kind,
                          uint8_t* q, uint8_t* block_scales, float* tensor_scale, void* workspace, size_t ws_bytes,
                          hipStream_t stream);

/* Dequantize: MX y = decode(q) * 2^e (scale byte 255 gives NaN); NV
 * y = RN32(decode(q) * S), S = RN32(m * s_t); then RNE bf16 when y_dt is
 * FP8_DT_BF16.  Shapes and alignment as for fp4_quantize. */
fp8_status_t fp4_dequantize(const uint8_t* q, const uint8_t* block_scales, const float* tensor_scale,
                            int64_t rows, int64_t cols, fp4_scaling_t kind, void* y, fp8_dtype_t y_dt,
                            hipStream_t stream);

/* FP4 block-scaled GEMM: out[m, n] = sum_k deq(a[m, k]) deq(b[n, k]) for
 * packed E2M1 operands a [M, K/2] and b [N, K/2] (both K-contiguous) of the
 * same kind:
 *   FP4_SCALE_MX  sum_k qa 2^ea qb 2^eb      (a_scales [M, K/32], b_scales [N, K/32])
 *   FP4_SCALE_NV  s_ta s_tb sum_k (qa ma)(qb mb)   (E4M3 microscales [M, K/16],
 *                 [N, K/16]; tensor scales a_tensor_scale, b_tensor_scale)
 * ("Illustrated GPU kernels, Part 8", "Low precision: FP8, FP4, and
 * microscaling": the scale factors travel with the data into the matrix
 * multiply.)  MX runs on the FP4 matrix cores: each 32-element block's
 * products are summed exactly, scaled by 2^(ea + eb), and the block sums are
 * added in fp32.  NV expands each code times its microscale exactly to fp16,
 * sums in fp32 on the fp16 matrix cores, and multiplies the result by the
 * tensor scales.  M <= 64 (decode shapes) runs a kernel that streams b once.
 * Meets |out - exact| <= 1e-4 sum_k |deq products| (plus half
 * a bf16 ulp for bf16 output) while the scaled products stay inside fp32's
 * range.
 * Shapes: M % 16 == 0, N % 16 == 0, K % 256 == 0, K <= 2^22.  a, b, out
 * 16-byte aligned; scale arrays 4-byte aligned.  out_dt FP8_DT_F32 or
 * FP8_DT_BF16.  K == 0 writes zeros. */
fp8_status_t fp4_gemm_blockscaled(const uint8_t* a, const uint8_t* a_scales, const float* a_tensor_scale,
                                  const uint8_t* b, const uint8_t* b_scales, const float* b_tensor_scale,
                                  int64_t M, int64_t N, int64_t K, fp4_scaling_t kind, void* out,
                                  fp8_dtype_t out_dt, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8BLK_H */
