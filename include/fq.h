/*
 * libfq -- fused small-matrix transform + dynamic low-bit quantization for AMD
 * Instinct MI355X (gfx950).
 *
 * The operator is the one stated on the page "aclnnFlatQuantV2 算子拆解：两步矩阵乘 +
 * 动态量化，CANN 上怎么写一次讲清" (cited as [FQV2] with the page's section names).
 * For every slice x_k [M, N] of x [K, M, N]:
 *
 *   T   = round_to_dtype(x_k . P2)          [FQV2] 拆开算, 第1步 (skipped when P2 is [0, 0])
 *   y_k = P1 . T   (fp32, never stored)     [FQV2] 拆开算, 第2步
 *
 * then one of two dynamic quantizations ([FQV2] 拆开算, 第3步 and 第4步):
 *
 *   per token (out INT32 or INT4):
 *       quantScale[k] = max|y_k| / (7 / clipRatio)              (fp32)
 *       code          = clamp(round_half_even(y / quantScale[k]), -8, 7)
 *   per group of 32 consecutive elements of the flattened slice (out FLOAT4_E2M1):
 *       dstTypeMax == 0  (V1): e8m0 = floor(log2(group max)) - 2 + 127, clamped to [0, 254]
 *       dstTypeMax in [6, 12] (V2): S = group max / dstTypeMax (fp32); e8m0 = the biased
 *           exponent of S, plus one when S is normal, the exponent is below 254 and the
 *           mantissa is non-zero
 *       code = E2M1(y * 2^(127 - e8m0)), round half to even, saturating at +-6
 *
 * Readings of points the page leaves open: the intermediate T is rounded to x's dtype
 * (the transforms must have x's dtype), y stays fp32, rounding is half-to-even
 * everywhere, int4 clamps to [-8, 7], the V1 exponent offset is 2 (E2M1's largest value
 * 6 = 1.5 * 2^2), 4-bit codes are packed low nibble first (INT32 words little-endian),
 * groups may span rows, a last partial group uses the elements present, the pad byte of
 * an odd group count is 0, and an all-zero slice or group gets scale 0 and codes 0.
 *
 * Calling pattern ([FQV2] 两段式接口): the first call validates, sizes the workspace
 * and returns an executor that holds every parameter; the caller allocates the
 * workspace only when its size is non-zero; the second call enqueues the work on a HIP
 * stream and takes no tensors.
 */
#ifndef FQ_H
#define FQ_H

#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ([FQV2] 容易踩的坑) ------------------------------------------
 * FQ_ERR_PARAM_NULLPTR: one of the five tensors (or its data pointer) is NULL, or an
 *   output pointer of the call is NULL.
 * FQ_ERR_PARAM_INVALID: every other failed check -- shape, dtype, clipRatio,
 *   dstTypeMax, an empty P2 outside the per-group mode, a workspace that is too small,
 *   an executor that is not live.
 * FQ_ERR_RUNTIME: the device is not gfx950, or a HIP call failed while enqueueing. */
typedef int32_t fq_status;
#define FQ_SUCCESS 0
#define FQ_ERR_PARAM_NULLPTR 161001
#define FQ_ERR_PARAM_INVALID 161002
#define FQ_ERR_RUNTIME 161003

/* ---- tensor descriptors ----------------------------------------------------------
 * [FQV2] 参数速查: all tensors are ND.
 *   x            FLOAT16 | BFLOAT16       [K, M, N], 1 <= K <= 262144, 1 <= M, N <= 256
 *   kroneckerP1  same dtype as x          [M, M]
 *   kroneckerP2  same dtype as x          [N, N], or [0, 0] (per-group mode only)
 *   out          INT32        [K, M, N/8]  (N % 8 == 0; 8 int4 codes per word)
 *                INT4         [K, M, N]    (N even; 2 codes per byte)
 *                FLOAT4_E2M1  [K, M*N]     (N even; 2 codes per byte)
 *                INT8 | FLOAT8_E4M3FN | FLOAT8_E5M2  [K, M, N]   (1 code per byte)
 *   quantScale   FLOAT32      [K]                          with INT32 / INT4 / 8-bit out
 *                FLOAT8_E8M0  [K, ceilDiv(M*N, 64), 2]     with FLOAT4_E2M1 out
 * The 8-bit outputs extend the per-token mode with the dynamic per-row quantization of
 * the dequant_swiglu_quant page (section 3.4): scale_k = fl32(max|y_k| /
 * fl32(max_val / clipRatio)) with max_val 127 (INT8), 448 (FLOAT8_E4M3FN), 57344
 * (FLOAT8_E5M2); INT8 codes clamp(RNE(y / scale), -127, 127) as two's-complement bytes;
 * FP8 codes the OCP E4M3FN / E5M2 value nearest clamp(y / scale, -max_val, max_val), a
 * tie to the even code, keeping y's sign.  They need a [N, N] P2 (as INT32 / INT4 do).
 * `data` is a device pointer; it is never dereferenced by fq_get_workspace_size.
 * `strides` are in elements of the tensor's dtype (for INT4 and FLOAT4_E2M1, in 4-bit
 * elements).  Inputs may have any non-negative strides.  Outputs may be strided too,
 * but the innermost dimension of INT4 / FLOAT4_E2M1 must have stride 1 and their other
 * strides must be even (whole bytes).  Non-contiguous tensors are staged through the
 * workspace, except an x whose innermost stride is 1 and whose other strides are multiples
 * of 8 elements (16-byte aligned data): the generic and one-wave-per-slice kernels read such
 * an x in place.  The caller owns all tensor memory; it must stay valid until the work
 * enqueued by fq_run has completed on the stream. */
typedef enum {
  FQ_DT_FLOAT16 = 1,
  FQ_DT_BFLOAT16 = 2,
  FQ_DT_FLOAT32 = 3,
  FQ_DT_INT32 = 4,
  FQ_DT_INT4 = 5,
  FQ_DT_FLOAT4_E2M1 = 6,
  FQ_DT_FLOAT8_E8M0 = 7,
  FQ_DT_INT8 = 8,           /* per-token 8-bit codes (see fq_get_workspace_size) */
  FQ_DT_FLOAT8_E4M3FN = 9,
  FQ_DT_FLOAT8_E5M2 = 10
} fq_dtype;

typedef struct {
  void* data;
  int32_t dtype;      /* fq_dtype */
  int32_t ndim;       /* 0 .. 4 */
  int64_t shape[4];
  int64_t strides[4];
} fq_tensor;

typedef struct fq_executor fq_executor; /* opaque, owned by the library */

/* ---- first stage ([FQV2] 两段式接口, 容易踩的坑) ------------------------------------
 * Validates the call, chooses the kernels and sizes the workspace.
 *   clipRatio   in (0, 1]; used by the per-token mode only ([FQV2] 标量参数).
 *   dstTypeMax  0.0 or in [6.0, 12.0]; used by the FLOAT4_E2M1 mode only; 0.0 is V1.
 * Checks run in this order: NULL pointers (FQ_ERR_PARAM_NULLPTR), then clipRatio and
 * the ranges of x's dimensions, then dtypes, shapes and dstTypeMax
 * (FQ_ERR_PARAM_INVALID).  On success *workspaceSize holds the bytes fq_run needs and
 * *executor a new executor: the staged copies of non-contiguous tensors, plus 256 bytes
 * for a slice counter when the pipelined 256 x 256 kernel (variant 4: both transforms,
 * int4 per-token codes) can run the call; 0 when every tensor is contiguous and that kernel
 * does not apply.  On failure no executor is created.  Host only: makes no HIP call and
 * may run without a GPU. */
fq_status fq_get_workspace_size(const fq_tensor* x, const fq_tensor* kroneckerP1,
                                const fq_tensor* kroneckerP2, double clipRatio, double dstTypeMax,
                                const fq_tensor* out, const fq_tensor* quantScale,
                                uint64_t* workspaceSize, fq_executor** executor);

/* The first stage in the V1 form ([FQV2] V1 还是 V2): the same call without dstTypeMax.
 * The page states that V2 with dstTypeMax = 0.0 behaves exactly as V1, so this plans the
 * V2 call with dstTypeMax = 0.0 -- same checks, same statuses, same executor, run with
 * fq_run. */
fq_status fq_v1_get_workspace_size(const fq_tensor* x, const fq_tensor* kroneckerP1,
                                   const fq_tensor* kroneckerP2, double clipRatio, const fq_tensor* out,
                                   const fq_tensor* quantScale, uint64_t* workspaceSize, fq_executor** executor);

/* ---- second stage ------------------------------------------------------------------
 * Enqueues the fused computation on `stream` (0 = the null stream) and returns without
 * synchronizing.  `workspace` is device memory of at least workspaceSize bytes (may be
 * NULL when the planned size is 0); its contents need not be initialised (fq_run sets
 * what it reads, on the stream), and work enqueued with one workspace must not overlap in
 * time with other work using the same bytes.  By default the executor is single-use: fq_run
 * releases it, whether it succeeds or fails.  A repeatable executor
 * (fq_executor_set_repeatable) survives and must be released with fq_executor_destroy.
 * Results are deterministic: the same inputs give the same bits on every run.
 * Errors: NULL executor -> FQ_ERR_PARAM_NULLPTR; workspace NULL while needed ->
 * FQ_ERR_PARAM_NULLPTR; workspace too small or executor not live ->
 * FQ_ERR_PARAM_INVALID; not a gfx950 device, or a launch failure -> FQ_ERR_RUNTIME.
 * Calls with distinct executors may come from different host threads. */
fq_status fq_run(void* workspace, uint64_t workspaceSize, fq_executor* executor, hipStream_t stream);

/* ---- second stage without a workspace allocation ------------------------------------------
 * For callers that cannot allocate device memory (code under HIP graph capture, serving loops
 * that forbid hipMalloc, harnesses that forbid it): fq_run with the staging buffer of
 * non-contiguous tensors taken from a device array inside the library instead of a
 * caller-allocated workspace.  The array holds FQ_NO_ALLOC_SCRATCH_BYTES (64 MiB) on every
 * device the library runs on, until the process ends.  No hipMalloc, hipFree or other
 * allocating call is made.  Behaviour otherwise as fq_run (single-use executors are released
 * whatever the outcome).  Errors: NULL executor -> FQ_ERR_PARAM_NULLPTR; executor not live,
 * or a planned workspace above FQ_NO_ALLOC_SCRATCH_BYTES -> FQ_ERR_PARAM_INVALID (checked
 * before any HIP call; fq_last_error() names the sizes); not a gfx950 device or a launch
 * failure -> FQ_ERR_RUNTIME.  Every call on one device shares that device's array: calls that
 * overlap in time on one device (different streams, or different host threads) race on it and
 * must be ordered by the caller.  The array is overwritten before it is read on every call. */
#define FQ_NO_ALLOC_SCRATCH_BYTES (64ull << 20)
fq_status fq_run_no_alloc(fq_executor* executor, hipStream_t stream);

/* ---- dequantization ------------------------------------------------------------------
 * The values of the codes fq_run writes, in a 16-bit float dtype: the second half of a
 * quantize -> dequantize ("fake-quant") round trip, e.g. to measure the RMS error
 * (the APT-LLM page, section 5.2, checks |dequantize(quantize(x)) - x| this way; the
 * ModelOpt page, section 6.4, uses such a round trip as a reference).
 *   per token (codes INT32 [K, M, N/8] or INT4 [K, M, N], scale FLOAT32 [K]):
 *       value = q * scale[k], q the two's-complement int4 code (the APT-LLM page, section
 *       2.1: the symmetric integer format dequantizes as q * scale)
 *   per group (codes FLOAT4_E2M1 [K, M*N], scale FLOAT8_E8M0 [K, ceilDiv(M*N, 64), 2]):
 *       value = E2M1(code) * 2^(e8m0 - 127), E2M1 magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 with
 *       the sign bit on top (the ModelOpt page, section 6.1; [FQV2] 第3步 pergroup)
 *   per token, 8-bit (codes INT8 | FLOAT8_E4M3FN | FLOAT8_E5M2 [K, M, N], scale FLOAT32 [K]):
 *       value = q * scale[k], q the INT8 integer or the FP8 value of the code (the codes of
 *       the dynamic per-row quantization of the dequant_swiglu_quant page, section 3.4);
 *       INT8 -128 and the FP8 NaN / infinity encodings, which fq_run never writes, are
 *       outside the domain
 * The product is formed in IEEE fp32 (per group it is exact, or overflows to infinity; an
 * e8m0 byte 0xFF, NaN in the MX encoding, makes its group NaN) and rounded once, to
 * nearest even, to out's dtype.
 *   out   FLOAT16 | BFLOAT16 [K, M, N]; K, M, N in the ranges of x above; 4-byte aligned.
 * All three tensors must be contiguous device memory owned by the caller (valid until the
 * work completes on the stream).  The work is enqueued on `stream` without synchronizing;
 * no workspace.  Errors: a NULL tensor or data pointer -> FQ_ERR_PARAM_NULLPTR; any shape,
 * dtype, stride or alignment mismatch -> FQ_ERR_PARAM_INVALID (these checks make no HIP
 * call); not a gfx950 device, or a launch failure -> FQ_ERR_RUNTIME. */
fq_status fq_dequant(const fq_tensor* codes, const fq_tensor* scale, const fq_tensor* out, hipStream_t stream);

/* ---- int4 consumer GEMM ------------------------------------------------------------
 * The product that follows the per-token int4 quantizer in a FlatQuant linear layer:
 *     C[t, o] = fl32( fl32(acc[t, o]) * fl32(a_scale[t] * w_scale[o]) ),
 *     acc[t, o] = sum_h qa[t, h] * qw[o, h]   (exact: int32 accumulation, |acc| <= 64 H)
 * with qa the int4 codes fq_run writes per token ([FQV2] 第3步 pertoken; its INT32 and INT4
 * outputs are the same bytes, so out viewed as INT4 [K, M*N] is a with T = K, H = M*N) and its
 * FLOAT32 [K] quantScale as a_scale; W int4 weights with one fp32 scale per output channel.
 * The symmetric integer format dequantizes as q * scale (the APT-LLM page, section 2.1).
 *   a        INT4    [T, H]     two's complement, 2 codes per byte, low nibble first; H % 128 == 0
 *   a_scale  FLOAT32 [T]
 *   w        INT4    [O, H]
 *   w_scale  FLOAT32 [O]
 *   c        BFLOAT16 | FLOAT32 [T, O]   (a bf16 C is the fp32 value rounded to nearest even)
 * All tensors contiguous device memory owned by the caller; a and w 16-byte aligned, the
 * scales 4-byte aligned; (T + 256) * H / 2 and (O + 256) * H / 2 below 2^31.  Enqueued on
 * `stream` without synchronizing; no workspace.  Errors: a NULL tensor or data pointer ->
 * FQ_ERR_PARAM_NULLPTR; any shape, dtype, stride, size or alignment mismatch ->
 * FQ_ERR_PARAM_INVALID (no HIP call is made before these checks); not a gfx950 device, or a
 * launch failure -> FQ_ERR_RUNTIME. */
fq_status fq_int4_gemm(const fq_tensor* a, const fq_tensor* a_scale, const fq_tensor* w, const fq_tensor* w_scale,
                       const fq_tensor* c, hipStream_t stream);

/* ---- int8 consumer GEMM ------------------------------------------------------------
 * The same product of the per-token int8 codes (out INT8 [K, M, N] viewed as [K, M*N]: T = K, H = M*N) with their
 * FLOAT32 [K] quantScale:
 *     C[t, o] = fl32( fl32(acc[t, o]) * fl32(a_scale[t] * w_scale[o]) ),   acc[t, o] = sum_h qa[t, h] * qw[o, h]
 * (exact: int32 accumulation, |acc| <= 2^14 H).
 *   a        INT8    [T, H]     16 <= H < 2^17, H % 16 == 0
 *   a_scale  FLOAT32 [T]
 *   w        INT8    [O, H]
 *   w_scale  FLOAT32 [O]
 *   c        FLOAT32 | FLOAT16 | BFLOAT16 [T, O]   (a 16-bit C is the fp32 value rounded to nearest even)
 * All tensors contiguous device memory owned by the caller; a and w 16-byte aligned, the scales 4-byte; T and O below
 * 2^26 (either may be 0: nothing to do, and empty tensors may have NULL data), ceilDiv(T, 128) * ceilDiv(O, 128) < 2^23.
 * Enqueued on `stream` without synchronizing; no workspace; the same inputs give the same bits.  Errors as for fq_int4_gemm. */
fq_status fq_int8_gemm(const fq_tensor* a, const fq_tensor* a_scale, const fq_tensor* w, const fq_tensor* w_scale,
                       const fq_tensor* c, hipStream_t stream);

/* ---- MXFP4 consumer GEMM ----------------------------------------------------------------
 * The product that follows the quantizer in a FlatQuant linear layer:
 *     C[t, o] = sum_h value(a[t, h]) * value(w[o, h])
 * with both operands in the per-group format fq_run writes ([FQV2] 第3步 pergroup / 第4步:
 * E2M1 codes, one e8m0 power of two per 32 consecutive elements of a row; the E2M1 values
 * from the ModelOpt page, section 6.1), so the quantizer's out / quantScale of a FLOAT4_E2M1
 * call feed it directly as a / a_scale (T = K, H = M*N).
 *   a        FLOAT4_E2M1  [T, H]                     H a multiple of 128
 *   a_scale  FLOAT8_E8M0  [T, ceilDiv(H, 64), 2]
 *   w        FLOAT4_E2M1  [O, H]
 *   w_scale  FLOAT8_E8M0  [O, ceilDiv(H, 64), 2]
 *   c        BFLOAT16 | FLOAT32 [T, O]
 * The products are accumulated in fp32 (the order is unspecified: the result lies within
 * gamma(H) * sum|terms| of the exact sum, gamma(n) = n u / (1 - n u), u = 2^-24) and rounded
 * once to c's dtype (round to nearest even).  Scales whose products leave the fp32 normal
 * range, and the e8m0 byte 0xFF (NaN), are outside the supported domain; the quantizer
 * writes neither.  All tensors contiguous device memory owned by the caller; a and w 16-byte
 * aligned; (T + 256) * H / 2 and (O + 256) * H / 2 below 2^31.  Enqueued on `stream` without
 * synchronizing; no workspace.  Errors: a NULL tensor or data pointer -> FQ_ERR_PARAM_NULLPTR;
 * any shape, dtype, stride, size or alignment mismatch -> FQ_ERR_PARAM_INVALID (no HIP call
 * is made before these checks); not a gfx950 device, or a launch failure -> FQ_ERR_RUNTIME. */
fq_status fq_mx_gemm(const fq_tensor* a, const fq_tensor* a_scale, const fq_tensor* w, const fq_tensor* w_scale,
                     const fq_tensor* c, hipStream_t stream);

/* ---- paged key-value cache -------------------------------------------------------------
 * The keys and values of an attention layer, kept in the formats the quantizer writes.  A cache
 * is two sides (keys, values) of the same shape; each is a codes tensor and, for the low-bit
 * formats, a scale tensor, over pages of P tokens:
 *   codes  FLOAT16 | BFLOAT16                    [pages, Hkv, P, D]
 *          INT8 | FLOAT8_E4M3FN                  [pages, Hkv, P, D]   scale FLOAT32 [pages, Hkv, P]
 *          INT4          (2 codes per byte)      [pages, Hkv, P, D]   scale FLOAT32 [pages, Hkv, P]
 *          FLOAT4_E2M1   (2 codes per byte)      [pages, Hkv, P, D]   scale FLOAT8_E8M0
 *                                                             [pages, Hkv, P, 2 * ceilDiv(D, 64)]
 *   P a power of two, 16 <= P <= 1024; 8 <= D <= 256, D % 8 == 0 (% 32 for FLOAT4_E2M1);
 *   1 <= Hkv <= 1024; pages * P < 2^31.  The scale pointers are NULL for the 16-bit formats.
 * A row -- one token's D elements of one head -- is quantized as the quantizer's per-token and
 * per-group rules quantize a slice: scale = fl32(max|x| / fl32(max_val / clipRatio)) (max_val
 * 127, 448, 7) and code = clamp(round_half_even(fl32(x / scale))); or one e8m0 byte per 32
 * elements by dstTypeMax's rule and E2M1 codes (bytes past D/32 in the scale row are 0).  An
 * all-zero row (group) gets scale 0 and codes 0.  A row (group) that holds an infinity or NaN
 * reads back as NaN throughout: its scale is stored non-finite (e8m0 0xFF).
 * Every dimension but the first must be contiguous; the first may have any stride that is a
 * multiple of 16 bytes, so one allocation can interleave the two sides.  Codes and scales
 * 16-byte aligned.  Token t of a sequence lies in page block_table[sequence, t / P] at offset
 * t % P.  All tensors are device memory owned by the
 * caller, valid until the work completes on the stream; all calls enqueue on `stream` without
 * synchronizing, allocate nothing, may be captured in a graph, and read slots, block tables and
 * lengths on the device, where every index is checked: one outside the cache is never followed.
 *
 * 16-bit row tensors (k, v, q, outputs) are FLOAT16 | BFLOAT16 [rows, heads, D] with innermost
 * stride 1, the other strides multiples of 8 elements (below 2^40) and data 16-byte aligned; an
 * empty one (a dimension of 0) may have NULL data, and a call with no rows does nothing.  Strides
 * of inputs may be 0; the elements of an output lie apart from each other (its smaller outer stride
 * at least D, the larger one at least what the smaller one spans).
 * Errors of all these calls: a required tensor or data pointer NULL -> FQ_ERR_PARAM_NULLPTR;
 * any dtype, shape, stride, alignment or scalar outside the above -> FQ_ERR_PARAM_INVALID (no
 * HIP call is made before these checks); not a gfx950 device, or a launch failure ->
 * FQ_ERR_RUNTIME.
 *
 * A call writes or reads at most (2^24 - 1) * 32 tokens with D up to 64, * 16 up to 128, * 8 up to 256.
 *
 * fq_kv_write: rows k[i], v[i] ([T, Hkv, D]) go to slot slots[i] = page * P + offset (INT32
 * [T]).  A negative slot, or one beyond the cache, writes nothing (padding).  No slot may occur
 * twice in a call.  clipRatio in (0, 1] acts on the per-token formats, dstTypeMax (0, or 6 to
 * 12) on FLOAT4_E2M1; a 16-bit cache must have k's dtype and stores the rows unchanged. */
fq_status fq_kv_write(const fq_tensor* k, const fq_tensor* v, const fq_tensor* slots, double clipRatio,
                      double dstTypeMax, const fq_tensor* k_cache, const fq_tensor* k_scale,
                      const fq_tensor* v_cache, const fq_tensor* v_scale, hipStream_t stream);

/* fq_kv_read: the first cu[b+1] - cu[b] tokens of every sequence b, as values, packed: token t
 * of sequence b goes to row cu[b] + t of k_out and v_out ([T, Hkv, D]).  block_table INT32
 * [B, pages per sequence] (innermost stride 1), cu INT32 [B+1] ascending from 0.  The value is
 * code * scale in fp32 rounded once to the output's dtype (a 16-bit cache must have the
 * output's dtype).  Rows from cu[B] on are not written; a token whose table entry is missing or
 * outside the cache gives zeros. */
fq_status fq_kv_read(const fq_tensor* k_cache, const fq_tensor* k_scale, const fq_tensor* v_cache,
                     const fq_tensor* v_scale, const fq_tensor* block_table, const fq_tensor* cu,
                     const fq_tensor* k_out, const fq_tensor* v_out, hipStream_t stream);

/* ---- norms and rotation of queries and keys -------------------------------------------------
 * What stands between the projection and the attention.  A row (one token's D elements of one head) is
 * first, where the side has a weight [D], divided by its root mean square,
 *     y = x / sqrt(mean(x^2) + eps) * w
 * (eps from 2^-126 to 2^127; a NULL weight: no norm), and then the pairs (a, b) of its first R elements
 * are turned by the token's position,
 *     (a, b) -> (a cos t - b sin t, b cos t + a sin t),   t = position * inv_freq[i],
 * pair i of R / 2 being elements (i, i + R / 2), or (2 i, 2 i + 1) with interleaved != 0.
 *   inv_freq   FLOAT32 [R / 2]: R a multiple of 8, at most D; empty: no rotation
 *   positions  INT32 [T] (contiguous); with axes [A, T], 1 <= A <= 16, innermost stride 1
 *   axes       NULL, or INT32 [R / 2]: the row of positions that turns each pair (time, height and width of
 *              a video, say); a pair whose axis is not in 0 .. A-1 is not turned
 *   weights    FLOAT32 | FLOAT16 | BFLOAT16 [D], contiguous
 * All of it is fp32, the angle's product with the position fp64 before its whole turns are taken off, and rounded
 * once at the end.  Squares have to sum within fp32's range (|x| up to 1e18).
 *
 * fq_qk_rope: q, k (either may be NULL with its output) to q_out, k_out, 16-bit rows as above, of one dtype, each with heads
 * of its own, 0 to 65536.  An output may be its own input (the same tensor, that is); it must not overlap otherwise.
 *
 * fq_kv_append: the same on q (may be NULL with q_out) and k, and k and v written to the cache as by fq_kv_write, in
 * one launch.  The keys' codes come from the unrounded rows; the values' are fq_kv_write's.  A token whose slot is negative
 * or beyond the cache still has its q turned. */
fq_status fq_qk_rope(const fq_tensor* q, const fq_tensor* k, const fq_tensor* q_weight, const fq_tensor* k_weight, double eps,
                     const fq_tensor* positions, const fq_tensor* inv_freq, const fq_tensor* axes, int32_t interleaved,
                     const fq_tensor* q_out, const fq_tensor* k_out, hipStream_t stream);
fq_status fq_kv_append(const fq_tensor* q, const fq_tensor* k, const fq_tensor* v, const fq_tensor* slots,
                       const fq_tensor* q_weight, const fq_tensor* k_weight, double eps, const fq_tensor* positions,
                       const fq_tensor* inv_freq, const fq_tensor* axes, int32_t interleaved, double clipRatio,
                       double dstTypeMax, const fq_tensor* k_cache, const fq_tensor* k_scale, const fq_tensor* v_cache,
                       const fq_tensor* v_scale, const fq_tensor* q_out, hipStream_t stream);

/* ---- attention of one new token over the cache --------------------------------------------
 *     out[b, h] = sum_t p[t] v[t, h / g],  p = softmax over t < lengths[b] of scale * <q[b, h], k[t, h / g]>
 * with g = Hq / Hkv (a whole number) query heads sharing a cache head.  q, out FLOAT16 |
 * BFLOAT16 [B, Hq, D] of one dtype (a 16-bit cache must have it too), lengths INT32 [B] (the
 * newest token included; capped at the table's reach), block_table as above, 1 <= Hq <= 65536;
 * reach = the table's width * P < 2^31 - 65536, B * Hkv * ceilDiv(g, 16) < 2^24 and that times
 * (ceilDiv(reach, 128) + 3) < 2^31.
 * `lse`, when not NULL, is FLOAT32 [B, Hq] (contiguous) and receives log sum_t exp(scale *
 * <q, k[t]>).  A length of 0 (an idle place of a fixed batch) gives zeros and lse = -infinity.
 * A token whose table entry is outside the cache is left out of the sum; cache contents past a
 * sequence's length are never used, whatever they hold.  |scale| <= 2^127; 0 means 1/sqrt(D).
 * Scores, softmax statistics and sums are fp32.  The products are the matrix cores', of 16-bit
 * operands.  Codes enter them exactly, but for E2M1 groups more than 2^26 below the largest among the
 * 32 tokens beside them (keys) or 2^25 below the largest of the sequence (values), which lose bits.
 * Weights enter with 22 bits (bf16 caches 16) where g <= 8.  With more heads a cache head they are
 * rounded once: 11 bits (bf16 caches 8), to 2^-32 of the sequence's largest weight at the least (2^-30
 * in the formats with a scale a token, where it is the weight times the token's value scale that is
 * rounded).  Results do not depend on the run: the same inputs give the same bits.
 * An infinite value that is seen with a weight above 0, however small, makes its element infinite (in
 * a 16-bit cache; the other formats hold none).
 * The cache is read once for every 16 query heads of a cache head, split over its length across the
 * device and joined; the partial sums
 * live in `workspace` (device memory, 16-byte aligned, of at least the size that
 * fq_attn_decode_get_workspace_size gives for the same q, cache and table; contents need not be
 * initialised; calls that overlap in time must not share it). */
fq_status fq_attn_decode_get_workspace_size(const fq_tensor* q, const fq_tensor* k_cache, const fq_tensor* block_table,
                                            uint64_t* workspaceSize);
fq_status fq_attn_decode(const fq_tensor* q, const fq_tensor* k_cache, const fq_tensor* k_scale,
                         const fq_tensor* v_cache, const fq_tensor* v_scale, const fq_tensor* block_table,
                         const fq_tensor* lengths, double scale, const fq_tensor* out, const fq_tensor* lse,
                         void* workspace, uint64_t workspaceSize, hipStream_t stream);

/* ---- attention over packed prompts -----------------------------------------------------------
 * Sequences of different lengths packed row after row: sequence b has the query rows cu_q[b] ..
 * cu_q[b+1]-1 of q, out [Tq, Hq, D] and the key rows cu_k[b] .. cu_k[b+1]-1 of k, v [Tk, Hkv, D]
 * (all of one dtype; cu_q, cu_k INT32 [B+1], ascending from 0).  With causal != 0 query row i
 * of a sequence sees its keys 0 .. (Lk - Lq) + i: the queries are the sequence's last rows, so
 * a prompt's chunk attends to the part before it (read back with fq_kv_read) and to itself.
 * With causal == 0 it sees all Lk.  A row that sees no key gives zeros and lse = -infinity.
 * Infinities and NaN in keys and values reach only the rows that see them, an infinite value with a
 * weight above 0 as an infinity.  Scores, statistics and sums are fp32; the weights are rounded to q's
 * dtype for the second product (11 bits and 2^-32 of the row's largest at the least, in bf16 8 bits).
 * The row strides of k and v are at most 2^23 elements.
 * `lse` (optional) FLOAT32 [Tq, Hq].  g = Hq / Hkv and scale as above; 1 <= B <= 65536 and
 * (floor(Tq / 128) + B) * Hq < 2^24.  Rows of out past cu_q[B] are not written.  A call with few rows over many keys splits the keys and joins
 * the parts in `workspace` (as for fq_attn_decode, of the size that
 * fq_attn_prefill_get_workspace_size gives for the same tensors; 0 for most calls). */
fq_status fq_attn_prefill_get_workspace_size(const fq_tensor* q, const fq_tensor* k, const fq_tensor* cu_q, int32_t causal,
                                             uint64_t* workspaceSize);
fq_status fq_attn_prefill(const fq_tensor* q, const fq_tensor* k, const fq_tensor* v, const fq_tensor* cu_q,
                          const fq_tensor* cu_k, int32_t causal, double scale, const fq_tensor* out,
                          const fq_tensor* lse, void* workspace, uint64_t workspaceSize, hipStream_t stream);

/* ---- attention of new tokens over the cache ---------------------------------------------------
 * Sequences of a running batch with one or more new tokens each, whose keys and values the cache holds already: sequence b has
 * the query rows cu_q[b] .. cu_q[b+1]-1 of q, out [Tq, Hq, D] (INT32 [B+1], ascending from 0) and lengths[b] cached tokens
 * (INT32 [B], the new ones included; capped at the table's reach).  Its last query row stands at its last token, and row i at
 * position p = lengths[b] - (cu_q[b+1] - cu_q[b]) + i sees the keys j <= p; with window > 0 of those only the ones with
 * j > p - window and the first ones, j < sinks, which stay visible.  window 0: all of them (sinks is not used then).  So chunks of prompts,
 * drafted tokens that are checked and single tokens can share one call; the work is cut by the mean rows of a sequence, so
 * that long chunks and single tokens take less time in calls of their own, and each workgroup looks at all B sequences: more
 * than about 1000 are better dealt to several calls.
 * q, out, the cache, block_table, scale (within 2^118 where f16 rows meet an int8 or int4 cache), lse FLOAT32 [Tq, Hq] and the
 * workspace as for fq_attn_decode (of the size that
 * fq_attn_chunk_get_workspace_size gives for the same q, cache, table, cu_q, window and sinks; its contents need not be
 * initialised; calls that overlap in time must not share it); 1 <= B <= 65536, Hq <= 65536; reach and Tq below 2^31 - 65536,
 * and (floor(Tq / t) + min(B, Tq)) * Hkv * n * (ceilDiv(seen, 64) + 5) < 2^31, with row tiles of r rows (the first of 32, 64
 * and 128 that ceilDiv(Tq, B) * g rows fit, else 128), n = ceilDiv(g, r) of them for a token's heads, t = floor(r / ceilDiv(g,
 * n)) tokens of one, and `seen` the keys that such a tile can see (reach + t, or window + t + 126 and the sinks).
 * A row that sees nothing (more rows than cached tokens, no page) gives zeros and lse = -infinity.  A token whose table entry
 * is outside the cache is left out.  What a row does not see never reaches it, infinities and NaN included; rows of out past
 * cu_q[B] are not written.  The same inputs give the same bits.
 * Scores, statistics and sums are fp32, codes enter the products exactly (E2M1 groups more than 2^26 below the largest of
 * their row lose bits, and a bf16 query's elements more than 2^28 below the largest of its row).  The weights are rounded for
 * the second product: to 11 bits and 2^-32 of the row's largest at the least over an f16 cache, 8 bits over a bf16 one; over
 * the low-bit formats a weight, off by up to 2^-17 of itself where value scales are far from 1, times its value's scale to 11
 * bits, and to 2^-30 of the largest of these.  Twice as many bits (as fq_attn_decode's) where r is 32, so for single tokens and
 * few drafts, and, over 16-bit caches or with f16 rows, where r is 64.  Value scales below 2^-80 lose bits (E2M1: values below
 * 2^-80), and below 2^-16 where some of 128 neighbouring rows of a cache head see ones above 2^96. */
fq_status fq_attn_chunk_get_workspace_size(const fq_tensor* q, const fq_tensor* k_cache, const fq_tensor* block_table, const fq_tensor* cu_q,
                                           int32_t window, int32_t sinks, uint64_t* workspaceSize);
fq_status fq_attn_chunk(const fq_tensor* q, const fq_tensor* k_cache, const fq_tensor* k_scale, const fq_tensor* v_cache,
                        const fq_tensor* v_scale, const fq_tensor* block_table, const fq_tensor* cu_q, const fq_tensor* lengths,
                        int32_t window, int32_t sinks, double scale, const fq_tensor* out, const fq_tensor* lse, void* workspace,
                        uint64_t workspaceSize, hipStream_t stream);

/* Releases an executor that will not be run (or a repeatable one).  NULL is a no-op. */
void fq_executor_destroy(fq_executor* executor);

/* Keeps the executor alive across fq_run calls (repeat != 0), e.g. to launch the same
 * problem many times.  Returns FQ_ERR_PARAM_NULLPTR / FQ_ERR_PARAM_INVALID for a NULL or
 * dead executor. */
fq_status fq_executor_set_repeatable(fq_executor* executor, int32_t repeat);

/* Kernel variant the executor will launch: 0 = the automatic choice, 1 = the generic
 * kernel (any shape), 2 = the small-slice MFMA kernel (one wave per slice; M and N up to
 * 128, run at the next of 16, 32, 64, 128 with zero padding where they are not one of
 * them: per token N a multiple of 8, per group N one of 32, 64, 128), 3 = the
 * whole-workgroup MFMA kernel for 256 x 256 slices, which also takes the slices with a side
 * above 128 (M, N up to 256; N a multiple of 8, per group of 32), zero-padded to 256 x 256
 * (an empty P2 as the identity), 4 = its pipelined form for 256 x 256
 * slices with both transforms and per-token int4 codes (INT32 / INT4 out; the automatic
 * choice there), 5 = the streaming MFMA kernel for 256 x 256 slices with an empty P2 and
 * FLOAT4_E2M1 out (x through an LDS ring filled by DMA, P1 in registers; the automatic
 * choice there).  Selecting a variant that does not support the planned problem returns
 * FQ_ERR_PARAM_INVALID and leaves the executor unchanged.  Meant for tests and
 * benchmarks. */
fq_status fq_executor_set_kernel(fq_executor* executor, int32_t variant);

/* The variant the executor will launch (1 .. 5), or a negative value for NULL. */
int32_t fq_executor_kernel(const fq_executor* executor);

/* A static, human-readable name for a status code. */
const char* fq_status_string(fq_status status);

/* Detail of the last FQ_ERR_RUNTIME returned on the calling thread: the HIP call that
 * failed and the runtime's error text, or "" when there was none.  The string is owned by
 * the library and stays valid until the thread's next call into it. */
const char* fq_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* FQ_H */
