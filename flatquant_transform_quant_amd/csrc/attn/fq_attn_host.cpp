// Host side of the key-value cache and attention calls of include/fq.h: checks and dispatch.
#include <hip/hip_runtime.h>

#include "fq_attn_checks.h"

using namespace fq;

extern "C" {

fq_status fq_kv_write(const fq_tensor* k, const fq_tensor* v, const fq_tensor* slots, double clipRatio,
                      double dstTypeMax, const fq_tensor* k_cache, const fq_tensor* k_scale, const fq_tensor* v_cache,
                      const fq_tensor* v_scale, hipStream_t stream) {
  clear_last_error();
  if (missing(k) || missing(v) || missing(slots)) return FQ_ERR_PARAM_NULLPTR;
  fq_status st = cache_null(k_cache, k_scale, v_cache, v_scale);
  if (st != FQ_SUCCESS) return st;
  if (!write_scalars_ok(clipRatio, dstTypeMax)) return FQ_ERR_PARAM_INVALID;
  KvCache c;
  st = cache_of(k_cache, k_scale, v_cache, v_scale, &c);
  if (st != FQ_SUCCESS) return st;
  if (k->ndim != 3) return FQ_ERR_PARAM_INVALID;
  const int64_t T = k->shape[0];
  Rows16 kr, vr;
  if (row_dtype(k->dtype) == 0 || !tokens_ok(T, c.D) ||
      !rows_ok(*k, T, c.Hkv, c.D, k->dtype, &kr) || !rows_ok(*v, T, c.Hkv, c.D, k->dtype, &vr) || !i32_vec(*slots, T))
    return FQ_ERR_PARAM_INVALID;
  if (c.mode == kKv16 && c.dtype != row_dtype(k->dtype)) return FQ_ERR_PARAM_INVALID;
  c.dtype = row_dtype(k->dtype);
  if (T == 0) return FQ_SUCCESS;
  if (!device_is_gfx950()) return fail_runtime("the current device is not gfx950", hipSuccess);
  const hipError_t err = launch_kv_write(c, T, kr, vr, static_cast<const int32_t*>(slots->data),
                                         write_divisor(c.mode, clipRatio), static_cast<float>(dstTypeMax), stream);
  return err == hipSuccess ? FQ_SUCCESS : fail_runtime("cache write kernel launch", err);
}

fq_status fq_kv_read(const fq_tensor* k_cache, const fq_tensor* k_scale, const fq_tensor* v_cache,
                     const fq_tensor* v_scale, const fq_tensor* block_table, const fq_tensor* cu,
                     const fq_tensor* k_out, const fq_tensor* v_out, hipStream_t stream) {
  clear_last_error();
  if (missing(block_table) || missing(cu) || missing(k_out) || missing(v_out)) return FQ_ERR_PARAM_NULLPTR;
  fq_status st = cache_null(k_cache, k_scale, v_cache, v_scale);
  if (st != FQ_SUCCESS) return st;
  KvCache c;
  st = cache_of(k_cache, k_scale, v_cache, v_scale, &c);
  if (st != FQ_SUCCESS) return st;
  if (block_table->ndim != 2 || k_out->ndim != 3) return FQ_ERR_PARAM_INVALID;
  const int64_t B = block_table->shape[0], T = k_out->shape[0];
  Rows16 kr, vr;
  BlockTable bt;
  if (B < 0 || B > 65536 || !tokens_ok(T, c.D) || row_dtype(k_out->dtype) == 0 ||
      !table_ok(*block_table, B, &bt) || !i32_vec(*cu, B + 1) || !out_rows_ok(*k_out, T, c.Hkv, c.D, k_out->dtype, &kr) ||
      !out_rows_ok(*v_out, T, c.Hkv, c.D, k_out->dtype, &vr))
    return FQ_ERR_PARAM_INVALID;
  if (c.mode == kKv16 && c.dtype != row_dtype(k_out->dtype)) return FQ_ERR_PARAM_INVALID;
  c.dtype = row_dtype(k_out->dtype);
  if (T == 0 || B == 0) return FQ_SUCCESS;
  if (!device_is_gfx950()) return fail_runtime("the current device is not gfx950", hipSuccess);
  const hipError_t err =
      launch_kv_read(c, T, static_cast<int32_t>(B), bt, static_cast<const int32_t*>(cu->data), kr, vr, stream);
  return err == hipSuccess ? FQ_SUCCESS : fail_runtime("cache read kernel launch", err);
}

// The parts of a decode call that its workspace depends on.
static bool decode_sizes(const fq_tensor* q, const fq_tensor* k_cache, const fq_tensor* block_table, int64_t* reach) {
  if (q->ndim != 3 || k_cache->ndim != 4 || block_table->ndim != 2) return false;
  const int64_t B = q->shape[0], Hq = q->shape[1], D = q->shape[2], Hkv = k_cache->shape[1], P = k_cache->shape[2];
  if (B < 0 || B > 65536 || Hq < 1 || Hq > 65536 || Hkv < 1 || Hkv > 1024 || Hq % Hkv != 0 || D < 8 || D > 256 ||
      D != k_cache->shape[3] || P < 16 || P > 1024 || block_table->shape[1] < 0 || block_table->shape[1] >= (int64_t(1) << 31))
    return false;
  *reach = block_table->shape[1] * P;
  if (*reach >= (int64_t(1) << 31) - 65536) return false;  // (a step past the last token stays within 31 bits)
  // segments (a sequence, cache head and 16 query heads: a workgroup each of the join, or of calls without
  // one), and units of work (128 tokens of a segment, and up to 3 more for its start) counted in 31 bits
  const int64_t segments = B * Hkv * ceil_div(Hq / Hkv, 16);
  return segments <= kWorkgroups && segments * (ceil_div(*reach, 128) + 3) < (int64_t(1) << 31);
}

fq_status fq_attn_decode_get_workspace_size(const fq_tensor* q, const fq_tensor* k_cache, const fq_tensor* block_table,
                                            uint64_t* workspaceSize) {
  clear_last_error();
  if (!q || !k_cache || !block_table || !workspaceSize) return FQ_ERR_PARAM_NULLPTR;
  int64_t reach;
  if (!decode_sizes(q, k_cache, block_table, &reach)) return FQ_ERR_PARAM_INVALID;
  *workspaceSize = attn_decode_workspace(static_cast<int32_t>(q->shape[0]), static_cast<int32_t>(q->shape[1]),
                                         static_cast<int32_t>(k_cache->shape[1]), static_cast<int32_t>(q->shape[2]), reach);
  return FQ_SUCCESS;
}

fq_status fq_attn_decode(const fq_tensor* q, const fq_tensor* k_cache, const fq_tensor* k_scale,
                         const fq_tensor* v_cache, const fq_tensor* v_scale, const fq_tensor* block_table,
                         const fq_tensor* lengths, double scale, const fq_tensor* out, const fq_tensor* lse,
                         void* workspace, uint64_t workspaceSize, hipStream_t stream) {
  clear_last_error();
  if (missing(q) || missing(block_table) || missing(lengths) || missing(out) || (lse && missing(lse)))
    return FQ_ERR_PARAM_NULLPTR;
  fq_status st = cache_null(k_cache, k_scale, v_cache, v_scale);
  if (st != FQ_SUCCESS) return st;
  DecodeArgs a;
  st = cache_of(k_cache, k_scale, v_cache, v_scale, &a.c);
  if (st != FQ_SUCCESS) return st;
  int64_t reach;
  if (!decode_sizes(q, k_cache, block_table, &reach) || row_dtype(q->dtype) == 0 ||
      !scale_ok(scale, q->shape[2], &a.scale))
    return FQ_ERR_PARAM_INVALID;
  const int64_t B = q->shape[0], Hq = q->shape[1], D = q->shape[2];
  if (!table_ok(*block_table, B, &a.bt) || !i32_vec(*lengths, B) || !rows_ok(*q, B, Hq, D, q->dtype, &a.q) ||
      !out_rows_ok(*out, B, Hq, D, q->dtype, &a.out) || !lse_ok(lse, B, Hq))
    return FQ_ERR_PARAM_INVALID;
  if (a.c.mode == kKv16 && a.c.dtype != row_dtype(q->dtype)) return FQ_ERR_PARAM_INVALID;
  a.c.dtype = row_dtype(q->dtype);
  a.lengths = static_cast<const int32_t*>(lengths->data);
  a.lse = lse ? static_cast<float*>(lse->data) : nullptr;
  a.B = static_cast<int32_t>(B);
  a.Hq = static_cast<int32_t>(Hq);
  a.g = static_cast<int32_t>(Hq / a.c.Hkv);
  const uint64_t need = attn_decode_workspace(a.B, a.Hq, a.c.Hkv, a.c.D, reach);
  if (need > 0 && !workspace) return FQ_ERR_PARAM_NULLPTR;
  if (workspaceSize < need || (need > 0 && !aligned(workspace, 16))) return FQ_ERR_PARAM_INVALID;
  if (B == 0) return FQ_SUCCESS;
  if (!device_is_gfx950()) return fail_runtime("the current device is not gfx950", hipSuccess);
  const hipError_t err = launch_attn_decode(a, workspace, stream);
  return err == hipSuccess ? FQ_SUCCESS : fail_runtime("decode attention kernel launch", err);
}

// The parts of a prompt call that its workspace depends on.
static bool prefill_sizes(const fq_tensor* q, const fq_tensor* k, const fq_tensor* cu_q) {
  if (q->ndim != 3 || k->ndim != 3 || cu_q->ndim != 1) return false;
  const int64_t Tq = q->shape[0], Hq = q->shape[1], D = q->shape[2], Tk = k->shape[0], Hkv = k->shape[1];
  const int64_t B = cu_q->shape[0] - 1, lim = (int64_t(1) << 31) - 65536;
  return B >= 1 && B <= 65536 && Tq >= 0 && Tk >= 0 && Tq < lim && Tk < lim && Hq >= 1 && Hq <= 65536 && Hkv >= 1 &&
         Hkv <= 1024 && Hq % Hkv == 0 && D >= 8 && D <= 256 && D % 8 == 0 &&
         (Tq / 128 + B) * Hq <= kWorkgroups;  // (a row tile and head each; only few are cut into parts)
}

fq_status fq_attn_prefill_get_workspace_size(const fq_tensor* q, const fq_tensor* k, const fq_tensor* cu_q, int32_t /*causal*/,
                                             uint64_t* workspaceSize) {
  clear_last_error();
  if (!q || !k || !cu_q || !workspaceSize) return FQ_ERR_PARAM_NULLPTR;
  if (!prefill_sizes(q, k, cu_q)) return FQ_ERR_PARAM_INVALID;
  *workspaceSize = attn_prefill_workspace(q->shape[0], k->shape[0], cu_q->shape[0] - 1, q->shape[1], q->shape[2]);
  return FQ_SUCCESS;
}

fq_status fq_attn_prefill(const fq_tensor* q, const fq_tensor* k, const fq_tensor* v, const fq_tensor* cu_q,
                          const fq_tensor* cu_k, int32_t causal, double scale, const fq_tensor* out,
                          const fq_tensor* lse, void* workspace, uint64_t workspaceSize, hipStream_t stream) {
  clear_last_error();
  for (const fq_tensor* t : {q, k, v, cu_q, cu_k, out})
    if (missing(t)) return FQ_ERR_PARAM_NULLPTR;
  if (lse && missing(lse)) return FQ_ERR_PARAM_NULLPTR;
  PrefillArgs a;
  if (!prefill_sizes(q, k, cu_q) || row_dtype(q->dtype) == 0 || !scale_ok(scale, q->shape[2], &a.scale)) return FQ_ERR_PARAM_INVALID;
  const int64_t Tq = q->shape[0], Hq = q->shape[1], D = q->shape[2], Tk = k->shape[0], Hkv = k->shape[1];
  const int64_t B = cu_q->shape[0] - 1;
  if (!rows_ok(*q, Tq, Hq, D, q->dtype, &a.q) || !out_rows_ok(*out, Tq, Hq, D, q->dtype, &a.out) ||
      !rows_ok(*k, Tk, Hkv, D, q->dtype, &a.k) || !rows_ok(*v, Tk, Hkv, D, q->dtype, &a.v) || !i32_vec(*cu_q, B + 1) ||
      !i32_vec(*cu_k, B + 1) || !lse_ok(lse, Tq, Hq))
    return FQ_ERR_PARAM_INVALID;
  // a tile of 64 key rows within 31-bit offsets
  if (Tk > 1 && (k->strides[0] > (int64_t(1) << 23) || v->strides[0] > (int64_t(1) << 23))) return FQ_ERR_PARAM_INVALID;
  const uint64_t need = attn_prefill_workspace(Tq, Tk, B, Hq, D);
  if (need > 0 && !workspace) return FQ_ERR_PARAM_NULLPTR;
  if (workspaceSize < need || (need > 0 && !aligned(workspace, 16))) return FQ_ERR_PARAM_INVALID;
  if (Tq == 0) return FQ_SUCCESS;
  if (!device_is_gfx950()) return fail_runtime("the current device is not gfx950", hipSuccess);
  a.lse = lse ? static_cast<float*>(lse->data) : nullptr;
  a.cu_q = static_cast<const int32_t*>(cu_q->data);
  a.cu_k = static_cast<const int32_t*>(cu_k->data);
  a.B = static_cast<int32_t>(B);
  a.Tq = static_cast<int32_t>(Tq);
  a.Tk = static_cast<int32_t>(Tk);
  a.Hq = static_cast<int32_t>(Hq);
  a.g = static_cast<int32_t>(Hq / Hkv);
  a.D = static_cast<int32_t>(D);
  a.dtype = row_dtype(q->dtype);
  a.causal = causal ? 1 : 0;
  const hipError_t err = launch_attn_prefill(a, workspace, stream);
  return err == hipSuccess ? FQ_SUCCESS : fail_runtime("prompt attention kernel launch", err);
}

}  // extern "C"
