// Host side of the key-value cache and attention calls of include/fq.h: checks and dispatch.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>

#include "fq.h"
#include "fq_attn.h"
#include "fq_host_util.h"

using namespace fq;

namespace {

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

bool empty(const fq_tensor& t) {
  if (t.ndim < 0 || t.ndim > 4) return false;
  for (int d = 0; d < t.ndim; ++d)
    if (t.shape[d] == 0) return true;
  return false;
}

// NULL tensors, or NULL data of a tensor that is not empty
bool missing(const fq_tensor* t) { return !t || (!t->data && !empty(*t)); }

// 16-bit rows [n, heads, D]
bool rows_ok(const fq_tensor& t, int64_t n, int64_t heads, int64_t D, int32_t dtype, Rows16* r) {
  if (!strides_ok(t) || t.dtype != dtype || !shape_is(t, 3, n, heads, D)) return false;
  r->p = static_cast<uint16_t*>(t.data);
  r->row = t.strides[0];
  r->head = t.strides[1];
  if (empty(t)) return true;
  const int64_t lim = int64_t(1) << 40;
  return (t.strides[2] == 1 || D == 1) && (n == 1 || t.strides[0] % 8 == 0) && (heads == 1 || t.strides[1] % 8 == 0) &&
         t.strides[0] < lim && t.strides[1] < lim && aligned(t.data, 16);
}

// The same of rows that are written: no two elements at one place, so that nothing depends on the order of the writes.
bool out_rows_ok(const fq_tensor& t, int64_t n, int64_t heads, int64_t D, int32_t dtype, Rows16* r) {
  if (!rows_ok(t, n, heads, D, dtype, r)) return false;
  if (empty(t) || (n == 1 && heads == 1)) return true;
  if (n == 1) return r->head >= D;
  if (heads == 1) return r->row >= D;
  // (below 2^57: strides below 2^40, at most 2^17 heads; for the rows compare by division)
  return r->row >= r->head ? r->head >= D && r->row >= (heads - 1) * r->head + D
                           : r->row >= D && (r->head - D) / r->row >= n - 1;
}

bool i32_vec(const fq_tensor& t, int64_t n) {
  return strides_ok(t) && t.dtype == FQ_DT_INT32 && shape_is(t, 1, n) && is_contiguous(t) && aligned(t.data, 4);
}

// all dimensions but the first contiguous
bool inner_contiguous(const fq_tensor& t) {
  int64_t expect = 1;
  for (int d = t.ndim - 1; d >= 1; --d) {
    if (t.shape[d] != 1 && t.strides[d] != expect) return false;
    expect *= t.shape[d];
  }
  return t.shape[0] == 1 || t.strides[0] >= expect;
}

// One side of the cache; `first` is the side that fixed c's sizes (null for that side itself).
fq_status side_of(const fq_tensor* codes, const fq_tensor* scale, bool first, KvCache* c, KvSide* sd) {
  if (!strides_ok(*codes) || codes->ndim != 4) return FQ_ERR_PARAM_INVALID;
  const int64_t pages = codes->shape[0], H = codes->shape[1], P = codes->shape[2], D = codes->shape[3];
  int32_t mode, dtype = 0, bits;
  switch (codes->dtype) {
    case FQ_DT_FLOAT16: mode = kKv16; dtype = kF16; bits = 16; break;
    case FQ_DT_BFLOAT16: mode = kKv16; dtype = kBF16; bits = 16; break;
    case FQ_DT_INT8: mode = kKvInt8; bits = 8; break;
    case FQ_DT_FLOAT8_E4M3FN: mode = kKvE4M3; bits = 8; break;
    case FQ_DT_INT4: mode = kKvInt4; bits = 4; break;
    case FQ_DT_FLOAT4_E2M1: mode = kKvFp4; bits = 4; break;
    default: return FQ_ERR_PARAM_INVALID;
  }
  if (pages < 1 || H < 1 || H > 1024 || P < 16 || P > 1024 || (P & (P - 1)) != 0 || D < 8 || D > 256 ||
      D % (mode == kKvFp4 ? 32 : 8) != 0 || pages >= (int64_t(1) << 31) / P)
    return FQ_ERR_PARAM_INVALID;
  int32_t log = 0;
  while ((int64_t(1) << log) < P) ++log;
  if (first) {
    c->mode = mode;
    c->dtype = dtype;
    c->Hkv = static_cast<int32_t>(H);
    c->D = static_cast<int32_t>(D);
    c->pages = static_cast<int32_t>(pages);
    c->page_log = log;
  } else if (c->mode != mode || c->dtype != dtype || c->Hkv != H || c->D != D || c->pages != pages || c->page_log != log) {
    return FQ_ERR_PARAM_INVALID;
  }
  const int64_t lim = int64_t(1) << 40;
  const int64_t stride0 = pages == 1 ? 0 : codes->strides[0];
  if (!inner_contiguous(*codes) || !aligned(codes->data, 16) || stride0 * bits % 128 != 0 || stride0 >= lim)
    return FQ_ERR_PARAM_INVALID;
  sd->codes = static_cast<uint8_t*>(codes->data);
  sd->page_b = stride0 * bits / 8;
  sd->scale = nullptr;
  sd->scale_page_b = 0;
  if (mode == kKv16) return FQ_SUCCESS;
  if (!strides_ok(*scale) || !aligned(scale->data, 16)) return FQ_ERR_PARAM_INVALID;
  int64_t eb;
  if (mode == kKvFp4) {
    if (scale->dtype != FQ_DT_FLOAT8_E8M0 || scale->ndim != 4 || scale->shape[0] != pages || scale->shape[1] != H ||
        scale->shape[2] != P || scale->shape[3] != 2 * ceil_div(D, 64))
      return FQ_ERR_PARAM_INVALID;
    eb = 1;
  } else {
    if (scale->dtype != FQ_DT_FLOAT32 || !shape_is(*scale, 3, pages, H, P)) return FQ_ERR_PARAM_INVALID;
    eb = 4;
  }
  const int64_t sstride0 = pages == 1 ? 0 : scale->strides[0];
  if (!inner_contiguous(*scale) || sstride0 * eb % 16 != 0 || sstride0 >= lim) return FQ_ERR_PARAM_INVALID;
  sd->scale = static_cast<uint8_t*>(scale->data);
  sd->scale_page_b = sstride0 * eb;
  return FQ_SUCCESS;
}

// Both sides.  The scale tensors are required for the low-bit formats only.
fq_status cache_null(const fq_tensor* k, const fq_tensor* ks, const fq_tensor* v, const fq_tensor* vs) {
  if (!k || !v || !k->data || !v->data) return FQ_ERR_PARAM_NULLPTR;
  const bool wide = k->dtype == FQ_DT_FLOAT16 || k->dtype == FQ_DT_BFLOAT16;
  if (!wide && (!ks || !vs || !ks->data || !vs->data)) return FQ_ERR_PARAM_NULLPTR;
  return FQ_SUCCESS;
}

fq_status cache_of(const fq_tensor* k, const fq_tensor* ks, const fq_tensor* v, const fq_tensor* vs, KvCache* c) {
  if (v->dtype != k->dtype) return FQ_ERR_PARAM_INVALID;
  const fq_status st = side_of(k, ks, true, c, &c->k);
  return st != FQ_SUCCESS ? st : side_of(v, vs, false, c, &c->v);
}

// Workgroups of a launch: all kernels here have 256 threads, and a grid has fewer than 2^32 of them in x.
constexpr int64_t kWorkgroups = (int64_t(1) << 24) - 1;

// T tokens as the cache kernels deal them out: D / 8 lanes, rounded up to 8, 16 or 32, a token
bool tokens_ok(int64_t T, int64_t D) {
  return T >= 0 && T <= kWorkgroups * (D <= 64 ? 32 : D <= 128 ? 16 : 8);
}

int32_t row_dtype(int32_t t) { return t == FQ_DT_FLOAT16 ? kF16 : t == FQ_DT_BFLOAT16 ? kBF16 : 0; }

bool table_ok(const fq_tensor& t, int64_t B, BlockTable* bt) {
  if (!strides_ok(t) || t.dtype != FQ_DT_INT32 || t.ndim != 2 || t.shape[0] != B || t.shape[1] < 0 ||
      t.shape[1] >= (int64_t(1) << 31))
    return false;
  bt->p = static_cast<const int32_t*>(t.data);
  bt->stride = t.strides[0];
  bt->width = static_cast<int32_t>(t.shape[1]);
  return empty(t) || ((t.shape[1] == 1 || t.strides[1] == 1) && aligned(t.data, 4));
}

// The scale of the scores in fp32.  The kernels multiply by scale * log2(e), which has to stay finite, and a
// scale too small for fp32 is its smallest number, not 0: a masked score is -infinity times it, and the
// weights come out as 1 either way.
bool scale_ok(double scale, int64_t D, float* out) {
  if (!(std::fabs(scale) <= 0x1p127)) return false;
  const float f = scale == 0.0 ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(D))) : static_cast<float>(scale);
  *out = std::fabs(f) > 0.0f ? f : std::copysign(0x1p-149f, static_cast<float>(scale));
  return true;
}

bool lse_ok(const fq_tensor* t, int64_t n, int64_t heads) {
  return !t || (strides_ok(*t) && t->dtype == FQ_DT_FLOAT32 && shape_is(*t, 2, n, heads) && is_contiguous(*t) && aligned(t->data, 4));
}

}  // namespace

extern "C" {

fq_status fq_kv_write(const fq_tensor* k, const fq_tensor* v, const fq_tensor* slots, double clipRatio,
                      double dstTypeMax, const fq_tensor* k_cache, const fq_tensor* k_scale, const fq_tensor* v_cache,
                      const fq_tensor* v_scale, hipStream_t stream) {
  clear_last_error();
  if (missing(k) || missing(v) || missing(slots)) return FQ_ERR_PARAM_NULLPTR;
  fq_status st = cache_null(k_cache, k_scale, v_cache, v_scale);
  if (st != FQ_SUCCESS) return st;
  if (!(clipRatio > 0.0 && clipRatio <= 1.0) || !(dstTypeMax == 0.0 || (dstTypeMax >= 6.0 && dstTypeMax <= 12.0)))
    return FQ_ERR_PARAM_INVALID;
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
  const double qmax = c.mode == kKvInt8 ? 127.0 : c.mode == kKvE4M3 ? 448.0 : 7.0;
  const hipError_t err = launch_kv_write(c, T, kr, vr, static_cast<const int32_t*>(slots->data),
                                         static_cast<float>(qmax / clipRatio), static_cast<float>(dstTypeMax), stream);
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
