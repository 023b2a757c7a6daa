// Checks of the key-value cache's and attention's host files: descriptors to kernel arguments.
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>

#include "fq.h"
#include "fq_attn.h"
#include "fq_host_util.h"

namespace fq {

inline bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

inline bool empty(const fq_tensor& t) {
  if (t.ndim < 0 || t.ndim > 4) return false;
  for (int d = 0; d < t.ndim; ++d)
    if (t.shape[d] == 0) return true;
  return false;
}

// NULL tensors, or NULL data of a tensor that is not empty
inline bool missing(const fq_tensor* t) { return !t || (!t->data && !empty(*t)); }

// 16-bit rows [n, heads, D]
inline bool rows_ok(const fq_tensor& t, int64_t n, int64_t heads, int64_t D, int32_t dtype, Rows16* r) {
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
inline bool out_rows_ok(const fq_tensor& t, int64_t n, int64_t heads, int64_t D, int32_t dtype, Rows16* r) {
  if (!rows_ok(t, n, heads, D, dtype, r)) return false;
  if (empty(t) || (n == 1 && heads == 1)) return true;
  if (n == 1) return r->head >= D;
  if (heads == 1) return r->row >= D;
  // (below 2^57: strides below 2^40, at most 2^17 heads; for the rows compare by division)
  return r->row >= r->head ? r->head >= D && r->row >= (heads - 1) * r->head + D
                           : r->row >= D && (r->head - D) / r->row >= n - 1;
}

inline bool i32_vec(const fq_tensor& t, int64_t n) {
  return strides_ok(t) && t.dtype == FQ_DT_INT32 && shape_is(t, 1, n) && is_contiguous(t) && aligned(t.data, 4);
}

// all dimensions but the first contiguous
inline bool inner_contiguous(const fq_tensor& t) {
  int64_t expect = 1;
  for (int d = t.ndim - 1; d >= 1; --d) {
    if (t.shape[d] != 1 && t.strides[d] != expect) return false;
    expect *= t.shape[d];
  }
  return t.shape[0] == 1 || t.strides[0] >= expect;
}

// One side of the cache; `first` is the side that fixed c's sizes (null for that side itself).
inline fq_status side_of(const fq_tensor* codes, const fq_tensor* scale, bool first, KvCache* c, KvSide* sd) {
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
inline fq_status cache_null(const fq_tensor* k, const fq_tensor* ks, const fq_tensor* v, const fq_tensor* vs) {
  if (!k || !v || !k->data || !v->data) return FQ_ERR_PARAM_NULLPTR;
  const bool wide = k->dtype == FQ_DT_FLOAT16 || k->dtype == FQ_DT_BFLOAT16;
  if (!wide && (!ks || !vs || !ks->data || !vs->data)) return FQ_ERR_PARAM_NULLPTR;
  return FQ_SUCCESS;
}

inline fq_status cache_of(const fq_tensor* k, const fq_tensor* ks, const fq_tensor* v, const fq_tensor* vs, KvCache* c) {
  if (v->dtype != k->dtype) return FQ_ERR_PARAM_INVALID;
  const fq_status st = side_of(k, ks, true, c, &c->k);
  return st != FQ_SUCCESS ? st : side_of(v, vs, false, c, &c->v);
}

// Workgroups of a launch: all kernels here have 256 threads, and a grid has fewer than 2^32 of them in x.
constexpr int64_t kWorkgroups = (int64_t(1) << 24) - 1;

// T tokens as the cache kernels deal them out: D / 8 lanes, rounded up to 8, 16 or 32, a token
inline bool tokens_ok(int64_t T, int64_t D) {
  return T >= 0 && T <= kWorkgroups * (D <= 64 ? 32 : D <= 128 ? 16 : 8);
}

// the scalars of a call that writes the cache, and the divisor of the formats with a scale a token
inline bool write_scalars_ok(double clipRatio, double dstTypeMax) {
  return clipRatio > 0.0 && clipRatio <= 1.0 && (dstTypeMax == 0.0 || (dstTypeMax >= 6.0 && dstTypeMax <= 12.0));
}
inline float write_divisor(int32_t mode, double clipRatio) {
  return static_cast<float>((mode == kKvInt8 ? 127.0 : mode == kKvE4M3 ? 448.0 : 7.0) / clipRatio);
}

inline int32_t row_dtype(int32_t t) { return t == FQ_DT_FLOAT16 ? kF16 : t == FQ_DT_BFLOAT16 ? kBF16 : 0; }

inline bool table_ok(const fq_tensor& t, int64_t B, BlockTable* bt) {
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
inline bool scale_ok(double scale, int64_t D, float* out) {
  if (!(std::fabs(scale) <= 0x1p127)) return false;
  const float f = scale == 0.0 ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(D))) : static_cast<float>(scale);
  *out = std::fabs(f) > 0.0f ? f : std::copysign(0x1p-149f, static_cast<float>(scale));
  return true;
}

inline bool lse_ok(const fq_tensor* t, int64_t n, int64_t heads) {
  return !t || (strides_ok(*t) && t->dtype == FQ_DT_FLOAT32 && shape_is(*t, 2, n, heads) && is_contiguous(*t) && aligned(t->data, 4));
}

}  // namespace fq
