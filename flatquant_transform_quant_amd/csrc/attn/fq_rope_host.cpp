// Host side of the norm and rotation calls of include/fq.h: checks and dispatch.
#include "fq_attn_checks.h"

using namespace fq;

namespace {

// What the two calls share.  q or k may be NULL (none of these rows); D comes from the one that is there.
fq_status rope_null(const fq_tensor* q, const fq_tensor* q_out, const fq_tensor* q_weight, const fq_tensor* k_weight,
                    const fq_tensor* positions, const fq_tensor* inv_freq, const fq_tensor* axes) {
  if ((q && missing(q)) || (q && missing(q_out)) || (q_weight && missing(q_weight)) || (k_weight && missing(k_weight)) ||
      missing(positions) || missing(inv_freq) || (axes && missing(axes)))
    return FQ_ERR_PARAM_NULLPTR;
  return FQ_SUCCESS;
}

bool norm_ok(const fq_tensor* t, int64_t D, RopeNorm* n) {
  *n = RopeNorm{nullptr, 0};
  if (!t) return true;
  const bool wide = t->dtype == FQ_DT_FLOAT32;
  if (!strides_ok(*t) || (!wide && row_dtype(t->dtype) == 0) || !shape_is(*t, 1, D) || !is_contiguous(*t) || !aligned(t->data, wide ? 4 : 2))
    return false;
  *n = RopeNorm{t->data, wide ? kNormF32 : row_dtype(t->dtype)};
  return true;
}

// positions, frequencies, axes, norms and queries into `a`, whose T, D, dtype and Hkv are set
bool rope_ok(const fq_tensor* q, const fq_tensor* q_out, const fq_tensor* q_weight, const fq_tensor* k_weight, double eps,
             const fq_tensor* positions, const fq_tensor* inv_freq, const fq_tensor* axes, int32_t interleaved, RopeArgs* a) {
  const int64_t T = a->T, D = a->D;
  a->q = a->q_out = Rows16{nullptr, 0, 0};
  a->Hq = 0;
  if (q) {
    if (q->ndim != 3 || q->shape[1] < 0 || q->shape[1] > 65536 || !rows_ok(*q, T, q->shape[1], D, q->dtype, &a->q) ||
        !out_rows_ok(*q_out, T, q->shape[1], D, q->dtype, &a->q_out))
      return false;
    a->Hq = static_cast<int32_t>(q->shape[1]);
  }
  if (!norm_ok(q_weight, D, &a->qn) || !norm_ok(k_weight, D, &a->kn)) return false;
  if (!(eps >= 0x1p-126 && eps <= 0x1p127)) return false;
  a->eps = static_cast<float>(eps);
  if (!strides_ok(*inv_freq) || inv_freq->ndim != 1 || inv_freq->dtype != FQ_DT_FLOAT32 || !is_contiguous(*inv_freq) ||
      !aligned(inv_freq->data, 4) || inv_freq->shape[0] < 0 || inv_freq->shape[0] > D / 2 || inv_freq->shape[0] % 4 != 0)
    return false;
  a->R = static_cast<int32_t>(2 * inv_freq->shape[0]);
  a->inv_freq = static_cast<const float*>(inv_freq->data);
  const fq_tensor& p = *positions;
  if (!strides_ok(p) || p.dtype != FQ_DT_INT32 || !aligned(p.data, 4)) return false;
  if (axes) {
    if (p.ndim != 2 || p.shape[0] < 1 || p.shape[0] > 16 || p.shape[1] != T || !i32_vec(*axes, a->R / 2)) return false;
    a->axes = static_cast<int32_t>(p.shape[0]);
    a->pos_axis = p.strides[0];
    if ((T > 1 && p.strides[1] != 1) || p.strides[0] >= int64_t(1) << 40) return false;
    a->axis = static_cast<const int32_t*>(axes->data);
  } else {
    if (!i32_vec(p, T)) return false;
    a->axes = 1;
    a->pos_axis = 0;
    a->axis = nullptr;
  }
  a->pos = static_cast<const int32_t*>(p.data);
  a->interleaved = interleaved ? 1 : 0;
  return true;
}

bool head_dim_ok(int64_t D) { return D >= 8 && D <= 256 && D % 8 == 0; }

}  // namespace

extern "C" {

fq_status fq_qk_rope(const fq_tensor* q, const fq_tensor* k, const fq_tensor* q_weight, const fq_tensor* k_weight, double eps,
                     const fq_tensor* positions, const fq_tensor* inv_freq, const fq_tensor* axes, int32_t interleaved,
                     const fq_tensor* q_out, const fq_tensor* k_out, hipStream_t stream) {
  clear_last_error();
  const fq_status st = rope_null(q, q_out, q_weight, k_weight, positions, inv_freq, axes);
  if (st != FQ_SUCCESS) return st;
  if ((!q && !k) || (k && (missing(k) || missing(k_out)))) return FQ_ERR_PARAM_NULLPTR;
  const fq_tensor& one = q ? *q : *k;
  RopeArgs a{};
  if (one.ndim != 3 || row_dtype(one.dtype) == 0 || !head_dim_ok(one.shape[2]) || !tokens_ok(one.shape[0], one.shape[2]))
    return FQ_ERR_PARAM_INVALID;
  a.T = one.shape[0];
  a.D = static_cast<int32_t>(one.shape[2]);
  a.dtype = row_dtype(one.dtype);
  if (k) {
    if (k->ndim != 3 || k->shape[1] < 0 || k->shape[1] > 65536 || !rows_ok(*k, a.T, k->shape[1], a.D, one.dtype, &a.k) ||
        !out_rows_ok(*k_out, a.T, k->shape[1], a.D, one.dtype, &a.k_out))
      return FQ_ERR_PARAM_INVALID;
    a.Hkv = static_cast<int32_t>(k->shape[1]);
  }
  if (!rope_ok(q, q_out, q_weight, k_weight, eps, positions, inv_freq, axes, interleaved, &a)) return FQ_ERR_PARAM_INVALID;
  if (a.T == 0 || a.Hq + a.Hkv == 0) return FQ_SUCCESS;
  if (!device_is_gfx950()) return fail_runtime("the current device is not gfx950", hipSuccess);
  const hipError_t err = launch_rope(a, stream);
  return err == hipSuccess ? FQ_SUCCESS : fail_runtime("rotation kernel launch", err);
}

fq_status fq_kv_append(const fq_tensor* q, const fq_tensor* k, const fq_tensor* v, const fq_tensor* slots, const fq_tensor* q_weight,
                       const fq_tensor* k_weight, double eps, const fq_tensor* positions, const fq_tensor* inv_freq,
                       const fq_tensor* axes, int32_t interleaved, double clipRatio, double dstTypeMax, const fq_tensor* k_cache,
                       const fq_tensor* k_scale, const fq_tensor* v_cache, const fq_tensor* v_scale, const fq_tensor* q_out,
                       hipStream_t stream) {
  clear_last_error();
  fq_status st = rope_null(q, q_out, q_weight, k_weight, positions, inv_freq, axes);
  if (st != FQ_SUCCESS) return st;
  if (missing(k) || missing(v) || missing(slots)) return FQ_ERR_PARAM_NULLPTR;
  st = cache_null(k_cache, k_scale, v_cache, v_scale);
  if (st != FQ_SUCCESS) return st;
  RopeArgs a{};
  if (!write_scalars_ok(clipRatio, dstTypeMax)) return FQ_ERR_PARAM_INVALID;
  st = cache_of(k_cache, k_scale, v_cache, v_scale, &a.c);
  if (st != FQ_SUCCESS) return st;
  if (k->ndim != 3) return FQ_ERR_PARAM_INVALID;
  a.T = k->shape[0];
  a.D = a.c.D;
  a.Hkv = a.c.Hkv;
  a.dtype = row_dtype(k->dtype);
  if (a.dtype == 0 || !tokens_ok(a.T, a.D) || (q && q->dtype != k->dtype) || !rows_ok(*k, a.T, a.Hkv, a.D, k->dtype, &a.k) ||
      !rows_ok(*v, a.T, a.Hkv, a.D, k->dtype, &a.v) || !i32_vec(*slots, a.T) || (a.c.mode == kKv16 && a.c.dtype != a.dtype))
    return FQ_ERR_PARAM_INVALID;
  if (!rope_ok(q, q_out, q_weight, k_weight, eps, positions, inv_freq, axes, interleaved, &a)) return FQ_ERR_PARAM_INVALID;
  if (a.T == 0) return FQ_SUCCESS;
  if (!device_is_gfx950()) return fail_runtime("the current device is not gfx950", hipSuccess);
  a.slots = static_cast<const int32_t*>(slots->data);
  a.append = 1;
  a.d = write_divisor(a.c.mode, clipRatio);
  a.dmax = static_cast<float>(dstTypeMax);
  const hipError_t err = launch_rope(a, stream);
  return err == hipSuccess ? FQ_SUCCESS : fail_runtime("cache append kernel launch", err);
}

}  // extern "C"
