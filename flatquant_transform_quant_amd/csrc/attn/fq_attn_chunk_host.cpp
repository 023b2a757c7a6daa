// Host side of attention of new tokens over the cache (include/fq.h): checks, sizes and dispatch.
#include <algorithm>

#include "fq_attn_checks.h"

using namespace fq;

namespace {

constexpr int64_t kKeys = 64;               // of a key tile
constexpr int64_t kPlaces = 5;              // key tiles that a segment's places may have above those of its span
// Workgroups of a launch: two a CU, one of heads above 128 (their LDS and registers).  A run of fewer than kLeast tiles
// costs more in parts to join than it gains.
constexpr int64_t kLeast = 8;
// Key tiles of the longest walk up to which every row tile is one workgroup's, without parts and a second launch.  us with 12, 24 and
// 48: 32 single tokens with a window of 1024 46.9, 31.6, 31.6; four 23.8, 21.5, 21.8; 32 of 300 to 1500 42.3, 36.5, 36.4; 128 of
// them in int4, 64 heads 92.8, 76.4, 77.0.
constexpr int64_t kShort = 24;

// The parts of a call that its workspace depends on, into a's sizes.
bool chunk_sizes(const fq_tensor* q, const fq_tensor* k_cache, const fq_tensor* block_table, const fq_tensor* cu_q, int32_t window,
                 int32_t sinks, ChunkArgs* a) {
  if (q->ndim != 3 || k_cache->ndim != 4 || block_table->ndim != 2 || cu_q->ndim != 1 || window < 0 || sinks < 0) return false;
  const int64_t Tq = q->shape[0], Hq = q->shape[1], D = q->shape[2], Hkv = k_cache->shape[1], P = k_cache->shape[2];
  const int64_t B = cu_q->shape[0] - 1, lim = (int64_t(1) << 31) - 65536;
  if (B < 1 || B > 65536 || Tq < 0 || Tq >= lim || Hq < 1 || Hq > 65536 || Hkv < 1 || Hkv > 1024 || Hq % Hkv != 0 || D < 8 || D > 256 ||
      D != k_cache->shape[3] || P < 16 || P > 1024 || block_table->shape[1] < 0 || block_table->shape[1] >= (int64_t(1) << 31) ||
      block_table->shape[1] * P >= lim)
    return false;
  const int64_t reach = block_table->shape[1] * P, g = Hq / Hkv;
  a->reach = static_cast<int32_t>(reach);
  a->B = static_cast<int32_t>(B);
  a->Tq = static_cast<int32_t>(Tq);
  a->Hq = static_cast<int32_t>(Hq);
  a->g = static_cast<int32_t>(g);
  const int64_t rows = ceil_div(Tq, B) * g;  // of a sequence and cache head, the mean
  a->tile_rows = rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
  a->head_tiles = static_cast<int32_t>(ceil_div(g, a->tile_rows));
  a->tile_heads = static_cast<int32_t>(ceil_div(g, a->head_tiles));
  a->tokens = a->tile_rows / a->tile_heads;
  a->heads = static_cast<int32_t>(Hkv * a->head_tiles);
  a->window = window >= reach ? 0 : window;  // (one of the whole reach hides nothing)
  a->sinks = a->window > 0 ? static_cast<int32_t>(std::min<int64_t>(sinks, reach)) : 0;
  // places of all segments, counted in 31 bits: row tiles of all sequences (at most one partial one each)
  const int64_t segments = (Tq / a->tokens + std::min(B, Tq)) * a->heads;
  if (segments >= int64_t(1) << 31) return false;
  int64_t span = reach + a->tokens;
  if (a->window > 0) span = std::min(span, int64_t(a->window) + a->tokens + 126) + ceil_div(a->sinks, kKeys) * kKeys;
  const int64_t places = segments * (ceil_div(span, kKeys) + kPlaces);
  if (places >= int64_t(1) << 31) return false;
  a->single = ceil_div(span, kKeys) <= kShort && segments < (int64_t(1) << 24) - 8 ? 1 : 0;
  a->runs = static_cast<int32_t>(a->single ? std::max<int64_t>(1, segments)
                                           : std::max<int64_t>(1, std::min<int64_t>(D > 128 ? 256 : 512, places / kLeast)));
  return true;
}

uint64_t chunk_workspace(const ChunkArgs& a, int64_t D) {
  const uint64_t padded = D <= 64 ? 64 : D <= 128 ? 128 : 256;
  return a.runs == 1 || a.single ? 0 : static_cast<uint64_t>(2 * a.runs) * (padded + 2) * a.tile_rows * sizeof(float);
}

}  // namespace

extern "C" {

fq_status fq_attn_chunk_get_workspace_size(const fq_tensor* q, const fq_tensor* k_cache, const fq_tensor* block_table, const fq_tensor* cu_q,
                                           int32_t window, int32_t sinks, uint64_t* workspaceSize) {
  clear_last_error();
  if (!q || !k_cache || !block_table || !cu_q || !workspaceSize) return FQ_ERR_PARAM_NULLPTR;
  ChunkArgs a{};
  if (!chunk_sizes(q, k_cache, block_table, cu_q, window, sinks, &a)) return FQ_ERR_PARAM_INVALID;
  *workspaceSize = chunk_workspace(a, q->shape[2]);
  return FQ_SUCCESS;
}

fq_status fq_attn_chunk(const fq_tensor* q, const fq_tensor* k_cache, const fq_tensor* k_scale, const fq_tensor* v_cache,
                        const fq_tensor* v_scale, const fq_tensor* block_table, const fq_tensor* cu_q, const fq_tensor* lengths,
                        int32_t window, int32_t sinks, double scale, const fq_tensor* out, const fq_tensor* lse, void* workspace,
                        uint64_t workspaceSize, hipStream_t stream) {
  clear_last_error();
  for (const fq_tensor* t : {q, block_table, cu_q, lengths, out})
    if (missing(t)) return FQ_ERR_PARAM_NULLPTR;
  if (lse && missing(lse)) return FQ_ERR_PARAM_NULLPTR;
  fq_status st = cache_null(k_cache, k_scale, v_cache, v_scale);
  if (st != FQ_SUCCESS) return st;
  ChunkArgs a{};
  st = cache_of(k_cache, k_scale, v_cache, v_scale, &a.c);
  if (st != FQ_SUCCESS) return st;
  if (!chunk_sizes(q, k_cache, block_table, cu_q, window, sinks, &a) || row_dtype(q->dtype) == 0 || !scale_ok(scale, q->shape[2], &a.scale))
    return FQ_ERR_PARAM_INVALID;
  const int64_t Tq = q->shape[0], Hq = q->shape[1], D = q->shape[2], B = a.B;
  if (!table_ok(*block_table, B, &a.bt) || !i32_vec(*cu_q, B + 1) || !i32_vec(*lengths, B) || !rows_ok(*q, Tq, Hq, D, q->dtype, &a.q) ||
      !out_rows_ok(*out, Tq, Hq, D, q->dtype, &a.out) || !lse_ok(lse, Tq, Hq) || (a.c.mode == kKv16 && a.c.dtype != row_dtype(q->dtype)))
    return FQ_ERR_PARAM_INVALID;
  a.c.dtype = row_dtype(q->dtype);
  // (integer codes are operands of 2^-9 of theirs, and f16 rows go in as they are, so that the scores' factor is 2^9 times the scale)
  if ((a.c.mode == kKvInt8 || a.c.mode == kKvInt4) && a.c.dtype == kF16 && std::fabs(a.scale) > 0x1p118f) return FQ_ERR_PARAM_INVALID;
  const uint64_t need = chunk_workspace(a, D);
  if (need > 0 && !workspace) return FQ_ERR_PARAM_NULLPTR;
  if (workspaceSize < need || (need > 0 && !aligned(workspace, 16))) return FQ_ERR_PARAM_INVALID;
  if (Tq == 0) return FQ_SUCCESS;
  if (!device_is_gfx950()) return fail_runtime("the current device is not gfx950", hipSuccess);
  a.cu_q = static_cast<const int32_t*>(cu_q->data);
  a.lengths = static_cast<const int32_t*>(lengths->data);
  a.lse = lse ? static_cast<float*>(lse->data) : nullptr;
  const auto launch = a.c.mode == kKv16     ? launch_attn_chunk_16
                      : a.c.mode == kKvInt8 ? launch_attn_chunk_int8
                      : a.c.mode == kKvE4M3 ? launch_attn_chunk_e4m3
                      : a.c.mode == kKvInt4 ? launch_attn_chunk_int4
                                            : launch_attn_chunk_fp4;
  const hipError_t err = launch(a, workspace, stream);
  return err == hipSuccess ? FQ_SUCCESS : fail_runtime("chunk attention kernel launch", err);
}

}  // extern "C"
