// Internal interface of the key-value cache and attention kernels (host checks -> launchers).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "fq_internal.h"

namespace fq {

// Storage of a cache row of D elements (kKv16: the rows' own 16-bit type).
enum KvMode : int32_t { kKv16 = 0, kKvInt8 = 1, kKvE4M3 = 2, kKvInt4 = 3, kKvFp4 = 4 };

// bytes of a row's codes; bytes of its scale (0 for kKv16)
__host__ __device__ inline int64_t kv_row_bytes(int32_t mode, int64_t D) {
  return mode == kKv16 ? 2 * D : (mode == kKvInt8 || mode == kKvE4M3) ? D : D / 2;
}
__host__ __device__ inline int64_t kv_scale_bytes(int32_t mode, int64_t D) {
  return mode == kKv16 ? 0 : mode == kKvFp4 ? 2 * ceil_div(D, 64) : 4;
}

// One side (keys or values) of a paged cache: [pages, Hkv, P] rows of codes, of scales.
struct KvSide {
  uint8_t* codes;
  uint8_t* scale;
  int64_t page_b, scale_page_b;  // bytes from one page to the next
};

struct KvCache {
  KvSide k, v;
  int32_t mode;   // KvMode
  int32_t dtype;  // of the rows: kF16 | kBF16
  int32_t Hkv, D;
  int32_t pages, page_log;  // P = 1 << page_log
};

struct Rows16 {  // 16-bit rows [n, heads, D], innermost stride 1; strides in elements
  uint16_t* p;
  int64_t row, head;
};

struct BlockTable {  // int32 [B, width], rows `stride` apart
  const int32_t* p;
  int64_t stride;
  int32_t width;
};

hipError_t launch_kv_write(const KvCache& c, int64_t T, const Rows16& k, const Rows16& v, const int32_t* slots, float d,
                           float dmax, hipStream_t s);
hipError_t launch_kv_read(const KvCache& c, int64_t T, int32_t B, const BlockTable& bt, const int32_t* cu, const Rows16& k,
                          const Rows16& v, hipStream_t s);

struct DecodeArgs {
  KvCache c;
  BlockTable bt;
  const int32_t* lengths;
  Rows16 q, out;
  float* lse;  // [B, Hq] or null
  int32_t B, Hq, g;
  float scale;  // of the scores, natural log domain
};
uint64_t attn_decode_workspace(int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int64_t max_tokens);
hipError_t launch_attn_decode(const DecodeArgs& a, void* ws, hipStream_t s);

struct PrefillArgs {
  Rows16 q, k, v, out;
  float* lse;  // [Tq, Hq] or null
  const int32_t *cu_q, *cu_k;
  int32_t B, Tq, Tk, Hq, g, D, dtype, causal;
  float scale;
};
uint64_t attn_prefill_workspace(int64_t Tq, int64_t Tk, int64_t B, int64_t Hq, int64_t D);
hipError_t launch_attn_prefill(const PrefillArgs& a, void* ws, hipStream_t s);

}  // namespace fq
