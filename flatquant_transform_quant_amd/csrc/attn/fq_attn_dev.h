// Device helpers of the key-value cache and attention kernels.
#pragma once

#include <hip/hip_runtime.h>

#include "fq_attn.h"
#include "fq_codec.h"
#include "fq_mfma_common.h"

namespace fq {

typedef __attribute__((ext_vector_type(2))) uint32_t u32x2_t;
typedef __attribute__((ext_vector_type(2))) float f32x2_t;

// Inclusive sum over the lanes up to each lane (DPP row shifts, then the rows' last lanes).
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
  return v;
}

// Index of token t of a sequence as (page, offset): page < 0 where the table has no page of this
// cache for it (short table, entry out of range), and such a token is not followed further.
__device__ __forceinline__ int32_t kv_page(const BlockTable& bt, int64_t b, int32_t t, int32_t page_log, int32_t pages) {
  const int32_t i = t >> page_log;
  if (i >= bt.width) return -1;
  const int32_t p = bt.p[b * bt.stride + i];
  return static_cast<uint32_t>(p) < static_cast<uint32_t>(pages) ? p : -1;
}

// Eight consecutive elements of a row from their codes (w: 16, 8 or 4 bytes) in fp32:
// code * scale, one rounding (exact for E2M1).  e8 255 is NaN.
template <int MODE, int DT>
__device__ __forceinline__ void kv_decode8(const u32x4_t w, float scale, uint32_t e8, float (&v)[8]) {
  if constexpr (MODE == kKv16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = load16<DT>(static_cast<uint16_t>(w[i]));
      v[2 * i + 1] = load16<DT>(static_cast<uint16_t>(w[i] >> 16));
    }
  } else if constexpr (MODE == kKvInt8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(static_cast<int8_t>(w[i / 4] >> (8 * (i % 4)))) * scale;
  } else if constexpr (MODE == kKvE4M3) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[i]), false);
      const f32x2_t b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[i]), true);
      v[4 * i] = a[0] * scale;
      v[4 * i + 1] = a[1] * scale;
      v[4 * i + 2] = b[0] * scale;
      v[4 * i + 3] = b[1] * scale;
    }
  } else if constexpr (MODE == kKvInt4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(static_cast<int32_t>(w[0] << (28 - 4 * i)) >> 28) * scale;
  } else {
    const float s = e8m0_to_float(e8);
    const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], s, 0);
    const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], s, 1);
    const f32x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], s, 2);
    const f32x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], s, 3);
    const float x[8] = {a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = e8 == 255u ? __uint_as_float(0x7FC00000u) : x[i];
  }
}

// Bit 15 of each half that is infinite or NaN.
template <int DT>
__device__ __forceinline__ uint32_t not_finite16(uint32_t x) {
  constexpr uint32_t e = DT == kBF16 ? 0x7F807F80u : 0x7C007C00u, one = DT == kBF16 ? 0x00800080u : 0x04000400u;
  return ((x & e) + one) & 0x80008000u;
}
// All bits of each half that is infinite or NaN.
template <int DT>
__device__ __forceinline__ uint32_t not_finite16_mask(uint32_t x) { return (not_finite16<DT>(x) >> 15) * 0xFFFFu; }

// Factor of sums when the softmax's maximum moves up from `m` to `to`.  A sum may hold the infinity of an element that
// was seen, which has to stay one however far the maximum moves: never 0 (what 2^-126 leaves of a finite sum is far
// below one rounding of any weight near the maximum).
__device__ __forceinline__ float rescale(float m, float to) { return fmaxf(__builtin_amdgcn_exp2f(m - to), 0x1p-126f); }

// Two halves u 2^-24 (u the biased code, an f16 subnormal) -> (u - bias) 2^-9, exact.
__device__ __forceinline__ uint32_t unbias_f16(uint32_t a, uint32_t minus) {
  typedef __attribute__((ext_vector_type(2))) _Float16 h16x2;
  const h16x2 up = __builtin_bit_cast(h16x2, 0x78007800u);  // 2^15
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(h16x2, a), up, __builtin_bit_cast(h16x2, minus)));
}
constexpr uint32_t kMinus8 = 0xA400A400u, kMinus128 = 0xB400B400u;  // -8 2^-9, -128 2^-9
template <int SEL>
__device__ __forceinline__ uint32_t fp4_to_f16x2(uint32_t w, float s) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, SEL));
}
template <bool HI>
__device__ __forceinline__ uint32_t fp8_to_f16x2(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
}

// 2^e as fp32 for e in [-126, 127]; 0 below (e never passes 127 here)
__device__ __forceinline__ float pow2(int e) { return e < -126 ? 0.0f : __int_as_float((e + 127) << 23); }

// The codes of elements 8c .. 8c+7 of a row.
template <int MODE>
__device__ __forceinline__ u32x4_t kv_load8(const uint8_t* row, int c) {
  if constexpr (MODE == kKv16) {
    return *reinterpret_cast<const u32x4_t*>(row + 16 * c);
  } else if constexpr (MODE == kKvInt8 || MODE == kKvE4M3) {
    const u32x2_t r = *reinterpret_cast<const u32x2_t*>(row + 8 * c);
    return u32x4_t{r[0], r[1], 0u, 0u};
  } else {
    return u32x4_t{*reinterpret_cast<const uint32_t*>(row + 4 * c), 0u, 0u, 0u};
  }
}

}  // namespace fq
