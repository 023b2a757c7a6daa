// A cache row quantized and stored, eight elements a lane: what every kernel that writes the cache ends with.
#pragma once

#include "fq_attn_dev.h"

namespace fq {

// Max over aligned groups of SPAN lanes, as integers: |x| as fp32 bits orders finite values,
// then infinity, then NaN, so a row that holds either shows it in its maximum.
template <int SPAN>
__device__ __forceinline__ uint32_t group_umax(uint32_t v) {
  v = max(v, dpp_u<kDppQuadXor1>(v));
  v = max(v, dpp_u<kDppQuadXor2>(v));
  if constexpr (SPAN >= 8) v = max(v, dpp_u<kDppRowHalfMirror>(v));
  if constexpr (SPAN >= 16) v = max(v, dpp_u<kDppRowMirror>(v));
  if constexpr (SPAN >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(r[0], r[1]);
  }
  return v;
}

// One 8-element piece (number ch) of a row of fp32 values quantized and stored: codes and scale rows at `codes`, `scale`.
// The LPR lanes of a row come here together, those past D with zeros.
template <int MODE, int DT, int LPR, int SV>
__device__ __forceinline__ void kv_store8(const float (&x)[8], uint8_t* codes, uint8_t* scale, int ch, int D, float d, float dmax, bool store) {
  if constexpr (MODE == kKv16) {
    if (store)
      *reinterpret_cast<u32x4_t*>(codes + 16 * ch) =
          u32x4_t{round16x2<DT>(x[0], x[1]), round16x2<DT>(x[2], x[3]), round16x2<DT>(x[4], x[5]), round16x2<DT>(x[6], x[7])};
  } else {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    top = group_umax<MODE == kKvFp4 ? 4 : LPR>(top);
    const bool finite = top < 0x7F800000u;
    if constexpr (MODE == kKvFp4) {
      uint32_t e8 = e8m0_code_v<SV>(__uint_as_float(top), dmax, 0.0f);
      const float s = e8m0_to_float(e8);
      uint32_t w = fp4x2<0>(0u, x[0], x[1], s);
      w = fp4x2<1>(w, x[2], x[3], s);
      w = fp4x2<2>(w, x[4], x[5], s);
      w = fp4x2<3>(w, x[6], x[7], s);
      if (!finite) {
        w = 0u;
        e8 = 255u;
      }
      if (store) {
        *reinterpret_cast<uint32_t*>(codes + 4 * ch) = w;
        if (ch % 4 == 0) {
          const int n = D / 32;
          scale[ch / 4] = static_cast<uint8_t>(e8);
          if ((n & 1) && ch / 4 == n - 1) scale[n] = 0;  // the pad byte of an odd group count
        }
      }
    } else {
      const float sc = __uint_as_float(top) / d;
      // q = x / sc, correctly rounded, from one reciprocal a row: with inv the rounded 1 / sc, q0 = x inv
      // is within an ulp or so, the fused remainder x - q0 sc is exact, and q0 + remainder * inv
      // rounds to the quotient (Markstein's correction).  Scales near the ends of the exponent range,
      // where the remainder could underflow, divide.
      const bool mid = sc > 0x1p-90f && sc < 0x1p100f;
      const float inv = mid ? 1.0f / sc : 0.0f;
      float q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float q0 = x[i] * inv;
        q[i] = __builtin_fmaf(__builtin_fmaf(-q0, sc, x[i]), inv, q0);
        if constexpr (MODE == kKvE4M3) q[i] = __builtin_copysignf(q[i], x[i]);  // (the sum of a +0 and a -0 is +0)
      }
      if (!mid) {
        const bool some = finite && sc > 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = some ? x[i] / sc : 0.0f;
      }
      if (store) {
        if constexpr (MODE == kKvInt4) {
          uint32_t w = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) w |= int4_nibble(q[i]) << (4 * i);
          *reinterpret_cast<uint32_t*>(codes + 4 * ch) = w;
        } else {
          constexpr int CM = MODE == kKvInt8 ? kPerTokenInt8 : kPerTokenE4M3;
          *reinterpret_cast<u32x2_t*>(codes + 8 * ch) =
              u32x2_t{code8x4<CM>(q[0], q[1], q[2], q[3]), code8x4<CM>(q[4], q[5], q[6], q[7])};
        }
        if (ch == 0) *reinterpret_cast<float*>(scale) = sc;
      }
    }
  }
}

// The same of a piece of a 16-bit row, which a 16-bit cache takes unchanged.
template <int MODE, int DT, int LPR, int SV>
__device__ __forceinline__ void kv_store8(const u32x4_t raw, uint8_t* codes, uint8_t* scale, int ch, int D, float d, float dmax, bool store) {
  if constexpr (MODE == kKv16) {
    if (store) *reinterpret_cast<u32x4_t*>(codes + 16 * ch) = raw;
  } else {
    float x[8];
    kv_decode8<kKv16, DT>(raw, 1.0f, 0, x);
    kv_store8<MODE, DT, LPR, SV>(x, codes, scale, ch, D, d, dmax, store);
  }
}

// How many tokens a workgroup of `threads` takes, whose lane groups of `lpr` lanes own a row each: one a lane group
// where that gives `enough` workgroups; fewer spread a small call over more of them, the lane groups of a token
// sharing its `heads`, down to a lane group per head.
inline int tokens_of(int64_t T, int heads, int lpr, int threads, int enough) {
  int tokens = threads / lpr;
  while (tokens > 1 && tokens / 2 * heads >= threads / lpr && ceil_div(T, tokens) < enough) tokens >>= 1;
  return tokens;
}

// f(lanes of a row)
template <typename F>
void by_lanes(int D, F&& f) {
  if (D <= 64) f(std::integral_constant<int, 8>{});
  else if (D <= 128) f(std::integral_constant<int, 16>{});
  else f(std::integral_constant<int, 32>{});
}

}  // namespace fq
