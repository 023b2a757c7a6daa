// The paged key-value cache: rows quantized as they are written, and read back as values.
//
// A row is one token's D elements of one head.  Per token: scale = fl32(max|x| / d), d =
// fl32(max_val / clipRatio), code = the integer or FP8 value nearest x / scale (the quantizer's
// per-token rules, fq_codec.h).  Per group of 32: the e8m0 rule of dstTypeMax and E2M1 codes.
// Both kernels only stream: a lane takes 8 elements (16 bytes of 16-bit values against 16, 8 or
// 4 bytes of codes), D / 8 lanes (rounded up to 8, 16 or 32) a row, and the row's or group's
// maximum is taken between those lanes with DPP moves.
#include <hip/hip_runtime.h>

#include "fq_attn_dev.h"

namespace fq {
namespace {

constexpr int kThreads = 256;
constexpr int kReadTokens = 16;  // tokens of a workgroup of the read kernel

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

// MODE, the rows' dtype, lanes per row, e8m0 rule (kE8V1 or kE8V2Div)
template <int MODE, int DT, int LPR, int SV>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(KvCache c, uint32_t items, Rows16 kin, Rows16 vin,
                                                             const int32_t* __restrict__ slots, float d, float dmax) {
  // item = (token, head, side), the side fastest: a wave's 64 / LPR rows
  const uint32_t item = blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR;
  const int ch = threadIdx.x % LPR;  // elements 8 ch .. 8 ch + 7
  const bool in_row = 8 * ch < c.D;
  const uint32_t side = item & 1u, th = item >> 1;
  const uint32_t t = th / static_cast<uint32_t>(c.Hkv), h = th - t * static_cast<uint32_t>(c.Hkv);
  const bool live = item < items && in_row;
  const int32_t slot = item < items ? slots[t] : -1;
  u32x4_t raw = {0u, 0u, 0u, 0u};
  if (live) {
    const Rows16& in = side ? vin : kin;
    raw = *reinterpret_cast<const u32x4_t*>(in.p + t * in.row + h * in.head + 8 * ch);
  }
  const int32_t page = slot >> c.page_log;  // a negative slot stays negative
  const bool store = live && page >= 0 && page < c.pages;
  const KvSide& sd = side ? c.v : c.k;
  const int64_t row = (static_cast<int64_t>(h) << c.page_log) + (slot & ((1 << c.page_log) - 1));
  if constexpr (MODE == kKv16) {
    if (store)
      *reinterpret_cast<u32x4_t*>(sd.codes + page * sd.page_b + row * 2 * c.D + 16 * ch) = raw;
  } else {
    float x[8];
    kv_decode8<kKv16, DT>(raw, 1.0f, 0, x);
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
        *reinterpret_cast<uint32_t*>(sd.codes + page * sd.page_b + row * (c.D / 2) + 4 * ch) = w;
        const int n = c.D / 32, sb = 2 * ((c.D + 63) / 64);
        uint8_t* sc = sd.scale + page * sd.scale_page_b + row * sb;
        if (ch % 4 == 0) {
          sc[ch / 4] = static_cast<uint8_t>(e8);
          if (n < sb && ch / 4 == n - 1) sc[n] = 0;  // the pad byte of an odd group count
        }
      }
    } else {
      const float scale = __uint_as_float(top) / d;
      // q = x / scale, correctly rounded, from one reciprocal a row: with inv the rounded 1 / scale,
      // q0 = x inv is within an ulp or so, the fused remainder x - q0 scale is exact, and q0 +
      // remainder * inv rounds to the quotient (Markstein's correction).  Scales near the ends of
      // the exponent range, where the remainder could underflow, divide.
      const bool mid = scale > 0x1p-90f && scale < 0x1p100f;
      const float inv = mid ? 1.0f / scale : 0.0f;
      float q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float q0 = x[i] * inv;
        q[i] = __builtin_fmaf(__builtin_fmaf(-q0, scale, x[i]), inv, q0);
        if constexpr (MODE == kKvE4M3) q[i] = __builtin_copysignf(q[i], x[i]);  // (the sum of a +0 and a -0 is +0)
      }
      if (!mid) {
        const bool some = finite && scale > 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = some ? x[i] / scale : 0.0f;
      }
      if (store) {
        uint8_t* const codes = sd.codes + page * sd.page_b;
        if constexpr (MODE == kKvInt4) {
          uint32_t w = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) w |= int4_nibble(q[i]) << (4 * i);
          *reinterpret_cast<uint32_t*>(codes + row * (c.D / 2) + 4 * ch) = w;
        } else {
          constexpr int CM = MODE == kKvInt8 ? kPerTokenInt8 : kPerTokenE4M3;
          *reinterpret_cast<u32x2_t*>(codes + row * c.D + 8 * ch) =
              u32x2_t{code8x4<CM>(q[0], q[1], q[2], q[3]), code8x4<CM>(q[4], q[5], q[6], q[7])};
        }
        if (ch == 0) *reinterpret_cast<float*>(sd.scale + page * sd.scale_page_b + row * 4) = scale;
      }
    }
  }
}

template <int MODE, int DT, int LPR>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvCache c, int32_t T, int32_t B, BlockTable bt,
                                                            const int32_t* __restrict__ cu, Rows16 kout, Rows16 vout) {
  // this workgroup's tokens: their sequences by bisection of cu, their pages from the table
  __shared__ int32_t s_page[kReadTokens], s_off[kReadTokens];
  const int32_t t0 = blockIdx.x * kReadTokens;
  if (threadIdx.x < kReadTokens) {
    const int32_t t = t0 + static_cast<int32_t>(threadIdx.x);
    int32_t page = -2, off = 0;  // -2: not a row of any sequence, not written
    if (t < T && t < cu[B]) {
      int32_t lo = 0, hi = B;  // cu[lo] <= t < cu[hi]
      while (hi - lo > 1) {
        const int32_t m = (lo + hi) >> 1;
        if (cu[m] <= t) lo = m; else hi = m;
      }
      const int32_t pos = t - cu[lo];
      page = pos >= 0 ? kv_page(bt, lo, pos, c.page_log, c.pages) : -2;
      off = pos & ((1 << c.page_log) - 1);
    }
    s_page[threadIdx.x] = page;
    s_off[threadIdx.x] = off;
  }
  __syncthreads();
  // items (side, head, token), the token fastest, LPR lanes each
  const int ch = threadIdx.x % LPR;
  const int n = 2 * c.Hkv * kReadTokens;
  if (8 * ch >= c.D) return;
#pragma unroll 4
  for (int it = threadIdx.x / LPR; it < n; it += kThreads / LPR) {
    const int tk = it % kReadTokens, sh = it / kReadTokens;
    const int side = sh >= c.Hkv, h = sh - (side ? c.Hkv : 0);
    const int32_t page = s_page[tk];
    if (page == -2) continue;
    const KvSide& sd = side ? c.v : c.k;
    u32x4_t o = {0u, 0u, 0u, 0u};
    if (page >= 0) {
      const int64_t row = (static_cast<int64_t>(h) << c.page_log) + s_off[tk];
      const u32x4_t w = kv_load8<MODE>(sd.codes + page * sd.page_b + row * kv_row_bytes(MODE, c.D), ch);
      if constexpr (MODE == kKv16) {
        o = w;
      } else {
        const uint8_t* sc = sd.scale + page * sd.scale_page_b;
        float scale = 0.0f, v[8];
        uint32_t e8 = 0;
        if constexpr (MODE == kKvFp4)
          e8 = sc[row * (2 * ((c.D + 63) / 64)) + ch / 4];
        else
          scale = *reinterpret_cast<const float*>(sc + row * 4);
        kv_decode8<MODE, DT>(w, scale, e8, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = round16x2<DT>(v[2 * i], v[2 * i + 1]);
      }
    }
    const Rows16& out = side ? vout : kout;
    __builtin_nontemporal_store(o, reinterpret_cast<u32x4_t*>(out.p + (t0 + tk) * out.row + h * out.head + 8 * ch));
  }
}

template <int MODE, int DT>
hipError_t write_mode(const KvCache& c, int64_t T, const Rows16& k, const Rows16& v, const int32_t* slots, float d,
                      float dmax, hipStream_t s) {
  const uint32_t items = static_cast<uint32_t>(2 * T * c.Hkv);
  auto go = [&](auto lpr, auto sv) {
    constexpr int L = decltype(lpr)::value, SV = decltype(sv)::value;
    kv_write_kernel<MODE, DT, L, SV><<<static_cast<uint32_t>(ceil_div(items, kThreads / L)), kThreads, 0, s>>>(
        c, items, k, v, slots, d, dmax);
  };
  auto by_rule = [&](auto lpr) {
    if constexpr (MODE == kKvFp4) {
      if (dmax != 0.0f) return go(lpr, std::integral_constant<int, kE8V2Div>{});
    }
    go(lpr, std::integral_constant<int, kE8V1>{});
  };
  if (c.D <= 64) by_rule(std::integral_constant<int, 8>{});
  else if (c.D <= 128) by_rule(std::integral_constant<int, 16>{});
  else by_rule(std::integral_constant<int, 32>{});
  return hipGetLastError();
}

template <int MODE, int DT>
hipError_t read_mode(const KvCache& c, int64_t T, int32_t B, const BlockTable& bt, const int32_t* cu, const Rows16& k,
                     const Rows16& v, hipStream_t s) {
  const uint32_t grid = static_cast<uint32_t>(ceil_div(T, kReadTokens));
  auto go = [&](auto lpr) {
    kv_read_kernel<MODE, DT, decltype(lpr)::value><<<grid, kThreads, 0, s>>>(c, static_cast<int32_t>(T), B, bt, cu, k, v);
  };
  if (c.D <= 64) go(std::integral_constant<int, 8>{});
  else if (c.D <= 128) go(std::integral_constant<int, 16>{});
  else go(std::integral_constant<int, 32>{});
  return hipGetLastError();
}

// f(mode constant, dtype constant); a 16-bit cache is copied whatever its dtype
template <typename F>
hipError_t by_mode(const KvCache& c, F&& f) {
  using std::integral_constant;
  auto dt = [&](auto m) {
    return c.dtype == kF16 ? f(m, integral_constant<int, kF16>{}) : f(m, integral_constant<int, kBF16>{});
  };
  switch (c.mode) {
    case kKv16: return f(integral_constant<int, kKv16>{}, integral_constant<int, kBF16>{});
    case kKvInt8: return dt(integral_constant<int, kKvInt8>{});
    case kKvE4M3: return dt(integral_constant<int, kKvE4M3>{});
    case kKvInt4: return dt(integral_constant<int, kKvInt4>{});
    default: return dt(integral_constant<int, kKvFp4>{});
  }
}

}  // namespace

hipError_t launch_kv_write(const KvCache& c, int64_t T, const Rows16& k, const Rows16& v, const int32_t* slots, float d,
                           float dmax, hipStream_t s) {
  return by_mode(c, [&](auto m, auto dt) { return write_mode<decltype(m)::value, decltype(dt)::value>(c, T, k, v, slots, d, dmax, s); });
}

hipError_t launch_kv_read(const KvCache& c, int64_t T, int32_t B, const BlockTable& bt, const int32_t* cu, const Rows16& k,
                          const Rows16& v, hipStream_t s) {
  return by_mode(c, [&](auto m, auto dt) { return read_mode<decltype(m)::value, decltype(dt)::value>(c, T, B, bt, cu, k, v, s); });
}

}  // namespace fq
