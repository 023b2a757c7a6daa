// The paged key-value cache: rows quantized as they are written, and read back as values.
//
// A row is one token's D elements of one head.  Per token: scale = fl32(max|x| / d), d =
// fl32(max_val / clipRatio), code = the integer or FP8 value nearest x / scale (the quantizer's
// per-token rules, fq_codec.h).  Per group of 32: the e8m0 rule of dstTypeMax and E2M1 codes.
// Both kernels only stream: a lane takes 8 elements (16 bytes of 16-bit values against 16, 8 or
// 4 bytes of codes), D / 8 lanes (rounded up to 8, 16 or 32) a row, and the row's or group's
// maximum is taken between those lanes with DPP moves.
//
// Bound by memory: contexts of 16 sequences of up to 32768 tokens read from E2M1, 8 heads of 128 (1.41 GB
// with the 2048 new tokens written): 275 us, 5.1 TB/s, a large copy's rate (5.2); six of up to 9001 in
// int4 with 512 written (153 MB): 30 us, 5.0 TB/s.  One token and 33 read back: 2.5 and 4 us of the
// device, less than the two calls take on the host (8 us each).
#include <hip/hip_runtime.h>

#include "fq_kv_store.h"

namespace fq {
namespace {

constexpr int kThreads = 256;
constexpr int kEnough = 512;   // workgroups of a launch that need no more spreading

// Both kernels: a lane group of LPR lanes owns one token of the workgroup's `tokens` and walks the
// heads, kInFlight heads' keys and values at a time (all loaded before the first is used); with
// fewer tokens than lane groups, the groups of a token share its heads.  So the page lookup
// and the 64-bit addresses are formed once a token, and each head adds a constant.  The lane groups
// of neighbouring tokens read (or write) neighbouring rows of a page.  us with one, two and four heads in
// flight, 16 sequences of up to 18000 tokens, 8 heads of 128: reading int8 342, 320, reading E2M1 294, 279,
// writing 2048 tokens each in int8 34.2, 33.8, 34.1; writing 512 tokens each of 6 in int4 5.7, 5.8, 9.3.
constexpr int kInFlight = 2;

// Small calls are spread over more workgroups (tokens_of).  us without and with: one token, 8 heads of 128,
// int8, written 9.2 and 3.2, 33 read 4.3 and 3.2; 128 written in int4 8.0 and 3.3; 6 x 512 8.7 and 5.8 (spread
// over 2048 workgroups: 9.1).

// MODE, the rows' dtype, lanes per row, e8m0 rule (kE8V1 or kE8V2Div)
template <int MODE, int DT, int LPR, int SV>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(KvCache c, int32_t T, int32_t tokens, Rows16 kin, Rows16 vin,
                                                             const int32_t* __restrict__ slots, float d, float dmax) {
  const int ch = threadIdx.x % LPR, r = threadIdx.x / LPR;  // elements 8 ch .. 8 ch + 7
  const int tk = r % tokens, h0 = r / tokens, dh = (kThreads / LPR) / tokens;
  const int32_t t = blockIdx.x * tokens + tk;
  const int32_t slot = t < T ? slots[t] : -1;
  const int32_t page = slot >> c.page_log;  // a negative slot stays negative
  const bool there = page >= 0 && page < c.pages && 8 * ch < c.D;  // (all lanes stay for the maxima)
  const int64_t rowb = kv_row_bytes(MODE, c.D), sb = kv_scale_bytes(MODE, c.D);
  const int64_t off = slot & ((1 << c.page_log) - 1);
  const int64_t first = (static_cast<int64_t>(h0) << c.page_log) + off;
  const uint16_t* src[2] = {kin.p + t * kin.row + h0 * kin.head + 8 * ch, vin.p + t * vin.row + h0 * vin.head + 8 * ch};
  uint8_t* codes[2] = {c.k.codes + (page * c.k.page_b + first * rowb), c.v.codes + (page * c.v.page_b + first * rowb)};
  uint8_t* scale[2] = {c.k.scale + (page * c.k.scale_page_b + first * sb), c.v.scale + (page * c.v.scale_page_b + first * sb)};
  const int64_t src_d[2] = {dh * kin.head, dh * vin.head}, codes_d = (dh * rowb) << c.page_log, scale_d = (dh * sb) << c.page_log;
  for (int h = h0; h < c.Hkv; h += dh * kInFlight) {
    u32x4_t raw[2][kInFlight];
#pragma unroll
    for (int i = 0; i < kInFlight; ++i)
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        raw[side][i] = u32x4_t{0u, 0u, 0u, 0u};
        if (there && h + i * dh < c.Hkv) raw[side][i] = *reinterpret_cast<const u32x4_t*>(src[side] + i * src_d[side]);
      }
#pragma unroll
    for (int side = 0; side < 2; ++side) {
#pragma unroll
      for (int i = 0; i < kInFlight; ++i) {
        if (i * dh >= c.Hkv) break;  // (a lane group per head has no second one: one token 3.7 us without this line, 3.2 with)
        kv_store8<MODE, DT, LPR, SV>(raw[side][i], codes[side] + i * codes_d, scale[side] + i * scale_d, ch, c.D, d, dmax,
                                     there && h + i * dh < c.Hkv);
      }
      src[side] += kInFlight * src_d[side];
      codes[side] += kInFlight * codes_d;
      scale[side] += kInFlight * scale_d;
    }
  }
}

template <int MODE, int DT, int LPR>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvCache c, int32_t T, int32_t B, int32_t tokens, BlockTable bt,
                                                            const int32_t* __restrict__ cu, Rows16 kout, Rows16 vout) {
  // this workgroup's tokens: their sequences by bisection of cu, their pages from the table
  __shared__ int32_t s_page[kThreads / LPR], s_off[kThreads / LPR];
  const int32_t t0 = blockIdx.x * tokens;
  if (threadIdx.x < static_cast<uint32_t>(tokens)) {
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
  const int ch = threadIdx.x % LPR, r = threadIdx.x / LPR;
  const int tk = r % tokens, h0 = r / tokens, dh = (kThreads / LPR) / tokens;
  const int32_t page = s_page[tk];
  if (8 * ch >= c.D || page == -2) return;
  const bool there = page >= 0;  // a token without a page gives zeros
  const int64_t rowb = kv_row_bytes(MODE, c.D), sb = kv_scale_bytes(MODE, c.D), off = s_off[tk];
  const int64_t first = (static_cast<int64_t>(h0) << c.page_log) + off, t = t0 + tk;
  uint16_t* dst[2] = {kout.p + t * kout.row + h0 * kout.head + 8 * ch, vout.p + t * vout.row + h0 * vout.head + 8 * ch};
  const uint8_t* codes[2] = {c.k.codes + (page * c.k.page_b + first * rowb), c.v.codes + (page * c.v.page_b + first * rowb)};
  const uint8_t* scale[2] = {c.k.scale + (page * c.k.scale_page_b + first * sb), c.v.scale + (page * c.v.scale_page_b + first * sb)};
  const int64_t dst_d[2] = {dh * kout.head, dh * vout.head}, codes_d = (dh * rowb) << c.page_log, scale_d = (dh * sb) << c.page_log;
  for (int h = h0; h < c.Hkv; h += dh * kInFlight) {
    u32x4_t w[2][kInFlight];
    float sc[2][kInFlight];
    uint32_t e8[2][kInFlight];
#pragma unroll
    for (int i = 0; i < kInFlight; ++i)
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        w[side][i] = u32x4_t{0u, 0u, 0u, 0u};
        sc[side][i] = 0.0f;
        e8[side][i] = 0u;
        if (there && h + i * dh < c.Hkv) {
          w[side][i] = kv_load8<MODE>(codes[side] + i * codes_d, ch);
          if constexpr (MODE == kKvFp4)
            e8[side][i] = scale[side][i * scale_d + ch / 4];
          else if constexpr (MODE != kKv16)
            sc[side][i] = *reinterpret_cast<const float*>(scale[side] + i * scale_d);
        }
      }
#pragma unroll
    for (int side = 0; side < 2; ++side) {
#pragma unroll
      for (int i = 0; i < kInFlight; ++i) {
        if (h + i * dh >= c.Hkv) break;
        u32x4_t o = w[side][i];
        if constexpr (MODE != kKv16) {
          float v[8];
          kv_decode8<MODE, DT>(w[side][i], sc[side][i], e8[side][i], v);
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] = round16x2<DT>(v[2 * j], v[2 * j + 1]);
        }
        __builtin_nontemporal_store(o, reinterpret_cast<u32x4_t*>(dst[side] + i * dst_d[side]));
      }
      dst[side] += kInFlight * dst_d[side];
      codes[side] += kInFlight * codes_d;
      scale[side] += kInFlight * scale_d;
    }
  }
}

template <int MODE, int DT>
hipError_t write_mode(const KvCache& c, int64_t T, const Rows16& k, const Rows16& v, const int32_t* slots, float d,
                      float dmax, hipStream_t s) {
  auto go = [&](auto lpr, auto sv) {
    constexpr int L = decltype(lpr)::value, SV = decltype(sv)::value;
    const int tokens = tokens_of(T, c.Hkv, L, kThreads, kEnough);
    kv_write_kernel<MODE, DT, L, SV><<<static_cast<uint32_t>(ceil_div(T, tokens)), kThreads, 0, s>>>(
        c, static_cast<int32_t>(T), tokens, k, v, slots, d, dmax);
  };
  by_lanes(c.D, [&](auto lpr) {
    if constexpr (MODE == kKvFp4) {
      if (dmax != 0.0f) return go(lpr, std::integral_constant<int, kE8V2Div>{});
    }
    go(lpr, std::integral_constant<int, kE8V1>{});
  });
  return hipGetLastError();
}

template <int MODE, int DT>
hipError_t read_mode(const KvCache& c, int64_t T, int32_t B, const BlockTable& bt, const int32_t* cu, const Rows16& k,
                     const Rows16& v, hipStream_t s) {
  by_lanes(c.D, [&](auto lpr) {
    constexpr int L = decltype(lpr)::value;
    const int tokens = tokens_of(T, c.Hkv, L, kThreads, kEnough);
    kv_read_kernel<MODE, DT, L><<<static_cast<uint32_t>(ceil_div(T, tokens)), kThreads, 0, s>>>(c, static_cast<int32_t>(T), B, tokens,
                                                                                              bt, cu, k, v);
  });
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
