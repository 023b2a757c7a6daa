// Queries and keys between the projection and the attention: the root-mean-square norm of each head's row
// (optional), then the rotation of its pairs by the token's position, in one pass; the keys to rows, or with the
// values straight into the paged cache, quantized.
//
//     y = x / sqrt(mean(x^2) + eps) * w;   (a, b) -> (a cos t - b sin t, b cos t + a sin t),   t = position * inv_freq[i]
// for the pairs i of the first R elements: (i, i + R/2), or (2 i, 2 i + 1) interleaved.  Everything is fp32 and rounded
// once, to the rows' type or to the cache's codes (which therefore come from unrounded values).
//
// A lane takes 8 elements and D / 8 lanes (rounded up to 8, 16 or 32) a row; a lane group owns a token and walks its heads.
// So the angles, the only expensive part, are formed once a token and lane: the product with the position in fp64 (exact
// below 2^29), its fraction of a turn in fp64, sine and cosine of that in fp32.  The other element of a pair is R/2 away
// in another lane; its lane reads it too (a second request to lines that the row's own loads bring into the cache).
//
// Bound by HBM: 16384 tokens of 72 heads of 128 in f16 (604 MB there and back) take 130 us, 4.6 TB/s (of 5.2 that a copy reaches);
// pairs side by side, which need no second request, 122.  A token's weights times its cosines and sines are formed once, not once a head (146 us,
// so 141).  Rows go out past the caches, which they only fill: 141 us, so 130; 2048 tokens of 40 heads 18.6, so 15.7.  More
// heads of a token side by side in a wave (its rows lie one behind the other) cost as many more angles: 142 to 174 us.
#include <hip/hip_runtime.h>

#include "fq_kv_store.h"

namespace fq {
namespace {

constexpr int kThreads = 256;
constexpr int kEnough = 512;  // workgroups of a launch that need no more spreading
constexpr int kInFlight = 4;  // heads whose rows are loaded before the first is used
constexpr int kRows = -1;     // the place of a cache mode: keys go to rows, and there are no values

// Sum over aligned groups of SPAN lanes, in an order that does not depend on the lane.
template <int SPAN>
__device__ __forceinline__ float group_sum(float v) {
  v += dpp_f<kDppQuadXor1>(v);
  v += dpp_f<kDppQuadXor2>(v);
  if constexpr (SPAN >= 8) v += dpp_f<kDppRowHalfMirror>(v);
  if constexpr (SPAN >= 16) v += dpp_f<kDppRowMirror>(v);
  if constexpr (SPAN >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

// Eight weights of a norm from element e on (e a multiple of 4; the upper four from e1).
__device__ __forceinline__ void weights8(const RopeNorm& n, int e0, int e1, float (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = i < 4 ? e0 + i : e1 + i - 4;
    w[i] = n.dtype == kNormF32 ? static_cast<const float*>(n.w)[e]
           : n.dtype == kF16   ? load16<kF16>(static_cast<const uint16_t*>(n.w)[e])
                               : load16<kBF16>(static_cast<const uint16_t*>(n.w)[e]);
  }
}

// What a lane's elements have in common over the heads of a token.
struct Turn {
  float c[8], s[8];  // y = x c + other s, the sign of the sine included (weights come to these)
  int o0, o1;        // the others' places in the row, of the lower and the upper four; -1: none (not turned)
};

template <int DT>
__device__ __forceinline__ void widen(const u32x4_t raw, float (&x)[8]) { kv_decode8<kKv16, DT>(raw, 1.0f, 0, x); }

template <int MODE, int DT, int LPR, int SV>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a, int32_t tokens) {
  const int ch = threadIdx.x % LPR, r = threadIdx.x / LPR;  // elements 8 ch .. 8 ch + 7
  const int tk = r % tokens, h0 = r / tokens, dh = (kThreads / LPR) / tokens;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * tokens + tk;
  const bool mine = t < a.T && 8 * ch < a.D;  // (all lanes stay for the sums and maxima)

  Turn tn;
  const int half = a.R / 2;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    tn.c[i] = 1.0f;
    tn.s[i] = 0.0f;
  }
  tn.o0 = tn.o1 = -1;
  auto angle = [&](int i, float& sn, float& cs) __attribute__((always_inline)) {  // of pair i
    const int ax = a.axis ? a.axis[i] : 0;
    const int32_t pos = static_cast<uint32_t>(ax) < static_cast<uint32_t>(a.axes) ? a.pos[ax * a.pos_axis + t] : 0;
    const double turns = static_cast<double>(pos) * static_cast<double>(a.inv_freq[i]) * 0.15915494309189533577;
    sincospif(static_cast<float>(2.0 * (turns - __builtin_rint(turns))), &sn, &cs);
  };
  if (mine) {
    if (a.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (8 * ch + 2 * i >= a.R) break;
        float sn;
        angle(4 * ch + i, sn, tn.c[2 * i]);
        tn.c[2 * i + 1] = tn.c[2 * i];
        tn.s[2 * i] = -sn;
        tn.s[2 * i + 1] = sn;
      }
    } else {
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int e = 8 * ch + 4 * g;
        if (e >= a.R) break;
        const bool low = e < half;
        (g == 0 ? tn.o0 : tn.o1) = low ? e + half : e - half;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float sn;
          angle((low ? e : e - half) + i, sn, tn.c[4 * g + i]);
          tn.s[4 * g + i] = low ? -sn : sn;
        }
      }
    }
  }

  // One row: normed where there are weights, and turned.  `other`: the row's elements at o0 and o1, four each; w, wo: weights times cosines
  // and sines.  (An element that is not turned is left as it is: a zero's sign, and whatever the other one holds.)
  auto turned = [&](const RopeNorm& n, const float (&w)[8], const float (&wo)[8], const u32x4_t raw, const u32x4_t other, float (&y)[8])
                    __attribute__((always_inline)) {
    float x[8], o[8];
    widen<DT>(raw, x);
    if (a.interleaved) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = x[i ^ 1];
    } else {
      widen<DT>(other, o);
    }
    if (n.w) {
      float q = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) q = __builtin_fmaf(x[i], x[i], q);
      const float inv = 1.0f / __builtin_sqrtf(group_sum<LPR>(q) / static_cast<float>(a.D) + a.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] *= inv;
        o[i] *= inv;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = tn.s[i] != 0.0f ? __builtin_fmaf(x[i], w[i], o[i] * wo[i]) : x[i] * w[i];
  };

  // The heads of one side, kInFlight rows at a time; sink(head, values, there).
  auto side = [&](const Rows16& in, int heads, const RopeNorm& n, auto sink) __attribute__((always_inline)) {
    float w[8], wo[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = wo[i] = 1.0f;
    if (n.w && mine) {
      weights8(n, 8 * ch, 8 * ch + 4, w);
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) wo[i] = w[i ^ 1];
      } else {
        weights8(n, max(tn.o0, 0), max(tn.o1, 0), wo);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] *= tn.c[i];
      wo[i] *= tn.s[i];
    }
    const uint16_t* src = in.p + (t * in.row + h0 * in.head);
    const int64_t step = dh * in.head;
    for (int h = h0; h < heads; h += dh * kInFlight) {
      u32x4_t raw[kInFlight], other[kInFlight];
#pragma unroll
      for (int i = 0; i < kInFlight; ++i) {
        raw[i] = other[i] = u32x4_t{0u, 0u, 0u, 0u};
        if (mine && h + i * dh < heads) {
          const uint16_t* const row = src + i * step;
          raw[i] = *reinterpret_cast<const u32x4_t*>(row + 8 * ch);
          if (tn.o0 >= 0) {
            const u32x2_t v = *reinterpret_cast<const u32x2_t*>(row + tn.o0);
            other[i][0] = v[0];
            other[i][1] = v[1];
          }
          if (tn.o1 >= 0) {
            const u32x2_t v = *reinterpret_cast<const u32x2_t*>(row + tn.o1);
            other[i][2] = v[0];
            other[i][3] = v[1];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kInFlight; ++i) {
        if (h + i * dh >= heads) break;
        float y[8];
        turned(n, w, wo, raw[i], other[i], y);
        sink(h + i * dh, y, mine);
      }
      src += kInFlight * step;
    }
  };
  auto to_rows = [&](const Rows16& out) __attribute__((always_inline)) {
    return [&, out](int h, const float (&y)[8], bool there) __attribute__((always_inline)) {
      if (there)
        __builtin_nontemporal_store(u32x4_t{round16x2<DT>(y[0], y[1]), round16x2<DT>(y[2], y[3]), round16x2<DT>(y[4], y[5]), round16x2<DT>(y[6], y[7])},
                                    reinterpret_cast<u32x4_t*>(out.p + (t * out.row + h * out.head + 8 * ch)));
    };
  };

  side(a.q, a.Hq, a.qn, to_rows(a.q_out));
  if constexpr (MODE == kRows) {
    side(a.k, a.Hkv, a.kn, to_rows(a.k_out));
  } else {
    const KvCache& c = a.c;
    const int32_t slot = t < a.T ? a.slots[t] : -1;
    const int32_t page = slot >> c.page_log;  // a negative slot stays negative
    const bool held = page >= 0 && page < c.pages;
    const int64_t rowb = kv_row_bytes(MODE, c.D), sb = kv_scale_bytes(MODE, c.D);
    const int64_t off = slot & ((1 << c.page_log) - 1);
    side(a.k, a.Hkv, a.kn, [&](int h, const float (&y)[8], bool there) __attribute__((always_inline)) {
      const int64_t row = (static_cast<int64_t>(h) << c.page_log) + off;
      kv_store8<MODE, DT, LPR, SV>(y, c.k.codes + (page * c.k.page_b + row * rowb), c.k.scale + (page * c.k.scale_page_b + row * sb), ch,
                                   c.D, a.d, a.dmax, there && held);
    });
    // the values, as the cache's own write stores them
    for (int h = h0; h < a.Hkv; h += dh * kInFlight) {
      u32x4_t raw[kInFlight];
#pragma unroll
      for (int i = 0; i < kInFlight; ++i) {
        raw[i] = u32x4_t{0u, 0u, 0u, 0u};
        if (mine && held && h + i * dh < a.Hkv)
          raw[i] = *reinterpret_cast<const u32x4_t*>(a.v.p + (t * a.v.row + (h + i * dh) * a.v.head + 8 * ch));
      }
#pragma unroll
      for (int i = 0; i < kInFlight; ++i) {
        if (h + i * dh >= a.Hkv) break;
        const int64_t row = (static_cast<int64_t>(h + i * dh) << c.page_log) + off;
        kv_store8<MODE, DT, LPR, SV>(raw[i], c.v.codes + (page * c.v.page_b + row * rowb), c.v.scale + (page * c.v.scale_page_b + row * sb),
                                     ch, c.D, a.d, a.dmax, mine && held);
      }
    }
  }
}

template <int MODE, int DT>
hipError_t go(const RopeArgs& a, hipStream_t s) {
  auto run = [&](auto lpr, auto sv) {
    constexpr int L = decltype(lpr)::value, SV = decltype(sv)::value;
    const int tokens = tokens_of(a.T, a.Hq + (MODE == kRows ? 1 : 2) * a.Hkv, L, kThreads, kEnough);
    rope_kernel<MODE, DT, L, SV><<<static_cast<uint32_t>(ceil_div(a.T, tokens)), kThreads, 0, s>>>(a, tokens);
  };
  by_lanes(a.D, [&](auto lpr) {
    if constexpr (MODE == kKvFp4) {
      if (a.dmax != 0.0f) return run(lpr, std::integral_constant<int, kE8V2Div>{});
    }
    run(lpr, std::integral_constant<int, kE8V1>{});
  });
  return hipGetLastError();
}

template <int DT>
hipError_t by_cache(const RopeArgs& a, hipStream_t s) {
  if (!a.append) return go<kRows, DT>(a, s);
  switch (a.c.mode) {
    case kKv16: return go<kKv16, DT>(a, s);
    case kKvInt8: return go<kKvInt8, DT>(a, s);
    case kKvE4M3: return go<kKvE4M3, DT>(a, s);
    case kKvInt4: return go<kKvInt4, DT>(a, s);
    default: return go<kKvFp4, DT>(a, s);
  }
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t s) { return a.dtype == kF16 ? by_cache<kF16>(a, s) : by_cache<kBF16>(a, s); }

}  // namespace fq
