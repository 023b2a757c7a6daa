// Attention of new tokens over the paged cache: the kernels, instantiated by cache format in fq_attn_chunk_*.hip.
//
// Sequence b has the query rows cu_q[b] .. cu_q[b+1]-1, its newest tokens, whose keys and values the cache holds already
// among its lengths[b] tokens.  Row i sees the keys up to its own position, with a window only the last W of them and
// the first S: o = sum_j p_j v_j, p = softmax over the visible keys of scale * <q, k_j>.
//
// A workgroup of four waves takes 128 query rows, 32 a wave: the g query heads of one cache head for 128 / g
// neighbouring tokens (a cached byte is read once for all of them), and walks the keys in tiles of 64 as the prompt
// kernel does: two LDS buffers, S^T = K Q^T and O^T = V^T P^T with 32 x 32 x 16 products, a lane owning one row's
// statistics, the maximum moved only when a score passes m + 8 in base-2 units.  LDS layouts as there.
// A tile's keys lie in pages of 16 tokens at least: each wave brings the 16 rows that are one page's (16 bits by LDS-DMA).
//
// Low-bit formats: the codes go through registers, are widened to f16 numbers there, exactly, and written to LDS;
// a tile's bytes are widened once for all 128 rows.  Widened: int8 and int4 the code times 2^-9, E4M3 the code, E2M1 the code
// times its group's power of two over the row's largest, times 2^13 (a group more than 2^26 below the largest of its
// row loses bits).  So every format has one factor a row: a key's multiplies its scores, a value's its weights, both in fp32 out of
// LDS.  A bf16 q is brought to f16 by a power of two a row (28 binades below its largest element keep all bits).
// Weights times value scales go to f16 relative to a reference exponent R, a row's own: w = exp2(s - m - R + 5) scale, where
// R is at least the exponent of the scales seen, less one (w stays below 2^15).  The sum l is of exp2(s - m - R + 5), so the
// quotient needs neither; m + R is what the parts of a walk are joined by.
//
// Split: every (sequence, cache head, row tile) is a segment of key tiles; all segments one after the other are dealt to
// the grid in equal runs.  A segment's place in that order has a closed form in its tile number (its walk's
// length is linear in it, up to the window), so a run finds its first segment by a scan over the sequences and a
// bisection.  A run that has a segment in part leaves its sums in the workspace, at most two such parts a run,
// and a second launch joins them in order.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>

#include "fq_attn_tile.h"

namespace fq {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kRows = 32 * kWaves;  // query rows of a workgroup
constexpr int kKeys = 64;           // keys of a tile
constexpr int kStart = 2;           // tiles that a segment's beginning and end count as when the work is dealt
constexpr int kAhead = 4;           // fragments read ahead of their products
constexpr float kLazy = 8.0f;

template <int MODE>
constexpr int kCodeBits = MODE == kKv16 ? 16 : (MODE == kKvInt8 || MODE == kKvE4M3) ? 8 : 4;
// a key's and a value's operand for 1 (E2M1: the keys' is in their factors)
template <int MODE>
constexpr float kUnitK = MODE == kKvInt8 || MODE == kKvInt4 ? 512.0f : 1.0f;
template <int MODE>
constexpr float kUnitV = MODE == kKvFp4 ? 0x1p-13f : kUnitK<MODE>;
// The reference R lies between these.  From kLeastRef on a walk's 2^31 weights sum below 2^127; up to kMostRef a weight of 1 is
// well within fp32's normal numbers.
constexpr int kLeastRef = -82, kMostRef = 120;
// weights enter the second product 2^kUpW times above the row's reference
template <int MODE, int DT>
constexpr float kUpW = MODE == kKv16 ? kUp<DT> : 5.0f;

// ---- the plan ------------------------------------------------------------------------------

struct Seq {
  int q0, lq, lk, off;  // its first row and rows (tokens), its keys, keys ahead of the first row
  int tiles, places;    // row tiles, and what one head's count for
};

// Places of a sequence's row tiles before tile j, in key tiles: the sums of spans in tokens, over 64, rounded down.  A
// tile's span: kStart + 1 tiles, the whole tiles of the first tokens, and the keys up to behind its last token (at most
// behind the last key) or what a window of all its tokens can touch.  (So that it has a place for each of its key tiles.)
// With a workgroup a segment it is one place.
__device__ __forceinline__ int places_before(const ChunkArgs& a, int off, int lk, int j) {
  if (a.single) return j;
  const int64_t a0 = max(off, 0), R = a.tokens;
  int64_t cap = lk + R, more = (kStart + 1) * kKeys;
  if (a.window > 0) {
    cap = min(cap, static_cast<int64_t>(a.window) + R + 126);
    more += (a.sinks + kKeys - 1) / kKeys * static_cast<int64_t>(kKeys);
  }
  const int64_t n = cap > a0 ? min(static_cast<int64_t>(j), static_cast<int64_t>(static_cast<uint32_t>(cap - a0) / static_cast<uint32_t>(a.tokens))) : 0;
  return static_cast<int>((n * a0 + R * (n * (n + 1) / 2) + (j - n) * cap + j * more) >> 6);
}

__device__ __forceinline__ Seq seq_of(const ChunkArgs& a, int b) {
  Seq s{0, 0, 0, 0, 0, 0};
  if (b < a.B) {
    s.q0 = max(0, min(a.cu_q[b], a.Tq));
    s.lq = max(0, min(a.cu_q[b + 1], a.Tq) - s.q0);
    s.lk = max(0, min(a.lengths[b], a.reach));
    s.off = s.lk - s.lq;
    s.tiles = (s.lq + a.tokens - 1) / a.tokens;
    s.places = places_before(a, s.off, s.lk, s.tiles);
  }
  return s;
}
__device__ __forceinline__ Seq lane_seq(const Seq& s, int w) {  // a lane's, for the whole wave
  return Seq{__builtin_amdgcn_readlane(s.q0, w),  __builtin_amdgcn_readlane(s.lq, w),    __builtin_amdgcn_readlane(s.lk, w),
             __builtin_amdgcn_readlane(s.off, w), __builtin_amdgcn_readlane(s.tiles, w), __builtin_amdgcn_readlane(s.places, w)};
}

// Run i of `runs` (at most `most`) has the places from start(i) up to start(i + 1).
struct Deal {
  uint32_t total, runs, q, r;
  __device__ Deal(uint32_t places, uint32_t most) : total(places), runs(min(places, most)) {
    q = runs ? total / runs : 0u;
    r = total - q * runs;
  }
  __device__ int start(uint32_t i) const { return static_cast<int>(i * q + i * r / runs); }
};

// All places (wave by wave, no barrier).
__device__ __forceinline__ int all_places(const ChunkArgs& a) {
  const int lane = threadIdx.x & 63;
  int total = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) total += __builtin_amdgcn_readlane(wave_scan(seq_of(a, b0 + lane).places), 63) * a.heads;
  return total;
}

// A segment: a row tile of one (sequence, cache head and heads' tile), and the first of its places.
struct Segment {
  Seq s;
  int b, head, tile, at;
};

// The segment that holds place x (below all of them).
__device__ __forceinline__ Segment segment_at(const ChunkArgs& a, int x) {
  const int lane = threadIdx.x & 63;
  Segment g;
  int before = 0;
  for (int b0 = 0;; b0 += 64) {
    const Seq s = seq_of(a, b0 + lane);
    const int incl = wave_scan(s.places) * a.heads;
    const uint64_t holds = __ballot(before + incl > x);
    if (holds == 0 && b0 + 64 < a.B) {
      before += __builtin_amdgcn_readlane(incl, 63);
      continue;
    }
    const int w = __builtin_ctzll(holds | (uint64_t(1) << 63));
    g.s = lane_seq(s, w);
    g.b = b0 + w;
    g.at = before + __builtin_amdgcn_readlane(incl - s.places * a.heads, w);
    break;
  }
  const int p = max(1, g.s.places);
  g.head = min((x - g.at) / p, a.heads - 1);
  g.at += g.head * p;
  int lo = 0, hi = max(1, g.s.tiles);  // the tile's first place is at or before x, that of tile hi behind it
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (g.at + places_before(a, g.s.off, g.s.lk, mid) <= x) lo = mid; else hi = mid;
  }
  g.tile = lo;
  g.at += places_before(a, g.s.off, g.s.lk, lo);
  return g;
}

// The key tiles that a row tile walks: the first `sinks` ones, then those from `lo` on; n in all.
struct Walk {
  int row0, row1;  // its first and last token
  int n, sinks, lo;
  __device__ int tile(int u) const { return u < sinks ? u : lo + u - sinks; }
};
__device__ __forceinline__ Walk walk_of(const ChunkArgs& a, const Seq& s, int tile) {
  Walk w;
  w.row0 = tile * a.tokens;
  w.row1 = min(w.row0 + a.tokens, s.lq) - 1;
  const int last = s.off + w.row1;  // the last key that is seen
  w.sinks = w.lo = 0;
  w.n = 0;
  if (last < 0) return w;
  if (a.window > 0) {
    w.sinks = (min(a.sinks, last + 1) + kKeys - 1) / kKeys;
    w.lo = max(w.sinks, max(0, s.off + w.row0 - a.window + 1) / kKeys);
  }
  w.n = w.sinks + last / kKeys + 1 - w.lo;
  return w;
}

// ---- codes to f16 operands -------------------------------------------------------------------

// Eight int4 codes (two's complement, low nibble first) -> f16 values code 2^-9, in order: each byte goes to both halves of
// a dword, one nibble of it is kept in each (16 times as much in the upper), and both are brought to the same unit.
__device__ __forceinline__ u32x4_t int4_to_f16(uint32_t w) {
  typedef __attribute__((ext_vector_type(2))) _Float16 h16x2;
  const h16x2 up = __builtin_bit_cast(h16x2, 0x68007800u), minus = __builtin_bit_cast(h16x2, kMinus8);  // 2^11, 2^15
  const uint32_t x = w ^ 0x88888888u;
  u32x4_t o;
  const uint32_t b[4] = {__builtin_amdgcn_perm(0u, x, 0x0C000C00u), __builtin_amdgcn_perm(0u, x, 0x0C010C01u),
                         __builtin_amdgcn_perm(0u, x, 0x0C020C02u), __builtin_amdgcn_perm(0u, x, 0x0C030C03u)};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(h16x2, b[i] & 0x00F0000Fu), up, minus));
  return o;
}

// Elements 8 e .. 8 e + 7 of a piece; s: the E2M1 group's factor.
template <int MODE, int W>
__device__ __forceinline__ u32x4_t widened(const uint32_t (&w)[W], int e, float s) {
  if constexpr (MODE == kKvInt8) {
    const uint32_t a = w[2 * e] ^ 0x80808080u, b = w[2 * e + 1] ^ 0x80808080u;
    return u32x4_t{unbias_f16(__builtin_amdgcn_perm(0u, a, 0x0C010C00u), kMinus128), unbias_f16(__builtin_amdgcn_perm(0u, a, 0x0C030C02u), kMinus128),
                   unbias_f16(__builtin_amdgcn_perm(0u, b, 0x0C010C00u), kMinus128), unbias_f16(__builtin_amdgcn_perm(0u, b, 0x0C030C02u), kMinus128)};
  } else if constexpr (MODE == kKvE4M3) {
    return u32x4_t{fp8_to_f16x2<false>(w[2 * e]), fp8_to_f16x2<true>(w[2 * e]), fp8_to_f16x2<false>(w[2 * e + 1]), fp8_to_f16x2<true>(w[2 * e + 1])};
  } else if constexpr (MODE == kKvInt4) {
    return int4_to_f16(w[e]);
  } else {
    return u32x4_t{fp4_to_f16x2<0>(w[e], s), fp4_to_f16x2<1>(w[e], s), fp4_to_f16x2<2>(w[e], s), fp4_to_f16x2<3>(w[e], s)};
  }
}
constexpr int kUpE = 13, kLeastE = 46;  // E2M1: a row's largest group goes in 2^kUpE up; below kLeastE it counts as that

template <int W>
__device__ __forceinline__ void load_piece(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t (&o)[W]) {
  if constexpr (W == 4) {
    const u32x4_t x = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = x[i];
  } else if constexpr (W == 2) {
    const u32x2_t x = __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0);
    o[0] = x[0];
    o[1] = x[1];
  } else {
    o[0] = __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
  }
}

// Max over aligned groups of SPAN lanes (4, 8, 16 or 32).
template <int SPAN>
__device__ __forceinline__ int lanes_max(int v) {
  v = max(v, static_cast<int>(dpp_u<kDppQuadXor1>(v)));
  v = max(v, static_cast<int>(dpp_u<kDppQuadXor2>(v)));
  if constexpr (SPAN >= 8) v = max(v, static_cast<int>(dpp_u<kDppRowHalfMirror>(v)));
  if constexpr (SPAN >= 16) v = max(v, static_cast<int>(dpp_u<kDppRowMirror>(v)));
  if constexpr (SPAN >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(static_cast<int>(r[0]), static_cast<int>(r[1]));
  }
  return v;
}

// What of a tile's low-bit rows one wave brings: its 16 rows' pieces and scales of both sides.
template <int MODE, int DP, bool PAD>
struct Low {
  static constexpr int bits = kCodeBits<MODE>;
  static constexpr int CE = PAD ? 8 : (128 / bits < DP / 4 ? 128 / bits : DP / 4);  // elements of a piece
  static constexpr int LPR = DP / CE;         // lanes of a row
  static constexpr int N = 16 * LPR / 64;     // pieces of a lane and side
  static constexpr int W = CE * bits / 32;    // dwords of a piece
  uint32_t w[2][N][W];
  uint32_t e8[2][MODE == kKvFp4 ? N : 1];
  float scale[2];  // of row lane % 16
};

// ---- the walk ----------------------------------------------------------------------------------

template <int MODE, int DT, int DP, bool PAD>
__global__ __launch_bounds__(kThreads, DP == 256 ? 1 : 2) void chunk_kernel(ChunkArgs a, float* __restrict__ ws) {
  constexpr bool kLow = MODE != kKv16;
  constexpr int ODT = kLow ? kF16 : DT;  // the operands' type
  constexpr bool kOdd = MODE == kKv16 || MODE == kKvFp4;  // values may be infinite or NaN one by one
  constexpr float kW = kUpW<MODE, DT>;
  constexpr int KS = DP / 16;            // products of a score block
  constexpr int DB = DP / 32;            // 32-row blocks of O^T
  constexpr int kRowB = DP * 2;          // bytes of a tile row
  constexpr int kTileB = kKeys * kRowB;  // bytes of a tile (keys or values)
  constexpr int kPieces = DP / 8;        // 16-byte pieces of a row
  constexpr int NL = kTileB / 1024 / kWaves;
  using L = Low<kLow ? MODE : kKvInt8, DP, PAD>;
  __shared__ __align__(16) uint8_t lds[4 * kTileB];  // buffer b: keys at 2 b, values at 2 b + 1
  __shared__ __align__(16) float s_scale[kLow ? 2 : 1][2][kLow ? kKeys : 1];  // [buffer][keys, values]
  __shared__ __align__(16) float s_top[kLow ? 2 : 1][kWaves];                 // largest value scale of 16 keys
  const lds_u8* const lds_l = (const lds_u8*)lds;
  const uint32_t lds_addr = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds_l));

  const KvCache& cc = a.c;
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 31, hf = lane >> 5;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int D = PAD ? cc.D : DP;
  const int rowb = static_cast<int>(kv_row_bytes(MODE, D)), sb = static_cast<int>(kv_scale_bytes(MODE, D));

  // ---- this workgroup's run (neighbouring runs, which share keys, on one XCD's L2)
  const Deal deal(all_places(a), a.single ? ~0u : a.runs);
  const int per_xcd = (deal.runs + 7) / 8, run = static_cast<int>(blockIdx.x & 7) * per_xcd + static_cast<int>(blockIdx.x >> 3);
  if (static_cast<int>(blockIdx.x >> 3) >= per_xcd || run >= static_cast<int>(deal.runs)) return;
  const int first = deal.start(run), last = deal.start(run + 1);
  Segment sg = segment_at(a, first);

  // LDS-DMA of 16-bit rows: load i of a wave fills the 16-byte places 64 (NL w + i) + lane of a tile, its 16 rows in all
  uint32_t koff[NL], voff[NL];
  if constexpr (!kLow) {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int at = 64 * (NL * wv + i) + lane, r = at / kPieces, p = at % kPieces;
      const int kp = p ^ (DP == 64 ? (r >> 1) & 7 : r & 15), vp = p ^ (4 * (DP == 64 ? (r >> 1) & 1 : r & 3));
      koff[i] = !PAD || 8 * kp < D ? static_cast<uint32_t>((r & 15) * rowb + 16 * kp) : kOut;
      voff[i] = !PAD || 8 * vp < D ? static_cast<uint32_t>((r & 15) * rowb + 16 * vp) : kOut;
    }
  }
  int step = 0;  // of this workgroup; tile of step s is in buffer s % 2

  for (;;) {
    const Walk wk = walk_of(a, sg.s, sg.tile);
    const int base = sg.at + kStart;  // the place of the segment's first key tile
    const int u0 = a.single ? 0 : min(wk.n, max(0, first - base)), u1 = a.single ? wk.n : max(u0, min(wk.n, last - base));
    const bool whole = wk.n == 0 ? sg.at >= first && sg.at < last : u0 == 0 && u1 == wk.n;
    if (whole || u0 < u1) {
      const int hk = sg.head / a.head_tiles, ht = sg.head - hk * a.head_tiles;
      const int hn = min(a.tile_heads, a.g - ht * a.tile_heads);  // heads of this tile
      const int lk = sg.s.lk, off = sg.s.off;
      // this lane's row: a token of the sequence and a head (rows past the last token or head repeat it)
      const int row = 32 * wv + col;
      const int tok = wk.row0 + row / a.tile_heads, hr = row % a.tile_heads;
      const bool mine = tok <= wk.row1 && row < a.tokens * a.tile_heads && hr < hn;
      const int token = min(tok, wk.row1), head = hk * a.g + ht * a.tile_heads + min(hr, hn - 1);
      auto token_of = [&](int r) __attribute__((always_inline)) { return min(wk.row0 + r / a.tile_heads, wk.row1); };
      const int first_tok = token_of(32 * wv), last_tok = token_of(32 * wv + 31);
      // keys that this lane's row sees: from lo up to lim, and below the sinks
      const int lim = off + token;
      const int lim_first = off + first_tok, lim_last = off + last_tok;
      auto low_of = [&](int l) __attribute__((always_inline)) { return a.window > 0 ? max(0, l - a.window + 1) : 0; };
      const int lo = low_of(lim), lo_first = low_of(lim_first), lo_last = low_of(lim_last);

      // ---- the query rows as B operands (a negative scale goes into their sign); c: base-2 scores' factor
      float c = __builtin_fabsf(a.scale) * 1.44269504f;
      u32x4_t qf[KS];
      {
        const uint16_t* qp = a.q.p + (sg.s.q0 + token) * a.q.row + head * a.q.head;
        const uint32_t sign = a.scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const int d = 16 * ks + 8 * hf;
          qf[ks] = u32x4_t{0u, 0u, 0u, 0u};
          if (!PAD || d < D) qf[ks] = *reinterpret_cast<const u32x4_t*>(qp + d);
          qf[ks] ^= u32x4_t{sign, sign, sign, sign};
        }
        if constexpr (kLow && DT == kBF16) {
          uint32_t top = 0;  // the largest exponent, in place
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int i = 0; i < 4; ++i) top = max(top, max(qf[ks][i] & 0x7F800000u, (qf[ks][i] << 16) & 0x7F800000u));
          const int e = min(static_cast<int>(__float_as_uint(half_max(__uint_as_float(top))) >> 23), 254) - 127;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              qf[ks][i] = round16x2<kF16>(__builtin_amdgcn_ldexpf(__uint_as_float(qf[ks][i] << 16), 14 - e),
                                          __builtin_amdgcn_ldexpf(__uint_as_float(qf[ks][i] & 0xFFFF0000u), 14 - e));
          c = __builtin_amdgcn_ldexpf(c, e - 14);
        }
        c = fminf(fmaxf(c * kUnitK<MODE>, 0x1p-126f), 0x1.fffffep127f);  // (a hidden score is -infinity times it)
      }

      // ---- the pages of 16 tiles at a time: lane 4 i + w has that of the w-th 16 keys of the i-th of them
      int pages = -1, pages_u = -(1 << 30);
      uint64_t there = 0;
      auto fetch_pages = [&](int u) __attribute__((always_inline)) {
        const int i = u + (lane >> 2);
        const int t = i < wk.n ? wk.tile(i) * kKeys + 16 * (lane & 3) : a.reach;
        pages = t < lk ? kv_page(a.bt, sg.b, t, cc.page_log, cc.pages) : -1;
        there = __ballot(pages >= 0 || t >= lk);
        pages_u = u;
      };
      auto rows_of = [&](int u) __attribute__((always_inline)) {
        return __builtin_amdgcn_readfirstlane(max(0, min(16, lk - (wk.tile(u) * kKeys + 16 * wv))));
      };
      auto row_of = [&](int u) __attribute__((always_inline)) {
        return (static_cast<int64_t>(hk) << cc.page_log) + ((wk.tile(u) * kKeys + 16 * wv) & ((1 << cc.page_log) - 1));
      };
      auto dma = [&](int u, int buf) __attribute__((always_inline)) {
        if (u >= pages_u + 16 || u < pages_u) fetch_pages(u);
        const int64_t pg = __builtin_amdgcn_readlane(pages, 4 * (u - pages_u) + wv);
        const uint32_t bytes = pg < 0 ? 0u : static_cast<uint32_t>(rows_of(u) * rowb);
        const int64_t at = max(pg, int64_t(0)), r = row_of(u) * rowb;
        const i32x4_t rk = rsrc4(cc.k.codes + (at * cc.k.page_b + r), bytes), rv = rsrc4(cc.v.codes + (at * cc.v.page_b + r), bytes);
        const uint32_t to = lds_addr + buf * (2 * kTileB) + 1024 * NL * wv;
#pragma unroll
        for (int i = 0; i < NL; ++i) dma16(to + 1024 * i, koff[i], rk);
#pragma unroll
        for (int i = 0; i < NL; ++i) dma16(to + kTileB + 1024 * i, voff[i], rv);
      };
      auto load_low = [&](int u, L& x) __attribute__((always_inline)) {
        if (u >= pages_u + 16 || u < pages_u) fetch_pages(u);
        const int pg = __builtin_amdgcn_readlane(pages, 4 * (u - pages_u) + wv), rows = rows_of(u);
        const int64_t at = max(pg, 0), r = row_of(u);
#pragma unroll
        for (int side = 0; side < 2; ++side) {
          const KvSide& sd = side ? cc.v : cc.k;
          const auto rc = __builtin_amdgcn_make_buffer_rsrc(sd.codes + (at * sd.page_b + r * rowb), static_cast<int16_t>(0),
                                                            pg < 0 ? 0 : rows * rowb, kBufferWord3);
          const auto rs = __builtin_amdgcn_make_buffer_rsrc(sd.scale + (at * sd.scale_page_b + r * sb), static_cast<int16_t>(0),
                                                            pg < 0 ? 0 : rows * sb, kBufferWord3);
#pragma unroll
          for (int i = 0; i < L::N; ++i) {
            const int rr = (64 * i + lane) / L::LPR, p = (64 * i + lane) % L::LPR;
            const bool in = !PAD || L::CE * p < D;
            load_piece<L::W>(rc, in ? static_cast<uint32_t>(rr * rowb + p * (L::CE * L::bits / 8)) : kOut, x.w[side][i]);
            if constexpr (MODE == kKvFp4)
              x.e8[side][i] = __builtin_amdgcn_raw_buffer_load_b8(rs, in ? static_cast<uint32_t>(rr * sb + L::CE * p / 32) : kOut, 0, 0);
          }
          if constexpr (MODE != kKvFp4) x.scale[side] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, 4 * (lane & 15), 0, 0));
        }
      };
      // the wave's rows, widened, and their factors to buffer `buf`
      auto store_low = [&](const L& x, int buf) __attribute__((always_inline)) {
        float big = 0.0f;  // of this lane's value scales
#pragma unroll
        for (int side = 0; side < 2; ++side) {
#pragma unroll
          for (int i = 0; i < L::N; ++i) {
            const int rr = (64 * i + lane) / L::LPR, p = (64 * i + lane) % L::LPR, r = 16 * wv + rr;
            float s = 1.0f;
            bool nan = false;
            if constexpr (MODE == kKvFp4) {
              const int e = static_cast<int>(x.e8[side][i]);
              nan = e == 255;
              const int top = max(kLeastE, lanes_max<L::LPR>(nan ? 0 : e));
              s = pow2(max(e - top + kUpE, -126));
              float f = pow2(top - 127 - (side == 0 ? kUpE : 0));
              if (side == 0) {
                if (lanes_max<L::LPR>(nan ? 1 : 0)) f = __builtin_nanf("");
              } else {
                big = fmaxf(big, f);
              }
              if (p == 0) s_scale[buf][side][r] = f;
            }
            uint8_t* const to = lds + (buf * 2 + side) * kTileB + r * kRowB;
            const int sw = side == 0 ? (DP == 64 ? (r >> 1) & 7 : r & 15) : 4 * (DP == 64 ? (r >> 1) & 1 : r & 3);
#pragma unroll
            for (int e = 0; e < L::CE / 8; ++e) {
              u32x4_t o = widened<MODE>(x.w[side][i], e, s);
              if (MODE == kKvFp4 && side == 1 && nan) o = u32x4_t{0x7E007E00u, 0x7E007E00u, 0x7E007E00u, 0x7E007E00u};
              *reinterpret_cast<u32x4_t*>(to + 16 * (((L::CE / 8) * p + e) ^ sw)) = o;
            }
          }
          if constexpr (MODE != kKvFp4) {
            if (lane < 16) s_scale[buf][side][16 * wv + lane] = x.scale[side];
            if (side == 1) big = __builtin_fabsf(x.scale[1]) < kInf ? __builtin_fabsf(x.scale[1]) : 0.0f;  // (neither infinity nor NaN)
          }
        }
        big = fmaxf(big, dpp_f<kDppQuadXor1>(big));
        big = fmaxf(big, dpp_f<kDppQuadXor2>(big));
        big = fmaxf(big, dpp_f<kDppRowHalfMirror>(big));
        big = fmaxf(big, dpp_f<kDppRowMirror>(big));
        if constexpr (MODE == kKvFp4) big = fmaxf(half_max(big), __shfl_xor(half_max(big), 16));
        if (lane == 0) s_top[buf][wv] = big;
      };

      const uint32_t krd = col * kRowB, kx = hf ^ (DP == 64 ? (col >> 1) & 7 : col & 15);
      const int rj = (lane & 15) >> 2;
      const uint32_t vrd = (4 * hf + rj) * kRowB + 32 * ((lane >> 4) & 1) + 8 * (lane & 3), vx = DP == 64 ? rj >> 1 : rj;

      f32x16_t acc[DB];
      float m, l;
      int ref;  // R
      auto walk = [&](auto careful) __attribute__((always_inline)) {
        constexpr bool CAREFUL = decltype(careful)::value;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[d][i] = 0.0f;
        m = -kInf;
        l = 0.0f;
        ref = kLow ? kLeastRef : 0;
        L x;
        if (u0 < u1) {
          if constexpr (kLow) {
            load_low(u0, x);
            store_low(x, step & 1);
          } else {
            dma(u0, step & 1);
          }
        }
        for (int u = u0; u < u1; ++u, ++step) {
          const int buf = step & 1, t = wk.tile(u);
          const uint32_t in = static_cast<uint32_t>(there >> (4 * (u - pages_u))) & 15u;  // which 16 keys have a page
          tile_barrier();
          if (u + 1 < u1) {
            if constexpr (kLow)
              load_low(u + 1, x);
            else
              dma(u + 1, buf ^ 1);
          }
          const int k0 = t * kKeys;
          // (waves none of whose rows sees the tile go on)
          if (k0 <= lim_last && (k0 + kKeys > lo_first || k0 < a.sinks)) {
            const lds_u8* const kt = lds_l + buf * (2 * kTileB);
            const lds_u8* const vt = kt + kTileB;
            auto key = [&](int ks, int b) __attribute__((always_inline)) {
              return *(const __attribute__((address_space(3))) u32x4_t*)(kt + krd + 16 * (kx ^ (2 * ks)) + b * 32 * kRowB);
            };
            auto value = [&](int d, int g) __attribute__((always_inline)) {
              const lds_u8* const p = vt + vrd + 64 * (d ^ vx) + 16 * g * kRowB;
              const u32x2_t lo2 = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)p));
              const u32x2_t hi2 = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(p + 8 * kRowB)));
              return u32x4_t{lo2[0], lo2[1], hi2[0], hi2[1]};
            };
            // a row factor of the keys of accumulator registers 4 j .. 4 j + 3 of block b
            auto factors = [&](int side, int b, int j) __attribute__((always_inline)) {
              return *reinterpret_cast<const f32x4_t*>(&s_scale[buf][side][32 * b + 8 * j + 4 * hf]);
            };
            f32x16_t s[2];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
              for (int i = 0; i < 16; ++i) s[b][i] = 0.0f;
            {
              u32x4_t kf[2 * KS];
#pragma unroll
              for (int i = 0; i < kAhead; ++i) kf[i] = key(i / 2, i % 2);
              static_for<0, 2 * KS>([&](auto ic) __attribute__((always_inline)) {
                constexpr int i = decltype(ic)::value;
                if constexpr (i + kAhead < 2 * KS) kf[i + kAhead] = key((i + kAhead) / 2, (i + kAhead) % 2);
                __builtin_amdgcn_sched_barrier(0);
                s[i % 2] = mfma32x32x16<ODT>(kf[i], qf[i / 2], s[i % 2]);
                __builtin_amdgcn_sched_barrier(0);
              });
            }
            f32x4_t vs[kLow ? 8 : 1];
            if constexpr (kLow) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const f32x4_t f = factors(0, j / 4, j % 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) s[j / 4][4 * (j % 4) + i] *= f[i];
                vs[j] = factors(1, j / 4, j % 4);
              }
            }
            u32x4_t vf[4 * DB];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) vf[i] = value(i % DB, i / DB);
            __builtin_amdgcn_sched_barrier(0);
            const bool masked = k0 + kKeys - 1 > lim_first || (k0 < lo_last && k0 + kKeys > a.sinks) || in != 15u;
            if (masked) {
              // this lane's places (4 hf less than the key in the tile): seen up to `left`, and from `from` on or below `sk`
              const int left = lim - k0 - 4 * hf, from = lo - k0 - 4 * hf, sk = a.sinks - k0 - 4 * hf;
#pragma unroll
              for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const int place = 32 * b + 8 * (i / 4) + i % 4;
                  const bool seen = place <= left && (place >= from || place < sk) && ((in >> (2 * b + i / 8)) & 1u);
                  if (!seen) {
                    s[b][i] = -kInf;
                    if constexpr (kLow) vs[4 * b + i / 4][i % 4] = 0.0f;
                  }
                }
            }
            uint64_t seen = 0;  // CAREFUL: keys of the tile with a score above -infinity for this lane's row
            if constexpr (CAREFUL) {
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                uint32_t w = 0;
#pragma unroll
                for (int i = 0; i < 16; ++i) w |= (s[b][i] > -kInf ? 1u : 0u) << (8 * (i / 4) + i % 4);
                w <<= 4 * hf;
                w |= __shfl_xor(w, 32);
                seen |= static_cast<uint64_t>(w) << (32 * b);
              }
            }
            float top = s[0][0];
#pragma unroll
            for (int i = 1; i < 32; ++i) top = fmaxf(top, s[i / 16][i % 16]);
            int ev = kLeastRef;  // exponent of the largest value scale that is seen
            if constexpr (kLow) {
              float big;
              if (masked) {
                big = 0.0f;
#pragma unroll
                for (int j = 0; j < 32; ++j) big = fmaxf(big, __builtin_fabsf(vs[j / 4][j % 4]) < kInf ? __builtin_fabsf(vs[j / 4][j % 4]) : 0.0f);
              } else {
                const f32x4_t q = *reinterpret_cast<const f32x4_t*>(s_top[buf]);
                big = fmaxf(fmaxf(q[0], q[1]), fmaxf(q[2], q[3]));
              }
              ev = static_cast<int>(__float_as_uint(big) >> 23) - 127;
            }
            if (__any(top * c > m + kLazy || (kLow && ev > ref + 1))) {
              const float mn = fmaxf(m, half_max(top) * c);
              int rn = ref;
              if constexpr (kLow) {
                const auto r = __builtin_amdgcn_permlane32_swap(ev, ev, false, false);
                rn = max(ref, min(kMostRef, max(static_cast<int>(r[0]), static_cast<int>(r[1]))));
              }
              const float to = mn + static_cast<float>(rn), from = m + static_cast<float>(ref);
              const float f = mn == -kInf ? 1.0f : CAREFUL ? rescale(from, to) : __builtin_amdgcn_exp2f(from - to);
              m = mn;
              ref = rn;
              l *= f;
#pragma unroll
              for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[d][i] *= f;
            }
            const float ms = m == -kInf ? 0.0f : m + static_cast<float>(ref) - kW;
            u32x4_t pf[4];
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int e = 8 * (g % 2) + 2 * i;
                float x0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[g / 2][e], c, -ms));
                float x1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[g / 2][e + 1], c, -ms));
                l += x0 + x1;
                if constexpr (kLow) {
                  x0 *= vs[4 * (g / 2) + e / 4][e % 4];
                  x1 *= vs[4 * (g / 2) + e / 4][e % 4 + 1];
                }
                pf[g][i] = round16x2<ODT>(x0, x1);
              }
            __builtin_amdgcn_sched_barrier(0);
            uint32_t odd = 0;
            static_for<0, 4 * DB>([&](auto ic) __attribute__((always_inline)) {
              constexpr int i = decltype(ic)::value;
              if constexpr (i + kAhead < 4 * DB) vf[i + kAhead] = value((i + kAhead) % DB, (i + kAhead) / DB);
              if constexpr (CAREFUL) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  odd |= not_finite16<ODT>(vf[i][j]);
                  vf[i][j] &= ~not_finite16_mask<ODT>(vf[i][j]);
                }
              }
              __builtin_amdgcn_sched_barrier(0);
              acc[i % DB] = mfma32x32x16<ODT>(vf[i], pf[i / DB], acc[i % DB]);
              __builtin_amdgcn_sched_barrier(0);
            });
            if constexpr (CAREFUL) {
              const bool any = __any(odd != 0);
              for (int j = 0; any && j < kKeys; ++j) {
                if (!((seen >> j) & 1)) continue;
#pragma unroll
                for (int d = 0; d < DB; ++d)
#pragma unroll
                  for (int i = 0; i < 16; ++i) {
                    const int e = 32 * d + 8 * (i / 4) + 4 * hf + i % 4;
                    const uint16_t v = *(const __attribute__((address_space(3))) uint16_t*)(
                        vt + j * kRowB + 16 * ((e / 8) ^ (4 * (DP == 64 ? (j >> 1) & 1 : j & 3))) + 2 * (e % 8));
                    if (not_finite16<ODT>(v)) acc[d][i] += load16<ODT>(v);
                  }
              }
            }
          }
          if constexpr (kLow) {
            if (u + 1 < u1) store_low(x, buf ^ 1);
          }
        }
      };
      walk(std::false_type{});
      if constexpr (kOdd) {
        float odd = 0.0f;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) odd = __builtin_fmaf(acc[d][i], 0.0f, odd);
        if (__syncthreads_or(odd != odd)) walk(std::true_type{});
      }
      // (no barrier here: the next segment's first tile takes the buffer that was last read a step before the last one)

      l = half_sum(l);
      if (!whole) {  // the part's sums as they are, [element][row], with m + R and l
        float* const o = ws + static_cast<int64_t>(2 * run + (u0 == 0 ? 1 : 0)) * ((DP + 2) * kRows) + row;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[(32 * d + 8 * (i / 4) + 4 * hf + i % 4) * kRows] = acc[d][i];
        if (hf == 0) {
          o[DP * kRows] = m + static_cast<float>(ref);
          o[(DP + 1) * kRows] = l;
        }
      } else if (mine) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int64_t to = sg.s.q0 + token;
        uint16_t* const out = a.out.p + to * a.out.row + head * a.out.head;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = 32 * d + 8 * i + 4 * hf;
            if (PAD && e >= D) continue;
            float o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = acc[d][4 * i + j] * inv * kUnitV<MODE>;
            *reinterpret_cast<u32x2_t*>(out + e) = u32x2_t{round16x2<DT>(o[0], o[1]), round16x2<DT>(o[2], o[3])};
          }
        if (a.lse && hf == 0)
          a.lse[to * a.Hq + head] = l == 0.0f ? -kInf : (m + static_cast<float>(ref) - kW + __builtin_amdgcn_logf(l)) * 0.693147181f;
      }
    }

    // ---- the next segment
    sg.at += places_before(a, sg.s.off, sg.s.lk, sg.tile + 1) - places_before(a, sg.s.off, sg.s.lk, sg.tile);
    if (sg.at >= last) return;
    if (++sg.tile == sg.s.tiles) {
      sg.tile = 0;
      if (++sg.head == a.heads) {
        sg.head = 0;
        do sg.s = seq_of(a, ++sg.b); while (sg.s.tiles == 0 && sg.b < a.B);
        sg.s = lane_seq(sg.s, 0);
      }
    }
  }
}

// Joins the parts of a segment that several runs share: the workgroups of run i do the one that begins in run i and
// goes on behind it; a workgroup 32 elements, a thread a row and 16 of them.
template <int MODE, int DT, int DP>
__global__ __launch_bounds__(kThreads) void chunk_join_kernel(ChunkArgs a, const float* __restrict__ ws) {
  const Deal deal(all_places(a), a.runs);
  const int run = blockIdx.x;
  if (run + 1 >= static_cast<int>(deal.runs)) return;
  const int end = deal.start(run + 1);
  const Segment sg = segment_at(a, end - 1);
  const Walk wk = walk_of(a, sg.s, sg.tile);
  const int base = sg.at + kStart;
  if (deal.start(run) > base || end <= base || end - base >= wk.n) return;  // its first tile is not here, or its last one is
  const int hk = sg.head / a.head_tiles, ht = sg.head - hk * a.head_tiles, hn = min(a.tile_heads, a.g - ht * a.tile_heads);
  const int r = threadIdx.x % kRows, e = 32 * blockIdx.y + 16 * (threadIdx.x / kRows);
  const int token = wk.row0 + r / a.tile_heads, hr = r % a.tile_heads, head = hk * a.g + ht * a.tile_heads + hr;
  if (token > wk.row1 || r >= a.tokens * a.tile_heads || hr >= hn || e >= a.c.D) return;
  float m = -kInf, l = 0.0f, o[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) o[j] = 0.0f;
  for (int i = run;; ++i) {
    const float* const p = ws + static_cast<int64_t>(2 * i + (i == run ? 1 : 0)) * ((DP + 2) * kRows) + r;
    const float mi = p[DP * kRows], li = p[(DP + 1) * kRows];
    float x[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = p[(e + j) * kRows];
    const float mn = fmaxf(m, mi);
    const float f0 = m == -kInf ? 0.0f : rescale(m, mn), f1 = mi == -kInf ? 0.0f : rescale(mi, mn);
    m = mn;
    l = li == 0.0f ? l * f0 : __builtin_fmaf(l, f0, li * f1);  // (nothing seen, or NaN)
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j] = __builtin_fmaf(o[j], f0, x[j] * f1);
    if (deal.start(i + 1) - base >= wk.n) break;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int64_t to = sg.s.q0 + token;
  uint16_t* const out = a.out.p + to * a.out.row + head * a.out.head + e;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (e + 8 * h >= a.c.D) break;
    u32x4_t w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = round16x2<DT>(o[8 * h + 2 * j] * inv * kUnitV<MODE>, o[8 * h + 2 * j + 1] * inv * kUnitV<MODE>);
    *reinterpret_cast<u32x4_t*>(out + 8 * h) = w;
  }
  if (a.lse && e == 0)
    a.lse[to * a.Hq + head] = l == 0.0f ? -kInf : (m - kUpW<MODE, DT> + __builtin_amdgcn_logf(l)) * 0.693147181f;
}

template <int MODE, int DT, int DP, bool PAD>
hipError_t chunk_go(const ChunkArgs& a, float* ws, hipStream_t s) {
  chunk_kernel<MODE, DT, DP, PAD><<<static_cast<uint32_t>(8 * ceil_div(a.runs, 8)), kThreads, 0, s>>>(a, ws);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || a.runs == 1 || a.single) return err;
  chunk_join_kernel<MODE, DT, DP><<<dim3(static_cast<uint32_t>(a.runs - 1), static_cast<uint32_t>(ceil_div(a.c.D, 32))), kThreads, 0, s>>>(a, ws);
  return hipGetLastError();
}

template <int MODE, int DT>
hipError_t chunk_by_size(const ChunkArgs& a, float* ws, hipStream_t s) {
  const int D = a.c.D;
  if (D == 64) return chunk_go<MODE, DT, 64, false>(a, ws, s);
  if (D == 128) return chunk_go<MODE, DT, 128, false>(a, ws, s);
  if (D == 256) return chunk_go<MODE, DT, 256, false>(a, ws, s);
  if (D < 64) return chunk_go<MODE, DT, 64, true>(a, ws, s);
  return D < 128 ? chunk_go<MODE, DT, 128, true>(a, ws, s) : chunk_go<MODE, DT, 256, true>(a, ws, s);
}

template <int MODE>
hipError_t chunk_mode(const ChunkArgs& a, void* ws, hipStream_t s) {
  float* const w = static_cast<float*>(ws);
  return a.c.dtype == kF16 ? chunk_by_size<MODE, kF16>(a, w, s) : chunk_by_size<MODE, kBF16>(a, w, s);
}

}  // namespace
}  // namespace fq
