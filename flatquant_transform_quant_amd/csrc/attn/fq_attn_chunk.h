// Attention of new tokens over the paged cache: the kernels, instantiated by cache format in fq_attn_chunk_*.hip.
//
// Sequence b has the query rows cu_q[b] .. cu_q[b+1]-1, its newest tokens, whose keys and values the cache holds already
// among its lengths[b] tokens.  Row i sees the keys up to its own position, with a window only the last W of them and
// the first S: o = sum_j p_j v_j, p = softmax over the visible keys of scale * <q, k_j>.
//
// A workgroup of four waves takes a row tile: the g query heads of one cache head for neighbouring tokens (a cached byte is read
// once for all of them), 128, 64 or 32 rows, the smallest that the mean rows of a sequence and cache head fit.  With 128 a wave has
// 32 rows; with 64 waves 2 and 3 have the rows of 0 and 1 and the other half of the keys; with 32 each wave has all rows and keys
// of its own, in LDS of its own without barriers (24 sequences of 5 drafts, 40 rows, over int8, in tiles of 128 265 us, of 64 122;
// see kShort for single tokens).  It walks the keys in tiles of 64 as the prompt kernel does: two LDS buffers, S^T = K Q^T and O^T
// = V^T P^T with 32 x 32 x 16 products, a lane owning one row's statistics, the maximum moved only when a score passes m + 8 in
// base-2 units.  LDS layouts as there.  A tile's keys lie in pages of 16 tokens at least: each wave brings the 16 rows that are one
// page's (16 bits by LDS-DMA).
//
// Low-bit formats: the codes go through registers, are widened to f16 numbers there, exactly, and written to LDS;
// a tile's bytes are widened once for all of its rows.  Widened: int8 and int4 the code times 2^-9, E4M3 the code, E2M1 the code
// times its group's power of two over the row's largest, times 2^13 (a group more than 2^26 below the largest of its
// row loses bits).  So every format has one factor a row: a key's multiplies its scores, a value's its weights, both in fp32 out of
// LDS.  A bf16 q is brought to f16 by a power of two a row (28 binades below its largest element keep all bits).
// Weights times value scales go to f16 relative to a reference exponent R, a row's own: w = exp2(s - m - R + 5) scale, where
// R is at least the exponent of the scales seen, less one (w stays below 2^15).  The sum l is of exp2(s - m - R + 5), so the
// quotient needs neither, and parts of a walk are joined as means with their weights' sums, without R.
//
// Split: every (sequence, cache head, row tile) is a segment of key tiles; all segments one after the other are dealt to
// the grid in equal runs.  A segment's place in that order has a closed form in its tile number (its walk's
// length is linear in it, up to the window), so a run finds its first segment by a scan over the sequences and a
// bisection.  A run that has a segment in part leaves its sums in the workspace, at most two such parts a run,
// and a second launch joins them in order.  (Cuts moved to a segment's edge where that is near save few parts and cost as much: no gain.)
//
// Bound, with 64 query heads on 8 or 32 on 8, D = 128: 16384 rows in f16 with a window of 4096, 305 to 324 us, up to 0.79 PFLOP/s,
// matrix cores 37% and vector unit 42% busy, one after the other in a wave, two waves a SIMD; 5 chunks of 1024 over int4, 577 us,
// 0.63 PFLOP/s: widening and softmax, vector unit 51%; 24 x 5 drafts over up to 16384 int8 tokens, 113 us, 2.9 TB/s: vector unit
// 43%, of which 24 of 64 rows are padding's; 32 single tokens of 1028 keys in bf16, 36 us, 3.8 TB/s.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "fq_attn_tile.h"
#include "fq_attn_chunk_plan.h"

namespace fq {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kAhead = 4;           // fragments read ahead of their products
constexpr float kLazy = 8.0f;
// Workgroups a CU that there are registers for.  Heads of 64: 1024 single tokens of 8 heads on 2, int8, with a window of 1024, 154
// us where there are for two, 128 for three.
template <int DP>
constexpr int kGroups = DP == 256 ? 1 : DP == 64 ? 3 : 2;

template <int MODE>
constexpr int kCodeBits = MODE == kKvInt8 || MODE == kKvE4M3 ? 8 : 4;
// a key's and a value's operand for 1 (E2M1: the keys' is in their factors)
template <int MODE>
constexpr float kUnitK = MODE == kKvInt8 || MODE == kKvInt4 ? 512.0f : 1.0f;
template <int MODE>
constexpr float kUnitV = MODE == kKvFp4 ? 0x1p-13f : kUnitK<MODE>;
// The reference R lies between these.  From kLeastRef on a walk's 2^31 weights sum below 2^127; up to kMostRef a weight of 1 is
// well within fp32's normal numbers.  Above kFullRef those 2^-35 of the largest are not (exp2 gives 0 below 2^-126): the walk is
// done again with value scales 2^-kDown of what they are, which are far below the largest where that is a subnormal number.
constexpr int kLeastRef = -82, kMostRef = 120, kFullRef = 96, kDown = 64;
// Whether the weights of row tiles of 32 RB rows enter the second product in two parts, the rounded weight and what the rounding
// left, and so with 16 bits (bf16) or 22.  Rounded once they add as much to an output's error as its own rounding where that has as
// many bits: 1.4 times the error in all (single tokens over a bf16 cache 2.2e-3 of the output, so 1.6e-3).  us without and with: 32
// single tokens of 1028 keys in bf16 35.0, 35.8, like all tiles of 32, which wait for memory; 24 x 5 drafts over int8 in tiles of
// 64 113.8, 122.5, so not for bf16 rows, whose output has 8 bits to these weights' 11; tiles of 128 keep one part, a document of
// 16384 rows in f16 314, 405, 5 chunks of 1024 over int4 575, 656: matrix and vector unit are what bounds them.
template <int MODE, int DT, int RB>
constexpr bool kRest = RB == 1 || (RB == 2 && (MODE == kKv16 || DT == kF16));
// weights enter the second product 2^kUpW times above the row's reference
template <int MODE, int DT>
constexpr float kUpW = MODE == kKv16 ? kUp<DT> : 5.0f;

// The lane's number, opaque to the compiler from here on: what is formed from it is not kept from before (a kernel's phases each have
// many addresses that depend on the lane alone; all of them held through the walk were more registers than there are).
__device__ __forceinline__ int lane_here() {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  return lane & 63;  // (so that its range stays known)
}

// A kernel's arguments (its first ones), read anew from here on, for the same reason: scalar registers.
__device__ __forceinline__ const ChunkArgs& args_here() {
  uint64_t p = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const ChunkArgs*)(const __attribute__((address_space(4))) ChunkArgs*)p;
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

// Rows of a tile that one wave brings through registers, NR of them (16 a page): their pieces and scales, of both sides.
template <int MODE, int DP, bool PAD, int NR>
struct Rows {
  static_assert(MODE != kKv16, "16-bit rows go to LDS by LDS-DMA");
  static constexpr int bits = kCodeBits<MODE>;
  static constexpr int CE = PAD ? 8 : (128 / bits < DP / 4 ? 128 / bits : DP / 4);  // elements of a piece
  static constexpr int LPR = DP / CE;        // lanes of a row
  static constexpr int N = NR * LPR / 64;    // pieces of a lane and side
  static constexpr int NH = 16 * LPR / 64;   // of one page
  static constexpr int W = CE * bits / 32;   // dwords of a piece
  uint32_t w[2][N][W];
  uint32_t e8[2][MODE == kKvFp4 ? N : 1];
  float scale[2][NR / 16];                   // of row lane % 16 of a page
};

// LDS places of 16-byte pieces: piece c of a key row r sits at c ^ key_swz, of a value row at c ^ value_swz.
template <int DP>
__device__ __forceinline__ int key_swz(int r) { return DP == 64 ? (r >> 1) & 7 : r & 15; }
template <int DP>
__device__ __forceinline__ int value_swz(int r) { return 4 * (DP == 64 ? (r >> 1) & 1 : r & 3); }

// Loads of page `pg` (below 0: none, zeros come) into the pieces of half `half`: `rows` rows from row `r` of the side on.
template <int MODE, int DP, bool PAD, int NR>
__device__ __forceinline__ void load_rows(Rows<MODE, DP, PAD, NR>& x, const KvCache& c, int lane, int half, int pg, int64_t r, int rows, int rowb, int sb, int D) {
  using R = Rows<MODE, DP, PAD, NR>;
  const int64_t at = max(pg, 0);
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const KvSide& sd = side ? c.v : c.k;
    const auto rc = __builtin_amdgcn_make_buffer_rsrc(sd.codes + (at * sd.page_b + r * rowb), static_cast<int16_t>(0), pg < 0 ? 0 : rows * rowb,
                                                      kBufferWord3);
#pragma unroll
    for (int i = 0; i < R::NH; ++i) {
      const int rr = (64 * i + lane) / R::LPR, p = (64 * i + lane) % R::LPR;
      load_piece<R::W>(rc, !PAD || R::CE * p < D ? static_cast<uint32_t>(rr * rowb + p * (R::CE * R::bits / 8)) : kOut, x.w[side][half * R::NH + i]);
    }
    const auto rs = __builtin_amdgcn_make_buffer_rsrc(sd.scale + (at * sd.scale_page_b + r * sb), static_cast<int16_t>(0), pg < 0 ? 0 : rows * sb,
                                                      kBufferWord3);
    if constexpr (MODE == kKvFp4) {
#pragma unroll
      for (int i = 0; i < R::NH; ++i) {
        const int rr = (64 * i + lane) / R::LPR, p = (64 * i + lane) % R::LPR;
        x.e8[side][half * R::NH + i] =
            __builtin_amdgcn_raw_buffer_load_b8(rs, !PAD || R::CE * p < D ? static_cast<uint32_t>(rr * sb + R::CE * p / 32) : kOut, 0, 0);
      }
    } else {
      x.scale[side][half] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, 4 * (lane & 15), 0, 0));
    }
  }
}

// The rows, widened, to LDS: keys from row `row0` of the tile at kt on, values of that at vt, their factors to ks and vs.
// Returns the largest value scale (neither infinity nor NaN) of them.  Values that are not finite become f16 NaN, with a factor of 0 or
// of the row's other groups.  Values' factors are `down` of what they are.
template <int MODE, int DP, bool PAD, int NR>
__device__ __forceinline__ float store_rows(const Rows<MODE, DP, PAD, NR>& x, int lane, uint8_t* kt, uint8_t* vt, float* ks, float* vs, int row0, float down) {
  using R = Rows<MODE, DP, PAD, NR>;
  float big = 0.0f;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
#pragma unroll
    for (int i = 0; i < R::N; ++i) {
      const int half = i / R::NH, rr = (64 * (i % R::NH) + lane) / R::LPR, p = (64 * i + lane) % R::LPR, r = row0 + 16 * half + rr;
      float s = 1.0f;
      bool nan = false;  // the piece's values are NaN
      if constexpr (MODE == kKvFp4) {
        const int e = static_cast<int>(x.e8[side][i]);
        nan = e == 255;
        const int top = max(kLeastE, lanes_max<R::LPR>(nan ? 0 : e));
        s = pow2(max(e - top + kUpE, -126));
        float f = pow2(top - 127 - (side == 0 ? kUpE : 0));
        if (side == 0) {
          if (lanes_max<R::LPR>(nan ? 1 : 0)) f = __builtin_nanf("");
        } else {
          f *= down;
          big = fmaxf(big, f);
        }
        if (p == 0) (side == 0 ? ks : vs)[r] = f;
      } else if (side == 1) {
        nan = !(__shfl(__builtin_fabsf(x.scale[1][half]), rr) < kInf);
      }
      uint8_t* const to = (side == 0 ? kt : vt) + r * (2 * DP);
      const int sw = side == 0 ? key_swz<DP>(r) : value_swz<DP>(r);
#pragma unroll
      for (int e = 0; e < R::CE / 8; ++e) {
        u32x4_t o = widened<MODE>(x.w[side][i], e, s);
        if (side == 1 && nan) o = u32x4_t{0x7E007E00u, 0x7E007E00u, 0x7E007E00u, 0x7E007E00u};
        *reinterpret_cast<u32x4_t*>(to + 16 * (((R::CE / 8) * p + e) ^ sw)) = o;
      }
    }
    if constexpr (MODE != kKvFp4) {
#pragma unroll
      for (int h = 0; h < NR / 16; ++h) {
        const bool fine = side == 0 || __builtin_fabsf(x.scale[1][h]) < kInf;
        const float f = !fine ? 0.0f : side == 0 ? x.scale[0][h] : x.scale[1][h] * down;
        if (lane < 16) (side == 0 ? ks : vs)[row0 + 16 * h + lane] = f;
        if (side == 1) big = fmaxf(big, __builtin_fabsf(f));
      }
    }
  }
  big = fmaxf(big, dpp_f<kDppQuadXor1>(big));
  big = fmaxf(big, dpp_f<kDppQuadXor2>(big));
  big = fmaxf(big, dpp_f<kDppRowHalfMirror>(big));
  big = fmaxf(big, dpp_f<kDppRowMirror>(big));
  if constexpr (MODE == kKvFp4) {  // (the others have the same 16 scales in every row of 16 lanes)
    big = half_max(big);
    big = fmaxf(big, __shfl_xor(big, 16));
  }
  return big;
}

// ---- a segment's rows and pages ------------------------------------------------------------------

// 32 query rows of a row tile: what a lane knows of its own (column lane % 32 of the products), and the wave of all.
struct Place {
  bool mine;       // not a repeated row
  int token, head; // of the sequence, of all query heads
  int lim, lo;     // the last key seen, the first in the window
  int lim_first, lim_last, lo_first, lo_last;  // of the first and last of the wave's rows
};
__device__ __forceinline__ Place place_of_rows(const ChunkArgs& a, const Segment& sg, const Walk& wk, int lane, int row0) {
  const int hk = sg.head / a.head_tiles, ht = sg.head - hk * a.head_tiles;
  const int hn = min(a.tile_heads, a.g - ht * a.tile_heads);  // heads of this tile
  const int row = row0 + (lane & 31);
  const int tok = wk.row0 + row / a.tile_heads, hr = row % a.tile_heads;
  Place p;
  p.mine = tok <= wk.row1 && row < a.tokens * a.tile_heads && hr < hn;
  p.token = min(tok, wk.row1);
  p.head = hk * a.g + ht * a.tile_heads + min(hr, hn - 1);
  const int off = sg.s.off;
  auto low_of = [&](int l) __attribute__((always_inline)) { return a.window > 0 ? max(0, l - a.window + 1) : 0; };
  p.lim = off + p.token;
  p.lo = low_of(p.lim);
  p.lim_first = off + min(wk.row0 + row0 / a.tile_heads, wk.row1);
  p.lim_last = off + min(wk.row0 + (row0 + 31) / a.tile_heads, wk.row1);
  p.lo_first = low_of(p.lim_first);
  p.lo_last = low_of(p.lim_last);
  return p;
}

// The pages of 16 tiles of a walk at a time: lane 4 i + w has that of the w-th 16 keys of the i-th tile.
struct Pages {
  int page, from;  // from: the walk's tile of lane 0
  uint64_t there;  // keys with a page (or past the sequence's end), a bit a lane
  __device__ __forceinline__ void need(const ChunkArgs& a, const Segment& sg, const Walk& wk, int u) {
    if (u >= from && u < from + 16) return;
    const int lane = threadIdx.x & 63, i = u + (lane >> 2);
    const int t = i < wk.n ? wk.tile(i) * kKeys + 16 * (lane & 3) : a.reach;
    page = t < sg.s.lk ? kv_page(a.bt, sg.b, t, a.c.page_log, a.c.pages) : -1;
    there = __ballot(page >= 0 || t >= sg.s.lk);
    from = u;
  }
  __device__ __forceinline__ int of(int u, int sub) const { return __builtin_amdgcn_readlane(page, 4 * (u - from) + sub); }
  __device__ __forceinline__ uint32_t bits(int u) const { return static_cast<uint32_t>(there >> (4 * (u - from))) & 15u; }
};
// rows that a page's 16 keys from key k on have, and the row of a side that they begin at
__device__ __forceinline__ int rows_at(const Segment& sg, int k) { return __builtin_amdgcn_readfirstlane(max(0, min(16, sg.s.lk - k))); }
__device__ __forceinline__ int64_t row_at(const ChunkArgs& a, int hk, int k) {
  return (static_cast<int64_t>(hk) << a.c.page_log) + (k & ((1 << a.c.page_log) - 1));
}

// The same with the addresses of the 16 rows on both sides and their bytes, so that a tile's LDS-DMA needs no more than to pick a
// lane's, and starts before the tile's products (formed a tile at a time from arguments read anew, under the first products:
// document of 16384 rows 317 us, so 309; the earlier start alone changes nothing).
struct PageRows : Pages {
  uint64_t at[2];
  int bytes;
  __device__ __forceinline__ void need(const ChunkArgs& a, const Segment& sg, const Walk& wk, int u, int hk, int rowb) {
    if (u >= from && u < from + 16) return;
    Pages::need(a, sg, wk, u);
    const int lane = threadIdx.x & 63, i = u + (lane >> 2), k = i < wk.n ? wk.tile(i) * kKeys + 16 * (lane & 3) : a.reach;
    const int64_t pg = max(page, 0), r = row_at(a, hk, k) * rowb;
    bytes = page < 0 ? 0 : max(0, min(16, sg.s.lk - k)) * rowb;
    at[0] = reinterpret_cast<uint64_t>(a.c.k.codes) + (pg * a.c.k.page_b + r);
    at[1] = reinterpret_cast<uint64_t>(a.c.v.codes) + (pg * a.c.v.page_b + r);
  }
  __device__ __forceinline__ i32x4_t rows(int u, int sub, int side) const {
    const int lane = 4 * (u - from) + sub;
    const uint32_t high = __builtin_amdgcn_readlane(static_cast<int>(at[side] >> 32), lane), low = __builtin_amdgcn_readlane(static_cast<int>(at[side]), lane);
    return rsrc4(reinterpret_cast<const void*>(static_cast<uint64_t>(high) << 32 | low), static_cast<uint32_t>(__builtin_amdgcn_readlane(bytes, lane)));
  }
};

// a = acc[D] times f where `need` (the wave's) is not 0.  The compiler copies the 16-register blocks to other registers and back
// around such a branch, for every tile, which waits for the products besides (document of 16384 rows 363 us, so 315); so each block
// has a place that the statements ask for, and the branch is inside: nothing is left to copy.  With it the wait states between the
// products that wrote the block and this read (at most 18), and between this write and the products that read it.
template <int D>
__device__ __forceinline__ void scale_block(f32x16_t& a, float f, int need) {
  need = __builtin_amdgcn_readfirstlane(need);
#define FQ_SCALE(N, R0, R1, R2, R3, R4, R5, R6, R7, R8, R9, R10, R11, R12, R13, R14, R15) \
  if constexpr (D == N) \
    asm("s_cmp_eq_u32 %2, 0\n\ts_cbranch_scc1 .Lfq_scaled%=\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7\n\t" \
        "v_mul_f32 v" #R0 ", %1, v" #R0 "\n\t" "v_mul_f32 v" #R1 ", %1, v" #R1 "\n\t" \
        "v_mul_f32 v" #R2 ", %1, v" #R2 "\n\t" "v_mul_f32 v" #R3 ", %1, v" #R3 "\n\t" \
        "v_mul_f32 v" #R4 ", %1, v" #R4 "\n\t" "v_mul_f32 v" #R5 ", %1, v" #R5 "\n\t" \
        "v_mul_f32 v" #R6 ", %1, v" #R6 "\n\t" "v_mul_f32 v" #R7 ", %1, v" #R7 "\n\t" \
        "v_mul_f32 v" #R8 ", %1, v" #R8 "\n\t" "v_mul_f32 v" #R9 ", %1, v" #R9 "\n\t" \
        "v_mul_f32 v" #R10 ", %1, v" #R10 "\n\t" "v_mul_f32 v" #R11 ", %1, v" #R11 "\n\t" \
        "v_mul_f32 v" #R12 ", %1, v" #R12 "\n\t" "v_mul_f32 v" #R13 ", %1, v" #R13 "\n\t" \
        "v_mul_f32 v" #R14 ", %1, v" #R14 "\n\t" "v_mul_f32 v" #R15 ", %1, v" #R15 "\n\t" \
        "s_nop 3\n.Lfq_scaled%=:" : "={v[" #R0 ":" #R15 "]}"(a) : "v"(f), "s"(need), "0"(a) : "scc")
  FQ_SCALE(0, 16, 17, 18, 19, 20, 21, 22, 23, 24, 25, 26, 27, 28, 29, 30, 31);
  FQ_SCALE(1, 32, 33, 34, 35, 36, 37, 38, 39, 40, 41, 42, 43, 44, 45, 46, 47);
  FQ_SCALE(2, 48, 49, 50, 51, 52, 53, 54, 55, 56, 57, 58, 59, 60, 61, 62, 63);
  FQ_SCALE(3, 64, 65, 66, 67, 68, 69, 70, 71, 72, 73, 74, 75, 76, 77, 78, 79);
  FQ_SCALE(4, 80, 81, 82, 83, 84, 85, 86, 87, 88, 89, 90, 91, 92, 93, 94, 95);
  FQ_SCALE(5, 96, 97, 98, 99, 100, 101, 102, 103, 104, 105, 106, 107, 108, 109, 110, 111);
  FQ_SCALE(6, 112, 113, 114, 115, 116, 117, 118, 119, 120, 121, 122, 123, 124, 125, 126, 127);
  FQ_SCALE(7, 128, 129, 130, 131, 132, 133, 134, 135, 136, 137, 138, 139, 140, 141, 142, 143);
#undef FQ_SCALE
}

// Holds a[d] at the registers that scale_block has for it.
template <int D>
__device__ __forceinline__ void pin_block(f32x16_t& a) {
  if constexpr (D == 0) asm("" : "={v[16:31]}"(a) : "0"(a));
  if constexpr (D == 1) asm("" : "={v[32:47]}"(a) : "0"(a));
  if constexpr (D == 2) asm("" : "={v[48:63]}"(a) : "0"(a));
  if constexpr (D == 3) asm("" : "={v[64:79]}"(a) : "0"(a));
  if constexpr (D == 4) asm("" : "={v[80:95]}"(a) : "0"(a));
  if constexpr (D == 5) asm("" : "={v[96:111]}"(a) : "0"(a));
  if constexpr (D == 6) asm("" : "={v[112:127]}"(a) : "0"(a));
  if constexpr (D == 7) asm("" : "={v[128:143]}"(a) : "0"(a));
}

// Means of two or more parts are joined by their weights' sums l, brought to one maximum: a part's share of them.  (A mean may hold
// the infinity of an element that was seen: a share is never 0 but where nothing was.)
__device__ __forceinline__ float part_weight(float l, float m, float to) { return m == -kInf ? 0.0f : l * rescale(m, to); }
__device__ __forceinline__ float part_share(float w, float inv) {  // (inv: 1 over all; NaN stays)
  const float s = w * inv;
  return s < 0x1p-126f && w != 0.0f ? 0x1p-126f : s;
}
// (the part with the maximum has a weight of 1 at the least; all parts' are 0 where nothing was seen)
__device__ __forceinline__ float over_all(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }

// ---- the products of 32 keys with 32 query rows ------------------------------------------------------

template <int MODE, int DT, int DP, bool PAD>
struct Block {
  static constexpr bool kLow = MODE != kKv16;
  static constexpr int ODT = kLow ? kF16 : DT;  // the operands' type
  static constexpr int KS = DP / 16;            // products of a score block
  static constexpr int DB = DP / 32;            // 32-row blocks of O^T
  static constexpr int kRowB = DP * 2;          // bytes of a tile row
  static constexpr float kW = kUpW<MODE, DT>;

  u32x4_t qf[KS];  // the query rows as B operands
  float c;         // base-2 scores' factor
  f32x16_t acc[DB];
  float m, l;  // m: the maximum as a score, before its factor
  int ref;     // R
  int far;     // whether some row's maximum of the wave is beyond kFar

  __device__ __forceinline__ void load_q(const ChunkArgs& a, const Segment& sg, const Place& p, int lane) {
    const int hf = lane >> 5, D = PAD ? a.c.D : DP;
    c = __builtin_fabsf(a.scale) * 1.44269504f;
    const uint16_t* const qp = a.q.p + (sg.s.q0 + p.token) * a.q.row + p.head * a.q.head;
    const uint32_t sign = a.scale < 0.0f ? 0x80008000u : 0u;  // (a negative scale goes into the rows' sign)
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

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[d][i] = 0.0f;
    m = -kInf;
    l = 0.0f;
    ref = kLow ? kLeastRef : 0;
    far = 0;
  }

  // Whether some of the wave's rows see a key of k0 .. k0 + n - 1.
  static __device__ __forceinline__ bool sees(const Place& p, int sinks, int k0, int n) {
    return k0 <= p.lim_last && (k0 + n > p.lo_first || k0 < sinks);
  }

  // Keys k0 .. k0 + 32 NB - 1, their rows at kt and vt in LDS (from a multiple of 32 on), their factors at ks and vs.  in: which 16
  // of them have a page; big: the largest value scale.  `scored` is called when
  // the score products are under way, before a value is read.
  template <int NB, bool REST, typename F>
  __device__ __forceinline__ void step(const Place& p, int lane, int sinks, int k0, uint32_t in, float big, const lds_u8* kt, const lds_u8* vt,
                                       const float* ks_, const float* vs_, F&& scored) {
    const int col = lane & 31, hf = lane >> 5;
    const uint32_t krd = col * kRowB, kx = hf ^ key_swz<DP>(col);
    const int rj = (lane & 15) >> 2;
    const uint32_t vrd = (4 * hf + rj) * kRowB + 32 * ((lane >> 4) & 1) + 8 * (lane & 3), vx = DP == 64 ? rj >> 1 : rj;
    auto key = [&](int ks, int b) __attribute__((always_inline)) {
      return *(const __attribute__((address_space(3))) u32x4_t*)(kt + krd + 16 * (kx ^ (2 * ks)) + b * 32 * kRowB);
    };
    auto value = [&](int d, int g) __attribute__((always_inline)) {
      const lds_u8* const q = vt + vrd + 64 * (d ^ vx) + 16 * g * kRowB;
      const u32x2_t lo2 = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)q));
      const u32x2_t hi2 = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(q + 8 * kRowB)));
      return u32x4_t{lo2[0], lo2[1], hi2[0], hi2[1]};
    };
    // the factors of the keys of registers 4 j .. 4 j + 3 of the scores
    auto factors = [&](const float* f, int j) __attribute__((always_inline)) { return *reinterpret_cast<const f32x4_t*>(f + 8 * j + 4 * hf); };

    f32x16_t s[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[b][i] = 0.0f;
    {
      u32x4_t kf[NB * KS];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) kf[i] = key(i / NB, i % NB);
      static_for<0, NB * KS>([&](auto ic) __attribute__((always_inline)) {
        constexpr int i = decltype(ic)::value;
        if constexpr (i + kAhead < NB * KS) kf[i + kAhead] = key((i + kAhead) / NB, (i + kAhead) % NB);
        __builtin_amdgcn_sched_barrier(0);
        s[i % NB] = mfma32x32x16<ODT>(kf[i], qf[i / NB], s[i % NB]);
        __builtin_amdgcn_sched_barrier(0);
      });
    }
    scored();
    if constexpr (kLow) {
#pragma unroll
      for (int j = 0; j < 4 * NB; ++j) {
        const f32x4_t f = factors(ks_, j);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[j / 4][4 * (j % 4) + i] *= f[i];
      }
    }
    u32x4_t vf[2 * NB * DB];
#pragma unroll
    for (int i = 0; i < kAhead && i < 2 * NB * DB; ++i) vf[i] = value(i % DB, i / DB);
    __builtin_amdgcn_sched_barrier(0);
    const bool masked = k0 + 32 * NB - 1 > p.lim_first || (k0 < p.lo_last && k0 + 32 * NB > sinks) || in != (1u << (2 * NB)) - 1u;
    if (masked) {
      asm volatile("");  // (a branch: as selects, this is done for every tile)
      // this lane's places (4 hf less than the key among these): seen up to `left`, and from `from` on or below `sk`
      const int left = p.lim - k0 - 4 * hf, from = p.lo - k0 - 4 * hf, sk = sinks - k0 - 4 * hf;
#pragma unroll
      for (int i = 0; i < 16 * NB; ++i) {
        const int place = 8 * (i / 4) + i % 4;
        const bool seen = place <= left && (place >= from || place < sk) && ((in >> (i / 8)) & 1u);
        if (!seen) s[i / 16][i % 16] = -kInf;
      }
    }
    float top = s[0][0];
#pragma unroll
    for (int i = 1; i < 16 * NB; ++i) top = fmaxf(top, s[i / 16][i % 16]);
    int ev = kLeastRef;  // exponent of the largest value scale that is seen
    if constexpr (kLow) {
      if (masked) {
        big = 0.0f;
#pragma unroll
        for (int j = 0; j < 4 * NB; ++j) {
          const f32x4_t f = factors(vs_, j);
#pragma unroll
          for (int i = 0; i < 4; ++i) big = fmaxf(big, s[j / 4][4 * (j % 4) + i] == -kInf ? 0.0f : __builtin_fabsf(f[i]));
        }
      }
      ev = static_cast<int>(__float_as_uint(big) >> 23) - 127;
    }
    float f = 1.0f;
    const int need = __any((top - m) * c > kLazy || (kLow && ev > ref + 1));
    if (need) {
      const float mn = fmaxf(m, half_max(top));
      int rn = ref;
      if constexpr (kLow) {
        const auto r = __builtin_amdgcn_permlane32_swap(ev, ev, false, false);
        rn = max(ref, min(kMostRef, max(static_cast<int>(r[0]), static_cast<int>(r[1]))));
      }
      f = mn == -kInf ? 1.0f : __builtin_amdgcn_exp2f((m - mn) * c);
      m = mn;
      l *= f;
      if constexpr (kLow) {  // (R may rise by more than exp2 can say)
        f = __builtin_amdgcn_ldexpf(f, ref - rn);
        l = __builtin_amdgcn_ldexpf(l, ref - rn);
        ref = rn;
      }
      far = __any(m != -kInf && __builtin_fabsf(m) * c > kFar);
    }
    static_for<0, DB>([&](auto dc) __attribute__((always_inline)) { scale_block<decltype(dc)::value>(acc[decltype(dc)::value], f, need); });
    const float m0 = m == -kInf ? 0.0f : m;
    float ms = __builtin_fmaf(m0, c, static_cast<float>(ref) - kW);
    if (far) {
      // A maximum that large is off by units as an fp32 number in base 2 (its weight 2^8, infinite or 0 where it has to be 1): it is
      // taken off as a score.
      asm volatile("");
#pragma unroll
      for (int i = 0; i < 16 * NB; ++i) s[i / 16][i % 16] -= m0;
      ms = static_cast<float>(ref) - kW;
    }
    u32x4_t pf[2 * NB], rest[REST ? 2 * NB : 1];
#pragma unroll
    for (int g = 0; g < 2 * NB; ++g) {
      f32x4_t vs[2];
      if constexpr (kLow) {
        vs[0] = factors(vs_, 2 * g);
        vs[1] = factors(vs_, 2 * g + 1);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = 8 * (g % 2) + 2 * i;
        float x0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[g / 2][e], c, -ms));
        float x1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[g / 2][e + 1], c, -ms));
        l += x0 + x1;
        if constexpr (kLow) {
          x0 *= vs[i / 2][2 * (i % 2)];
          x1 *= vs[i / 2][2 * (i % 2) + 1];
        }
        pf[g][i] = round16x2<ODT>(x0, x1);
        if constexpr (REST)
          rest[g][i] = round16x2<ODT>(x0 - load16<ODT>(static_cast<uint16_t>(pf[g][i])), x1 - load16<ODT>(static_cast<uint16_t>(pf[g][i] >> 16)));
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    static_for<0, 2 * NB * DB>([&](auto ic) __attribute__((always_inline)) {
      constexpr int i = decltype(ic)::value;
      if constexpr (i + kAhead < 2 * NB * DB) vf[i + kAhead] = value((i + kAhead) % DB, (i + kAhead) / DB);
      __builtin_amdgcn_sched_barrier(0);
      acc[i % DB] = mfma32x32x16<ODT>(vf[i], pf[i / DB], acc[i % DB]);
      if constexpr (REST) acc[i % DB] = mfma32x32x16<ODT>(vf[i], rest[i / DB], acc[i % DB]);
      __builtin_amdgcn_sched_barrier(0);
    });
  }

  // Where a sum is not finite, the walk is done again with the values that are infinite or NaN taken out of the products: they
  // are noted for the rows that see them, a bit an element of a lane's sums for infinity, for minus infinity or both (NaN), in
  // LDS (words 2 w and 2 w + 1 of each lane), and added at the end, so that a seen infinity stays one, however small its weight ...
  static constexpr int kWords = DB / 2;
  typedef uint32_t Odd[2 * kWords][64];
  static __device__ __forceinline__ void no_odd(Odd& o) {
#pragma unroll
    for (int w = 0; w < 2 * kWords; ++w) o[w][threadIdx.x & 63] = 0u;
  }
  static __device__ __forceinline__ void note_odd(Odd& o, const Place& p, int sinks, int k0, uint32_t in, const lds_u8* vt) {
    const int lane = lane_here(), hf = lane >> 5;
#pragma clang loop unroll(disable)
    for (int j = 0; j < 32; ++j) {
      bool odd = false;
      for (int e = 2 * lane; e < DP; e += 128)
        odd |= not_finite16<ODT>(*(const __attribute__((address_space(3))) uint32_t*)(vt + j * kRowB + 2 * e)) != 0;
      if (!__any(odd) || !((in >> (j / 16)) & 1u)) continue;
      const int k = k0 + j;
      if (!(k <= p.lim && (k >= p.lo || k < sinks))) continue;
#pragma clang loop unroll(disable)
      for (int w = 0; w < kWords; ++w) {
        uint32_t up = 0, down = 0;
#pragma clang loop unroll(disable)
        for (int i = 0; i < 32; ++i) {
          const int e = 64 * w + 8 * (i / 4) + 4 * hf + i % 4;
          const uint16_t v = *(const __attribute__((address_space(3))) uint16_t*)(vt + j * kRowB + 16 * ((e / 8) ^ value_swz<DP>(j)) + 2 * (e % 8));
          const float x = load16<ODT>(v);
          const uint32_t bit = not_finite16<ODT>(v) ? 1u << i : 0u;
          up |= x < 0.0f ? 0u : bit;
          down |= x > 0.0f ? 0u : bit;
        }
        o[2 * w][lane] |= up;
        o[2 * w + 1][lane] |= down;
      }
    }
  }
  __device__ __forceinline__ void add_odd(const Odd& o) {
    const int lane = lane_here();
#pragma unroll
    for (int d = 0; d < DB; ++d) {
      const uint32_t up = o[2 * (d / 2)][lane], down = o[2 * (d / 2) + 1][lane];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int bit = 16 * (d % 2) + i;
        acc[d][i] += ((up >> bit) & 1u ? kInf : 0.0f) + ((down >> bit) & 1u ? -kInf : 0.0f);
      }
    }
  }
  // ... and taken out of the products, `rows` rows at vt.
  static __device__ __forceinline__ void drop_odd(lds_u8* vt, int rows) {
#pragma clang loop unroll(disable)
    for (int i = lane_here(); i < rows * (DP / 2); i += 64) {
      __attribute__((address_space(3))) uint32_t* const at = (__attribute__((address_space(3))) uint32_t*)(vt + 4 * i);
      const uint32_t v = *at;
      *at = v & ~not_finite16_mask<ODT>(v);
    }
  }
  __device__ __forceinline__ void pin() {
    static_for<0, DB>([&](auto dc) __attribute__((always_inline)) { pin_block<decltype(dc)::value>(acc[decltype(dc)::value]); });
  }
  // Whether the walk has to be done again: a sum is infinite or NaN, or the reference beyond kFullRef (`high`).
  __device__ __forceinline__ bool again() const { return odd() || high(); }
  __device__ __forceinline__ bool high() const { return kLow && ref > kFullRef; }
  // The walk's end: the sums become means of the values (0 where nothing was seen), l the sum of the weights, 2^kW times what they are
  // relative to m, without R, and m is in base-2 units.  Value scales were `down` of what they are.
  __device__ __forceinline__ void finish(float down) {
    l = half_sum(l);
    float inv = over_all(l);
    constexpr bool kFirst = kUnitV<MODE> < 1.0f;  // (E2M1's sums are up to 2^13 above the values: that goes first)
    const float up = kLow ? kUnitV<MODE> / down : 1.0f;
    if (kFirst) inv *= up;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[d][i] = kFirst || !kLow ? acc[d][i] * inv : acc[d][i] * inv * up;
    if constexpr (kLow) l = __builtin_amdgcn_ldexpf(l, ref);
    m *= c;
  }
  __device__ __forceinline__ bool odd() const {
    float o = 0.0f;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o = __builtin_fmaf(acc[d][i], 0.0f, o);
    return o != o;
  }
};

// A part for the join: its means [element][row] of TR rows, then m and l.
template <int DP, int TR>
constexpr int kPart = (DP + 2) * TR;

// ---- row tiles of 128 or 64: 32 rows a wave, the tile's keys shared -------------------------------------

// RB blocks of 32 rows: 4, a wave each; or 2, where waves 2 and 3 have the same rows as 0 and 1 and the tile's other 32 keys, and
// their sums are joined at the segment's end.
template <int MODE, int DT, int DP, bool PAD, int RB>
__global__ __launch_bounds__(kThreads, kGroups<DP>) void chunk_wide_kernel(ChunkArgs, float* __restrict__ ws) {
  using BK = Block<MODE, DT, DP, PAD>;
  constexpr bool kLow = BK::kLow;
  using RW = Rows<kLow ? MODE : kKvInt8, DP, PAD, 16>;  // (16 bits: not used)
  constexpr int DB = BK::DB, kRowB = BK::kRowB, kTR = 32 * RB;
  constexpr int kTileB = kKeys * kRowB;  // bytes of a tile (keys or values)
  constexpr int kPieces = DP / 8;        // 16-byte pieces of a row
  constexpr int NL = kTileB / 1024 / kWaves;
  __shared__ __align__(16) uint8_t lds[4 * kTileB];  // buffer b: keys at 2 b, values at 2 b + 1
  __shared__ __align__(16) float s_scale[kLow ? 2 : 1][2][kLow ? kKeys : 1];  // [buffer][keys, values]
  __shared__ __align__(16) float s_top[kLow ? 2 : 1][kWaves];                 // largest value scale of 16 keys
  __shared__ float s_m[2][RB == 2 ? 64 : 1];                                   // of waves 2 and 3: m, l
  __shared__ typename BK::Odd s_odd[kWaves];
  lds_u8* const lds_l = (lds_u8*)lds;
  const uint32_t lds_addr = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds_l));

  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int D = PAD ? args_here().c.D : DP;
  const int rowb = static_cast<int>(kv_row_bytes(MODE, D)), sb = static_cast<int>(kv_scale_bytes(MODE, D));
  const Run run = run_of(args_here());
  if (run.last <= run.first) return;
  Segment sg = segment_at(args_here(), run.first);
  if (sg.s.tiles == 0) return;

  // LDS-DMA of 16-bit rows: load i of a wave fills the 16-byte places 64 (NL w + i) + lane of a tile, its 16 rows in all
  uint32_t koff[NL], voff[NL];
  if constexpr (!kLow) {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int at = 64 * (NL * wv + i) + (threadIdx.x & 63), r = at / kPieces, p = at % kPieces;
      const int kp = p ^ key_swz<DP>(r), vp = p ^ value_swz<DP>(r);
      koff[i] = !PAD || 8 * kp < D ? static_cast<uint32_t>((r & 15) * rowb + 16 * kp) : kOut;
      voff[i] = !PAD || 8 * vp < D ? static_cast<uint32_t>((r & 15) * rowb + 16 * vp) : kOut;
    }
  }
  int step = 0;  // of this workgroup; the tile of step s is in buffer s % 2

  do {
    const ChunkArgs& a = args_here();
    const KvCache& cc = a.c;
    const Walk wk = walk_of(a, sg.s, sg.tile);
    const Share sh = share_of(a, run, sg, wk);
    if (!sh.whole && sh.u0 >= sh.u1) continue;
    const int hk = sg.head / a.head_tiles, lane = lane_here();
    const Place pl = place_of_rows(a, sg, wk, lane, 32 * (wv % RB));
    BK bk;
    bk.load_q(a, sg, pl, lane);
    std::conditional_t<kLow, Pages, PageRows> pages{};
    pages.from = -(1 << 30);
    auto dma = [&](int u, int buf) __attribute__((always_inline)) {
      if constexpr (!kLow) {
        pages.need(a, sg, wk, u, hk, rowb);
        const i32x4_t rk = pages.rows(u, wv, 0), rv = pages.rows(u, wv, 1);
        const uint32_t to = lds_addr + buf * (2 * kTileB) + 1024 * NL * wv;
#pragma unroll
        for (int i = 0; i < NL; ++i) dma16(to + 1024 * i, koff[i], rk);
#pragma unroll
        for (int i = 0; i < NL; ++i) dma16(to + kTileB + 1024 * i, voff[i], rv);
      }
    };
    RW x;
    auto load = [&](int u) __attribute__((always_inline)) {
      if constexpr (kLow) {
        pages.need(a, sg, wk, u);
        const int k = wk.tile(u) * kKeys + 16 * wv;
        load_rows(x, cc, lane, 0, pages.of(u, wv), row_at(a, hk, k), rows_at(sg, k), rowb, sb, D);
      }
    };
    float down = 1.0f;
    auto store = [&](int buf) __attribute__((always_inline)) {
      if constexpr (kLow) {
        const float big = store_rows(x, lane, lds + buf * (2 * kTileB), lds + buf * (2 * kTileB) + kTileB, s_scale[buf][0], s_scale[buf][1], 16 * wv, down);
        if (lane == 0) s_top[buf][wv] = big;
      }
    };
    for (bool careful = false;;) {
      bk.clear();
      if (sh.u0 < sh.u1) {
        if constexpr (kLow) {
          load(sh.u0);
          store(step & 1);
        } else {
          dma(sh.u0, step & 1);
        }
      }
      for (int u = sh.u0; u < sh.u1; ++u, ++step) {
        const int buf = step & 1, k0 = wk.tile(u) * kKeys;
        const uint32_t in = pages.bits(u);  // which 16 keys have a page
        tile_barrier();
        // the next tile's rows: to LDS, or to registers until this tile is done (loaded under its first products 24 x 5 drafts over int8
        // take 113 us in place of 111, 5 chunks of 1024 over int4 582 in place of 574)
        if (u + 1 < sh.u1) {
          if constexpr (kLow)
            load(u + 1);
          else
            dma(u + 1, buf ^ 1);
        }
        lds_u8* const kt = lds_l + buf * (2 * kTileB);
        lds_u8* const vt = kt + kTileB;
        if (careful) {
          for (int b = RB == 2 ? wv / 2 : 0; b < (RB == 2 ? wv / 2 + 1 : 2); ++b) BK::note_odd(s_odd[wv], pl, a.sinks, k0 + 32 * b, (in >> (2 * b)) & 3u, vt + 32 * b * kRowB);
          __syncthreads();
          BK::drop_odd(vt + 16 * wv * kRowB, 16);
          __syncthreads();
        }
        // 64 keys at a time in 16 bits, 32 where the widening of codes needs registers too
        constexpr int NB = kLow || RB == 2 ? 1 : 2;
#pragma unroll
        for (int i = 0; i < (RB == 2 ? 1 : 2 / NB); ++i) {
          const int b = RB == 2 ? wv / 2 : i;
          if (!BK::sees(pl, a.sinks, k0 + 32 * b, 32 * NB)) continue;
          const float big = kLow ? fmaxf(s_top[buf][2 * b], s_top[buf][2 * b + 1]) : 0.0f;
          bk.template step<NB, kRest<MODE, DT, RB>>(pl, lane, a.sinks, k0 + 32 * b, (in >> (2 * b)) & ((1u << (2 * NB)) - 1u), big,
                               kt + 32 * b * kRowB, vt + 32 * b * kRowB, &s_scale[buf][0][32 * b], &s_scale[buf][1][32 * b], [] {});
        }
        if constexpr (kLow) {
          if (u + 1 < sh.u1) store(buf ^ 1);
        }
      }
      bk.pin();
      if (careful || !__syncthreads_or(bk.again())) {
        if (careful) bk.add_odd(s_odd[wv]);
        break;
      }
      if (kLow && __syncthreads_or(bk.high())) down = pow2(-kDown);
      careful = true;
      BK::no_odd(s_odd[wv]);
    }
    // (no barrier needed here: the next segment's first tile takes the buffer that was last read a step before the last one)

    const int end = lane_here(), col = end & 31, hf = end >> 5;
    const ChunkArgs& z = args_here();
    bk.finish(down);
    if constexpr (RB == 2) {  // waves 2 and 3 hand their sums over in the other buffer
      float* const at = reinterpret_cast<float*>(lds + ((step & 1) ^ 1) * (2 * kTileB)) + (wv & 1) * (32 * DP) + col;
      __syncthreads();
      if (wv >= 2) {
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) at[(32 * d + 8 * (i / 4) + 4 * hf + i % 4) * 32] = bk.acc[d][i];
        if (hf == 0) {
          s_m[0][32 * (wv & 1) + col] = bk.m;
          s_m[1][32 * (wv & 1) + col] = bk.l;
        }
      }
      __syncthreads();
      if (wv >= 2) continue;
      const float mo = s_m[0][32 * wv + col], mn = fmaxf(bk.m, mo);
      const float w0 = part_weight(bk.l, bk.m, mn), w1 = part_weight(s_m[1][32 * wv + col], mo, mn);
      bk.m = mn;
      bk.l = w0 + w1;
      const float inv = over_all(bk.l), f0 = part_share(w0, inv), f1 = part_share(w1, inv);
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) bk.acc[d][i] = __builtin_fmaf(bk.acc[d][i], f0, at[(32 * d + 8 * (i / 4) + 4 * hf + i % 4) * 32] * f1);
    }
    if (!sh.whole) {
      float* const o = ws + static_cast<int64_t>(part_at(run.i, sh.u0)) * kPart<DP, kTR> + 32 * (wv % RB) + col;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[(32 * d + 8 * (i / 4) + 4 * hf + i % 4) * kTR] = bk.acc[d][i];
      if (hf == 0) {
        o[DP * kTR] = bk.m;
        o[(DP + 1) * kTR] = bk.l;
      }
    } else if (pl.mine) {
      const int64_t to = sg.s.q0 + pl.token;
      uint16_t* const out = z.out.p + to * z.out.row + pl.head * z.out.head;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = 32 * d + 8 * i + 4 * hf;
          if (PAD && e >= D) continue;
          *reinterpret_cast<u32x2_t*>(out + e) = u32x2_t{round16x2<DT>(bk.acc[d][4 * i], bk.acc[d][4 * i + 1]),
                                                         round16x2<DT>(bk.acc[d][4 * i + 2], bk.acc[d][4 * i + 3])};
        }
      if (z.lse && hf == 0) z.lse[to * z.Hq + pl.head] = bk.l == 0.0f ? -kInf : (bk.m - BK::kW + __builtin_amdgcn_logf(bk.l)) * 0.693147181f;
    }
  } while (next_segment(args_here(), run, sg));
}

// ---- row tiles of 32: every wave has all of them, and keys of its own --------------------------------------

// A wave takes every fourth 32 keys of the walk into an LDS region of its own: no barrier before the segment's end, where the
// waves' sums are joined.  Low-bit rows go through registers, the next 32 on their way during the products of these; 16-bit ones by
// LDS-DMA, the next keys as soon as the scores are done with these, the next values behind the second products.
template <int MODE, int DT, int DP, bool PAD>
__global__ __launch_bounds__(kThreads, kGroups<DP>) void chunk_narrow_kernel(ChunkArgs, float* __restrict__ ws) {
  using BK = Block<MODE, DT, DP, PAD>;
  constexpr bool kLow = BK::kLow;
  using RW = Rows<kLow ? MODE : kKvInt8, DP, PAD, 32>;  // (16 bits: not used)
  constexpr int DB = BK::DB, kRowB = BK::kRowB, kTR = 32;
  constexpr int kSideB = 32 * kRowB;  // bytes of a wave's keys (or values); both: 32 rows of DP sums in fp32
  constexpr int kPieces = DP / 8;     // 16-byte pieces of a row
  constexpr int NL = kSideB / 1024;   // LDS-DMA loads of a side
  __shared__ __align__(16) uint8_t lds[kWaves][2 * kSideB];
  __shared__ __align__(16) float s_scale[kLow ? kWaves : 1][2][32];
  __shared__ float s_m[kWaves][32], s_l[kWaves][32];
  __shared__ typename BK::Odd s_odd[kWaves];

  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int D = PAD ? args_here().c.D : DP;
  const int rowb = static_cast<int>(kv_row_bytes(MODE, D)), sb = static_cast<int>(kv_scale_bytes(MODE, D));
  const Run run = run_of(args_here());
  if (run.last <= run.first) return;
  Segment sg = segment_at(args_here(), run.first);
  if (sg.s.tiles == 0) return;
  lds_u8* const kt = (lds_u8*)lds[wv];
  lds_u8* const vt = kt + kSideB;
  const uint32_t k_addr = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(kt));

  do {
    const ChunkArgs& a = args_here();
    const KvCache& cc = a.c;
    const Walk wk = walk_of(a, sg.s, sg.tile);
    const Share sh = share_of(a, run, sg, wk);
    if (!sh.whole && sh.u0 >= sh.u1) continue;
    const int hk = sg.head / a.head_tiles, lane = lane_here();
    Pages pages{-1, -(1 << 30), 0};
    // The v-th 32 keys of the walk: which 16 of them have a page, with the pages looked up.
    auto bits = [&](int v) __attribute__((always_inline)) {
      pages.need(a, sg, wk, v >> 1);
      return (pages.bits(v >> 1) >> (2 * (v & 1))) & 3u;
    };
    auto key_of = [&](int v) __attribute__((always_inline)) { return wk.tile(v >> 1) * kKeys + 32 * (v & 1); };
    RW x;
    auto load = [&](int v) __attribute__((always_inline)) {
      if constexpr (kLow) {
        const int k = key_of(v);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          load_rows(x, cc, lane, h, pages.of(v >> 1, 2 * (v & 1) + h), row_at(a, hk, k + 16 * h), rows_at(sg, k + 16 * h), rowb, sb, D);
      }
    };
    // load i of a side fills the 16-byte places 64 i + lane; the first half of them is the first page's
    auto dma = [&](int v, int side) __attribute__((always_inline)) {
      const int k = key_of(v);
      const KvSide& sd = side ? cc.v : cc.k;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t pg = pages.of(v >> 1, 2 * (v & 1) + h);
        const i32x4_t rs = rsrc4(sd.codes + (max(pg, int64_t(0)) * sd.page_b + row_at(a, hk, k + 16 * h) * rowb),
                                 pg < 0 ? 0u : static_cast<uint32_t>(rows_at(sg, k + 16 * h) * rowb));
#pragma unroll
        for (int i = 0; i < NL / 2; ++i) {
          const int at = 64 * (NL / 2 * h + i) + lane, r = at / kPieces, p = (at % kPieces) ^ (side ? value_swz<DP>(r) : key_swz<DP>(r));
          dma16(k_addr + side * kSideB + 1024 * (NL / 2 * h + i), !PAD || 8 * p < D ? static_cast<uint32_t>((r & 15) * rowb + 16 * p) : kOut, rs);
        }
      }
    };
    // everything but the last `NL` loads has landed (more: the other side's are on their way)
    auto landed = [&](bool more) __attribute__((always_inline)) {
      if (more)
        asm volatile("s_waitcnt vmcnt(%0)" : : "i"(NL) : "memory");
      else
        asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
    };
    auto lds_done = [] __attribute__((always_inline)) { asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); };
    const int v0 = 2 * sh.u0 + wv, v1 = 2 * sh.u1;
    const Place pl = place_of_rows(a, sg, wk, lane, 0);
    BK bk;
    bk.load_q(a, sg, pl, lane);
    float down = 1.0f;
    for (bool careful = false;;) {
      bk.clear();
      uint32_t in = 0;
      if (v0 < v1) {
        in = bits(v0);
        if constexpr (kLow) {
          load(v0);
        } else {
          dma(v0, 0);
          dma(v0, 1);
        }
      }
      for (int v = v0; v < v1; v += kWaves) {
        const int k0 = key_of(v);
        const uint32_t now = in;
        const bool more = v + kWaves < v1;
        float big = 0.0f;
        if constexpr (kLow) {
          big = store_rows(x, lane, lds[wv], lds[wv] + kSideB, s_scale[wv][0], s_scale[wv][1], 0, down);
          lds_done();  // (other lanes' rows are read below)
        }
        if constexpr (kLow) {
          if (more) {
            in = bits(v + kWaves);
            load(v + kWaves);
          }
        }
        if (careful) {
          if constexpr (!kLow) landed(false);
          BK::note_odd(s_odd[wv], pl, a.sinks, k0, now, vt);
          lds_done();
          BK::drop_odd(vt, 32);
          lds_done();
        }
        if constexpr (kLow) {
          if (BK::sees(pl, a.sinks, k0, 32)) bk.template step<1, kRest<MODE, DT, 1>>(pl, lane, a.sinks, k0, now, big, kt, vt, s_scale[wv][0], s_scale[wv][1], [] {});
          lds_done();  // (before the next rows take their places)
        } else {  // (keys that no row sees, at most the rest of 64 of them, are masked like others)
          landed(true);  // (the keys)
          bk.template step<1, kRest<MODE, DT, 1>>(pl, lane, a.sinks, k0, now, big, kt, vt, nullptr, nullptr, [&] __attribute__((always_inline)) {
            lds_done();
            if (more) {
              in = bits(v + kWaves);
              dma(v + kWaves, 0);
            }
            landed(more);  // (the values)
          });
          lds_done();
          if (more) dma(v + kWaves, 1);
        }
      }
      bk.pin();
      if (careful || !__syncthreads_or(bk.again())) {
        if (careful) bk.add_odd(s_odd[wv]);
        break;
      }
      if (kLow && __syncthreads_or(bk.high())) down = pow2(-kDown);
      careful = true;
      BK::no_odd(s_odd[wv]);
    }

    // ---- the waves' means: [element][row] of each wave, then a wave joins a quarter of the elements
    bk.finish(down);
    const int end = lane_here(), col = end & 31, hf = end >> 5;
    const ChunkArgs& z = args_here();
    float* const mine = reinterpret_cast<float*>(lds[wv]);
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) mine[(32 * d + 8 * (i / 4) + 4 * hf + i % 4) * 32 + col] = bk.acc[d][i];
    if (hf == 0) {
      s_m[wv][col] = bk.m;
      s_l[wv][col] = bk.l;
    }
    __syncthreads();
    float m = -kInf, l = 0.0f, f[kWaves];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) m = fmaxf(m, s_m[w][col]);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      f[w] = part_weight(s_l[w][col], s_m[w][col], m);
      l += f[w];
    }
    const float inv = over_all(l);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) f[w] = part_share(f[w], inv);
    // this lane's elements: DP / 8 from e0 on
    constexpr int NE = DP / 8;
    const int e0 = (2 * wv + hf) * NE;
    float o[NE];
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      o[j] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float v = reinterpret_cast<const float*>(lds[w])[(e0 + j) * 32 + col];
        o[j] = f[w] == 0.0f ? o[j] : __builtin_fmaf(v, f[w], o[j]);
      }
    }
    __syncthreads();  // (before these places are written again)
    if (!sh.whole) {
      float* const to = ws + static_cast<int64_t>(part_at(run.i, sh.u0)) * kPart<DP, kTR> + col;
#pragma unroll
      for (int j = 0; j < NE; ++j) to[(e0 + j) * kTR] = o[j];
      if (wv == 0 && hf == 0) {
        to[DP * kTR] = m;
        to[(DP + 1) * kTR] = l;
      }
    } else if (pl.mine) {
      const int64_t to = sg.s.q0 + pl.token;
      uint16_t* const out = z.out.p + to * z.out.row + pl.head * z.out.head + e0;
#pragma unroll
      for (int j = 0; j < NE; j += 8) {
        if (PAD && e0 + j >= D) break;
        u32x4_t w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = round16x2<DT>(o[j + 2 * i], o[j + 2 * i + 1]);
        *reinterpret_cast<u32x4_t*>(out + j) = w;
      }
      if (z.lse && wv == 0 && hf == 0) z.lse[to * z.Hq + pl.head] = l == 0.0f ? -kInf : (m - BK::kW + __builtin_amdgcn_logf(l)) * 0.693147181f;
    }
  } while (next_segment(args_here(), run, sg));
}

// Joins the parts of a segment that several runs share: the workgroups of run i do the one that begins in run i and
// goes on behind it; a workgroup 32 elements, a thread a row and TR / 8 of them.
template <int MODE, int DT, int DP, int TR>
__global__ __launch_bounds__(kThreads) void chunk_join_kernel(ChunkArgs a, const float* __restrict__ ws) {
  constexpr int NE = TR / 8;
  // parts whose loads are on their way together (tiles of 128 rows have 16 loads of a thread in each: document of 16384 rows with
  // 1, 2 and 4 parts 312.7, 314.3, 319.9 us, 5 chunks over int4 578, 581, 585; 16 x 3 drafts behind up to 8000 int8 tokens one
  // after the other 51.2 us, by four 48.2)
  constexpr int kAtOnce = TR == 128 ? 1 : 4;
  const int run = blockIdx.x;
  const Shared sh = shared_from(a, run);
  if (sh.parts == 0) return;
  const Segment& sg = sh.sg;
  const Walk& wk = sh.wk;
  const int hk = sg.head / a.head_tiles, ht = sg.head - hk * a.head_tiles, hn = min(a.tile_heads, a.g - ht * a.tile_heads);
  const int r = threadIdx.x % TR, e = 32 * blockIdx.y + NE * (threadIdx.x / TR);
  const int token = wk.row0 + r / a.tile_heads, hr = r % a.tile_heads, head = hk * a.g + ht * a.tile_heads + hr;
  if (token > wk.row1 || r >= a.tokens * a.tile_heads || hr >= hn || e >= a.c.D) return;
  float m = -kInf, l = 0.0f, o[NE];
#pragma unroll
  for (int j = 0; j < NE; ++j) o[j] = 0.0f;
  for (int i = 0; i <= sh.parts; i += kAtOnce) {
    float mi[kAtOnce], li[kAtOnce], x[kAtOnce][NE];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int part = min(i + k, sh.parts);
      const float* const p = ws + static_cast<int64_t>(part_at(run + part, part)) * kPart<DP, TR> + r;
      mi[k] = p[DP * TR];
      li[k] = p[(DP + 1) * TR];
#pragma unroll
      for (int j = 0; j < NE; ++j) x[k][j] = p[(e + j) * TR];
    }
    const int n = min(kAtOnce, sh.parts + 1 - i);
    const float m0 = m, l0 = l;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) m = fmaxf(m, mi[k]);
    float w[kAtOnce];
    l = part_weight(l0, m0, m);
    const float before = l;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      w[k] = k < n ? part_weight(li[k], mi[k], m) : 0.0f;
      l += w[k];
    }
    const float inv = over_all(l), f0 = part_share(before, inv);
#pragma unroll
    for (int j = 0; j < NE; ++j) o[j] *= f0;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (k >= n) break;
      const float f = part_share(w[k], inv);
#pragma unroll
      for (int j = 0; j < NE; ++j) o[j] = __builtin_fmaf(x[k][j], f, o[j]);
    }
  }
  const int64_t to = sg.s.q0 + token;
  uint16_t* const out = a.out.p + to * a.out.row + head * a.out.head + e;
#pragma unroll
  for (int j = 0; j < NE; j += 4) {
    if (e + j >= a.c.D) break;
    *reinterpret_cast<u32x2_t*>(out + j) = u32x2_t{round16x2<DT>(o[j], o[j + 1]), round16x2<DT>(o[j + 2], o[j + 3])};
  }
  if (a.lse && e == 0)
    a.lse[to * a.Hq + head] = l == 0.0f ? -kInf : (m - kUpW<MODE, DT> + __builtin_amdgcn_logf(l)) * 0.693147181f;
}

template <int MODE, int DT, int DP, bool PAD, int TR>
hipError_t chunk_go(const ChunkArgs& a, float* ws, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(8 * ceil_div(a.runs, 8)));
  if constexpr (TR == 32)
    chunk_narrow_kernel<MODE, DT, DP, PAD><<<grid, kThreads, 0, s>>>(a, ws);
  else
    chunk_wide_kernel<MODE, DT, DP, PAD, TR / 32><<<grid, kThreads, 0, s>>>(a, ws);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || a.runs == 1 || a.single) return err;
  chunk_join_kernel<MODE, DT, DP, TR><<<dim3(static_cast<uint32_t>(a.runs - 1), static_cast<uint32_t>(ceil_div(a.c.D, 32))), kThreads, 0, s>>>(a, ws);
  return hipGetLastError();
}

template <int MODE, int DT, int DP, bool PAD>
hipError_t chunk_by_rows(const ChunkArgs& a, float* ws, hipStream_t s) {
  return a.tile_rows == 128  ? chunk_go<MODE, DT, DP, PAD, 128>(a, ws, s)
         : a.tile_rows == 64 ? chunk_go<MODE, DT, DP, PAD, 64>(a, ws, s)
                             : chunk_go<MODE, DT, DP, PAD, 32>(a, ws, s);
}

template <int MODE, int DT>
hipError_t chunk_by_size(const ChunkArgs& a, float* ws, hipStream_t s) {
  const int D = a.c.D;
  if (D == 64) return chunk_by_rows<MODE, DT, 64, false>(a, ws, s);
  if (D == 128) return chunk_by_rows<MODE, DT, 128, false>(a, ws, s);
  if (D == 256) return chunk_by_rows<MODE, DT, 256, false>(a, ws, s);
  if (D < 64) return chunk_by_rows<MODE, DT, 64, true>(a, ws, s);
  return D < 128 ? chunk_by_rows<MODE, DT, 128, true>(a, ws, s) : chunk_by_rows<MODE, DT, 256, true>(a, ws, s);
}

template <int MODE>
hipError_t chunk_mode(const ChunkArgs& a, void* ws, hipStream_t s) {
  float* const w = static_cast<float*>(ws);
  return a.c.dtype == kF16 ? chunk_by_size<MODE, kF16>(a, w, s) : chunk_by_size<MODE, kBF16>(a, w, s);
}

}  // namespace
}  // namespace fq
