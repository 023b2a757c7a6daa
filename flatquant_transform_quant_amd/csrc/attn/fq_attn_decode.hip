// Attention of one new token per sequence over the paged cache.
//
// For a cache head and its g query heads: s[t, h] = <q_h, k_t>, p = softmax over t, o_h = sum_t
// p[t, h] v_t.  Every cached byte is used for up to 16 heads at once, so the products run on the
// matrix cores with the heads as the 16 columns of a tile (heads beyond 16 take further tiles, which read
// the cache again) and the kernel is bound by reading the cache: int8, 8 cache heads of 128, 64 query heads, 64
// sequences of 1047 to 16384 tokens (756 MB) 148 us, 5.1 TB/s, two of up to 131072 (492 MB) 97 us, 5.0;
// a large copy moves 5.2.  4 bits are bound by the vector instructions that widen them: 128 sequences of
// the same lengths (783 MB) 171 us in int4, 174 in E2M1, 4.6 and 4.5 TB/s.  Small calls are a chain of latencies: workgroups
// start over 2 to 4 us, a run's plan takes 1.5 to 3, its pages and first keys 3, a step of 128 tokens 2 (3 at
// full bandwidth), the join 5 (37 sequences of up to 2000 tokens, E4M3, 39 MB: 20.4 us).
//
// One wave and 32 tokens (two subtiles of 16), v_mfma_f32_16x16x32:
//   S^T = K Q^T: the A operand's row is a token, so a lane reads pieces of one key row straight
//     from memory into operand position -- no LDS, no transpose.  Lane l ends with tokens
//     16 a + 4 (l / 16) + 0..3 of both subtiles a, for head l % 16.
//   O^T = V^T P^T: those 8 weights of a lane are, rounded to 16 bits, its B operand as they
//     stand (contraction slot j of lane group l / 16 is token 16 (j / 4) + 4 (l / 16) + j % 4).
//     V^T's row is an element d; a lane reads EC consecutive elements of its 8 tokens and pairs
//     them across tokens with byte permutes: product jj takes element EC (l % 16) + jj.
// Codes enter the products as f16 numbers, exactly but for what is said of E2M1 (16-bit caches: as they are):
//   int8, int4: the code plus 128 or 8 (u >= 0) in the low bits of a half is the f16 subnormal
//     u 2^-24, so widening costs a byte permute or a mask; one packed fused multiply-add makes it
//     the number (u - 128) 2^-9 or (u - 8) 2^-9, exactly.  (Subnormals themselves as operands lose
//     accuracy in the products' internal alignment -- scores were off by 2^-17 -- and a bias left
//     in and taken off the sums costs as much where a row's codes are small.)  Nibbles masked at
//     bits 4..7 are 16 u: q carries 1/16 at those elements, the output is divided by 16.
//   E4M3, E2M1: the converting instructions; E2M1 takes its group's power of two, relative to
//     the largest of the 32 tokens (keys) or to a running reference (values), along with it, and 2^13 (2^12) more:
//     a group 2^26 (2^25) smaller is still of normal f16 numbers, one 2^36 smaller is gone.
// A bf16 q is brought to f16 by a power of two per row (28 binades keep full precision).  The
// value scale of a token multiplies its weight: w = p scale 2^-R rounded to f16, with R a
// running reference exponent, so that w stays in range.
// The weights are the second product's operand and have its type: 11 bits (8 where the cache is bf16), and in f16
// no less than 2^-24; kUpP below puts them at the upper end of that.  Their rounding would be most of the
// result's error.  With at most 8 heads in a group the
// tile has columns to spare: they take the same heads with the remainders w - f16(w) as weights, so
// the weights count with twice the bits and the matrix cores have no more to do.  The remainders go in
// times 2^11: those of weights below 2^-14, where f16 has fewer bits, keep theirs.  With more heads there is no
// such room: a weight is off by 2^-11 (2^-8) of itself, or 2^-32 of the largest one (2^-30 where it carries a
// scale), and a token whose scale is below 2^-19 of the largest in its sequence loses bits in proportion.
// Softmax statistics are fp32: the running maximum m (base-2 scores) is only moved when a score
// passes m + 8 (weights then reach 2^8, far inside f16's range), so the common tile has no
// cross-lane step and no rescaling.
//
// Split: the units of work are 128 tokens (4 waves x 32) of a (sequence, cache head, head tile);
// all units in order are dealt to the grid in equal runs, whatever the lengths; a segment counts two
// or three units more than it has, for its page lookup, first loads and rows out (else the runs over
// many short segments end last: the 64 sequences above, int8, 153 us without, 150, 147, 149, 155 with one
// to four; the 128 in int4 189, 182, 175, 171, 172, in E2M1 191, 184, 178, 174, 175).  A run that
// holds only part of a segment leaves its unnormalised sums and (m, l) in the workspace, and a second
// launch joins them in a fixed order.  A segment's first loads are under way while the rows of the one
// before are written.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "fq_attn_dev.h"

namespace fq {
namespace {

constexpr int kThreads = 256, kWaves = 4;
constexpr int kTile = 32;                    // tokens of a wave's step
constexpr int kUnit = kWaves * kTile;        // tokens of a unit
constexpr int kBatch = 31;                   // steps per fetch of the block table (64 subtiles cover one step more)
constexpr int kMaxGrid = 1024;               // workgroups of a launch at most: four on each of 256 CUs
constexpr int kHeldLengths = 512;            // lengths kept in LDS (those of later sequences are read again)
constexpr float kLazy = 8.0f;                // base-2 slack of the running maximum
constexpr float kInf = __builtin_inff();

// Exponents that widen the range of the f16 operands at no cost (all exact, taken off again at the end):
//   kUpP: of the weights.  They reach 2^8 above the running maximum's, and at most 2^2 more by a token's value scale
//     (see ref_lim), so this ends at 2^15.
//   kUpK, kUpV: of E2M1 keys and values, at most 6 (values 6 2^1, see ref), so these end below 2^16.
template <int MODE, int PDT>
constexpr int kUpP = PDT != kF16 ? 0 : (MODE == kKv16 || MODE == kKvFp4) ? 7 : 5;
constexpr int kUpK = 13, kUpV = 12;

template <int MODE>
constexpr int kBits = MODE == kKv16 ? 16 : (MODE == kKvInt8 || MODE == kKvE4M3) ? 8 : 4;

// Sizes of a lane's pieces.  DP: D rounded up to 64, 128 or 256; PAD: D < DP, where pieces at
// or past D are zeros (pieces are then 8 elements, which D's multiple of 8 never cuts).
template <int MODE, int DP, bool PAD>
struct Shape {
  static constexpr int bits = kBits<MODE>;
  static constexpr int CE = PAD ? 8 : (128 / bits < DP / 4 ? 128 / bits : DP / 4);  // elements of a key piece
  static constexpr int KC = DP / (4 * CE);                                         // pieces of a lane in a key row
  static constexpr int KW = CE * bits / 32;                                        // dwords of a piece
  static constexpr int EC = DP / 16 < 8 ? DP / 16 : 8;                             // elements of a value piece
  static constexpr int NH = DP / (16 * EC);
  static constexpr int VB = EC * bits / 8;                                         // bytes of a value piece
  static constexpr int VW = VB < 4 ? 1 : VB / 4;
  static constexpr int KS = DP / 32;                                               // products of a score
  // units that a segment's beginning and end (page lookup, first loads, rows out) count as, see above
  static constexpr int start = bits == 4 ? 3 : 2;
  // Workgroups of a CU (waves of a SIMD): as many as registers and, at 256, LDS hold without spills in
  // the loop.  us with 1, 2, 3, 4: the 64 sequences above, int8 at 128: 182, 148, 173, 483; the 128, int4:
  // 308, 198, 171, 241; 32 of 147 to 4096, 32 heads on 8, 16 bits at 128: 33, 38, 52, 82; 32 of 535 to 4096, 16
  // heads on 4, at 256, 16 bits: 45, 111, 51, 59, int8: 35, 35, 50, 62, int4: 31, 29, 46, 58; 64 of 1041 to 8192,
  // 16 heads at 64, int8: 167, 106, 94, 98, int4: 146, 93, 79, 74, 16 bits: 164, 163, 169, 167 -- and 37 of 43 to
  // 2000 there, E4M3: 29, 21, 20, 20.
  static constexpr int per_cu = DP == 256 ? (bits == 16 ? 1 : 2) : DP == 64 ? 4 : bits == 4 ? 3 : 2;
};

template <int MODE, int DP, bool PAD>
struct Keys {
  using S = Shape<MODE, DP, PAD>;
  uint32_t w[2][S::KC][S::KW];
  f32x4_t scale[MODE == kKv16 || MODE == kKvFp4 ? 1 : 2];
  uint32_t e8[MODE == kKvFp4 ? 2 : 1][S::KC];
};
template <int MODE, int DP, bool PAD>
struct Values {
  using S = Shape<MODE, DP, PAD>;
  uint32_t w[8][S::NH][S::VW];
  f32x4_t scale[MODE == kKv16 || MODE == kKvFp4 ? 1 : 2];
  uint32_t e8[MODE == kKvFp4 ? 8 : 1][S::NH];
};

constexpr uint32_t kOut = 0x80000000u;  // an offset past every resource

template <int W>
__device__ __forceinline__ void load_words(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t (&o)[W]) {
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

template <int DT>
__device__ __forceinline__ uint32_t h2(float a, float b) { return round16x2<DT>(a, b); }

// Operand of 8 key elements from a piece's dwords (e: which 8); s: the E2M1 group's factor.
template <int MODE, int KW>
__device__ __forceinline__ u32x4_t key_operand(const uint32_t (&w)[KW], int e, float s) {
  if constexpr (MODE == kKv16) {
    return u32x4_t{w[0], w[1], w[2], w[3]};
  } else if constexpr (MODE == kKvInt8) {
    const uint32_t a = w[2 * e] ^ 0x80808080u, b = w[2 * e + 1] ^ 0x80808080u;
    return u32x4_t{unbias_f16(__builtin_amdgcn_perm(0u, a, 0x0C010C00u), kMinus128), unbias_f16(__builtin_amdgcn_perm(0u, a, 0x0C030C02u), kMinus128),
                   unbias_f16(__builtin_amdgcn_perm(0u, b, 0x0C010C00u), kMinus128), unbias_f16(__builtin_amdgcn_perm(0u, b, 0x0C030C02u), kMinus128)};
  } else if constexpr (MODE == kKvE4M3) {
    return u32x4_t{fp8_to_f16x2<false>(w[2 * e]), fp8_to_f16x2<true>(w[2 * e]), fp8_to_f16x2<false>(w[2 * e + 1]),
                   fp8_to_f16x2<true>(w[2 * e + 1])};
  } else if constexpr (MODE == kKvInt4) {  // order n0 n4 n1 n5 n2 n6 n3 n7, the odd ones x 16
    const uint32_t x = w[e] ^ 0x88888888u, y = x >> 8;
    return u32x4_t{unbias_f16(x & 0x000F000Fu, kMinus8), unbias_f16(x & 0x00F000F0u, kMinus128), unbias_f16(y & 0x000F000Fu, kMinus8),
                   unbias_f16(y & 0x00F000F0u, kMinus128)};
  } else {
    return u32x4_t{fp4_to_f16x2<0>(w[e], s), fp4_to_f16x2<1>(w[e], s), fp4_to_f16x2<2>(w[e], s), fp4_to_f16x2<3>(w[e], s)};
  }
}

// Element of q at place j of such an operand, and the factor it carries.
template <int MODE>
__device__ __forceinline__ constexpr int q_place(int j) {
  constexpr int order[8] = {0, 4, 1, 5, 2, 6, 3, 7};
  return MODE == kKvInt4 ? order[j] : j;
}

// max over the four lanes that share l % 16
__device__ __forceinline__ float column_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float column_sum(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}
__device__ __forceinline__ int wave_imax(int v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v = max(v, __shfl_xor(v, o));
  return v;
}

// the same value, opaque to the compiler from here on
__device__ __forceinline__ uint32_t here(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}

__device__ __forceinline__ int32_t length_of(const DecodeArgs& a, int b) {
  const int64_t reach = static_cast<int64_t>(a.bt.width) << a.c.page_log;
  return static_cast<int32_t>(max(int64_t(0), min(static_cast<int64_t>(a.lengths[b]), reach)));
}
__device__ __forceinline__ int32_t units_of(int32_t n) { return n / kUnit + (n % kUnit != 0); }
// what a segment counts as when the work is dealt (see the top)
__device__ __forceinline__ int32_t weight_of(int32_t n, int start) { return n > 0 ? units_of(n) + start : 0; }

// Workgroup i of `runs` (at most `total`; all below 2^31, which the host checks) has the units from
// start(i) = i total / runs up to start(i + 1); unit u is in run of(u).
struct Runs {
  uint32_t total, runs, q, r;
  __device__ Runs(uint32_t units, uint32_t grid) : total(units), runs(min(units, grid)) {
    q = runs ? total / runs : 0u;
    r = total - q * runs;
  }
  __device__ uint32_t start(uint32_t i) const { return i * q + i * r / runs; }
  __device__ uint32_t of(uint32_t u) const { return static_cast<uint32_t>(((u + uint64_t(1)) * runs - 1) / total); }
};

template <int MODE, int DT, int DP, bool PAD>
__global__ __launch_bounds__(kThreads, (Shape<MODE, DP, PAD>::per_cu)) void decode_kernel(DecodeArgs a, float* __restrict__ part, int32_t nht, int32_t gh,
                                                             bool single) {
  using S = Shape<MODE, DP, PAD>;
  constexpr bool kScaled = MODE == kKvInt8 || MODE == kKvE4M3 || MODE == kKvInt4;  // a scale per token
  constexpr int PDT = MODE == kKv16 ? DT : kF16;                                   // operands' type
  constexpr float kCode = MODE == kKvInt8 || MODE == kKvInt4 ? 512.0f : 1.0f;       // 1 / the operand's unit
  constexpr float kUp = PDT == kF16 ? 2048.0f : 1.0f;                               // of the weights' remainders
  constexpr int LDH = 17;  // row pitch of the output exchange (heads)
  __shared__ float s_o[kWaves][DP * LDH];
  __shared__ float s_m[kWaves][16], s_l[kWaves][16];
  __shared__ int32_t s_sum[kWaves], s_len[kHeldLengths], s_b, s_at;

  const KvCache& c = a.c;
  const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, kb = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int D = PAD ? c.D : DP;
  const int per_b = c.Hkv * nht;  // segments of a sequence
  const int rowb = D * S::bits / 8;
  const int sb = MODE == kKvFp4 ? 2 * ((D + 63) / 64) : 4;

  // ---- this workgroup's run of units
  int u = 0, u_end = 0;  // units from the start of sequence b on
  int b = 0;
  if (single) {  // a workgroup a segment: no plan, no join
    b = blockIdx.x / per_b;
    u = blockIdx.x - b * per_b;
    u_end = u + 1;
  } else if (a.B <= 64) {  // the plan below with a sequence a lane, by each wave for itself (1 us less a call)
    const int32_t n = lane < a.B ? length_of(a, lane) : 0;
    s_len[lane] = n;
    const int weight = weight_of(n, S::start), incl = wave_scan(weight);
    const Runs run(__builtin_amdgcn_readlane(incl, 63) * per_b, gridDim.x);
    if (blockIdx.x >= run.runs) return;
    const int first = __builtin_amdgcn_readfirstlane(run.start(blockIdx.x)), last = __builtin_amdgcn_readfirstlane(run.start(blockIdx.x + 1));
    b = __builtin_ctzll(__ballot(incl * per_b > first));
    const int at = __builtin_amdgcn_readlane(incl - weight, b) * per_b;
    u = first - at;
    u_end = last - at;
  } else {
    // the units of all sequences, then the sequence that holds the first unit: scans over the
    // lengths, 256 at a time; the first pass over them keeps the first scan
    int mine = 0, incl = 0, n0 = 0;
    for (int i = tid; i < a.B; i += kThreads) {
      const int32_t n = length_of(a, i);
      if (i < kHeldLengths) s_len[i] = n;
      mine += weight_of(n, S::start);
      if (i == tid) n0 = mine;
    }
    incl = wave_scan(n0);
    const int all = a.B <= kThreads ? incl : wave_scan(mine);
    if (lane == 63) s_sum[wv] = all;
    __syncthreads();
    const Runs run((s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3]) * per_b, gridDim.x);
    if (blockIdx.x >= run.runs) return;
    const int first = run.start(blockIdx.x), last = run.start(blockIdx.x + 1);
    int base = 0;
    for (int i0 = 0; i0 < a.B; i0 += kThreads) {
      const int i = i0 + tid;
      if (a.B > kThreads) {
        n0 = i < a.B ? weight_of(i < kHeldLengths ? s_len[i] : length_of(a, i), S::start) : 0;
        incl = wave_scan(n0);
        __syncthreads();
        if (lane == 63) s_sum[wv] = incl;
        __syncthreads();
      }
      int end = base + incl;
      for (int w = 0; w < wv; ++w) end += s_sum[w];
      if (first >= (end - n0) * per_b && first < end * per_b) {
        s_b = i;
        s_at = (end - n0) * per_b;
      }
      base += s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
      if (first < base * per_b) break;
    }
    __syncthreads();
    b = __builtin_amdgcn_readfirstlane(s_b);
    const int at = __builtin_amdgcn_readfirstlane(s_at);
    u = first - at;
    u_end = last - at;
  }

  bool first_seg = true;
  int32_t pages = -1;                 // lane 2 i + s: the page of subtile s of step (batch) + i
  int pages_b = -1, pages_t = -1;     // the sequence and first token they were fetched for
  const bool two = a.g <= 8;          // weights in two halves, see below
  // ---- the segment at hand: its sequence, length, heads and units, this wave's first token and steps
  int32_t n = 0;
  int nu = 0, seg = 0, ua = 0, ue = 0, t_first = 0, steps = 0;
  auto next_segment = [&]() __attribute__((always_inline)) {  // false: nothing of it is this run's
    int nw;
    for (;; ++b) {
      n = __builtin_amdgcn_readfirstlane(!single && b < kHeldLengths ? s_len[b] : length_of(a, b));
      nw = single ? 1 : weight_of(n, S::start);
      if (u < nw * per_b) break;
      u -= nw * per_b;
      u_end -= nw * per_b;
    }
    nu = single ? max(1, units_of(n)) : units_of(n);
    seg = __builtin_amdgcn_readfirstlane(u / nw);
    const int start = single ? 0 : S::start, at = u - seg * nw, take = min(nw - at, u_end - u);
    u += take;
    ua = max(0, at - start);
    ue = single ? nu : at + take - start;
    // this wave's steps: tokens kUnit (ua + i) + kTile wv ..
    t_first = kUnit * ua + kTile * wv;
    const int t_last = min(n, kUnit * ue);
    steps = t_first < t_last ? (t_last - t_first + kUnit - 1) / kUnit : 0;
    return ua < ue;
  };

  auto fetch_pages = [&](int step) __attribute__((always_inline)) {
    const int64_t t = static_cast<int64_t>(t_first) + static_cast<int64_t>(kUnit) * (step + (lane >> 1)) + 16 * (lane & 1);
    pages = t < n ? kv_page(a.bt, b, static_cast<int32_t>(t), c.page_log, c.pages) : -1;
    pages_b = b;
    pages_t = t_first + kUnit * step;
  };
  const uint32_t koff = r16 * rowb + kb * (S::CE * S::bits / 8), keoff = r16 * sb + (S::CE * kb) / 32;
  const uint32_t voff = 4 * kb * rowb + r16 * S::VB, veoff = 4 * kb * sb + (S::EC * r16) / 32;
  // Loads go through a buffer resource per subtile that starts at its first row and ends behind
  // its last token (at nothing for a subtile without a page): rows past n, and the pieces of
  // padded lanes, whose offset is kOut, are zeros without a branch.
  auto rows_of = [&](int step, int s) __attribute__((always_inline)) {
    // (as a scalar: a clamp runs in a vector register, and a resource there costs a loop a load)
    return __builtin_amdgcn_readfirstlane(max(0, min(16, n - (t_first + kUnit * step + 16 * s))));
  };
  auto resource = [&](const uint8_t* base, int64_t page_b, int row_b, int step, int s, int idx) __attribute__((always_inline)) {
    const int32_t pg = __builtin_amdgcn_readlane(pages, 2 * idx + s);
    const int off = (t_first + kUnit * step + 16 * s) & ((1 << c.page_log) - 1);
    const int bytes = rows_of(step, s) * row_b;
    const int64_t row = (static_cast<int64_t>(seg / nht) << c.page_log) + off;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base) + (max(pg, 0) * page_b + row * row_b), static_cast<int16_t>(0),
                                             pg < 0 ? 0 : bytes, kBufferWord3);
  };
  auto load_keys = [&](Keys<MODE, DP, PAD>& x, int step, int idx) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const auto rc = resource(c.k.codes, c.k.page_b, rowb, step, s, idx);
#pragma unroll
      for (int p = 0; p < S::KC; ++p)
        load_words<S::KW>(rc, (PAD && S::CE * (4 * p + kb) >= D ? kOut : koff) + p * (4 * S::CE * S::bits / 8), x.w[s][p]);
      if constexpr (MODE != kKv16) {
        const auto rs = resource(c.k.scale, c.k.scale_page_b, sb, step, s, idx);
        if constexpr (MODE == kKvFp4) {
#pragma unroll
          for (int p = 0; p < S::KC; ++p)
            x.e8[s][p] = __builtin_amdgcn_raw_buffer_load_b8(rs, (PAD && S::CE * (4 * p + kb) >= D ? kOut : keoff) + S::CE * 4 * p / 32, 0, 0);
        } else {
          x.scale[s] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, 16 * kb, 0, 0));
        }
      }
    }
  };
  auto load_values = [&](Values<MODE, DP, PAD>& x, int step, int idx) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const auto rc = resource(c.v.codes, c.v.page_b, rowb, step, s, idx);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < S::NH; ++h) {
          const uint32_t o = (PAD && 128 * h + S::EC * r16 >= D ? kOut : voff) + i * rowb + h * (16 * S::VB);
          if constexpr (S::VB == 2)
            x.w[4 * s + i][h][0] = __builtin_amdgcn_raw_buffer_load_b16(rc, o, 0, 0);
          else
            load_words<S::VW>(rc, o, x.w[4 * s + i][h]);
        }
      if constexpr (MODE != kKv16) {
        const auto rs = resource(c.v.scale, c.v.scale_page_b, sb, step, s, idx);
        if constexpr (MODE == kKvFp4) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < S::NH; ++h)
              x.e8[4 * s + i][h] = __builtin_amdgcn_raw_buffer_load_b8(rs, (PAD && 128 * h + S::EC * r16 >= D ? kOut : veoff) + i * sb + 4 * h, 0, 0);
        } else {
          x.scale[s] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, 16 * kb, 0, 0));
        }
      }
    }
  };
  // the rows a lane's four tokens of a subtile have left (0 .. 4): for steps that are not whole
  auto mine = [&](int step, int s, int idx) __attribute__((always_inline)) {
    const int rows = rows_of(step, s);
    return (__builtin_amdgcn_readlane(pages, 2 * idx + s) < 0 ? 0 : rows) - 4 * kb;
  };

  // the first step's loads of a segment
  Keys<MODE, DP, PAD> kx;
  Values<MODE, DP, PAD> vx;
  auto begin = [&]() __attribute__((always_inline)) {
    if (steps > 0) {
      if (pages_b != b || pages_t != t_first) fetch_pages(0);
      load_keys(kx, 0, 0);
      load_values(vx, 0, 0);
    }
  };

  if (!next_segment()) return;
  begin();
  for (bool more = true; more;) {
    const int b0 = b, hk = seg / nht, ht = seg - hk * nht;
    const bool all = ua == 0 && ue == nu;
    // This lane's head within the group.  Of at most 8 heads the tile's columns 8 .. 15 take the same
    // heads again, with what the rounding of the weights left over: their sums are added to the others'.
    const int head = ht * 16 + (two ? r16 & 7 : r16);
    const bool my_head = head < a.g;
    const float up = r16 < 8 ? 1.0f : kUp, minus = r16 < 8 ? -0.0f : -kUp;

    // ---- state of the segment
    f32x4_t acc[S::NH][S::EC];
#pragma unroll
    for (int h = 0; h < S::NH; ++h)
#pragma unroll
      for (int j = 0; j < S::EC; ++j) acc[h][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    float m = -kInf, l = 0.0f;
    int ref = -100000;      // exponent R of the value scales (wave-uniform); far below any
    float ref_inv = 0.0f;   // 2^-R
    float ref_lim = 0.0f;   // a scale at or above 2^(R + 2) moves R

    // ---- q as the B operand, and the column's constants
    u32x4_t qf[S::KS];
    float cq = a.scale * 1.44269504f;  // (times kCode with q's exponent below: that product alone could overflow)
    {
      const uint16_t* qp = a.q.p + b0 * a.q.row + static_cast<int64_t>(hk * a.g + (my_head ? head : 0)) * a.q.head;
      u32x4_t raw[S::KS];
#pragma unroll
      for (int ks = 0; ks < S::KS; ++ks) {
        const int d = S::CE * (4 * (ks / (S::CE / 8)) + kb) + 8 * (ks % (S::CE / 8));
        raw[ks] = u32x4_t{0u, 0u, 0u, 0u};
        if (my_head && d < D) raw[ks] = *reinterpret_cast<const u32x4_t*>(qp + d);
      }
      if constexpr (MODE == kKv16) {
#pragma unroll
        for (int ks = 0; ks < S::KS; ++ks) qf[ks] = raw[ks];
      } else {
        float top = 0.0f;
#pragma unroll
        for (int ks = 0; ks < S::KS; ++ks) {
          float x[8];
          kv_decode8<kKv16, DT>(raw[ks], 1.0f, 0, x);
#pragma unroll
          for (int j = 0; j < 8; ++j) top = fmaxf(top, __builtin_fabsf(x[j]));
        }
        // |q| < 2^(e + 1) at its largest; brought to [2^13, 2^14)
        const int e = static_cast<int>((__float_as_uint(column_max(top)) >> 23) & 0xFFu) - 127;
#pragma unroll
        for (int ks = 0; ks < S::KS; ++ks) {
          float x[8], y[8];
          kv_decode8<kKv16, DT>(raw[ks], 1.0f, 0, x);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            y[j] = __builtin_amdgcn_ldexpf(x[q_place<MODE>(j)], 13 - e);
            if (MODE == kKvInt4 && (j & 2)) y[j] *= 0.0625f;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) qf[ks][i] = h2<kF16>(y[2 * i], y[2 * i + 1]);
        }
        cq = __builtin_amdgcn_ldexpf(cq, e - 13 + (kCode == 512.0f ? 9 : 0));
      }
    }

    // base-2 scores of a step
    auto score = [&](const Keys<MODE, DP, PAD>& x, int step, int idx, bool whole, float (&s)[8]) __attribute__((always_inline)) {
      int ek = 0;  // E2M1: the tile's largest exponent
      if constexpr (MODE == kKvFp4) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int p = 0; p < S::KC; ++p) ek = max(ek, static_cast<int>(x.e8[s][p]));
        ek = __builtin_amdgcn_readfirstlane(wave_imax(ek));
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        f32x4_t z = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int ks = 0; ks < S::KS; ++ks) {
          constexpr int E = S::CE / 8;
          const float f = MODE == kKvFp4 ? (x.e8[t][ks / E] == 255u ? __builtin_nanf("") : pow2(static_cast<int>(x.e8[t][ks / E]) - ek + kUpK)) : 0.0f;
          z = mfma16x16x32<PDT>(key_operand<MODE, S::KW>(x.w[t][ks / E], ks % E, f), qf[ks], z);
        }
        const float cf = MODE == kKvFp4 ? __builtin_amdgcn_ldexpf(cq, ek - 127 - kUpK) : cq;
#pragma unroll
        for (int i = 0; i < 4; ++i) s[4 * t + i] = z[i] * (kScaled ? cf * x.scale[t][i] : cf);
      }
      if (!whole) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int left = mine(step, t, idx);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i >= left) s[4 * t + i] = -kInf;
        }
      }
    };

    // 16-bit values that are infinite or NaN.  Their products are formed apart, with weights of 1 (0 for a score
    // of -infinity), and they are left out of the weighted ones: a weight that rounds to 0 would make a NaN of
    // an infinity that every weight above 0 keeps.
    auto take_odd = [&](Values<MODE, DP, PAD>& x, const float (&s)[8]) __attribute__((always_inline)) {
      uint32_t odd = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int h = 0; h < S::NH; ++h)
#pragma unroll
          for (int w = 0; w < S::VW; ++w) odd |= not_finite16<DT>(x.w[i][h][w]);
      if (!__any(odd != 0)) return;
      u32x4_t one;
#pragma unroll
      for (int i = 0; i < 4; ++i) one[i] = h2<DT>(s[2 * i] > -kInf ? 1.0f : 0.0f, s[2 * i + 1] > -kInf ? 1.0f : 0.0f);
#pragma unroll
      for (int h = 0; h < S::NH; ++h)
#pragma unroll
        for (int w = 0; w < S::VW; ++w) {  // elements 2 w, 2 w + 1
          uint32_t a[4], b[4];
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            uint32_t& y0 = x.w[2 * p][h][w];
            uint32_t& y1 = x.w[2 * p + 1][h][w];
            const uint32_t m0 = not_finite16_mask<DT>(y0), m1 = not_finite16_mask<DT>(y1);
            a[p] = __builtin_amdgcn_perm(y1 & m1, y0 & m0, 0x05040100u);
            b[p] = __builtin_amdgcn_perm(y1 & m1, y0 & m0, 0x07060302u);
            y0 &= ~m0;
            y1 &= ~m1;
          }
          acc[h][2 * w] = mfma16x16x32<DT>(u32x4_t{a[0], a[1], a[2], a[3]}, one, acc[h][2 * w]);
          acc[h][2 * w + 1] = mfma16x16x32<DT>(u32x4_t{b[0], b[1], b[2], b[3]}, one, acc[h][2 * w + 1]);
        }
    };

    // their weights p = exp2(s - m), the running maximum and sum moved along
    auto weigh = [&](float (&s)[8]) __attribute__((always_inline)) {
      float top = s[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) top = fmaxf(top, s[i]);
      if (__any(top > m + kLazy)) {
        const float mn = fmaxf(m, column_max(top));
        const float f = mn == -kInf ? 1.0f : rescale(m, mn);
        m = mn;
        l *= f;
#pragma unroll
        for (int h = 0; h < S::NH; ++h)
#pragma unroll
          for (int j = 0; j < S::EC; ++j) acc[h][j] *= f;
      }
      const float ms = m == -kInf ? 0.0f : m - kUpP<MODE, PDT>;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[i] = __builtin_amdgcn_exp2f(s[i] - ms);
        l += s[i];
      }
    };

    // the weighted values
    auto add = [&](Values<MODE, DP, PAD>& x, int step, int idx, bool whole, float (&w)[8]) __attribute__((always_inline)) {
      auto move_ref = [&](int r) __attribute__((always_inline)) {  // sums to the reference 2^r
        const float f = ref < -1000 ? 0.0f : pow2(max(ref - r, -127));
#pragma unroll
        for (int h = 0; h < S::NH; ++h)
#pragma unroll
          for (int j = 0; j < S::EC; ++j) acc[h][j] *= f;
        ref = r;
      };
      if constexpr (MODE == kKvFp4) {
        int ev = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int h = 0; h < S::NH; ++h) ev = max(ev, x.e8[i][h] == 255u ? 0 : static_cast<int>(x.e8[i][h]));  // (255: NaN)
        if (__any(ev > ref + 1)) move_ref(__builtin_amdgcn_readfirstlane(wave_imax(ev)));
      }
      if constexpr (kScaled) {
        if (!whole) {  // (the scales of tokens past n may be anything)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int left = mine(step, t, idx);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (i >= left) x.scale[t][i] = 0.0f;
          }
        }
        float big = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) big = fmaxf(big, x.scale[i / 4][i % 4]);
        if (__any(big >= ref_lim)) {
          // (a tile of zero scales leaves the reference where it is)
          const int r = __builtin_amdgcn_readfirstlane(wave_imax(static_cast<int>((__float_as_uint(big) >> 23) & 0xFFu) - 127));
          if (r > ref && r > -127) {
            move_ref(r);
            ref_inv = pow2(min(-r, 127));
            ref_lim = r + 2 > 127 ? kInf : pow2(max(r + 2, -126));
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] *= x.scale[i / 4][i % 4] * ref_inv;
      }
      u32x4_t pf;
#pragma unroll
      for (int i = 0; i < 4; ++i) pf[i] = h2<PDT>(w[2 * i], w[2 * i + 1]);
      if (two) {  // (w - hi) up in the columns of the remainders, else w
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t hi = pf[i];
          pf[i] = h2<PDT>(__builtin_fmaf(load16<PDT>(static_cast<uint16_t>(hi)), minus, w[2 * i] * up),
                          __builtin_fmaf(load16<PDT>(static_cast<uint16_t>(hi >> 16)), minus, w[2 * i + 1] * up));
        }
      }
#pragma unroll
      for (int h = 0; h < S::NH; ++h) {
#pragma unroll
        for (int q = 0; q < S::EC / 4; ++q) {  // elements 4 q .. 4 q + 3
          uint32_t o[4][4];  // operand dwords: tokens 2 p, 2 p + 1 of an element
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const auto& y0 = x.w[2 * p][h];
            const auto& y1 = x.w[2 * p + 1][h];
            if constexpr (MODE == kKvInt8) {
              constexpr uint32_t sel[4] = {0x0C040C00u, 0x0C050C01u, 0x0C060C02u, 0x0C070C03u};
#pragma unroll
              for (int j = 0; j < 4; ++j)
                o[j][p] = unbias_f16(__builtin_amdgcn_perm(y1[q] ^ 0x80808080u, y0[q] ^ 0x80808080u, sel[j]), kMinus128);
            } else if constexpr (MODE == kKvInt4) {
              const uint32_t z = __builtin_amdgcn_perm(y1[0], y0[0], q ? 0x07060302u : 0x05040100u) ^ 0x88888888u, zz = z >> 8;
              o[0][p] = unbias_f16(z & 0x000F000Fu, kMinus8);
              o[1][p] = unbias_f16(z & 0x00F000F0u, kMinus128);
              o[2][p] = unbias_f16(zz & 0x000F000Fu, kMinus8);
              o[3][p] = unbias_f16(zz & 0x00F000F0u, kMinus128);
            } else {
              uint32_t e0[2], e1[2];  // the elements of both tokens as halves
              if constexpr (MODE == kKv16) {
                e0[0] = y0[2 * q];
                e0[1] = y0[2 * q + 1];
                e1[0] = y1[2 * q];
                e1[1] = y1[2 * q + 1];
              } else if constexpr (MODE == kKvE4M3) {
                e0[0] = fp8_to_f16x2<false>(y0[q]);
                e0[1] = fp8_to_f16x2<true>(y0[q]);
                e1[0] = fp8_to_f16x2<false>(y1[q]);
                e1[1] = fp8_to_f16x2<true>(y1[q]);
              } else {
                const uint32_t b0 = x.e8[2 * p][h], b1 = x.e8[2 * p + 1][h];
                const float f0 = b0 == 255u ? __builtin_nanf("") : pow2(static_cast<int>(b0) - ref + kUpV);
                const float f1 = b1 == 255u ? __builtin_nanf("") : pow2(static_cast<int>(b1) - ref + kUpV);
                e0[0] = q ? fp4_to_f16x2<2>(y0[0], f0) : fp4_to_f16x2<0>(y0[0], f0);
                e0[1] = q ? fp4_to_f16x2<3>(y0[0], f0) : fp4_to_f16x2<1>(y0[0], f0);
                e1[0] = q ? fp4_to_f16x2<2>(y1[0], f1) : fp4_to_f16x2<0>(y1[0], f1);
                e1[1] = q ? fp4_to_f16x2<3>(y1[0], f1) : fp4_to_f16x2<1>(y1[0], f1);
              }
#pragma unroll
              for (int j = 0; j < 4; ++j)
                o[j][p] = __builtin_amdgcn_perm(e1[j / 2], e0[j / 2], j % 2 ? 0x07060302u : 0x05040100u);
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[h][4 * q + j] = mfma16x16x32<PDT>(u32x4_t{o[j][0], o[j][1], o[j][2], o[j][3]}, pf, acc[h][4 * q + j]);
          __builtin_amdgcn_sched_barrier(0);  // (bounds the operands alive at once)
        }
      }
    };

    // ---- the steps, in a pipeline: the next step's keys are loaded as soon as this one's scores
    // are formed, its values as soon as this one's are added, so a wave always has one of the
    // two in flight.
    if (steps > 0) {
      float s[8];
      int base = 0;
      for (int i = 0; i < steps; ++i) {
        const int idx = i - base;
        const bool whole = t_first + kUnit * i + kTile <= n && __builtin_amdgcn_readlane(pages, 2 * idx) >= 0 &&
                           __builtin_amdgcn_readlane(pages, 2 * idx + 1) >= 0;
        score(kx, i, idx, whole, s);
        if (i + 1 < steps) load_keys(kx, i + 1, idx + 1);
        if constexpr (MODE == kKv16) take_odd(vx, s);
        weigh(s);
        add(vx, i, idx, whole, s);
        if (i + 1 < steps) load_values(vx, i + 1, idx + 1);
        if (idx + 1 == kBatch) {  // the last fetched step is under way: fetch from it on
          base = i + 1;
          fetch_pages(base);
        }
      }
    }

    // ---- the next segment's first loads, under way while this one's rows are written
    more = u < u_end && next_segment();
    if (more) begin();

    // ---- the four waves' sums joined; the whole segment's rows out, or its part to the workspace
    // (lane indices redefined: what derives from them is not kept in registers across the steps)
    const int el = static_cast<int>(here(lane)), er = el & 15, eb = el >> 4;
    constexpr float down = 1.0f / (1 << kUpP<MODE, PDT>);
    l = column_sum(l) * down;
    if (eb == 0) {
      s_m[wv][er] = m;
      s_l[wv][er] = l;
    }
    __syncthreads();
    {
      float mx = -kInf;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) mx = fmaxf(mx, s_m[w][er]);
      float f = m == -kInf ? 0.0f : rescale(m, mx);
      if (m != m || mx == kInf) f = __builtin_nanf("");
      f *= kCode * down;
      const int e = kScaled ? (ref < -1000 ? 0 : ref) : MODE == kKvFp4 ? (ref < -1000 ? 0 : ref - 127 - kUpV) : 0;
#pragma unroll
      for (int h = 0; h < S::NH; ++h)
#pragma unroll
        for (int j = 0; j < S::EC; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float g = MODE == kKvInt4 && (j & 1) ? f * 0.0625f : f;
            s_o[wv][(128 * h + S::EC * (4 * eb + i) + j) * LDH + er] = __builtin_amdgcn_ldexpf(acc[h][j][i] * g, e);
          }
    }
    __syncthreads();
    const int heads = min(16, a.g - ht * 16);
    float* slot = part + (static_cast<int64_t>(blockIdx.x) * 2 + (first_seg ? 0 : 1)) * (static_cast<int64_t>(gh) * (DP + 2));
    for (int i = static_cast<int>(here(tid)); i < heads * DP; i += kThreads) {
      const int hd = i / DP, d = i - hd * DP;
      float mx = -kInf, ls = 0.0f, o = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) mx = fmaxf(mx, s_m[w][hd]);
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float mw = s_m[w][hd];
        ls += s_l[w][hd] == 0.0f ? 0.0f : s_l[w][hd] * __builtin_amdgcn_exp2f(mw - mx);  // (nothing seen, or NaN)
        const float x = s_o[w][d * LDH + hd];
        o += x;
        // (a seen infinity stands in both columns, the sum is that of x)
        if (two && __builtin_fabsf(x) < kInf) o += s_o[w][d * LDH + hd + 8] * (1.0f / kUp);
      }
      const int hq = hk * a.g + ht * 16 + hd;
      if (all) {
        if (!PAD || d < D) a.out.p[b0 * a.out.row + hq * a.out.head + d] = round16<DT>(ls == 0.0f ? 0.0f : o / ls);
        if (a.lse && d == 0)
          a.lse[static_cast<int64_t>(b0) * a.Hq + hq] = ls == 0.0f ? -kInf : (mx + __builtin_amdgcn_logf(ls)) * 0.693147181f;
      } else {
        slot[hd * DP + d] = o;
        if (d == 0) {
          slot[gh * DP + hd] = mx;
          slot[gh * (DP + 1) + hd] = ls;
        }
      }
    }
    __syncthreads();
    first_seg = false;
  }
}

// Joins the parts of the segments that were split, and writes the rows of empty sequences.  One
// workgroup per segment and, with gridDim.y > 1, every gridDim.y-th of its heads; with gridDim.z > 1 that
// part of the elements, whose threads then share the parts among more groups.
template <int DT, int DP>
__global__ __launch_bounds__(kThreads) void decode_join_kernel(DecodeArgs a, const float* __restrict__ part, int32_t nht,
                                                               int32_t gh, int32_t grid, int32_t start) {
  const int E = DP / gridDim.z, G = kThreads / E;  // its elements; threads that share an element's parts
  constexpr int kBatch = 8;         // parts of a thread in flight (2: 2 x 131072 tokens 106 us, not 103)
  constexpr int kFew = 4;           // parts that all elements are joined of at once: 64 x 16384 in int8 160 us
                                    // by the general loop, 151 so
  __shared__ int32_t s_sum[2][kWaves];
  __shared__ float s_m[kThreads], s_l[kThreads], s_o[kThreads];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int per_b = a.c.Hkv * nht, D = a.c.D;
  const int b = blockIdx.x / per_b, seg = blockIdx.x - b * per_b, hk = seg / nht, ht = seg - hk * nht;
  const int heads = min(16, a.g - ht * 16);
  const int at = tid & (E - 1), d = E * blockIdx.z + at, gr = tid / E;
  const int32_t n = length_of(a, b);
  int sum = 0, before = 0;  // of all sequences, of those before b
  if (a.B <= 64) {
    const int weight = lane < a.B ? weight_of(length_of(a, lane), start) : 0, incl = wave_scan(weight);
    sum = __builtin_amdgcn_readlane(incl, 63);
    before = __builtin_amdgcn_readlane(incl - weight, b);
  } else {
    for (int i = tid; i < a.B; i += kThreads) {
      const int k = weight_of(length_of(a, i), start);
      sum += k;
      if (i < b) before += k;
    }
    sum = wave_scan(sum);
    before = wave_scan(before);
    if (lane == 63) {
      s_sum[0][wv] = sum;
      s_sum[1][wv] = before;
    }
    __syncthreads();
    sum = s_sum[0][0] + s_sum[0][1] + s_sum[0][2] + s_sum[0][3];
    before = s_sum[1][0] + s_sum[1][1] + s_sum[1][2] + s_sum[1][3];
  }
  for (int hd = blockIdx.y; n == 0 && hd < heads; hd += gridDim.y) {
    const int hq = hk * a.g + ht * 16 + hd;
    if (gr == 0 && d < D) a.out.p[b * a.out.row + hq * a.out.head + d] = 0;
    if (a.lse && gr == 0 && d == 0) a.lse[static_cast<int64_t>(b) * a.Hq + hq] = -kInf;
  }
  if (n == 0) return;
  const Runs run(sum * per_b, grid);
  const int nw = weight_of(n, start);
  const uint32_t ua = before * per_b + seg * nw;
  const int i0 = run.of(ua + start), i1 = run.of(ua + nw - 1);
  if (i0 == i1) return;  // one workgroup had it all and wrote the rows
  const int np = i1 - i0 + 1;
  const int64_t pitch = static_cast<int64_t>(gh) * (DP + 2);
  // run i's part is its first one unless the run began before this segment (only i0 can have)
  const float* const p0 = part + (static_cast<int64_t>(i0) * 2 + (run.start(i0) < ua ? 1 : 0)) * pitch;
  const float* const p1 = part + static_cast<int64_t>(i0) * 2 * pitch;  // + 2 i pitch for run i0 + i
  if (np <= kFew) {  // (short segments: all parts of four elements of a thread in flight)
    if (blockIdx.z > 0) return;
    for (int e0 = blockIdx.y * 4 * kThreads + tid; e0 < heads * DP; e0 += gridDim.y * 4 * kThreads) {
      float pm[4][kFew], pl[4][kFew], po[4][kFew];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int e = e0 + x * kThreads, hd = e / DP;
#pragma unroll
        for (int i = 0; i < kFew; ++i) {
          const float* const p = i == 0 ? p0 : p1 + 2 * pitch * i;
          const bool in = i < np && e < heads * DP;
          pm[x][i] = in ? p[gh * DP + hd] : -kInf;
          pl[x][i] = in ? p[gh * (DP + 1) + hd] : 0.0f;
          po[x][i] = in ? p[e] : 0.0f;
        }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int e = e0 + x * kThreads, hd = e / DP, de = e - hd * DP, hq = hk * a.g + ht * 16 + hd;
        float m = -kInf, l = 0.0f, o = 0.0f;
#pragma unroll
        for (int i = 0; i < kFew; ++i) m = fmaxf(m, pm[x][i]);
#pragma unroll
        for (int i = 0; i < kFew; ++i) {
          const float w = pm[x][i] == -kInf ? 0.0f : rescale(pm[x][i], m);
          l += pl[x][i] * w;
          o += po[x][i] * w;
        }
        if (e < heads * DP && de < D) a.out.p[b * a.out.row + hq * a.out.head + de] = round16<DT>(l == 0.0f ? 0.0f : o / l);
        if (a.lse && e < heads * DP && de == 0)
          a.lse[static_cast<int64_t>(b) * a.Hq + hq] = l == 0.0f ? -kInf : (m + __builtin_amdgcn_logf(l)) * 0.693147181f;
      }
    }
    return;
  }
  for (int hd = blockIdx.y; hd < heads; hd += gridDim.y) {
    float m = -kInf, l = 0.0f, o = 0.0f;
    for (int k = gr; k < np; k += G * kBatch) {
      float pm[kBatch], pl[kBatch], po[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = k + j * G;
        const float* const p = i == 0 ? p0 : p1 + 2 * pitch * i;
        pm[j] = i < np ? p[gh * DP + hd] : -kInf;
        pl[j] = i < np ? p[gh * (DP + 1) + hd] : 0.0f;
        po[j] = i < np ? p[hd * DP + d] : 0.0f;
      }
      float mn = m;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) mn = fmaxf(mn, pm[j]);
      const float f = m == -kInf ? 0.0f : rescale(m, mn);
      l *= f;
      o *= f;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const float w = pm[j] == -kInf ? 0.0f : rescale(pm[j], mn);
        l += pl[j] * w;
        o += po[j] * w;
      }
      m = mn;
    }
    if (G > 1) {
      s_m[tid] = m;
      s_l[tid] = l;
      s_o[tid] = o;
      __syncthreads();
      float mn = m;
      for (int g = 0; g < G; ++g) mn = fmaxf(mn, s_m[g * E + at]);
      l = o = 0.0f;
      for (int g = 0; g < G; ++g) {
        const float mg = s_m[g * E + at], w = mg == -kInf ? 0.0f : rescale(mg, mn);
        l += s_l[g * E + at] * w;
        o += s_o[g * E + at] * w;
      }
      m = mn;
      __syncthreads();
    }
    const int hq = hk * a.g + ht * 16 + hd;
    if (gr == 0 && d < D) a.out.p[b * a.out.row + hq * a.out.head + d] = round16<DT>(l == 0.0f ? 0.0f : o / l);
    if (a.lse && gr == 0 && d == 0)
      a.lse[static_cast<int64_t>(b) * a.Hq + hq] = l == 0.0f ? -kInf : (m + __builtin_amdgcn_logf(l)) * 0.693147181f;
  }
}

// Whether a segment is one workgroup's whatever its length, with no plan and no join: a table that
// reaches 4 units at most, or 8 with a segment for each CU.  us a call split and joined, and so (8 of either are
// the host's): one sequence of 250 tokens, 32 heads on 8 of 128, bf16 (8 segments) 12.2 and 9.5, of 510 12.9
// and 10.0, of 880 12.5 and 13.2; 32 of 65 to 500 (256 segments) 15.7 and 10.3, of 131 to 1000 19.1 and 17.3, of
// 261 to 2000 30.0 and 28.5; 64 of 1000, int8, 28.6 and 26.3, of 2000 50.3 and 47.7; 37 of 22 to 1000, E4M3, 16
// heads of 64 16.0 and 15.3, of 43 to 2000 20.3 and 26.6.
bool single_of(int64_t segments, int64_t reach) { return reach <= (segments >= 256 ? 8 : 4) * kUnit; }

int padded(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

template <int MODE, int DT, int DP, bool PAD>
hipError_t go(const DecodeArgs& a, float* part, hipStream_t s) {
  const int nht = (a.g + 15) / 16, gh = a.g < 16 ? a.g : 16;
  const int64_t reach = static_cast<int64_t>(a.bt.width) << a.c.page_log;
  const int64_t segments = static_cast<int64_t>(a.B) * a.c.Hkv * nht;
  const bool single = single_of(segments, reach);
  if (single) {
    decode_kernel<MODE, DT, DP, PAD><<<static_cast<uint32_t>(segments), kThreads, 0, s>>>(a, part, nht, gh, true);
    return hipGetLastError();
  }
  constexpr int grid = 256 * Shape<MODE, DP, PAD>::per_cu;
  decode_kernel<MODE, DT, DP, PAD><<<grid, kThreads, 0, s>>>(a, part, nht, gh, false);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  // Enough workgroups of the join to fill the device, at most one a head.  us with one a segment, and so: 2
  // sequences of 87381 and 131072 tokens, int8, 64 heads on 8: 120 and 93; 16 of 1150 to 8192, 32 heads on 1: 65
  // and 24; 8 of 254 to 1500, 32 on 8: 18 and 14.
  const uint32_t ny = static_cast<uint32_t>(std::min<int64_t>(gh, ceil_div(512, segments)));
  // And where that leaves few, slices of 16 elements at least: one sequence of 131072 tokens, int4, 8 heads on
  // 1, 75 us whole and 25 so, of 60883, 16 heads of 64 on 2, 31 and 18, of 8192, 32 on 8, 18.7 and 15.5; the two
  // long ones 93 and 92; the eight short ones the same.
  uint32_t nz = 1;
  while (nz < DP / 16 && segments * ny * nz * 2 <= 256) nz *= 2;
  decode_join_kernel<DT, DP><<<dim3(static_cast<uint32_t>(segments), ny, nz), kThreads, 0, s>>>(a, part, nht, gh, grid, Shape<MODE, DP, PAD>::start);
  return hipGetLastError();
}

template <int MODE, int DT>
hipError_t by_size(const DecodeArgs& a, float* part, hipStream_t s) {
  switch (a.c.D) {
    case 64: return go<MODE, DT, 64, false>(a, part, s);
    case 128: return go<MODE, DT, 128, false>(a, part, s);
    case 256: return go<MODE, DT, 256, false>(a, part, s);
    default: break;
  }
  switch (padded(a.c.D)) {
    case 64: return go<MODE, DT, 64, true>(a, part, s);
    case 128: return go<MODE, DT, 128, true>(a, part, s);
    default: return go<MODE, DT, 256, true>(a, part, s);
  }
}

template <int MODE>
hipError_t by_dtype(const DecodeArgs& a, float* part, hipStream_t s) {
  return a.c.dtype == kF16 ? by_size<MODE, kF16>(a, part, s) : by_size<MODE, kBF16>(a, part, s);
}

}  // namespace

uint64_t attn_decode_workspace(int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int64_t max_tokens) {
  const int g = Hq / Hkv, gh = g < 16 ? g : 16;
  if (B == 0 || single_of(static_cast<int64_t>(B) * Hkv * ceil_div(g, 16), max_tokens)) return 0;
  return static_cast<uint64_t>(kMaxGrid) * 2 * gh * (padded(D) + 2) * sizeof(float);
}

hipError_t launch_attn_decode(const DecodeArgs& a, void* ws, hipStream_t s) {
  float* part = static_cast<float*>(ws);
  switch (a.c.mode) {
    case kKv16: return by_dtype<kKv16>(a, part, s);
    case kKvInt8: return by_dtype<kKvInt8>(a, part, s);
    case kKvE4M3: return by_dtype<kKvE4M3>(a, part, s);
    case kKvInt4: return by_dtype<kKvInt4>(a, part, s);
    default: return by_dtype<kKvFp4>(a, part, s);
  }
}

}  // namespace fq
