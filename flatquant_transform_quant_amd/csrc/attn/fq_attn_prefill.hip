// Attention over packed prompts: for every query row i of a sequence and query head h,
//     o = sum_j p_j v_j,  p = softmax over the visible keys j of scale * <q, k_j>
// in one pass over the keys, with the running maximum m and sum l of the softmax in fp32.
//
// A workgroup of four waves takes 128 query rows of one head (32 a wave) and walks the keys in
// tiles of 64, copied by LDS-DMA into one of two buffers while the other is used; two workgroups
// share a CU, so that one wave's softmax runs beside another's products.  Per wave and tile,
// v_mfma_f32_32x32x16:
//   S^T = K Q^T: A rows are keys (16-byte LDS reads), B columns the wave's query rows, kept in
//     registers for the whole walk.  A lane ends with 32 scores of ONE query row (l % 32; the
//     other half of the keys is with lane l ^ 32), so the softmax needs no step between lanes
//     but a maximum between those two, and that only when m moves.
//   O^T = V^T P^T: the weights, rounded to 16 bits, are the B operand exactly as they lie in
//     the accumulators (contraction slot 4 x + i of half h is key 16 g + 8 x + 4 h + i); the A
//     operand is read from the row-major V tile by the transposing LDS read, whose runs of
//     four keys are just those slots.
// LDS layouts: the 16-byte piece c of tile row r sits at c ^ (r & 15) (keys) or c ^ 4 (r & 3)
// (values); with rows of 128 bytes, where two rows share the 64 banks, at c ^ ((r >> 1) & 7) and
// c ^ 4 ((r >> 1) & 1): both kinds of read then touch every bank once.
// The weights have the values' type, as the instruction asks: 11 bits, in bf16 8 (the sums l take them unrounded).
// The result's error is 1.0 to 1.4 times what fp32 weights leave, the output's own rounding in both; a second
// product with the remainders would cost half as much matrix time again.
// The maximum is moved only when a score passes m + 8 in base-2 units (weights then reach 2^8):
// the accumulators are rescaled a few times a walk instead of every tile.
// Tiles of all sequences are handed out longest walk first; where they do not fill the device, the
// long walks are cut into parts whose sums a second launch joins.
// A weight of 0 times an infinite or NaN value is NaN: for a key that is hidden, in a partly masked tile, and for
// one whose weight rounds to 0, where the infinity should stay.  The walk ignores that; if a result is not
// finite, the workgroup walks again, this time taking such values out of the products and adding them to the
// rows that do see them.
//
// What bounds it: one 32768-row prompt, 8 heads on one cache head of 128, takes 1.93 to 2.03 ms (1.08 to
// 1.14 PFLOP/s; a large library product reaches 1.25 to 1.39 here) with the matrix cores busy 61% of the
// time at a clock of 1.8 GHz, which the power of products, LDS reads, copies and exponentials together
// sets: without any one of them the rate is 1.25 to 1.27, without all but the products 1.67.  Smaller
// calls run at 2.0 GHz and 47%: nine packed prompts of 242 to 4096 rows, 32 heads, 306 to 314 us (910 to 930 TFLOP/s),
// where a workgroup spends 3.4 us before its first and after its last tile each (places, query rows,
// rows out) and 1.76 us a tile; four chunks of 313 to 1024 rows behind 2507 to 8192 keys, 212 to 230 us (800 to 870),
// where the device's 512 places are 81% busy, the longest walk being 133 tiles and the mean 97.
// Tile and schedule, TFLOP/s on those three (prompt, packed, chunks) and 2 x 8192 rows of 64:
//   128 rows, 4 waves (this)                                          1128  867  669*  826
//   256 rows, 8 waves                                                 1167  847  611*  795
//   64 rows a wave, each LDS fragment for two products, 1 wave a SIMD  221  179  144   511
//   scores of the next 32 keys under the softmax of these              1015  811  800   758  (this: 1077 887 855 870)
// (*: before walks were ordered by length.)
#include <hip/hip_runtime.h>

#include <algorithm>

#include "fq_attn_dev.h"

namespace fq {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kRows = 32 * kWaves;  // query rows of a workgroup
constexpr int kKeys = 64;           // keys of a tile
constexpr int kAhead = 4;           // fragments read ahead of their products (2, 6 and 8: the same to 2% slower)
constexpr int kMaxParts = 32, kMinChunk = 8, kEnough = 512;  // see parts_of()
constexpr float kLazy = 8.0f;
// Weights as they enter the second product are 2^kUp times those above (at most 2^(8 + kUp), f16's largest binade):
// an f16 weight is then off by 2^-32 of the largest one where it is subnormal, not by 2^-25, which many keys far
// below one that stands out lost altogether (20000 of them 17.5 nats below: 5e-4 of the weights).
template <int DT>
constexpr float kUp = DT == kF16 ? 7.0f : 0.0f;
constexpr float kInf = __builtin_inff();
constexpr uint32_t kOut = 0x80000000u;  // an offset past every resource

typedef __attribute__((ext_vector_type(16))) float f32x16_t;
typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4_t;
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) bf16x4_t lds_bf16x4;
typedef int i32x4_t __attribute__((ext_vector_type(4)));

template <int DT>
__device__ __forceinline__ f32x16_t mfma32x32x16(u32x4_t a, u32x4_t b, f32x16_t c) {
  if constexpr (DT == kBF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

// Buffer resource over `bytes` bytes from p as scalar registers; 0 bytes: every access is out of
// range (a load returns zeros and touches no memory).
__device__ __forceinline__ i32x4_t rsrc4(const void* p, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  return i32x4_t{static_cast<int>(static_cast<uint32_t>(a)), static_cast<int>(static_cast<uint32_t>(a >> 32) & 0xFFFF),
                 static_cast<int>(bytes), kBufferWord3};
}

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// One LDS-DMA load: lane l's 16 bytes at rs + voff go to LDS lds + 16 l.  (As inline assembly: the
// compiler would wait for every such load before any LDS read.  A load that takes its place from m0
// needs one wait state after m0's write.)
__device__ __forceinline__ void dma16(uint32_t lds, uint32_t voff, i32x4_t rs) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" : : "s"(lds), "v"(voff), "s"(rs) : "memory", "m0");
}
#pragma clang diagnostic pop

// This wave's loads landed and its LDS reads done, then the workgroup barrier.
__device__ __forceinline__ void tile_barrier() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" : : : "memory"); }

__device__ __forceinline__ float half_max(float v) {  // with lane ^ 32
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// the largest over the wave
__device__ __forceinline__ int wave_top(int v) {
  v = max(v, __builtin_amdgcn_update_dpp(v, v, 0x111, 0xF, 0xF, false));
  v = max(v, __builtin_amdgcn_update_dpp(v, v, 0x112, 0xF, 0xF, false));
  v = max(v, __builtin_amdgcn_update_dpp(v, v, 0x114, 0xF, 0xF, false));
  v = max(v, __builtin_amdgcn_update_dpp(v, v, 0x118, 0xF, 0xF, false));
  v = max(v, __builtin_amdgcn_update_dpp(v, v, 0x142, 0xA, 0xF, false));
  v = max(v, __builtin_amdgcn_update_dpp(v, v, 0x143, 0xC, 0xF, false));
  return __builtin_amdgcn_readlane(v, 63);
}
__device__ __forceinline__ int wave_total(int v) { return __builtin_amdgcn_readlane(wave_scan(v), 63); }

// The 128 query rows and the head that workgroup number `id` works on.
struct Place {
  int seq;       // -1: none left for this workgroup
  int tile;      // tile of the sequence
  int q0, lq;    // its query rows
  int k0, lk;    // its key rows
  int head;
  int chunk;     // key tiles of a part, where the walk is split (the longest walk over `parts`)
};

// the last key that query row r of a sequence sees
__device__ __forceinline__ int last_key(const PrefillArgs& a, int off, int lk, int r) { return a.causal ? min(off + r, lk - 1) : lk - 1; }
__device__ __forceinline__ int key_tiles(const PrefillArgs& a, int off, int lk, int lq, int tile) {
  return max(0, (last_key(a, off, lk, min((tile + 1) * kRows, lq) - 1) + kKeys) / kKeys);
}

// Tiles are handed out longest walk first, over all sequences: a tile's level is the number of
// whole 128-key blocks before its last row's key, every sequence has at most one tile of a level,
// so the level of the rank-th tile is found by bisection on the number of tiles at or above a
// level.  More than 64 sequences, or no causal mask: sequence by sequence, last tile first.
__device__ __forceinline__ Place place_of(const PrefillArgs& a, int id, int parts) {
  const int lane = threadIdx.x & 63;
  Place p;
  p.head = id % a.Hq;
  int rank = id / a.Hq;
  // (workgroups go to the 8 XCDs in turn: neighbouring heads, which share keys, on one XCD's L2)
  if (a.Hq % 8 == 0) p.head = (p.head % 8) * (a.Hq / 8) + p.head / 8;
  p.seq = -1;
  p.tile = p.q0 = p.lq = 0;
  p.chunk = 1 << 30;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    const int b = b0 + lane;
    int s = 0, n = 0, ks = 0, kn = 0;
    if (b < a.B) {
      s = max(0, min(a.cu_q[b], a.Tq));
      n = max(0, min(a.cu_q[b + 1], a.Tq) - s);
      ks = max(0, min(a.cu_k[b], a.Tk));
      kn = max(0, min(a.cu_k[b + 1], a.Tk) - ks);
    }
    const int nt = (n + kRows - 1) / kRows;
    if (parts > 1) p.chunk = max(kMinChunk, (wave_top(nt > 0 ? key_tiles(a, kn - n, kn, n, nt - 1) : 0) + parts - 1) / parts);
    int w;
    if (a.causal && a.B <= 64) {
      const int total = wave_total(nt);
      if (rank >= total) return p;
      const int first = max(0, kn - n + kRows - 1) / kRows;  // level of the sequence's tile 0 (0 where no key is ahead)
      auto above = [&](int level) { return max(0, min(nt, first + nt - level)); };  // this sequence's tiles at or above
      int lo = 0, hi = wave_top(first + nt);  // tiles at or above lo: more than rank; at or above hi: not
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (wave_total(above(mid)) > rank) lo = mid; else hi = mid;
      }
      const int in = rank - wave_total(above(lo + 1));  // the in-th sequence with a tile of level lo
      w = __builtin_ctzll(__ballot(wave_scan(above(lo) - above(lo + 1)) > in));
      p.tile = lo - __builtin_amdgcn_readlane(first, w);
    } else {
      const int incl = wave_scan(nt), sum = __builtin_amdgcn_readlane(incl, 63);
      if (rank >= sum) {
        rank -= sum;
        continue;
      }
      w = __builtin_ctzll(__ballot(incl > rank));
      p.tile = __builtin_amdgcn_readlane(incl, w) - 1 - rank;
    }
    p.seq = b0 + w;
    p.q0 = __builtin_amdgcn_readlane(s, w);
    p.lq = __builtin_amdgcn_readlane(n, w);
    p.k0 = __builtin_amdgcn_readlane(ks, w);
    p.lk = __builtin_amdgcn_readlane(kn, w);
    return p;
  }
  return p;
}

// (heads of 64: registers for three workgroups a CU, which the plain walk alone would leave, and the careful one not)
template <int DT, int DP, bool PAD>
__global__ __launch_bounds__(kThreads, DP == 256 ? 1 : DP == 64 ? 3 : 2) void prefill_kernel(PrefillArgs a, int parts, float* __restrict__ ws) {
  constexpr int KS = DP / 16;            // products of a score block
  constexpr int DB = DP / 32;            // 32-row blocks of O^T
  constexpr int kRowB = DP * 2;          // bytes of a tile row
  constexpr int kTileB = kKeys * kRowB;  // bytes of a tile (keys or values)
  constexpr int kPieces = DP / 8;        // 16-byte pieces of a row
  constexpr int NL = kTileB / 1024 / kWaves;
  __shared__ __align__(16) uint8_t lds[4 * kTileB];  // buffer b: keys at 2 b, values at 2 b + 1
  const lds_u8* const lds_l = (const lds_u8*)lds;
  const uint32_t lds_addr = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds_l));

  const int tid = threadIdx.x, lane = tid & 63, col = lane & 31, hf = lane >> 5;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int D = PAD ? a.D : DP;

  // ---- which rows, and which part of their walk
  const int part = parts > 1 ? static_cast<int>(blockIdx.x / a.Hq) % parts : 0;
  const Place pl = place_of(a, parts > 1 ? static_cast<int>(blockIdx.x % a.Hq + blockIdx.x / (a.Hq * parts) * a.Hq) : blockIdx.x, parts);
  if (pl.seq < 0) return;
  const int head = pl.head, q0 = pl.q0, lq = pl.lq, k0 = pl.k0, lk = pl.lk;
  const int row0 = pl.tile * kRows;
  const int row = row0 + 32 * wv + col;  // this lane's query row in the sequence
  const int off = lk - lq;               // keys ahead of the first row
  // the last key that this lane's row, the wave's first and last rows see; the walk's tiles
  const int lim = last_key(a, off, lk, row);
  const int lim_first = last_key(a, off, lk, row0 + 32 * wv), lim_last = last_key(a, off, lk, min(row0 + 32 * wv + 31, lq - 1));
  const int all_tiles = key_tiles(a, off, lk, lq, pl.tile);
  const bool split = all_tiles > pl.chunk;
  const int t_first = split ? part * pl.chunk : 0, t_end = split ? min(all_tiles, t_first + pl.chunk) : all_tiles;
  if (part > 0 && (!split || t_first >= t_end)) return;
  const int hk = head / a.g;

  // ---- LDS-DMA: load i of wave w fills the 16-byte places 64 (NL w + i) + lane of a tile
  uint32_t koff[NL], voff[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int at = 64 * (NL * wv + i) + lane, r = at / kPieces, p = at % kPieces;
    const int kp = p ^ (DP == 64 ? (r >> 1) & 7 : r & 15), vp = p ^ (4 * (DP == 64 ? (r >> 1) & 1 : r & 3));
    koff[i] = !PAD || 8 * kp < D ? static_cast<uint32_t>(r * a.k.row * 2 + 16 * kp) : kOut;
    voff[i] = !PAD || 8 * vp < D ? static_cast<uint32_t>(r * a.v.row * 2 + 16 * vp) : kOut;
  }
  auto dma = [&](int t, int buf) __attribute__((always_inline)) {
    const int left = min(kKeys, lk - t * kKeys);
    const int64_t r = k0 + static_cast<int64_t>(t) * kKeys;
    const i32x4_t rk = rsrc4(a.k.p + (r * a.k.row + hk * a.k.head), left > 0 ? static_cast<uint32_t>((left - 1) * a.k.row + D) * 2u : 0u);
    const i32x4_t rv = rsrc4(a.v.p + (r * a.v.row + hk * a.v.head), left > 0 ? static_cast<uint32_t>((left - 1) * a.v.row + D) * 2u : 0u);
    const uint32_t at = lds_addr + buf * (2 * kTileB) + 1024 * NL * wv;
#pragma unroll
    for (int i = 0; i < NL; ++i) dma16(at + 1024 * i, koff[i], rk);
#pragma unroll
    for (int i = 0; i < NL; ++i) dma16(at + kTileB + 1024 * i, voff[i], rv);
  };

  // (the first tile is on its way before the query rows are waited for)
  if (t_first < t_end) dma(t_first, t_first & 1);

  // ---- the query rows as B operands (a negative scale goes into their sign)
  const float c = __builtin_fabsf(a.scale) * 1.44269504f;
  u32x4_t qf[KS];
  {
    const uint16_t* qp = a.q.p + (q0 + min(row, lq - 1)) * a.q.row + head * a.q.head;
    const uint32_t sign = a.scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int d = 16 * ks + 8 * hf;
      qf[ks] = u32x4_t{0u, 0u, 0u, 0u};
      if (!PAD || d < D) qf[ks] = *reinterpret_cast<const u32x4_t*>(qp + d);
      qf[ks] ^= u32x4_t{sign, sign, sign, sign};
    }
  }

  // ---- LDS reads: keys, piece 2 ks + hf of row col (+ 32); values, runs of the transposing read
  const uint32_t krd = col * kRowB, kx = hf ^ (DP == 64 ? (col >> 1) & 7 : col & 15);
  const int rj = (lane & 15) >> 2;
  const uint32_t vrd = (4 * hf + rj) * kRowB + 32 * ((lane >> 4) & 1) + 8 * (lane & 3), vx = DP == 64 ? rj >> 1 : rj;

  f32x16_t acc[DB];
  float m, l;
  auto walk = [&](auto careful) __attribute__((always_inline)) {
    constexpr bool CAREFUL = decltype(careful)::value;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[d][i] = 0.0f;
    m = -kInf;
    l = 0.0f;
    if (CAREFUL && t_first < t_end) dma(t_first, t_first & 1);
    for (int t = t_first; t < t_end; ++t) {
      const int buf = t & 1;
      tile_barrier();
      if (t + 1 < t_end) dma(t + 1, buf ^ 1);
      if (t * kKeys > lim_last) continue;  // no row of this wave sees the tile
      const lds_u8* const kt = lds_l + buf * (2 * kTileB);
      const lds_u8* const vt = kt + kTileB;
      // Fragments are read kAhead products before their use, the first of the values before the
      // softmax; the scheduling barriers keep the compiler from moving each read to its use.
      auto key = [&](int ks, int b) __attribute__((always_inline)) {
        return *(const __attribute__((address_space(3))) u32x4_t*)(kt + krd + 16 * (kx ^ (2 * ks)) + b * 32 * kRowB);
      };
      auto value = [&](int d, int g) __attribute__((always_inline)) {
        const lds_u8* const p = vt + vrd + 64 * (d ^ vx) + 16 * g * kRowB;
        const u32x2_t lo = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)p));
        const u32x2_t hi = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(p + 8 * kRowB)));
        return u32x4_t{lo[0], lo[1], hi[0], hi[1]};
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
          s[i % 2] = mfma32x32x16<DT>(kf[i], qf[i / 2], s[i % 2]);
          __builtin_amdgcn_sched_barrier(0);
        });
      }
      u32x4_t vf[4 * DB];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) vf[i] = value(i % DB, i / DB);
      __builtin_amdgcn_sched_barrier(0);
      const bool masked = t * kKeys + kKeys - 1 > lim_first;
      if (masked) {
        const int left = lim - t * kKeys - 4 * hf;  // visible: place <= left
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (32 * b + 8 * (i / 4) + i % 4 > left) s[b][i] = -kInf;
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
      if (__any(top * c > m + kLazy)) {
        const float mn = fmaxf(m, half_max(top) * c);
        const float f = mn == -kInf ? 1.0f : CAREFUL ? rescale(m, mn) : __builtin_amdgcn_exp2f(m - mn);
        m = mn;
        l *= f;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[d][i] *= f;
      }
      const float ms = m == -kInf ? 0.0f : m - kUp<DT>;
      u32x4_t pf[4];
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[g / 2][8 * (g % 2) + 2 * i], c, -ms));
          const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(s[g / 2][8 * (g % 2) + 2 * i + 1], c, -ms));
          pf[g][i] = round16x2<DT>(x, y);
          l += x + y;
        }
      __builtin_amdgcn_sched_barrier(0);
      uint32_t odd = 0;
      static_for<0, 4 * DB>([&](auto ic) __attribute__((always_inline)) {
        constexpr int i = decltype(ic)::value;
        if constexpr (i + kAhead < 4 * DB) vf[i + kAhead] = value((i + kAhead) % DB, (i + kAhead) / DB);
        if constexpr (CAREFUL) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            odd |= not_finite16<DT>(vf[i][j]);
            vf[i][j] &= ~not_finite16_mask<DT>(vf[i][j]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        acc[i % DB] = mfma32x32x16<DT>(vf[i], pf[i / DB], acc[i % DB]);
        __builtin_amdgcn_sched_barrier(0);
      });
      if constexpr (CAREFUL) {
        const bool any = __any(odd != 0);
        for (int j = 0; any && j < kKeys; ++j) {
          if (t * kKeys + j > lim) break;
          const float w = (seen >> j) & 1 ? 1.0f : 0.0f;
#pragma unroll
          for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int e = 32 * d + 8 * (i / 4) + 4 * hf + i % 4;
              const uint16_t v = *(const __attribute__((address_space(3))) uint16_t*)(
                  vt + j * kRowB + 16 * ((e / 8) ^ (4 * (DP == 64 ? (j >> 1) & 1 : j & 3))) + 2 * (e % 8));
              if (not_finite16<DT>(v)) acc[d][i] += w * load16<DT>(v);
            }
        }
      }
    }
  };
  walk(std::false_type{});
  {
    float odd = 0.0f;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) odd = __builtin_fmaf(acc[d][i], 0.0f, odd);
    if (__syncthreads_or(odd != odd)) walk(std::true_type{});
  }

  l = half_sum(l);
  const float down = DT == kF16 ? 0x1p-7f : 1.0f;  // 2^-kUp
  if (split) {  // the part's sums as they are, [element][row], with m and l
    float* const o = ws + (static_cast<int64_t>(blockIdx.x)) * ((DP + 2) * kRows) + 32 * wv + col;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[(32 * d + 8 * (i / 4) + 4 * hf + i % 4) * kRows] = acc[d][i] * down;
    if (hf == 0) {
      o[DP * kRows] = m;
      o[(DP + 1) * kRows] = l * down;
    }
    return;
  }

  // ---- rows out: through LDS (each wave its own 32 rows, pieces placed as in a key tile), so that a
  // store instruction writes whole rows
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  __syncthreads();  // the last tile's reads are done
  uint8_t* const mine = lds + 32 * wv * kRowB;
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 32 * d + 8 * i + 4 * hf;
      *reinterpret_cast<u32x2_t*>(mine + col * kRowB + 16 * ((e / 8) ^ (DP == 64 ? (col >> 1) & 7 : col & 15)) + 8 * hf) =
          u32x2_t{round16x2<DT>(acc[d][4 * i] * inv, acc[d][4 * i + 1] * inv),
                  round16x2<DT>(acc[d][4 * i + 2] * inv, acc[d][4 * i + 3] * inv)};
    }
  if (a.lse && hf == 0 && row < lq)
    a.lse[static_cast<int64_t>(q0 + row) * a.Hq + head] = l == 0.0f ? -kInf : (m + __builtin_amdgcn_logf(l * down)) * 0.693147181f;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 32 * kPieces / 64; ++i) {
    const int at = 64 * i + lane, r = at / kPieces, p = at % kPieces;
    const u32x4_t w = *reinterpret_cast<const u32x4_t*>(mine + r * kRowB + 16 * (p ^ (DP == 64 ? (r >> 1) & 7 : r & 15)));
    const int to = row0 + 32 * wv + r;
    if (to < lq && (!PAD || 8 * p < D))
      *reinterpret_cast<u32x4_t*>(a.out.p + (q0 + to) * a.out.row + head * a.out.head + 8 * p) = w;
  }
}

// Joins the parts of the walks that were split: a workgroup per 128 rows, head and 32 elements, a thread
// per row and 16 elements.
template <int DT, int DP>
__global__ __launch_bounds__(kThreads) void prefill_join_kernel(PrefillArgs a, int parts, const float* __restrict__ ws) {
  const Place pl = place_of(a, blockIdx.x, parts);
  if (pl.seq < 0) return;
  const int tiles = key_tiles(a, pl.lk - pl.lq, pl.lk, pl.lq, pl.tile);
  if (tiles <= pl.chunk) return;
  const int n = (tiles + pl.chunk - 1) / pl.chunk;
  const int r = threadIdx.x % kRows, row = pl.tile * kRows + r, e = 32 * blockIdx.y + 16 * (threadIdx.x / kRows);
  if (row >= pl.lq || e >= a.D) return;
  // part i of this workgroup's rows was number (rank parts + i) Hq + head's place of the first launch
  const int64_t first = static_cast<int64_t>(blockIdx.x / a.Hq) * parts * a.Hq + blockIdx.x % a.Hq;
  const float* p = ws + first * ((DP + 2) * kRows) + r;
  float m = -kInf, l = 0.0f, o[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) o[j] = 0.0f;
  for (int i = 0; i < n; ++i, p += static_cast<int64_t>(a.Hq) * ((DP + 2) * kRows)) {
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
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint16_t* const out = a.out.p + (pl.q0 + row) * a.out.row + pl.head * a.out.head + e;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (e + 8 * h >= a.D) break;
    u32x4_t w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = round16x2<DT>(o[8 * h + 2 * j] * inv, o[8 * h + 2 * j + 1] * inv);
    *reinterpret_cast<u32x4_t*>(out + 8 * h) = w;
  }
  if (a.lse && e == 0)
    a.lse[static_cast<int64_t>(pl.q0 + row) * a.Hq + pl.head] = l == 0.0f ? -kInf : (m + __builtin_amdgcn_logf(l)) * 0.693147181f;
}

int padded(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

// workgroups of a launch that does not split: tiles of all sequences (at most one partial one each)
int64_t workgroups(int64_t Tq, int64_t B, int64_t Hq) { return (Tq / kRows + B) * Hq; }

// Parts that the longest walk may be cut into.  The device runs 512 workgroups at a time (two a CU; 768 of heads
// of 64); with fewer, the longest walk alone is the whole time.  us in one part and so: 128 rows behind 32768 keys, 32
// heads (64 workgroups) 546 and 88 (without a mask 538 and 85); 64 rows, 8 heads 540 and 44; 16 rows behind 131072, 8
// heads 2137 and 97; 200 behind 2800, 32 heads 56 and 26; 512 behind 16384, 64 heads (320) 293 and 268; 1855 rows, 8
// heads of 256 70 and 41; 1024 rows, 8 heads 23 and 19; 1000, 32 heads 25 and 24.  In up to 8, 16, 32 and 64 parts
// (on a slower card): 128 rows behind 32768 97, 96, 96, 96; 64 82, 53, 46, 46; 16 behind 131072 284, 157, 105, 124.
// A part's sums go through memory (66 KB at 128), so nothing is split once the device is full:
// chunks of 313 to 1024 rows behind up to 8192 keys, 32 heads (736): 204 whole, 227 in two parts, 261 in three
// (cut at the mean load alone 226; dealt out in equal runs 241, as walks that no longer go side by side
// share fewer keys in L2).  Parts of 8 tiles at least: 1024 rows, 8 heads 19 us, of 16 tiles 23.  Where two
// a CU would be shorter, one a CU: 1000 rows, 32 heads 26 us, in two parts each 31; 1855, 8 heads of 256 43
// and 63; 200 behind 2800, 32 heads 28 and 31.  Few keys for so many sequences are short walks, which a
// second launch would only hold up.
int parts_of(int64_t Tq, int64_t Tk, int64_t B, int64_t Hq) {
  const int64_t w = workgroups(Tq, B, Hq);
  if (B > 64 || w >= kEnough || Tk <= kKeys * kMinChunk * std::min<int64_t>(B, 4)) return 1;
  const int64_t two = ceil_div(kEnough, w), one = ceil_div(kEnough / 2, w), least = Tk / (kKeys * kMinChunk);
  return static_cast<int>(std::min(int64_t(kMaxParts), std::max(int64_t(1), two <= least ? two : std::min(one, least + 1))));
}

template <int DT, int DP, bool PAD>
hipError_t go(const PrefillArgs& a, float* ws, hipStream_t s) {
  const int64_t w = workgroups(a.Tq, a.B, a.Hq);
  const int parts = parts_of(a.Tq, a.Tk, a.B, a.Hq);
  prefill_kernel<DT, DP, PAD><<<static_cast<uint32_t>(w * parts), kThreads, 0, s>>>(a, parts, ws);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || parts == 1) return err;
  prefill_join_kernel<DT, DP><<<dim3(static_cast<uint32_t>(w), static_cast<uint32_t>(ceil_div(a.D, 32))), kThreads, 0, s>>>(a, parts, ws);
  return hipGetLastError();
}

template <int DT>
hipError_t by_size(const PrefillArgs& a, float* ws, hipStream_t s) {
  if (a.D == 64) return go<DT, 64, false>(a, ws, s);
  if (a.D == 128) return go<DT, 128, false>(a, ws, s);
  if (a.D == 256) return go<DT, 256, false>(a, ws, s);
  if (a.D < 64) return go<DT, 64, true>(a, ws, s);
  return a.D < 128 ? go<DT, 128, true>(a, ws, s) : go<DT, 256, true>(a, ws, s);
}

}  // namespace

uint64_t attn_prefill_workspace(int64_t Tq, int64_t Tk, int64_t B, int64_t Hq, int64_t D) {
  const int parts = Tq == 0 ? 1 : parts_of(Tq, Tk, B, Hq);
  if (parts == 1) return 0;
  return static_cast<uint64_t>(workgroups(Tq, B, Hq)) * parts * (padded(static_cast<int>(D)) + 2) * kRows * sizeof(float);
}

hipError_t launch_attn_prefill(const PrefillArgs& a, void* ws, hipStream_t s) {
  float* const w = static_cast<float*>(ws);
  return a.dtype == kF16 ? by_size<kF16>(a, w, s) : by_size<kBF16>(a, w, s);
}

}  // namespace fq
