// int8 consumer GEMM: C[t, o] = fl32(sum_h qa[t, h] qw[o, h]) * fl32(sa[t] * sw[o]) with A the quantizer's per-token int8
// codes (its INT8 [K, M, N] output viewed as [K, M N]) and their fp32 scales, W int8 weights with one fp32 scale per output
// channel.  The integer sums are exact in int32 (|sum| <= 2^14 H, H < 2^17), so C is one defined value, rounded once more to a 16-bit C.
//
// Tiles: a workgroup computes a BT x BO tile on v_mfma_i32_16x16x64_i8, 128 bytes of the contraction a stage: the stage's rows of
// A and W are copied by LDS-DMA into one of NB buffers while others feed the products, one barrier a stage; chunk c of row r
// sits at c ^ (r & 7); W is the first operand, so a lane's four results are four consecutive columns of one row.  A half-stage's
// fragments are read among the products of the one before (read in front of their own: 64 x 64 tiles 26 us where they then
// took 19, 100 x 1024 x 8192).  Each XCD takes neighbouring tiles, in groups of four row bands.
// Bound by the walk over the contraction while the device holds all tiles at once (100 x 1024 x 8192: 17.5 us, 270 ns a stage of barrier,
// LDS reads and products); at 8192^3, 443 us (2.48 POP/s, half of the dense int8 peak, matrix cores 58% busy), by LDS: the reads and
// copies of a stage take as many cycles as its products.
// Rows (up to 32, as in single steps): bound by reading W once, 4 x 10240 x 8192 (84 MB) 20.4 us, 4.1 TB/s.  A workgroup of eight
// waves has 16 or 32 channels; the waves take 128 bytes of the contraction in turn, straight from memory into operand registers (both
// operands relabel the contraction the same way: lane group kb has bytes 32 kb .. 32 kb + 31 of the 128), and their sums are added
// up in LDS.
#include <hip/hip_runtime.h>

#include "attn/fq_attn_tile.h"

namespace fq {
namespace {

constexpr int kStage = 128;  // bytes of the contraction a stage
constexpr int kGroup = 4;    // row bands walked together
enum Out : int { kOutF32 = 0, kOutF16 = kF16, kOutBF16 = kBF16 };

struct Gemm {
  const uint8_t *a, *w;
  const float *sa, *sw;
  void* c;
  int32_t T, O, H;
  int32_t vec;  // rows of C are a whole number of four elements, aligned
};

// Four columns o .. o + 3 of row t from their sums.
template <int OUT>
__device__ __forceinline__ void put4(const Gemm& g, int t, int o, i32x4_t acc, float sa, f32x4_t sw) {
  f32x4_t v;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = static_cast<float>(acc[e]) * (sa * sw[e]);
  const int64_t at = static_cast<int64_t>(t) * g.O + o;
  if (g.vec && o + 4 <= g.O) {
    if constexpr (OUT == kOutF32)
      *reinterpret_cast<f32x4_t*>(static_cast<float*>(g.c) + at) = v;
    else
      *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(g.c) + at) = u32x2_t{round16x2<OUT>(v[0], v[1]), round16x2<OUT>(v[2], v[3])};
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (o + e >= g.O) break;
      if constexpr (OUT == kOutF32)
        static_cast<float*>(g.c)[at + e] = v[e];
      else
        static_cast<uint16_t*>(g.c)[at + e] = round16<OUT>(v[e]);
    }
  }
}

// ---- tiles ------------------------------------------------------------------------------------

// BT x BO a workgroup, WT x WO waves, NB buffers
template <int BT, int BO, int WT, int WO, int NB, int OUT>
__global__ __launch_bounds__(64 * WT * WO) void tile_kernel(Gemm g, int32_t nT, int32_t nO) {
  constexpr int NW = WT * WO, NI = BT / WT / 16, NJ = BO / WO / 16;
  constexpr int LA = BT / 8 / NW, LW = BO / 8 / NW;  // LDS-DMA loads of a wave and stage: 8 rows each
  constexpr int kStageB = (BT + BO) * kStage;
  __shared__ __align__(16) uint8_t lds[NB][kStageB];
  const lds_u8* const lds_l = (const lds_u8*)lds[0];
  const uint32_t lds_addr = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds_l));
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);

  // dispatch goes round-robin over the 8 XCDs: each takes neighbouring tiles, which share rows of A and W in its L2
  const int n = nT * nO, b = static_cast<int>(blockIdx.x & 7) * ((n + 7) / 8) + static_cast<int>(blockIdx.x >> 3);
  if (b >= n) return;
  const int grp = b / (kGroup * nO), gfirst = grp * kGroup, gsz = min(nT - gfirst, kGroup);
  const int rem = b - grp * kGroup * nO;
  const int t0 = (gfirst + rem % gsz) * BT, o0 = (rem / gsz) * BO;

  // operand rows past T or O read zeros through resources that end with the tile's last row
  const int H = g.H, rows_a = min(BT, g.T - t0), rows_w = min(BO, g.O - o0);
  const i32x4_t ra = rsrc4(g.a + static_cast<int64_t>(t0) * H, static_cast<uint32_t>(rows_a * H));
  const i32x4_t rw = rsrc4(g.w + static_cast<int64_t>(o0) * H, static_cast<uint32_t>(rows_w * H));
  // load j of wave wv fills rows 8 (NW j + wv) .. + 7; lane l has chunk (l % 8) ^ (row & 7) of row l / 8
  const int crow = 8 * wv + (lane >> 3), chunk = (lane & 7) ^ (lane >> 3);
  uint32_t off[LA > LW ? LA : LW];
#pragma unroll
  for (int j = 0; j < (LA > LW ? LA : LW); ++j) off[j] = static_cast<uint32_t>((8 * NW * j + crow) * H + 16 * chunk);
  auto dma = [&](int buf, int kt) __attribute__((always_inline)) {
    const uint32_t to = lds_addr + buf * kStageB + 1024 * wv;
    const uint32_t past = kStage * kt + 16 * chunk < H ? 0u : kOut;  // (the last stage may be short)
#pragma unroll
    for (int j = 0; j < LA; ++j) dma16(to + 1024 * NW * j, (off[j] + kStage * kt) | past, ra);
#pragma unroll
    for (int j = 0; j < LW; ++j) dma16(to + BT * kStage + 1024 * NW * j, (off[j] + kStage * kt) | past, rw);
  };

  const int wm = wv / WO, wn = wv % WO;
  const int r16 = lane & 15, kb = lane >> 4;
  i32x4_t acc[NI][NJ];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};

  // the fragments of 64 bytes of the contraction, and their products
  struct Half {
    i32x4_t w[NJ], a[NI];
  } x, y;
  auto place = [&](int buf, int h) __attribute__((always_inline)) { return lds_l + buf * kStageB + 16 * ((4 * h + kb) ^ (r16 & 7)); };
  auto read_w = [&](Half& f, const lds_u8* st, int j) __attribute__((always_inline)) {
    f.w[j] = *(const __attribute__((address_space(3))) i32x4_t*)(st + (BT + 16 * (NJ * wn + j) + r16) * kStage);
  };
  auto read_a = [&](Half& f, const lds_u8* st, int i) __attribute__((always_inline)) {
    f.a[i] = *(const __attribute__((address_space(3))) i32x4_t*)(st + (16 * (NI * wm + i) + r16) * kStage);
  };
  // the products of f, and the reads of `next` (from `st`) spread among them
  auto phase = [&](const Half& f, Half& next, const lds_u8* st) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
#pragma unroll
      for (int j = i * NJ / NI; j < (i + 1) * NJ / NI; ++j) read_w(next, st, j);
      read_a(next, st, i);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.w[j], f.a[i], acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // A stage's loads have landed when at most those of the `behind` stages after it are outstanding; its second half's
  // fragments are read under the first one's products, the next stage's first ones under the second one's.  So a stage's
  // buffer is free, all waves' reads of it done, at the barrier in its middle.
  const int nkt = (H + kStage - 1) / kStage;
  auto landed = [&](auto behind) __attribute__((always_inline)) {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "i"(decltype(behind)::value * (LA + LW)) : "memory");
  };
#pragma unroll
  for (int i = 0; i < NB; ++i)
    if (i < nkt) dma(i, i);
  if (nkt >= NB)
    landed(std::integral_constant<int, NB - 1>{});
  else
    tile_barrier();
#pragma unroll
  for (int j = 0; j < NJ; ++j) read_w(x, place(0, 0), j);
#pragma unroll
  for (int i = 0; i < NI; ++i) read_a(x, place(0, 0), i);
  for (int kt = 0, buf = 0; kt < nkt; ++kt) {
    phase(x, y, place(buf, 1));
    if (kt + NB <= nkt)
      landed(std::integral_constant<int, NB - 2>{});
    else
      tile_barrier();
    if (kt + NB < nkt) dma(buf, kt + NB);
    buf = buf + 1 == NB ? 0 : buf + 1;
    phase(y, x, place(buf, 0));  // (behind the last stage: of no use)
  }

  // lane l holds C[t][o .. o + 3] with t = .. + 16 i + l % 16, o = .. + 16 j + 4 (l / 16)
  const auto rsw = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(g.sw), static_cast<int16_t>(0), g.O * 4, kBufferWord3);
  f32x4_t sw[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      sw[j][e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rsw, 4 * (o0 + 16 * (NJ * wn + j) + 4 * kb + e), 0, 0));
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int t = t0 + 16 * (NI * wm + i) + r16;
    if (t >= g.T) continue;
    const float sa = g.sa[t];
#pragma unroll
    for (int j = 0; j < NJ; ++j) put4<OUT>(g, t, o0 + 16 * (NJ * wn + j) + 4 * kb, acc[i][j], sa, sw[j]);
  }
}

// ---- rows ---------------------------------------------------------------------------------------

constexpr int kRowWaves = 8;
constexpr int kRowAhead = 4;  // 128-byte pieces of W on their way (6 and 8: 24.5 us where 4 takes 20.4; four waves with 8: 21.1)

// 16 NT rows of A (blockIdx.y) by 16 NO channels
template <int NT, int NO, int OUT>
__global__ __launch_bounds__(64 * kRowWaves) void rows_kernel(Gemm g) {
  __shared__ __align__(16) i32x4_t s_acc[kRowWaves][NT * NO][64];
  const int lane = threadIdx.x & 63, r16 = lane & 15, kb = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int H = g.H, o0 = 16 * NO * blockIdx.x, t0 = 16 * NT * blockIdx.y;
  const auto rw = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(g.w) + static_cast<int64_t>(o0) * H, static_cast<int16_t>(0),
                                                    min(16 * NO, g.O - o0) * H, kBufferWord3);
  const auto ra = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(g.a) + static_cast<int64_t>(t0) * H, static_cast<int16_t>(0),
                                                    min(16 * NT, g.T - t0) * H, kBufferWord3);
  i32x4_t acc[NT][NO];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < NO; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};
  struct Piece {
    u32x4_t w[NO][2], a[NT][2];
  } p[kRowAhead];
  auto load = [&](Piece& x, int k) __attribute__((always_inline)) {  // bytes k .. k + 127 of the rows
    const int at = k + 32 * kb;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t past = at + 16 * h < H ? 0u : kOut;
#pragma unroll
      for (int j = 0; j < NO; ++j) x.w[j][h] = __builtin_amdgcn_raw_buffer_load_b128(rw, static_cast<uint32_t>((16 * j + r16) * H + at + 16 * h) | past, 0, 0);
#pragma unroll
      for (int i = 0; i < NT; ++i) x.a[i][h] = __builtin_amdgcn_raw_buffer_load_b128(ra, static_cast<uint32_t>((16 * i + r16) * H + at + 16 * h) | past, 0, 0);
    }
  };
  constexpr int kStep = kRowWaves * kStage;
  const int k0 = kStage * wv;
#pragma unroll
  for (int q = 0; q < kRowAhead; ++q) load(p[q], k0 + q * kStep);  // (past the end: zeros, and no memory is touched)
  for (int k = k0; k < H; k += kRowAhead * kStep) {
#pragma unroll
    for (int q = 0; q < kRowAhead; ++q) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int j = 0; j < NO; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, p[q].w[j][h]), __builtin_bit_cast(i32x4_t, p[q].a[i][h]),
                                                              acc[i][j], 0, 0, 0);
      load(p[q], k + (kRowAhead + q) * kStep);
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < NO; ++j) s_acc[wv][i * NO + j][lane] = acc[i][j];
  __syncthreads();
  for (int x = threadIdx.x; x < NT * NO * 64; x += 64 * kRowWaves) {
    const int ij = x >> 6, l = x & 63;
    i32x4_t sum = s_acc[0][ij][l];
#pragma unroll
    for (int w = 1; w < kRowWaves; ++w) sum += s_acc[w][ij][l];
    const int t = t0 + 16 * (ij / NO) + (l & 15), o = o0 + 16 * (ij % NO) + 4 * (l >> 4);
    if (t >= g.T || o >= g.O) continue;
    f32x4_t sw;
#pragma unroll
    for (int e = 0; e < 4; ++e) sw[e] = g.sw[min(o + e, g.O - 1)];
    put4<OUT>(g, t, o, sum, g.sa[t], sw);
  }
}

// The smallest tile whose number the device still holds at once has the shortest walk (64 x 64: two a CU, the others one); more of
// them than that read A and W too often, where there is more than one band of rows.  us of 64 x 64, 128 x 128, 256 x 256, with eight waves:
//   200 x 8192 x 8192   29.2  40.8  89.8      1024 x 8192 x 8192    119  72.7  96.2
//   333 x 8200 x 4112   39.4  24.5  55.9      2048 x 4096 x 4096   60.7  39.3  53.3
//   320 x 8192 x 4096   27.2  21.8            4096 x 4096 x 4096    122  88.3  62.6
// and 128 x 256, where it fits: 1024 x 8192 x 8192 70.4, 2048 x 4096 x 4096 38.5.  Four waves a workgroup hide less of a stage's
// waits: 100 x 1024 x 8192 19.3 (eight: 17.5), 128 x 4096 x 4096 11.6 (10.8), 512 x 8192 x 8192 53.6 (42.5).
// One band of rows reads W once whatever its tiles are, and taller ones multiply zeros; us of 64 x 64, 128 x 128, 128 x 256, 256 x 256:
//   48 x 131072 x 4096   107  126  126  137      100 x 131072 x 4096   152  137  135  145
//   64 x 65536 x 8192    113  122  125  135      128 x 65536 x 8192    179  129  131  141
//   64 x 32832 x 8192   71.4 91.2 68.9 90.8      65 x 65536 x 4096    76.6 69.5 67.8 70.8
// Up to 32 rows without tiles: 20 x 8192 x 8192 20.2 us; 50 rows took 26.8 that way, in 64 x 64 tiles 18.6.
template <int OUT>
hipError_t go(const Gemm& g, hipStream_t s) {
  auto tiles = [&](int bt, int bo) { return static_cast<int64_t>(ceil_div(g.T, bt)) * ceil_div(g.O, bo); };
  auto run = [&](auto bt, auto bo, auto nb) {
    constexpr int BT = decltype(bt)::value, BO = decltype(bo)::value, NB = decltype(nb)::value;
    tile_kernel<BT, BO, 2, 4, NB, OUT><<<static_cast<uint32_t>(8 * ceil_div(tiles(BT, BO), 8)), 512, 0, s>>>(
        g, static_cast<int32_t>(ceil_div(g.T, BT)), static_cast<int32_t>(ceil_div(g.O, BO)));
  };
  if (g.T <= 32) {
    if (g.T <= 16) rows_kernel<1, 1, OUT><<<static_cast<uint32_t>(ceil_div(g.O, 16)), 64 * kRowWaves, 0, s>>>(g);
    else rows_kernel<2, 2, OUT><<<static_cast<uint32_t>(ceil_div(g.O, 32)), 64 * kRowWaves, 0, s>>>(g);
  } else if (g.T <= 64 || tiles(64, 64) <= 512) {
    run(std::integral_constant<int, 64>{}, std::integral_constant<int, 64>{}, std::integral_constant<int, 4>{});
  } else if (tiles(128, 128) <= 256) {
    run(std::integral_constant<int, 128>{}, std::integral_constant<int, 128>{}, std::integral_constant<int, 3>{});
  } else if (g.T <= 128 || tiles(128, 256) <= 256) {
    run(std::integral_constant<int, 128>{}, std::integral_constant<int, 256>{}, std::integral_constant<int, 3>{});
  } else {
    run(std::integral_constant<int, 256>{}, std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_gemm(int64_t T, int64_t O, int64_t H, const uint8_t* a, const float* sa, const uint8_t* w, const float* sw, void* c,
                            int32_t out, hipStream_t s) {
  const uintptr_t al = out == kOutF32 ? 16 : 8;
  const Gemm g{a, w, sa, sw, c, static_cast<int32_t>(T), static_cast<int32_t>(O), static_cast<int32_t>(H),
               O % 4 == 0 && reinterpret_cast<uintptr_t>(c) % al == 0};
  return out == kOutF32 ? go<kOutF32>(g, s) : out == kOutF16 ? go<kOutF16>(g, s) : go<kOutBF16>(g, s);
}

}  // namespace fq
