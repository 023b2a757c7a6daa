// Pieces of the attention kernels that work on tiles of keys in LDS: 32 x 32 x 16 products, LDS-DMA loads, steps between lanes.
#pragma once

#include <hip/hip_runtime.h>

#include "fq_attn_dev.h"

namespace fq {

// Weights as they enter the second product are 2^kUp times those above (at most 2^(8 + kUp), f16's largest binade):
// an f16 weight is then off by 2^-32 of the largest one where it is subnormal, not by 2^-25, which many keys far
// below one that stands out lost altogether (20000 of them 17.5 nats below: 5e-4 of the weights).
template <int DT>
constexpr float kUp = DT == kF16 ? 7.0f : 0.0f;
// Scores up to this far from 0, in base-2 units, have their maximum taken off within the weights' exponent; its rounding is 2^-5 there.
constexpr float kFar = 0x1p20f;
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

// a b, rounded by itself (not within a fused sum)
__device__ __forceinline__ float product(float a, float b) {
#pragma clang fp contract(off)
  return a * b;
}

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

}  // namespace fq
