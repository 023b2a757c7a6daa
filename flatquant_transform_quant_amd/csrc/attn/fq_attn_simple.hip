// Attention, the simplest form: one wave per (query row, query head).  Lane l scores key 64 i + l
// of step i by an fp32 dot product; the step's weights exp(s - m) are then handed round and
// every lane accumulates its elements of the output, with the running maximum m and sum l of
// the softmax in fp32.
#include <hip/hip_runtime.h>

#include "fq_attn_dev.h"

namespace fq {
namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// row(side, t): pointers of token t's codes and scale, or null if it has none
template <int MODE, int DT, typename Row>
__device__ __forceinline__ void attend(const uint16_t* q, uint16_t* out, float* lse, int D, int n, float scale, Row&& row) {
  __shared__ float qs[256];
  const int lane = threadIdx.x;
  for (int d = lane; d < D; d += 64) qs[d] = load16<DT>(q[d]) * scale;
  __syncthreads();
  float m = -__builtin_inff(), l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int t0 = 0; t0 < n; t0 += 64) {
    const int t = t0 + lane;
    const uint8_t *kp = nullptr, *ks = nullptr;
    if (t < n) row(0, t, kp, ks);
    float s = -__builtin_inff();
    if (kp) {
      s = 0.0f;
      for (int c = 0; 8 * c < D; ++c) {
        float x[8];
        kv_decode8<MODE, DT>(kv_load8<MODE>(kp, c), MODE == kKv16 || MODE == kKvFp4 ? 0.0f : *reinterpret_cast<const float*>(ks),
                             MODE == kKvFp4 ? ks[c / 4] : 0, x);
        for (int i = 0; i < 8; ++i) s = __builtin_fmaf(x[i], qs[8 * c + i], s);
      }
    }
    const float mn = fmaxf(m, wave_max(s)), ms = mn == -__builtin_inff() ? 0.0f : mn;
    const float a = __expf(m - ms), p = kp ? __expf(s - ms) : 0.0f;
    l = l * a + p;
    m = mn;
    for (int j = 0; j < 4; ++j) o[j] *= a;
    for (int i = 0; i < 64 && t0 + i < n; ++i) {
      const float pi = __shfl(p, i);
      const uint8_t *vp = nullptr, *vs = nullptr;
      row(1, t0 + i, vp, vs);
      if (!vp) continue;
      for (int j = 0; j < 4; ++j) {
        const int d = lane + 64 * j;
        if (d >= D) break;
        float x[8];
        kv_decode8<MODE, DT>(kv_load8<MODE>(vp, d / 8), MODE == kKv16 || MODE == kKvFp4 ? 0.0f : *reinterpret_cast<const float*>(vs),
                             MODE == kKvFp4 ? vs[d / 32] : 0, x);
        float v = x[0];
        for (int e = 1; e < 8; ++e) v = (d & 7) == e ? x[e] : v;
        o[j] = __builtin_fmaf(pi, v, o[j]);
      }
    }
  }
  l = wave_sum(l);
  for (int j = 0; j < 4; ++j)
    if (lane + 64 * j < D) out[lane + 64 * j] = round16<DT>(l == 0.0f ? 0.0f : o[j] / l);
  if (lse && lane == 0) *lse = l == 0.0f ? -__builtin_inff() : m + __logf(l);
}

template <int DT>
__global__ __launch_bounds__(64) void prefill_simple_kernel(PrefillArgs a) {
  const int t = blockIdx.y, h = blockIdx.x, hk = h / a.g;
  if (t >= a.cu_q[a.B]) return;
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (a.cu_q[m] <= t) lo = m; else hi = m;
  }
  const int q0 = a.cu_q[lo], lq = a.cu_q[lo + 1] - q0;
  const int k0 = max(0, min(a.cu_k[lo], a.Tk)), lk = max(0, min(a.cu_k[lo + 1], a.Tk) - k0);
  const int n = a.causal ? max(0, min(lk, lk - lq + (t - q0) + 1)) : lk;
  attend<kKv16, DT>(a.q.p + t * a.q.row + h * a.q.head, a.out.p + t * a.out.row + h * a.out.head,
                    a.lse ? a.lse + static_cast<int64_t>(t) * a.Hq + h : nullptr, a.D, n, a.scale,
                    [&](int side, int j, const uint8_t*& p, const uint8_t*&) {
                      const Rows16& r = side ? a.v : a.k;
                      p = reinterpret_cast<const uint8_t*>(r.p + (k0 + j) * r.row + hk * r.head);
                    });
}

}  // namespace

hipError_t launch_attn_prefill(const PrefillArgs& a, hipStream_t s) {
  const dim3 grid(a.Hq, a.Tq);
  if (a.dtype == kF16)
    prefill_simple_kernel<kF16><<<grid, 64, 0, s>>>(a);
  else
    prefill_simple_kernel<kBF16><<<grid, 64, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace fq
