// Attention of one new token per sequence over a paged key-value cache.
#include "wq_device.cuh"
#include "wq_internal.h"

#include <cuda_fp8.h>
#include <math_constants.h>

namespace wq {
namespace {

__device__ __forceinline__ float e4m3_to_float(uint8_t b) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
}

// One warp per (sequence, query head): a lane holds D / 32 values of the
// query and of the running sum.
template <int D, bool kE4m3>
__global__ void kv_attn_kernel(const KvCache a, const uint16_t* __restrict__ q, int64_t q_stride,
                               const int32_t* __restrict__ lens, int64_t Hq, float sm_scale, int64_t window,
                               uint16_t* __restrict__ out, float* __restrict__ lse, int32_t* __restrict__ bad) {
  constexpr int E = D / 32;
  const int64_t b = blockIdx.x / Hq, hq = blockIdx.x % Hq, G = Hq / a.Hkv, h = hq / G;
  const int lane = threadIdx.x;
  float qv[E], acc[E] = {};
#pragma unroll
  for (int e = 0; e < E; ++e) qv[e] = bf16_bits_to_float(q[b * q_stride + hq * D + lane + 32 * e]);
  int64_t len = lens[b];
  if (len > a.W * a.S) len = a.W * a.S;
  const int64_t first = window > 0 && len > window ? len - window : 0;
  const float ks = kE4m3 ? a.k_scale[h] * sm_scale : sm_scale, vs = kE4m3 ? a.v_scale[h] : 1.0f;
  float m = -CUDART_INF_F, l = 0.0f;
  for (int64_t t = first; t < len; ++t) {
    const int64_t page = a.table[b * a.W + t / a.S];
    if (page < 0 || page >= a.P) {
      if (bad != nullptr && lane == 0 && hq == 0 && (t % a.S == 0 || t == first)) atomicAdd(bad, 1);
      continue;
    }
    const int64_t kr = ((page * 2 * a.Hkv + h) * a.S + t % a.S) * D, vr = kr + a.Hkv * a.S * D;
    float x = 0.0f, vv[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int64_t i = lane + 32 * e;
      float kk;
      if constexpr (kE4m3) {
        kk = e4m3_to_float(static_cast<const uint8_t*>(a.kv)[kr + i]);
        vv[e] = e4m3_to_float(static_cast<const uint8_t*>(a.kv)[vr + i]);
      } else {
        kk = bf16_bits_to_float(static_cast<const uint16_t*>(a.kv)[kr + i]);
        vv[e] = bf16_bits_to_float(static_cast<const uint16_t*>(a.kv)[vr + i]);
      }
      x += qv[e] * kk;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    x *= ks;
    const float m2 = fmaxf(m, x), base = m2 == -CUDART_INF_F ? 0.0f : m2;
    const float w = expf(m - base), p = expf(x - base);
    m = m2;
    l = l * w + p;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * w + p * vv[e];
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    out[(b * Hq + hq) * D + lane + 32 * e] = float_to_bf16_bits_rn(l == 0.0f ? 0.0f : acc[e] * vs / l);
  if (lse != nullptr && lane == 0) lse[b * Hq + hq] = l == 0.0f ? -CUDART_INF_F : m + logf(l);
}

template <int D>
void launch_d(const Ctx& c, const KvCache& a, const uint16_t* q, int64_t q_stride, const int32_t* lens, int64_t Hq,
              float sm_scale, int64_t window, uint16_t* out, float* lse, int32_t* bad) {
  const unsigned grid = static_cast<unsigned>(a.B * Hq);
  if (a.type == WQ_KV_E4M3)
    kv_attn_kernel<D, true><<<grid, 32, 0, c.stream>>>(a, q, q_stride, lens, Hq, sm_scale, window, out, lse, bad);
  else
    kv_attn_kernel<D, false><<<grid, 32, 0, c.stream>>>(a, q, q_stride, lens, Hq, sm_scale, window, out, lse, bad);
}

}  // namespace

size_t kv_attn_ws_bytes(int64_t, int64_t, int64_t, int64_t) { return 0; }

cudaError_t launch_kv_attn(const Ctx& c, const KvCache& a, const uint16_t* q, int64_t q_stride, const int32_t* lens,
                           int64_t Hq, float sm_scale, int64_t window, uint16_t* out, float* lse, int32_t* bad,
                           void*) {
  switch (a.D) {
    case 64: launch_d<64>(c, a, q, q_stride, lens, Hq, sm_scale, window, out, lse, bad); break;
    case 96: launch_d<96>(c, a, q, q_stride, lens, Hq, sm_scale, window, out, lse, bad); break;
    case 128: launch_d<128>(c, a, q, q_stride, lens, Hq, sm_scale, window, out, lse, bad); break;
    case 192: launch_d<192>(c, a, q, q_stride, lens, Hq, sm_scale, window, out, lse, bad); break;
    case 256: launch_d<256>(c, a, q, q_stride, lens, Hq, sm_scale, window, out, lse, bad); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace wq
