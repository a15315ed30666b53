// Writes new keys and values into the pages of a paged cache (bf16 as they
// are, or rounded to e4m3 with a scale per key head).
#include "wq_device.cuh"
#include "wq_internal.h"

#include <cuda_fp8.h>

namespace wq {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// One thread per 8 values: chunk i of token t, keys first.
template <bool kE4m3>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvCache a, const uint16_t* __restrict__ k,
                                                            const uint16_t* __restrict__ v, int64_t k_stride,
                                                            int64_t v_stride, int64_t T,
                                                            const int32_t* __restrict__ seq,
                                                            const int32_t* __restrict__ pos,
                                                            int32_t* __restrict__ bad) {
  const int row = static_cast<int>(a.Hkv * a.D / 8);  // chunks of a token's keys
  const int64_t u = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t t = u / (2 * row);
  if (t >= T) return;
  const int i = static_cast<int>(u - t * 2 * row);
  const int side = i >= row, at = i - side * row;

  const int64_t s = seq != nullptr ? seq[t] : t;
  const int64_t p = pos[t];
  int64_t page = -1;
  if (s >= 0 && s < a.B && p >= 0 && p < a.W * a.S) page = a.table[s * a.W + p / a.S];
  if (page < 0 || page >= a.P) {
    if (i == 0 && bad != nullptr) atomicAdd(bad, 1);
    return;
  }
  const int per_head = static_cast<int>(a.D / 8);
  const int h = at / per_head, d = (at - h * per_head) * 8;
  const uint16_t* src = side ? v + t * v_stride : k + t * k_stride;
  const uint4 x = *reinterpret_cast<const uint4*>(src + h * a.D + d);
  const int64_t dst = (((page * 2 + side) * a.Hkv + h) * a.S + p % a.S) * a.D + d;
  if constexpr (!kE4m3) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.kv) + dst) = x;
  } else {
    const float w = side ? a.v_scale[h] : a.k_scale[h];
    const uint32_t r[4] = {x.x, x.y, x.z, x.w};
    uint32_t o[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t b[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t y = r[2 * j + e];
        b[e] = e4m3x2(__fdiv_rn(__uint_as_float(y << 16), w), __fdiv_rn(__uint_as_float(y & 0xFFFF0000u), w));
      }
      o[j] = b[0] | (b[1] << 16);
    }
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.kv) + dst) = make_uint2(o[0], o[1]);
  }
}

}  // namespace

cudaError_t launch_kv_append(const Ctx& c, const KvCache& a, const uint16_t* k, const uint16_t* v, int64_t k_stride,
                             int64_t v_stride, int64_t T, const int32_t* seq, const int32_t* pos, int32_t* bad) {
  const int64_t chunks = T * 2 * (a.Hkv * a.D / 8);
  const int64_t grid = (chunks + kThreads - 1) / kThreads;
  if (grid > kMaxDim) return cudaErrorInvalidConfiguration;
  if (a.type == WQ_KV_E4M3)
    kv_append_kernel<true><<<static_cast<unsigned>(grid), kThreads, 0, c.stream>>>(a, k, v, k_stride, v_stride, T,
                                                                                  seq, pos, bad);
  else
    kv_append_kernel<false><<<static_cast<unsigned>(grid), kThreads, 0, c.stream>>>(a, k, v, k_stride, v_stride, T,
                                                                                   seq, pos, bad);
  return cudaGetLastError();
}

}  // namespace wq
