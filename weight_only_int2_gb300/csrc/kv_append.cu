// Writes new keys and values into the pages of a paged cache (bf16 as they
// are, or rounded to e4m3 with a scale per key head).
//
// Bound: a token's place takes three loads one after the other (its sequence and
// position, then the page id), so a few tokens cost that latency (64 tokens of 8
// key heads by 128: 1.8 us, nearly all of it the launch), and many the read and
// the write of their values, if enough of them are on their way: a thread loads
// its values before it knows where they go, with many tokens for two in a row, in
// no more than 32 registers, so that an SM holds its 2048 threads. 12289 tokens of
// 8 key heads by 128 into e4m3, 75.7 MB: 16 us, 4.7 TB/s; there the issue is
// next (three quarters of its slots: the codes and the indexes; with float32
// operations one by one 1.2 us more); into bf16, 100.7 MB, 17.8 us, 5.7 TB/s. Where two tokens a thread took 18.5
// us, one took 19.2, four 20.3 (72 registers), eight 23.6; blocks of 512 threads 19.3.
//
// The e4m3 code is that of the IEEE quotient x / w. With y = RN(1 / w),
// q = RN(x y) and r = x - q w (exact in one fma), RN(q + r y) is the correctly
// rounded quotient (Markstein, IBM J. Res. Dev. 34(1), 1990). x is clamped to
// +-500 w first (rounded up to bf16, beyond the largest code), and both are
// multiplied by a power of two that is not 1 for w outside 2^-64 .. 2^64, so that on
// the way nothing overflows and r loses no bits where the code is not 0 anyway.
#include "wq_cluster.cuh"
#include "wq_device.cuh"
#include "wq_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp8.h>

namespace wq {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint64_t pair(float x, float y) {
  return static_cast<uint64_t>(__float_as_uint(y)) << 32 | __float_as_uint(x);
}
__device__ __forceinline__ float low_of(uint64_t p) { return __uint_as_float(static_cast<uint32_t>(p)); }
__device__ __forceinline__ float high_of(uint64_t p) { return __uint_as_float(static_cast<uint32_t>(p >> 32)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// A scale for pairs of values: with f the power of two, -f, w = scale f,
// -RN(1 / w) and the two bf16 limits.
struct Scale {
  uint64_t minus_f, w, minus_y;
  uint32_t lim;
  __device__ explicit Scale(float s) {
    const __nv_bfloat16 top = __float2bfloat16_ru(fminf(500.0f * s, 3.3895313892515355e38f));
    const __nv_bfloat162 l = __nv_bfloat162(top, top);
    lim = *reinterpret_cast<const uint32_t*>(&l);
    const float f = s < 5.421010862427522e-20f ? 3.8685626227668134e+25f : (s > 1.8446744073709552e19f ? 5.421010862427522e-20f : 1.0f);
    const float r = -__frcp_rn(s * f);
    minus_f = pair(-f, -f);
    w = pair(s * f, s * f);
    minus_y = pair(r, r);
  }
};

// Two bf16 numbers (the halves of p) over w as two e4m3 codes. (With the signs as
// they are here, -0.0 stays -0.0.)
__device__ __forceinline__ uint32_t codes_of(uint32_t p, const Scale& s) {
  asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(p) : "r"(s.lim));
  asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(p) : "r"(s.lim | 0x80008000u));
  const uint64_t minus_x = mul2(pair(__uint_as_float(p << 16), __uint_as_float(p & 0xFFFF0000u)), s.minus_f);
  const uint64_t z = mul2(minus_x, s.minus_y), q = fma2(fma2(z, s.w, minus_x), s.minus_y, z);
  return __nv_cvt_float2_to_fp8x2(make_float2(low_of(q), high_of(q)), __NV_SATFINITE, __NV_E4M3);
}

// By scales beyond kHuge an infinite number clamped to bf16's largest does not
// saturate: the thread writes the codes of those among its values once more. (A call
// that finds everything again, so that the kernel keeps its registers.)
constexpr float kHuge = 3.3e35f;
__device__ __noinline__ void infinite_by_huge(uint8_t* kv, int side, const int32_t* table, int64_t B, int64_t W,
                                              int64_t S, int64_t P, int Hkv, int D, const uint16_t* src, int64_t stride,
                                              int tokens, int64_t T, const int32_t* seq, const int32_t* pos) {
  const int row = Hkv * D / 16;
  const int64_t u = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x, t0 = u / (2 * row) * tokens;
  const int at = static_cast<int>(u % (2 * row)) % row * 16, h = at / D;
#pragma unroll 1
  for (int64_t t = t0; t < t0 + tokens && t < T; ++t) {
    const int64_t s = seq != nullptr ? seq[t] : t, p = pos[t];
    if (s < 0 || s >= B || p < 0 || p >= W * S) continue;
    const int64_t page = table[s * W + p / S];
    if (page < 0 || page >= P) continue;
    uint8_t* dst = kv + (((page * 2 + side) * Hkv + h) * S + p % S) * D + (at - h * D);
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {
      const uint32_t x = src[t * stride + at + i];
      if ((x & 0x7FFFu) == 0x7F80u) dst[i] = static_cast<uint8_t>(x >> 15 << 7 | 0x7Eu);
    }
  }
}

// One thread per 16 bytes of the cache (8 bf16 values or 16 codes) of kTokens
// tokens in a row: chunk i of a token, keys first.
template <bool kE4m3, int kTokens>
__global__ void __launch_bounds__(kThreads, 8) kv_append_kernel(const KvCache a, const uint16_t* __restrict__ k,
                                                            const uint16_t* __restrict__ v, int64_t k_stride,
                                                            int64_t v_stride, int64_t T,
                                                            const int32_t* __restrict__ seq,
                                                            const int32_t* __restrict__ pos,
                                                            int32_t* __restrict__ bad) {
  constexpr int kValues = kE4m3 ? 16 : 8, kLoads = kValues / 8;
  const uint32_t per_head = static_cast<uint32_t>(a.D) / kValues, row = static_cast<uint32_t>(a.Hkv) * per_head;
  // (64-bit places are divided only where they are past 32 bits)
  const int64_t u0 = static_cast<int64_t>(blockIdx.x) * kThreads;
  const int64_t g0 = u0 <= 0xFFFFFFFFll ? static_cast<uint32_t>(u0) / (2 * row) : u0 / (2 * row);
  const uint32_t in = static_cast<uint32_t>(u0 - g0 * 2 * row) + threadIdx.x;
  const int64_t t0 = (g0 + in / (2 * row)) * kTokens;
  if (t0 >= T) return;
  const uint32_t i = in % (2 * row), side = i >= row, at = i - side * row, h = at / per_head, d = (at - h * per_head) * kValues;

  cl::griddep_wait();
  uint4 x[kTokens][kLoads];
  int32_t s[kTokens], p[kTokens];
#pragma unroll
  for (int j = 0; j < kTokens; ++j) {
    s[j] = p[j] = -1;
    if (t0 + j >= T) continue;
    s[j] = seq != nullptr ? seq[t0 + j] : static_cast<int32_t>(t0 + j);
    p[j] = pos[t0 + j];
    const uint16_t* src = side ? v + (t0 + j) * v_stride : k + (t0 + j) * k_stride;
#pragma unroll
    for (int l = 0; l < kLoads; ++l) x[j][l] = __ldcs(reinterpret_cast<const uint4*>(src + h * a.D + d) + l);
  }
  int32_t page[kTokens];
  const uint32_t S = static_cast<uint32_t>(a.S);
#pragma unroll
  for (int j = 0; j < kTokens; ++j) {
    page[j] = -1;
    if (s[j] >= 0 && s[j] < a.B && p[j] >= 0 && p[j] < a.W * a.S)
      page[j] = a.table[static_cast<int64_t>(s[j]) * a.W + static_cast<uint32_t>(p[j]) / S];
  }
  float w = 1.0f;
  if constexpr (kE4m3) w = side ? a.v_scale[h] : a.k_scale[h];
  const Scale scale(w);
#pragma unroll
  for (int j = 0; j < kTokens; ++j) {
    if (page[j] < 0 || page[j] >= a.P) {
      if (i == 0 && bad != nullptr && t0 + j < T) atomicAdd(bad, 1);
      continue;
    }
    const int64_t dst = (((static_cast<int64_t>(page[j]) * 2 + side) * a.Hkv + h) * a.S + static_cast<uint32_t>(p[j]) % S) * a.D + d;
    if constexpr (!kE4m3) {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.kv) + dst) = x[j][0];
    } else {
      uint32_t o[4];
#pragma unroll
      for (int l = 0; l < 2; ++l) {
        o[2 * l] = codes_of(x[j][l].x, scale) | codes_of(x[j][l].y, scale) << 16;
        o[2 * l + 1] = codes_of(x[j][l].z, scale) | codes_of(x[j][l].w, scale) << 16;
      }
      *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.kv) + dst) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
  if (kE4m3 && w > kHuge)
    infinite_by_huge(static_cast<uint8_t*>(a.kv), side, a.table, a.B, a.W, a.S, a.P, static_cast<int>(a.Hkv),
                     static_cast<int>(a.D), side ? v : k, side ? v_stride : k_stride, kTokens, T, seq, pos);
}

}  // namespace

cudaError_t launch_kv_append(const Ctx& c, const KvCache& a, const uint16_t* k, const uint16_t* v, int64_t k_stride,
                             int64_t v_stride, int64_t T, const int32_t* seq, const int32_t* pos, int32_t* bad) {
  const bool e4m3 = a.type == WQ_KV_E4M3;
  const int64_t chunks = 2 * a.Hkv * a.D / (e4m3 ? 16 : 8);
  // one token a thread while the SMs hold them all at once (64 tokens: two a
  // thread take 0.3 us more)
  const bool many = T * chunks > int64_t{8} * kThreads * c.sm_count;
  const int64_t grid = ((many ? (T + 1) / 2 : T) * chunks + kThreads - 1) / kThreads;
  if (grid > kMaxDim) return cudaErrorInvalidConfiguration;
  const auto kern = e4m3 ? (many ? kv_append_kernel<true, 2> : kv_append_kernel<true, 1>)
                         : (many ? kv_append_kernel<false, 2> : kv_append_kernel<false, 1>);
  return launch_early(c, grid, kThreads, 0, kern, a, k, v, k_stride, v_stride, T, seq, pos, bad);
}

}  // namespace wq
