// The router of a mixture of experts and its gradient, and the rows of the tokens'
// choices: spread to the experts' order, brought back with weights, and that
// gradient.
#include "wq_cluster.cuh"
#include "wq_device.cuh"
#include "wq_internal.h"

namespace wq {
namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kThreads = 256;

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
  return x;
}
// The largest of the lanes' numbers (NaN only where all are).
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kAll, x, o));
  return x;
}

// ---------------------------------------------------------------- router
//
// A warp per token; lane l holds the experts l, l + 32, .. as keys in the order of
// the choice (larger logits first, NaN before all, 0.0 and -0.0 equal; 0 for -inf,
// which is never chosen). A choice is two reductions of the warp: the largest key,
// then the lowest expert that has it; only the lane that held it looks for its next.
// Bound: a decode batch by the launch, many tokens by the issue of the choices.

__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return kAll;
  const uint32_t b = __float_as_uint(x + 0.0f);
  if (b == 0xFF800000u) return 0;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  if (k == kAll) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

template <bool kF32>
__device__ __forceinline__ float logit(const void* row, int64_t e) {
  if constexpr (kF32) return static_cast<const float*>(row)[e];
  return bf16_bits_to_float(static_cast<const uint16_t*>(row)[e]);
}

__device__ __forceinline__ float sigmoid(float x) {
  const float e = expf(-fabsf(x));
  return x >= 0.0f ? 1.0f / (1.0f + e) : e / (1.0f + e);
}

// The chosen logits' weights without the scale, one a lane (lane j's logit x, `held`
// if it is a choice). top: their largest.
__device__ __forceinline__ float chosen_weight(float x, bool held, float top, int score, bool renormalize) {
  float p = 0.0f;
  if (score == WQ_SCORE_SOFTMAX) {
    p = held ? expf(x - top) : 0.0f;  // (only renormalized: their own softmax)
  } else if (renormalize && top < -20.0f) {
    p = held ? expf(x - top) : 0.0f;  // sigmoid(x) = exp(x) to 2^-28 of itself, and all may be below 2^-126
  } else {
    p = held ? sigmoid(x) : 0.0f;
  }
  if (!renormalize) return p;
  const float sum = warp_sum(p);
  return held ? p / sum : 0.0f;
}

template <bool kF32, int kPer>
__global__ void __launch_bounds__(kThreads) route_kernel(const RouteArgs a, int32_t* __restrict__ ids,
                                                         float* __restrict__ weights) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  cl::griddep_wait();
  cl::griddep_launch_dependents();
  if (t >= a.T) return;
  const char* row = static_cast<const char*>(a.logits) + t * a.ld * (kF32 ? 4 : 2);
  const int E = static_cast<int>(a.E);
  uint32_t key[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) key[i] = 32 * i + lane < E ? order_key(logit<kF32>(row, 32 * i + lane)) : 0u;
  float sum = 1.0f, top_all = 0.0f;
  if (a.score == WQ_SCORE_SOFTMAX && !a.renormalize) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) best = max(best, key[i]);
    best = __reduce_max_sync(kAll, best);
    top_all = best != 0 ? key_value(best) : 0.0f;
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += key[i] != 0 ? expf(key_value(key[i]) - top_all) : 0.0f;
    sum = warp_sum(sum);
  }
  uint32_t mine = 0;  // this lane's largest key not chosen yet
  int at = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (key[i] > mine) mine = key[i], at = i;
  uint32_t chosen = 0;
  int id = -1;
  for (int j = 0; j < a.k; ++j) {
    const uint32_t best = __reduce_max_sync(kAll, mine);
    const uint32_t e = __reduce_min_sync(kAll, mine == best ? 32u * at + lane : kAll);
    if (best != 0 && (e & 31) == lane) {
      // (the key itself goes, then its lane's next largest, the first among equals)
      mine = 0;
      const int gone = at;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (i == gone) key[i] = 0;
        if (key[i] > mine) mine = key[i], at = i;
      }
    }
    if (lane == j && best != 0) chosen = best, id = static_cast<int>(e);
  }
  const bool held = id >= 0;
  const float x = held ? key_value(chosen) : 0.0f;
  const float top = __shfl_sync(kAll, x, 0);
  float w;
  if (a.score == WQ_SCORE_SOFTMAX && !a.renormalize)
    w = held ? expf(x - top_all) / sum : 0.0f;
  else
    w = chosen_weight(x, held, top, a.score, a.renormalize != 0);
  if (lane < a.k) {
    ids[t * a.k + lane] = id;
    weights[t * a.k + lane] = a.scale * w;
  }
}

template <bool kF32>
__device__ __forceinline__ void put(void* row, int64_t e, float v) {
  if constexpr (kF32)
    static_cast<float*>(row)[e] = v;
  else
    static_cast<uint16_t*>(row)[e] = float_to_bf16_bits_rn(v);
}

// The sum of v over the lanes with this lane's id (as a rule, no other has it).
__device__ __forceinline__ float sum_of_same(float v, int id) {
  const uint32_t same = __match_any_sync(kAll, id >= 0 ? id : -1 - static_cast<int>(threadIdx.x & 31));
  if (!__any_sync(kAll, __popc(same) > 1)) return v;
  float s = 0.0f;
  for (int j = 0; j < 32; ++j) {
    const float o = __shfl_sync(kAll, v, j);
    if (same >> j & 1) s += o;
  }
  return s;
}

// With g = scale dweights at the choices: softmax over all experts gives
// p_e (g_e - sum g p), with g_e = 0 elsewhere; the other scores reach the chosen
// logits only: renormalized p (g - sum g p), times 1 - sigmoid where that is the
// score, and plain sigmoid g p (1 - p). A lane holds a choice; the warp writes the
// row's other values first.
template <bool kF32, int kPer>
__global__ void __launch_bounds__(kThreads) route_grad_kernel(const RouteArgs a, const int32_t* __restrict__ ids,
                                                              const float* __restrict__ dweights, void* dlogits) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  cl::griddep_wait();
  cl::griddep_launch_dependents();
  if (t >= a.T) return;
  const int E = static_cast<int>(a.E);
  const char* row = static_cast<const char*>(a.logits) + t * a.ld * (kF32 ? 4 : 2);
  char* drow = static_cast<char*>(dlogits) + t * a.E * (kF32 ? 4 : 2);
  int id = -1;
  float g = 0.0f;
  if (lane < a.k) {
    id = ids[t * a.k + lane];
    g = a.scale * dweights[t * a.k + lane];
  }
  if (id >= E) id = -1;
  float x = id >= 0 ? logit<kF32>(row, id) : -INFINITY;
  if (x == -INFINITY) id = -1;
  const bool held = id >= 0;
  if (!held) g = 0.0f;
  const bool over_all = a.score == WQ_SCORE_SOFTMAX && !a.renormalize;
  float d;
  if (over_all) {
    float v[kPer], top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      v[i] = 32 * i + lane < E ? logit<kF32>(row, 32 * i + lane) : -INFINITY;
      top = fmaxf(top, v[i]);
    }
    top = warp_max(top);
    if (top == -INFINITY) top = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      v[i] = expf(v[i] - top);
      sum += v[i];
    }
    sum = warp_sum(sum);
    const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
    const float p = held ? expf(x - top) * inv : 0.0f;
    const float mean = warp_sum(g * p);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (32 * i + lane < E) put<kF32>(drow, 32 * i + lane, -mean * (v[i] * inv));
    d = p * (sum_of_same(g, id) - mean);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (32 * i + lane < E) put<kF32>(drow, 32 * i + lane, 0.0f);
    const float top = warp_max(x);
    const float p = chosen_weight(held ? x : 0.0f, held, top, a.score, a.renormalize != 0);
    const float mean = a.renormalize ? warp_sum(g * p) : 0.0f;
    d = p * (g - mean);
    if (a.score == WQ_SCORE_SIGMOID) d *= sigmoid(-x);
    d = sum_of_same(held ? d : 0.0f, id);
  }
  __syncwarp();
  if (held) put<kF32>(drow, id, d);
}

// ---------------------------------------------------------------- rows
//
// Bound: HBM; nothing but the rows is read or written. A thread has 16 bytes of a
// token's row and goes over the token's choices: spread reads them once and writes k
// times, combine has its k loads on their way at once, which many threads turn into
// enough bytes in flight. Rows whose length is no multiple of 8 go value by value.

struct Place {
  int64_t t;
  int64_t c;
};
// This thread's token and place in its row of C pieces, flat over all tokens.
__device__ __forceinline__ Place flat_place(int64_t C) {
  const int64_t u0 = static_cast<int64_t>(blockIdx.x) * kThreads;
  // (64-bit places are divided only where they are past 32 bits)
  const int64_t t0 = u0 <= 0xFFFFFFFFll ? static_cast<uint32_t>(u0) / static_cast<uint32_t>(C) : u0 / C;
  const uint32_t in = static_cast<uint32_t>(u0 - t0 * C) + threadIdx.x;
  const uint32_t more = in / static_cast<uint32_t>(C);
  return Place{t0 + more, static_cast<int64_t>(in - more * static_cast<uint32_t>(C))};
}

template <int kVec>
struct Piece;  // kVec bf16 values
template <>
struct Piece<8> {
  using type = uint4;
  __device__ static void widen(const uint4& p, float (&v)[8]) {
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ static uint4 narrow(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Piece<1> {
  using type = uint16_t;
  __device__ static void widen(const uint16_t& p, float (&v)[1]) { v[0] = bf16_bits_to_float(p); }
  __device__ static uint16_t narrow(const float (&v)[1]) { return float_to_bf16_bits_rn(v[0]); }
};

constexpr int kBatch = 8;  // choices whose rows are on their way at once

template <int kVec>
__global__ void __launch_bounds__(kThreads) spread_kernel(const ChoiceRows a, const uint16_t* __restrict__ x,
                                                          int64_t x_stride, uint16_t* __restrict__ out) {
  using V = typename Piece<kVec>::type;
  const Place p = flat_place(a.D / kVec);
  cl::griddep_wait();
  cl::griddep_launch_dependents();
  if (p.t >= a.T) return;
  const V v = reinterpret_cast<const V*>(x + p.t * x_stride)[p.c];
  const int32_t* slots = a.slots + p.t * a.k;
  for (int j0 = 0; j0 < a.k; j0 += kBatch) {
    int32_t s[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) s[j] = j0 + j < a.k ? slots[j0 + j] : -1;
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (s[j] >= 0 && s[j] < a.R) reinterpret_cast<V*>(out + s[j] * a.D)[p.c] = v;
  }
}

template <int kVec>
__global__ void __launch_bounds__(kThreads) combine_kernel(const ChoiceRows a, const uint16_t* __restrict__ y,
                                                           const uint16_t* residual, uint16_t* out) {
  using P = Piece<kVec>;
  using V = typename P::type;
  const Place p = flat_place(a.D / kVec);
  cl::griddep_wait();
  cl::griddep_launch_dependents();
  if (p.t >= a.T) return;
  float acc[kVec] = {};
  if (residual != nullptr) P::widen(reinterpret_cast<const V*>(residual + p.t * a.D)[p.c], acc);
  const int64_t at = p.t * a.k;
  for (int j0 = 0; j0 < a.k; j0 += kBatch) {
    int32_t s[kBatch];
    float w[kBatch];
    V v[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) s[j] = j0 + j < a.k ? a.slots[at + j0 + j] : -1;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      w[j] = 0.0f;
      v[j] = V{};
      if (s[j] < 0 || s[j] >= a.R) continue;
      w[j] = a.weights != nullptr ? a.weights[at + j0 + j] : 1.0f;
      v[j] = reinterpret_cast<const V*>(y + s[j] * a.D)[p.c];
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      float f[kVec];
      P::widen(v[j], f);
#pragma unroll
      for (int i = 0; i < kVec; ++i) acc[i] = fmaf(w[j], f[i], acc[i]);
    }
  }
  reinterpret_cast<V*>(out + p.t * a.D)[p.c] = P::narrow(acc);
}

// The sums over the lanes of 8 numbers: lane l has that of number l / 4. Halves of
// the numbers go to halves of the lanes, so that 9 exchanges do.
__device__ __forceinline__ float eight_sums(const float (&v)[8]) {
  const int lane = threadIdx.x & 31;
  float u[4], w[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float keep = lane & 16 ? v[4 + i] : v[i], give = lane & 16 ? v[i] : v[4 + i];
    u[i] = keep + __shfl_xor_sync(kAll, give, 16);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float keep = lane & 8 ? u[2 + i] : u[i], give = lane & 8 ? u[i] : u[2 + i];
    w[i] = keep + __shfl_xor_sync(kAll, give, 8);
  }
  const float keep = lane & 4 ? w[1] : w[0], give = lane & 4 ? w[0] : w[1];
  float s = keep + __shfl_xor_sync(kAll, give, 4);
  s += __shfl_xor_sync(kAll, s, 2);
  return s + __shfl_xor_sync(kAll, s, 1);
}

// A block per token: dy's rows are written as y's are read, and the products with
// dout are summed over the block in a fixed order.
template <int kVec>
__global__ void __launch_bounds__(kThreads) combine_grad_kernel(const ChoiceRows a, const uint16_t* __restrict__ dout,
                                                                const uint16_t* __restrict__ y, uint16_t* dy,
                                                                float* __restrict__ dweights) {
  using P = Piece<kVec>;
  using V = typename P::type;
  __shared__ float part[kThreads / 32][kBatch];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t t = blockIdx.x, at = t * a.k;
  const int C = static_cast<int>(a.D / kVec);
  cl::griddep_wait();
  cl::griddep_launch_dependents();
  for (int j0 = 0; j0 < a.k; j0 += kBatch) {
    int32_t s[kBatch];
    float w[kBatch], dot[kBatch] = {};
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      s[j] = j0 + j < a.k ? a.slots[at + j0 + j] : -1;
      if (s[j] >= a.R) s[j] = -1;
      w[j] = s[j] >= 0 ? a.weights[at + j0 + j] : 0.0f;
    }
    for (int c = threadIdx.x; c < C; c += blockDim.x) {
      float g[kVec];
      V v[kBatch];
      P::widen(reinterpret_cast<const V*>(dout + t * a.D)[c], g);
#pragma unroll
      for (int j = 0; j < kBatch; ++j) v[j] = s[j] >= 0 ? reinterpret_cast<const V*>(y + s[j] * a.D)[c] : V{};
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (s[j] < 0) continue;
        float f[kVec];
        P::widen(v[j], f);
#pragma unroll
        for (int i = 0; i < kVec; ++i) dot[j] = fmaf(g[i], f[i], dot[j]);
#pragma unroll
        for (int i = 0; i < kVec; ++i) f[i] = w[j] * g[i];
        reinterpret_cast<V*>(dy + s[j] * a.D)[c] = P::narrow(f);
      }
    }
    const float sum = eight_sums(dot);
    if ((lane & 3) == 0) part[warp][lane >> 2] = sum;
    __syncthreads();
    if (threadIdx.x < kBatch && j0 + static_cast<int>(threadIdx.x) < a.k) {
      float d = 0.0f;
      for (int i = 0; i < warps; ++i) d += part[i][threadIdx.x];
      dweights[at + j0 + threadIdx.x] = d;
    }
    __syncthreads();
  }
}

template <bool kF32>
auto route_of(int64_t E) {
  return E <= 32    ? route_kernel<kF32, 1>
         : E <= 64  ? route_kernel<kF32, 2>
         : E <= 128 ? route_kernel<kF32, 4>
         : E <= 256 ? route_kernel<kF32, 8>
         : E <= 512 ? route_kernel<kF32, 16>
                    : route_kernel<kF32, 32>;
}
template <bool kF32>
auto route_grad_of(int64_t E) {
  return E <= 32    ? route_grad_kernel<kF32, 1>
         : E <= 64  ? route_grad_kernel<kF32, 2>
         : E <= 128 ? route_grad_kernel<kF32, 4>
         : E <= 256 ? route_grad_kernel<kF32, 8>
         : E <= 512 ? route_grad_kernel<kF32, 16>
                    : route_grad_kernel<kF32, 32>;
}

}  // namespace

cudaError_t launch_moe_route(const Ctx& c, const RouteArgs& a, int32_t* ids, float* weights) {
  const int64_t grid = (a.T + kThreads / 32 - 1) / (kThreads / 32);
  return launch_early(c, grid, kThreads, 0, a.type == WQ_LOGITS_F32 ? route_of<true>(a.E) : route_of<false>(a.E), a,
                      ids, weights);
}

cudaError_t launch_moe_route_grad(const Ctx& c, const RouteArgs& a, const int32_t* ids, const float* dweights,
                                  void* dlogits) {
  const int64_t grid = (a.T + kThreads / 32 - 1) / (kThreads / 32);
  return launch_early(c, grid, kThreads, 0,
                      a.type == WQ_LOGITS_F32 ? route_grad_of<true>(a.E) : route_grad_of<false>(a.E), a, ids,
                      dweights, dlogits);
}

namespace {
int64_t flat_grid(int64_t T, int64_t C) { return (T * C + kThreads - 1) / kThreads; }
}  // namespace

cudaError_t launch_moe_spread(const Ctx& c, const ChoiceRows& a, const uint16_t* x, int64_t x_stride, uint16_t* out) {
  const bool vec = a.D % 8 == 0 && x_stride % 8 == 0;
  const int64_t grid = flat_grid(a.T, vec ? a.D / 8 : a.D);
  if (grid > kMaxDim) return cudaErrorInvalidConfiguration;
  return launch_early(c, grid, kThreads, 0, vec ? spread_kernel<8> : spread_kernel<1>, a, x, x_stride, out);
}

cudaError_t launch_moe_combine(const Ctx& c, const ChoiceRows& a, const uint16_t* y, const uint16_t* residual,
                               uint16_t* out) {
  const bool vec = a.D % 8 == 0;
  const int64_t grid = flat_grid(a.T, vec ? a.D / 8 : a.D);
  if (grid > kMaxDim) return cudaErrorInvalidConfiguration;
  return launch_early(c, grid, kThreads, 0, vec ? combine_kernel<8> : combine_kernel<1>, a, y, residual, out);
}

cudaError_t launch_moe_combine_grad(const Ctx& c, const ChoiceRows& a, const uint16_t* dout, const uint16_t* y,
                                    uint16_t* dy, float* dweights) {
  return launch_early(c, a.T, kThreads, 0, a.D % 8 == 0 ? combine_grad_kernel<8> : combine_grad_kernel<1>, a, dout, y,
                      dy, dweights);
}

}  // namespace wq
