// Log probabilities of given tokens, entropy and the best alternatives, from
// logits.
#include "wq_device.cuh"
#include "wq_internal.h"

#include <math_constants.h>

namespace wq {
namespace {

constexpr int kThreads = 512;

template <bool kBf16>
__device__ __forceinline__ float logit(const void* row, int64_t i) {
  if constexpr (kBf16) return bf16_bits_to_float(static_cast<const uint16_t*>(row)[i]);
  else return static_cast<const float*>(row)[i];
}

// The order of the tokens as one number: a larger logit is larger (NaN above
// all, -0.0 as 0.0), then a smaller id.
__device__ __forceinline__ uint64_t order_key(float x, uint32_t id) {
  uint32_t u = __float_as_uint(x + 0.0f);
  u = x != x ? 0xFFFFFFFFu : ((u >> 31) != 0 ? ~u : u | 0x80000000u);
  return static_cast<uint64_t>(u) << 32 | (0xFFFFFFFFu - id);
}

template <typename X, typename Op>
__device__ X block_reduce(X v, Op op) {
  __shared__ X part[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = part[0];
  for (int i = 1; i < kThreads / 32; ++i) v = op(v, part[i]);
  return v;
}

// One block per row: the largest logit, then the sums, then the best top_k by
// as many passes.
template <bool kBf16>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LogprobArgs a) {
  const int64_t t = blockIdx.x;
  const void* row = static_cast<const uint8_t*>(a.logits) + t * a.ld * (kBf16 ? 2 : 4);
  auto max_op = [](uint64_t x, uint64_t y) { return x > y ? x : y; };
  auto add = [](float x, float y) { return x + y; };
  uint64_t best = 0;
  for (int64_t i = threadIdx.x; i < a.V; i += kThreads) best = max_op(best, order_key(logit<kBf16>(row, i), i));
  best = block_reduce(best, max_op);
  const float m = logit<kBf16>(row, 0xFFFFFFFFu - static_cast<uint32_t>(best));
  const bool none = m == -CUDART_INF_F;

  const int64_t id = a.ids != nullptr ? a.ids[t] : -1;
  const bool given = id >= 0 && id < a.V;
  const float xt = given ? logit<kBf16>(row, id) : 0.0f;
  const uint64_t key_t = given ? order_key(xt, id) : 0;
  const float inv = 1.0f / a.temperature;
  float l = 0.0f, s = 0.0f;
  int before = 0;
  for (int64_t i = threadIdx.x; i < a.V; i += kThreads) {
    const float x = logit<kBf16>(row, i);
    before += order_key(x, i) > key_t;
    const float d = none ? 0.0f : (x - m) * inv, e = expf(d);
    l += e;
    if (!(d == -CUDART_INF_F)) s += e * d;
  }
  l = block_reduce(l, add);
  s = block_reduce(s, add);
  before = block_reduce(before, [](int x, int y) { return x + y; });
  const float log_l = logf(l);
  if (threadIdx.x == 0) {
    if (a.ids != nullptr) {
      a.logprob[t] = given && !none ? (xt - m) * inv - log_l : -CUDART_INF_F;
      a.rank[t] = given ? 1 + before : 0;
      if (!given && a.bad != nullptr) atomicAdd(a.bad, 1);
    }
    if (a.entropy != nullptr) a.entropy[t] = none ? 0.0f : log_l - s / l;
  }
  for (int j = 0; j < a.top_k; ++j) {
    const uint32_t tok = 0xFFFFFFFFu - static_cast<uint32_t>(best);
    if (threadIdx.x == 0) {
      a.top_ids[t * a.top_k + j] = static_cast<int32_t>(tok);
      a.top_logprobs[t * a.top_k + j] = none ? -CUDART_INF_F : (logit<kBf16>(row, tok) - m) * inv - log_l;
    }
    const uint64_t last = best;
    best = 0;
    for (int64_t i = threadIdx.x; i < a.V; i += kThreads) {
      const uint64_t k = order_key(logit<kBf16>(row, i), i);
      if (k < last) best = max_op(best, k);
    }
    best = block_reduce(best, max_op);
  }
}

}  // namespace

size_t logprobs_ws_bytes(int64_t, int64_t, int) { return 0; }

cudaError_t launch_logprobs(const Ctx& c, const LogprobArgs& a) {
  if (a.type == WQ_LOGITS_BF16)
    logprobs_kernel<true><<<static_cast<unsigned>(a.T), kThreads, 0, c.stream>>>(a);
  else
    logprobs_kernel<false><<<static_cast<unsigned>(a.T), kThreads, 0, c.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace wq
