// The router of a mixture of experts and its gradient, and the rows of the tokens'
// choices: spread to the experts' order, brought back with weights, and that
// gradient.
#include "wq_cluster.cuh"
#include "wq_device.cuh"
#include "wq_internal.h"

#include <algorithm>

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
// the choice: larger logits first, NaN before all, 0.0 and -0.0 equal; 0 for -inf,
// which is never chosen. The key's lowest bits make room for the expert (lower ones
// are larger numbers), so that one reduction of the warp finds a choice, all keys
// differ, and a lane sorts its own by minima and maxima alone; the lane whose largest
// was chosen moves on to its next. A bf16 logit's key has those bits to spare. Two
// float32 logits may differ in them alone: where neighbours among the chosen (or the
// last one and one that was not) have equal keys but for the expert, the token is
// done again by whole keys, equal logits too (16384 rows of 256 logits that were bf16
// before: 16.4 us; nothing but equal ones: 21.2).
// Bound: a decode batch by the launch (64 tokens: 1.7 us), many tokens by the issue
// (550 instructions a token of 256 experts, 80 % of the slots): 16384 rows of 256
// float32 logits, 8 chosen, 10.2 us. With two reductions and a search through the
// lane's keys a choice 20.5; with loads behind branches, each of which waited for the
// one before it, 15.1.

// (x + 0 is 0.0 for -0.0, and 0x7FFFFFFF for every NaN)
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
  const uint32_t key = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
  return key > 0x007FFFFFu ? key : 0u;  // -inf is 0x007FFFFF, the lowest
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

// The lane's logits, -inf beyond the last (all loads on their way at once).
template <bool kF32, int kPer>
__device__ __forceinline__ void load_row(const void* row, int E, float (&x)[kPer]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < kPer; ++i) x[i] = logit<kF32>(row, min(32 * i + lane, E - 1));
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (32 * i + lane >= E) x[i] = -INFINITY;
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

// This token's choices by whole keys: lane j's expert, -1 if none is left.
template <bool kF32, int kPer>
__device__ __noinline__ int choose_exactly(const void* row, int E, int k) {
  const int lane = threadIdx.x & 31;
  uint32_t key[kPer];
  {
    float x[kPer];
    load_row<kF32>(row, E, x);
#pragma unroll
    for (int i = 0; i < kPer; ++i) key[i] = order_key(x[i]);
  }
  int id = -1;
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    uint32_t mine = 0, at = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (key[i] > mine) mine = key[i], at = i;
    const uint32_t best = __reduce_max_sync(kAll, mine);
    if (best == 0) break;
    const uint32_t e = __reduce_min_sync(kAll, mine == best ? 32u * at + lane : kAll);
    if (lane == j) id = static_cast<int>(e);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (32u * i + lane == e) key[i] = 0;
  }
  return id;
}

// The larger keys first (Batcher's odd-even merge sort).
template <int kPer, int kP = 1, int kK = 1>
__device__ __forceinline__ void sort_down(uint32_t (&v)[kPer]) {
  if constexpr (kP < kPer) {
#pragma unroll
    for (int i = 0; i + kK < kPer; ++i) {
      constexpr int kFirst = kK % kP;
      if (i >= kFirst && (i - kFirst) % (2 * kK) < kK && i / (2 * kP) == (i + kK) / (2 * kP)) {
        const uint32_t x = v[i], y = v[i + kK];
        v[i] = max(x, y);
        v[i + kK] = min(x, y);
      }
    }
    if constexpr (kK > 1)
      sort_down<kPer, kP, kK / 2>(v);
    else
      sort_down<kPer, 2 * kP, 2 * kP>(v);
  }
}

template <bool kF32, int kPer>
__global__ void __launch_bounds__(kThreads) route_kernel(const RouteArgs a, int32_t* __restrict__ ids,
                                                         float* __restrict__ weights) {
  constexpr uint32_t kExpert = 32 * kPer - 1;  // the bits of the expert
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  cl::griddep_wait();
  cl::griddep_launch_dependents();
  if (t >= a.T) return;
  const char* row = static_cast<const char*>(a.logits) + t * a.ld * (kF32 ? 4 : 2);
  const int E = static_cast<int>(a.E);
  const bool over_all = a.score == WQ_SCORE_SOFTMAX && !a.renormalize;
  uint32_t key[kPer];
  float sum = 1.0f, top_all = 0.0f;
  {
    float x[kPer];
    load_row<kF32>(row, E, x);
#pragma unroll
    for (int i = 0; i < kPer; ++i) key[i] = order_key(x[i]);
    if (over_all) {
      uint32_t best = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) best = max(best, key[i]);
      best = __reduce_max_sync(kAll, best);
      top_all = best != 0 ? key_value(best) : 0.0f;
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) sum += expf(x[i] - top_all);  // (exp(-inf) is 0)
      sum = warp_sum(sum);
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (key[i] != 0) key[i] = (key[i] & ~kExpert) | (kExpert - (32 * i + lane));
  sort_down(key);
  uint32_t chosen = 0, last = 0;
  bool close = false;
  for (int j = 0; j < a.k; ++j) {
    const uint32_t best = __reduce_max_sync(kAll, key[0]);
    if (best == 0) break;
    if (lane == j) chosen = best;
    if (key[0] == best) {
#pragma unroll
      for (int i = 0; i + 1 < kPer; ++i) key[i] = key[i + 1];
      key[kPer - 1] = 0;
    }
    close |= (best ^ last) <= kExpert;
    last = best;
  }
  int id = chosen != 0 ? static_cast<int>(kExpert - (chosen & kExpert)) : -1;
  if constexpr (kF32) {
    close |= (key[0] ^ last) <= kExpert && key[0] != 0;
    if (__any_sync(kAll, close)) id = choose_exactly<kF32, kPer>(row, E, a.k);
  }
  const bool held = id >= 0;
  const float x = held ? logit<kF32>(row, id) : 0.0f;
  const float top = __shfl_sync(kAll, x, 0);
  float w;
  if (over_all)
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
    load_row<kF32>(row, E, v);
#pragma unroll
    for (int i = 0; i < kPer; ++i) top = fmaxf(top, v[i]);
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
// Bound: HBM; nothing but the rows is read or written. kLanes threads go along a
// token's row, 8 values at a time, and over its
// choices: spread reads a piece once and writes it k times, combine has its k loads
// on their way at once. Few tokens are cut into parts, so that more SMs have work.
// Measured for 8192 tokens of 8 choices of 5120: combine 129 us, 6.5 TB/s (a thread a
// piece, flat over all tokens, 143: many short blocks; 256 threads a token 137), its
// gradient 209 us, 6.8 TB/s, spread 113 us, 6.7 TB/s.

constexpr int kRowThreads = 128;  // of a block, unless a token has more

// 8 bf16 values.
__device__ __forceinline__ void widen(const uint4& p, float (&v)[8]) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 narrow(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Rows that do not begin at 16 bytes (kOdd) are written in whole pieces of 16 bytes,
// and read by two of them and a shift; a warp takes the values at the row's ends one a
// lane. (4096 tokens of 6 choices of 2049: spread 32 us, combine 49,
// its gradient 55; value by value 63, 88 and 78.)
//
// Values i .. i + 7, whose 16-byte pieces both lie in the array, as two loads without
// a branch (so that many are on their way at once) and a shift.
struct Odd8 {
  uint4 a, b;
  __device__ __forceinline__ void load(const uint16_t* p, int64_t i) {
    const uint4* v = reinterpret_cast<const uint4*>(p) + (i >> 3);
    a = v[0];
    b = v[(i & 7) != 0];
  }
  __device__ __forceinline__ uint4 get(int64_t i) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t s[7], t[5];
#pragma unroll
    for (int l = 0; l < 7; ++l) s[l] = i & 2 ? w[l + 1] : w[l];
#pragma unroll
    for (int l = 0; l < 5; ++l) t[l] = i & 4 ? s[l + 2] : s[l];
    const int half = 16 * static_cast<int>(i & 1);
    return make_uint4(__funnelshift_r(t[0], t[1], half), __funnelshift_r(t[1], t[2], half),
                      __funnelshift_r(t[2], t[3], half), __funnelshift_r(t[3], t[4], half));
  }
};
// A row of D that begins at value i of the array that is written: `head` values, then
// `full` pieces, then at most 15 values.
struct Ends {
  int64_t D;
  int head, full;
  __device__ __forceinline__ Ends(int64_t i, int64_t D_) : D(D_) {
    head = static_cast<int>(min(-i & 7, D));
    full = static_cast<int>((D - head) / 8);
  }
  // One piece less where the last one's second load would pass the end of the array of
  // n values that is read from value i on.
  __device__ __forceinline__ void within(int64_t i, int64_t n) {
    const int64_t at = i + head + 8 * (static_cast<int64_t>(full) - 1);
    if (full > 0 && (at & 7) != 0 && (at >> 3) * 8 + 16 > n) --full;
  }
  // The value at an end that this lane takes, or -1.
  __device__ __forceinline__ int64_t value(int lane) const {
    const int64_t e = lane < 8 ? lane : head + 8 * static_cast<int64_t>(full) + lane - 8;
    return (lane < 8 ? lane < head : e < D) ? e : -1;
  }
};
constexpr int kOddBatch = 4;

constexpr int kBatch = 8;  // choices whose rows are on their way at once

// This thread's token, and its pieces: the first and the step.
struct Along {
  int64_t t;
  int c, step;
};
template <int kLanes>
constexpr int kBlock = kLanes > kRowThreads ? kLanes : kRowThreads;
template <int kLanes>
__device__ __forceinline__ Along along(int parts) {
  const uint32_t part = blockIdx.x % parts, group = blockIdx.x / parts;
  return Along{static_cast<int64_t>(group) * (kBlock<kLanes> / kLanes) + threadIdx.x / kLanes,
               static_cast<int>(part * kLanes + threadIdx.x % kLanes), parts * kLanes};
}

// Writes the token's row to kBatch rows of out (-1: none).
template <bool kOdd>
__device__ __forceinline__ void spread_row(const ChoiceRows& a, const Along& p, const uint16_t* x, int64_t x_stride,
                                           uint16_t* out, const int32_t (&s)[kBatch]) {
  const int64_t D = a.D, from = p.t * x_stride;
  if constexpr (kOdd) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (s[j] < 0) continue;
      const int64_t i = s[j] * D;
      Ends ends(i, D);
      ends.within(from, (a.T - 1) * x_stride + D);
      const int64_t e = p.c < 32 ? ends.value(p.c) : -1;
      if (e >= 0) out[i + e] = x[from + e];
#pragma unroll 2
      for (int c = p.c; c < ends.full; c += p.step) {
        const int64_t at = ends.head + 8 * static_cast<int64_t>(c);
        Odd8 v;
        v.load(x, from + at);
        *reinterpret_cast<uint4*>(out + i + at) = v.get(from + at);
      }
    }
  } else {
    const int64_t C = D / 8;
    for (int64_t c = p.c; c < C; c += p.step) {
      const uint4 v = reinterpret_cast<const uint4*>(x + from)[c];
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (s[j] >= 0) reinterpret_cast<uint4*>(out + s[j] * D)[c] = v;
    }
  }
}

template <bool kOdd, int kLanes>
__global__ void __launch_bounds__(kRowThreads) spread_kernel(const ChoiceRows a, const uint16_t* __restrict__ x,
                                                             int64_t x_stride, uint16_t* __restrict__ out, int parts) {
  const Along p = along<kLanes>(parts);
  cl::griddep_wait();
  cl::griddep_launch_dependents();
  if (p.t >= a.T) return;
  const int32_t* slots = a.slots + p.t * a.k;
  for (int j0 = 0; j0 < a.k; j0 += kBatch) {
    int32_t s[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      s[j] = slots[min(j0 + j, a.k - 1)];
      if (j0 + j >= a.k || s[j] >= a.R) s[j] = -1;
    }
    spread_row<kOdd>(a, p, x, x_stride, out, s);
  }
}

__device__ __forceinline__ float eight_sums(const float (&v)[8]);

// Few choices: a token's blocks find its places themselves, each the number of
// choices that come before by (expert, choice), and one more block counts the
// experts' (a launch less: 64 tokens of 8 choices of 5120 2.9 us, with one 5.2; 256
// tokens 8.0, and 257 in two launches 9.6).
constexpr int kFewChoices = 2048;

template <bool kOdd>
__global__ void __launch_bounds__(kRowThreads) sort_few_kernel(const ChoiceRows a, const int32_t* __restrict__ ids,
                                                               int E, const uint16_t* __restrict__ x, int64_t x_stride,
                                                               uint16_t* __restrict__ out, int32_t* slots,
                                                               int32_t* __restrict__ offsets, int32_t* bad, int parts) {
  __shared__ float part[2][kRowThreads / 32][kBatch];
  __shared__ int count[kMaxGroups + 1];
  const int n = static_cast<int>(a.T) * a.k, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool counts = blockIdx.x == gridDim.x - 1;
  if (counts) {
    for (int e = threadIdx.x; e <= E; e += kRowThreads) count[e] = 0;
    __syncthreads();
  }
  cl::griddep_wait();
  cl::griddep_launch_dependents();
  auto group_of = [&](int i) {  // ids outside [0, E) come last
    const int id = ids[i];
    return id < 0 || id >= E ? E : id;
  };
  if (counts) {
    for (int i = threadIdx.x; i < n; i += kRowThreads) atomicAdd(&count[group_of(i)], 1);
    __syncthreads();
    if (warp == 0) {
      int before = 0;
      for (int e0 = 0; e0 <= E; e0 += 32) {
        const int e = e0 + lane, c = e <= E ? count[e] : 0;
        int sum = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(kAll, sum, o);
          if (lane >= o) sum += v;
        }
        if (e <= E) offsets[e] = before + sum - c;
        before += __shfl_sync(kAll, sum, 31);
      }
      if (lane == 0 && bad != nullptr && count[E] > 0) atomicAdd(bad, count[E]);
    }
    return;
  }
  const Along p = along<kRowThreads>(parts);
  const int own = static_cast<int>(p.t) * a.k;
  for (int j0 = 0; j0 < a.k; j0 += kBatch) {
    // the (expert, choice) pairs as numbers
    int key[kBatch], before[kBatch] = {};
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = own + min(j0 + j, a.k - 1);
      key[j] = group_of(i) * kFewChoices + i;
    }
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kRowThreads) {
      const int other = group_of(i) * kFewChoices + i;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) before[j] += other < key[j];
    }
    float f[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) f[j] = static_cast<float>(before[j]);
    const float sum = eight_sums(f);  // (at most 2048: exact)
    float(&sums)[kRowThreads / 32][kBatch] = part[(j0 / kBatch) & 1];
    if ((lane & 3) == 0) sums[warp][lane >> 2] = sum;
    __syncthreads();
    int32_t s[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      s[j] = static_cast<int32_t>((sums[0][j] + sums[1][j]) + (sums[2][j] + sums[3][j]));
      if (key[j] >= E * kFewChoices) s[j] = -1;
      if (p.c == j && j0 + j < a.k) slots[own + j0 + j] = s[j];
      if (j0 + j >= a.k) s[j] = -1;
    }
    if (out != nullptr) spread_row<kOdd>(a, p, x, x_stride, out, s);
  }
}

template <bool kOdd, int kLanes>
__global__ void __launch_bounds__(kRowThreads) combine_kernel(const ChoiceRows a, const uint16_t* __restrict__ y,
                                                              const uint16_t* residual, uint16_t* out, int parts) {
  const Along p = along<kLanes>(parts);
  cl::griddep_wait();
  cl::griddep_launch_dependents();
  if (p.t >= a.T) return;
  const int64_t D = a.D, at = p.t * a.k, row = p.t * D;
  int32_t s[kBatch];
  float w[kBatch];
  auto choices = [&](int j0) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      s[j] = a.slots[at + min(j0 + j, a.k - 1)];
      w[j] = 1.0f;
    }
    if (a.weights != nullptr) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) w[j] = a.weights[at + min(j0 + j, a.k - 1)];
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (j0 + j >= a.k || s[j] >= a.R) s[j] = -1;
  };
  float acc[8];
  auto add = [&](int j, const uint4& v) {
    float f[8];
    widen(v, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = fmaf(w[j], f[i], acc[i]);
  };
  choices(0);
  if constexpr (kOdd) {
    Ends ends(row, D);
    int full = ends.full;
    for (int j0 = 0; j0 < a.k; j0 += kBatch) {
      if (a.k > kBatch) choices(j0);
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        Ends of(row, D);
        of.within(max(s[j], 0) * D, a.R * D);
        full = min(full, of.full);
      }
    }
    ends.full = full;
    const int64_t e = p.c < 32 ? ends.value(p.c) : -1;
    if (e >= 0) {
      float sum = residual != nullptr ? bf16_bits_to_float(residual[row + e]) : 0.0f;
      for (int j0 = 0; j0 < a.k; j0 += kBatch) {
        if (a.k > kBatch) choices(j0);
        uint16_t v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) v[j] = y[max(s[j], 0) * D + e];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (s[j] >= 0) sum = fmaf(w[j], bf16_bits_to_float(v[j]), sum);
      }
      out[row + e] = float_to_bf16_bits_rn(sum);
    }
#pragma unroll 1
    for (int c = p.c; c < full; c += p.step) {
      const int64_t i = ends.head + 8 * static_cast<int64_t>(c);
      uint4 first = make_uint4(0, 0, 0, 0);
      if (residual != nullptr) first = *reinterpret_cast<const uint4*>(residual + row + i);
      widen(first, acc);
      for (int j0 = 0; j0 < a.k; j0 += kBatch) {
        if (a.k > kBatch) choices(j0);
#pragma unroll
        for (int l = 0; l < kBatch; l += kOddBatch) {
          Odd8 v[kOddBatch];
#pragma unroll
          for (int j = 0; j < kOddBatch; ++j) v[j].load(y, max(s[l + j], 0) * D + i);
#pragma unroll
          for (int j = 0; j < kOddBatch; ++j)
            if (s[l + j] >= 0) add(l + j, v[j].get(s[l + j] * D + i));
        }
      }
      *reinterpret_cast<uint4*>(out + row + i) = narrow(acc);
    }
  } else {
    const int64_t C = D / 8;
#pragma unroll 1
    for (int64_t c = p.c; c < C; c += p.step) {
      uint4 first = make_uint4(0, 0, 0, 0);
      if (residual != nullptr) first = reinterpret_cast<const uint4*>(residual + row)[c];
      widen(first, acc);
      for (int j0 = 0; j0 < a.k; j0 += kBatch) {
        if (a.k > kBatch) choices(j0);
        uint4 v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          v[j] = s[j] >= 0 ? reinterpret_cast<const uint4*>(y + s[j] * D)[c] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (s[j] >= 0) add(j, v[j]);
      }
      reinterpret_cast<uint4*>(out + row)[c] = narrow(acc);
    }
  }
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

// dy's rows are written as y's are read; the products with dout are summed over a
// token's threads in a fixed order.
template <bool kOdd, int kLanes>
__global__ void __launch_bounds__(kBlock<kLanes>, kOdd ? 1 : 768 / kBlock<kLanes>)
    combine_grad_kernel(const ChoiceRows a, const uint16_t* __restrict__ dout, const uint16_t* __restrict__ y,
                        uint16_t* dy, float* __restrict__ dweights) {
  constexpr int kGroupWarps = kLanes / 32;
  __shared__ float part[kBlock<kLanes> / 32][kBatch];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Along p = along<kLanes>(1);
  cl::griddep_wait();
  cl::griddep_launch_dependents();
  const bool real = p.t < a.T;  // (the block's barriers want every thread)
  const int64_t t = real ? p.t : a.T - 1, at = t * a.k, D = a.D, C = real ? D / 8 : 0;
  for (int j0 = 0; j0 < a.k; j0 += kBatch) {
    int32_t s[kBatch];
    float w[kBatch], dot[kBatch] = {};
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      s[j] = a.slots[at + min(j0 + j, a.k - 1)];
      w[j] = a.weights[at + min(j0 + j, a.k - 1)];
      if (j0 + j >= a.k || s[j] >= a.R) s[j] = -1;
    }
    auto term = [&](int j, const uint4& yv, const float (&g)[8]) {
      float f[8];
      widen(yv, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) dot[j] = fmaf(g[i], f[i], dot[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = w[j] * g[i];
      return narrow(f);
    };
    if constexpr (kOdd) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (s[j] < 0 || !real) continue;
        const int64_t i = s[j] * D;  // y's and dy's pieces lie alike
        Ends ends(i, D);
        ends.within(t * D, a.T * D);
        const int64_t e = p.c < 32 ? ends.value(p.c) : -1;
        if (e >= 0) {
          const float g = bf16_bits_to_float(dout[t * D + e]);
          dot[j] = fmaf(g, bf16_bits_to_float(y[i + e]), dot[j]);
          dy[i + e] = float_to_bf16_bits_rn(w[j] * g);
        }
#pragma unroll 2
        for (int c = p.c; c < ends.full; c += kLanes) {
          const int64_t l = ends.head + 8 * static_cast<int64_t>(c);
          Odd8 v;
          v.load(dout, t * D + l);
          const uint4 yv = *reinterpret_cast<const uint4*>(y + i + l);
          float g[8];
          widen(v.get(t * D + l), g);
          *reinterpret_cast<uint4*>(dy + i + l) = term(j, yv, g);
        }
      }
    } else {
#pragma unroll 1
      for (int64_t c = p.c; c < C; c += kLanes) {
        float g[8];
        uint4 v[kBatch];
        widen(reinterpret_cast<const uint4*>(dout + t * D)[c], g);
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          v[j] = s[j] >= 0 ? reinterpret_cast<const uint4*>(y + s[j] * D)[c] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (s[j] >= 0) reinterpret_cast<uint4*>(dy + s[j] * D)[c] = term(j, v[j], g);
      }
    }
    const float sum = eight_sums(dot);
    if constexpr (kGroupWarps == 1) {
      if (real && (lane & 3) == 0 && j0 + (lane >> 2) < a.k) dweights[at + j0 + (lane >> 2)] = sum;
    } else {
      const int own = threadIdx.x % kLanes;
      if ((lane & 3) == 0) part[warp][lane >> 2] = sum;
      __syncthreads();
      if (real && own < kBatch && j0 + own < a.k) {
        float d = 0.0f;
#pragma unroll
        for (int i = 0; i < kGroupWarps; ++i) d += part[threadIdx.x / kLanes * kGroupWarps + i][own];
        dweights[at + j0 + own] = d;
      }
      __syncthreads();
    }
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

// How the rows go: in whole 16 bytes or not, threads a token (a warp for short
// rows), parts a token is cut into, blocks.
struct RowPlan {
  bool odd;
  int lanes, parts, threads;
  int64_t grid;
};
RowPlan row_plan(int64_t T, int64_t D, int64_t stride, int lanes, int64_t cut_below) {
  RowPlan p;
  p.odd = D % 8 != 0 || stride % 8 != 0;
  const int64_t C = std::max<int64_t>(D / 8, 1);
  p.lanes = C <= 64 ? 32 : lanes;
  p.threads = p.lanes < kRowThreads ? kRowThreads : p.lanes;
  const int64_t groups = (T * p.lanes - 1) / p.threads + 1;
  p.parts = groups < cut_below ? static_cast<int>((C - 1) / p.lanes + 1) : 1;
  if (groups * p.parts > kMaxDim) p.parts = 1;
  p.grid = groups * p.parts;
  return p;
}

}  // namespace

#define WQ_ROW_KERNEL(kern, p)                                                       \
  ((p).lanes == 32 ? ((p).odd ? kern<true, 32> : kern<false, 32>)                    \
                   : ((p).odd ? kern<true, kRowThreads> : kern<false, kRowThreads>))

cudaError_t launch_moe_sort(const Ctx& c, const ChoiceRows& a, const int32_t* ids, int64_t E, const uint16_t* x,
                            int64_t x_stride, uint16_t* out, int32_t* offsets, int32_t* slots, int32_t* bad) {
  const int64_t n = a.T * a.k;
  if (n > 0 && n <= kFewChoices) {
    const bool odd = a.D % 8 != 0 || x_stride % 8 != 0;
    const int64_t parts = std::max<int64_t>(1, (a.D / 8 - 1) / kRowThreads + 1);
    return launch_early(c, a.T * parts + 1, kRowThreads, 0, odd ? sort_few_kernel<true> : sort_few_kernel<false>, a, ids,
                        static_cast<int>(E), x, x_stride, out, slots, offsets, bad, static_cast<int>(parts));
  }
  GroupArgs g{};
  g.ids = ids;
  g.n = n;
  g.E = static_cast<int>(E);
  g.slots = slots;
  g.offsets = offsets;
  g.bad = bad;
  const cudaError_t e = launch_group(c, g);
  if (e != cudaSuccess || out == nullptr || n == 0) return e;
  // (a thread a piece: its k writes need no loop, 5 us of 122 for 8192 tokens of 8 choices of 5120)
  const bool wide = a.D % 8 == 0 && x_stride % 8 == 0;
  const RowPlan p = row_plan(a.T, a.D, x_stride, kRowThreads, wide ? kMaxDim : 4 * c.sm_count);
  return launch_early(c, p.grid, p.threads, 0, WQ_ROW_KERNEL(spread_kernel, p), a, x, x_stride, out, p.parts);
}

cudaError_t launch_moe_combine(const Ctx& c, const ChoiceRows& a, const uint16_t* y, const uint16_t* residual,
                               uint16_t* out) {
  const RowPlan p = row_plan(a.T, a.D, a.D, kRowThreads, 4 * c.sm_count);
  return launch_early(c, p.grid, p.threads, 0, WQ_ROW_KERNEL(combine_kernel, p), a, y, residual, out, p.parts);
}

cudaError_t launch_moe_combine_grad(const Ctx& c, const ChoiceRows& a, const uint16_t* dout, const uint16_t* y,
                                    uint16_t* dy, float* dweights) {
  // 128 threads a token: 4099 tokens of 6 choices of 2048 31 us (64: 31, 256: 36); few tokens of long rows 512 (64
  // tokens of 8 choices of 5120 5.8 us, with 256 6.7, with 128 8.8)
  if (a.T < 2 * c.sm_count && a.D > 2048) {
    const RowPlan p = row_plan(a.T, a.D, a.D, 512, 0);
    return launch_early(c, p.grid, p.threads, 0, p.odd ? combine_grad_kernel<true, 512> : combine_grad_kernel<false, 512>,
                        a, dout, y, dy, dweights);
  }
  const RowPlan p = row_plan(a.T, a.D, a.D, kRowThreads, 0);
  return launch_early(c, p.grid, p.threads, 0, WQ_ROW_KERNEL(combine_grad_kernel, p), a, dout, y, dy, dweights);
}

}  // namespace wq
