// Log probabilities of given tokens, entropy and the best alternatives, from
// logits.
//
// Mathematics, with c = log2(e) / temperature and any reference m (a maximum
// seen so far): u_i = (x_i - m) c (the difference of near logits is exact),
// l = sum 2^u_i, t = sum 2^u_i u_i. Raising m by d / c turns (l, t) into
// 2^-d (l, t - d l), so all comes from one pass, and with the final sums
//   logprob = ln 2 (u_id - log2 l),  entropy = ln 2 (log2 l - t / l).
// The t of a row that is nearly certain is small beside no other number, so the
// entropy does not lose digits.
//
// Bound: the read of the logits, and right behind it the issue of about seven
// instructions per logit (at the copy rate an SM gets 12 bf16 logits a clock and
// issues 128 lanes). So: everything in one pass; pairs of float32 operations
// where there are such; the rank by packed compares; no running maximum but a
// test per 8 logits (4 for float32) against the reference and against the
// top_k'th best so far. Measured: 64 rows of 8 M bf16 logits 6.8 TB/s without ids
// and best, 6.6 with ids, 5.8 with the best 5; 2049 rows of 248320, 1.02 GB, 151
// us (6.7 TB/s), 176, 218 and with the best 20 267: a row's ends, the barriers of
// its notes and the notes themselves, about 10 us a row at three rows an SM, are
// what the other two blocks do not hide. 1 row with the best 20: 12 us, of which
// the join is 4; 96 float32 rows of 100003 with the best 8: 26 us.
//  - All rows are one line of units of 4 KB (a 16-byte vector per thread), cut
//    into equal shares, one per block, several blocks per SM; a second kernel
//    joins rows that were cut, in the order of their parts: bits do not depend on
//    timing, and one row keeps many SMs busy.
//  - A thread copies its own vectors to shared memory, two rounds of four units
//    ahead (cp.async), and reads them back itself: no barrier.
//  - The best top_k are kept as 64-bit keys (logit, then id) in shared memory: the
//    first round's bound is the top_k'th largest of 32 groups' maxima; later
//    logits are noted only above the bound, which is raised after 2, 4, 8 ..
//    rounds: a few notes per row in the usual order. Where they do not fit
//    (ascending rows), the piece's best are found again with a bound for every
//    round, by bisection over the keys. -inf is not noted: where too few logits
//    are above it (a grammar's mask), the first of them follow at the end.
//  - Short rows take a kernel of their own, a warp per row.
#include "wq_cluster.cuh"
#include "wq_device.cuh"
#include "wq_internal.h"

#include <math_constants.h>

namespace wq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlocksPerSm = 3;
constexpr int kRound = 4;      // units a block takes at a time
constexpr int kStages = 3;     // rounds in shared memory
constexpr int kRowCost = 4;    // what beginning and ending a row costs, in units
constexpr int kLeast = 2;      // units of a share at least
constexpr int kNotes = 512;    // keys noted at a time
constexpr int kMaxShares = 160 * kBlocksPerSm;
constexpr float kSlack = 4.0f;  // the reference is raised when a logit passes it by more (in powers of two)

// A row's sums, or those of a part of it.
struct Sums {
  float m, l, t;  // m = -inf: nothing yet
  int before;     // tokens that come before the given one
};
struct Part {
  Sums s;
  uint64_t keys[kMaxTopK];  // best first; 0: none
};

struct Args {
  LogprobArgs a;
  float c;         // log2(e) / temperature
  int units;       // of a row
  int64_t share;   // places of a share
  int64_t shares;
  Part* parts;     // two per share
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float x, float y) {
  float z;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}

// A logit's place in the order as an unsigned number: NaN above all, -0.0 as 0.0.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return x != x ? 0xFFFFFFFFu : ((u >> 31) != 0 ? ~u : u | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t order) {
  if (order == 0xFFFFFFFFu) return CUDART_NAN_F;
  return __uint_as_float((order >> 31) != 0 ? order & 0x7FFFFFFFu : ~order);
}
__device__ __forceinline__ uint64_t key_of(float x, uint32_t id) {
  return static_cast<uint64_t>(order_of(x)) << 32 | (0xFFFFFFFFu - id);
}
__device__ __forceinline__ uint32_t id_of(uint64_t key) { return 0xFFFFFFFFu - static_cast<uint32_t>(key); }

// (A difference beyond 200 leaves no weight, as 200 does; it may be infinite, as from
// the type's lowest value, and t - d l would be so, too.)
__device__ __forceinline__ void raise(Sums& s, float m, float c) {
  const float d = s.m == -CUDART_INF_F || s.m == m ? 0.0f : fminf((m - s.m) * c, 200.0f);
  const float f = s.m == -CUDART_INF_F ? 0.0f : exp2_fast(-d);
  s.t = f * (s.t - d * s.l);
  s.l = f * s.l;
  s.m = m;
}
// The sums of both.
__device__ __forceinline__ void join(Sums& s, Sums o, float c) {
  const float m = fmaxf(s.m, o.m);
  if (m != -CUDART_INF_F) {
    raise(s, m, c);
    raise(o, m, c);
  }
  s.l += o.l;
  s.t += o.t;
  s.before += o.before;
}

// The given token's logit.
__device__ __forceinline__ float given_logit(const LogprobArgs& a, int64_t row, int32_t id) {
  if (id < 0 || id >= a.V) return 0.0f;
  return a.type == WQ_LOGITS_BF16 ? bf16_bits_to_float(static_cast<const uint16_t*>(a.logits)[row * a.ld + id])
                                  : static_cast<const float*>(a.logits)[row * a.ld + id];
}

// The number before x, which logits that are not below x are not at or below
// (NaN, unordered with all, where there is none).
template <bool kBf16>
__device__ __forceinline__ float next_below(float x) {
  constexpr uint32_t kOne = kBf16 ? 0x10000u : 1u;
  if (x == -CUDART_INF_F) return CUDART_NAN_F;
  return __uint_as_float(x > 0.0f ? __float_as_uint(x) - kOne : (x == 0.0f ? 0x80000000u + kOne : __float_as_uint(x) + kOne));
}

// A row's results from its sums and keys (lanes 0 .. top_k - 1 and 0).
__device__ __forceinline__ void put(const Args& g, int64_t row, int i, const Sums& s, uint64_t key, bool given, float xt) {
  const LogprobArgs& a = g.a;
  const bool none = s.m == -CUDART_INF_F && s.l == 0.0f;
  const float log_l = log2f(s.l), ref = s.m == -CUDART_INF_F ? 0.0f : s.m;
  const auto lp = [&](float x) {
    const float u = (x - ref) * g.c;
    if (none) return -CUDART_INF_F;
    // (in powers of two the type's lowest value overflows, in nats it need not)
    return u == -CUDART_INF_F ? (x - ref) / a.temperature - 0.6931471805599453f * log_l : 0.6931471805599453f * (u - log_l);
  };
  if (i < a.top_k) {
    a.top_ids[row * a.top_k + i] = static_cast<int32_t>(id_of(key));
    a.top_logprobs[row * a.top_k + i] = lp(value_of(static_cast<uint32_t>(key >> 32)));
  }
  if (i == 0) {
    if (a.ids != nullptr) {
      a.logprob[row] = given ? lp(xt) : -CUDART_INF_F;
      a.rank[row] = given ? 1 + s.before : 0;
      if (!given && a.bad != nullptr) atomicAdd(a.bad, 1);
    }
    if (a.entropy != nullptr) a.entropy[row] = none ? 0.0f : 0.6931471805599453f * (log_l - s.t / s.l);
  }
}

// Pairs of float32 operations.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  return static_cast<uint64_t>(__float_as_uint(y)) << 32 | __float_as_uint(x);
}
__device__ __forceinline__ float low_of(uint64_t p) { return __uint_as_float(static_cast<uint32_t>(p)); }
__device__ __forceinline__ float high_of(uint64_t p) { return __uint_as_float(static_cast<uint32_t>(p >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// A 16-byte vector of logits: 8 bf16 or 4 float32.
template <bool kBf16>
struct Vec {
  static constexpr int kN = kBf16 ? 8 : 4;
  uint32_t w[4];
  __device__ __forceinline__ float at(int i) const {
    if constexpr (kBf16) return __uint_as_float((i & 1) ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
    else return __uint_as_float(w[i]);
  }
  __device__ __forceinline__ static Vec from(const uint8_t* p) {
    const uint4 y = *reinterpret_cast<const uint4*>(p);
    return Vec{{y.x, y.y, y.z, y.w}};
  }
  // The larger of each pair of words' logits, NaN before all.
  __device__ __forceinline__ static uint32_t max_word(uint32_t x, uint32_t y) {
    uint32_t z;
    if constexpr (kBf16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(z) : "r"(x), "r"(y));
    else z = __float_as_uint(max_nan(__uint_as_float(x), __uint_as_float(y)));
    return z;
  }
  __device__ __forceinline__ uint32_t max_word() const {
    return max_word(max_word(w[0], w[1]), max_word(w[2], w[3]));
  }
  __device__ __forceinline__ static float top_of(uint32_t x) {
    if constexpr (kBf16) return max_nan(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
    else return __uint_as_float(x);
  }
  // The largest, NaN if there is one.
  __device__ __forceinline__ float top() const { return top_of(max_word()); }
  // Adds how many logits are above `than` (or NaN): for bf16 a sum of masks,
  // 0xFFFF for each half that is above, that count_of() takes apart.
  __device__ __forceinline__ void add_above(float than, uint32_t& sum) const {
    if constexpr (kBf16) {
      const uint32_t than2 = __byte_perm(__float_as_uint(than), 0u, 0x3232);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sum += __hgtu2_mask(*reinterpret_cast<const __nv_bfloat162*>(&w[i]),
                            *reinterpret_cast<const __nv_bfloat162*>(&than2));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) sum += !(at(i) <= than);
    }
  }
  __device__ __forceinline__ static int count_of(uint32_t sum) {
    if constexpr (kBf16) {  // L low and H high ones, below 2^16: sum = (L - H) 2^16 - L
      const uint32_t low = -sum & 0xFFFFu, high = (low - ((sum + low) >> 16)) & 0xFFFFu;
      return static_cast<int>(low + high);
    } else {
      return static_cast<int>(sum);
    }
  }
};

// The vectors of a row: vector v has logits v kN - head .. v kN - head + kN - 1.
template <bool kBf16>
struct Row {
  const uint8_t* base;  // 16-byte aligned
  int nvec, head;
  __device__ void set(const LogprobArgs& a, int64_t row) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.logits) + row * a.ld * (kBf16 ? 2 : 4);
    base = reinterpret_cast<const uint8_t*>(p & ~uintptr_t{15});
    head = static_cast<int>(p & 15) / (kBf16 ? 2 : 4);
    nvec = static_cast<int>((a.V + head + Vec<kBf16>::kN - 1) / Vec<kBf16>::kN);
  }
  // The id of logit i of vector v (before the row: above any V).
  __device__ __forceinline__ uint32_t id(int v, int i) const {
    return static_cast<uint32_t>(v) * Vec<kBf16>::kN + i - head;
  }
};

struct Shared {
  uint8_t ring[kStages][kRound][kThreads * 16];
  uint64_t notes[kNotes];
  uint64_t best[kMaxTopK];
  uint32_t groups[kWarps][32];
  Sums sums[kWarps];
  int noted, count;
};

// Sorts the n <= kNotes noted keys' best top_k to the front (by counting, keys
// are distinct): 8 to 1 threads a key. All threads; n is the same for all.
// Returns how many are kept.
__device__ __forceinline__ int keep_best(Shared& sh, int n, int top_k) {
  n = n < kNotes ? n : kNotes;
  const int shift = n <= 32 ? 3 : (n <= 64 ? 2 : (n <= 128 ? 1 : 0)), per = 1 << shift;
  for (int i0 = 0; i0 < n; i0 += kThreads >> shift) {
    const int i = i0 + (static_cast<int>(threadIdx.x) >> shift);
    const uint64_t mine = i < n ? sh.notes[i] : 0;
    int rank = 0;
    for (int j = threadIdx.x & (per - 1); j < n; j += per) rank += sh.notes[j] > mine;
    for (int o = 1; o < per; o <<= 1) rank += __shfl_xor_sync(0xFFFFFFFFu, rank, o);
    if (i < n && rank < top_k) sh.best[rank] = mine;
  }
  __syncthreads();
  const int kept = n < top_k ? n : top_k;
  if (threadIdx.x < kept) sh.notes[threadIdx.x] = sh.best[threadIdx.x];
  if (threadIdx.x == 0) sh.noted = kept;
  __syncthreads();
  return kept;
}

// A vector in shared memory with logits id, id + 1 .., which may be its row's
// first or last or none of it: what lies outside becomes -inf. Returns how many
// of its logits come before the given token.
template <bool kBf16>
__device__ __noinline__ int look_closer(uint8_t* x, uint32_t id, uint32_t V, uint64_t key_t) {
  int before = 0;
  for (int i = 0; i < Vec<kBf16>::kN; ++i) {
    if constexpr (kBf16) {
      uint16_t& y = reinterpret_cast<uint16_t*>(x)[i];
      if (id + i < V) before += key_of(bf16_bits_to_float(y), id + i) > key_t;
      else y = 0xFF80u;
    } else {
      float& y = reinterpret_cast<float*>(x)[i];
      if (id + i < V) before += key_of(y, id + i) > key_t;
      else y = -CUDART_INF_F;
    }
  }
  return before;
}

// A vector's terms with a difference for each exponent: l and t.
template <bool kBf16>
__device__ __noinline__ float2 far_sums(const uint8_t* x, float m, float c) {
  float2 s = make_float2(0.0f, 0.0f);
  for (int i = 0; i < Vec<kBf16>::kN; ++i) {
    float y;
    if constexpr (kBf16) y = bf16_bits_to_float(reinterpret_cast<const uint16_t*>(x)[i]);
    else y = reinterpret_cast<const float*>(x)[i];
    const float d = max_nan((y - m) * c, -200.0f), e = exp2_fast(d);
    s.x += e;
    s.y = fmaf(e, d, s.y);
  }
  return s;
}

// Notes a logit of the row.
__device__ __noinline__ void note(Shared& sh, float x, uint32_t id, uint32_t V) {
  if (id >= V) return;
  const int to = atomicAdd(&sh.noted, 1);
  if (to < kNotes) sh.notes[to] = key_of(x, id);
}

// The best top_k of units [unit, end) of a row, in whatever order they come:
// sorted in sh.notes, sh.noted of them. Reads the logits again.
template <bool kBf16>
__device__ __noinline__ void best_of(Shared& sh, const LogprobArgs& a, int64_t row, int unit, int end) {
  constexpr int kN = Vec<kBf16>::kN;
  const int tid = threadIdx.x;
  const void* x = static_cast<const uint8_t*>(a.logits) + row * a.ld * (kBf16 ? 2 : 4);
  Row<kBf16> r;
  r.set(a, row);
  // logits unit .. end - 1 hold, in steps of what a block reads at once
  const int64_t first = static_cast<int64_t>(unit) * kThreads * kN - r.head, last = static_cast<int64_t>(end) * kThreads * kN - r.head;
  const int64_t from = first < 0 ? 0 : first, to = last < a.V ? last : a.V;
  constexpr int kPer = 8;
  __syncthreads();
  if (tid == 0) sh.noted = 0;
  __syncthreads();
  for (int64_t i0 = from; i0 < to; i0 += kThreads * kPer) {
    const int kept = sh.noted;
    uint64_t key[kPer];
    const uint64_t bound = kept == a.top_k ? sh.notes[kept - 1] : 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int64_t i = i0 + j * kThreads + tid;
      float y = 0.0f;
      if (i < to) {
        if constexpr (kBf16) y = bf16_bits_to_float(static_cast<const uint16_t*>(x)[i]);
        else y = static_cast<const float*>(x)[i];
      }
      key[j] = i < to ? key_of(y, static_cast<uint32_t>(i)) : 0;
      if (key[j] <= bound) key[j] = 0;  // none, or not among the best
    }
    // all of them if they fit; else a bound that at least top_k of them reach:
    // the top_k'th largest found bit by bit, or an earlier one that few enough reach
    uint64_t least = 1;
    for (int bit = 64; bit >= 0; --bit) {
      const uint64_t trial = bit == 64 ? 1 : ((bit == 63 ? 0 : least) | uint64_t{1} << bit);
      __syncthreads();
      if (tid == 0) sh.count = 0;
      __syncthreads();
      int c = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) c += key[j] >= trial;
      c = __reduce_add_sync(0xFFFFFFFFu, c);
      if ((tid & 31) == 0) atomicAdd(&sh.count, c);
      __syncthreads();
      const int n = sh.count;
      if (bit == 64) {
        if (n <= kNotes - kMaxTopK) break;
        continue;
      }
      if (bit == 63) least = 0;
      if (n < a.top_k) continue;
      least = trial;
      if (n <= kNotes - kMaxTopK) break;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (key[j] != 0 && key[j] >= least) {
        const int n = atomicAdd(&sh.noted, 1);
        if (n < kNotes) sh.notes[n] = key[j];
      }
    __syncthreads();
    const int n = sh.noted;
    __syncthreads();
    if (n > kept) keep_best(sh, n, a.top_k);
  }
}

// Adds the first -inf of units [unit, end) of a row to its kept keys, up to
// top_k. One warp; returns how many there are then.
template <bool kBf16>
__device__ __noinline__ int fill(Shared& sh, const LogprobArgs& a, int64_t row, int unit, int end, int kept) {
  const int lane = threadIdx.x & 31;
  Row<kBf16> r;
  r.set(a, row);
  const int64_t first = static_cast<int64_t>(unit) * kThreads * Vec<kBf16>::kN - r.head;
  const int64_t last = static_cast<int64_t>(end) * kThreads * Vec<kBf16>::kN - r.head;
  const int64_t from = first < 0 ? 0 : first, to = last < a.V ? last : a.V;
  for (int64_t i0 = from; i0 < to && i0 < from + 2 * kMaxTopK && kept < a.top_k; i0 += 32) {
    const int64_t i = i0 + lane;
    const bool none = i < to && given_logit(a, row, static_cast<int32_t>(i)) == -CUDART_INF_F;
    const unsigned who = __ballot_sync(0xFFFFFFFFu, none);
    const int at = kept + __popc(who & ((1u << lane) - 1u));
    if (none && at < a.top_k) sh.notes[at] = key_of(-CUDART_INF_F, static_cast<uint32_t>(i));
    kept += __popc(who);
  }
  __syncwarp();
  return kept < a.top_k ? kept : a.top_k;
}

template <bool kBf16, bool kIds>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) logprobs_kernel(const Args g) {
  constexpr int kN = Vec<kBf16>::kN, kElem = kBf16 ? 2 : 4;
  extern __shared__ __align__(128) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  const LogprobArgs& a = g.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int places = g.units + kRowCost;
  const uint32_t V = static_cast<uint32_t>(a.V);
  const float slack = kSlack / g.c;
  cl::griddep_wait();
  cl::griddep_launch_dependents();  // the join may start; it waits for this kernel's end

  // a piece: units [unit, end) of row, `left` places of the share from there on
  const int64_t total = a.T * places, first = g.share * blockIdx.x;
  if (first >= total) return;
  int left = static_cast<int>(first + g.share < total ? g.share : total - first);
  int row = static_cast<int>(first / places);
  int unit = static_cast<int>(first - static_cast<int64_t>(row) * places) - kRowCost;
  if (unit < 0) {
    left += unit;
    unit = 0;
  }
  if (left <= 0) return;
  Row<kBf16> r;
  r.set(a, row);

  // ---- the copies: rounds of the share's pieces, kStages - 1 ahead
  uint8_t* const mine = sh.ring[0][0] + tid * 16;
  const uint32_t mine_s = smem_u32(mine);
  constexpr int kUnitBytes = kThreads * 16, kStageBytes = kRound * kUnitBytes;
  Row<kBf16> lr = r;
  int l_row = row, l_left = left, l_unit = unit;
  const uint8_t* l_src = nullptr;  // of the next round, where it is known to be a whole one
  const auto copy = [&](const uint8_t* src, int stage, int j, int bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(mine_s + stage * kStageBytes +
                                                                                j * kUnitBytes),
                 "l"(src + j * kUnitBytes), "r"(bytes)
                 : "memory");
  };
  auto copy_round = [&](int stage) {
    if (l_left > 0) {
      const int end = g.units - l_unit < l_left ? g.units : l_unit + l_left;
      const int row_end = (lr.head + static_cast<int>(V & 7)) * kElem & 15;  // bytes of the last vector, 0: all
      const uint8_t* src = lr.base + (static_cast<int64_t>(l_unit) * kThreads + tid) * 16;
      if (l_unit + kRound <= end && (l_unit + kRound) * kThreads < lr.nvec) {
#pragma unroll
        for (int j = 0; j < kRound; ++j) copy(src, stage, j, 16);
      } else {
        for (int j = 0; j < kRound; ++j) {
          const int v = (l_unit + j) * kThreads + tid;
          if (l_unit + j < end && v < lr.nvec) copy(src, stage, j, v == lr.nvec - 1 && row_end != 0 ? row_end : 16);  // not past the row
        }
      }
      const int n = end - l_unit < kRound ? end - l_unit : kRound;
      l_left -= n;
      l_unit += n;
      if (l_unit == g.units) {
        l_left -= kRowCost;
        l_unit = 0;
        if (l_left > 0) lr.set(a, ++l_row);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) copy_round(i);
  int stage = 0;

  // the given token and its logit, and the next row's token
  const auto id_of_row = [&](int t) { return kIds && t < a.T ? a.ids[t] : -1; };
  int32_t id = id_of_row(row), id2 = id_of_row(row + 1);
  float xt = given_logit(a, row, id);
  while (true) {
    const int end = g.units - unit < left ? g.units : unit + left;
    const bool begins = unit == 0, whole = begins && end == g.units;
    const bool given = kIds && id >= 0 && id < a.V;
    const uint64_t key_t = given ? key_of(xt, static_cast<uint32_t>(id)) : ~uint64_t{0};
    const int v_id = given ? static_cast<int>((static_cast<uint32_t>(id) + r.head) / kN) : -1;
    const float low = next_below<kBf16>(xt);  // vectors before v_id count logits that are not below xt

    Sums s{-CUDART_INF_F, 0.0f, 0.0f, 0};
    float limit = -CUDART_INF_F, bound = -CUDART_INF_F;
    float gate = CUDART_NAN_F;  // a vector above it (always, for NaN) needs more than its terms
    // The terms are added up in pairs, relative to ref = m c rounded (one fma for
    // an exponent); flush() brings them to m. Where that rounding is no small
    // number (`far`), each exponent is a difference's.
    uint64_t l2 = 0, t2 = 0;
    float ref = 0.0f;
    bool far = false;
    const auto flush = [&]() {
      if (far) {
        l2 = t2 = 0;
        return;
      }
      const float l = low_of(l2) + high_of(l2), t = low_of(t2) + high_of(t2);
      const float off = s.m == -CUDART_INF_F ? 0.0f : fmaf(s.m, g.c, -ref), f = exp2_fast(-off);
      s.l += f * l;
      s.t += f * (t - off * l);
      l2 = t2 = 0;
    };
    bool closed = a.top_k == 0, lost = false;
    // the opening's bound does for the second round, too, unless most of its groups
    // have to be above it (top_k 32: 355 us with a raise after the first round, 1070
    // without; 5: 222 and 218)
    int raise_at = a.top_k > 24 ? 1 : 2;
    if (tid == 0) sh.noted = 0;
    // logits this far below the reference (-inf among them) have weight 0; they
    // count as this one, so that every term is finite
    uint32_t floor_word = 0;
    const auto set_floor = [&]() {
      const float f = (s.m == -CUDART_INF_F ? 0.0f : s.m) - 160.0f / g.c;
      floor_word = __float_as_uint(f);
      if constexpr (kBf16) {  // rounded down
        floor_word += (floor_word >> 31) != 0 ? 0xFFFFu : 0u;
        floor_word = __byte_perm(floor_word, 0u, 0x3232);
      }
    };
    set_floor();
    // whole rounds without a special vector that follow, for which also the copy
    // is a whole round's; the logit to compare theirs with
    int fast = 0;
    float than_fast = xt;
    uint32_t above = 0;

    for (int u = unit, rounds = 1; u < end; u += kRound, ++rounds) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      uint8_t* in = mine + stage * kStageBytes;
      const int v0 = u * kThreads + warp * 32, freed = stage == 0 ? kStages - 1 : stage - 1;  // read in the round before
      unsigned special = 0;
      bool plain = true;
      float than = than_fast;
      if (fast > 0) {
        --fast;
#pragma unroll
        for (int j = 0; j < kRound; ++j) copy(l_src, freed, j, 16);
        asm volatile("cp.async.commit_group;" ::: "memory");
        l_src += kStageBytes;
        l_unit += kRound;
        l_left -= kRound;
      } else {
        copy_round(freed);
        // the row's first and last vector where it is not all the row's, the given
        // token's, and what lies outside the piece: logit by logit, by their warp
        // the row's whole vectors: [head, full)
        const int head = r.head > 0, full = static_cast<int>((V + r.head) / kN);
        plain = v0 >= head && v0 + (kRound - 1) * kThreads + 32 <= full && u + kRound <= end &&
                (v_id < v0 || v_id >= v0 + (kRound - 1) * kThreads + 32) && xt == xt;
        than = v_id >= v0 ? low : xt;
        if (!plain) {
          for (int j = 0; j < kRound; ++j) {
            const int w0 = v0 + j * kThreads, v = w0 + lane;
            if (w0 >= head && w0 + 32 <= full && u + j < end && (v_id < w0 || v_id >= w0 + 32) && xt == xt) continue;
            special |= 1u << j;
            const uint32_t id0 = u + j < end && v < r.nvec ? r.id(v, 0) : 0xFFFFFF00u;  // none: above any V
            s.before += look_closer<kBf16>(in + j * kUnitBytes, id0, V, key_t);
          }
          if constexpr (kIds) {
            for (int j = 0; j < kRound; ++j)
              if ((special >> j & 1u) == 0)
                Vec<kBf16>::from(in + j * kUnitBytes).add_above(v_id >= v0 + j * kThreads ? low : xt, above);
          }
        }
        const int u2 = u + kRound, l_end = g.units - l_unit < l_left ? g.units : l_unit + l_left;
        const int whole = full / kThreads, l_whole = (lr.nvec - 1) / kThreads;
        fast = ((end < whole ? end : whole) - u2) / kRound;
        const int l_fast = l_left > 0 ? ((l_end < l_whole ? l_end : l_whole) - l_unit) / kRound : 0;
        fast = fast < l_fast ? fast : l_fast;
        than_fast = xt;
        if (v_id >= u2 * kThreads) {
          than_fast = low;
          const int to_id = (v_id / kThreads - u2) / kRound;
          fast = fast < to_id ? fast : to_id;
        }
        if (xt != xt) fast = 0;
        l_src = lr.base + (static_cast<int64_t>(l_unit) * kThreads + tid) * 16;
      }
      // far: always; before there is a reference, and for NaN: always
      const auto set_gate = [&]() {
        gate = far || limit == -CUDART_INF_F ? CUDART_NAN_F : (closed || limit < bound ? limit : bound);
      };
      if (rounds == 1) {
        // The opening: the largest logit of the block's round is everyone's first
        // reference, and the top_k'th largest of 32 groups' maxima the first bound
        // (top_k logits are not below it).
        float tops[kRound];
#pragma unroll
        for (int j = 0; j < kRound; ++j) tops[j] = Vec<kBf16>::from(in + j * kUnitBytes).top();
        uint32_t o = 0;
#pragma unroll
        for (int j = 0; j < kRound; ++j) o = max(o, order_of(tops[j]));
        sh.groups[warp][lane] = o;  // (a group: a lane of every warp, so that a short piece's logits are in all)
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWarps; ++i) o = max(o, sh.groups[i][lane]);
        const float top = value_of(__reduce_max_sync(0xFFFFFFFFu, o));
        if (top > -CUDART_INF_F) {  // not NaN
          s.m = top;
          limit = top + slack;
          ref = top * g.c;
          far = !(fabsf(ref) < 16777216.0f);
          set_floor();
        }
        if (!closed) {
          int rank = 0;
#pragma unroll 4
          for (int i = 0; i < 32; ++i) {
            const uint32_t y = __shfl_sync(0xFFFFFFFFu, o, i);
            rank += y > o || (y == o && i < lane);
          }
          const int from = __ffs(__ballot_sync(0xFFFFFFFFu, rank == a.top_k - 1)) - 1;
          const uint32_t least = __shfl_sync(0xFFFFFFFFu, o, from);
          // (NaN: only NaN is as good; noting more does no harm)
          const float from_here = least == 0xFFFFFFFFu ? CUDART_INF_F : value_of(least);
          const auto note_it = [&](float y) { return !(y < from_here) && y != -CUDART_INF_F; };
#pragma unroll 1
          for (int j = 0; j < kRound; ++j) {
            const int v = v0 + j * kThreads + lane;
            const Vec<kBf16> x = Vec<kBf16>::from(in + j * kUnitBytes);
            if (!note_it(x.top()) || u + j >= end || v >= r.nvec) continue;
#pragma unroll
            for (int i = 0; i < kN; ++i)
              if (note_it(x.at(i))) note(sh, x.at(i), r.id(v, i), V);
          }
          if (least != 0xFFFFFFFFu) bound = from_here;  // (equal ones that come later are behind)
        }
        set_gate();
      }
      Vec<kBf16> x[kRound];
#pragma unroll
      for (int j = 0; j < kRound; ++j) x[j] = Vec<kBf16>::from(in + j * kUnitBytes);
      uint32_t word = x[0].max_word();
#pragma unroll
      for (int j = 1; j < kRound; ++j) word = Vec<kBf16>::max_word(word, x[j].max_word());
      const float top = Vec<kBf16>::top_of(word);
      if (!(top <= gate)) {
        if (top > limit) {
          flush();
          raise(s, top, g.c);
          limit = top + slack;
          ref = top * g.c;
          far = !(fabsf(ref) < 16777216.0f);
          set_floor();
        }
        if (far) {
#pragma unroll 1
          for (int j = 0; j < kRound; ++j) {
            const float2 y = far_sums<kBf16>(in + j * kUnitBytes, s.m, g.c);
            s.l += y.x;
            s.t += y.y;
          }
        }
        if (!closed && rounds > 1 && !(top <= bound)) {
          // (what lies outside the piece is -inf: not above any bound)
#pragma unroll
          for (int j = 0; j < kRound; ++j) {
            if (x[j].top() <= bound) continue;
#pragma unroll
            for (int i = 0; i < kN; ++i)
              if (!(x[j].at(i) <= bound)) note(sh, x[j].at(i), r.id(v0 + j * kThreads + lane, i), V);
          }
        }
        set_gate();
      }
      if (kIds && plain) {
#pragma unroll
        for (int j = 0; j < kRound; ++j) x[j].add_above(than, above);
      }
      {
        const uint64_t c2 = pair(g.c, g.c), m2 = pair(-ref, -ref);  // (of no use where `far`: flush() drops these)
#pragma unroll
        for (int j = 0; j < kRound; ++j) {
#pragma unroll
          for (int i = 0; i < 4; ++i) x[j].w[i] = Vec<kBf16>::max_word(x[j].w[i], floor_word);
#pragma unroll
          for (int i = 0; i < kN; i += 2) {
            const uint64_t d = fma2(pair(x[j].at(i), x[j].at(i + 1)), c2, m2);
            const uint64_t e = pair(exp2_fast(low_of(d)), exp2_fast(high_of(d)));
            l2 = add2(l2, e);
            t2 = fma2(e, d, t2);
          }
        }
      }
      if ((rounds & 1023) == 0) {  // before the counts of 16 a round pass 16 bits
        s.before += Vec<kBf16>::count_of(above);
        above = 0;
      }

      // ---- the best top_k: the bound is raised after 2, 4, 8 .. rounds (a raise
      // costs a block about ten notes, and twice the logits bring top_k notes;
      // fourfold steps, top_k 5: 215 us for 218, 20: 302 for 267)
      if (!closed && rounds == raise_at) {
        raise_at *= 2;
        __syncthreads();
        const int n = sh.noted;
        if (n > kNotes) {
          closed = lost = true;
        } else if (keep_best(sh, n, a.top_k) == a.top_k) {
          // (equal ones that come later are behind it)
          bound = value_of(static_cast<uint32_t>(sh.notes[a.top_k - 1] >> 32));
          closed = bound != bound;  // NaN: nothing that comes later is better
        }  // else fewer than top_k are above -inf
        set_gate();
      }
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }

    // ---- the end of the piece
    flush();
    s.before += Vec<kBf16>::count_of(above);
    const int done_row = row;
    const float done_xt = xt;
    const int done_unit = unit;
    left -= end - unit;
    if (end == g.units) {
      left -= kRowCost;
      ++row;
      unit = 0;
    } else {
      unit = end;
    }
    if (left > 0) {  // the next row's token and its logit
      id = id2;
      xt = given_logit(a, row, id);
      id2 = id_of_row(row + 1);
    }
    // mostly everyone's reference is still the opening's
    const bool same = __all_sync(0xFFFFFFFFu, s.m == __shfl_sync(0xFFFFFFFFu, s.m, 0));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Sums y{same ? s.m : __shfl_xor_sync(0xFFFFFFFFu, s.m, o), __shfl_xor_sync(0xFFFFFFFFu, s.l, o),
                   __shfl_xor_sync(0xFFFFFFFFu, s.t, o), __shfl_xor_sync(0xFFFFFFFFu, s.before, o)};
      if (same) {
        s.l += y.l;
        s.t += y.t;
        s.before += y.before;
      } else {
        join(s, y, g.c);
      }
    }
    if (lane == 0) sh.sums[warp] = s;
    __syncthreads();
    int kept = 0;
    if (a.top_k > 0) {
      kept = sh.noted;
      if (lost || kept > kNotes) {
        best_of<kBf16>(sh, a, done_row, done_unit, end);
        kept = sh.noted;
      } else {
        kept = keep_best(sh, kept, a.top_k);
      }
    }
    if (warp == 0) {
      // -inf is not noted: where less than top_k is above it, all the piece's other
      // logits are -inf, and the first of them are among its first 2 kMaxTopK
      if (kept < a.top_k && !lost) kept = fill<kBf16>(sh, a, done_row, done_unit, end, kept);
      s = sh.sums[lane % kWarps];
#pragma unroll
      for (int o = kWarps / 2; o > 0; o >>= 1) {
        const Sums y{__shfl_xor_sync(0xFFFFFFFFu, s.m, o), __shfl_xor_sync(0xFFFFFFFFu, s.l, o),
                     __shfl_xor_sync(0xFFFFFFFFu, s.t, o), __shfl_xor_sync(0xFFFFFFFFu, s.before, o)};
        join(s, y, g.c);
      }
      const uint64_t key = lane < kept ? sh.notes[lane] : 0;
      if (whole) {
        put(g, done_row, lane, s, key, given, done_xt);
      } else {
        // slot 1 for the row's first part, 0 for a continued one
        Part& p = g.parts[static_cast<int64_t>(blockIdx.x) * 2 + begins];
        if (lane == 0) p.s = s;
        if (lane < a.top_k) p.keys[lane] = key;
      }
    }
    if (left <= 0) return;
    r.set(a, row);  // (what warp 0 still reads is written again only after the next opening's barrier)
  }
}

// Joins the parts of rows that several shares hold, in their order: a block per
// end of a share, which works if it is the first inside a row. Of n sorted lists,
// the r'th largest of their j'th keys bounds the best top_k from below where
// r j >= top_k; what reaches it (at most top_k lists of top_k keys) is ranked by
// counting.
constexpr int kMaxParts = kMaxShares + 1;

__global__ void __launch_bounds__(kThreads) join_kernel(const Args g) {
  __shared__ uint64_t lead[kMaxParts], some[kMaxTopK * kMaxTopK], best[kMaxTopK];
  __shared__ Sums sums[kWarps];
  __shared__ uint64_t bound;
  __shared__ int count;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, k = g.a.top_k;
  const int64_t p0 = blockIdx.x, places = g.units + kRowCost, row = (p0 + 1) * g.share / places;
  const int64_t first = row * places + kRowCost, last = first + g.units - 1;
  // A block with nothing to join waits all the same: where no row is cut that is
  // every block, and whoever comes next in the stream waits for this grid alone.
  if (row >= g.a.T || first < p0 * g.share || first >= (p0 + 1) * g.share) {
    cl::griddep_wait();
    return;
  }
  const int n = static_cast<int>(last / g.share - p0) + 1;
  const int32_t id = g.a.ids != nullptr ? g.a.ids[row] : -1;
  const float xt = given_logit(g.a, row, id);
  if (tid == 0) {
    count = 0;
    bound = 0;
  }
  if (tid < kMaxTopK) best[tid] = 0;
  cl::griddep_wait();
  const auto part = [&](int p) -> const Part& { return g.parts[(p0 + p) * 2 + (p == 0)]; };
  const int j = (k + n - 1) / n, r = j > 0 ? (k + j - 1) / j : 0;
  Sums s{-CUDART_INF_F, 0.0f, 0.0f, 0};
  for (int p = tid; p < n; p += kThreads) {
    const Part& x = part(p);
    if (k > 0) lead[p] = x.keys[j - 1];
    join(s, x.s, g.c);
  }
  if (warp * 32 < n) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Sums y{__shfl_xor_sync(0xFFFFFFFFu, s.m, o), __shfl_xor_sync(0xFFFFFFFFu, s.l, o),
                   __shfl_xor_sync(0xFFFFFFFFu, s.t, o), __shfl_xor_sync(0xFFFFFFFFu, s.before, o)};
      join(s, y, g.c);
    }
  }
  if (lane == 0) sums[warp] = s;
  __syncthreads();
  if (k > 0) {
    for (int p = tid; p < n; p += kThreads) {
      const uint64_t mine = lead[p];
      int rank = 0;
      for (int i = 0; i < n; ++i) rank += lead[i] > mine;
      if (rank == r - 1) bound = mine;  // (no keys at all: 0, from whichever)
    }
    __syncthreads();
    const uint64_t least = bound > 0 ? bound : 1;
    for (int i = tid; i < n * k; i += kThreads) {
      const int p = i / k;
      const uint64_t key = part(p).keys[i - p * k];
      if (key >= least) some[atomicAdd(&count, 1)] = key;
    }
    __syncthreads();
    const int c = count;
    for (int i = tid; i < c; i += kThreads) {
      const uint64_t mine = some[i];
      int rank = 0;
      for (int q = 0; q < c; ++q) rank += some[q] > mine;
      if (rank < k) best[rank] = mine;
    }
    __syncthreads();
  }
  if (warp == 0) {
    s = sums[0];
    for (int w = 1; w < kWarps && w * 32 < n; ++w) join(s, sums[w], g.c);
    put(g, row, lane, s, best[lane], id >= 0 && id < g.a.V, xt);
  }
}

// ---- short rows: a warp per row
//
// A share's block spends about 10 us on a row whatever its length (the opening,
// the barriers of the notes, the end), which many short rows cannot hide. Here a
// row needs no barrier: a lane has every 32nd vector, four on their way, each
// exponent is a difference, and the notes are taken by ballot, so that the list
// never overflows: it is cut to the best as soon as it holds 16 more. 4096 rows
// of 500 bf16 logits, best 5: 10.7 us (88 us in shares); 16384 rows of 8001
// without the best: 78 us, 3.4 TB/s (176), with the best 20 200 us (359). The
// issue bounds it: about eight instructions per logit, and the notes. Two vectors
// on their way or fewer registers (five blocks) cost 5 to 10 %.

constexpr int kAhead = 4;  // vectors of a lane on their way
constexpr int kSpare = 16;  // notes beyond top_k that are kept until the next cut
constexpr int kWarpNotes = kMaxTopK + kSpare + 32 * 8;

// Vector v of a row; what lies outside it is -inf and is not read.
template <bool kBf16>
__device__ __forceinline__ Vec<kBf16> load(const Row<kBf16>& r, int v, uint32_t V) {
  constexpr int kN = Vec<kBf16>::kN;
  const uint32_t id = r.id(v, 0);
  const uint8_t* p = r.base + static_cast<int64_t>(v) * 16;
  if (v < r.nvec && id < V && V - id >= kN) {
    const uint4 y = __ldcs(reinterpret_cast<const uint4*>(p));
    return Vec<kBf16>{{y.x, y.y, y.z, y.w}};
  }
  Vec<kBf16> x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kBf16) {
      x.w[i] = 0xFF80FF80u;
      if (v < r.nvec) {
        if (id + 2 * i < V) x.w[i] = (x.w[i] & 0xFFFF0000u) | reinterpret_cast<const uint16_t*>(p)[2 * i];
        if (id + 2 * i + 1 < V)
          x.w[i] = (x.w[i] & 0xFFFFu) | static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[2 * i + 1]) << 16;
      }
    } else {
      x.w[i] = v < r.nvec && id + i < V ? reinterpret_cast<const uint32_t*>(p)[i] : 0xFF800000u;
    }
  }
  return x;
}

// Sorts the n noted keys' best top_k to the front; returns how many are kept.
__device__ __noinline__ int keep_best_warp(uint64_t* notes, uint64_t* best, int n, int top_k) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
  for (int i = lane; i < n; i += 32) {
    const uint64_t mine = notes[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += notes[j] > mine;
    if (rank < top_k) best[rank] = mine;
  }
  __syncwarp();
  n = n < top_k ? n : top_k;
  if (lane < n) notes[lane] = best[lane];
  __syncwarp();
  return n;
}

// Notes the logits id, id + 1 .. that are of the row and have keys above the
// bound, whose logit is `least`; returns how many there are then. (Not inlined:
// four copies of it, unrolled, are slower than the calls, by half at top_k 20.)
template <bool kBf16>
__device__ __noinline__ int note_warp(Vec<kBf16> x, uint32_t id, uint32_t V, uint64_t bound, float least,
                                      uint64_t* notes, int noted) {
  const uint32_t before = (1u << (threadIdx.x & 31)) - 1u;
#pragma unroll
  for (int i = 0; i < Vec<kBf16>::kN; ++i) {
    if (!__any_sync(0xFFFFFFFFu, !(x.at(i) < least))) continue;
    const uint64_t key = key_of(x.at(i), id + i);
    const bool take = id + i < V && key > bound;
    const unsigned who = __ballot_sync(0xFFFFFFFFu, take);
    if (take) notes[noted + __popc(who & before)] = key;
    noted += __popc(who);
  }
  return noted;
}

template <bool kBf16, bool kIds>
__global__ void __launch_bounds__(kThreads, 4) short_rows_kernel(const Args g) {
  constexpr int kN = Vec<kBf16>::kN;
  __shared__ uint64_t all_notes[kWarps][kWarpNotes], all_best[kWarps][kMaxTopK];
  cl::griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const LogprobArgs& a = g.a;
  if (row >= a.T) return;
  const uint32_t V = static_cast<uint32_t>(a.V);
  uint64_t* const notes = all_notes[warp];
  Row<kBf16> r;
  r.set(a, row);
  const int32_t id = kIds ? a.ids[row] : -1;
  const bool given = kIds && id >= 0 && id < a.V;
  const float xt = kIds ? given_logit(a, row, id) : 0.0f;
  const uint64_t key_t = given ? key_of(xt, static_cast<uint32_t>(id)) : ~uint64_t{0};
  const int v_id = given ? static_cast<int>((static_cast<uint32_t>(id) + r.head) / kN) : -1;
  const float low = next_below<kBf16>(xt);

  Sums s{-CUDART_INF_F, 0.0f, 0.0f, 0};
  uint64_t l2 = 0, t2 = 0;  // added up in pairs
  const auto add_up = [&]() {
    s.l += low_of(l2) + high_of(l2);
    s.t += low_of(t2) + high_of(t2);
    l2 = t2 = 0;
  };
  uint32_t above = 0;
  uint64_t bound = 0;  // keys up to it are not among the best
  float least = 0.0f;  // its logit
  int noted = 0;
  for (int v0 = 0; v0 < r.nvec; v0 += 32 * kAhead) {
    Vec<kBf16> x[kAhead];
    float tops[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) x[j] = load<kBf16>(r, v0 + j * 32 + lane, V);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) tops[j] = x[j].top();

    float top = tops[0];
#pragma unroll
    for (int j = 1; j < kAhead; ++j) top = max_nan(top, tops[j]);
    if (top > s.m) {
      add_up();
      raise(s, top, g.c);
    }
    const float m = s.m == -CUDART_INF_F ? 0.0f : s.m;
    const uint64_t c2 = pair(g.c, g.c), m2 = pair(-m, -m);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (v0 + j * 32 >= r.nvec) break;
#pragma unroll
      for (int i = 0; i < kN; i += 2) {
        uint64_t d = mul2(add2(pair(x[j].at(i), x[j].at(i + 1)), m2), c2);
        d = pair(max_nan(low_of(d), -200.0f), max_nan(high_of(d), -200.0f));
        const uint64_t e = pair(exp2_fast(low_of(d)), exp2_fast(high_of(d)));
        l2 = add2(l2, e);
        t2 = fma2(e, d, t2);
      }
    }

    if (given) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int v = v0 + j * 32 + lane;
        if (v >= r.nvec) continue;
        const uint32_t id0 = r.id(v, 0);
        if (v != v_id && id0 < V && V - id0 >= kN && xt == xt) {
          x[j].add_above(v < v_id ? low : xt, above);
        } else {
#pragma unroll
          for (int i = 0; i < kN; ++i) s.before += id0 + i < V && key_of(x[j].at(i), id0 + i) > key_t;
        }
      }
    }

    if (a.top_k > 0) {
      if (v0 == 0) {
        // top_k logits are not below the top_k'th largest of the lanes' maxima
        const uint32_t o = lane < r.nvec ? order_of(top) : 0u;
        int rank = 0;
#pragma unroll 8
        for (int i = 0; i < 32; ++i) {
          const uint32_t y = __shfl_sync(0xFFFFFFFFu, o, i);
          rank += y > o || (y == o && i < lane);
        }
        const int from = __ffs(__ballot_sync(0xFFFFFFFFu, rank == a.top_k - 1)) - 1;
        bound = static_cast<uint64_t>(__shfl_sync(0xFFFFFFFFu, o, from)) << 32;
        least = value_of(static_cast<uint32_t>(bound >> 32));
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (!__any_sync(0xFFFFFFFFu, !(tops[j] < least))) continue;
        const int v = v0 + j * 32 + lane;
        noted = note_warp(x[j], v < r.nvec ? r.id(v, 0) : 0xFFFFFF00u, V, bound, least, notes, noted);
        if (noted > a.top_k + kSpare) {
          noted = keep_best_warp(notes, all_best[warp], noted, a.top_k);
          if (noted == a.top_k) bound = notes[noted - 1];
          least = value_of(static_cast<uint32_t>(bound >> 32));
        }
      }
    }
  }
  add_up();
  s.before += Vec<kBf16>::count_of(above);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Sums y{__shfl_xor_sync(0xFFFFFFFFu, s.m, o), __shfl_xor_sync(0xFFFFFFFFu, s.l, o),
                 __shfl_xor_sync(0xFFFFFFFFu, s.t, o), __shfl_xor_sync(0xFFFFFFFFu, s.before, o)};
    join(s, y, g.c);
  }
  if (a.top_k > 0) noted = keep_best_warp(notes, all_best[warp], noted, a.top_k);
  put(g, row, lane, s, lane < noted ? notes[lane] : 0, given, xt);
}

}  // namespace

size_t logprobs_ws_bytes(int64_t, int64_t, int) { return sizeof(Part) * 2 * kMaxShares; }

cudaError_t launch_logprobs(const Ctx& c, const LogprobArgs& a) {
  Args g{};
  g.a = a;
  g.c = 1.4426950408889634f / a.temperature;
  const bool bf16 = a.type == WQ_LOGITS_BF16, ids = a.ids != nullptr;
  const int64_t per = bf16 ? 8 : 4;
  // A warp per row for rows of 2 KB, and up to 32 KB where there are many: 1 row of
  // 1000 bf16 logits with the best 20 takes 7.6 us this way, 9.3 in shares; of 4001,
  // 20 and 9.7; but 16384 rows of 1000 48 and 370, 4096 of 8001 61 and 94, 2048 of
  // 8001 22 and 27 without the best, 256 of 2000 14 and 12.
  const int64_t vectors = (a.V + per - 1) / per;
  if (vectors <= 128 || (vectors <= 2048 && a.T >= 2 * vectors)) {
    const auto kern = bf16 ? (ids ? short_rows_kernel<true, true> : short_rows_kernel<true, false>)
                           : (ids ? short_rows_kernel<false, true> : short_rows_kernel<false, false>);
    return launch_early(c, (a.T + kWarps - 1) / kWarps, kThreads, 0, kern, g);
  }
  // a row may begin anywhere within its first vector
  g.units = static_cast<int>(((a.V + 2 * (per - 1)) / per + kThreads - 1) / kThreads);
  const int64_t total = a.T * (g.units + kRowCost);
  int64_t blocks = static_cast<int64_t>(kBlocksPerSm) * c.sm_count;
  if (blocks > kMaxShares) blocks = kMaxShares;
  g.share = (total + blocks - 1) / blocks;
  if (g.share < kLeast) g.share = kLeast;
  g.shares = (total + g.share - 1) / g.share;
  g.parts = static_cast<Part*>(a.ws);
  static SmemLimit lim[4];
  const auto kern = bf16 ? (ids ? logprobs_kernel<true, true> : logprobs_kernel<true, false>)
                         : (ids ? logprobs_kernel<false, true> : logprobs_kernel<false, false>);
  cudaError_t e = raise_smem_limit(lim[bf16 * 2 + ids], kern, c.device, sizeof(Shared));
  if (e != cudaSuccess) return e;
  e = launch_early(c, g.shares, kThreads, sizeof(Shared), kern, g);
  if (e != cudaSuccess || g.shares < 2) return e;
  return launch_early(c, g.shares - 1, kThreads, 0, join_kernel, g);
}

}  // namespace wq
