// Attention of one new token per sequence over a paged key-value cache.
//
// Mathematics: x_t = sm_scale <q, k_t>, out = sum_t e^(x_t) v_t / sum_t e^(x_t),
// in one pass over the tokens with the running maximum m and sum l of the
// softmax; two parts (m1, l1, o1), (m2, l2, o2) of one sequence join to
// m = max, l = sum l_i e^(m_i - m), o = sum o_i e^(m_i - m).
//
// Each key and value is used by the G = Hq / Hkv query heads of its key head
// only, G flop per byte of bf16 cache, so the bound is the cache's read from
// HBM (or, for a few hundred tokens, the chain of latencies: lengths, page
// ids, keys, weights, values). Everything follows from that:
//  - the work of all sequences and key heads is one line of units of 64
//    tokens, cut into equal shares, one per block, two blocks per SM (one where
//    the stages need the shared memory); a share may begin and end inside a
//    sequence. The pieces of a cut (sequence, head) are joined by the block
//    that finishes last, in their order, so the bits do not depend on timing;
//  - a warp takes 16 of a unit's 64 tokens through its own ring of stages
//    filled with cp.async (rows found through the page table one step ahead,
//    rows outside the sequence zero-filled and never read), so warps wait for
//    nothing but their own loads until a (sequence, head) ends;
//  - the products run on warp-level MMAs (m16n8k16): the 16 rows are the heads
//    of the group, and with G <= 8 the second 8 rows carry the low part of the
//    weights: p = hi + lo in two 16-bit numbers keeps the weights to 2^-17
//    (2^-22 for e4m3, whose values are exact in fp16) at no further cost;
//  - e4m3 caches are widened in registers; their scales are factors of the
//    scores and of the output.
#include "wq_device.cuh"
#include "wq_internal.h"

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math_constants.h>

namespace wq {
namespace {

constexpr int kStep = 16;        // tokens a warp takes at a time
// A (sequence, head) of at most this many units is not cut: a join costs
// about as much as a few units in a row.
constexpr int kMinShare = 2;
// What beginning and ending an item costs, in units: every item takes so many
// places more in the line, so that shares with many short items take no longer.
constexpr int kItemCost = 1;
constexpr int kMaxBlocks = 512;  // shares (the partial results' space)

// A head chunk is at most 16 query heads of one key head (kR16), or 8.
template <int D, bool kE4m3, bool kR16>
struct Cfg {
  static constexpr int kRows = kR16 ? 16 : 8;
  static constexpr int kRowBytes = D * (kE4m3 ? 1 : 2);
  static constexpr int kPitch = kRowBytes + 16;  // an odd number of 16-byte words: ldmatrix without conflicts
  static constexpr int kSide = kStep * kPitch;   // a step's keys (or values)
  static constexpr int kStage = 2 * kSide;
  static constexpr int kMisc = 3072;
  // Warps of a block and blocks of an SM: as many warps as the registers (a
  // warp keeps D / 2 or more running sums a thread) and stages allow.
  static constexpr int kBlocksPerSm = D == 64 ? 2 : 1;
  static constexpr int kRoom = (kBlocksPerSm == 2 ? 113 : 227) * 1024 - kMisc;
  static constexpr int kWarps = D <= 128 && D > 64 && kE4m3 ? 12 : (16 * kStage <= kRoom ? 8 : 4);
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kUnit = kStep * kWarps;  // tokens a block takes at a time
  static constexpr int kFit = kRoom / (kWarps * kStage);
  static constexpr int kStages = kFit < 6 ? kFit : 6;
  static constexpr int kSmem = kMisc + kWarps * kStages * kStage;
  // A warp's sums on their way to the block's: kOut rows in the stage that was
  // read last. The pitch keeps 8 rows of a store apart.
  static constexpr int kOPitch = D + (kE4m3 ? 16 : 8);  // floats
  static constexpr int kOut = kE4m3 && kR16 ? 8 : kRows;
  static_assert(kOut * kOPitch * 4 <= kStage, "the sums fit a stage");
  // lanes that load one row (16 bytes each at a time)
  static constexpr int kLanes = kRowBytes % 128 == 0 ? 8 : (kRowBytes % 64 == 0 ? 4 : 2);
  static constexpr int kRowsPerLane = kStep * kLanes / 32;
  static constexpr int kChunks = kRowBytes / (16 * kLanes);
  // registers of 4 for the queries: 16 columns each, or 32 of e4m3 codes (twice with kR16)
  static constexpr int kQ = kE4m3 && !kR16 ? D / 32 : D / 16;
  static_assert(kStages >= 2, "at least two stages");
};

struct Args {
  KvCache kv;
  const uint16_t* q;
  int64_t q_stride;
  const int32_t* lens;
  int Hq, G, chunks;  // query heads, heads per key head, head chunks per key head
  float scale;        // sm_scale log2(e)
  int64_t window;
  uint16_t* out;
  float* lse;
  int32_t* bad;
  float* parts;       // partial results, two per block
  unsigned* arrived;  // one per (sequence, head chunk), zero at rest
  uint32_t div_mul;   // t / S = (t * div_mul) >> div_shift for t < 2^31
  int div_shift;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool kF16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    mma_bf16_16816(c, a[0], a[1], a[2], a[3], b0, b1);
}
__device__ __forceinline__ void mma_e4m3(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four bf16 numbers times `up` as hi + lo, four e4m3 codes each.
__device__ __forceinline__ void split_e4m3(uint2 w, float up, uint32_t& hi, uint32_t& lo) {
  hi = lo = 0u;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t p = j ? w.y : w.x;
    const float x = __uint_as_float(p << 16) * up, y = __uint_as_float(p & 0xFFFF0000u) * up;
    const __nv_fp8x2_storage_t c = __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
    const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3)));
    const __nv_fp8x2_storage_t d = __nv_cvt_float2_to_fp8x2(make_float2(x - f.x, y - f.y), __NV_SATFINITE, __NV_E4M3);
    hi |= static_cast<uint32_t>(c) << (16 * j);
    lo |= static_cast<uint32_t>(d) << (16 * j);
  }
}
// Two e4m3 codes (the low or high half of w) as two fp16 numbers, exactly.
__device__ __forceinline__ uint32_t widen(uint32_t w, bool high) {
  const __nv_fp8x2_storage_t v = static_cast<__nv_fp8x2_storage_t>(high ? w >> 16 : w & 0xFFFFu);
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(v, __NV_E4M3);
  return static_cast<uint32_t>(h.x) | static_cast<uint32_t>(h.y) << 16;
}
// x, y rounded to 16 bits (hi), and what that leaves (lo), packed.
template <bool kF16>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t& hi, uint32_t& lo) {
  if constexpr (kF16) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    const __half2 r = __floats2half2_rn(x - f.x, y - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    const __nv_bfloat162 r = __floats2bfloat162_rn(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xFFFF0000u));
    lo = *reinterpret_cast<const uint32_t*>(&r);
  }
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The tokens of a sequence that count, in units.
struct Span {
  unsigned first, end;  // below 2^31, but a unit may reach past that
  int units;
};
template <int kUnit>
__device__ __forceinline__ Span span_of(const Args& a, int64_t b) {
  int64_t len = a.lens[b];
  const int64_t cap = a.kv.W * a.kv.S;
  if (len > cap) len = cap;
  if (len < 0) len = 0;
  Span s;
  s.end = static_cast<unsigned>(len);
  s.first = a.window > 0 && len > a.window ? static_cast<unsigned>(len - a.window) : 0u;
  s.units = static_cast<int>((s.end - s.first + kUnit - 1) / kUnit);
  return s;
}

// Places of an item in the line: its cost, then its units.
__device__ __forceinline__ int places(const Span& s) { return s.units == 0 ? 0 : s.units + kItemCost; }

// Unit `unit` of head chunk `hc` of sequence b, at place `at` of the line.
template <int kUnit>
struct Cursor {
  int64_t b, at;
  int hc, unit;
  Span s;
  __device__ void next(const Args& a, int per_seq) {
    ++at;
    if (++unit < s.units) return;
    at += kItemCost;
    unit = 0;
    if (++hc < per_seq) return;
    hc = 0;
    do {
      if (++b >= a.kv.B) return;
      s = span_of<kUnit>(a, b);
    } while (s.units == 0);
  }
};

// (m, l) of two parts of a softmax together, into the first.
__device__ __forceinline__ void join(float& m, float& l, float m2, float l2) {
  const float top = fmaxf(m, m2), base = top == -CUDART_INF_F ? 0.0f : top;
  l = l * exp2_fast(m - base) + l2 * exp2_fast(m2 - base);
  m = top;
}

// Four columns of a result.
template <int D>
__device__ __forceinline__ void put(const Args& a, int64_t b, int hq, int d, float4 o, float m, float l, float vs) {
  const float f = l == 0.0f ? 0.0f : vs / l;
  const __nv_bfloat162 x = __floats2bfloat162_rn(o.x * f, o.y * f), y = __floats2bfloat162_rn(o.z * f, o.w * f);
  *reinterpret_cast<uint2*>(a.out + (b * a.Hq + hq) * D + d) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  if (a.lse != nullptr && d == 0)
    a.lse[b * a.Hq + hq] = l == 0.0f ? -CUDART_INF_F : (m + log2f(l)) * 0.6931471805599453f;
}

template <int D, bool kE4m3, bool kR16>
__global__ void __launch_bounds__(Cfg<D, kE4m3, kR16>::kThreads, Cfg<D, kE4m3, kR16>::kBlocksPerSm)
    attn_kernel(const Args a) {
  using C = Cfg<D, kE4m3, kR16>;
  constexpr int kK = D / 16, kN = D / 8, kWarps = C::kWarps, kThreads = C::kThreads, kUnit = C::kUnit;
  extern __shared__ __align__(128) uint8_t smem[];
  float* ml = reinterpret_cast<float*>(smem + kWarps * C::kStages * C::kStage);  // [kWarps][16][2]
  uint32_t* vmask = reinterpret_cast<uint32_t*>(ml + kWarps * 16 * 2);           // [kWarps][kStages]
  int64_t* share = reinterpret_cast<int64_t*>(vmask + 96);  // [0] places of a share, [1] b, [2] those before b, [3] all
  float* whole_ml = reinterpret_cast<float*>(share + 4);                         // [16][2] of a join
  unsigned* last = reinterpret_cast<unsigned*>(whole_ml + 32);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = lane >> 2, col = lane & 3;
  const int per_seq = static_cast<int>(a.kv.Hkv) * a.chunks;

  if (warp == 1) {  // sequences without tokens
    for (int64_t b = blockIdx.x; b < a.kv.B; b += gridDim.x) {
      if (span_of<kUnit>(a, b).units != 0) continue;
      for (int64_t i = lane; i < static_cast<int64_t>(a.Hq) * D / 2; i += 32)
        reinterpret_cast<uint32_t*>(a.out + b * a.Hq * D)[i] = 0;
      if (a.lse != nullptr)
        for (int i = lane; i < a.Hq; i += 32) a.lse[b * a.Hq + i] = -CUDART_INF_F;
    }
  }
  // this block's share: warp 0 adds up the units, each lane some sequences
  if (warp == 0) {
    const int64_t each = (a.kv.B + 31) / 32;
    const int64_t b0 = lane * each, b1 = b0 + each < a.kv.B ? b0 + each : a.kv.B;
    int64_t sum = 0;
    int most = 0;
    for (int64_t b = b0; b < b1; ++b) {
      const int u = places(span_of<kUnit>(a, b));
      sum += u;
      most = u > most ? u : most;
    }
    int64_t upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += y;
    }
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    const int64_t total = __shfl_sync(0xFFFFFFFFu, upto, 31) * per_seq;
    int64_t c = (total + gridDim.x - 1) / gridDim.x;
    const int least = most < kMinShare + kItemCost ? most : kMinShare + kItemCost;
    if (c < least) c = least;
    const int64_t start = c * blockIdx.x;
    if (lane == 0) {
      share[0] = c;
      share[1] = -1;
      share[3] = total;
    }
    __syncwarp();
    if (start < total && start >= (upto - sum) * per_seq && start < upto * per_seq) {
      int64_t before = upto - sum;
      for (int64_t b = b0; b < b1; ++b) {
        const int u = places(span_of<kUnit>(a, b));
        if (start < (before + u) * per_seq) {
          share[1] = b;
          share[2] = before;
          break;
        }
        before += u;
      }
    }
  }
  __syncthreads();
  const int64_t c = share[0], total = share[3];
  if (share[1] < 0) return;
  const int64_t start = c * blockIdx.x, stop = start + c < total ? start + c : total;
  Cursor<kUnit> cur;
  cur.b = share[1];
  cur.s = span_of<kUnit>(a, cur.b);
  {
    const int64_t rel = start - share[2] * per_seq;
    cur.hc = static_cast<int>(rel / places(cur.s));
    const int in = static_cast<int>(rel - static_cast<int64_t>(cur.hc) * places(cur.s));
    cur.unit = in < kItemCost ? 0 : in - kItemCost;
    cur.at = start + (in < kItemCost ? kItemCost - in : 0);
  }

  // ---- the loads: a cursor of their own, the page ids one step ahead
  const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kStage;
  Cursor<kUnit> ld = cur;
  const unsigned S = static_cast<unsigned>(a.kv.S);
  const int64_t to_v = a.kv.Hkv * a.kv.S * C::kRowBytes;
  int ld_slot = 0;
  int32_t ld_page = -1;
  bool ld_in = false;
  auto look_up = [&]() {  // lanes 0..15 (and again 16..31): one token each
    const unsigned t = ld.s.first + static_cast<unsigned>(ld.unit) * kUnit + warp * kStep + (lane & 15);
    ld_in = t < ld.s.end;
    const unsigned j = static_cast<unsigned>((static_cast<uint64_t>(t) * a.div_mul) >> a.div_shift);
    ld_slot = static_cast<int>(t - j * S);
    ld_page = ld_in ? a.kv.table[ld.b * a.kv.W + j] : -1;
  };
  auto load = [&](int stage) {
    const bool ok = ld_in && ld_page >= 0 && ld_page < a.kv.P;
    if (ld_in && !ok && a.bad != nullptr && ld.hc == 0 && lane < 16 &&
        (ld_slot == 0 || (ld.unit == 0 && warp == 0 && lane == 0)))
      atomicAdd(a.bad, 1);
    // a row that is left out reads nothing: its copies have no bytes
    const int h = ld.hc / a.chunks;
    uint64_t from = reinterpret_cast<uint64_t>(a.kv.kv);
    if (ok) from += ((static_cast<int64_t>(ld_page) * 2 * a.kv.Hkv + h) * a.kv.S + ld_slot) * C::kRowBytes;
    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, ok) & 0xFFFFu;
    if (lane == 0) vmask[warp * C::kStages + stage] = mask;
    const uint32_t base = ring + stage * C::kStage + (lane / C::kLanes) * C::kPitch + (lane % C::kLanes) * 16;
#pragma unroll
    for (int i = 0; i < C::kRowsPerLane; ++i) {
      const int r = lane / C::kLanes + i * (32 / C::kLanes);
      const uint64_t src = __shfl_sync(0xFFFFFFFFu, from, r) + (lane % C::kLanes) * 16;
      const uint32_t bytes = (mask >> r & 1u) * 16u;
      const uint32_t dst = base + i * (32 / C::kLanes) * C::kPitch;
#pragma unroll
      for (int j = 0; j < C::kChunks; ++j) {
        cp_async16(dst + j * C::kLanes * 16, reinterpret_cast<const void*>(src + j * C::kLanes * 16), bytes);
        cp_async16(dst + C::kSide + j * C::kLanes * 16, reinterpret_cast<const void*>(src + to_v + j * C::kLanes * 16),
                   bytes);
      }
    }
    ld.next(a, per_seq);
    if (ld.at < stop) look_up();
  };
  if (ld.at < stop) look_up();
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) {
    if (ld.at < stop) load(i);
    cp_async_commit();
  }

  // ---- the pieces of (sequence, head chunk) items
  int stage = 0;
  while (cur.at < stop) {
    const int h = cur.hc / a.chunks, chunk = cur.hc - h * a.chunks;
    const int hq0 = h * a.G + chunk * 16;
    const int rows = a.G - chunk * 16 < 16 ? a.G - chunk * 16 : 16;
    const int64_t item0 = cur.at - cur.unit, item1 = item0 + cur.s.units;
    const int units = static_cast<int>((item1 < stop ? item1 : stop) - cur.at);

    // the queries as the MMA's row operand. For an e4m3 cache they are split
    // into two e4m3 numbers behind a power of two that puts the row's largest
    // in [2^7, 2^8): q = q1 + q2 exactly, but for numbers below 2^-9 of the
    // largest, which are off by at most 2^-17 of it
    uint32_t qa[C::kQ][4];
    float scale[2] = {a.scale, a.scale};
    {
      const uint16_t* qp = a.q + cur.b * a.q_stride + static_cast<int64_t>(hq0) * D;
#pragma unroll
      for (int half = 0; half < (kR16 ? 2 : 1); ++half) {
        const int r = row + 8 * half;
        const bool in = r < rows;
        if constexpr (!kE4m3) {
#pragma unroll
          for (int k = 0; k < kK; ++k) {
            const uint32_t* p = reinterpret_cast<const uint32_t*>(qp + r * D + k * 16 + 2 * col);
            qa[k][half] = in ? p[0] : 0u;      // columns 2 col, 2 col + 1
            qa[k][half + 2] = in ? p[4] : 0u;  // and 8 further
            if constexpr (!kR16) qa[k][1] = qa[k][3] = 0u;
          }
        } else {
          // 4 columns at 4 col of every 16
          uint2 w[kK];
          uint32_t top = 0;
#pragma unroll
          for (int k = 0; k < kK; ++k) {
            w[k] = in ? *reinterpret_cast<const uint2*>(qp + r * D + k * 16 + 4 * col) : make_uint2(0u, 0u);
            top = __vmaxu2(top, __vmaxu2(w[k].x & 0x7FFF7FFFu, w[k].y & 0x7FFF7FFFu));
          }
          top = (top >> 16) > (top & 0xFFFFu) ? top >> 16 : top & 0xFFFFu;
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
          const bool wrong = top >= 0x7F80u;     // an infinite or NaN query: NaN
          int e = static_cast<int>(top >> 7) - 127;  // the largest is in [2^e, 2^(e + 1))
          e = top == 0 || wrong ? 7 : (e < -93 ? -93 : (e > 107 ? 107 : e));
          const float up = __int_as_float((7 - e + 127) << 23), down = __int_as_float((e - 7 + 127) << 23);
          scale[half] = a.scale * a.kv.k_scale[h] * down;
#pragma unroll
          for (int k = 0; k < kK; ++k) {
            uint32_t hi, lo;
            split_e4m3(w[k], up, hi, lo);
            if (wrong) hi = 0x7F7F7F7Fu;
            if constexpr (kR16) {  // q1 and q2 in operands of their own
              qa[k >> 1][half + 2 * (k & 1)] = hi;
              qa[kK / 2 + (k >> 1)][half + 2 * (k & 1)] = lo;
            } else {  // q2 in the rows 8 below
              qa[k >> 1][2 * (k & 1)] = hi;
              qa[k >> 1][2 * (k & 1) + 1] = lo;
            }
          }
        }
      }
    }

    float acc[kN][4];
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
    float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.0f, 0.0f};

    for (int u = 0; u < units; ++u) {
      cp_async_wait<C::kStages - 2>();
      __syncwarp();
      // the stage read in the step before is free again
      if (ld.at < stop) load(stage == 0 ? C::kStages - 1 : stage - 1);
      cp_async_commit();
      const uint32_t mask = vmask[warp * C::kStages + stage];
      const uint32_t kbase = ring + stage * C::kStage, vbase = kbase + C::kSide;
      if (mask != 0) {
        // scores of 16 tokens: s[j] has tokens 8 j + 2 col, + 1 of rows `row` and row + 8
        float s[2][4] = {}, s2[2][4] = {};  // two chains
        if constexpr (!kE4m3) {
          const uint32_t addr = kbase + ((lane & 7) + (lane >> 4) * 8) * C::kPitch + ((lane >> 3) & 1) * 16;
#pragma unroll
          for (int k = 0; k < kK; ++k) {
            uint32_t b[4];
            ldsm4(addr + k * 32, b);
            mma<false>((k & 1) ? s2[0] : s[0], qa[k], b[0], b[1]);
            mma<false>((k & 1) ? s2[1] : s[1], qa[k], b[2], b[3]);
          }
        } else {
          const uint32_t addr = kbase + (lane & 15) * C::kPitch + (lane >> 4) * 16;
#pragma unroll
          for (int k = 0; k < kK / 2; ++k) {
            uint32_t b[4];  // 16 codes of tokens 0-7, 8-15, then the next 16
            ldsm4(addr + k * 32, b);
            mma_e4m3((k & 1) ? s2[0] : s[0], qa[k], b[0], b[2]);
            mma_e4m3((k & 1) ? s2[1] : s[1], qa[k], b[1], b[3]);
            if constexpr (kR16) {
              mma_e4m3((k & 1) ? s[0] : s2[0], qa[kK / 2 + k], b[0], b[2]);
              mma_e4m3((k & 1) ? s[1] : s2[1], qa[kK / 2 + k], b[1], b[3]);
            }
          }
          if constexpr (!kR16) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                s[j][i] += s[j][i + 2];
                s2[j][i] += s2[j][i + 2];
              }
          }
        }
        float top[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < (kR16 ? 4 : 2); ++i) {
            s[j][i] = (s[j][i] + s2[j][i]) * scale[i >> 1];
            if (mask != 0xFFFFu && ((mask >> (8 * j + 2 * col + (i & 1))) & 1u) == 0) s[j][i] = -CUDART_INF_F;
            top[i >> 1] = fmaxf(top[i >> 1], s[j][i]);
          }
        bool raised = false;
        float base[2], shrink[2];
#pragma unroll
        for (int i = 0; i < (kR16 ? 2 : 1); ++i) {
          top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 1));
          top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 2));
          const float m2 = fmaxf(m[i], top[i]);
          raised |= m2 > m[i];
          base[i] = m2 == -CUDART_INF_F ? 0.0f : m2;
          shrink[i] = exp2_fast(m[i] - base[i]);
          m[i] = m2;
        }
        if (__any_sync(0xFFFFFFFFu, raised)) {
#pragma unroll
          for (int n = 0; n < kN; ++n) {
            acc[n][0] *= shrink[0];
            acc[n][1] *= shrink[0];
            acc[n][2] *= shrink[kR16 ? 1 : 0];
            acc[n][3] *= shrink[kR16 ? 1 : 0];
          }
#pragma unroll
          for (int i = 0; i < (kR16 ? 2 : 1); ++i) l[i] *= shrink[i];
        }
        uint32_t hi[2][2], lo[2][2];  // [tokens 8 j ..][rows, rows + 8]
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < (kR16 ? 2 : 1); ++i) {
            const float p0 = exp2_fast(s[j][2 * i] - base[i]), p1 = exp2_fast(s[j][2 * i + 1] - base[i]);
            l[i] += p0 + p1;
            split_pair<kE4m3>(p0, p1, hi[j][i], lo[j][i]);
          }
        // values: b[0], b[1] the tokens' halves of 8 columns, b[2], b[3] of the next 8
        const uint32_t addr = vbase + (lane & 15) * C::kPitch + (lane >> 4) * 16;
        auto accumulate = [&](int n, uint32_t b0, uint32_t b1) {
          if constexpr (kR16) {
            mma<kE4m3>(acc[n], {hi[0][0], hi[0][1], hi[1][0], hi[1][1]}, b0, b1);
            mma<kE4m3>(acc[n], {lo[0][0], lo[0][1], lo[1][0], lo[1][1]}, b0, b1);
          } else {
            mma<kE4m3>(acc[n], {hi[0][0], lo[0][0], hi[1][0], lo[1][0]}, b0, b1);
          }
        };
        if constexpr (!kE4m3) {
#pragma unroll
          for (int n2 = 0; n2 < kN / 2; ++n2) {
            uint32_t b[4];
            ldsm4_trans(addr + n2 * 32, b);
            accumulate(2 * n2, b[0], b[1]);
            accumulate(2 * n2 + 1, b[2], b[3]);
          }
        } else {
          // 16 columns of codes: a register holds columns 2 row, 2 row + 1 of
          // two tokens; the even columns make one tile, the odd ones another
#pragma unroll
          for (int n4 = 0; n4 < kN / 4; ++n4) {
            uint32_t b[4];
            ldsm4_trans(addr + n4 * 32, b);
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = __byte_perm(b[j], 0u, 0x3120);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              accumulate(4 * n4 + 2 * j, widen(b[2 * j], false), widen(b[2 * j + 1], false));
              accumulate(4 * n4 + 2 * j + 1, widen(b[2 * j], true), widen(b[2 * j + 1], true));
            }
          }
        }
      }
      stage = stage + 1 == C::kStages ? 0 : stage + 1;
    }
    // to the piece's last unit; next() below leaves the item or ends the share
    cur.unit += units - 1;
    cur.at += units - 1;

    // ---- the warps' parts, in their order: each puts its sums where the stage
    // of the step just done lies (the next load into it comes after the
    // barriers), then every thread adds up some columns of all warps
    if constexpr (!kR16) {
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        acc[n][0] += acc[n][2];
        acc[n][1] += acc[n][3];
      }
    }
#pragma unroll
    for (int i = 0; i < (kR16 ? 2 : 1); ++i) {
      l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 1);
      l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 2);
      if (col == 0) {
        ml[(warp * 16 + row + 8 * i) * 2] = m[i];
        ml[(warp * 16 + row + 8 * i) * 2 + 1] = l[i];
      }
    }
    const bool whole = item0 >= start && item1 <= stop;
    const float vs = kE4m3 ? a.kv.v_scale[h] : 1.0f;
    uint8_t* outs = smem + (stage == 0 ? C::kStages - 1 : stage - 1) * C::kStage;
    // a part of several: rows of D sums, then (m, l) of each row; slot 1 for
    // the item's first part, 0 for a continued one
    float* part = a.parts + (static_cast<int64_t>(blockIdx.x) * 2 + (item0 >= start)) * C::kRows * (D + 2);
    __syncwarp();  // all lanes have read the stage
#pragma unroll
    for (int r0 = 0; r0 < C::kRows; r0 += C::kOut) {
      float* mine = reinterpret_cast<float*>(outs + warp * C::kStages * C::kStage);
      if (r0 > 0) __syncthreads();
#pragma unroll
      for (int i = r0 / 8; i < (r0 + C::kOut) / 8; ++i) {
        float* p = mine + (row + 8 * i - r0) * C::kOPitch;
        if constexpr (!kE4m3) {
#pragma unroll
          for (int n = 0; n < kN; ++n)
            *reinterpret_cast<float2*>(p + 8 * n + 2 * col) = make_float2(acc[n][2 * i], acc[n][2 * i + 1]);
        } else {  // tiles n and n + 1 hold the even and the odd columns
#pragma unroll
          for (int n = 0; n < kN; n += 2)
            *reinterpret_cast<float4*>(p + 8 * n + 4 * col) =
                make_float4(acc[n][2 * i], acc[n + 1][2 * i], acc[n][2 * i + 1], acc[n + 1][2 * i + 1]);
        }
      }
      __syncthreads();
      const int here = rows - r0 < C::kOut ? rows - r0 : C::kOut;
      for (int i = tid; i < here * (D / 4); i += kThreads) {
        const int r = i / (D / 4), d = 4 * (i - r * (D / 4));
        const float* p = ml + (r0 + r) * 2;
        float M = p[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) M = fmaxf(M, p[w * 32]);
        const float base = M == -CUDART_INF_F ? 0.0f : M;
        float L = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = exp2_fast(p[w * 32] - base);
          const float4 v = *reinterpret_cast<const float4*>(outs + w * C::kStages * C::kStage + (r * C::kOPitch + d) * 4);
          L += p[w * 32 + 1] * f;
          o.x += v.x * f;
          o.y += v.y * f;
          o.z += v.z * f;
          o.w += v.w * f;
        }
        if (whole) {
          put<D>(a, cur.b, hq0 + r0 + r, d, o, M, L, vs);
        } else {
          *reinterpret_cast<float4*>(part + (r0 + r) * D + d) = o;
          if (d == 0) *reinterpret_cast<float2*>(part + C::kRows * D + (r0 + r) * 2) = make_float2(M, L);
        }
      }
    }
    __syncthreads();
    if (!whole) {
      const int64_t p0 = item0 / c;
      const int n_parts = static_cast<int>((item1 - 1) / c - p0) + 1;
      if (tid == 0) {
        unsigned* count = a.arrived + cur.b * per_seq + cur.hc;
        __threadfence();
        const bool is_last = atom_add_acq_rel_gpu(count, 1u) == static_cast<unsigned>(n_parts - 1);
        if (is_last) *count = 0;  // nobody else will: all parts are here
        *last = is_last;
      }
      __syncthreads();
      if (*last) {
        __threadfence();
        const auto at = [&](int p) { return a.parts + ((p0 + p) * 2 + (p == 0)) * C::kRows * (D + 2); };
        // (m, l) of the whole: a warp per row, parts over the lanes
        for (int r = warp; r < rows; r += kWarps) {
          float M = -CUDART_INF_F, L = 0.0f;
#pragma unroll 4
          for (int p = lane; p < n_parts; p += 32) {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(at(p) + C::kRows * D + r * 2));
            join(M, L, v.x, v.y);
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const float M2 = __shfl_xor_sync(0xFFFFFFFFu, M, o), L2 = __shfl_xor_sync(0xFFFFFFFFu, L, o);
            join(M, L, M2, L2);
          }
          if (lane == 0) {
            whole_ml[2 * r] = M;
            whole_ml[2 * r + 1] = L;
          }
        }
        __syncthreads();
        // 4 columns a thread; the parts over the warp's four groups of 8 lanes
        for (int i0 = warp * 8; i0 < rows * (D / 4); i0 += kWarps * 8) {
          const int i = i0 + (lane & 7), r = i / (D / 4), d = 4 * (i - r * (D / 4));  // rows * D / 4 is a multiple of 8
          const float M = whole_ml[2 * r], base = M == -CUDART_INF_F ? 0.0f : M;
          float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
          for (int p = lane >> 3; p < n_parts; p += 4) {
            const float* q = at(p);
            const float4 v = __ldcg(reinterpret_cast<const float4*>(q + r * D + d));
            const float f = exp2_fast(__ldcg(q + C::kRows * D + r * 2) - base);
            o.x += v.x * f;
            o.y += v.y * f;
            o.z += v.z * f;
            o.w += v.w * f;
          }
#pragma unroll
          for (int x = 8; x < 32; x <<= 1) {
            o.x += __shfl_xor_sync(0xFFFFFFFFu, o.x, x);
            o.y += __shfl_xor_sync(0xFFFFFFFFu, o.y, x);
            o.z += __shfl_xor_sync(0xFFFFFFFFu, o.z, x);
            o.w += __shfl_xor_sync(0xFFFFFFFFu, o.w, x);
          }
          if (lane < 8) put<D>(a, cur.b, hq0 + r, d, o, M, whole_ml[2 * r + 1], vs);
        }
      }
    }
    cur.next(a, per_seq);
  }
}

template <int D, bool kE4m3, bool kR16>
cudaError_t launch(const Ctx& c, const Args& a) {
  using C = Cfg<D, kE4m3, kR16>;
  static SmemLimit lim;
  cudaError_t e = raise_smem_limit(lim, attn_kernel<D, kE4m3, kR16>, c.device, C::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t cap = a.kv.W * a.kv.S, most = a.window > 0 && a.window < cap ? a.window : cap;
  const int64_t items = a.kv.B * a.kv.Hkv * a.chunks, units = (most + C::kUnit - 1) / C::kUnit;
  int64_t grid = static_cast<int64_t>(C::kBlocksPerSm) * c.sm_count;
  if (grid > kMaxBlocks) grid = kMaxBlocks;
  if (items < grid && items * units < grid) grid = items * units;
  attn_kernel<D, kE4m3, kR16><<<static_cast<unsigned>(grid), C::kThreads, C::kSmem, c.stream>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const Ctx& c, const Args& a) {
  const bool e4m3 = a.kv.type == WQ_KV_E4M3, r16 = a.G > 8;
  if (e4m3) return r16 ? launch<D, true, true>(c, a) : launch<D, true, false>(c, a);
  return r16 ? launch<D, false, true>(c, a) : launch<D, false, false>(c, a);
}

}  // namespace

// Partial results first, in a space that does not depend on the batch, then
// the arrival counters: a call of another shape never writes partial results
// where counters must be zero.
constexpr size_t kPartsBytes = static_cast<size_t>(kMaxBlocks) * 2 * 16 * (256 + 2) * 4;

size_t kv_attn_ws_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t D) {
  const int64_t G = Hq / Hkv;
  (void)D;
  return kPartsBytes + static_cast<size_t>(B) * Hkv * ((G + 15) / 16) * 4;
}

cudaError_t launch_kv_attn(const Ctx& c, const KvCache& kv, const uint16_t* q, int64_t q_stride, const int32_t* lens,
                           int64_t Hq, float sm_scale, int64_t window, uint16_t* out, float* lse, int32_t* bad,
                           void* ws) {
  Args a{};
  a.kv = kv;
  a.q = q;
  a.q_stride = q_stride;
  a.lens = lens;
  a.Hq = static_cast<int>(Hq);
  a.G = static_cast<int>(Hq / kv.Hkv);
  a.chunks = (a.G + 15) / 16;
  a.scale = sm_scale * 1.4426950408889634f;
  a.window = window;
  a.out = out;
  a.lse = lse;
  a.bad = bad;
  a.parts = static_cast<float*>(ws);
  a.arrived = reinterpret_cast<unsigned*>(static_cast<uint8_t*>(ws) + kPartsBytes);
  int l = 0;
  while ((int64_t{1} << l) < kv.S) ++l;
  a.div_shift = 31 + l;
  a.div_mul = static_cast<uint32_t>((uint64_t{1} << (31 + l)) / static_cast<uint64_t>(kv.S) + 1);
  switch (kv.D) {
    case 64: return launch_d<64>(c, a);
    case 96: return launch_d<96>(c, a);
    case 128: return launch_d<128>(c, a);
    case 192: return launch_d<192>(c, a);
    case 256: return launch_d<256>(c, a);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace wq
