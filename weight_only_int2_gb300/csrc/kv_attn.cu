// Attention of one new token per sequence over a paged key-value cache.
//
// Mathematics: x_t = sm_scale <q, k_t>, out = sum_t e^(x_t) v_t / sum_t e^(x_t),
// in one pass over the tokens with a reference m (a maximum seen so far) and
// the sum l of the softmax; two parts (m1, l1, o1), (m2, l2, o2) of one sequence
// join to m = max, l = sum l_i e^(m_i - m), o = sum o_i e^(m_i - m).
//
// Each key and value is used by the G = Hq / Hkv query heads of its key head
// only, G flop per byte of bf16 cache, so the bound is the cache's read from
// HBM (or, for a few hundred tokens, the chain of latencies: lengths, page
// ids, keys, weights, values). Everything follows from that:
//  - the work of all sequences and key heads is one line of units, cut into
//    equal shares, one per block, as many blocks as fit the GPU at once; a share
//    may begin and end inside a sequence. A second kernel joins the pieces of
//    a cut (sequence, head) in their order, so the bits do not depend on timing;
//  - a warp takes 16 of a unit's tokens through its own ring of stages filled
//    with cp.async (rows found through the page table one step ahead, rows
//    outside the sequence zero-filled and never read), so warps wait for
//    nothing but their own loads until a (sequence, head) ends;
//  - the products run on warp-level MMAs with the tokens (scores) and the
//    columns (output) as the 16 rows and 8 query heads as the columns: no row
//    is padding, and a thread keeps D / 4 sums for 8 heads. The weights go into
//    the second product as hi + lo, two 16-bit numbers, which keeps each to 2^-17
//    of itself, however small it is beside the others;
//  - e4m3 keys are multiplied as they are, by queries split into two e4m3
//    numbers; e4m3 values are transposed as codes and widened to fp16 in
//    registers, or to bf16 (three more instructions for two values) with 16
//    tokens among whose weights there are some that fp16 is too short for: where
//    all are so, D = 64 takes 109 us for 100 (64 sequences of up to 16011), D = 128
//    181 to 184 either way, 16 heads 118 for 107, D = 256 152 for 143. The caches'
//    scales are factors of the scores and of the output.
//
// Measured (of a copy's 6.8 TB/s): 64 sequences of 1 to 8192 tokens, 8 key heads
// of 4 query heads, D = 128, bf16, 1.07 GB: 174 us, 6.2 TB/s; one of 131071
// tokens, 40 query heads, 537 MB: 92 us, 5.9 TB/s; 48 of up to 16384 tokens, 4
// key heads of 6, D = 256, e4m3, 0.95 GB: 160 to 165 us, 5.8 TB/s, where a third of
// the issue and of the tensor pipe is taken. A call has about 12 us
// that do not stream: the start, the last block's end and the join (8 us by
// itself, half of it under the first kernel's end). 77 tokens: 3.8 us. From L2 the
// same loops run at 10.7 TB/s, so they are not the bound. Several waves of shares
// instead of one (the one long sequence: 145 us), shares taken by tickets (124 us)
// and a join by the block that comes last (6 to 25 us more) were slower.
#include "wq_cluster.cuh"
#include "wq_device.cuh"
#include "wq_internal.h"

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math_constants.h>

#include <type_traits>

namespace wq {
namespace {

// What beginning and ending an item costs, in units: every item takes so many
// places more in the line, so that shares with many short items take no longer.
constexpr int kItemCost = 1;
// Shares of so many units are not made smaller (a join costs about as much).
constexpr int least_units(int unit) { return unit > 64 ? 2 : 4; }
// The weights are relative to a reference that is raised when a score passes it
// by more than this (in powers of two), so that most steps need no maximum.
constexpr float kSlack = 8.0f;
// fp16 holds 2^-24 to 2^15: for e4m3 the reference lies so far below the first
// largest score that weights come up to 2^15, and hi + lo, off by at most 2^-25,
// is within 2^-17 of weights of kLeastF16 and more.
constexpr float kDown = 7.0f;
constexpr float kLeastF16 = 0.00390625f;

// Blocks that share an SM: as many as the registers allow (a thread keeps D / 4
// sums and D / 8 registers of queries for 8 heads, twice that for 16, and with
// e4m3 two parts of a step) and the stages leave room for.
constexpr int blocks_per_sm(int64_t d, bool e4m3, bool r16) {
  if (r16 && e4m3) return 2;
  if (r16) return d <= 64 ? 4 : (d <= 128 ? 3 : 2);
  if (e4m3) return d <= 128 ? 3 : 2;
  return d <= 96 ? 4 : (d == 128 ? 3 : 2);
}
// Shares that the space for partial results is for (a GB300 has 152 SMs).
constexpr int max_shares(int64_t d, bool e4m3, bool r16) { return 160 * blocks_per_sm(d, e4m3, r16); }

// A head chunk is at most 16 query heads of one key head (kR16), or 8.
template <int D, bool kE4m3, bool kR16>
struct Cfg {
  static constexpr int kRows = kR16 ? 16 : 8;
  static constexpr int kTiles = kRows / 8;       // MMA columns of 8 heads
  static constexpr int kRowBytes = D * (kE4m3 ? 1 : 2);
  static constexpr int kPitch = kRowBytes + 16;  // an odd number of 16-byte words: ldmatrix without conflicts
  // Tokens a warp takes at a time: of e4m3 codes twice as many, the same bytes, so
  // that the places are found once for 32 (D = 64: 98 us for 113; 16 heads of
  // D = 128: 245 for 304); not where the sums of 16 heads leave no registers for
  // it (D = 256: 215 us for 158).
  static constexpr int kStep = kE4m3 && (!kR16 || D <= 192) ? 32 : 16;
  static constexpr int kSide = kStep * kPitch;   // a step's keys (or values)
  static constexpr int kStage = 2 * kSide;
  static constexpr int kMisc = 1024;
  // Several blocks share an SM, so that one streams while another begins or
  // ends a share.
  static constexpr int kBlocksPerSm = blocks_per_sm(D, kE4m3, kR16);
  static constexpr int kRoom = 226 * 1024 / kBlocksPerSm - kMisc;
  static constexpr int kWarps = 8 * kStage <= kRoom ? 4 : 3;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kUnit = kStep * kWarps;  // tokens a block takes at a time
  static constexpr int kFit = kRoom / (kWarps * kStage);
  static constexpr int kStages = kFit < 6 ? kFit : 6;
  static constexpr int kSmem = kMisc + kWarps * kStages * kStage;
  // A warp's sums on their way to the block's: kOut heads in the stage that was
  // read last. The pitch keeps the 32 words of a store apart.
  static constexpr int kOPitch = D + 4;  // floats
  static constexpr int kOut = kE4m3 && kR16 && kStep == 16 ? 8 : kRows;
  static_assert(kOut * kOPitch * 4 <= kStage, "the sums fit a stage");
  // lanes that load one row (16 bytes each at a time)
  static constexpr int kLanes = kRowBytes % 128 == 0 ? 8 : (kRowBytes % 64 == 0 ? 4 : 2);
  static constexpr int kRowsPerLane = kStep * kLanes / 32;
  static constexpr int kChunks = kRowBytes / (16 * kLanes);
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
  float* parts;      // partial results, two per share
  int shares;        // at most
  bool direct;       // a share per item, nothing cut
  bool by_cut;       // the join has per_join blocks for every end of a share, else for every sequence
  int per_join;
  uint32_t div_mul;  // t / S = (t * div_mul) >> div_shift for t < 2^31
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
// Two matrices of 16 x 16 8-bit numbers: of columns lane / 4 and lane / 4 + 8 the
// rows 4 (lane % 4) .. + 3, for either.
__device__ __forceinline__ void ldsm2_codes(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// A matrix of 8 x 8 16-bit numbers, transposed across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <bool kF16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  if constexpr (kF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
  else
    mma_bf16_16816(c, a[0], a[1], a[2], a[3], b[0], b[1]);
}
__device__ __forceinline__ void mma_e4m3(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
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
// Four e4m3 codes as fp16 numbers, exactly: the low two and the high two.
__device__ __forceinline__ void widen(uint32_t w, uint32_t& low, uint32_t& high) {
  asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\ncvt.rn.f16x2.e4m3x2 %0, l;\ncvt.rn.f16x2.e4m3x2 %1, h;\n}"
      : "=r"(low), "=r"(high)
      : "r"(w));
}
// The same as bf16 numbers, exactly, too.
__device__ __forceinline__ void widen_bf16(uint32_t w, uint32_t& low, uint32_t& high) {
  uint32_t h[2];
  widen(w, h[0], h[1]);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h[0]));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&h[1]));
  low = __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
  high = __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x7632);
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

// n / d of numbers that are rarely large (a 64-bit division takes a while).
__device__ __forceinline__ int64_t quotient(int64_t n, int64_t d) {
  if ((n >> 32) == 0 && (d >> 32) == 0) return static_cast<uint32_t>(n) / static_cast<uint32_t>(d);
  return n / d;
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

// Unit `unit` of head chunk `hc` of sequence b, with `left` places of the share
// from there on (a share of 2^31 places would take years).
template <int kUnit>
struct Cursor {
  int64_t b;
  int hc, unit, left;
  Span s;
  // To the next unit; true where that is another item's.
  __device__ bool next(const Args& a, int per_seq) {
    --left;
    if (++unit < s.units) return false;
    left -= kItemCost;
    unit = 0;
    if (++hc < per_seq) return true;
    hc = 0;
    do {
      if (++b >= a.kv.B) {
        left = 0;
        return true;
      }
      s = span_of<kUnit>(a, b);
    } while (s.units == 0);
    return true;
  }
};

// The line of all items, found by a warp: each lane adds up the places of
// sequences b0 .. b1 - 1, which lie at before .. upto - 1 (times the items of a
// sequence); `share` places make a share.
struct Line {
  int64_t total, share, before, upto, b0, b1;
};
template <int kUnit>
__device__ __forceinline__ Line line_of(const Args& a, int per_seq, int shares) {
  const int lane = threadIdx.x & 31;
  const int64_t each = (a.kv.B + 31) / 32;
  Line x;
  x.b0 = lane * each;
  x.b1 = x.b0 + each < a.kv.B ? x.b0 + each : a.kv.B;
  int64_t sum = 0;
  int most = 0;
#pragma unroll 4
  for (int64_t b = x.b0; b < x.b1; ++b) {
    const int u = places(span_of<kUnit>(a, b));
    sum += u;
    most = u > most ? u : most;
  }
  x.upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x.upto, o);
    if (lane >= o) x.upto += y;
  }
  x.before = x.upto - sum;
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  x.total = __shfl_sync(0xFFFFFFFFu, x.upto, 31) * per_seq;
  x.share = quotient(x.total + shares - 1, shares);
  const int least = most < least_units(kUnit) + kItemCost ? most : least_units(kUnit) + kItemCost;
  x.share = x.share > least ? x.share : least;
  return x;
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
  constexpr int kK = kE4m3 ? D / 32 : D / 16, kT = D / 16, kWarps = C::kWarps, kThreads = C::kThreads;
  constexpr int kUnit = C::kUnit, kTiles = C::kTiles, kStep = C::kStep, kParts = kStep / 16;
  constexpr uint32_t kFull = kStep == 32 ? 0xFFFFFFFFu : 0xFFFFu;
  extern __shared__ __align__(128) uint8_t smem[];
  float* ml = reinterpret_cast<float*>(smem + kWarps * C::kStages * C::kStage);  // [kWarps][16][2]
  int64_t* share = reinterpret_cast<int64_t*>(ml + kWarps * 16 * 2);  // [0] places of a share, [1] b, [2] those before b, [3] all
  uint32_t* vmask = reinterpret_cast<uint32_t*>(share + 4);           // [kWarps][kStages]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = lane >> 2, col = lane & 3;
  const int per_seq = static_cast<int>(a.kv.Hkv) * a.chunks;

  cl::griddep_wait();
  cl::griddep_launch_dependents();  // the join may start; it waits for this kernel's end
  if (warp == 1) {  // sequences without tokens
    for (int64_t b = blockIdx.x; b < a.kv.B; b += gridDim.x) {
      if (span_of<kUnit>(a, b).units != 0) continue;
      for (int64_t i = lane; i < static_cast<int64_t>(a.Hq) * D / 2; i += 32)
        reinterpret_cast<uint32_t*>(a.out + b * a.Hq * D)[i] = 0;
      if (a.lse != nullptr)
        for (int i = lane; i < a.Hq; i += 32) a.lse[b * a.Hq + i] = -CUDART_INF_F;
    }
  }
  if (warp == 0 && !a.direct) {
    const Line line = line_of<kUnit>(a, per_seq, gridDim.x);
    const int64_t start = line.share * blockIdx.x;
    if (lane == 0) {
      share[0] = line.share;
      share[1] = -1;
      share[3] = line.total;
    }
    __syncwarp();
    if (start < line.total && start >= line.before * per_seq && start < line.upto * per_seq) {
      int64_t before = line.before;
      for (int64_t b = line.b0; b < line.b1; ++b) {
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
  int64_t start = 0, stop = 0;
  Cursor<kUnit> cur;
  if (a.direct) {
    cur.b = blockIdx.x / per_seq;
    cur.hc = static_cast<int>(blockIdx.x - cur.b * per_seq);
    cur.s = span_of<kUnit>(a, cur.b);
    cur.unit = 0;
    cur.left = cur.s.units;
  } else {
    __syncthreads();
    const int64_t c = share[0], total = share[3];
    if (share[1] < 0) return;
    start = c * blockIdx.x;
    stop = start + c < total ? start + c : total;
    cur.b = share[1];
    cur.s = span_of<kUnit>(a, cur.b);
    const int64_t rel = start - share[2] * per_seq;
    cur.hc = static_cast<int>(quotient(rel, places(cur.s)));
    const int in = static_cast<int>(rel - static_cast<int64_t>(cur.hc) * places(cur.s));
    cur.unit = in < kItemCost ? 0 : in - kItemCost;
    cur.left = static_cast<int>(stop - start) - (in < kItemCost ? kItemCost - in : 0);
  }
  if (cur.left <= 0) return;

  // ---- the loads: a cursor of their own, the page ids one step ahead
  const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kStage;
  Cursor<kUnit> ld = cur;
  const unsigned S = static_cast<unsigned>(a.kv.S);
  const uint32_t to_v = static_cast<uint32_t>(a.kv.Hkv) * S * C::kRowBytes;  // a page has fewer than 2^32 bytes
  const int32_t P = static_cast<int32_t>(a.kv.P);
  struct Rows {  // a step's, one token each in lanes 0 .. kStep - 1 (16: and again in 16..31)
    unsigned place;  // of the row within its page's keys; bit 0: count the page if it is out of range
    int32_t page;    // -1 also where there is no token
    bool in;
  };
  const int32_t* ld_table = nullptr;  // the item's
  unsigned ld_head = 0;
  auto new_item = [&]() {
    ld_table = a.kv.table + ld.b * a.kv.W;
    ld_head = static_cast<unsigned>(ld.hc) / static_cast<unsigned>(a.chunks) * S * C::kRowBytes;
  };
  new_item();
  auto look_up = [&](Rows& r) {
    const unsigned t = ld.s.first + static_cast<unsigned>(ld.unit) * kUnit + warp * kStep + (lane & (kStep - 1));
    const unsigned j = static_cast<unsigned>((static_cast<uint64_t>(t) * a.div_mul) >> a.div_shift);
    const unsigned at = t - j * S;
    r.in = t < ld.s.end;
    r.place = ld_head + at * C::kRowBytes;
    if (ld.hc == 0 && (at == 0 || t == ld.s.first)) r.place |= 1u;
    r.page = r.in ? ld_table[j] : -1;
    if (ld.next(a, per_seq) && ld.left > 0) new_item();
  };
  auto load = [&](const Rows& x, int stage) {
    const bool ok = static_cast<uint32_t>(x.page) < static_cast<uint32_t>(P);
    if (!ok && x.in && (x.place & 1u) && a.bad != nullptr && lane < kStep) atomicAdd(a.bad, 1);
    // a row that is left out reads nothing: its copies have no bytes
    uint64_t from = reinterpret_cast<uint64_t>(a.kv.kv);
    if (ok) from += static_cast<uint64_t>(static_cast<uint32_t>(x.page)) * (2 * to_v) + (x.place & ~1u);
    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, ok) & kFull;
    if (lane == 0) vmask[warp * C::kStages + stage] = mask;
    const uint32_t base = ring + stage * C::kStage + (lane / C::kLanes) * C::kPitch + (lane % C::kLanes) * 16;
    const auto rows_from = [&](auto whole) {
#pragma unroll
      for (int i = 0; i < C::kRowsPerLane; ++i) {
        const int r = lane / C::kLanes + i * (32 / C::kLanes);
        const uint64_t src = __shfl_sync(0xFFFFFFFFu, from, r) + (lane % C::kLanes) * 16;
        const uint32_t bytes = whole() ? 16u : (mask >> r & 1u) * 16u;
        const uint32_t dst = base + i * (32 / C::kLanes) * C::kPitch;
#pragma unroll
        for (int j = 0; j < C::kChunks; ++j) {
          cp_async16(dst + j * C::kLanes * 16, reinterpret_cast<const void*>(src + j * C::kLanes * 16), bytes);
          cp_async16(dst + C::kSide + j * C::kLanes * 16,
                     reinterpret_cast<const void*>(src + to_v + j * C::kLanes * 16), bytes);
        }
      }
    };
    if (mask == kFull) rows_from([] { return true; });
    else rows_from([] { return false; });
  };
  Rows ahead{};  // the step to load next
  bool have;     // whether there is one
  {
    Rows x[C::kStages - 1];  // the first steps' page ids all at once
    bool got[C::kStages - 1];
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) {
      got[i] = ld.left > 0;
      if (got[i]) look_up(x[i]);
    }
    have = ld.left > 0;
    if (have) look_up(ahead);
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) {
      if (got[i]) load(x[i], i);
      cp_async_commit();
    }
  }

  // ---- the pieces of (sequence, head chunk) items
  int stage = 0;
  while (cur.left > 0) {
    const int h = cur.hc / a.chunks, chunk = cur.hc - h * a.chunks;
    const int hq0 = h * a.G + chunk * 16;
    const int rows = a.G - chunk * 16 < 16 ? a.G - chunk * 16 : 16;
    const int to_end = cur.s.units - cur.unit, units = to_end < cur.left ? to_end : cur.left;
    const bool begins = cur.unit == 0, whole = begins && units == to_end;  // the item's first part, all of it

    // the queries as the MMA's column operand, head 8 j + row in this lane.
    // For an e4m3 cache they are split into two e4m3 numbers behind a power of
    // two that puts the head's largest in [2^7, 2^8): q = q1 + q2 exactly, but
    // for numbers below 2^-9 of the largest, which are off by at most 2^-17 of it
    // (for any finite largest; below 2^-119 the power stays at 2^126)
    uint32_t q1[kTiles][kK][2], q2[kTiles][kE4m3 ? kK : 1][2];
    float scale[kTiles][2];  // of heads 8 j + 2 col, + 1
#pragma unroll
    for (int j = 0; j < kTiles; ++j) {
      const int r = 8 * j + row;
      const uint16_t* qp = a.q + cur.b * a.q_stride + static_cast<int64_t>(hq0 + r) * D;
      if constexpr (!kE4m3) {
#pragma unroll
        for (int k = 0; k < kK; ++k) {
          const uint32_t* p = reinterpret_cast<const uint32_t*>(qp + k * 16 + 2 * col);
          q1[j][k][0] = r < rows ? p[0] : 0u;  // columns 2 col, 2 col + 1
          q1[j][k][1] = r < rows ? p[4] : 0u;  // and 8 further
        }
        scale[j][0] = scale[j][1] = a.scale;
      } else {
        uint2 w[kT];  // 4 columns at 4 col of every 16
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < kT; ++k) {
          w[k] = r < rows ? *reinterpret_cast<const uint2*>(qp + k * 16 + 4 * col) : make_uint2(0u, 0u);
          top = __vmaxu2(top, __vmaxu2(w[k].x & 0x7FFF7FFFu, w[k].y & 0x7FFF7FFFu));
        }
        top = (top >> 16) > (top & 0xFFFFu) ? top >> 16 : top & 0xFFFFu;
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        const bool wrong = top >= 0x7F80u;         // an infinite or NaN query: NaN
        int e = static_cast<int>(top >> 7) - 127;  // the largest is in [2^e, 2^(e + 1))
        e = top == 0 || wrong ? 7 : (e < -119 ? -119 : e);
        const float up = __int_as_float((7 - e + 127) << 23), down = __int_as_float((e - 7 + 127) << 23);
        const float mine = a.scale * a.kv.k_scale[h] * down;
        scale[j][0] = __shfl_sync(0xFFFFFFFFu, mine, 8 * col);
        scale[j][1] = __shfl_sync(0xFFFFFFFFu, mine, 8 * col + 4);
#pragma unroll
        for (int k = 0; k < kT; ++k) {
          uint32_t hi, lo;
          split_e4m3(w[k], up, hi, lo);
          q1[j][k >> 1][k & 1] = wrong ? 0x7F7F7F7Fu : hi;
          q2[j][k >> 1][k & 1] = lo;
        }
      }
    }

    float acc[kTiles][kT][4];  // columns 16 t + row (and + 8) of heads 8 j + 2 col, + 1
    float m[kTiles][2], l[kTiles][2];  // the reference (0 before the first score) and the sum
    float limit[kTiles][2];           // the reference is raised for scores above
#pragma unroll
    for (int j = 0; j < kTiles; ++j) {
#pragma unroll
      for (int t = 0; t < kT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][t][i] = 0.0f;
      m[j][0] = m[j][1] = 0.0f;
      limit[j][0] = limit[j][1] = -CUDART_INF_F;
      l[j][0] = l[j][1] = 0.0f;
    }

    for (int u = 0; u < units; ++u) {
      cp_async_wait<C::kStages - 2>();
      __syncwarp();
      // the stage read in the step before is free again
      if (have) load(ahead, stage == 0 ? C::kStages - 1 : stage - 1);
      cp_async_commit();
      have = ld.left > 0;
      if (have) look_up(ahead);
      const uint32_t mask = vmask[warp * C::kStages + stage];
      const uint32_t kbase = ring + stage * C::kStage, vbase = kbase + C::kSide;
      if (mask != 0) {
        // scores: s[part][j] has tokens row (and + 8) of heads 8 j + 2 col, + 1
        float s[kParts][kTiles][4] = {}, s2[kParts][kTiles][4] = {};  // two chains
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
          // (e4m3: the second 8 rows are tokens 12-15 and 8-11, see the values)
          const int token = kE4m3 ? (lane & 15) ^ ((lane & 8) >> 1) : lane & 15;
          const uint32_t addr = kbase + (part * 16 + token) * C::kPitch + (lane >> 4) * 16;
#pragma unroll
          for (int k = 0; k < kK; ++k) {
            uint32_t b[4];
            ldsm4(addr + k * 32, b);
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
              if constexpr (kE4m3) {
                mma_e4m3(s[part][j], b, q1[j][k]);
                mma_e4m3(s2[part][j], b, q2[j][k]);
              } else {
                mma<false>((k & 1) ? s2[part][j] : s[part][j], b, q1[j][k]);
              }
            }
          }
        }
        bool above = false;
#pragma unroll
        for (int part = 0; part < kParts; ++part)
#pragma unroll
          for (int j = 0; j < kTiles; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float& x = s[part][j][i];
              x = (x + s2[part][j][i]) * scale[j][i & 1];
              const int token = part * 16 + ((i >> 1) == 0 ? row : 8 + (kE4m3 ? row ^ 4 : row));
              if (mask != kFull && ((mask >> token) & 1u) == 0) x = -CUDART_INF_F;
              above |= x > limit[j][i & 1];
            }
        if (__any_sync(0xFFFFFFFFu, above)) {
#pragma unroll
          for (int j = 0; j < kTiles; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float top = fmaxf(s[0][j][i], s[0][j][i + 2]);
              if constexpr (kParts == 2) top = fmaxf(top, fmaxf(s[1][j][i], s[1][j][i + 2]));
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
              const bool raise = top > limit[j][i];
              // (rounded towards each other: no score is more than kSlack + kDown above)
              const float ref = kE4m3 ? __fadd_ru(top, -kDown) : top;
              float shrink = exp2_fast(limit[j][i] == -CUDART_INF_F ? -CUDART_INF_F : m[j][i] - ref);
              shrink = raise ? shrink : 1.0f;
              m[j][i] = raise ? ref : m[j][i];
              limit[j][i] = raise ? __fadd_rd(top, kSlack) : limit[j][i];
              l[j][i] *= shrink;
#pragma unroll
              for (int t = 0; t < kT; ++t) {
                acc[j][t][i] *= shrink;
                acc[j][t][i + 2] *= shrink;
              }
            }
        }
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
          bool tiny = false;
#pragma unroll
          for (int j = 0; j < kTiles; ++j) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float& p = s[part][j][i];
              p = exp2_fast(p - m[j][i & 1]);
              l[j][i & 1] += p;
              tiny |= p < kLeastF16 && p != 0.0f;
            }
          }
          const auto products = [&](auto f16) {
            constexpr bool kF16 = decltype(f16)::value;
            uint32_t hi[kTiles][2], lo[kTiles][2];  // tokens 0-7 and 8-15 of head 8 j + row
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                split_pair<kF16>(s[part][j][2 * i], s[part][j][2 * i + 1], hi[j][i], lo[j][i]);
                hi[j][i] = transpose8(hi[j][i]);
                lo[j][i] = transpose8(lo[j][i]);
              }
            }
            // values, their columns as rows: b[0], b[1] 8 columns each of tokens
            // 0-7, b[2], b[3] of tokens 8-15
            auto accumulate = [&](int t, const uint32_t(&b)[4]) {
#pragma unroll
              for (int j = 0; j < kTiles; ++j) {
                mma<kF16>(acc[j][t], b, hi[j]);
                mma<kF16>(acc[j][t], b, lo[j]);
              }
            };
            if constexpr (!kE4m3) {
              const uint32_t addr = vbase + (part * 16 + (lane & 7) + (lane >> 4) * 8) * C::kPitch + ((lane >> 3) & 1) * 16;
#pragma unroll
              for (int t = 0; t < kT; ++t) {
                uint32_t b[4];
                ldsm4_trans(addr + t * 32, b);
                accumulate(t, b);
              }
            } else {
              // 16 x 16 codes a matrix: a register holds a column's codes of rows 4 col
              // .. 4 col + 3, of which the first two go with weights 2 col, 2 col + 1 of
              // tokens 0-7, the others of 8-15. The rows are the tokens that the
              // weights have there; with 12-15 before 8-11 no 8 rows share a bank. (With
              // 16-bit matrices and byte permutes D = 64 took 4 % longer, 128 2 %.)
              const int at = (lane >> 2 & 3) * 2 + (lane & 1), token = (lane & 2) != 0 ? 8 + (at ^ 4) : at;
              const uint32_t addr = vbase + (part * 16 + token) * C::kPitch + (lane >> 4) * 16;
#pragma unroll
              for (int t = 0; t < kT; t += 2) {
                uint32_t b[4];
                ldsm2_codes(addr + t * 16, b);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  uint32_t c[4];
                  if constexpr (kF16) {
                    widen(b[2 * i], c[0], c[2]);
                    widen(b[2 * i + 1], c[1], c[3]);
                  } else {
                    widen_bf16(b[2 * i], c[0], c[2]);
                    widen_bf16(b[2 * i + 1], c[1], c[3]);
                  }
                  accumulate(t + i, c);
                }
              }
            }
          };
          if (kE4m3 && !__any_sync(0xFFFFFFFFu, tiny)) products(std::true_type{});
          else products(std::false_type{});
        }
      }
      stage = stage + 1 == C::kStages ? 0 : stage + 1;
    }

    // ---- the warps' parts, in their order: each puts its sums where the stage
    // of the step just done lies (the next load into it comes after the
    // barriers), then every thread adds up some columns of all warps
#pragma unroll
    for (int j = 0; j < kTiles; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[j][i] += __shfl_xor_sync(0xFFFFFFFFu, l[j][i], o);
        if (row == 0) {
          // no score yet: nothing, from -inf (but NaN stays)
          ml[(warp * 16 + 8 * j + 2 * col + i) * 2] = limit[j][i] == -CUDART_INF_F ? -CUDART_INF_F : m[j][i];
          ml[(warp * 16 + 8 * j + 2 * col + i) * 2 + 1] = l[j][i];
        }
      }
    const float vs = kE4m3 ? a.kv.v_scale[h] : 1.0f;
    uint8_t* outs = smem + (stage == 0 ? C::kStages - 1 : stage - 1) * C::kStage;
    // a part of several: rows of D sums, then (m, l) of each row; slot 1 for
    // the item's first part, 0 for a continued one
    float* part = a.parts + (static_cast<int64_t>(blockIdx.x) * 2 + begins) * C::kRows * (D + 2);
    __syncwarp();  // all lanes have read the stage
#pragma unroll
    for (int r0 = 0; r0 < C::kRows; r0 += C::kOut) {
      float* mine = reinterpret_cast<float*>(outs + warp * C::kStages * C::kStage);
      if (r0 > 0) __syncthreads();
#pragma unroll
      for (int j = r0 / 8; j < (r0 + C::kOut) / 8; ++j)
#pragma unroll
        for (int t = 0; t < kT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int d = t * 16 + (i >> 1) * 8 + row;
            mine[(8 * j - r0 + 2 * col + (i & 1)) * C::kOPitch + d] = acc[j][t][i];
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
    // to the piece's last unit: next() leaves the item or ends the share
    cur.unit += units - 1;
    cur.left -= units - 1;
    cur.next(a, per_seq);
    __syncthreads();  // the stage may be loaded again
  }
}

// Joins the parts of an item that several shares hold, in their order: a block
// per query head, each thread with 4 columns of every kGroups-th part. It is
// launched with the kernel above and finds its parts before that one has ended;
// what is left after its end is one round of loads.
constexpr int kJoinThreads = 128;

template <int D, bool kE4m3, bool kR16>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const Args a) {
  constexpr int kRows = kR16 ? 16 : 8, kCols = D / 4, kGroups = kJoinThreads / kCols, kBatch = 8;
  constexpr int kUnit = Cfg<D, kE4m3, kR16>::kUnit;
  __shared__ int64_t found[4];  // share, sequence (-1: none), places before it, its places
  __shared__ float4 some[kGroups][kCols];
  __shared__ float2 some_ml[kGroups];
  const int tid = threadIdx.x;
  const int per_seq = static_cast<int>(a.kv.Hkv) * a.chunks;
  // the head of this block, or the end of a share and a row of the item there
  const int64_t at = blockIdx.x / a.per_join;
  const int part = static_cast<int>(blockIdx.x - at * a.per_join);
  if (tid < 32) {
    const Line line = line_of<kUnit>(a, per_seq, a.shares);
    const int64_t place = (at + 1) * line.share;
    if (tid == 0) found[1] = -1;
    __syncwarp();
    if (a.by_cut ? place >= line.before * per_seq && place < line.upto * per_seq : at >= line.b0 && at < line.b1) {
      int64_t before = line.before;
      for (int64_t b = line.b0; b < line.b1; ++b) {
        const int u = places(span_of<kUnit>(a, b));
        if (a.by_cut ? place < (before + u) * per_seq : b == at) {
          found[0] = line.share;
          found[1] = b;
          found[2] = before;
          found[3] = u;
          break;
        }
        before += u;
      }
    }
  }
  __syncthreads();
  const int64_t c = found[0], b = found[1], before = found[2], len = found[3];
  int hc = 0, r = part, hq = part, n = 0;
  int64_t p0 = 0;
  if (b >= 0 && len > 0) {
    if (a.by_cut) {
      hc = static_cast<int>(quotient((at + 1) * c - before * per_seq, len));
    } else {
      const int in = hq % a.G;
      hc = hq / a.G * a.chunks + (in >> 4);
      r = in & 15;
    }
    const int64_t item0 = before * per_seq + hc * len + kItemCost, item1 = item0 + len - kItemCost;
    p0 = quotient(item0, c);
    n = static_cast<int>(quotient(item1 - 1, c) - p0) + 1;
    if (a.by_cut) {
      // an item is joined at the first end of a share inside it
      const int chunk = hc % a.chunks;
      if (p0 != at || r >= a.G - chunk * 16) n = 0;
      hq = hc / a.chunks * a.G + chunk * 16 + r;
    }
  }
  const int g = tid / kCols, d = 4 * (tid - g * kCols);
  cl::griddep_wait();
  if (n <= 1) return;
  float M = -CUDART_INF_F, L = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (g < kGroups) {
    for (int p = g; p < n; p += kBatch * kGroups) {
      float4 v[kBatch];
      float2 ml[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int part = p + i * kGroups < n ? p + i * kGroups : p;
        const float* q = a.parts + ((p0 + part) * 2 + (part == 0)) * kRows * (D + 2);
        v[i] = __ldcg(reinterpret_cast<const float4*>(q + r * D + d));
        ml[i] = __ldcg(reinterpret_cast<const float2*>(q + kRows * D + r * 2));
      }
      float top = M;
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (p + i * kGroups < n) top = fmaxf(top, ml[i].x);
      const float base = top == -CUDART_INF_F ? 0.0f : top, shrink = exp2_fast(M - base);
      M = top;
      L *= shrink;
      o.x *= shrink;
      o.y *= shrink;
      o.z *= shrink;
      o.w *= shrink;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (p + i * kGroups >= n) continue;
        const float f = exp2_fast(ml[i].x - base);
        L += ml[i].y * f;
        o.x += v[i].x * f;
        o.y += v[i].y * f;
        o.z += v[i].z * f;
        o.w += v[i].w * f;
      }
    }
    some[g][d / 4] = o;
    if (d == 0) some_ml[g] = make_float2(M, L);
  }
  __syncthreads();
  if (tid < kCols) {
    M = some_ml[0].x;
#pragma unroll
    for (int i = 1; i < kGroups; ++i) M = fmaxf(M, some_ml[i].x);
    const float base = M == -CUDART_INF_F ? 0.0f : M;
    L = 0.0f;
    o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const float f = exp2_fast(some_ml[i].x - base);
      const float4 v = some[i][tid];
      L += some_ml[i].y * f;
      o.x += v.x * f;
      o.y += v.y * f;
      o.z += v.z * f;
      o.w += v.w * f;
    }
    put<D>(a, b, hq, 4 * tid, o, M, L, kE4m3 ? a.kv.v_scale[hq / a.G] : 1.0f);
  }
}

template <int D, bool kE4m3, bool kR16>
cudaError_t launch(const Ctx& c, Args a) {
  using C = Cfg<D, kE4m3, kR16>;
  static SmemLimit lim;
  cudaError_t e = raise_smem_limit(lim, attn_kernel<D, kE4m3, kR16>, c.device, C::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t cap = a.kv.W * a.kv.S, most = a.window > 0 && a.window < cap ? a.window : cap;
  const int64_t items = a.kv.B * a.kv.Hkv * a.chunks, units = (most + C::kUnit - 1) / C::kUnit;
  int64_t grid = C::kBlocksPerSm * c.sm_count;
  if (grid > max_shares(D, kE4m3, kR16)) grid = max_shares(D, kE4m3, kR16);
  // A block per item, nothing cut, where no item can be longer than a least share,
  // or than 1024 tokens with an item for every block: 256 sequences of 1000, 8 key
  // heads of D = 128: 159 us (171 in shares), 64 of 1 to 300: 12 (17); 64 of 1000,
  // 512 items for 456 blocks, 56 (52). One item's 1024 tokens are about 12 us.
  a.direct = (units <= least_units(C::kUnit) || (most <= 1024 && items >= grid)) && items <= kMaxDim;
  if (a.direct) grid = items;
  else if (items < grid && items * units < grid) grid = items * units;
  a.shares = static_cast<int>(grid);
  e = launch_early(c, grid, C::kThreads, C::kSmem, attn_kernel<D, kE4m3, kR16>, a);
  if (e != cudaSuccess || a.direct) return e;
  const int64_t heads = a.kv.B * a.Hq, rows = a.G < 16 ? a.G : 16, cuts = (grid - 1) * rows;
  a.by_cut = cuts < heads;
  a.per_join = static_cast<int>(a.by_cut ? rows : a.Hq);
  if (cuts == 0) return cudaSuccess;  // one share
  return launch_early(c, a.by_cut ? cuts : heads, kJoinThreads, 0, join_kernel<D, kE4m3, kR16>, a);
}

template <int D>
cudaError_t launch_d(const Ctx& c, const Args& a) {
  const bool e4m3 = a.kv.type == WQ_KV_E4M3, r16 = a.G > 8;
  if (e4m3) return r16 ? launch<D, true, true>(c, a) : launch<D, true, false>(c, a);
  return r16 ? launch<D, false, true>(c, a) : launch<D, false, false>(c, a);
}

}  // namespace

size_t kv_attn_ws_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t D) {
  const bool r16 = Hq / Hkv > 8;
  const int rows = r16 ? 16 : 8, x = max_shares(D, true, r16), y = max_shares(D, false, r16), shares = x > y ? x : y;
  (void)B;
  return static_cast<size_t>(shares) * 2 * rows * (D + 2) * 4;  // two parts for each share
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
