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

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStep = 16;               // tokens a warp takes at a time
constexpr int kUnit = kStep * kWarps;   // tokens a block takes at a time
// A (sequence, head) of at most this many units is not cut: a join costs
// about as much as four units in a row.
constexpr int kMinShare = 4;
constexpr int kMaxBlocks = 512;         // shares (the partial results' space)

// Row base of a head chunk: at most 16 query heads of one key head.
template <int D, bool kE4m3, bool kR16>
struct Cfg {
  static constexpr int kRows = kR16 ? 16 : 8;
  static constexpr int kRowBytes = D * (kE4m3 ? 1 : 2);
  static constexpr int kPitch = kRowBytes + 16;  // an odd number of 16-byte words: ldmatrix without conflicts
  static constexpr int kSide = kStep * kPitch;   // a step's keys (or values)
  static constexpr int kStage = 2 * kSide;
  static constexpr int kOPitch = D + 8;          // floats
  static constexpr int kOBuf = kRows * kOPitch * 4;
  static constexpr int kMisc = 1024;
  static constexpr int kFixed = 2 * kOBuf + kMisc;
  static constexpr int kFit2 = (113 * 1024 - kFixed) / (kWarps * kStage);
  static constexpr int kFit1 = (226 * 1024 - kFixed) / (kWarps * kStage);
  static constexpr int kBlocksPerSm = kFit2 >= 3 ? 2 : 1;
  static constexpr int kFit = kBlocksPerSm == 2 ? kFit2 : kFit1;
  static constexpr int kStages = kFit < 6 ? kFit : 6;
  static constexpr int kSmem = kFixed + kWarps * kStages * kStage;
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
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (kF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    mma_bf16_16816(c, a0, a1, a2, a3, b0, b1);
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

// A place in the line of units: unit `unit` of head chunk `hc` of sequence b.
struct Cursor {
  int64_t b;
  int hc, unit;
  Span s;
  __device__ void next(const Args& a, int per_seq) {
    if (++unit < s.units) return;
    unit = 0;
    if (++hc < per_seq) return;
    hc = 0;
    do {
      if (++b >= a.kv.B) return;
      s = span_of(a, b);
    } while (s.units == 0);
  }
};

template <int D, bool kE4m3, bool kR16>
__global__ void __launch_bounds__(kThreads) attn_kernel(const Args a) {
  using C = Cfg<D, kE4m3, kR16>;
  constexpr int kK = D / 16, kN = D / 8;
  extern __shared__ __align__(128) uint8_t smem[];
  float* obuf = reinterpret_cast<float*>(smem + kWarps * C::kStages * C::kStage);
  float* ml = obuf + 2 * C::kOBuf / 4;                                  // [kWarps][16][2]
  uint32_t* vmask = reinterpret_cast<uint32_t*>(ml + kWarps * 16 * 2);  // [kWarps][kStages]
  int64_t* share = reinterpret_cast<int64_t*>(vmask + 32);              // [0] share, [1] b, [2] units before b
  unsigned* last = reinterpret_cast<unsigned*>(share + 4);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = lane >> 2, col = lane & 3;
  const int per_seq = static_cast<int>(a.kv.Hkv) * a.chunks;

  if (warp == 1) {  // sequences without tokens
    for (int64_t b = blockIdx.x; b < a.kv.B; b += gridDim.x) {
      if (span_of(a, b).units != 0) continue;
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
      const int u = span_of(a, b).units;
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
    const int least = most < kMinShare ? most : kMinShare;
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
        const int u = span_of(a, b).units;
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
  Cursor cur;
  cur.b = share[1];
  cur.s = span_of(a, cur.b);
  int64_t before = share[2] * per_seq;  // units before sequence cur.b
  cur.hc = static_cast<int>((start - before) / cur.s.units);
  cur.unit = static_cast<int>((start - before) % cur.s.units);

  // ---- the loads: a cursor of their own, the page ids one step ahead
  const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kStage;
  Cursor ld = cur;
  int64_t to_load = stop - start;
  const unsigned S = static_cast<unsigned>(a.kv.S);
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
    const int h = ld.hc / a.chunks;
    const bool ok = ld_in && ld_page >= 0 && ld_page < a.kv.P;
    if (ld_in && !ok && a.bad != nullptr && ld.hc == 0 && lane < 16 &&
        (ld_slot == 0 || (ld.unit == 0 && warp == 0 && lane == 0)))
      atomicAdd(a.bad, 1);
    int64_t off = -1;
    if (ok) off = ((static_cast<int64_t>(ld_page) * 2 * a.kv.Hkv + h) * a.kv.S + ld_slot) * C::kRowBytes;
    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, ok) & 0xFFFFu;
    if (lane == 0) vmask[warp * C::kStages + stage] = mask;
    const uint32_t base = ring + stage * C::kStage;
    const int64_t to_v = a.kv.Hkv * a.kv.S * C::kRowBytes;
    const uint8_t* kv = static_cast<const uint8_t*>(a.kv.kv);
#pragma unroll
    for (int i = 0; i < C::kRowsPerLane; ++i) {
      const int r = lane / C::kLanes + i * (32 / C::kLanes);
      const int64_t o = __shfl_sync(0xFFFFFFFFu, off, r);
      const uint32_t bytes = o >= 0 ? 16u : 0u;
      const uint8_t* src = kv + (o >= 0 ? o : 0) + (lane % C::kLanes) * 16;
      const uint32_t dst = base + r * C::kPitch + (lane % C::kLanes) * 16;
      const int64_t v = o >= 0 ? to_v : 0;
#pragma unroll
      for (int j = 0; j < C::kChunks; ++j) {
        cp_async16(dst + j * C::kLanes * 16, src + j * C::kLanes * 16, bytes);
        cp_async16(dst + C::kSide + j * C::kLanes * 16, src + v + j * C::kLanes * 16, bytes);
      }
    }
    ld.next(a, per_seq);
    --to_load;
    if (to_load > 0) look_up();
  };
  look_up();
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) {
    if (to_load > 0) load(i);
    cp_async_commit();
  }

  // ---- the pieces of (sequence, head chunk) items
  int64_t done = start;
  int stage = 0;
  while (done < stop) {
    const int h = cur.hc / a.chunks, chunk = cur.hc - h * a.chunks;
    const int hq0 = h * a.G + chunk * 16;
    const int rows = a.G - chunk * 16 < 16 ? a.G - chunk * 16 : 16;
    const int64_t item0 = before + static_cast<int64_t>(cur.hc) * cur.s.units, item1 = item0 + cur.s.units;
    const int units = static_cast<int>((item1 < stop ? item1 : stop) - done);

    // the queries as the MMA's row operand; e4m3: in fp16 behind a power of
    // two that puts the row's largest at 2^13 (exact but for numbers below
    // 2^-38 of it)
    uint32_t qa[kK][kR16 ? 4 : 2];
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
            qa[k][half] = in ? p[0] : 0u;                      // columns 2 col, 2 col + 1
            qa[k][half + (kR16 ? 2 : 1)] = in ? p[4] : 0u;     // and 8 further
          }
        } else {
          // columns 4 col .. 4 col + 3 of each 16: the order in which a row of
          // codes comes out of ldmatrix
          uint32_t top = 0;
#pragma unroll
          for (int k = 0; k < kK; ++k) {
            const uint2 w = in ? *reinterpret_cast<const uint2*>(qp + r * D + k * 16 + 4 * col) : make_uint2(0u, 0u);
            qa[k][half] = w.x;
            qa[k][half + (kR16 ? 2 : 1)] = w.y;
            const uint32_t m1 = __vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu);
            top = __vmaxu2(top, m1);
          }
          top = (top >> 16) > (top & 0xFFFFu) ? top >> 16 : top & 0xFFFFu;
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
          int e = static_cast<int>(top >> 7) - 127;  // the largest is in [2^e, 2^(e + 1))
          if (top == 0 || top >= 0x7F80u) e = 13;
          e = 13 - e < -100 ? 113 : (13 - e > 100 ? -87 : e);
          const float up = __int_as_float((13 - e + 127) << 23), down = __int_as_float((e - 13 + 127) << 23);
          scale[half] = a.scale * a.kv.k_scale[h] * down;
#pragma unroll
          for (int k = 0; k < kK; ++k)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t w = qa[k][half + j * (kR16 ? 2 : 1)];
              const __half2 f = __floats2half2_rn(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xFFFF0000u) * up);
              qa[k][half + j * (kR16 ? 2 : 1)] = *reinterpret_cast<const uint32_t*>(&f);
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
      if (to_load > 0) load(stage == 0 ? C::kStages - 1 : stage - 1);
      cp_async_commit();
      const uint32_t mask = vmask[warp * C::kStages + stage];
      const uint32_t kbase = ring + stage * C::kStage, vbase = kbase + C::kSide;
      if (mask != 0) {
        // scores of 16 tokens: s[j] has tokens 8 j + 2 col, + 1 of rows `row` and row + 8
        float s[2][4] = {};
        if constexpr (!kE4m3) {
          const uint32_t addr = kbase + ((lane & 7) + (lane >> 4) * 8) * C::kPitch + ((lane >> 3) & 1) * 16;
#pragma unroll
          for (int k = 0; k < kK; ++k) {
            uint32_t b[4];
            ldsm4(addr + k * 32, b);
            if constexpr (kR16) {
              mma<false>(s[0], qa[k][0], qa[k][1], qa[k][2], qa[k][3], b[0], b[1]);
              mma<false>(s[1], qa[k][0], qa[k][1], qa[k][2], qa[k][3], b[2], b[3]);
            } else {
              mma<false>(s[0], qa[k][0], 0u, qa[k][1], 0u, b[0], b[1]);
              mma<false>(s[1], qa[k][0], 0u, qa[k][1], 0u, b[2], b[3]);
            }
          }
        } else {
          const uint32_t addr = kbase + (lane & 15) * C::kPitch + (lane >> 4) * 16;
#pragma unroll
          for (int k2 = 0; k2 < kK / 2; ++k2) {
            uint32_t b[4];  // 16 columns of tokens 0-7, 8-15, then the next 16 columns
            ldsm4(addr + k2 * 32, b);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int k = 2 * k2 + (j >> 1);
              const uint32_t b0 = widen(b[j], false), b1 = widen(b[j], true);
              if constexpr (kR16) mma<true>(s[j & 1], qa[k][0], qa[k][1], qa[k][2], qa[k][3], b0, b1);
              else mma<true>(s[j & 1], qa[k][0], 0u, qa[k][1], 0u, b0, b1);
            }
          }
        }
        float top[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < (kR16 ? 4 : 2); ++i) {
            s[j][i] *= scale[i >> 1];
            if (((mask >> (8 * j + 2 * col + (i & 1))) & 1u) == 0) s[j][i] = -CUDART_INF_F;
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
            mma<kE4m3>(acc[n], hi[0][0], hi[0][1], hi[1][0], hi[1][1], b0, b1);
            mma<kE4m3>(acc[n], lo[0][0], lo[0][1], lo[1][0], lo[1][1], b0, b1);
          } else {
            mma<kE4m3>(acc[n], hi[0][0], lo[0][0], hi[1][0], lo[1][0], b0, b1);
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
      cur.unit++;
    }
    done += units;

    // ---- the four warps' parts, in their order
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
    __syncthreads();
    float mm[2], ll[2];
#pragma unroll
    for (int i = 0; i < (kR16 ? 2 : 1); ++i) {
      const float* p = ml + (row + 8 * i) * 2;
      mm[i] = p[0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) mm[i] = fmaxf(mm[i], p[w * 32]);
      const float base = mm[i] == -CUDART_INF_F ? 0.0f : mm[i];
      ll[i] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) ll[i] += p[w * 32 + 1] * exp2_fast(p[w * 32] - base);
      const float f = exp2_fast(m[i] - base);
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        acc[n][2 * i] *= f;
        acc[n][2 * i + 1] *= f;
      }
    }
    auto exchange = [&](int buf, bool store) {
#pragma unroll
      for (int i = 0; i < (kR16 ? 2 : 1); ++i)
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          float2* p = reinterpret_cast<float2*>(obuf + buf * (C::kOBuf / 4) + (row + 8 * i) * C::kOPitch + 8 * n + 2 * col);
          if (store) {
            *p = make_float2(acc[n][2 * i], acc[n][2 * i + 1]);
          } else {
            const float2 v = *p;
            acc[n][2 * i] += v.x;
            acc[n][2 * i + 1] += v.y;
          }
        }
    };
    if (warp >= 2) exchange(warp - 2, true);
    __syncthreads();
    if (warp < 2) exchange(warp, false);
    if (warp == 1) exchange(1, true);
    __syncthreads();
    const bool whole = item0 >= start && item1 <= stop;
    // column of acc[n][2 i + e]: e4m3 tiles hold the even or the odd columns
    auto column = [&](int n, int e) { return kE4m3 ? (n >> 1) * 16 + 2 * (2 * col + e) + (n & 1) : 8 * n + 2 * col + e; };
    const float vs = kE4m3 ? a.kv.v_scale[h] : 1.0f;
    if (warp == 0) {
      exchange(1, false);
      if (whole) {
#pragma unroll
        for (int i = 0; i < (kR16 ? 2 : 1); ++i) {
          const int r = row + 8 * i;
          if (r >= rows) continue;
          const float f = ll[i] == 0.0f ? 0.0f : vs / ll[i];
          uint16_t* o = a.out + (cur.b * a.Hq + hq0 + r) * D;
          if constexpr (!kE4m3) {
#pragma unroll
            for (int n = 0; n < kN; ++n) {
              const __nv_bfloat162 v = __floats2bfloat162_rn(acc[n][2 * i] * f, acc[n][2 * i + 1] * f);
              *reinterpret_cast<__nv_bfloat162*>(o + 8 * n + 2 * col) = v;
            }
          } else {
#pragma unroll
            for (int n = 0; n < kN; n += 2) {
              const __nv_bfloat162 v0 = __floats2bfloat162_rn(acc[n][2 * i] * f, acc[n + 1][2 * i] * f);
              const __nv_bfloat162 v1 = __floats2bfloat162_rn(acc[n][2 * i + 1] * f, acc[n + 1][2 * i + 1] * f);
              *reinterpret_cast<uint2*>(o + column(n, 0)) = make_uint2(*reinterpret_cast<const uint32_t*>(&v0),
                                                                      *reinterpret_cast<const uint32_t*>(&v1));
            }
          }
          if (a.lse != nullptr && col == 0)
            a.lse[cur.b * a.Hq + hq0 + r] = ll[i] == 0.0f ? -CUDART_INF_F : (mm[i] + log2f(ll[i])) * 0.6931471805599453f;
        }
      } else {
        // one part of several: rows of D + 2 floats (o, m, l); slot 1 for the
        // item's first part, 0 for a continued one
        float* part = a.parts + (static_cast<int64_t>(blockIdx.x) * 2 + (item0 >= start)) * C::kRows * (D + 2);
#pragma unroll
        for (int i = 0; i < (kR16 ? 2 : 1); ++i) {
          const int r = row + 8 * i;
          if (r >= rows) continue;
#pragma unroll
          for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) part[r * (D + 2) + column(n, e)] = acc[n][2 * i + e];
          if (col == 0) {
            part[r * (D + 2) + D] = mm[i];
            part[r * (D + 2) + D + 1] = ll[i];
          }
        }
        __threadfence();
        __syncwarp();
        if (lane == 0) {
          const int64_t p0 = item0 / c, n_parts = (item1 - 1) / c - p0 + 1;
          unsigned* count = a.arrived + cur.b * per_seq + cur.hc;
          const bool is_last = atom_add_acq_rel_gpu(count, 1u) == static_cast<unsigned>(n_parts - 1);
          if (is_last) *count = 0;  // nobody else will: all parts are here
          *last = is_last;
        }
      }
    }
    if (!whole) {
      __syncthreads();
      if (*last) {
        __threadfence();
        const int64_t p0 = item0 / c, p1 = (item1 - 1) / c;
        for (int i = tid; i < rows * (D / 2); i += kThreads) {
          const int r = i / (D / 2), d = 2 * (i - r * (D / 2));
          float M = -CUDART_INF_F, L = 0.0f;
          float2 o = make_float2(0.0f, 0.0f);
#pragma unroll 4
          for (int64_t p = p0; p <= p1; ++p) {
            const float* part = a.parts + (p * 2 + (p == p0)) * C::kRows * (D + 2) + r * (D + 2);
            const float2 v = __ldcg(reinterpret_cast<const float2*>(part + d));
            const float2 s = __ldcg(reinterpret_cast<const float2*>(part + D));
            const float M2 = fmaxf(M, s.x), base = M2 == -CUDART_INF_F ? 0.0f : M2;
            const float f = exp2_fast(M - base), g = exp2_fast(s.x - base);
            M = M2;
            L = L * f + s.y * g;
            o.x = o.x * f + v.x * g;
            o.y = o.y * f + v.y * g;
          }
          const float f = L == 0.0f ? 0.0f : vs / L;
          *reinterpret_cast<__nv_bfloat162*>(a.out + (cur.b * a.Hq + hq0 + r) * D + d) =
              __floats2bfloat162_rn(o.x * f, o.y * f);
          if (a.lse != nullptr && d == 0)
            a.lse[cur.b * a.Hq + hq0 + r] = L == 0.0f ? -CUDART_INF_F : (M + log2f(L)) * 0.6931471805599453f;
        }
      }
    }
    // the next item
    cur.unit--;
    const int64_t b = cur.b;
    const int64_t units_b = static_cast<int64_t>(cur.s.units) * per_seq;
    cur.next(a, per_seq);
    if (cur.b != b) before += units_b;
  }
}

template <int D, bool kE4m3, bool kR16>
cudaError_t launch(const Ctx& c, const Args& a) {
  using C = Cfg<D, kE4m3, kR16>;
  static SmemLimit lim;
  cudaError_t e = raise_smem_limit(lim, attn_kernel<D, kE4m3, kR16>, c.device, C::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t cap = a.kv.W * a.kv.S, most = a.window > 0 && a.window < cap ? a.window : cap;
  const int64_t items = a.kv.B * a.kv.Hkv * a.chunks, units = (most + kUnit - 1) / kUnit;
  int64_t grid = static_cast<int64_t>(C::kBlocksPerSm) * c.sm_count;
  if (grid > kMaxBlocks) grid = kMaxBlocks;
  if (items < grid && items * units < grid) grid = items * units;
  attn_kernel<D, kE4m3, kR16><<<static_cast<unsigned>(grid), kThreads, C::kSmem, c.stream>>>(a);
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
