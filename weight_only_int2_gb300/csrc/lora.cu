// Low-rank adapters beside a shared projection: row m of y is
//   base[m] + scale[a] (x[m] A[a]^T) B[a]^T,   a = adapter[m],
// and base[m] for a row without an adapter.
//
// Two products, with the rows grouped by adapter into tiles, so that every A and B is
// read by few blocks (up to 128 rows each block groups them itself, more are grouped
// by a launch before, group.cu). x A^T stays as two bf16 numbers a value on its way
// into the second product (2^-16 of itself; one would cost the sum bf16's 2^-8 once
// more), whose float32 sums begin with base or have it added at their end (on tcgen05),
// and are rounded once, to y.
//  - The first contracts over K: a block takes a tile and a share of K, as many shares
//    as it takes to fill the GPU (a rule on the number of tiles, which is on the
//    device), and writes float32 partial sums.
//  - The second adds them up in their order and scales (for larger ranks of many rows a
//    launch between the two does), and takes a tile and some of the columns; base and y
//    are read and written 16 bytes a thread: the columns of four MMAs are dealt out so
//    that a thread holds 8 in a row.
//
// Bound: HBM, where there is enough to read. 8192 rows, K 5120, N 17408, r 16, 658 MB:
// 115 us, 5.7 TB/s (the second product 91 us of it; three blocks an SM instead of two
// 145, since more places in base and y are open at once); r 64 144 us and r 128 171, both
// products by tcgen05 there. 64 rows of 41 adapters, 40 MB: 14.2 us, the chain rows ->
// order -> A, x -> sums -> B, twice a launch. One row: 4.8 us.
#include "wq_cluster.cuh"
#include "wq_device.cuh"
#include "wq_internal.h"
#include "wq_tc.cuh"

#include <cuda_bf16.h>

#include <algorithm>

namespace wq {
namespace {

constexpr int kThreads = 128;    // of a block of the first product
constexpr int kWarps = kThreads / 32;
constexpr int kMaxShares = 32;
constexpr int kMaxGrid = 1024;   // blocks of the first product

// Rows of a tile. A decode batch has a few rows of each adapter: they are the 8
// columns of an MMA, and A's or B's values its 16 rows. From kManyRows rows on tiles
// are 64 rows, 16 a warp, and A's or B's values the columns. (512 rows, tiles of 8 and of
// 64: r 16, 5 adapters 21.3 and 19.4 us; r 64, 5 adapters 25.8 and 20.3, 60 adapters 33.2
// and 36.0; r 128, 5 adapters 38.7 and 24.0; r 16, 60 adapters 17.7 and 23.1.)
constexpr int64_t kManyRows = 512;
constexpr int kFewTile = 8;
constexpr int tile_of(int64_t M) { return M < kManyRows ? kFewTile : 64; }
// Up to so many rows every block groups them itself, one a thread.
constexpr int64_t kFewRows = kThreads;

struct Ws {
  int4* tiles;     // as launch_group writes them
  int32_t* order;  // [M] the row at each place
  float* part;     // [shares][rows with an adapter][r]
  uint4* low;      // many rows: x A^T as the second product's MMAs read it, [tiles][r / 64][128][8]
};
int64_t most_tiles(int64_t M, int64_t n) { return M / tile_of(M) + std::min(M, n + 1); }
size_t part_bytes(int64_t M, int64_t r) {
  // shares * rows <= max(rows, blocks * tile), and shares <= kMaxShares
  return static_cast<size_t>(std::max(M, std::min(kMaxShares * M, int64_t{kMaxGrid} * tile_of(M)))) * r * 4;
}
size_t round16(size_t b) { return (b + 15) / 16 * 16; }
// r as the kernels have it.
constexpr int rank_of(int64_t r) { return r <= 16 ? 16 : (r <= 32 ? 32 : (r <= 64 ? 64 : 128)); }
// Whether a kernel of its own adds up the shares of many rows (below).
constexpr bool joined(int64_t r) { return r > 32; }
size_t low_bytes(int64_t M, int64_t n, int64_t r) {
  return tile_of(M) == 64 && joined(r) ? static_cast<size_t>(most_tiles(M, n)) * 64 * rank_of(r) * 4 : 0;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  const int size = real ? 16 : 0;  // 0: zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&d)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
               : "r"(addr)
               : "memory");
}

// How K is shared among blocks: `shares` of `per` stages each. (Shares are added up a
// few at a time: beyond 16 they have four stages at least.)
struct Shares {
  int shares, per;
};
__device__ __forceinline__ Shares shares_of(int stages, int tiles, int grid) {
  int s = tiles > 0 ? grid / tiles : 1;
  s = max(1, min(min(s, kMaxShares), min(stages, max(16, stages / 4))));
  const int per = (stages + s - 1) / s;
  return Shares{(stages + per - 1) / per, per};
}

// ---------------------------------------------------------------- rows by adapter

// What both products know of the rows' order: as launch_group wrote it, or of few
// rows in shared memory, found by the block itself (a launch less).
struct Few {
  int key[kFewRows];      // (adapter, row) by row
  int id[kFewRows + 1];   // adapters by place; id[0]: none
  int32_t order[kFewRows];
  int4 tiles[1 + kFewRows];
};
struct Rows {
  const int4* tiles;
  const int32_t* order;
  // (past the first level cache, as all that is read before the wait: nothing says that it holds no earlier call's)
  __device__ int4 tile(int i) const { return __ldcg(tiles + i); }
  __device__ int row(int i) const { return __ldcg(order + i); }
};
struct FewRows {
  const Few* f;
  __device__ int4 tile(int i) const { return f->tiles[i]; }
  __device__ int row(int i) const { return f->order[i]; }
};
// Every thread has a row, whose place is the number of rows before it by (adapter,
// row); then it has the place with its number, and a tile begins at the places 0, 8,
// 16 .. of a group.
__device__ __forceinline__ void group_few(Few& f, const int32_t* ids, int M, int n) {
  static_assert(kFewRows == kThreads && kMaxGroups < (1 << 24), "a row a thread");
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
  int id = i < M ? __ldcg(ids + i) : 0x7FFFFF;
  if (i < M && (id < 0 || id >= n)) id = n;
  const int key = id << 7 | i;
  f.key[i] = key;
  if (i == 0) f.id[0] = -1;
  __syncthreads();
  int place = i;
  if (32 * warp < M) {
    place = 0;
#pragma unroll 4
    for (int j = 0; j < M; j += 4) {
      const int4 k = *reinterpret_cast<const int4*>(f.key + j);
      place += (k.x < key) + (k.y < key) + (k.z < key) + (k.w < key);
    }
  }
  f.id[1 + place] = id;
  f.order[place] = i;
  __syncthreads();
  // the groups' first places as bits, then the tiles'
  uint32_t first[kFewRows / 32], begin[kFewRows / 32];
  int rows = 0, tiles = 0, inside = 0;
#pragma unroll
  for (int w = 0; w < kFewRows / 32; ++w) {
    const int at = f.id[1 + 32 * w + lane], p = 32 * w + lane;
    first[w] = __ballot_sync(0xFFFFFFFFu, p < M && at != f.id[p]);
    const uint32_t have = __ballot_sync(0xFFFFFFFFu, p < M && at < n);
    int start = 0;  // place p's group's
#pragma unroll
    for (int v = 0; v <= w; ++v) {
      const uint32_t m = v < w ? first[v] : first[v] & (0xFFFFFFFFu >> (31 - lane));
      if (m != 0) start = 32 * v + 31 - __clz(m);
    }
    begin[w] = __ballot_sync(0xFFFFFFFFu, p < M && (p - start) % kFewTile == 0);
    rows += __popc(have);
    inside += __popc(begin[w] & have);
    if (w == warp && (begin[w] >> lane & 1) != 0) {
      const int t = tiles + __popc(begin[w] & ((1u << lane) - 1));
      int end = p + 1;
      while (end < M && end < p + kFewTile && f.id[1 + end] == at) ++end;
      f.tiles[1 + t] = make_int4(at < n ? at : -1, p, end - p, 0);
    }
    tiles += __popc(begin[w]);
  }
  if (i == 0) f.tiles[0] = make_int4(inside, tiles, rows, 0);
  __syncthreads();
}

// ---------------------------------------------------------------- x A^T

// Tiles of 8 rows. Few rows use A: a lane copies what it needs itself in the MMA's
// layout (16 bytes are 8 values of K in a row, dealt out alike on x's side) into its
// own places of a ring of stages of 32 of K, so that nothing waits for another lane.
// The block's four warps take 128 of K in turn along its share and are added up at
// its end.
template <int kR>
struct Shrink8 {
  static constexpr int kCols = 512;  // of a stage of the shares: four warps' 128
  static constexpr int kStages = kR == 128 ? 3 : 4;
  static constexpr int kStageBytes = (kR / 8 + 1) * 512;
  static constexpr int kSums = kWarps * 8 * kR * 4;
  static constexpr int kSmem = kWarps * kStages * kStageBytes;
  static constexpr int kAll = kSmem + kSums + static_cast<int>(sizeof(Few)) + 1024;
  static constexpr int kFit = 228 * 1024 / kAll < 4 ? 228 * 1024 / kAll : 4;
};

template <int kR, bool kFew>
__global__ void __launch_bounds__(kThreads, Shrink8<kR>::kFit) shrink8_kernel(const LoraArgs a, const Ws ws) {
  using C = Shrink8<kR>;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float sums[kWarps][8 * kR];
  cl::griddep_wait();
  cl::griddep_launch_dependents();
  const auto rows = [&] {
    if constexpr (kFew) {
      __shared__ Few few;
      group_few(few, a.adapter, static_cast<int>(a.M), static_cast<int>(a.n));
      return FewRows{&few};
    } else {
      return Rows{ws.tiles, ws.order};
    }
  }();
  const int4 head = rows.tile(0);
  const int K = static_cast<int>(a.K), r = static_cast<int>(a.r), stages = (K - 1) / C::kCols + 1;
  const Shares sh = shares_of(stages, head.x, gridDim.x);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const uint8_t* own = ring + warp * C::kStages * C::kStageBytes + lane * 16;
  const uint32_t own_at = smem_u32(own);
  const int units = head.x * sh.shares;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int t = u / sh.shares, share = u - t * sh.shares;
    const int4 tile = rows.tile(1 + t);
    const bool mine = g < tile.z;
    const uint16_t* x = a.x + (mine ? rows.row(tile.y + g) : 0) * a.x_stride;
    const uint16_t* A = a.A + (static_cast<int64_t>(tile.x) * r + g) * K;
    const int k0 = share * sh.per * C::kCols + warp * 128 + q * 8;  // (stages end below 2^31 + 2^9)
    const int blocks = 4 * (min(sh.per * (share + 1), stages) - share * sh.per);
    auto fetch = [&](int b, uint32_t slot) {
      const int k = k0 + (b >> 2) * C::kCols + (b & 3) * 32;
      const bool in = k >= 0 && k < K;
      const uint16_t* src = A + k;
#pragma unroll
      for (int n = 0; n < kR / 8; ++n) {
        const bool real = in && 8 * n < r;
        cp_async16(own_at + slot + n * 512, real ? src : a.A, real);
        src += static_cast<int64_t>(8) * K;
      }
      cp_async16(own_at + slot + (kR / 8) * 512, in && mine ? x + k : a.x, in && mine);
    };
#pragma unroll
    for (int b = 0; b < C::kStages - 1; ++b) {
      if (b < blocks) fetch(b, b * C::kStageBytes);
      cp_commit();
    }
    float acc[kR / 16][4] = {};
    uint32_t slot = 0, ahead = (C::kStages - 1) * C::kStageBytes;
#pragma unroll 1
    for (int b = 0; b < blocks; ++b) {
      if (b + C::kStages - 1 < blocks) fetch(b + C::kStages - 1, ahead);
      cp_commit();
      cp_wait<C::kStages - 1>();
      const uint4 xv = *reinterpret_cast<const uint4*>(own + slot + (kR / 8) * 512);
#pragma unroll
      for (int n = 0; n < kR / 16; ++n) {
        const uint4 lo = *reinterpret_cast<const uint4*>(own + slot + (2 * n) * 512);
        const uint4 hi = *reinterpret_cast<const uint4*>(own + slot + (2 * n + 1) * 512);
        mma_bf16_16816(acc[n], lo.x, hi.x, lo.y, hi.y, xv.x, xv.y);
        mma_bf16_16816(acc[n], lo.z, hi.z, lo.w, hi.w, xv.z, xv.w);
      }
      ahead = slot;
      slot = slot + C::kStageBytes == C::kStages * C::kStageBytes ? 0 : slot + C::kStageBytes;
    }
#pragma unroll
    for (int n = 0; n < kR / 16; ++n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) sums[warp][(2 * q + (i & 1)) * kR + 16 * n + g + 8 * (i >> 1)] = acc[n][i];
    }
    __syncthreads();
    float* part = ws.part + (static_cast<int64_t>(share) * head.z + tile.y) * r;
    for (int i = threadIdx.x; i < tile.z * kR; i += kThreads) {
      const int row = i / kR, col = i % kR;
      const float s = (sums[0][i] + sums[1][i]) + (sums[2][i] + sums[3][i]);
      if (col < r) part[row * r + col] = s;
    }
    __syncthreads();
  }
}

// Tiles of 64 rows: a ring of cp.async stages of x's rows and A's.
template <int kR>
struct Shrink64 {
  static constexpr int kCols = 64;  // of a stage
  static constexpr int kRowBytes = 2 * kCols;
  static constexpr int kChunks = kRowBytes / 16;
  static constexpr int kStages = kR == 128 ? 4 : 6;
  static constexpr int kStageBytes = (64 + kR) * kRowBytes;
  static constexpr int kSmem = kStages * kStageBytes + (joined(kR) ? 1024 : 0);
  static constexpr int kStep = kThreads / kChunks;  // rows that the block copies at once
  static constexpr int kXs = 64 / kStep;            // rows of x a thread copies
  static constexpr int kAs = kR / kStep;            // and of A
};

template <int kR>
__global__ void __launch_bounds__(kThreads) shrink64_kernel(const LoraArgs a, const Ws ws) {
  using C = Shrink64<kR>;
  extern __shared__ __align__(128) uint8_t ring[];
  cl::griddep_wait();
  cl::griddep_launch_dependents();
  const Rows rows{ws.tiles, ws.order};
  const int4 head = rows.tile(0);
  const int K = static_cast<int>(a.K), r = static_cast<int>(a.r), stages = (K - 1) / C::kCols + 1;
  const Shares sh = shares_of(stages, head.x, gridDim.x);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunk = threadIdx.x % C::kChunks, row0 = threadIdx.x / C::kChunks;
  const uint32_t ring_at = smem_u32(ring);
  const int64_t units = static_cast<int64_t>(head.x) * sh.shares;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int t = static_cast<int>(u / sh.shares), share = static_cast<int>(u - static_cast<int64_t>(t) * sh.shares);
    const int4 tile = rows.tile(1 + t);
    const int first = share * sh.per, last = min(first + sh.per, stages);
    const uint16_t* src_x[C::kXs];
#pragma unroll
    for (int i = 0; i < C::kXs; ++i) {
      const int row = row0 + i * C::kStep;
      src_x[i] = row < tile.z ? a.x + rows.row(tile.y + row) * a.x_stride : nullptr;
    }
    const uint16_t* src_a = a.A + static_cast<int64_t>(tile.x) * r * K;
    auto fetch = [&](int s, int slot) {
      const int col = s * C::kCols + chunk * 8;  // (stages end below 2^31 + 2^6)
      const bool in = col >= 0 && col < K;
      const uint32_t at = ring_at + slot * C::kStageBytes;
#pragma unroll
      for (int i = 0; i < C::kXs; ++i) {
        const int row = row0 + i * C::kStep;
        const bool real = in && src_x[i] != nullptr;
        cp_async16(at + row * C::kRowBytes + ((chunk ^ (row & 7)) << 4), real ? src_x[i] + col : a.x, real);
      }
#pragma unroll
      for (int i = 0; i < C::kAs; ++i) {
        const int row = row0 + i * C::kStep;
        const bool real = in && row < r;
        cp_async16(at + (64 + row) * C::kRowBytes + ((chunk ^ (row & 7)) << 4),
                   real ? src_a + static_cast<int64_t>(row) * K + col : a.A, real);
      }
    };
    float acc[kR / 8][4] = {};
#pragma unroll
    for (int s = 0; s < C::kStages - 1; ++s) {
      if (first + s < last) fetch(first + s, s);
      cp_commit();
    }
    int slot = 0;
    for (int s = first; s < last; ++s) {
      cp_wait<C::kStages - 2>();
      __syncthreads();
      if (s + C::kStages - 1 < last) fetch(s + C::kStages - 1, slot == 0 ? C::kStages - 1 : slot - 1);
      cp_commit();
      const uint32_t at = ring_at + slot * C::kStageBytes;
      slot = slot + 1 == C::kStages ? 0 : slot + 1;
#pragma unroll
      for (int kk = 0; kk < C::kCols / 16; ++kk) {
        const int xr = warp * 16 + (lane & 15);
        uint32_t x[4];
        ldmatrix4(x, at + xr * C::kRowBytes + (((2 * kk + (lane >> 4)) ^ (xr & 7)) << 4));
#pragma unroll
        for (int n = 0; n < kR / 16; ++n) {
          const int ar = n * 16 + (lane & 7) + ((lane >> 4) << 3);
          uint32_t b[4];
          ldmatrix4(b, at + (64 + ar) * C::kRowBytes + (((2 * kk + ((lane >> 3) & 1)) ^ (ar & 7)) << 4));
          mma_bf16_16816(acc[2 * n], x[0], x[1], x[2], x[3], b[0], b[1]);
          mma_bf16_16816(acc[2 * n + 1], x[0], x[1], x[2], x[3], b[2], b[3]);
        }
      }
    }
    __syncthreads();
    float* part = ws.part + (static_cast<int64_t>(share) * head.z + tile.y) * r;
    const int g = lane >> 2, q = 2 * (lane & 3);
#pragma unroll
    for (int n = 0; n < kR / 8; ++n) {
      const int col = n * 8 + q, row = warp * 16 + g;
      if (col >= r) break;
      if (row < tile.z) *reinterpret_cast<float2*>(part + row * r + col) = make_float2(acc[n][0], acc[n][1]);
      if (row + 8 < tile.z) *reinterpret_cast<float2*>(part + (row + 8) * r + col) = make_float2(acc[n][2], acc[n][3]);
    }
  }
}

// 16 lanes by 32 columns of tensor memory, as the sums of four MMAs of a warp's own.
__device__ __forceinline__ void tmem_ld_sums(uint32_t at, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(at));
}

// The same for larger ranks on the tcgen05 tensor cores: x's rows and A's lie in a stage
// as the descriptors want them, the sums in tensor memory (8192 rows, r 128: 171 us for
// the call, by mma.sync 179; 2049 rows, K 17408, r 64: 39 and 41.5; 512 rows of 60
// adapters, r 64: 35 and 38).
template <int kR>
__global__ void __launch_bounds__(kThreads) shrink_many_kernel(const LoraArgs a, const Ws ws, unsigned* status) {
  using C = Shrink64<kR>;
  extern __shared__ uint8_t smem[];
  __shared__ uint64_t done[C::kStages];  // a stage's MMAs
  __shared__ uint32_t tmem_at;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t ring_at = (smem_u32(smem) + 1023) & ~1023u;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) mbar_init(&done[i], 1);
    fence_mbar_init();
  }
  // (before the next kernel may start, so that it cannot take the columns from a block that it then waits for)
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_at)), "r"(kR)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = tmem_at;
  cl::griddep_wait();
  cl::griddep_launch_dependents();
  const Rows rows{ws.tiles, ws.order};
  const int4 head = rows.tile(0);
  const int K = static_cast<int>(a.K), r = static_cast<int>(a.r), stages = (K - 1) / C::kCols + 1;
  const Shares sh = shares_of(stages, head.x, gridDim.x);
  const int chunk = threadIdx.x % C::kChunks, row0 = threadIdx.x / C::kChunks;
  const int64_t units = static_cast<int64_t>(head.x) * sh.shares;
  uint32_t slot = 0, parity = 0;  // of the next stage; bit i: of slot i
  bool ok = true;
  auto wait = [&](uint32_t i) {  // for the MMAs of slot i's stage (after one wait that gave up without another)
    if (ok) ok = mbar_wait_bounded(&done[i], parity >> i & 1);
    parity ^= 1u << i;
  };
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int t = static_cast<int>(u / sh.shares), share = static_cast<int>(u - static_cast<int64_t>(t) * sh.shares);
    const int4 tile = rows.tile(1 + t);
    const int first = share * sh.per, last = min(first + sh.per, stages);
    const uint16_t* src_x[C::kXs];
#pragma unroll
    for (int i = 0; i < C::kXs; ++i) {
      const int row = row0 + i * C::kStep;
      src_x[i] = row < tile.z ? a.x + rows.row(tile.y + row) * a.x_stride : nullptr;
    }
    const uint16_t* src_a = a.A + static_cast<int64_t>(tile.x) * r * K;
    auto fetch = [&](int s, int slot) {
      const int col = s * C::kCols + chunk * 8;  // (stages end below 2^31 + 2^6)
      const bool in = col >= 0 && col < K;
      const uint32_t at = ring_at + slot * C::kStageBytes;
#pragma unroll
      for (int i = 0; i < C::kXs; ++i) {
        const int row = row0 + i * C::kStep;
        const bool real = in && src_x[i] != nullptr;
        cp_async16(at + row * C::kRowBytes + ((chunk ^ (row & 7)) << 4), real ? src_x[i] + col : a.x, real);
      }
#pragma unroll
      for (int i = 0; i < C::kAs; ++i) {
        const int row = row0 + i * C::kStep;
        const bool real = in && row < r;
        cp_async16(at + (64 + row) * C::kRowBytes + ((chunk ^ (row & 7)) << 4),
                   real ? src_a + static_cast<int64_t>(row) * K + col : a.A, real);
      }
    };
    uint32_t into = slot;
#pragma unroll 1
    for (int s = 0; s < C::kStages - 1; ++s) {
      if (first + s < last) fetch(first + s, into);
      cp_commit();
      into = into + 1 == C::kStages ? 0 : into + 1;
    }
#pragma unroll 1
    for (int s = first; s < last; ++s) {
      cp_wait<C::kStages - 2>();
      fence_proxy_async_smem();
      tc::tc_fence_before();
      __syncthreads();
      if (threadIdx.x == 0) {
        tc::tc_fence_after();
        const uint32_t at = ring_at + slot * C::kStageBytes;
        const uint64_t x_desc = tc::sw128_desc(at), a_desc = tc::sw128_desc(at + 64 * C::kRowBytes);
#pragma unroll
        for (int k = 0; k < C::kCols / 16; ++k) {
          asm volatile(
              "{\n\t.reg .pred p;\n\t"
              "setp.ne.b32 p, %4, 0;\n\t"
              "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(tmem),
              "l"(x_desc + 2 * k), "l"(a_desc + 2 * k), "r"(tc::make_idesc(64, kR)), "r"(s > first || k > 0 ? 1 : 0)
              : "memory");
        }
        tc::umma_commit(&done[slot]);
      }
      if (s > first) wait(into);  // the slot of the stage before
      if (s + C::kStages - 1 < last) fetch(s + C::kStages - 1, into);
      cp_commit();
      into = slot;
      slot = slot + 1 == C::kStages ? 0 : slot + 1;
    }
    wait(into);
    __syncwarp();
    tc::tc_fence_after();
    float* part = ws.part + (static_cast<int64_t>(share) * head.z + tile.y) * r;
    const int row = warp * 16 + (lane >> 2), q = 2 * (lane & 3);
#pragma unroll
    for (int c = 0; c < kR; c += 32) {
      uint32_t v[16];
      tmem_ld_sums(tmem + (static_cast<uint32_t>(warp) << 21) + c, v);
      tc::tmem_wait_ld_all(v);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = c + j * 8 + q;
        if (col >= r) break;
        if (row < tile.z)
          *reinterpret_cast<float2*>(part + row * r + col) = make_float2(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]));
        if (row + 8 < tile.z)
          *reinterpret_cast<float2*>(part + (row + 8) * r + col) = make_float2(__uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
      }
    }
  }
  if (!ok) record_status(status, kStatusTimeout);
  asm volatile("cp.async.wait_all;" ::: "memory");
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kR) : "memory");
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
// Two values as pairs of bf16 numbers of the values' own signs, neither of them 0 where the
// value is not: an infinite value of B, or sums beyond float32's range, are infinite in both
// products, or have the same sign in both, where a nearest number and its remainder gave NaN
// (0 or a number of the other sign times infinity) and values next to the largest became
// infinite. The first number is the largest below the value (of its size), the second the
// rest rounded, so that the pair is the value to 2^-16 (or 2^-132). Nearest numbers, to
// 2^-17, with the two products told apart where one is not finite took 1 to 14 % more of
// a call of many rows. (x, y: results of sums, whose NaN is 0x7FFFFFFF.)
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  uint32_t first[2];
  float rest[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float v = i == 0 ? x : y;
    const uint32_t b = __float_as_uint(v), size = b & 0x7FFFFFFFu;
    const uint32_t h = (b & 0x80000000u) | ((max(size, 0x00010001u) - 1) & 0xFFFF0000u);
    first[i] = size != 0 ? h : 0u;
    rest[i] = size != 0 ? copysignf(fmaxf(fabsf(v - __uint_as_float(h)), 0x1p-133f), v) : 0.0f;
  }
  hi = __byte_perm(first[0], first[1], 0x7632);
  lo = pack2(rest[0], rest[1]);
}

// Where the descriptors of the tensor cores have 16 bytes of a row of kRows: rows of 128
// bytes, swizzled by their number; the ranks from 64 on lie behind all rows.
template <int kRows>
__device__ __forceinline__ uint32_t tile_place(int row, int chunk) {
  return ((chunk >> 3) * kRows + row) * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

// Many rows, larger ranks: the shares added up in their order, scaled and written as
// the MMAs of the second product read them, so that its blocks, which come to a tile
// many times, find them ready (2049 rows, r 64, K 17408, 8 shares, both products by
// mma.sync: 42 us for the call, 47 where they added up the shares themselves; with r 16
// the launch costs the 2 us that it saves). A thread has two values of a row side by side; rows behind a tile's
// last stay as they are.
template <int kR>
__global__ void __launch_bounds__(256) join_kernel(const LoraArgs a, const Ws ws, int shrink_grid, int shrink_cols) {
  cl::griddep_wait();
  cl::griddep_launch_dependents();
  const Rows rows{ws.tiles, ws.order};
  const int4 head = rows.tile(0);
  const int r = static_cast<int>(a.r);
  const Shares sh = shares_of((static_cast<int>(a.K) - 1) / shrink_cols + 1, head.x, shrink_grid);
  const int64_t stride = static_cast<int64_t>(head.z) * r, all = static_cast<int64_t>(head.x) * (32 * kR);
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; u < all; u += int64_t{256} * gridDim.x) {
    const int t = static_cast<int>(u / (32 * kR)), pair = static_cast<int>(u % (32 * kR));
    const int row = pair / (kR / 2), col = 2 * (pair % (kR / 2));
    const int4 tile = rows.tile(1 + t);
    if (row >= tile.z) continue;
    float sx = 0.0f, sy = 0.0f;
    if (col < r) {
      const float* p = ws.part + (static_cast<int64_t>(tile.y) + row) * r + col;
      for (int j0 = 0; j0 < sh.shares; j0 += 8) {
        float2 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)  // (without branches: a load behind one waits for the load before it)
          v[j] = __ldcg(reinterpret_cast<const float2*>(p + min(j0 + j, sh.shares - 1) * stride));
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j0 + j < sh.shares) sx += v[j].x, sy += v[j].y;
      }
      const float scale = a.scale != nullptr ? a.scale[tile.x] : 1.0f;
      sx *= scale, sy *= scale;
    }
    uint32_t hi, lo;
    split2(sx, sy, hi, lo);
    uint8_t* dst = reinterpret_cast<uint8_t*>(ws.low + static_cast<int64_t>(t) * (64 * kR / 4)) +
                   tile_place<128>(row / 16 * 32 + row % 16, col >> 3) + 2 * (col & 7);
    *reinterpret_cast<uint32_t*>(dst) = hi;
    *reinterpret_cast<uint32_t*>(dst + 16 * 128) = lo;  // (the 17th row from there is swizzled alike)
  }
}

// ---------------------------------------------------------------- y = base + (x A^T) B^T

// Where B's row of column c lies: the columns of MMA j of 32, which are 8 i + 2 j and
// the next, one after another; and a piece of it, swizzled so that the 8 rows of an
// ldmatrix are in different banks.
template <int kR>
__device__ __forceinline__ uint32_t b_place(int row, int chunk) {
  static_assert(kR == 16 || kR == 32, "larger ranks lie as tile_place has them");
  const int sw = kR == 16 ? row >> 2 & 1 : row >> 1 & 3;
  return row * (2 * kR) + ((chunk ^ sw) << 4);
}
__device__ __forceinline__ int b_row(int c) { return (c & ~31) + (c >> 1 & 3) * 8 + (c >> 3 & 3) * 2 + (c & 1); }

// x A^T of 16 rows as the MMA's left operand, each value as two bf16 numbers.
template <int kR>
struct Low {
  uint4 hi[kR / 16], lo[kR / 16];
  // h: float32 [rows][kR]; row: this thread's first
  __device__ __forceinline__ void load(const float* h, int row, int q) {
#pragma unroll
    for (int s = 0; s < kR / 16; ++s) {
      const float* p = h + row * kR + 16 * s + 2 * q;
      split2(p[0], p[1], hi[s].x, lo[s].x);
      split2(p[8 * kR], p[8 * kR + 1], hi[s].y, lo[s].y);
      split2(p[8], p[9], hi[s].z, lo[s].z);
      split2(p[8 * kR + 8], p[8 * kR + 9], hi[s].w, lo[s].w);
    }
  }
  // acc += x A^T B^T for 32 columns whose rows of B begin at `at`
  __device__ __forceinline__ void times(uint32_t at, float (&acc)[4][4], int lane) const {
#pragma unroll
    for (int s = 0; s < kR / 16; ++s) {
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        uint32_t b[4];  // both halves of 16 values of r, for two MMAs
        ldmatrix4(b, at + b_place<kR>(j * 8 + (lane & 7) + (lane >> 4) * 8, 2 * s + (lane >> 3 & 1)));
        mma_bf16_16816(acc[j], lo[s].x, lo[s].y, lo[s].z, lo[s].w, b[0], b[1]);
        mma_bf16_16816(acc[j + 1], lo[s].x, lo[s].y, lo[s].z, lo[s].w, b[2], b[3]);
        mma_bf16_16816(acc[j], hi[s].x, hi[s].y, hi[s].z, hi[s].w, b[0], b[1]);
        mma_bf16_16816(acc[j + 1], hi[s].x, hi[s].y, hi[s].z, hi[s].w, b[2], b[3]);
      }
    }
  }
};

// The shares of x A^T of a tile's rows added up in their order and scaled, into h
// [kTile][kR] float32; rows and columns that are not there are zeros. By `threads`
// threads, `kSums` shares on their way at once.
template <int kTile, int kR, int kSums>
__device__ __forceinline__ void add_shares(float* h, const LoraArgs& a, const float* part, int4 tile, int64_t rows,
                                           int shares, int thread, int threads) {
  const float scale = a.scale != nullptr ? a.scale[tile.x] : 1.0f;
  const int r = static_cast<int>(a.r);
  const int64_t stride = rows * r;
#pragma unroll 1
  for (int i = thread; i < kTile * kR / 4; i += threads) {
    const int row = i / (kR / 4), col = i % (kR / 4) * 4;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (row < tile.z && col < r) {
      const float* p = part + (static_cast<int64_t>(tile.y) + row) * r + col;
#pragma unroll 1
      for (int j0 = 0; j0 < shares; j0 += kSums) {
        float4 v[kSums];
#pragma unroll
        for (int j = 0; j < kSums; ++j)  // (without branches: a load behind one waits for the load before it)
          v[j] = __ldcg(reinterpret_cast<const float4*>(p + min(j0 + j, shares - 1) * stride));
#pragma unroll
        for (int j = 0; j < kSums; ++j)
          if (j0 + j < shares) s.x += v[j].x, s.y += v[j].y, s.z += v[j].z, s.w += v[j].w;
      }
      s.x *= scale, s.y *= scale, s.z *= scale, s.w *= scale;
    }
    *reinterpret_cast<float4*>(h + row * kR + col) = s;
  }
}

// The MMAs' sums begin with base: 8 columns of this thread's row g + 8 i.
__device__ __forceinline__ void begin_with(float (&acc)[4][4], int i, const uint4& b) {
  const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    acc[j][2 * i] = __uint_as_float(w[j] << 16);
    acc[j][2 * i + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 rounded(const float (&acc)[4][4], int i) {
  return make_uint4(pack2(acc[0][2 * i], acc[0][2 * i + 1]), pack2(acc[1][2 * i], acc[1][2 * i + 1]),
                    pack2(acc[2][2 * i], acc[2][2 * i + 1]), pack2(acc[3][2 * i], acc[3][2 * i + 1]));
}

// 16 rows by 32 columns of base and y that lie at any 2-byte address: lanes side by
// side along a row, through a warp's own shared memory (kOddRow values a row).
constexpr int kOddRow = 34;
struct OddRows {
  uint16_t* stage;
  int64_t m;  // lane l < 16: the row, or -1
  __device__ __forceinline__ void read(const LoraArgs& a, int64_t col, int lane, float (&acc)[4][4]) const {
    const bool in = col + lane < a.N;
    __syncwarp();
#pragma unroll 8
    for (int i = 0; i < 16; ++i) {
      const int64_t row = __shfl_sync(0xFFFFFFFFu, m, i);
      stage[i * kOddRow + lane] = in && row >= 0 ? a.base[row * a.base_stride + col + lane] : 0;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(stage + ((lane >> 2) + 8 * i) * kOddRow + 8 * (lane & 3));
      begin_with(acc, i, make_uint4(p[0], p[1], p[2], p[3]));
    }
  }
  // (without an adapter the stage holds what was read)
  __device__ __forceinline__ void write(const LoraArgs& a, int64_t col, int lane, const float (&acc)[4][4],
                                        bool adapted) const {
    const bool in = col + lane < a.N;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!adapted) break;
      uint32_t* p = reinterpret_cast<uint32_t*>(stage + ((lane >> 2) + 8 * i) * kOddRow + 8 * (lane & 3));
      const uint4 v = rounded(acc, i);
      p[0] = v.x, p[1] = v.y, p[2] = v.z, p[3] = v.w;
    }
    __syncwarp();
#pragma unroll 8
    for (int i = 0; i < 16; ++i) {
      const int64_t row = __shfl_sync(0xFFFFFFFFu, m, i);
      if (in && row >= 0) a.y[row * a.y_stride + col + lane] = stage[i * kOddRow + lane];
    }
  }
};

// Where a run of units (a tile's columns, some at a time) stands.
struct Walk {
  int t, c;  // tile, place in its columns
  __device__ __forceinline__ void to(int64_t u, int per_tile) {
    t = static_cast<int>(u / per_tile);
    c = static_cast<int>(u - static_cast<int64_t>(t) * per_tile);
  }
  // true: a new tile
  __device__ __forceinline__ bool next(int per_tile) {
    if (++c < per_tile) return false;
    c = 0;
    ++t;
    return true;
  }
};

// Tiles of 8 rows: a warp for itself, 64 columns at a time, without barriers. B, which
// few rows use, is the left operand of four MMAs of 16 columns, dealt out so that a
// lane's are 8 in a row of two rows of y; x A^T is the right one. A lane copies its
// values of B and base itself into its own places of a ring of stages; of ranks up to
// 16 it reads 8 bytes of a row, and the warp copies whole pieces of 16 (the copies of 8
// go through the first level cache, which what is read before the wait must not).
template <int kR>
struct Expand8 {
  static constexpr bool kShared = kR == 16;  // the warp's pieces
  static constexpr int kPieces = kShared ? 1 : kR / 32;  // a lane's of a row of B
  static constexpr int kBBytes = 64 * kR * 2;
  static constexpr int kStageBytes = kBBytes + 2 * 16 * 32;
  static constexpr int kStages = kR == 16 || kR == 128 ? 2 : 3;
  static constexpr int kWarpBytes = kStages * kStageBytes + 8 * kR * 4;
  static constexpr int kSmem = kWarps * kWarpBytes;
  static constexpr int kAll = kSmem + static_cast<int>(sizeof(Few)) + 1024;
  static constexpr int kFit = 228 * 1024 / kAll < 4 ? 228 * 1024 / kAll : 4;
};
constexpr int kFewCols = 64;
// Rank 16: where the row of B of column c of 64 lies (the rows that a quarter of the
// lanes reads at once are in different banks).
__device__ __forceinline__ int b16_place(int c) { return (c ^ (c >> 3 & 3)) * 32; }

template <int kR, bool kVec, bool kFew>
__global__ void __launch_bounds__(kThreads, Expand8<kR>::kFit)
    expand8_kernel(const LoraArgs a, const Ws ws, int shrink_grid, int shrink_cols) {
  using C = Expand8<kR>;
  extern __shared__ __align__(128) uint8_t ring[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  float* h = reinterpret_cast<float*>(ring + warp * C::kWarpBytes + C::kStages * C::kStageBytes);
  const uint8_t* own_b = ring + warp * C::kWarpBytes + (C::kShared ? 0 : lane * 16);
  const uint8_t* own_base = ring + warp * C::kWarpBytes + C::kBBytes + lane * 16;
  const uint32_t own_b_at = smem_u32(own_b), own_base_at = smem_u32(own_base);
  // What comes before the wait reads the order of the rows, base and B, all complete
  // when the first product's kernel began its own work.
  const auto rows = [&] {
    if constexpr (kFew) {
      __shared__ Few few;
      group_few(few, a.adapter, static_cast<int>(a.M), static_cast<int>(a.n));
      return FewRows{&few};
    } else {
      return Rows{ws.tiles, ws.order};
    }
  }();
  const int4 head = rows.tile(0);
  const int r = static_cast<int>(a.r), N = static_cast<int>(a.N), per_tile = (N - 1) / kFewCols + 1;
  const int64_t units = static_cast<int64_t>(a.y == a.base ? head.x : head.y) * per_tile;
  // (neighbours in the line of units go to different blocks)
  const uint32_t w = warp * gridDim.x + blockIdx.x, all = gridDim.x * kWarps;
  Walk f;
  int todo;
  if (units <= 0x7FFFFFFF) {  // (divisions of 64 bits take as long as a few units)
    const uint32_t each = static_cast<uint32_t>(units) / all, more = static_cast<uint32_t>(units) - each * all;
    const uint32_t u0 = w * each + min(w, more);
    todo = static_cast<int>(each + (w < more ? 1 : 0));
    f.t = static_cast<int>(u0 / static_cast<uint32_t>(per_tile));
    f.c = static_cast<int>(u0 - static_cast<uint32_t>(f.t) * per_tile);
  } else {
    f.to(units / all * w, per_tile);
    todo = static_cast<int>(units / all + (w == all - 1 ? units % all : 0));
  }
  const Shares sh = shares_of((static_cast<int>(a.K) - 1) / shrink_cols + 1, head.x, shrink_grid);
  Walk now = f;
  int left = todo;  // units not fetched yet
  int4 ftile;
  const uint16_t *fB, *fbase[2];
  // this lane's rows of y are 2 q and 2 q + 1, its columns 8 g .. 8 g + 7; what it copies of B begins at this column
  // and value of r
  const int b_col = C::kShared ? lane >> 1 : 8 * g, piece = C::kShared ? 8 * (lane & 1) : 8 * q;
  auto fetch_tile = [&] {
    ftile = rows.tile(1 + f.t);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      fbase[i] = 2 * q + i < ftile.z ? a.base + rows.row(ftile.y + 2 * q + i) * a.base_stride + 8 * g : nullptr;
    fB = a.B + (static_cast<int64_t>(ftile.x) * N + b_col) * r + piece;
  };
  if (left > 0) fetch_tile();
  auto fetch = [&](uint32_t slot) {
    if (left <= 0) return;
    --left;
    const int col = f.c * kFewCols;
    if (ftile.x >= 0) {
      const uint16_t* src = fB + static_cast<int64_t>(col) * r;
      const bool whole = r == kR && N - col >= kFewCols;  // (col + 64 may be 2^31)
      if constexpr (C::kShared) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool real = whole || (col + b_col + 16 * j < N && piece < r);
          cp_async16(own_b_at + slot + b16_place(b_col + 16 * j) + 2 * piece, real ? src + 16 * j * r : a.B, real);
        }
      } else if (whole) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
          for (int i = 0; i < C::kPieces; ++i)
            cp_async16(own_b_at + slot + (j * C::kPieces + i) * 512, src + j * kR + 32 * i, true);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
          for (int i = 0; i < C::kPieces; ++i) {
            const bool real = col + b_col + j < N && piece + 32 * i < r;
            cp_async16(own_b_at + slot + (j * C::kPieces + i) * 512, real ? src + j * r + 32 * i : a.B, real);
          }
        }
      }
    }
    if constexpr (kVec) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (fbase[i] != nullptr && col + 8 * g < N) cp_async16(own_base_at + slot + i * 512, fbase[i] + col, true);
    }
    if (f.next(per_tile) && left > 0) fetch_tile();
  };
#pragma unroll 1
  for (int s = 0; s < C::kStages - 1; ++s) {
    fetch(s * C::kStageBytes);
    cp_commit();
  }
  cl::griddep_wait();
  cl::griddep_launch_dependents();

  int4 tile;
  const uint16_t* base[2];
  uint16_t* y[2];
  uint32_t hi[kR / 16][2], lo[kR / 16][2];
  bool fresh = true;
  uint32_t slot = 0, ahead = (C::kStages - 1) * C::kStageBytes;
#pragma unroll 1
  for (int u = 0; u < todo; ++u) {
    if constexpr (C::kShared) __syncwarp();  // (no lane reads the stage of the unit before any more)
    fetch(ahead);
    cp_commit();
    if (fresh) {
      tile = rows.tile(1 + now.t);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        base[i] = nullptr, y[i] = nullptr;
        if (2 * q + i < tile.z) {
          const int64_t m = rows.row(tile.y + 2 * q + i);
          base[i] = a.base + m * a.base_stride + 8 * g;
          y[i] = a.y + m * a.y_stride + 8 * g;
        }
      }
      if (tile.x >= 0) {
        __syncwarp();
        add_shares<8, kR, 12>(h, a, ws.part, tile, head.z, sh.shares, lane, 32);
        __syncwarp();
#pragma unroll
        for (int s = 0; s < kR / 16; ++s) {
          const int col = kR == 16 ? 4 * q : 32 * (s >> 1) + 8 * q + 4 * (s & 1);
          const float4 v = *reinterpret_cast<const float4*>(h + g * kR + col);
          split2(v.x, v.y, hi[s][0], lo[s][0]);
          split2(v.z, v.w, hi[s][1], lo[s][1]);
        }
      }
    }
    cp_wait<C::kStages - 1>();
    if constexpr (C::kShared) __syncwarp();  // (the other lanes' pieces)
    const int col = now.c * kFewCols;
    // MMA j: its rows g and g + 8 are columns 8 g + 2 j and the next of y, its columns rows of y
    float acc[4][4];
    uint4 was[2];  // base, as it is
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint4& v = was[i];
      v = make_uint4(0, 0, 0, 0);
      if constexpr (kVec) {
        v = *reinterpret_cast<const uint4*>(own_base + slot + i * 512);
      } else if (base[i] != nullptr) {
        uint32_t e[8];
#pragma unroll
        for (int l = 0; l < 8; ++l) e[l] = col + 8 * g + l < N ? base[i][col + l] : 0;
        v = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
      }
      const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[j][i] = __uint_as_float(w4[j] << 16);
        acc[j][2 + i] = __uint_as_float(w4[j] & 0xFFFF0000u);
      }
    }
    if (tile.x >= 0) {
#pragma unroll
      for (int i = 0; i < C::kPieces; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (C::kShared) {
            const uint2 e = *reinterpret_cast<const uint2*>(own_b + slot + b16_place(8 * g + 2 * j) + 8 * q);
            const uint2 o = *reinterpret_cast<const uint2*>(own_b + slot + b16_place(8 * g + 2 * j + 1) + 8 * q);
            mma_bf16_16816(acc[j], e.x, o.x, e.y, o.y, lo[0][0], lo[0][1]);
            mma_bf16_16816(acc[j], e.x, o.x, e.y, o.y, hi[0][0], hi[0][1]);
          } else {
            const uint8_t* at = own_b + slot + (2 * j * C::kPieces + i) * 512;
            const uint4 e = *reinterpret_cast<const uint4*>(at);
            const uint4 o = *reinterpret_cast<const uint4*>(at + C::kPieces * 512);
            mma_bf16_16816(acc[j], e.x, o.x, e.y, o.y, lo[2 * i][0], lo[2 * i][1]);
            mma_bf16_16816(acc[j], e.z, o.z, e.w, o.w, lo[2 * i + 1][0], lo[2 * i + 1][1]);
            mma_bf16_16816(acc[j], e.x, o.x, e.y, o.y, hi[2 * i][0], hi[2 * i][1]);
            mma_bf16_16816(acc[j], e.z, o.z, e.w, o.w, hi[2 * i + 1][0], hi[2 * i + 1][1]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (y[i] == nullptr) continue;
      uint32_t o[4] = {was[i].x, was[i].y, was[i].z, was[i].w};
      if (tile.x >= 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = pack2(acc[j][i], acc[j][2 + i]);
      }
      if constexpr (kVec) {
        if (col + 8 * g < N) *reinterpret_cast<uint4*>(y[i] + col) = make_uint4(o[0], o[1], o[2], o[3]);
      } else {
#pragma unroll
        for (int l = 0; l < 8; ++l)
          if (col + 8 * g + l < N) y[i][col + l] = static_cast<uint16_t>(o[l / 2] >> (16 * (l % 2)));
      }
    }
    fresh = now.next(per_tile);
    ahead = slot;
    slot = slot + C::kStageBytes == C::kStages * C::kStageBytes ? 0 : slot + C::kStageBytes;
  }
}

// Tiles of 64 rows: 8 warps, 16 rows and half of the columns each, share a ring of
// stages of B's rows and base's.
template <int kR>
struct Expand64 {
  static constexpr int kWarps = 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kUnit = 128;  // columns of a stage
  static constexpr int kStages = 3;
  static constexpr int kBaseBytes = 64 * kUnit * 2;
  static constexpr int kStageBytes = kBaseBytes + kUnit * kR * 2;
  static constexpr int kSmem = kStages * kStageBytes + 64 * kR * 4;
  static constexpr int kBaseChunks = kUnit / 8;             // 16-byte pieces of a row
  static constexpr int kBaseStep = kThreads / kBaseChunks;  // rows that the block copies at once
  static constexpr int kBases = 64 / kBaseStep;             // rows a thread copies
  static constexpr int kBs = kUnit * (kR / 8) / kThreads;   // pieces of B a thread copies
  static constexpr int kFit = 2;
  static_assert(kFit * (kSmem + 1024) <= 228 * 1024, "");
};

template <int kR, bool kVec>
__global__ void __launch_bounds__(Expand64<kR>::kThreads, Expand64<kR>::kFit)
    expand64_kernel(const LoraArgs a, const Ws ws, int shrink_grid, int shrink_cols) {
  using C = Expand64<kR>;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(16) uint16_t odd_stage[kVec ? 8 : C::kWarps * 16 * kOddRow];
  const uint32_t ring_at = smem_u32(ring);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  // What comes before the wait reads the order of the rows, base and B, all complete
  // when the kernel before this one began its own work.
  const Rows rows{ws.tiles, ws.order};
  const int4 head = rows.tile(0);
  const int r = static_cast<int>(a.r), N = static_cast<int>(a.N), per_tile = (N - 1) / C::kUnit + 1;
  const int64_t units = static_cast<int64_t>(a.y == a.base ? head.x : head.y) * per_tile;
  const int64_t u0 = units * blockIdx.x / gridDim.x;
  const int todo = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x - u0);

  const Shares sh = shares_of((static_cast<int>(a.K) - 1) / shrink_cols + 1, head.x, shrink_grid);
  Walk f, now;
  f.to(u0, per_tile);
  now = f;
  int left = todo;  // units not fetched yet
  int4 ftile;
  int base_row[C::kBases];
  const uint16_t* fB;
  const int base_chunk = threadIdx.x % C::kBaseChunks, base_row0 = threadIdx.x / C::kBaseChunks;
  const int b_chunk = threadIdx.x % (kR / 8), b_col0 = threadIdx.x / (kR / 8);
  constexpr int kBStep = C::kThreads / (kR / 8);  // columns whose rows of B the block copies at once
  auto fetch_tile = [&] {
    ftile = rows.tile(1 + f.t);
    if constexpr (kVec) {
#pragma unroll
      for (int i = 0; i < C::kBases; ++i) {
        const int row = base_row0 + i * C::kBaseStep;
        base_row[i] = row < ftile.z ? rows.row(ftile.y + row) : -1;
      }
    }
    fB = a.B + static_cast<int64_t>(ftile.x) * N * r + b_col0 * r + b_chunk * 8;
  };
  if (left > 0) fetch_tile();
  auto fetch = [&](uint32_t slot) {
    if (left <= 0) return;
    --left;
    const int col = f.c * C::kUnit;
    const uint32_t at = ring_at + slot;
    if constexpr (kVec) {
      const uint16_t* src = a.base + col + base_chunk * 8;
      const bool in = col + base_chunk * 8 < N;
#pragma unroll
      for (int i = 0; i < C::kBases; ++i) {
        const int row = base_row0 + i * C::kBaseStep;
        if (in && base_row[i] >= 0)
          cp_async16(at + row * (2 * C::kUnit) + ((base_chunk ^ (row & 1) << 2) << 4),
                     src + base_row[i] * a.base_stride, true);
      }
    }
    if (ftile.x >= 0) {
      const uint16_t* src = fB + static_cast<int64_t>(col) * r;
#pragma unroll
      for (int i = 0; i < C::kBs; ++i) {
        const int c = b_col0 + i * kBStep;
        const bool real = b_chunk * 8 < r && col + c < N;
        cp_async16(at + C::kBaseBytes + b_place<kR>(b_row(c), b_chunk), real ? src + i * kBStep * r : a.B, real);
      }
    }
    if (f.next(per_tile) && left > 0) fetch_tile();
  };
#pragma unroll 1
  for (int s = 0; s < C::kStages - 1; ++s) {
    fetch(s * C::kStageBytes);
    cp_commit();
  }
  cl::griddep_wait();
  cl::griddep_launch_dependents();

  const int row0 = (warp & 3) * 16 + g;
  Low<kR> low;
  int4 tile;
  uint16_t* y[2];
  OddRows odd{odd_stage + warp * 16 * kOddRow, -1};
  bool fresh = true;
  uint32_t slot = 0, ahead = (C::kStages - 1) * C::kStageBytes;
#pragma unroll 1
  for (int u = 0; u < todo; ++u) {
    cp_wait<C::kStages - 2>();
    __syncthreads();
    fetch(ahead);
    cp_commit();
    if (fresh) {
      tile = rows.tile(1 + now.t);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        y[i] = row0 + 8 * i < tile.z ? a.y + rows.row(tile.y + row0 + 8 * i) * a.y_stride + 8 * q : nullptr;
      if constexpr (!kVec) {
        const int row = (warp & 3) * 16 + (lane & 15);
        odd.m = row < tile.z ? rows.row(tile.y + row) : -1;
      }
      if (tile.x >= 0) {
        float* h = reinterpret_cast<float*>(ring + C::kStages * C::kStageBytes);
        add_shares<64, kR, 4>(h, a, ws.part, tile, head.z, sh.shares, threadIdx.x, C::kThreads);
        __syncthreads();
        low.load(h, row0, q);
        // (the next tile's sums are written after the barrier of its first unit)
      }
    }
    const int col0 = now.c * C::kUnit;
    const uint8_t* stage = ring + slot;
#pragma unroll
    for (int step = 0; step < C::kUnit / 64; ++step) {
      const int c0 = (warp >> 2) * (C::kUnit / 2) + step * 32;  // of the unit
      const int col = col0 + c0;
      float acc[4][4];
      if constexpr (kVec) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = row0 + 8 * i;
          begin_with(acc, i, *reinterpret_cast<const uint4*>(stage + row * (2 * C::kUnit) +
                                                             (((c0 / 8 + q) ^ (row & 1) << 2) << 4)));
        }
      } else {
        odd.read(a, col, lane, acc);
      }
      if (tile.x >= 0) low.times(ring_at + slot + C::kBaseBytes + c0 * (2 * kR), acc, lane);
      if constexpr (kVec) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (y[i] == nullptr || col + 8 * q >= N) continue;
          const int row = row0 + 8 * i;
          *reinterpret_cast<uint4*>(y[i] + col) =
              tile.x >= 0 ? rounded(acc, i)
                          : *reinterpret_cast<const uint4*>(stage + row * (2 * C::kUnit) + (((c0 / 8 + q) ^ (row & 1) << 2) << 4));
        }
      } else {
        odd.write(a, col, lane, acc, tile.x >= 0);
      }
    }
    fresh = now.next(per_tile);
    ahead = slot;
    slot += C::kStageBytes;
    if (slot == C::kStages * C::kStageBytes) slot = 0;
  }
}

// Tiles of 64 rows, larger ranks: the same on the tcgen05 tensor cores. The two numbers
// of a value are two of an MMA's 128 rows (16 rows' higher ones, their lower ones, the
// next 16 ..), so that a warp finds both sums of its rows in its own lanes of tensor
// memory, and reads them as its own MMAs would hold them: base, y and the order of the
// columns are as above. What a block waits for (loads, MMAs, sums) the other on its SM
// covers, or its 16 warps. 8192 rows, K 5120, N 17408: r 64 144 us, r 128 171 (two blocks
// of 8 warps and 64 columns 179); finishing a unit while the next one's MMAs run, which
// costs a stage, 144 and 176; the numbers as separate MMAs of 64 rows 144 and 189; by
// mma.sync 146 and 270. (Three blocks of r 64 take 139, but 207 where a block has to wait
// for a place, since each has its part of the units from the start.)
template <int kR, bool kVec>
struct ExpandMany {
  static constexpr int kUnit = kR == 64 ? 64 : 128;  // columns of a stage
  static constexpr int kFit = kR == 64 ? 2 : 1;
  static constexpr int kStages = 4;
  static constexpr int kWarps = kUnit / 8;  // 16 rows and 32 columns each
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kOdds = kVec ? 8 : kWarps * 16 * kOddRow;
  static constexpr int kBaseBytes = kVec ? 64 * kUnit * 2 : 0;  // (rows at any address are read later)
  static constexpr int kStageBytes = kBaseBytes + kUnit * kR * 2;
  static constexpr int kLowBytes = 64 * kR * 4;
  static constexpr int kSmem = 1024 + kLowBytes + kStages * kStageBytes;
  static constexpr int kBaseChunks = kUnit / 8;             // 16-byte pieces of a row
  static constexpr int kBaseStep = kThreads / kBaseChunks;  // rows that the block copies at once
  static constexpr int kBases = 64 / kBaseStep;             // rows a thread copies
  static constexpr int kBs = kUnit * (kR / 8) / kThreads;   // pieces of B a thread copies
  static constexpr int kLows = kLowBytes / 16 / kThreads;   // and of x A^T
  static_assert(kFit * kUnit <= 512 && kFit * (kSmem + 2 * kOdds + 1024 + 64) <= 228 * 1024, "");
};

template <int kR, bool kVec>
__global__ void __launch_bounds__(ExpandMany<kR, kVec>::kThreads, ExpandMany<kR, kVec>::kFit)
    expand_many_kernel(const LoraArgs a, const Ws ws, unsigned* status) {
  using C = ExpandMany<kR, kVec>;
  extern __shared__ uint8_t smem[];
  __shared__ __align__(16) uint16_t odd_stage[C::kOdds];
  __shared__ uint64_t done;  // a unit's MMAs
  __shared__ uint32_t tmem_at;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const uint32_t skip = -smem_u32(smem) & 1023;
  uint4* const low = reinterpret_cast<uint4*>(smem + skip);
  uint8_t* const ring = smem + skip + C::kLowBytes;
  const uint32_t ring_at = smem_u32(ring);
  if (threadIdx.x == 0) {
    mbar_init(&done, 1);
    fence_mbar_init();
  }
  // (before the next kernel may start, so that it cannot take the columns from a block that it then waits for)
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_at)),
                 "r"(C::kUnit)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = tmem_at;
  // What comes before the wait reads the order of the rows, base and B, all complete
  // when the kernel before this one began its own work.
  const Rows rows{ws.tiles, ws.order};
  const int4 head = rows.tile(0);
  const int r = static_cast<int>(a.r), N = static_cast<int>(a.N), per_tile = (N - 1) / C::kUnit + 1;
  const int64_t units = static_cast<int64_t>(a.y == a.base ? head.x : head.y) * per_tile;
  const int64_t u0 = units * blockIdx.x / gridDim.x;
  const int todo = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x - u0);

  Walk f, now;
  f.to(u0, per_tile);
  now = f;
  int left = todo;  // units not fetched yet
  int4 ftile;
  int base_row[C::kBases];
  const uint16_t* fB;
  const int base_chunk = threadIdx.x % C::kBaseChunks, base_row0 = threadIdx.x / C::kBaseChunks;
  const int b_chunk = threadIdx.x % (kR / 8), b_col0 = threadIdx.x / (kR / 8);
  constexpr int kBStep = C::kThreads / (kR / 8);  // columns whose rows of B the block copies at once
  auto fetch_tile = [&] {
    ftile = rows.tile(1 + f.t);
    if constexpr (kVec) {
#pragma unroll
      for (int i = 0; i < C::kBases; ++i) {
        const int row = base_row0 + i * C::kBaseStep;
        base_row[i] = row < ftile.z ? rows.row(ftile.y + row) : -1;
      }
    }
    fB = a.B + static_cast<int64_t>(ftile.x) * N * r + b_col0 * r + b_chunk * 8;
  };
  if (left > 0) fetch_tile();
  auto fetch = [&](uint32_t slot) {
    if (left <= 0) return;
    --left;
    const int col = f.c * C::kUnit;
    const uint32_t at = ring_at + slot;
    if constexpr (kVec) {
      const uint16_t* src = a.base + col + base_chunk * 8;
      const bool in = col + base_chunk * 8 < N;
#pragma unroll
      for (int i = 0; i < C::kBases; ++i) {
        const int row = base_row0 + i * C::kBaseStep;
        if (in && base_row[i] >= 0)
          cp_async16(at + row * (2 * C::kUnit) + ((base_chunk ^ (row & 1) << 2) << 4),
                     src + base_row[i] * a.base_stride, true);
      }
    }
    if (ftile.x >= 0) {
      const uint16_t* src = fB + static_cast<int64_t>(col) * r;
#pragma unroll
      for (int i = 0; i < C::kBs; ++i) {
        const int c = b_col0 + i * kBStep;
        const bool real = b_chunk * 8 < r && col + c < N;
        cp_async16(at + C::kBaseBytes + tile_place<C::kUnit>(b_row(c), b_chunk), real ? src + i * kBStep * r : a.B, real);
      }
    }
    if (f.next(per_tile) && left > 0) fetch_tile();
  };
#pragma unroll 1
  for (int s = 0; s < C::kStages - 1; ++s) {
    fetch(s * C::kStageBytes);
    cp_commit();
  }
  cl::griddep_wait();
  cl::griddep_launch_dependents();

  const int row0 = (warp & 3) * 16 + g, c0 = (warp >> 2) * 32;  // of the unit
  int4 tile;
  uint16_t* y[2];
  OddRows odd{odd_stage + warp * 16 * kOddRow, -1};
  bool fresh = true, ok = true;
  uint32_t slot = 0, ahead = (C::kStages - 1) * C::kStageBytes, parity = 0;
  const uint64_t x_desc = tc::sw128_desc(smem_u32(low)), b_desc = tc::sw128_desc(ring_at + C::kBaseBytes);
#pragma unroll 1
  for (int u = 0; u < todo; ++u) {
    cp_wait<C::kStages - 2>();
    fence_proxy_async_smem();
    tc::tc_fence_before();
    __syncthreads();  // (nothing reads the stage, the sums and x A^T of the unit before any more)
    if (fresh) {
      tile = rows.tile(1 + now.t);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        y[i] = row0 + 8 * i < tile.z ? a.y + rows.row(tile.y + row0 + 8 * i) * a.y_stride + 8 * q : nullptr;
      if constexpr (!kVec) {
        const int row = (warp & 3) * 16 + (lane & 15);
        odd.m = row < tile.z ? rows.row(tile.y + row) : -1;
      }
      if (tile.x >= 0) {
        const uint4* src = ws.low + static_cast<int64_t>(now.t) * (C::kLowBytes / 16) + threadIdx.x;
        uint4 v[C::kLows];
#pragma unroll
        for (int i = 0; i < C::kLows; ++i) v[i] = __ldcg(src + i * C::kThreads);
#pragma unroll
        for (int i = 0; i < C::kLows; ++i) low[threadIdx.x + i * C::kThreads] = v[i];
        fence_proxy_async_smem();
        __syncthreads();
      }
    }
    if (tile.x >= 0 && threadIdx.x == 0) {
      tc::tc_fence_after();
      const uint64_t b = b_desc + (slot >> 4);
#pragma unroll
      for (int i = 0; i < kR / 16; ++i) {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(tmem),
            "l"(x_desc + (i / 4 * (128 * 128 / 16) + 2 * (i % 4))), "l"(b + (i / 4 * (C::kUnit * 128 / 16) + 2 * (i % 4))),
            "r"(tc::make_idesc(128, C::kUnit)), "r"(i > 0 ? 1 : 0)
            : "memory");
      }
      tc::umma_commit(&done);
    }
    fetch(ahead);
    cp_commit();
    const int col = now.c * C::kUnit + c0;
    const uint8_t* stage = ring + slot;
    float acc[4][4];
    if constexpr (kVec) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = row0 + 8 * i;
        begin_with(acc, i, *reinterpret_cast<const uint4*>(stage + row * (2 * C::kUnit) +
                                                           (((c0 / 8 + q) ^ (row & 1) << 2) << 4)));
      }
    } else {
      odd.read(a, col, lane, acc);
    }
    if (tile.x >= 0) {
      if (ok) ok = mbar_wait_bounded(&done, parity);  // (after one wait that gave up without another)
      parity ^= 1;
      __syncwarp();
      tc::tc_fence_after();
      const uint32_t at = tmem + (static_cast<uint32_t>(warp & 3) << 21) + c0;
      uint32_t hi[16], lo[16];
      tmem_ld_sums(at, hi);
      tmem_ld_sums(at + (16u << 16), lo);
      tc::tmem_wait_ld_all(hi);
      tc::tmem_wait_ld_all(lo);
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i >> 2][i & 3] += __uint_as_float(lo[i]) + __uint_as_float(hi[i]);
    }
    if constexpr (kVec) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (y[i] == nullptr || col + 8 * q >= N) continue;
        const int row = row0 + 8 * i;
        *reinterpret_cast<uint4*>(y[i] + col) =
            tile.x >= 0 ? rounded(acc, i)
                        : *reinterpret_cast<const uint4*>(stage + row * (2 * C::kUnit) + (((c0 / 8 + q) ^ (row & 1) << 2) << 4));
      }
    } else {
      odd.write(a, col, lane, acc, tile.x >= 0);
    }
    fresh = now.next(per_tile);
    ahead = slot;
    slot = slot + C::kStageBytes == C::kStages * C::kStageBytes ? 0 : slot + C::kStageBytes;
  }
  if (!ok) record_status(status, kStatusTimeout);
  asm volatile("cp.async.wait_all;" ::: "memory");
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kUnit) : "memory");
}

bool sixteen_bytes(const LoraArgs& a) {
  return a.N % 8 == 0 && a.base_stride % 8 == 0 && a.y_stride % 8 == 0 && aligned16(a.base) && aligned16(a.y);
}

template <int kR, bool kFew>
cudaError_t launch_8(const Ctx& c, const LoraArgs& a, const Ws& ws) {
  using S = Shrink8<kR>;
  using E = Expand8<kR>;
  static SmemLimit lim;
  cudaError_t e = raise_smem_limit(lim, shrink8_kernel<kR, kFew>, c.device, S::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = most_tiles(a.M, a.n), stages = (a.K - 1) / S::kCols + 1;
  const int64_t grid = std::min({int64_t{S::kFit} * c.sm_count, int64_t{kMaxGrid}, tiles * std::min<int64_t>(stages, kMaxShares)});
  e = launch_early(c, grid, kThreads, S::kSmem, shrink8_kernel<kR, kFew>, a, ws);
  if (e != cudaSuccess) return e;
  const int64_t units = tiles * ((a.N - 1) / kFewCols + 1);
  const int64_t grid2 = std::min<int64_t>((units - 1) / kWarps + 1, E::kFit * c.sm_count);
  const auto expand = [&](SmemLimit& limit, auto kern) {
    const cudaError_t err = raise_smem_limit(limit, kern, c.device, E::kSmem);
    return err != cudaSuccess ? err
                              : launch_early(c, grid2, kThreads, E::kSmem, kern, a, ws, static_cast<int>(grid),
                                             int{S::kCols});
  };
  static SmemLimit vec, odd;
  return sixteen_bytes(a) ? expand(vec, expand8_kernel<kR, true, kFew>) : expand(odd, expand8_kernel<kR, false, kFew>);
}

template <int kR>
cudaError_t launch_64(const Ctx& c, const LoraArgs& a, const Ws& ws) {
  using S = Shrink64<kR>;
  static SmemLimit lim;
  const int64_t tiles = most_tiles(a.M, a.n), stages = (a.K - 1) / S::kCols + 1;
  const int64_t grid = std::min({int64_t{220 * 1024 / S::kSmem} * c.sm_count, int64_t{kMaxGrid}, tiles * std::min<int64_t>(stages, kMaxShares)});
  cudaError_t e;
  if constexpr (joined(kR)) {
    e = raise_smem_limit(lim, shrink_many_kernel<kR>, c.device, S::kSmem);
    if (e == cudaSuccess) e = launch_early(c, grid, kThreads, S::kSmem, shrink_many_kernel<kR>, a, ws, c.status);
  } else {
    e = raise_smem_limit(lim, shrink64_kernel<kR>, c.device, S::kSmem);
    if (e == cudaSuccess) e = launch_early(c, grid, kThreads, S::kSmem, shrink64_kernel<kR>, a, ws);
  }
  if (e != cudaSuccess) return e;
  static SmemLimit vec, odd;
  if constexpr (joined(kR)) {
    e = launch_early(c, std::min<int64_t>(tiles * (32 * kR / 256), 8 * c.sm_count), 256, 0, join_kernel<kR>, a, ws,
                     static_cast<int>(grid), int{S::kCols});
    if (e != cudaSuccess) return e;
    const auto expand = [&](SmemLimit& limit, auto kern, auto E) {
      const cudaError_t err = raise_smem_limit(limit, kern, c.device, E.kSmem);
      const int64_t grid2 = std::min<int64_t>(tiles * ((a.N - 1) / E.kUnit + 1), E.kFit * c.sm_count);
      return err != cudaSuccess ? err : launch_early(c, grid2, int{E.kThreads}, E.kSmem, kern, a, ws, c.status);
    };
    return sixteen_bytes(a) ? expand(vec, expand_many_kernel<kR, true>, ExpandMany<kR, true>{})
                            : expand(odd, expand_many_kernel<kR, false>, ExpandMany<kR, false>{});
  } else {
    using E = Expand64<kR>;
    const int64_t grid2 = std::min<int64_t>(tiles * ((a.N - 1) / E::kUnit + 1), E::kFit * c.sm_count);
    const auto expand = [&](SmemLimit& limit, auto kern) {
      const cudaError_t err = raise_smem_limit(limit, kern, c.device, E::kSmem);
      return err != cudaSuccess ? err
                                : launch_early(c, grid2, E::kThreads, E::kSmem, kern, a, ws, static_cast<int>(grid),
                                               int{S::kCols});
    };
    return sixteen_bytes(a) ? expand(vec, expand64_kernel<kR, true>) : expand(odd, expand64_kernel<kR, false>);
  }
}

template <int kR>
cudaError_t launch_rank(const Ctx& c, const LoraArgs& a, const Ws& ws) {
  if (a.M <= kFewRows) return launch_8<kR, true>(c, a, ws);
  return tile_of(a.M) == kFewTile ? launch_8<kR, false>(c, a, ws) : launch_64<kR>(c, a, ws);
}

}  // namespace

size_t lora_ws_bytes(int64_t M, int64_t n, int64_t r) {
  return round16(16 * (1 + most_tiles(M, n))) + round16(4 * M) + round16(part_bytes(M, r)) + low_bytes(M, n, r);
}

cudaError_t launch_lora(const Ctx& c, const LoraArgs& a) {
  Ws ws;
  uint8_t* p = static_cast<uint8_t*>(a.ws);
  ws.tiles = reinterpret_cast<int4*>(p);
  p += round16(16 * (1 + most_tiles(a.M, a.n)));
  ws.order = reinterpret_cast<int32_t*>(p);
  p += round16(4 * a.M);
  ws.part = reinterpret_cast<float*>(p);
  p += round16(part_bytes(a.M, a.r));
  ws.low = reinterpret_cast<uint4*>(p);
  if (a.M > kFewRows) {
    GroupArgs g{};
    g.ids = a.adapter;
    g.n = a.M;
    g.E = static_cast<int>(a.n);
    g.order = ws.order;
    g.tiles = ws.tiles;
    g.tile = tile_of(a.M);
    const cudaError_t e = launch_group(c, g);
    if (e != cudaSuccess) return e;
  }
  if (a.r <= 16) return launch_rank<16>(c, a, ws);
  if (a.r <= 32) return launch_rank<32>(c, a, ws);
  if (a.r <= 64) return launch_rank<64>(c, a, ws);
  return launch_rank<128>(c, a, ws);
}

}  // namespace wq
