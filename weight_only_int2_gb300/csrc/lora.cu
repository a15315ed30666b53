// Low-rank adapters beside a shared projection: row m of y is
//   base[m] + scale[a] (x[m] A[a]^T) B[a]^T,   a = adapter[m],
// and base[m] for a row without an adapter.
//
// Three kernels. The rows are grouped by adapter into tiles (group.cu), so that every
// A and B is read by few blocks. The first product contracts over K: a block takes a
// tile and a share of K (as many shares as it takes to fill the GPU, a rule on the
// number of tiles, which is on the device) through a ring of cp.async stages into
// warp MMAs, and writes float32 partial sums. The second adds the shares up in their
// order, scales, and takes a tile and a run of columns: x A^T stays in registers as
// two bf16 numbers a value (2^-17 of itself; one would cost the sum bf16's 2^-9 once
// more), B comes straight from memory in the MMA's layout, and base and y are read
// and written 16 bytes a thread: the columns of four MMAs are dealt out so that a
// thread holds 8 in a row.
//
// Bound: HBM. With r up to 64 the MMAs take less time than base and y do; what a
// decode batch reads is each adapter's A and B once.
#include "wq_cluster.cuh"
#include "wq_device.cuh"
#include "wq_internal.h"

#include <cuda_bf16.h>

#include <algorithm>

namespace wq {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kStages = 4;
constexpr int kMaxShares = 32;
constexpr int kMaxGrid = 1024;   // blocks of the first product
constexpr int kUnit = 128;       // columns of a unit of the second product's work

// Rows of a tile. A decode batch has a few rows of each adapter: one MMA's 16 rows,
// the four warps side by side along K or the columns. From kManyRows rows on a warp
// has 16 rows of its own.
constexpr int64_t kManyRows = 512;
constexpr int tile_of(int64_t M) { return M < kManyRows ? 16 : 64; }

struct Ws {
  int4* tiles;     // as launch_group writes them
  int32_t* order;  // [M] the row at each place
  float* part;     // [shares][rows with an adapter][r]
};
int64_t most_tiles(int64_t M, int64_t n) { return M / tile_of(M) + std::min(M, n + 1); }
size_t part_bytes(int64_t M, int64_t r) {
  // shares * rows <= max(rows, blocks * tile), and shares <= kMaxShares
  return static_cast<size_t>(std::max(M, std::min(kMaxShares * M, int64_t{kMaxGrid} * tile_of(M)))) * r * 4;
}
size_t round16(size_t b) { return (b + 15) / 16 * 16; }

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

// How K is shared among blocks: `shares` of `per` stages each.
struct Shares {
  int shares, per;
};
__device__ __forceinline__ Shares shares_of(int stages, int tiles, int grid) {
  int s = tiles > 0 ? grid / tiles : 1;
  s = max(1, min(min(s, kMaxShares), stages));
  const int per = (stages + s - 1) / s;
  return Shares{(stages + per - 1) / per, per};
}

// ---------------------------------------------------------------- x A^T

template <int kTile, int kR>
struct Shrink {
  static constexpr int kCols = kTile == 16 ? 128 : 64;  // of a stage
  static constexpr int kRowBytes = 2 * kCols;
  static constexpr int kChunks = kRowBytes / 16;
  static constexpr int kRows = kTile + kR;
  static constexpr int kStageBytes = kRows * kRowBytes;
  static constexpr int kSmem = kStages * kStageBytes;
  static constexpr int kStep = kThreads / kChunks;        // rows that the block copies at once
  static constexpr int kXs = kTile / kStep;               // rows of x a thread copies
  static constexpr int kAs = (kR + kStep - 1) / kStep;    // and of A
  static_assert(kTile % kStep == 0, "");
  static_assert(kTile == 64 || kWarps * 16 * kR * 4 <= kSmem, "the warps' sums lie in the ring");
};

template <int kTile, int kR>
__global__ void __launch_bounds__(kThreads) shrink_kernel(const LoraArgs a, const Ws ws) {
  using C = Shrink<kTile, kR>;
  extern __shared__ __align__(128) uint8_t ring[];
  cl::griddep_wait();
  cl::griddep_launch_dependents();
  const int4 head = ws.tiles[0];
  const int stages_all = static_cast<int>((a.K + C::kCols - 1) / C::kCols);
  const Shares sh = shares_of(stages_all, head.x, gridDim.x);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunk = threadIdx.x % C::kChunks, row0 = threadIdx.x / C::kChunks;
  const uint32_t ring_at = smem_u32(ring);
  const int64_t units = static_cast<int64_t>(head.x) * sh.shares;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int t = static_cast<int>(u / sh.shares), share = static_cast<int>(u - static_cast<int64_t>(t) * sh.shares);
    const int4 tile = ws.tiles[1 + t];
    const int first = share * sh.per, last = min(first + sh.per, stages_all);
    const uint16_t* src_x[C::kXs];
    bool real_x[C::kXs];
#pragma unroll
    for (int i = 0; i < C::kXs; ++i) {
      const int row = row0 + i * C::kStep;
      real_x[i] = row < tile.z;
      src_x[i] = a.x + (real_x[i] ? ws.order[tile.y + row] : 0) * a.x_stride;
    }
    const uint16_t* src_a = a.A + static_cast<int64_t>(tile.x) * a.r * a.K;
    auto fetch = [&](int s, int slot) {
      const int64_t col = static_cast<int64_t>(s) * C::kCols + chunk * 8;
      const bool in = col < a.K;
      const uint32_t at = ring_at + slot * C::kStageBytes;
#pragma unroll
      for (int i = 0; i < C::kXs; ++i) {
        const int row = row0 + i * C::kStep;
        cp_async16(at + row * C::kRowBytes + ((chunk ^ (row & 7)) << 4), in ? src_x[i] + col : a.x, in && real_x[i]);
      }
#pragma unroll
      for (int i = 0; i < C::kAs; ++i) {
        const int row = row0 + i * C::kStep;
        if (C::kAs * C::kStep > kR && row >= kR) break;
        const bool real = in && row < a.r;
        cp_async16(at + (kTile + row) * C::kRowBytes + ((chunk ^ (row & 7)) << 4),
                   real ? src_a + row * a.K + col : a.A, real);
      }
    };
    float acc[kR / 8][4] = {};
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
      if (first + s < last) fetch(first + s, s);
      cp_commit();
    }
    int slot = 0;
    for (int s = first; s < last; ++s) {
      cp_wait<kStages - 2>();
      __syncthreads();
      if (s + kStages - 1 < last) fetch(s + kStages - 1, (slot + kStages - 1) % kStages);
      cp_commit();
      const uint32_t at = ring_at + slot * C::kStageBytes;
      slot = (slot + 1) % kStages;
#pragma unroll
      for (int kk = 0; kk < C::kCols / 16; ++kk) {
        if (kTile == 16 && (kk & (kWarps - 1)) != warp) continue;
        const int xr = (kTile == 16 ? 0 : warp * 16) + (lane & 15);
        uint32_t x[4];
        ldmatrix4(x, at + xr * C::kRowBytes + (((2 * kk + (lane >> 4)) ^ (xr & 7)) << 4));
#pragma unroll
        for (int n = 0; n < kR / 16; ++n) {
          const int ar = n * 16 + (lane & 7) + ((lane >> 4) << 3);
          uint32_t b[4];
          ldmatrix4(b, at + (kTile + ar) * C::kRowBytes + (((2 * kk + ((lane >> 3) & 1)) ^ (ar & 7)) << 4));
          mma_bf16_16816(acc[2 * n], x[0], x[1], x[2], x[3], b[0], b[1]);
          mma_bf16_16816(acc[2 * n + 1], x[0], x[1], x[2], x[3], b[2], b[3]);
        }
      }
    }
    __syncthreads();
    float* part = ws.part + (static_cast<int64_t>(share) * head.z + tile.y) * a.r;
    const int g = lane >> 2, q = 2 * (lane & 3);
    if constexpr (kTile == 16) {
      float* sums = reinterpret_cast<float*>(ring);
#pragma unroll
      for (int n = 0; n < kR / 8; ++n) {
        float* p = sums + (warp * 16 + g) * kR + n * 8 + q;
        p[0] = acc[n][0], p[1] = acc[n][1];
        p[8 * kR] = acc[n][2], p[8 * kR + 1] = acc[n][3];
      }
      __syncthreads();
      for (int i = threadIdx.x; i < 16 * kR; i += kThreads) {
        const int row = i / kR, col = i % kR;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += sums[w * 16 * kR + i];
        if (row < tile.z && col < a.r) part[row * a.r + col] = s;
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int n = 0; n < kR / 8; ++n) {
        const int col = n * 8 + q, row = warp * 16 + g;
        if (col >= a.r) break;
        if (row < tile.z) *reinterpret_cast<float2*>(part + row * a.r + col) = make_float2(acc[n][0], acc[n][1]);
        if (row + 8 < tile.z)
          *reinterpret_cast<float2*>(part + (row + 8) * a.r + col) = make_float2(acc[n][2], acc[n][3]);
      }
    }
  }
}

// ---------------------------------------------------------------- y = base + (x A^T) B^T

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
// Two values as pairs of bf16 numbers, whose sums are the values to 2^-17. (An
// infinite value has no second number, so that it stays one.)
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack2(x, y);
  const float xh = __uint_as_float(hi << 16), yh = __uint_as_float(hi & 0xFFFF0000u);
  lo = pack2(fabsf(xh) < INFINITY ? x - xh : 0.0f, fabsf(yh) < INFINITY ? y - yh : 0.0f);
}

template <int kTile, int kR, bool kVec>
__global__ void __launch_bounds__(kThreads) expand_kernel(const LoraArgs a, const Ws ws, int shrink_grid,
                                                          int shrink_cols) {
  constexpr int kSteps = kR / 16;
  constexpr int kPiece = kR == 16 ? 4 : 8;  // values of B's row that a thread holds in a row: the MMA's order of r
                                            // is dealt out alike on both sides
  __shared__ float h[kTile * kR];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  cl::griddep_wait();
  cl::griddep_launch_dependents();
  const int4 head = ws.tiles[0];
  const bool in_place = a.y == a.base;
  const int tiles = in_place ? head.x : head.y;
  const int per_tile = static_cast<int>((a.N + kUnit - 1) / kUnit);
  const int64_t units = static_cast<int64_t>(tiles) * per_tile;
  int64_t u = units * blockIdx.x / gridDim.x;
  const int64_t u_end = units * (blockIdx.x + 1) / gridDim.x;
  const Shares sh = shares_of(static_cast<int>((a.K + shrink_cols - 1) / shrink_cols), head.x, shrink_grid);
  while (u < u_end) {
    const int t = static_cast<int>(u / per_tile);
    const int c0 = static_cast<int>(u - static_cast<int64_t>(t) * per_tile);
    const int c1 = static_cast<int>(min(static_cast<int64_t>(per_tile), c0 + (u_end - u)));
    u += c1 - c0;
    const int4 tile = ws.tiles[1 + t];
    const bool adapted = tile.x >= 0;
    uint32_t hi[kSteps][4], lo[kSteps][4];
    const int rowA = (kTile == 16 ? 0 : warp * 16) + g;
    if (adapted) {
      __syncthreads();
      const float scale = a.scale != nullptr ? a.scale[tile.x] : 1.0f;
      const int64_t stride = static_cast<int64_t>(head.z) * a.r;
      for (int i = threadIdx.x; i < kTile * kR / 4; i += kThreads) {
        const int row = i / (kR / 4), col = i % (kR / 4) * 4;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (row < tile.z && col < a.r) {
          const float* p = ws.part + static_cast<int64_t>(tile.y + row) * a.r + col;
#pragma unroll 8
          for (int j = 0; j < sh.shares; ++j) {
            const float4 v = *reinterpret_cast<const float4*>(p + j * stride);
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
          }
          s.x *= scale, s.y *= scale, s.z *= scale, s.w *= scale;
        }
        *reinterpret_cast<float4*>(h + row * kR + col) = s;
      }
      __syncthreads();
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int col = kR == 16 ? q * 4 : (s / 2) * 32 + q * 8 + (s % 2) * 4;
        const float4 top = *reinterpret_cast<const float4*>(h + rowA * kR + col);
        const float4 low = *reinterpret_cast<const float4*>(h + (rowA + 8) * kR + col);
        split2(top.x, top.y, hi[s][0], lo[s][0]);
        split2(low.x, low.y, hi[s][1], lo[s][1]);
        split2(top.z, top.w, hi[s][2], lo[s][2]);
        split2(low.z, low.w, hi[s][3], lo[s][3]);
      }
    }
    const bool real0 = rowA < tile.z, real1 = rowA + 8 < tile.z;
    const int64_t m0 = real0 ? ws.order[tile.y + rowA] : 0, m1 = real1 ? ws.order[tile.y + rowA + 8] : 0;
    const uint16_t* base0 = a.base + m0 * a.base_stride;
    const uint16_t* base1 = a.base + m1 * a.base_stride;
    uint16_t* y0 = a.y + m0 * a.y_stride;
    uint16_t* y1 = a.y + m1 * a.y_stride;
    const uint16_t* Bt = a.B + static_cast<int64_t>(adapted ? tile.x : 0) * a.N * a.r;
    const int64_t col_end = min(a.N, static_cast<int64_t>(c1) * kUnit);
    for (int64_t col = static_cast<int64_t>(c0) * kUnit + (kTile == 16 ? warp * 32 : 0); col < col_end;
         col += kTile == 16 ? kUnit : 32) {
      const int64_t mine = col + 8 * q;  // this thread's 8 columns
      uint4 b0 = make_uint4(0, 0, 0, 0), b1 = b0;
      if constexpr (kVec) {
        if (real0 && mine < a.N) b0 = *reinterpret_cast<const uint4*>(base0 + mine);
        if (real1 && mine < a.N) b1 = *reinterpret_cast<const uint4*>(base1 + mine);
      }
      float acc[4][4] = {};
      if (adapted) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // MMA j's column g is column 8 (g / 2) + 2 j + g % 2 of the 32
          const int64_t n = min(col + 8 * (g >> 1) + 2 * j + (g & 1), a.N - 1);
          const uint16_t* row = Bt + n * a.r + q * kPiece;
          if constexpr (kR == 16) {
            uint2 b = make_uint2(0, 0);
            if (q * 4 < a.r) b = *reinterpret_cast<const uint2*>(row);
            mma_bf16_16816(acc[j], lo[0][0], lo[0][1], lo[0][2], lo[0][3], b.x, b.y);
            mma_bf16_16816(acc[j], hi[0][0], hi[0][1], hi[0][2], hi[0][3], b.x, b.y);
          } else {
#pragma unroll
            for (int s = 0; s < kR / 32; ++s) {
              uint4 b = make_uint4(0, 0, 0, 0);
              if (s * 32 + q * 8 < a.r) b = *reinterpret_cast<const uint4*>(row + s * 32);
              mma_bf16_16816(acc[j], lo[2 * s][0], lo[2 * s][1], lo[2 * s][2], lo[2 * s][3], b.x, b.y);
              mma_bf16_16816(acc[j], lo[2 * s + 1][0], lo[2 * s + 1][1], lo[2 * s + 1][2], lo[2 * s + 1][3], b.z, b.w);
              mma_bf16_16816(acc[j], hi[2 * s][0], hi[2 * s][1], hi[2 * s][2], hi[2 * s][3], b.x, b.y);
              mma_bf16_16816(acc[j], hi[2 * s + 1][0], hi[2 * s + 1][1], hi[2 * s + 1][2], hi[2 * s + 1][3], b.z, b.w);
            }
          }
        }
      }
      if constexpr (kVec) {
        auto add = [](uint32_t b, float x, float y) {
          return pack2(__uint_as_float(b << 16) + x, __uint_as_float(b & 0xFFFF0000u) + y);
        };
        if (adapted) {
          b0 = make_uint4(add(b0.x, acc[0][0], acc[0][1]), add(b0.y, acc[1][0], acc[1][1]),
                          add(b0.z, acc[2][0], acc[2][1]), add(b0.w, acc[3][0], acc[3][1]));
          b1 = make_uint4(add(b1.x, acc[0][2], acc[0][3]), add(b1.y, acc[1][2], acc[1][3]),
                          add(b1.z, acc[2][2], acc[2][3]), add(b1.w, acc[3][2], acc[3][3]));
        }
        if (real0 && mine < a.N) *reinterpret_cast<uint4*>(y0 + mine) = b0;
        if (real1 && mine < a.N) *reinterpret_cast<uint4*>(y1 + mine) = b1;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (mine + i >= a.N) break;
          if (real0) {
            const uint16_t b = base0[mine + i];
            y0[mine + i] = adapted ? float_to_bf16_bits_rn(bf16_bits_to_float(b) + acc[i / 2][i % 2]) : b;
          }
          if (real1) {
            const uint16_t b = base1[mine + i];
            y1[mine + i] = adapted ? float_to_bf16_bits_rn(bf16_bits_to_float(b) + acc[i / 2][2 + i % 2]) : b;
          }
        }
      }
    }
  }
}

template <int kTile, int kR>
cudaError_t launch_products(const Ctx& c, const LoraArgs& a, const Ws& ws) {
  using C = Shrink<kTile, kR>;
  static SmemLimit lim;
  cudaError_t e = raise_smem_limit(lim, shrink_kernel<kTile, kR>, c.device, C::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t stages = (a.K + C::kCols - 1) / C::kCols, tiles = most_tiles(a.M, a.n);
  const int fit = std::max(1, std::min(8, 220 * 1024 / C::kSmem));
  const int64_t grid = std::min({int64_t{fit} * c.sm_count, int64_t{kMaxGrid}, tiles * std::min<int64_t>(stages, kMaxShares)});
  e = launch_early(c, grid, kThreads, C::kSmem, shrink_kernel<kTile, kR>, a, ws);
  if (e != cudaSuccess) return e;
  const bool vec = a.N % 8 == 0 && a.base_stride % 8 == 0 && a.y_stride % 8 == 0 && aligned16(a.base) && aligned16(a.y);
  const int64_t units = tiles * ((a.N + kUnit - 1) / kUnit);
  const int64_t grid2 = std::min<int64_t>(units, int64_t{8} * c.sm_count);
  return launch_early(c, grid2, kThreads, 0, vec ? expand_kernel<kTile, kR, true> : expand_kernel<kTile, kR, false>, a,
                      ws, static_cast<int>(grid), int{C::kCols});
}

template <int kTile>
cudaError_t launch_ranks(const Ctx& c, const LoraArgs& a, const Ws& ws) {
  if (a.r <= 16) return launch_products<kTile, 16>(c, a, ws);
  if (a.r <= 32) return launch_products<kTile, 32>(c, a, ws);
  if (a.r <= 64) return launch_products<kTile, 64>(c, a, ws);
  return launch_products<kTile, 128>(c, a, ws);
}

}  // namespace

size_t lora_ws_bytes(int64_t M, int64_t n, int64_t r) {
  return round16(16 * (1 + most_tiles(M, n))) + round16(4 * M) + part_bytes(M, r);
}

cudaError_t launch_lora(const Ctx& c, const LoraArgs& a) {
  Ws ws;
  uint8_t* p = static_cast<uint8_t*>(a.ws);
  ws.tiles = reinterpret_cast<int4*>(p);
  p += round16(16 * (1 + most_tiles(a.M, a.n)));
  ws.order = reinterpret_cast<int32_t*>(p);
  p += round16(4 * a.M);
  ws.part = reinterpret_cast<float*>(p);
  GroupArgs g{};
  g.ids = a.adapter;
  g.n = a.M;
  g.E = static_cast<int>(a.n);
  g.order = ws.order;
  g.tiles = ws.tiles;
  g.tile = tile_of(a.M);
  const cudaError_t e = launch_group(c, g);
  if (e != cudaSuccess) return e;
  return tile_of(a.M) == 16 ? launch_ranks<16>(c, a, ws) : launch_ranks<64>(c, a, ws);
}

}  // namespace wq
