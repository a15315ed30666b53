// Groups entries by a small id, stably: entry i of id e gets the place
// #{i' : (id', i') < (e, i)}, so that the entries of each id follow one another in
// their own order. The experts' rows of a batch and the tiles of its adapters
// begin with it.
//
// The ids are a few KB to a few hundred KB, so latency bounds it. A warp counts a
// run of entries in its own row of counters (the lanes that share an id find each
// other by votes on its bits, so nothing depends on the order of atomics; the
// instruction that matches whole numbers is far slower), the rows and the blocks are
// summed up, and what was counted before an entry is its place. Few entries take one
// block; more take a cluster of 8 that exchange their counts through distributed
// shared memory. 65536 ids of 128 experts: about 7 us of a sort's 121 (by matches 13).
#include "wq_cluster.cuh"
#include "wq_device.cuh"
#include "wq_internal.h"

namespace wq {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kRun = 8;  // ids a lane holds between the two passes
constexpr int64_t kGroupOneBlock = 4096;

// Exclusive prefix sum over the block of two counts a thread; *total receives the sum.
__device__ int block_scan(int a, int b, int* warp_sum, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = a + b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  int s = warp_sum[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, s, o);
    if (lane >= o) s += y;
  }
  *total = __shfl_sync(0xFFFFFFFFu, s, 31);
  const int before = warp > 0 ? __shfl_sync(0xFFFFFFFFu, s, warp - 1) : 0;
  __syncthreads();
  return before + x - a - b;
}

// The lanes whose number of `bits` bits is this lane's.
__device__ __forceinline__ uint32_t lanes_with(uint32_t x, int bits) {
  uint32_t same = 0xFFFFFFFFu;
#pragma unroll 4
  for (int b = 0; b < bits; ++b) {
    const uint32_t set = __ballot_sync(0xFFFFFFFFu, x >> b & 1);
    same &= x >> b & 1 ? set : ~set;
  }
  return same;
}

template <int kBlocks>
__global__ void __cluster_dims__(kBlocks, 1, 1) __launch_bounds__(kThreads) group_kernel(const GroupArgs a) {
  extern __shared__ int32_t smem[];
  __shared__ int warp_sum[kWarps];
  const int E1 = a.E + 1;               // ids outside [0, E) are the last group
  int32_t* hist = smem;                 // [kWarps][E1] counts, then places given out before, of each warp
  int32_t* count = hist + kWarps * E1;  // [E1] of this block
  int32_t* first = count + E1;          // [E1] this block's first place of each id
  int32_t* start = first + E1;          // [E1 + 1] the id's first place, and n
  int32_t* tile0 = start + E1 + 1;      // [E1 + 1] tiles before the id's
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = kBlocks > 1 ? static_cast<int>(cl::cluster_rank()) : 0;
  const int64_t per = (a.n + kBlocks * kThreads - 1) / (kBlocks * kThreads) * 32;
  const int64_t lo = (static_cast<int64_t>(rank) * kWarps + warp) * per, hi = lo + per < a.n ? lo + per : a.n;
  for (int i = threadIdx.x; i < kWarps * E1; i += kThreads) hist[i] = 0;
  cl::griddep_wait();
  cl::griddep_launch_dependents();
  int32_t* mine = hist + warp * E1;
  const int bits = 32 - __clz(E1);  // of E1, which stands for no entry
  int32_t id[kRun], before[kRun];
  auto load = [&](int64_t i0) {
    if (i0 >= hi) return;
#pragma unroll
    for (int j = 0; j < kRun; ++j) {  // (without branches: a load behind one waits for the load before it)
      const int64_t i = i0 + 32 * j + lane;
      id[j] = a.ids[i < hi ? i : hi - 1];
      if (id[j] < 0 || id[j] >= a.E) id[j] = a.E;
      if (i >= hi) id[j] = E1;
    }
  };
  // counts the run's ids: before[j] of the same id come before this lane's
  auto counted = [&](int64_t i0) {
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      if (i0 + 32 * j >= hi) break;
      const uint32_t same = lanes_with(id[j], bits), lower = same & ((1u << lane) - 1);
      const int have = id[j] < E1 ? mine[id[j]] : 0;
      before[j] = have + __popc(lower);
      __syncwarp();
      if (id[j] < E1 && lower == 0) mine[id[j]] = have + __popc(same);
      __syncwarp();
    }
  };
  load(lo);
  __syncthreads();
  for (int64_t i0 = lo; i0 < hi; i0 += 32 * kRun) {
    if (i0 > lo) load(i0);
    counted(i0);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E1; e += kThreads) {
    int c[kWarps], run = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) c[w] = hist[w * E1 + e];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      hist[w * E1 + e] = run;
      run += c[w];
    }
    count[e] = run;
  }
  if (kBlocks > 1) {
    cl::cluster_arrive();
    cl::cluster_wait();
  } else {
    __syncthreads();
  }
  // two ids a thread: E + 1 <= 1025
  int lower[2] = {}, all[2] = {};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = 2 * threadIdx.x + i;
    if (e >= E1) continue;
    if constexpr (kBlocks == 1) {
      all[i] = count[e];
    } else {
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        int c;
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(c) : "r"(cl::map_peer(smem_u32(count + e), b)));
        if (b < rank) lower[i] += c;
        all[i] += c;
      }
    }
  }
  if (kBlocks > 1) cl::cluster_arrive();  // this block reads no other's counts any more
  int total;
  int at = block_scan(all[0], all[1], warp_sum, &total);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = 2 * threadIdx.x + i;
    if (e < E1) {
      first[e] = at + lower[i];
      start[e] = at;
      if (rank == 0) {
        if (a.offsets != nullptr) a.offsets[e] = at;
        if (e == a.E && a.bad != nullptr && all[i] > 0) atomicAdd(a.bad, all[i]);
      }
    }
    at += all[i];
  }
  if (a.tiles != nullptr && rank == 0) {
    const int t0 = all[0] / a.tile + (all[0] % a.tile != 0), t1 = all[1] / a.tile + (all[1] % a.tile != 0);
    int tiles;
    const int tb = block_scan(t0, t1, warp_sum, &tiles);
    if (2 * threadIdx.x < E1) tile0[2 * threadIdx.x] = tb;
    if (2 * threadIdx.x + 1 < E1) tile0[2 * threadIdx.x + 1] = tb + t0;
    if (threadIdx.x == 0) start[E1] = total;
    __syncthreads();
    if (threadIdx.x == 0) a.tiles[0] = make_int4(tile0[a.E], tiles, start[a.E], 0);
    for (int t = threadIdx.x; t < tiles; t += kThreads) {
      int e = 0, end = E1;  // the last id whose tiles begin at t or before
      while (end - e > 1) {
        const int mid = (e + end) >> 1;
        if (tile0[mid] <= t) e = mid; else end = mid;
      }
      const int r0 = start[e] + (t - tile0[e]) * a.tile, rows = start[e + 1] - r0;
      a.tiles[1 + t] = make_int4(e < a.E ? e : -1, r0, rows < a.tile ? rows : a.tile, 0);
    }
  }
  if (kBlocks > 1) cl::cluster_wait();
  __syncthreads();
  // (a run that the registers do not hold is counted once more, from the places given out before it)
  const bool again = per > 32 * kRun;
  for (int64_t i0 = lo; i0 < hi; i0 += 32 * kRun) {
    if (again) {
      load(i0);
      counted(i0);
    }
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      const int64_t i = i0 + 32 * j + lane;
      if (i >= hi) continue;
      const int place = first[id[j]] + (again ? 0 : mine[id[j]]) + before[j];
      if (a.slots != nullptr) a.slots[i] = id[j] < a.E ? place : -1;
      if (a.order != nullptr) a.order[place] = static_cast<int32_t>(i);
    }
  }
}

}  // namespace

cudaError_t launch_group(const Ctx& c, const GroupArgs& a) {
  const size_t smem = sizeof(int32_t) * ((kWarps + 2) * (static_cast<size_t>(a.E) + 1) + 2 * (a.E + 2));
  // (2056 ids: a sort takes 9.6 us with one block and 10.3 with a cluster; 8192: an adapter call 116 and 115)
  if (a.n <= kGroupOneBlock) {
    static SmemLimit lim;
    const cudaError_t e = raise_smem_limit(lim, group_kernel<1>, c.device, smem);
    return e != cudaSuccess ? e : launch_early(c, 1, kThreads, smem, group_kernel<1>, a);
  }
  static SmemLimit lim;
  const cudaError_t e = raise_smem_limit(lim, group_kernel<8>, c.device, smem);
  return e != cudaSuccess ? e : launch_early(c, 8, kThreads, smem, group_kernel<8>, a);
}

}  // namespace wq
