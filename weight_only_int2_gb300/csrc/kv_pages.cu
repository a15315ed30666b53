// Page management of a paged key-value cache: copy, fork, reserve, free and
// compact.
//
// Two kinds of work, in a launch each. The tables, lengths and counts are a few
// hundred KB: latency bounds them (one block alone took 20 to 40 us for 65536
// pages), so a cluster of 8 blocks shares every step, with the cluster's barrier
// between the steps and running counts exchanged through distributed shared
// memory; all choices (which page to whom) follow from prefix sums over
// ascending ids, so nothing depends on timing. The pages themselves are moved by
// a second kernel that reads the (source, destination) list from device memory;
// it is bound by HBM and is launched before the first one has ended.
// Measured: fork of 16 sequences in a pool of 1024 pages with its copies 8.6 us,
// free and reserve for 256 sequences in a pool of 65536 pages 8.2 us each (one block:
// 32 and 31 us), compact's first kernel for 4096 pages 10 us, all latency:
// barriers and dependent loads. Pages: 1.07 GB moved in 160 us, 6.7 TB/s.
#include "wq_cluster.cuh"
#include "wq_device.cuh"
#include "wq_internal.h"

namespace wq {
namespace {

constexpr int kMeta = 512;    // threads of a block that works on the tables
constexpr int kBlocks = 8;    // such blocks, one cluster
constexpr int kMetaWarps = kMeta / 32;
constexpr int kAll = kMeta * kBlocks;
constexpr int kPer = 8;       // counts a thread looks at per pass

// Scratch of the calls.
struct Scratch {
  int64_t* off;    // [n] free pages asked for before sequence or pair i
  int64_t* asked;  // [1] by all
  int32_t* count;  // [4]: [0] pairs in the lists below
  int32_t* ids;    // [P] free pages in ascending order
  int32_t* src;    // [max(n, P)] pages to copy; -1: none
  int32_t* dst;    // [max(n, P)]
  int32_t* len;    // [n] the parents' lengths before the call
};
Scratch split_scratch(void* p, int64_t n, int64_t P) {
  int64_t* off = static_cast<int64_t*>(p);
  int32_t* w = reinterpret_cast<int32_t*>(off + n + 1);
  const int64_t pairs = n > P ? n : P;
  return Scratch{off, off + n, w, w + 4, w + 4 + P, w + 4 + P + pairs, w + 4 + P + 2 * pairs};
}

// A block's place in the cluster and what its blocks exchange.
struct Team {
  uint64_t (*counts)[kBlocks];  // [2][kBlocks] a pass's counts of every block, in turn
  uint64_t* warps;              // [kMetaWarps] of every warp
  int rank, turn;
  __device__ void sync() const {
    cl::cluster_arrive();
    cl::cluster_wait();
  }
  // What the warps before this one counted in this pass (warps of lower blocks
  // first), and all of them; `mine` is a warp's, the same in its lanes. Two
  // counts may share the 64 bits. A barrier of the cluster.
  __device__ uint64_t before(uint64_t mine, uint64_t* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) warps[warp] = mine;
    __syncthreads();
    uint64_t x = lane < kMetaWarps ? warps[lane] : 0;
    const uint64_t own = x;
#pragma unroll
    for (int o = 1; o < kMetaWarps; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    const uint64_t block = __shfl_sync(0xFFFFFFFFu, x, kMetaWarps - 1);
    const uint64_t in_block = __shfl_sync(0xFFFFFFFFu, x - own, warp);
    if (threadIdx.x < kBlocks) {
      const uint32_t to = cl::map_peer(smem_u32(&counts[turn][rank]), threadIdx.x);
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to), "l"(block) : "memory");
    }
    sync();
    uint64_t lower = 0, sum = 0;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      const uint64_t c = counts[turn][i];
      if (i < rank) lower += c;
      sum += c;
    }
    turn ^= 1;
    *all = sum;
    return lower + in_block;
  }
};
#define WQ_TEAM(team)                                  \
  __shared__ uint64_t team_counts[2][kBlocks];         \
  __shared__ uint64_t team_warps[kMetaWarps];          \
  Team team{team_counts, team_warps, static_cast<int>(cl::cluster_rank()), 0}

// Exclusive prefix sum of v over the block; *total receives the block's sum.
__device__ int64_t block_scan(int64_t v, int64_t* total) {
  __shared__ int64_t warp_sum[kMetaWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  int64_t before = 0, sum = 0;
#pragma unroll
  for (int i = 0; i < kMetaWarps; ++i) {
    const int64_t w = warp_sum[i];
    if (i < warp) before += w;
    sum += w;
  }
  __syncthreads();
  *total = sum;
  return before + x - v;
}

// dst = src by all blocks.
__device__ void copy_array(const Team& team, const int32_t* src, int32_t* dst, int64_t n) {
  if (src == dst) return;
  const int64_t first = static_cast<int64_t>(team.rank) * kMeta + threadIdx.x;
  if (((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 15) == 0) {
    const int64_t n4 = n / 4;
#pragma unroll 4
    for (int64_t i = first; i < n4; i += kAll) reinterpret_cast<int4*>(dst)[i] = reinterpret_cast<const int4*>(src)[i];
    if (first < n - 4 * n4) dst[4 * n4 + first] = src[4 * n4 + first];
  } else {
#pragma unroll 4
    for (int64_t i = first; i < n; i += kAll) dst[i] = src[i];
  }
}

// Pages that `len` tokens take, 0 for a negative length, at most W.
__device__ __forceinline__ int pages_of(int64_t len, int64_t S, int64_t W) {
  if (len <= 0) return 0;
  const int64_t p = (len + S - 1) / S;
  return static_cast<int>(p < W ? p : W);
}

// One pass over kAll * kPer counts from p0 on: a warp has 32 kPer pages in a
// row, bit i of a lane's result is page 32 i + lane of them.
__device__ __forceinline__ uint32_t in_use(const Team& team, const int32_t* ref, int64_t p0, int64_t P,
                                           int64_t* first, uint32_t* there) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  *first = p0 + static_cast<int64_t>(team.rank * kMetaWarps + warp) * 32 * kPer;
  int32_t c[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t p = *first + 32 * i + lane;
    c[i] = p < P ? ref[p] : 0;
  }
  uint32_t used = 0;
  *there = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    used |= static_cast<uint32_t>(c[i] != 0) << i;
    *there |= static_cast<uint32_t>(*first + 32 * i + lane < P) << i;
  }
  return used;
}
// The rank of page 32 i + lane among the warp's pages with a bit of `bits`, for
// one i after the other; `seen` counts those of the i before.
__device__ __forceinline__ int rank_of(uint32_t bits, int i, int& seen) {
  const uint32_t votes = __ballot_sync(0xFFFFFFFFu, (bits >> i & 1u) != 0);
  const int r = seen + __popc(votes & ((1u << (threadIdx.x & 31)) - 1u));
  seen += __popc(votes);
  return r;
}

// The free pages in ascending order, into ids: as many as *asked, which block 0
// writes before the call. Returns how many there are (at most *asked). Ends with
// a barrier of the cluster; whatever was written before it is seen after it.
__device__ int64_t find_free(Team& team, const int32_t* ref, int64_t P, const int64_t* asked, int32_t* ids) {
  int64_t got = 0, want = 1;  // (known after the first pass's barrier)
  for (int64_t p0 = 0; p0 < P && got < want; p0 += static_cast<int64_t>(kAll) * kPer) {
    int64_t first;
    uint32_t there;
    const uint32_t used = in_use(team, ref, p0, P, &first, &there), free = there & ~used;
    const int mine = __reduce_add_sync(0xFFFFFFFFu, __popc(free));
    uint64_t all;
    const int64_t r0 = got + static_cast<int64_t>(team.before(mine, &all));
    want = __ldcg(asked);
    int seen = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t r = r0 + rank_of(free, i, seen);
      if ((free >> i & 1u) != 0 && r < want) ids[r] = static_cast<int32_t>(first + 32 * i + (threadIdx.x & 31));
    }
    got += static_cast<int64_t>(all);
  }
  team.sync();
  return got < want ? got : want;
}

__global__ void __cluster_dims__(kBlocks, 1, 1) __launch_bounds__(kMeta)
    fork_kernel(SeqTables t, const int32_t* parent, const int32_t* child, int n, int32_t* table_out,
                int32_t* lens_out, int32_t* ref_out, int32_t* granted, Scratch w) {
  WQ_TEAM(team);
  cl::griddep_wait();
  cl::cluster_arrive();
  cl::griddep_launch_dependents();  // the copy may start; it waits for this kernel's end
  const int64_t cap = t.W * t.S;
  auto good = [&](int i) {
    const int64_t p = parent[i], ch = child[i];
    return p >= 0 && p < t.B && ch >= 0 && ch < t.B && p != ch;
  };
  // the lengths before anything is written, and the free pages that the pairs
  // up to each ask for
  if (team.rank == 0) {
    int64_t asked = 0;
    for (int i0 = 0; i0 < n; i0 += kMeta) {
      const int i = i0 + threadIdx.x;
      int64_t len = i < n && good(i) ? t.lens[parent[i]] : 0;
      len = len < 0 ? 0 : (len > cap ? cap : len);
      const int64_t need = len % t.S != 0;
      int64_t total;
      const int64_t o = asked + block_scan(need, &total);
      if (i < n) {
        w.off[i] = o;
        w.len[i] = static_cast<int32_t>(len);
      }
      asked += total;
    }
    if (threadIdx.x == 0) {
      *w.asked = asked;
      w.count[0] = n;
    }
  }
  copy_array(team, t.ref, ref_out, t.P);
  copy_array(team, t.table, table_out, t.B * t.W);
  copy_array(team, t.lens, lens_out, t.B);
  cl::cluster_wait();  // every block runs, before the first store into another's shared memory
  const int64_t have = find_free(team, t.ref, t.P, w.asked, w.ids);
  const int lane = threadIdx.x & 31;
  for (int i = team.rank * kMetaWarps + (threadIdx.x >> 5); i < n; i += kBlocks * kMetaWarps) {  // a warp per pair
    const bool ok0 = good(i);
    const int64_t len = __ldcg(w.len + i), off = __ldcg(w.off + i), ch = child[i];
    const int full = static_cast<int>(len / t.S), need = len % t.S != 0;
    const bool ok = ok0 && (need == 0 || off < have);
    int32_t from = -1, to = -1;
    if (ok) {
      for (int j = lane; j < full; j += 32) {
        const int32_t page = t.table[parent[i] * t.W + j];
        table_out[ch * t.W + j] = page;
        if (page >= 0 && page < t.P) atomicAdd(ref_out + page, 1);
      }
      if (need) {
        from = t.table[parent[i] * t.W + full];
        to = __ldcg(w.ids + off);
        if (lane == 0) {
          table_out[ch * t.W + full] = to;
          ref_out[to] = 1;
        }
      }
    }
    if (lane == 0) {
      granted[i] = ok;
      if (ch >= 0 && ch < t.B) lens_out[ch] = static_cast<int32_t>(ok ? len : 0);
      w.src[i] = from;
      w.dst[i] = to;
    }
  }
}

__global__ void __cluster_dims__(kBlocks, 1, 1) __launch_bounds__(kMeta)
    reserve_kernel(SeqTables t, const int32_t* new_lens, int32_t* table_out, int32_t* ref_out, int32_t* granted,
                   Scratch w) {
  WQ_TEAM(team);
  cl::griddep_wait();
  cl::cluster_arrive();
  const int64_t cap = t.W * t.S;
  auto needs = [&](int64_t b) -> int64_t {
    if (new_lens[b] > cap) return 0;
    const int d = pages_of(new_lens[b], t.S, t.W) - pages_of(t.lens[b], t.S, t.W);
    return d > 0 ? d : 0;
  };
  if (team.rank == 0) {
    int64_t asked = 0;
    for (int64_t b0 = 0; b0 < t.B; b0 += kMeta) {
      const int64_t b = b0 + threadIdx.x;
      const int64_t need = b < t.B ? needs(b) : 0;
      int64_t total;
      const int64_t o = asked + block_scan(need, &total);
      if (b < t.B) w.off[b] = o;
      asked += total;
    }
    if (threadIdx.x == 0) *w.asked = asked;
  }
  copy_array(team, t.ref, ref_out, t.P);
  copy_array(team, t.table, table_out, t.B * t.W);
  cl::cluster_wait();  // every block runs, before the first store into another's shared memory
  const int64_t have = find_free(team, t.ref, t.P, w.asked, w.ids);
  const int lane = threadIdx.x & 31;
  for (int64_t b = team.rank * kMetaWarps + (threadIdx.x >> 5); b < t.B; b += kBlocks * kMetaWarps) {
    const int64_t need = needs(b), o = __ldcg(w.off + b);
    const bool ok = new_lens[b] <= cap && (need == 0 || o + need <= have);
    if (ok) {
      const int first = pages_of(t.lens[b], t.S, t.W);
      for (int64_t j = lane; j < need; j += 32) {
        const int32_t page = __ldcg(w.ids + o + j);
        table_out[b * t.W + first + j] = page;
        ref_out[page] = 1;
      }
    }
    if (lane == 0) granted[b] = ok;
  }
}

__global__ void __cluster_dims__(kBlocks, 1, 1) __launch_bounds__(kMeta)
    free_kernel(SeqTables t, const int32_t* seqs, int64_t n, int32_t* lens_out, int32_t* ref_out, int32_t* bad) {
  WQ_TEAM(team);
  cl::griddep_wait();
  const int lane = threadIdx.x & 31;
  copy_array(team, t.ref, ref_out, t.P);
  copy_array(team, t.lens, lens_out, t.B);
  // a warp per sequence; the first one's pages are on their way before the barrier
  int64_t i = team.rank * kMetaWarps + (threadIdx.x >> 5), b = -1;
  int have = 0;
  int32_t page[kPer];
  const auto pages_from = [&](int j0) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int j = j0 + 32 * k + lane;
      page[k] = j < have ? t.table[b * t.W + j] : -1;
    }
  };
  const auto begin = [&]() {
    if (i >= n) return;
    b = seqs[i];
    have = b >= 0 && b < t.B ? pages_of(t.lens[b], t.S, t.W) : 0;
    pages_from(0);
  };
  begin();
  team.sync();
  for (; i < n; i += kBlocks * kMetaWarps, begin()) {
    if (b < 0 || b >= t.B) {
      if (lane == 0 && bad != nullptr) atomicAdd(bad, 1);
      continue;
    }
    for (int j0 = 0; j0 < have; j0 += 32 * kPer) {
      if (j0 > 0) pages_from(j0);
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (j0 + 32 * k + lane >= have) continue;
        bool wrong = page[k] < 0 || page[k] >= t.P;
        if (!wrong && atomicSub(ref_out + page[k], 1) <= 0) {
          atomicAdd(ref_out + page[k], 1);
          wrong = true;
        }
        if (wrong && bad != nullptr) atomicAdd(bad, 1);
      }
    }
    if (lane == 0) lens_out[b] = 0;  // (in place: nobody else reads it)
  }
}

__global__ void __cluster_dims__(kBlocks, 1, 1) __launch_bounds__(kMeta)
    compact_kernel(SeqTables t, int32_t* table_out, int32_t* ref_out, int32_t* remap, int32_t* n_live, Scratch w) {
  WQ_TEAM(team);
  cl::griddep_wait();
  cl::griddep_launch_dependents();  // the copy may start; it waits for this kernel's end
  const int lane = threadIdx.x & 31;
  team.sync();  // every block runs, before the first store into another's shared memory
  const int64_t step = static_cast<int64_t>(kAll) * kPer, gid = static_cast<int64_t>(team.rank) * kMeta + threadIdx.x;
  int64_t live = 0, first;
  uint32_t there, used = 0;
  for (int64_t p0 = 0; p0 < t.P; p0 += step) {
    used = in_use(team, t.ref, p0, t.P, &first, &there);
    uint64_t all;
    team.before(__reduce_add_sync(0xFFFFFFFFu, __popc(used)), &all);
    live += static_cast<int64_t>(all);
  }
  // the j-th page in use at or above `live` takes the j-th free one below it
  uint64_t done = 0;  // holes << 32 | movers
  for (int64_t p0 = 0; p0 < t.P; p0 += step) {
    if (t.P > step) used = in_use(team, t.ref, p0, t.P, &first, &there);  // else it is still at hand
    uint32_t low = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) low |= static_cast<uint32_t>(first + 32 * i + lane < live) << i;
    const uint32_t hole = there & low & ~used, mover = used & ~low;
    const uint64_t mine = static_cast<uint64_t>(__reduce_add_sync(0xFFFFFFFFu, __popc(hole))) << 32 |
                          static_cast<uint32_t>(__reduce_add_sync(0xFFFFFFFFu, __popc(mover)));
    uint64_t all;
    const uint64_t r0 = done + team.before(mine, &all);
    int holes = 0, movers = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t p = first + 32 * i + lane;
      const int64_t rh = static_cast<int64_t>(r0 >> 32) + rank_of(hole, i, holes);
      const int64_t rm = static_cast<int64_t>(r0 & 0xFFFFFFFFu) + rank_of(mover, i, movers);
      if ((hole >> i & 1u) != 0) w.dst[rh] = static_cast<int32_t>(p);
      if ((mover >> i & 1u) != 0) w.src[rm] = static_cast<int32_t>(p);
      else if ((there >> i & 1u) != 0) remap[p] = (used >> i & 1u) != 0 ? static_cast<int32_t>(p) : -1;
    }
    done += all;
  }
  const int64_t movers = static_cast<int64_t>(done & 0xFFFFFFFFu);
  team.sync();
  for (int64_t j = gid; j < movers; j += kAll) {
    const int32_t src = __ldcg(w.src + j), dst = __ldcg(w.dst + j);
    remap[src] = dst;
    ref_out[dst] = t.ref[src];
  }
  if (ref_out != t.ref)
    for (int64_t p = gid; p < live; p += kAll)
      if (t.ref[p] != 0) ref_out[p] = t.ref[p];
  if (gid == 0) {
    w.count[0] = static_cast<int32_t>(movers);
    n_live[0] = static_cast<int32_t>(live);
  }
  team.sync();
  for (int64_t p = live + gid; p < t.P; p += kAll) ref_out[p] = 0;
  const int64_t cells = t.B * t.W;
  for (int64_t i = gid; i < cells; i += kAll) {
    const int64_t b = i / t.W;
    const int32_t page = t.table[i];
    if (i - b * t.W < pages_of(t.lens[b], t.S, t.W)) table_out[i] = page >= 0 && page < t.P ? __ldcg(remap + page) : -1;
    else if (table_out != t.table) table_out[i] = page;
  }
}

// Moves pages src[i] -> dst[i] in every layer, i < n or *count. A unit is 64
// bytes a thread of one page of one layer, all of them on their way before the
// first store: 16 KB with blocks of 256, 4 KB with blocks of 64 for small pages.
// Several times as many blocks as fit the GPU at once: 1.07 GB moved in 160 us
// (6.7 TB/s); with just as many, in a loop, 180 us: nothing hid the index
// arithmetic and the ids' loads.
constexpr int kCopyThreads = 256, kSmallCopyThreads = 64;
constexpr int kVecs = 4;

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(PagePool p, const int32_t* src, const int32_t* dst,
                                                           int64_t n, const int32_t* count, int32_t* bad) {
  cl::griddep_wait();
  if (count != nullptr) n = __ldcg(count);
  const int threads = blockDim.x;
  const int64_t unit = threads * kVecs * 16, per_page = (p.page_bytes + unit - 1) / unit, per_pair = p.L * per_page, units = n * per_pair;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    int64_t i, layer, r;
    if (units <= 0x7FFFFFFF) {  // (32-bit divisions take a fraction of the others' time)
      i = static_cast<uint32_t>(u) / static_cast<uint32_t>(per_pair);
      r = u - i * per_pair;
      layer = static_cast<uint32_t>(r) / static_cast<uint32_t>(per_page);
    } else {
      i = u / per_pair;
      r = u - i * per_pair;
      layer = r / per_page;
    }
    const int64_t s = __ldcg(src + i), d = __ldcg(dst + i);
    if (s < 0 || s >= p.P || d < 0 || d >= p.P) {
      if (bad != nullptr && r == 0 && threadIdx.x == 0) atomicAdd(bad, 1);
      continue;
    }
    const int64_t at = (r - layer * per_page) * unit + threadIdx.x * 16;
    const uint8_t* from = static_cast<const uint8_t*>(p.kv) + (layer * p.P + s) * p.page_bytes;
    uint8_t* to = static_cast<uint8_t*>(p.kv) + (layer * p.P + d) * p.page_bytes;
    uint4 x[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int64_t o = at + j * threads * 16;
      if (o < p.page_bytes) x[j] = __ldcs(reinterpret_cast<const uint4*>(from + o));
    }
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int64_t o = at + j * threads * 16;
      if (o < p.page_bytes) __stcs(reinterpret_cast<uint4*>(to + o), x[j]);
    }
  }
}

cudaError_t copy_pages(const Ctx& c, const PagePool& p, const int32_t* src, const int32_t* dst, int64_t most,
                       const int32_t* count, int32_t* bad) {
  if (most == 0) return cudaSuccess;
  const int threads = p.page_bytes > kCopyThreads * kVecs * 8 ? kCopyThreads : kSmallCopyThreads;
  const int64_t unit = threads * kVecs * 16, per_page = (p.page_bytes + unit - 1) / unit;
  int64_t grid = (threads == kCopyThreads ? 64 : 256) * static_cast<int64_t>(c.sm_count);
  if (most < grid && most * p.L < grid && most * p.L * per_page < grid) grid = most * p.L * per_page;
  return launch_early(c, grid, threads, 0, copy_kernel, p, src, dst, most, count, bad);
}

}  // namespace

size_t kv_pages_scratch(int64_t n, int64_t, int64_t, int64_t P) {
  const int64_t pairs = n > P ? n : P;
  return static_cast<size_t>(8 * (n + 1) + 4 * (4 + P + 2 * pairs + n));
}

cudaError_t launch_pages_copy(const Ctx& c, const PagePool& p, const int32_t* src, const int32_t* dst, int64_t n,
                              int32_t* bad) {
  return copy_pages(c, p, src, dst, n, nullptr, bad);
}

cudaError_t launch_pages_fork(const Ctx& c, const PagePool& p, const SeqTables& t, const int32_t* parent,
                              const int32_t* child, int64_t n, int32_t* table_out, int32_t* lens_out,
                              int32_t* ref_out, int32_t* granted, void* scratch) {
  const Scratch w = split_scratch(scratch, n, t.P);
  cudaError_t e = launch_early(c, kBlocks, kMeta, 0, fork_kernel, t, parent, child, static_cast<int>(n), table_out,
                               lens_out, ref_out, granted, w);
  if (e == cudaSuccess) e = copy_pages(c, p, w.src, w.dst, n, w.count, nullptr);
  return e;
}

cudaError_t launch_pages_reserve(const Ctx& c, const SeqTables& t, const int32_t* new_lens, int32_t* table_out,
                                 int32_t* ref_out, int32_t* granted, void* scratch) {
  return launch_early(c, kBlocks, kMeta, 0, reserve_kernel, t, new_lens, table_out, ref_out, granted,
                      split_scratch(scratch, t.B, t.P));
}

cudaError_t launch_pages_free(const Ctx& c, const SeqTables& t, const int32_t* seqs, int64_t n, int32_t* lens_out,
                              int32_t* ref_out, int32_t* bad) {
  return launch_early(c, kBlocks, kMeta, 0, free_kernel, t, seqs, n, lens_out, ref_out, bad);
}

cudaError_t launch_pages_compact(const Ctx& c, const PagePool& p, const SeqTables& t, int32_t* table_out,
                                 int32_t* ref_out, int32_t* remap, int32_t* n_live, void* scratch) {
  const Scratch w = split_scratch(scratch, 0, t.P);
  cudaError_t e = launch_early(c, kBlocks, kMeta, 0, compact_kernel, t, table_out, ref_out, remap, n_live, w);
  if (e == cudaSuccess) e = copy_pages(c, p, w.src, w.dst, t.P / 2, w.count, nullptr);
  return e;
}

}  // namespace wq
