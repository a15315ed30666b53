// Page management of a paged key-value cache: copy, fork, reserve, free and
// compact. The tables, lengths and counts are worked on by one block; the
// pages themselves are moved by a second launch that reads the list of
// (source, destination) pairs from device memory.
#include "wq_device.cuh"
#include "wq_internal.h"

namespace wq {
namespace {

constexpr int kMeta = 1024;  // threads of the block that works on the tables

// Exclusive prefix sum of v over the block; *total receives the block's sum.
template <typename I>
__device__ I block_scan(I v, I* total) {
  __shared__ I warp_sum[kMeta / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  I x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const I y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  if (warp == 0) {
    I s = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const I y = __shfl_up_sync(0xFFFFFFFFu, s, o);
      if (lane >= o) s += y;
    }
    warp_sum[lane] = s;
  }
  __syncthreads();
  const I before = warp == 0 ? 0 : warp_sum[warp - 1];
  *total = warp_sum[kMeta / 32 - 1];
  __syncthreads();
  return before + x - v;
}

__device__ void copy_array(const int32_t* src, int32_t* dst, int64_t n) {
  if (src == dst) return;
  for (int64_t i = threadIdx.x; i < n; i += kMeta) dst[i] = src[i];
}

// Pages that `len` tokens take, 0 for a negative length, at most W.
__device__ __forceinline__ int pages_of(int64_t len, int64_t S, int64_t W) {
  if (len <= 0) return 0;
  const int64_t p = (len + S - 1) / S;
  return static_cast<int>(p < W ? p : W);
}

// Scratch of the calls.
struct Scratch {
  int64_t* off;    // [n] free pages asked for before sequence or pair i
  int32_t* count;  // [4]: [0] pairs in the lists below
  int32_t* ids;    // [P] free pages in ascending order
  int32_t* src;    // [max(n, P)] pages to copy; -1: none
  int32_t* dst;    // [max(n, P)]
  int32_t* len;    // [n] the parents' lengths before the call
};
Scratch split_scratch(void* p, int64_t n, int64_t P) {
  int64_t* off = static_cast<int64_t*>(p);
  int32_t* w = reinterpret_cast<int32_t*>(off + n);
  const int64_t pairs = n > P ? n : P;
  return Scratch{off, w, w + 4, w + 4 + P, w + 4 + P + pairs, w + 4 + P + 2 * pairs};
}

// The first `want` free pages in ascending order, into ids; returns how many
// there are (at most want). Ends with a barrier.
__device__ int64_t find_free(const int32_t* ref, int64_t P, int64_t want, int32_t* ids) {
  int64_t got = 0;
  for (int64_t p0 = 0; p0 < P && got < want; p0 += kMeta) {
    const int64_t p = p0 + threadIdx.x;
    const int f = p < P && ref[p] == 0;
    int total;
    const int64_t r = got + block_scan(f, &total);
    if (f && r < want) ids[r] = static_cast<int32_t>(p);
    got += total;
  }
  __syncthreads();
  return got < want ? got : want;
}

__global__ void __launch_bounds__(kMeta) fork_kernel(SeqTables t, const int32_t* parent, const int32_t* child, int n,
                                                    int32_t* table_out, int32_t* lens_out, int32_t* ref_out,
                                                    int32_t* granted, Scratch w) {
  copy_array(t.table, table_out, t.B * t.W);
  copy_array(t.lens, lens_out, t.B);
  copy_array(t.ref, ref_out, t.P);
  const int64_t cap = t.W * t.S;
  auto good = [&](int i) {
    const int64_t p = parent[i], ch = child[i];
    return p >= 0 && p < t.B && ch >= 0 && ch < t.B && p != ch;
  };
  auto length = [&](int i) {
    const int64_t len = t.lens[parent[i]];
    return len < 0 ? int64_t{0} : (len > cap ? cap : len);
  };
  int64_t need_all = 0;
  for (int i0 = 0; i0 < n; i0 += kMeta) {
    const int i = i0 + threadIdx.x;
    const int64_t len = i < n && good(i) ? length(i) : 0, need = len % t.S != 0;
    int64_t total;
    const int64_t o = need_all + block_scan(need, &total);
    if (i < n) {
      w.off[i] = o;
      w.len[i] = static_cast<int32_t>(len);
    }
    need_all += total;
  }
  const int64_t have = find_free(t.ref, t.P, need_all, w.ids);
  for (int i = threadIdx.x >> 5; i < n; i += kMeta / 32) {  // one warp per pair
    const int lane = threadIdx.x & 31;
    const bool ok0 = good(i);
    const int64_t len = w.len[i], ch = child[i];
    const int full = static_cast<int>(len / t.S), need = len % t.S != 0;
    const bool ok = ok0 && (need == 0 || w.off[i] < have);
    int32_t from = -1, to = -1;
    if (ok) {
      for (int j = lane; j < full; j += 32) {
        const int32_t page = t.table[parent[i] * t.W + j];
        table_out[ch * t.W + j] = page;
        if (page >= 0 && page < t.P) atomicAdd(ref_out + page, 1);
      }
      if (need) {
        from = t.table[parent[i] * t.W + full];
        to = w.ids[w.off[i]];
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
  if (threadIdx.x == 0) w.count[0] = n;
}

__global__ void __launch_bounds__(kMeta) reserve_kernel(SeqTables t, const int32_t* new_lens, int32_t* table_out,
                                                       int32_t* ref_out, int32_t* granted, Scratch w) {
  copy_array(t.table, table_out, t.B * t.W);
  copy_array(t.ref, ref_out, t.P);
  const int64_t cap = t.W * t.S;
  auto needs = [&](int64_t b) -> int64_t {
    if (new_lens[b] > cap) return 0;
    const int d = pages_of(new_lens[b], t.S, t.W) - pages_of(t.lens[b], t.S, t.W);
    return d > 0 ? d : 0;
  };
  int64_t need_all = 0;
  for (int64_t b0 = 0; b0 < t.B; b0 += kMeta) {
    const int64_t b = b0 + threadIdx.x;
    const int64_t need = b < t.B ? needs(b) : 0;
    int64_t total;
    const int64_t o = need_all + block_scan(need, &total);
    if (b < t.B) w.off[b] = o;
    need_all += total;
  }
  const int64_t have = find_free(t.ref, t.P, need_all, w.ids);
  for (int64_t b = threadIdx.x >> 5; b < t.B; b += kMeta / 32) {
    const int lane = threadIdx.x & 31;
    const int64_t need = needs(b), o = w.off[b];
    const bool ok = new_lens[b] <= cap && (need == 0 || o + need <= have);
    if (ok) {
      const int first = pages_of(t.lens[b], t.S, t.W);
      for (int64_t j = lane; j < need; j += 32) {
        const int32_t page = w.ids[o + j];
        table_out[b * t.W + first + j] = page;
        ref_out[page] = 1;
      }
    }
    if (lane == 0) granted[b] = ok;
  }
}

__global__ void __launch_bounds__(kMeta) free_kernel(SeqTables t, const int32_t* seqs, int64_t n, int32_t* lens_out,
                                                    int32_t* ref_out, int32_t* bad) {
  // the lengths are read here, before the in-place update below
  copy_array(t.ref, ref_out, t.P);
  __syncthreads();
  for (int64_t i = threadIdx.x >> 5; i < n; i += kMeta / 32) {
    const int lane = threadIdx.x & 31;
    const int64_t b = seqs[i];
    if (b < 0 || b >= t.B) {
      if (lane == 0 && bad != nullptr) atomicAdd(bad, 1);
      continue;
    }
    const int have = pages_of(t.lens[b], t.S, t.W);
    for (int j = lane; j < have; j += 32) {
      const int32_t page = t.table[b * t.W + j];
      bool wrong = page < 0 || page >= t.P;
      if (!wrong && atomicSub(ref_out + page, 1) <= 0) {
        atomicAdd(ref_out + page, 1);
        wrong = true;
      }
      if (wrong && bad != nullptr) atomicAdd(bad, 1);
    }
  }
  __syncthreads();
  copy_array(t.lens, lens_out, t.B);
  __syncthreads();
  for (int64_t i = threadIdx.x; i < n; i += kMeta) {
    const int64_t b = seqs[i];
    if (b >= 0 && b < t.B) lens_out[b] = 0;
  }
}

__global__ void __launch_bounds__(kMeta) compact_kernel(SeqTables t, int32_t* table_out, int32_t* ref_out,
                                                       int32_t* remap, int32_t* n_live, Scratch w) {
  int64_t live = 0;
  for (int64_t p0 = 0; p0 < t.P; p0 += kMeta) {
    const int64_t p = p0 + threadIdx.x;
    live += __syncthreads_count(p < t.P && t.ref[p] != 0);
  }
  // the j-th page in use at or above `live` takes the j-th free one below it
  int64_t holes = 0, movers = 0;
  for (int64_t p0 = 0; p0 < t.P; p0 += kMeta) {
    const int64_t p = p0 + threadIdx.x;
    const bool used = p < t.P && t.ref[p] != 0;
    const int hole = p < live && !used, mover = p >= live && used;
    int nh, nm;
    const int64_t rh = holes + block_scan(hole, &nh), rm = movers + block_scan(mover, &nm);
    if (hole) w.dst[rh] = static_cast<int32_t>(p);
    if (mover) w.src[rm] = static_cast<int32_t>(p);
    if (p < t.P && !mover) remap[p] = used ? static_cast<int32_t>(p) : -1;
    holes += nh;
    movers += nm;
  }
  __syncthreads();
  for (int64_t j = threadIdx.x; j < movers; j += kMeta) {
    remap[w.src[j]] = w.dst[j];
    ref_out[w.dst[j]] = t.ref[w.src[j]];
  }
  if (ref_out != t.ref)
    for (int64_t p = threadIdx.x; p < live; p += kMeta)
      if (t.ref[p] != 0) ref_out[p] = t.ref[p];
  __syncthreads();
  for (int64_t p = live + threadIdx.x; p < t.P; p += kMeta) ref_out[p] = 0;
  for (int64_t i = threadIdx.x; i < t.B * t.W; i += kMeta) {
    const int64_t b = i / t.W;
    const int32_t page = t.table[i];
    if (i - b * t.W < pages_of(t.lens[b], t.S, t.W)) table_out[i] = page >= 0 && page < t.P ? remap[page] : -1;
    else if (table_out != t.table) table_out[i] = page;
  }
  if (threadIdx.x == 0) {
    w.count[0] = static_cast<int32_t>(movers);
    n_live[0] = static_cast<int32_t>(live);
  }
}

// Moves pages src[i] -> dst[i] in every layer, i < n or *count. A unit is
// kUnit bytes of one page of one layer.
constexpr int kCopyThreads = 256;
constexpr int64_t kUnit = 16384;

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(PagePool p, const int32_t* __restrict__ src,
                                                           const int32_t* __restrict__ dst, int64_t n,
                                                           const int32_t* __restrict__ count, int32_t* bad) {
  if (count != nullptr) n = *count;
  const int64_t per_page = (p.page_bytes + kUnit - 1) / kUnit, units = n * p.L * per_page;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t i = u / (p.L * per_page), r = u - i * p.L * per_page, layer = r / per_page, at = r - layer * per_page;
    const int64_t s = src[i], d = dst[i];
    if (s < 0 || s >= p.P || d < 0 || d >= p.P) {
      if (bad != nullptr && r == 0 && threadIdx.x == 0) atomicAdd(bad, 1);
      continue;
    }
    const int64_t first = at * kUnit, last = first + kUnit < p.page_bytes ? first + kUnit : p.page_bytes;
    const uint8_t* from = static_cast<const uint8_t*>(p.kv) + (layer * p.P + s) * p.page_bytes;
    uint8_t* to = static_cast<uint8_t*>(p.kv) + (layer * p.P + d) * p.page_bytes;
    for (int64_t o = first + threadIdx.x * 16; o < last; o += kCopyThreads * 16)
      *reinterpret_cast<uint4*>(to + o) = *reinterpret_cast<const uint4*>(from + o);
  }
}

cudaError_t copy_pages(const Ctx& c, const PagePool& p, const int32_t* src, const int32_t* dst, int64_t most,
                       const int32_t* count, int32_t* bad) {
  if (most == 0) return cudaSuccess;
  const int64_t per_page = (p.page_bytes + kUnit - 1) / kUnit;
  int64_t grid = 8 * static_cast<int64_t>(c.sm_count);
  if (most < grid && most * p.L < grid && most * p.L * per_page < grid) grid = most * p.L * per_page;
  copy_kernel<<<static_cast<unsigned>(grid), kCopyThreads, 0, c.stream>>>(p, src, dst, most, count, bad);
  return cudaGetLastError();
}

}  // namespace

size_t kv_pages_scratch(int64_t n, int64_t, int64_t, int64_t P) {
  const int64_t pairs = n > P ? n : P;
  return static_cast<size_t>(8 * n + 4 * (4 + P + 2 * pairs + n));
}

cudaError_t launch_pages_copy(const Ctx& c, const PagePool& p, const int32_t* src, const int32_t* dst, int64_t n,
                              int32_t* bad) {
  return copy_pages(c, p, src, dst, n, nullptr, bad);
}

cudaError_t launch_pages_fork(const Ctx& c, const PagePool& p, const SeqTables& t, const int32_t* parent,
                              const int32_t* child, int64_t n, int32_t* table_out, int32_t* lens_out,
                              int32_t* ref_out, int32_t* granted, void* scratch) {
  const Scratch w = split_scratch(scratch, n, t.P);
  fork_kernel<<<1, kMeta, 0, c.stream>>>(t, parent, child, static_cast<int>(n), table_out, lens_out, ref_out,
                                         granted, w);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && n > 0) e = copy_pages(c, p, w.src, w.dst, n, w.count, nullptr);
  return e;
}

cudaError_t launch_pages_reserve(const Ctx& c, const SeqTables& t, const int32_t* new_lens, int32_t* table_out,
                                 int32_t* ref_out, int32_t* granted, void* scratch) {
  reserve_kernel<<<1, kMeta, 0, c.stream>>>(t, new_lens, table_out, ref_out, granted,
                                            split_scratch(scratch, t.B, t.P));
  return cudaGetLastError();
}

cudaError_t launch_pages_free(const Ctx& c, const SeqTables& t, const int32_t* seqs, int64_t n, int32_t* lens_out,
                              int32_t* ref_out, int32_t* bad) {
  free_kernel<<<1, kMeta, 0, c.stream>>>(t, seqs, n, lens_out, ref_out, bad);
  return cudaGetLastError();
}

cudaError_t launch_pages_compact(const Ctx& c, const PagePool& p, const SeqTables& t, int32_t* table_out,
                                 int32_t* ref_out, int32_t* remap, int32_t* n_live, void* scratch) {
  const Scratch w = split_scratch(scratch, 0, t.P);
  compact_kernel<<<1, kMeta, 0, c.stream>>>(t, table_out, ref_out, remap, n_live, w);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = copy_pages(c, p, w.src, w.dst, t.P / 2, w.count, nullptr);
  return e;
}

}  // namespace wq
