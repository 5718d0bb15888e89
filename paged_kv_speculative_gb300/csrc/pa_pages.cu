// Page operations on the pool: fork, resize (grow, trim, free, copy on write),
// compact and copy. A free page is one whose reference count is 0 and pages
// are taken lowest number first, so there is no free list to keep: every
// result is a function of the block table, the lengths and the counts. Counts
// change by integer atomics, whose order does not change the result.
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "pa_prefill.h"

namespace pav {

namespace {

constexpr int kThreads = 1024;
constexpr int kTicketInts = 64;
constexpr int kPagesPerBlock = 4096;  // compact: pages of one block (4 a thread)

__device__ __forceinline__ int pages_of(int len) { return (len + kPage - 1) / kPage; }

__device__ __forceinline__ void flag(uint32_t* err, uint32_t bits) {
  if (err) atomicOr(err, bits);
}

// Exclusive prefix sum of v over the block's 1024 threads; *total gets the sum. Two block barriers.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* total, T* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, m);
    if (lane >= m) x += y;
  }
  __syncthreads();  // red is free again
  if (lane == 31) red[warp] = x;
  __syncthreads();
  T w = red[lane];  // 32 warps
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, w, m);
    if (lane >= m) w += y;
  }
  const T before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  *total = __shfl_sync(0xffffffffu, w, 31);
  return x - v + (warp ? before : T(0));
}

// ---------------------------------------------------------------- fork
// One block an entry: an entry is valid on its own reading of the whole list, so no block waits for another and
// none reads a length that another writes (a parent is no entry's child, and a child has one valid entry).
__global__ void __launch_bounds__(256) pages_fork_kernel(PagesDesc d, int32_t* __restrict__ table, int32_t* lens,
                                                         int32_t* __restrict__ ref, const int32_t* __restrict__ parents,
                                                         const int32_t* __restrict__ children, int n, uint32_t* err) {
  chained_start();
  const int i = blockIdx.x;
  const int parent = parents[i], child = children[i];
  bool bad = parent < 0 || parent >= d.num_seqs || child < 0 || child >= d.num_seqs;
  for (int j = threadIdx.x; j < n; j += blockDim.x) {
    const int c = children[j];
    bad |= c == parent || (j < i && c == child);
  }
  int len = 0;
  if (!__syncthreads_or(bad)) {
    len = lens[parent];
    bad = lens[child] != 0 || len < 0 || len > static_cast<int64_t>(d.stride) * kPage;
  }
  if (__syncthreads_or(bad)) {  // also: every thread has read the child's length before it is written
    if (threadIdx.x == 0) flag(err, kErrLengths);
    return;
  }
  const int32_t* from = table + static_cast<size_t>(parent) * d.stride;
  int32_t* to = table + static_cast<size_t>(child) * d.stride;
  for (int k = threadIdx.x; k < pages_of(len); k += blockDim.x) {
    const int p = from[k];
    to[k] = p;
    if (p < 0 || p >= d.num_pages) flag(err, kErrPageRange);
    else if (atomicAdd(ref + p, 1) <= 0) flag(err, kErrRefs);
  }
  if (threadIdx.x == 0) lens[child] = len;
}

// ---------------------------------------------------------------- resize
// A shrinking row drops the pages behind its new end; `tid` of `threads` threads share the row. The caller has read the
// length before (a barrier stands between that and the write here).
__device__ __forceinline__ void release_row(const PagesDesc& d, int b, int len, int to, const int32_t* table, int32_t* lens,
                                            int32_t* ref, uint32_t* err, int tid, int threads) {
  if (to < 0) return;
  const int64_t most = static_cast<int64_t>(d.stride) * kPage;
  if (len < 0 || len > most || to > most) {
    if (tid == 0) flag(err, kErrLengths);
    return;
  }
  if (to >= len) return;
  const int32_t* row = table + static_cast<size_t>(b) * d.stride;
  for (int k = pages_of(to) + tid; k < pages_of(len); k += threads) {
    const int p = row[k];
    if (p < 0 || p >= d.num_pages) {
      flag(err, kErrPageRange);
    } else if (atomicSub(ref + p, 1) <= 0) {
      atomicAdd(ref + p, 1);
      flag(err, kErrRefs);
    }
  }
  if (tid == 0) lens[b] = to;
}

constexpr int kSmallList = 4096;  // free pages of one call that are listed in shared memory

// One launch. The shrinking rows first: one block for all of them when the table is small (a warp a row), else a block a
// row; the block that finishes last (a ticket in the workspace, put back to 0) then serves the growing rows, thread b row b:
// what each needs, the lowest free pages by a scan of the counts that stops as soon as there are enough, the tables. What
// other blocks wrote is read past the L1 cache.
__global__ void __launch_bounds__(kThreads) pages_resize_kernel(PagesDesc d, int32_t* table, int32_t* lens, int32_t* ref,
                                                                const int32_t* __restrict__ new_lens,
                                                                int32_t* __restrict__ copy_src, int32_t* __restrict__ copy_dst,
                                                                uint32_t* err, uint32_t* ticket, int32_t* far_list) {
  chained_start();
  __shared__ long long red64[32];
  __shared__ int red[32];
  __shared__ int tails[kThreads];
  __shared__ long long s_first[kThreads];  // the row's first place in the list
  __shared__ int s_have[kThreads];         // pages it has (~: the first of the list replaces the last of them); INT_MIN: refused
  __shared__ int32_t s_list[kSmallList];
  __shared__ int s_growers[kThreads];      // growing rows by their shared page's hash
  const int b = threadIdx.x, lane = b & 31;
  if (gridDim.x == 1) {
    for (int r = b >> 5; r < d.num_seqs; r += kThreads / 32) {
      const int len = lens[r], to = new_lens[r];
      __syncwarp();
      release_row(d, r, len, to, table, lens, ref, err, lane, 32);
    }
    __syncthreads();
  } else {
    for (int r = blockIdx.x; r < d.num_seqs; r += gridDim.x) {
      const int len = lens[r], to = new_lens[r];
      __syncthreads();
      release_row(d, r, len, to, table, lens, ref, err, b, kThreads);
    }
    __threadfence();
    __syncthreads();
    int last = 0;
    if (b == 0) last = atomicAdd(ticket, 1u) == gridDim.x - 1;
    if (!__syncthreads_or(last)) return;
    if (b == 0) *ticket = 0;
    __threadfence();
  }

  int len = 0, to = -1, tail = -1;
  bool grows = false;
  if (b < d.num_seqs) {
    len = __ldcg(lens + b);
    to = new_lens[b];
    grows = to > len && len >= 0 && to <= static_cast<int64_t>(d.stride) * kPage;
  }
  int32_t* row = table + static_cast<size_t>(b) * d.stride;
  int held = 0;
  if (grows && len % kPage) {
    const int p = row[pages_of(len) - 1];
    if (p < 0 || p >= d.num_pages) flag(err, kErrPageRange);
    else {
      held = __ldcg(ref + p);
      if (held > 1) tail = p;
      if (held <= 0) {  // a page that the search below may hand out: the row may not write on into it
        flag(err, kErrRefs);
        grows = false;
      }
    }
  }
  const int have = pages_of(grows ? len : 0), want = pages_of(grows ? to : 0);
  tails[b] = tail;
  s_growers[b] = 0;
  const bool any_shared = __syncthreads_or(tail >= 0);
  bool copy = tail >= 0;
  if (any_shared) {
    // the page's growing rows, or more (other pages may have the same hash): fewer than its holders, and nobody keeps it
    if (copy) atomicAdd(s_growers + tail % kThreads, 1);
    __syncthreads();
    if (copy && s_growers[tail % kThreads] >= held) {
      int rank = 0;  // growing rows before this one with the same shared page
      for (int j = 0; j < b; ++j) rank += tails[j] == tail;
      copy = rank != held - 1;  // every holder grows and this is the last: it keeps the page
      if (rank >= held) {       // more holders than the count knows: taking it down further would free a page that one of them keeps
        flag(err, kErrRefs);
        grows = copy = false;
      }
    }
  }
  // a row cannot get more pages than there are: the sum stays in range
  const long long need = grows ? min(static_cast<long long>(want - have) + copy, static_cast<long long>(d.num_pages) + 1) : 0;
  long long total;
  const long long first = block_scan<long long>(need, &total, red64);

  // the lowest free pages, in order, until there are `total`
  int32_t* list = total <= kSmallList ? s_list : far_list;
  long long found = 0;
  constexpr int kEach = 8;
  for (int64_t base = 0; base < d.num_pages && found < total; base += kThreads * kEach) {
    const int64_t p0 = base + static_cast<int64_t>(b) * kEach;
    uint32_t free_bits = 0;
    if (p0 + kEach <= d.num_pages && (reinterpret_cast<uintptr_t>(ref) & 15) == 0) {
      int4 r[kEach / 4];
#pragma unroll
      for (int k = 0; k < kEach / 4; ++k) r[k] = __ldcg(reinterpret_cast<const int4*>(ref + p0) + k);
#pragma unroll
      for (int k = 0; k < kEach / 4; ++k)
        free_bits |= (r[k].x == 0 ? 1u : 0u) << (4 * k) | (r[k].y == 0 ? 2u : 0u) << (4 * k) | (r[k].z == 0 ? 4u : 0u) << (4 * k) |
                     (r[k].w == 0 ? 8u : 0u) << (4 * k);
    } else {
      for (int k = 0; k < kEach; ++k)
        if (p0 + k < d.num_pages && __ldcg(ref + p0 + k) == 0) free_bits |= 1u << k;
    }
    int here;
    long long at = found + block_scan<int>(__popc(free_bits), &here, red);
    for (; free_bits && at < total; free_bits &= free_bits - 1, ++at)
      list[at] = static_cast<int32_t>(p0 + __ffs(free_bits) - 1);
    found += here;
  }
  const bool granted = grows && first + need <= found;
  if (grows && !granted) flag(err, kErrNoPages);
  __syncthreads();  // list and every read of ref above are done
  int src = -1, dst = -1;
  if (granted && copy) {
    src = tail;
    dst = list[first];
    atomicSub(ref + src, 1);
    ref[dst] = 1;
    row[have - 1] = dst;
  }
  if (b < d.num_seqs) {
    copy_src[b] = src;
    copy_dst[b] = dst;
    if (granted) lens[b] = to;
  }
  s_first[b] = first;
  s_have[b] = !granted ? INT_MIN : copy ? ~have : have;
  __syncthreads();
  // new pages: a thread a page, its row the last that starts at or before it (rows that need none start where the next does)
  const long long last = total < found ? total : found;
  for (long long k = b; k < last; k += kThreads) {
    int lo = 0, hi = kThreads - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_first[mid] <= k) lo = mid;
      else hi = mid - 1;
    }
    const int h = s_have[lo];
    if (h == INT_MIN) continue;
    const long long i = k - s_first[lo] - (h < 0 ? 1 : 0);
    if (i < 0) continue;  // the copy's
    const int p = list[k];
    table[static_cast<size_t>(lo) * d.stride + (h < 0 ? ~h : h) + i] = p;
    ref[p] = 1;
  }
}

// ---------------------------------------------------------------- compact
// Live pages of each block of 4096.
__global__ void __launch_bounds__(kThreads) pages_count_kernel(int num_pages, const int32_t* __restrict__ ref,
                                                               int32_t* __restrict__ counts) {
  chained_start();
  int n = 0;
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kPagesPerBlock;
#pragma unroll
  for (int k = 0; k < kPagesPerBlock / kThreads; ++k) {
    const int64_t p = base + k * kThreads + threadIdx.x;
    n += __syncthreads_count(p < num_pages && ref[p] > 0);
  }
  if (threadIdx.x == 0) counts[blockIdx.x] = n;
}

// Every block sums the counts for itself (n_live, its own first rank, the live pages below n_live), then ranks its
// pages: live ones at or above n_live are the sources, free ones below it the destinations.
__global__ void __launch_bounds__(kThreads) pages_rank_kernel(int num_pages, const int32_t* __restrict__ ref,
                                                              const int32_t* __restrict__ counts, int blocks,
                                                              int32_t* __restrict__ copy_src, int32_t* __restrict__ copy_dst,
                                                              int32_t* __restrict__ num_moves, int32_t* __restrict__ to) {
  chained_start();
  __shared__ int red[32];
  int sum = 0, before = 0;
  for (int c = threadIdx.x; c < blocks; c += kThreads) {
    const int n = counts[c];
    sum += n;
    if (c < static_cast<int>(blockIdx.x)) before += n;
  }
  int live, first;
  block_scan<int>(sum, &live, red);
  block_scan<int>(before, &first, red);
  const int edge = live / kPagesPerBlock;  // the block that n_live falls in
  int low = 0;
  for (int c = threadIdx.x; c < edge; c += kThreads) low += counts[c];
  for (int64_t p = static_cast<int64_t>(edge) * kPagesPerBlock + threadIdx.x; p < live; p += kThreads) low += ref[p] > 0;
  int stay;  // live pages below n_live
  block_scan<int>(low, &stay, red);
  const int moves = live - stay;
  const int64_t p0 = static_cast<int64_t>(blockIdx.x) * kPagesPerBlock + 4 * threadIdx.x;
  int n = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) n += p0 + k < num_pages && ref[p0 + k] > 0;
  int total;
  int rank = first + block_scan<int>(n, &total, red);  // live pages before p0
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t p = p0 + k;
    if (p >= num_pages) break;
    const bool is_live = ref[p] > 0;
    int t = is_live ? static_cast<int>(p) : -1;  // where the page's entries go; -1: it is free
    if (is_live && p >= live) {
      copy_src[rank - stay] = static_cast<int32_t>(p);
      t = -2 - (rank - stay);  // its destination stands at that rank
    }
    if (!is_live && p < live) copy_dst[p - rank] = static_cast<int32_t>(p);
    to[p] = t;
    rank += is_live;
  }
  for (int64_t r = moves + static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; r < num_pages / 2;
       r += static_cast<int64_t>(gridDim.x) * kThreads) {
    copy_src[r] = -1;
    copy_dst[r] = -1;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    num_moves[0] = moves;
    to[num_pages] = live;
  }
}

// Tables and counts. A thread that moves a page's count is the only one that touches the two counts, so ref_out may be ref.
__global__ void __launch_bounds__(256) pages_rewrite_kernel(PagesDesc d, const int32_t* table, const int32_t* __restrict__ lens,
                                                            const int32_t* ref, int32_t* table_out, int32_t* ref_out,
                                                            const int32_t* __restrict__ copy_dst,
                                                            const int32_t* __restrict__ to, uint32_t* err) {
  chained_start();
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x, t0 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  for (int64_t p = t0; p < d.num_pages; p += step) {
    const int t = to[p];
    if (t >= 0) {
      ref_out[p] = ref[p];
    } else if (t < -1) {
      ref_out[copy_dst[-2 - t]] = ref[p];
      ref_out[p] = 0;
    } else if (p >= to[d.num_pages]) {
      ref_out[p] = ref[p];  // a free page that stays free (below n_live it receives a mover's count)
    }
  }
  const int64_t cells = static_cast<int64_t>(d.num_seqs) * d.stride;
  for (int64_t c = t0; c < cells; c += step) {
    const int b = static_cast<int>(c / d.stride), k = static_cast<int>(c - static_cast<int64_t>(b) * d.stride);
    int p = table[c];
    const int len = lens[b];
    if (len < 0 || len > static_cast<int64_t>(d.stride) * kPage) {
      if (k == 0) flag(err, kErrLengths);
    } else if (k < pages_of(len)) {
      if (p < 0 || p >= d.num_pages) flag(err, kErrPageRange);
      else {
        const int t = to[p];
        if (t == -1) flag(err, kErrRefs);
        else if (t < -1) p = copy_dst[-2 - t];
      }
    }
    table_out[c] = p;
  }
}

// A small pool in one launch: one block, its `to` and the destinations in shared memory.
constexpr int kSmallPool = 8192, kSmallCells = 65536;

__global__ void __launch_bounds__(kThreads) pages_compact_small_kernel(PagesDesc d, const int32_t* table,
                                                                       const int32_t* __restrict__ lens, const int32_t* ref,
                                                                       int32_t* table_out, int32_t* ref_out,
                                                                       int32_t* __restrict__ copy_src,
                                                                       int32_t* __restrict__ copy_dst,
                                                                       int32_t* __restrict__ num_moves, uint32_t* err) {
  chained_start();
  constexpr int kEach = kSmallPool / kThreads;
  __shared__ int red[32];
  __shared__ int32_t s_dst[kSmallPool / 2];
  __shared__ int16_t s_to[kSmallPool];  // -1: free, -2: stays, else its rank among the movers
  const int p0 = threadIdx.x * kEach;
  int counts[kEach], n = 0;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    counts[k] = p0 + k < d.num_pages ? ref[p0 + k] : 0;
    n += counts[k] > 0;
  }
  int live, stay;
  int rank = block_scan<int>(n, &live, red);  // live pages before p0
  int low = 0;
#pragma unroll
  for (int k = 0; k < kEach; ++k) low += p0 + k < live && counts[k] > 0;
  block_scan<int>(low, &stay, red);
  const int moves = live - stay;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int p = p0 + k;
    if (p < d.num_pages) {
      const bool is_live = counts[k] > 0;
      int t = is_live ? -2 : -1;
      if (is_live && p >= live) {
        t = rank - stay;
        copy_src[t] = p;
      }
      if (!is_live && p < live) {
        s_dst[p - rank] = p;
        copy_dst[p - rank] = p;
      }
      s_to[p] = static_cast<int16_t>(t);
      rank += is_live;
    }
  }
  for (int r = moves + threadIdx.x; r < d.num_pages / 2; r += kThreads) {
    copy_src[r] = -1;
    copy_dst[r] = -1;
  }
  if (threadIdx.x == 0) num_moves[0] = moves;
  __syncthreads();  // every count has been read: ref_out may be ref
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int p = p0 + k;
    if (p < d.num_pages) {
      const int t = s_to[p];
      if (t >= 0) {
        ref_out[s_dst[t]] = counts[k];
        ref_out[p] = 0;
      } else if (t == -2 || p >= live) {
        ref_out[p] = counts[k];
      }
    }
  }
  const int cells = d.num_seqs * d.stride;
  for (int c = threadIdx.x; c < cells; c += kThreads) {
    const int b = c / d.stride, k = c - b * d.stride;
    int p = table[c];
    const int len = lens[b];
    if (len < 0 || len > static_cast<int64_t>(d.stride) * kPage) {
      if (k == 0) flag(err, kErrLengths);
    } else if (k < pages_of(len)) {
      if (p < 0 || p >= d.num_pages) flag(err, kErrPageRange);
      else if (s_to[p] == -1) flag(err, kErrRefs);
      else if (s_to[p] >= 0) p = s_dst[s_to[p]];
    }
    table_out[c] = p;
  }
}

// ---------------------------------------------------------------- copy
__global__ void __launch_bounds__(128) pages_copy_kernel(PoolCopy c) {
  chained_start();
  int n = c.max_pairs;
  if (c.num_pairs) n = min(n, *c.num_pairs);
  const int per = 2 * c.layers;  // K and V of each layer
  const int64_t items = static_cast<int64_t>(n) * per;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int i = static_cast<int>(it / per), which = static_cast<int>(it - static_cast<int64_t>(i) * per);
    const int src = c.src[i], dst = c.dst[i];
    if (src < 0 || dst < 0) continue;
    if (src >= c.num_pages || dst >= c.num_pages) {
      if (threadIdx.x == 0) flag(c.err, kErrPageRange);
      continue;
    }
    const uint4* from = static_cast<const uint4*>(c.data[which]) + static_cast<size_t>(src) * c.page_units;
    uint4* to = static_cast<uint4*>(c.data[which]) + static_cast<size_t>(dst) * c.page_units;
    for (int u = threadIdx.x; u < c.page_units; u += blockDim.x) to[u] = from[u];
    if (c.scale_units) {
      const uint4* sf = reinterpret_cast<const uint4*>(c.scale[which]) + static_cast<size_t>(src) * c.scale_units;
      uint4* st = reinterpret_cast<uint4*>(c.scale[which]) + static_cast<size_t>(dst) * c.scale_units;
      for (int u = threadIdx.x; u < c.scale_units; u += blockDim.x) st[u] = sf[u];
    }
  }
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

// Workspace: resize's ticket (256 bytes), then one int per page (+ 1): resize's list of free pages, or compact's `to` with n_live behind it;
// then compact's counts.
size_t pages_workspace_bytes(const PagesDesc& d) {
  const size_t blocks = (static_cast<size_t>(d.num_pages) + kPagesPerBlock - 1) / kPagesPerBlock;
  return 4 * kTicketInts + up256((static_cast<size_t>(d.num_pages) + 1) * 4) + up256(4 * blocks);
}

cudaError_t launch_pages_fork(const PagesDesc& d, int32_t* table, int32_t* lens, int32_t* ref, const int32_t* parents,
                              const int32_t* children, int n, uint32_t* err, cudaStream_t stream) {
  return launch_chained(pages_fork_kernel, n, 256, 0, stream, d, table, lens, ref, parents, children, n, err);
}

cudaError_t launch_pages_resize(const PagesDesc& d, int32_t* table, int32_t* lens, int32_t* ref, const int32_t* new_lens,
                                int32_t* copy_src, int32_t* copy_dst, uint32_t* err, void* ws, cudaStream_t stream) {
  const bool small = static_cast<int64_t>(d.num_seqs) * d.stride <= 16384;
  const int grid = small ? 1 : d.num_seqs < 304 ? d.num_seqs : 304;  // at most two blocks for each of GB300's 152 SMs
  return launch_chained(pages_resize_kernel, grid, kThreads, 0, stream, d, table, lens, ref, new_lens, copy_src, copy_dst, err,
                                                     static_cast<uint32_t*>(ws), static_cast<int32_t*>(ws) + kTicketInts);
}

cudaError_t launch_pages_compact(const PagesDesc& d, const int32_t* table, const int32_t* lens, const int32_t* ref,
                                 int32_t* table_out, int32_t* ref_out, int32_t* copy_src, int32_t* copy_dst,
                                 int32_t* num_moves, uint32_t* err, void* ws, cudaStream_t stream) {
  if (d.num_pages <= kSmallPool && static_cast<int64_t>(d.num_seqs) * d.stride <= kSmallCells) {
    return launch_chained(pages_compact_small_kernel, 1, kThreads, 0, stream, d, table, lens, ref, table_out, ref_out, copy_src, copy_dst, num_moves, err);
  }
  const int blocks = static_cast<int>((static_cast<int64_t>(d.num_pages) + kPagesPerBlock - 1) / kPagesPerBlock);
  int32_t* to = static_cast<int32_t*>(ws) + kTicketInts;
  int32_t* counts = reinterpret_cast<int32_t*>(reinterpret_cast<uint8_t*>(to) + up256((static_cast<size_t>(d.num_pages) + 1) * 4));
  cudaError_t e = launch_chained(pages_count_kernel, blocks, kThreads, 0, stream, d.num_pages, ref, counts);
  if (e != cudaSuccess) return e;
  e = launch_chained(pages_rank_kernel, blocks, kThreads, 0, stream, d.num_pages, ref, counts, blocks, copy_src, copy_dst, num_moves, to);
  if (e != cudaSuccess) return e;
  const int64_t work = static_cast<int64_t>(d.num_seqs) * d.stride + d.num_pages;
  const int grid = static_cast<int>(work / 256 + 1 < 2048 ? work / 256 + 1 : 2048);
  return launch_chained(pages_rewrite_kernel, grid, 256, 0, stream, d, table, lens, ref, table_out, ref_out, copy_dst, to, err);
}

cudaError_t launch_pages_copy(const PoolCopy& c, cudaStream_t stream) {
  const int64_t items = static_cast<int64_t>(c.max_pairs) * 2 * c.layers;
  const int grid = static_cast<int>(items < 4096 ? items : 4096);
  return launch_chained(pages_copy_kernel, grid, 128, 0, stream, c);
}

}  // namespace pav
