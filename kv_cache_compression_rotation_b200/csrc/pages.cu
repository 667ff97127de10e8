// Pages of a cache: reference counts, allocation, forks, compaction and the copies they need.
//
// A page is free while its count is 0.  Allocation takes the free pages of the lowest ids in the
// order of the requests, so a call's result depends on its arguments alone; there is no free list
// to keep in step.  Ranks of free (or live) pages come from counts of chunks of 4096 pages, then
// from a scan inside the chunk.  A call that cannot be served whole (too few free pages, a bad or
// repeated row, a source row that lacks pages) changes nothing: the kernel that would change something
// first sees the counts of all chunks and the verdict on all requests, which the kernel before it wrote.
//
// The bookkeeping reads 4 bytes a page and is bound by launch and memory latency; the copies are
// bound by bytes, 2 a byte moved, and go in slices of 16 KB with four 16-byte loads in flight a
// thread.  Pools of up to 16384 pages take one block of 1024 threads, which holds all counts in its
// registers and the requests in shared memory, in place of the counting and the assigning kernel.
// Measured: 48 children of 16 parents of some 45 pages freed and forked 13 us, 144 of 48 parents of some
// 90 pages 19 us (11 and 15 without the look through the source rows' entries; 20 us with the counting and
// the assigning kernel), 0.8 GB moved by a compaction 290 us, 5.7 TB/s.
#include "pages.h"

#include <algorithm>

#include "device_common.cuh"
#include "launchers.h"

namespace tq {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = kPageChunk / kThreads;  // counts a thread
constexpr int kSmallThreads = 1024;
constexpr int kSmallPages = kSmallThreads * kPer, kSmallRequests = 2048, kSmallRows = 16384;
// Source entries of a fork (requests x columns of the table) that one block looks through; their number in a
// row is kept in 16 bits.  One block / the three kernels, freed and forked: 32639 entries 17 / 22 us, 65535
// entries 21.5 / 21.7, 131327 entries 31 / 23.
constexpr int kSmallEntries = 65535;
static_assert(kCheckBlocks <= kThreads, "a thread reads one verdict");

// Sum over the block; every thread gets it.
template <int N = kThreads, typename T>
__device__ __forceinline__ T block_sum(T x, T* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  __syncthreads();
  if (lane == 0) sh[warp] = x;
  __syncthreads();
  T t = 0;
#pragma unroll
  for (int w = 0; w < N / 32; ++w) t += sh[w];
  return t;
}

// Sum over the threads before this one.
template <typename T>
__device__ __forceinline__ T block_before(T x, T* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = s;
  __syncthreads();
  T t = s - x;
  for (int w = 0; w < warp; ++w) t += sh[w];
  return t;
}

// Pages that requests want (their sum may pass 32 bits); no pool has as many as INT32_MAX.
using Wanted = long long;
__device__ __forceinline__ int pages_wanted(Wanted n) { return static_cast<int>(min(n, static_cast<Wanted>(INT32_MAX))); }

__device__ __forceinline__ int pages_of(int len, int page) { return (len + page - 1) / page; }

// Counts of this thread's pages p0 .. p0 + kPer - 1 (pages past the pool count as live).
__device__ __forceinline__ void load_refs(const tq_page_pool& pool, int64_t p0, int (&r)[kPer]) {
  if (p0 + kPer <= pool.num_pages) {
#pragma unroll
    for (int k = 0; k < kPer; k += 4) {
      const int4 v = *reinterpret_cast<const int4*>(pool.refs + p0 + k);
      r[k] = v.x; r[k + 1] = v.y; r[k + 2] = v.z; r[k + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < kPer; ++k) r[k] = p0 + k < pool.num_pages ? pool.refs[p0 + k] : 1;
  }
}

__device__ __forceinline__ int count_free(const int (&r)[kPer]) {
  int n = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) n += r[k] <= 0;
  return n;
}

// Marks row `r` of bitmap `m`; true if it was marked before.
__device__ __forceinline__ bool mark(uint32_t* m, int r) {
  const uint32_t bit = 1u << (r & 31);
  return atomicOr(m + (r >> 5), bit) & bit;
}

// Request i: its row, what it wants of it, and whether it is in range.
template <bool FORK>
__device__ __forceinline__ bool request(const PagesParams& p, int i, int& row, int& src, int& want) {
  const int cap = p.pool.max_pages * p.pool.page_size, len = p.lens[i];
  row = p.rows[i];
  want = src = 0;
  if (row < 0 || row >= p.pool.rows || len < 0 || len > cap) return false;
  if (FORK) {
    src = p.src[i];
    want = len % p.pool.page_size ? 1 : 0;
    return src >= 0 && src < p.pool.rows;
  }
  const int old = p.old_lens[i];
  want = max(0, pages_of(len, p.pool.page_size) - pages_of(old, p.pool.page_size));
  return old >= 0 && old <= cap;
}

// The last block: what the requests want, and whether they can be served at all.
template <bool FORK>
__device__ void scan_requests(const PagesParams& p) {
  __shared__ Wanted sh[kThreads / 32];
  __shared__ int bad;
  const int words = (p.pool.rows + 31) / 32;
  if (threadIdx.x == 0) bad = 0;
  for (int i = threadIdx.x; i < 2 * words; i += kThreads) p.marks[i] = 0;
  __syncthreads();
  Wanted run = 0;
  for (int i0 = 0; i0 < p.n; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    int want = 0;
    if (i < p.n) {
      int row, src;
      const bool ok = request<FORK>(p, i, row, src, want);
      if (!ok) want = 0;
      if (FORK && ok) mark(p.marks + words, src);
      if (!ok || mark(p.marks, row)) atomicOr(&bad, 1);
    }
    const Wanted before = block_before(static_cast<Wanted>(want), sh);
    if (i < p.n) p.prefix[i] = pages_wanted(run + before);
    run += block_sum(static_cast<Wanted>(want), sh);
  }
  __syncthreads();
  if (FORK)                                  // a row that is made must not be copied from too
    for (int i = threadIdx.x; i < words; i += kThreads)
      if (p.marks[i] & p.marks[words + i]) atomicOr(&bad, 1);
  __syncthreads();
  if (threadIdx.x == 0) p.prefix[p.n] = bad ? -1 : pages_wanted(run);
}

enum : int { COUNT_FORK = 0, COUNT_RESERVE = 1, COUNT_COMPACT = 2 };

// Blocks: the chunks, one for the requests, and for a fork those that look through the source rows.
template <int MODE>
__global__ void __launch_bounds__(kThreads) count_kernel(const PagesParams p) {
  __shared__ int sh[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  if (MODE != COUNT_COMPACT && static_cast<int>(blockIdx.x) == p.chunks) {
    scan_requests<MODE == COUNT_FORK>(p);
    return;
  }
  if (MODE == COUNT_FORK && static_cast<int>(blockIdx.x) > p.chunks) {
    const int first = blockIdx.x - p.chunks - 1;
    bool ok = true;
    for (int i = first; i < p.n; i += kCheckBlocks) {
      int row, src, want;
      if (!request<true>(p, i, row, src, want)) continue;        // (refused by the block of the requests)
      const int used = pages_of(p.lens[i], p.pool.page_size);
      const int32_t* from = p.pool.block_table + static_cast<int64_t>(src) * p.pool.max_pages;
#pragma unroll 4
      for (int c = threadIdx.x; c < used; c += kThreads) {
        const int id = from[c];
        ok &= id >= 0 && id < p.pool.num_pages && p.pool.refs[id] > 0;
      }
    }
    const int bad = __syncthreads_or(!ok);
    if (threadIdx.x == 0) p.bad[first] = bad;
    return;
  }
  int r[kPer];
  load_refs(p.pool, static_cast<int64_t>(blockIdx.x) * kPageChunk + threadIdx.x * kPer, r);
  const int n = block_sum(count_free(r), sh);
  if (threadIdx.x == 0) p.chunk_free[blockIdx.x] = n;
}

// Free pages of the chunks before `chunk`, and of all.
__device__ __forceinline__ void chunk_sums(const PagesParams& p, int chunk, int* sh, int& before, int& all) {
  int b = 0, a = 0;
  for (int c = threadIdx.x; c < p.chunks; c += kThreads) {
    const int n = p.chunk_free[c];
    a += n;
    if (c < chunk) b += n;
  }
  before = block_sum(b, sh);
  all = block_sum(a, sh);
}

// Request i of a fork: its row shares the parent's whole pages (one block).
__device__ __forceinline__ void share_pages(const PagesParams& p, int i) {
  const tq_page_pool& pool = p.pool;
  const int full = p.lens[i] / pool.page_size;
  const int32_t* from = pool.block_table + static_cast<int64_t>(p.src[i]) * pool.max_pages;
  int32_t* to = pool.block_table + static_cast<int64_t>(p.rows[i]) * pool.max_pages;
  for (int c = threadIdx.x; c < full; c += kThreads) {
    const int id = from[c];
    to[c] = id;
    atomicAdd(pool.refs + id, 1);
  }
}

// The page that request i of a fork copies (-1: none).
__device__ __forceinline__ int tail_page(const PagesParams& p, int i) {
  const tq_page_pool& pool = p.pool;
  const int len = p.lens[i];
  return len % pool.page_size ? pool.block_table[static_cast<int64_t>(p.src[i]) * pool.max_pages + len / pool.page_size] : -1;
}

// Gives page `id`, of rank `rank` among the free ones, to the request that wants it.
template <bool FORK>
__device__ __forceinline__ void hand_out(const PagesParams& p, const int* prefix, int rank, int id) {
  const tq_page_pool& pool = p.pool;
  int lo = 0, hi = p.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= rank) lo = mid; else hi = mid - 1;
  }
  const int col = FORK ? p.lens[lo] / pool.page_size : pages_of(p.old_lens[lo], pool.page_size) + rank - prefix[lo];
  pool.block_table[static_cast<int64_t>(p.rows[lo]) * pool.max_pages + col] = id;
  pool.refs[id] = 1;
  if (FORK) p.to[lo] = id;
}

// Small pools: counts, requests and pages in one block.  A fork leaves prefix[n] = -1 where it changes
// nothing.
template <bool FORK>
__global__ void __launch_bounds__(kSmallThreads, 1) small_assign_kernel(const PagesParams p) {
  __shared__ Wanted sh_wanted[kSmallThreads / 32];
  __shared__ int sh[kSmallThreads / 32], prefix[kSmallRequests];
  __shared__ uint32_t marks[2][kSmallRows / 32];
  __shared__ uint16_t free_ids[kSmallPages];
  __shared__ uint16_t in_use[kSmallThreads];   // bit k of word t: page t * kPer + k
  __shared__ int bad;
  // (before free_ids is filled) a fork's source rows, and how many of their pages it asks for
  uint16_t* srcs = free_ids;
  uint16_t* used = free_ids + kSmallRequests;
  const int tid = threadIdx.x, words = (p.pool.rows + 31) / 32;
  for (int i = tid; i < words; i += kSmallThreads) marks[0][i] = marks[1][i] = 0;
  if (tid == 0) bad = 0;
  pdl_wait();
  pdl_trigger();
  int r[kPer];
  const int64_t p0 = tid * kPer;
  load_refs(p.pool, p0, r);
  if (FORK) {
    uint32_t bits = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) bits |= (r[k] > 0 ? 1u : 0u) << k;
    in_use[tid] = static_cast<uint16_t>(bits);
  }
  __syncthreads();
  Wanted sum = 0;
  for (int i0 = 0; i0 < p.n; i0 += kSmallThreads) {
    const int i = i0 + tid;
    int row = 0, src = 0, want = 0;
    if (i < p.n) {
      const bool ok = request<FORK>(p, i, row, src, want);
      if (!ok) want = 0;
      if (FORK) {
        if (ok) mark(marks[1], src);
        srcs[i] = static_cast<uint16_t>(src);
        used[i] = static_cast<uint16_t>(ok ? pages_of(p.lens[i], p.pool.page_size) : 0);
      }
      if (!ok || mark(marks[0], row)) bad = 1;
    }
    const Wanted before = block_before(static_cast<Wanted>(want), sh_wanted);
    if (i < p.n) prefix[i] = pages_wanted(sum + before);
    sum += block_sum<kSmallThreads>(static_cast<Wanted>(want), sh_wanted);
  }
  const int need = pages_wanted(sum);
  __syncthreads();
  if (FORK)                                  // a row that is made must not be copied from too
    for (int i = tid; i < words; i += kSmallThreads)
      if (marks[0][i] & marks[1][i]) bad = 1;
  if (FORK) {                                // every source row holds what it is asked for
    // A warp takes two requests at a time, four steps of 32 entries of each, whose loads are in flight together.
    constexpr int kWarps = kSmallThreads / 32;
    bool ok = true;
    for (int i = tid / 32; i < p.n; i += 2 * kWarps) {
      const int i2 = min(i + kWarps, p.n - 1), n0 = used[i], n1 = used[i2];
      const int32_t* from0 = p.pool.block_table + static_cast<int64_t>(srcs[i]) * p.pool.max_pages;
      const int32_t* from1 = p.pool.block_table + static_cast<int64_t>(srcs[i2]) * p.pool.max_pages;
      for (int c = tid % 32; c < max(n0, n1); c += 128) {
        int id[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          id[k] = c + 32 * k < n0 ? from0[c + 32 * k] : 0;
          id[4 + k] = c + 32 * k < n1 ? from1[c + 32 * k] : 0;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (c + 32 * (k & 3) < (k < 4 ? n0 : n1))
            ok &= id[k] >= 0 && id[k] < p.pool.num_pages && (in_use[id[k] / kPer] >> id[k] % kPer & 1);
      }
    }
    if (!ok) bad = 1;
  }
  const int mine = count_free(r);
  int rank = block_before(mine, sh);
  const int all = block_sum<kSmallThreads>(mine, sh);
  const bool refused = bad, short_of = refused || all < need;        // (block_sum's barriers stand between)
  if (tid == 0) {
    *p.shortfall = refused ? -1 : max(0, need - all);
    if (refused) report_status(p.status, TQ_ERR_INVALID_ARG);
    if (FORK) p.prefix[p.n] = short_of ? -1 : need;
  }
  if (short_of) return;
#pragma unroll
  for (int k = 0; k < kPer; ++k)
    if (r[k] <= 0) {
      if (rank < need) free_ids[rank] = static_cast<uint16_t>(p0 + k);
      ++rank;
    }
  if (FORK)
    for (int i = tid; i < p.n; i += kSmallThreads) {
      p.from[i] = tail_page(p, i);
      if (p.lens[i] % p.pool.page_size == 0) p.to[i] = -1;
    }
  __syncthreads();
  for (int k = tid; k < need; k += kSmallThreads) hand_out<FORK>(p, prefix, k, free_ids[k]);
}

// Blocks 0 .. chunks - 1 hand out the free pages of their chunk; fork has one more block a
// request, which shares the parent's whole pages.
template <bool FORK>
__global__ void __launch_bounds__(kThreads) assign_kernel(const PagesParams p) {
  __shared__ int sh[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const tq_page_pool& pool = p.pool;
  int need = p.prefix[p.n];
  if (FORK && __syncthreads_or(static_cast<int>(threadIdx.x) < min(p.n, kCheckBlocks) && p.bad[threadIdx.x])) need = -1;
  int before, all;
  chunk_sums(p, blockIdx.x, sh, before, all);
  const bool short_of = need < 0 || all < need;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *p.shortfall = need < 0 ? -1 : max(0, need - all);
    if (need < 0) report_status(p.status, TQ_ERR_INVALID_ARG);
  }
  if (FORK && static_cast<int>(blockIdx.x) >= p.chunks) {
    const int i = blockIdx.x - p.chunks;
    const int len = p.lens[i];
    if (short_of) {
      if (threadIdx.x == 0) p.to[i] = -1;
      return;
    }
    share_pages(p, i);
    if (threadIdx.x == 0) {
      p.from[i] = tail_page(p, i);
      if (len % p.pool.page_size == 0) p.to[i] = -1;
    }
    return;
  }
  if (short_of || before >= need) return;
  int r[kPer];
  const int64_t p0 = static_cast<int64_t>(blockIdx.x) * kPageChunk + threadIdx.x * kPer;
  load_refs(pool, p0, r);
  int rank = before + block_before(count_free(r), sh);
#pragma unroll 1
  for (int k = 0; k < kPer && rank < need; ++k)
    if (r[k] <= 0) hand_out<FORK>(p, p.prefix, rank++, static_cast<int>(p0 + k));
}

__global__ void __launch_bounds__(kThreads) free_kernel(const PagesParams p) {
  pdl_wait();
  pdl_trigger();
  const tq_page_pool& pool = p.pool;
  const int i = blockIdx.x, row = p.rows[i], cap = pool.max_pages * pool.page_size;
  int len = p.lens[i];
  if (row < 0 || row >= pool.rows || len < 0 || len > cap) {
    if (threadIdx.x == 0) report_status(p.status, TQ_ERR_INVALID_ARG);
    return;
  }
  const int used = pages_of(len, pool.page_size);
  for (int c = threadIdx.x; c < used; c += kThreads) {
    // a row that is named twice gives its pages back once
    const int id = atomicExch(pool.block_table + static_cast<int64_t>(row) * pool.max_pages + c, -1);
    if (id == -1) continue;
    if (id < 0 || id >= pool.num_pages) {
      report_status(p.status, TQ_ERR_INVALID_ARG);
    } else if (atomicSub(pool.refs + id, 1) <= 0) {
      atomicAdd(pool.refs + id, 1);          // it was free already
      report_status(p.status, TQ_ERR_INVALID_ARG);
    }
  }
}

// Compaction, pass 2: with L live pages, the live ones at ids >= L move, in their order, to the
// free ids below L in theirs.  map: own id, -1 (free), or -2 - j for the j-th page that moves.
__global__ void __launch_bounds__(kThreads) compact_plan_kernel(const PagesParams p) {
  __shared__ int sh[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const tq_page_pool& pool = p.pool;
  int before, all;
  chunk_sums(p, blockIdx.x, sh, before, all);
  const int64_t L = pool.num_pages - all;    // live pages
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.live = static_cast<int>(L);
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kPageChunk, p0 = c0 + threadIdx.x * kPer;
  // free pages below L: those of the chunks before L's, and of the part of L's chunk
  int low_free = 0;
  if (c0 + kPageChunk > L) {
    const int lc = static_cast<int>(min(L / kPageChunk, static_cast<int64_t>(p.chunks)));
    int n = 0;
    for (int c = threadIdx.x; c < lc; c += kThreads) n += p.chunk_free[c];
    for (int64_t q = static_cast<int64_t>(lc) * kPageChunk + threadIdx.x; q < L; q += kThreads) n += pool.refs[q] <= 0;
    low_free = block_sum(n, sh);
  }
  int r[kPer];
  load_refs(pool, p0, r);
  int frank = before + block_before(count_free(r), sh);       // free pages before p0
#pragma unroll 1
  for (int k = 0; k < kPer && p0 + k < pool.num_pages; ++k) {
    const int64_t id = p0 + k;
    int m = -1;
    if (r[k] > 0) {
      m = static_cast<int>(id);
      if (id >= L) {
        const int j = static_cast<int>(id - frank - (L - low_free));
        p.from[j] = static_cast<int>(id);
        m = -2 - j;
      }
    } else {
      if (id < L) p.to[frank] = static_cast<int>(id);
      ++frank;
    }
    p.page_map[id] = m;
  }
}

// Compaction of a small pool, both passes in one block.  live: live pages; chunk_free[0]: pages that move.
__global__ void __launch_bounds__(kSmallThreads) small_compact_kernel(const PagesParams p) {
  __shared__ int sh[kSmallThreads / 32];
  pdl_wait();
  pdl_trigger();
  const tq_page_pool& pool = p.pool;
  int r[kPer];
  const int64_t p0 = threadIdx.x * kPer;
  load_refs(pool, p0, r);
  const int mine = count_free(r);
  int frank = block_before(mine, sh);
  const int L = static_cast<int>(pool.num_pages) - block_sum<kSmallThreads>(mine, sh);
  int low = 0;                               // free pages below L
#pragma unroll
  for (int k = 0; k < kPer; ++k) low += r[k] <= 0 && p0 + k < L;
  const int low_free = block_sum<kSmallThreads>(low, sh);
  if (threadIdx.x == 0) {
    *p.live = L;
    p.chunk_free[0] = low_free;
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int id = static_cast<int>(p0) + k;
    if (id >= pool.num_pages) break;
    int m = -1;
    if (r[k] > 0) {
      m = id;
      if (id >= L) {
        const int j = id - frank - (L - low_free);
        p.from[j] = id;
        m = -2 - j;
      }
    } else {
      if (id < L) p.to[frank] = id;
      ++frank;
    }
    p.page_map[id] = m;
  }
}

template <typename V, int N>
__device__ __forceinline__ void copy_units(V* dst, const V* src, int units) {
  int i = threadIdx.x;
  for (; i + (N - 1) * kThreads < units; i += N * kThreads) {
    V v[N];
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = __ldcs(src + i + k * kThreads);
#pragma unroll
    for (int k = 0; k < N; ++k) __stcs(dst + i + k * kThreads, v[k]);
  }
  for (; i < units; i += kThreads) dst[i] = src[i];
}

enum : int { COPY_LIST = 0, COPY_FORK = 1, COPY_COMPACT = 2, COPY_SMALL_FORK = 3, COPY_SMALL_COMPACT = 4 };

// Moves the pages of the pairs in from / to, one slice of one array a step.
template <int KIND>
__global__ void __launch_bounds__(kThreads) copy_kernel(const PagesParams p) {
  constexpr int MODE = KIND == COPY_SMALL_FORK ? COPY_FORK : KIND == COPY_SMALL_COMPACT ? COPY_COMPACT : KIND;
  pdl_wait();
  pdl_trigger();
  const int64_t n_pages = p.pool.num_pages;
  int64_t pairs = p.n;
  if (KIND == COPY_SMALL_FORK) {
    if (p.prefix[p.n] < 0) return;
    for (int i = blockIdx.x; i < p.n; i += gridDim.x) share_pages(p, i);
  }
  if (KIND == COPY_SMALL_COMPACT) pairs = p.chunk_free[0];
  if (KIND == COPY_COMPACT) {
    // pages that move: free pages below the live count
    __shared__ int sh[kThreads / 32];
    const int64_t L = *p.live;
    const int lc = static_cast<int>(L / kPageChunk);
    int n = 0;
    for (int c = threadIdx.x; c < lc; c += kThreads) n += p.chunk_free[c];
    for (int64_t q = static_cast<int64_t>(lc) * kPageChunk + threadIdx.x; q < L; q += kThreads) {
      // the counts are being moved by other blocks; the map is not, for pages below L
      n += p.page_map[q] == -1;
    }
    pairs = block_sum(n, sh);
  }
  if (MODE == COPY_COMPACT) {
    // entries of the table, by the map (-2 - j: the page that pair j leads to)
    const int64_t entries = static_cast<int64_t>(p.pool.rows) * p.pool.max_pages;
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; e < entries;
         e += static_cast<int64_t>(gridDim.x) * kThreads) {
      const int id = p.pool.block_table[e];
      if (id < 0) continue;
      if (id >= n_pages) { report_status(p.status, TQ_ERR_INVALID_ARG); continue; }
      int m = *static_cast<volatile int32_t*>(p.page_map + id);
      if (m <= -2) m = p.to[-2 - m];
      if (m != id) p.pool.block_table[e] = m;
    }
    // counts and map of the pages that move, whether or not the pool has arrays
    for (int64_t j = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; j < pairs;
         j += static_cast<int64_t>(gridDim.x) * kThreads) {
      const int from = p.from[j], to = p.to[j];
      p.pool.refs[to] = p.pool.refs[from];
      p.pool.refs[from] = 0;
      *static_cast<volatile int32_t*>(p.page_map + from) = to;
    }
  }
  const int slices = p.copy.slice0[p.copy.n];
  for (int64_t w = blockIdx.x; w < pairs * slices; w += gridDim.x) {
    const int64_t j = w / slices;
    const int s = static_cast<int>(w - j * slices);
    int from, to;
    if (MODE == COPY_LIST) { from = p.src[j]; to = p.rows[j]; }
    else { to = p.to[j]; from = MODE == COPY_FORK && to < 0 ? -1 : p.from[j]; }
    if (MODE == COPY_FORK && to < 0) continue;
    if (from < 0 || from >= n_pages || to < 0 || to >= n_pages) {
      if (threadIdx.x == 0) report_status(p.status, TQ_ERR_INVALID_ARG);
      continue;
    }
    if (from == to) continue;
    int a = 0;
    while (s >= p.copy.slice0[a + 1]) ++a;
    const int64_t pb = p.copy.page_bytes[a], off = static_cast<int64_t>(s - p.copy.slice0[a]) * kCopySlice;
    const int bytes = static_cast<int>(min(pb - off, static_cast<int64_t>(kCopySlice)));
    char* dst = p.copy.data[a] + to * pb + off;
    const char* src = p.copy.data[a] + from * pb + off;
    if (pb % 16 == 0) copy_units<uint4, 4>(reinterpret_cast<uint4*>(dst), reinterpret_cast<const uint4*>(src), bytes / 16);
    else copy_units<uint32_t, 4>(reinterpret_cast<uint32_t*>(dst), reinterpret_cast<const uint32_t*>(src), bytes / 4);
  }
}

// Blocks of a copy: all slices (or rounds of the lists, where there are no arrays) where they are few,
// else eight an SM.
unsigned copy_grid(int64_t pairs, const PagesParams& p, int sms) {
  const int64_t all = std::max<int64_t>(pairs * p.copy.slice0[p.copy.n], (pairs + kThreads - 1) / kThreads);
  return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(all, 8ll * sms)));
}

}  // namespace

cudaError_t launch_pages_free(const PagesParams& p, cudaStream_t s) {
  return launch_pdl(free_kernel, dim3(p.n), dim3(kThreads), 0, s, p);
}

// One block does it (small_assign_kernel).
static bool is_small(const PagesParams& p) {
  return p.pool.num_pages <= kSmallPages && p.n <= kSmallRequests && p.pool.rows <= kSmallRows &&
         (!p.src || static_cast<int64_t>(p.n) * p.pool.max_pages <= kSmallEntries);
}

cudaError_t launch_pages_reserve(const PagesParams& p, cudaStream_t s) {
  if (is_small(p)) return launch_pdl(small_assign_kernel<false>, dim3(1), dim3(kSmallThreads), 0, s, p);
  cudaError_t e = launch_pdl(count_kernel<COUNT_RESERVE>, dim3(p.chunks + 1), dim3(kThreads), 0, s, p);
  return e != cudaSuccess ? e : launch_pdl(assign_kernel<false>, dim3(p.chunks), dim3(kThreads), 0, s, p);
}

cudaError_t launch_pages_fork(const PagesParams& p, int sms, cudaStream_t s) {
  if (is_small(p)) {
    cudaError_t e = launch_pdl(small_assign_kernel<true>, dim3(1), dim3(kSmallThreads), 0, s, p);
    const unsigned grid = std::max(copy_grid(p.n, p, sms), std::min(static_cast<unsigned>(p.n), 8u * sms));
    return e != cudaSuccess ? e : launch_pdl(copy_kernel<COPY_SMALL_FORK>, dim3(grid), dim3(kThreads), 0, s, p);
  }
  cudaError_t e = launch_pdl(count_kernel<COUNT_FORK>, dim3(p.chunks + 1 + std::min(p.n, kCheckBlocks)), dim3(kThreads), 0, s, p);
  if (e == cudaSuccess) e = launch_pdl(assign_kernel<true>, dim3(p.chunks + p.n), dim3(kThreads), 0, s, p);
  if (e == cudaSuccess) e = launch_pdl(copy_kernel<COPY_FORK>, dim3(copy_grid(p.n, p, sms)), dim3(kThreads), 0, s, p);
  return e;
}

cudaError_t launch_pages_compact(const PagesParams& p, int sms, cudaStream_t s) {
  const unsigned grid = copy_grid(p.pool.num_pages / 2 + 1, p, sms);
  if (p.pool.num_pages <= kSmallPages) {
    cudaError_t e = launch_pdl(small_compact_kernel, dim3(1), dim3(kSmallThreads), 0, s, p);
    return e != cudaSuccess ? e : launch_pdl(copy_kernel<COPY_SMALL_COMPACT>, dim3(grid), dim3(kThreads), 0, s, p);
  }
  cudaError_t e = launch_pdl(count_kernel<COUNT_COMPACT>, dim3(p.chunks), dim3(kThreads), 0, s, p);
  if (e == cudaSuccess) e = launch_pdl(compact_plan_kernel, dim3(p.chunks), dim3(kThreads), 0, s, p);
  if (e == cudaSuccess) e = launch_pdl(copy_kernel<COPY_COMPACT>, dim3(grid), dim3(kThreads), 0, s, p);
  return e;
}

cudaError_t launch_pages_copy(const PagesParams& p, int sms, cudaStream_t s) {
  return launch_pdl(copy_kernel<COPY_LIST>, dim3(copy_grid(p.n, p, sms)), dim3(kThreads), 0, s, p);
}

}  // namespace tq
