// pages.cu -- the pages of a paged cache: taking and freeing (cp_pages_resize),
// forking (cp_pages_fork), compacting (cp_pages_compact) and copying
// (cp_pages_copy): C ABI and kernels.
//
// The state is two sorts of arrays on the device: refs[page], how many table
// entries hold the page (0: it is free), and tables with their rows' counts of
// pages.  There is no list of free pages: the k-th page that a call takes is
// the k-th free one by number, found by counting the zeros of refs.  So results
// hang neither on the order of threads nor on the calls' history, and counts
// are changed by integer atomics alone.
//
// The three calls that change tables are bound by latency: dependent loads, code
// that runs once, and a count of refs (4 bytes a page).  Each is one cluster of
// CTAs, so that its steps are separated by the cluster's hardware barrier, not by
// launches, and their counts are exchanged through distributed shared memory.
// refs is cut into up to 2048 chunks, dealt out among the warps in turn, as the
// free pages of the lowest numbers lie together; their finders only list them,
// and all threads of the CTA place them in the tables (in one stretch a warp, and placed where
// they are found, 30K pages of a million took 57 us).  In a graph: 64 rows and
// 16K pages 5.3 us a call, 4096 rows and a million pages 11.0, of which letting
// go and taking 20K pages.
//
// The copies are bound by memory: a compaction that moves 1.0 GB in pages of 131
// KB takes 313 us in all (0.98 of a copy's rate), in 20 blocks of 2048 pieces of
// 16 bytes an SM; in 8 an SM, of which some end late, 324.
#include <cuda_runtime.h>

#include <climits>

#define CP_TU_ID ::cpattn::kTuPages
#include "host.h"
#include "paged.cuh"

namespace cpattn {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kMaxTableRows = kMaxEntries;
constexpr int kChunks = 2 * kThreads;  // of refs, at most
constexpr int kList = 16384;   // pages that a call places at a time
constexpr int kQueue = 1024;

// Shared memory of a CTA.
struct PagesShared {
  int start[kMaxTableRows + 1];  // pages that the rows before take
  int warp_sums[kWarps];
  int free_before[kChunks + 1];  // free pages in the chunks before
  int counts[kChunks];           // free pages of this CTA's chunks: number i is chunk i * cluster + rank
  int moved, need;               // what one CTA has found and tells the others
  int queued, queue[kQueue];     // rows with many pages to let go
  int listed;
  int2 list[kList + 256];        // free pages that this CTA has found, and how many lie before each
};
extern __shared__ __align__(16) unsigned char pages_shared[];

__device__ __forceinline__ int cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return static_cast<int>(r);
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// All threads of the cluster; what they wrote before, to global memory too, is
// seen after (read past L1 where this kernel itself has written).
__device__ __forceinline__ void cluster_barrier(int cluster) {
  if (cluster == 1) {
    __syncthreads();
  } else {
    cluster_arrive();
    cluster_wait();
  }
}
// What is at the address of `local` in the shared memory of CTA `rank`; v to it.
__device__ __forceinline__ int ld_cluster(const int* local, int rank) {
  const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(local));
  uint32_t remote;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster(int* local, int rank, int v) {
  const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(local));
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(a), "r"(rank));
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(remote), "r"(v) : "memory");
}

struct Table {
  int rows, columns;
  int32_t* pages;
  int32_t* held;
};

// refs of four pages; -1 behind the last.
__device__ __forceinline__ int4 load_refs(const int32_t* refs, int page, int pages) {
  if (page + 4 <= pages) return __ldcg(reinterpret_cast<const int4*>(refs + page));
  int4 v = make_int4(-1, -1, -1, -1);
  if (page < pages) v.x = __ldcg(refs + page);
  if (page + 1 < pages) v.y = __ldcg(refs + page + 1);
  if (page + 2 < pages) v.z = __ldcg(refs + page + 2);
  return v;
}
__device__ __forceinline__ unsigned free_bits(const int4& v) {
  return (v.x == 0) | (v.y == 0) << 1 | (v.z == 0) << 2 | (v.w == 0) << 3;
}

// refs in chunks of a multiple of 128 pages; warp `gw` of the cluster has every warps-th.
// It goes through a chunk 128 pages at a time, four to a lane.
struct Chunks {
  const int32_t* refs;
  int pages, size, count, gw, warps;
  int counted;              // chunks that have been counted
  int chunk, time;          // the next that this warp counts, and how many times 128 pages lie before
  unsigned long long mask;  // the lane's free pages in the first 16 such times
  __device__ __forceinline__ Chunks(const int32_t* r, int n, int warp, int all)
      : refs(r), pages(n), gw(warp), warps(all), counted(0), chunk(warp), time(0), mask(0) {
    const int most = all == kWarps ? kWarps : kChunks;  // one CTA: a chunk a warp
    size = ((n + most - 1) / most + 127) & ~127;
    count = (n + size - 1) / size;
  }
  // Counts the chunks up to number `to`: leaves the free pages of all before each in
  // sh.free_before (and behind the last).  All threads of the cluster; has a barrier of it, and arrives
  // at another, which no CTA may leave or count on without (leave).  A CTA runs
  // this once and its code comes from L2, some 12 clocks an instruction: it is written to be short.
  __device__ __forceinline__ void count_free(PagesShared& sh, int cluster, int to) {
    constexpr int kAhead = 4;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int sum = 0, at = 0;
    // Whole chunks of four times, as large pools have them.
#pragma unroll 1
    while (size % (128 * kAhead) == 0 && chunk < to && (chunk + 1LL) * size <= pages) {
      const int4* from = reinterpret_cast<const int4*>(refs + static_cast<size_t>(chunk) * size + at) + lane;
      int4 v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) v[i] = __ldcg(from + 32 * i);
      unsigned bits = 0;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) bits |= free_bits(v[i]) << 4 * i;
      if (time < 16) mask |= static_cast<unsigned long long>(bits) << 4 * time;
      time += kAhead;
      sum += __popc(bits);
      at += 128 * kAhead;
      if (at >= size) {
        sum = __reduce_add_sync(0xffffffffu, sum);
        if (lane == 0) sh.counts[chunk / cluster] = sum;
        sum = at = 0;
        chunk += warps;
      }
    }
    int load_chunk = chunk, load_at = 4 * lane;  // the next to load
#pragma unroll 1
    while (chunk < to) {
      int4 v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const long long p = static_cast<long long>(load_chunk) * size + load_at;
        v[i] = make_int4(-1, -1, -1, -1);
        if (load_chunk < to && p + 4 <= pages) v[i] = __ldcg(reinterpret_cast<const int4*>(refs + p));
        load_at += 128;
        if (load_at >= size) load_at = 4 * lane, load_chunk += warps;
      }
      unsigned all = 0;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) all |= free_bits(v[i]) << 4 * i;
#pragma unroll 1
      for (int i = 0; i < kAhead && chunk < to; ++i, ++time) {
        unsigned bits = all & 15u;
        all >>= 4;
        const int p = chunk * size + at + 4 * lane;
        if (p < pages && p + 4 > pages) bits = free_bits(load_refs(refs, p, pages));
        if (time < 16) mask |= static_cast<unsigned long long>(bits) << 4 * time;
        sum += __popc(bits);
        at += 128;
        if (at >= size) {
          sum = __reduce_add_sync(0xffffffffu, sum);
          if (lane == 0) sh.counts[chunk / cluster] = sum;
          sum = at = 0;
          chunk += warps;
        }
      }
    }
    cluster_barrier(cluster);
    // Of each CTA's chunks, those from number `counted` on.
    const int i0 = counted / cluster, blocks = ((to + cluster - 1) / cluster - i0 + 31) / 32;
#pragma unroll 1
    for (int b = warp; b < blocks * cluster; b += kWarps) {
      const int from = b / blocks, i = i0 + (b - from * blocks) * 32 + lane, c = i * cluster + from;
      if (c >= counted && c < to) sh.free_before[c + 1] = cluster == 1 ? sh.counts[i] : ld_cluster(&sh.counts[i], from);
    }
    if (cluster > 1) cluster_arrive();
    if (counted == 0 && threadIdx.x == 0) sh.free_before[0] = 0;
    __syncthreads();
    // Running sums, two chunks to a thread.
    const int c = counted + 2 * threadIdx.x, x = c < to ? sh.free_before[c + 1] : 0, y = c + 1 < to ? sh.free_before[c + 2] : 0;
    const int base = sh.free_before[counted];
    int upto = x + y;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += z;
    }
    if (lane == 31) sh.warp_sums[warp] = upto;
    __syncthreads();
    const int behind = base + __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_sums[lane] : 0) + upto;
    if (c < to) sh.free_before[c + 1] = behind - y;
    if (c + 1 < to) sh.free_before[c + 2] = behind;
    counted = to;
    __syncthreads();
  }
  // Behind it no CTA reads this one's shared memory.
  __device__ __forceinline__ void leave(int cluster) const {
    if (cluster > 1) cluster_wait();
  }
  // Free pages of four of the lane, from page p on of the warp's time number `time`.
  __device__ __forceinline__ unsigned bits(int p, int time) const {
    return time < 16 ? static_cast<unsigned>(mask >> 4 * time) & 15u : free_bits(load_refs(refs, p + 4 * (threadIdx.x & 31), pages));
  }
  // f(first page, the lane's free bits of it and the three behind, free pages before the first, of all lanes)
  // for the warp's runs of 128 pages that have free ones numbered base .. end - 1.
  template <typename F>
  __device__ __forceinline__ void each_run(const PagesShared& sh, int base, int end, F&& f) const {
    const unsigned lower = (1u << (threadIdx.x & 31)) - 1;
    int time = 0;
#pragma unroll 1
    for (int chunk = gw; chunk < counted; chunk += warps) {
      int before = sh.free_before[chunk];
      if (before >= end) break;
      if (sh.free_before[chunk + 1] <= base) {
        time += size / 128;
        continue;
      }
#pragma unroll 1
      for (int at = 0; at < size; at += 128, ++time) {
        const int p = chunk * size + at;
        const unsigned b = bits(p, time);
        int mine = before, all = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const unsigned ones = __ballot_sync(0xffffffffu, b >> i & 1);
          mine += __popc(ones & lower);
          all += __popc(ones);
        }
        if (before + all > base && before < end) f(p + 4 * (threadIdx.x & 31), b, mine, all);
        before += all;
      }
    }
  }
};

__device__ __forceinline__ int add_up(int a, int b) {  // of numbers from 0 on, no further than INT_MAX
  return static_cast<int>(min(static_cast<unsigned>(a) + static_cast<unsigned>(b), static_cast<unsigned>(INT_MAX)));
}

// start[r] = need(0) + .. + need(r - 1), no further than INT_MAX, for 0 <= r <= rows.
template <typename F>
__device__ __forceinline__ void scan_rows(PagesShared& sh, int* start, int rows, F&& need) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int each = (rows + kThreads - 1) / kThreads, r0 = min(static_cast<int>(threadIdx.x) * each, rows), r1 = min(r0 + each, rows);
  int sum = 0;
#pragma unroll 1
  for (int r = r0; r < r1; ++r) {
    start[r] = need(r);
    sum = add_up(sum, start[r]);
  }
  int upto = sum;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto = add_up(upto, y);
  }
  int at = __shfl_up_sync(0xffffffffu, upto, 1);
  if (lane == 0) at = 0;
  if (lane == 31) sh.warp_sums[warp] = upto;
  __syncthreads();
  int before = lane < warp ? sh.warp_sums[lane] : 0;
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) before = add_up(before, __shfl_xor_sync(0xffffffffu, before, o));
  at = add_up(before, at);
#pragma unroll 1
  for (int r = r0; r < r1; ++r) {
    const int x = start[r];
    start[r] = at;
    at = add_up(at, x);
  }
  if (threadIdx.x == kThreads - 1) start[rows] = at;
  __syncthreads();
}

// The first CTA's number of pages to take, for all: with it they go through the
// same barriers, even if the arrays should change under the kernel.  Waits for the
// cluster's CTAs to have begun, and ends with a barrier of it.
__device__ __forceinline__ int agree_on_need(PagesShared& sh, int need, int cluster) {
  if (cluster > 1) {
    cluster_wait();
    if (cluster_rank() == 0 && static_cast<int>(threadIdx.x) < cluster) st_cluster(&sh.need, threadIdx.x, need);
    cluster_barrier(cluster);
    return sh.need;
  }
  __syncthreads();
  return need;
}

// The row that item k falls to: the last with start[r] <= k.
__device__ __forceinline__ int row_of(const int* start, int rows, int k) {
  int lo = 0, hi = rows - 1;
  while (lo < hi) {
    const int m = (lo + hi + 1) / 2;
    if (start[m] <= k) lo = m; else hi = m - 1;
  }
  return lo;
}

// place(page, k, free) for the k-th free page, k < need as far as there are any;
// returns how many are free, or fewer, but then `need`.  All threads of the cluster.
template <typename F>
__device__ __forceinline__ int take_pages(PagesShared& sh, const int32_t* refs, int pages, int need, int cluster, F&& place) {
  const int lane = threadIdx.x & 31, rank = cluster_rank();
  if (threadIdx.x == 0) sh.listed = 0;
  // First a chunk a warp, which in a large pool may be enough, then the rest.
  Chunks chunks(refs, pages, (threadIdx.x >> 5) * cluster + rank, cluster * kWarps);
  chunks.count_free(sh, cluster, min(chunks.count, chunks.warps));
  if (sh.free_before[chunks.counted] < need && chunks.counted < chunks.count) {
    chunks.leave(cluster);
    __syncthreads();
    chunks.count_free(sh, cluster, chunks.count);
  }
  const int free_pages = sh.free_before[chunks.counted], given = min(need, free_pages);
  // As many at a time as this CTA's list holds; of the cluster's, mostly all.
  int mine = cluster == 1 ? given : 0;
  for (int i = lane; i * cluster + rank < chunks.counted && cluster > 1; i += 32)
    if (sh.free_before[i * cluster + rank] < given) mine += sh.counts[i];
  if (cluster > 1) mine = __reduce_add_sync(0xffffffffu, mine);
  const int window = mine <= kList ? given : kList;
  // From the highest on: a chunk that is looked at again then lacks only pages
  // behind those that are counted.
#pragma unroll 1
  for (int base = given > 0 ? (given - 1) / window * window : -1; base >= 0; base -= window) {
    const int end = given - base < window ? given : base + window;
    chunks.each_run(sh, base, end, [&](int page, unsigned bits, int k, int all) {
      int to = 0;
      if (lane == 0) to = atomicAdd(&sh.listed, all);
      to = __shfl_sync(0xffffffffu, to, 0) + k - __shfl_sync(0xffffffffu, k, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (bits >> i & 1) {
          // The run's free pages have places side by side; those outside the window
          // leave theirs empty, in a first and a last run.
          if (to < kList + 256) sh.list[to] = make_int2(k >= base && k < end ? page + i : -1, k);
          ++to, ++k;
        }
    });
    __syncthreads();
    const int listed = min(sh.listed, kList + 256);  // more only where refs changes under the kernel
    for (int i = threadIdx.x; i < listed; i += kThreads)
      if (sh.list[i].x >= 0) place(sh.list[i].x, sh.list[i].y, free_pages);
    __syncthreads();
    if (threadIdx.x == 0) sh.listed = 0;
    __syncthreads();
  }
  chunks.leave(cluster);
  return free_pages;
}

struct ResizeArgs {
  Table table;
  int32_t* refs;
  int num_pages, page_shift;
  const int32_t* tokens;
  int32_t* served;
  int32_t* status;
};

// Pages that a row should hold; -1: it is left alone; -2: it cannot be (bad).
__device__ __forceinline__ int wanted(const ResizeArgs& a, int r, int held) {
  const int t = a.tokens[r];
  if (t < 0) return -1;
  const int want = static_cast<int>((static_cast<long long>(t) + (1 << a.page_shift) - 1) >> a.page_shift);
  return held < 0 || held > a.table.columns || want > a.table.columns ? -2 : want;
}

__device__ __forceinline__ void let_go(const ResizeArgs& a, int r, int c) {
  if (!CP_CHECK_DATA(c >= 0 && c < a.table.columns, a.status)) return;
  int32_t* entry = a.table.pages + static_cast<size_t>(r) * a.table.columns + c;
  const int page = *entry;
  *entry = -1;
  if (!CP_CHECK_DATA(page >= 0 && page < a.num_pages, a.status)) return;
  if (!CP_CHECK_DATA(atomicSub(a.refs + page, 1) > 0, a.status)) atomicAdd(a.refs + page, 1);
}

__global__ void __launch_bounds__(kThreads, 1) pages_resize_kernel(const __grid_constant__ ResizeArgs a, int cluster) {
  constexpr int kFew = 4;  // pages that a row's thread lets go itself
  PagesShared& sh = *reinterpret_cast<PagesShared*>(pages_shared);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rank = cluster_rank();
  const int rows = a.table.rows;
  if (cluster > 1) cluster_arrive();
  if (threadIdx.x == 0) sh.queued = 0;
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  // Every CTA counts what all rows take; each lets go of the pages of its share of them.
  scan_rows(sh, sh.start, rows, [&](int r) {
    const int held = a.table.held[r], want = wanted(a, r, held);
    if (r % cluster == rank) {
      if (want == -2) debug_bounds_fail(a.status, __LINE__, CP_TU_ID);
      if (want >= 0 && want < held) {
        int k = kQueue;
        if (held - want > kFew) k = atomicAdd(&sh.queued, 1);
        if (k < kQueue) {
          sh.queue[k] = r;
        } else {
          for (int c = want; c < held; ++c) let_go(a, r, c);
        }
      }
    }
    return want >= 0 ? max(want - held, 0) : 0;
  });
  const int queued = min(sh.queued, kQueue);
  if (queued > 0) {
    // Pages of rows with many, shared out to all threads.
    int* first = sh.free_before;
    scan_rows(sh, first, queued, [&](int i) {
      const int r = sh.queue[i], held = a.table.held[r];
      return max(held - max(wanted(a, r, held), 0), 0);
    });
#pragma unroll 1
    for (int k = threadIdx.x; k < first[queued]; k += kThreads) {
      const int i = row_of(first, queued, k), r = sh.queue[i];
      let_go(a, r, a.table.held[r] - 1 - (k - first[i]));
    }
  }
  const int need = agree_on_need(sh, sh.start[rows], cluster);  // behind it all has been let go
  int free_pages = 0;
  if (need > 0)
    free_pages = take_pages(sh, a.refs, a.num_pages, need, cluster, [&](int page, int k, int free) {
      const int r = row_of(sh.start, rows, k);
      if (sh.start[r + 1] > free) return;  // served in order, as long as pages last
      const int want = static_cast<int>((static_cast<long long>(a.tokens[r]) + (1 << a.page_shift) - 1) >> a.page_shift);
      const int c = want - (sh.start[r + 1] - k);
      if (!CP_CHECK_DATA(c >= 0 && c < a.table.columns, a.status)) return;  // only where the arrays change under the kernel
      a.refs[page] = 1;
      a.table.pages[static_cast<size_t>(r) * a.table.columns + c] = page;
    });
  for (int r = rank * kThreads + threadIdx.x; r < rows; r += cluster * kThreads) {
    const int held = a.table.held[r], want = wanted(a, r, held);
    const bool ok = want != -2 && (want <= held || sh.start[r + 1] <= free_pages);
    if (ok && want >= 0) a.table.held[r] = want;
    a.served[r] = ok;
  }
}

struct ForkArgs {
  Table src, dst;
  int32_t* refs;
  int num_pages, page_shift;
  const int32_t* parent;
  const int32_t* tokens;
  int32_t* served;
  int32_t* count;  // of the moves
  int32_t* move_src;
  int32_t* move_dst;
  int32_t* move_tokens;
  int32_t* status;
};

// 1: row r is a child as it should be; 0: none; -1: its data are bad.
__device__ __forceinline__ int is_child(const ForkArgs& a, int r) {
  const int p = a.parent[r], t = a.tokens[r];
  if (p < 0) return 0;
  if (p >= a.src.rows || t < 0 || a.dst.held[r] != 0) return -1;
  const long long held = a.src.held[p], want = (static_cast<long long>(t) + (1 << a.page_shift) - 1) >> a.page_shift;
  return held >= want && held <= a.src.columns && want <= a.dst.columns ? 1 : -1;
}

__global__ void __launch_bounds__(kThreads, 1) pages_fork_kernel(const __grid_constant__ ForkArgs a, int cluster) {
  __shared__ int8_t child[kMaxTableRows];
  PagesShared& sh = *reinterpret_cast<PagesShared*>(pages_shared);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = cluster_rank(), gw = rank * kWarps + warp, warps = cluster * kWarps;
  const int rows = a.dst.rows, rest = (1 << a.page_shift) - 1;
  if (cluster > 1) cluster_arrive();
  pdl_wait();
  pdl_launch_dependents();
  scan_rows(sh, sh.start, rows, [&](int r) {
    const int c = is_child(a, r);
    child[r] = static_cast<int8_t>(c);
    if (c < 0 && rank == 0) debug_bounds_fail(a.status, __LINE__, CP_TU_ID);
    return c > 0 && (a.tokens[r] & rest) ? 1 : 0;
  });
  const int need = agree_on_need(sh, sh.start[rows], cluster);  // behind it every row's data have been read
  int free_pages = 0;
  if (need > 0)
    free_pages = take_pages(sh, a.refs, a.num_pages, need, cluster, [&](int page, int k, int) {
      const int r = row_of(sh.start, rows, k);  // its part page
      const int t = a.tokens[r], full = t >> a.page_shift, parent = a.parent[r];
      // Only where the arrays change under the kernel.
      if (!CP_CHECK_DATA(parent >= 0 && parent < a.src.rows && full < a.dst.columns && full < a.src.columns, a.status)) return;
      a.refs[page] = 1;
      a.dst.pages[static_cast<size_t>(r) * a.dst.columns + full] = page;
      a.move_src[k] = a.src.pages[static_cast<size_t>(parent) * a.src.columns + full];
      a.move_dst[k] = page;
      a.move_tokens[k] = t & rest;
    });
  if (rank == 0 && threadIdx.x == 0) *a.count = min(need, free_pages);
  for (int r = gw; r < rows; r += warps) {
    const bool ok = child[r] >= 0 && (sh.start[r + 1] == sh.start[r] || sh.start[r + 1] <= free_pages);
    if (lane == 0) a.served[r] = ok;
    if (!ok || child[r] == 0) continue;
    const int full = a.tokens[r] >> a.page_shift, parent = a.parent[r];
    if (!CP_CHECK_DATA(full <= a.dst.columns && full <= a.src.columns && parent >= 0 && parent < a.src.rows, a.status)) continue;  // as above
    const int32_t* from = a.src.pages + static_cast<size_t>(parent) * a.src.columns;
    int32_t* to = a.dst.pages + static_cast<size_t>(r) * a.dst.columns;
    for (int c = lane; c < full; c += 32) {
      const int page = from[c];
      const bool there = CP_CHECK_DATA(page >= 0 && page < a.num_pages, a.status);
      if (there) atomicAdd(a.refs + page, 1);
      to[c] = there ? page : -1;
    }
    if (lane == 0) a.dst.held[r] = full + (sh.start[r + 1] - sh.start[r]);
  }
}

struct CompactArgs {
  const int32_t* refs;
  int32_t* refs_out;
  int num_pages;
  int32_t* count;
  int32_t* move_src;
  int32_t* move_dst;
  int32_t* move_tokens;
  int page_size;
  int32_t* used;   // the caller's, or null
  int32_t* total;  // workspace: the same
  int32_t* to;     // workspace: where a page from the used-th on goes, -1: nowhere
  int32_t* status;
};

__global__ void __launch_bounds__(kThreads, 1) pages_compact_kernel(const __grid_constant__ CompactArgs a, int cluster) {
  PagesShared& sh = *reinterpret_cast<PagesShared*>(pages_shared);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = cluster_rank(), gw = warp * cluster + rank, warps = cluster * kWarps;
  const int P = a.num_pages;
  if (cluster > 1) cluster_arrive();
  pdl_wait();
  pdl_launch_dependents();
  Chunks chunks(a.refs, P, gw, warps);
  if (cluster > 1) cluster_wait();
  chunks.count_free(sh, cluster, chunks.count);
  chunks.leave(cluster);
  // Held pages from number `used` on move to the free ones below it, which are
  // as many: `moves`, the free pages before number `used`, counted by the warp of that chunk.
  const int used = P - sh.free_before[chunks.counted], chunk_of_used = used / chunks.size;
  if (used < P && chunk_of_used % warps == gw) {
    int n = 0;
    for (int p = chunk_of_used * chunks.size; p < used; p += 128) {
      const unsigned bits = free_bits(load_refs(a.refs, p + 4 * lane, P));
#pragma unroll
      for (int i = 0; i < 4; ++i) n += (bits >> i & 1) && p + 4 * lane + i < used;
    }
    n = sh.free_before[chunk_of_used] + __reduce_add_sync(0xffffffffu, n);
    if (cluster == 1) sh.moved = n;
    else if (lane < cluster) st_cluster(&sh.moved, lane, n);
  }
  cluster_barrier(cluster);
  const int moves = used < P ? sh.moved : 0;
  // Free pages below `used` in order, held ones from there on in order.
  const unsigned lower = (1u << lane) - 1;
#pragma unroll 1
  for (int chunk = gw; chunk < chunks.count; chunk += warps) {
    int n = sh.free_before[chunk];
#pragma unroll 1
    for (int p = chunk * chunks.size; p < min((chunk + 1) * chunks.size, P); p += 128) {
      const int at = p + 4 * lane;
      const int4 v = load_refs(a.refs, at, P);
      const unsigned bits = free_bits(v);
      int rank_of = n;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const unsigned b = __ballot_sync(0xffffffffu, bits >> i & 1);
        rank_of += __popc(b & lower);
        n += __popc(b);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int page = at + i, held = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
        if (page >= P) break;
        const bool free_page = bits >> i & 1;
        if (a.refs_out != a.refs) a.refs_out[page] = page < used ? held : 0;
        if (page < used && free_page) {
          if (CP_CHECK_DATA(rank_of < P / 2, a.status)) a.move_dst[rank_of] = page;
        } else if (page >= used) {
          a.to[page] = -1;
          // page - rank_of held ones lie before it, used - moves of them below `used`.
          const int k = page - rank_of - (used - moves);
          if (!free_page && CP_CHECK_DATA(k >= 0 && k < P / 2, a.status)) a.move_src[k] = page;
        }
        rank_of += free_page;
      }
    }
  }
  cluster_barrier(cluster);
  for (int i = rank * kThreads + threadIdx.x; i < min(moves, P / 2); i += cluster * kThreads) {
    const int src = __ldcg(a.move_src + i), dst = __ldcg(a.move_dst + i);
    // These and the checks above fail only where refs changes under the kernel.
    if (!CP_CHECK_DATA(src >= 0 && src < P && dst >= 0 && dst < P, a.status)) continue;
    a.move_tokens[i] = a.page_size;
    a.to[src] = dst;
    const int r = __ldcg(a.refs + src);
    a.refs_out[dst] = r;
    a.refs_out[src] = 0;
  }
  if (rank == 0 && threadIdx.x == 0) {
    *a.count = moves;
    *a.total = used;
    if (a.used) *a.used = used;
  }
}

struct RenameArgs {
  int n;
  Table table[CP_PAGES_MAX_TABLES];
  int32_t* out[CP_PAGES_MAX_TABLES];
  int num_pages;
  const int32_t* total;
  const int32_t* to;
  int32_t* status;
};

constexpr int kRenameThreads = 256, kRenameChunk = 1024;

// Tables after a compaction: a block takes kRenameChunk entries of a row.
__global__ void __launch_bounds__(kRenameThreads) pages_rename_kernel(const __grid_constant__ RenameArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int used = *a.total;
  long long first = 0;
  for (int k = 0; k < a.n; ++k) {
    const Table& t = a.table[k];
    const int chunks = (t.columns + kRenameChunk - 1) / kRenameChunk;
    const long long all = static_cast<long long>(t.rows) * chunks;
    // Blocks go on in turn from where the table before left off.
    long long i = blockIdx.x - first % gridDim.x;
    if (i < 0) i += gridDim.x;
    for (; i < all; i += gridDim.x) {
      const int r = static_cast<int>(i / chunks), c0 = static_cast<int>(i % chunks) * kRenameChunk;
      int held = t.held[r];
      if (!CP_CHECK_DATA(held >= 0 && held <= t.columns, a.status)) continue;
      const int end = min(held, c0 + kRenameChunk);
      const int32_t* from = t.pages + static_cast<size_t>(r) * t.columns;
      int32_t* out = a.out[k] + static_cast<size_t>(r) * t.columns;
      for (int c = c0 + threadIdx.x; c < end; c += kRenameThreads) {
        int page = from[c];
        if (CP_CHECK_DATA(page >= 0 && page < a.num_pages, a.status) && page >= used && CP_IN_BOUNDS(c < t.columns, a.status)) {
          const int to = a.to[page];
          if (CP_CHECK_DATA(to >= 0, a.status)) page = to;
        }
        out[c] = page;
      }
    }
    first += all;
  }
}

struct CopyArgs {
  int n, d, Hkv, page_shift;
  int src_pages, dst_pages, capacity;
  const int32_t* count;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* tokens;
  int64_t src_page, src_token, src_head, dst_page, dst_token, dst_head;  // strides in elements
  int heads_first;  // of the order in which a page's rows are numbered
  int linear;       // pages of both are the same contiguous block
  int parts;        // of a page
  int32_t* status;
  const void* from[CP_PAGES_MAX_CACHES][2];
  void* to[CP_PAGES_MAX_CACHES][2];
};

constexpr int kCopyThreads = 256, kCopyAhead = 8;
constexpr int kCopyPart = kCopyThreads * kCopyAhead;  // 16-byte pieces that a block copies at a time

// A block copies one part of one page of one cache's K or V at a time.
__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const __grid_constant__ CopyArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int count = *a.count;
  if (!CP_CHECK_DATA(count >= 0 && count <= a.capacity, a.status)) return;
  const unsigned per_move = 2u * a.n * a.parts;
  const long long units = static_cast<long long>(count) * per_move;
  const int shift = a.d == 128 ? 4 : 3;  // 16-byte pieces of a row
  const int ps = 1 << a.page_shift;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int m = static_cast<int>(u / per_move);
    const unsigned in = static_cast<unsigned>(u - static_cast<long long>(m) * per_move);
    const unsigned which = in / a.parts, part = in - which * a.parts;
    const int src = a.src[m], dst = a.dst[m], tokens = a.tokens[m];
    if (!CP_CHECK_DATA(src >= 0 && src < a.src_pages && dst >= 0 && dst < a.dst_pages && tokens >= 0 && tokens <= ps, a.status)) continue;
    const uint16_t* from = static_cast<const uint16_t*>(a.from[which >> 1][which & 1]) + src * a.src_page;
    uint16_t* to = static_cast<uint16_t*>(a.to[which >> 1][which & 1]) + dst * a.dst_page;
    const int first = static_cast<int>(part) * kCopyPart + threadIdx.x;
    const int pieces = (a.heads_first ? ps : tokens) * a.Hkv << shift;
    uint4 x[kCopyAhead];
    int64_t at[kCopyAhead];
#pragma unroll
    for (int i = 0; i < kCopyAhead; ++i) {
      const int piece = first + i * kCopyThreads;
      at[i] = -1;
      if (piece >= pieces) continue;
      const int row = piece >> shift, col = (piece & ((1 << shift) - 1)) * 8;
      int64_t get;
      if (a.linear) {
        if (a.heads_first && (row & (ps - 1)) >= tokens) continue;
        get = at[i] = static_cast<int64_t>(piece) * 8;
      } else {
        const int h = a.heads_first ? row >> a.page_shift : row % a.Hkv, t = a.heads_first ? row & (ps - 1) : row / a.Hkv;
        if (t >= tokens) continue;
        get = t * a.src_token + h * a.src_head + col;
        at[i] = t * a.dst_token + h * a.dst_head + col;
        if (!CP_IN_BOUNDS(h < a.Hkv && t < ps, a.status)) at[i] = -1;
      }
      x[i] = *reinterpret_cast<const uint4*>(from + get);
    }
#pragma unroll
    for (int i = 0; i < kCopyAhead; ++i)
      if (at[i] >= 0) *reinterpret_cast<uint4*>(to + at[i]) = x[i];
  }
}

// CTAs of a call that looks at `pages` counts and `rows` rows, of which a CTA does `each` well.
int cluster_for(int pages, int rows, int each) {
  int c = 1;
  while (c < kMaxCluster && (pages > 32768 * c || rows > each * c)) c *= 2;
  return c;
}

template <typename K, typename A>
int launch_cluster(std::atomic<int> (&known)[64], K kernel, const A& a, int cluster, cudaStream_t stream) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CP_ERR_CUDA;
  if (!known[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(PagesShared)) != cudaSuccess)
      return CP_ERR_CUDA;
    known[dev].store(1, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(PagesShared);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a, cluster) == cudaSuccess ? CP_OK : CP_ERR_CUDA;
}

// The host's checks.
constexpr int kMaxPages = 1 << 30;
int check_refs(int32_t num_pages, const int32_t* refs) {
  if (num_pages <= 0 || num_pages > kMaxPages || !refs) return CP_ERR_INVALID_ARG;
  return aligned(refs, 16) ? CP_OK : CP_ERR_ALIGNMENT;
}
int check_table(const cp_page_table_t* t, int page_shift) {
  if (!t || t->rows <= 0 || t->rows > kMaxTableRows || t->columns <= 0 || !t->pages || !t->held) return CP_ERR_INVALID_ARG;
  if (static_cast<long long>(t->columns) << page_shift >= 1LL << 30) return CP_ERR_INVALID_ARG;
  return aligned(t->pages, 4) && aligned(t->held, 4) ? CP_OK : CP_ERR_ALIGNMENT;
}
int check_moves(const cp_page_moves_t* m, int least) {
  if (!m || m->capacity < 0 || m->capacity < least || !m->count) return CP_ERR_INVALID_ARG;
  if (m->capacity > 0 && (!m->src || !m->dst || !m->tokens)) return CP_ERR_INVALID_ARG;
  return aligned(m->count, 4) && aligned(m->src, 4) && aligned(m->dst, 4) && aligned(m->tokens, 4) ? CP_OK : CP_ERR_ALIGNMENT;
}
Table table_of(const cp_page_table_t& t) { return Table{t.rows, t.columns, t.pages, t.held}; }

}  // namespace
}  // namespace cpattn

using namespace cpattn;

extern "C" {

int cp_pages_resize(const cp_paged_t* plan, int32_t num_pages, int32_t* refs, const cp_page_table_t* table, const int32_t* tokens,
                    int32_t* served, cudaStream_t stream) {
  if (!plan) return CP_ERR_INVALID_ARG;
  ResizeArgs a = {};
  a.page_shift = paged_page_shift(plan);
  int rc = check_refs(num_pages, refs);
  if (rc == CP_OK) rc = check_table(table, a.page_shift);
  if (rc == CP_OK && (!tokens || !served || served == tokens || served == table->held || tokens == table->held)) rc = CP_ERR_INVALID_ARG;
  if (rc == CP_OK && (!aligned(tokens, 4) || !aligned(served, 4))) rc = CP_ERR_ALIGNMENT;
  if (rc == CP_OK) rc = check_arch();
  if (rc != CP_OK) return rc;
  a.table = table_of(*table);
  a.refs = refs;
  a.num_pages = num_pages;
  a.tokens = tokens;
  a.served = served;
  a.status = device_status_ptr();
  if (!a.status) return CP_ERR_CUDA;
  NvtxRange range("cp_pages_resize");
  static std::atomic<int> known[64];
  return launch_cluster(known, pages_resize_kernel, a, cluster_for(num_pages, table->rows, 256), stream);
}

int cp_pages_fork(const cp_paged_t* plan, int32_t num_pages, int32_t* refs, const cp_page_table_t* src, const cp_page_table_t* dst,
                  const int32_t* parent, const int32_t* tokens, const cp_page_moves_t* moves, int32_t* served, cudaStream_t stream) {
  if (!plan) return CP_ERR_INVALID_ARG;
  ForkArgs a = {};
  a.page_shift = paged_page_shift(plan);
  int rc = check_refs(num_pages, refs);
  if (rc == CP_OK) rc = check_table(src, a.page_shift);
  if (rc == CP_OK) rc = check_table(dst, a.page_shift);
  if (rc == CP_OK) rc = check_moves(moves, dst->rows);
  if (rc == CP_OK && (!parent || !tokens || !served || served == parent || served == tokens || served == src->held || served == dst->held ||
                      parent == dst->held || tokens == dst->held))
    rc = CP_ERR_INVALID_ARG;
  if (rc == CP_OK && (!aligned(parent, 4) || !aligned(tokens, 4) || !aligned(served, 4))) rc = CP_ERR_ALIGNMENT;
  if (rc == CP_OK) rc = check_arch();
  if (rc != CP_OK) return rc;
  a.src = table_of(*src);
  a.dst = table_of(*dst);
  a.refs = refs;
  a.num_pages = num_pages;
  a.parent = parent;
  a.tokens = tokens;
  a.served = served;
  a.count = moves->count;
  a.move_src = moves->src;
  a.move_dst = moves->dst;
  a.move_tokens = moves->tokens;
  a.status = device_status_ptr();
  if (!a.status) return CP_ERR_CUDA;
  NvtxRange range("cp_pages_fork");
  static std::atomic<int> known[64];
  return launch_cluster(known, pages_fork_kernel, a, cluster_for(num_pages, dst->rows, 64), stream);
}

int cp_pages_workspace_size(int32_t num_pages, size_t* bytes) {
  if (num_pages <= 0 || num_pages > kMaxPages || !bytes) return CP_ERR_INVALID_ARG;
  *bytes = 16 + 4 * static_cast<size_t>(num_pages);
  return CP_OK;
}

int cp_pages_compact(const cp_paged_t* plan, int32_t num_pages, const int32_t* refs, int32_t* refs_out, int32_t n_tables,
                     const cp_page_table_t* tables, const cp_page_table_t* tables_out, const cp_page_moves_t* moves, int32_t* used,
                     void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!plan || n_tables < 1 || n_tables > CP_PAGES_MAX_TABLES || !tables || !tables_out) return CP_ERR_INVALID_ARG;
  const int shift = paged_page_shift(plan);
  int rc = check_refs(num_pages, refs);
  if (rc == CP_OK) rc = check_refs(num_pages, refs_out);
  if (rc == CP_OK) rc = check_moves(moves, num_pages / 2);
  RenameArgs b = {};
  long long chunks = 0;
  for (int i = 0; rc == CP_OK && i < n_tables; ++i) {
    rc = check_table(tables + i, shift);
    if (rc == CP_OK && (!tables_out[i].pages || tables_out[i].rows != tables[i].rows || tables_out[i].columns != tables[i].columns))
      rc = CP_ERR_INVALID_ARG;
    if (rc == CP_OK && !aligned(tables_out[i].pages, 4)) rc = CP_ERR_ALIGNMENT;
    if (rc != CP_OK) break;
    b.table[i] = table_of(tables[i]);
    b.out[i] = tables_out[i].pages;
    chunks += static_cast<long long>(tables[i].rows) * ((tables[i].columns + kRenameChunk - 1) / kRenameChunk);
  }
  if (rc == CP_OK && (!aligned(used, 4) || !aligned(workspace, 16))) rc = CP_ERR_ALIGNMENT;
  size_t bytes = 0;
  if (rc == CP_OK) rc = cp_pages_workspace_size(num_pages, &bytes);
  if (rc == CP_OK && (!workspace || workspace_bytes < bytes)) rc = CP_ERR_WORKSPACE;
  if (rc == CP_OK) rc = check_arch();
  if (rc != CP_OK) return rc;
  CompactArgs a = {};
  a.refs = refs;
  a.refs_out = refs_out;
  a.num_pages = num_pages;
  a.count = moves->count;
  a.move_src = moves->src;
  a.move_dst = moves->dst;
  a.move_tokens = moves->tokens;
  a.page_size = 1 << shift;
  a.used = used;
  a.total = static_cast<int32_t*>(workspace);
  a.to = a.total + 4;
  a.status = device_status_ptr();
  if (!a.status) return CP_ERR_CUDA;
  b.n = n_tables;
  b.num_pages = num_pages;
  b.total = a.total;
  b.to = a.to;
  b.status = a.status;
  NvtxRange range("cp_pages_compact");
  static std::atomic<int> known[64];
  rc = launch_cluster(known, pages_compact_kernel, a, cluster_for(num_pages, 0, 1), stream);
  if (rc != CP_OK) return rc;
  const unsigned grid = static_cast<unsigned>(chunks < 152 * 8 ? chunks : 152 * 8);
  return launch(pages_rename_kernel, grid, kRenameThreads, 0, stream, b);
}

int cp_pages_copy(const cp_paged_t* plan, int32_t n_caches, const cp_paged_cache_t* src, const cp_paged_cache_t* dst,
                  const cp_page_moves_t* moves, cudaStream_t stream) {
  if (!plan || n_caches < 1 || n_caches > CP_PAGES_MAX_CACHES || !src || !dst) return CP_ERR_INVALID_ARG;
  int rc = check_moves(moves, 0);
  CopyArgs a = {};
  for (int i = 0; rc == CP_OK && i < n_caches; ++i) {
    rc = paged_check_cache(plan, src[i]);
    if (rc == CP_OK) rc = paged_check_cache(plan, dst[i]);
    // The layers' caches are alike.
    const cp_paged_cache_t* c[2][2] = {{src, src + i}, {dst, dst + i}};
    for (int k = 0; rc == CP_OK && k < 2; ++k)
      if (c[k][0]->num_pages != c[k][1]->num_pages || c[k][0]->page_stride != c[k][1]->page_stride ||
          c[k][0]->token_stride != c[k][1]->token_stride || c[k][0]->head_stride != c[k][1]->head_stride)
        rc = CP_ERR_INVALID_ARG;
    a.from[i][0] = src[i].k;
    a.from[i][1] = src[i].v;
    a.to[i][0] = dst[i].k;
    a.to[i][1] = dst[i].v;
  }
  if (rc == CP_OK) rc = check_arch();
  if (rc != CP_OK || moves->capacity == 0) return rc;
  a.n = n_caches;
  paged_rows(plan, &a.Hkv, &a.d);
  a.page_shift = paged_page_shift(plan);
  a.src_pages = src->num_pages;
  a.dst_pages = dst->num_pages;
  a.capacity = moves->capacity;
  a.count = moves->count;
  a.src = moves->src;
  a.dst = moves->dst;
  a.tokens = moves->tokens;
  a.src_page = src->page_stride;
  a.src_token = src->token_stride;
  a.src_head = src->head_stride;
  a.dst_page = dst->page_stride;
  a.dst_token = dst->token_stride;
  a.dst_head = dst->head_stride;
  const int64_t ps = 1LL << a.page_shift;
  a.heads_first = a.dst_token < a.dst_head;
  // With one head, or pages of one token's order, the strides that no row takes say nothing.
  const auto dense = [&](const cp_paged_cache_t& c) {
    return a.heads_first ? c.token_stride == a.d && (a.Hkv == 1 || c.head_stride == ps * a.d)
                         : (a.Hkv == 1 || c.head_stride == a.d) && c.token_stride == static_cast<int64_t>(a.Hkv) * a.d;
  };
  a.linear = dense(*src) && dense(*dst);
  a.status = device_status_ptr();
  if (!a.status) return CP_ERR_CUDA;
  const long long pieces = ps * a.Hkv * (a.d / 8);
  if (pieces > 1 << 30) return CP_ERR_UNSUPPORTED;
  a.parts = static_cast<int>((pieces + kCopyPart - 1) / kCopyPart);
  const long long units = 2LL * n_caches * a.parts * moves->capacity;  // at most; the moves' count is on the device
  const unsigned grid = static_cast<unsigned>(units < 152 * 20 ? units : 152 * 20);
  NvtxRange range("cp_pages_copy");
  return launch(pages_copy_kernel, grid, kCopyThreads, 0, stream, a);
}

}  // extern "C"
