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
// The three calls that change tables are bound by latency: a few dependent
// loads and a count of refs (4 bytes a page).  Each is one cluster of CTAs, so that its
// steps are separated by the cluster's hardware barrier, not by launches, and
// their counts are exchanged through distributed shared memory.  The copies are bound
// by memory.
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
constexpr int kRowsPerThread = kMaxTableRows / kThreads;

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// All threads of the cluster; what they wrote before, to global memory too, is
// seen after (read past L1 where this kernel itself has written).
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ int ld_cluster(const int* local, unsigned rank) {
  const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(local));
  uint32_t remote;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
  return v;
}

struct Table {
  int rows, columns;
  int32_t* pages;
  int32_t* held;
};

// Each warp of the cluster counts its own stretch of refs, a multiple of 128 pages.
struct Stretch {
  int lo, hi;
  __device__ __forceinline__ Stretch(int pages, int warp, int warps) {
    const int per = ((pages + warps - 1) / warps + 127) & ~127;
    lo = static_cast<int>(min(static_cast<long long>(warp) * per, static_cast<long long>(pages)));
    hi = static_cast<int>(min(static_cast<long long>(lo) + per, static_cast<long long>(pages)));
  }
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

// Free pages of the warp's stretch.
__device__ __forceinline__ int count_free(const int32_t* refs, const Stretch& s, int pages) {
  constexpr int kAhead = 4;
  const int lane = threadIdx.x & 31;
  int n = 0;
  for (int p = s.lo; p < s.hi; p += 128 * kAhead) {
    int4 v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int at = p + 128 * i + 4 * lane;
      v[i] = p + 128 * i < s.hi ? load_refs(refs, at, pages) : make_int4(-1, -1, -1, -1);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) n += __popc(free_bits(v[i]));
  }
  return __reduce_add_sync(0xffffffffu, n);
}

// f(page, free pages before it) for the free pages of the warp's stretch, of
// which `before` lie before it, as long as fewer than `most` do.
template <typename F>
__device__ __forceinline__ void each_free(const int32_t* refs, const Stretch& s, int pages, int before, int most, F&& f) {
  const int lane = threadIdx.x & 31;
  const unsigned lower = (1u << lane) - 1;
  for (int p = s.lo; p < s.hi && before < most; p += 128) {
    const int at = p + 4 * lane;
    const unsigned bits = free_bits(load_refs(refs, at, pages));
    int mine = before, all = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned b = __ballot_sync(0xffffffffu, bits >> i & 1);
      mine += __popc(b & lower);
      all += __popc(b);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (bits >> i & 1) f(at + i, mine++);
    before += all;
  }
}

// Sums over the cluster of one number a warp: the sum of the warps before this
// one, and of all.  Two cluster barriers.
__device__ __forceinline__ int cluster_scan(int mine, int cluster, int* warp_sums, int* cta_sum, int* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) warp_sums[warp] = mine;
  __syncthreads();
  const int x = warp_sums[lane];
  if (threadIdx.x == 0) *cta_sum = 0;
  __syncthreads();
  const int here = __reduce_add_sync(0xffffffffu, x);
  const int before_here = __reduce_add_sync(0xffffffffu, lane < warp ? x : 0);
  if (threadIdx.x == 0) *cta_sum = here;
  cluster_barrier();
  const unsigned rank = cluster_rank();
  const int other = lane < cluster ? ld_cluster(cta_sum, lane) : 0;
  *all = __reduce_add_sync(0xffffffffu, other);
  const int before = before_here + __reduce_add_sync(0xffffffffu, lane < static_cast<int>(rank) ? other : 0);
  cluster_barrier();
  return before;
}

// start[r] = need(0) + .. + need(r - 1), cut off at INT_MAX, for 0 <= r <= rows.
template <typename F>
__device__ __forceinline__ void scan_rows(int rows, int* start, long long* warp_totals, F&& need) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int each = (rows + kThreads - 1) / kThreads, r0 = threadIdx.x * each;
  int x[kRowsPerThread];
  long long sum = 0;
#pragma unroll
  for (int i = 0; i < kRowsPerThread; ++i) {
    x[i] = i < each && r0 + i < rows ? need(r0 + i) : 0;
    sum += x[i];
  }
  long long upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) warp_totals[warp] = upto;
  __syncthreads();
  long long at = upto - sum;
  for (int w = 0; w < warp; ++w) at += warp_totals[w];
#pragma unroll
  for (int i = 0; i < kRowsPerThread; ++i) {
    if (i < each && r0 + i < rows) start[r0 + i] = static_cast<int>(min(at, static_cast<long long>(INT_MAX)));
    at += x[i];
  }
  if (threadIdx.x == kThreads - 1) start[rows] = static_cast<int>(min(at, static_cast<long long>(INT_MAX)));
  __syncthreads();
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

__global__ void __launch_bounds__(kThreads) pages_resize_kernel(const __grid_constant__ ResizeArgs a, int cluster) {
  __shared__ int start[kMaxTableRows + 1];
  __shared__ long long warp_totals[kWarps];
  __shared__ int warp_sums[kWarps], cta_sum;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = static_cast<int>(cluster_rank()), gw = rank * kWarps + warp, warps = cluster * kWarps;
  const int rows = a.table.rows;
  pdl_wait();
  pdl_launch_dependents();
  scan_rows(rows, start, warp_totals, [&](int r) {
    const int held = a.table.held[r], want = wanted(a, r, held);
    if (want == -2 && rank == 0) debug_bounds_fail(a.status, __LINE__, CP_TU_ID);
    return want >= 0 ? max(want - held, 0) : 0;
  });
  // Pages behind those that a row should hold are let go.
  for (int r = gw; r < rows; r += warps) {
    const int held = a.table.held[r], want = wanted(a, r, held);
    if (want < 0 || !CP_IN_BOUNDS(held <= a.table.columns, a.status)) continue;  // wanted() has looked at held
    int32_t* pages = a.table.pages + static_cast<size_t>(r) * a.table.columns;
    for (int c = want + lane; c < held; c += 32) {
      const int page = pages[c];
      pages[c] = -1;
      if (!CP_CHECK_DATA(page >= 0 && page < a.num_pages, a.status)) continue;
      if (!CP_CHECK_DATA(atomicSub(a.refs + page, 1) > 0, a.status)) atomicAdd(a.refs + page, 1);
    }
  }
  const int need = start[rows];
  cluster_barrier();
  int free_pages = 0;
  if (need > 0) {
    const Stretch s(a.num_pages, gw, warps);
    const int before = cluster_scan(count_free(a.refs, s, a.num_pages), cluster, warp_sums, &cta_sum, &free_pages);
    each_free(a.refs, s, a.num_pages, before, min(need, free_pages), [&](int page, int k) {
      if (k >= need) return;
      const int r = row_of(start, rows, k);
      if (start[r + 1] > free_pages) return;  // served in order, as long as pages last
      const int want = static_cast<int>((static_cast<long long>(a.tokens[r]) + (1 << a.page_shift) - 1) >> a.page_shift);
      const int c = want - (start[r + 1] - k);
      if (!CP_CHECK_DATA(c >= 0 && c < a.table.columns, a.status)) return;  // only where the arrays change under the kernel
      a.refs[page] = 1;
      a.table.pages[static_cast<size_t>(r) * a.table.columns + c] = page;
    });
  }
  for (int r = rank * kThreads + threadIdx.x; r < rows; r += cluster * kThreads) {
    const int want = wanted(a, r, a.table.held[r]);
    const bool ok = want != -2 && (start[r + 1] == start[r] || start[r + 1] <= free_pages);
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

__global__ void __launch_bounds__(kThreads) pages_fork_kernel(const __grid_constant__ ForkArgs a, int cluster) {
  __shared__ int start[kMaxTableRows + 1];
  __shared__ int8_t child[kMaxTableRows];
  __shared__ long long warp_totals[kWarps];
  __shared__ int warp_sums[kWarps], cta_sum;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = static_cast<int>(cluster_rank()), gw = rank * kWarps + warp, warps = cluster * kWarps;
  const int rows = a.dst.rows, rest = (1 << a.page_shift) - 1;
  pdl_wait();
  pdl_launch_dependents();
  scan_rows(rows, start, warp_totals, [&](int r) {
    const int c = is_child(a, r);
    child[r] = static_cast<int8_t>(c);
    if (c < 0 && rank == 0) debug_bounds_fail(a.status, __LINE__, CP_TU_ID);
    return c > 0 && (a.tokens[r] & rest) ? 1 : 0;
  });
  const int need = start[rows];
  // Every row's data have been read by the whole cluster behind the scan's barriers.
  const Stretch s(a.num_pages, gw, warps);
  int free_pages;
  const int before = cluster_scan(need > 0 ? count_free(a.refs, s, a.num_pages) : 0, cluster, warp_sums, &cta_sum, &free_pages);
  const int given = min(need, free_pages);
  each_free(a.refs, s, a.num_pages, before, given, [&](int page, int k) {
    if (k >= given) return;
    const int r = row_of(start, rows, k);  // its part page
    const int t = a.tokens[r], full = t >> a.page_shift, parent = a.parent[r];
    if (!CP_CHECK_DATA(parent >= 0 && parent < a.src.rows && full < a.dst.columns && full < a.src.columns, a.status)) return;  // as above
    a.refs[page] = 1;
    a.dst.pages[static_cast<size_t>(r) * a.dst.columns + full] = page;
    a.move_src[k] = a.src.pages[static_cast<size_t>(parent) * a.src.columns + full];
    a.move_dst[k] = page;
    a.move_tokens[k] = t & rest;
  });
  if (rank == 0 && threadIdx.x == 0) *a.count = given;
  for (int r = gw; r < rows; r += warps) {
    const bool ok = child[r] >= 0 && (start[r + 1] == start[r] || start[r + 1] <= free_pages);
    if (lane == 0) a.served[r] = ok;
    if (!ok || child[r] == 0) continue;
    const int full = a.tokens[r] >> a.page_shift, parent = a.parent[r];
    if (!CP_CHECK_DATA(full <= a.dst.columns && full <= a.src.columns && parent >= 0 && parent < a.src.rows, a.status)) continue;
    const int32_t* from = a.src.pages + static_cast<size_t>(parent) * a.src.columns;
    int32_t* to = a.dst.pages + static_cast<size_t>(r) * a.dst.columns;
    for (int c = lane; c < full; c += 32) {
      const int page = from[c];
      const bool there = CP_CHECK_DATA(page >= 0 && page < a.num_pages, a.status);
      if (there) atomicAdd(a.refs + page, 1);
      to[c] = there ? page : -1;
    }
    if (lane == 0) a.dst.held[r] = full + (start[r + 1] - start[r]);
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

__global__ void __launch_bounds__(kThreads) pages_compact_kernel(const __grid_constant__ CompactArgs a, int cluster) {
  __shared__ int warp_sums[kWarps], cta_sum, moved_here;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = static_cast<int>(cluster_rank()), gw = rank * kWarps + warp, warps = cluster * kWarps;
  const int P = a.num_pages;
  pdl_wait();
  pdl_launch_dependents();
  const Stretch s(P, gw, warps);
  int free_pages;
  const int before = cluster_scan(count_free(a.refs, s, P), cluster, warp_sums, &cta_sum, &free_pages);
  // Held pages from number `used` on move to the free ones below it, which are
  // as many: `moves`, the free pages before number `used`, known to the warp of that stretch.
  const int used = P - free_pages;
  const int per = ((P + warps - 1) / warps + 127) & ~127;
  const int owner = used / per;  // P / per at most, that is, perhaps behind the last warp
  if (gw == owner) {
    int n = before;
    each_free(a.refs, s, P, before, INT_MAX, [&](int page, int) { n += page < used; });
    n = before + __reduce_add_sync(0xffffffffu, n - before);
    if (lane == 0) moved_here = n;
  }
  cluster_barrier();
  const int moves = used < P ? ld_cluster(&moved_here, owner / kWarps) : 0;
  // Free pages below `used` in order, held ones from there on in order.
  const unsigned lower = (1u << lane) - 1;
  int n = before;
  for (int p = s.lo; p < s.hi; p += 128) {
    const int at = p + 4 * lane;
    const int4 v = load_refs(a.refs, at, P);
    const unsigned bits = free_bits(v);
    int mine = n;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned b = __ballot_sync(0xffffffffu, bits >> i & 1);
      mine += __popc(b & lower);
      n += __popc(b);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int page = at + i, held = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
      if (page >= P) break;
      const bool free_page = bits >> i & 1;
      if (a.refs_out != a.refs) a.refs_out[page] = page < used ? held : 0;
      if (page < used && free_page) {
        if (CP_CHECK_DATA(mine < P / 2, a.status)) a.move_dst[mine] = page;
      } else if (page >= used) {
        a.to[page] = -1;
        // page - mine held ones lie before it, used - moves of them below `used`.
        const int k = page - mine - (used - moves);
        if (!free_page && CP_CHECK_DATA(k >= 0 && k < P / 2, a.status)) a.move_src[k] = page;
      }
      mine += free_page;
    }
  }
  cluster_barrier();
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

// CTAs of a call that looks at `pages` counts and `rows` rows.
int cluster_for(int pages, int rows) {
  int c = 1;
  while (c < kMaxCluster && (pages > 8192 * c || rows > 256 * c)) c *= 2;
  return c;
}

template <typename K, typename A>
int launch_cluster(std::atomic<int> (&known)[64], K kernel, const A& a, int cluster, cudaStream_t stream) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CP_ERR_CUDA;
  if (!known[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) return CP_ERR_CUDA;
    known[dev].store(1, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster);
  cfg.blockDim = dim3(kThreads);
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
  if (!m || m->capacity < least || !m->count || !m->src || !m->dst || !m->tokens) return CP_ERR_INVALID_ARG;
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
  if (rc == CP_OK && (!tokens || !served)) rc = CP_ERR_INVALID_ARG;
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
  return launch_cluster(known, pages_resize_kernel, a, cluster_for(num_pages, table->rows), stream);
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
  if (rc == CP_OK && (!parent || !tokens || !served)) rc = CP_ERR_INVALID_ARG;
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
  return launch_cluster(known, pages_fork_kernel, a, cluster_for(num_pages, dst->rows), stream);
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
  rc = launch_cluster(known, pages_compact_kernel, a, cluster_for(num_pages, 0), stream);
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
  const unsigned grid = static_cast<unsigned>(units < 152 * 8 ? units : 152 * 8);
  NvtxRange range("cp_pages_copy");
  return launch(pages_copy_kernel, grid, kCopyThreads, 0, stream, a);
}

}  // extern "C"
