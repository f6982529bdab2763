// paged.cuh -- what the paged-cache kernels share: the walk over a worker's
// units, the targets of its rows, TMA boxes of the cache, launches.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "debug.cuh"
#include "paged.h"
#include "ptx.cuh"
#include "tmap.h"

namespace cpattn {

// File ids of the status record, after those in debug.cuh.
enum : int32_t { kTuPagedAppend = 6, kTuPagedAttn = 7, kTuRope = 8, kTuVerify = 9, kTuPages = 10 };

// The batch arrays and page numbers are data that no host check has seen;
// these checks are therefore in every build, unlike CP_IN_BOUNDS.
#define CP_CHECK_DATA(cond, status) ((cond) || ::cpattn::debug_bounds_fail((status), __LINE__, CP_TU_ID))

// mbar_wait (ptx.cuh) with the clock first looked at after 16 failed tries:
// reading %globaltimer takes longer than most of these kernels' waits.  The
// same limit, abort flag and status.
__device__ __forceinline__ bool mbar_wait_short(uint32_t bar, uint32_t parity, volatile int* abort, int32_t* status) {
  for (int i = 0; i < 16; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait(bar, parity, abort, status);
}

// Number of the n elements of the ascending array `a` that are <= t.  Executed
// by a whole warp: 32 probes a round, so 1024 elements take two dependent
// loads.  Ends after log32(n) rounds whatever the data.
__device__ __forceinline__ int warp_count_le(const int32_t* a, int n, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;
  while (hi - lo > 32) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step + step - 1;
    const int c = __popc(__ballot_sync(0xffffffffu, i < hi && a[i] <= t));
    lo = min(hi, lo + c * step);
    hi = min(hi, lo + step);
  }
  const int i = lo + lane;
  return lo + __popc(__ballot_sync(0xffffffffu, i < hi && a[i] <= t));
}

// Prefix of sequence s, or -1: the p with prefix_first[p] <= s < prefix_first[p + 1].
__device__ __forceinline__ int warp_prefix_of(const PagedGeom& g, int s) {
  if (g.NP == 0 || g.prefix_first[0] > s) return -1;
  const int p = warp_count_le(g.prefix_first + 1, g.NP, s);
  return p < g.NP ? p : -1;
}

// Programmatic dependent launch: `launch_dependents` lets the next kernel of
// the stream begin as SMs fall free; `wait` returns once the kernel before
// this one has completed and its writes are visible.  Every kernel here is
// launched so, and
//   - touches no memory before its wait, except the merge, which reads the
//     batch's arrays first: the attention kernel lets it begin only after its
//     own wait, that is, when all that the arrays may come from is done;
//   - waits in every block, so that whoever waits for it waits for all before.
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ long long shfl64(long long x, int lane) { return __shfl_sync(0xffffffffu, x, lane); }

// Debug builds (debug.cuh): whether rows of the workspace, tokens and query
// heads of the batch, and boxes of the cache are there.
__device__ __forceinline__ bool part_rows_in(const PagedAttnArgs& a, long long row, int n) {
  return row >= 0 && row + n <= static_cast<long long>(a.rows);
}
__device__ __forceinline__ bool token_in(const PagedGeom& g, long long token, int head) {
  return token >= 0 && token < g.N && head >= 0 && head < g.Hq;
}
__device__ __forceinline__ bool cache_box_in(const PagedGeom& g, int row, int rows, int head, int page) {
  return row >= 0 && row + rows <= 1 << g.page_shift && head >= 0 && head < g.Hkv && page >= 0 && page < g.num_pages;
}

// Sine and cosine of pos * turns / 2^64 of a full circle (paged_append.cu says
// to what they are good).
__device__ __forceinline__ void sincos_turns(int pos, uint64_t turns, float* s, float* c) {
  const uint64_t x = static_cast<uint64_t>(static_cast<int64_t>(pos)) * turns;
  sincospif(static_cast<float>(static_cast<int32_t>(x >> 32)) * 4.656612873077393e-10f, s, c);  // 2^-31
}

// A barrier of the block's first `threads` threads.
__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("barrier.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Which share a warp takes up: of the units of sum `sum` under cut number
// `cut`, as worker `worker` of at most max_workers with at least min_units
// units each; its slots.
struct PagedRole {
  int sum, cut, worker, max_workers, min_units, slots, slot_rows;
};

__device__ __noinline__ inline long long paged_entry_units_call(int n, int keys, int limit0, PagedCut c) {
  return paged_entry_units(c, PagedEntry{0, n, keys, limit0, nullptr, false});
}

// Walks a worker's units, one warp, 32 entries at a time, an entry a lane.
// Every warp that walks totals the units and chooses; a CTA's one that fetches
// goes on to walk.  SUMS: 1, a batch for warps alone, or kUnitSums.
//
// Code that a CTA runs once comes from L2 line by line, the same lines for
// all SMs at once, some 12 clocks an instruction: this is written to be short.
// Of kUnitSums the entries' units are counted by a call, in one copy (for one
// sum the call costs more than it saves: decode_1x1000 8.0 -> 8.2 us).
template <int SUMS>
struct PagedWalker {
  static constexpr int kCuts = SUMS == 1 ? 1 : 2;
  const PagedAttnArgs& a;
  const PagedGeom& g;
  const PagedCut (&cuts)[kCuts];
  PagedCut cut;
  int sum = 0;                 // the role's
  PagedPlace place;
  int E;
  PagedShares shares;
  long long u, end;            // this worker's next unit and last + 1
  int base = -1;               // first entry of the window; -1: none is held
  long long before;            // units before the window
  PagedEntry entry;            // the lane's
  long long head_units, upto;  // its units of one head; units of the window up to and including it
  const int32_t* table;        // page table of the last segment's entry
  bool once;                   // no other token tile reads its keys

  __device__ __forceinline__ PagedWalker(const PagedAttnArgs& args, const PagedCut (&c)[kCuts])
      : a(args), g(args.g), cuts(c), E(args.g.B + args.g.NP), shares(0, 1, 1) {}

  // The window from entry `first` on, and the units of the lane's entry.
  __device__ __forceinline__ void load(int first, long long (&x)[SUMS]) {
    const int lane = threadIdx.x & 31;
    base = first;
    entry = PagedEntry{0, 0, 0, 0, nullptr, false};
    if (base + lane < E) entry = paged_entry(g, base + lane);
    if (entry.bad) debug_bounds_fail(a.status, __LINE__, kTuPagedAttn);
    if constexpr (SUMS == 1)
      x[0] = paged_entry_units(cuts[0], entry);
    else
      paged_unit_sums(g, cuts, entry, x, [](const PagedCut& c, const PagedEntry& e) {
        return paged_entry_units_call(e.n, e.keys, e.limit0, c);
      });
  }
  __device__ __forceinline__ long long pick(const long long (&x)[SUMS]) const {
    long long r = x[0];
#pragma unroll
    for (int i = 1; i < SUMS; ++i) r = sum == i ? x[i] : r;
    return r;
  }
  __device__ __forceinline__ void scan(long long of_head) {
    const int lane = threadIdx.x & 31;
    head_units = of_head;
    upto = head_units * g.Hkv;
#pragma unroll 1
    for (int x = 1; x < 32; x <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, upto, x);
      if (lane >= x) upto += y;
    }
  }

  // The worker's place among the units.  Called by the block's first `warps`
  // warps: they total the units (`sums`: SUMS numbers in shared memory for
  // each window of 32 entries), and choose(units) returns the PagedRole of the
  // calling warp.  False: nothing for it.  `sums` is free once every warp has
  // returned.
  template <typename F>
  __device__ __forceinline__ bool start(long long* sums, int warps, F&& choose) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int windows = (E + 31) / 32;
    const bool alone = windows == 1;
    place.covered0 = g.NP > 0 ? g.prefix_first[0] : 0;
    place.covered1 = g.NP > 0 ? g.prefix_first[g.NP] : 0;
    long long x[SUMS], units[SUMS];
    bool chosen = false;
    int w = alone ? 0 : warp;
#pragma unroll 1
    while (true) {
      if (w < windows) {
        load(w * 32, x);
        if (chosen) break;
#pragma unroll
        for (int i = 0; i < SUMS; ++i) {
          const long long y = x[i] * g.Hkv;  // below 2^48: two 24-bit sums of 32 each
          const unsigned lo = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(y & 0xffffff));
          const unsigned hi = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(y >> 24));
          units[i] = (static_cast<long long>(hi) << 24) + lo;
          if (!alone && lane == 0) sums[w * SUMS + i] = units[i];
        }
      }
      if (!alone) {
        w += warps;
        if (w < windows) continue;
        named_barrier(1, warps * 32);
#pragma unroll
        for (int i = 0; i < SUMS; ++i) {
          units[i] = 0;
#pragma unroll 1
          for (int k = 0; k < windows; ++k) units[i] += sums[k * SUMS + i];
        }
      }
      const PagedRole r = choose(units);
      cut = cuts[kCuts == 1 ? 0 : r.cut];
      sum = r.sum;
      place.worker = r.worker;
      place.slots = r.slots;
      place.slot_rows = r.slot_rows;
      place.home = static_cast<int>(a.rows_large_end);
      place.home_prefix = place.home + a.max_tokens * g.Hq;
      place.B = g.B;
      place.G = g.G;
      place.Hq = g.Hq;
      shares = PagedShares(pick(units), r.max_workers, r.min_units);
      before = 0;
      if (r.worker >= shares.workers) return false;
      u = shares.first(r.worker);
      end = shares.first(r.worker + 1);
      if (alone) break;
#pragma unroll 1
      for (w = 0; w + 1 < windows && before + sums[w * SUMS + sum] <= u; ++w) before += sums[w * SUMS + sum];
      chosen = true;
    }
    scan(pick(x));
    return true;
  }

  // The next segment (warp-uniform), nt == 0 behind the last.  The run that
  // begins a token tile's keys also records where the tile's parts are.
  __device__ __forceinline__ PagedSegment next() {
    PagedSegment s{0, 0, 0, 0, 0, 0, 0, 0, 0};
    while (u < end) {
      long long total = shfl64(upto, 31);
      while (u >= before + total) {
        if (base + 32 >= E) {  // only where the arrays changed under the kernel
          end = u;
          return s;
        }
        before += total;
        long long x[SUMS];
        load(base + 32, x);
        scan(pick(x));
        total = shfl64(upto, 31);
      }
      long long rel = u - before;
      const int at = __ffs(__ballot_sync(0xffffffffu, upto > rel)) - 1;  // exists: rel < total
      const long long hu = shfl64(head_units, at);
      rel -= shfl64(upto, at) - hu * g.Hkv;
      const int id = base + at;
      PagedEntry e;
      e.t0 = __shfl_sync(0xffffffffu, entry.t0, at);
      e.n = __shfl_sync(0xffffffffu, entry.n, at);
      e.keys = __shfl_sync(0xffffffffu, entry.keys, at);
      e.limit0 = __shfl_sync(0xffffffffu, entry.limit0, at);
      once = e.n <= cut.tile_tokens;
      const bool prefix = id >= g.B;
      table = prefix ? g.prefix_table + static_cast<size_t>(id - g.B) * g.prefix_stride
                     : g.page_table + static_cast<size_t>(id) * g.table_stride;
      PagedRecord rec;
      u += paged_take(cut, shares, place, id, e, hu, rel, u, end - u, s, rec);
      if (s.nt == 0) continue;
      if (rec.count > 0) {
        PagedParts* parts = a.parts + (prefix ? static_cast<size_t>(a.max_tokens) * g.Hkv : 0);
        for (int i = threadIdx.x & 31; i < s.nt; i += 32)
          if (CP_IN_BOUNDS(s.t0 >= 0 && s.t0 + i < a.max_tokens && s.h < g.Hkv, a.status))
            parts[static_cast<size_t>(s.t0 + i) * g.Hkv + s.h] =
                PagedParts{rec.first + i * rec.first_step, rec.second + i * g.G, rec.count, rec.stride};
      }
      break;
    }
    return s;
  }
};

template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float2 unpack(uint32_t x) {
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_bf16x2(lo, hi); }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ float2 unpack(uint32_t x) {
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};

// Weights are 2^(s - m + kBias).  The running maximum m is raised only when a
// score exceeds it by kSlack (log2 units), so O is rescaled rarely; the final
// division uses the same m.  bf16 has fp32's exponents and needs no bias.  In
// fp16 a weight below 2^-14 loses bits and one below 2^-25 vanishes, which the
// flat tail of a long context would show: with the bias a weight keeps its
// bits down to 2^-23 of the largest, and a million keys below that are off by
// at most 2^-14 of the sum, under fp16's own half step of 2^-11.
// kSpecSum and kSpecMax bound weights taken before their maximum is known
// (paged_attn_large.cu): a sum of weights, and one score over m.  kBelow: what
// the first of a weight's two halves is the rounding of (paged_small.cuh).
template <typename T>
struct Weight {
  static constexpr float kBias = 0.f, kSlack = 8.f, kSpecSum = 65536.f, kSpecMax = 16.f;
  static constexpr float kBelow = 1.f - 0x1p-8f - 0x1p-14f;
};
template <>
struct Weight<__half> {
  static constexpr float kBias = 9.f, kSlack = 2.f, kSpecSum = 60000.f, kSpecMax = 6.5f;
  static constexpr float kBelow = 1.f - 0x1p-11f - 0x1p-13f;
};

// L2 policy of keys that are read once, and of all that warps read: first to
// go, so that a step's stream of keys does not push out the queries, the parts
// and the kernels' own code (64 sequences on a prefix of 32K keys 74.8 -> 68.5 us).  Warps beside CTAs have it
// for short entries of up to 16 token tiles too, that read their keys again: a
// policy by entry there took 256 sequences on prefixes from 93.5 to 95.9 us.
__device__ __forceinline__ uint64_t read_once_policy() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint64_t read_again_policy() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z, int w,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, %4, "
      "%5, %6}], [%2], %7;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w),
      "l"(policy)
      : "memory");
}

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z, int w,
                                            int v, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, %4, "
      "%5, %6, %7}], [%2], %8;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w),
      "r"(v), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y), "r"(z)
               : "memory");
}
// At most N of the thread's groups have yet to read their source; all of them
// have written.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// 16 bytes from global to shared memory, asynchronously; both addresses
// 16-byte aligned.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr) : "memory");
  return r;
}

// ---------------------------------------------------------------- host side

// 4-D map over the cache: columns, tokens of a page, heads, pages; boxes of
// 64 columns (128 bytes, swizzled) x box_rows tokens.  L2 fetches 128 bytes at
// a time: with 256, a row of d = 64 brings the next head's, which has left
// again when it is wanted (24 sequences of 64K keys, 4 heads of 64 side by
// side: 343 us with 256, 257 with 128; rows of 256 bytes are indifferent).
inline bool make_cache_map(CUtensorMap* m, const PagedGeom& g, const void* base, int box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(g.d), static_cast<cuuint64_t>(1) << g.page_shift,
                        static_cast<cuuint64_t>(g.Hkv), static_cast<cuuint64_t>(g.num_pages)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(g.token_stride) * 2, static_cast<cuuint64_t>(g.head_stride) * 2,
                           static_cast<cuuint64_t>(g.page_stride) * 2};
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_rows), 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(m, g.dtype == CP_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
             const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same with the 64-column pieces of a head as a dimension of their own: a
// box is box_rows tokens of the whole head, piece by piece.
inline bool make_cache_map_whole(CUtensorMap* m, const PagedGeom& g, const void* base, int box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint32_t pieces = g.d / 64;
  cuuint64_t dims[5] = {64, static_cast<cuuint64_t>(1) << g.page_shift, pieces, static_cast<cuuint64_t>(g.Hkv),
                        static_cast<cuuint64_t>(g.num_pages)};
  cuuint64_t strides[4] = {static_cast<cuuint64_t>(g.token_stride) * 2, 128, static_cast<cuuint64_t>(g.head_stride) * 2,
                           static_cast<cuuint64_t>(g.page_stride) * 2};
  cuuint32_t box[5] = {64, static_cast<cuuint32_t>(box_rows), pieces, 1, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return enc(m, g.dtype == CP_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5,
             const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A launch that may begin while the kernel before it in the stream still
// runs (it calls griddepcontrol.wait before it reads that kernel's results).
template <typename... P, typename... A>
int launch(void (*kernel)(P...), unsigned grid, int threads, int smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? CP_OK : CP_ERR_CUDA;
}

// The current device's SM count, and the kernel's shared-memory limit raised
// there; once per device (concurrent first calls do the same).
template <typename K>
int prepare_kernel(std::atomic<int> (&known)[64], K kernel, int smem, int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CP_ERR_CUDA;
  int n = known[dev].load(std::memory_order_acquire);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return CP_ERR_CUDA;
    known[dev].store(n, std::memory_order_release);
  }
  *sms = n;
  return CP_OK;
}

}  // namespace cpattn
