// paged.h -- geometry of a batch over the paged key/value cache, shared by
// the host layer (paged.cu) and the kernels (paged_append.cu,
// paged_attn.cu).  Not part of the public ABI.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime_api.h>

#include "cp_attn.h"

namespace cpattn {

constexpr int kMaxRopePairs = 64;  // rope_dim <= d <= 128

// Plan and batch, passed to the kernels by value.  The int32 arrays are the
// caller's device arrays; nothing in them is trusted: every row, page and
// length read from them is checked against the bounds held here.
struct PagedGeom {
  int Hq, Hkv, G, d;
  int page_shift;          // log2 of the page size
  int num_pages;
  int causal;
  int dtype;               // CP_DTYPE_*
  int B, N, NP;            // sequences, token rows, prefixes
  int max_new;             // most new tokens of one sequence
  int table_stride;        // columns of page_table
  int prefix_stride;       // columns of prefix_table
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* page_table;
  const int32_t* prefix_first;
  const int32_t* prefix_len;
  const int32_t* prefix_table;
  const int32_t* positions;
  int64_t page_stride, token_stride, head_stride;  // of the cache, in elements
  float scale;
};

// What the sequences share with the kernels' index arithmetic is in 32 bits:
// keys, rows and workspace rows stay below 2^30; units of work, cache offsets
// and byte offsets are 64-bit.

// One set of keys and the token rows that attend to it: entry e < B is
// sequence e with its own pages, entry B + p is prefix p with the rows of
// all its sequences.  n == 0: nothing to do.  Row i (of n) sees the first
// min(keys, limit0 + i) keys.
struct PagedEntry {
  int t0, n, keys, limit0;
  const int32_t* table;
  bool bad;  // the arrays break their bounds; n == 0
};

__host__ __device__ inline PagedEntry paged_entry(const PagedGeom& g, int e) {
  PagedEntry r{0, 0, 0, 0, nullptr, false};
  int a, b;
  long long cap;
  if (e < g.B) {
    a = g.q_start[e];
    b = g.q_start[e + 1];
    r.keys = g.kv_len[e];
    cap = static_cast<long long>(g.table_stride) << g.page_shift;
    r.table = g.page_table + static_cast<size_t>(e) * g.table_stride;
    r.bad = b - static_cast<long long>(a) > g.max_new;
  } else {
    const int p = e - g.B;
    const int f0 = g.prefix_first[p], f1 = g.prefix_first[p + 1];
    if (f0 < 0 || f1 < f0 || f1 > g.B) {
      r.bad = true;
      return r;
    }
    a = g.q_start[f0];
    b = g.q_start[f1];
    r.keys = g.prefix_len[p];
    cap = static_cast<long long>(g.prefix_stride) << g.page_shift;
    r.table = g.prefix_table + static_cast<size_t>(p) * g.prefix_stride;
  }
  if (r.bad || a < 0 || b < a || b > g.N || r.keys < 0 || r.keys > cap) {
    r.bad = true;
    r.keys = 0;
    return r;
  }
  r.t0 = a;
  r.n = b - a;
  r.limit0 = (e < g.B && g.causal) ? r.keys - r.n + 1 : r.keys;
  return r;
}

// How the attention of a batch is cut into work.  A cut takes the entries
// whose rows (tokens x query heads of a KV head) lie in [min_rows, max_rows],
// cuts their tokens into tiles of tile_tokens and each tile's visible keys
// into tiles of 2^key_shift.  One key tile of one token tile and KV head is a
// unit, and the loading and writing of its rows a few more; units are numbered entry by entry, KV head by KV head, token tile by
// token tile, and each of the W workers (CTAs) takes an equal, contiguous
// share of the numbers.  A token tile whose units fall to several workers
// has as many parts, merged afterwards by their log-sum-exp.  The cut depends
// on the batch's lengths alone, so the result does too.
struct PagedCut {
  int min_rows, max_rows;
  int tile_tokens, key_shift;  // tiles of 2^key_shift keys
  int lead;                    // units without keys that stand for a token tile's own cost
};

// Units of token tile `rb` of entry `e`: `lead`, then the key tiles it sees;
// none if it sees no key.
__host__ __device__ inline int paged_tile_units(const PagedCut& c, const PagedEntry& e, int rb) {
  const int last = (rb + 1) * c.tile_tokens < e.n ? (rb + 1) * c.tile_tokens - 1 : e.n - 1;
  const int seen = e.limit0 + last < e.keys ? e.limit0 + last : e.keys;
  return seen > 0 ? c.lead + ((seen + (1 << c.key_shift) - 1) >> c.key_shift) : 0;
}

// Units of entry `e` for one KV head.
__host__ __device__ inline long long paged_head_units(const PagedGeom& g, const PagedCut& c, const PagedEntry& e) {
  const long long rows = static_cast<long long>(e.n) * g.G;
  if (e.n <= 0 || rows < c.min_rows || rows > c.max_rows) return 0;
  if (e.n <= c.tile_tokens) return paged_tile_units(c, e, 0);
  const int tiles = (e.n + c.tile_tokens - 1) / c.tile_tokens;
  if (e.limit0 >= e.keys) return static_cast<long long>(tiles) * paged_tile_units(c, e, 0);  // all rows see all keys
  long long sum = 0;
  for (int rb = 0; rb < tiles; ++rb) sum += paged_tile_units(c, e, rb);
  return sum;
}

// Quotient of numbers that nearly always fit in 32 bits: a 64-bit division
// takes the device some 500 clocks, and a worker's start is a chain of them.
__host__ __device__ inline long long paged_div(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// `units` in `workers` contiguous shares, the first `extra` one larger.  At
// least min_units each, so that a short batch is not cut finer than its merge
// costs.
struct PagedShares {
  long long units, per;
  int workers, extra;
  __host__ __device__ PagedShares(long long n, int max_workers, int min_units) : units(n), per(0), workers(0), extra(0) {
    if (n <= 0) return;
    const long long most = paged_div(n + min_units - 1, min_units);
    workers = most < max_workers ? static_cast<int>(most) : max_workers;
    per = paged_div(n, workers);
    extra = static_cast<int>(n - per * workers);
  }
  __host__ __device__ long long first(int w) const { return w * per + (w < extra ? w : extra); }
  __host__ __device__ int worker_of(long long u) const {
    const long long large = extra * (per + 1);
    return static_cast<int>(u < large ? paged_div(u, per + 1) : extra + paged_div(u - large, per));
  }
};

// Workers and slots.  A worker holds at most two incomplete token tiles: the
// one its share begins in (its slot 2w) and the one its share ends in (slot
// 2w + 1); a part that is complete but has a partner (own keys and a prefix)
// goes to a home row of its own.
//
// Small: a warp (paged_small.cuh), 16 keys a tile, up to 8 or 16 rows, or 32
// where the batch has nothing larger; at least kSmallMinUnits tiles each.  Large: a
// CTA (paged_attn_large.cu), two blocks of up to 128 rows, 128 keys a tile.
constexpr int kSmallWorkers = 1216, kSmallRows = 32, kSmallKeyShift = 4;
constexpr int kSmallMinUnits = 4;
constexpr int kSmallLead = 2;
constexpr int kLargeWorkers = 152, kLargeRows = 256, kLargeKeyShift = 7;
constexpr int kLargeLead = 4;
constexpr int kMaxEntries = 8192;

inline __host__ __device__ PagedCut paged_cut_small(int G, int rows) {
  return PagedCut{1, rows, G <= rows ? rows / G : 1, kSmallKeyShift, kSmallLead};
}
inline __host__ __device__ PagedCut paged_cut_large(int G, int small_rows) {
  return PagedCut{small_rows + 1, 0x7fffffff, 2 * (kLargeRows / 2 / G), kLargeKeyShift, kLargeLead};
}

// Where a (token, KV head)'s parts over one entry are: G consecutive rows each.
struct PagedParts {
  int32_t first, second;  // rows of part 0 and part 1
  int32_t count, stride;  // parts, and rows from part 1 to part 2, ...
};

// The workspace: parts [2][N][Hkv] (own, prefix), then the rows' log-sum-exp
// (log2 units) and their normalised fp32 O.
struct PagedWorkspace {
  long long rows_small, rows_large_end, rows;  // small slots end, large slots end (home rows begin), all
  size_t parts, lse, o, total;             // byte offsets
};
inline __host__ __device__ PagedWorkspace paged_workspace(long long max_tokens, int Hq, int Hkv, int d, bool prefixes) {
  PagedWorkspace w;
  w.rows_small = 2LL * kSmallWorkers * kSmallRows;
  w.rows_large_end = w.rows_small + 2LL * kLargeWorkers * kLargeRows;
  w.rows = w.rows_large_end + (prefixes ? 2LL * max_tokens * Hq : 0);
  w.parts = 0;
  w.lse = (static_cast<size_t>(2 * max_tokens) * Hkv * sizeof(PagedParts) + 255) & ~size_t(255);
  w.o = w.lse + ((static_cast<size_t>(w.rows) * 4 + 255) & ~size_t(255));
  w.total = w.o + static_cast<size_t>(w.rows) * d * 4;
  return w;
}

struct AppendArgs {
  PagedGeom g;
  const void* q;           // or null
  const void* k;
  const void* v;
  void* q_out;
  void* k_cache;
  void* v_cache;
  int64_t q_stride, k_stride, v_stride, q_out_stride;  // between tokens, in elements
  int rope_dim, interleaved;
  // Pair j turns by pos * turns[j] / 2^64 of a full circle.
  uint64_t turns[kMaxRopePairs];
  int32_t* status;
};

int launch_paged_append(const AppendArgs& a, cudaStream_t stream);

struct PagedAttnArgs {
  PagedGeom g;
  const void* q;
  int64_t q_stride;        // between tokens, in elements
  const void* k_cache;
  const void* v_cache;
  void* o;                 // [N][Hq][d], the plan's type or fp32 (out_fp32)
  int out_fp32;
  float* lse;              // [Hq][N]
  PagedParts* parts;       // the workspace (PagedWorkspace)
  float* part_lse;
  float* part_o;
  long long rows_small, rows_large_end;
  int max_tokens;          // of the plan: home rows of prefixes follow max_tokens * Hq of the own keys
  int32_t* status;
};

int launch_paged_attn(const PagedAttnArgs& a, cudaStream_t stream);
// For batches that may have entries of more than kSmallRows rows (paged_attn_large.cu).
int launch_paged_large(const PagedAttnArgs& a, cudaStream_t stream);

// Device address of the status words on the current device (cp_attn.cu).
int32_t* device_status_ptr();

}  // namespace cpattn
