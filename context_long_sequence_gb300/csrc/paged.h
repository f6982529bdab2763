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

// Keys, rows and workspace rows stay below 2^30 and are held in 32 bits; units
// of work, cache offsets and byte offsets are 64-bit.

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

// How the attention of a batch is cut into work.  A cut takes some of the
// entries, cuts their tokens into tiles of tile_tokens and each tile's visible
// keys into tiles of 2^key_shift.  One key tile of one token tile and
// KV head is a unit, and the loading and writing of its rows a few more; units
// are numbered entry by entry, KV head by KV head, token tile by token tile,
// and each of the workers (warps or CTAs) takes an equal, contiguous share of
// the numbers.  A token tile whose units fall to several workers has as many
// parts, merged afterwards by their log-sum-exp.  The cut depends on the
// batch's lengths alone, so the result does too.
//
// Two sorts of worker.  A warp (paged_small.cuh): 16 keys a tile, and 8, 16 or
// (d = 64) 32 rows (tokens x query heads of a KV head), the fewest that hold a
// batch's entries.  A CTA (paged_attn_large.cu): two blocks of up to 128 rows,
// 128 keys a tile; in such a batch warps of 8 rows take some entries too.
//
// Between 8 and 32 rows, in us: 24 sequences of 20 rows on up to 30K keys take
// 446 by warps at d = 128 (their registers spill), 258 by CTAs; at d = 64 and
// 16K keys 75 by warps, 115 by CTAs.  Beside CTAs 16 rows spill in the loop over
// the keys: 40 sequences of 1 to 40 new tokens on up to 8K keys take 170 with
// warps of 8 rows, 396 with 16.  (With 8 the kernel of both stores 24 bytes a
// thread at d = 128 and 36 at d = 64, by the compiler's account.)
//
// Which kernel a batch gets goes by the most rows that its plan's max_new and
// the batch's n_tokens allow an entry, not by the lengths, which are on the
// device: a plan with room to spare gets the kernel of both (64 sequences of up
// to 16K keys 326 us by paged_small_kernel, 331 by paged_large_kernel's warps; 24
// drafts of 5 tokens at d = 64 20.8 and 30.0, after 16K keys 75 and 115).
struct PagedCut {
  int tile_tokens, key_shift;  // tiles of 2^key_shift keys
  int lead;                    // units without keys that stand for a token tile's own cost
};

constexpr int kSmallWarps = 8;  // workers of a CTA
constexpr int kSmallWorkers = 1216, kSmallRows = 32, kSmallKeyShift = 4;
constexpr int kSmallMinUnits = 3;  // of a worker, at least
constexpr int kSmallLead = 3;
constexpr int kBesideRows = 8, kBesideMaxRows = 128, kBesideWeight = 12;
constexpr int kLightUnits = 12;
constexpr int kLargeWorkers = 152, kLargeRows = 256, kLargeKeyShift = 7;
constexpr int kLargeLead = 4;
constexpr int kMaxEntries = 8192;

// Warps of `rows` rows.
inline __host__ __device__ PagedCut paged_cut_small(int G, int rows) {
  return PagedCut{G <= rows ? rows / G : 1, kSmallKeyShift, kSmallLead};
}
inline __host__ __device__ PagedCut paged_cut_large(int G) {
  return PagedCut{2 * (kLargeRows / 2 / G), kLargeKeyShift, kLargeLead};
}

// Whether an entry is the warps' in a batch that CTAs work on too: one of up
// to 8 rows, and one whose tiles of 8 rows, that read the keys once each, cost
// less than a CTA's one tile: short ones.  (In us, at weights 0, 8, 12, 16: 420
// sequences of 24 rows on up to 36 keys 149, 44, 44, 44; beside a prefix of 1000,
// 64 of 8 to 24 rows on 1000 keys 90, 90, 79, 79, and 64 of 12 on 1000 to 4000
// 139, 140, 178, 205.)
__host__ __device__ inline bool paged_by_warps(const PagedGeom& g, const PagedEntry& e) {
  const long long rows = static_cast<long long>(e.n) * g.G;
  if (rows <= kBesideRows) return true;
  if (g.G > kBesideRows || rows > kBesideMaxRows) return false;
  const long long warps = (rows + kBesideRows - 1) / kBesideRows * (((e.keys + 15) >> kSmallKeyShift) + kSmallLead);
  return warps <= kBesideWeight * (((e.keys + 127) >> kLargeKeyShift) + kLargeLead);
}

// Units of token tile `rb` of entry `e`: `lead`, then the key tiles it sees;
// none if it sees no key.
__host__ __device__ inline int paged_tile_units(const PagedCut& c, const PagedEntry& e, int rb) {
  const int last = (rb + 1) * c.tile_tokens < e.n ? (rb + 1) * c.tile_tokens - 1 : e.n - 1;
  const int seen = e.limit0 + last < e.keys ? e.limit0 + last : e.keys;
  return seen > 0 ? c.lead + ((seen + (1 << c.key_shift) - 1) >> c.key_shift) : 0;
}

// Units of entry `e` for one KV head.
__host__ __device__ inline long long paged_entry_units(const PagedCut& c, const PagedEntry& e) {
  if (e.n <= 0) return 0;
  if (e.n <= c.tile_tokens) return paged_tile_units(c, e, 0);
  const int tiles = (e.n + c.tile_tokens - 1) / c.tile_tokens;
  if (e.limit0 >= e.keys) return static_cast<long long>(tiles) * paged_tile_units(c, e, 0);  // all rows see all keys
  long long sum = 0;
  for (int rb = 0; rb < tiles; ++rb) sum += paged_tile_units(c, e, rb);
  return sum;
}

// The sums that decide how a batch with entries for CTAs is shared out: units
// of the entries that the warps take beside CTAs, of the CTAs' entries, and of
// all entries if the warps took them (too many where they cannot).  An entry's
// for one KV head, under cuts[0] of the warps and cuts[1] of the CTAs.
enum : int { kUnitsBeside = 0, kUnitsLarge = 1, kUnitsLight = 2, kUnitSums = 3 };
template <typename F>
__host__ __device__ inline void paged_unit_sums(const PagedGeom& g, const PagedCut (&cuts)[2], const PagedEntry& e,
                                                long long (&units)[kUnitSums], F&& entry_units) {
  const bool warps = paged_by_warps(g, e);
  units[kUnitsLight] = kLightUnits * kSmallWorkers + 1;
  if (warps || (g.G <= kBesideRows && static_cast<long long>(e.n) * g.G <= kBesideMaxRows))
    units[kUnitsLight] = entry_units(cuts[0], e);
  units[kUnitsBeside] = warps ? units[kUnitsLight] : 0;
  units[kUnitsLarge] = warps ? 0 : entry_units(cuts[1], e);
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

// A batch is light if all its entries, of up to 128 rows, are a few units for
// every warp in tiles of 8 rows: 7 sequences on a prefix of 2000 keys take 13.8
// us so and 17.2 with CTAs, 16 sequences 16.9 and 17.8; at kLightUnits 16, 7 on
// 8000 keys would take 22.2 and not 21.0.
inline __host__ __device__ bool paged_is_light(long long units, int ctas) {
  return units > 0 && units <= static_cast<long long>(kLightUnits) * kSmallWarps * ctas;
}

// Workers and slots.  A worker holds at most two incomplete token tiles: the
// one its share begins in (its slot 2w) and the one its share ends in (slot
// 2w + 1); a part that is complete but has a partner (own keys and a prefix)
// goes to a home row of its own.

// Where a (token, KV head)'s parts over one entry are: G consecutive rows each.
struct alignas(16) PagedParts {
  int32_t first, second;  // rows of part 0 and part 1
  int32_t count, stride;  // parts, and rows from part 1 to part 2, ...
};
// Whether the parts of G rows each lie among `rows` rows.  Where the batch's
// arrays are not ascending, entries overlap, and a row's record may be
// another entry's or none of this call's.
__host__ __device__ inline bool paged_parts_in(const PagedParts& p, int G, uint32_t rows) {
  if (p.count == 0) return true;
  const uint32_t count = static_cast<uint32_t>(p.count), first = static_cast<uint32_t>(p.first);
  const uint32_t second = static_cast<uint32_t>(p.second), stride = static_cast<uint32_t>(p.stride), last = rows - G;
  if (count > kSmallWorkers || first > last) return false;
  return count == 1 || (second <= last && stride <= 2 * kLargeRows && second + (count - 2) * stride <= last);
}

// CTAs for the entries of many rows, where a batch has both, by the time of
// their units: one is 256 rows x 128 keys, some 2750 clocks on the tensor core
// and the exponentials; one of few rows is 16 keys, about a twentieth of that
// for a CTA's eight warps (112 GB/s).  (64 sequences on a prefix of 32K keys,
// and 256 on two of 16K and 9K, in us at weights 12: 64.8, 106.5; 16: 60.5,
// 99.4; 20: 59.0, 96.1; 22: 58.7, 91.4; 24: 59.8, 93.1; 28: 63.2, 100.3.)
__host__ __device__ inline int paged_large_ctas(long long small, long long large, int ctas) {
  if (large == 0) return 0;
  if (small == 0) return ctas;
  const long long all = 22 * large + small;
  const int n = static_cast<int>(paged_div(22 * large * ctas + all / 2, all));
  return n < 1 ? 1 : n > ctas - 1 ? ctas - 1 : n;
}

// The most rows that an entry of the batch may have, and those that an entry
// of own keys may have.
__host__ __device__ inline long long paged_most_own_rows(const PagedGeom& g) {
  return static_cast<long long>(g.N < g.max_new ? g.N : g.max_new) * g.G;
}
__host__ __device__ inline long long paged_most_rows(const PagedGeom& g) {
  return g.NP > 0 ? static_cast<long long>(g.N) * g.G : paged_most_own_rows(g);
}
// Whether a batch of at most `most` rows an entry may have large entries; if
// not, the rows of the small workers' tiles.
__host__ __device__ inline int paged_small_rows(long long most) { return most <= 8 ? 8 : most <= 16 ? 16 : kSmallRows; }
__host__ __device__ inline bool paged_has_large(long long most, int d) { return most > (d == 64 ? kSmallRows : 16); }

// One run of key tiles of one token tile and KV head, as a worker gets it and
// as the fetching warp hands it to the others through shared memory.
struct PagedSegment {
  int t0, nt;                 // the tile's tokens; nt == 0: no more segments
  int h;                      // KV head
  int keys, limit0;           // keys of the entry; token t0 + i sees min(keys, limit0 + i)
  int tile0, tile1;           // key tiles of this run
  // Where the rows go: straight to o and lse (final), or to part rows: row of
  // (token, head) is row + token * Hq + head (home), row r of the token tile
  // is row + r (slot).
  int mode, row;
};
enum : int { kRowsFinal = 0, kRowsHome = 1, kRowsSlot = 2 };

// Where the parts of token `i` of a segment's tile are, for the run that
// begins the tile's keys: the token's G rows from first + i * first_step and
// second + i * G on.
struct PagedRecord {
  int first, first_step, second, count, stride;
};

// What a worker takes of entry `id` from unit `rel` of the entry on, of the
// `left` units that it still has: fills `s` (nt == 0: only a lead) and `rec`
// (count == 0: the run does not begin its token tile), and returns the units
// taken.
struct PagedPlace {
  int worker, slots, slot_rows;  // the cut's first slot row and rows of a slot
  int home, home_prefix;         // first home row of own keys and of prefixes
  int covered0, covered1;        // sequences that belong to some prefix
  int B, G, Hq;
};
__host__ __device__ inline long long paged_take(const PagedCut& c, const PagedShares& shares, const PagedPlace& at, int id,
                                                const PagedEntry& e, long long head_units, long long rel, long long u,
                                                long long left, PagedSegment& s, PagedRecord& rec) {
  s.h = static_cast<int>(paged_div(rel, head_units));
  rel -= s.h * head_units;
  int rb = 0, tiles = paged_tile_units(c, e, 0);
  while (rel >= tiles && (rb + 1) * c.tile_tokens < e.n) {
    rel -= tiles;
    tiles = paged_tile_units(c, e, ++rb);
  }
  const long long u0 = u - rel;  // the token tile's first unit
  const int stop = static_cast<int>(rel + left < tiles ? rel + left : tiles);
  s.t0 = e.t0 + rb * c.tile_tokens;
  s.nt = e.n - rb * c.tile_tokens < c.tile_tokens ? e.n - rb * c.tile_tokens : c.tile_tokens;
  s.keys = e.keys;
  s.limit0 = e.limit0 + rb * c.tile_tokens;
  s.tile0 = rel > c.lead ? static_cast<int>(rel) - c.lead : 0;
  s.tile1 = stop - c.lead;
  rec.count = 0;
  if (s.tile1 <= s.tile0) {  // only its lead falls to this worker
    s.nt = 0;
    return stop - rel;
  }
  const bool prefix = id >= at.B, begins = s.tile0 == 0, whole = begins && stop == tiles;
  if (whole) {
    s.mode = prefix || (id >= at.covered0 && id < at.covered1) ? kRowsHome : kRowsFinal;
    s.row = prefix ? at.home_prefix : at.home;
  } else {
    s.mode = kRowsSlot;
    s.row = at.slots + (2 * at.worker + (begins ? 1 : 0)) * at.slot_rows;
  }
  if (begins) {
    rec.first = s.mode == kRowsSlot ? s.row : s.row + s.t0 * at.Hq + s.h * at.G;
    rec.first_step = s.mode == kRowsSlot ? at.G : at.Hq;
    rec.second = at.slots + 2 * (at.worker + 1) * at.slot_rows;
    rec.count = (whole ? at.worker : shares.worker_of(u0 + tiles - 1)) - at.worker + 1;
    rec.stride = 2 * at.slot_rows;
  }
  return stop - rel;
}

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
  uint32_t rows;           // all of them
  int max_tokens;          // of the plan: home rows of prefixes follow max_tokens * Hq of the own keys
  int32_t* status;
};

int launch_paged_attn(const PagedAttnArgs& a, cudaStream_t stream);
// For batches that may have entries of more rows than paged_small_kernel's tiles
// (paged_has_large): 16 at d = 128, 32 at d = 64 (paged_attn_large.cu).
int launch_paged_large(const PagedAttnArgs& a, cudaStream_t stream);

// Device address of the status words on the current device (cp_attn.cu).
int32_t* device_status_ptr();

}  // namespace cpattn
