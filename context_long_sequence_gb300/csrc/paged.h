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
  void* workspace;
  int32_t* status;
};

int launch_paged_attn(const PagedAttnArgs& a, cudaStream_t stream);

// Device address of the status words on the current device (cp_attn.cu).
int32_t* device_status_ptr();

}  // namespace cpattn
