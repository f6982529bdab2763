// paged.cu -- the C ABI of the paged key/value cache (include/cp_attn.h):
// plan validation, workspace sizing and argument checks of cp_cache_append
// and cp_attn_paged.  Host code only; the kernels live in paged_append.cu and
// paged_attn.cu.
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cmath>
#include <new>

#include "paged.h"

using cpattn::PagedGeom;

struct cp_paged {
  cp_paged_desc_t desc;
  int page_shift;
  float scale;
  uint64_t turns[cpattn::kMaxRopePairs];  // of a full circle per position, 64-bit fraction
};

namespace {

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

constexpr long long kMaxKeys = 1LL << 30;  // of one page table row; key indices and limits stay in 32 bits
constexpr long long kMaxRows = 1LL << 30;  // of the workspace's home rows
constexpr int64_t kMaxStride = 1LL << 36;  // elements; a tensor map takes strides below 2^40 bytes
constexpr int64_t kMaxSpan = 1LL << 60;    // elements from the cache's first to its last; offsets stay in 64 bits

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The kernels are built for sm_103 alone; asked once per device.
int check_arch() {
  static int known[64];  // 0 unknown, 1 sm_103, -1 other; racing calls store the same value
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CP_ERR_CUDA;
  int k = __atomic_load_n(&known[dev], __ATOMIC_RELAXED);
  if (k == 0) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
      return CP_ERR_CUDA;
    k = major == 10 && minor == 3 ? 1 : -1;
    __atomic_store_n(&known[dev], k, __ATOMIC_RELAXED);
  }
  return k > 0 ? CP_OK : CP_ERR_ARCH;
}

int check_cache(const cp_paged_desc_t& d, const cp_paged_cache_t& c) {
  if (!c.k || !c.v || c.num_pages <= 0) return CP_ERR_INVALID_ARG;
  if (!aligned(c.k, 16) || !aligned(c.v, 16)) return CP_ERR_ALIGNMENT;
  const int64_t s[3] = {c.page_stride, c.token_stride, c.head_stride};
  const int64_t n[3] = {c.num_pages, d.page_size, d.Hkv};
  for (int i = 0; i < 3; ++i)
    if (s[i] < d.d || s[i] >= kMaxStride || s[i] % 8) return CP_ERR_INVALID_ARG;
  // Rows do not overlap: in ascending order each stride spans what lies below it.
  int o[3] = {0, 1, 2};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (s[o[j]] > s[o[j + 1]]) {
        const int x = o[j];
        o[j] = o[j + 1];
        o[j + 1] = x;
      }
  int64_t span = d.d;
  for (int i = 0; i < 3; ++i) {
    if (n[o[i]] == 1) continue;
    if (s[o[i]] < span || n[o[i]] - 1 > (kMaxSpan - span) / s[o[i]]) return CP_ERR_INVALID_ARG;
    span += s[o[i]] * (n[o[i]] - 1);
  }
  return CP_OK;
}

int check_batch(const cp_paged_desc_t& d, const cp_paged_batch_t& b) {
  if (b.n_seqs < 0 || b.n_seqs > d.max_seqs || b.n_tokens < 0 || b.n_tokens > d.max_tokens) return CP_ERR_INVALID_ARG;
  if (b.n_prefixes < 0 || b.n_prefixes > d.max_prefixes) return CP_ERR_INVALID_ARG;
  if (b.n_seqs > 0 && b.n_tokens > 0) {
    if (!b.q_start || !b.kv_len || !b.page_table) return CP_ERR_INVALID_ARG;
    if (b.n_prefixes > 0 && (!b.prefix_first || !b.prefix_len || !b.prefix_table)) return CP_ERR_INVALID_ARG;
  }
  const void* arrays[] = {b.q_start, b.kv_len, b.page_table, b.prefix_first, b.prefix_len, b.prefix_table, b.positions};
  for (const void* a : arrays)
    if (!aligned(a, 4)) return CP_ERR_ALIGNMENT;
  return CP_OK;
}

// A token-major tensor: heads contiguous, tokens `stride` elements apart.
int check_tokens(const void* p, int64_t stride, int heads, int d) {
  if (!p || stride < static_cast<int64_t>(heads) * d || stride >= kMaxStride || stride % 8) return CP_ERR_INVALID_ARG;
  return aligned(p, 16) ? CP_OK : CP_ERR_ALIGNMENT;
}

// The fraction of a full circle in x >= 0 turns, in units of 2^-64.
uint64_t fraction(double x) { return static_cast<uint64_t>(std::ldexp(x - std::floor(x), 64)); }

// f radians as a fraction of a full circle: f / 2 pi = high + low, high the
// rounded product and low what it leaves out, with 1 / 2 pi to 110 bits.  Off
// by at most 2^-63 for |f| up to 2^42 (two cuts at 2^-64; the constant and
// low's rounding stay below |f| 2^-106); f / 2 pi in one double would be off by
// 2^-54 times itself, which a position of 2^31 makes 10^-5 radians at f = 100.
uint64_t turns_of(double f) {
  constexpr double kHigh = 0.15915494309189535, kLow = -9.839338337591243e-18;
  const double x = std::fabs(f);
  const volatile double product = x * kHigh;  // rounded: never fused with what follows
  const double high = product, low = std::fma(x, kLow, std::fma(x, kHigh, -high));
  const uint64_t rest = fraction(std::fabs(low));
  const uint64_t turns = fraction(high) + (low < 0 ? 0 - rest : rest);
  return f < 0 ? 0 - turns : turns;
}

PagedGeom geom(const cp_paged& p, const cp_paged_cache_t& c, const cp_paged_batch_t& b) {
  const cp_paged_desc_t& d = p.desc;
  PagedGeom g;
  g.Hq = d.Hq;
  g.Hkv = d.Hkv;
  g.G = d.Hq / d.Hkv;
  g.d = d.d;
  g.page_shift = p.page_shift;
  g.num_pages = c.num_pages;
  g.causal = d.causal;
  g.dtype = d.dtype;
  g.B = b.n_seqs;
  g.N = b.n_tokens;
  g.NP = b.n_prefixes;
  g.max_new = d.max_new;
  g.table_stride = d.max_pages;
  g.prefix_stride = d.max_prefix_pages;
  g.q_start = b.q_start;
  g.kv_len = b.kv_len;
  g.page_table = b.page_table;
  g.prefix_first = b.prefix_first;
  g.prefix_len = b.prefix_len;
  g.prefix_table = b.prefix_table;
  g.positions = b.positions;
  g.page_stride = c.page_stride;
  g.token_stride = c.token_stride;
  g.head_stride = c.head_stride;
  g.scale = p.scale;
  return g;
}

}  // namespace

extern "C" {

int cp_paged_create(const cp_paged_desc_t* desc, cp_paged_t** out) {
  if (!desc || !out) return CP_ERR_INVALID_ARG;
  const cp_paged_desc_t& d = *desc;
  if (d.version != CP_PAGED_VERSION) return CP_ERR_INVALID_ARG;
  if (d.dtype != CP_DTYPE_BF16 && d.dtype != CP_DTYPE_FP16) return CP_ERR_INVALID_ARG;
  if (d.Hq <= 0 || d.Hkv <= 0 || d.Hq % d.Hkv) return CP_ERR_INVALID_ARG;
  if (d.page_size <= 0 || d.max_seqs <= 0 || d.max_tokens <= 0 || d.max_new <= 0 || d.max_pages <= 0)
    return CP_ERR_INVALID_ARG;
  if (d.max_prefixes < 0 || d.max_prefix_pages < 0 || (d.max_prefixes > 0) != (d.max_prefix_pages > 0))
    return CP_ERR_INVALID_ARG;
  if ((d.causal | 1) != 1 || (d.out_fp32 | 1) != 1 || (d.rope_interleaved | 1) != 1) return CP_ERR_INVALID_ARG;
  if (!(d.softmax_scale >= 0.f) || std::isinf(d.softmax_scale * 1.4426950408889634f)) return CP_ERR_INVALID_ARG;  // scores are in log2 units
  if (d.rope_dim < 0 || d.rope_dim > d.d) return CP_ERR_INVALID_ARG;
  if (static_cast<long long>(d.max_pages) * d.page_size >= kMaxKeys ||
      static_cast<long long>(d.max_prefix_pages) * d.page_size >= kMaxKeys ||
      2LL * d.max_tokens * d.Hq >= kMaxRows ||
      static_cast<long long>(d.max_seqs) + d.max_prefixes > cpattn::kMaxEntries)
    return CP_ERR_INVALID_ARG;
  if (d.d != 64 && d.d != 128) return CP_ERR_UNSUPPORTED;
  if (d.page_size < 16 || d.page_size > 65536 || (d.page_size & (d.page_size - 1))) return CP_ERR_UNSUPPORTED;
  if (d.Hq / d.Hkv > 128 || d.rope_dim % 16) return CP_ERR_UNSUPPORTED;
  if (d.rope_dim > 0 && !d.rope_freqs && !(d.rope_base > 0 && std::isfinite(d.rope_base))) return CP_ERR_INVALID_ARG;
  if (d.rope_dim > 0 && d.rope_freqs)
    for (int j = 0; j < d.rope_dim / 2; ++j)
      if (!std::isfinite(d.rope_freqs[j])) return CP_ERR_INVALID_ARG;
  cp_paged* p = new (std::nothrow) cp_paged();
  if (!p) return CP_ERR_CUDA;
  p->desc = d;
  p->desc.rope_freqs = nullptr;
  for (p->page_shift = 0; (1 << p->page_shift) < d.page_size;) ++p->page_shift;
  p->scale = d.softmax_scale > 0.f ? d.softmax_scale : 1.0f / std::sqrt(static_cast<float>(d.d));
  for (int j = 0; j < d.rope_dim / 2; ++j)
    p->turns[j] = turns_of(d.rope_freqs ? d.rope_freqs[j] : std::pow(d.rope_base, -2.0 * j / d.rope_dim));
  *out = p;
  return CP_OK;
}

void cp_paged_destroy(cp_paged_t* p) { delete p; }

int cp_paged_workspace_size(const cp_paged_t* p, size_t* bytes) {
  if (!p || !bytes) return CP_ERR_INVALID_ARG;
  const cp_paged_desc_t& d = p->desc;
  *bytes = cpattn::paged_workspace(d.max_tokens, d.Hq, d.Hkv, d.d, d.max_prefixes > 0).total;
  return CP_OK;
}

int cp_paged_shares(const cp_paged_t* p, const cp_paged_batch_t* batch, int32_t ctas, int32_t* rows, int64_t capacity,
                    int64_t* n_rows) {
  if (!p || !batch || !n_rows || ctas < 2 || ctas > cpattn::kLargeWorkers || capacity < 0 || (capacity > 0 && !rows))
    return CP_ERR_INVALID_ARG;
  const cp_paged_desc_t& d = p->desc;
  const int rc = check_batch(d, *batch);
  if (rc != CP_OK) return rc;
  *n_rows = 0;
  if (batch->n_seqs == 0 || batch->n_tokens == 0) return CP_OK;
  using namespace cpattn;
  cp_paged_cache_t none = {};
  const PagedGeom g = geom(*p, none, *batch);
  const PagedWorkspace w = paged_workspace(d.max_tokens, d.Hq, d.Hkv, d.d, d.max_prefixes > 0);
  const long long most = paged_most_rows(g);
  const bool both = paged_has_large(most, g.d);
  const PagedCut cuts[2] = {paged_cut_small(g.G, both ? kBesideRows : paged_small_rows(most)), paged_cut_large(g.G)};
  // Units of an entry for one KV head, of the sum `which`.
  const auto head_units = [&](const PagedEntry& e, int which) {
    if (!both) return which == kUnitsBeside ? paged_entry_units(cuts[0], e) : 0;
    long long x[kUnitSums];
    paged_unit_sums(g, cuts, e, x, paged_entry_units);
    return x[which];
  };
  long long units[kUnitSums] = {0, 0, 0};
  for (int e = 0; e < g.B + g.NP; ++e)
    for (int i = 0; i < kUnitSums; ++i) units[i] += head_units(paged_entry(g, e), i) * g.Hkv;
  const bool light = both && paged_is_light(units[kUnitsLight], ctas);
  const int large = both && !light ? paged_large_ctas(units[kUnitsBeside], units[kUnitsLarge], ctas) : 0;
  for (int c = 0; c < 2; ++c) {
    const int which = c == 0 && light ? kUnitsLight : c == 0 ? kUnitsBeside : kUnitsLarge;
    if (c == 1 && light) break;
    const PagedShares shares(units[which], c ? large : kSmallWarps * (ctas - large), c ? 1 : kSmallMinUnits);
    PagedPlace at;
    at.slots = c ? static_cast<int>(w.rows_small) : 0;
    at.slot_rows = c ? kLargeRows : kSmallRows;
    at.home = static_cast<int>(w.rows_large_end);
    at.home_prefix = at.home + d.max_tokens * d.Hq;
    at.covered0 = g.NP > 0 ? g.prefix_first[0] : 0;
    at.covered1 = g.NP > 0 ? g.prefix_first[g.NP] : 0;
    at.B = g.B;
    at.G = g.G;
    at.Hq = g.Hq;
    long long before = 0;  // units of the entries before
    int e = 0;
    for (at.worker = 0; at.worker < shares.workers; ++at.worker) {
      long long u = shares.first(at.worker);
      const long long end = shares.first(at.worker + 1);
      while (u < end) {
        const PagedEntry entry = paged_entry(g, e);
        const long long hu = head_units(entry, which);
        if (u >= before + hu * g.Hkv) {
          before += hu * g.Hkv;
          ++e;
          continue;
        }
        PagedSegment s;
        PagedRecord rec;
        u += paged_take(cuts[c], shares, at, e, entry, hu, u - before, u, end - u, s, rec);
        if (s.nt == 0) continue;
        if (*n_rows < capacity) {
          int32_t* o = rows + *n_rows * 14;
          const int key1 = s.tile1 << cuts[c].key_shift;
          const int32_t v[14] = {c, at.worker, e, s.h, s.t0, s.nt, s.tile0 << cuts[c].key_shift, key1 < s.keys ? key1 : s.keys,
                                 s.mode, s.row, rec.count, rec.count ? rec.first : 0, rec.count ? rec.second : 0,
                                 rec.count ? rec.stride : 0};
          for (int i = 0; i < 14; ++i) o[i] = v[i];
        }
        ++*n_rows;
      }
    }
  }
  return capacity > 0 && *n_rows > capacity ? CP_ERR_WORKSPACE : CP_OK;
}

int cp_cache_append(const cp_paged_t* p, const cp_paged_cache_t* cache, const cp_paged_batch_t* batch, const void* q,
                    int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride, void* q_out,
                    int64_t q_out_stride, cudaStream_t stream) {
  if (!p || !cache || !batch) return CP_ERR_INVALID_ARG;
  const cp_paged_desc_t& d = p->desc;
  int rc = check_cache(d, *cache);
  if (rc == CP_OK) rc = check_batch(d, *batch);
  if (rc == CP_OK && (batch->n_seqs == 0 || batch->n_tokens == 0)) return CP_OK;
  if (rc == CP_OK) rc = check_tokens(k, k_stride, d.Hkv, d.d);
  if (rc == CP_OK) rc = check_tokens(v, v_stride, d.Hkv, d.d);
  if (rc == CP_OK && q) rc = check_tokens(q, q_stride, d.Hq, d.d);
  if (rc == CP_OK && q) rc = check_tokens(q_out, q_out_stride, d.Hq, d.d);
  if (rc == CP_OK && q && q == q_out && q_stride != q_out_stride) rc = CP_ERR_INVALID_ARG;
  if (rc == CP_OK) rc = check_arch();
  if (rc != CP_OK) return rc;
  cpattn::AppendArgs a;
  a.g = geom(*p, *cache, *batch);
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_out = q_out;
  a.k_cache = cache->k;
  a.v_cache = cache->v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out_stride = q_out_stride;
  a.rope_dim = d.rope_dim;
  a.interleaved = d.rope_interleaved;
  for (int j = 0; j < cpattn::kMaxRopePairs; ++j) a.turns[j] = p->turns[j];
  a.status = cpattn::device_status_ptr();
  if (!a.status) return CP_ERR_CUDA;
  NvtxRange range("cp_cache_append");
  return cpattn::launch_paged_append(a, stream);
}

int cp_attn_paged(const cp_paged_t* p, const cp_paged_cache_t* cache, const cp_paged_batch_t* batch, const void* q,
                  int64_t q_stride, void* o, float* lse, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!p || !cache || !batch) return CP_ERR_INVALID_ARG;
  const cp_paged_desc_t& d = p->desc;
  int rc = check_cache(d, *cache);
  if (rc == CP_OK) rc = check_batch(d, *batch);
  if (rc == CP_OK && (batch->n_seqs == 0 || batch->n_tokens == 0)) return CP_OK;
  if (rc == CP_OK && (!o || !lse)) rc = CP_ERR_INVALID_ARG;
  if (rc == CP_OK) rc = check_tokens(q, q_stride, d.Hq, d.d);
  if (rc == CP_OK && (!aligned(o, 16) || !aligned(lse, 16) || !aligned(workspace, 16))) rc = CP_ERR_ALIGNMENT;
  size_t need = 0;
  if (rc == CP_OK) rc = cp_paged_workspace_size(p, &need);
  if (rc == CP_OK && (!workspace || workspace_bytes < need)) rc = CP_ERR_WORKSPACE;
  if (rc == CP_OK) rc = check_arch();
  if (rc != CP_OK) return rc;
  cpattn::PagedAttnArgs a;
  a.g = geom(*p, *cache, *batch);
  a.q = q;
  a.q_stride = q_stride;
  a.k_cache = cache->k;
  a.v_cache = cache->v;
  a.o = o;
  a.out_fp32 = d.out_fp32;
  a.lse = lse;
  const cpattn::PagedWorkspace w = cpattn::paged_workspace(d.max_tokens, d.Hq, d.Hkv, d.d, d.max_prefixes > 0);
  char* ws = static_cast<char*>(workspace);
  a.parts = reinterpret_cast<cpattn::PagedParts*>(ws + w.parts);
  a.part_lse = reinterpret_cast<float*>(ws + w.lse);
  a.part_o = reinterpret_cast<float*>(ws + w.o);
  a.rows_small = w.rows_small;
  a.rows_large_end = w.rows_large_end;
  a.rows = static_cast<uint32_t>(w.rows);
  a.max_tokens = d.max_tokens;
  a.status = cpattn::device_status_ptr();
  if (!a.status) return CP_ERR_CUDA;
  NvtxRange range("cp_attn_paged");
  return cpattn::launch_paged_attn(a, stream);
}

}  // extern "C"
