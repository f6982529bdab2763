// paged_attn.cu -- attention of a batch's new tokens over the paged
// key/value cache, shared prefixes included.
//
// For one token row and query head, over the keys that it sees (its
// sequence's own, up to the causal limit, and its prefix's):
//   m = max_k s_k,  l = sum_k e^(s_k - m),  O = sum_k e^(s_k - m) v_k / l,
//   LSE = m + ln l,   s_k = scale * q . k_k,
// in one pass over the keys with running m and l.  The keys are cut into
// equal shares for the whole card (PagedCut); a row whose keys fall to several
// workers, or that has a prefix, is joined by its parts' log-sum-exp.
//
//   paged_small_kernel   batches whose entries have few rows (tokens x query
//                        heads of a KV head): bound by reading the cache (the
//                        work is in paged_small.cuh).
//   paged_large_kernel   batches that have larger ones too (paged_attn_large.cu).
//   paged_merge_kernel   joins the parts.
#include <cuda.h>
#include <cuda_runtime.h>

#include <type_traits>

#define CP_TU_ID ::cpattn::kTuPagedAttn
#include "paged.cuh"
#include "paged_small.cuh"

namespace cpattn {
namespace {

// ---------------------------------------------------------------- few rows
template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(kSmallWarps * 32, 1)
    paged_small_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ PagedAttnArgs args) {
  using SM = SmallSmem<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    small_init<D>(smem, warp);
  }
  __syncwarp();
  pdl_wait();
  pdl_launch_dependents();
  if (smem_u32(smem) & 1023) {  // the swizzle is a function of the address
    debug_bounds_fail(args.status, __LINE__, CP_TU_ID);
    return;
  }
  const PagedCut cuts[1] = {paged_cut_small(args.g.G, ROWS)};
  PagedWalker<1> walk(args, cuts);
  // Workers of different SMs first, so that a short batch has the whole card.
  const auto role = [&](const long long (&)[1]) {
    return PagedRole{0, 0, warp * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x), kSmallWarps * static_cast<int>(gridDim.x),
                     kSmallMinUnits, 0, kSmallRows};
  };
  if (walk.start(reinterpret_cast<long long*>(smem + SM::offSums), kSmallWarps, role))
    small_worker<SmallRows<T, D, ROWS>, D>(smem, warp, tm_k, tm_v, walk);
}

// ---------------------------------------------------------------- merge
//
// O = sum_p 2^(lse_p - m) O_p / sum_p 2^(lse_p - m) over a row's parts, its own
// keys' first, then its prefix's, in key order; rows whose only part went
// straight to the output are left alone.  What it reads is small and in L2, so
// its time is latency: eight loads of 16 bytes a lane are in flight, or ten.
//   kMergeBlock  a block per (token, query head), its warps share the parts:
//                few rows, many parts (a decode of one sequence 9.7 us without,
//                8.0 with; 20 sequences on a prefix of 30K keys, 640 rows, 39.8
//                and 37.0).  Ten parts a warp at a time: 7 sequences on a
//                prefix 13.7 us, 14.4 with eight, 13.9 with sixteen.
//   kMergeHead   a warp per (token, query head), eight parts at a time (24
//                drafts of 5 tokens 27.3 us without, 21.0 with; 64 sequences on
//                a prefix 64.8 and 60.5).
//   kMergeGroup  a warp per (token, KV head), four heads x two parts at a time:
//                a batch whose rows would be several waves of warps (256
//                sequences on prefixes 105.8 us without, 99.1 with).
//   kMergeToken  a warp per token, four heads x two parts at a time: prompts,
//                whose rows have one part (and are left) or two (chunks of 2K
//                tokens 412 us without, 392 with).  A decode batch that large
//                joins every row, one KV head after another: on a prefix of 2000
//                keys 1024 sequences of 8 KV heads take 94.0 us (kMergeGroup),
//                1025 98.1; 256 of 32 heads of one query head each 56.6, 257
//                86.7; 64 of 128 heads on 500 keys 50.2, 65 134.
enum MergeBy { kMergeBlock, kMergeHead, kMergeGroup, kMergeToken };
constexpr int kMergeWarps = 4;
constexpr int kMergeBlocks = 152 * 12;  // at most; they loop
constexpr long long kMergeBlockRows = 1216;                        // (token, query head)s up to which BY is kMergeBlock,
constexpr long long kMergeHeadGroups = 1216, kMergeGroups = 8192;  // (token, KV head)s: kMergeHead, kMergeGroup

// Join the parts `a` (own keys) and `b` (prefix) of token t's query heads
// h0 .. h1 - 1 of KV head hk.  `joint`: kMergeBlock's warps' sums.
template <typename T, int D, MergeBy BY>
__device__ __forceinline__ void join_parts(const PagedAttnArgs& args, const PagedParts& a, const PagedParts& b, int t, int hk,
                                           int h0, int h1, float (*joint)[32][D / 32 + 2]) {
  constexpr int E = D / 32, HB = BY >= kMergeGroup ? 4 : 1, PB = BY == kMergeBlock ? 10 : 8 / HB;  // heads and parts at a time
  constexpr int step = BY == kMergeBlock ? kMergeWarps : 1;               // between a warp's parts
  using Vec = typename std::conditional<E == 4, float4, float2>::type;
  const PagedGeom& g = args.g;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = a.count + b.count;
  for (int sub = h0; sub < h1; sub += HB) {
    float m[HB], sum[HB], o[HB][E];
#pragma unroll
    for (int h = 0; h < HB; ++h) {
      m[h] = -INFINITY;
      sum[h] = 0.f;
#pragma unroll
      for (int j = 0; j < E; ++j) o[h][j] = 0.f;
    }
    for (int i0 = BY == kMergeBlock ? warp : 0; i0 < n; i0 += PB * step) {
      float lse[PB][HB];
      Vec v[PB][HB];
#pragma unroll
      for (int k = 0; k < PB; ++k) {
        const int i = i0 + k * step;
        const bool in_a = i < a.count;
        const int at = in_a ? i : i - a.count;
        const int first = in_a ? a.first : b.first, second = in_a ? a.second : b.second, next = in_a ? a.stride : b.stride;
        const long long row = (at == 0 ? first : second + (at - 1) * next) + sub;
#pragma unroll
        for (int h = 0; h < HB; ++h) {
          lse[k][h] = -INFINITY;
          if (i < n && sub + h < h1 && CP_IN_BOUNDS(part_rows_in(args, row + h, 1), args.status)) {
            lse[k][h] = args.part_lse[row + h];
            v[k][h] = *reinterpret_cast<const Vec*>(args.part_o + (row + h) * D + lane * E);
          }
        }
      }
#pragma unroll
      for (int h = 0; h < HB; ++h) {
        float top = m[h];
#pragma unroll
        for (int k = 0; k < PB; ++k) top = fmaxf(top, lse[k][h]);
        const float z = top == -INFINITY ? 0.f : top, f = ex2_approx(m[h] - z);
        m[h] = top;
        sum[h] *= f;
#pragma unroll
        for (int j = 0; j < E; ++j) o[h][j] *= f;
#pragma unroll
        for (int k = 0; k < PB; ++k) {
          if (lse[k][h] == -INFINITY) continue;
          const float wt = ex2_approx(lse[k][h] - z);
          sum[h] += wt;
          const float* y = reinterpret_cast<const float*>(&v[k][h]);
#pragma unroll
          for (int j = 0; j < E; ++j) o[h][j] = fmaf(wt, y[j], o[h][j]);
        }
      }
    }
    if constexpr (BY == kMergeBlock) {
      __syncthreads();  // the last item's are read
#pragma unroll
      for (int j = 0; j < E; ++j) joint[warp][lane][j] = o[0][j];
      joint[warp][lane][E] = m[0];
      joint[warp][lane][E + 1] = sum[0];
      __syncthreads();
      if (warp > 0) return;
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < kMergeWarps; ++k) top = fmaxf(top, joint[k][lane][E]);
      const float z = top == -INFINITY ? 0.f : top;
      m[0] = top;
      sum[0] = 0.f;
#pragma unroll
      for (int j = 0; j < E; ++j) o[0][j] = 0.f;
#pragma unroll
      for (int k = 0; k < kMergeWarps; ++k) {
        const float f = ex2_approx(joint[k][lane][E] - z);
        sum[0] = fmaf(f, joint[k][lane][E + 1], sum[0]);
#pragma unroll
        for (int j = 0; j < E; ++j) o[0][j] = fmaf(f, joint[k][lane][j], o[0][j]);
      }
    }
#pragma unroll
    for (int h = 0; h < HB; ++h) {
      if (sub + h >= h1) continue;
      const float inv = sum[h] != 0.f ? __fdividef(1.f, sum[h]) : 0.f;
      const int head = hk * g.G + sub + h;
      if (!CP_IN_BOUNDS(token_in(g, t, head), args.status)) continue;
      const long long at = (static_cast<long long>(t) * g.Hq + head) * D + lane * E;
      if (args.out_fp32) {
        float* dst = static_cast<float*>(args.o) + at;
#pragma unroll
        for (int j = 0; j < E; ++j) dst[j] = o[h][j] * inv;
      } else {
        uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<T*>(args.o) + at);
#pragma unroll
        for (int j = 0; j < E / 2; ++j) dst[j] = Elem<T>::pack(o[h][2 * j] * inv, o[h][2 * j + 1] * inv);
      }
      if (lane == 0)
        args.lse[static_cast<long long>(head) * g.N + t] = sum[h] != 0.f ? (m[h] + lg2_approx(sum[h])) * 0.69314718055994531f : -INFINITY;
    }
  }
}

template <typename T, int D, MergeBy BY>
__global__ void __launch_bounds__(kMergeWarps * 32) paged_merge_kernel(const __grid_constant__ PagedAttnArgs args) {
  __shared__ float joint[BY == kMergeBlock ? kMergeWarps : 1][32][D / 32 + 2];
  pdl_launch_dependents();
  const PagedGeom& g = args.g;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per_token = BY == kMergeToken ? 1 : BY == kMergeGroup ? g.Hkv : g.Hq;
  const long long items = static_cast<long long>(g.N) * per_token;
  const long long stride = static_cast<long long>(gridDim.x) * (BY == kMergeBlock ? 1 : kMergeWarps);
  const int covered0 = g.NP > 0 ? g.prefix_first[0] : 0, covered1 = g.NP > 0 ? g.prefix_first[g.NP] : 0;  // as PagedWalker has it
  bool waited = false;
  for (long long w = BY == kMergeBlock ? blockIdx.x : static_cast<long long>(blockIdx.x) * kMergeWarps + warp; w < items; w += stride) {
    const int t = static_cast<int>(w / per_token);
    const int s = warp_count_le(g.q_start + 1, g.B, t);
    if (s >= g.B) break;  // this token and those after it belong to no sequence
    const PagedEntry own = paged_entry(g, s);
    if (own.bad || t < own.t0 || t >= own.t0 + own.n) continue;
    const bool covered = s >= covered0 && s < covered1;
    const int p = covered ? warp_prefix_of(g, s) : -1;
    const PagedEntry pre = p >= 0 ? paged_entry(g, g.B + p) : PagedEntry{0, 0, 0, 0, nullptr, false};
    const bool prefix = pre.keys > 0 && t >= pre.t0 && t < pre.t0 + pre.n;
    const bool sees_own = min(own.keys, own.limit0 + (t - own.t0)) > 0;
    const PagedParts* own_parts = args.parts + static_cast<size_t>(t) * g.Hkv;
    const PagedParts* prefix_parts = own_parts + static_cast<size_t>(args.max_tokens) * g.Hkv;
    if (!waited) pdl_wait();
    waited = true;
    if constexpr (BY != kMergeToken) {
      const int x = static_cast<int>(w - static_cast<long long>(t) * per_token);
      const int hk = BY == kMergeGroup ? x : x / g.G, h = BY == kMergeGroup ? 0 : x - hk * g.G;
      PagedParts a{0, 0, 0, 0}, b{0, 0, 0, 0};
      if (sees_own) a = own_parts[hk];
      if (prefix) b = prefix_parts[hk];
      if ((a.count != 1 || covered) &&
          CP_CHECK_DATA(paged_parts_in(a, g.G, args.rows) && paged_parts_in(b, g.G, args.rows), args.status))
        join_parts<T, D, BY>(args, a, b, t, hk, h, BY == kMergeGroup ? g.G : h + 1, joint);
    } else {
      // A lane looks up one of 32 KV heads; the warp goes through those that
      // have parts to join.
      for (int h0 = 0; h0 < g.Hkv; h0 += 32) {
        PagedParts a{0, 0, 0, 0}, b{0, 0, 0, 0};
        const bool there = h0 + lane < g.Hkv;
        if (there && sees_own) a = own_parts[h0 + lane];
        if (there && prefix) b = prefix_parts[h0 + lane];
        const bool joins = there && (a.count != 1 || covered) &&
                           CP_CHECK_DATA(paged_parts_in(a, g.G, args.rows) && paged_parts_in(b, g.G, args.rows), args.status);
        for (unsigned todo = __ballot_sync(0xffffffffu, joins); todo; todo &= todo - 1) {
          const int from = __ffs(todo) - 1;
          auto of = [&](const PagedParts& x) {
            return PagedParts{__shfl_sync(0xffffffffu, x.first, from), __shfl_sync(0xffffffffu, x.second, from),
                              __shfl_sync(0xffffffffu, x.count, from), __shfl_sync(0xffffffffu, x.stride, from)};
          };
          join_parts<T, D, BY>(args, of(a), of(b), t, h0 + from, 0, g.G, joint);
        }
      }
    }
  }
  if (!waited) pdl_wait();  // whoever waits for this kernel waits for those before it too
}

// ---------------------------------------------------------------- launch

template <typename T, int D, int ROWS>
int launch_small(const PagedAttnArgs& a, cudaStream_t stream) {
  static std::atomic<int> known[64];
  int sms = 0;
  const int rc = prepare_kernel(known, paged_small_kernel<T, D, ROWS>, SmallSmem<D>::kBytes, &sms);
  if (rc != CP_OK) return rc;
  CUtensorMap mk, mv;
  if (!make_cache_map_whole(&mk, a.g, a.k_cache, 16) || !make_cache_map_whole(&mv, a.g, a.v_cache, 16)) return CP_ERR_CUDA;
  const int ctas = sms < kSmallWorkers / kSmallWarps ? sms : kSmallWorkers / kSmallWarps;
  return launch(paged_small_kernel<T, D, ROWS>, ctas, kSmallWarps * 32, SmallSmem<D>::kBytes, stream, mk, mv, a);
}

template <typename T, int D>
int launch_attn_d(const PagedAttnArgs& a, cudaStream_t stream) {
  const PagedGeom& g = a.g;
  const long long most = paged_most_rows(g);
  int rc;
  if (paged_has_large(most, D))
    rc = launch_paged_large(a, stream);
  else if (paged_small_rows(most) == 8)
    rc = launch_small<T, D, 8>(a, stream);
  else if (paged_small_rows(most) == 16)
    rc = launch_small<T, D, 16>(a, stream);
  else if constexpr (D == 64)
    rc = launch_small<T, D, kSmallRows>(a, stream);
  else
    rc = CP_ERR_UNSUPPORTED;  // paged_has_large
  if (rc != CP_OK) return rc;
  const long long rows = static_cast<long long>(g.N) * g.Hq;
  const auto blocks = [](long long n) { return static_cast<unsigned>(n < kMergeBlocks ? n : kMergeBlocks); };
  if (rows <= kMergeBlockRows)
    return launch(paged_merge_kernel<T, D, kMergeBlock>, blocks(rows), kMergeWarps * 32, 0, stream, a);
  const long long groups = static_cast<long long>(g.N) * g.Hkv;
  if (groups <= kMergeHeadGroups)
    return launch(paged_merge_kernel<T, D, kMergeHead>, blocks((rows + kMergeWarps - 1) / kMergeWarps), kMergeWarps * 32, 0, stream, a);
  if (groups <= kMergeGroups)
    return launch(paged_merge_kernel<T, D, kMergeGroup>, blocks((groups + kMergeWarps - 1) / kMergeWarps), kMergeWarps * 32, 0, stream, a);
  return launch(paged_merge_kernel<T, D, kMergeToken>, blocks((static_cast<long long>(g.N) + kMergeWarps - 1) / kMergeWarps),
                kMergeWarps * 32, 0, stream, a);
}

}  // namespace

int launch_paged_attn(const PagedAttnArgs& a, cudaStream_t stream) {
  const bool bf16 = a.g.dtype == CP_DTYPE_BF16;
  if (a.g.d == 128) return bf16 ? launch_attn_d<__nv_bfloat16, 128>(a, stream) : launch_attn_d<__half, 128>(a, stream);
  if (a.g.d == 64) return bf16 ? launch_attn_d<__nv_bfloat16, 64>(a, stream) : launch_attn_d<__half, 64>(a, stream);
  return CP_ERR_UNSUPPORTED;
}

}  // namespace cpattn
