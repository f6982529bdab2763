// verify.cu -- verification of drafted tokens against the target's
// probabilities from given random numbers: C ABI and kernel of
// cp_verify_drafts.
//
// Row i of a sequence's n new tokens holds the target's probabilities p_i of
// the token behind it; the draft x is the next row's token, drawn from q_i (or
// certain: q_i(x) = 1).  Drafts are accepted while u_i q_i(x) < p_i(x).  At the
// first one that is not, row a, the next token is drawn from max(p_a - q_a, 0);
// behind the last accepted one from p_a: the least k with w_0 + ... + w_k > r
// (w_0 + ... + w_V-1).  So the tokens are distributed as the target's own.
//
// Exactness.  Which k comes out hangs on sums over the whole vocabulary: with
// sums good to e, one in about 1 / (2 V e) draws lands beside a border and comes
// out differently: with fp32 sums (1e-7) of V = 10^5 numbers, one in 50.  So
// differences and sums are kept in pairs of fp32 numbers whose sum is the
// value (exact sum and difference of two floats: Knuth, Dekker), some 2^-46 of
// it off, and a warp's totals in fp64 from there on: one in 10^8.  fp64 for
// each element would be bound by the fp64 units (2 a clock and SM): two such
// operations of 128K elements of 64 rows take 30 us, the pairs' 11 of fp32 5.
//
// Bound by memory (each sequence's one row of p, and of q where it counts, is
// read once) and, for few sequences, by a chain of dependent loads: lengths,
// tokens, their probabilities, the row.  A cluster of up to 16 CTAs shares a
// row, each warp a stretch of it, so that one sequence uses 16 SMs; the warps' totals
// are exchanged through distributed shared memory; the CTA in whose stretch the
// border lies reads it again, from L2, and looks closer.
#include <cuda_runtime.h>

#define CP_TU_ID ::cpattn::kTuVerify
#include "host.h"
#include "paged.cuh"

namespace cpattn {
namespace {

constexpr int kVerifyThreads = 512, kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyMaxCluster = 16;

struct VerifyArgs {
  int B, N, V, max_new;
  const int32_t* q_start;
  const int32_t* kv_len;
  const void* p;
  const void* q;               // or null
  int64_t p_stride, q_stride;  // between rows, in elements
  const int32_t* tokens;
  const float* accept_u;
  const float* sample_u;
  int32_t* accepted;
  int32_t* out_tokens;
  int32_t* kv_out;             // or null
  int32_t* status;
};

// A weight: finite and above zero, else zero.
__device__ __forceinline__ float weight(float x) { return x > 0.f && x < INFINITY ? x : 0.f; }

// The sum hi + lo of many numbers, exactly but for the rounding of lo.
struct Pair {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x, float rest) {
    const float s = __fadd_rn(hi, x), b = __fadd_rn(s, -hi);
    const float e = __fadd_rn(__fadd_rn(hi, -__fadd_rn(s, -b)), __fadd_rn(x, -b));
    hi = s;
    lo = __fadd_rn(lo, __fadd_rn(e, rest));
  }
  __device__ __forceinline__ double value() const { return static_cast<double>(hi) + static_cast<double>(lo); }
};

template <typename T>
__device__ __forceinline__ float to_float(T x) {
  return static_cast<float>(x);
}

// The numbers of 16 bytes.
template <typename T>
struct Granule {
  static constexpr int kN = 16 / sizeof(T);
  float x[kN];
  __device__ __forceinline__ void from(const uint4& r) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        x[i] = __uint_as_float(w[i]);
      } else {
        const float2 u = Elem<T>::unpack(w[i]);
        x[2 * i] = u.x;
        x[2 * i + 1] = u.y;
      }
    }
  }
};

// A row of weights, in granules of 16 aligned bytes of p: granule g holds the
// elements g * kN - skew .. + kN - 1, as far as they are in [0, V).
template <typename T>
struct Row {
  static constexpr int kN = Granule<T>::kN;
  const T* p;
  const T* q;   // null: no second row
  int V, skew, granules;
  int x;        // with no second row: the rejected draft, which loses 1; else -1
  bool alike;   // q's granules are aligned where p's are

  __device__ __forceinline__ void set(const T* p_row, const T* q_row, int vocab, int draft) {
    p = p_row;
    q = q_row;
    V = vocab;
    x = draft;
    skew = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    alike = !q || ((reinterpret_cast<uintptr_t>(q) ^ reinterpret_cast<uintptr_t>(p)) & 15) == 0;
    granules = static_cast<int>((static_cast<long long>(V) + skew + kN - 1) / kN);
  }
  __device__ __forceinline__ void none() {
    p = q = nullptr;
    V = skew = granules = 0;
    x = -1;
    alike = true;
  }
  __device__ __forceinline__ int first(int g) const { return g * kN - skew; }
  __device__ __forceinline__ bool whole(int g) const { return alike && g > 0 && g < granules - 1; }
  __device__ __forceinline__ void load_whole(int g, uint4& a, uint4& b) const {
    a = *reinterpret_cast<const uint4*>(p + first(g));
    if (q) b = *reinterpret_cast<const uint4*>(q + first(g));
  }
  // The granule's numbers one by one: at the row's ends, and where p and q are
  // not aligned alike.
  __device__ __forceinline__ void load_edge(int g, Granule<T>& a, Granule<T>& b) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int e = first(g) + i;
      const bool in = e >= 0 && e < V;
      a.x[i] = in ? to_float(p[e]) : 0.f;
      b.x[i] = in && q ? to_float(q[e]) : 0.f;
    }
  }
  // Weight of element e, of which p and q are given: d + rest exactly.
  __device__ __forceinline__ void diff(int e, float of_p, float of_q, float& d, float& rest) const {
    const float u = weight(of_p), v = e == x ? 1.f : of_q > 0.f ? of_q : 0.f;
    d = __fadd_rn(u, -v);
    rest = __fadd_rn(__fadd_rn(u, -d), -v);  // exact where u >= v >= 0
    if (!(u > v)) d = rest = 0.f;
  }
  __device__ __forceinline__ void add(int g, const Granule<T>& a, const Granule<T>& b, Pair& sum) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      float d, rest;
      diff(first(g) + i, a.x[i], b.x[i], d, rest);
      sum.add(d, rest);
    }
  }
  __device__ __forceinline__ void weight_of(int e, float& d, float& rest) const {
    diff(e, to_float(p[e]), q ? to_float(q[e]) : 0.f, d, rest);
  }
};

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) v += __shfl_xor_sync(0xffffffffu, v, x);
  return v;
}

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
// The double at the address of `local` in the shared memory of CTA `rank`.
__device__ __forceinline__ double ld_cluster(const double* local, unsigned rank) {
  const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(local));
  uint32_t remote;
  double v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(remote) : "memory");
  return v;
}

// Totals of granules [g0, g1) of the row, lane by lane.
template <typename T>
__device__ __forceinline__ double sum_granules(const Row<T>& row, int g0, int g1) {
  constexpr int kAhead = 4;
  const int lane = threadIdx.x & 31;
  Pair sum;
  for (int g = g0 + lane; g < g1; g += 32 * kAhead) {
    uint4 a[kAhead], b[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      a[i] = b[i] = make_uint4(0, 0, 0, 0);
      if (g + 32 * i < g1 && row.whole(g + 32 * i)) row.load_whole(g + 32 * i, a[i], b[i]);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int at = g + 32 * i;
      if (at >= g1) break;
      Granule<T> u, v;
      u.from(a[i]);
      v.from(b[i]);
      if (!row.whole(at)) row.load_edge(at, u, v);
      row.add(at, u, v, sum);
    }
  }
  return sum.value();
}

// One cluster a sequence.
template <typename T>
__global__ void __launch_bounds__(kVerifyThreads, 2) verify_kernel(const __grid_constant__ VerifyArgs a, int cluster) {
  constexpr int kEach = kVerifyMaxCluster * kVerifyWarps / 32;
  __shared__ double totals[kVerifyWarps + 1];                 // this CTA's warps', read by the cluster; whether there is a residual
  __shared__ double sums[kVerifyMaxCluster * kVerifyWarps];   // all warps'
  __shared__ double close[kVerifyWarps];
  __shared__ double found_total, found_before;
  __shared__ int found_accepted, found_warp;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = static_cast<int>(cluster_rank()), s = blockIdx.x / cluster;
  pdl_wait();
  pdl_launch_dependents();
  const int t0 = a.q_start[s], t1 = a.q_start[s + 1], n = t1 - t0;
  // Every CTA goes through the same cluster barriers, whatever it finds in the arrays.
  const bool good = CP_CHECK_DATA(t0 >= 0 && t1 >= t0 && t1 <= a.N && n <= a.max_new, a.status);
  const T* p = static_cast<const T*>(a.p);
  const T* q = static_cast<const T*>(a.q);
  // Drafts accepted: 32 at a time, by every CTA's first warp.
  if (warp == 0) {
    int accepted = good ? max(n - 1, 0) : 0;
    for (int i0 = 0; good && i0 < n - 1; i0 += 32) {
      const int i = i0 + lane;
      bool ok = true;
      if (i < n - 1) {
        const int x = a.tokens[t0 + i + 1];
        ok = CP_CHECK_DATA(x >= 0 && x < a.V, a.status);
        if (ok) {
          const float px = weight(to_float(p[(t0 + i) * a.p_stride + x]));
          float qx = 1.f;
          if (q) qx = to_float(q[(t0 + i) * a.q_stride + x]);
          if (!(qx > 0.f)) qx = 0.f;
          // A product of two floats is exact in fp64.
          ok = static_cast<double>(a.accept_u[t0 + i]) * static_cast<double>(qx) < static_cast<double>(px);
        }
      }
      const unsigned no = __ballot_sync(0xffffffffu, !ok);
      if (no) {
        accepted = i0 + __ffs(no) - 1;
        break;
      }
    }
    if (lane == 0) found_accepted = accepted;
  }
  __syncthreads();
  const int accepted = found_accepted;
  const bool live = good && n > 0, rejected = live && accepted < n - 1;
  const int64_t t = static_cast<int64_t>(t0) + accepted;
  Row<T> row;
  row.none();
  if (live && CP_IN_BOUNDS(t < a.N, a.status))
    row.set(p + t * a.p_stride, rejected && q ? q + t * a.q_stride : nullptr, a.V, rejected && !q ? a.tokens[t + 1] : -1);
  const int warps = cluster * kVerifyWarps;
  int per = 0;
  for (int turn = 0; turn < 2; ++turn) {
    // A stretch of whole granules for each warp of the cluster, a multiple of 32 where there are enough.
    per = (row.granules + warps - 1) / warps;
    if (per > 32) per = (per + 31) & ~31;
    const int w = rank * kVerifyWarps + warp;
    const int g0 = min(w * per, row.granules), g1 = min(g0 + per, row.granules);
    const double v = warp_sum(sum_granules(row, g0, g1));
    if (lane == 0) totals[warp] = v;
    if (threadIdx.x == 0) totals[kVerifyWarps] = rejected ? 1 : 0;
    cluster_sync_all();
    if (static_cast<int>(threadIdx.x) < warps) sums[threadIdx.x] = ld_cluster(&totals[threadIdx.x % kVerifyWarps], threadIdx.x / kVerifyWarps);
    const bool again = turn == 0 && ld_cluster(&totals[kVerifyWarps], 0) != 0;
    cluster_sync_all();  // no CTA leaves, or writes its totals again, before all have read them
    if (warp == 0) {
      // Running sums of up to 256 numbers, eight to a lane; the first with any
      // weight of its own that ends above the border, or else (rounding) the last with any.
      double x[kEach], own = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        x[i] = lane * kEach + i < warps ? sums[lane * kEach + i] : 0.0;
        own += x[i];
      }
      double upto = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      double at = __shfl_up_sync(0xffffffffu, upto, 1);
      if (lane == 0) at = 0;
      const double total = __shfl_sync(0xffffffffu, upto, 31);
      const float r = live ? a.sample_u[s] : 0.f;
      const double border = total * static_cast<double>(r >= 0.f ? fminf(r, 0x1.fffffep-1f) : 0.f);
      int which = -1, any = -1;
      double which_before = 0, any_before = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const double end = at + x[i];
        if (x[i] > 0) {
          any = lane * kEach + i;
          any_before = at;
          if (which < 0 && end > border) which = any, which_before = at;
        }
        at = end;
      }
      const unsigned above = __ballot_sync(0xffffffffu, which >= 0), some = __ballot_sync(0xffffffffu, any >= 0);
      if (lane == 0) found_total = total, found_warp = -1;
      __syncwarp();
      if (above ? lane == __ffs(above) - 1 : some && lane == 31 - __clz(some)) {
        found_warp = above ? which : any;
        found_before = above ? which_before : any_before;
        found_total = total;
      }
    }
    __syncthreads();
    // Nothing left of p: no residual (the rows are not what they should be), so p itself.
    if (found_total > 0 || !again) break;
    if (live) row.set(row.p, nullptr, a.V, -1);
    __syncthreads();
  }
  if (!live) {
    if (good && rank == 0 && threadIdx.x == 0) {
      a.accepted[s] = 0;
      if (a.kv_out) a.kv_out[s] = a.kv_len[s];
    }
    return;
  }
  const int mine = found_warp;
  if (mine >= 0 && mine / kVerifyWarps == rank) {
    // This CTA's warps share that stretch, then one of them its lanes.
    const float r = a.sample_u[s];
    const double border = found_total * static_cast<double>(r >= 0.f ? fminf(r, 0x1.fffffep-1f) : 0.f);
    const int g0 = min(mine * per, row.granules), g1 = min(g0 + per, row.granules);
    const int part = (g1 - g0 + kVerifyWarps - 1) / kVerifyWarps;
    const int c0 = min(g0 + warp * part, g1), c1 = min(c0 + part, g1);
    const double v = warp_sum(sum_granules(row, c0, c1));
    if (lane == 0) close[warp] = v;
    __syncthreads();
    if (warp == 0) {
      // The part that holds the border; rounding apart, there is one.  Else the last with any weight.
      int k = -1;
      double before = 0, at = found_before;
      for (int i = 0; i < kVerifyWarps; ++i) {
        const double end = at + close[i];
        if (close[i] > 0) {
          k = i;
          before = at;
          if (end > border) break;
        }
        at = end;
      }
      if (k >= 0) {
        const int d0 = min(g0 + k * part, g1), d1 = min(d0 + part, g1);
        const int each = (d1 - d0 + 31) / 32;
        const int e0 = min(d0 + lane * each, d1), e1 = min(e0 + each, d1);
        Pair lane_sum;
        Granule<T> u, w;
        for (int g = e0; g < e1; ++g) {
          row.load_edge(g, u, w);
          row.add(g, u, w, lane_sum);
        }
        const double own = lane_sum.value();
        double upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double y = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += y;
        }
        const unsigned above = __ballot_sync(0xffffffffu, own > 0 && before + upto > border);
        const unsigned any = __ballot_sync(0xffffffffu, own > 0);
        if (any && lane == (above ? __ffs(above) - 1 : 31 - __clz(any))) {
          double sum = before + (upto - own);
          int token = -1;
          for (int e = max(row.first(e0), 0), end = min(row.first(e1), a.V); e < end; ++e) {
            float d, rest;
            row.weight_of(e, d, rest);
            if (!(d > 0.f)) continue;
            token = e;
            sum += static_cast<double>(d) + static_cast<double>(rest);
            if (sum > border) break;
          }
          a.out_tokens[t] = token;
        }
      }
    }
  } else if (mine < 0 && rank == 0 && threadIdx.x == 0) {
    a.out_tokens[t] = -1;
  }
  if (rank == 0 && warp == kVerifyWarps - 1) {
    for (int i = lane; i < n; i += 32)
      if (i != accepted) a.out_tokens[t0 + i] = i < accepted ? a.tokens[t0 + i + 1] : -1;
    if (lane == 0) {
      a.accepted[s] = accepted;
      if (a.kv_out) a.kv_out[s] = a.kv_len[s] - (n - 1 - accepted);
    }
  }
}

template <typename T>
int launch_verify(const VerifyArgs& a, cudaStream_t stream) {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CP_ERR_CUDA;
  if (!known[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(verify_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) return CP_ERR_CUDA;
    known[dev].store(1, std::memory_order_release);
  }
  // As many CTAs a sequence as fill the card twice, none with less than 512 granules of 16 bytes.
  int cluster = 1;
  while (cluster < kVerifyMaxCluster && a.B * cluster < 2 * 152 && a.V / cluster > 1024) cluster *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * cluster);
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_kernel<T>, a, cluster) == cudaSuccess ? CP_OK : CP_ERR_CUDA;
}

}  // namespace
}  // namespace cpattn

using namespace cpattn;

extern "C" {

int cp_verify_drafts(const cp_paged_t* plan, const cp_paged_batch_t* batch, const cp_verify_t* verify, cudaStream_t stream) {
  if (!plan || !batch || !verify) return CP_ERR_INVALID_ARG;
  const cp_verify_t& v = *verify;
  const int max_new = paged_max_new(plan, *batch);
  if (max_new < 0) return max_new;
  if (v.dtype < CP_DTYPE_BF16 || v.dtype > CP_DTYPE_FP32) return CP_ERR_INVALID_ARG;
  if (v.vocab <= 0 || v.vocab > 1 << 30 || v.p_stride < v.vocab || v.p_stride >= kMaxStride) return CP_ERR_INVALID_ARG;
  if (v.q && (v.q_stride < v.vocab || v.q_stride >= kMaxStride)) return CP_ERR_INVALID_ARG;
  if (batch->n_seqs == 0) return CP_OK;
  if (!batch->q_start || !batch->kv_len || !v.accepted) return CP_ERR_INVALID_ARG;
  // Without rows every sequence has none, which its outputs say.
  if (batch->n_tokens > 0 && (!v.p || !v.tokens || !v.accept_u || !v.sample_u || !v.out_tokens)) return CP_ERR_INVALID_ARG;
  if (!aligned(v.p, 16) || !aligned(v.q, 16)) return CP_ERR_ALIGNMENT;
  const void* arrays[] = {v.tokens, v.accept_u, v.sample_u, v.accepted, v.out_tokens, v.kv_len_out};
  for (const void* x : arrays)
    if (!aligned(x, 4)) return CP_ERR_ALIGNMENT;
  const int rc = check_arch();
  if (rc != CP_OK) return rc;
  VerifyArgs a = {};
  a.B = batch->n_seqs;
  a.N = batch->n_tokens;
  a.V = v.vocab;
  a.max_new = max_new;
  a.q_start = batch->q_start;
  a.kv_len = batch->kv_len;
  a.p = v.p;
  a.q = v.q;
  a.p_stride = v.p_stride;
  a.q_stride = v.q_stride;
  a.tokens = v.tokens;
  a.accept_u = v.accept_u;
  a.sample_u = v.sample_u;
  a.accepted = v.accepted;
  a.out_tokens = v.out_tokens;
  a.kv_out = v.kv_len_out;
  a.status = device_status_ptr();
  if (!a.status) return CP_ERR_CUDA;
  NvtxRange range("cp_verify_drafts");
  return v.dtype == CP_DTYPE_FP32   ? launch_verify<float>(a, stream)
         : v.dtype == CP_DTYPE_BF16 ? launch_verify<__nv_bfloat16>(a, stream)
                                    : launch_verify<__half>(a, stream);
}

}  // extern "C"
