// rope.cu -- rotary positions of whole sequences, with one position or
// several (time, height, width) a token: C ABI and kernel of cp_rope.
//
// Pair j of a head turns by theta = pos[axis(j)][t] * f_j: (a, b) ->
// (a cos - b sin, b cos + a sin); the gradient of that is the turn by -theta.
// Angles are paged_append.cu's: 64-bit fractions of a circle, good at every
// position.  The rotation is in fp32 with one rounding at the end.
//
// Bound by memory: each value is read once and written once.  As in the
// append a warp owns a token (or a share of its heads), a lane two pieces of 16 bytes of
// a head that hold both halves of eight pairs (four in fp32), so that its
// sines and cosines serve every head it visits, queries and keys alike.  The
// warp's lanes compute a pair each, while the first pieces are on their way, and hand them on
// through shared memory.  64K tokens of 32 + 8 heads of 128 in bf16 (1.34 GB) take
// 196 us, 1.02 of the copy's rate; 20000 of 16 + 4 heads 0.76 to 0.96 of it in
// 16 bits (d = 64 to 256), 0.96 to 0.99 in fp32, 0.85 to 1.0 from fp32 to 16 bits.  With few heads (13805 tokens of 2)
// the angles count: 12 us for 28 MB.
#include <cuda_runtime.h>

#include <cmath>
#include <new>

#define CP_TU_ID ::cpattn::kTuRope
#include "host.h"
#include "paged.cuh"

struct cp_rope_plan {
  cp_rope_desc_t desc;
  uint64_t turns[128];
  uint8_t axis[128];
};

namespace cpattn {
namespace {

constexpr int kRopeMaxDim = 256;
constexpr int kRopeWarps = 2;
constexpr int kRopeFillWarps = 152 * 32;  // warps that keep the memory busy

struct RopeJob {
  const void* in;
  void* out;
  int64_t in_stride, out_stride;
  int first;  // its first head among those of all jobs
};

struct RopeArgs {
  int n, d, rope_dim, interleaved, inverse, heads, jobs, axes;
  const int32_t* positions;  // [axes][n]
  RopeJob job[CP_ROPE_MAX_JOBS];
  uint64_t turns[kRopeMaxDim / 2];
  uint8_t axis[kRopeMaxDim / 2];
  int32_t* status;
};

// N elements as they lie in memory, 8 or 16 bytes at a time.
template <typename T, int N>
struct Piece {
  static constexpr int kBytes = N * static_cast<int>(sizeof(T));
  using Vector = typename std::conditional<kBytes % 16 == 0, uint4, uint2>::type;
  static constexpr int kVectors = kBytes / static_cast<int>(sizeof(Vector));
  Vector r[kVectors];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kVectors; ++i) r[i] = reinterpret_cast<const Vector*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < kVectors; ++i) reinterpret_cast<Vector*>(p)[i] = r[i];
  }
  __device__ __forceinline__ void get(float (&x)[N]) const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(r);
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const float2 u = Elem<T>::unpack(w[i]);
        x[2 * i] = u.x;
        x[2 * i + 1] = u.y;
      }
    }
  }
  __device__ __forceinline__ void set(const float (&x)[N]) {
    uint32_t* w = reinterpret_cast<uint32_t*>(r);
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = __float_as_uint(x[i]);
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) w[i] = Elem<T>::pack(x[2 * i], x[2 * i + 1]);
    }
  }
};

// Elements of a lane's piece of a head: 16 bytes.
template <typename TI>
constexpr __host__ __device__ int rope_piece() {
  return 16 / static_cast<int>(sizeof(TI));
}

// Parameters that each lane wants another of, by the way of global memory: the
// constant bank gives one address at a time (13805 tokens of 2 heads of 256
// elements took 28 us, 4 of them for the memory).
__device__ __forceinline__ uint64_t param_u64(const uint64_t* p) {
  uint64_t v;
  asm("ld.b64 %0, [%1];" : "=l"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t param_u8(const uint8_t* p) {
  uint32_t v;
  asm("ld.u8 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

template <typename TI, typename TO>
__global__ void __launch_bounds__(kRopeWarps * 32) rope_kernel(const __grid_constant__ RopeArgs args, unsigned units) {
  constexpr int N = rope_piece<TI>();
  // Groups of heads whose loads are in flight together: more pay only where the
  // pieces stored are half as large (20000 tokens of 20 heads of 192, fp32 to bf16, 85 us
  // with 2, 73 with 3 or 4; fp32 throughout 94 and, with 3, 109; bf16 53 and 57).
  constexpr int kAhead = sizeof(TI) > sizeof(TO) ? 4 : 2;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const unsigned w = blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
  const unsigned t = w / units, unit = w - t * units;
  if (t >= static_cast<unsigned>(args.n)) return;
  const int lph = args.d / (2 * N), hpg = 32 / lph;  // lanes per head, heads per group
  const int sub = lane / lph, j = lane - sub * lph;
  const bool rotated = j < args.rope_dim / (2 * N), halves = rotated && !args.interleaved;
  const int ea = halves ? N * j : 2 * N * j;  // first elements of the lane's two pieces
  const int eb = halves ? args.rope_dim / 2 + N * j : 2 * N * j + N;
  Piece<TI, N> a[kAhead], b[kAhead];
  TO* dst[kAhead];
  // The pieces of group g.
  const auto load = [&](int i, int g) {
    const int h = g * hpg + sub;
    dst[i] = nullptr;
    if (sub >= hpg || h >= args.heads || !CP_IN_BOUNDS(ea + N <= args.d && eb + N <= args.d, args.status)) return;
    int k = 0;
#pragma unroll
    for (int x = 1; x < CP_ROPE_MAX_JOBS; ++x) k += x < args.jobs && h >= args.job[x].first;
    const RopeJob& job = args.job[k];
    const int64_t at = static_cast<int64_t>(h - job.first) * args.d;
    const TI* src = static_cast<const TI*>(job.in) + t * job.in_stride + at;
    dst[i] = static_cast<TO*>(job.out) + t * job.out_stride + at;
    a[i].load(src + ea);
    b[i].load(src + eb);
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(i, unit + i * units);  // on their way while the angles are computed
  __shared__ __align__(16) float2 turned[kRopeWarps][kRopeMaxDim / 2];  // cosine, sine
  float2* mine = turned[threadIdx.x >> 5];
  const int of_lane = lane < args.axes ? args.positions[static_cast<size_t>(lane) * args.n + t] : 0;
#pragma unroll 1
  for (int i = 0; i < args.rope_dim / 2; i += 32) {
    const int pair = min(i + lane, args.rope_dim / 2 - 1);
    float c, sn;
    sincos_turns(__shfl_sync(0xffffffffu, of_lane, static_cast<int>(param_u8(args.axis + pair))), param_u64(args.turns + pair), &sn, &c);
    mine[pair] = make_float2(c, args.inverse ? -sn : sn);  // the last one's lanes agree
  }
  __syncwarp();
  float c[N], sn[N];
  if (rotated) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float4 v = reinterpret_cast<const float4*>(mine + N * j)[i];
      c[2 * i] = v.x;
      sn[2 * i] = v.y;
      c[2 * i + 1] = v.z;
      sn[2 * i + 1] = v.w;
    }
  }
  const auto turn = [&](int i) {
    float x[N], y[N];
    a[i].get(x);
    b[i].get(y);
    if (halves) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float u = x[e], v = y[e];
        x[e] = u * c[e] - v * sn[e];
        y[e] = v * c[e] + u * sn[e];
      }
    } else if (rotated) {
#pragma unroll
      for (int e = 0; e < N / 2; ++e) {
        const float u = x[2 * e], v = x[2 * e + 1], p = y[2 * e], q = y[2 * e + 1];
        x[2 * e] = u * c[e] - v * sn[e];
        x[2 * e + 1] = v * c[e] + u * sn[e];
        y[2 * e] = p * c[N / 2 + e] - q * sn[N / 2 + e];
        y[2 * e + 1] = q * c[N / 2 + e] + p * sn[N / 2 + e];
      }
    }
    Piece<TO, N> o;
    o.set(x);
    o.store(dst[i] + ea);
    o.set(y);
    o.store(dst[i] + eb);
  };
  const int groups = (args.heads + hpg - 1) / hpg;
  // As soon as a group is stored another is asked for.
  for (int g0 = unit; g0 < groups; g0 += kAhead * static_cast<int>(units)) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (dst[i]) turn(i);
      load(i, g0 + (kAhead + i) * static_cast<int>(units));
    }
  }
}

template <typename TI, typename TO>
int launch_rope(const RopeArgs& a, cudaStream_t stream) {
  const int hpg = 32 / (a.d / (2 * rope_piece<TI>())), groups = (a.heads + hpg - 1) / hpg;
  // Few tokens: a warp for each group of heads, for latency.  Many: a warp
  // takes more of its token's heads, as one set of sines serves them all.
  const long long fill = (static_cast<long long>(a.n) + kRopeFillWarps - 1) / a.n;  // n itself may be 2^31 - 1
  const int units = static_cast<int>(fill > groups ? groups : fill);
  const long long warps = static_cast<long long>(a.n) * units;  // below 2^31 + kRopeFillWarps + n
  const long long grid = (warps + kRopeWarps - 1) / kRopeWarps;
  return launch(rope_kernel<TI, TO>, static_cast<unsigned>(grid), kRopeWarps * 32, 0, stream, a, static_cast<unsigned>(units));
}

template <typename TI>
int launch_rope_from(const RopeArgs& a, int out_dtype, cudaStream_t stream) {
  if (out_dtype == CP_DTYPE_FP32) return launch_rope<TI, float>(a, stream);
  if constexpr (std::is_same<TI, float>::value) {
    return out_dtype == CP_DTYPE_BF16 ? launch_rope<TI, __nv_bfloat16>(a, stream) : launch_rope<TI, __half>(a, stream);
  } else {
    return launch_rope<TI, TI>(a, stream);
  }
}

}  // namespace
}  // namespace cpattn

using namespace cpattn;

extern "C" {

int cp_rope_create(const cp_rope_desc_t* desc, cp_rope_t** out) {
  if (!desc || !out || desc->version != CP_ROPE_VERSION) return CP_ERR_INVALID_ARG;
  const cp_rope_desc_t& d = *desc;
  if (d.d <= 0 || d.rope_dim <= 0 || d.rope_dim > d.d || (d.rope_interleaved | 1) != 1) return CP_ERR_INVALID_ARG;
  if (d.d % 16 || d.d > kRopeMaxDim || d.rope_dim % 16) return CP_ERR_UNSUPPORTED;
  cp_rope_plan* r = new (std::nothrow) cp_rope_plan();
  if (!r) return CP_ERR_CUDA;
  const int rc = rope_pairs(d.rope_dim, d.rope_base, d.rope_freqs, d.rope_axes, d.rope_axis, r->turns, r->axis);
  if (rc != CP_OK) {
    delete r;
    return rc;
  }
  r->desc = d;
  r->desc.rope_freqs = nullptr;
  r->desc.rope_axis = nullptr;
  *out = r;
  return CP_OK;
}

void cp_rope_destroy(cp_rope_t* r) { delete r; }

int cp_rope(const cp_rope_t* r, int32_t n_tokens, const int32_t* positions, int32_t n_jobs, const cp_rope_job_t* jobs, int32_t in_dtype,
            int32_t out_dtype, int32_t inverse, cudaStream_t stream) {
  if (!r || n_tokens < 0 || n_jobs < 1 || n_jobs > CP_ROPE_MAX_JOBS || !jobs || (inverse | 1) != 1) return CP_ERR_INVALID_ARG;
  if (in_dtype < CP_DTYPE_BF16 || in_dtype > CP_DTYPE_FP32 || out_dtype < CP_DTYPE_BF16 || out_dtype > CP_DTYPE_FP32)
    return CP_ERR_INVALID_ARG;
  if (in_dtype != out_dtype && in_dtype != CP_DTYPE_FP32 && out_dtype != CP_DTYPE_FP32) return CP_ERR_UNSUPPORTED;
  const cp_rope_desc_t& d = r->desc;
  const int64_t in_unit = in_dtype == CP_DTYPE_FP32 ? 4 : 8, out_unit = out_dtype == CP_DTYPE_FP32 ? 4 : 8;  // of 16 bytes
  RopeArgs a = {};
  for (int i = 0; i < n_jobs; ++i) {
    const cp_rope_job_t& j = jobs[i];
    if (j.heads <= 0 || j.heads > 65536) return CP_ERR_INVALID_ARG;
    const int64_t row = static_cast<int64_t>(j.heads) * d.d;
    if (j.in_stride < row || j.in_stride >= kMaxStride || j.in_stride % in_unit || j.out_stride < row || j.out_stride >= kMaxStride ||
        j.out_stride % out_unit)
      return CP_ERR_INVALID_ARG;
    if (n_tokens > 0 && (!j.in || !j.out)) return CP_ERR_INVALID_ARG;
    if (!aligned(j.in, 16) || !aligned(j.out, 16)) return CP_ERR_ALIGNMENT;
    if (j.in && j.in == j.out && (j.in_stride != j.out_stride || in_dtype != out_dtype)) return CP_ERR_INVALID_ARG;
    a.job[i] = RopeJob{j.in, j.out, j.in_stride, j.out_stride, a.heads};
    a.heads += j.heads;
  }
  if (n_tokens == 0) return CP_OK;
  if (!positions) return CP_ERR_INVALID_ARG;
  if (!aligned(positions, 4)) return CP_ERR_ALIGNMENT;
  const int rc = check_arch();
  if (rc != CP_OK) return rc;
  a.n = n_tokens;
  a.d = d.d;
  a.rope_dim = d.rope_dim;
  a.interleaved = d.rope_interleaved;
  a.inverse = inverse;
  a.jobs = n_jobs;
  a.axes = d.rope_axes;
  a.positions = positions;
  for (int j = 0; j < d.rope_dim / 2; ++j) a.turns[j] = r->turns[j], a.axis[j] = r->axis[j];
  a.status = device_status_ptr();
  if (!a.status) return CP_ERR_CUDA;
  NvtxRange range("cp_rope");
  return in_dtype == CP_DTYPE_FP32   ? launch_rope_from<float>(a, out_dtype, stream)
         : in_dtype == CP_DTYPE_BF16 ? launch_rope_from<__nv_bfloat16>(a, out_dtype, stream)
                                     : launch_rope_from<__half>(a, out_dtype, stream);
}

}  // extern "C"
