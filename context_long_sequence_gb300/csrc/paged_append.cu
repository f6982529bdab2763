// paged_append.cu -- a step's new keys and values into the paged cache, the
// keys (and the step's queries) turned by their rotary position angles.
//
// Pair (a, b) number j of a head at position pos turns by the angle
// theta = pos * f_j: (a cos - b sin, b cos + a sin).  An angle of a far
// position needs more than fp32: at pos = 10^6, pos * f_0 has an fp32 step of
// 0.06 rad.  The host therefore gives f_j / 2 pi as a 64-bit binary fraction
// of a circle, good to 2^-63 for |f_j| up to 2^42 (turns_of in paged.cu).  pos *
// that, modulo 2^64, is one integer product, good to pos * 2^-63 turns, 2^-32 at
// the farthest position; its upper 32 bits, cut at 2^-32 turns and rounded to
// fp32 (at most 2^-25 half-turns), go to sincospif as a number of half-turns in
// [-1, 1).  rope_base's f_j is a double itself, off by 2^-53 of it.
//
// Bound by memory: every new row is read once and written once (16K tokens of
// 32 + 2 x 8 heads of 128: 403 MB in 62.4 us, 6.45 TB/s), and for few tokens
// by the launch (3.3 us in a graph).  A warp owns one token (or a share of its
// heads): a lane holds 16 elements of a head, two 16-byte pieces that hold
// both halves of eight pairs, so its eight sines and cosines serve every head
// it visits; four groups of heads are loaded before the first is stored.
//
// The rotation is in fp32 with one rounding at the end.
#include <cuda_runtime.h>

#define CP_TU_ID ::cpattn::kTuPagedAppend
#include "paged.cuh"

namespace cpattn {
namespace {

constexpr int kAppendWarps = 2;
constexpr int kAhead = 4;            // groups of heads whose loads are in flight together
constexpr int kFillWarps = 152 * 32;  // warps that keep the memory busy

// Eight pairs: a[i], b[i].  Halves: the pairs are (a, b) of the two pieces.
// Interleaved: neighbours, four pairs in each piece.
template <typename T>
__device__ __forceinline__ void turn(uint4& a, uint4& b, const float (&c)[8], const float (&s)[8], bool interleaved) {
  uint32_t* x = reinterpret_cast<uint32_t*>(&a);
  uint32_t* y = reinterpret_cast<uint32_t*>(&b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = Elem<T>::unpack(x[i]), w = Elem<T>::unpack(y[i]);
    if (interleaved) {
      x[i] = Elem<T>::pack(u.x * c[i] - u.y * s[i], u.y * c[i] + u.x * s[i]);
      y[i] = Elem<T>::pack(w.x * c[4 + i] - w.y * s[4 + i], w.y * c[4 + i] + w.x * s[4 + i]);
    } else {
      x[i] = Elem<T>::pack(u.x * c[2 * i] - w.x * s[2 * i], u.y * c[2 * i + 1] - w.y * s[2 * i + 1]);
      y[i] = Elem<T>::pack(w.x * c[2 * i] + u.x * s[2 * i], w.y * c[2 * i + 1] + u.y * s[2 * i + 1]);
    }
  }
}

// Warp `unit` of `units` of a token visits every units-th group of heads; a
// group is 512 elements, 32 lanes of 16.
template <typename T, int D, bool AXES>
__global__ void __launch_bounds__(kAppendWarps * 32)
    paged_append_kernel(const __grid_constant__ AppendArgs args, int units) {
  constexpr int LPH = D / 16;       // lanes per head
  constexpr int HPG = 32 / LPH;     // heads per group
  const PagedGeom& g = args.g;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long w = static_cast<long long>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
  const int t = static_cast<int>(w / units), unit = static_cast<int>(w % units);
  if (t >= g.N) return;
  const int s = warp_count_le(g.q_start + 1, g.B, t);
  if (s >= g.B) return;  // a row behind the last sequence
  const PagedEntry e = paged_entry(g, s);
  if (!CP_CHECK_DATA(!e.bad, args.status) || t < e.t0 || t >= e.t0 + e.n) return;
  const int at = e.keys - e.n + (t - e.t0);  // place among the sequence's own keys
  const int page = CP_CHECK_DATA(at >= 0, args.status) ? e.table[at >> g.page_shift] : -1;
  if (!CP_CHECK_DATA(page >= 0 && page < g.num_pages, args.status)) return;
  const int64_t row = page * g.page_stride + (at & ((1 << g.page_shift) - 1)) * g.token_stride;

  const int j = lane % LPH, sub = lane / LPH;
  const bool rotated = j < args.rope_dim / 16;
  const bool halves = rotated && !args.interleaved;
  const int ea = halves ? 8 * j : 16 * j;                       // first elements of the lane's two pieces
  const int eb = halves ? args.rope_dim / 2 + 8 * j : 16 * j + 8;
  float c[8], sn[8];
  int pos = at;
  if (g.positions) {
    if constexpr (!AXES) pos = g.positions[t];
  } else if (args.rope_dim > 0) {
    // Looked up by the whole warp, the lanes behind rope_dim too.  A bad prefix,
    // or one whose rows this is not among, is none: as in the attention.
    const int p = warp_prefix_of(g, s);
    if (p >= 0) {
      const PagedEntry pre = paged_entry(g, g.B + p);
      if (CP_CHECK_DATA(!pre.bad, args.status) && t >= pre.t0 && t < pre.t0 + pre.n) pos += pre.keys;
    }
  }
  if (rotated) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (AXES) {
        if (g.positions) pos = g.positions[static_cast<size_t>(args.axis[8 * j + i]) * g.N + t];
      }
      sincos_turns(pos, args.turns[8 * j + i], &sn[i], &c[i]);
    }
  }
  const int heads = g.Hq + 2 * g.Hkv, groups = (heads + HPG - 1) / HPG;
  // Four groups at a time, their loads before the first store.
  for (int g0 = unit; g0 < groups; g0 += kAhead * units) {
    uint4 a[kAhead], b[kAhead];
    T* dst[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int h = (g0 + i * units) * HPG + sub;
      const T* src = nullptr;
      dst[i] = nullptr;
      if (h < g.Hq) {
        if (args.q) {
          src = static_cast<const T*>(args.q) + t * args.q_stride + h * D;
          dst[i] = static_cast<T*>(args.q_out) + t * args.q_out_stride + h * D;
        }
      } else if (h < g.Hq + g.Hkv) {
        src = static_cast<const T*>(args.k) + t * args.k_stride + (h - g.Hq) * D;
        dst[i] = static_cast<T*>(args.k_cache) + row + (h - g.Hq) * g.head_stride;
      } else if (h < heads) {
        src = static_cast<const T*>(args.v) + t * args.v_stride + (h - g.Hq - g.Hkv) * D;
        dst[i] = static_cast<T*>(args.v_cache) + row + (h - g.Hq - g.Hkv) * g.head_stride;
      }
      if (src && !CP_IN_BOUNDS(ea + 8 <= D && eb + 8 <= D && e.t0 + e.n <= g.N, args.status)) src = nullptr, dst[i] = nullptr;
      if (src) {
        a[i] = *reinterpret_cast<const uint4*>(src + ea);
        b[i] = *reinterpret_cast<const uint4*>(src + eb);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (!dst[i]) continue;
      if (rotated && (g0 + i * units) * HPG + sub < g.Hq + g.Hkv) turn<T>(a[i], b[i], c, sn, args.interleaved != 0);
      *reinterpret_cast<uint4*>(dst[i] + ea) = a[i];
      *reinterpret_cast<uint4*>(dst[i] + eb) = b[i];
    }
  }
}

template <typename T, int D, bool AXES>
int launch_append_axes(const AppendArgs& a, cudaStream_t stream) {
  const int groups = (a.g.Hq + 2 * a.g.Hkv + 512 / D - 1) / (512 / D);
  // Few tokens: a warp for each group of heads, for latency.  Many: a warp
  // takes more of its token's heads, as one set of sines serves them all.
  int units = (kFillWarps + a.g.N - 1) / a.g.N;
  units = units < 1 ? 1 : units > groups ? groups : units;
  const long long warps = static_cast<long long>(a.g.N) * units;
  const long long grid = (warps + kAppendWarps - 1) / kAppendWarps;
  if (grid > 0x7fffffffLL) return CP_ERR_UNSUPPORTED;
  return launch(paged_append_kernel<T, D, AXES>, static_cast<unsigned>(grid), kAppendWarps * 32, 0, stream, a, units);
}

// A plan of several axes looks its positions up pair by pair.
template <typename T, int D>
int launch_append_d(const AppendArgs& a, cudaStream_t stream) {
  return a.axes > 1 ? launch_append_axes<T, D, true>(a, stream) : launch_append_axes<T, D, false>(a, stream);
}

}  // namespace

int launch_paged_append(const AppendArgs& a, cudaStream_t stream) {
  const bool bf16 = a.g.dtype == CP_DTYPE_BF16;
  if (a.g.d == 128) return bf16 ? launch_append_d<__nv_bfloat16, 128>(a, stream) : launch_append_d<__half, 128>(a, stream);
  if (a.g.d == 64) return bf16 ? launch_append_d<__nv_bfloat16, 64>(a, stream) : launch_append_d<__half, 64>(a, stream);
  return CP_ERR_UNSUPPORTED;
}

}  // namespace cpattn
