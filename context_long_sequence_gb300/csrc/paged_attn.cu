// paged_attn.cu -- attention of a batch's new tokens over the paged
// key/value cache, shared prefixes included.
//
// For one token row and query head, over the keys that it sees (its
// sequence's own, up to the causal limit, and its prefix's):
//   m = max_k s_k,  l = sum_k e^(s_k - m),  O = sum_k e^(s_k - m) v_k / l,
//   LSE = m + ln l,   s_k = scale * q . k_k.
//
// One warp takes one (token, query head): lane i holds elements i, i + 32, ..
// of the row, the running maximum and sum stay in fp32, one pass over the
// keys.
#include <cuda_runtime.h>

#define CP_TU_ID ::cpattn::kTuPagedAttn
#include "paged.cuh"

namespace cpattn {
namespace {

constexpr int kWarps = 4;

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) paged_attn_kernel(const __grid_constant__ PagedAttnArgs args) {
  constexpr int E = D / 32;
  const PagedGeom& g = args.g;
  const int lane = threadIdx.x & 31;
  const long long w = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int t = static_cast<int>(w / g.Hq), h = static_cast<int>(w % g.Hq);
  if (t >= g.N) return;
  const int s = warp_count_le(g.q_start + 1, g.B, t);
  if (s >= g.B) return;
  const PagedEntry own = paged_entry(g, s);
  if (!CP_CHECK_DATA(!own.bad, args.status) || t < own.t0 || t >= own.t0 + own.n) return;
  const int p = warp_prefix_of(g, s);
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] = static_cast<float>(static_cast<const T*>(args.q)[t * args.q_stride + h * D + i * 32 + lane]) * g.scale;
    o[i] = 0.f;
  }
  for (int part = p >= 0 ? 0 : 1; part < 2; ++part) {
    const PagedEntry e = part ? own : paged_entry(g, g.B + p);
    if (!CP_CHECK_DATA(!e.bad, args.status)) continue;
    const int keys = min(e.keys, e.limit0 + (t - e.t0));
    for (int k = 0; k < keys; ++k) {
      const int page = e.table[k >> g.page_shift];
      if (!CP_CHECK_DATA(page >= 0 && page < g.num_pages, args.status)) continue;
      const int64_t at = page * g.page_stride + (k & ((1 << g.page_shift) - 1)) * g.token_stride + (h / g.G) * g.head_stride;
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) dot = fmaf(q[i], static_cast<float>(static_cast<const T*>(args.k_cache)[at + i * 32 + lane]), dot);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, x);
      const float m_new = fmaxf(m, dot);
      const float alpha = expf(m - m_new), pk = expf(dot - m_new);
      m = m_new;
      l = l * alpha + pk;
#pragma unroll
      for (int i = 0; i < E; ++i)
        o[i] = fmaf(pk, static_cast<float>(static_cast<const T*>(args.v_cache)[at + i * 32 + lane]), o[i] * alpha);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const int64_t row = (static_cast<int64_t>(t) * g.Hq + h) * D;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    if (args.out_fp32)
      static_cast<float*>(args.o)[row + i * 32 + lane] = o[i] * inv;
    else
      static_cast<T*>(args.o)[row + i * 32 + lane] = static_cast<T>(o[i] * inv);
  }
  if (lane == 0) args.lse[static_cast<int64_t>(h) * g.N + t] = l > 0.f ? m + logf(l) : -INFINITY;
}

template <typename T, int D>
int launch_attn_d(const PagedAttnArgs& a, cudaStream_t stream) {
  const long long warps = static_cast<long long>(a.g.N) * a.g.Hq;
  const long long grid = (warps + kWarps - 1) / kWarps;
  if (grid > 0x7fffffffLL) return CP_ERR_UNSUPPORTED;
  paged_attn_kernel<T, D><<<static_cast<unsigned>(grid), kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? CP_OK : CP_ERR_CUDA;
}

}  // namespace

int launch_paged_attn(const PagedAttnArgs& a, cudaStream_t stream) {
  const bool bf16 = a.g.dtype == CP_DTYPE_BF16;
  if (a.g.d == 128) return bf16 ? launch_attn_d<__nv_bfloat16, 128>(a, stream) : launch_attn_d<__half, 128>(a, stream);
  if (a.g.d == 64) return bf16 ? launch_attn_d<__nv_bfloat16, 64>(a, stream) : launch_attn_d<__half, 64>(a, stream);
  return CP_ERR_UNSUPPORTED;
}

}  // namespace cpattn
