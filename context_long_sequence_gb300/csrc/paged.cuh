// paged.cuh -- device helpers shared by the paged-cache kernels.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "debug.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace cpattn {

// The batch arrays and page numbers are data that no host check has seen;
// these checks are therefore in every build, unlike CP_IN_BOUNDS.
#define CP_CHECK_DATA(cond, status) ((cond) || ::cpattn::debug_bounds_fail((status), __LINE__, CP_TU_ID))

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

}  // namespace cpattn
