// host.h -- what the C-ABI files of the paged cache and of the calls around its
// attention share on the host: argument checks, the architecture check, NVTX ranges.
#pragma once
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cstdint>

#include "cp_attn.h"

namespace cpattn {

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

constexpr int64_t kMaxStride = 1LL << 36;  // elements; a tensor map takes strides below 2^40 bytes

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The kernels are built for sm_103 alone; asked once per device.
inline int check_arch() {
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

// f radians as a fraction of a full circle, in units of 2^-64 (paged.cu).
uint64_t turns_of(double f);

// The pairs of a rotation (paged.cu): turns[j] of pair j's frequency, freqs[j]
// or base^(-2j/rope_dim), and its axis, below axes.  CP_OK, or why not.
int rope_pairs(int rope_dim, double base, const double* freqs, int axes, const int32_t* axis_of, uint64_t* turns, uint8_t* axis);

// What a plan and a batch say to calls that have files of their own (paged.cu):
// the plan's max_new, or a CP_ERR_* code if the batch leaves its bounds.
int paged_max_new(const cp_paged_t* plan, const cp_paged_batch_t& batch);
// log2 of its page size; the heads and dimension of its pages; what is wrong with a cache.
int paged_page_shift(const cp_paged_t* plan);
void paged_rows(const cp_paged_t* plan, int* Hkv, int* d);
int paged_check_cache(const cp_paged_t* plan, const cp_paged_cache_t& cache);

}  // namespace cpattn
