// paged_small.cuh -- attention over the paged cache for entries of few rows
// (a decode step, short drafts), by single warps.
//
// Bound by reading the cache: at 16 rows a key's 4 d bytes take 64 d flops.
// A warp is a worker of its own: it fetches its 16-key tiles (one TMA box each
// for K and V, 128-byte swizzle) into a ring of stages, multiplies with
// mma.sync (8 rows at a time, where tcgen05 would waste 120 of 128) and writes
// its part.  Nothing is shared between warps, so none waits for another, and
// the eight of an SM hide each other's latencies; the many parts cost little
// to merge, a row of d floats each for few rows.
//
// Measured (32 query heads on 8 of d = 128, keys of one step): 64 sequences of
// up to 16K keys, 2.16 GB from DRAM in 324 us, 6.65 TB/s; a sequence of 2^20
// keys 4.3 GB in 636 us, 6.75 TB/s.  An SM by itself reads 112 GB/s: 79 with a
// copy for each 64 columns, 87 with one a tile and rows as the MMA's rows.
// With few keys the time is latency: 1000 keys of one sequence, 8.1 us with
// the merge, most of it instructions that come from L2 once.
#pragma once
#include <type_traits>

#include "paged.cuh"

namespace cpattn {

template <int D>
struct SmallSmem {
  static constexpr int kHalf = 16 * 128;                 // 64 columns of a tile, 128 bytes a row
  static constexpr int kKV = 16 * D * 2;                 // K or V of a stage
  static constexpr int kStages = 24 * 1024 / (2 * kKV);  // 3 (d = 128) or 6: 192 KB in flight on an SM
  static constexpr int kWarp = kStages * 2 * kKV;        // of one warp; a multiple of 1 KB
  // Segments known: those of the tiles in flight (a segment may be one tile)
  // and the end mark.
  static constexpr int kSegs = kStages + 1;
  static constexpr int offSums = kSmallWarps * kWarp;    // the walker's window sums, three a window
  static constexpr int offBar = offSums + 3 * kMaxEntries / 32 * 8;
  static constexpr int offSeg = offBar + kSmallWarps * kStages * 8;
  static constexpr int kBytes = offSeg + kSmallWarps * kSegs * static_cast<int>(sizeof(PagedSegment));
};

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// A weight in two halves of the cache's type, p = hi + lo, for the product with
// V (the sum is taken in fp32 before): what is left out is under 1.02 2^-15 of it
// in bf16, 1.13 2^-21 in fp16 (or 2^-25, 2^-34 of the largest weight), where one
// half leaves 2^-8 and 2^-11.  hi is the rounding of a little less than p, so that
// lo is positive where p is (down to 2^-12 in fp16): an infinite value in V stays what it is, which 0 and negative
// halves would make a NaN.  With u the half step, hi = c p (1 + e), |e| <= u, and
// c = 1 - u - s: s p <= lo <= (2 u + s) p, rounded to u of it.  In us, one half
// and two: 64 sequences of up to 16K keys at 4 query heads a KV head 319 and
// 320, at 16 336 and 341 (d = 128), 194 and 181 (d = 64); one of 2^20 keys 620
// and 624: the keys' bytes hide the second product.  At 32 rows (24 sequences of
// 20 rows on 16K keys, d = 64) the products are the bound, 75 and 84, as they
// are for CTAs, where the second would be a third of the MMAs: those round a
// weight once, to half a step of the cache's type.
template <typename T>
__device__ __forceinline__ void split_weights(float p0, float p1, uint32_t& hi, uint32_t& lo) {
  hi = Elem<T>::pack(p0 * Weight<T>::kBelow, p1 * Weight<T>::kBelow);
  const float2 h = Elem<T>::unpack(hi);
  lo = Elem<T>::pack(p0 - h.x, p1 - h.y);
}

// The barriers of warp `warp`, by one lane.
template <int D>
__device__ __forceinline__ void small_init(uint8_t* smem, int warp) {
  using SM = SmallSmem<D>;
  for (int i = 0; i < SM::kStages; ++i) mbar_init(smem_u32(smem) + SM::offBar + 8u * (warp * SM::kStages + i), 1);
  fence_mbar_init();
}

// 8 x 8 transpose of 16-bit elements across the warp.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Places of the lane's ldmatrix rows in a 16 x D tile, for 16-column steps
// k = 0..3 (steps 4..7 lie kHalf further): `a` takes the 8 x 8 pieces in the
// order of the MMA's A operand (rows first), `b` columns first.
__device__ __forceinline__ uint32_t place_a(int k) {
  const int lane = threadIdx.x & 31, row = (((lane >> 3) & 1) << 3) + (lane & 7);
  return row * 128 + (((k * 2 + (lane >> 4)) ^ (row & 7)) << 4);
}
__device__ __forceinline__ uint32_t place_b(int k) {
  const int lane = threadIdx.x & 31, row = ((lane >> 4) << 3) + (lane & 7);
  return row * 128 + (((k * 2 + ((lane >> 3) & 1)) ^ (row & 7)) << 4);
}

// r / G for a row r < 256 of a token tile: with 65536 / G rounded up, the
// product is too large by less than r / 65536 < 1 / G.
struct RowsOf {
  uint32_t inverse;
  __device__ __forceinline__ explicit RowsOf(int G) : inverse((65535u + G) / G) {}
  __device__ __forceinline__ int token(int r) const { return static_cast<int>((r * inverse) >> 16); }
};

// Raise a running maximum (log2 units) to t, the score's, if it exceeds it by
// kSlack; the factor for what was summed under the old one.
template <typename T>
__device__ __forceinline__ float raise_max(float& m, float t) {
  const float up = t > m + Weight<T>::kSlack ? t : m;
  const float f = up > m ? ex2_approx(m - up) : 1.f;
  m = up;
  return f;
}

// One row's weight sum, maximum and place, for its log-sum-exp.  A NaN among
// the scores is one in the sum (the maximum passes over it) and in the result.
template <typename T>
__device__ __forceinline__ void store_lse(const PagedAttnArgs& a, const PagedSegment& seg, int token, int head, long long at,
                                          float sum, float m) {
  const float lse2 = sum != 0.f ? m + lg2_approx(sum) - Weight<T>::kBias : -INFINITY;
  if (seg.mode == kRowsFinal)
    a.lse[static_cast<long long>(head) * a.g.N + token] = lse2 * 0.69314718055994531f;
  else
    a.part_lse[at] = lse2;
}

// Up to 8 rows, as the MMAs' columns: S^T = K Q^T and O^T = V^T P^T, with 16
// keys (then 16 columns of V) as the rows.  A group of 4 or 8 query heads
// fills half or all of the 8 columns; as the MMA's 16 rows it would take twice
// the products, exponentials and accumulators.  (One SM reads 112 GB/s of
// keys this way, 87 the other.)
template <typename T, int D>
struct SmallColumns {
  static constexpr int kRows = 8;
  int lim[2];  // keys seen by rows c2, c2 + 1
  uint32_t q[D / 16][2];
  float o[D / 16][4], m[2], l[2];
  uint32_t at_k[4], at_v[4];
  const RowsOf of;

  __device__ __forceinline__ SmallColumns(uint32_t k, uint32_t v, int G) : of(G) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      at_k[i] = k + place_a(i);
      at_v[i] = v + place_b(i);
    }
  }

  __device__ __forceinline__ void begin(const PagedAttnArgs& a, const PagedSegment& seg) {
    const int lane = threadIdx.x & 31, r = lane >> 2, c2 = 2 * (lane & 3), G = a.g.G, rows = seg.nt * G;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      lim[y] = c2 + y < rows ? min(seg.keys, seg.limit0 + of.token(c2 + y)) : 0;
      m[y] = -INFINITY;
      l[y] = 0.f;
    }
    const int i = of.token(r);
    const T* p = static_cast<const T*>(a.q) + (static_cast<long long>(seg.t0) + i) * a.q_stride + (seg.h * G + r - i * G) * D + c2;
    const bool there = r < rows && CP_IN_BOUNDS(token_in(a.g, seg.t0 + i, seg.h * G + r - i * G), a.status);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      q[k][0] = there ? *reinterpret_cast<const uint32_t*>(p + k * 16) : 0u;
      q[k][1] = there ? *reinterpret_cast<const uint32_t*>(p + k * 16 + 8) : 0u;
#pragma unroll
      for (int x = 0; x < 4; ++x) o[k][x] = 0.f;
    }
  }

  // 16 keys from key0 on; `clean`: fetched and seen by every row; keep[]: V's
  // keys that hold something, for the lane's pairs.
  __device__ __forceinline__ void tile(uint32_t stage, int key0, bool there, bool clean, const uint32_t (&keep)[2], float sl2) {
    constexpr uint32_t kAll = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    float c[2][4];  // two chains
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i >> 2][i & 3] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint32_t f[4];
      ldmatrix4<false>(f, at_k[k & 3] + stage + (k >> 2) * SmallSmem<D>::kHalf);
      mma16816<T>(c[k & 1], f, q[k][0], q[k][1]);
    }
    float x[4];  // keys lane / 4 (0, 1) and 8 further (2, 3) of rows c2, c2 + 1
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = c[0][i] + c[1][i];
      if (!clean && (!there || key0 + (lane >> 2) + (i >> 1) * 8 >= lim[i & 1])) x[i] = -INFINITY;
    }
    float t[2] = {fmaxf(x[0], x[2]) * sl2, fmaxf(x[1], x[3]) * sl2};
    if (!__all_sync(kAll, t[0] <= m[0] + Weight<T>::kSlack && t[1] <= m[1] + Weight<T>::kSlack)) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
#pragma unroll
        for (int z = 4; z < 32; z <<= 1) t[y] = fmaxf(t[y], __shfl_xor_sync(kAll, t[y], z));
        const float f = raise_max<T>(m[y], t[y]);
        l[y] *= f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          o[i][y] *= f;
          o[i][2 + y] *= f;
        }
      }
    }
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = ex2_approx(fmaf(x[i], sl2, Weight<T>::kBias - (m[i & 1] == -INFINITY ? 0.f : m[i & 1])));
    l[0] += p[0] + p[2];
    l[1] += p[1] + p[3];
    uint32_t hi[2], lo[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      split_weights<T>(p[2 * i], p[2 * i + 1], hi[i], lo[i]);
      hi[i] = movmatrix_trans(hi[i]);
      lo[i] = movmatrix_trans(lo[i]);
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      uint32_t f[4];
      ldmatrix4<true>(f, at_v[i & 3] + stage + (i >> 2) * SmallSmem<D>::kHalf);
      if (!clean) {
        f[0] &= keep[0];
        f[1] &= keep[0];
        f[2] &= keep[1];
        f[3] &= keep[1];
      }
      mma16816<T>(o[i], f, hi[0], hi[1]);
      mma16816<T>(o[i], f, lo[0], lo[1]);
    }
  }

  __device__ __forceinline__ void finish(const PagedAttnArgs& a, const PagedSegment& seg) {
    const int lane = threadIdx.x & 31, d0 = lane >> 2, G = a.g.G;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      float sum = l[y];
#pragma unroll
      for (int z = 4; z < 32; z <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, z);
      const int r = 2 * (lane & 3) + y, i = of.token(r);
      if (r >= seg.nt * G) continue;
      const float inv = sum != 0.f ? __fdividef(1.f, sum) : 0.f;
      const int token = seg.t0 + i, head = seg.h * G + r - i * G;
      const long long row = static_cast<long long>(token) * a.g.Hq + head, at = seg.row + (seg.mode == kRowsHome ? row : r);
      if (!CP_IN_BOUNDS(token_in(a.g, token, head) && (seg.mode == kRowsFinal || part_rows_in(a, at, 1)), a.status)) continue;
      // Column 8 j + d0.
      if (seg.mode == kRowsFinal && !a.out_fp32) {
        T* dst = static_cast<T*>(a.o) + row * D + d0;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) dst[j * 8] = static_cast<T>(o[j >> 1][(j & 1) * 2 + y] * inv);
      } else {
        float* dst = (seg.mode == kRowsFinal ? static_cast<float*>(a.o) + row * D : a.part_o + at * D) + d0;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) dst[j * 8] = o[j >> 1][(j & 1) * 2 + y] * inv;
      }
      if (d0 == 0) store_lse<T>(a, seg, token, head, at, sum, m[y]);
    }
  }
};

// Up to 16 NB rows, as the MMAs' rows: S = Q K^T, O = P V.  NB = 2 at d = 64
// only: at d = 128 its registers spill (PagedCut).  24 sequences of 20 rows on
// 16K keys, d = 64: 75.7 us (5.2 TB/s) with NB = 2, 122 with two tiles of NB =
// 1, that read the keys twice.
template <typename T, int D, int NB>
struct SmallBlocks {
  static constexpr int kRows = 16 * NB;
  int lim[NB][2];  // keys seen by rows lane / 4 and 8 further of a block
  uint32_t q[NB][D / 16][4];
  float o[NB][D / 8][4], m[NB][2], l[NB][2];
  uint32_t at_k[4], at_v[4];
  const RowsOf of;

  __device__ __forceinline__ SmallBlocks(uint32_t k, uint32_t v, int G) : of(G) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      at_k[i] = k + place_b(i);
      at_v[i] = v + place_a(i);
    }
  }

  __device__ __forceinline__ void begin(const PagedAttnArgs& a, const PagedSegment& seg) {
    const int lane = threadIdx.x & 31, G = a.g.G, rows = seg.nt * G;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int r = b * 16 + y * 8 + (lane >> 2), i = of.token(r);
        lim[b][y] = r < rows ? min(seg.keys, seg.limit0 + i) : 0;
        m[b][y] = -INFINITY;
        l[b][y] = 0.f;
        const T* p = static_cast<const T*>(a.q) + (static_cast<long long>(seg.t0) + i) * a.q_stride +
                     (seg.h * G + r - i * G) * D + 2 * (lane & 3);
        const bool there = r < rows && CP_IN_BOUNDS(token_in(a.g, seg.t0 + i, seg.h * G + r - i * G), a.status);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          q[b][k][y] = there ? *reinterpret_cast<const uint32_t*>(p + k * 16) : 0u;
          q[b][k][2 + y] = there ? *reinterpret_cast<const uint32_t*>(p + k * 16 + 8) : 0u;
        }
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i) o[b][i][0] = o[b][i][1] = o[b][i][2] = o[b][i][3] = 0.f;
    }
  }

  __device__ __forceinline__ void tile(uint32_t stage, int key0, bool there, bool clean, const uint32_t (&keep)[2], float sl2) {
    constexpr uint32_t kAll = 0xffffffffu;
    constexpr int CH = NB == 1 ? 2 : 1;  // chains per 8 keys
    const int c2 = 2 * (threadIdx.x & 3);
    float c[NB][CH][2][4];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < CH * 8; ++i) c[b][i / 8][(i / 4) & 1][i & 3] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint32_t f[4];
      ldmatrix4<false>(f, at_k[k & 3] + stage + (k >> 2) * SmallSmem<D>::kHalf);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        mma16816<T>(c[b][k % CH][0], q[b][k], f[0], f[1]);
        mma16816<T>(c[b][k % CH][1], q[b][k], f[2], f[3]);
      }
    }
    constexpr bool kTwo = NB == 1;  // halves of a weight (split_weights)
    uint32_t hi[NB][4], lo[NB][4];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float x[8];  // first row: 0, 1, 4, 5; second: 2, 3, 6, 7
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = c[b][0][i >> 2][i & 3] + (CH == 2 ? c[b][CH - 1][i >> 2][i & 3] : 0.f);
        if (!clean && (!there || key0 + (i >> 2) * 8 + c2 + (i & 1) >= lim[b][(i >> 1) & 1])) x[i] = -INFINITY;
      }
      float t[2] = {fmaxf(fmaxf(x[0], x[1]), fmaxf(x[4], x[5])) * sl2, fmaxf(fmaxf(x[2], x[3]), fmaxf(x[6], x[7])) * sl2};
      if (!__all_sync(kAll, t[0] <= m[b][0] + Weight<T>::kSlack && t[1] <= m[b][1] + Weight<T>::kSlack)) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          t[y] = fmaxf(t[y], __shfl_xor_sync(kAll, t[y], 1));
          t[y] = fmaxf(t[y], __shfl_xor_sync(kAll, t[y], 2));
          const float f = raise_max<T>(m[b][y], t[y]);
          l[b][y] *= f;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            o[b][i][2 * y] *= f;
            o[b][i][2 * y + 1] *= f;
          }
        }
      }
      float p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float top = m[b][(i >> 1) & 1];
        p[i] = ex2_approx(fmaf(x[i], sl2, Weight<T>::kBias - (top == -INFINITY ? 0.f : top)));
      }
      l[b][0] += (p[0] + p[1]) + (p[4] + p[5]);
      l[b][1] += (p[2] + p[3]) + (p[6] + p[7]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (kTwo)
          split_weights<T>(p[2 * i], p[2 * i + 1], hi[b][i], lo[b][i]);
        else
          hi[b][i] = Elem<T>::pack(p[2 * i], p[2 * i + 1]);
      }
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      uint32_t f[4];
      ldmatrix4<true>(f, at_v[i & 3] + stage + (i >> 2) * SmallSmem<D>::kHalf);
      if (!clean) {
        f[0] &= keep[0];
        f[1] &= keep[1];
        f[2] &= keep[0];
        f[3] &= keep[1];
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        mma16816<T>(o[b][2 * i], hi[b], f[0], f[1]);
        mma16816<T>(o[b][2 * i + 1], hi[b], f[2], f[3]);
        if constexpr (kTwo) {
          mma16816<T>(o[b][2 * i], lo[b], f[0], f[1]);
          mma16816<T>(o[b][2 * i + 1], lo[b], f[2], f[3]);
        }
      }
    }
  }

  __device__ __forceinline__ void finish(const PagedAttnArgs& a, const PagedSegment& seg) {
    const int lane = threadIdx.x & 31, G = a.g.G;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float sum = l[b][y];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const int r = b * 16 + y * 8 + (lane >> 2), i = of.token(r);
        if (r >= seg.nt * G) continue;
        const float inv = sum != 0.f ? __fdividef(1.f, sum) : 0.f;
        const int token = seg.t0 + i, head = seg.h * G + r - i * G;
        const long long row = static_cast<long long>(token) * a.g.Hq + head, at = seg.row + (seg.mode == kRowsHome ? row : r);
        if (!CP_IN_BOUNDS(token_in(a.g, token, head) && (seg.mode == kRowsFinal || part_rows_in(a, at, 1)), a.status)) continue;
        if (seg.mode == kRowsFinal && !a.out_fp32) {
          T* dst = static_cast<T*>(a.o) + row * D + 2 * (lane & 3);
#pragma unroll
          for (int j = 0; j < D / 8; ++j)
            *reinterpret_cast<uint32_t*>(dst + j * 8) = Elem<T>::pack(o[b][j][2 * y] * inv, o[b][j][2 * y + 1] * inv);
        } else {
          float* dst = (seg.mode == kRowsFinal ? static_cast<float*>(a.o) + row * D : a.part_o + at * D) + 2 * (lane & 3);
#pragma unroll
          for (int j = 0; j < D / 8; ++j)
            *reinterpret_cast<float2*>(dst + j * 8) = make_float2(o[b][j][2 * y] * inv, o[b][j][2 * y + 1] * inv);
        }
        if ((lane & 3) == 0) store_lse<T>(a, seg, token, head, at, sum, m[b][y]);
      }
  }
};

// The kind for entries of up to 8, 16 or 32 rows.
template <typename T, int D, int ROWS>
using SmallRows = typename std::conditional<ROWS == 8, SmallColumns<T, D>, SmallBlocks<T, D, ROWS <= 16 ? 1 : 2>>::type;

// The share of the block's warp `warp`, whose walk has begun and whose
// barriers are set.
template <typename Rows, int D, typename Walk>
__device__ __forceinline__ void small_worker(uint8_t* smem, int warp, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                             Walk& walk) {
  using SM = SmallSmem<D>;
  constexpr int S = SM::kStages;
  constexpr uint32_t kAll = 0xffffffffu;
  const uint32_t s0 = smem_u32(smem) + warp * SM::kWarp;
  const uint32_t full0 = smem_u32(smem) + SM::offBar + 8u * (warp * S);
  const int lane = threadIdx.x & 31;
  const PagedAttnArgs& args = walk.a;
  const PagedGeom& g = args.g;
  int32_t* status = args.status;
  PagedSegment* segs = reinterpret_cast<PagedSegment*>(smem + SM::offSeg) + warp * SM::kSegs;

  // ---- Fetching, S tiles ahead of the computing.
  const uint64_t policy = read_once_policy();
  int f_seg = 0, f_n = 0, f_st = 0;    // segments walked, tiles fetched, the next one's stage
  uint32_t held = 0;                   // stages whose page was fetched
  int f_tile = 0, f_end = 0, f_h = 0;  // of the segment being fetched
  int f_pages = -1, f_next = -1;       // lane: page of tile (f_tile & ~31) + lane, and of the 32 after
  bool f_more = true;
  const int32_t* f_table = nullptr;
  auto pages_of = [&](int tile) { return tile < f_end ? f_table[static_cast<long long>(tile) * 16 >> g.page_shift] : -1; };
  auto fetch = [&]() {
    if (!f_more) return;
    if (f_tile == f_end) {
      const PagedSegment s = walk.next();
      if (lane == 0) segs[f_seg % SM::kSegs] = s;
      __syncwarp();
      ++f_seg;
      if (!(f_more = s.nt > 0)) return;
      f_tile = s.tile0;
      f_end = s.tile1;
      f_h = s.h;
      f_table = walk.table;
      f_pages = pages_of((f_tile & ~31) + lane);
      f_next = pages_of((f_tile & ~31) + 32 + lane);
    } else if ((f_tile & 31) == 0) {
      f_pages = f_next;
      f_next = pages_of(f_tile + 32 + lane);
    }
    const int page = __shfl_sync(kAll, f_pages, f_tile & 31);
    const bool there = page >= 0 && page < g.num_pages;
    held = (held & ~(1u << f_st)) | (there ? 1u << f_st : 0u);
    if (lane == 0) {
      const uint32_t full = full0 + 8u * f_st, dst = s0 + f_st * 2 * SM::kKV;
      const int row = (f_tile * 16) & ((1 << g.page_shift) - 1);
      mbar_arrive_expect_tx(full, there ? 2 * SM::kKV : 0);
      if (CP_CHECK_DATA(there, status)) {
        (void)CP_IN_BOUNDS(cache_box_in(g, row, 16, f_h, page), status);
        tma_load_5d(dst, &tm_k, full, 0, row, 0, f_h, page, policy);
        tma_load_5d(dst + SM::kKV, &tm_v, full, 0, row, 0, f_h, page, policy);
      }
    }
    __syncwarp();
    f_st = f_st + 1 == S ? 0 : f_st + 1;
    ++f_n;
    ++f_tile;
  };
#pragma unroll 1
  for (int i = 0; i < S; ++i) fetch();

  // ---- Computing.
  const float sl2 = g.scale * 1.4426950408889634f;
  Rows rows(s0, s0 + SM::kKV, g.G);
  int n = 0, st = 0;    // tiles computed, the next one's stage
  uint32_t phase = 0;
  bool ok = true;
#pragma unroll 1
  for (int c_seg = 0; ok; ++c_seg) {
    const PagedSegment seg = segs[c_seg % SM::kSegs];
    if (seg.nt == 0) break;
    const int lim_all = min(seg.keys, seg.limit0);  // seen by every row
    rows.begin(args, seg);
#pragma unroll 1
    for (int tile = seg.tile0; tile < seg.tile1; ++tile, ++n) {
      const int key0 = tile * 16;
      ok = __all_sync(kAll, mbar_wait_short(full0 + 8u * st, phase, nullptr, status));
      if (!ok) break;
      const bool there = (held >> st) & 1u, clean = there && key0 + 16 <= lim_all;
      uint32_t keep[2] = {kAll, kAll};
      if (!clean) {
        // What lies behind the last key may be anything, NaN included: 0 * NaN
        // would reach O.  An MMA's lane holds V's keys c, c + 1 and 8 further.
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!there || key0 + (i >> 1) * 8 + 2 * (lane & 3) + (i & 1) >= seg.keys) keep[i >> 1] &= i & 1 ? 0x0000ffffu : 0xffff0000u;
      }
      rows.tile(st * 2 * SM::kKV, key0, there, clean, keep, sl2);
      __syncwarp();  // the stage is read: the next tile may land on it
      st = st + 1 == S ? 0 : st + 1;
      phase ^= st == 0;
      fetch();
    }
    if (!ok) break;
    rows.finish(args, seg);
  }
  if (!ok)  // let every copy still in flight land
    for (; n < f_n; ++n) mbar_wait(full0 + 8u * (n % S), (n / S) & 1, nullptr, status);
}

}  // namespace cpattn
