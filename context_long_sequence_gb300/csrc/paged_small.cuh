// paged_small.cuh -- attention over the paged cache for entries of few rows
// (a decode step, short drafts), by single warps.
//
// Bound by reading the cache: at 16 rows a key's 4 d bytes take 64 d flops.
// A warp is a worker of its own: it fetches its 16-key tiles (TMA boxes,
// 128-byte swizzle) into a ring of stages, multiplies with mma.sync (8 rows at
// a time, where tcgen05 would waste 120 of 128) and writes its part.  Nothing is
// shared between warps, so none waits for another, and the eight of an SM hide
// each other's latencies; the many parts cost little to merge, a row of d
// floats each for few rows.
#pragma once
#include "paged.cuh"

namespace cpattn {

constexpr int kSmallWarps = 8;  // workers of a CTA, one CTA an SM

template <int D>
struct SmallSmem {
  static constexpr int kHalf = 16 * 128;                 // 64 columns of a tile, 128 bytes a row
  static constexpr int kKV = 16 * D * 2;                 // K or V of a stage
  static constexpr int kStages = 24 * 1024 / (2 * kKV);  // 3 (d = 128) or 6: 192 KB in flight on an SM
  static constexpr int kWarp = kStages * 2 * kKV;        // of one warp; a multiple of 1 KB
  // Segments known: those of the tiles in flight (a segment may be one tile)
  // and the end mark.
  static constexpr int kSegs = kStages + 1;
  static constexpr int offSums = kSmallWarps * kWarp;    // the walker's window sums, two cuts
  static constexpr int offBar = offSums + 2 * kMaxEntries / 32 * 8;
  static constexpr int offSeg = offBar + kSmallWarps * kStages * 8;
  static constexpr int offHeld = offSeg + kSmallWarps * kSegs * static_cast<int>(sizeof(PagedSegment));
  static constexpr int kBytes = offHeld + kSmallWarps * kStages * 4;  // held: whether the stage's page was fetched
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

// The share of the block's warp `warp`, whose walk has begun and whose
// barriers are set.  Entries have up to 8 NT rows.
//
// The products are taken transposed, S^T = K Q^T and O^T = V^T P^T, with keys
// (then columns of V) as the 16 rows of an MMA and 8 query rows as its
// columns: a group of 4 or 8 query heads fills half or all of that, where as
// the MMA's rows it would fill a quarter or half.
template <typename T, int D, int NT>
__device__ __forceinline__ void small_worker(uint8_t* smem, int warp, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                             PagedWalker& walk) {
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
  volatile int* held = reinterpret_cast<volatile int*>(smem + SM::offHeld) + warp * S;

  // ---- Fetching, S tiles ahead of the computing.
  const uint64_t policy = read_once_policy();
  int f_seg = 0, f_n = 0;              // segments walked, tiles fetched
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
    const int page = __shfl_sync(kAll, f_pages, f_tile & 31), st = f_n % S;
    const bool there = page >= 0 && page < g.num_pages;
    if (lane == 0) {
      const uint32_t full = full0 + 8u * st, dst = s0 + st * 2 * SM::kKV;
      const int row = (f_tile * 16) & ((1 << g.page_shift) - 1);
      held[st] = there;
      mbar_arrive_expect_tx(full, there ? 2 * SM::kKV : 0);
      if (CP_CHECK_DATA(there, status)) {
        tma_load_5d(dst, &tm_k, full, 0, row, 0, f_h, page, policy);
        tma_load_5d(dst + SM::kKV, &tm_v, full, 0, row, 0, f_h, page, policy);
      }
    }
    __syncwarp();
    ++f_n;
    ++f_tile;
  };
#pragma unroll 1
  for (int i = 0; i < S; ++i) fetch();

  // ---- Computing.
  const float sl2 = g.scale * 1.4426950408889634f;
  const int r8 = lane >> 2, c2 = 2 * (lane & 3);  // row and first column of the lane in an MMA fragment
  // ldmatrix places of the lane, relative to a stage: K as [keys][columns] and
  // V, transposed on the way, as [columns][keys]; 16-column steps k and k + 4
  // lie kHalf apart.
  uint32_t at_k[4], at_v[4];
  {
    const int row_k = (((lane >> 3) & 1) << 3) + (lane & 7), piece_k = lane >> 4;
    const int row_v = ((lane >> 4) << 3) + (lane & 7), piece_v = (lane >> 3) & 1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      at_k[k] = s0 + row_k * 128 + (((k * 2 + piece_k) ^ (row_k & 7)) << 4);
      at_v[k] = s0 + SM::kKV + row_v * 128 + (((k * 2 + piece_v) ^ (row_v & 7)) << 4);
    }
  }
  int n = 0;
  bool ok = true;
#pragma unroll 1
  for (int c_seg = 0; ok; ++c_seg) {
    const PagedSegment seg = segs[c_seg % SM::kSegs];
    if (seg.nt == 0) break;
    const int rows = seg.nt * g.G;
    const int lim_all = min(seg.keys, seg.limit0);  // seen by every row
    int lim[NT][2];                                 // seen by rows c2, c2 + 1 of each eight
    uint32_t q[NT][D / 16][2];
#pragma unroll
    for (int b = 0; b < NT; ++b) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int r = b * 8 + c2 + y;
        lim[b][y] = r < rows ? min(seg.keys, seg.limit0 + r / g.G) : 0;
      }
      const int r = b * 8 + r8, i = r / g.G;
      const T* p = static_cast<const T*>(args.q) + (static_cast<long long>(seg.t0) + i) * args.q_stride + (seg.h * g.G + r - i * g.G) * D + c2;
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int x = 0; x < 2; ++x) q[b][k][x] = r < rows ? *reinterpret_cast<const uint32_t*>(p + k * 16 + x * 8) : 0u;
    }
    float o[NT][D / 16][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int b = 0; b < NT; ++b) {
      m[b][0] = m[b][1] = -INFINITY;
      l[b][0] = l[b][1] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[b][i][0] = o[b][i][1] = o[b][i][2] = o[b][i][3] = 0.f;
    }
#pragma unroll 1
    for (int tile = seg.tile0; tile < seg.tile1; ++tile, ++n) {
      const int st = n % S, key0 = tile * 16;
      ok = __all_sync(kAll, mbar_wait_short(full0 + 8u * st, (n / S) & 1, nullptr, status));
      if (!ok) break;
      const bool there = held[st];
      const bool clean = there && key0 + 16 <= lim_all;
      const uint32_t stage = st * 2 * SM::kKV;
      // S^T for 16 keys; few rows leave room for two chains.
      constexpr int CH = NT <= 2 ? 2 : 1;
      float c[NT][CH][4];
#pragma unroll
      for (int b = 0; b < NT; ++b)
#pragma unroll
        for (int i = 0; i < CH * 4; ++i) c[b][i / 4][i & 3] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t f[4];
        ldmatrix4<false>(f, at_k[k & 3] + stage + (k >> 2) * SM::kHalf);
#pragma unroll
        for (int b = 0; b < NT; ++b) mma16816<T>(c[b][k % CH], f, q[b][k][0], q[b][k][1]);
      }
      uint32_t keep0 = kAll, keep1 = kAll;  // V rows that hold keys, for the lane's two pairs
      if (!clean) {
        // What lies behind the last key may be anything, NaN included: 0 * NaN would reach O.
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!there || key0 + (i >> 1) * 8 + c2 + (i & 1) >= seg.keys) (i & 2 ? keep1 : keep0) &= i & 1 ? 0x0000ffffu : 0xffff0000u;
      }
      uint32_t pb[NT][2];
#pragma unroll
      for (int b = 0; b < NT; ++b) {
        float x[4];  // keys r8 (0, 1) and r8 + 8 (2, 3) of rows c2, c2 + 1
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = CH == 2 ? c[b][0][i] + c[b][CH - 1][i] : c[b][0][i];
        if (!clean) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!there || key0 + r8 + (i >> 1) * 8 >= lim[b][i & 1]) x[i] = -INFINITY;
        }
        const float mx0 = fmaxf(x[0], x[2]) * sl2, mx1 = fmaxf(x[1], x[3]) * sl2;
        if (!__all_sync(kAll, mx0 <= m[b][0] + Weight<T>::kSlack && mx1 <= m[b][1] + Weight<T>::kSlack)) {
          float t[2] = {mx0, mx1};
#pragma unroll
          for (int y = 0; y < 2; ++y) {
#pragma unroll
            for (int z = 4; z < 32; z <<= 1) t[y] = fmaxf(t[y], __shfl_xor_sync(kAll, t[y], z));
            const float up = t[y] > m[b][y] + Weight<T>::kSlack ? t[y] : m[b][y];
            const float f = up > m[b][y] ? ex2_approx(m[b][y] - up) : 1.f;
            m[b][y] = up;
            l[b][y] *= f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              o[b][i][y] *= f;
              o[b][i][2 + y] *= f;
            }
          }
        }
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          p[i] = ex2_approx(fmaf(x[i], sl2, Weight<T>::kBias - (m[b][i & 1] == -INFINITY ? 0.f : m[b][i & 1])));
        l[b][0] += p[0] + p[2];
        l[b][1] += p[1] + p[3];
        // The weights are rounded to the cache's type for the product with V;
        // their sum is not.
        pb[b][0] = movmatrix_trans(Elem<T>::pack(p[0], p[1]));
        pb[b][1] = movmatrix_trans(Elem<T>::pack(p[2], p[3]));
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t f[4];
        ldmatrix4<true>(f, at_v[i & 3] + stage + (i >> 2) * SM::kHalf);
        if (!clean) {
          f[0] &= keep0;
          f[1] &= keep0;
          f[2] &= keep1;
          f[3] &= keep1;
        }
#pragma unroll
        for (int b = 0; b < NT; ++b) mma16816<T>(o[b][i], f, pb[b][0], pb[b][1]);
      }
      __syncwarp();  // the stage is read: the next tile may land on it
      fetch();
    }
    if (!ok) break;
    const bool final_rows = seg.mode == kRowsFinal;
#pragma unroll
    for (int b = 0; b < NT; ++b)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float sum = l[b][y];
#pragma unroll
        for (int z = 4; z < 32; z <<= 1) sum += __shfl_xor_sync(kAll, sum, z);
        const int r = b * 8 + c2 + y, i = r / g.G;
        if (r >= rows) continue;
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        const int token = seg.t0 + i, head = seg.h * g.G + r - i * g.G;
        const long long row = static_cast<long long>(token) * g.Hq + head;
        const long long at = seg.row + (seg.mode == kRowsHome ? row : r);
        // Column 16 j + 8 half + r8.
        if (final_rows && !args.out_fp32) {
          T* dst = static_cast<T*>(args.o) + row * D + r8;
#pragma unroll
          for (int j = 0; j < D / 8; ++j) dst[j * 8] = static_cast<T>(o[b][j >> 1][(j & 1) * 2 + y] * inv);
        } else {
          float* dst = (final_rows ? static_cast<float*>(args.o) + row * D : args.part_o + at * D) + r8;
#pragma unroll
          for (int j = 0; j < D / 8; ++j) dst[j * 8] = o[b][j >> 1][(j & 1) * 2 + y] * inv;
        }
        if (r8 == 0) {
          const float lse2 = sum > 0.f ? m[b][y] + log2f(sum) - Weight<T>::kBias : -INFINITY;
          if (final_rows)
            args.lse[static_cast<long long>(head) * g.N + token] = lse2 * 0.69314718055994531f;
          else
            args.part_lse[at] = lse2;
        }
      }
  }
  if (!ok)  // let every copy still in flight land
    for (; n < f_n; ++n) mbar_wait(full0 + 8u * (n % S), (n / S) & 1, nullptr, status);
}

}  // namespace cpattn
