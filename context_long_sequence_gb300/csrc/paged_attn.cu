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
//   paged_small_kernel   entries of up to 64 rows (tokens x query heads of a
//                        KV head): bound by reading the cache.
//   paged_large_kernel   the others (paged_attn_large.cu).
//   paged_merge_kernel   joins the parts.
#include <cuda.h>
#include <cuda_runtime.h>

#include <type_traits>

#define CP_TU_ID ::cpattn::kTuPagedAttn
#include "paged.cuh"

namespace cpattn {
namespace {

// ---------------------------------------------------------------- few rows
//
// A CTA walks its share of 64-key tiles with a ring of shared-memory stages:
// warp 4 fetches (TMA boxes of up to one page, 128-byte swizzle; page numbers
// one tile ahead), warps 0..3 compute with mma.sync (at these row counts the
// tensor work is a fraction of the time its keys take to arrive, and a row
// block of 16 wastes less than tcgen05's 128).  Two CTAs share an SM, each
// with 96 KB of keys in flight.
//
// Up to 16 rows: the four warps take 16 keys of the tile each, with running
// maxima and sums of their own, and meet only at the end of a segment.  Up to
// 32 rows: two row blocks, two key halves; up to 64: a row block each.
constexpr int kSmallThreads = 160;
constexpr int kBox = 64;  // keys per stage

template <int D>
struct SmallSmem {
  static constexpr int kHalf = kBox * 128;               // 64 columns of a tile, 128 bytes a row
  static constexpr int kKV = kBox * D * 2;               // K or V of a stage
  static constexpr int kStages = 96 * 1024 / (2 * kKV);  // 3 (d = 128) or 6
  static constexpr int offJoin = kStages * 2 * kKV;      // half of four warps' O; first the walker's window sums
  static constexpr int kJoin = 2 * 16 * D * 4;
  static constexpr int offMl = offJoin + kJoin;          // [4 warps][16 rows] m, l
  // Segments on their way: one more than stages, so that the segment whose
  // place is taken has given its last stage back.
  static constexpr int kSegs = kStages + 1;
  static constexpr int offBar = offMl + 4 * 16 * 8;      // full, empty (stages), segment, join, read
  static constexpr int offSeg = offBar + (2 * kStages + kSegs + 2) * 8;
  static constexpr int offMask = offSeg + kSegs * static_cast<int>(sizeof(PagedSegment));  // boxes of the stage that hold keys
  static constexpr int offAbort = offMask + kStages * 4;
  static constexpr int kBytes = offAbort + 4;
};
static_assert(2 * (SmallSmem<128>::kBytes + 1024) <= 228 * 1024, "two CTAs an SM");
static_assert(SmallSmem<128>::kJoin >= kMaxEntries / 32 * 8 && SmallSmem<64>::kJoin >= kMaxEntries / 32 * 8, "window sums");

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

template <typename T, int D>
__global__ void __launch_bounds__(kSmallThreads, 2)
    paged_small_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ PagedAttnArgs args, const PagedCut cut, int min_units, int box_rows) {
  using SM = SmallSmem<D>;
  constexpr int NH = D / 64, S = SM::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t s0 = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedGeom& g = args.g;
  int32_t* status = args.status;
  auto full = [&](int i) { return s0 + SM::offBar + 8u * i; };
  auto empty = [&](int i) { return s0 + SM::offBar + 8u * (S + i); };
  auto seg_full = [&](int i) { return s0 + SM::offBar + 8u * (2 * S + i); };
  const uint32_t join_bar = s0 + SM::offBar + 8u * (2 * S + SM::kSegs), read_bar = join_bar + 8;
  PagedSegment* segs = reinterpret_cast<PagedSegment*>(smem + SM::offSeg);
  volatile uint32_t* mask = reinterpret_cast<volatile uint32_t*>(smem + SM::offMask);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SM::offAbort);
  pdl_launch_dependents();
  if (s0 & 1023) {  // the swizzle is a function of the address
    debug_bounds_fail(status, __LINE__, CP_TU_ID);
    pdl_wait();
    return;
  }
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    for (int i = 0; i < S; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), 4);
    }
    for (int i = 0; i < SM::kSegs; ++i) mbar_init(seg_full(i), 1);
    mbar_init(join_bar, 4);
    mbar_init(read_bar, 4);
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  PagedWalker walk(args, cut, kSmallRows, 0);
  const bool any = walk.start(reinterpret_cast<long long*>(smem + SM::offJoin), blockIdx.x, gridDim.x, min_units);
  if (!any) {
    // nothing for this worker
  } else if (warp == 4) {
    // ------------------------------------------------------------ fetch
    // Lane: one box of the tile, one 64-column half, K or V.
    const int boxes = kBox / box_rows;
    const int kv = lane & 1, half = (lane >> 1) % NH, box = (lane >> 1) / NH;
    const bool mine = box < boxes;
    const CUtensorMap* map = kv ? &tm_v : &tm_k;
    const uint32_t dst0 = s0 + kv * SM::kKV + half * SM::kHalf + box * box_rows * 128;
    const int page_mask = (1 << g.page_shift) - 1;
    int n = 0, nseg = 0;
    bool ok = true;
    while (ok) {
      const PagedSegment seg = walk.next();
      if (lane == 0) {
        segs[nseg % SM::kSegs] = seg;
        mbar_arrive(seg_full(nseg % SM::kSegs));
      }
      ++nseg;
      if (seg.nt == 0) break;
      auto page_of = [&](int tile) {
        const int key = tile * kBox + box * box_rows;
        return mine && tile < seg.tile1 && key < seg.keys ? walk.table[key >> g.page_shift] : -2;
      };
      int page = page_of(seg.tile0);
      for (int tile = seg.tile0; tile < seg.tile1; ++tile, ++n) {
        const int ahead = page_of(tile + 1);
        const int st = n % S;
        ok = __all_sync(0xffffffffu, mbar_wait(empty(st), ((n / S) & 1) ^ 1, abort_flag, status));
        if (!ok) break;
        const int key = tile * kBox + box * box_rows;
        bool load = page != -2;
        if (load && !CP_CHECK_DATA(page >= 0 && page < g.num_pages, status)) load = false;
        const uint32_t all = __ballot_sync(0xffffffffu, load);
        if (lane == 0) {
          uint32_t held = 0;
          for (int b = 0; b < boxes; ++b) held |= ((all >> (2 * NH * b)) & 1u) << b;
          mask[st] = held;
          mbar_arrive_expect_tx(full(st), __popc(all) * box_rows * 128);
        }
        __syncwarp();
        if (load) tma_load_4d(dst0 + st * 2 * SM::kKV, map, full(st), half * 64, key & page_mask, seg.h, page);
        page = ahead;
      }
    }
    if (!ok)  // let every copy still in flight land
      for (int i = n < S ? 0 : n - S; i < n; ++i) mbar_wait(full(i % S), (i / S) & 1, nullptr, status);
  } else {
    // ------------------------------------------------------------ compute
    const float sl2 = g.scale * 1.4426950408889634f;
    const uint32_t box_all = (1u << (kBox / box_rows)) - 1;
    const int box_shift = 31 - __clz(box_rows);
    const int qr = lane >> 2, qc = 2 * (lane & 3);  // row and first column of the lane in an MMA fragment
    // ldmatrix rows of the lane: K (16 keys x 16 columns) and V (the same, transposed on the way).
    const int k_row = ((lane >> 4) << 3) + (lane & 7), k_piece = (lane >> 3) & 1;
    const int v_row = (((lane >> 3) & 1) << 3) + (lane & 7), v_piece = lane >> 4;
    float* ml = reinterpret_cast<float*>(smem + SM::offMl);
    float4* join = reinterpret_cast<float4*>(smem + SM::offJoin);
    int n = 0, nseg = 0;
    uint32_t joins = 0, njoin = 0;
    bool ok = true;
    // All four warps here: a bounded wait, unlike a hardware barrier.
    auto join_sync = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(join_bar);
      return __all_sync(0xffffffffu, mbar_wait(join_bar, joins++ & 1, abort_flag, status));
    };
    while (true) {
      ok = __all_sync(0xffffffffu, mbar_wait(seg_full(nseg % SM::kSegs), (nseg / SM::kSegs) & 1, abort_flag, status));
      if (!ok) break;
      const PagedSegment seg = segs[nseg % SM::kSegs];
      ++nseg;
      if (seg.nt == 0) break;
      const int rows = seg.nt * g.G;
      const int nrb = rows <= 16 ? 1 : rows <= 32 ? 2 : 4, nks = 4 / nrb;
      const int rb = warp % nrb, ks = warp / nrb;
      const int r0 = rb * 16 + qr, r1 = r0 + 8;
      const int i0 = r0 / g.G, i1 = r1 / g.G;  // tokens of the lane's two rows
      const int lim0 = r0 < rows ? min(seg.keys, seg.limit0 + i0) : 0;
      const int lim1 = r1 < rows ? min(seg.keys, seg.limit0 + i1) : 0;
      const int lim_all = min(seg.keys, seg.limit0);                  // seen by every row
      const int lim_any = min(seg.keys, seg.limit0 + seg.nt - 1);     // seen by some row
      uint32_t q[D / 16][4];
      {
        const T* p0 = static_cast<const T*>(args.q) + (seg.t0 + i0) * args.q_stride + (seg.h * g.G + r0 - i0 * g.G) * D + qc;
        const T* p1 = static_cast<const T*>(args.q) + (seg.t0 + i1) * args.q_stride + (seg.h * g.G + r1 - i1 * g.G) * D + qc;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          q[k][0] = r0 < rows ? *reinterpret_cast<const uint32_t*>(p0 + k * 16) : 0u;
          q[k][1] = r1 < rows ? *reinterpret_cast<const uint32_t*>(p1 + k * 16) : 0u;
          q[k][2] = r0 < rows ? *reinterpret_cast<const uint32_t*>(p0 + k * 16 + 8) : 0u;
          q[k][3] = r1 < rows ? *reinterpret_cast<const uint32_t*>(p1 + k * 16 + 8) : 0u;
        }
      }
      float o[D / 8][4];
#pragma unroll
      for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

      for (int tile = seg.tile0; tile < seg.tile1; ++tile, ++n) {
        const int st = n % S;
        ok = __all_sync(0xffffffffu, mbar_wait(full(st), (n / S) & 1, abort_flag, status));
        if (!ok) break;
        const uint32_t held = mask[st];
        const bool clean = held == box_all && (tile + 1) * kBox <= lim_all;
        const uint32_t sk = s0 + st * 2 * SM::kKV, sv = sk + SM::kKV;
        for (int sl = ks; sl < 4; sl += nks) {
          const int key0 = tile * kBox + sl * 16;
          if (key0 >= lim_any) break;
          // S = Q K^T for 16 rows x 16 keys, two chains per 8 keys.
          float c[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) c[i][0] = c[i][1] = c[i][2] = c[i][3] = 0.f;
          const int kr = sl * 16 + k_row;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            uint32_t b[4];
            ldmatrix4<false>(b, sk + (k >> 2) * SM::kHalf + kr * 128 + ((((k & 3) * 2 + k_piece) ^ (kr & 7)) << 4));
            mma16816<T>(c[(k & 1) * 2], q[k], b[0], b[1]);
            mma16816<T>(c[(k & 1) * 2 + 1], q[k], b[2], b[3]);
          }
          float x[8];  // row r0: 0, 1, 4, 5; row r1: 2, 3, 6, 7
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = (c[0][i] + c[2][i]) * sl2;
            x[4 + i] = (c[1][i] + c[3][i]) * sl2;
          }
          uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;  // V rows that hold keys, for the lane's two pairs
          if (!clean) {
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const int in = sl * 16 + half * 8 + qc + j, key = tile * kBox + in;
                const bool there = (held >> (in >> box_shift)) & 1u;
                if (!there || key >= lim0) x[half * 4 + j] = -INFINITY;
                if (!there || key >= lim1) x[half * 4 + 2 + j] = -INFINITY;
                // What lies behind the last key may be anything, NaN included: 0 * NaN would reach O.
                if (!there || key >= seg.keys) (half ? keep1 : keep0) &= j ? 0x0000ffffu : 0xffff0000u;
              }
          }
          const float mx0 = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[4], x[5]));
          const float mx1 = fmaxf(fmaxf(x[2], x[3]), fmaxf(x[6], x[7]));
          if (!__all_sync(0xffffffffu, mx0 <= m0 + Weight<T>::kSlack && mx1 <= m1 + Weight<T>::kSlack)) {
            float t0 = mx0, t1 = mx1;
#pragma unroll
            for (int y = 1; y < 4; y <<= 1) {
              t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, y));
              t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, y));
            }
            const float n0 = t0 > m0 + Weight<T>::kSlack ? t0 : m0, n1 = t1 > m1 + Weight<T>::kSlack ? t1 : m1;
            const float a0 = n0 > m0 ? ex2_approx(m0 - n0) : 1.f, a1 = n1 > m1 ? ex2_approx(m1 - n1) : 1.f;
            m0 = n0;
            m1 = n1;
            l0 *= a0;
            l1 *= a1;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
              o[i][0] *= a0;
              o[i][1] *= a0;
              o[i][2] *= a1;
              o[i][3] *= a1;
            }
          }
          const float b0 = Weight<T>::kBias - (m0 == -INFINITY ? 0.f : m0), b1 = Weight<T>::kBias - (m1 == -INFINITY ? 0.f : m1);
          float p[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) p[i] = ex2_approx(x[i] + ((i & 2) ? b1 : b0));
          l0 += (p[0] + p[1]) + (p[4] + p[5]);
          l1 += (p[2] + p[3]) + (p[6] + p[7]);
          // The weights are rounded to the cache's type for the product with V;
          // their sum is not.
          const uint32_t pa[4] = {Elem<T>::pack(p[0], p[1]), Elem<T>::pack(p[2], p[3]), Elem<T>::pack(p[4], p[5]),
                                  Elem<T>::pack(p[6], p[7])};
          const int vr = sl * 16 + v_row;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            uint32_t b[4];
            ldmatrix4<true>(b, sv + (i >> 2) * SM::kHalf + vr * 128 + ((((i & 3) * 2 + v_piece) ^ (vr & 7)) << 4));
            if (!clean) {
              b[0] &= keep0;
              b[1] &= keep1;
              b[2] &= keep0;
              b[3] &= keep1;
            }
            mma16816<T>(o[2 * i], pa, b[0], b[1]);
            mma16816<T>(o[2 * i + 1], pa, b[2], b[3]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty(st));
      }

      if (!ok) break;

      // Join the warps that shared the rows.  Each pair (w, w ^ 2) swaps
      // halves of the columns, then, where four warps share, (w, w ^ 1)
      // quarters, so every warp ends with the whole sum of its share of the
      // columns and all four write.
#pragma unroll
      for (int y = 1; y < 4; y <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, y);
        l1 += __shfl_xor_sync(0xffffffffu, l1, y);
      }
      constexpr int H = D / 16, Q = D / 32;  // 8-column pieces of half and a quarter of a row
      int col = 0, pieces = D / 8;           // the warp's share
      if (nks > 1) {
        const bool upper = warp & 2;
        // The last readers of these places were two joins ago or have passed `read_bar`.
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(read_bar, (njoin & 1) ^ 1, abort_flag, status)))) break;
        if ((lane & 3) == 0) {
          ml[(warp * 16 + qr) * 2] = m0;
          ml[(warp * 16 + qr) * 2 + 1] = l0;
          ml[(warp * 16 + qr + 8) * 2] = m1;
          ml[(warp * 16 + qr + 8) * 2 + 1] = l1;
        }
        float4* give = join + (warp ^ 2) * H * 32 + lane;
        float4* got = join + warp * H * 32 + lane;
#pragma unroll
        for (int i = 0; i < H; ++i)
          give[i * 32] = upper ? make_float4(o[i][0], o[i][1], o[i][2], o[i][3])
                               : make_float4(o[H + i][0], o[H + i][1], o[H + i][2], o[H + i][3]);
        if (!(ok = join_sync())) break;
        float n0 = -INFINITY, n1 = -INFINITY;
        for (int k = 0; k < nks; ++k) {
          const float* x = ml + ((rb + nrb * k) * 16 + qr) * 2;
          n0 = fmaxf(n0, x[0]);
          n1 = fmaxf(n1, x[16]);
        }
        const float z0 = n0 == -INFINITY ? 0.f : n0, z1 = n1 == -INFINITY ? 0.f : n1;
        l0 = l1 = 0.f;
        for (int k = 0; k < nks; ++k) {
          const float* x = ml + ((rb + nrb * k) * 16 + qr) * 2;
          l0 += x[1] * ex2_approx(x[0] - z0);
          l1 += x[17] * ex2_approx(x[16] - z1);
        }
        const float f0 = ex2_approx(m0 - z0), f1 = ex2_approx(m1 - z1);
        const float* x = ml + ((warp ^ 2) * 16 + qr) * 2;
        const float g0 = ex2_approx(x[0] - z0), g1 = ex2_approx(x[16] - z1);
        m0 = n0;
        m1 = n1;
#pragma unroll
        for (int i = 0; i < H; ++i) {
          const float4 y = got[i * 32];
          o[i][0] = (upper ? o[H + i][0] : o[i][0]) * f0 + y.x * g0;
          o[i][1] = (upper ? o[H + i][1] : o[i][1]) * f0 + y.y * g0;
          o[i][2] = (upper ? o[H + i][2] : o[i][2]) * f1 + y.z * g1;
          o[i][3] = (upper ? o[H + i][3] : o[i][3]) * f1 + y.w * g1;
        }
        col = upper ? D / 2 : 0;
        pieces = H;
        if (nks == 4) {
          const bool odd = warp & 1;
          // Over what this warp has just read; only its partner reads it there.
#pragma unroll
          for (int i = 0; i < Q; ++i)
            got[i * 32] = odd ? make_float4(o[i][0], o[i][1], o[i][2], o[i][3])
                              : make_float4(o[Q + i][0], o[Q + i][1], o[Q + i][2], o[Q + i][3]);
          if (!(ok = join_sync())) break;
          const float4* other = join + (warp ^ 1) * H * 32 + lane;
#pragma unroll
          for (int i = 0; i < Q; ++i) {
            const float4 y = other[i * 32];
            o[i][0] = (odd ? o[Q + i][0] : o[i][0]) + y.x;
            o[i][1] = (odd ? o[Q + i][1] : o[i][1]) + y.y;
            o[i][2] = (odd ? o[Q + i][2] : o[i][2]) + y.z;
            o[i][3] = (odd ? o[Q + i][3] : o[i][3]) + y.w;
          }
          col += odd ? D / 4 : 0;
          pieces = Q;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(read_bar);
        ++njoin;
      }
      const bool final_rows = seg.mode == kRowsFinal;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = half ? r1 : r0, i = half ? i1 : i0;
        if (r >= rows) continue;
        const float l = half ? l1 : l0, m = half ? m1 : m0;
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const int token = seg.t0 + i, head = seg.h * g.G + r - i * g.G;
        const long long row = static_cast<long long>(token) * g.Hq + head;
        const long long at = seg.row + (seg.mode == kRowsHome ? row : r);
        if (final_rows && !args.out_fp32) {
          T* dst = static_cast<T*>(args.o) + row * D + col + qc;
#pragma unroll
          for (int j = 0; j < D / 8; ++j)
            if (j < pieces)
              *reinterpret_cast<uint32_t*>(dst + j * 8) = Elem<T>::pack(o[j][2 * half] * inv, o[j][2 * half + 1] * inv);
        } else {
          float* dst = (final_rows ? static_cast<float*>(args.o) + row * D : args.part_o + at * D) + col + qc;
#pragma unroll
          for (int j = 0; j < D / 8; ++j)
            if (j < pieces)
              *reinterpret_cast<float2*>(dst + j * 8) = make_float2(o[j][2 * half] * inv, o[j][2 * half + 1] * inv);
        }
        if (ks == 0 && (lane & 3) == 0) {
          const float lse2 = l > 0.f ? m + log2f(l) - Weight<T>::kBias : -INFINITY;
          if (final_rows)
            args.lse[static_cast<long long>(head) * g.N + token] = lse2 * 0.69314718055994531f;
          else
            args.part_lse[at] = lse2;
        }
      }
    }
  }
  pdl_wait();  // a kernel that waits for this one also waits for those before it
}

// ---------------------------------------------------------------- merge
//
// O = sum_p 2^(lse_p - m) O_p / sum_p 2^(lse_p - m) over a row's parts, its own
// keys' first, then its prefix's, in key order; rows whose only part went
// straight to the output are left alone.  What it reads is in L2 and small, so
// its time is latency: a lane asks for eight parts at once, and with few rows
// (SPLIT) the four warps of a block share the parts of one row.
constexpr int kMergeWarps = 4;
constexpr int kMergeAhead = 8;
constexpr long long kMergeSplitRows = 2048;

template <typename T, int D, bool SPLIT>
__global__ void __launch_bounds__(kMergeWarps * 32) paged_merge_kernel(const __grid_constant__ PagedAttnArgs args) {
  constexpr int E = D / 32;
  using Vec = typename std::conditional<E == 4, float4, float2>::type;
  __shared__ float joint[SPLIT ? kMergeWarps : 1][32][E + 2];
  const PagedGeom& g = args.g;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // SPLIT: a block per (token, query head); else a warp per (token, KV head).
  const long long w = SPLIT ? static_cast<long long>(blockIdx.x) : static_cast<long long>(blockIdx.x) * kMergeWarps + warp;
  const int per_token = SPLIT ? g.Hq : g.Hkv;
  const int t = static_cast<int>(w / per_token), x = static_cast<int>(w % per_token);
  if (t >= g.N) return;
  const int s = warp_count_le(g.q_start + 1, g.B, t);
  if (s >= g.B) return;
  const PagedEntry own = paged_entry(g, s);
  if (own.bad || t < own.t0 || t >= own.t0 + own.n) return;
  const int p = warp_prefix_of(g, s);
  const bool covered = g.NP > 0 && s >= g.prefix_first[0] && s < g.prefix_first[g.NP];  // as PagedWalker has it
  const bool prefix = p >= 0 && paged_entry(g, g.B + p).keys > 0;
  const int hk = SPLIT ? x / g.G : x;
  const PagedParts* parts = args.parts + static_cast<size_t>(t) * g.Hkv + hk;
  PagedParts a{0, 0, 0, 0}, b{0, 0, 0, 0};
  pdl_wait();
  if (min(own.keys, own.limit0 + (t - own.t0)) > 0) a = *parts;
  if (prefix) b = parts[static_cast<size_t>(args.max_tokens) * g.Hkv];
  if (a.count == 1 && !covered) return;
  const int n = a.count + b.count;
  const int sub0 = SPLIT ? x - hk * g.G : 0, sub1 = SPLIT ? sub0 + 1 : g.G;
  for (int sub = sub0; sub < sub1; ++sub) {
    float m = -INFINITY, sum = 0.f, o[E];
#pragma unroll
    for (int j = 0; j < E; ++j) o[j] = 0.f;
    for (int i0 = SPLIT ? warp : 0; i0 < n; i0 += kMergeAhead * (SPLIT ? kMergeWarps : 1)) {
      float lse[kMergeAhead];
      Vec v[kMergeAhead];
#pragma unroll
      for (int k = 0; k < kMergeAhead; ++k) {
        const int i = i0 + k * (SPLIT ? kMergeWarps : 1);
        const bool in_a = i < a.count;
        const int at = in_a ? i : i - a.count;
        const int first = in_a ? a.first : b.first, second = in_a ? a.second : b.second, stride = in_a ? a.stride : b.stride;
        const long long row = (at == 0 ? first : second + (at - 1) * stride) + sub;
        lse[k] = -INFINITY;
        if (i < n) {
          lse[k] = args.part_lse[row];
          v[k] = *reinterpret_cast<const Vec*>(args.part_o + row * D + lane * E);
        }
      }
      float top = m;
#pragma unroll
      for (int k = 0; k < kMergeAhead; ++k) top = fmaxf(top, lse[k]);
      const float z = top == -INFINITY ? 0.f : top;
      const float f = ex2_approx(m - z);
      m = top;
      sum *= f;
#pragma unroll
      for (int j = 0; j < E; ++j) o[j] *= f;
#pragma unroll
      for (int k = 0; k < kMergeAhead; ++k) {
        if (lse[k] == -INFINITY) continue;
        const float wt = ex2_approx(lse[k] - z);
        sum += wt;
        const float* y = reinterpret_cast<const float*>(&v[k]);
#pragma unroll
        for (int j = 0; j < E; ++j) o[j] = fmaf(wt, y[j], o[j]);
      }
    }
    if constexpr (SPLIT) {
#pragma unroll
      for (int j = 0; j < E; ++j) joint[warp][lane][j] = o[j];
      joint[warp][lane][E] = m;
      joint[warp][lane][E + 1] = sum;
      __syncthreads();
      if (warp > 0) return;
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < kMergeWarps; ++k) top = fmaxf(top, joint[k][lane][E]);
      const float z = top == -INFINITY ? 0.f : top;
      m = top;
      sum = 0.f;
#pragma unroll
      for (int j = 0; j < E; ++j) o[j] = 0.f;
#pragma unroll
      for (int k = 0; k < kMergeWarps; ++k) {
        const float f = ex2_approx(joint[k][lane][E] - z);
        sum = fmaf(f, joint[k][lane][E + 1], sum);
#pragma unroll
        for (int j = 0; j < E; ++j) o[j] = fmaf(f, joint[k][lane][j], o[j]);
      }
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    const int h = hk * g.G + sub;
    const long long at = (static_cast<long long>(t) * g.Hq + h) * D + lane * E;
    if (args.out_fp32) {
      float* dst = static_cast<float*>(args.o) + at;
#pragma unroll
      for (int j = 0; j < E; ++j) dst[j] = o[j] * inv;
    } else {
      uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<T*>(args.o) + at);
#pragma unroll
      for (int j = 0; j < E / 2; ++j) dst[j] = Elem<T>::pack(o[2 * j] * inv, o[2 * j + 1] * inv);
    }
    if (lane == 0)
      args.lse[static_cast<long long>(h) * g.N + t] = sum > 0.f ? (m + log2f(sum)) * 0.69314718055994531f : -INFINITY;
  }
}

// ---------------------------------------------------------------- launch

template <typename T, int D>
int launch_attn_d(const PagedAttnArgs& a, cudaStream_t stream) {
  const PagedGeom& g = a.g;
  static std::atomic<int> small_known[64];
  int sms = 0;
  int rc = prepare_kernel(small_known, paged_small_kernel<T, D>, SmallSmem<D>::kBytes, &sms);
  if (rc != CP_OK) return rc;
  const int page = 1 << g.page_shift, box = page < kBox ? page : kBox;
  CUtensorMap mk, mv;
  if (!make_cache_map(&mk, g, a.k_cache, box) || !make_cache_map(&mv, g, a.v_cache, box)) return CP_ERR_CUDA;
  const int workers = 2 * sms < kSmallWorkers ? 2 * sms : kSmallWorkers;
  // Whether an entry may have more rows than this kernel takes.
  const long long most = static_cast<long long>(g.NP > 0 || g.N < g.max_new ? g.N : g.max_new) * g.G;
  const bool large = most > kSmallRows;
  if (large && (rc = launch_paged_large(a, stream)) != CP_OK) return rc;
  rc = launch(paged_small_kernel<T, D>, workers, kSmallThreads, SmallSmem<D>::kBytes, large, stream, mk, mv, a,
              paged_cut_small(g.G), 1, box);
  if (rc != CP_OK) return rc;
  const long long rows = static_cast<long long>(g.N) * g.Hq;
  if (rows <= kMergeSplitRows)
    return launch(paged_merge_kernel<T, D, true>, static_cast<unsigned>(rows), kMergeWarps * 32, 0, true, stream, a);
  const long long warps = static_cast<long long>(g.N) * g.Hkv;
  return launch(paged_merge_kernel<T, D, false>, static_cast<unsigned>((warps + kMergeWarps - 1) / kMergeWarps),
                kMergeWarps * 32, 0, true, stream, a);
}

}  // namespace

int launch_paged_attn(const PagedAttnArgs& a, cudaStream_t stream) {
  const bool bf16 = a.g.dtype == CP_DTYPE_BF16;
  if (a.g.d == 128) return bf16 ? launch_attn_d<__nv_bfloat16, 128>(a, stream) : launch_attn_d<__half, 128>(a, stream);
  if (a.g.d == 64) return bf16 ? launch_attn_d<__nv_bfloat16, 64>(a, stream) : launch_attn_d<__half, 64>(a, stream);
  return CP_ERR_UNSUPPORTED;
}

}  // namespace cpattn
