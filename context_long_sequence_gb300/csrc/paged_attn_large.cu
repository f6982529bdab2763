// paged_attn_large.cu -- attention over the paged cache for batches with
// entries of many rows: a prefix with the rows of all its sequences, or a
// sequence with a chunk of new tokens.
//
// Rows are (token, query head of the KV head) pairs, token by token; a token
// tile holds two blocks of up to 128 rows, whole tokens each, that share
// every K and V tile.  Per 128-key tile, as in the forward over whole
// sequences (attn_fwd.cu):
//
//   S_t = Q_t K^T        tcgen05.mma, operands in shared memory, S in TMEM
//   online softmax       one thread per row; P_t packed back over S_t, rounded
//                        once to the cache's type (its sum is not): what is left
//                        over as a second operand (split_weights in
//                        paged_small.cuh) would make three products of two, and
//                        the tensor core is the bound here
//   O_t += P_t V         tcgen05.mma with A read from TMEM
//
// and the two row blocks ping-pong on the tensor core (issue order QK_0,
// PV_1 of the tile before, QK_1, PV_0).  Unlike there, a CTA is one of 152
// workers that each walk an equal share of the batch's units (PagedCut): a
// batch has few token tiles and many keys, so the keys are what is shared
// out, and the runs' (O, LSE) are merged.  K and V come page by page.
//
// At 256 rows a 128-key tile is 256 flops a byte, the card's own balance:
// fewer rows are bound by the cache's bytes, more by the tensor core.  A tile
// of 256 rows takes 2750 clocks, 2165 of them the MMAs'.  Measured (32 query
// heads on 8, d = 128): chunks of up to 2K tokens after up to 14K keys, 569
// GFLOP in 382 us, 1.49 PFLOP/s (tensor pipe 66 % active; the rest is the
// softmax's share of a tile and the change from one segment to the next); 64
// sequences on a prefix of 32K keys, 274 MB and 35 GFLOP in 52 us of the
// kernel's own, 59 with the merge: the first tile's rows are done 11 us in (the
// shares 3, the segment 2, Q, K and S 4, its exponentials 2, all of them code
// that comes from L2 once), and tiles follow every 1.4 us.
//
// Rows leave through shared memory: as TMA boxes of 32 rows where they lie
// together, else as lines of 128 bytes (256 sequences on prefixes 98.8 us with
// lines alone, 95.3 with boxes).
//
// A batch's entries of few rows are taken by other CTAs of the same launch
// (paged_small.cuh, eight workers a CTA), in proportion to their work
// (paged_large_ctas): work bound by the tensor core and work bound by the
// cache's bytes share the card better side by side than one after the other.
//
// Warps (320 threads): 0 fetches, 1 issues the MMAs (and holds the TMEM),
// 2..5 and 6..9 load Q, take the softmax and write the rows of block 0 and 1.
#include <cuda.h>
#include <cuda_runtime.h>

#define CP_TU_ID ::cpattn::kTuPagedAttn
#include "paged.cuh"
#include "paged_small.cuh"

namespace cpattn {
namespace {

constexpr int BM = 128, BN = 128;
constexpr uint32_t HALF_BYTES = 128 * 128;  // one 64-column swizzled half of a 128-row tile
constexpr int kThreads = 320;
constexpr int kSlots = 5;      // K/V ring: K of key tile j is load 2j, V load 2j + 1
constexpr int kTileBars = 3;   // key tiles in flight at most

enum Bar {
  BAR_Q = 0,                             // both blocks' Q written (8 warps)
  BAR_T_FULL = 1,                        // +key tile % kTileBars: its K and V landed
  BAR_KV_EMPTY = 1 + kTileBars,          // +slot
  BAR_S_FULL = 1 + kTileBars + kSlots,   // +block
  BAR_P_HALF = 3 + kTileBars + kSlots,   // +block: P of keys 0-63 written
  BAR_P_FULL = 5 + kTileBars + kSlots,   // +block
  BAR_O = 7 + kTileBars + kSlots,        // +block: every MMA of the segment's block completed
  BAR_SEG = 9 + kTileBars + kSlots,      // +segment % kSegs: handed over
  NUM_BARS = 9 + kTileBars + kSlots + 4
};
// Segments on their way.  A tile's slots are those of the tile three before it
// (5 slots, 2 a tile), so a segment four back has given its last tile back,
// and everybody has read it: its MMAs waited for all row warps' Q.
constexpr int kSegs = 4;

template <int D>
struct LargeSmem {
  static constexpr uint32_t kQ = BM * D * 2;
  static constexpr uint32_t kKV = BN * D * 2;
  static constexpr uint32_t offKV = 2 * kQ;
  static constexpr uint32_t offBar = offKV + kSlots * kKV;
  static constexpr uint32_t offMisc = offBar + NUM_BARS * 8;  // TMEM address, abort flag, box masks
  static constexpr uint32_t offSeg = offMisc + 8 + kTileBars * 4;
  static constexpr uint32_t kUsed = offSeg + kSegs * sizeof(PagedSegment);
  // D = 64 is padded so that one CTA (and its 512 TMEM columns) is on an SM.
  static constexpr uint32_t kBytes = kUsed < 120 * 1024 ? 120 * 1024 : kUsed;
};

__device__ __forceinline__ bool warp_all(bool x) { return __all_sync(0xffffffffu, x); }

// kind::f16 instruction descriptor: fp32 accumulator, A and B both T.
template <typename T>
constexpr uint32_t idesc(int n, int b_mn_major) {
  const uint32_t d = idesc_bf16_f32(BM, n, b_mn_major);
  return sizeof(T) == 2 && Weight<T>::kBias > 0.f ? d & ~((1u << 7) | (1u << 10)) : d;
}

// A row block's view of the keys: its first row sees keys below lo, its last
// those below hi; hi == 0: no rows.
struct RowBlock {
  int lo, hi;
  __device__ __forceinline__ bool sees(int key0) const { return key0 < hi; }
};
__device__ __forceinline__ RowBlock row_block(const PagedSegment& s, int t, int tokens) {
  const int first = t * tokens, n = min(tokens, s.nt - first);
  if (n <= 0) return RowBlock{0, 0};
  return RowBlock{min(s.keys, s.limit0 + first), min(s.keys, s.limit0 + first + n - 1)};
}

template <int D>
constexpr uint32_t kLaunchBytes =
    LargeSmem<D>::kBytes > SmallSmem<D>::kBytes ? LargeSmem<D>::kBytes : static_cast<uint32_t>(SmallSmem<D>::kBytes);
static_assert(kLaunchBytes<128> <= 227 * 1024, "one CTA an SM");

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_large_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ CUtensorMap tm_k16, const __grid_constant__ CUtensorMap tm_v16,
                       const __grid_constant__ CUtensorMap tm_part, const __grid_constant__ CUtensorMap tm_o,
                       const __grid_constant__ PagedAttnArgs args, int box_rows, int o_boxes) {
  using SM = LargeSmem<D>;
  constexpr int NH = D / 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t s0 = smem_u32(smem), sQ = s0, sKV = s0 + SM::offKV;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedGeom& g = args.g;
  int32_t* status = args.status;
  auto bar = [&](int i) { return s0 + SM::offBar + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM::offMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SM::offMisc + 4);
  volatile uint32_t* mask = reinterpret_cast<volatile uint32_t*>(smem + SM::offMisc + 8);
  if (threadIdx.x == kThreads - 32) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_k16);
    tma_prefetch_desc(&tm_v16);
  }
  pdl_wait();
  pdl_launch_dependents();
  if (s0 & 1023) {  // the swizzle is a function of the address
    debug_bounds_fail(status, __LINE__, CP_TU_ID);
    return;
  }
  PagedSegment* segs = reinterpret_cast<PagedSegment*>(smem + SM::offSeg);
  const PagedCut cuts[2] = {paged_cut_small(g.G, kBesideRows), paged_cut_large(g.G)};
  PagedWalker<kUnitSums> walk(args, cuts);
  int large = 0;  // CTAs that take the entries of many rows
  const auto role = [&](const long long (&units)[kUnitSums]) {
    const int ctas = gridDim.x, b = blockIdx.x;
    const bool light = paged_is_light(units[kUnitsLight], ctas);
    if (!light) large = paged_large_ctas(units[kUnitsBeside], units[kUnitsLarge], ctas);
    return b < large ? PagedRole{kUnitsLarge, 1, b, large, 1, static_cast<int>(args.rows_small), kLargeRows}
                     : PagedRole{light ? kUnitsLight : kUnitsBeside, 0, warp * (ctas - large) + b - large,
                                 kSmallWarps * (ctas - large), kSmallMinUnits, 0, kSmallRows};
  };
  // The sums lie behind the small workers' stages, and where V will be for the large.
  const bool any = walk.start(reinterpret_cast<long long*>(smem + SmallSmem<D>::offSums), kThreads / 32, role);
  if (static_cast<int>(blockIdx.x) >= large) {
    // Entries of few rows: a warp each, eight of the ten.
    if (warp < kSmallWarps && any) {
      if (lane == 0) small_init<D>(smem, warp);
      __syncwarp();
      small_worker<SmallColumns<T, D>, D>(smem, warp, tm_k16, tm_v16, walk);
    }
    return;
  }
  if (!any) return;  // the whole block
  const int block_tokens = cuts[1].tile_tokens / 2;
  const uint32_t box_all = 0xffffffffu >> (32 - 2 * NH * (BN / box_rows));  // every box of a tile held

  if (threadIdx.x == 0) {
    mbar_init(bar(BAR_Q), 8);
    for (int i = 0; i < kTileBars; ++i) mbar_init(bar(BAR_T_FULL + i), 1);
    for (int i = 0; i < kSlots; ++i) mbar_init(bar(BAR_KV_EMPTY + i), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(BAR_S_FULL + i), 1);
      mbar_init(bar(BAR_P_HALF + i), 4);
      mbar_init(bar(BAR_P_FULL + i), 4);
      mbar_init(bar(BAR_O + i), 1);
    }
    for (int i = 0; i < kSegs; ++i) mbar_init(bar(BAR_SEG + i), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  fence_proxy_async_smem();  // the sums were read before the first copy lands on them
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;  // S_t at 128 t (P_t packed in its first 64 columns), O_t at 256 + D t
  // Segment number n, once handed over.
  auto take = [&](int n, PagedSegment& seg) {
    if (!warp_all(mbar_wait_short(bar(BAR_SEG + n % kSegs), (n / kSegs) & 1, abort_flag, status))) return false;
    seg = segs[n % kSegs];
    return seg.nt > 0;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ fetch
    // Lane: one box of the tile, one 64-column half, K or V (at most 8 x 2 x 2).
    const int boxes = BN / box_rows;
    const int kv = lane & 1, half = (lane >> 1) % NH, box = (lane >> 1) / NH;
    const bool mine = box < boxes;
    const CUtensorMap* map = kv ? &tm_v : &tm_k;
    const uint32_t dst0 = sKV + half * HALF_BYTES + box * box_rows * 128;
    const int page_mask = (1 << g.page_shift) - 1;
    int nt = 0, nseg = 0;  // key tiles fetched, segments handed over
    bool ok = true;
    while (ok) {
      const PagedSegment seg = walk.next();
      if (lane == 0) {
        segs[nseg % kSegs] = seg;
        mbar_arrive(bar(BAR_SEG + nseg % kSegs));
      }
      ++nseg;
      if (seg.nt == 0) break;
      const uint64_t policy = walk.once ? read_once_policy() : read_again_policy();
      // Whether the lane has a box of the tile, and the page that it is in: any
      // number, as it stands in the table.
      auto wants = [&](int tile) { return mine && tile < seg.tile1 && tile * BN + box * box_rows < seg.keys; };
      auto page_of = [&](int tile) {
        return wants(tile) ? walk.table[(tile * BN + box * box_rows) >> g.page_shift] : 0;
      };
      int page = page_of(seg.tile0);
      for (int tile = seg.tile0; tile < seg.tile1; ++tile, ++nt) {
        const int ahead = page_of(tile + 1);
        const int n = 2 * nt, slk = n % kSlots, slv = (n + 1) % kSlots;
        ok = warp_all(mbar_wait_short(bar(BAR_KV_EMPTY + slk), ((n / kSlots) & 1) ^ 1, abort_flag, status) &&
                      mbar_wait_short(bar(BAR_KV_EMPTY + slv), (((n + 1) / kSlots) & 1) ^ 1, abort_flag, status));
        if (!ok) break;
        const uint32_t tb = bar(BAR_T_FULL + nt % kTileBars);
        bool load = wants(tile);
        if (load && !CP_CHECK_DATA(page >= 0 && page < g.num_pages, status)) load = false;
        const uint32_t all = __ballot_sync(0xffffffffu, load);
        if (lane == 0) {
          mask[nt % kTileBars] = all;  // 2 NH bits a box
          mbar_arrive_expect_tx(tb, __popc(all) * box_rows * 128);
        }
        __syncwarp();
        const int key = tile * BN + box * box_rows;
        (void)CP_IN_BOUNDS(!load || cache_box_in(g, key & page_mask, box_rows, seg.h, page), status);
        if (load) tma_load_4d(dst0 + (kv ? slv : slk) * SM::kKV, map, tb, half * 64, key & page_mask, seg.h, page, policy);
        page = ahead;
      }
    }
    if (!ok)  // let every copy still in flight land
      for (int i = max(0, nt - kTileBars); i < nt; ++i)
        mbar_wait(bar(BAR_T_FULL + i % kTileBars), (i / kTileBars) & 1, nullptr, status);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issue
    constexpr uint32_t idesc_qk = idesc<T>(BN, 0), idesc_pv = idesc<T>(D, 1);
    const uint64_t dq0 = smem_desc_sw128(sQ, 16, 1024), dq1 = smem_desc_sw128(sQ + SM::kQ, 16, 1024);
    const uint64_t dk0 = smem_desc_sw128(sKV, 16, 1024);          // slot 0 read as K (K-major)
    const uint64_t dv0 = smem_desc_sw128(sKV, HALF_BYTES, 1024);  // slot 0 read as V (MN-major)
    constexpr uint64_t kSlotStep = SM::kKV >> 4;
    int npv[2] = {0, 0};   // PVs issued per block, over all segments
    bool fresh[2] = {true, true};  // the segment's first PV overwrites O
    auto issue_qk = [&](int t, int slot) {
      const uint64_t a0 = t ? dq1 : dq0, b0 = dk0 + static_cast<uint64_t>(slot) * kSlotStep;
      if constexpr (D == 128)
        mma_bf16_ss_k128_warp<HALF_BYTES>(tmem + 128 * t, a0, b0, idesc_qk, 0u);
      else
        mma_bf16_ss_k64_warp(tmem + 128 * t, a0, b0, idesc_qk, 0u);
      mma_commit_warp(bar(BAR_S_FULL + t));
    };
    auto issue_pv = [&](int t, int sl, bool release_v) -> bool {
      if (!warp_all(mbar_wait_short(bar(BAR_P_HALF + t), npv[t] & 1, abort_flag, status))) return false;
      tc_fence_after();
      const uint64_t b0 = dv0 + static_cast<uint64_t>(sl) * kSlotStep;
      mma_bf16_ts_k64_warp(tmem + 256 + D * t, tmem + 128 * t, b0, idesc_pv, fresh[t] ? 0u : 1u);
      if (!warp_all(mbar_wait_short(bar(BAR_P_FULL + t), npv[t] & 1, abort_flag, status))) return false;
      tc_fence_after();
      mma_bf16_ts_k64_warp(tmem + 256 + D * t, tmem + 128 * t + 32, b0 + 512, idesc_pv, 1u);
      if (release_v) mma_commit_warp(bar(BAR_KV_EMPTY + sl));
      fresh[t] = false;
      ++npv[t];
      return true;
    };
    int j = 0, ring = 0, nseg = 0;  // key tiles walked, slot of the next K, segments
    bool ok = true;
    PagedSegment seg;
    while (ok && take(nseg, seg)) {
      const RowBlock b0 = row_block(seg, 0, block_tokens), b1 = row_block(seg, 1, block_tokens);
      fresh[0] = fresh[1] = true;
      int pend = -1;  // V slot of a PV_1 still to issue
      ok = warp_all(mbar_wait_short(bar(BAR_Q), nseg & 1, abort_flag, status));
      for (int tile = seg.tile0; ok && tile < seg.tile1; ++tile, ++j) {
        const bool v0 = b0.sees(tile * BN), v1 = b1.sees(tile * BN);
        const int kslot = ring, vslot = ring + 1 == kSlots ? 0 : ring + 1;
        ring = vslot + 1 == kSlots ? 0 : vslot + 1;
        ok = warp_all(mbar_wait_short(bar(BAR_T_FULL + j % kTileBars), (j / kTileBars) & 1, abort_flag, status));
        if (!ok) break;
        tc_fence_after();
        if (v0) issue_qk(0, kslot);
        if (pend >= 0) {
          if (!(ok = issue_pv(1, pend, true))) break;
          pend = -1;
        }
        if (v1) issue_qk(1, kslot);
        mma_commit_warp(bar(BAR_KV_EMPTY + kslot));
        if (v0 && !(ok = issue_pv(0, vslot, !v1))) break;
        if (v1) pend = vslot;
      }
      mma_commit_warp(bar(BAR_O));  // block 0's rows are written while block 1's last PV runs
      if (ok && pend >= 0) ok = issue_pv(1, pend, true);
      mma_commit_warp(bar(BAR_O + 1));
      ++nseg;
    }
    // Every MMA issued has completed before TMEM and shared memory are
    // released: the last commit tracks them all.
    if (nseg > 0) mbar_wait(bar(BAR_O + 1), (nseg - 1) & 1, nullptr, status);
  } else {
    // ------------------------------------------------------------ rows
    // A warp loads, exponentiates and writes 32 rows; one without rows only
    // keeps the barriers going (its lanes of S, P and O hold anything: rows do
    // not mix).  Loops that run once a segment are kept short rather than
    // unrolled: cold code costs some 10 clocks an instruction here.
    const int t = (warp - 2) >> 2;  // row block
    const int wq = warp & 3, row = wq * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tSt = tmem + 128 * t + lane_off, tOt = tmem + 256 + D * t + lane_off;
    const uint32_t sW = sQ + t * SM::kQ + wq * 32 * 128;  // the warp's rows of Q, first half; then its staging
    const float sl2 = g.scale * 1.4426950408889634f;
    constexpr float kBias = Weight<T>::kBias;
    const int tok = row / g.G;  // token of the block's, and query head within the KV head's
    const int sub = row - tok * g.G;
    const int box_shift = 31 - __clz(box_rows);
    int j = 0, k = 0, nseg = 0;  // key tiles walked, seen, segments
    bool ok = true;
    PagedSegment seg;
    while (ok && take(nseg, seg)) {
      const RowBlock w = row_block(seg, t, block_tokens);
      const int first = t * block_tokens;
      const int n_rows = max(0, min(block_tokens, seg.nt - first)) * g.G;
      const bool row_valid = row < n_rows, busy = wq * 32 < n_rows;
      const int my_lim = row_valid ? min(seg.keys, seg.limit0 + first + tok) : 0;
      // Row of (token, head) from the tile's first token on.
      const int my_off = tok * g.Hq + sub;
      const long long tile_row = (static_cast<long long>(seg.t0) + first) * g.Hq + seg.h * g.G;
      if (busy) {
        // Q: 16 bytes a lane and step; a row's pieces side by side.
        constexpr int P = D / 8;  // pieces of a row
        const int piece = lane % P;
        const T* q0 = static_cast<const T*>(args.q) + (static_cast<long long>(seg.t0) + first) * args.q_stride +
                      static_cast<long long>(seg.h) * g.G * D + piece * 8;
        const uint32_t dst = sW + (piece >> 3) * HALF_BYTES;
        const int mine = min(32, n_rows - wq * 32);
        // Straight to shared memory, every row's copy in flight at once.
#pragma unroll 4
        for (int n = 0; n < P; ++n) {
          const int r = n * (32 / P) + lane / P;
          const int i = __shfl_sync(0xffffffffu, tok, r), h = __shfl_sync(0xffffffffu, sub, r);
          if (r < mine && CP_IN_BOUNDS(token_in(g, seg.t0 + first + i, seg.h * g.G + h), status))
            cp_async16(dst + r * 128 + (((piece & 7) ^ (r & 7)) << 4), q0 + i * args.q_stride + h * D);
        }
        cp_async_wait_all();
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_Q));
      float m = -INFINITY, l = 0.f;
      const int k0 = k;
      for (int tile = seg.tile0; ok && tile < seg.tile1; ++tile, ++j) {
        const int key0 = tile * BN;
        if (!w.sees(key0)) continue;
        // K, V and the box mask of the tile are visible through the tile's barrier.
        ok = warp_all(mbar_wait_short(bar(BAR_T_FULL + j % kTileBars), (j / kTileBars) & 1, abort_flag, status) &&
                      mbar_wait_short(bar(BAR_S_FULL + t), k & 1, abort_flag, status));
        if (!ok) break;
        tc_fence_after();
        const uint32_t held = mask[j % kTileBars];
        const bool full = held == box_all && key0 + BN <= w.lo;
        auto signal = [&](int b) {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(b + t));
        };
        if (held != box_all || key0 + BN > seg.keys) {
          // V rows behind the last key (or in a page that was not fetched) may
          // hold anything, NaN included; a zero weight does not remove a NaN.
          if (!((held >> ((row >> box_shift) * 2 * NH)) & 1u) || key0 + row >= seg.keys) {
            const uint32_t v = sKV + ((2 * j + 1) % kSlots) * SM::kKV + row * 128;
#pragma unroll 1
            for (int b = 0; b < 8 * NH; ++b) st_shared_v4(v + (b >> 3) * HALF_BYTES + (b & 7) * 16, 0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        if (!busy) {
          signal(BAR_P_HALF);
          signal(BAR_P_FULL);
          ++k;
          continue;
        }
        // A tile that all rows see whole is exponentiated against the running
        // maximum m before its own is taken: the sum of keys 0-63 bounds each
        // of them, and the maximum of keys 64-127 (found while those
        // exponentials run) the rest.  `exact`: m is raised first -- on a
        // segment's first tile, on masked ones, and where the bounds fail.
        // Both ways share the exponentials' code, whose first pass through the
        // instruction caches costs as much as five tiles.
        bool exact = !(full && warp_all(m != -INFINITY || !row_valid));
        float alpha = 1.f;
        while (true) {
          if (exact) {
            float mx = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < BN / 32; ++c) {
              uint32_t r[32];
              tmem_ld32(tSt + c * 32, r);
              tmem_wait_ld();
              reg_fence(r);
              if (!full) {
                // Hidden keys become -inf in S.  Boxes are 16 keys or more:
                // two bits cover 32 columns.
                const uint32_t in0 = (held >> (((c * 32) >> box_shift) * 2 * NH)) & 1u, in1 = (held >> (((c * 32 + 16) >> box_shift) * 2 * NH)) & 1u;
                const int left = my_lim - key0 - c * 32;
                const int n0 = in0 ? left : 0, n1 = in1 ? left : 0;
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (e >= (e < 16 ? n0 : n1)) r[e] = 0xff800000u;
                tmem_st32(tSt + c * 32, r);
              }
              float m4[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) m4[i] = __uint_as_float(r[i]);
#pragma unroll
              for (int e = 4; e < 32; e += 4)
#pragma unroll
                for (int i = 0; i < 4; ++i) m4[i] = fmaxf(m4[i], __uint_as_float(r[e + i]));
              mx = fmax3(mx, fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
            }
            tmem_wait_st();
            const float m_new = fmaxf(m, mx * sl2);
            if (m_new > m + Weight<T>::kSlack) {
              alpha = ex2_approx(m - m_new);
              m = m_new;
            }
            // O is stable here: this tile's S came after the PV before it.
            if (k > k0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t ov[32];
                tmem_ld32(tOt + c * 32, ov);
                tmem_wait_ld();
                reg_fence(ov);
#pragma unroll
                for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                tmem_st32(tOt + c * 32, ov);
              }
            }
          }
          uint32_t sr[BN];
          float* x = reinterpret_cast<float*>(sr);
          auto col32 = [&](int c) -> uint32_t(&)[32] { return *reinterpret_cast<uint32_t(*)[32]>(&sr[c * 32]); };
          const f32x2 sl2x2 = make_f32x2(sl2, sl2), zero2 = make_f32x2(0.f, 0.f);
          const float off = kBias - (m == -INFINITY ? 0.f : m);
          auto exp32 = [&](int c, f32x2 (&rs2)[4], uint32_t (&pk)[16]) {
            const f32x2 off2 = make_f32x2(off, off);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float a0, a1;
              split_f32x2(fma_f32x2(make_f32x2(x[c * 32 + e], x[c * 32 + e + 1]), sl2x2, off2), a0, a1);
              const float p0 = ex2_approx(a0), p1 = ex2_approx(a1);
              rs2[(e >> 1) & 3] = add_f32x2(rs2[(e >> 1) & 3], make_f32x2(p0, p1));
              pk[e >> 1] = Elem<T>::pack(p0, p1);
            }
          };
          auto sum4 = [](const f32x2 (&rs2)[4]) {
            float lo[4], hi[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) split_f32x2(rs2[i], lo[i], hi[i]);
            return ((lo[0] + hi[0]) + (lo[1] + hi[1])) + ((lo[2] + hi[2]) + (lo[3] + hi[3]));
          };
          tmem_ld32(tSt, col32(0));
          tmem_ld32(tSt + 32, col32(1));
          tmem_wait_ld();
          reg_fence(col32(0));
          reg_fence(col32(1));
          tmem_ld32(tSt + 64, col32(2));  // in flight while keys 0-63 are exponentiated
          tmem_ld32(tSt + 96, col32(3));
          f32x2 rs2[4] = {zero2, zero2, zero2, zero2};
          uint32_t pk0[16], pk1[16];
          exp32(0, rs2, pk0);
          exp32(1, rs2, pk1);
          tmem_wait_ld();
          reg_fence(col32(2));
          reg_fence(col32(3));
          float m4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) m4[i] = fmaxf(x[64 + i], x[68 + i]);
#pragma unroll
          for (int e = 72; e < BN; e += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i) m4[i] = fmax3(m4[i], x[e + i], x[e + 4 + i]);
          const float mx_hi = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          const float s_lo = sum4(rs2);
          if (!exact && !warp_all((s_lo < Weight<T>::kSpecSum && mx_hi * sl2 < m + Weight<T>::kSpecMax) || !row_valid)) {
            exact = true;  // S is as it was
            continue;
          }
          tmem_st16(tSt, pk0);
          tmem_st16(tSt + 16, pk1);
          signal(BAR_P_HALF);
          f32x2 rh[4] = {zero2, zero2, zero2, zero2};
          exp32(2, rh, pk0);
          tmem_st16(tSt + 32, pk0);
          exp32(3, rh, pk1);
          tmem_st16(tSt + 48, pk1);
          signal(BAR_P_FULL);
          l = l * alpha + (s_lo + sum4(rh));
          ++k;
          break;
        }
      }
      // The block's MMAs of this segment have completed: O is whole, and Q's
      // shared memory free for staging and for the next segment.
      if (ok) ok = warp_all(mbar_wait_short(bar(BAR_O + t), nseg & 1, abort_flag, status));
      ++nseg;
      if (!ok) break;
      if (!busy) continue;
      tc_fence_after();
      const bool final_rows = seg.mode == kRowsFinal;
      const float inv = l != 0.f ? __fdividef(1.f, l) : 0.f;
      // A thread holds a row, but rows leave as whole lines: 128 bytes of 32
      // rows at a time pass through shared memory (16-byte pieces, swizzled).
      const bool narrow = final_rows && !args.out_fp32;  // 64 columns are 128 bytes, else 32
      const int lines = narrow ? D / 64 : D / 32;
      char* base;
      int my_line;  // the row's number from base on
      if (seg.mode == kRowsSlot) {
        base = reinterpret_cast<char*>(args.part_o + (seg.row + first * static_cast<long long>(g.G)) * D);
        my_line = row;
      } else {
        base = final_rows ? static_cast<char*>(args.o) + tile_row * D * (narrow ? 2 : 4)
                          : reinterpret_cast<char*>(args.part_o + (seg.row + tile_row) * D);
        my_line = my_off;
      }
      const int row_bytes = D * (narrow ? 2 : 4);
      const int mine = min(32, n_rows - wq * 32);
      // 32 rows that lie together (a slot's; or whole tokens' heads of o) go as
      // TMA boxes, others as lines of 128 bytes by plain stores.
      const bool boxes = mine == 32 && (seg.mode == kRowsSlot || (narrow && o_boxes));
#pragma unroll 1
      for (int c = 0; c < lines; ++c) {
        const uint32_t stage = sW + (NH > 1 ? (c & 1) * HALF_BYTES : 0);
        const uint32_t my_stage = stage + lane * 128;
        if (boxes && c >= NH) {  // the box before has left this place
          if (lane == 0) bulk_wait_read<NH - 1>();
          __syncwarp();
        }
        uint32_t ov[32];
        auto fetch = [&](int col) {
          if (k > k0) {
            tmem_ld32(tOt + col, ov);
            tmem_wait_ld();
            reg_fence(ov);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] = k > k0 ? __float_as_uint(__uint_as_float(ov[e]) * inv) : 0u;
        };
        if (narrow) {
#pragma unroll 1
          for (int hh = 0; hh < 2; ++hh) {
            fetch(c * 64 + hh * 32);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              auto two = [&](int e) { return Elem<T>::pack(__uint_as_float(ov[e]), __uint_as_float(ov[e + 1])); };
              st_shared_v4(my_stage + (((hh * 4 + p) ^ (lane & 7)) << 4), two(8 * p), two(8 * p + 2), two(8 * p + 4), two(8 * p + 6));
            }
          }
        } else {
          fetch(c * 32);
#pragma unroll
          for (int p = 0; p < 8; ++p)
            st_shared_v4(my_stage + ((p ^ (lane & 7)) << 4), ov[4 * p], ov[4 * p + 1], ov[4 * p + 2], ov[4 * p + 3]);
        }
        if (boxes) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            const int slot_row = seg.row + first * g.G + wq * 32, token = seg.t0 + first + wq * 32 / g.G;
            if (seg.mode == kRowsSlot) {
              if (CP_IN_BOUNDS(slot_row >= args.rows_small && slot_row + 32 <= args.rows_large_end, status))
                tma_store_2d(&tm_part, stage, c * 32, slot_row);
            } else if (CP_IN_BOUNDS(token_in(g, token, seg.h * g.G) && token_in(g, token + 32 / g.G - 1, seg.h * g.G + g.G - 1), status)) {
              tma_store_3d(&tm_o, stage, c * 64, seg.h * g.G, token);
            }
            bulk_commit();
          }
          continue;
        }
        __syncwarp();
        uint4 y[8];
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const int r = n * 4 + (lane >> 3), p = lane & 7;
          y[n] = ld_shared_v4(stage + r * 128 + ((p ^ (r & 7)) << 4));
        }
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const int r = n * 4 + (lane >> 3), p = lane & 7;
          const int line = __shfl_sync(0xffffffffu, my_line, r);
          if (r < mine && CP_IN_BOUNDS(final_rows ? tile_row + line < static_cast<long long>(g.N) * g.Hq
                                       : part_rows_in(args, seg.row + (seg.mode == kRowsHome ? tile_row : first * g.G) + line, 1), status))
            *reinterpret_cast<uint4*>(base + static_cast<long long>(line) * row_bytes + c * 128 + p * 16) = y[n];
        }
        if (NH == 1) __syncwarp();  // one staging place; with two, the step between orders them
      }
      if (boxes && lane == 0) bulk_wait_read<0>();
      const long long my_row = seg.row + (seg.mode == kRowsHome ? tile_row + my_off : first * g.G + row);
      if (row_valid && CP_IN_BOUNDS(token_in(g, seg.t0 + first + tok, seg.h * g.G + sub) &&
                                        (final_rows || part_rows_in(args, my_row, 1)), status)) {
        const float lse2 = l != 0.f ? m + lg2_approx(l) - kBias : -INFINITY;
        if (final_rows)
          args.lse[static_cast<long long>(seg.h * g.G + sub) * g.N + seg.t0 + first + tok] = lse2 * 0.69314718055994531f;
        else
          args.part_lse[my_row] = lse2;
      }
      __syncwarp();      // the staging is read before the next segment's Q lands on it
      tc_fence_before();  // O was read before this warp's next arrival lets a PV overwrite it
    }
    bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Boxes of 32 rows x 128 bytes (swizzled) over the part rows, and over o as
// [tokens][heads][columns].
bool make_part_map(CUtensorMap* m, const void* base, int d, long long rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(d) * 4};
  cuuint32_t box[2] = {32, 32}, estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool make_o_map(CUtensorMap* m, const PagedGeom& g, const void* base) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(g.d), static_cast<cuuint64_t>(g.Hq), static_cast<cuuint64_t>(g.N)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(g.d) * 2, static_cast<cuuint64_t>(g.d) * 2 * g.Hq};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(g.G), static_cast<cuuint32_t>(32 / g.G)}, estr[3] = {1, 1, 1};
  return enc(m, g.dtype == CP_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
             const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D>
int launch_large_d(const PagedAttnArgs& a, cudaStream_t stream) {
  const PagedGeom& g = a.g;
  static std::atomic<int> known[64];
  int sms = 0;
  int rc = prepare_kernel(known, paged_large_kernel<T, D>, kLaunchBytes<D>, &sms);
  if (rc != CP_OK) return rc;
  const int page = 1 << g.page_shift, box = page < BN ? page : BN;
  CUtensorMap mk, mv, mk16, mv16;
  if (!make_cache_map(&mk, g, a.k_cache, box) || !make_cache_map(&mv, g, a.v_cache, box) ||
      !make_cache_map_whole(&mk16, g, a.k_cache, 16) || !make_cache_map_whole(&mv16, g, a.v_cache, 16))
    return CP_ERR_CUDA;
  // Boxes of 32 rows: of the slots, and of o where 32 rows are whole tokens.
  const bool o_boxes = !a.out_fp32 && 32 % g.G == 0;
  CUtensorMap mp, mo;
  if (!make_part_map(&mp, a.part_o, g.d, a.rows_large_end) || (o_boxes && !make_o_map(&mo, g, a.o))) return CP_ERR_CUDA;
  if (!o_boxes) mo = mp;  // not used
  const int workers = sms < kLargeWorkers ? sms : kLargeWorkers;
  return launch(paged_large_kernel<T, D>, workers, kThreads, kLaunchBytes<D>, stream, mk, mv, mk16, mv16, mp, mo,
                a, box, o_boxes ? 1 : 0);
}

}  // namespace

int launch_paged_large(const PagedAttnArgs& a, cudaStream_t stream) {
  const bool bf16 = a.g.dtype == CP_DTYPE_BF16;
  if (a.g.d == 128) return bf16 ? launch_large_d<__nv_bfloat16, 128>(a, stream) : launch_large_d<__half, 128>(a, stream);
  if (a.g.d == 64) return bf16 ? launch_large_d<__nv_bfloat16, 64>(a, stream) : launch_large_d<__half, 64>(a, stream);
  return CP_ERR_UNSUPPORTED;
}

}  // namespace cpattn
