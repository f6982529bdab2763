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
// differences and sums are kept as pairs of fp32 numbers whose sum is the
// value (exact sum and difference of two floats: Knuth, Dekker), good to some 2^-44:
// one in 10^8.  In fp64 each element would cost two operations of units that
// do two a clock and SM (128K elements of 64 rows: 27 us an operation).  From a
// warp's totals on, the search counts in whole numbers, the row's sum being some 2^60.
//
// Bound by memory (each sequence's one row of p, and of q where it counts, is
// read once) and, for few sequences, by a chain of dependent loads: lengths,
// tokens, their probabilities, the row.  A cluster of up to 16 CTAs shares a
// row, each warp a stretch of it, so that one sequence uses 16 SMs; the warps' totals
// are exchanged through distributed shared memory; the warp in whose stretch the
// border lies looks closer, at its lanes' sums and then at one lane's elements.
//
// In a graph: one sequence of 5 drafts, V = 100003, 7.3 us (a third of it the
// row's sums, the rest the chain); 64 sequences, 49 MB, 17.0 us; 256 without q,
// 26 MB of bf16, 14.9 us: 0.9 to the accepted drafts, 6 for the row (4.7 on SMs with two
// CTAs, 6.6 with four), 1.5 for the exchange, 2.9 for the search behind it, and
// the launch.  Where each row has one CTA, the time is that of a CTA on its way
// through the row, whatever runs beside it: V = 128000 in bf16, 305 rows 40 us, 400
// 42, 608 43 (152 SMs of four CTAs), 700 74; 304 rows, two CTAs each, 25.  At 400 the issue slots
// are half used, and half of the warps' time is spent on loads.  What was tried on these and not kept:
// CTAs of 128 or 512 threads, or 3 or 5 on an SM (5: 7.6, 20.8, 19.1); granules
// through shared memory by asynchronous copies (27.7 and 23.2); a prefetch of the stretch
// into L2 (7.4, 19.5, 15.3); the next step's granules in registers, or without q
// four of p at a time (7.6, 18.1, 16.0; 400 rows 44 to 42); sums in packed additions (7.4, 17.1, 15.6)
// or above a power of two that spares the minimum and maximum (7.5, 16.9, 16.0).
#include <cuda_runtime.h>

#include <climits>

#define CP_TU_ID ::cpattn::kTuVerify
#include "host.h"
#include "paged.cuh"

namespace cpattn {
namespace {

constexpr int kVerifyThreads = 256, kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyMaxCluster = 16, kVerifyResident = 4;  // CTAs of an SM
constexpr int kVerifySums = kVerifyMaxCluster * kVerifyWarps;
constexpr int kVerifySlots = 4;
constexpr int kVerifyAhead = 2;                 // granules of a lane in a step
constexpr int kVerifyStep = 32 * kVerifyAhead;  // and of a warp

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

// The number hi + lo.
struct Pair {
  float hi = 0.f, lo = 0.f;
  // += x + rest, exactly but for the rounding of lo (Knuth's sum of two numbers).
  __device__ __forceinline__ void add(float x, float rest) {
    const float s = __fadd_rn(hi, x), b = __fadd_rn(s, -hi);
    const float e = __fadd_rn(__fadd_rn(hi, -__fadd_rn(s, -b)), __fadd_rn(x, -b));
    hi = s;
    lo = __fadd_rn(lo, __fadd_rn(e, rest));
  }
  // += x >= 0 where hi >= 0: the sum's rounding from the larger of the two (Dekker).
  __device__ __forceinline__ void add(float x) {
    const float s = __fadd_rn(hi, x);
    lo = __fadd_rn(lo, __fadd_rn(fminf(hi, x), -__fadd_rn(s, -fmaxf(hi, x))));
    hi = s;
  }
};

// Numbers of a row in units of which its sum, about `sum`, is 2^60 to 2^61.
struct Units {
  float a = 0.f, b = 0.f;  // their product: 2^187 over the sum's power of two, with the exponent's bias
  __device__ __forceinline__ void set(float sum) {
    const int e = max(static_cast<int>(__float_as_uint(sum) >> 23), 1), k = 187 - e;
    a = __uint_as_float((127 + k / 2) << 23);
    b = __uint_as_float((127 + k - k / 2) << 23);
  }
  // At least 1 where there is anything.
  __device__ __forceinline__ long long of(float hi, float lo) const {
    const long long x = __float2ll_rn(hi * a * b) + __float2ll_rn(lo * a * b);
    return hi > 0.f && x < 1 ? 1 : x;
  }
};

// Code that a CTA runs once comes from L2 line by line, some 12 clocks an
// instruction, and an fp64 operation takes a warp 64 clocks: from here on the code is
// in loops and one copy, and counts in whole numbers.

// The sum over the warp's lanes, the same bits in all of them: hi is, as the sum of two
// numbers does not hang on their order; lo + (e + rest) does, by a rounding, and the
// search wants each stretch's share to be one number for every lane and CTA (of
// equal stretches up to all of the borders between them had no owner, or two).
__device__ __forceinline__ Pair warp_sum(Pair v) {
#pragma unroll 1
  for (int x = 16; x > 0; x >>= 1) v.add(__shfl_xor_sync(0xffffffffu, v.hi, x), __shfl_xor_sync(0xffffffffu, v.lo, x));
  v.lo = __shfl_sync(0xffffffffu, v.lo, 0);
  return v;
}

// The same of whole numbers of up to 61 bits, 27 of them at a time.
__device__ __forceinline__ long long warp_sum(long long v) {
  constexpr unsigned kMask = (1u << 27) - 1;
  const unsigned a = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(v) & kMask);
  const unsigned b = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(v >> 27) & kMask);
  const unsigned c = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(v >> 54));
  return a + (static_cast<long long>(b) << 27) + (static_cast<long long>(c) << 54);
}

struct Found {
  int lane;
  long long before, end;
};

// Of the lanes, each with a share `own` behind `before` and those of the lanes below it,
// the first that ends above the border and has any weight, or else the last with
// any; -1 without any.  What lies before that lane's share, and behind the last lane's.
__device__ __noinline__ Found find_lane(long long own, long long before, long long border) {
  const int lane = threadIdx.x & 31;
  long long upto = own;
#pragma unroll 1
  for (int x = 1; x < 32; x <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, upto, x);
    if (lane >= x) upto += y;
  }
  upto += before;
  const unsigned some = __ballot_sync(0xffffffffu, own > 0), above = __ballot_sync(0xffffffffu, own > 0 && upto > border);
  const int who = above ? __ffs(above) - 1 : some ? 31 - __clz(some) : -1;
  return Found{who, __shfl_sync(0xffffffffu, upto - own, max(who, 0)), __shfl_sync(0xffffffffu, upto, 31)};
}

// A row of weights w = max(p - q, 0), or p where there is no q; with draft x >= 0
// and no q, max(p - 1, 0) there.
template <typename T>
struct Row {
  static constexpr int kN = 16 / sizeof(T);  // elements of a granule, 16 aligned bytes of p
  const T* p;
  const T* q;
  int x, V, skew;  // granule g begins at element g * kN - skew
  bool alike;      // q's granules are aligned where p's are

  __device__ __forceinline__ Row(const T* p_row, const T* q_row, int vocab, int draft) : p(p_row), q(q_row), x(draft), V(vocab) {
    skew = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    alike = !q || ((reinterpret_cast<uintptr_t>(q) ^ reinterpret_cast<uintptr_t>(p)) & 15) == 0;
  }
  __device__ __forceinline__ int granules() const { return static_cast<int>((static_cast<long long>(V) + skew + kN - 1) / kN); }
  // First element of granule g, within the row.
  __device__ __forceinline__ int element(int g) const {
    const long long e = static_cast<long long>(g) * kN - skew;
    return static_cast<int>(e < 0 ? 0 : e > V ? V : e);
  }
  // w = d + rest exactly: where u >= v >= 0 the difference's rounding is a float
  // (Dekker).  u: p, or 0 where that is negative or NaN.
  static __device__ __forceinline__ void diff(float u, float of_q, float& d, float& rest) {
    const float v = fminf(fmaxf(of_q, 0.f), u);
    d = __fadd_rn(u, -v);
    rest = __fadd_rn(__fadd_rn(u, -d), -v);
  }
  __device__ __forceinline__ void element_weight(int e, float& d, float& rest) const {
    diff(weight(static_cast<float>(p[e])), q ? static_cast<float>(q[e]) : e == x ? 1.f : 0.f, d, rest);
  }
};

template <typename T>
__device__ __forceinline__ void unpack(const uint4& r, float (&x)[16 / sizeof(T)]) {
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

// How the lanes of a warp share granules: in each step of a slot of `steps` a lane
// takes those number lane * lane_step + step * step_size + i * next, i < kVerifyAhead.
struct Share {
  int steps, lane_step, step_size, next;
};
// Neighbouring lanes take neighbours, as the memory likes it, or a lane takes neighbours.
__device__ __forceinline__ Share by_granule(int steps) { return Share{steps, 1, kVerifyStep, 32}; }
__device__ __forceinline__ Share by_lane(int steps) { return Share{steps, kVerifyAhead * steps, kVerifyAhead, 1}; }

// The lane's sum of granules [g0, g1) of the row; of each slot its sum goes to `slots`.
// An infinite element makes the sum infinite or NaN, unless it is taken one by one.
template <typename T>
__device__ __forceinline__ Pair sum_granules(const Row<T>& row, int g0, int g1, const Share& share, float2 (*slots)[32]) {
  constexpr int kN = Row<T>::kN, kAhead = kVerifyAhead;
  const int lane = threadIdx.x & 31;
  Pair sum;
  const uint4* p = reinterpret_cast<const uint4*>(row.p - row.skew);
  const uint4* q = row.q ? reinterpret_cast<const uint4*>(row.q - row.skew) : nullptr;
  // Granules that are vectors: not the row's first and last where they are not
  // whole, nor the one of the draft that loses 1, and none where p and q are not
  // aligned alike.
  const int v0 = max(g0, row.alike ? row.skew > 0 : INT_MAX), v1 = min(g1, row.granules() - ((row.V + row.skew) % kN > 0));
  const unsigned vectors = static_cast<unsigned>(max(v1 - v0, 0));
  const int gx = !q && row.x >= 0 ? (row.x + row.skew) / kN : -1;
  const int size = share.steps * kVerifyStep;
  int number = 0;
#pragma unroll 1
  for (int slot = g0; slot < g1; slot += size) {
    Pair part;
    const int slot_end = min(slot + size, g1);
    int g = slot + lane * share.lane_step;
#pragma unroll 1
    for (int step = 0; step < share.steps; ++step, g += share.step_size) {
      uint4 x[kAhead], y[kAhead];
      bool whole = true;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) whole &= static_cast<unsigned>(g + i * share.next - v0) < vectors && g + i * share.next != gx;
      const bool all = __all_sync(0xffffffffu, whole);
      if (all) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          x[i] = p[g + i * share.next];
          if (q) y[i] = q[g + i * share.next];
        }
      } else {
        if (!__any_sync(0xffffffffu, g < slot_end)) break;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int at = g + i * share.next;
          x[i] = y[i] = make_uint4(0, 0, 0, 0);
          if (at >= slot_end) continue;
          if (static_cast<unsigned>(at - v0) < vectors && at != gx) {
            x[i] = p[at];
            if (q) y[i] = q[at];
          } else {  // not a vector
#pragma unroll 1
            for (int e = row.element(at), end = row.element(at + 1); e < end; ++e) {
              float d, rest;
              row.element_weight(e, d, rest);
              part.add(d, rest);
            }
          }
        }
      }
      // fmaxf: neither negative nor NaN.
      if (q) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          float u[kN], v[kN];
          unpack<T>(x[i], u);
          unpack<T>(y[i], v);
#pragma unroll
          for (int e = 0; e < kN; ++e) {
            float d, rest;
            Row<T>::diff(fmaxf(u[e], 0.f), v[e], d, rest);
            part.add(d);
            part.lo = __fadd_rn(part.lo, rest);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          float u[kN];
          unpack<T>(x[i], u);
#pragma unroll
          for (int e = 0; e < kN; ++e) part.add(fmaxf(u[e], 0.f));
        }
      }
    }
    slots[number++][lane] = make_float2(part.hi, part.lo);
    sum.add(part.hi, part.lo);
  }
  return sum;
}

__device__ __forceinline__ int cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return static_cast<int>(r);
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// v to the address of `local` in the shared memory of CTA `rank`.
__device__ __forceinline__ void st_cluster(float2* local, int rank, float x, float y) {
  const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(local));
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(a), "r"(rank));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(remote), "f"(x), "f"(y) : "memory");
}

// A draft's place in a row; -1: none.
__device__ __forceinline__ int draft_at(int x, int V) { return x >= 0 && x < V ? x : -1; }

// One cluster a sequence.
template <typename T>
__global__ void __launch_bounds__(kVerifyThreads, kVerifyResident) verify_kernel(const __grid_constant__ VerifyArgs a, int cluster) {
  __shared__ float2 sums[3][kVerifySums + 1];  // all warps', for each turn; behind them whether there is a residual
  __shared__ float2 slots[kVerifyWarps][kVerifySlots][32];
  __shared__ int found_accepted;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = cluster_rank(), s = blockIdx.x / cluster;
  cluster_arrive();  // waited for before the first store to another CTA, which has begun then
  pdl_wait();
  pdl_launch_dependents();
  const int t0 = a.q_start[s], t1 = a.q_start[s + 1], n = t1 - t0;
  const float of_all = a.N > 0 ? a.sample_u[s] : 0.f;  // without rows the array may be null
  // Every CTA goes through the same cluster barriers, whatever it finds in the arrays.
  const bool good = CP_CHECK_DATA(t0 >= 0 && t1 >= t0 && t1 <= a.N && n <= a.max_new, a.status);
  const T* p = static_cast<const T*>(a.p);
  const T* q = static_cast<const T*>(a.q);
  // Drafts accepted: 32 at a time, by every CTA's first warp.
  if (warp == 0) {
    int accepted = good ? max(n - 1, 0) : 0;
#pragma unroll 1
    for (int i0 = 0; good && i0 < n - 1; i0 += 32) {
      const int i = i0 + lane;
      bool ok = true;
      if (i < n - 1) {
        const int x = a.tokens[t0 + i + 1];
        const float u = a.accept_u[t0 + i];
        ok = CP_CHECK_DATA(x >= 0 && x < a.V, a.status);
        if (ok) {
          const float px = weight(static_cast<float>(p[(t0 + i) * a.p_stride + x]));
          float qx = 1.f;
          if (q) qx = static_cast<float>(q[(t0 + i) * a.q_stride + x]);
          if (!(qx > 0.f)) qx = 0.f;
          // A product of two floats is exact in fp64.
          ok = static_cast<double>(u) * static_cast<double>(qx) < static_cast<double>(px);
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
  const bool there = live && CP_IN_BOUNDS(t < a.N, a.status);
  Row<T> row(there ? p + t * a.p_stride : nullptr, there && rejected && q ? q + t * a.q_stride : nullptr, there ? a.V : 0,
             there && rejected && !q ? draft_at(a.tokens[t + 1], a.V) : -1);
  // A stretch of granules for each warp of the cluster, in slots of `steps` steps.
  const int warps = cluster * kVerifyWarps, granules = row.granules(), w = rank * kVerifyWarps + warp;
  const int per = (granules + warps - 1) / warps, steps = (per + kVerifySlots * kVerifyStep - 1) / (kVerifySlots * kVerifyStep);
  const int size = steps * kVerifyStep;
  int g0 = min(w * per, granules), g1 = min(g0 + per, granules);
  Share share = by_granule(steps);
  Units units;
  long long at = 0, border = 0;
  Pair v;
  bool clean = false, plain = false, found = false;
  // First every warp its stretch, in one turn and seldom more; then the warp that
  // has found the border in its stretch one slot of that: in one copy of the code.
#pragma unroll 1
  for (int turn = 0;; ++turn) {
    v = sum_granules<T>(row, g0, g1, share, slots[warp]);
    if (found) break;
    v = warp_sum(v);
    if (turn == 0) cluster_wait();
    if (lane < cluster) {
      st_cluster(&sums[turn][w], lane, v.hi, v.lo);
      if (w == 0) st_cluster(&sums[turn][kVerifySums], lane, rejected ? 1.f : 0.f, 0.f);
    }
    cluster_arrive();
    cluster_wait();
    // Every warp: what lies before its stretch, and in all.
    float about = 0.f;
#pragma unroll 1
    for (int k = lane; k < warps; k += 32) about += sums[turn][k].x;
#pragma unroll 1
    for (int x = 16; x > 0; x >>= 1) about += __shfl_xor_sync(0xffffffffu, about, x);
    long long total = 0;
    if (about > 0.f && about < INFINITY) {
      units.set(about);
#pragma unroll 1
      for (int k = lane; k < warps; k += 32) {
        const long long x = units.of(sums[turn][k].x, sums[turn][k].y);
        total += x;
        if (k < w) at += x;
      }
      at = warp_sum(at);
      total = warp_sum(total);
    } else if (turn < 2 && (about != 0.f ? !clean : !plain && sums[0][kVerifySums].x != 0.f)) {
      // Seldom, and the same for all warps of the cluster, who decide it by what
      // they have exchanged.  Infinite elements: again, one by one, without them.
      // Nothing left of p (the rows are not what they should be): p itself.
      if (about != 0.f) {
        clean = true;
        row.alike = false;
      } else {
        plain = true;
        row.q = nullptr;
        row.x = -1;
      }
      continue;
    }
    if (rank == 0 && warp == kVerifyWarps - 1 && good) {
      for (int i = lane; i < n; i += 32)
        if (i != accepted) a.out_tokens[t0 + i] = i < accepted ? a.tokens[t0 + i + 1] : -1;
      if (lane == 0) {
        a.accepted[s] = accepted;
        if (a.kv_out) a.kv_out[s] = a.kv_len[s] - max(n - 1 - accepted, 0);
        if (live && total == 0) a.out_tokens[t] = -1;
      }
    }
    // r of the total, cut to a whole number, which no sum of whole numbers can tell from it.
    unsigned long long r = 0;
    if (of_all > 0.f) r = __float2ull_rz(fminf(of_all, 0x1.fffffep-1f) * 0x1p64f);
    border = static_cast<long long>(__umul64hi(static_cast<unsigned long long>(total), r));
    if (!live || at > border || border >= at + units.of(v.hi, v.lo)) return;
    // This warp's stretch holds it: which of its slots.  Their sums are rounded
    // otherwise than the stretch's: where none ends above the border, it is the last with any weight.
    int slot = -1;
    long long before = at;
#pragma unroll 1
    for (int k = 0; g0 + k * size < g1 && at <= border; ++k) {
      const long long x = warp_sum(units.of(slots[warp][k][lane].x, slots[warp][k][lane].y));
      if (x > 0) slot = k, before = at;
      at += x;
    }
    if (slot < 0) return;  // not so: the stretch has weight
    at = before;
    g0 += slot * size;
    g1 = min(g0 + size, g1);
    share = by_lane(steps);
    found = true;
  }
  // Which lane's part of the slot, and which of its elements.
  Found f = find_lane(units.of(v.hi, v.lo), at, border);
  if (f.lane < 0) return;
  const int part = steps * kVerifyAhead, e1 = row.element(min(g0 + (f.lane + 1) * part, g1));
  int token = -1;
  at = f.before;
#pragma unroll 1
  for (int e0 = row.element(g0 + f.lane * part); e0 < e1 && at <= border; e0 += 32) {
    float d = 0.f, rest = 0.f;
    if (e0 + lane < e1) row.element_weight(e0 + lane, d, rest);
    f = find_lane(units.of(d, rest), at, border);
    at = f.end;
    if (f.lane >= 0) token = e0 + f.lane;
  }
  if (lane == 0) a.out_tokens[t] = token;
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
  // As many CTAs a sequence as the card holds at once, none with less than 2048
  // elements; 16 only for up to 8 sequences, as so many that have to start
  // together wait for one another (V = 128000, 8 and 16 CTAs: 2 sequences 8.8 and 7.4 us, 8
  // 8.9 and 8.5, 16 9.7 and 9.8, 32 12.3 and 16.8; V = 32000: 1 5.8 and 5.9, 8 6.0 and 6.6).
  int cluster = 1;
  while (a.B * cluster * 2 <= kVerifyResident * 152 && a.V / cluster > 4096 && cluster < (a.B <= 8 ? kVerifyMaxCluster : 8)) cluster *= 2;
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
  // Without rows every sequence has none, which its outputs say; the kernel reads none of these then.
  if (batch->n_tokens > 0 && (!v.p || !v.tokens || !v.accept_u || !v.sample_u || !v.out_tokens)) return CP_ERR_INVALID_ARG;
  // No output is another array, save that kv_len_out may be kv_len.  Without rows theirs are not touched.
  const void* in[] = {batch->q_start, batch->kv_len, v.tokens, v.accept_u, v.sample_u, v.p, v.q};
  const void* out[] = {v.accepted, v.kv_len_out, v.out_tokens};
  const int ins = batch->n_tokens > 0 ? 7 : 2, outs = batch->n_tokens > 0 ? 3 : 2;
  for (int i = 0; i < outs; ++i) {
    for (int k = 0; k < ins; ++k)
      if (out[i] && out[i] == in[k] && !(i == 1 && k == 1)) return CP_ERR_INVALID_ARG;
    for (int k = 0; k < i; ++k)
      if (out[i] && out[i] == out[k]) return CP_ERR_INVALID_ARG;
  }
  const uintptr_t element = v.dtype == CP_DTYPE_FP32 ? 4 : 2;
  if (!aligned(v.p, element) || !aligned(v.q, element)) return CP_ERR_ALIGNMENT;
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
