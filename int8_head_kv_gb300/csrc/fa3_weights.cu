// Attention weight that each cached token gets (tcgen05, sm_103a): what an eviction goes by.
//
// For token t of a sequence and KV head g, over the sequence's packed new rows i that see it and the G query heads of g:
//   w[t] = sum_{i, h} exp(s[t] - lse[i, h]),   s[t] = (q[i, h] . k8[t, g]) * k_scale[t's block, g] * softmax_scale
// which is added to the token's weight; the new rows' own tokens begin with nothing.
//
// Only keys are read, and the scores are turned round: keys are the rows of the MMA (A), queries its columns (B), so that
// a thread has a key and sums along its own TMEM lane.  bf16 queries go in as they are, and an int8 code is exact
// in bf16, so the products are exact and the sums float32.
//
// The row's log-sum-exp goes into the product as well: with f the key's factor (its scale, softmax_scale and log2(e)), the exponent
// is f (S - lse / f), and lse / f is a product of a number of the key's and one of the column's.  Both are split into
// three bf16 parts, exactly, and the eight products of parts that count (what is left out is below 2^-31 of it) are one more
// slice of the contraction.  It is the last, and taken relative to the lse of the step's first column, where that is a common
// number, which the exponent gets in float32: the tensor pipe cuts its sums off relative to their largest term, which
// lse / f would be (weights of 4096 rows on 8192 keys were off by 1.5e-6 of them in the mean with all of it as the first slice,
// 6e-7 as the last, 1.2e-7 so; 308, 309 and 312 us).  A thread then reads little but its scores: with the log-sum-exps in shared
// memory, each warp reading them anew, that memory was the bound (4460 cycles for 512 keys x 128 columns; the MMAs alone take 2048).
//
// Work.  A unit is 512 keys of one sequence and KV head, as four row tiles; a step is the scores of P new tokens x G heads
// (up to 128 columns) with all four.  All units lie on one line that is cut into equal parts, one per SM; a cut unit's
// parts leave their sums in the workspace, and weights_combine_kernel adds them up in order, so results do not
// depend on which CTA is first.
//
// Roles in the CTA (768 threads).  Warp 0 issues the MMAs, warp 1 brings the query tiles by TMA, warp 2 plans, warp 3 writes the
// columns' parts of the log-sum-exps.  Warps 4-7, 8-11, 12-15 and 16-19 (a key a lane) sum up the four row tiles' scores, each in a
// quarter of TMEM.  Warps 20-23 bring the int8 keys and write them as bf16, and the keys' parts of the log-sum-exps.
//
// What bounds it (64 query and 8 KV heads, one GB300).  4096 new rows on a context of 8192: 312 us, 1320 TFLOP/s (exponentials
// not counted).  The tensor pipe is active for 45 % of the time; the warps that sum, each row tile's four, wait for TMEM,
// multiply, exponentiate and add, and are busy for 80 %.  Their fast loop is for steps of 128 columns, that is groups that divide
// 128 and calls with rows enough on average; in other groups every step is read with its mask, 680 to 730 TFLOP/s (56 query
// and 8 KV heads: 493 us, 24 and 8: 225, 28 and 4: 254).  With few columns a unit's keys are what costs (their way to shared
// memory as bf16, some 8 us a unit): 16 contexts of 4096 keys take 51 us with 8 columns each as with 128, so few columns go to
// fa3_few.cu's kernel.
//
// Every wait is bounded; on time-out the kernel sets FA3_DEVERR_TIMEOUT, waits for its
// copies and MMAs, frees its TMEM and returns.
#include "fa3_few.cuh"
#include "fa3_packed.cuh"
#include "fa3_pipe.cuh"

#include <math_constants.h>

#include <algorithm>
#include <atomic>
#include <cmath>

namespace fa3 {
namespace {

constexpr int kD = 128;
constexpr int kTilesW = 4, kKeysW = 128 * kTilesW;         // row tiles of the MMA and keys of a unit
constexpr int kCols = 128;         // columns of a step, at most
constexpr int kThreadsW = 768;
constexpr uint32_t kHalfTile = 128 * 128;                  // 128 rows of 64 values of d, 128-byte swizzle
constexpr uint32_t kTile = 2 * kHalfTile;                  // 128 rows of 128 values
constexpr uint32_t kQStages = 2;
constexpr uint32_t kSlice = 128 * 32;                      // 128 rows of 16 values, in two chunks of 8
constexpr uint32_t OFF_KW = 0;                             // four row tiles
constexpr uint32_t OFF_QW = OFF_KW + 4 * kTile;
constexpr uint32_t OFF_KX = OFF_QW + kQStages * kTile;     // the row tiles' slices of the log-sum-exp
constexpr uint32_t OFF_QX = OFF_KX + kTilesW * kSlice;     // the columns', a stage each
constexpr uint32_t kRingW = 4, kPartBytesW = 48;
constexpr uint32_t OFF_PARTSW = OFF_QX + kQStages * kSlice;
constexpr uint32_t OFF_BARW = OFF_PARTSW + kRingW * kPartBytesW;
enum {
  W_K_FULL = 0, W_K_EMPTY = 1,     // a unit's keys written; all its MMAs done
  W_S_FULL = 2, W_S_EMPTY = 6,     // [4]: a row tile's scores of a step; read
  W_Q_FULL = 10, W_Q_EMPTY = 12,   // [2]: a step's queries and log-sum-exps
  W_DRAIN = 14,
  W_PART_FULL = 15, W_PART_EMPTY = 19,   // [4]
  W_N = 23
};
__constant__ const uint8_t kArrivalsW[W_N] = {4, 1, 1, 1, 1, 1, 4, 4, 4, 4, 2, 2, 1, 1, 1, 1, 1, 1, 1, 23, 23, 23, 23};
constexpr uint32_t OFF_TSLOTW = OFF_BARW + 8 * W_N;
constexpr uint32_t OFF_ABORTW = OFF_TSLOTW + 4;
constexpr uint32_t SMEM_WEIGHTS = OFF_ABORTW + 4 + 1024;   // + alignment slack
static_assert(SMEM_WEIGHTS <= 232448, "shared memory");

// The line's unit is a step.  kUnitSteps: what a unit costs beside its steps (its keys' way to shared memory); kLeastSteps: the
// least part of the line a CTA takes, enough for a part inside a unit to hold a step.
constexpr int kUnitSteps = 2, kLeastSteps = 4;
static_assert(kLeastSteps > kUnitSteps, "a part inside a unit, behind its fixed cost, holds a step");

struct CutW {
  int b, g, tile, first, last;     // unit, CTAs that have parts of it; first < 0: none begins here
};

struct WeightParams {
  const int8_t* k;                 // [pool rows][Hkv][128]
  const float* ks;
  const float* lse;                // [n][Hq]
  float* weights;                  // [num_pages][Hkv][page_size]
  const int32_t* q_start;
  const int32_t* kv_lens;
  float* part;                     // [2 * CTAs][512]: sums of a cut unit's parts
  CutW* cuts;                      // [CTAs]
  int32_t* err;
  Pages pg;
  int n, B, Hq, G, P, ctas, narrow;
  DivU32 div_G, div_P;
  float sm_log2;
  uint32_t wait_ticks;             // of a wait for a unit's work
  CUtensorMap map_q;               // bf16 [n][Hq][128] in boxes of [P][G][64]
};

struct SeqW {
  int q0, nq, nkv;
};
// nq = 0: nothing to do; -1: q_start falls.
__device__ __forceinline__ SeqW sequence_of(const WeightParams& p, int b, bool report) {
  SeqW s;
  s.q0 = p.q_start[b];
  const int q1 = p.q_start[b + 1];
  s.nkv = p.kv_lens[b];
  s.nq = q1 - s.q0;
  if (s.q0 < 0 || q1 < s.q0 || q1 > p.n || (s.nq > 0 && (s.nkv < s.nq || s.nkv > p.pg.T_max))) {
    if (report) set_dev_err(p.err, FA3_DEVERR_LENS);
    s.nq = q1 < s.q0 ? -1 : 0;
  }
  return s;
}
__device__ __forceinline__ int tiles_of(const SeqW& s) { return s.nq > 0 ? (int)(((uint32_t)s.nkv + kKeysW - 1) / kKeysW) : 0; }
// Column tiles of the sequence's rows, and the first that sees key tile j: row i sees key t from t = nkv - nq + i down.
__device__ __forceinline__ int col_tiles(const WeightParams& p, const SeqW& s) {
  return (int)divu32((uint32_t)(s.nq + p.P - 1), p.div_P);
}
__device__ __forceinline__ int first_col_tile(const WeightParams& p, const SeqW& s, int j) {
  const int i0 = j * kKeysW - (s.nkv - s.nq);
  return i0 <= 0 ? 0 : (int)divu32((uint32_t)i0, p.div_P);
}
// The first column tile that sees a key of row tile x of key tile j, as all behind it do (col_tiles: none does).
__device__ __forceinline__ int first_of_tile(const WeightParams& p, const SeqW& s, int j, int x) {
  return j * kKeysW + 128 * x < s.nkv ? first_col_tile(p, SeqW{s.q0, s.nq, s.nkv - 128 * x}, j) : col_tiles(p, s);
}
__device__ __forceinline__ int steps_of(const WeightParams& p, const SeqW& s, int j) { return col_tiles(p, s) - first_col_tile(p, s, j); }
// Cost of all units of one KV head.
template <class I>
__device__ __forceinline__ I sequence_cost(const WeightParams& p, const SeqW& s) {
  const int nt = tiles_of(s);
  if (nt == 0) return 0;
  I c = (I)nt * (I)(kUnitSteps + col_tiles(p, s));
  const int js = (s.nkv - s.nq) / kKeysW + 1;                // the first tile whose first key some row does not see
  if (js < nt) c -= floor_sum<I>((I)(nt - js), (I)p.P, (I)kKeysW, (I)js * kKeysW - (I)(s.nkv - s.nq));
  return c;
}

// What a CTA does of a unit: steps [s0, s1) of n.
struct PartW {
  int b, g, tile, q0, nq, nkv, s0, s1, n;
};
static_assert(sizeof(PartW) <= kPartBytesW, "ring of parts");

__device__ __forceinline__ SeqW lane_of(const SeqW& s, int l) {
  return SeqW{__shfl_sync(0xffffffffu, s.q0, l), __shfl_sync(0xffffffffu, s.nq, l), __shfl_sync(0xffffffffu, s.nkv, l)};
}
__device__ __forceinline__ SeqW sequence_or_none(const WeightParams& p, int b, bool report) {
  return b < p.B ? sequence_of(p, b, report) : SeqW{0, 0, 0};
}

// A CTA's parts in order (the warp together), each given to `put`; the record of the cut behind its part.
template <class I, class Put>
__device__ __forceinline__ void walk_parts(const WeightParams& p, int cta, int lane, Put put) {
  CutW cut = {0, 0, 0, -1, -1};
  Line<I> line;
  line.total = 0;
  bool falls = false;
#pragma unroll 1
  for (int base = 0; base < p.B; base += 32) {
    const SeqW s = sequence_or_none(p, base + lane, cta == 0);
    falls |= s.nq < 0;
    I c = sequence_cost<I>(p, s) * (I)p.pg.Hkv;
#pragma unroll
    for (int o = 16; o; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    line.total += c;
  }
  if (__any_sync(0xffffffffu, falls)) line.total = 0;        // sequences might share rows, or tokens be counted twice
  const I most = line.total / kLeastSteps;
  line.parts = most < 1 ? 1 : most < (I)p.ctas ? (int)most : p.ctas;
  line.each = line.total / (I)line.parts;
  line.rest = (int)(line.total - line.each * (I)line.parts);
  I x = line.begin(cta), left = line.begin(cta + 1) - x;
  I skip = x;                                                // of the line, in front of the sequence looked at
#pragma unroll 1
  for (int base = 0; base < p.B && left > 0; base += 32) {
    const SeqW mine = sequence_or_none(p, base + lane, false);
    const I per_head = sequence_cost<I>(p, mine), all = per_head * (I)p.pg.Hkv;
    const I upto = warp_scan<I>(all, lane), sum = __shfl_sync(0xffffffffu, upto, 31);
    if (sum <= skip) {
      skip -= sum;
      continue;
    }
    unsigned todo = __ballot_sync(0xffffffffu, upto > skip && all > 0);
    bool first = true;
#pragma unroll 1
    while (todo && left > 0) {
      const int l = __ffs(todo) - 1;
      todo &= todo - 1;
      const SeqW s = lane_of(mine, l);
      const I head = __shfl_sync(0xffffffffu, per_head, l);
      I off = first ? skip - (__shfl_sync(0xffffffffu, upto, l) - head * (I)p.pg.Hkv) : 0;
      first = false;
      int g = (int)(off / head);
      off -= (I)g * head;
      const int nt = tiles_of(s);
#pragma unroll 1
      for (; g < p.pg.Hkv && left > 0; ++g) {
        // the unit that holds `off`
        int j = 0;
        if (off > 0) {
#pragma unroll 1
          for (;; j += 32) {
            const I c = j + lane < nt ? (I)(kUnitSteps + steps_of(p, s, j + lane)) : 0, u = warp_scan<I>(c, lane);
            const unsigned beyond = __ballot_sync(0xffffffffu, u > off);
            if (beyond) {
              const int k = __ffs(beyond) - 1;
              off -= __shfl_sync(0xffffffffu, u - c, k);
              j += k;
              break;
            }
            off -= __shfl_sync(0xffffffffu, u, 31);
          }
        }
#pragma unroll 1
        for (; j < nt && left > 0; ++j) {
          const int n = steps_of(p, s, j);
          const I cost = (I)(kUnitSteps + n), take = min(cost - off, left);
          auto step_at = [&](I o) { return o <= (I)kUnitSteps ? 0 : (int)(o - (I)kUnitSteps); };
          const int s0 = step_at(off), s1 = off + take == cost ? n : step_at(off + take);
          if (s0 < s1) {
            if (s0 == 0 && s1 < n) cut = CutW{base + l, g, j, cta, line.owner(x + (cost - off) - 1)};
            if (!put(PartW{base + l, g, j, s.q0, s.nq, s.nkv, s0, s1, n})) left = take;
          }
          left -= take;
          x += take;
          off = 0;
        }
        off = 0;
      }
    }
    skip = 0;
  }
  if (lane == 0) p.cuts[cta] = cut;
}

// Adds `sum` to the weight of token t: one call a token and head.  Pages may be shared by sequences, old tokens' weights
// are added to atomically then.
__device__ __forceinline__ void add_weight(const WeightParams& p, int b, int g, int t, bool is_new, float sum) {
  const uint32_t pi = divu32((uint32_t)t, p.pg.div_ps);
  const int page = p.pg.table[(int64_t)b * p.pg.max_pages + pi];
  if ((uint32_t)page >= (uint32_t)p.pg.num_pages) {
    set_dev_err(p.err, FA3_DEVERR_PAGE);
    return;
  }
  float* w = p.weights + ((int64_t)page * p.pg.Hkv + g) * p.pg.page_size + (t - (int)pi * p.pg.page_size);
  if (is_new)
    *w = sum;
  else
    atomicAdd(w, sum);
}

// Four signed int8 codes -> two bf16x2 (exact): with the low seven bits as the mantissa of 128, c = (128 + low) - (128 or
// 256), where 256 has the sign bit's place in bf16.
__device__ __forceinline__ void i8x4_to_bf16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  auto two = [](uint32_t p) {                                // 0x43cc in each half
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(p & 0xff7fff7fu), "r"(p & 0xff80ff80u));
    return r;
  };
  lo = two(__byte_perm(w, 0x43434343u, 0x4140));
  hi = two(__byte_perm(w, 0x43434343u, 0x4342));
}

constexpr float kMostLse = 268435456.f;                      // 2^28: log-sum-exps relative to a step's, in log2 units

// A step's exponents are taken relative to its first column's: -lse log2(e), or 0 where that is 64 or more.  A column's weights
// are off by the rounding of the centre's size as well as of its own log-sum-exp's, and rows of large scores stand beside rows
// of small ones: with a centre of 1000 their weights were off by 1e-4.
__device__ __forceinline__ float center_of(float lse) {
  const float c = lse * -1.4426950408889634f;
  return fabsf(c) < 64.f ? c : 0.f;
}

// A number as the sum of three bf16 numbers, exactly (24 bits are three times 8; each is the rest's upper half).
__device__ __forceinline__ void three_parts(float x, uint32_t (&p)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    p[i] = __float_as_uint(x) >> 16;
    x -= __uint_as_float(p[i] << 16);
  }
}
// The factor of a key's scores: not so small that its inverse times kMostLse leaves float32's range (with queries below 2^60, a
// smaller one gives every score 0 as well).
constexpr float kLeastFactor = 3.1554436208840472e-30f;      // 2^-98
__device__ __forceinline__ float key_factor(const WeightParams& p, int page, int at, int g) {
  const float ks = (uint32_t)page < (uint32_t)p.pg.num_pages
                       ? p.ks[((int64_t)page * p.pg.per_page + divu32((uint32_t)at, p.pg.div_block)) * p.pg.Hkv + g]
                       : 0.f;                                 // outside the pool: the keys' loader reports it
  return fmaxf(ks * p.sm_log2, kLeastFactor);
}

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* tm, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(c2), "r"(bar) : "memory");
}

__global__ void __launch_bounds__(kThreadsW, 1) weights_kernel(const __grid_constant__ WeightParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + OFF_ABORTW);
  auto bar = [&](int i) { return sbase + OFF_BARW + 8u * (uint32_t)i; };
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(sbase + OFF_TSLOTW), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (warp == 1) {
    if (lane < W_N) mbar_init(bar(lane), kArrivalsW[lane]);
    if (lane == 0) *abort_flag = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (lane == 0) prefetch_map(&p.map_q);
  }
  // the slices' second chunks are zero
  for (int i = tid; i < (int)((kTilesW + kQStages) * 128); i += kThreadsW)
    sts128(sbase + OFF_KX + (uint32_t)(i >> 7) * kSlice + 2048u + (uint32_t)(i & 127) * 16u, make_uint4(0u, 0u, 0u, 0u));
  fence_proxy_async();
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + OFF_TSLOTW);
  pdl_launch_dependents();

  PartW* const ring = reinterpret_cast<PartW*>(smem + OFF_PARTSW);
  uint32_t parts = 0;                                         // taken (by warp 2: written)
  auto next_part = [&]() {                                    // false: none left
    return warp_wait(bar(W_PART_FULL) + 8u * (parts % kRingW), (parts / kRingW) & 1u, lane, abort_flag, p.err, p.wait_ticks) &&
           ring[parts % kRingW].n >= 0;
  };
  auto part_read = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(W_PART_EMPTY) + 8u * (parts % kRingW));
    ++parts;
  };
  auto warp_arrive = [&](int which) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(which));
  };

  if (warp == 2) {
    auto put = [&](const PartW& u) {
      if (!warp_wait(bar(W_PART_EMPTY) + 8u * (parts % kRingW), ((parts / kRingW) & 1u) ^ 1u, lane, abort_flag, p.err, p.wait_ticks))
        return false;
      if (lane == 0) {
        ring[parts % kRingW] = u;
        mbar_arrive(bar(W_PART_FULL) + 8u * (parts % kRingW));
      }
      ++parts;
      return true;
    };
    if (p.narrow)
      walk_parts<uint32_t>(p, blockIdx.x, lane, put);
    else
      walk_parts<int64_t>(p, blockIdx.x, lane, put);
    PartW end = {};
    end.n = -1;
    put(end);
  } else if (warp == 0) {
    // ------------------------------------------------------------ MMA issuer
    uint32_t units = 0, qs = 0, q_par = 0, done = 0;          // done: parities of the row tiles' steps, a bit each
    bool ok = true;
    const uint32_t lead = elect_one();
    while (ok && next_part()) {
      const PartW u = ring[parts % kRingW];
      part_read();
      ok = warp_all(wait_long(bar(W_K_FULL), units & 1u, abort_flag, p.err, p.wait_ticks));
      const SeqW sq = {u.q0, u.nq, u.nkv};
      const int rt0 = first_col_tile(p, sq, u.tile);
      int seen[kTilesW];                                      // the first step that sees a row tile
#pragma unroll
      for (int x = 0; x < kTilesW; ++x) seen[x] = first_of_tile(p, sq, u.tile, x) - rt0;
#pragma unroll 1
      for (int s = u.s0; s < u.s1 && ok; ++s) {
        ok = warp_all(wait_long(bar(W_Q_FULL) + 8u * qs, q_par, abort_flag, p.err));
        const int cols = min(p.P, u.nq - (rt0 + s) * p.P) * p.G;
        const uint32_t id = idesc_f16(128, (cols + 15) & ~15, true, false);
#pragma unroll
        for (uint32_t x = 0; x < kTilesW; ++x) {
          if (!ok || s < seen[x]) continue;
          ok = warp_all(wait_long(bar(W_S_EMPTY) + 8u * x, ((done >> x) & 1u) ^ 1u, abort_flag, p.err));
          if (!ok) continue;
          tc_fence_after();
          // S = K.Q^T: both K-major, 128-byte swizzle: 8-row groups 1024 B apart, 16 values of d 32 B apart within a half; the
          // slice of the log-sum-exp without swizzle, as 8-row groups 128 B and chunks of 8 values 2048 B apart
          uint32_t a = desc_lo(sbase + OFF_KW + x * kTile, 16), bd = desc_lo(sbase + OFF_QW + qs * kTile, 16);
#pragma unroll 2
          for (int kk = 0; kk < kD / 16; ++kk) {
            mma_ss<desc_hi(1024, true), desc_hi(1024, true)>(lead, tmem + x * 128, a, bd, id, (uint32_t)(kk > 0));
            const uint32_t next = kk == 3 ? (kHalfTile >> 4) - 3 * (32 >> 4) : 32 >> 4;
            a += next;
            bd += next;
          }
          mma_ss<desc_hi(128, false), desc_hi(128, false)>(lead, tmem + x * 128, desc_lo(sbase + OFF_KX + x * kSlice, 2048),
                                                           desc_lo(sbase + OFF_QX + qs * kSlice, 2048), id, 1u);
          commit_if(lead, bar(W_S_FULL) + 8u * x);
          done ^= 1u << x;
        }
        if (!ok) break;
        commit_if(lead, bar(W_Q_EMPTY) + 8u * qs);
        if (++qs == kQStages) qs = 0, q_par ^= 1u;
      }
      if (ok) commit_if(lead, bar(W_K_EMPTY));
      ++units;
    }
    commit_if(lead, bar(W_DRAIN));                            // every MMA issued has completed before TMEM is freed
    wait_long(bar(W_DRAIN), 0, abort_flag, p.err);
  } else if (warp == 1) {
    // ------------------------------------------------------ TMA: query tiles
    uint32_t qs = 0, q_par = 1, sent = 0;
    bool ok = true;
    while (ok && next_part()) {
      const PartW u = ring[parts % kRingW];
      part_read();
      const int rt0 = first_col_tile(p, SeqW{u.q0, u.nq, u.nkv}, u.tile);
#pragma unroll 1
      for (int s = u.s0; s < u.s1 && ok; ++s) {
        ok = warp_wait(bar(W_Q_EMPTY) + 8u * qs, q_par, lane, abort_flag, p.err);
        if (!ok) break;
        const uint32_t full = bar(W_Q_FULL) + 8u * qs, dst = sbase + OFF_QW + qs * kTile;
        if (lane == 0) {
          mbar_expect_tx(full, (uint32_t)(p.P * p.G) * 256u);
          tma_3d(dst, &p.map_q, 0, u.g * p.G, u.q0 + (rt0 + s) * p.P, full);
          tma_3d(dst + kHalfTile, &p.map_q, 64, u.g * p.G, u.q0 + (rt0 + s) * p.P, full);
        }
        ++sent;
        if (++qs == kQStages) qs = 0, q_par ^= 1u;
      }
    }
    // What was sent off lands before the block ends, also after a time-out elsewhere (a bounded wait).
    if (lane < (int)min(sent, kQStages)) {
      const uint32_t k = sent - 1 - (uint32_t)lane, t = k % kQStages, par = (k / kQStages) & 1u;
      const uint64_t t0 = global_ns();
      while (!mbar_try(bar(W_Q_FULL) + 8u * t, par) && global_ns() - t0 < kWaitNs / 50) {}
    }
  } else if (warp == 3) {
    // ------------------------------------------------------ log-sum-exps of a step's columns
    // -lse log2(e) in parts b1, b2, b3 meets the keys' a1, a2, a3 as a1 b1, a1 b2, a2 b1, a1 b3, a2 b2, a3 b1, a2 b3, a3 b2.  A step's
    // values are asked for two steps ahead: their way is longer than a step.
    uint32_t qs = 0, q_par = 1;
    bool ok = true;
    while (ok && next_part()) {
      const PartW u = ring[parts % kRingW];
      part_read();
      const int rt0 = first_col_tile(p, SeqW{u.q0, u.nq, u.nkv}, u.tile);
      float v[3][4];
      auto ask = [&](int s, float (&to)[4]) {
        const int i0 = (rt0 + s) * p.P, cols = s < u.s1 ? min(p.P, u.nq - i0) * p.G : 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = lane + 32 * k, i = (int)divu32((uint32_t)c, p.div_G);
          to[k] = c < cols ? p.lse[(int64_t)(u.q0 + i0 + i) * p.Hq + u.g * p.G + c - i * p.G] : 0.f;
        }
      };
      ask(u.s0, v[0]);
      ask(u.s0 + 1, v[1]);
#pragma unroll 1
      for (int s = u.s0; s < u.s1 && ok; s += 3) {
#pragma unroll
        for (int x = 0; x < 3; ++x) {
          if (s + x < u.s1 && ok) {
            ask(s + x + 2, v[(x + 2) % 3]);
            ok = warp_wait(bar(W_Q_EMPTY) + 8u * qs, q_par, lane, abort_flag, p.err);
            if (ok) {
              const float center = center_of(__shfl_sync(0xffffffffu, v[x][0], 0));
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                // with scores below 2^26 only an infinite lse, whose row's weights are nothing, lies outside; NaN passes
                uint32_t b[3];
                const float y = v[x][k] * -1.4426950408889634f - center;
                three_parts(y < -kMostLse ? -kMostLse : y > kMostLse ? kMostLse : y, b);
                sts128(sbase + OFF_QX + qs * kSlice + (uint32_t)(lane + 32 * k) * 16u,
                       make_uint4(b[0] | b[1] << 16, b[0] | b[2] << 16, b[1] | b[0] << 16, b[2] | b[1] << 16));
              }
              fence_proxy_async();
              warp_arrive(W_Q_FULL + (int)qs);
              if (++qs == kQStages) qs = 0, q_par ^= 1u;
            }
          }
        }
      }
    }
  } else if (warp >= 20) {
    // ------------------------------------------------------ int8 keys -> bf16
    // A warp has a row tile, in four times 32 keys, a lane 16 bytes of eight of them: bytes 16 (l % 8) .. of row l / 8, lanes
    // l % 8 >= 4 of the row's neighbour (l / 8) ^ 1, so that the eight lanes of a store hit different banks of the swizzled
    // rows.  A lane looks four keys up, the others get their rows by shuffles.
    const int cw = warp - 20, cl = lane & 7, rl = (lane >> 3) ^ (cl >> 2);
    const uint32_t dst = sbase + OFF_KW + (uint32_t)cw * kTile + (uint32_t)(cl >> 2) * kHalfTile + (uint32_t)rl * 128;
    const uint32_t at0 = ((uint32_t)(2 * cl & 7) ^ (uint32_t)rl) * 16;   // n % 8 = rl, or rl + 4 for odd i
    const int row_stride = p.pg.Hkv * kD;
    uint32_t units = 0;
    bool ok = true;
    while (ok && next_part()) {
      const PartW u = ring[parts % kRingW];
      part_read();
      const int8_t* base = p.k + u.g * kD + cl * 16;
      int rows[4];
      float factor[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const uint32_t t = (uint32_t)min(u.tile * kKeysW + 128 * cw + 32 * h + lane, u.nkv - 1), pi = divu32(t, p.pg.div_ps);
        int page = p.pg.table[(int64_t)u.b * p.pg.max_pages + pi];
        if ((uint32_t)page >= (uint32_t)p.pg.num_pages) {      // outside the pool: any page of it
          set_dev_err(p.err, FA3_DEVERR_PAGE);
          page = 0;
        }
        const int at = (int)(t - pi * (uint32_t)p.pg.page_size);
        rows[h] = page * p.pg.page_size + at;
        factor[h] = key_factor(p, page, at, u.g);
        prefetch_line(p.k + u.g * kD + (int64_t)rows[h] * row_stride);
      }
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        uint4 r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          r[i] = load_once(base + (int64_t)__shfl_sync(0xffffffffu, rows[h], 4 * i + rl) * row_stride);
        if (h == 0) ok = warp_wait(bar(W_K_EMPTY), (units & 1u) ^ 1u, lane, abort_flag, p.err, p.wait_ticks);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint4 o0, o1;
          i8x4_to_bf16x4(r[i].x, o0.x, o0.y);
          i8x4_to_bf16x4(r[i].y, o0.z, o0.w);
          i8x4_to_bf16x4(r[i].z, o1.x, o1.y);
          i8x4_to_bf16x4(r[i].w, o1.z, o1.w);
          const uint32_t at = at0 ^ ((uint32_t)(i & 1) << 6);
          sts128(dst + (32 * h + 4 * i) * 128 + at, o0);
          sts128(dst + (32 * h + 4 * i) * 128 + (at ^ 16u), o1);
        }
        uint32_t a[3];
        three_parts(__fdiv_rn(1.f, factor[h]), a);
        sts128(sbase + OFF_KX + (uint32_t)cw * kSlice + (uint32_t)(32 * h + lane) * 16u,
               make_uint4(a[0] | a[0] << 16, a[1] | a[0] << 16, a[1] | a[2] << 16, a[1] | a[2] << 16));
      }
      if (!ok) break;
      fence_proxy_async();
      warp_arrive(W_K_FULL);
      ++units;
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------ sums of exponentials, a key a lane
    const int x = (warp - 4) >> 2, quarter = (warp - 4) & 3;  // row tile, quarter of its lanes
    const int r = 128 * x + quarter * 32 + lane;
    const uint32_t scol = tmem + ((uint32_t)(quarter * 32) << 16) + x * 128;
    uint32_t done = 0;                                        // steps of this row tile
    bool ok = true;
    while (ok && next_part()) {
      const PartW u = ring[parts % kRingW];
      part_read();
      const int t = u.tile * kKeysW + r, c = u.nkv - u.nq;
      float f;
      {
        const uint32_t tv = (uint32_t)min(t, u.nkv - 1), pi = divu32(tv, p.pg.div_ps);
        const int page = p.pg.table[(int64_t)u.b * p.pg.max_pages + pi];
        f = key_factor(p, page, (int)(tv - pi * (uint32_t)p.pg.page_size), u.g);
      }
      const SeqW sq = {u.q0, u.nq, u.nkv};
      const int rt0 = first_col_tile(p, sq, u.tile), seen = first_of_tile(p, sq, u.tile, x) - rt0;
      // From step `clear` on all rows see all of the row tile's keys (what lanes behind the context hold is not used); before step
      // `full` all 128 columns are rows.
      const int clear = (max(min(u.tile * kKeysW + 128 * x + 128, u.nkv) - 1 - c, 0) + p.P - 1) / p.P - rt0;
      const int full = p.P * p.G == kCols ? u.nq / p.P - rt0 : 0;
      float total = 0.f, lost = 0.f;                          // the sum, and what its roundings lost (Kahan)
      const int first = max(u.s0, seen);
      const float* const lse = p.lse + (int64_t)(u.q0 + rt0 * p.P) * p.Hq + u.g * p.G;   // the first column's
      float next = first < u.s1 ? lse[(int64_t)first * p.P * p.Hq] : 0.f;
#pragma unroll 1
      for (int s = first; s < u.s1; ++s) {
        const float mu = center_of(next);
        if (s + 1 < u.s1) next = lse[(int64_t)(s + 1) * p.P * p.Hq];
        ok = warp_wait(bar(W_S_FULL) + 8u * x, done & 1u, lane, abort_flag, p.err);
        if (!ok) break;
        ++done;
        tc_fence_after();
        float a0 = 0.f, a1 = 0.f, b0 = 0.f, b1 = 0.f;
        if (s >= clear && s < full) {
          uint32_t v[16];
          FA3_TMEM_LD16(scol, v);
#pragma unroll 1
          for (uint32_t k = 16;; k += 16) {
            wait_ld16(v);
            float y[16];
#pragma unroll
            for (int e = 0; e < 16; e += 2) fma2(y[e], y[e + 1], __uint_as_float(v[e]), __uint_as_float(v[e + 1]), f, f, mu, mu);
            if (k < kCols) {
              FA3_TMEM_LD16(scol + k, v);
            } else {
              tc_fence_before();                              // the scores are all in registers
              warp_arrive(W_S_EMPTY + x);
            }
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              add2(a0, a1, a0, a1, ex2_approx(y[e]), ex2_approx(y[e + 1]));
              add2(b0, b1, b0, b1, ex2_approx(y[e + 2]), ex2_approx(y[e + 3]));
            }
            if (k == kCols) break;
          }
        } else {
          // the first column that sees the key; the mask also drops what columns without a row hold
          const int i0 = (rt0 + s) * p.P, cols = min(p.P, u.nq - i0) * p.G, from = min(max(t - c - i0, 0), kCols) * p.G;
#pragma unroll 1
          for (int k = 0; k < cols; k += 16) {
            uint32_t v[16];
            FA3_TMEM_LD16(scol + k, v);
            wait_ld16(v);
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const float y = ex2_approx(fmaf(__uint_as_float(v[e]), f, mu)), z = ex2_approx(fmaf(__uint_as_float(v[e + 1]), f, mu));
              a0 += k + e >= from && k + e < cols ? y : 0.f;
              a1 += k + e + 1 >= from && k + e + 1 < cols ? z : 0.f;
            }
          }
          tc_fence_before();
          warp_arrive(W_S_EMPTY + x);
        }
        const float d = (a0 + a1) + (b0 + b1) - lost, z = total + d;
        lost = (z - total) - d;
        total = z;
      }
      if (!ok) break;
      if (u.s0 == 0 && u.s1 == u.n) {
        if (t < u.nkv) add_weight(p, u.b, u.g, t, t >= c, total);
      } else {
        p.part[(int64_t)(2 * (int)blockIdx.x + (u.s0 == 0 ? 1 : 0)) * kKeysW + r] = total;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// Adds up the parts of the unit whose first cut lies behind CTA blockIdx.x's part.
__global__ void __launch_bounds__(kKeysW) weights_combine_kernel(const __grid_constant__ WeightParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const CutW u = p.cuts[blockIdx.x];
  if (u.first < 0) return;
  const int nkv = p.kv_lens[u.b], nq = p.q_start[u.b + 1] - p.q_start[u.b], t = u.tile * kKeysW + (int)threadIdx.x;
  if (t >= nkv) return;
  float total = 0.f, lost = 0.f;
  for (int c = u.first; c <= u.last; ++c) {
    const float y = p.part[(int64_t)(2 * c + (c == u.first ? 1 : 0)) * kKeysW + threadIdx.x] - lost, z = total + y;
    lost = (z - total) - y;
    total = z;
  }
  add_weight(p, u.b, u.g, t, t >= nkv - nq, total);
}

size_t weights_bytes_of(int ctas) { return (size_t)ctas * (2 * kKeysW * sizeof(float) + sizeof(CutW)); }

}  // namespace
}  // namespace fa3

using namespace fa3;

FA3_API size_t fa3_attn_weights_workspace_size(void) {
  int sms = 0;
  if (check_device(&sms) != FA3_OK) sms = 152;
  return weights_bytes_of(sms);
}

FA3_API int fa3_attn_weights_gqa_block_paged(const uint16_t* q, const int8_t* k_cache, const float* k_scale, const float* lse,
                                             float* weights, const int32_t* q_start, const int32_t* kv_lens,
                                             const int32_t* block_table, int n, int B, int Hq, int Hkv, int D,
                                             int64_t q_stride, int num_pages, int page_size, int max_pages, int block,
                                             float softmax_scale, void* workspace, size_t workspace_bytes,
                                             int32_t* dev_err, void* stream) {
  if (!q || !k_cache || !k_scale || !lse || !weights || !q_start || !kv_lens) return FA3_EINVAL;
  if (n <= 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || Hq % Hkv != 0) return FA3_EINVAL;
  if (!(softmax_scale > 0.f) || !std::isfinite(softmax_scale)) return FA3_EINVAL;
  WeightParams p;
  int st = pages_of(block_table, B, Hkv, num_pages, page_size, max_pages, block, &p.pg);
  if (st != FA3_OK) return st;
  p.G = Hq / Hkv;
  if (D != kD || p.G > kCols || n >= (1 << 27) - 1 || q_stride < 0 || q_stride % 8 != 0) return FA3_ERANGE;
  if (n > 1 && q_stride < (int64_t)Hq * kD) return FA3_ERANGE;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned4(k_scale) || !aligned4(lse) || !aligned4(weights)) return FA3_ERANGE;
  int sms = 0;
  st = check_device(&sms);
  if (st != FA3_OK) return st;
  if (!workspace || workspace_bytes < weights_bytes_of(sms) || !aligned16(workspace)) return FA3_EWORKSPACE;
  if (few_rows_weights(n, B, Hkv, p.G, p.pg.T_max)) {
    const FewCall c = {q, k_cache, nullptr, k_scale, nullptr, q_start, kv_lens, nullptr, const_cast<float*>(lse), q_stride, n, B,
                       Hq, p.G, sms, softmax_scale * 1.4426950408889634f, dev_err};
    return cuda_status(few_rows_weights_attn(c, weights, block_table, num_pages, page_size, max_pages, block, Hkv,
                                             static_cast<cudaStream_t>(stream)));
  }
  p.k = k_cache; p.ks = k_scale; p.lse = lse; p.weights = weights; p.q_start = q_start; p.kv_lens = kv_lens;
  p.part = static_cast<float*>(workspace);
  p.cuts = reinterpret_cast<CutW*>(p.part + (size_t)2 * sms * kKeysW);
  p.err = dev_err; p.n = n; p.B = B; p.Hq = Hq; p.ctas = sms;
  // New tokens of a step: as many as fill its columns, but no more than a sequence has on average (a step's queries are
  // brought whole, also those that are another sequence's).
  p.P = std::max(1, std::min(kCols / p.G, (n + B - 1) / B));
  p.div_G = make_divu32((uint32_t)p.G);
  p.div_P = make_divu32((uint32_t)p.P);
  p.narrow = (double)Hkv * (p.pg.T_max / kKeysW + 1.0) * ((double)B * (kUnitSteps + 1) + (double)n / p.P) < 16777216.0;
  p.sm_log2 = softmax_scale * 1.4426950408889634f;
  p.wait_ticks = 4 * kWaitTicks + (uint32_t)(n / p.P >> 7);   // 4 s and 8 us a step
  const auto encode = tensor_map_encoder();
  if (!encode) return FA3_ECUDA;
  const cuuint64_t dims[3] = {kD, (cuuint64_t)Hq, (cuuint64_t)n};
  const cuuint64_t strides[2] = {kD * 2, (cuuint64_t)(n > 1 ? q_stride : (int64_t)Hq * kD) * 2};
  const cuuint32_t boxes[3] = {64, (cuuint32_t)p.G, (cuuint32_t)p.P}, step[3] = {1, 1, 1};
  if (encode(&p.map_q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(q), dims, strides, boxes, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return FA3_ECUDA;
  static std::atomic<bool> set[64];                          // the kernel's attribute, once a device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return FA3_ECUDA;
  if (dev >= 64 || !set[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(weights_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_WEIGHTS) != cudaSuccess)
      return FA3_ECUDA;
    if (dev < 64) set[dev].store(true, std::memory_order_release);
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const LaunchTogether together(s);
  if (launch_pdl(weights_kernel, dim3((unsigned)sms), dim3(kThreadsW), SMEM_WEIGHTS, s, p) != cudaSuccess) return FA3_ECUDA;
  return cuda_status(launch_pdl(weights_combine_kernel, dim3((unsigned)sms), dim3(kKeysW), 0, s, p));
}
