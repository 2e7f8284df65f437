// Attention of few packed rows a sequence (decode steps, drafts) over a block-scaled paged INT8 cache.
//
// The call's arithmetic is fa3_chunk.cu's (block-scaled variant); here it is HBM-bound: each KV byte meets a handful of
// query columns, too few for the 128 rows of tcgen05.mma.  A column is a new row's query head; a column tile is RT rows x the
// group's G heads, up to 8 NT columns (8, 16 or 32), as the N side of warp-level MMAs with 16 tokens as the M side:
//   * scores  S^T[16 tokens x 8 columns] = K . Q^T by m16n8k16 f16, int8 codes exact in fp16, bf16 queries exact after a
//     power of two by column; the contraction order is permuted so that a thread's K and Q words are the bytes it holds;
//   * x = s log2(e) + log2(value scale), P = 2^(x - m) as fp16, O^T += V^T . P^T on V's bare codes, and the row sum takes P
//     over the value scale: a step of 16 tokens lies in one block of the cache, so its scales are one number each;
//   * P lies 2^7 to 2^15 above fp16's normal range's end for the row's largest, which moves lazily.
//
// Work.  A unit is a column tile of one sequence and KV head; its steps of 16 tokens and all others lie on one line that is
// cut into equal parts, one per resident CTA, so ragged batches and one long context fill the GPU alike.  A CTA's four
// warps take a unit's steps in turn, each through its own cp.async ring, and merge at its end; a cut unit's parts meet in
// few_combine_kernel.
//
// What bounds it (one GB300, 64 query and 8 KV heads).  16 one-token rows of 4096 keys take 29.5 us, of 16384 keys 89 to 93 us and
// of 1024 14.5 us: HBM at 6.5 to 6.8 TB/s behind some 10 us that every call pays (launch, plan, a chain of lengths, page and first
// keys, the combine kernel).  With more columns the MMAs, conversions and exponentials of a step count as well: two rows each
// 33 us, four 46 (half of the issue slots, three and two warps a scheduler).  A merge by whoever comes last to a unit, in place
// of the second kernel, took 33.5 us for the first case.
#include "fa3_few.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

namespace fa3 {
namespace {

constexpr int kD = 128;
constexpr int kStep = 16;          // tokens of a warp's step
constexpr int kWarps = 4, kThreadsF = 32 * kWarps;
constexpr int kStageBytes = 2 * kStep * kD;                // K, then V rows
// The attention kernel's shared memory: rings, and where the columns are too many for registers their queries and constants.
template <int NT>
struct FewSmem {
  static constexpr bool kQueries = NT > 2;
  static constexpr int kStages = NT > 2 ? 4 : 2, kCtas = NT == 1 ? 4 : NT == 2 ? 3 : 2;   // of a ring; an SM
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kBytes = kRing + (kQueries ? NT * (4 * 32 + 4) * 16 : 0);
};

constexpr float kNone = -1e30f;    // the reference of a column that has seen no key
// What a unit costs beside its steps, and the least part of the line a CTA takes (enough for a part inside a unit to hold a
// step), in steps of a CTA's warp.
constexpr int kUnitSteps = 16, kLeastSteps = 20;
static_assert(kLeastSteps > kUnitSteps, "a part inside a unit, behind its fixed cost, holds a step");

struct CutF {
  int row0, cols, g, first, last;  // the unit's first row, columns and KV head, CTAs that have parts of it; first < 0: none begins here
};

struct FewParams {
  const uint16_t* q;
  const int8_t* k;
  const int8_t* v;
  const float* ks;
  const float* vs;
  const int32_t* q_start;
  const int32_t* kv_lens;
  __nv_bfloat16* out;
  float* lse;
  float* part_o;                   // [2 * CTAs][columns][128]
  float2* part_ml;                 // [2 * CTAs][columns]
  CutF* cuts;                      // [CTAs]
  int32_t* err;
  int64_t q_stride;
  Pages pg;
  int n, B, Hq, G, RT, ctas;
  DivU32 div_RT, div_G;
  float sm_log2;
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four signed int8 codes -> two f16x2 (exact).
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  lo = __byte_perm(u, 0x64646464u, 0x4140);
  hi = __byte_perm(u, 0x64646464u, 0x4342);
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(0x64806480u));
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(0x64806480u));
}
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Row values 4 lane .. 4 lane + 3 of a row whose weighted sum is a and whose weights' is l.  (A row sees a key at least, so l is
// positive where its scores are finite; infinite or NaN scores make l NaN, or 0 with all at -inf, and the row NaN.)
__device__ __forceinline__ void put_row(__nv_bfloat16* row, int lane, const float (&a)[4], float l) {
  const float inv = 1.f / l;
  const __nv_bfloat162 x = __floats2bfloat162_rn(a[0] * inv, a[1] * inv), y = __floats2bfloat162_rn(a[2] * inv, a[3] * inv);
  *reinterpret_cast<uint2*>(row + 4 * lane) = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}

struct SeqF {
  int q0, nq, nkv;
};
// nq = 0: nothing to do; -1: q_start falls.
template <class P>
__device__ __forceinline__ SeqF sequence_of(const P& p, int b, bool report) {
  SeqF s;
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
// Column tiles, and the cost of one (all of a sequence's count as its last).
__device__ __forceinline__ int tiles_of(const FewParams& p, const SeqF& s) {
  return s.nq > 0 ? (int)divu32((uint32_t)(s.nq + p.RT - 1), p.div_RT) : 0;
}
__device__ __forceinline__ int cost_of(const SeqF& s) { return kUnitSteps + (int)(((uint32_t)s.nkv + kStep - 1) / kStep); }
__device__ __forceinline__ uint32_t sequence_cost(const FewParams& p, const SeqF& s) {
  return s.nq > 0 ? (uint32_t)(tiles_of(p, s) * p.pg.Hkv * cost_of(s)) : 0u;
}

// The line's parts: CTA c takes [begin(c), begin(c + 1)).  Its numbers fit 31 bits (few_rows), and it is planned by every warp
// for itself, in registers: with 64-bit numbers, shared memory and barriers, the way to the first key took some 2 us more.
struct LineF {
  uint32_t total, each, rest;
  int parts;
  __device__ __forceinline__ uint32_t begin(int c) const {
    return c >= parts ? total : each * (uint32_t)c + rest * (uint32_t)c / (uint32_t)parts;
  }
  __device__ __forceinline__ int owner(uint32_t x) const {
    int c = min((int)(x / each), parts - 1);
    while (c > 0 && begin(c) > x) --c;
    while (c + 1 < parts && begin(c + 1) <= x) ++c;
    return c;
  }
};
struct Begin {
  SeqF s;
  int b;
  uint32_t off;                    // of the CTA's begin in sequence b
};
// The line, and the sequence that holds the begin of CTA `cta`'s part (the warp together; none if the part is empty).
template <class P>
__device__ __forceinline__ LineF find_begin(const P& p, int cta, int lane, Begin* at) {
  // a lane has `per` sequences that follow one another
  const int per = (p.B + 31) >> 5, b0 = lane * per;
  SeqF s = {0, 0, 0};
  uint32_t mine = 0;
  bool falls = false;
#pragma unroll 4
  for (int i = 0; i < per; ++i) {
    if (b0 + i < p.B) {
      s = sequence_of(p, b0 + i, cta == 0 && threadIdx.x < 32);
      falls |= s.nq < 0;
      mine += sequence_cost(p, s);
    }
  }
  uint32_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  LineF l;
  l.total = __any_sync(0xffffffffu, falls) ? 0u : __shfl_sync(0xffffffffu, upto, 31);
  l.parts = (int)max(1u, min(l.total / kLeastSteps, (uint32_t)p.ctas));
  l.each = l.total / (uint32_t)l.parts;
  l.rest = l.total - l.each * (uint32_t)l.parts;
  const uint32_t x = l.begin(cta);
  if (x >= l.total) return l;
  int k = __ffs(__ballot_sync(0xffffffffu, upto > x)) - 1;
  at->off = x - __shfl_sync(0xffffffffu, upto - mine, k);
  at->b = k * per;
#pragma unroll 1
  for (int base = 0; per > 1; base += 32) {                  // which of that lane's
    s = base + lane < per && at->b + base + lane < p.B ? sequence_of(p, at->b + base + lane, false) : SeqF{0, 0, 0};
    const uint32_t c = sequence_cost(p, s);
    uint32_t u = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, u, o);
      if (lane >= o) u += y;
    }
    const unsigned beyond = __ballot_sync(0xffffffffu, u > at->off);
    if (beyond) {
      k = __ffs(beyond) - 1;
      at->off -= __shfl_sync(0xffffffffu, u - c, k);
      at->b += base + k;
      break;
    }
    at->off -= __shfl_sync(0xffffffffu, u, 31);
  }
  at->s = SeqF{__shfl_sync(0xffffffffu, s.q0, k), __shfl_sync(0xffffffffu, s.nq, k), __shfl_sync(0xffffffffu, s.nkv, k)};
  return l;
}

template <int NT>
__global__ void __launch_bounds__(kThreadsF, FewSmem<NT>::kCtas) few_rows_kernel(const __grid_constant__ FewParams p) {
  // A 128-byte row stores its 16-byte chunk c at position c ^ f(row & 7), f(r) = (r & 6) ^ 4 (r & 1): every 8-lane
  // phase of the K and V fragment loads below then touches 8 distinct 16-byte bank groups.
  extern __shared__ __align__(128) uint8_t fsm[];
  constexpr int kCols = 8 * NT, kStages = FewSmem<NT>::kStages;
  constexpr bool kShared = FewSmem<NT>::kQueries;
  uint4* const sm_q = reinterpret_cast<uint4*>(fsm + FewSmem<NT>::kRing);   // [tile][4][32]: fragments of Q^T
  float4* const sm_c = reinterpret_cast<float4*>(sm_q + NT * 4 * 32);       // [tile][4]: two columns' factors and last keys
  float (*sm_o)[kCols][kD] = reinterpret_cast<float (*)[kCols][kD]>(fsm);   // at a unit's end, in the rings' place
  static_assert(kWarps * kCols * kD * 4 <= FewSmem<NT>::kRing, "partial O fits in the rings");
  __shared__ float sm_m[kWarps][kCols], sm_l[kWarps][kCols];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
  const int r = lane >> 2, qd = lane & 3;
  Begin w = {{0, 0, 0}, p.B, 0u};
  const LineF line = find_begin(p, cta, lane, &w);
  uint32_t x = line.begin(cta), left = line.begin(cta + 1) - x;
  CutF cut = {0, 0, 0, -1, -1};
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(fsm) + (uint32_t)(warp * kStages * kStageBytes);
  auto swz = [](int row) { return (row & 6) ^ ((row & 1) << 2); };
  auto chunk_addr = [&](uint32_t base, int row, int col) { return base + row * 128 + ((col ^ swz(row)) << 4); };
  const int64_t tok_stride = (int64_t)p.pg.Hkv * kD;

  SeqF s = w.s;
  int tile = 0, g = 0, off = 0;
  if (left > 0) {
    const uint32_t u = w.off / (uint32_t)cost_of(s);
    off = (int)(w.off - u * (uint32_t)cost_of(s));
    tile = (int)(u / (uint32_t)p.pg.Hkv);
    g = (int)u - tile * p.pg.Hkv;
  }
  while (left > 0) {
    const int cost = cost_of(s), take = (int)min((uint32_t)(cost - off), left);
    // the unit's rows, columns, keys and steps
    const int i0 = tile * p.RT, cols = min(p.RT, s.nq - i0) * p.G;
    const int c0 = s.nkv - s.nq, keys = c0 + min(s.nq, i0 + p.RT), steps = (keys + kStep - 1) / kStep;
    auto step_at = [&](int o) { return min(max(o - kUnitSteps, 0), steps); };
    const int s0 = step_at(off), s1 = off + take == cost ? steps : step_at(off + take);
    if (s0 < s1) {
      const bool whole = s0 == 0 && s1 == steps;
      // Q^T fragments: thread (r, qd) holds column 8 nt + r's values [16 qd, +16) and [64 + 16 qd, +16) as fp16, times a
      // power of two that brings the column's largest to [2^14, 2^15).  The values are asked for before all else.
      // (Where they are shared, a warp makes one tile's.)
      constexpr int NQ = kShared ? 1 : NT;
      static_assert(!kShared || NT == kWarps, "a tile a warp");
      uint4 qv[NQ][4];
#pragma unroll
      for (int nt = 0; nt < NQ; ++nt) {
        const int col = 8 * (kShared ? warp : nt) + r, ri = (int)divu32((uint32_t)col, p.div_G);
        const uint16_t* row = p.q + (int64_t)(s.q0 + i0 + ri) * p.q_stride + (int64_t)(g * p.G + col - ri * p.G) * kD;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          qv[nt][i] = col < cols ? *reinterpret_cast<const uint4*>(row + (i >> 1) * 64 + 16 * qd + 8 * (i & 1))
                                 : make_uint4(0u, 0u, 0u, 0u);
      }
      const int n_my = s1 - s0 > warp ? (s1 - s0 - warp + kWarps - 1) / kWarps : 0;   // steps s0 + warp, + 4, ...
      // A lane looks one of the next 32 steps up: its first row in the pool, and its scales.
      int row_of = 0;
      float ks_of = 0.f, lv_of = 0.f, rv_of = 0.f, ks_next = 0.f, vs_next = 0.f;
      auto look_up = [&](int m) {
        const uint32_t t = (uint32_t)((s0 + warp + kWarps * min(m + lane, n_my - 1)) * kStep), pi = divu32(t, p.pg.div_ps);
        int page = p.pg.table[(int64_t)w.b * p.pg.max_pages + pi];
        if ((uint32_t)page >= (uint32_t)p.pg.num_pages) {           // outside the pool: any page of it
          set_dev_err(p.err, FA3_DEVERR_PAGE);
          page = 0;
        }
        const int at = (int)(t - pi * (uint32_t)p.pg.page_size);
        row_of = page * p.pg.page_size + at;
        const int64_t sc = ((int64_t)page * p.pg.per_page + (int)divu32((uint32_t)at, p.pg.div_block)) * p.pg.Hkv + g;
        ks_next = p.ks[sc];
        vs_next = p.vs[sc];
      };
      // A step's 16 rows of K and of V: a lane has 16 bytes of rows l / 8, l / 8 + 4, ..  Rows behind the context are read as
      // they are (they lie in the same page) and masked.
      const int64_t lane_off = (int64_t)(lane >> 3) * tok_stride + g * kD + (lane & 7) * 16;
      const uint32_t lane_dst = ring + (uint32_t)(lane >> 3) * 128;
      const uint32_t dst_even = ((lane & 7) ^ swz(lane >> 3)) << 4, dst_odd = ((lane & 7) ^ swz((lane >> 3) + 4)) << 4;
      auto issue = [&](int m, int stage) {
        const int64_t at = (int64_t)__shfl_sync(0xffffffffu, row_of, m & 31) * tok_stride + lane_off;
        const int8_t *ka = p.k + at, *va = p.v + at;
        const uint32_t dst = lane_dst + stage * kStageBytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          cp_async16(dst + 512 * i + (i & 1 ? dst_odd : dst_even), ka + 4 * i * tok_stride);
          cp_async16(dst + 2048 + 512 * i + (i & 1 ? dst_odd : dst_even), va + 4 * i * tok_stride);
        }
      };
      if (n_my > 0) look_up(0);
#pragma unroll
      for (int m = 0; m < kStages - 1; ++m) {
        if (m < n_my) issue(m, m);
        cp_async_commit();
      }
      uint32_t qh[NQ][8][2];
      float f0[NQ], f1[NQ];
      int lim0[NQ], lim1[NQ];                                   // last key of columns 8 nt + 2 qd, + 1; -1: no column
#pragma unroll
      for (int nt = 0; nt < NQ; ++nt) {
        const uint4 (&v)[4] = qv[nt];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu),
                                       __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu)));
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t e = max(top >> 7, 15u);                  // the largest's exponent: 2^(e - 127)
        const float f = __uint_as_float((268u - e) << 23);
        auto two = [&](uint32_t y) { return pack_f16x2(__uint_as_float(y << 16) * f, __uint_as_float(y & 0xffff0000u) * f); };
#pragma unroll
        for (int st = 0; st < 8; ++st) {
          qh[nt][st][0] = two(word(v[st >> 1], 2 * (st & 1)));
          qh[nt][st][1] = two(word(v[st >> 1], 2 * (st & 1) + 1));
        }
        const float inv = __uint_as_float((e - 14u) << 23) * p.sm_log2;
        f0[nt] = __shfl_sync(0xffffffffu, inv, 4 * (2 * qd));
        f1[nt] = __shfl_sync(0xffffffffu, inv, 4 * (2 * qd + 1));
        const int ca = 8 * (kShared ? warp : nt) + 2 * qd;
        lim0[nt] = ca < cols ? c0 + i0 + (int)divu32((uint32_t)ca, p.div_G) : -1;
        lim1[nt] = ca + 1 < cols ? c0 + i0 + (int)divu32((uint32_t)(ca + 1), p.div_G) : -1;
      }
      if constexpr (kShared) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          sm_q[(warp * 4 + i) * 32 + lane] = make_uint4(qh[0][2 * i][0], qh[0][2 * i][1], qh[0][2 * i + 1][0], qh[0][2 * i + 1][1]);
        if (r == 0) sm_c[warp * 4 + qd] = make_float4(f0[0], f1[0], __int_as_float(lim0[0]), __int_as_float(lim1[0]));
        __syncthreads();
      }
      // kNone in place of -infinity: differences of references stay numbers
      float m0[NT], m1[NT], l0[NT], l1[NT], o[NT][8][4];
      const int lim = cols == kCols ? c0 + i0 : -1;             // the last key that all columns see
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        m0[nt] = m1[nt] = kNone;
        l0[nt] = l1[nt] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
      }
      for (int m = 0; m < n_my; ++m) {
        const int t0 = (s0 + warp + kWarps * m) * kStep;
        if ((m & 31) == 0) {
          const float vs = fmaxf(vs_next, kLeastScale);
          ks_of = ks_next;
          lv_of = __log2f(vs);
          rv_of = __fdividef(1.f, vs);
        }
        const float ks = __shfl_sync(0xffffffffu, ks_of, m & 31), lv = __shfl_sync(0xffffffffu, lv_of, m & 31),
                    rv = __shfl_sync(0xffffffffu, rv_of, m & 31);
        if (m + kStages - 1 < n_my) {
          if (((m + kStages - 1) & 31) == 0) look_up(m + kStages - 1);
          issue(m + kStages - 1, (m + kStages - 1) % kStages);
        }
        cp_async_commit();
        cp_async_wait<kStages - 1>();
        __syncwarp();
        const uint32_t kst = ring + (m % kStages) * kStageBytes, vst = kst + 2048;
        float cf[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) cf[nt][0] = cf[nt][1] = cf[nt][2] = cf[nt][3] = 0.f;
        {
          const uint4 k0 = lds128(chunk_addr(kst, r, qd)), k1 = lds128(chunk_addr(kst, r, 4 + qd)),
                      k2 = lds128(chunk_addr(kst, r + 8, qd)), k3 = lds128(chunk_addr(kst, r + 8, 4 + qd));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t ka[2][4];                                  // row r: the thread's values 4 st .. 4 st + 3; row r + 8
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int st = 2 * i + e;
              codes_to_f16(word(st < 4 ? k0 : k1, st & 3), ka[e][0], ka[e][2]);
              codes_to_f16(word(st < 4 ? k2 : k3, st & 3), ka[e][1], ka[e][3]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint4 b;
              if constexpr (kShared) b = sm_q[(nt * 4 + i) * 32 + lane];
              else b = make_uint4(qh[nt][2 * i][0], qh[nt][2 * i][1], qh[nt][2 * i + 1][0], qh[nt][2 * i + 1][1]);
              mma16816(cf[nt], ka[0][0], ka[0][1], ka[0][2], ka[0][3], b.x, b.y);
              mma16816(cf[nt], ka[1][0], ka[1][1], ka[1][2], ka[1][3], b.z, b.w);
            }
          }
        }
        const uint4 v0 = lds128(chunk_addr(vst, 2 * qd, r)), v1 = lds128(chunk_addr(vst, 2 * qd + 1, r)),
                    v2 = lds128(chunk_addr(vst, 2 * qd + 8, r)), v3 = lds128(chunk_addr(vst, 2 * qd + 9, r));
        __syncwarp();                                           // every lane has its fragments: the stage may be refilled
        const bool masked = t0 + kStep - 1 > lim;
        uint32_t b0[NT], b1[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float fa, fb;
          int la, lb;
          if constexpr (kShared) {
            const float4 c = sm_c[nt * 4 + qd];
            fa = c.x, fb = c.y, la = __float_as_int(c.z), lb = __float_as_int(c.w);
          } else {
            fa = f0[nt], fb = f1[nt], la = lim0[nt], lb = lim1[nt];
          }
          const float e0 = fa * ks, e1 = fb * ks;
          float y[4];
          auto exponents = [&]() {                              // of tokens r, r + 8 and columns 2 qd, 2 qd + 1
            const float a0 = lv - m0[nt], a1 = lv - m1[nt];
            y[0] = fmaf(cf[nt][0], e0, a0);
            y[1] = fmaf(cf[nt][1], e1, a1);
            y[2] = fmaf(cf[nt][2], e0, a0);
            y[3] = fmaf(cf[nt][3], e1, a1);
            if (masked) {
              const int ta = t0 + r, tb = ta + 8;
              y[0] = ta <= la ? y[0] : -CUDART_INF_F;
              y[1] = ta <= lb ? y[1] : -CUDART_INF_F;
              y[2] = tb <= la ? y[2] : -CUDART_INF_F;
              y[3] = tb <= lb ? y[3] : -CUDART_INF_F;
            }
          };
          exponents();
          // The reference lies 7 below the column's largest when it is set, and moves when one is 15 or more above it:
          // P stays below 2^15 (a little above, by the rounding of y), which is below fp16's end.
          if (__any_sync(0xffffffffu, fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])) > 15.f)) {
            auto x_of = [&](int e) { return y[e] == -CUDART_INF_F ? y[e] : fmaf(cf[nt][e], e & 1 ? e1 : e0, lv); };
            float x0 = fmaxf(x_of(0), x_of(2)), x1 = fmaxf(x_of(1), x_of(3));
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) {
              x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, k));
              x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, k));
            }
            const float n0 = x0 - 7.f > m0[nt] + 8.f ? x0 - 7.f : m0[nt], n1 = x1 - 7.f > m1[nt] + 8.f ? x1 - 7.f : m1[nt];
            const float al0 = ex2_approx(m0[nt] - n0), al1 = ex2_approx(m1[nt] - n1);
            l0[nt] *= al0;
            l1[nt] *= al1;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              o[nt][i][0] *= al0; o[nt][i][1] *= al1; o[nt][i][2] *= al0; o[nt][i][3] *= al1;
            }
            m0[nt] = n0;
            m1[nt] = n1;
            exponents();
          }
          const float p0 = ex2_approx(y[0]), p1 = ex2_approx(y[1]), p2 = ex2_approx(y[2]), p3 = ex2_approx(y[3]);
          l0[nt] = fmaf(p0 + p2, rv, l0[nt]);
          l1[nt] = fmaf(p1 + p3, rv, l1[nt]);
          b0[nt] = movmatrix_trans(pack_f16x2(p0, p1));
          b1[nt] = movmatrix_trans(pack_f16x2(p2, p3));
        }
        // O^T += V^T . P^T; m-tile i covers values 16 r + 2 i (row r) and 16 r + 2 i + 1 (row r + 8)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
          uint32_t a0, a1, a2, a3;
          codes_to_f16(__byte_perm(word(v0, i >> 1), word(v1, i >> 1), sel), a0, a1);
          codes_to_f16(__byte_perm(word(v2, i >> 1), word(v3, i >> 1), sel), a2, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][i], a0, a1, a2, a3, b0[nt], b1[nt]);
        }
      }
      cp_async_wait<0>();
      // ---- merge the warps (the rings become the partial-O buffer)
      __syncthreads();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int o_ = 4; o_ < 32; o_ <<= 1) {
          l0[nt] += __shfl_xor_sync(0xffffffffu, l0[nt], o_);
          l1[nt] += __shfl_xor_sync(0xffffffffu, l1[nt], o_);
        }
        const int ca = 8 * nt + 2 * qd;
        if (r == 0) {
          sm_m[warp][ca] = m0[nt]; sm_m[warp][ca + 1] = m1[nt];
          sm_l[warp][ca] = l0[nt]; sm_l[warp][ca + 1] = l1[nt];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          *reinterpret_cast<float2*>(&sm_o[warp][ca][16 * r + 2 * i]) = make_float2(o[nt][i][0], o[nt][i][2]);
          *reinterpret_cast<float2*>(&sm_o[warp][ca + 1][16 * r + 2 * i]) = make_float2(o[nt][i][1], o[nt][i][3]);
        }
      }
      __syncthreads();
      // a warp has every fourth column, a lane four values
      for (int col = warp; col < cols; col += kWarps) {
        float M = kNone;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) M = fmaxf(M, sm_m[k][col]);
        float L = 0.f, a[4] = {};
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
          const float fk = ex2_approx(sm_m[k][col] - M);
          const float4 ok = *reinterpret_cast<const float4*>(&sm_o[k][col][4 * lane]);
          L = fmaf(sm_l[k][col], fk, L);
          a[0] = fmaf(ok.x, fk, a[0]); a[1] = fmaf(ok.y, fk, a[1]); a[2] = fmaf(ok.z, fk, a[2]); a[3] = fmaf(ok.w, fk, a[3]);
        }
        const int ri = (int)divu32((uint32_t)col, p.div_G);
        const int64_t orow = (int64_t)(s.q0 + i0 + ri) * p.Hq + g * p.G + col - ri * p.G;
        if (whole) {
          put_row(p.out + orow * kD, lane, a, L);
          if (lane == 0 && p.lse) p.lse[orow] = log_sum(M, L);
        } else {
          const int64_t slot = (int64_t)(2 * cta + (s0 == 0 ? 1 : 0)) * kCols + col;
          *reinterpret_cast<float4*>(p.part_o + slot * kD + 4 * lane) = make_float4(a[0], a[1], a[2], a[3]);
          if (lane == 0) p.part_ml[slot] = make_float2(M, L);
        }
      }
      // The part that begins a unit records its cut; the costs count some steps that only the last tile has, so the last CTA
      // with any is the one that holds the last step.
      if (s0 == 0 && !whole) cut = CutF{s.q0 + i0, cols, g, cta, line.owner(x + (uint32_t)(kUnitSteps + steps - off) - 1u)};
      __syncthreads();                                          // the rings are the next unit's
    }
    left -= take;
    x += take;
    off = 0;
    if (++g == p.pg.Hkv) {
      g = 0;
      if (++tile == tiles_of(p, s) && left > 0) {
        tile = 0;
        do {
          s = ++w.b < p.B ? sequence_of(p, w.b, false) : SeqF{0, 1, 0};
        } while (s.nq <= 0);
      }
    }
  }
  if (tid == 0) p.cuts[cta] = cut;
}

// Merges the parts of the unit whose first cut lies behind CTA blockIdx.x's part.  MW warps have a column, each every MW-th
// part, eight at once.
constexpr int kMergeCols = 4, kMergeLoads = 8;
template <int NT, int MW>
__global__ void __launch_bounds__(32 * MW * kMergeCols) few_combine_kernel(const __grid_constant__ FewParams p) {
  constexpr int kCols = 8 * NT;
  __shared__ float4 sm_a[kMergeCols][MW][32];
  __shared__ float2 sm_ml[kMergeCols][MW];
  // No early start of what follows: its blocks would be placed around these, and the next attention call's, which fill the GPU
  // exactly, unevenly (16 one-token rows of 4096 keys 36.2 us a call instead of 32.0, of 16384 keys 107 instead of 89).
  pdl_wait();
  const CutF u = p.cuts[blockIdx.x];
  if (u.first < 0) return;
  const int lane = threadIdx.x & 31, part = (threadIdx.x >> 5) % MW, mine = threadIdx.x / (32 * MW);
  const int col = blockIdx.y * kMergeCols + mine;
  float M = kNone, L = 0.f, a[4] = {};
  if (col < u.cols) {
    auto slot = [&](int c) { return (int64_t)(2 * c + (c == u.first ? 1 : 0)) * kCols + col; };
#pragma unroll 1
    for (int c = u.first + part; c <= u.last; c += kMergeLoads * MW) {
      float2 ml[kMergeLoads];
      float4 o[kMergeLoads];
#pragma unroll
      for (int k = 0; k < kMergeLoads; ++k) {
        const int64_t at = slot(min(c + k * MW, u.last));
        ml[k] = p.part_ml[at];
        o[k] = *reinterpret_cast<const float4*>(p.part_o + at * kD + 4 * lane);
      }
      float top = M;
#pragma unroll
      for (int k = 0; k < kMergeLoads; ++k) top = fmaxf(top, ml[k].x);
      const float f = ex2_approx(M - top);
      L *= f;
#pragma unroll
      for (int e = 0; e < 4; ++e) a[e] *= f;
      M = top;
#pragma unroll
      for (int k = 0; k < kMergeLoads; ++k) {
        const float fk = c + k * MW <= u.last ? ex2_approx(ml[k].x - M) : 0.f;
        L = fmaf(ml[k].y, fk, L);
        a[0] = fmaf(o[k].x, fk, a[0]); a[1] = fmaf(o[k].y, fk, a[1]); a[2] = fmaf(o[k].z, fk, a[2]); a[3] = fmaf(o[k].w, fk, a[3]);
      }
    }
  }
  if constexpr (MW > 1) {
    sm_a[mine][part][lane] = make_float4(a[0], a[1], a[2], a[3]);
    if (lane == 0) sm_ml[mine][part] = make_float2(M, L);
    __syncthreads();
    if (part) return;
    M = kNone;
#pragma unroll
    for (int k = 0; k < MW; ++k) M = fmaxf(M, sm_ml[mine][k].x);
    L = a[0] = a[1] = a[2] = a[3] = 0.f;
#pragma unroll
    for (int k = 0; k < MW; ++k) {
      const float2 ml = sm_ml[mine][k];
      const float4 o = sm_a[mine][k][lane];
      const float f = ex2_approx(ml.x - M);
      L = fmaf(ml.y, f, L);
      a[0] = fmaf(o.x, f, a[0]); a[1] = fmaf(o.y, f, a[1]); a[2] = fmaf(o.z, f, a[2]); a[3] = fmaf(o.w, f, a[3]);
    }
  }
  if (col >= u.cols) return;
  const int ri = (int)divu32((uint32_t)col, p.div_G);
  const int64_t orow = (int64_t)(u.row0 + ri) * p.Hq + u.g * p.G + col - ri * p.G;
  put_row(p.out + orow * kD, lane, a, L);
  if (lane == 0 && p.lse) p.lse[orow] = log_sum(M, L);
}

// ------------------------------------------------------------------ attention weights of few rows
// fa3_weights.cu's sums where few columns meet each key: only keys are read, once for every 64 columns of a sequence, and the
// scores are those above, with the sum over columns (2 a thread, then the four threads of a token) in place of the softmax.
// Tokens have nothing to do with one another, so a part of the line is a run of tokens and there is nothing to merge.
// 16 one-token rows of 4096 keys, 64 query and 8 KV heads: 17.6 us, 10 of them HBM's; each 8 columns more take 2.6 us
// (MMAs and exponentials).
constexpr int kChunkCols = 64, kWStages = 3;
constexpr uint32_t kWRing = kWarps * kWStages * kStep * kD;                    // int8 rows of K
constexpr uint32_t OFF_WQ = kWRing;                                            // [tile][4][32] uint4: fragments of Q^T
constexpr uint32_t OFF_WC = OFF_WQ + kChunkCols / 8 * 4 * 32 * 16;             // [tile][4] float4: two columns' factors and -lse
constexpr uint32_t OFF_WL = OFF_WC + kChunkCols / 8 * 4 * 16;                  // [tile][4] int2: the last key that sees them
constexpr uint32_t SMEM_FEW_WEIGHTS = OFF_WL + kChunkCols / 8 * 4 * 8;
constexpr int kWUnit = 16;         // what a unit costs beside its steps

struct FewWeightParams {
  const uint16_t* q;
  const int8_t* k;
  const float* ks;
  const float* lse;
  float* weights;
  const int32_t* q_start;
  const int32_t* kv_lens;
  int32_t* err;
  int64_t q_stride;
  Pages pg;
  int n, B, Hq, G, RC, ctas;       // RC: rows of a chunk
  DivU32 div_RC, div_G;
  float sm_log2;
};
__device__ __forceinline__ int chunks_of(const FewWeightParams& p, const SeqF& s) { return (int)divu32((uint32_t)(s.nq + p.RC - 1), p.div_RC); }
__device__ __forceinline__ uint32_t unit_cost(const FewWeightParams& p, const SeqF& s) {
  return kWUnit + (uint32_t)(((uint32_t)s.nkv + kStep - 1) / kStep) * (uint32_t)chunks_of(p, s);
}
__device__ __forceinline__ uint32_t sequence_cost(const FewWeightParams& p, const SeqF& s) {
  return s.nq > 0 ? (uint32_t)p.pg.Hkv * unit_cost(p, s) : 0u;
}

__global__ void __launch_bounds__(kThreadsF, 4) few_weights_kernel(const __grid_constant__ FewWeightParams p) {
  extern __shared__ __align__(128) uint8_t fsm[];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
  const int r = lane >> 2, qd = lane & 3;
  Begin w = {{0, 0, 0}, p.B, 0u};
  const LineF line = find_begin(p, cta, lane, &w);
  uint32_t left = line.begin(cta + 1) - line.begin(cta);
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(fsm) + (uint32_t)(warp * kWStages * kStep * kD);
  auto swz = [](int row) { return (row & 6) ^ ((row & 1) << 2); };
  auto chunk_addr = [&](uint32_t base, int row, int col) { return base + row * 128 + ((col ^ swz(row)) << 4); };
  const int64_t tok_stride = (int64_t)p.pg.Hkv * kD;
  uint4* const sm_q = reinterpret_cast<uint4*>(fsm + OFF_WQ);
  float4* const sm_c = reinterpret_cast<float4*>(fsm + OFF_WC);
  int2* const sm_lim = reinterpret_cast<int2*>(fsm + OFF_WL);
  SeqF s = w.s;
  int g = 0;
  uint32_t off = 0;
  if (left > 0) {
    g = (int)(w.off / unit_cost(p, s));
    off = w.off - (uint32_t)g * unit_cost(p, s);
  }
  while (left > 0) {
    const uint32_t cost = unit_cost(p, s), take = min(cost - off, left);
    const int chunks = chunks_of(p, s), c0 = s.nkv - s.nq;
    // a part begins with the first step that begins behind its begin
    auto step_at = [&](uint32_t o) { return o <= kWUnit ? 0 : (int)((o - kWUnit + (uint32_t)chunks - 1u) / (uint32_t)chunks); };
    const int s0 = step_at(off), s1 = step_at(off + take);
    const int n_my = s1 - s0 > warp ? (s1 - s0 - warp + kWarps - 1) / kWarps : 0;   // steps s0 + warp, + 4, ...
    for (int chunk = 0; chunk < chunks && s0 < s1; ++chunk) {
      const int i0 = chunk * p.RC, cols = min(p.RC, s.nq - i0) * p.G, tiles = (cols + 7) >> 3;
      // A lane looks one of the next 32 steps up: its page and row there, and its scale.
      int page_of = 0, at_of = 0;
      float ks_of = 0.f, ks_next = 0.f;
      int page_next = 0, at_next = 0;
      auto look_up = [&](int m) {
        const uint32_t t = (uint32_t)((s0 + warp + kWarps * min(m + lane, n_my - 1)) * kStep), pi = divu32(t, p.pg.div_ps);
        page_next = p.pg.table[(int64_t)w.b * p.pg.max_pages + pi];
        at_next = (int)(t - pi * (uint32_t)p.pg.page_size);
        if ((uint32_t)page_next >= (uint32_t)p.pg.num_pages) {      // outside the pool: its tokens get nothing
          set_dev_err(p.err, FA3_DEVERR_PAGE);
          page_next = -1;
        }
        ks_next = p.ks[((int64_t)max(page_next, 0) * p.pg.per_page + (int)divu32((uint32_t)at_next, p.pg.div_block)) * p.pg.Hkv + g];
      };
      const int64_t lane_off = (int64_t)(lane >> 3) * tok_stride + g * kD + (lane & 7) * 16;
      const uint32_t lane_dst = ring + (uint32_t)(lane >> 3) * 128;
      const uint32_t dst_even = ((lane & 7) ^ swz(lane >> 3)) << 4, dst_odd = ((lane & 7) ^ swz((lane >> 3) + 4)) << 4;
      auto issue = [&](int m) {
        const int pg = __shfl_sync(0xffffffffu, page_next, m & 31), at = __shfl_sync(0xffffffffu, at_next, m & 31);
        const int8_t* ka = p.k + ((int64_t)max(pg, 0) * p.pg.page_size + at) * tok_stride + lane_off;
        const uint32_t dst = lane_dst + (m % kWStages) * (kStep * kD);
#pragma unroll
        for (int i = 0; i < 4; ++i) cp_async16(dst + 512 * i + (i & 1 ? dst_odd : dst_even), ka + 4 * i * tok_stride);
      };
      if (n_my > 0) look_up(0);
#pragma unroll
      for (int m = 0; m < kWStages - 1; ++m) {
        if (m < n_my) issue(m);
        cp_async_commit();
      }
      // Q^T fragments as above, a tile of 8 columns a warp
      for (int tile = warp; tile < tiles; tile += kWarps) {
        const int col = 8 * tile + r, ri = (int)divu32((uint32_t)col, p.div_G), h = g * p.G + col - ri * p.G;
        const int64_t row = s.q0 + i0 + ri;
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = col < cols ? *reinterpret_cast<const uint4*>(p.q + row * p.q_stride + (int64_t)h * kD + (i >> 1) * 64 +
                                                                  16 * qd + 8 * (i & 1))
                            : make_uint4(0u, 0u, 0u, 0u);
        const float lse = col < cols ? p.lse[row * p.Hq + h] * -1.4426950408889634f : 0.f;
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu),
                                       __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu)));
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t e = max(top >> 7, 15u);
        const float f = __uint_as_float((268u - e) << 23), inv = __uint_as_float((e - 14u) << 23) * p.sm_log2;
        auto two = [&](uint32_t y) { return pack_f16x2(__uint_as_float(y << 16) * f, __uint_as_float(y & 0xffff0000u) * f); };
#pragma unroll
        for (int i = 0; i < 4; ++i)
          sm_q[(tile * 4 + i) * 32 + lane] = make_uint4(two(v[i].x), two(v[i].y), two(v[i].z), two(v[i].w));
        const int lim = col < cols ? c0 + i0 + ri : -1;
        const float f0 = __shfl_sync(0xffffffffu, inv, 8 * qd), f1 = __shfl_sync(0xffffffffu, inv, 8 * qd + 4);
        const float l0 = __shfl_sync(0xffffffffu, lse, 8 * qd), l1 = __shfl_sync(0xffffffffu, lse, 8 * qd + 4);
        const int m0 = __shfl_sync(0xffffffffu, lim, 8 * qd), m1 = __shfl_sync(0xffffffffu, lim, 8 * qd + 4);
        if (r == 0) {
          sm_c[tile * 4 + qd] = make_float4(f0, f1, l0, l1);
          sm_lim[tile * 4 + qd] = make_int2(m0, m1);
        }
      }
      __syncthreads();
      const int lim_min = (cols & 7) ? -1 : c0 + i0;             // the last key that all of the chunk's columns see
      for (int m = 0; m < n_my; ++m) {
        const int t0 = (s0 + warp + kWarps * m) * kStep;
        if ((m & 31) == 0) page_of = page_next, at_of = at_next, ks_of = ks_next;
        const float ks = __shfl_sync(0xffffffffu, ks_of, m & 31);
        const int page = __shfl_sync(0xffffffffu, page_of, m & 31), at = __shfl_sync(0xffffffffu, at_of, m & 31);
        if (m + kWStages - 1 < n_my) {
          if (((m + kWStages - 1) & 31) == 0) look_up(m + kWStages - 1);
          issue(m + kWStages - 1);
        }
        cp_async_commit();
        cp_async_wait<kWStages - 1>();
        __syncwarp();
        const uint32_t kst = ring + (m % kWStages) * (kStep * kD);
        uint32_t a[8][4];
        {
          const uint4 k0 = lds128(chunk_addr(kst, r, qd)), k1 = lds128(chunk_addr(kst, r, 4 + qd)),
                      k2 = lds128(chunk_addr(kst, r + 8, qd)), k3 = lds128(chunk_addr(kst, r + 8, 4 + qd));
#pragma unroll
          for (int st = 0; st < 8; ++st) {
            codes_to_f16(word(st < 4 ? k0 : k1, st & 3), a[st][0], a[st][2]);
            codes_to_f16(word(st < 4 ? k2 : k3, st & 3), a[st][1], a[st][3]);
          }
        }
        __syncwarp();                                            // every lane has its fragments: the stage may be refilled
        const bool masked = t0 + kStep - 1 > lim_min;
        const int ta = t0 + r, tb = ta + 8;
        float sa = 0.f, sb = 0.f;
        // N column tiles at once: a tile's MMAs are a chain (16 sequences of 4096 keys, 64 columns each: 39.4 us one by one, 36.1 by
        // twos, 36.1 by fours)
        auto add = [&](auto n, int tile) {
          constexpr int N = decltype(n)::value;
          float cf[N][4] = {};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int k = 0; k < N; ++k) {
              const uint4 b = sm_q[((tile + k) * 4 + i) * 32 + lane];
              mma16816(cf[k], a[2 * i][0], a[2 * i][1], a[2 * i][2], a[2 * i][3], b.x, b.y);
              mma16816(cf[k], a[2 * i + 1][0], a[2 * i + 1][1], a[2 * i + 1][2], a[2 * i + 1][3], b.z, b.w);
            }
          }
#pragma unroll
          for (int k = 0; k < N; ++k) {
            const float4 c = sm_c[(tile + k) * 4 + qd];
            const float e0 = c.x * ks, e1 = c.y * ks;
            float y0 = ex2_approx(fmaf(cf[k][0], e0, c.z)), y1 = ex2_approx(fmaf(cf[k][1], e1, c.w)),
                  y2 = ex2_approx(fmaf(cf[k][2], e0, c.z)), y3 = ex2_approx(fmaf(cf[k][3], e1, c.w));
            if (masked) {
              const int2 lim = sm_lim[(tile + k) * 4 + qd];
              y0 = ta <= lim.x ? y0 : 0.f;
              y1 = ta <= lim.y ? y1 : 0.f;
              y2 = tb <= lim.x ? y2 : 0.f;
              y3 = tb <= lim.y ? y3 : 0.f;
            }
            sa += y0 + y1;
            sb += y2 + y3;
          }
        };
        int tile = 0;
#pragma unroll 1
        for (; tile + 2 <= tiles; tile += 2) add(std::integral_constant<int, 2>(), tile);
        if (tile < tiles) add(std::integral_constant<int, 1>(), tile);
        sa += __shfl_xor_sync(0xffffffffu, sa, 1);
        sb += __shfl_xor_sync(0xffffffffu, sb, 1);
        sa += __shfl_xor_sync(0xffffffffu, sa, 2);
        sb += __shfl_xor_sync(0xffffffffu, sb, 2);
        const int t = qd ? tb : ta;
        if (qd < 2 && page >= 0 && t < s.nkv) {
          float* to = p.weights + ((int64_t)page * p.pg.Hkv + g) * p.pg.page_size + at + r + 8 * qd;
          // a new token begins with nothing; old ones may lie in pages that sequences share
          if (t >= c0 && chunk == 0)
            *to = qd ? sb : sa;
          else
            atomicAdd(to, qd ? sb : sa);
        }
      }
      cp_async_wait<0>();
      __syncthreads();                                           // the fragments are the next chunk's
    }
    left -= take;
    off = 0;
    if (++g == p.pg.Hkv && left > 0) {
      g = 0;
      do {
        s = ++w.b < p.B ? sequence_of(p, w.b, false) : SeqF{0, 1, 0};
      } while (s.nq <= 0);
    }
  }
}

// Columns of a sequence on average (whole rows, for some of n may be nobody's).
int64_t columns_of(int n, int B, int G) { return (int64_t)std::max(1, n / B) * G; }
// Units of 8, 16 or 32 columns, as sequences have on average.  16 sequences of 4096 keys, 16 columns each: 33 us in units of 16,
// 43 of 32; 32 columns: 54.5 in two units of 16, 46 in one of 32, whose keys are read and converted once (but half as many
// warps are there to hide the waits, and its queries have to lie in shared memory).
int n_tiles(int n, int B, int G) {
  const int64_t cols = columns_of(n, B, G);
  return cols <= 8 ? 1 : cols <= 16 ? 2 : 4;
}
int ctas_of(int nt, int sms) { return sms * (nt == 1 ? FewSmem<1>::kCtas : nt == 2 ? FewSmem<2>::kCtas : FewSmem<4>::kCtas); }
size_t bytes_of(int nt, int ctas) {
  return (size_t)ctas * (2 * 8 * nt * (kD * sizeof(float) + sizeof(float2)) + sizeof(CutF));
}

template <int NT>
cudaError_t launch(FewParams& p, void* workspace, cudaStream_t s) {
  static std::atomic<bool> set[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return cudaErrorInvalidDevice;
  if (dev >= 64 || !set[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(few_rows_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, FewSmem<NT>::kBytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) set[dev].store(true, std::memory_order_release);
  }
  p.RT = 8 * NT / p.G;
  p.div_RT = make_divu32((uint32_t)p.RT);
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + (size_t)2 * p.ctas * 8 * NT * kD);
  p.cuts = reinterpret_cast<CutF*>(p.part_ml + (size_t)2 * p.ctas * 8 * NT);
  const LaunchTogether together(s);
  cudaError_t e = launch_pdl(few_rows_kernel<NT>, dim3((unsigned)p.ctas), dim3(kThreadsF), FewSmem<NT>::kBytes, s, p);
  if (e != cudaSuccess) return e;
  // Four warps a column where units may have many parts; one token of 32768 keys (76 parts a unit): 25.5 us with one warp,
  // 22.5 with four; but 16 of 1024 keys: 14.4 and 17.0, for its more blocks.
  const dim3 grid((unsigned)p.ctas, 8 * NT / kMergeCols);
  if (p.ctas > 16 * (int64_t)p.B * p.pg.Hkv) return launch_pdl(few_combine_kernel<NT, 4>, grid, dim3(128 * kMergeCols), 0, s, p);
  return launch_pdl(few_combine_kernel<NT, 1>, grid, dim3(32 * kMergeCols), 0, s, p);
}

}  // namespace

bool few_rows(int n, int B, int Hkv, int G, int T_max) {
  const double units = (double)n + B;
  // Up to 32 columns a sequence: 16 sequences of 4096 keys, 64 query and 8 KV heads, with 1, 2, 3, 4 and 5 rows each take 29.5, 33, 45,
  // 46 and 78 us here, and 58 to 61 in fa3_chunk.cu's kernel.  The lengths are on the device, so the rule goes by the call's average,
  // and was measured on calls of equal sequences.  A chunk beside many single tokens is the wrong way round for one of them: 512
  // rows beside 128 tokens (4 rows on average, all here) take 517 us, the parts by themselves 82 (there) and 181 (here); beside 64
  // (8 rows, all there) 248, by themselves 82 and 96.
  return G <= 16 && columns_of(n, B, G) <= 32 && units * Hkv * (T_max / kStep + kUnitSteps + 1.0) < 2147483648.0;
}
size_t few_rows_workspace(int n, int B, int G, int sms) {
  if (G > 16) return 0;
  const int nt = n_tiles(n, B, G);
  return bytes_of(nt, ctas_of(nt, sms));
}
cudaError_t few_rows_attn(const FewCall& c, const int32_t* table, int num_pages, int page_size, int max_pages, int block,
                          int Hkv, void* workspace, cudaStream_t s) {
  FewParams p;
  if (pages_of(table, c.B, Hkv, num_pages, page_size, max_pages, block, &p.pg) != FA3_OK) return cudaErrorInvalidValue;
  p.q = c.q; p.k = c.k; p.v = c.v; p.ks = c.ks; p.vs = c.vs; p.q_start = c.q_start; p.kv_lens = c.kv_lens;
  p.out = reinterpret_cast<__nv_bfloat16*>(c.out); p.lse = c.lse; p.err = c.err; p.q_stride = c.q_stride;
  p.n = c.n; p.B = c.B; p.Hq = c.Hq; p.G = c.G; p.sm_log2 = c.sm_log2;
  p.div_G = make_divu32((uint32_t)c.G);
  const int nt = n_tiles(c.n, c.B, c.G);
  p.ctas = ctas_of(nt, c.sms);
  return nt == 1 ? launch<1>(p, workspace, s) : nt == 2 ? launch<2>(p, workspace, s) : launch<4>(p, workspace, s);
}

bool few_rows_weights(int n, int B, int Hkv, int G, int T_max) {
  const double chunks = (double)n / (kChunkCols / std::min(G, kChunkCols)) + B;
  // Up to some 96 columns a sequence: 16 sequences of 4096 keys, 64 query and 8 KV heads, with 1, 4, 8 and 16 rows each take
  // 17.6, 24.8, 36.0 and 64.7 us here and 50.7, 51.1, 52.5 and 51.6 in fa3_weights.cu's kernel.  By the call's average, as above:
  // 512 rows beside 64 single tokens (9 rows on average, all here) take 473 us, by themselves 42 (there) and 53 (here).
  return G <= kChunkCols && (int64_t)n * G <= (int64_t)96 * B &&
         Hkv * ((double)B * kWUnit + chunks * (T_max / kStep + 1.0)) < 2147483648.0;
}
cudaError_t few_rows_weights_attn(const FewCall& c, float* weights, const int32_t* table, int num_pages, int page_size,
                                  int max_pages, int block, int Hkv, cudaStream_t s) {
  FewWeightParams p;
  if (pages_of(table, c.B, Hkv, num_pages, page_size, max_pages, block, &p.pg) != FA3_OK) return cudaErrorInvalidValue;
  static std::atomic<bool> set[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return cudaErrorInvalidDevice;
  if (dev >= 64 || !set[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(few_weights_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_FEW_WEIGHTS);
    if (e != cudaSuccess) return e;
    if (dev < 64) set[dev].store(true, std::memory_order_release);
  }
  p.q = c.q; p.k = c.k; p.ks = c.ks; p.lse = c.lse; p.weights = weights; p.q_start = c.q_start; p.kv_lens = c.kv_lens;
  p.err = c.err; p.q_stride = c.q_stride; p.n = c.n; p.B = c.B; p.Hq = c.Hq; p.G = c.G; p.sm_log2 = c.sm_log2;
  p.RC = kChunkCols / c.G;
  p.div_RC = make_divu32((uint32_t)p.RC);
  p.div_G = make_divu32((uint32_t)c.G);
  p.ctas = 4 * c.sms;
  return launch_pdl(few_weights_kernel, dim3((unsigned)p.ctas), dim3(kThreadsF), SMEM_FEW_WEIGHTS, s, p);
}

}  // namespace fa3
