// Attention of packed new rows over an INT8 KV cache (tcgen05, sm_103a): a chunk of new
// tokens over a paged cache, causally, and cross attention to an encoder's states.
//
// The new rows of all sequences are packed: rows q_start[b] .. q_start[b + 1] - 1 of q
// and out belong to sequence b.  With n_b new rows and kv_len_b keys, for row i of
// sequence b, query head h and its KV head g = h / G, G = Hq / Hkv:
//
//   s[t] = (q8[i, h] . k8[t, g]) * q_scale[h] * k_scale[g] * softmax_scale
//   out[i, h] = bf16( v_scale[g] * sum_t softmax(s)_t * v8[t, g] )
//   t <= kv_len_b - n_b + i  (chunk)      t < kv_len_b  (cross)
//
// Work.  A unit is a row block of one sequence and KV head: up to 2 x P positions x the
// group's G heads (P = 128 / G), so that a converted K/V tile of 128 keys feeds up to 256
// rows.  The pipe works in steps, Q.K^T and P.V of 128 rows and 128 keys:
//   * two row tiles: each key tile is two steps, of tile 0 and of tile 1;
//   * one row tile (up to P positions left, a decode token or a short draft): the key tiles
//     alternate between the two score and accumulator buffers, and the two results are
//     merged in the CTA.  Either way step t works on buffer t & 1, and while a buffer's
//     softmax runs the tensor pipe has the other buffer's step.
// All units lie on one line, as long as their measured costs, that is cut into equal
// parts, one per SM: a CTA takes whole units and at most one part of a unit at either
// end.  A cut unit's parts leave unnormalised O, maximum and sum in the workspace, and
// chunk_combine_kernel merges them, so one long sequence and a ragged batch both fill the GPU.
//
// Roles in the CTA (512 threads).  Warp 0 issues the MMAs.  Warp 1 looks pages up in the
// block table and brings int8 K and V tiles to shared memory by TMA.  Warp 2 records the
// cut before the CTA's part for the combine kernel.  Warp 3 finds the CTA's parts of the
// line and hands them to the others through a ring.  Warps 4-7 and 8-11 (a row a lane)
// run the softmax of buffers 0 and 1.  Warps 12, 13 (K) and 14, 15 (V) write the int8
// tiles as fp16 into one of two stages.
//
// Numbers.  int8 codes are exact in fp16 and a 128-term sum of their products stays
// below 2^24, so kind::f16 MMAs with float32 accumulation give the exact integer score
// (the integer tensor rate of sm_103a is far below it).  P is rounded to fp16 relative to
// a reference that the row's maximum lies 2^7 to 2^15 above (it moves lazily): a weight is off by
// 2^-11 of itself, or by 2^-32 of the row's largest where fp16 is subnormal, so T keys are off by
// T 2^-32 of max|v| beside the bf16 rounding of the result, 2^-8 of it.  (With the maximum at 1
// the weights below 2^-25 were lost, but counted in the row sum: 131072 keys off by 2^-8 of max|v|.)
// The row sum is float32 over the unrounded weights, and O, partial results
// and their merging are float32.  P is written over its scores in TMEM and is the A operand
// of P.V.  TMEM: O_0, O_1, S_0, S_1, 128 columns each.
//
// What bounds it (64 query and 8 KV heads, one GB300).  4096 new rows on a context of
// 8192: 682 us, 1209 TFLOP/s.  The tensor pipe works half of the time: the rest is the chain
// scores, softmax, P.V, scores of each of the two buffers with a barrier at every arrow
// (the softmax reads every score from TMEM twice, for the maximum and for the weight), and
// shared memory, which moves 320 KB a key tile (int8 tile in and out, fp16 tile in, Q, K and V
// into the MMAs: 2500 cycles at 128 bytes each).  16 one-token rows of 4096 keys: 50 us,
// 2.7 TB/s.  A key tile takes 2500 cycles of the same chain, for 8 rows of 128; neither a second
// int8 tile on its way nor four warps on a tile's softmax shortened it (53.7 and 55.1 us where
// it took 51.4 and 53.6), and more code costs every case: the roles' loops share the SM's
// instruction cache.  About 8 us of a small call are the launch, the plan (2 us), the first
// tiles' way (3 us) and the combine kernel (3 us).
//
// Every wait is bounded; on time-out the kernel sets FA3_DEVERR_TIMEOUT, waits for its
// copies and MMAs, frees its TMEM and returns.
#include "fa3_common.cuh"
#include "fa3_tc.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include <algorithm>
#include <atomic>
#include <cmath>

namespace fa3 {
namespace {

constexpr int kD = 128;            // head dim
constexpr int kKeys = 128;         // keys per tile
constexpr int kRows = 128;         // rows (TMEM lanes) per row tile
constexpr int kThreadsC = 512;     // warp 0: MMA; 1: TMA; 4-7 / 8-11: softmax of buffer 0 / 1; 12-15: converters
constexpr uint32_t TM_O = 0, TM_S = 256;                   // O_x [128x, +128), S_x [256 + 128x, +128)
constexpr uint32_t KV_TILE = kKeys * kD * 2;               // 32 KB of fp16
constexpr uint32_t KV_HALF = KV_TILE / 2;                  // 64 values of d: 128 keys x 128 B, 128-byte swizzle
constexpr uint32_t Q_TILE = kRows * kD * 2;                // 32 KB of fp16
constexpr uint32_t OFF_Q = 0;                              // 2 x fp16 query rows, K-major
constexpr uint32_t OFF_K = OFF_Q + 2 * Q_TILE;             // 2 stages
constexpr uint32_t OFF_V = OFF_K + 2 * KV_TILE;            // 2 stages
constexpr uint32_t OFF_RAW = OFF_V + 2 * KV_TILE;          // int8 K and V tile on their way: 128 keys x 128 B each
constexpr uint32_t RAW_TILE = kKeys * kD;
constexpr uint32_t OFF_ML = OFF_Q + Q_TILE;                // [2][128] float2: (m, l) of a single row tile's halves,
                                                           // in the second row tile's place
constexpr uint32_t OFF_PARTS = OFF_RAW + 2 * RAW_TILE;     // the ring of parts
constexpr uint32_t kRing = 4, kPartBytes = 48;
constexpr uint32_t OFF_BAR = OFF_PARTS + kRing * kPartBytes;
enum {
  B_K_FULL = 0, B_K_EMPTY = 2, B_V_FULL = 4, B_V_EMPTY = 6,
  B_S_FULL = 8,                    // [2]: buffer x's scores of its next step
  B_P_FULL = 10,                   // [2]: P written over S_x
  B_PV_DONE = 12,                  // [2]: P_x.V done (O_x holds it; S_x free)
  B_ML = 14,                       // [2]: buffer x's (m, l) of a single row tile written
  B_READ = 16,                     // [2]: warps of buffer x have read both O of a single row tile
  B_RAW_FULL = 18,                 // [2]: int8 K, V tile arrived
  B_RAW_EMPTY = 20,                // [2]: int8 K, V tile taken into registers
  B_Q_READY = 22, B_DRAIN = 23,
  B_PART_FULL = 24, B_PART_EMPTY = 28,   // [4]: part of the ring written, read by all
  B_N = 32
};
__constant__ const uint8_t kArrivals[B_N] = {2, 2, 1, 1, 2, 2, 1, 1, 1, 1, 4, 4, 1, 1, 4, 4, 4, 4, 1, 1, 2, 2, 8, 1, 1, 1, 1, 1, 14, 14, 14, 14};
constexpr uint32_t OFF_TSLOT = OFF_BAR + 8 * B_N;
constexpr uint32_t OFF_ABORT = OFF_TSLOT + 4;
constexpr uint32_t SMEM_CHUNK = OFF_ABORT + 4 + 1024;      // + alignment slack
static_assert(SMEM_CHUNK <= 232448, "shared memory");

// The line's unit is an eighth of a step with two row tiles: what a key tile costs with two row tiles and with one, a
// unit's cost beside its steps (its query rows, pipeline fill and epilogue), the least part of the line a CTA takes,
// and the least where short units go one to a CTA (16 one-token units of 128 keys: 17 us in parts of two such units,
// 12 so).  A part of 40 is a short unit of one key tile: one token of 1024 keys takes 18.8 us in parts of 64, 16.7 of
// 40 and 15.8 of 32, which cut short units (one token of 64 keys 10.2 instead of 10.0, of 4096 keys 22.5 instead of
// 21.4).  Fitted over the CTAs of ragged batches: 1950 cycles a step with two row tiles, 2200 with one, 7000 to 8000 a
// unit.  Eight sequences of up to 512 new rows took 113 us with a unit counted as 2 steps, 98.6 as 3 and every step
// alike, 92.3 so (87 now).
constexpr int kTileDual = 16, kTileSingle = 9, kUnitCost = 30, kLeastPart = 40, kLeastInner = 32;
static_assert(kLeastInner >= kTileDual, "a part inside a unit, behind its fixed cost, holds a key tile");

// What the combine kernel has to know of the cut before a CTA's part: nothing (owner < 0) unless it is the
// first cut of its unit.
struct Cut {
  int row0, left, g, dual;      // first packed row of the row block, positions from there on, KV head, two row tiles
  int owner, last, own, end;    // CTAs of the unit's begin and end; whether their parts hold any key tile
};

struct ChunkParams {
  const int8_t* q;              // [n][Hq][128]
  const int8_t* k;              // page pool [pool rows][Hkv][128], or [B][T][Hkv][128]
  const int8_t* v;
  const float* q_scale;         // [Hq]
  const float* k_scale;         // [Hkv]
  const float* v_scale;
  const int32_t* q_start;       // [B + 1]
  const int32_t* kv_lens;       // [B]
  const int32_t* block_table;   // [B][max_pages], or nullptr: sequence b's keys are rows b*T ..
  uint16_t* out;                // bf16 [n][Hq][128]
  float4* part_o;               // [2 * CTAs][32][rows_max]: O of a cut unit's part, column group by row
  float2* part_ml;              // [2 * CTAs][rows_max]
  Cut* cuts;                    // [CTAs]
  int32_t* err;
  int n, B, T, Hq, Hkv, G, P, causal, ctas, rows_max;
  int page_size, max_pages, num_pages;
  DivU32 div_ps, div_2p;        // / page_size, / (2 P)
  int narrow;                   // the line's numbers fit 24 bits
  float sm_log2;                // softmax_scale * log2(e)
  int box;                      // rows of a TMA box; 0: pages too ragged for boxes, loads through registers
  CUtensorMap map_k, map_v;     // [cache rows][Hkv * 128] in boxes of [box][128]
};

// Keys come in boxes of consecutive cache rows, the largest power of two that divides the page size (and the
// tile), from 8 rows on: a tile's 16 boxes are then a half warp's.  Other page sizes go through registers.  The TMA unit
// takes some 31 cycles a box: with a row a box, 16 one-token rows of 4096 keys took 126 us, through registers 67
// and in boxes of 64 rows 63 at that time; 2 x 16 boxes of 8 rows hide behind a tile's 2600 cycles.
constexpr int kLeastBox = 8;

// ------------------------------------------------------------------ the line of steps
struct Seq {
  int q0, nq, nkv;
};
// The new rows and keys of sequence b; nq = 0 for an empty or invalid sequence, -1 for one that ends before it begins.
__device__ __forceinline__ Seq sequence_of(const ChunkParams& p, int b, bool report) {
  Seq s;
  s.q0 = p.q_start[b];
  const int q1 = p.q_start[b + 1];
  s.nkv = p.kv_lens[b];
  s.nq = q1 - s.q0;
  if (s.q0 < 0 || q1 < s.q0 || q1 > p.n || (s.nq > 0 && (s.nkv < (p.causal ? s.nq : 0) || s.nkv > p.T))) {
    if (report) set_dev_err(p.err, FA3_DEVERR_LENS);
    s.nq = q1 < s.q0 ? -1 : 0;
  }
  return s;
}
__device__ __forceinline__ int blocks_of(const ChunkParams& p, const Seq& s) {
  return (int)divu32((uint32_t)(s.nq + 2 * p.P - 1), p.div_2p);
}
// Key tiles of row block rb, and its cost.
__device__ __forceinline__ int tiles_of(const ChunkParams& p, const Seq& s, int rb) {
  const int keys = p.causal ? s.nkv - s.nq + min(s.nq, (rb + 1) * 2 * p.P) : s.nkv;
  return (int)(((uint32_t)keys + kKeys - 1) / kKeys);
}
__device__ __forceinline__ bool is_dual(const ChunkParams& p, const Seq& s, int rb) { return s.nq - rb * 2 * p.P > p.P; }
__device__ __forceinline__ int cost_of(const ChunkParams& p, const Seq& s, int rb) {
  return kUnitCost + tiles_of(p, s, rb) * (is_dual(p, s, rb) ? kTileDual : kTileSingle);
}

// The line's numbers are I: uint32_t where they fit 24 bits (the host's bound), int64_t otherwise.  The plan is on
// every call's way, and 64-bit divisions and scans take several times as long (16 sequences: 6600 cycles with int64_t,
// 3200 with uint32_t).

// Sum over r < n of floor((at + r step) / mod): whole multiples come out, then the roles of step and mod change
// (the lattice points under a line, counted along the other axis: Graham, Knuth and Patashnik, "Concrete Mathematics",
// section 3.5, with Euclid's steps).
template <class I>
__device__ __forceinline__ I floor_sum(I n, I mod, I step, I at) {
  I total = 0;
#pragma unroll 1
  for (;;) {
    total += n * (n - 1) / 2 * (step / mod) + n * (at / mod);
    step %= mod;
    at %= mod;
    const I top = step * n + at;
    if (top < mod) return total;
    n = top / mod;
    at = top % mod;
    const I t = mod;
    mod = step;
    step = t;
  }
}
// Cost of all row blocks of one KV head of the sequence.
template <class I>
__device__ __forceinline__ I sequence_cost(const ChunkParams& p, const Seq& s) {
  const int nb = blocks_of(p, s);
  if (nb == 0) return 0;
  I c = (I)cost_of(p, s, nb - 1) + (I)(nb - 1) * kUnitCost;
  if (nb > 1)
    c += kTileDual * (p.causal ? floor_sum<I>((I)(nb - 1), kKeys, (I)(2 * p.P), (I)(s.nkv - s.nq) + 2 * p.P + kKeys - 1)
                       : (I)(nb - 1) * (I)tiles_of(p, s, 0));
  return c;
}

template <class I>
__device__ __forceinline__ I warp_scan(I v, int lane) {     // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const I y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// The line and its parts: CTA c takes [begin(c), begin(c + 1)).
template <class I>
struct Line {
  I total, each;
  int parts, rest;
  __device__ __forceinline__ I begin(int c) const {
    return c >= parts ? total : each * (I)c + (I)((uint32_t)rest * (uint32_t)c / (uint32_t)parts);
  }
  // The part that position x lies in.
  __device__ __forceinline__ int owner(I x) const {
    int c = (int)(((x + 1) * (I)parts - 1) / total);
    while (c > 0 && begin(c) > x) --c;
    while (c + 1 < parts && begin(c + 1) <= x) ++c;
    return c;
  }
};
// The first 32 sequences, a lane each: cost of a KV head and, summed over all heads, up to and with this one.
template <class I>
struct Ahead {
  Seq s;
  I per_head, upto;
};
// The warp together; s0: sequence `lane`.
template <class I>
__device__ __forceinline__ Line<I> make_line(const ChunkParams& p, int lane, bool report, const Seq& s0, Ahead<I>& a) {
  a.s = s0;
  a.per_head = sequence_cost<I>(p, s0);
  a.upto = warp_scan<I>(a.per_head * (I)p.Hkv, lane);
  int blocks = blocks_of(p, s0);
  bool falls = s0.nq < 0;
  Line<I> l;
  l.total = __shfl_sync(0xffffffffu, a.upto, 31);
  if (p.B > 32) {
    I sum = 0;
#pragma unroll 1
    for (int b = 32 + lane; b < p.B; b += 32) {
      const Seq s = sequence_of(p, b, report);
      sum += sequence_cost<I>(p, s);
      blocks += blocks_of(p, s);
      falls |= s.nq < 0;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l.total += sum * (I)p.Hkv;
  }
  blocks = __reduce_add_sync(0xffffffffu, blocks);
  // A q_start that falls: where it rises again sequences may share rows, which two units would write, and the rows may be more
  // than n, which the bounds of I rest on.  There is no plan, then.
  if (__any_sync(0xffffffffu, falls)) {
    l.total = 0;
    blocks = 0;
  }
  // Parts of kLeastPart or more; short units go one to a CTA, though (parts of kLeastInner or more, so that a part
  // inside a unit still holds a key tile).
  const I units = min((I)blocks * (I)p.Hkv, l.total / kLeastInner), most = max(l.total / kLeastPart, units);
  l.parts = most < 1 ? 1 : most < (I)p.ctas ? (int)most : p.ctas;
  l.each = l.total / (I)l.parts;
  l.rest = (int)(l.total - l.each * (I)l.parts);
  return l;
}

// A position on the line: unit (b, g, rb) and the offset into it.
template <class I>
struct Cursor {
  int b, g, rb;
  Seq s;
  I off;
};
__device__ __forceinline__ Seq lane_of(const Seq& s, int l) {
  return Seq{__shfl_sync(0xffffffffu, s.q0, l), __shfl_sync(0xffffffffu, s.nq, l), __shfl_sync(0xffffffffu, s.nkv, l)};
}
// First sequence from b on with new rows (the warp together); b = B when there is none.
template <class I>
__device__ __forceinline__ void to_sequence(const ChunkParams& p, Cursor<I>& c, int b, const Seq& s0, int lane) {
#pragma unroll 1
  for (int base = b & ~31; base < p.B; base += 32) {
    Seq s = s0;
    if (base > 0) {
      s = Seq{0, 0, 0};
      if (base + lane < p.B) s = sequence_of(p, base + lane, false);
    }
    const unsigned have = __ballot_sync(0xffffffffu, s.nq > 0 && base + lane >= b);
    if (have) {
      const int l = __ffs(have) - 1;
      c.b = base + l;
      c.s = lane_of(s, l);
      return;
    }
  }
  c.b = p.B;
  c.s = Seq{0, 0, 0};
}
// The unit that holds position x of the line (x < total).
template <class I>
__device__ __forceinline__ Cursor<I> seek(const ChunkParams& p, I x, const Ahead<I>& first, int lane) {
  Cursor<I> c = {p.B, 0, 0, {0, 0, 0}, 0};
#pragma unroll 1
  for (int base = 0; base < p.B; base += 32) {
    Seq s = first.s;
    I mine = first.per_head, upto = first.upto;
    if (base > 0) {
      s = Seq{0, 0, 0};
      if (base + lane < p.B) s = sequence_of(p, base + lane, false);
      mine = sequence_cost<I>(p, s);
      upto = warp_scan<I>(mine * (I)p.Hkv, lane);
    }
    const unsigned beyond = __ballot_sync(0xffffffffu, upto > x);
    if (beyond) {
      const int l = __ffs(beyond) - 1;
      const I per_head = __shfl_sync(0xffffffffu, mine, l);
      x -= __shfl_sync(0xffffffffu, upto, l) - per_head * (I)p.Hkv;
      c.b = base + l;
      c.s = lane_of(s, l);
      c.g = (int)(x / per_head);
      x -= (I)c.g * per_head;
      break;
    }
    x -= __shfl_sync(0xffffffffu, upto, 31);
  }
  const int nb = blocks_of(p, c.s);
  c.off = x;
#pragma unroll 1
  for (int base = 0; base < nb && nb > 1; base += 32) {
    const I mine = base + lane < nb ? (I)cost_of(p, c.s, base + lane) : 0, upto = warp_scan<I>(mine, lane);
    const unsigned beyond = __ballot_sync(0xffffffffu, upto > x);
    if (beyond) {
      const int l = __ffs(beyond) - 1;
      c.rb = base + l;
      c.off = x - __shfl_sync(0xffffffffu, upto - mine, l);
      break;
    }
    x -= __shfl_sync(0xffffffffu, upto, 31);
  }
  return c;
}

// Key tile at which a part that begins `off` into a unit begins.
template <class I>
__device__ __forceinline__ int tile_at(I off, bool dual, int nt) {
  const I at = off <= kUnitCost ? 0 : off - kUnitCost, t = dual ? at / kTileDual : at / kTileSingle;
  return t < (I)nt ? (int)t : nt;
}

// The record of the cut before CTA cta's part (the warp together).
template <class I>
__device__ __forceinline__ void record_cut(const ChunkParams& p, const Seq& s0, int cta, int lane) {
  Ahead<I> first;
  const Line<I> line = make_line<I>(p, lane, false, s0, first);
  Cut cut = {0, 0, 0, 0, -1, 0, 0, 0};
  const I x = line.begin(cta);
  if (cta > 0 && cta < line.parts && x < line.total) {
    const Cursor<I> c = seek<I>(p, x, first, lane);
    const I begin = x - c.off;                               // of the unit
    if (c.off > 0 && line.begin(cta - 1) <= begin) {         // its first cut
      const int nt = tiles_of(p, c.s, c.rb);
      const bool dual = is_dual(p, c.s, c.rb);
      const I end = begin + (I)cost_of(p, c.s, c.rb);
      cut.row0 = c.s.q0 + c.rb * 2 * p.P;
      cut.left = c.s.nq - c.rb * 2 * p.P;
      cut.g = c.g;
      cut.dual = dual;
      cut.owner = cta - 1;
      cut.last = line.owner(end - 1);
      // a CTA between the two has kLeastInner or more of the line, which is a key tile at least; only this one,
      // right behind the unit's begin, may have none
      cut.own = tile_at<I>(c.off, dual, nt) > 0;
      if (cta < cut.last && tile_at<I>(line.begin(cta + 1) - begin, dual, nt) == 0) cut.owner = cta;
      cut.end = tile_at<I>(line.begin(cut.last) - begin, dual, nt) < nt;
    }
  }
  if (lane == 0) p.cuts[cta] = cut;
}

// What a CTA does of a unit: key tiles [t0, t1) of nt, for row block rb.
struct Part {
  int b, g, rb, q0, nq, nkv, t0, t1, nt;
  bool dual, first;                 // first: the part holds the unit's begin
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == nt; }
};

static_assert(sizeof(Part) <= kPartBytes, "ring of parts");

// Rows of queries without a key (the warp together).
__device__ __forceinline__ void zero_rows(const ChunkParams& p, int row0, int count, int g, int lane) {
#pragma unroll 1
  for (int i = lane >> 4; i < count * p.G; i += 2) {
    const int at = i / p.G;
    reinterpret_cast<uint4*>(p.out + ((int64_t)(row0 + at) * p.Hq + g * p.G + i - at * p.G) * kD)[lane & 15] = make_uint4(0u, 0u, 0u, 0u);
  }
}
// A CTA's parts in order (the warp together), each given to `put`.  The roles look a key tile ahead, so a part
// in the ring has one at least: rows without a key are written here.
template <class I, class Put>
__device__ __forceinline__ void walk_parts(const ChunkParams& p, const Seq& s0, int cta, int lane, Put put) {
  Ahead<I> first;
  const Line<I> line = make_line<I>(p, lane, cta == 0, s0, first);
  const I x = line.begin(cta);
  I left = line.begin(cta + 1) - x;
  if (left == 0) return;
  Cursor<I> c = seek<I>(p, x, first, lane);
#pragma unroll 1
  while (left > 0) {
    const int nt = tiles_of(p, c.s, c.rb);
    const bool dual = is_dual(p, c.s, c.rb);
    const I cost = (I)cost_of(p, c.s, c.rb), take = min(cost - c.off, left);
    const bool first_part = c.off == 0;
    const Part u = {c.b, c.g, c.rb, c.s.q0, c.s.nq, c.s.nkv, tile_at<I>(c.off, dual, nt),
                    c.off + take == cost ? nt : tile_at<I>(c.off + take, dual, nt), nt, dual, first_part};
    if (nt == 0) {
      if (first_part) zero_rows(p, c.s.q0 + c.rb * 2 * p.P, min(c.s.nq - c.rb * 2 * p.P, 2 * p.P), c.g, lane);
    } else if (u.t0 < u.t1 && !put(u)) {
      return;
    }
    left -= take;
    c.off = 0;
    if (++c.rb == blocks_of(p, c.s)) {
      c.rb = 0;
      if (++c.g == p.Hkv) {
        c.g = 0;
        if (left > 0) to_sequence<I>(p, c, c.b + 1, s0, lane);
      }
    }
  }
}

// wait_bar for short waits, with bounded_wait's rare look at the clock, in ticks of 2^20 ns (1.05 ms).  A second for a wait
// within a unit; a wait for a part of the ring may last as long as a unit of the longest context takes (2.3 us a key
// tile), and has four seconds and 8 us a key tile.
constexpr uint32_t kWaitTicks = 954;
__device__ __forceinline__ uint32_t part_ticks(const ChunkParams& p) { return 4 * kWaitTicks + ((uint32_t)p.T >> 14); }
__device__ __forceinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, int32_t* err,
                                          uint32_t limit = kWaitTicks) {
  const Waited w = bounded_wait([&] { return mbar_try(bar, parity); }, [&] { return *abort_flag != 0u; },
                                [] { return (uint32_t)(global_ns() >> 20); }, limit);
  if (w == Waited::kLate) {
    *abort_flag = 1u;
    set_dev_err(err, FA3_DEVERR_TIMEOUT);
  }
  return w == Waited::kDone;
}
// The same for a warp, whose lanes have to agree.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int lane, volatile uint32_t* abort_flag,
                                          int32_t* err, uint32_t limit = kWaitTicks) {
  return warp_all(wait_long(bar, parity, abort_flag, err, limit));
}

// The wait for this thread's TMEM loads, which also orders the uses of v behind it.
__device__ __forceinline__ void wait_ld16(uint32_t* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
               :: "memory");
}

// 32 columns' maximum, by the load itself; the columns go to v all the same.
__device__ __forceinline__ void tmem_ld_max32(uint32_t taddr, uint32_t (&v)[32], float& m) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
        "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
        "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31]),
        "=f"(m)
      : "r"(taddr));
}
__device__ __forceinline__ void wait_max(float& a) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+f"(a) :: "memory");
}

// 16 bytes that this SM reads once: the L1 (what shared memory leaves of it) is passed by.
__device__ __forceinline__ uint4 load_once(const int8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* tm, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]) : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* tm) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tm)) : "memory");
}
__device__ __forceinline__ void prefetch_line(const int8_t* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// MMAs on descriptors given by their low words (address and leading stride; the step along the contraction
// is one 32-bit addition).  The whole warp runs the issuing code, converged, so that its addresses stay in
// uniform registers, and the elected lane's predicate guards the instruction itself.
__host__ __device__ constexpr uint32_t desc_hi(uint32_t sbo, bool swizzle) { return (sbo >> 4) | (1u << 14) | (swizzle ? 2u << 29 : 0u); }
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return (addr >> 4) | ((lbo >> 4) << 16); }
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e;
}
template <uint32_t HI_A, uint32_t HI_B>
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p, e;\n.reg .b64 a, b;\nsetp.ne.b32 e, %0, 0;\nsetp.ne.b32 p, %5, 0;\n"
      "mov.b64 a, {%2, %6};\nmov.b64 b, {%3, %7};\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%1], a, b, %4, p;\n}\n"
      ::"r"(lead), "r"(d), "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "n"(HI_A), "n"(HI_B) : "memory");
}
template <uint32_t HI>
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p, e;\n.reg .b64 b;\nsetp.ne.b32 e, %0, 0;\nsetp.ne.b32 p, %5, 0;\nmov.b64 b, {%3, %6};\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], b, %4, p;\n}\n"
      ::"r"(lead), "r"(d), "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(acc), "n"(HI) : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n.reg .pred e;\nsetp.ne.b32 e, %1, 0;\n"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar), "r"(lead)
      : "memory");
}

__global__ void __launch_bounds__(kThreadsC, 1) gqa_chunk_kernel(const __grid_constant__ ChunkParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + OFF_ABORT);
  auto bar = [&](int i) { return sbase + OFF_BAR + 8u * (uint32_t)i; };
  // Set-up that reads nothing another kernel writes goes before the wait for it.
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(sbase + OFF_TSLOT), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (warp == 1) {
    static_assert(B_N == 32, "a lane a barrier");
    mbar_init(bar(lane), lane >= B_PART_EMPTY && !p.box ? 13 : kArrivals[lane]);   // without boxes warp 1 has nothing to do
    if (lane == 0) *abort_flag = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (lane == 0 && p.box) {
      prefetch_map(&p.map_k);
      prefetch_map(&p.map_v);
    }
  }
  pdl_wait();
  Seq s0 = {0, 0, 0};                                         // of warps 2 and 3: on its way while the others set up
  if ((warp & ~1) == 2 && lane < p.B) s0 = sequence_of(p, lane, blockIdx.x == 0 && warp == 3);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + OFF_TSLOT);
  pdl_launch_dependents();

  // The CTA's parts come from warp 3 through a ring; a part with nt < 0 is the end.
  Part* const ring = reinterpret_cast<Part*>(smem + OFF_PARTS);
  uint32_t parts = 0;                                         // taken (by warp 3: written)
  auto next_part = [&]() {                                    // false: none left; otherwise the part is ring[parts % kRing]
    return warp_wait(bar(B_PART_FULL) + 8u * (parts % kRing), (parts / kRing) & 1u, lane, abort_flag, p.err, part_ticks(p)) &&
           ring[parts % kRing].nt >= 0;
  };
  auto part_read = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(B_PART_EMPTY) + 8u * (parts % kRing));
    ++parts;
  };

  if (warp == 3) {
    auto put = [&](const Part& u) {
      if (!warp_wait(bar(B_PART_EMPTY) + 8u * (parts % kRing), ((parts / kRing) & 1u) ^ 1u, lane, abort_flag, p.err,
                     part_ticks(p)))
        return false;
      if (lane == 0) {
        ring[parts % kRing] = u;
        mbar_arrive(bar(B_PART_FULL) + 8u * (parts % kRing));
      }
      ++parts;
      return true;
    };
    if (p.narrow)
      walk_parts<uint32_t>(p, s0, blockIdx.x, lane, put);
    else
      walk_parts<int64_t>(p, s0, blockIdx.x, lane, put);
    Part end = {};
    end.nt = -1;
    put(end);
  } else if (warp == 2) {
    if (p.narrow)
      record_cut<uint32_t>(p, s0, blockIdx.x, lane);
    else
      record_cut<int64_t>(p, s0, blockIdx.x, lane);
  } else if (warp == 0) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t id_qk = idesc_f16(kRows, kKeys, false, false);
    const uint32_t id_pv = idesc_f16(kRows, kD, false, true);
    uint32_t kc = 0, done0 = 0, done1 = 0, units = 0;         // key tiles, steps of each buffer, units so far
    bool ok = true;
    const uint32_t lead = elect_one();
    while (ok && next_part()) {
      const Part& now = ring[parts % kRing];
      const struct { int t0, t1; bool dual; } u = {now.t0, now.t1, now.dual};
      part_read();
      const int nk = u.t1 - u.t0, steps = u.dual ? 2 * nk : nk;
      ok = warp_all(wait_long(bar(B_Q_READY), units & 1u, abort_flag, p.err));
      // Step t: buffer t & 1, key tile t (or t / 2 with two row tiles).  P.V of step t, then Q.K^T of step t + 2.
      // All roles' loops are kept rolled: together they have to stay in the SM's instruction cache, and an MMA lasts
      // longer than an iteration (4096 rows on 8192 keys, the MMA loops unrolled by 1, 2, 4, 8: 691, 682, 700, 702 us).
      const uint32_t per = u.dual ? 1u : 0u;
#pragma unroll 1
      for (int t = -2; t < steps && ok; ++t) {
        const uint32_t x = (uint32_t)t & 1u;
        if (t >= 0) {
          // O_x += P_x.V: P_x (fp16, over S_x: column k holds keys 2k, 2k + 1) is the A operand in
          // TMEM, V the MN-major B operand (128-byte swizzle: 8-key groups 1024 B apart, halves of d 16 KB).
          const uint32_t kt = kc + ((uint32_t)t >> per), s = kt & 1u, d = (x ? done1 : done0) + ((uint32_t)t >> 1);
          ok = ((u.dual && x) || warp_all(wait_long(bar(B_V_FULL) + 8u * s, (kt >> 1) & 1u, abort_flag, p.err))) &&
               warp_all(wait_long(bar(B_P_FULL) + 8u * x, d & 1u, abort_flag, p.err));
          if (!ok) break;
          tc_fence_after();
          uint32_t bd = desc_lo(sbase + OFF_V + s * KV_TILE, KV_HALF), ap = tmem + TM_S + x * 128;
          uint32_t acc = t >= 2 ? 1u : 0u;
#pragma unroll 2
          for (int kk = 0; kk < kKeys / 16; ++kk) {
            mma_ts<desc_hi(1024, true)>(lead, tmem + TM_O + x * 128, ap, bd, id_pv, acc);
            bd += 2048 >> 4;
            ap += 8;
            acc = 1u;
          }
          commit_if(lead, bar(B_PV_DONE) + 8u * x);
          if (!u.dual || x) commit_if(lead, bar(B_V_EMPTY) + 8u * s);
        }
        if (t + 2 < steps) {
          // S_x = Q.K^T: the row tile's K-major A operand in shared memory (8-row core groups 128 B
          // apart, 8-wide d groups 2048 B apart), K the K-major B operand (128-byte swizzle: 8-key groups
          // 1024 B apart, 16 values of d 32 B apart within a half).  S_x holds the P of step t until its P.V is done.
          const uint32_t t2 = (uint32_t)(t + 2), kt = kc + (t2 >> per), s = kt & 1u;
          ok = (u.dual && x) || warp_all(wait_long(bar(B_K_FULL) + 8u * s, (kt >> 1) & 1u, abort_flag, p.err));
          if (ok && t >= 0)
            ok = warp_all(wait_long(bar(B_PV_DONE) + 8u * x, ((x ? done1 : done0) + ((uint32_t)t >> 1)) & 1u, abort_flag, p.err));
          if (!ok) break;
          tc_fence_after();
          uint32_t a = desc_lo(sbase + OFF_Q + (u.dual ? x : 0u) * Q_TILE, 2048), bd = desc_lo(sbase + OFF_K + s * KV_TILE, 16);
          uint32_t acc = 0u;
#pragma unroll 2
          for (int kk = 0; kk < kD / 16; ++kk) {
            mma_ss<desc_hi(128, false), desc_hi(1024, true)>(lead, tmem + TM_S + x * 128, a, bd, id_qk, acc);
            a += 4096 >> 4;
            bd += kk == 3 ? (KV_HALF >> 4) - 3 * (32 >> 4) : 32 >> 4;
            acc = 1u;
          }
          commit_if(lead, bar(B_S_FULL) + 8u * x);
          if (!u.dual || x) commit_if(lead, bar(B_K_EMPTY) + 8u * s);    // all steps of this key tile have it
        }
      }
      kc += (uint32_t)nk;
      done0 += (uint32_t)(steps + 1) / 2;
      done1 += (uint32_t)steps / 2;
      ++units;
    }
    // Drain: every MMA issued has completed before TMEM is freed.
    commit_if(lead, bar(B_DRAIN));
    wait_long(bar(B_DRAIN), 0, abort_flag, p.err);
  } else if (warp == 1) {
    // ------------------------------------------------------ TMA: int8 tiles of K and V
    // Lanes 0 .. 15 have a box of K each, lanes 16 .. 31 of V (fewer boxes: fewer lanes).  A lane looks up the
    // page of its box's first key one tile ahead.  Boxes past the end are the last box again.
    if (p.box) {
      const int kv = lane >> 4, boxes = kKeys / p.box, i = lane & 15;
      const bool mine = i < boxes;
      int j = 0, t_end = 0, n_keys = 0, b = 0, g = 0;        // the tile to look up next
      int pg = 0, at = 0, g_at = 0;                          // the tile looked up
      auto look_up = [&]() {                                 // false: nothing left
        while (j >= t_end) {
          if (!next_part()) return false;
          const Part& u = ring[parts % kRing];
          j = u.t0;
          t_end = u.t1;
          b = u.b;
          g = u.g;
          n_keys = p.causal ? u.nkv - u.nq + min(u.nq, (u.rb + 1) * 2 * p.P) : u.nkv;
          part_read();
        }
        const uint32_t t = (uint32_t)min(j * kKeys + i * p.box, (n_keys - 1) & ~(p.box - 1));
        if (p.block_table) {
          const uint32_t pi = divu32(t, p.div_ps);
          pg = mine ? __ldg(p.block_table + (int64_t)b * p.max_pages + pi) : 0;
          at = (int)(t - pi * (uint32_t)p.page_size);
        } else {
          at = b * p.T + (int)t;
        }
        g_at = g;
        ++j;
        return true;
      };
      const CUtensorMap* map = kv ? &p.map_v : &p.map_k;
      const uint32_t dst = sbase + OFF_RAW + kv * RAW_TILE + (uint32_t)(i * p.box) * kD;
      bool more = look_up(), ok = true;
      uint32_t kc = 0;
      for (; more && ok; ++kc) {
        if ((uint32_t)pg >= (uint32_t)p.num_pages && p.block_table) {   // outside the pool: any page of it
          set_dev_err(p.err, FA3_DEVERR_PAGE);
          pg = 0;
        }
        const int row = at + (p.block_table ? pg * p.page_size : 0), col = g_at * kD;
        more = look_up();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ok = ok && warp_wait(bar(B_RAW_EMPTY + h), (kc & 1u) ^ 1u, lane, abort_flag, p.err);
          if (!ok) break;
          if (lane == 0) mbar_expect_tx(bar(B_RAW_FULL + h), RAW_TILE);
          __syncwarp();
          if (kv == h && mine) tma_2d(dst, map, col, row, bar(B_RAW_FULL + h));
        }
      }
      // What was sent off lands before the block ends, also after a time-out elsewhere (a bounded wait; of the
      // last tile K alone may be on its way, then V's last is the one before).
      if (lane < 2 && kc > 0) {
        const uint64_t t0 = global_ns();
        for (uint32_t back = 1; back <= (ok ? 1u : 2u) && back <= kc; ++back)
          while (!mbar_try(bar(B_RAW_FULL + lane), (kc - back) & 1u) && global_ns() - t0 < kWaitNs / 50) {}
      }
    }
  } else if (warp >= 12) {
    // ------------------------------------------------------ int8 -> fp16 converters
    // Warps 12 and 13 have K, 14 and 15 V (each in a chain of its own: 16 x 4096 keys, one token each, 57.5 -> 53.6 us
    // against all four on K and then V).  A warp has 64 keys of a tile, a lane 16 bytes of sixteen of them: bytes
    // 16 (l % 8) .. of row l / 8, lanes l % 8 >= 4 of the row's neighbour (l / 8) ^ 1.  The two 16-byte fp16 chunks they
    // become go to chunks 2c and 2c + 1 of the key's swizzled row; the neighbour's row has the other parity, so
    // the eight lanes of a store hit different banks.  Without boxes the bytes come from the cache itself: a lane
    // looks two keys up, the others get their rows by shuffles, and the rows of the next tile are asked of HBM into
    // L2 a tile ahead.
    const int cw = warp & 1, kv = (warp - 12) >> 1, cl = lane & 7, rl = (lane >> 3) ^ (cl >> 2);
    const uint32_t src = sbase + OFF_RAW + kv * RAW_TILE + (uint32_t)(64 * cw + rl) * kD + cl * 16;
    // chunk 2 cl (and 2 cl + 1) of key n: half cl / 4, row n, chunk ((2 cl) % 8) ^ (n % 8)
    const uint32_t dst0 = sbase + (uint32_t)(cl >> 2) * KV_HALF + (uint32_t)(64 * cw + rl) * 128;
    const uint32_t at0 = ((uint32_t)(2 * cl & 7) ^ (uint32_t)rl) * 16;   // n % 8 = rl, or rl + 4 for odd i
    const int row_stride = p.Hkv * kD;
    int j = 0, t_end = 0, n_keys = 0, b = 0, g = 0;          // the tile to look up next
    int mine[2] = {0, 0}, head = 0, head_next = 0;                   // the tile looked up: this lane's row, offset of the KV head
    auto look_up = [&]() {                                   // false: nothing left
      while (j >= t_end) {
        if (!next_part()) return false;
        const Part& u = ring[parts % kRing];
        j = u.t0;
        t_end = u.t1;
        b = u.b;
        g = u.g;
        n_keys = p.causal ? u.nkv - u.nq + min(u.nq, (u.rb + 1) * 2 * p.P) : u.nkv;
        part_read();
      }
      if (!p.box) {
        head_next = g * kD;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t t = (uint32_t)min(j * kKeys + 64 * cw + 32 * h + lane, n_keys - 1), pi = divu32(t, p.div_ps);
          int pg = __ldg(p.block_table + (int64_t)b * p.max_pages + pi);
          if ((uint32_t)pg >= (uint32_t)p.num_pages) {         // outside the pool: any page of it
            set_dev_err(p.err, FA3_DEVERR_PAGE);
            pg = 0;
          }
          mine[h] = pg * p.page_size + (int)(t - pi * (uint32_t)p.page_size);
          prefetch_line((kv ? p.v : p.k) + (int64_t)mine[h] * row_stride + head_next);
        }
      }
      ++j;
      return true;
    };
    bool more = look_up(), ok = true;
    for (uint32_t kc = 0; more && ok; ++kc) {
      const uint32_t s = kc & 1u, par = ((kc >> 1) & 1u) ^ 1u;
      const int rows[2] = {mine[0], mine[1]};                // of this tile
      head = head_next;
      more = look_up();
      const uint32_t dst = dst0 + OFF_K + (OFF_V - OFF_K) * kv + s * KV_TILE;
      uint4 r[16];
      if (p.box) {
        // The int8 tile is given back as soon as it is in registers, before the wait for the fp16 tile's place (the same
        // workload: 63 -> 57.5 us).  The fence holds the TMA's next writes behind these reads: without it
        // one warp in some thousands read its part of the next tile.
        ok = warp_wait(bar(B_RAW_FULL) + 8u * kv, kc & 1u, lane, abort_flag, p.err);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 16; ++i) r[i] = lds128(src + 4 * i * kD);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_RAW_EMPTY) + 8u * kv);
      } else {
        const int8_t* base = (kv ? p.v : p.k) + head + cl * 16;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          r[i] = load_once(base + (int64_t)__shfl_sync(0xffffffffu, rows[i >> 3], (4 * i & 31) + rl) * row_stride);
      }
      ok = warp_wait(bar(B_K_EMPTY) + 8u * (s + (B_V_EMPTY - B_K_EMPTY) * kv), par, lane, abort_flag, p.err);
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        uint4 o0, o1;
        i8x4_to_f16x4(r[i].x, o0.x, o0.y);
        i8x4_to_f16x4(r[i].y, o0.z, o0.w);
        i8x4_to_f16x4(r[i].z, o1.x, o1.y);
        i8x4_to_f16x4(r[i].w, o1.z, o1.w);
        const uint32_t at = at0 ^ ((uint32_t)(i & 1) << 6);
        sts128(dst + 4 * i * 128 + at, o0);
        sts128(dst + 4 * i * 128 + (at ^ 16u), o1);
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_K_FULL) + 8u * (s + (B_V_FULL - B_K_FULL) * kv));
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax warps
    const int x = (warp - 4) >> 2;                          // buffer
    const int r = ((warp - 4) & 3) * 32 + lane;             // row == TMEM lane
    const uint32_t lane_base = (uint32_t)(((warp - 4) & 3) * 32) << 16;
    const uint32_t o_col = tmem + lane_base + TM_O + x * 128;
    const uint32_t scol = tmem + lane_base + TM_S + x * 128;
    float2* ml = reinterpret_cast<float2*>(smem + OFF_ML);
    auto warp_arrive = [&](int which) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(which));
    };
    uint32_t done = 0, done_other = 0, merges = 0;          // steps of this buffer and the other, merged units
    bool ok = true;
    while (ok && next_part()) {
      const Part u = ring[parts % kRing];
      part_read();
      const int nk = u.t1 - u.t0, steps = u.dual ? 2 * nk : nk, mine = (steps + 1 - x) / 2;
      const int pl = r / p.G, hh = u.g * p.G + r - pl * p.G;  // position in the row tile, query head
      const int i = u.rb * 2 * p.P + (u.dual ? x * p.P : 0) + pl;
      const bool active = pl < p.P && i < u.nq;
      const bool warp_active = __any_sync(0xffffffffu, active);
      const int64_t orow = (int64_t)(u.q0 + (active ? i : 0)) * p.Hq + hh;   // row of q and out
      // The row's query codes as fp16 into the row tile's K-major A operand (chunk of 8 d at
      // (d / 8) * 2048 + row * 16).
      if (u.dual || x == 0) {
        const int8_t* qrow = p.q + orow * kD;
        uint8_t* qdst = smem + OFF_Q + (u.dual ? x : 0) * Q_TILE + r * 16;
#pragma unroll
        for (int c16 = 0; c16 < 8; ++c16) {
          uint4 xq = make_uint4(0u, 0u, 0u, 0u);
          if (active) xq = __ldg(reinterpret_cast<const uint4*>(qrow + 16 * c16));
          uint4 o0, o1;
          i8x4_to_f16x4(xq.x, o0.x, o0.y);
          i8x4_to_f16x4(xq.y, o0.z, o0.w);
          i8x4_to_f16x4(xq.z, o1.x, o1.y);
          i8x4_to_f16x4(xq.w, o1.z, o1.w);
          *reinterpret_cast<uint4*>(qdst + (2 * c16) * 2048) = o0;
          *reinterpret_cast<uint4*>(qdst + (2 * c16 + 1) * 2048) = o1;
        }
        fence_proxy_async();
      }
      warp_arrive(B_Q_READY);
      const int pos = !active ? -1 : p.causal ? u.nkv - u.nq + i : u.nkv - 1;   // last key this row sees
      const int pos_min = __reduce_min_sync(0xffffffffu, active ? pos : 0x7fffffff);
      // positive, so that -inf * c stays -inf; with a scale of zero every score still rounds to weight 1
      const float c = active ? fmaxf(p.q_scale[hh] * p.k_scale[u.g] * p.sm_log2, 1e-37f) : 1.f;
      float m_run = -CUDART_INF_F, l_run = 0.f;
      for (int st = 0; st < mine && ok; ++st) {
        const uint32_t ph = done + (uint32_t)st;
        if (!warp_wait(bar(B_S_FULL + x), ph & 1u, lane, abort_flag, p.err)) {
          ok = false;
          break;
        }
        if (warp_active) {
          tc_fence_after();
          const int t0 = (u.t0 + (u.dual ? st : 2 * st + x)) * kKeys;   // the tile's first key
          if (t0 + kKeys - 1 > pos_min) {
            // some active row of the warp does not see all keys: their scores become -inf
            const int last = pos - t0;
#pragma unroll 1
            for (int c16 = 0; c16 < 8; ++c16) {
              uint32_t w[16];
              FA3_TMEM_LD16(scol + c16 * 16, w);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = 16 * c16 + e <= last ? w[e] : 0xff800000u;
              FA3_TMEM_ST16(scol + c16 * 16, w);
            }
            tmem_wait_st();
          }
          // the row's maximum of the integer scores
          uint32_t v0[16], v1[16];
          float mx = -CUDART_INF_F;
#pragma unroll 1
          for (uint32_t k = 0; k < 128; k += 32) {
            uint32_t w[32];
            float m;
            tmem_ld_max32(scol + k, w, m);
            wait_max(m);
            mx = fmaxf(mx, m);
          }
          FA3_TMEM_LD16(scol, v0);
          // The reference, 7 (log2 units) below the row's maximum.  Rounded up, and the difference below is exact where
          // it matters: P stays below 2^15 whatever the size of the scores.
          mx = __fadd_ru(__fmul_ru(mx, c), -7.f);
          // Lazy rescale: the reference moves only when it would by more than 8; then O (P.V up to this buffer's
          // step before) is scaled in place.  No key yet: -inf - (-inf) is no difference.
          const bool grow = mx - m_run > 8.f;
          const bool scale_o = grow && m_run != -CUDART_INF_F;
          if (__any_sync(0xffffffffu, scale_o)) {
            if (!warp_wait(bar(B_PV_DONE + x), (ph - 1u) & 1u, lane, abort_flag, p.err)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const float f = scale_o ? ex2_approx(m_run - mx) : 1.f;
#pragma unroll 1
            for (int c16 = 0; c16 < 8; ++c16) {
              uint32_t w[16];
              FA3_TMEM_LD16(o_col + c16 * 16, w);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * f);
              FA3_TMEM_ST16(o_col + c16 * 16, w);
            }
          }
          if (grow) {
            l_run = m_run == -CUDART_INF_F ? 0.f : l_run * ex2_approx(m_run - mx);
            m_run = mx;
          }
          const float mc = m_run == -CUDART_INF_F ? 0.f : -m_run;
          // P = exp2(s c - m) as fp16 pairs over the S columns (keys 32 c4 .. 32 c4 + 31 go to columns
          // 16 c4 .. 16 c4 + 15); the row sum takes the weights before the rounding.
          float l0 = 0.f, l1 = 0.f;
          auto weigh = [&](const uint32_t (&w)[16], uint32_t (&pk)[8]) {
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              float p0, p1;
              fma2(p0, p1, __uint_as_float(w[e]), __uint_as_float(w[e + 1]), c, c, mc, mc);
              p0 = ex2_approx(p0);
              p1 = ex2_approx(p1);
              add2(l0, l1, l0, l1, p0, p1);
              pk[e / 2] = pack_f16x2(p0, p1);
            }
          };
          uint32_t pa[8], pb[8];
          wait_ld16(v0);
          FA3_TMEM_LD16(scol + 16, v1);
          weigh(v0, pa);
#pragma unroll 1
          for (uint32_t k = 0; k < 96; k += 32) {
            wait_ld16(v1);
            FA3_TMEM_LD16(scol + k + 32, v0);
            weigh(v1, pb);
            tmem_st8(scol + k / 2, pa);
            wait_ld16(v0);
            FA3_TMEM_LD16(scol + k + 48, v1);
            weigh(v0, pa);
            tmem_st8(scol + k / 2 + 8, pb);
          }
          wait_ld16(v1);
          weigh(v1, pb);
          tmem_st8(scol + 48, pa);
          tmem_st8(scol + 56, pb);
          l_run += l0 + l1;
          tmem_wait_st();
          tc_fence_before();
        }
        warp_arrive(B_P_FULL + x);
      }
      if (!ok) break;
      done += (uint32_t)mine;
      done_other += (uint32_t)(steps - mine);
      // ---------------------------------------------------------- epilogue
      // O_x is complete when the buffer's last P.V is.  A single row tile has both buffers' results for
      // the same rows: both warpgroups read both and write half of the columns each.
      if (mine > 0) ok = warp_wait(bar(B_PV_DONE + x), (done - 1u) & 1u, lane, abort_flag, p.err);
      float f_mine = 1.f, f_other = 0.f;
      bool both = false;
      if (!u.dual) {
        ml[x * kRows + r] = make_float2(m_run, l_run);
        warp_arrive(B_ML + x);
        ok = ok && warp_wait(bar(B_ML + (x ^ 1)), merges & 1u, lane, abort_flag, p.err);
        both = steps > mine;
        if (ok && both) ok = warp_wait(bar(B_PV_DONE + (x ^ 1)), (done_other - 1u) & 1u, lane, abort_flag, p.err);
        if (!ok) break;
        const float2 o = ml[(x ^ 1) * kRows + r];
        const float m = fmaxf(m_run, o.x);
        f_mine = m_run == -CUDART_INF_F ? 0.f : ex2_approx(m_run - m);
        f_other = o.x == -CUDART_INF_F ? 0.f : ex2_approx(o.x - m);
        l_run = l_run * f_mine + o.y * f_other;
        m_run = m;
        ++merges;
      }
      if (!ok) break;
      tc_fence_after();
      if (warp_active) {
        const bool whole = u.whole();
        const float inv = !whole ? 1.f : l_run > 0.f ? p.v_scale[u.g] / l_run : 0.f;
        f_mine *= inv;
        f_other *= inv;
        const int slot = 2 * (int)blockIdx.x + (u.first ? 1 : 0);
        const int prow = (u.dual ? x * kRows : 0) + r;
        float4* po = p.part_o + (int64_t)slot * (kD / 4) * p.rows_max + prow;
        const int c_begin = u.dual ? 0 : x * 4, c_end = u.dual ? 8 : c_begin + 4;      // groups of 16 columns
#pragma unroll 1
        for (int c16 = c_begin; c16 < c_end; ++c16) {
          uint32_t a[16], b2[16];
          if (mine > 0) FA3_TMEM_LD16(o_col + c16 * 16, a);
          if (both) FA3_TMEM_LD16(tmem + lane_base + TM_O + (x ^ 1) * 128 + c16 * 16, b2);
          tmem_wait_ld();
          float f[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            f[e] = f_mine == 0.f || mine == 0 ? 0.f : __uint_as_float(a[e]) * f_mine;
            if (both && f_other != 0.f) f[e] = fmaf(__uint_as_float(b2[e]), f_other, f[e]);
          }
          if (active) {
            if (whole) {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                const __nv_bfloat162 bb = __floats2bfloat162_rn(f[e], f[e + 1]);
                w[e / 2] = *reinterpret_cast<const uint32_t*>(&bb);
              }
              uint4* o = reinterpret_cast<uint4*>(p.out + orow * kD + c16 * 16);
              o[0] = make_uint4(w[0], w[1], w[2], w[3]);
              o[1] = make_uint4(w[4], w[5], w[6], w[7]);
            } else {
#pragma unroll
              for (int q4 = 0; q4 < 4; ++q4)
                po[(int64_t)(c16 * 4 + q4) * p.rows_max] = make_float4(f[4 * q4], f[4 * q4 + 1], f[4 * q4 + 2], f[4 * q4 + 3]);
            }
          }
        }
        if (!whole && active && (u.dual || x == 0)) p.part_ml[(int64_t)slot * p.rows_max + prow] = make_float2(m_run, l_run);
      }
      if (!u.dual) {
        // the other warpgroup's next P.V may overwrite what this one reads, and this one's that one's
        tc_fence_before();
        warp_arrive(B_READ + x);
        ok = warp_wait(bar(B_READ + (x ^ 1)), (merges - 1u) & 1u, lane, abort_flag, p.err);
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

// Merges the parts of cut units.  Block (c - 1, rows): the unit whose first cut lies before CTA c's part; rows
// 32 blockIdx.y .. + 31.  A lane has a row, a warp 16 columns.  It is launched while the main kernel runs and takes
// about 3 us behind its end, for a few MB at most; the cuts come from the main kernel, because finding them
// here again took 2 us more.
__global__ void __launch_bounds__(256) chunk_combine_kernel(const __grid_constant__ ChunkParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int prow = blockIdx.y * 32 + lane;                   // row tile x 128 + row
  const int r = prow & (kRows - 1), pl = r / p.G, i = (prow >= kRows ? p.P : 0) + pl;
  pdl_wait();
  pdl_launch_dependents();
  const Cut cut = p.cuts[blockIdx.x + 1];
  if (cut.owner < 0 || cut.last - cut.owner - 1 + cut.own + cut.end < 2) return;   // no cut, or one CTA has all keys
  if ((prow >= kRows && !cut.dual) || pl >= p.P || i >= cut.left) return;
  const int k0 = cut.owner + (cut.own ? 0 : 1), k1 = cut.last - (cut.end ? 0 : 1);
  auto slot_of = [&](int cta) { return 2 * (int64_t)cta + (cta == cut.owner ? 1 : 0); };
  float m = -CUDART_INF_F;
  for (int k = k0; k <= k1; ++k) m = fmaxf(m, p.part_ml[slot_of(k) * p.rows_max + prow].x);
  float l = 0.f, o[16] = {};
  for (int k = k0; k <= k1; ++k) {
    const float2 ml = p.part_ml[slot_of(k) * p.rows_max + prow];
    if (ml.x == -CUDART_INF_F) continue;
    const float f = ex2_approx(ml.x - m);
    l = fmaf(ml.y, f, l);
    const float4* po = p.part_o + slot_of(k) * (kD / 4) * p.rows_max + prow;
#pragma unroll
    for (int q4 = 0; q4 < 4; ++q4) {
      const float4 a = po[(int64_t)(warp * 4 + q4) * p.rows_max];
      o[4 * q4] = fmaf(a.x, f, o[4 * q4]);
      o[4 * q4 + 1] = fmaf(a.y, f, o[4 * q4 + 1]);
      o[4 * q4 + 2] = fmaf(a.z, f, o[4 * q4 + 2]);
      o[4 * q4 + 3] = fmaf(a.w, f, o[4 * q4 + 3]);
    }
  }
  const float inv = l > 0.f ? p.v_scale[cut.g] / l : 0.f;
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 16; e += 2) {
    const __nv_bfloat162 bb = __floats2bfloat162_rn(o[e] * inv, o[e + 1] * inv);
    w[e / 2] = *reinterpret_cast<const uint32_t*>(&bb);
  }
  const int h = cut.g * p.G + r - pl * p.G;
  uint4* out = reinterpret_cast<uint4*>(p.out + ((int64_t)(cut.row0 + i) * p.Hq + h) * kD + warp * 16);
  out[0] = make_uint4(w[0], w[1], w[2], w[3]);
  out[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// Rows of a unit's partial result: one row tile when no sequence can fill more.
int rows_max_of(int n, int G) { return n > kRows / G ? 2 * kRows : kRows; }

size_t workspace_bytes_of(int ctas, int rows_max) {
  return (size_t)2 * ctas * rows_max * (kD * sizeof(float) + sizeof(float2)) + (size_t)ctas * sizeof(Cut);
}

}  // namespace
}  // namespace fa3

using namespace fa3;

FA3_API size_t fa3_chunk_workspace_size(int n, int B, int Hq, int Hkv, int D) {
  if (n <= 0 || B <= 0 || Hq <= 0 || Hkv <= 0 || D != kD || Hq % Hkv != 0 || Hq / Hkv > kRows) return 0;
  int sms = 0;
  if (check_device(&sms) != FA3_OK) sms = 152;
  return workspace_bytes_of(sms, rows_max_of(n, Hq / Hkv));
}

namespace {
// The cache as [rows][Hkv * 128] bytes in boxes of box rows of one KV head.
bool cache_map(CUtensorMap* map, const int8_t* base, int Hkv, int64_t rows, int box) {
  const auto encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)Hkv * kD, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)Hkv * kD};
  const cuuint32_t boxes[2] = {kD, (cuuint32_t)box}, step[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(base), dims, strides, boxes, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int chunk_attn(ChunkParams& p, int D, float softmax_scale, void* workspace, size_t workspace_bytes, void* stream) {
  if (!p.q || !p.k || !p.v || !p.q_scale || !p.k_scale || !p.v_scale || !p.q_start || !p.kv_lens || !p.out)
    return FA3_EINVAL;
  if (p.n <= 0 || p.B <= 0 || p.T <= 0 || p.Hq <= 0 || p.Hkv <= 0 || D <= 0 || p.Hq % p.Hkv != 0) return FA3_EINVAL;
  if (!(softmax_scale > 0.f) || !std::isfinite(softmax_scale)) return FA3_EINVAL;
  p.G = p.Hq / p.Hkv;
  if (D != kD || p.G > kRows || p.Hkv > 65535 || p.n >= (1 << 27) - 1 || p.B > kMostSequences) return FA3_ERANGE;
  if ((p.block_table ? (int64_t)p.num_pages * p.page_size : (int64_t)p.B * p.T) >= ((int64_t)1 << 31)) return FA3_ERANGE;
  if (!aligned16(p.q) || !aligned16(p.k) || !aligned16(p.v) || !aligned16(p.out)) return FA3_ERANGE;
  p.P = kRows / p.G;
  p.div_2p = make_divu32((uint32_t)(2 * p.P));
  p.narrow = ((double)p.n / (2 * p.P) + p.B) * p.Hkv * (kUnitCost + kTileDual * (p.T / kKeys + 1.0)) < 16777216.0;
  p.sm_log2 = softmax_scale * 1.4426950408889634f;
  int sms = 0;
  const int st = check_device(&sms);
  if (st != FA3_OK) return st;
  p.ctas = sms;
  p.rows_max = rows_max_of(p.n, p.G);
  if (!workspace || workspace_bytes < workspace_bytes_of(sms, p.rows_max) || !aligned16(workspace)) return FA3_EWORKSPACE;
  p.part_o = static_cast<float4*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + (size_t)2 * sms * (kD / 4) * p.rows_max);
  p.cuts = reinterpret_cast<Cut*>(p.part_ml + (size_t)2 * sms * p.rows_max);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t cache_rows = p.block_table ? (int64_t)p.num_pages * p.page_size : (int64_t)p.B * p.T;
  p.box = p.block_table ? std::min(kKeys, p.page_size & -p.page_size) : kKeys;
  if (p.box < kLeastBox) p.box = 0;
  if (p.box && (!cache_map(&p.map_k, p.k, p.Hkv, cache_rows, p.box) || !cache_map(&p.map_v, p.v, p.Hkv, cache_rows, p.box)))
    return FA3_ECUDA;
  static std::atomic<bool> set[64];                          // the kernel's attribute, once a device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return FA3_ECUDA;
  if (dev >= 64 || !set[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(gqa_chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_CHUNK) != cudaSuccess)
      return FA3_ECUDA;
    if (dev < 64) set[dev].store(true, std::memory_order_release);
  }
  const LaunchTogether together(s);
  if (launch_pdl(gqa_chunk_kernel, dim3((unsigned)sms), dim3(kThreadsC), SMEM_CHUNK, s, p) != cudaSuccess)
    return FA3_ECUDA;
  if (sms > 1 && launch_pdl(chunk_combine_kernel, dim3((unsigned)(sms - 1), (unsigned)(p.rows_max / 32)), dim3(256), 0, s,
                            p) != cudaSuccess)
    return FA3_ECUDA;
  return FA3_OK;
}
}  // namespace

FA3_API int fa3_prefill_attn_gqa_paged(const int8_t* q, const int8_t* k, const int8_t* v, const float* q_scale,
                                       const float* k_scale, const float* v_scale, const int32_t* q_start,
                                       const int32_t* kv_lens, const int32_t* block_table, uint16_t* out, int n, int B,
                                       int Hq, int Hkv, int D, int num_pages, int page_size, int max_pages,
                                       float softmax_scale, void* workspace, size_t workspace_bytes, int32_t* dev_err,
                                       void* stream) {
  if (!block_table || num_pages <= 0 || page_size <= 0 || max_pages <= 0) return FA3_EINVAL;
  if ((int64_t)max_pages * page_size >= ((int64_t)1 << 31)) return FA3_ERANGE;
  ChunkParams p = {};
  p.q = q; p.k = k; p.v = v; p.q_scale = q_scale; p.k_scale = k_scale; p.v_scale = v_scale; p.q_start = q_start;
  p.kv_lens = kv_lens; p.block_table = block_table; p.out = out; p.err = dev_err;
  p.n = n; p.B = B; p.T = max_pages * page_size; p.Hq = Hq; p.Hkv = Hkv; p.causal = 1;
  p.page_size = page_size; p.max_pages = max_pages; p.num_pages = num_pages;
  p.div_ps = make_divu32((uint32_t)page_size);
  return chunk_attn(p, D, softmax_scale, workspace, workspace_bytes, stream);
}

FA3_API int fa3_cross_attn_gqa(const int8_t* q, const int8_t* k, const int8_t* v, const float* q_scale,
                               const float* k_scale, const float* v_scale, const int32_t* q_start,
                               const int32_t* enc_lens, uint16_t* out, int n, int B, int T, int Hq, int Hkv, int D,
                               float softmax_scale, void* workspace, size_t workspace_bytes, int32_t* dev_err,
                               void* stream) {
  ChunkParams p = {};
  p.q = q; p.k = k; p.v = v; p.q_scale = q_scale; p.k_scale = k_scale; p.v_scale = v_scale; p.q_start = q_start;
  p.kv_lens = enc_lens; p.out = out; p.err = dev_err;
  p.n = n; p.B = B; p.T = T; p.Hq = Hq; p.Hkv = Hkv; p.causal = 0;
  return chunk_attn(p, D, softmax_scale, workspace, workspace_bytes, stream);
}
