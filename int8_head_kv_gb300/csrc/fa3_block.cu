// A paged INT8 cache that needs no calibration: every block of tokens has, for each KV head, a scale of its own for its
// keys and one for its values.  Here: the append that writes it, and the eviction that cuts it down.
//
// Append.  For each block that gets new rows, x the values of one head's new rows in it, a = max |x| of the finite ones:
//   s = fl(a / 127); if the block has tokens already (codes c, scale s0): s = max(s, s0), c = RNE(c * fl(s0 / s))
//   code = clamp(RNE(fl(x / s)), -127, 127)       (s = 0 -> 0)
// A block's scale only grows, so a token's codes are rewritten when a later one is larger, each time off by half a step at
// most, and what the scale is does not depend on how the block's tokens were split over calls.
//
// A ragged batch of 6168 new tokens (8 heads, blocks of 32) takes 12.9 us, 16 single tokens 3.4 us: one wave of blocks, each a chain of
// lengths, page, rows, the greatest of them and the codes; 38 MB are 5.6 us of HBM.
#include "fa3_packed.cuh"

#include <algorithm>
#include <atomic>

namespace fa3 {
namespace {

constexpr int kAppendThreads = 256;

struct AppendArgs {
  const uint16_t* x[2];            // bf16 rows of k, v
  int8_t* cache[2];
  float* scale[2];
  int64_t stride[2];               // elements from row to row
  const int32_t* q_start;
  const int32_t* kv_lens;
  int32_t* err;
  Pages pg;
  int n, B, D, chunks, wide;       // chunks: groups of 8 values a row; wide: rows 16-byte aligned
  DivU32 div_chunks;
};

__device__ __forceinline__ uint4 load8(const uint16_t* p, bool wide) {
  if (wide) return *reinterpret_cast<const uint4*>(p);
  const uint2 a = reinterpret_cast<const uint2*>(p)[0], b = reinterpret_cast<const uint2*>(p)[1];
  return make_uint4(a.x, a.y, b.x, b.y);
}
// The largest magnitude of 8 bf16 values, as its 15 bits (their order is the magnitudes'); of those that are finite.
__device__ __forceinline__ uint32_t amax8(uint4 v, uint32_t m) {
  return __vmaxu2(m, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
}
__device__ __forceinline__ uint32_t amax8_finite(uint4 v, uint32_t m) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t a = w[k] & 0x7fff7fffu;
    m = __vmaxu2(m, a & __vcmpltu2(a, 0x7f807f80u));
  }
  return m;
}
// Codes of eight bf16 values, quant_code's.
__device__ __noinline__ uint2 codes8_divided(uint4 v, float s) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[2] = {0u, 0u};
#pragma unroll 1
  for (int e = 0; e < 8; ++e) {
    const uint32_t x = (e & 4 ? (e & 2 ? w[3] : w[2]) : (e & 2 ? w[1] : w[0])) >> (16 * (e & 1));
    c[e >> 2] |= ((uint32_t)quant_code(bf16_to_float(x & 0xffffu), s) & 0xffu) << (8 * (e & 3));
  }
  return make_uint2(c[0], c[1]);
}
// The same where `plain`: s in [2^-100, 2^100], every value finite and at most 127 s in magnitude.  Values next to half
// steps are no rare case here: with a the block's greatest, x / s = 127 x / a is a half step, but for s's rounding, whenever the
// eight bits of x and a are such, which a warp's 256 values meet two times in three.  So the float32 quotient itself decides: two
// corrections of x rs by its residual, which one fused operation gives exactly, round it correctly (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990; rs is 1 / s rounded correctly), and adding 1.5 2^23
// rounds it to a whole number, half to even.
__device__ __forceinline__ uint2 codes8(uint4 v, float s, float rs, bool plain) {
  if (!plain) return codes8_divided(v, s);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const unsigned long long rs2 = f32x2_pack(rs, rs), s2 = f32x2_pack(-s, -s), one2 = f32x2_pack(1.f, 1.f),
                           zero2 = f32x2_pack(0.f, 0.f), magic2 = f32x2_pack(kCodeMagic, kCodeMagic);
  uint32_t q[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const unsigned long long x = f32x2_pack(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
    unsigned long long y = f32x2_fma(x, rs2, zero2);
    y = f32x2_fma(f32x2_fma(y, s2, x), rs2, y);
    y = f32x2_fma(f32x2_fma(y, s2, x), rs2, y);
    float t0, t1;
    f32x2_unpack(f32x2_fma(y, one2, magic2), t0, t1);
    q[2 * k] = __float_as_uint(t0);
    q[2 * k + 1] = __float_as_uint(t1);
  }
  return make_uint2(__byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410));
}

// Block (piece, heads, k or v): W warps have a block of tokens of one head.  A thread keeps up to 8 groups of 8 values, in shared
// memory, so that they are read once where W warps hold a block; larger blocks are read again (from L2).  The loops stay
// short: with 16 groups in registers and all their code in a row, instructions were what the warps waited for (a ragged batch
// of 6168 new tokens, 8 heads, blocks of 32: 54 us; 13.1 so).
constexpr int kHeld = 8, kAsk = 8;
constexpr int kAppendSmem = kAppendThreads * kHeld * 16;
static_assert(kAppendSmem + 1024 <= 48 * 1024, "no attribute of the kernel's needed");
template <int W>
__global__ void __launch_bounds__(kAppendThreads) block_append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int kHeads = kAppendThreads / 32 / W;
  __shared__ Piece found;
  __shared__ uint32_t warp_max[kAppendThreads / 32];
  extern __shared__ uint4 kept[];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, kv = blockIdx.z, h = blockIdx.y * kHeads + warp / W;
  const int tid = threadIdx.x % (32 * W);                    // in the block of tokens
  const Piece p = find_piece(a.q_start, a.kv_lens, a.B, a.n, a.pg.T_max, a.pg.div_block, 2, blockIdx.x,
                             (blockIdx.x | blockIdx.y | blockIdx.z) == 0, a.err, &found);
  if (p.b < 0) return;
  // Tokens [lo, hi) of the block are new, [base, lo) were there.
  const int start = p.nkv - p.nq, blk = (int)divu32((uint32_t)start, a.pg.div_block) + p.index;
  const int base = blk * a.pg.block, lo = max(base, start), hi = min(base + a.pg.block, p.nkv);
  if (base >= p.nkv) return;
  const bool mine = h < a.pg.Hkv;
  const int items = mine ? (hi - lo) * a.chunks : 0;
  const int pi = (int)divu32((uint32_t)base, a.pg.div_ps), page = a.pg.table[(int64_t)p.b * a.pg.max_pages + pi];
  const uint16_t* x = a.x[kv] + (int64_t)(p.q0 + lo - start) * a.stride[kv] + (int64_t)h * a.D;
  // A thread's groups are 32 W apart: their offsets go on from one to the next.
  const int rows_on = (int)divu32(32u * W, a.div_chunks), chunks_on = 32 * W - rows_on * a.chunks;
  const int row0 = (int)divu32((uint32_t)tid, a.div_chunks), c0 = tid - row0 * a.chunks;
  struct Walk {
    int c;
    int64_t off;
  };
  auto begin = [&](int64_t stride) { return Walk{c0, row0 * stride + c0 * 8}; };
  auto next = [&](Walk& w, int64_t stride) {
    w.c += chunks_on;
    w.off += rows_on * stride + chunks_on * 8;
    if (w.c >= a.chunks) {
      w.c -= a.chunks;
      w.off += stride - a.chunks * 8;
    }
  };
  const int64_t x_step = a.stride[kv];
  const bool wide = a.wide;
  uint32_t m = 0;
  Walk in = begin(x_step);
  int i = tid;
#pragma unroll 1
  for (int k = 0; k < kHeld && i < items; k += kAsk) {
    uint4 v[kAsk];
#pragma unroll
    for (int e = 0; e < kAsk; ++e, i += 32 * W) {
      v[e] = make_uint4(0u, 0u, 0u, 0u);
      if (i < items) v[e] = load8(x + in.off, wide);
      next(in, x_step);
    }
#pragma unroll
    for (int e = 0; e < kAsk; ++e) {
      m = amax8(v[e], m);
      kept[(k + e) * kAppendThreads + threadIdx.x] = v[e];
    }
  }
  if ((uint32_t)page >= (uint32_t)a.pg.num_pages) {
    if (threadIdx.x == 0) set_dev_err(a.err, FA3_DEVERR_PAGE);
    return;
  }
  const int at = base - pi * a.pg.page_size;                 // of the block in its page
  float* scale = a.scale[kv] + ((int64_t)page * a.pg.per_page + (int)divu32((uint32_t)at, a.pg.div_block)) * a.pg.Hkv + (mine ? h : 0);
  const float before = lo > base ? *scale : 0.f;
  for (; i < items; i += 32 * W) {
    m = amax8(load8(x + in.off, wide), m);
    next(in, x_step);
  }
  bool plain = max(m & 0xffffu, m >> 16) < 0x7f80u;
  if (!plain) {                                              // some value is not finite: again, without those
    m = 0;
    in = begin(x_step);
    for (i = tid; i < items; i += 32 * W) {
      m = amax8_finite(load8(x + in.off, wide), m);
      next(in, x_step);
    }
  }
  m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
  if constexpr (W > 1) {
    if ((threadIdx.x & 31) == 0) warp_max[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) m = max(m, warp_max[warp / W * W + w]);
  } else {
    __syncwarp();
  }
  if (!mine) return;
  float s = __fdiv_rn(bf16_to_float(m), 127.f);
  int8_t* rows0 = a.cache[kv] + ((int64_t)page * a.pg.page_size + at) * a.pg.Hkv * a.D + (int64_t)h * a.D;   // token `base`
  const int64_t step = (int64_t)a.pg.Hkv * a.D;
  if (lo > base) {
    if (s > before) {
      const float ratio = __fdiv_rn(before, s);
      for (int i = tid; i < (lo - base) * a.chunks; i += 32 * W) {
        const int row = (int)divu32((uint32_t)i, a.div_chunks);
        uint2* c = reinterpret_cast<uint2*>(rows0 + row * step + (i - row * a.chunks) * 8);
        const uint2 w = *c;
        *c = make_uint2(rescaled(w.x, ratio), rescaled(w.y, ratio));
      }
    } else {
      s = before;
    }
  }
  if (tid == 0) *scale = s;                                  // all have read it: the barrier above
  const float rs = __fdiv_rn(1.f, s);
  plain = plain && exact_scale(s);
  int8_t* out = rows0 + (lo - base) * step;
  in = begin(x_step);
  Walk to = begin(step);
  i = tid;
#pragma unroll 2
  for (int k = 0; k < kHeld; ++k, i += 32 * W) {
    if (i < items) *reinterpret_cast<uint2*>(out + to.off) = codes8(kept[k * kAppendThreads + threadIdx.x], s, rs, plain);
    next(in, x_step);
    next(to, step);
  }
  for (; i < items; i += 32 * W) {
    *reinterpret_cast<uint2*>(out + to.off) = codes8(load8(x + in.off, wide), s, rs, plain);
    next(in, x_step);
    next(to, step);
  }
}

// ------------------------------------------------------------------ eviction
// Of each sequence and KV head the first `sinks` tokens stay, the last `recent`, and of the others those with the
// greatest weights, the earliest of equal ones, up to `budget` in all; a context that fits the budget stays whole.
//
// The choice is a radix selection by one block a head and sequence: 16 contexts of 4096 tokens and 8 heads take 8.8 us, three of
// up to 20001 tokens and 5 heads 13.0 (15 blocks: latency, barriers and instructions, far from HBM).  A cluster of blocks a head
// was slower.  Contexts beyond kMostKeys are read again for each digit (a whole call on one of 49000 tokens, 8 heads: 35 us, of 60000
// 72, of 100000 110).  Shared memory goes by the table's width, the lengths being on the device: one block an SM instead of
// two from 20000 tokens on (128 contexts of 2048 cut to 1024: 164 us, with a table for 131072 tokens 184).
constexpr int kPickThreads = 1024;
constexpr int kDigitBits = 11, kBins = 1 << kDigitBits;
constexpr int kMostKeys = 48 * 1024;                       // of a context that shared memory holds

struct EvictArgs {
  int8_t* cache[2];
  float* scale[2];
  float* weights;                  // [num_pages][Hkv][page_size]
  const int32_t* kv_lens;
  const int32_t* new_table;        // [B][new_pages]
  int32_t* kept;                   // [B][Hkv][budget]
  int32_t* new_lens;               // [B]
  int32_t* err;
  Pages pg;
  int B, D, new_pages, budget, sinks, recent, cached;
  int rows, unit, chunks;          // tokens of a block of evict_move_kernel; bytes it moves at once, how many times a row
  DivU32 div_chunks;
};

// Order-preserving bits: NaN above all, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive prefix sums over the block's 1024 threads (`tmp` holds 32 values).
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* tmp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  __syncthreads();
  if (lane == 31) tmp[warp] = s;
  __syncthreads();
  if (warp == 0) {
    uint32_t t = tmp[lane];
    const uint32_t mine = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += y;
    }
    tmp[lane] = t - mine;
  }
  __syncthreads();
  return tmp[warp] + s - v;
}

// Block (head, sequence): the tokens that stay, in order, to `kept`.
constexpr int kFewKeys = 4096;
__global__ void __launch_bounds__(kPickThreads) evict_pick_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ __align__(16) uint32_t keys[];           // of all tokens that are chosen from, where they fit
  __shared__ uint32_t bins[2][kBins], sums[2][32], tmp[32], few[kFewKeys], n_few;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, g = blockIdx.x, b = blockIdx.y;
  const int T = a.kv_lens[b];
  int32_t* kept = a.kept + ((int64_t)b * a.pg.Hkv + g) * a.budget;
  if (T < 0 || T > a.pg.T_max) {
    if (tid == 0 && g == 0) set_dev_err(a.err, FA3_DEVERR_LENS);
    return;
  }
  const int left = min(T, a.budget);
  if (tid == 0 && g == 0) a.new_lens[b] = left;
  for (int i = left + tid; i < a.budget; i += kPickThreads) kept[i] = -1;
  if (T <= a.budget) {
    for (int i = tid; i < T; i += kPickThreads) kept[i] = i;
    return;
  }
  for (int i = tid; i < a.sinks; i += kPickThreads) kept[i] = i;
  for (int i = tid; i < a.recent; i += kPickThreads) kept[a.budget - a.recent + i] = T - a.recent + i;
  const int c0 = a.sinks, c1 = T - a.recent, want = a.budget - a.sinks - a.recent;   // want < c1 - c0
  if (want == 0) return;
  // Tokens go by fours, which lie in one page: group q holds tokens base + 4 q .. + 3, with key 0, which no weight has, outside
  // [c0, c1).  kLoads groups a thread are on their way at once.
  constexpr int kLoads = 4;
  const int base = c0 & ~3, groups = (c1 - base + 3) >> 2;
  const int32_t* table = a.pg.table + (int64_t)b * a.pg.max_pages;
  auto load = [&](int q0, int stride, uint4 (&k)[kLoads]) {
    int page[kLoads];
    uint32_t t[kLoads];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      t[i] = (uint32_t)(base + 4 * min(q0 + i * stride, groups - 1));
      page[i] = table[divu32(t[i], a.pg.div_ps)];
    }
    float4 w[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if ((uint32_t)page[i] >= (uint32_t)a.pg.num_pages) {   // outside the pool: any page of it
        bad = true;
        page[i] = 0;
      }
      const int at = (int)(t[i] - divu32(t[i], a.pg.div_ps) * (uint32_t)a.pg.page_size);
      w[i] = *reinterpret_cast<const float4*>(a.weights + ((int64_t)page[i] * a.pg.Hkv + g) * a.pg.page_size + at);
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      auto in = [&](int e, float x) {
        const int u = (int)t[i] + e;
        return u >= c0 && u < c1 ? weight_key(x) : 0u;
      };
      k[i] = make_uint4(in(0, w[i].x), in(1, w[i].y), in(2, w[i].z), in(3, w[i].w));
    }
    if (bad) set_dev_err(a.err, FA3_DEVERR_PAGE);
  };
  const bool cached = 4 * groups <= a.cached;
  uint4* const keys4 = reinterpret_cast<uint4*>(keys);
  // A thread's run of groups (an odd number of them: eight threads' groups then lie in different banks).
  const int per = ((groups + kPickThreads - 1) / kPickThreads) | 1;
  const int g0 = (int)min((int64_t)groups, (int64_t)tid * per), g1 = (int)min((int64_t)groups, (int64_t)tid * per + per);
  // calls use(group, its keys) for this thread's run, in order
  auto run = [&](auto use) {
    if (cached) {
      for (int q = g0; q < g1; ++q) use(q, keys4[q]);
    } else {
      for (int q = g0; q < g1; q += kLoads) {
        uint4 k[kLoads];
        load(q, 1, k);
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          if (q + i < g1) use(q + i, k[i]);
      }
    }
  };
  auto four = [](uint4 k, auto use) {
    use(0, k.x);
    use(1, k.y);
    use(2, k.z);
    use(3, k.w);
  };
  // The want-th greatest key, digit by digit from the top.  Behind the first digit few keys are left as a rule, which are put
  // aside.  Of a run that shared memory holds, a bit a token says from there on which are above that digit and which have it, so
  // the run is not read again.
  static_assert(4 * ((kMostKeys / 4 + kPickThreads - 1) / kPickThreads | 1) <= 64, "bits of a run");
  unsigned long long above = 0, among = 0;
  auto bits_of = [](unsigned long long m, auto use) {
    for (; m; m &= m - 1) use(__ffsll((long long)m) - 1);
  };
  uint32_t prefix = 0, need = (uint32_t)want;
  bool aside = false;
  for (int i = tid; i < kBins; i += kPickThreads) bins[0][i] = 0;
  if (tid == 0) n_few = 0;
  __syncthreads();
#pragma unroll 1
  for (int shift = 32, buf = 0; shift > 0; buf ^= 1) {
    const int bits = min(kDigitBits, shift), rest = shift - bits;
    const uint32_t mask = (1u << bits) - 1u;
    uint32_t* const count = bins[buf];
    if (shift == 32) {
      // tokens that nothing looked at are many: counted by the thread
      constexpr uint32_t kZero = 0x80000000u;
      uint32_t zeros = 0;
      for (int q = tid; q < groups; q += kLoads * kPickThreads) {
        uint4 k[kLoads];
        load(q, kPickThreads, k);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          if (q + i * kPickThreads < groups) {
            if (cached) keys4[q + i * kPickThreads] = k[i];
            four(k[i], [&](int, uint32_t x) {
              if (x == kZero) ++zeros; else if (x) atomicAdd(&count[x >> rest], 1u);
            });
          }
        }
      }
      zeros = __reduce_add_sync(0xffffffffu, zeros);
      if (lane == 0 && zeros) atomicAdd(&count[kZero >> rest], zeros);
    } else if (aside) {
      const int n = (int)n_few;
      for (int i = tid; i < n; i += kPickThreads)
        if (few[i] >> shift == prefix) atomicAdd(&count[(few[i] >> rest) & mask], 1u);
    } else {
      // all keys again: many are equal then, and equal neighbours are counted by the thread
      uint32_t last = 0, times = 0;
      run([&](int, uint4 k) {
        four(k, [&](int, uint32_t x) {
          if (!x || x >> shift != prefix) return;
          if (x != last) {
            if (times) atomicAdd(&count[(last >> rest) & mask], times);
            last = x;
            times = 0;
          }
          ++times;
        });
      });
      if (times) atomicAdd(&count[(last >> rest) & mask], times);
    }
    __syncthreads();
    // A thread has two bins, the greatest first, and a warp the sum of its 64; then every warp finds the digit for itself.  The other
    // bins, which all have read, are cleared meanwhile.
    const uint32_t mine = __reduce_add_sync(0xffffffffu, count[kBins - 1 - 2 * tid] + count[kBins - 2 - 2 * tid]);
    if (lane == 0) sums[buf][tid >> 5] = mine;
    for (int i = tid; i < kBins; i += kPickThreads) bins[buf ^ 1][i] = 0;
    __syncthreads();
    // the lane whose values, summed up from lane 0 on, reach `need`; what lies in front of them is taken off it
    auto reach = [&](uint32_t v) {
      uint32_t upto = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      const int l = __ffs(__ballot_sync(0xffffffffu, upto >= need)) - 1;
      need -= __shfl_sync(0xffffffffu, upto - v, l);
      return l;
    };
    const int w = reach(sums[buf][lane]), hi = kBins - 1 - 64 * w;
    const uint32_t n0 = count[hi - 2 * lane], n1 = count[hi - 2 * lane - 1];
    const int l = reach(n0 + n1);
    const uint32_t f0 = __shfl_sync(0xffffffffu, n0, l), f1 = __shfl_sync(0xffffffffu, n1, l);
    const bool second = f0 < need;
    if (second) need -= f0;
    prefix = (shift == 32 ? 0u : prefix << bits) | (uint32_t)(hi - 2 * l - second);
    if (shift == 32) {
      if (cached) {
        for (int q = g0; q < g1; ++q) {
          const uint4 k = keys4[q];
          uint32_t up = 0, here = 0;
          four(k, [&](int e, uint32_t x) {
            up |= (uint32_t)(x >> rest > prefix) << e;
            here |= (uint32_t)(x && x >> rest == prefix) << e;
          });
          above |= (unsigned long long)up << (4 * (q - g0));
          among |= (unsigned long long)here << (4 * (q - g0));
        }
      }
      if ((second ? f1 : f0) <= kFewKeys) {
        aside = true;
        if (cached) {
          if (among) {
            uint32_t to = atomicAdd(&n_few, (uint32_t)__popcll(among));
            bits_of(among, [&](int i) { few[to++] = keys[4 * g0 + i]; });
          }
        } else {
          run([&](int, uint4 k) {
            four(k, [&](int, uint32_t x) {
              if (x && x >> rest == prefix) few[atomicAdd(&n_few, 1u)] = x;
            });
          });
        }
        __syncthreads();
      }
    }
    shift = rest;
  }
  // Kept: greater than `prefix`, or equal to it and one of the first `need` such.
  uint32_t more = 0, same = 0;
  unsigned long long equal = 0;
  if (cached) {
    bits_of(among, [&](int i) {
      const uint32_t x = keys[4 * g0 + i];
      above |= (unsigned long long)(x > prefix) << i;
      equal |= (unsigned long long)(x == prefix) << i;
    });
    more = (uint32_t)__popcll(above);
    same = (uint32_t)__popcll(equal);
  } else {
    run([&](int, uint4 k) {
      four(k, [&](int, uint32_t x) {
        more += x > prefix;
        same += x == prefix;
      });
    });
  }
  uint32_t seen, at;
  if (cached) {                                              // both counts at once: they stay below 2^16
    static_assert(kMostKeys < 65536, "counts in 16 bits");
    const uint32_t before = block_scan(more << 16 | same, tmp);
    seen = before & 0xffffu;
    at = before >> 16;
  } else {
    seen = block_scan(same, tmp);
    at = block_scan(more, tmp);
  }
  at += min(seen, need);
  if (cached) {
    bits_of(above | equal, [&](int i) {
      const bool is_equal = equal >> i & 1;
      if (!is_equal || seen < need) kept[a.sinks + at++] = base + 4 * g0 + i;
      seen += is_equal;
    });
  } else {
    run([&](int q, uint4 k) {
      four(k, [&](int e, uint32_t x) {
        const bool stays = x > prefix || (x == prefix && seen < need);
        seen += x == prefix;
        if (stays) kept[a.sinks + at++] = base + 4 * q + e;
      });
    });
  }
}

constexpr int kMoveThreads = 128, kMoveTokens = 32;         // tokens of a block, whose blocks of scales stay together

// Block (rows, head, sequence): `rows` tokens of the new context, whole blocks of it, as codes at the greatest of their block's
// scales, and their weights.  A thread's pieces, of 16 bytes where rows allow it, are on their way at once and while the
// scales are found.  Its way is a chain of four loads (positions, pages, scales, codes), so many blocks an SM, and small
// ones, are what hides it: 16 contexts of 4096 tokens cut to 1024 take 25.5 us a call so, 28.0 with 5 blocks an SM of 256
// threads and 64 tokens, 25.5 with 7 (an odd batch of three long contexts alike).  17 of them are this kernel's, 4 TB/s: pieces of 128
// bytes, a head's row of one token, from all over the pool.  Asking for the rows from evict_pick_kernel, into L2, was slower
// (28.8 us; the odd batch 27.0 where it takes 18.4).
template <class V>
__global__ void __launch_bounds__(kMoveThreads, 12) evict_move_kernel(const __grid_constant__ EvictArgs a) {
  // per token: row in the old pages and in the new ones (head rows; -1: no such page), scales of k and v; per block: their greatest
  extern __shared__ int64_t src_row[];
  int64_t* const dst_row = src_row + a.rows;
  float* const scale = reinterpret_cast<float*>(dst_row + a.rows);
  int* const most = reinterpret_cast<int*>(scale + 2 * a.rows);
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, g = blockIdx.y, b = blockIdx.z, blocks = a.rows / a.pg.block;
  const int T = a.kv_lens[b];
  if (T < 0 || T > a.pg.T_max) return;
  const int base = blockIdx.x * a.rows, rows = min(a.rows, min(T, a.budget) - base);
  if (rows <= 0) return;
  const int32_t* kept = a.kept + ((int64_t)b * a.pg.Hkv + g) * a.budget + base;
  for (int i = tid; i < 2 * blocks; i += kMoveThreads) most[i] = 0;
  float s[2] = {0.f, 0.f};
  for (int i = tid; i < rows; i += kMoveThreads) {
    const int t = kept[i];
    const uint32_t sp = divu32((uint32_t)t, a.pg.div_ps), dp = divu32((uint32_t)(base + i), a.pg.div_ps);
    int from = a.pg.table[(int64_t)b * a.pg.max_pages + sp];
    const int to = a.new_table[(int64_t)b * a.new_pages + dp];
    if ((uint32_t)from >= (uint32_t)a.pg.num_pages) {        // outside the pool: any page of it
      set_dev_err(a.err, FA3_DEVERR_PAGE);
      from = 0;
    }
    const bool lost = (uint32_t)to >= (uint32_t)a.pg.num_pages;
    if (lost) set_dev_err(a.err, FA3_DEVERR_PAGE);
    const int in = t - (int)sp * a.pg.page_size, at = base + i - (int)dp * a.pg.page_size;
    src_row[i] = ((int64_t)from * a.pg.page_size + in) * a.pg.Hkv + g;
    dst_row[i] = lost ? -1 : ((int64_t)to * a.pg.page_size + at) * a.pg.Hkv + g;
    const float w = a.weights[((int64_t)from * a.pg.Hkv + g) * a.pg.page_size + in];
    const int64_t sc = ((int64_t)from * a.pg.per_page + (int)divu32((uint32_t)in, a.pg.div_block)) * a.pg.Hkv + g;
    s[0] = a.scale[0][sc];
    s[1] = a.scale[1][sc];
    scale[i] = s[0];
    scale[a.rows + i] = s[1];
    if (!lost) a.weights[((int64_t)to * a.pg.Hkv + g) * a.pg.page_size + at] = w;
  }
  __syncthreads();
  // the first pieces are asked for; scales are not negative, so their bits are in their order
  constexpr int kLoads = 4;
  const int items = rows * a.chunks;
  auto where = [&](int j, int& kv, int& row, int& c) {
    kv = j >= items;
    const int i = j - kv * items;
    row = (int)divu32((uint32_t)i, a.div_chunks);
    c = (i - row * a.chunks) * (int)sizeof(V);
  };
  auto load = [&](int j, V (&v)[kLoads]) {
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      int kv, row, c;
      where(min(j + k * kMoveThreads, 2 * items - 1), kv, row, c);
      v[k] = __ldcs(reinterpret_cast<const V*>(a.cache[kv] + src_row[row] * a.D + c));
    }
  };
  V v[kLoads];
  load(tid, v);
  for (int i = tid; i < rows; i += kMoveThreads) {
    const int blk = (int)divu32((uint32_t)i, a.pg.div_block);
    atomicMax(&most[blk], __float_as_int(scale[i]));
    atomicMax(&most[blocks + blk], __float_as_int(scale[a.rows + i]));
  }
  __syncthreads();
  for (int i = tid; i < 2 * rows; i += kMoveThreads) {
    const int kv = i >= rows, row = i - kv * rows, blk = (int)divu32((uint32_t)row, a.pg.div_block);
    const float old = scale[kv * a.rows + row], now = __int_as_float(most[kv * blocks + blk]);
    scale[kv * a.rows + row] = old == now ? 1.f : __fdiv_rn(old, now);   // 0 / 0 with it
    if (row == blk * a.pg.block && dst_row[row] >= 0) {
      const uint32_t dp = divu32((uint32_t)(base + row), a.pg.div_ps);
      const int at = base + row - (int)dp * a.pg.page_size, to = a.new_table[(int64_t)b * a.new_pages + dp];
      a.scale[kv][((int64_t)to * a.pg.per_page + (int)divu32((uint32_t)at, a.pg.div_block)) * a.pg.Hkv + g] = now;
    }
  }
  __syncthreads();
  for (int j = tid; j < 2 * items; j += kLoads * kMoveThreads) {
    if (j != tid) load(j, v);
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      if (j + k * kMoveThreads >= 2 * items) break;
      int kv, row, c;
      where(j + k * kMoveThreads, kv, row, c);
      const float r = scale[kv * a.rows + row];
      uint32_t* w = reinterpret_cast<uint32_t*>(&v[k]);
      if (r != 1.f) {
#pragma unroll
        for (int e = 0; e < (int)sizeof(V) / 4; ++e) w[e] = rescaled(w[e], r);
      }
      if (dst_row[row] >= 0) *reinterpret_cast<V*>(a.cache[kv] + dst_row[row] * a.D + c) = v[k];
    }
  }
}

inline bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

}  // namespace
}  // namespace fa3

using namespace fa3;

FA3_API int fa3_append_gqa_block_paged(const uint16_t* k, const uint16_t* v, int8_t* k_cache, int8_t* v_cache,
                                       float* k_scale, float* v_scale, const int32_t* block_table,
                                       const int32_t* q_start, const int32_t* kv_lens, int n, int B, int Hkv, int D,
                                       int64_t k_stride, int64_t v_stride, int num_pages, int page_size, int max_pages,
                                       int block, int32_t* dev_err, void* stream) {
  if (!k || !v || !k_cache || !v_cache || !k_scale || !v_scale || !q_start || !kv_lens) return FA3_EINVAL;
  if (n <= 0 || D <= 0) return FA3_EINVAL;
  AppendArgs a;
  int st = pages_of(block_table, B, Hkv, num_pages, page_size, max_pages, block, &a.pg);
  if (st != FA3_OK) return st;
  if (D % 8 != 0 || D > 256 || k_stride < 0 || v_stride < 0 || k_stride % 4 != 0 || v_stride % 4 != 0) return FA3_ERANGE;
  if (!aligned8(k) || !aligned8(v) || !aligned8(k_cache) || !aligned8(v_cache) || !aligned4(k_scale) || !aligned4(v_scale))
    return FA3_ERANGE;
  const int64_t pieces = pieces_of(n, B, block, 2);
  if (pieces >= ((int64_t)1 << 31)) return FA3_ERANGE;
  st = check_device(nullptr);
  if (st != FA3_OK) return st;
  a.x[0] = k; a.x[1] = v; a.cache[0] = k_cache; a.cache[1] = v_cache; a.scale[0] = k_scale; a.scale[1] = v_scale;
  a.stride[0] = k_stride; a.stride[1] = v_stride;
  a.q_start = q_start; a.kv_lens = kv_lens; a.err = dev_err; a.n = n; a.B = B; a.D = D; a.chunks = D / 8;
  a.wide = aligned16(k) && aligned16(v) && k_stride % 8 == 0 && v_stride % 8 == 0;
  a.div_chunks = make_divu32((uint32_t)a.chunks);
  // as many warps a block of tokens as hold it
  const int warps = kAppendThreads / 32, need = (block * a.chunks + 32 * kHeld - 1) / (32 * kHeld);
  const int W = need <= 1 ? 1 : need <= 2 ? 2 : need <= 4 ? 4 : 8;
  auto* kernel = W == 1 ? block_append_kernel<1> : W == 2 ? block_append_kernel<2> : W == 4 ? block_append_kernel<4>
                                                                                            : block_append_kernel<8>;
  const int heads = warps / W;
  return cuda_status(launch_pdl(kernel, dim3((unsigned)pieces, (unsigned)((Hkv + heads - 1) / heads), 2), dim3(kAppendThreads), kAppendSmem,
                                static_cast<cudaStream_t>(stream), a));
}

FA3_API int fa3_evict_gqa_block_paged(int8_t* k_cache, int8_t* v_cache, float* k_scale, float* v_scale, float* weights,
                                      const int32_t* block_table, const int32_t* kv_lens, const int32_t* new_table,
                                      int32_t* kept, int32_t* new_lens, int B, int Hkv, int D, int num_pages,
                                      int page_size, int max_pages, int block, int new_pages, int budget, int sinks,
                                      int recent, int32_t* dev_err, void* stream) {
  if (!k_cache || !v_cache || !k_scale || !v_scale || !weights || !kv_lens || !new_table || !kept || !new_lens)
    return FA3_EINVAL;
  if (D <= 0 || new_pages <= 0 || budget <= 0 || sinks < 0 || recent < 0) return FA3_EINVAL;
  EvictArgs a;
  int st = pages_of(block_table, B, Hkv, num_pages, page_size, max_pages, block, &a.pg);
  if (st != FA3_OK) return st;
  if ((int64_t)sinks + recent > budget || (int64_t)budget > (int64_t)new_pages * page_size) return FA3_EINVAL;
  if (D % 8 != 0 || D > 256 || B > 65535 || (int64_t)budget > ((int64_t)1 << 31) - 65536) return FA3_ERANGE;
  if (!aligned8(k_cache) || !aligned8(v_cache) || !aligned4(k_scale) || !aligned4(v_scale) || !aligned16(weights))
    return FA3_ERANGE;
  // (the blocks of other heads would read the lengths that the first has written)
  if (new_lens < kv_lens + B && kv_lens < new_lens + B) return FA3_EINVAL;
  st = check_device(nullptr);
  if (st != FA3_OK) return st;
  a.cache[0] = k_cache; a.cache[1] = v_cache; a.scale[0] = k_scale; a.scale[1] = v_scale; a.weights = weights;
  a.kv_lens = kv_lens; a.new_table = new_table; a.kept = kept; a.new_lens = new_lens; a.err = dev_err;
  a.B = B; a.D = D; a.new_pages = new_pages; a.budget = budget; a.sinks = sinks; a.recent = recent;
  const bool wide = D % 16 == 0 && aligned16(k_cache) && aligned16(v_cache);
  a.unit = wide ? 16 : 8;
  a.chunks = D / a.unit;
  a.div_chunks = make_divu32((uint32_t)a.chunks);
  a.rows = block * std::max(1, kMoveTokens / block);
  a.cached = std::min(a.pg.T_max / 4 * 4 + 8, kMostKeys);   // (up to three tokens more, in front and behind)
  const int smem = a.cached * 4;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const auto move = wide ? evict_move_kernel<uint4> : evict_move_kernel<uint2>;
  const int move_smem = a.rows * 24 + a.rows / block * 8;
  static std::atomic<bool> set[64];                          // the kernels' attributes, once a device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return FA3_ECUDA;
  if (dev >= 64 || !set[dev].load(std::memory_order_acquire)) {
    constexpr auto kMost = cudaFuncAttributeMaxDynamicSharedMemorySize;
    if (cudaFuncSetAttribute(evict_pick_kernel, kMost, kMostKeys * 4) != cudaSuccess ||
        cudaFuncSetAttribute(evict_move_kernel<uint4>, kMost, kMostBlock * 24 + 8) != cudaSuccess ||
        cudaFuncSetAttribute(evict_move_kernel<uint2>, kMost, kMostBlock * 24 + 8) != cudaSuccess)
      return FA3_ECUDA;
    if (dev < 64) set[dev].store(true, std::memory_order_release);
  }
  const LaunchTogether together(s);
  if (launch_pdl(evict_pick_kernel, dim3((unsigned)Hkv, (unsigned)B), dim3(kPickThreads), (size_t)smem, s, a) != cudaSuccess)
    return FA3_ECUDA;
  const unsigned blocks = (unsigned)((budget + a.rows - 1) / a.rows);
  return cuda_status(launch_pdl(move, dim3(blocks, (unsigned)Hkv, (unsigned)B), dim3(kMoveThreads), (size_t)move_smem, s, a));
}
