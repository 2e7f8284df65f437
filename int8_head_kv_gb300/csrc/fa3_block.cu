// A paged INT8 cache that needs no calibration: every block of tokens has, for each KV head, a scale of its own for its
// keys and one for its values.  Here: the append that writes it, and the eviction that cuts it down.
//
// Append.  For each block that gets new rows, x the values of one head's new rows in it, a = max |x| of the finite ones:
//   s = fl(a / 127); if the block has tokens already (codes c, scale s0): s = max(s, s0), c = RNE(c * fl(s0 / s))
//   code = clamp(RNE(fl(x / s)), -127, 127)       (s = 0 -> 0)
// A block's scale only grows, so a token's codes are rewritten when a later one is larger, each time off by half a step at
// most, and what the scale is does not depend on how the block's tokens were split over calls.
#include "fa3_packed.cuh"

#include <algorithm>

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
// The largest magnitude of 8 bf16 values that are finite, as its 15 bits (their order is the magnitudes').
__device__ __forceinline__ uint32_t amax8(uint4 v, uint32_t m) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t a = w[k] & 0x7fff7fffu;
    m = __vmaxu2(m, a & __vcmpltu2(a, 0x7f807f80u));
  }
  return m;
}

// Block (piece, head, k or v).
__global__ void __launch_bounds__(kAppendThreads) block_append_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ Piece found;
  __shared__ uint32_t warp_max[kAppendThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, h = blockIdx.y, kv = blockIdx.z;
  const Piece p = find_piece(a.q_start, a.kv_lens, a.B, a.n, a.pg.T_max, a.pg.div_block, 2, blockIdx.x,
                             (blockIdx.x | blockIdx.y | blockIdx.z) == 0, a.err, &found);
  if (p.b < 0) return;
  // Tokens [lo, hi) of the block are new, [blk * block, lo) were there.
  const int start = p.nkv - p.nq, blk = (int)divu32((uint32_t)start, a.pg.div_block) + p.index;
  const int base = blk * a.pg.block, lo = max(base, start), hi = min(base + a.pg.block, p.nkv);
  if (base >= p.nkv) return;
  const int pi = (int)divu32((uint32_t)base, a.pg.div_ps), page = a.pg.table[(int64_t)p.b * a.pg.max_pages + pi];
  if ((uint32_t)page >= (uint32_t)a.pg.num_pages) {
    if (tid == 0 && h == 0 && kv == 0) set_dev_err(a.err, FA3_DEVERR_PAGE);
    return;
  }
  const int at = base - pi * a.pg.page_size;                 // of the block in its page
  const int rows = hi - lo, items = rows * a.chunks;
  const uint16_t* x = a.x[kv] + (int64_t)(p.q0 + lo - start) * a.stride[kv] + (int64_t)h * a.D;
  constexpr int kHeld = 4;                                   // groups of 8 values that a thread keeps
  uint4 held[kHeld];
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int i = tid + k * kAppendThreads;
    held[k] = make_uint4(0u, 0u, 0u, 0u);
    if (i < items) {
      const int row = (int)divu32((uint32_t)i, a.div_chunks);
      held[k] = load8(x + row * a.stride[kv] + (i - row * a.chunks) * 8, a.wide);
    }
  }
#pragma unroll
  for (int k = 0; k < kHeld; ++k) m = amax8(held[k], m);
  for (int i = tid + kHeld * kAppendThreads; i < items; i += kAppendThreads) {
    const int row = (int)divu32((uint32_t)i, a.div_chunks);
    m = amax8(load8(x + row * a.stride[kv] + (i - row * a.chunks) * 8, a.wide), m);
  }
  m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
  if ((tid & 31) == 0) warp_max[tid >> 5] = m;
  float* scale = a.scale[kv] + ((int64_t)page * a.pg.per_page + (int)divu32((uint32_t)at, a.pg.div_block)) * a.pg.Hkv + h;
  const float before = lo > base ? *scale : 0.f;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kAppendThreads / 32; ++w) m = max(m, warp_max[w]);
  float s = __fdiv_rn(bf16_to_float(m), 127.f);
  int8_t* rows0 = a.cache[kv] + ((int64_t)page * a.pg.page_size + at) * a.pg.Hkv * a.D + (int64_t)h * a.D;   // token `base`
  const int64_t step = (int64_t)a.pg.Hkv * a.D;
  if (lo > base) {
    if (s > before) {
      const float ratio = __fdiv_rn(before, s);
      for (int i = tid; i < (lo - base) * a.chunks; i += kAppendThreads) {
        const int row = (int)divu32((uint32_t)i, a.div_chunks);
        uint2* c = reinterpret_cast<uint2*>(rows0 + row * step + (i - row * a.chunks) * 8);
        const uint2 w = *c;
        *c = make_uint2(rescaled(w.x, ratio), rescaled(w.y, ratio));
      }
    } else {
      s = before;
    }
  }
  if (tid == 0) *scale = s;                                  // every thread has read it: the barrier above
  const float rs = rcp_approx(s);
  const bool exact = exact_scale(s);
  int8_t* out = rows0 + (lo - base) * step;
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int i = tid + k * kAppendThreads;
    if (i < items) {
      const int row = (int)divu32((uint32_t)i, a.div_chunks);
      *reinterpret_cast<uint2*>(out + row * step + (i - row * a.chunks) * 8) = quant_group8(held[k], s, rs, exact);
    }
  }
  for (int i = tid + kHeld * kAppendThreads; i < items; i += kAppendThreads) {
    const int row = (int)divu32((uint32_t)i, a.div_chunks);
    const uint4 v = load8(x + row * a.stride[kv] + (i - row * a.chunks) * 8, a.wide);
    *reinterpret_cast<uint2*>(out + row * step + (i - row * a.chunks) * 8) = quant_group8(v, s, rs, exact);
  }
}

// ------------------------------------------------------------------ eviction
// Of each sequence and KV head the first `sinks` tokens stay, the last `recent`, and of the others those with the
// greatest weights, the earliest of equal ones, up to `budget` in all; a context that fits the budget stays whole.
constexpr int kPickThreads = 1024;
constexpr int kDigitBits = 11, kBins = 1 << kDigitBits;

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
  int B, D, new_pages, budget, sinks, recent, chunks, cached;
  DivU32 div_chunks;
};

// Order-preserving bits: NaN above all, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive prefix sums over the block's threads, and the total (1024 threads; `tmp` holds 33 values).
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* tmp, uint32_t* total) {
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
    if (lane == 31) tmp[32] = t;
  }
  __syncthreads();
  *total = tmp[32];
  return tmp[warp] + s - v;
}

// Block (head, sequence): the tokens that stay, in order, to `kept`.
__global__ void __launch_bounds__(kPickThreads) evict_pick_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ uint32_t keys[];                         // of the whole context, where they fit
  __shared__ uint32_t bins[kBins], tmp[33], found[2];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, g = blockIdx.x, b = blockIdx.y, lane = tid & 31, warp = tid >> 5;
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
  const int c0 = a.sinks, c1 = T - a.recent, want = a.budget - a.sinks - a.recent;   // want < c1 - c0
  auto load = [&](int t) -> uint32_t {
    const uint32_t pi = divu32((uint32_t)t, a.pg.div_ps);
    int page = a.pg.table[(int64_t)b * a.pg.max_pages + pi];
    if ((uint32_t)page >= (uint32_t)a.pg.num_pages) {        // outside the pool: any page of it
      set_dev_err(a.err, FA3_DEVERR_PAGE);
      page = 0;
    }
    return weight_key(a.weights[((int64_t)page * a.pg.Hkv + g) * a.pg.page_size + (t - (int)pi * a.pg.page_size)]);
  };
  const bool cached = c1 - c0 <= a.cached;
  if (cached) {
    for (int t = c0 + tid; t < c1; t += kPickThreads) keys[t - c0] = load(t);
  }
  auto key = [&](int t) { return cached ? keys[t - c0] : load(t); };
  // The want-th greatest key, digit by digit from the top: `above` keys are greater than every one with these digits.
  uint32_t prefix = 0, need = (uint32_t)want;
  int shift = 32;
  while (shift > 0 && want > 0) {
    const int bits = min(kDigitBits, shift), rest = shift - bits;
    for (int i = tid; i < kBins; i += kPickThreads) bins[i] = 0;
    __syncthreads();
    for (int t = c0 + tid; t < c1; t += kPickThreads) {
      const uint32_t k = key(t);
      if (shift == 32 || k >> shift == prefix) atomicAdd(&bins[(k >> rest) & ((1u << bits) - 1u)], 1u);
    }
    __syncthreads();
    // a thread has two bins, the greatest first
    const int hi = kBins - 1 - 2 * tid;
    const uint32_t n0 = bins[hi], n1 = bins[hi - 1];
    uint32_t total;
    const uint32_t before = block_scan(n0 + n1, tmp, &total);
    if (before < need && before + n0 + n1 >= need) {
      const bool second = before + n0 < need;
      found[0] = (uint32_t)(second ? hi - 1 : hi);
      found[1] = need - before - (second ? n0 : 0u);
    }
    __syncthreads();
    prefix = (shift == 32 ? 0u : prefix << bits) | found[0];
    need = found[1];
    shift = rest;
  }
  // Kept: greater than `prefix`, or equal to it and one of the first `need` such.  A warp has a run of tokens.
  const int count = c1 - c0, per = ((count + kPickThreads - 1) / kPickThreads) * 32;
  const int w0 = c0 + (int)min((int64_t)count, (int64_t)warp * per), w1 = c0 + (int)min((int64_t)count, (int64_t)(warp + 1) * per);
  uint32_t more = 0, same = 0;
  for (int t0 = w0; t0 < w1; t0 += 32) {
    const uint32_t k = t0 + lane < w1 ? key(t0 + lane) : 0u;
    more += __popc(__ballot_sync(0xffffffffu, t0 + lane < w1 && want > 0 && k > prefix));
    same += __popc(__ballot_sync(0xffffffffu, t0 + lane < w1 && want > 0 && k == prefix));
  }
  uint32_t total;
  const uint32_t same_before = __shfl_sync(0xffffffffu, block_scan(lane == 0 ? same : 0u, tmp, &total), 0);
  const uint32_t take = same_before >= need ? 0u : min(same, need - same_before);
  const uint32_t before = __shfl_sync(0xffffffffu, block_scan(lane == 0 ? more + take : 0u, tmp, &total), 0);
  uint32_t at = before, seen = same_before;
  for (int t0 = w0; t0 < w1; t0 += 32) {
    const bool in = t0 + lane < w1 && want > 0;
    const uint32_t k = in ? key(t0 + lane) : 0u;
    const uint32_t eq = __ballot_sync(0xffffffffu, in && k == prefix), below = (1u << lane) - 1u;
    const bool stays = in && (k > prefix || (k == prefix && seen + __popc(eq & below) < need));
    const uint32_t all = __ballot_sync(0xffffffffu, stays);
    if (stays) kept[a.sinks + at + __popc(all & below)] = t0 + lane;
    at += __popc(all);
    seen += __popc(eq);
  }
  for (int i = tid; i < a.sinks; i += kPickThreads) kept[i] = i;
  for (int i = tid; i < a.recent; i += kPickThreads) kept[a.budget - a.recent + i] = c1 + i;
}

constexpr int kMoveThreads = 128;

// Block (destination block, head, sequence): its tokens' codes, at the greatest of their scales, and weights.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ int64_t src_row[];                       // [block], then float ratio[2][block]
  float* ratio = reinterpret_cast<float*>(src_row + a.pg.block);
  __shared__ float warp_max[2][kMoveThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, g = blockIdx.y, b = blockIdx.z, bs = a.pg.block;
  const int T = a.kv_lens[b];
  if (T < 0 || T > a.pg.T_max) return;
  const int left = min(T, a.budget), base = blockIdx.x * bs, rows = min(bs, left - base);
  if (rows <= 0) return;
  const int pi = (int)divu32((uint32_t)base, a.pg.div_ps), page = a.new_table[(int64_t)b * a.new_pages + pi];
  if ((uint32_t)page >= (uint32_t)a.pg.num_pages) {
    if (tid == 0) set_dev_err(a.err, FA3_DEVERR_PAGE);
    return;
  }
  const int at = base - pi * a.pg.page_size;
  const int32_t* kept = a.kept + ((int64_t)b * a.pg.Hkv + g) * a.budget + base;
  const int64_t to = ((int64_t)page * a.pg.page_size + at) * a.pg.Hkv + g;             // in head rows
  float m[2] = {0.f, 0.f};
  for (int i = tid; i < rows; i += kMoveThreads) {
    const int t = kept[i];
    const uint32_t sp = divu32((uint32_t)t, a.pg.div_ps);
    int from = a.pg.table[(int64_t)b * a.pg.max_pages + sp];
    if ((uint32_t)from >= (uint32_t)a.pg.num_pages) {
      set_dev_err(a.err, FA3_DEVERR_PAGE);
      from = 0;
    }
    const int in = t - (int)sp * a.pg.page_size;
    src_row[i] = ((int64_t)from * a.pg.page_size + in) * a.pg.Hkv + g;
    a.weights[((int64_t)page * a.pg.Hkv + g) * a.pg.page_size + at + i] =
        a.weights[((int64_t)from * a.pg.Hkv + g) * a.pg.page_size + in];
    const int64_t sc = ((int64_t)from * a.pg.per_page + (int)divu32((uint32_t)in, a.pg.div_block)) * a.pg.Hkv + g;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const float s = a.scale[kv][sc];
      ratio[kv * bs + i] = s;
      m[kv] = fmaxf(m[kv], s);
    }
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
    for (int o = 16; o; o >>= 1) m[kv] = fmaxf(m[kv], __shfl_xor_sync(0xffffffffu, m[kv], o));
    if ((tid & 31) == 0) warp_max[kv][tid >> 5] = m[kv];
  }
  __syncthreads();
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
    for (int w = 0; w < kMoveThreads / 32; ++w) m[kv] = fmaxf(m[kv], warp_max[kv][w]);
    if (tid == 0)
      a.scale[kv][((int64_t)page * a.pg.per_page + (int)divu32((uint32_t)at, a.pg.div_block)) * a.pg.Hkv + g] = m[kv];
    for (int i = tid; i < rows; i += kMoveThreads) {
      const float s = ratio[kv * bs + i];
      ratio[kv * bs + i] = s == m[kv] ? 1.f : __fdiv_rn(s, m[kv]);   // 0 / 0 with it
    }
  }
  __syncthreads();
  const int items = rows * a.chunks;
  for (int j = tid; j < 2 * items; j += kMoveThreads) {
    const int kv = j >= items, i = j - kv * items;
    const int row = (int)divu32((uint32_t)i, a.div_chunks), c = (i - row * a.chunks) * 8;
    uint2 w = *reinterpret_cast<const uint2*>(a.cache[kv] + src_row[row] * a.D + c);
    const float r = ratio[kv * bs + row];
    if (r != 1.f) w = make_uint2(rescaled(w.x, r), rescaled(w.y, r));
    *reinterpret_cast<uint2*>(a.cache[kv] + (to + (int64_t)row * a.pg.Hkv) * a.D + c) = w;
  }
}

inline bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

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
  return cuda_status(launch_pdl(block_append_kernel, dim3((unsigned)pieces, (unsigned)Hkv, 2), dim3(kAppendThreads), 0,
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
  if (D % 8 != 0 || D > 256 || B > 65535) return FA3_ERANGE;
  if (!aligned8(k_cache) || !aligned8(v_cache) || !aligned4(k_scale) || !aligned4(v_scale) || !aligned4(weights))
    return FA3_ERANGE;
  st = check_device(nullptr);
  if (st != FA3_OK) return st;
  a.cache[0] = k_cache; a.cache[1] = v_cache; a.scale[0] = k_scale; a.scale[1] = v_scale; a.weights = weights;
  a.kv_lens = kv_lens; a.new_table = new_table; a.kept = kept; a.new_lens = new_lens; a.err = dev_err;
  a.B = B; a.D = D; a.new_pages = new_pages; a.budget = budget; a.sinks = sinks; a.recent = recent; a.chunks = D / 8;
  a.div_chunks = make_divu32((uint32_t)a.chunks);
  a.cached = std::min(a.pg.T_max, 48 * 1024);
  const int smem = a.cached * 4;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaFuncSetAttribute(evict_pick_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 48 * 1024 * 4) != cudaSuccess ||
      cudaFuncSetAttribute(evict_move_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 4096 * 16) != cudaSuccess)
    return FA3_ECUDA;
  const LaunchTogether together(s);
  if (launch_pdl(evict_pick_kernel, dim3((unsigned)Hkv, (unsigned)B), dim3(kPickThreads), (size_t)smem, s, a) != cudaSuccess)
    return FA3_ECUDA;
  const unsigned blocks = (unsigned)((budget + block - 1) / block);
  return cuda_status(launch_pdl(evict_move_kernel, dim3(blocks, (unsigned)Hkv, (unsigned)B), dim3(kMoveThreads),
                                (size_t)block * 16, s, a));
}
