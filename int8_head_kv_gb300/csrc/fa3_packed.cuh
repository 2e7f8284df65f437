// What the calls on packed rows over a block-scaled paged cache share: which sequence a piece of work belongs to, and
// where a block of tokens and its scales lie.
#pragma once

#include <math_constants.h>
#include <stdint.h>

#include "fa3_common.cuh"

namespace fa3 {
namespace {

constexpr int kLeastBlock = 16, kMostBlock = 4096;   // tokens that share a scale: a multiple of the one, up to the other

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The pages: token t of sequence b lies in row t % page_size of page block_table[b][t / page_size].
struct Pages {
  const int32_t* table;            // [B][max_pages]
  int max_pages, num_pages, page_size, T_max;
  int block, per_page, Hkv;        // tokens a scale, scales a page and head
  DivU32 div_ps, div_block;
};

// Checks of what every call on such a cache is given; fills *p.
inline int pages_of(const int32_t* table, int B, int Hkv, int num_pages, int page_size, int max_pages, int block, Pages* p) {
  if (!table || B <= 0 || Hkv <= 0 || num_pages <= 0 || page_size <= 0 || max_pages <= 0 || block <= 0) return FA3_EINVAL;
  if (page_size % block != 0) return FA3_EINVAL;
  if (block % kLeastBlock != 0 || block > kMostBlock || B > kMostSequences || Hkv > 65535) return FA3_ERANGE;
  // (kernels look some tokens behind a context's last in 32-bit numbers)
  if ((int64_t)max_pages * page_size > ((int64_t)1 << 31) - 65536 || (int64_t)num_pages * page_size >= ((int64_t)1 << 31))
    return FA3_ERANGE;
  *p = Pages{table, max_pages, num_pages, page_size, max_pages * page_size, block, page_size / block, Hkv,
             make_divu32((uint32_t)page_size), make_divu32((uint32_t)block)};
  return FA3_OK;
}

// A piece of work of a packed call: `index` counts the pieces of sequence b; q0 .. q0 + nq its rows, nkv its context.
struct Piece {
  int b, index, q0, nq, nkv;
};

// Pieces of `step` rows: sequence b has the numbers from q_start[b] / step + extra * b on, up to those of the next.  That is
// no fewer than ceil(n_b / step) + extra - 1, whatever q_start[b] is, and the whole call has n / step + extra * B.
inline int64_t pieces_of(int64_t n, int64_t B, int64_t step, int64_t extra) { return n / step + extra * B; }

// Finds piece x (the block together; `found` is shared).  b < 0: there is none, or the sequence's lengths are bad, or
// q_start falls somewhere (two sequences might share rows then: the call does nothing).  All threads read q_start at
// once, one load's latency for B up to the block's threads.  With `report`, bad lengths set FA3_DEVERR_LENS.
__device__ __forceinline__ Piece find_piece(const int32_t* __restrict__ q_start, const int32_t* __restrict__ kv_lens, int B, int n,
                                            int T_max, DivU32 div_step, int extra, int64_t x, bool report, int32_t* err,
                                            Piece* found) {
  if (threadIdx.x == 0) found->b = -1;
  __syncthreads();
  bool falls = false, bad = false;
  for (int b = threadIdx.x; b < B; b += blockDim.x) {
    const int q0 = q_start[b], q1 = q_start[b + 1];
    const int nkv = kv_lens[b];
    falls |= q1 < q0;
    const bool wrong = q0 < 0 || q1 > n || (q1 > q0 && (nkv < q1 - q0 || nkv > T_max));
    bad |= wrong;
    if (wrong || q1 <= q0) continue;
    const int64_t first = (int64_t)divu32((uint32_t)q0, div_step) + (int64_t)extra * b;
    const int64_t next = (int64_t)divu32((uint32_t)q1, div_step) + (int64_t)extra * (b + 1);
    if (x >= first && x < next) *found = Piece{b, (int)(x - first), q0, q1 - q0, nkv};
  }
  if (report && (falls || bad)) set_dev_err(err, FA3_DEVERR_LENS);
  falls = __syncthreads_or(falls);
  Piece p = *found;
  if (falls) p.b = -1;
  return p;
}

// RNE(code * ratio), exactly: one fused operation rounds the exact product to a whole number (|code * ratio| <= 127).  Codes
// become float32 as the low byte of 2^23 (+ 128), by byte moves and packed sums: conversion instructions go at 16 a cycle, and were
// what an eviction waited for.
__device__ __forceinline__ uint32_t rescaled(uint32_t codes4, float ratio) {
  const uint32_t u = codes4 ^ 0x80808080u;
  const unsigned long long less = f32x2_pack(-8388736.f, -8388736.f), by = f32x2_pack(ratio, ratio), one = f32x2_pack(1.f, 1.f),
                           magic = f32x2_pack(kCodeMagic, kCodeMagic);
  uint32_t q[4];
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    const unsigned long long x = f32x2_pack(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 + e)),
                                            __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7441 + e)));
    float t0, t1;
    f32x2_unpack(f32x2_fma(f32x2_fma(x, one, less), by, magic), t0, t1);
    q[e] = __float_as_uint(t0);
    q[e + 1] = __float_as_uint(t1);
  }
  return __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
}

constexpr float kLeastScale = 8.271806125530277e-25f;      // 2^-80: attention takes a smaller value scale as this

// Natural logarithm of a row's sum of exponentials: the sum of 2^(.. - m) is l.  Scores that are not finite make l NaN, or 0
// with all at -inf: NaN, as the row is.
__device__ __forceinline__ float log_sum(float m, float l) { return l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : CUDART_NAN_F; }

}  // namespace
}  // namespace fa3
