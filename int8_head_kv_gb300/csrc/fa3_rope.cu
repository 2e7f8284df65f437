// The input side of attention: per-head RMS norm and position rotation of q and k,
// to floating point (what calibration looks at) or to INT8 codes on the way into the
// paged cache.
//
// For a head row x of D values at position p:
//   a = x * (mean(x^2) + eps)^-1/2 * w                      (no weight: a = x)
//   (y1, y2) = (a1 c - a2 s, a2 c + a1 s)                   c, s = cos_sin[p][i], cos_sin[p][rot/2 + i]
// over the pairs i of the first rot values, (i, i + rot/2) or (2i, 2i + 1); values
// beyond rot pass.  msModelSlim FA3量化 (原理 / 算法流程) calibrates and quantizes q
// and k as attention sees them, that is after this step.
//
// All of it is one read of x and one write of y (3 to 6 bytes a value), so a lane
// holds both members of its pairs: lane i of a head row owns values 4i .. 4i+3 and
// rot/2 + 4i .. rot/2 + 4i+3 (or 8i .. 8i+7 for neighbouring pairs and for values that
// pass), which needs no exchange between lanes, reads each table value once and lets
// the floating-point call work in place.  A row takes 8, 16 or 32 lanes (D up to 256),
// a warp 4, 2 or 1 rows at a time.  Numbers are float32 throughout and rounded once, to
// the output's type or to a code.
#include "fa3_common.cuh"

#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

namespace fa3 {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeWarps = kRopeThreads / 32;

// One tensor of head rows: row (b, s, h) starts at x + b * sb + s * ss + h * sh.
struct HeadRows {
  const uint16_t* x;
  const uint16_t* weight;   // [D] or nullptr
  int64_t sb, ss, sh;
};

struct HeadOut {
  void* y;
  int64_t sb, ss, sh;
};

struct RotArgs {
  const float* cos_sin;     // [table_len][rot], or nullptr: no rotation
  int table_len, rot, interleaved, D;
  float eps, inv_D, inv_D_lo;                 // inv_D + inv_D_lo = 1 / D
};

// A lane's eight values of a row: two groups of four at o1 and o2.
struct Lane8 {
  int o1, o2;
  bool in, rotated;
};
__device__ __forceinline__ Lane8 lane_place(int i, const RotArgs& r) {
  Lane8 p;
  p.in = 8 * i < r.D;
  p.rotated = r.cos_sin != nullptr && 8 * i < r.rot;
  const bool halves = p.rotated && !r.interleaved;
  p.o1 = halves ? 4 * i : 8 * i;
  p.o2 = halves ? r.rot / 2 + 4 * i : 8 * i + 4;
  return p;
}

__device__ __forceinline__ void bf16x4(uint2 v, float* f) {
  f[0] = __uint_as_float(v.x << 16);
  f[1] = __uint_as_float(v.x & 0xffff0000u);
  f[2] = __uint_as_float(v.y << 16);
  f[3] = __uint_as_float(v.y & 0xffff0000u);
}
__device__ __forceinline__ uint2 load4(const uint16_t* p) { return *reinterpret_cast<const uint2*>(p); }

// The pair e of a lane's eight values is (f[first(e)], f[second(e)]).
template <bool INTER>
__device__ __forceinline__ constexpr int first(int e) { return INTER ? 2 * e : e; }
template <bool INTER>
__device__ __forceinline__ constexpr int second(int e) { return INTER ? 2 * e + 1 : 4 + e; }

using f2 = unsigned long long;          // two floats for the packed instructions
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float rsqrt_approx(float x) {          // relative 2^-22.9
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {  // a NaN is dropped
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Two 16-bit codes clamped to [-127, 127].
__device__ __forceinline__ uint32_t clamp_code2(uint32_t v) {
  uint32_t r;
  asm("{\n.reg .b32 x;\nmax.s16x2 x, %1, %2;\nmin.s16x2 %0, x, %3;\n}" : "=r"(r) : "r"(v), "r"(0xff81ff81u), "r"(0x007f007fu));
  return r;
}

// Sum over the LANES lanes of a row.
template <int LANES, typename T>
__device__ __forceinline__ T row_sum(T v) {
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A lane's values of a row as packed pair members: a[j] = (a_2j, a_2j+1), b likewise.
struct Pairs {
  f2 a[2], b[2];
};
template <bool INTER>
__device__ __forceinline__ Pairs unpack_pairs(uint2 lo, uint2 hi) {
  float f[8];
  bf16x4(lo, f);
  bf16x4(hi, f + 4);
  Pairs p;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    p.a[j] = f32x2_pack(f[first<INTER>(2 * j)], f[first<INTER>(2 * j + 1)]);
    p.b[j] = f32x2_pack(f[second<INTER>(2 * j)], f[second<INTER>(2 * j + 1)]);
  }
  return p;
}

// The row's sum of squares: squares of bf16 values are exact in float32, the sum is eight
// to ten roundings deep.
template <int LANES>
__device__ __forceinline__ float row_squares(const Pairs& p) {
  f2 acc = mul2(p.a[0], p.a[0]);
  acc = f32x2_fma(p.a[1], p.a[1], acc);
  acc = f32x2_fma(p.b[0], p.b[0], acc);
  acc = f32x2_fma(p.b[1], p.b[1], acc);
  float lo, hi;
  f32x2_unpack(acc, lo, hi);
  return row_sum<LANES>(lo + hi);
}

// What a token and a weight multiply a lane's pairs by: y_a = a * ac - b * bs,
// y_b = b * bc + a * as, times the row's 1 / rms.  The products of weight and angle are
// taken once for all heads of the task (one rounding).
struct Turn {
  f2 ac[2], nbs[2], bc[2], as[2];
};
template <bool INTER>
__device__ __forceinline__ Turn make_turn(const Lane8& p, const RotArgs& r, int pos, const uint16_t* weight, int i) {
  float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
  float4 c4 = make_float4(1.f, 1.f, 1.f, 1.f), s4 = make_float4(0.f, 0.f, 0.f, 0.f);
  if (weight && p.in) {
    bf16x4(load4(weight + p.o1), w);
    bf16x4(load4(weight + p.o2), w + 4);
  }
  if (p.rotated) {
    const float* row = r.cos_sin + (int64_t)pos * r.rot + 4 * i;
    c4 = *reinterpret_cast<const float4*>(row);
    s4 = *reinterpret_cast<const float4*>(row + r.rot / 2);
  }
  const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
  Turn t;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int e = 2 * j;
    const float wa0 = w[first<INTER>(e)], wa1 = w[first<INTER>(e + 1)];
    const float wb0 = w[second<INTER>(e)], wb1 = w[second<INTER>(e + 1)];
    t.ac[j] = f32x2_pack(wa0 * c[e], wa1 * c[e + 1]);
    t.as[j] = f32x2_pack(wa0 * s[e], wa1 * s[e + 1]);
    t.bc[j] = f32x2_pack(wb0 * c[e], wb1 * c[e + 1]);
    t.nbs[j] = f32x2_pack(-wb0 * s[e], -wb1 * s[e + 1]);
  }
  return t;
}

// ------------------------------------------------------------------- norm_rope
struct NormRopeArgs {
  HeadRows q, k;
  HeadOut qo, ko;
  RotArgs r;
  const int32_t* pos;       // [B * S]
  int S, Hq, Hkv;
  uint32_t tokens, chunks, q_chunks, per_chunk;   // a warp's task: per_chunk heads of a token
  DivU32 div_chunks, div_S;
  int32_t* err;
};

template <typename OUT>
__device__ __forceinline__ void store4(OUT* dst, const float* f);
template <>
__device__ __forceinline__ void store4<float>(float* dst, const float* f) {
  *reinterpret_cast<float4*>(dst) = make_float4(f[0], f[1], f[2], f[3]);
}
template <>
__device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16* dst, const float* f) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(f[0], f[1]), hi = __floats2bfloat162_rn(f[2], f[3]);
  *reinterpret_cast<uint2*>(dst) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// Tasks of a token: chunks of per_chunk heads that lie within q or within k, so that
// pointers, strides and weights are the warp's.  Two passes (32 / LANES rows each) are
// loaded while the two before them are worked on.
//
// Bounded by HBM where there is enough of it: 8192 tokens of 64 + 8 heads of 128 (302 MB
// in and out) take 53 us, 5.8 TB/s of the 6.7 that a copy reaches.  Packed arithmetic on
// pairs of values and 64 registers (8 blocks an SM) brought that from 68; up to some
// hundred tokens it is the launch, 2 to 5 us.
template <typename OUT, int LANES, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 8) norm_rope_kernel(const NormRopeArgs a) {
  constexpr int rows = 32 / LANES;
  const int lane = threadIdx.x & 31;
  const int i = lane % LANES, sub = lane / LANES;
  const Lane8 p = lane_place(i, a.r);
  const uint32_t nt = a.tokens * a.chunks;
  pdl_wait();
  pdl_launch_dependents();
  for (uint32_t t = blockIdx.x * kRopeWarps + (threadIdx.x >> 5); t < nt; t += gridDim.x * kRopeWarps) {
    const uint32_t tok = divu32(t, a.div_chunks), chunk = t - tok * a.chunks;
    const uint32_t b = divu32(tok, a.div_S), s = tok - b * (uint32_t)a.S;
    const bool is_q = chunk < a.q_chunks;
    const HeadRows T = is_q ? a.q : a.k;
    const int h_first = (int)((is_q ? chunk : chunk - a.q_chunks) * a.per_chunk);
    const int n = min((int)a.per_chunk, (is_q ? a.Hq : a.Hkv) - h_first) - sub;   // rows from this half on
    const uint16_t* x = T.x + b * T.sb + s * T.ss + (h_first + sub) * T.sh;
    const int64_t step = rows * T.sh;
    uint2 cur[2][2], nxt[2][2];
    auto fetch = [&](uint2 (&d)[2][2], int h, const uint16_t* at) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        d[u][0] = d[u][1] = make_uint2(0u, 0u);
        if (h + u * rows < n && p.in) {
          d[u][0] = load4(at + u * step + p.o1);
          d[u][1] = load4(at + u * step + p.o2);
        }
      }
    };
    fetch(cur, 0, x);
    int pos = 0;
    if (a.r.cos_sin) {
      pos = a.pos[tok];
      if (pos < 0 || pos >= a.r.table_len) {
        if (lane == 0) set_dev_err(a.err, FA3_DEVERR_POS);
        continue;
      }
    }
    const Turn w = make_turn<INTER>(p, a.r, pos, T.weight, i);
    const HeadOut O = is_q ? a.qo : a.ko;
    OUT* y = (OUT*)O.y + b * O.sb + s * O.ss + (h_first + sub) * O.sh;
    for (int h = 0; h < n + sub; h += 2 * rows) {                      // n + sub: the same for the whole warp
      x += 2 * step;
      fetch(nxt, h + 2 * rows, x);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (u && h + rows >= n + sub) break;
        const Pairs v = unpack_pairs<INTER>(cur[u][0], cur[u][1]);
        f2 r2 = 0;
        if (T.weight) {
          const float rstd = rsqrtf(row_squares<LANES>(v) * a.r.inv_D + a.r.eps);
          r2 = f32x2_pack(rstd, rstd);
        }
        float f[8];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          // values that pass stay apart from their neighbours: 0 * inf is no 0
          f2 ya = p.rotated ? f32x2_fma(v.a[j], w.ac[j], mul2(v.b[j], w.nbs[j])) : mul2(v.a[j], w.ac[j]);
          f2 yb = p.rotated ? f32x2_fma(v.b[j], w.bc[j], mul2(v.a[j], w.as[j])) : mul2(v.b[j], w.bc[j]);
          if (T.weight) {
            ya = mul2(ya, r2);
            yb = mul2(yb, r2);
          }
          f32x2_unpack(ya, f[first<INTER>(2 * j)], f[first<INTER>(2 * j + 1)]);
          f32x2_unpack(yb, f[second<INTER>(2 * j)], f[second<INTER>(2 * j + 1)]);
        }
        if (h + u * rows < n && p.in) {
          store4(y + u * rows * O.sh + p.o1, f);
          store4(y + u * rows * O.sh + p.o2, f + 4);
        }
      }
      y += 2 * rows * O.sh;
#pragma unroll
      for (int u = 0; u < 2; ++u) cur[u][0] = nxt[u][0], cur[u][1] = nxt[u][1];
    }
  }
}

// ------------------------------------------------------------- append into pages
struct RopeAppendArgs {
  HeadRows q, k, v;          // packed rows: ss = row stride, sh = head stride; sb unused
  const float *q_scale, *k_scale, *v_scale;
  int8_t *q_out, *k_cache, *v_cache;
  RotArgs r;
  const int32_t *block_table, *q_start, *kv_lens;
  int n, B, Hq, Hkv, num_pages, page_size, max_pages, T_max;
  uint32_t chunks, q_chunks, k_chunks, per_chunk;   // a warp's task: per_chunk heads of q, k or v of a token
  DivU32 div_chunks, div_ps;
  int32_t* err;
};

// Sequence of packed row `row`: the last b with q_start[b] <= row, found by the warp
// 32 entries at a time (one dependent load per factor of 32 in B).
__device__ __forceinline__ int find_sequence(const int32_t* q_start, int B, int row, int lane) {
  int lo = 0, len = B + 1;
  while (len > 1) {
    const int step = (len + 31) / 32;
    const int at = lo + lane * step;
    const bool le = lane * step < len && q_start[at] <= row;
    const int c = __popc(__ballot_sync(0xffffffffu, le));
    if (c == 0) return -1;
    const int off = (c - 1) * step;
    lo += off;
    len = min(step, len - off);
  }
  return lo;
}

// Codes in float32, and where that cannot decide, in float64.
//
// Fast path: with f = 1 / (rms s), t = y f by one fma onto 1.5 * 2^23, which rounds half
// to even in the low mantissa bits; d is what the rounding left.  In units of u = 2^-24
// and relative to m = |a ac| + |b bs|, t is off by: product and fma 2, reciprocal of s
// 1.65, and with the norm ten roundings of the sum, mean and eps halved by the root 6,
// rsqrtf 4, f 1, weight times angle 1; together 3.7 (15.7).  A t whose half step is
// nearer than 8 (20) u (|a| + |b|) max(|ac|, |bs|, |bc|, |as|) is decided again: one or
// two values in 10^4 of normal data.
//
// Again, by the whole warp because the row's sum of squares is needed: everything as unevaluated pairs of
// float32 (Dekker's products by fma, Knuth's sums; float64 runs at a small fraction of the float32 rate here),
// 1 / sqrt by one correction of the hardware's, and the sign of y - h s for the half step h next to t.  The pairs are off
// by up to 2^-44.7 of the terms |a c| + |b s| (the worst of 60,000 rows of three head sizes), so where y - h s is within
// 2^-40 of them the pairs cannot tell a value on the half step from one beside it.  There, and for what float32 cannot
// carry (a scale outside [2^-100, 2^100], a sum of squares outside [2^-100, 2^100], infinities and NaN), float64 decides, in
// the order of the definition: x / rms, times the weight, the two products, their sum, the quotient.
constexpr float kTieNorm = 20.f / 16777216.f, kTiePlain = 8.f / 16777216.f;

__device__ __forceinline__ int code64(double y, double s) {
  if (s == 0.0) return 0;
  return __double2int_rn(fmin(fmax(y / s, -127.0), 127.0));
}

struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair product(float a, float b) {          // exact
  const float h = __fmul_rn(a, b);
  return Pair{h, fmaf(a, b, -h)};
}
__device__ __forceinline__ Pair sum(float a, float b) {              // exact
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return Pair{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}

// Value e of a lane's eight (x: the values, w: the weights or ones, c and sn the angles of its four pairs, r:
// 1 / rms), decided as described above; near: the pairs cannot tell.
constexpr float kPairBand = 9.094947017729282e-13f;                  // 2^-40
template <bool INTER>
__device__ __forceinline__ int decide(const float (&x)[8], const float (&w)[8], const float (&c)[4],
                                      const float (&sn)[4], int e, Pair r, bool norm, bool turn, float s, float rs, bool& near) {
  const int pe = INTER ? e / 2 : e % 4;
  const bool sec = INTER ? (e & 1) != 0 : e >= 4;
  const int o = sec ? first<INTER>(pe) : second<INTER>(pe);
  Pair y = {x[e] * w[e], 0.f};                                       // bf16 x bf16: exact
  float terms = fabsf(y.hi);
  if (turn) {
    const float other = x[o] * w[o];
    const Pair p = product(y.hi, c[pe]), q = product(other, sec ? sn[pe] : -sn[pe]);
    const Pair z = sum(p.hi, q.hi);
    terms = fabsf(p.hi) + fabsf(q.hi);
    y = sum(z.hi, __fadd_rn(z.lo, __fadd_rn(p.lo, q.lo)));
  }
  if (norm) {
    const Pair p = product(y.hi, r.hi);
    terms *= r.hi;
    y = Pair{p.hi, __fadd_rn(p.lo, fmaf(y.hi, r.lo, __fmul_rn(y.lo, r.hi)))};
  }
  const float lo = floorf(y.hi * rs), h = lo + 0.5f;                 // the half step next to y / s
  const Pair g = product(h, s);
  const float over = __fadd_rn(__fsub_rn(y.hi, g.hi), __fsub_rn(y.lo, g.lo));
  near = (norm || turn) && fabsf(over) <= terms * kPairBand;          // x alone is exact
  const int code = (int)(over > 0.0f ? lo + 1.f : over < 0.0f ? lo : rintf(h));
  return max(-127, min(127, code));
}
// The same in float64, one rounding an operation: value x with weight w and angle c, its partner xo, wo and, with the
// sign of their product, so.
__device__ __noinline__ int decide64(float x, float w, float c, float xo, float wo, float so, double rms, bool norm,
                                     bool turn, float s) {
  double y = norm ? __dmul_rn((double)x / rms, (double)w) : (double)x;
  if (turn) {
    const double other = norm ? __dmul_rn((double)xo / rms, (double)wo) : (double)xo;
    y = __dadd_rn(__dmul_rn(y, (double)c), __dmul_rn(other, (double)so));
  }
  return code64(y, (double)s);
}

// The lane's codes with those of `again` (a bit each) decided again; every lane of the warp calls it.  Out of
// line: it is rare, and its registers are not the loop's.
template <int LANES, bool INTER>
__device__ __noinline__ uint2 decide_row(const RotArgs& r, const uint16_t* weight, uint2 x1, uint2 x2, float s,
                                         uint2 codes, uint32_t again, bool sound, bool is_v, int pos, int i) {
  const Lane8 p = lane_place(i, r);
  float x[8], w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}, c[4] = {}, sn[4] = {};
  bf16x4(x1, x);
  bf16x4(x2, x + 4);
  Pair rms = {1.f, 0.f};                                             // 1 / rms
  if (weight) {
    Pair ss = {0.f, 0.f};                                            // the squares are exact
    auto add = [&](float v) {
      const Pair z = sum(ss.hi, v);
      ss = Pair{z.hi, __fadd_rn(ss.lo, z.lo)};
    };
#pragma unroll
    for (int e = 0; e < 8; ++e) add(x[e] * x[e]);
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) {
      const float h2 = __shfl_xor_sync(0xffffffffu, ss.hi, o), l2 = __shfl_xor_sync(0xffffffffu, ss.lo, o);
      add(h2);
      ss.lo = __fadd_rn(ss.lo, l2);
    }
    // m = ss / D + eps, then r0 + r0 (e / 2 + 3 e^2 / 8) with e = 1 - m r0^2
    const Pair d = product(ss.hi, r.inv_D);
    Pair m = sum(d.hi, r.eps);
    m = sum(m.hi, __fadd_rn(m.lo, __fadd_rn(d.lo, fmaf(ss.hi, r.inv_D_lo, __fmul_rn(ss.lo, r.inv_D)))));
    const float r0 = rsqrt_approx(m.hi);
    const Pair t = product(r0, r0), u = product(m.hi, t.hi);
    const float e = __fsub_rn(__fsub_rn(__fsub_rn(1.f, u.hi), u.lo), fmaf(m.hi, t.lo, __fmul_rn(m.lo, t.hi)));
    rms = Pair{r0, r0 * (e * fmaf(0.375f, e, 0.5f))};
  }
  if (weight && again) {
    bf16x4(load4(weight + p.o1), w);
    bf16x4(load4(weight + p.o2), w + 4);
  }
  if (p.rotated && again) {
    const float* tr = r.cos_sin + (int64_t)pos * r.rot + 4 * i;
    const float4 c4 = *reinterpret_cast<const float4*>(tr), s4 = *reinterpret_cast<const float4*>(tr + r.rot / 2);
    c[0] = c4.x, c[1] = c4.y, c[2] = c4.z, c[3] = c4.w;
    sn[0] = s4.x, sn[1] = s4.y, sn[2] = s4.z, sn[3] = s4.w;
  }
  const float rs = rcp_approx(s);
  uint32_t q[2] = {codes.x, codes.y};
  auto set = [&](int e, int code) {
    q[e / 4] = (q[e / 4] & ~(0xffu << (8 * (e % 4)))) | (((uint32_t)code & 0xffu) << (8 * (e % 4)));
  };
  uint32_t left = is_v || sound ? 0u : again;                        // for float64
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if ((again & ~left) >> e & 1u) {
      bool near = false;
      set(e, is_v ? quant_code(x[e], s) : decide<INTER>(x, w, c, sn, e, rms, weight != nullptr, p.rotated, s, rs, near));
      if (near) left |= 1u << e;
    }
  if (__any_sync(0xffffffffu, left != 0u)) {
    double root = 1.0;
    if (weight) {
      double sd = 0.0;
#pragma unroll
      for (int k = 0; k < 8; ++k) sd = fma((double)x[k], (double)x[k], sd);
      root = sqrt(row_sum<LANES>(sd) / (double)r.D + (double)r.eps);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (left >> e & 1u) {
        const int pe = INTER ? e / 2 : e % 4;
        const bool sec = INTER ? (e & 1) != 0 : e >= 4;
        const int o = sec ? first<INTER>(pe) : second<INTER>(pe);
        set(e, decide64(x[e], w[e], c[pe], x[o], w[o], sec ? sn[pe] : -sn[pe], root, weight != nullptr, p.rotated, s));
      }
  }
  return make_uint2(q[0], q[1]);
}

// Where a packed row goes: its position and the pool row.
struct Place {
  int pos;
  int64_t pool_row;          // -1: the page lies outside the pool
  bool ok;
};
__device__ __forceinline__ Place place_row(const RopeAppendArgs& a, int row, int lane) {
  Place pl = {0, -1, false};
  const int b = find_sequence(a.q_start, a.B, row, lane);
  if (b < 0 || b >= a.B) return pl;                        // behind the last sequence
  const int q0 = a.q_start[b], q1 = a.q_start[b + 1], kv = a.kv_lens[b];
  // In a q_start that falls and rises the search may end at a sequence that begins behind the row: its position would
  // be below 0, and the reads of the table and of the pages outside both.
  if (q0 < 0 || q0 > row || q1 <= row || q1 > a.n || kv < q1 - q0 || kv > a.T_max) return pl;   // check_lengths reports it
  pl.pos = kv - (q1 - row);
  if (a.r.cos_sin && pl.pos >= a.r.table_len) {
    if (lane == 0) set_dev_err(a.err, FA3_DEVERR_POS);
    return pl;
  }
  pl.ok = true;
  const uint32_t pi = divu32((uint32_t)pl.pos, a.div_ps);
  const int pg = a.block_table[(int64_t)b * a.max_pages + pi];
  if (pg >= 0 && pg < a.num_pages)
    pl.pool_row = (int64_t)pg * a.page_size + (pl.pos - (int)pi * a.page_size);
  else if (lane == 0)
    set_dev_err(a.err, FA3_DEVERR_PAGE);
  return pl;
}

// Reports bad lengths of any sequence.  The rows cannot: a sequence that ends before it begins has none, and in a
// q_start that falls a row may find another sequence that holds it.  A block of its own, so that no row waits for it.
__device__ __forceinline__ void check_lengths(const RopeAppendArgs& a) {
  for (int b = threadIdx.x; b < a.B; b += kRopeThreads) {
    const int q0 = a.q_start[b], q1 = a.q_start[b + 1], kv = a.kv_lens[b];
    if (q0 < 0 || q1 < q0 || q1 > a.n || (q1 > q0 && (kv < q1 - q0 || kv > a.T_max))) set_dev_err(a.err, FA3_DEVERR_LENS);
  }
}

// The same walk over chunks of heads of q, k or v, of which each row ends as codes: q's
// in q_out, k's and v's in the token's place in the pages.
//
// 3080 tokens of 64 + 8 + 8 heads of 128 (95 MB) take 37 us, 2.6 TB/s.  Bounded by latency at
// low occupancy: about 190 instructions for the 256 values of a warp's pass (a code and the
// test of its neighbourhood take six a value) fill 59 % of the issue slots, and 16 warps an
// SM at 124 registers do not cover the rest (instructions wait for results before them,
// shared-memory exchanges and loads, in this order).  With 96 registers (5 blocks an SM) or 80
// (6) the rows spill, 45 and 51 us.  A token's look-ups (sequence, lengths, page) are loads
// that wait for one another, so the first rows are asked for before them: 16 one-token
// sequences take 4 us.
template <int LANES, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const __grid_constant__ RopeAppendArgs a) {
  constexpr int rows = 32 / LANES;
  const int lane = threadIdx.x & 31;
  const int i = lane % LANES, sub = lane / LANES;
  const Lane8 p = lane_place(i, a.r);
  const uint32_t nt = (uint32_t)a.n * a.chunks;
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x == 0) {
    check_lengths(a);
    return;
  }
  for (uint32_t t = (blockIdx.x - 1) * kRopeWarps + (threadIdx.x >> 5); t < nt; t += (gridDim.x - 1) * kRopeWarps) {
    const int row = (int)divu32(t, a.div_chunks);
    uint32_t chunk = t - (uint32_t)row * a.chunks;
    const bool is_q = chunk < a.q_chunks;
    if (!is_q) chunk -= a.q_chunks;
    const bool is_v = !is_q && chunk >= a.k_chunks;
    if (is_v) chunk -= a.k_chunks;
    const HeadRows T = is_q ? a.q : is_v ? a.v : a.k;
    const float* scale = is_q ? a.q_scale : is_v ? a.v_scale : a.k_scale;
    const int H = is_q ? a.Hq : a.Hkv;
    const int h_first = (int)(chunk * a.per_chunk) + sub;
    const int n_all = min((int)a.per_chunk, H - (h_first - sub));      // the task's rows
    const int n_in = p.in ? n_all - sub : 0;                           // as this lane counts them
    const int64_t step = (int64_t)rows * T.sh;
    const uint16_t* x1 = T.x + row * T.ss + (int64_t)h_first * T.sh + p.o1;
    const int gap = p.o2 - p.o1;
    const float* sp = scale + h_first;
    // Two passes (rows rows each) are loaded while the two before them are worked on; the
    // first ones' loads go out before the look-ups of the token's place.
    uint2 cur[2][2], nxt[2][2];
    float s_cur[2], s_nxt[2];
    auto fetch = [&](uint2 (&d)[2][2], float (&sc)[2], int h) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        d[u][0] = d[u][1] = make_uint2(0u, 0u);
        sc[u] = 1.f;
        if (h + u * rows < n_in) {
          d[u][0] = load4(x1 + u * step);
          d[u][1] = load4(x1 + u * step + gap);
          sc[u] = sp[u * rows];
        }
      }
      x1 += 2 * step;
      sp += 2 * rows;
    };
    fetch(cur, s_cur, 0);
    const Place pl = place_row(a, row, lane);
    if (!pl.ok || (!is_q && pl.pool_row < 0)) continue;
    int8_t* y1 = (is_q ? a.q_out + (int64_t)row * a.Hq * a.r.D
                       : (is_v ? a.v_cache : a.k_cache) + pl.pool_row * a.Hkv * a.r.D) + (int64_t)h_first * a.r.D + p.o1;
    const int y_step = rows * a.r.D;
    const bool norm = T.weight != nullptr;
    Lane8 pt = p;
    pt.rotated = p.rotated && !is_v;                        // v: multiplied by 1 and 0
    const Turn w = make_turn<INTER>(pt, a.r, pl.pos, T.weight, i);
    float band = 0.f;                                       // the largest factor (NaN if one is), times the tie band
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float g0, g1, g2, g3;
      f32x2_unpack(w.ac[j], g0, g1);
      f32x2_unpack(w.nbs[j], g2, g3);
      band = max3_nan(max3_nan(band, fabsf(g0), fabsf(g1)), fabsf(g2), fabsf(g3));
      f32x2_unpack(w.bc[j], g0, g1);
      f32x2_unpack(w.as[j], g2, g3);
      band = max3_nan(max3_nan(band, fabsf(g0), fabsf(g1)), fabsf(g2), fabsf(g3));
    }
    band *= norm ? kTieNorm : kTiePlain;
    const float lim_min = 0.5f - 32768.f * (norm ? kTieNorm : kTiePlain);
    const f2 magic = f32x2_pack(kCodeMagic, kCodeMagic);
    for (int h = 0; h < n_all; h += 2 * rows) {
      fetch(nxt, s_nxt, h + 2 * rows);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (u && h + rows >= n_all) break;
        const float s = s_cur[u];
        const Pairs v = unpack_pairs<INTER>(cur[u][0], cur[u][1]);
        float f = rcp_approx(s);
        bool sound = exact_scale(s);
        if (norm) {
          const float ss = row_squares<LANES>(v);
          sound = sound & (ss >= 7.8886e-31f) & (ss <= 1.2676e30f);
          f *= rsqrt_approx(fmaf(ss, a.r.inv_D, a.r.eps));
        }
        const f2 ff = f32x2_pack(f, f);
        uint32_t t[8];
        float d[8], m = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const f2 ya = f32x2_fma(v.a[j], w.ac[j], mul2(v.b[j], w.nbs[j]));
          const f2 yb = f32x2_fma(v.b[j], w.bc[j], mul2(v.a[j], w.as[j]));
          const f2 ta = f32x2_fma(ya, ff, magic), tb = f32x2_fma(yb, ff, magic);          // magic + RNE(t)
          const f2 da = f32x2_fma(ya, ff, f32x2_sub(magic, ta)), db = f32x2_fma(yb, ff, f32x2_sub(magic, tb));
          const int at[4] = {first<INTER>(2 * j), first<INTER>(2 * j + 1), second<INTER>(2 * j), second<INTER>(2 * j + 1)};
          float t0, t1, t2, t3, a0, a1, b0, b1;
          f32x2_unpack(ta, t0, t1);
          f32x2_unpack(tb, t2, t3);
          t[at[0]] = __float_as_uint(t0), t[at[1]] = __float_as_uint(t1);
          t[at[2]] = __float_as_uint(t2), t[at[3]] = __float_as_uint(t3);
          f32x2_unpack(da, d[at[0]], d[at[1]]);
          f32x2_unpack(db, d[at[2]], d[at[3]]);
          f32x2_unpack(v.a[j], a0, a1);
          f32x2_unpack(v.b[j], b0, b1);
          m = max3_nan(m, fabsf(a0) + fabsf(b0), fabsf(a1) + fabsf(b1));
        }
        // codes: the low 16 bits of t, clamped in pairs, then the low bytes
        uint2 code;
        code.x = __byte_perm(clamp_code2(__byte_perm(t[0], t[1], 0x5410)), clamp_code2(__byte_perm(t[2], t[3], 0x5410)), 0x6420);
        code.y = __byte_perm(clamp_code2(__byte_perm(t[4], t[5], 0x5410)), clamp_code2(__byte_perm(t[6], t[7], 0x5410)), 0x6420);
        const float lim = fmaf(-m * band, f, 0.5f);
        const float dm = max3(max3(fabsf(d[0]), fabsf(d[1]), fabsf(d[2])), max3(fabsf(d[3]), fabsf(d[4]), fabsf(d[5])),
                              fmaxf(fabsf(d[6]), fabsf(d[7])));
        sound = sound & (lim >= lim_min);                     // |t| below 2^15 and no infinity or NaN
        const bool sure = sound & (dm <= lim);
        const bool live = h + u * rows < n_in;
        if (__any_sync(0xffffffffu, live & !sure)) {
          uint32_t again = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (live & (!sound | !(fabsf(d[e]) <= lim))) again |= 1u << e;
          code = decide_row<LANES, INTER>(a.r, T.weight, cur[u][0], cur[u][1], s, code, again, sound, is_v, pl.pos, i);
        }
        if (live) {
          *reinterpret_cast<uint32_t*>(y1 + u * y_step) = code.x;
          *reinterpret_cast<uint32_t*>(y1 + u * y_step + gap) = code.y;
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) cur[u][0] = nxt[u][0], cur[u][1] = nxt[u][1], s_cur[u] = s_nxt[u];
      y1 += 2 * y_step;
    }
  }
}

template <int LANES>
auto append_kernel(bool inter) {
  return inter ? rope_append_kernel<LANES, true> : rope_append_kernel<LANES, false>;
}
template <int LANES>
auto norm_kernel(bool inter, bool f32) {
  return f32 ? (inter ? norm_rope_kernel<float, LANES, true> : norm_rope_kernel<float, LANES, false>)
             : (inter ? norm_rope_kernel<__nv_bfloat16, LANES, true> : norm_rope_kernel<__nv_bfloat16, LANES, false>);
}

inline bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

// Checks shared by the two calls; fills *r.
int rot_args(const float* cos_sin, int table_len, int rot_dim, int interleaved, float eps, int D, RotArgs* r) {
  if (D <= 0 || !(eps >= 0.f) || !std::isfinite(eps)) return FA3_EINVAL;
  if (D % 8 != 0 || D > 256) return FA3_ERANGE;
  if (cos_sin) {
    if (table_len <= 0 || rot_dim <= 0 || rot_dim > D) return FA3_EINVAL;
    if (rot_dim % 8 != 0 || !aligned16(cos_sin)) return FA3_ERANGE;
  } else {
    rot_dim = 0;
    table_len = 0;
  }
  *r = RotArgs{cos_sin, table_len, rot_dim, interleaved ? 1 : 0, D, eps, 1.f / (float)D, (float)(1.0 / D - (double)(1.f / (float)D))};
  return FA3_OK;
}

int lanes_per_row(int D) { return D <= 64 ? 8 : D <= 128 ? 16 : 32; }

// Head rows a warp takes of one token: enough warps to fill the GPU come first (24 an SM),
// then longer tasks, which read a token's table row and place once for more heads.  With
// 64 warps an SM first, 999 tokens of 20 + 5 heads of 80 took 6.9 us instead of 4.8, and a
// ragged append of as many heads 13 instead of 10; large calls are the same with either.
int heads_per_task(int64_t tokens, int heads, int rows, int sms) {
  const int64_t passes = tokens * ((heads + rows - 1) / rows);
  const int64_t per = std::max<int64_t>(1, std::min<int64_t>(8, passes / ((int64_t)sms * 24)));
  return (int)per * rows;
}

}  // namespace
}  // namespace fa3

using namespace fa3;

FA3_API int fa3_norm_rope(const uint16_t* q, const uint16_t* k, const uint16_t* q_weight, const uint16_t* k_weight,
                          float eps, const float* cos_sin, int table_len, int rot_dim, int interleaved,
                          const int32_t* pos, void* q_out, void* k_out, int out_f32, int B, int S, int Hq, int Hkv,
                          int D, int64_t q_sb, int64_t q_ss, int64_t q_sh, int64_t k_sb, int64_t k_ss, int64_t k_sh,
                          int64_t qo_sb, int64_t qo_ss, int64_t qo_sh, int64_t ko_sb, int64_t ko_ss, int64_t ko_sh,
                          int32_t* dev_err, void* stream) {
  if (!q || !q_out || (cos_sin && !pos)) return FA3_EINVAL;
  if ((k == nullptr) != (k_out == nullptr) || (Hkv > 0 && !k)) return FA3_EINVAL;
  if (k && (q_weight == nullptr) != (k_weight == nullptr)) return FA3_EINVAL;
  if (B <= 0 || S <= 0 || Hq <= 0 || Hkv < 0 || (k && Hkv <= 0)) return FA3_EINVAL;
  NormRopeArgs a;
  int st = rot_args(cos_sin, table_len, rot_dim, interleaved, eps, D, &a.r);
  if (st != FA3_OK) return st;
  const int64_t strides[12] = {q_sb, q_ss, q_sh, k_sb, k_ss, k_sh, qo_sb, qo_ss, qo_sh, ko_sb, ko_ss, ko_sh};
  for (int i = 0; i < 12; ++i)
    if (strides[i] < 0 || strides[i] % 4 != 0) return FA3_ERANGE;
  if (!aligned8(q) || !aligned8(k) || !aligned8(q_weight) || !aligned8(k_weight) || !aligned16(q_out) ||
      !aligned16(k_out))
    return FA3_ERANGE;
  if ((int64_t)B * S >= ((int64_t)1 << 31) || (int64_t)Hq + Hkv > 65535) return FA3_ERANGE;
  int sms = 0;
  st = check_device(&sms);
  if (st != FA3_OK) return st;
  a.q = HeadRows{q, q_weight, q_sb, q_ss, q_sh};
  a.k = HeadRows{k, k_weight, k_sb, k_ss, k_sh};
  a.qo = HeadOut{q_out, qo_sb, qo_ss, qo_sh};
  a.ko = HeadOut{k_out, ko_sb, ko_ss, ko_sh};
  a.pos = pos; a.S = S; a.Hq = Hq; a.Hkv = Hkv; a.err = dev_err;
  const int lanes = lanes_per_row(D), rows = 32 / lanes, heads = Hq + Hkv;
  a.tokens = (uint32_t)((int64_t)B * S);
  a.per_chunk = (uint32_t)heads_per_task(a.tokens, heads, rows, sms);
  a.q_chunks = (Hq + a.per_chunk - 1) / a.per_chunk;
  a.chunks = a.q_chunks + (Hkv + a.per_chunk - 1) / a.per_chunk;
  const int64_t tasks = (int64_t)a.tokens * a.chunks;
  if (tasks >= ((int64_t)1 << 31)) return FA3_ERANGE;
  a.div_chunks = make_divu32(a.chunks);
  a.div_S = make_divu32((uint32_t)S);
  const int64_t blocks = std::min<int64_t>((tasks + kRopeWarps - 1) / kRopeWarps, (int64_t)sms * 8);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool inter = a.r.interleaved != 0, f32 = out_f32 != 0;
  auto* kernel = lanes == 8 ? norm_kernel<8>(inter, f32) : lanes == 16 ? norm_kernel<16>(inter, f32)
                                                                       : norm_kernel<32>(inter, f32);
  return cuda_status(launch_pdl(kernel, dim3((unsigned)blocks), dim3(kRopeThreads), 0, s, a));
}

FA3_API int fa3_rope_append_gqa_paged(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                      const uint16_t* q_weight, const uint16_t* k_weight, float eps,
                                      const float* cos_sin, int table_len, int rot_dim, int interleaved,
                                      const float* q_scale, const float* k_scale, const float* v_scale, int8_t* q_out,
                                      int8_t* k_cache, int8_t* v_cache, const int32_t* block_table,
                                      const int32_t* q_start, const int32_t* kv_lens, int n, int B, int Hq, int Hkv,
                                      int D, int64_t q_stride, int64_t k_stride, int64_t v_stride, int num_pages,
                                      int page_size, int max_pages, int32_t* dev_err, void* stream) {
  if (!k || !v || !k_scale || !v_scale || !k_cache || !v_cache || !block_table || !q_start || !kv_lens)
    return FA3_EINVAL;
  if ((q == nullptr) != (q_out == nullptr) || (q && !q_scale) || (q_weight && !q)) return FA3_EINVAL;
  if (n <= 0 || B <= 0 || Hkv <= 0 || Hq < 0 || (q && Hq <= 0) || D <= 0) return FA3_EINVAL;
  if (num_pages <= 0 || page_size <= 0 || max_pages <= 0) return FA3_EINVAL;
  if (!q) Hq = 0;
  RopeAppendArgs a;
  int st = rot_args(cos_sin, table_len, rot_dim, interleaved, eps, D, &a.r);
  if (st != FA3_OK) return st;
  if ((int64_t)max_pages * page_size >= ((int64_t)1 << 31) || B > kMostSequences) return FA3_ERANGE;
  if (q_stride < 0 || k_stride < 0 || v_stride < 0 || q_stride % 4 != 0 || k_stride % 4 != 0 || v_stride % 4 != 0)
    return FA3_ERANGE;
  if (!aligned8(q) || !aligned8(k) || !aligned8(v) || !aligned8(q_weight) || !aligned8(k_weight) || !aligned8(q_out) ||
      !aligned8(k_cache) || !aligned8(v_cache))
    return FA3_ERANGE;
  if ((int64_t)Hq + 2 * (int64_t)Hkv > 65535) return FA3_ERANGE;
  int sms = 0;
  st = check_device(&sms);
  if (st != FA3_OK) return st;
  a.q = HeadRows{q, q_weight, 0, q_stride, D};
  a.k = HeadRows{k, k_weight, 0, k_stride, D};
  a.v = HeadRows{v, nullptr, 0, v_stride, D};
  a.q_scale = q_scale; a.k_scale = k_scale; a.v_scale = v_scale;
  a.q_out = q_out; a.k_cache = k_cache; a.v_cache = v_cache;
  a.block_table = block_table; a.q_start = q_start; a.kv_lens = kv_lens;
  a.n = n; a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.num_pages = num_pages; a.page_size = page_size; a.max_pages = max_pages;
  a.T_max = max_pages * page_size; a.err = dev_err;
  const int lanes = lanes_per_row(D), rows = 32 / lanes, heads = Hq + 2 * Hkv;
  a.per_chunk = (uint32_t)heads_per_task(n, heads, rows, sms);
  a.q_chunks = (Hq + a.per_chunk - 1) / a.per_chunk;
  a.k_chunks = (Hkv + a.per_chunk - 1) / a.per_chunk;
  a.chunks = a.q_chunks + 2 * a.k_chunks;
  const int64_t tasks = (int64_t)n * a.chunks;
  if (tasks >= ((int64_t)1 << 31)) return FA3_ERANGE;
  a.div_chunks = make_divu32(a.chunks);
  a.div_ps = make_divu32((uint32_t)page_size);
  const int64_t blocks = std::min<int64_t>((tasks + kRopeWarps - 1) / kRopeWarps, (int64_t)sms * 8);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool inter = a.r.interleaved != 0;
  auto* kernel = lanes == 8 ? append_kernel<8>(inter) : lanes == 16 ? append_kernel<16>(inter)
                                                                    : append_kernel<32>(inter);
  return cuda_status(launch_pdl(kernel, dim3((unsigned)blocks + 1), dim3(kRopeThreads), 0, s, a));
}
