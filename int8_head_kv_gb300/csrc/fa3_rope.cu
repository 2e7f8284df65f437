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
// a warp 4, 2 or 1 rows at a time.
#include "fa3_common.cuh"

#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

namespace fa3 {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;

// One tensor of head rows: row (b, s, h) starts at x + b * sb + s * ss + h * sh.
struct HeadRows {
  const uint16_t* x;
  const uint16_t* weight;   // [D] or nullptr
  int64_t sb, ss, sh;
};

struct RotArgs {
  const float* cos_sin;     // [table_len][rot], or nullptr: no rotation
  int table_len, rot, interleaved, D;
  float eps;
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

// f[0..7] = values at o1, o2 -> pair members a[e], b[e] (and back).
template <typename T>
__device__ __forceinline__ void to_pairs(const T* f, bool inter, T* a, T* b) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    a[e] = inter ? f[2 * e] : f[e];
    b[e] = inter ? f[2 * e + 1] : f[4 + e];
  }
}
template <typename T>
__device__ __forceinline__ void from_pairs(const T* a, const T* b, bool inter, T* f) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (inter) {
      f[2 * e] = a[e];
      f[2 * e + 1] = b[e];
    } else {
      f[e] = a[e];
      f[4 + e] = b[e];
    }
  }
}

// Sum over the lanes of a row (row_lanes a power of two).
template <typename T>
__device__ __forceinline__ T row_sum(T v, int row_lanes) {
  for (int o = row_lanes >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The transform in type T; x and w are the lane's values of the row and its weight.
template <typename T>
__device__ __forceinline__ void transform(const float (&x)[8], const float (&w)[8], bool norm, const Lane8& p,
                                          const RotArgs& r, float4 c4, float4 s4, int row_lanes, T (&y)[8]) {
  T f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = (T)x[e];
  if (norm) {
    T ss = (T)0;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss += f[e] * f[e];
    const T rstd = (T)1 / sqrt(row_sum(ss, row_lanes) / (T)r.D + (T)r.eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = f[e] * rstd * (T)w[e];
  }
  if (p.rotated) {
    T a[4], b[4], ya[4], yb[4];
    to_pairs(f, r.interleaved != 0, a, b);
    const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      ya[e] = a[e] * (T)c[e] - b[e] * (T)s[e];
      yb[e] = b[e] * (T)c[e] + a[e] * (T)s[e];
    }
    from_pairs(ya, yb, r.interleaved != 0, y);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = f[e];
  }
}

// ------------------------------------------------------------------- norm_rope
struct NormRopeArgs {
  HeadRows q, k;
  void *q_out, *k_out;
  int64_t qo_sb, qo_ss, qo_sh, ko_sb, ko_ss, ko_sh;
  RotArgs r;
  const int32_t* pos;       // [B * S]
  int S, Hq, Hkv;
  uint32_t tokens, chunks, per_chunk;   // head rows per warp task
  int row_lanes;
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

template <typename OUT>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(const NormRopeArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int i = lane & (a.row_lanes - 1), sub = lane / a.row_lanes, rows = 32 / a.row_lanes;
  const Lane8 p = lane_place(i, a.r);
  const uint32_t nt = a.tokens * a.chunks;
  for (uint32_t t = blockIdx.x * kRopeWarps + (threadIdx.x >> 5); t < nt; t += gridDim.x * kRopeWarps) {
    const uint32_t tok = divu32(t, a.div_chunks), chunk = t - tok * a.chunks;
    const uint32_t b = divu32(tok, a.div_S), s = tok - b * (uint32_t)a.S;
    float4 c4 = make_float4(1.f, 1.f, 1.f, 1.f), s4 = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.r.cos_sin) {
      const int pos = a.pos[tok];
      if (pos < 0 || pos >= a.r.table_len) {
        if (lane == 0) set_dev_err(a.err, FA3_DEVERR_POS);
        continue;
      }
      if (p.rotated) {
        const float* row = a.r.cos_sin + (int64_t)pos * a.r.rot + 4 * i;
        c4 = *reinterpret_cast<const float4*>(row);
        s4 = *reinterpret_cast<const float4*>(row + a.r.rot / 2);
      }
    }
    const int h_end = min((int)((chunk + 1) * a.per_chunk), a.Hq + a.Hkv);
    for (int h0 = chunk * a.per_chunk; h0 < h_end; h0 += rows) {
      const int hh = h0 + sub;
      const bool live = hh < h_end && p.in;
      const bool is_q = hh < a.Hq;
      const int h = is_q ? hh : hh - a.Hq;
      const HeadRows& T = is_q ? a.q : a.k;
      float x[8] = {}, w[8] = {}, y[8];
      if (live) {
        const uint16_t* xr = T.x + b * T.sb + s * T.ss + h * T.sh;
        bf16x4(load4(xr + p.o1), x);
        bf16x4(load4(xr + p.o2), x + 4);
        if (T.weight) {
          bf16x4(load4(T.weight + p.o1), w);
          bf16x4(load4(T.weight + p.o2), w + 4);
        }
      }
      transform<float>(x, w, a.q.weight != nullptr || a.k.weight != nullptr, p, a.r, c4, s4, a.row_lanes, y);
      if (live) {
        OUT* yr = is_q ? (OUT*)a.q_out + b * a.qo_sb + s * a.qo_ss + h * a.qo_sh
                       : (OUT*)a.k_out + b * a.ko_sb + s * a.ko_ss + h * a.ko_sh;
        store4(yr + p.o1, y);
        store4(yr + p.o2, y + 4);
      }
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
  uint32_t chunks, per_chunk;
  int row_lanes;
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

__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeAppendArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int i = lane & (a.row_lanes - 1), sub = lane / a.row_lanes, rows = 32 / a.row_lanes;
  const Lane8 p = lane_place(i, a.r);
  const Lane8 pass = {8 * i, 8 * i + 4, p.in, false};
  const uint32_t nt = (uint32_t)a.n * a.chunks;
  const int heads = a.Hq + 2 * a.Hkv;
  for (uint32_t t = blockIdx.x * kRopeWarps + (threadIdx.x >> 5); t < nt; t += gridDim.x * kRopeWarps) {
    const int row = (int)divu32(t, a.div_chunks);
    const int chunk = (int)(t - (uint32_t)row * a.chunks);
    const int b = find_sequence(a.q_start, a.B, row, lane);
    if (b < 0 || b >= a.B) continue;                       // behind the last sequence
    const int q0 = a.q_start[b], q1 = a.q_start[b + 1], kv = a.kv_lens[b];
    if (q0 < 0 || q1 <= row || q1 > a.n || kv < q1 - q0 || kv > a.T_max) {
      if (lane == 0) set_dev_err(a.err, FA3_DEVERR_LENS);
      continue;
    }
    const int pos = kv - (q1 - row);
    float4 c4 = make_float4(1.f, 1.f, 1.f, 1.f), s4 = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.r.cos_sin) {
      if (pos >= a.r.table_len) {
        if (lane == 0) set_dev_err(a.err, FA3_DEVERR_POS);
        continue;
      }
      if (p.rotated) {
        const float* tr = a.r.cos_sin + (int64_t)pos * a.r.rot + 4 * i;
        c4 = *reinterpret_cast<const float4*>(tr);
        s4 = *reinterpret_cast<const float4*>(tr + a.r.rot / 2);
      }
    }
    const uint32_t pi = divu32((uint32_t)pos, a.div_ps);
    const int pg = a.block_table[(int64_t)b * a.max_pages + pi];
    const bool page_ok = pg >= 0 && pg < a.num_pages;
    if (!page_ok && lane == 0) set_dev_err(a.err, FA3_DEVERR_PAGE);
    const int64_t pool_row = (int64_t)pg * a.page_size + (pos - (int)pi * a.page_size);
    const int h_end = min((chunk + 1) * (int)a.per_chunk, heads);
    for (int h0 = chunk * (int)a.per_chunk; h0 < h_end; h0 += rows) {
      const int hh = h0 + sub;
      const int kind = hh < a.Hq ? 0 : hh < a.Hq + a.Hkv ? 1 : 2;
      const int h = kind == 0 ? hh : kind == 1 ? hh - a.Hq : hh - a.Hq - a.Hkv;
      const bool live = hh < h_end && p.in && (kind == 0 ? a.q_out != nullptr : page_ok);
      const HeadRows& T = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
      const Lane8 pl = kind == 2 ? pass : p;
      float x[8] = {}, w[8] = {};
      float sc = 0.f;
      if (live) {
        const uint16_t* xr = T.x + row * T.ss + h * T.sh;
        bf16x4(load4(xr + pl.o1), x);
        bf16x4(load4(xr + pl.o2), x + 4);
        if (T.weight) {
          bf16x4(load4(T.weight + pl.o1), w);
          bf16x4(load4(T.weight + pl.o2), w + 4);
        }
        sc = (kind == 0 ? a.q_scale : kind == 1 ? a.k_scale : a.v_scale)[h];
      }
      const bool norm = kind < 2 && T.weight != nullptr;
      double y[8];
      {
        double f[8], ss = 0.0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          f[e] = (double)x[e];
          ss += f[e] * f[e];
        }
        ss = row_sum(ss, a.row_lanes);
        if (norm) {
          const double rstd = 1.0 / sqrt(ss / (double)a.r.D + (double)a.r.eps);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = f[e] * rstd * (double)w[e];
        }
        if (pl.rotated) {
          double pa[4], pb[4], ya[4], yb[4];
          to_pairs(f, a.r.interleaved != 0, pa, pb);
          const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            ya[e] = pa[e] * (double)c[e] - pb[e] * (double)s[e];
            yb[e] = pb[e] * (double)c[e] + pa[e] * (double)s[e];
          }
          from_pairs(ya, yb, a.r.interleaved != 0, y);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = f[e];
        }
      }
      if (live) {
        uint32_t packed[2] = {0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          int code = 0;
          if (kind == 2) {
            code = quant_code(x[e], sc);
          } else if (sc != 0.f) {
            code = __double2int_rn(fmin(fmax(y[e] / (double)sc, -127.0), 127.0));
          }
          packed[e >> 2] |= ((uint32_t)code & 0xffu) << (8 * (e & 3));
        }
        int8_t* dst = kind == 0 ? a.q_out + ((int64_t)row * a.Hq + h) * a.r.D
                                : (kind == 1 ? a.k_cache : a.v_cache) + (pool_row * a.Hkv + h) * a.r.D;
        *reinterpret_cast<uint32_t*>(dst + pl.o1) = packed[0];
        *reinterpret_cast<uint32_t*>(dst + pl.o2) = packed[1];
      }
    }
  }
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
  *r = RotArgs{cos_sin, table_len, rot_dim, interleaved ? 1 : 0, D, eps};
  return FA3_OK;
}

int lanes_per_row(int D) { return D <= 64 ? 8 : D <= 128 ? 16 : 32; }

// Head rows a warp takes of one token: enough warps to fill the GPU come first, then
// longer tasks, which read a token's table row and place once for more heads.
int heads_per_task(int64_t tokens, int heads, int rows, int sms) {
  const int64_t passes = tokens * ((heads + rows - 1) / rows);
  const int64_t per = std::max<int64_t>(1, std::min<int64_t>(8, passes / ((int64_t)sms * 64)));
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
  a.q_out = q_out; a.k_out = k_out;
  a.qo_sb = qo_sb; a.qo_ss = qo_ss; a.qo_sh = qo_sh; a.ko_sb = ko_sb; a.ko_ss = ko_ss; a.ko_sh = ko_sh;
  a.pos = pos; a.S = S; a.Hq = Hq; a.Hkv = Hkv; a.err = dev_err;
  a.row_lanes = lanes_per_row(D);
  const int rows = 32 / a.row_lanes, heads = Hq + Hkv;
  a.tokens = (uint32_t)((int64_t)B * S);
  a.per_chunk = (uint32_t)heads_per_task(a.tokens, heads, rows, sms);
  a.chunks = (heads + a.per_chunk - 1) / a.per_chunk;
  const int64_t tasks = (int64_t)a.tokens * a.chunks;
  if (tasks >= ((int64_t)1 << 31)) return FA3_ERANGE;
  a.div_chunks = make_divu32(a.chunks);
  a.div_S = make_divu32((uint32_t)S);
  const int64_t blocks = std::min<int64_t>((tasks + kRopeWarps - 1) / kRopeWarps, (int64_t)sms * 8);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(launch_pdl(out_f32 ? norm_rope_kernel<float> : norm_rope_kernel<__nv_bfloat16>,
                                dim3((unsigned)blocks), dim3(kRopeThreads), 0, s, a));
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
  if ((int64_t)max_pages * page_size >= ((int64_t)1 << 31)) return FA3_ERANGE;
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
  a.row_lanes = lanes_per_row(D);
  const int rows = 32 / a.row_lanes, heads = Hq + 2 * Hkv;
  a.per_chunk = (uint32_t)heads_per_task(n, heads, rows, sms);
  a.chunks = (heads + a.per_chunk - 1) / a.per_chunk;
  const int64_t tasks = (int64_t)n * a.chunks;
  if (tasks >= ((int64_t)1 << 31)) return FA3_ERANGE;
  a.div_chunks = make_divu32(a.chunks);
  a.div_ps = make_divu32((uint32_t)page_size);
  const int64_t blocks = std::min<int64_t>((tasks + kRopeWarps - 1) / kRopeWarps, (int64_t)sms * 8);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(launch_pdl(rope_append_kernel, dim3((unsigned)blocks), dim3(kRopeThreads), 0, s, a));
}
