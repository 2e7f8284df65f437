// What the persistent tcgen05 kernels on packed rows share (fa3_chunk.cu, fa3_weights.cu): the line of work and its parts,
// bounded waits for warps, loads and stores, and MMAs issued from converged warps.
#pragma once

#include "fa3_tc.cuh"

namespace fa3 {
namespace {

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
// wait_bar for short waits, with bounded_wait's rare look at the clock, in ticks of 2^20 ns (1.05 ms).  A second, unless
// the caller says otherwise.
constexpr uint32_t kWaitTicks = 954;
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

// 16 bytes that this SM reads once: the L1 (what shared memory leaves of it) is passed by.  (Not as read-only data: the call
// before may have written them after this kernel had begun.)
__device__ __forceinline__ uint4 load_once(const int8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
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
__device__ __forceinline__ void commit_if(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n.reg .pred e;\nsetp.ne.b32 e, %1, 0;\n"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar), "r"(lead)
      : "memory");
}

}  // namespace
}  // namespace fa3
