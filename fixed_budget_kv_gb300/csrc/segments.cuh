// What the persistent attention kernels share: work shared out over the CTAs, places in a ring
// of tiles, and MMAs issued by a warp in step.
#pragma once

#include "common.cuh"

namespace kvpop {

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// mbar_wait and report_error with their long parts out of line: a persistent kernel's roles wait in
// dozens of places, and with all of them inline its loops leave the instruction cache (the received
// weight of decode rows: a quarter of the fetches missed).
static __device__ __noinline__ bool bar_wait_long(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return mbar_wait(bar, parity, abort_flag);
}
static __device__ __noinline__ void give_up(int* status, int site, int detail, volatile int* abort_flag) {
  report_error(status, KVPOP_ERR_TIMEOUT, site, detail);
  *abort_flag = 1;
}
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return mbar_try_wait(bar, parity) || bar_wait_long(bar, parity, abort_flag);
}
__device__ __forceinline__ bool bar_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, bar_wait(bar, parity, abort_flag));
}

__device__ __forceinline__ int scan_incl(int x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane_id() >= o) x += y;
  }
  return x;
}

// U units over C CTAs: the first U mod C of them take one more.
struct Share {
  int q, r;
  __device__ __forceinline__ Share(int U, int C) : q(U / C), r(U - U / C * C) {}
  __device__ __forceinline__ int first(int c) const { return q * c + min(c, r); }
  __device__ __forceinline__ int cta_of(int u) const {
    const int big = r * (q + 1);
    return u < big ? u / (q + 1) : r + (u - big) / q;
  }
};

// The MMA wrappers for a whole warp: one elected lane issues.
__device__ __forceinline__ void mma_ss_elect(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 a, b;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHiSw128)
      : "memory");
}
__device__ __forceinline__ void mma_ts_elect(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 b;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHiSw128)
      : "memory");
}
__device__ __forceinline__ void mma_commit_elect(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}

// Place of a key tile's K and V among the segment's 2 NT loads: the order in which
// the MMA warp uses them (S runs two events ahead of P V).
__device__ __forceinline__ int pos_v(bool two, int NT, int t) { return two ? 2 * t + 1 : min(NT, t + 2) + t; }

// A place in a ring of N stages and the parity of its use.
template <int N>
struct Ring {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void skip(int d) {  // d < N
    st += d;
    if (st >= N) {
      st -= N;
      ph ^= 1;
    }
  }
  __device__ __forceinline__ void jump(int d) {
    ph ^= d / N & 1;
    skip(d % N);
  }
};

}  // namespace kvpop
