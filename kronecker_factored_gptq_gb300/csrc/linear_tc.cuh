// Building blocks of the linear layer's tcgen05 kernels: 16-bit matrix
// instructions, TMEM access, waits and the position in a ring of stages.
#pragma once

#include "linear.cuh"
#include "tc_common.cuh"

namespace bakron {
namespace tc {

__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

template <typename H>
struct IdescType;
template <>
struct IdescType<__half> { static constexpr uint32_t v = 0; };
template <>
struct IdescType<__nv_bfloat16> { static constexpr uint32_t v = 1; };
template <typename H>
__device__ __forceinline__ uint32_t idesc_f16(int n) {
  return (1u << 4) | (IdescType<H>::v << 7) | (IdescType<H>::v << 10) | ((uint32_t)(n >> 3) << 17) |
         ((128u >> 4) << 24);
}

// Bounded wait; the clock is read only once the first try has failed.  When it
// runs out the block records BAKRON_ERR_TIMEOUT and its other roles stop.
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, int* abort, int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  volatile int* ab = abort;
  if (mbar_wait(bar, parity, ab)) return true;
  atomicCAS(status, 0, (int)BAKRON_ERR_TIMEOUT);
  *ab = 1;
  return false;
}
// Position in a ring of stages, advanced without divisions: stage s and the
// parity of its current use.
struct Ring {
  int s = 0;
  uint32_t parity = 0;
  bool first = true;      // first time round: the stage is free
  __device__ __forceinline__ void advance(int by, int stages) {
    s += by;
    if (s >= stages) {
      s -= stages;
      parity ^= 1;
      first = false;
    }
  }
};
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

}  // namespace tc
}  // namespace bakron
