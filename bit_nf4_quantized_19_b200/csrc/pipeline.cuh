// Device helpers of the 8-bit operators' kernels beside common.cuh: barrier tests and
// warp-wide waits, a single elected lane, programmatic dependent launch, the two halves of
// a cluster barrier.
#pragma once
#include "common.cuh"

namespace qlora {

// Whether the phase is complete now.  (mbar_try_wait may suspend the thread for
// microseconds before it answers no.)
QDEV bool mbar_test(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// wait_bar by a whole warp, which leaves it with one answer.
QDEV bool wait_bar_warp(uint64_t *bar, uint32_t parity, const Waiter &w) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, w) ? 1 : 0) != 0;
}

// One lane of a converged warp.
QDEV bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// ------------------------------------------------------------------ programmatic dependent launch
// A kernel launched as a programmatic dependent may start while the kernel before it in the
// stream still runs: it does its setup, and touches global memory only after pdl_wait,
// which returns once that kernel has finished and its writes are visible.  pdl_trigger lets
// the kernel after this one do the same.  A kernel that triggers only after its own wait
// promises its dependent that everything older than itself has finished: a dependent that
// needs nothing of the kernel before it may then start its work at once and wait at its end
// (so that it, too, finishes after everything older).
QDEV void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
QDEV void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Loads behind a pdl_wait.  The kernel before may have written the words while this grid already
// lived, which the non-coherent path (__ldg, const __restrict__) rules out; these are coherent and,
// like the wait, volatile, so they stay behind it.
QDEV uint32_t ld_global_u8(const uint8_t *p) {
  uint32_t v;
  asm volatile("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
QDEV uint32_t ld_global_u32(const void *p) {
  uint32_t v;
  asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
QDEV uint2 ld_global_v2(const void *p) {
  uint2 v;
  asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
// (streamed data; with the wider L2 fetch the quantizer takes what it did on the non-coherent path:
// 8192 x 22016 90 us and 89, 8192 x 8192 35 and 37; without it 93 and 38)
QDEV uint4 ld_global_v4(const void *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
QDEV float4 ld_global_f4(const float *p) {
  float4 v;
  asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
  return v;
}

// The two halves of a cluster barrier, for work between them.
QDEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
QDEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

}  // namespace qlora
