// Copies and waits of the tensor-core attention kernels.
#pragma once

#include "prefill.cuh"
#include "tcgen05.cuh"

namespace skv {
namespace {

__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap* map, int x, int y,
                                         uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// A whole warp's bounded wait, with one answer for all its lanes: each lane reads the timer for
// itself, and where some gave up while others went on, the rest of the warp's code (TMEM loads,
// votes) would run without them. mbar_wait_bounded in fewer instructions: this kernel has thirty
// waits.
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity,
                                             unsigned long long limit_ns) {
  bool ok = true;
  uint64_t t0 = 0;
  while (!mbar_try_wait(bar, parity)) {
    const uint64_t t = global_timer_ns();
    if (t0 == 0) t0 = t;
    if (t - t0 > limit_ns) {
      ok = false;
      break;
    }
  }
  return __all_sync(0xffffffffu, ok);
}
// 64 columns of a tile's rows: G heads of 128 / G tokens of the query tensor [T][Hq][D].
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int x, int head,
                                         int token, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(head), "r"(token),
        "r"(smem_addr(bar)) : "memory");
}

// A value that is the same in every lane, said so that the compiler keeps it, and what follows
// from it, in uniform registers: the products' descriptors come from there.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Hint: bring the 128-byte line holding p into L1.
__device__ __forceinline__ void prefetch_l1(const void* p) {
  asm volatile("prefetch.global.L1 [%0];" ::"l"(p));
}

}  // namespace
}  // namespace skv
