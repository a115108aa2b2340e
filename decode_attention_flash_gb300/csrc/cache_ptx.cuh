// cache_ptx.cuh -- PTX that the cache kernels and the 4-bit float decode use beside ptx.cuh.
#pragma once

#include "ptx.cuh"

namespace da {

// A shared-memory word that one warp writes and another reads (release / acquire in the block).
__device__ __forceinline__ void st_release_cta(uint32_t *p, uint32_t v) {
  asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(smem_u32(p)), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_acquire_cta(const uint32_t *p) {
  uint32_t v;
  asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(v) : "r"(smem_u32(p)) : "memory");
  return v;
}

// ---------------------------------------------------------------- dependent launches
// Kernels launched with launch_dependent (cache_ops.h) may start while the previous
// kernel of the stream is still running: nothing that it may have written is read,
// and nothing at all is written, before this returns. They are alive while that kernel
// writes, so what a kernel of a serving step may write (slots, positions, tables, queries,
// cache rows) is read by ordinary loads, which the wait orders; __ldg, whose memory nobody may
// write during a kernel's life, takes constants alone: cosines, head scales, masks.
__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next kernel of the stream start its blocks (they wait as above).
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---------------------------------------------------------------- cp.async

// 16 bytes to the shared address `smem_dst` (both sides 16-byte aligned), past L1.
__device__ __forceinline__ void cp_async_16(uint32_t smem_dst, const void *gsrc) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_dst),
               "l"(reinterpret_cast<uint64_t>(gsrc))
               : "memory");
}

}  // namespace da
