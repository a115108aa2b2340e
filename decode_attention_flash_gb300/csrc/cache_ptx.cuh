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

// Both: how a kernel that has nothing to do before the wait begins.
__device__ __forceinline__ void begin_dependent() {
  wait_for_previous_kernel();
  let_next_kernel_start();
}

// ---------------------------------------------------------------- packed fp32

// Two floats in a register pair, added or multiplied by one instruction (sm_100 and later), each
// result rounded by itself as by __fadd_rn, __fsub_rn, __fmul_rn.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pack(float a, float b) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack(Pair v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair sub2(Pair a, Pair b) {
  Pair r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// ---------------------------------------------------------------- cp.async

// 16 bytes to the shared address `smem_dst` (both sides 16-byte aligned), past L1.
__device__ __forceinline__ void cp_async_16(uint32_t smem_dst, const void *gsrc) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_dst),
               "l"(reinterpret_cast<uint64_t>(gsrc))
               : "memory");
}

}  // namespace da
