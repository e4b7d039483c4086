// Further tcgen05 helpers: the lane that issues, and the single-CTA (cta_group::1)
// forms next to the CTA pairs' ones of bl_device.cuh.
#pragma once

#include <cstdint>

#include "bl_device.cuh"

namespace bl {

// One lane of the (converged) warp. A loop that loads or multiplies runs in all lanes of
// its warp and this one issues: code after elect.sync keeps the instructions' descriptors
// in uniform registers. (Under `lane == 0` each tcgen05.mma took 63 cycles to issue, a
// stage of four and its waits 530, for 512 of the tensor cores'.)
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.b32 %0, 1, 0, q;\n\t}" : "=r"(yes));
  return yes != 0;
}

// A bounded wait of a whole (converged) warp, decided by all of its lanes: where the wait
// runs out, or another warp gives up, between two lanes' looks at the barrier, no lane
// goes on alone to an instruction that takes the whole warp.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, err));
}

// Single-CTA (cta_group::1) forms.
__device__ __forceinline__ void tmem_alloc_one(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)), "r"(ncols)
               : "memory");
}

__device__ __forceinline__ void tmem_relinquish_one() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc_one(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

__device__ __forceinline__ void mma_i8_one(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrives once on the barrier when all MMAs previously issued by this thread
// complete.
__device__ __forceinline__ void mma_commit_one(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

}  // namespace bl
