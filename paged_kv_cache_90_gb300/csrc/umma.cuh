// umma.cuh — issuing tcgen05 MMAs from a whole warp: one elected lane issues, every lane runs
// the code around it.  The descriptors are then the same in all lanes, and the compiler keeps
// them in uniform registers; issued from a branch of one lane they are moved there one by one,
// which takes longer than the MMA.
#pragma once

#include "tcgen05.cuh"

namespace pkv {
namespace umma {

// D (tmem) [+]= A (smem) * B (smem)
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile("{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
               "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
               ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
// D (tmem) [+]= A (tmem) * B (smem)
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile("{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
               "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
               ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
// arrive once on `bar` when every MMA the elected lane issued before has completed
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
               "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
               ::"r"(smem_addr(bar)) : "memory");
}

}  // namespace umma
}  // namespace pkv
