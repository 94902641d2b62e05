// pba_ptx_more.cuh -- further PTX of the kernels around the attention block.  Apart
// from pba_ptx.cuh, whose text is part of the attention kernel's and of its
// measured traffic's record.
#pragma once

#include "pba_ptx.cuh"

namespace pba {

// cp_async16 with the first `bytes` (0 to 16) read and the rest filled with zeros.
__device__ __forceinline__ void cp_async16_part(void *dst_smem, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst_smem)), "l"(src), "r"(bytes)
               : "memory");
}
// Waits until at most N committed copy groups of this thread are under way.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One lane of a converged warp (the same one every time).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

}  // namespace pba
