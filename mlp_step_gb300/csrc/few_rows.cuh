// What the kernels for a few rows share: a thread's ring of asynchronously
// copied pieces of W, and reads of another CTA's sums.
#pragma once

#include "ptx.cuh"
#include "rowvec.cuh"

namespace mlp {

// One piece of W into the thread's slot: asynchronously where it is whole and
// aligned, else value by value (the same thread reads it, in program order).
template <typename T>
__device__ __forceinline__ void few_issue(uint4* slot, const T* p, int n, bool vec) {
  if (vec && n >= RowVec<T>::N) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(slot)), "l"(p)
                 : "memory");
  } else {
    *slot = load_piece(p, n, false);
  }
}
__device__ __forceinline__ void few_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void few_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

}  // namespace mlp
