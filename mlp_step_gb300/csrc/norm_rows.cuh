// Rows of a matrix held in registers by the norms' kernels: blocks, sums over a
// row, parameter vectors, and the size of a launch that walks over rows.
#pragma once

#include "rowvec.cuh"

namespace mlp {

namespace {

constexpr int kPerThread = 16;        // values of a row per thread
constexpr int kHeldWidth = 16 * 512;  // widest row held by one block's registers

// Threads of the blocks that hold rows with WPR warps each.
template <int WPR>
struct HeldBlock {
  static constexpr int ROWS = WPR >= 8 ? 1 : 8 / WPR;  // rows at a time
  static constexpr int THREADS = 32 * WPR * ROWS;
};

// Waits for the warps that share a row (the whole block where it holds one).
template <int WPR>
__device__ __forceinline__ void row_barrier(int slot) {
  if constexpr (WPR == 1) __syncwarp();
  else if constexpr (WPR >= 8) __syncthreads();
  else asm volatile("bar.sync %0, %1;" ::"r"(slot + 1), "r"(32 * WPR) : "memory");
}

// Sums of NV values over the row's threads, the same in each and in a fixed
// order.  `part`: NV * WPR floats of the row's slot, of which callers use two
// in turn so that one barrier a call is enough.
template <int WPR, int NV>
__device__ __forceinline__ void row_sums(float (&v)[NV], float* part, int slot, int warp_in_row) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int i = 0; i < NV; ++i) part[i * WPR + warp_in_row] = v[i];
    row_barrier<WPR>(slot);
    // one load and log2(WPR) exchanges (a load per partial, in every thread,
    // was two loads per value of a row of 8,192)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[i] = part[i * WPR + (threadIdx.x & (WPR - 1))];
#pragma unroll
      for (int o = WPR / 2; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
  }
}

// N parameter values (fp32) from column c (a multiple of N), `fill` past n values
// or without a vector.
template <int N, bool FULL = false>
__device__ __forceinline__ void load_param(const float* p, int c, int n, float fill,
                                           float (&v)[N]) {
  if (p && (FULL ? n > 0 : n >= N)) {
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(p + c + j));
      v[j] = f.x;
      v[j + 1] = f.y;
      v[j + 2] = f.z;
      v[j + 3] = f.w;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = !FULL && p && j < n ? __ldg(p + c + j) : fill;
}

bool row_vec(const void* p, long long ld, int esz, int bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * esz % bytes == 0;
}

// Blocks of a row-walking launch: as many as are resident at once (more would
// run as a second, ragged wave), at most one per row set.
template <typename K>
int walk_blocks(K kernel, int threads, PerDevice& resident, long long T, int rows_per_block,
                int smem = 0) {
  const int per_sm = resident.get(current_device(), [&] {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess) {
      cudaGetLastError();
      n = 1;
    }
    return n > 0 ? n : 1;
  });
  const long long need = (T + rows_per_block - 1) / rows_per_block;
  const long long most = (long long)num_sms() * per_sm;
  return (int)(need < most ? need : most);
}

}  // namespace

}  // namespace mlp
