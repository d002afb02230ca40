// What stands between two blocks of a network: the norm of the block's output,
// its gate, dropout, the scaled residual, and the norm before the next block.
//   forward   c = post_gain b rb,  rb = 1 / sqrt(mean b^2 + eps)   (or post_gain b)
//             h = x + scale G dropout(c),  G = z, 1 / (1 + e^(-z)) or 1
//             n = next_gain h rh,  rh = 1 / sqrt(mean h^2 + eps)
//   backward  t = dn next_gain,  dh' = dh + rh (t - hh mean(t hh)),  hh = h rh
//             dx = dh',  e = scale dh' keep
//             dz = e c G',  v = e G,  dpost_gain = sum v bb,  bb = b rb
//             db = rb (v post_gain - bb mean(v post_gain bb))   (or v post_gain)
//             dnext_gain = sum dn hh
// n is taken from the unrounded h.  All of it is bound by HBM (forward up to 10,
// backward up to 16 bytes per bf16 value), so a row is read once and stays in
// registers between its two reductions; everything between load and store is
// fp32, and the dropout mask is computed where it is used (philox.cuh).
//
// A row is held by WPR warps, 16 values per thread as in k_layernorm.cu; rows
// wider than a block holds (8,192) are held by a cluster of up to eight blocks,
// whose sums meet in distributed shared memory, so they too are read once.
// Parameter gradients stay in registers over a block's rows and leave as one
// row of partial sums per block (cluster): no atomics, the same in every run.
#include "act.cuh"
#include "few_rows.cuh"
#include "kernels.cuh"
#include "norm_rows.cuh"
#include "philox.cuh"
#include "rowvec.cuh"
#include "trace.cuh"

namespace mlp {

namespace {

constexpr int kMaxCluster = 8;

// Bits of ResNorm::vec: 16-byte pieces of that matrix's rows are aligned.
enum { kXVec = 1, kBVec = 2, kZVec = 4, kHVec = 8, kNVec = 16, kDxVec = 32, kDbVec = 64,
       kDzVec = 128 };

// Sums of one value over the row: over a block's warps, then (WIDE) over the
// cluster's blocks in rank order.  Callers alternate `turn`, so that one barrier
// a call (each) is enough.
template <int WPR, bool WIDE, int ROWS>
struct RowSum {
  float (*part)[ROWS][WPR];  // [2][ROWS][WPR]
  float* mine;               // WIDE: [2] in this block's shared memory
  int slot, warp_in_row, cluster, turn;
  __device__ __forceinline__ float operator()(float v) {
    float s[1] = {v};
    row_sums<WPR>(s, part[turn][slot], slot, warp_in_row);
    if constexpr (WIDE) {
      if (threadIdx.x == 0) mine[turn] = s[0];
      ptx::cluster_sync();
      const uint32_t at = ptx::smem_u32(mine + turn);
      s[0] = 0.f;
      for (int r = 0; r < cluster; ++r)
        s[0] += ld_cluster_f32(ptx::mapa_shared(at, (uint32_t)r));
    }
    turn ^= 1;
    return s[0];
  }
};

// The logistic function s of two values, and what s' is s times: 1 - s =
// e^(-z) s, which keeps its precision where s is near 1 (e^(-z) held to a finite
// value, where s makes the product 0).  The accurate functions for fp32 rows.
template <typename T>
__device__ __forceinline__ F2 logistic2(F2 z, F2& one_minus) {
  F2 e, s;
  if constexpr (sizeof(T) == 4) {
    e = f2(expf(-z.x), expf(-z.y));
    s = f2(__fdividef(1.f, 1.f + e.x), __fdividef(1.f, 1.f + e.y));
  } else {
    const F2 t = mul2(z, f2(-1.4426950408889634f));
    e = f2(ex2_fast(t.x), ex2_fast(t.y));
    const F2 d = add2(e, f2(1.f));
    s = f2(rcp_fast(d.x), rcp_fast(d.y));
  }
  one_minus = mul2(f2(fminf(e.x, 5e34f), fminf(e.y, 5e34f)), s);
  return s;
}

template <typename T, int WPR, bool FULL, bool WIDE>
__global__ void __launch_bounds__(HeldBlock<WPR>::THREADS,
                                  (sizeof(T) == 2 ? 768 : 512) / HeldBlock<WPR>::THREADS)
    resnorm_fwd_kernel(const ResNorm p, int cluster) {
  constexpr int N = RowVec<T>::N, NV = kPerThread / N, ROWS = HeldBlock<WPR>::ROWS;
  __shared__ float part[2][ROWS][WPR];
  __shared__ float mine[2];
  pdl_wait();
  pdl_launch_dependents();
  const int slot = threadIdx.x / (32 * WPR), t = threadIdx.x % (32 * WPR);
  const int rank = WIDE ? (int)(blockIdx.x % cluster) : 0;
  const int c_first = rank * kHeldWidth + t * N;  // piece i at c_first + i 32 WPR N
  const long long stride = WIDE ? gridDim.x / cluster : (long long)gridDim.x * ROWS;
  long long row = WIDE ? blockIdx.x / cluster : (long long)blockIdx.x * ROWS + slot;
  const float inv_d = 1.f / (float)p.d;
  const bool block = p.b != nullptr, gate = p.z != nullptr;
  const DropKey key(p.drop);
  RowSum<WPR, WIDE, ROWS> sum{part, mine, slot, t >> 5, cluster, 0};
  uint4 rx[NV], rb[NV], rz[NV];
  auto load = [&](long long r) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c_first + i * 32 * WPR * N;
      const int n = r < p.T ? p.d - c : 0;
      rx[i] = load_piece_of<FULL>(static_cast<const T*>(p.x) + r * p.ldx + c, n, p.vec & kXVec);
      if (block)
        rb[i] = load_piece_of<FULL>(static_cast<const T*>(p.b) + r * p.ldb + c, n, p.vec & kBVec);
      if (gate)
        rz[i] = load_piece_of<FULL>(static_cast<const T*>(p.z) + r * p.ldz + c, n, p.vec & kZVec);
    }
  };
  load(row);
  for (; row < p.T; row += stride) {  // uniform over the threads that share a row
    F2 v[NV][N / 2];
    if (block) {
      F2 s2 = f2(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        unpack_piece<T>(rb[i], v[i]);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) s2 = fma2(v[i][j], v[i][j], s2);
      }
      float rho = 1.f;
      if (p.post) {
        rho = rsqrtf(sum(s2.x + s2.y) * inv_d + p.eps);  // two ulp
        if (p.b_rstd && rank == 0 && t == 0) p.b_rstd[row] = rho;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = c_first + i * 32 * WPR * N, n = p.d - c;
        float g[N];
        load_param<N, FULL>(p.post_gain, c, n, 1.f, g);
        const uint32_t bits =
            p.drop.threshold ? drop_bits<N>(p.drop, key, (uint32_t)row, c) : 0u;
        F2 x[N / 2], z[N / 2];
        unpack_piece<T>(rx[i], x);
        if (gate) unpack_piece<T>(rz[i], z);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          F2 e = mul2(mul2(v[i][j], f2(rho)), f2(g[2 * j], g[2 * j + 1]));
          if (p.drop.threshold) e = drop2(e, bits, 2 * j, p.drop.scale);
          if (gate) {
            F2 rest;
            e = mul2(e, p.sigmoid ? logistic2<T>(z[j], rest) : z[j]);
          }
          v[i][j] = fma2(e, f2(p.scale), x[j]);
          // past the row's end (where 0 times a scale that is not finite would not be 0)
          if (2 * j >= n) v[i][j].x = 0.f;
          if (2 * j + 1 >= n) v[i][j].y = 0.f;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) unpack_piece<T>(rx[i], v[i]);
    }
    load(row + stride);
    if (p.h) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = c_first + i * 32 * WPR * N;
        store_piece_of<FULL>(static_cast<T*>(p.h) + row * p.ldh + c,
                             reinterpret_cast<const float(&)[N]>(v[i]), p.d - c, p.vec & kHVec);
      }
    }
    if (p.n) {
      F2 s2 = f2(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < N / 2; ++j) s2 = fma2(v[i][j], v[i][j], s2);
      const float rho = rsqrtf(sum(s2.x + s2.y) * inv_d + p.eps);
      if (p.h_rstd && rank == 0 && t == 0) p.h_rstd[row] = rho;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = c_first + i * 32 * WPR * N, n = p.d - c;
        float g[N];
        load_param<N, FULL>(p.next_gain, c, n, 1.f, g);
#pragma unroll
        for (int j = 0; j < N / 2; ++j)
          v[i][j] = mul2(mul2(v[i][j], f2(rho)), f2(g[2 * j], g[2 * j + 1]));
        store_piece_of<FULL>(static_cast<T*>(p.n) + row * p.ldn + c,
                             reinterpret_cast<const float(&)[N]>(v[i]), n, p.vec & kNVec);
      }
    }
  }
  if constexpr (WIDE) ptx::cluster_sync();  // no block leaves while its sums may be read
}

template <typename T, int WPR, bool FULL, bool WIDE>
__global__ void __launch_bounds__(HeldBlock<WPR>::THREADS,
                                  sizeof(T) == 2 ? 512 / HeldBlock<WPR>::THREADS : 1)
    resnorm_bwd_kernel(const ResNorm p, int cluster) {
  constexpr int N = RowVec<T>::N, NV = kPerThread / N, ROWS = HeldBlock<WPR>::ROWS;
  __shared__ float part[2][ROWS][WPR];
  __shared__ float mine[2];
  extern __shared__ __align__(16) float sums_mem[];  // ROWS > 1: one slot's values at a time
  pdl_wait();
  pdl_launch_dependents();
  const int slot = threadIdx.x / (32 * WPR), t = threadIdx.x % (32 * WPR);
  const int rank = WIDE ? (int)(blockIdx.x % cluster) : 0;
  const int c_first = rank * kHeldWidth + t * N;
  const long long stride = WIDE ? gridDim.x / cluster : (long long)gridDim.x * ROWS;
  long long row = WIDE ? blockIdx.x / cluster : (long long)blockIdx.x * ROWS + slot;
  const float inv_d = 1.f / (float)p.d;
  const bool block = p.b != nullptr, gate = p.z != nullptr, next = p.n != nullptr;
  const DropKey key(p.drop);
  RowSum<WPR, WIDE, ROWS> sum{part, mine, slot, t >> 5, cluster, 0};
  F2 dnext[NV][N / 2], dpost[NV][N / 2];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < N / 2; ++j) dnext[i][j] = dpost[i][j] = f2(0.f);
  uint4 rx[NV], rn[NV], rh[NV];
  auto load = [&](long long r) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c_first + i * 32 * WPR * N;
      const int n = r < p.T ? p.d - c : 0;
      if (next) {
        rn[i] = load_piece_of<FULL>(static_cast<const T*>(p.n) + r * p.ldn + c, n, p.vec & kNVec);
        rh[i] = load_piece_of<FULL>(static_cast<const T*>(p.h) + r * p.ldh + c, n, p.vec & kHVec);
      }
      rx[i] = p.x ? load_piece_of<FULL>(static_cast<const T*>(p.x) + r * p.ldx + c, n,
                                        p.vec & kXVec)
                  : make_uint4(0, 0, 0, 0);
    }
  };
  load(row);
  for (; row < p.T; row += stride) {
    // this row's b and z are in flight over the first reduction
    uint4 rb[NV], rz[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c_first + i * 32 * WPR * N;
      if (block)
        rb[i] = load_piece_of<FULL>(static_cast<const T*>(p.b) + row * p.ldb + c, p.d - c,
                                    p.vec & kBVec);
      if (gate)
        rz[i] = load_piece_of<FULL>(static_cast<const T*>(p.z) + row * p.ldz + c, p.d - c,
                                    p.vec & kZVec);
    }
    F2 v[NV][N / 2];  // dh'
    if (next) {
      const float rho = p.h_rstd[row];
      F2 hh[NV][N / 2];
      F2 s2 = f2(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = c_first + i * 32 * WPR * N, n = p.d - c;
        float g[N];
        load_param<N, FULL>(p.next_gain, c, n, 1.f, g);
        unpack_piece<T>(rn[i], v[i]);
        unpack_piece<T>(rh[i], hh[i]);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          hh[i][j] = mul2(hh[i][j], f2(rho));
          if (2 * j >= n) hh[i][j].x = 0.f;
          if (2 * j + 1 >= n) hh[i][j].y = 0.f;
          dnext[i][j] = fma2(v[i][j], hh[i][j], dnext[i][j]);
          v[i][j] = mul2(v[i][j], f2(g[2 * j], g[2 * j + 1]));
          s2 = fma2(v[i][j], hh[i][j], s2);
        }
      }
      const float m = sum(s2.x + s2.y) * inv_d;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        F2 x[N / 2];
        unpack_piece<T>(rx[i], x);
#pragma unroll
        for (int j = 0; j < N / 2; ++j)
          v[i][j] = fma2(fma2(hh[i][j], f2(-m), v[i][j]), f2(rho), x[j]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) unpack_piece<T>(rx[i], v[i]);
    }
    load(row + stride);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c_first + i * 32 * WPR * N;
      store_piece_of<FULL>(static_cast<T*>(p.dx) + row * p.lddx + c,
                           reinterpret_cast<const float(&)[N]>(v[i]), p.d - c, p.vec & kDxVec);
    }
    if (!block) continue;
    const float rho = p.post ? p.b_rstd[row] : 1.f;
    F2 s2 = f2(0.f);
    F2 bb[NV][N / 2];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c_first + i * 32 * WPR * N, n = p.d - c;
      float g[N];
      load_param<N, FULL>(p.post_gain, c, n, 1.f, g);
      const uint32_t bits = p.drop.threshold ? drop_bits<N>(p.drop, key, (uint32_t)row, c) : 0u;
      unpack_piece<T>(rb[i], bb[i]);
      F2 z[N / 2], dz[N / 2];
      if (gate) unpack_piece<T>(rz[i], z);
#pragma unroll
      for (int j = 0; j < N / 2; ++j) {
        bb[i][j] = mul2(bb[i][j], f2(rho));
        if (2 * j >= n) bb[i][j].x = 0.f;
        if (2 * j + 1 >= n) bb[i][j].y = 0.f;
        const F2 g2 = f2(g[2 * j], g[2 * j + 1]);
        F2 e = mul2(v[i][j], f2(p.scale));
        if (gate) {
          const F2 c2 = mul2(bb[i][j], g2);
          dz[j] = mul2(e, p.drop.threshold ? drop2(c2, bits, 2 * j, p.drop.scale) : c2);
          if (p.sigmoid) {
            F2 rest;
            z[j] = logistic2<T>(z[j], rest);
            dz[j] = mul2(dz[j], mul2(z[j], rest));
          }
          e = mul2(e, z[j]);
        }
        if (p.drop.threshold) e = drop2(e, bits, 2 * j, p.drop.scale);
        dpost[i][j] = fma2(e, bb[i][j], dpost[i][j]);
        v[i][j] = mul2(e, g2);
        s2 = fma2(v[i][j], bb[i][j], s2);
      }
      if (gate)
        store_piece_of<FULL>(static_cast<T*>(p.dz) + row * p.lddz + c,
                             reinterpret_cast<const float(&)[N]>(dz), n, p.vec & kDzVec);
    }
    float m = 0.f;
    if (p.post) m = sum(s2.x + s2.y) * inv_d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c_first + i * 32 * WPR * N;
#pragma unroll
      for (int j = 0; j < N / 2; ++j)
        if (p.post) v[i][j] = mul2(fma2(bb[i][j], f2(-m), v[i][j]), f2(rho));
      store_piece_of<FULL>(static_cast<T*>(p.db) + row * p.lddb + c,
                           reinterpret_cast<const float(&)[N]>(v[i]), p.d - c, p.vec & kDbVec);
    }
  }
  if (p.part) {
    // this block's partial sums, row slots added in order
    float* out = p.part + (long long)(WIDE ? blockIdx.x / cluster : blockIdx.x) * 2 * p.d;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      F2(&a)[NV][N / 2] = which ? dpost : dnext;
      if constexpr (ROWS > 1) {
        F2* sums = reinterpret_cast<F2*>(sums_mem) + t;  // value k at [k * 32 WPR]
        for (int k = 1; k < ROWS; ++k) {
          __syncthreads();
          if (slot == k)
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
              for (int j = 0; j < N / 2; ++j) sums[(i * N / 2 + j) * 32 * WPR] = a[i][j];
          __syncthreads();
          if (slot == 0)
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
              for (int j = 0; j < N / 2; ++j)
                a[i][j] = add2(a[i][j], sums[(i * N / 2 + j) * 32 * WPR]);
        }
      }
      if (slot == 0)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = c_first + i * 32 * WPR * N;
          float* o = out + (long long)which * p.d + c;
#pragma unroll
          for (int j = 0; j < N / 2; ++j) {
            if (c + 2 * j < p.d) o[2 * j] = a[i][j].x;
            if (c + 2 * j + 1 < p.d) o[2 * j + 1] = a[i][j].y;
          }
        }
    }
  }
  if constexpr (WIDE) ptx::cluster_sync();  // no block leaves while its sums may be read
}

// ------------------------------------------------------------ launches

// Blocks in clusters of `cluster` (1: none).
template <typename K>
mlp_status launch_rows(K* kernel, int blocks, int threads, int smem, int cluster, const ResNorm& p,
                       cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  cudaLaunchKernelEx(&cfg, kernel, p, cluster);
  return launch_status();
}

// The most partial rows of a backward launch (sizes its workspace, so it
// depends on the sizes alone).  Launches take as many of them as are resident.
constexpr int kBwdBlocks = 304;
int bwd_blocks(long long T, int d) {
  const int rows = d <= 512 ? 8 : d <= 1024 ? 4 : d <= 2048 ? 2 : 1;
  const long long need = (T + rows - 1) / rows;
  return (int)(need < kBwdBlocks ? need : kBwdBlocks);
}

template <typename T, int WPR, bool FULL, bool WIDE>
mlp_status fwd_of(const ResNorm& p, cudaStream_t st) {
  using B = HeldBlock<WPR>;
  auto kernel = resnorm_fwd_kernel<T, WPR, FULL, WIDE>;
  static PerDevice per_sm;
  const int cluster = WIDE ? (p.d + kHeldWidth - 1) / kHeldWidth : 1;
  int blocks = walk_blocks(kernel, B::THREADS, per_sm, WIDE ? 1ll << 40 : p.T, B::ROWS);
  if (WIDE) {
    blocks /= cluster;
    if (blocks < 1) blocks = 1;
    if (blocks > p.T) blocks = (int)p.T;
    blocks *= cluster;
  }
  LaunchScope ls("resnorm_fwd", st, p.T, p.d, sizeof(T));
  return launch_rows(kernel, blocks, B::THREADS, 0, cluster, p, st);
}

template <typename T, int WPR, bool FULL, bool WIDE>
mlp_status bwd_of(const ResNorm& p, int* rows, cudaStream_t st) {
  using B = HeldBlock<WPR>;
  auto kernel = resnorm_bwd_kernel<T, WPR, FULL, WIDE>;
  static PerDevice per_sm;
  const int cluster = WIDE ? (p.d + kHeldWidth - 1) / kHeldWidth : 1;
  int resident = walk_blocks(kernel, B::THREADS, per_sm, WIDE ? 1ll << 40 : p.T, B::ROWS);
  if (WIDE) resident = resident / cluster > 0 ? resident / cluster : 1;
  if (resident < *rows) *rows = resident;
  const size_t smem = B::ROWS > 1 && p.part ? (size_t)32 * WPR * kPerThread * 4 : 0;
  LaunchScope ls("resnorm_bwd", st, p.T, p.d, sizeof(T));
  return launch_rows(kernel, *rows * cluster, B::THREADS, (int)smem, cluster, p, st);
}

template <typename T, int WPR, bool WIDE, bool BWD>
mlp_status of_form(const ResNorm& p, bool full, int* rows, cudaStream_t st) {
  if constexpr (BWD)
    return full ? bwd_of<T, WPR, true, WIDE>(p, rows, st) : bwd_of<T, WPR, false, WIDE>(p, rows, st);
  else
    return full ? fwd_of<T, WPR, true, WIDE>(p, st) : fwd_of<T, WPR, false, WIDE>(p, st);
}

template <typename T, bool BWD>
mlp_status of_type(ResNorm p, int* rows, cudaStream_t st) {
  p.vec = 0;
  bool full = p.d % RowVec<T>::N == 0;
  auto look = [&](const void* m, long long ld, int bit) {
    if (!m) return;
    if (row_vec(m, ld, sizeof(T), 16)) p.vec |= bit;
    else full = false;
  };
  look(p.x, p.ldx, kXVec);
  look(p.b, p.ldb, kBVec);
  look(p.z, p.ldz, kZVec);
  look(p.h, p.ldh, kHVec);
  look(p.n, p.ldn, kNVec);
  if (BWD) {
    look(p.dx, p.lddx, kDxVec);
    look(p.db, p.lddb, kDbVec);
    look(p.dz, p.lddz, kDzVec);
  }
  if (p.d <= 512) return of_form<T, 1, false, BWD>(p, full, rows, st);
  if (p.d <= 1024) return of_form<T, 2, false, BWD>(p, full, rows, st);
  if (p.d <= 2048) return of_form<T, 4, false, BWD>(p, full, rows, st);
  if (p.d <= 4096) return of_form<T, 8, false, BWD>(p, full, rows, st);
  if (p.d <= kHeldWidth) return of_form<T, 16, false, BWD>(p, full, rows, st);
  return of_form<T, 16, true, BWD>(p, full, rows, st);
}

template <bool BWD>
mlp_status of_any(const ResNorm& p, int* rows, cudaStream_t st) {
  switch (p.dtype) {
    case MLP_DTYPE_BF16: return of_type<__nv_bfloat16, BWD>(p, rows, st);
    case MLP_DTYPE_F16: return of_type<__half, BWD>(p, rows, st);
    default: return of_type<float, BWD>(p, rows, st);
  }
}

}  // namespace

size_t resnorm_ws_bytes(long long T, int d) {
  return (size_t)bwd_blocks(T, d) * 2 * d * sizeof(float);
}

mlp_status launch_resnorm_fwd(const ResNorm& a, cudaStream_t st) {
  return of_any<false>(a, nullptr, st);
}

mlp_status launch_resnorm_bwd(const ResNorm& a, float* dnext_gain, float* dpost_gain,
                              cudaStream_t st) {
  int rows = bwd_blocks(a.T, a.d);
  MLP_CHECK(of_any<true>(a, &rows, st));
  const long long ld = 2ll * a.d;
  if (dnext_gain && dpost_gain)
    return launch_partial_sums(a.part, rows, 2 * a.d, ld, dnext_gain, a.d, dpost_gain, st);
  if (dnext_gain)
    return launch_partial_sums(a.part, rows, a.d, ld, dnext_gain, a.d, nullptr, st);
  if (dpost_gain)
    return launch_partial_sums(a.part + a.d, rows, a.d, ld, dpost_gain, a.d, nullptr, st);
  return MLP_OK;
}

}  // namespace mlp
