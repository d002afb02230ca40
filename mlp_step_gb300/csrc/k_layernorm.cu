// Layer norm over the rows of a matrix, forward and backward.
//   mu = mean_i x_i,  rho = 1 / sqrt(mean_i (x_i - mu)^2 + eps)
//   xh = (x - mu) rho,  y = xh gain + shift
//   g = dy gain,  dx = rho (g - mean(g) - xh mean(g xh)) + dres
//   dgain = sum_t dy xh,  dshift = sum_t dy
// All of it is bound by HBM (forward 4, backward 6 to 8 bytes per bf16 value),
// so a row is read once and stays in registers between its reductions: the
// variance is taken about the mean that was just found (two passes over
// registers), not as a difference of moments, which would cancel for rows
// whose mean is large against their spread.  Everything between load and
// store is fp32.
//
// A row is held by WPR warps, 16 values per thread (two 16-byte pieces in 16
// bits, four in fp32), piece i at column (i * 32 WPR + thread) * N: every load
// of a warp is one contiguous run and a group of 32 values for the 8-bit form
// is 4 (8) neighbouring lanes.  Blocks walk over rows with a grid stride; the
// next row's loads are issued before this row's reductions.
// Measured: 65,536 x 512 bf16 with the 8-bit form of x written 35 us forward,
// read 49 us backward (4.8 TB/s both); 16,384 x 8,192 fp16 117 us and 157 us
// (4.6 and 5.1 TB/s: the block-wide reductions of a row, two barriers forward,
// are not hidden by the one other block that an SM's registers hold).
#include "ckpt8.cuh"
#include "kernels.cuh"
#include "rowvec.cuh"
#include "trace.cuh"

namespace mlp {

namespace {

constexpr int kPerThread = 16;        // values of a row per thread
constexpr int kHeldWidth = 16 * 512;  // widest row held by one block's registers
constexpr int kLoopThreads = 512;

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

// The 8-bit form of a piece at column c of a row (its group's lanes together).
template <typename T, bool FULL = false>
__device__ __forceinline__ void store_ckpt(const float (&v)[RowVec<T>::N], int8_t* qrow,
                                           uint8_t* srow, int c, int n, bool vec) {
  constexpr int N = RowVec<T>::N, LANES = kCkptGroup / N;
  uint32_t amax = amax_bits_of(v);
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1)
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  uint32_t w[N / 4];
  const uint32_t b = ckpt8_piece(v, amax, w);
  if (n > 0) {
    store_q<N, FULL>(qrow + c, n, vec, w);
    if ((threadIdx.x & (LANES - 1)) == 0) srow[c / kCkptGroup] = (uint8_t)b;
  }
}

// ------------------------------------------------------------ forward

// Registers: 64 per thread (128 for fp32 rows, whose pieces are twice as many)
// keep 32 (16) warps on an SM, each with its next row in flight.
template <typename T, int WPR, bool FULL>
__global__ void __launch_bounds__(HeldBlock<WPR>::THREADS,
                                  (sizeof(T) == 2 ? 1024 : 512) / HeldBlock<WPR>::THREADS)
    ln_fwd_kernel(const LayerNormFwd p) {
  constexpr int N = RowVec<T>::N, NV = kPerThread / N, ROWS = HeldBlock<WPR>::ROWS;
  __shared__ float part[2][ROWS][WPR];
  pdl_wait();
  pdl_launch_dependents();
  const int slot = threadIdx.x / (32 * WPR), t = threadIdx.x % (32 * WPR);
  const long long stride = (long long)gridDim.x * ROWS;
  long long row = (long long)blockIdx.x * ROWS + slot;
  const float inv_d = 1.f / (float)p.d;
  const T* x = static_cast<const T*>(p.x);
  uint4 raw[NV];
  auto load = [&](long long r) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * 32 * WPR + t) * N;
      raw[i] = load_piece_of<FULL>(x + r * p.ldx + c, r < p.T ? p.d - c : 0, p.x_vec);
    }
  };
  load(row);
  for (; row < p.T; row += stride) {  // uniform over the warps that share a row
    F2 v[NV][N / 2];
    F2 s2 = f2(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      unpack_piece<T>(raw[i], v[i]);
#pragma unroll
      for (int j = 0; j < N / 2; ++j) s2 = add2(s2, v[i][j]);
    }
    load(row + stride);
    float s[1] = {s2.x + s2.y};
    row_sums<WPR>(s, part[0][slot], slot, t >> 5);
    const float mu = s[0] * inv_d;
    s2 = f2(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int n = p.d - (i * 32 * WPR + t) * N;
      if (FULL ? n > 0 : n >= N) {
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          const F2 c = add2(v[i][j], f2(-mu));
          s2 = fma2(c, c, s2);
        }
      } else if (!FULL) {
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          const float c0 = 2 * j < n ? v[i][j].x - mu : 0.f;
          const float c1 = 2 * j + 1 < n ? v[i][j].y - mu : 0.f;
          s2 = fma2(f2(c0, c1), f2(c0, c1), s2);
        }
      }
    }
    s[0] = s2.x + s2.y;
    row_sums<WPR>(s, part[1][slot], slot, t >> 5);
    const float rho = rsqrtf(s[0] * inv_d + p.eps);  // two ulp
    if (t == 0) {
      if (p.mean) p.mean[row] = mu;
      if (p.rstd) p.rstd[row] = rho;
    }
    T* y = static_cast<T*>(p.y) + row * p.ldy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * 32 * WPR + t) * N;
      const int n = p.d - c;
      if (p.q)
        store_ckpt<T, FULL>(reinterpret_cast<const float(&)[N]>(v[i]), p.q + row * p.ldq,
                            p.scale + row * p.lds, c, n, p.q_vec);
      float a[N], b[N];
      load_param<N, FULL>(p.gain, c, n, 1.f, a);
      load_param<N, FULL>(p.shift, c, n, 0.f, b);
#pragma unroll
      for (int j = 0; j < N / 2; ++j)
        v[i][j] = fma2(mul2(add2(v[i][j], f2(-mu)), f2(rho)), f2(a[2 * j], a[2 * j + 1]),
                       f2(b[2 * j], b[2 * j + 1]));
      store_piece_of<FULL>(y + c, reinterpret_cast<const float(&)[N]>(v[i]), n, p.y_vec);
    }
  }
}

// Rows wider than the registers of a block: one block per row, which reads the
// row three times (the second and third mostly from L1 and L2): 4,096 x 16,384
// fp32 107 us, 5.0 TB/s of one read and one write.
template <typename T>
__global__ void __launch_bounds__(kLoopThreads) ln_fwd_wide_kernel(const LayerNormFwd p) {
  constexpr int N = RowVec<T>::N, WPR = kLoopThreads / 32;
  __shared__ float part[2][WPR];
  pdl_wait();
  pdl_launch_dependents();
  const int t = threadIdx.x;
  const float inv_d = 1.f / (float)p.d;
  // whole warps walk together past the row's end, so that group shuffles are full
  const int end = (p.d + 32 * N - 1) / (32 * N) * (32 * N);
  for (long long row = blockIdx.x; row < p.T; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    float s[1] = {0.f};
    for (int c = t * N; c < p.d; c += kLoopThreads * N) {
      float v[N];
      unpack_piece<T>(load_piece(x + c, p.d - c, p.x_vec), v);
#pragma unroll
      for (int j = 0; j < N; ++j) s[0] += v[j];
    }
    row_sums<WPR>(s, part[0], 0, t >> 5);
    const float mu = s[0] * inv_d;
    s[0] = 0.f;
    for (int c = t * N; c < p.d; c += kLoopThreads * N) {
      float v[N];
      unpack_piece<T>(load_piece(x + c, p.d - c, p.x_vec), v);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float e = c + j < p.d ? v[j] - mu : 0.f;
        s[0] = fmaf(e, e, s[0]);
      }
    }
    row_sums<WPR>(s, part[1], 0, t >> 5);
    const float rho = rsqrtf(s[0] * inv_d + p.eps);  // two ulp
    if (t == 0) {
      if (p.mean) p.mean[row] = mu;
      if (p.rstd) p.rstd[row] = rho;
    }
    for (int c = t * N; c < end; c += kLoopThreads * N) {
      const int n = p.d - c;
      float v[N], a[N], b[N];
      unpack_piece<T>(load_piece(x + c, n, p.x_vec), v);
      if (p.q) store_ckpt<T>(v, p.q + row * p.ldq, p.scale + row * p.lds, c, n, p.q_vec);
      load_param<N>(p.gain, c, n, 1.f, a);
      load_param<N>(p.shift, c, n, 0.f, b);
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = fmaf((v[j] - mu) * rho, a[j], b[j]);
      store_piece(static_cast<T*>(p.y) + row * p.ldy + c, v, n, p.y_vec);
    }
  }
}

// ------------------------------------------------------------ backward

// A piece of the forward's input: its raw 16 bytes, or the 8-bit words and the
// group's scale byte.
template <typename T, bool CK, bool FULL = false>
struct XPiece {
  static constexpr int N = RowVec<T>::N;
  uint4 raw;
  uint32_t w[N / 4], b;
  __device__ __forceinline__ void load(const LayerNormBwd& p, long long row, int c, int n) {
    if constexpr (CK) {
      load_q<N, FULL>(p.q + row * p.ldq + c, n, p.q_vec, w);
      b = n > 0 ? p.scale[row * p.lds + c / kCkptGroup] : 0u;
    } else {
      raw = load_piece_of<FULL>(static_cast<const T*>(p.x) + row * p.ldx + c, n, p.x_vec);
    }
  }
  __device__ __forceinline__ void values(F2 (&v)[N / 2]) const {
    if constexpr (CK) {
      const float step = ckpt8_step(b);
#pragma unroll
      for (int k = 0; k < N / 4; ++k) {
        const uint32_t f = ckpt8_flip(w[k]);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          v[2 * k + e] = mul2(add2(f2(ckpt8_biased(f, 2 * e), ckpt8_biased(f, 2 * e + 1)),
                                   f2(-kCkptBias)),
                              f2(step));
      }
    } else {
      unpack_piece<T>(raw, v);
    }
  }
  __device__ __forceinline__ void values(float (&v)[N]) const {
    if constexpr (CK) {
      const float step = ckpt8_step(b);
#pragma unroll
      for (int k = 0; k < N / 4; ++k) {
        const uint32_t f = ckpt8_flip(w[k]);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * k + e] = ckpt8_value(f, e, step);
      }
    } else {
      unpack_piece<T>(raw, v);
    }
  }
};

// Per row: s1 = sum g, s2 = sum g xh, then dx; the sums of dy xh and dy over
// the block's rows stay in registers (each thread always has the same
// columns), are added over the block's row slots in order at the end, and
// leave as one row of partial sums per block: no atomics, so the gradients
// are the same in every run.
template <typename T, int WPR, bool CK, bool FULL>
__global__ void __launch_bounds__(HeldBlock<WPR>::THREADS,
                                  sizeof(T) == 2 ? 512 / HeldBlock<WPR>::THREADS : 1)
    ln_bwd_kernel(const LayerNormBwd p) {
  constexpr int N = RowVec<T>::N, NV = kPerThread / N, ROWS = HeldBlock<WPR>::ROWS;
  __shared__ float part[2][ROWS][2 * WPR];
  extern __shared__ __align__(16) float sums_mem[];  // ROWS > 1: one slot's values at a time
  pdl_wait();
  pdl_launch_dependents();
  const int slot = threadIdx.x / (32 * WPR), t = threadIdx.x % (32 * WPR);
  const long long stride = (long long)gridDim.x * ROWS;
  long long row = (long long)blockIdx.x * ROWS + slot;
  const float inv_d = 1.f / (float)p.d;
  const T* dy = static_cast<const T*>(p.dy);
  const T* dres = static_cast<const T*>(p.dres);
  F2 dg[NV][N / 2], ds[NV][N / 2];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < N / 2; ++j) dg[i][j] = ds[i][j] = f2(0.f);
  uint4 rdy[NV];
  XPiece<T, CK, FULL> rx[NV];
  float mu_n = 0.f, rho_n = 0.f;
  auto load = [&](long long r) {
    const bool in = r < p.T;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * 32 * WPR + t) * N;
      const int n = in ? p.d - c : 0;
      rdy[i] = load_piece_of<FULL>(dy + r * p.lddy + c, n, p.dy_vec);
      rx[i].load(p, r, c, n);
    }
    if (in) {
      mu_n = p.mean[r];
      rho_n = p.rstd[r];
    }
  };
  load(row);
  int turn = 0;
  for (; row < p.T; row += stride, turn ^= 1) {
    const float mu = mu_n, rho = rho_n;
    F2 g[NV][N / 2], xh[NV][N / 2];
    F2 s1 = f2(0.f), s2 = f2(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * 32 * WPR + t) * N, n = p.d - c;
      float gain[N];  // from L1: as registers they would cost a block per SM
      load_param<N, FULL>(p.gain, c, n, 1.f, gain);
      unpack_piece<T>(rdy[i], g[i]);
      rx[i].values(xh[i]);
#pragma unroll
      for (int j = 0; j < N / 2; ++j) xh[i][j] = mul2(add2(xh[i][j], f2(-mu)), f2(rho));
      // past the row's end xh is set to 0 (dy reads as 0 there, but 0 times a
      // mean or scale that is not finite would not be)
      if (FULL ? n <= 0 : n < N) {
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          if (FULL || 2 * j >= n) xh[i][j].x = 0.f;
          if (FULL || 2 * j + 1 >= n) xh[i][j].y = 0.f;
        }
      }
#pragma unroll
      for (int j = 0; j < N / 2; ++j) {
        dg[i][j] = fma2(g[i][j], xh[i][j], dg[i][j]);
        ds[i][j] = add2(ds[i][j], g[i][j]);
        g[i][j] = mul2(g[i][j], f2(gain[2 * j], gain[2 * j + 1]));
        s1 = add2(s1, g[i][j]);
        s2 = fma2(g[i][j], xh[i][j], s2);
      }
    }
    uint4 rr[NV];  // this row's residual gradient, in flight over the reductions
    if (dres) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * 32 * WPR + t) * N;
        rr[i] = load_piece_of<FULL>(dres + row * p.ldr + c, p.d - c, p.r_vec);
      }
    }
    load(row + stride);
    float s[2] = {s1.x + s1.y, s2.x + s2.y};
    row_sums<WPR>(s, part[turn][slot], slot, t >> 5);
    const float m1 = s[0] * inv_d, m2 = s[1] * inv_d;
    T* dx = static_cast<T*>(p.dx) + row * p.lddx;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * 32 * WPR + t) * N;
      // rho (g - (m1 + xh m2))
#pragma unroll
      for (int j = 0; j < N / 2; ++j)
        g[i][j] = mul2(add2(g[i][j], fma2(xh[i][j], f2(-m2), f2(-m1))), f2(rho));
      if (dres) {
        F2 r[N / 2];
        unpack_piece<T>(rr[i], r);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) g[i][j] = add2(g[i][j], r[j]);
      }
      store_piece_of<FULL>(dx + c, reinterpret_cast<const float(&)[N]>(g[i]), p.d - c, p.dx_vec);
    }
  }
  // this block's partial sums, row slots added in order
  float* out = p.part + (long long)blockIdx.x * 2 * p.d;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    F2(&a)[NV][N / 2] = which ? ds : dg;
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
        const int c = (i * 32 * WPR + t) * N;
        float* o = out + (long long)which * p.d + c;
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          if (FULL ? c < p.d : c + 2 * j < p.d) o[2 * j] = a[i][j].x;
          if (FULL ? c < p.d : c + 2 * j + 1 < p.d) o[2 * j + 1] = a[i][j].y;
        }
      }
  }
}

// Wide rows, dx: one block per row, dy and x read twice (4,096 x 16,384 fp32
// 172 us, 4.7 TB/s of two reads and one write).
template <typename T, bool CK>
__global__ void __launch_bounds__(kLoopThreads) ln_bwd_wide_kernel(const LayerNormBwd p) {
  constexpr int N = RowVec<T>::N, WPR = kLoopThreads / 32;
  __shared__ float part[2][2 * WPR];
  pdl_wait();
  pdl_launch_dependents();
  const int t = threadIdx.x;
  const float inv_d = 1.f / (float)p.d;
  int turn = 0;
  for (long long row = blockIdx.x; row < p.T; row += gridDim.x, turn ^= 1) {
    const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
    const float mu = p.mean[row], rho = p.rstd[row];
    float s[2] = {0.f, 0.f};
    auto piece = [&](int c, float(&g)[N], float(&xh)[N]) {
      XPiece<T, CK> x;
      float gain[N];
      x.load(p, row, c, p.d - c);
      x.values(xh);
      unpack_piece<T>(load_piece(dy + c, p.d - c, p.dy_vec), g);
      load_param<N>(p.gain, c, p.d - c, 1.f, gain);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        xh[j] = c + j < p.d ? (xh[j] - mu) * rho : 0.f;
        g[j] *= gain[j];
      }
    };
    for (int c = t * N; c < p.d; c += kLoopThreads * N) {
      float g[N], xh[N];
      piece(c, g, xh);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        s[0] += g[j];
        s[1] = fmaf(g[j], xh[j], s[1]);
      }
    }
    row_sums<WPR>(s, part[turn], 0, t >> 5);
    const float m1 = s[0] * inv_d, m2 = s[1] * inv_d;
    for (int c = t * N; c < p.d; c += kLoopThreads * N) {
      float g[N], xh[N];
      piece(c, g, xh);
#pragma unroll
      for (int j = 0; j < N; ++j) g[j] = rho * (g[j] - fmaf(xh[j], m2, m1));
      if (p.dres) {
        float r[N];
        unpack_piece<T>(
            load_piece(static_cast<const T*>(p.dres) + row * p.ldr + c, p.d - c, p.r_vec), r);
#pragma unroll
        for (int j = 0; j < N; ++j) g[j] += r[j];
      }
      store_piece(static_cast<T*>(p.dx) + row * p.lddx + c, g, p.d - c, p.dx_vec);
    }
  }
}

// Wide rows, partial sums of dy xh and dy: block (x, y) adds rows y, y + chunks,
// ... of its 256-piece stripe of columns (4,096 x 16,384 fp32 94 us, 5.7 TB/s).
template <typename T, bool CK>
__global__ void __launch_bounds__(256) ln_bwd_wide_sums_kernel(const LayerNormBwd p) {
  constexpr int N = RowVec<T>::N;
  pdl_wait();
  pdl_launch_dependents();
  const int c = (blockIdx.x * 256 + threadIdx.x) * N;
  if (c >= p.d) return;
  float dg[N], ds[N];
#pragma unroll
  for (int j = 0; j < N; ++j) dg[j] = ds[j] = 0.f;
#pragma unroll 4
  for (long long row = blockIdx.y; row < p.T; row += gridDim.y) {
    XPiece<T, CK> x;
    float g[N], xh[N];
    x.load(p, row, c, p.d - c);
    x.values(xh);
    unpack_piece<T>(
        load_piece(static_cast<const T*>(p.dy) + row * p.lddy + c, p.d - c, p.dy_vec), g);
    const float mu = p.mean[row], rho = p.rstd[row];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      dg[j] = fmaf(g[j], (xh[j] - mu) * rho, dg[j]);
      ds[j] += g[j];
    }
  }
  float* out = p.part + (long long)blockIdx.y * 2 * p.d;
#pragma unroll
  for (int j = 0; j < N; ++j)
    if (c + j < p.d) {
      out[c + j] = dg[j];
      out[p.d + c + j] = ds[j];
    }
}

// ------------------------------------------------------------ launches

bool row_vec(const void* p, long long ld, int esz, int bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * esz % bytes == 0;
}

// Blocks of a row-walking launch: as many as are resident at once (more would
// run as a second, ragged wave), at most one per row set.
template <typename K>
int walk_blocks(K kernel, int threads, PerDevice& resident, long long T, int rows_per_block) {
  const int per_sm = resident.get(current_device(), [&] {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0) != cudaSuccess) {
      cudaGetLastError();
      n = 1;
    }
    return n > 0 ? n : 1;
  });
  const long long need = (T + rows_per_block - 1) / rows_per_block;
  const long long most = (long long)num_sms() * per_sm;
  return (int)(need < most ? need : most);
}

template <typename T, int WPR, bool FULL>
mlp_status fwd_held_of(const LayerNormFwd& p, cudaStream_t st) {
  using B = HeldBlock<WPR>;
  static PerDevice per_sm;
  const int blocks = walk_blocks(ln_fwd_kernel<T, WPR, FULL>, B::THREADS, per_sm, p.T, B::ROWS);
  launch_k(ln_fwd_kernel<T, WPR, FULL>, dim3(blocks), dim3(B::THREADS), 0, st, p);
  return launch_status();
}

template <typename T, int WPR>
mlp_status fwd_held(const LayerNormFwd& p, cudaStream_t st) {
  const bool full = p.d % RowVec<T>::N == 0 && p.x_vec && p.y_vec && (!p.q || p.q_vec);
  return full ? fwd_held_of<T, WPR, true>(p, st) : fwd_held_of<T, WPR, false>(p, st);
}

template <typename T>
mlp_status fwd_t(LayerNormFwd p, cudaStream_t st) {
  p.x_vec = row_vec(p.x, p.ldx, sizeof(T), 16);
  p.y_vec = row_vec(p.y, p.ldy, sizeof(T), 16);
  p.q_vec = p.q && row_vec(p.q, p.ldq, 1, RowVec<T>::N);
  LaunchScope ls("layernorm_fwd", st, p.T, p.d, sizeof(T));
  if (p.d <= 512) return fwd_held<T, 1>(p, st);
  if (p.d <= 1024) return fwd_held<T, 2>(p, st);
  if (p.d <= 2048) return fwd_held<T, 4>(p, st);
  if (p.d <= 4096) return fwd_held<T, 8>(p, st);
  if (p.d <= kHeldWidth) return fwd_held<T, 16>(p, st);
  static PerDevice per_sm;
  const int blocks = walk_blocks(ln_fwd_wide_kernel<T>, kLoopThreads, per_sm, p.T, 1);
  launch_k(ln_fwd_wide_kernel<T>, dim3(blocks), dim3(kLoopThreads), 0, st, p);
  return launch_status();
}

// The most partial rows of a backward launch (sizes its workspace, so it
// depends on the sizes alone): 304 blocks of 256 threads are two per SM, all
// that the registers hold.  Launches take as many of them as are resident.
constexpr int kBwdBlocks = 304;
int bwd_blocks(long long T, int d) {
  // (wide rows: eight rows to a partial row, so that few rows do not leave more
  // partial sums than they are: 380 x 10,480 bf16 takes 33 us for the sums with
  // a row each, 14 with eight)
  const int rows = d <= 512 || d > kHeldWidth ? 8 : d <= 1024 ? 4 : d <= 2048 ? 2 : 1;
  const long long need = (T + rows - 1) / rows;
  return (int)(need < kBwdBlocks ? need : kBwdBlocks);
}

template <typename T, int WPR, bool CK, bool FULL>
mlp_status bwd_held_of(const LayerNormBwd& p, int* blocks, cudaStream_t st) {
  using B = HeldBlock<WPR>;
  static PerDevice per_sm;
  const int resident =
      walk_blocks(ln_bwd_kernel<T, WPR, CK, FULL>, B::THREADS, per_sm, p.T, B::ROWS);
  if (resident < *blocks) *blocks = resident;
  const size_t smem = B::ROWS > 1 ? (size_t)32 * WPR * kPerThread * 4 : 0;
  LaunchScope ls("layernorm_bwd", st, p.T, p.d, sizeof(T));
  launch_k(ln_bwd_kernel<T, WPR, CK, FULL>, dim3(*blocks), dim3(B::THREADS), smem, st, p);
  return launch_status();
}

template <typename T, int WPR, bool CK>
mlp_status bwd_held(const LayerNormBwd& p, int* blocks, cudaStream_t st) {
  const bool full = p.d % RowVec<T>::N == 0 && p.dy_vec && p.dx_vec &&
                    (!p.dres || p.r_vec) && (CK ? p.q_vec : p.x_vec);
  return full ? bwd_held_of<T, WPR, CK, true>(p, blocks, st)
              : bwd_held_of<T, WPR, CK, false>(p, blocks, st);
}

template <typename T, bool CK>
mlp_status bwd_t(LayerNormBwd p, cudaStream_t st) {
  p.dy_vec = row_vec(p.dy, p.lddy, sizeof(T), 16);
  p.x_vec = CK ? 0 : row_vec(p.x, p.ldx, sizeof(T), 16);
  p.q_vec = CK ? row_vec(p.q, p.ldq, 1, RowVec<T>::N) : 0;
  p.r_vec = row_vec(p.dres, p.ldr, sizeof(T), 16);
  p.dx_vec = row_vec(p.dx, p.lddx, sizeof(T), 16);
  int blocks = bwd_blocks(p.T, p.d);
  if (p.d <= 512) MLP_CHECK((bwd_held<T, 1, CK>(p, &blocks, st)));
  else if (p.d <= 1024) MLP_CHECK((bwd_held<T, 2, CK>(p, &blocks, st)));
  else if (p.d <= 2048) MLP_CHECK((bwd_held<T, 4, CK>(p, &blocks, st)));
  else if (p.d <= 4096) MLP_CHECK((bwd_held<T, 8, CK>(p, &blocks, st)));
  else if (p.d <= kHeldWidth) MLP_CHECK((bwd_held<T, 16, CK>(p, &blocks, st)));
  else {
    // the sums first: they read dy once more, which dx may overwrite
    {
      LaunchScope ls("layernorm_bwd_wide_sums", st, p.T, p.d, sizeof(T));
      const int stripe = 256 * RowVec<T>::N;
      launch_k(ln_bwd_wide_sums_kernel<T, CK>, dim3((p.d + stripe - 1) / stripe, blocks),
               dim3(256), 0, st, p);
      MLP_CHECK(launch_status());
    }
    LaunchScope ls("layernorm_bwd_wide", st, p.T, p.d, sizeof(T));
    static PerDevice per_sm;
    launch_k(ln_bwd_wide_kernel<T, CK>,
             dim3(walk_blocks(ln_bwd_wide_kernel<T, CK>, kLoopThreads, per_sm, p.T, 1)),
             dim3(kLoopThreads), 0, st, p);
    MLP_CHECK(launch_status());
  }
  return launch_partial_sums(p.part, blocks, 2 * p.d, 2 * p.d, p.dgain, p.d, p.dshift, st);
}

template <typename T>
mlp_status bwd_ck(const LayerNormBwd& p, cudaStream_t st) {
  return p.q ? bwd_t<T, true>(p, st) : bwd_t<T, false>(p, st);
}

}  // namespace

size_t layernorm_ws_bytes(long long T, int d) {
  return (size_t)bwd_blocks(T, d) * 2 * d * sizeof(float);
}

mlp_status launch_layernorm_fwd(const LayerNormFwd& a, cudaStream_t st) {
  switch (a.dtype) {
    case MLP_DTYPE_BF16: return fwd_t<__nv_bfloat16>(a, st);
    case MLP_DTYPE_F16: return fwd_t<__half>(a, st);
    default: return fwd_t<float>(a, st);
  }
}

mlp_status launch_layernorm_bwd(const LayerNormBwd& a, cudaStream_t st) {
  switch (a.dtype) {
    case MLP_DTYPE_BF16: return bwd_ck<__nv_bfloat16>(a, st);
    case MLP_DTYPE_F16: return bwd_ck<__half>(a, st);
    default: return bwd_ck<float>(a, st);
  }
}

}  // namespace mlp
