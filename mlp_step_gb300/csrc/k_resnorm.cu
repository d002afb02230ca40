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
// A row is held by WPR warps, two 16-byte pieces per thread as in k_layernorm.cu;
// rows wider than a block holds (8,192) are held by a cluster of up to eight
// blocks, whose sums meet in distributed shared memory, so they too are read once.
// The next row is on its way to shared memory while this one is worked on.
// Parameter gradients stay in registers over a block's rows and leave as one
// row of partial sums per block (cluster): no atomics, the same in every run.
// Measured with events, launches back to back, the backward with its sums' launch:
// 65,536 x 512 bf16 with both norms, gate and dropout 57 us forward and 97
// backward (5.8 and 5.5 TB/s; with rows loaded to registers 63 and 173); 16,384 x
// 8,192 fp16 without gate and dropout 170 and 319 (6.3 and 5.0 TB/s; 226 and 483):
// the backward's one block an SM waits at two block-wide sums a row.
#include <cfloat>

#include "act.cuh"
#include "few_rows.cuh"
#include "kernels.cuh"
#include "norm_rows.cuh"
#include "philox.cuh"
#include "rowvec.cuh"
#include "trace.cuh"

namespace mlp {

namespace {

constexpr int kBlockWidth = 8192;  // widest row held by one block
constexpr int kMaxCluster = 8;

// Values of a row per thread: two 16-byte pieces.
template <typename T>
constexpr int vpt() {
  return 2 * RowVec<T>::N;
}

// Bits of ResNorm::vec: 16-byte pieces of that matrix's rows are aligned.
enum { kXVec = 1, kBVec = 2, kZVec = 4, kHVec = 8, kNVec = 16, kDxVec = 32, kDbVec = 64,
       kDzVec = 128 };

// What the blocks of a cluster exchange for a row's sum: each sends its own to
// every block's `in` (asynchronous stores, counted in bytes by the receiver's
// barrier) and waits for all.  Nothing else is ordered by it, where a cluster
// barrier would wait for the row's stores.  Two turns: a block sends for a turn
// again only after the other turn's sums arrived, which were sent after all
// threads had read this one's.
struct Exchange {
  float in[2][kMaxCluster];
  unsigned long long full[2];
};

__device__ __forceinline__ void send_f32(uint32_t to, float v, uint32_t bar) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(to),
      "r"(__float_as_uint(v)), "r"(bar)
      : "memory");
}

// Sums of one value over the row: over a block's warps, then (WIDE) over the
// cluster's blocks in rank order.  Callers' turns alternate, so that one barrier
// a call (each) is enough.  A wait that runs out is recorded, and no more are
// begun: the rows are then finished with what is there.
template <int WPR, bool WIDE, int ROWS>
struct RowSum {
  float (*part)[ROWS][WPR];  // [2][ROWS][WPR]
  Exchange* ex;              // WIDE: in this block's shared memory
  int slot, warp_in_row, rank, cluster;
  unsigned long long wait_ns;
  int* err;
  int turn = 0;
  uint32_t phase = 0;  // of this turn's barrier
  bool dead = false;
  __device__ __forceinline__ float operator()(float v) {
    float s[1] = {v};
    row_sums<WPR>(s, part[turn][slot], slot, warp_in_row);
    if constexpr (WIDE) {
      uint64_t* bar = reinterpret_cast<uint64_t*>(&ex->full[turn]);
      if (threadIdx.x == 0) ptx::mbar_arrive_expect_tx(bar, (uint32_t)cluster * 4u);
      if (threadIdx.x < 32 && (int)threadIdx.x < cluster)
        send_f32(ptx::mapa_shared(ptx::smem_u32(&ex->in[turn][rank]), threadIdx.x), s[0],
                 ptx::mapa_shared(ptx::smem_u32(bar), threadIdx.x));
      if (!dead)
        dead = !ptx::mbar_wait_cluster_bounded(bar, phase, wait_ns, err, DEVERR_TIMEOUT_PEER);
      s[0] = 0.f;
      for (int r = 0; r < cluster; ++r) s[0] += ex->in[turn][r];
      if (turn) phase ^= 1;
    }
    turn ^= 1;
    return s[0];
  }
  __device__ __forceinline__ void begin() {
    if constexpr (WIDE) {
      if (threadIdx.x == 0) {
        ptx::mbar_init(reinterpret_cast<uint64_t*>(&ex->full[0]), 1);
        ptx::mbar_init(reinterpret_cast<uint64_t*>(&ex->full[1]), 1);
        ptx::fence_mbar_init();
      }
      ptx::cluster_sync();
    }
  }
};

// The logistic function s of two values, and what s' is s times: 1 - s =
// e^(-z) s, which keeps its precision where s is near 1 and is 1 where s is tiny,
// as far as s is not 0: it reads as 0 once e^(-z) is past 2^126 (z below -87.3).
// An infinite e^(-z) is held to the largest finite value, which s makes 0.  The
// accurate functions for fp32 rows.
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
  one_minus = mul2(f2(fminf(e.x, FLT_MAX), fminf(e.y, FLT_MAX)), s);
  return s;
}

// A thread's pieces of the rows ahead, in shared memory: `mats` matrices (those
// that the call has: what the ring leaves is L1, where the gains are kept),
// AHEAD + 1 rows, each 16-byte piece at a place of its own that this thread alone
// fills (asynchronous copies) and reads.  So what is in flight takes no registers
// and no barrier.
template <typename T, int AHEAD, int THREADS>
struct Ring {
  static constexpr int NV = vpt<T>() / RowVec<T>::N;
  static constexpr int bytes(int mats) { return mats * (AHEAD + 1) * NV * THREADS * 16; }
  uint4* mine;
  int mats;
  int stage;  // of the current row
  __device__ __forceinline__ uint4* at(int s, int m, int i) const {
    return mine + ((s * mats + m) * NV + i) * THREADS;
  }
  // piece i of matrix m of the current row
  __device__ __forceinline__ uint4 operator()(int m, int i) const { return *at(stage, m, i); }
  // Zeros in a piece that no row has, which no copy writes.
  __device__ __forceinline__ void clear(int i) const {
    for (int m = 0; m < mats * (AHEAD + 1); ++m) *at(0, m, i) = make_uint4(0, 0, 0, 0);
  }
};

// Piece of n values at p into its place: asynchronously in 16 bytes, for fp32 rows
// that start anywhere in 4 (10,007 x 1,001 fp32 forward 66 us, 99 with loads and
// stores of the thread's own), else by the thread.
template <typename T, bool FULL>
__device__ __forceinline__ void issue_piece(uint4* place, const T* p, int n, bool vec) {
  if constexpr (FULL) {
    n = RowVec<T>::N;
    vec = true;
  }
  if constexpr (sizeof(T) == 4 && !FULL) {
    if (!(vec && n >= 4)) {
      const uint32_t to = ptx::smem_u32(place);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j < n)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + 4 * j), "l"(p + j)
                       : "memory");
        else
          asm volatile("st.shared.b32 [%0], 0;" ::"r"(to + 4 * j) : "memory");
      }
      return;
    }
  }
  few_issue(place, p, n, vec);
}

// Values past the row's end, where 0 times a scale that is not finite would not
// be 0 (FULL: whole pieces only).
template <bool FULL, int N>
__device__ __forceinline__ void zero_past(F2 (&v)[N / 2], int n) {
  if (FULL ? n <= 0 : n < N) {
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      if (FULL || 2 * j >= n) v[j].x = 0.f;
      if (FULL || 2 * j + 1 >= n) v[j].y = 0.f;
    }
  }
}

// v times the N values of a parameter vector from column c (without one: 1).
template <bool FULL, int N>
__device__ __forceinline__ void times(F2 (&v)[N / 2], const float* gain, int c, int n) {
  if (!gain) return;
  float g[N];
  load_param<N, FULL>(gain, c, n, 1.f, g);
#pragma unroll
  for (int j = 0; j < N / 2; ++j) v[j] = mul2(v[j], f2(g[2 * j], g[2 * j + 1]));
}

// FORM: what the launch promises of the rows.  kFull: whole aligned pieces,
// kExact: and exactly as many as the threads that share a row hold.
enum { kAny, kFull, kExact };

// Where a thread's share of the rows lies: piece i at column c0 + i 32 WPR N.
template <typename T, int WPR, bool WIDE>
struct Place {
  static constexpr int ROWS = HeldBlock<WPR>::ROWS, N = RowVec<T>::N;
  static constexpr int WIDTH = vpt<T>() * 32 * WPR;  // columns of a block
  int slot, t, rank, c0;
  uint32_t row, stride;  // (unsigned: a row number past T is below 2^32)
  __device__ __forceinline__ explicit Place(int cluster) {
    slot = threadIdx.x / (32 * WPR);
    t = threadIdx.x % (32 * WPR);
    rank = WIDE ? (int)(blockIdx.x % cluster) : 0;
    c0 = rank * WIDTH + t * N;
    stride = WIDE ? gridDim.x / cluster : gridDim.x * ROWS;
    row = WIDE ? blockIdx.x / cluster : blockIdx.x * ROWS + slot;
  }
  __device__ __forceinline__ int col(int i) const { return c0 + i * 32 * WPR * N; }
  // columns from piece i's first to the row's end (EXACT: known to hold the piece)
  template <bool EXACT>
  __device__ __forceinline__ int left(int d, int i) const {
    return EXACT ? N : d - col(i);
  }
  // this thread's first value of row r of a matrix (pitches are ints at the C
  // boundary: one widening multiplication)
  __device__ __forceinline__ T* in(const void* m, long long ld, uint32_t r) const {
    return static_cast<T*>(const_cast<void*>(m)) + ((uint64_t)r * (uint32_t)ld + c0);
  }
};

template <typename T, int WPR, int FORM, bool WIDE>
__global__ void __launch_bounds__(HeldBlock<WPR>::THREADS,
                                  1024 / HeldBlock<WPR>::THREADS)
    resnorm_fwd_kernel(const ResNorm p, int cluster) {
  constexpr int N = RowVec<T>::N, NV = vpt<T>() / N, ROWS = HeldBlock<WPR>::ROWS;
  constexpr int THREADS = HeldBlock<WPR>::THREADS, step = 32 * WPR * N;
  constexpr bool FULL = FORM != kAny, EXACT = FORM == kExact;
  __shared__ float part[2][ROWS][WPR];
  __shared__ Exchange ex;
  extern __shared__ __align__(16) uint8_t ring_mem[];
  pdl_wait();
  pdl_launch_dependents();
  Place<T, WPR, WIDE> at(cluster);
  const uint32_t rows = (uint32_t)p.T;
  const float inv_d = 1.f / (float)p.d;
  const bool block = p.b != nullptr, gate = p.z != nullptr;
  const DropKey key(p.drop);
  RowSum<WPR, WIDE, ROWS> sum{part, &ex, at.slot, at.t >> 5, at.rank, cluster, p.wait_ns, p.err};
  sum.begin();
  Ring<T, 1, THREADS> ring{reinterpret_cast<uint4*>(ring_mem) + threadIdx.x, 1 + block + gate, 0};
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (FULL && !EXACT && at.col(i) >= p.d) ring.clear(i);
  auto issue = [&](int s, uint32_t r) {
    if (r < rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int n = at.template left<EXACT>(p.d, i);
        if (FULL && n <= 0) continue;
        issue_piece<T, FULL>(ring.at(s, 0, i), at.in(p.x, p.ldx, r) + i * step, n, p.vec & kXVec);
        if (block)
          issue_piece<T, FULL>(ring.at(s, 1, i), at.in(p.b, p.ldb, r) + i * step, n, p.vec & kBVec);
        if (gate)
          issue_piece<T, FULL>(ring.at(s, 2, i), at.in(p.z, p.ldz, r) + i * step, n, p.vec & kZVec);
      }
    }
    few_commit();
  };
  issue(0, at.row);
  for (; at.row < rows; at.row += at.stride) {  // uniform over the threads that share a row
    const uint32_t row = at.row;
    issue(ring.stage ^ 1, row + at.stride);
    few_wait<1>();
    F2 v[NV][N / 2];
    if (block) {
#pragma unroll
      for (int i = 0; i < NV; ++i) unpack_piece<T>(ring(1, i), v[i]);
      float rho = 1.f;
      if (p.post) {
        F2 s2 = f2(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < N / 2; ++j) s2 = fma2(v[i][j], v[i][j], s2);
        rho = rsqrtf(sum(s2.x + s2.y) * inv_d + p.eps);  // two ulp
        if (p.b_rstd && at.rank == 0 && at.t == 0) p.b_rstd[row] = rho;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = at.col(i), n = at.template left<EXACT>(p.d, i);
        if (p.post) {
#pragma unroll
          for (int j = 0; j < N / 2; ++j) v[i][j] = mul2(v[i][j], f2(rho));
        }
        times<FULL, N>(v[i], p.post_gain, c, n);
        if (p.drop.threshold) {
          uint32_t w[N / 2];
          drop_words<N>(p.drop, key, row, c, w);
#pragma unroll
          for (int j = 0; j < N / 2; ++j) v[i][j] = drop2(v[i][j], w[j], key, p.drop.scale);
        }
        if (gate) {
          F2 z[N / 2], rest;
          unpack_piece<T>(ring(2, i), z);
          if (p.sigmoid) {
#pragma unroll
            for (int j = 0; j < N / 2; ++j) z[j] = logistic2<T>(z[j], rest);
          }
#pragma unroll
          for (int j = 0; j < N / 2; ++j) v[i][j] = mul2(v[i][j], z[j]);
        }
        F2 x[N / 2];
        unpack_piece<T>(ring(0, i), x);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) v[i][j] = fma2(v[i][j], f2(p.scale), x[j]);
        zero_past<FULL, N>(v[i], n);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) unpack_piece<T>(ring(0, i), v[i]);
    }
    if (p.h) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        store_piece_of<FULL>(at.in(p.h, p.ldh, row) + i * step,
                             reinterpret_cast<const float(&)[N]>(v[i]), at.template left<EXACT>(p.d, i),
                             p.vec & kHVec);
    }
    if (p.n) {
      F2 s2 = f2(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < N / 2; ++j) s2 = fma2(v[i][j], v[i][j], s2);
      const float rho = rsqrtf(sum(s2.x + s2.y) * inv_d + p.eps);
      if (p.h_rstd && at.rank == 0 && at.t == 0) p.h_rstd[row] = rho;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = at.col(i), n = at.template left<EXACT>(p.d, i);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) v[i][j] = mul2(v[i][j], f2(rho));
        times<FULL, N>(v[i], p.next_gain, c, n);
        store_piece_of<FULL>(at.in(p.n, p.ldn, row) + i * step,
                             reinterpret_cast<const float(&)[N]>(v[i]), n, p.vec & kNVec);
      }
    }
    ring.stage ^= 1;
  }
  if constexpr (WIDE) ptx::cluster_sync();  // no block leaves while its sums may be read
}

// Rows ahead in the backward's ring: one; none for fp32 rows of 512 threads, where
// a second row would not fit: the places of what has been read are filled with
// the next row's at once.
template <typename T, int WPR>
constexpr int bwd_ahead() {
  return sizeof(T) == 4 && WPR == 32 ? 0 : 1;
}

template <typename T, int WPR, int FORM, bool WIDE>
__global__ void __launch_bounds__(HeldBlock<WPR>::THREADS,
                                  WPR == 32 ? 1 : 512 / HeldBlock<WPR>::THREADS)
    resnorm_bwd_kernel(const ResNorm p, int cluster) {
  constexpr int N = RowVec<T>::N, NV = vpt<T>() / N, ROWS = HeldBlock<WPR>::ROWS;
  constexpr int THREADS = HeldBlock<WPR>::THREADS, step = 32 * WPR * N;
  constexpr bool FULL = FORM != kAny, EXACT = FORM == kExact;
  __shared__ float part[2][ROWS][WPR];
  __shared__ Exchange ex;
  extern __shared__ __align__(16) uint8_t ring_mem[];
  pdl_wait();
  pdl_launch_dependents();
  Place<T, WPR, WIDE> at(cluster);
  const uint32_t rows = (uint32_t)p.T;
  const float inv_d = 1.f / (float)p.d;
  const bool block = p.b != nullptr, gate = p.z != nullptr, next = p.n != nullptr;
  const DropKey key(p.drop);
  RowSum<WPR, WIDE, ROWS> sum{part, &ex, at.slot, at.t >> 5, at.rank, cluster, p.wait_ns, p.err};
  sum.begin();
  F2 dnext[NV][N / 2], dpost[NV][N / 2];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < N / 2; ++j) dnext[i][j] = dpost[i][j] = f2(0.f);
  constexpr int AHEAD = bwd_ahead<T, WPR>();
  // places of dh, b and z behind dn and h
  const int mx = next ? 2 : 0, mb = mx + (p.x != nullptr), mz = mb + 1;
  Ring<T, AHEAD, THREADS> ring{reinterpret_cast<uint4*>(ring_mem) + threadIdx.x,
                               mb + block + gate, 0};
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (FULL && !EXACT && at.col(i) >= p.d) ring.clear(i);
  float rh_n = 0.f, rb_n = 0.f;  // the next row's
  // dn, h and dh of row r, one group of copies, and b and z, another
  auto issue_norm = [&](int s, uint32_t r) {
    if (r < rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int n = at.template left<EXACT>(p.d, i);
        if (FULL && n <= 0) continue;
        if (next) {
          issue_piece<T, FULL>(ring.at(s, 0, i), at.in(p.n, p.ldn, r) + i * step, n, p.vec & kNVec);
          issue_piece<T, FULL>(ring.at(s, 1, i), at.in(p.h, p.ldh, r) + i * step, n, p.vec & kHVec);
        }
        if (p.x)
          issue_piece<T, FULL>(ring.at(s, mx, i), at.in(p.x, p.ldx, r) + i * step, n, p.vec & kXVec);
      }
      if (next) rh_n = p.h_rstd[r];
    }
    few_commit();
  };
  auto issue_block = [&](int s, uint32_t r) {
    if (r < rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int n = at.template left<EXACT>(p.d, i);
        if (FULL && n <= 0) continue;
        if (block)
          issue_piece<T, FULL>(ring.at(s, mb, i), at.in(p.b, p.ldb, r) + i * step, n, p.vec & kBVec);
        if (gate)
          issue_piece<T, FULL>(ring.at(s, mz, i), at.in(p.z, p.ldz, r) + i * step, n, p.vec & kZVec);
      }
      if (p.post) rb_n = p.b_rstd[r];
    }
    few_commit();
  };
  issue_norm(0, at.row);
  issue_block(0, at.row);
  for (; at.row < rows; at.row += at.stride) {
    const uint32_t row = at.row, then = row + at.stride;
    const float rh = rh_n, rb = p.post ? rb_n : 1.f;
    if constexpr (AHEAD) {
      issue_norm(ring.stage ^ 1, then);
      issue_block(ring.stage ^ 1, then);
      few_wait<2>();
    } else {
      few_wait<1>();
    }
    F2 v[NV][N / 2];  // dh'
    if (next) {
      F2 hh[NV][N / 2];
      F2 s2 = f2(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = at.col(i), n = at.template left<EXACT>(p.d, i);
        unpack_piece<T>(ring(0, i), v[i]);
        unpack_piece<T>(ring(1, i), hh[i]);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) hh[i][j] = mul2(hh[i][j], f2(rh));
        zero_past<FULL, N>(hh[i], n);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) dnext[i][j] = fma2(v[i][j], hh[i][j], dnext[i][j]);
        times<FULL, N>(v[i], p.next_gain, c, n);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) s2 = fma2(v[i][j], hh[i][j], s2);
      }
      const float m = sum(s2.x + s2.y) * inv_d;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < N / 2; ++j)
          v[i][j] = mul2(fma2(hh[i][j], f2(-m), v[i][j]), f2(rh));
      if (p.x) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          F2 x[N / 2];
          unpack_piece<T>(ring(mx, i), x);
#pragma unroll
          for (int j = 0; j < N / 2; ++j) v[i][j] = add2(v[i][j], x[j]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) unpack_piece<T>(ring(mx, i), v[i]);
    }
    if constexpr (!AHEAD) {
      issue_norm(0, then);
      few_wait<1>();
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      store_piece_of<FULL>(at.in(p.dx, p.lddx, row) + i * step,
                           reinterpret_cast<const float(&)[N]>(v[i]), at.template left<EXACT>(p.d, i),
                           p.vec & kDxVec);
    if (!block) {
      if constexpr (AHEAD) ring.stage ^= 1;
      else issue_block(0, then);
      continue;
    }
    F2 s2 = f2(0.f);
    F2 bb[NV][N / 2];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = at.col(i), n = at.template left<EXACT>(p.d, i);
      uint32_t w[N / 2];
      if (p.drop.threshold) drop_words<N>(p.drop, key, row, c, w);
      unpack_piece<T>(ring(mb, i), bb[i]);
      if (p.post) {
#pragma unroll
        for (int j = 0; j < N / 2; ++j) bb[i][j] = mul2(bb[i][j], f2(rb));
        zero_past<FULL, N>(bb[i], n);
      }
#pragma unroll
      for (int j = 0; j < N / 2; ++j) v[i][j] = mul2(v[i][j], f2(p.scale));
      zero_past<FULL, N>(v[i], n);
      if (gate) {
        F2 z[N / 2], dz[N / 2];
        unpack_piece<T>(ring(mz, i), z);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) dz[j] = bb[i][j];
        times<FULL, N>(dz, p.post_gain, c, n);
        if (p.drop.threshold) {
#pragma unroll
          for (int j = 0; j < N / 2; ++j) dz[j] = drop2(dz[j], w[j], key, p.drop.scale);
        }
#pragma unroll
        for (int j = 0; j < N / 2; ++j) dz[j] = mul2(dz[j], v[i][j]);
        if (p.sigmoid) {
#pragma unroll
          for (int j = 0; j < N / 2; ++j) {
            F2 rest;
            z[j] = logistic2<T>(z[j], rest);
            dz[j] = mul2(dz[j], mul2(z[j], rest));
          }
        }
        store_piece_of<FULL>(at.in(p.dz, p.lddz, row) + i * step,
                             reinterpret_cast<const float(&)[N]>(dz), n, p.vec & kDzVec);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) v[i][j] = mul2(v[i][j], z[j]);
      }
      if (p.drop.threshold) {
#pragma unroll
        for (int j = 0; j < N / 2; ++j) v[i][j] = drop2(v[i][j], w[j], key, p.drop.scale);
      }
#pragma unroll
      for (int j = 0; j < N / 2; ++j) dpost[i][j] = fma2(v[i][j], bb[i][j], dpost[i][j]);
      times<FULL, N>(v[i], p.post_gain, c, n);
#pragma unroll
      for (int j = 0; j < N / 2; ++j) s2 = fma2(v[i][j], bb[i][j], s2);
    }
    if constexpr (AHEAD) ring.stage ^= 1;
    else issue_block(0, then);
    if (p.post) {
      const float m = sum(s2.x + s2.y) * inv_d;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < N / 2; ++j)
          v[i][j] = mul2(fma2(bb[i][j], f2(-m), v[i][j]), f2(rb));
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      store_piece_of<FULL>(at.in(p.db, p.lddb, row) + i * step,
                           reinterpret_cast<const float(&)[N]>(v[i]), at.template left<EXACT>(p.d, i),
                           p.vec & kDbVec);
  }
  if (p.part) {
    // this block's partial sums, row slots added in order, in the ring's place
    few_wait<0>();
    float* out = p.part + (long long)(WIDE ? blockIdx.x / cluster : blockIdx.x) * 2 * p.d;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      F2(&a)[NV][N / 2] = which ? dpost : dnext;
      if constexpr (ROWS > 1) {
        F2* sums = reinterpret_cast<F2*>(ring_mem) + at.t;  // value k at [k * 32 WPR]
        for (int k = 1; k < ROWS; ++k) {
          __syncthreads();
          if (at.slot == k)
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
              for (int j = 0; j < N / 2; ++j) sums[(i * N / 2 + j) * 32 * WPR] = a[i][j];
          __syncthreads();
          if (at.slot == 0)
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
              for (int j = 0; j < N / 2; ++j)
                a[i][j] = add2(a[i][j], sums[(i * N / 2 + j) * 32 * WPR]);
        }
      }
      if (at.slot == 0)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = at.col(i);
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

template <typename T, int WPR, int FORM, bool WIDE>
mlp_status fwd_of(const ResNorm& p, cudaStream_t st) {
  using B = HeldBlock<WPR>;
  constexpr int kWidth = vpt<T>() * 32 * WPR;
  auto kernel = resnorm_fwd_kernel<T, WPR, FORM, WIDE>;
  static PerDevice per_sm;
  using R = Ring<T, 1, B::THREADS>;
  constexpr int kSmem = R::bytes(3);
  static_assert(kSmem <= 225 * 1024, "shared memory");
  static PerDevice configured;
  if (!allow_smem(configured, kernel, kSmem)) return MLP_ERR_CUDA;
  const int cluster = WIDE ? (p.d + kWidth - 1) / kWidth : 1;
  int blocks = walk_blocks(kernel, B::THREADS, per_sm, WIDE ? 1ll << 40 : p.T, B::ROWS, kSmem);
  if (WIDE) {
    blocks /= cluster;
    if (blocks < 1) blocks = 1;
    if (blocks > p.T) blocks = (int)p.T;
    blocks *= cluster;
  }
  LaunchScope ls("resnorm_fwd", st, p.T, p.d, sizeof(T));
  return launch_rows(kernel, blocks, B::THREADS, R::bytes(1 + !!p.b + !!p.z), cluster, p, st);
}

template <typename T, int WPR, int FORM, bool WIDE>
mlp_status bwd_of(const ResNorm& p, int* rows, cudaStream_t st) {
  using B = HeldBlock<WPR>;
  constexpr int kWidth = vpt<T>() * 32 * WPR;
  auto kernel = resnorm_bwd_kernel<T, WPR, FORM, WIDE>;
  static PerDevice per_sm;
  using R = Ring<T, bwd_ahead<T, WPR>(), B::THREADS>;
  constexpr int kSmem = R::bytes(5);
  static_assert(kSmem <= 225 * 1024, "shared memory");
  static_assert(B::ROWS == 1 || 32 * WPR * vpt<T>() * 4 <= R::bytes(1),
                "sums in the ring's place");
  static PerDevice configured;
  if (!allow_smem(configured, kernel, kSmem)) return MLP_ERR_CUDA;
  const int cluster = WIDE ? (p.d + kWidth - 1) / kWidth : 1;
  int resident = walk_blocks(kernel, B::THREADS, per_sm, WIDE ? 1ll << 40 : p.T, B::ROWS, kSmem);
  if (WIDE) resident = resident / cluster > 0 ? resident / cluster : 1;
  if (resident < *rows) *rows = resident;
  LaunchScope ls("resnorm_bwd", st, p.T, p.d, sizeof(T));
  return launch_rows(kernel, *rows * cluster, B::THREADS,
                     R::bytes(2 * !!p.n + !!p.x + !!p.b + !!p.z), cluster, p, st);
}

// kExact where it applies (us with it and with kFull, 2^25 values, 2^26 from 2,048 and
// 2^27 from 8,192 columns on: forward bf16 512 columns 50 and 53, 1,024 51 and 55, 4,096 89
// and 98, 8,192 169 and 185, with gate and dropout 61 and 64, 62 and 69, 119 and 136, 226
// and 255; backward 73 and 77, 76 and 83, 170 and 178, 327 and 331).  With gate and
// dropout its 16-bit backward spills 24 to 48 bytes a thread at two to eight warps a
// row and is the slower one there (bf16 1,024 columns 117 and 112, 2,048 236 and 216, 4,096
// 267 and 238, 8,192 549 and 525; fp16 113 and 110, 225 and 216, 253 and 240, but 8,192 499
// and 538, and 512 98 and 101, 96 and 100).
template <typename T, int WPR, bool WIDE, bool BWD>
mlp_status of_form(const ResNorm& p, bool full, int* rows, cudaStream_t st) {
  const bool exact = full && p.d % (vpt<T>() * 32 * WPR) == 0;
  if constexpr (BWD)
    return exact  ? bwd_of<T, WPR, kExact, WIDE>(p, rows, st)
           : full ? bwd_of<T, WPR, kFull, WIDE>(p, rows, st)
                  : bwd_of<T, WPR, kAny, WIDE>(p, rows, st);
  else
    return exact  ? fwd_of<T, WPR, kExact, WIDE>(p, st)
           : full ? fwd_of<T, WPR, kFull, WIDE>(p, st)
                  : fwd_of<T, WPR, kAny, WIDE>(p, st);
}

template <typename T, bool BWD>
mlp_status of_type(ResNorm p, int* rows, cudaStream_t st) {
  p.wait_ns = wait_limit_ns();
  p.err = device_error_word();
  if (!p.err) return MLP_ERR_CUDA;
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
  const int warps = (p.d + 32 * vpt<T>() - 1) / (32 * vpt<T>());
  if (warps <= 1) return of_form<T, 1, false, BWD>(p, full, rows, st);
  if (warps <= 2) return of_form<T, 2, false, BWD>(p, full, rows, st);
  if (warps <= 4) return of_form<T, 4, false, BWD>(p, full, rows, st);
  if (warps <= 8) return of_form<T, 8, false, BWD>(p, full, rows, st);
  constexpr int kMost = kBlockWidth / (32 * vpt<T>());  // 16, or 32 for fp32
  if (kMost > 16 && warps <= 16) return of_form<T, 16, false, BWD>(p, full, rows, st);
  if (warps <= kMost) return of_form<T, kMost, false, BWD>(p, full, rows, st);
  return of_form<T, kMost, true, BWD>(p, full, rows, st);
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
