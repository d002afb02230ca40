// Dropout of a matrix with an optional residual, y = residual + keep x scale:
// the backward is the same kernel on dy.  The mask is computed where it is used
// (philox.cuh), so the traffic is x, the residual and y alone.
// Bound by HBM: 262,144 x 512 bf16 with a residual 128 us (6.3 TB/s, 19 instructions
// a value); rows that start anywhere move a value at a time, 10,007 x 1,001 fp32
// 18 us with cold caches (4.5 TB/s).
#include "kernels.cuh"
#include "philox.cuh"
#include "rowvec.cuh"
#include "trace.cuh"

namespace mlp {

namespace {

constexpr int kThreads = 256;
constexpr int kPerSm = 5;  // blocks
constexpr int kAhead = 2;  // pieces of a thread whose loads are in flight together

// A thread's pieces (16 bytes) lie a grid's stride apart, row and column
// carried along (step_rows rows and step_cols pieces, wrapping).  FULL: all rows
// are whole aligned pieces.
template <typename T, bool FULL>
__global__ void __launch_bounds__(kThreads, kPerSm)
    dropout_kernel(const Dropout p, uint32_t per_row, uint32_t step_rows, uint32_t step_cols) {
  constexpr int N = RowVec<T>::N;
  pdl_wait();
  pdl_launch_dependents();
  const T* x = static_cast<const T*>(p.x);
  const T* res = static_cast<const T*>(p.res);
  T* y = static_cast<T*>(p.y);
  const DropKey key(p.drop);
  // pitches and row numbers are ints at the C boundary: one widening
  // multiplication a piece
  const uint32_t rows = (uint32_t)p.T;
  const uint32_t ldx = (uint32_t)p.ldx, ldr = (uint32_t)p.ldr, ldy = (uint32_t)p.ldy;
  const unsigned long long first = (unsigned long long)blockIdx.x * kThreads + threadIdx.x;
  uint32_t row = (uint32_t)(first / per_row), q = (uint32_t)(first % per_row);
  while (row < rows) {
    uint4 rx[kAhead], rr[kAhead];
    uint32_t at[kAhead], col[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      at[k] = row;
      col[k] = q * N;
      const int n = row < rows ? p.d - (int)col[k] : 0;
      rx[k] = load_piece_of<FULL>(x + (uint64_t)row * ldx + col[k], n, p.x_vec);
      if (res) rr[k] = load_piece_of<FULL>(res + (uint64_t)row * ldr + col[k], n, p.r_vec);
      row += step_rows;
      q += step_cols;
      if (q >= per_row) {
        q -= per_row;
        ++row;
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (at[k] >= rows) break;
      F2 v[N / 2];
      unpack_piece<T>(rx[k], v);
      if (p.drop.threshold) {
        uint32_t w[N / 2];
        drop_words<N>(p.drop, key, at[k], (int)col[k], w);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) v[j] = drop2(v[j], w[j], key, p.drop.scale);
      }
      if (res) {
        F2 r[N / 2];
        unpack_piece<T>(rr[k], r);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) v[j] = add2(v[j], r[j]);
      }
      store_piece_of<FULL>(y + (uint64_t)at[k] * ldy + col[k],
                           reinterpret_cast<const float(&)[N]>(v), p.d - (int)col[k], p.y_vec);
    }
  }
}

template <typename T, bool FULL>
mlp_status launch_of(const Dropout& p, cudaStream_t st) {
  constexpr int N = RowVec<T>::N;
  const uint32_t per_row = (uint32_t)((p.d - 1) / N + 1);
  const long long pieces = p.T * per_row;
  const long long most = (long long)num_sms() * kPerSm;
  long long blocks = (pieces + kThreads - 1) / kThreads;
  if (blocks > most) blocks = most;
  const uint32_t step = (uint32_t)blocks * kThreads;
  LaunchScope ls("dropout", st, p.T, p.d, sizeof(T));
  launch_k(dropout_kernel<T, FULL>, dim3((unsigned)blocks), dim3(kThreads), 0, st, p, per_row,
           step / per_row, step % per_row);
  return launch_status();
}

template <typename T>
mlp_status launch_t(Dropout p, cudaStream_t st) {
  auto vec = [](const void* m, long long ld) {
    return m && aligned16(m) && ld * (long long)sizeof(T) % 16 == 0;
  };
  p.x_vec = vec(p.x, p.ldx);
  p.r_vec = vec(p.res, p.ldr);
  p.y_vec = vec(p.y, p.ldy);
  const bool full = p.d % RowVec<T>::N == 0 && p.x_vec && p.y_vec && (!p.res || p.r_vec);
  return full ? launch_of<T, true>(p, st) : launch_of<T, false>(p, st);
}

}  // namespace

mlp_status launch_dropout(const Dropout& p, cudaStream_t st) {
  switch (p.dtype) {
    case MLP_DTYPE_BF16: return launch_t<__nv_bfloat16>(p, st);
    case MLP_DTYPE_F16: return launch_t<__half>(p, st);
    default: return launch_t<float>(p, st);
  }
}

}  // namespace mlp
