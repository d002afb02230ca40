// Dropout of a matrix with an optional residual, y = residual + keep x scale:
// the backward is the same kernel on dy.  The mask is computed where it is used
// (philox.cuh), so the traffic is x, the residual and y alone.
#include "kernels.cuh"
#include "philox.cuh"
#include "rowvec.cuh"
#include "trace.cuh"

namespace mlp {

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // pieces of a thread whose loads are in flight together

// A thread's pieces (16 bytes) lie a grid's stride apart, row and column
// carried along (step_rows rows and step_cols pieces, wrapping).
template <typename T>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const Dropout p, int per_row,
                                                           long long step_rows, int step_cols) {
  constexpr int N = RowVec<T>::N;
  pdl_wait();
  pdl_launch_dependents();
  const T* x = static_cast<const T*>(p.x);
  const T* res = static_cast<const T*>(p.res);
  T* y = static_cast<T*>(p.y);
  const DropKey key(p.drop);
  const long long first = (long long)blockIdx.x * kThreads + threadIdx.x;
  long long row = first / per_row;
  int q = (int)(first - row * per_row);
  while (row < p.T) {
    uint4 rx[kAhead], rr[kAhead];
    long long at[kAhead];
    int col[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      at[k] = row;
      col[k] = q * N;
      const int n = row < p.T ? p.d - col[k] : 0;
      rx[k] = load_piece(x + row * p.ldx + col[k], n, p.x_vec);
      if (res) rr[k] = load_piece(res + row * p.ldr + col[k], n, p.r_vec);
      row += step_rows;
      q += step_cols;
      if (q >= per_row) {
        q -= per_row;
        ++row;
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (at[k] >= p.T) break;
      F2 v[N / 2];
      unpack_piece<T>(rx[k], v);
      if (p.drop.threshold) {
        const uint32_t bits = drop_bits<N>(p.drop, key, (uint32_t)at[k], col[k]);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) v[j] = drop2(v[j], bits, 2 * j, p.drop.scale);
      }
      if (res) {
        F2 r[N / 2];
        unpack_piece<T>(rr[k], r);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) v[j] = add2(v[j], r[j]);
      }
      store_piece(y + at[k] * p.ldy + col[k], reinterpret_cast<const float(&)[N]>(v),
                  p.d - col[k], p.y_vec);
    }
  }
}

template <typename T>
mlp_status launch_t(Dropout p, cudaStream_t st) {
  constexpr int N = RowVec<T>::N;
  auto vec = [](const void* m, long long ld) {
    return m && aligned16(m) && ld * (long long)sizeof(T) % 16 == 0;
  };
  p.x_vec = vec(p.x, p.ldx);
  p.r_vec = vec(p.res, p.ldr);
  p.y_vec = vec(p.y, p.ldy);
  const int per_row = (p.d - 1) / N + 1;
  const long long pieces = p.T * per_row;
  const long long most = (long long)num_sms() * 8;
  long long blocks = (pieces + kThreads - 1) / kThreads;
  if (blocks > most) blocks = most;
  const long long step = blocks * kThreads;
  LaunchScope ls("dropout", st, p.T, p.d, sizeof(T));
  launch_k(dropout_kernel<T>, dim3((unsigned)blocks), dim3(kThreads), 0, st, p, per_row,
           step / per_row, (int)(step % per_row));
  return launch_status();
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
