// 8-bit activation checkpoints (format: ckpt8.cuh): encode and decode of a
// matrix.  Both are one pass over the data and bound by HBM: 2 + 33/32 bytes
// per bf16 value either way.
//
// Work item = one 16-byte piece of a row (8 16-bit or 4 fp32 values), so a
// group of 32 is 4 or 8 neighbouring lanes, every load and store of a warp is
// one contiguous run, and the group's largest magnitude is two or three
// shuffles.  A thread takes four items a block-width apart, all loads first:
// with 64 bytes in flight per thread and full occupancy the loads cover the
// latency without a staging pipeline.
// Measured: 262,144 x 512 bf16 encoded in 62 us and decoded in 59 (6.6 and 6.9
// TB/s, the copy rate); 10,007 x 1,001 fp32, whose rows start anywhere and move
// value by value, in 16 and 18 (3.2 and 2.7 TB/s, bound by
// instruction issue; 26 us both ways where L2 holds the matrix).
#include "ckpt8.cuh"
#include "kernels.cuh"
#include "rowvec.cuh"
#include "trace.cuh"

namespace mlp {

namespace {

constexpr int kThreads = 256;
constexpr int kItems = 4;  // per thread

// Pieces of a row, padded to whole groups so that a group's lanes never
// straddle two rows.
template <typename T>
__host__ __device__ constexpr long long pieces_per_row(long long cols) {
  return (cols + kCkptGroup - 1) / kCkptGroup * (kCkptGroup / RowVec<T>::N);
}

// Where a block's items lie.  FLAT: matrices without padding whose rows are
// whole groups are one long row, item i its piece i (the divisions below cost
// more than the encoding: 262,144 x 512 bf16 90 us with them).  Otherwise one
// 64-bit division per block gives its first row and piece, and the items
// divide a small offset.
template <bool FLAT>
struct Span {
  long long row0;
  unsigned off0;
  int per_row;
  __device__ __forceinline__ explicit Span(int per_row_) : row0(0), off0(0), per_row(per_row_) {
    const long long base = (long long)blockIdx.x * (kThreads * kItems);
    if constexpr (!FLAT) {
      row0 = base / per_row;
      off0 = (unsigned)(base - row0 * per_row);
    }
  }
  // row and first column of item k of this thread
  template <int N>
  __device__ __forceinline__ void item(int k, long long& row, long long& col) const {
    const unsigned o = off0 + k * kThreads + threadIdx.x;
    if constexpr (FLAT) {
      row = 0;
      col = ((long long)blockIdx.x * (kThreads * kItems) + o) * N;
    } else {
      const unsigned r = o / (unsigned)per_row;
      row = row0 + r;
      col = (long long)(o - r * per_row) * N;
    }
  }
};

__device__ __forceinline__ int columns_left(long long cols, long long col) {
  const long long n = cols - col;
  return n > kCkptGroup ? kCkptGroup : (int)n;
}

template <typename T, bool FLAT>
__global__ void __launch_bounds__(kThreads)
    ckpt8_encode_kernel(const T* __restrict__ x, long long rows, long long cols, long long ldx,
                        int8_t* __restrict__ q, long long ldq, uint8_t* __restrict__ scale,
                        long long lds, int x_vec, int q_vec) {
  constexpr int N = RowVec<T>::N;
  constexpr int LANES = kCkptGroup / N;  // lanes of a group
  pdl_wait();
  pdl_launch_dependents();
  const Span<FLAT> sp(FLAT ? 1 : (int)pieces_per_row<T>(cols));
  long long row[kItems], col[kItems];
  uint4 raw[kItems];
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    sp.template item<N>(k, row[k], col[k]);
    raw[k] = load_piece(x + row[k] * ldx + col[k], row[k] < rows ? columns_left(cols, col[k]) : 0, x_vec);
  }
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    float v[N];
    unpack_piece<T>(raw[k], v);
    uint32_t amax = amax_bits_of(v);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    uint32_t w[N / 4];
    const uint32_t b = ckpt8_piece(v, amax, w);
    if (row[k] < rows && col[k] < cols) {
      store_q<N>(q + row[k] * ldq + col[k], columns_left(cols, col[k]), q_vec, w);
      if ((threadIdx.x & (LANES - 1)) == 0) scale[row[k] * lds + col[k] / kCkptGroup] = (uint8_t)b;
    }
  }
}

template <typename T, bool FLAT>
__global__ void __launch_bounds__(kThreads)
    ckpt8_decode_kernel(const int8_t* __restrict__ q, long long ldq,
                        const uint8_t* __restrict__ scale, long long lds, long long rows,
                        long long cols,
                        T* __restrict__ out, long long ldo, int q_vec, int o_vec) {
  constexpr int N = RowVec<T>::N;
  pdl_wait();
  pdl_launch_dependents();
  const Span<FLAT> sp(FLAT ? 1 : (int)pieces_per_row<T>(cols));
  long long row[kItems], col[kItems];
  uint32_t w[kItems][N / 4], b[kItems];
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    sp.template item<N>(k, row[k], col[k]);
    const int n = row[k] < rows ? columns_left(cols, col[k]) : 0;
    load_q<N>(q + row[k] * ldq + col[k], n, q_vec, w[k]);
    b[k] = n > 0 ? scale[row[k] * lds + col[k] / kCkptGroup] : 0u;
  }
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const float step = ckpt8_step(b[k]);
    float v[N];
#pragma unroll
    for (int j = 0; j < N / 4; ++j) {
      const uint32_t f = ckpt8_flip(w[k][j]);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * j + e] = ckpt8_value(f, e, step);
    }
    if (row[k] < rows)
      store_piece(out + row[k] * ldo + col[k], v, columns_left(cols, col[k]), o_vec);
  }
}

// Rows of pitch ld (elements of size esz) keep pieces of `bytes` aligned?
bool rows_aligned(const void* p, long long ld, int esz, int bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * esz % bytes == 0;
}

// The whole matrix as one row of whole groups?
bool one_row(long long rows, int cols, long long ld, long long ldq, long long lds) {
  return cols % kCkptGroup == 0 &&
         (rows == 1 || (ld == cols && ldq == cols && lds == cols / kCkptGroup));
}

template <typename T>
mlp_status encode_t(const T* x, long long rows, int cols, long long ldx, int8_t* q, long long ldq,
                    uint8_t* scale, long long lds, cudaStream_t st) {
  const long long items = rows * pieces_per_row<T>(cols);
  const long long blocks = (items + kThreads * kItems - 1) / (kThreads * kItems);
  if (blocks > 0x7fffffffll) return MLP_ERR_UNSUPPORTED_SHAPE;
  LaunchScope ls("ckpt8_encode", st, rows, cols, sizeof(T));
  const bool flat = one_row(rows, cols, ldx, ldq, lds);
  launch_k(flat ? ckpt8_encode_kernel<T, true> : ckpt8_encode_kernel<T, false>,
           dim3((unsigned)blocks), dim3(kThreads), 0, st, x, flat ? 1ll : rows,
           flat ? rows * cols : (long long)cols, ldx, q, ldq, scale, lds,
           (int)rows_aligned(x, ldx, sizeof(T), 16), (int)rows_aligned(q, ldq, 1, RowVec<T>::N));
  return launch_status();
}

template <typename T>
mlp_status decode_t(const int8_t* q, long long ldq, const uint8_t* scale, long long lds,
                    long long rows, int cols, T* out, long long ldo, cudaStream_t st) {
  const long long items = rows * pieces_per_row<T>(cols);
  const long long blocks = (items + kThreads * kItems - 1) / (kThreads * kItems);
  if (blocks > 0x7fffffffll) return MLP_ERR_UNSUPPORTED_SHAPE;
  LaunchScope ls("ckpt8_decode", st, rows, cols, sizeof(T));
  const bool flat = one_row(rows, cols, ldo, ldq, lds);
  launch_k(flat ? ckpt8_decode_kernel<T, true> : ckpt8_decode_kernel<T, false>,
           dim3((unsigned)blocks), dim3(kThreads), 0, st, q, ldq, scale, lds, flat ? 1ll : rows,
           flat ? rows * cols : (long long)cols, out, ldo,
           (int)rows_aligned(q, ldq, 1, RowVec<T>::N), (int)rows_aligned(out, ldo, sizeof(T), 16));
  return launch_status();
}

}  // namespace

mlp_status launch_ckpt8_encode(const void* x, int dtype, long long rows, int cols, long long ldx,
                               int8_t* q, long long ldq, uint8_t* scale, long long lds,
                               cudaStream_t st) {
  switch (dtype) {
    case MLP_DTYPE_BF16:
      return encode_t(static_cast<const __nv_bfloat16*>(x), rows, cols, ldx, q, ldq, scale, lds, st);
    case MLP_DTYPE_F16:
      return encode_t(static_cast<const __half*>(x), rows, cols, ldx, q, ldq, scale, lds, st);
    default:
      return encode_t(static_cast<const float*>(x), rows, cols, ldx, q, ldq, scale, lds, st);
  }
}

mlp_status launch_ckpt8_decode(const int8_t* q, long long ldq, const uint8_t* scale, long long lds,
                               long long rows, int cols, void* out, int dtype, long long ldo,
                               cudaStream_t st) {
  switch (dtype) {
    case MLP_DTYPE_BF16:
      return decode_t(q, ldq, scale, lds, rows, cols, static_cast<__nv_bfloat16*>(out), ldo, st);
    case MLP_DTYPE_F16:
      return decode_t(q, ldq, scale, lds, rows, cols, static_cast<__half*>(out), ldo, st);
    default:
      return decode_t(q, ldq, scale, lds, rows, cols, static_cast<float*>(out), ldo, st);
  }
}

}  // namespace mlp
