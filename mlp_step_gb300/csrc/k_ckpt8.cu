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
// TB/s, the copy rate).  Rows that start anywhere: the kernels of a value per
// lane below.
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

// Rows that start anywhere: a value per lane, so that a group is a warp (its
// largest magnitude one reduction) and unaligned runs still leave as whole
// lines.  A warp takes eight groups of a row, all loads first.  (10,007 x 1,001,
// encoded and decoded: fp32 9.9 and 7.6 us, bf16 9.9 and 7.1; by pieces, whose
// values then move one by one, 12.5 and 12.7, 14.3 and 28.4.)
constexpr int kRowGroups = 8, kRowChunk = kRowGroups * kCkptGroup;

template <typename T>
__global__ void __launch_bounds__(kThreads)
    ckpt8_encode_rows_kernel(const T* __restrict__ x, unsigned units, unsigned chunks, int cols,
                             long long ldx, int8_t* __restrict__ q, long long ldq,
                             uint8_t* __restrict__ scale, long long lds) {
  pdl_wait();
  pdl_launch_dependents();
  const unsigned unit = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (unit >= units) return;
  const int lane = threadIdx.x & 31;
  const unsigned row = unit / chunks;
  const int g0 = (int)(unit - row * chunks) * kRowGroups, c = g0 * kCkptGroup + lane;
  const T* px = x + row * ldx + c;
  int8_t* pq = q + row * ldq + c;
  float v[kRowGroups];
#pragma unroll
  for (int g = 0; g < kRowGroups; ++g)
    v[g] = c + g * kCkptGroup < cols ? to_f32(px[g * kCkptGroup]) : 0.f;
  uint32_t mine = 0;
#pragma unroll
  for (int g = 0; g < kRowGroups; ++g) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(v[g]) & 0x7fffffffu);
    const uint32_t b = ckpt8_byte(top);
    if (ckpt8_must_hold(top)) v[g] = ckpt8_hold(v[g], ckpt8_step(b));
    const uint32_t w = b == kCkptNanByte ? 0u : ckpt8_q(v[g], ckpt8_inv_step(b));
    if (c + g * kCkptGroup < cols) pq[g * kCkptGroup] = (int8_t)w;
    if (lane == g) mine = b;
  }
  if (lane < kRowGroups && (g0 + lane) * kCkptGroup < cols)
    scale[row * lds + g0 + lane] = (uint8_t)mine;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    ckpt8_decode_rows_kernel(const int8_t* __restrict__ q, long long ldq,
                             const uint8_t* __restrict__ scale, long long lds, unsigned units,
                             unsigned chunks, int cols, T* __restrict__ out, long long ldo) {
  pdl_wait();
  pdl_launch_dependents();
  const unsigned unit = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (unit >= units) return;
  const int lane = threadIdx.x & 31;
  const unsigned row = unit / chunks;
  const int g0 = (int)(unit - row * chunks) * kRowGroups, c = g0 * kCkptGroup + lane;
  const int8_t* pq = q + row * ldq + c;
  T* po = out + row * ldo + c;
  uint32_t b = 0;
  if (lane < kRowGroups && (g0 + lane) * kCkptGroup < cols) b = scale[row * lds + g0 + lane];
  int w[kRowGroups];
#pragma unroll
  for (int g = 0; g < kRowGroups; ++g)
    w[g] = c + g * kCkptGroup < cols ? pq[g * kCkptGroup] : 0;
  const float step = ckpt8_step(b);
#pragma unroll
  for (int g = 0; g < kRowGroups; ++g) {
    const float s = __shfl_sync(0xffffffffu, step, g);
    if (c + g * kCkptGroup < cols) from_f32((float)w[g] * s, po[g * kCkptGroup]);
  }
}

// Units of those kernels; 0 where they are too many for their 32-bit numbers, or
// rows so narrow that they leave a warp's chunk mostly empty (100,000 x 45 fp32:
// encoded in 22 us by rows, 9 by pieces).
unsigned row_units(long long rows, int cols, unsigned* chunks) {
  *chunks = (cols + kRowChunk - 1) / kRowChunk;
  if (cols < kRowChunk * 3 / 4) return 0u;
  const long long units = rows * *chunks;
  return units < 0x7fffffffll ? (unsigned)units : 0u;
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
  const int x_vec = rows_aligned(x, ldx, sizeof(T), 16), q_vec = rows_aligned(q, ldq, 1, RowVec<T>::N);
  unsigned chunks;
  const unsigned units = flat || (x_vec && q_vec) ? 0u : row_units(rows, cols, &chunks);
  if (units) {
    launch_k(ckpt8_encode_rows_kernel<T>, dim3((units + kThreads / 32 - 1) / (kThreads / 32)),
             dim3(kThreads), 0, st, x, units, chunks, cols, ldx, q, ldq, scale, lds);
    return launch_status();
  }
  launch_k(flat ? ckpt8_encode_kernel<T, true> : ckpt8_encode_kernel<T, false>,
           dim3((unsigned)blocks), dim3(kThreads), 0, st, x, flat ? 1ll : rows,
           flat ? rows * cols : (long long)cols, ldx, q, ldq, scale, lds,
           x_vec, q_vec);
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
  const int q_vec = rows_aligned(q, ldq, 1, RowVec<T>::N), o_vec = rows_aligned(out, ldo, sizeof(T), 16);
  unsigned chunks;
  const unsigned units = flat || (q_vec && o_vec) ? 0u : row_units(rows, cols, &chunks);
  if (units) {
    launch_k(ckpt8_decode_rows_kernel<T>, dim3((units + kThreads / 32 - 1) / (kThreads / 32)),
             dim3(kThreads), 0, st, q, ldq, scale, lds, units, chunks, cols, out, ldo);
    return launch_status();
  }
  launch_k(flat ? ckpt8_decode_kernel<T, true> : ckpt8_decode_kernel<T, false>,
           dim3((unsigned)blocks), dim3(kThreads), 0, st, q, ldq, scale, lds, flat ? 1ll : rows,
           flat ? rows * cols : (long long)cols, out, ldo,
           q_vec, o_vec);
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
