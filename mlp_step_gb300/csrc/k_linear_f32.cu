// fp32 products of the linear layers: raw sums into planes [splits][T][ldp]
// that launch_linear_finish turns into the layer's outputs.
//   forward  P = x W,    W [K][N];     backward  P = dy W^T,  W [N][K]
//
// Bound: fp32 FMA issue (no tensor cores: their operands are 19 bits at most).
// A block computes 128 x 128 outputs, a thread 8 x 8 of them: per step of K
// four 16-byte shared-memory loads feed 64 FMAs, issued as 32 packed ones
// (scalar FMAs: 1.12 times the time; the 64 x 64 tiles of the general fp32
// product, 4 x 4 per thread, load half as much for 16: 26,823 x 2,502 x 354
// 2,990 us there, 1,060 here = 45 TFLOP/s, 56 % of the FMA rate).  Both operands lie in
// shared memory as [k][128 rows or columns]; matrices whose rows run along K
// are transposed by the copies themselves (4-byte asynchronous copies, which
// take any pitch), W [K][N] goes in 16-byte pieces where its rows allow.
// Three stages of 16 of K, so two are in flight.  Sums run over ascending k in
// one fused multiply-add chain per output and split.
#include "f32x2.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "trace.cuh"

namespace mlp {

namespace {

constexpr int kThreads = 256;
constexpr int TM = 128, TN = 128, TK = 16, STAGES = 3;
constexpr int PITCH = 132;  // floats per k: rows stay 16-byte aligned
constexpr int kSmem = STAGES * 2 * TK * PITCH * 4;

// `bytes` of src into dst, zeros past the matrix (ok false reads nothing).
template <int BYTES>
__device__ __forceinline__ void copy(float* dst, const float* src, bool ok) {
  const uint32_t d = ptx::smem_u32(dst);
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src),
                 "r"(ok ? 16 : 0)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(d), "l"(src),
                 "r"(ok ? 4 : 0)
                 : "memory");
}

// A thread's part of staging rows [r0, r0 + 128) x 16 columns of a matrix whose
// rows run along K, transposed into s[k][row]: column tid % 16 of rows
// tid / 16 + 16 i.  Addresses and the rows that exist are worked out once.
struct RowStager {
  const float* p;
  long long step;  // 16 rows
  unsigned rows;   // bit i: row i exists
  __device__ __forceinline__ RowStager(const float* base, long long ld, long long r0,
                                       long long n_rows, int k_lo, int tid) {
    const long long r = r0 + (tid >> 4);
    p = base + r * ld + k_lo + (tid & 15);
    step = 16 * ld;
    rows = 0;
#pragma unroll
    for (int i = 0; i < TM / 16; ++i) rows |= (unsigned)(r + 16 * i < n_rows) << i;
  }
  // columns [k0, k0 + 16), of which `left` exist; then moves on
  __device__ __forceinline__ void stage(float* s, int left, const float* any, int tid) {
    float* d = s + (tid & 15) * PITCH + (tid >> 4);
    const unsigned ok = (tid & 15) < left ? rows : 0u;
    const float* q = p;
#pragma unroll
    for (int i = 0; i < TM / 16; ++i) {
      const bool in = ok >> i & 1;
      copy<4>(d + 16 * i, in ? q : any, in);
      q += step;
    }
    p += TK;
  }
};

// Rows [k0, k0 + 16) x columns [c0, c0 + 128) of a matrix [K][cols].
__device__ __forceinline__ void stage_cols(float* s, const float* base, long long ld, int c0,
                                           int cols, int k0, int k_hi, bool vec, int tid) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = (tid >> 5) + 8 * i, c = (tid & 31) * 4;
      const bool row = k0 + k < k_hi;
      if (c0 + c + 4 <= cols || !row || c0 + c >= cols) {
        const bool ok = row && c0 + c < cols;
        copy<16>(s + k * PITCH + c, ok ? base + (long long)(k0 + k) * ld + c0 + c : base, ok);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool ok = c0 + c + e < cols;
          copy<4>(s + k * PITCH + c + e, ok ? base + (long long)(k0 + k) * ld + c0 + c + e : base,
                  ok);
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = (tid >> 7) + 2 * i, c = tid & 127;
      const bool ok = k0 + k < k_hi && c0 + c < cols;
      copy<4>(s + k * PITCH + c, ok ? base + (long long)(k0 + k) * ld + c0 + c : base, ok);
    }
  }
}

template <bool BWD>
__global__ void __launch_bounds__(kThreads, 2) linear_f32_kernel(const LinearArgs a, int k_per,
                                                                 int w_vec) {
  extern __shared__ __align__(16) float smem[];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const unsigned tiles_n = (a.N + TN - 1) / TN, tm = blockIdx.x / tiles_n;
  const long long r0 = (long long)tm * TM;
  const int c0 = (int)(blockIdx.x - tm * tiles_n) * TN;
  const int k_lo = blockIdx.y * k_per, k_hi = min(a.K, k_lo + k_per);
  const float* x = static_cast<const float*>(a.x);
  // of two products of the same x: the second's weight and planes
  const bool second = !BWD && blockIdx.z;
  const float* w = static_cast<const float*>(second ? a.w2 : a.w);
  const long long ldw = second ? a.ldw2 : a.ldw;
  RowStager xs(x, a.ldx, r0, a.T, k_lo, tid);
  RowStager wr(w, ldw, c0, BWD ? a.N : 0, k_lo, tid);
  auto stage = [&](int st, int k0) {
    float* sa = smem + st * 2 * TK * PITCH;
    float* sb = sa + TK * PITCH;
    if (k0 < k_hi) {
      xs.stage(sa, k_hi - k0, x, tid);
      if constexpr (BWD) wr.stage(sb, k_hi - k0, w, tid);
      else stage_cols(sb, w, ldw, c0, a.N, k0, k_hi, w_vec, tid);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // rows ty * 4 + {0..3} and 64 + ty * 4 + {0..3}; columns alike from tx
  F2 acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f2(0.f);
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) stage(s, k_lo + s * TK);
  int st = 0;
  for (int k0 = k_lo; k0 < k_hi; k0 += TK) {
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
    __syncthreads();  // this stage has landed for all; the one before is free
    stage(st == 0 ? STAGES - 1 : st - 1, k0 + (STAGES - 1) * TK);
    const float* sa = smem + st * 2 * TK * PITCH + ty * 4;
    const float* sb = smem + (st * 2 + 1) * TK * PITCH + tx * 4;
#pragma unroll
    for (int k = 0; k < TK; ++k) {
      const float4 a0 = *reinterpret_cast<const float4*>(sa + k * PITCH);
      const float4 a1 = *reinterpret_cast<const float4*>(sa + k * PITCH + 64);
      const float4 b0 = *reinterpret_cast<const float4*>(sb + k * PITCH);
      const float4 b1 = *reinterpret_cast<const float4*>(sb + k * PITCH + 64);
      const float av[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
      const F2 bv[4] = {f2(b0.x, b0.y), f2(b0.z, b0.w), f2(b1.x, b1.y), f2(b1.z, b1.w)};
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fma2(f2(av[i]), bv[j], acc[i][j]);
    }
    st = st + 1 == STAGES ? 0 : st + 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  // planes have whole 32-column pieces (ldp a multiple of 32): only whole
  // quads past ldp are left out
  float* out = a.partial + (long long)(blockIdx.z * gridDim.y + blockIdx.y) * a.T * a.ldp;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const long long r = r0 + (i < 4 ? 0 : 64) + ty * 4 + (i & 3);
    if (r >= a.T) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = c0 + 64 * h + tx * 4;
      if (c < a.ldp)
        *reinterpret_cast<float4*>(out + r * a.ldp + c) =
            make_float4(acc[i][2 * h].x, acc[i][2 * h].y, acc[i][2 * h + 1].x,
                        acc[i][2 * h + 1].y);
    }
  }
}

}  // namespace

// The split of K with the smallest estimated time (cycles): rounds of blocks
// over 304 places, each k taking an SM 260 cycles with one block on it and 380
// with two (49 and 67 % of the FMA rate), and the raw sums' way through memory
// and the pass that adds them, four planes at a time.
int linear_f32_splits(long long T, int K, int N, int products) {
  const long long tiles = (T + TM - 1) / TM * ((N + TN - 1) / TN) * products;
  int best = 1;
  double best_cycles = 1e300;
  for (int s = 1; s <= 32; ++s) {
    if (s > 1 && s > K / 64) break;
    const int per = ((K + s - 1) / s + TK - 1) / TK * TK;
    const int splits = (K + per - 1) / per;
    const long long blocks = tiles * splits, waves = (blocks + 303) / 304;
    const double cycles = (blocks <= 152 ? 260. : waves * 380.) * per + waves * 6000. +
                          splits * (double)T * N * products * 8 / 3000 + (splits + 3) / 4 * 1500.;
    if (cycles < best_cycles) {
      best_cycles = cycles;
      best = splits;
    }
  }
  return best;
}

mlp_status launch_linear_f32(const LinearArgs& a, bool bwd, cudaStream_t st) {
  const long long tiles = (a.T + TM - 1) / TM * ((a.N + TN - 1) / TN);
  if (tiles > 0x7fffffffll) return MLP_ERR_UNSUPPORTED_SHAPE;
  const dim3 grid((unsigned)tiles, a.splits, a.w2 ? 2 : 1);
  const int per = ((a.K + a.splits - 1) / a.splits + TK - 1) / TK * TK;
  const int w_vec = reinterpret_cast<uintptr_t>(a.w) % 16 == 0 && a.ldw % 4 == 0 &&
                    (!a.w2 || (reinterpret_cast<uintptr_t>(a.w2) % 16 == 0 && a.ldw2 % 4 == 0));
  auto kernel = bwd ? linear_f32_kernel<true> : linear_f32_kernel<false>;
  static PerDevice configured[2];
  if (!allow_smem(configured[bwd], kernel, kSmem)) return MLP_ERR_CUDA;
  LaunchScope ls(bwd ? "linear_bwd_f32" : "linear_fwd_f32", st, a.T, a.N, a.K);
  launch_k(kernel, grid, dim3(kThreads), kSmem, st, a, per, w_vec);
  return launch_status();
}

}  // namespace mlp
