// Gated units outside the tensor-core tiles (formulas: k_glu.cu, k_glu_bwd.cu):
// the one-launch kernel for a few rows (single tokens), and the epilogues as
// passes of their own over raw sums (split-K partial planes, fp32 products).
// A warp finishes 32 columns of a row at a time, one per lane: memory is
// touched in whole rows of 32 values and a group of the 8-bit form is one warp.
// The passes are bound by latency and issue, so an address costs one widening
// multiplication.  Whole fp32 calls of 784 and 1,001 columns with cold caches, against
// a 64-bit product for every element: 1,003 rows forward 87.6 and 87.2 us, backward
// 51 and 52; 129 rows 28.6 and 37.7, 18.2 and 19.8.
#include "act.cuh"
#include "ckpt8.cuh"
#include "few_rows.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "rowvec.cuh"
#include "trace.cuh"

namespace mlp {

namespace {

constexpr int kThreads = 256;
constexpr int kRowsAhead = 4;  // rows loaded before the first is finished

// Value at column c of row m (pitches are ints at the C boundary: one widening
// multiplication).
template <typename T>
__device__ __forceinline__ T* at(void* base, long long ld, long long m, int c) {
  return static_cast<T*>(base) + ((unsigned long long)(uint32_t)m * (uint32_t)ld + (uint32_t)c);
}
template <typename T>
__device__ __forceinline__ const T* at(const void* base, long long ld, long long m, int c) {
  return static_cast<const T*>(base) +
         ((unsigned long long)(uint32_t)m * (uint32_t)ld + (uint32_t)c);
}

// Element (m, c) of kept matrix k: the pre-activation z in the operand type or
// in 8 bits (whole warps, lane = column of a 32-column group).
template <typename T>
__device__ __forceinline__ void keep(const GluArgs& a, int k, long long m, int c, bool ok,
                                     float z) {
  if (a.o[k]) {
    if (ok) from_f32(z, *at<T>(a.o[k], a.ldo[k], m, c));
  } else if (a.q[k]) {
    const uint32_t top =
        __reduce_max_sync(0xffffffffu, ok ? __float_as_uint(z) & 0x7fffffffu : 0u);
    const uint32_t b = ckpt8_byte(top);
    if (ok) {
      const float held = ckpt8_must_hold(top) ? ckpt8_hold(z, ckpt8_step(b)) : z;
      *at<int8_t>(a.q[k], a.ldq[k], m, c) =
          b == kCkptNanByte ? (int8_t)0 : (int8_t)ckpt8_q(held, ckpt8_inv_step(b));
    }
    if ((c & 31) == 0) *at<uint8_t>(a.scale[k], a.lds[k], m, c / kCkptGroup) = (uint8_t)b;
  }
}

// Forward outputs of element (m, c) from its raw sums.
template <typename T, int ACT>
__device__ __forceinline__ void glu_out(const GluArgs& a, long long m, int c, bool ok, float g,
                                        float u, float bg, float bu) {
  g += bg;
  u += bu;
  keep<T>(a, 0, m, c, ok, g);
  keep<T>(a, 1, m, c, ok, u);
  const float y = act_value_of<sizeof(T) == 4, ACT>(g, a.slope) * u;
  if (ok) from_f32(y, *at<T>(a.y, a.ldy, m, c));
}

__device__ __forceinline__ float bias_of(const float* b, int c, bool ok) {
  return b && ok ? __ldg(b + c) : 0.f;
}

// ------------------------------------------------------------ epilogue passes

// Sums of rows m0 .. m0 + rows - 1 at column c over the planes in order, four
// planes of all rows in flight.  (Planes have whole 32-column pieces, so lanes
// past the last column read as well.)
__device__ __forceinline__ void add_planes(const float* p, long long plane, int splits, int ldp,
                                           int rows, float (&v)[kRowsAhead]) {
#pragma unroll
  for (int k = 0; k < kRowsAhead; ++k) v[k] = 0.f;
#pragma unroll 1
  for (int s = 0; s < splits; s += 4, p += 4 * plane) {
    float q[4][kRowsAhead];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int k = 0; k < kRowsAhead; ++k)
        q[j][k] = s + j < splits && k < rows ? __ldcs(p + j * plane + k * ldp) : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int k = 0; k < kRowsAhead; ++k) v[k] += q[j][k];
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) glu_finish_fwd_kernel(const GluArgs a, int groups,
                                                                  long long units) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (unit >= units) return;
  const long long rb = unit / groups;
  const int c = (int)(unit - rb * groups) * 32 + lane;
  const bool ok = c < a.N;
  const long long m0 = rb * kRowsAhead, plane = a.T * a.ldp;
  const int rows = (int)min((long long)kRowsAhead, a.T - m0);
  const float bg = bias_of(a.bias[0], c, ok), bu = bias_of(a.bias[1], c, ok);
  float g[kRowsAhead], u[kRowsAhead];
  const float* p = a.partial + m0 * a.ldp + c;
  add_planes(p, plane, a.splits, (int)a.ldp, rows, g);
  add_planes(p + a.splits * plane, plane, a.splits, (int)a.ldp, rows, u);
  with_act(a.act, [&](auto tag) {
#pragma unroll
    for (int k = 0; k < kRowsAhead; ++k)
      if (k < rows)  // warp-uniform
        glu_out<T, decltype(tag)::value>(a, m0 + k, c, ok, g[k], u[k], bg, bu);
  });
}

// Warp unit: a.part_rows rows of 32 columns, whose column sums it adds in row
// order into one row of colpart.
template <typename T>
__global__ void __launch_bounds__(kThreads) glu_finish_bwd_kernel(const GluArgs a, int groups,
                                                                  long long units) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (unit >= units) return;
  const long long rb = unit / groups;
  const int c = (int)(unit - rb * groups) * 32 + lane;
  const bool ok = c < a.N;
  const long long m_end = min(a.T, (rb + 1) * a.part_rows), plane = a.T * a.ldp;
  float s0 = 0.f, s1 = 0.f;
  auto saved = [&](int k, long long m, bool in) {
    if (!in) return 0.f;
    if (a.q[k])
      return (float)*at<int8_t>(a.q[k], a.ldq[k], m, c) *
             ckpt8_step(*at<uint8_t>(a.scale[k], a.lds[k], m, c / kCkptGroup));
    return to_f32(*at<T>(a.in[k], a.ld_in[k], m, c));
  };
  with_act(a.act, [&](auto tag) {
    for (long long m0 = rb * a.part_rows; m0 < m_end; m0 += kRowsAhead) {
      const int rows = (int)min((long long)kRowsAhead, m_end - m0);
      float g[kRowsAhead], u[kRowsAhead], da[kRowsAhead];
#pragma unroll
      for (int k = 0; k < kRowsAhead; ++k) {
        g[k] = saved(0, m0 + k, ok && k < rows);
        u[k] = saved(1, m0 + k, ok && k < rows);
      }
      add_planes(a.partial + m0 * a.ldp + c, plane, a.splits, (int)a.ldp, rows, da);
#pragma unroll
      for (int k = 0; k < kRowsAhead; ++k) {
        if (k >= rows) break;  // warp-uniform
        const long long m = m0 + k;
        float f;
        const float df = act_grad_of<sizeof(T) == 4, decltype(tag)::value>(g[k], a.slope, f);
        const float dg = da[k] * (u[k] * df), du = da[k] * f;
        s0 += dg;
        s1 += du;
        if (ok) {
          from_f32(dg, *at<T>(a.o[0], a.ldo[0], m, c));
          from_f32(du, *at<T>(a.o[1], a.ldo[1], m, c));
          if (a.y) from_f32(f * u[k], *at<T>(a.y, a.ldy, m, c));
        }
      }
    }
  });
  if (a.colpart && ok) {
    float* o = a.colpart + rb * a.ldcp + c;
    o[0] = s0;
    o[a.N] = s1;
  }
}

// ------------------------------------------------------------ a few rows
//
// Up to 8 rows: bound by reading both weights once.  A cluster of S CTAs takes
// COLS accumulators, half of them gate and half up columns of the same hidden
// columns, each CTA one slice of K; the S partial results meet in distributed
// shared memory and the cluster's warps run the epilogue, so the call is one
// launch without a workspace.  Each CTA: 256 threads, each with a ring of
// 16-byte pieces of its weight that it alone fills (asynchronous copies) and
// reads, so the stream needs no barriers and the depth of the ring, not the
// registers, sets the bytes in flight; the rows of x are in shared memory as
// fp32.  A thread keeps 16 bytes of columns and walks down K (runs of 128 bytes
// of either weight per 128 accumulators in 16 bits).  All CTAs of a launch are
// resident at once up to 152 kPerSm tiles; more run on in further waves (clusters
// do not wait for one another).  8,192 -> 8,192 bf16, one row, back to back: 42.5 us, 6.3 TB/s;
// 512 -> 1,408 5 us from L2, 12 with cold caches.

constexpr int kFewX = 4096;  // values of x staged at a time (all rows)
constexpr int kFewRing = 8;  // pieces of a thread's ring

template <int MT, int COLS>
struct FewShape {
  static constexpr int kPerSm = MT <= 2 ? 4 : MT == 4 ? 3 : 2;  // CTAs an SM holds (registers)
  static constexpr int kChunk = kFewX / MT;
  // ring (the reduction takes its place), x, this CTA's sums
  static constexpr int kRing = kFewRing * kThreads * 16;
  static constexpr int kSmem = kRing + kFewX * 4 + MT * COLS * 4;
  static_assert(8 * MT * COLS * 4 <= kRing, "reduction in the ring's place");
};

template <typename T, int MT, int COLS>
__global__ void __launch_bounds__(kThreads, FewShape<MT, COLS>::kPerSm)
    glu_few_kernel(const GluArgs a, int cluster, int slice, int w_vec) {
  using Shape = FewShape<MT, COLS>;
  constexpr int N = RowVec<T>::N;
  constexpr int HALF = COLS / 2;      // hidden columns of a cluster
  constexpr int LPR = COLS / N;       // lanes across the accumulators
  constexpr int KP = kThreads / LPR;  // rows of the weights per step
  constexpr int CHUNK = Shape::kChunk;
  constexpr int D = kFewRing;
  static_assert(LPR <= 32 && HALF % 32 == 0, "columns of a CTA");
  static_assert(KP == 8 || LPR < 32, "a warp's lanes share a row");
  extern __shared__ __align__(16) uint8_t few_smem[];
  float* xs = reinterpret_cast<float*>(few_smem + Shape::kRing);  // [k][MT]
  float* red = reinterpret_cast<float*>(few_smem);                // [warp][MT][COLS]
  float* part = xs + kFewX;  // [MT][COLS]: this CTA's sums, read by the cluster
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint4* ring = reinterpret_cast<uint4*>(few_smem) + tid;  // slot i at [i * kThreads]
  pdl_wait();
  pdl_launch_dependents();
  const int rank = blockIdx.x % cluster;
  const int c0 = (int)(blockIdx.x / cluster) * HALF;
  const int k_lo = rank * slice, k_hi = min(a.K, k_lo + slice);
  const T* x = static_cast<const T*>(a.x);
  const int which = tid % LPR / (LPR / 2);  // gate or up
  const long long ldw = which ? a.ldw[1] : a.ldw[0];
  const int c = c0 + tid % (LPR / 2) * N, cols = a.N - c;
  const T* w = static_cast<const T*>(which ? a.w[1] : a.w[0]) + c;
  const int k_first = tid / LPR;

  float acc[MT][N];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < N; ++j) acc[m][j] = 0.f;

  for (int kc = k_lo; kc < k_hi; kc += CHUNK) {
    const int len = min(CHUNK, k_hi - kc);
    if (kc > k_lo) __syncthreads();  // the previous chunk has been read
    // step s: row k_first + s KP of the chunk
    const T* wp = w + (long long)(kc + k_first) * ldw;
    const long long step = (long long)KP * ldw;
    const int steps = (len - k_first + KP - 1) / KP;
    auto issue = [&](int st, int slot) {
      if (st < steps) few_issue(ring + slot * kThreads, wp + st * step, cols, w_vec);
      few_commit();
    };
#pragma unroll
    for (int i = 0; i < D - 1; ++i) issue(i, i);
#pragma unroll 4
    for (int i = tid; i < len * MT; i += kThreads) {
      const int m = MT == 1 ? 0 : i / len, k = i - m * len;  // coalesced along k
      xs[k * MT + m] = m < a.T ? to_f32(x[m * a.ldx + kc + k]) : 0.f;
    }
    __syncthreads();
    for (int s0 = 0; s0 < steps; s0 += D) {
#pragma unroll
      for (int i = 0; i < D; ++i) {
        few_wait<D - 2>();  // step s0 + i has landed
        if (s0 + i < steps) {
          F2 wv[N / 2];
          float xv[MT];
          unpack_piece<T>(ring[i * kThreads], wv);
          const float* xk = xs + (k_first + (s0 + i) * KP) * MT;
          if constexpr (MT >= 4) {
#pragma unroll
            for (int m = 0; m < MT; m += 4) {
              const float4 f = *reinterpret_cast<const float4*>(xk + m);
              xv[m] = f.x;
              xv[m + 1] = f.y;
              xv[m + 2] = f.z;
              xv[m + 3] = f.w;
            }
          } else {
#pragma unroll
            for (int m = 0; m < MT; ++m) xv[m] = xk[m];
          }
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < N; j += 2) {
              const F2 r = fma2(f2(xv[m]), wv[j / 2], f2(acc[m][j], acc[m][j + 1]));
              acc[m][j] = r.x;
              acc[m][j + 1] = r.y;
            }
        }
        issue(s0 + i + D - 1, (i + D - 1) % D);
      }
    }
    few_wait<0>();
  }

  // this CTA's sums into part[m][accumulator]
  __syncthreads();  // every thread is done with its ring
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < N; ++j) {
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) acc[m][j] += __shfl_xor_sync(0xffffffffu, acc[m][j], o);
      if (lane < LPR) red[(warp * MT + m) * COLS + lane * N + j] = acc[m][j];
    }
  __syncthreads();
  for (int i = tid; i < MT * COLS; i += kThreads) {
    float s = red[i];
#pragma unroll
    for (int q = 1; q < 8; ++q) s += red[q * MT * COLS + i];
    part[i] = s;
  }
  ptx::cluster_sync();  // every CTA's sums are in place (a cluster of one: a block barrier)

  // Epilogue: (row, 32-column group) units dealt over the cluster's warps.
  const uint32_t part0 = ptx::smem_u32(part);
  constexpr int G = HALF / 32;
  const int units = G * (int)a.T;
  for (int u = rank + cluster * warp; u < units; u += cluster * (kThreads / 32)) {
    const int m = u / G, g = u % G;
    if (c0 + g * 32 >= a.N) continue;  // warp-uniform
    const int cc = c0 + g * 32 + lane;
    const bool ok = cc < a.N;
    const float bg = bias_of(a.bias[0], cc, ok), bu = bias_of(a.bias[1], cc, ok);
    float z[2] = {0.f, 0.f};
    for (int r = 0; r < cluster; ++r)  // in slice order
#pragma unroll
      for (int k = 0; k < 2; ++k)
        z[k] += ld_cluster_f32(ptx::mapa_shared(
            part0 + (uint32_t)(m * COLS + k * HALF + g * 32 + lane) * 4u, (uint32_t)r));
    with_act(a.act, [&](auto tag) {
      glu_out<T, decltype(tag)::value>(a, m, cc, ok, z[0], z[1], bg, bu);
    });
  }
  ptx::cluster_sync();  // no CTA leaves while its sums may still be read
}

template <typename T, int MT, int COLS>
mlp_status few_launch(const GluArgs& a, cudaStream_t st) {
  using Shape = FewShape<MT, COLS>;
  static PerDevice configured;
  if (!allow_smem(configured, glu_few_kernel<T, MT, COLS>, Shape::kSmem)) return MLP_ERR_CUDA;
  // The widest cluster with which all CTAs are resident (on 152 SMs) and each still
  // has 64 of K; 1 where there are more tiles than places.  From the shape alone, as
  // the order of the sums follows from it.
  const long long tiles = (a.N + COLS / 2 - 1) / (COLS / 2);
  int cluster = 8;
  while (cluster > 1 && (tiles * cluster > 152 * Shape::kPerSm || a.K < 64 * cluster)) --cluster;
  const int per = (a.K + cluster - 1) / cluster;
  const int slice = (per + 63) / 64 * 64;
  if (tiles * cluster > 0x7fffffffll) return MLP_ERR_UNSUPPORTED_SHAPE;
  const int w_vec = aligned16(a.w[0]) && aligned16(a.w[1]) && a.ldw[0] * sizeof(T) % 16 == 0 &&
                    a.ldw[1] * sizeof(T) % 16 == 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Shape::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  LaunchScope ls("glu_fwd_few", st, a.T, a.N, a.K);
  cudaLaunchKernelEx(&cfg, glu_few_kernel<T, MT, COLS>, a, cluster, slice, w_vec);
  return launch_status();
}

// 128 accumulators a cluster, whose runs of the weights are longer (us with 128 and
// 64, one row, bf16: 512 -> 1,408 8.8 and 10.8, 4,096 -> 11,008 35.5 and 39.4, 8,192
// -> 8,192 47.6 and 53.8; four rows of the last 62 and 70); 64 for eight rows, whose
// sums would not fit the registers.
template <typename T>
mlp_status few_rows(const GluArgs& a, cudaStream_t st) {
  if (a.T <= 1) return few_launch<T, 1, 128>(a, st);
  if (a.T <= 2) return few_launch<T, 2, 128>(a, st);
  if (a.T <= 4) return few_launch<T, 4, 128>(a, st);
  return few_launch<T, 8, 64>(a, st);
}

template <typename T>
mlp_status finish_launch(const GluArgs& a, bool bwd, cudaStream_t st) {
  const int groups = (a.N + 31) / 32;
  const int unit_rows = bwd ? a.part_rows : kRowsAhead;
  const long long units = (a.T + unit_rows - 1) / unit_rows * groups;
  const long long blocks = (units + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7fffffffll) return MLP_ERR_UNSUPPORTED_SHAPE;
  LaunchScope ls(bwd ? "glu_bwd_finish" : "glu_fwd_finish", st, a.T, a.N, a.splits);
  launch_k(bwd ? glu_finish_bwd_kernel<T> : glu_finish_fwd_kernel<T>, dim3((unsigned)blocks),
           dim3(kThreads), 0, st, a, groups, units);
  return launch_status();
}

}  // namespace

// Up to 8 rows for fp32, whose tiled product computes 128 rows whatever T is (us
// here and there with cold weights: 784 -> 1,001, rows that start anywhere, T = 1 14.5
// and 15.5, 4 15.6 and 16.7, 8 10.6 and 15.9; 512 -> 1,408 T = 1 6.0 and 16.6, 8 7.4
// and 17.9; 4,096 -> 11,008 T = 1 71 and 397, 4 74 and 398, 8 148 and 399).
// In 16 bits the tensor cores take over once the FMAs, not the reading of the
// weights, bound this kernel: above 2 rows, 8 of small weights (us here and there
// with cold weights, bf16: 512 -> 1,408 T = 1 9 and 13, 4 11 and 13, 8 13 and 13; 1,024
// -> 2,816 T = 2 13 and 15, 4 15 and 15, 8 17 and 15; 8,192 -> 8,192 T = 1 48 and 54, 2
// 52 and 54, 3 62 and 54, 8 140 and 54).
bool glu_takes_few(long long T, int K, int N, int dtype) {
  if (dtype == MLP_DTYPE_F32) return T <= 8;
  return T <= 2 || (T <= 8 && (long long)K * N <= (1ll << 20));
}

mlp_status launch_glu_few(const GluArgs& a, cudaStream_t st) {
  switch (a.dtype) {
    case MLP_DTYPE_BF16: return few_rows<__nv_bfloat16>(a, st);
    case MLP_DTYPE_F16: return few_rows<__half>(a, st);
    default: return few_rows<float>(a, st);
  }
}

mlp_status launch_glu_finish(const GluArgs& a, bool bwd, cudaStream_t st) {
  switch (a.dtype) {
    case MLP_DTYPE_BF16: return finish_launch<__nv_bfloat16>(a, bwd, st);
    case MLP_DTYPE_F16: return finish_launch<__half>(a, bwd, st);
    default: return finish_launch<float>(a, bwd, st);
  }
}

}  // namespace mlp
