// Linear layers outside the tensor-core tiles (formulas: k_linear.cu): the
// one-launch kernel for a few rows (single tokens), and the epilogue as a pass
// of its own over raw sums (split-K partial planes, fp32 products) or over dy
// (the activation's backward without a product).
//
// In both a warp finishes 32 columns of a row at a time, one per lane: memory
// is touched in whole rows of 32 values and a group of the 8-bit form is one
// warp, its largest magnitude one warp reduction.
#include "act.cuh"
#include "ckpt8.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "rowvec.cuh"
#include "trace.cuh"

namespace mlp {

namespace {

constexpr int kThreads = 256;

// What the epilogue of element (m, c) reads beside the raw sum: the residual
// (forward) or the saved pre-activation (backward).
template <typename T, bool BWD>
__device__ __forceinline__ float epi_load(const LinearArgs& a, long long m, int c, bool ok) {
  if (!ok) return 0.f;
  if constexpr (BWD) {
    if (a.q) return (float)a.q[m * a.ldq + c] * ckpt8_step(a.scale[m * a.lds + c / kCkptGroup]);
    if (a.u_in) return to_f32(static_cast<const T*>(a.u_in)[m * a.ldu_in + c]);
  } else if (a.res) {
    return a.out_f32 ? static_cast<const float*>(a.res)[m * a.ldr + c]
                     : to_f32(static_cast<const T*>(a.res)[m * a.ldr + c]);
  }
  return 0.f;
}

// Finishes element (m, c) from its raw sum; whole warps, lane = column of a
// 32-column group.  Returns the stored value before rounding.
template <typename T, bool BWD>
__device__ __forceinline__ float epi_finish(const LinearArgs& a, long long m, int c, bool ok,
                                            float v, float bias, float extra) {
  constexpr bool ACC = sizeof(T) == 4;  // fp32 layers: the exact functions
  if constexpr (!BWD) {
    v += bias;
    if (a.u_out && ok) from_f32(v, static_cast<T*>(a.u_out)[m * a.ldu_out + c]);
    if (a.q) {
      const uint32_t top =
          __reduce_max_sync(0xffffffffu, ok ? __float_as_uint(v) & 0x7fffffffu : 0u);
      const uint32_t b = ckpt8_byte(top);
      const float held = ckpt8_must_hold(top) ? ckpt8_hold(v, ckpt8_step(b)) : v;
      if (ok)
        a.q[m * a.ldq + c] =
            b == kCkptNanByte ? (int8_t)0 : (int8_t)ckpt8_q(held, ckpt8_inv_step(b));
      if ((c & (kCkptGroup - 1)) == 0 && ok) a.scale[m * a.lds + c / kCkptGroup] = (uint8_t)b;
    }
    with_act(a.act, [&](auto tag) {
      v = act_value_of<ACC, decltype(tag)::value>(v, a.slope) + extra;
    });
  } else if (a.act != MLP_ACT_NONE || a.u_out) {
    float f = 0.f;
    with_act(a.act, [&](auto tag) {
      v *= act_grad_of<ACC, decltype(tag)::value>(extra, a.slope, f);
    });
    if (a.u_out && ok) from_f32(f, static_cast<T*>(a.u_out)[m * a.ldu_out + c]);
  }
  if (ok) {
    if (a.out_f32) static_cast<float*>(a.y)[m * a.ldy + c] = v;
    else from_f32(v, static_cast<T*>(a.y)[m * a.ldy + c]);
  }
  return v;
}

// ------------------------------------------------------------ epilogue pass

constexpr int kRowsAhead = 4;  // rows loaded before the first is finished
constexpr int kUnitRows = 32;  // rows of a backward unit (one row of colpart)

// Warp unit: `unit_rows` rows of 32 columns; in the backward 32 rows, whose
// column sums it adds in row order into one row of colpart.
template <typename T, bool BWD, bool ELT>
__global__ void __launch_bounds__(kThreads) linear_finish_kernel(const LinearArgs a, int groups,
                                                                 int unit_rows,
                                                                 long long units) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (unit >= units) return;
  const long long rb = unit / groups;
  const int c = (int)(unit - rb * groups) * 32 + lane;
  const bool ok = c < a.N;
  const long long m_end = min(a.T, (rb + 1) * unit_rows);
  const float bias = !BWD && a.bias && ok ? __ldg(a.bias + c) : 0.f;
  float sum = 0.f;
  for (long long m0 = rb * unit_rows; m0 < m_end; m0 += kRowsAhead) {
    float v[kRowsAhead], extra[kRowsAhead];
#pragma unroll
    for (int k = 0; k < kRowsAhead; ++k) {
      const bool in = ok && m0 + k < m_end;
      if constexpr (ELT) {
        v[k] = in ? to_f32(static_cast<const T*>(a.x)[(m0 + k) * a.ldx + c]) : 0.f;
      } else {
        v[k] = 0.f;
        if (in) {
          const float* p = a.partial + (m0 + k) * a.ldp + c;
          for (int s = 0; s < a.splits; ++s) v[k] += __ldcs(p + (long long)s * a.T * a.ldp);
        }
      }
      extra[k] = epi_load<T, BWD>(a, m0 + k, c, in);
    }
#pragma unroll
    for (int k = 0; k < kRowsAhead; ++k) {
      if (m0 + k >= m_end) break;  // warp-uniform
      v[k] = epi_finish<T, BWD>(a, m0 + k, c, ok, v[k], bias, extra[k]);
      sum += v[k];
    }
  }
  if (BWD && a.colpart && ok) a.colpart[rb * a.ldcp + c] = sum;
}

// ------------------------------------------------------------ a few rows
//
// Up to 8 rows: bound by reading W once.  A cluster of S CTAs takes 64 or 128
// output columns, each CTA one slice of K; the S partial results meet in
// distributed shared memory and the cluster's warps run the epilogue, so the
// call is one launch without a workspace.  Each CTA: 256 threads, 16-byte
// loads of W straight to registers (every element is used by this CTA alone;
// shared memory would only add a hop), the rows of x in shared memory as fp32.
//   forward, W [K][N]: a thread keeps 16 bytes of columns and walks down K
//   (256-byte runs of W per 128 columns), the next loads in flight while the
//   last are used;
//   backward, W [N][K]: a warp keeps 8 of the 64 columns and its lanes walk
//   along K.
// All CTAs of a launch are resident at once: a second wave of a few would
// double the time.

constexpr int kFewX = 4096;  // values of x staged at a time (all rows)

// CTAs that an SM holds (by registers), and the K values staged at a time.
template <int MT, bool BWD>
struct FewShape {
  static constexpr int kPerSm = (MT == 1 ? 4 : MT == 2 ? 3 : MT == 4 ? 3 : 2) - (BWD ? 1 : 0);
  static constexpr int kChunk = kFewX / MT;
};

// Sums of V <= 32 values over the warp's lanes: lane L gets that of value
// L % V.  Halving rounds as in a transposition, then a butterfly.
template <int V>
__device__ __forceinline__ float lane_sums(float (&v)[V], int lane) {
#pragma unroll
  for (int o = V / 2; o > 0; o >>= 1) {
    const bool upper = lane & o;
#pragma unroll
    for (int j = 0; j < o; ++j) {
      const float give = upper ? v[j] : v[j + o];
      const float keep = upper ? v[j + o] : v[j];
      v[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
#pragma unroll
  for (int o = V; o < 32; o <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  return v[0];
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

template <typename T, int MT, bool BWD, int COLS>
__global__ void __launch_bounds__(kThreads, FewShape<MT, BWD>::kPerSm)
    linear_few_kernel(const LinearArgs a, int cluster, int slice, int w_vec, float* dbias) {
  constexpr int N = RowVec<T>::N;
  constexpr int LPR = COLS / N < 32 ? COLS / N : 32;  // forward: lanes across the columns
  constexpr int KP = kThreads / LPR;                  // forward: rows of W per step
  constexpr int U = 4;                                // loads a thread issues together
  constexpr int CHUNK = FewShape<MT, BWD>::kChunk;
  static_assert(LPR * N == COLS && (!BWD || COLS == 64), "columns of a CTA");
  __shared__ __align__(16) float xs[CHUNK * MT];   // forward [k][MT], backward [MT][k]
  __shared__ float red[BWD ? 1 : 8 * MT * COLS];   // forward: [warp][MT][COLS]
  __shared__ float part[MT * COLS];                // this CTA's sums, read by the cluster
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % cluster;
  const int c0 = (int)(blockIdx.x / cluster) * COLS;
  const int k_lo = rank * slice, k_hi = min(a.K, k_lo + slice);
  const T* x = static_cast<const T*>(a.x);
  const T* w = static_cast<const T*>(a.w);

  constexpr int V = BWD ? 8 : N;  // columns per thread
  float acc[MT][V];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < V; ++j) acc[m][j] = 0.f;

  for (int kc = k_lo; kc < k_hi; kc += CHUNK) {
    const int len = min(CHUNK, k_hi - kc);
    if (kc > k_lo) __syncthreads();  // the previous chunk has been read
    auto stage_x = [&] {
#pragma unroll 4
      for (int i = tid; i < len * MT; i += kThreads) {
        const int m = MT == 1 ? 0 : i / len, k = i - m * len;  // coalesced along k
        xs[BWD ? m * CHUNK + k : k * MT + m] = m < a.T ? to_f32(x[m * a.ldx + kc + k]) : 0.f;
      }
      if (BWD)  // the last piece of a row of W may reach past K; its x reads as zero
        for (int i = tid; i < MT * N; i += kThreads)
          if (len + i % N < CHUNK) xs[i / N * CHUNK + len + i % N] = 0.f;
      __syncthreads();
    };
    if constexpr (!BWD) {
      const int c = c0 + (tid % LPR) * N;
      const int cols = a.N - c;
      const T* wp = w + (long long)(kc + tid / LPR) * a.ldw + c;
      uint4 raw[U];
      auto load = [&](int k0) {
#pragma unroll
        for (int i = 0; i < U; ++i)
          raw[i] = load_piece(wp + (long long)(k0 + i * KP) * a.ldw,
                              k0 + tid / LPR + i * KP < len ? cols : 0, w_vec);
      };
      load(0);
      stage_x();
      for (int k0 = 0; k0 < len; k0 += KP * U) {
        uint4 cur[U];
#pragma unroll
        for (int i = 0; i < U; ++i) cur[i] = raw[i];
        if (k0 + KP * U < len) load(k0 + KP * U);
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int k = k0 + tid / LPR + i * KP;
          if (k >= len) break;
          float wv[N], xv[MT];
          unpack_piece<T>(cur[i], wv);
#pragma unroll
          for (int m = 0; m < MT; ++m) xv[m] = xs[k * MT + m];
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < N; ++j) acc[m][j] = fmaf(xv[m], wv[j], acc[m][j]);
        }
      }
    } else {
      // steps of four of the warp's eight columns and 32 N of K
      uint4 raw[4];
      auto load = [&](int k, int h) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = c0 + warp * 8 + h + j;
          raw[j] = load_piece(w + (long long)c * a.ldw + kc + k, c < a.N ? len - k : 0, w_vec);
        }
      };
      load(lane * N, 0);
      stage_x();
      for (int k = lane * N; k < len; k += 32 * N) {
#pragma unroll
        for (int h = 0; h < 8; h += 4) {
          float wv[4][N];
#pragma unroll
          for (int j = 0; j < 4; ++j) unpack_piece<T>(raw[j], wv[j]);
          if (h == 0) load(k, 4);
          else if (k + 32 * N < len) load(k + 32 * N, 0);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            float xv[N];
#pragma unroll
            for (int e = 0; e < N; e += 4) {
              const float4 f = *reinterpret_cast<const float4*>(xs + m * CHUNK + k + e);
              xv[e] = f.x;
              xv[e + 1] = f.y;
              xv[e + 2] = f.z;
              xv[e + 3] = f.w;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int e = 0; e < N; ++e) acc[m][h + j] = fmaf(xv[e], wv[j][e], acc[m][h + j]);
          }
        }
      }
    }
  }

  // this CTA's sums into part[m][column]
  if constexpr (!BWD) {
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
  } else {
    // four rows (32 values) at a time
    constexpr int MB = MT < 4 ? MT : 4;
#pragma unroll
    for (int mb = 0; mb < MT; mb += MB) {
      float v[MB * 8];
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[m * 8 + j] = acc[mb + m][j];
      const float s = lane_sums<MB * 8>(v, lane);
      if (lane < MB * 8) part[(mb + lane / 8) * COLS + warp * 8 + lane % 8] = s;
    }
  }
  ptx::cluster_sync();  // every CTA's sums are in place (a cluster of one: a block barrier)

  // Epilogue: (row, 32-column group) units dealt over the cluster's warps; in
  // the backward a unit takes all rows, so it also has the column sums.
  const uint32_t part0 = ptx::smem_u32(part);
  constexpr int G = COLS / 32;
  const int units = BWD ? G : G * (int)a.T;
  for (int u = rank + cluster * warp; u < units; u += cluster * (kThreads / 32)) {
    const int g = u % G;
    const int c = c0 + g * 32 + lane;
    if (c0 + g * 32 >= a.N) continue;  // warp-uniform
    const bool ok = c < a.N;
    const float bias = !BWD && a.bias && ok ? __ldg(a.bias + c) : 0.f;
    float sum = 0.f;
    const int m_lo = BWD ? 0 : u / G, m_hi = BWD ? (int)a.T : m_lo + 1;
    for (int m = m_lo; m < m_hi; ++m) {
      const float extra = epi_load<T, BWD>(a, m, c, ok);
      float v = 0.f;
      for (int r = 0; r < cluster; ++r)  // in slice order
        v += ld_cluster_f32(ptx::mapa_shared(
            part0 + (uint32_t)(m * COLS + g * 32 + lane) * 4u, (uint32_t)r));
      sum += epi_finish<T, BWD>(a, m, c, ok, v, bias, extra);
    }
    if (BWD && dbias && ok) dbias[c] = sum;
  }
  ptx::cluster_sync();  // no CTA leaves while its sums may still be read
}

template <typename T, int MT, bool BWD, int COLS>
mlp_status few_launch(const LinearArgs& a, float* dbias, cudaStream_t st) {
  // the widest cluster with which all CTAs are resident (on 152 SMs) and each
  // still has 128 of K
  const long long tiles = (a.N + COLS - 1) / COLS;
  int cluster = 8;
  while (cluster > 1 &&
         (tiles * cluster > 152 * FewShape<MT, BWD>::kPerSm || a.K < 128 * cluster))
    --cluster;
  const int per = (a.K + cluster - 1) / cluster;
  const int slice = (per + 63) / 64 * 64;  // slices start on whole 16-byte pieces
  if (tiles * cluster > 0x7fffffffll) return MLP_ERR_UNSUPPORTED_SHAPE;
  const int w_vec = reinterpret_cast<uintptr_t>(a.w) % 16 == 0 && a.ldw * sizeof(T) % 16 == 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  LaunchScope ls(BWD ? "linear_bwd_few" : "linear_fwd_few", st, a.T, a.N, a.K);
  cudaLaunchKernelEx(&cfg, linear_few_kernel<T, MT, BWD, COLS>, a, cluster, slice, w_vec, dbias);
  return launch_status();
}

template <typename T, int MT, bool BWD>
mlp_status few_cols(const LinearArgs& a, float* dbias, cudaStream_t st) {
  // 128 columns a cluster (longer runs of W) where they still give enough CTAs
  if constexpr (!BWD && MT <= 4) {
    if ((long long)a.N / 128 * 8 >= 304) return few_launch<T, MT, BWD, 128>(a, dbias, st);
  }
  return few_launch<T, MT, BWD, 64>(a, dbias, st);
}

template <typename T, bool BWD>
mlp_status few_rows(const LinearArgs& a, float* dbias, cudaStream_t st) {
  if (a.T <= 1) return few_cols<T, 1, BWD>(a, dbias, st);
  if (a.T <= 2) return few_cols<T, 2, BWD>(a, dbias, st);
  if (a.T <= 4) return few_cols<T, 4, BWD>(a, dbias, st);
  return few_cols<T, 8, BWD>(a, dbias, st);
}

template <typename T, bool BWD, bool ELT>
mlp_status finish_launch(const LinearArgs& a, cudaStream_t st) {
  const int groups = (a.N + 31) / 32;
  const int unit_rows = BWD ? kUnitRows : kRowsAhead;
  const long long units = (a.T + unit_rows - 1) / unit_rows * groups;
  const long long blocks = (units + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7fffffffll) return MLP_ERR_UNSUPPORTED_SHAPE;
  LaunchScope ls(ELT ? "act_bwd" : BWD ? "linear_bwd_finish" : "linear_fwd_finish", st, a.T, a.N,
                 a.splits);
  launch_k(linear_finish_kernel<T, BWD, ELT>, dim3((unsigned)blocks), dim3(kThreads), 0, st, a,
           groups, unit_rows, units);
  return launch_status();
}

template <typename T>
mlp_status finish_t(const LinearArgs& a, bool bwd, bool elementwise, cudaStream_t st) {
  if (elementwise) return finish_launch<T, true, true>(a, st);
  return bwd ? finish_launch<T, true, false>(a, st) : finish_launch<T, false, false>(a, st);
}

}  // namespace

mlp_status launch_linear_few(const LinearArgs& a, bool bwd, float* dbias, cudaStream_t st) {
  switch (a.dtype) {
    case MLP_DTYPE_BF16:
      return bwd ? few_rows<__nv_bfloat16, true>(a, dbias, st)
                 : few_rows<__nv_bfloat16, false>(a, nullptr, st);
    case MLP_DTYPE_F16:
      return bwd ? few_rows<__half, true>(a, dbias, st) : few_rows<__half, false>(a, nullptr, st);
    default:
      return bwd ? few_rows<float, true>(a, dbias, st) : few_rows<float, false>(a, nullptr, st);
  }
}

mlp_status launch_linear_finish(const LinearArgs& a, bool bwd, bool elementwise, cudaStream_t st) {
  switch (a.dtype) {
    case MLP_DTYPE_BF16: return finish_t<__nv_bfloat16>(a, bwd, elementwise, st);
    case MLP_DTYPE_F16: return finish_t<__half>(a, bwd, elementwise, st);
    default: return finish_t<float>(a, bwd, elementwise, st);
  }
}

}  // namespace mlp
