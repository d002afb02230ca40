// Linear layers outside the tensor-core tiles (formulas: k_linear.cu): the
// one-launch kernel for a few rows (single tokens), the epilogue as a pass of
// its own over raw sums (split-K partial planes, fp32 products), and the
// activation's backward without a product.
//
// In the first two a warp finishes 32 columns of a row at a time, one per
// lane: memory is touched in whole rows of 32 values and a group of the 8-bit
// form is one warp, its largest magnitude one warp reduction.
#include <type_traits>

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
template <typename T, bool BWD, int ACT>
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
    v = act_value_of<ACC, ACT>(v, a.slope) + extra;
  } else if (ACT != MLP_ACT_NONE || a.u_out) {
    float f;
    v *= act_grad_of<ACC, ACT>(extra, a.slope, f);
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

// Warp unit: `unit_rows` rows of 32 columns; in the backward it adds their
// column sums in row order into one row of colpart.  Bound by reading the
// planes (26,823 x 354 fp32, five planes, GELU: 88 us, the issue slots 75 %
// taken), or by latency for the few rows that are split most (168 x 325, 15
// planes: 10 us with cold caches).
template <typename T, bool BWD>
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
  with_act(a.act, [&](auto tag) {
    for (long long m0 = rb * unit_rows; m0 < m_end; m0 += kRowsAhead) {
      float v[kRowsAhead], extra[kRowsAhead];
#pragma unroll
      for (int k = 0; k < kRowsAhead; ++k) {
        v[k] = 0.f;
        extra[k] = epi_load<T, BWD>(a, m0 + k, c, ok && m0 + k < m_end);
      }
      // planes in order, four of all rows at a time in flight
      const float* p = a.partial + m0 * a.ldp + c;
      const long long plane = a.T * a.ldp;
#pragma unroll 1
      for (int s = 0; s < a.splits; s += 4) {
        float q[kRowsAhead][4];
#pragma unroll
        for (int k = 0; k < kRowsAhead; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            q[k][j] = ok && m0 + k < m_end && s + j < a.splits
                          ? __ldcs(p + (s + j) * plane + k * a.ldp)
                          : 0.f;
#pragma unroll
        for (int k = 0; k < kRowsAhead; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j) v[k] += q[k][j];
      }
#pragma unroll
      for (int k = 0; k < kRowsAhead; ++k) {
        if (m0 + k >= m_end) break;  // warp-uniform
        v[k] = epi_finish<T, BWD, decltype(tag)::value>(a, m0 + k, c, ok, v[k], bias, extra[k]);
        sum += v[k];
      }
    }
  });
  if (BWD && a.colpart && ok) a.colpart[rb * a.ldcp + c] = sum;
}

// ------------------------------------------------------------ activation backward
//
// du = dy f'(u), a = f(u) and partial column sums: bound by HBM.  A warp takes
// 32 (8) rows of 32 V columns, V per lane: four where all rows keep them aligned
// (8- and 16-byte accesses), else one (whole 32-value runs at any alignment).
// Two batches of rows are in flight: the next one's loads are issued before
// this one's arithmetic.  Measured with GELU (tanh) and column sums: 65,536 x
// 1,536 bf16 108 us (5.6 TB/s), fp32 188 (6.4 TB/s); 10,007 x 1,001 fp32, a
// value per lane and 64 instructions each, 27 (4.4 TB/s, the issue slots 75 %
// taken; with one batch at a time 52).

// V neighbouring values as they lie in memory, in whole registers.
template <typename T, int V>
union Cols {
  static constexpr int BYTES = sizeof(T) * V, WORDS = (BYTES + 3) / 4;
  uint32_t w[WORDS];
  T t[V];
  __device__ __forceinline__ Cols() {}
  // Nothing computed from the words moves to before this point.  (The compiler
  // converts 16-bit values where they are loaded, and so waits for the load.)
  __device__ __forceinline__ void pin() {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) asm volatile("" : "+r"(w[i]));
  }
};

// ... of which the first n exist (none where the row does not); V > 1 only
// where rows keep them aligned.
template <typename T, int V>
__device__ __forceinline__ Cols<T, V> load_cols(const T* p, bool in, int n) {
  using C = Cols<T, V>;
  C r;
#pragma unroll
  for (int i = 0; i < C::WORDS; ++i) r.w[i] = 0u;
  if (in && n >= V) {
    if constexpr (C::BYTES == 16) {
      const uint4 q = *reinterpret_cast<const uint4*>(p);
      r.w[0] = q.x, r.w[1] = q.y, r.w[2] = q.z, r.w[3] = q.w;
    } else if constexpr (C::BYTES == 8) {
      const uint2 q = *reinterpret_cast<const uint2*>(p);
      r.w[0] = q.x, r.w[1] = q.y;
    } else if constexpr (C::BYTES == 4) {
      r.w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (C::BYTES == 2) {
      r.w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else {
      r.w[0] = *reinterpret_cast<const uint8_t*>(p);
    }
  } else if (V > 1 && in) {
#pragma unroll
    for (int j = 0; j < V - 1; ++j)
      if (j < n) r.t[j] = p[j];
  }
  return r;
}
template <typename T, int V>
__device__ __forceinline__ void store_cols(T* p, int n, const float (&v)[V]) {
  using C = Cols<T, V>;
  C r;
#pragma unroll
  for (int j = 0; j < V; ++j) from_f32(v[j], r.t[j]);
  if (n >= V) {
    if constexpr (C::BYTES == 16)
      *reinterpret_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    else if constexpr (C::BYTES == 8) *reinterpret_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
    else *p = r.t[0];
  } else {
#pragma unroll
    for (int j = 0; j < V - 1; ++j)
      if (j < n) p[j] = r.t[j];
  }
}

template <typename T, int V, bool CK>
__global__ void __launch_bounds__(kThreads, 3) act_bwd_kernel(const LinearArgs a, int groups,
                                                              long long units) {
  constexpr bool ACC = sizeof(T) == 4;
  constexpr int R = V > 1 && ACC ? 2 : 4;  // rows of a batch
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (unit >= units) return;
  const long long rb = unit / groups;
  const int c = ((int)(unit - rb * groups) * 32 + lane) * V;
  const int n = a.N - c;  // this lane's columns that exist
  const long long m0 = rb * a.part_rows;
  const int rows = (int)min((long long)a.part_rows, a.T - m0);
  const bool has_u = CK || a.u_in != nullptr;
  // pitches are ints at the C boundary: products with a row number are one
  // widening multiplication
  const int ldx = (int)a.ldx, ldu = (int)a.ldu_in, ldq = (int)a.ldq, lds = (int)a.lds;
  const int ldy = (int)a.ldy, ldo = (int)a.ldu_out;
  const T* dy = static_cast<const T*>(a.x) + m0 * ldx + c;
  const T* u = static_cast<const T*>(a.u_in) + m0 * ldu + c;
  const int8_t* q = a.q + m0 * ldq + c;
  const uint8_t* sc = a.scale + m0 * lds + c / kCkptGroup;
  T* du = static_cast<T*>(a.y) + m0 * ldy + c;
  T* ao = static_cast<T*>(a.u_out) + m0 * ldo + c;
  // A batch as it lies in memory: whatever is computed from a load waits for
  // it, so nothing is until the batch's turn (converted on arrival, 65,536 x
  // 1,536 bf16 took 302 us instead of 108).
  using S = typename std::conditional<CK, int8_t, T>::type;  // of the saved values
  struct Batch {
    Cols<T, V> g[R];
    Cols<S, V> x[R];
    uint32_t b[R];
  };
  auto load = [&](int r0) {
    Batch t;
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int r = r0 + k;
      const bool in = r < rows;
      t.g[k] = load_cols<T, V>(dy + (long long)r * ldx, in, n);
      if constexpr (CK) {
        t.x[k] = load_cols<int8_t, V>(q + (long long)r * ldq, in, n);
        t.b[k] = in && n > 0 ? sc[(long long)r * lds] : 0;
      } else {
        t.x[k] = load_cols<T, V>(u + (long long)r * ldu, in && has_u, n);
      }
    }
    return t;
  };
  float sum[V];
#pragma unroll
  for (int j = 0; j < V; ++j) sum[j] = 0.f;
  Batch next = load(0);
  with_act(a.act, [&](auto tag) {
    constexpr int ACT = decltype(tag)::value;
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += R) {
      Batch t = next;
#pragma unroll
      for (int k = 0; k < R; ++k) {
        t.g[k].pin();
        t.x[k].pin();
      }
      if (r0 + R < rows) next = load(r0 + R);
      // two values at a time: neighbours, or a column of two rows
      constexpr int KP = V == 1 ? 2 : 1;
#pragma unroll
      for (int k = 0; k < R; k += KP) {
        float g[KP][V], x[KP][V], f[KP][V];
#pragma unroll
        for (int e = 0; e < KP; ++e) {
          const Cols<T, V>& tg = t.g[k + e];
          const Cols<S, V>& tx = t.x[k + e];
          const float step = CK ? ckpt8_step(t.b[k + e]) : 0.f;
#pragma unroll
          for (int j = 0; j < V; ++j) {
            g[e][j] = to_f32(tg.t[j]);
            if constexpr (CK) x[e][j] = (float)tx.t[j] * step;
            else x[e][j] = to_f32(tx.t[j]);
          }
        }
        float* gv = &g[0][0];
        float* fv = &f[0][0];
        const float* xv = &x[0][0];
#pragma unroll
        for (int i = 0; i < KP * V; i += 2) {
          if constexpr (ACC) {
            gv[i] *= act_grad_of<true, ACT>(xv[i], a.slope, fv[i]);
            gv[i + 1] *= act_grad_of<true, ACT>(xv[i + 1], a.slope, fv[i + 1]);
          } else {
            F2 w;
            const F2 d = mul2(f2(gv[i], gv[i + 1]), act_grad2<ACT>(f2(xv[i], xv[i + 1]), a.slope, w));
            gv[i] = d.x;
            gv[i + 1] = d.y;
            fv[i] = w.x;
            fv[i + 1] = w.y;
          }
        }
#pragma unroll
        for (int e = 0; e < KP; ++e) {
          if (r0 + k + e >= rows) break;  // warp-uniform
#pragma unroll
          for (int j = 0; j < V; ++j) sum[j] += g[e][j];
          store_cols<T, V>(du + (long long)(r0 + k + e) * ldy, n, g[e]);
          if (a.u_out) store_cols<T, V>(ao + (long long)(r0 + k + e) * ldo, n, f[e]);
        }
      }
    }
  });
  if (a.colpart) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j < n) a.colpart[rb * a.ldcp + c + j] = sum[j];
  }
}

// ------------------------------------------------------------ a few rows
//
// Up to 8 rows: bound by reading W once.  A cluster of S CTAs takes 64 or 128
// output columns, each CTA one slice of K; the S partial results meet in
// distributed shared memory and the cluster's warps run the epilogue, so the
// call is one launch without a workspace.  Each CTA: 256 threads, each with a
// ring of 16-byte pieces of W that it alone fills (asynchronous copies) and
// reads, so the stream needs no barriers and the depth of the ring, not the
// registers, sets the bytes in flight; the rows of x are in shared memory as
// fp32.
//   forward, W [K][N]: a thread keeps 16 bytes of columns and walks down K
//   (256-byte runs of W per 128 columns);
//   backward, W [N][K]: a warp keeps 8 of the 64 columns and its lanes walk
//   along K.
// All CTAs of a launch are resident at once: a second wave of a few would
// double the time (8,192 x 8,192 bf16, one row: 70 us; all resident 23 us =
// 5.8 TB/s; 512 x 1,536 with cold caches 8 us).

constexpr int kFewX = 4096;   // values of x staged at a time (all rows)
constexpr int kFewRing = 8;   // pieces of a thread's ring

template <int MT, bool BWD, int COLS>
struct FewShape {
  static constexpr int kPerSm = MT <= 2 ? 4 : MT == 4 ? 3 : 2;  // CTAs an SM holds (registers)
  static constexpr int kChunk = kFewX / MT;
  // ring (the forward's reduction takes its place), x, this CTA's sums
  static constexpr int kRing = kFewRing * kThreads * 16;
  static constexpr int kSmem = kRing + kFewX * 4 + MT * COLS * 4;
  static_assert(8 * MT * COLS * 4 <= kRing, "reduction in the ring's place");
};

// One piece of W into the thread's slot: asynchronously where it is whole and
// aligned, else value by value (the same thread reads it, in program order).
template <typename T>
__device__ __forceinline__ void few_issue(uint4* slot, const T* p, int n, bool vec) {
  if (vec && n >= RowVec<T>::N) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(slot)), "l"(p)
                 : "memory");
  } else {
    *slot = load_piece(p, n, false);
  }
}
__device__ __forceinline__ void few_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void few_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

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
__global__ void __launch_bounds__(kThreads, FewShape<MT, BWD, COLS>::kPerSm)
    linear_few_kernel(const LinearArgs a, int cluster, int slice, int w_vec, float* dbias) {
  using Shape = FewShape<MT, BWD, COLS>;
  constexpr int N = RowVec<T>::N;
  constexpr int LPR = COLS / N;       // forward: lanes across the columns
  constexpr int KP = kThreads / LPR;  // forward: rows of W per step
  constexpr int CHUNK = Shape::kChunk;
  constexpr int D = kFewRing;
  static_assert(LPR <= 32 && (!BWD || COLS == 64), "columns of a CTA");
  extern __shared__ __align__(16) uint8_t few_smem[];
  float* xs = reinterpret_cast<float*>(few_smem + Shape::kRing);  // forward [k][MT], backward [MT][k]
  float* red = reinterpret_cast<float*>(few_smem);                // forward: [warp][MT][COLS]
  float* part = xs + kFewX;  // [MT][COLS]: this CTA's sums, read by the cluster
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint4* ring = reinterpret_cast<uint4*>(few_smem) + tid;  // slot i at [i * kThreads]
  pdl_wait();
  pdl_launch_dependents();
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
      // step s: row tid / LPR + s KP of the chunk
      const int k_first = tid / LPR;
      const int c = c0 + (tid % LPR) * N, cols = a.N - c;
      const T* wp = w + (long long)(kc + k_first) * a.ldw + c;
      const long long step = (long long)KP * a.ldw;
      const int steps = (len - k_first + KP - 1) / KP;
      auto issue = [&](int st, int slot) {
        if (st < steps) few_issue(ring + slot * kThreads, wp + st * step, cols, w_vec);
        few_commit();
      };
#pragma unroll
      for (int i = 0; i < D - 1; ++i) issue(i, i);
      stage_x();
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
    } else {
      // step s: column s % 8 of the warp, piece lane + 32 (s / 8) of the chunk
      static_assert(D == 8, "a ring turn is the warp's eight columns");
      const T* wp = w + (long long)(c0 + warp * 8) * a.ldw + kc + lane * N;
      auto issue = [&](int k, int j) {  // k: offset from the lane's first piece
        if (k + lane * N < len)
          few_issue(ring + j * kThreads, wp + j * a.ldw + k,
                    c0 + warp * 8 + j < a.N ? len - k - lane * N : 0, w_vec);
        few_commit();
      };
#pragma unroll
      for (int j = 0; j < D - 1; ++j) issue(0, j);
      stage_x();
      for (int k = 0; k < len; k += 32 * N) {  // warp-uniform
        const bool in = k + lane * N < len;
#pragma unroll
        for (int j = 0; j < D; j += 2) {
          // two columns share the x fragments
          few_wait<D - 3>();
          if (in) {
            F2 w0[N / 2], w1[N / 2];
            unpack_piece<T>(ring[j * kThreads], w0);
            unpack_piece<T>(ring[(j + 1) * kThreads], w1);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              F2 s0 = f2(acc[m][j], 0.f), s1 = f2(acc[m][j + 1], 0.f);
#pragma unroll
              for (int e = 0; e < N; e += 4) {
                const float4 f =
                    *reinterpret_cast<const float4*>(xs + m * CHUNK + k + lane * N + e);
                s0 = fma2(f2(f.x, f.y), w0[e / 2], s0);
                s1 = fma2(f2(f.x, f.y), w1[e / 2], s1);
                s0 = fma2(f2(f.z, f.w), w0[e / 2 + 1], s0);
                s1 = fma2(f2(f.z, f.w), w1[e / 2 + 1], s1);
              }
              acc[m][j] = s0.x + s0.y;
              acc[m][j + 1] = s1.x + s1.y;
            }
          }
          if (j == 0) issue(k, D - 1);
          else issue(k + 32 * N, j - 1);
          issue(k + 32 * N, j);
        }
      }
      few_wait<0>();
    }
  }

  // this CTA's sums into part[m][column]
  if constexpr (!BWD) {
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
      with_act(a.act, [&](auto tag) {
        sum += epi_finish<T, BWD, decltype(tag)::value>(a, m, c, ok, v, bias, extra);
      });
    }
    if (BWD && dbias && ok) dbias[c] = sum;
  }
  ptx::cluster_sync();  // no CTA leaves while its sums may still be read
}

template <typename T, int MT, bool BWD, int COLS>
mlp_status few_launch(const LinearArgs& a, float* dbias, cudaStream_t st) {
  using Shape = FewShape<MT, BWD, COLS>;
  static PerDevice configured;
  if (!allow_smem(configured, linear_few_kernel<T, MT, BWD, COLS>, Shape::kSmem))
    return MLP_ERR_CUDA;
  // the widest cluster with which all CTAs are resident (on 152 SMs) and each
  // still has 128 of K
  const long long tiles = (a.N + COLS - 1) / COLS;
  int cluster = 8;
  while (cluster > 1 &&
         (tiles * cluster > 152 * Shape::kPerSm || a.K < 128 * cluster))
    --cluster;
  const int per = (a.K + cluster - 1) / cluster;
  const int slice = (per + 63) / 64 * 64;  // slices start on whole 16-byte pieces
  if (tiles * cluster > 0x7fffffffll) return MLP_ERR_UNSUPPORTED_SHAPE;
  const int w_vec = reinterpret_cast<uintptr_t>(a.w) % 16 == 0 && a.ldw * sizeof(T) % 16 == 0;
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

template <typename T, bool BWD>
mlp_status finish_launch(const LinearArgs& a, cudaStream_t st) {
  const int groups = (a.N + 31) / 32;
  const int unit_rows = BWD ? a.part_rows : kRowsAhead;
  const long long units = (a.T + unit_rows - 1) / unit_rows * groups;
  const long long blocks = (units + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7fffffffll) return MLP_ERR_UNSUPPORTED_SHAPE;
  LaunchScope ls(BWD ? "linear_bwd_finish" : "linear_fwd_finish", st, a.T, a.N, a.splits);
  launch_k(linear_finish_kernel<T, BWD>, dim3((unsigned)blocks), dim3(kThreads), 0, st, a, groups,
           unit_rows, units);
  return launch_status();
}

template <typename T, int V, bool CK>
mlp_status act_launch(const LinearArgs& a, cudaStream_t st) {
  const int groups = (a.N + 32 * V - 1) / (32 * V);
  const long long units = (a.T + a.part_rows - 1) / a.part_rows * groups;
  const long long blocks = (units + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7fffffffll) return MLP_ERR_UNSUPPORTED_SHAPE;
  LaunchScope ls("act_bwd", st, a.T, a.N, sizeof(T));
  launch_k(act_bwd_kernel<T, V, CK>, dim3((unsigned)blocks), dim3(kThreads), 0, st, a, groups,
           units);
  return launch_status();
}

template <typename T>
mlp_status act_t(const LinearArgs& a, cudaStream_t st) {
  // four columns per lane where every matrix keeps them aligned (base pointers
  // are 16-byte aligned)
  const bool vec = a.ldx % 4 == 0 && a.ldy % 4 == 0 && (!a.u_in || a.ldu_in % 4 == 0) &&
                   (!a.q || a.ldq % 4 == 0) && (!a.u_out || a.ldu_out % 4 == 0);
  if (a.q) return vec ? act_launch<T, 4, true>(a, st) : act_launch<T, 1, true>(a, st);
  return vec ? act_launch<T, 4, false>(a, st) : act_launch<T, 1, false>(a, st);
}

}  // namespace

// Up to 8 rows, all that this kernel takes, for fp32, whose tiled kernel computes
// 128 rows whatever T is (8 rows, here and there: 512 x 1,536 4.8 and 11.5 us,
// 8,192 x 8,192 65 and 298; backward 9.5 and 12.7, 112 and 292).
// In 16 bits the tensor cores take over once the FMAs, not the reading of W,
// bound this kernel: above 2 rows of a large W (8,192 x 8,192, 4 rows: 49 us
// here, 36 there), above 8 of a small one, 4 in the backward, whose x
// fragments are per lane (1,536 x 512, 8 rows: forward 6.3 here, 8.7 there;
// backward 11.9 and 9.6).
bool linear_takes_few(long long T, int K, int N, int dtype, bool bwd) {
  if (dtype == MLP_DTYPE_F32) return T <= 8;
  return T <= 2 || (T <= (bwd ? 4 : 8) && (long long)K * N <= (1ll << 22));
}

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

mlp_status launch_linear_finish(const LinearArgs& a, bool bwd, cudaStream_t st) {
  switch (a.dtype) {
    case MLP_DTYPE_BF16:
      return bwd ? finish_launch<__nv_bfloat16, true>(a, st)
                 : finish_launch<__nv_bfloat16, false>(a, st);
    case MLP_DTYPE_F16:
      return bwd ? finish_launch<__half, true>(a, st) : finish_launch<__half, false>(a, st);
    default: return bwd ? finish_launch<float, true>(a, st) : finish_launch<float, false>(a, st);
  }
}

mlp_status launch_act_bwd(const LinearArgs& a, cudaStream_t st) {
  switch (a.dtype) {
    case MLP_DTYPE_BF16: return act_t<__nv_bfloat16>(a, st);
    case MLP_DTYPE_F16: return act_t<__half>(a, st);
    default: return act_t<float>(a, st);
  }
}

}  // namespace mlp
