// C-ABI entry points of the feed-forward operators: layer norm, linear layers
// with a fused epilogue, and 8-bit activation checkpoints (include/mlp_step.h).
// Argument checks, workspace carving and the enqueue order; every computation
// is a kernel launch.
#include "ckpt8.cuh"
#include "kernels.cuh"
#include "trace.cuh"

using namespace mlp;

namespace {

inline cudaStream_t S(void* s) { return static_cast<cudaStream_t>(s); }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

bool float_dtype(int t) {
  return t == MLP_DTYPE_F32 || t == MLP_DTYPE_BF16 || t == MLP_DTYPE_F16;
}
bool known_act(int act) { return act >= MLP_ACT_NONE && act <= MLP_ACT_SILU; }

constexpr int kMaxWidth = 65536;    // layer-norm rows
constexpr int kMaxLinear = 1 << 24; // widths of linear layers

int scale_cols(int cols) { return (cols - 1) / kCkptGroup + 1; }  // cols >= 1

// Widths that the entry points take; a size query for others is 0.
bool linear_widths(int d_in, int d_out) {
  return d_in > 0 && d_in <= kMaxLinear && d_out > 0 && d_out <= kMaxLinear;
}

// A checkpoint argument pair: both given with pitches that hold `cols`
// columns, or neither.
bool ckpt_ok(const void* q, int ldq, const void* scale, int lds, int cols) {
  if (!q && !scale) return true;
  return q && scale && ldq >= cols && lds >= scale_cols(cols);
}

template <typename... P>
bool all_aligned(P... p) {
  return (aligned16(p) && ...);  // null pointers are
}

}  // namespace

extern "C" {

// ------------------------------------------------------------ checkpoints

int mlp_ckpt8_scale_cols(int cols) { return cols > 0 ? scale_cols(cols) : 0; }

mlp_status mlp_ckpt8_encode(const void* x, int x_dtype, int rows, int cols, int ldx, int8_t* q,
                            int ldq, uint8_t* scale, int lds, void* stream) {
  NvtxRange nvtx_range("mlp_ckpt8_encode");
  if (rows < 0 || cols < 0 || !float_dtype(x_dtype)) return MLP_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return MLP_OK;
  if (cols > kMaxLinear) return MLP_ERR_UNSUPPORTED_SHAPE;
  if (!x || !q || !scale || ldx < cols || !ckpt_ok(q, ldq, scale, lds, cols))
    return MLP_ERR_INVALID_ARG;
  if (!all_aligned(x, q, scale)) return MLP_ERR_MISALIGNED;
  return launch_ckpt8_encode(x, x_dtype, rows, cols, ldx, q, ldq, scale, lds, S(stream));
}

mlp_status mlp_ckpt8_decode(const int8_t* q, int ldq, const uint8_t* scale, int lds, int rows,
                            int cols, void* out, int out_dtype, int ldo, void* stream) {
  NvtxRange nvtx_range("mlp_ckpt8_decode");
  if (rows < 0 || cols < 0 || !float_dtype(out_dtype)) return MLP_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return MLP_OK;
  if (cols > kMaxLinear) return MLP_ERR_UNSUPPORTED_SHAPE;
  if (!out || !q || !scale || ldo < cols || !ckpt_ok(q, ldq, scale, lds, cols))
    return MLP_ERR_INVALID_ARG;
  if (!all_aligned(out, q, scale)) return MLP_ERR_MISALIGNED;
  return launch_ckpt8_decode(q, ldq, scale, lds, rows, cols, out, out_dtype, ldo, S(stream));
}

// ------------------------------------------------------------ layer norm

mlp_status mlp_layernorm_fwd(const void* x, int dtype, int ldx, const float* gain,
                             const float* shift, int T, int d, float eps, void* y, int ldy,
                             float* mean_out, float* rstd_out, int8_t* x_q, int ldq,
                             uint8_t* x_scale, int lds, void* stream) {
  NvtxRange nvtx_range("mlp_layernorm_fwd");
  if (T < 0 || d <= 0 || !float_dtype(dtype) || !(eps >= 0.f)) return MLP_ERR_INVALID_ARG;
  if (d > kMaxWidth) return MLP_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return MLP_OK;
  if (!x || !y || ldx < d || ldy < d || !ckpt_ok(x_q, ldq, x_scale, lds, d))
    return MLP_ERR_INVALID_ARG;
  if (!all_aligned(x, y, gain, shift, mean_out, rstd_out, x_q, x_scale)) return MLP_ERR_MISALIGNED;
  LayerNormFwd a{};
  a.dtype = dtype;
  a.x = x; a.ldx = ldx;
  a.gain = gain; a.shift = shift;
  a.T = T; a.d = d; a.eps = eps;
  a.y = y; a.ldy = ldy;
  a.mean = mean_out; a.rstd = rstd_out;
  a.q = x_q; a.ldq = ldq; a.scale = x_scale; a.lds = lds;
  return launch_layernorm_fwd(a, S(stream));
}

size_t mlp_layernorm_workspace_bytes(int T, int d) {
  if (T <= 0 || d <= 0 || d > kMaxWidth) return 0;
  return layernorm_ws_bytes(T, d);
}

mlp_status mlp_layernorm_bwd(const void* dy, int dtype, int lddy, const void* x, int ldx,
                             const int8_t* x_q, int ldq, const uint8_t* x_scale, int lds,
                             const float* mean, const float* rstd, const float* gain,
                             const void* dres, int ldr, int T, int d, void* dx, int lddx,
                             float* dgain, float* dshift, void* workspace, size_t ws_bytes,
                             void* stream) {
  NvtxRange nvtx_range("mlp_layernorm_bwd");
  if (T < 0 || d <= 0 || !float_dtype(dtype)) return MLP_ERR_INVALID_ARG;
  if (d > kMaxWidth) return MLP_ERR_UNSUPPORTED_SHAPE;
  if (!dgain || !dshift) return MLP_ERR_INVALID_ARG;
  if (!all_aligned(dgain, dshift)) return MLP_ERR_MISALIGNED;
  if (T == 0) {
    // a sum over no rows
    if (cudaMemsetAsync(dgain, 0, (size_t)d * 4, S(stream)) != cudaSuccess ||
        cudaMemsetAsync(dshift, 0, (size_t)d * 4, S(stream)) != cudaSuccess)
      return MLP_ERR_CUDA;
    return MLP_OK;
  }
  if (!dy || !dx || !mean || !rstd || lddy < d || lddx < d || (dres && ldr < d))
    return MLP_ERR_INVALID_ARG;
  // the forward's input in exactly one form
  if (!x == !x_q || (x && (ldx < d || x_scale)) || !ckpt_ok(x_q, ldq, x_scale, lds, d))
    return MLP_ERR_INVALID_ARG;
  if (!workspace || ws_bytes < layernorm_ws_bytes(T, d)) return MLP_ERR_INVALID_ARG;
  if (!all_aligned(dy, x, x_q, x_scale, mean, rstd, gain, dres, dx, workspace))
    return MLP_ERR_MISALIGNED;
  LayerNormBwd a{};
  a.dtype = dtype;
  a.dy = dy; a.lddy = lddy;
  a.x = x; a.ldx = ldx;
  a.q = x_q; a.ldq = ldq; a.scale = x_scale; a.lds = lds;
  a.mean = mean; a.rstd = rstd; a.gain = gain;
  a.dres = dres; a.ldr = ldr;
  a.T = T; a.d = d;
  a.dx = dx; a.lddx = lddx;
  a.dgain = dgain; a.dshift = dshift;
  a.part = static_cast<float*>(workspace);
  return launch_layernorm_bwd(a, S(stream));
}

}  // extern "C"

// ------------------------------------------------------------ linear layers

namespace {

// How a product [T][K] x [K][N] runs, and its workspace: raw sums of the paths
// that finish in a second pass, then (backward) the partial column sums.
struct LinearPath {
  bool few;      // launch_linear_few: no workspace
  int splits;    // planes of raw sums (0: the epilogue is in the product's kernel)
  size_t sums, part;
  int part_rows;
  long long ldp, ldcp;
  long long parts(long long T) const { return (T + part_rows - 1) / part_rows; }
};

LinearPath linear_path(long long T, int K, int N, int dtype, bool bwd) {
  LinearPath p{};
  p.few = linear_takes_few(T, K, N, dtype, bwd);
  if (p.few) return p;
  if (dtype == MLP_DTYPE_F32) {
    p.splits = linear_f32_splits(T, K, N);
  } else {
    p.splits = linear_tc_splits(T, K, N);
    if (p.splits == 1) p.splits = 0;
  }
  p.ldp = (N + 31) / 32 * 32;  // whole pieces of the tensor-core kernel
  p.sums = align256((size_t)p.splits * T * p.ldp * 4);
  if (bwd) {
    p.ldcp = (N + 31) / 32 * 32;  // whole 128-byte lines
    p.part_rows = p.splits && T < 2048 ? kPartRowsFew : kPartRows;
    p.part = align256((size_t)p.parts(T) * p.ldcp * 4);
  }
  return p;
}

mlp_status zero_sums(float* dbias, int n, cudaStream_t st) {
  if (dbias && cudaMemsetAsync(dbias, 0, (size_t)n * 4, st) != cudaSuccess) return MLP_ERR_CUDA;
  return MLP_OK;
}

mlp_status run_linear(LinearArgs a, const LinearPath& lp, bool bwd, float* dbias, void* workspace,
                      cudaStream_t st) {
  if (lp.few) return launch_linear_few(a, bwd, dbias, st);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.splits = lp.splits ? lp.splits : 1;
  a.partial = lp.splits ? reinterpret_cast<float*>(ws) : nullptr;
  a.ldp = lp.ldp;
  a.colpart = dbias ? reinterpret_cast<float*>(ws + lp.sums) : nullptr;
  a.ldcp = lp.ldcp;
  a.part_rows = lp.part_rows;
  MLP_CHECK(a.dtype == MLP_DTYPE_F32 ? launch_linear_f32(a, bwd, st) : launch_linear_tc(a, bwd, st));
  if (lp.splits) MLP_CHECK(launch_linear_finish(a, bwd, st));
  if (!dbias) return MLP_OK;
  return launch_partial_sums(a.colpart, lp.parts(a.T), a.N, a.ldcp, dbias, a.N, nullptr,
                             st);
}

// The shapes and types that a product's entry points share.
mlp_status check_linear(int T, int d_in, int d_out, int dtype, int out_dtype, int act) {
  if (T < 0 || d_in < 1 || d_out < 1 || !float_dtype(dtype) || !known_act(act))
    return MLP_ERR_INVALID_ARG;
  if (out_dtype != dtype && out_dtype != MLP_DTYPE_F32) return MLP_ERR_INVALID_ARG;
  if (d_in > kMaxLinear || d_out > kMaxLinear) return MLP_ERR_UNSUPPORTED_SHAPE;
  return MLP_OK;
}

}  // namespace

extern "C" {

size_t mlp_linear_workspace_bytes(int T, int d_in, int d_out, int dtype) {
  if (T <= 0 || !linear_widths(d_in, d_out) || !float_dtype(dtype)) return 0;
  return linear_path(T, d_in, d_out, dtype, false).sums;
}

mlp_status mlp_linear_fwd(const void* x, int ldx, const void* w, int ldw, int T, int d_in,
                          int d_out, int dtype, const float* bias, int act, float slope,
                          const void* residual, int ldr, void* y, int ldy, int y_dtype,
                          void* u_out, int ldu, int8_t* u_q, int ldq, uint8_t* u_scale, int lds,
                          void* workspace, size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("mlp_linear_fwd");
  MLP_CHECK(check_linear(T, d_in, d_out, dtype, y_dtype, act));
  if (T == 0) return MLP_OK;
  if (!x || !w || !y || ldx < d_in || ldw < d_out || ldy < d_out || (residual && ldr < d_out) ||
      (u_out && ldu < d_out) || !ckpt_ok(u_q, ldq, u_scale, lds, d_out))
    return MLP_ERR_INVALID_ARG;
  if (!all_aligned(x, w, bias, residual, y, u_out, u_q, u_scale, workspace))
    return MLP_ERR_MISALIGNED;
  if (dtype != MLP_DTYPE_F32 && (ldx % 8 != 0 || ldw % 8 != 0)) return MLP_ERR_MISALIGNED;
  const LinearPath lp = linear_path(T, d_in, d_out, dtype, false);
  if (lp.sums > 0 && (!workspace || ws_bytes < lp.sums)) return MLP_ERR_INVALID_ARG;
  LinearArgs a{};
  a.dtype = dtype;
  a.T = T; a.K = d_in; a.N = d_out;
  a.x = x; a.ldx = ldx;
  a.w = w; a.ldw = ldw;
  a.act = act; a.slope = slope;
  a.bias = bias;
  a.res = residual; a.ldr = ldr;
  a.y = y; a.ldy = ldy;
  a.out_f32 = y_dtype == MLP_DTYPE_F32 ? 1 : 0;
  a.u_out = u_out; a.ldu_out = ldu;
  a.q = u_q; a.ldq = ldq; a.scale = u_scale; a.lds = lds;
  return run_linear(a, lp, false, nullptr, workspace, S(stream));
}

size_t mlp_linear_bwd_workspace_bytes(int T, int d_in, int d_out, int dtype) {
  if (T <= 0 || !linear_widths(d_in, d_out) || !float_dtype(dtype)) return 0;
  const LinearPath lp = linear_path(T, d_out, d_in, dtype, true);
  return lp.sums + lp.part;
}

mlp_status mlp_linear_bwd(const void* dy, int lddy, const void* w, int ldw, int T, int d_in,
                          int d_out, int dtype, int act, float slope, const void* u, int ldu,
                          const int8_t* u_q, int ldq, const uint8_t* u_scale, int lds, void* du,
                          int lddu, int du_dtype, float* dbias, void* a_out, int lda,
                          void* workspace, size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("mlp_linear_bwd");
  MLP_CHECK(check_linear(T, d_in, d_out, dtype, du_dtype, act));
  if (!all_aligned(dbias)) return MLP_ERR_MISALIGNED;
  if (T == 0) return zero_sums(dbias, d_in, S(stream));
  if (!dy || !w || !du || lddy < d_out || ldw < d_out || lddu < d_in || (a_out && lda < d_in) ||
      (u && (ldu < d_in || u_q || u_scale)) || !ckpt_ok(u_q, ldq, u_scale, lds, d_in))
    return MLP_ERR_INVALID_ARG;
  if (!u && !u_q && (act != MLP_ACT_NONE || a_out)) return MLP_ERR_INVALID_ARG;
  if (!all_aligned(dy, w, u, u_q, u_scale, du, a_out, workspace)) return MLP_ERR_MISALIGNED;
  if (dtype != MLP_DTYPE_F32 && (lddy % 8 != 0 || ldw % 8 != 0)) return MLP_ERR_MISALIGNED;
  const LinearPath lp = linear_path(T, d_out, d_in, dtype, true);
  const size_t need = lp.sums + (dbias ? lp.part : 0);
  if (need > 0 && (!workspace || ws_bytes < need)) return MLP_ERR_INVALID_ARG;
  LinearArgs a{};
  a.dtype = dtype;
  a.T = T; a.K = d_out; a.N = d_in;
  a.x = dy; a.ldx = lddy;
  a.w = w; a.ldw = ldw;
  a.act = act; a.slope = slope;
  a.y = du; a.ldy = lddu;
  a.out_f32 = du_dtype == MLP_DTYPE_F32 ? 1 : 0;
  a.u_out = a_out; a.ldu_out = lda;
  a.u_in = u; a.ldu_in = ldu;
  a.q = const_cast<int8_t*>(u_q); a.ldq = ldq;
  a.scale = const_cast<uint8_t*>(u_scale); a.lds = lds;
  return run_linear(a, lp, true, dbias, workspace, S(stream));
}

size_t mlp_act_bwd_workspace_bytes(int T, int n) {
  if (T <= 0 || !linear_widths(n, n)) return 0;
  const int rows = act_part_rows(T, n);
  return align256((size_t)(((long long)T + rows - 1) / rows) * ((n + 31) / 32 * 32) * 4);
}

mlp_status mlp_act_bwd(const void* dy, int lddy, int T, int n, int dtype, int act, float slope,
                       const void* u, int ldu, const int8_t* u_q, int ldq,
                       const uint8_t* u_scale, int lds, void* du, int lddu, float* dbias,
                       void* a_out, int lda, void* workspace, size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("mlp_act_bwd");
  MLP_CHECK(check_linear(T, n, n, dtype, dtype, act));
  if (!all_aligned(dbias)) return MLP_ERR_MISALIGNED;
  if (T == 0) return zero_sums(dbias, n, S(stream));
  if (!dy || !du || lddy < n || lddu < n || (a_out && lda < n) ||
      (u && (ldu < n || u_q || u_scale)) || !ckpt_ok(u_q, ldq, u_scale, lds, n))
    return MLP_ERR_INVALID_ARG;
  if (!u && !u_q && (act != MLP_ACT_NONE || a_out)) return MLP_ERR_INVALID_ARG;
  if (!all_aligned(dy, u, u_q, u_scale, du, a_out, workspace)) return MLP_ERR_MISALIGNED;
  if (dbias && (!workspace || ws_bytes < mlp_act_bwd_workspace_bytes(T, n)))
    return MLP_ERR_INVALID_ARG;
  LinearArgs a{};
  a.dtype = dtype;
  a.T = T; a.N = n;
  a.x = dy; a.ldx = lddy;
  a.act = act; a.slope = slope;
  a.y = du; a.ldy = lddu;
  a.out_f32 = dtype == MLP_DTYPE_F32 ? 1 : 0;
  a.u_out = a_out; a.ldu_out = lda;
  a.u_in = u; a.ldu_in = ldu;
  a.q = const_cast<int8_t*>(u_q); a.ldq = ldq;
  a.scale = const_cast<uint8_t*>(u_scale); a.lds = lds;
  a.ldcp = (n + 31) / 32 * 32;
  a.part_rows = act_part_rows(T, n);
  a.colpart = dbias ? static_cast<float*>(workspace) : nullptr;
  MLP_CHECK(launch_act_bwd(a, S(stream)));
  if (!dbias) return MLP_OK;
  return launch_partial_sums(a.colpart, ((long long)T + a.part_rows - 1) / a.part_rows, n, a.ldcp,
                             dbias, n, nullptr, S(stream));
}

}  // extern "C"
