// C-ABI entry points of the gated units (include/mlp_step.h).  Argument checks,
// workspace carving and the enqueue order; every computation is a kernel launch.
#include "ckpt8.cuh"
#include "kernels.cuh"
#include "trace.cuh"

using namespace mlp;

namespace {

inline cudaStream_t S(void* s) { return static_cast<cudaStream_t>(s); }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

constexpr int kMaxWidth = 1 << 24;

bool widths_ok(int a, int b) { return a > 0 && a <= kMaxWidth && b > 0 && b <= kMaxWidth; }

bool known_dtype(int t) {
  return t == MLP_DTYPE_F32 || t == MLP_DTYPE_BF16 || t == MLP_DTYPE_F16;
}

mlp_status check(int T, int k, int n, int dtype, int act) {
  if (T < 0 || k < 1 || n < 1 || !known_dtype(dtype) || act < MLP_ACT_NONE ||
      act > MLP_ACT_SILU)
    return MLP_ERR_INVALID_ARG;
  return widths_ok(k, n) ? MLP_OK : MLP_ERR_UNSUPPORTED_SHAPE;
}

template <typename... P>
bool all_aligned(P... p) {
  return (aligned16(p) && ...);  // null pointers are
}

// The gate's and the up projection's matrices of one form, n columns: both
// given with pitches that hold them, or neither.
bool pair_ok(const void* g, int ldg, const void* u, int ldu, int n) {
  if (!g && !u) return true;
  return g && u && ldg >= n && ldu >= n;
}
// ... in 8 bits, with their scales
bool ckpt_pair_ok(const void* gq, int ldgq, const void* gs, int ldgs, const void* uq, int lduq,
                  const void* us, int ldus, int n) {
  const int groups = (n - 1) / kCkptGroup + 1;
  return pair_ok(gq, ldgq, uq, lduq, n) && pair_ok(gs, ldgs, us, ldus, groups) && !gq == !gs;
}

// How a product [T][K] x [K][N] runs, and its workspace: planes of raw sums
// where the epilogue is a pass of its own, then (backward) partial column sums.
struct GluPath {
  bool few;    // launch_glu_few: no workspace
  int splits;  // planes of raw sums of a projection (0: the epilogue is in the product's kernel)
  size_t sums, part;
  int part_rows;
  long long ldp, ldcp;
  long long parts(long long T) const { return (T + part_rows - 1) / part_rows; }
};

GluPath glu_path(long long T, int K, int N, int dtype, bool bwd) {
  GluPath p{};
  p.few = !bwd && glu_takes_few(T, K, N, dtype);
  if (p.few) return p;
  if (dtype == MLP_DTYPE_F32) {
    p.splits = linear_f32_splits(T, K, N, bwd ? 1 : 2);
  } else {
    p.splits = glu_tc_splits(T, K, N, bwd);
    if (p.splits == 1) p.splits = 0;
  }
  p.ldp = (N + 31) / 32 * 32;  // whole pieces of the tensor-core kernel
  p.sums = align256((size_t)p.splits * (bwd ? 1 : 2) * T * p.ldp * 4);
  if (bwd) {
    p.ldcp = (2ll * N + 31) / 32 * 32;  // whole 128-byte lines
    p.part_rows = p.splits && T < 2048 ? kPartRowsFew : kPartRows;
    p.part = align256((size_t)p.parts(T) * p.ldcp * 4);
  }
  return p;
}

mlp_status run_glu(GluArgs a, const GluPath& gp, bool bwd, float* db_gate, float* db_up,
                   void* workspace, cudaStream_t st) {
  if (gp.few) return launch_glu_few(a, st);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.splits = gp.splits ? gp.splits : 1;
  a.partial = gp.splits ? reinterpret_cast<float*>(ws) : nullptr;
  a.ldp = gp.ldp;
  a.colpart = db_gate ? reinterpret_cast<float*>(ws + gp.sums) : nullptr;
  a.ldcp = gp.ldcp;
  a.part_rows = gp.part_rows;
  if (a.dtype == MLP_DTYPE_F32) {
    LinearArgs l{};
    l.dtype = a.dtype;
    l.T = a.T; l.K = a.K; l.N = a.N;
    l.x = a.x; l.ldx = a.ldx;
    l.ldp = a.ldp;
    l.splits = a.splits;
    l.w = a.w[0]; l.ldw = a.ldw[0];
    l.w2 = a.w[1]; l.ldw2 = a.ldw[1];  // (none in the backward)
    l.partial = a.partial;
    MLP_CHECK(launch_linear_f32(l, bwd, st));
  } else {
    MLP_CHECK(launch_glu_tc(a, bwd, st));
  }
  if (gp.splits) MLP_CHECK(launch_glu_finish(a, bwd, st));
  if (!db_gate) return MLP_OK;
  return launch_partial_sums(a.colpart, gp.parts(a.T), 2 * a.N, a.ldcp, db_gate, a.N, db_up, st);
}

}  // namespace

extern "C" {

size_t mlp_glu_workspace_bytes(int T, int d_in, int hidden, int dtype) {
  if (T <= 0 || !widths_ok(d_in, hidden) || !known_dtype(dtype)) return 0;
  return glu_path(T, d_in, hidden, dtype, false).sums;
}

mlp_status mlp_glu_fwd(const void* x, int ldx, const void* w_gate, int ldwg, const void* w_up,
                       int ldwu, int T, int d_in, int hidden, int dtype, const float* b_gate,
                       const float* b_up, int act, float slope, void* y, int ldy, void* g_out,
                       int ldg, void* u_out, int ldu, int8_t* g_q, int ldgq, uint8_t* g_scale,
                       int ldgs, int8_t* u_q, int lduq, uint8_t* u_scale, int ldus,
                       void* workspace, size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("mlp_glu_fwd");
  MLP_CHECK(check(T, d_in, hidden, dtype, act));
  if (T == 0) return MLP_OK;
  if (!x || !w_gate || !w_up || !y || ldx < d_in || ldwg < hidden || ldwu < hidden ||
      ldy < hidden || !pair_ok(g_out, ldg, u_out, ldu, hidden) ||
      !ckpt_pair_ok(g_q, ldgq, g_scale, ldgs, u_q, lduq, u_scale, ldus, hidden) ||
      (g_out && g_q))
    return MLP_ERR_INVALID_ARG;
  if (!all_aligned(x, w_gate, w_up, b_gate, b_up, y, g_out, u_out, g_q, g_scale, u_q, u_scale,
                   workspace))
    return MLP_ERR_MISALIGNED;
  if (dtype != MLP_DTYPE_F32 && (ldx % 8 != 0 || ldwg % 8 != 0 || ldwu % 8 != 0))
    return MLP_ERR_MISALIGNED;
  const GluPath gp = glu_path(T, d_in, hidden, dtype, false);
  if (gp.sums > 0 && (!workspace || ws_bytes < gp.sums)) return MLP_ERR_INVALID_ARG;
  GluArgs a{};
  a.dtype = dtype;
  a.T = T; a.K = d_in; a.N = hidden;
  a.x = x; a.ldx = ldx;
  a.w[0] = w_gate; a.ldw[0] = ldwg;
  a.w[1] = w_up; a.ldw[1] = ldwu;
  a.act = act; a.slope = slope;
  a.bias[0] = b_gate; a.bias[1] = b_up;
  a.y = y; a.ldy = ldy;
  a.o[0] = g_out; a.ldo[0] = ldg;
  a.o[1] = u_out; a.ldo[1] = ldu;
  a.q[0] = g_q; a.ldq[0] = ldgq; a.scale[0] = g_scale; a.lds[0] = ldgs;
  a.q[1] = u_q; a.ldq[1] = lduq; a.scale[1] = u_scale; a.lds[1] = ldus;
  return run_glu(a, gp, false, nullptr, nullptr, workspace, S(stream));
}

size_t mlp_glu_bwd_workspace_bytes(int T, int hidden, int d_out, int dtype) {
  if (T <= 0 || !widths_ok(hidden, d_out) || !known_dtype(dtype)) return 0;
  const GluPath gp = glu_path(T, d_out, hidden, dtype, true);
  return gp.sums + gp.part;
}

mlp_status mlp_glu_bwd(const void* dy, int lddy, const void* w_down, int ldw, int T, int hidden,
                       int d_out, int dtype, int act, float slope, const void* g, int ldg,
                       const void* u, int ldu, const int8_t* g_q, int ldgq,
                       const uint8_t* g_scale, int ldgs, const int8_t* u_q, int lduq,
                       const uint8_t* u_scale, int ldus, void* dg, int lddg, void* du, int lddu,
                       float* db_gate, float* db_up, void* a_out, int lda, void* workspace,
                       size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("mlp_glu_bwd");
  MLP_CHECK(check(T, d_out, hidden, dtype, act));
  if (!db_gate != !db_up) return MLP_ERR_INVALID_ARG;
  if (!all_aligned(db_gate, db_up)) return MLP_ERR_MISALIGNED;
  if (T == 0) {
    // sums over no rows
    for (float* d : {db_gate, db_up})
      if (d && cudaMemsetAsync(d, 0, (size_t)hidden * 4, S(stream)) != cudaSuccess)
        return MLP_ERR_CUDA;
    return MLP_OK;
  }
  if (!dy || !w_down || !dg || !du || lddy < d_out || ldw < d_out || lddg < hidden ||
      lddu < hidden || (a_out && lda < hidden) || !pair_ok(g, ldg, u, ldu, hidden) ||
      !ckpt_pair_ok(g_q, ldgq, g_scale, ldgs, u_q, lduq, u_scale, ldus, hidden) ||
      !g == !g_q)  // the pre-activations in exactly one form
    return MLP_ERR_INVALID_ARG;
  if (!all_aligned(dy, w_down, g, u, g_q, g_scale, u_q, u_scale, dg, du, a_out, workspace))
    return MLP_ERR_MISALIGNED;
  if (dtype != MLP_DTYPE_F32 && (lddy % 8 != 0 || ldw % 8 != 0)) return MLP_ERR_MISALIGNED;
  const GluPath gp = glu_path(T, d_out, hidden, dtype, true);
  const size_t need = gp.sums + (db_gate ? gp.part : 0);
  if (need > 0 && (!workspace || ws_bytes < need)) return MLP_ERR_INVALID_ARG;
  GluArgs a{};
  a.dtype = dtype;
  a.T = T; a.K = d_out; a.N = hidden;
  a.x = dy; a.ldx = lddy;
  a.w[0] = w_down; a.ldw[0] = ldw;
  a.act = act; a.slope = slope;
  a.y = a_out; a.ldy = lda;
  a.o[0] = dg; a.ldo[0] = lddg;
  a.o[1] = du; a.ldo[1] = lddu;
  a.in[0] = g; a.ld_in[0] = ldg;
  a.in[1] = u; a.ld_in[1] = ldu;
  a.q[0] = const_cast<int8_t*>(g_q); a.ldq[0] = ldgq;
  a.scale[0] = const_cast<uint8_t*>(g_scale); a.lds[0] = ldgs;
  a.q[1] = const_cast<int8_t*>(u_q); a.ldq[1] = lduq;
  a.scale[1] = const_cast<uint8_t*>(u_scale); a.lds[1] = ldus;
  return run_glu(a, gp, true, db_gate, db_up, workspace, S(stream));
}

}  // extern "C"
