// C-ABI entry points of dropout and of the residual norm (include/mlp_step.h).
// Argument checks; every computation is a kernel launch.
#include <cmath>

#include "kernels.cuh"
#include "trace.cuh"

using namespace mlp;

namespace {

inline cudaStream_t S(void* s) { return static_cast<cudaStream_t>(s); }

constexpr int kMaxNorm = 65536;      // widths of the norm
constexpr int kMaxDropout = 1 << 24; // ... of dropout alone

bool known_dtype(int t) {
  return t == MLP_DTYPE_F32 || t == MLP_DTYPE_BF16 || t == MLP_DTYPE_F16;
}

template <typename... P>
bool all_aligned(P... p) {
  return (aligned16(p) && ...);  // null pointers are
}

// A matrix that may be missing, d columns.
bool mat_ok(const void* m, int ld, int d) { return !m || ld >= d; }

bool drop_ok(float p, const void* rng) { return p >= 0.f && p <= 1.f && (p == 0.f || rng); }

DropArgs drop_args(float p, const uint64_t* rng, uint32_t site) {
  DropArgs a{};
  a.threshold = (uint32_t)std::floor((double)p * 65536.0 + 0.5);
  a.rng = reinterpret_cast<const unsigned long long*>(rng);
  a.site = site;
  a.scale = a.threshold < 65536u ? (float)(65536.0 / (65536.0 - a.threshold)) : 0.f;
  return a;
}

bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7) == 0; }

}  // namespace

extern "C" {

mlp_status mlp_dropout(const void* x, int ldx, const void* residual, int ldr, int T, int d,
                       int dtype, float p, const uint64_t* rng, uint32_t site, void* y, int ldy,
                       void* stream) {
  NvtxRange nvtx_range("mlp_dropout");
  if (T < 0 || d <= 0 || !known_dtype(dtype) || !drop_ok(p, rng)) return MLP_ERR_INVALID_ARG;
  if (d > kMaxDropout) return MLP_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return MLP_OK;
  if (!x || !y || ldx < d || ldy < d || !mat_ok(residual, ldr, d)) return MLP_ERR_INVALID_ARG;
  if (!all_aligned(x, residual, y) || !aligned8(rng)) return MLP_ERR_MISALIGNED;
  Dropout a{};
  a.dtype = dtype;
  a.x = x; a.ldx = ldx;
  a.res = residual; a.ldr = ldr;
  a.T = T; a.d = d;
  a.drop = drop_args(p, rng, site);
  a.y = y; a.ldy = ldy;
  return launch_dropout(a, S(stream));
}

mlp_status mlp_resnorm_fwd(const void* x, int ldx, const void* b, int ldb, int dtype,
                           int post_norm, const float* post_gain, const void* gate, int ldgate,
                           int gate_act, float scale, float p, const uint64_t* rng,
                           uint32_t site, int T, int d, float eps, const float* next_gain,
                           void* h, int ldh, void* n, int ldn, float* b_rstd_out,
                           float* h_rstd_out, void* stream) {
  NvtxRange nvtx_range("mlp_resnorm_fwd");
  if (T < 0 || d <= 0 || !known_dtype(dtype) || !(eps >= 0.f) || !drop_ok(p, rng) ||
      (gate_act != MLP_GATE_PLAIN && gate_act != MLP_GATE_SIGMOID))
    return MLP_ERR_INVALID_ARG;
  if (d > kMaxNorm) return MLP_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return MLP_OK;
  // without a block output there is the norm of x alone; h comes with b
  if (!b && (post_norm || post_gain || gate || p > 0.f)) return MLP_ERR_INVALID_ARG;
  if (!x || !b != !h || (!h && !n) || (!n && (next_gain || h_rstd_out)) ||
      (!post_norm && b_rstd_out))
    return MLP_ERR_INVALID_ARG;
  if (ldx < d || !mat_ok(b, ldb, d) || !mat_ok(gate, ldgate, d) || !mat_ok(h, ldh, d) ||
      !mat_ok(n, ldn, d))
    return MLP_ERR_INVALID_ARG;
  if (!all_aligned(x, b, post_gain, gate, next_gain, h, n, b_rstd_out, h_rstd_out) ||
      !aligned8(rng))
    return MLP_ERR_MISALIGNED;
  ResNorm a{};
  a.dtype = dtype;
  a.T = T; a.d = d; a.eps = eps;
  a.x = x; a.ldx = ldx;
  a.b = b; a.ldb = ldb;
  a.z = gate; a.ldz = ldgate;
  a.sigmoid = gate_act == MLP_GATE_SIGMOID;
  a.scale = scale;
  a.post = post_norm != 0;
  a.post_gain = post_gain; a.next_gain = next_gain;
  a.drop = drop_args(p, rng, site);
  a.h = h; a.ldh = ldh;
  a.n = n; a.ldn = ldn;
  a.b_rstd = b_rstd_out; a.h_rstd = h_rstd_out;
  return launch_resnorm_fwd(a, S(stream));
}

size_t mlp_resnorm_workspace_bytes(int T, int d) {
  if (T <= 0 || d <= 0 || d > kMaxNorm) return 0;
  return resnorm_ws_bytes(T, d);
}

mlp_status mlp_resnorm_bwd(const void* dh, int lddh, const void* dn, int lddn, const void* h,
                           int ldh, const float* h_rstd, const float* next_gain, const void* b,
                           int ldb, int dtype, int post_norm, const float* post_gain,
                           const float* b_rstd, const void* gate, int ldgate, int gate_act,
                           float scale, float p, const uint64_t* rng, uint32_t site, int T, int d,
                           void* dx, int lddx, void* db, int lddb, void* dgate, int lddgate,
                           float* dpost_gain, float* dnext_gain, void* workspace, size_t ws_bytes,
                           void* stream) {
  NvtxRange nvtx_range("mlp_resnorm_bwd");
  if (T < 0 || d <= 0 || !known_dtype(dtype) || !drop_ok(p, rng) ||
      (gate_act != MLP_GATE_PLAIN && gate_act != MLP_GATE_SIGMOID))
    return MLP_ERR_INVALID_ARG;
  if (d > kMaxNorm) return MLP_ERR_UNSUPPORTED_SHAPE;
  if (!all_aligned(dpost_gain, dnext_gain)) return MLP_ERR_MISALIGNED;
  if (T == 0) {
    // sums over no rows
    for (float* g : {dpost_gain, dnext_gain})
      if (g && cudaMemsetAsync(g, 0, (size_t)d * 4, S(stream)) != cudaSuccess)
        return MLP_ERR_CUDA;
    return MLP_OK;
  }
  if (!b && (post_norm || post_gain || gate || p > 0.f || dpost_gain)) return MLP_ERR_INVALID_ARG;
  if ((!dh && !dn) || !dx || !b != !db || !gate != !dgate || (post_norm && !b_rstd) ||
      (dn && (!h || !h_rstd)) || (!dn && (next_gain || dnext_gain)))
    return MLP_ERR_INVALID_ARG;
  if (!mat_ok(dh, lddh, d) || !mat_ok(dn, lddn, d) || (dn && ldh < d) || !mat_ok(b, ldb, d) ||
      !mat_ok(gate, ldgate, d) || lddx < d || !mat_ok(db, lddb, d) || !mat_ok(dgate, lddgate, d))
    return MLP_ERR_INVALID_ARG;
  const bool sums = dpost_gain || dnext_gain;
  if (sums && (!workspace || ws_bytes < resnorm_ws_bytes(T, d))) return MLP_ERR_INVALID_ARG;
  if (!all_aligned(dh, dn, h, h_rstd, next_gain, b, post_gain, b_rstd, gate, dx, db, dgate,
                   workspace) ||
      !aligned8(rng))
    return MLP_ERR_MISALIGNED;
  ResNorm a{};
  a.dtype = dtype;
  a.T = T; a.d = d;
  a.x = dh; a.ldx = lddh;
  a.b = b; a.ldb = ldb;
  a.z = gate; a.ldz = ldgate;
  a.sigmoid = gate_act == MLP_GATE_SIGMOID;
  a.scale = scale;
  a.post = post_norm != 0;
  a.post_gain = post_gain; a.next_gain = next_gain;
  a.drop = drop_args(p, rng, site);
  if (dn) {
    a.h = const_cast<void*>(h); a.ldh = ldh;
    a.n = const_cast<void*>(dn); a.ldn = lddn;
    a.h_rstd = const_cast<float*>(h_rstd);
  }
  a.b_rstd = const_cast<float*>(b_rstd);
  a.dx = dx; a.lddx = lddx;
  a.db = db; a.lddb = lddb;
  a.dz = dgate; a.lddz = lddgate;
  a.part = sums ? static_cast<float*>(workspace) : nullptr;
  return launch_resnorm_bwd(a, dnext_gain, dpost_gain, S(stream));
}

}  // extern "C"
