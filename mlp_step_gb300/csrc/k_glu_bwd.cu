// Gated units on the tensor cores, backward: through the down projection and
// the gate in one kernel,
//   da = dy Wd^T,  dg = da u f'(g),  du = da f(g),  a = f(g) u,
// with the column sums of dg and du (the bias gradients).  g and u are read in
// the operand type or from 8 bits.
//
// Tiles as in k_glu.cu, without the second weight (256 x 256 of a CTA pair,
// 128 x 128 or 128 x 64 of one CTA).  Bound by HBM for K of a few hundred:
// beside the product, 8 to 10 bytes move per value of da.  So the saved values
// of an epilogue warp's next piece (32 x 32) are on their way by TMA while it
// works on this one, and every output leaves by TMA from a box of its own.
// Measured at 65,536 x 512 <- 1,408 bf16, SiLU: from 16 bits without a and sums 138
// us (5.8 TB/s); from 8 bits with both 176, of which the column sums and their
// launch are 32, bound by the epilogue's instructions (35 an output, issued in
// 55 % of the slots).
#include "glu_launch.cuh"

namespace mlp {

namespace {

// 16-bit saved values take boxes twice as large as 8-bit ones: beside twelve
// epilogue warps a ring of three operand stages, which long K feels, beside
// eight one of four (us with twelve and eight, K = 512 194 and 210, 1,024 134
// and 118, 1,536 224 and 198, 8,192 425 and 374).  Registers spill a little, in
// bytes a thread: twelve warps from 16 bits 16 (ragged pieces 20), from 8 bits none
// (12), eight warps 4 (20), the 128-column single tile 36.
constexpr int kShortK = 12;  // k-blocks

template <int H16, int MODE>
mlp_status launch(const GluMaps& maps, const GluParams& p, GluTile tile, cudaStream_t st) {
  if (tile == kGluPair) {
    if constexpr (MODE == kGluBwd) {
      if (p.k_blocks > kShortK)
        return glu_whole(p, true) ? launch_glu_pair<4, 8, H16, MODE, true>(maps, p, st)
                                  : launch_glu_pair<4, 8, H16, MODE, false>(maps, p, st);
    }
    constexpr int STAGES = MODE == kGluBwd ? 3 : 4;
    return glu_whole(p, true) ? launch_glu_pair<STAGES, 12, H16, MODE, true>(maps, p, st)
                              : launch_glu_pair<STAGES, 12, H16, MODE, false>(maps, p, st);
  }
  if (tile == kGluWide) return launch_glu_single<128, 4, 8, 128, H16, MODE>(maps, p, st);
  return launch_glu_single<64, 7, 4, 128, H16, MODE>(maps, p, st);
}

}  // namespace

mlp_status launch_glu_bwd_tc(const GluArgs& a, const GluPlan& pl, cudaStream_t st) {
  GluMaps maps;
  GluParams p;
  MLP_CHECK(glu_setup(a, pl, true, maps, p));
  const bool h16 = a.dtype == MLP_DTYPE_F16;
  if (a.q[0])
    return h16 ? launch<1, kGluBwdCkpt>(maps, p, pl.tile, st)
               : launch<0, kGluBwdCkpt>(maps, p, pl.tile, st);
  return h16 ? launch<1, kGluBwd>(maps, p, pl.tile, st) : launch<0, kGluBwd>(maps, p, pl.tile, st);
}

}  // namespace mlp
