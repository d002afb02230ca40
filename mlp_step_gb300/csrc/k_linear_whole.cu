// The 16-bit linear layers in CTA pairs whose pieces are all whole: N in 64s,
// 16-bit outputs, every matrix of the epilogue addressable by TMA.  The usual
// case, compiled without the other ones (bias, residual and the 8-bit output
// stay run-time choices): 65,536 x 512 -> 1,536 with GELU and 8-bit
// pre-activations takes 151 us in the general form and 105 in this one.
#include "linear_tc.cuh"

namespace mlp {

namespace {

template <int H16>
mlp_status launch(const LinMaps& maps, const LinParams& p, int mode, int form, cudaStream_t st) {
  if (mode == kFwd)
    return form == kWhole64 ? launch_pairs<H16, kFwd, kWhole64>(maps, p, st)
                            : launch_pairs<H16, kFwd, kWhole32>(maps, p, st);
  if (mode == kBwd) return launch_pairs<H16, kBwd, kWhole64>(maps, p, st);
  return form == kWhole64 ? launch_pairs<H16, kBwdCkpt, kWhole64>(maps, p, st)
                          : launch_pairs<H16, kBwdCkpt, kWhole32>(maps, p, st);
}

}  // namespace

mlp_status launch_linear_whole(const LinMaps& maps, const LinParams& p, int mode, int form,
                               cudaStream_t st) {
  return p.a.dtype == MLP_DTYPE_F16 ? launch<1>(maps, p, mode, form, st)
                                    : launch<0>(maps, p, mode, form, st);
}

}  // namespace mlp
