// Gated units on the tensor cores, forward: both projections of x, the
// activation and the product in one kernel,
//   g = x Wg + bg,  u = x Wu + bu,  y = f(g) u,
// fp32 from the accumulators to the one rounding of each output; g and u are
// optionally stored, in the operand type or in 8 bits.
//
// One accumulator holds the gate and the up columns of the same hidden columns
// side by side: a tile of a CTA pair (256 rows, cta_group::2, N = 256) is 128
// hidden columns, of which the even CTA stages the gate's weights and the odd
// one the up projection's, so the MMAs are those of an ordinary product of
// twice the width and the epilogue finds both factors of an output in one row
// of tensor memory, 128 columns apart.  x is read once for both products and g
// and u never leave the SM unless they are kept.  Where such tiles are few, a
// single CTA does the same on 128 rows (128 or 64 hidden columns), with the
// contraction split over CTAs when even those are few (raw sums to a
// workspace, finished by launch_glu_finish).  Warps: TMA producer, MMA issuer,
// four to twelve epilogue warps; two accumulators, so that the epilogue of one
// tile overlaps the MMAs of the next.  The body is in glu_tc.cuh.
//
// Bound: the MMAs for long K (4,096 x 8,192 -> 8,192 fp16 610 us = 1.80 PFLOP/s, 94 %
// of the library's rate, with both pre-activations kept 614, in short runs; called
// again and again, under the power cap, 714).  For K of a few
// hundred the epilogue (65,536 x 512 -> 1,408 bf16 SiLU: 122 us = 1.55 PFLOP/s, of
// which loads and MMAs alone take 104 and the accumulators' way to registers 5; with
// g and u kept 149, in 8 bits 151).
#include "glu_launch.cuh"

namespace mlp {

namespace {

// From the shape alone (so that workspace sizes do not depend on the device).
// Pairs from 40 of their tiles on (us in pairs and in the best single tiles, K =
// 512 and 4,096: forward 33 tiles 14.8 and 12.8, 31 and 29; 44 tiles 14.8 and 14.8, 31
// and 35; 55 tiles 14.8 and 16.9, 31 and 35; backward 36 tiles 23 and 21, 42 and 37; 48
// tiles 23 and 27, 42 and 54).  Otherwise the single-CTA tile and the split of K with
// the smallest estimated time: rounds of units over ~152 CTAs, each as long as its
// MMAs (a 64-deep block takes about 512 cycles whatever the tile's width) or its
// epilogue, and the weights' way from memory.  A split costs the second launch and
// the raw sums' way through memory.
GluPlan plan(long long T, int K, int N, bool bwd) {
  const int kb = (K + GBK - 1) / GBK, pair_hid = bwd ? 256 : 128;
  if (T > 128 && N > pair_hid / 2 &&
      (T + 255) / 256 * ((N + pair_hid - 1) / pair_hid) >= 40)
    return {kGluPair, pair_hid, 1, kb};
  GluPlan best{};
  double best_cycles = 1e300;
  for (int i = 0; i < 2; ++i) {
    const GluTile tile = bwd ? (i ? kGluNarrow : kGluWide) : (i ? kGluWide : kGluTall);
    const int hid = i ? 64 : 128;
    if (i == 0 && N <= hid / 2) continue;
    const long long tiles = (T + 127) / 128 * ((N + hid - 1) / hid);
    for (int s = 1; s <= 16; ++s) {
      if (s > 1 && (s > kb / 2 || tiles * s > 304)) break;
      const int per = (kb + s - 1) / s, splits = (kb + per - 1) / per;
      const double rounds = (double)((tiles * splits + 151) / 152);
      const double epilogue = tile == kGluTall ? (splits > 1 ? 8000 : 12000) : 4500;
      const double mma = per * 512., read = (double)K * N * (bwd ? 2 : 4) / 3500;
      double cycles = rounds * (mma > epilogue ? mma : epilogue);
      cycles = (cycles > read ? cycles : read) + epilogue;
      if (splits > 1) cycles += 5000 + splits * (double)T * N * (bwd ? 8 : 16) / 1750;
      if (cycles < best_cycles) {
        best_cycles = cycles;
        best = {tile, hid, splits, per};
      }
    }
  }
  return best;
}

// Epilogue warps of a pair: twelve, whose 128 registers hold a unit of the forward
// without spills (65,536 x 512 -> 1,408 bf16 SiLU with 8-bit g and u: sixteen 167 us,
// twelve 151, eight 153; without kept values 127, 122, 120; GELU and 8-bit values
// 174, 164, 167); eight where both are kept in 16 bits, whose boxes would take an
// operand stage beside twelve (171, 163, 149).
template <int H16, int MODE>
mlp_status launch(const GluMaps& maps, const GluParams& p, GluTile tile, cudaStream_t st) {
  constexpr int EW = MODE == kGluFwdKeep ? 8 : 12;
  if (tile == kGluPair)
    return glu_whole(p, false) ? launch_glu_pair<5, EW, H16, MODE, true>(maps, p, st)
                               : launch_glu_pair<5, EW, H16, MODE, false>(maps, p, st);
  // Up to 32 rows a stage holds just those, and five stages fit instead of four (us
  // with this and with whole tiles, 16 to 32 rows, cold weights: 4,096 -> 11,008 42.5
  // and 45.4; 4,096 -> 1,361, 512 -> 1,408 and 8,192 -> 8,192 the same within 0.2).
  if (tile == kGluTall)
    return p.a_bytes <= 32 * GBK * 2 ? launch_glu_single<256, 5, 4, 32, H16, MODE>(maps, p, st)
                                     : launch_glu_single<256, 4, 4, 128, H16, MODE>(maps, p, st);
  return launch_glu_single<128, 5, 8, 128, H16, MODE>(maps, p, st);
}

template <int H16>
mlp_status launch_mode(const GluMaps& maps, const GluParams& p, GluTile tile, cudaStream_t st) {
  return p.a.o[0] ? launch<H16, kGluFwdKeep>(maps, p, tile, st)
                  : launch<H16, kGluFwd>(maps, p, tile, st);
}

}  // namespace

int glu_tc_splits(long long T, int K, int N, bool bwd) { return plan(T, K, N, bwd).splits; }

mlp_status launch_glu_tc(const GluArgs& a, bool bwd, cudaStream_t st) {
  const GluPlan pl = plan(a.T, a.K, a.N, bwd);
  if (bwd) return launch_glu_bwd_tc(a, pl, st);
  GluMaps maps;
  GluParams p;
  MLP_CHECK(glu_setup(a, pl, false, maps, p));
  return a.dtype == MLP_DTYPE_F16 ? launch_mode<1>(maps, p, pl.tile, st)
                                  : launch_mode<0>(maps, p, pl.tile, st);
}

}  // namespace mlp
