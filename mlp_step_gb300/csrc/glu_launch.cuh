// How a gated unit's product is tiled, and the launch of its kernels; included
// by k_glu.cu (forward) and k_glu_bwd.cu.
#pragma once

#include <cstring>

#include "glu_tc.cuh"

namespace mlp {

// Tiles of a CTA pair, or of one CTA: 256 accumulator columns (forward only),
// 128, 64 (backward only).
enum GluTile { kGluPair, kGluTall, kGluWide, kGluNarrow };

struct GluPlan {
  GluTile tile;
  int hid;  // hidden columns of a tile
  int splits, kb_per_split;
};

namespace {

template <int BN, int STAGES, int EW, int AROWS, int H16, int MODE>
__global__ void
    __launch_bounds__(GluLayout<0, BN, STAGES, EW, AROWS, MODE>::THREADS, 1)
    glu_kernel(const __grid_constant__ GluMaps maps, const __grid_constant__ GluParams p) {
  glu_body<0, BN, STAGES, EW, AROWS, H16, MODE, false>(maps, p);
}

template <int BN, int STAGES, int EW, int AROWS, int H16, int MODE>
mlp_status launch_glu_single(const GluMaps& maps, const GluParams& p, cudaStream_t st) {
  using L = GluLayout<0, BN, STAGES, EW, AROWS, MODE>;
  auto kernel = glu_kernel<BN, STAGES, EW, AROWS, H16, MODE>;
  static PerDevice configured;
  if (!allow_smem(configured, kernel, L::SMEM)) return MLP_ERR_CUDA;
  const int grid = p.units < num_sms() ? p.units : num_sms();
  LaunchScope ls(glu_is_bwd(MODE) ? "glu_bwd" : "glu_fwd", st, p.a.T, p.a.N, p.a.K);
  launch_k(kernel, dim3(grid), dim3(L::THREADS), L::SMEM, st, maps, p);
  return launch_status();
}

// Everything of a launch but the choice of its kernel.
mlp_status glu_setup(const GluArgs& a, const GluPlan& pl, bool bwd, GluMaps& maps, GluParams& p) {
  const int tile_m = pl.tile == kGluPair ? 256 : 128;
  const long long tm = (a.T + tile_m - 1) / tile_m, tn = (a.N + pl.hid - 1) / pl.hid;
  if (tm * tn * pl.splits > (1ll << 30)) return MLP_ERR_UNSUPPORTED_SHAPE;
  p = GluParams{};
  p.a = a;
  p.a.splits = pl.splits;
  p.tiles_m = (int)tm;
  p.tiles_n = (int)tn;
  p.units = (int)(tm * tn * pl.splits);
  p.magic = (unsigned)(((1ull << 32) + 8 * tn - 1) / (8 * tn));
  p.k_blocks = (a.K + GBK - 1) / GBK;
  p.kb_per_split = pl.kb_per_split;
  p.wait_ns = wait_limit_ns();
  p.err = device_error_word();
  if (!p.err) return MLP_ERR_CUDA;
  memset(&maps, 0, sizeof(maps));
  auto operand = [](CUtensorMap* map, const void* base, long long cols, long long rows,
                    long long ld, unsigned box_cols, unsigned box_rows) {
    return encode_tmap_bf16_2d(map, base, cols, rows, (unsigned long long)ld * 2, box_cols,
                               box_rows);
  };
  // A single-CTA tile of few rows loads just those (in eights): the stale rows
  // behind them only feed accumulator rows that are never stored.
  const int a_rows = pl.tile != kGluPair && a.T < 128 ? (int)(a.T + 7) / 8 * 8 : 128;
  p.a_bytes = a_rows * GBK * 2;
  bool ok = operand(&maps.x, a.x, a.K, a.T, a.ldx, GBK, a_rows);
  if (bwd) {
    ok = ok && operand(&maps.w[0], a.w[0], a.K, a.N, a.ldw[0], GBK,
                       pl.tile == kGluPair ? 128 : pl.hid);
  } else {
    for (int k = 0; k < 2; ++k)
      ok = ok && operand(&maps.w[k], a.w[k], a.N, a.K, a.ldw[k], 64, GBK);
  }
  // What the epilogue reads and writes moves by TMA where rows start on 16 bytes.
  if (pl.splits == 1) {
    auto rows16 = [](const void* ptr, long long ld, int esz) {
      return ptr && aligned16(ptr) && ld * esz % 16 == 0;
    };
    auto box16 = [&](CUtensorMap* map, const void* base, long long ld) {
      return encode_tmap_out_2d(map, base, 0, a.N, a.T, (unsigned long long)ld * 2, 32, 32);
    };
    auto box8 = [&](CUtensorMap* map, const void* base, long long ld) {
      return encode_tmap_u8_2d(map, base, a.N, a.T, (unsigned long long)ld, 32, 32);
    };
    const bool q16 = rows16(a.q[0], a.ldq[0], 1) && rows16(a.q[1], a.ldq[1], 1);
    p.tma_y = rows16(a.y, a.ldy, 2);
    if (p.tma_y) ok = ok && box16(&maps.y, a.y, a.ldy);
    if (a.o[0]) p.tma_o = rows16(a.o[0], a.ldo[0], 2) && rows16(a.o[1], a.ldo[1], 2);
    else if (!bwd && a.q[0]) p.tma_o = q16;
    if (bwd) p.tma_in = a.q[0] ? q16 : rows16(a.in[0], a.ld_in[0], 2) && rows16(a.in[1], a.ld_in[1], 2);
    for (int k = 0; k < 2; ++k) {
      if (p.tma_o)
        ok = ok && (a.o[0] ? box16(&maps.o[k], a.o[k], a.ldo[k])
                           : box8(&maps.o[k], a.q[k], a.ldq[k]));
      if (p.tma_in)
        ok = ok && (a.q[0] ? box8(&maps.in[k], a.q[k], a.ldq[k])
                           : box16(&maps.in[k], a.in[k], a.ld_in[k]));
    }
  }
  return ok ? MLP_OK : MLP_ERR_CUDA;
}

// Whether all pieces are whole and everything present moves by TMA.
bool glu_whole(const GluParams& p, bool bwd) {
  const GluArgs& a = p.a;
  const bool kept = bwd || a.o[0] || a.q[0];
  return a.N % 32 == 0 && (!a.y || p.tma_y) && (!kept || p.tma_o) && (!bwd || p.tma_in);
}

}  // namespace

// k_glu_bwd.cu
mlp_status launch_glu_bwd_tc(const GluArgs& a, const GluPlan& pl, cudaStream_t st);

}  // namespace mlp
