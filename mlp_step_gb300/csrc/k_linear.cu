// Linear layers on the tensor cores: the product of 16-bit operands with the
// whole layer in its epilogue, fp32 from the accumulator to the one rounding
// of each output.
//   forward:   u = x W + bias,  y = f(u) + residual;  u optionally stored, in
//              the operand type or in 8 bits
//   backward:  du = (dy W^T) f'(u), u read from either form; optionally
//              a = f(u) (the operand of the next weight gradient) and the
//              column sums of du (the bias gradient)
// A group of the 8-bit form is 32 columns of a row: exactly the piece of the
// accumulator that one thread reads from tensor memory at a time, so its
// largest magnitude needs no exchange between threads.
//
// Tiles: CTA pairs (cta_group::2) on 256 x 256 tiles where there are enough
// of them to fill the GPU, single CTAs on 128 rows x 64 to 256 columns
// otherwise, with the contraction split over CTAs when even those are few
// (raw sums to a workspace, finished by launch_linear_finish).  Warps: TMA
// producer, MMA issuer, four to sixteen epilogue warps (a tensor-memory lane
// quarter and a share of the columns each); two accumulators, so that the
// epilogue of one tile overlaps the MMAs of the next.  W is read as it is
// stored: [K][N] as an N-major operand, [N][K] (backward) as a K-major one.
// The kernel's body is in linear_tc.cuh; pairs whose pieces are all whole run
// the form of k_linear_whole.cu, this file has the rest and the choice.
//
// Bound: the MMAs for long K (16,384 x 8,192 -> 8,192 fp16, SiLU and residual:
// 1,240 us = 1.77 PFLOP/s, 93 % of the library's rate; 65,536 x 1,536 -> 512
// bf16 with residual: 75 us = 1.38 PFLOP/s).  For K of a few hundred, the
// operands' way into shared memory (65,536 x 512 -> 1,536 bf16 without an
// activation: 82 us, of which 64 are loads and MMAs) or the epilogue (GELU and
// 8-bit pre-activations: 105 us, backward with kept outputs and column sums:
// 163 us = 22 and 31 instructions an output, issued in 55 and 57 % of the slots:
// the latencies of the rest are what sixteen warps, all that the registers
// hold, leave uncovered).
#include <cstring>

#include "linear_tc.cuh"

namespace mlp {

namespace {

template <int BN, int STAGES, int EW, int AROWS, int H16, int MODE>
__global__ void __launch_bounds__(LinLayout<0, BN, STAGES, EW, AROWS>::THREADS, 1)
    linear_kernel(const __grid_constant__ LinMaps maps, const __grid_constant__ LinParams p) {
  linear_body<0, BN, STAGES, EW, AROWS, H16, MODE, kAny>(maps, p);
}

// ------------------------------------------------------------ plan and launch

// Output tiles: 256 x 256 of a CTA pair, or 128 rows of one CTA.
enum Tile { kPair, kTall, kWide, kNarrow };
constexpr int kTileN[] = {256, 256, 128, 64};

struct LinPlan {
  Tile tile;
  int splits, kb_per_split;
};

// From the shape alone (so that workspace sizes do not depend on the device).
// Pairs when their tiles fill most of ~76 pairs: at 48 tiles a K of 512 takes
// 13.0 us in the best single tiles and 11.1 in pairs, 4,096 takes 35.0 and 27.2;
// at 36 9.3 and 10.7, 24.8 and 26.1 (residual; from 39 on the single tiles need a
// second round and pairs are ahead there too: 12.6 and 10.9 at 40).  Otherwise the single-CTA tile
// and the split of K with the smallest estimated time: rounds of units over
// ~152 CTAs, each as long as its MMAs or its epilogue.  A 64-deep block takes
// about 512 cycles of a CTA's MMAs whatever the tile's width (measured: 500 in
// 128 x 64 tiles), so wide tiles win as soon as they are enough to go round,
// and splitting K makes them enough for few rows (16 rows x 8,192 x 8,192: 42
// us in 128 x 64 tiles, 31 in 128 x 256 with K in two).  A split costs the
// second launch and the raw sums' way through memory.
LinPlan linear_plan(long long T, int K, int N) {
  const int kb = (K + BK - 1) / BK;
  if (T > 128 && N > 128 && (T + 255) / 256 * ((N + 255) / 256) >= 48) return {kPair, 1, kb};
  LinPlan best{};
  double best_cycles = 1e300;
  for (int tile = kTall; tile <= kNarrow; ++tile) {
    if (tile != kNarrow && N <= kTileN[tile] / 2) continue;
    const long long tiles = (T + 127) / 128 * ((N + kTileN[tile] - 1) / kTileN[tile]);
    for (int s = 1; s <= 16; ++s) {
      if (s > 1 && (s > kb / 2 || tiles * s > 304)) break;
      const int per = (kb + s - 1) / s, splits = (kb + per - 1) / per;
      const double rounds = (double)((tiles * splits + 151) / 152);
      const double epilogue = tile == kTall ? (splits > 1 ? 8000 : 12000) : 4000;
      const double mma = per * 512., read = (double)K * N * 2 / 3500;  // W at ~6.8 TB/s
      double cycles = rounds * (mma > epilogue ? mma : epilogue);
      cycles = (cycles > read ? cycles : read) + epilogue;
      if (splits > 1) cycles += 5000 + splits * (double)T * N * 8 / 1750;  // at half that
      if (cycles < best_cycles) {
        best_cycles = cycles;
        best = {(Tile)tile, splits, per};
      }
    }
  }
  return best;
}

template <int BN, int STAGES, int EW, int AROWS, int H16, int MODE>
mlp_status launch_single(const LinMaps& maps, const LinParams& p, cudaStream_t st) {
  using L = LinLayout<0, BN, STAGES, EW, AROWS>;
  auto kernel = linear_kernel<BN, STAGES, EW, AROWS, H16, MODE>;
  static PerDevice configured;
  if (!allow_smem(configured, kernel, L::SMEM)) return MLP_ERR_CUDA;
  const int grid = p.units < num_sms() ? p.units : num_sms();
  LaunchScope ls(MODE != kFwd ? "linear_bwd" : "linear_fwd", st, p.a.T, p.a.N, p.a.K);
  launch_k(kernel, dim3(grid), dim3(L::THREADS), L::SMEM, st, maps, p);
  return launch_status();
}

template <int H16, int MODE>
mlp_status launch_tile(const LinMaps& maps, const LinParams& p, Tile tile, cudaStream_t st) {
  switch (tile) {
    case kPair:
      return launch_pairs<H16, MODE, kAny>(maps, p, st);
    case kTall:
      return p.a_bytes <= 32 * BK * 2 ? launch_single<256, 5, 4, 32, H16, MODE>(maps, p, st)
                                      : launch_single<256, 4, 4, 128, H16, MODE>(maps, p, st);
    case kWide: return launch_single<128, 5, 8, 128, H16, MODE>(maps, p, st);
    default: return launch_single<64, 7, 4, 128, H16, MODE>(maps, p, st);
  }
}

}  // namespace

int linear_tc_splits(long long T, int K, int N) { return linear_plan(T, K, N).splits; }

mlp_status launch_linear_tc(const LinearArgs& a, bool bwd, cudaStream_t st) {
  const LinPlan pl = linear_plan(a.T, a.K, a.N);
  const int tile_m = pl.tile == kPair ? 256 : 128;
  const int tile_n = kTileN[pl.tile];
  const long long tm = (a.T + tile_m - 1) / tile_m, tn = (a.N + tile_n - 1) / tile_n;
  if (tm * tn * pl.splits > (1ll << 30)) return MLP_ERR_UNSUPPORTED_SHAPE;
  LinParams p{};
  p.a = a;
  p.a.splits = pl.splits;
  p.tiles_m = (int)tm;
  p.tiles_n = (int)tn;
  p.units = (int)(tm * tn * pl.splits);
  p.magic = (unsigned)(((1ull << 32) + 8 * tn - 1) / (8 * tn));
  p.k_blocks = (a.K + BK - 1) / BK;
  p.kb_per_split = pl.kb_per_split;
  p.wait_ns = wait_limit_ns();
  p.err = device_error_word();
  if (!p.err) return MLP_ERR_CUDA;

  LinMaps maps;
  memset(&maps, 0, sizeof(maps));
  auto map16 = [](CUtensorMap* map, const void* base, long long cols, long long rows, long long ld,
                  unsigned box_cols, unsigned box_rows) {
    return encode_tmap_bf16_2d(map, base, cols, rows, (unsigned long long)ld * 2, box_cols,
                               box_rows);
  };
  // A single-CTA tile of few rows loads just those (in eights): the stale rows
  // behind them only feed accumulator rows that are never stored.
  const int a_rows = pl.tile != kPair && a.T < 128 ? (int)(a.T + 7) / 8 * 8 : 128;
  p.a_bytes = a_rows * BK * 2;
  if (!map16(&maps.a, a.x, a.K, a.T, a.ldx, BK, a_rows)) return MLP_ERR_CUDA;
  if (!(bwd ? map16(&maps.b, a.w, a.K, a.N, a.ldw, BK, pl.tile == kPair ? 128 : tile_n)
            : map16(&maps.b, a.w, a.N, a.K, a.ldw, 64, BK)))
    return MLP_ERR_CUDA;
  // What the epilogue reads and writes moves by TMA where rows start on 16
  // bytes.  (A row per thread straight between registers and memory touches 32
  // lines an instruction: 65,536 x 512 -> 1,536 took 70 us more for a residual
  // that way, 42 us for the 8-bit values.)
  if (pl.splits == 1) {
    auto rows16 = [](const void* ptr, long long ld, int esz) {
      return ptr && aligned16(ptr) && ld * esz % 16 == 0;
    };
    const int esz = a.out_f32 ? 4 : 2;
    p.y64 = !a.out_f32 && !a.u_out;
    if (rows16(a.y, a.ldy, esz)) {
      if (!(p.y64 ? map16(&maps.y, a.y, a.N, a.T, a.ldy, 64, 32)
                  : encode_tmap_out_2d(&maps.y, a.y, a.out_f32, a.N, a.T,
                                       (unsigned long long)a.ldy * esz, 32, 32)))
        return MLP_ERR_CUDA;
      p.tma_y = 1;
    }
    if (!a.out_f32 && rows16(a.u_out, a.ldu_out, 2)) {
      if (!encode_tmap_out_2d(&maps.u, a.u_out, 0, a.N, a.T, (unsigned long long)a.ldu_out * 2, 32,
                              32))
        return MLP_ERR_CUDA;
      p.tma_u = 1;
    }
    const void* in = bwd ? a.u_in : a.res;
    const long long ld_in = bwd ? a.ldu_in : a.ldr;
    if (p.y64 && rows16(in, ld_in, 2)) {
      if (!map16(&maps.in, in, a.N, a.T, ld_in, 64, 32)) return MLP_ERR_CUDA;
      p.tma_in = 1;
    }
    if (rows16(a.q, a.ldq, 1)) {
      if (!encode_tmap_u8_2d(&maps.q, a.q, a.N, a.T, a.ldq, 64, 32)) return MLP_ERR_CUDA;
      p.tma_q = 1;
    }
  }
  const void* in16 = bwd ? a.u_in : a.res;
  if (pl.tile == kPair && a.N % 64 == 0 && !a.out_f32 && p.tma_y && (!a.q || p.tma_q)) {
    const int mode = !bwd ? kFwd : a.q ? kBwdCkpt : kBwd;
    if (!a.u_out && (!in16 || p.tma_in)) return launch_linear_whole(maps, p, mode, kWhole64, st);
    if (p.tma_u && !in16 && mode != kBwd) return launch_linear_whole(maps, p, mode, kWhole32, st);
  }
  const bool h16 = a.dtype == MLP_DTYPE_F16;
  if (!bwd)
    return h16 ? launch_tile<1, kFwd>(maps, p, pl.tile, st)
               : launch_tile<0, kFwd>(maps, p, pl.tile, st);
  if (a.q)
    return h16 ? launch_tile<1, kBwdCkpt>(maps, p, pl.tile, st)
               : launch_tile<0, kBwdCkpt>(maps, p, pl.tile, st);
  return h16 ? launch_tile<1, kBwd>(maps, p, pl.tile, st)
             : launch_tile<0, kBwd>(maps, p, pl.tile, st);
}

}  // namespace mlp
