// The kernel body of the 16-bit gated units (k_glu.cu tells its shape), its
// parameters, and the launch of CTA pairs.
#pragma once

#include "act.cuh"
#include "ckpt8.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "tile_epilogue.cuh"
#include "trace.cuh"

namespace mlp {

struct GluParams {
  GluArgs a;
  int tiles_m, tiles_n, units, k_blocks, kb_per_split;
  unsigned magic;  // of tile_of
  int a_bytes;     // of a stage's x tile: fewer than 128 rows when there are fewer
  // What moves by TMA: y (backward a); the kept pre-activations (backward dg
  // and du); the backward's saved pre-activations
  int tma_y, tma_o, tma_in;
  unsigned long long wait_ns;
  int* err;
};

// Tensor maps of a launch: operands (w[1]: the forward's up projection), y / a,
// kept / gradients, saved.
struct GluMaps {
  CUtensorMap x, w[2], y, o[2], in[2];
};

namespace {

constexpr int GBK = 64;
constexpr int kGluBox = 2048;  // 32 rows x 64 bytes (8-bit values: 32 bytes a row)

// MODE: forward that keeps its pre-activations in 16 bits, or in 8 or not at all;
// backward from 16-bit pre-activations, from 8-bit ones.
enum { kGluFwdKeep, kGluFwd, kGluBwd, kGluBwdCkpt };
constexpr bool glu_is_bwd(int mode) { return mode >= kGluBwd; }

// EW: epilogue warps.  AROWS: rows of x that a stage holds; with fewer than 128
// the MMA reads on into what follows, which only feeds accumulator rows that
// are never stored.  The forward's accumulator is half gate, half up columns of
// the same hidden columns.  Staging boxes of an epilogue warp: y, g, u (8-bit
// ones are half as large); backward: saved g and u, dg, du, a.
template <int PAIR, int BN, int STAGES, int EW, int AROWS, int MODE>
struct GluLayout {
  static constexpr bool BWD = glu_is_bwd(MODE);
  static constexpr int A_BYTES = AROWS * GBK * 2;
  static constexpr int B_COLS = PAIR ? 128 : BN;  // operand columns staged per CTA
  static constexpr int B_BYTES = B_COLS * GBK * 2;
  static constexpr int ACC = PAIR ? 256 : BN;       // accumulator columns per CTA
  static constexpr int HID = BWD ? ACC : ACC / 2;   // hidden columns of a tile
  static constexpr int PIECES = HID / 32;           // units of a lane quarter's warps in a tile
  static constexpr int SHARE = EW / 4;              // ... and these warps
  static constexpr int KEPT = MODE == kGluFwdKeep || MODE == kGluBwd ? kGluBox : kGluBox / 2;
  static constexpr int STAGE = (BWD ? 3 : 1) * kGluBox + 2 * KEPT;
  static constexpr int THREADS = 64 + 32 * EW;      // + producer, MMA issuer
  static constexpr int SMEM = 1024 + STAGES * (A_BYTES + B_BYTES) + EW * STAGE + 1024;
  static constexpr uint32_t TMEM_COLS = 2 * ACC;
  static_assert(PIECES >= SHARE, "every epilogue warp has a unit of every tile");
  static_assert(SMEM <= 232448, "shared memory");
};

// 32 accumulator columns of this warp's rows.
__device__ __forceinline__ void take32(uint32_t addr, F2 (&v)[16]) {
  uint32_t r[32];
  __syncwarp();
  ptx::tmem_ld_32x32b_x32(addr, r);
  ptx::tmem_ld_wait();
#pragma unroll
  for (int j = 0; j < 16; ++j)
    v[j] = f2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
}

// A piece's raw sums into their plane (whole 32-column pieces: ldp a multiple of 32).
__device__ __forceinline__ void store_raw(float* p, const F2 (&v)[16]) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    reinterpret_cast<float4*>(p)[k] =
        make_float4(v[2 * k].x, v[2 * k].y, v[2 * k + 1].x, v[2 * k + 1].y);
}

// WHOLE: every piece is whole, everything moves by TMA and K is not split, so
// that the epilogue's scalar work is decided when it is compiled.
template <int PAIR, int BN, int STAGES, int EW, int AROWS, int H16, int MODE, bool WHOLE>
__device__ __forceinline__ void glu_body(const GluMaps& maps, const GluParams& p) {
  constexpr bool BWD = glu_is_bwd(MODE), CK = MODE == kGluBwdCkpt;
  using L = GluLayout<PAIR, BN, STAGES, EW, AROWS, MODE>;
  constexpr int KEPT = L::KEPT;
  static_assert(AROWS == 128 || (STAGES * L::B_BYTES >= 16384 && !PAIR), "reads past the x ring");
  constexpr int ACC = L::ACC, HID = L::HID;
  constexpr int TILE_M = PAIR ? 256 : 128;
  constexpr bool B_MN = !BWD;  // W [K][N] is an N-major operand, W [N][K] a K-major one
  const GluArgs& a = p.a;
  const int splits = WHOLE ? 1 : a.splits;
  const bool tma_y = WHOLE || p.tma_y, tma_o = WHOLE || p.tma_o, tma_in = WHOLE || p.tma_in;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + STAGES * L::A_BYTES;
  uint8_t* stg = sB + STAGES * L::B_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(stg + EW * L::STAGE);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  uint64_t* in_full = done + 1;  // per epilogue warp: its saved values have landed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(in_full + EW);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  // warp-uniform to the compiler, which then keeps what follows from it in
  // uniform registers
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? blockIdx.x & 1u : 0u;  // in the cluster of two
  const int worker = PAIR ? blockIdx.x >> 1 : blockIdx.x;
  const int workers = PAIR ? gridDim.x >> 1 : gridDim.x;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 1);
    }
    for (int k = 0; k < 2; ++k) {
      ptx::mbar_init(&tfull[k], 1);
      ptx::mbar_init(&tempty[k], PAIR ? 2 * EW : EW);
    }
    for (int w = 0; w < EW; ++w) ptx::mbar_init(&in_full[w], 1);
    ptx::mbar_init(done, 1);
    *s_abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&maps.x);
    ptx::prefetch_tensormap(&maps.w[0]);
    if (!BWD) ptx::prefetch_tensormap(&maps.w[1]);
    if (p.tma_y) ptx::prefetch_tensormap(&maps.y);
    for (int k = 0; k < 2; ++k) {
      if (p.tma_o) ptx::prefetch_tensormap(&maps.o[k]);
      if (p.tma_in) ptx::prefetch_tensormap(&maps.in[k]);
    }
  }
  if (warp == 1) {
    if constexpr (PAIR) ptx::tmem_alloc_pair(tmem_slot, L::TMEM_COLS);
    else ptx::tmem_alloc(tmem_slot, L::TMEM_COLS);
  }
  ptx::tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) ptx::cluster_sync();  // both CTAs' barriers exist before any signal
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  pdl_launch_dependents();

  // k-blocks of unit u's split
  auto k_range = [&](int u, int& kb0, int& kb1) {
    kb0 = u % splits * p.kb_per_split;
    kb1 = min(p.k_blocks, kb0 + p.kb_per_split);
  };
  int last_parity[STAGES];  // of the producer's stages: what may be in flight after an abort

  if (warp == 0) {
    if (lane == 0) {
      for (int s = 0; s < STAGES; ++s) last_parity[s] = -1;
      const uint32_t full0 = PAIR ? ptx::mapa_shared(ptx::smem_u32(full), 0) : 0u;
      int stage = 0;
      uint32_t phase = 0;
      for (int u = worker; u < p.units && !*s_abort; u += workers) {
        int tm, tn, kb0, kb1;
        tile_of(p, splits == 1 ? u : u / splits, tm, tn);
        k_range(u, kb0, kb1);
        const int m0 = tm * TILE_M + (int)rank * 128;
        // forward: the hidden columns of both weights (of a pair, the even CTA
        // stages the gate's and the odd one the up projection's)
        const int n0 = tn * HID + (BWD ? (int)rank * L::B_COLS : 0);
        for (int kb = kb0; kb < kb1; ++kb) {
          const bool ok = PAIR ? ptx::mbar_wait_cluster_bounded(&empty[stage], phase ^ 1, p.wait_ns,
                                                                p.err, DEVERR_TIMEOUT_PRODUCER)
                               : ptx::mbar_wait_bounded(&empty[stage], phase ^ 1, p.wait_ns, p.err,
                                                        DEVERR_TIMEOUT_PRODUCER);
          if (!ok) {
            *s_abort = 1;
            break;
          }
          uint8_t* da = sA + stage * L::A_BYTES;
          uint8_t* db = sB + stage * L::B_BYTES;
          const int k0 = kb * GBK;
          if constexpr (PAIR) {
            if (rank == 0) {
              ptx::mbar_arrive_expect_tx(&full[stage], 2 * (L::A_BYTES + L::B_BYTES));
              last_parity[stage] = (int)phase;
            }
            const uint32_t bar = full0 + (uint32_t)stage * 8u;
            ptx::tma_load_2d_pair(da, &maps.x, bar, k0, m0);
            if constexpr (B_MN) {
              const CUtensorMap* w = rank ? &maps.w[1] : &maps.w[0];
              ptx::tma_load_2d_pair(db, w, bar, n0, k0);
              ptx::tma_load_2d_pair(db + 8192, w, bar, n0 + 64, k0);
            } else {
              ptx::tma_load_2d_pair(db, &maps.w[0], bar, k0, n0);
            }
          } else {
            // 64-wide boxes entirely past N are not loaded: they only feed
            // accumulator columns that are never stored
            constexpr int HB = BN / 128;  // boxes of either weight
            uint32_t bytes = p.a_bytes + L::B_BYTES;
            if constexpr (B_MN) {
#pragma unroll
              for (int j = 1; j < HB; ++j)
                if (n0 + 64 * j >= a.N) bytes -= 2 * 8192u;
            }
            ptx::mbar_arrive_expect_tx(&full[stage], bytes);
            last_parity[stage] = (int)phase;
            ptx::tma_load_2d(da, &maps.x, &full[stage], k0, m0);
            if constexpr (B_MN) {
#pragma unroll
              for (int j = 0; j < HB; ++j)
                if (j == 0 || n0 + 64 * j < a.N) {
                  ptx::tma_load_2d(db + 8192 * j, &maps.w[0], &full[stage], n0 + 64 * j, k0);
                  ptx::tma_load_2d(db + 8192 * (HB + j), &maps.w[1], &full[stage], n0 + 64 * j,
                                   k0);
                }
            } else {
              ptx::tma_load_2d(db, &maps.w[0], &full[stage], k0, n0);
            }
          }
          if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = ptx::idesc_16_f32<H16>(TILE_M, ACC, 0, B_MN ? 1 : 0);
      constexpr uint32_t b_lbo = B_MN ? 8192u : 16u, b_kstep = B_MN ? 2048u : 32u;
      const uint64_t ad0 = ptx::sw128_desc(ptx::smem_u32(sA), 16, 1024);
      const uint64_t bd0 = ptx::sw128_desc(ptx::smem_u32(sB), b_lbo, 1024);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      for (int u = worker; u < p.units && !*s_abort; u += workers) {
        const bool free = PAIR ? ptx::mbar_wait_cluster_bounded(&tempty[acc], acc_phase ^ 1,
                                                                p.wait_ns, p.err,
                                                                DEVERR_TIMEOUT_MMA)
                               : ptx::mbar_wait_bounded(&tempty[acc], acc_phase ^ 1, p.wait_ns,
                                                        p.err, DEVERR_TIMEOUT_MMA);
        if (!free) {
          *s_abort = 1;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t d = tmem_base + (uint32_t)(acc * ACC);
        int kb0, kb1;
        k_range(u, kb0, kb1);
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!ptx::mbar_wait_bounded(&full[stage], phase, p.wait_ns, p.err, DEVERR_TIMEOUT_MMA)) {
            *s_abort = 1;
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint64_t ad = ad0 + (uint32_t)(stage * (L::A_BYTES >> 4));
          const uint64_t bd = bd0 + (uint32_t)(stage * (L::B_BYTES >> 4));
#pragma unroll
          for (int k = 0; k < GBK / 16; ++k) {
            const uint32_t add = kb > kb0 || k > 0;
            if constexpr (PAIR)
              ptx::mma_bf16_pair(d, ad + k * 2, bd + k * (b_kstep >> 4), idesc, add);
            else
              ptx::mma_bf16(d, ad + k * 2, bd + k * (b_kstep >> 4), idesc, add);
          }
          if constexpr (PAIR) ptx::mma_commit_pair_multicast(&empty[stage], 3);
          else ptx::mma_commit(&empty[stage]);
          if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
        if (!ok) break;
        if constexpr (PAIR) ptx::mma_commit_pair_multicast(&tfull[acc], 3);
        else ptx::mma_commit(&tfull[acc]);
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
      if constexpr (PAIR) ptx::mma_commit_pair_multicast(done, 1);
      else ptx::mma_commit(done);
      ptx::mbar_wait_bounded(done, 0, p.wait_ns, p.err, DEVERR_TIMEOUT_TEARDOWN);
    }
  } else {
    const int ew = warp - 2;
    const int quarter = warp & 3;  // tensor-memory lanes [32 q, 32 q + 32)
    const uint32_t tempty0 = PAIR ? ptx::mapa_shared(ptx::smem_u32(tempty), 0) : 0u;
    uint8_t* in_box = stg + ew * L::STAGE;                  // backward: saved g, u
    uint8_t* out_box = in_box + (BWD ? 2 * KEPT : 0);       // y, g, u; dg, du, a
    bool stores = false;      // a store of this warp may still read its boxes
    bool in_flight = false;   // saved values are on their way
    uint32_t in_phase = 0;
    uint32_t sb[2] = {0, 0};  // their scale bytes of this row

    // One unit is 32 columns of the warp's 32 rows; units go tile by tile, dealt
    // in turn over the warps of a lane quarter: `start` is this warp's first in
    // the tile.
    struct Unit {
      int row0, n0;
    };
    auto locate = [&](int u, int c) {
      Unit t{0, a.N};
      if (u < p.units) {
        int tm, tn;
        tile_of(p, splits == 1 ? u : u / splits, tm, tn);
        t.row0 = tm * TILE_M + (int)rank * 128 + quarter * 32;
        t.n0 = tn * HID + c;
      }
      return t;
    };
    auto exists = [&](const Unit& t) { return t.n0 < a.N && t.row0 < a.T; };
    auto boxes_free = [&] {
      if (stores) {
        if (lane == 0) ptx::bulk_wait_group_read<0>();
        __syncwarp();
        stores = false;
      }
    };
    // Requests the saved values of a unit, once every lane has read the last ones.
    auto request = [&](const Unit& t) {
      if (!exists(t)) return;
      if constexpr (CK) {
        const long long m = (long long)t.row0 + lane;
        if (m < a.T) {
#pragma unroll
          for (int k = 0; k < 2; ++k) sb[k] = a.scale[k][m * a.lds[k] + t.n0 / kCkptGroup];
        }
      }
      if (tma_in) {
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(&in_full[ew], 2 * KEPT);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            ptx::tma_load_2d(in_box + k * KEPT, &maps.in[k], &in_full[ew], t.n0, t.row0);
        }
        in_flight = true;
      }
    };
    // The accumulator goes back to the MMA issuer as soon as the warp's last
    // piece of it is in registers.  Relaxed: nothing in memory is handed over
    // (the tensor-memory reads have completed).
    int acc = 0;
    uint32_t acc_phase = 0;
    auto release = [&] {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) ptx::mbar_arrive_relaxed(&tempty[acc]);
        else ptx::mbar_arrive_remote_relaxed(tempty0 + (uint32_t)acc * 8u);
      }
    };

    int start = ew >> 2;
    Unit next = locate(worker, 32 * start);
    if (BWD && splits == 1) request(next);
    for (int u = worker; u < p.units; u += workers) {
      if (*s_abort) break;
      bool ready = false;
      int c = 32 * start;
      start -= L::PIECES % L::SHARE;
      if (start < 0) start += L::SHARE;
      for (; c < HID; c += 32 * L::SHARE) {
        const Unit t = next;
        const bool last = c + 32 * L::SHARE >= HID;
        if (last) next = locate(u + workers, 32 * start);
        else next.n0 += 32 * L::SHARE;
        const long long m = (long long)t.row0 + lane;
        const bool row_ok = m < a.T;
        if (!ready) {
          ready = PAIR ? ptx::mbar_wait_cluster_bounded(&tfull[acc], acc_phase, p.wait_ns, p.err,
                                                        DEVERR_TIMEOUT_EPILOGUE)
                       : ptx::mbar_wait_bounded(&tfull[acc], acc_phase, p.wait_ns, p.err,
                                                DEVERR_TIMEOUT_EPILOGUE);
          if (!ready) break;
          ptx::tc_fence_after();
        }
        if (!exists(t)) {  // warp-uniform
          if (last) release();
          if (BWD && splits == 1) request(next);
          continue;
        }
        const int cols = WHOLE ? 32 : min(32, a.N - t.n0);
        const int rows = (int)min(32ll, a.T - t.row0);
        const uint32_t from = tmem_base + ((uint32_t)(quarter * 32) << 16) +
                              (uint32_t)(acc * ACC + c);
        F2 v[16], w[16];
        if (!WHOLE && splits > 1) {
          // raw sums: gate planes, then (forward) up planes
          const long long plane = a.T * a.ldp;
          float* pr = a.partial + (u % splits) * plane + m * a.ldp + t.n0;
          take32(from, v);
          if (BWD && last) release();
          if (row_ok) store_raw(pr, v);
          if constexpr (!BWD) {
            take32(from + HID, v);
            if (last) release();
            if (row_ok) store_raw(pr + splits * plane, v);
          }
          continue;
        }
        // Ragged pieces do not leave by TMA: the bulk stores write whole 16-byte
        // units, so they would touch columns past N.
        const bool whole = WHOLE || cols == 32;
        auto copy16 = [&](uint8_t* box, void* base, long long ld) {
          warp_copy<true>(box, 64, static_cast<uint8_t*>(base) + (t.row0 * ld + t.n0) * 2, ld * 2,
                          rows, cols * 2, 2, lane);
        };
        if constexpr (!BWD) {
          boxes_free();
          // one projection's piece: bias, and the kept form into its box
          auto projection = [&](int k, F2 (&z)[16]) {
            const float* bias = a.bias[k];
            if (bias && whole) {
              float4 b4[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) b4[j] = load_bias4(bias + t.n0 + 4 * j);
              take32(from + k * HID, z);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                z[2 * j] = add2(z[2 * j], f2(b4[j].x, b4[j].y));
                z[2 * j + 1] = add2(z[2 * j + 1], f2(b4[j].z, b4[j].w));
              }
            } else {
              take32(from + k * HID, z);
            }
            if (k == 1 && last) release();
            if (!whole) {
              // columns past N: zero, so that they take no part in the 8-bit
              // group's scale
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const bool e = 2 * j < cols, o = 2 * j + 1 < cols;
                z[j].x = e ? z[j].x + (bias ? __ldg(bias + t.n0 + 2 * j) : 0.f) : 0.f;
                z[j].y = o ? z[j].y + (bias ? __ldg(bias + t.n0 + 2 * j + 1) : 0.f) : 0.f;
              }
            }
            uint8_t* kept = out_box + kGluBox + k * KEPT;
            if (MODE == kGluFwdKeep) {
              pack_row<H16>(kept, 64, lane, 0, z);
            } else if (a.q[k]) {
              uint32_t q[8];
              const uint32_t b = ckpt8_group(reinterpret_cast<const float(&)[32]>(z), q);
              if (row_ok) a.scale[k][m * a.lds[k] + t.n0 / kCkptGroup] = (uint8_t)b;
              *reinterpret_cast<uint4*>(chunk_at(kept, 32, lane, 0)) =
                  make_uint4(q[0], q[1], q[2], q[3]);
              *reinterpret_cast<uint4*>(chunk_at(kept, 32, lane, 1)) =
                  make_uint4(q[4], q[5], q[6], q[7]);
            }
          };
          projection(0, v);
          with_act(a.act, [&](auto tag) {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = act_value2<decltype(tag)::value>(v[j], a.slope);
          });
          projection(1, w);
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = mul2(v[j], w[j]);
          pack_row<H16>(out_box, 64, lane, 0, v);
          const bool kept = MODE == kGluFwdKeep || a.q[0];
          const bool by_y = tma_y && whole, by_o = kept && tma_o && whole;
          if (by_y || by_o) {
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              // rows past T are clipped by the stores
              if (by_y) ptx::tma_store_2d(&maps.y, out_box, t.n0, t.row0);
              if (by_o) {
                ptx::tma_store_2d(&maps.o[0], out_box + kGluBox, t.n0, t.row0);
                ptx::tma_store_2d(&maps.o[1], out_box + kGluBox + KEPT, t.n0, t.row0);
              }
              ptx::bulk_commit_group();
            }
            stores = true;
          }
          if (!by_y) copy16(out_box, a.y, a.ldy);
          if (kept && !by_o) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              if (MODE == kGluFwdKeep) copy16(out_box + kGluBox + k * KEPT, a.o[k], a.ldo[k]);
              else
                warp_copy<true>(out_box + kGluBox + k * KEPT, 32,
                                reinterpret_cast<uint8_t*>(a.q[k]) + t.row0 * a.ldq[k] + t.n0,
                                a.ldq[k], rows, cols, 1, lane);
            }
          }
        } else {
          // the saved values of this piece, raw
          if (in_flight) {
            if (!ptx::mbar_wait_bounded(&in_full[ew], in_phase, p.wait_ns, p.err,
                                        DEVERR_TIMEOUT_EPILOGUE)) {
              ready = false;
              break;
            }
            in_phase ^= 1;
            in_flight = false;
          }
          if (!tma_in) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              if (CK)
                warp_copy<false>(in_box + k * KEPT, 32,
                                 reinterpret_cast<uint8_t*>(a.q[k]) + t.row0 * a.ldq[k] + t.n0,
                                 a.ldq[k], rows, cols, 1, lane);
              else
                warp_copy<false>(in_box + k * KEPT, 64,
                                 static_cast<uint8_t*>(const_cast<void*>(a.in[k])) +
                                     (t.row0 * a.ld_in[k] + t.n0) * 2,
                                 a.ld_in[k] * 2, rows, cols * 2, 2, lane);
            }
          }
          constexpr int RAW = CK ? 8 : 16;
          uint32_t raw[2][RAW];
          float step[2] = {0.f, 0.f};
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (CK) step[k] = ckpt8_step(sb[k]);
#pragma unroll
            for (int j = 0; j < RAW / 4; ++j) {
              const uint4 q = *reinterpret_cast<const uint4*>(
                  chunk_at(in_box + k * KEPT, CK ? 32 : 64, lane, j));
              raw[k][4 * j] = q.x;
              raw[k][4 * j + 1] = q.y;
              raw[k][4 * j + 2] = q.z;
              raw[k][4 * j + 3] = q.w;
            }
          }
          if (!tma_in) __syncwarp();
          request(next);
          take32(from, v);
          if (last) release();
          boxes_free();
          // values 8 g .. 8 g + 7 of saved matrix k
          auto saved = [&](int k, int g, F2 (&x)[4]) {
            if constexpr (CK) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t f = ckpt8_flip(raw[k][2 * g + e]);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                  x[2 * e + j] = mul2(add2(f2(ckpt8_biased(f, 2 * j), ckpt8_biased(f, 2 * j + 1)),
                                           f2(-kCkptBias)),
                                      f2(step[k]));
              }
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) x[j] = unpack2<H16>(raw[k][4 * g + j]);
            }
          };
          // v: da -> dg,  w: du
          with_act(a.act, [&](auto tag) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              F2 x[4], y[4];
              saved(0, g, x);
              saved(1, g, y);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                F2 f;
                const F2 df = act_grad2<decltype(tag)::value>(x[j], a.slope, f);
                w[4 * g + j] = mul2(v[4 * g + j], f);
                v[4 * g + j] = mul2(v[4 * g + j], mul2(y[j], df));
                x[j] = mul2(f, y[j]);
              }
              if (a.y) pack_row<H16>(out_box + 2 * kGluBox, 64, lane, g, x);
            }
          });
          pack_row<H16>(out_box, 64, lane, 0, v);
          pack_row<H16>(out_box + kGluBox, 64, lane, 0, w);
          const bool by_o = tma_o && whole, by_y = a.y && tma_y && whole;
          if (by_o || by_y) {
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (by_o) {
                ptx::tma_store_2d(&maps.o[0], out_box, t.n0, t.row0);
                ptx::tma_store_2d(&maps.o[1], out_box + kGluBox, t.n0, t.row0);
              }
              if (by_y) ptx::tma_store_2d(&maps.y, out_box + 2 * kGluBox, t.n0, t.row0);
              ptx::bulk_commit_group();
            }
            stores = true;
          }
          if (!by_o) {
            copy16(out_box, a.o[0], a.ldo[0]);
            copy16(out_box + kGluBox, a.o[1], a.ldo[1]);
          }
          if (a.y && !by_y) copy16(out_box + 2 * kGluBox, a.y, a.ldy);
          if (a.colpart) {
            if (!row_ok) {
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] = w[j] = f2(0.f);
            }
            const float s0 = column_sums(v, lane), s1 = column_sums(w, lane);
            if (lane < cols) {
              float* o = a.colpart + (long long)(t.row0 / 32) * a.ldcp + t.n0 + lane;
              o[0] = s0;
              o[a.N] = s1;
            }
          }
        }
      }
      if (!ready) {
        *s_abort = 1;
        break;
      }
      if (++acc == 2) { acc = 0; acc_phase ^= 1; }
    }
    // saved values requested for a unit that an abort skipped
    if (in_flight)
      ptx::mbar_wait_bounded(&in_full[ew], in_phase, p.wait_ns, p.err, DEVERR_TIMEOUT_TEARDOWN);
    // bulk stores read shared memory: they finish before the CTA leaves
    if (lane == 0) ptx::bulk_wait_group<0>();
    __syncwarp();
  }

  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (*s_abort && warp == 0 && lane == 0) {
    for (int s = 0; s < STAGES; ++s)
      if (last_parity[s] >= 0)
        ptx::mbar_wait_bounded(&full[s], (uint32_t)last_parity[s], p.wait_ns, p.err,
                               DEVERR_TIMEOUT_TEARDOWN);
  }
  __syncwarp();
  __syncthreads();
  // neither CTA of a pair frees its tensor memory or leaves while the pair's
  // MMAs or signals may still reach it
  if constexpr (PAIR) ptx::cluster_sync();
  if (warp == 1) {
    __syncwarp();
    if constexpr (PAIR) ptx::tmem_dealloc_pair(tmem_base, L::TMEM_COLS);
    else ptx::tmem_dealloc(tmem_base, L::TMEM_COLS);
  }
}

template <int STAGES, int EW, int H16, int MODE, bool WHOLE>
__global__ void __cluster_dims__(2, 1, 1)
    __launch_bounds__(GluLayout<1, 256, STAGES, EW, 128, MODE>::THREADS, 1)
    glu_pair_kernel(const __grid_constant__ GluMaps maps, const __grid_constant__ GluParams p) {
  glu_body<1, 256, STAGES, EW, 128, H16, MODE, WHOLE>(maps, p);
}

template <int STAGES, int EW, int H16, int MODE, bool WHOLE>
mlp_status launch_glu_pair(const GluMaps& maps, const GluParams& p, cudaStream_t st) {
  using L = GluLayout<1, 256, STAGES, EW, 128, MODE>;
  auto kernel = glu_pair_kernel<STAGES, EW, H16, MODE, WHOLE>;
  static PerDevice resident;
  const int max_pairs = resident_pairs(resident, kernel, L::THREADS, L::SMEM);
  if (max_pairs < 1) return MLP_ERR_CUDA;
  const int pairs = p.units < max_pairs ? p.units : max_pairs;
  LaunchScope ls(glu_is_bwd(MODE) ? "glu_bwd_pair" : "glu_fwd_pair", st, p.a.T, p.a.N, p.a.K);
  launch_k(kernel, dim3(2 * pairs), dim3(L::THREADS), L::SMEM, st, maps, p);
  return launch_status();
}

}  // namespace

}  // namespace mlp
