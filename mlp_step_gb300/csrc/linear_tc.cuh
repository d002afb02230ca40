// The kernel body of the 16-bit linear layers (k_linear.cu tells its shape),
// its parameters, and the launch of CTA pairs.
#pragma once

#include "act.cuh"
#include "ckpt8.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "tile_epilogue.cuh"
#include "trace.cuh"

namespace mlp {

struct LinParams {
  LinearArgs a;
  int tiles_m, tiles_n, units, k_blocks, kb_per_split;
  unsigned magic;  // of tile_of
  int a_bytes;  // of a stage's x tile: fewer than 128 rows when there are fewer
  int y64;  // y / du in boxes of 64 columns (16-bit, no u_out), else of 32
  // What moves by TMA: y / du; u_out; the 16-bit residual / u (into the y64 box,
  // where the output replaces it); the 8-bit values
  int tma_y, tma_u, tma_in, tma_q;
  unsigned long long wait_ns;
  int* err;
};

// Tensor maps of a launch: operands, outputs, the epilogue's input, 8-bit values.
struct LinMaps {
  CUtensorMap a, b, y, u, in, q;
};

namespace {

constexpr int BK = 64;
// Staging bytes of an epilogue warp: 32 rows x 128 bytes for y / du (or two
// boxes of 32 rows x 64 bytes, for y / du and u / a), then 32 rows x 64 bytes
// of 8-bit values.  Everything that the epilogue reads and writes beside the
// accumulator passes through these boxes, so its arithmetic has one form; rows
// that TMA cannot address, and ragged columns, are moved between box and
// matrix by the warp's own copies.
constexpr int kBox = 4096, kWarpStage = kBox + 2048;

// EW: epilogue warps.  AROWS: rows of x that a stage holds; with fewer than 128
// the MMA reads on into what follows, which only feeds accumulator rows that
// are never stored.
template <int PAIR, int BN, int STAGES, int EW, int AROWS = 128>
struct LinLayout {
  static constexpr int A_BYTES = AROWS * BK * 2;
  static constexpr int B_COLS = PAIR ? 128 : BN;  // operand columns staged per CTA
  static constexpr int B_BYTES = B_COLS * BK * 2;
  static constexpr int ACC = PAIR ? 256 : BN;     // accumulator columns per CTA
  static constexpr int SPAN = ACC / (EW / 4);     // columns of an epilogue warp
  static constexpr int THREADS = 64 + 32 * EW;    // + producer, MMA issuer
  static constexpr int BAR_BYTES = 1024;
  static constexpr int SMEM =
      1024 + STAGES * (A_BYTES + B_BYTES) + EW * kWarpStage + BAR_BYTES;
  static constexpr uint32_t TMEM_COLS = 2 * ACC;
  static_assert(SPAN % 64 == 0, "an epilogue unit is 64 columns");
  static_assert(SMEM <= 232448, "shared memory");
};

// ------------------------------------------------------------ the kernel

// MODE: forward, backward from 16-bit (or no) pre-activations, backward from
// 8-bit ones.
enum { kFwd, kBwd, kBwdCkpt };

// FORM: what the launch promises of its pieces, so that the epilogue's scalar
// work (half of its instructions otherwise) is decided when it is compiled.
//   kAny      nothing
//   kWhole64  whole 64-column units, 16-bit y / du in 64-column boxes, all of
//             the epilogue's matrices moved by TMA
//   kWhole32  the same with u_out: both outputs in 32-column boxes (and no
//             16-bit input, which would need a third)
enum { kAny, kWhole64, kWhole32 };

template <int PAIR, int BN, int STAGES, int EW, int AROWS, int H16, int MODE, int FORM>
__device__ __forceinline__ void linear_body(const LinMaps& maps, const LinParams& p) {
  using L = LinLayout<PAIR, BN, STAGES, EW, AROWS>;
  static_assert(AROWS == 128 || (STAGES * L::B_BYTES >= 16384 && !PAIR), "reads past the x ring");
  constexpr int ACC = L::ACC;
  constexpr int TILE_M = PAIR ? 256 : 128, TILE_N = ACC;
  constexpr bool BWD = MODE != kFwd, CK = MODE == kBwdCkpt;
  constexpr bool B_MN = !BWD;  // W [K][N] is an N-major operand, W [N][K] a K-major one
  constexpr bool WHOLE = FORM != kAny;
  static_assert(!WHOLE || PAIR, "whole pieces only in pairs");
  const LinearArgs& a = p.a;
  const int splits = WHOLE ? 1 : a.splits;
  const bool out_f32 = !WHOLE && a.out_f32;
  const bool y64 = FORM == kAny ? p.y64 : FORM == kWhole64;
  const bool u_out = FORM == kAny ? a.u_out != nullptr : FORM == kWhole32;
  const bool tma_y = WHOLE || p.tma_y, tma_u = WHOLE || p.tma_u, tma_q = WHOLE || p.tma_q;
  const bool tma_in = FORM != kWhole32 && !CK && p.tma_in;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + STAGES * L::A_BYTES;
  uint8_t* stg = sB + STAGES * L::B_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(stg + EW * kWarpStage);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  uint64_t* in_full = done + 1;  // per epilogue warp: its input box has landed
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
    ptx::prefetch_tensormap(&maps.a);
    ptx::prefetch_tensormap(&maps.b);
    if (p.tma_y) ptx::prefetch_tensormap(&maps.y);
    if (p.tma_u) ptx::prefetch_tensormap(&maps.u);
    if (p.tma_in) ptx::prefetch_tensormap(&maps.in);
    if (p.tma_q) ptx::prefetch_tensormap(&maps.q);
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
        const int n0 = tn * TILE_N + (int)rank * L::B_COLS;
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
          const int k0 = kb * BK;
          if constexpr (PAIR) {
            if (rank == 0) {
              ptx::mbar_arrive_expect_tx(&full[stage], 2 * (L::A_BYTES + L::B_BYTES));
              last_parity[stage] = (int)phase;
            }
            const uint32_t bar = full0 + (uint32_t)stage * 8u;
            ptx::tma_load_2d_pair(da, &maps.a, bar, k0, m0);
            if constexpr (B_MN) {
              ptx::tma_load_2d_pair(db, &maps.b, bar, n0, k0);
              ptx::tma_load_2d_pair(db + 8192, &maps.b, bar, n0 + 64, k0);
            } else {
              ptx::tma_load_2d_pair(db, &maps.b, bar, k0, n0);
            }
          } else {
            // 64-wide boxes entirely past N are not loaded: they only feed
            // accumulator columns that are never stored
            uint32_t bytes = p.a_bytes + L::B_BYTES;
            if constexpr (B_MN) {
#pragma unroll
              for (int j = 1; j < BN / 64; ++j)
                if (n0 + 64 * j >= a.N) bytes -= 8192u;
            }
            ptx::mbar_arrive_expect_tx(&full[stage], bytes);
            last_parity[stage] = (int)phase;
            ptx::tma_load_2d(da, &maps.a, &full[stage], k0, m0);
            if constexpr (B_MN) {
#pragma unroll
              for (int j = 0; j < BN / 64; ++j)
                if (j == 0 || n0 + 64 * j < a.N)
                  ptx::tma_load_2d(db + 8192 * j, &maps.b, &full[stage], n0 + 64 * j, k0);
            } else {
              ptx::tma_load_2d(db, &maps.b, &full[stage], k0, n0);
            }
          }
          if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = ptx::idesc_16_f32<H16>(TILE_M, TILE_N, 0, B_MN ? 1 : 0);
      constexpr uint32_t b_lbo = B_MN ? 8192u : 16u, b_kstep = B_MN ? 2048u : 32u;
      // Descriptors of stage 0; the address field (16-byte units, low bits)
      // advances by plain addition.  The issuing warp shares its scheduler
      // with four epilogue warps, so every instruction here costs several
      // issue slots of waiting.
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
          for (int k = 0; k < BK / 16; ++k) {
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
    const int c_first = (ew >> 2) * L::SPAN;
    const uint32_t tempty0 = PAIR ? ptx::mapa_shared(ptx::smem_u32(tempty), 0) : 0u;
    uint8_t* box = stg + ew * kWarpStage;
    uint8_t* qbox = box + kBox;
    bool stores = false;      // a store of this warp may still read its boxes
    bool in_flight = false;   // an input box is on its way
    uint32_t in_phase = 0;
    uint32_t sb[2] = {0, 0};  // backward: the scale bytes of this row's two groups

    // One unit is 64 columns of the warp's 32 rows; units go tile by tile.
    struct Unit {
      int row0, n0;
    };
    auto locate = [&](int u, int c) {
      Unit t{0, a.N};
      if (u < p.units) {
        int tm, tn;
        tile_of(p, splits == 1 ? u : u / splits, tm, tn);
        t.row0 = tm * TILE_M + (int)rank * 128 + quarter * 32;
        t.n0 = tn * TILE_N + c_first + c;
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
    // Requests what the epilogue of a unit reads by TMA.
    auto request = [&](const Unit& t) {
      if (!exists(t)) return;
      if constexpr (CK) {
        const long long m = (long long)t.row0 + lane;
        if (m < a.T) {
#pragma unroll
          for (int g = 0; g < 2; ++g)
            sb[g] = WHOLE || t.n0 + 32 * g < a.N ? a.scale[m * a.lds + t.n0 / kCkptGroup + g] : 0u;
        }
        if (tma_q) {
          __syncwarp();  // every lane has read the box
          if (lane == 0) {
            ptx::mbar_arrive_expect_tx(&in_full[ew], 2048);
            ptx::tma_load_2d(qbox, &maps.q, &in_full[ew], t.n0, t.row0);
          }
          in_flight = true;
        }
      }
      if (tma_in) {
        // A unit that left by the warp's own copy wrote the box with ordinary
        // stores; each lane orders its own before the copy's writes.  (Whole
        // pieces always leave by TMA, behind the fence before that store.)
        if (!WHOLE) ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(&in_full[ew], kBox);
          ptx::tma_load_2d(box, &maps.in, &in_full[ew], t.n0, t.row0);
        }
        in_flight = true;
      }
    };
    // The accumulator goes back to the MMA issuer as soon as the warp's last
    // piece of it is in registers.  Relaxed: nothing in memory is handed over
    // (the tensor-memory reads have completed), and a release at cluster scope
    // would wait for all of the warp's global accesses.
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

    Unit next = locate(worker, 0);
    if (CK && splits == 1) request(next);
    for (int u = worker; u < p.units; u += workers) {
      if (*s_abort) break;
      bool ready = false;
      for (int c = 0; c < L::SPAN; c += 64) {
        const Unit t = next;
        const bool last_unit = c + 64 >= L::SPAN;
        next = last_unit ? locate(u + workers, 0) : locate(u, c + 64);
        const long long m = (long long)t.row0 + lane;
        const bool row_ok = m < a.T;
        // the 8-bit input is requested a unit ahead; one that lands in the
        // output's box once that has been read by its store
        if (tma_in) {
          boxes_free();
          request(t);
        }
        if (!ready) {
          ready = PAIR ? ptx::mbar_wait_cluster_bounded(&tfull[acc], acc_phase, p.wait_ns, p.err,
                                                        DEVERR_TIMEOUT_EPILOGUE)
                       : ptx::mbar_wait_bounded(&tfull[acc], acc_phase, p.wait_ns, p.err,
                                                DEVERR_TIMEOUT_EPILOGUE);
          if (!ready) break;
          ptx::tc_fence_after();
        }
        const bool real = exists(t);  // warp-uniform
        if (real && splits == 1) {
          if (!tma_in) boxes_free();
          if (in_flight) {
            if (!ptx::mbar_wait_bounded(&in_full[ew], in_phase, p.wait_ns, p.err,
                                        DEVERR_TIMEOUT_EPILOGUE)) {
              ready = false;
              break;
            }
            in_phase ^= 1;
            in_flight = false;
          }
        }
        // Ragged units do not leave by TMA: the bulk stores write whole 16-byte
        // units, so they would touch columns past N.
        const bool whole = WHOLE || t.n0 + 64 <= a.N;
        const int rows = (int)min(32ll, a.T - t.row0);
        const int esz = out_f32 ? 4 : 2;
        const int y_bytes = y64 || out_f32 ? 128 : 64;  // of a box row
        // the 16-bit input: residual (forward) or u (backward)
        const uint8_t* in16 = reinterpret_cast<const uint8_t*>(
            CK || FORM == kWhole32 ? nullptr : BWD ? a.u_in : out_f32 ? nullptr : a.res);
        const long long ld_in = (BWD ? a.ldu_in : a.ldr) * 2;
        if (real && splits == 1) {
          const int cols = min(64, a.N - t.n0);
          if (!WHOLE && in16 && y64 && !tma_in)
            warp_copy<false>(box, 128,
                             const_cast<uint8_t*>(in16) + t.row0 * ld_in + (long long)t.n0 * 2,
                             ld_in, rows, cols * 2, 2, lane);
          if (CK && !tma_q)
            warp_copy<false>(qbox, 64, reinterpret_cast<uint8_t*>(a.q) + t.row0 * a.ldq + t.n0,
                             a.ldq, rows, cols, 1, lane);
        }
#pragma unroll(BWD && FORM == kWhole64 ? 2 : 1)
        for (int h = 0; h < 2; ++h) {
          const int n0 = t.n0 + 32 * h;
          const int cols = WHOLE ? 32 : min(32, a.N - n0);
          const bool last = last_unit && h == 1;
          if (!real || cols <= 0) {  // warp-uniform
            if (last) release();
            continue;
          }
          const bool end = h == 1 || (!WHOLE && a.N - n0 <= 32);  // the unit's last piece
          F2 v[16];
          {
            float4 b4[8];
            if constexpr (!BWD) {
              if (a.bias && cols == 32 && splits == 1) {
#pragma unroll
                for (int k = 0; k < 8; ++k) b4[k] = load_bias4(a.bias + n0 + 4 * k);
              } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) b4[k] = make_float4(0.f, 0.f, 0.f, 0.f);
              }
            }
            uint32_t r[32];
            __syncwarp();
            ptx::tmem_ld_32x32b_x32(tmem_base + ((uint32_t)(quarter * 32) << 16) +
                                        (uint32_t)(acc * ACC + c_first + c + 32 * h),
                                    r);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j)
              v[j] = f2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
            if (last) release();
            if constexpr (!BWD) {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                v[2 * k] = add2(v[2 * k], f2(b4[k].x, b4[k].y));
                v[2 * k + 1] = add2(v[2 * k + 1], f2(b4[k].z, b4[k].w));
              }
              if (cols < 32 && splits == 1) {
                // columns past N: zero, so that they take no part in the
                // 8-bit group's scale
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                  const bool e = 2 * j < cols, o = 2 * j + 1 < cols;
                  v[j].x = e ? v[j].x + (a.bias ? __ldg(a.bias + n0 + 2 * j) : 0.f) : 0.f;
                  v[j].y = o ? v[j].y + (a.bias ? __ldg(a.bias + n0 + 2 * j + 1) : 0.f) : 0.f;
                }
              }
            }
          }
          if (splits > 1) {
            // raw sums: planes have whole 32-column pieces (ldp a multiple of 32)
            if (row_ok) {
              float* pr = a.partial + ((long long)(u % splits) * a.T + m) * a.ldp + n0;
#pragma unroll
              for (int k = 0; k < 8; ++k)
                reinterpret_cast<float4*>(pr)[k] =
                    make_float4(v[2 * k].x, v[2 * k].y, v[2 * k + 1].x, v[2 * k + 1].y);
            }
            continue;
          }
          if (h == 1 && !y64) boxes_free();
          // u / a leaves through the second box; beside an fp32 output, whose
          // box is the whole space, at once and through the same space
          uint8_t* u_box = out_f32 ? box : box + kBox / 2;
          auto copy_u = [&] {
            if (!(tma_u && whole))
              warp_copy<true>(u_box, 64,
                              static_cast<uint8_t*>(a.u_out) +
                                  ((long long)t.row0 * a.ldu_out + n0) * 2,
                              a.ldu_out * 2, rows, cols * 2, 2, lane);
          };
          // the 16-bit input's piece into the box, where the unit did not bring it
          auto stage16 = [&] {
            if (!y64)
              warp_copy<false>(box, 64,
                               const_cast<uint8_t*>(in16) + t.row0 * ld_in + (long long)n0 * 2,
                               ld_in, rows, cols * 2, 2, lane);
          };

          if constexpr (!BWD) {
            if (a.q) {
              uint32_t w[8];
              const uint32_t b = ckpt8_group(reinterpret_cast<const float(&)[32]>(v), w);
              if (row_ok) a.scale[m * a.lds + n0 / kCkptGroup] = (uint8_t)b;
              *reinterpret_cast<uint4*>(chunk_at(qbox, 64, lane, 2 * h)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
              *reinterpret_cast<uint4*>(chunk_at(qbox, 64, lane, 2 * h + 1)) =
                  make_uint4(w[4], w[5], w[6], w[7]);
            }
            if (u_out) {
              pack_row<H16>(u_box, 64, lane, 0, v);
              copy_u();
            }
            with_act(a.act, [&](auto tag) {
#pragma unroll
              for (int j = 0; j < 16; ++j)
                v[j] = act_value2<decltype(tag)::value>(v[j], a.slope);
            });
            if (in16) {
              stage16();
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint4 q = *reinterpret_cast<const uint4*>(
                    chunk_at(box, y64 ? 128 : 64, lane, (y64 ? 4 * h : 0) + k));
                v[4 * k] = add2(v[4 * k], unpack2<H16>(q.x));
                v[4 * k + 1] = add2(v[4 * k + 1], unpack2<H16>(q.y));
                v[4 * k + 2] = add2(v[4 * k + 2], unpack2<H16>(q.z));
                v[4 * k + 3] = add2(v[4 * k + 3], unpack2<H16>(q.w));
              }
              __syncwarp();
            } else if (!WHOLE && a.res) {
              warp_copy<false>(box, 128,
                               static_cast<uint8_t*>(const_cast<void*>(a.res)) +
                                   ((long long)t.row0 * a.ldr + n0) * 4,
                               a.ldr * 4, rows, cols * 4, 4, lane);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float4 f =
                    *reinterpret_cast<const float4*>(chunk_at(box, 128, lane, k));
                v[2 * k] = add2(v[2 * k], f2(f.x, f.y));
                v[2 * k + 1] = add2(v[2 * k + 1], f2(f.z, f.w));
              }
            }
          } else {
            // the saved values of this piece, raw (decoded half a piece at a
            // time below, which keeps the registers within the launch's limit)
            uint32_t raw[CK ? 8 : 16];
            auto take = [&](int k, const uint4& q) {
              raw[4 * k] = q.x;
              raw[4 * k + 1] = q.y;
              raw[4 * k + 2] = q.z;
              raw[4 * k + 3] = q.w;
            };
            float step = 0.f;
            if constexpr (CK) {
              step = ckpt8_step(h ? sb[1] : sb[0]);
#pragma unroll
              for (int k = 0; k < 2; ++k)
                take(k, *reinterpret_cast<const uint4*>(chunk_at(qbox, 64, lane, 2 * h + k)));
              // this unit's values are in registers: bring the next unit's
              if (end) request(next);
            } else if (in16) {
              stage16();
#pragma unroll
              for (int k = 0; k < 4; ++k)
                take(k, *reinterpret_cast<const uint4*>(
                            chunk_at(box, y64 ? 128 : 64, lane, (y64 ? 4 * h : 0) + k)));
              __syncwarp();
            } else {
#pragma unroll
              for (int k = 0; k < 16; ++k) raw[k] = 0u;
            }
            // v <- v f'(u), f(u) into its box
            with_act(a.act, [&](auto tag) {
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                F2 x[8];
                if constexpr (CK) {
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const uint32_t f = ckpt8_flip(raw[4 * g + e]);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                      x[2 * e + j] = mul2(
                          add2(f2(ckpt8_biased(f, 2 * j), ckpt8_biased(f, 2 * j + 1)),
                               f2(-kCkptBias)),
                          f2(step));
                  }
                } else {
#pragma unroll
                  for (int j = 0; j < 8; ++j) x[j] = unpack2<H16>(raw[8 * g + j]);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  F2 f;
                  v[8 * g + j] = mul2(v[8 * g + j],
                                      act_grad2<decltype(tag)::value>(x[j], a.slope, f));
                  x[j] = f;
                }
                if (u_out) pack_row<H16>(u_box, 64, lane, 2 * g, x);
              }
            });
            if (u_out) copy_u();
          }

          // the output into its box, and out
          if (out_f32) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<float4*>(chunk_at(box, 128, lane, k)) =
                  make_float4(v[2 * k].x, v[2 * k].y, v[2 * k + 1].x, v[2 * k + 1].y);
          } else {
            pack_row<H16>(box, y_bytes, lane, y64 ? 4 * h : 0, v);
          }
          const bool flush_y = end || !y64, flush_q = !BWD && a.q && end;
          const bool by_tma_y = flush_y && tma_y && whole;
          const bool by_tma_q = flush_q && tma_q && whole;
          const bool by_tma_u = u_out && tma_u && whole;
          if (by_tma_y || by_tma_q || by_tma_u) {
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              // rows past T are clipped by the stores
              if (by_tma_y) ptx::tma_store_2d(&maps.y, box, y64 ? t.n0 : n0, t.row0);
              if (by_tma_u) ptx::tma_store_2d(&maps.u, box + kBox / 2, n0, t.row0);
              if (by_tma_q) ptx::tma_store_2d(&maps.q, qbox, t.n0, t.row0);
              ptx::bulk_commit_group();
            }
            stores = true;
          }
          if (flush_y && !by_tma_y)
            warp_copy<true>(box, y_bytes,
                            static_cast<uint8_t*>(a.y) +
                                ((long long)t.row0 * a.ldy + (y64 ? t.n0 : n0)) * esz,
                            a.ldy * esz, rows, (y64 ? min(64, a.N - t.n0) : cols) * esz, esz,
                            lane);
          if (flush_q && !by_tma_q)
            warp_copy<true>(qbox, 64, reinterpret_cast<uint8_t*>(a.q) + t.row0 * a.ldq + t.n0,
                            a.ldq, rows, min(64, a.N - t.n0), 1, lane);
          if constexpr (BWD) {
            if (a.colpart) {
              if (!row_ok) {
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = f2(0.f);
              }
              const float s1 = column_sums(v, lane);
              if (lane < cols)
                a.colpart[(long long)(t.row0 / 32) * a.ldcp + n0 + lane] = s1;
            }
          }
        }
        // (a unit that does not exist in this tile has none to wait for, but
        // the next one may)
        if (CK && !real && splits == 1) request(next);
      }
      if (!ready) {
        *s_abort = 1;
        break;
      }
      if (++acc == 2) { acc = 0; acc_phase ^= 1; }
    }
    // an input box requested for a unit that an abort skipped
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

template <int STAGES, int EW, int H16, int MODE, int FORM>
__global__ void __cluster_dims__(2, 1, 1)
    __launch_bounds__(LinLayout<1, 256, STAGES, EW>::THREADS, 1)
    linear_pair_kernel(const __grid_constant__ LinMaps maps, const __grid_constant__ LinParams p) {
  linear_body<1, 256, STAGES, EW, 128, H16, MODE, FORM>(maps, p);
}

template <int STAGES, int EW, int H16, int MODE, int FORM>
mlp_status launch_pair(const LinMaps& maps, const LinParams& p, cudaStream_t st) {
  using L = LinLayout<1, 256, STAGES, EW>;
  auto kernel = linear_pair_kernel<STAGES, EW, H16, MODE, FORM>;
  static PerDevice resident;
  const int max_pairs = resident_pairs(resident, kernel, L::THREADS, L::SMEM);
  if (max_pairs < 1) return MLP_ERR_CUDA;
  const int pairs = p.units < max_pairs ? p.units : max_pairs;
  LaunchScope ls(MODE != kFwd ? "linear_bwd_pair" : "linear_fwd_pair", st, p.a.T, p.a.N, p.a.K);
  launch_k(kernel, dim3(2 * pairs), dim3(L::THREADS), L::SMEM, st, maps, p);
  return launch_status();
}

// Pairs: for short K the epilogue is as long as the product, so it gets
// sixteen warps and the operand ring four stages (65,536 x 512 -> 1,536, no
// activation: 64 us of MMAs and loads with four stages, 63 with five); for
// long K eight warps leave room for a fifth stage.  Sixteen and eight warps,
// 65,536 rows -> 1,536, GELU with 8-bit pre-activations: K = 512 101 and 126 us,
// 768 137 and 138, 1,024 175 and 163, 1,536 234 and 222; the backward with column
// sums 137 and 163, 151 and 179, 178 and 179, 235 and 241; without an activation
// eight are ahead from 512 (79 and 70) to 1,536 (187 and 178).
constexpr int kShortK = 16;  // k-blocks

// The pairs of either operand ring.
template <int H16, int MODE, int FORM>
mlp_status launch_pairs(const LinMaps& maps, const LinParams& p, cudaStream_t st) {
  return p.k_blocks <= kShortK ? launch_pair<4, 16, H16, MODE, FORM>(maps, p, st)
                               : launch_pair<5, 8, H16, MODE, FORM>(maps, p, st);
}

}  // namespace

// Pairs of whole pieces (k_linear_whole.cu): mode and form as above.
mlp_status launch_linear_whole(const LinMaps& maps, const LinParams& p, int mode, int form,
                               cudaStream_t st);

}  // namespace mlp
