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
// of them to fill the GPU, single CTAs on 128 x 128 or 128 x 64 tiles
// otherwise, with the contraction split over CTAs when even those are few
// (raw sums to a workspace, finished by launch_linear_finish).  Warps: TMA
// producer, MMA issuer, eight or sixteen epilogue warps (a tensor-memory lane
// quarter and a share of the columns each); two accumulators, so that the
// epilogue of one tile overlaps the MMAs of the next.  W is read as it is stored: [K][N] as an
// N-major operand, [N][K] (backward) as a K-major one.
//
// Bound: the MMAs for long K; for K of a few hundred, the epilogue's
// instruction issue (an activation is 10 to 20 instructions per output).
#include <cstring>

#include "act.cuh"
#include "ckpt8.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "trace.cuh"

namespace mlp {

namespace {

constexpr int BK = 64;
constexpr int kStage = 4096;  // output staging bytes per epilogue warp

struct LinParams {
  LinearArgs a;
  int tiles_m, tiles_n, units, k_blocks, kb_per_split;
  int tma_y, tma_u;  // y / du and u_out leave through their tensor maps
  unsigned long long wait_ns;
  int* err;
};

template <int PAIR, int BN, int STAGES>
struct LinLayout {
  static constexpr int A_BYTES = 128 * BK * 2;
  static constexpr int B_COLS = PAIR ? 128 : BN;  // operand columns staged per CTA
  static constexpr int B_BYTES = B_COLS * BK * 2;
  static constexpr int ACC = PAIR ? 256 : BN;     // accumulator columns per CTA
  // Epilogue warps: four per scheduler, where the tile has 32 columns for
  // each; with two per scheduler the epilogue's latencies (tensor-memory
  // loads, the proxy fence before each store) left half of the issue slots
  // empty.
  static constexpr int EPI_WARPS = ACC >= 128 ? 16 : 8;
  static constexpr int THREADS = 64 + 32 * EPI_WARPS;  // + producer, MMA issuer
  static constexpr int BAR_BYTES = 1024;
  static constexpr int SMEM =
      1024 + STAGES * (A_BYTES + B_BYTES) + BAR_BYTES + EPI_WARPS * kStage;
  static constexpr uint32_t TMEM_COLS = 2 * ACC;
  static_assert(SMEM <= 232448, "shared memory");
};

// Eight tile rows at a time sweep all tile columns, so that CTAs that run
// together share row and column blocks in L2.
__device__ __forceinline__ void tile_of(int t, int tiles_m, int tiles_n, int& tm, int& tn) {
  constexpr int G = 8;
  const int first = t / (G * tiles_n) * G;
  const int gm = min(tiles_m - first, G);
  const int r = t - first * tiles_n;
  tm = first + r % gm;
  tn = r / gm;
}

// ------------------------------------------------------------ epilogue pieces

template <int H16>
__device__ __forceinline__ F2 unpack2(uint32_t w) {
  if constexpr (H16) {
    const float2 f = __half22float2(*reinterpret_cast<__half2*>(&w));
    return f2(f.x, f.y);
  } else {
    return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
}

// 32 consecutive values of a row as they lie in memory: 64 bytes of a 16-bit
// type, or 32 int8 and a scale byte.
struct Saved {
  uint4 q[4];
  uint32_t b;
};

__device__ __forceinline__ void load_row16(const void* base, long long ld, long long m, int n0,
                                           int N, Saved& s) {
  const uint16_t* p = static_cast<const uint16_t*>(base) + m * ld + n0;
  if (n0 + 32 <= N && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
#pragma unroll
    for (int k = 0; k < 4; ++k) s.q[k] = *(reinterpret_cast<const uint4*>(p) + k);
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(s.q);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const uint32_t lo = n0 + 2 * k < N ? p[2 * k] : 0u;
      const uint32_t hi = n0 + 2 * k + 1 < N ? p[2 * k + 1] : 0u;
      w[k] = lo | hi << 16;
    }
  }
}

__device__ __forceinline__ void load_row8(const LinearArgs& a, long long m, int n0, Saved& s) {
  const int8_t* p = a.q + m * a.ldq + n0;
  s.b = a.scale[m * a.lds + n0 / kCkptGroup];
  if (n0 + 32 <= a.N && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    s.q[0] = *reinterpret_cast<const uint4*>(p);
    s.q[1] = *(reinterpret_cast<const uint4*>(p) + 1);
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(s.q);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      w[k] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n0 + 4 * k + e < a.N) w[k] |= (uint32_t)(uint8_t)p[4 * k + e] << (8 * e);
    }
  }
}

// Where a piece's 32 values of one output go: a row of a staging box that a
// TMA store then moves (32 rows x 32 columns; 16-bit boxes in the 64-byte
// swizzle their tensor map names, fp32 ones in the 128-byte swizzle), or the
// matrix itself, for ragged pieces, unaligned rows and small outputs.
struct Sink {
  uint8_t* box;  // this lane's row of the box, or nullptr
  uint8_t* mem;  // this lane's row of the matrix at the piece's first column
  int f32, lane, n;  // n: columns that exist (0: a row past the end)
};

template <int H16>
__device__ __forceinline__ void sink8(const Sink& s, int k, const F2 (&v)[4]) {
  if (s.f32) {
    const float4 lo = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    const float4 hi = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
    if (s.box) {
      *reinterpret_cast<float4*>(s.box + (((2 * k) ^ (s.lane & 7)) << 4)) = lo;
      *reinterpret_cast<float4*>(s.box + (((2 * k + 1) ^ (s.lane & 7)) << 4)) = hi;
    } else {
      float* p = reinterpret_cast<float*>(s.mem) + 8 * k;
      if (8 * k + 8 <= s.n && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        reinterpret_cast<float4*>(p)[0] = lo;
        reinterpret_cast<float4*>(p)[1] = hi;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (8 * k + j < s.n) p[j] = j & 1 ? v[j / 2].y : v[j / 2].x;
      }
    }
    return;
  }
  const uint4 o = make_uint4(pack16x2<H16>(v[0].x, v[0].y), pack16x2<H16>(v[1].x, v[1].y),
                             pack16x2<H16>(v[2].x, v[2].y), pack16x2<H16>(v[3].x, v[3].y));
  if (s.box) {
    *reinterpret_cast<uint4*>(s.box + ((k ^ ((s.lane >> 1) & 3)) << 4)) = o;
  } else {
    uint16_t* p = reinterpret_cast<uint16_t*>(s.mem) + 8 * k;
    if (8 * k + 8 <= s.n && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
      *reinterpret_cast<uint4*>(p) = o;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (8 * k + j < s.n) p[j] = f32_to_16<H16>(j & 1 ? v[j / 2].y : v[j / 2].x);
    }
  }
}

// Column sums of a warp's 32 x 32 piece (row = lane): each round a lane hands
// half of its columns to its partner and adds the partner's half of its own,
// so after five rounds lane j holds the sum of column j.  31 exchanges for 32
// columns, in a fixed order.
__device__ __forceinline__ float column_sums(F2 (&p)[16], int lane) {
  float* v = reinterpret_cast<float*>(p);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool upper = lane & o;
#pragma unroll
    for (int j = 0; j < o; ++j) {
      const float give = upper ? v[j] : v[j + o];
      const float keep = upper ? v[j + o] : v[j];
      v[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  return v[0];
}

// ------------------------------------------------------------ the kernel

template <int PAIR, int BN, int STAGES, int H16, int BWD>
__device__ __forceinline__ void linear_body(const CUtensorMap& tmA, const CUtensorMap& tmB,
                                            const CUtensorMap& tmY, const CUtensorMap& tmU,
                                            const LinParams& p) {
  using L = LinLayout<PAIR, BN, STAGES>;
  constexpr int ACC = L::ACC;
  constexpr int TILE_M = PAIR ? 256 : 128, TILE_N = ACC;
  constexpr bool B_MN = !BWD;  // W [K][N] is an N-major operand, W [N][K] a K-major one
  const LinearArgs& a = p.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + STAGES * L::A_BYTES;
  uint8_t* stg = sB + STAGES * L::B_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(stg + L::EPI_WARPS * kStage);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? ptx::cluster_ctarank() : 0u;
  const int worker = PAIR ? blockIdx.x >> 1 : blockIdx.x;
  const int workers = PAIR ? gridDim.x >> 1 : gridDim.x;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 1);
    }
    for (int k = 0; k < 2; ++k) {
      ptx::mbar_init(&tfull[k], 1);
      ptx::mbar_init(&tempty[k], PAIR ? 2 * L::EPI_WARPS : L::EPI_WARPS);
    }
    ptx::mbar_init(done, 1);
    *s_abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&tmA);
    ptx::prefetch_tensormap(&tmB);
    if (p.tma_y) ptx::prefetch_tensormap(&tmY);
    if (p.tma_u) ptx::prefetch_tensormap(&tmU);
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
    kb0 = u % a.splits * p.kb_per_split;
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
        tile_of(u / a.splits, p.tiles_m, p.tiles_n, tm, tn);
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
            ptx::tma_load_2d_pair(da, &tmA, bar, k0, m0);
            if constexpr (B_MN) {
              ptx::tma_load_2d_pair(db, &tmB, bar, n0, k0);
              ptx::tma_load_2d_pair(db + 8192, &tmB, bar, n0 + 64, k0);
            } else {
              ptx::tma_load_2d_pair(db, &tmB, bar, k0, n0);
            }
          } else {
            // 64-wide boxes entirely past N are not loaded: they only feed
            // accumulator columns that are never stored
            uint32_t bytes = L::A_BYTES + L::B_BYTES;
            if constexpr (B_MN) {
#pragma unroll
              for (int j = 1; j < BN / 64; ++j)
                if (n0 + 64 * j >= a.N) bytes -= 8192u;
            }
            ptx::mbar_arrive_expect_tx(&full[stage], bytes);
            last_parity[stage] = (int)phase;
            ptx::tma_load_2d(da, &tmA, &full[stage], k0, m0);
            if constexpr (B_MN) {
#pragma unroll
              for (int j = 0; j < BN / 64; ++j)
                if (j == 0 || n0 + 64 * j < a.N)
                  ptx::tma_load_2d(db + 8192 * j, &tmB, &full[stage], n0 + 64 * j, k0);
            } else {
              ptx::tma_load_2d(db, &tmB, &full[stage], k0, n0);
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
          const uint32_t ab = ptx::smem_u32(sA + stage * L::A_BYTES);
          const uint32_t bb = ptx::smem_u32(sB + stage * L::B_BYTES);
#pragma unroll
          for (int k = 0; k < BK / 16; ++k) {
            const uint64_t ad = ptx::sw128_desc(ab + k * 32, 16, 1024);
            const uint64_t bd = ptx::sw128_desc(bb + k * b_kstep, b_lbo, 1024);
            const uint32_t add = kb > kb0 || k > 0;
            if constexpr (PAIR) ptx::mma_bf16_pair(d, ad, bd, idesc, add);
            else ptx::mma_bf16(d, ad, bd, idesc, add);
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
    const int quarter = warp & 3;  // tensor-memory lanes [32 q, 32 q + 32)
    constexpr int SPAN = ACC / (L::EPI_WARPS / 4);  // columns of a warp
    const int c_first = ((warp - 2) >> 2) * SPAN;
    const uint32_t tempty0 = PAIR ? ptx::mapa_shared(ptx::smem_u32(tempty), 0) : 0u;
    // staging: both outputs' boxes (or one fp32 box) fill the warp's 4 KiB,
    // one 16-bit output takes its two halves in turn
    uint8_t* boxes = stg + (warp - 2) * kStage;
    const int turns = a.out_f32 || p.tma_u ? 1 : 2;
    int staged = 0;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int u = worker; u < p.units; u += workers) {
      if (*s_abort) break;
      int tm, tn;
      tile_of(u / a.splits, p.tiles_m, p.tiles_n, tm, tn);
      const int row0 = tm * TILE_M + (int)rank * 128 + quarter * 32;  // this warp's first row
      const long long m = (long long)row0 + lane;
      const bool row_ok = m < a.T;
      const int n_first = tn * TILE_N + c_first;
      const int n_end = min(a.N, n_first + SPAN);
      // what the epilogue reads beside the accumulator: requested before the
      // wait for the accumulator, then as soon as the last piece's is used
      auto fetch = [&](int n0, Saved& s) {
        if (!row_ok || n0 >= n_end || a.splits > 1) return;
        if constexpr (BWD) {
          if (a.q) load_row8(a, m, n0, s);
          else if (a.u_in) load_row16(a.u_in, a.ldu_in, m, n0, a.N, s);
        } else {
          if (a.res && !a.out_f32) load_row16(a.res, a.ldr, m, n0, a.N, s);
        }
      };
      Saved cur;
      cur.b = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) cur.q[k] = make_uint4(0, 0, 0, 0);
      fetch(n_first, cur);
      const bool ready = PAIR ? ptx::mbar_wait_cluster_bounded(&tfull[acc], acc_phase, p.wait_ns,
                                                               p.err, DEVERR_TIMEOUT_EPILOGUE)
                              : ptx::mbar_wait_bounded(&tfull[acc], acc_phase, p.wait_ns, p.err,
                                                       DEVERR_TIMEOUT_EPILOGUE);
      if (!ready) {
        *s_abort = 1;
        break;
      }
      ptx::tc_fence_after();
      // the accumulator goes back to the MMA issuer once this warp's last
      // piece of it is in registers
      auto release = [&] {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (rank == 0) ptx::mbar_arrive(&tempty[acc]);
          else ptx::mbar_arrive_remote(tempty0 + (uint32_t)acc * 8u);
        }
      };
      if (n_first >= a.N) release();
#pragma unroll 1
      for (int n0 = n_first; n0 < n_end; n0 += 32) {  // warp-uniform
        F2 v[16];
        {
          uint32_t r[32];
          __syncwarp();
          ptx::tmem_ld_32x32b_x32(tmem_base + ((uint32_t)(quarter * 32) << 16) +
                                      (uint32_t)(acc * ACC + c_first + n0 - n_first),
                                  r);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            v[j] = f2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
        }
        if (n0 + 32 >= n_end) release();
        if (a.splits > 1) {
          // raw sums: planes have whole 32-column pieces (ldp a multiple of 32)
          if (row_ok) {
            float* pr = a.partial + ((long long)(u % a.splits) * a.T + m) * a.ldp + n0;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              reinterpret_cast<float4*>(pr)[k] =
                  make_float4(v[2 * k].x, v[2 * k].y, v[2 * k + 1].x, v[2 * k + 1].y);
          }
          continue;
        }
        if (row0 >= a.T) continue;  // warp-uniform: no row of this warp exists

        // A ragged last piece leaves from registers: the bulk store writes
        // whole 16-byte units, so it would touch columns past N.
        const int cols = a.N - n0;
        const bool whole = cols >= 32;
        const bool box_y = p.tma_y && whole, box_u = p.tma_u && whole;
        uint8_t* box = boxes + (turns == 2 ? (staged & 1) * 2048 : 0);
        if ((box_y || box_u) && staged >= turns) {
          if (lane == 0) {
            if (turns == 2) ptx::bulk_wait_group_read<1>();
            else ptx::bulk_wait_group_read<0>();
          }
          __syncwarp();
        }
        const int n_ok = row_ok ? cols : 0;
        const Sink to_y{box_y ? box + lane * (a.out_f32 ? 128 : 64) : nullptr,
                        static_cast<uint8_t*>(a.y) + (m * a.ldy + n0) * (a.out_f32 ? 4 : 2),
                        a.out_f32, lane, n_ok};
        uint8_t* ubox = box + (p.tma_y ? 2048 : 0);
        const Sink to_u{box_u ? ubox + lane * 64 : nullptr,
                        static_cast<uint8_t*>(a.u_out) + (m * a.ldu_out + n0) * 2, 0, lane, n_ok};
        const uint32_t* sw = reinterpret_cast<const uint32_t*>(cur.q);

        if constexpr (!BWD) {
          if (a.bias) {
            if (whole) {
              const float4* bp = reinterpret_cast<const float4*>(a.bias + n0);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float4 b4 = __ldg(bp + k);
                v[2 * k] = add2(v[2 * k], f2(b4.x, b4.y));
                v[2 * k + 1] = add2(v[2 * k + 1], f2(b4.z, b4.w));
              }
            } else {
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                if (2 * j < cols) v[j].x += __ldg(a.bias + n0 + 2 * j);
                if (2 * j + 1 < cols) v[j].y += __ldg(a.bias + n0 + 2 * j + 1);
              }
            }
          }
          if (a.q) {
            if (!whole) {  // columns past N take no part in the group's scale
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                if (2 * j >= cols) v[j].x = 0.f;
                if (2 * j + 1 >= cols) v[j].y = 0.f;
              }
            }
            uint32_t w[8];
            const uint32_t b = ckpt8_group(reinterpret_cast<const float(&)[32]>(v), w);
            if (row_ok) {
              int8_t* qp = a.q + m * a.ldq + n0;
              a.scale[m * a.lds + n0 / kCkptGroup] = (uint8_t)b;
              if (whole && (reinterpret_cast<uintptr_t>(qp) & 15) == 0) {
                reinterpret_cast<uint4*>(qp)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                reinterpret_cast<uint4*>(qp)[1] = make_uint4(w[4], w[5], w[6], w[7]);
              } else {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (j < cols) qp[j] = (int8_t)(w[j / 4] >> (8 * (j & 3)));
              }
            }
          }
          if (a.u_out) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              sink8<H16>(to_u, k, reinterpret_cast<const F2(&)[4]>(v[4 * k]));
          }
          with_act(a.act, [&](auto tag) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              v[j] = act_value2<decltype(tag)::value>(v[j], a.slope);
          });
          if (a.res) {
            if (!a.out_f32) {
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] = add2(v[j], unpack2<H16>(sw[j]));
            } else if (row_ok) {
              const float* rp = static_cast<const float*>(a.res) + m * a.ldr + n0;
              if (whole && (reinterpret_cast<uintptr_t>(rp) & 15) == 0) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const float4 f = *(reinterpret_cast<const float4*>(rp) + k);
                  v[2 * k] = add2(v[2 * k], f2(f.x, f.y));
                  v[2 * k + 1] = add2(v[2 * k + 1], f2(f.z, f.w));
                }
              } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                  if (2 * j < cols) v[j].x += rp[2 * j];
                  if (2 * j + 1 < cols) v[j].y += rp[2 * j + 1];
                }
              }
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            sink8<H16>(to_y, k, reinterpret_cast<const F2(&)[4]>(v[4 * k]));
        } else {
          const float step = a.q ? ckpt8_step(cur.b) : 0.f;
          with_act(a.act, [&](auto tag) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              F2 f[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                F2 uv;
                if (a.q) {
                  const uint32_t w = ckpt8_flip(sw[2 * k + j / 2]);
                  uv = mul2(add2(f2(ckpt8_biased(w, 2 * (j & 1)),
                                    ckpt8_biased(w, 2 * (j & 1) + 1)),
                                 f2(-kCkptBias)),
                            f2(step));
                } else {
                  uv = unpack2<H16>(sw[4 * k + j]);
                }
                v[4 * k + j] = mul2(
                    v[4 * k + j], act_grad2<decltype(tag)::value>(uv, a.slope, f[j]));
              }
              if (a.u_out) sink8<H16>(to_u, k, f);
              sink8<H16>(to_y, k, reinterpret_cast<const F2(&)[4]>(v[4 * k]));
            }
          });
        }
        fetch(n0 + 32, cur);
        if (box_y || box_u) {
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            // rows past T are clipped by the stores
            if (box_y) ptx::tma_store_2d(&tmY, box, n0, row0);
            if (box_u) ptx::tma_store_2d(&tmU, ubox, n0, row0);
            ptx::bulk_commit_group();
          }
          ++staged;
        }
        if constexpr (BWD) {
          if (a.colpart) {
            if (!row_ok) {
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] = f2(0.f);
            }
            const float s = column_sums(v, lane);
            if (lane < cols) a.colpart[(long long)(row0 / 32) * a.ldcp + n0 + lane] = s;
          }
        }
      }
      if (++acc == 2) { acc = 0; acc_phase ^= 1; }
    }
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

template <int STAGES, int H16, int BWD>
__global__ void __cluster_dims__(2, 1, 1)
    __launch_bounds__(LinLayout<1, 256, STAGES>::THREADS, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tmA,
                       const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmY,
                       const __grid_constant__ CUtensorMap tmU,
                       const __grid_constant__ LinParams p) {
  linear_body<1, 256, STAGES, H16, BWD>(tmA, tmB, tmY, tmU, p);
}

template <int BN, int STAGES, int H16, int BWD>
__global__ void __launch_bounds__(LinLayout<0, BN, STAGES>::THREADS, 1)
    linear_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmU,
                  const __grid_constant__ LinParams p) {
  linear_body<0, BN, STAGES, H16, BWD>(tmA, tmB, tmY, tmU, p);
}

// ------------------------------------------------------------ plan and launch

enum Tile { kPair, kWide, kNarrow };  // 256 x 256 pairs, 128 x 128, 128 x 64

struct LinPlan {
  Tile tile;
  int splits, kb_per_split;
};

// From the shape alone, so that workspace sizes do not depend on the device.
// Pairs when their tiles fill most of ~76 pairs; otherwise single CTAs, 128
// wide when that gives ~100 tiles, else 64 wide; and when those are fewer than
// half of ~152 SMs and K is long, K is split over CTAs, at least four 64-deep
// blocks each.
LinPlan linear_plan(long long T, int K, int N) {
  LinPlan pl;
  const int kb = (K + BK - 1) / BK;
  const long long pair = ((T + 255) / 256) * ((N + 255) / 256);
  const long long wide = ((T + 127) / 128) * ((N + 127) / 128);
  const long long narrow = ((T + 127) / 128) * ((N + 63) / 64);
  int s = 1;
  if (pair >= 48 && N > 128 && T > 128) {
    pl.tile = kPair;
  } else if (wide >= 100 && N > 64) {
    pl.tile = kWide;
  } else {
    pl.tile = kNarrow;
    if (narrow < 76) {
      s = (int)(152 / narrow);
      if (s > 16) s = 16;
      if (s > kb / 4) s = kb / 4;
      if (s < 1) s = 1;
    }
  }
  const int per = (kb + s - 1) / s;
  pl.splits = (kb + per - 1) / per;
  pl.kb_per_split = per;
  return pl;
}

template <int BN, int STAGES, int H16, int BWD>
mlp_status launch_single(const CUtensorMap (&tm)[4], const LinParams& p, cudaStream_t st) {
  using L = LinLayout<0, BN, STAGES>;
  static const cudaError_t configured =
      cudaFuncSetAttribute(linear_kernel<BN, STAGES, H16, BWD>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
  if (configured != cudaSuccess) return MLP_ERR_CUDA;
  const int grid = p.units < num_sms() ? p.units : num_sms();
  LaunchScope ls(BWD ? "linear_bwd" : "linear_fwd", st, p.a.T, p.a.N, p.a.K);
  launch_k(linear_kernel<BN, STAGES, H16, BWD>, dim3(grid), dim3(L::THREADS), L::SMEM, st, tm[0],
           tm[1], tm[2], tm[3], p);
  return launch_status();
}

template <int STAGES, int H16, int BWD>
mlp_status launch_pair(const CUtensorMap (&tm)[4], const LinParams& p, cudaStream_t st) {
  using L = LinLayout<1, 256, STAGES>;
  auto kernel = linear_pair_kernel<STAGES, H16, BWD>;
  // pairs that fit at once (a GPC with an odd number of free SMs leaves one over)
  static const int max_pairs = [&] {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM) !=
        cudaSuccess)
      return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (num_sms() / 2));
    cfg.blockDim = dim3(L::THREADS);
    cfg.dynamicSmemBytes = L::SMEM;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = num_sms() / 2;
    }
    return n;
  }();
  if (max_pairs < 1) return MLP_ERR_CUDA;
  const int pairs = p.units < max_pairs ? p.units : max_pairs;
  LaunchScope ls(BWD ? "linear_bwd_pair" : "linear_fwd_pair", st, p.a.T, p.a.N, p.a.K);
  launch_k(kernel, dim3(2 * pairs), dim3(L::THREADS), L::SMEM, st, tm[0], tm[1], tm[2], tm[3], p);
  return launch_status();
}

template <int H16, int BWD>
mlp_status launch_tile(const CUtensorMap (&tm)[4], const LinParams& p, Tile tile,
                       cudaStream_t st) {
  switch (tile) {
    case kPair: return launch_pair<5, H16, BWD>(tm, p, st);
    case kWide: return launch_single<128, 5, H16, BWD>(tm, p, st);
    default: return launch_single<64, 6, H16, BWD>(tm, p, st);
  }
}

}  // namespace

int linear_tc_splits(long long T, int K, int N) { return linear_plan(T, K, N).splits; }

mlp_status launch_linear_tc(const LinearArgs& a, bool bwd, cudaStream_t st) {
  const LinPlan pl = linear_plan(a.T, a.K, a.N);
  const int tile_m = pl.tile == kPair ? 256 : 128;
  const int tile_n = pl.tile == kPair ? 256 : pl.tile == kWide ? 128 : 64;
  const long long tm = (a.T + tile_m - 1) / tile_m, tn = (a.N + tile_n - 1) / tile_n;
  if (tm * tn * pl.splits > (1ll << 30)) return MLP_ERR_UNSUPPORTED_SHAPE;
  LinParams p{};
  p.a = a;
  p.a.splits = pl.splits;
  p.tiles_m = (int)tm;
  p.tiles_n = (int)tn;
  p.units = (int)(tm * tn * pl.splits);
  p.k_blocks = (a.K + BK - 1) / BK;
  p.kb_per_split = pl.kb_per_split;
  p.wait_ns = wait_limit_ns();
  p.err = device_error_word();
  if (!p.err) return MLP_ERR_CUDA;

  CUtensorMap maps[4];
  memset(maps, 0, sizeof(maps));
  if (!encode_tmap_bf16_2d(&maps[0], a.x, a.K, a.T, (unsigned long long)a.ldx * 2, BK, 128))
    return MLP_ERR_CUDA;
  const bool okb = bwd ? encode_tmap_bf16_2d(&maps[1], a.w, a.K, a.N, (unsigned long long)a.ldw * 2,
                                             BK, pl.tile == kNarrow ? 64 : 128)
                       : encode_tmap_bf16_2d(&maps[1], a.w, a.N, a.K, (unsigned long long)a.ldw * 2,
                                             64, BK);
  if (!okb) return MLP_ERR_CUDA;
  // large outputs with 16-byte rows leave through TMA stores of staged boxes;
  // for small ones the staging round trip is latency
  if (pl.splits == 1 && a.T * a.N >= (1ll << 20)) {
    const int esz = a.out_f32 ? 4 : 2;
    if (a.ldy * esz % 16 == 0 && aligned16(a.y)) {
      if (!encode_tmap_out_2d(&maps[2], a.y, a.out_f32, a.N, a.T,
                              (unsigned long long)a.ldy * esz, 32, 32))
        return MLP_ERR_CUDA;
      p.tma_y = 1;
    }
    // (an fp32 box leaves no room for a second one)
    if (a.u_out && !a.out_f32 && a.ldu_out * 2 % 16 == 0 && aligned16(a.u_out)) {
      if (!encode_tmap_out_2d(&maps[3], a.u_out, 0, a.N, a.T, (unsigned long long)a.ldu_out * 2,
                              32, 32))
        return MLP_ERR_CUDA;
      p.tma_u = 1;
    }
  }
  const bool h16 = a.dtype == MLP_DTYPE_F16;
  if (bwd) return h16 ? launch_tile<1, 1>(maps, p, pl.tile, st) : launch_tile<0, 1>(maps, p, pl.tile, st);
  return h16 ? launch_tile<1, 0>(maps, p, pl.tile, st) : launch_tile<0, 0>(maps, p, pl.tile, st);
}

}  // namespace mlp
