// What the tensor-core kernels with an epilogue of their own share (linear
// layers, gated units): the order of tiles, and the pieces of an epilogue warp's
// work between accumulator, staging boxes and matrices.
#pragma once

#include "f32x2.cuh"
#include "ptx.cuh"

namespace mlp {

namespace {

// Eight tile rows at a time sweep all tile columns, so that CTAs that run
// together share row and column blocks in L2.  Every warp does this for every
// tile, so the division by the tiles of a group is a multiplication (`magic` =
// ceil(2^32 / (8 tiles_n)): the quotient or one more) and full groups shift.
template <typename P>
__device__ __forceinline__ void tile_of(const P& p, int t, int& tm, int& tn) {
  const int per = 8 * p.tiles_n;
  int group = (int)__umulhi((unsigned)t, p.magic);
  if (group * per > t) --group;
  const int first = group * 8, r = t - group * per;
  const int gm = min(p.tiles_m - first, 8);
  if (gm == 8) {
    tm = first + (r & 7);
    tn = r >> 3;
  } else {
    tm = first + r % gm;
    tn = r / gm;
  }
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

// 16-byte chunk c of row r of a box whose rows are 32, 64 or 128 bytes, in the
// swizzle that a tensor map of that width names.
__device__ __forceinline__ uint8_t* chunk_at(uint8_t* box, int row_bytes, int r, int c) {
  const int swz = row_bytes == 128 ? r & 7 : row_bytes == 64 ? (r >> 1) & 3 : (r >> 2) & 1;
  return box + r * row_bytes + ((c ^ swz) << 4);
}

// One value per lane and row; what is read from memory four rows at a time, so
// that their latencies overlap (backward of 43,599 x 144 -> 1,241 fp16 from u
// kept at an odd pitch: 480 us one by one, 261 this way).
template <bool OUT, typename V>
__device__ __forceinline__ void warp_copy_values(uint8_t* box, int row_bytes, uint8_t* mem,
                                                 long long ld, int rows, int n, int lane) {
  constexpr int B = OUT ? 1 : 4;  // rows at a time (more spill)
#pragma unroll 1
  for (int j = lane; j < n; j += 32) {
    const int o = j * (int)sizeof(V);
#pragma unroll 1
    for (int r = 0; r < rows; r += B) {
      V v[B];
#pragma unroll
      for (int k = 0; k < B; ++k) {
        const uint8_t* bp = chunk_at(box, row_bytes, r + k, o >> 4) + (o & 15);
        if (r + k < rows)
          v[k] = *reinterpret_cast<const V*>(OUT ? bp : mem + (r + k) * ld + o);
      }
#pragma unroll
      for (int k = 0; k < B; ++k) {
        uint8_t* bp = chunk_at(box, row_bytes, r + k, o >> 4) + (o & 15);
        if (r + k < rows) *reinterpret_cast<V*>(OUT ? mem + (r + k) * ld + o : bp) = v[k];
      }
    }
  }
}

// The warp's own copy between a box and a matrix: `rows` rows of `bytes` bytes,
// `esz` per value, at mem with a pitch of ld bytes.  16-byte pieces where rows
// and widths allow, else one value per lane (runs of 32 values either way).
template <bool OUT>
__device__ __forceinline__ void warp_copy(uint8_t* box, int row_bytes, uint8_t* mem, long long ld,
                                          int rows, int bytes, int esz, int lane) {
  __syncwarp();
  if ((reinterpret_cast<uintptr_t>(mem) & 15) == 0 && (ld & 15) == 0 && (bytes & 15) == 0) {
    const int per = bytes >> 4;
#pragma unroll 1
    for (int i = lane; i < rows * per; i += 32) {
      const int r = i / per, c = i - r * per;
      uint4* b = reinterpret_cast<uint4*>(chunk_at(box, row_bytes, r, c));
      uint4* m = reinterpret_cast<uint4*>(mem + r * ld + c * 16);
      if (OUT) *m = *b;
      else *b = *m;
    }
  } else if (esz == 1) {
    warp_copy_values<OUT, uint8_t>(box, row_bytes, mem, ld, rows, bytes, lane);
  } else if (esz == 2) {
    warp_copy_values<OUT, uint16_t>(box, row_bytes, mem, ld, rows, bytes >> 1, lane);
  } else {
    warp_copy_values<OUT, uint32_t>(box, row_bytes, mem, ld, rows, bytes >> 2, lane);
  }
  __syncwarp();
}

// Values into this lane's row of a 16-bit box, from chunk `c0`.
template <int H16, int PAIRS>
__device__ __forceinline__ void pack_row(uint8_t* box, int row_bytes, int lane, int c0,
                                         const F2 (&v)[PAIRS]) {
#pragma unroll
  for (int k = 0; k < PAIRS / 4; ++k)
    *reinterpret_cast<uint4*>(chunk_at(box, row_bytes, lane, c0 + k)) =
        make_uint4(pack16x2<H16>(v[4 * k].x, v[4 * k].y),
                   pack16x2<H16>(v[4 * k + 1].x, v[4 * k + 1].y),
                   pack16x2<H16>(v[4 * k + 2].x, v[4 * k + 2].y),
                   pack16x2<H16>(v[4 * k + 3].x, v[4 * k + 3].y));
}

// Four consecutive bias values.  Volatile, so that the loads stay ahead of the
// accumulator's (the compiler would sink them to their use, behind it).
__device__ __forceinline__ float4 load_bias4(const float* p) {
  float4 f;
  asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w)
               : "l"(p));
  return f;
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

}  // namespace

}  // namespace mlp
