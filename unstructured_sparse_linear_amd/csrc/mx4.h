// mx4.h -- device helpers of the 4-bit microscaled matrices (mx4.hip,
// mx4_matmul.hip, mx4_mma.hip).
//
// A row holds blocks of 32 elements: 16 bytes of codes (element 2j is the low half
// of byte j; sign, two bits of exponent, one of mantissa) and one scale byte s that
// stands for 2^(s - 127), or NaN at 255.  gfx950 converts pairs of elements with
// the scale applied in one instruction, exactly as far as the target type holds the
// value: bf16 and f32 hold all of them (scales from 253 on pass their range), f16
// those of the scales 104 to 140.  The conversions take the scale as the exponent
// field of an f32, where zero stands for 2^-127 and 255 for NaN.
#pragma once

#include "common.h"

namespace spops {

constexpr int kMx4Block = 32;

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float mx4_scale(uint32_t code) { return __uint_as_float(code << 23); }

// Elements 2 S and 2 S + 1 of a word of eight, as a pair of 16 bits.
template <int S>
__device__ __forceinline__ uint32_t mx4_pair(uint32_t w, float scale, bf16_t*) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, S));
}
template <int S>
__device__ __forceinline__ uint32_t mx4_pair(uint32_t w, float scale, _Float16*) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, S));
}
template <int S>
__device__ __forceinline__ f32x2 mx4_pair_f32(uint32_t w, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, S);
}

// A word of eight elements as eight values of 16 bits.
template <typename T>
__device__ __forceinline__ uint4 mx4_eight(uint32_t w, float scale) {
  T* const t = nullptr;
  return make_uint4(mx4_pair<0>(w, scale, t), mx4_pair<1>(w, scale, t), mx4_pair<2>(w, scale, t),
                    mx4_pair<3>(w, scale, t));
}

// The scale byte of a block whose largest magnitude has the f32 bits `top`: the
// largest power of two with top below 8 times it, so that the largest element (6)
// is reached and values between 6 and 8 times it saturate.  A block of zeros has
// scale 1, one that holds an infinity or a NaN has 255.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t top) {
  if (top >= 0x7f800000u) return 255u;
  if (top == 0u) return 127u;
  const int e = (int)(top >> 23) - 2;
  return e > 0 ? (uint32_t)e : 0u;
}

// Eight values to eight codes (round to nearest even, saturating).
__device__ __forceinline__ uint32_t mx4_encode(const float (&v)[8], float scale) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
  return w;
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Eight values of x as they were loaded.
template <typename T>
struct Raw {
  uint32_t w[2 * sizeof(T)];
};

template <typename T>
__device__ __forceinline__ float raw_value(const Raw<T>& r, int i) {
  if constexpr (sizeof(T) == 4)
    return __uint_as_float(r.w[i]);
  else
    return i % 2 ? hi_f32(r.w[i / 2], (T*)nullptr) : lo_f32(r.w[i / 2], (T*)nullptr);
}

// Part p of eight values, as bf16 pairs: the upper 16 bits of the value, of what is
// left, of what is left then.  An infinity or a NaN is all in the first part.
template <typename T, int P>
__device__ __forceinline__ void split(const Raw<T>& r, uint4 (&part)[P]) {
  if constexpr (P == 1) {
    part[0] = __builtin_bit_cast(uint4, r);
  } else {
    uint32_t w[P][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[2] = {raw_value(r, 2 * i), raw_value(r, 2 * i + 1)};
#pragma unroll
      for (int p = 0; p < P; ++p) {
        uint32_t b[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          b[j] = __float_as_uint(v[j]);
          // a NaN whose upper bits are an infinity's stays a NaN
          if (p == 0 && magnitude(v[j]) > 0x7f800000u) b[j] |= 0x400000u;
          const float rest = v[j] - __uint_as_float(b[j] & 0xffff0000u);
          v[j] = magnitude(v[j]) >= 0x7f800000u ? 0.f : rest;
        }
        w[p][i] = __builtin_amdgcn_perm(b[1], b[0], 0x07060302u);
      }
    }
#pragma unroll
    for (int p = 0; p < P; ++p) part[p] = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
  }
}

// Eight values of x from element `at` on, of which those from `end` on are not read.
template <typename T>
__device__ __forceinline__ Raw<T> load_until(const T* x, int64_t at, int64_t end) {
  Raw<T> r;
  if (at + 8 <= end) {
    __builtin_memcpy(&r, x + at, sizeof(r));
    return r;
  }
#pragma unroll
  for (int i = 0; i < (int)(2 * sizeof(T)); ++i) r.w[i] = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (at + i >= end) break;
    if constexpr (sizeof(T) == 4)
      r.w[i] = __float_as_uint(x[at + i]);
    else
      r.w[i / 2] |= (uint32_t)bits16(x[at + i]) << (16 * (i % 2));
  }
  return r;
}

typedef __attribute__((address_space(3))) i16x4* Lds4;

// Eight consecutive k of one column of a tile of rows of k, from the four lanes' rows
// at `at` and four rows further: each group of 16 lanes reads four rows of 16 columns
// and gets, in lane i, column i of them.
__device__ __forceinline__ bf16x8_t turned(const char* at, int four_rows) {
  const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds4)at);
  const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds4)(at + four_rows));
  struct {
    i16x4 a, b;
  } v = {lo, hi};
  return __builtin_bit_cast(bf16x8_t, v);
}

// Workgroup index -> logical index, so that neighbours run on one XCD (workgroup b is
// on XCD b mod 8).
__device__ __forceinline__ uint32_t xcd_index(uint32_t b, uint32_t n) {
  const uint32_t q = b % 8, each = n / 8, more = n % 8;
  return q * each + min(q, more) + b / 8;
}

// What a workgroup makes: whole tiles first, then the rest of them in pieces of the
// inner size.  Tiles go four columns at a time, so that an XCD's workgroups share rows
// and columns.
struct Mx4Cut {
  uint32_t tiles_m, tiles_n;
  uint32_t whole;          // tiles made whole (a multiple of 8, or all)
  uint32_t pieces;         // of each of the others
  int32_t steps;           // in a piece
};
struct Mx4Place {
  uint32_t m, n;           // tile
  uint32_t rest, piece;    // of the tiles in pieces, which
  bool cut;
};
__host__ __device__ inline void mx4_place(const Mx4Cut& c, uint32_t tile, uint32_t& m,
                                          uint32_t& n) {
  const uint32_t band = tile / (4 * c.tiles_m), in = tile % (4 * c.tiles_m);
  const uint32_t left = c.tiles_n - 4 * band, wide = left < 4 ? left : 4;
  m = in / wide;
  n = 4 * band + in % wide;
}
__device__ __forceinline__ Mx4Place mx4_place(const Mx4Cut& c, uint32_t block) {
  Mx4Place p{0, 0, 0, 0, block >= c.whole};
  uint32_t tile;
  if (!p.cut) {
    tile = xcd_index(block, c.whole);
  } else {
    const uint32_t rest = c.tiles_m * c.tiles_n - c.whole;
    const uint32_t i = xcd_index(block - c.whole, rest * c.pieces);
    // a tile's pieces on one XCD, where they are added too: their sums are in its L2
    // (f32 gradient of 512 tokens, 2048 x 2048: 36.6 us, 43.2 with pieces apart)
    p.rest = i / c.pieces;
    p.piece = i % c.pieces;
    tile = c.whole + p.rest;
  }
  mx4_place(c, tile, p.m, p.n);
  return p;
}
inline uint32_t mx4_blocks(const Mx4Cut& c) {
  return c.whole + (c.tiles_m * c.tiles_n - c.whole) * c.pieces;
}
inline size_t mx4_part_bytes(const Mx4Cut& c, int64_t bm, int64_t bn) {
  return (size_t)(c.tiles_m * c.tiles_n - c.whole) * c.pieces * bm * bn * 4;
}

// A wave's memory is written before it is read by other lanes, and read before it is
// written again.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Shared memory a wave needs for mx4_write.
constexpr int kWriteBytes = 32 * (256 + 16);

// TN results of v_mfma_f32_32x32x* side by side whose rows are tokens and whose columns
// are rows of W: a lane holds row r0 + lane % 32 and runs of four tokens.  They go
// through shared memory, up to 256 bytes of a row at a time, so that a row's tokens are
// stored 16 bytes a lane side by side (stored as they are held, 8 bytes of 32 rows at a
// time, they took 25 of 80 us of 4096^2 in four bits on 4096 tokens).
template <typename E, int TN>
__device__ __forceinline__ void mx4_write(const f32x16 (&acc)[TN], char* lds, int64_t r0,
                                          int64_t t0, int64_t M, int64_t tokens, E* out,
                                          int64_t ld) {
  constexpr int N = TN * sizeof(E) < 8 ? TN : 8 / sizeof(E);  // results at a time
  constexpr int kRow = N * 32 * sizeof(E) + 16, kEach = 16 / sizeof(E);
  constexpr int kLanes = N * 32 / kEach, kRows = 64 / kLanes;
  const int lane = lane_id();
#pragma unroll
  for (int n0 = 0; n0 < TN; n0 += N) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint32_t v[sizeof(E)];
        if constexpr (sizeof(E) == 2) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            v[i] = pair16(acc[n0 + n][4 * g + 2 * i], acc[n0 + n][4 * g + 2 * i + 1], (E*)nullptr);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(acc[n0 + n][4 * g + i]);
        }
        char* const to = lds + lane % 32 * kRow + (32 * n + 8 * g + 4 * (lane / 32)) * sizeof(E);
        __builtin_memcpy(__builtin_assume_aligned(to, 4 * sizeof(E)), v, sizeof(v));
      }
    wave_fence();
    const int64_t t = t0 + 32 * n0 + lane % kLanes * kEach;
#pragma unroll
    for (int i = 0; i < 32 / kRows; ++i) {
      const int r = i * kRows + lane / kLanes;
      if (r0 + r >= M || t >= tokens) continue;
      E v[kEach];
      __builtin_memcpy(v, __builtin_assume_aligned(lds + r * kRow + lane % kLanes * 16, 16), 16);
      E* const p = out + (r0 + r) * ld + t;
      if (t + kEach <= tokens) {
        __builtin_memcpy(p, v, 16);
      } else {
#pragma unroll
        for (int j = 0; j < kEach; ++j)
          if (t + j < tokens) p[j] = v[j];
      }
    }
    wave_fence();
  }
}

// out = the sums of the pieces of the tiles that were cut (bm rows x bn tokens each),
// added in order (mx4.hip); part is [piece][tile][bm][bn].
hipError_t launch_mx4_sum(const float* part, const Mx4Cut& c, int bm, int bn, int64_t M,
                          int64_t tokens, void* out, int dtype, int64_t ldo, hipStream_t s);

}  // namespace spops
