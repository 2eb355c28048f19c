// lowrank.h -- device helpers of the low-rank adapter kernels (lowrank.hip).
//
// Every product runs on 16x16 MFMA tiles over K blocks of 32.  A lane holds
// eight consecutive k of one row (k = 8 (lane / 16) + s, row = lane % 16): for
// f16 and bf16 that is one v_mfma_f32_16x16x32; for f32 the eight values feed
// eight v_mfma_f32_16x16x4, whose k index is lane / 16, so the same fragment
// serves (the order of k inside the block does not matter to the sum).  The
// result tile has column n = lane % 16 and rows m = 4 (lane / 16) + i.
#pragma once

#include "common.h"

namespace spops {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

template <typename T>
struct Frag {
  uint32_t w[2 * sizeof(T)];  // eight elements
};

__device__ __forceinline__ f32x4 mma(const Frag<bf16_t>& a, const Frag<bf16_t>& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(const Frag<_Float16>& a, const Frag<_Float16>& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(const Frag<float>& a, const Frag<float>& b, f32x4 c) {
#pragma unroll
  for (int s = 0; s < 8; ++s)
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.w[s]), __uint_as_float(b.w[s]), c,
                                             0, 0, 0);
  return c;
}

// Eight consecutive elements; the address is aligned to the element only
// (gfx950 takes unaligned global accesses of any width).
template <typename T>
__device__ __forceinline__ Frag<T> load8(const T* p) {
  Frag<T> f;
  __builtin_memcpy(&f, p, sizeof(f));
  return f;
}

__device__ __forceinline__ uint32_t raw_bits(const float* p) { return __float_as_uint(*p); }
__device__ __forceinline__ uint32_t raw_bits(const _Float16* p) { return bits16(*p); }
__device__ __forceinline__ uint32_t raw_bits(const bf16_t* p) { return p->bits; }

// The first `cnt` (0..8) of eight elements, zeros for the rest.
template <typename T>
__device__ __forceinline__ Frag<T> load8_count(const T* p, int cnt) {
  Frag<T> f;
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    const uint32_t b = s < cnt ? raw_bits(p + s) : 0u;
    if (sizeof(T) == 4)
      f.w[s] = b;
    else if (s % 2 == 0)
      f.w[s / 2] = b;
    else
      f.w[s / 2] |= b << 16;
  }
  return f;
}

// Keeps element s where bit s of m is set, zeros the others (a select, not a
// product: a NaN or infinity in a masked place leaves nothing behind).
template <typename T>
__device__ __forceinline__ void mask8(Frag<T>& f, uint32_t m) {
  if (sizeof(T) == 4) {
#pragma unroll
    for (int s = 0; s < 8; ++s) f.w[s] = (m >> s) & 1u ? f.w[s] : 0u;
  } else {
#pragma unroll
    for (int s = 0; s < 4; ++s)
      f.w[s] &= ((m >> (2 * s)) & 1u ? 0xffffu : 0u) | ((m >> (2 * s)) & 2u ? 0xffff0000u : 0u);
  }
}

// Infinities and NaN made finite where `on` (the largest value of their sign), other
// values as they are.  Compared as integers: a positive value's bits grow with it,
// and a negative one's, unsigned, with its magnitude.  Two packed instructions per
// pair and no branch, which would cut the schedule of the products around it (64
// requests of one token, 11008 x 4096, 16 ranks: 20.8 us, 20.3 without; 64 ranks'
// gradients of 4096 tokens 76.3 and 76.2).
typedef int16_t i16x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t largest_pair(bf16_t*) { return 0x7f7f7f7fu; }
__device__ __forceinline__ uint32_t largest_pair(_Float16*) { return 0x7bff7bffu; }
template <typename T>
__device__ __forceinline__ Frag<T> made_finite(Frag<T> f, bool on) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t most = on ? largest_pair((T*)nullptr) : 0x7fff7fffu;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const i16x2 v = __builtin_elementwise_min(__builtin_bit_cast(i16x2, f.w[i]),
                                                __builtin_bit_cast(i16x2, most));
      const u16x2 w = __builtin_elementwise_min(__builtin_bit_cast(u16x2, v),
                                                __builtin_bit_cast(u16x2, most | 0x80008000u));
      f.w[i] = __builtin_bit_cast(uint32_t, w);
    }
  }
  return f;
}

// V consecutive elements of one row of a matrix whose rows run along k.
template <typename T, int V>
struct Row {
  uint32_t w[(V * sizeof(T) + 3) / 4];
};
template <typename T, int V>
__device__ __forceinline__ Row<T, V> load_row(const T* p) {
  Row<T, V> r;
  if constexpr (V * sizeof(T) == 2)
    r.w[0] = raw_bits(p);
  else
    __builtin_memcpy(&r, p, V * sizeof(T));
  return r;
}
template <typename T, int V>
__device__ __forceinline__ void zero_row(Row<T, V>& r) {
#pragma unroll
  for (int i = 0; i < (int)(sizeof(r.w) / 4); ++i) r.w[i] = 0u;
}

// Eight rows (k) of V columns, turned in registers: the fragment of column j.
// 16-bit pairs are joined with one v_perm per word, so a block costs half an
// instruction per element and no shared memory.
template <typename T, int V>
__device__ __forceinline__ Frag<T> column(const Row<T, V> (&r)[8], int j) {
  Frag<T> f;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int s = 0; s < 8; ++s) f.w[s] = r[s].w[j];
  } else {
#pragma unroll
    for (int p = 0; p < 4; ++p)
      f.w[p] = __builtin_amdgcn_perm(r[2 * p + 1].w[j / 2], r[2 * p].w[j / 2],
                                     j % 2 ? 0x07060302u : 0x05040100u);
  }
  return f;
}

// ------------------------------------------- the inner product's two halves --
//
// u = A x is kept in fp32.  As an operand of a 16-bit MFMA it is split into
// hi + lo of the storage type, each product run twice (or, for ranks up to 16,
// once: hi and lo fill the two halves of the 32-wide K block), so that the
// second product sees 16 (bf16) to 22 (f16) bits of u and the result's one
// rounding is the output's.  f16 has a narrow exponent range: its operand is
// scaled by a power of two that brings the largest finite |u| near one, and the fp32
// result is scaled back.  The other operand meets hi as it is and lo with its
// infinities and NaN made finite: infinity times u is infinity times hi, whose
// sign is u's, and a lo that is zero or of the other sign must not turn it into NaN.

// hi or lo of u (one element's bits).  bf16: hi truncates, so it never
// overflows; the remainder is exact and rounded once.  A non-finite u goes
// into hi alone.  f16: under 2^-25 of the largest, u counts as zero.
__device__ __forceinline__ uint32_t split_bits(float u, bool lo, bf16_t*) {
  const uint32_t hb = __float_as_uint(u) & 0xffff0000u;
  if (!lo) return (__float_as_uint(u) & 0x7fffffffu) > 0x7f800000u ? 0x7fc0u : hb >> 16;
  const float rest = u - __uint_as_float(hb);
  const uint32_t r = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)rest);
  return (__float_as_uint(u) & 0x7f800000u) == 0x7f800000u ? 0u : r;
}
__device__ __forceinline__ uint32_t split_bits(float u, bool lo, _Float16*) {
  const _Float16 h = (_Float16)u;
  if (!lo) return bits16(h);
  const float hf = (float)h;
  const uint32_t r = bits16((_Float16)(u - hf));
  return (__float_as_uint(hf) & 0x7f800000u) == 0x7f800000u ? 0u : r;
}

template <typename T>
__device__ __forceinline__ Frag<T> split8(const float (&u)[8], bool lo) {
  Frag<T> f;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int s = 0; s < 8; ++s) f.w[s] = __float_as_uint(u[s]);
  } else {
#pragma unroll
    for (int s = 0; s < 8; s += 2)
      f.w[s / 2] = split_bits(u[s], lo, (T*)nullptr) | split_bits(u[s + 1], lo, (T*)nullptr) << 16;
  }
  return f;
}

// The larger of m and |u|, or m where u is infinite or NaN: finite values keep
// their range beside it.
constexpr float kMaxFloat = 3.402823466e38f;
__device__ __forceinline__ float max_finite(float m, float u) {
  u = fabsf(u);
  return u > m && u <= kMaxFloat ? u : m;
}

// 2^-e and 2^e for the exponent e of m, the largest finite |u|.
struct Pow2 {
  float down, up;
};
__device__ __forceinline__ Pow2 pow2_of(float m) {
  uint32_t b = (__float_as_uint(m) >> 23) & 255u;
  b = b < 2u ? 2u : b > 252u ? 252u : b;
  Pow2 p;
  p.down = __uint_as_float((254u - b) << 23);
  p.up = __uint_as_float(b << 23);
  return p;
}

// fp32 -> storage, the hardware's round to nearest even.
__device__ __forceinline__ uint32_t out_bits(float x, bf16_t*) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x);
}
__device__ __forceinline__ uint32_t out_bits(float x, _Float16*) { return bits16((_Float16)x); }
__device__ __forceinline__ uint32_t out_bits(float x, float*) { return __float_as_uint(x); }

__device__ __forceinline__ void store_bits(float* p, uint32_t b) { *p = __uint_as_float(b); }
__device__ __forceinline__ void store_bits(_Float16* p, uint32_t b) {
  *p = __builtin_bit_cast(_Float16, (uint16_t)b);
}
__device__ __forceinline__ void store_bits(bf16_t* p, uint32_t b) { p->bits = (uint16_t)b; }

// Element e of a row as fp32.
template <typename T, int V>
__device__ __forceinline__ float row_f32(const Row<T, V>& r, int e) {
  const uint32_t b = r.w[e * sizeof(T) / 4];
  if constexpr (sizeof(T) == 4)
    return __uint_as_float(b);
  else
    return e % 2 ? hi_f32(b, (T*)nullptr) : lo_f32(b, (T*)nullptr);
}

// C consecutive elements as fp32, and back; the first `cnt` only where the
// row ends inside.
template <typename T, int C>
__device__ __forceinline__ void load_chunk(const T* p, int cnt, float (&v)[C]) {
  Row<T, C> r;
  if (cnt >= C) {
    r = load_row<T, C>(p);
  } else {
    zero_row(r);
#pragma unroll
    for (int e = 0; e < C; ++e)
      if (e < cnt) r.w[e * sizeof(T) / 4] |= raw_bits(p + e) << (e * sizeof(T) * 8 % 32);
  }
#pragma unroll
  for (int e = 0; e < C; ++e) {
    const uint32_t b = r.w[e * sizeof(T) / 4];
    if constexpr (sizeof(T) == 4)
      v[e] = __uint_as_float(b);
    else
      v[e] = e % 2 ? hi_f32(b, (T*)nullptr) : lo_f32(b, (T*)nullptr);
  }
}
template <typename T, int C>
__device__ __forceinline__ void store_chunk(T* p, int cnt, const float (&v)[C]) {
  uint32_t b[C];
#pragma unroll
  for (int e = 0; e < C; ++e) b[e] = out_bits(v[e], (T*)nullptr);
  if (cnt >= C) {
    Row<T, C> r;
    zero_row(r);
#pragma unroll
    for (int e = 0; e < C; ++e) r.w[e * sizeof(T) / 4] |= b[e] << (e * sizeof(T) * 8 % 32);
    if constexpr (C * sizeof(T) == 2)
      store_bits(p, r.w[0]);
    else
      __builtin_memcpy(p, &r, C * sizeof(T));
  } else {
#pragma unroll
    for (int e = 0; e < C; ++e)
      if (e < cnt) store_bits(p + e, b[e]);
  }
}

__device__ __forceinline__ int clampi(int64_t v, int lo, int hi) {
  return v < lo ? lo : v > hi ? hi : (int)v;
}

}  // namespace spops
