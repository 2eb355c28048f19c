// mx4_few.hip -- products of a 4-bit microscaled matrix with the few tokens of a
// decode step, out = W x.
//
// W is read once, which bounds a single token; with more, x is brought again by every
// workgroup and staged by each wave for itself.  A workgroup of eight waves makes 16 RT rows of W times up
// to 16 NT tokens; the waves take turns at slabs of 128 k, so that together they read
// 512 neighbouring bytes of each row, and add their sums through shared memory at the
// end.  In a slab, lanes 16 g + r hold block g of row r: 16 bytes, one scale, four
// v_mfma_f32_16x16x32 whose k are 32 g + 8 s + j.  The codes of two slabs are in flight
// (four: no faster), and the scales of both come in one load a row, handed on between
// the lanes (a load of each scale cost 2.3 of 10 us on 48 rows a workgroup).
//
// x is taken through shared memory, a part of its own for each wave, where eight k of
// a token are read turned; a single token's x needs no turning and is loaded as it
// is.
//
// 4096 x 4096 in bf16: one token 4.3 to 4.9 us (a launch that only reads W 2.3 to 2.6, an
// empty one 1.6), 16 tokens 5.6; 4096 -> 11008: one 7.8 (only reading 4.4 to 5.0), 32 tokens
// of f16 11.4.
#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "mx4.h"

namespace spops {
namespace {

constexpr int kWaves = 8, kSlab = 128, kAhead = 2;

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <typename T>
struct Cut {
  static constexpr int parts = sizeof(T) == 4 ? 3 : 1;
};

__device__ __forceinline__ f32x4 mma(bf16x8_t a, bf16x8_t b, f32x4 c, bf16_t*) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(bf16x8_t a, bf16x8_t b, f32x4 c, _Float16*) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

// ONE: a single token whose x is contiguous.
template <typename T, int RT, int NT, bool ONE>
__global__ __launch_bounds__(64 * kWaves) void mx4_few_kernel(Mx4MatmulArgs a) {
  constexpr int P = Cut<T>::parts;
  // a row of x: 16 NT tokens; 32 rows and then a gap, so that the rows of two lane
  // groups which are read at once lie in different banks
  constexpr int kRow = 32 * NT, kGroup = 32 * kRow + (NT == 1 ? 128 : 32);
  constexpr int kPart = 4 * kGroup, kX = ONE ? 0 : P * kPart;
  constexpr int kSums = RT * NT * 1024;
  __shared__ __attribute__((aligned(16))) char lds[kWaves * (kX > kSums ? kX : kSums)];

  const Mx4 W = a.W;
  const int64_t nb = (W.cols + kMx4Block - 1) / kMx4Block;
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int g = lane / 16, l16 = lane % 16;
  const int64_t r0 = (int64_t)blockIdx.x * (16 * RT), t0 = (int64_t)blockIdx.y * (16 * NT);
  const int64_t slabs = (W.cols + kSlab - 1) / kSlab;
  const T* const x = (const T*)a.x;
  const int64_t end = (W.cols - 1) * a.ldx + a.T;  // of x
  char* const xs = lds + wave * kX;

  // codes and scales relative to the workgroup's first row; rows past the last read it
  // again, and their sums are not written
  const uint8_t* const wcodes = W.codes + r0 * nb * 16;
  const uint8_t* const wscales = W.scales + r0 * nb;
  uint32_t row_at[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
    row_at[r] = (uint32_t)(min((int64_t)(16 * r + l16), W.rows - 1 - r0) * nb);
  uint4 codes[kAhead][RT];
  const auto load = [&](int64_t slab, uint4 (&c)[RT]) {
    // x is zero past the last column, so any finite block will do there
    const uint32_t b = 4 * (uint32_t)slab + g, last = (uint32_t)nb - 1;
#pragma unroll
    for (int r = 0; r < RT; ++r)
      c[r] = *(const uint4*)(wcodes + (row_at[r] + min(b, last)) * 16u);
  };
  // The scales of kAhead slabs in one load a row: lane group g brings the word of slab g.
  // Past the last block, ones.
  uint32_t words_now[RT], words_next[RT];
  const auto load_scales = [&](int64_t slab, uint32_t (&w)[RT]) {
    const uint32_t b = 4 * (uint32_t)slab;
    if (b + 4 <= (uint32_t)nb) {
#pragma unroll
      for (int r = 0; r < RT; ++r) __builtin_memcpy(&w[r], wscales + row_at[r] + b, 4);
    } else {
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        w[r] = 0x7f7f7f7fu;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (b + i < (uint32_t)nb)
            w[r] = (w[r] & ~(0xffu << (8 * i))) | ((uint32_t)wscales[row_at[r] + b + i] << (8 * i));
      }
    }
  };

  f32x4 acc[RT][NT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[r][n] = (f32x4){0.f, 0.f, 0.f, 0.f};

  // x of one slab as it is loaded: 2 NT lanes a row, or, of a single token, a lane's own
  // eight k of each instruction
  const int xrow = lane / (2 * NT), xchunk = lane % (2 * NT);
  constexpr int kPass = 32 / NT;  // rows of a pass
  constexpr int kRaw = ONE ? 4 : 4 * NT;
  constexpr int kXAhead = ONE && sizeof(T) == 2 ? kAhead : 1;
  Raw<T> raw[kXAhead][kRaw];
  const uint32_t ld = (uint32_t)a.ldx;
  const auto load_x = [&](int64_t slab, Raw<T> (&v)[kRaw]) {
    const int64_t first = slab * kSlab * (ONE ? 1 : a.ldx) + t0;
    const T* const from = x + first;
    // every load of all slabs but the last ones lies inside x
    if (ONE ? first + kSlab <= end : first + (kSlab - 1) * a.ldx + 16 * NT <= end) {
#pragma unroll
      for (int i = 0; i < kRaw; ++i) {
        const uint32_t at =
            ONE ? (uint32_t)(32 * g + 8 * i) : (kPass * i + xrow) * ld + 8 * xchunk;
        __builtin_memcpy(&v[i], from + at, sizeof(v[i]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < kRaw; ++i) {
        if constexpr (ONE) {
          v[i] = load_until(x, first + 32 * g + 8 * i, end);
        } else {
          const int64_t k = slab * kSlab + kPass * i + xrow, t = t0 + 8 * xchunk;
          // a token past the last may hold anything: its column is not written
          v[i] = load_until(x, k * a.ldx + t, k < W.cols && t < a.T ? end : 0);
        }
      }
    }
  };
  // The products of a slab; F: with W in f16.
  const auto slab_product = [&](const uint4 (&c)[RT], const uint32_t (&sc)[RT],
                                const Raw<T> (&one)[kRaw], auto fast) {
    constexpr bool F = decltype(fast)::value;
    if constexpr (ONE && sizeof(T) == 4) {
      // one f32 token: two conversions and fused products a pair of weights cost less
      // than x in three parts
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const uint32_t words[4] = {c[r].x, c[r].y, c[r].z, c[r].w};
          const float scale = mx4_scale(sc[r]);
          const f32x2 w[4] = {mx4_pair_f32<0>(words[s], scale), mx4_pair_f32<1>(words[s], scale),
                              mx4_pair_f32<2>(words[s], scale), mx4_pair_f32<3>(words[s], scale)};
#pragma unroll
          for (int j = 0; j < 8; ++j)
            acc[r][0][0] = fmaf(w[j / 2][j % 2], __uint_as_float(one[s].w[j]), acc[r][0][0]);
        }
      return;
    }
    constexpr int Q = F || __is_same(T, bf16_t) ? 1 : __is_same(T, float) ? 3 : 2;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      bf16x8_t wf[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const uint32_t words[4] = {c[r].x, c[r].y, c[r].z, c[r].w};
        wf[r] = F ? __builtin_bit_cast(bf16x8_t, mx4_eight<_Float16>(words[s], mx4_scale(sc[r])))
                  : __builtin_bit_cast(bf16x8_t, mx4_eight<bf16_t>(words[s], mx4_scale(sc[r])));
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        bf16x8_t xf[Q];
        if constexpr (sizeof(T) == 4 && !ONE) {
#pragma unroll
          for (int q = 0; q < Q; ++q)
            xf[q] = turned(xs + q * kPart + g * kGroup + (8 * s + l16 / 4) * kRow + 32 * n +
                               8 * (l16 % 4),
                           4 * kRow);
        } else {
          Raw<T> v;
          if constexpr (ONE)
            v = one[s];
          else
            v = __builtin_bit_cast(Raw<T>, turned(xs + g * kGroup + (8 * s + l16 / 4) * kRow +
                                                      32 * n + 8 * (l16 % 4),
                                                  4 * kRow));
          uint4 part[Q];
          split<T, Q>(v, part);
#pragma unroll
          for (int q = 0; q < Q; ++q) xf[q] = __builtin_bit_cast(bf16x8_t, part[q]);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int q = 0; q < Q; ++q)
            acc[r][n] = F ? mma(xf[q], wf[r], acc[r][n], (_Float16*)nullptr)
                          : mma(xf[q], wf[r], acc[r][n], (bf16_t*)nullptr);
      }
    }
  };
  // A wave takes two neighbouring slabs, whose codes are whole lines of 128 bytes.
  const auto slab_at = [&](int64_t first, int i) {
    return first + (i / 2) * (2 * kWaves) + 2 * wave + i % 2;
  };
  load_scales(slab_at(0, g % kAhead), words_now);
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(slab_at(0, i), codes[i]);
#pragma unroll
  for (int i = 0; i < kXAhead; ++i) load_x(slab_at(0, i), raw[i]);
  for (int64_t first = 0; slab_at(first, 0) < slabs; first += kAhead * kWaves) {
    // the registers of a slab are loaded again as soon as it is done
    const int64_t then = first + kAhead * kWaves;
    const bool more = slab_at(then, 0) < slabs;
    if (more) load_scales(slab_at(then, g % kAhead), words_next);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t slab = slab_at(first, i);
      if (slab >= slabs) break;
      constexpr int kOne = kXAhead;
      if constexpr (!ONE) {
#pragma unroll
        for (int j = 0; j < kRaw; ++j) {
          const int first_row = kPass * j;  // of 32 rows no pass crosses the end
          uint4 part[P];
          split<T, P>(raw[0][j], part);
#pragma unroll
          for (int p = 0; p < P; ++p)
            *(uint4*)(xs + p * kPart + (first_row / 32) * kGroup +
                      (first_row % 32 + xrow) * kRow + 16 * xchunk) = part[p];
        }
        wave_fence();
        load_x(i + 1 < kAhead ? slab_at(first, i + 1) : slab_at(then, 0), raw[0]);
      }
      uint32_t scale[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r)
        scale[r] = ((uint32_t)__shfl((int)words_now[r], 16 * i + l16, 64) >> (8 * g)) & 0xffu;
      const Raw<T>(&one)[kRaw] = raw[i % kOne];
      if constexpr (__is_same(T, _Float16)) {
        // scales that f16 does not hold: the slab runs on bf16, with x in two parts
        bool wide = false;
#pragma unroll
        for (int r = 0; r < RT; ++r) wide |= scale[r] - 104u > 36u;
        if (__any(wide))
          slab_product(codes[i], scale, one, std::false_type());
        else
          slab_product(codes[i], scale, one, std::true_type());
      } else {
        slab_product(codes[i], scale, one, std::false_type());
      }
      if (more) load(slab_at(then, i), codes[i]);
      if constexpr (ONE) {
        if (kXAhead == kAhead)
          if (more) load_x(slab_at(then, i), raw[i % kOne]);
        if (kXAhead == 1)
          load_x(i + 1 < kAhead ? slab_at(first, i + 1) : slab_at(then, 0), raw[0]);
      } else {
        wave_fence();
      }
    }
    if (more) {
#pragma unroll
      for (int r = 0; r < RT; ++r) words_now[r] = words_next[r];
    }
  }
  if constexpr (ONE && sizeof(T) == 4) {
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      acc[r][0][0] += __shfl_xor(acc[r][0][0], 16, 64);
      acc[r][0][0] += __shfl_xor(acc[r][0][0], 32, 64);
    }
  }

  // the waves' sums: a lane holds row lane % 16 and tokens 4 (lane / 16) + i
  __syncthreads();
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n)
      *(f32x4*)(lds + wave * kSums + ((r * NT + n) * 64 + lane) * 16) = acc[r][n];
  __syncthreads();
  for (int i = tid; i < RT * NT * 64; i += 64 * kWaves) {
    f32x4 v = *(const f32x4*)(lds + i * 16);
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += *(const f32x4*)(lds + w * kSums + i * 16);
    const int l = i % 64, n = i / 64 % NT, r = i / 64 / NT;
    const int64_t row = r0 + 16 * r + l % 16, t = t0 + 16 * n + 4 * (l / 16);
    if (row >= W.rows) continue;
    T* const p = (T*)a.out + row * a.ldo + t;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (t + j < a.T) p[j] = from_f32<T>(v[j]);
  }
}

template <typename T, int RT, int NT, bool ONE>
hipError_t launch(const Mx4MatmulArgs& a, hipStream_t s) {
  const dim3 grid((uint32_t)cdiv(a.W.rows, 16 * RT), (uint32_t)cdiv(a.T, 16 * NT));
  mx4_few_kernel<T, RT, NT, ONE><<<grid, 64 * kWaves, 0, s>>>(a);
  return hipGetLastError();
}

// As few rows a workgroup as leave one workgroup a compute unit: more of them bring the
// same x again (11008 rows, 32 tokens f16: 11.4 us with 48 rows, 19 with 32, 20 with 16).
template <typename T, int NT, bool ONE>
hipError_t rows(const Mx4MatmulArgs& a, hipStream_t s) {
  switch (cdiv(a.W.rows, 16 * 256)) {
    case 1: return launch<T, 1, NT, ONE>(a, s);
    case 2: return launch<T, 2, NT, ONE>(a, s);
    case 3: return launch<T, 3, NT, ONE>(a, s);
    default: return launch<T, 4, NT, ONE>(a, s);
  }
}

template <typename T>
hipError_t few(const Mx4MatmulArgs& a, hipStream_t s) {
  if (a.T == 1 && (a.ldx == 1 || a.W.cols == 1)) return rows<T, 1, true>(a, s);
  if constexpr (sizeof(T) == 2) {
    // 64 tokens: on 4096 rows 12.0 us at once and 13.8 in two tiles, on 11008 26.8 and 23.6
    if (a.T > 32 && a.W.rows <= 4096) return launch<T, 1, 4, false>(a, s);
    if (a.T > 16) return rows<T, 2, false>(a, s);
  }
  return rows<T, 1, false>(a, s);
}

}  // namespace

hipError_t launch_mx4_few(const Mx4MatmulArgs& a, int dtype, hipStream_t s) {
  if (dtype == kF32) return few<float>(a, s);
  if (dtype == kF16) return few<_Float16>(a, s);
  return few<bf16_t>(a, s);
}

}  // namespace spops
