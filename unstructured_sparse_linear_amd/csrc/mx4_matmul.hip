// mx4_matmul.hip -- products of a 4-bit microscaled matrix W with dense activations.
//
//   out = W x    (x [cols][T], out [rows][T]),
//   out = W^T x  (x [rows][T], out [cols][T], the gradient of the input).
//
// An element of W times its scale has two significant bits, so bf16 holds it and its
// product with a bf16 value is exact in f32.  x of f32 is cut into three bf16 parts
// of eight bits each and x of f16 into two, which loses nothing (of f32 values under
// 2^-109 the bits below 2^-133, the smallest bf16); every product is then exact and the
// sums are f32.  Eight consecutive elements of the inner size (k)
// feed one half of v_mfma_f32_32x32x16_bf16 (row = lane % 32, half = lane / 32).
//
// A workgroup makes BM rows x BN tokens in steps of 64 k.  In a step, half h holds
// the elements 32 h + 8 s + j of instruction s, so that the 16 bytes which a lane
// loads of W are one block of one row, with one scale, for four instructions.
#include <algorithm>

#include "kernels.h"
#include "mx4.h"

namespace spops {
namespace {

constexpr int kStep = 64;

template <typename T>
struct Parts;
template <>
struct Parts<bf16_t> {
  static constexpr int n = 1;
};
template <>
struct Parts<_Float16> {
  static constexpr int n = 2;
};
template <>
struct Parts<float> {
  static constexpr int n = 3;
};

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

// Eight values of row k from token t on; zeros past the matrix.
template <typename T>
__device__ __forceinline__ Raw<T> load_edge(const T* x, int64_t ldx, int64_t k, int64_t t,
                                            int64_t K, int64_t tokens) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < (int)(2 * sizeof(T)); ++i) r.w[i] = 0u;
  if (k >= K || t >= tokens) return r;
  const T* const p = x + k * ldx + t;
  if (t + 8 <= tokens) {
    __builtin_memcpy(&r, p, sizeof(r));
    return r;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (t + i >= tokens) break;
    if constexpr (sizeof(T) == 4)
      r.w[i] = __float_as_uint(p[i]);
    else
      r.w[i / 2] |= (uint32_t)bits16(p[i]) << (16 * (i % 2));
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

// Block b of row r of W; past the matrix, zeros.
struct Block {
  uint4 c;
  uint32_t s;
};
__device__ __forceinline__ Block load_block(const Mx4& W, int64_t nb, int64_t r, int64_t b) {
  Block v{make_uint4(0u, 0u, 0u, 0u), 127u};
  if (r < W.rows && b < nb) {
    v.c = *(const uint4*)(W.codes + (r * nb + b) * 16);
    v.s = W.scales[r * nb + b];
  }
  return v;
}

template <typename T, bool TR, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void mx4_tile_kernel(Mx4MatmulArgs a,
                                                                   uint32_t tiles_m,
                                                                   uint32_t tiles_n) {
  constexpr int P = Parts<T>::n, kThreads = 64 * WM * WN;
  constexpr int TM = BM / WM / 32, TN = BN / WN / 32;
  constexpr int kChunks = BN / 8, kRows = kThreads / kChunks, kPasses = kStep / kRows;
  constexpr int kXBytes = kStep * BN * 2, kWBytes = TR ? kStep * BM * 2 : 0;
  constexpr int kBlocks = BM / 32;  // of a row of W, transposed
  static_assert(!TR || kThreads == kStep * kBlocks, "a block a thread");
  __shared__ __attribute__((aligned(16))) char lds[2 * (P * kXBytes + kWBytes)];

  const Mx4 W = a.W;
  const int64_t nb = (W.cols + kMx4Block - 1) / kMx4Block;
  const int64_t M = TR ? W.cols : W.rows, K = TR ? W.rows : W.cols;
  const uint32_t index = xcd_index(blockIdx.x, gridDim.x);
  const uint32_t tile = index % (tiles_m * tiles_n), piece = index / (tiles_m * tiles_n);
  // four columns of tiles at a time, so that an XCD's workgroups share rows and columns
  const uint32_t band = tile / (4 * tiles_m), in = tile % (4 * tiles_m);
  const uint32_t wide = min(4u, tiles_n - 4 * band);
  const int64_t m0 = (int64_t)(in / wide) * BM, t0 = (int64_t)(4 * band + in % wide) * BN;
  const int64_t first = (int64_t)piece * a.steps;
  const int64_t last = min(first + a.steps, (K + kStep - 1) / kStep);

  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int wm = wave / WN, wn = wave % WN, half = lane / 32;
  // x is stored with the 64-byte groups of a row turned by the row, so that the four
  // rows that are read at once lie in different banks
  const int xrow = tid / kChunks, xchunk = tid % kChunks;
  const int64_t xt = t0 + 8 * xchunk;
  const int xstore = (xrow * kChunks + (xchunk ^ ((xrow & 3) << 2))) * 16;
  const int l16 = lane % 16, sub = (lane / 16) % 2;
  const int chunk = 2 * sub + (l16 % 4) / 2, byte = 8 * (l16 & 1), trow = 32 * half + l16 / 4;
  int xread[TN];
#pragma unroll
  for (int n = 0; n < TN; ++n)
    xread[n] = (trow * kChunks + ((4 * (wn * TN + n) + chunk) ^ ((l16 / 4) << 2))) * 16 + byte;
  // transposed, W is stored as bf16 in the same way, a block's four pieces turned by
  // the block
  const int wrow = tid / kBlocks, wblock = tid % kBlocks;
  int wread[TM];
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    const int b = wm * TM + m;
    wread[m] = (trow * (BM / 8) + ((4 * b + (chunk ^ ((b >> 2) & 3))) ^ ((l16 / 4) << 2))) * 16 +
               byte;
  }

  Raw<T> xr[kPasses];
  Block wr[TR ? 1 : TM], wc[TR ? 1 : TM];
  const T* const x = (const T*)a.x;
  const auto load = [&](int64_t step) {
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
      xr[i] = load_edge(x, a.ldx, step * kStep + i * kRows + xrow, xt, K, a.T);
    if constexpr (TR) {
      wr[0] = load_block(W, nb, step * kStep + wrow, m0 / kMx4Block + wblock);
    } else {
#pragma unroll
      for (int m = 0; m < TM; ++m)
        wr[m] = load_block(W, nb, m0 + (wm * TM + m) * 32 + lane % 32, 2 * step + half);
    }
  };
  const auto store = [&](int buffer) {
    char* const xs = lds + buffer * P * kXBytes;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      uint4 part[P];
      split<T, P>(xr[i], part);
#pragma unroll
      for (int p = 0; p < P; ++p)
        *(uint4*)(xs + p * kXBytes + xstore + i * kRows * kChunks * 16) = part[p];
    }
    if constexpr (TR) {
      char* const ws = lds + 2 * P * kXBytes + buffer * kWBytes;
      const uint32_t words[4] = {wr[0].c.x, wr[0].c.y, wr[0].c.z, wr[0].c.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = (4 * wblock + (i ^ ((wblock >> 2) & 3))) ^ ((wrow & 3) << 2);
        *(uint4*)(ws + (wrow * (BM / 8) + at) * 16) =
            mx4_eight<bf16_t>(words[i], mx4_scale(wr[0].s));
      }
    } else {
#pragma unroll
      for (int m = 0; m < TM; ++m) wc[m] = wr[m];
    }
  };

  f32x16 acc[TM][TN];
#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int n = 0; n < TN; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[m][n][i] = 0.f;

  if (first < last) {
    load(first);
    store(0);
  }
  __syncthreads();
  for (int64_t step = first; step < last; ++step) {
    const int buffer = (int)(step - first) & 1;
    const bool more = step + 1 < last;
    if (more) load(step + 1);
    const char* const xs = lds + buffer * P * kXBytes;
    const char* const ws = lds + 2 * P * kXBytes + buffer * kWBytes;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      bf16x8_t wf[TM];
#pragma unroll
      for (int m = 0; m < TM; ++m) {
        if constexpr (TR) {
          wf[m] = turned(ws + wread[m] + s * 8 * BM * 2, 4 * BM * 2);
        } else {
          const uint32_t words[4] = {wc[m].c.x, wc[m].c.y, wc[m].c.z, wc[m].c.w};
          wf[m] = __builtin_bit_cast(bf16x8_t, mx4_eight<bf16_t>(words[s], mx4_scale(wc[m].s)));
        }
      }
#pragma unroll
      for (int n = 0; n < TN; ++n)
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const bf16x8_t xf = turned(xs + p * kXBytes + xread[n] + s * 8 * BN * 2, 4 * BN * 2);
#pragma unroll
          for (int m = 0; m < TM; ++m)
            acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(xf, wf[m], acc[m][n], 0, 0, 0);
        }
    }
    if (more) store(buffer ^ 1);
    __syncthreads();
  }

#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int n = 0; n < TN; ++n)
      mx4_write<T>(acc[m][n], m0 + (wm * TM + m) * 32, t0 + (wn * TN + n) * 32, M, a.T, a.out, a.ldo,
                   a.part, piece);
}

struct Cut {
  bool large;        // the large tiles
  uint32_t tiles_m, tiles_n;
  int32_t pieces, steps;
};
// Large tiles where they fill half of the GPU; small ones cut along the inner size
// until they fill it too, in pieces of at least four steps.
Cut cut(const Mx4& W, int transposed, int dtype, int64_t T) {
  const int64_t M = transposed ? W.cols : W.rows, K = transposed ? W.rows : W.cols;
  const int64_t steps = cdiv(K, kStep);
  Cut c;
  c.large = dtype != kF32 && cdiv(M, 256) * cdiv(T, dtype == kF16 ? 128 : 256) >= 128;
  c.tiles_m = (uint32_t)cdiv(M, c.large ? 256 : 128);
  c.tiles_n = (uint32_t)cdiv(T, c.large && dtype != kF16 ? 256 : 128);
  const int64_t tiles = (int64_t)c.tiles_m * c.tiles_n;
  int64_t pieces = c.large || tiles >= 256 ? 1 : std::min<int64_t>(512 / tiles, steps / 4);
  pieces = std::max<int64_t>(pieces, 1);
  c.steps = (int32_t)cdiv(steps, pieces);
  c.pieces = (int32_t)cdiv(steps, c.steps);
  return c;
}

template <typename T, bool TR>
void launch(const Mx4MatmulArgs& a, const Cut& c, hipStream_t s) {
  const uint32_t blocks = c.tiles_m * c.tiles_n * (uint32_t)c.pieces;
  if constexpr (sizeof(T) == 2) {
    constexpr int BN = Parts<T>::n == 1 ? 256 : 128;
    if (c.large) {
      mx4_tile_kernel<T, TR, 256, BN, 4, 2><<<blocks, 512, 0, s>>>(a, c.tiles_m, c.tiles_n);
      return;
    }
  }
  mx4_tile_kernel<T, TR, 128, 128, 2, 2><<<blocks, 256, 0, s>>>(a, c.tiles_m, c.tiles_n);
}

template <typename T>
hipError_t matmul(Mx4MatmulArgs a, int transposed, int dtype, hipStream_t s) {
  const Cut c = cut(a.W, transposed, dtype, a.T);
  const int64_t M = transposed ? a.W.cols : a.W.rows;
  a.pieces = c.pieces;
  a.steps = c.steps;
  if (c.pieces == 1) a.part = nullptr;
  if (transposed)
    launch<T, true>(a, c, s);
  else
    launch<T, false>(a, c, s);
  if (c.pieces > 1) return launch_mx4_sum(a.part, c.pieces, M, a.T, a.out, dtype, a.ldo, s);
  return hipGetLastError();
}

}  // namespace

size_t mx4_matmul_bytes(const Mx4& W, int transposed, int dtype, int64_t T) {
  const Cut c = cut(W, transposed, dtype, T);
  if (c.pieces == 1) return 0;
  return (size_t)c.pieces * (size_t)(transposed ? W.cols : W.rows) * (size_t)T * 4;
}

hipError_t launch_mx4_matmul(const Mx4MatmulArgs& a, int transposed, int dtype, hipStream_t s) {
  if (dtype == kF32) return matmul<float>(a, transposed, dtype, s);
  if (dtype == kF16) return matmul<_Float16>(a, transposed, dtype, s);
  return matmul<bf16_t>(a, transposed, dtype, s);
}

}  // namespace spops
