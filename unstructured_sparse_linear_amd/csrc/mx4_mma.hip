// mx4_mma.hip -- product of two 4-bit microscaled matrices, out = W X^T.
//
// W [rows][cols] and X [tokens][cols] both run along the inner size, and
// v_mfma_scale_f32_32x32x64 takes both as they are stored: a lane holds one block of
// one row (row = lane % 32, block = lane / 32) and its scale byte.  Products are
// exact, the sums f32.
#include <algorithm>

#include "kernels.h"
#include "mx4.h"

namespace spops {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kStep = 128;  // k of a step: four blocks

struct Args {
  Mx4 W, X;
  void* out;
  int64_t ldo;
  float* part;
  int32_t steps;
};

__device__ __forceinline__ i32x8 operand(const uint4& c) {
  i32x8 v = {(int)c.x, (int)c.y, (int)c.z, (int)c.w, 0, 0, 0, 0};
  return v;
}

// Block b of row r; past the matrix, zeros.
__device__ __forceinline__ uint4 load_codes(const Mx4& A, int64_t nb, int64_t r, int64_t b) {
  if (r >= A.rows || b >= nb) return make_uint4(0u, 0u, 0u, 0u);
  return *(const uint4*)(A.codes + (r * nb + b) * 16);
}
// Scales of four blocks from b on; past the matrix, ones.
__device__ __forceinline__ uint32_t load_scales(const Mx4& A, int64_t nb, int64_t r, int64_t b) {
  uint32_t w = 0x7f7f7f7fu;
  if (r >= A.rows) return w;
  const uint8_t* const p = A.scales + r * nb + b;
  if (b + 4 <= nb) {
    __builtin_memcpy(&w, p, 4);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (b + i < nb) w = (w & ~(0xffu << (8 * i))) | ((uint32_t)p[i] << (8 * i));
  }
  return w;
}

// BM rows x BN tokens; WM x WN waves.
template <typename T, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void mx4_mma_kernel(Args a, uint32_t tiles_m,
                                                                  uint32_t tiles_n) {
  constexpr int kThreads = 64 * WM * WN, kRows = kThreads / 4;
  constexpr int TM = BM / WM / 32, TN = BN / WN / 32;
  static_assert(BM % kRows == 0 && BN % kRows == 0 && BM + BN <= kThreads, "whole passes");
  constexpr int kStage = (BM + BN) * 68;  // codes, then scales
  __shared__ __attribute__((aligned(16))) char lds[2 * kStage];

  const int64_t nb = (a.W.cols + kMx4Block - 1) / kMx4Block;
  const uint32_t index = xcd_index(blockIdx.x, gridDim.x);
  const uint32_t tile = index % (tiles_m * tiles_n), piece = index / (tiles_m * tiles_n);
  const uint32_t band = tile / (4 * tiles_m), in = tile % (4 * tiles_m);
  const uint32_t wide = min(4u, tiles_n - 4 * band);
  const int64_t m0 = (int64_t)(in / wide) * BM, t0 = (int64_t)(4 * band + in % wide) * BN;
  const int64_t first = (int64_t)piece * a.steps;
  const int64_t last = min(first + a.steps, (a.W.cols + kStep - 1) / kStep);

  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int wm = wave / WN, wn = wave % WN, half = lane / 32;
  // rows of four blocks, turned by the row, so that 16 rows read at once lie in
  // different banks
  const int srow = tid / 4, sblock = tid % 4;
  uint4 wr[BM / kRows], xr[BN / kRows];
  uint32_t sr = 0;
  const auto load = [&](int64_t step) {
#pragma unroll
    for (int i = 0; i < BM / kRows; ++i)
      wr[i] = load_codes(a.W, nb, m0 + i * kRows + srow, 4 * step + sblock);
#pragma unroll
    for (int i = 0; i < BN / kRows; ++i)
      xr[i] = load_codes(a.X, nb, t0 + i * kRows + srow, 4 * step + sblock);
    if (tid < BM)
      sr = load_scales(a.W, nb, m0 + tid, 4 * step);
    else if (tid < BM + BN)
      sr = load_scales(a.X, nb, t0 + tid - BM, 4 * step);
  };
  const auto store = [&](int buffer) {
    char* const s = lds + buffer * kStage;
#pragma unroll
    for (int i = 0; i < BM / kRows; ++i) {
      const int r = i * kRows + srow;
      *(uint4*)(s + r * 64 + 16 * (sblock ^ ((r >> 2) & 3))) = wr[i];
    }
#pragma unroll
    for (int i = 0; i < BN / kRows; ++i) {
      const int r = BM + i * kRows + srow;
      *(uint4*)(s + r * 64 + 16 * (sblock ^ ((r >> 2) & 3))) = xr[i];
    }
    if (tid < BM + BN) *(uint32_t*)(s + (BM + BN) * 64 + tid * 4) = sr;
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
    const char* const s = lds + buffer * kStage;
    int ws[TM], xs[TN];
#pragma unroll
    for (int m = 0; m < TM; ++m)
      ws[m] = *(const int*)(s + (BM + BN) * 64 + ((wm * TM + m) * 32 + lane % 32) * 4) >> (8 * half);
#pragma unroll
    for (int n = 0; n < TN; ++n)
      xs[n] = *(const int*)(s + (BM + BN) * 64 + (BM + (wn * TN + n) * 32 + lane % 32) * 4) >>
              (8 * half);
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      uint4 wf[TM], xf[TN];
#pragma unroll
      for (int m = 0; m < TM; ++m) {
        const int r = (wm * TM + m) * 32 + lane % 32;
        wf[m] = *(const uint4*)(s + r * 64 + 16 * ((2 * sub + half) ^ ((r >> 2) & 3)));
      }
#pragma unroll
      for (int n = 0; n < TN; ++n) {
        const int r = BM + (wn * TN + n) * 32 + lane % 32;
        xf[n] = *(const uint4*)(s + r * 64 + 16 * ((2 * sub + half) ^ ((r >> 2) & 3)));
      }
#pragma unroll
      for (int n = 0; n < TN; ++n)
#pragma unroll
        for (int m = 0; m < TM; ++m)
          acc[m][n] = sub == 0 ? __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                                     operand(xf[n]), operand(wf[m]), acc[m][n], 4, 4, 0, xs[n], 0,
                                     ws[m])
                               : __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                                     operand(xf[n]), operand(wf[m]), acc[m][n], 4, 4, 2, xs[n], 2,
                                     ws[m]);
    }
    if (more) store(buffer ^ 1);
    __syncthreads();
  }
#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int n = 0; n < TN; ++n)
      mx4_write<T>(acc[m][n], m0 + (wm * TM + m) * 32, t0 + (wn * TN + n) * 32, a.W.rows, a.X.rows,
                   a.out, a.ldo, a.part, piece);
}

struct Cut {
  bool large;
  uint32_t tiles_m, tiles_n;
  int32_t pieces, steps;
};
// Large tiles where they fill half of the GPU; small ones cut along the inner size
// until they fill it too, in pieces of at least four steps.
Cut cut(const Mx4& W, int64_t T) {
  const int64_t steps = cdiv(W.cols, kStep);
  Cut c;
  c.large = cdiv(W.rows, 256) * cdiv(T, 256) >= 128;
  const int64_t side = c.large ? 256 : 128;
  c.tiles_m = (uint32_t)cdiv(W.rows, side);
  c.tiles_n = (uint32_t)cdiv(T, side);
  const int64_t tiles = (int64_t)c.tiles_m * c.tiles_n;
  int64_t pieces = c.large || tiles >= 256 ? 1 : std::min<int64_t>(512 / tiles, steps / 4);
  pieces = std::max<int64_t>(pieces, 1);
  c.steps = (int32_t)cdiv(steps, pieces);
  c.pieces = (int32_t)cdiv(steps, c.steps);
  return c;
}

template <typename T>
hipError_t matmul4(Args a, const Cut& c, int dtype, hipStream_t s) {
  const uint32_t blocks = c.tiles_m * c.tiles_n * (uint32_t)c.pieces;
  if (c.large)
    mx4_mma_kernel<T, 256, 256, 4, 2><<<blocks, 512, 0, s>>>(a, c.tiles_m, c.tiles_n);
  else
    mx4_mma_kernel<T, 128, 128, 2, 2><<<blocks, 256, 0, s>>>(a, c.tiles_m, c.tiles_n);
  if (c.pieces > 1)
    return launch_mx4_sum(a.part, c.pieces, a.W.rows, a.X.rows, a.out, dtype, a.ldo, s);
  return hipGetLastError();
}

}  // namespace

size_t mx4_matmul4_bytes(const Mx4& W, int64_t T) {
  const Cut c = cut(W, T);
  return c.pieces == 1 ? 0 : (size_t)c.pieces * (size_t)W.rows * (size_t)T * 4;
}

hipError_t launch_mx4_matmul4(const Mx4& W, const Mx4& X, void* out, int dtype, int64_t ldo,
                              void* ws, hipStream_t s) {
  const Cut c = cut(W, X.rows);
  const Args a{W, X, out, ldo, c.pieces > 1 ? (float*)ws : nullptr, c.steps};
  if (dtype == kF32) return matmul4<float>(a, c, dtype, s);
  if (dtype == kF16) return matmul4<_Float16>(a, c, dtype, s);
  return matmul4<bf16_t>(a, c, dtype, s);
}

}  // namespace spops
