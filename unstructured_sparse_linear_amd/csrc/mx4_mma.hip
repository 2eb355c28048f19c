// mx4_mma.hip -- product of two 4-bit microscaled matrices, out = W X^T.
//
// W [rows][cols] and X [tokens][cols] both run along the inner size, and
// v_mfma_scale_f32_32x32x64 takes both as they are stored: a lane holds one block of
// one row (row = lane % 32, block = lane / 32) and its scale byte.  Products are
// exact, the sums f32.
//
// A step of 256 k takes whole lines (128 bytes) of each row's codes through shared
// memory, and scales come for two steps at a time.  8192 tokens, 4096 -> 11008, bf16 out:
// 290 us, 2.5 PFLOP/s (the matrix cores reach 6.0 on random operands, and are busy for
// 26% of the cycles): one workgroup a compute unit, whose steps are a few hundred clocks
// between barriers and whose output nothing overlaps.  Bytes do not bound it (1.5 GB from
// the L2s, 64 us at their 24 TB/s).  300 tokens, 4096 x 4096: 15.4 us, bound by the chain
// of a tile's steps.
#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "mx4.h"

namespace spops {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kStep = 256;           // k of a step: eight blocks, 128 bytes of a row
constexpr int kBlocks = kStep / 32;

struct Args {
  Mx4 W, X;
  void* out;
  int64_t ldo;
  float* part;
};

__device__ __forceinline__ i32x8 operand(const u32x4& c) {
  i32x8 v = {(int)c[0], (int)c[1], (int)c[2], (int)c[3], 0, 0, 0, 0};
  return v;
}

// BM rows x BN tokens; KG groups of WM x WN waves, each with a part of the steps and shared
// memory of its own.
template <typename T, int BM, int BN, int WM, int WN, int KG>
__global__ __launch_bounds__(64 * WM * WN * KG, 2) void mx4_mma_kernel(Args a, Mx4Cut cut) {
  constexpr int kThreads = 64 * WM * WN, kRows = BM + BN, kLoads = kRows * kBlocks / kThreads;
  constexpr int TM = BM / WM / 32, TN = BN / WN / 32;
  static_assert(kRows == kThreads && BM % 64 == 0, "a row of scales a thread, waves of one matrix");
  constexpr int kCodes = kRows * 128, kScales = kRows * 16;
  static_assert(BM * kBlocks % kThreads == 0 &&
                    WM * WN * kWriteBytes <= 2 * (kCodes + kScales),
                "whole loads of each matrix, room for the output");
  constexpr int kGroupBytes = 2 * (kCodes + kScales);
  static_assert(KG == 1 || BM * BN * 4 <= kGroupBytes, "room for the sums");
  __shared__ __attribute__((aligned(16))) char all[KG * kGroupBytes];

  const int64_t nb = (a.W.cols + kMx4Block - 1) / kMx4Block;
  const Mx4Place place = mx4_place(cut, blockIdx.x);
  const int64_t m0 = (int64_t)place.m * BM, t0 = (int64_t)place.n * BN;
  const int64_t steps = (nb + kBlocks - 1) / kBlocks;
  const int64_t from = place.cut ? (int64_t)place.piece * cut.steps : 0;
  const int64_t to = place.cut ? min(from + cut.steps, steps) : steps;
  const int group = KG == 1 ? 0 : wave_uniform((int)threadIdx.x / kThreads);
  const int64_t each = KG == 1 ? to - from : (to - from + KG - 1) / KG;
  const int64_t first = from + group * each, last = min(first + each, to);
  char* const lds = all + group * kGroupBytes;
  const int64_t rest = cut.tiles_m * cut.tiles_n - cut.whole;
  float* const part =
      place.cut ? a.part + (place.piece * rest + place.rest) * (BM * BN) : nullptr;

  const int tid = (int)threadIdx.x % kThreads, lane = tid % 64, wave = tid / 64;
  const int wm = wave / WN, wn = wave % WN, half = lane / 32;
  // a row's eight blocks are turned by the row, so that 16 rows read at once lie in
  // different banks
  int wread[TM], xread[TN];
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    const int r = (wm * TM + m) * 32 + lane % 32;
    wread[m] = r * 128 + 16 * (half ^ ((r >> 1) & 7));
  }
#pragma unroll
  for (int n = 0; n < TN; ++n) {
    const int r = BM + (wn * TN + n) * 32 + lane % 32;
    xread[n] = r * 128 + 16 * (half ^ ((r >> 1) & 7));
  }

  // Rows and blocks past the last read it again: what the rows give is not written, and
  // the blocks are stored as zeros of scale one.
  const int block = tid % kBlocks;
  u32x4 codes[kLoads], scales;
  const auto load = [&](int64_t step) {
    const int64_t b = min(kBlocks * step + block, nb - 1);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const Mx4& A = i < BM * kBlocks / kThreads ? a.W : a.X;
      const int r = (tid + i * kThreads) / kBlocks;
      const int64_t row = min(i < BM * kBlocks / kThreads ? m0 + r : t0 + r - BM, A.rows - 1);
      codes[i] = *(const u32x4*)(A.codes + (row * nb + b) * 16);
    }
  };
  // scales of two steps
  const Mx4& mine_of = tid < BM ? a.W : a.X;
  const uint8_t* const my_scales =
      mine_of.scales + min(tid < BM ? m0 + tid : t0 + tid - BM, mine_of.rows - 1) * nb;
  const auto load_scales = [&](int64_t step) {
    const int64_t b = kBlocks * step;
    if (b + 16 <= nb) {
      typedef uint32_t bytes16 __attribute__((ext_vector_type(4), aligned(1)));
      scales = *(const bytes16*)(my_scales + b);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w = 0x7f7f7f7fu;
#pragma unroll 1
        for (int j = 0; j < 4 && b + 4 * i + j < nb; ++j)
          w = (w & ~(0xffu << (8 * j))) | ((uint32_t)my_scales[b + 4 * i + j] << (8 * j));
        scales[i] = w;
      }
    }
  };
  const auto store = [&](int64_t step) {
    char* const to = lds + ((int)(step - first) & 1) * kCodes;
    const uint32_t keep = kBlocks * step + block < nb ? ~0u : 0u;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int r = (tid + i * kThreads) / kBlocks;
      *(u32x4*)(to + r * 128 + 16 * (block ^ ((r >> 1) & 7))) = codes[i] & keep;
    }
  };
  const auto store_scales = [&](int64_t step) {
    *(u32x4*)(lds + 2 * kCodes + ((int)(step - first) >> 1 & 1) * kScales + tid * 16) = scales;
  };

  f32x16 acc[TM][TN];
#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int n = 0; n < TN; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[m][n][i] = 0.f;

  // One step; U: whether it is the second of a pair.
  const auto products = [&](int64_t step, auto second) {
    constexpr int U = decltype(second)::value;
    const char* const c = lds + ((int)(step - first) & 1) * kCodes;
    const char* const s = lds + 2 * kCodes + ((int)(step - first) >> 1 & 1) * kScales + 8 * U;
    int ws[TM][2], xs[TN][2];
#pragma unroll
    for (int m = 0; m < TM; ++m) {
      const uint2 v = *(const uint2*)(s + ((wm * TM + m) * 32 + lane % 32) * 16);
      ws[m][0] = (int)(v.x >> (8 * half)), ws[m][1] = (int)(v.y >> (8 * half));
    }
#pragma unroll
    for (int n = 0; n < TN; ++n) {
      const uint2 v = *(const uint2*)(s + (BM + (wn * TN + n) * 32 + lane % 32) * 16);
      xs[n][0] = (int)(v.x >> (8 * half)), xs[n][1] = (int)(v.y >> (8 * half));
    }
#pragma unroll
    for (int sub = 0; sub < 4; ++sub) {
      u32x4 wf[TM], xf[TN];
#pragma unroll
      for (int m = 0; m < TM; ++m) wf[m] = *(const u32x4*)(c + (wread[m] ^ (32 * sub)));
#pragma unroll
      for (int n = 0; n < TN; ++n) xf[n] = *(const u32x4*)(c + (xread[n] ^ (32 * sub)));
#pragma unroll
      for (int n = 0; n < TN; ++n)
#pragma unroll
        for (int m = 0; m < TM; ++m)
          acc[m][n] = sub % 2 == 0
                          ? __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                                operand(xf[n]), operand(wf[m]), acc[m][n], 4, 4, 0, xs[n][sub / 2],
                                0, ws[m][sub / 2])
                          : __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                                operand(xf[n]), operand(wf[m]), acc[m][n], 4, 4, 2, xs[n][sub / 2],
                                2, ws[m][sub / 2]);
    }
  };

  // A step is made while the next one's loads come; loads past the last step are not
  // used.  (The scheduling barriers keep the loads before the products: below them they
  // would be waited for.  Loads two steps ahead were no faster.)
  if (first < last) {
    load(first);
    load_scales(first);
    store(first);
    store_scales(first);
  }
  __syncthreads();
  for (int64_t step = first; step < first + each; step += 2) {
    load(step + 1);
    if (step + 2 < last) load_scales(step + 2);
    __builtin_amdgcn_sched_barrier(0);
    if (KG == 1 || step < last) products(step, std::integral_constant<int, 0>());
    store(step + 1);
    __syncthreads();
    load(step + 2);
    __builtin_amdgcn_sched_barrier(0);
    if (step + 1 < last) products(step + 1, std::integral_constant<int, 1>());
    store(step + 2);
    store_scales(step + 2);
    __syncthreads();
  }
  // (every wave is past the last step's barrier)
  if constexpr (KG > 1) {
    const auto at = [&](int g, int m, int n, int i) {
      return (f32x4*)(all + g * kGroupBytes) +
             (((m * TN + n) * 4 + i) * WM * WN + wave) * 64 + lane;
    };
    if (group > 0) {
#pragma unroll
      for (int m = 0; m < TM; ++m)
#pragma unroll
        for (int n = 0; n < TN; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *at(group, m, n, i) = (f32x4){acc[m][n][4 * i], acc[m][n][4 * i + 1],
                                          acc[m][n][4 * i + 2], acc[m][n][4 * i + 3]};
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 1; g < KG; ++g)
#pragma unroll
      for (int m = 0; m < TM; ++m)
#pragma unroll
        for (int n = 0; n < TN; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f32x4 v = *at(g, m, n, i);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[m][n][4 * i + j] += v[j];
          }
  }
  char* const mine = lds + wave * kWriteBytes;
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    const int64_t r = (wm * TM + m) * 32, t = wn * TN * 32;
    if (part)
      mx4_write(acc[m], mine, r, t, a.W.rows - m0, a.X.rows - t0, part, BN);
    else
      mx4_write(acc[m], mine, m0 + r, t0 + t, a.W.rows, a.X.rows, (T*)a.out, a.ldo);
  }
}

struct Cut : Mx4Cut {
  int side;
};
// Tiles of 256, 128 or 64 square, the largest that fill the GPU (4096 x 4096, 2560
// tokens: 43.5 us with 256, 46.0 with 128; 2048: 51.9 and 31.5; 1024: 22.2 with 128, 26.7
// with 64; 640: 20.9 and 22.2; 512: 21.9 and 15.1; 128: 13.4 and 11.0); few small ones are
// cut along the inner size, in pieces of at least four steps, which two groups of waves
// make (64 tokens: 9.0 us, 10.3 in pieces for four groups).
Cut cut(const Mx4& W, int64_t T) {
  const int64_t steps = cdiv(W.cols, kStep);
  Cut c;
  c.side = 64;
  if (cdiv(W.rows, 128) * cdiv(T, 128) >= 256) c.side = 128;
  if (cdiv(W.rows, 256) * cdiv(T, 256) >= 160) c.side = 256;
  c.tiles_m = (uint32_t)cdiv(W.rows, c.side);
  c.tiles_n = (uint32_t)cdiv(T, c.side);
  const int64_t tiles = (int64_t)c.tiles_m * c.tiles_n;
  const int64_t pieces = std::max<int64_t>(1, std::min<int64_t>(256 / tiles, steps / 4));
  c.whole = (uint32_t)(pieces > 1 ? 0 : tiles);
  c.steps = (int32_t)cdiv(steps, pieces);
  c.pieces = (uint32_t)cdiv(steps, c.steps);
  return c;
}

template <typename T>
hipError_t matmul4(const Args& a, const Cut& c, int dtype, hipStream_t s) {
  const uint32_t blocks = mx4_blocks(c);
  if (c.side == 256)
    mx4_mma_kernel<T, 256, 256, 4, 2, 1><<<blocks, 512, 0, s>>>(a, c);
  else if (c.side == 128)
    mx4_mma_kernel<T, 128, 128, 2, 2, 1><<<blocks, 256, 0, s>>>(a, c);
  else if (c.steps >= 4)
    // two waves a tile leave its steps one after the other: two groups of them 15.4 us for
    // 300 tokens, 4096 x 4096, one 18.4, four (a workgroup a compute unit) 21.1; of 512 x
    // 512 x 512, two steps, one 4.4 us, two 5.9
    mx4_mma_kernel<T, 64, 64, 2, 1, 2><<<blocks, 256, 0, s>>>(a, c);
  else
    mx4_mma_kernel<T, 64, 64, 2, 1, 1><<<blocks, 128, 0, s>>>(a, c);
  if (c.whole < c.tiles_m * c.tiles_n)
    return launch_mx4_sum(a.part, c, c.side, c.side, a.W.rows, a.X.rows, a.out, dtype, a.ldo, s);
  return hipGetLastError();
}

}  // namespace

size_t mx4_matmul4_bytes(const Mx4& W, int64_t T) {
  const Cut c = cut(W, T);
  return mx4_part_bytes(c, c.side, c.side);
}

hipError_t launch_mx4_matmul4(const Mx4& W, const Mx4& X, void* out, int dtype, int64_t ldo,
                              void* ws, hipStream_t s) {
  const Cut c = cut(W, X.rows);
  const Args a{W, X, out, ldo, (float*)ws};
  if (dtype == kF32) return matmul4<float>(a, c, dtype, s);
  if (dtype == kF16) return matmul4<_Float16>(a, c, dtype, s);
  return matmul4<bf16_t>(a, c, dtype, s);
}

}  // namespace spops
