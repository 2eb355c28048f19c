// mx4_matmul.hip -- products of a 4-bit microscaled matrix W with dense activations.
//
//   out = W x    (x [cols][T], out [rows][T]),
//   out = W^T x  (x [rows][T], out [cols][T], the gradient of the input).
//
// An element of W times its scale has two significant bits, so bf16 holds it and its
// product with a bf16 value is exact in f32.  x of f32 is cut into three bf16 parts
// of eight bits each, which loses nothing (of values under 2^-109 the bits below
// 2^-133, the smallest bf16).  f16 holds the elements of the scales 104 to 140: with x
// of f16 a workgroup first looks its scales through (32 KB of a tile of 256 x 4096) and
// runs on f16, or, where others are among them, on bf16 with x in two parts.  So every
// product is exact, and the sums are f32.  Eight consecutive elements of the inner size (k)
// feed one half of v_mfma_f32_32x32x16_bf16 (row = lane % 32, half = lane / 32).
//
// A workgroup makes BM rows x BN tokens in steps of 64 k.  In a step, half h holds
// the elements 32 h + 8 s + j of instruction s, so that 16 bytes of W are one block of
// one row, with one scale, for four instructions.  x goes through shared memory as it
// lies (rows of k) and is read turned; W goes through it as codes, two steps (64 bytes
// a row) at a time, and is converted where it is used.  (Read by each lane for itself,
// 16 bytes of 32 rows at a time, W took lines of the L1 four times over: 4096 x 4096,
// 1024 tokens 65 us, so 52.)  W^T x converts W into shared memory and reads it turned.
//
// Bound by the matrix cores at the clock that their power leaves: with operands of
// random bits they reach 1.69 PFLOP/s and no more.  8192 tokens, 4096 -> 11008, bf16:
// 643 us, 1.15 PFLOP/s (a library's dense bf16 product of that size 701); gradient of
// 4096 tokens, 4096 x 4096: 118 us, 1.16.
#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "mx4.h"

namespace spops {
namespace {

constexpr int kStep = 64;

// One tile, and the steps of its inner size; part: where the sums of a tile in pieces go.
struct Tile {
  int64_t m0, t0, first, last;
  float* part;
  int bn;  // its row
};
// F: on f16.  SB: x in a single buffer.
template <typename T, bool F>
constexpr int kParts = sizeof(T) == 4 ? 3 : __is_same(T, _Float16) && !F ? 2 : 1;
template <typename T, bool TR, int BM, int BN, bool F, bool SB>
constexpr int kTileBytes = (SB ? 1 : 2) * kParts<T, F> * BN * 2 * kStep +
                           2 * BM * (TR ? 2 * kStep : 4 * 16 + 4);

template <typename T, bool TR, int BM, int BN, int WM, int WN, bool F, bool SB>
__device__ __forceinline__ void tile_product(const Mx4MatmulArgs& a, const Tile& tile, char* lds) {
  constexpr int P = kParts<T, F>, kThreads = 64 * WM * WN;
  constexpr int TM = BM / WM / 32, TN = BN / WN / 32;
  constexpr int kChunks = BN / 8, kRows = kThreads / kChunks, kPasses = kStep / kRows;
  constexpr int kXBytes = kStep * BN * 2;
  constexpr int kBlocks = BM / 32;  // of a row of W, transposed
  // W in shared memory: transposed a step as 16-bit values, otherwise two steps as they
  // are, 64 bytes of codes and 4 scales a row
  constexpr int kWBytes = TR ? kStep * BM * 2 : BM * 68;
  constexpr int kW = TR ? 1 : BM * 4 / kThreads;  // loads of codes
  // transposed, a block a thread, of the first threads
  constexpr int kLoaders = kStep * kBlocks;
  static_assert(!TR || kThreads >= kLoaders, "a block a thread");
  static_assert(WM * WN * kWriteBytes <= kTileBytes<T, TR, BM, BN, F, SB>, "room for output");
  static_assert(TR || (BM * 4 % kThreads == 0 && BM <= kThreads), "whole loads");
  using E = std::conditional_t<F, _Float16, bf16_t>;

  const Mx4 W = a.W;
  const int64_t nb = (W.cols + kMx4Block - 1) / kMx4Block;
  const int64_t M = TR ? W.cols : W.rows, K = TR ? W.rows : W.cols;
  const int64_t m0 = tile.m0, t0 = tile.t0, first = tile.first, last = tile.last;
  char* const wlds = lds + (SB ? 1 : 2) * P * kXBytes;

  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int wm = wave / WN, wn = wave % WN, half = lane / 32;
  // x is stored with the 64-byte groups of a row turned by the row, so that the four
  // rows that are read at once lie in different banks
  const int xrow = tid / kChunks, xchunk = tid % kChunks;
  const int xstore = (xrow * kChunks + (xchunk ^ ((xrow & 3) << 2))) * 16;
  const int l16 = lane % 16, sub = (lane / 16) % 2;
  const int chunk = 2 * sub + (l16 % 4) / 2, byte = 8 * (l16 & 1), trow = 32 * half + l16 / 4;
  int xread[TN];
#pragma unroll
  for (int n = 0; n < TN; ++n)
    xread[n] = (trow * kChunks + ((4 * (wn * TN + n) + chunk) ^ ((l16 / 4) << 2))) * 16 + byte;
  // transposed, W is stored in the same way, a block's four pieces turned by the block;
  // otherwise a row's four blocks are turned by the row, for the 16 rows read at once
  const int wrow = tid / kBlocks, wblock = tid % kBlocks;
  int wread[TM];
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    const int b = wm * TM + m, r = 32 * b + lane % 32;
    wread[m] = TR ? (trow * (BM / 8) + ((4 * b + (chunk ^ ((b >> 2) & 3))) ^ ((l16 / 4) << 2))) *
                            16 + byte
                  : r * 64 + 16 * (half ^ ((r >> 2) & 3));
  }

  const T* const x = (const T*)a.x;
  const int64_t end = (K - 1) * a.ldx + a.T;  // of x
  const int64_t xlane = xrow * a.ldx + 8 * xchunk;
  // transposed, small tiles of 16 bits load two steps ahead (gradient of 1024 tokens,
  // 4096 x 4096: 49.4 us, 55.1 one ahead; no faster where W comes for two steps anyhow,
  // nor on large tiles)
  constexpr bool kTwo = TR && BM == 128 && sizeof(T) == 2 && !SB;
  Raw<T> xr[1 + kTwo][kPasses];
  // Nothing in a load looks at what another brings, so that they come while the step
  // before is made.  Inside: every load of the step lies inside x (tokens past the last
  // may hold anything, as their columns are not written).  Rows that start between two
  // words are loaded as they are: words from the one before on, shifted when they are
  // stored, took longer (f16, 2011 tokens, 4090 -> 4097: 98.7 us, 91.5 so).
  const auto load_x = [&](int64_t step, auto inside, int to = 0) {
    const int64_t at = step * kStep * a.ldx + t0;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      if constexpr (decltype(inside)::value) {
        __builtin_memcpy(&xr[to][i], x + at + i * kRows * a.ldx + xlane, sizeof(xr[to][i]));
      } else {
        const int64_t k = step * kStep + i * kRows + xrow, t = t0 + 8 * xchunk;
        xr[to][i] = load_until(x, k * a.ldx + t, k < K && t < a.T ? end : 0);
      }
    }
  };
  // the steps up to here lie inside
  const int64_t room = end - BN - t0 - (kStep - 1) * a.ldx;
  const int64_t inside_end = room < 0 ? 0 : room / (kStep * a.ldx) + 1;
  const auto load_x_any = [&](int64_t step) {
    if (step < inside_end)
      load_x(step, std::true_type());
    else
      load_x(step, std::false_type());
  };
  const auto store_x = [&](int64_t step, int from = 0) {
    char* const xs = lds + (SB ? 0 : (int)(step - first) & 1) * P * kXBytes;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      uint4 part[P];
      split<T, P>(xr[from][i], part);
#pragma unroll
      for (int p = 0; p < P; ++p)
        *(uint4*)(xs + p * kXBytes + xstore + i * kRows * kChunks * 16) = part[p];
    }
  };

  // W of one step (transposed) or of two.  Rows and blocks past the last read the last
  // again: what they give meets zeros of x, for which scales past the inner size are
  // made finite, or is not written.
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  u32x4 wr[1 + kTwo][kW];
  uint32_t ws[1 + kTwo] = {};
  const auto load_w = [&](int64_t step, auto inside, int into = 0) {
    constexpr bool I = decltype(inside)::value;
    if constexpr (TR) {
      if (kThreads > kLoaders && tid >= kLoaders) return;
      const int64_t r = step * kStep + wrow;
      const int64_t at = (I ? r : min(r, W.rows - 1)) * nb + min(m0 / kMx4Block + wblock, nb - 1);
      wr[into][0] = *(const u32x4*)(W.codes + at * 16);
      ws[into] = W.scales[at];
    } else {
#pragma unroll
      for (int i = 0; i < kW; ++i) {
        const int id = tid + i * kThreads;
        const int64_t r = min(m0 + id / 4, W.rows - 1), b = 2 * step + id % 4;
        wr[into][i] = *(const u32x4*)(W.codes + (r * nb + (I ? b : min(b, nb - 1))) * 16);
      }
      if (BM == kThreads || tid < BM) {
        const uint8_t* const p = W.scales + min(m0 + tid, W.rows - 1) * nb + 2 * step;
        if constexpr (I) {
          typedef uint32_t word __attribute__((aligned(1)));
          ws[into] = *(const word*)p;
        } else {
          uint32_t w = 0x7f7f7f7fu;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (2 * step + i < nb) w = (w & ~(0xffu << (8 * i))) | ((uint32_t)p[i] << (8 * i));
          ws[into] = w;
        }
      }
    }
  };
  // the steps up to here lie inside x and W, and so do the loads of W that go with them
  const int64_t hot_end =
      min(min(last, inside_end), TR ? last : nb < 4 ? 0 : (nb - 4) / 2 + 1);
  const auto store_w = [&](int64_t step, int from = 0) {
    char* const to = wlds + ((int)(step - first) >> (TR ? 0 : 1) & 1) * kWBytes;
    if constexpr (TR) {
      if (kThreads > kLoaders && tid >= kLoaders) return;
      const float scale = mx4_scale(step * kStep + wrow < W.rows ? ws[from] : 127u);
      const u32x4 c = wr[from][0];
      const uint32_t words[4] = {c[0], c[1], c[2], c[3]};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = (4 * wblock + (i ^ ((wblock >> 2) & 3))) ^ ((wrow & 3) << 2);
        *(uint4*)(to + (wrow * (BM / 8) + at) * 16) = mx4_eight<E>(words[i], scale);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kW; ++i) {
        const int id = tid + i * kThreads, r = id / 4;
        *(u32x4*)(to + r * 64 + 16 * ((id % 4) ^ ((r >> 2) & 3))) = wr[from][i];
      }
      if (BM == kThreads || tid < BM) *(uint32_t*)(to + BM * 64 + tid * 4) = ws[from];
    }
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
    const int at = (int)(step - first);
    const char* const xs = lds + (SB ? 0 : at & 1) * P * kXBytes;
    const char* const wl = wlds + (TR ? at & 1 : at >> 1 & 1) * kWBytes;
    uint4 wc[TM];
    float scale[TM];
    if constexpr (!TR) {
#pragma unroll
      for (int m = 0; m < TM; ++m) {
        wc[m] = *(const uint4*)(wl + (wread[m] ^ (32 * U)));
        const uint32_t s4 =
            *(const uint32_t*)(wl + BM * 64 + ((wm * TM + m) * 32 + lane % 32) * 4);
        scale[m] = mx4_scale((s4 >> (16 * U + 8 * half)) & 0xffu);
      }
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      bf16x8_t wf[TM];
#pragma unroll
      for (int m = 0; m < TM; ++m) {
        if constexpr (TR) {
          wf[m] = turned(wl + wread[m] + s * 8 * BM * 2, 4 * BM * 2);
        } else {
          const uint32_t words[4] = {wc[m].x, wc[m].y, wc[m].z, wc[m].w};
          wf[m] = __builtin_bit_cast(bf16x8_t, mx4_eight<E>(words[s], scale[m]));
        }
      }
#pragma unroll
      for (int n = 0; n < TN; ++n)
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const bf16x8_t xf = turned(xs + p * kXBytes + xread[n] + s * 8 * BN * 2, 4 * BN * 2);
#pragma unroll
          for (int m = 0; m < TM; ++m)
            acc[m][n] = F ? __builtin_amdgcn_mfma_f32_32x32x16_f16(
                                __builtin_bit_cast(f16x8_t, xf),
                                __builtin_bit_cast(f16x8_t, wf[m]), acc[m][n], 0, 0, 0)
                          : __builtin_amdgcn_mfma_f32_32x32x16_bf16(xf, wf[m], acc[m][n], 0, 0, 0);
        }
    }
  };

  // A step is made while the next one's loads come.  (The scheduling barriers keep the
  // loads before the products: below them they would be waited for.)
  int64_t step = first;
  if (step < last) {
    load_w(step, std::false_type());
    load_x_any(step);
    store_w(step);
    store_x(step);
  }
  __syncthreads();
  if constexpr (kTwo) {
    // (step + 1 is on its way already)
    if (step + 3 < hot_end) {
      load_x(step + 1, std::true_type(), 1);
      load_w(step + 1, std::true_type(), 1);
    }
    for (; step + 3 < hot_end; step += 2) {
      load_x(step + 2, std::true_type());
      load_w(step + 2, std::true_type());
      __builtin_amdgcn_sched_barrier(0);
      products(step, std::integral_constant<int, 0>());
      store_x(step + 1, 1);
      store_w(step + 1, 1);
      __syncthreads();
      load_x(step + 3, std::true_type(), 1);
      load_w(step + 3, std::true_type(), 1);
      __builtin_amdgcn_sched_barrier(0);
      products(step + 1, std::integral_constant<int, 1>());
      store_x(step + 2);
      store_w(step + 2);
      __syncthreads();
    }
  } else if constexpr (!SB) {
    for (; step + 2 < hot_end; step += 2) {
      load_x(step + 1, std::true_type());
      load_w(step + (TR ? 1 : 2), std::true_type());
      __builtin_amdgcn_sched_barrier(0);
      products(step, std::integral_constant<int, 0>());
      store_x(step + 1);
      if constexpr (TR) store_w(step + 1);
      __syncthreads();
      load_x(step + 2, std::true_type());
      if constexpr (TR) load_w(step + 2, std::true_type());
      __builtin_amdgcn_sched_barrier(0);
      products(step + 1, std::integral_constant<int, 1>());
      store_x(step + 2);
      store_w(step + 2);
      __syncthreads();
    }
  }
  const auto next = [&](int64_t to, bool w) {
    if (to >= last) return;
    if (SB) load_x_any(to);
    if (SB) __syncthreads();
    store_x(to);
    if (w) store_w(to);
  };
  for (; step < last; step += 2) {
    if (!SB && step + 1 < last) load_x_any(step + 1);
    if (step + 1 < last) load_w(step + (TR ? 1 : 2), std::false_type());
    products(step, std::integral_constant<int, 0>());
    next(step + 1, TR);
    __syncthreads();
    if (step + 1 >= last) break;
    if (!SB && step + 2 < last) load_x_any(step + 2);
    if (TR && step + 2 < last) load_w(step + 2, std::false_type());
    products(step + 1, std::integral_constant<int, 1>());
    next(step + 2, true);
    __syncthreads();
  }

  // (every wave is past the last step's barrier)
  char* const mine = lds + wave * kWriteBytes;
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    const int64_t r = (wm * TM + m) * 32, t = wn * TN * 32;
    if (tile.part)
      mx4_write(acc[m], mine, r, t, M - m0, a.T - t0, tile.part, tile.bn);
    else
      mx4_write(acc[m], mine, m0 + r, t0 + t, M, a.T, (T*)a.out, a.ldo);
  }
}

// Whether any of `n` scales of `rows` rows from p on, `ld` apart, is one that f16 does
// not hold.  Four to a word: those under 128 have to be 104 at least, the others 140 at
// most.
template <int THREADS>
__device__ __forceinline__ bool wide_scales(const uint8_t* p, int64_t rows, int64_t n, int64_t ld) {
  const auto outside = [](uint32_t w) {
    const uint32_t low = (w | 0x80808080u) - 0x68686868u, high = (w | 0x80808080u) - 0x0d0d0d0du;
    return ((~w & ~low) | (w & high)) & 0x80808080u;
  };
  uint32_t bad = 0;
  const int64_t words = (n + 7) / 8;
  for (int64_t i = threadIdx.x; i < rows * words; i += THREADS) {
    const int64_t r = i / words, c = 8 * (i - r * words);
    const uint8_t* const q = p + r * ld + c;
    if (c + 8 <= n) {
      uint32_t w[2];
      __builtin_memcpy(w, q, 8);
      bad |= outside(w[0]) | outside(w[1]);
    } else {
      for (int64_t j = 0; c + j < n; ++j) bad |= (uint32_t)q[j] - 104u > 36u;
    }
  }
  return __syncthreads_or(bad != 0);
}

template <typename T, bool TR, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void mx4_tile_kernel(Mx4MatmulArgs a, Mx4Cut c) {
  constexpr bool H = __is_same(T, _Float16);
  __shared__ __attribute__((aligned(16))) char
      lds[std::max(kTileBytes<T, TR, BM, BN, H, false>,
                   H ? kTileBytes<T, TR, BM, 128, false, true> : 0)];
  const Mx4Place p = mx4_place(c, blockIdx.x);
  const int64_t K = TR ? a.W.rows : a.W.cols, steps = (K + kStep - 1) / kStep;
  Tile tile;
  tile.m0 = (int64_t)p.m * BM;
  tile.t0 = (int64_t)p.n * BN;
  tile.first = p.cut ? (int64_t)p.piece * c.steps : 0;
  tile.last = p.cut ? min(tile.first + c.steps, steps) : steps;
  const int64_t rest = c.tiles_m * c.tiles_n - c.whole;
  tile.part = p.cut ? a.part + (p.piece * rest + p.rest) * (BM * BN) : nullptr;
  tile.bn = BN;
  if constexpr (H) {
    const int64_t nb = (a.W.cols + kMx4Block - 1) / kMx4Block;
    const int64_t r0 = TR ? tile.first * kStep : tile.m0, b0 = TR ? tile.m0 / 32 : 2 * tile.first;
    const int64_t rows = min(a.W.rows - r0, TR ? (tile.last - tile.first) * kStep : (int64_t)BM);
    const int64_t n = min(nb - b0, TR ? (int64_t)BM / 32 : 2 * (tile.last - tile.first));
    if (wide_scales<64 * WM * WN>(a.W.scales + r0 * nb + b0, rows, n, nb)) {
      // in two parts x takes twice the room: 128 tokens at a time
      for (int i = 0; i < BN / 128; ++i, tile.t0 += 128, tile.part += tile.part ? 128 : 0) {
        tile_product<T, TR, BM, 128, WM, WN, false, true>(a, tile, lds);
        // the output of the last 128 has left shared memory before the next begin
        __syncthreads();
      }
      return;
    }
  }
  tile_product<T, TR, BM, BN, WM, WN, H, false>(a, tile, lds);
}

constexpr int kSlots = 256;  // compute units

struct Cut : Mx4Cut {
  bool large;
  int bm, bn;
};
// Large tiles (256 rows; transposed 256 tokens too) where they fill the GPU (4096 x 4096,
// 2048 tokens: 76 us, 84 with small ones; gradient of 3000 tokens, 192 large tiles: 109 us,
// 123 with small ones; of 2048, 128 tiles: 106 and 82).  Fewer tiles than compute units are cut along
// the inner size until they do, in pieces of at least four steps (4096 x 4096, 256
// tokens: 24.6 us in four pieces, 28.7 in eight, 42 whole: the pieces are written and
// read again).  Of a few more than a round of them those past it are cut, so that they do
// not take a round of their own (2304 tokens, 32 tiles past it: 103 us whole, 81 in four
// pieces, 85 in eight or two; gradient of 4352 tokens, 16 past it: 215 whole, 145 in eight
// pieces, 154 in sixteen or four; of 5120, 64 past it: 172 in four, 180 in two).
Cut cut(const Mx4& W, int transposed, int dtype, int64_t T) {
  const int64_t M = transposed ? W.cols : W.rows, K = transposed ? W.rows : W.cols;
  const int64_t steps = cdiv(K, kStep);
  Cut c;
  const int64_t wide = transposed ? 256 : 128;
  c.large = dtype != kF32 && cdiv(M, 256) * cdiv(T, wide) >= (transposed ? 160 : 256);
  c.bm = c.large ? 256 : 128;
  c.bn = c.large ? (int)wide : 128;
  c.tiles_m = (uint32_t)cdiv(M, c.bm);
  c.tiles_n = (uint32_t)cdiv(T, c.bn);
  const int64_t tiles = (int64_t)c.tiles_m * c.tiles_n, rest = tiles % kSlots;
  // the transposed large tiles have a compute unit each, others share one
  const int64_t few = tiles < kSlots ? (c.large ? 0 : kSlots) : c.large && transposed ? 128 : 85;
  int64_t pieces = 1;
  if (rest > 0 && rest <= few) {
    pieces = kSlots / rest;
    if (tiles > kSlots) pieces = std::max(std::min<int64_t>(pieces, 4), kSlots / 2 / rest);
    pieces = std::min(pieces, steps / 4);
  }
  c.whole = (uint32_t)(pieces > 1 ? tiles - rest : tiles);
  c.steps = (int32_t)cdiv(steps, std::max<int64_t>(pieces, 1));
  c.pieces = (uint32_t)cdiv(steps, c.steps);
  return c;
}

template <typename T, bool TR>
void launch(const Mx4MatmulArgs& a, const Cut& c, hipStream_t s) {
  const uint32_t blocks = mx4_blocks(c);
  if constexpr (sizeof(T) == 2) {
    if (c.large) {
      if constexpr (TR)
        mx4_tile_kernel<T, TR, 256, 256, 4, 2><<<blocks, 512, 0, s>>>(a, c);
      else
        mx4_tile_kernel<T, TR, 256, 128, 4, 1><<<blocks, 256, 0, s>>>(a, c);
      return;
    }
  }
  // f32, whose x takes the whole shared memory in its three parts: eight waves (gradient of
  // 512 tokens, 2048 x 2048: 31.9 us, 35.7 with four; 2048 tokens, 4096 x 4096: 256, 316)
  if constexpr (sizeof(T) == 4)
    mx4_tile_kernel<T, TR, 128, 128, 2, 4><<<blocks, 512, 0, s>>>(a, c);
  else
    mx4_tile_kernel<T, TR, 128, 128, 2, 2><<<blocks, 256, 0, s>>>(a, c);
}

// Up to this many tokens the kernel of few tokens is the faster (bf16 4096 -> 11008, 64
// tokens: 23.9 us, 30.4 in tiles; 128: 44.6 and 31.7; f32 4096 x 4096, 32: 23.8 and 26.0).
bool is_few(int transposed, int dtype, int64_t T) {
  return !transposed && T <= (dtype == kF32 ? 32 : 64);
}

template <typename T>
hipError_t matmul(Mx4MatmulArgs a, int transposed, int dtype, hipStream_t s) {
  Cut c = cut(a.W, transposed, dtype, a.T);
  // rows of x further apart than the kernel of few tokens counts: no workspace, so whole
  if (is_few(transposed, dtype, a.T)) c.whole = c.tiles_m * c.tiles_n;
  const int64_t M = transposed ? a.W.cols : a.W.rows;
  if (transposed)
    launch<T, true>(a, c, s);
  else
    launch<T, false>(a, c, s);
  if (c.whole < c.tiles_m * c.tiles_n)
    return launch_mx4_sum(a.part, c, c.bm, c.bn, M, a.T, a.out, dtype, a.ldo, s);
  return hipGetLastError();
}

}  // namespace

size_t mx4_matmul_bytes(const Mx4& W, int transposed, int dtype, int64_t T) {
  if (is_few(transposed, dtype, T)) return 0;
  const Cut c = cut(W, transposed, dtype, T);
  return mx4_part_bytes(c, c.bm, c.bn);
}

hipError_t launch_mx4_matmul(const Mx4MatmulArgs& a, int transposed, int dtype, hipStream_t s) {
  if (is_few(transposed, dtype, a.T) && a.ldx <= kMx4FewLd) return launch_mx4_few(a, dtype, s);
  if (dtype == kF32) return matmul<float>(a, transposed, dtype, s);
  if (dtype == kF16) return matmul<_Float16>(a, transposed, dtype, s);
  return matmul<bf16_t>(a, transposed, dtype, s);
}

}  // namespace spops
