// mx4.hip -- matrices to and from 4-bit microscaled form.
//
// quantise: s = 2^(floor(log2(max |w|)) - 2) of each block of 32 along a row,
// element = w / s rounded to nearest even among 0, 0.5, 1, 1.5, 2, 3, 4, 6.
//
// Both directions are bound by memory: 11008 x 4096 bf16 quantised in 22.3 us (5.1 TB/s),
// dequantised in 17.8 (6.4, part of it in the memory-side cache); 2047 tokens x 4096 of
// f16 along the columns in 9.3 and 5.4.
#include <algorithm>

#include "kernels.h"
#include "mx4.h"

namespace spops {
namespace {

constexpr int kThreads = 256;

// Rows of unit stride: four lanes a block, eight elements a lane.
template <typename T>
__global__ __launch_bounds__(kThreads) void mx4_quantize_rows(const T* w, int64_t rows,
                                                              int64_t cols, int64_t ld,
                                                              uint32_t* codes, uint8_t* scales) {
  const int64_t nb = (cols + kMx4Block - 1) / kMx4Block;
  const uint32_t words = 4 * (uint32_t)nb, id = blockIdx.x * kThreads + threadIdx.x;
  const uint32_t r = id / words, word = id - r * words;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
  if (r < rows) {
    const T* p = w + r * ld + 8 * word;
    if (8 * word + 8 <= cols) {
      T t[8];
      __builtin_memcpy(t, p, sizeof(t));
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = to_f32(t[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (8 * word + i < cols) v[i] = to_f32(p[i]);
    }
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, magnitude(v[i]));
  top = max(top, (uint32_t)__shfl_xor((int)top, 1, 64));
  top = max(top, (uint32_t)__shfl_xor((int)top, 2, 64));
  const uint32_t s = mx4_scale_byte(top);
  if (r >= rows) return;
  codes[id] = s == 255u ? 0u : mx4_encode(v, mx4_scale(s));
  if ((word & 3) == 0) scales[id / 4] = (uint8_t)s;
}

// Columns of unit stride (activations of features x tokens, quantised as tokens x
// features): 128 rows (tokens) x 8 blocks a workgroup, a wave a block.  A lane holds the
// 32 elements of two neighbouring rows, so that a load of the wave is 256 neighbouring
// bytes and a block's maximum needs no other lane; codes go through shared memory, so
// that a row's eight blocks are stored as one line.  Neighbouring workgroups take
// neighbouring rows: in the other order, columns a power of two apart meet in few memory
// channels (8192 tokens x 4096, bf16: 13.7 us, 16.3 so).  Where there are few of them,
// neighbours share an XCD, as lines cross tiles (300 tokens x 4096 and their product of
// two: 20.9 us, 21.7 apart; 8192 tokens: 16.0).
constexpr int kTileRows = 128, kTileBlocks = 8;
template <typename T>
__global__ __launch_bounds__(64 * kTileBlocks) void mx4_quantize_columns(const T* w, int64_t rows,
                                                                         int64_t cols, int64_t ld,
                                                                         uint32_t tiles,
                                                                         uint8_t* codes,
                                                                         uint8_t* scales) {
  // a row's codes, and 16 bytes so that neighbouring rows begin in other banks
  constexpr int kRow = 16 * kTileBlocks + 16;
  __shared__ __attribute__((aligned(16))) char lds[kTileRows * kRow];
  __shared__ __attribute__((aligned(8))) uint8_t bytes[kTileRows * kTileBlocks];
  const int64_t nb = (cols + kMx4Block - 1) / kMx4Block;
  const uint32_t index = tiles < 16 ? xcd_index(blockIdx.x, gridDim.x) : blockIdx.x;
  const int64_t r0 = (int64_t)(index % tiles) * kTileRows;
  const int64_t b0 = (int64_t)(index / tiles) * kTileBlocks;
  const int tid = threadIdx.x, lane = tid % 64, wave = wave_uniform(tid / 64);
  const int64_t r = r0 + 2 * lane, k0 = (b0 + wave) * kMx4Block;
  if (k0 < cols) {
    struct Pair {
      T v[2];
    } p[kMx4Block];
    const int n = (int)min((int64_t)kMx4Block, cols - k0);
    const T* const from = w + k0 * ld + r;
    if (n == kMx4Block && r0 + kTileRows <= rows) {
#pragma unroll
      for (int i = 0; i < kMx4Block; ++i) __builtin_memcpy(&p[i], from + i * ld, sizeof(Pair));
    } else {
#pragma unroll
      for (int i = 0; i < kMx4Block; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          p[i].v[j] = i < n && r + j < rows ? from[i * ld + j] : from_f32<T>(0.f);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < kMx4Block; ++i) top = max(top, magnitude(to_f32(p[i].v[j])));
      const uint32_t s = mx4_scale_byte(top);
      uint32_t q[4] = {0u, 0u, 0u, 0u};
      if (s != 255u) {
        const float scale = mx4_scale(s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = to_f32(p[8 * i + e].v[j]);
          q[i] = mx4_encode(v, scale);
        }
      }
      *(uint4*)(lds + (2 * lane + j) * kRow + 16 * wave) = make_uint4(q[0], q[1], q[2], q[3]);
      bytes[(2 * lane + j) * kTileBlocks + wave] = (uint8_t)s;
    }
  }
  __syncthreads();
  const int64_t blocks = min((int64_t)kTileBlocks, nb - b0);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int at = (tid + 512 * i) / kTileBlocks, b = tid % kTileBlocks;
    if (r0 + at < rows && b < blocks)
      *(uint4*)(codes + ((r0 + at) * nb + b0 + b) * 16) = *(const uint4*)(lds + at * kRow + 16 * b);
  }
  if (tid < kTileRows && r0 + tid < rows) {
    uint8_t* const to = scales + (r0 + tid) * nb + b0;
    if (blocks == kTileBlocks)
      __builtin_memcpy(to, bytes + tid * kTileBlocks, kTileBlocks);
    else
      for (int b = 0; b < blocks; ++b) to[b] = bytes[tid * kTileBlocks + b];
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void mx4_dequantize_kernel(const uint32_t* codes,
                                                                  const uint8_t* scales,
                                                                  int64_t rows, int64_t cols,
                                                                  T* out, int64_t ldo) {
  const int64_t nb = (cols + kMx4Block - 1) / kMx4Block;
  const uint32_t words = 4 * (uint32_t)nb, id = blockIdx.x * kThreads + threadIdx.x;
  const uint32_t r = id / words, word = id - r * words;
  if (r >= rows || 8 * word >= cols) return;
  const uint32_t w = codes[id];
  const float s = mx4_scale(scales[id / 4]);
  T t[8];
  if constexpr (sizeof(T) == 2) {
    const uint4 v = mx4_eight<T>(w, s);
    __builtin_memcpy(t, &v, sizeof(t));
  } else {
    const f32x2 v[4] = {mx4_pair_f32<0>(w, s), mx4_pair_f32<1>(w, s), mx4_pair_f32<2>(w, s),
                        mx4_pair_f32<3>(w, s)};
    __builtin_memcpy(t, v, sizeof(t));
  }
  T* p = out + r * ldo + 8 * word;
  if (8 * word + 8 <= cols) {
    __builtin_memcpy(p, t, sizeof(t));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (8 * word + i < cols) p[i] = t[i];
  }
}

// out = the pieces' sums, added in order: four tokens of a row a thread, the pieces'
// loads in flight together.
template <typename T>
__global__ __launch_bounds__(256) void mx4_sum_kernel(const float* part, Mx4Cut c, int bm, int bn,
                                                      int64_t rows, int64_t tokens, T* out,
                                                      int64_t ldo) {
  const uint32_t rest = c.tiles_m * c.tiles_n - c.whole, blocks = bm * bn / 1024;
  const uint32_t index = xcd_index(blockIdx.x, gridDim.x);
  const uint32_t tile = index / blocks, at = (index % blocks * 256 + threadIdx.x) * 4;
  uint32_t m, n;
  mx4_place(c, c.whole + tile, m, n);
  const int64_t r = (int64_t)m * bm + at / bn, t = (int64_t)n * bn + at % bn;
  if (r >= rows || t >= tokens) return;
  const int64_t each = (int64_t)rest * bm * bn;
  const float* p = part + (int64_t)tile * bm * bn + at;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (uint32_t i = 0; i < c.pieces; ++i, p += each) {
    // (tokens past the last were not written, and are not written here)
    const float4 w = *(const float4*)p;
    v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
  }
  const T w[4] = {from_f32<T>(v.x), from_f32<T>(v.y), from_f32<T>(v.z), from_f32<T>(v.w)};
  T* const q = out + r * ldo + t;
  if (t + 4 <= tokens) {
    __builtin_memcpy(q, w, sizeof(w));
  } else {
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (t + j < tokens) q[j] = w[j];
  }
}

// Threads of a launch (under 2^32); larger matrices take several.
constexpr int64_t kMostItems = (int64_t)1 << 31;

template <typename T>
hipError_t quantize(const void* w, int64_t rows, int64_t cols, int64_t rs, int64_t cs,
                    uint8_t* codes, uint8_t* scales, hipStream_t s) {
  const int64_t nb = cdiv(cols, kMx4Block);
  // rows of a launch
  const int64_t most = kMostItems / (4 * nb) / kThreads * kThreads;
  for (int64_t r = 0; r < rows; r += most) {
    const int64_t n = std::min(most, rows - r);
    const T* const from = (const T*)w + r * rs;
    uint8_t* const c = codes + r * nb * 16;
    if (cs == 1) {
      mx4_quantize_rows<T><<<(uint32_t)cdiv(n * 4 * nb, kThreads), kThreads, 0, s>>>(
          from, n, cols, rs, (uint32_t*)c, scales + r * nb);
    } else {
      const uint32_t tiles = (uint32_t)cdiv(n, kTileRows);
      mx4_quantize_columns<T>
          <<<(uint32_t)cdiv(nb, kTileBlocks) * tiles, 64 * kTileBlocks, 0, s>>>(from, n, cols, cs, tiles,
                                                                            c, scales + r * nb);
    }
  }
  return hipGetLastError();
}

template <typename T>
hipError_t dequantize(const Mx4& W, T* out, int64_t ldo, hipStream_t s) {
  const int64_t nb = cdiv(W.cols, kMx4Block), most = kMostItems / (4 * nb);
  for (int64_t r = 0; r < W.rows; r += most) {
    const int64_t n = std::min(most, W.rows - r);
    mx4_dequantize_kernel<T><<<(uint32_t)cdiv(n * 4 * nb, kThreads), kThreads, 0, s>>>(
        (const uint32_t*)(W.codes + r * nb * 16), W.scales + r * nb, n, W.cols, out + r * ldo, ldo);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx4_quantize(const void* w, int dtype, int64_t rows, int64_t cols, int64_t rs,
                               int64_t cs, uint8_t* codes, uint8_t* scales, hipStream_t s) {
  if (dtype == kF32) return quantize<float>(w, rows, cols, rs, cs, codes, scales, s);
  if (dtype == kF16) return quantize<_Float16>(w, rows, cols, rs, cs, codes, scales, s);
  return quantize<bf16_t>(w, rows, cols, rs, cs, codes, scales, s);
}

hipError_t launch_mx4_dequantize(const Mx4& W, void* out, int dtype, int64_t ldo, hipStream_t s) {
  if (dtype == kF32) return dequantize(W, (float*)out, ldo, s);
  if (dtype == kF16) return dequantize(W, (_Float16*)out, ldo, s);
  return dequantize(W, (bf16_t*)out, ldo, s);
}

hipError_t launch_mx4_sum(const float* part, const Mx4Cut& c, int bm, int bn, int64_t M,
                          int64_t tokens, void* out, int dtype, int64_t ldo, hipStream_t s) {
  const uint32_t blocks = (c.tiles_m * c.tiles_n - c.whole) * (uint32_t)(bm * bn / 1024);
  if (dtype == kF32)
    mx4_sum_kernel<<<blocks, 256, 0, s>>>(part, c, bm, bn, M, tokens, (float*)out, ldo);
  else if (dtype == kF16)
    mx4_sum_kernel<<<blocks, 256, 0, s>>>(part, c, bm, bn, M, tokens, (_Float16*)out, ldo);
  else
    mx4_sum_kernel<<<blocks, 256, 0, s>>>(part, c, bm, bn, M, tokens, (bf16_t*)out, ldo);
  return hipGetLastError();
}

}  // namespace spops
