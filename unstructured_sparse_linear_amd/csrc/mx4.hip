// mx4.hip -- matrices to and from 4-bit microscaled form.
//
// quantise: s = 2^(floor(log2(max |w|)) - 2) of each block of 32 along a row,
// element = w / s rounded to nearest even among 0, 0.5, 1, 1.5, 2, 3, 4, 6.
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
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t r = id / (4 * nb), word = id - r * 4 * nb;
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
  codes[r * 4 * nb + word] = s == 255u ? 0u : mx4_encode(v, mx4_scale(s));
  if ((word & 3) == 0) scales[r * nb + word / 4] = (uint8_t)s;
}

// Columns of unit stride (activations of features x tokens, quantised as tokens x
// features): one thread a block, neighbouring threads in neighbouring rows.
template <typename T>
__global__ __launch_bounds__(kThreads) void mx4_quantize_columns(const T* w, int64_t rows,
                                                                 int64_t cols, int64_t ld,
                                                                 uint32_t* codes,
                                                                 uint8_t* scales) {
  const int64_t nb = (cols + kMx4Block - 1) / kMx4Block;
  const int64_t r = (int64_t)(blockIdx.x / nb) * kThreads + threadIdx.x, b = blockIdx.x % nb;
  if (r >= rows) return;
  const int64_t k0 = b * kMx4Block;
  float v[4][8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kMx4Block; ++i) {
    v[i / 8][i % 8] = k0 + i < cols ? to_f32(w[(k0 + i) * ld + r]) : 0.f;
    top = max(top, magnitude(v[i / 8][i % 8]));
  }
  const uint32_t s = mx4_scale_byte(top);
  uint4 q = make_uint4(0u, 0u, 0u, 0u);
  if (s != 255u) {
    const float scale = mx4_scale(s);
    q = make_uint4(mx4_encode(v[0], scale), mx4_encode(v[1], scale), mx4_encode(v[2], scale),
                   mx4_encode(v[3], scale));
  }
  *(uint4*)(codes + (r * nb + b) * 4) = q;
  scales[r * nb + b] = (uint8_t)s;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void mx4_dequantize_kernel(const uint32_t* codes,
                                                                  const uint8_t* scales,
                                                                  int64_t rows, int64_t cols,
                                                                  T* out, int64_t ldo) {
  const int64_t nb = (cols + kMx4Block - 1) / kMx4Block;
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t r = id / (4 * nb), word = id - r * 4 * nb;
  if (r >= rows || 8 * word >= cols) return;
  const uint32_t w = codes[r * 4 * nb + word];
  const float s = mx4_scale(scales[r * nb + word / 4]);
  T t[8];
  const f32x2 a = mx4_pair_f32<0>(w, s), b = mx4_pair_f32<1>(w, s), c = mx4_pair_f32<2>(w, s),
              d = mx4_pair_f32<3>(w, s);
  t[0] = from_f32<T>(a[0]), t[1] = from_f32<T>(a[1]), t[2] = from_f32<T>(b[0]);
  t[3] = from_f32<T>(b[1]), t[4] = from_f32<T>(c[0]), t[5] = from_f32<T>(c[1]);
  t[6] = from_f32<T>(d[0]), t[7] = from_f32<T>(d[1]);
  T* p = out + r * ldo + 8 * word;
  if (8 * word + 8 <= cols) {
    __builtin_memcpy(p, t, sizeof(t));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (8 * word + i < cols) p[i] = t[i];
  }
}

// out = the pieces' sums, added in order.
template <typename T>
__global__ __launch_bounds__(256) void mx4_sum_kernel(const float* part, int pieces, int64_t M,
                                                      int64_t tokens, T* out, int64_t ldo) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= M * tokens) return;
  float v = 0.f;
  for (int i = 0; i < pieces; ++i) v += part[i * M * tokens + id];
  const int64_t r = id / tokens;
  out[r * ldo + id - r * tokens] = from_f32<T>(v);
}

// Threads of a launch (under 2^32); larger matrices take several.
constexpr int64_t kMostItems = (int64_t)1 << 31;

template <typename T>
hipError_t quantize(const void* w, int64_t rows, int64_t cols, int64_t rs, int64_t cs,
                    uint8_t* codes, uint8_t* scales, hipStream_t s) {
  const int64_t nb = cdiv(cols, kMx4Block);
  const int64_t each = cs == 1 ? 4 * nb : nb;
  const int64_t most = kMostItems / each / kThreads * kThreads;
  for (int64_t r = 0; r < rows; r += most) {
    const int64_t n = std::min(most, rows - r);
    const T* const from = (const T*)w + r * rs;
    uint32_t* const c = (uint32_t*)(codes + r * nb * 16);
    if (cs == 1)
      mx4_quantize_rows<T><<<(uint32_t)cdiv(n * each, kThreads), kThreads, 0, s>>>(
          from, n, cols, rs, c, scales + r * nb);
    else
      mx4_quantize_columns<T><<<(uint32_t)(cdiv(n, kThreads) * nb), kThreads, 0, s>>>(
          from, n, cols, cs, c, scales + r * nb);
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

hipError_t launch_mx4_sum(const float* part, int pieces, int64_t M, int64_t tokens, void* out,
                          int dtype, int64_t ldo, hipStream_t s) {
  const uint32_t blocks = (uint32_t)cdiv(M * tokens, 256);
  if (dtype == kF32)
    mx4_sum_kernel<<<blocks, 256, 0, s>>>(part, pieces, M, tokens, (float*)out, ldo);
  else if (dtype == kF16)
    mx4_sum_kernel<<<blocks, 256, 0, s>>>(part, pieces, M, tokens, (_Float16*)out, ldo);
  else
    mx4_sum_kernel<<<blocks, 256, 0, s>>>(part, pieces, M, tokens, (bf16_t*)out, ldo);
  return hipGetLastError();
}

}  // namespace spops
