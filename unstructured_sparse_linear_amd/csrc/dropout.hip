// dropout.hip -- dropout whose mask is never stored.
//
// out = keep ? x * 65536 / (65536 - limit) : 0, keep = r >= limit, limit = p * 65536
// rounded, r 16 random bits of the element.  The bits come from Philox 4x32 of seven
// rounds (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2,
// 3", 2011; seven is the least number that passed all their tests): the counter is
// (column / 8, row, step), the key the seed, and the eight halves of its result go to
// eight neighbouring columns, so that a group of columns costs one evaluation (16 bits
// of probability instead of 32).  So the mask depends on the element's place alone, and
// the gradient is the same call.
//
// Bound by memory: 11008 x 8192 bf16 61 to 66 us (5.4 to 5.9 TB/s), f32 133.  A lane
// holds one group, 16 bytes of 16-bit values; halves are compared and masked in pairs
// and bf16 rounded in pairs (one value at a time: 87 us, bound by the vector unit; f16,
// whose conversions are single, 80).
#include <algorithm>

#include "common.h"
#include "kernels.h"

namespace spops {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMostItems = (int64_t)1 << 31;  // threads of a launch (under 2^32)

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

struct Four {
  uint32_t v[4];
};

__device__ __forceinline__ Four philox7(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                        uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    const uint64_t p0 = (uint64_t)0xD2511F53u * c0, p1 = (uint64_t)0xCD9E8D57u * c2;
    const uint32_t n0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0, n2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
    c1 = (uint32_t)p1;
    c3 = (uint32_t)p0;
    c0 = n0;
    c2 = n2;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return {{c0, c1, c2, c3}};
}

template <typename T>
__global__ __launch_bounds__(kThreads) void dropout_kernel(DropoutArgs a) {
  const uint32_t groups = (uint32_t)((a.cols + 7) / 8), id = blockIdx.x * kThreads + threadIdx.x;
  const uint32_t row = id / groups, g = id - row * groups;
  const int64_t r = a.row0 + row;
  if (r >= a.rows) return;
  const uint64_t seed = a.state ? a.state[0] : a.seed, step = a.state ? a.state[1] : a.step;
  const Four f = philox7((uint32_t)g, (uint32_t)r, (uint32_t)step, (uint32_t)(step >> 32),
                         (uint32_t)seed, (uint32_t)(seed >> 32));
  const T* p = (const T*)a.x + r * a.ldx + 8 * (int64_t)g;
  T* q = (T*)a.out + r * a.ldo + 8 * (int64_t)g;
  const int64_t c = 8 * (int64_t)g;
  const bool whole = c + 8 <= a.cols;
  union {
    T t[8];
    uint32_t w[2 * sizeof(T)];
  } v;
  if (whole) {
    __builtin_memcpy(v.t, p, sizeof(v.t));
  } else {
#pragma unroll
    for (int i = 0; i < (int)(2 * sizeof(T)); ++i) v.w[i] = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < a.cols) v.t[i] = p[i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // all ones where a half is kept: max(half, limit) is the half itself
    const u16x2 half = __builtin_bit_cast(u16x2, f.v[i]);
    const u16x2 drop = __builtin_elementwise_max(half, (u16x2)(uint16_t)a.limit) ^ half;
    uint32_t keep = __builtin_bit_cast(
        uint32_t, (u16x2)(__builtin_elementwise_min(drop, (u16x2)(uint16_t)1) - (uint16_t)1));
    if (a.limit > 65535u) keep = 0u;
    if constexpr (sizeof(T) == 2) {
      T* const t = nullptr;
      v.w[i] = pair16(lo_f32(v.w[i], t) * a.scale, hi_f32(v.w[i], t) * a.scale, t) & keep;
    } else {
      v.w[2 * i] = __float_as_uint(__uint_as_float(v.w[2 * i]) * a.scale) &
                   (uint32_t)((int32_t)(keep << 16) >> 16);
      v.w[2 * i + 1] = __float_as_uint(__uint_as_float(v.w[2 * i + 1]) * a.scale) &
                       (uint32_t)((int32_t)keep >> 16);
    }
  }
  if (whole) {
    __builtin_memcpy(q, v.t, sizeof(v.t));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < a.cols) q[i] = v.t[i];
  }
}

}  // namespace

hipError_t launch_dropout(DropoutArgs a, int dtype, hipStream_t s) {
  const int64_t groups = cdiv(a.cols, 8), most = std::max<int64_t>(1, kMostItems / groups);
  const int64_t rows = a.rows;
  for (a.row0 = 0; a.row0 < rows; a.row0 = a.rows) {
    // the last workgroup reaches past the launch's rows
    a.rows = std::min(rows, a.row0 + most);
    const uint32_t blocks = (uint32_t)cdiv((a.rows - a.row0) * groups, kThreads);
    if (dtype == kF32)
      dropout_kernel<float><<<blocks, kThreads, 0, s>>>(a);
    else if (dtype == kF16)
      dropout_kernel<_Float16><<<blocks, kThreads, 0, s>>>(a);
    else
      dropout_kernel<bf16_t><<<blocks, kThreads, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace spops
