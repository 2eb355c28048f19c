// dropout.hip -- dropout whose mask is never stored.
//
// out = keep ? x * 65536 / (65536 - limit) : 0, keep = r >= limit, limit = p * 65536
// rounded, r 16 random bits of the element.  The bits come from Philox 4x32 of seven
// rounds (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2,
// 3", 2011; seven is the least number that passed their tests, three more would cost
// as much as the memory takes): the counter is (column / 8, row, step), the key the
// seed, and the eight halves of its result go to eight neighbouring columns.  So the
// mask depends on the element's place alone, and the gradient is the same call.
#include <algorithm>

#include "common.h"
#include "kernels.h"

namespace spops {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMostItems = (int64_t)1 << 31;  // threads of a launch (under 2^32)

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
  const int64_t groups = (a.cols + 7) / 8;
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  int64_t r = id / groups;
  const int64_t g = id - r * groups;
  r += a.row0;
  if (r >= a.rows) return;
  const uint64_t seed = a.state ? a.state[0] : a.seed, step = a.state ? a.state[1] : a.step;
  const Four f = philox7((uint32_t)g, (uint32_t)r, (uint32_t)step, (uint32_t)(step >> 32),
                         (uint32_t)seed, (uint32_t)(seed >> 32));
  const T* p = (const T*)a.x + r * a.ldx + 8 * g;
  T* q = (T*)a.out + r * a.ldo + 8 * g;
  const bool whole = 8 * g + 8 <= a.cols;
  T t[8];
  if (whole) {
    __builtin_memcpy(t, p, sizeof(t));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (8 * g + i < a.cols) t[i] = p[i];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t bits = (f.v[i / 2] >> (16 * (i % 2))) & 0xffffu;
    t[i] = bits >= a.limit ? from_f32<T>(to_f32(t[i]) * a.scale) : from_f32<T>(0.f);
  }
  if (whole) {
    __builtin_memcpy(q, t, sizeof(t));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (8 * g + i < a.cols) q[i] = t[i];
  }
}

}  // namespace

hipError_t launch_dropout(DropoutArgs a, int dtype, hipStream_t s) {
  const int64_t groups = cdiv(a.cols, 8), most = std::max<int64_t>(1, kMostItems / groups);
  for (a.row0 = 0; a.row0 < a.rows; a.row0 += most) {
    const uint32_t blocks =
        (uint32_t)cdiv(std::min(most, a.rows - a.row0) * groups, kThreads);
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
