// clip.hip -- the norm of many gradients together, and clipping by it.
//
//   norm = sqrt(sum over all tensors of g^2),  c = min(1, max_norm / (norm + 1e-6)),
//   out = c g   (in place, or into other tensors; a NaN norm gives NaN)
//
// Two launches for up to 128 tensors (and two more for each further 128): the
// squares' sums, one per workgroup; then every workgroup adds those sums in
// the same order and scales its part.  The tensors' table travels in the
// kernel arguments, so a call copies nothing to the device and may be
// captured.  Sums are fp64: no square overflows, and the norm is exact to its
// fp32 rounding.  Bound by memory: the gradients are read twice and written
// once.  The second pass runs through them backwards, so that what the first
// read last is still in the 256 MB memory-side cache.
#include <math.h>

#include "kernels.h"
#include "lowrank.h"

namespace spops {
namespace {

constexpr int kThreads = 256;
constexpr int kTable = 128;      // tensors in one launch's arguments (under 4 KiB)
constexpr int64_t kChunk = 8192; // elements of a workgroup's step
constexpr int64_t kMaxBlocks = 1024;  // four workgroups on each of the 256 CUs

struct Table {
  const void* grad[kTable];
  void* out[kTable];
  int64_t numel[kTable];
  uint8_t dtype[kTable];
  int32_t first[kTable + 1];  // first chunk of each tensor
  int32_t count;
};

struct Piece {
  int tensor;
  int64_t at;  // first element
  int n;
};

// The tensor of chunk c: each lane compares two of the table's starts.
__device__ __forceinline__ Piece find_piece(const Table& t, int c) {
  const int l = lane_id();
  const uint64_t lo = __ballot(l < t.count && t.first[l] <= c);
  const uint64_t hi = __ballot(l + kWave < t.count && t.first[l + kWave] <= c);
  // empty tensors share their start with the next: the last start wins
  Piece p;
  p.tensor = __builtin_popcountll(lo) + __builtin_popcountll(hi) - 1;
  p.at = (int64_t)(c - t.first[p.tensor]) * kChunk;
  const int64_t left = t.numel[p.tensor] - p.at;
  p.n = left < kChunk ? (int)left : (int)kChunk;
  return p;
}

__device__ __forceinline__ double block_sum(double v, double* red) {
  const int tid = threadIdx.x;
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  if (tid % kWave == 0) red[tid / kWave] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < kThreads / kWave; ++w) v += red[w];
  __syncthreads();
  return v;
}

template <typename T>
__device__ __forceinline__ double squares(const T* g, int n) {
  constexpr int C = 16 / sizeof(T), STEP = kThreads * C;
  double s = 0.0;
  if (n == kChunk) {
    float v[kChunk / STEP][C];
#pragma unroll
    for (int k = 0; k < kChunk / STEP; ++k)
      load_chunk<T, C>(g + k * STEP + threadIdx.x * C, C, v[k]);
#pragma unroll
    for (int k = 0; k < kChunk / STEP; ++k)
#pragma unroll
      for (int e = 0; e < C; ++e) s = __builtin_fma((double)v[k][e], (double)v[k][e], s);
  } else {
    for (int i = threadIdx.x * C; i < n; i += STEP) {
      float v[C];
      load_chunk<T, C>(g + i, n - i, v);
#pragma unroll
      for (int e = 0; e < C; ++e) s = __builtin_fma((double)v[e], (double)v[e], s);
    }
  }
  return s;
}

template <typename T>
__device__ __forceinline__ void scaled(const T* g, T* out, int n, float c) {
  constexpr int C = 16 / sizeof(T), STEP = kThreads * C;
  if (n == kChunk) {
    float v[kChunk / STEP][C];
#pragma unroll
    for (int k = 0; k < kChunk / STEP; ++k)
      load_chunk<T, C>(g + k * STEP + threadIdx.x * C, C, v[k]);
#pragma unroll
    for (int k = 0; k < kChunk / STEP; ++k) {
#pragma unroll
      for (int e = 0; e < C; ++e) v[k][e] *= c;
      store_chunk<T, C>(out + k * STEP + threadIdx.x * C, C, v[k]);
    }
  } else {
    for (int i = threadIdx.x * C; i < n; i += STEP) {
      float v[C];
      load_chunk<T, C>(g + i, n - i, v);
#pragma unroll
      for (int e = 0; e < C; ++e) v[e] *= c;
      store_chunk<T, C>(out + i, n - i, v);
    }
  }
}

__global__ __launch_bounds__(kThreads) void clip_norm_kernel(const Table t, double* partial) {
  __shared__ double red[kThreads / kWave];
  double s = 0.0;
  for (int c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
    const Piece p = find_piece(t, c);
    const void* g = t.grad[p.tensor];
    const int dt = t.dtype[p.tensor];
    if (dt == kF32)
      s += squares((const float*)g + p.at, p.n);
    else if (dt == kF16)
      s += squares((const _Float16*)g + p.at, p.n);
    else
      s += squares((const bf16_t*)g + p.at, p.n);
  }
  s = block_sum(s, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__global__ __launch_bounds__(kThreads) void clip_scale_kernel(const Table t, const double* partial,
                                                              int partials, double max_norm,
                                                              float* norm_out) {
  __shared__ double red[kThreads / kWave];
  double s = 0.0;
  for (int i = threadIdx.x; i < partials; i += kThreads) s += partial[i];
  const double norm = sqrt(block_sum(s, red));
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  const double q = max_norm / (norm + 1e-6);
  const float coef = q > 1.0 ? 1.f : (float)q;
  const int chunks = t.first[t.count];
  for (int b = blockIdx.x; b < chunks; b += gridDim.x) {
    const Piece p = find_piece(t, chunks - 1 - b);
    const void* g = t.grad[p.tensor];
    void* out = t.out[p.tensor];
    if (out == g && coef == 1.f) continue;  // nothing changes
    const int dt = t.dtype[p.tensor];
    if (dt == kF32)
      scaled((const float*)g + p.at, (float*)out + p.at, p.n, coef);
    else if (dt == kF16)
      scaled((const _Float16*)g + p.at, (_Float16*)out + p.at, p.n, coef);
    else
      scaled((const bf16_t*)g + p.at, (bf16_t*)out + p.at, p.n, coef);
  }
}

// The table of tensors [i, count) as far as it goes; returns the next i.  The
// caller keeps numel under kClipMaxNumel, so a full table has under 2^31 chunks.
int64_t fill_table(const ClipTensor* ts, int64_t i, int64_t count, Table& t) {
  t.count = 0;
  int64_t chunks = 0;
  for (; i < count && t.count < kTable; ++i) {
    const int64_t c = cdiv(ts[i].numel, kChunk);
    if (c == 0) continue;
    t.grad[t.count] = ts[i].grad;
    t.out[t.count] = ts[i].out;
    t.numel[t.count] = ts[i].numel;
    t.dtype[t.count] = (uint8_t)ts[i].dtype;
    t.first[t.count++] = (int32_t)chunks;
    chunks += c;
  }
  t.first[t.count] = (int32_t)chunks;
  return i;
}

int blocks_of(const Table& t) {
  const int64_t c = t.first[t.count];
  return (int)(c < kMaxBlocks ? c : kMaxBlocks);
}

}  // namespace

size_t clip_workspace_bytes(int64_t count) {
  return (size_t)((cdiv(count, kTable) + 1) * kMaxBlocks * 8);  // one fp64 sum per workgroup
}

hipError_t launch_clip(const ClipTensor* ts, int64_t count, double max_norm, float* norm, void* ws,
                       hipStream_t s) {
  double* partial = (double*)ws;
  Table t;
  int partials = 0;
  for (int64_t i = 0; i < count;) {
    i = fill_table(ts, i, count, t);
    const int blocks = blocks_of(t);
    if (blocks == 0) continue;
    hipLaunchKernelGGL(clip_norm_kernel, dim3(blocks), dim3(kThreads), 0, s, t, partial + partials);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    partials += blocks;
  }
  bool first = true;
  for (int64_t i = 0; i < count || first;) {
    i = fill_table(ts, i, count, t);
    const int blocks = blocks_of(t);
    if (blocks == 0 && !(first && i >= count)) continue;
    hipLaunchKernelGGL(clip_scale_kernel, dim3(blocks ? blocks : 1), dim3(kThreads), 0, s, t,
                       partial, partials, max_norm, first ? norm : nullptr);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    first = false;
  }
  return hipSuccess;
}

}  // namespace spops
