// clip.hip -- the norm of many gradients together, and clipping by it.
//
//   norm = sqrt(sum over all tensors of g^2),  c = min(1, max_norm / (norm + 1e-6)),
//   out = c g   (in place, or into other tensors; a NaN norm gives NaN; an
//                infinite max_norm gives c = 1 whatever the norm)
//
// Two launches for up to 250 tensors (and two more for each further 250): the
// squares' sums, one per workgroup; then every workgroup adds those sums in
// the same order and scales its part, its first values already requested.  More
// sums than one launch leaves are added once, by a launch between (2000 tensors of
// 65536 bf16 values: 244 us, 336 where each workgroup adds them; 500 of 1000 values:
// 22 us, 24 with it).  The
// tensors' table travels in the kernel arguments, 16 bytes a tensor with the
// first launch (which leaves it in the workspace for the second) and 8 with the
// second, so a call copies nothing to the device and may be captured.  Sums are
// fp64: no square overflows, and the norm is exact to its fp32 rounding.  Bound
// by memory: the gradients are read twice and written once (1.08 GB of f32:
// 597 us, 5.4 TB/s).  The second pass runs through them backwards, towards what the
// 256 MB memory-side cache may still hold of the first (609 us forwards).  In place
// and below the limit they are read once (211 us).
#include <math.h>

#include "kernels.h"
#include "lowrank.h"

namespace spops {
namespace {

constexpr int kThreads = 256;
// Tensors of one launch: its arguments stay under 4 KiB, and a full table of
// the largest tensors has fewer chunks than an int counts.
constexpr int kTable = 250;
constexpr int64_t kChunk = 8192; // elements of a workgroup's step
// Workgroups: six on each of the 256 CUs, for the tensors of a model's adapters
// in one round (200 tensors, 12 million values: 28 us, 38 with four); four for
// long streams (270 million f32 values: 599 us, 617 with six).
constexpr int64_t kMaxBlocks = 1536;
constexpr int64_t kStreamBlocks = 1024, kStreamChunks = 4 * kMaxBlocks;

struct Table {
  const void* grad[kTable];
  int32_t first[kTable + 1];  // first chunk of each tensor
  // Elements of its last chunk less one, dtype above bit 13.  A word, not 16 bits:
  // with both widths under one index the compiler (ROCm 7.2) forms the address of
  // `first` from two halves of it, of which scalar loads drop the odd bits.
  int32_t tail[kTable];
  int32_t count;
};
struct Outs {
  void* out[kTable];
};
static_assert(kTable * (kClipMaxNumel / kChunk) + kMaxBlocks < INT32_MAX, "chunks");
static_assert(sizeof(Table) + 16 <= 4096 && sizeof(Outs) + 64 <= 4096, "kernel arguments");

struct Piece {
  int tensor, dtype, n;
  int64_t at;  // first element
};

// The tensor of chunk c: lanes compare the table's starts.
__device__ __forceinline__ Piece find_piece(const Table& t, int c) {
  int before = 0;
#pragma unroll
  for (int h = 0; h < (kTable + kWave - 1) / kWave; ++h) {
    const int i = h * kWave + lane_id();
    before += __builtin_popcountll(__ballot(i < t.count && t.first[i < kTable ? i : 0] <= c));
  }
  Piece p;
  p.tensor = before - 1;
  const int tail = t.tail[p.tensor];
  p.at = (int64_t)(c - t.first[p.tensor]) * kChunk;
  p.dtype = tail >> 13;
  p.n = c + 1 == t.first[p.tensor + 1] ? (tail & 8191) + 1 : (int)kChunk;
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

// A whole chunk, 16 bytes a thread and load.
struct Held {
  Row<float, 4> w[kChunk * 4 / 16 / kThreads];
};
template <typename T>
__device__ __forceinline__ void hold(const T* g, Held& h) {
#pragma unroll
  for (int k = 0; k < (int)(kChunk * sizeof(T) / 16 / kThreads); ++k)
    __builtin_memcpy(&h.w[k], g + (k * kThreads + threadIdx.x) * (16 / sizeof(T)), 16);
}
template <typename T>
__device__ __forceinline__ void scale_held(const Held& h, T* out, float c) {
  constexpr int C = 16 / sizeof(T);
#pragma unroll
  for (int k = 0; k < (int)(kChunk / C / kThreads); ++k) {
    const Row<T, C> r = __builtin_bit_cast(Row<T, C>, h.w[k]);
    float v[C];
#pragma unroll
    for (int e = 0; e < C; ++e) v[e] = row_f32<T, C>(r, e) * c;
    store_chunk<T, C>(out + (k * kThreads + threadIdx.x) * C, C, v);
  }
}
template <typename T>
__device__ __forceinline__ void scaled(const T* g, T* out, int n, float c) {
  constexpr int C = 16 / sizeof(T), STEP = kThreads * C;
  for (int i = threadIdx.x * C; i < n; i += STEP) {
    float v[C];
    load_chunk<T, C>(g + i, n - i, v);
#pragma unroll
    for (int e = 0; e < C; ++e) v[e] *= c;
    store_chunk<T, C>(out + i, n - i, v);
  }
}

// f(typed null) for the storage type.
template <typename F>
__device__ __forceinline__ void with_type(int dtype, F f) {
  if (dtype == kF32)
    f((float*)nullptr);
  else if (dtype == kF16)
    f((_Float16*)nullptr);
  else
    f((bf16_t*)nullptr);
}
template <typename T>
__device__ __forceinline__ T* typed(void* p, int64_t at, T*) {
  return (T*)p + at;
}
template <typename T>
__device__ __forceinline__ const T* typed(const void* p, int64_t at, T*) {
  return (const T*)p + at;
}

__global__ __launch_bounds__(kThreads, 6) void clip_norm_kernel(const Table t, double* partial,
                                                             Table* kept) {
  __shared__ double red[kThreads / kWave];
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < (int)(sizeof(Table) / 4); i += kThreads)
      ((uint32_t*)kept)[i] = ((const uint32_t*)&t)[i];
  double s = 0.0;
  for (int c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
    const Piece p = find_piece(t, c);
    with_type(p.dtype, [&](auto* as) { s += squares(typed(t.grad[p.tensor], p.at, as), p.n); });
  }
  s = block_sum(s, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// The sum of the workgroups' sums, in the order of clip_scale_kernel's.
__global__ __launch_bounds__(kThreads) void clip_total_kernel(const double* partial, int partials,
                                                              double* total) {
  __shared__ double red[kThreads / kWave];
  double s = 0.0;
#pragma unroll 8
  for (int i = threadIdx.x; i < partials; i += kThreads) s += partial[i];
  s = block_sum(s, red);
  if (threadIdx.x == 0) *total = s;
}

__global__ __launch_bounds__(kThreads) void clip_scale_kernel(const Outs outs, const Table* table,
                                                              const double* partial, int partials,
                                                              double max_norm, float* norm_out) {
  __shared__ double red[kThreads / kWave];
  const Table& t = *table;
  const int chunks = table ? t.first[t.count] : 0;
  Held held;
  Piece p{};
  int b = blockIdx.x;
  if (b < chunks) {
    p = find_piece(t, chunks - 1 - b);
    if (p.n == kChunk)
      with_type(p.dtype, [&](auto* as) { hold(typed(t.grad[p.tensor], p.at, as), held); });
  }
  double s = 0.0;
  for (int i = threadIdx.x; i < partials; i += kThreads) s += partial[i];
  const double norm = sqrt(block_sum(s, red));
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  const double q = max_norm / (norm + 1e-6);
  // without a limit nothing changes, also where the norm is infinite or NaN
  const float coef = q > 1.0 || isinf(max_norm) ? 1.f : (float)q;
  while (b < chunks) {
    const void* g = t.grad[p.tensor];
    void* out = outs.out[p.tensor];
    if (out != g || coef != 1.f)  // or nothing changes
      with_type(p.dtype, [&](auto* as) {
        if (p.n == kChunk)
          scale_held(held, typed(out, p.at, as), coef);
        else
          scaled(typed(g, p.at, as), typed(out, p.at, as), p.n, coef);
      });
    b += gridDim.x;
    if (b >= chunks) break;
    p = find_piece(t, chunks - 1 - b);
    if (p.n == kChunk && (coef != 1.f || outs.out[p.tensor] != t.grad[p.tensor]))
      with_type(p.dtype, [&](auto* as) { hold(typed(t.grad[p.tensor], p.at, as), held); });
  }
}

// The table of tensors [i, count) as far as it goes; returns the next i.
int64_t fill_table(const ClipTensor* ts, int64_t i, int64_t count, Table& t, Outs& o) {
  t.count = 0;
  int64_t chunks = 0;
  for (; i < count && t.count < kTable; ++i) {
    const int64_t c = cdiv(ts[i].numel, kChunk);
    if (c == 0) continue;
    o.out[t.count] = ts[i].out;
    t.grad[t.count] = ts[i].grad;
    t.tail[t.count] = (int32_t)((ts[i].numel - 1) % kChunk) | ts[i].dtype << 13;
    t.first[t.count++] = (int32_t)chunks;
    chunks += c;
  }
  t.first[t.count] = (int32_t)chunks;
  return i;
}

int blocks_of(const Table& t) {
  const int64_t c = t.first[t.count];
  return (int)(c < kMaxBlocks ? c : c < kStreamChunks ? kMaxBlocks : kStreamBlocks);
}

}  // namespace

// A table for each launch of a pass, then one fp64 sum per workgroup.
size_t clip_workspace_bytes(int64_t count) {
  return (size_t)(cdiv(count, kTable) + 1) * (sizeof(Table) + kMaxBlocks * 8);
}

hipError_t launch_clip(const ClipTensor* ts, int64_t count, double max_norm, float* norm, void* ws,
                       hipStream_t s) {
  Table* tables = (Table*)ws;
  double* partial = (double*)(tables + cdiv(count, kTable) + 1);
  Table t;
  Outs o;
  int partials = 0, launches = 0;
  for (int64_t i = 0; i < count;) {
    i = fill_table(ts, i, count, t, o);
    const int blocks = blocks_of(t);
    if (blocks == 0) continue;
    hipLaunchKernelGGL(clip_norm_kernel, dim3(blocks), dim3(kThreads), 0, s, t, partial + partials,
                       tables + launches++);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    partials += blocks;
  }
  if (launches == 0) {  // no values: the norm alone
    hipLaunchKernelGGL(clip_scale_kernel, dim3(1), dim3(kThreads), 0, s, o, (const Table*)nullptr,
                       partial, 0, max_norm, norm);
    return hipGetLastError();
  }
  if (partials > kMaxBlocks) {
    hipLaunchKernelGGL(clip_total_kernel, dim3(1), dim3(kThreads), 0, s, partial, partials,
                       partial + partials);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    partial += partials;
    partials = 1;
  }
  launches = 0;
  for (int64_t i = 0; i < count;) {
    i = fill_table(ts, i, count, t, o);
    const int blocks = blocks_of(t);
    if (blocks == 0) continue;
    hipLaunchKernelGGL(clip_scale_kernel, dim3(blocks), dim3(kThreads), 0, s, o,
                       (const Table*)(tables + launches), partial, partials, max_norm,
                       launches == 0 ? norm : nullptr);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    ++launches;
  }
  return hipSuccess;
}

}  // namespace spops
