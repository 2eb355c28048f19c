// lowrank.hip -- low-rank adapters of many requests beside a shared projection.
//
// A request i owns the tokens [offsets[i], offsets[i+1]) and one adapter
// a = adapter[i] of a stacked pool A [n, R, in], B [n, out, R] (or none).  On
// its tokens, with k_a = ranks[a] <= R used ranks:
//   u  = scale_a A_a x          (k_a x tokens)
//   y += B_a u                   low_rank_add (given y), low_rank_project
//                                (y = W x, the product made here)
//   du = scale_a B_a^T dy
//   dx = A_a^T du,  dA_a = sum du x^T,  dB_a = sum dy u^T      low_rank_backward
// Activations are feature-major (features x tokens).
//
// Every call is bound by memory: a token's adapter costs 2 R (in + out)
// multiply-adds against in + 2 out values moved, R/1.5 operations a byte in
// f16, far below the matrix cores' rate over the memory's for the ranks in
// use.  So the tiles are chosen for the streams of x, y and dy, and the
// products ride along on MFMA.
//
// Kernels:
//   shrink   u (and du) as fp32 partial sums over slices of the features
//   join     adds the slices (backward, where u is read many times)
//   expand   y + B u
//   dx       A^T du
//   outer    dA and dB, one workgroup per adapter and 64 features
//   project  W x + B u on few tokens
// Requests meet the tiles only through each token's adapter, which the shrink
// kernel finds and writes once.  A tile whose tokens have several adapters is
// computed once per distinct adapter and the results selected per token (never
// multiplied by zero: another request's NaN or infinity stays its own).
#include "kernels.h"
#include "lowrank.h"

namespace spops {
namespace {

constexpr int kThreads = 256;       // shrink, expand, dx, join: four waves
constexpr int kWaves = kThreads / kWave;
constexpr int kOuterThreads = 512;  // outer, project: eight waves
constexpr int kOuterWaves = kOuterThreads / kWave;

// ------------------------------------------------------ adapters of tokens --

template <int TT>
struct TokenTile {
  int mark[TT];  // position of the request that starts at this token, or -1
  int end[TT];   // that request's end and adapter
  int ad[TT];
  int tok[TT];   // the answer: each token's adapter, or -1
};

// Adapters of the tokens [t0, t0 + TT) by all threads of the workgroup: every
// request that meets the tile marks its first token there, and a running
// maximum over the marks gives each token its request.  One pass over the
// offsets, no search.  Out-of-range adapters and adapters without ranks count
// as none; offsets that do not ascend give unspecified adapters, nothing else.
template <int TT, int THREADS>
__device__ __forceinline__ void token_adapters(const LowRankArgs& a, int64_t t0, TokenTile<TT>& s) {
  const int tid = threadIdx.x;
  for (int t = tid; t < TT; t += THREADS) s.mark[t] = -1;
  __syncthreads();
  const int64_t last = t0 + TT < a.T ? t0 + TT : a.T;
  for (int i = tid; i < a.S; i += THREADS) {
    const int64_t b = a.offsets[i], e = a.offsets[i + 1];
    const int64_t lo = b > t0 ? b : t0, hi = e < last ? e : last;
    if (lo < hi) {
      int ad = a.adapter[i];
      if (ad < 0 || ad >= a.n || (a.ranks && a.ranks[ad] <= 0)) ad = -1;
      const int p = (int)(lo - t0);
      s.mark[p] = p;
      s.end[p] = (int)(hi - t0);
      s.ad[p] = ad;
    }
  }
  __syncthreads();
  if (tid < kWave) {
    int before = -1;
#pragma unroll
    for (int h = 0; h < (TT + kWave - 1) / kWave; ++h) {
      const int t = h * kWave + tid;
      int m = t < TT ? s.mark[t] : -1;
#pragma unroll
      for (int o = 1; o < kWave; o <<= 1) {
        const int up = __shfl_up(m, o, kWave);
        if (tid >= o) m = up > m ? up : m;
      }
      m = before > m ? before : m;
      before = __shfl(m, kWave - 1, kWave);
      if (t < TT) s.tok[t] = m >= 0 && t < s.end[m] ? s.ad[m] : -1;
    }
  }
  __syncthreads();
}

// The distinct adapters of a tile, one after another (wave-uniform).
template <int TT>
struct AdapterWalk {
  int a0, a1;
  uint64_t m0, m1;
  __device__ __forceinline__ AdapterWalk(const int* tok) {
    const int l = lane_id();
    a0 = l < TT ? tok[l] : -1;
    a1 = TT > kWave ? tok[l + kWave < TT ? l + kWave : l] : -1;
    m0 = __ballot(a0 >= 0);
    m1 = __ballot(a1 >= 0);
  }
  __device__ __forceinline__ bool next(int& ad) {
    if (!(m0 | m1)) return false;
    ad = m0 ? __builtin_amdgcn_readlane(a0, __builtin_ctzll(m0))
            : __builtin_amdgcn_readlane(a1, __builtin_ctzll(m1));
    m0 &= ~__ballot(a0 == ad);
    m1 &= ~__ballot(a1 == ad);
    return true;
  }
  __device__ __forceinline__ bool done() const { return !(m0 | m1); }
};

__device__ __forceinline__ int rank_of(const LowRankArgs& a, int ad) {
  return a.ranks ? clampi(a.ranks[ad], 0, a.R) : a.R;
}

// -------------------------------------------------------------- tree sum --

// Sums the waves' tiles into wave 0's, in a fixed order.
template <int N, int WAVES>
__device__ __forceinline__ void wave_tree_sum(f32x4 (&acc)[N], f32x4* red) {
  const int wave = threadIdx.x / kWave, lane = lane_id();
#pragma unroll
  for (int h = WAVES / 2; h > 0; h >>= 1) {
    if (wave >= h && wave < 2 * h) {
#pragma unroll
      for (int k = 0; k < N; ++k) red[((wave - h) * N + k) * kWave + lane] = acc[k];
    }
    __syncthreads();
    if (wave < h) {
#pragma unroll
      for (int k = 0; k < N; ++k) acc[k] += red[(wave * N + k) * kWave + lane];
    }
    __syncthreads();
  }
}

// ----------------------------------------------------------------- shrink --

// One product u = F x: x is K x T (ldx), F is [n][R][K] or, TR, [n][K][R].
struct ShrinkJob {
  const void* x;
  const void* f;
  float* u;        // [slices][R][Tp]
  int64_t ldx, K;
  int slices;
};

// Accumulates 32-feature steps [s0, s1) for the tokens tok..tok+V-1 of each
// lane and 16 NR ranks from r0.  x is read V tokens wide, eight rows a lane,
// and turned in registers; the same turn serves a factor stored [K][R].
template <typename T, int V, int NR, bool TR, bool PACK>
__device__ __forceinline__ void shrink_steps(const T* x, int64_t ldx, int64_t K, const T* f, int R,
                                             int r0, int64_t tok, int64_t s0, int64_t s1,
                                             f32x4 (&acc)[NR * V], T* packed) {
  const int lane = lane_id(), n = lane % 16, g = lane / 16;
  struct Buf {
    Row<T, V> x[8];
    Frag<T> f[TR ? 1 : NR];
    Row<T, TR ? NR : 1> ft[8];
  } cur, nxt;
  int64_t frow[NR];
#pragma unroll
  for (int b = 0; b < NR; ++b) {
    const int r = r0 + b * 16 + n;
    frow[b] = (int64_t)(r < R ? r : R - 1) * K;
  }
  const int fcol = TR ? (r0 + n * NR < R - NR ? r0 + n * NR : R - NR) : 0;
  auto load = [&](int64_t step, Buf& b) {
    const int64_t k0 = step * 32 + g * 8;
    const bool whole = step * 32 + 32 <= K;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const int64_t k = whole || k0 + s < K ? k0 + s : K - 1;
      b.x[s] = load_row<T, V>(x + k * ldx + tok);
      if constexpr (TR) b.ft[s] = load_row<T, NR>(f + k * R + fcol);
    }
    if constexpr (!TR) {
#pragma unroll
      for (int q = 0; q < NR; ++q)
        b.f[q] = whole ? load8(f + frow[q] + k0)
                       : load8_count(f + frow[q] + k0, clampi(K - k0, 0, 8));
    }
    if (!whole) {
#pragma unroll
      for (int s = 0; s < 8; ++s)
        if (k0 + s >= K) {
          zero_row(b.x[s]);
          if constexpr (TR) zero_row(b.ft[s]);
        }
    }
  };
  auto compute = [&](int64_t step, const Buf& b) {
    Frag<T> ff[NR];
#pragma unroll
    for (int q = 0; q < NR; ++q) {
      if constexpr (TR)
        ff[q] = column<T, NR>(b.ft, q);
      else
        ff[q] = b.f[q];
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const Frag<T> fx = column<T, V>(b.x, j);
      if constexpr (PACK) __builtin_memcpy(packed + ((step * V + j) * kWave + lane) * 8, &fx, sizeof(fx));
#pragma unroll
      for (int q = 0; q < NR; ++q) acc[q * V + j] = mma(fx, ff[q], acc[q * V + j]);
    }
  };
  if (s0 >= s1) return;
  load(s0, cur);
  for (int64_t s = s0; s < s1; s += 2) {
    if (s + 1 < s1) load(s + 1, nxt);
    compute(s, cur);
    if (s + 2 < s1) load(s + 2, cur);
    if (s + 1 < s1) compute(s + 1, nxt);
  }
}

template <typename T, int V, int NR, bool TR, bool PACK>
__device__ __forceinline__ void shrink_tile(const LowRankArgs& a, const ShrinkJob& job, int slice,
                                            int groups, f32x4* red, TokenTile<16 * V>& tile) {
  constexpr int TT = 16 * V;
  const int lane = lane_id(), n = lane % 16, g = lane / 16, wave = threadIdx.x / kWave;
  // the last tile is moved back to end at T (its shared tokens get the same
  // values twice), and a lane's V tokens are moved back likewise: no load
  // passes the end of a row
  int64_t t0 = (int64_t)blockIdx.x * TT;
  if (t0 > a.T - TT) t0 = a.T > TT ? a.T - TT : 0;
  token_adapters<TT, kThreads>(a, t0, tile);
  const int rc = blockIdx.y / groups, group = blockIdx.y % groups;
  if (blockIdx.y == 0 && blockIdx.z == 0)
    for (int t = threadIdx.x; t < TT; t += kThreads)
      if (t0 + t < a.T) a.tokad[t0 + t] = tile.tok[t];
  const int64_t lim = a.T - V;
  const int64_t tok = t0 + n * V < lim ? t0 + n * V : lim;
  const int64_t steps = cdiv(job.K, 32), units = (int64_t)job.slices * kWaves;
  const int64_t unit = (int64_t)slice * kWaves + wave;
  const int64_t s0 = steps * unit / units, s1 = steps * (unit + 1) / units;
  const T* x = (const T*)job.x;
  const int r0 = rc * 64;
  T* packed = PACK && blockIdx.y == 0
                  ? (T*)a.packed + (int64_t)blockIdx.x * steps * V * kWave * 8
                  : nullptr;
  AdapterWalk<TT> walk(tile.tok);
  int ad, count = 0;
  bool packing = packed != nullptr;
  // a tile without adapters still packs its x
  if (packing && walk.done()) {
    f32x4 acc[NR * V];
#pragma unroll
    for (int k = 0; k < NR * V; ++k) acc[k] = f32x4{0.f, 0.f, 0.f, 0.f};
    shrink_steps<T, V, NR, TR, PACK>(x, job.ldx, job.K, (const T*)job.f, a.R, r0, tok, s0, s1, acc,
                                     packed);
  }
  while (walk.next(ad)) {
    const bool only = count == 0 && walk.done();
    if (count++ % groups != group) continue;
    f32x4 acc[NR * V];
#pragma unroll
    for (int k = 0; k < NR * V; ++k) acc[k] = f32x4{0.f, 0.f, 0.f, 0.f};
    const T* f = (const T*)job.f + (int64_t)ad * a.R * job.K;
    if (packing)
      shrink_steps<T, V, NR, TR, PACK>(x, job.ldx, job.K, f, a.R, r0, tok, s0, s1, acc, packed);
    else
      shrink_steps<T, V, NR, TR, false>(x, job.ldx, job.K, f, a.R, r0, tok, s0, s1, acc, nullptr);
    packing = false;
    wave_tree_sum<NR * V, kWaves>(acc, red);
    if (wave == 0) {
      const float sc = a.scale ? a.scale[ad] : 1.f;
      const int rank = rank_of(a, ad);
#pragma unroll
      for (int q = 0; q < NR; ++q) {
        int r;
        if (TR)
          r = (r0 + n * NR < a.R - NR ? r0 + n * NR : a.R - NR) + q;
        else
          r = r0 + q * 16 + n;
        if (r >= a.R) continue;
        float* u = job.u + ((int64_t)slice * a.R + r) * a.Tp;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t t1 = t0 + (g * 4 + i) * V < lim ? t0 + (g * 4 + i) * V : lim;
          float v[V];
#pragma unroll
          for (int j = 0; j < V; ++j) v[j] = r < rank ? acc[q * V + j][i] * sc : 0.f;
          if (only) {
            __builtin_memcpy(u + t1, v, sizeof(v));
          } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
              if (tile.tok[t1 - t0 + j] == ad) u[t1 + j] = v[j];
          }
        }
      }
    }
  }
}

template <typename T, int V, int NR, bool BACKWARD, bool PACK>
__global__ __launch_bounds__(kThreads) void lowrank_shrink_kernel(LowRankArgs a, ShrinkJob jx,
                                                                  ShrinkJob jy, int groups) {
  __shared__ f32x4 red[kWaves / 2 * NR * V * kWave];
  __shared__ TokenTile<16 * V> tile;
  if (!BACKWARD || (int)blockIdx.z < jx.slices)
    shrink_tile<T, V, NR, false, PACK>(a, jx, blockIdx.z, groups, red, tile);
  else
    shrink_tile<T, V, NR, true, false>(a, jy, blockIdx.z - jx.slices, groups, red, tile);
}

// ------------------------------------------------------------------- join --

// Adds the slices of u and du into slice 0, in order.
__global__ __launch_bounds__(kThreads) void lowrank_join_kernel(LowRankArgs a, int su, int sd) {
  float* u = blockIdx.y ? a.du : a.u;
  const int slices = blockIdx.y ? sd : su;
  const int64_t size = (int64_t)a.R * a.Tp;
  const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4;  // Tp is a multiple of 32
  if (i >= size) return;
  f32x4 v = *(const f32x4*)(u + i);
  for (int s = 1; s < slices; ++s) v += *(const f32x4*)(u + s * size + i);
  *(f32x4*)(u + i) = v;
}

// --------------------------------------------- u as an operand, from shared --

// Width of a staged row: the ranks rounded up to the K block (16, or 32 a
// step), plus four words that spread the rows over the banks.
__host__ __device__ inline int staged_width(int R) {
  return (R <= 16 ? 16 : (R + 31) / 32 * 32) + 4;
}

// Stages u of the tile's tokens as [token][rank] fp32, slices added in order.
template <int TT, int THREADS>
__device__ __forceinline__ void stage_u(const LowRankArgs& a, const float* u, int slices,
                                        int64_t t0, float* us) {
  const int rs = staged_width(a.R);
  for (int i = threadIdx.x; i < TT * (rs - 4); i += THREADS) {
    const int t = i % TT, r = i / TT;
    float v = 0.f;
    if (r < a.R && t0 + t < a.T) {
      const float* p = u + (int64_t)r * a.Tp + t0 + t;
      for (int s = 0; s < slices; ++s) v += p[(int64_t)s * a.R * a.Tp];
    }
    us[t * rs + r] = v;
  }
}

// Scales of a token row (one and one but for f16).
template <typename T>
__device__ __forceinline__ Pow2 row_pow2(const float* row, int R) {
  if constexpr (__is_same(T, _Float16)) {
    const int g = lane_id() / 16;
    float m = 0.f;
    for (int r = g * 4; r < staged_width(R) - 4; r += 16)
#pragma unroll
      for (int s = 0; s < 4; ++s) m = fmaxf(m, fabsf(row[r + s]));
    m = fmaxf(m, __shfl_xor(m, 16, kWave));
    m = fmaxf(m, __shfl_xor(m, 32, kWave));
    return pow2_of(m);
  } else {
    return Pow2{1.f, 1.f};
  }
}

// How a token row's ranks fill K blocks.  SMALL (R <= 16): one block; 16-bit
// types put hi in its lower half and lo in its upper, f32 uses four of the
// eight steps.  Otherwise 32 ranks a block, hi and lo apart.
template <typename T, bool SMALL>
__device__ __forceinline__ int rank_base(int step) {
  const int g = lane_id() / 16;
  if (!SMALL) return step * 32 + g * 8;
  return sizeof(T) == 4 ? g * 4 : (g % 2) * 8;
}
template <typename T, bool SMALL>
__device__ __forceinline__ Frag<T> u_frag(const float* row, int step, bool lo, float down) {
  const int r = rank_base<T, SMALL>(step);
  float v[8];
#pragma unroll
  for (int s = 0; s < 8; ++s)
    v[s] = SMALL && sizeof(T) == 4 && s >= 4 ? 0.f : row[r + s] * down;
  if (SMALL) lo = lane_id() >= 32;
  return split8<T>(v, lo);
}

// c + u F^T for one K block, F's fragment laid out the same way.
template <typename T, bool SMALL>
__device__ __forceinline__ f32x4 u_mma(const Frag<T>& hi, const Frag<T>& lo, const Frag<T>& f,
                                       f32x4 c) {
  if constexpr (SMALL && sizeof(T) == 4) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(hi.w[s]), __uint_as_float(f.w[s]),
                                               c, 0, 0, 0);
    return c;
  } else {
    c = mma(hi, f, c);
    if constexpr (!SMALL && sizeof(T) == 2) c = mma(lo, f, c);
    return c;
  }
}

// Fragment of B_ad's row o: ranks from rank_base, zero from the adapter's rank
// on (what lies there is not the adapter's).
template <typename T, bool SMALL>
__device__ __forceinline__ Frag<T> b_frag(const LowRankArgs& a, int ad, int64_t o, int rank,
                                          int step) {
  constexpr int W = SMALL && sizeof(T) == 4 ? 4 : 8;
  const int r = rank_base<T, SMALL>(step);
  const int64_t at = ((int64_t)ad * a.n_out + o) * a.R + r;
  const int cnt = clampi(rank - r, 0, W);
  const T* p = (const T*)a.B + at;
  if (cnt < W && at + 8 > (int64_t)a.n * a.n_out * a.R) return load8_count(p, cnt);
  if (W == 4 && at + 8 > (int64_t)a.n * a.n_out * a.R) return load8_count(p, cnt);
  Frag<T> f = load8(p);
  if (cnt < 8) mask8(f, (1u << cnt) - 1u);
  return f;
}

// Token order of the streaming kernels: result row m of product q stands for
// this token of the tile, so that a lane's rows over q are runs of eight
// (Q >= 2) or four tokens in memory.
template <int Q>
__device__ __forceinline__ int tile_token(int q, int m) {
  return Q == 1 ? m : (q / 2) * 32 + (m / 4) * 8 + (q % 2) * 4 + m % 4;
}

// The tile's u rows as operands: kept in registers for up to STEPS K blocks,
// read from shared memory again where there are more.
template <typename T, int Q, int STEPS, bool SMALL>
struct UOperand {
  Frag<T> hi[Q][STEPS > 0 ? STEPS : 1], lo[Q][STEPS > 0 ? STEPS : 1];
  float down[Q];
  f32x4 up[Q];
  const float* row[Q];
  int blocks;
  __device__ __forceinline__ UOperand(const LowRankArgs& a, const float* us) {
    const int m = lane_id() % 16, g = lane_id() / 16;
    blocks = SMALL ? 1 : (a.R + 31) / 32;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      row[q] = us + tile_token<Q>(q, m) * staged_width(a.R);
      const Pow2 p = row_pow2<T>(row[q], a.R);
      down[q] = p.down;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        up[q][i] = __is_same(T, _Float16) ? __shfl(p.up, g * 4 + i, kWave) : 1.f;
#pragma unroll
      for (int k = 0; k < STEPS; ++k) {
        hi[q][k] = u_frag<T, SMALL>(row[q], k, false, down[q]);
        if constexpr (!SMALL && sizeof(T) == 2) lo[q][k] = u_frag<T, SMALL>(row[q], k, true, down[q]);
      }
    }
  }
  // acc[q] += u_q F^T for block k (not yet scaled by up)
  __device__ __forceinline__ void product(int k, const Frag<T>& f, f32x4 (&acc)[Q]) const {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      if constexpr (STEPS > 0) {
        acc[q] = u_mma<T, SMALL>(hi[q][k], lo[q][k], f, acc[q]);
      } else {
        const Frag<T> h = u_frag<T, SMALL>(row[q], k, false, down[q]);
        const Frag<T> l = sizeof(T) == 2 ? u_frag<T, SMALL>(row[q], k, true, down[q]) : h;
        acc[q] = u_mma<T, SMALL>(h, l, f, acc[q]);
      }
    }
  }
};

// Adapters of the result rows a lane holds.
template <int Q>
__device__ __forceinline__ void row_adapters(const int* tok, int (&ra)[Q][4]) {
  const int g = lane_id() / 16;
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) ra[q][i] = tok[tile_token<Q>(q, g * 4 + i)];
}

template <int TT, int THREADS>
__device__ __forceinline__ void load_tokad(const LowRankArgs& a, int64_t t0, int* tok) {
  for (int t = threadIdx.x; t < TT; t += THREADS) tok[t] = t0 + t < a.T ? a.tokad[t0 + t] : -1;
}

// ----------------------------------------------------------------- expand --

// out = y + B u.  A wave takes 16 output rows at a time: y's values go through
// registers in the products' own layout, eight tokens (16 bytes in f16) a
// lane, and are stored once.  out may be y itself.
template <typename T, int Q, int STEPS, bool SMALL>
__global__ __launch_bounds__(kThreads) void lowrank_expand_kernel(LowRankArgs a, int slices,
                                                                  int rows_per_block,
                                                                  int row_blocks) {
  constexpr int TT = 16 * Q, C = Q == 1 ? 4 : 8, P = TT / (4 * C);
  extern __shared__ float us[];
  __shared__ int tok[TT];
  const int lane = lane_id(), n = lane % 16, g = lane / 16, wave = threadIdx.x / kWave;
  const int block = blockIdx.x % row_blocks;
  const int64_t t0 = (int64_t)(blockIdx.x / row_blocks) * TT;
  load_tokad<TT, kThreads>(a, t0, tok);
  stage_u<TT, kThreads>(a, a.u, slices, t0, us);
  __syncthreads();
  const UOperand<T, Q, STEPS, SMALL> u(a, us);
  int ra[Q][4];
  row_adapters<Q>(tok, ra);
  const int64_t o_end0 = (int64_t)(block + 1) * rows_per_block;
  const int64_t o_end = o_end0 < a.n_out ? o_end0 : a.n_out;
  const int64_t left = a.T - t0;
  const T* y = (const T*)a.y + t0;
  T* out = (T*)a.out + t0;
  for (int64_t ob = (int64_t)block * rows_per_block + wave * 16; ob < o_end;
       ob += kWaves * 16) {
    const int64_t o = ob + n < a.n_out ? ob + n : a.n_out - 1;
    float v[P][C];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int t = p * 4 * C + g * C;
      load_chunk<T, C>(y + o * a.ldy + t, clampi(left - t, 0, C), v[p]);
    }
    AdapterWalk<TT> walk(tok);
    int ad;
    while (walk.next(ad)) {
      const int rank = rank_of(a, ad);
      f32x4 acc[Q];
#pragma unroll
      for (int q = 0; q < Q; ++q) acc[q] = f32x4{0.f, 0.f, 0.f, 0.f};
      const int blocks = STEPS > 0 ? STEPS : u.blocks;
      for (int k = 0; k < blocks; ++k) u.product(k, b_frag<T, SMALL>(a, ad, o, rank, k), acc);
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float& d = v[q * 4 / C][(q * 4) % C + i];
          d = ra[q][i] == ad ? d + acc[q][i] * u.up[q][i] : d;
        }
    }
    if (ob + n < a.n_out) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int t = p * 4 * C + g * C;
        store_chunk<T, C>(out + o * a.ldo + t, clampi(left - t, 0, C), v[p]);
      }
    }
  }
}

// --------------------------------------------------------------------- dx --

// dx = A^T du, zero where a token has no adapter.  A's rows run along the
// features: eight ranks of V features a lane are turned as x is in shrink, and
// product j gives the features f0 + V n + j.
template <typename T, int Q, int V, int STEPS, bool SMALL>
__global__ __launch_bounds__(kThreads) void lowrank_dx_kernel(LowRankArgs a, int slices,
                                                              int rows_per_block, int row_blocks) {
  constexpr int TT = 16 * Q, C = Q == 1 ? 4 : 8, P = TT / (4 * C);
  constexpr int KR = SMALL && sizeof(T) == 4 ? 4 : 8;  // ranks a lane holds of a block
  extern __shared__ float us[];
  __shared__ int tok[TT];
  const int lane = lane_id(), n = lane % 16, g = lane / 16, wave = threadIdx.x / kWave;
  const int block = blockIdx.x % row_blocks;
  const int64_t t0 = (int64_t)(blockIdx.x / row_blocks) * TT;
  load_tokad<TT, kThreads>(a, t0, tok);
  stage_u<TT, kThreads>(a, a.du, slices, t0, us);
  __syncthreads();
  const UOperand<T, Q, STEPS, SMALL> u(a, us);
  int ra[Q][4];
  row_adapters<Q>(tok, ra);
  const int64_t f_end0 = (int64_t)(block + 1) * rows_per_block;
  const int64_t f_end = f_end0 < a.n_in ? f_end0 : a.n_in;
  const int64_t left = a.T - t0;
  T* out = (T*)a.out + t0;
  for (int64_t fb = (int64_t)block * rows_per_block + wave * 16 * V; fb < f_end;
       fb += kWaves * 16 * V) {
    const int64_t f = fb + n * V < a.n_in - V ? fb + n * V : a.n_in - V;
    f32x4 res[V][Q];
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int q = 0; q < Q; ++q) res[j][q] = f32x4{0.f, 0.f, 0.f, 0.f};
    AdapterWalk<TT> walk(tok);
    int ad;
    while (walk.next(ad)) {
      const int rank = rank_of(a, ad);
      const T* A = (const T*)a.A + (int64_t)ad * a.R * a.n_in + f;
      f32x4 acc[V][Q];
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int q = 0; q < Q; ++q) acc[j][q] = f32x4{0.f, 0.f, 0.f, 0.f};
      const int blocks = STEPS > 0 ? STEPS : u.blocks;
      for (int k = 0; k < blocks; ++k) {
        const int r = rank_base<T, SMALL>(k);
        Row<T, V> rows[8];
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          zero_row(rows[s]);
          if (s < KR && r + s < rank) rows[s] = load_row<T, V>(A + (int64_t)(r + s) * a.n_in);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) u.product(k, column<T, V>(rows, j), acc[j]);
      }
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            res[j][q][i] = ra[q][i] == ad ? acc[j][q][i] * u.up[q][i] : res[j][q][i];
    }
    if (fb + n * V < a.n_in) {
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const int t = p * 4 * C + g * C;
          float v[C];
#pragma unroll
          for (int e = 0; e < C; ++e) v[e] = res[j][(p * C + e) / 4][e % 4];
          store_chunk<T, C>(out + (f + j) * a.ldo + t, clampi(left - t, 0, C), v);
        }
    }
  }
}

// ------------------------------------------------------------------ outer --

// dA_a = sum over the adapter's tokens of du x^T, and dB_a = sum of dy u^T:
// one workgroup takes 16 FF features of x (or of dy), one adapter and up to 64
// ranks.  Its waves walk the 32-token blocks in turn, skip those without a
// token of the adapter, and mask the others' tokens out of both operands; the
// waves' sums are added in a fixed order.  f16: u's block is scaled by rank
// (its largest |u| among the block's tokens of this adapter), and the block's
// product is scaled back in fp32.
template <typename T, int FF, int NR>
__global__ __launch_bounds__(kOuterThreads) void lowrank_outer_kernel(LowRankArgs a, int xblocks) {
  __shared__ f32x4 red[kOuterWaves / 2 * FF * NR * kWave];
  const int lane = lane_id(), n = lane % 16, g = lane / 16, wave = threadIdx.x / kWave;
  const bool is_x = (int)blockIdx.x < xblocks;
  const int64_t F = is_x ? a.n_in : a.n_out, ld = is_x ? a.ldx : a.ldy;
  const T* src = (const T*)(is_x ? a.x : a.y);
  const float* u = is_x ? a.du : a.u;
  const int64_t f0 = (int64_t)(is_x ? blockIdx.x : blockIdx.x - xblocks) * (16 * FF);
  const int ad = blockIdx.y, r0 = blockIdx.z * 64;
  const T* row[FF];
#pragma unroll
  for (int k = 0; k < FF; ++k) {
    const int64_t f = f0 + k * 16 + n;
    row[k] = src + (f < F ? f : F - 1) * ld;
  }
  const float* urow[NR];
#pragma unroll
  for (int q = 0; q < NR; ++q) {
    const int r = r0 + q * 16 + n;
    urow[q] = u + (int64_t)(r < a.R ? r : a.R - 1) * a.Tp;
  }
  f32x4 acc[FF * NR];
#pragma unroll
  for (int k = 0; k < FF * NR; ++k) acc[k] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int64_t blocks = cdiv(a.T, 32);
  for (int64_t b = wave; b < blocks; b += kOuterWaves) {
    const int64_t t = b * 32 + g * 8;
    const int cnt = clampi(a.T - t, 0, 8);
    uint32_t m = 0;
    if (cnt == 8) {
      int ta[8];
      __builtin_memcpy(ta, __builtin_assume_aligned(a.tokad + t, 16), sizeof(ta));
#pragma unroll
      for (int s = 0; s < 8; ++s) m |= (ta[s] == ad ? 1u : 0u) << s;
    } else {
      for (int s = 0; s < cnt; ++s) m |= (a.tokad[t + s] == ad ? 1u : 0u) << s;
    }
    if (__ballot(m != 0) == 0) continue;
    Frag<T> fx[FF];
#pragma unroll
    for (int k = 0; k < FF; ++k) fx[k] = cnt == 8 ? load8(row[k] + t) : load8_count(row[k] + t, cnt);
    float uv[NR][8];
#pragma unroll
    for (int q = 0; q < NR; ++q)
      __builtin_memcpy(uv[q], __builtin_assume_aligned(urow[q] + t, 16), sizeof(uv[q]));
    if (__ballot(m != 255u) != 0) {
#pragma unroll
      for (int k = 0; k < FF; ++k) mask8(fx[k], m);
#pragma unroll
      for (int q = 0; q < NR; ++q)
#pragma unroll
        for (int s = 0; s < 8; ++s) uv[q][s] = (m >> s) & 1u ? uv[q][s] : 0.f;
    }
#pragma unroll
    for (int q = 0; q < NR; ++q) {
      if constexpr (__is_same(T, _Float16)) {
        float big = 0.f;
#pragma unroll
        for (int s = 0; s < 8; ++s) big = fmaxf(big, fabsf(uv[q][s]));
        big = fmaxf(big, __shfl_xor(big, 16, kWave));
        big = fmaxf(big, __shfl_xor(big, 32, kWave));
        const Pow2 p = pow2_of(big);
#pragma unroll
        for (int s = 0; s < 8; ++s) uv[q][s] *= p.down;
        const Frag<T> hi = split8<T>(uv[q], false), lo = split8<T>(uv[q], true);
#pragma unroll
        for (int k = 0; k < FF; ++k) {
          const f32x4 c = mma(fx[k], lo, mma(fx[k], hi, f32x4{0.f, 0.f, 0.f, 0.f}));
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[k * NR + q][i] = __builtin_fmaf(c[i], p.up, acc[k * NR + q][i]);
        }
      } else {
        const Frag<T> hi = split8<T>(uv[q], false);
#pragma unroll
        for (int k = 0; k < FF; ++k) acc[k * NR + q] = mma(fx[k], hi, acc[k * NR + q]);
        if constexpr (sizeof(T) == 2) {
          const Frag<T> lo = split8<T>(uv[q], true);
#pragma unroll
          for (int k = 0; k < FF; ++k) acc[k * NR + q] = mma(fx[k], lo, acc[k * NR + q]);
        }
      }
    }
  }
  wave_tree_sum<FF * NR, kOuterWaves>(acc, red);
  if (wave != 0) return;
  const int rank = rank_of(a, ad);
  T* out = (T*)(is_x ? a.dA : a.dB) + (int64_t)ad * a.R * F;
#pragma unroll
  for (int k = 0; k < FF; ++k)
#pragma unroll
    for (int q = 0; q < NR; ++q) {
      const int r = r0 + q * 16 + n;
      const int64_t f = f0 + k * 16 + g * 4;
      const int cnt = clampi(F - f, 0, 4);
      if (r >= a.R || cnt == 0) continue;
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = r < rank ? acc[k * NR + q][i] : 0.f;
      if (is_x) {
        store_chunk<T, 4>(out + (int64_t)r * F + f, cnt, v);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < cnt) store_bits(out + (f + i) * a.R + r, out_bits(v[i], (T*)nullptr));
      }
    }
}

// ---------------------------------------------------------------- project --

// y = W x + B u on a tile of 16 V tokens: a workgroup takes 16 MO rows of W,
// its waves a slice of the features each; x comes as the fragments that the
// shrink kernel packed.  The waves' sums meet in shared memory, where the
// adapters' part is added.
template <typename T, int V, int MO, bool SMALL>
__global__ __launch_bounds__(kOuterThreads) void lowrank_project_kernel(LowRankArgs a, int slices,
                                                                        int row_blocks) {
  constexpr int TT = 16 * V;
  extern __shared__ float us[];
  __shared__ f32x4 red[kOuterWaves * MO * V * kWave];
  __shared__ int tok[TT];
  const int lane = lane_id(), n = lane % 16, g = lane / 16, wave = threadIdx.x / kWave;
  const int block = blockIdx.x % row_blocks;
  const int64_t tile = blockIdx.x / row_blocks;
  int64_t t0 = tile * TT;
  if (t0 > a.T - TT) t0 = a.T > TT ? a.T - TT : 0;
  load_tokad<TT, kOuterThreads>(a, t0, tok);
  stage_u<TT, kOuterThreads>(a, a.u, slices, t0, us);
  const int64_t steps = cdiv(a.n_in, 32);
  const int64_t s0 = steps * wave / kOuterWaves, s1 = steps * (wave + 1) / kOuterWaves;
  const int64_t o0 = (int64_t)block * (16 * MO);
  const T* w[MO];
#pragma unroll
  for (int k = 0; k < MO; ++k) {
    const int64_t o = o0 + k * 16 + n;
    w[k] = (const T*)a.W + (o < a.n_out ? o : a.n_out - 1) * a.ldw;
  }
  const T* xp = (const T*)a.packed + (tile * steps * V * kWave + lane) * 8;
  f32x4 acc[MO * V];
#pragma unroll
  for (int k = 0; k < MO * V; ++k) acc[k] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int64_t whole = a.n_in / 32 < s1 ? a.n_in / 32 : s1;
  int64_t s = s0;
  for (; s < whole; ++s) {
    Frag<T> fw[MO], fx[V];
#pragma unroll
    for (int k = 0; k < MO; ++k) fw[k] = load8(w[k] + s * 32 + g * 8);
#pragma unroll
    for (int j = 0; j < V; ++j) fx[j] = load8(xp + (s * V + j) * kWave * 8);
#pragma unroll
    for (int k = 0; k < MO; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) acc[k * V + j] = mma(fx[j], fw[k], acc[k * V + j]);
  }
  if (s < s1) {
    const int cnt = clampi(a.n_in - s * 32 - g * 8, 0, 8);
#pragma unroll
    for (int k = 0; k < MO; ++k) {
      const Frag<T> fw = load8_count(w[k] + s * 32 + g * 8, cnt);
#pragma unroll
      for (int j = 0; j < V; ++j)
        acc[k * V + j] = mma(load8(xp + (s * V + j) * kWave * 8), fw, acc[k * V + j]);
    }
  }
#pragma unroll
  for (int k = 0; k < MO * V; ++k) red[(wave * MO * V + k) * kWave + lane] = acc[k];
  __syncthreads();
  const int64_t lim = a.T - V;
  const int blocks = SMALL ? 1 : (a.R + 31) / 32;
  for (int k = wave; k < MO * V; k += kOuterWaves) {
    f32x4 v = red[k * kWave + lane];
#pragma unroll
    for (int h = 1; h < kOuterWaves; ++h) v += red[(h * MO * V + k) * kWave + lane];
    const int j = k % V;
    const int64_t o = o0 + k / V * 16 + n, oc = o < a.n_out ? o : a.n_out - 1;
    auto local = [&](int m) {
      const int64_t t = t0 + m * V;
      return (int)((t < lim ? t : lim) - t0) + j;
    };
    const float* row = us + local(n) * staged_width(a.R);
    const Pow2 p = row_pow2<T>(row, a.R);
    AdapterWalk<TT> walk(tok);
    int ad;
    while (walk.next(ad)) {
      const int rank = rank_of(a, ad);
      f32x4 c = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int b = 0; b < blocks; ++b) {
        const Frag<T> hi = u_frag<T, SMALL>(row, b, false, p.down);
        const Frag<T> lo = u_frag<T, SMALL>(row, b, true, p.down);
        c = u_mma<T, SMALL>(hi, lo, b_frag<T, SMALL>(a, ad, oc, rank, b), c);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float up = __is_same(T, _Float16) ? __shfl(p.up, g * 4 + i, kWave) : 1.f;
        v[i] = tok[local(g * 4 + i)] == ad ? v[i] + c[i] * up : v[i];
      }
    }
    if (o < a.n_out) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        store_bits((T*)a.out + o * a.ldo + t0 + local(g * 4 + i), out_bits(v[i], (T*)nullptr));
    }
  }
}

// --------------------------------------------------------------- launches --

constexpr int64_t kFillBlocks = 512;  // two workgroups on each of the 256 CUs

// Tokens a lane holds of a row in the shrink kernel.
int token_width(int op, int dtype, int64_t T) {
  const int most = op == kLowRankProject ? 4 : dtype == kF32 ? 4 : 8;
  int v = 1;
  while (v < most && T > 16 * v) v *= 2;
  return v;
}

// Distinct adapters that share a tile are spread over this many workgroups:
// the tile's mean number of requests, at most the adapters there are.
int adapter_groups(int64_t T, int64_t S, int64_t n, int64_t tile) {
  const int64_t t = T < tile ? T : tile;
  int64_t g = S * t / (T > 0 ? T : 1);
  g = g < n ? g : n;
  return (int)(g < 1 ? 1 : g > 64 ? 64 : g);
}

int slices_for(int64_t blocks, int64_t K) {
  int64_t s = cdiv(kFillBlocks, blocks > 0 ? blocks : 1);
  const int64_t most = cdiv(K, 32) / (2 * kWaves);  // two steps a wave at least
  s = s < most ? s : most;
  return (int)(s < 1 ? 1 : s > 16 ? 16 : s);
}

template <typename T, int V, bool BACKWARD, bool PACK>
hipError_t shrink_v(const LowRankArgs& a, const LowRankLayout& l, hipStream_t s) {
  const int rcs = (int)cdiv(a.R, 64);
  ShrinkJob jx{a.x, a.A, a.u, a.ldx, a.n_in, l.slices_u};
  ShrinkJob jy{a.y, a.B, a.du, a.ldy, a.n_out, l.slices_du};
  const dim3 grid((unsigned)cdiv(a.T, 16 * V), (unsigned)(l.groups * rcs),
                  (unsigned)(l.slices_u + (BACKWARD ? l.slices_du : 0)));
  const int nr = a.R <= 16 ? 1 : a.R <= 32 ? 2 : 4;
  if (nr == 1)
    hipLaunchKernelGGL((lowrank_shrink_kernel<T, V, 1, BACKWARD, PACK>), grid, dim3(kThreads), 0, s,
                       a, jx, jy, l.groups);
  else if (nr == 2)
    hipLaunchKernelGGL((lowrank_shrink_kernel<T, V, 2, BACKWARD, PACK>), grid, dim3(kThreads), 0, s,
                       a, jx, jy, l.groups);
  else
    hipLaunchKernelGGL((lowrank_shrink_kernel<T, V, 4, BACKWARD, PACK>), grid, dim3(kThreads), 0, s,
                       a, jx, jy, l.groups);
  return hipGetLastError();
}

template <typename T, bool BACKWARD, bool PACK>
hipError_t shrink(const LowRankArgs& a, const LowRankLayout& l, hipStream_t s) {
  switch (l.width) {
    case 1: return shrink_v<T, 1, BACKWARD, PACK>(a, l, s);
    case 2: return shrink_v<T, 2, BACKWARD, PACK>(a, l, s);
    case 4: return shrink_v<T, 4, BACKWARD, PACK>(a, l, s);
  }
  if constexpr (sizeof(T) == 2 && !PACK) return shrink_v<T, 8, BACKWARD, PACK>(a, l, s);
  return hipErrorInvalidValue;
}

size_t staged_bytes(int64_t tokens, int R) { return (size_t)tokens * staged_width(R) * 4; }

// Rows a workgroup of expand or dx takes: enough that staging u is a small
// part of the streams, few enough that the launch fills the GPU.
int64_t rows_per_block(int64_t rows, int64_t tiles, int64_t unit) {
  int64_t blocks = cdiv(4 * kFillBlocks, tiles);
  int64_t per = cdiv(cdiv(rows, blocks), unit) * unit;
  return per < 512 ? per : cdiv(512, unit) * unit;
}

template <typename T, int Q>
hipError_t expand_q(const LowRankArgs& a, const LowRankLayout& l, hipStream_t s) {
  const int64_t tiles = cdiv(a.T, 16 * Q), per = rows_per_block(a.n_out, tiles, 16 * kWaves);
  const int64_t rb = cdiv(a.n_out, per);
  const dim3 grid((unsigned)(rb * tiles));
  const size_t lds = staged_bytes(16 * Q, a.R);
  if (a.R <= 16)
    hipLaunchKernelGGL((lowrank_expand_kernel<T, Q, 1, true>), grid, dim3(kThreads), lds, s, a,
                       l.slices_u, (int)per, (int)rb);
  else if (a.R <= 32)
    hipLaunchKernelGGL((lowrank_expand_kernel<T, Q, 1, false>), grid, dim3(kThreads), lds, s, a,
                       l.slices_u, (int)per, (int)rb);
  else if (a.R <= 64)
    hipLaunchKernelGGL((lowrank_expand_kernel<T, Q, 2, false>), grid, dim3(kThreads), lds, s, a,
                       l.slices_u, (int)per, (int)rb);
  else
    hipLaunchKernelGGL((lowrank_expand_kernel<T, Q, 0, false>), grid, dim3(kThreads), lds, s, a,
                       l.slices_u, (int)per, (int)rb);
  return hipGetLastError();
}

template <typename T, int Q, int V>
hipError_t dx_qv(const LowRankArgs& a, hipStream_t s) {
  const int64_t tiles = cdiv(a.T, 16 * Q), per = rows_per_block(a.n_in, tiles, 16 * V * kWaves);
  const int64_t rb = cdiv(a.n_in, per);
  const dim3 grid((unsigned)(rb * tiles));
  const size_t lds = staged_bytes(16 * Q, a.R);
  if (a.R <= 16)
    hipLaunchKernelGGL((lowrank_dx_kernel<T, Q, V, 1, true>), grid, dim3(kThreads), lds, s, a, 1,
                       (int)per, (int)rb);
  else if (a.R <= 32)
    hipLaunchKernelGGL((lowrank_dx_kernel<T, Q, V, 1, false>), grid, dim3(kThreads), lds, s, a, 1,
                       (int)per, (int)rb);
  else if (a.R <= 64)
    hipLaunchKernelGGL((lowrank_dx_kernel<T, Q, V, 2, false>), grid, dim3(kThreads), lds, s, a, 1,
                       (int)per, (int)rb);
  else
    hipLaunchKernelGGL((lowrank_dx_kernel<T, Q, V, 0, false>), grid, dim3(kThreads), lds, s, a, 1,
                       (int)per, (int)rb);
  return hipGetLastError();
}

template <typename T, int FF>
hipError_t outer_f(const LowRankArgs& a, hipStream_t s) {
  const int xblocks = (int)cdiv(a.n_in, 16 * FF), yblocks = (int)cdiv(a.n_out, 16 * FF);
  const dim3 grid((unsigned)(xblocks + yblocks), (unsigned)a.n, (unsigned)cdiv(a.R, 64));
  if (a.R <= 16)
    hipLaunchKernelGGL((lowrank_outer_kernel<T, FF, 1>), grid, dim3(kOuterThreads), 0, s, a, xblocks);
  else if (a.R <= 32)
    hipLaunchKernelGGL((lowrank_outer_kernel<T, FF, 2>), grid, dim3(kOuterThreads), 0, s, a, xblocks);
  else
    hipLaunchKernelGGL((lowrank_outer_kernel<T, FF, 4>), grid, dim3(kOuterThreads), 0, s, a, xblocks);
  return hipGetLastError();
}

template <typename T, int V, int MO>
hipError_t project_v(const LowRankArgs& a, const LowRankLayout& l, hipStream_t s) {
  const int64_t rb = cdiv(a.n_out, 16 * MO);
  const dim3 grid((unsigned)(rb * cdiv(a.T, 16 * V)));
  const size_t lds = staged_bytes(16 * V, a.R);
  if (a.R <= 16)
    hipLaunchKernelGGL((lowrank_project_kernel<T, V, MO, true>), grid, dim3(kOuterThreads), lds, s,
                       a, l.slices_u, (int)rb);
  else
    hipLaunchKernelGGL((lowrank_project_kernel<T, V, MO, false>), grid, dim3(kOuterThreads), lds, s,
                       a, l.slices_u, (int)rb);
  return hipGetLastError();
}

template <typename T>
hipError_t add_t(const LowRankArgs& a, const LowRankLayout& l, hipStream_t s) {
  hipError_t e = shrink<T, false, false>(a, l, s);
  if (e != hipSuccess) return e;
  return a.T <= 16 * 8 ? expand_q<T, 1>(a, l, s) : expand_q<T, 4>(a, l, s);
}

template <typename T>
hipError_t backward_t(const LowRankArgs& a, const LowRankLayout& l, hipStream_t s) {
  if (a.T == 0) return outer_f<T, 2>(a, s);  // zeros
  hipError_t e = shrink<T, true, false>(a, l, s);
  if (e != hipSuccess) return e;
  if (l.slices_u > 1 || l.slices_du > 1) {
    const dim3 grid((unsigned)cdiv((int64_t)a.R * a.Tp, 4 * kThreads), 2);
    hipLaunchKernelGGL(lowrank_join_kernel, grid, dim3(kThreads), 0, s, a, l.slices_u, l.slices_du);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  e = a.n_in < 4 ? dx_qv<T, 4, 1>(a, s) : dx_qv<T, 4, 4>(a, s);
  if (e != hipSuccess) return e;
  return outer_f<T, 2>(a, s);
}

template <typename T>
hipError_t project_t(const LowRankArgs& a, const LowRankLayout& l, hipStream_t s) {
  hipError_t e = shrink<T, false, true>(a, l, s);
  if (e != hipSuccess) return e;
  switch (l.width) {
    case 1: return project_v<T, 1, 1>(a, l, s);
    case 2: return project_v<T, 2, 1>(a, l, s);
    default: return project_v<T, 4, 1>(a, l, s);
  }
}

}  // namespace

LowRankLayout lowrank_layout(int op, int dtype, int64_t T, int64_t S, int64_t n, int64_t R,
                             int64_t n_in, int64_t n_out) {
  LowRankLayout l{};
  const int64_t eb = dtype == kF32 ? 4 : 2;
  l.Tp = cdiv(T, 32) * 32;
  l.width = token_width(op, dtype, T);
  l.groups = adapter_groups(T, S, n, 16 * l.width);
  const int64_t tiles = cdiv(T, 16 * l.width);
  const int64_t blocks = tiles * l.groups * cdiv(R, 64) * (op == kLowRankBackward ? 2 : 1);
  l.slices_u = slices_for(blocks, n_in);
  l.slices_du = op == kLowRankBackward ? slices_for(blocks, n_out) : 0;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  l.at_tokad = take((size_t)l.Tp * 4);
  l.at_u = take((size_t)l.slices_u * R * l.Tp * 4);
  l.at_du = take((size_t)l.slices_du * R * l.Tp * 4);
  l.at_packed = take(op == kLowRankProject
                         ? (size_t)(tiles * cdiv(n_in, 32) * l.width * kWave * 8 * eb)
                         : 0);
  l.bytes = at;
  return l;
}

hipError_t launch_lowrank(int op, int dtype, LowRankArgs a, void* ws, hipStream_t s) {
  const LowRankLayout l = lowrank_layout(op, dtype, a.T, a.S, a.n, a.R, a.n_in, a.n_out);
  char* w = (char*)ws;
  a.Tp = l.Tp;
  a.tokad = (int32_t*)(w + l.at_tokad);
  a.u = (float*)(w + l.at_u);
  a.du = (float*)(w + l.at_du);
  a.packed = w + l.at_packed;
  switch (dtype) {
    case kF32:
      return op == kLowRankAdd ? add_t<float>(a, l, s)
             : op == kLowRankProject ? project_t<float>(a, l, s) : backward_t<float>(a, l, s);
    case kF16:
      return op == kLowRankAdd ? add_t<_Float16>(a, l, s)
             : op == kLowRankProject ? project_t<_Float16>(a, l, s) : backward_t<_Float16>(a, l, s);
    case kBF16:
      return op == kLowRankAdd ? add_t<bf16_t>(a, l, s)
             : op == kLowRankProject ? project_t<bf16_t>(a, l, s) : backward_t<bf16_t>(a, l, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace spops
