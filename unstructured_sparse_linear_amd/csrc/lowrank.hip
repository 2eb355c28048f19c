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
//   pack     adds the slices and splits them into operands, where they are
//            read many times
//   expand   y + B u
//   gradients  dA and dB, one workgroup per adapter and 32 or 64 features, and
//            dx = A^T du
//   project  W x + B u on the tokens of a decode step
//   few      either forward on a few tokens in one launch
// Requests meet the tiles only through each token's adapter, which the shrink
// kernel finds and writes once.  A tile whose tokens have several adapters is
// computed once per distinct adapter and the results selected per token (never
// multiplied by zero: another request's NaN or infinity stays its own).
#include "kernels.h"
#include "lowrank.h"

namespace spops {
namespace {

template <int N>
struct Int {
  static constexpr int value = N;
};

constexpr int kThreads = 256;     // four waves
constexpr int kWaves = kThreads / kWave;
constexpr int kProjectWaves = 8;  // that stream W

// Workgroup b of N runs on XCD b % 8.  Each XCD takes one contiguous part of
// the work list: neighbouring tiles share lines, factors and pages of one L2.
__device__ __forceinline__ uint32_t xcd_chunk(uint32_t b, uint32_t N) {
  const uint32_t x = b % 8, q = N / 8, r = N % 8;
  return x * q + (x < r ? x : r) + b / 8;
}

__device__ __forceinline__ uint32_t block_of(const LowRankArgs& a) { return a.block0 + blockIdx.x; }

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
    int ad = a.adapter[i];
    const int64_t lo = b > t0 ? b : t0, hi = e < last ? e : last;
    if (lo < hi) {
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

// Eight rows of V tokens from p on.
template <typename T, int V>
__device__ __forceinline__ void shrink_load(const T* p, int64_t ld, Row<T, V> (&r)[8]) {
#pragma unroll
  for (int s = 0; s < 8; ++s) r[s] = load_row<T, V>(p + s * ld);
}
// The `left` (0 or less: none) of them that there are, zeros for the rest; the
// others' addresses are moved back to the last there is.
template <typename T, int V>
__device__ __forceinline__ void shrink_load_count(const T* p, int64_t ld, int64_t left,
                                                  Row<T, V> (&r)[8]) {
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    r[s] = load_row<T, V>(p + (s < left ? s : left - 1) * ld);
    if (s >= left) zero_row(r[s]);
    __builtin_amdgcn_sched_barrier(0);  // rare: one address at a time
  }
}

// Accumulates the steps [s0, s1) of 32 features for the tokens tok..tok+V-1 of
// each lane and 16 NR ranks from r0.  x is read V tokens wide, eight rows a
// lane, and turned in registers; the same turn serves a factor stored [K][R].
// Two steps' rows are in flight where the sums leave room for them, at two waves a
// SIMD (67 MB of x and dy, 16 ranks: 18.8 us; one step at three waves 19.7, at four,
// with registers in memory, 22.1).
template <typename T, int V, int NR, bool TR, bool PACK>
__device__ __forceinline__ void shrink_steps(const T* x, int64_t ldx, int64_t K, const T* f, int R,
                                             int r0, int64_t tok, int64_t s0, int64_t s1,
                                             f32x4 (&acc)[NR * V], T* packed) {
  const int lane = lane_id(), n = lane % 16, g = lane / 16;
  const int64_t k0 = s0 * 32 + g * 8, whole = K / 32 < s1 ? K / 32 : s1;
  const T* xp = x + k0 * ldx + tok;
  const T* fp[TR ? 1 : NR];
  if constexpr (TR) {
    fp[0] = f + k0 * R + (r0 + n * NR < R - NR ? r0 + n * NR : R - NR);
  } else {
#pragma unroll
    for (int q = 0; q < NR; ++q) {
      const int r = r0 + q * 16 + n;
      fp[q] = f + (int64_t)(r < R ? r : R - 1) * K + k0;
    }
  }
  constexpr int D = V * NR <= 8 ? 2 : 1;  // steps in flight
  Row<T, V> xr[D][8];
  auto compute = [&](int64_t step, const Row<T, V>(&rows)[8], const Frag<T>(&ff)[NR]) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const Frag<T> fx = column<T, V>(rows, j);
      if (PACK && packed)
        __builtin_memcpy(packed + ((step * V + j) * kWave + lane) * 8, &fx, sizeof(fx));
#pragma unroll
      for (int q = 0; q < NR; ++q) acc[q * V + j] = mma(fx, ff[q], acc[q * V + j]);
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d) {
    if (s0 + d < whole) shrink_load<T, V>(xp, ldx, xr[d]);
    if (s0 + d < whole) xp += 32 * ldx;
  }
#pragma unroll 1
  for (int64_t at = s0; at < whole; at += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int64_t step = at + d;
      if (d > 0 && step >= whole) break;
      Frag<T> ff[NR];
      if constexpr (TR) {
        Row<T, NR> ft[8];
        shrink_load<T, NR>(fp[0], R, ft);
        fp[0] += 32 * (int64_t)R;
#pragma unroll
        for (int q = 0; q < NR; ++q) ff[q] = column<T, NR>(ft, q);
      } else {
#pragma unroll
        for (int q = 0; q < NR; ++q) {
          ff[q] = load8(fp[q]);
          fp[q] += 32;
        }
      }
      compute(step, xr[d], ff);
      if (step + D < whole) {
        shrink_load<T, V>(xp, ldx, xr[d]);
        xp += 32 * ldx;
      }
    }
  }
  if (s0 < s1 && whole < s1) {  // the features past the last 32
    const int64_t left = K - whole * 32 - g * 8;
    shrink_load_count<T, V>(xp, ldx, left, xr[0]);
    Frag<T> ff[NR];
    if constexpr (TR) {
      Row<T, NR> ft[8];
      shrink_load_count<T, NR>(fp[0], R, left, ft);
#pragma unroll
      for (int q = 0; q < NR; ++q) ff[q] = column<T, NR>(ft, q);
    } else {
#pragma unroll
      for (int q = 0; q < NR; ++q) ff[q] = load8_count(fp[q], clampi(left, 0, 8));
    }
    compute(whole, xr[0], ff);
  }
}

// One exchange between the waves w and w ^ BIT: of 2 H tiles each, one ends with
// the sums of the lower half, the other with those of the upper.
template <int H, int BIT, int N>
__device__ __forceinline__ void exchange(f32x4 (&acc)[N], f32x4* red) {
  const int wave = threadIdx.x / kWave, lane = lane_id();
  const bool upper = __builtin_amdgcn_readfirstlane(wave & BIT);
  if (upper) {
#pragma unroll
    for (int k = 0; k < H; ++k) {
      red[(wave * H + k) * kWave + lane] = acc[k];
      acc[k] = acc[k + H];
    }
  } else {
#pragma unroll
    for (int k = 0; k < H; ++k) red[(wave * H + k) * kWave + lane] = acc[k + H];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < H; ++k) acc[k] += red[((wave ^ BIT) * H + k) * kWave + lane];
  __syncthreads();
}

// Sums the four waves' N tiles: each wave ends with N / 4 of them, in
// acc[0..N/4), which are tiles wave * N / 4 and on (N >= 4); or wave 0 with all.
template <int N>
__device__ __forceinline__ void spread_sum(f32x4 (&acc)[N], f32x4* red) {
  static_assert(kWaves == 4, "two exchanges");
  if constexpr (N < 4) {
    wave_tree_sum<N, kWaves>(acc, red);
  } else {
    exchange<N / 2, 2>(acc, red);
    exchange<N / 4, 1>(acc, red);
  }
}

template <typename T, int V, int NR, bool TR, bool PACK>
__device__ __forceinline__ void shrink_tile(const LowRankArgs& a, const ShrinkJob& job, int slice,
                                            int tile_id, int part, bool first, int groups,
                                            f32x4* red, TokenTile<16 * V>& tile) {
  constexpr int TT = 16 * V, N = NR * V;
  const int lane = lane_id(), n = lane % 16, g = lane / 16, wave = threadIdx.x / kWave;
  // the last tile is moved back to end at T (its shared tokens get the same
  // values twice), and a lane's V tokens are moved back likewise: no load
  // passes the end of a row
  int64_t t0 = (int64_t)tile_id * TT;
  if (t0 > a.T - TT) t0 = a.T > TT ? a.T - TT : 0;
  const int64_t lim = a.T - V;
  const int64_t tok = t0 + n * V < lim ? t0 + n * V : lim;
  const int64_t steps = cdiv(job.K, 32), units = (int64_t)job.slices * kWaves;
  const int64_t unit = (int64_t)slice * kWaves + wave;
  const int64_t s0 = steps * unit / units, s1 = steps * (unit + 1) / units;
  const T* x = (const T*)job.x;
  token_adapters<TT, kThreads>(a, t0, tile);
  const int rc = part / groups, group = part % groups;
  if (first)
    for (int t = threadIdx.x; t < TT; t += kThreads)
      if (t0 + t < a.T) a.tokad[t0 + t] = tile.tok[t];
  const int r0 = rc * 64;
  T* packed = PACK && part == 0
                  ? (T*)a.packed + (int64_t)tile_id * steps * V * kWave * 8
                  : nullptr;
  AdapterWalk<TT> walk(tile.tok);
  int count = 0;
  f32x4 acc[N];
  for (;;) {
    int ad = -1;
    const bool any = walk.next(ad), only = count == 0 && walk.done();
    if (any && count++ % groups != group) continue;
    if (!any && !packed) break;  // a tile without adapters still packs its x
#pragma unroll
    for (int k = 0; k < N; ++k) acc[k] = f32x4{0.f, 0.f, 0.f, 0.f};
    int64_t from = tok;
    if (any && !only && !packed) {
      // lanes without a token of this adapter read along with one that has
      bool mine = false;
#pragma unroll
      for (int j = 0; j < V; ++j) mine |= tile.tok[tok - t0 + j] == ad;
      const int lead = (int)__builtin_ctzll(__ballot(mine)) % 16;
      const int64_t there = t0 + lead * V < lim ? t0 + lead * V : lim;
      from = mine ? tok : there;
    }
    shrink_steps<T, V, NR, TR, PACK>(x, job.ldx, job.K,
                                     (const T*)job.f + (int64_t)(any ? ad : 0) * a.R * job.K, a.R,
                                     r0, from, s0, s1, acc, packed);
    packed = nullptr;
    if (!any) break;
    spread_sum<N>(acc, red);
    constexpr int M = N < 4 ? N : N / 4, J = M < V ? M : V;  // tiles of a wave, tokens in a run
    if (N < 4 && wave != 0) continue;
    const float sc = a.scale ? a.scale[ad] : 1.f;
    const int rank = rank_of(a, ad), k0 = N < 4 ? 0 : wave * M;
#pragma unroll
    for (int k = 0; k < M; k += J) {
      const int q = (k0 + k) / V, j0 = (k0 + k) % V;
      const int r = TR ? (r0 + n * NR < a.R - NR ? r0 + n * NR : a.R - NR) + q : r0 + q * 16 + n;
      if (r >= a.R) continue;
      float* u = job.u + ((int64_t)slice * a.R + r) * a.Tp;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t t1 = (t0 + (g * 4 + i) * V < lim ? t0 + (g * 4 + i) * V : lim) + j0;
        float v[J];
#pragma unroll
        for (int j = 0; j < J; ++j) v[j] = r < rank ? acc[k + j][i] * sc : 0.f;
        if (only) {
          __builtin_memcpy(u + t1, v, sizeof(v));
        } else {
#pragma unroll
          for (int j = 0; j < J; ++j)
            if (tile.tok[t1 - t0 + j] == ad) u[t1 + j] = v[j];
        }
      }
    }
  }
}

template <typename T, int V, int NR, bool BACKWARD, bool PACK>
__global__ __launch_bounds__(kThreads, V * NR >= 8 ? 2 : 3) void lowrank_shrink_kernel(LowRankArgs a, ShrinkJob jx,
                                                                  ShrinkJob jy, int groups) {
  __shared__ f32x4 red[kWaves / 2 * NR * V * kWave];
  __shared__ TokenTile<16 * V> tile;
  // tiles are the fastest index, then the parts of a tile, then the slices
  const int tiles = (int)((a.T + 16 * V - 1) / (16 * V)), parts = groups * ((a.R + 63) / 64);
  const uint32_t b = xcd_chunk(block_of(a), a.blocks);
  const int tile_id = b % tiles, part = b / tiles % parts, z = b / tiles / parts;
  if (!BACKWARD || z < jx.slices)
    shrink_tile<T, V, NR, false, PACK>(a, jx, z, tile_id, part, b < (uint32_t)tiles, groups, red,
                                       tile);
  else
    shrink_tile<T, V, NR, true, false>(a, jy, z - jx.slices, tile_id, part, false, groups, red,
                                       tile);
}

// ------------------------------------------------------------------- pack --

// Bytes of a token's packed ranks: 64 for ranks up to 16, else 128 per 32
// ranks (hi and lo of a 16-bit type, or fp32).
__host__ __device__ inline int packed_row(int R) { return R <= 16 ? 64 : (R + 31) / 32 * 128; }

constexpr int kPackTokens = 32;  // small tiles: the launch is short and wants many workgroups

// Adds the slices of u (or du) in order and writes them as the operands that
// the later kernels load, so that the sum and the split into halves are made
// once and not by every workgroup that reads them:
//   rows   [token][ranks], for expand (u) and dx (du); f16: scaled by token
//   ru, rdu  [hi, lo][rank][token], for outer; f16: scaled by rank over the
//          tokens of one adapter in a block of 32, the exponent kept beside
template <typename T, bool BACKWARD>
__global__ __launch_bounds__(kThreads) void lowrank_pack_kernel(LowRankArgs a, int su, int sd) {
  constexpr int TT = kPackTokens, LD = TT + 1;
  extern __shared__ float us[];
  __shared__ float down[TT];
  const bool is_du = BACKWARD && blockIdx.y == 1;
  const float* u = is_du ? a.du : a.u;
  const int slices = is_du ? sd : su, tid = threadIdx.x, R = a.R;
  const int64_t t0 = (int64_t)block_of(a) * TT, size = (int64_t)R * a.Tp;
  for (int i = tid; i < R * (TT / 4); i += kThreads) {
    const int r = i / (TT / 4), t = i % (TT / 4) * 4;
    const float* p = u + (int64_t)r * a.Tp + t0 + t;
    f32x4 v = *(const f32x4*)p;
#pragma unroll 8
    for (int s = 1; s < slices; ++s) v += *(const f32x4*)(p + s * size);
#pragma unroll
    for (int e = 0; e < 4; ++e) us[r * LD + t + e] = v[e];
  }
  __syncthreads();
  if (!BACKWARD || is_du) {
    if constexpr (__is_same(T, _Float16)) {
      if (tid < TT) {
        float m = 0.f;
        for (int r = 0; r < R; ++r) m = fmaxf(m, fabsf(us[r * LD + tid]));
        if (m > kMaxFloat) {
          m = 0.f;
          for (int r = 0; r < R; ++r) m = max_finite(m, us[r * LD + tid]);
        }
        const Pow2 p = pow2_of(m);
        down[tid] = p.down;
        a.up[t0 + tid] = p.up;
      }
      __syncthreads();
    }
    const int pieces = packed_row(R) / 16;
    for (int i = tid; i < TT * pieces; i += kThreads) {
      const int t = i / pieces, c = i % pieces;
      uint32_t w[4];
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = c * 4 + e < R ? __float_as_uint(us[(c * 4 + e) * LD + t]) : 0u;
      } else {
        const bool lo = R <= 16 ? c >= 2 : c % 8 >= 4;
        const int r = R <= 16 ? c % 2 * 8 : c / 8 * 32 + c % 4 * 8;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[e] = r + e < R ? us[(r + e) * LD + t] : 0.f;
          if constexpr (__is_same(T, _Float16)) v[e] *= down[t];
        }
        const Frag<T> f = split8<T>(v, lo);
        __builtin_memcpy(w, &f, 16);
      }
      __builtin_memcpy(__builtin_assume_aligned((char*)a.rows + (t0 + t) * (pieces * 16) + c * 16, 16),
                       w, 16);
    }
  }
  if constexpr (BACKWARD) {
    const int lane = tid % TT;
    const int64_t t = t0 + lane;
    const int ad = __is_same(T, _Float16) && t < a.T ? a.tokad[t] : -1;
    for (int r = tid / TT; r < R; r += kThreads / TT) {
      float v = us[r * LD + lane];
      const int64_t at = (int64_t)r * a.Tp + t;
      if constexpr (sizeof(T) == 4) {
        ((float*)(is_du ? a.rdu : a.ru))[at] = v;
      } else {
        if constexpr (__is_same(T, _Float16)) {
          float big = 0.f;
          // both ranks of the wave hold the same tokens
          uint32_t rest = (uint32_t)__ballot(ad >= 0);
          while (rest) {
            const bool same = ad == __shfl(ad, __builtin_ctz(rest), kWave);
            float m = same ? max_finite(0.f, v) : 0.f;
#pragma unroll
            for (int o = 1; o < TT; o <<= 1) m = fmaxf(m, __shfl_xor(m, o, kWave));
            big = same ? m : big;
            rest &= ~(uint32_t)__ballot(same);
          }
          const Pow2 p = pow2_of(big);
          v *= p.down;
          (is_du ? a.edu : a.eu)[at] = (uint8_t)(__float_as_uint(p.up) >> 23);
        }
        T* out = (T*)(is_du ? a.rdu : a.ru) + at;
        store_bits(out, split_bits(v, false, (T*)nullptr));
        store_bits(out + size, split_bits(v, true, (T*)nullptr));
      }
    }
  }
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
#pragma unroll 8
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
      for (int s = 0; s < 4; ++s) m = max_finite(m, row[r + s]);
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

// A factor's fragment as hi and lo meet it.  SMALL: one fragment for both, the
// lanes of the block's upper half for lo.
template <typename T, bool SMALL>
struct Halves {
  Frag<T> hi, lo;
  __device__ __forceinline__ explicit Halves(const Frag<T>& f)
      : hi(SMALL ? made_finite(f, lane_id() >= 32) : f), lo(SMALL ? hi : made_finite(f, true)) {}
};

// c + F u for one K block: result rows are F's, columns are u's tokens.
template <typename T, bool SMALL>
__device__ __forceinline__ f32x4 u_mma(const Halves<T, SMALL>& f, const Frag<T>& hi,
                                       const Frag<T>& lo, f32x4 c) {
  if constexpr (SMALL && sizeof(T) == 4) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(f.hi.w[s]),
                                               __uint_as_float(hi.w[s]), c, 0, 0, 0);
    return c;
  } else {
    c = mma(f.hi, hi, c);
    if constexpr (!SMALL && sizeof(T) == 2) c = mma(f.lo, lo, c);
    return c;
  }
}

// The same turned: rows are u's tokens.
template <typename T, bool SMALL>
__device__ __forceinline__ f32x4 token_mma(const Frag<T>& hi, const Frag<T>& lo,
                                           const Halves<T, SMALL>& f, f32x4 c) {
  if constexpr (SMALL && sizeof(T) == 4) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(hi.w[s]),
                                               __uint_as_float(f.hi.w[s]), c, 0, 0, 0);
    return c;
  } else {
    c = mma(hi, f.hi, c);
    if constexpr (!SMALL && sizeof(T) == 2) c = mma(lo, f.lo, c);
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

// Fragment of feature f of A_ad, likewise (A's rows run along the features).
template <typename T, bool SMALL>
__device__ __forceinline__ Frag<T> at_frag(const LowRankArgs& a, int ad, int64_t f, int rank,
                                           int step) {
  constexpr int W = SMALL && sizeof(T) == 4 ? 4 : 8;
  const int r = rank_base<T, SMALL>(step);
  const T* p = (const T*)a.A + (int64_t)ad * a.R * a.n_in + f;
  uint32_t b[8];
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    b[s] = 0u;
    if (s < W) {
      const uint32_t v = raw_bits(p + (int64_t)(r + s < a.R ? r + s : a.R - 1) * a.n_in);
      b[s] = r + s < rank ? v : 0u;
    }
  }
  Frag<T> out;
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    if (sizeof(T) == 4)
      out.w[s] = b[s];
    else if (s % 2 == 0)
      out.w[s / 2] = b[s] | b[s + 1] << 16;
  }
  return out;
}

// The adapters of a tile of tokens: each token's own, and the distinct ones
// with their ranks, in order of their first token.
template <int TT>
struct TileAdapters {
  int tok[TT];
  int ad[TT];
  int rank[TT];
  float up[TT];  // scale of the token's packed ranks (f16)
  int count;
};

template <int TT, int THREADS>
__device__ __forceinline__ void load_tokad(const LowRankArgs& a, int64_t t0, int* tok) {
  for (int t = threadIdx.x; t < TT; t += THREADS) {
    const int ad = t0 + t < a.T ? a.tokad[t0 + t] : -1;
    tok[t] = ad < a.n ? ad : -1;
  }
}

// By all threads; ends with a barrier.
template <int TT, int THREADS>
__device__ __forceinline__ void tile_adapters(const LowRankArgs& a, int64_t t0, bool scaled,
                                              TileAdapters<TT>& s) {
  load_tokad<TT, THREADS>(a, t0, s.tok);
  if (scaled && threadIdx.x < TT) s.up[threadIdx.x] = a.up[t0 + threadIdx.x];
  __syncthreads();
  if (threadIdx.x < kWave) {
    AdapterWalk<TT> walk(s.tok);
    int ad, c = 0, mine0 = -1, mine1 = -1;
    while (walk.next(ad)) {
      if (c % kWave == lane_id()) (c < kWave ? mine0 : mine1) = ad;
      ++c;
    }
    const int l = lane_id();
    if (l < c) {
      s.ad[l] = mine0;
      s.rank[l] = rank_of(a, mine0);
    }
    if (TT > kWave && l + kWave < c) {
      s.ad[l + kWave] = mine1;
      s.rank[l + kWave] = rank_of(a, mine1);
    }
    if (l == 0) s.count = c;
  }
  __syncthreads();
}

// The tile's ranks as operands.  Column n of product q is the token V n + q,
// so that a lane's V columns are neighbours in memory.  Ranks up to 16 stay in
// registers, one fragment a product; more of them would leave one wave a SIMD
// (64 ranks: 128 registers, 145 us where shared memory takes
// 97 us for 8192 tokens and 11008 rows), so they stay in shared memory as
// pack wrote them, rows ordered by product for reads without bank conflicts.
// A tile of single tokens (V = 1) has its ranks staged there as fp32 instead.
template <int V>
__host__ __device__ inline int operand_bytes(int R) {
  return V == 1 ? 16 * staged_width(R) * 4 : R <= 16 ? 0 : 16 * V * (packed_row(R) + 16);
}

template <int V, int THREADS>
__device__ __forceinline__ void copy_rows(const LowRankArgs& a, int64_t t0, char* lds) {
  const int row = packed_row(a.R), pieces = row / 16;
  const char* from = (const char*)a.rows + t0 * row;
  for (int i = threadIdx.x; i < 16 * V * pieces; i += THREADS) {
    const int t = i / pieces, c = i % pieces;
    __builtin_memcpy(__builtin_assume_aligned(lds + (t % V * 16 + t / V) * (row + 16) + c * 16, 16),
                     __builtin_assume_aligned(from + (int64_t)i * 16, 16), 16);
  }
}

template <typename T, int V, bool SMALL>
struct UOperand {
  Frag<T> reg[SMALL ? V : 1];
  float up, down;  // of staged ranks
  const char* lds;
  int row, blocks;

  __device__ __forceinline__ UOperand(const LowRankArgs& a, int64_t t0, const char* staged) {
    const int n = lane_id() % 16, g = lane_id() / 16;
    blocks = SMALL ? 1 : (a.R + 31) / 32;
    row = V == 1 ? staged_width(a.R) * 4 : packed_row(a.R) + 16;
    lds = staged + n * row;
    up = down = 1.f;
    if constexpr (V == 1) {
      const Pow2 p = row_pow2<T>((const float*)lds, a.R);
      up = p.up;
      down = p.down;
      if constexpr (SMALL) reg[0] = u_frag<T, true>((const float*)lds, 0, false, down);
    } else if constexpr (SMALL) {
#pragma unroll
      for (int q = 0; q < V; ++q)
        __builtin_memcpy(&reg[q],
                         __builtin_assume_aligned((const char*)a.rows + (t0 + n * V + q) * 64 + g * 16, 16),
                         16);
    }
  }
  // acc[q] += f u_q for block k (not yet scaled by up)
  __device__ __forceinline__ void product(int k, const Frag<T>& factor, f32x4 (&acc)[V]) const {
    const int g = lane_id() / 16;
    const Halves<T, SMALL> f(factor);
#pragma unroll
    for (int q = 0; q < V; ++q) {
      Frag<T> h, l;
      if constexpr (SMALL) {
        h = l = reg[q];
      } else if constexpr (V == 1) {
        h = u_frag<T, false>((const float*)lds, k, false, down);
        l = u_frag<T, false>((const float*)lds, k, true, down);
      } else {
        const char* p = lds + q * 16 * row + k * 128 + g * (int)sizeof(h);
        __builtin_memcpy(&h, __builtin_assume_aligned(p, 16), sizeof(h));
        if constexpr (sizeof(T) == 2)
          __builtin_memcpy(&l, __builtin_assume_aligned(p + 64, 16), sizeof(l));
        else
          l = h;
      }
      acc[q] = u_mma<T, SMALL>(f, h, l, acc[q]);
    }
  }
};

// --------------------------------------------------------- expand and dx --

// Rows ob + 4 (lane / 16) + i of a matrix, V tokens from `t` a lane.
template <typename T, int V>
__device__ __forceinline__ void load_rows(const T* p, int64_t ld, int64_t ob, int64_t rows,
                                          int64_t t, int cnt, Row<T, V> (&y)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = ob + lane_id() / 16 * 4 + i;
    const T* at = p + (r < rows ? r : rows - 1) * ld + t;
    if (cnt >= V) {
      y[i] = load_row<T, V>(at);
    } else {
      zero_row(y[i]);
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e < cnt) y[i].w[e * sizeof(T) / 4] |= raw_bits(at + e) << (e * sizeof(T) * 8 % 32);
    }
  }
}

// expand: out = y + B u (out may be y itself; 8192 tokens x 11008 rows, 16 ranks,
// bf16: 76 us, 4.7 TB/s; 64 ranks: 95 us).  DX: out = A^T du, zero where a
// token has no adapter.  A workgroup keeps the ranks of 16 V tokens (in
// registers up to 16 ranks, past them in shared memory) and walks rows of the
// output, 16 a wave at a time: sixteen lanes
// hold 16 V neighbouring tokens of a row (256 bytes), four rows a load.  The
// next rows' values and factors are requested before the present ones are
// used.  Distinct adapters are computed for the whole tile one after another
// (D at a time in flight) and selected per token.
template <typename T, int V, int STEPS, bool SMALL, bool DX>
__device__ __forceinline__ void stream_rows(const LowRankArgs& a, const TileAdapters<16 * V>& tile,
                                            const char* staged, int64_t t0, int64_t row0,
                                            int64_t row_end) {
  constexpr int D = V != 1 ? 1 : SMALL && sizeof(T) == 2 ? 8 : 4, N = STEPS > 0 ? STEPS : 1;
  const int lane = lane_id(), n = lane % 16, wave = threadIdx.x / kWave;
  const UOperand<T, V, SMALL> u(a, t0, staged);
  const int64_t rows = DX ? a.n_in : a.n_out, t = t0 + n * V;
  const int cnt = clampi(a.T - t, 0, V);
  const int count = __builtin_amdgcn_readfirstlane(tile.count);
  const T* y = (const T*)a.y;
  T* out = (T*)a.out;
  auto factor = [&](int c, int64_t ob, int k) {
    const int at = c < count ? c : count - 1;
    const int ad = __builtin_amdgcn_readfirstlane(tile.ad[at]);
    const int rank = __builtin_amdgcn_readfirstlane(tile.rank[at]);
    const int64_t r = ob + n < rows ? ob + n : rows - 1;
    if constexpr (DX)
      return at_frag<T, SMALL>(a, ad, r, rank, k);
    else
      return b_frag<T, SMALL>(a, ad, r, rank, k);
  };
  Row<T, V> yv[4], yn[4];
  Frag<T> f[D][N], fn[D][N];
  int64_t ob = row0 + wave * 16;
  if (ob >= row_end) return;
  if constexpr (!DX) load_rows<T, V>(y, a.ldy, ob, rows, t, cnt, yn);
  if (STEPS > 0 && count > 0) {
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
      for (int k = 0; k < N; ++k) fn[d][k] = factor(d, ob, k);
  }
  for (; ob < row_end; ob += kWaves * 16) {
    const int64_t next = ob + kWaves * 16;
    const bool more = next < row_end;
    float v[4][V];
    if constexpr (!DX) {
#pragma unroll
      for (int i = 0; i < 4; ++i) yv[i] = yn[i];
      if (more) load_rows<T, V>(y, a.ldy, next, rows, t, cnt, yn);
    }
    if (STEPS > 0 && count > 0) {
#pragma unroll
      for (int d = 0; d < D; ++d)
#pragma unroll
        for (int k = 0; k < N; ++k) {
          f[d][k] = fn[d][k];
          if (more) fn[d][k] = factor(d, next, k);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int q = 0; q < V; ++q) v[i][q] = DX ? 0.f : row_f32<T, V>(yv[i], q);
    for (int c0 = 0; c0 < count; c0 += D) {
      if (STEPS > 0 && c0 > 0) {
#pragma unroll
        for (int d = 0; d < D; ++d)
#pragma unroll
          for (int k = 0; k < N; ++k) f[d][k] = factor(c0 + d, ob, k);
      }
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (d > 0 && c0 + d >= count) break;
        // what is in shared memory is not to be kept in registers over the
        // loops (or one wave a SIMD is left)
        asm volatile("" ::: "memory");
        const int ad = __builtin_amdgcn_readfirstlane(tile.ad[c0 + d]);
        f32x4 acc[V];
#pragma unroll
        for (int q = 0; q < V; ++q) acc[q] = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (STEPS > 0) {
#pragma unroll
          for (int k = 0; k < STEPS; ++k) u.product(k, f[d][k], acc);
        } else {
          for (int k = 0; k < u.blocks; ++k) u.product(k, factor(c0 + d, ob, k), acc);
        }
#pragma unroll
        for (int q = 0; q < V; ++q) {
          const bool mine = tile.tok[n * V + q] == ad;
          const float up = !__is_same(T, _Float16) ? 1.f : V == 1 ? u.up : tile.up[n * V + q];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float w = __is_same(T, _Float16) ? acc[q][i] * up : acc[q][i];
            v[i][q] = !mine ? v[i][q] : DX ? w : v[i][q] + w;
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t r = ob + lane / 16 * 4 + i;
      if (r < rows) store_chunk<T, V>(out + r * a.ldo + t, cnt, v[i]);
    }
  }
}

// Token tiles are the fastest index, so that neighbouring workgroups stream
// neighbouring parts of the same rows.
// Waves a SIMD that expand's registers are fitted to: three, two where three
// would spill.
template <typename T, int V, int STEPS, bool SMALL>
constexpr int expand_waves() {
  return V == 1 ? (STEPS == 2 && sizeof(T) == 4 ? 2 : 3)
                : (__is_same(T, _Float16) && (SMALL || STEPS == 2) ? 2 : 3);
}

template <typename T, int V, int STEPS, bool SMALL>
__global__ __launch_bounds__(kThreads, (expand_waves<T, V, STEPS, SMALL>())) void lowrank_expand_kernel(LowRankArgs a, int slices,
                                                                  int tiles, int rows_per_block) {
  constexpr int TT = 16 * V;
  extern __shared__ __attribute__((aligned(16))) char operand[];
  __shared__ TileAdapters<TT> tile;
  const uint32_t b = xcd_chunk(block_of(a), a.blocks);
  const int64_t t0 = (int64_t)(b % tiles) * TT, row0 = (int64_t)(b / tiles) * rows_per_block;
  const int64_t end = row0 + rows_per_block < a.n_out ? row0 + rows_per_block : a.n_out;
  if constexpr (V == 1)
    stage_u<TT, kThreads>(a, a.u, slices, t0, (float*)operand);
  else if constexpr (!SMALL)
    copy_rows<V, kThreads>(a, t0, operand);
  tile_adapters<TT, kThreads>(a, t0, __is_same(T, _Float16) && V != 1, tile);
  stream_rows<T, V, STEPS, SMALL, false>(a, tile, operand, t0, row0, end);
}

// ------------------------------------------------------------------ outer --

constexpr int kListTokens = 32 * kThreads;

template <int FF, int NR>
struct OuterShared {
  f32x4 red[kWaves / 2 * FF * NR * kWave];
  uint32_t mask[kThreads];
  uint16_t block[kThreads];
  int waves[kWaves];
};

// dA_a = sum over the adapter's tokens of du x^T, and dB_a = sum of dy u^T:
// one workgroup takes 16 FF features of x (or of dy), one adapter and up to 64
// ranks.  It lists the 32-token blocks that hold a token of the adapter, its
// waves take them in turn, two together where registers allow, the next ones'
// loads in flight; other adapters' tokens are masked out of both operands.
// The waves' sums are added in a fixed order.  f16: the block's product is
// scaled back in fp32 by the exponent that pack chose for the rank.
template <typename T, int NR, int FF>
__device__ __forceinline__ void outer_tile(const LowRankArgs& a, bool is_x, int64_t f0, int ad,
                                           int r0, OuterShared<FF, NR>& sh) {
  constexpr int P = NR * sizeof(T) > 4 || FF > 2 ? 1 : 2;
  constexpr bool F16 = __is_same(T, _Float16), HALVES = sizeof(T) == 2;
  const int tid = threadIdx.x, lane = lane_id(), n = lane % 16, g = lane / 16, wave = tid / kWave;
  const int64_t F = is_x ? a.n_in : a.n_out, ld = is_x ? a.ldx : a.ldy;
  const T* src = (const T*)(is_x ? a.x : a.y);
  const T* u = (const T*)(is_x ? a.rdu : a.ru);
  const uint8_t* ex = is_x ? a.edu : a.eu;
  const int64_t half = (int64_t)a.R * a.Tp;
  const T* row[FF];
#pragma unroll
  for (int k = 0; k < FF; ++k) {
    const int64_t f = f0 + k * 16 + n;
    row[k] = src + (f < F ? f : F - 1) * ld;
  }
  int64_t urow[NR];
#pragma unroll
  for (int q = 0; q < NR; ++q) {
    const int r = r0 + q * 16 + n;
    urow[q] = (int64_t)(r < a.R ? r : a.R - 1) * a.Tp;
  }
  f32x4 acc[FF * NR];
#pragma unroll
  for (int k = 0; k < FF * NR; ++k) acc[k] = f32x4{0.f, 0.f, 0.f, 0.f};
  // 16-bit rows that start between two words are read as the words around them
  // and shifted in registers: loads that are not aligned to a word take several
  // times as long in this pattern (2047 tokens: 71 us where this takes 46)
  const bool odd = HALVES && ((((uintptr_t)src) | (uintptr_t)(ld * (int64_t)sizeof(T))) & 2);
  uint32_t shift[FF];
#pragma unroll
  for (int k = 0; k < FF; ++k) shift[k] = HALVES ? (uint32_t)((uintptr_t)row[k] & 2) * 8 : 0u;
  struct Raw {
    uint32_t w[2 * sizeof(T) + (HALVES ? 1 : 0)];
  };
  auto aligned = [&](const Raw& r, uint32_t sh) {
    Frag<T> f;
#pragma unroll
    for (int i = 0; i < (int)(2 * sizeof(T)); ++i)
      f.w[i] = HALVES ? __builtin_amdgcn_alignbit(r.w[HALVES ? i + 1 : i], r.w[i], sh) : r.w[i];
    return f;
  };
  struct Buf {
    Raw x[P][FF];
    Frag<T> hi[P][NR], lo[P][HALVES ? NR : 1];
    uint32_t e[P][F16 ? NR : 1], m[P];
  } cur, nxt;
  for (int64_t c0 = 0; c0 < a.T; c0 += kListTokens) {
    // this chunk's blocks with a token of the adapter
    uint32_t m = 0;
    const int64_t tb = c0 + (int64_t)tid * 32;
    if (tb < a.T) {
      int ta[32];
      __builtin_memcpy(ta, __builtin_assume_aligned(a.tokad + tb, 16), sizeof(ta));
      const int left = clampi(a.T - tb, 0, 32);
#pragma unroll
      for (int s = 0; s < 32; ++s) m |= (ta[s] == ad && s < left ? 1u : 0u) << s;
    }
    const uint64_t any = __ballot(m != 0);
    if (lane == 0) sh.waves[wave] = __builtin_popcountll(any);
    sh.mask[tid] = m;
    __syncthreads();
    int before = 0, count = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      before += w < wave ? sh.waves[w] : 0;
      count += sh.waves[w];
    }
    if (m != 0) sh.block[before + __builtin_popcountll(any & lanemask_lt())] = (uint16_t)tid;
    __syncthreads();
    count = __builtin_amdgcn_readfirstlane(count);
    auto load = [&](int e, Buf& b) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int at = e + p < count ? e + p : count - 1;
        const int blk = __builtin_amdgcn_readfirstlane((int)sh.block[at]);
        b.m[p] = e + p < count ? __builtin_amdgcn_readfirstlane(sh.mask[blk]) : 0u;
        const int64_t bt = c0 + (int64_t)blk * 32, t = bt + g * 8;
        const bool whole = bt + 32 <= a.T;
        if (!whole) {
#pragma unroll
          for (int k = 0; k < FF; ++k) {
            const Frag<T> f = load8_count(row[k] + t, clampi(a.T - t, 0, 8));
            uint32_t below = 0;
#pragma unroll
            for (int i = 0; i < (int)(2 * sizeof(T)); ++i) {
              b.x[p][k].w[i] = shift[k] ? __builtin_amdgcn_alignbit(f.w[i], below, 16) : f.w[i];
              below = f.w[i];
            }
            if constexpr (HALVES) b.x[p][k].w[4] = below >> 16;
          }
        } else if (odd) {
          // each word holds an element of the row: none lies outside its memory
#pragma unroll
          for (int k = 0; k < FF; ++k) {
            const uint32_t* q = (const uint32_t*)((uintptr_t)(row[k] + t) & ~(uintptr_t)3);
            __builtin_memcpy(b.x[p][k].w, q, 16);
            if constexpr (HALVES) b.x[p][k].w[4] = q[shift[k] ? 4 : 3];
          }
        } else {
#pragma unroll
          for (int k = 0; k < FF; ++k) {
            __builtin_memcpy(b.x[p][k].w, row[k] + t, sizeof(Frag<T>));
            if constexpr (HALVES) b.x[p][k].w[4] = 0u;
          }
        }
#pragma unroll
        for (int q = 0; q < NR; ++q) {
          __builtin_memcpy(&b.hi[p][q], __builtin_assume_aligned(u + urow[q] + t, 16),
                           sizeof(Frag<T>));
          if constexpr (HALVES)
            __builtin_memcpy(&b.lo[p][q], __builtin_assume_aligned(u + half + urow[q] + t, 16),
                             sizeof(Frag<T>));
          // any token of the adapter in the block has the scale
          if constexpr (F16) b.e[p][q] = ex[urow[q] + bt + (b.m[p] ? __builtin_ctz(b.m[p]) : 0)];
        }
      }
    };
    auto compute = [&](Buf& b) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        if (b.m[p] == 0) continue;
        Frag<T> x[FF];
#pragma unroll
        for (int k = 0; k < FF; ++k) x[k] = aligned(b.x[p][k], shift[k]);
        if (b.m[p] != ~0u) {
          const uint32_t m8 = (b.m[p] >> (g * 8)) & 255u;
#pragma unroll
          for (int k = 0; k < FF; ++k) mask8(x[k], m8);
#pragma unroll
          for (int q = 0; q < NR; ++q) {
            mask8(b.hi[p][q], m8);
            if constexpr (HALVES) mask8(b.lo[p][q], m8);
          }
        }
#pragma unroll
        for (int k = 0; k < FF; ++k) {
          const Halves<T, false> h(x[k]);
#pragma unroll
          for (int q = 0; q < NR; ++q) {
            f32x4& d = acc[k * NR + q];
            if constexpr (F16) {
              const float up = __uint_as_float(b.e[p][q] << 23);
              const f32x4 c = mma(h.lo, b.lo[p][q],
                                  mma(h.hi, b.hi[p][q], f32x4{0.f, 0.f, 0.f, 0.f}));
#pragma unroll
              for (int i = 0; i < 4; ++i) d[i] = __builtin_fmaf(c[i], up, d[i]);
            } else {
              d = mma(h.hi, b.hi[p][q], d);
              if constexpr (HALVES) d = mma(h.lo, b.lo[p][q], d);
            }
          }
        }
      }
    };
    if (wave * P < count) load(wave * P, nxt);
    for (int e = wave * P; e < count; e += kWaves * P) {
      cur = nxt;
      if (e + kWaves * P < count) load(e + kWaves * P, nxt);
      __builtin_amdgcn_sched_barrier(0);
      compute(cur);
    }
    __syncthreads();
  }
  wave_tree_sum<FF * NR, kWaves>(acc, sh.red);
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

// dA, dB and dx in one launch: they need the same packed ranks and nothing of
// each other, and the reads of the first two go beside the writes of the last.
template <typename T, int NR, int STEPS, bool SMALL, int FF>
__global__ __launch_bounds__(kThreads, 3) void lowrank_gradients_kernel(LowRankArgs a, int xblocks,
                                                                     int yblocks, int tiles,
                                                                     int rows_per_block) {
  constexpr int V = 16 / sizeof(T), TT = 16 * V;
  extern __shared__ __attribute__((aligned(16))) char operand[];
  __shared__ union {
    OuterShared<FF, NR> outer;
    TileAdapters<TT> tile;
  } sh;
  const int rcs = (a.R + 63) / 64;
  const int64_t outer = (int64_t)(xblocks + yblocks) * a.n * rcs;
  const uint32_t block = block_of(a);
  if (block < outer) {
    const uint32_t b = xcd_chunk(block, (uint32_t)outer);
    const int per = a.n * rcs, fb = b / per, rest = b % per;
    const bool is_x = fb < xblocks;
    outer_tile<T, NR, FF>(a, is_x, (int64_t)(is_x ? fb : fb - xblocks) * (16 * FF), rest / rcs,
                      rest % rcs * 64, sh.outer);
  } else {
    const int64_t b = xcd_chunk(block - outer, a.blocks - outer), t0 = b % tiles * TT,
                  row0 = b / tiles * rows_per_block;
    const int64_t end = row0 + rows_per_block < a.n_in ? row0 + rows_per_block : a.n_in;
    if constexpr (!SMALL) copy_rows<V, kThreads>(a, t0, operand);
    tile_adapters<TT, kThreads>(a, t0, __is_same(T, _Float16), sh.tile);
    stream_rows<T, V, STEPS, SMALL, true>(a, sh.tile, operand, t0, row0, end);
  }
}

// ---------------------------------------------------------------- project --

// y = W x + B u on a tile of 16 V tokens: a workgroup takes 16 MO rows of W,
// eight waves a slice of the features each; x comes as the fragments that the
// shrink kernel packed, and is read once for the MO row tiles.  V more waves make the adapters' part of 16 tokens each
// meanwhile: their chain of dependent loads (u, adapter, B) is as long as the
// stream of W and would double the time behind it.  All meet in shared memory.
template <typename T, int V, int MO, bool SMALL>
__global__ __launch_bounds__((kProjectWaves + V) * kWave) void lowrank_project_kernel(
    LowRankArgs a, int slices, int row_blocks) {
  constexpr int TT = 16 * V, D = 4;
  extern __shared__ float us[];
  __shared__ f32x4 red[(kProjectWaves + 1) * MO * V * kWave];
  const int lane = lane_id(), n = lane % 16, g = lane / 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int block = block_of(a) % row_blocks;
  const int64_t tile = block_of(a) / row_blocks;
  int64_t t0 = tile * TT;
  if (t0 > a.T - TT) t0 = a.T > TT ? a.T - TT : 0;
  const int64_t lim = a.T - V, o0 = (int64_t)block * (16 * MO);
  auto row_of = [&](int k) {
    const int64_t o = o0 + k * 16 + n;
    return o < a.n_out ? o : a.n_out - 1;
  };
  // token of row m of tile j
  auto token = [&](int m, int j) {
    const int64_t t = t0 + m * V;
    return (t < lim ? t : lim) + j;
  };
  if (wave < kProjectWaves) {
    const int64_t steps = cdiv(a.n_in, 32);
    const int64_t s0 = steps * wave / kProjectWaves, s1 = steps * (wave + 1) / kProjectWaves;
    const T* w[MO];
#pragma unroll
    for (int k = 0; k < MO; ++k) w[k] = (const T*)a.W + row_of(k) * a.ldw + g * 8;
    const T* xp = (const T*)a.packed + (tile * steps * V * kWave + lane) * 8;
    f32x4 acc[MO * V];
#pragma unroll
    for (int k = 0; k < MO * V; ++k) acc[k] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int64_t whole = a.n_in / 32 < s1 ? a.n_in / 32 : s1;
    // U steps' loads are issued together
    constexpr int U = MO == 1 ? 8 / V : V == 4 ? 2 : 4;
    auto run = [&](int64_t at, auto steps_together) {
      constexpr int N = decltype(steps_together)::value;
      Frag<T> fw[N][MO], fx[N][V];
#pragma unroll
      for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int k = 0; k < MO; ++k) fw[i][k] = load8(w[k] + (at + i) * 32);
#pragma unroll
        for (int j = 0; j < V; ++j) fx[i][j] = load8(xp + ((at + i) * V + j) * kWave * 8);
      }
      __builtin_amdgcn_sched_barrier(0);  // or the loads are spread among the products
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int k = 0; k < MO; ++k)
#pragma unroll
          for (int j = 0; j < V; ++j) acc[k * V + j] = mma(fx[i][j], fw[i][k], acc[k * V + j]);
    };
    int64_t s = s0;
#pragma unroll 1
    for (; s + U <= whole; s += U) run(s, Int<U>{});
#pragma unroll 1
    for (; s < whole; ++s) run(s, Int<1>{});
    if (s < s1) {
      const int cnt = clampi(a.n_in - s * 32 - g * 8, 0, 8);
#pragma unroll
      for (int k = 0; k < MO; ++k) {
        const Frag<T> fw = load8_count(w[k] + s * 32, cnt);
#pragma unroll
        for (int j = 0; j < V; ++j)
          acc[k * V + j] = mma(load8(xp + (s * V + j) * kWave * 8), fw, acc[k * V + j]);
      }
    }
#pragma unroll
    for (int k = 0; k < MO * V; ++k) red[(wave * MO * V + k) * kWave + lane] = acc[k];
  } else {
    const int j = wave - kProjectWaves, rs = staged_width(a.R);
    float* mine = us + j * 16 * rs;
    const int64_t tn = token(n, j);
    int ad_n = tn < a.T ? a.tokad[tn] : -1;
    ad_n = ad_n < a.n ? ad_n : -1;
    for (int r = g; r < rs - 4; r += 4) {
      float v = 0.f;
      if (r < a.R) {
        const float* p = a.u + (int64_t)r * a.Tp + tn;
#pragma unroll 8
        for (int s = 0; s < slices; ++s) v += p[(int64_t)s * a.R * a.Tp];
      }
      mine[n * rs + r] = v;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the wave alone reads its ranks
    __builtin_amdgcn_wave_barrier();
    const float* row = mine + n * rs;
    const Pow2 p = row_pow2<T>(row, a.R);
    const int blocks = SMALL ? 1 : (a.R + 31) / 32;
    int ra[4];
    float up[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ra[i] = __shfl(ad_n, g * 4 + i, kWave);
      up[i] = __is_same(T, _Float16) ? __shfl(p.up, g * 4 + i, kWave) : 1.f;
    }
    f32x4 v[MO];
#pragma unroll
    for (int m = 0; m < MO; ++m) v[m] = f32x4{0.f, 0.f, 0.f, 0.f};
    uint64_t rest = __ballot(ad_n >= 0);
    while (rest) {
      // D distinct adapters, their factors requested together
      int ads[D], ranks[D], count = 0;
#pragma unroll
      for (int d = 0; d < D; ++d) {
        ads[d] = d > 0 ? ads[d - 1] : 0;
        if (rest) {
          ads[d] = __builtin_amdgcn_readlane(ad_n, __builtin_ctzll(rest));
          rest &= ~__ballot(ad_n == ads[d]);
          ++count;
        }
      }
#pragma unroll
      for (int d = 0; d < D; ++d) ranks[d] = rank_of(a, ads[d]);
      f32x4 c[MO][D];
#pragma unroll
      for (int m = 0; m < MO; ++m)
#pragma unroll
        for (int d = 0; d < D; ++d) c[m][d] = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int k = 0; k < blocks; ++k) {
        const Frag<T> hi = u_frag<T, SMALL>(row, k, false, p.down);
        const Frag<T> lo = u_frag<T, SMALL>(row, k, true, p.down);
        Frag<T> f[MO][D];
#pragma unroll
        for (int d = 0; d < D; ++d)
#pragma unroll
          for (int m = 0; m < MO; ++m) f[m][d] = b_frag<T, SMALL>(a, ads[d], row_of(m), ranks[d], k);
#pragma unroll
        for (int d = 0; d < D; ++d)
#pragma unroll
          for (int m = 0; m < MO; ++m)
            c[m][d] = token_mma<T, SMALL>(hi, lo, Halves<T, SMALL>(f[m][d]), c[m][d]);
      }
#pragma unroll
      for (int d = 0; d < D; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool mine_too = d < count && ra[i] == ads[d];
#pragma unroll
          for (int m = 0; m < MO; ++m) v[m][i] = mine_too ? c[m][d][i] * up[i] : v[m][i];
        }
    }
#pragma unroll
    for (int m = 0; m < MO; ++m) red[((kProjectWaves * MO + m) * V + j) * kWave + lane] = v[m];
  }
  __syncthreads();
  for (int k = wave; k < MO * V; k += kProjectWaves + V) {
    f32x4 v = red[k * kWave + lane];
#pragma unroll
    for (int h = 1; h < kProjectWaves; ++h) v += red[(h * MO * V + k) * kWave + lane];
    const f32x4 add = red[(kProjectWaves * MO * V + k) * kWave + lane];
    const int64_t o = o0 + k / V * 16 + n;
    if (o < a.n_out) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t t = token(g * 4 + i, k % V);
        if (t < a.T) store_bits((T*)a.out + o * a.ldo + t, out_bits(v[i] + add[i], (T*)nullptr));
      }
    }
  }
}

// -------------------------------------------------------------------- few --

constexpr int kFewTokens = 16;
constexpr int kFewThreads = 1024;
constexpr int kFewWaves = kFewThreads / kWave;

// A few tokens with one adapter at most, in one launch: every workgroup makes
// u = A x for itself, from its XCD's L2 (128 KB for 16 ranks of 4096 features in 16
// bits; `few` bounds it).
// add: sixteen waves split A's features, then take 16 rows of B each.  project:
// a workgroup takes 16 rows of W, whose features eight waves split; the other
// eight find the adapter and make u and B u meanwhile.
template <typename T, bool PROJECT, int NR>
__global__ __launch_bounds__(kFewThreads) void lowrank_few_kernel(LowRankArgs a) {
  constexpr bool SMALL = NR == 1;
  constexpr int AW = PROJECT ? kFewWaves - kProjectWaves : kFewWaves;  // waves that split A
  __shared__ float us[16 * (16 * NR + 4)];
  __shared__ f32x4 red[(AW * NR + (PROJECT ? kProjectWaves : 0)) * kWave];
  f32x4* redw = red + AW * NR * kWave;
  const int lane = lane_id(), n = lane % 16, g = lane / 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const bool stream = PROJECT && wave >= AW;  // a wave of W
  const int64_t K = a.n_in, steps = cdiv(K, 32);
  const int parts = stream ? kProjectWaves : AW, part = stream ? wave - AW : wave;
  const int64_t s0 = steps * part / parts, s1 = steps * (part + 1) / parts;
  const int64_t whole = K / 32 < s1 ? K / 32 : s1;
  constexpr int rs = 16 * NR + 4;
  const T* x = (const T*)a.x + (n < a.T ? n : (int)a.T - 1);
  const bool neighbours = a.ldx == 1;  // one token: the features lie together
  auto x_frag = [&](int64_t k0, auto tail) {
    uint32_t b[8];
    const T* p = x + k0 * a.ldx;
#pragma unroll
    for (int s = 0; s < 8; ++s)
      b[s] = !decltype(tail)::value || k0 + s < K ? raw_bits(p + s * a.ldx) : 0u;
    Frag<T> f;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      if (sizeof(T) == 4)
        f.w[s] = b[s];
      else if (s % 2 == 0)
        f.w[s / 2] = b[s] | b[s + 1] << 16;
    }
    return f;
  };
  // rows of length K against x, over this wave's features
  auto dots = [&](auto count, const T* const* rows, f32x4* acc) {
    constexpr int M = decltype(count)::value;
    int64_t s = s0;
    auto run = [&](auto together, auto near) {
      constexpr int N = decltype(together)::value;
      Frag<T> f[N][M], fx[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int64_t k0 = (s + i) * 32 + g * 8;
#pragma unroll
        for (int m = 0; m < M; ++m) f[i][m] = load8(rows[m] + k0);
        if constexpr (decltype(near)::value)
          fx[i] = load8(x + k0);
        else
          fx[i] = x_frag(k0, Int<0>{});
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int m = 0; m < M; ++m) acc[m] = mma(f[i][m], fx[i], acc[m]);
      s += N;
    };
    constexpr int U = sizeof(T) == 4 ? 4 : 8;
    if (neighbours) {
#pragma unroll 1
      while (s + U <= whole) run(Int<U>{}, Int<1>{});
    } else {
#pragma unroll 1
      while (s + 2 <= whole) run(Int<2>{}, Int<0>{});
    }
#pragma unroll 1
    while (s < whole) run(Int<1>{}, Int<0>{});
    if (s < s1) {
      const int64_t k0 = s * 32 + g * 8;
      const Frag<T> fx = x_frag(k0, Int<1>{});
#pragma unroll
      for (int m = 0; m < M; ++m)
        acc[m] = mma(load8_count(rows[m] + k0, clampi(K - k0, 0, 8)), fx, acc[m]);
    }
  };
  const int64_t o0 = PROJECT ? (int64_t)blockIdx.x * 16
                             : ((int64_t)blockIdx.x * kFewWaves + wave) * 16;
  const int64_t oc = o0 + n < a.n_out ? o0 + n : a.n_out - 1;
  const bool finish = PROJECT ? wave == 0 : o0 < a.n_out;  // waves that write rows
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  int ad = -1, rank = 0;
  float sc = 1.f;
  uint32_t mine = 0;  // tokens of the adapter
  Frag<T> fb{};
  if (stream) {
    f32x4 acc[1] = {f32x4{0.f, 0.f, 0.f, 0.f}};
    const T* rows[1] = {(const T*)a.W + oc * a.ldw};
    dots(Int<1>{}, rows, acc);
    redw[part * kWave + lane] = acc[0];
  } else {
    if (!PROJECT && finish && n < a.T) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t r = o0 + g * 4 + i;
        if (r < a.n_out) v[i] = to_f32(((const T*)a.y)[r * a.ldy + n]);
      }
    }
    for (int i0 = 0; i0 < a.S; i0 += kWave) {
      const int i = i0 + lane;
      uint32_t m = 0;
      int of = -1;
      if (i < a.S) {
        of = a.adapter[i];
        const int lo = clampi(a.offsets[i], 0, (int)a.T), hi = clampi(a.offsets[i + 1], 0, (int)a.T);
        if (lo < hi && of >= 0 && of < a.n) m = (1u << hi) - (1u << lo);
      }
      const uint64_t some = __ballot(m != 0);
      if (some) {
        if (ad < 0) ad = __builtin_amdgcn_readlane(of, __builtin_ctzll(some));
        if (of != ad) m = 0;
#pragma unroll
        for (int o = 1; o < kWave; o <<= 1) m |= (uint32_t)__shfl_xor((int)m, o, kWave);
        mine |= m;
      }
    }
    if (ad >= 0) {
      if (a.scale) sc = a.scale[ad];
      rank = rank_of(a, ad);
      if (rank == 0) mine = 0;
      if (finish) fb = b_frag<T, SMALL>(a, ad, oc, rank, 0);
      f32x4 acc[NR];
      const T* rows[NR];
#pragma unroll
      for (int q = 0; q < NR; ++q) {
        const int r = q * 16 + n;
        rows[q] = (const T*)a.A + ((int64_t)ad * a.R + (r < a.R ? r : a.R - 1)) * K;
        acc[q] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
      dots(Int<NR>{}, rows, acc);
#pragma unroll
      for (int q = 0; q < NR; ++q) red[(wave * NR + q) * kWave + lane] = acc[q];
    }
  }
  __syncthreads();
  if (wave < NR) {
    f32x4 t = f32x4{0.f, 0.f, 0.f, 0.f};
    if (ad >= 0) {
#pragma unroll
      for (int h = 0; h < AW; ++h) t += red[(h * NR + wave) * kWave + lane];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = wave * 16 + g * 4 + i;
      us[n * rs + r] = r < rank && ((mine >> n) & 1u) ? t[i] * sc : 0.f;
    }
  }
  __syncthreads();
  if (!finish) return;
  if constexpr (PROJECT) {
    f32x4 w = redw[lane];
#pragma unroll
    for (int h = 1; h < kProjectWaves; ++h) w += redw[h * kWave + lane];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = w[i];
  }
  const float* row = us + n * rs;
  const Pow2 p = row_pow2<T>(row, a.R);
  const Frag<T> hi = u_frag<T, SMALL>(row, 0, false, p.down);
  const Frag<T> lo = u_frag<T, SMALL>(row, 0, true, p.down);
  const f32x4 c = u_mma<T, SMALL>(Halves<T, SMALL>(fb), hi, lo, f32x4{0.f, 0.f, 0.f, 0.f});
  if (n < a.T) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t r = o0 + g * 4 + i;
      const float f = (mine >> n) & 1u ? v[i] + c[i] * p.up : v[i];
      if (r < a.n_out) store_bits((T*)a.out + r * a.ldo + n, out_bits(f, (T*)nullptr));
    }
  }
}

// --------------------------------------------------------------- launches --

constexpr size_t kSharedBytes = 160 * 1024;  // of a workgroup
// The largest takers besides: expand and dx at 256 ranks (their tile's rows and
// the adapters or the sums of outer), project with two row tiles.
static_assert(128 * (1024 + 16) + sizeof(OuterShared<2, 4>) + 1024 <= kSharedBytes, "dx");
static_assert((kProjectWaves + 1) * 2 * 4 * kWave * 16 + 64 * (256 + 4) * 4 <= kSharedBytes, "project");

constexpr int64_t kFillBlocks = 512;  // two workgroups on each of the 256 CUs
// Busy workgroups of the shrink kernel.  More of them mean more partial sums
// (8192 tokens, 16 ranks: 25 us at 256, 27 at 384, 32 at 1024), fewer leave
// tiles of several adapters behind (2047 tokens of 23 requests, both products:
// 54 us at 256, 41 at 384, 48 at 512).
constexpr int64_t kShrinkBlocks = 384;

// Tokens a lane holds of a row in the shrink kernel: 16 bytes a load of a 16-bit
// type up to 32 ranks.  Past them the sums of eight tokens (32 tiles of a 16-row
// product, four registers each) would leave one wave a SIMD; with four tokens two
// fit, as with eight up to 32 ranks, and narrower forms leave three.
int token_width(int op, int dtype, int64_t T, int64_t R) {
  const int most = op == kLowRankProject || dtype == kF32 || R > 32 ? 4 : 8;
  int v = 1;
  while (v < most && T > 16 * v) v *= 2;
  return v;
}

// Distinct adapters that share a tile are spread over this many workgroups:
// one more than the mean number of requests that start in a tile, for the one
// that reaches into it.  Where few tiles have a second adapter, those take
// twice the time instead of every tile an idle workgroup.
int adapter_groups(double mean, int64_t S, int64_t n) {
  if (mean < 0.25) return 1;
  int64_t g = (int64_t)mean + 2;
  g = g < n ? g : n;
  g = g < S ? g : S;
  return (int)(g < 1 ? 1 : g > 64 ? 64 : g);
}

int slices_for(double blocks, int64_t K) {
  int64_t s = (int64_t)(kShrinkBlocks / blocks);
  const int64_t most = cdiv(K, 32) / (2 * kWaves);  // two steps a wave at least
  s = s < most ? s : most;
  return (int)(s < 1 ? 1 : s > 16 ? 16 : s);
}

// launch(arguments, grid) for workgroups of `threads`.  A launch has fewer than
// 2^32 work-items; what is more goes into further ones.  Parts of whole rounds over
// the XCDs keep each XCD's share together.
template <typename F>
hipError_t in_parts(LowRankArgs a, int64_t blocks, int threads, F launch) {
  const int64_t most = (int64_t)(UINT32_MAX / (uint32_t)threads) / 8 * 8;
  a.blocks = (uint32_t)blocks;
  for (int64_t b = 0; b < blocks; b += most) {
    a.block0 = (uint32_t)b;
    launch(a, (unsigned)(blocks - b < most ? blocks - b : most));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T, int V, bool BACKWARD, bool PACK>
hipError_t shrink_v(const LowRankArgs& a, const LowRankLayout& l, hipStream_t s) {
  ShrinkJob jx{a.x, a.A, a.u, a.ldx, a.n_in, l.slices_u};
  ShrinkJob jy{a.y, a.B, a.du, a.ldy, a.n_out, l.slices_du};
  auto launch = [&](auto ranks) {
    return in_parts(a, l.shrink_blocks, kThreads, [&](const LowRankArgs& p, unsigned grid) {
      hipLaunchKernelGGL((lowrank_shrink_kernel<T, V, decltype(ranks)::value, BACKWARD, PACK>),
                         dim3(grid), dim3(kThreads), 0, s, p, jx, jy, l.groups);
    });
  };
  if (a.R <= 16) return launch(Int<1>{});
  if (a.R <= 32) return launch(Int<2>{});
  if constexpr (V <= 4) return launch(Int<4>{});
  return hipErrorInvalidValue;  // token_width keeps such tiles narrow
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

// Rows a workgroup of expand or dx takes: enough that loading its tokens'
// ranks is a small part of the streams, few enough that the launch fills the
// GPU.
int64_t rows_per_block(int64_t rows, int64_t tiles) {
  const int64_t unit = 16 * kWaves, blocks = cdiv(4 * kFillBlocks, tiles);
  const int64_t per = cdiv(cdiv(rows, blocks), unit) * unit;
  return per < 512 ? per : 512;
}

// Whether the ranks are packed for expand's wide tiles, or staged by its
// 16-token tiles without that launch: staged for few tokens, and for some more
// where most tiles have many adapters (which a wide tile computes one after
// another).  4096 x 4096, 16 ranks, bf16, staged against packed, us: one request
// of 128 tokens 12.8 and 16.1, of 192 13.8 and 16.3, of 256 16.8 and 16.1; 256
// requests of one token 34 and 43, 512 45.7 and 44.9.
bool packs(int op, int64_t T, int64_t S) {
  if (op != kLowRankAdd) return op == kLowRankBackward;
  return T > (S >= T / 8 ? 256 : 192);
}

template <typename T, bool BACKWARD>
hipError_t pack(const LowRankArgs& a, const LowRankLayout& l, hipStream_t s) {
  return in_parts(a, a.Tp / kPackTokens, kThreads, [&](const LowRankArgs& p, unsigned grid) {
    hipLaunchKernelGGL((lowrank_pack_kernel<T, BACKWARD>), dim3(grid, BACKWARD ? 2 : 1),
                       dim3(kThreads), (size_t)a.R * (kPackTokens + 1) * 4, s, p, l.slices_u,
                       l.slices_du);
  });
}

template <typename T, int V>
hipError_t expand_v(const LowRankArgs& a, const LowRankLayout& l, hipStream_t s) {
  const int64_t tiles = cdiv(a.T, 16 * V), per = rows_per_block(a.n_out, tiles);
  auto launch = [&](auto steps, auto small) {
    return in_parts(a, cdiv(a.n_out, per) * tiles, kThreads,
                    [&](const LowRankArgs& p, unsigned grid) {
      hipLaunchKernelGGL((lowrank_expand_kernel<T, V, decltype(steps)::value,
                                                decltype(small)::value != 0>),
                         dim3(grid), dim3(kThreads), operand_bytes<V>(a.R), s, p, l.slices_u,
                         (int)tiles, (int)per);
    });
  };
  if (a.R <= 16) return launch(Int<1>{}, Int<1>{});
  if (a.R <= 32) return launch(Int<1>{}, Int<0>{});
  if (a.R <= 64) return launch(Int<2>{}, Int<0>{});
  return launch(Int<0>{}, Int<0>{});
}

template <typename T, int FF>
hipError_t gradients_f(const LowRankArgs& a, hipStream_t s) {
  constexpr int TT = 256 / sizeof(T);
  const int64_t xb = cdiv(a.n_in, 16 * FF), yb = cdiv(a.n_out, 16 * FF);
  const int64_t tiles = cdiv(a.T, TT), per = rows_per_block(a.n_in, tiles > 0 ? tiles : 1);
  const int64_t blocks = (xb + yb) * a.n * cdiv(a.R, 64) + cdiv(a.n_in, per) * tiles;
  const size_t lds = operand_bytes<16 / sizeof(T)>(a.R);
  const int t = (int)(tiles > 0 ? tiles : 1);
  auto launch = [&](auto nr, auto steps, auto small) {
    return in_parts(a, blocks, kThreads, [&](const LowRankArgs& p, unsigned grid) {
      hipLaunchKernelGGL((lowrank_gradients_kernel<T, decltype(nr)::value, decltype(steps)::value,
                                                   decltype(small)::value != 0, FF>),
                         dim3(grid), dim3(kThreads), lds, s, p, (int)xb, (int)yb, t, (int)per);
    });
  };
  if (a.R <= 16) return launch(Int<1>{}, Int<1>{}, Int<1>{});
  if constexpr (FF > 2) {
    return launch(Int<2>{}, Int<1>{}, Int<0>{});  // up to 32 ranks
  } else {
    if (a.R <= 32) return launch(Int<2>{}, Int<1>{}, Int<0>{});
    if (a.R <= 64) return launch(Int<4>{}, Int<2>{}, Int<0>{});
    return launch(Int<4>{}, Int<0>{}, Int<0>{});
  }
}

// Features of an outer workgroup: 64 share each load of u where that still
// gives two workgroups a CU and the sums fit the registers (2048 tokens, 6 adapters of 32 ranks, f16: 42 us
// against 75 with 32), else 32 (one adapter of 4096 x 4096).
template <typename T>
hipError_t gradients(const LowRankArgs& a, hipStream_t s) {
  const int64_t wide = cdiv(a.n_in + a.n_out, 64) * a.n;
  return a.R <= 32 && wide >= kFillBlocks ? gradients_f<T, 4>(a, s) : gradients_f<T, 2>(a, s);
}

// Row tiles of a workgroup: as many as leave one workgroup to a CU, so that no
// second round runs half empty and x is read less often (32 tokens, 11008 x
// 4096 f16: 44 us with one, 28 with three).
template <typename T, int V, int MO>
hipError_t project_vm(const LowRankArgs& a, const LowRankLayout& l, hipStream_t s) {
  const int64_t rb = cdiv(a.n_out, 16 * MO);
  constexpr int threads = (kProjectWaves + V) * kWave;
  auto launch = [&](auto small) {
    return in_parts(a, rb * cdiv(a.T, 16 * V), threads, [&](const LowRankArgs& p, unsigned grid) {
      hipLaunchKernelGGL((lowrank_project_kernel<T, V, MO, decltype(small)::value != 0>),
                         dim3(grid), dim3(threads), staged_bytes(16 * V, a.R), s, p, l.slices_u,
                         (int)rb);
    });
  };
  return a.R <= 16 ? launch(Int<1>{}) : launch(Int<0>{});
}

template <typename T, int V>
hipError_t project_v(const LowRankArgs& a, const LowRankLayout& l, hipStream_t s) {
  const int64_t tiles = cdiv(a.n_out, 16) * cdiv(a.T, 16 * V);
  if (tiles <= 256) return project_vm<T, V, 1>(a, l, s);
  // three tiles' sums of 64 tokens leave no room for the ranks past 192
  const size_t three = (kProjectWaves + 1) * 3 * V * kWave * sizeof(f32x4) + staged_bytes(16 * V, a.R);
  if (tiles <= 512 || three > kSharedBytes) return project_vm<T, V, 2>(a, l, s);
  return project_vm<T, V, 3>(a, l, s);
}

// One launch for up to 16 tokens that cannot have more than one adapter, of up
// to 32 ranks, where what every workgroup reads for itself costs less than a second
// launch.  Its workgroups read x while others write: not where out shares memory
// with x.  us, one launch and two, one token, bf16:
//   add: all of A (its ranks rounded up to 16).  16 ranks of 4096 features 9.2 and
//   10.6, of 4608 10.0 and 10.8, of 6144 11.8 and 10.8, of 11008 17.4 and 11.3;
//   32 ranks of 2048 9.3 and 10.4, of 4096 13.2 and 11.1.
//   project: A and 16 rows of W, in as many rounds as the rows take with one such
//   workgroup a CU, against 48 rows each in the other form.  16 ranks of 4096 x 4096
//   13.0 and 17.0, of 8192 features 21.6 and 21.9, 4096 features and 11008 rows 34.1
//   and 27.8, 1024 and 11008 15.1 and 17.6, 4096 and 16384 45.9 and 49.1.  More
//   tokens read x a value at a time: 16 of 6144 x 4096 21.0 and 19.5, of 2048 x
//   11008 24.1 and 19.3.
bool few(int op, int64_t eb, int64_t T, int64_t S, int64_t n, int64_t R, int64_t n_in,
         int64_t n_out) {
  if (op == kLowRankBackward || T > kFewTokens || R > 32 || (T > 1 && S > 1 && n > 1)) return false;
  const int64_t row = n_in * eb, ranks = R <= 16 ? 16 : 32;
  if (op == kLowRankAdd) return ranks * row <= 144 * 1024;
  const int64_t rounds = cdiv(n_out, 16 * 256), others = cdiv(n_out, 48 * 256);
  return (ranks + 16) * row * rounds / others <=
         (T <= 1 ? 512 : rounds == 1 ? 384 : 288) * 1024;
}

template <typename T, bool PROJECT>
hipError_t few_t(const LowRankArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)cdiv(a.n_out, PROJECT ? 16 : 16 * kFewWaves)), block(kFewThreads);
  if (a.R <= 16)
    hipLaunchKernelGGL((lowrank_few_kernel<T, PROJECT, 1>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((lowrank_few_kernel<T, PROJECT, 2>), grid, block, 0, s, a);
  return hipGetLastError();
}

template <typename T>
hipError_t add_t(const LowRankArgs& a, const LowRankLayout& l, hipStream_t s) {
  if (l.few) return few_t<T, false>(a, s);
  hipError_t e = shrink<T, false, false>(a, l, s);
  if (e != hipSuccess) return e;
  if (!packs(kLowRankAdd, a.T, a.S)) return expand_v<T, 1>(a, l, s);
  if ((e = pack<T, false>(a, l, s)) != hipSuccess) return e;
  return expand_v<T, 16 / sizeof(T)>(a, l, s);
}

template <typename T>
hipError_t backward_t(const LowRankArgs& a, const LowRankLayout& l, hipStream_t s) {
  if (a.T > 0) {
    hipError_t e = shrink<T, true, false>(a, l, s);
    if (e != hipSuccess) return e;
    if ((e = pack<T, true>(a, l, s)) != hipSuccess) return e;
  }
  return gradients<T>(a, s);  // zeros where there are no tokens
}

template <typename T>
hipError_t project_t(const LowRankArgs& a, const LowRankLayout& l, hipStream_t s) {
  if (l.few) return few_t<T, true>(a, s);
  hipError_t e = shrink<T, false, true>(a, l, s);
  if (e != hipSuccess) return e;
  switch (l.width) {
    case 1: return project_v<T, 1>(a, l, s);
    case 2: return project_v<T, 2>(a, l, s);
    default: return project_v<T, 4>(a, l, s);
  }
}

}  // namespace

LowRankLayout lowrank_layout(int op, bool over_x, int dtype, int64_t T, int64_t S, int64_t n,
                             int64_t R, int64_t n_in, int64_t n_out) {
  LowRankLayout l{};
  const int64_t eb = dtype == kF32 ? 4 : 2;
  l.few = !over_x && few(op, eb, T, S, n, R, n_in, n_out);
  if (l.few) return l;   // one launch, nothing between
  if (T == 0) return l;  // the gradients' zeros alone
  l.Tp = cdiv(T, 128) * 128;  // whole tiles
  l.width = token_width(op, dtype, T, R);
  const int64_t tiles = cdiv(T, 16 * l.width);
  const double mean = (double)S / (double)(tiles > 0 ? tiles : 1);
  l.groups = adapter_groups(mean, S, n);
  // busy workgroups: an adapter in the mean, or each request that starts
  const double busy = mean < 1 ? 1 : mean < l.groups ? mean : l.groups;
  const double blocks = (double)tiles * busy * (double)cdiv(R, 64) * (op == kLowRankBackward ? 2 : 1);
  l.slices_u = slices_for(blocks, n_in);
  l.slices_du = op == kLowRankBackward ? slices_for(blocks, n_out) : 0;
  l.shrink_blocks = tiles * l.groups * cdiv(R, 64) * (l.slices_u + l.slices_du);
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
  const bool rows = packs(op, T, S), sides = op == kLowRankBackward;
  l.at_rows = take(rows ? (size_t)l.Tp * packed_row((int)R) : 0);
  l.at_up = take(rows ? (size_t)l.Tp * 4 : 0);
  l.at_ru = take(sides ? (size_t)R * l.Tp * 4 : 0);
  l.at_rdu = take(sides ? (size_t)R * l.Tp * 4 : 0);
  l.at_eu = take(sides ? (size_t)R * l.Tp : 0);
  l.at_edu = take(sides ? (size_t)R * l.Tp : 0);
  l.bytes = at;
  return l;
}

hipError_t launch_lowrank(int op, bool over_x, int dtype, LowRankArgs a, void* ws,
                          hipStream_t s) {
  const LowRankLayout l = lowrank_layout(op, over_x, dtype, a.T, a.S, a.n, a.R, a.n_in, a.n_out);
  char* w = (char*)ws;
  a.Tp = l.Tp;
  a.tokad = (int32_t*)(w + l.at_tokad);
  a.u = (float*)(w + l.at_u);
  a.du = (float*)(w + l.at_du);
  a.packed = w + l.at_packed;
  a.rows = w + l.at_rows;
  a.up = (float*)(w + l.at_up);
  a.ru = w + l.at_ru;
  a.rdu = w + l.at_rdu;
  a.eu = (uint8_t*)(w + l.at_eu);
  a.edu = (uint8_t*)(w + l.at_edu);
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
