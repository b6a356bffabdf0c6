// Cross entropy of singles over a vocabulary, its gradients, without the
// logits: z[t, v] = scale x_t . W_v is formed tile by tile on the matrix cores.
//
// Forward: a workgroup forms a tile of z transposed (vocabulary x tokens), so a
// lane holds one token and the tile's maximum and sum of powers are mostly in
// its registers; they go to the workspace, one pair for each token and tile, and
// a second kernel joins them. Backward: pieces of the vocabulary; for each,
// d = (g_nll + g_lse) exp(z - lse) - g_nll [v = target] goes to the workspace in
// the operands' type, then g_x += scale d W and g_W = scale d^T x are products
// over it. The weights' gradient is fp32, which one bf16 of d (2^-9 of each
// value) would not fill: it takes d as a pair of bf16, hi + lo (2^-17), in two
// products; g_x is rounded to bf16 itself and takes hi alone.
//
// Tokens without a target take no part: the others' rows are listed first, the
// forward reads x through the list, the backward copies the listed rows (with
// zeros behind the last one), so what an ignored row holds reaches nothing.
// Nothing is added with atomics; sums have one order.
#include "nt_internal.hpp"
#include "nt_product_tile.hpp"

#include <math.h>

#include <algorithm>

namespace nt {
namespace {

constexpr int kTlListThreads = 1024;
constexpr int64_t kTlListChunk = 4 * kTlListThreads;  // targets of a workgroup of the list

// Rows that have a target, in order: rows[0 .. *live), by workgroups that each
// count what lies before their own stretch of targets (that is read from cache,
// and spares launches). The others' results are zeros: nll, lse (forward) or the
// rows of g_x (backward).
__global__ __launch_bounds__(kTlListThreads) void k_tl_list(const int32_t* targets, int64_t T,
                                                            int32_t* rows, int64_t* live,
                                                            float* nll, float* lse) {
  __shared__ int part[kTlListThreads / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t first = (int64_t)blockIdx.x * kTlListChunk;
  int before = 0;
  for (int64_t t = threadIdx.x; t < first; t += kTlListThreads) before += targets[t] >= 0;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) before += __shfl_xor(before, m);
  if (lane == 0) part[wave] = before;
  __syncthreads();
  int64_t at = 0;
  for (int w = 0; w < kTlListThreads / 64; ++w) at += part[w];
  for (int u = 0; u < 4; ++u) {
    const int64_t t = first + u * kTlListThreads + threadIdx.x;
    const bool is = t < T && targets[t] >= 0;
    const unsigned long long who = __ballot(is);
    __syncthreads();
    if (lane == 0) part[wave] = __popcll(who);
    __syncthreads();
    int64_t mine = at;
    for (int w = 0; w < kTlListThreads / 64; ++w) {
      if (w < wave) mine += part[w];
      at += part[w];
    }
    if (is) {
      rows[mine + __popcll(who & ((1ull << lane) - 1))] = (int32_t)t;
    } else if (t < T && nll) {
      nll[t] = 0.0f;
      lse[t] = 0.0f;
    }
  }
  if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) *live = at;
}

// The listed rows of x, one after another, zeros behind them up to a whole tile.
template <typename T>
__global__ __launch_bounds__(256) void k_tl_gather(const T* x, const int32_t* rows,
                                                   const int64_t* live, T* out, int64_t chunks,
                                                   int64_t padded) {
  constexpr int V = 16 / (int)sizeof(T);
  const int64_t n = *live, most = (n + 255) / 256 * 256;
  const int64_t end = (most < padded ? most : padded) * chunks;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < end; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / chunks, c = i - r * chunks;
    Vec16<T> v;
    if (r < n) {
      v = load16(x + ((int64_t)rows[r] * chunks + c) * V);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) v.set(e, 0.0f);
    }
    store16(out + i * V, v);
  }
}

template <typename T> struct TlForward {
  const T* x;
  const T* W;
  const int32_t* targets;
  const int32_t* rows;
  const int64_t* live;
  float2* part;   // [tiles of the vocabulary][T]: maximum (in powers of 2) and sum
  float* at;      // [T] the target's logit, in powers of 2
  int64_t tokens, V;
  int C;
  float scale2;   // scale log2(e)
  uint32_t tiles_m, tiles_n;
};

__device__ __forceinline__ float tl_halves_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x),
                                                  __builtin_bit_cast(uint32_t, x), false, false);
  return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}

template <typename S>
__global__ __launch_bounds__(S::threads) void k_tl_forward(TlForward<typename S::type> p) {
  typedef typename S::type T;
  typedef PtAlong<T, S::m, S::threads> A;
  typedef PtAlong<T, S::n, S::threads> B;
  __shared__ __attribute__((aligned(16))) char smem[2 * S::bytes];
  uint32_t tm, tn;
  if (!pt_tile(blockIdx.x, p.tiles_m, p.tiles_n, &tm, &tn)) return;
  const int64_t v0 = (int64_t)tm * S::m, t0 = (int64_t)tn * S::n, live = *p.live;
  if (t0 >= live) return;
  const A la([&](int r) { return p.W + (v0 + r < p.V ? v0 + r : p.V - 1) * p.C; });
  const B lb([&](int r) {
    return p.x + (int64_t)p.rows[t0 + r < live ? t0 + r : live - 1] * p.C;
  });
  f32x16 z[S::mt][S::nt];
  pt_product<S, A, B>(z, smem, (p.C + S::bk - 1) / S::bk, [&](int64_t j, uint32_t to) {
    la.start(j * S::bk, p.C, to);
    lb.start(j * S::bk, p.C, to + S::m * 128);
  });

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5;
  const int m0 = wave / S::wn * 32 * S::mt, n0 = wave % S::wn * 32 * S::nt;
  const int64_t past = p.V - v0 - m0 - 4 * h;  // the vocabulary's end from the lane's rows on
  const int left = past < 0 ? 0 : past < S::m ? (int)past : S::m;
  float2* stats = reinterpret_cast<float2*>(smem);  // [wm][n]
  __syncthreads();
#pragma unroll
  for (int j = 0; j < S::nt; ++j) {
    const int64_t t = t0 + n0 + 32 * j + (lane & 31);
    int target = -1;  // from the lane's rows on, where it is among them
    if (t < live) {
      const int64_t from = p.targets[p.rows[t]] - v0 - m0 - 4 * h;
      // the other half of the wave holds every other four rows
      if (from >= 0 && from < 32 * S::mt && !(from & 4)) target = (int)from;
    }
    float most = -INFINITY;
#pragma unroll
    for (int i = 0; i < S::mt; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        z[i][j][e] *= p.scale2;
        most = fmaxf(most, z[i][j][e]);
      }
    if (v0 + S::m > p.V) {  // the last tile of the vocabulary
      int end = left;
      asm volatile("" : "+v"(end)::"memory");  // not compared ahead for every j
      most = -INFINITY;
#pragma unroll
      for (int i = 0; i < S::mt; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if (32 * i + 8 * (e >> 2) + (e & 3) >= end) z[i][j][e] = -INFINITY;
          most = fmaxf(most, z[i][j][e]);
        }
    }
    if (__ballot(target >= 0)) {
      at_rare();
      float found = 0.0f;
#pragma unroll
      for (int i = 0; i < S::mt; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          found = 32 * i + 8 * (e >> 2) + (e & 3) == target ? z[i][j][e] : found;
      if (target >= 0) p.at[t] = found;
    }
    most = at_halves_max(most);
    const float base = most == -INFINITY ? 0.0f : most;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < S::mt; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) sum += __builtin_amdgcn_exp2f(z[i][j][e] - base);
    sum = tl_halves_sum(sum);
    if (h == 0) stats[wave / S::wn * S::n + n0 + 32 * j + lane] = make_float2(most, sum);
  }
  __syncthreads();
  for (int c = threadIdx.x; c < S::n; c += S::threads) {
    if (t0 + c >= live) break;
    float most = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int w = 0; w < S::wm; ++w) most = fmaxf(most, stats[w * S::n + c].x);
    const float base = most == -INFINITY ? 0.0f : most;
#pragma unroll
    for (int w = 0; w < S::wm; ++w) {
      const float2 s = stats[w * S::n + c];
      sum += s.y * __builtin_amdgcn_exp2f(s.x - base);
    }
    p.part[(int64_t)tm * p.tokens + t0 + c] = make_float2(most, sum);
  }
}

// Joins the tiles' statistics: 16 tokens a workgroup, 16 threads a token.
__global__ __launch_bounds__(256) void k_tl_join(const float2* part, const float* at,
                                                 const int32_t* targets, const int32_t* rows,
                                                 const int64_t* live, float* nll, float* lse,
                                                 int64_t tokens, int64_t V, uint32_t tiles) {
  __shared__ float2 stats[16][17];
  const int c = threadIdx.x & 15, k = threadIdx.x >> 4;
  const int64_t n = *live;
  for (int64_t first = (int64_t)blockIdx.x * 16; first < n; first += (int64_t)gridDim.x * 16) {
    const int64_t t = first + c;
    __syncthreads();  // stats may still be read
    float most = -INFINITY, sum = 0.0f;
    if (t < n)
      for (uint32_t i = k; i < tiles; i += 16) {
        const float2 s = part[(int64_t)i * tokens + t];
        const float m = fmaxf(most, s.x), base = m == -INFINITY ? 0.0f : m;
        sum = sum * __builtin_amdgcn_exp2f(most - base) + s.y * __builtin_amdgcn_exp2f(s.x - base);
        most = m;
      }
    stats[k][c] = make_float2(most, sum);
    __syncthreads();
    if (k || t >= n) continue;
    for (int i = 1; i < 16; ++i) most = fmaxf(most, stats[i][c].x);
    const float base = most == -INFINITY ? 0.0f : most;
    sum = 0.0f;
    for (int i = 0; i < 16; ++i) sum += stats[i][c].y * __builtin_amdgcn_exp2f(stats[i][c].x - base);
    const float rest = __builtin_amdgcn_logf(sum);  // log2
    const int64_t row = rows[t];
    lse[row] = (most + rest) * kLn2;
    // a target that the vocabulary does not hold
    nll[row] = targets[row] < V ? ((most - at[t]) + rest) * kLn2 : __builtin_nanf("");
  }
}

template <typename T> struct TlGrad {
  const T* x;     // the listed rows, one after another
  const T* W;
  const int32_t* targets;
  const int32_t* rows;
  const int64_t* live;
  const float* lse;
  const float* g_nll;
  const float* g_lse;
  T* d;           // [padded tokens][piece], in bf16 hi, then lo behind `plane` elements
  int64_t plane, piece;
  int64_t v_first, V;  // the piece's first row of W, and all rows
  float* sums;    // products: [splits][...] fp32
  float* out;     // g_W
  int64_t tokens; // capacity of the lists
  int C, splits, accumulate;
  float scale, scale2;
  uint32_t tiles_m, tiles_n;
};

// d of a tile: rows of W (m) x tokens (n).
template <typename S>
__global__ __launch_bounds__(S::threads) void k_tl_logit_grad(TlGrad<typename S::type> p) {
  typedef typename S::type T;
  typedef PtAlong<T, S::m, S::threads> A;
  typedef PtAlong<T, S::n, S::threads> B;
  __shared__ __attribute__((aligned(16))) char smem[2 * S::bytes];
  uint32_t tm, tn;
  if (!pt_tile(blockIdx.x, p.tiles_m, p.tiles_n, &tm, &tn)) return;
  const int64_t c0 = (int64_t)tm * S::m, v0 = p.v_first + c0, t0 = (int64_t)tn * S::n;
  const int64_t live = *p.live;
  if (t0 >= live) return;
  const A la([&](int r) { return p.W + (v0 + r < p.V ? v0 + r : p.V - 1) * p.C; });
  const B lb([&](int r) { return p.x + (t0 + r) * p.C; });
  f32x16 z[S::mt][S::nt];
  pt_product<S, A, B>(z, smem, (p.C + S::bk - 1) / S::bk, [&](int64_t j, uint32_t to) {
    la.start(j * S::bk, p.C, to);
    lb.start(j * S::bk, p.C, to + S::m * 128);
  });

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5;
  const int m0 = wave / S::wn * 32 * S::mt, n0 = wave % S::wn * 32 * S::nt;
#pragma unroll
  for (int j = 0; j < S::nt; ++j) {
    const int64_t t = t0 + n0 + 32 * j + (lane & 31);
    float both = 0.0f, one = 0.0f, base = 0.0f;
    int target = -1, left = 0;  // from the lane's rows of W on
    if (t < live) {
      const int64_t row = p.rows[t], past = p.V - v0 - m0 - 4 * h;
      const int64_t from = p.targets[row] - v0 - m0 - 4 * h;
      if (from >= 0 && from < 32 * S::mt) target = (int)from;
      left = past < 0 ? 0 : past < S::m ? (int)past : S::m;
      one = p.g_nll[row];
      both = (p.g_lse ? one + p.g_lse[row] : one) * p.scale;
      one *= p.scale;
      base = p.lse[row] * kLog2e;
      if (p.targets[row] >= p.V) both = __builtin_nanf("");
    }
    T* to = p.d + t * p.piece + c0 + m0 + 4 * h;
#pragma unroll
    for (int i = 0; i < S::mt; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int v = 32 * i + 8 * g + e;
          f[e] = both * __builtin_amdgcn_exp2f(z[i][j][4 * g + e] * p.scale2 - base);
          if (v == target) f[e] -= one;
          // rows of W that are not there, and tokens behind the last one
          if (v >= left) f[e] = 0.0f;
        }
        at_store4(to + 32 * i + 8 * g, f[0], f[1], f[2], f[3]);
        if constexpr (sizeof(T) == 2) {
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] -= (float)(T)f[e];
          at_store4(to + p.plane + 32 * i + 8 * g, f[0], f[1], f[2], f[3]);
        }
      }
  }
}

// sums[split][t][c] (+)= sum over the split's rows v of the piece of d[t, v] W[v, c].
template <typename S>
__global__ __launch_bounds__(S::threads) void k_tl_x_grad(TlGrad<typename S::type> p) {
  typedef typename S::type T;
  typedef PtAcross<T, S::m, S::threads> A;
  typedef PtAlong<T, S::n, S::threads> B;
  __shared__ __attribute__((aligned(16))) char smem[2 * S::bytes];
  uint32_t tm, tn;
  if (!pt_tile(blockIdx.x, p.tiles_m, p.tiles_n, &tm, &tn)) return;
  const int64_t c0 = (int64_t)tm * S::m, t0 = (int64_t)tn * S::n, live = *p.live;
  if (t0 >= live) return;
  const int64_t K = p.V - p.v_first < p.piece ? p.V - p.v_first : p.piece;
  const int64_t tiles = (K + S::bk - 1) / S::bk, each = (tiles + p.splits - 1) / p.splits;
  const int64_t begin = blockIdx.y * each, end = begin + each < tiles ? begin + each : tiles;
  const A la(p.W + p.v_first * p.C + c0, p.C - c0, p.C);
  const B lb([&](int r) { return p.d + (t0 + r) * p.piece; });
  f32x16 acc[S::mt][S::nt];
  pt_product<S, A, B>(acc, smem, end - begin, [&](int64_t j, uint32_t to) {
    la.start((begin + j) * S::bk, K, to);
    lb.start((begin + j) * S::bk, p.piece, to + S::m * 128);
  });
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5;
  const int m0 = wave / S::wn * 32 * S::mt, n0 = wave % S::wn * 32 * S::nt;
#pragma unroll
  for (int j = 0; j < S::nt; ++j) {
    const int64_t t = t0 + n0 + 32 * j + (lane & 31);
    if (t >= live) continue;
    float* to = p.sums + ((int64_t)blockIdx.y * p.tokens + t) * p.C;
#pragma unroll
    for (int i = 0; i < S::mt; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int64_t c = c0 + m0 + 32 * i + 8 * g + 4 * h;
        if (c >= p.C) continue;
        f32x4 f = {acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2],
                   acc[i][j][4 * g + 3]};
        if (p.accumulate) f += *reinterpret_cast<const f32x4*>(to + c);
        *reinterpret_cast<f32x4*>(to + c) = f;
      }
  }
}

// g_W[v][c] (+)= sum over tokens of d[t, v] x[t, c], d as hi and lo in turn; with
// more than one split the parts go to sums[split][v][c].
template <typename S>
__global__ __launch_bounds__(S::threads) void k_tl_w_grad(TlGrad<typename S::type> p) {
  typedef typename S::type T;
  typedef PtAcross<T, S::m, S::threads> A;
  typedef PtAcross<T, S::n, S::threads> B;
  __shared__ __attribute__((aligned(16))) char smem[2 * S::bytes];
  uint32_t tm, tn;
  if (!pt_tile(blockIdx.x, p.tiles_m, p.tiles_n, &tm, &tn)) return;
  const int64_t c0 = (int64_t)tm * S::m, n_first = (int64_t)tn * S::n, live = *p.live;
  const int64_t one = (live + S::bk - 1) / S::bk;
  const int64_t tiles = sizeof(T) == 2 ? 2 * one : one, each = (tiles + p.splits - 1) / p.splits;
  const int64_t begin = blockIdx.y * each, end = begin + each < tiles ? begin + each : tiles;
  const A la(p.x + c0, p.C - c0, p.C);
  const B lb(p.d + n_first, p.piece - n_first, p.piece);
  B lo = lb;
  lo.base += p.plane;
  f32x16 acc[S::mt][S::nt];
  pt_product<S, A, B>(acc, smem, end - begin, [&](int64_t j, uint32_t to) {
    const bool low = begin + j >= one;
    const int64_t k0 = (begin + j - (low ? one : 0)) * S::bk;
    la.start(k0, p.tokens, to);
    (low ? lo : lb).start(k0, p.tokens, to + S::m * 128);
  });
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5;
  const int m0 = wave / S::wn * 32 * S::mt, n0 = wave % S::wn * 32 * S::nt;
  const int64_t rows = p.V - p.v_first < p.piece ? p.V - p.v_first : p.piece;
#pragma unroll
  for (int j = 0; j < S::nt; ++j) {
    const int64_t v = n_first + n0 + 32 * j + (lane & 31);
    if (v >= rows) continue;
    float* to = p.splits > 1 ? p.sums + ((int64_t)blockIdx.y * p.piece + v) * p.C
                             : p.out + (p.v_first + v) * p.C;
#pragma unroll
    for (int i = 0; i < S::mt; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int64_t c = c0 + m0 + 32 * i + 8 * g + 4 * h;
        if (c >= p.C) continue;
        f32x4 f = {acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2],
                   acc[i][j][4 * g + 3]};
        if (p.splits == 1 && p.accumulate) f += *reinterpret_cast<const f32x4*>(to + c);
        *reinterpret_cast<f32x4*>(to + c) = f;
      }
  }
}

// The splits of g_x joined and rounded, each listed row at its token's place, zeros at the others.
template <typename T>
__global__ __launch_bounds__(256) void k_tl_x_join(const float* sums, const int32_t* targets,
                                                   const int32_t* rows, const int64_t* live,
                                                   T* g_x, int64_t tokens, int64_t capacity,
                                                   int C, int splits) {
  // one thread takes 4 columns
  const int64_t quads = C / 4, n = *live;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < tokens * quads;
       i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / quads, c = (i - r * quads) * 4;
    if (r < n) {
      f32x4 f = *reinterpret_cast<const f32x4*>(sums + r * C + c);
      for (int s = 1; s < splits; ++s)
        f += *reinterpret_cast<const f32x4*>(sums + ((int64_t)s * capacity + r) * C + c);
      at_store4(g_x + (int64_t)rows[r] * C + c, f[0], f[1], f[2], f[3]);
    }
    if (targets[r] < 0) at_store4(g_x + r * C + c, 0.0f, 0.0f, 0.0f, 0.0f);
  }
}

// The splits of a piece of g_W joined.
__global__ __launch_bounds__(256) void k_tl_w_join(const float* sums, float* out, int64_t quads,
                                                   int64_t each, int splits, int accumulate) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < quads; i += (int64_t)gridDim.x * 256) {
    f32x4 f = *reinterpret_cast<const f32x4*>(sums + 4 * i);
    for (int s = 1; s < splits; ++s) f += *reinterpret_cast<const f32x4*>(sums + s * each + 4 * i);
    if (accumulate) f += *reinterpret_cast<const f32x4*>(out + 4 * i);
    *reinterpret_cast<f32x4*>(out + 4 * i) = f;
  }
}

__global__ void k_tl_fill(float* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    p[i] = 0.0f;
}

int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }
int64_t tiles_of(int64_t x, int64_t tile) { return (x + tile - 1) / tile; }
// Workgroups of a kernel that walks on with its grid.
uint32_t blocks_of(int64_t x, int64_t each) {
  return (uint32_t)std::min<int64_t>(tiles_of(x, each), 1 << 16);
}

typedef PtShape<bf16, 4, 2, 2, 4> Big;                       // 256 x 256, 8 waves
template <typename T> using Mid = PtShape<T, 2, 2, 2, 2>;   // 128 x 128, 4 waves
template <typename T> using Thin = PtShape<T, 1, 1, 4, 1>;  // 128 x 32, 4 waves

constexpr int64_t kCus = 256;
constexpr int64_t kPieceBytes = int64_t(512) << 20;  // of d
constexpr int kMostSplits = 16;

struct Plan {
  int64_t padded, piece, planes;
  int x_splits, w_splits;
  // the workspace
  size_t rows, live, part, at, x, d, x_sums, w_sums, total;
};

// Tiles of 256 x 256 where they fill the card once. Only in bf16: fp32 products
// take sixteen times as long, and a tile of 128 x 128 keeps up with its loads.
bool big_tiles(int64_t m, int64_t n, bool narrow) {
  return narrow && tiles_of(m, 256) * tiles_of(n, 256) >= kCus;
}

int splits_of(int64_t tiles, int64_t steps) {
  // about one workgroup for each compute unit and half as many again, eight steps each at least
  int64_t s = tiles >= kCus ? 1 : (kCus + kCus / 2) / tiles;
  if (s > steps / 8) s = steps / 8;
  if (s > kMostSplits) s = kMostSplits;
  return s < 1 ? 1 : (int)s;
}

int64_t forward_m(int64_t T, int64_t V, bool narrow) {
  return T > 32 && big_tiles(V, T, narrow) ? 256 : 128;
}

Plan forward_plan(int64_t T, int64_t V, nt_dtype dtype) {
  Plan p = {};
  size_t at = 0;
  p.rows = at; at = align256(at + sizeof(int32_t) * T);
  p.live = at; at = align256(at + sizeof(int64_t));
  p.at = at; at = align256(at + sizeof(float) * T);
  p.part = at; at = align256(at + sizeof(float2) * T * tiles_of(V, forward_m(T, V, dtype == NT_BF16)));
  p.total = at;
  return p;
}

Plan backward_plan(int64_t T, int64_t V, int64_t C, nt_dtype dtype) {
  Plan p = {};
  const int64_t es = dtype == NT_BF16 ? 2 : 4;
  p.planes = dtype == NT_BF16 ? 2 : 1;
  p.padded = up(T, 256);
  const int64_t most = std::max<int64_t>(256, kPieceBytes / (p.padded * es * p.planes) / 256 * 256);
  const int64_t pieces = tiles_of(V, most);
  p.piece = up(tiles_of(V, pieces), 256);
  const int64_t bk = 128 / es;
  const bool bx = big_tiles(C, T, p.planes == 2), bw = big_tiles(C, p.piece, p.planes == 2);
  const int64_t x_tiles = bx ? tiles_of(C, 256) * tiles_of(T, 256) : tiles_of(C, 128) * tiles_of(T, 128);
  const int64_t w_tiles = bw ? tiles_of(C, 256) * tiles_of(p.piece, 256)
                             : tiles_of(C, 128) * tiles_of(std::min(p.piece, up(V, 128)), 128);
  p.x_splits = splits_of(x_tiles, p.piece / bk);
  p.w_splits = splits_of(w_tiles, p.planes * p.padded / bk);
  size_t at = 0;
  p.rows = at; at = align256(at + sizeof(int32_t) * T);
  p.live = at; at = align256(at + sizeof(int64_t));
  p.x = at; at = align256(at + es * p.padded * C);
  p.d = at; at = align256(at + es * p.planes * p.padded * p.piece);
  p.x_sums = at; at = align256(at + sizeof(float) * p.x_splits * p.padded * C);
  p.w_sums = at;
  if (p.w_splits > 1) at = align256(at + sizeof(float) * p.w_splits * p.piece * C);
  p.total = at;
  return p;
}

template <typename S>
hipError_t run_forward(TlForward<typename S::type> a, hipStream_t s) {
  a.tiles_m = (uint32_t)tiles_of(a.V, S::m);
  a.tiles_n = (uint32_t)tiles_of(a.tokens, S::n);
  k_tl_forward<S><<<dim3((uint32_t)pt_grid((int64_t)a.tiles_m * a.tiles_n)), S::threads, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t forward(const void* x, const void* W, const int32_t* targets, float* nll, float* lse,
                   int64_t tokens, int64_t V, int C, float scale, char* ws, nt_dtype dtype, hipStream_t s) {
  const Plan p = forward_plan(tokens, V, dtype);
  int32_t* rows = reinterpret_cast<int32_t*>(ws + p.rows);
  int64_t* live = reinterpret_cast<int64_t*>(ws + p.live);
  k_tl_list<<<(uint32_t)tiles_of(tokens, kTlListChunk), kTlListThreads, 0, s>>>(targets, tokens,
                                                                               rows, live, nll, lse);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  TlForward<T> a = {static_cast<const T*>(x), static_cast<const T*>(W), targets, rows, live,
                    reinterpret_cast<float2*>(ws + p.part), reinterpret_cast<float*>(ws + p.at),
                    tokens, V, C, scale * kLog2e, 0, 0};
  const int64_t m = forward_m(tokens, V, dtype == NT_BF16);
  if constexpr (sizeof(T) == 2)
    e = m == 256 ? run_forward<Big>(a, s)
                 : tokens <= 32 ? run_forward<Thin<T>>(a, s) : run_forward<Mid<T>>(a, s);
  else
    e = tokens <= 32 ? run_forward<Thin<T>>(a, s) : run_forward<Mid<T>>(a, s);
  if (e != hipSuccess) return e;
  k_tl_join<<<blocks_of(tokens, 16), 256, 0, s>>>(
      a.part, a.at, targets, rows, live, nll, lse, tokens, V, (uint32_t)tiles_of(V, m));
  return hipGetLastError();
}

// One of the gradient's products, m x n results, in tiles of the size that fits.
enum Product { kLogits, kSingles, kWeights };
template <typename S, Product P> hipError_t run_tiles(TlGrad<typename S::type> a, int64_t m, int64_t n, hipStream_t s) {
  a.tiles_m = (uint32_t)tiles_of(m, S::m);
  a.tiles_n = (uint32_t)tiles_of(n, S::n);
  const dim3 grid((uint32_t)pt_grid((int64_t)a.tiles_m * a.tiles_n), a.splits);
  if constexpr (P == kLogits) k_tl_logit_grad<S><<<grid, S::threads, 0, s>>>(a);
  if constexpr (P == kSingles) k_tl_x_grad<S><<<grid, S::threads, 0, s>>>(a);
  if constexpr (P == kWeights) k_tl_w_grad<S><<<grid, S::threads, 0, s>>>(a);
  return hipGetLastError();
}
template <Product P, typename T>
hipError_t run_product(const TlGrad<T>& a, bool big, int64_t m, int64_t n, hipStream_t s) {
  if constexpr (sizeof(T) == 2)
    if (big) return run_tiles<Big, P>(a, m, n, s);
  return run_tiles<Mid<T>, P>(a, m, n, s);
}

template <typename T>
hipError_t backward(const void* x, const void* W, const int32_t* targets, const float* lse,
                    const float* g_nll, const float* g_lse, void* g_x, float* g_W, int64_t tokens,
                    int64_t V, int C, float scale, bool accumulate, char* ws, nt_dtype dtype,
                    hipStream_t s) {
  const Plan p = backward_plan(tokens, V, C, dtype);
  const bool narrow = dtype == NT_BF16;
  int32_t* rows = reinterpret_cast<int32_t*>(ws + p.rows);
  int64_t* live = reinterpret_cast<int64_t*>(ws + p.live);
  T* xs = reinterpret_cast<T*>(ws + p.x);
  k_tl_list<<<(uint32_t)tiles_of(tokens, kTlListChunk), kTlListThreads, 0, s>>>(
      targets, tokens, rows, live, nullptr, nullptr);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t chunks = C * (int64_t)sizeof(T) / 16;
  k_tl_gather<T><<<blocks_of(p.padded * chunks, 256), 256, 0, s>>>(
      static_cast<const T*>(x), rows, live, xs, chunks, p.padded);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  TlGrad<T> a = {xs, static_cast<const T*>(W), targets, rows, live, lse, g_nll, g_lse,
                 reinterpret_cast<T*>(ws + p.d), p.padded * p.piece, p.piece, 0, V,
                 reinterpret_cast<float*>(ws + p.x_sums), g_W, p.padded, C, 1, 0, scale,
                 scale * kLog2e, 0, 0};
  for (int64_t v = 0; v < V; v += p.piece) {
    const int64_t n = std::min(p.piece, V - v);
    a.v_first = v;
    a.accumulate = 0;
    a.splits = 1;
    // whole tiles of d: the products read up to the next multiple of a step of k
    const int64_t m = std::min(p.piece, up(n, 256));
    e = run_product<kLogits>(a, big_tiles(m, tokens, narrow), m, tokens, s);
    if (e != hipSuccess) return e;
    if (g_x) {
      a.accumulate = v > 0;
      a.splits = p.x_splits;
      e = run_product<kSingles>(a, big_tiles(C, tokens, narrow), C, tokens, s);
      if (e != hipSuccess) return e;
    }
    if (g_W) {
      TlGrad<T> b = a;
      b.accumulate = accumulate;
      b.splits = p.w_splits;
      b.sums = reinterpret_cast<float*>(ws + p.w_sums);
      e = run_product<kWeights>(b, big_tiles(C, p.piece, narrow), C, n, s);
      if (e != hipSuccess) return e;
      if (p.w_splits > 1) {
        const int64_t quads = n * C / 4;
        k_tl_w_join<<<blocks_of(quads, 256), 256, 0, s>>>(
            b.sums, g_W + v * C, quads, p.piece * C, p.w_splits, accumulate);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
      }
    }
  }
  if (!g_x) return hipSuccess;
  k_tl_x_join<T><<<blocks_of(tokens * (C / 4), 256), 256, 0, s>>>(
      a.sums, targets, rows, live, static_cast<T*>(g_x), tokens, p.padded, C, p.x_splits);
  return hipGetLastError();
}

}  // namespace

size_t token_loss_ws_bytes(int64_t tokens, int64_t V, nt_dtype dtype) {
  return tokens ? forward_plan(tokens, V, dtype).total : 0;
}

size_t token_loss_backward_ws_bytes(int64_t tokens, int64_t V, int C, nt_dtype dtype) {
  return tokens ? backward_plan(tokens, V, C, dtype).total : 0;
}

hipError_t launch_token_loss(const void* x, const void* W, const int32_t* targets, float* nll,
                             float* lse, int64_t tokens, int64_t V, int C, float scale,
                             nt_dtype dtype, void* ws, hipStream_t s) {
  if (tokens == 0) return hipSuccess;
  char* w = static_cast<char*>(ws);
  return dtype == NT_BF16 ? forward<bf16>(x, W, targets, nll, lse, tokens, V, C, scale, w, dtype, s)
                          : forward<float>(x, W, targets, nll, lse, tokens, V, C, scale, w, dtype, s);
}

hipError_t launch_token_loss_backward(const void* x, const void* W, const int32_t* targets,
                                      const float* lse, const float* g_nll, const float* g_lse,
                                      void* g_x, float* g_W, int64_t tokens, int64_t V, int C,
                                      float scale, bool accumulate, nt_dtype dtype, void* ws,
                                      hipStream_t s) {
  if (tokens == 0) {  // nothing to add
    if (!g_W || accumulate) return hipSuccess;
    const int64_t n = V * C;
    k_tl_fill<<<blocks_of(n, 256), 256, 0, s>>>(g_W, n);
    return hipGetLastError();
  }
  char* w = static_cast<char*>(ws);
  return dtype == NT_BF16 ? backward<bf16>(x, W, targets, lse, g_nll, g_lse, g_x, g_W, tokens, V, C,
                                           scale, accumulate, w, dtype, s)
                          : backward<float>(x, W, targets, lse, g_nll, g_lse, g_x, g_W, tokens, V,
                                            C, scale, accumulate, w, dtype, s);
}

}  // namespace nt
