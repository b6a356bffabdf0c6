// Cross entropy of singles over a vocabulary, its gradients, without the
// logits: z[t, v] = scale x_t . W_v is formed tile by tile on the matrix cores.
//
// Forward: a workgroup forms a tile of z transposed (vocabulary x tokens), so a
// lane holds one token and the tile's maximum and sum of powers are mostly in
// its registers; they go to the workspace, one pair for each token and tile, and
// a second kernel joins them. Backward: pieces of the vocabulary; for each,
// d = (g_nll + g_lse) exp(z - lse) - g_nll [v = target] goes to the workspace in
// the operands' type, then g_x += scale d W and g_W = scale d^T x are products
// over it. In bf16 one rounding of d (2^-9 of each value) would be seen in both: g_W is
// fp32, and g_x, which is rounded once itself, would be off by up to its own half step
// again where terms cancel. Both take d as a pair of bf16, hi + lo (2^-17), in two products.
//
// Tokens without a target take no part: the others' rows are listed first, the
// forward reads x through the list, the backward copies the listed rows (with
// zeros behind the last one), so what an ignored row holds reaches nothing.
// Nothing is added with atomics; sums have one order.
#include "nt_internal.hpp"
#include "nt_product_tile.hpp"
#include "nt_token_loss_plan.hpp"

#include <math.h>

#include <algorithm>

namespace nt {
namespace {

using namespace token_loss;

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

// Rows of an array [rows, C] transposed, to [C][ld], and (copy given) as they are,
// to [..][C]: the rows of a list (list given), or the rows from `first` on. Columns of the
// result from `*live` (or `rows`) on are zeros up to a whole tile of 256. Tiles of 64
// x 64 pass through LDS, so both sides are whole lines.
template <typename T> struct TlTranspose {
  const T* from;
  T* to;
  T* copy;
  const int32_t* list;
  const int64_t* live;
  int64_t rows, ld;
  int C;
};
// Two arrays in one launch, the second one (blockIdx.z 1) where there is one.
template <typename T>
__global__ __launch_bounds__(256) void k_tl_transpose(TlTranspose<T> p, TlTranspose<T> second) {
  if (blockIdx.z) p = second;
  constexpr int V = 16 / (int)sizeof(T), kChunks = 64 / V;  // of a tile's row
  __shared__ T tile[64][64 + V];
  const int64_t rows = p.live ? *p.live : p.rows;
  const int64_t r0 = (int64_t)blockIdx.x * 64;
  const int c0 = (int)blockIdx.y * 64;
  if (r0 >= (rows + 255) / 256 * 256) return;
#pragma unroll
  for (int i = threadIdx.x; i < 64 * kChunks; i += 256) {
    const int r = i / kChunks, c = i % kChunks * V;
    Vec16<T> v;
#pragma unroll
    for (int e = 0; e < V; ++e) v.set(e, 0.0f);
    if (c0 + c < p.C) {
      if (r0 + r < rows) v = load16(p.from + (p.list ? p.list[r0 + r] : r0 + r) * p.C + c0 + c);
      if (p.copy) store16(p.copy + (r0 + r) * p.C + c0 + c, v);
    }
    store16(&tile[r][c], v);
  }
  __syncthreads();
  if (!p.to) return;
#pragma unroll
  for (int i = threadIdx.x; i < 64 * kChunks; i += 256) {
    const int c = i / kChunks, r = i % kChunks * V;
    Vec16<T> v;
#pragma unroll
    for (int e = 0; e < V; ++e) v.v[e] = tile[r + e][c];
    if (c0 + c < p.C) store16(p.to + (c0 + c) * p.ld + r0 + r, v);
  }
}

template <typename T> struct TlForward {
  const T* x;
  const T* W;
  const int32_t* targets;
  const int32_t* rows;
  const int64_t* live;
  float2* part;   // [tiles of the vocabulary][T]: base (in powers of 2) and sum of the powers
  float* at;      // [T] the target's logit before its scale
  int64_t tokens, V;
  int C;
  float scale2;   // scale log2(e)
  uint32_t tiles_m;
};

// A value of the four lanes that hold a token joined.
__device__ __forceinline__ float tl_max4(float x) {
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float tl_sum4(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

// Bound by the matrix cores at the clock that the card's power leaves: 8,007 tokens over
// 65,537 words of 2,048 in bf16 1.73 ms, 1,240 TFLOP/s, cores busy for 66 % of the cycles.
// What is not: a tile's first loads and its statistics (a workgroup that walks over tiles
// with the next one's loads ahead of the statistics took 1.72 ms and was not kept).
template <typename S>
__global__ __launch_bounds__(S::threads) void k_tl_forward(TlForward<typename S::type> p) {
  typedef typename S::type T;
  typedef PtAlong<T, S::m, S::threads> A;
  typedef PtAlong<T, S::n, S::threads> B;
  __shared__ __attribute__((aligned(256))) char smem[S::lds];
  uint32_t tm, tn;
  const int64_t live = *p.live;
  if (!pt_tile(blockIdx.x, p.tiles_m, (uint32_t)((live + S::n - 1) / S::n), &tm, &tn)) return;
  const int64_t v0 = (int64_t)tm * S::m, t0 = (int64_t)tn * S::n;
  const A la(p.W + v0 * p.C, p.C, [&](int r) { return v0 + r < p.V ? r : p.V - 1 - v0; });
  const B lb(p.x, p.C, [&](int r) {
    return (int64_t)p.rows[t0 + r < live ? t0 + r : live - 1];
  });
  PtSums<S> z;
  pt_product<true, S, A, B>(
      z, smem, (p.C + S::bk - 1) / S::bk,
      [&](int64_t j, uint32_t to) { la.start(j * S::bk, p.C, to); },
      [&](int64_t j, uint32_t to) { lb.start(j * S::bk, p.C, to); });

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4;
  const int m0 = z.first_m(), n0 = z.first_n();
  const int64_t past = p.V - v0 - m0 - 4 * g;  // the vocabulary's end from the lane's rows on
  const int left = past < 0 ? 0 : past < S::m ? (int)past : S::m;
  float2* stats = reinterpret_cast<float2*>(smem);  // [wm][n]
  const float factor = fabsf(p.scale2);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < S::nt; ++j) {
    const int64_t t = t0 + n0 + 16 * j + (lane & 15);
    int target = -1;  // from the lane's rows on, where it is among them
    if (t < live) {
      const int64_t from = p.targets[p.rows[t]] - v0 - m0 - 4 * g;
      if (from >= 0 && from < 16 * S::mt && from % 16 < 4) target = (int)from;
    }
    if (p.scale2 < 0.0f) {  // then all logits the other way round
      at_rare();
#pragma unroll
      for (int i = 0; i < S::mt; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) z.d[i][j][e] = -z.d[i][j][e];
    }
    if (v0 + S::m > p.V) {  // the last tile of the vocabulary
      int end = left;
      asm volatile("" : "+v"(end)::"memory");  // not compared ahead for every j
#pragma unroll
      for (int i = 0; i < S::mt; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (16 * i + e >= end) z.d[i][j][e] = -INFINITY;
    }
    if (__ballot(target >= 0)) {
      at_rare();
      float found = 0.0f;
#pragma unroll
      for (int i = 0; i < S::mt; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) found = 16 * i + e == target ? z.d[i][j][e] : found;
      if (target >= 0) p.at[t] = found;
    }
    float most = -INFINITY;
#pragma unroll
    for (int i = 0; i < S::mt; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) most = fmaxf(most, z.d[i][j][e]);
    // The powers count from the base as it is rounded here, the join as well, and the
    // target's logit is taken from it unrounded (a product and a sum in one rounding), so
    // that what the base lost cancels in nll. (-inf times a factor of 0 would be NaN.)
    most = tl_max4(most);
    most = most == -INFINITY ? most : most * factor;
    const float base = most == -INFINITY ? 0.0f : most;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < S::mt; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        sum += __builtin_amdgcn_exp2f(__builtin_fmaf(z.d[i][j][e], factor, -base));
    sum = tl_sum4(sum);
    if (g == 0) stats[wave / S::wn * S::n + n0 + 16 * j + lane] = make_float2(most, sum);
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
                                                 int64_t tokens, int64_t V, uint32_t tiles,
                                                 float factor) {
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
    nll[row] = targets[row] < V ? (rest - __builtin_fmaf(at[t], factor, -most)) * kLn2
                                : __builtin_nanf("");
  }
}

// Few tokens (at most 32, one new token of each sample): the rows of W are read once
// and that bounds it, so they go from memory to the matrix cores' registers as they
// are, 16 rows a wave, without LDS and barriers, several loads of each lane in flight
// and all waves of the card at it. A wave keeps each token's
// maximum and sum over the rows that it takes. The list of tokens is a ballot. x lies in
// LDS, 64 KiB of it at a time: fragments of x from the cache would be as many loads again
// as those of W (40 us where this takes 34). Measured at 16 tokens, 32,000 words of 2,048
// (131 MB): 28 us, 4.6 TB/s, and the join 5; 131,072 words of 4,096 200 us, 5.3 TB/s.
// Where it ends: 32 tokens here and 33 in tiles take 36 and 53 us over 32,000 words of
// 2,048, 13.5 and 17.5 over 4,099 of 384, 228 and 231 over 131,072 of 4,096; in fp32 72 and
// 99, 13.6 and 19.7, 475 and 626.

// Of the calling wave's lanes, whether the lane's token has a target, and its place among those.
struct TlFew {
  unsigned long long mask;
  __device__ __forceinline__ TlFew(const int32_t* targets, int tokens) {
    const int lane = threadIdx.x & 63;
    mask = __ballot(lane < tokens && targets[lane < tokens ? lane : 0] >= 0);
  }
  __device__ __forceinline__ bool is(int t) const { return mask >> t & 1; }
  __device__ __forceinline__ int place(int t) const { return __popcll(mask & ((1ull << t) - 1)); }
  __device__ __forceinline__ int count() const { return __popcll(mask); }
};

template <typename T> struct TlThin {
  const T* x;
  const T* W;
  const int32_t* targets;
  float2* part;  // [workgroups][tokens]
  float* at;     // [tokens]
  int64_t V;
  int tokens, C;
  float scale2;
};

// Values k .. k + 7 of a row as a fragment.
__device__ __forceinline__ bf16x8 tl_values(const bf16* p) {
  return *reinterpret_cast<const bf16x8*>(p);
}
__device__ __forceinline__ f32x8 tl_values(const float* p) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
  return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

template <typename T, int NT>
__global__ __launch_bounds__(64 * kThinWaves) void k_tl_thin(TlThin<T> p) {
  constexpr int kSteps = (sizeof(T) == 2 ? 8 : 4) / NT;  // of 32 values of k, in flight
  constexpr int kVec = 16 / (int)sizeof(T);
  constexpr int kRow = 65536 / (16 * NT * (int)sizeof(T));  // values of k of a token in LDS
  typedef typename AtFrag<T>::type Frag;
  __shared__ __attribute__((aligned(256))) T held[16 * NT * kRow];
  __shared__ int rows[kThinTokens];
  __shared__ float2 stats[kThinWaves][16 * NT];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4;
  const TlFew few(p.targets, p.tokens);
  const int live = few.count();
  if (live == 0) return;
  if (threadIdx.x < kThinTokens && few.is(lane)) rows[few.place(lane)] = lane;
  __syncthreads();
  int target[NT];
  float most[NT], sum[NT];
  const float factor = fabsf(p.scale2);
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int t = 16 * j + (lane & 15);
    target[j] = t < live ? p.targets[rows[t]] : -1;
    most[j] = -INFINITY;
    sum[j] = 0.0f;
  }
  // 16-byte chunks of a token's row, turned by the token: the 16 tokens of a fragment's
  // chunk lie in different banks
  const auto place = [](int t, int chunk) { return (t * (kRow / kVec) + (chunk ^ (t & 15))) * kVec; };
  const auto hold = [&](int k0) {
    const int chunks = (p.C - k0 < kRow ? p.C - k0 : kRow) / kVec;
    const uint32_t to = at_lds(held) + wave * 1024;
    for (int i = threadIdx.x; i < 16 * NT * (kRow / kVec); i += 64 * kThinWaves) {
      const int t = i / (kRow / kVec), c = i % (kRow / kVec) ^ (t & 15);
      if (t < live && c < chunks)
        at_load_lds<16>(p.x + (int64_t)rows[t] * p.C + k0 + c * kVec,
                        to + (i - threadIdx.x) * 16);
    }
  };
  const auto value = [&](int j, int k) -> Frag {  // of token 16 j + l % 16, values k ..
    const int t = 16 * j + (lane & 15);
    if constexpr (sizeof(T) == 2) {
      return tl_values(held + place(t, k / kVec));
    } else {
      const f32x4 a = *reinterpret_cast<const f32x4*>(held + place(t, k / kVec));
      const f32x4 b = *reinterpret_cast<const f32x4*>(held + place(t, k / kVec + 1));
      return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    }
  };
  const auto row = [&](int64_t base) {
    const int64_t v = base + wave * 16 + (lane & 15);
    return p.W + (v < p.V ? v : p.V - 1) * p.C;
  };
  const auto load = [&](const T* w, int k, Frag (&f)[kSteps]) {
#pragma unroll
    for (int u = 0; u < kSteps; ++u) f[u] = tl_values(w + k + 32 * u + 8 * g);
  };
  hold(0);
  Frag a[2][kSteps];
  if (p.C >= 32 * kSteps) load(row((int64_t)blockIdx.x * kThinWaves * 16), 0, a[0]);
  at_arrive<0>();
  for (int64_t base = (int64_t)blockIdx.x * kThinWaves * 16; base < p.V;
       base += (int64_t)gridDim.x * kThinWaves * 16) {
    const int64_t v0 = base + wave * 16;
    const bool begun = base == (int64_t)blockIdx.x * kThinWaves * 16;
    f32x4 z[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) z[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int k0 = 0; k0 < p.C; k0 += kRow) {
      if (p.C > kRow && (k0 || !begun)) {
        __syncthreads();
        hold(k0);
        at_arrive<0>();
      }
      const T* w = row(base) + k0;
      const int n = p.C - k0 < kRow ? p.C - k0 : kRow;
      // the fragments of the next steps are on their way while these are multiplied
      const auto multiply = [&](int k, const Frag (&f)[kSteps]) {
#pragma unroll
        for (int u = 0; u < kSteps; ++u)
#pragma unroll
          for (int j = 0; j < NT; ++j) z[j] = pt_mma(f[u], value(j, k + 32 * u + 8 * g), z[j]);
      };
      constexpr int kStep = 32 * kSteps;
      const int whole = n / kStep * kStep;
      if (whole && (k0 || !begun)) load(w, 0, a[0]);
      for (int k = 0; k < whole; k += 2 * kStep) {
        if (k + kStep < whole) load(w, k + kStep, a[1]);
        multiply(k, a[0]);
        if (k + kStep >= whole) break;
        if (k + 2 * kStep < whole) load(w, k + 2 * kStep, a[0]);
        multiply(k + kStep, a[1]);
      }
      if (whole < n) {  // the rest, zeros behind it
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
          const int at = whole + 32 * u + 8 * g;
          a[0][u] = tl_values(w + (at < n ? at : 0));
        }
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
          const int at = whole + 32 * u + 8 * g;
          const Frag zero = {};
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const Frag y = value(j, at < n ? at : 0);
            z[j] = pt_mma(at < n ? a[0][u] : zero, at < n ? y : zero, z[j]);
          }
        }
      }
    }
    const int64_t first = v0 + 4 * g;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float top = -INFINITY;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (p.scale2 < 0.0f) z[j][e] = -z[j][e];
        if (first + e >= p.V) z[j][e] = -INFINITY;
        if (first + e == target[j]) p.at[16 * j + (lane & 15)] = z[j][e];
        top = fmaxf(top, z[j][e]);
      }
      top = fmaxf(most[j], top == -INFINITY ? top : top * factor);
      const float base = top == -INFINITY ? 0.0f : top;
      sum[j] *= __builtin_amdgcn_exp2f(most[j] - base);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        sum[j] += __builtin_amdgcn_exp2f(__builtin_fmaf(z[j][e], factor, -base));
      most[j] = top;
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const float top = tl_max4(most[j]), base = top == -INFINITY ? 0.0f : top;
    const float s = tl_sum4(sum[j] * __builtin_amdgcn_exp2f(most[j] - base));
    if (g == 0) stats[wave][16 * j + lane] = make_float2(top, s);
  }
  __syncthreads();
  const int t = threadIdx.x;
  if (t >= live) return;
  float top = -INFINITY, s = 0.0f;
#pragma unroll
  for (int w = 0; w < kThinWaves; ++w) top = fmaxf(top, stats[w][t].x);
  const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
  for (int w = 0; w < kThinWaves; ++w)
    s += stats[w][t].y * __builtin_amdgcn_exp2f(stats[w][t].x - base);
  p.part[(int64_t)blockIdx.x * p.tokens + t] = make_float2(top, s);
}

// One workgroup: 32 threads a token, at most 32 pairs each, all loaded at once.
__global__ __launch_bounds__(1024) void k_tl_thin_join(const float2* part, const float* at,
                                                       const int32_t* targets, float* nll,
                                                       float* lse, int tokens, int64_t V,
                                                       int blocks, float factor) {
  constexpr int kEach = kThinBlocks / 32;
  __shared__ float2 stats[32][33];
  const int t = threadIdx.x & 31, k = threadIdx.x >> 5;
  const TlFew few(targets, tokens);
  const int live = few.count();
  float2 s[kEach];
  float most = -INFINITY, sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int b = k + 32 * i;
    s[i] = t < live && b < blocks ? part[(int64_t)b * tokens + t] : make_float2(-INFINITY, 0.0f);
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) most = fmaxf(most, s[i].x);
  float base = most == -INFINITY ? 0.0f : most;
#pragma unroll
  for (int i = 0; i < kEach; ++i) sum += s[i].y * __builtin_amdgcn_exp2f(s[i].x - base);
  stats[k][t] = make_float2(most, sum);
  __syncthreads();
  if (k || t >= tokens) return;
  if (!few.is(t)) {
    nll[t] = 0.0f;
    lse[t] = 0.0f;
    return;
  }
  const int c = few.place(t);
  most = -INFINITY;
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) most = fmaxf(most, stats[i][c].x);
  base = most == -INFINITY ? 0.0f : most;
#pragma unroll
  for (int i = 0; i < 32; ++i) sum += stats[i][c].y * __builtin_amdgcn_exp2f(stats[i][c].x - base);
  const float rest = __builtin_amdgcn_logf(sum);  // log2
  lse[t] = (most + rest) * kLn2;
  // a target that the vocabulary does not hold has no logit
  nll[t] = targets[t] < V ? (rest - __builtin_fmaf(at[c], factor, -most)) * kLn2
                          : __builtin_nanf("");
}

template <typename T> struct TlGrad {
  const T* x;     // the listed rows, one after another
  const T* xT;    // transposed, [C][ldt]
  const T* W;
  const T* WT;    // the piece transposed, [C][ldv]
  const int32_t* targets;
  const int32_t* rows;
  const int64_t* live;
  const float* lse;
  const float* g_nll;
  const float* g_lse;
  T* d;           // [piece][ldt], in bf16 hi, then lo `plane` elements on
  int64_t plane, piece, ldv, ldt;
  int64_t v_first, V;  // the piece's first row of W, and all rows
  float* sums;    // products: [splits][...] fp32
  float* out;     // g_W
  int64_t tokens; // of the copies, a multiple of 256
  int64_t x_budget;  // numbers in the sums of g_x
  int C, w_most, accumulate;
  float scale, scale2;
  uint32_t tiles_m, tiles_n;
};

// A wave's results in the operands' type, to memory by way of LDS, so that rows are
// stored as whole lines (stores of the four consecutive m that a lane holds took a
// quarter of the kernel). In LDS a row is an n; its 16-byte chunks are turned by the
// row, which spreads the accesses over the banks. A wave's part of LDS is its own.
template <typename S> struct TlTurn {
  typedef typename S::type T;
  static constexpr int width = 16 * S::mt, rows = 16 * S::nt;  // of the wave
  static constexpr int vec = 16 / (int)sizeof(T), chunks = width / vec;
  static_assert(S::wm * S::wn * rows * width * (int)sizeof(T) <= S::lds, "fits the tiles' LDS");
  static __device__ __forceinline__ int at(int r, int c) {
    return r * width + ((c / vec) ^ (r & (chunks - 1))) * vec + c % vec;
  }
  static __device__ __forceinline__ T* tile(char* smem) {
    return reinterpret_cast<T*>(smem) + (threadIdx.x >> 6) * (rows * width);
  }
  static __device__ __forceinline__ void put(const PtSums<S>& x, T* tile) {
    const int lane = threadIdx.x & 63, g = lane >> 4;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int j = 0; j < S::nt; ++j)
#pragma unroll
      for (int i = 0; i < S::mt; ++i)
        at_store4(tile + at(16 * j + (lane & 15), 16 * i + 4 * g), x.d[i][j][0], x.d[i][j][1],
                  x.d[i][j][2], x.d[i][j][3]);
    __builtin_amdgcn_wave_barrier();
  }
  // Rows of m, n contiguous: a lane takes 16 bytes of a row, the 4 quarters of a wave
  // 64 of 16 rows. In bf16 by the transposing read (lane i's address is that of row
  // i / 4 and columns 4 (i % 4) .. of its quarter).
  static __device__ __forceinline__ void store(const T* tile, T* to, int64_t pitch) {
    const int lane = threadIdx.x & 63, g = lane >> 4, i = lane & 15;
#pragma unroll
    for (int b = 0; b < S::mt; ++b)
#pragma unroll
      for (int k = 0; k < rows / (4 * vec); ++k) {
        const int n = k * 4 * vec + vec * g;
        Vec16<T> v;
        if constexpr (sizeof(T) == 2) {
          const at_bf16x4 x = at_read_tr(tile + at(n + (i >> 2), 16 * b + 4 * (i & 3)));
          const at_bf16x4 y = at_read_tr(tile + at(n + 4 + (i >> 2), 16 * b + 4 * (i & 3)));
          v.v = bf16x8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
        } else {
#pragma unroll
          for (int e = 0; e < vec; ++e) v.v[e] = tile[at(n + e, 16 * b + i)];
        }
        store16(to + (16 * b + i) * pitch + n, v);
      }
  }
};

// d of a tile, rows of W (m) x tokens (n), to d[v][t], in bf16 hi and lo. (The order that
// both products would read along k, [t][v] for the gradient of x, costs more to store
// than its product gains from it: workgroups come to their stores at the same time, so
// every byte is paid.) 8,007 tokens x 16,128 rows of
// 2,048, bf16: 560 us, cores busy for 48 % of the cycles, 0.9 TB/s of d to memory in bursts.
template <typename S>
__global__ __launch_bounds__(S::threads) void k_tl_logit_grad(TlGrad<typename S::type> p) {
  typedef typename S::type T;
  typedef PtAlong<T, S::m, S::threads> A;
  typedef PtAlong<T, S::n, S::threads> B;
  __shared__ __attribute__((aligned(256))) char smem[S::lds];
  uint32_t tm, tn;
  const int64_t live = *p.live;
  if (!pt_tile(blockIdx.x, p.tiles_m, (uint32_t)((live + S::n - 1) / S::n), &tm, &tn)) return;
  const int64_t c0 = (int64_t)tm * S::m, v0 = p.v_first + c0, t0 = (int64_t)tn * S::n;
  // a tile may begin behind the vocabulary: d is whole tiles of 256
  const int64_t from = v0 < p.V ? v0 : p.V - 1;
  const A la(p.W + from * p.C, p.C, [&](int r) { return from + r < p.V ? r : p.V - 1 - from; });
  const B lb(p.x + t0 * p.C, p.C, [](int r) { return (int64_t)r; });
  PtSums<S> z;
  pt_product<true, S, A, B>(
      z, smem, (p.C + S::bk - 1) / S::bk,
      [&](int64_t j, uint32_t to) { la.start(j * S::bk, p.C, to); },
      [&](int64_t j, uint32_t to) { lb.start(j * S::bk, p.C, to); });

  const int lane = threadIdx.x & 63, g = lane >> 4, m0 = z.first_m(), n0 = z.first_n();
#pragma unroll
  for (int j = 0; j < S::nt; ++j) {
    const int64_t t = t0 + n0 + 16 * j + (lane & 15), first = v0 + m0 + 4 * g;
    float both = 0.0f, one = 0.0f, base = 0.0f;
    int target = -1;  // from the lane's rows of W on, where it is among them
    if (t < live) {
      const int64_t row = p.rows[t], place = p.targets[row] - first;
      if (place >= 0 && place < 16 * S::mt && place % 16 < 4) target = (int)place;
      one = p.g_nll[row];
      both = (p.g_lse ? one + p.g_lse[row] : one) * p.scale;
      one *= p.scale;
      base = p.lse[row] * kLog2e;
      if (p.targets[row] >= p.V) both = __builtin_nanf("");
    }
#pragma unroll
    for (int i = 0; i < S::mt; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        z.d[i][j][e] =
            both * __builtin_amdgcn_exp2f(__builtin_fmaf(z.d[i][j][e], p.scale2, -base));
    if (__ballot(target >= 0)) {
      at_rare();
#pragma unroll
      for (int i = 0; i < S::mt; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) z.d[i][j][e] -= 16 * i + e == target ? one : 0.0f;
    }
    if (v0 + S::m > p.V || t0 + S::n > live) {
      // zeros for rows of W that are not there and for tokens behind the last one
      const int64_t past = p.V - first;
      int left = t >= live || past < 0 ? 0 : past < S::m ? (int)past : S::m;
      asm volatile("" : "+v"(left)::"memory");  // not compared ahead for every j
#pragma unroll
      for (int i = 0; i < S::mt; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (16 * i + e >= left) z.d[i][j][e] = 0.0f;
    }
  }
  __syncthreads();  // the tiles have been read
  T* tile = TlTurn<S>::tile(smem);
  TlTurn<S>::put(z, tile);
  T* to = p.d + (c0 + m0) * p.ldt + t0 + n0;
  TlTurn<S>::store(tile, to, p.ldt);
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int j = 0; j < S::nt; ++j)
#pragma unroll
      for (int i = 0; i < S::mt; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) z.d[i][j][e] -= (float)(T)z.d[i][j][e];
    TlTurn<S>::put(z, tile);
    TlTurn<S>::store(tile, to + p.plane, p.ldt);
  }
}

// How many parts k is cut into: as many as the launched workgroups allow for this many tiles
// of results (how many tokens have a target is known here only), up to `most`, each of
// eight tiles of k at least.
__device__ __forceinline__ int tl_splits(int64_t tiles, int64_t steps, int64_t launched,
                                         int64_t most) {
  int64_t s = launched / ((tiles + 7) / 8 * 8);
  if (s > steps / 8) s = steps / 8;
  if (s > most) s = most;
  return s < 1 ? 1 : (int)s;
}

// The parts of g_x that `budget` fp32 numbers hold.
__device__ __forceinline__ int64_t tl_most(int64_t budget, int64_t live, int C) {
  const int64_t most = live ? budget / (live * C) : 1;
  return most < kMostSplits ? most : kMostSplits;
}

// A workgroup's tile of results and its part of the tiles of k.
struct TlPart {
  uint32_t m, n;
  int split, splits;
  int64_t begin, count;
  __device__ __forceinline__ bool take(uint32_t tiles_m, uint32_t tiles_n, int64_t steps,
                                       int64_t most) {
    const int64_t tiles = (int64_t)tiles_m * tiles_n, each = (tiles + 7) / 8 * 8;
    if (tiles == 0) return false;
    splits = tl_splits(tiles, steps, gridDim.x, most);
    split = (int)(blockIdx.x / each);
    if (split >= splits) return false;
    const int64_t length = (steps + splits - 1) / splits;
    begin = split * length;
    count = (begin + length < steps ? begin + length : steps) - begin;
    return pt_tile((uint32_t)(blockIdx.x - split * each), tiles_m, tiles_n, &m, &n);
  }
};

// A wave's results to rows of n in fp32, m contiguous: columns below `columns` of rows below
// `rows`, added to what is there with `add`.
template <typename S>
__device__ __forceinline__ void tl_store(const PtSums<S>& acc, float* to, int64_t pitch,
                                         int64_t first, int64_t rows, int64_t column,
                                         int64_t columns, bool add) {
  const int lane = threadIdx.x & 63, g = lane >> 4;
#pragma unroll
  for (int j = 0; j < S::nt; ++j) {
    const int64_t r = first + acc.first_n() + 16 * j + (lane & 15);
    if (r >= rows) continue;
#pragma unroll
    for (int i = 0; i < S::mt; ++i) {
      const int64_t c = column + acc.first_m() + 16 * i + 4 * g;
      if (c >= columns) continue;
      f32x4* at = reinterpret_cast<f32x4*>(to + r * pitch + c);
      *at = add ? acc.d[i][j] + *at : acc.d[i][j];
    }
  }
}

// Either product reaches 1,250 TFLOP/s (840 us a piece of 16,128 rows, for hi and lo) at 8,007
// tokens of 2,048 in bf16, the matrix cores busy for 59 to 60 % of the cycles.
//
// The product of g_x, sums[split][t][c] (+)= sum over the split's rows v of the piece of
// d[t, v] W[v, c], d as hi and lo in turn, and that of g_W: both sides of a launch and of its
// join count alike.
template <int TILE> __device__ __forceinline__ int64_t tl_tokens(int64_t live) {
  return (live + TILE - 1) / TILE;
}

template <typename S>
__global__ __launch_bounds__(S::threads) void k_tl_x_grad(TlGrad<typename S::type> p) {
  typedef typename S::type T;
  typedef PtAlong<T, S::m, S::threads> A;
  typedef PtAcross<T, S::n, S::threads> B;
  __shared__ __attribute__((aligned(256))) char smem[S::lds];
  const int64_t live = *p.live;
  const int64_t K = p.V - p.v_first < p.piece ? p.V - p.v_first : p.piece;
  TlPart part;
  constexpr int kPlanes = sizeof(T) == 2 ? 2 : 1;
  // parts of the first piece, which may be cut finer than a shorter last one could
  if (!part.take(p.tiles_m, (uint32_t)tl_tokens<S::n>(live), kPlanes * (p.piece / S::bk),
                 tl_most(p.x_budget, live, p.C)))
    return;
  const int64_t one = (K + S::bk - 1) / S::bk, steps = kPlanes * one;
  const int64_t count = part.begin + part.count < steps ? part.count : steps - part.begin;
  const int64_t c0 = (int64_t)part.m * S::m, t0 = (int64_t)part.n * S::n;
  const A la(p.WT + c0 * p.ldv, p.ldv, [&](int r) { return c0 + r < p.C ? r : p.C - 1 - c0; });
  const B lb(p.d + t0, p.ldt);
  PtSums<S> acc;
  pt_product<false, S, A, B>(
      acc, smem, count,
      [&](int64_t j, uint32_t to) {
        const int64_t k = part.begin + j;
        la.start((k < one ? k : k - one) * S::bk, p.piece, to);
      },
      [&](int64_t j, uint32_t to) {
        const int64_t k = part.begin + j;
        lb.start((k < one ? k : k - one) * S::bk, to, k < one ? 0 : p.plane);
      });
  tl_store(acc, p.sums + part.split * live * p.C, p.C, t0, live, c0, p.C, p.accumulate);
}

// g_W[v][c] (+)= sum over tokens of d[t, v] x[t, c], d as hi and lo in turn; with
// more than one split the parts go to sums[split][v][c].
template <typename S>
__global__ __launch_bounds__(S::threads) void k_tl_w_grad(TlGrad<typename S::type> p) {
  typedef typename S::type T;
  typedef PtAlong<T, S::m, S::threads> A;
  typedef PtAlong<T, S::n, S::threads> B;
  __shared__ __attribute__((aligned(256))) char smem[S::lds];
  const int64_t one = (*p.live + S::bk - 1) / S::bk;
  TlPart part;
  if (!part.take(p.tiles_m, p.tiles_n, sizeof(T) == 2 ? 2 * one : one, p.w_most)) return;
  const int64_t c0 = (int64_t)part.m * S::m, n0 = (int64_t)part.n * S::n;
  const A la(p.xT + c0 * p.ldt, p.ldt,
             [&](int r) { return c0 + r < p.C ? r : p.C - 1 - c0; });
  const B lb(p.d + n0 * p.ldt, p.ldt, [](int r) { return (int64_t)r; });
  PtSums<S> acc;
  pt_product<false, S, A, B>(
      acc, smem, part.count,
      [&](int64_t j, uint32_t to) {
        const int64_t k = part.begin + j;
        la.start((k < one ? k : k - one) * S::bk, p.tokens, to);
      },
      [&](int64_t j, uint32_t to) {
        const int64_t k = part.begin + j;
        lb.start((k < one ? k : k - one) * S::bk, p.tokens, to, k < one ? 0 : p.plane);
      });
  const int64_t rows = p.V - p.v_first < p.piece ? p.V - p.v_first : p.piece;
  if (part.splits > 1)
    tl_store(acc, p.sums + part.split * rows * p.C, p.C, n0, rows, c0, p.C, false);
  else
    tl_store(acc, p.out + p.v_first * p.C, p.C, n0, rows, c0, p.C, p.accumulate);
}

// How a product was cut, for its join.
struct TlCut {
  int tile_m, tile_n, bk, planes;
  int64_t launched;
};

// The splits of g_x joined and rounded, each listed row at its token's place, zeros at the
// others.
template <typename T>
__global__ __launch_bounds__(256) void k_tl_x_join(const float* sums, const int32_t* targets,
                                                   const int32_t* rows, const int64_t* live,
                                                   T* g_x, int64_t tokens, int64_t piece,
                                                   int64_t budget, int C, TlCut cut) {
  const int64_t n = *live;
  const int64_t tiles = (int64_t)((C + cut.tile_m - 1) / cut.tile_m) *
                        ((n + cut.tile_n - 1) / cut.tile_n);
  const int64_t steps = cut.planes * (piece / cut.bk);
  const int splits = n ? tl_splits(tiles, steps, cut.launched, tl_most(budget, n, C)) : 1;
  for (int64_t r = blockIdx.x; r < tokens; r += gridDim.x) {
    T* to = g_x + (int64_t)(r < n ? rows[r] : 0) * C;
    const bool absent = targets[r] < 0;
    for (int c = 4 * threadIdx.x; c < C; c += 4 * 256) {
      if (r < n) {
        f32x4 f = *reinterpret_cast<const f32x4*>(sums + r * C + c);
        for (int s = 1; s < splits; ++s)
          f += *reinterpret_cast<const f32x4*>(sums + (s * n + r) * C + c);
        at_store4(to + c, f[0], f[1], f[2], f[3]);
      }
      if (absent) at_store4(g_x + r * C + c, 0.0f, 0.0f, 0.0f, 0.0f);
    }
  }
}

// The splits of a piece of g_W (`rows` rows) joined, where there are several.
__global__ __launch_bounds__(256) void k_tl_w_join(const float* sums, const int64_t* live,
                                                   float* out, int64_t rows, int C, int64_t most,
                                                   int accumulate, TlCut cut) {
  const int64_t tiles = (int64_t)((C + cut.tile_m - 1) / cut.tile_m) *
                        ((rows + cut.tile_n - 1) / cut.tile_n);
  const int64_t steps = cut.planes * ((*live + cut.bk - 1) / cut.bk), quads = rows * C / 4;
  const int splits = tl_splits(tiles, steps, cut.launched, most);
  if (splits == 1) return;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < quads; i += (int64_t)gridDim.x * 256) {
    f32x4 f = *reinterpret_cast<const f32x4*>(sums + 4 * i);
    for (int s = 1; s < splits; ++s)
      f += *reinterpret_cast<const f32x4*>(sums + s * rows * C + 4 * i);
    if (accumulate) f += *reinterpret_cast<const f32x4*>(out + 4 * i);
    *reinterpret_cast<f32x4*>(out + 4 * i) = f;
  }
}

__global__ void k_tl_fill(float* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    p[i] = 0.0f;
}

// Workgroups of a kernel that walks on with its grid.
uint32_t blocks_of(int64_t x, int64_t each) {
  return (uint32_t)std::min<int64_t>(tiles_of(x, each), 1 << 16);
}

// Two tiles for each type. fp32 products take sixteen times as long as bf16's, so smaller
// tiles keep up with their loads.
template <typename T> struct Tiles;
template <> struct Tiles<bf16> {
  typedef PtShape<bf16, 8, 4, 2, 4> Large;  // 256 x 256, 8 waves, one workgroup a compute unit
  typedef PtShape<bf16, 4, 4, 2, 2> Small;  // 128 x 128, 4 waves, two of them
};
template <> struct Tiles<float> {
  typedef PtShape<float, 4, 4, 2, 2> Large;  // 128 x 128, 4 waves, two of them
  typedef PtShape<float, 2, 2, 2, 2> Small;  // 64 x 64, 4 waves, four of them
};

hipError_t list(const int32_t* targets, int64_t tokens, int32_t* rows, int64_t* live, float* nll,
                float* lse, hipStream_t s) {
  k_tl_list<<<(uint32_t)tiles_of(tokens, kTlListChunk), kTlListThreads, 0, s>>>(
      targets, tokens, rows, live, nll, lse);
  return hipGetLastError();
}

template <typename S>
hipError_t run_forward(TlForward<typename S::type> a, float* nll, float* lse, hipStream_t s) {
  a.tiles_m = (uint32_t)tiles_of(a.V, S::m);
  k_tl_forward<S><<<(uint32_t)up(a.tiles_m * tiles_of(a.tokens, S::n), 8), S::threads, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_tl_join<<<blocks_of(a.tokens, 16), 256, 0, s>>>(a.part, a.at, a.targets, a.rows, a.live, nll,
                                                    lse, a.tokens, a.V, a.tiles_m,
                                                    fabsf(a.scale2));
  return hipGetLastError();
}

template <typename T>
hipError_t forward_thin(const T* x, const T* W, const int32_t* targets, float* nll, float* lse,
                        int tokens, int64_t V, int C, float scale, char* ws, const Plan& p,
                        hipStream_t s) {
  const TlThin<T> a = {x, W, targets, reinterpret_cast<float2*>(ws + p.part),
                       reinterpret_cast<float*>(ws + p.at), V, tokens, C, scale * kLog2e};
  const int blocks = thin_blocks(V);
  if (tokens <= 16)
    k_tl_thin<T, 1><<<blocks, 64 * kThinWaves, 0, s>>>(a);
  else
    k_tl_thin<T, 2><<<blocks, 64 * kThinWaves, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_tl_thin_join<<<1, 1024, 0, s>>>(a.part, a.at, targets, nll, lse, tokens, V, blocks,
                                    fabsf(a.scale2));
  return hipGetLastError();
}

template <typename T>
hipError_t forward(const T* x, const T* W, const int32_t* targets, float* nll, float* lse,
                   int64_t T_, int64_t V, int C, float scale, char* ws, nt_dtype dtype,
                   hipStream_t s) {
  const Plan p = forward_plan(T_, V, C, dtype == NT_BF16);
  if (thin(T_)) return forward_thin(x, W, targets, nll, lse, (int)T_, V, C, scale, ws, p, s);
  int32_t* rows = reinterpret_cast<int32_t*>(ws + p.rows);
  int64_t* live = reinterpret_cast<int64_t*>(ws + p.live);
  for (int64_t t = 0; t < T_; t += p.tokens) {
    const int64_t n = std::min(p.tokens, T_ - t);
    hipError_t e = list(targets + t, n, rows, live, nll + t, lse + t, s);
    if (e != hipSuccess) return e;
    const TlForward<T> a = {x + t * C, W, targets + t, rows, live,
                            reinterpret_cast<float2*>(ws + p.part),
                            reinterpret_cast<float*>(ws + p.at), n, V, C, scale * kLog2e, 0};
    e = p.logits.large ? run_forward<typename Tiles<T>::Large>(a, nll + t, lse + t, s)
                       : run_forward<typename Tiles<T>::Small>(a, nll + t, lse + t, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// One of the gradient's products, m x n results.
enum Product { kLogits, kSingles, kWeights };
template <typename S, Product P>
hipError_t run_tiles(TlGrad<typename S::type> a, const Cut& cut, int64_t m, int64_t n,
                     hipStream_t s) {
  a.tiles_m = (uint32_t)tiles_of(m, S::m);
  a.tiles_n = (uint32_t)tiles_of(n, S::n);
  const uint32_t grid = (uint32_t)std::max(cut.launched, up((int64_t)a.tiles_m * a.tiles_n, 8));
  if constexpr (P == kLogits) k_tl_logit_grad<S><<<grid, S::threads, 0, s>>>(a);
  if constexpr (P == kSingles) k_tl_x_grad<S><<<grid, S::threads, 0, s>>>(a);
  if constexpr (P == kWeights) k_tl_w_grad<S><<<grid, S::threads, 0, s>>>(a);
  return hipGetLastError();
}
template <Product P, typename T>
hipError_t run_product(const TlGrad<T>& a, const Cut& cut, int64_t m, int64_t n, hipStream_t s) {
  if (cut.large) return run_tiles<typename Tiles<T>::Large, P>(a, cut, m, n, s);
  return run_tiles<typename Tiles<T>::Small, P>(a, cut, m, n, s);
}

// b: with `b_rows` rows, or none of them.
template <typename T>
hipError_t transpose(const TlTranspose<T>& a, int64_t a_rows, const TlTranspose<T>& b,
                     int64_t b_rows, hipStream_t s) {
  const int64_t rows = std::max(a_rows, b_rows);
  const dim3 grid((uint32_t)(up(rows, 256) / 64), (uint32_t)tiles_of(a.C, 64), b_rows ? 2 : 1);
  k_tl_transpose<T><<<grid, 256, 0, s>>>(a, b);
  return hipGetLastError();
}

// A pass.
template <typename T>
hipError_t backward(const Plan& p, const T* x, const T* W, const int32_t* targets, const float* lse,
                    const float* g_nll, const float* g_lse, T* g_x, float* g_W, int64_t tokens,
                    int64_t V, int C, float scale, bool accumulate, char* ws, hipStream_t s) {
  int32_t* rows = reinterpret_cast<int32_t*>(ws + p.rows);
  int64_t* live = reinterpret_cast<int64_t*>(ws + p.live);
  T* xs = reinterpret_cast<T*>(ws + p.x);
  T* xT = reinterpret_cast<T*>(ws + p.xT);
  T* WT = reinterpret_cast<T*>(ws + p.WT);
  hipError_t e = list(targets, tokens, rows, live, nullptr, nullptr, s);
  if (e != hipSuccess) return e;
  // x, and the first piece of W
  const auto piece = [&](int64_t v, int64_t n) {
    return TlTranspose<T>{W + v * C, WT, nullptr, nullptr, nullptr, n, p.ldv, C};
  };
  const int64_t first = std::min(p.piece, V);
  e = transpose(TlTranspose<T>{x, g_W ? xT : nullptr, xs, rows, live, tokens, p.ldt, C}, tokens,
                piece(0, first), g_x ? first : 0, s);
  if (e != hipSuccess) return e;
  TlGrad<T> a = {xs, xT, W, WT, targets, rows, live, lse, g_nll, g_lse,
                 reinterpret_cast<T*>(ws + p.d), p.ldt * p.piece, p.piece, p.ldv, p.ldt, 0, V,
                 nullptr, g_W, p.padded, p.x_budget, C, p.w_most, 0, scale, scale * kLog2e, 0, 0};
  float* x_sums = reinterpret_cast<float*>(ws + p.x_sums);
  float* w_sums = reinterpret_cast<float*>(ws + p.w_sums);
  const int bk = 128 / (int)sizeof(T);
  for (int64_t v = 0; v < V; v += p.piece) {
    const int64_t n = std::min(p.piece, V - v);
    a.v_first = v;
    // whole tiles of d: the products read up to the next multiple of a step of k
    e = run_product<kLogits>(a, p.logits, up(n, 256), tokens, s);
    if (e != hipSuccess) return e;
    if (g_x) {
      if (v) e = transpose(piece(v, n), n, piece(v, n), 0, s);
      if (e != hipSuccess) return e;
      a.sums = x_sums;
      a.accumulate = v > 0;
      e = run_product<kSingles>(a, p.singles, C, tokens, s);
      if (e != hipSuccess) return e;
    }
    if (g_W) {
      a.sums = w_sums;
      a.accumulate = accumulate;
      e = run_product<kWeights>(a, p.weights, C, n, s);
      if (e != hipSuccess) return e;
      if (p.w_most > 1) {
        const int t = p.weights.tile;
        const int64_t launched =
            std::max(p.weights.launched, up(tiles_of(C, t) * tiles_of(n, t), 8));
        k_tl_w_join<<<blocks_of(n * C / 4, 256), 256, 0, s>>>(
            w_sums, live, g_W + v * C, n, C, p.w_most, accumulate,
            TlCut{t, t, bk, (int)p.planes, launched});
        e = hipGetLastError();
        if (e != hipSuccess) return e;
      }
    }
  }
  if (!g_x) return hipSuccess;
  const int t = p.singles.tile;
  const int64_t launched = std::max(p.singles.launched, up(tiles_of(C, t) * tiles_of(tokens, t), 8));
  k_tl_x_join<T><<<blocks_of(tokens, 1), 256, 0, s>>>(
      x_sums, targets, rows, live, g_x, tokens, p.piece, p.x_budget, C,
      TlCut{t, t, bk, (int)p.planes, launched});
  return hipGetLastError();
}

template <typename T>
hipError_t backward(const void* x, const void* W, const int32_t* targets, const float* lse,
                    const float* g_nll, const float* g_lse, void* g_x, float* g_W, int64_t tokens,
                    int64_t V, int C, float scale, bool accumulate, void* ws, nt_dtype dtype,
                    hipStream_t s) {
  const Plan p = backward_plan(tokens, V, C, dtype == NT_BF16);
  for (int64_t t = 0; t < tokens; t += p.tokens) {
    const hipError_t e = backward<T>(
        p, static_cast<const T*>(x) + t * C, static_cast<const T*>(W), targets + t, lse + t,
        g_nll + t, g_lse ? g_lse + t : nullptr, g_x ? static_cast<T*>(g_x) + t * C : nullptr, g_W,
        std::min(p.tokens, tokens - t), V, C, scale, accumulate || t > 0, static_cast<char*>(ws), s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

size_t token_loss_ws_bytes(int64_t tokens, int64_t V, int C, nt_dtype dtype) {
  return tokens ? forward_plan(tokens, V, C, dtype == NT_BF16).total : 0;
}

size_t token_loss_backward_ws_bytes(int64_t tokens, int64_t V, int C, nt_dtype dtype) {
  return tokens ? backward_plan(tokens, V, C, dtype == NT_BF16).total : 0;
}

hipError_t launch_token_loss(const void* x, const void* W, const int32_t* targets, float* nll,
                             float* lse, int64_t tokens, int64_t V, int C, float scale,
                             nt_dtype dtype, void* ws, hipStream_t s) {
  if (tokens == 0) return hipSuccess;
  char* w = static_cast<char*>(ws);
  if (dtype == NT_BF16)
    return forward(static_cast<const bf16*>(x), static_cast<const bf16*>(W), targets, nll, lse,
                   tokens, V, C, scale, w, dtype, s);
  return forward(static_cast<const float*>(x), static_cast<const float*>(W), targets, nll, lse,
                 tokens, V, C, scale, w, dtype, s);
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
  return dtype == NT_BF16 ? backward<bf16>(x, W, targets, lse, g_nll, g_lse, g_x, g_W, tokens, V, C,
                                           scale, accumulate, ws, dtype, s)
                          : backward<float>(x, W, targets, lse, g_nll, g_lse, g_x, g_W, tokens, V,
                                            C, scale, accumulate, ws, dtype, s);
}

}  // namespace nt
