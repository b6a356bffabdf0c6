// Gradients of the attention of pair rows over pair columns, which recompute
// the probabilities from the scores and the forward's log sums.
//
// Two walks, each with its own order of sums and no atomics, so results
// repeat bit by bit. The first owns 32 virtual rows (queries of one key head,
// as in the forward) in a wave and walks over the keys: it forms S^T = K Q^T and
// dP^T = V G^T, and their dS^T is, as it stands, the fragment of
// g_q^T += K^T dS^T. It also leaves each row's base (its log sum) and delta, prepared and
// row by row for each head, to the second (where both go out in one launch a
// small kernel before it does), which owns 32 keys in a wave and
// walks over the rows of each query head of the group in turn: S = Q K^T and
// dP = G V^T give P and dS as fragments of g_v^T += G^T P and g_k^T += Q^T dS,
// and shared key heads sum in registers. The scores and dP are formed twice (7
// products instead of 5); joining the walks would need g_q summed across
// workgroups. Causal lengths 4096, 2500, 1111, 300 (16 heads over 8, D 64) 235 us, 62 %
// of the rate of a large matrix product over the 7 products: of a CU's cycles the
// matrix cores are busy for 36 %, the vector unit (exponentials, differences,
// conversions) for 43 %, LDS for 24 % without conflicts, and with two waves a SIMD the
// first two do not overlap much. Lengths 1024, 768, 384, 96 with a bias and its gradient
// (12 heads, D 32) 50 us: 60 MB fetched (the bias, 43 MB, comes from memory 1.3 times),
// 47 written, and the chain of a tile.
#include <math.h>

#include "nt_attention_tile.hpp"
#include "nt_internal.hpp"

namespace nt {
namespace {

struct AbArgs {
  const int64_t *eta, *mu, *cell0;
  const int32_t *rows, *cols;
  int64_t T, cells, slots, ld_q, ld_k, ld_v, ld_gq, ld_gk, ld_gv;
  int B, H, K, D, causal;
  float scale;
  const void *q, *k, *v, *bias, *o, *g_o;
  const float* lse;
  void *g_q, *g_k, *g_v, *g_bias;
  float *base, *share, *delta;  // [H, T]
  int *sharing;  // [units of 32 virtual rows, K]: whether one of them has a share
};

// Tiles in flight: two where that leaves room for a second workgroup on the CU.
constexpr int ab_ahead(int pair_bytes) { return 3 * pair_bytes <= 80 * 1024 ? 2 : 1; }

__device__ __forceinline__ float ab_dot(const bf16x8& a, const bf16x8& b) {
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) s += (float)a[j] * (float)b[j];
  return s;
}
__device__ __forceinline__ float ab_dot(const f32x8& a, const f32x8& b) {
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) s += a[j] * b[j];
  return s;
}

// A row's probabilities are exp(S - base) share. Its log sum is the base, with a
// share of 1, as long as half a step of it, which is the relative error of all of
// the row's probabilities, stays below 2^-14. Beyond that (all of a row's scores
// near a mask of -1e9 or of the type's lowest value, or a large offset that they
// have in common) the sum is lost in it: at the lowest value every probability
// would be 1. There the base is the row's maximum, whose differences to the scores
// are exact, and the share one over the sum, both found by a walk over the keys of
// its own, which only waves with such a row take. The search for such rows costs the
// others 0.5 us of 50 (lengths 1024 .. 96, bias) to 4 of 230 (causal 4096 .. 300).
constexpr float kAbLarge = 1024.0f;
__device__ __forceinline__ bool ab_large(float lse) {
  return fabsf(lse) >= kAbLarge && fabsf(lse) < INFINITY;
}

// The base of a row whose share is 1, in powers of two without a bias. A row that
// saw nothing gives nothing.
template <bool BIAS> __device__ __forceinline__ float ab_base(float lse) {
  const float x = lse == -INFINITY ? INFINITY : lse;
  return BIAS ? x : x * kLog2e;
}

// The maximum of a wave's 32 rows' scores (queries q, as fragments) and the sum of
// their powers, each lane over the keys of its half: of the row's first `last`, at
// most `most` of the m at k, the pieces of keys that begin at from, from +
// step, ... bias: the cells of the lane's row. The scores are formed as in the
// walks; a piece's loads are on their way together (pieces twice as long leave the
// small kernel before the joint walks fewer waves: 15 us instead of 13, causal 4096 ..
// 300). Lengths 1024, 768, 384, 96 with one row of lowest-value masks each: 65 us
// instead of 51; with nothing else 98.
template <typename T, int DP> struct AbNormalise {
  static constexpr int blocks = sizeof(T) == 2 && DP <= 64 ? 2 : 1, keys = 32 * blocks;
};
template <typename T, int DP, bool BIAS>
__device__ __forceinline__ void ab_normalise(const AbArgs& a, const typename AtFrag<T>::type* q,
                                             const T* k, const T* bias, int m, int most, int last,
                                             int from, int step, float* to_top, float* to_sum) {
  typedef typename AtFrag<T>::type Frag;
  typedef T Cells __attribute__((ext_vector_type(4)));
  typedef AbNormalise<T, DP> P;
  constexpr int KS = DP / 16;
  const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
  const float unit = a.scale * kLog2e;
  float top = -INFINITY, sum = 0.0f;
  for (int c = from; c < most; c += step) {
    Frag f[P::blocks][KS];
    Cells z[P::blocks][4];
#pragma unroll
    for (int b = 0; b < P::blocks; ++b) {
      const int row = c + 32 * b + l32;
      const T* kp = k + (int64_t)(row < m ? row : m - 1) * a.ld_k;
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        f[b][x] = Frag{};
        if (16 * x + 8 * h < a.D) f[b][x] = at_row(kp, x, h);
      }
      if (BIAS) {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int key = c + 32 * b + 8 * y + 4 * h;
          z[b][y] = Cells{};
          if (key + 4 <= m) {
            __builtin_memcpy(&z[b][y], bias + key, sizeof(Cells));
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (key + e < m) z[b][y][e] = bias[key + e];
          }
        }
      }
    }
#pragma unroll
    for (int b = 0; b < P::blocks; ++b) {
      f32x16 s = {};
#pragma unroll
      for (int x = 0; x < KS; ++x) s = at_mma(f[b][x], q[x], s);
      float now = top, v[16];
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const int key = c + 32 * b + 8 * (x / 4) + 4 * h + x % 4;
        v[x] = BIAS ? __builtin_fmaf(s[x], a.scale, to_f32((T)z[b][x / 4][x % 4])) : s[x] * unit;
        if (key >= last) v[x] = -INFINITY;
        now = fmaxf(now, v[x]);
      }
      now = at_halves_max(now);
      const float zero = now == -INFINITY ? 0.0f : now;
      sum *= __builtin_amdgcn_exp2f((top - zero) * (BIAS ? kLog2e : 1.0f));
#pragma unroll
      for (int x = 0; x < 16; ++x)
        if (v[x] != -INFINITY)
          sum += __builtin_amdgcn_exp2f(BIAS ? (v[x] - zero) * kLog2e
                                             : __builtin_fmaf(s[x], unit, -zero));
      top = now;
    }
  }
  *to_top = top;
  *to_sum = sum;
}
// A row's base and share from them (a row without a sum gives nothing).
__device__ __forceinline__ void ab_base_share(float top, float sum, float* base, float* share) {
  const bool none = sum == 0.0f;
  *base = none ? INFINITY : top;
  *share = none ? 1.0f : 1.0f / sum;
}

// g_q of 32 virtual rows a wave, and their statistics. As in the forward, QW
// waves own different rows, and KW waves the same rows and different keys.
template <typename T, int DP, int QW, int KW, int NB, bool BIAS> struct AbQ {
  static constexpr int THREADS = 64 * QW * KW, ROWS = 32 * QW, KEYS = 32 * KW * NB;
  static constexpr int TILE = KEYS * AtTile<T, DP>::pitch, kPair = 2 * TILE * (int)sizeof(T);
  static constexpr int AHEAD = BIAS ? 1 : ab_ahead(kPair), BUFS = AHEAD + 1;
  static constexpr int kTiles = BUFS * kPair, kJoin = (KW - 1) * QW * DP / 2 * 64 * 4;
  static constexpr int kBias = kTiles > kJoin ? kTiles : kJoin;  // where the bias tiles are
  static constexpr int kLds = kBias + (BIAS ? BUFS * ROWS * KEYS * (int)sizeof(T) : 0);
};
// READY: the statistics are there already.
template <typename T, int DP, int QW, int KW, int NB, bool BIAS, bool READY>
__device__ __forceinline__ void ab_queries(const AbArgs& a, char* lds_bytes, uint32_t block) {
  typedef AbQ<T, DP, QW, KW, NB, BIAS> P;
  constexpr int KS = DP / 16, DT = DP / 32, THREADS = P::THREADS;
  constexpr int ROWS = P::ROWS, KEYS = P::KEYS;
  typedef typename AtFrag<T>::type Frag;
  typedef AtLoad<T, KEYS, DP, THREADS> Load;
  constexpr int TILE = P::TILE, kPair = P::kPair, AHEAD = P::AHEAD, BUFS = P::BUFS;
  constexpr int BEHIND = (AHEAD - 1) * 2 * Load::kPieces;
  typedef AtBiasTile<T, ROWS, KEYS, THREADS> Bias;
  T* lds_bias = reinterpret_cast<T*>(lds_bytes + P::kBias);
  const T* lds = reinterpret_cast<const T*>(lds_bytes);
  const uint32_t lds_at = at_lds(lds_bytes);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l32 = lane & 31, h = lane >> 5;
  const int qw = wave / KW, kw = wave % KW;
  // as in the forward: key heads fastest, a causal sample's longest rows first
  const int hk = block % a.K;
  const int64_t slot = a.slots - 1 - block / a.K;
  const int G = a.H / a.K;
  const int i = at_sample_of(a.eta, a.B, G, ROWS, slot);
  const int64_t tile = slot - (a.eta[i] * G / ROWS + i);
  const int64_t n = a.rows[i], m = a.cols[i];
  if (tile * ROWS >= n * G) return;

  const int64_t vr = tile * ROWS + qw * 32 + l32;
  const bool live = vr < n * G;
  const int64_t r = (live ? vr : n * G - 1) / G;
  const int hq = hk * G + (int)((live ? vr : n * G - 1) % G);
  const int64_t t = a.eta[i] + r, at = t * a.H + hq;
  const int64_t seen64 = a.causal ? r + 1 + m - n : m;
  const int64_t seen = seen64 < 0 ? 0 : seen64 < m ? seen64 : m;
  int64_t c1 = m;
  if (a.causal) {
    const int64_t vlast = tile * ROWS + ROWS - 1;
    const int64_t rl = (vlast < n * G ? vlast : n * G - 1) / G;
    c1 = rl + 1 + m - n;
    c1 = c1 < 0 ? 0 : c1 < m ? c1 : m;
  }
  const int keys = (int)m, last = (int)seen;
  const int seen0 = a.causal ? __builtin_amdgcn_readfirstlane(last) : keys;

  Frag q[KS], g[KS];
  const T* qp = static_cast<const T*>(a.q) + t * a.ld_q + (int64_t)hq * a.D;
  const T* gp = static_cast<const T*>(a.g_o) + at * a.D;
  const T* op = static_cast<const T*>(a.o) + at * a.D;
  float delta = 0.0f;
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    q[s] = g[s] = Frag{};
    if (16 * s + 8 * h < a.D) {
      q[s] = at_row(qp, s, h);
      g[s] = at_row(gp, s, h);
      if (!READY) delta += ab_dot(g[s], at_row(op, s, h));
    }
  }
  const T* kp = static_cast<const T*>(a.k) + a.mu[i] * a.ld_k + (int64_t)hk * a.D;
  const T* vp = static_cast<const T*>(a.v) + a.mu[i] * a.ld_v + (int64_t)hk * a.D;
  float base, share = 1.0f;  // (a row's share enters its g_q at the end)
  if (READY) {
    base = a.base[hq * a.T + t];
    share = a.share[hq * a.T + t];
    delta = a.delta[hq * a.T + t];
  } else {
    base = ab_base<BIAS>(a.lse[at]);
    const bool large = ab_large(a.lse[at]), any = __any(large);
    if (lane == 0 && kw == 0 && live)
      a.sharing[(a.eta[i] * G / 32 + i + tile * QW + qw) * a.K + hk] = any;
    if (any) {
      at_rare();
      float top, sum;
      ab_normalise<T, DP, BIAS>(
          a, q, kp, BIAS ? static_cast<const T*>(a.bias) + hq * a.cells + a.cell0[i] + r * m : nullptr,
          keys, (int)c1, last, 0, AbNormalise<T, DP>::keys, &top, &sum);
      sum += __shfl_xor(sum, 32);
      if (large) ab_base_share(top, sum, &base, &share);
    }
    delta += __shfl_xor(delta, 32);
    if (live && h == 0 && kw == 0) {
      a.base[hq * a.T + t] = base;
      a.share[hq * a.T + t] = share;
      a.delta[hq * a.T + t] = delta;
    }
  }
  f32x16 gq[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) gq[d] = f32x16{};
  const float unit = a.scale * kLog2e;
  const Load load_k(a.ld_k), load_v(a.ld_v);
  // the bias as in the forward: loaded BUFS tiles ahead, put into LDS one ahead
  Bias biases[BUFS];
  const T* cells[Bias::kPieces];
  int cells_left = keys;
  if (BIAS) {
#pragma unroll
    for (int u = 0; u < Bias::kPieces; ++u) {
      const int64_t x = tile * ROWS + Bias::row(u) < n * G ? tile * ROWS + Bias::row(u) : n * G - 1;
      cells[u] = static_cast<const T*>(a.bias) + (hk * G + x % G) * a.cells + a.cell0[i] +
                 x / G * m + Bias::col(u);
    }
  }
  auto load_bias = [&](Bias& to_load) {
    to_load.load(cells, cells_left);
#pragma unroll
    for (int u = 0; u < Bias::kPieces; ++u) cells[u] += KEYS;
    cells_left -= KEYS;
  };
  const int mine = 32 * kw * NB;  // this wave's first key in a tile
  const int tiles = (int)((c1 + KEYS - 1) / KEYS);
  int left = keys, to = 0;  // keys from the tile to load on; its buffer
  auto start = [&]() {
    load_k.start(kp, a.ld_k, left, a.D, lds_at + to * kPair);
    load_v.start(vp, a.ld_v, left, a.D, lds_at + to * kPair + kPair / 2);
    kp += KEYS * a.ld_k;
    vp += KEYS * a.ld_v;
    left -= KEYS;
    to = to + 1 == BUFS ? 0 : to + 1;
  };
#pragma unroll
  for (int j = 0; j < AHEAD; ++j)
    if (j < tiles) start();
  if (BIAS) {
#pragma unroll
    for (int j = 0; j < BUFS; ++j)
      if (j < tiles) load_bias(biases[j]);
    if (tiles > 0) biases[0].put(lds_bias);
  }
  int c = 0;
  auto step = [&](int j, auto index) {
    constexpr int buf = decltype(index)::value;
    if (j + AHEAD - 1 < tiles) at_arrive<BEHIND>();
    else at_arrive<0>();
    if (BIAS && j + 1 < tiles)
      biases[(buf + 1) % BUFS].put(lds_bias + (buf + 1) % BUFS * ROWS * KEYS);
    if (j + AHEAD < tiles) start();
    if (BIAS && j + BUFS < tiles) load_bias(biases[buf]);
    const T* lk = lds + buf * 2 * TILE;
    const T* lv = lk + TILE;
    f32x16 s[NB], dp[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      s[b] = dp[b] = f32x16{};
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        s[b] = at_mma(at_along<DP>(lk, mine + 32 * b + l32, x, h), q[x], s[b]);
        dp[b] = at_mma(at_along<DP>(lv, mine + 32 * b + l32, x, h), g[x], dp[b]);
      }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        at_f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
        if (BIAS) {
          const auto cell = at_cells<KEYS>(lds_bias + buf * ROWS * KEYS, 32 * qw + l32,
                                           mine + 32 * b + 8 * y + 4 * h);
#pragma unroll
          for (int e = 0; e < 4; ++e) z[e] = to_f32((T)cell[e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int x = 4 * y + e;
          s[b][x] = BIAS ? (__builtin_fmaf(s[b][x], a.scale, z[e]) - base) * kLog2e
                         : __builtin_fmaf(s[b][x], unit, -base);
          s[b][x] = __builtin_amdgcn_exp2f(s[b][x]) * (dp[b][x] - delta);
        }
      }
    if (c + KEYS > seen0) {
      at_rare();
      const int end = last - c - mine - 4 * h;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int x = 0; x < 16; ++x)
          if (32 * b + 8 * (x / 4) + x % 4 >= end) s[b][x] = 0.0f;
    }
#pragma unroll
    for (int x = 0; x < 2 * NB; ++x) {
      Frag f;
      at_pack(s[x / 2], 8 * (x % 2), f);
#pragma unroll
      for (int d = 0; d < DT; ++d)
        gq[d] = at_mma(at_across<DP>(lk, mine + 16 * x, 32 * d), f, gq[d]);
    }
    c += KEYS;
  };
  at_each<BUFS>(tiles, step);
  if (KW > 1) {  // the waves of the same rows, in order
    __syncthreads();
    float* join = reinterpret_cast<float*>(lds_bytes);
    if (kw > 0) {
      float* p = join + ((kw - 1) * QW + qw) * DT * 16 * 64 + lane;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int x = 0; x < 16; ++x) p[(16 * d + x) * 64] = gq[d][x];
    }
    __syncthreads();
    if (kw > 0) return;
#pragma unroll
    for (int w = 1; w < KW; ++w) {
      const float* p = join + ((w - 1) * QW + qw) * DT * 16 * 64 + lane;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int x = 0; x < 16; ++x) gq[d][x] += p[(16 * d + x) * 64];
    }
  }
  if (!live) return;
  const float unit_q = a.scale * share;
  T* out = static_cast<T*>(a.g_q) + t * a.ld_gq + (int64_t)hq * a.D;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int y = 0; y < 4; ++y)
      if (32 * d + 8 * y + 4 * h < a.D)
        at_store4(out + 32 * d + 8 * y + 4 * h, gq[d][4 * y] * unit_q, gq[d][4 * y + 1] * unit_q,
                  gq[d][4 * y + 2] * unit_q, gq[d][4 * y + 3] * unit_q);
}

template <typename T, int DP, int QW, int KW, int NB, bool BIAS>
__global__ __launch_bounds__(64 * QW * KW, sizeof(T) == 4 && (DP > 64 || BIAS) ? 1 : 2) void k_attention_bwd_q(
    AbArgs a) {
  __shared__ __align__(16) char lds[AbQ<T, DP, QW, KW, NB, BIAS>::kLds];
  ab_queries<T, DP, QW, KW, NB, BIAS, false>(a, lds, blockIdx.x);
}

// g_k and g_v of 32 keys a wave, and the bias's gradient dS: a store covers 64
// bytes of two rows, 5 us for 21.5 million cells. (From the first kernel, whose
// lanes hold four cells each of 32 rows, 14 us; put through LDS there and stored
// as whole lines, both kernels together took 56 us against 51, since the first
// one also fetches the bias from memory.) KW waves of a
// workgroup own different keys; RW waves own the same keys and take different
// blocks of 32 rows of each tile, and their sums are joined at the end in
// order, so few keys still fill the card.
template <typename T, int DP, int KW, int RW, int NB, bool BIAS> struct AbK {
  static constexpr int THREADS = 64 * KW * RW, KEYS = 32 * KW;
  static constexpr int ROWS = 32 * RW * NB;  // of a tile: NB blocks of a wave
  static constexpr int TILE = ROWS * AtTile<T, DP>::pitch, kPair = 2 * TILE * (int)sizeof(T);
  static constexpr int AHEAD = BIAS ? 1 : ab_ahead(kPair), BUFS = AHEAD + 1;
  static constexpr int kTiles = BUFS * kPair, kJoin = (RW - 1) * KW * 2 * DP * 32 * 4;
  // the rows' bases and deltas, the shares of those that have one, then the bias tiles
  static constexpr int kStats = kTiles > kJoin ? kTiles : kJoin;
  static constexpr int kShares = kStats + BUFS * KW * RW * 2 * 32 * NB * 4;
  static constexpr int kBias = kShares + KW * RW * 32 * 4;
  static constexpr int kLds = kBias + (BIAS ? BUFS * ROWS * KEYS * (int)sizeof(T) : 0);
  static constexpr int kWaves = DP > 64 || (BIAS && (sizeof(T) == 4 || (RW == 4 && DP > 32))) ? 1 : 2;
};
template <typename T, int DP, int KW, int RW, int NB, bool BIAS>
__device__ __forceinline__ void ab_keys(const AbArgs& a, char* lds_bytes, uint32_t block) {
  typedef AbK<T, DP, KW, RW, NB, BIAS> P;
  constexpr int KS = DP / 16, DT = DP / 32, THREADS = P::THREADS, KEYS = P::KEYS, ROWS = P::ROWS;
  typedef typename AtFrag<T>::type Frag;
  typedef AtLoad<T, ROWS, DP, THREADS> Load;
  constexpr int TILE = P::TILE, kPair = P::kPair, AHEAD = P::AHEAD, BUFS = P::BUFS;
  constexpr int BEHIND = (AHEAD - 1) * (2 * Load::kPieces + NB);  // the next tile's loads
  typedef AtBiasTile<T, ROWS, KEYS, THREADS> Bias;
  // each wave's own rows: bases, then deltas
  typedef float Stats[KW * RW][2][32 * NB];
  Stats* stats = reinterpret_cast<Stats*>(lds_bytes + P::kStats);
  typedef float Shares[32];
  Shares* shares = reinterpret_cast<Shares*>(lds_bytes + P::kShares);
  T* lds_bias = reinterpret_cast<T*>(lds_bytes + P::kBias);
  const T* lds = reinterpret_cast<const T*>(lds_bytes);
  const uint32_t lds_at = at_lds(lds_bytes);
  const uint32_t stats_at = at_lds(stats);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l32 = lane & 31, h = lane >> 5;
  const int kw = wave / RW, rw = wave % RW;
  // a causal sample's first keys, which the most rows see, begin first
  const int hk = block % a.K;
  const int64_t slot = block / a.K;
  const int G = a.H / a.K;
  const int i = at_sample_of(a.mu, a.B, 1, KEYS, slot);
  const int64_t tile = slot - (a.mu[i] / KEYS + i);
  const int64_t n = a.rows[i], m = a.cols[i];
  if (tile * KEYS >= m) return;
  const int64_t k0 = tile * KEYS + kw * 32, key = k0 + l32;
  const bool live = key < m;
  const int64_t keyc = live ? key : m - 1, t = a.mu[i] + keyc;

  Frag k[KS], v[KS];
  const T* kp = static_cast<const T*>(a.k) + t * a.ld_k + (int64_t)hk * a.D;
  const T* vp = static_cast<const T*>(a.v) + t * a.ld_v + (int64_t)hk * a.D;
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    k[s] = v[s] = Frag{};
    if (16 * s + 8 * h < a.D) {
      k[s] = at_row(kp, s, h);
      v[s] = at_row(vp, s, h);
    }
  }
  f32x16 gk[DT], gv[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) gk[d] = gv[d] = f32x16{};
  const float unit = a.scale * kLog2e;
  // Whether a row of the walk has a share, known before the walk. (Found from each
  // tile's bases: causal 4096 .. 300 3 us more.)
  bool sharing = false;
  const int64_t units = a.eta[i] * G / 32 + i, unit_end = units + (n * G + 31) / 32;
  for (int64_t x = units + lane; x < unit_end; x += 64) sharing |= a.sharing[x * a.K + hk] != 0;
  sharing = __any(sharing);

  // Rows from the first that sees a key of this workgroup, for each query head
  // in turn; the cells of the bias's gradient before it are zero.
  const int64_t ahead = a.causal ? m - n : 0;  // row r sees keys up to r + ahead
  int64_t first = 0;
  if (a.causal) {
    first = tile * KEYS - ahead;
    first = first < 0 ? 0 : first < n ? first : n;
  }
  T* g_bias = static_cast<T*>(a.g_bias) + a.cell0[i];
  if (BIAS && a.g_bias && live)
    for (int g = 0; g < G; ++g)
      for (int64_t r = 2 * rw + h; r < first; r += 2 * RW)
        g_bias[(int64_t)(hk * G + g) * a.cells + r * m + key] = from_f32<T>(0.0f);
  const int rows = (int)n, from = (int)first;
  const int tiles = (int)((n - first + ROWS - 1) / ROWS) * G;

  // The loads run ahead of the products: their own head and row.
  const Load load_q(a.ld_q), load_g((int64_t)a.H * a.D);
  int load_h = hk * G, load_r = from, to = 0;
  auto start = [&]() {
    const int left = rows - load_r;
    const int64_t t0 = a.eta[i] + load_r;
    load_q.start(static_cast<const T*>(a.q) + t0 * a.ld_q + (int64_t)load_h * a.D, a.ld_q, left,
                 a.D, lds_at + to * kPair);
    load_g.start(static_cast<const T*>(a.g_o) + (t0 * a.H + load_h) * a.D, (int64_t)a.H * a.D,
                 left, a.D, lds_at + to * kPair + kPair / 2);
    const float* p = a.base + load_h * a.T + t0;
    const float* d = a.delta + load_h * a.T + t0;
    const uint32_t stats_to = stats_at + (to * KW * RW + wave) * 2 * 32 * NB * 4;
    if (NB == 1) {  // a half of the wave each
      const int x = 32 * rw + l32, y = x < left ? x : left - 1;
      at_load_lds<4>((h ? d : p) + y, stats_to);
    } else {
      const int x = 64 * rw + lane, y = x < left ? x : left - 1;
      at_load_lds<4>(p + y, stats_to);
      at_load_lds<4>(d + y, stats_to + 32 * NB * 4);
    }
    to = to + 1 == BUFS ? 0 : to + 1;
    load_r += ROWS;
    if (load_r >= rows) {
      load_r = from;
      ++load_h;
    }
  };
  // The bias as in the forward, for the tiles of rows in turn. Its gradient's
  // rows are m elements apart from a uniform base, the lane's key and its half's
  // four rows are one register's distance (T_cols < 2^23 with a bias).
  const uint32_t row_bytes = (uint32_t)(m * sizeof(T));
  const uint32_t b_off = 4 * h * row_bytes + (uint32_t)(keyc * sizeof(T));
  Bias biases[BUFS];
  int bias_h = hk * G, bias_r = from;  // of the tile whose bias is loaded next
  const int cells_left = (int)(m - tile * KEYS);
  auto load_bias = [&](Bias& to_load) {
    const T* p = static_cast<const T*>(a.bias) + (int64_t)bias_h * a.cells + a.cell0[i] +
                 bias_r * m + tile * KEYS;
    const T* cells[Bias::kPieces];
#pragma unroll
    for (int u = 0; u < Bias::kPieces; ++u) {
      const int r = Bias::row(u) < rows - bias_r ? Bias::row(u) : rows - bias_r - 1;
      cells[u] = p + r * m + Bias::col(u);
    }
    to_load.load(cells, cells_left);
    bias_r += ROWS;
    if (bias_r >= rows) {
      bias_r = from;
      ++bias_h;
    }
  };
#pragma unroll
  for (int j = 0; j < AHEAD; ++j)
    if (j < tiles) start();
  if (BIAS) {
#pragma unroll
    for (int j = 0; j < BUFS; ++j)
      if (j < tiles) load_bias(biases[j]);
    if (tiles > 0) biases[0].put(lds_bias);
  }
  int hq = hk * G, r0 = from;
  auto step = [&](int j, auto index) {
    constexpr int buf = decltype(index)::value;
    if (j + AHEAD - 1 < tiles) at_arrive<BEHIND>();
    else at_arrive<0>();
    if (BIAS && j + 1 < tiles)
      biases[(buf + 1) % BUFS].put(lds_bias + (buf + 1) % BUFS * ROWS * KEYS);
    if (j + AHEAD < tiles) start();
    if (BIAS && j + BUFS < tiles) load_bias(biases[buf]);
    const T* lq = lds + buf * 2 * TILE;
    const T* lg = lq + TILE;
    const int mine = 32 * rw * NB;  // this wave's first row in the tile
    f32x16 s[NB], dp[NB];
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      s[u] = dp[u] = f32x16{};
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        s[u] = at_mma(at_along<DP>(lq, mine + 32 * u + l32, x, h), k[x], s[u]);
        dp[u] = at_mma(at_along<DP>(lg, mine + 32 * u + l32, x, h), v[x], dp[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      Frag cell[2] = {};
      if (BIAS)
#pragma unroll
        for (int x = 0; x < 2; ++x)
          cell[x] = at_across<KEYS>(lds_bias + buf * ROWS * KEYS, mine + 32 * u + 16 * x, 32 * kw);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int w = 32 * u + 8 * y + 4 * h;
        const f32x4 z = *reinterpret_cast<const f32x4*>(&stats[buf][wave][0][w]);
        const f32x4 d = *reinterpret_cast<const f32x4*>(&stats[buf][wave][1][w]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int x = 4 * y + e;
          const float p = __builtin_amdgcn_exp2f(
              BIAS ? (__builtin_fmaf(s[u][x], a.scale, to_f32((T)cell[x / 8][x % 8])) - z[e]) * kLog2e
                   : __builtin_fmaf(s[u][x], unit, -z[e]));
          s[u][x] = p;
          dp[u][x] = p * (dp[u][x] - d[e]);
        }
      }
    }
    // rows of this tile from this wave's first on, and the first that sees its keys
    const int left = rows - r0 - mine;
    if (sharing || left < 32 * NB || (a.causal && k0 + 31 > r0 + mine + ahead)) {
      at_rare();
      if (sharing) {
#pragma unroll
        for (int u = 0; u < NB; ++u) {
          const int r = r0 + mine + 32 * u + l32;
          shares[wave][l32] = a.share[hq * a.T + a.eta[i] + (r < rows ? r : rows - 1)];
          __builtin_amdgcn_wave_barrier();  // (the wave's own rows: no other wave writes here)
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const f32x4 f = *reinterpret_cast<const f32x4*>(&shares[wave][8 * y + 4 * h]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              s[u][4 * y + e] *= f[e];
              dp[u][4 * y + e] *= f[e];
            }
          }
          __builtin_amdgcn_wave_barrier();
        }
      }
      const int past = a.causal ? (int)(key - ahead) - r0 - mine - 4 * h : 0;
      const int end = left - 4 * h;
#pragma unroll
      for (int u = 0; u < NB; ++u)
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const int w = 32 * u + 8 * (x / 4) + x % 4;
          if (w < past || w >= end) s[u][x] = dp[u][x] = 0.0f;
        }
    }
    if (BIAS && a.g_bias && live) {
      T* p = g_bias + (int64_t)hq * a.cells + (int64_t)(r0 + mine) * m;
      if (left >= 32 * NB) {
        const AtBuffer buffer(p);
#pragma unroll
        for (int u = 0; u < NB; ++u)
#pragma unroll
          for (int x = 0; x < 16; ++x)
            buffer.store<T>(from_f32<T>(dp[u][x]), b_off, (32 * u + 8 * (x / 4) + x % 4) * row_bytes);
      } else {
        const int64_t step = at_opaque(m);
#pragma unroll
        for (int u = 0; u < NB; ++u)
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const int r = 32 * u + 8 * (x / 4) + 4 * h + x % 4;
            if (r < left) p[r * step + key] = from_f32<T>(dp[u][x]);
          }
      }
    }
#pragma unroll
    for (int x = 0; x < 2 * NB; ++x) {
      Frag fp, fs;
      at_pack(s[x / 2], 8 * (x % 2), fp);
      at_pack(dp[x / 2], 8 * (x % 2), fs);
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        gv[d] = at_mma(at_across<DP>(lg, mine + 16 * x, 32 * d), fp, gv[d]);
        gk[d] = at_mma(at_across<DP>(lq, mine + 16 * x, 32 * d), fs, gk[d]);
      }
    }
    r0 += ROWS;
    if (r0 >= rows) {
      r0 = from;
      ++hq;
    }
  };
  at_each<BUFS>(tiles, step);
  if (RW > 1) {  // the waves of the same keys, in order
    __syncthreads();
    float* join = reinterpret_cast<float*>(lds_bytes);
    if (rw > 0) {
      float* p = join + ((rw - 1) * KW + kw) * 2 * DT * 16 * 64 + lane;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          p[(32 * d + x) * 64] = gk[d][x];
          p[(32 * d + 16 + x) * 64] = gv[d][x];
        }
    }
    __syncthreads();
    if (rw > 0) return;
#pragma unroll
    for (int w = 1; w < RW; ++w) {
      const float* p = join + ((w - 1) * KW + kw) * 2 * DT * 16 * 64 + lane;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          gk[d][x] += p[(32 * d + x) * 64];
          gv[d][x] += p[(32 * d + 16 + x) * 64];
        }
    }
  }
  if (!live) return;
  T* ok = static_cast<T*>(a.g_k) + t * a.ld_gk + (int64_t)hk * a.D;
  T* ov = static_cast<T*>(a.g_v) + t * a.ld_gv + (int64_t)hk * a.D;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int c = 32 * d + 8 * y + 4 * h;
      if (c < a.D) {
        at_store4(ok + c, gk[d][4 * y] * a.scale, gk[d][4 * y + 1] * a.scale,
                  gk[d][4 * y + 2] * a.scale, gk[d][4 * y + 3] * a.scale);
        at_store4(ov + c, gv[d][4 * y], gv[d][4 * y + 1], gv[d][4 * y + 2], gv[d][4 * y + 3]);
      }
    }
}

template <typename T, int DP, int KW, int RW, int NB, bool BIAS>
__global__ __launch_bounds__(64 * KW * RW, (AbK<T, DP, KW, RW, NB, BIAS>::kWaves)) void k_attention_bwd_k(
    AbArgs a) {
  __shared__ __align__(16) char lds[AbK<T, DP, KW, RW, NB, BIAS>::kLds];
  ab_keys<T, DP, KW, RW, NB, BIAS>(a, lds, blockIdx.x);
}

// Both walks in one launch, the keys' (the longer ones) first, behind a kernel
// that prepares the rows' statistics.
template <typename T, int DP, bool BIAS>
__global__ __launch_bounds__(256, (AbK<T, DP, 2, 2, 1, BIAS>::kWaves)) void k_attention_bwd_both(
    AbArgs a, uint32_t key_blocks) {
  constexpr int kQ = AbQ<T, DP, 2, 2, 1, BIAS>::kLds, kK = AbK<T, DP, 2, 2, 1, BIAS>::kLds;
  __shared__ __align__(16) char lds[kQ > kK ? kQ : kK];
  if (blockIdx.x < key_blocks) ab_keys<T, DP, 2, 2, 1, BIAS>(a, lds, blockIdx.x);
  else ab_queries<T, DP, 2, 2, 1, BIAS, true>(a, lds, blockIdx.x - key_blocks);
}

// The statistics of rows whose log sum is large, of 128 virtual rows, and which 32 of
// them hold one: the four waves look at 32 each, then share the keys of those that do.
template <typename T, int DP, bool BIAS>
__device__ __forceinline__ void ab_large_rows(const AbArgs& a, uint32_t block) {
  constexpr int KS = DP / 16, ROWS = 128, KEYS = AbNormalise<T, DP>::keys;
  __shared__ float tops[4][32], sums[4][32];
  __shared__ int some[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l32 = lane & 31, h = lane >> 5;
  const int hk = block % a.K, G = a.H / a.K;
  const int64_t slot = block / a.K;
  const int i = at_sample_of(a.eta, a.B, G, ROWS, slot);
  const int64_t tile = (slot - (a.eta[i] * G / ROWS + i)) * ROWS;
  const int64_t n = a.rows[i], m = a.cols[i], end = n * G;
  if (tile >= end) return;
  {
    const int64_t vr = tile + 32 * wave + l32;
    const bool any = __any(vr < end && ab_large(a.lse[(a.eta[i] + vr / G) * a.H + hk * G + vr % G]));
    if (lane == 0) {
      some[wave] = any;
      if (vr < end) a.sharing[(a.eta[i] * G / 32 + i + vr / 32) * a.K + hk] = any;
    }
  }
  __syncthreads();
  for (int w = 0; w < 4; ++w) {
    if (!some[w]) continue;
    const int64_t first = tile + 32 * w;
    const bool live = first + l32 < end;
    const int64_t vr = live ? first + l32 : end - 1, r = vr / G, t = a.eta[i] + r;
    const int hq = hk * G + (int)(vr % G);
    // the keys of this row, and of the last of the 32
    const int64_t last_r = (first + 31 < end ? first + 31 : end - 1) / G;
    int64_t seen = a.causal ? r + 1 + m - n : m, most = a.causal ? last_r + 1 + m - n : m;
    seen = seen < 0 ? 0 : seen < m ? seen : m;
    most = most < 0 ? 0 : most < m ? most : m;
    typename AtFrag<T>::type q[KS];
    const T* qp = static_cast<const T*>(a.q) + t * a.ld_q + (int64_t)hq * a.D;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      q[s] = typename AtFrag<T>::type{};
      if (16 * s + 8 * h < a.D) q[s] = at_row(qp, s, h);
    }
    float top, sum;
    ab_normalise<T, DP, BIAS>(
        a, q, static_cast<const T*>(a.k) + a.mu[i] * a.ld_k + (int64_t)hk * a.D,
        BIAS ? static_cast<const T*>(a.bias) + hq * a.cells + a.cell0[i] + r * m : nullptr, (int)m,
        (int)most, (int)seen, wave * KEYS, 4 * KEYS, &top, &sum);
    sum += __shfl_xor(sum, 32);
    if (h == 0) {
      tops[wave][l32] = top;
      sums[wave][l32] = sum;
    }
    __syncthreads();
    if (wave == 0 && h == 0 && live && ab_large(a.lse[t * a.H + hq])) {  // in the waves' order
      for (int x = 1; x < 4; ++x) top = fmaxf(top, tops[x][l32]);
      const float zero = top == -INFINITY ? 0.0f : top;
      sum = 0.0f;
      for (int x = 0; x < 4; ++x)
        sum += sums[x][l32] * __builtin_amdgcn_exp2f((tops[x][l32] - zero) * (BIAS ? kLog2e : 1.0f));
      float base, share;
      ab_base_share(top, sum, &base, &share);
      a.base[hq * a.T + t] = base;
      a.share[hq * a.T + t] = share;
    }
    __syncthreads();
  }
}

// The base, share and delta = o . g_o of every row and head: 8 dimensions a lane,
// the next power of two of D / 8 lanes a group; behind those workgroups, ones that
// look for rows with a large log sum, and write their base and share and where
// they are.
template <typename T, int DP, bool BIAS>
__global__ __launch_bounds__(256) void k_attention_bwd_rows(AbArgs a, int lanes, uint32_t blocks) {
  if (blockIdx.x >= blocks) return ab_large_rows<T, DP, BIAS>(a, blockIdx.x - blocks);
  // a head's rows one after another: the statistics are written as whole lines
  // (T H < 2^29: a grid of 32-row tiles fits)
  const uint32_t per = 256 / lanes, rows = (uint32_t)a.T;
  const uint32_t to = blockIdx.x * per + threadIdx.x / lanes;  // head T + t
  const int e0 = threadIdx.x % lanes * 8;
  const bool live = to < rows * a.H;
  const int64_t at = live ? (int64_t)(to % rows) * a.H + to / rows : 0;
  float delta = 0.0f;
  if (live && e0 < a.D)
    delta = ab_dot(at_row(static_cast<const T*>(a.g_o) + at * a.D + e0, 0, 0),
                   at_row(static_cast<const T*>(a.o) + at * a.D + e0, 0, 0));
  for (int x = 1; x < lanes; x <<= 1) delta += __shfl_xor(delta, x);
  if (!live || e0) return;
  a.delta[to] = delta;
  const float lse = a.lse[at];
  if (ab_large(lse)) return;
  a.base[to] = ab_base<BIAS>(lse);
  a.share[to] = 1.0f;
}

template <typename T, int DP, int QW, int KW, int NB, bool BIAS>
hipError_t run_q(const nt_partition& p, AbArgs x, hipStream_t stream) {
  x.slots = at_slots(p.T, p.B, x.H / x.K, 32 * QW);
  k_attention_bwd_q<T, DP, QW, KW, NB, BIAS>
      <<<(unsigned)(x.slots * x.K), 64 * QW * KW, 0, stream>>>(x);
  return hipGetLastError();
}
template <typename T, int DP, int KW, int RW, int NB, bool BIAS>
hipError_t run_k(const nt_partition& p, AbArgs x, hipStream_t stream) {
  x.slots = at_slots(p.T_cols, p.B, 1, 32 * KW);
  k_attention_bwd_k<T, DP, KW, RW, NB, BIAS>
      <<<(unsigned)(x.slots * x.K), 64 * KW * RW, 0, stream>>>(x);
  return hipGetLastError();
}

// Waves share a tile of 128 rows (keys) where that makes eight workgroups a CU,
// and two of them each 64 otherwise; fewer than one and a half workgroups of 64
// keys a CU are split once more (bf16). Four waves against two sharing, uniform
// 8 x 2,048 (D 64, 16 heads, 2,048 workgroups of 128): queries 271 us against
// 291, keys 381 against 476; causal lengths 4096 .. 300 (D 64, 8 key heads, 528):
// 124 against 112, 228 against 184. Keys in one wave against two: 2,000 rows
// (D 128, 4 key heads, 128 workgroups of 64) 94 us against 143; lengths 1024 .. 96
// with a bias (D 32, 12 heads, 468): 36 against 32.
//
// Up to 3,200 workgroups of both walks go out in one launch (512 where the keys'
// registers leave one workgroup a CU): neither walk alone fills the card to its
// end. Against two launches: 1,000 + 500 + 300 with a bias (D 64, 12 heads, about 750) 56
// us against 84, (D 128, 8 heads, 500) 82 against 123; 8 x 512 (D 32, 12 heads, 1,700) 34
// against 38; 8 x 1,024 with a bias (D 32, 8 heads, 2,176) 136 against 145. Near the limit
// they are alike (causal 4096 .. 300, 3,064: 251 against 249; 8 x 1,024 of D 32, 12
// heads, 3,264: 95 against 96), beyond it one launch loses: 8 x 1,024 of D 64, 16
// heads (4,352) 186 against 181, causal 8,192 (4,128) 601 against 581. D 128: 2,000 rows,
// 8 heads (512) 110 against 117, 16 heads (1,024) 208 against 185; 8 x 512 with a bias
// (1,152) 109 against 94. Shared key heads with few keys are better split (2,000 rows,
// D 64, 16 heads over 4: 91 us, in one launch 124).
template <typename T, int DP, bool BIAS>
hipError_t run(const nt_partition& p, AbArgs x, hipStream_t stream) {
  // (two blocks of 32 at a time; a bias or fp32 fragments would not leave it the registers)
  constexpr bool can_share = sizeof(T) == 2 && !BIAS;
  typedef AbK<T, DP, 2, 2, 1, BIAS> Keys;
  if constexpr (Keys::kLds <= 86 * 1024) {  // (not wide fp32 heads, whose tiles fill LDS)
    const int64_t q_blocks = at_slots(p.T, p.B, x.H / x.K, 64) * x.K;
    const int64_t k_blocks = at_slots(p.T_cols, p.B, 1, 64) * x.K;
    if (p.T && p.T_cols && q_blocks + k_blocks <= (Keys::kWaves == 2 ? 3200 : 512) &&
        (x.H == x.K || k_blocks >= 384)) {
      int lanes = 1;
      while (lanes * 8 < x.D) lanes *= 2;
      const int64_t rows = (p.T * x.H * lanes + 255) / 256;
      const int64_t tiles = at_slots(p.T, p.B, x.H / x.K, 128) * x.K;
      k_attention_bwd_rows<T, DP, BIAS>
          <<<(unsigned)(rows + tiles), 256, 0, stream>>>(x, lanes, (uint32_t)rows);
      hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      x.slots = at_slots(p.T, p.B, x.H / x.K, 64);
      k_attention_bwd_both<T, DP, BIAS>
          <<<(unsigned)(q_blocks + k_blocks), 256, 0, stream>>>(x, (uint32_t)k_blocks);
      return hipGetLastError();
    }
  }
  if (p.T) {
    bool many = false;
    if constexpr (can_share) many = at_slots(p.T, p.B, x.H / x.K, 128) * x.K >= 2048;
    hipError_t e = hipSuccess;
    if constexpr (can_share)
      if (many) e = run_q<T, DP, 4, 1, 2, BIAS>(p, x, stream);
    if (!many) e = run_q<T, DP, 2, 2, 1, BIAS>(p, x, stream);
    if (e != hipSuccess) return e;
  }
  if (!p.T_cols) return hipSuccess;
  if constexpr (can_share)
    if (at_slots(p.T_cols, p.B, 1, 128) * x.K >= 2048) return run_k<T, DP, 4, 1, 2, BIAS>(p, x, stream);
  if constexpr (sizeof(T) == 2)  // its tiles of 128 rows fit LDS
    if (at_slots(p.T_cols, p.B, 1, 64) * x.K < 384) return run_k<T, DP, 1, 4, 1, BIAS>(p, x, stream);
  // (wide fp32 tiles leave LDS for a bias tile of 32 keys)
  if constexpr (sizeof(T) == 4 && DP > 64 && BIAS) return run_k<T, DP, 1, 2, 1, BIAS>(p, x, stream);
  else return run_k<T, DP, 2, 2, 1, BIAS>(p, x, stream);
}

template <typename T, int DP>
hipError_t run(const nt_partition& p, const AbArgs& x, hipStream_t stream) {
  return x.bias ? run<T, DP, true>(p, x, stream) : run<T, DP, false>(p, x, stream);
}

template <typename T>
hipError_t backward(const nt_partition& p, const AbArgs& x, hipStream_t stream) {
  if (x.D <= 32) return run<T, 32>(p, x, stream);
  if (x.D <= 64) return run<T, 64>(p, x, stream);
  if (x.D <= 96) return run<T, 96>(p, x, stream);
  return run<T, 128>(p, x, stream);
}

}  // namespace

size_t attention_backward_ws_bytes(const nt_partition& p, const nt_attention& a, nt_dtype) {
  const int64_t units = at_slots(p.T, p.B, a.heads / a.kv_heads, 32) * a.kv_heads;
  return (size_t)p.T * a.heads * 3 * sizeof(float) + (size_t)units * sizeof(int);
}

hipError_t launch_attention_backward(const nt_partition& p, const nt_attention& a, const void* q,
                                     const void* k, const void* v, const void* bias,
                                     const void* o, const float* lse, const void* g_o,
                                     const nt_attention_grads& g, nt_dtype dtype, void* ws,
                                     hipStream_t stream) {
  AbArgs x;
  x.eta = p.single_offsets;
  x.mu = p.col_offsets;
  x.cell0 = p.pair_offsets;
  x.rows = p.lengths;
  x.cols = p.col_lengths;
  x.T = p.T;
  x.cells = p.cells;
  x.slots = 0;
  x.ld_q = a.ld_q;
  x.ld_k = a.ld_k;
  x.ld_v = a.ld_v;
  x.ld_gq = g.ld_q;
  x.ld_gk = g.ld_k;
  x.ld_gv = g.ld_v;
  x.B = p.B;
  x.H = a.heads;
  x.K = a.kv_heads;
  x.D = a.head_dim;
  x.causal = a.causal;
  x.scale = a.scale;
  x.q = q;
  x.k = k;
  x.v = v;
  x.bias = bias;
  x.o = o;
  x.g_o = g_o;
  x.lse = lse;
  x.g_q = g.q;
  x.g_k = g.k;
  x.g_v = g.v;
  x.g_bias = g.bias;
  x.base = static_cast<float*>(ws);
  x.share = x.base + p.T * a.heads;
  x.delta = x.share + p.T * a.heads;
  x.sharing = reinterpret_cast<int*>(x.delta + p.T * a.heads);
  return dtype == NT_BF16 ? backward<bf16>(p, x, stream) : backward<float>(p, x, stream);
}

}  // namespace nt
