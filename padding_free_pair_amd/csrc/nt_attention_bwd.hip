// Gradients of the attention of pair rows over pair columns, which recompute
// the probabilities from the scores and the forward's log sums.
//
// Two kernels, each with its own order of sums and no atomics, so results
// repeat bit by bit. The first owns 32 virtual rows (queries of one key head,
// as in the forward) in a wave and walks over the keys: it forms S^T = K Q^T and
// dP^T = V G^T, and their dS^T is, as it stands, the fragment of
// g_q^T += K^T dS^T. It also leaves each row's delta for the second, which owns
// 32 keys in a wave and walks over the virtual rows: S = Q K^T and dP = G V^T
// give P and dS as fragments of g_v^T += G^T P and g_k^T += Q^T dS; the rows of
// all query heads of the group pass by, so shared key heads sum in registers.
// The scores and dP are formed twice (7 products instead of 5); joining the
// walks would need g_q summed across workgroups.
#include <math.h>
#include <stdlib.h>

#include "nt_attention_tile.hpp"
#include "nt_internal.hpp"

namespace nt {
namespace {

constexpr int kAbTile = 64;  // rows of a tile in LDS: keys, or virtual rows

struct AbArgs {
  const int64_t *eta, *mu, *cell0;
  const int32_t *rows, *cols;
  int64_t cells, slots, ld_q, ld_k, ld_v, ld_gq, ld_gk, ld_gv;
  int B, H, K, D, causal;
  float scale;
  const void *q, *k, *v, *bias, *o, *g_o;
  const float* lse;
  void *g_q, *g_k, *g_v, *g_bias;
  float* delta;  // [T, H]
};

template <typename T>
__device__ __forceinline__ float ab_dot(const bf16x8& a, const bf16x8& b) {
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) s += (float)a[j] * (float)b[j];
  return s;
}
template <typename T> __device__ __forceinline__ float ab_dot(const f32x8& a, const f32x8& b) {
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) s += a[j] * b[j];
  return s;
}

// g_q of 32 virtual rows a wave, and their delta.
template <typename T, int DP, int WAVES, bool BIAS>
__global__ __launch_bounds__(64 * WAVES, sizeof(T) == 4 && DP > 64 ? 1 : 2) void k_attention_bwd_q(
    AbArgs a) {
  constexpr int KS = DP / 16, DT = DP / 32, THREADS = 64 * WAVES, ROWS = 32 * WAVES;
  typedef AtBoth<T, DP> L;
  constexpr int TILE = kAbTile * L::pitch;
  typedef typename AtFrag<T>::type Frag;
  __shared__ __align__(16) T lds[2][2 * TILE];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l32 = lane & 31, h = lane >> 5;
  // as in the forward: key heads fastest, a causal sample's longest rows first
  const int hk = blockIdx.x % a.K;
  const int64_t slot = a.slots - 1 - blockIdx.x / a.K;
  const int G = a.H / a.K;
  const int i = at_sample_of(a.eta, a.B, G, ROWS, slot);
  const int64_t tile = slot - (a.eta[i] * G / ROWS + i);
  const int64_t n = a.rows[i], m = a.cols[i];
  if (tile * ROWS >= n * G) return;

  const int64_t vr = tile * ROWS + wave * 32 + l32;
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
  const int keys = (int)m, end = (int)c1, last = (int)seen;
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
      delta += ab_dot<T>(g[s], at_row(op, s, h));
    }
  }
  delta += __shfl_xor(delta, 32);
  if (live && h == 0) a.delta[at] = delta;
  // a row that saw nothing gives nothing
  const float lse = a.lse[at] == -INFINITY ? INFINITY : a.lse[at];
  const T* kp = static_cast<const T*>(a.k) + a.mu[i] * a.ld_k + (int64_t)hk * a.D;
  const T* vp = static_cast<const T*>(a.v) + a.mu[i] * a.ld_v + (int64_t)hk * a.D;
  const T* bp = BIAS ? static_cast<const T*>(a.bias) + hq * a.cells + a.cell0[i] + r * m : nullptr;

  f32x16 gq[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) gq[d] = f32x16{};
  const float unit = a.scale * kLog2e, base = lse * kLog2e;
  AtStage<T, kAbTile, DP, THREADS> sk(a.ld_k), sv(a.ld_v);
  if (end > 0) {
    sk.load(kp, a.ld_k, keys, a.D);
    sv.load(vp, a.ld_v, keys, a.D);
    sk.template put<L>(lds[0]);
    sv.template put<L>(lds[0] + TILE);
  }
  __syncthreads();
  int buf = 0;
  for (int c = 0; c < end; c += kAbTile, buf ^= 1) {
    const bool more = c + kAbTile < end;
    if (more) {
      kp += kAbTile * a.ld_k;
      vp += kAbTile * a.ld_v;
      sk.load(kp, a.ld_k, keys - c - kAbTile, a.D);
      sv.load(vp, a.ld_v, keys - c - kAbTile, a.D);
    }
    const T* lk = lds[buf];
    const T* lv = lds[buf] + TILE;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      f32x16 s = f32x16{}, dp = f32x16{};
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        s = at_mma(at_along<L>(lk, 32 * b + l32, x, h), q[x], s);
        dp = at_mma(at_along<L>(lv, 32 * b + l32, x, h), g[x], dp);
      }
      if (BIAS) {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          float f[4];
          at_bias4(bp, c + 32 * b + 8 * y + 4 * h, keys, f);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[4 * y + e] = (s[4 * y + e] * a.scale + f[e] - lse) * kLog2e;
        }
      } else {
#pragma unroll
        for (int x = 0; x < 16; ++x) s[x] = s[x] * unit - base;
      }
#pragma unroll
      for (int x = 0; x < 16; ++x) s[x] = __builtin_amdgcn_exp2f(s[x]) * (dp[x] - delta);
      if (c + kAbTile > seen0) {
        at_rare();
        const int left = last - c - 4 * h;
#pragma unroll
        for (int x = 0; x < 16; ++x)
          if (32 * b + 8 * (x / 4) + x % 4 >= left) s[x] = 0.0f;
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        Frag f;
        at_pack(s, 8 * x, f);
#pragma unroll
        for (int d = 0; d < DT; ++d)
          gq[d] = at_mma(at_across<L>(lk, 32 * b + 16 * x, 32 * d), f, gq[d]);
      }
    }
    if (more) {
      sk.template put<L>(lds[buf ^ 1]);
      sv.template put<L>(lds[buf ^ 1] + TILE);
    }
    __syncthreads();
  }
  if (!live) return;
  T* out = static_cast<T*>(a.g_q) + t * a.ld_gq + (int64_t)hq * a.D;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int y = 0; y < 4; ++y)
      if (32 * d + 8 * y + 4 * h < a.D)
        at_store4(out + 32 * d + 8 * y + 4 * h, gq[d][4 * y] * a.scale, gq[d][4 * y + 1] * a.scale,
                  gq[d][4 * y + 2] * a.scale, gq[d][4 * y + 3] * a.scale);
}

// g_k and g_v of 32 keys a wave, and the bias's gradient. KW waves of a
// workgroup own different keys; RW waves own the same keys and take different
// blocks of 32 rows of each tile, and their sums are joined at the end in
// order, so few keys still fill the card.
template <typename T, int DP, int KW, int RW, bool BIAS>
__global__ __launch_bounds__(64 * KW * RW, DP > 64 ? 1 : 2) void k_attention_bwd_k(AbArgs a) {
  constexpr int KS = DP / 16, DT = DP / 32, THREADS = 64 * KW * RW, KEYS = 32 * KW;
  constexpr int NB = RW == 1 ? 2 : 1, ROWS = 32 * RW * NB;  // blocks of a wave, rows of a tile
  typedef AtBoth<T, DP> L;
  constexpr int TILE = ROWS * L::pitch;
  constexpr int kLds = 2 * 2 * TILE * (int)sizeof(T), kJoin = (RW - 1) * KW * 2 * DP * 32 * 4;
  typedef typename AtFrag<T>::type Frag;
  __shared__ __align__(16) char lds_bytes[kLds > kJoin ? kLds : kJoin];
  __shared__ __align__(16) float stats[2][2][ROWS];  // [buffer][log sum, delta]
  T* lds = reinterpret_cast<T*>(lds_bytes);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l32 = lane & 31, h = lane >> 5;
  const int kw = wave / RW, rw = wave % RW;
  // a causal sample's first keys, which the most rows see, begin first
  const int hk = blockIdx.x % a.K;
  const int64_t slot = blockIdx.x / a.K;
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

  // Rows from the first that sees a key of this workgroup, for each query head
  // in turn; the cells of the bias's gradient before it are zero.
  const int64_t ahead = a.causal ? m - n : 0;  // row r sees keys up to r + ahead
  int64_t first = 0;
  if (a.causal) {
    first = tile * KEYS - ahead;
    first = first < 0 ? 0 : first < n ? first : n;
  }
  const T* bias = static_cast<const T*>(a.bias) + a.cell0[i];
  T* g_bias = static_cast<T*>(a.g_bias) + a.cell0[i];
  if (BIAS && a.g_bias && live)
    for (int g = 0; g < G; ++g)
      for (int64_t r = 2 * rw + h; r < first; r += 2 * RW)
        g_bias[(int64_t)(hk * G + g) * a.cells + r * m + key] = from_f32<T>(0.0f);
  const int rows = (int)n, per_head = (int)((n - first + ROWS - 1) / ROWS), tiles = per_head * G;

  AtStage<T, ROWS, DP, THREADS> sq(a.ld_q), sg((int64_t)a.H * a.D);
  float row_lse = 0.0f, row_delta = 0.0f;
  // Bias of this lane's key at its rows. Rows are m elements apart from a uniform
  // base; a lane's distance from it, of its key and its half's four rows, is
  // one register (T_cols < 2^27 with a bias).
  T b_now[NB][16], b_next[NB][16];
  const uint32_t b_off = (uint32_t)((4 * h * (uint32_t)m + (uint32_t)keyc) * sizeof(T));
  int next_h = hk * G, next_r = (int)first;  // head and first row of the tile to fetch
  auto fetch = [&]() {
    const int hq = next_h, r0 = next_r;
    next_r += ROWS;
    if (next_r >= rows) {
      next_r = (int)first;
      ++next_h;
    }
    const int64_t t0 = a.eta[i] + r0;
    sq.load(static_cast<const T*>(a.q) + t0 * a.ld_q + (int64_t)hq * a.D, a.ld_q, rows - r0, a.D);
    sg.load(static_cast<const T*>(a.g_o) + (t0 * a.H + hq) * a.D, (int64_t)a.H * a.D, rows - r0, a.D);
    if (threadIdx.x < ROWS) {
      const bool in = r0 + (int)threadIdx.x < rows;
      const int64_t at = (t0 + (in ? threadIdx.x : 0)) * a.H + hq;
      const float z = a.lse[at];
      // a row that saw nothing, or is none, gives nothing
      row_lse = in && z != -INFINITY ? (BIAS ? z : z * kLog2e) : INFINITY;
      row_delta = a.delta[at];
    }
    if (BIAS) {
      const T* p = bias + (int64_t)hq * a.cells + r0 * m;
      if (r0 + ROWS <= rows) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const T* pr = p + (32 * (rw * NB + b) + 8 * (x / 4) + x % 4) * m;
            b_next[b][x] = *reinterpret_cast<const T*>(reinterpret_cast<const char*>(pr) + b_off);
          }
      } else {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const int r = 32 * (rw * NB + b) + 8 * (x / 4) + 4 * h + x % 4;
            b_next[b][x] = p[(r < rows - r0 ? r : rows - r0 - 1) * m + keyc];
          }
      }
    }
  };
  auto put = [&](int buf) {
    sq.template put<L>(lds + buf * 2 * TILE);
    sg.template put<L>(lds + buf * 2 * TILE + TILE);
    if (threadIdx.x < ROWS) {
      stats[buf][0][threadIdx.x] = row_lse;
      stats[buf][1][threadIdx.x] = row_delta;
    }
  };
  if (tiles > 0) {
    fetch();
    put(0);
  }
  __syncthreads();
  int buf = 0;
  for (int j = 0, hq = hk * G, r0 = (int)first; j < tiles; ++j, buf ^= 1) {
    const bool more = j + 1 < tiles;
    if (BIAS) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int x = 0; x < 16; ++x) b_now[b][x] = b_next[b][x];
    }
    if (more) fetch();
    const T* lq = lds + buf * 2 * TILE;
    const T* lg = lq + TILE;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int rb = 32 * (rw * NB + b);  // first row of the block in the tile
      f32x16 s = f32x16{}, dp = f32x16{};
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        s = at_mma(at_along<L>(lq, rb + l32, x, h), k[x], s);
        dp = at_mma(at_along<L>(lg, rb + l32, x, h), v[x], dp);
      }
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const f32x4 z = *reinterpret_cast<const f32x4*>(&stats[buf][0][rb + 8 * y + 4 * h]);
        const f32x4 d = *reinterpret_cast<const f32x4*>(&stats[buf][1][rb + 8 * y + 4 * h]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int x = 4 * y + e;
          const float p = __builtin_amdgcn_exp2f(
              BIAS ? (s[x] * a.scale + to_f32(b_now[b][x]) - z[e]) * kLog2e : s[x] * unit - z[e]);
          s[x] = p;
          dp[x] = p * (dp[x] - d[e]);
        }
      }
      if (a.causal && k0 + 31 > r0 + rb + ahead) {
        at_rare();
        const int past = (int)(key - ahead) - r0 - rb - 4 * h;  // rows before it do not see the key
#pragma unroll
        for (int x = 0; x < 16; ++x)
          if (8 * (x / 4) + x % 4 < past) s[x] = dp[x] = 0.0f;
      }
      if (BIAS && a.g_bias && live) {
        T* p = g_bias + (int64_t)hq * a.cells + (int64_t)(r0 + rb) * m;
        const int left = rows - r0 - rb;
        if (left >= 32) {
#pragma unroll
          for (int x = 0; x < 16; ++x)
            *reinterpret_cast<T*>(reinterpret_cast<char*>(p + (8 * (x / 4) + x % 4) * m) + b_off) =
                from_f32<T>(dp[x]);
        } else {
          at_rare();
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const int r = 8 * (x / 4) + 4 * h + x % 4;
            if (r < left) p[r * m + key] = from_f32<T>(dp[x]);
          }
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        Frag fp, fs;
        at_pack(s, 8 * x, fp);
        at_pack(dp, 8 * x, fs);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          gv[d] = at_mma(at_across<L>(lg, rb + 16 * x, 32 * d), fp, gv[d]);
          gk[d] = at_mma(at_across<L>(lq, rb + 16 * x, 32 * d), fs, gk[d]);
        }
      }
    }
    if (more) put(buf ^ 1);
    __syncthreads();
    r0 += ROWS;
    if (r0 >= rows) {
      r0 = (int)first;
      ++hq;
    }
  }
  if (RW > 1) {  // the waves of the same keys, in order
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

template <typename T, int DP, int KW, int RW, bool BIAS>
hipError_t run_k(const nt_partition& p, AbArgs x, hipStream_t stream) {
  x.slots = at_slots(p.T_cols, p.B, 1, 32 * KW);
  k_attention_bwd_k<T, DP, KW, RW, BIAS>
      <<<(unsigned)(x.slots * x.K), 64 * KW * RW, 0, stream>>>(x);
  return hipGetLastError();
}

template <typename T, int DP, bool BIAS>
hipError_t run(const nt_partition& p, AbArgs x, hipStream_t stream) {
  if (p.T) {
    x.slots = at_slots(p.T, p.B, x.H / x.K, 128);
    k_attention_bwd_q<T, DP, 4, BIAS><<<(unsigned)(x.slots * x.K), 256, 0, stream>>>(x);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!p.T_cols) return hipSuccess;
  const int64_t groups = at_slots(p.T_cols, p.B, 1, 128) * x.K;
  if (const char* ev = getenv("NT_BK")) {
    const int c = atoi(ev);
    if (c == 41) return run_k<T, DP, 4, 1, BIAS>(p, x, stream);
    if (c == 22) return run_k<T, DP, 2, 2, BIAS>(p, x, stream);
    if (c == 21) return run_k<T, DP, 2, 1, BIAS>(p, x, stream);
    if (c == 12) return run_k<T, DP, 1, 2, BIAS>(p, x, stream);
    if constexpr (sizeof(T) == 2) { if (c == 14) return run_k<bf16, DP, 1, 4, BIAS>(p, x, stream); }
  }
  if (groups >= 2048) return run_k<T, DP, 4, 1, BIAS>(p, x, stream);
  return run_k<T, DP, 2, 2, BIAS>(p, x, stream);
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
  return (size_t)p.T * a.heads * sizeof(float);
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
  x.delta = static_cast<float*>(ws);
  return dtype == NT_BF16 ? backward<bf16>(p, x, stream) : backward<float>(p, x, stream);
}

}  // namespace nt
