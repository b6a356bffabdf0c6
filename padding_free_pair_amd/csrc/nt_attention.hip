// Attention of each pair row's query over its sample's pair columns, in one
// pass over the keys with a running maximum and sum.
//
// A wave owns 32 virtual rows: the queries of one sample that read one key
// head, (row, head of the group) with the head fastest, so shared key heads
// fill the rows of a tile and are read once for their group. It forms the
// scores transposed, S^T = K Q^T: a lane then holds one row's scores for 32 of
// a tile's 64 keys, its softmax is within the lane and its partner in the
// other half, and the probabilities are, as they stand, the fragments of the
// second product O^T = V^T P^T: they never leave the registers. Four waves
// share each tile of keys and values in LDS; the next tile's loads are in
// flight meanwhile, into the other of two buffers.
#include <math.h>

#include "nt_attention_tile.hpp"
#include "nt_internal.hpp"

namespace nt {
namespace {

constexpr int kAtWaves = 4;
constexpr int kAtThreads = 64 * kAtWaves;
constexpr int kAtRows = 32 * kAtWaves;  // virtual rows of a workgroup
constexpr int kAtKeys = 64;             // keys of a tile

struct AtArgs {
  const int64_t *eta, *mu, *cell0;
  const int32_t *rows, *cols;
  int64_t cells, slots, ld_q, ld_k, ld_v;
  int64_t part_rows;  // split keys: rows of one split's partial results
  int B, H, K, D, splits;
  float scale;
  const void *q, *k, *v, *bias;
  void* o;
  float* lse;
  float *part_o, *part_ml;
};

template <typename T, int DP, bool BIAS, bool CAUSAL>
__global__ __launch_bounds__(kAtThreads, sizeof(T) == 4 && DP > 64 ? 1 : 2) void k_attention(AtArgs a) {
  constexpr int KS = DP / 16, DT = DP / 32;
  typedef AtAlong<T, DP> LK;
  typedef AtAcross<T, DP> LV;
  typedef typename AtFrag<T>::type Frag;
  __shared__ __align__(16) T lds[2][kAtKeys * (LK::pitch + LV::pitch)];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l32 = lane & 31, h = lane >> 5;
  // Key heads fastest: with 8 of them (or 4, 16 ..) an XCD, which takes every
  // eighth workgroup, stays with its own heads' keys, and all heads advance
  // together. Tiles in reverse, so that a causal sample's longest rows begin
  // first and the short ones fill the end.
  const int hk = blockIdx.x % a.K;
  const int split = blockIdx.x / a.K % a.splits;
  const int64_t slot = a.slots - 1 - blockIdx.x / a.K / a.splits;
  const int G = a.H / a.K;
  const int i = at_sample_of(a.eta, a.B, G, kAtRows, slot);
  const int64_t tile = slot - (a.eta[i] * G / kAtRows + i);
  const int64_t n = a.rows[i], m = a.cols[i];
  if (tile * kAtRows >= n * G) return;

  // this lane's row
  const int64_t vr = tile * kAtRows + wave * 32 + l32;
  const bool live = vr < n * G;
  const int64_t r = (live ? vr : n * G - 1) / G;
  const int hq = hk * G + (int)((live ? vr : n * G - 1) % G);
  const int64_t t = a.eta[i] + r;
  const int64_t seen64 = CAUSAL ? r + 1 + m - n : m;
  const int64_t seen = seen64 < 0 ? 0 : seen64 < m ? seen64 : m;
  // keys of this split, up to the last that a row of the workgroup sees
  int64_t c1 = m;
  if (CAUSAL) {
    const int64_t vlast = tile * kAtRows + kAtRows - 1;
    const int64_t rl = (vlast < n * G ? vlast : n * G - 1) / G;
    c1 = rl + 1 + m - n;
    c1 = c1 < 0 ? 0 : c1 < m ? c1 : m;
  }
  int64_t c0 = 0;
  if (a.splits > 1) {
    const int64_t per = ((c1 + a.splits - 1) / a.splits + kAtKeys - 1) / kAtKeys * kAtKeys;
    c0 = split * per < c1 ? split * per : c1;
    c1 = c0 + per < c1 ? c0 + per : c1;
  }
  const int keys = (int)m, end = (int)c1, last = (int)seen;
  // the fewest keys that a row of this wave sees: no masks below it
  const int seen0 = __builtin_amdgcn_readfirstlane(last);

  // queries as fragments; the scale's sign goes with them
  Frag q[KS];
  const T* qp = static_cast<const T*>(a.q) + t * a.ld_q + (int64_t)hq * a.D;
  // (and a scale of zero is one of zero queries)
  const float scale = a.scale == 0.0f ? 1.0f : fabsf(a.scale);
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    q[s] = Frag{};
    if (16 * s + 8 * h < a.D && a.scale != 0.0f) q[s] = at_row(qp, s, h);
    if (a.scale < 0.0f) q[s] = -q[s];
  }
  const T* kp = static_cast<const T*>(a.k) + a.mu[i] * a.ld_k + (int64_t)hk * a.D;
  const T* vp = static_cast<const T*>(a.v) + a.mu[i] * a.ld_v + (int64_t)hk * a.D;
  const T* bp = BIAS ? static_cast<const T*>(a.bias) + hq * a.cells + a.cell0[i] + r * m : nullptr;

  f32x16 o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) o[d] = f32x16{};
  float most = -INFINITY, sum = 0.0f;  // of this row; sum: this half's keys
  const float unit = BIAS ? 1.0f : scale * kLog2e;  // a score's unit in powers of two
  AtStage<T, kAtKeys, DP, kAtThreads> sk(a.ld_k), sv(a.ld_v);
  kp += c0 * a.ld_k;
  vp += c0 * a.ld_v;
  if (c0 < c1) {
    sk.load(kp, a.ld_k, keys - (int)c0, a.D);
    sv.load(vp, a.ld_v, keys - (int)c0, a.D);
    sk.template put<LK>(lds[0]);
    sv.template put<LV>(lds[0] + kAtKeys * LK::pitch);
  }
  __syncthreads();
  int buf = 0;
  for (int c = (int)c0; c < end; c += kAtKeys, buf ^= 1) {
    const bool more = c + kAtKeys < end;
    if (more) {
      kp += kAtKeys * a.ld_k;
      vp += kAtKeys * a.ld_v;
      sk.load(kp, a.ld_k, keys - c - kAtKeys, a.D);
      sv.load(vp, a.ld_v, keys - c - kAtKeys, a.D);
    }
    const T* lk = lds[buf];
    const T* lv = lds[buf] + kAtKeys * LK::pitch;
    f32x16 s[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      s[b] = f32x16{};
#pragma unroll
      for (int x = 0; x < KS; ++x) s[b] = at_mma(at_along<LK>(lk, 32 * b + l32, x, h), q[x], s[b]);
    }
    if (BIAS) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          float f[4];
          at_bias4(bp, c + 32 * b + 8 * g + 4 * h, keys, f);
#pragma unroll
          for (int e = 0; e < 4; ++e) s[b][4 * g + e] = s[b][4 * g + e] * scale + f[e];
        }
    }
    if (c + kAtKeys > (CAUSAL ? seen0 : keys)) {
      at_rare();
      const int left = last - c - 4 * h;
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int x = 0; x < 16; ++x)
          if (32 * b + 8 * (x / 4) + x % 4 >= left) s[b][x] = -INFINITY;
    }
    float top = s[0][0];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int x = 0; x < 16; ++x) top = fmaxf(top, s[b][x]);
    top = at_halves_max(top);
    if (__any(top > most)) {
      at_rare();
      const float now = fmaxf(most, top);
      const float keep = now == -INFINITY ? 1.0f
                                          : __builtin_amdgcn_exp2f((most - now) * (BIAS ? kLog2e : unit));
      most = now;
      sum *= keep;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int x = 0; x < 16; ++x) o[d][x] *= keep;
    }
    const float base = most == -INFINITY ? 0.0f : most;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const float p = BIAS ? __builtin_amdgcn_exp2f((s[b][x] - base) * kLog2e)
                             : __builtin_amdgcn_exp2f(s[b][x] * unit - base * unit);
        s[b][x] = p;
        sum += p;
      }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      Frag p;
      at_pack(s[x / 2], 8 * (x % 2), p);
#pragma unroll
      for (int d = 0; d < DT; ++d)
        o[d] = at_mma(at_across<LV>(lv, 16 * x, 32 * d), p, o[d]);
    }
    if (more) {
      sk.template put<LK>(lds[buf ^ 1]);
      sv.template put<LV>(lds[buf ^ 1] + kAtKeys * LK::pitch);
    }
    __syncthreads();
  }
  sum += __shfl_xor(sum, 32);
  if (!live) return;
  const int64_t at = t * a.H + hq;
  if (a.splits > 1) {
    float* po = a.part_o + ((int64_t)split * a.part_rows + at) * a.D;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        if (32 * d + 8 * g + 4 * h < a.D)
          at_store4(po + 32 * d + 8 * g + 4 * h, o[d][4 * g], o[d][4 * g + 1], o[d][4 * g + 2],
                    o[d][4 * g + 3]);
    if (h == 0) {
      float* ml = a.part_ml + ((int64_t)split * a.part_rows + at) * 2;
      ml[0] = BIAS ? most : most * scale;
      ml[1] = sum;
    }
    return;
  }
  const float inv = sum > 0.0f ? 1.0f / sum : 1.0f;
  T* op = static_cast<T*>(a.o) + at * a.D;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      if (32 * d + 8 * g + 4 * h < a.D)
        at_store4(op + 32 * d + 8 * g + 4 * h, o[d][4 * g] * inv, o[d][4 * g + 1] * inv,
                  o[d][4 * g + 2] * inv, o[d][4 * g + 3] * inv);
  if (h == 0) a.lse[at] = (BIAS ? most : most * scale) + logf(sum);
}

// Joins the splits of a row: one wave for each, a dimension or two a lane.
template <typename T>
__global__ __launch_bounds__(256) void k_attention_join(const float* part_o, const float* part_ml,
                                                        int splits, int64_t rows, int D, T* o,
                                                        float* lse) {
  const int lane = threadIdx.x & 63;
  for (int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); at < rows;
       at += (int64_t)gridDim.x * 4) {
    float most = -INFINITY, sum = 0.0f, acc[2] = {0.0f, 0.0f};
    for (int s = 0; s < splits; ++s) most = fmaxf(most, part_ml[(s * rows + at) * 2]);
    const float base = most == -INFINITY ? 0.0f : most;
    for (int s = 0; s < splits; ++s) {
      const float* ml = part_ml + (s * rows + at) * 2;
      const float w = expf(ml[0] - base);
      sum += w * ml[1];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (lane + 64 * e < D) acc[e] += w * part_o[(s * rows + at) * D + lane + 64 * e];
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (lane + 64 * e < D)
        o[at * D + lane + 64 * e] = from_f32<T>(sum > 0.0f ? acc[e] / sum : 0.0f);
    if (lane == 0) lse[at] = most + logf(sum);
  }
}

// In how many parts the keys are split: one, unless the rows alone leave the
// card idle and there are keys to share out.
int splits_of(const nt_partition& p, const nt_attention& a) {
  if (p.T == 0 || p.B == 0) return 1;
  const int64_t groups = at_slots(p.T, p.B, a.heads / a.kv_heads, kAtRows) * a.kv_heads;
  const int64_t keys = p.T_cols / p.B;
  if (groups >= 512 || keys < 512) return 1;
  int64_t s = 2048 / groups;
  if (s > keys / 128) s = keys / 128;
  return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}

template <typename T, int DP>
hipError_t run(const AtArgs& x, bool causal, hipStream_t stream) {
  const unsigned g = (unsigned)(x.slots * x.splits * x.K);
  if (x.bias) {
    if (causal) k_attention<T, DP, true, true><<<g, kAtThreads, 0, stream>>>(x);
    else k_attention<T, DP, true, false><<<g, kAtThreads, 0, stream>>>(x);
  } else {
    if (causal) k_attention<T, DP, false, true><<<g, kAtThreads, 0, stream>>>(x);
    else k_attention<T, DP, false, false><<<g, kAtThreads, 0, stream>>>(x);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t forward(const nt_partition& p, const nt_attention& a, AtArgs x, hipStream_t stream) {
  hipError_t e;
  if (a.head_dim <= 32) e = run<T, 32>(x, a.causal, stream);
  else if (a.head_dim <= 64) e = run<T, 64>(x, a.causal, stream);
  else if (a.head_dim <= 96) e = run<T, 96>(x, a.causal, stream);
  else e = run<T, 128>(x, a.causal, stream);
  if (e != hipSuccess || x.splits == 1) return e;
  const int64_t rows = p.T * a.heads, blocks = (rows + 3) / 4;
  k_attention_join<T><<<(unsigned)(blocks < (1 << 20) ? blocks : (1 << 20)), 256, 0, stream>>>(
      x.part_o, x.part_ml, x.splits, rows, a.head_dim, static_cast<T*>(x.o), x.lse);
  return hipGetLastError();
}

}  // namespace

// A grid holds fewer than 2^32 threads an axis.
bool attention_fits(const nt_partition& p, const nt_attention& a) {
  const int64_t most = (int64_t(1) << 32) / kAtThreads;
  // the smallest tiles that any kernel here or of the gradients takes
  return at_slots(p.T, p.B, a.heads / a.kv_heads, 64) * splits_of(p, a) * a.kv_heads < most &&
         at_slots(p.T_cols, p.B, 1, 64) * a.kv_heads < most;
}

size_t attention_ws_bytes(const nt_partition& p, const nt_attention& a, nt_dtype) {
  const int s = splits_of(p, a);
  if (s == 1) return 0;
  return (size_t)s * p.T * a.heads * (a.head_dim + 2) * sizeof(float);
}

hipError_t launch_attention(const nt_partition& p, const nt_attention& a, const void* q,
                            const void* k, const void* v, const void* bias, void* o, float* lse,
                            nt_dtype dtype, void* ws, hipStream_t stream) {
  if (p.T == 0) return hipSuccess;
  AtArgs x;
  x.eta = p.single_offsets;
  x.mu = p.col_offsets;
  x.cell0 = p.pair_offsets;
  x.rows = p.lengths;
  x.cols = p.col_lengths;
  x.cells = p.cells;
  x.slots = at_slots(p.T, p.B, a.heads / a.kv_heads, kAtRows);
  x.ld_q = a.ld_q;
  x.ld_k = a.ld_k;
  x.ld_v = a.ld_v;
  x.part_rows = p.T * a.heads;
  x.B = p.B;
  x.H = a.heads;
  x.K = a.kv_heads;
  x.D = a.head_dim;
  x.splits = splits_of(p, a);
  x.scale = a.scale;
  x.q = q;
  x.k = k;
  x.v = v;
  x.bias = bias;
  x.o = o;
  x.lse = lse;
  x.part_o = static_cast<float*>(ws);
  x.part_ml = x.part_o + (int64_t)x.splits * x.part_rows * a.head_dim;
  return dtype == NT_BF16 ? forward<bf16>(p, a, x, stream) : forward<float>(p, a, x, stream);
}

}  // namespace nt
