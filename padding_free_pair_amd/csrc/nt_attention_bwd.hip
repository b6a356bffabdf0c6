// Gradients of the attention of pair rows over pair columns.
//
// One wave for a query and head (its gradient and the bias's), and one for a
// key and key head, which takes the queries of its group's heads in turn; the
// lanes hold the head's dimensions, two each.
#include <math.h>

#include "nt_device.hpp"
#include "nt_internal.hpp"

namespace nt {
namespace {

constexpr int kAbThreads = 256;

__device__ __forceinline__ float ab_wave_sum(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

template <typename T> struct AbArgs {
  const int64_t *eta, *mu, *cell0;
  const int32_t *rows, *cols, *row_sample;
  int64_t T_rows, T_cols, cells;
  int B, H, K, D, causal;
  float scale;
  int64_t ld_q, ld_k, ld_v, ld_gq, ld_gk, ld_gv;
  const T *q, *k, *v, *bias, *o, *g_o;
  const float* lse;
  T *g_q, *g_k, *g_v, *g_bias;
};

template <typename T> __device__ __forceinline__ void ab_load(const T* p, int D, float* f) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int e = 0; e < 2; ++e) f[e] = lane + 64 * e < D ? to_f32(p[lane + 64 * e]) : 0.0f;
}
template <typename T> __device__ __forceinline__ void ab_store(T* p, int D, const float* f) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (lane + 64 * e < D) p[lane + 64 * e] = from_f32<T>(f[e]);
}
__device__ __forceinline__ float ab_dot(const float* a, const float* b) {
  return ab_wave_sum(a[0] * b[0] + a[1] * b[1]);
}

template <typename T> __global__ __launch_bounds__(kAbThreads) void k_attention_bwd_q(AbArgs<T> a) {
  const int lane = threadIdx.x & 63;
  for (int64_t w = (int64_t)blockIdx.x * (kAbThreads / 64) + (threadIdx.x >> 6);
       w < a.T_rows * a.H; w += (int64_t)gridDim.x * (kAbThreads / 64)) {
    const int64_t t = w / a.H;
    const int h = (int)(w - t * a.H), hk = h / (a.H / a.K);
    const int i = a.row_sample[t];
    const int64_t r = t - a.eta[i], m = a.cols[i];
    const int64_t past = a.causal ? r + 1 + m - a.rows[i] : m;
    const int64_t cell = (int64_t)h * a.cells + a.cell0[i] + r * m;
    float q[2], o[2], g[2], acc[2] = {0.0f, 0.0f};
    ab_load(a.q + t * a.ld_q + h * a.D, a.D, q);
    ab_load(a.o + w * a.D, a.D, o);
    ab_load(a.g_o + w * a.D, a.D, g);
    const float delta = ab_dot(g, o), lse = a.lse[w];
    for (int64_t c = 0; c < m; ++c) {
      float ds = 0.0f;
      if (c < past && lse != -INFINITY) {
        float k[2], v[2];
        ab_load(a.k + (a.mu[i] + c) * a.ld_k + hk * a.D, a.D, k);
        ab_load(a.v + (a.mu[i] + c) * a.ld_v + hk * a.D, a.D, v);
        float s = ab_dot(q, k) * a.scale;
        if (a.bias) s += to_f32(a.bias[cell + c]);
        const float p = expf(s - lse);
        ds = p > 0.0f ? p * (ab_dot(g, v) - delta) : p;
        acc[0] += ds * k[0];
        acc[1] += ds * k[1];
      }
      if (a.g_bias && lane == 0) a.g_bias[cell + c] = from_f32<T>(ds);
    }
    acc[0] *= a.scale;
    acc[1] *= a.scale;
    ab_store(a.g_q + t * a.ld_gq + h * a.D, a.D, acc);
  }
}

template <typename T> __global__ __launch_bounds__(kAbThreads) void k_attention_bwd_k(AbArgs<T> a) {
  for (int64_t w = (int64_t)blockIdx.x * (kAbThreads / 64) + (threadIdx.x >> 6);
       w < a.T_cols * a.K; w += (int64_t)gridDim.x * (kAbThreads / 64)) {
    const int64_t t = w / a.K;
    const int hk = (int)(w - t * a.K), G = a.H / a.K;
    const int i = find_segment(a.mu, 0, a.B, t);
    const int64_t c = t - a.mu[i], m = a.cols[i], n = a.rows[i];
    float k[2], v[2], gk[2] = {0.0f, 0.0f}, gv[2] = {0.0f, 0.0f};
    ab_load(a.k + t * a.ld_k + hk * a.D, a.D, k);
    ab_load(a.v + t * a.ld_v + hk * a.D, a.D, v);
    int64_t r0 = a.causal ? c - m + n : 0;
    if (r0 < 0) r0 = 0;
    for (int h = hk * G; h < (hk + 1) * G; ++h)
      for (int64_t r = r0; r < n; ++r) {
        const int64_t at = (a.eta[i] + r) * a.H + h;
        const float lse = a.lse[at];
        if (lse == -INFINITY) continue;
        float q[2], o[2], g[2];
        ab_load(a.q + (a.eta[i] + r) * a.ld_q + h * a.D, a.D, q);
        ab_load(a.o + at * a.D, a.D, o);
        ab_load(a.g_o + at * a.D, a.D, g);
        float s = ab_dot(q, k) * a.scale;
        if (a.bias) s += to_f32(a.bias[(int64_t)h * a.cells + a.cell0[i] + r * m + c]);
        const float p = expf(s - lse);
        const float ds = p > 0.0f ? p * (ab_dot(g, v) - ab_dot(g, o)) : p;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          gk[e] += a.scale * ds * q[e];
          gv[e] += p * g[e];
        }
      }
    ab_store(a.g_k + t * a.ld_gk + hk * a.D, a.D, gk);
    ab_store(a.g_v + t * a.ld_gv + hk * a.D, a.D, gv);
  }
}

template <typename T>
hipError_t backward(const nt_partition& p, const nt_attention& x, const void* q, const void* k,
                    const void* v, const void* bias, const void* o, const float* lse,
                    const void* g_o, const nt_attention_grads& g, hipStream_t stream) {
  AbArgs<T> a;
  a.eta = p.single_offsets;
  a.mu = p.col_offsets;
  a.cell0 = p.pair_offsets;
  a.rows = p.lengths;
  a.cols = p.col_lengths;
  a.row_sample = p.row_sample;
  a.T_rows = p.T;
  a.T_cols = p.T_cols;
  a.cells = p.cells;
  a.B = p.B;
  a.H = x.heads;
  a.K = x.kv_heads;
  a.D = x.head_dim;
  a.causal = x.causal;
  a.scale = x.scale;
  a.ld_q = x.ld_q;
  a.ld_k = x.ld_k;
  a.ld_v = x.ld_v;
  a.ld_gq = g.ld_q;
  a.ld_gk = g.ld_k;
  a.ld_gv = g.ld_v;
  a.q = (const T*)q;
  a.k = (const T*)k;
  a.v = (const T*)v;
  a.bias = (const T*)bias;
  a.o = (const T*)o;
  a.g_o = (const T*)g_o;
  a.lse = lse;
  a.g_q = (T*)g.q;
  a.g_k = (T*)g.k;
  a.g_v = (T*)g.v;
  a.g_bias = (T*)g.bias;
  auto grid = [](int64_t items) {
    const int64_t b = (items + kAbThreads / 64 - 1) / (kAbThreads / 64);
    return (unsigned)(b < (1 << 20) ? b : (1 << 20));
  };
  if (p.T) k_attention_bwd_q<T><<<grid(p.T * x.heads), kAbThreads, 0, stream>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.T_cols == 0) return e;
  k_attention_bwd_k<T><<<grid(p.T_cols * x.kv_heads), kAbThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t attention_backward_ws_bytes(const nt_partition&, const nt_attention&, nt_dtype) { return 0; }

hipError_t launch_attention_backward(const nt_partition& p, const nt_attention& a, const void* q,
                                     const void* k, const void* v, const void* bias,
                                     const void* o, const float* lse, const void* g_o,
                                     const nt_attention_grads& g, nt_dtype dtype, void*,
                                     hipStream_t stream) {
  return dtype == NT_BF16 ? backward<bf16>(p, a, q, k, v, bias, o, lse, g_o, g, stream)
                          : backward<float>(p, a, q, k, v, bias, o, lse, g_o, g, stream);
}

}  // namespace nt
