// Attention of each pair row's query over its sample's pair columns.
//
// One wave for a query and head: the lanes hold the head's dimensions, two
// each, and take the keys in turn with a running maximum and sum.
#include <math.h>

#include "nt_device.hpp"
#include "nt_internal.hpp"

namespace nt {
namespace {

constexpr int kAtThreads = 256;

__device__ __forceinline__ float at_wave_sum(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

template <typename T>
__global__ __launch_bounds__(kAtThreads) void k_attention(
    const int64_t* eta, const int64_t* mu, const int64_t* cell0, const int32_t* rows,
    const int32_t* cols, const int32_t* row_sample, int64_t T_rows, int64_t cells, int H, int K,
    int D, int causal, float scale, int64_t ld_q, int64_t ld_k, int64_t ld_v, const T* q,
    const T* k, const T* v, const T* bias, T* o, float* lse) {
  const int lane = threadIdx.x & 63;
  const int64_t items = T_rows * H;
  for (int64_t w = (int64_t)blockIdx.x * (kAtThreads / 64) + (threadIdx.x >> 6); w < items;
       w += (int64_t)gridDim.x * (kAtThreads / 64)) {
    const int64_t t = w / H;
    const int h = (int)(w - t * H), hk = h / (H / K);
    const int i = row_sample[t];
    const int64_t r = t - eta[i], m = cols[i];
    const int64_t seen = causal ? (r + 1 + m - rows[i] < m ? r + 1 + m - rows[i] : m) : m;
    const T* kb = k + mu[i] * ld_k + hk * D;
    const T* vb = v + mu[i] * ld_v + hk * D;
    const T* b = bias ? bias + (int64_t)h * cells + cell0[i] + r * m : nullptr;
    float x[2], acc[2] = {0.0f, 0.0f}, most = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 2; ++e) x[e] = lane + 64 * e < D ? to_f32(q[t * ld_q + h * D + lane + 64 * e]) : 0.0f;
    for (int64_t c = 0; c < seen; ++c) {
      float dot = 0.0f, y[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool in = lane + 64 * e < D;
        if (in) dot += x[e] * to_f32(kb[c * ld_k + lane + 64 * e]);
        y[e] = in ? to_f32(vb[c * ld_v + lane + 64 * e]) : 0.0f;
      }
      float s = at_wave_sum(dot) * scale;
      if (b) s += to_f32(b[c]);
      const float now = fmaxf(most, s);
      if (now == -INFINITY) continue;
      const float keep = expf(most - now), p = expf(s - now);
      most = now;
      sum = sum * keep + p;
#pragma unroll
      for (int e = 0; e < 2; ++e) acc[e] = acc[e] * keep + p * y[e];
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (lane + 64 * e < D)
        o[(t * H + h) * D + lane + 64 * e] = from_f32<T>(sum > 0.0f ? acc[e] / sum : acc[e]);
    if (lane == 0) lse[w] = most + logf(sum);
  }
}

}  // namespace

size_t attention_ws_bytes(const nt_partition&, const nt_attention&, nt_dtype) { return 0; }

hipError_t launch_attention(const nt_partition& p, const nt_attention& a, const void* q,
                            const void* k, const void* v, const void* bias, void* o, float* lse,
                            nt_dtype dtype, void*, hipStream_t stream) {
  const int64_t items = p.T * a.heads;
  if (items == 0) return hipSuccess;
  const int64_t need = (items + kAtThreads / 64 - 1) / (kAtThreads / 64);
  const unsigned grid = (unsigned)(need < (1 << 20) ? need : (1 << 20));
#define NT_LAUNCH(E)                                                                             \
  k_attention<E><<<grid, kAtThreads, 0, stream>>>(                                               \
      p.single_offsets, p.col_offsets, p.pair_offsets, p.lengths, p.col_lengths, p.row_sample,   \
      p.T, p.cells, a.heads, a.kv_heads, a.head_dim, a.causal, a.scale, a.ld_q, a.ld_k, a.ld_v,  \
      (const E*)q, (const E*)k, (const E*)v, (const E*)bias, (E*)o, lse)
  if (dtype == NT_BF16) NT_LAUNCH(bf16);
  else NT_LAUNCH(float);
#undef NT_LAUNCH
  return hipGetLastError();
}

}  // namespace nt
