// Norms of queries and keys for each head with the position rotation in the
// same pass, their gradient, and the rotation's table.
//
// One group of lanes takes one token and a chunk of its heads: 8 consecutive
// dimensions a lane, the next power of two of head_dim / 8 lanes a group. The
// cosines, sines and norm weights of the lane's dimensions are read once and
// kept in registers over the heads; a head is read once (16-byte loads of
// bf16), its sum of squares is joined across the group by lane exchanges,
// and it is written once. The rotation needs each dimension's partner: in the
// interleaved layout it is in the same lane; in the half layout the lane
// reads its partners' values again, from the line that the group has just
// read. Memory bounds both directions.
#include <math.h>

#include "nt_device.hpp"
#include "nt_internal.hpp"

namespace nt {
namespace {

constexpr int kNrThreads = 256;
constexpr int kNrVec = 8;        // dimensions of a lane
constexpr int kNrHeadsAtOnce = 2;
constexpr int64_t kNrMostBlocks = int64_t(1) << 20;

// How a lane finds the partners of its dimensions.
enum { kPairsInLane = 0, kPairsInLine = 1, kPairsAnywhere = 2 };

template <typename T> struct NrSide {
  const T* x;
  const T* g;      // backward: gradient of the output, contiguous
  T* y;            // forward: output; backward: gradient of the input
  const float* w;
  const int32_t* positions;
  const int64_t* offsets;      // of the side's singles
  const int32_t* row_sample;   // null: searched in offsets
  float* part;                 // backward: partial weight gradients [blocks][D]
  int64_t tokens, ld, ld_y;
  int heads, per_chunk, chunks;
};

template <typename T> __device__ __forceinline__ void nr_load(const T* p, float* f);
template <> __device__ __forceinline__ void nr_load<bf16>(const bf16* p, float* f) {
  const bf16x8 v = *reinterpret_cast<const bf16x8*>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = (float)v[i];
}
template <> __device__ __forceinline__ void nr_load<float>(const float* p, float* f) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = a[i];
    f[4 + i] = b[i];
  }
}
template <typename T> __device__ __forceinline__ void nr_store(T* p, const float* f);
template <> __device__ __forceinline__ void nr_store<bf16>(bf16* p, const float* f) {
  bf16x8 v;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (bf16)f[i];
  *reinterpret_cast<bf16x8*>(p) = v;
}
template <> __device__ __forceinline__ void nr_store<float>(float* p, const float* f) {
  f32x4 a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = f[i];
    b[i] = f[4 + i];
  }
  *reinterpret_cast<f32x4*>(p) = a;
  *reinterpret_cast<f32x4*>(p + 4) = b;
}

__device__ __forceinline__ float nr_group_sum(float v, int lanes) {
  for (int m = 1; m < lanes; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

// The dimension that dimension e turns with (itself outside the rotated part).
__device__ __forceinline__ int nr_partner(int e, int R, bool interleaved) {
  if (e >= R) return e;
  if (interleaved) return e ^ 1;
  return e < R / 2 ? e + R / 2 : e - R / 2;
}

// cos and signed sin of the lane's dimensions at a token: out_e = y_e c_e +
// y_partner s_e. A position that the table does not hold gives NaN.
__device__ __forceinline__ void nr_angles(const float* table, int64_t at, int64_t positions, int R,
                                          bool interleaved, int e0, float* c, float* s) {
  const bool inside = at >= 0 && at < positions;
  const float* row = table + (inside ? at : 0) * R;
#pragma unroll
  for (int i = 0; i < kNrVec; ++i) {
    const int e = e0 + i;
    c[i] = 1.0f;
    s[i] = 0.0f;
    if (e < R) {
      const int j = interleaved ? e >> 1 : (e < R / 2 ? e : e - R / 2);
      const bool first = interleaved ? !(e & 1) : e < R / 2;
      c[i] = row[j];
      s[i] = first ? -row[R / 2 + j] : row[R / 2 + j];
    }
    if (!inside) c[i] = __builtin_nanf("");
  }
}

// Values of the partners of the lane's dimensions of one head.
template <typename T, int PAIRS>
__device__ __forceinline__ void nr_partners(const T* head, const float* own, int e0, int R,
                                            float* f) {
  if (PAIRS == kPairsInLane) {
#pragma unroll
    for (int i = 0; i < kNrVec; ++i) f[i] = own[i ^ 1];
  } else if (PAIRS == kPairsInLine) {
    nr_load<T>(head + nr_partner(e0, R, false), f);
  } else {
#pragma unroll
    for (int i = 0; i < kNrVec; ++i) f[i] = to_f32(head[nr_partner(e0 + i, R, false)]);
  }
}

template <typename T>
__device__ __forceinline__ int64_t nr_position(const NrSide<T>& a, int64_t t, int B) {
  if (a.positions) return a.positions[t];
  const int i = a.row_sample ? a.row_sample[t] : find_segment(a.offsets, 0, B, t);
  return t - a.offsets[i];
}

// grid: x over groups of tokens, y over the head chunks of q, then of k.
template <typename T, int PAIRS>
__global__ __launch_bounds__(kNrThreads) void k_norm_rotary(NrSide<T> q, NrSide<T> k,
                                                            const float* table, int64_t positions,
                                                            int B, int D, int R, int lanes,
                                                            float eps) {
  const bool is_q = (int)blockIdx.y < q.chunks;
  const NrSide<T>& a = is_q ? q : k;
  const int chunk = is_q ? blockIdx.y : blockIdx.y - q.chunks;
  const int groups = kNrThreads / lanes;
  const int e0 = (threadIdx.x % lanes) * kNrVec;
  const bool live = e0 < D;
  const int h0 = chunk * a.per_chunk;
  const int h1 = h0 + a.per_chunk < a.heads ? h0 + a.per_chunk : a.heads;
  float w[kNrVec], wp[kNrVec];
#pragma unroll
  for (int i = 0; i < kNrVec; ++i) {
    w[i] = a.w && live ? a.w[e0 + i] : 1.0f;
    wp[i] = a.w && live ? a.w[nr_partner(e0 + i, R, PAIRS == kPairsInLane)] : 1.0f;
  }
  // whole groups leave together
  for (int64_t t = (int64_t)blockIdx.x * groups + threadIdx.x / lanes; t < a.tokens;
       t += (int64_t)gridDim.x * groups) {
    float c[kNrVec], s[kNrVec];
#pragma unroll
    for (int i = 0; i < kNrVec; ++i) {
      c[i] = 1.0f;
      s[i] = 0.0f;
    }
    if (R && live)
      nr_angles(table, nr_position(a, t, B), positions, R, PAIRS == kPairsInLane, e0, c, s);
    const T* x = a.x + t * a.ld;
    T* y = a.y + t * a.ld_y;
    for (int h = h0; h < h1; h += kNrHeadsAtOnce) {
      float v[kNrHeadsAtOnce][kNrVec], f[kNrHeadsAtOnce][kNrVec];
      // the heads' loads first: their stores may write the same array
#pragma unroll
      for (int u = 0; u < kNrHeadsAtOnce; ++u) {
        const int hu = h + u < h1 ? h + u : h;
#pragma unroll
        for (int i = 0; i < kNrVec; ++i) v[u][i] = f[u][i] = 0.0f;
        if (live) {
          nr_load<T>(x + hu * D + e0, v[u]);
          nr_partners<T, PAIRS>(x + hu * D, v[u], e0, R, f[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < kNrHeadsAtOnce; ++u) {
        float r = 1.0f;
        if (a.w) {
          float sum = 0.0f;
#pragma unroll
          for (int i = 0; i < kNrVec; ++i) sum += v[u][i] * v[u][i];
          r = 1.0f / sqrtf(nr_group_sum(sum, lanes) / (float)D + eps);
        }
#pragma unroll
        for (int i = 0; i < kNrVec; ++i)
          v[u][i] = v[u][i] * r * w[i] * c[i] + f[u][i] * r * wp[i] * s[i];
        if (live && h + u < h1) nr_store<T>(y + (h + u) * D + e0, v[u]);
      }
    }
  }
}

// The gradient. A workgroup walks over tokens gridDim.x groups apart and
// keeps the weight gradient of its lanes' dimensions in registers; the
// workgroup's sums go to part[blockIdx.x + gridDim.x chunk].
template <typename T, int PAIRS>
__global__ __launch_bounds__(kNrThreads) void k_norm_rotary_bwd(NrSide<T> q, NrSide<T> k,
                                                                const float* table,
                                                                int64_t positions, int B, int D,
                                                                int R, int lanes, float eps) {
  __shared__ float sums[kNrThreads * kNrVec];
  const bool is_q = (int)blockIdx.y < q.chunks;
  const NrSide<T>& a = is_q ? q : k;
  const int chunk = is_q ? blockIdx.y : blockIdx.y - q.chunks;
  const int groups = kNrThreads / lanes;
  const int e0 = (threadIdx.x % lanes) * kNrVec;
  const bool live = e0 < D;
  const int h0 = chunk * a.per_chunk;
  const int h1 = h0 + a.per_chunk < a.heads ? h0 + a.per_chunk : a.heads;
  float w[kNrVec], gw[kNrVec];
#pragma unroll
  for (int i = 0; i < kNrVec; ++i) {
    w[i] = a.w && live ? a.w[e0 + i] : 1.0f;
    gw[i] = 0.0f;
  }
  for (int64_t t = (int64_t)blockIdx.x * groups + threadIdx.x / lanes; t < a.tokens;
       t += (int64_t)gridDim.x * groups) {
    float c[kNrVec], s[kNrVec];
#pragma unroll
    for (int i = 0; i < kNrVec; ++i) {
      c[i] = 1.0f;
      s[i] = 0.0f;
    }
    if (R && live)
      nr_angles(table, nr_position(a, t, B), positions, R, PAIRS == kPairsInLane, e0, c, s);
    const T* x = a.x + t * a.ld;
    const T* g = a.g + t * (int64_t)a.heads * D;
    T* y = a.y + t * a.ld_y;
    for (int h = h0; h < h1; h += kNrHeadsAtOnce) {
      float v[kNrHeadsAtOnce][kNrVec], d[kNrHeadsAtOnce][kNrVec], f[kNrHeadsAtOnce][kNrVec];
#pragma unroll
      for (int u = 0; u < kNrHeadsAtOnce; ++u) {
        const int hu = h + u < h1 ? h + u : h;
#pragma unroll
        for (int i = 0; i < kNrVec; ++i) v[u][i] = d[u][i] = f[u][i] = 0.0f;
        if (live) {
          if (a.w) nr_load<T>(x + hu * D + e0, v[u]);
          nr_load<T>(g + hu * D + e0, d[u]);
          nr_partners<T, PAIRS>(g + hu * D, d[u], e0, R, f[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < kNrHeadsAtOnce; ++u) {
        const bool mine = live && h + u < h1;
#pragma unroll
        for (int i = 0; i < kNrVec; ++i) d[u][i] = d[u][i] * c[i] - f[u][i] * s[i];
        if (a.w) {
          float sum = 0.0f, dot = 0.0f;
#pragma unroll
          for (int i = 0; i < kNrVec; ++i) sum += v[u][i] * v[u][i];
          const float r = 1.0f / sqrtf(nr_group_sum(sum, lanes) / (float)D + eps);
#pragma unroll
          for (int i = 0; i < kNrVec; ++i) {
            v[u][i] *= r;  // xhat
            if (mine) gw[i] += d[u][i] * v[u][i];
            d[u][i] *= w[i];
            dot += live ? d[u][i] * v[u][i] : 0.0f;
          }
          dot = nr_group_sum(dot, lanes) / (float)D;
#pragma unroll
          for (int i = 0; i < kNrVec; ++i) d[u][i] = r * (d[u][i] - v[u][i] * dot);
        }
        if (mine) nr_store<T>(y + (h + u) * D + e0, d[u]);
      }
    }
  }
  if (!a.w) return;
#pragma unroll
  for (int i = 0; i < kNrVec; ++i) sums[threadIdx.x * kNrVec + i] = gw[i];
  __syncthreads();
  // dimension e of group n is sums[n lanes 8 + e]: added in group order
  for (int e = threadIdx.x; e < D; e += kNrThreads) {
    float sum = 0.0f;
    for (int n = 0; n < groups; ++n) sum += sums[n * lanes * kNrVec + e];
    a.part[((int64_t)chunk * gridDim.x + blockIdx.x) * D + e] = sum;
  }
}

// Weight gradients: the partial sums added in a fixed order in fp64 (there
// are up to 4,096 of them). Block y: q or k; 16 dimensions a block.
__global__ __launch_bounds__(256) void k_norm_weight_sum(const float* part_q, const float* part_k,
                                                         int rows_q, int rows_k, float* g_q,
                                                         float* g_k, int D) {
  __shared__ double sums[256];
  const float* part = blockIdx.y ? part_k : part_q;
  const int rows = blockIdx.y ? rows_k : rows_q;
  float* g = blockIdx.y ? g_k : g_q;
  const int col = threadIdx.x & 15, e = blockIdx.x * 16 + col;
  double sum = 0.0;
  if (g && e < D)
    for (int r = threadIdx.x >> 4; r < rows; r += 16) sum += (double)part[(int64_t)r * D + e];
  sums[threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.x >= 16 || !g || e >= D) return;
  for (int r = 1; r < 16; ++r) sum += sums[r * 16 + col];
  g[e] = (float)sum;
}

__global__ __launch_bounds__(256) void k_rotary_table(float* table, int64_t positions, int R,
                                                      int scaling, double base, double factor,
                                                      double original, double beta_fast,
                                                      double beta_slow, double magnitude) {
  // blocks along y: a frequency; along x the positions
  const int half = R / 2, j = blockIdx.y;
  double f = pow(base, -2.0 * j / R);
  if (scaling == NT_ROTARY_LINEAR) f /= factor;
  if (scaling == NT_ROTARY_PARTS) {
    const double turns = original * f / (2.0 * M_PI);
    double keep = (turns - beta_slow) / (beta_fast - beta_slow);
    keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
    f = f * keep + f / factor * (1.0 - keep);
  }
  for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < positions;
       at += (int64_t)gridDim.x * 256) {
    double sn, cs;
    sincos((double)at * f, &sn, &cs);
    table[at * R + j] = (float)(cs * magnitude);
    table[at * R + half + j] = (float)(sn * magnitude);
  }
}

int group_lanes(int D) {
  int lanes = 1;
  while (lanes * kNrVec < D) lanes *= 2;
  return lanes;
}

// Heads that one group takes in turn: all of them, unless that leaves fewer
// than 2,048 workgroups (8 for each CU); then fewer, down to one.
int chunk_heads(int64_t tokens, int heads, int lanes) {
  const int64_t blocks = (tokens * lanes + kNrThreads - 1) / kNrThreads;
  int per = heads;
  while (per > 1 && blocks * ((heads + per - 1) / per) < 2048) per = (per + 1) / 2;
  return per < 1 ? 1 : per;
}

template <typename T>
NrSide<T> side(const nt_partition& p, const nt_norm_rotary& n, bool is_q, int lanes, const void* x,
               const float* w, const int32_t* positions, void* y) {
  NrSide<T> a = {};
  a.x = static_cast<const T*>(x);
  a.y = static_cast<T*>(y);
  a.w = w;
  a.positions = positions;
  const bool square = p.col_offsets == p.single_offsets;
  a.offsets = is_q ? p.single_offsets : p.col_offsets;
  a.row_sample = is_q || square ? p.row_sample : nullptr;
  a.heads = is_q ? n.heads : n.kv_heads;
  a.tokens = a.heads ? (is_q ? p.T : p.T_cols) : 0;
  const int64_t packed = (int64_t)a.heads * n.head_dim;
  a.ld = is_q ? n.ld_q : n.ld_k;
  if (!a.ld) a.ld = packed;
  a.ld_y = is_q ? n.ld_q_out : n.ld_k_out;
  if (!a.ld_y) a.ld_y = packed;
  a.per_chunk = chunk_heads(a.tokens, a.heads, lanes);
  a.chunks = a.tokens ? (a.heads + a.per_chunk - 1) / a.per_chunk : 0;
  return a;
}

int pairs_of(const nt_norm_rotary& n) {
  if (n.interleaved || n.rot_dim == 0) return kPairsInLane;
  return n.rot_dim % 16 == 0 ? kPairsInLine : kPairsAnywhere;
}

// Workgroups along x of the backward: every group of tokens, at most 256.
int64_t bwd_blocks(int64_t tokens, int lanes) {
  const int64_t b = (tokens * lanes + kNrThreads - 1) / kNrThreads;
  return b < 256 ? b : 256;
}

template <typename T>
hipError_t forward(const nt_partition& p, const nt_norm_rotary& n, const void* q, const void* k,
                   const float* w_q, const float* w_k, const float* table, const int32_t* pos_q,
                   const int32_t* pos_k, void* q_out, void* k_out, hipStream_t stream) {
  const int lanes = group_lanes(n.head_dim);
  const NrSide<T> a = side<T>(p, n, true, lanes, q, w_q, pos_q, q_out);
  const NrSide<T> b = side<T>(p, n, false, lanes, k, w_k, pos_k, k_out);
  const int64_t tokens = a.tokens > b.tokens ? a.tokens : b.tokens;
  if (tokens == 0) return hipSuccess;
  int64_t bx = (tokens * lanes + kNrThreads - 1) / kNrThreads;
  if (bx > kNrMostBlocks) bx = kNrMostBlocks;  // a grid holds fewer than 2^32 threads an axis
  const dim3 grid((unsigned)bx, a.chunks + b.chunks);
#define NT_LAUNCH(P)                                                                           \
  k_norm_rotary<T, P><<<grid, kNrThreads, 0, stream>>>(a, b, table, n.positions, p.B, n.head_dim, \
                                                       n.rot_dim, lanes, n.eps)
  switch (pairs_of(n)) {
    case kPairsInLane: NT_LAUNCH(kPairsInLane); break;
    case kPairsInLine: NT_LAUNCH(kPairsInLine); break;
    default: NT_LAUNCH(kPairsAnywhere);
  }
#undef NT_LAUNCH
  return hipGetLastError();
}

template <typename T>
hipError_t backward(const nt_partition& p, const nt_norm_rotary& n, const void* q, const void* k,
                    const void* g_q, const void* g_k, const float* w_q, const float* w_k,
                    const float* table, const int32_t* pos_q, const int32_t* pos_k, void* g_q_in,
                    void* g_k_in, float* g_w_q, float* g_w_k, void* ws, hipStream_t stream) {
  const int lanes = group_lanes(n.head_dim);
  NrSide<T> a = side<T>(p, n, true, lanes, q, w_q, pos_q, g_q_in);
  NrSide<T> b = side<T>(p, n, false, lanes, k, w_k, pos_k, g_k_in);
  a.g = static_cast<const T*>(g_q);
  b.g = static_cast<const T*>(g_k);
  const int64_t tokens = a.tokens > b.tokens ? a.tokens : b.tokens;
  const int64_t bx = bwd_blocks(tokens, lanes);
  a.part = static_cast<float*>(ws);
  b.part = a.part + (int64_t)a.chunks * bx * n.head_dim;
  if (tokens) {
    const dim3 grid((unsigned)bx, a.chunks + b.chunks);
#define NT_LAUNCH(P)                                                                         \
  k_norm_rotary_bwd<T, P><<<grid, kNrThreads, 0, stream>>>(a, b, table, n.positions, p.B,    \
                                                           n.head_dim, n.rot_dim, lanes, n.eps)
    switch (pairs_of(n)) {
      case kPairsInLane: NT_LAUNCH(kPairsInLane); break;
      case kPairsInLine: NT_LAUNCH(kPairsInLine); break;
      default: NT_LAUNCH(kPairsAnywhere);
    }
#undef NT_LAUNCH
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!w_q && !w_k) return hipSuccess;
  k_norm_weight_sum<<<dim3((n.head_dim + 15) / 16, 2), 256, 0, stream>>>(
      a.part, b.part, (int)(a.chunks * bx), (int)(b.chunks * bx), w_q ? g_w_q : nullptr,
      w_k ? g_w_k : nullptr, n.head_dim);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rotary_table(const nt_rotary& r, float* table, int64_t positions,
                               hipStream_t stream) {
  if (positions == 0) return hipSuccess;
  const int64_t bx = (positions + 255) / 256;
  k_rotary_table<<<dim3((unsigned)(bx < 1024 ? bx : 1024), r.rot_dim / 2), 256, 0, stream>>>(
      table, positions, r.rot_dim, r.scaling, r.base, r.factor, r.original, r.beta_fast,
      r.beta_slow, r.magnitude);
  return hipGetLastError();
}

hipError_t launch_norm_rotary(const nt_partition& p, const nt_norm_rotary& n, const void* q,
                              const void* k, const float* w_q, const float* w_k,
                              const float* table, const int32_t* pos_q, const int32_t* pos_k,
                              void* q_out, void* k_out, nt_dtype dtype, hipStream_t stream) {
  return dtype == NT_BF16 ? forward<bf16>(p, n, q, k, w_q, w_k, table, pos_q, pos_k, q_out, k_out,
                                          stream)
                          : forward<float>(p, n, q, k, w_q, w_k, table, pos_q, pos_k, q_out,
                                           k_out, stream);
}

size_t norm_rotary_backward_ws_bytes(const nt_partition& p, const nt_norm_rotary& n) {
  const int lanes = group_lanes(n.head_dim);
  const NrSide<float> a = side<float>(p, n, true, lanes, nullptr, nullptr, nullptr, nullptr);
  const NrSide<float> b = side<float>(p, n, false, lanes, nullptr, nullptr, nullptr, nullptr);
  const int64_t tokens = a.tokens > b.tokens ? a.tokens : b.tokens;
  return (size_t)(a.chunks + b.chunks) * bwd_blocks(tokens, lanes) * n.head_dim * sizeof(float);
}

hipError_t launch_norm_rotary_backward(const nt_partition& p, const nt_norm_rotary& n,
                                       const void* q, const void* k, const void* g_q,
                                       const void* g_k, const float* w_q, const float* w_k,
                                       const float* table, const int32_t* pos_q,
                                       const int32_t* pos_k, void* g_q_in, void* g_k_in,
                                       float* g_w_q, float* g_w_k, void* ws, nt_dtype dtype,
                                       hipStream_t stream) {
  return dtype == NT_BF16
             ? backward<bf16>(p, n, q, k, g_q, g_k, w_q, w_k, table, pos_q, pos_k, g_q_in, g_k_in,
                              g_w_q, g_w_k, ws, stream)
             : backward<float>(p, n, q, k, g_q, g_k, w_q, w_k, table, pos_q, pos_k, g_q_in,
                               g_k_in, g_w_q, g_w_k, ws, stream);
}

}  // namespace nt
