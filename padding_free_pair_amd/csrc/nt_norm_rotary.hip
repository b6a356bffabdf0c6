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
// read. Memory bounds both directions: 16,384 tokens of 32 + 8 heads of 128
// (bf16, read from one projected array) take 84 us, 4.0 TB/s where a large copy
// reaches 4.95; the gradient of 16 + 4 heads 58 us and its weight sums 5, 4.0
// TB/s together. Small batches (810 tokens of 4 + 4 heads of 32) take 5 us on the
// GPU, and the call's host side bounds them.
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
template <int PAIRS>
__device__ __forceinline__ void nr_angles(const float* table, int64_t at, int64_t positions, int R,
                                          int e0, float* c, float* s) {
  const bool inside = at >= 0 && at < positions;
  const float* row = table + (inside ? at : 0) * R;
  if (PAIRS == kPairsInLine) {  // eight angles in a row, and half a head is whole lanes
    if (e0 < R) {
      const bool first = e0 < R / 2;
      const float* p = row + (first ? e0 : e0 - R / 2);
      nr_load<float>(p, c);
      nr_load<float>(p + R / 2, s);
#pragma unroll
      for (int i = 0; i < kNrVec; ++i) s[i] = first ? -s[i] : s[i];
    }
  } else if (PAIRS == kPairsInLane && R % 8 == 0) {  // four angles in a row
    if (e0 < R) {
      const f32x4 u = *reinterpret_cast<const f32x4*>(row + e0 / 2);
      const f32x4 v = *reinterpret_cast<const f32x4*>(row + R / 2 + e0 / 2);
#pragma unroll
      for (int i = 0; i < kNrVec; ++i) {
        c[i] = u[i / 2];
        s[i] = i & 1 ? v[i / 2] : -v[i / 2];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kNrVec; ++i) {
      const int e = e0 + i;
      if (e < R) {
        const int j = PAIRS == kPairsInLane ? e >> 1 : (e < R / 2 ? e : e - R / 2);
        const bool first = PAIRS == kPairsInLane ? !(e & 1) : e < R / 2;
        c[i] = row[j];
        s[i] = first ? -row[R / 2 + j] : row[R / 2 + j];
      }
    }
  }
  if (!inside)
#pragma unroll
    for (int i = 0; i < kNrVec; ++i) c[i] = __builtin_nanf("");
}

// The lane's part of a head as it is stored, and its partners' part.
template <typename T, int PAIRS> struct NrHead {
  T own[kNrVec], other[kNrVec];
  __device__ __forceinline__ void load(const T* head, int e0, int R, bool partners) {
    typedef T Vec __attribute__((ext_vector_type(16 / sizeof(T))));
    constexpr int n = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < kNrVec; i += n)
      *reinterpret_cast<Vec*>(own + i) = *reinterpret_cast<const Vec*>(head + e0 + i);
    if (PAIRS == kPairsInLane || !partners) return;
    if (PAIRS == kPairsInLine) {
      const int p = nr_partner(e0, R, false);
#pragma unroll
      for (int i = 0; i < kNrVec; i += n)
        *reinterpret_cast<Vec*>(other + i) = *reinterpret_cast<const Vec*>(head + p + i);
    } else {
#pragma unroll
      for (int i = 0; i < kNrVec; ++i) other[i] = head[nr_partner(e0 + i, R, false)];
    }
  }
  __device__ __forceinline__ float partner(int i) const {
    return to_f32(PAIRS == kPairsInLane ? own[i ^ 1] : other[i]);
  }
};

template <typename T>
__device__ __forceinline__ int64_t nr_position(const NrSide<T>& a, int64_t t, int B) {
  if (a.positions) return a.positions[t];
  const int i = a.row_sample ? a.row_sample[t] : find_segment(a.offsets, 0, B, t);
  return t - a.offsets[i];
}

// grid: x over groups of tokens, y over the head chunks of q, then of k. The
// next heads are loaded before the present ones are stored (which may be in
// the same array, at heads already read).
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
  const int ec = live ? e0 : 0;  // lanes past the head read its first dimensions
  const int h0 = chunk * a.per_chunk;
  const int h1 = h0 + a.per_chunk < a.heads ? h0 + a.per_chunk : a.heads;
  float w[kNrVec], wp[kNrVec];
#pragma unroll
  for (int i = 0; i < kNrVec; ++i) {
    w[i] = a.w ? a.w[ec + i] : 1.0f;
    wp[i] = a.w ? a.w[nr_partner(ec + i, R, PAIRS == kPairsInLane)] : 1.0f;
  }
  // whole groups leave together
  for (int64_t t = (int64_t)blockIdx.x * groups + threadIdx.x / lanes; t < a.tokens;
       t += (int64_t)gridDim.x * groups) {
    const T* x = a.x + t * a.ld;
    T* y = a.y + t * a.ld_y;
    NrHead<T, PAIRS> now[kNrHeadsAtOnce], next[kNrHeadsAtOnce];
#pragma unroll
    for (int u = 0; u < kNrHeadsAtOnce; ++u)
      next[u].load(x + (h0 + u < h1 ? h0 + u : h0) * D, ec, R, R > 0);
    float c[kNrVec], s[kNrVec];
#pragma unroll
    for (int i = 0; i < kNrVec; ++i) {
      c[i] = 1.0f;
      s[i] = 0.0f;
    }
    if (R) nr_angles<PAIRS>(table, nr_position(a, t, B), positions, R, ec, c, s);
    for (int h = h0; h < h1; h += kNrHeadsAtOnce) {
#pragma unroll
      for (int u = 0; u < kNrHeadsAtOnce; ++u) now[u] = next[u];
      if (h + kNrHeadsAtOnce < h1) {
#pragma unroll
        for (int u = 0; u < kNrHeadsAtOnce; ++u) {
          const int hu = h + kNrHeadsAtOnce + u;
          next[u].load(x + (hu < h1 ? hu : h1 - 1) * D, ec, R, R > 0);
        }
      }
#pragma unroll
      for (int u = 0; u < kNrHeadsAtOnce; ++u) {
        float r = 1.0f, v[kNrVec];
        if (a.w) {
          float sum = 0.0f;
#pragma unroll
          for (int i = 0; i < kNrVec; ++i) sum += to_f32(now[u].own[i]) * to_f32(now[u].own[i]);
          r = 1.0f / sqrtf(nr_group_sum(live ? sum : 0.0f, lanes) / (float)D + eps);
        }
#pragma unroll
        for (int i = 0; i < kNrVec; ++i) {
          v[i] = to_f32(now[u].own[i]) * r * w[i] * c[i];
          // (a select, not a product with zero: an infinity behind the rotated part stays one)
          const float turned = v[i] + now[u].partner(i) * r * wp[i] * s[i];
          v[i] = ec + i < R ? turned : v[i];
        }
        if (live && h + u < h1) nr_store<T>(y + (h + u) * D + e0, v);
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
  __shared__ float sums[kNrThreads / 64][16 * kNrVec];
  const bool is_q = (int)blockIdx.y < q.chunks;
  const NrSide<T>& a = is_q ? q : k;
  const int chunk = is_q ? blockIdx.y : blockIdx.y - q.chunks;
  const int groups = kNrThreads / lanes;
  const int e0 = (threadIdx.x % lanes) * kNrVec;
  const bool live = e0 < D;
  const int ec = live ? e0 : 0;
  const int h0 = chunk * a.per_chunk;
  const int h1 = h0 + a.per_chunk < a.heads ? h0 + a.per_chunk : a.heads;
  float w[kNrVec], gw[kNrVec];
#pragma unroll
  for (int i = 0; i < kNrVec; ++i) {
    w[i] = a.w ? a.w[ec + i] : 1.0f;
    gw[i] = 0.0f;
  }
  for (int64_t t = (int64_t)blockIdx.x * groups + threadIdx.x / lanes; t < a.tokens;
       t += (int64_t)gridDim.x * groups) {
    const T* x = a.x + t * a.ld;
    const T* g = a.g + t * (int64_t)a.heads * D;
    T* y = a.y + t * a.ld_y;
    NrHead<T, PAIRS> gn[kNrHeadsAtOnce], gc[kNrHeadsAtOnce];
    NrHead<T, kPairsInLane> xn[kNrHeadsAtOnce], xc[kNrHeadsAtOnce];
#pragma unroll
    for (int u = 0; u < kNrHeadsAtOnce; ++u) {
      const int hu = h0 + u < h1 ? h0 + u : h0;
      gn[u].load(g + hu * D, ec, R, R > 0);
      if (a.w) xn[u].load(x + hu * D, ec, R, false);
    }
    float c[kNrVec], s[kNrVec];
#pragma unroll
    for (int i = 0; i < kNrVec; ++i) {
      c[i] = 1.0f;
      s[i] = 0.0f;
    }
    if (R) nr_angles<PAIRS>(table, nr_position(a, t, B), positions, R, ec, c, s);
    for (int h = h0; h < h1; h += kNrHeadsAtOnce) {
#pragma unroll
      for (int u = 0; u < kNrHeadsAtOnce; ++u) {
        gc[u] = gn[u];
        xc[u] = xn[u];
      }
      if (h + kNrHeadsAtOnce < h1) {
#pragma unroll
        for (int u = 0; u < kNrHeadsAtOnce; ++u) {
          const int hu = h + kNrHeadsAtOnce + u < h1 ? h + kNrHeadsAtOnce + u : h1 - 1;
          gn[u].load(g + hu * D, ec, R, R > 0);
          if (a.w) xn[u].load(x + hu * D, ec, R, false);
        }
      }
#pragma unroll
      for (int u = 0; u < kNrHeadsAtOnce; ++u) {
        const bool mine = live && h + u < h1;
        float d[kNrVec];
#pragma unroll
        for (int i = 0; i < kNrVec; ++i) {
          d[i] = to_f32(gc[u].own[i]) * c[i];
          const float turned = d[i] - gc[u].partner(i) * s[i];
          d[i] = ec + i < R ? turned : d[i];
        }
        if (a.w) {
          float sum = 0.0f, dot = 0.0f, v[kNrVec];
#pragma unroll
          for (int i = 0; i < kNrVec; ++i) {
            v[i] = to_f32(xc[u].own[i]);
            sum += v[i] * v[i];
            dot += d[i] * w[i] * v[i];
          }
          sum = nr_group_sum(live ? sum : 0.0f, lanes);
          dot = nr_group_sum(live ? dot : 0.0f, lanes);
          const float r = 1.0f / sqrtf(sum / (float)D + eps);
          dot = dot * r / (float)D;  // mean of h w xhat
#pragma unroll
          for (int i = 0; i < kNrVec; ++i) {
            v[i] *= r;  // xhat
            if (mine) gw[i] += d[i] * v[i];
            d[i] = r * (d[i] * w[i] - v[i] * dot);
          }
        }
        if (mine) nr_store<T>(y + (h + u) * D + e0, d);
      }
    }
  }
  if (!a.w) return;
  // the wave's groups by lane exchanges, then the waves in order
#pragma unroll
  for (int i = 0; i < kNrVec; ++i) {
    for (int m = lanes; m < 64; m <<= 1) gw[i] += __shfl_xor(gw[i], m);
    if ((threadIdx.x & 63) < lanes && live) sums[threadIdx.x >> 6][e0 + i] = gw[i];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < D; e += kNrThreads) {
    float sum = 0.0f;
    for (int n = 0; n < kNrThreads / 64; ++n) sum += sums[n][e];
    a.part[((int64_t)chunk * gridDim.x + blockIdx.x) * D + e] = sum;
  }
}

// Weight gradients: the partial sums added in a fixed order in fp64 (there
// are up to a few thousand of them). Block y: q or k; 4 dimensions a block,
// so 64 threads share the rows of each.
__global__ __launch_bounds__(256) void k_norm_weight_sum(const float* part_q, const float* part_k,
                                                         int rows_q, int rows_k, float* g_q,
                                                         float* g_k, int D) {
  __shared__ double sums[4][4];
  const float* part = blockIdx.y ? part_k : part_q;
  const int rows = blockIdx.y ? rows_k : rows_q;
  float* g = blockIdx.y ? g_k : g_q;
  if (!g) return;
  const int e = blockIdx.x * 4 + (threadIdx.x & 3);
  double sum = 0.0;
#pragma unroll 8
  for (int r = threadIdx.x >> 2; r < rows; r += 64) sum += (double)part[(int64_t)r * D + e];
  for (int m = 4; m < 64; m <<= 1) sum += __shfl_xor(sum, m);
  if ((threadIdx.x & 63) < 4) sums[threadIdx.x >> 6][threadIdx.x & 3] = sum;
  __syncthreads();
  if (threadIdx.x < 4)
    g[e] = (float)(sums[0][threadIdx.x] + sums[1][threadIdx.x] + sums[2][threadIdx.x] +
                   sums[3][threadIdx.x]);
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

// Heads that one group takes in turn: all of them, so that a token's angles are
// read once, unless that leaves fewer than 2,048 workgroups (8 for each CU);
// then fewer, down to one.
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
  k_norm_weight_sum<<<dim3(n.head_dim / 4, 2), 256, 0, stream>>>(
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
