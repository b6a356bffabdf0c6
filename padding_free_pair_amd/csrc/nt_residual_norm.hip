// The singles' norm with the residual's addition in the same pass, its output
// in the storage type or in 8 bits with scales, and its gradient.
//
// h = x + residual is rounded to the storage type once and y = h / sqrt(mean
// h^2 + eps) w is that of the rounded sum, so that the gradient, which reads h,
// sees the numbers that the forward used. A team of lanes takes a row, 8
// consecutive columns a lane and chunk, and keeps the row in registers: every
// array is read and written once, which is what bounds both directions. Teams
// are 8 to 64 lanes for rows of up to 2,048 columns (sums by lane exchanges), a
// workgroup for wider ones.
//
// 8 bits: e4m3 codes in units of a scale, the largest magnitude of the row or of
// each `group` columns times the fp32 number next to 1/448 (the format of the
// optimizer's states). The magnitudes are those of y in fp32, before any
// rounding.
//
// Gradient: with r = 1 / sqrt(mean h^2 + eps) and xhat = h r,
//   g = r (g_y w - xhat mean(g_y w xhat)) + g_h,   g_w = sum over rows of g_y xhat.
// Both row sums join in one exchange. A team walks over rows and keeps its
// columns' weight sums in registers; workgroups write theirs, and a second
// kernel adds them in order.
//
// Measured, 16,384 rows of 4,096 in bf16: forward with the residual to 8 bits 99 us for
// 470 MB, 4.8 TB/s; gradient with g_h 102 us for 537 MB, 5.3 TB/s, and 6.5 us for g_w.
#include <math.h>

#include <algorithm>

#include "nt_device.hpp"
#include "nt_internal.hpp"

namespace nt {
namespace {

constexpr int kRnThreads = 256;
constexpr int64_t kRnMostGrid = int64_t(1) << 20;
constexpr int kRnMostBlocks = 512;  // of the gradient: two for each compute unit

template <typename T> __device__ __forceinline__ void rn_load(const T* p, float* f);
template <> __device__ __forceinline__ void rn_load<bf16>(const bf16* p, float* f) {
  const bf16x8 v = *reinterpret_cast<const bf16x8*>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = (float)v[i];
}
template <> __device__ __forceinline__ void rn_load<float>(const float* p, float* f) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = a[i];
    f[4 + i] = b[i];
  }
}
template <typename T> __device__ __forceinline__ void rn_store(T* p, const float* f);
template <> __device__ __forceinline__ void rn_store<bf16>(bf16* p, const float* f) {
  bf16x8 v;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (bf16)f[i];
  *reinterpret_cast<bf16x8*>(p) = v;
}
template <> __device__ __forceinline__ void rn_store<float>(float* p, const float* f) {
  *reinterpret_cast<f32x4*>(p) = f32x4{f[0], f[1], f[2], f[3]};
  *reinterpret_cast<f32x4*>(p + 4) = f32x4{f[4], f[5], f[6], f[7]};
}

// Eight columns of a row as they lie in memory.
template <typename T> struct RnRaw {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ float get(int e) const {
    T t[8];
    __builtin_memcpy(t, v, sizeof(t));
    return (float)t[e];
  }
};

struct RnSum {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct RnMax {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

// A value of every lane of a team joined over `lanes` of them (a power of two;
// the whole team where lanes is LANES). scratch: LDS of one float a wave.
template <int LANES, typename Op>
__device__ __forceinline__ float rn_join(float v, int lanes, const Op& op, float* scratch) {
  for (int m = 1; m < (lanes < 64 ? lanes : 64); m <<= 1) v = op(v, __shfl_xor(v, m));
  if (LANES > 64 && lanes > 64) {
    __syncthreads();  // the scratch may still be read
    if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = v;
    __syncthreads();
    v = scratch[0];
#pragma unroll
    for (int w = 1; w < LANES / 64; ++w) v = op(v, scratch[w]);
  }
  return v;
}

template <typename T> struct RnForward {
  const T* x;
  const T* residual;
  const float* w;
  T* h;        // null without a residual
  T* y;
  uint8_t* codes;
  float* scales;
  int64_t rows;
  int C, group;  // group 0: the row
  float eps;
};

template <typename T, int LANES, int NV, bool CODES>
__device__ __forceinline__ void rn_forward(const RnForward<T>& p, int64_t row, float* scratch) {
  const int lane = threadIdx.x % LANES;
  // teams without a row take the last one and store nothing: lane exchanges stay whole
  const int64_t at = (row < p.rows ? row : p.rows - 1) * p.C;
  const bool store = row < p.rows;
  float f[NV][8], sum = 0.0f;
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int c = (lane + u * LANES) * 8;
    if (c < p.C) {
      rn_load<T>(p.x + at + c, f[u]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[u][e] = 0.0f;
    }
  }
  if (p.residual) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int c = (lane + u * LANES) * 8;
      if (c < p.C) {
        float g[8];
        rn_load<T>(p.residual + at + c, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[u][e] = (float)(T)(f[u][e] + g[e]);
        if (store) rn_store<T>(p.h + at + c, f[u]);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < NV; ++u)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += f[u][e] * f[u][e];
  sum = rn_join<LANES>(sum, LANES, RnSum(), scratch);
  const float r = 1.0f / sqrtf(sum / (float)p.C + p.eps);
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int c = (lane + u * LANES) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[u][e] *= r;
    if (p.w && c < p.C) {
      float w[8];
      rn_load<float>(p.w + c, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[u][e] *= w[e];
    }
  }
  if constexpr (!CODES) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int c = (lane + u * LANES) * 8;
      if (store && c < p.C) rn_store<T>(p.y + at + c, f[u]);
    }
  } else {
    float top[NV];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      top[u] = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) top[u] = fmaxf(top[u], isfinite(f[u][e]) ? fabsf(f[u][e]) : 0.0f);
    }
    if (p.group) {
#pragma unroll
      for (int u = 0; u < NV; ++u) top[u] = rn_join<LANES>(top[u], p.group / 8, RnMax(), scratch);
    } else {
#pragma unroll
      for (int u = 1; u < NV; ++u) top[0] = fmaxf(top[0], top[u]);
      top[0] = rn_join<LANES>(top[0], LANES, RnMax(), scratch);
#pragma unroll
      for (int u = 1; u < NV; ++u) top[u] = top[0];
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int c = (lane + u * LANES) * 8;
      const float scale = top[u] * (1.0f / 448.0f);
      // the quotients as products with the scale's inverse (one more rounding of
      // fp32, 2^-24); small scales times 2^64 first, so that the inverse is finite
      const float lift = scale < 1.0f ? 0x1p64f : 1.0f;
      const float inverse = scale > 0.0f ? 1.0f / (scale * lift) : 0.0f;
      float q[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = f[u][e] * lift * inverse;
      // A normal scale leaves nothing past 448 but roundings. A subnormal one may be rounded to
      // far less than the largest value's 448th, and the conversion makes NaN of what is past
      // its range. NaN and infinities do become the NaN code.
      if (scale < 0x1p-126f) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (isfinite(q[e])) q[e] = fminf(fmaxf(q[e], -448.0f), 448.0f);
      }
      uint32_t a = 0, b = 0;
      a = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], a, false);
      a = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], a, true);
      b = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], b, false);
      b = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], b, true);
      if (store && c < p.C) {
        *reinterpret_cast<uint2*>(p.codes + at + c) = make_uint2(a, b);
        if (p.group) {
          if (c % p.group == 0) p.scales[(at + c) / p.group] = scale;
        } else if (c == 0) {
          p.scales[row] = scale;
        }
      }
    }
  }
}

template <typename T, int LANES, int NV, bool CODES>
__global__ __launch_bounds__(kRnThreads) void k_rn_forward(RnForward<T> p) {
  constexpr int kTeams = kRnThreads / LANES;
  __shared__ float scratch[kRnThreads / 64];
  for (int64_t first = (int64_t)blockIdx.x * kTeams; first < p.rows;
       first += (int64_t)gridDim.x * kTeams)
    rn_forward<T, LANES, NV, CODES>(p, first + threadIdx.x / LANES, scratch);
}

template <typename T> struct RnBackward {
  const T* h;
  const T* g_y;
  const T* g_h;
  const float* w;
  T* g;
  float* part;  // [workgroups][C], null without w
  int64_t rows;
  int C;
  float eps;
};

// Two values of every lane of a team summed in one exchange.
template <int LANES> __device__ __forceinline__ float2 rn_sum2(float2 v, float2* scratch) {
#pragma unroll
  for (int m = 1; m < (LANES < 64 ? LANES : 64); m <<= 1) {
    v.x += __shfl_xor(v.x, m);
    v.y += __shfl_xor(v.y, m);
  }
  if (LANES > 64) {
    if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = v;
    __syncthreads();
    v = scratch[0];
#pragma unroll
    for (int w = 1; w < LANES / 64; ++w) {
      v.x += scratch[w].x;
      v.y += scratch[w].y;
    }
  }
  return v;
}

template <typename T, int LANES, int NV>
__global__ __launch_bounds__(kRnThreads) void k_rn_backward(RnBackward<T> p) {
  constexpr int kTeams = kRnThreads / LANES;
  __shared__ float2 scratch[2][kRnThreads / 64];  // in turn, so that one barrier a row is enough
  const int lane = threadIdx.x % LANES, team = threadIdx.x / LANES;
  float w[NV][8], sums[NV][8];
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int c = (lane + u * LANES) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[u][e] = 1.0f;
      sums[u][e] = 0.0f;
    }
    if (p.w && c < p.C) rn_load<float>(p.w + c, w[u]);
  }
  const int64_t step = (int64_t)gridDim.x * kTeams;
  // the next row is loaded while this one is worked on (rows of up to 8,192 columns: the
  // wider ones have no registers left)
  constexpr bool kAhead = NV <= 4;
  RnRaw<T> h[NV], g[NV], more[NV];
  const auto load = [&](int64_t first) {
    const int64_t row = first + team;
    const int64_t at = (row < p.rows ? row : p.rows - 1) * p.C;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int c = (lane + u * LANES) * 8;
      more[u].zero();
      if (c < p.C) {
        h[u].load(p.h + at + c);
        g[u].load(p.g_y + at + c);
        if (p.g_h) more[u].load(p.g_h + at + c);
      } else {
        h[u].zero();
        g[u].zero();
      }
    }
  };
  int turn = 0;
  if (kAhead) load((int64_t)blockIdx.x * kTeams);
  for (int64_t first = (int64_t)blockIdx.x * kTeams; first < p.rows; first += step, turn ^= 1) {
    const int64_t row = first + team;
    const bool is = row < p.rows;  // the others keep the lane exchanges whole
    if (!kAhead) load(first);
    const int64_t at = row * p.C;
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s.x += h[u].get(e) * h[u].get(e);
        s.y += h[u].get(e) * (g[u].get(e) * w[u][e]);
      }
    s = rn_sum2<LANES>(s, scratch[turn]);
    const float r = 1.0f / sqrtf(s.x / (float)p.C + p.eps);
    const float mean = r * s.y / (float)p.C;  // of g_y w xhat
    float out[NV][8];
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xhat = h[u].get(e) * r;
        out[u][e] = r * (g[u].get(e) * w[u][e] - xhat * mean) + more[u].get(e);
        if (is) sums[u][e] += g[u].get(e) * xhat;
      }
    if (kAhead && first + step < p.rows) load(first + step);
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int c = (lane + u * LANES) * 8;
      if (is && c < p.C) rn_store<T>(p.g + at + c, out[u]);
    }
  }
  if (!p.part) return;
  // the teams' sums of a column, in their order
  float* part = p.part + (int64_t)blockIdx.x * p.C;
  if constexpr (kTeams == 1) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int c = (lane + u * LANES) * 8;
      if (c < p.C) rn_store<float>(part + c, sums[u]);
    }
  } else {
    __shared__ float all[kTeams][LANES * NV * 8];
#pragma unroll
    for (int u = 0; u < NV; ++u) rn_store<float>(&all[team][(lane + u * LANES) * 8], sums[u]);
    __syncthreads();
    for (int c = threadIdx.x; c < p.C; c += kRnThreads) {
      float s = all[0][c];
      for (int k = 1; k < kTeams; ++k) s += all[k][c];
      part[c] = s;
    }
  }
}

// g_w[c] = the workgroups' sums added: 32 columns x 32 stretches of workgroups, 8 loads
// of a thread in flight (8 stretches and one load after the other: 17 us).
constexpr int kRnWeightThreads = 1024;
__global__ __launch_bounds__(kRnWeightThreads) void k_rn_weights(const float* part, float* g_w,
                                                                 int blocks, int C) {
  __shared__ double all[32][33];
  const int lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane, k = threadIdx.x >> 5;
  double s = 0.0;
  if (c < C)
    for (int b = k; b < blocks; b += 256) {
      float f[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) f[u] = b + 32 * u < blocks ? part[(int64_t)(b + 32 * u) * C + c] : 0.0f;
#pragma unroll
      for (int u = 0; u < 8; ++u) s += (double)f[u];
    }
  all[k][lane] = s;
  __syncthreads();
  if (k || c >= C) return;
#pragma unroll
  for (int i = 1; i < 32; ++i) s += all[i][lane];
  g_w[c] = (float)s;
}

// The team of a row of C columns: run(lanes, chunks of a lane).
template <int LANES, int NV> struct RnTeam {
  static constexpr int lanes = LANES, nv = NV;
};
template <typename Run> hipError_t rn_teams(int C, const Run& run) {
  const int chunks = C / 8;
  if (chunks <= 8) return run(RnTeam<8, 1>());
  if (chunks <= 16) return run(RnTeam<16, 1>());
  if (chunks <= 32) return run(RnTeam<32, 1>());
  if (chunks <= 64) return run(RnTeam<64, 1>());
  if (chunks <= 128) return run(RnTeam<64, 2>());
  if (chunks <= 256) return run(RnTeam<64, 4>());
  if (chunks <= 512) return run(RnTeam<256, 2>());
  if (chunks <= 1024) return run(RnTeam<256, 4>());
  return run(RnTeam<256, 8>());
}

int rn_teams_of_block(int C) { return C > 2048 ? 1 : C <= 64 ? 32 : C <= 128 ? 16 : C <= 256 ? 8 : 4; }

int backward_blocks(int64_t rows, int C) {
  const int64_t teams = rn_teams_of_block(C);
  return (int)std::min<int64_t>((rows + teams - 1) / teams, kRnMostBlocks);
}

template <typename T>
hipError_t forward(const RnForward<T>& p, hipStream_t s) {
  return rn_teams(p.C, [&](auto team) {
    typedef decltype(team) Team;
    const int64_t teams = kRnThreads / Team::lanes;
    const uint32_t grid = (uint32_t)std::min<int64_t>((p.rows + teams - 1) / teams, kRnMostGrid);
    if (p.codes)
      k_rn_forward<T, Team::lanes, Team::nv, true><<<grid, kRnThreads, 0, s>>>(p);
    else
      k_rn_forward<T, Team::lanes, Team::nv, false><<<grid, kRnThreads, 0, s>>>(p);
    return hipGetLastError();
  });
}

template <typename T>
hipError_t backward(const RnBackward<T>& p, float* g_w, hipStream_t s) {  // g_w: null without w
  const int blocks = backward_blocks(p.rows, p.C);
  hipError_t e = hipSuccess;
  if (blocks) {
    e = rn_teams(p.C, [&](auto team) {
      typedef decltype(team) Team;
      k_rn_backward<T, Team::lanes, Team::nv><<<blocks, kRnThreads, 0, s>>>(p);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  if (!p.w) return hipSuccess;
  k_rn_weights<<<(p.C + 31) / 32, kRnWeightThreads, 0, s>>>(p.part, g_w, blocks, p.C);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_residual_norm(const void* x, const void* residual, const float* w, void* h,
                                void* y, uint8_t* codes, float* scales, int64_t rows, int C,
                                int group, float eps, nt_dtype dtype, hipStream_t s) {
  if (rows == 0) return hipSuccess;
  if (dtype == NT_BF16)
    return forward(RnForward<bf16>{static_cast<const bf16*>(x), static_cast<const bf16*>(residual),
                                   w, static_cast<bf16*>(h), static_cast<bf16*>(y), codes, scales,
                                   rows, C, group, eps},
                   s);
  return forward(RnForward<float>{static_cast<const float*>(x), static_cast<const float*>(residual),
                                  w, static_cast<float*>(h), static_cast<float*>(y), codes, scales,
                                  rows, C, group, eps},
                 s);
}

size_t residual_norm_backward_ws_bytes(int64_t rows, int C) {
  return align256(sizeof(float) * (size_t)backward_blocks(rows, C) * C);
}

hipError_t launch_residual_norm_backward(const void* h, const void* g_y, const void* g_h,
                                         const float* w, void* g, float* g_w, int64_t rows, int C,
                                         float eps, nt_dtype dtype, void* ws, hipStream_t s) {
  float* part = w ? static_cast<float*>(ws) : nullptr;
  if (dtype == NT_BF16)
    return backward(RnBackward<bf16>{static_cast<const bf16*>(h), static_cast<const bf16*>(g_y),
                                     static_cast<const bf16*>(g_h), w, static_cast<bf16*>(g), part,
                                     rows, C, eps},
                    g_w, s);
  return backward(RnBackward<float>{static_cast<const float*>(h), static_cast<const float*>(g_y),
                                    static_cast<const float*>(g_h), w, static_cast<float*>(g), part,
                                    rows, C, eps},
                  g_w, s);
}

}  // namespace nt
