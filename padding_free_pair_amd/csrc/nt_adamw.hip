// AdamW over many tensors in one launch, states in 32 bits or in 8.
//
// Memory bounds it (28 bytes an element of fp32 parameters with fp32 states,
// about 15 operations), so every array is read and written once in pieces of
// 4 elements a lane and nothing else is moved: the table of tensors travels
// in the kernel's arguments, a workgroup finds its tensor by comparing its
// index with all first workgroups at once (one lane each), and the bias
// corrections are two numbers. A wave takes whole blocks of 256 elements, the
// span of one 8-bit scale, so a block's largest magnitude is a lane exchange
// and no scratch memory is needed. The 8-bit codes are e4m3 values in units
// of the block's scale: v_cvt_pk_fp8_f32 rounds to nearest even. Measured: 71
// million bf16 parameters with fp32 masters and 8-bit states (18 bytes an
// element) 253 us, 5.1 TB/s, where a large copy reaches 4.95; 20 fp32 tensors
// of 49,152 or 65,536 elements 8.5 us in one launch.
#include <math.h>

#include "nt_device.hpp"
#include "nt_internal.hpp"

namespace nt {
namespace {

constexpr int kAwThreads = 256;
constexpr int kAwTensors = 40;                    // of one launch: 64 bytes of arguments each
constexpr int kAwBlock = NT_ADAMW_BLOCK;          // elements of a wave's piece
constexpr int kAwPieces = 4;                      // pieces of a wave
constexpr int64_t kAwChunk = int64_t(kAwBlock) * kAwPieces * (kAwThreads / 64);
constexpr float kE4m3Max = 448.0f;
constexpr float kE4m3Least = 0.001953125f;  // 2^-9

typedef unsigned char u8x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

struct AdamwArgs {
  nt_adamw_tensor t[kAwTensors];
  uint32_t first[kAwTensors];  // first workgroup of each tensor
  int count;
};

struct AdamwNumbers {
  float lr, beta1, rest1, beta2, rest2, eps, decay;
  float c1, c2;          // 1 / (1 - beta^step)
  double b1, b2, wd64;
  const int64_t* step_device;
  const float* lr_device;
};

// Four elements at p + i, the ones past n as zeros.
template <typename T> __device__ __forceinline__ void aw_load(const T* p, int64_t i, int64_t n,
                                                              float* f) {
  typedef T T4 __attribute__((ext_vector_type(4)));
  if (i + 4 <= n) {
    const T4 v = *reinterpret_cast<const T4*>(p + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = (float)v[e];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = i + e < n ? (float)p[i + e] : 0.0f;
  }
}
template <typename T> __device__ __forceinline__ void aw_store(T* p, int64_t i, int64_t n,
                                                               const float* f) {
  typedef T T4 __attribute__((ext_vector_type(4)));
  if (i + 4 <= n) {
    T4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (T)f[e];
    *reinterpret_cast<T4*>(p + i) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < n) p[i + e] = (T)f[e];
  }
}

__device__ __forceinline__ uint32_t aw_load_codes(const uint8_t* p, int64_t i, int64_t n) {
  if (i + 4 <= n) return *reinterpret_cast<const uint32_t*>(p + i);
  uint32_t c = 0;
  for (int e = 0; e < 4; ++e)
    if (i + e < n) c |= (uint32_t)p[i + e] << (8 * e);
  return c;
}
__device__ __forceinline__ void aw_store_codes(uint8_t* p, int64_t i, int64_t n, uint32_t c) {
  if (i + 4 <= n) {
    *reinterpret_cast<uint32_t*>(p + i) = c;
    return;
  }
  for (int e = 0; e < 4; ++e)
    if (i + e < n) p[i + e] = (uint8_t)(c >> (8 * e));
}

__device__ __forceinline__ void aw_values(uint32_t c, float scale, float* f) {
  f[0] = __builtin_amdgcn_cvt_f32_fp8(c, 0) * scale;
  f[1] = __builtin_amdgcn_cvt_f32_fp8(c, 1) * scale;
  f[2] = __builtin_amdgcn_cvt_f32_fp8(c, 2) * scale;
  f[3] = __builtin_amdgcn_cvt_f32_fp8(c, 3) * scale;
}

__device__ __forceinline__ float aw_wave_max(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v = fmaxf(v, __shfl_xor(v, m));
  return v;
}

// The codes of a wave's 256 values and their scale, which is their largest
// magnitude times the rounded 1/448, not the rounded quotient (part of the format:
// a state is read back with the scale that it was written with). Values that are not
// finite get the NaN code and do not enter the scale.
__device__ __forceinline__ uint32_t aw_codes(const float* f, bool positive, float* scale) {
  float top = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) top = fmaxf(top, isfinite(f[e]) ? fabsf(f[e]) : 0.0f);
  *scale = aw_wave_max(top) * (1.0f / kE4m3Max);
  float y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    y[e] = *scale > 0.0f ? f[e] / *scale : 0.0f;
    y[e] = fminf(fmaxf(y[e], -kE4m3Max), kE4m3Max);
    if (positive && f[e] > 0.0f) y[e] = fmaxf(y[e], kE4m3Least);
  }
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], c, false);
  c = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], c, true);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (!isfinite(f[e])) c = (c & ~(0xffu << (8 * e))) | (0x7fu << (8 * e));
  return c;
}

// The moments and the codes' quotients are formed by separately rounded fp32
// operations in the order written (no contraction to fused multiply-adds):
// a code that lies next to a rounding border is then the one that any
// program gets that follows the formulas in fp32, a resumed run on another
// machine among them.
template <typename T, int BITS>
__global__ __launch_bounds__(kAwThreads) void k_adamw(AdamwArgs args, AdamwNumbers h) {
#pragma clang fp contract(off)
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool before = lane < args.count && args.first[lane < args.count ? lane : 0] <= blockIdx.x;
  const int which = __builtin_amdgcn_readfirstlane(__popcll(__ballot(before)) - 1);
  const nt_adamw_tensor t = args.t[which];
  const int64_t chunk = (int64_t)(blockIdx.x - args.first[which]) * kAwChunk;
  float lr = h.lr, c1 = h.c1, c2 = h.c2, decay = h.decay;
  if (h.step_device) {
    const double step = (double)*h.step_device;
    c1 = (float)(1.0 / (1.0 - pow(h.b1, step)));
    c2 = (float)(1.0 / (1.0 - pow(h.b2, step)));
  }
  if (h.lr_device) {
    lr = *h.lr_device;
    decay = (float)(1.0 - (double)lr * h.wd64);
  }
  T* param = static_cast<T*>(t.param);
#pragma unroll
  for (int u = 0; u < kAwPieces; ++u) {
    const int64_t piece = chunk + (int64_t)(u * (kAwThreads / 64) + wave) * kAwBlock;
    if (piece >= t.n) return;  // whole waves
    const int64_t i = piece + lane * 4;
    float g[4], p[4], m[4], v[4];
    aw_load(t.grad, i, t.n, g);
    if (t.master) aw_load(t.master, i, t.n, p);
    else aw_load(param, i, t.n, p);
    if (BITS == 8) {
      const int64_t b = piece / kAwBlock;
      aw_values(aw_load_codes(static_cast<const uint8_t*>(t.m), i, t.n), t.m_scale[b], m);
      aw_values(aw_load_codes(static_cast<const uint8_t*>(t.v), i, t.n), t.v_scale[b], v);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= v[e];
    } else {
      aw_load(static_cast<const float*>(t.m), i, t.n, m);
      aw_load(static_cast<const float*>(t.v), i, t.n, v);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      m[e] = h.beta1 * m[e] + h.rest1 * g[e];
      v[e] = h.beta2 * v[e] + h.rest2 * g[e] * g[e];
      p[e] = p[e] * decay - lr * (m[e] * c1) / (sqrtf(v[e] * c2) + h.eps);
    }
    if (t.master) aw_store(t.master, i, t.n, p);
    aw_store(param, i, t.n, p);
    if (BITS == 8) {
      float sm, sv;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = sqrtf(v[e]);
      const uint32_t cm = aw_codes(m, false, &sm), cv = aw_codes(v, true, &sv);
      aw_store_codes(static_cast<uint8_t*>(t.m), i, t.n, cm);
      aw_store_codes(static_cast<uint8_t*>(t.v), i, t.n, cv);
      if (lane == 0) {
        const int64_t b = piece / kAwBlock;
        t.m_scale[b] = sm;
        t.v_scale[b] = sv;
      }
    } else {
      aw_store(static_cast<float*>(t.m), i, t.n, m);
      aw_store(static_cast<float*>(t.v), i, t.n, v);
    }
  }
}

}  // namespace

hipError_t launch_adamw(const nt_adamw_tensor* tensors, int32_t count, const nt_adamw& h,
                        nt_dtype dtype, hipStream_t stream) {
  AdamwNumbers x;
  x.lr = (float)h.lr;
  x.beta1 = (float)h.beta1;
  x.rest1 = (float)(1.0 - h.beta1);
  x.beta2 = (float)h.beta2;
  x.rest2 = (float)(1.0 - h.beta2);
  x.eps = (float)h.eps;
  x.decay = (float)(1.0 - h.lr * h.weight_decay);
  x.c1 = (float)(1.0 / (1.0 - pow(h.beta1, (double)h.step)));
  x.c2 = (float)(1.0 / (1.0 - pow(h.beta2, (double)h.step)));
  x.b1 = h.beta1;
  x.b2 = h.beta2;
  x.wd64 = h.weight_decay;
  x.step_device = h.step_device;
  x.lr_device = h.lr_device;
  AdamwArgs args;
  args.count = 0;
  uint64_t blocks = 0;
  for (int32_t i = 0; i <= count; ++i) {
    const uint64_t more =
        i < count ? (uint64_t)((tensors[i].n + kAwChunk - 1) / kAwChunk) : 0;
    const bool full = args.count == kAwTensors || blocks + more > kAdamwMostBlocks;
    if (args.count && (i == count || full)) {
#define NT_LAUNCH(T, BITS) k_adamw<T, BITS><<<(unsigned)blocks, kAwThreads, 0, stream>>>(args, x)
      if (dtype == NT_BF16) {
        if (h.state_bits == 8) NT_LAUNCH(bf16, 8);
        else NT_LAUNCH(bf16, 32);
      } else {
        if (h.state_bits == 8) NT_LAUNCH(float, 8);
        else NT_LAUNCH(float, 32);
      }
#undef NT_LAUNCH
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      args.count = 0;
      blocks = 0;
    }
    if (i == count || more == 0) continue;
    args.t[args.count] = tensors[i];
    args.first[args.count++] = (uint32_t)blocks;
    blocks += more;
  }
  return hipSuccess;
}

}  // namespace nt
