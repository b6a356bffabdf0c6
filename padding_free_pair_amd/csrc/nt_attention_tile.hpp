// Pieces that the attention kernels and their gradients share: matrix-core
// fragments of both storage types, tiles of token rows in LDS, and the map
// from workgroups to samples.
//
// Fragments are those of the 32 x 32 x 16 bf16 product: lane l holds row (or
// column) l % 32 and, of the 16 values of k, the 8 of its half h = l / 32. The
// fp32 product takes the same fragments as eight 32 x 32 x 2 products, the
// j-th over the j-th values of both halves, so one kernel serves both types.
// A product's result holds column l % 32 in lane l, rows 8 (i / 4) + 4 h + i % 4
// for i = 0 .. 15. Eight consecutive results of a lane are rows {4 h + 0 .. 3,
// 8 + 4 h + 0 .. 3} of a block of 16: as a fragment of the next product they
// are its 16 values of k in another order, which the other operand takes too.
#pragma once

#include "nt_device.hpp"

namespace nt {

constexpr float kLog2e = 1.44269504088896340736f;

typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef short at_i16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 at_bf16x4 __attribute__((ext_vector_type(4)));
typedef float at_f32x4 __attribute__((ext_vector_type(4)));

template <typename T> struct AtFrag;
template <> struct AtFrag<bf16> { typedef bf16x8 type; };
template <> struct AtFrag<float> { typedef f32x8 type; };

__device__ __forceinline__ f32x16 at_mma(const bf16x8& a, const bf16x8& b, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 at_mma(const f32x8& a, const f32x8& b, f32x16 c) {
#pragma unroll
  for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
  return c;
}

// Where a tile of token rows keeps its elements in LDS, by the fragments that
// are read from it, without bank conflicts.
// AtAlong: along rows only. 16 rows are read at once, 16 bytes of each: a pitch
// of an odd number of 16 bytes.
template <typename T, int DP> struct AtAlong {
  static constexpr int pitch = DP + 16 / (int)sizeof(T);
  static __device__ __forceinline__ int at(int r, int c) { return r * pitch + c; }
};
// AtAcross: across rows only. bf16: four rows at once, 64 bytes of each: a pitch
// of 64 bytes modulo 256, or of 192. fp32: rows 4 apart on different halves of
// the banks.
template <typename T, int DP> struct AtAcross {
  static constexpr int pitch = sizeof(T) == 4 ? DP + 8 : DP % 64 == 0 ? DP + 32 : DP;
  static __device__ __forceinline__ int at(int r, int c) { return r * pitch + c; }
};
// AtBoth: both. bf16: rows of 16-byte chunks, chunk c of row r at c ^ f(r);
// along a row, 16 rows read one chunk each, which f must send to the 16 chunks
// of 256 bytes; across rows, 4 rows read 4 neighbouring chunks each, which f
// must send to the 4 different 64-byte pieces: f's high bits are r's low ones.
// fp32: AtAlong's pitch, which serves the other kind half.
template <typename T, int DP> struct AtBoth;
template <int DP> struct AtBoth<bf16, DP> {
  static constexpr int pitch = DP == 96 ? 128 : DP;
  static __device__ __forceinline__ int at(int r, int c) {
    const int f = pitch == 128 ? (r & 3) << 2 | ((r >> 2) & 3)
                  : pitch == 64 ? ((r >> 1) & 1) << 2 | ((r >> 2) & 3) : (r >> 2) & 3;
    return r * pitch + (((c >> 3) ^ f) << 3) + (c & 7);
  }
};
template <int DP> struct AtBoth<float, DP> : AtAlong<float, DP> {};

// Values 16 s + 8 h .. of a row in global memory as a fragment.
__device__ __forceinline__ bf16x8 at_row(const bf16* row, int s, int h) {
  return *reinterpret_cast<const bf16x8*>(row + 16 * s + 8 * h);
}
__device__ __forceinline__ f32x8 at_row(const float* row, int s, int h) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(row + 16 * s + 8 * h);
  const f32x4 b = *reinterpret_cast<const f32x4*>(row + 16 * s + 8 * h + 4);
  return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// Fragment along row r of a tile, values 16 s + 8 h ..
template <typename L> __device__ __forceinline__ bf16x8 at_along(const bf16* tile, int r, int s, int h) {
  return *reinterpret_cast<const bf16x8*>(tile + L::at(r, 16 * s + 8 * h));
}
template <typename L> __device__ __forceinline__ f32x8 at_along(const float* tile, int r, int s, int h) {
  return at_row(tile + L::at(r, 0), s, h);
}

// Four bf16 by the transposing LDS read: within each 16 lanes, lane j's
// element e is element j % 4 of the 8 bytes at the address of lane 4 e + j / 4.
__device__ __forceinline__ at_bf16x4 at_read_tr(const bf16* p) {
  const at_i16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) at_i16x4*)(p));
  return __builtin_bit_cast(at_bf16x4, v);
}

// Fragment across rows: column c0 + l % 32 of the tile, rows r0 + {4 h + 0 ..
// 3, 8 + 4 h + 0 .. 3} (the order of a product's results).
template <typename L> __device__ __forceinline__ bf16x8 at_across(const bf16* tile, int r0, int c0) {
  const int lane = threadIdx.x & 63, h = lane >> 5, q = lane & 15, g = lane >> 4;
  const int r = r0 + 4 * h + (q >> 2), c = c0 + 16 * (g & 1) + 4 * (q & 3);
  const at_bf16x4 a = at_read_tr(tile + L::at(r, c));
  const at_bf16x4 b = at_read_tr(tile + L::at(r + 8, c));
  return bf16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}
template <typename L> __device__ __forceinline__ f32x8 at_across(const float* tile, int r0, int c0) {
  const int lane = threadIdx.x & 63, h = lane >> 5;
  constexpr int P = L::pitch;
  const float* p = tile + (r0 + 4 * h) * P + c0 + (lane & 31);
  f32x8 f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[j] = p[j * P];
    f[4 + j] = p[(8 + j) * P];
  }
  return f;
}

// Eight results of a product, from the i-th, as a fragment.
__device__ __forceinline__ void at_pack(const f32x16& x, int i, bf16x8& f) {
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = (bf16)x[i + j];
}
__device__ __forceinline__ void at_pack(const f32x16& x, int i, f32x8& f) {
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = x[i + j];
}

// Four consecutive values to global memory.
__device__ __forceinline__ void at_store4(bf16* p, float a, float b, float c, float d) {
  *reinterpret_cast<at_bf16x4*>(p) = at_bf16x4{(bf16)a, (bf16)b, (bf16)c, (bf16)d};
}
__device__ __forceinline__ void at_store4(float* p, float a, float b, float c, float d) {
  *reinterpret_cast<at_f32x4*>(p) = at_f32x4{a, b, c, d};
}

// Four bias values of a row, from column c on; the ones past `m` as zeros. A row
// begins at any element, so the four are one unaligned load.
__device__ __forceinline__ void at_bias4(const bf16* p, int64_t c, int64_t m, float* f) {
  if (c + 4 <= m) {
    at_bf16x4 v;
    __builtin_memcpy(&v, p + c, 8);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = (float)v[e];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = c + e < m ? (float)p[c + e] : 0.0f;
  }
}
__device__ __forceinline__ void at_bias4(const float* p, int64_t c, int64_t m, float* f) {
  if (c + 4 <= m) {
    __builtin_memcpy(f, p + c, 16);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = c + e < m ? p[c + e] : 0.0f;
  }
}

// A tile of ROWS token rows of D elements (D <= DP) on its way to LDS: pieces
// of 16 bytes, one after another over the THREADS threads. The distances of a
// thread's pieces from the tile's first row stay the same from tile to tile
// (ld <= 2^22 keeps them in 32 bits), so a load is a uniform base and one
// register. Rows past the last one read the last one (their weight is zero).
template <typename T, int ROWS, int DP, int THREADS> struct AtStage {
  static constexpr int kVec = 16 / sizeof(T);
  static constexpr int kPieces = ROWS * DP / kVec / THREADS;
  static_assert(ROWS * DP % (kVec * THREADS) == 0, "whole pieces");
  typedef T Vec __attribute__((ext_vector_type(16 / sizeof(T))));
  Vec v[kPieces];
  uint32_t off[kPieces];
  static __device__ __forceinline__ int row(int u) { return (threadIdx.x + u * THREADS) * kVec / DP; }
  static __device__ __forceinline__ int col(int u) { return (threadIdx.x + u * THREADS) * kVec % DP; }
  __device__ __forceinline__ AtStage(int64_t ld) {
#pragma unroll
    for (int u = 0; u < kPieces; ++u)
      off[u] = (uint32_t)((row(u) * (uint32_t)ld + col(u)) * sizeof(T));
  }
  // first: the tile's first row; rows: how many there are from it on (>= 1)
  __device__ __forceinline__ void load(const T* first, int64_t ld, int rows, int D) {
    const char* base = reinterpret_cast<const char*>(first);
    if (rows >= ROWS && D == DP) {
#pragma unroll
      for (int u = 0; u < kPieces; ++u) v[u] = *reinterpret_cast<const Vec*>(base + off[u]);
    } else {
#pragma unroll
      for (int u = 0; u < kPieces; ++u) {
        const int r = row(u) < rows ? row(u) : rows - 1, c = col(u);
        v[u] = Vec{};
        if (c < D) v[u] = *reinterpret_cast<const Vec*>(first + r * ld + c);
      }
    }
  }
  template <typename L> __device__ __forceinline__ void put(T* tile) const {
#pragma unroll
    for (int u = 0; u < kPieces; ++u)
      *reinterpret_cast<Vec*>(tile + L::at(row(u), col(u))) = v[u];
  }
};

// Keeps the compiler from turning a branch that few tiles take into selects
// that every tile pays for.
__device__ __forceinline__ void at_rare() { asm volatile("" ::: "memory"); }

// The larger of a lane's value and its partner's in the other half.
__device__ __forceinline__ float at_halves_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x),
                                                  __builtin_bit_cast(uint32_t, x), false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}

// Tiles of `tile` rows of ragged samples without a list of them: sample i
// owns the slots [off_i mult / tile + i, off_{i+1} mult / tile + i + 1), at
// least ceil(n_i mult / tile) of them, so a launch takes total mult / tile + B
// slots and the few that are left over return. The sample of a slot is found
// by a search in which a wave compares 64 offsets at once.
__device__ __forceinline__ int at_sample_of(const int64_t* off, int B, int mult, int tile,
                                            int64_t slot) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = B;  // the last i in [lo, lo + n) whose first slot is <= slot
  while (n > 1) {
    const int step = (n + 63) / 64;
    const int i = lo + lane * step;
    const bool before = lane * step < n && off[i] * mult / tile + i <= slot;
    const int k = __popcll(__ballot(before)) - 1;
    const int next = lo + k * step;
    n = n - k * step < step ? n - k * step : step;
    lo = next;
  }
  return lo;
}
inline int64_t at_slots(int64_t total, int B, int mult, int tile) {
  return total * mult / tile + B;
}

}  // namespace nt
