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

#include "nt_attention_index.hpp"
#include "nt_device.hpp"

namespace nt {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

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

template <typename T, int DP> struct AtTile : AtTileMap<(int)sizeof(T), DP> {};

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
template <int DP> __device__ __forceinline__ bf16x8 at_along(const bf16* tile, int r, int s, int h) {
  return *reinterpret_cast<const bf16x8*>(tile + AtTile<bf16, DP>::at(r, 16 * s + 8 * h));
}
template <int DP> __device__ __forceinline__ f32x8 at_along(const float* tile, int r, int s, int h) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(tile + AtTile<float, DP>::at(r, 16 * s + 8 * h));
  const f32x4 b =
      *reinterpret_cast<const f32x4*>(tile + AtTile<float, DP>::at(r, 16 * s + 8 * h + 4));
  return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
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
template <int DP> __device__ __forceinline__ bf16x8 at_across(const bf16* tile, int r0, int c0) {
  const int lane = threadIdx.x & 63, h = lane >> 5, q = lane & 15, g = lane >> 4;
  const int r = r0 + 4 * h + (q >> 2), c = c0 + 16 * (g & 1) + 4 * (q & 3);
  const at_bf16x4 a = at_read_tr(tile + AtTile<bf16, DP>::at(r, c));
  const at_bf16x4 b = at_read_tr(tile + AtTile<bf16, DP>::at(r + 8, c));
  return bf16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}
template <int DP> __device__ __forceinline__ f32x8 at_across(const float* tile, int r0, int c0) {
  const int lane = threadIdx.x & 63, r = r0 + 4 * (lane >> 5), c = c0 + (lane & 31);
  f32x8 f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[j] = tile[AtTile<float, DP>::at(r + j, c)];
    f[4 + j] = tile[AtTile<float, DP>::at(r + 8 + j, c)];
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

// Four consecutive values to global memory, at any element.
__device__ __forceinline__ void at_store4(bf16* p, float a, float b, float c, float d) {
  const at_bf16x4 v = {(bf16)a, (bf16)b, (bf16)c, (bf16)d};
  __builtin_memcpy(p, &v, sizeof(v));
}
__device__ __forceinline__ void at_store4(float* p, float a, float b, float c, float d) {
  const at_f32x4 v = {a, b, c, d};
  __builtin_memcpy(p, &v, sizeof(v));
}

// Keeps the compiler from turning a branch that few tiles take into selects
// that every tile pays for.
__device__ __forceinline__ void at_rare() { asm volatile("" ::: "memory"); }

// An address that is the same for the wave, in scalar registers.
__device__ __forceinline__ uint64_t at_uniform(const void* p) {
  const uint64_t x = reinterpret_cast<uint64_t>(p);
  return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(x >> 32)) << 32 |
         (uint32_t)__builtin_amdgcn_readfirstlane((int)x);
}

// The LDS address of a __shared__ array.
__device__ __forceinline__ uint32_t at_lds(const void* array) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)array;
}

// Loads that write LDS themselves, without passing a register: 64 lanes of
// BYTES each, from an address a lane, to consecutive places from LDS address
// `to` (the same for the wave). They have no result to wait for; at_arrive
// waits. In assembly, because the compiler would wait for the builtin's loads
// before every transposing LDS read, and with that for the tiles on their way.
template <int BYTES> __device__ __forceinline__ void at_load_lds(const void* from, uint32_t to) {
  static_assert(BYTES == 16 || BYTES == 4, "a lane loads one or four words");
  const uint32_t lds = (uint32_t)__builtin_amdgcn_readfirstlane((int)to);
  const uint64_t at = reinterpret_cast<uint64_t>(from);
  if constexpr (BYTES == 16)
    asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %1, off" ::"{m0}"(lds), "v"(at) : "memory");
  else
    asm volatile("s_nop 4\n\tglobal_load_lds_dword %1, off" ::"{m0}"(lds), "v"(at) : "memory");
}
// The same from a uniform base and a lane's distance in bytes. The base may have
// been written by a vector instruction just before (v_readfirstlane, or the return
// of a register that was put aside in a vector one): five wait states must pass
// before a load reads it, which the compiler does not see to within assembly.
__device__ __forceinline__ void at_load_lds16(const char* base, uint32_t lane, uint32_t to) {
  const uint32_t lds = (uint32_t)__builtin_amdgcn_readfirstlane((int)to);
  const uint64_t at = at_uniform(base);
  asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %1, %2"
               ::"{m0}"(lds), "v"(lane), "s"(at) : "memory");
}

// Waits until all but the last OPS vector memory operations of the wave, and its
// LDS reads, are done, then for the workgroup's other waves.
template <int OPS> __device__ __forceinline__ void at_arrive() {
  constexpr int N = OPS < 64 ? OPS : 63;  // the counter has six bits
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 7 << 4);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The buffer of a tile as a constant, so that its LDS addresses are a register
// of the loop's and an immediate.
template <int I> struct AtIndex {
  static constexpr int value = I;
};
// step(j, AtIndex<j % BUFS>) for j = 0 .. n - 1.
template <int BUFS, typename Step> __device__ __forceinline__ void at_each(int n, const Step& step) {
  static_assert(BUFS == 2 || BUFS == 3, "one or two tiles ahead");
  for (int j = 0; j < n; j += BUFS) {
    step(j, AtIndex<0>());
    if (j + 1 < n) step(j + 1, AtIndex<1>());
    if constexpr (BUFS == 3)
      if (j + 2 < n) step(j + 2, AtIndex<2>());
  }
}

__device__ const f32x4 kAtZeros = {0.0f, 0.0f, 0.0f, 0.0f};

// A tile of ROWS token rows of D elements (D <= DP) on its way to LDS, THREADS
// threads taking chunks one after another. A thread's distances from the
// tile's first row stay the same from tile to tile. Rows past the last one read
// the last one (their weight is zero); where a tile is not whole, columns past D
// read zeros.
template <typename T, int ROWS, int DP, int THREADS> struct AtLoad {
  typedef AtLoadMap<(int)sizeof(T), ROWS, DP, THREADS> Map;
  static constexpr int kPieces = Map::pieces;  // loads of a wave
  uint32_t off[kPieces];
  __device__ __forceinline__ explicit AtLoad(int64_t ld) {
#pragma unroll
    for (int u = 0; u < kPieces; ++u) off[u] = Map::whole(threadIdx.x, u, (uint32_t)ld);
  }
  // first: the tile's first row; rows: how many there are from it on (>= 1);
  // tile: its LDS address
  __device__ __forceinline__ void start(const T* first, int64_t ld, int rows, int D,
                                        uint32_t tile) const {
    const char* base = reinterpret_cast<const char*>(first);
    const uint32_t to = tile + (threadIdx.x & ~63) * 16;
    if (rows >= ROWS && D == DP) {
#pragma unroll
      for (int u = 0; u < kPieces; ++u) at_load_lds16(base, off[u], to + u * THREADS * 16);
    } else {
#pragma unroll
      for (int u = 0; u < kPieces; ++u) {
        const int row = Map::row(threadIdx.x, u), c = Map::col(threadIdx.x, u);
        const int r = row < rows ? row : rows - 1;
        const void* from = c < D ? (const void*)(first + r * ld + c) : (const void*)&kAtZeros;
        at_load_lds<16>(from, to + u * THREADS * 16);
      }
    }
  }
};

// A count (the same for the wave) that the compiler may not compute with ahead
// of its use: what follows from it stays in the branch that needs it.
__device__ __forceinline__ int64_t at_opaque(int64_t x) {
  int y = __builtin_amdgcn_readfirstlane((int)x);
  asm volatile("" : "+s"(y));
  return y;
}

// Stores of single elements at a uniform base, a lane's distance and a uniform
// one (both in bytes, below 2^31): a buffer instruction adds the three itself,
// where a global one would take a 64-bit addition for each.
struct AtBuffer {
  __amdgpu_buffer_rsrc_t r;
  __device__ __forceinline__ explicit AtBuffer(const void* p) {
    r = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(at_uniform(p)), 0, 0xffffffff,
                                          0x00027000);
  }
  template <typename T>
  __device__ __forceinline__ void store(T x, uint32_t lane, uint32_t uniform) const {
    if constexpr (sizeof(T) == 2)
      __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, x), r, lane, uniform, 0);
    else
      __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, x), r, lane, uniform, 0);
  }
};

// The larger of a lane's value and its partner's in the other half.
__device__ __forceinline__ float at_halves_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x),
                                                  __builtin_bit_cast(uint32_t, x), false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}

// A tile of the bias, ROWS rows of COLS cells, on its way to LDS through
// registers (a row begins at any element, which loads to LDS do not allow): 16
// bytes a thread and piece, consecutive threads along a row, so a row of the
// tile is read as whole lines, where lanes that read their own scores' cells
// touch 32 rows each time. In LDS it is an AtTile, read along or across rows.
// Rows past the last one read the last one; cells past a row's end read zeros (and
// their scores are masked).
template <typename T, int ROWS, int COLS, int THREADS> struct AtBiasTile {
  typedef AtTile<T, COLS> L;
  typedef T Vec __attribute__((ext_vector_type(16 / sizeof(T))));
  static constexpr int kPieces = ROWS * L::chunks / THREADS;
  static_assert(ROWS * L::chunks % THREADS == 0, "whole pieces");
  Vec v[kPieces];
  static __device__ __forceinline__ int row(int u) {
    return (threadIdx.x + u * THREADS) / L::chunks;
  }
  static __device__ __forceinline__ int col(int u) {
    return (threadIdx.x + u * THREADS) % L::chunks * L::vec;
  }
  // at[u]: the cell of the thread's u-th piece; cells: how many of the row
  // there are from the tile's first column on
  __device__ __forceinline__ void load(const T* const (&at)[kPieces], int cells) {
    if (cells >= COLS) {
#pragma unroll
      for (int u = 0; u < kPieces; ++u) __builtin_memcpy(&v[u], at[u], sizeof(Vec));
    } else {
      at_rare();
#pragma unroll
      for (int u = 0; u < kPieces; ++u)
#pragma unroll
        for (int e = 0; e < L::vec; ++e) v[u][e] = col(u) + e < cells ? at[u][e] : (T)0.0f;
    }
  }
  __device__ __forceinline__ void put(T* tile) const {
#pragma unroll
    for (int u = 0; u < kPieces; ++u)
      *reinterpret_cast<Vec*>(tile + L::at(row(u), col(u))) = v[u];
  }
};

// Four cells of a bias tile's row, from column c (a multiple of 4) on.
template <int COLS> __device__ __forceinline__ at_bf16x4 at_cells(const bf16* tile, int r, int c) {
  return *reinterpret_cast<const at_bf16x4*>(tile + AtTile<bf16, COLS>::at(r, c));
}
template <int COLS> __device__ __forceinline__ at_f32x4 at_cells(const float* tile, int r, int c) {
  return *reinterpret_cast<const at_f32x4*>(tile + AtTile<float, COLS>::at(r, c));
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
