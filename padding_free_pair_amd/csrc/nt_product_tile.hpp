// A product of two matrices by one workgroup, D[m, n] = sum_k A(m, k) B(n, k),
// for the kernels that put something of their own in the place of D's store.
//
// An operand lies along k (a row of k's for each m or n) or across it (a row of m's
// or n's for each k). A tile of BK values of k, 128 bytes of every row along k, is
// loaded straight to LDS as it lies; the chunks of a row are turned (across k as those
// of the attention's tiles, AtTileMap), so that fragments along k are read without
// conflicts. Fragments across k take the transposing LDS read, which moves 8 bytes a
// lane where the plain one moves 16: a product with both operands across k reached 1,120
// TFLOP/s, so at least one of them is better transposed in memory once.
//
// Products are 16 x 16 x 32 in bf16: lane l holds row (or column) l % 16 of a
// block and, of the 32 values of k, the 8 of its quarter g = l / 16; in fp32 the
// same fragments are eight 16 x 16 x 4 products, the j-th over the j-th values
// of all quarters. The result of a wave is MT x NT blocks: lane l holds column
// n = l % 16 of a block and rows m = 4 g + 0 .. 3.
//
// Measured at 16,384 x 8,192 x 2,048 (bf16, results summed, not stored), 256 x
// 256 tiles of 8 waves: 1,430 TFLOP/s (the library's products of these sizes
// reach 1,260 to 1,380). With blocks of 32 x 32 x 16 1,345; with all of a tile's
// loads behind the barrier at once 1,280; with tiles of 64 bytes in a ring of four
// or five 1,240; 4 waves of 128 x 128 1,260; tiles of 128 x 128 1,115.
#pragma once

#include "nt_attention_tile.hpp"

namespace nt {

template <typename T, int MT, int NT, int WM, int WN> struct PtShape {
  typedef T type;
  static constexpr int mt = MT, nt = NT, wm = WM, wn = WN;
  static constexpr int m = 16 * MT * WM, n = 16 * NT * WN, threads = 64 * WM * WN;
  static constexpr int bk = 128 / (int)sizeof(T);  // values of k in a tile
  static constexpr int bytes = (m + n) * 128;      // of LDS for one tile of each operand
  static constexpr int lds = 2 * bytes;
};

__device__ __forceinline__ f32x4 pt_mma(const bf16x8& a, const bf16x8& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 pt_mma(const f32x8& a, const f32x8& b, f32x4 c) {
#pragma unroll
  for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
  return c;
}
// The products of all blocks, in fp32 one value of k of all blocks after the other, so
// that none waits for the one before it.
template <int MT, int NT>
__device__ __forceinline__ void pt_mma(const bf16x8 (&a)[MT], const bf16x8 (&b)[NT],
                                       f32x4 (&c)[MT][NT]) {
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) c[i][j] = pt_mma(a[i], b[j], c[i][j]);
}
template <int MT, int NT>
__device__ __forceinline__ void pt_mma(const f32x8 (&a)[MT], const f32x8 (&b)[NT],
                                       f32x4 (&c)[MT][NT]) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
        c[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i][k], b[j][k], c[i][j], 0, 0, 0);
}

// The thread's index where few tiles need it: nothing that follows from it is kept in
// registers over the walk.
__device__ __forceinline__ int pt_thread() {
  int t = threadIdx.x;
  asm volatile("" : "+v"(t)::"memory");
  return t;
}

template <typename V> __device__ __forceinline__ V pt_lds(uint32_t at) {
  return *(const __attribute__((address_space(3))) V*)(uintptr_t)at;
}

// Tiles of an operand that lies along k: ROWS rows of 128 bytes, the loads of a
// thread, and the fragments.
template <typename T, int ROWS, int THREADS> struct PtRows {
  static constexpr int vec = 16 / (int)sizeof(T);  // elements of a chunk, 8 chunks a row
  static constexpr int pieces = ROWS * 8 / THREADS;
  static_assert(ROWS * 8 % THREADS == 0, "whole pieces");
  static constexpr bool S32 = sizeof(T) == 4;
  // A row's chunks are turned (XOR) by its place in 16 rows. Two rows are a line of the 64
  // banks, so rows 2 r and 2 r + 1 share a turn and the 8 of them differ. The 16 lanes that
  // are served together hold rows 0 .. 3 and 12 .. 15 of one quarter and 4 .. 11 of the next
  // one, whose chunk differs in bit 0 (fp32: 1): that bit is the row's bit 1, which takes
  // either value in both groups. (With its bit 2 there half of the reads' cycles were
  // conflicts, and a loss of 8,007 tokens over 65,537 words took 8.6e8 cycles of the compute
  // units where it takes 8.2e8, LDS busy for 48 % of them where it is for 25.)
  static __device__ __forceinline__ int turn(int r) {
    return S32 ? (r >> 3 & 1) << 2 | (r >> 1 & 1) << 1 | (r >> 2 & 1) : r >> 1 & 7;
  }
  static __device__ __forceinline__ int row(int thread, int u) { return (thread + u * THREADS) / 8; }
  static __device__ __forceinline__ int col(int thread, int u) {
    return ((thread + u * THREADS) % 8 ^ turn(row(thread, u))) * vec;
  }
  // The lane's bytes in a tile: row r + l % 16, values 8 g ..; r is a multiple of 16.
  static __device__ __forceinline__ uint32_t lane(int r) {
    const int l = threadIdx.x & 63;
    return (uint32_t)((r + (l & 15)) * 128 + (8 * (l >> 4) / vec ^ turn(l & 15)) * 16);
  }
  // Block i (16 rows on), values 32 s + 8 g .., at the LDS address of lane(r). The turn
  // of a row's chunks goes by its place in 16 rows; steps and halves are bits of the chunk.
  static __device__ __forceinline__ auto frag(uint32_t at, int i, int s) {
    const uint32_t p = (at ^ (uint32_t)(64 * s)) + (uint32_t)(i * 16 * 128);
    if constexpr (!S32) {
      return pt_lds<bf16x8>(p);
    } else {
      const f32x4 a = pt_lds<f32x4>(p), b = pt_lds<f32x4>(p ^ 16);
      return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    }
  }
};

// Rows of one array: place(r) is the array's row, from `base` on, of the tile's row r.
template <typename T, int ROWS, int THREADS> struct PtAlong : PtRows<T, ROWS, THREADS> {
  typedef PtRows<T, ROWS, THREADS> Base;
  using Base::pieces;
  uint32_t off[Base::pieces];
  const T* base;
  // ld: elements from row to row; all places are within 4 GiB of base
  template <typename Place>
  __device__ __forceinline__ PtAlong(const T* b, int64_t ld, const Place& place) : base(b) {
#pragma unroll
    for (int u = 0; u < pieces; ++u) {
      off[u] = (uint32_t)((place(Base::row(threadIdx.x, u)) * ld + Base::col(threadIdx.x, u)) *
                          (int64_t)sizeof(T));
      asm volatile("" : "+v"(off[u]));  // one register, not the 64 bits it comes from
    }
  }
  // Values k0 .. of all rows to LDS address `tile`, zeros from K on, of the array that lies
  // `plane` elements on.
  __device__ __forceinline__ void start(int64_t k0, int64_t K, uint32_t tile,
                                        int64_t plane = 0) const {
    const uint32_t to = tile + (threadIdx.x & ~63) * 16;
    const char* from = reinterpret_cast<const char*>(base + plane + k0);
    if (k0 + 8 * Base::vec <= K) {
#pragma unroll
      for (int u = 0; u < pieces; ++u) at_load_lds16(from, off[u], to + u * THREADS * 16);
    } else {
      const int thread = pt_thread();
#pragma unroll
      for (int u = 0; u < pieces; ++u) {
        uint32_t o = off[u];
        asm volatile("" : "+v"(o));
        at_load_lds<16>(k0 + Base::col(thread, u) < K ? (const void*)(from + o)
                                                      : (const void*)&kAtZeros,
                        to + u * THREADS * 16);
      }
    }
  }
};

// Tiles of an operand that lies across k: BK rows of COLS columns, in pieces of
// 256 bytes a row. All rows and columns of a tile are there.
template <typename T, int COLS, int THREADS> struct PtAcross {
  static constexpr int sub = 256 / (int)sizeof(T), bk = 128 / (int)sizeof(T);
  typedef AtTile<T, sub> L;
  static constexpr int pieces = COLS * 8 / THREADS;
  static_assert(COLS % sub == 0 && COLS * 8 % THREADS == 0, "whole pieces");
  uint32_t off[pieces];
  const T* base;
  int64_t ld;
  // base: the tile's first column in row 0; ld: elements from row to row (bk of them within
  // 4 GiB)
  __device__ __forceinline__ PtAcross(const T* b, int64_t l) : base(b), ld(l) {
#pragma unroll
    for (int u = 0; u < pieces; ++u) {
      const int i = threadIdx.x + u * THREADS, row = i / 16 % bk;
      const int col = i / (16 * bk) * sub + (i % 16 ^ L::turn(row)) * L::vec;
      off[u] = (uint32_t)((row * ld + col) * (int64_t)sizeof(T));
      asm volatile("" : "+v"(off[u]));
    }
  }
  // Rows k0 .. to LDS address `tile`, of the array that lies `plane` elements on.
  __device__ __forceinline__ void start(int64_t k0, uint32_t tile, int64_t plane = 0) const {
    const uint32_t to = tile + (threadIdx.x & ~63) * 16;
    const char* from = reinterpret_cast<const char*>(base + plane + k0 * ld);
#pragma unroll
    for (int u = 0; u < pieces; ++u) at_load_lds16(from, off[u], to + u * THREADS * 16);
  }
  // The lane's bytes in a tile, of columns c .. (a multiple of a wave's columns). In bf16:
  // within each 16 lanes the transposing read gives lane j the values j % 4 of the lanes
  // 4 e + j / 4, so lane i's address is that of row i / 4, columns 4 (i % 4) ..
  static __device__ __forceinline__ uint32_t lane(int c) {
    const int l = threadIdx.x & 63, g = l >> 4, i = l & 15;
    const int at = sizeof(T) == 2 ? L::at(8 * g + (i >> 2), c % sub + 4 * (i & 3))
                                  : L::at(8 * g, c % sub + i);
    return (uint32_t)((c / sub * (bk * sub) + at) * (int)sizeof(T));
  }
  // Column c + 16 i + l % 16, rows 32 s + 8 g ..: blocks are bits of the chunk, and the
  // turn of a row's chunks goes by its place in 16 rows.
  static __device__ __forceinline__ auto frag(uint32_t at, int i, int s) {
    if constexpr (sizeof(T) == 2) {
      const uint32_t p = at ^ (uint32_t)(32 * i);
      const at_bf16x4 a = tr(p + 32 * 256 * s), b = tr((p ^ 16) + 32 * 256 * s + 4 * 256);
      return bf16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    } else {
      f32x8 f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        f[j] = pt_lds<float>((at ^ (uint32_t)(64 * i ^ 16 * (j >> 2 << 3 | (j & 3)))) +
                             (32 * s + j) * 256);
      return f;
    }
  }
  static __device__ __forceinline__ at_bf16x4 tr(uint32_t at) {
    return __builtin_bit_cast(
        at_bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                       (__attribute__((address_space(3))) at_i16x4*)(uintptr_t)at));
  }
};

// The results of a wave.
template <typename S> struct PtSums {
  f32x4 d[S::mt][S::nt];
  static __device__ __forceinline__ int first_m() {  // of the wave, within the tile
    return (int)(threadIdx.x >> 6) / S::wn * 16 * S::mt;
  }
  static __device__ __forceinline__ int first_n() {
    return (int)(threadIdx.x >> 6) % S::wn * 16 * S::nt;
  }
};

// The fragments of one step of 32 values of k, of a wave's blocks.
template <typename S> struct PtFrags {
  typename AtFrag<typename S::type>::type a[S::mt], b[S::nt];
  // at: LDS addresses of the lane's part of both tiles. They pass through an empty
  // statement, or the compiler keeps every block's address in a register of its own.
  template <typename A, typename B>
  __device__ __forceinline__ void read(uint32_t at_a, uint32_t at_b, int s) {
    asm volatile("" : "+v"(at_a), "+v"(at_b));
#pragma unroll
    for (int i = 0; i < S::mt; ++i) a[i] = A::frag(at_a, i, s);
#pragma unroll
    for (int j = 0; j < S::nt; ++j) b[j] = B::frag(at_b, j, s);
  }
  __device__ __forceinline__ void multiply(PtSums<S>& acc) const {
    __builtin_amdgcn_sched_barrier(0);
    pt_mma(a, b, acc.d);
    __builtin_amdgcn_sched_barrier(0);
  }
};

// The walk over k: tiles t = 0 .. n - 1; load_a(t, LDS address), load_b start the
// loads of tile t. Two tiles in LDS; fragments are read one step ahead of their
// products. The barrier between two tiles stands before the last step's products,
// whose fragments are in registers by then: behind it the next tile's first
// fragments are read and one operand's part of the tile after it starts on its way,
// while the matrix cores go on; the other operand's part follows a step later, so that
// the loads of a tile do not stand in one queue. The first one has two steps to arrive, the
// other one: A_FIRST where A comes from further away.
template <bool A_FIRST, typename S, typename A, typename B, typename LoadA, typename LoadB>
__device__ __forceinline__ void pt_product(PtSums<S>& acc, char* smem, int64_t n,
                                           const LoadA& load_a, const LoadB& load_b) {
  constexpr int kSteps = S::bk / 32;
  constexpr uint32_t kB = S::m * 128;  // where B's tile lies behind A's
  const uint32_t lds = at_lds(smem);
  const uint32_t at_a = lds + A::lane(acc.first_m()), at_b = lds + kB + B::lane(acc.first_n());
  const auto first = [&](int64_t t, uint32_t buffer) {
    if (A_FIRST) load_a(t, lds + buffer); else load_b(t, lds + buffer + kB);
  };
  const auto second = [&](int64_t t, uint32_t buffer) {
    if (A_FIRST) load_b(t, lds + buffer + kB); else load_a(t, lds + buffer);
  };
#pragma unroll
  for (int i = 0; i < S::mt; ++i)
#pragma unroll
    for (int j = 0; j < S::nt; ++j) acc.d[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (n <= 0) return;
  first(0, 0);
  second(0, 0);
  if (n > 1) first(1, S::bytes);
  if (kSteps == 1 && n > 1) second(1, S::bytes);
  if (n > 1)
    at_arrive<(A_FIRST ? A::pieces : B::pieces) +
              (kSteps > 1 ? 0 : A_FIRST ? B::pieces : A::pieces)>();
  else
    at_arrive<0>();
  PtFrags<S> f[2];
  f[0].template read<A, B>(at_a, at_b, 0);
  // tile t in the buffer `here` bytes on, its first fragments in f[F]
  const auto step = [&](int64_t t, uint32_t here, auto which) {
    constexpr int F = decltype(which)::value;
    const uint32_t there = S::bytes - here;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if (s + 1 < kSteps) {
        f[(F + s + 1) & 1].template read<A, B>(at_a + here, at_b + here, s + 1);
        if (s == 0 && t + 1 < n) second(t + 1, there);
      } else if (t + 1 < n) {
        at_arrive<0>();  // the next tile is there, and every wave has read all of this one
        f[(F + kSteps) & 1].template read<A, B>(at_a + there, at_b + there, 0);
        if (t + 2 < n) {
          first(t + 2, here);
          if (kSteps == 1) second(t + 2, here);
        }
      }
      f[(F + s) & 1].multiply(acc);
    }
  };
  if constexpr (kSteps % 2 == 0) {
    for (int64_t t = 0; t < n; ++t) step(t, (uint32_t)(t & 1) * S::bytes, AtIndex<0>());
  } else {
    for (int64_t t = 0; t < n; t += 2) {
      step(t, 0, AtIndex<0>());
      if (t + 1 < n) step(t + 1, S::bytes, AtIndex<1>());
    }
  }
}

// Tiles over the eight dies: workgroups go to the dies in turn, so each die
// takes a stretch of the tiles' order, and in that order four tiles of m stay
// together over all tiles of n: what the 32 workgroups of a die read at a time
// is 4 + 8 strips of the operands, which its cache holds. A launch has the tiles' number
// rounded up to whole eights of workgroups.
constexpr int kPtGroup = 4;
__device__ __forceinline__ bool pt_tile(uint32_t id, uint32_t tiles_m, uint32_t tiles_n, uint32_t* m,
                                        uint32_t* n) {
  const uint32_t total = tiles_m * tiles_n, each = (total + 7) / 8;
  const uint32_t at = (id & 7) * each + (id >> 3);
  if (id >> 3 >= each || at >= total) return false;
  const uint32_t group = at / (kPtGroup * tiles_n), in = at - group * kPtGroup * tiles_n;
  const uint32_t first = group * kPtGroup;
  const uint32_t have = tiles_m - first < kPtGroup ? tiles_m - first : kPtGroup;
  *m = first + in % have;
  *n = in / have;
  return true;
}

}  // namespace nt
