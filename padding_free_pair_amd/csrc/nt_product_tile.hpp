// A product of two matrices by one workgroup, D[m, n] = sum_k A(m, k) B(n, k),
// for the kernels that put something of their own in the place of D's store.
//
// Each operand lies in memory along k (a row of k's for each m or n) or across
// it (a row of m's or n's for each k). A tile of BK values of k, 128 bytes, is
// loaded straight to LDS as it lies; fragments of operands across k are read
// by the transposing LDS read. The layouts in LDS are those of the attention's
// tiles (AtTileMap), which no fragment read of either kind conflicts in. The
// result of a wave is MT x NT blocks of 32 x 32: lane l holds column n = l % 32
// of a block and rows m = 8 (i / 4) + 4 (l / 32) + i % 4.
#pragma once

#include "nt_attention_tile.hpp"

namespace nt {

template <typename T, int MT, int NT, int WM, int WN> struct PtShape {
  typedef T type;
  static constexpr int mt = MT, nt = NT, wm = WM, wn = WN;
  static constexpr int m = 32 * MT * WM, n = 32 * NT * WN, threads = 64 * WM * WN;
  static constexpr int bk = 128 / (int)sizeof(T);   // values of k in a tile
  static constexpr int sub = 256 / (int)sizeof(T);  // columns of a piece of a tile across k
  static constexpr int bytes = (m + n) * 128;       // of LDS for one tile of each operand
};

// Loads of tiles of an operand that lies along k: ROWS rows of 128 bytes.
template <typename T, int ROWS, int THREADS> struct PtAlong {
  typedef AtTile<T, 128 / (int)sizeof(T)> L;
  static constexpr int pieces = ROWS * 8 / THREADS;
  static_assert(ROWS * 8 % THREADS == 0, "whole pieces");
  const char* at[pieces];
  static __device__ __forceinline__ int row(int u) { return (threadIdx.x + u * THREADS) / 8; }
  static __device__ __forceinline__ int col(int u) {
    return ((threadIdx.x + u * THREADS) % 8 ^ L::turn(row(u))) * L::vec;
  }
  // where(r): the first element of the tile's row r, of a row that is there
  template <typename Where> __device__ __forceinline__ explicit PtAlong(const Where& where) {
#pragma unroll
    for (int u = 0; u < pieces; ++u)
      at[u] = reinterpret_cast<const char*>(where(row(u)) + col(u));
  }
  // Values k0 .. of all rows to LDS address `tile`; zeros from K on.
  __device__ __forceinline__ void start(int64_t k0, int64_t K, uint32_t tile) const {
    const uint32_t to = tile + (threadIdx.x & ~63) * 16;
    if (k0 + L::pitch <= K) {
#pragma unroll
      for (int u = 0; u < pieces; ++u)
        at_load_lds<16>(at[u] + k0 * (int64_t)sizeof(T), to + u * THREADS * 16);
    } else {
      at_rare();
#pragma unroll
      for (int u = 0; u < pieces; ++u) {
        const void* from = k0 + col(u) < K ? (const void*)(at[u] + k0 * (int64_t)sizeof(T))
                                           : (const void*)&kAtZeros;
        at_load_lds<16>(from, to + u * THREADS * 16);
      }
    }
  }
  // Fragment of row r (of the lane), values 16 s + 8 h ..
  static __device__ __forceinline__ auto frag(const char* tile, int r, int s) {
    return at_along<128 / (int)sizeof(T)>(reinterpret_cast<const T*>(tile), r + (threadIdx.x & 31),
                                          s, (threadIdx.x & 63) >> 5);
  }
};

// The same of an operand that lies across k: BK rows of COLS columns, in pieces
// of 256 bytes a row.
template <typename T, int COLS, int THREADS> struct PtAcross {
  static constexpr int sub = 256 / (int)sizeof(T), bk = 128 / (int)sizeof(T);
  typedef AtTile<T, sub> L;
  static constexpr int pieces = COLS * 8 / THREADS;
  static_assert(COLS % sub == 0 && COLS * 8 % THREADS == 0, "whole pieces");
  uint32_t off[pieces];
  const T* base;
  int64_t ld;
  static __device__ __forceinline__ int row(int u) {
    return (threadIdx.x + u * THREADS) / 16 % bk;
  }
  static __device__ __forceinline__ int col(int u) {
    const int i = threadIdx.x + u * THREADS;
    return i / (16 * bk) * sub + (i % 16 ^ L::turn(row(u))) * L::vec;
  }
  // base: the tile's first column in row 0; cols: how many columns there are
  // from it on (a multiple of 8), ld: elements from row to row (bk ld bytes fit 32 bits).
  // Columns that are not there read the row's first ones.
  __device__ __forceinline__ PtAcross(const T* b, int64_t cols, int64_t l) : base(b), ld(l) {
#pragma unroll
    for (int u = 0; u < pieces; ++u)
      off[u] = (uint32_t)((row(u) * ld + (col(u) < cols ? col(u) : 0)) * (int64_t)sizeof(T));
  }
  // Rows k0 .. of the array's K to LDS; rows from K on read the last one.
  __device__ __forceinline__ void start(int64_t k0, int64_t K, uint32_t tile) const {
    const uint32_t to = tile + (threadIdx.x & ~63) * 16;
    const char* from = reinterpret_cast<const char*>(base + k0 * ld);
    if (k0 + bk <= K) {
#pragma unroll
      for (int u = 0; u < pieces; ++u) at_load_lds16(from, off[u], to + u * THREADS * 16);
    } else {
      at_rare();
#pragma unroll
      for (int u = 0; u < pieces; ++u) {
        const int64_t past = k0 + row(u) - (K - 1);
        at_load_lds<16>(from + off[u] - (past > 0 ? past * ld * (int64_t)sizeof(T) : 0),
                        to + u * THREADS * 16);
      }
    }
  }
  // Fragment of column c + l % 32, rows 16 s + 8 h ..
  static __device__ __forceinline__ bf16x8 frag_of(const bf16* tile, int c, int s) {
    const int lane = threadIdx.x & 63, h = lane >> 5, q = lane & 15, g = lane >> 4;
    const int r = 16 * s + 8 * h + (q >> 2), x = c + 16 * (g & 1) + 4 * (q & 3);
    const at_bf16x4 a = at_read_tr(tile + L::at(r, x));
    const at_bf16x4 b = at_read_tr(tile + L::at(r + 4, x));
    return bf16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  }
  static __device__ __forceinline__ f32x8 frag_of(const float* tile, int c, int s) {
    const int lane = threadIdx.x & 63, r = 16 * s + 8 * (lane >> 5), x = c + (lane & 31);
    f32x8 f;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = tile[L::at(r + j, x)];
    return f;
  }
  static __device__ __forceinline__ auto frag(const char* tile, int c, int s) {
    const T* t = reinterpret_cast<const T*>(tile) + (c / sub) * (bk * sub);
    return frag_of(t, c % sub, s);
  }
};

// The walk over k: tiles j = 0 .. n - 1, load(j, LDS address) starts the loads of
// tile j of both operands (B behind A), one tile ahead of the products.
template <typename S, typename A, typename B, typename Load>
__device__ __forceinline__ void pt_product(f32x16 (&acc)[S::mt][S::nt], char* smem, int64_t n,
                                           const Load& load) {
  const int wave = threadIdx.x >> 6, m0 = wave / S::wn * 32 * S::mt, n0 = wave % S::wn * 32 * S::nt;
  const uint32_t lds = at_lds(smem);
#pragma unroll
  for (int i = 0; i < S::mt; ++i)
#pragma unroll
    for (int j = 0; j < S::nt; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  if (n > 0) load((int64_t)0, lds);
  for (int64_t t = 0; t < n; ++t) {
    at_arrive<0>();  // tile t is there, and every wave is done with tile t - 1
    if (t + 1 < n) load(t + 1, lds + (uint32_t)((t + 1) & 1) * S::bytes);
    const char* a = smem + (t & 1) * S::bytes;
    const char* b = a + S::m * 128;
#pragma unroll
    for (int s = 0; s < S::bk / 16; ++s) {
      typename AtFrag<typename S::type>::type fa[S::mt], fb[S::nt];
#pragma unroll
      for (int i = 0; i < S::mt; ++i) fa[i] = A::frag(a, m0 + 32 * i, s);
#pragma unroll
      for (int j = 0; j < S::nt; ++j) fb[j] = B::frag(b, n0 + 32 * j, s);
#pragma unroll
      for (int i = 0; i < S::mt; ++i)
#pragma unroll
        for (int j = 0; j < S::nt; ++j) acc[i][j] = at_mma(fa[i], fb[j], acc[i][j]);
    }
  }
}

// Tiles over the eight dies: workgroups go to the dies in turn, so each die
// takes a stretch of the tiles' order, and in that order four tiles of m stay
// together over all tiles of n: what the 32 workgroups of a die read at a time
// is 4 + 8 strips of the operands, which its cache holds.
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
inline int64_t pt_grid(int64_t tiles) { return (tiles + 7) / 8 * 8; }

}  // namespace nt
