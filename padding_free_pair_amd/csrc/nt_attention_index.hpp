// Index arithmetic of the attention kernels' tiles: where a tile of token rows
// keeps its elements in LDS, and which elements of the array its loads read.
// Plain constant expressions, so that a host program can check every index.
#pragma once

#include <stdint.h>

namespace nt {

// Where a tile of token rows keeps its elements in LDS: rows of 16-byte chunks
// without padding (so that loads can write them as they come), chunk c of row
// r at c ^ f(r). Fragments along rows read one chunk of 16 rows at once, which f
// must send to the 16 chunks of 256 bytes. Fragments across rows read, in bf16,
// 4 neighbouring chunks of 4 rows at once, which f must send to the 4 different
// 64-byte pieces: f's high bits are r's low ones. In fp32 they read 8 chunks of
// two rows 4 apart, which f sends to the two halves where a row has 16 chunks.
template <int SIZE, int DP> struct AtTileMap {
  static constexpr int vec = 16 / SIZE;                 // elements of a chunk
  static constexpr int pitch = DP == 96 ? 128 : DP;     // elements of a row
  static constexpr int chunks = pitch / vec;            // of a row
  static constexpr int turn(int r) {                    // f
    return SIZE == 2 ? (chunks == 16  ? (r & 3) << 2 | ((r >> 2) & 3)
                        : chunks == 8 ? ((r >> 1) & 1) << 2 | ((r >> 2) & 3)
                                      : (r >> 2) & 3)
                     : (chunks == 8 ? (r >> 1) & 7
                                    : ((r >> 2) & 1) << 3 | ((r >> 3) & 1) << 2 | (r & 3));
  }
  static constexpr int at(int r, int c) {
    return r * pitch + ((c / vec) ^ turn(r)) * vec + c % vec;
  }
};

// The chunks of a tile of ROWS token rows, THREADS threads taking them one after
// another: the element of the array that a thread's u-th chunk begins with.
template <int SIZE, int ROWS, int DP, int THREADS> struct AtLoadMap {
  typedef AtTileMap<SIZE, DP> L;
  static constexpr int pieces = ROWS * L::chunks / THREADS;  // chunks of a thread
  static_assert(ROWS * L::chunks % THREADS == 0, "whole pieces");
  static constexpr int row(int thread, int u) { return (thread + u * THREADS) / L::chunks; }
  static constexpr int col(int thread, int u) {
    return ((thread + u * THREADS) % L::chunks ^ L::turn(row(thread, u))) * L::vec;
  }
  // Bytes from the tile's first row on where a whole tile of DP columns is loaded
  // (ld <= 2^22 keeps them in 32 bits). A row of LDS may be longer than DP: its
  // chunks past the head, which no fragment reads, take the head's first one, so
  // that no load leaves the row.
  static constexpr uint32_t whole(int thread, int u, uint32_t ld) {
    return (row(thread, u) * ld + (col(thread, u) < DP ? col(thread, u) : 0)) * (uint32_t)SIZE;
  }
};

}  // namespace nt
