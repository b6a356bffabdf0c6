// How the cross entropy over a vocabulary is cut into passes, pieces, tiles and parts, and
// where its workspace holds what. Host arithmetic only, so that a program without a GPU can
// say which kernels sizes lead to.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

namespace nt {
namespace token_loss {

constexpr int kMostSplits = 16;
constexpr int kThinTokens = 32;
constexpr int kThinWaves = 4;
constexpr int kThinBlocks = 1024;  // of a launch, four for each compute unit

inline int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }
inline int64_t tiles_of(int64_t x, int64_t tile) { return (x + tile - 1) / tile; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

constexpr int64_t kCus = 256;
constexpr int64_t kPieceBytes = int64_t(512) << 20;  // of d, and of the copy of the piece's rows of W
constexpr int64_t kSumsBytes = int64_t(256) << 20;   // of the parts of g_x or g_W, where there are

// How a product of m x n results over k is cut: its tile, and the workgroups launched,
// which cut k into parts where there are more of them than tiles.
struct Cut {
  bool large;
  int tile;
  int64_t launched;
  double cost;
};

// The cheaper tile, counted in steps of k that a compute unit spends on a small tile:
// whole rounds of all units (in fp32 and half a one: tokens without a target leave the last
// one fuller or emptier, and the small tile costs little more), 4 for a large tile and 1.3
// for a small one (measured in bf16: 1,430 and 1,115 TFLOP/s where the rounds are full;
// fp32: 129 and 122, 1.07), a tile's beginning and end as 300 steps more (fp32: 40), and the
// results' way through memory, `bytes` each and 8 more for each part where there are
// several, at 4 TB/s. Measured at 13 sizes in fp32 and 18 in bf16 (256 to 8,007 tokens, all of
// them or half with a target, 1,000 to 32,000 words of 256 to 2,048), forward and gradient, by
// this rule, in large tiles and in small ones, in us:
//   fp32, 1,866 (half) over 4,099 of 384: gradient 139, 188, 137; forward 44, 66, 44
//   fp32, 500 over 32,000 of 1,024:       gradient 915, 925, 933; forward 294, 273, 294
//   fp32, 4,000 over 16,000 of 256:       gradient 980, 946, 913; forward 306, 307, 311
//   bf16, 1,000 over 16,000 of 384:       gradient 139, 155, 142; forward 28, 27, 36
//   bf16, 4,096 over 8,000 of 2,048:      gradient 592, 580, 787; forward 114, 115, 165
//   bf16, 2,272 (half) over 8,000 of 2,048: gradient 248, 235, 313; forward 80, 55, 80
// The last one is the rule's worst; elsewhere it is within 15 % of the better tile in bf16
// and 8 % in fp32. The half round is fp32's alone: without it the forward of the first size
// takes 66, and with it in bf16 gradients take up to 27 % longer (4,096 over 8,000: 750) and
// forwards up to 38 %, as large tiles gain a third there and next to nothing in fp32.
inline double step_of(bool narrow) { return narrow ? 5.9e-9 : 1.4e-8; }  // seconds
inline Cut cut_of(int64_t m, int64_t n, int64_t k, double bytes, bool narrow, bool split) {
  Cut best = {};
  const double step = step_of(narrow);
  const int64_t bk = narrow ? 64 : 32;
  for (int large = 0; large < 2; ++large) {
    const int64_t tile = (narrow ? 128 : 64) << large;
    const int64_t tiles = tiles_of(m, tile) * tiles_of(n, tile);
    // as many workgroups as there is room for at a time
    const int64_t room = kCus * (large ? (narrow ? 1 : 2) : (narrow ? 2 : 4));
    const int64_t launched = split ? std::max(up(tiles, 8), room) : up(tiles, 8);
    int64_t s = std::min<int64_t>(launched / up(tiles, 8), std::min<int64_t>(kMostSplits, k / (8 * bk)));
    if (s < 1) s = 1;
    const double cost = ((double)tiles_of(tiles * s, kCus) + (narrow ? 0.0 : 0.5)) *
                            (large ? 4.0 : narrow ? 1.3 : 1.07) *
                            ((double)tiles_of(k, s) + (narrow ? 300.0 : 40.0)) +
                        (double)m * (double)n * ((s > 1 ? (double)s * 8.0 : 0.0) + bytes) / 4e12 / step;
    if (!large || cost < best.cost) best = {large != 0, (int)tile, launched, cost};
  }
  return best;
}

struct Plan {
  int64_t tokens, padded, piece, planes, ldv, ldt, x_budget;
  int w_most;
  Cut logits, singles, weights;
  // the workspace
  size_t rows, live, part, at, x, xT, WT, d, x_sums, w_sums, total;
};

// Tokens of a pass: an array of them spans 4 GiB at most, and the statistics of 128
// rows of the vocabulary each 512 MiB (or those of 256 tokens).
inline int64_t pass_of(int64_t T, int64_t V) {
  const int64_t most = (int64_t(1) << 26) / tiles_of(V, 128) / 256 * 256;
  return std::min(T, std::max<int64_t>(256, std::min<int64_t>(most, 1 << 16)));
}

inline bool thin(int64_t T) { return T <= kThinTokens; }
inline int thin_blocks(int64_t V) { return (int)std::min<int64_t>(tiles_of(V, 16 * kThinWaves), kThinBlocks); }

inline Plan forward_plan(int64_t T, int64_t V, int64_t C, bool narrow) {
  Plan p = {};
  p.tokens = pass_of(T, V);
  p.logits = cut_of(V, p.tokens, C, 0.0, narrow, false);
  size_t at = 0;
  if (thin(T)) {
    p.at = at; at = align256(at + sizeof(float) * T);
    p.part = at; at = align256(at + 2 * sizeof(float) * T * thin_blocks(V));
    p.total = at;
    return p;
  }
  p.rows = at; at = align256(at + sizeof(int32_t) * p.tokens);
  p.live = at; at = align256(at + sizeof(int64_t));
  p.at = at; at = align256(at + sizeof(float) * p.tokens);
  p.part = at; at = align256(at + 2 * sizeof(float) * p.tokens * tiles_of(V, p.logits.tile));
  p.total = at;
  return p;
}

inline Plan backward_plan(int64_t T, int64_t V, int64_t C, bool narrow) {
  Plan p = {};
  const int64_t es = narrow ? 2 : 4;
  p.tokens = pass_of(T, V);
  p.padded = up(p.tokens, 256);
  p.planes = narrow ? 2 : 1;  // of d
  // Rows of a power of two of bytes would put the same values of k of all rows in one
  // channel of the cache: a line more
  const int64_t line = 128 / es;
  p.ldt = p.padded + line;
  // rows that both the piece's arrays hold: many tokens make d the larger one, few the copy of W
  const int64_t rows = std::min(kPieceBytes / (p.ldt * es * p.planes), kPieceBytes / (C * es) - line);
  const int64_t most = std::max<int64_t>(256, rows / 256 * 256);
  // the number of pieces, from the least one on, that fills whole rounds best; each is some
  // launches more, 20 us where the card is not filled (256 tokens over 131,072 words of 8,192 in
  // bf16: five pieces by this take 4.6 ms, eight without it 5.1)
  const double launches = 2e-5 / step_of(narrow);
  double best = 0.0;
  for (int64_t pieces = tiles_of(V, most), last = pieces + 8; pieces < last; ++pieces) {
    const int64_t piece = up(tiles_of(V, pieces), 256), n = std::min(piece, V);
    const Cut l = cut_of(n, p.tokens, C, (double)(es * p.planes), narrow, false);
    const Cut x = cut_of(C, p.tokens, p.planes * n, 8.0, narrow, true);
    const Cut w = cut_of(C, n, p.planes * p.tokens, 4.0, narrow, true);
    const double cost = (double)tiles_of(V, piece) * (l.cost + x.cost + w.cost + launches);
    if (!p.piece || cost < best) {
      best = cost;
      p.piece = piece;
      p.logits = l;
      p.singles = x;
      p.weights = w;
    }
  }
  p.ldv = p.piece + line;
  const int64_t numbers = kSumsBytes / (int64_t)sizeof(float);
  // room for all parts that the workgroups allow, or for 256 MiB of them (fewer tokens with
  // a target allow more parts of fewer rows, which take no more room)
  const int64_t x_tiles = tiles_of(C, p.singles.tile) * tiles_of(p.tokens, p.singles.tile);
  const int64_t x_parts = std::min<int64_t>(kMostSplits, p.singles.launched / up(x_tiles, 8));
  p.x_budget = std::max(p.padded * C, std::min(x_parts * p.padded * C, numbers));
  const int64_t w_tiles = tiles_of(C, p.weights.tile) * tiles_of(std::min(p.piece, V), p.weights.tile);
  const int64_t w_rows = std::min(p.piece, V) * C;
  p.w_most = (int)std::max<int64_t>(
      1, std::min(std::min<int64_t>(kMostSplits, p.weights.launched / up(w_tiles, 8)), numbers / w_rows));
  size_t at = 0;
  p.rows = at; at = align256(at + sizeof(int32_t) * p.tokens);
  p.live = at; at = align256(at + sizeof(int64_t));
  p.x = at; at = align256(at + es * p.padded * C);
  p.xT = at; at = align256(at + es * p.ldt * C);
  p.WT = at; at = align256(at + es * p.ldv * C);
  p.d = at; at = align256(at + es * p.planes * p.ldt * p.piece);
  p.x_sums = at; at = align256(at + sizeof(float) * p.x_budget);
  p.w_sums = at;
  if (p.w_most > 1) at = align256(at + sizeof(float) * p.w_most * w_rows);
  p.total = at;
  return p;
}

}  // namespace token_loss
}  // namespace nt
