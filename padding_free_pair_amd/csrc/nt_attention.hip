// Attention of each pair row's query over its sample's pair columns, in one
// pass over the keys with a running maximum and sum.
//
// A wave owns 32 virtual rows: the queries of one sample that read one key
// head, (row, head of the group) with the head fastest, so shared key heads
// fill the rows of a tile and are read once for their group. It forms the
// scores transposed, S^T = K Q^T: a lane then holds one row's scores for 32 of
// a tile's keys, its softmax is within the lane and its partner in the
// other half, and the probabilities are, as they stand, the fragments of the
// second product O^T = V^T P^T: they never leave the registers. The waves of a
// workgroup share each tile of keys and values in LDS, which loads write
// directly, one or two tiles ahead. QW waves own
// different rows; KW waves own the same rows and take different blocks of 32
// keys of each tile, each with its own running maximum, and are joined at the
// end: few or short samples then still fill the card.
//
// Measured: causal lengths 6000, 4097, 1500, 257 (16 heads over 4, D 128) 237 us,
// 950 TFLOP/s of the 1190 that a large matrix product reaches: the matrix cores (53 %
// of their cycles), with the vector unit's exponentials beside them (48 %). 16 samples of 231 .. 256 tokens with a bias
// (12 heads, D 32) 17 us: the bias, 23 MB, and the few tiles of a workgroup, whose
// first loads nothing hides. One token each of 16 samples over 8192 .. 1 keys (32
// heads over 8, D 128) 46 us, 35 of them this kernel's and 4 the join's: the keys
// and values, 148 MB.
#include <math.h>

#include "nt_attention_tile.hpp"
#include "nt_internal.hpp"

namespace nt {
namespace {

constexpr int kAtThreads = 256;

struct AtArgs {
  const int64_t *eta, *mu, *cell0;
  const int32_t *rows, *cols;
  int64_t cells, slots, ld_q, ld_k, ld_v;
  int64_t part_rows;  // split keys: rows of one split's partial results
  int B, H, K, D, splits, chunk;
  float scale;
  const void *q, *k, *v, *bias;
  void* o;
  float* lse;
  float *part_o, *part_ml;
};

// The base of a row's powers, in powers of two: its running maximum times the
// scores' unit, rounded. Without a bias the unit carries the scale, the powers are
// formed from unrounded products less this number, and whatever brings two bases
// together (a move, the waves' join) takes the difference of the rounded ones:
// beside scores of 10^5 the unrounded difference is off by up to 2^-7.
__device__ __forceinline__ float at_base(float most, float unit) {
#pragma clang fp contract(off)
  return most * unit;
}

template <typename T, int DP, int QW, int KW, int NB, bool BIAS, bool CAUSAL>
__global__ __launch_bounds__(kAtThreads, sizeof(T) == 4 && (DP > 64 || BIAS) ? 1 : 2) void k_attention(
    AtArgs a) {
  static_assert(64 * QW * KW == kAtThreads, "four waves");
  constexpr int KS = DP / 16, DT = DP / 32;
  constexpr int ROWS = 32 * QW, KEYS = 32 * KW * NB;  // of a workgroup; of a tile
  typedef typename AtFrag<T>::type Frag;
  typedef AtLoad<T, KEYS, DP, kAtThreads> Load;
  constexpr int TILE = KEYS * AtTile<T, DP>::pitch, kPair = 2 * TILE * (int)sizeof(T);
  // Tiles in flight: two where three pairs of tiles leave room for a second
  // workgroup on the CU (160 KB), else one.
  constexpr int AHEAD = !BIAS && 3 * kPair <= 80 * 1024 ? 2 : 1, BUFS = AHEAD + 1;
  constexpr int kLds = BUFS * kPair, kJoin = (KW - 1) * QW * (DP / 2 + 2) * 64 * 4;
  // Operations behind a tile's own loads when it is needed: the next tile's.
  constexpr int BEHIND = (AHEAD - 1) * 2 * Load::kPieces;
  typedef AtBiasTile<T, ROWS, KEYS, kAtThreads> Bias;
  __shared__ __align__(16) char lds_bytes[kLds > kJoin ? kLds : kJoin];
  __shared__ __align__(16) T lds_bias[BIAS ? BUFS * ROWS * KEYS : 1];
  const T* lds = reinterpret_cast<const T*>(lds_bytes);
  const uint32_t lds_at = at_lds(lds_bytes);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l32 = lane & 31, h = lane >> 5;
  const int qw = wave / KW, kw = wave % KW;
  // Key heads fastest: with 8 of them (or 4, 16 ..) an XCD, which takes every
  // eighth workgroup, stays with its own heads' keys, and all heads advance
  // together. Tiles in reverse, so that a causal sample's longest rows begin
  // first and the short ones fill the end.
  const int hk = blockIdx.x % a.K;
  const int64_t all = blockIdx.x / a.K;
  const int split = (int)((uint32_t)all / (uint32_t)a.slots);
  const int64_t slot = a.slots - 1 - (uint32_t)all % (uint32_t)a.slots;
  const int G = a.H / a.K;
  const int i = at_sample_of(a.eta, a.B, G, ROWS, slot);
  const int64_t tile = slot - (a.eta[i] * G / ROWS + i);
  const int64_t n = a.rows[i], m = a.cols[i];
  if (tile * ROWS >= n * G) return;

  // this lane's row
  const int64_t vr = tile * ROWS + qw * 32 + l32;
  const bool live = vr < n * G;
  const int64_t r = (live ? vr : n * G - 1) / G;
  const int hq = hk * G + (int)((live ? vr : n * G - 1) % G);
  const int64_t t = a.eta[i] + r;
  const int64_t seen64 = CAUSAL ? r + 1 + m - n : m;
  const int64_t seen = seen64 < 0 ? 0 : seen64 < m ? seen64 : m;
  // keys of this split, up to the last that a row of the workgroup sees
  int64_t c1 = m;
  if (CAUSAL) {
    const int64_t vlast = tile * ROWS + ROWS - 1;
    const int64_t rl = (vlast < n * G ? vlast : n * G - 1) / G;
    c1 = rl + 1 + m - n;
    c1 = c1 < 0 ? 0 : c1 < m ? c1 : m;
  }
  int64_t c0 = 0;
  if (a.splits > 1) {
    int64_t per = ((c1 + a.splits - 1) / a.splits + KEYS - 1) / KEYS * KEYS;
    per = per < a.chunk ? a.chunk : per;
    c0 = split * per < c1 ? split * per : c1;
    c1 = c0 + per < c1 ? c0 + per : c1;
    if (c0 == c1 && split > 0) {
      if (live && kw == 0 && h == 0) {
        float* ml = a.part_ml + ((int64_t)split * a.part_rows + t * a.H + hq) * 2;
        ml[0] = -INFINITY;
        ml[1] = 0.0f;
      }
      return;
    }
  }
  const int keys = (int)m, last = (int)seen;
  // the fewest keys that a row of this wave sees: no masks below it
  const int seen0 = __builtin_amdgcn_readfirstlane(last);

  // queries as fragments; the scale's sign goes with them
  Frag q[KS];
  const T* qp = static_cast<const T*>(a.q) + t * a.ld_q + (int64_t)hq * a.D;
  // (and a scale of zero is one of zero queries)
  const float scale = a.scale == 0.0f ? 1.0f : fabsf(a.scale);
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    q[s] = Frag{};
    if (16 * s + 8 * h < a.D && a.scale != 0.0f) q[s] = at_row(qp, s, h);
    if (a.scale < 0.0f) q[s] = -q[s];
  }
  const T* kp = static_cast<const T*>(a.k) + a.mu[i] * a.ld_k + (int64_t)hk * a.D;
  const T* vp = static_cast<const T*>(a.v) + a.mu[i] * a.ld_v + (int64_t)hk * a.D;

  f32x16 o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) o[d] = f32x16{};
  float most = -INFINITY, sum = 0.0f;  // of this row; sum: this half's keys
  const float unit = BIAS ? 1.0f : scale * kLog2e;
  const float step = BIAS ? kLog2e : unit;  // a score's unit in powers of two
  const Load load_k(a.ld_k), load_v(a.ld_v);
  // The bias: tile j's cells are loaded BUFS tiles ahead and put into LDS one
  // ahead, so that a wait for them leaves the loads of the tiles between.
  Bias biases[BUFS];
  const T* cells[Bias::kPieces];
  int cells_left = keys - (int)c0;
  if (BIAS) {
#pragma unroll
    for (int u = 0; u < Bias::kPieces; ++u) {
      const int64_t x = tile * ROWS + Bias::row(u) < n * G ? tile * ROWS + Bias::row(u) : n * G - 1;
      cells[u] = static_cast<const T*>(a.bias) + (hk * G + x % G) * a.cells + a.cell0[i] +
                 x / G * m + c0 + Bias::col(u);
    }
  }
  auto load_bias = [&](Bias& to_load) {
    to_load.load(cells, cells_left);
#pragma unroll
    for (int u = 0; u < Bias::kPieces; ++u) cells[u] += KEYS;
    cells_left -= KEYS;
  };
  const int mine = 32 * kw * NB;  // this wave's first key in a tile
  const int tiles = (int)((c1 - c0 + KEYS - 1) / KEYS);
  kp += c0 * a.ld_k;
  vp += c0 * a.ld_v;
  int left = keys - (int)c0, to = 0;  // keys from the tile to load on; its buffer
  auto start = [&]() {
    load_k.start(kp, a.ld_k, left, a.D, lds_at + to * kPair);
    load_v.start(vp, a.ld_v, left, a.D, lds_at + to * kPair + kPair / 2);
    kp += KEYS * a.ld_k;
    vp += KEYS * a.ld_v;
    left -= KEYS;
    to = to + 1 == BUFS ? 0 : to + 1;
  };
#pragma unroll
  for (int j = 0; j < AHEAD; ++j)
    if (j < tiles) start();
  if (BIAS) {
#pragma unroll
    for (int j = 0; j < BUFS; ++j)
      if (j < tiles) load_bias(biases[j]);
    if (tiles > 0) biases[0].put(lds_bias);
  }
  int c = (int)c0;
  auto tile_step = [&](int j, auto index) {
    constexpr int buf = decltype(index)::value;
    if (j + AHEAD - 1 < tiles) at_arrive<BEHIND>();
    else at_arrive<0>();
    if (BIAS && j + 1 < tiles)
      biases[(buf + 1) % BUFS].put(lds_bias + (buf + 1) % BUFS * ROWS * KEYS);
    if (j + AHEAD < tiles) start();
    if (BIAS && j + BUFS < tiles) load_bias(biases[buf]);
    // (the loads go out before the products: mixed with them by the compiler, long
    // causal 258 us, in this order 233)
    __builtin_amdgcn_sched_barrier(0);
    const T* lk = lds + buf * 2 * TILE;
    const T* lv = lk + TILE;
    f32x16 s[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      s[b] = f32x16{};
#pragma unroll
      for (int x = 0; x < KS; ++x)
        s[b] = at_mma(at_along<DP>(lk, mine + 32 * b + l32, x, h), q[x], s[b]);
    }
    if (BIAS) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const auto z = at_cells<KEYS>(lds_bias + buf * ROWS * KEYS, 32 * qw + l32,
                                        mine + 32 * b + 8 * y + 4 * h);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[b][4 * y + e] = s[b][4 * y + e] * scale + to_f32((T)z[e]);
        }
    }
    if (c + KEYS > (CAUSAL ? seen0 : keys)) {
      at_rare();
      const int left = last - c - mine - 4 * h;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int x = 0; x < 16; ++x)
          if (32 * b + 8 * (x / 4) + x % 4 >= left) s[b][x] = -INFINITY;
    }
    float top = s[0][0];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int x = 0; x < 16; ++x) top = fmaxf(top, s[b][x]);
    top = at_halves_max(top);
    // The base of a row's powers moves when its maximum has outgrown it by 2^8,
    // not at every new maximum: until then the powers stay below 2^8, which costs
    // neither bf16 nor fp32 any precision, and the sums carry the same base. (Of 32
    // rows one has a new maximum in most of the first 30 tiles, and moving scales
    // all of o: 16 D / 32 products a lane.)
    if (__any((top - most) * step > 8.0f)) {
      at_rare();
      const float now = fmaxf(most, top);
      const float moved = BIAS ? (most - now) * step : at_base(most, step) - at_base(now, step);
      const float keep = now == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(moved);
      most = now;
      sum *= keep;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int x = 0; x < 16; ++x) o[d][x] *= keep;
    }
    const float base = most == -INFINITY ? 0.0f : most;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const float p = BIAS ? __builtin_amdgcn_exp2f((s[b][x] - base) * kLog2e)
                             : __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][x], unit, -at_base(base, unit)));
        s[b][x] = p;
        sum += p;
      }
#pragma unroll
    for (int x = 0; x < 2 * NB; ++x) {
      Frag p;
      at_pack(s[x / 2], 8 * (x % 2), p);
#pragma unroll
      for (int d = 0; d < DT; ++d)
        o[d] = at_mma(at_across<DP>(lv, mine + 16 * x, 32 * d), p, o[d]);
    }
    c += KEYS;
  };
  at_each<BUFS>(tiles, tile_step);
  sum += __shfl_xor(sum, 32);
  if (KW > 1) {  // the waves of the same rows, in order, at their common maximum
    __syncthreads();
    float* join = reinterpret_cast<float*>(lds_bytes);
    constexpr int kPart = (16 * DT + 2) * 64;
    if (kw > 0) {
      float* p = join + ((kw - 1) * QW + qw) * kPart + lane;
      p[0] = most;
      p[64] = sum;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int x = 0; x < 16; ++x) p[(2 + 16 * d + x) * 64] = o[d][x];
    }
    __syncthreads();
    if (kw > 0) return;
    float now = most;
#pragma unroll
    for (int w = 1; w < KW; ++w) now = fmaxf(now, join[((w - 1) * QW + qw) * kPart + lane]);
    const float base = now == -INFINITY ? 0.0f : now;
    auto keep_of = [&](float x) {
      return __builtin_amdgcn_exp2f(BIAS ? (x - base) * step : at_base(x, step) - at_base(base, step));
    };
    float keep = keep_of(most);
    sum *= keep;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int x = 0; x < 16; ++x) o[d][x] *= keep;
#pragma unroll
    for (int w = 1; w < KW; ++w) {
      const float* p = join + ((w - 1) * QW + qw) * kPart + lane;
      keep = keep_of(p[0]);
      sum += p[64] * keep;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int x = 0; x < 16; ++x) o[d][x] += p[(2 + 16 * d + x) * 64] * keep;
    }
    most = now;
  }
  if (!live) return;
  const int64_t at = t * a.H + hq;
  // what the rounding of its base adds to a row's powers, as a power of two
  const float added = BIAS || most == -INFINITY ? 0.0f : __builtin_fmaf(most, step, -at_base(most, step));
  if (a.splits > 1) {
    const float keep = __builtin_amdgcn_exp2f(-added);
    float* po = a.part_o + ((int64_t)split * a.part_rows + at) * a.D;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        if (32 * d + 8 * g + 4 * h < a.D)
          at_store4(po + 32 * d + 8 * g + 4 * h, o[d][4 * g] * keep, o[d][4 * g + 1] * keep,
                    o[d][4 * g + 2] * keep, o[d][4 * g + 3] * keep);
    if (h == 0) {
      float* ml = a.part_ml + ((int64_t)split * a.part_rows + at) * 2;
      ml[0] = most;
      ml[1] = sum * keep;
    }
    return;
  }
  const float inv = sum > 0.0f ? 1.0f / sum : 1.0f;
  T* op = static_cast<T*>(a.o) + at * a.D;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      if (32 * d + 8 * g + 4 * h < a.D)
        at_store4(op + 32 * d + 8 * g + 4 * h, o[d][4 * g] * inv, o[d][4 * g + 1] * inv,
                  o[d][4 * g + 2] * inv, o[d][4 * g + 3] * inv);
  if (h == 0) a.lse[at] = (BIAS ? most : most * scale) + (logf(sum) - added * kLn2);
}

// Joins the splits of a row: a wave for each. The lanes first hold the splits'
// maxima (of scores that `scale` is still to multiply) and sums (at most 64), then
// the dimensions, two each.
template <typename T>
__global__ __launch_bounds__(256) void k_attention_join(const float* part_o, const float* part_ml,
                                                        int splits, int64_t rows, int D, float scale,
                                                        T* o, float* lse) {
  const int lane = threadIdx.x & 63;
  for (int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); at < rows;
       at += (int64_t)gridDim.x * 4) {
    float most = -INFINITY, sum = 0.0f;
    if (lane < splits) {
      most = part_ml[(lane * rows + at) * 2];
      sum = part_ml[(lane * rows + at) * 2 + 1];
    }
    // splits behind the row's last key hold nothing
    const int used = 64 - __builtin_clzll(__ballot(sum != 0.0f) | 1);
    float top = most;
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
    const float w = lane < splits ? expf((most - (top == -INFINITY ? 0.0f : top)) * scale) : 0.0f;
    sum *= w;
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) sum += __shfl_xor(sum, x);
    float acc[2] = {0.0f, 0.0f};
    const int d0 = lane < D ? lane : 0, d1 = lane + 64 < D ? lane + 64 : 0;
    for (int s = 0; s < used; s += 8) {  // eight loads at a time
      float v[8][2];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float* p = part_o + ((s + u < used ? s + u : s) * rows + at) * D;
        v[u][0] = p[d0];
        v[u][1] = p[d1];
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (s + u < used) {
          const float ws = __shfl(w, s + u);
          acc[0] += ws * v[u][0];
          acc[1] += ws * v[u][1];
        }
      }
    }
    const float inv = sum > 0.0f ? 1.0f / sum : 1.0f;
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (lane + 64 * e < D) o[at * D + lane + 64 * e] = from_f32<T>(acc[e] * inv);
    if (lane == 0) lse[at] = top * scale + logf(sum);
  }
}

// How the waves of a workgroup are shared out, in how many parts the keys are
// split over workgroups, and the fewest keys of a part.
struct AtPlan {
  int qw, splits, chunk;
};
// Without a bias, workgroups of 128 rows read each tile of keys half as often as
// those of 64, and leave fewer of them: taken where there are 1,024 or more. 64 against
// 128 rows, bf16: 8 x 1,024 of D 32, 12 heads (864 workgroups of 128) 33 against 37 us,
// 16 heads (1,152) 47 against 44; 16 x 256 of D 64, 32 heads (1,536) 29 against 25; 8 x
// 1,024 of D 128, 16 heads (1,152) 103 against 86; causal 6000 .. 257 (D 128, 1,496) 293
// against 253, causal 2 x 4,096 (D 64, 1,056) 105 against 107. Wide heads would gain
// from fewer already (4 x 1,024 of D 128, 16 heads, 576 workgroups: 54 against 47), D 64
// not always (8 x 1,024, 8 heads, 576: 34 against 36).
//
// A split costs its partial sums (fp32, written and read) and a second launch,
// 5 us at least. Where a sample's rows fill half a tile of 64 or less (decoding)
// they are small beside the keys, and parts of about 512 keys also even out
// samples of different lengths; below that, parts as short as make 512
// workgroups. The launch holds twice the parts that the mean length fills, and
// those behind a sample's last key return: one row each of 16 samples of 8,192 ..
// 1 keys (32 heads over 8, D 128): 44 to 46 us; with 1,024 workgroups 46, 2,048: 50;
// with four times the mean's parts 48, once 69. 64 such samples: 133 us, unsplit
// 191; 256: 494. One of 8,192 keys: 20. The mean length decides: 16 of 512 keys take 15
// us, unsplit 13, of 700 keys 17 and 16; one of 16,384 keys among 63 of 200 is not split
// (mean 453) and takes 204.
// With more rows only few workgroups over many keys gain, from about 1,536 keys on: 256
// rows (D 64, 8 heads) over 1,000 keys 14 us either way, over 1,536 17 -> 15, 2,048 22 ->
// 16, 8,192 73 -> 21; 500 rows (D 128, 8 heads) over 1,536 24 either way, 3,000 41 -> 27;
// 1,000 over 1,000 (D 32, 12 heads) would go 12 -> 18. 1,600 over 1,600 (6 heads) loses,
// 16 -> 19.
AtPlan plan_of(const nt_partition& p, const nt_attention& a) {
  if (p.T == 0 || p.B == 0) return {4, 1, 0};
  const int G = a.heads / a.kv_heads;
  auto groups = [&](int qw) { return at_slots(p.T, p.B, G, 32 * qw) * a.kv_heads; };
  const int qw = groups(4) >= 1024 ? 4 : 2;
  const int64_t keys = p.T_cols / p.B;
  const bool few = p.T * G <= 32 * (int64_t)p.B;
  int64_t s = 1, chunk = 0;
  if (keys >= 512 && (few ? groups(qw) < 4096 : groups(qw) <= 192 && p.T_cols >= 1536)) {
    chunk = (keys * groups(qw) / 512 + 63) / 64 * 64;
    const int64_t most = keys / 4 > 512 ? keys / 4 : 512;
    if (few && chunk > most) chunk = most / 64 * 64;
    if (chunk < 128) chunk = 128;
    s = 2 * keys / chunk;
    if (s > 64) s = 64;
    if (s < 1) s = 1;
  }
  return {qw, (int)s, (int)(chunk < (1 << 30) ? chunk : 1 << 30)};
}

template <typename T, int DP, int QW, int KW, int NB, bool BIAS>
hipError_t run(const AtArgs& x, bool causal, hipStream_t stream) {
  const unsigned g = (unsigned)(x.slots * x.splits * x.K);
  if (causal) k_attention<T, DP, QW, KW, NB, BIAS, true><<<g, kAtThreads, 0, stream>>>(x);
  else k_attention<T, DP, QW, KW, NB, BIAS, false><<<g, kAtThreads, 0, stream>>>(x);
  return hipGetLastError();
}
template <typename T, int DP>
hipError_t run(const AtArgs& x, int qw, bool causal, hipStream_t stream) {
  if (x.bias) return run<T, DP, 2, 2, 1, true>(x, causal, stream);
  if (qw == 4) return run<T, DP, 4, 1, 2, false>(x, causal, stream);
  return run<T, DP, 2, 2, 1, false>(x, causal, stream);
}

template <typename T>
hipError_t forward(const nt_partition& p, const nt_attention& a, const AtArgs& x, int qw,
                   hipStream_t stream) {
  hipError_t e;
  if (a.head_dim <= 32) e = run<T, 32>(x, qw, a.causal, stream);
  else if (a.head_dim <= 64) e = run<T, 64>(x, qw, a.causal, stream);
  else if (a.head_dim <= 96) e = run<T, 96>(x, qw, a.causal, stream);
  else e = run<T, 128>(x, qw, a.causal, stream);
  if (e != hipSuccess || x.splits == 1) return e;
  const int64_t rows = p.T * a.heads, blocks = (rows + 3) / 4;
  k_attention_join<T><<<(unsigned)(blocks < (1 << 20) ? blocks : (1 << 20)), 256, 0, stream>>>(
      x.part_o, x.part_ml, x.splits, rows, a.head_dim,
      x.bias || a.scale == 0.0f ? 1.0f : fabsf(a.scale), static_cast<T*>(x.o), x.lse);
  return hipGetLastError();
}

}  // namespace

// A grid holds fewer than 2^32 threads an axis.
bool attention_fits(const nt_partition& p, const nt_attention& a) {
  const int64_t most = (int64_t(1) << 32) / kAtThreads;
  // the smallest tiles that any kernel here or of the gradients takes
  return at_slots(p.T, p.B, a.heads / a.kv_heads, 32) * plan_of(p, a).splits * a.kv_heads < most &&
         at_slots(p.T_cols, p.B, 1, 32) * a.kv_heads < most;
}

size_t attention_ws_bytes(const nt_partition& p, const nt_attention& a, nt_dtype) {
  const int s = plan_of(p, a).splits;
  if (s == 1) return 0;
  return (size_t)s * p.T * a.heads * (a.head_dim + 2) * sizeof(float);
}

hipError_t launch_attention(const nt_partition& p, const nt_attention& a, const void* q,
                            const void* k, const void* v, const void* bias, void* o, float* lse,
                            nt_dtype dtype, void* ws, hipStream_t stream) {
  if (p.T == 0) return hipSuccess;
  AtArgs x;
  x.eta = p.single_offsets;
  x.mu = p.col_offsets;
  x.cell0 = p.pair_offsets;
  x.rows = p.lengths;
  x.cols = p.col_lengths;
  x.cells = p.cells;
  x.ld_q = a.ld_q;
  x.ld_k = a.ld_k;
  x.ld_v = a.ld_v;
  x.part_rows = p.T * a.heads;
  x.B = p.B;
  x.H = a.heads;
  x.K = a.kv_heads;
  x.D = a.head_dim;
  const AtPlan plan = plan_of(p, a);
  const int qw = bias ? 2 : plan.qw;  // (the workspace's size does not depend on the bias)
  x.slots = at_slots(p.T, p.B, a.heads / a.kv_heads, 32 * qw);
  x.splits = plan.splits;
  x.chunk = plan.chunk;
  x.scale = a.scale;
  x.q = q;
  x.k = k;
  x.v = v;
  x.bias = bias;
  x.o = o;
  x.lse = lse;
  x.part_o = static_cast<float*>(ws);
  x.part_ml = x.part_o + (int64_t)x.splits * x.part_rows * a.head_dim;
  return dtype == NT_BF16 ? forward<bf16>(p, a, x, qw, stream)
                          : forward<float>(p, a, x, qw, stream);
}

}  // namespace nt
