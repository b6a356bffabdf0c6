// Embedding of tokens as singles, and its gradient by sorted tokens.
//
// Forward: out[t] = scale table[token t], 8 columns a lane; a lookup moves bytes
// and nothing else. Tokens below zero are absent (zeros), tokens that the table
// does not hold give NaN.
//
// Gradient: g_table[v] = scale sum over the places t of token v of g[t], in the
// places' order whatever the launch does (no atomics on values). Three kernels:
// 1. Sort. Each workgroup owns every W-th token of the vocabulary (W a power of two:
//    the frequent ones, which often stand together, are spread) and reads all
//    tokens (from cache: 4 bytes each): it counts those of the workgroups before it,
//    which is where its own go in the sorted order, and lists its own in order, so
//    one launch sorts without an exchange between workgroups. Its list is then
//    sorted by token in LDS counters, one set a wave.
// 2. Sums. The sorted places are cut into parts of equal length, so that a token
//    that is everywhere costs the sums no more than many rare ones (the sort is one
//    workgroup's then). A team of lanes
//    adds the rows of a part, 8 columns a lane, and writes a token's row at the
//    end of its run; runs that cross the part's ends go to the workspace. Workgroups
//    behind the parts' write the zeros of the tokens that no place holds, which is most
//    of what a large vocabulary moves (in the first kernel they kept the sums waiting:
//    67 us where this takes 49, 16,384 places over 50,021 tokens of 1,024, on one table's
//    gradient; on six of them in turn, which no cache holds, 58, of which this kernel 41
//    for 238 MB, 5.9 TB/s).
// 3. Join. The part where a crossing run begins adds its pieces in order.
// Few places over a small vocabulary (an alphabet) take one launch instead: a workgroup
// for each token and 64 columns lists the token's places and adds their rows.
#include <algorithm>

#include "nt_device.hpp"
#include "nt_internal.hpp"

namespace nt {
namespace {

constexpr int kTeThreads = 256;
constexpr int kTeSortThreads = 1024;
constexpr int kTeSortWaves = kTeSortThreads / 64;
constexpr int kTeRange = 512;       // most tokens of a workgroup
constexpr int kTeAhead = 8;         // rows in flight
constexpr int64_t kTeMostGrid = int64_t(1) << 20;
constexpr int64_t kTeZeroBlocks = 1024;  // four for each compute unit

template <typename T> __device__ __forceinline__ void te_load(const T* p, float* f);
template <> __device__ __forceinline__ void te_load<bf16>(const bf16* p, float* f) {
  const bf16x8 v = *reinterpret_cast<const bf16x8*>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = (float)v[i];
}
template <> __device__ __forceinline__ void te_load<float>(const float* p, float* f) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = a[i];
    f[4 + i] = b[i];
  }
}
__device__ __forceinline__ void te_store(bf16* p, const float* f) {
  bf16x8 v;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (bf16)f[i];
  *reinterpret_cast<bf16x8*>(p) = v;
}
__device__ __forceinline__ void te_store(float* p, const float* f) {
  *reinterpret_cast<f32x4*>(p) = f32x4{f[0], f[1], f[2], f[3]};
  *reinterpret_cast<f32x4*>(p + 4) = f32x4{f[4], f[5], f[6], f[7]};
}

template <typename T, int LANES>
__global__ __launch_bounds__(kTeThreads) void k_te_lookup(const T* table, const int32_t* tokens,
                                                          T* out, int64_t n, int64_t V, int C,
                                                          float scale) {
  constexpr int kTeams = kTeThreads / LANES;
  for (int64_t t = (int64_t)blockIdx.x * kTeams + threadIdx.x / LANES; t < n;
       t += (int64_t)gridDim.x * kTeams) {
    const int64_t token = tokens[t];
    const bool is = token >= 0 && token < V;
    const float other = token < 0 ? 0.0f : __builtin_nanf("");
    const T* from = table + (is ? token : 0) * C;
    for (int c = threadIdx.x % LANES * 8; c < C; c += LANES * 8) {
      float f[8];
      te_load(from + c, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = is ? f[e] * scale : other;
      te_store(out + t * C + c, f);
    }
  }
}

struct TeSorted {
  int2* list;       // a workgroup's places and its number of their tokens, in order
  int32_t* place;   // sorted
  int32_t* token;   // of each sorted place
  int64_t* count;   // of places that hold a token of the table
  uint8_t* held;    // whether a place holds each token
};

__global__ __launch_bounds__(kTeSortThreads) void k_te_sort(const int32_t* tokens, int64_t n,
                                                            int64_t V, int shift, TeSorted s) {
  __shared__ int64_t below[kTeSortWaves], inside[kTeSortWaves];
  __shared__ int32_t counts[kTeSortWaves][kTeRange];
  __shared__ int32_t sums[kTeSortWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // its tokens are blockIdx.x + (k << shift), k below `have`
  const uint32_t mask = (1u << shift) - 1, mine = blockIdx.x, all_tokens = (uint32_t)V;
  const uint32_t have = (all_tokens - mine + mask) >> shift;
  for (int k = threadIdx.x; k < kTeSortWaves * kTeRange; k += kTeSortThreads) (&counts[0][0])[k] = 0;
  // A wave takes a stretch of the places, 4 neighbouring ones a lane at a time; absent
  // tokens are large unsigned numbers.
  const int64_t each = ((n + kTeSortWaves - 1) / kTeSortWaves + 255) / 256 * 256;
  const int64_t begin = std::min<int64_t>(n, wave * each), end = std::min<int64_t>(n, begin + each);
  const auto load = [&](int64_t i, uint32_t (&x)[4]) {
    if (i + 4 <= end) {
      __builtin_memcpy(x, tokens + i, 16);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = i + e < end ? (uint32_t)tokens[i + e] : 0xffffffffu;
    }
  };
  int under = 0, own = 0;
  for (int64_t i = begin + 4 * lane; i < end; i += 1024) {
    uint32_t x[4][4];
#pragma unroll
    for (int u = 0; u < 4; ++u) load(i + 256 * u, x[u]);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        under += x[u][e] < all_tokens && (x[u][e] & mask) < mine;
        own += x[u][e] < all_tokens && (x[u][e] & mask) == mine;
      }
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    under += __shfl_xor(under, m);
    own += __shfl_xor(own, m);
  }
  if (lane == 0) {
    below[wave] = under;
    inside[wave] = own;
  }
  __syncthreads();
  int64_t base = 0, total = 0, at = 0;
  for (int w = 0; w < kTeSortWaves; ++w) {
    base += below[w];
    if (w < wave) at += inside[w];
    total += inside[w];
  }
  if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) *s.count = base + total;
  for (int64_t i0 = begin; own && i0 < end; i0 += 1024) {
    const int64_t i = i0 + 4 * lane;
    uint32_t x[4][4];
#pragma unroll
    for (int u = 0; u < 4; ++u) load(i + 256 * u, x[u]);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      // behind the matches of the lanes before this one, then its own in order
      int place = 0, all = 0;
      bool is[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        is[e] = x[u][e] < all_tokens && (x[u][e] & mask) == mine;
        const unsigned long long who = __ballot(is[e]);
        place += __popcll(who & ((1ull << lane) - 1));
        all += __popcll(who);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (is[e])
          s.list[base + at + place++] =
              make_int2((int)(i + 256 * u + e), (int)(x[u][e] >> shift));
      at += all;
    }
  }
  __syncthreads();
  // how often each wave's stretch of the list holds each token
  const int64_t part = (total + kTeSortWaves - 1) / kTeSortWaves;
  const int64_t l0 = std::min<int64_t>(total, wave * part), l1 = std::min<int64_t>(total, l0 + part);
  for (int64_t i = l0 + lane; i < l1; i += 64 * kTeAhead) {
    int x[kTeAhead];
#pragma unroll
    for (int u = 0; u < kTeAhead; ++u) x[u] = i + 64 * u < l1 ? s.list[base + i + 64 * u].y : 0;
#pragma unroll
    for (int u = 0; u < kTeAhead; ++u)
      if (i + 64 * u < l1) atomicAdd(&counts[wave][x[u]], 1);
  }
  __syncthreads();
  // the first place of each token and wave: a token a thread, then over the tokens
  int all = 0;
  if (threadIdx.x < kTeRange)
    for (int w = 0; w < kTeSortWaves; ++w) all += counts[w][threadIdx.x];
  int before = all;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const int y = __shfl_up(before, m);
    if (lane >= m) before += y;
  }
  if (lane == 63) sums[wave] = before;
  __syncthreads();
  before -= all;
  for (int w = 0; w < wave; ++w) before += sums[w];
  if (threadIdx.x < kTeRange)
    for (int w = 0; w < kTeSortWaves; ++w) {
      const int x = counts[w][threadIdx.x];
      counts[w][threadIdx.x] = before;
      before += x;
    }
  if (threadIdx.x < have) s.held[mine + ((int64_t)threadIdx.x << shift)] = all != 0;
  __syncthreads();
  // places of equal tokens keep their order: the wave's next place of the token,
  // and behind it one for each earlier lane with the same token
  for (int64_t i = l0; i < l1; i += 64 * kTeAhead) {
    int2 ahead[kTeAhead];
#pragma unroll
    for (int u = 0; u < kTeAhead; ++u)
      ahead[u] = i + 64 * u + lane < l1 ? s.list[base + i + 64 * u + lane] : make_int2(0, 0);
#pragma unroll
    for (int u = 0; u < kTeAhead; ++u) {
      if (i + 64 * u >= l1) break;
      const bool is = i + 64 * u + lane < l1;
      const int2 x = ahead[u];
      unsigned long long same = __ballot(is);
#pragma unroll
      for (int b = 0; b < 9; ++b) {
        const unsigned long long one = __ballot(x.y >> b & 1);
        same &= x.y >> b & 1 ? one : ~one;
      }
      if (is) {
        const int rank = __popcll(same & ((1ull << lane) - 1));
        const int to = counts[wave][x.y] + rank;
        s.place[base + to] = x.x;
        s.token[base + to] = (int)(mine + ((uint32_t)x.y << shift));
      }
      __builtin_amdgcn_wave_barrier();
      if (is && same >> lane == 1) counts[wave][x.y] += __popcll(same);
      __builtin_amdgcn_wave_barrier();
    }
  }
}

template <typename T> struct TeSums {
  const T* g;
  float* g_table;
  float* pieces;          // [2 parts][C]: of the run that a part begins with, and ends with
  const int32_t* place;
  const int32_t* token;
  const int64_t* count;
  const uint8_t* held;
  int64_t parts, V;
  int part, C, accumulate;
  int blocks;             // workgroups of the sums; the ones behind them write zeros
  float scale;
};

template <typename T>
__device__ __forceinline__ void te_row(const TeSums<T>& p, int64_t token, int c, float* f) {
  float* to = p.g_table + token * p.C + c;
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] *= p.scale;
  if (p.accumulate) {
    float old[8];
    te_load<float>(to, old);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] += old[e];
  }
  te_store(to, f);
}

// Zeros in the rows of tokens that no place holds, a wave a row.
template <typename T> __device__ __forceinline__ void te_zeros(const TeSums<T>& p) {
  const int64_t step = (int64_t)(gridDim.x - p.blocks) * (kTeThreads / 64);
  for (int64_t v = (int64_t)(blockIdx.x - p.blocks) * (kTeThreads / 64) + threadIdx.x / 64; v < p.V;
       v += step)
    if (!p.held[v])
      for (int c = (threadIdx.x & 63) * 4; c < p.C; c += 256)
        *reinterpret_cast<f32x4*>(p.g_table + v * p.C + c) = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
}

template <typename T, int LANES>
__global__ __launch_bounds__(kTeThreads) void k_te_sums(TeSums<T> p) {
  if ((int)blockIdx.x >= p.blocks) {
    if (blockIdx.y == 0) te_zeros(p);
    return;
  }
  const int64_t k = (int64_t)blockIdx.x * (kTeThreads / LANES) + threadIdx.x / LANES;
  const int c = (int)(blockIdx.y * LANES + threadIdx.x % LANES) * 8;
  const int64_t n = *p.count, begin = k * p.part;
  if (k >= p.parts || begin >= n || c >= p.C) return;
  const int64_t end = begin + p.part < n ? begin + p.part : n;
  const int before = begin ? p.token[begin - 1] : -1, after = end < n ? p.token[end] : -1;
  float sum[8] = {};
  int now = p.token[begin];
  bool first = true;  // the run that the part begins with
  for (int64_t i = begin; i < end; i += kTeAhead) {
    float f[kTeAhead][8];
    int token[kTeAhead];
#pragma unroll
    for (int u = 0; u < kTeAhead; ++u) {
      const int64_t at = i + u < end ? i + u : end - 1;
      token[u] = p.token[at];
      te_load<T>(p.g + (int64_t)p.place[at] * p.C + c, f[u]);
    }
#pragma unroll
    for (int u = 0; u < kTeAhead; ++u) {
      if (i + u >= end) break;
      if (token[u] != now) {
        if (first && now == before)
          te_store(p.pieces + 2 * k * p.C + c, sum);
        else
          te_row(p, now, c, sum);
        first = false;
        now = token[u];
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += f[u][e];
    }
  }
  if (first && now == before)
    te_store(p.pieces + 2 * k * p.C + c, sum);
  else if (now == after)
    te_store(p.pieces + (2 * k + 1) * p.C + c, sum);
  else
    te_row(p, now, c, sum);
}

// A workgroup for each part: where a run begins in it and goes on behind it, the
// run's pieces are added, a stretch of them a team, then the teams' sums.
template <typename T, int LANES>
__global__ __launch_bounds__(kTeThreads) void k_te_join(TeSums<T> p) {
  constexpr int kTeams = kTeThreads / LANES;
  __shared__ float all[kTeams][LANES * 8];
  const int64_t k = blockIdx.x, n = *p.count, begin = k * p.part, end = begin + p.part;
  if (end >= n) return;
  const int now = p.token[end - 1];
  if (p.token[end] != now || (begin && p.token[begin - 1] == now)) return;
  // the last part that begins with the run's token, 64 parts looked at at once
  int64_t last = k + 1;
  for (;;) {
    const int64_t next = last + 1 + (threadIdx.x & 63);
    const bool on = next < p.parts && next * p.part < n && p.token[next * p.part] == now;
    const int more = __popcll(__ballot(on));
    last += more;
    if (more < 64) break;
  }
  const int64_t pieces = last - k + 1;
  const int team = threadIdx.x / LANES, c = (int)(blockIdx.y * LANES + threadIdx.x % LANES) * 8;
  const int64_t each = (pieces + kTeams - 1) / kTeams;
  const int64_t from = k + team * each, to = from + each < last + 1 ? from + each : last + 1;
  float sum[8] = {};
  if (c < p.C)
    for (int64_t i = from; i < to; i += kTeAhead) {
      float f[kTeAhead][8];
#pragma unroll
      for (int u = 0; u < kTeAhead; ++u) {
        const int64_t at = i + u < to ? i + u : to - 1;
        te_load<float>(p.pieces + (2 * at + (at == k)) * p.C + c, f[u]);
      }
#pragma unroll
      for (int u = 0; u < kTeAhead; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += i + u < to ? f[u][e] : 0.0f;
    }
  te_store(&all[team][threadIdx.x % LANES * 8], sum);
  __syncthreads();
  if (team || c >= p.C) return;
  for (int w = 1; w < kTeams; ++w)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] += all[w][threadIdx.x % LANES * 8 + e];
  te_row(p, now, c, sum);
}

// A token v and 64 columns a workgroup: the places of v in order, in LDS, as many as it
// holds at a time; then 32 teams of 8 lanes add every 32nd of them, and the teams' sums
// are added in order.
constexpr int kTePlaces = 4096;
template <typename T>
__global__ __launch_bounds__(kTeThreads) void k_te_direct(const int32_t* tokens, const T* g,
                                                          float* g_table, int n, int C,
                                                          float scale, int accumulate) {
  __shared__ int32_t places[kTePlaces];
  __shared__ int counts[kTeThreads / 64];
  __shared__ float all[32][65];
  const int v = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // each wave lists a stretch of the places: its count first, then they go behind the others'
  const int each = ((n + kTeThreads / 64 - 1) / (kTeThreads / 64) + 63) / 64 * 64;
  const int begin = min(n, wave * each), end = min(n, begin + each);
  int mine = 0;
  for (int i = begin; i < end; i += 512) {
    int x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) x[u] = i + 64 * u + lane < end ? tokens[i + 64 * u + lane] : -1;
#pragma unroll
    for (int u = 0; u < 8; ++u) mine += __popcll(__ballot(x[u] == v));
  }
  if (lane == 0) counts[wave] = mine;
  __syncthreads();
  int at = 0, total = 0;
  for (int w = 0; w < kTeThreads / 64; ++w) {
    if (w < wave) at += counts[w];
    total += counts[w];
  }
  for (int i = begin; mine && i < end; i += 64) {
    const bool is = i + lane < end && tokens[i + lane] == v;
    const unsigned long long who = __ballot(is);
    if (is) places[at + __popcll(who & ((1ull << lane) - 1))] = i + lane;
    at += __popcll(who);
  }
  __syncthreads();
  const int team = threadIdx.x / 8, c = (int)blockIdx.y * 64 + threadIdx.x % 8 * 8;
  float sum[8] = {};
  if (c < C)
    for (int i = team; i < total; i += 32 * 4) {
      float f[4][8];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        te_load(g + (int64_t)places[i + 32 * u < total ? i + 32 * u : i] * C + c, f[u]);
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += i + 32 * u < total ? f[u][e] : 0.0f;
    }
#pragma unroll
  for (int e = 0; e < 8; ++e) all[team][threadIdx.x % 8 * 8 + e] = sum[e];
  __syncthreads();
  // 64 columns x 4 stretches of teams, then those
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) s += all[8 * wave + k][lane];
  __syncthreads();
  all[wave][lane] = s;
  __syncthreads();
  const int column = (int)blockIdx.y * 64 + lane;
  if (wave || column >= C) return;
  s = (all[0][lane] + all[1][lane]) + (all[2][lane] + all[3][lane]);
  float* to = g_table + (int64_t)v * C + column;
  if (!accumulate)
    *to = s * scale;
  else if (total)
    *to += s * scale;
}

// One launch while the places fit LDS and there are at most 4,096 workgroups, each of which
// reads all tokens. In us on the GPU, here and by sorting (fp32): 2,272 places, 33 tokens and
// 384 columns 4.6 and 16.3, with 4,096 places 5.9 and 17.4, one token in all of them 13.9 and
// 28.4; at 4,000 or 4,096 workgroups, 4,096 places over 1,000 tokens of 256 14.7 and 18.5, over
// 4,096 of 64 13.1 and 20.3, 300 places 6.0 and 15.7. Beyond: 8,000 workgroups and 1,000 places
// 10.9 and 16.6, 16,000 17.6 and 17.0, 16,384 and 4,096 places 28.7 and 21.0, 64,000 and 300
// places 52 and 17.
bool direct(int64_t T, int64_t V, int C) {
  return T <= kTePlaces && V * ((C + 63) / 64) <= 4096;
}

__global__ __launch_bounds__(kTeThreads) void k_te_fill(f32x4* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * kTeThreads + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * kTeThreads)
    p[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
}

template <int LANES> struct TeTeam {
  static constexpr int lanes = LANES;
};
// The team of a row of C columns, at most `MOST` lanes.
template <int MOST, typename Run> hipError_t te_teams(int C, const Run& run) {
  if (C <= 64) return run(TeTeam<8>());
  if (C <= 128) return run(TeTeam<16>());
  if (C <= 256) return run(TeTeam<32>());
  if (MOST == 64 || C <= 512) return run(TeTeam<64>());
  if (C <= 1024) return run(TeTeam<MOST < 128 ? MOST : 128>());
  return run(TeTeam<MOST>());
}

struct Plan {
  int64_t parts;
  int part, shift;
  size_t list, place, token, count, held, pieces, total;
};

Plan plan_of(int64_t T, int64_t V, int C) {
  Plan p = {};
  // 16 places a part, more of them where that would be over 2,048 parts
  p.part = (int)std::max<int64_t>(16, (T + 2047) / 2048);
  p.parts = (T + p.part - 1) / p.part;
  // a workgroup for each compute unit, or more where one would have too many tokens
  p.shift = 8;
  while ((V >> p.shift) >= kTeRange) ++p.shift;
  size_t at = 0;
  p.list = at; at = align256(at + sizeof(int2) * T);
  p.place = at; at = align256(at + sizeof(int32_t) * T);
  p.token = at; at = align256(at + sizeof(int32_t) * T);
  p.count = at; at = align256(at + sizeof(int64_t));
  p.held = at; at = align256(at + V);
  p.pieces = at; at = align256(at + sizeof(float) * 2 * p.parts * C);
  p.total = at;
  return p;
}

template <typename T>
hipError_t lookup(const void* table, const int32_t* tokens, void* out, int64_t n, int64_t V, int C,
                  float scale, hipStream_t s) {
  return te_teams<256>(C, [&](auto team) {
    constexpr int L = decltype(team)::lanes;
    const int64_t rows = kTeThreads / L;
    const uint32_t grid = (uint32_t)std::min<int64_t>((n + rows - 1) / rows, kTeMostGrid);
    k_te_lookup<T, L><<<grid, kTeThreads, 0, s>>>(
        static_cast<const T*>(table), tokens, static_cast<T*>(out), n, V, C, scale);
    return hipGetLastError();
  });
}

template <typename T>
hipError_t backward(const int32_t* tokens, const void* g, float* g_table, int64_t n, int64_t V,
                    int C, float scale, bool accumulate, char* ws, hipStream_t s) {
  if (direct(n, V, C)) {
    k_te_direct<T><<<dim3((uint32_t)V, (uint32_t)((C + 63) / 64)), kTeThreads, 0, s>>>(
        tokens, static_cast<const T*>(g), g_table, (int)n, C, scale, accumulate);
    return hipGetLastError();
  }
  const Plan p = plan_of(n, V, C);
  const TeSorted sorted = {reinterpret_cast<int2*>(ws + p.list),
                           reinterpret_cast<int32_t*>(ws + p.place),
                           reinterpret_cast<int32_t*>(ws + p.token),
                           reinterpret_cast<int64_t*>(ws + p.count),
                           reinterpret_cast<uint8_t*>(ws + p.held)};
  k_te_sort<<<(uint32_t)std::min<int64_t>(V, int64_t(1) << p.shift), kTeSortThreads, 0, s>>>(
      tokens, n, V, p.shift, sorted);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  TeSums<T> a = {static_cast<const T*>(g), g_table, reinterpret_cast<float*>(ws + p.pieces),
                 sorted.place, sorted.token, sorted.count, sorted.held, p.parts, V, p.part, C,
                 accumulate, 0, scale};
  return te_teams<64>(C, [&](auto team) {
    constexpr int L = decltype(team)::lanes;
    const int64_t rows = kTeThreads / L;
    const uint32_t slices = (uint32_t)((C / 8 + L - 1) / L);
    a.blocks = (int)((p.parts + rows - 1) / rows);
    const int64_t zeros = accumulate ? 0 : std::min<int64_t>((V + 3) / 4, kTeZeroBlocks);
    k_te_sums<T, L><<<dim3((uint32_t)(a.blocks + zeros), slices), kTeThreads, 0, s>>>(a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || p.parts < 2) return err;
    k_te_join<T, L><<<dim3((uint32_t)(p.parts - 1), slices), kTeThreads, 0, s>>>(a);
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_token_embedding(const void* table, const int32_t* tokens, void* out, int64_t T,
                                  int64_t V, int C, float scale, nt_dtype dtype, hipStream_t s) {
  if (T == 0) return hipSuccess;
  return dtype == NT_BF16 ? lookup<bf16>(table, tokens, out, T, V, C, scale, s)
                          : lookup<float>(table, tokens, out, T, V, C, scale, s);
}

size_t token_embedding_backward_ws_bytes(int64_t T, int64_t V, int C) {
  return T && !direct(T, V, C) ? plan_of(T, V, C).total : 0;
}

hipError_t launch_token_embedding_backward(const int32_t* tokens, const void* g_out,
                                           float* g_table, int64_t T, int64_t V, int C,
                                           float scale, bool accumulate, nt_dtype dtype, void* ws,
                                           hipStream_t s) {
  if (T == 0) {  // nothing to add
    if (accumulate) return hipSuccess;
    const int64_t n = V * C / 4;
    k_te_fill<<<(uint32_t)std::min<int64_t>((n + kTeThreads - 1) / kTeThreads, 4096), kTeThreads, 0,
                s>>>(reinterpret_cast<f32x4*>(g_table), n);
    return hipGetLastError();
  }
  char* w = static_cast<char*>(ws);
  return dtype == NT_BF16
             ? backward<bf16>(tokens, g_out, g_table, T, V, C, scale, accumulate, w, s)
             : backward<float>(tokens, g_out, g_table, T, V, C, scale, accumulate, w, s);
}

}  // namespace nt
