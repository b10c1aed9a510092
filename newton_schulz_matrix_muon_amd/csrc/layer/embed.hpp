// Token embeddings: rows of a table looked up and scaled, and the table's gradient.
//
//   y[t]  = scale table[token[t]]
//   dT[v] = scale sum over the t with token[t] = v of dy[t]
//
// A token outside 0 .. V - 1 (padding) gives a row of zeros and adds to no gradient.
//
// The gradient is a dense table (the optimizer takes it as it is), summed without float atomics: the
// positions are sorted by token, ties by position, and cut into tiles of 32. A thread walks a tile
// for one 16-byte unit of columns and adds up rows of one token in order, in fp32; what lies within
// the tile goes to the table at once, the parts of a token that crosses a tile's end go to the
// workspace and are added up tile by tile, for many tiles of one token in two steps. The work is in
// proportion to the positions whatever their tokens. Equal calls give equal bits.
//
// Bound by HBM: dy is read once and the table, mostly zeros, written once. One MI355X: 16384 rows of 163840 x 7168
// bf16 looked up in 83 us (5.7 TB/s); the gradient of 8192 positions of that table 405 to 440 us in embed_grad at 5.6 to 6.1
// TB/s and 31 in the sort and the join; of 30011 positions of 8191 x 1021 fp32 30 us at 5.0 TB/s, and 30 in the rest.
#pragma once

#include "mx8.hpp"
#include "norm.hpp"

namespace mns {

// The token of position t, or -1.
template <typename ID>
__device__ inline int token_of(const void* tokens, int64_t t, int vocab) {
  const ID v = reinterpret_cast<const ID*>(tokens)[t];
  return v >= 0 && v < (ID)vocab ? (int)v : -1;
}

// 16 bytes of a row (V elements) or, in rows shorter than that, one element. Rows begin anywhere; a
// row's last unit ends with the row, so it shares elements with the one before, of the same value.
template <typename T, int V>
struct EmbedUnit {
  static __device__ inline int at(int u, int cols) { return V > 1 ? min(u * V, cols - V) : u; }
  u32x4 v;
  __device__ inline void load(const T* row, int c) {
    if constexpr (V > 1) v = *reinterpret_cast<const u32x4_any*>(row + c);
    else v[0] = __float_as_uint(as_f32(row[c]));
  }
  __device__ inline void unpack(float (&f)[V]) const {
    if constexpr (V == 8) VecIO<T>::unpack(v, f);
    else
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] = __uint_as_float(v[e]);
  }
  static __device__ inline void store(T* row, int c, const float (&f)[V]) {
    if constexpr (V == 8) {
      *reinterpret_cast<u32x4_any*>(row + c) = u32x4{pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7])};
    } else if constexpr (V == 4) {
      *reinterpret_cast<u32x4_any*>(row + c) = u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
    } else {
      row[c] = from_f32<T>(f[0]);
    }
  }
};

// Whole rows of the smallest units: (row, unit) of item first + x, where first = row0 * units + rest.
struct EmbedArgs {
  const char* table; int64_t table_ld;   // bytes per row
  char* y; int64_t y_ld;
  const void* tokens;
  int64_t n;                       // positions
  int vocab, cols, units;
  float scale;
};

template <typename T, typename ID, int V>
__global__ void __launch_bounds__(256) embed_rows(const EmbedArgs p) {
  const int64_t first = block_id() * 256;
  const int64_t t0 = first / p.units;
  const unsigned x = (unsigned)(first - t0 * p.units) + threadIdx.x;
  const unsigned q = x / (unsigned)p.units;
  const int64_t t = t0 + q;
  if (t >= p.n) return;
  const int c = EmbedUnit<T, V>::at((int)(x - q * (unsigned)p.units), p.cols);
  const int v = token_of<ID>(p.tokens, t, p.vocab);
  // padding reads row 0 and keeps nothing of it
  EmbedUnit<T, V> u;
  u.load(reinterpret_cast<const T*>(p.table + (int64_t)max(v, 0) * p.table_ld), c);
  float f[V];
  u.unpack(f);
#pragma unroll
  for (int e = 0; e < V; ++e) f[e] = v >= 0 ? f[e] * p.scale : 0.f;
  EmbedUnit<T, V>::store(reinterpret_cast<T*>(p.y + t * p.y_ld), c, f);
}

// ------------------------------------------------------------------------------------- sort
// Positions by token: a radix sort from the lowest digit up, stable, in passes of up to ten bits.
// Up to EMBED_ONE positions one workgroup takes every pass in one launch; more go in two launches a
// pass, counts and places, with one step of 64 positions a wave. A pass of one workgroup costs 3.6 us at
// 1024 positions, 7 at 4096, 11.5 at 8192 and 21 at 16384; one of two launches 10 to 12 us at any of
// these. The whole gradient (80 columns, 19478 rows, bf16): 30.7 us against 31.5 at 4096 positions, 36.0
// against 32.1 at 6000, 59.5 against 33.5 at 16384.
constexpr int EMBED_WAVES = 16, EMBED_NT = 64 * EMBED_WAVES;
constexpr int EMBED_DIGITS = 1024;
constexpr int64_t EMBED_ONE = 4096;

struct EmbedSortArgs {
  const void* tokens;
  int64_t n;
  int vocab;
  int bits, passes;                // per pass
  int steps;                       // 64-position steps per wave: a workgroup takes EMBED_NT * steps positions
  int nblocks;
  int2* sorted[2];                 // token (vocab: none) and position, after even and odd passes
  int32_t* hist;                   // [nblocks][EMBED_DIGITS]
  uint8_t* marks;                  // [vocab]: whether the token occurs
};

// A wave's positions of one pass, 64 at a time: digit -1 past the end. Held in registers from the counts to
// the places, and loaded together, so that a pass waits for memory once.
template <int STEPS>
struct EmbedRun {
  int key[STEPS], pos[STEPS], digit[STEPS];
};
template <typename ID, int STEPS>
__device__ inline void embed_load(const EmbedSortArgs& p, int pass, int64_t s0, EmbedRun<STEPS>& d) {
  const int from = (pass - 1) & 1;
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int64_t s = min(s0 + 64 * i, p.n - 1);
    if (pass == 0) {
      const int v = token_of<ID>(p.tokens, s, p.vocab);
      d.key[i] = v < 0 ? p.vocab : v;
      d.pos[i] = (int)s;
    } else {
      const int2 kp = p.sorted[from][s];
      d.key[i] = kp.x;
      d.pos[i] = kp.y;
    }
  }
#pragma unroll
  for (int i = 0; i < STEPS; ++i) d.digit[i] = s0 + 64 * i < p.n ? (d.key[i] >> (pass * p.bits)) & ((1 << p.bits) - 1) : -1;
}

// Each wave's positions by digit into at[wave].
template <int STEPS>
__device__ inline void embed_count(const EmbedRun<STEPS>& d, int (*at)[EMBED_DIGITS]) {
  const int wv = threadIdx.x >> 6;
#pragma unroll
  for (int w = 0; w < EMBED_WAVES; ++w) at[w][threadIdx.x] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < STEPS; ++i)
    if (d.digit[i] >= 0) atomicAdd(&at[wv][d.digit[i]], 1);
  __syncthreads();
}

// Counts in at to the places where each wave's digits begin: behind the smaller digits, and of one
// digit behind `before` of earlier workgroups and the earlier waves of this one. EMBED_NT threads,
// one digit each.
__device__ inline void embed_places(int total, int before, int (*at)[EMBED_DIGITS], int* scan) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, e = threadIdx.x;
  int run = total;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(run, o);
    if (lane >= o) run += v;
  }
  if (lane == 63) scan[wv] = run;
  __syncthreads();
  int next = run - total + before;
  for (int w = 0; w < wv; ++w) next += scan[w];
  for (int w = 0; w < EMBED_WAVES; ++w) {
    const int n = at[w][e];
    at[w][e] = next;
    next += n;
  }
  __syncthreads();
}

// The positions to their places: a wave ranks 64 at a time, equal digits by lane number.
template <int STEPS>
__device__ inline void embed_place(const EmbedSortArgs& p, int pass, const EmbedRun<STEPS>& d, int (*at)[EMBED_DIGITS]) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int digit = d.digit[i];
    uint64_t same = __ballot(digit >= 0);
    for (int b = 0; b < p.bits; ++b) {
      const uint64_t m = __ballot((digit >> b) & 1);
      same &= (digit >> b) & 1 ? m : ~m;
    }
    const int lead = __builtin_ctzll(same | (1ull << 63));
    int next = 0;
    if (digit >= 0 && lane == lead) next = atomicAdd(&at[wv][digit], __builtin_popcountll(same));
    next = __shfl(next, lead);
    if (digit >= 0) {
      const int to = next + __builtin_popcountll(same & ((1ull << lane) - 1));
      p.sorted[pass & 1][to] = int2{d.key[i], d.pos[i]};
      if (pass == 0 && d.key[i] < p.vocab) p.marks[d.key[i]] = 1;
    }
  }
}

// Every pass in one workgroup, and the marks. At least one position.
template <typename ID, int STEPS>
__global__ void __launch_bounds__(EMBED_NT) embed_sort_one(const EmbedSortArgs p) {
  __shared__ int at[EMBED_WAVES][EMBED_DIGITS];
  __shared__ int scan[EMBED_WAVES];
  // the workspace begins at a multiple of 16 bytes, and so do the marks, with room behind them
  for (int64_t i = (int64_t)threadIdx.x * 16; i < p.vocab; i += EMBED_NT * 16) *reinterpret_cast<u32x4*>(p.marks + i) = u32x4{0, 0, 0, 0};
  const int64_t s0 = (int64_t)(threadIdx.x >> 6) * 64 * STEPS + (threadIdx.x & 63);
  for (int pass = 0; pass < p.passes; ++pass) {
    EmbedRun<STEPS> d;
    embed_load<ID>(p, pass, s0, d);
    embed_count(d, at);
    int total = 0;
#pragma unroll
    for (int w = 0; w < EMBED_WAVES; ++w) total += at[w][threadIdx.x];
    embed_places(total, 0, at, scan);
    embed_place(p, pass, d, at);
    __syncthreads();
  }
}

// No position: every row of the table is zeros.
template <int NT>
__global__ void __launch_bounds__(NT) embed_no_marks(const EmbedSortArgs p) {
  const int64_t i = ((int64_t)blockIdx.x * NT + threadIdx.x) * 16;
  if (i < p.vocab) *reinterpret_cast<u32x4*>(p.marks + i) = u32x4{0, 0, 0, 0};
}

template <typename ID>
__global__ void __launch_bounds__(EMBED_NT) embed_sort_count(const EmbedSortArgs p, int pass) {
  __shared__ int at[EMBED_DIGITS];
  if (pass == 0)
    for (int64_t i = ((int64_t)blockIdx.x * EMBED_NT + threadIdx.x) * 16; i < p.vocab; i += (int64_t)gridDim.x * EMBED_NT * 16)
      *reinterpret_cast<u32x4*>(p.marks + i) = u32x4{0, 0, 0, 0};
  at[threadIdx.x] = 0;
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * EMBED_NT * p.steps;
  for (int i = 0; i < p.steps; ++i) {
    EmbedRun<1> d;
    embed_load<ID>(p, pass, lo + (int64_t)i * EMBED_NT + threadIdx.x, d);
    if (d.digit[0] >= 0) atomicAdd(&at[d.digit[0]], 1);
  }
  __syncthreads();
  p.hist[(int64_t)blockIdx.x * EMBED_DIGITS + threadIdx.x] = at[threadIdx.x];
}

// Every workgroup adds up the counts itself: all of them for the digits before, the earlier
// workgroups' for its own positions, a step of each wave at a time. 6 us for 8 workgroups, 9.5 for 64.
template <typename ID>
__global__ void __launch_bounds__(EMBED_NT) embed_sort_place(const EmbedSortArgs p, int pass) {
  __shared__ int at[EMBED_WAVES][EMBED_DIGITS];
  __shared__ int scan[EMBED_WAVES];
  const int64_t lo = (int64_t)blockIdx.x * EMBED_NT * p.steps;
  EmbedRun<1> d;
  embed_load<ID>(p, pass, lo + threadIdx.x, d);
  int total = 0, before = 0;
  for (int b0 = 0; b0 < p.nblocks; b0 += 16) {
    int n[16];
#pragma unroll
    for (int b = 0; b < 16; ++b) n[b] = b0 + b < p.nblocks ? p.hist[(int64_t)(b0 + b) * EMBED_DIGITS + threadIdx.x] : 0;
#pragma unroll
    for (int b = 0; b < 16; ++b) {
      total += n[b];
      before += b0 + b < (int)blockIdx.x ? n[b] : 0;
    }
  }
  for (int i = 0; i < p.steps; ++i) {
    if (i) embed_load<ID>(p, pass, lo + (int64_t)i * EMBED_NT + threadIdx.x, d);
    embed_count(d, at);
    int mine = 0;
#pragma unroll
    for (int w = 0; w < EMBED_WAVES; ++w) mine += at[w][threadIdx.x];
    embed_places(total, before, at, scan);
    embed_place(p, pass, d, at);
    before += mine;
    __syncthreads();
  }
}

// --------------------------------------------------------------------------------- gradient
// Positions of a tile: a thread has eight rows of a tile in flight. The next eight positions loaded ahead as well took
// 0.7 us off small calls and cost large ones 7 % (registers).
constexpr int EMBED_TILE = 32;

struct EmbedGradArgs {
  const char* dy; int64_t dy_ld;   // bytes per row
  char* dt; int64_t dt_ld;
  const int2* sorted;              // tokens (x) and positions (y)
  const uint8_t* marks;
  float* part;                     // [2 * tiles][cols]: a tile's part of the token that came in from the tile before, of the one that goes on
  int64_t n, tiles;
  bool gathered;                   // embed_gather ran
  int64_t tile_blocks, zero_blocks;
  int vocab, cols, units;
  float scale;
};

constexpr int EMBED_ZERO = 8;      // units of 256 threads a workgroup looks at for rows of zeros

template <typename T, int V>
__device__ inline void embed_zero(const EmbedGradArgs& p, int64_t block) {
  const int64_t first = block * 256 * EMBED_ZERO;
  const int64_t v0 = first / p.units;
  const unsigned rest = (unsigned)(first - v0 * p.units) + threadIdx.x;
  float zero[V];
#pragma unroll
  for (int e = 0; e < V; ++e) zero[e] = 0.f;
#pragma unroll
  for (int i = 0; i < EMBED_ZERO; ++i) {
    const unsigned x = rest + i * 256;
    const unsigned q = x / (unsigned)p.units;
    const int64_t v = v0 + q;
    if (v < p.vocab && !p.marks[v])
      EmbedUnit<T, V>::store(reinterpret_cast<T*>(p.dt + v * p.dt_ld), EmbedUnit<T, V>::at((int)(x - q * (unsigned)p.units), p.cols), zero);
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(256) embed_grad(const EmbedGradArgs p) {
  constexpr int U = 8;             // rows in flight
  const int64_t block = block_id();
  if (block >= p.tile_blocks) {
    if (block - p.tile_blocks < p.zero_blocks) embed_zero<T, V>(p, block - p.tile_blocks);
    return;
  }
  const int64_t first = block * 256;
  const int64_t k0 = first / p.units;
  const unsigned x = (unsigned)(first - k0 * p.units) + threadIdx.x;
  const unsigned q = x / (unsigned)p.units;
  const int64_t tile = k0 + q;
  if (tile >= p.tiles) return;
  const int c = EmbedUnit<T, V>::at((int)(x - q * (unsigned)p.units), p.cols);
  const int64_t lo = tile * EMBED_TILE, hi = min(lo + EMBED_TILE, p.n);
  const int after = hi < p.n ? p.sorted[hi].x : -1;
  int now = p.sorted[lo].x;
  bool came = lo > 0 && p.sorted[lo - 1].x == now;
  float acc[V];
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.f;
  // the sum of token `now` leaves: to the table if it lies within the tile, or as a part
  auto leave = [&](bool goes) {
    if (came || goes) {
      float* part = p.part + (2 * tile + (came ? 0 : 1)) * p.cols + c;
#pragma unroll
      for (int e = 0; e < V; ++e) part[e] = acc[e];
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] *= p.scale;
      EmbedUnit<T, V>::store(reinterpret_cast<T*>(p.dt + (int64_t)now * p.dt_ld), c, acc);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
    came = false;
  };
  for (int64_t s = lo; s < hi; s += U) {
    int2 at[U];
    EmbedUnit<T, V> row[U];
    // the rows behind the tile's end read the tile's last and are left out: no branch between the loads
#pragma unroll
    for (int u = 0; u < U; ++u) at[u] = p.sorted[min(s + u, hi - 1)];
#pragma unroll
    for (int u = 0; u < U; ++u) row[u].load(reinterpret_cast<const T*>(p.dy + (int64_t)at[u].y * p.dy_ld), c);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s + u >= hi) continue;
      if (at[u].x != now) {
        leave(false);
        now = at[u].x;
      }
      if (now >= p.vocab) return;  // sorted behind all tokens
      float f[V];
      row[u].unpack(f);
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += f[e];
    }
  }
  if (now < p.vocab) leave(now == after);
}

// Many tiles of one token: the parts of EMBED_GROUP tiles that lie within one token, added up into the first
// one's, so that embed_join has fewer to go through. Workgroup (group, 512 columns), each of its four waves
// a quarter of the tiles in turns of four. One token at all of 65536 positions of 1024 columns: 131 us
// without, 67 with; at 2^20 positions of 64 columns 1299 and 140; with tokens that occur alike 2 to 3 us more for
// the launch, which is why fewer groups go without.
constexpr int EMBED_GROUP = 64;
constexpr int64_t EMBED_GROUPS = 16;   // from so many groups on
__device__ inline void embed_load_parts(const EmbedGradArgs& p, int64_t tile, int64_t c0, float (&v)[8]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = p.part[2 * tile * p.cols + min(c0 + e * 64 + lane, (int64_t)p.cols - 1)];
}
// Sums of four waves in the first, in order.
__device__ inline void embed_meet(float (&acc)[8], float (*sum)[8][64]) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  if (wv)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[wv - 1][e][lane] = acc[e];
  __syncthreads();
  if (wv) return;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    for (int w = 0; w < 3; ++w) acc[e] += sum[w][e][lane];
}
template <int NT>
__global__ void __launch_bounds__(NT) embed_gather(const EmbedGradArgs p) {
  __shared__ float sum[3][8][64];
  const int64_t t0 = block_id() * EMBED_GROUP, t1 = t0 + EMBED_GROUP - 1;
  if (t0 == 0 || t1 >= p.tiles) return;
  const int token = p.sorted[t1 * EMBED_TILE].x;
  if (token >= p.vocab || p.sorted[t0 * EMBED_TILE - 1].x != token) return;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t c0 = (int64_t)blockIdx.z * 512;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int i = wv; i < EMBED_GROUP; i += 16) {
    float v[4][8];
#pragma unroll
    for (int u = 0; u < 4; ++u) embed_load_parts(p, t0 + i + 4 * u, c0, v[u]);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += v[u][e];
  }
  embed_meet(acc, sum);   // every load of the first tile's part has landed
  if (wv) return;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c0 + e * 64 + lane < p.cols) p.part[2 * t0 * p.cols + c0 + e * 64 + lane] = acc[e];
}

// A token that crosses ends of tiles: its parts added up in the tiles' order. Workgroup (end between
// two tiles, 512 columns) works where a token begins in the tile before the end and goes on behind it;
// its four waves take every fourth tile, or group of tiles that embed_gather has added up.
template <typename T>
__global__ void __launch_bounds__(256) embed_join(const EmbedGradArgs p) {
  __shared__ float sum[3][8][64];
  const int64_t a = block_id();    // the tile that it begins in
  if (a + 1 >= p.tiles) return;
  const int64_t hi = (a + 1) * EMBED_TILE;
  const int token = p.sorted[hi].x, last = p.sorted[hi - 1].x, begin = p.sorted[a * EMBED_TILE].x, ahead = a > 0 ? p.sorted[a * EMBED_TILE - 1].x : -1;
  if (token >= p.vocab || last != token) return;
  if (begin == token && ahead == token) return;   // it came from further ahead
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  // the first tile behind that does not begin within the token: 64 places looked at together
  int64_t lo = a + 1, end = p.tiles;
  while (end - lo > 1) {
    const int64_t step = (end - lo + 63) / 64, t = lo + lane * step;
    const int in = __builtin_popcountll(__ballot(t < end && p.sorted[min(t, end - 1) * EMBED_TILE].x == token));
    lo += (in - 1) * step;                        // the first of them is lo itself
    end = min(lo + step, end);
  }
  // what there is to add up: the tiles before the first whole group, the whole groups, the tiles behind
  const int64_t g0 = min((a + EMBED_GROUP) / EMBED_GROUP * EMBED_GROUP, end), g1 = p.gathered ? max(g0, end / EMBED_GROUP * EMBED_GROUP) : g0;
  const int64_t head = g0 - (a + 1), groups = (g1 - g0) / EMBED_GROUP, items = head + groups + (end - g1);
  auto tile_of = [&](int64_t i) {
    return i < head ? a + 1 + i : i < head + groups ? g0 + (i - head) * EMBED_GROUP : g1 + (i - head - groups);
  };
  const int64_t c0 = (int64_t)blockIdx.z * 512;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (wv == 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = p.part[(2 * a + 1) * p.cols + min(c0 + e * 64 + lane, (int64_t)p.cols - 1)];
  }
  // four parts in flight; those behind the last read the last and are left out
  for (int64_t i = wv; i < items; i += 16) {
    float v[4][8];
#pragma unroll
    for (int u = 0; u < 4; ++u) embed_load_parts(p, tile_of(min(i + 4 * u, items - 1)), c0, v[u]);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += i + 4 * u < items ? v[u][e] : 0.f;
  }
  embed_meet(acc, sum);
  if (wv) return;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c0 + e * 64 + lane < p.cols) reinterpret_cast<T*>(p.dt + (int64_t)token * p.dt_ld)[c0 + e * 64 + lane] = from_f32<T>(acc[e] * p.scale);
}

}  // namespace mns
