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
// workspace and are added up tile by tile. The work is in proportion to the positions whatever
// their tokens, so a token that occurs everywhere costs no more than others. Equal calls give equal
// bits.
//
// Bound by HBM: dy is read once and the table, mostly zeros, written once.
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
// pass, counts and places.
constexpr int EMBED_WAVES = 16, EMBED_NT = 64 * EMBED_WAVES;
constexpr int EMBED_DIGITS = 1024;
constexpr int64_t EMBED_ONE = 16384;

struct EmbedSortArgs {
  const void* tokens;
  int64_t n;
  int vocab;
  int bits, passes;                // per pass
  int steps;                       // 64-position steps per wave: a workgroup takes EMBED_NT * steps positions
  int nblocks;
  int32_t* key[2];                 // token (vocab: none) of the sorted positions, after even and odd passes
  int32_t* pos[2];                 // and the positions
  int32_t* hist;                   // [nblocks][EMBED_DIGITS]
  uint8_t* marks;                  // [vocab]: whether the token occurs
};

struct EmbedDigit {
  int key, pos, digit;             // digit -1: past the end
};
template <typename ID>
__device__ inline EmbedDigit embed_digit(const EmbedSortArgs& p, int pass, int64_t s) {
  if (s >= p.n) return {0, 0, -1};
  EmbedDigit d;
  if (pass == 0) {
    const int v = token_of<ID>(p.tokens, s, p.vocab);
    d.key = v < 0 ? p.vocab : v;
    d.pos = (int)s;
  } else {
    d.key = p.key[(pass - 1) & 1][s];
    d.pos = p.pos[(pass - 1) & 1][s];
  }
  d.digit = (d.key >> (pass * p.bits)) & ((1 << p.bits) - 1);
  return d;
}

// Each wave's positions by digit into at[wave], for this workgroup's run of positions.
template <typename ID>
__device__ inline void embed_count(const EmbedSortArgs& p, int pass, int64_t s0, int (*at)[EMBED_DIGITS]) {
  const int wv = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < EMBED_DIGITS; e += EMBED_NT)
#pragma unroll
    for (int w = 0; w < EMBED_WAVES; ++w) at[w][e] = 0;
  __syncthreads();
  for (int i = 0; i < p.steps; ++i) {
    const int d = embed_digit<ID>(p, pass, s0 + 64 * i).digit;
    if (d >= 0) atomicAdd(&at[wv][d], 1);
  }
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
template <typename ID>
__device__ inline void embed_place(const EmbedSortArgs& p, int pass, int64_t s0, int (*at)[EMBED_DIGITS]) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  for (int i = 0; i < p.steps; ++i) {
    const EmbedDigit d = embed_digit<ID>(p, pass, s0 + 64 * i);
    uint64_t same = __ballot(d.digit >= 0);
    for (int b = 0; b < p.bits; ++b) {
      const uint64_t m = __ballot((d.digit >> b) & 1);
      same &= (d.digit >> b) & 1 ? m : ~m;
    }
    const int lead = __builtin_ctzll(same | (1ull << 63));
    int next = 0;
    if (d.digit >= 0 && lane == lead) next = atomicAdd(&at[wv][d.digit], __builtin_popcountll(same));
    next = __shfl(next, lead);
    if (d.digit < 0) continue;
    const int to = next + __builtin_popcountll(same & ((1ull << lane) - 1));
    p.key[pass & 1][to] = d.key;
    p.pos[pass & 1][to] = d.pos;
    if (pass == 0 && d.key < p.vocab) p.marks[d.key] = 1;
  }
}

// Every pass in one workgroup, and the marks.
template <typename ID>
__global__ void __launch_bounds__(EMBED_NT) embed_sort_one(const EmbedSortArgs p) {
  __shared__ int at[EMBED_WAVES][EMBED_DIGITS];
  __shared__ int scan[EMBED_WAVES];
  // the workspace begins at a multiple of 16 bytes, and so do the marks, with room behind them
  for (int64_t i = (int64_t)threadIdx.x * 16; i < p.vocab; i += EMBED_NT * 16) *reinterpret_cast<u32x4*>(p.marks + i) = u32x4{0, 0, 0, 0};
  const int64_t s0 = (int64_t)(threadIdx.x >> 6) * 64 * p.steps + (threadIdx.x & 63);
  for (int pass = 0; pass < p.passes; ++pass) {
    embed_count<ID>(p, pass, s0, at);
    int total = 0;
    for (int w = 0; w < EMBED_WAVES; ++w) total += at[w][threadIdx.x];
    embed_places(total, 0, at, scan);
    embed_place<ID>(p, pass, s0, at);
    __syncthreads();
  }
}

template <typename ID>
__global__ void __launch_bounds__(EMBED_NT) embed_sort_count(const EmbedSortArgs p, int pass) {
  __shared__ int at[EMBED_WAVES][EMBED_DIGITS];
  if (pass == 0)
    for (int64_t i = ((int64_t)blockIdx.x * EMBED_NT + threadIdx.x) * 16; i < p.vocab; i += (int64_t)gridDim.x * EMBED_NT * 16)
      *reinterpret_cast<u32x4*>(p.marks + i) = u32x4{0, 0, 0, 0};
  const int64_t s0 = ((int64_t)blockIdx.x * EMBED_WAVES + (threadIdx.x >> 6)) * 64 * p.steps + (threadIdx.x & 63);
  embed_count<ID>(p, pass, s0, at);
  int total = 0;
  for (int w = 0; w < EMBED_WAVES; ++w) total += at[w][threadIdx.x];
  p.hist[(int64_t)blockIdx.x * EMBED_DIGITS + threadIdx.x] = total;
}

// Every workgroup adds up the counts itself: all of them for the digits before, the earlier
// workgroups' for its own positions.
template <typename ID>
__global__ void __launch_bounds__(EMBED_NT) embed_sort_place(const EmbedSortArgs p, int pass) {
  __shared__ int at[EMBED_WAVES][EMBED_DIGITS];
  __shared__ int scan[EMBED_WAVES];
  const int64_t s0 = ((int64_t)blockIdx.x * EMBED_WAVES + (threadIdx.x >> 6)) * 64 * p.steps + (threadIdx.x & 63);
  embed_count<ID>(p, pass, s0, at);
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
  embed_places(total, before, at, scan);
  embed_place<ID>(p, pass, s0, at);
}

// --------------------------------------------------------------------------------- gradient
constexpr int EMBED_TILE = 32;

struct EmbedGradArgs {
  const char* dy; int64_t dy_ld;   // bytes per row
  char* dt; int64_t dt_ld;
  const int32_t* key; const int32_t* pos;   // sorted
  const uint8_t* marks;
  float* part;                     // [2 * tiles][cols]: a tile's part of the token that came in from the tile before, of the one that goes on
  int64_t n, tiles;
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
  const int after = hi < p.n ? p.key[hi] : -1;
  int now = p.key[lo];
  bool came = lo > 0 && p.key[lo - 1] == now;
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
    int key[U];
    EmbedUnit<T, V> row[U];
#pragma unroll
    for (int u = 0; u < U; ++u) key[u] = s + u < hi ? p.key[s + u] : p.vocab;
    // the rows behind the tile's end read the tile's last and are left out: no branch between the loads
#pragma unroll
    for (int u = 0; u < U; ++u) row[u].load(reinterpret_cast<const T*>(p.dy + (int64_t)p.pos[min(s + u, hi - 1)] * p.dy_ld), c);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s + u >= hi) continue;
      if (key[u] != now) {
        leave(false);
        now = key[u];
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

// A token that crosses ends of tiles: its parts added up in the tiles' order. Workgroup (end between
// two tiles, 512 columns) works where a token begins in the tile before the end and goes on behind it;
// its four waves take every fourth tile.
template <typename T>
__global__ void __launch_bounds__(256) embed_join(const EmbedGradArgs p) {
  __shared__ float sum[3][8][64];
  const int64_t a = block_id();    // the tile that it begins in
  if (a + 1 >= p.tiles) return;
  const int64_t hi = (a + 1) * EMBED_TILE;
  const int token = p.key[hi];
  if (token >= p.vocab || p.key[hi - 1] != token) return;
  if (a > 0 && p.key[a * EMBED_TILE] == token && p.key[a * EMBED_TILE - 1] == token) return;   // it came from further ahead
  // the first tile behind that does not begin within the token
  int64_t lo = a + 1, end = p.tiles;
  while (end - lo > 1) {
    const int64_t mid = (lo + end) / 2;
    if (p.key[mid * EMBED_TILE] == token) lo = mid;
    else end = mid;
  }
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  for (int64_t c0 = (int64_t)blockIdx.z * 512; c0 < p.cols; c0 += (int64_t)gridDim.z * 512) {
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    auto add = [&](const float* part) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c0 + e * 64 + lane < p.cols) acc[e] += part[c0 + e * 64 + lane];
    };
    if (wv == 0) add(p.part + (2 * a + 1) * p.cols);
    for (int64_t t = a + 1 + wv; t < end; t += 4) add(p.part + 2 * t * p.cols);
    if (wv)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[wv - 1][e][lane] = acc[e];
    __syncthreads();
    if (wv == 0)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        for (int w = 0; w < 3; ++w) acc[e] += sum[w][e][lane];
        if (c0 + e * 64 + lane < p.cols) reinterpret_cast<T*>(p.dt + (int64_t)token * p.dt_ld)[c0 + e * 64 + lane] = from_f32<T>(acc[e] * p.scale);
      }
    __syncthreads();
  }
}

}  // namespace mns
