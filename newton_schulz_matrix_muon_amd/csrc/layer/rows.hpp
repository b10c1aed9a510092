// Tokens sorted by expert, and back.
//
// T tokens pick k of E experts each: S = T k slots, slot t k + j holding token t's j-th pick. The
// slots are sorted by expert (ties by slot, so the order is unique); rank[t][j] is the sorted row
// of a slot and offsets[e] .. offsets[e + 1] are expert e's rows. A slot whose pick is outside
// 0 .. E-1 (a padded token, an expert that lives elsewhere) gets rank -1 and no row; the rows
// from offsets[E] to S belong to nobody and are written as zeros.
//
//   dispatch          xs[rank[t][j]] = x[t]
//   its gradient      dx[t] = sum_j dxs[rank[t][j]]
//   combine           y[t] = sum_j w[t][j] ys[rank[t][j]]
//   its gradient      dys[rank[t][j]] = w[t][j] dy[t],  dw[t][j] = sum(dy[t] ys[rank[t][j]])
//
// Bound by HBM. The token side is read or written once and the row side once, in whole rows; each
// token's slots are handled together, so the gradients of its k copies meet in registers and no
// kernel needs atomics (sums run over j in order, in fp32, rounded once). One MI355X (a large copy
// reaches 5.0 to 5.3 TB/s): 8192 tokens of 7168 bf16, 8 of 384 experts each, sort 12 us, dispatch
// 207 us at 5.1 TB/s, combine 200 us at 5.3; 4099 tokens of 2048 fp16, 6 of 64, the dispatch's
// gradient 22 us at 5.3 TB/s, the combine's 51 us at 4.3.
//
// A rank outside 0 .. S-1 is treated as "no row", whatever the caller's buffer holds.
#pragma once

#include "norm.hpp"

namespace mns {

// ------------------------------------------------------------------------------------- sort
constexpr int SORT_WAVES = 8, SORT_NT = 64 * SORT_WAVES;
constexpr int SORT_MAX_E = 1024;

struct SortArgs {
  const void* ids;
  int64_t slots;
  int experts;
  int steps;              // 64-slot steps per wave: a workgroup takes SORT_NT * steps slots
  int nblocks;
  int32_t* hist;          // [nblocks][experts]: each workgroup's slots per expert
  int32_t* offsets;
  int32_t* rank;
};

// The expert of slot s, or -1.
template <typename ID>
__device__ inline int expert_of(const SortArgs& p, int64_t s) {
  if (s >= p.slots) return -1;
  const ID e = reinterpret_cast<const ID*>(p.ids)[s];
  return e >= 0 && e < (ID)p.experts ? (int)e : -1;
}

template <typename ID>
__global__ void __launch_bounds__(SORT_NT) sort_count(const SortArgs p) {
  __shared__ int h[SORT_MAX_E];
  for (int e = threadIdx.x; e < p.experts; e += SORT_NT) h[e] = 0;
  __syncthreads();
  const int64_t s0 = (int64_t)blockIdx.x * SORT_NT * p.steps;
  for (int i = 0; i < p.steps; ++i) {
    const int e = expert_of<ID>(p, s0 + (int64_t)i * SORT_NT + threadIdx.x);
    if (e >= 0) atomicAdd(&h[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.experts; e += SORT_NT) p.hist[(int64_t)blockIdx.x * p.experts + e] = h[e];
}

// Every workgroup adds up the counts itself (its own expert bases and, before its own slots, the
// earlier workgroups' slots), then places its slots: each wave walks its run of slots 64 at a
// time and ranks the lanes of one expert by their lane number. 65536 slots, 384 experts: count 4.8 us,
// place 7.5 (20 with the counts read one after the other; eight are in flight).
template <typename ID>
__global__ void __launch_bounds__(SORT_NT) sort_place(const SortArgs p) {
  __shared__ int at[SORT_WAVES][SORT_MAX_E];   // next row of (wave, expert)
  __shared__ int scan[SORT_WAVES];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < p.experts; e += SORT_NT)
#pragma unroll
    for (int w = 0; w < SORT_WAVES; ++w) at[w][e] = 0;
  __syncthreads();
  const int64_t s0 = ((int64_t)blockIdx.x * SORT_WAVES + wv) * 64 * p.steps + lane;
  for (int i = 0; i < p.steps; ++i) {
    const int e = expert_of<ID>(p, s0 + 64 * i);
    if (e >= 0) atomicAdd(&at[wv][e], 1);
  }
  __syncthreads();
  int base0 = 0;                               // rows of the experts before this pass
  for (int e0 = 0; e0 < p.experts; e0 += SORT_NT) {
    const int e = e0 + threadIdx.x;
    int total = 0, before = 0;
    if (e < p.experts) {
      if (p.nblocks == 1) {
        for (int w = 0; w < SORT_WAVES; ++w) total += at[w][e];
      } else {
        for (int b0 = 0; b0 < p.nblocks; b0 += 16) {
          int n[16];
#pragma unroll
          for (int b = 0; b < 16; ++b) n[b] = b0 + b < p.nblocks ? p.hist[(int64_t)(b0 + b) * p.experts + e] : 0;
#pragma unroll
          for (int b = 0; b < 16; ++b) {
            total += n[b];
            before += b0 + b < (int)blockIdx.x ? n[b] : 0;
          }
        }
      }
    }
    int run = total;                           // inclusive sum over the wave, then over the waves
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(run, o);
      if (lane >= o) run += v;
    }
    if (lane == 63) scan[wv] = run;
    __syncthreads();
    int first = base0 + run - total, all = 0;
    for (int w = 0; w < SORT_WAVES; ++w) {
      if (w < wv) first += scan[w];
      all += scan[w];
    }
    base0 += all;
    if (e < p.experts) {
      if (blockIdx.x == 0) p.offsets[e] = first;
      int next = first + before;
      for (int w = 0; w < SORT_WAVES; ++w) {
        const int n = at[w][e];
        at[w][e] = next;
        next += n;
      }
    }
    __syncthreads();
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) p.offsets[p.experts] = base0;
  const int bits = 32 - __builtin_clz(p.experts);
  for (int i = 0; i < p.steps; ++i) {
    const int64_t s = s0 + 64 * i;
    const int e = expert_of<ID>(p, s);
    uint64_t same = __ballot(e >= 0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t m = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? m : ~m;
    }
    const int lead = __builtin_ctzll(same | (1ull << 63));
    int next = 0;
    if (e >= 0 && lane == lead) next = atomicAdd(&at[wv][e], __builtin_popcountll(same));
    next = __shfl(next, lead);
    if (s < p.slots) p.rank[s] = e >= 0 ? next + __builtin_popcountll(same & ((1ull << lane) - 1)) : -1;
  }
}

// ------------------------------------------------------------------------------ copies, sums
struct RowsArgs {
  const char* tok; int64_t tok_ld;   // token side: x, dx, y, dy (bytes per row)
  const char* row; int64_t row_ld;   // row side: xs, dxs, ys (bytes per row)
  char* out; int64_t out_ld;         // dys of the combine's gradient (bytes per row)
  const int32_t* rank;
  const int32_t* offsets;            // for the rows of nobody
  const void* weights; int w_dt;
  void* dweights;
  int64_t tokens, slots;
  int k, experts;
  int units;                         // accesses per row
};

constexpr int ROWS_NT = 256;
constexpr int ROWS_KU = 8;           // slots of a token that are in flight together

// (token, unit) of this thread: 256 consecutive units of the token-major sequence a workgroup.
__device__ inline bool token_unit(const RowsArgs& p, int64_t* t, int* u) {
  const int64_t first = block_id() * ROWS_NT;
  const int64_t t0 = first / p.units;
  const unsigned x = (unsigned)(first - t0 * p.units) + threadIdx.x;
  const unsigned q = x / (unsigned)p.units;
  *t = t0 + q;
  *u = (int)(x - q * (unsigned)p.units);
  return *t < p.tokens;
}

__device__ inline bool has_row(const RowsArgs& p, int r) { return (unsigned)r < (uint64_t)p.slots; }

// Zeros to the rows of nobody; the workgroups share them row by row.
template <typename U, int NT>
__device__ inline void zero_rest(const RowsArgs& p, char* rows, int64_t ld) {
  int64_t r = p.offsets[p.experts];
  r = r < 0 ? 0 : r;
  for (r += block_id(); r < p.slots; r += (int64_t)gridDim.x * gridDim.y)
    for (int u = threadIdx.x; u < p.units; u += NT) reinterpret_cast<U*>(rows + r * ld)[u] = U{};
}

template <typename U>
__global__ void __launch_bounds__(ROWS_NT) rows_dispatch(const RowsArgs p) {
  int64_t t;
  int u;
  if (token_unit(p, &t, &u)) {
    const U v = reinterpret_cast<const U*>(p.tok + t * p.tok_ld)[u];
    for (int j0 = 0; j0 < p.k; j0 += ROWS_KU) {
      int r[ROWS_KU];
#pragma unroll
      for (int j = 0; j < ROWS_KU; ++j) r[j] = j0 + j < p.k ? p.rank[t * p.k + j0 + j] : -1;
#pragma unroll
      for (int j = 0; j < ROWS_KU; ++j)
        if (has_row(p, r[j])) reinterpret_cast<U*>(p.out + r[j] * p.out_ld)[u] = v;
    }
  }
  zero_rest<U, ROWS_NT>(p, p.out, p.out_ld);
}

// V consecutive elements of type T, as loaded, as fp32, and back (V = 8: whole 16-byte vectors;
// V = 1: any alignment).
template <typename T, int V> struct Unit {
  typename VecIO<T>::raw v;
  __device__ inline void load(const char* row, int u) { v = VecIO<T>::load_raw(row, (int64_t)u * 8); }
  __device__ inline void unpack(float (&f)[V]) const { VecIO<T>::unpack(v, f); }
};
template <typename T> struct Unit<T, 1> {
  T v;
  __device__ inline void load(const char* row, int u) { v = reinterpret_cast<const T*>(row)[u]; }
  __device__ inline void unpack(float (&f)[1]) const { f[0] = as_f32(v); }
};
template <typename T, int V>
__device__ inline void store_v(char* row, int u, const float (&v)[V]) {
  if constexpr (V == 8) VecIO<T>::store(row, (int64_t)u * 8, v);
  else reinterpret_cast<T*>(row)[u] = from_f32<T>(v[0]);
}

// Sum of a token's rows, weighted (the combine) or not (the dispatch's gradient).
template <typename T, int V, bool WEIGHTED>
__global__ void __launch_bounds__(ROWS_NT) rows_gather(const RowsArgs p) {
  int64_t t;
  int u;
  if (!token_unit(p, &t, &u)) return;
  float acc[V];
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.f;
  for (int j0 = 0; j0 < p.k; j0 += ROWS_KU) {
    int r[ROWS_KU];
    float w[ROWS_KU];
    Unit<T, V> v[ROWS_KU];
#pragma unroll
    for (int j = 0; j < ROWS_KU; ++j) {
      r[j] = j0 + j < p.k ? p.rank[t * p.k + j0 + j] : -1;
      w[j] = WEIGHTED && j0 + j < p.k ? load_elem(p.weights, p.w_dt, t * p.k + j0 + j) : 1.f;
    }
    // a slot without a row reads row 0 and is left out of the sum: no branch between the loads
#pragma unroll
    for (int j = 0; j < ROWS_KU; ++j)
      if (j0 + j < p.k) v[j].load(p.row + (has_row(p, r[j]) ? r[j] : 0) * p.row_ld, u);
#pragma unroll
    for (int j = 0; j < ROWS_KU; ++j)
      if (has_row(p, r[j])) {
        float f[V];
        v[j].unpack(f);
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] += w[j] * f[e];
      }
  }
  store_v<T, V>(p.out + t * p.out_ld, u, acc);
}

// The combine's gradient: one workgroup per token. Bound by the
// scattered rows' traffic, read and written; 4099 tokens of 2048 fp16, 6 rows each: 51 us (one wave a
// token 56).
template <typename T, int V>
__global__ void __launch_bounds__(ROWS_NT) rows_combine_bwd(const RowsArgs p) {
  constexpr int NT = ROWS_NT;
  __shared__ float red[NT / 64][ROWS_KU];
  const int64_t t = block_id();
  const char* dy = p.tok + t * p.tok_ld;
  for (int j0 = 0; j0 < p.k && t < p.tokens; j0 += ROWS_KU) {
    int r[ROWS_KU];
    float w[ROWS_KU], dot[ROWS_KU];
#pragma unroll
    for (int j = 0; j < ROWS_KU; ++j) {
      r[j] = j0 + j < p.k ? p.rank[t * p.k + j0 + j] : -1;
      w[j] = has_row(p, r[j]) ? load_elem(p.weights, p.w_dt, t * p.k + j0 + j) : 0.f;
      dot[j] = 0.f;
    }
    for (int u = threadIdx.x; u < p.units; u += NT) {
      Unit<T, V> gu, y[ROWS_KU];
      gu.load(dy, u);
#pragma unroll
      for (int j = 0; j < ROWS_KU; ++j)
        if (j0 + j < p.k) y[j].load(p.row + (has_row(p, r[j]) ? r[j] : 0) * p.row_ld, u);
      float g[V];
      gu.unpack(g);
#pragma unroll
      for (int j = 0; j < ROWS_KU; ++j)
        if (has_row(p, r[j])) {
          float f[V], o[V];
          y[j].unpack(f);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            dot[j] += g[e] * f[e];
            o[e] = w[j] * g[e];
          }
          store_v<T, V>(p.out + r[j] * p.out_ld, u, o);
        }
    }
#pragma unroll
    for (int j = 0; j < ROWS_KU; ++j) dot[j] = wave_sum(dot[j]);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int j = 0; j < ROWS_KU; ++j) red[threadIdx.x >> 6][j] = dot[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < ROWS_KU; ++j) {
      dot[j] = 0.f;
#pragma unroll
      for (int i = 0; i < NT / 64; ++i) dot[j] += red[i][j];
    }
    if (threadIdx.x == 0)
#pragma unroll
      for (int j = 0; j < ROWS_KU; ++j)
        if (j0 + j < p.k) store_elem(p.dweights, p.w_dt, t * p.k + j0 + j, has_row(p, r[j]) ? dot[j] : 0.f);
  }
  if constexpr (V == 8 && sizeof(T) == 4) {
    RowsArgs q = p;
    q.units *= 2;
    zero_rest<u32x4, NT>(q, p.out, p.out_ld);
  } else if constexpr (V == 8) {
    zero_rest<u32x4, NT>(p, p.out, p.out_ld);
  } else if constexpr (sizeof(T) == 4) {
    zero_rest<uint32_t, NT>(p, p.out, p.out_ld);
  } else {
    zero_rest<uint16_t, NT>(p, p.out, p.out_ld);
  }
}

}  // namespace mns
