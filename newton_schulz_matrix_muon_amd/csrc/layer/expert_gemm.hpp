// The experts' matrix products over rows sorted by expert.
//
//   forward            Y[s][n]     = sum_k X[s][k] W[e][n][k]     s in expert e's rows
//   input gradient     dX[s][k]    = sum_n dY[s][n] W[e][n][k]
//   weight gradient    dW[e][n][k] = sum_s dY[s][n] X[s][k]       s over expert e's rows
//
// expert e's rows are offsets[e] .. offsets[e + 1]; W and dW are batches of rows x cols matrices,
// the layout the Muon step takes. Rows of nobody (from offsets[E] on) get zeros, an expert
// without rows a zero gradient. Each product is C[i][j] = sum_c A(i, c) B(j, c) on MFMA with fp32
// accumulation, rounded once; an operand is read contraction-contiguous or contraction-major
// ("KM"), through gfx950's transposing LDS reads, so nothing is ever transposed in memory:
//
//                  i, j, c         A            B
//   forward        s, n, k         X            W
//   input grad     s, k, n         dY           W   KM
//   weight grad    n, k, s         dY  KM       X   KM
//
// The row counts live on the GPU only: every workgroup reads the offsets, adds up the experts'
// tiles in LDS and walks its share of them, so a call never waits for the host. Offsets that run
// outside 0 .. S are cut to it, and an expert whose end lies before its beginning has no rows.
#pragma once

#include <type_traits>

#include "norm.hpp"

namespace mns {

constexpr int EXPERT_MAX = 1024;

// Which product: forward, input gradient, weight gradient; the same of two matrices side by side (gated.hpp).
enum { EX_FWD = 0, EX_DX = 1, EX_DW = 2, EX_GATE = 3, EX_DX2 = 4, EX_DW2 = 5 };
__host__ __device__ constexpr bool ex_fwd(int mode) { return mode == EX_FWD || mode == EX_GATE; }
__host__ __device__ constexpr bool ex_dx(int mode) { return mode == EX_DX || mode == EX_DX2; }
__host__ __device__ constexpr bool ex_dw(int mode) { return mode == EX_DW || mode == EX_DW2; }

struct ExpertArgs {
  const char* A; int64_t lda;       // elements
  const char* B; int64_t ldb, sB;   // sB, sC: from matrix to matrix, where there is one per expert
  char* C; int64_t ldc, sC;
  const int32_t* offsets;
  int experts;
  int64_t rows;                     // S
  int n;                            // columns of C (extent of j)
  int m, k;                         // extents of i / of the contraction, where fixed
  int tiles_n;
  int c_vec;                        // 16-byte stores fit C
};

// Two matrices W and W2 per expert over the same rows.
//   EX_GATE  C = act(A B^T) * (A B2^T), and the two products to C2 and C3 where they are kept
//   EX_DX2   C = A B + A2 B2
//   EX_DW2   C = A^T B, C2 = A2^T B
// A tile of EX_GATE holds blocks of 32 columns of W and W2 in turn, so that a wave has both products
// of its columns; EX_DX2's contraction runs over A and B, then over A2 and B2; EX_DW2 takes C and
// C2 as the results of two experts.
struct GatedArgs : ExpertArgs {
  const char* A2;                   // rows like A's
  const char* B2; int64_t ldb2, sB2;
  char* C2; int64_t ldc2, sC2;
  char* C3; int64_t ldc3;
  int act;
  // expert_gemm_pp, SPLIT: sums of the parts, 256 x 256 floats a workgroup, and workgroups per XCD
  float* parts; int wgs;
};
enum { ACT_SILU = 0, ACT_GELU = 1, ACT_RELU = 2 };
template <int MODE> struct ArgsOf { typedef ExpertArgs type; };
template <> struct ArgsOf<EX_GATE> { typedef GatedArgs type; };
template <> struct ArgsOf<EX_DX2> { typedef GatedArgs type; };
template <> struct ArgsOf<EX_DW2> { typedef GatedArgs type; };

// Columns of C that a tile of BN columns of B makes.
template <int MODE, class CFG> constexpr int tile_cols() { return MODE == EX_GATE ? CFG::BN / 2 : CFG::BN; }
// Matrices that the weight gradient's tiles belong to.
template <int MODE> __host__ __device__ inline int dw_matrices(const ExpertArgs& p) { return MODE == EX_DW2 ? 2 * p.experts : p.experts; }

// Beginning and end of expert e's rows; e = E: the rows of nobody. No offsets: one expert has all rows.
__host__ __device__ inline void expert_rows(const ExpertArgs& p, int e, int* lo, int* hi) {
  const int rows = (int)p.rows;
  if (!p.offsets) {
    *lo = e < p.experts ? 0 : rows;
    *hi = rows;
    return;
  }
  const int a = p.offsets[e], b = e < p.experts ? p.offsets[e + 1] : rows;
  *lo = min(max(a, 0), rows);
  *hi = min(max(b, *lo), rows);
}

// The arithmetic of the tile list in plain functions, which a test compiles for the host.
//
// Tile rows before an expert, cut so that their number of tiles fits 32 bits. The host keeps a
// call's tiles below 2^31, so nothing is cut but what offsets that fall and rise again make: experts
// that share rows have up to E / 2 times the tile rows that S rows have.
__host__ __device__ inline int list_rows(int64_t tile_rows, int tiles_n) {
  return (int)min(tile_rows, (int64_t)(0x7fffffff / tiles_n));
}

// Whether all tiles up to expert i's last lie before or at tile t of the list.
__host__ __device__ inline bool ends_by(const int* first, int i, int tiles_n, int t) { return first[i + 1] * tiles_n <= t; }

// Tile r of an expert with tm x tiles_n of them: in bands of EXPERT_BAND tile rows, down a band,
// then one tile column right.
constexpr int EXPERT_BAND = 8;
struct TileAt {
  int row, col;
};
__host__ __device__ inline TileAt tile_at(int r, int tm, int tiles_n) {
  const int band = r / (EXPERT_BAND * tiles_n), high = min(tm - band * EXPERT_BAND, EXPERT_BAND);
  r -= band * EXPERT_BAND * tiles_n;
  return {band * EXPERT_BAND + r % high, r / high};
}

// What a tile of a weight gradient costs, in stages of 64 rows: three more than it has, for its stores and
// the tile's begin (one MI355X, 256 x 256 tiles: 1.66 us a stage, 5.3 us a tile without any).
__host__ __device__ inline int dw_cost(int rows) { return (rows + 63) / 64 + 3; }

// first[e] = tile rows (of BM) of the experts before e, as list_rows cuts them, e = 0 .. E + 1: entry
// E begins the tile rows over the rows of nobody, entry E + 1 is the total. rows (ROWS): beginning and number of each
// expert's rows. COST: first[e] = what a tile of each of the experts before e costs. Ends with a barrier.
template <int NT, int BM, bool ROWS = false, bool COST = false>
__device__ inline void expert_tiles(const ExpertArgs& p, int* first, int* wsum, int2* rows = nullptr) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  int base = 0;
  for (int e0 = 0; e0 <= p.experts; e0 += NT) {
    const int e = e0 + threadIdx.x;
    int n = 0;
    if (e <= p.experts) {
      int lo, hi;
      expert_rows(p, e, &lo, &hi);
      n = COST ? (e < p.experts ? dw_cost(hi - lo) : 0) : (hi - lo + BM - 1) / BM;
      if constexpr (ROWS) rows[e] = int2{lo, hi - lo};
    }
    int run = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(run, o);
      if (lane >= o) run += v;
    }
    if (lane == 63) wsum[wv] = run;
    __syncthreads();
    int before = base, all = 0;
    for (int w = 0; w < NT / 64; ++w) {
      if (w < wv) before += wsum[w];
      all += wsum[w];
    }
    base += all;
    if (e <= p.experts) first[e] = COST ? before + run - n : list_rows(before + run - n, p.tiles_n);
    if (e == p.experts) first[e + 1] = COST ? before + run : list_rows(before + run, p.tiles_n);
    __syncthreads();
  }
}

// One output tile: its expert's operands and result, where it lies in the result, and what it
// sums over. Equal in every lane.
struct ExpertTile {
  int row0, col0;         // of the tile, within its expert's result
  int m, k;               // rows of the expert's result, contraction length
  const char* a; const char* b;
  char* c;
  const char* a2; const char* b2;   // EX_GATE, EX_DX2
  char* c2; char* c3;               // EX_GATE
  int64_t ldc;                      // EX_DW2
};

// 16 bytes at any element's address
typedef u32x4 u32x4_any __attribute__((aligned(2)));

// How the 16-byte chunks of an operand's rows are loaded: rows of whole aligned chunks; rows of any
// length from a chunk on, at any address, which the hardware's loads take as it is; rows shorter
// than a chunk, element by element.
enum { CHUNK_TINY, CHUNK_ANY, CHUNK_ALIGNED };

// Elements e0 .. of a row `len` long. The row has the whole chunk, but for CHUNK_TINY, which gives
// zeros past the end.
template <typename T, int FIT>
__device__ inline u32x4 load_chunk(const T* row, int e0, int len) {
  constexpr int N = 16 / (int)sizeof(T);
  if constexpr (FIT == CHUNK_ALIGNED) {
    return *reinterpret_cast<const u32x4*>(row + e0);
  } else if constexpr (FIT == CHUNK_ANY) {
    return *reinterpret_cast<const u32x4_any*>(row + e0);
  } else {
    typedef T TN __attribute__((ext_vector_type(N)));
    TN v;
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = e0 + e < len ? row[e0 + e] : (T)0.f;
    return __builtin_bit_cast(u32x4, v);
  }
}

// v without its first `by` elements, zeros behind.
template <typename T>
__device__ inline u32x4 drop_first(u32x4 v, int by) {
  constexpr int N = 16 / (int)sizeof(T);
  const unsigned __int128 w = __builtin_bit_cast(unsigned __int128, v);
  return by < N ? __builtin_bit_cast(u32x4, w >> (by * (int)sizeof(T) * 8)) : u32x4{0, 0, 0, 0};
}


// The part of the launch's tile list that one XCD takes (an eighth, so that neighbouring tiles
// share an L2), for the workgroups on it to walk side by side.
struct ExpertList {
  int lo, n;
};
template <int MODE, class CFG>
__device__ inline ExpertList expert_list(const ExpertArgs& p, const int* first) {
  // below 2^31: a weight gradient's by the host's check, the others' also by list_rows
  const int64_t total = (int64_t)p.tiles_n * (ex_dw(MODE) ? dw_matrices<MODE>(p) * ((p.m + CFG::BM - 1) / CFG::BM) : wave_uniform(first[p.experts + 1]));
  const int xcd = blockIdx.x & 7;
  const int lo = (int)(total * xcd / 8);
  return {wave_uniform(lo), wave_uniform((int)(total * (xcd + 1) / 8) - lo)};
}

// The same for a weight gradient whose experts' tiles cost as COST says: eight parts of equal cost, so that
// experts with many rows do not fall to one XCD. cost_begin: where part x begins, in tiles; first, T (tiles
// per expert) as above; which: the expert that the part begins in.
__host__ __device__ inline int64_t cost_target(const int* first, int experts, int64_t T, int x) { return first[experts] * T * x / 8; }
__host__ __device__ inline int cost_begin(const int* first, int experts, int64_t T, int x, int which) {
  if (which >= experts) return (int)(experts * T);
  return (int)(which * T + (cost_target(first, experts, T, x) - first[which] * T) / (first[which + 1] - first[which]));
}
__device__ inline ExpertList cost_list(const ExpertArgs& p, const int* first, int64_t T) {
  const int xcd = blockIdx.x & 7, lane = threadIdx.x & 63;
  int begin[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int64_t target = cost_target(first, p.experts, T, xcd + s);
    int e = 0;
    for (int i = lane; i - lane < p.experts; i += 64) e += __builtin_popcountll(__ballot(i < p.experts && first[i + 1] * T <= target));
    begin[s] = wave_uniform(cost_begin(first, p.experts, T, xcd + s, e));
  }
  return {begin[0], begin[1] - begin[0]};
}

// Tile t of an XCD's list. Tiles go expert by expert, within one in bands (tile_at), so that the
// tiles that run together share panels of both operands in L2. *from: the expert of the tile
// before, or 0. rows (ROWS): as expert_tiles left them.
template <int MODE, typename T, class CFG, bool ROWS = false>
__device__ inline ExpertTile expert_tile(const typename ArgsOf<MODE>::type& p, const int* first, const ExpertList& l, int t, int* from,
                                         const int2* rows = nullptr) {
  t += l.lo;
  constexpr int ES = sizeof(T);
  ExpertTile x;
  int e, r, tm;
  bool second = false;
  if constexpr (ex_dw(MODE)) {
    tm = (p.m + CFG::BM - 1) / CFG::BM;
    e = t / (tm * p.tiles_n);
    r = t - e * tm * p.tiles_n;
    if constexpr (MODE == EX_DW2) {
      second = e & 1;
      e >>= 1;
    }
  } else {
    // the expert whose tiles hold t: the last tile's, or as many as end at or before t
    e = *from;
    if (wave_uniform(first[e + 1]) * p.tiles_n <= t) {
      const int lane = threadIdx.x & 63;
      e = 0;
      for (int i = lane; i - lane <= p.experts; i += 64)
        e += __builtin_popcountll(__ballot(i <= p.experts && ends_by(first, i, p.tiles_n, t)));
    }
    *from = e;
    const int f = wave_uniform(first[e]);
    tm = wave_uniform(first[e + 1]) - f;
    r = t - f * p.tiles_n;
  }
  int lo, hi;
  if constexpr (ROWS) {
    lo = rows[e].x;
    hi = lo + rows[e].y;
  } else {
    expert_rows(p, e, &lo, &hi);
  }
  lo = wave_uniform(lo);
  hi = wave_uniform(hi);
  const TileAt at = tile_at(r, tm, p.tiles_n);
  x.row0 = at.row * CFG::BM;
  x.col0 = at.col * tile_cols<MODE, CFG>();
  x.a = p.A + (int64_t)lo * p.lda * ES;
  if constexpr (ex_dw(MODE)) {
    x.m = p.m;
    x.k = hi - lo;
    x.b = p.B + (int64_t)lo * p.ldb * ES;
    x.c = p.C + (int64_t)e * p.sC * ES;
    if constexpr (MODE == EX_DW2) {
      x.ldc = second ? p.ldc2 : p.ldc;
      if (second) {
        x.a = p.A2 + (int64_t)lo * p.lda * ES;
        x.c = p.C2 + (int64_t)e * p.sC2 * ES;
      }
    }
  } else {
    x.m = hi - lo;
    x.k = e < p.experts ? p.k : 0;
    x.b = p.B + (int64_t)(e < p.experts ? e : 0) * p.sB * ES;
    x.c = p.C + (int64_t)lo * p.ldc * ES;
    if constexpr (MODE == EX_GATE || MODE == EX_DX2) x.b2 = p.B2 + (int64_t)(e < p.experts ? e : 0) * p.sB2 * ES;
    if constexpr (MODE == EX_DX2) x.a2 = p.A2 + (int64_t)lo * p.lda * ES;
    if constexpr (MODE == EX_GATE) {
      x.c2 = p.C2 ? p.C2 + (int64_t)lo * p.ldc2 * ES : nullptr;
      x.c3 = p.C2 ? p.C3 + (int64_t)lo * p.ldc3 * ES : nullptr;
    }
  }
  return x;
}

// From one row of a tile's result to the next.
template <int MODE, class P>
__device__ inline int64_t row_step(const P& p, const ExpertTile& x) {
  if constexpr (MODE == EX_DW2) return x.ldc;
  else return p.ldc;
}

// Elements c .. c + 7 of a row of n, at any address.
template <typename T>
__device__ inline void store_eight(T* out, int c, int n, const f32x4& a, const f32x4& b) {
  constexpr int DT = sizeof(T) == 4 ? F32 : (__is_same(T, __bf16) ? BF16 : F16);
  const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  if (c + 8 <= n) {
    u32x4_any* o = reinterpret_cast<u32x4_any*>(out + c);
    if constexpr (sizeof(T) == 4) {
      o[0] = __builtin_bit_cast(u32x4, a);
      o[1] = __builtin_bit_cast(u32x4, b);
    } else {
      o[0] = u32x4{pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7])};
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < n) store_elem(out, DT, c + e, v[e]);
  }
}

// exp(x) for rows of T: fp32 to an ulp; for 16 bits as exp2 of a rounded argument, off by |x| 2^-24 of it, which is far below
// the rows' half step wherever the activation is not 0 in them.
template <typename T>
__device__ inline float row_exp(float x) {
  return sizeof(T) == 4 ? expf(x) : __expf(x);
}

// F(g), the normal distribution's part below g, and exp(-g^2 / 2). By erfc, not 1 + erf, which has lost the digits of a part
// near 0 (all of them from g = -5.4 on). For rows of 16 bits, whose half step is 2^-12 of the value at least, the part below -|g| as
// t P(t) exp(-g^2 / 2) with t = 1 / (1 + 0.3 |g| / sqrt 2): the polynomial is fitted to erfcx by reweighted least
// squares (2e-8 off, 5e-7 as evaluated near 0). With erff, which is two branches of polynomials, a forward product of
// 64 x 1408 x 2048 with 384 rows each took 431 us for gelu, 375 for relu.
template <typename T>
__device__ inline float normal_part(float g, float* density) {
  *density = row_exp<T>(-0.5f * g * g);
  if constexpr (sizeof(T) == 4) return 0.5f * erfcf(-0.70710678118654752f * g);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.21213204f, __builtin_fabsf(g), 1.f));
  constexpr float P[9] = {0.084594116f, 0.085356005f, 0.074179493f, 0.10742909f, -0.047254566f, 0.27376783f, -0.25606576f, 0.24274902f, -0.064755239f};
  float s = P[8];
#pragma unroll
  for (int i = 7; i >= 0; --i) s = __builtin_fmaf(s, t, P[i]);
  s *= t * *density;
  return g < 0.f ? s : 1.f - s;
}

// The activation of a gate's value; for results of 16 bits quotients by the reciprocal to 1 ulp.
template <typename T, int ACT>
__device__ inline float activated(float g) {
  if constexpr (ACT == ACT_RELU) {
    return g <= 0.f ? 0.f : g;   // a maximum instruction would turn a NaN into 0
  } else if constexpr (ACT == ACT_SILU) {
    const float d = 1.f + row_exp<T>(-g);
    return sizeof(T) == 2 ? g * __builtin_amdgcn_rcpf(d) : g / d;
  } else {
    float density;
    return g * normal_part<T>(g, &density);
  }
}
// f(the activation as a constant): chosen once, not once a value.
template <class F>
__device__ inline void with_activation(int act, F&& f) {
  if (act == ACT_SILU) f(std::integral_constant<int, ACT_SILU>{});
  else if (act == ACT_GELU) f(std::integral_constant<int, ACT_GELU>{});
  else f(std::integral_constant<int, ACT_RELU>{});
}

// Columns lc .. lc + 7 of row lr of a slab's tile to C (EX_GATE: from blocks of 32 columns of both products, to C and
// where they are kept to C2 and C3). read(column): four sums of the row.
template <int MODE, typename T, class P, class R>
__device__ inline void store_from(const P& p, const ExpertTile& x, int r, int c, int lc, R&& read) {
  if constexpr (MODE == EX_GATE) {
    const int at = (lc >> 5) * 64 + (lc & 31);
    const f32x4 g0 = read(at), g1 = read(at + 4), u0 = read(at + 32), u1 = read(at + 36);
    f32x4 h0, h1;
    with_activation(p.act, [&](auto act) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h0[e] = activated<T, act.value>(g0[e]) * u0[e];
        h1[e] = activated<T, act.value>(g1[e]) * u1[e];
      }
    });
    store_eight(reinterpret_cast<T*>(x.c) + (int64_t)r * p.ldc, c, p.n, h0, h1);
    if (x.c2) {
      store_eight(reinterpret_cast<T*>(x.c2) + (int64_t)r * p.ldc2, c, p.n, g0, g1);
      store_eight(reinterpret_cast<T*>(x.c3) + (int64_t)r * p.ldc3, c, p.n, u0, u1);
    }
  } else {
    store_eight(reinterpret_cast<T*>(x.c) + (int64_t)r * row_step<MODE>(p, x), c, p.n, read(lc), read(lc + 4));
  }
}

// Accumulators to C: through an fp32 slab in LDS, whole rows of 16-byte vectors out.
template <int MODE, typename T, class CFG>
__device__ inline void expert_store(const typename ArgsOf<MODE>::type& p, const ExpertTile& x, char* lds, const f32x16 (&acc)[CFG::TM][CFG::TN], int lane) {
  constexpr int NT = CFG::NT, WTM = CFG::WTM, CP = CFG::CP;
  constexpr int SR = CFG::SR, SROWS = SR * WTM, VPR = tile_cols<MODE, CFG>() / 8;
  const int wave = wave_uniform(threadIdx.x >> 6), tid = wave * 64 + lane;
  const int wm = wave / CFG::WVN, wn = wave % CFG::WVN;
  float* Cs = reinterpret_cast<float*>(lds);
  for (int sl = 0; sl < CFG::WVM / SR; ++sl) {
    if (wm / SR == sl) acc_to_slab<CFG>(Cs, acc, lane, wn, (wm % SR) * WTM);
    lds_barrier();
#pragma unroll 1
    for (int idx = tid; idx < SROWS * VPR; idx += NT) {
      const int lr = idx / VPR, lc = (idx - lr * VPR) * 8;
      const int r = x.row0 + sl * SROWS + lr, c = x.col0 + lc;
      if (r < x.m && c < p.n)
        store_from<MODE, T>(p, x, r, c, lc, [&](int at) { return *reinterpret_cast<const f32x4*>(Cs + lr * CP + at); });
    }
    lds_barrier();
  }
}

// kmajor_swizzle and kmajor_frag_off of gemm.hpp for rows of C chunks, 8 as well as 16.
template <int C>
__device__ constexpr int stage_swizzle(int s) { return kmajor_swizzle(s) & (C - 1); }
template <int RB>
__device__ inline int stage_frag_off(int lane, int n0) {
  const int j16 = lane & 15, qo = (lane >> 4) & 1, hi = lane >> 5;
  const int n = n0 + 16 * qo + 4 * (j16 & 3);
  return (8 * hi + (j16 >> 2)) * RB + (((n >> 3) ^ stage_swizzle<RB / 16>(j16 >> 2)) << 4) + 8 * (j16 & 1);
}

// G waves' sums of one tile to C, added up in the waves' order.
template <int MODE, typename T, class CFG, int G>
__device__ inline void expert_store_split(const typename ArgsOf<MODE>::type& p, const ExpertTile& x, char* lds, const f32x16 (&acc)[CFG::TM][CFG::TN], int lane) {
  constexpr int BM = CFG::BM, CP = CFG::CP, VPR = tile_cols<MODE, CFG>() / 8;
  const int wave = wave_uniform(threadIdx.x >> 6);
  acc_to_slab<CFG>(reinterpret_cast<float*>(lds + wave * CFG::STAGE), acc, lane, 0, 0);
  lds_barrier();
#pragma unroll 1
  for (int idx = wave * 64 + lane; idx < BM * VPR; idx += 64 * G) {
    const int lr = idx / VPR, lc = (idx - lr * VPR) * 8;
    const int r = x.row0 + lr, c = x.col0 + lc;
    if (r < x.m && c < p.n)
      store_from<MODE, T>(p, x, r, c, lc, [&](int at) {
        f32x4 a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int g = 0; g < G; ++g) a += *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(lds + g * CFG::STAGE) + lr * CP + at);
        return a;
      });
  }
  lds_barrier();
}

// Operands staged through registers: every type, any alignment and length (FIT). 128 x 128 tiles of
// 4 waves, one stage of K ahead in registers (two ahead gained 1 % at 50 registers more), 64 KB of
// LDS and two workgroups a CU, so that one computes while the other waits.
//
// One MI355X, bf16, 64 experts with 64 rows on average: 1408 x 2048 forward 108 us, input gradient 82,
// weight gradient 147; 1405 x 2045, whose rows begin anywhere, 122, 95, 189. Loads element by
// element for such rows took 3 times as long, loads under a condition per lane 1.3 to 2 times (the
// compiler waits for one before the next). fp32 is bound by its MFMAs, so blocks of 32 rows that have none are left out.
//
// G > 1 (few tiles): 64 x 64 tiles whose G waves take every G-th stage each, on their own: a wave
// stages into its own piece of LDS, where its reads and writes keep their order without a barrier,
// and the sums meet at the end. A stage of a 128 x 128 tile alone on its CU takes about 1 us (loads,
// LDS, barrier, MFMAs one after the other; fp32 1.8), so eight waves side by side cut the time of a
// long contraction to a third: 3 experts of 504 x 4000 bf16, 256 rows each, 61 us to 20.
template <int MODE, typename T, int FIT, class CFG, int G = 1>
__global__ void __launch_bounds__(CFG::NT * G, CFG::OCC) expert_gemm_staged(const typename ArgsOf<MODE>::type p) {
  constexpr int ES = sizeof(T), BM = CFG::BM, BN = CFG::BN, NT = CFG::NT, KB = CFG::KB, ROWB = CFG::ROWB;
  constexpr int EPC = 16 / ES, BK = KB / ES, CPR = CFG::CPR, TM = CFG::TM, TN = CFG::TN;
  constexpr bool AKM = ex_dw(MODE), BKM = !ex_fwd(MODE);
  constexpr int CPM = BM * ES / 16, CPN = BN * ES / 16;   // chunks per contraction-major row
  static_assert(G == 1 || (CFG::NT == 64 && CFG::STAGE >= CFG::SLAB), "the parts of a split tile are waves");
  __shared__ __align__(16) char lds_all[G > 1 ? G * CFG::STAGE : CFG::LDS];
  __shared__ int first[EXPERT_MAX + 2];
  __shared__ int wsum[NT * G / 64];
  const int part = G > 1 ? wave_uniform(threadIdx.x >> 6) : 0;
  char* lds = lds_all + part * CFG::STAGE;
  const int tid = G > 1 ? threadIdx.x & 63 : threadIdx.x, lane = tid & 63, wave = G > 1 ? 0 : wave_uniform(tid >> 6);
  const int wm = wave / CFG::WVN, wn = wave % CFG::WVN;
  if constexpr (!ex_dw(MODE)) expert_tiles<NT * G, BM>(p, first, wsum);
  const ExpertList l = expert_list<MODE, CFG>(p, first);
  int from = 0;
  for (int t = blockIdx.x >> 3; t < l.n; t += gridDim.x >> 3) {
    const ExpertTile x = expert_tile<MODE, T, CFG>(p, first, l, t, &from);
    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    const int nh = (x.k + BK - 1) / BK;            // stages of a contraction, EX_DX2: of either
    const int nk = MODE == EX_DX2 ? 2 * nh : nh;
    // A thread's chunks of a stage: loaded without a branch from places clamped into the operand,
    // so that the loads of a stage are all in flight together; what the clamps moved is put right
    // when the registers go to LDS, in the stages and tiles that have an edge. Only the contraction
    // needs its zeros: rows and columns past C's are not stored.
    u32x4 ra[CFG::CA], rb[CFG::CB];
    constexpr int RPQ = NT / CPR;       // rows that one chunk of every thread covers
    constexpr bool CLAMP = FIT != CHUNK_TINY;
    // A of EX_DX2 and EX_DW2 has rows of whole chunks, zeros behind the end
    const int klen = MODE == EX_DX2 && CLAMP ? (x.k + EPC - 1) / EPC * EPC : x.k;
    const int mlen = MODE == EX_DW2 && CLAMP ? (x.m + EPC - 1) / EPC * EPC : x.m;
    auto load_rows = [&](const T* src, int64_t ld, int row0, int rows, int k0, auto& r) {
      const int e0 = k0 + (tid % CPR) * EPC, row = tid / CPR;
#pragma unroll
      for (int q = 0; q < (int)(sizeof(r) / 16); ++q) {
        const int first = row0 + RPQ * q;
        if (first >= rows) break;       // equal in every lane
        const T* at = src + (int64_t)min(first + row, rows - 1) * ld;
        r[q] = load_chunk<T, FIT>(at, CLAMP ? min(e0, klen - EPC) : e0, klen);
      }
    };
    auto load_deep = [&](const T* src, int64_t ld, int col0, int cols, int k0, auto& r, auto cpr_c) {
      constexpr int C = decltype(cpr_c)::value;
      const int c0 = col0 + (tid % C) * EPC;
#pragma unroll
      for (int q = 0; q < (int)(sizeof(r) / 16); ++q) {
        const T* at = src + (int64_t)min(k0 + tid / C + NT / C * q, x.k - 1) * ld;
        r[q] = load_chunk<T, FIT>(at, CLAMP ? min(c0, cols - EPC) : c0, cols);
      }
    };
    auto mend_rows = [&](int k0, auto& r) {
      const int e0 = k0 + (tid % CPR) * EPC;
#pragma unroll
      for (int q = 0; q < (int)(sizeof(r) / 16); ++q) {
        if constexpr (FIT == CHUNK_ALIGNED) r[q] = e0 < klen ? r[q] : u32x4{0, 0, 0, 0};
        else if constexpr (CLAMP) r[q] = drop_first<T>(r[q], e0 - min(e0, klen - EPC));
      }
    };
    auto mend_deep = [&](int col0, int cols, int k0, auto& r, auto cpr_c) {
      constexpr int C = decltype(cpr_c)::value;
      const int c0 = col0 + (tid % C) * EPC;
#pragma unroll
      for (int q = 0; q < (int)(sizeof(r) / 16); ++q) {
        if constexpr (FIT == CHUNK_ANY) r[q] = drop_first<T>(r[q], c0 - min(c0, cols - EPC));
        r[q] = k0 + tid / C + NT / C * q < x.k ? r[q] : u32x4{0, 0, 0, 0};
      }
    };
    // the columns' rows of both matrices, a block of 32 of either in turn
    auto load_gated = [&](int k0, auto& r) {
      const int e0 = k0 + (tid % CPR) * EPC, row = tid / CPR;
#pragma unroll
      for (int q = 0; q < (int)(sizeof(r) / 16); ++q) {
        constexpr int BLOCK = 32;
        const int block = RPQ * q / BLOCK, first = x.col0 + (block >> 1) * BLOCK + RPQ * q % BLOCK;
        if (first >= p.n) continue;     // equal in every lane
        const T* src = reinterpret_cast<const T*>(block & 1 ? x.b2 : x.b);
        int64_t ld = p.ldb;
        if constexpr (MODE == EX_GATE)
          if (block & 1) ld = p.ldb2;
        const T* at = src + (int64_t)min(first + row, p.n - 1) * ld;
        r[q] = load_chunk<T, FIT>(at, CLAMP ? min(e0, x.k - EPC) : e0, x.k);
      }
    };
    using CM = std::integral_constant<int, CPM>;
    using CN = std::integral_constant<int, CPN>;
    // where stage kt begins in its contraction, and the operands of that one
    auto begin_of = [&](int kt) { return (MODE == EX_DX2 && kt >= nh ? kt - nh : kt) * BK; };
    auto load_stage = [&](int kt) {
      const int k0 = begin_of(kt);
      const T* A = reinterpret_cast<const T*>(x.a);
      const T* B = reinterpret_cast<const T*>(x.b);
      int64_t ldb = p.ldb;
      if constexpr (MODE == EX_DX2) {
        if (kt >= nh) {
          A = reinterpret_cast<const T*>(x.a2);
          B = reinterpret_cast<const T*>(x.b2);
          ldb = p.ldb2;
        }
      }
      if constexpr (AKM) load_deep(A, p.lda, x.row0, mlen, k0, ra, CM{});
      else load_rows(A, p.lda, x.row0, x.m, k0, ra);
      if constexpr (BKM) load_deep(B, ldb, x.col0, p.n, k0, rb, CN{});
      else if constexpr (MODE == EX_GATE) load_gated(k0, rb);
      else load_rows(B, ldb, x.col0, p.n, k0, rb);
    };
    auto store_stage = [&](int buf, int kt) {
      const int k0 = begin_of(kt);
      char* As = lds + buf * CFG::STAGE;
      char* Bs = As + BM * ROWB;
      const bool cut = k0 + BK > x.k;
      if constexpr (AKM) {
        if (cut || (FIT == CHUNK_ANY && x.row0 + BM > mlen)) mend_deep(x.row0, mlen, k0, ra, CM{});
      } else {
        if (cut) mend_rows(k0, ra);
      }
      if constexpr (BKM) {
        if (cut || (FIT == CHUNK_ANY && x.col0 + BN > p.n)) mend_deep(x.col0, p.n, k0, rb, CN{});
      } else {
        if (cut) mend_rows(k0, rb);
      }
#pragma unroll
      for (int q = 0; q < CFG::CA; ++q) {
        const int c = tid + NT * q;
        if constexpr (AKM)
          *reinterpret_cast<u32x4*>(As + (c / CPM) * (BM * ES) + (((c % CPM) ^ stage_swizzle<CPM>((c / CPM) & 3)) << 4)) = ra[q];
        else
          *reinterpret_cast<u32x4*>(As + (c / CPR) * ROWB + (c % CPR) * 16) = ra[q];
      }
#pragma unroll
      for (int q = 0; q < CFG::CB; ++q) {
        const int c = tid + NT * q;
        if constexpr (BKM)
          *reinterpret_cast<u32x4*>(Bs + (c / CPN) * (BN * ES) + (((c % CPN) ^ stage_swizzle<CPN>((c / CPN) & 3)) << 4)) = rb[q];
        else
          *reinterpret_cast<u32x4*>(Bs + (c / CPR) * ROWB + (c % CPR) * 16) = rb[q];
      }
    };
    typedef typename Frag<T>::type F;
    int aoff[TM], boff[TN];
#pragma unroll
    for (int i = 0; i < TM; ++i) aoff[i] = AKM ? stage_frag_off<BM * ES>(lane, wm * CFG::WTM + i * 32) : 0;
#pragma unroll
    for (int j = 0; j < TN; ++j) boff[j] = BKM ? stage_frag_off<BN * ES>(lane, wn * CFG::WTN + j * 32) : 0;
    // A stage's products of the wave's first R row blocks.
    auto compute = [&](int buf, auto r_c) {
      constexpr int R = decltype(r_c)::value;
      F fa[R], fb[TN];
      const char* As = lds + buf * CFG::STAGE;
      const char* Bs = As + BM * ROWB;
#pragma unroll
      for (int g = 0; g < CFG::NG; ++g) {
        if constexpr (!AKM)
          load_frags<T, R, TN, ROWB, !BKM>(As + (wm * CFG::WTM) * ROWB, Bs + (wn * CFG::WTN) * ROWB, lane, g, fa, fb);
        else if constexpr (ES == 2)
          load_b_kmajor<T, R, BM * ES>(As, aoff, g, fa);
        else
          load_b_kmajor_f32<R, BM * ES>(As, lane, wm * CFG::WTM, g, fa);
        if constexpr (BKM && ES == 2)
          load_b_kmajor<T, TN, BN * ES>(Bs, boff, g, fb);
        else if constexpr (BKM)
          load_b_kmajor_f32<TN, BN * ES>(Bs, lane, wn * CFG::WTN, g, fb);
        mma<T, R, TN>(fa, fb, reinterpret_cast<f32x16(&)[R][TN]>(acc));
      }
    };
    // the wave's row blocks that hold any row: fp32 products of few rows are bound by MFMAs
    const int nb = (x.m - x.row0 - wm * CFG::WTM + 31) / 32;
    auto products = [&](int buf) {
      if constexpr (AKM && ES == 2) {
        if (nb > 0) compute(buf, std::integral_constant<int, TM>{});
      } else {
        if (nb >= TM) compute(buf, std::integral_constant<int, TM>{});
        else if (nb > 0) compute(buf, std::integral_constant<int, 1>{});
      }
    };
    if constexpr (G > 1) {
      if (part < nk) load_stage(part);
      for (int kt = part; kt < nk; kt += G) {
        store_stage(0, kt);
        __builtin_amdgcn_wave_barrier();
        if (kt + G < nk) load_stage(kt + G);
        products(0);
        __builtin_amdgcn_wave_barrier();
      }
      expert_store_split<MODE, T, CFG, G>(p, x, lds_all, acc, lane);
      continue;
    }
    if (nk) {
      load_stage(0);
      store_stage(0, 0);
      __syncthreads();
    }
    for (int kt = 0; kt < nk; ++kt) {
      if (kt + 1 < nk) load_stage(kt + 1);
      products(kt & 1);
      if (kt + 1 < nk) store_stage((kt & 1) ^ 1, kt + 1);
      __syncthreads();
    }
    expert_store<MODE, T, CFG>(p, x, lds, acc, lane);
  }
}

}  // namespace mns
