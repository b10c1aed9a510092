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

#include "norm.hpp"

namespace mns {

constexpr int EXPERT_MAX = 1024;

// Which product: forward, input gradient, weight gradient.
enum { EX_FWD = 0, EX_DX = 1, EX_DW = 2 };

struct ExpertArgs {
  const char* A; int64_t lda, sA;   // elements; s: matrix stride of W, unused for row operands
  const char* B; int64_t ldb, sB;
  char* C; int64_t ldc, sC;
  const int32_t* offsets;
  int experts;
  int64_t rows;                     // S
  int n;                            // columns of C (extent of j)
  int m, k;                         // extents of i / of the contraction, where fixed
  int tiles_n;
  int c_vec;                        // 16-byte stores fit C
};

// Beginning and end of expert e's rows; e = E: the rows of nobody.
__device__ inline void expert_rows(const ExpertArgs& p, int e, int* lo, int* hi) {
  const int rows = (int)p.rows, a = p.offsets[e], b = e < p.experts ? p.offsets[e + 1] : rows;
  *lo = min(max(a, 0), rows);
  *hi = min(max(b, *lo), rows);
}

// first[e] = tile rows (of BM) of the experts before e, e = 0 .. E + 1: entry E begins the tile
// rows over the rows of nobody, entry E + 1 is the total. Ends with a barrier.
template <int NT, int BM>
__device__ inline void expert_tiles(const ExpertArgs& p, int* first, int* wsum) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  int base = 0;
  for (int e0 = 0; e0 <= p.experts; e0 += NT) {
    const int e = e0 + threadIdx.x;
    int n = 0;
    if (e <= p.experts) {
      int lo, hi;
      expert_rows(p, e, &lo, &hi);
      n = (hi - lo + BM - 1) / BM;
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
    if (e <= p.experts) first[e] = before + run - n;
    if (e == p.experts) first[e + 1] = before + run;
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
};

// 16 bytes of an operand row: elements e0 .. of a row `len` long, zero past the end.
template <typename T, bool VEC>
__device__ inline u32x4 load_chunk(const T* row, int e0, int len) {
  constexpr int N = 16 / (int)sizeof(T);
  if constexpr (VEC) {
    return e0 < len ? *reinterpret_cast<const u32x4*>(row + e0) : u32x4{0, 0, 0, 0};
  } else {
    typedef T TN __attribute__((ext_vector_type(N)));
    TN v;
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = e0 + e < len ? row[e0 + e] : (T)0.f;
    return __builtin_bit_cast(u32x4, v);
  }
}

// The part of the launch's tile list that one XCD takes (an eighth, so that neighbouring tiles
// share an L2), for the workgroups on it to walk side by side. When the last round of whole tiles
// would leave half of them idle or more, its tiles are cut into an upper and a lower half: the
// round then takes about 0.6 of a whole one (a half tile still brings all of its columns of W).
struct ExpertList {
  int64_t lo;       // first tile
  int64_t whole;    // whole tiles, then
  int64_t n;        // all pieces
};
template <int MODE, class CFG>
__device__ inline ExpertList expert_list(const ExpertArgs& p, const int* first) {
  const int64_t total = (int64_t)p.tiles_n * (MODE == EX_DW ? p.experts * ((p.m + CFG::BM - 1) / CFG::BM) : wave_uniform(first[p.experts + 1]));
  const int xcd = blockIdx.x & 7, wgs = gridDim.x >> 3;
  ExpertList l;
  l.lo = total * xcd / 8;
  l.n = l.whole = total * (xcd + 1) / 8 - l.lo;
  const int rest = (int)(l.n % wgs);
  if (2 * rest <= wgs) {
    l.whole -= rest;
    l.n += rest;
  }
  return l;
}

// Piece t of an XCD's list. Tiles go expert by expert, within one in bands of EXPERT_BAND tile
// rows, down a band, then one tile column right, so that the tiles that run together share panels
// of both operands in L2.
constexpr int EXPERT_BAND = 8;
template <int MODE, typename T, class CFG>
__device__ inline ExpertTile expert_tile(const ExpertArgs& p, const int* first, const ExpertList& l, int64_t t) {
  const int half = t < l.whole ? 0 : 1 + (int)((t - l.whole) & 1);   // 0: whole, 1: upper, 2: lower
  t = l.lo + (half ? l.whole + ((t - l.whole) >> 1) : t);
  constexpr int ES = sizeof(T);
  ExpertTile x;
  int e, r, tm;
  if constexpr (MODE == EX_DW) {
    tm = (p.m + CFG::BM - 1) / CFG::BM;
    e = (int)(t / (tm * p.tiles_n));
    r = (int)(t - (int64_t)e * tm * p.tiles_n);
  } else {
    // the expert whose tiles hold t
    e = 0;
    int top = p.experts;
    while (e < top) {
      const int mid = (e + top + 1) >> 1;
      if ((int64_t)wave_uniform(first[mid]) * p.tiles_n <= t) e = mid; else top = mid - 1;
    }
    const int f = wave_uniform(first[e]);
    tm = wave_uniform(first[e + 1]) - f;
    r = (int)(t - (int64_t)f * p.tiles_n);
  }
  int lo, hi;
  expert_rows(p, e, &lo, &hi);
  lo = wave_uniform(lo);
  hi = wave_uniform(hi);
  const int band = r / (EXPERT_BAND * p.tiles_n), high = min(tm - band * EXPERT_BAND, EXPERT_BAND);
  r -= band * EXPERT_BAND * p.tiles_n;
  x.row0 = (band * EXPERT_BAND + r % high) * CFG::BM;
  x.col0 = (r / high) * CFG::BN;
  x.a = p.A + (int64_t)lo * p.lda * ES;
  if constexpr (MODE == EX_DW) {
    x.m = p.m;
    x.k = hi - lo;
    x.b = p.B + (int64_t)lo * p.ldb * ES;
    x.c = p.C + (int64_t)e * p.sC * ES;
  } else {
    x.m = hi - lo;
    x.k = e < p.experts ? p.k : 0;
    x.b = p.B + (int64_t)(e < p.experts ? e : 0) * p.sB * ES;
    x.c = p.C + (int64_t)lo * p.ldc * ES;
  }
  if (half == 1) x.m = min(x.m, x.row0 + CFG::BM / 2);
  if (half == 2) {
    x.row0 += CFG::BM / 2;
    if (x.row0 >= x.m) x.k = 0;   // nothing there: nothing is read, and no store is in range
  }
  return x;
}

// Accumulators to C: through an fp32 slab in LDS, whole rows of 16-byte vectors out.
template <typename T, class CFG>
__device__ inline void expert_store(const ExpertArgs& p, const ExpertTile& x, char* lds, const f32x16 (&acc)[CFG::TM][CFG::TN], int lane) {
  constexpr int BN = CFG::BN, NT = CFG::NT, WTM = CFG::WTM, CP = CFG::CP;
  constexpr int SR = CFG::SR, SROWS = SR * WTM, VPR = BN / 8;
  const int wave = wave_uniform(threadIdx.x >> 6), tid = wave * 64 + lane;
  const int wm = wave / CFG::WVN, wn = wave % CFG::WVN;
  constexpr int DT = sizeof(T) == 4 ? F32 : (__is_same(T, __bf16) ? BF16 : F16);
  float* Cs = reinterpret_cast<float*>(lds);
  for (int sl = 0; sl < CFG::WVM / SR; ++sl) {
    if (wm / SR == sl) acc_to_slab<CFG>(Cs, acc, lane, wn, (wm % SR) * WTM);
    lds_barrier();
#pragma unroll 1
    for (int idx = tid; idx < SROWS * VPR; idx += NT) {
      const int lr = idx / VPR, lc = (idx - lr * VPR) * 8;
      const int r = x.row0 + sl * SROWS + lr, c = x.col0 + lc;
      if (r < x.m && c < p.n) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(Cs + lr * CP + lc);
        const f32x4 b = *reinterpret_cast<const f32x4*>(Cs + lr * CP + lc + 4);
        const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
        T* out = reinterpret_cast<T*>(x.c) + (int64_t)r * p.ldc;
        if (p.c_vec && c + 8 <= p.n) {
          VecIO<T>::store(out, c, v);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c + e < p.n) store_elem(out, DT, c + e, v[e]);
        }
      }
    }
    lds_barrier();
  }
}

// Operands staged through registers: every type and any alignment (VEC: rows of whole 16-byte
// chunks). 128 x 128 tiles of 4 waves.
template <int MODE, typename T, bool VEC, class CFG>
__global__ void __launch_bounds__(CFG::NT, CFG::OCC) expert_gemm_staged(const ExpertArgs p) {
  constexpr int ES = sizeof(T), BM = CFG::BM, BN = CFG::BN, NT = CFG::NT, KB = CFG::KB, ROWB = CFG::ROWB;
  constexpr int EPC = 16 / ES, BK = KB / ES, CPR = CFG::CPR, TM = CFG::TM, TN = CFG::TN;
  constexpr bool AKM = MODE == EX_DW, BKM = MODE != EX_FWD;
  constexpr int CPM = BM * ES / 16, CPN = BN * ES / 16;   // chunks per contraction-major row
  __shared__ __align__(16) char lds[CFG::LDS];
  __shared__ int first[EXPERT_MAX + 2];
  __shared__ int wsum[NT / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_uniform(tid >> 6);
  const int wm = wave / CFG::WVN, wn = wave % CFG::WVN;
  if constexpr (MODE != EX_DW) expert_tiles<NT, BM>(p, first, wsum);
  const ExpertList l = expert_list<MODE, CFG>(p, first);
  for (int64_t t = blockIdx.x >> 3; t < l.n; t += gridDim.x >> 3) {
    const ExpertTile x = expert_tile<MODE, T, CFG>(p, first, l, t);
    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    const T* A = reinterpret_cast<const T*>(x.a);
    const T* B = reinterpret_cast<const T*>(x.b);
    u32x4 ra[CFG::CA], rb[CFG::CB];
    const u32x4 zero = {0, 0, 0, 0};
    auto load_stage = [&](int k0) {
#pragma unroll
      for (int q = 0; q < CFG::CA; ++q) {
        const int c = tid + NT * q;
        if constexpr (AKM) {
          const int k = k0 + c / CPM, i = x.row0 + (c % CPM) * EPC;
          ra[q] = k < x.k ? load_chunk<T, VEC>(A + (int64_t)k * p.lda, i, x.m) : zero;
        } else {
          const int i = x.row0 + c / CPR;
          ra[q] = i < x.m ? load_chunk<T, VEC>(A + (int64_t)i * p.lda, k0 + (c % CPR) * EPC, x.k) : zero;
        }
      }
#pragma unroll
      for (int q = 0; q < CFG::CB; ++q) {
        const int c = tid + NT * q;
        if constexpr (BKM) {
          const int k = k0 + c / CPN, j = x.col0 + (c % CPN) * EPC;
          rb[q] = k < x.k ? load_chunk<T, VEC>(B + (int64_t)k * p.ldb, j, p.n) : zero;
        } else {
          const int j = x.col0 + c / CPR;
          rb[q] = j < p.n ? load_chunk<T, VEC>(B + (int64_t)j * p.ldb, k0 + (c % CPR) * EPC, x.k) : zero;
        }
      }
    };
    auto store_stage = [&](int buf) {
      char* As = lds + buf * CFG::STAGE;
      char* Bs = As + BM * ROWB;
#pragma unroll
      for (int q = 0; q < CFG::CA; ++q) {
        const int c = tid + NT * q;
        if constexpr (AKM)
          *reinterpret_cast<u32x4*>(As + (c / CPM) * (BM * ES) + (((c % CPM) ^ kmajor_swizzle((c / CPM) & 3)) << 4)) = ra[q];
        else
          *reinterpret_cast<u32x4*>(As + (c / CPR) * ROWB + (c % CPR) * 16) = ra[q];
      }
#pragma unroll
      for (int q = 0; q < CFG::CB; ++q) {
        const int c = tid + NT * q;
        if constexpr (BKM)
          *reinterpret_cast<u32x4*>(Bs + (c / CPN) * (BN * ES) + (((c % CPN) ^ kmajor_swizzle((c / CPN) & 3)) << 4)) = rb[q];
        else
          *reinterpret_cast<u32x4*>(Bs + (c / CPR) * ROWB + (c % CPR) * 16) = rb[q];
      }
    };
    typedef typename Frag<T>::type F;
    F fa[TM], fb[TN];
    int aoff[TM], boff[TN];
#pragma unroll
    for (int i = 0; i < TM; ++i) aoff[i] = AKM ? kmajor_frag_off<BM * ES>(lane, wm * CFG::WTM + i * 32) : 0;
#pragma unroll
    for (int j = 0; j < TN; ++j) boff[j] = BKM ? kmajor_frag_off<BN * ES>(lane, wn * CFG::WTN + j * 32) : 0;
    const int nk = (x.k + BK - 1) / BK;
    if (nk) {
      load_stage(0);
      store_stage(0);
      __syncthreads();
    }
    for (int kt = 0; kt < nk; ++kt) {
      if (kt + 1 < nk) load_stage((kt + 1) * BK);
      const char* As = lds + (kt & 1) * CFG::STAGE;
      const char* Bs = As + BM * ROWB;
#pragma unroll
      for (int g = 0; g < CFG::NG; ++g) {
        if constexpr (!AKM)
          load_frags<T, TM, TN, ROWB, !BKM>(As + (wm * CFG::WTM) * ROWB, Bs + (wn * CFG::WTN) * ROWB, lane, g, fa, fb);
        else if constexpr (ES == 2)
          load_b_kmajor<T, TM, BM * ES>(As, aoff, g, fa);
        else
          load_b_kmajor_f32<TM, BM * ES>(As, lane, wm * CFG::WTM, g, fa);
        if constexpr (BKM && ES == 2)
          load_b_kmajor<T, TN, BN * ES>(Bs, boff, g, fb);
        else if constexpr (BKM)
          load_b_kmajor_f32<TN, BN * ES>(Bs, lane, wn * CFG::WTN, g, fb);
        mma<T, TM, TN>(fa, fb, acc);
      }
      if (kt + 1 < nk) store_stage((kt & 1) ^ 1);
      __syncthreads();
    }
    expert_store<T, CFG>(p, x, lds, acc, lane);
  }
}

// ---------------------------------------------------------------- large products, 16-bit types
// 256 x 256 tiles, 16 waves of 64 x 64 at four per SIMD, operands DMA'd global -> LDS into a ring
// of two 128-byte (64-element) stages, as the Newton-Schulz products. The tiles of a workgroup
// form one stream of stages: the next tile's first stage is on its way during this tile's last
// one and its stores, so a tile pays neither a first wait nor an epilogue in LDS. The stores
// leave the registers directly: the MFMAs run with the operands swapped, so a lane holds runs of
// four columns of one row, and one swap of lane halves makes them 16 bytes.

// A value the compiler cannot see through: what is computed from it is computed where it stands
// and not kept in registers across the loops.
__device__ inline int opaque(int v) {
  __asm__ __volatile__("" : "+v"(v));
  return v;
}

// acc[i][j] += B_j A_i^T: lane (l, h) register r holds row 32 i + l, column 32 j + 8 (r / 4) + 4 h + r % 4.
template <typename T, int TM, int TN>
__device__ inline void mma_swapped(const typename Frag<T>::type (&a)[TM], const typename Frag<T>::type (&b)[TN], f32x16 (&acc)[TM][TN]) {
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      if constexpr (__is_same(T, __bf16)) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[j], a[i], acc[i][j], 0, 0, 0);
      else acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(b[j], a[i], acc[i][j], 0, 0, 0);
    }
}

// The fragments of one k-group: two 32-row blocks of either operand, from a contraction-major
// stage (KM: two transposing reads a block, see load_b_kmajor) or a contraction-contiguous one (a
// 16-byte read a block). Reads and their wait stand in one block: for reads that it can see, the
// compiler waits for the whole DMA queue first, because the next stage's DMA writes the same
// array (2048 x 7168, 27 experts, 32768 rows: 1100 us with such waits).
template <typename T, bool AKM, bool BKM, int RBA, int RBB, int NEXT>
__device__ inline void load_frags_asm(unsigned a0, unsigned a1, unsigned b0, unsigned b1, typename Frag<T>::type (&a)[2],
                                      typename Frag<T>::type (&b)[2]) {
  typedef typename Frag<T>::type F;
  auto join = [](s16x4 lo, s16x4 hi) {
    return __builtin_bit_cast(F, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  if constexpr (AKM && BKM) {
    s16x4 al0, ah0, al1, ah1, bl0, bh0, bl1, bh1;
    __asm__ __volatile__(
        "ds_read_b64_tr_b16 %0, %8\n\t"
        "ds_read_b64_tr_b16 %1, %8 offset:%12\n\t"
        "ds_read_b64_tr_b16 %2, %9\n\t"
        "ds_read_b64_tr_b16 %3, %9 offset:%12\n\t"
        "ds_read_b64_tr_b16 %4, %10\n\t"
        "ds_read_b64_tr_b16 %5, %10 offset:%13\n\t"
        "ds_read_b64_tr_b16 %6, %11\n\t"
        "ds_read_b64_tr_b16 %7, %11 offset:%13\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(al0), "=&v"(ah0), "=&v"(al1), "=&v"(ah1), "=&v"(bl0), "=&v"(bh0), "=&v"(bl1), "=&v"(bh1)
        : "v"(a0), "v"(a1), "v"(b0), "v"(b1), "i"(4 * RBA), "i"(4 * RBB)
        : "memory");
    a[0] = join(al0, ah0);
    a[1] = join(al1, ah1);
    b[0] = join(bl0, bh0);
    b[1] = join(bl1, bh1);
  } else if constexpr (BKM) {
    s16x4 bl0, bh0, bl1, bh1;
    __asm__ __volatile__(
        "ds_read_b128 %0, %6\n\t"
        "ds_read_b128 %1, %6 offset:%9\n\t"
        "ds_read_b64_tr_b16 %2, %7\n\t"
        "ds_read_b64_tr_b16 %3, %7 offset:%10\n\t"
        "ds_read_b64_tr_b16 %4, %8\n\t"
        "ds_read_b64_tr_b16 %5, %8 offset:%10\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(a[0]), "=&v"(a[1]), "=&v"(bl0), "=&v"(bh0), "=&v"(bl1), "=&v"(bh1)
        : "v"(a0), "v"(b0), "v"(b1), "i"(NEXT), "i"(4 * RBB)
        : "memory");
    b[0] = join(bl0, bh0);
    b[1] = join(bl1, bh1);
  } else {
    __asm__ __volatile__(
        "ds_read_b128 %0, %4\n\t"
        "ds_read_b128 %1, %4 offset:%6\n\t"
        "ds_read_b128 %2, %5\n\t"
        "ds_read_b128 %3, %5 offset:%6\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(a[0]), "=&v"(a[1]), "=&v"(b[0]), "=&v"(b[1])
        : "v"(a0), "v"(b0), "i"(NEXT)
        : "memory");
  }
}

// Accumulators to C: 16-byte stores, 32 contiguous bytes of 32 rows each. Rows and columns past
// the end fall to the buffer's range check, so every wave issues TM * TN * 2 stores whatever its
// tile (the stage stream counts them).
template <typename T, class CFG>
__device__ inline void expert_store_direct(const ExpertArgs& p, const ExpertTile& x, const f32x16 (&acc)[CFG::TM][CFG::TN], int lane, int wm, int wn) {
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(x.c + ((int64_t)x.row0 * p.ldc + x.col0) * 2, 0x7ffffff0u);
  const int h = lane >> 5;
#pragma unroll
  for (int i = 0; i < CFG::TM; ++i) {
    const int r = wm * CFG::WTM + i * 32 + (lane & 31);
    const bool rin = x.row0 + r < x.m;
#pragma unroll
    for (int j = 0; j < CFG::TN; ++j)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int c = wn * CFG::WTN + j * 32 + q * 16 + h * 8;
        uint32_t w[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 2; ++e) w[u][e] = pack2<T>(acc[i][j][q * 8 + u * 4 + 2 * e], acc[i][j][q * 8 + u * 4 + 2 * e + 1]);
        const auto s0 = __builtin_amdgcn_permlane32_swap(w[0][0], w[1][0], false, false);
        const auto s1 = __builtin_amdgcn_permlane32_swap(w[0][1], w[1][1], false, false);
        const u32x4 v = {s0[0], s1[0], s0[1], s1[1]};
        const uint32_t off = rin && x.col0 + c < p.n ? (uint32_t)(r * (int)p.ldc + c) * 2 : OOB;
        __builtin_amdgcn_raw_buffer_store_b128(v, rs, off, 0, 0);
      }
  }
}

template <int MODE, typename T, class CFG>
__global__ void __launch_bounds__(CFG::NT, CFG::OCC) expert_gemm_dma(const ExpertArgs p) {
  constexpr int ES = 2, BM = CFG::BM, BN = CFG::BN, NT = CFG::NT, KB = CFG::KB;
  constexpr int BK = KB / ES, CPR = CFG::CPR, TM = CFG::TM, TN = CFG::TN, STG = CFG::STG;
  constexpr bool AKM = MODE == EX_DW, BKM = MODE != EX_FWD;
  constexpr int NWAVE = NT / 64;
  constexpr int AW = NWAVE * BM / (BM + BN);           // waves that bring A; the others bring B
  constexpr int D = (BM + BN) * KB / 1024 / NWAVE;     // 1 KB pieces a wave brings per stage
  constexpr int STORES = TM * TN * 2;
  static_assert(sizeof(T) == 2 && TM == 2 && TN == 2 && CPR == 8 && CFG::NST == 2, "tile");
  static_assert(AW * D * 1024 == BM * KB && (NWAVE - AW) * D * 1024 == BN * KB, "pieces divide over the waves");
  static_assert(D % 4 == 0, "a wave's pieces begin at a multiple of four");
  __shared__ __align__(1024) char lds[2 * STG];
  __shared__ int first[EXPERT_MAX + 2];
  __shared__ int wsum[NWAVE];
  const int wave = wave_uniform(threadIdx.x >> 6);
  const int wm = wave / CFG::WVN, wn = wave % CFG::WVN;
  const int lane0 = threadIdx.x & 63;
  if constexpr (MODE != EX_DW) expert_tiles<NT, BM>(p, first, wsum);
  const ExpertList l = expert_list<MODE, CFG>(p, first);
  const int64_t step = gridDim.x >> 3;
  int64_t t = blockIdx.x >> 3;
  if (t >= l.n) return;

  // what this wave brings of the tile whose stages are being issued: where its operand begins,
  // bytes from one contraction index to the next, and per piece the lane's offset (past the
  // range where it lies outside) and contraction index within the stage
  const bool isa = wave < AW;
  const int piece0 = (isa ? wave : wave - AW) * D;
  char* const dst = lds + (isa ? 0 : BM * KB) + piece0 * 1024;
  const char* src = nullptr;
  int64_t kstep = 0;
  uint32_t goff[D];
  int kin[D];
  int klen = 0;
  auto aim = [&](const ExpertTile& x) {
    const bool km = isa ? AKM : BKM;
    const int64_t ld = isa ? p.lda : p.ldb;
    const int lo = isa ? x.row0 : x.col0, ext = (isa ? x.m : p.n) - lo;   // extent of i or j from the tile on
    klen = x.k;
    kstep = km ? ld * ES : ES;
    src = (isa ? x.a : x.b) + (km ? (int64_t)lo * ES : (int64_t)lo * ld * ES);
    const int lane = opaque(lane0);
#pragma unroll
    for (int j = 0; j < D; ++j) {
      if (km) {
        constexpr int CPK = BM * ES / 16;                // chunks of a contraction row (BM = BN)
        const int k = (piece0 + j) * (1024 / (BM * ES)) + lane / CPK;
        const int c = ((lane % CPK) ^ kmajor_swizzle(k & 3)) * 8;
        kin[j] = k;
        goff[j] = c < ext ? (uint32_t)(k * (int)ld + c) * ES : OOB;
      } else {
        const int r = (piece0 + j) * 8 + lane / CPR;
        const int c = ((lane % CPR) ^ chunk_swizzle<CPR>(r)) * 8;
        kin[j] = c;
        goff[j] = r < ext ? (uint32_t)(r * (int)ld + c) * ES : OOB;
      }
    }
  };
  static_assert(BM == BN, "one row length of the contraction-major stages");
  auto issue = [&](int k0, int slot) {
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(src + k0 * kstep, 0x7ffffff0u);
#pragma unroll
    for (int j = 0; j < D; ++j) dma16(rs, dst + slot * STG + j * 1024, k0 + kin[j] < klen ? goff[j] : OOB);
  };

  typedef __attribute__((address_space(3))) const char* lds_ptr;
  typename Frag<T>::type fa[TM], fb[TN];
  f32x16 acc[TM][TN];
  // one stage: all but its last group's products; that group's fragments stay in fa, fb
  auto stage = [&](int s) {
    const unsigned sb = (unsigned)(size_t)(lds_ptr)lds + s * STG;
    const int lane = opaque(lane0);
    // block 0 and 1 of either operand, k-group 0; a contraction-major group is 16 rows further,
    // a contiguous one two chunks, whose place depends on the row
    const unsigned a0 = sb + (AKM ? kmajor_frag_off<BM * ES>(lane, wm * CFG::WTM) : (wm * CFG::WTM + (lane & 31)) * KB);
    const unsigned a1 = AKM ? sb + kmajor_frag_off<BM * ES>(lane, wm * CFG::WTM + 32) : 0u;
    const unsigned bb = sb + BM * KB;
    const unsigned b0 = bb + (BKM ? kmajor_frag_off<BN * ES>(lane, wn * CFG::WTN) : (wn * CFG::WTN + (lane & 31)) * KB);
    const unsigned b1 = BKM ? bb + kmajor_frag_off<BN * ES>(lane, wn * CFG::WTN + 32) : 0u;
    const int sw = chunk_swizzle<CPR>(lane & 31);
#pragma unroll
    for (int g = 0; g < CFG::NG; ++g) {
      const unsigned ck = ((2 * g + (lane >> 5)) ^ sw) << 4;
      load_frags_asm<T, AKM, BKM, BM * ES, BN * ES, 32 * KB>(a0 + (AKM ? 16 * g * BM * ES : ck), a1 + 16 * g * BM * ES,
                                                             b0 + (BKM ? 16 * g * BN * ES : ck), b1 + 16 * g * BN * ES, fa, fb);
      if (g + 1 < CFG::NG) mma_swapped<T, TM, TN>(fa, fb, acc);
    }
  };

  ExpertTile x = expert_tile<MODE, T, CFG>(p, first, l, t);
  aim(x);
  int slot = 0;                      // of the tile's first stage
  if (x.k > 0) issue(0, 0);
  bool begin = true;
  for (;;) {
    const int nk = (x.k + BK - 1) / BK;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    if (nk) {
      // this tile's first stage: only the stores of the tile before it were issued after it
      if (begin) wait_vmcnt<0>(); else wait_vmcnt<STORES>();
      barrier_nofence();
    }
    // a wave whose rows all lie outside only brings operands
    const bool busy = x.row0 + wm * CFG::WTM < x.m;
    for (int kt = 0; kt + 1 < nk; ++kt) {
      // the last group of the stage before, whose fragments were read before the barrier
      if (kt && busy) mma_swapped<T, TM, TN>(fa, fb, acc);
      issue((kt + 1) * BK, (slot + kt + 1) & 1);
      if (busy) stage((slot + kt) & 1);
      wait_vmcnt<0>();
      barrier_nofence();
      if (busy) pin_frags<T, TM, TN>(fa, fb);
    }
    if (nk > 1 && busy) mma_swapped<T, TM, TN>(fa, fb, acc);
    // the last stage, and the next tile's first one into the slot before it
    const ExpertTile now = x;
    const int last = slot + nk - 1;
    slot = (slot + nk) & 1;
    t += step;
    const bool more = t < l.n;
    if (more) {
      x = expert_tile<MODE, T, CFG>(p, first, l, t);
      aim(x);
      if (x.k > 0) issue(0, slot);
    }
    if (nk) {
      if (busy) stage(last & 1);
      barrier_nofence();
      if (busy) {
        pin_frags<T, TM, TN>(fa, fb);
        mma_swapped<T, TM, TN>(fa, fb, acc);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    expert_store_direct<T, CFG>(p, now, acc, opaque(lane0), wm, wn);
    __builtin_amdgcn_sched_barrier(0);
    if (!more) break;
    begin = false;
  }
}

}  // namespace mns
