// Host side of the layer operators of include/muon_ns.h: layer norm, rows sorted by expert and
// the experts' matrix products, each with its gradient. As in muon_ns.hip, validation happens
// before any HIP call and a call only enqueues kernels on the caller's stream.

#include "muon_ns.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../host.hpp"
#include "expert_few.hpp"
#include "expert_gemm.hpp"
#include "expert_pingpong.hpp"
#include "norm.hpp"
#include "overlap.hpp"
#include "rows.hpp"

using namespace mns;

namespace {

constexpr int64_t kMaxRows = 1 << 24, kMaxCols = 1 << 20;

// A buffer of rows: like the matrices of the Newton-Schulz calls, but zero rows are allowed and
// offsets may pass 32 bits.
int check_rows(const mns_tensor* t) {
  if (!t) return MNS_ERR_ARG;
  if (!valid_dtype(t->dtype)) return MNS_ERR_DTYPE;
  if (t->batch < 1 || t->rows < 0 || t->cols < 1) return MNS_ERR_SHAPE;
  if (t->batch > kMaxRows || t->rows > kMaxRows || t->batch * t->rows > kMaxRows) return MNS_ERR_SHAPE;
  if (t->cols > kMaxCols || t->ld < t->cols || t->ld > kMaxCols) return MNS_ERR_SHAPE;
  if (t->batch > 1 && (t->stride < t->rows * t->ld || t->stride > (int64_t(1) << 40))) return MNS_ERR_SHAPE;
  if (!t->ptr && t->rows > 0) return MNS_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(t->ptr) % dtype_size(t->dtype)) return MNS_ERR_ARG;
  return MNS_OK;
}

Span span(const mns_tensor* t) { return mns::span(t, dtype_size(t->dtype)); }
using mns::span;

bool same_rows(const mns_tensor* a, const mns_tensor* b) {
  return a->batch == b->batch && a->rows == b->rows && a->cols == b->cols;
}

// Every row of t begins at a multiple of 16 bytes and is whole 16-byte chunks long.
bool vec_rows(const mns_tensor* t) {
  const int64_t es = dtype_size(t->dtype);
  return reinterpret_cast<uintptr_t>(t->ptr) % 16 == 0 && t->cols * es % 16 == 0 && (t->rows <= 1 || t->ld * es % 16 == 0) &&
         (t->batch == 1 || t->stride * es % 16 == 0);
}
bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// f(element of the buffer's type) for a runtime dtype.
template <class F>
int by_type(int dt, F&& f) {
  if (dt == F32) return f(float{});
  if (dt == BF16) return f(__bf16{});
  return f(_Float16{});
}

// At least n workgroups of up to 1024 threads, numbered by block_id().
dim3 grid_of(int64_t n) {
  const int64_t x = std::min<int64_t>(n, 1 << 21);
  return dim3((unsigned)x, (unsigned)((n + x - 1) / x));
}

hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

// ------------------------------------------------------------------------------- layer norm

RowsRef rows_ref(const mns_tensor* t) { return {reinterpret_cast<char*>(t->ptr), std::max<int64_t>(t->rows, 1), t->ld, t->stride}; }

// The affine parameters' type: the rows' own or fp32.
int check_wdtype(const mns_tensor* x, int32_t wdtype) {
  if (!valid_dtype(wdtype)) return MNS_ERR_DTYPE;
  return wdtype == x->dtype || wdtype == F32 ? MNS_OK : MNS_ERR_DTYPE;
}

// Columns that NT threads of VPT pieces hold.
constexpr int held(int nt, int vpt) { return nt * vpt * 8; }
constexpr int kNormHeld = held(1024, 2);   // longer rows take the kernels that read them again

// Workgroups that share the rows of a backward pass, each with a part of dweight and dbias: enough
// to fill the chip (two of 512 threads a CU, or four of 256 where rows are short), but at least
// four turns of rows each once every CU has one, because each part costs as much traffic as two
// fp32 rows (1021 x 2047 fp32 with a part a row: 12 us and 8 for the parts' sum; four rows a part:
// 12 and 4).
int norm_parts(int64_t rows, int64_t cols) {
  const int64_t turns = cols <= held(64, 2) ? (rows + 3) / 4 : rows;   // four rows at a time where a wave holds one
  const int64_t most = cols <= held(256, 1) ? 1024 : 512;
  return (int)std::max<int64_t>(1, turns <= 256 ? turns : std::min(most, std::max<int64_t>(256, turns / 4)));
}

template <typename T, typename WT, bool VEC>
void launch_norm_fwd(const NormArgs& a, hipStream_t s) {
  const dim3 one = grid_of(a.rows), four = grid_of((a.rows + 3) / 4);
  if (a.cols <= held(64, 1)) hipLaunchKernelGGL((norm_fwd_row<T, WT, 64, 1, VEC>), four, dim3(256), 0, s, a);
  else if (a.cols <= held(64, 2)) hipLaunchKernelGGL((norm_fwd_row<T, WT, 64, 2, VEC>), four, dim3(256), 0, s, a);
  else if (a.cols <= held(64, 4)) hipLaunchKernelGGL((norm_fwd_row<T, WT, 64, 4, VEC>), four, dim3(256), 0, s, a);
  else if (a.cols <= held(256, 2)) hipLaunchKernelGGL((norm_fwd_row<T, WT, 256, 2, VEC>), one, dim3(256), 0, s, a);
  else if (a.cols <= held(256, 4)) hipLaunchKernelGGL((norm_fwd_row<T, WT, 256, 4, VEC>), one, dim3(256), 0, s, a);
  else if (a.cols <= held(1024, 2)) hipLaunchKernelGGL((norm_fwd_row<T, WT, 1024, 2, VEC>), one, dim3(1024), 0, s, a);
  else hipLaunchKernelGGL((norm_fwd_any<T, WT>), one, dim3(256), 0, s, a);
}

template <typename T, typename WT, bool VEC>
void launch_norm_bwd(const NormArgs& a, hipStream_t s) {
  const dim3 g((unsigned)a.nparts);
  if (a.cols <= held(64, 1)) hipLaunchKernelGGL((norm_bwd_row<T, WT, 64, 1, VEC>), g, dim3(256), 0, s, a);
  else if (a.cols <= held(64, 2)) hipLaunchKernelGGL((norm_bwd_row<T, WT, 64, 2, VEC>), g, dim3(256), 0, s, a);
  else if (a.cols <= held(256, 1)) hipLaunchKernelGGL((norm_bwd_row<T, WT, 256, 1, VEC>), g, dim3(256), 0, s, a);
  else if (a.cols <= held(256, 2)) hipLaunchKernelGGL((norm_bwd_row<T, WT, 256, 2, VEC>), g, dim3(256), 0, s, a);
  else if (a.cols <= held(512, 2)) {
    // wider elements, or single ones, need the registers of two pieces for one
    if constexpr (VEC && sizeof(T) == 2) hipLaunchKernelGGL((norm_bwd_row<T, WT, 512, 2, VEC>), g, dim3(512), 0, s, a);
    else hipLaunchKernelGGL((norm_bwd_row<T, WT, 1024, 1, VEC>), g, dim3(1024), 0, s, a);
  } else hipLaunchKernelGGL((norm_bwd_row<T, WT, 1024, 2, VEC>), g, dim3(1024), 0, s, a);
}

template <class F>
int by_norm_types(int dt, int wdt, F&& f) {
  return by_type(dt, [&](auto x) {
    if (wdt == F32) return f(x, float{});
    return f(x, x);
  });
}

// ------------------------------------------------------------------------------------- rows

int check_rank(const int32_t* rank, int64_t tokens, int32_t k) {
  if (k < 1 || k > kMaxCols) return MNS_ERR_SHAPE;
  if (tokens * k > kMaxRows) return MNS_ERR_SHAPE;
  if (tokens && !rank) return MNS_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(rank) % 4) return MNS_ERR_ARG;
  return MNS_OK;
}

int check_experts(const int32_t* offsets, int32_t experts) {
  if (experts < 1 || experts > EXPERT_MAX) return MNS_ERR_SHAPE;
  if (!offsets || reinterpret_cast<uintptr_t>(offsets) % 4) return MNS_ERR_ARG;
  return MNS_OK;
}

// Token side and row side of one routing: T x D and T k x D of one type.
int check_sides(const mns_tensor* tok, const mns_tensor* row, const int32_t* rank, int32_t k) {
  if (int st = check_rows(tok)) return st;
  if (int st = check_rows(row)) return st;
  if (tok->dtype != row->dtype) return MNS_ERR_DTYPE;
  if (tok->batch != 1 || row->batch != 1 || tok->cols != row->cols) return MNS_ERR_SHAPE;
  if (int st = check_rank(rank, tok->rows, k)) return st;
  return row->rows == tok->rows * k ? MNS_OK : MNS_ERR_SHAPE;
}

int64_t row_bytes(const mns_tensor* t) { return t->ld * dtype_size(t->dtype); }

int64_t rank_bytes(int64_t tokens, int32_t k) { return 4 * tokens * k; }

RowsArgs rows_args(const mns_tensor* tok, const int32_t* rank, int32_t k) {
  RowsArgs a{};
  a.rank = rank;
  a.k = k;
  a.tokens = tok->rows;
  a.slots = tok->rows * k;
  return a;
}

// Workgroups of the (token, unit) kernels: at most 2^24 x 2^20 / 256, two dimensions hold them.
dim3 rows_grid(const RowsArgs& a) { return grid_of((a.tokens * a.units + ROWS_NT - 1) / ROWS_NT); }

template <bool WEIGHTED>
int gather(RowsArgs a, const mns_tensor* row, const mns_tensor* tok, hipStream_t s) {
  a.row = reinterpret_cast<const char*>(row->ptr);
  a.row_ld = row_bytes(row);
  a.out = reinterpret_cast<char*>(tok->ptr);
  a.out_ld = row_bytes(tok);
  const bool vec = vec_rows(row) && vec_rows(tok) && tok->cols % 8 == 0;
  a.units = (int)(vec ? tok->cols / 8 : tok->cols);
  const dim3 g = rows_grid(a);
  return by_type(tok->dtype, [&](auto x) {
    using T = decltype(x);
    return launch(K_ROUTE, s, [&] {
      if (vec) hipLaunchKernelGGL((rows_gather<T, 8, WEIGHTED>), g, dim3(ROWS_NT), 0, s, a);
      else hipLaunchKernelGGL((rows_gather<T, 1, WEIGHTED>), g, dim3(ROWS_NT), 0, s, a);
    });
  });
}

struct SortPlan {
  int steps, nblocks;
};
// One workgroup up to 8 steps of each wave; past that 1024 slots a workgroup, at most 256 of them.
SortPlan sort_plan(int64_t slots) {
  const int64_t waves = (slots + SORT_NT - 1) / SORT_NT;   // 64-slot steps per wave of one workgroup
  if (waves <= 8) return {(int)std::max<int64_t>(1, waves), 1};
  const int64_t steps = std::max<int64_t>(2, (waves + 255) / 256);
  return {(int)steps, (int)((waves + steps - 1) / steps)};
}

// ------------------------------------------------------------------------------- the products

int check_product(const mns_tensor* in, const mns_tensor* w, const int32_t* offsets, const mns_tensor* out) {
  for (const mns_tensor* t : {in, w, out})
    if (int st = check_rows(t)) return st;
  if (in->dtype != w->dtype || out->dtype != w->dtype) return MNS_ERR_DTYPE;
  if (w->rows < 1 || w->batch > EXPERT_MAX) return MNS_ERR_SHAPE;
  return check_experts(offsets, (int32_t)w->batch);
}

// Persistent grid: enough workgroups for every tile the rows could make, at most those the chip
// holds at once, the same number on each of the eight XCDs.
template <class CFG>
unsigned gemm_grid(int mode, const ExpertArgs& a, int64_t cols_n) {
  const int64_t tn = (cols_n + CFG::BN - 1) / CFG::BN;
  const int64_t tm = mode == EX_DW ? a.experts * ((a.m + CFG::BM - 1) / CFG::BM)
                                   : (a.rows + CFG::BM - 1) / CFG::BM + std::min<int64_t>(a.experts, a.rows) + 1;
  const int per_cu = std::max(1, std::min((160 * 1024) / (CFG::LDS + 8192), 4 * CFG::OCC / (CFG::NT / 64)));
  const int64_t most = (int64_t)device_cus() * per_cu;
  return (unsigned)(8 * std::max<int64_t>(1, (std::min(tm * tn, most) + 7) / 8));
}

// CHUNK_*: how a product's operand rows are loaded (the row operands' and W's widths, but for the
// contraction of a weight gradient, which runs along the rows).
template <int MODE>
int chunk_fit(const ExpertArgs& a, int dt, bool vec) {
  const int chunk = 16 / (int)dtype_size(dt);
  if (vec) return CHUNK_ALIGNED;
  return (MODE == EX_DW ? a.m : a.k) < chunk || (MODE != EX_FWD && a.n < chunk) ? CHUNK_TINY : CHUNK_ANY;
}

template <int MODE, class CFG>
int run_staged(ExpertArgs a, int dt, bool vec, hipStream_t s) {
  a.tiles_n = (a.n + CFG::BN - 1) / CFG::BN;
  const unsigned g = gemm_grid<CFG>(MODE, a, a.n);
  const int fit = chunk_fit<MODE>(a, dt, vec);
  return by_type(dt, [&](auto x) {
    using T = decltype(x);
    return launch(K_EXPERT_GEMM, s, [&] {
      if (fit == CHUNK_ALIGNED) hipLaunchKernelGGL((expert_gemm_staged<MODE, T, CHUNK_ALIGNED, CFG>), dim3(g), dim3(CFG::NT), 0, s, a);
      else if (fit == CHUNK_ANY) hipLaunchKernelGGL((expert_gemm_staged<MODE, T, CHUNK_ANY, CFG>), dim3(g), dim3(CFG::NT), 0, s, a);
      else hipLaunchKernelGGL((expert_gemm_staged<MODE, T, CHUNK_TINY, CFG>), dim3(g), dim3(CFG::NT), 0, s, a);
    });
  });
}

using Tile64 = TileCfg<64, 64, 1, 1, 128, 1, 2>;

// Few tiles: 64 x 64 ones, each split over eight waves, one workgroup a CU.
template <int MODE>
int run_split(ExpertArgs a, int dt, bool vec, hipStream_t s) {
  constexpr int G = 8;
  a.tiles_n = (a.n + 63) / 64;
  const int64_t tm = MODE == EX_DW ? a.experts * ((a.m + 63) / 64) : a.rows / 64 + std::min<int64_t>(a.experts, a.rows) + 1;
  const dim3 g((unsigned)(8 * ((std::min<int64_t>(tm * a.tiles_n, device_cus()) + 7) / 8)));
  const int fit = chunk_fit<MODE>(a, dt, vec);
  return by_type(dt, [&](auto x) {
    using T = decltype(x);
    return launch(K_EXPERT_GEMM, s, [&] {
      if (fit == CHUNK_ALIGNED) hipLaunchKernelGGL((expert_gemm_staged<MODE, T, CHUNK_ALIGNED, Tile64, G>), g, dim3(64 * G), 0, s, a);
      else if (fit == CHUNK_ANY) hipLaunchKernelGGL((expert_gemm_staged<MODE, T, CHUNK_ANY, Tile64, G>), g, dim3(64 * G), 0, s, a);
      else if constexpr (MODE != EX_FWD)   // whose contraction would be one short row
        hipLaunchKernelGGL((expert_gemm_staged<MODE, T, CHUNK_TINY, Tile64, G>), g, dim3(64 * G), 0, s, a);
    });
  });
}

template <int MODE>
int run_pingpong(ExpertArgs a, int dt, hipStream_t s) {
  a.tiles_n = (a.n + TilePP::BN - 1) / TilePP::BN;
  const unsigned g = gemm_grid<TilePP>(MODE, a, a.n);
  return launch(K_EXPERT_GEMM, s, [&] {
    if (dt == BF16) hipLaunchKernelGGL((expert_gemm_pp<MODE, __bf16>), dim3(g), dim3(TilePP::NT), 0, s, a);
    else hipLaunchKernelGGL((expert_gemm_pp<MODE, _Float16>), dim3(g), dim3(TilePP::NT), 0, s, a);
  });
}

// Few rows: a workgroup per 16 rows of each weight matrix that can have any.
int run_few(const ExpertArgs& a, int dt, bool vec, hipStream_t s) {
  const dim3 g((a.n + 15) / 16, (unsigned)std::min<int64_t>(a.experts, a.rows) + 1);
  const int fit = chunk_fit<EX_FWD>(a, dt, vec);
  return by_type(dt, [&](auto x) {
    using T = decltype(x);
    return launch(K_EXPERT_GEMM, s, [&] {
      if (fit == CHUNK_ALIGNED) hipLaunchKernelGGL((expert_few_fwd<T, CHUNK_ALIGNED>), g, dim3(256), 0, s, a);
      else if (fit == CHUNK_ANY) hipLaunchKernelGGL((expert_few_fwd<T, CHUNK_ANY>), g, dim3(256), 0, s, a);
      else hipLaunchKernelGGL((expert_few_fwd<T, CHUNK_TINY>), g, dim3(256), 0, s, a);
    });
  });
}

// Whether the forward product has few enough rows for the kernel that reads the weights once
// (expert_few.hpp). One MI355X, rows per expert on average (a router's picks), its time against the
// 128 x 128 tiles':
//   64 x 1408 x 2048, bf16: 4 rows 75 to 94 us, 8 rows 85 to 99; 27 x 2048 x 7168: 4 rows 150 to 153,
//   8 rows 178 to 154; fp32, 64 x 1408 x 2048: 8 rows 184 to 241 (split tiles 160), 32 rows 460 to 390
//   (229). Rows that begin anywhere, 64 x 1405 x 2045: bf16 1 row 84 to 60, fp32 4 rows 203 to 244, 16
//   rows 332 to 245 (181). 16-bit with short rows of W, 0.2 rows: 131 x 3432 x 440 18 to 25, 98 x 5872 x
//   296 20 to 21, 244 x 4112 x 112 (224 bytes) 36 to 21, 260 x 5088 x 80 47 to 25.
// Tiles for less than half of the CUs are bound by the latency of their stages, so it takes four
// times the rows, but for 16-bit rows that begin anywhere; against split tiles, 8 x 1000 x 776, bf16:
// 16 rows 7.1 to 8.4 us, 32 rows 9.5 to 8.9; fp32 (1001 x 777) 16 rows 16.2 to 16.4; bf16 8 x 1001 x 777: 8
// rows 9.8 to 8.9; 3 x 505 x 4001: 1 row 15 to 17, 8 rows 19 to 18.
bool few_rows(const ExpertArgs& a, int dt, int fit) {
  const int64_t tiles = std::min<int64_t>(a.experts, a.rows) * ((a.n + 127) / 128);
  const int64_t most = (fit == CHUNK_ALIGNED ? 4 : 2) * (dt == F32 ? 2 : 1) * (int64_t)a.experts;
  const bool whole = fit == CHUNK_ALIGNED || dt == F32;
  if (2 * tiles <= device_cus()) return a.rows <= (whole ? 4 * most : most);
  return a.rows <= most && a.k * dtype_size(dt) >= 512 && whole;
}

// Whether a product takes 64 x 64 tiles, each split along the contraction over eight waves: where
// they fit the CUs at once (fp32, whose MFMAs bound it: nine times that) and the contraction has
// four stages or more. One MI355X, 128 x 128 against split tiles, bf16: 8 experts of 1000 x 776,
// forward 64 rows (192 tiles) 17.3 to 9.7 us, 256 rows (576) 20 to 22; 3 of 504 x 4000, forward 256
// rows (108) 61 to 20, input gradient 32 rows (189) 11.7 to 7.6, 256 rows (850) 14 to 21; 12 of 5361 x
// 2944, 26 rows (1008) 75 to 79. fp32, 64 of 1405 x 2045, forward 16 rows (1408) 245 to 183, 64 rows
// (2112) 399 to 380, input gradient 1 row (2112) 206 to 131. Weight gradients: 6 of 152 x 88 fp32, 1093
// rows (36 tiles) 99 to 27; 8 of 1001 x 777 fp32 (1664) 17 to 40.
template <int MODE>
bool split_tiles(const ExpertArgs& a, int dt) {
  const int64_t stage = 128 / dtype_size(dt);
  const int64_t some = std::min<int64_t>(a.experts, a.rows);   // experts that can have rows
  const int64_t high = MODE == EX_DW ? a.experts * ((a.m + 63) / 64) : std::max(some, a.rows / 64 + some / 2);
  const int64_t tiles = high * ((a.n + 63) / 64), deep = MODE == EX_DW ? a.rows / a.experts : a.k;
  return deep >= 4 * stage && tiles <= (dt == F32 && MODE != EX_DW ? 9 : 1) * (int64_t)device_cus();
}

// The kernel of a product. The 256 x 256 tiles need 16-bit types, whole 16-byte chunks everywhere,
// extents that do not leave half of a tile empty, and enough tiles for half of the CUs. One
// MI355X, bf16, rows per expert on average (a router's picks), 256 x 256 against 128 x 128 tiles: 27
// experts of 2048 x 7168, 8 rows, forward 144 against 154 us, weight gradient 173 against 237; 256
// rows 317 against 417, 380 against 496 (exactly 256 rows each: 218 against 318, 362 against 449); 64
// experts of 1408 x 2048, 16 rows 100 against 100 us, weight gradient 83 against 115; 128 rows 115
// against 132, 138 against 183; 128 experts of 512 x 512 (264 tiles), 32 rows 22 against 20 us, weight
// gradient 20 against 22; 64 rows 24 against 22, 22 against 25; 512 rows 63 against 75; 8 experts of
// 1000 x 776 (64 tiles), 320 rows 23 against 19 us, weight gradient (128 tiles) 17 against 15.
template <int MODE>
int run_product(const ExpertArgs& a, int dt, bool vec, hipStream_t s) {
  // the largest list of the smallest tiles
  const int64_t tn = (a.n + 127) / 128, tm = MODE == EX_DW ? a.experts * ((a.m + 127) / 128) : a.rows / 128 + a.experts + 1;
  if (tn * tm > INT32_MAX) return MNS_ERR_SHAPE;
  if (MODE == EX_FWD && few_rows(a, dt, chunk_fit<EX_FWD>(a, dt, vec))) return run_few(a, dt, vec, s);
  const bool whole = vec && a.c_vec && a.n % 8 == 0 && dt != F32 && a.n > 128 && (MODE != EX_DW || a.m > 128);
  const int64_t high = MODE == EX_DW ? a.experts * ((a.m + 255) / 256) : a.rows / 256 + std::min<int64_t>(a.experts, a.rows);
  if (whole && 2 * high * ((a.n + 255) / 256) >= device_cus()) return run_pingpong<MODE>(a, dt, s);
  if (split_tiles<MODE>(a, dt)) return run_split<MODE>(a, dt, vec, s);
  return run_staged<MODE, Tile128>(a, dt, vec, s);
}

ExpertArgs product_args(const mns_tensor* A, const mns_tensor* B, const mns_tensor* C, const int32_t* offsets, int experts, int64_t rows) {
  ExpertArgs a{};
  a.A = reinterpret_cast<const char*>(A->ptr);
  a.lda = A->ld;
  a.B = reinterpret_cast<const char*>(B->ptr);
  a.ldb = B->ld;
  a.sB = B->batch > 1 ? B->stride : 0;
  a.C = reinterpret_cast<char*>(C->ptr);
  a.ldc = C->ld;
  a.sC = C->batch > 1 ? C->stride : 0;
  a.offsets = offsets;
  a.experts = experts;
  a.rows = rows;
  a.n = (int)C->cols;
  const int64_t es = dtype_size(C->dtype);
  a.c_vec = aligned16(C->ptr) && C->ld * es % 16 == 0 && (C->batch == 1 || C->stride * es % 16 == 0);
  return a;
}

int64_t offsets_bytes(int64_t experts) { return 4 * (experts + 1); }

}  // namespace

// ==========================================================================================
extern "C" {

int layer_norm(const mns_tensor* X, const void* weight, const void* bias, int32_t wdtype, float eps, const mns_tensor* Y,
               float* mean, float* rstd, void* stream) {
  if (int st = check_rows(X)) return st;
  if (int st = check_rows(Y)) return st;
  if (Y->dtype != X->dtype) return MNS_ERR_DTYPE;
  if (!same_rows(X, Y)) return MNS_ERR_SHAPE;
  if (int st = check_wdtype(X, wdtype)) return st;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return MNS_ERR_ARG;
  const int64_t rows = X->batch * X->rows;
  if (!rows) return MNS_OK;
  if (!mean || !rstd) return MNS_ERR_ARG;
  const int64_t wb = X->cols * dtype_size(wdtype);
  if (clash({span(Y), span(mean, 4 * rows), span(rstd, 4 * rows)}, {span(X), span(weight, wb), span(bias, wb)})) return MNS_ERR_ARG;
  NormArgs a{};
  a.x = rows_ref(X);
  a.y = rows_ref(Y);
  a.w = weight;
  a.b = bias;
  a.mean = mean;
  a.rstd = rstd;
  a.rows = rows;
  a.cols = (int)X->cols;
  a.eps = eps;
  a.n = (float)X->cols;
  const bool vec = vec_rows(X) && vec_rows(Y) && X->cols % 8 == 0 && aligned16(weight) && aligned16(bias);
  const hipStream_t s = as_stream(stream);
  return by_norm_types(X->dtype, wdtype, [&](auto x, auto w) {
    using T = decltype(x);
    using WT = decltype(w);
    return launch(K_LAYER_NORM, s, [&] {
      if (vec) launch_norm_fwd<T, WT, true>(a, s);
      else launch_norm_fwd<T, WT, false>(a, s);
    });
  });
}

int mns_layer_norm_workspace_bytes(const mns_tensor* X, size_t* bytes) {
  if (!X || !bytes) return MNS_ERR_ARG;
  mns_tensor t = *X;
  t.ptr = nullptr;
  if (t.rows > 0) t.ptr = reinterpret_cast<void*>(16);   // the pointer does not matter here
  if (int st = check_rows(&t)) return st;
  *bytes = (size_t)norm_parts(X->batch * X->rows, X->cols) * 2 * (size_t)X->cols * 4;
  return MNS_OK;
}

int layer_norm_backward(const mns_tensor* dY, const mns_tensor* X, const float* mean, const float* rstd, const void* weight,
                        int32_t wdtype, const mns_tensor* dX, void* dweight, void* dbias, void* ws, size_t ws_bytes, void* stream) {
  for (const mns_tensor* t : {dY, X, dX})
    if (int st = check_rows(t)) return st;
  if (dY->dtype != X->dtype || dX->dtype != X->dtype) return MNS_ERR_DTYPE;
  if (!same_rows(X, dY) || !same_rows(X, dX)) return MNS_ERR_SHAPE;
  if (int st = check_wdtype(X, wdtype)) return st;
  const int64_t rows = X->batch * X->rows;
  if (rows && (!mean || !rstd)) return MNS_ERR_ARG;
  const bool grads = dweight || dbias;
  const size_t need = (size_t)norm_parts(rows, X->cols) * 2 * (size_t)X->cols * 4;
  if (grads && rows && (!ws || ws_bytes < need || !aligned16(ws))) return MNS_ERR_WORKSPACE;
  const int64_t wb = X->cols * dtype_size(wdtype);
  if (clash({span(dX), span(dweight, wb), span(dbias, wb), span(grads ? ws : nullptr, (int64_t)need)},
            {span(dY), span(X), span(mean, 4 * rows), span(rstd, 4 * rows), span(weight, wb)}))
    return MNS_ERR_ARG;
  NormArgs a{};
  a.x = rows_ref(X);
  a.dy = rows_ref(dY);
  a.dx = rows_ref(dX);
  a.w = weight;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.rows = rows;
  a.cols = (int)X->cols;
  a.n = (float)X->cols;
  a.part = grads ? reinterpret_cast<float*>(ws) : nullptr;
  a.nparts = rows ? norm_parts(rows, X->cols) : 0;
  a.dw = dweight;
  a.db = dbias;
  const bool vec = vec_rows(X) && vec_rows(dY) && vec_rows(dX) && X->cols % 8 == 0 && aligned16(weight);
  const hipStream_t s = as_stream(stream);
  return by_norm_types(X->dtype, wdtype, [&](auto x, auto w) {
    using T = decltype(x);
    using WT = decltype(w);
    if (rows && a.cols <= kNormHeld) {
      if (int st = launch(K_LAYER_NORM, s, [&] {
            if (vec) launch_norm_bwd<T, WT, true>(a, s);
            else launch_norm_bwd<T, WT, false>(a, s);
          }))
        return st;
    } else if (rows) {
      if (int st = launch(K_LAYER_NORM, s, [&] { hipLaunchKernelGGL((norm_dx_any<T, WT>), grid_of(rows), dim3(256), 0, s, a); })) return st;
      if (grads)
        if (int st = launch(K_LAYER_NORM, s, [&] {
              hipLaunchKernelGGL((norm_dw_any<T>), dim3((a.cols + 255) / 256, a.nparts), dim3(256), 0, s, a);
            }))
          return st;
    }
    if (!grads) return (int)MNS_OK;
    return launch(K_LAYER_NORM, s, [&] { hipLaunchKernelGGL((norm_dw_sum<WT>), dim3((a.cols + 63) / 64, 2), dim3(1024), 0, s, a); });
  });
}

int mns_expert_sort_workspace_bytes(int64_t slots, int32_t experts, size_t* bytes) {
  if (!bytes) return MNS_ERR_ARG;
  if (slots < 0 || slots > kMaxRows || experts < 1 || experts > EXPERT_MAX) return MNS_ERR_SHAPE;
  const SortPlan sp = sort_plan(slots);
  *bytes = sp.nblocks > 1 ? (size_t)sp.nblocks * experts * 4 : 0;
  return MNS_OK;
}

int expert_sort(const void* ids, int32_t id_bytes, int64_t slots, int32_t experts, int32_t* offsets, int32_t* rank, void* ws,
                size_t ws_bytes, void* stream) {
  static_assert(SORT_MAX_E == EXPERT_MAX, "one limit on the number of experts");
  if (id_bytes != 4 && id_bytes != 8) return MNS_ERR_DTYPE;
  size_t need = 0;
  if (int st = mns_expert_sort_workspace_bytes(slots, experts, &need)) return st;
  if (int st = check_experts(offsets, experts)) return st;
  if (slots && (!ids || !rank || reinterpret_cast<uintptr_t>(ids) % id_bytes || reinterpret_cast<uintptr_t>(rank) % 4)) return MNS_ERR_ARG;
  if (need && (!ws || ws_bytes < need || !aligned16(ws))) return MNS_ERR_WORKSPACE;
  if (clash({span(offsets, offsets_bytes(experts)), span(rank, 4 * slots), span(need ? ws : nullptr, (int64_t)need)}, {span(ids, id_bytes * slots)}))
    return MNS_ERR_ARG;
  const SortPlan sp = sort_plan(slots);
  SortArgs a{ids, slots, experts, sp.steps, sp.nblocks, reinterpret_cast<int32_t*>(ws), offsets, rank};
  const hipStream_t s = as_stream(stream);
  auto run = [&](auto id) {
    using ID = decltype(id);
    if (sp.nblocks > 1)
      if (int st = launch(K_ROUTE, s, [&] { hipLaunchKernelGGL((sort_count<ID>), dim3(sp.nblocks), dim3(SORT_NT), 0, s, a); })) return st;
    return launch(K_ROUTE, s, [&] { hipLaunchKernelGGL((sort_place<ID>), dim3(sp.nblocks), dim3(SORT_NT), 0, s, a); });
  };
  return id_bytes == 4 ? run(int32_t{}) : run(int64_t{});
}

int expert_dispatch(const mns_tensor* X, const int32_t* rank, int32_t k, const int32_t* offsets, int32_t experts,
                    const mns_tensor* XS, void* stream) {
  if (int st = check_sides(X, XS, rank, k)) return st;
  if (int st = check_experts(offsets, experts)) return st;
  if (clash({span(XS)}, {span(X), span(rank, rank_bytes(X->rows, k)), span(offsets, offsets_bytes(experts))})) return MNS_ERR_ARG;
  if (!X->rows) return MNS_OK;
  RowsArgs a = rows_args(X, rank, k);
  a.tok = reinterpret_cast<const char*>(X->ptr);
  a.tok_ld = row_bytes(X);
  a.out = reinterpret_cast<char*>(XS->ptr);
  a.out_ld = row_bytes(XS);
  a.offsets = offsets;
  a.experts = experts;
  const bool vec = vec_rows(X) && vec_rows(XS);
  const int es = dtype_size(X->dtype);
  a.units = (int)(vec ? X->cols * es / 16 : X->cols);
  const dim3 g = rows_grid(a);
  const hipStream_t s = as_stream(stream);
  return launch(K_ROUTE, s, [&] {
    if (vec) hipLaunchKernelGGL((rows_dispatch<u32x4>), g, dim3(ROWS_NT), 0, s, a);
    else if (es == 4) hipLaunchKernelGGL((rows_dispatch<uint32_t>), g, dim3(ROWS_NT), 0, s, a);
    else hipLaunchKernelGGL((rows_dispatch<uint16_t>), g, dim3(ROWS_NT), 0, s, a);
  });
}

int expert_dispatch_backward(const mns_tensor* dXS, const int32_t* rank, int32_t k, const mns_tensor* dX, void* stream) {
  if (int st = check_sides(dX, dXS, rank, k)) return st;
  if (clash({span(dX)}, {span(dXS), span(rank, rank_bytes(dX->rows, k))})) return MNS_ERR_ARG;
  if (!dX->rows) return MNS_OK;
  return gather<false>(rows_args(dX, rank, k), dXS, dX, as_stream(stream));
}

int expert_combine(const mns_tensor* YS, const void* weights, int32_t wdtype, const int32_t* rank, int32_t k, const mns_tensor* Y,
                   void* stream) {
  if (int st = check_sides(Y, YS, rank, k)) return st;
  if (int st = check_wdtype(Y, wdtype)) return st;
  if (Y->rows && (!weights || reinterpret_cast<uintptr_t>(weights) % dtype_size(wdtype))) return MNS_ERR_ARG;
  if (clash({span(Y)}, {span(YS), span(rank, rank_bytes(Y->rows, k)), span(weights, Y->rows * k * dtype_size(wdtype))})) return MNS_ERR_ARG;
  if (!Y->rows) return MNS_OK;
  RowsArgs a = rows_args(Y, rank, k);
  a.weights = weights;
  a.w_dt = wdtype;
  return gather<true>(a, YS, Y, as_stream(stream));
}

int expert_combine_backward(const mns_tensor* dY, const mns_tensor* YS, const void* weights, int32_t wdtype, const int32_t* rank,
                            int32_t k, const int32_t* offsets, int32_t experts, const mns_tensor* dYS, void* dweights, void* stream) {
  if (int st = check_sides(dY, YS, rank, k)) return st;
  if (int st = check_sides(dY, dYS, rank, k)) return st;
  if (int st = check_wdtype(dY, wdtype)) return st;
  if (int st = check_experts(offsets, experts)) return st;
  const int64_t wb = dY->rows * k * dtype_size(wdtype);
  for (const void* w : {weights, (const void*)dweights})
    if (dY->rows && (!w || reinterpret_cast<uintptr_t>(w) % dtype_size(wdtype))) return MNS_ERR_ARG;
  if (clash({span(dYS), span(dweights, wb)},
            {span(dY), span(YS), span(weights, wb), span(rank, rank_bytes(dY->rows, k)), span(offsets, offsets_bytes(experts))}))
    return MNS_ERR_ARG;
  if (!dY->rows) return MNS_OK;
  RowsArgs a = rows_args(dY, rank, k);
  a.tok = reinterpret_cast<const char*>(dY->ptr);
  a.tok_ld = row_bytes(dY);
  a.row = reinterpret_cast<const char*>(YS->ptr);
  a.row_ld = row_bytes(YS);
  a.out = reinterpret_cast<char*>(dYS->ptr);
  a.out_ld = row_bytes(dYS);
  a.weights = weights;
  a.w_dt = wdtype;
  a.dweights = dweights;
  a.offsets = offsets;
  a.experts = experts;
  const bool vec = vec_rows(dY) && vec_rows(YS) && vec_rows(dYS) && dY->cols % 8 == 0;
  a.units = (int)(vec ? dY->cols / 8 : dY->cols);
  const hipStream_t s = as_stream(stream);
  const dim3 g = grid_of(a.tokens);
  return by_type(dY->dtype, [&](auto x) {
    using T = decltype(x);
    return launch(K_ROUTE, s, [&] {
      if (vec) hipLaunchKernelGGL((rows_combine_bwd<T, 8>), g, dim3(ROWS_NT), 0, s, a);
      else hipLaunchKernelGGL((rows_combine_bwd<T, 1>), g, dim3(ROWS_NT), 0, s, a);
    });
  });
}

int expert_matmul(const mns_tensor* X, const mns_tensor* W, const int32_t* offsets, const mns_tensor* Y, void* stream) {
  if (int st = check_product(X, W, offsets, Y)) return st;
  if (X->batch != 1 || Y->batch != 1 || X->rows != Y->rows || X->cols != W->cols || Y->cols != W->rows) return MNS_ERR_SHAPE;
  if (clash({span(Y)}, {span(X), span(W), span(offsets, offsets_bytes(W->batch))})) return MNS_ERR_ARG;
  if (!X->rows) return MNS_OK;
  ExpertArgs a = product_args(X, W, Y, offsets, (int)W->batch, X->rows);
  a.k = (int)W->cols;
  return run_product<EX_FWD>(a, W->dtype, vec_rows(X) && vec_rows(W), as_stream(stream));
}

int expert_matmul_grad_input(const mns_tensor* dY, const mns_tensor* W, const int32_t* offsets, const mns_tensor* dX, void* stream) {
  if (int st = check_product(dY, W, offsets, dX)) return st;
  if (dY->batch != 1 || dX->batch != 1 || dY->rows != dX->rows || dY->cols != W->rows || dX->cols != W->cols) return MNS_ERR_SHAPE;
  if (clash({span(dX)}, {span(dY), span(W), span(offsets, offsets_bytes(W->batch))})) return MNS_ERR_ARG;
  if (!dY->rows) return MNS_OK;
  ExpertArgs a = product_args(dY, W, dX, offsets, (int)W->batch, dY->rows);
  a.k = (int)W->rows;
  return run_product<EX_DX>(a, W->dtype, vec_rows(dY) && vec_rows(W), as_stream(stream));
}

int expert_matmul_grad_weight(const mns_tensor* dY, const mns_tensor* X, const int32_t* offsets, const mns_tensor* dW, void* stream) {
  if (int st = check_product(dY, dW, offsets, X)) return st;
  if (dY->batch != 1 || X->batch != 1 || dY->rows != X->rows || dY->cols != dW->rows || X->cols != dW->cols) return MNS_ERR_SHAPE;
  if (clash({span(dW)}, {span(dY), span(X), span(offsets, offsets_bytes(dW->batch))})) return MNS_ERR_ARG;
  ExpertArgs a = product_args(dY, X, dW, offsets, (int)dW->batch, dY->rows);
  a.m = (int)dW->rows;
  return run_product<EX_DW>(a, dW->dtype, vec_rows(dY) && vec_rows(X), as_stream(stream));
}

}  // extern "C"
