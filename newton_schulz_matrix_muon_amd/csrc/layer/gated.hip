// Host side of the gated block (gated.hpp). As in layer.hip, validation happens before any HIP call and a
// call only enqueues kernels on the caller's stream.

#include "muon_ns.h"

#include <hip/hip_runtime.h>

#include <algorithm>

#include "checks.hpp"
#include "expert_pingpong.hpp"
#include "gated.hpp"

using namespace mns;

namespace {

using Tile64 = TileCfg<64, 64, 1, 1, 128, 1, 2>;

// Tile rows and columns of a product over all experts, as the kernels cut them.
template <int MODE, class CFG>
int64_t tile_rows(const GatedArgs& a) {
  if (ex_dw(MODE)) return (int64_t)dw_matrices<MODE>(a) * ((a.m + CFG::BM - 1) / CFG::BM);
  return (a.rows + CFG::BM - 1) / CFG::BM + std::min<int64_t>(a.experts, a.rows) + 1;
}
template <int MODE, class CFG>
int tile_columns(const GatedArgs& a) { return (a.n + tile_cols<MODE, CFG>() - 1) / tile_cols<MODE, CFG>(); }

// Persistent grid: enough workgroups for every tile, at most those the chip holds at once, the same
// number on each of the eight XCDs.
template <int MODE, class CFG>
unsigned grid_for(const GatedArgs& a, int per_cu) {
  const int64_t tiles = tile_rows<MODE, CFG>(a) * a.tiles_n;
  return (unsigned)(8 * std::max<int64_t>(1, (std::min(tiles, (int64_t)device_cus() * per_cu) + 7) / 8));
}

template <int MODE, class CFG, int G>
int run_staged(GatedArgs a, int dt, int fit, hipStream_t s) {
  a.tiles_n = tile_columns<MODE, CFG>(a);
  const int per_cu = G > 1 ? 1 : std::max(1, std::min((160 * 1024) / (CFG::LDS + 8192), 4 * CFG::OCC / (CFG::NT / 64)));
  const dim3 g(grid_for<MODE, CFG>(a, per_cu)), b(CFG::NT * G);
  return by_type(dt, [&](auto x) {
    using T = decltype(x);
    return launch(K_EXPERT_GEMM, s, [&] {
      if (fit == CHUNK_ALIGNED) hipLaunchKernelGGL((expert_gemm_staged<MODE, T, CHUNK_ALIGNED, CFG, G>), g, b, 0, s, a);
      else if (fit == CHUNK_ANY) hipLaunchKernelGGL((expert_gemm_staged<MODE, T, CHUNK_ANY, CFG, G>), g, b, 0, s, a);
      else if constexpr (G == 1 || !ex_fwd(MODE))   // a split forward product's contraction would be one short row
        hipLaunchKernelGGL((expert_gemm_staged<MODE, T, CHUNK_TINY, CFG, G>), g, b, 0, s, a);
    });
  });
}

template <int MODE>
int run_pingpong(GatedArgs a, int dt, hipStream_t s) {
  a.tiles_n = tile_columns<MODE, TilePP>(a);
  const unsigned g = grid_for<MODE, TilePP>(a, 1);
  return launch(K_EXPERT_GEMM, s, [&] {
    if (dt == BF16) hipLaunchKernelGGL((expert_gemm_pp<MODE, __bf16>), dim3(g), dim3(TilePP::NT), 0, s, a);
    else hipLaunchKernelGGL((expert_gemm_pp<MODE, _Float16>), dim3(g), dim3(TilePP::NT), 0, s, a);
  });
}

// A dense product whose last round of 256 x 256 tiles would leave half of the CUs idle or more: that round's tiles are
// cut along the contraction (last_round). The workspace has room for a part of every workgroup.
int64_t split_bytes() { return (int64_t)round_up(device_cus(), 8) * 256 * 256 * 4; }

template <int MODE>
int run_split_pingpong(GatedArgs a, int dt, hipStream_t s) {
  a.tiles_n = tile_columns<MODE, TilePP>(a);
  a.wgs = (int)round_up(device_cus(), 8) / 8;
  const unsigned g = 8 * a.wgs;
  auto both = [&](auto x) {
    using T = decltype(x);
    if (int st = launch(K_EXPERT_GEMM, s, [&] { hipLaunchKernelGGL((expert_gemm_pp<MODE, T, true>), dim3(g), dim3(TilePP::NT), 0, s, a); })) return st;
    return launch(K_EXPERT_GEMM, s, [&] { hipLaunchKernelGGL((expert_split_sum<MODE, T>), dim3(256 * (a.wgs / 2)), dim3(64), 0, s, a); });
  };
  return dt == BF16 ? both(__bf16{}) : both(_Float16{});
}

// Whether cutting the last round is worth its sum: host arithmetic on a dense product's tiles. Forward products
// with and without (us, 128 x 64 tiles): 1000 x 2048 x 2048 (32 stages) 46 and 36, 600 x 4096 x 3000 (47) 58 and 61,
// 400 x 7168 x 4096 (64) 73 and 83.
template <int MODE>
bool split_pays(const GatedArgs& a) {
  if (MODE == EX_DW2 || !a.parts || a.offsets) return false;
  const int wgs = (int)round_up(device_cus(), 8) / 8;
  const int64_t tiles = (a.rows + 255) / 256 * tile_columns<MODE, TilePP>(a);
  const LastRound last = last_round((int)((tiles + 7) / 8), wgs);
  const int64_t stages = (a.k + 63) / 64 * (MODE == EX_DX2 ? 2 : 1);
  return last.parts > 1 && stages >= 40;
}

int run_few(const GatedArgs& a, int dt, int fit, hipStream_t s) {
  const dim3 g((a.n + 15) / 16, (unsigned)std::min<int64_t>(a.experts, a.rows) + 1);
  return by_type(dt, [&](auto x) {
    using T = decltype(x);
    return launch(K_EXPERT_GEMM, s, [&] {
      if (fit == CHUNK_ALIGNED) hipLaunchKernelGGL((expert_few_gated<T, CHUNK_ALIGNED>), g, dim3(256), 0, s, a);
      else if (fit == CHUNK_ANY) hipLaunchKernelGGL((expert_few_gated<T, CHUNK_ANY>), g, dim3(256), 0, s, a);
      else hipLaunchKernelGGL((expert_few_gated<T, CHUNK_TINY>), g, dim3(256), 0, s, a);
    });
  });
}

// Few rows: the kernel that reads the weights once for 16 rows of an expert. It wins where there are few tiles, and where a row
// of W is short, so that the tiles' first stages count; it has nothing to hide its latency under where W's rows begin anywhere.
// us with it and without (bf16; fp32):
//   64 experts of 1408 x 2048  6 experts with a row 17 and 24; 42 and 55;  16: 37 and 51; 84 and 87;  one row each 124 and 157;
//                              297 and 309;  four each 132 and 158; 311 and 311;  six each 140 and 159; 320 and 310
//   27 of 2048 x 7168          6 (192 tiles) 79 and 80; 166 and 184;  16 (512) 173 and 161; 403 and 369;  one row each 295 and 286; 694 and 629
//   12 of 5360 x 2944          6 (504) 83 and 85; 175 and 157;  one row each 135 and 137; 339 and 306
//   dense 4096 x 3000          1 row 17 and 20; 27 and 40;  16 rows 18 and 21; 33 and 42;  24 rows 25 and 22; 51 and 44
//   dense 18432 x 7168 (288)   1 row 105 and 127; 237 and 242;  4 rows 112 and 127; 247 and 241;  8 rows 121 and 127; 260 and 244
//   64 of 1405 x 2045          6 (132) 34 and 26; 47 and 55;  16 (352) 64 and 57; 101 and 87
bool few_rows(const GatedArgs& a, int dt, int fit) {
  const int64_t tiles = std::min<int64_t>(a.experts, a.rows) * ((a.n + 63) / 64), cus = device_cus(), row = a.k * dtype_size(dt);
  const bool aligned = fit == CHUNK_ALIGNED, whole = aligned || dt == F32;
  const int64_t most = (whole ? 4 : 2) * (int64_t)a.experts;
  if (2 * tiles <= cus) return a.rows <= (whole ? 4 * most : most);
  if (a.rows > most || row < 512 || !whole) return false;
  return aligned ? 2 * tiles <= 3 * cus || row <= 8192 : tiles <= cus;
}

// 64 x 64 tiles whose contraction eight waves share: where larger tiles would leave CUs idle, or would be mostly
// empty. us with these tiles and without: 16-bit forward products of 400 x 2048 x 2048 (448 tiles) 26 and 34,
// 200 x 4096 x 3000 (512) 36 and 45, 300 x 4096 x 3000 (640) 49 and 48; input gradients of 300 x 7168 x 4096
// (320) 110 and 85. fp32 has no larger pipelined tiles: 64 experts of 1408 x 2048 with 32 rows each 445 and
// 760, with 64 rows 698 and 778, with 96 rows 912 and 800.
template <int MODE>
bool split_tiles(const GatedArgs& a, int dt) {
  const int64_t stage = 128 / dtype_size(dt);
  const int64_t some = std::min<int64_t>(a.experts, a.rows);   // experts that can have rows
  const int64_t high = ex_dw(MODE) ? tile_rows<MODE, Tile64>(a) : a.experts > 1 ? std::max(some, a.rows / 64 + some / 2) : (a.rows + 63) / 64;
  const int64_t tiles = high * tile_columns<MODE, Tile64>(a), deep = ex_dw(MODE) ? a.rows / a.experts : MODE == EX_DX2 ? 2 * (int64_t)a.k : a.k;
  if (deep < 4 * stage) return false;
  if (dt == F32 && !ex_dw(MODE)) return tiles <= 9 * (int64_t)device_cus() || a.rows <= 72 * some;
  return tiles <= (MODE == EX_GATE ? 2 : 1) * (int64_t)device_cus();
}

// Whether the 256 x 256 tiles fit a product's types, rows and extents.
template <int MODE>
bool whole_tiles(const GatedArgs& a, int dt, bool vec) {
  return vec && a.c_vec && a.n % 8 == 0 && dt != F32 && a.n > (MODE == EX_GATE ? 64 : 128) && (!ex_dw(MODE) || a.m > 128);
}

// Whether a dense product of rows x n results and contractions of k takes the cut last round if it has room for it.
template <int MODE>
bool takes_split(int64_t rows, int64_t n, int64_t k, int dt) {
  GatedArgs a{};
  float room;
  a.parts = &room;
  a.c_vec = 1;
  a.experts = 1;
  a.rows = rows;
  a.n = (int)n;
  a.k = (int)k;
  return whole_tiles<MODE>(a, dt, true) && !(MODE == EX_GATE && few_rows(a, dt, CHUNK_ALIGNED)) && split_pays<MODE>(a) && !split_tiles<MODE>(a, dt);
}

// vec: operands' rows of whole aligned chunks.
template <int MODE>
int run_product(const GatedArgs& a, int dt, bool vec, hipStream_t s) {
  // the largest list of the smallest tiles of the persistent kernels
  if (tile_rows<MODE, Tile64>(a) * (int64_t)tile_columns<MODE, Tile64>(a) > INT32_MAX) return MNS_ERR_SHAPE;
  const int chunk = 16 / dtype_size(dt);
  const bool tiny = (ex_dw(MODE) ? a.m : a.k) < chunk || (!ex_fwd(MODE) && a.n < chunk);
  const int fit = vec ? CHUNK_ALIGNED : tiny ? CHUNK_TINY : CHUNK_ANY;
  if constexpr (MODE == EX_GATE)
    if (few_rows(a, dt, fit)) return run_few(a, dt, fit, s);
  const bool whole = whole_tiles<MODE>(a, dt, vec);
  const int64_t high = ex_dw(MODE) ? tile_rows<MODE, TilePP>(a) : a.rows / 256 + std::min<int64_t>(a.experts, a.rows);
  if constexpr (MODE != EX_DW2)
    if (whole && split_pays<MODE>(a) && !split_tiles<MODE>(a, dt)) return run_split_pingpong<MODE>(a, dt, s);
  // With as few rows as there are these tiles lose little: 64 experts of 1408 x 2048, 24 rows each, forward 154 us, with 128 x 64 tiles
  // 149; 64 rows 161 and 159, 128 rows 173 and 228; 27 experts of 2048 x 7168 291 and 295, 300 and 313, 346 and 460.
  if (whole && 2 * high * tile_columns<MODE, TilePP>(a) >= device_cus()) return run_pingpong<MODE>(a, dt, s);
  if (split_tiles<MODE>(a, dt)) return run_staged<MODE, Tile64, 8>(a, dt, fit, s);
  return run_staged<MODE, Tile128, 1>(a, dt, fit, s);
}

// Results that 16-byte stores fit.
bool vec_out(const mns_tensor* t) {
  const int64_t es = dtype_size(t->dtype);
  return aligned16(t->ptr) && t->ld * es % 16 == 0 && (t->batch == 1 || t->stride * es % 16 == 0);
}

// X: S x K, Wg and Wu: E matrices N x K.
int check_pair(const mns_tensor* X, const mns_tensor* Wg, const mns_tensor* Wu, const int32_t* offsets, int32_t act) {
  for (const mns_tensor* t : {X, Wg, Wu}) {
    if (int st = check_rows(t)) return st;
    if (t->dtype != X->dtype) return MNS_ERR_DTYPE;
  }
  if (X->batch != 1 || !same_rows(Wg, Wu) || Wg->rows < 1 || Wg->batch > EXPERT_MAX || X->cols != Wg->cols) return MNS_ERR_SHAPE;
  if (act != MNS_ACT_SILU && act != MNS_ACT_GELU && act != MNS_ACT_RELU) return MNS_ERR_ARG;
  static_assert(ACT_SILU == MNS_ACT_SILU && ACT_GELU == MNS_ACT_GELU && ACT_RELU == MNS_ACT_RELU, "one numbering");
  if (!offsets) return Wg->batch == 1 ? MNS_OK : MNS_ERR_ARG;
  return check_experts(offsets, (int32_t)Wg->batch);
}

// A buffer of S x N rows.
int check_inner(const mns_tensor* t, const mns_tensor* X, const mns_tensor* W) {
  if (int st = check_rows(t)) return st;
  if (t->dtype != X->dtype) return MNS_ERR_DTYPE;
  return t->batch == 1 && t->rows == X->rows && t->cols == W->rows ? MNS_OK : MNS_ERR_SHAPE;
}

GatedArgs gated_args(const mns_tensor* A, const mns_tensor* Wg, const mns_tensor* Wu, const mns_tensor* C, const int32_t* offsets,
                     int experts, int64_t rows) {
  GatedArgs a{};
  static_cast<ExpertArgs&>(a) = product_args(A, Wg, C, offsets, experts, rows);
  a.B2 = reinterpret_cast<const char*>(Wu->ptr);
  a.ldb2 = Wu->ld;
  a.sB2 = Wu->batch > 1 ? Wu->stride : 0;
  return a;
}

Span offsets_span(const int32_t* offsets, int64_t experts) { return span(offsets, offsets ? offsets_bytes(experts) : 0); }

// dgate and dup of a backward pass: rows of whole 16-byte chunks.
int64_t inner_ld(int64_t n) { return round_up(n, 8); }
int64_t inner_bytes(int64_t rows, int64_t n, int dt) { return round_up(rows * inner_ld(n) * dtype_size(dt), 16); }

}  // namespace

// ==========================================================================================
extern "C" {

int mns_expert_gated_workspace_bytes(int64_t rows, int64_t inner, int32_t experts, int32_t dtype, size_t* forward, size_t* backward) {
  if (!forward || !backward) return MNS_ERR_ARG;
  if (!valid_dtype(dtype)) return MNS_ERR_DTYPE;
  if (rows < 0 || rows > kMaxRows || inner < 1 || inner > kMaxCols || experts < 0 || experts > EXPERT_MAX) return MNS_ERR_SHAPE;
  *forward = rows && !experts && dtype != F32 ? (size_t)split_bytes() : 0;
  *backward = (size_t)(2 * inner_bytes(rows, inner, dtype)) + *forward;
  return MNS_OK;
}

int mns_expert_gated_dense_workspace_bytes(int64_t rows, int64_t inner, int64_t cols, int32_t dtype, size_t* forward, size_t* backward) {
  if (cols < 1 || cols > kMaxCols) return MNS_ERR_SHAPE;
  if (int st = mns_expert_gated_workspace_bytes(rows, inner, 0, dtype, forward, backward)) return st;
  if (!*forward) return MNS_OK;
  if (!takes_split<EX_DX2>(rows, cols, inner, dtype)) *backward -= *forward;
  if (!takes_split<EX_GATE>(rows, inner, cols, dtype)) *forward = 0;
  return MNS_OK;
}

int expert_gated(const mns_tensor* X, const mns_tensor* Wg, const mns_tensor* Wu, const int32_t* offsets, int32_t act, const mns_tensor* H,
                 const mns_tensor* G, const mns_tensor* U, void* ws, size_t ws_bytes, void* stream) {
  if (int st = check_pair(X, Wg, Wu, offsets, act)) return st;
  if ((G == nullptr) != (U == nullptr)) return MNS_ERR_ARG;
  for (const mns_tensor* t : {H, G ? G : H, U ? U : H})
    if (int st = check_inner(t, X, Wg)) return st;
  const Span none = span(static_cast<const void*>(nullptr), 0);
  // the workspace is for dense calls alone, and they do without
  const bool room = ws && !offsets && X->dtype != F32 && ws_bytes >= (size_t)split_bytes();
  if (room && !aligned16(ws)) return MNS_ERR_WORKSPACE;
  if (clash({span(H), G ? span(G) : none, U ? span(U) : none, room ? span(ws, split_bytes()) : none},
            {span(X), span(Wg), span(Wu), offsets_span(offsets, Wg->batch)}))
    return MNS_ERR_ARG;
  if (!X->rows) return MNS_OK;
  GatedArgs a = gated_args(X, Wg, Wu, H, offsets, (int)Wg->batch, X->rows);
  a.k = (int)X->cols;
  a.act = act;
  a.parts = room ? reinterpret_cast<float*>(ws) : nullptr;
  if (G) {
    a.C2 = reinterpret_cast<char*>(G->ptr);
    a.ldc2 = G->ld;
    a.C3 = reinterpret_cast<char*>(U->ptr);
    a.ldc3 = U->ld;
    a.c_vec = a.c_vec && vec_out(G) && vec_out(U);
  }
  return run_product<EX_GATE>(a, X->dtype, vec_rows(X) && vec_rows(Wg) && vec_rows(Wu), as_stream(stream));
}

int expert_gated_backward(const mns_tensor* dH, const mns_tensor* X, const mns_tensor* Wg, const mns_tensor* Wu, const mns_tensor* G,
                          const mns_tensor* U, const int32_t* offsets, int32_t act, const mns_tensor* dX, const mns_tensor* dWg,
                          const mns_tensor* dWu, void* ws, size_t ws_bytes, void* stream) {
  if (int st = check_pair(X, Wg, Wu, offsets, act)) return st;
  for (const mns_tensor* t : {dH, G, U})
    if (int st = check_inner(t, X, Wg)) return st;
  if ((dWg == nullptr) != (dWu == nullptr) || (!dX && !dWg)) return MNS_ERR_ARG;
  for (const mns_tensor* t : {dX ? dX : X, dWg ? dWg : Wg, dWu ? dWu : Wu}) {
    if (int st = check_rows(t)) return st;
    if (t->dtype != X->dtype) return MNS_ERR_DTYPE;
  }
  if ((dX && !same_rows(dX, X)) || (dWg && (!same_rows(dWg, Wg) || !same_rows(dWu, Wg)))) return MNS_ERR_SHAPE;
  const int64_t half = inner_bytes(X->rows, Wg->rows, X->dtype);
  if (X->rows && (!ws || ws_bytes < (size_t)(2 * half) || !aligned16(ws))) return MNS_ERR_WORKSPACE;
  const bool room = X->rows && !offsets && X->dtype != F32 && ws_bytes >= (size_t)(2 * half + split_bytes());
  const Span none = span(static_cast<const void*>(nullptr), 0);
  if (clash({dX ? span(dX) : none, dWg ? span(dWg) : none, dWu ? span(dWu) : none, X->rows ? span(ws, 2 * half + (room ? split_bytes() : 0)) : none},
            {span(dH), span(X), span(Wg), span(Wu), span(G), span(U), offsets_span(offsets, Wg->batch)}))
    return MNS_ERR_ARG;
  const hipStream_t s = as_stream(stream);
  // the rows of dgate and dup
  mns_tensor d = *X;
  d.ptr = ws;
  d.cols = Wg->rows;
  d.ld = inner_ld(Wg->rows);
  char* dup = reinterpret_cast<char*>(ws) + half;
  if (X->rows) {
    GatedGradArgs g{};
    g.dh = reinterpret_cast<const char*>(dH->ptr);
    g.gate = reinterpret_cast<const char*>(G->ptr);
    g.up = reinterpret_cast<const char*>(U->ptr);
    g.ldh = dH->ld;
    g.ldg = G->ld;
    g.ldu = U->ld;
    g.dgate = reinterpret_cast<char*>(ws);
    g.dup = dup;
    g.ld = d.ld;
    g.offsets = offsets;
    g.experts = (int)Wg->batch;
    g.rows = X->rows;
    g.n = (int)Wg->rows;
    g.units = (int)(d.ld / 8);
    if (int st = by_type(X->dtype, [&](auto x) {
          using T = decltype(x);
          return launch(K_EXPERT_GEMM, s, [&] { hipLaunchKernelGGL(gated_grad<T>, grid_of((g.rows * g.units + 255) / 256), dim3(256), 0, s, g, act); });
        }))
      return st;
  }
  // Their rows are whole chunks whatever N is: zeros behind the end meet rows of W behind its end, which
  // read as zeros, or are rows of dW behind its end, which are not stored.
  if (dX && X->rows) {
    GatedArgs a = gated_args(&d, Wg, Wu, dX, offsets, (int)Wg->batch, X->rows);
    a.A2 = dup;
    a.k = (int)Wg->rows;
    a.parts = room ? reinterpret_cast<float*>(dup + half) : nullptr;
    if (int st = run_product<EX_DX2>(a, X->dtype, vec_rows(Wg) && vec_rows(Wu), s)) return st;
  }
  if (!dWg) return MNS_OK;
  if (!X->rows) d.ptr = nullptr;
  GatedArgs a{};
  static_cast<ExpertArgs&>(a) = product_args(&d, X, dWg, offsets, (int)Wg->batch, X->rows);
  a.A2 = X->rows ? dup : nullptr;
  a.C2 = reinterpret_cast<char*>(dWu->ptr);
  a.ldc2 = dWu->ld;
  a.sC2 = dWu->batch > 1 ? dWu->stride : 0;
  a.c_vec = a.c_vec && vec_out(dWu);
  a.m = (int)Wg->rows;
  return run_product<EX_DW2>(a, X->dtype, vec_rows(X), s);
}

}  // extern "C"
