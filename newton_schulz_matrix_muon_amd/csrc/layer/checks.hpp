// What the host sides of the layer operators share (layer.hip, gated.hip, block.hip): checks of their
// arguments, dispatch by type, and the grids and arguments of the experts' products.
#pragma once

#include "muon_ns.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../host.hpp"
#include "expert_gemm.hpp"
#include "norm.hpp"
#include "overlap.hpp"

namespace mns {

constexpr int64_t kMaxRows = 1 << 24, kMaxCols = 1 << 20;

// A buffer of rows: like the matrices of the Newton-Schulz calls, but zero rows are allowed and
// offsets may pass 32 bits.
inline int check_rows(const mns_tensor* t) {
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

inline Span span(const mns_tensor* t) { return span(t, dtype_size(t->dtype)); }

inline bool same_rows(const mns_tensor* a, const mns_tensor* b) {
  return a->batch == b->batch && a->rows == b->rows && a->cols == b->cols;
}

// Every row of t begins at a multiple of 16 bytes and is whole 16-byte chunks long.
inline bool vec_rows(const mns_tensor* t) {
  const int64_t es = dtype_size(t->dtype);
  return reinterpret_cast<uintptr_t>(t->ptr) % 16 == 0 && t->cols * es % 16 == 0 && (t->rows <= 1 || t->ld * es % 16 == 0) &&
         (t->batch == 1 || t->stride * es % 16 == 0);
}
inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// f(element of the buffer's type) for a runtime dtype.
template <class F>
inline int by_type(int dt, F&& f) {
  if (dt == F32) return f(float{});
  if (dt == BF16) return f(__bf16{});
  return f(_Float16{});
}

// At least n workgroups of up to 1024 threads, numbered by block_id().
inline dim3 grid_of(int64_t n) {
  const int64_t x = std::min<int64_t>(n, 1 << 21);
  return dim3((unsigned)x, (unsigned)((n + x - 1) / x));
}

inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

inline RowsRef rows_ref(const mns_tensor* t) { return {reinterpret_cast<char*>(t->ptr), std::max<int64_t>(t->rows, 1), t->ld, t->stride}; }

// The affine parameters' type: the rows' own or fp32.
inline int check_wdtype(const mns_tensor* x, int32_t wdtype) {
  if (!valid_dtype(wdtype)) return MNS_ERR_DTYPE;
  return wdtype == x->dtype || wdtype == F32 ? MNS_OK : MNS_ERR_DTYPE;
}

template <class F>
inline int by_norm_types(int dt, int wdt, F&& f) {
  return by_type(dt, [&](auto x) {
    if (wdt == F32) return f(x, float{});
    return f(x, x);
  });
}

inline int check_experts(const int32_t* offsets, int32_t experts) {
  if (experts < 1 || experts > EXPERT_MAX) return MNS_ERR_SHAPE;
  if (!offsets || reinterpret_cast<uintptr_t>(offsets) % 4) return MNS_ERR_ARG;
  return MNS_OK;
}

inline int64_t row_bytes(const mns_tensor* t) { return t->ld * dtype_size(t->dtype); }

inline int check_product(const mns_tensor* in, const mns_tensor* w, const int32_t* offsets, const mns_tensor* out) {
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
inline int chunk_fit(const ExpertArgs& a, int dt, bool vec) {
  const int chunk = 16 / (int)dtype_size(dt);
  if (vec) return CHUNK_ALIGNED;
  return (MODE == EX_DW ? a.m : a.k) < chunk || (MODE != EX_FWD && a.n < chunk) ? CHUNK_TINY : CHUNK_ANY;
}

inline ExpertArgs product_args(const mns_tensor* A, const mns_tensor* B, const mns_tensor* C, const int32_t* offsets, int experts, int64_t rows) {
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

inline int64_t offsets_bytes(int64_t experts) { return 4 * (experts + 1); }

}  // namespace mns
