// Host side of the operators around the layer: rms norm with the residual stream, token embeddings and
// AdamW with states in 8 bits. As in layer.hip, validation happens before any HIP call and a call only
// enqueues kernels on the caller's stream.

#include "muon_ns.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "adamw8.hpp"
#include "checks.hpp"
#include "embed.hpp"
#include "rms.hpp"

using namespace mns;

namespace {

// -------------------------------------------------------------------------------- rms norm

constexpr int held(int nt, int vpt) { return nt * vpt * 8; }
constexpr int kRmsHeld = held(1024, 2);   // backward: longer rows take the kernels that read them again

// Threads that hold a row, a chunk each, in whole waves. whole: past 256 threads as many on each of a CU's four
// SIMDs, so that as many workgroups fit a CU as its registers allow (backward, 16384 x 2500 132 us without and 116 with);
// forward kernels do better with none idle: 16384 rows, us without and with, 16-bit of 4500 columns 116 and 128 (in 8 bits
// 107 and 132), of 2816 71 and 72 (60 and 66); fp32 of 4500 212 and 213 (186 and 188), of 2500 130 and 131 (103 and 106).
int row_threads(int64_t cols, bool whole) {
  const int64_t nt = (cols + 511) / 512 * 64;
  return (int)std::min<int64_t>(1024, !whole || nt <= 256 ? nt : round_up(nt, 256));
}

// Workgroups that share the rows of a backward pass, each with a part of dweight: as many as the chip holds at
// once, 20 waves a CU (h as dh, 65536 x 700 in bf16: 95 us, with 16 or 32 waves 109 and 114; 16384 x 7168: 189, 189 and 194).
int rms_parts(int64_t rows, int64_t cols) {
  const bool wave = cols <= held(64, 1);                 // four rows at a time where a wave holds one
  const int64_t turns = wave ? (rows + 3) / 4 : rows;
  return (int)std::max<int64_t>(1, std::min<int64_t>(turns, 256 * (20 / ((wave ? 256 : row_threads(cols, true)) / 64))));
}

// Workgroups of a forward pass of `turns` rows (fours of them where a wave holds one): a row each, or as many as a CU holds
// at once, each of which has the next row on its way. us of a workgroup a row, of 16 and of 32 waves a CU:
//   bf16  16384 x 4500 147, 191, 128;  16384 x 7168 177, 188, 179 (in 8 bits 180, 194, 161);  8192 x 12000 203, 163, 166
//   fp32  16384 x 2500 130, 132, 149;  16384 x 4500 226, 214, 229;  4096 x 12000 188, 156, 155;  65536 x 700 153, 166, 170
// Six workgroups of five waves, or three of ten, do not run on a CU at once: the last of them come when the others
// have ended. us with so many and with one less: 16384 x 2500 75 and 61 (in 8 bits 70 and 58), 16384 x 4864 145 and 117
// (133 and 115), 4096 x 5120 31 and 28 (31 and 29); five of six waves and three of nine do (2816 71 and 70, 4500 116 and 120).
unsigned rms_groups(int64_t turns, int nt, int64_t cols, int es) {
  if (es == 4 && (cols <= held(64, 1) || nt < 256)) return (unsigned)turns;   // fewer than 2^32 threads: 2^24 rows of 192
  const int waves = es == 4 || cols > held(1024, 1) ? 16 : 32;
  const int fit = 64 * waves / nt - (waves == 32 && (nt == 320 || nt == 640) ? 1 : 0);
  return (unsigned)std::min<int64_t>(turns, (int64_t)device_cus() * fit);
}

template <typename T, typename WT, bool MX>
void launch_rms_fwd(const RmsArgs& a, hipStream_t s) {
  const int nt = a.cols <= held(64, 1) ? 256 : row_threads(a.cols, false);
  const dim3 g(rms_groups(a.cols <= held(64, 1) ? (a.rows + 3) / 4 : a.rows, nt, a.cols, sizeof(T)));
  if (a.cols <= held(64, 1)) hipLaunchKernelGGL((rms_fwd_row<T, WT, true, 1, MX>), g, dim3(nt), 0, s, a);
  else if (a.cols <= held(1024, 1)) hipLaunchKernelGGL((rms_fwd_row<T, WT, false, 1, MX>), g, dim3(nt), 0, s, a);
  else if (a.cols <= held(1024, 2)) hipLaunchKernelGGL((rms_fwd_row<T, WT, false, 2, MX>), g, dim3(nt), 0, s, a);
  else hipLaunchKernelGGL((rms_fwd_long<T, WT, MX>), grid_of(a.rows), dim3(1024), 0, s, a);
}

template <typename T, typename WT>
void launch_rms_bwd(const RmsArgs& a, hipStream_t s) {
  const dim3 g((unsigned)a.nparts);
  const int nt = row_threads(a.cols, true);
  if (a.cols <= held(64, 1)) hipLaunchKernelGGL((rms_bwd_row<T, WT, true, 1>), g, dim3(256), 32 * 64, s, a);
  else if (a.cols <= held(1024, 1)) hipLaunchKernelGGL((rms_bwd_row<T, WT, false, 1>), g, dim3(nt), 32 * nt, s, a);
  else hipLaunchKernelGGL((rms_bwd_row<T, WT, false, 2>), g, dim3(1024), 64 * 1024, s, a);
}

// Whether `out` is the very buffer `in`: a row of it is read before it is written, by the same threads.
bool same_buffer(const mns_tensor* out, const mns_tensor* in) {
  return out && in && out->ptr == in->ptr && same_rows(out, in) && (in->rows <= 1 || out->ld == in->ld) &&
         (in->batch <= 1 || out->stride == in->stride);
}
const Span kNoSpan = span(static_cast<const void*>(nullptr), 0);
Span span_or_none(const mns_tensor* t) { return t ? span(t) : kNoSpan; }

// What both forward calls check; *a is filled but for the output.
int rms_forward_args(const mns_tensor* X, const mns_tensor* R, const void* weight, int32_t wdtype, float eps, const mns_tensor* H,
                     const float* rstd, RmsArgs* a) {
  if (int st = check_rows(X)) return st;
  if ((R == nullptr) != (H == nullptr)) return MNS_ERR_ARG;
  if (R)
    for (const mns_tensor* t : {R, H}) {
      if (int st = check_rows(t)) return st;
      if (t->dtype != X->dtype) return MNS_ERR_DTYPE;
      if (!same_rows(X, t)) return MNS_ERR_SHAPE;
    }
  if (int st = check_wdtype(X, wdtype)) return st;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return MNS_ERR_ARG;
  const int64_t rows = X->batch * X->rows;
  if (rows && !rstd) return MNS_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(rstd) % 4 || reinterpret_cast<uintptr_t>(weight) % dtype_size(wdtype)) return MNS_ERR_ARG;
  a->x = rows_ref(X);
  if (R) {
    a->r = rows_ref(R);
    a->h = rows_ref(H);
  }
  a->w = weight;
  a->rstd = const_cast<float*>(rstd);
  a->rows = rows;
  a->cols = (int)X->cols;
  a->eps = eps;
  a->n = (float)X->cols;
  return MNS_OK;
}

// ------------------------------------------------------------------------------- embeddings

int check_tokens(const void* tokens, int32_t id_bytes, int64_t n) {
  if (id_bytes != 4 && id_bytes != 8) return MNS_ERR_DTYPE;
  if (n < 0 || n > kMaxRows) return MNS_ERR_SHAPE;
  if (n && !tokens) return MNS_ERR_ARG;
  return reinterpret_cast<uintptr_t>(tokens) % id_bytes ? MNS_ERR_ARG : MNS_OK;
}

// f(element, elements of a unit): whole 16-byte units where a row holds one.
template <class F>
int by_unit(int dt, int64_t cols, F&& f) {
  return by_type(dt, [&](auto x) {
    using T = decltype(x);
    constexpr int V = 16 / (int)sizeof(T);
    return cols >= V ? f(x, std::integral_constant<int, V>{}) : f(x, std::integral_constant<int, 1>{});
  });
}
int units_of(int64_t cols, int v) { return (int)((cols + v - 1) / v); }

// The workspace of a gradient, in bytes from its beginning.
struct EmbedPlan {
  int bits, passes, steps, nblocks;
  int64_t tiles, marks, sorted[2], hist, part, total;
};
EmbedPlan embed_plan(int64_t n, int64_t vocab, int64_t cols) {
  EmbedPlan e{};
  int width = 1;
  while (vocab >> width) ++width;
  e.passes = (width + 9) / 10;
  e.bits = (width + e.passes - 1) / e.passes;
  const int64_t waves = (n + EMBED_NT - 1) / EMBED_NT;   // 64-position steps per wave of one workgroup
  e.steps = (int)(n <= EMBED_ONE ? std::max<int64_t>(1, waves) : (waves + 255) / 256);
  e.nblocks = (int)std::max<int64_t>(1, (waves + e.steps - 1) / e.steps);
  e.tiles = (n + EMBED_TILE - 1) / EMBED_TILE;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += round_up(bytes, 16);
    return here;
  };
  e.marks = take(vocab);
  for (int64_t& s : e.sorted) s = take(8 * n);
  e.hist = take(n > EMBED_ONE ? 4 * (int64_t)e.nblocks * EMBED_DIGITS : 0);
  e.part = take(e.tiles > 1 ? 8 * e.tiles * cols : 0);
  e.total = at;
  return e;
}

// ------------------------------------------------------------------------------------ AdamW

int run_adamw8(int nt, void* const* params, const void* const* grads, uint8_t* const* m, uint8_t* const* ms, uint8_t* const* r,
               uint8_t* const* rs, const int64_t* numels, int dt, const mns_adamw8_params* ap, hipStream_t s) {
  Adam8Table t;
  t.lr = (float)ap->lr;
  t.beta1 = (float)ap->beta1;
  t.beta2 = (float)ap->beta2;
  t.one_beta1 = (float)(1.0 - ap->beta1);
  t.one_beta2 = (float)(1.0 - ap->beta2);
  t.eps = (float)ap->eps;
  t.wd_mul = (float)(1.0 - ap->lr * ap->weight_decay);
  const bool dev = ap->device_step != nullptr;
  t.bc1 = ap->bias_correction && !dev ? (float)adam8_correction(ap->beta1, (uint32_t)ap->step) : 1.f;
  t.bc2 = ap->bias_correction && !dev ? (float)std::sqrt(adam8_correction(ap->beta2, (uint32_t)ap->step)) : 1.f;
  t.step = ap->device_step;
  t.seed = adam8_seed(ap->seed);
  t.correct = ap->bias_correction;
  t.wide1 = ap->beta1;
  t.wide2 = ap->beta2;
  int i = 0;
  while (i < nt) {
    int k = 0;
    int64_t blocks = 0;
    for (; i < nt && k < ADAM8_MAXT; ++i) {
      if (numels[i] == 0) continue;
      const int64_t b = (numels[i] + ADAM8_CHUNK - 1) / ADAM8_CHUNK;
      // a grid holds fewer than 2^32 threads; the largest tensor, 2^34 elements, takes half of them
      static_assert((int64_t(1) << 34) / ADAM8_CHUNK <= UINT32_MAX / ADAM8_BLOCK, "a tensor fits a launch");
      if (blocks + b > UINT32_MAX / ADAM8_BLOCK) break;
      t.p[k] = params[i];
      t.g[k] = grads[i];
      t.m[k] = m[i];
      t.ms[k] = ms[i];
      t.r[k] = r[i];
      t.rs[k] = rs[i];
      t.numel[k] = numels[i];
      t.blk_start[k] = (int)blocks;
      t.key[k] = dev ? (uint32_t)i : adam8_key(t.seed, (uint32_t)ap->step, (uint32_t)i);
      blocks += b;
      ++k;
    }
    if (k == 0) continue;                                // only empty tensors were left
    t.blk_start[k] = (int)blocks;
    t.nt = k;
    if (int st = by_type(dt, [&](auto x) {
          using T = decltype(x);
          return launch(K_ADAMW, s, [&] {
            if (dev) hipLaunchKernelGGL((adamw8_kernel<T, true>), dim3((unsigned)blocks), dim3(ADAM8_BLOCK), 0, s, t);
            else hipLaunchKernelGGL((adamw8_kernel<T, false>), dim3((unsigned)blocks), dim3(ADAM8_BLOCK), 0, s, t);
          });
        }))
      return st;
  }
  return MNS_OK;
}

}  // namespace

// ==========================================================================================
extern "C" {

int rms_norm(const mns_tensor* X, const mns_tensor* R, const void* weight, int32_t wdtype, float eps, const mns_tensor* Y,
             const mns_tensor* H, float* rstd, void* stream) {
  RmsArgs a{};
  if (int st = rms_forward_args(X, R, weight, wdtype, eps, H, rstd, &a)) return st;
  if (int st = check_rows(Y)) return st;
  if (Y->dtype != X->dtype) return MNS_ERR_DTYPE;
  if (!same_rows(X, Y)) return MNS_ERR_SHAPE;
  const Span w = span(weight, X->cols * dtype_size(wdtype)), st = span(rstd, 4 * a.rows), h = span_or_none(H), r = span_or_none(R);
  const bool kept = same_buffer(H, R);
  if (clash({span(Y), st}, {span(X), w, r, h}) || clash({h}, {span(X), w, st, kept ? kNoSpan : r})) return MNS_ERR_ARG;
  if (!a.rows) return MNS_OK;
  a.y = rows_ref(Y);
  const hipStream_t s = as_stream(stream);
  return by_norm_types(X->dtype, wdtype, [&](auto x, auto wt) {
    return launch(K_LAYER_NORM, s, [&] { launch_rms_fwd<decltype(x), decltype(wt), false>(a, s); });
  });
}

int rms_norm_mx8(const mns_tensor* X, const mns_tensor* R, const void* weight, int32_t wdtype, float eps, uint8_t* q, uint8_t* scales,
                 const mns_tensor* H, float* rstd, void* stream) {
  RmsArgs a{};
  if (int st = rms_forward_args(X, R, weight, wdtype, eps, H, rstd, &a)) return st;
  if (a.rows && (!q || !scales)) return MNS_ERR_ARG;
  a.blocks = (a.cols + MX_BLOCK - 1) / MX_BLOCK;
  const Span w = span(weight, X->cols * dtype_size(wdtype)), st = span(rstd, 4 * a.rows), h = span_or_none(H), r = span_or_none(R);
  const Span out = span(q, a.rows * a.cols), sc = span(scales, a.rows * a.blocks);
  const bool kept = same_buffer(H, R);
  if (clash({out, sc, st}, {span(X), w, r, h}) || clash({h}, {span(X), w, st, kept ? kNoSpan : r})) return MNS_ERR_ARG;
  if (!a.rows) return MNS_OK;
  a.q = q;
  a.scales = scales;
  const hipStream_t s = as_stream(stream);
  return by_norm_types(X->dtype, wdtype, [&](auto x, auto wt) {
    return launch(K_LAYER_NORM, s, [&] { launch_rms_fwd<decltype(x), decltype(wt), true>(a, s); });
  });
}

int mns_rms_norm_workspace_bytes(const mns_tensor* X, size_t* bytes) {
  if (!X || !bytes) return MNS_ERR_ARG;
  mns_tensor t = *X;
  t.ptr = t.rows > 0 ? reinterpret_cast<void*>(16) : nullptr;   // the pointer does not matter here
  if (int st = check_rows(&t)) return st;
  *bytes = (size_t)rms_parts(X->batch * X->rows, X->cols) * (size_t)X->cols * 4;
  return MNS_OK;
}

int rms_norm_backward(const mns_tensor* dY, const mns_tensor* H, const float* rstd, const void* weight, int32_t wdtype, const mns_tensor* dH,
                      const mns_tensor* dX, void* dweight, void* ws, size_t ws_bytes, void* stream) {
  for (const mns_tensor* t : {dY, H, dX, dH ? dH : dY}) {
    if (int st = check_rows(t)) return st;
    if (t->dtype != dY->dtype) return MNS_ERR_DTYPE;
    if (!same_rows(t, dY)) return MNS_ERR_SHAPE;
  }
  if (int st = check_wdtype(H, wdtype)) return st;
  const int64_t rows = H->batch * H->rows;
  if (rows && !rstd) return MNS_ERR_ARG;
  for (const void* w : {weight, (const void*)dweight})
    if (reinterpret_cast<uintptr_t>(w) % dtype_size(wdtype)) return MNS_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(rstd) % 4) return MNS_ERR_ARG;
  const size_t need = (size_t)rms_parts(rows, H->cols) * (size_t)H->cols * 4;
  if (dweight && rows && (!ws || ws_bytes < need || !aligned16(ws))) return MNS_ERR_WORKSPACE;
  const int64_t wb = H->cols * dtype_size(wdtype);
  if (clash({span(dX), span(dweight, wb), span(dweight ? ws : nullptr, (int64_t)need)},
            {span(dY), span(H), span(rstd, 4 * rows), span(weight, wb), same_buffer(dX, dH) ? kNoSpan : span_or_none(dH)}))
    return MNS_ERR_ARG;
  if (dH && clash({span(dweight, wb), span(dweight ? ws : nullptr, (int64_t)need)}, {span(dH)})) return MNS_ERR_ARG;
  RmsArgs a{};
  a.h = rows_ref(H);
  a.dy = rows_ref(dY);
  a.dx = rows_ref(dX);
  if (dH) a.dh = rows_ref(dH);
  a.w = weight;
  a.rstd = const_cast<float*>(rstd);
  a.rows = rows;
  a.cols = (int)H->cols;
  a.n = (float)H->cols;
  a.part = dweight ? reinterpret_cast<float*>(ws) : nullptr;
  a.nparts = rows ? rms_parts(rows, H->cols) : 0;
  a.dw = dweight;
  const hipStream_t s = as_stream(stream);
  return by_norm_types(H->dtype, wdtype, [&](auto x, auto w) {
    using T = decltype(x);
    using WT = decltype(w);
    if (rows && a.cols <= kRmsHeld) {
      if (int st = launch(K_LAYER_NORM, s, [&] { launch_rms_bwd<T, WT>(a, s); })) return st;
    } else if (rows) {
      if (int st = launch(K_LAYER_NORM, s, [&] { hipLaunchKernelGGL((rms_dx_long<T, WT>), grid_of(rows), dim3(1024), 0, s, a); })) return st;
      if (dweight)
        if (int st = launch(K_LAYER_NORM, s, [&] {
              hipLaunchKernelGGL((rms_dw_long<T>), dim3((a.cols + 2047) / 2048, a.nparts), dim3(256), 0, s, a);
            }))
          return st;
    }
    if (!dweight) return (int)MNS_OK;
    return launch(K_LAYER_NORM, s, [&] { hipLaunchKernelGGL((rms_dw_sum<WT>), dim3((a.cols + 31) / 32), dim3(1024), 0, s, a); });
  });
}

int embed(const void* tokens, int32_t id_bytes, const mns_tensor* table, float scale, const mns_tensor* Y, void* stream) {
  for (const mns_tensor* t : {table, Y})
    if (int st = check_rows(t)) return st;
  if (table->dtype != Y->dtype) return MNS_ERR_DTYPE;
  if (table->batch != 1 || Y->batch != 1 || table->rows < 1 || table->cols != Y->cols) return MNS_ERR_SHAPE;
  if (int st = check_tokens(tokens, id_bytes, Y->rows)) return st;
  if (!std::isfinite(scale)) return MNS_ERR_ARG;
  if (clash({span(Y)}, {span(table), span(tokens, id_bytes * Y->rows)})) return MNS_ERR_ARG;
  if (!Y->rows) return MNS_OK;
  EmbedArgs a{};
  a.table = reinterpret_cast<const char*>(table->ptr);
  a.table_ld = row_bytes(table);
  a.y = reinterpret_cast<char*>(Y->ptr);
  a.y_ld = row_bytes(Y);
  a.tokens = tokens;
  a.n = Y->rows;
  a.vocab = (int)table->rows;
  a.cols = (int)table->cols;
  a.scale = scale;
  const hipStream_t s = as_stream(stream);
  return by_unit(Y->dtype, a.cols, [&](auto x, auto v) {
    using T = decltype(x);
    constexpr int V = decltype(v)::value;
    a.units = units_of(a.cols, V);
    const dim3 g = grid_of((a.n * a.units + 255) / 256);
    return launch(K_ROUTE, s, [&] {
      if (id_bytes == 4) hipLaunchKernelGGL((embed_rows<T, int32_t, V>), g, dim3(256), 0, s, a);
      else hipLaunchKernelGGL((embed_rows<T, int64_t, V>), g, dim3(256), 0, s, a);
    });
  });
}

int mns_embed_workspace_bytes(int64_t tokens, int64_t vocab, int64_t cols, size_t* bytes) {
  if (!bytes) return MNS_ERR_ARG;
  if (tokens < 0 || tokens > kMaxRows || vocab < 1 || vocab > kMaxRows || cols < 1 || cols > kMaxCols) return MNS_ERR_SHAPE;
  *bytes = (size_t)embed_plan(tokens, vocab, cols).total;
  return MNS_OK;
}

int embed_backward(const mns_tensor* dY, const void* tokens, int32_t id_bytes, float scale, const mns_tensor* dT, void* ws, size_t ws_bytes,
                   void* stream) {
  for (const mns_tensor* t : {dY, dT})
    if (int st = check_rows(t)) return st;
  if (dY->dtype != dT->dtype) return MNS_ERR_DTYPE;
  if (dT->batch != 1 || dY->batch != 1 || dT->rows < 1 || dT->cols != dY->cols) return MNS_ERR_SHAPE;
  if (int st = check_tokens(tokens, id_bytes, dY->rows)) return st;
  if (!std::isfinite(scale)) return MNS_ERR_ARG;
  const EmbedPlan e = embed_plan(dY->rows, dT->rows, dT->cols);
  if (!ws || ws_bytes < (size_t)e.total || !aligned16(ws)) return MNS_ERR_WORKSPACE;
  if (clash({span(dT), span(ws, e.total)}, {span(dY), span(tokens, id_bytes * dY->rows)})) return MNS_ERR_ARG;
  char* base = reinterpret_cast<char*>(ws);
  EmbedSortArgs p{};
  p.tokens = tokens;
  p.n = dY->rows;
  p.vocab = (int)dT->rows;
  p.bits = e.bits;
  p.passes = e.passes;
  p.steps = e.steps;
  p.nblocks = e.nblocks;
  for (int i = 0; i < 2; ++i) p.sorted[i] = reinterpret_cast<int2*>(base + e.sorted[i]);
  p.hist = reinterpret_cast<int32_t*>(base + e.hist);
  p.marks = reinterpret_cast<uint8_t*>(base + e.marks);
  const hipStream_t s = as_stream(stream);
  auto sort = [&](auto id) {
    using ID = decltype(id);
    if (!p.n) return launch(K_ROUTE, s, [&] { hipLaunchKernelGGL(embed_no_marks<256>, dim3((p.vocab + 4095) / 4096), dim3(256), 0, s, p); });
    if (p.n <= EMBED_ONE)
      return launch(K_ROUTE, s, [&] {
        if (p.steps <= 1) hipLaunchKernelGGL((embed_sort_one<ID, 1>), dim3(1), dim3(EMBED_NT), 0, s, p);
        else hipLaunchKernelGGL((embed_sort_one<ID, 4>), dim3(1), dim3(EMBED_NT), 0, s, p);
      });
    for (int pass = 0; pass < p.passes; ++pass) {
      if (int st = launch(K_ROUTE, s, [&] { hipLaunchKernelGGL(embed_sort_count<ID>, dim3(p.nblocks), dim3(EMBED_NT), 0, s, p, pass); })) return st;
      if (int st = launch(K_ROUTE, s, [&] { hipLaunchKernelGGL(embed_sort_place<ID>, dim3(p.nblocks), dim3(EMBED_NT), 0, s, p, pass); })) return st;
    }
    return (int)MNS_OK;
  };
  if (int st = id_bytes == 4 ? sort(int32_t{}) : sort(int64_t{})) return st;
  EmbedGradArgs a{};
  a.dy = reinterpret_cast<const char*>(dY->ptr);
  a.dy_ld = row_bytes(dY);
  a.dt = reinterpret_cast<char*>(dT->ptr);
  a.dt_ld = row_bytes(dT);
  a.sorted = p.sorted[(p.passes - 1) & 1];
  a.marks = p.marks;
  a.part = reinterpret_cast<float*>(base + e.part);
  a.n = p.n;
  a.tiles = e.tiles;
  a.vocab = p.vocab;
  a.cols = (int)dT->cols;
  a.scale = scale;
  return by_unit(dT->dtype, a.cols, [&](auto x, auto v) {
    using T = decltype(x);
    constexpr int V = decltype(v)::value;
    a.units = units_of(a.cols, V);
    a.tile_blocks = (a.tiles * a.units + 255) / 256;
    a.zero_blocks = ((int64_t)a.vocab * a.units + 256 * EMBED_ZERO - 1) / (256 * EMBED_ZERO);
    if (int st = launch(K_ROUTE, s, [&] {
          hipLaunchKernelGGL((embed_grad<T, V>), grid_of(a.tile_blocks + a.zero_blocks), dim3(256), 0, s, a);
        }))
      return st;
    if (a.tiles < 2) return (int)MNS_OK;
    a.gathered = a.tiles >= EMBED_GROUPS * EMBED_GROUP;
    auto columns = [&](dim3 g) {
      g.z = (a.cols + 511) / 512;
      return g;
    };
    const dim3 groups = columns(grid_of((a.tiles + EMBED_GROUP - 1) / EMBED_GROUP)), g = columns(grid_of(a.tiles - 1));
    if (a.gathered)
      if (int st = launch(K_ROUTE, s, [&] { hipLaunchKernelGGL(embed_gather<256>, groups, dim3(256), 0, s, a); })) return st;
    return launch(K_ROUTE, s, [&] { hipLaunchKernelGGL(embed_join<T>, g, dim3(256), 0, s, a); });
  });
}

int adamw8_step(int ntensors, void* const* params, const void* const* grads, uint8_t* const* exp_avg, uint8_t* const* exp_avg_scale,
                uint8_t* const* root, uint8_t* const* root_scale, const int64_t* numels, int32_t dtype, const mns_adamw8_params* ap,
                void* stream) {
  if (ntensors < 1 || !params || !grads || !exp_avg || !exp_avg_scale || !root || !root_scale || !numels || !ap) return MNS_ERR_ARG;
  if (!valid_dtype(dtype)) return MNS_ERR_DTYPE;
  for (double x : {ap->lr, ap->beta1, ap->beta2, ap->eps, ap->weight_decay})
    if (!std::isfinite((float)x)) return MNS_ERR_ARG;
  if (ap->beta1 < 0. || ap->beta1 >= 1. || ap->beta2 < 0. || ap->beta2 >= 1. || ap->eps < 0.) return MNS_ERR_ARG;
  if ((ap->bias_correction != 0 && ap->bias_correction != 1) || (!ap->device_step && ap->step < 1)) return MNS_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(ap->device_step) % 8) return MNS_ERR_ARG;
  // every buffer there (unless empty) and aligned to its elements, no two of them overlapping
  std::vector<std::pair<uintptr_t, uintptr_t>> iv;
  if (const uintptr_t at = reinterpret_cast<uintptr_t>(ap->device_step)) iv.push_back({at, at + 8});
  const uintptr_t es = (uintptr_t)dtype_size(dtype);
  for (int i = 0; i < ntensors; ++i) {
    if (numels[i] < 0) return MNS_ERR_ARG;
    if (numels[i] == 0) continue;
    if (numels[i] > (int64_t(1) << 34)) return MNS_ERR_SHAPE;   // the workgroups of one launch
    const uintptr_t n = (uintptr_t)numels[i], blocks = (n + MX_BLOCK - 1) / MX_BLOCK;
    const std::pair<const void*, uintptr_t> bufs[6] = {{params[i], n * es}, {grads[i], n * es},   {exp_avg[i], n},
                                                       {exp_avg_scale[i], blocks}, {root[i], n}, {root_scale[i], blocks}};
    for (int b = 0; b < 6; ++b) {
      const uintptr_t lo = reinterpret_cast<uintptr_t>(bufs[b].first);
      if (!lo || (b < 2 && lo % es)) return MNS_ERR_ARG;
      iv.push_back({lo, lo + bufs[b].second});
    }
  }
  std::sort(iv.begin(), iv.end());
  for (size_t k = 1; k < iv.size(); ++k)
    if (iv[k].first < iv[k - 1].second) return MNS_ERR_ARG;
  return run_adamw8(ntensors, params, grads, exp_avg, exp_avg_scale, root, root_scale, numels, dtype, ap, as_stream(stream));
}

}  // extern "C"
