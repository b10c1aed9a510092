// Whether an output shares bytes with an input or another output (host code). Two buffers whose
// address ranges meet may still be apart: the halves of one wider buffer's columns, or every other
// matrix of a batch.
#pragma once

#include "muon_ns.h"

#include <cstdint>
#include <initializer_list>

namespace mns {

// A buffer's bytes, twice: pieces of `row_bytes` (its rows) every `row_step` bytes from lo on, and of
// `mat_bytes` (its matrices) every `mat_step`. A step of 0: one piece; of -1: at no common distance.
struct Span {
  uintptr_t lo, hi;
  int64_t row_step, row_bytes, mat_step, mat_bytes;
};

inline Span span(const void* p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  if (!p) bytes = 0;
  return {lo, lo + (uintptr_t)bytes, 0, bytes, 0, bytes};
}

inline Span span(const mns_tensor* t, int64_t elem) {
  if (!t->rows) return span(t->ptr, 0);
  const int64_t row = t->cols * elem, ld = t->ld * elem, mat = (t->rows - 1) * ld + row;
  const int64_t stride = t->batch > 1 ? t->stride * elem : 0;
  Span s = span(t->ptr, (t->batch - 1) * stride + mat);
  s.row_bytes = row;
  s.row_step = t->rows == 1 ? stride : t->batch == 1 || stride % ld == 0 ? ld : -1;
  s.mat_bytes = mat;
  s.mat_step = stride;
  return s;
}

// Whether pieces of `wa` bytes every `sa` bytes and of `wb` every `sb`, the first `ahead` bytes behind
// the others' first, are apart for their places within one step alone.
inline bool apart(int64_t sa, int64_t wa, int64_t sb, int64_t wb, int64_t ahead) {
  const int64_t step = sa ? sa : sb;
  if (step <= 0 || (sb && sb != step) || wa > step || wb > step) return false;
  const int64_t at = (ahead % step + step) % step;
  return at >= wa && at + wb <= step;
}

inline bool meet(const Span& a, const Span& b) {
  if (a.lo >= b.hi || b.lo >= a.hi) return false;
  const int64_t ahead = (int64_t)(b.lo - a.lo);
  return !apart(a.row_step, a.row_bytes, b.row_step, b.row_bytes, ahead) && !apart(a.mat_step, a.mat_bytes, b.mat_step, b.mat_bytes, ahead);
}

// Each of `out` against all.
inline bool clash(std::initializer_list<Span> out, std::initializer_list<Span> in) {
  for (auto a = out.begin(); a != out.end(); ++a) {
    if (a->lo == a->hi) continue;
    for (auto b = out.begin(); b != a; ++b)
      if (meet(*a, *b)) return true;
    for (const Span& b : in)
      if (meet(*a, b)) return true;
  }
  return false;
}

}  // namespace mns
