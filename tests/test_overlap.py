"""Which outputs count as overlapping: overlap.hpp, compiled for the host, against the sets of bytes themselves."""
import os
import shutil
import subprocess

import pytest

from newton_schulz_matrix_muon_amd import build as b

SOURCE = r"""
#include <cstdio>
#include <set>
#include "layer/overlap.hpp"
using namespace mns;

static unsigned long long x = 88172645463325252ull;
static int64_t below(int64_t n) {
  x ^= x << 13, x ^= x >> 7, x ^= x << 17;
  return (int64_t)(x % (unsigned long long)n);
}
static mns_tensor make(int64_t at, int64_t batch, int64_t rows, int64_t cols, int64_t ld, int64_t stride) {
  mns_tensor t{};
  t.ptr = reinterpret_cast<void*>(0x10000 + at);
  t.batch = batch, t.rows = rows, t.cols = cols, t.ld = ld, t.stride = stride;
  return t;
}
static std::set<uintptr_t> bytes(const mns_tensor& t, int64_t es) {
  std::set<uintptr_t> s;
  for (int64_t i = 0; i < t.batch; ++i)
    for (int64_t r = 0; r < t.rows; ++r)
      for (int64_t c = 0; c < t.cols * es; ++c) s.insert((uintptr_t)t.ptr + (i * t.stride + r * t.ld) * es + c);
  return s;
}
static bool share(const std::set<uintptr_t>& a, const std::set<uintptr_t>& b) {
  for (uintptr_t v : a)
    if (b.count(v)) return true;
  return false;
}
static int check(const char* what, const mns_tensor& a, const mns_tensor& c, int64_t es, bool want) {
  const bool got = meet(span(&a, es), span(&c, es)), back = meet(span(&c, es), span(&a, es));
  if (got == want && back == want) return 0;
  std::printf("%s: %d %d, expected %d\n", what, got, back, want);
  return 1;
}

int main() {
  int bad = 0;
  for (int64_t es : {2, 4}) {
    // halves of one buffer's columns, and a column too many
    bad |= check("left and right half", make(0, 1, 40, 64, 128, 0), make(64 * es, 1, 40, 64, 128, 0), es, false);
    bad |= check("one column shared", make(0, 1, 40, 65, 128, 0), make(64 * es, 1, 40, 64, 128, 0), es, true);
    bad |= check("the right half's end is the next row", make(0, 1, 40, 64, 128, 0), make(64 * es, 1, 40, 65, 128, 0), es, true);
    bad |= check("three parts", make(128 * es, 1, 7, 64, 200, 0), make(20 * es, 1, 9, 108, 200, 0), es, false);
    bad |= check("the same rows", make(0, 1, 40, 64, 128, 0), make(0, 1, 40, 64, 128, 0), es, true);
    bad |= check("rows apart by whole rows", make(0, 1, 40, 64, 128, 0), make(128 * 5 * es, 1, 40, 64, 128, 0), es, true);
    // every other matrix, and the upper and lower half of each matrix
    bad |= check("every other matrix", make(0, 3, 5, 8, 8, 80), make(40 * es, 3, 5, 8, 8, 80), es, false);
    bad |= check("halves of the matrices", make(0, 3, 5, 8, 8, 80), make(40 * es, 2, 4, 8, 8, 80), es, false);
    bad |= check("a row of the other half", make(0, 3, 6, 8, 8, 80), make(40 * es, 3, 5, 8, 8, 80), es, true);
    bad |= check("columns of batches", make(0, 3, 5, 8, 16, 80), make(8 * es, 3, 5, 8, 16, 80), es, false);
    // behind each other, and one row in the gap of another buffer's
    bad |= check("behind each other", make(0, 1, 4, 8, 8, 0), make(32 * es, 1, 4, 8, 8, 0), es, false);
    bad |= check("a row in a gap", make(0, 1, 4, 8, 32, 0), make(40 * es, 1, 1, 16, 16, 0), es, false);
  }
  // any pair: "apart" is never said of buffers that share a byte; of equal steps it is exact
  long apart_pairs = 0;
  for (int i = 0; i < 60000 && !bad; ++i) {
    const int64_t es = below(2) ? 2 : 4, ld = 1 + below(12), other = below(3) ? ld : 1 + below(12);
    auto any = [&](int64_t l) {
      const int64_t rows = 1 + below(5), cols = 1 + below(l), batch = 1 + below(3);
      return make(es * below(80), batch, rows, cols, l, rows * l + (below(2) ? l * below(3) : below(9)));
    };
    const mns_tensor a = any(ld), c = any(other);
    const bool got = meet(span(&a, es), span(&c, es)), shared = share(bytes(a, es), bytes(c, es));
    if (shared && !got) bad = 1, std::printf("shared bytes called apart in pair %d\n", i);
    if (got != meet(span(&c, es), span(&a, es))) bad = 1, std::printf("not symmetric in pair %d\n", i);
    apart_pairs += !got;
  }
  if (apart_pairs < 1000) bad = 1, std::printf("only %ld pairs apart\n", apart_pairs);
  mns_tensor none = make(0, 1, 0, 8, 8, 0), some = make(0, 1, 4, 8, 8, 0);
  if (clash({span(&none, 2)}, {span(&some, 2)}) || clash({span(&some, 2)}, {span((const void*)nullptr, 64)}) || !clash({span(&some, 2)}, {span(some.ptr, 1)})) bad = 1;
  if (!bad) std::puts("in order");
  return bad;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no compiler")
def test_buffers_that_share_no_byte(tmp_path):
    src, exe = tmp_path / "overlap.cpp", str(tmp_path / "overlap")
    src.write_text(SOURCE)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                        "-I", os.path.join(b.ROOT, "include"), "-I", b.CSRC, str(src), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "in order" in r.stdout, r.stdout + r.stderr
