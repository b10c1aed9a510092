"""The experts' tile list on the host: the functions of expert_gemm.hpp that the kernels walk it with, compiled for
the CPU, on offsets that expert_sort would not write. Whatever the offsets hold, a tile belongs to an expert that
exists and lies within the rows of its operands."""
import os
import subprocess

import pytest

from newton_schulz_matrix_muon_amd import build as b

SOURCE = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include <hip/hip_runtime.h>
#include "layer/expert_gemm.hpp"
using namespace mns;

static int bad(const char* what, long long a, long long b) { std::printf("%s: %lld %lld\n", what, a, b); return 1; }

// The list as expert_tiles, expert_list and expert_tile make it: 0 if every tile looked at is in order.
static int walk(int experts, int64_t rows, int n, int bm, const std::vector<int32_t>& offsets, int64_t* total) {
  ExpertArgs p{};
  p.offsets = offsets.data();
  p.experts = experts;
  p.rows = rows;
  p.tiles_n = (n + bm - 1) / bm;
  std::vector<int> first(experts + 2);
  int64_t sum = 0;
  for (int e = 0; e <= experts + 1; ++e) {
    first[e] = list_rows(sum, p.tiles_n);
    int lo = 0, hi = 0;
    if (e <= experts) expert_rows(p, e, &lo, &hi);
    if (lo < 0 || hi < lo || hi > rows) return bad("rows", lo, hi);
    sum += (hi - lo + bm - 1) / bm;
    if (sum > 0x7fffffff) return bad("tile rows past 32 bits", sum, 0);
  }
  for (int e = 0; e <= experts + 1; ++e)
    if ((int64_t)first[e] * p.tiles_n > 0x7fffffff) return bad("tiles past 32 bits before expert", e, (int64_t)first[e] * p.tiles_n);
  *total = (int64_t)first[experts + 1] * p.tiles_n;
  unsigned long long x = 88172645463325252ull;
  for (int i = 0; i < 4000 && *total; ++i) {
    x ^= x << 13, x ^= x >> 7, x ^= x << 17;
    const int t = (int)(i == 0 ? 0 : i == 1 ? *total - 1 : (int64_t)(x % (unsigned long long)*total));
    int e = 0;
    for (int k = 0; k <= experts; ++k) e += ends_by(first.data(), k, p.tiles_n, t);
    if (e > experts) return bad("no expert has tile", t, e);
    int lo, hi;
    expert_rows(p, e, &lo, &hi);
    const int tm = first[e + 1] - first[e], r = t - first[e] * p.tiles_n;
    const TileAt at = tile_at(r, tm, p.tiles_n);
    if (r < 0 || at.row < 0 || at.row >= tm || at.col < 0 || at.col >= p.tiles_n) return bad("place of tile", t, r);
    if (lo + (int64_t)at.row * bm >= hi) return bad("tile behind its expert's rows", t, e);
  }
  return 0;
}

int main() {
  int64_t total = 0, whole = 0;
  // in order: every tile is there, none is cut
  for (int bm : {64, 128, 256}) {
    std::vector<int32_t> o{0, 5, 5, 700, 1300};
    if (walk(4, 1400, 2048, bm, o, &total)) return 1;
    const int64_t want = ((5 + bm - 1) / bm + (695 + bm - 1) / bm + (600 + bm - 1) / bm + (100 + bm - 1) / bm) * (2048 / bm);
    if (total != want) return bad("tiles", total, want);
    // the most tiles that the host accepts (128 x 128 ones, in order) are all listed
    std::vector<int32_t> one(2, 1 << 24);
    one[0] = 0;
    if (walk(1, 1 << 24, 1 << 20, 256, one, &whole)) return 1;
    if (whole != (1ll << 16) * (1 << 12)) return bad("tiles of the largest product", whole, 0);
  }
  // offsets that fall and rise again, up to the limits on experts, rows and columns; and ones of no order at all
  for (int experts : {3, 64, 1024})
    for (int64_t rows : {int64_t(1) << 16, (int64_t(1) << 24) - 1, int64_t(1) << 24})
      for (int n : {64, 4096, 1 << 20})
        for (int bm : {64, 128, 256}) {
          std::vector<int32_t> o(experts + 1), any(experts + 1);
          for (int e = 0; e <= experts; ++e) {
            o[e] = e & 1 ? (int32_t)rows : 0;
            any[e] = (int32_t)(2654435761u * (unsigned)(e + 7));
          }
          if (walk(experts, rows, n, bm, o, &total) || walk(experts, rows, n, bm, any, &total)) {
            std::printf("experts %d rows %lld n %d tile %d\n", experts, (long long)rows, n, bm);
            return 1;
          }
        }
  std::puts("in order");
  return 0;
}
"""


def test_every_tile_of_any_offsets_lies_in_its_operands(tmp_path):
    if not os.path.exists("/opt/rocm/bin/hipcc"):
        pytest.skip("no compiler")
    src, exe = tmp_path / "list.hip", str(tmp_path / "list")
    src.write_text(SOURCE)
    flags = [f for f in b.HIPCC_FLAGS if f not in ("-O3", "-shared")]
    r = subprocess.run([b.hipcc(), *flags, "-O1", "--cuda-host-only", "-I", os.path.join(b.ROOT, "include"), "-I", b.CSRC,
                        str(src), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "in order" in r.stdout, r.stdout + r.stderr
