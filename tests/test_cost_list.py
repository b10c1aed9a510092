"""The parts of a weight gradient's tile list that the eight XCDs take, on the host: cost_begin of expert_gemm.hpp on experts
of any numbers of rows. The parts follow each other, cover every tile, and cost the same but for one tile."""
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

static int check(const std::vector<int>& rows, int64_t T, const char* name) {
  const int E = (int)rows.size();
  std::vector<int> first(E + 2);
  for (int e = 0; e < E; ++e) {
    const int64_t next = (int64_t)first[e] + dw_cost(rows[e]);
    if (next > 0x7fffffff) return std::printf("%s: cost past 32 bits\n", name), 1;
    first[e + 1] = (int)next;
  }
  first[E + 1] = first[E];
  int64_t begin[9];
  for (int x = 0; x <= 8; ++x) {
    const int64_t target = cost_target(first.data(), E, T, x);
    int e = 0;
    for (int i = 0; i < E; ++i) e += first[i + 1] * T <= target;
    begin[x] = cost_begin(first.data(), E, T, x, e);
  }
  if (begin[0] != 0 || begin[8] != E * T) return std::printf("%s: %lld to %lld of %lld tiles\n", name, (long long)begin[0], (long long)begin[8], (long long)(E * T)), 1;
  int most = 0;
  for (int r : rows) most = std::max(most, dw_cost(r));
  auto cost = [&](int64_t t) { const int64_t e = t / T; return e >= E ? first[E] * T : first[e] * T + (t - e * T) * dw_cost(rows[e]); };
  for (int x = 0; x < 8; ++x) {
    if (begin[x + 1] < begin[x]) return std::printf("%s: part %d ends before it begins\n", name, x), 1;
    const int64_t part = cost(begin[x + 1]) - cost(begin[x]), even = first[E] * T / 8;
    if (part > even + most + 1 || part < even - most - 1) return std::printf("%s: part %d costs %lld of %lld\n", name, x, (long long)part, (long long)even), 1;
  }
  return 0;
}

int main() {
  unsigned long long s = 88172645463325252ull;
  auto rnd = [&] { return s ^= s << 13, s ^= s >> 7, s ^= s << 17, s; };
  for (int E : {1, 2, 7, 64, 1024})
    for (int64_t T : {int64_t(1), int64_t(3), int64_t(96), (int64_t(1) << 31) / E - 1}) {
      std::vector<int> even(E, 384), none(E, 0), one(E, 0), any(E), all(E, 1 << 24);
      one[E / 2] = 1 << 24;
      for (int& r : any) r = (int)(rnd() % 2000);
      if (check(even, T, "even") || check(none, T, "none") || check(one, T, "one") || check(any, T, "any") || check(all, T, "all")) {
        std::printf("%d experts, %lld tiles each\n", E, (long long)T);
        return 1;
      }
    }
  std::puts("in order");
  return 0;
}
"""


def test_parts_of_equal_cost_cover_every_tile(tmp_path):
    if not os.path.exists("/opt/rocm/bin/hipcc"):
        pytest.skip("no compiler")
    src, exe = tmp_path / "cost.hip", str(tmp_path / "cost")
    src.write_text(SOURCE)
    flags = [f for f in b.HIPCC_FLAGS if f not in ("-O3", "-shared")]
    r = subprocess.run([b.hipcc(), *flags, "-O1", "--cuda-host-only", "-I", os.path.join(b.ROOT, "include"), "-I", b.CSRC,
                        str(src), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "in order" in r.stdout, r.stdout + r.stderr
