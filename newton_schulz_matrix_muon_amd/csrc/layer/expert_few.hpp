// The experts' forward product when each expert has few rows (tokens while text is generated): the
// time is that of reading the weights of the experts that have rows, once, so the work is cut
// along the weights, 16 of their rows a workgroup, until every CU reads.
//
// One MI355X, bf16, weights from HBM: 64 experts of 1408 x 2048, 6 rows 14.6 us (128 x 128 tiles:
// 33.4), 64 rows 51 us at 4.8 TB/s (60), 256 rows 77 us (103), 1024 rows 126 us (104); 27 experts
// of 2048 x 7168, 27 rows 93 us at 5.7 TB/s (146), 108 rows 145 us (156), 216 rows 174 us (158).
// So it serves up to four rows an expert. The input gradient stays on the tiles: they read W by
// whole rows, 5.2 TB/s from one row an expert on.
#pragma once

#include "expert_gemm.hpp"

namespace mns {

// The slot-th expert that has rows (counting the rows of nobody as expert E), or -1; its rows.
// Equal in every lane.
__device__ inline int nth_expert(const ExpertArgs& p, int slot, int* lo, int* hi) {
  const int lane = threadIdx.x & 63;
  for (int e0 = 0; e0 <= p.experts; e0 += 64) {
    int a = 0, b = 0;
    if (e0 + lane <= p.experts) expert_rows(p, e0 + lane, &a, &b);
    const uint64_t some = __ballot(b > a);
    const int n = __builtin_popcountll(some);
    if (slot < n) {
      uint64_t m = some;
      for (int i = 0; i < slot; ++i) m &= m - 1;
      const int l = __builtin_ctzll(m);
      *lo = __builtin_amdgcn_readlane(a, l);
      *hi = __builtin_amdgcn_readlane(b, l);
      return e0 + l;
    }
    slot -= n;
  }
  return -1;
}

template <typename T>
__device__ inline f32x4 mma16(const typename Frag<T>::type& a, const typename Frag<T>::type& b, f32x4 c) {
  if constexpr (__is_same(T, __bf16)) return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  else return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Forward: a workgroup takes 16 rows of one expert's W against 16 rows of X at a time; its four
// waves take every fourth 64-wide piece of K, whose 128 bytes four lanes of a row read whole (the
// order of the contraction within a piece does not matter as long as both operands agree), and
// their sums meet in LDS. One wave's pieces are loaded four at a time.
template <typename T>
__global__ void __launch_bounds__(256) expert_few_fwd(const ExpertArgs p) {
  typedef typename Frag<T>::type F;
  constexpr int U = 8;               // pieces of a wave in flight
  __shared__ f32x4 part[3][64];
  const int lane = threadIdx.x & 63, wave = wave_uniform(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 16, l16 = lane & 15, q = lane >> 4;
  int lo, hi;
  const int e = nth_expert(p, blockIdx.y, &lo, &hi);
  if (e < 0) return;
  const T* W = reinterpret_cast<const T*>(p.B) + (int64_t)(e < p.experts ? e : 0) * p.sB + (int64_t)min(n0 + l16, p.n - 1) * p.ldb;
  for (int r0 = lo; r0 < hi; r0 += 16) {
    const int r = r0 + l16;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    if (e < p.experts) {
      const T* X = reinterpret_cast<const T*>(p.A) + (int64_t)min(r, hi - 1) * p.lda;
      const F zero = {};
      for (int k0 = wave * 64; k0 < p.k; k0 += 4 * U * 64) {
        F a[U][2], b[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const int k = k0 + u * 256 + q * 16 + v * 8;
            const bool in = k < p.k;
            a[u][v] = in ? *reinterpret_cast<const F*>(W + k) : zero;
            b[u][v] = in && r < hi ? *reinterpret_cast<const F*>(X + k) : zero;
          }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int v = 0; v < 2; ++v) acc = mma16<T>(a[u][v], b[u][v], acc);
      }
    }
    if (wave) part[wave - 1][lane] = acc;
    __syncthreads();
    if (!wave) {
#pragma unroll
      for (int w = 0; w < 3; ++w) acc += part[w][lane];
      // lane (row l16 of X): columns n0 + 4 q .. + 3
      if (r < hi) {
        T* y = reinterpret_cast<T*>(p.C) + (int64_t)r * p.ldc + n0 + 4 * q;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n0 + 4 * q + i < p.n) y[i] = from_f32<T>(acc[i]);
      }
    }
    __syncthreads();
  }
}

}  // namespace mns
