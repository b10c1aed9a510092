// The experts' forward product when each expert has few rows (tokens while text is generated): the
// time is that of reading the weights of the experts that have rows, once, so the work is cut
// along the weights, 16 of their rows a workgroup, until every CU reads.
//
// One MI355X, bf16, weights from HBM (128 x 128 tiles in brackets), rows in all, each of an expert at
// random: 64 experts of 1408 x 2048, 6 rows 10.2 us (28), 64 rows 48 us at 4.9 TB/s (61), 256 rows 75 us
// (97); 27 experts of 2048 x 7168, 27 rows 96 us at 5.2 TB/s (147), 108 rows 150 us (153). The input gradient stays on the tiles: they read
// W by whole rows, 5.2 TB/s from one row an expert on.
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

// acc += the products of one 16-byte chunk of each operand's row: chunks of lanes q = 0..3 of a row
// are four parts of the contraction.
template <typename T>
__device__ inline f32x4 mma16(const u32x4& a, const u32x4& b, f32x4 c) {
  typedef typename Frag<T>::type F;
  const F x = __builtin_bit_cast(F, a), y = __builtin_bit_cast(F, b);
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[e], y[e], c, 0, 0, 0);
    return c;
  } else if constexpr (__is_same(T, __bf16)) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, c, 0, 0, 0);
  } else {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(x, y, c, 0, 0, 0);
  }
}

// Forward: a workgroup takes 16 rows of one expert's W against 16 rows of X at a time; its four
// waves take every fourth piece of K, whose 128 bytes four lanes of a row read whole (the order of
// the contraction within a piece does not matter as long as both operands agree), and their sums
// meet in LDS. One wave's pieces are loaded eight at a time.
// (Two waves a SIMD at least: up to 256 registers a lane the compiler takes the MFMAs whose sums are in
// vector registers. In accumulation registers it moves them out behind the loop's branch without the
// wait that the last product needs; build.py refuses a library with a kernel that has any.)
template <typename T, int FIT>
__global__ void __launch_bounds__(256, 2) expert_few_fwd(const ExpertArgs p) {
  constexpr int U = 8;               // pieces of a wave in flight
  constexpr int N = 16 / sizeof(T), PIECE = 8 * N;
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
      auto pieces = [&](int k0, auto cut_c) {
        constexpr bool cut = decltype(cut_c)::value, shift = cut && FIT == CHUNK_ANY;
        const u32x4 zero = {0, 0, 0, 0};
        u32x4 a[U][2], b[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const int k = k0 + u * 4 * PIECE + (q * 2 + v) * N, at = shift ? min(k, p.k - N) : k;
            const bool in = !cut || k < p.k;
            a[u][v] = in ? load_chunk<T, FIT>(W, at, p.k) : zero;
            b[u][v] = in && r < hi ? load_chunk<T, FIT>(X, at, p.k) : zero;
          }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            if constexpr (shift) {
              const int k = k0 + u * 4 * PIECE + (q * 2 + v) * N, by = k - min(k, p.k - N);
              a[u][v] = drop_first<T>(a[u][v], by);
              b[u][v] = drop_first<T>(b[u][v], by);
            }
            acc = mma16<T>(a[u][v], b[u][v], acc);
          }
      };
      int k0 = wave * PIECE;
      for (; k0 + (4 * U - 3) * PIECE <= p.k; k0 += 4 * U * PIECE) pieces(k0, std::false_type{});
      if (k0 < p.k) pieces(k0, std::true_type{});
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
