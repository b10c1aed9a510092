// The gated block of an expert (or of a dense layer): both projections, the activation and the product
// in one kernel, and its gradients.
//
//   gate = X Wg^T,  up = X Wu^T,  H = act(gate) * up
//   dgate = dH * up * act'(gate),  dup = dH * act(gate)
//   dX = dgate Wg + dup Wu,  dWg = dgate^T X,  dWu = dup^T X
//
//   silu  g s(g), s(g) = 1 / (1 + exp(-g));  slope s (1 + g (1 - s))
//   gelu  g F(g), F(g) = (1 + erf(g / sqrt 2)) / 2;  slope F + g exp(-g^2 / 2) / sqrt(2 pi)
//   relu  max(g, 0);  slope 1 where g > 0, else 0
//
// A gate that is no number stays one in every activation, so that H, dup and what they reach show it.
//
// The products are the experts' (expert_gemm.hpp, expert_pingpong.hpp) with two matrices each: a tile of the forward
// product holds 32 columns of either matrix side by side, so that a lane has gate and up of the same element; the
// input gradient's contraction runs through one matrix and on through the other; the weight gradients' tiles
// are those of both matrices, so X and its rows are shared in L2. Bound by MFMA and the board's power, by HBM where there
// are few rows. One MI355X: 32768 rows over 27 experts of 2048 x 7168 bf16, gate and up kept, 1760 us (1093
// TFLOP/s; a large plain product of the vendor's library 1360 to 1600); 24594 rows over 64 experts of 1408 x 2048 fp16, backward 800:
// gated_grad 70, input gradient 303 to 332, weight gradients 388 to 432; one token of 6 such experts 15.9 us (4.3
// TB/s with the launch).
//
// The activation takes the fp32 sums. What the backward pass needs is gate and up, kept in the rows' type.
// dgate and dup are rounded to that type as well, since they are operands of MFMAs: an error of half a
// step of independent sign per term, as much in the sums as the rounding of the result itself.
#pragma once

#include "expert_few.hpp"

namespace mns {

// The activation's value and slope.
template <typename T>
__device__ inline void activate_slope(float g, int act, float* a, float* slope) {
  if (act == ACT_SILU) {
    // 1 - s as t s: as a difference it is off by 2^-24, which g multiplies
    const float t = row_exp<T>(-g), s = 1.f / (1.f + t), rest = s > 0.f ? t * s : 1.f;
    *a = g * s;
    *slope = s * (1.f + g * rest);
  } else if (act == ACT_GELU) {
    float density;
    const float f = normal_part<T>(g, &density);
    *a = g * f;
    *slope = f + g * density * 0.39894228040143268f;
  } else {
    *a = g <= 0.f ? 0.f : g;   // NaN stays
    *slope = g > 0.f ? 1.f : 0.f;
  }
}

struct GatedGradArgs {
  const char* dh; const char* gate; const char* up;   // rows
  int64_t ldh, ldg, ldu;                              // elements
  char* dgate; char* dup; int64_t ld;                 // rows of whole 16-byte chunks, zeros behind the end
  const int32_t* offsets; int experts;                // may be null: every row is somebody's
  int64_t rows; int n, units;
};

// dgate and dup, eight columns a thread. Rows of nobody are left out: the products do not read them.
// Bound by HBM: three rows read and two written; 24594 x 1408 fp16 67 to 71 us at 4.9 to 5.2 TB/s.
template <typename T>
__global__ void __launch_bounds__(256) gated_grad(const GatedGradArgs p, int act) {
  constexpr int N = 16 / (int)sizeof(T);
  const int64_t first = block_id() * 256;
  const int64_t r0 = first / p.units;
  const unsigned x = (unsigned)(first - r0 * p.units) + threadIdx.x;
  const unsigned q = x / (unsigned)p.units;
  const int64_t r = r0 + q;
  bool own = r < p.rows && (!p.offsets || r < p.offsets[p.experts]);
  if (__any(!own && r < p.rows)) {
    // behind the last offset, which need not be the largest (expert_rows): no expert ends behind `end`
    int end = 0;
    for (int e = threadIdx.x & 63; e < p.experts; e += 64) end = max(end, p.offsets[e + 1] > p.offsets[e] ? p.offsets[e + 1] : 0);
#pragma unroll
    for (int o = 32; o; o >>= 1) end = max(end, __shfl_xor(end, o));
    own = r < min((int64_t)end, p.rows);
  }
  if (!own) return;
  const int c = (int)(x - q * (unsigned)p.units) * 8;
  auto load = [&](const char* base, int64_t ld, float (&f)[8]) {
    const T* row = reinterpret_cast<const T*>(base) + r * ld;
    if (c + 8 <= p.n) {
      u32x4 v[8 / N];
#pragma unroll
      for (int l = 0; l < 8 / N; ++l) v[l] = *reinterpret_cast<const u32x4_any*>(row + c + l * N);
      if constexpr (N == 8) VecIO<T>::unpack(v[0], f);
      else
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(v[e >> 2][e & 3]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = c + e < p.n ? as_f32(row[c + e]) : 0.f;
    }
  };
  float d[8], g[8], u[8], dg[8], du[8];
  load(p.dh, p.ldh, d);
  load(p.gate, p.ldg, g);
  load(p.up, p.ldu, u);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float a, slope;
    activate_slope<T>(g[e], act, &a, &slope);
    dg[e] = c + e < p.n ? d[e] * u[e] * slope : 0.f;
    du[e] = c + e < p.n ? d[e] * a : 0.f;
  }
  VecIO<T>::store(reinterpret_cast<T*>(p.dgate) + r * p.ld, c, dg);
  VecIO<T>::store(reinterpret_cast<T*>(p.dup) + r * p.ld, c, du);
}

// Few rows (generation): the time is that of reading both matrices once, as in expert_few_fwd: a
// workgroup takes 16 rows of either, its four waves every fourth piece of K.
template <typename T, int FIT>
__global__ void __launch_bounds__(256, 2) expert_few_gated(const GatedArgs p) {
  constexpr int U = 4;               // pieces of a wave in flight, of both matrices
  constexpr int N = 16 / sizeof(T), PIECE = 8 * N;
  __shared__ f32x4 part[3][2][64];
  const int lane = threadIdx.x & 63, wave = wave_uniform(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 16, l16 = lane & 15, q = lane >> 4;
  int lo, hi;
  const int e = nth_expert(p, blockIdx.y, &lo, &hi);
  if (e < 0) return;
  const int64_t own = e < p.experts ? e : 0, row = min(n0 + l16, p.n - 1);
  const T* G = reinterpret_cast<const T*>(p.B) + own * p.sB + row * p.ldb;
  const T* W = reinterpret_cast<const T*>(p.B2) + own * p.sB2 + row * p.ldb2;
  for (int r0 = lo; r0 < hi; r0 += 16) {
    const int r = r0 + l16;
    f32x4 gate = {0.f, 0.f, 0.f, 0.f}, up = gate;
    if (e < p.experts) {
      const T* X = reinterpret_cast<const T*>(p.A) + (int64_t)min(r, hi - 1) * p.lda;
      auto pieces = [&](int k0, auto cut_c) {
        constexpr bool cut = decltype(cut_c)::value, shift = cut && FIT == CHUNK_ANY;
        const u32x4 zero = {0, 0, 0, 0};
        u32x4 a[U][2], b[U][2], x[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const int k = k0 + u * 4 * PIECE + (q * 2 + v) * N, at = shift ? min(k, p.k - N) : k;
            const bool in = !cut || k < p.k;
            a[u][v] = in ? load_chunk<T, FIT>(G, at, p.k) : zero;
            b[u][v] = in ? load_chunk<T, FIT>(W, at, p.k) : zero;
            x[u][v] = in && r < hi ? load_chunk<T, FIT>(X, at, p.k) : zero;
          }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            if constexpr (shift) {
              const int k = k0 + u * 4 * PIECE + (q * 2 + v) * N, by = k - min(k, p.k - N);
              a[u][v] = drop_first<T>(a[u][v], by);
              b[u][v] = drop_first<T>(b[u][v], by);
              x[u][v] = drop_first<T>(x[u][v], by);
            }
            gate = mma16<T>(a[u][v], x[u][v], gate);
            up = mma16<T>(b[u][v], x[u][v], up);
          }
      };
      int k0 = wave * PIECE;
      for (; k0 + (4 * U - 3) * PIECE <= p.k; k0 += 4 * U * PIECE) pieces(k0, std::false_type{});
      if (k0 < p.k) pieces(k0, std::true_type{});
    }
    if (wave) {
      part[wave - 1][0][lane] = gate;
      part[wave - 1][1][lane] = up;
    }
    __syncthreads();
    if (!wave) {
#pragma unroll
      for (int w = 0; w < 3; ++w) {
        gate += part[w][0][lane];
        up += part[w][1][lane];
      }
      // lane (row l16 of X): columns n0 + 4 q .. + 3
      if (r < hi) {
        const int c = n0 + 4 * q;
        T* y = reinterpret_cast<T*>(p.C) + (int64_t)r * p.ldc + c;
        with_activation(p.act, [&](auto act) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (c + i < p.n) y[i] = from_f32<T>(activated<T, act.value>(gate[i]) * up[i]);
        });
        if (p.C2) {
          T* g = reinterpret_cast<T*>(p.C2) + (int64_t)r * p.ldc2 + c;
          T* w = reinterpret_cast<T*>(p.C3) + (int64_t)r * p.ldc3 + c;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (c + i < p.n) {
              g[i] = from_f32<T>(gate[i]);
              w[i] = from_f32<T>(up[i]);
            }
        }
      }
    }
    __syncthreads();
  }
}

}  // namespace mns
