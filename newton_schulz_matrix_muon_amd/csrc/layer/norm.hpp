// Layer norm over the columns of each row, and its gradients.
//
//   mean = sum(x) / D,  rstd = 1 / sqrt(sum((x - mean)^2) / D + eps),  xh = (x - mean) rstd
//   y  = xh w + b
//   g  = dy w,  dx = rstd (g - sum(g) / D - xh sum(g xh) / D)
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Every sum is fp32; y, dx, dw and db are rounded once, to their buffer's type. Sums run in a
// fixed order (no atomics), so a call's results are the same every time.
//
// Bound by HBM: the forward pass reads x and writes y, the backward pass reads x and dy and
// writes dx; a few flops per byte.
#pragma once

#include "../gemm.hpp"

namespace mns {

// A strided [batch][rows][cols] buffer seen as batch * rows rows.
struct RowsRef {
  char* p;
  int64_t rows_per, ld, stride;   // ld, stride in elements
};
template <typename T>
__device__ inline T* row_ptr(const RowsRef& a, int64_t r) {
  T* p = reinterpret_cast<T*>(a.p);
  if (r < a.rows_per) return p + r * a.ld;
  const int64_t b = r / a.rows_per;
  return p + b * a.stride + (r - b * a.rows_per) * a.ld;
}

struct NormArgs {
  RowsRef x, y, dy, dx;
  const void* w; const void* b;   // may be null: 1 and 0
  float* mean; float* rstd;
  int64_t rows; int cols;
  float eps, n;                  // n = cols
  float* part; int nparts;        // [nparts][2][cols]: dw and db of the rows part i took
  void* dw; void* db;             // may be null
};

template <typename T> __device__ inline float as_f32(T v) {
  if constexpr (__is_same(T, __bf16)) return bf16_bits_to_f32(__builtin_bit_cast(uint16_t, v));
  else return (float)v;
}
template <typename T> __device__ inline T from_f32(float v) {
  if constexpr (__is_same(T, __bf16)) return __builtin_bit_cast(__bf16, f32_to_bf16_bits(v));
  else return (T)v;
}

__device__ inline float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Sums of two values over the workgroup's NT threads, in every thread. `red`: 2 * 16 floats that
// no other reduction between two barriers uses.
template <int NT>
__device__ inline void block_sum2(float& a, float& b, float* red) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (NT > 64) {
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      red[2 * w] = a;
      red[2 * w + 1] = b;
    }
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) {
      a += red[2 * i];
      b += red[2 * i + 1];
    }
  }
}

// Rows of any length, any alignment: one workgroup per row, which it reads three times (twice
// from cache).
template <typename T, typename WT>
__global__ void __launch_bounds__(256) norm_fwd_any(const NormArgs p) {
  __shared__ float red[3][32];
  const int64_t r = blockIdx.x;
  const T* x = row_ptr<T>(p.x, r);
  T* y = row_ptr<T>(p.y, r);
  const WT* w = reinterpret_cast<const WT*>(p.w);
  const WT* b = reinterpret_cast<const WT*>(p.b);
  float s = 0.f, dummy = 0.f;
  for (int c = threadIdx.x; c < p.cols; c += 256) s += as_f32(x[c]);
  block_sum2<256>(s, dummy, red[0]);
  const float mean = s / p.n;
  float q = 0.f;
  for (int c = threadIdx.x; c < p.cols; c += 256) {
    const float d = as_f32(x[c]) - mean;
    q += d * d;
  }
  block_sum2<256>(q, dummy, red[1]);
  const float rstd = 1.f / __builtin_sqrtf(q / p.n + p.eps);
  for (int c = threadIdx.x; c < p.cols; c += 256) {
    float v = (as_f32(x[c]) - mean) * rstd;
    if (w) v *= as_f32(w[c]);
    if (b) v += as_f32(b[c]);
    y[c] = from_f32<T>(v);
  }
  if (threadIdx.x == 0) {
    p.mean[r] = mean;
    p.rstd[r] = rstd;
  }
}

template <typename T, typename WT>
__global__ void __launch_bounds__(256) norm_dx_any(const NormArgs p) {
  __shared__ float red[32];
  const int64_t r = blockIdx.x;
  const T* x = row_ptr<T>(p.x, r);
  const T* dy = row_ptr<T>(p.dy, r);
  T* dx = row_ptr<T>(p.dx, r);
  const WT* w = reinterpret_cast<const WT*>(p.w);
  const float mean = p.mean[r], rstd = p.rstd[r];
  float a = 0.f, b = 0.f;
  for (int c = threadIdx.x; c < p.cols; c += 256) {
    const float g = as_f32(dy[c]) * (w ? as_f32(w[c]) : 1.f), xh = (as_f32(x[c]) - mean) * rstd;
    a += g;
    b += g * xh;
  }
  block_sum2<256>(a, b, red);
  a /= p.n;
  b /= p.n;
  for (int c = threadIdx.x; c < p.cols; c += 256) {
    const float g = as_f32(dy[c]) * (w ? as_f32(w[c]) : 1.f), xh = (as_f32(x[c]) - mean) * rstd;
    dx[c] = from_f32<T>(rstd * (g - a - xh * b));
  }
}

// Partial dw and db: workgroup (column block, part) sums the part's rows, one column a thread.
template <typename T>
__global__ void __launch_bounds__(256) norm_dw_any(const NormArgs p) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  const int64_t part = blockIdx.y;
  if (c >= p.cols) return;
  float a = 0.f, b = 0.f;
  for (int64_t r = part; r < p.rows; r += p.nparts) {
    const float g = as_f32(row_ptr<T>(p.dy, r)[c]);
    a += g * ((as_f32(row_ptr<T>(p.x, r)[c]) - p.mean[r]) * p.rstd[r]);
    b += g;
  }
  p.part[part * 2 * p.cols + c] = a;
  p.part[(part * 2 + 1) * p.cols + c] = b;
}

// dw and db from the parts: 64 columns a workgroup, its 16 waves each take every 16th part.
template <typename WT>
__global__ void __launch_bounds__(1024) norm_dw_sum(const NormArgs p) {
  __shared__ float red[2][16][64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float a = 0.f, b = 0.f;
  if (c < p.cols)
    for (int i = wv; i < p.nparts; i += 16) {
      a += p.part[(int64_t)i * 2 * p.cols + c];
      b += p.part[((int64_t)i * 2 + 1) * p.cols + c];
    }
  red[0][wv][lane] = a;
  red[1][wv][lane] = b;
  __syncthreads();
  if (wv < 2 && c < p.cols) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += red[wv][i][lane];
    void* out = wv == 0 ? p.dw : p.db;
    if (out) reinterpret_cast<WT*>(out)[c] = from_f32<WT>(s);
  }
}

}  // namespace mns
