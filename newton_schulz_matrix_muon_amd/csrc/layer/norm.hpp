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
// writes dx; a few flops per byte. One MI355X, 16384 x 7168 bf16: forward 88 us, 5.3 TB/s (a large
// copy reaches 5.0 to 5.3); backward with dw and db 147 us, 4.8 TB/s.
#pragma once

#include "../gemm.hpp"

namespace mns {

// The workgroup's number in a grid of up to two dimensions: a dimension holds fewer than 2^32
// threads, which a workgroup per row can pass.
__device__ inline int64_t block_id() { return blockIdx.x + (int64_t)blockIdx.y * gridDim.x; }

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
    lds_barrier();   // the rows on their way and the stores of the last one stay in flight
    a = b = 0.f;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) {
      a += red[2 * i];
      b += red[2 * i + 1];
    }
  }
}

// Rows longer than the kernels below hold in registers: one workgroup per row, which it reads
// three times (twice from cache). 8192 x 16392 bf16: forward 384 us (1.4 TB/s), backward 538 (1.5).
template <typename T, typename WT>
__global__ void __launch_bounds__(256) norm_fwd_any(const NormArgs p) {
  __shared__ float red[3][32];
  const int64_t r = block_id();
  if (r >= p.rows) return;
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
  const int64_t r = block_id();
  if (r >= p.rows) return;
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

// ------------------------------------------------------------- a row in registers
// Eight elements of a row, as loaded: elements 8 u .. 8 u + 7 in one or two 16-byte accesses
// (VEC), or every nt-th element (any alignment; consecutive threads, consecutive elements).
// Elements past the row's end are zero and are not stored.
template <typename T, bool VEC>
struct Piece {
  typename VecIO<T>::raw v;
  T s[8];
  __device__ inline void load(const T* row, int i, int nt, int tid, int cols) {
    if constexpr (VEC) {
      const int c = (i * nt + tid) * 8;
      v = c < cols ? VecIO<T>::load_raw(row, c) : typename VecIO<T>::raw{};
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = (i * 8 + e) * nt + tid;
        s[e] = c < cols ? row[c] : (T)0.f;
      }
    }
  }
  __device__ inline void unpack(float (&f)[8]) const {
    if constexpr (VEC) {
      VecIO<T>::unpack(v, f);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = as_f32(s[e]);
    }
  }
};
template <bool VEC>
__device__ inline int piece_col(int i, int e, int nt, int tid) {
  return VEC ? (i * nt + tid) * 8 + e : (i * 8 + e) * nt + tid;
}
template <typename T, bool VEC>
__device__ inline void piece_store(T* row, int i, int nt, int tid, int cols, const float (&f)[8]) {
  if constexpr (VEC) {
    const int c = (i * nt + tid) * 8;
    if (c < cols) VecIO<T>::store(row, c, f);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = (i * 8 + e) * nt + tid;
      if (c < cols) row[c] = from_f32<T>(f[e]);
    }
  }
}

// Forward: NT threads hold a row, VPT pieces each; x is read once, the mean and then the variance
// come from the registers. NT = 64: four rows a workgroup, no barrier. 16384 x 7168 bf16: 390 us
// when a row is read three times (twice from cache), 88 so; one row 3.3 us.
template <typename T, typename WT, int NT, int VPT, bool VEC>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT) norm_fwd_row(const NormArgs p) {
  __shared__ float red[2][32];
  const int tid = threadIdx.x % NT;
  const int64_t r = block_id() * (NT < 256 ? 256 / NT : 1) + threadIdx.x / NT;
  if (r >= p.rows) return;   // whole waves (NT = 64), else the whole workgroup
  const T* x = row_ptr<T>(p.x, r);
  Piece<T, VEC> px[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) px[i].load(x, i, NT, tid, p.cols);
  Piece<WT, VEC> pw[VPT], pb[VPT];
  if (p.w) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) pw[i].load(reinterpret_cast<const WT*>(p.w), i, NT, tid, p.cols);
  }
  if (p.b) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) pb[i].load(reinterpret_cast<const WT*>(p.b), i, NT, tid, p.cols);
  }
  float v[VPT][8], s = 0.f, dummy = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    px[i].unpack(v[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) s += v[i][e];
  }
  block_sum2<NT>(s, dummy, red[0]);
  const float mean = s / p.n;
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[i][e] = piece_col<VEC>(i, e, NT, tid) < p.cols ? v[i][e] - mean : 0.f;
      q += v[i][e] * v[i][e];
    }
  block_sum2<NT>(q, dummy, red[1]);
  const float rstd = 1.f / __builtin_sqrtf(q / p.n + p.eps);
  T* y = row_ptr<T>(p.y, r);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = v[i][e] * rstd;
    if (p.w) {
      float w[8];
      pw[i].unpack(w);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= w[e];
    }
    if (p.b) {
      float b[8];
      pb[i].unpack(b);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] += b[e];
    }
    piece_store<T, VEC>(y, i, NT, tid, p.cols, f);
  }
  if (tid == 0) {
    p.mean[r] = mean;
    p.rstd[r] = rstd;
  }
}

// Backward: a workgroup walks every gridDim.x-th row (or four of them, NT = 64) with the next
// row's x and dy already on their way, and keeps its columns' dw and db in registers; they leave
// once, as one part, for norm_dw_sum to add up. 16384 x 7168 bf16: 345 us with a barrier that waits
// for the loads on their way as well, 141 with one that waits for LDS only and w in LDS, not in
// registers (which spilled); 1021 x 2047 fp32, any alignment, 11 us.
//
// From 8193 columns on (1024 threads, two pieces each) a lane's row and sums do not fit its 128 registers:
// 28 to 56 bytes of it lie in scratch, 188 to 196 where rows begin anywhere. 8192 rows bf16: 8192 columns
// 88 us (4.6 TB/s), 12000 columns 153 us (3.9), 12001 columns 793 us (0.7).
template <typename T, typename WT, int NT, int VPT, bool VEC>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT, NT >= 512 ? 4 : 1) norm_bwd_row(const NormArgs p) {
  constexpr int RPW = NT < 256 ? 256 / NT : 1;
  constexpr bool AHEAD = NT * VPT < 2048;   // the longest rows leave no registers for the next one
  __shared__ float red[2][32];
  __shared__ f32x4 w[VPT][2][NT];   // the weight: kept out of the registers
  const int tid = threadIdx.x % NT, sub = threadIdx.x / NT;
  float aw[VPT][8], ab[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) aw[i][e] = ab[i][e] = 0.f;
    if (sub == 0) {
      float f[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
      if (p.w) {
        Piece<WT, VEC> pw;
        pw.load(reinterpret_cast<const WT*>(p.w), i, NT, tid, p.cols);
        pw.unpack(f);
      }
      w[i][0][tid] = f32x4{f[0], f[1], f[2], f[3]};
      w[i][1][tid] = f32x4{f[4], f[5], f[6], f[7]};
    }
  }
  __syncthreads();
  const int64_t step = (int64_t)gridDim.x * RPW;
  int64_t r = (int64_t)blockIdx.x * RPW + sub;
  Piece<T, VEC> px[VPT], pg[VPT];
  float mean = 0.f, rstd = 0.f;
  auto fetch = [&](int64_t row) {
    const T* x = row_ptr<T>(p.x, row);
    const T* g = row_ptr<T>(p.dy, row);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      px[i].load(x, i, NT, tid, p.cols);
      pg[i].load(g, i, NT, tid, p.cols);
    }
    mean = p.mean[row];
    rstd = p.rstd[row];
  };
  if (AHEAD && r < p.rows) fetch(r);
  for (int flip = 0; r < p.rows; r += step, flip ^= 1) {
    if (!AHEAD) fetch(r);
    float xh[VPT][8], g[VPT][8], a = 0.f, b = 0.f;
    const float rs = rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      px[i].unpack(xh[i]);
      pg[i].unpack(g[i]);
      const f32x4 w0 = w[i][0][tid], w1 = w[i][1][tid];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xh[i][e] = (xh[i][e] - mean) * rs;
        aw[i][e] += g[i][e] * xh[i][e];
        ab[i][e] += g[i][e];
        g[i][e] *= e < 4 ? w0[e & 3] : w1[e & 3];
        a += g[i][e];
        b += g[i][e] * xh[i][e];
      }
    }
    if (AHEAD && r + step < p.rows) fetch(r + step);
    block_sum2<NT>(a, b, red[flip]);
    a /= p.n;
    b /= p.n;
    T* dx = row_ptr<T>(p.dx, r);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = rs * (g[i][e] - a - xh[i][e] * b);
      piece_store<T, VEC>(dx, i, NT, tid, p.cols, f);
    }
  }
  if (!p.part) return;
  if constexpr (RPW > 1) {   // the four waves' sums meet in the first, in order
    __shared__ float sum[RPW - 1][2][NT * VPT * 8];
    if (sub) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          sum[sub - 1][0][(i * 8 + e) * NT + tid] = aw[i][e];
          sum[sub - 1][1][(i * 8 + e) * NT + tid] = ab[i][e];
        }
    }
    __syncthreads();
    if (sub) return;
    for (int k = 0; k < RPW - 1; ++k)
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          aw[i][e] += sum[k][0][(i * 8 + e) * NT + tid];
          ab[i][e] += sum[k][1][(i * 8 + e) * NT + tid];
        }
  }
  float* part = p.part + (int64_t)blockIdx.x * 2 * p.cols;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    piece_store<float, VEC>(part, i, NT, tid, p.cols, aw[i]);
    piece_store<float, VEC>(part + p.cols, i, NT, tid, p.cols, ab[i]);
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

// dw (blockIdx.y = 0) or db (1) from the parts: 64 columns a workgroup, its 16 waves each take
// every 16th part, eight at a time: 6.4 us for 7168 columns of 512 parts.
template <typename WT>
__global__ void __launch_bounds__(1024) norm_dw_sum(const NormArgs p) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  void* out = blockIdx.y == 0 ? p.dw : p.db;
  if (!out) return;
  float a = 0.f;
  if (c < p.cols) {
    const float* part = p.part + (int64_t)blockIdx.y * p.cols + c;
    int i = wv;
    for (; i + 7 * 16 < p.nparts; i += 8 * 16) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = part[(int64_t)(i + 16 * u) * 2 * p.cols];
#pragma unroll
      for (int u = 0; u < 8; ++u) a += v[u];
    }
    for (; i < p.nparts; i += 16) a += part[(int64_t)i * 2 * p.cols];
  }
  red[wv][lane] = a;
  __syncthreads();
  if (wv == 0 && c < p.cols) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += red[i][lane];
    reinterpret_cast<WT*>(out)[c] = from_f32<WT>(s);
  }
}

}  // namespace mns
