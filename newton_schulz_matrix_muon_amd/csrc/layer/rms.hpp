// Root-mean-square norm over the columns of each row, with the residual stream's addition in front
// and an output in 8 bits, and its gradients.
//
//   h    = x + r, rounded to the rows' type (no residual: h = x)
//   rstd = 1 / sqrt(sum(h^2) / D + eps),  y = h rstd w
//   g    = dy w,  xh = h rstd,  dx = rstd (g - xh sum(g xh) / D) + dh
//   dw   = sum over rows of dy xh
//
// dh is the gradient that reaches h along the stream; dx is the gradient of x and of r. The norm
// reads the rounded h, so that the backward pass, which has the rounded h, differentiates what
// the forward pass computed. Sums are fp32 in a fixed order; each result is rounded once.
//
// Bound by HBM: a few flops per byte, every input read once and every output written once, a row
// held in registers.
#pragma once

#include "mx8.hpp"

namespace mns {

struct RmsArgs {
  RowsRef x, r, h, y;             // r, h: p = null without a residual
  RowsRef dy, dh, dx;             // backward: h is the kept sum, dh may be null
  const void* w;                  // may be null: 1
  float* rstd;
  int64_t rows; int cols;
  float eps, n;                   // n = cols
  uint8_t* q; uint8_t* scales;    // 8-bit output: rows x cols codes, rows x blocks bytes
  int blocks;
  float* part; int nparts;        // [nparts][cols]: dw of the rows part i took
  void* dw;
};

// Elements c .. c + 7 of a row, as loaded. Rows begin anywhere: the hardware's loads take any
// element's address, so a chunk is loaded whole from a place clamped into the row, without a branch
// between loads, and moved into place (zeros behind the end). Rows shorter than a chunk go element
// by element.
template <typename T>
struct Chunk {
  static constexpr int N = 16 / (int)sizeof(T), L = 8 / N;
  u32x4 v[L];
  __device__ inline void load(const T* row, int c, int cols) {
    if (cols < N) {
      typedef T TN __attribute__((ext_vector_type(N)));
#pragma unroll
      for (int l = 0; l < L; ++l) {
        TN s;
#pragma unroll
        for (int e = 0; e < N; ++e) s[e] = c + l * N + e < cols ? row[c + l * N + e] : (T)0.f;
        v[l] = __builtin_bit_cast(u32x4, s);
      }
      return;
    }
#pragma unroll
    for (int l = 0; l < L; ++l) v[l] = *reinterpret_cast<const u32x4_any*>(row + min(c + l * N, cols - N));
    if (cols % N) {
#pragma unroll
      for (int l = 0; l < L; ++l) {
        const int by = min(c + l * N - min(c + l * N, cols - N), N);
        const unsigned __int128 w = __builtin_bit_cast(unsigned __int128, v[l]);
        v[l] = by < N ? __builtin_bit_cast(u32x4, w >> (by * (int)sizeof(T) * 8)) : u32x4{0, 0, 0, 0};
      }
    } else {
#pragma unroll
      for (int l = 0; l < L; ++l) v[l] = c + l * N < cols ? v[l] : u32x4{0, 0, 0, 0};
    }
  }
  __device__ inline void unpack(float (&f)[8]) const {
    if constexpr (L == 2) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(v[e >> 2][e & 3]);
    } else {
      VecIO<T>::unpack(v[0], f);
    }
  }
  __device__ inline void pack(const float (&f)[8]) {
    if constexpr (L == 2) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e >> 2][e & 3] = __float_as_uint(f[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[0][e] = pack2<T>(f[2 * e], f[2 * e + 1]);
    }
  }
  __device__ inline void store(T* row, int c, int cols) const {
    if (c + 8 <= cols) {
#pragma unroll
      for (int l = 0; l < L; ++l) *reinterpret_cast<u32x4_any*>(row + c + l * N) = v[l];
    } else if (c < cols) {
      typedef T TN __attribute__((ext_vector_type(N)));
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e < cols) row[c + e] = __builtin_bit_cast(TN, v[e / N])[e % N];
    }
  }
};

template <int NT>
__device__ inline float block_sum(float v, float* red) {
  v = wave_sum(v);
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    lds_barrier();   // loads and stores on their way stay in flight
    v = 0.f;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) v += red[i];
  }
  return v;
}

// y of eight columns, as the rows' type or in 8 bits (MX).
template <typename T, bool MX>
__device__ inline void rms_store(const RmsArgs& p, int64_t r, T* y, int c, const float (&f)[8]) {
  if constexpr (MX) {
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, finite_size(f[e]));
    const int byte = mx_byte(quad_max(top));
    if (c >= p.cols) return;
    const u32x2 codes = mx_codes(f, mx_divisor(byte));
    uint8_t* q = p.q + r * p.cols + c;
    if (c + 8 <= p.cols) {
      *reinterpret_cast<u32x2_any*>(q) = codes;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e < p.cols) q[e] = (uint8_t)(codes[e >> 2] >> (8 * (e & 3)));
    }
    if (c % MX_BLOCK == 0) p.scales[r * p.blocks + c / MX_BLOCK] = (uint8_t)byte;
  } else {
    Chunk<T> o;
    o.pack(f);
    o.store(y, c, p.cols);
  }
}

// NT threads hold a row, VPT chunks each (NT = 64: four rows a workgroup, no barrier).
template <typename T, typename WT, int NT, int VPT, bool MX>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT) rms_fwd_row(const RmsArgs p) {
  __shared__ float red[16];
  const int tid = threadIdx.x % NT;
  const int64_t r = block_id() * (NT < 256 ? 256 / NT : 1) + threadIdx.x / NT;
  if (r >= p.rows) return;   // whole waves (NT = 64), else the whole workgroup
  const T* x = row_ptr<T>(p.x, r);
  Chunk<T> px[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) px[i].load(x, (i * NT + tid) * 8, p.cols);
  if (p.r.p) {
    Chunk<T> pr[VPT];
    const T* res = row_ptr<T>(p.r, r);
#pragma unroll
    for (int i = 0; i < VPT; ++i) pr[i].load(res, (i * NT + tid) * 8, p.cols);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float a[8], b[8];
      px[i].unpack(a);
      pr[i].unpack(b);
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] += b[e];
      px[i].pack(a);
    }
  }
  Chunk<WT> pw[VPT];
  if (p.w) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) pw[i].load(reinterpret_cast<const WT*>(p.w), (i * NT + tid) * 8, p.cols);
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    float v[8];
    px[i].unpack(v);
#pragma unroll
    for (int e = 0; e < 8; ++e) s += v[e] * v[e];
  }
  // every load of the row has landed behind this sum: h may lie in the residual's own buffer
  s = block_sum<NT>(s, red);
  const float rstd = 1.f / __builtin_sqrtf(s / p.n + p.eps);
  if (p.h.p) {
    T* h = row_ptr<T>(p.h, r);
#pragma unroll
    for (int i = 0; i < VPT; ++i) px[i].store(h, (i * NT + tid) * 8, p.cols);
  }
  T* y = MX ? nullptr : row_ptr<T>(p.y, r);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    float f[8];
    px[i].unpack(f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= rstd;
    if (p.w) {
      float w[8];
      pw[i].unpack(w);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= w[e];
    }
    rms_store<T, MX>(p, r, y, (i * NT + tid) * 8, f);
  }
  if (tid == 0) p.rstd[r] = rstd;
}

// Rows longer than the kernels above hold: a workgroup of 1024 threads reads x and r twice, the
// second time from cache. A thread writes only elements of h that it alone reads.
template <typename T, typename WT, bool MX>
__global__ void __launch_bounds__(1024) rms_fwd_long(const RmsArgs p) {
  __shared__ float red[16];
  const int64_t r = block_id();
  if (r >= p.rows) return;
  const T* x = row_ptr<T>(p.x, r);
  const T* res = p.r.p ? row_ptr<T>(p.r, r) : nullptr;
  auto sum = [&](int c, Chunk<T>& v) {
    v.load(x, c, p.cols);
    if (!res) return;
    Chunk<T> o;
    o.load(res, c, p.cols);
    float a[8], b[8];
    v.unpack(a);
    o.unpack(b);
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] += b[e];
    v.pack(a);
  };
  float s = 0.f;
  for (int c = threadIdx.x * 8; c < p.cols; c += 8192) {
    Chunk<T> v;
    float f[8];
    sum(c, v);
    v.unpack(f);
#pragma unroll
    for (int e = 0; e < 8; ++e) s += f[e] * f[e];
  }
  s = block_sum<1024>(s, red);
  const float rstd = 1.f / __builtin_sqrtf(s / p.n + p.eps);
  T* h = p.h.p ? row_ptr<T>(p.h, r) : nullptr;
  T* y = MX ? nullptr : row_ptr<T>(p.y, r);
  // whole quads of lanes go round together (the columns behind the end are zeros)
  for (int c = threadIdx.x * 8; c / MX_BLOCK * MX_BLOCK < p.cols; c += 8192) {
    Chunk<T> v;
    float f[8];
    sum(c, v);
    if (h) v.store(h, c, p.cols);
    v.unpack(f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= rstd;
    if (p.w) {
      Chunk<WT> o;
      float w[8];
      o.load(reinterpret_cast<const WT*>(p.w), c, p.cols);
      o.unpack(w);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= w[e];
    }
    rms_store<T, MX>(p, r, y, c, f);
  }
  if (threadIdx.x == 0) p.rstd[r] = rstd;
}

// Backward: a workgroup walks every gridDim.x-th row (or four of them, NT = 64) with the next
// row's h and dy already on their way (dh, which is needed last, with its own row), and keeps its columns' dw in registers; they leave once,
// as one part, for rms_dw_sum to add up.
template <typename T, typename WT, int NT, int VPT>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT, NT >= 512 ? 4 : 1) rms_bwd_row(const RmsArgs p) {
  constexpr int RPW = NT < 256 ? 256 / NT : 1;
  constexpr bool AHEAD = NT * VPT < 2048;   // the longest rows leave no registers for the next one
  __shared__ float red[2][16];
  __shared__ f32x4 w[VPT][2][NT];           // the weight: kept out of the registers
  const int tid = threadIdx.x % NT, sub = threadIdx.x / NT;
  float aw[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) aw[i][e] = 0.f;
    if (sub == 0) {
      float f[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
      if (p.w) {
        Chunk<WT> pw;
        pw.load(reinterpret_cast<const WT*>(p.w), (i * NT + tid) * 8, p.cols);
        pw.unpack(f);
      }
      w[i][0][tid] = f32x4{f[0], f[1], f[2], f[3]};
      w[i][1][tid] = f32x4{f[4], f[5], f[6], f[7]};
    }
  }
  __syncthreads();
  const int64_t step = (int64_t)gridDim.x * RPW;
  int64_t r = (int64_t)blockIdx.x * RPW + sub;
  Chunk<T> ph[VPT], pg[VPT], pd[VPT];
  float rstd = 0.f;
  auto fetch = [&](int64_t row) {
    const T* h = row_ptr<T>(p.h, row);
    const T* g = row_ptr<T>(p.dy, row);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      ph[i].load(h, (i * NT + tid) * 8, p.cols);
      pg[i].load(g, (i * NT + tid) * 8, p.cols);
    }
    rstd = p.rstd[row];
  };
  if (AHEAD && r < p.rows) fetch(r);
  for (int flip = 0; r < p.rows; r += step, flip ^= 1) {
    if (!AHEAD) fetch(r);
    float xh[VPT][8], g[VPT][8], a = 0.f;
    const float rs = rstd;
    if (p.dh.p) {
      const T* d = row_ptr<T>(p.dh, r);
#pragma unroll
      for (int i = 0; i < VPT; ++i) pd[i].load(d, (i * NT + tid) * 8, p.cols);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      ph[i].unpack(xh[i]);
      pg[i].unpack(g[i]);
      const f32x4 w0 = w[i][0][tid], w1 = w[i][1][tid];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xh[i][e] *= rs;
        aw[i][e] += g[i][e] * xh[i][e];
        g[i][e] *= e < 4 ? w0[e & 3] : w1[e & 3];
        a += g[i][e] * xh[i][e];
      }
    }
    if (AHEAD && r + step < p.rows) fetch(r + step);
    a = block_sum<NT>(a, red[flip]) / p.n;
    T* dx = row_ptr<T>(p.dx, r);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float f[8], s[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = rs * (g[i][e] - xh[i][e] * a);
      if (p.dh.p) {
        pd[i].unpack(s);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] += s[e];
      }
      Chunk<T> o;
      o.pack(f);
      o.store(dx, (i * NT + tid) * 8, p.cols);
    }
  }
  if (!p.part) return;
  if constexpr (RPW > 1) {   // the four waves' sums meet in the first, in order
    __shared__ float sum[RPW - 1][NT * VPT * 8];
    if (sub) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[sub - 1][(i * 8 + e) * NT + tid] = aw[i][e];
    }
    __syncthreads();
    if (sub) return;
    for (int k = 0; k < RPW - 1; ++k)
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) aw[i][e] += sum[k][(i * 8 + e) * NT + tid];
  }
  float* part = p.part + (int64_t)blockIdx.x * p.cols;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    Chunk<float> o;
    o.pack(aw[i]);
    o.store(part, (i * NT + tid) * 8, p.cols);
  }
}

// Longer rows: dx by rows, a workgroup of 1024 threads that reads them twice, and dw by columns.
template <typename T, typename WT>
__global__ void __launch_bounds__(1024) rms_dx_long(const RmsArgs p) {
  __shared__ float red[16];
  const int64_t r = block_id();
  if (r >= p.rows) return;
  const T* h = row_ptr<T>(p.h, r);
  const T* dy = row_ptr<T>(p.dy, r);
  const T* dh = p.dh.p ? row_ptr<T>(p.dh, r) : nullptr;
  T* dx = row_ptr<T>(p.dx, r);
  const float rs = p.rstd[r];
  auto terms = [&](int c, float (&xh)[8], float (&g)[8]) {
    Chunk<T> a, b;
    a.load(h, c, p.cols);
    b.load(dy, c, p.cols);
    a.unpack(xh);
    b.unpack(g);
#pragma unroll
    for (int e = 0; e < 8; ++e) xh[e] *= rs;
    if (!p.w) return;
    Chunk<WT> o;
    float w[8];
    o.load(reinterpret_cast<const WT*>(p.w), c, p.cols);
    o.unpack(w);
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] *= w[e];
  };
  float a = 0.f;
  for (int c = threadIdx.x * 8; c < p.cols; c += 8192) {
    float xh[8], g[8];
    terms(c, xh, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) a += g[e] * xh[e];
  }
  a = block_sum<1024>(a, red) / p.n;
  for (int c = threadIdx.x * 8; c < p.cols; c += 8192) {
    float xh[8], g[8];
    terms(c, xh, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = rs * (g[e] - xh[e] * a);
    if (dh) {
      Chunk<T> d;
      float s[8];
      d.load(dh, c, p.cols);
      d.unpack(s);
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] += s[e];
    }
    Chunk<T> o;
    o.pack(g);
    o.store(dx, c, p.cols);
  }
}

// Partial dw: workgroup (2048 columns, part) sums the part's rows, eight columns a thread.
template <typename T>
__global__ void __launch_bounds__(256) rms_dw_long(const RmsArgs p) {
  const int c = (blockIdx.x * 256 + threadIdx.x) * 8;
  if (c >= p.cols) return;
  float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int64_t r = blockIdx.y; r < p.rows; r += p.nparts) {
    Chunk<T> h, g;
    float x[8], y[8];
    h.load(row_ptr<T>(p.h, r), c, p.cols);
    g.load(row_ptr<T>(p.dy, r), c, p.cols);
    h.unpack(x);
    g.unpack(y);
    const float rs = p.rstd[r];
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] += y[e] * (x[e] * rs);
  }
  Chunk<float> o;
  o.pack(a);
  o.store(p.part + (int64_t)blockIdx.y * p.cols, c, p.cols);
}

// dw from the parts: 64 columns a workgroup, its 16 waves each take every 16th part, eight at a time.
template <typename WT>
__global__ void __launch_bounds__(1024) rms_dw_sum(const RmsArgs p) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float a = 0.f;
  if (c < p.cols) {
    const float* part = p.part + c;
    int i = wv;
    for (; i + 7 * 16 < p.nparts; i += 8 * 16) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = part[(int64_t)(i + 16 * u) * p.cols];
#pragma unroll
      for (int u = 0; u < 8; ++u) a += v[u];
    }
    for (; i < p.nparts; i += 16) a += part[(int64_t)i * p.cols];
  }
  red[wv][lane] = a;
  __syncthreads();
  if (wv == 0 && c < p.cols) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += red[i][lane];
    reinterpret_cast<WT*>(p.dw)[c] = from_f32<WT>(s);
  }
}

}  // namespace mns
