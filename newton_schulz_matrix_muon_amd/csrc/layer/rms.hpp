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
// held in registers. One MI355X (a large copy reaches 4.9 TB/s), with the residual: 16384 x 7168 bf16
// forward 178 us at 5.3 TB/s, in 8 bits 160 at 5.2, backward 219 at 4.3; fp32 342, 281 and 348 (5.4 TB/s);
// 16383 x 2047 fp16, rows at any address, 55, 52 and 66 (4.9, 4.5 and 4.1 TB/s).
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

// Sum over a wave's lanes, in every lane: moves within rows of 16 lanes, then swaps of rows and halves
// (in one instruction each; through LDS, as __shfl goes, the sum takes several times as long).
__device__ inline float lanes_sum(float v) {
  auto moved = [](float x, auto ctrl_c) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), decltype(ctrl_c)::value, 0xf, 0xf, true));
  };
  v += moved(v, std::integral_constant<int, 0xb1>{});    // quads: 1 0 3 2
  v += moved(v, std::integral_constant<int, 0x4e>{});    // quads: 2 3 0 1
  v += moved(v, std::integral_constant<int, 0x141>{});   // half rows backwards
  v += moved(v, std::integral_constant<int, 0x140>{});   // rows backwards
  const auto rows = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(rows[0]) + __uint_as_float(rows[1]);
  const auto halves = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(halves[0]) + __uint_as_float(halves[1]);
}

// Sum over the workgroup's waves (up to 16), in every thread; within the wave alone where a wave has a row
// (WAVE). red: 16 floats that no other sum between two barriers uses, zero where there is no wave.
template <bool WAVE>
__device__ inline float block_sum(float v, f32x4* red) {
  v = lanes_sum(v);
  if constexpr (!WAVE) {
    if ((threadIdx.x & 63) == 0) reinterpret_cast<float*>(red)[threadIdx.x >> 6] = v;
    lds_barrier();   // loads and stores on their way stay in flight
    const f32x4 s = (red[0] + red[1]) + (red[2] + red[3]);
    v = (s[0] + s[1]) + (s[2] + s[3]);
  }
  return v;
}
// Zeros where block_sum has no wave; a barrier follows before the first sum's reads.
__device__ inline void clear_sums(f32x4* red, int n) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) red[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  __syncthreads();
}

// y of eight columns, as the rows' type or in 8 bits (MX).
template <typename T, bool MX>
__device__ inline void rms_store(const RmsArgs& p, int64_t r, T* y, int c, const float (&f)[8]) {
  if constexpr (MX) {
    bool odd;
    const int byte = mx_byte(quad_max(mx_top(f, &odd)));
    const float d = mx_divisor(byte);
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = f[e] * d;
    const u32x2 codes = mx_codes(f, v, odd);
    if (c >= p.cols) return;
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

// A row is held by a wave (WAVE: four rows a workgroup, no barrier) or by the workgroup, as many waves as it
// takes, VPT chunks a thread. A workgroup walks every gridDim.x-th row (or four of them) with the weight
// in registers and the next row's x and r already on their way (16384 x 7168 bf16, a row a workgroup and sums through
// LDS 190 us, in 8 bits 194). The barrier waits for the sums alone. One row of 7168 takes 3.4 us.
template <typename T, typename WT, bool WAVE, int VPT, bool MX>
__global__ void __launch_bounds__(WAVE ? 256 : 1024, !WAVE && VPT == 1 && sizeof(T) == 2 ? 8 : 1) rms_fwd_row(const RmsArgs p) {
  constexpr int RPW = WAVE ? 4 : 1;
  constexpr bool AHEAD = VPT == 1;
  __shared__ f32x4 red[2][4];
  const int NT = WAVE ? 64 : blockDim.x, tid = WAVE ? threadIdx.x & 63 : threadIdx.x;
  if constexpr (!WAVE) clear_sums(red[0], 8);
  const int64_t step = (int64_t)gridDim.x * RPW;
  // whole waves leave together (NT = 64), else the whole workgroup
  int64_t r = (int64_t)blockIdx.x * RPW + (WAVE ? threadIdx.x >> 6 : 0);
  if (r >= p.rows) return;
  Chunk<T> nx[VPT], nr[VPT];
  auto fetch = [&](int64_t row) {
    const T* x = row_ptr<T>(p.x, row);
#pragma unroll
    for (int i = 0; i < VPT; ++i) nx[i].load(x, (i * NT + tid) * 8, p.cols);
    if (!p.r.p) return;
    const T* res = row_ptr<T>(p.r, row);
#pragma unroll
    for (int i = 0; i < VPT; ++i) nr[i].load(res, (i * NT + tid) * 8, p.cols);
  };
  fetch(r);
  Chunk<WT> pw[VPT];
  if (p.w) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) pw[i].load(reinterpret_cast<const WT*>(p.w), (i * NT + tid) * 8, p.cols);
  }
  for (int flip = 0; r < p.rows; r += step, flip ^= 1) {
    Chunk<T> px[VPT];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float a[8];
      px[i] = nx[i];
      if (p.r.p) {
        float b[8];
        px[i].unpack(a);
        nr[i].unpack(b);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] += b[e];
        px[i].pack(a);
      }
      px[i].unpack(a);
#pragma unroll
      for (int e = 0; e < 8; ++e) s += a[e] * a[e];
    }
    if (AHEAD && r + step < p.rows) fetch(r + step);
    // every load of this row has landed behind the sum: h may lie in the residual's own buffer
    s = block_sum<WAVE>(s, red[flip]);
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
    if (!AHEAD && r + step < p.rows) fetch(r + step);
  }
}

// Rows longer than the kernels above hold (16384 columns): a workgroup of 1024 threads reads x and r twice, the
// second time from cache. A thread writes only elements of h that it alone reads.
template <typename T, typename WT, bool MX>
__global__ void __launch_bounds__(1024) rms_fwd_long(const RmsArgs p) {
  __shared__ f32x4 red[4];
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
  s = block_sum<false>(s, red);
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
// row's (16-bit types: the next two rows') h, dy and dh already on their way, and keeps its columns' dw in registers; they leave once,
// as one part, for rms_dw_sum to add up. The weight waits in LDS and the row stays as it was loaded, which is what lets
// 20 waves fit a CU: 16384 x 7168 bf16 290 us with both in registers and one row ahead, 219 so.
template <typename T, typename WT, bool WAVE, int VPT>
__global__ void __launch_bounds__(WAVE ? 256 : 1024, 4) rms_bwd_row(const RmsArgs p) {
  constexpr int RPW = WAVE ? 4 : 1;
  constexpr bool AHEAD = VPT == 1;          // the longest rows leave no registers for the next one
  constexpr int DEEP = VPT == 1 && sizeof(T) == 2 ? 2 : 1;   // rows on their way
  __shared__ f32x4 red[2][4];
  extern __shared__ f32x4 w[];              // the weight, [VPT][2][threads of a row]: kept out of the registers
  const int NT = WAVE ? 64 : blockDim.x, tid = WAVE ? threadIdx.x & 63 : threadIdx.x, sub = WAVE ? threadIdx.x >> 6 : 0;
  if constexpr (!WAVE) clear_sums(red[0], 8);
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
      w[2 * i * NT + tid] = f32x4{f[0], f[1], f[2], f[3]};
      w[(2 * i + 1) * NT + tid] = f32x4{f[4], f[5], f[6], f[7]};
    }
  }
  __syncthreads();
  const int64_t step = (int64_t)gridDim.x * RPW;
  int64_t r = (int64_t)blockIdx.x * RPW + sub;
  int flip = 0;
  Chunk<T> ph[DEEP][VPT], pg[DEEP][VPT], pd[DEEP][VPT];
  float rstd[DEEP];
  auto fetch = [&](auto slot_c, int64_t row) {
    constexpr int S = decltype(slot_c)::value;
    if (row >= p.rows) return;
    const T* h = row_ptr<T>(p.h, row);
    const T* g = row_ptr<T>(p.dy, row);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      ph[S][i].load(h, (i * NT + tid) * 8, p.cols);
      pg[S][i].load(g, (i * NT + tid) * 8, p.cols);
    }
    if (p.dh.p) {
      const T* d = row_ptr<T>(p.dh, row);
#pragma unroll
      for (int i = 0; i < VPT; ++i) pd[S][i].load(d, (i * NT + tid) * 8, p.cols);
    }
    rstd[S] = p.rstd[row];
  };
  // row r from slot S, whose next row is ordered while this one is added up
  auto row = [&](auto slot_c) {
    constexpr int S = decltype(slot_c)::value;
    // this row, as loaded: unpacked twice, which takes fewer registers than to keep it unpacked
    Chunk<T> h[VPT], dy[VPT], dh[VPT];
    const float rs = rstd[S];
    float a = 0.f;
    auto terms = [&](int i, float (&xh)[8], float (&g)[8]) {
      h[i].unpack(xh);
      dy[i].unpack(g);
#pragma unroll
      for (int e = 0; e < 8; ++e) xh[e] *= rs;
    };
    auto weigh = [&](int i, float (&g)[8]) {
      const f32x4 w0 = w[2 * i * NT + tid], w1 = w[(2 * i + 1) * NT + tid];
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] *= e < 4 ? w0[e & 3] : w1[e & 3];
    };
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      h[i] = ph[S][i];
      dy[i] = pg[S][i];
      dh[i] = pd[S][i];
      float xh[8], g[8];
      terms(i, xh, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) aw[i][e] += g[e] * xh[e];
      weigh(i, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) a += g[e] * xh[e];
    }
    if (AHEAD) fetch(slot_c, r + DEEP * step);
    a = block_sum<WAVE>(a, red[flip]) / p.n;
    flip ^= 1;
    T* dx = row_ptr<T>(p.dx, r);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float xh[8], g[8];
      terms(i, xh, g);
      weigh(i, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = rs * (g[e] - xh[e] * a);
      if (p.dh.p) {
        dh[i].unpack(xh);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] += xh[e];
      }
      Chunk<T> o;
      o.pack(g);
      o.store(dx, (i * NT + tid) * 8, p.cols);
    }
    r += step;
  };
  using S0 = std::integral_constant<int, 0>;
  using S1 = std::integral_constant<int, DEEP - 1>;
  if (AHEAD) {
    fetch(S0{}, r);
    if (DEEP > 1) fetch(S1{}, r + step);
  }
  while (r < p.rows) {
    if (!AHEAD) fetch(S0{}, r);
    row(S0{});
    if (DEEP > 1 && r < p.rows) row(S1{});
  }
  if (!p.part) return;
  if constexpr (RPW > 1) {   // the four waves' sums meet in the first, in order
    __shared__ float sum[RPW - 1][64 * VPT * 8];
    if (sub) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[sub - 1][(i * 8 + e) * 64 + tid] = aw[i][e];
    }
    __syncthreads();
    if (sub) return;
    for (int k = 0; k < RPW - 1; ++k)
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) aw[i][e] += sum[k][(i * 8 + e) * 64 + tid];
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
  __shared__ f32x4 red[4];
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
  a = block_sum<false>(a, red) / p.n;
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

// dw from the parts: 32 columns a workgroup, whose 32 half waves each take every 32nd part, eight at a time: 5.6 us for
// 2047 columns of 1280 parts.
template <typename WT>
__global__ void __launch_bounds__(1024) rms_dw_sum(const RmsArgs p) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, half = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float a = 0.f;
  if (c < p.cols) {
    const float* part = p.part + c;
    int i = half;
    for (; i + 7 * 32 < p.nparts; i += 8 * 32) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = part[(int64_t)(i + 32 * u) * p.cols];
#pragma unroll
      for (int u = 0; u < 8; ++u) a += v[u];
    }
    for (; i < p.nparts; i += 32) a += part[(int64_t)i * p.cols];
  }
  red[half][lane] = a;
  __syncthreads();
  if (half == 0 && c < p.cols) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += red[i][lane];
    reinterpret_cast<WT*>(p.dw)[c] = from_f32<WT>(s);
  }
}

}  // namespace mns
