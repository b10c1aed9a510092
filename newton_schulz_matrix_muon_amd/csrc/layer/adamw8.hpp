// AdamW whose moments are held in 8 bits (mx8.hpp): m, and r = sqrt(v), whose range is half of v's in
// powers of two, each as codes and one power of two per 32 elements of the flat tensor.
//
//   m <- beta1 m + (1 - beta1) g;  r <- sqrt(beta2 r^2 + (1 - beta2) g^2);
//   p <- (1 - lr wd) p - lr m^ / (r^ + eps)
//
// The update takes m and r in fp32, before they are rounded to their codes. They are rounded up or
// down at random, in proportion, so that a moment's mean is right: with the nearest code a change
// below half a code's step is lost every time, and a step of e4m3 is 6 to 12 % where g = 0 moves r
// by (1 - beta2) / 2, so moments that should decay would stand still. A root that is not zero keeps
// the smallest code at least, so that an element that has seen a gradient never divides by eps
// alone; m / r stays within its block's range.
//
// Bound by HBM: 3 elements, 4 bytes of codes and an eighth of a byte of powers per parameter (10.1 bytes
// in bf16, 22 with moments in fp32) and, in 16 bits, as much by its arithmetic. One MI355X: 20480 x 7168 and eight
// 384 x 7168 (169 M) 324 to 329 us in bf16 at 5.2 TB/s, 498 in fp32 at 5.5; 122 tensors of 7168 in three launches of 6 to 8 us.
// With each code rounded on its own bits and a full-precision quotient it was 425 in bf16.
#pragma once

#include "../adamw.hpp"
#include "mx8.hpp"

namespace mns {

constexpr int ADAM8_MAXT = 48;                // tensors per launch (kernel-argument table)
constexpr int ADAM8_BLOCK = 256;
constexpr int ADAM8_CHUNK = ADAM8_BLOCK * 8;  // elements per workgroup (16 a thread: 169 M in bf16 337 us)

struct Adam8Table {
  void* p[ADAM8_MAXT];
  const void* g[ADAM8_MAXT];
  uint8_t* m[ADAM8_MAXT];
  uint8_t* ms[ADAM8_MAXT];
  uint8_t* r[ADAM8_MAXT];
  uint8_t* rs[ADAM8_MAXT];
  int64_t numel[ADAM8_MAXT];
  int blk_start[ADAM8_MAXT + 1];              // first workgroup of each tensor
  uint32_t key[ADAM8_MAXT];                   // of the tensor's random numbers; its place in the list where the step lies on the device
  int nt;
  float lr, beta1, beta2, eps, wd_mul;        // wd_mul = 1 - lr * weight_decay
  float one_beta1, one_beta2;                 // 1 - beta1, 1 - beta2, rounded once
  float bc1, bc2;                             // bias correction of m and of r (1 when off)
  // the step on the device (DEV): read when the kernel runs, so that a captured call's replays go on counting
  const int64_t* step;
  uint32_t seed;                              // adam8_seed
  int correct;                                // bias corrections of the step read
  double wide1, wide2;                        // beta1, beta2 for them
};

// Random bits: a number's bits mixed, which the tensor's key and an element's place go through.
constexpr uint32_t ADAM8_MIX0 = 0xdf50e7c3u, ADAM8_MIX1 = 0x3dd219bfu, ADAM8_MIX2 = 0xafd7c8e5u;
__host__ __device__ inline uint32_t adam8_mix(uint32_t x) {
  x ^= x >> 16;
  x *= ADAM8_MIX1;
  x ^= x >> 15;
  x *= ADAM8_MIX2;
  return x ^ (x >> 16);
}
__host__ __device__ inline uint32_t adam8_seed(uint64_t seed) { return adam8_mix(adam8_mix((uint32_t)seed) ^ (uint32_t)(seed >> 32)); }
__host__ __device__ inline uint32_t adam8_key(uint32_t seed, uint32_t step, uint32_t place) { return adam8_mix(adam8_mix(seed ^ step) ^ place); }
// 1 / (1 - beta^step), the power by squaring: the same bits from the host and from the kernel.
__host__ __device__ inline double adam8_correction(double beta, uint32_t step) {
#pragma clang fp contract(off)
  double power = 1.0;
  for (; step; step >>= 1, beta *= beta)
    if (step & 1) power *= beta;
  return 1.0 / (1.0 - power);
}
// Elements i .. i + 7 (i a multiple of 8): 16 bits for m (low) and 16 for r (high) each.
__device__ inline void adam8_bits(uint32_t key, int64_t i, uint32_t (&rnd)[8]) {
  if (i >> 32) key = adam8_mix(key ^ (uint32_t)(i >> 32));
  const uint32_t x = (uint32_t)i * ADAM8_MIX0 + key;
#pragma unroll
  for (uint32_t e = 0; e < 8; ++e) rnd[e] = adam8_mix(x + e * ADAM8_MIX0);
}

// A magnitude of at most 448 to a multiple of e4m3's step below or above it, above by the chance
// that rnd / 2^16 is under the rest. fp32 keeps 20 bits more than e4m3, which rnd is added to and which are
// then cut off; below 2^-6 the step is 2^-9 throughout, as it is for x + 2^-6.
__device__ inline float adam8_round(float x, uint32_t rnd) {
  const float low = x < 0x1p-6f ? 0x1p-6f : 0.f;
  return __uint_as_float((__float_as_uint(x + low) + (rnd << 4)) & 0xfff00000u) - low;
}

// Eight elements' new states as codes with their block's byte: adam8_round of the scaled magnitudes.
template <bool ROOT>
__device__ inline u32x2 adam8_codes(const float (&v)[8], const uint32_t (&rnd)[8], int* byte) {
  float q[8];
  bool odd;
  *byte = mx_byte(quad_max(mx_top(v, &odd)));
  const float d = mx_divisor(*byte);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float a = __builtin_fabsf(v[e]);
    float s = adam8_round(a * d, ROOT ? rnd[e] >> 16 : rnd[e] & 0xffffu);
    if (ROOT) s = fmaxf(s, a > 0.f ? 0x1p-9f : 0.f);
    q[e] = ROOT ? s : __builtin_copysignf(s, v[e]);
  }
  return mx_codes(v, q, odd);
}

// A moment's sum: every operation rounded and none contracted, and the root to half a step, so that the states of parameters
// of any type follow the formula in fp32 bit for bit. A last bit that differs moves one in some million roundings to the
// next code. The root is one correction of an estimate to an ulp, and right for every non-negative float (all 2^31 compared); small
// numbers are moved up by 2^64 first, which keeps the correction's rest exact. 169 M in bf16 328 us; 314 with
// contracted sums and a root to an ulp.
__device__ inline float adam8_sum(float a, float x, float b, float y) {
#pragma clang fp contract(off)
  return a * x + b * y;
}
__device__ inline float adam8_sqrt(float v) {
  const bool small = v < 0x1p-64f;
  const float x = v * (small ? 0x1p64f : 1.f);
  const float y = __builtin_amdgcn_rsqf(x), root = x * y;
  const float s = __builtin_fmaf(__builtin_fmaf(-root, root, x), 0.5f * y, root) * (small ? 0x1p-32f : 1.f);
  return __builtin_amdgcn_classf(v, 0x180) ? s : v;   // positive and finite; 0, infinity and NaN are their own roots
}

__device__ inline u32x2 adam8_load(const uint8_t* p, int64_t i, int64_t n) {
  if (i + 8 <= n) return *reinterpret_cast<const u32x2_any*>(p + i);
  u32x2 v = {0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (i + e < n) v[e >> 2] |= (uint32_t)p[i + e] << (8 * (e & 3));
  return v;
}
__device__ inline void adam8_store(uint8_t* p, int64_t i, int64_t n, const u32x2& v) {
  if (i + 8 <= n) {
    *reinterpret_cast<u32x2_any*>(p + i) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (i + e < n) p[i + e] = (uint8_t)(v[e >> 2] >> (8 * (e & 3)));
  }
}

// Eight elements at any element's address.
template <typename T>
struct Adam8Vec {
  static constexpr int N = 16 / (int)sizeof(T), L = 8 / N;
  u32x4 v[L];
  __device__ inline void load(const T* p, int64_t i, int64_t n) {
    if (i + 8 <= n) {
#pragma unroll
      for (int l = 0; l < L; ++l) v[l] = *reinterpret_cast<const u32x4_any*>(p + i + l * N);
    } else {
      typedef T TN __attribute__((ext_vector_type(N)));
#pragma unroll
      for (int l = 0; l < L; ++l) {
        TN s;
#pragma unroll
        for (int e = 0; e < N; ++e) s[e] = i + l * N + e < n ? p[i + l * N + e] : (T)0.f;
        v[l] = __builtin_bit_cast(u32x4, s);
      }
    }
  }
  __device__ inline void unpack(float (&f)[8]) const {
    if constexpr (L == 1) VecIO<T>::unpack(v[0], f);
    else
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(v[e >> 2][e & 3]);
  }
  static __device__ inline void store(T* p, int64_t i, int64_t n, const float (&f)[8]) {
    if (i + 8 <= n) {
      if constexpr (L == 1) {
        *reinterpret_cast<u32x4_any*>(p + i) = u32x4{pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7])};
      } else {
#pragma unroll
        for (int l = 0; l < 2; ++l)
          *reinterpret_cast<u32x4_any*>(p + i + 4 * l) =
              u32x4{__float_as_uint(f[4 * l]), __float_as_uint(f[4 * l + 1]), __float_as_uint(f[4 * l + 2]), __float_as_uint(f[4 * l + 3])};
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (i + e < n) p[i + e] = from_f32<T>(f[e]);
    }
  }
};

// DEV: the step, and with it the random numbers and the bias corrections, comes from the device's memory.
template <typename T, bool DEV>
__global__ void __launch_bounds__(ADAM8_BLOCK) adamw8_kernel(const Adam8Table t) {
  int ti = 0;
  while (ti + 1 < t.nt && (int)blockIdx.x >= t.blk_start[ti + 1]) ++ti;
  const int64_t n = t.numel[ti];
  const int64_t base = (int64_t)((int)blockIdx.x - t.blk_start[ti]) * ADAM8_CHUNK;
  T* p = reinterpret_cast<T*>(t.p[ti]);
  const T* g = reinterpret_cast<const T*>(t.g[ti]);
  uint8_t* m = t.m[ti];
  uint8_t* r = t.r[ti];
  // all loads of the thread first, then the arithmetic
  const int64_t i = base + (int64_t)threadIdx.x * 8;
  const bool in = i < n;
  Adam8Vec<T> pv, gv;
  u32x2 mc, rc;
  int mb, rb;
  if (in) {
    pv.load(p, i, n);
    gv.load(g, i, n);
    mc = adam8_load(m, i, n);
    rc = adam8_load(r, i, n);
    mb = t.ms[ti][i / MX_BLOCK];
    rb = t.rs[ti][i / MX_BLOCK];
  }
  uint32_t key = t.key[ti];
  float bc1 = t.bc1, bc2 = t.bc2;
  if constexpr (DEV) {
    const uint32_t step = (uint32_t)max((int64_t)1, min(*t.step, (int64_t)0x7fffffff));
    key = adam8_key(t.seed, step, key);
    if (t.correct) {                          // one wave works them out
      __shared__ float fix[2];
      if (threadIdx.x < 64) {
        const double c1 = adam8_correction(t.wide1, step), c2 = __builtin_sqrt(adam8_correction(t.wide2, step));
        if (threadIdx.x == 0) {
          fix[0] = (float)c1;
          fix[1] = (float)c2;
        }
      }
      __syncthreads();
      bc1 = fix[0];
      bc2 = fix[1];
    }
  }
  float pf[8], mf[8], rf[8];
  uint32_t rnd[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) pf[e] = mf[e] = rf[e] = 0.f;
  if (in) {
    float gf[8];
    pv.unpack(pf);
    gv.unpack(gf);
    mx_values(mc, mx_factor(mb), mf);
    mx_values(rc, mx_factor(rb), rf);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      mf[e] = adam8_sum(t.beta1, mf[e], t.one_beta1, gf[e]);
      rf[e] = adam8_sqrt(adam8_sum(t.beta2, rf[e] * rf[e], t.one_beta2, gf[e] * gf[e]));
      // the reciprocal to 1 ulp: its error in p is 2^-23 of the step
      pf[e] = t.wd_mul * pf[e] - t.lr * ((mf[e] * bc1) * __builtin_amdgcn_rcpf(rf[e] * bc2 + t.eps));
    }
  }
  adam8_bits(key, i, rnd);
  if (i + 8 > n) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (i + e >= n) mf[e] = rf[e] = 0.f;   // behind the end nothing counts for the block
  }
  // the quads' lanes meet here, those behind the end with zeros
  int bm, br;
  const u32x2 cm = adam8_codes<false>(mf, rnd, &bm), cr = adam8_codes<true>(rf, rnd, &br);
  if (!in) return;
  Adam8Vec<T>::store(p, i, n, pf);
  adam8_store(m, i, n, cm);
  adam8_store(r, i, n, cr);
  if (i % MX_BLOCK == 0) {
    t.ms[ti][i / MX_BLOCK] = (uint8_t)bm;
    t.rs[ti][i / MX_BLOCK] = (uint8_t)br;
  }
}

}  // namespace mns
