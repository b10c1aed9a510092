// 8-bit values in blocks of 32: e4m3 codes (OCP FP8, largest value 448, smallest 2^-9) and one
// power of two per block, held as the byte of its biased exponent (e8m0). A block's power is the
// smallest that brings its largest finite magnitude to 448 or less, so nothing is cut off; a block
// of zeros has byte 0. Values that are not finite become NaN codes and leave their block's power
// alone.
#pragma once

#include "norm.hpp"

namespace mns {

constexpr int MX_BLOCK = 32;

typedef u32x4 u32x4_any __attribute__((aligned(2)));      // 16 bytes at any element's address
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));

// top: the largest finite magnitude. 448 = 1.75 * 2^8.
__device__ inline int mx_byte(float top) {
  const uint32_t u = __float_as_uint(top);
  return max(0, (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0));
}
// 2^(127 - byte) and 2^(byte - 127); the byte of a block written here is at most 247.
__device__ inline float mx_divisor(int byte) { return __uint_as_float((uint32_t)(254 - byte) << 23); }
__device__ inline float mx_factor(int byte) { return byte ? __uint_as_float((uint32_t)byte << 23) : 0x1p-127f; }

// The largest finite magnitude of eight values, and whether any value of the wave is not finite (rare,
// equal in every lane). Magnitudes compare as their bits do.
__device__ inline float mx_top(const float (&v)[8], bool* odd) {
  constexpr uint32_t INF = 0x7f800000u;
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
  *odd = __any(top >= INF);
  if (*odd) {
    top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t u = __float_as_uint(v[e]) & 0x7fffffffu;
      top = max(top, u < INF ? u : 0u);
    }
  }
  return __uint_as_float(top);
}

// The maximum over the four lanes that hold a block, eight values each.
__device__ inline float quad_max(float v) {
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xb1, 0xf, 0xf, true)));    // lanes 1 0 3 2
  return fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4e, 0xf, 0xf, true)));  // lanes 2 3 0 1
}

// Four values to codes, rounded to nearest even (values of e4m3 stay as they are).
__device__ inline uint32_t mx_pack(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// Eight values as codes, q as scaled and rounded; odd: as mx_top found.
__device__ inline u32x2 mx_codes(const float (&v)[8], float (&q)[8], bool odd) {
  if (odd) {
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = __builtin_fabsf(v[e]) < __builtin_inff() ? q[e] : __builtin_nanf("");
  }
  return u32x2{mx_pack(q[0], q[1], q[2], q[3]), mx_pack(q[4], q[5], q[6], q[7])};
}

__device__ inline void mx_values(const u32x2& codes, float factor, float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes[h], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes[h], true);
    v[4 * h] = a[0] * factor;
    v[4 * h + 1] = a[1] * factor;
    v[4 * h + 2] = b[0] * factor;
    v[4 * h + 3] = b[1] * factor;
  }
}

}  // namespace mns
