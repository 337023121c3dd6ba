// Microscaled matrices: 32 consecutive elements of a row share a power of two. An element is
// e4m3 (8 bits, up to 448) or e2m1 (4 bits, up to 6), the power 2^(scale - 127) a byte (255:
// none of the block's values is a number).
#pragma once

#include "common.h"

namespace th {

constexpr int kMxBlock = 32;

template <int TYPE>
struct MxForm;
// kTop: exponent of the largest number's binade. kCarry: added to the bits of an fp32 number it
// carries into the exponent where the number, at this binade, would be rounded to the first one
// past the largest: above 464 = 1.8125 * 256 (464 itself goes to the even 448); from 7 = 1.75 * 4
// (which goes to the even 8) on.
template <>
struct MxForm<TH_MX_E4M3> {
  static constexpr int kBits = 8, kTop = 8;
  static constexpr unsigned kCarry = 0x17ffffu;
  static constexpr float kMost = 448.0f;
};
template <>
struct MxForm<TH_MX_E2M1> {
  static constexpr int kBits = 4, kTop = 2;
  static constexpr unsigned kCarry = 0x200000u;
  static constexpr float kMost = 6.0f;
};

typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// Scale byte of a block from the largest |x| of it (its bits): the smallest power at which no
// element, rounded to the nearest, passes the largest number; at the ends of the byte's range
// numbers become 0 or the largest.
template <int TYPE>
__device__ __forceinline__ unsigned mx_scale_of(unsigned top) {
  if (top >= 0x7f800000u) return 255u;
  const int e = (int)((top + MxForm<TYPE>::kCarry) >> 23) - MxForm<TYPE>::kTop;
  return (unsigned)min(max(e, 0), 254 - MxForm<TYPE>::kTop);
}

// 2^(127 - scale), and 0 for 255: what the block is multiplied by, exact for every scale above.
__device__ __forceinline__ float mx_inverse(unsigned scale) {
  return scale == 255u ? 0.f : __uint_as_float((254u - scale) << 23);
}
// 2^(scale - 127), NaN for 255.
__device__ __forceinline__ float mx_power(unsigned scale) {
  return __uint_as_float(scale == 255u ? 0x7fc00000u : (scale ? scale << 23 : 0x400000u));
}

// Eight scaled values as elements, rounded to nearest even by the conversion instructions. Past
// the largest number there are only what rounds to it and what the byte's range saturates.
__device__ __forceinline__ float mx_clamp(float x, float most) {
  return __builtin_amdgcn_fmed3f(x, -most, most);
}
__device__ __forceinline__ u32x2_t mx_encode8(const float (&v)[8], float inv,
                                              std::integral_constant<int, TH_MX_E4M3>) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = inv == 0.f ? 0.f : mx_clamp(v[i] * inv, 448.0f);
  u32x2_t r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i], x[4 * i + 1], 0, false);
    r[i] = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(x[4 * i + 2], x[4 * i + 3], w, true);
  }
  return r;
}
__device__ __forceinline__ unsigned mx_encode8(const float (&v)[8], float inv,
                                               std::integral_constant<int, TH_MX_E2M1>) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = inv == 0.f ? 0.f : mx_clamp(v[i] * inv, 6.0f);
  unsigned r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x[0], x[1], 1.0f, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x[2], x[3], 1.0f, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x[4], x[5], 1.0f, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x[6], x[7], 1.0f, 3);
  return r;
}

// Eight elements as numbers, before their scale.
__device__ __forceinline__ void mx_decode8(u32x2_t u, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)u[i], false);
    const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)u[i], true);
    v[4 * i] = lo[0];
    v[4 * i + 1] = lo[1];
    v[4 * i + 2] = hi[0];
    v[4 * i + 3] = hi[1];
  }
}
__device__ __forceinline__ void mx_decode8(unsigned u, float (&v)[8]) {
  f32x2_t p;
  p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, 1.0f, 0);
  v[0] = p[0], v[1] = p[1];
  p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, 1.0f, 1);
  v[2] = p[0], v[3] = p[1];
  p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, 1.0f, 2);
  v[4] = p[0], v[5] = p[1];
  p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u, 1.0f, 3);
  v[6] = p[0], v[7] = p[1];
}

// Eight elements in memory, of any alignment.
template <int TYPE>
struct MxWord {
  typedef u32x2_t value;
  typedef u32x2_t memory __attribute__((aligned(1)));
};
template <>
struct MxWord<TH_MX_E2M1> {
  typedef unsigned value;
  typedef unsigned memory __attribute__((aligned(1)));
};

// The eight elements from q of a row (q a multiple of 8) and, by the first lane of the four
// that share it, their block's scale. All four lanes call it together.
template <int TYPE>
__device__ __forceinline__ void mx_put8(const float (&v)[8], unsigned char* elements,
                                        unsigned char* scales, int64_t q) {
  unsigned top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  top = max(top, (unsigned)__shfl_xor((int)top, 1));
  top = max(top, (unsigned)__shfl_xor((int)top, 2));
  const unsigned scale = mx_scale_of<TYPE>(top);
  typedef MxWord<TYPE> Word;
  *(typename Word::memory*)(elements + q * MxForm<TYPE>::kBits / 8) =
      mx_encode8(v, mx_inverse(scale), std::integral_constant<int, TYPE>{});
  if (q % kMxBlock == 0) scales[q / kMxBlock] = (unsigned char)scale;
}

}  // namespace th
