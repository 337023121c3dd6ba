// Eight consecutive elements of a row (bf16 or fp32) at a time, shared by the kernels that
// stream rows.
#pragma once

#include "common.h"

namespace th {

// Eight elements, 16 bytes at a time, aligned like an element only: the memory system
// takes such accesses at any of their addresses, so that odd widths and pitches need no
// code of their own but for a row's last elements (65536 rows of 4095 in bf16: 329 us;
// element by element 587).
typedef u32x4_t bf16_row_t __attribute__((aligned(2)));
typedef f32x4_t f32_row_t __attribute__((aligned(4)));

struct Row8 {
  float v[8];
};

__device__ __forceinline__ Row8 load8(const unsigned short* p) {
  const u32x4_t u = *(const bf16_row_t*)p;
  Row8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = __uint_as_float(u[i] << 16);
    r.v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
  return r;
}
__device__ __forceinline__ Row8 load8(const float* p) {
  const f32x4_t a = *(const f32_row_t*)p, b = *(const f32_row_t*)(p + 4);
  return Row8{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
}
__device__ __forceinline__ void store8(unsigned short* p, const Row8& r) {
  u32x4_t u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    u[i] = (unsigned)f32_to_bf16_rne(r.v[2 * i]) | ((unsigned)f32_to_bf16_rne(r.v[2 * i + 1]) << 16);
  *(bf16_row_t*)p = u;
}
__device__ __forceinline__ void store8(float* p, const Row8& r) {
  *(f32_row_t*)p = f32x4_t{r.v[0], r.v[1], r.v[2], r.v[3]};
  *(f32_row_t*)(p + 4) = f32x4_t{r.v[4], r.v[5], r.v[6], r.v[7]};
}
__device__ __forceinline__ float load1(const unsigned short* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(unsigned short* p, float v) { *p = f32_to_bf16_rne(v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

// Elements q .. q+7 of a row of b: with a TAIL (b is no multiple of 8) those past its end
// are 0, and not stored.
template <bool TAIL, class T>
__device__ __forceinline__ Row8 row_load(const T* row, int64_t q, int64_t b) {
  if (!TAIL || q + 8 <= b) return load8(row + q);
  Row8 r;
#pragma unroll
  for (int e = 0; e < 8; ++e) r.v[e] = q + e < b ? load1(row + q + e) : 0.f;
  return r;
}
template <bool TAIL, class T>
__device__ __forceinline__ void row_store(T* row, int64_t q, int64_t b, const Row8& r) {
  if (!TAIL || q + 8 <= b) return store8(row + q, r);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (q + e < b) store1(row + q + e, r.v[e]);
}

}  // namespace th
