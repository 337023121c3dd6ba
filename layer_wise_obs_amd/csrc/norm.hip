// Root-mean-square norm of the rows of an activation matrix,
//   y_tq = x_tq / sqrt(mean_q x_tq^2 + eps) * w_q,
// which stands before the q/k/v and the gate/up projections of a block ("Pruning
// LLMs with Thanos", section "The compression target: linear layers").
//
// Bound by memory: one read and one write of the matrix. A workgroup takes one
// row and keeps it in registers between the sum and the product, so x is read
// once; every lane moves 8 consecutive elements (16 bytes of bf16) at a time. The
// sum of squares is fp32: 8 products per chunk and lane, then lanes, then waves.
// 131072 rows of 4096 in bf16: 358-412 us by box, 5.2-6.0 TB/s (torch's copy: 4.9).
// Rows below 512 elements are bound by launching workgroups: 100000 of 100, 54 us.
#include "common.h"

namespace th {

namespace {

constexpr int kNChunks = 4;  // register-held chunks of 8 elements per thread

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

// Sum over the T threads of a workgroup, the same value in every thread.
template <int T>
__device__ __forceinline__ float group_sum(float s, float* red) {
#pragma unroll
  for (int m = 32; m; m >>= 1) s += __shfl_xor(s, m);
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    s = 0.f;
#pragma unroll
    for (int w = 0; w < T / 64; ++w) s += red[w];
  }
  return s;
}

// 1 / sqrt(v). Root and reciprocal round once each; for fp32 outputs (EXACT) one step of
// Newton's with the product's own rounding makes that half a unit of the result (their
// error against 64 bits: 6.1e-8 -> 5.7e-8 rms at 4096 columns; for bf16 ones, whose
// rounding hides it, it would cost 0.4% of the time).
template <bool EXACT>
__device__ __forceinline__ float inverse_root(float v) {
  const float r = 1.0f / sqrtf(v);
  if constexpr (!EXACT) return r;
  const float h = v * r, rest = fmaf(v, r, -h);
  const float e = fmaf(-h, r, 1.0f) - rest * r;  // 1 - v r^2; NaN for roots of 0 and infinity
  return fabsf(e) < 1.0f ? fmaf(0.5f * r, e, r) : r;
}

template <class TI, class TO, int T, bool TAIL>
__global__ __launch_bounds__(T) void rms_norm_kernel(const TI* X, int64_t ldx, const TI* w, TO* Y,
                                                     int64_t ldy, int64_t b, float eps) {
  __shared__ float red[T / 64];
  const TI* x = X + (int64_t)blockIdx.x * ldx;
  TO* y = Y + (int64_t)blockIdx.x * ldy;
  Row8 kept[kNChunks];
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kNChunks; ++i) {
    const int64_t q = ((int64_t)i * T + threadIdx.x) * 8;
    if (q < b) kept[i] = row_load<TAIL>(x, q, b);
  }
#pragma unroll
  for (int i = 0; i < kNChunks; ++i) {
    if (((int64_t)i * T + threadIdx.x) * 8 < b) {
#pragma unroll
      for (int e = 0; e < 8; ++e) s += kept[i].v[e] * kept[i].v[e];
    }
  }
  // columns past the register-held part are read again for the product
  for (int64_t q = ((int64_t)kNChunks * T + threadIdx.x) * 8; q < b; q += T * 8) {
    const Row8 r = row_load<TAIL>(x, q, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) s += r.v[e] * r.v[e];
  }
  const float mean = group_sum<T>(s, red) / (float)b + eps;
  const float scale = inverse_root<std::is_same<TO, float>::value>(mean);
  auto put = [&](Row8 r, int64_t q) {
    const Row8 g = row_load<TAIL>(w, q, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) r.v[e] = r.v[e] * scale * g.v[e];
    row_store<TAIL>(y, q, b, r);
  };
#pragma unroll
  for (int i = 0; i < kNChunks; ++i) {
    const int64_t q = ((int64_t)i * T + threadIdx.x) * 8;
    if (q < b) put(kept[i], q);
  }
  for (int64_t q = ((int64_t)kNChunks * T + threadIdx.x) * 8; q < b; q += T * 8) put(row_load<TAIL>(x, q, b), q);
}

template <class TI, class TO, int T, bool TAIL>
hipError_t launch_rows(const void* X, int64_t ldx, const void* w, void* Y, int64_t ldy, int64_t n,
                       int64_t b, float eps, hipStream_t s) {
  const TI* x = (const TI*)X;
  TO* y = (TO*)Y;
  for (; n > 0; n -= kMaxGroups, x += kMaxGroups * ldx, y += kMaxGroups * ldy)
    hipLaunchKernelGGL((rms_norm_kernel<TI, TO, T, TAIL>),
                       dim3((unsigned)(n < kMaxGroups ? n : kMaxGroups)), dim3(T), 0, s, x, ldx,
                       (const TI*)w, y, ldy, b, eps);
  return hipGetLastError();
}

template <class TI, class TO>
hipError_t launch_typed(const void* X, int64_t ldx, const void* w, void* Y, int64_t ldy, int64_t n,
                        int64_t b, float eps, hipStream_t s) {
  if (b % 8)  // the whole rows' kernel needs fewer registers: tails cost it 7%
    return b <= 1024 ? launch_rows<TI, TO, 64, true>(X, ldx, w, Y, ldy, n, b, eps, s)
                     : launch_rows<TI, TO, 256, true>(X, ldx, w, Y, ldy, n, b, eps, s);
  return b <= 1024 ? launch_rows<TI, TO, 64, false>(X, ldx, w, Y, ldy, n, b, eps, s)
                   : launch_rows<TI, TO, 256, false>(X, ldx, w, Y, ldy, n, b, eps, s);
}

}  // namespace

hipError_t launch_rms_norm(const void* X, th_dtype xdt, int64_t ldx, const void* w, void* Y,
                           th_dtype ydt, int64_t ldy, int64_t n, int64_t b, float eps,
                           hipStream_t s) {
  typedef unsigned short h;
  if (xdt == TH_BF16)
    return ydt == TH_BF16 ? launch_typed<h, h>(X, ldx, w, Y, ldy, n, b, eps, s)
                          : launch_typed<h, float>(X, ldx, w, Y, ldy, n, b, eps, s);
  return ydt == TH_BF16 ? launch_typed<float, h>(X, ldx, w, Y, ldy, n, b, eps, s)
                        : launch_typed<float, float>(X, ldx, w, Y, ldy, n, b, eps, s);
}

}  // namespace th
