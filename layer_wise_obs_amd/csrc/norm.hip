// Root-mean-square norm of the rows of an activation matrix,
//   y_tq = x_tq / sqrt(mean_q x_tq^2 + eps) * w_q,
// which stands before the q/k/v and the gate/up projections of a block ("Pruning
// LLMs with Thanos", section "The compression target: linear layers").
//
// Bound by memory: one read and one write of the matrix. A workgroup takes one
// row and keeps it in registers between the sum and the product, so x is read
// once; every lane moves 8 consecutive elements (16 bytes of bf16) at a time. The
// sum of squares is fp32: 8 products per chunk and lane, then lanes, then waves.
// 131072 rows of 4096 in bf16: 354-380 us, 5.7-6.1 TB/s (a copy: 4.9).
#include "common.h"

namespace th {

namespace {

constexpr int kNChunks = 4;  // register-held chunks of 8 elements per thread

struct Row8 {
  float v[8];
};

__device__ __forceinline__ Row8 load8(const unsigned short* p) {
  const u32x4_t u = *(const u32x4_t*)p;
  Row8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = __uint_as_float(u[i] << 16);
    r.v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
  return r;
}
__device__ __forceinline__ Row8 load8(const float* p) {
  const f32x4_t a = ((const f32x4_t*)p)[0], b = ((const f32x4_t*)p)[1];
  return Row8{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
}
__device__ __forceinline__ void store8(unsigned short* p, const Row8& r) {
  u32x4_t u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    u[i] = (unsigned)f32_to_bf16_rne(r.v[2 * i]) | ((unsigned)f32_to_bf16_rne(r.v[2 * i + 1]) << 16);
  *(u32x4_t*)p = u;
}
__device__ __forceinline__ void store8(float* p, const Row8& r) {
  ((f32x4_t*)p)[0] = f32x4_t{r.v[0], r.v[1], r.v[2], r.v[3]};
  ((f32x4_t*)p)[1] = f32x4_t{r.v[4], r.v[5], r.v[6], r.v[7]};
}
__device__ __forceinline__ float load1(const unsigned short* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(unsigned short* p, float v) { *p = f32_to_bf16_rne(v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

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

template <class TI, class TO, int T>
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
    if (q < b) kept[i] = load8(x + q);
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
    const Row8 r = load8(x + q);
#pragma unroll
    for (int e = 0; e < 8; ++e) s += r.v[e] * r.v[e];
  }
  const float scale = 1.0f / sqrtf(group_sum<T>(s, red) / (float)b + eps);
  auto put = [&](Row8 r, int64_t q) {
    const Row8 g = load8(w + q);
#pragma unroll
    for (int e = 0; e < 8; ++e) r.v[e] = r.v[e] * scale * g.v[e];
    store8(y + q, r);
  };
#pragma unroll
  for (int i = 0; i < kNChunks; ++i) {
    const int64_t q = ((int64_t)i * T + threadIdx.x) * 8;
    if (q < b) put(kept[i], q);
  }
  for (int64_t q = ((int64_t)kNChunks * T + threadIdx.x) * 8; q < b; q += T * 8) put(load8(x + q), q);
}

// Any width, pitch and alignment: one element per thread and step.
template <class TI, class TO>
__global__ __launch_bounds__(256) void rms_norm_any_kernel(const TI* X, int64_t ldx, const TI* w,
                                                           TO* Y, int64_t ldy, int64_t b,
                                                           float eps) {
  __shared__ float red[4];
  const TI* x = X + (int64_t)blockIdx.x * ldx;
  TO* y = Y + (int64_t)blockIdx.x * ldy;
  float s = 0.f;
  for (int64_t q = threadIdx.x; q < b; q += 256) {
    const float v = load1(x + q);
    s += v * v;
  }
  const float scale = 1.0f / sqrtf(group_sum<256>(s, red) / (float)b + eps);
  for (int64_t q = threadIdx.x; q < b; q += 256) store1(y + q, load1(x + q) * scale * load1(w + q));
}

template <class TI, class TO>
hipError_t launch_typed(const void* X, int64_t ldx, const void* w, void* Y, int64_t ldy, int64_t n,
                        int64_t b, float eps, hipStream_t s) {
  // 16-byte accesses: 8 bf16 or 4 fp32 elements
  const bool vec = b % 8 == 0 && ldx % (16 / sizeof(TI)) == 0 && ldy % (16 / sizeof(TO)) == 0 &&
                   (((uintptr_t)X | (uintptr_t)w | (uintptr_t)Y) & 15) == 0;
  const TI* x = (const TI*)X;
  TO* y = (TO*)Y;
  for (; n > 0; n -= kMaxGroups, x += kMaxGroups * ldx, y += kMaxGroups * ldy) {
    const dim3 grid((unsigned)(n < kMaxGroups ? n : kMaxGroups));
    if (!vec)
      hipLaunchKernelGGL((rms_norm_any_kernel<TI, TO>), grid, dim3(256), 0, s, x, ldx,
                         (const TI*)w, y, ldy, b, eps);
    else if (b <= 1024)
      hipLaunchKernelGGL((rms_norm_kernel<TI, TO, 64>), grid, dim3(64), 0, s, x, ldx, (const TI*)w,
                         y, ldy, b, eps);
    else
      hipLaunchKernelGGL((rms_norm_kernel<TI, TO, 256>), grid, dim3(256), 0, s, x, ldx,
                         (const TI*)w, y, ldy, b, eps);
  }
  return hipGetLastError();
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
