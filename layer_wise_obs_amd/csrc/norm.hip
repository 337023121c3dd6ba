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
//
// With the addition of the residual before it, h = x + r rounded to the stream's type, and an
// output that may be microscaled (mx.h), what a product of 8- or 4-bit operands reads: the
// second kernel. There sums, root and products are in 64 bits, so that y is rounded once, from
// a value off by (b / (2 T) + 20) 2^-53 of itself at most, T lanes to a row (64 up to 2048 columns, else
// 256: 2^-48.2 at 4096, 2^-46.7 at 28672): where it lies next to a border between two
// elements, or the block's largest next to one between two scales, fp32's error of 2^-23
// decides for a step of 2^-4. Five 64-bit operations an element against 7 bytes are more than the
// vector units have time for, so only the sum is in 64 bits everywhere; a wave's products are in
// fp32, and again in 64 bits where one of them lies within 4 units of fp32 of a border. 65536 rows
// of 4096 with the residual, bf16 to 8 bits: 532 -> 345-359 us by card (5.3 TB/s; a copy of 4 GiB
// 4.7-4.9); 7 rows of 4096 from fp32 4.5, of which a launch is 2.3 and the 64-bit sum's way over the
// lanes 1 (rms_norm: 3.5).
#include "common.h"
#include "mx.h"
#include "row8.h"

namespace th {

namespace {

constexpr int kNChunks = 4;  // register-held chunks of 8 elements per thread

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

// ---------------------------------------------------------------- residual and norm

template <int W>
__device__ __forceinline__ double row_sum(double s, double* red) {
#pragma unroll
  for (int m = 32; m; m >>= 1) s += __shfl_xor(s, m);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    s = 0.0;
#pragma unroll
    for (int w = 0; w < W; ++w) s += red[w];
  }
  return s;
}

// fp64 to fp32, rounded to odd: where bits are lost, towards zero with the last bit set. A
// rounding of the result to fewer bits, or its comparison with a number of fewer bits, is then
// that of the value itself.
__device__ __forceinline__ float to_odd(double y) {
  const float f = (float)y;
  const double t = (double)f;
  unsigned u = __float_as_uint(f);
  if (t != y) u = (u - (fabs(t) > fabs(y) ? 1u : 0u)) | 1u;
  return __uint_as_float(u);
}

// Eight elements of the residual stream as they are held.
template <class T>
struct Held;
template <>
struct Held<unsigned short> {
  u32x4_t u;
  __device__ __forceinline__ float at(int e) const {
    return __uint_as_float(e & 1 ? u[e >> 1] & 0xffff0000u : u[e >> 1] << 16);
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      typedef __bf16 pair_t __attribute__((ext_vector_type(2)));
      u[i] = __builtin_bit_cast(unsigned, pair_t{(__bf16)v[2 * i], (__bf16)v[2 * i + 1]});
    }
  }
  template <bool TAIL>
  __device__ __forceinline__ void load(const unsigned short* p, int64_t q, int64_t b) {
    if (!TAIL || q + 8 <= b) {
      u = *(const bf16_row_t*)(p + q);
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      u[i] = (q + 2 * i < b ? p[q + 2 * i] : 0u) | (q + 2 * i + 1 < b ? (unsigned)p[q + 2 * i + 1] << 16 : 0u);
  }
  template <bool TAIL>
  __device__ __forceinline__ void store(unsigned short* p, int64_t q, int64_t b) const {
    if (!TAIL || q + 8 <= b) {
      *(bf16_row_t*)(p + q) = u;
      return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (q + e < b) p[q + e] = (unsigned short)(u[e >> 1] >> (16 * (e & 1)));
  }
};
template <>
struct Held<float> {
  Row8 r;
  __device__ __forceinline__ float at(int e) const { return r.v[e]; }
  __device__ __forceinline__ void set(const float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) r.v[e] = v[e];
  }
  template <bool TAIL>
  __device__ __forceinline__ void load(const float* p, int64_t q, int64_t b) {
    r = row_load<TAIL>(p, q, b);
  }
  template <bool TAIL>
  __device__ __forceinline__ void store(float* p, int64_t q, int64_t b) const {
    row_store<TAIL>(p, q, b, r);
  }
};

struct NormOut {  // Y, or the elements and scales of a microscaled one
  void* y;
  unsigned char* scales;
  int64_t ldy, lds;  // Y: elements; microscaled: bytes
};

// OUT: -1 bf16, -2 fp32, else a th_mx_type. W waves to a row of b elements.
template <class TI, int OUT, int W, bool TAIL>
__global__ __launch_bounds__(256) void add_rms_norm_kernel(const TI* X, int64_t ldx, const TI* R,
                                                           int64_t ldr, const TI* w, TI* S, int64_t ldsum,
                                                           NormOut out, int64_t n, int64_t b, double eps) {
  constexpr int kRows = 4 / W, T = 64 * W;
  __shared__ double red[4];
  const int64_t row = (int64_t)blockIdx.x * kRows + (W == 1 ? threadIdx.x / 64 : 0);
  if (row >= n) return;
  const int t = threadIdx.x % T;
  const TI* x = X + row * ldx;
  const TI* r = R ? R + row * ldr : nullptr;
  TI* sum = S ? S + row * ldsum : nullptr;
  typedef Held<TI> H;
  // the sum in the stream's type
  auto added = [&](const H& h, const H& a) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = h.at(e) + a.at(e);
    H z;
    z.set(v);
    return z;
  };
  auto stream = [&](int64_t q) {
    H h;
    h.template load<TAIL>(x, q, b);
    if (r) {
      H a;
      a.template load<TAIL>(r, q, b);
      h = added(h, a);
    }
    return h;
  };
  double s = 0.0;
  auto add = [&](const H& h) {
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fma((double)h.at(e), (double)h.at(e), s);
  };
  H kept[kNChunks];
  if (r) {  // all loads on their way before the first sum
    H other[kNChunks];
#pragma unroll
    for (int i = 0; i < kNChunks; ++i) {
      const int64_t q = ((int64_t)i * T + t) * 8;
      if (q < b) {
        kept[i].template load<TAIL>(x, q, b);
        other[i].template load<TAIL>(r, q, b);
      }
    }
#pragma unroll
    for (int i = 0; i < kNChunks; ++i) {
      const int64_t q = ((int64_t)i * T + t) * 8;
      if (q < b) {
        kept[i] = added(kept[i], other[i]);
        if (sum) kept[i].template store<TAIL>(sum, q, b);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kNChunks; ++i) {
      const int64_t q = ((int64_t)i * T + t) * 8;
      if (q < b) kept[i].template load<TAIL>(x, q, b);
    }
  }
#pragma unroll
  for (int i = 0; i < kNChunks; ++i)
    if (((int64_t)i * T + t) * 8 < b) add(kept[i]);
  // columns past the register-held part: formed and added here, read again for the product
  // (from the sum, which may have taken the place of x or r)
  for (int64_t q = ((int64_t)kNChunks * T + t) * 8; q < b; q += T * 8) {
    const H h = stream(q);
    add(h);
    if (sum) h.template store<TAIL>(sum, q, b);
  }
  const double scale = 1.0 / sqrt(row_sum<W>(s, red) / (double)b + eps);
  // The products in fp32 are off by less than four units of their last place. Only where one
  // lies that near to a place where roundings to the output's type meet, or scales do (its last
  // 16 bits tell: 1 in 7000), does fp64 have to decide: the wave then forms its eight again. So it
  // does where an element over the root is no normal number, or 0, beside a weight above 4: the places
  // that are lost, 2^-150, would then count (weights up to 4 keep them below 4 units of any result).
  const float near = (float)scale;
  const bool far = !(near > 0x1p-100f && near < 0x1p100f);
  auto put = [&](const H& h, int64_t q) {
    H g;
    g.template load<TAIL>(w, q, b);
    Row8 v;
    if constexpr (OUT == -2) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v.v[e] = (float)((double)h.at(e) * scale * (double)g.at(e));
      row_store<TAIL>((float*)out.y + row * out.ldy, q, b, v);
      return;
    }
    unsigned least = 0xffffffffu;
    float small = 1.0f, large = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = h.at(e) * near;
      small = fminf(small, fabsf(x));
      large = fmaxf(large, fabsf(g.at(e)));
      v.v[e] = x * g.at(e);
      least = min(least, (__float_as_uint(v.v[e]) + (OUT == -1 ? 0x8004u : 4u)) << 16);
    }
    if (__any(least <= 8u << 16 || (small < 0x1p-126f && large > 4.0f) || far)) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v.v[e] = to_odd((double)h.at(e) * scale * (double)g.at(e));
    }
    if constexpr (OUT == -1) {
      Held<unsigned short> y;
      y.set(v.v);
      y.template store<TAIL>((unsigned short*)out.y + row * out.ldy, q, b);
    } else if constexpr (OUT >= 0) {
      mx_put8<OUT>(v.v, (unsigned char*)out.y + row * out.ldy, out.scales + row * out.lds, q);
    }
  };
#pragma unroll
  for (int i = 0; i < kNChunks; ++i) {
    const int64_t q = ((int64_t)i * T + t) * 8;
    if (q < b) put(kept[i], q);
  }
  for (int64_t q = ((int64_t)kNChunks * T + t) * 8; q < b; q += T * 8) {
    H h;
    if (sum)
      h.template load<TAIL>(sum, q, b);
    else
      h = stream(q);
    put(h, q);
  }
}

template <class TI, int OUT, int W, bool TAIL>
hipError_t launch_add_rows(const TI* x, int64_t ldx, const TI* r, int64_t ldr, const TI* w, TI* sum,
                           int64_t ldsum, NormOut o, int64_t n, int64_t b, double eps, hipStream_t s) {
  constexpr int64_t kMost = kMaxGroups * (4 / W);
  const int64_t unit = OUT == -1 ? 2 : (OUT == -2 ? 4 : 1);
  for (; n > 0; n -= kMost) {
    const int64_t m = n < kMost ? n : kMost;
    hipLaunchKernelGGL((add_rms_norm_kernel<TI, OUT, W, TAIL>), dim3((unsigned)cdiv(m, 4 / W)),
                       dim3(256), 0, s, x, ldx, r, ldr, w, sum, ldsum, o, m, b, eps);
    x += kMost * ldx;
    if (r) r += kMost * ldr;
    if (sum) sum += kMost * ldsum;
    o.y = (char*)o.y + kMost * o.ldy * unit;
    if (o.scales) o.scales += kMost * o.lds;
  }
  return hipGetLastError();
}

template <class TI, int OUT>
hipError_t launch_add_typed(const void* X, int64_t ldx, const void* R, int64_t ldr, const void* w,
                            void* sum, int64_t ldsum, const NormOut& o, int64_t n, int64_t b,
                            double eps, hipStream_t s) {
  const TI *x = (const TI*)X, *r = (const TI*)R, *g = (const TI*)w;
  TI* h = (TI*)sum;
  // a wave to a row up to what its registers hold
  const bool one = b <= 64 * 8 * kNChunks;
  if constexpr (OUT < 0) {
    if (b % 8)
      return one ? launch_add_rows<TI, OUT, 1, true>(x, ldx, r, ldr, g, h, ldsum, o, n, b, eps, s)
                 : launch_add_rows<TI, OUT, 4, true>(x, ldx, r, ldr, g, h, ldsum, o, n, b, eps, s);
  }
  return one ? launch_add_rows<TI, OUT, 1, false>(x, ldx, r, ldr, g, h, ldsum, o, n, b, eps, s)
             : launch_add_rows<TI, OUT, 4, false>(x, ldx, r, ldr, g, h, ldsum, o, n, b, eps, s);
}

template <class TI>
hipError_t launch_add_out(const void* X, int64_t ldx, const void* R, int64_t ldr, const void* w,
                          void* sum, int64_t ldsum, void* Y, th_dtype ydt, int64_t ldy, const th_mx* m,
                          int64_t n, int64_t b, double eps, hipStream_t s) {
  if (m) {
    const NormOut o = {m->elements, (unsigned char*)m->scales, m->ld, m->lds};
    return m->type == TH_MX_E4M3
               ? launch_add_typed<TI, TH_MX_E4M3>(X, ldx, R, ldr, w, sum, ldsum, o, n, b, eps, s)
               : launch_add_typed<TI, TH_MX_E2M1>(X, ldx, R, ldr, w, sum, ldsum, o, n, b, eps, s);
  }
  const NormOut o = {Y, nullptr, ldy, 0};
  return ydt == TH_BF16 ? launch_add_typed<TI, -1>(X, ldx, R, ldr, w, sum, ldsum, o, n, b, eps, s)
                        : launch_add_typed<TI, -2>(X, ldx, R, ldr, w, sum, ldsum, o, n, b, eps, s);
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

hipError_t launch_add_rms_norm(const void* X, th_dtype xdt, int64_t ldx, const void* R, int64_t ldr,
                               const void* w, void* sum, int64_t ldsum, void* Y, th_dtype ydt,
                               int64_t ldy, const th_mx* m, int64_t n, int64_t b, double eps,
                               hipStream_t s) {
  return xdt == TH_BF16 ? launch_add_out<unsigned short>(X, ldx, R, ldr, w, sum, ldsum, Y, ydt, ldy, m,
                                                         n, b, eps, s)
                        : launch_add_out<float>(X, ldx, R, ldr, w, sum, ldsum, Y, ydt, ldy, m, n, b,
                                                eps, s);
}

}  // namespace th
