// Microscaled matrices from bf16 or fp32 and back: the form in which the pruned layers of a
// block are served ("Pruning LLMs with Thanos", section "The compression target: linear
// layers"), 4.25 or 8.25 bits a weight; zeros stay zeros.
//
//   E = the smallest exponent at which max |x| / 2^E rounds to a number of the type,
//   element = round to nearest even (x / 2^E),  value = element 2^E.
//
// Scaling by a power of two is exact and the conversion instructions round once, so an
// element is off by at most half a step of its type. (The usual choice, the exponent of the
// largest element's binade, clips up to a quarter of it: over normal weights of 4 bits the
// error is 0.1160 of their root mean square instead of 0.1123, pruned 2:4 0.1118 instead of
// 0.1048; 8 bits 0.0302 and 0.0269.)
//
// Bound by memory. Four lanes share a block, each moves eight elements (16 bytes of bf16, 32
// of fp32); a workgroup's lanes follow the rows one after another. 11008 x 4096 from fp32 to 4
// bits 30-32 us (6.6 TB/s, some of it from the last level cache), to bf16 from 4 bits 21-22; 65536 x
// 4096 of 8 bits to bf16 148-158 (5.3-5.5 TB/s); 5 rows of 11008 2.4 and 2.8, a launch's time.
#include "common.h"
#include "mx.h"
#include "row8.h"

namespace th {

namespace {

// Chunk i of eight elements is in row i / per_row; a launch has less than 2^31 chunks.
template <int TYPE, class T>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const T* X, int64_t ldx, unsigned chunks,
                                                          unsigned per_row, unsigned char* elements,
                                                          int64_t ld, unsigned char* scales,
                                                          int64_t lds) {
  const unsigned i = blockIdx.x * 256 + threadIdx.x;
  if (i >= chunks) return;  // blocks of four lanes end together
  const unsigned row = i / per_row;
  const int64_t q = (int64_t)(i - row * per_row) * 8;
  const Row8 r = load8(X + row * ldx + q);
  mx_put8<TYPE>(r.v, elements + row * ld, scales + row * lds, q);
}

template <int TYPE, class T>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const unsigned char* elements, int64_t ld,
                                                            const unsigned char* scales, int64_t lds,
                                                            unsigned chunks, unsigned per_row, T* Y,
                                                            int64_t ldy) {
  const unsigned i = blockIdx.x * 256 + threadIdx.x;
  if (i >= chunks) return;
  const unsigned row = i / per_row;
  const int64_t q = (int64_t)(i - row * per_row) * 8;
  typedef MxWord<TYPE> Word;
  const typename Word::value u =
      *(const typename Word::memory*)(elements + row * ld + q * MxForm<TYPE>::kBits / 8);
  const float power = mx_power(scales[row * lds + q / kMxBlock]);
  Row8 r;
  mx_decode8(u, r.v);
#pragma unroll
  for (int e = 0; e < 8; ++e) r.v[e] *= power;
  store8(Y + row * ldy + q, r);
}

// Rows of one launch: less than 2^31 chunks.
int64_t rows_at_once(int64_t b) { return (((int64_t)1 << 31) - 256) / (b / 8); }

template <int TYPE, class T>
hipError_t quantize_rows(const T* X, int64_t ldx, int64_t n, int64_t b, const th_mx& y, hipStream_t s) {
  unsigned char *e = (unsigned char*)y.elements, *sc = (unsigned char*)y.scales;
  const int64_t most = rows_at_once(b);
  for (int64_t r = 0; r < n; r += most) {
    const int64_t chunks = (n - r < most ? n - r : most) * (b / 8);
    hipLaunchKernelGGL((mx_quantize_kernel<TYPE, T>), dim3((unsigned)cdiv(chunks, 256)), dim3(256), 0,
                       s, X + r * ldx, ldx, (unsigned)chunks, (unsigned)(b / 8), e + r * y.ld, y.ld,
                       sc + r * y.lds, y.lds);
  }
  return hipGetLastError();
}

template <int TYPE, class T>
hipError_t dequantize_rows(const th_mx& x, int64_t n, int64_t b, T* Y, int64_t ldy, hipStream_t s) {
  const unsigned char *e = (const unsigned char*)x.elements, *sc = (const unsigned char*)x.scales;
  const int64_t most = rows_at_once(b);
  for (int64_t r = 0; r < n; r += most) {
    const int64_t chunks = (n - r < most ? n - r : most) * (b / 8);
    hipLaunchKernelGGL((mx_dequantize_kernel<TYPE, T>), dim3((unsigned)cdiv(chunks, 256)), dim3(256),
                       0, s, e + r * x.ld, x.ld, sc + r * x.lds, x.lds, (unsigned)chunks,
                       (unsigned)(b / 8), Y + r * ldy, ldy);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(const void* X, th_dtype xdt, int64_t ldx, int64_t n, int64_t b,
                              const th_mx& y, hipStream_t s) {
  typedef unsigned short h;
  if (y.type == TH_MX_E4M3)
    return xdt == TH_BF16 ? quantize_rows<TH_MX_E4M3>((const h*)X, ldx, n, b, y, s)
                          : quantize_rows<TH_MX_E4M3>((const float*)X, ldx, n, b, y, s);
  return xdt == TH_BF16 ? quantize_rows<TH_MX_E2M1>((const h*)X, ldx, n, b, y, s)
                        : quantize_rows<TH_MX_E2M1>((const float*)X, ldx, n, b, y, s);
}

hipError_t launch_mx_dequantize(const th_mx& x, int64_t n, int64_t b, void* Y, th_dtype ydt,
                                int64_t ldy, hipStream_t s) {
  typedef unsigned short h;
  if (x.type == TH_MX_E4M3)
    return ydt == TH_BF16 ? dequantize_rows<TH_MX_E4M3>(x, n, b, (h*)Y, ldy, s)
                          : dequantize_rows<TH_MX_E4M3>(x, n, b, (float*)Y, ldy, s);
  return ydt == TH_BF16 ? dequantize_rows<TH_MX_E2M1>(x, n, b, (h*)Y, ldy, s)
                        : dequantize_rows<TH_MX_E2M1>(x, n, b, (float*)Y, ldy, s);
}

}  // namespace th
