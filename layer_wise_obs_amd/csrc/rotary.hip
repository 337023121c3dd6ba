// Rotary positions of queries and keys, with the norm of each head in the same pass.
//
// A head x of d elements is first normed where a weight w is given,
//   x_e <- x_e / sqrt(mean_e x_e^2 + eps) * w_e,
// then the pairs of its first `rot` elements are turned by the token's position p
// times the pair's frequency f_i,
//   (a, b) <- amplitude * (a cos p f_i - b sin p f_i, b cos p f_i + a sin p f_i),
// with (a, b) = (x_i, x_{i + rot/2}) ("half") or (x_2i, x_2i+1) ("interleaved").
//
// Bound by memory: one read and one write of the heads. p f_i is formed and
// reduced to turns in fp64 (p f_i reaches 10^6 radians, where fp32 is off by 0.06),
// then sine and cosine are fp32. They depend on the token and the pair only, so a
// workgroup computes them once per token into LDS for all its heads of q and k.
// A head is held by a group of lanes with 8 consecutive elements each (16 bytes of
// bf16); a half-layout partner sits in another lane of the group.
#include "common.h"

namespace th {

namespace {

constexpr int kRThreads = 256;
constexpr int kRMaxTokens = 16;  // tokens per workgroup, at most
constexpr int kRMaxPairs = 128;
constexpr int kRBatch = 4;       // heads whose loads are in flight together

struct RotSide {
  const void* x;
  void* y;
  const void* w;
  int heads;
  int64_t xt, xh, yt, yh;
};

struct RotArgs {
  RotSide side[2];
  int64_t n;
  int d, rot, interleaved, tokens;
  const int32_t* pos;
  const double* freqs;
  float amplitude, eps;
};

// (cos, sin) of position p at frequency f, in fp32 from an angle reduced in fp64.
__device__ __forceinline__ float2 turn_of(double p, double f, float amplitude) {
  double t = p * f * 0.15915494309189533577;  // turns
  t -= rint(t);
  float s, c;
  sincospif((float)(2.0 * t), &s, &c);
  return make_float2(c * amplitude, s * amplitude);
}

__device__ __forceinline__ void unpack8(const u32x4_t& u, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void get8(const unsigned short* p, float (&v)[8]) {
  unpack8(*(const u32x4_t*)p, v);
}
__device__ __forceinline__ void get8(const float* p, float (&v)[8]) {
  const f32x4_t a = ((const f32x4_t*)p)[0], b = ((const f32x4_t*)p)[1];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}
__device__ __forceinline__ void put8(unsigned short* p, const float (&v)[8]) {
  u32x4_t u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    u[i] = (unsigned)f32_to_bf16_rne(v[2 * i]) | ((unsigned)f32_to_bf16_rne(v[2 * i + 1]) << 16);
  *(u32x4_t*)p = u;
}
__device__ __forceinline__ void put8(float* p, const float (&v)[8]) {
  ((f32x4_t*)p)[0] = f32x4_t{v[0], v[1], v[2], v[3]};
  ((f32x4_t*)p)[1] = f32x4_t{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ float get1(const unsigned short* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ float get1(const float* p) { return *p; }
__device__ __forceinline__ void put1(unsigned short* p, float v) { *p = f32_to_bf16_rne(v); }
__device__ __forceinline__ void put1(float* p, float v) { *p = v; }

// 16-byte accesses. G lanes (a power of two >= d / 8) hold a head; the workgroup's
// 256 / G groups are `tokens` tokens x `phases` heads at a time.
template <class T, int G, bool INTERLEAVED>
__global__ __launch_bounds__(kRThreads) void rotary_kernel(RotArgs a) {
  __shared__ float2 cs[kRMaxTokens * kRMaxPairs];
  const int pairs = a.rot >> 1;
  const int64_t token0 = (int64_t)blockIdx.x * a.tokens;
  for (int i = threadIdx.x; i < a.tokens * pairs; i += kRThreads) {
    const int t = i / pairs, p = i - t * pairs;
    const int64_t tok = token0 + t;
    if (tok < a.n)
      cs[i] = turn_of(a.pos ? (double)a.pos[tok] : (double)tok, a.freqs[p], a.amplitude);
  }
  __syncthreads();
  constexpr int groups = kRThreads / G;
  const int phases = groups / a.tokens;
  const int grp = threadIdx.x / G, lane = threadIdx.x % G;
  const int t = grp / phases, phase = grp - t * phases;
  const int64_t tok = token0 + t;
  if (t >= a.tokens || tok >= a.n) return;
  const int e0 = lane * 8;
  const bool mine = e0 < a.d, turned = e0 < a.rot;
  // this lane's pairs: 8 of them (half) or 4 (interleaved), the same for every head
  float cosv[INTERLEAVED ? 4 : 8], sinv[INTERLEAVED ? 4 : 8];
  const bool upper = !INTERLEAVED && e0 >= pairs;  // second element of its pairs
  if (turned) {
    const float2* c = cs + t * pairs + (INTERLEAVED ? e0 / 2 : (upper ? e0 - pairs : e0));
#pragma unroll
    for (int i = 0; i < (INTERLEAVED ? 4 : 8); ++i) {
      cosv[i] = c[i].x;
      sinv[i] = c[i].y;
    }
  }
  const int hops = pairs / 8;  // half: the partner's distance in lanes
  const int partner = (threadIdx.x & 63) + (upper ? -hops : hops);
  const int all = a.side[0].heads + a.side[1].heads;
  for (int h0 = phase; h0 < all; h0 += phases * kRBatch) {
    float v[kRBatch][8];
#pragma unroll
    for (int u = 0; u < kRBatch; ++u) {
      const int h = h0 + u * phases;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
      if (h < all && mine) {
        const bool k = h >= a.side[0].heads;
        const RotSide& sd = a.side[k ? 1 : 0];
        get8((const T*)sd.x + tok * sd.xt + (int64_t)(k ? h - a.side[0].heads : h) * sd.xh + e0, v[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kRBatch; ++u) {
      const int h = h0 + u * phases;
      if (h >= all) break;
      const bool k = h >= a.side[0].heads;
      const RotSide& sd = a.side[k ? 1 : 0];
      if (sd.w) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += v[u][i] * v[u][i];
#pragma unroll
        for (int m = G / 2; m; m >>= 1) s += __shfl_xor(s, m);
        const float scale = 1.0f / sqrtf(s / (float)a.d + a.eps);
        if (mine) {
          float w[8];
          get8((const T*)sd.w + e0, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[u][i] = v[u][i] * scale * w[i];
        }
      }
      if constexpr (INTERLEAVED) {
        if (turned) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = v[u][2 * i], y = v[u][2 * i + 1];
            v[u][2 * i] = x * cosv[i] - y * sinv[i];
            v[u][2 * i + 1] = y * cosv[i] + x * sinv[i];
          }
        }
      } else {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = __shfl(v[u][i], partner);
        if (turned) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            v[u][i] = upper ? v[u][i] * cosv[i] + o[i] * sinv[i] : v[u][i] * cosv[i] - o[i] * sinv[i];
        }
      }
      if (mine)
        put8((T*)sd.y + tok * sd.yt + (int64_t)(k ? h - a.side[0].heads : h) * sd.yh + e0, v[u]);
    }
  }
}

// Any head size, pitch and alignment: one wave per head, one pair per lane and step.
template <class T>
__global__ __launch_bounds__(kRThreads) void rotary_any_kernel(RotArgs a) {
  const int all = a.side[0].heads + a.side[1].heads;
  const int64_t row = (int64_t)blockIdx.x * (kRThreads / 64) + threadIdx.x / 64;
  const int64_t tok = row / all;
  const int lane = threadIdx.x & 63;
  if (tok >= a.n) return;
  int h = (int)(row - tok * all);
  const bool k = h >= a.side[0].heads;
  const RotSide& sd = a.side[k ? 1 : 0];
  if (k) h -= a.side[0].heads;
  const T* x = (const T*)sd.x + tok * sd.xt + (int64_t)h * sd.xh;
  T* y = (T*)sd.y + tok * sd.yt + (int64_t)h * sd.yh;
  const T* w = (const T*)sd.w;
  float scale = 1.0f;
  if (w) {
    float s = 0.f;
    for (int e = lane; e < a.d; e += 64) s += get1(x + e) * get1(x + e);
#pragma unroll
    for (int m = 32; m; m >>= 1) s += __shfl_xor(s, m);
    scale = 1.0f / sqrtf(s / (float)a.d + a.eps);
  }
  auto normed = [&](int e) { return w ? get1(x + e) * scale * get1(w + e) : get1(x + e); };
  const int pairs = a.rot >> 1;
  const double p = a.pos ? (double)a.pos[tok] : (double)tok;
  for (int i = lane; i < pairs; i += 64) {
    const int ea = a.interleaved ? 2 * i : i, eb = a.interleaved ? 2 * i + 1 : i + pairs;
    const float2 c = turn_of(p, a.freqs[i], a.amplitude);
    const float va = normed(ea), vb = normed(eb);
    put1(y + ea, va * c.x - vb * c.y);
    put1(y + eb, vb * c.x + va * c.y);
  }
  for (int e = a.rot + lane; e < a.d; e += 64) put1(y + e, normed(e));
}

template <class T, int G>
hipError_t launch_group(RotArgs a, hipStream_t s) {
  // a group of lanes takes at least kRBatch heads of its token where there are
  // that many, and the workgroup as many tokens as then have a group
  const int groups = kRThreads / G, all = a.side[0].heads + a.side[1].heads;
  int phases = 1;
  while (phases < groups && phases * kRBatch < all) phases *= 2;
  a.tokens = groups / phases;
  if (a.tokens > kRMaxTokens) a.tokens = kRMaxTokens;
  const dim3 grid((unsigned)cdiv(a.n, a.tokens));
  if (a.interleaved)
    hipLaunchKernelGGL((rotary_kernel<T, G, true>), grid, dim3(kRThreads), 0, s, a);
  else
    hipLaunchKernelGGL((rotary_kernel<T, G, false>), grid, dim3(kRThreads), 0, s, a);
  return hipGetLastError();
}

template <class T>
hipError_t launch_typed(const RotArgs& a, hipStream_t s) {
  // 16-byte accesses need whole chunks of 8 elements on either side of a pair
  const int64_t el = 16 / sizeof(T);
  bool vec = a.d % 8 == 0 && a.rot % 8 == 0 && (a.interleaved || a.rot % 16 == 0);
  for (const RotSide& sd : a.side) {
    if (!sd.heads) continue;
    vec = vec && sd.xt % el == 0 && sd.xh % el == 0 && sd.yt % el == 0 && sd.yh % el == 0 &&
          (((uintptr_t)sd.x | (uintptr_t)sd.y | (uintptr_t)sd.w) & 15) == 0;
  }
  if (!vec) {
    const int64_t rows = a.n * (a.side[0].heads + a.side[1].heads);
    hipLaunchKernelGGL((rotary_any_kernel<T>), dim3((unsigned)cdiv(rows, kRThreads / 64)),
                       dim3(kRThreads), 0, s, a);
    return hipGetLastError();
  }
  if (a.d <= 64) return launch_group<T, 8>(a, s);
  if (a.d <= 128) return launch_group<T, 16>(a, s);
  return launch_group<T, 32>(a, s);
}

RotSide side_of(const th_heads* h) {
  if (!h) return RotSide{nullptr, nullptr, nullptr, 0, 0, 0, 0, 0};
  return RotSide{h->x, h->y, h->norm, (int)h->heads, h->x_token, h->x_head, h->y_token, h->y_head};
}

}  // namespace

hipError_t launch_rotary(const th_heads* q, const th_heads* k, th_dtype dt, int64_t n, int64_t d,
                         int64_t rot, int interleaved, const int32_t* positions,
                         const double* freqs, float amplitude, float eps, hipStream_t s) {
  RotArgs a;
  a.side[0] = side_of(q);
  a.side[1] = side_of(k);
  a.n = n;
  a.d = (int)d;
  a.rot = (int)rot;
  a.interleaved = interleaved;
  a.tokens = 1;
  a.pos = positions;
  a.freqs = freqs;
  a.amplitude = amplitude;
  a.eps = eps;
  return dt == TH_BF16 ? launch_typed<unsigned short>(a, s) : launch_typed<float>(a, s);
}

}  // namespace th
