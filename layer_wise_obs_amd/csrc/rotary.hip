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
// and its sine and cosine are rounded to fp32 once. They depend on the token and the
// pair only, so a workgroup computes them once per token into LDS for all its heads of
// q and k, while its first heads are on their way.
// A head is held by a group of lanes with 8 consecutive elements each (16 bytes of
// bf16); a half-layout partner sits in another lane of the group, at the same place where
// rot / 2 is a multiple of 8, and is fetched through LDS where it is not.
#include "common.h"

namespace th {

namespace {

constexpr int kRThreads = 256;
constexpr int kRMaxTokens = 16;  // tokens per workgroup, at most
constexpr int kRMaxPairs = 128;
constexpr int kRBatch = 2;       // heads whose loads are in flight together (four or eight:
                                 // 3% more for 65536 tokens x 64 heads of 128)

struct RotSide {
  const void* x;
  void* y;
  const void* w;
  int heads;
  int64_t xt, xh, yt, yh;
};

struct RotArgs {
  RotSide side[2];
  int64_t from, n;  // tokens [from, n), at most kMaxGroups workgroups of them
  int d, rot, interleaved, tokens;
  const int32_t* pos;
  const double* freqs;
  float amplitude, eps, inv_d;
};

// (cos, sin) of position p at frequency f times the amplitude, formed in fp64 and rounded
// once. (In fp32 from an angle rounded to fp32, a sine or cosine is off by up to 2^-23.4
// however small it is: fp32 heads come out a tenth less exact, 5001 tokens of 28 heads of
// 96 take 20.95 us instead of 21.07.)
__device__ __forceinline__ float2 turn_of(double p, double f, float amplitude) {
  const double t = p * f * 0.15915494309189533577;  // turns
  double s, c;
  sincospi(2.0 * (t - rint(t)), &s, &c);
  return make_float2((float)(c * amplitude), (float)(s * amplitude));
}

// Eight elements as they are in memory, and as floats; aligned like an element only, which
// the memory system takes.
typedef u32x4_t bf16_row_t __attribute__((aligned(2)));
typedef f32x4_t f32_row_t __attribute__((aligned(4)));
template <class T>
struct Raw8;
template <>
struct Raw8<unsigned short> {
  u32x4_t u;
  __device__ __forceinline__ void load(const unsigned short* p) { u = *(const bf16_row_t*)p; }
  __device__ __forceinline__ void to(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
};
template <>
struct Raw8<float> {
  f32x4_t a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *(const f32_row_t*)p;
    b = *(const f32_row_t*)(p + 4);
  }
  __device__ __forceinline__ void to(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  }
};
__device__ __forceinline__ void put8(unsigned short* p, const float (&v)[8]) {
  u32x4_t u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    u[i] = (unsigned)f32_to_bf16_rne(v[2 * i]) | ((unsigned)f32_to_bf16_rne(v[2 * i + 1]) << 16);
  *(bf16_row_t*)p = u;
}
__device__ __forceinline__ void put8(float* p, const float (&v)[8]) {
  *(f32_row_t*)p = f32x4_t{v[0], v[1], v[2], v[3]};
  *(f32_row_t*)(p + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ float get1(const unsigned short* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ float get1(const float* p) { return *p; }
__device__ __forceinline__ void put1(unsigned short* p, float v) { *p = f32_to_bf16_rne(v); }
__device__ __forceinline__ void put1(float* p, float v) { *p = v; }

// Where the other element of a pair is. (29807 tokens, 64 heads of 88, half, normed: 239 us
// with 16-byte accesses and partners through LDS, 817 with a lane per pair; 11625 tokens, 64
// heads of 64, 62 elements interleaved: 34 and 197.)
enum Partner {
  kNext,    // interleaved: the pair is in one lane
  kLane,    // half, rot % 16 == 0: the same element of another lane
  kAnyLane  // half: any element of another lane
};

// 16-byte accesses (d % 8 == 0). G lanes (a power of two >= d / 8) hold a head; the
// workgroup's 256 / G groups are `tokens` tokens x `phases` heads at a time.
template <class T, int G, int PARTNER>
__global__ __launch_bounds__(kRThreads) void rotary_kernel(RotArgs a) {
  __shared__ float2 cs[kRMaxTokens * kRMaxPairs];
  __shared__ __attribute__((aligned(16))) float xs[PARTNER == kAnyLane ? kRThreads * 8 : 4];
  const int pairs = a.rot >> 1;
  const int64_t token0 = a.from + (int64_t)blockIdx.x * a.tokens;
  constexpr int groups = kRThreads / G;
  const int phases = groups / a.tokens;
  const int grp = threadIdx.x / G, lane = threadIdx.x % G;
  const int t = grp / phases, phase = grp - t * phases;
  const int64_t tok = token0 + t;
  const int e0 = lane * 8;
  const bool mine = e0 < a.d, turned = e0 < a.rot;
  const bool works = t < a.tokens && tok < a.n;
  const int all = a.side[0].heads + a.side[1].heads;
  // heads phase, phase + phases, ...: kRBatch of them in flight, the first ones while
  // the angles are formed
  Raw8<T> raw[kRBatch];
  auto fetch = [&](int h0) {
#pragma unroll
    for (int u = 0; u < kRBatch; ++u) {
      const int h = h0 + u * phases;
      if (works && mine && h < all) {
        const bool k = h >= a.side[0].heads;
        const RotSide& sd = a.side[k ? 1 : 0];
        raw[u].load((const T*)sd.x + tok * sd.xt + (int64_t)(k ? h - a.side[0].heads : h) * sd.xh + e0);
      }
    }
  };
  fetch(phase);
  for (int i = threadIdx.x; i < a.tokens * pairs; i += kRThreads) {
    const int ti = i / pairs, p = i - ti * pairs;
    const int64_t tt = token0 + ti;
    if (tt < a.n)
      cs[i] = turn_of(a.pos ? (double)a.pos[tt] : (double)tt, a.freqs[p], a.amplitude);
  }
  __syncthreads();
  if (!works) return;
  // this lane's pairs: 8 of them (half) or 4 (interleaved), the same for every head; an
  // upper element's turn is v cos + partner sin, a lower one's v cos - partner sin
  constexpr int kCs = PARTNER == kNext ? 4 : 8;
  float cosv[kCs], sinv[kCs];
  const bool upper = PARTNER == kLane && e0 >= pairs;  // second element of its pairs
  if (turned) {
    const float2* c = cs + t * pairs;
    if constexpr (PARTNER == kNext) {
      c += e0 / 2;
    } else if constexpr (PARTNER == kLane) {
      c += upper ? e0 - pairs : e0;
    }
#pragma unroll
    for (int i = 0; i < kCs; ++i) {
      const int e = e0 + (PARTNER == kNext ? 2 * i : i);
      if (PARTNER != kLane && e >= a.rot) break;  // kLane: a lane is turned whole or not
      const bool up = PARTNER == kLane ? upper : e >= pairs;
      const float2 w = c[PARTNER != kAnyLane ? i : (up ? e - pairs : e)];
      cosv[i] = w.x;
      sinv[i] = PARTNER == kNext || up ? w.y : -w.y;
    }
  }
  const int hops = pairs / 8;  // kLane: the partner's distance in lanes
  const int partner = (threadIdx.x & 63) + (upper ? -hops : hops);
  for (int h0 = phase; h0 < all; h0 += phases * kRBatch) {
    if (h0 != phase) fetch(h0);
#pragma unroll
    for (int u = 0; u < kRBatch; ++u) {
      const int h = h0 + u * phases;
      if (h >= all) break;
      const bool k = h >= a.side[0].heads;
      const RotSide& sd = a.side[k ? 1 : 0];
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (mine) raw[u].to(v);
      if (sd.w) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += v[i] * v[i];
#pragma unroll
        for (int m = G / 2; m; m >>= 1) s += __shfl_xor(s, m);
        const float scale = rsqrtf(s * a.inv_d + a.eps);
        if (mine) {
          Raw8<T> wr;
          float w[8];
          wr.load((const T*)sd.w + e0);
          wr.to(w);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = v[i] * scale * w[i];
        }
      }
      if constexpr (PARTNER == kNext) {
        if (turned) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (e0 + 2 * i >= a.rot) break;
            const float x = v[2 * i], y = v[2 * i + 1];
            v[2 * i] = x * cosv[i] - y * sinv[i];
            v[2 * i + 1] = y * cosv[i] + x * sinv[i];
          }
        }
      } else {
        float o[8];
        if constexpr (PARTNER == kLane) {
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = __shfl(v[i], partner);
        } else {
          float* head = xs + grp * G * 8;
          wave_sync();  // the head before has been read
          if (turned) {
            *(f32x4_t*)(head + e0) = f32x4_t{v[0], v[1], v[2], v[3]};
            *(f32x4_t*)(head + e0 + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
          }
          wave_sync();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int e = e0 + i;
            if (e < a.rot) o[i] = head[e < pairs ? e + pairs : e - pairs];
          }
        }
        if (turned) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (PARTNER == kLane || e0 + i < a.rot) v[i] = v[i] * cosv[i] + o[i] * sinv[i];
        }
      }
      if (mine)
        put8((T*)sd.y + tok * sd.yt + (int64_t)(k ? h - a.side[0].heads : h) * sd.yh + e0, v);
    }
  }
}

// Heads of any size: a workgroup per token, a wave per head at a
// time, one pair per lane and step.
template <class T>
__global__ __launch_bounds__(kRThreads) void rotary_any_kernel(RotArgs a) {
  __shared__ float2 cs[kRMaxPairs];
  const int64_t tok = a.from + blockIdx.x;
  const int pairs = a.rot >> 1;
  const double p = a.pos ? (double)a.pos[tok] : (double)tok;
  for (int i = threadIdx.x; i < pairs; i += kRThreads) cs[i] = turn_of(p, a.freqs[i], a.amplitude);
  __syncthreads();
  const int all = a.side[0].heads + a.side[1].heads;
  const int lane = threadIdx.x & 63;
  for (int hh = threadIdx.x / 64; hh < all; hh += kRThreads / 64) {
    const bool k = hh >= a.side[0].heads;
    const RotSide& sd = a.side[k ? 1 : 0];
    const int h = k ? hh - a.side[0].heads : hh;
    const T* x = (const T*)sd.x + tok * sd.xt + (int64_t)h * sd.xh;
    T* y = (T*)sd.y + tok * sd.yt + (int64_t)h * sd.yh;
    const T* w = (const T*)sd.w;
    float scale = 1.0f;
    if (w) {
      float s = 0.f;
      for (int e = lane; e < a.d; e += 64) s += get1(x + e) * get1(x + e);
#pragma unroll
      for (int m = 32; m; m >>= 1) s += __shfl_xor(s, m);
      scale = rsqrtf(s * a.inv_d + a.eps);
    }
    auto normed = [&](int e) { return w ? get1(x + e) * scale * get1(w + e) : get1(x + e); };
    for (int i = lane; i < pairs; i += 64) {
      const int ea = a.interleaved ? 2 * i : i, eb = a.interleaved ? 2 * i + 1 : i + pairs;
      const float2 c = cs[i];
      const float va = normed(ea), vb = normed(eb);
      put1(y + ea, va * c.x - vb * c.y);
      put1(y + eb, vb * c.x + va * c.y);
    }
    for (int e = a.rot + lane; e < a.d; e += 64) put1(y + e, normed(e));
  }
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
  for (; a.from < a.n; a.from += kMaxGroups * a.tokens) {
    const int64_t left = cdiv(a.n - a.from, a.tokens);
    const dim3 grid((unsigned)(left < kMaxGroups ? left : kMaxGroups));
    if (a.interleaved)
      hipLaunchKernelGGL((rotary_kernel<T, G, kNext>), grid, dim3(kRThreads), 0, s, a);
    else if (a.rot % 16 == 0)
      hipLaunchKernelGGL((rotary_kernel<T, G, kLane>), grid, dim3(kRThreads), 0, s, a);
    else
      hipLaunchKernelGGL((rotary_kernel<T, G, kAnyLane>), grid, dim3(kRThreads), 0, s, a);
  }
  return hipGetLastError();
}

template <class T>
hipError_t launch_typed(RotArgs a, hipStream_t s) {
  if (a.d % 8) {
    for (; a.from < a.n; a.from += kMaxGroups) {
      const int64_t left = a.n - a.from;
      hipLaunchKernelGGL((rotary_any_kernel<T>),
                         dim3((unsigned)(left < kMaxGroups ? left : kMaxGroups)), dim3(kRThreads), 0,
                         s, a);
    }
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
  a.from = 0;
  a.n = n;
  a.d = (int)d;
  a.rot = (int)rot;
  a.interleaved = interleaved;
  a.tokens = 1;
  a.pos = positions;
  a.freqs = freqs;
  a.amplitude = amplitude;
  a.eps = eps;
  a.inv_d = 1.0f / (float)d;
  return dt == TH_BF16 ? launch_typed<unsigned short>(a, s) : launch_typed<float>(a, s);
}

}  // namespace th
