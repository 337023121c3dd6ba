// Epilogue of the linear layers, act(z + bias) + residual in fp32, rounded once: shared by the
// products of bf16 and of microscaled operands.
#pragma once

#include "common.h"

namespace th {

// 16 bytes of a row of Y or the residual, aligned like its elements only: the memory
// system takes such accesses at any of their addresses, so that odd widths and pitches
// need no code of their own but for a row's last channels. (15485 tokens 2216 -> 9418, gelu
// and residual, bf16: 678 us; element by element, half as much again, 1022 against 694.)
typedef u32x4_t bf16_out_t __attribute__((aligned(2)));
typedef f32x4_t f32_out_t __attribute__((aligned(4)));

struct LinEpilogue {
  const unsigned short* bias;
  const void* residual;
  void* y;
  int64_t ldr, ldy;
  int act;       // th_activation
  int y_f32;     // Y and residual are fp32 (else bf16)
  int past_cache;  // stores past the caches, which Y would not stay in (MX below only)
};

// z Phi(z), Phi(-|z|) = erfc(|z| / sqrt 2) / 2 = e^(-z^2/2) t Q(t), t = 1 / (1 + |z| / 2), Q
// of degree 10 fitted here to erfcx by weighted least squares (2.2e-8 of itself at most, for
// |z| <= 13.8, past which the result is below fp32's range). Every |z| keeps its relative
// accuracy, (16 + 1.5 z^2) 2^-24 counted in roundings; 1 + erff(z / sqrt 2) has none left
// at z = -5. (16384 tokens 4096 -> 4096: 435 us, with erff 446, with erfcf 471.)
__device__ __forceinline__ float gelu(float z) {
  const float a = fabsf(z), t = __builtin_amdgcn_rcpf(fmaf(a, 0.5f, 1.0f));
  float q = -0.0370472595f;
  q = fmaf(q, t, 0.175881296f);
  q = fmaf(q, t, -0.28242594f);
  q = fmaf(q, t, 0.0463377908f);
  q = fmaf(q, t, 0.393810064f);
  q = fmaf(q, t, -0.43306008f);
  q = fmaf(q, t, 0.0639118254f);
  q = fmaf(q, t, 0.0201857612f);
  q = fmaf(q, t, 0.153776303f);
  q = fmaf(q, t, 0.19914858f);
  q = fmaf(q, t, 0.199481636f);
  const float h = q * t * __builtin_amdgcn_exp2f(z * z * -0.72134752044448170f);
  return z > 0.0f ? z * (1.0f - h) : z * h;
}

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case TH_ACT_RELU: return z > 0.0f || z != z ? z : 0.0f;
    case TH_ACT_SILU: return z / (1.0f + expf(-z));
    case TH_ACT_GELU: return gelu(z);
    default: return z;
  }
}

// z / (1 + e^-z) behind products of microscaled operands, by the value alone, whichever kernel forms
// it. From z = -88.7 on e^-z passes fp32's range, where the result, -2.4e-37 there, is still one of
// either type: below kSiluFar it is z e^z, e^z by its root, which is a normal number. NEAR, for outputs
// that are rounded to bf16: to 4 units and |z| 2^-23 of itself, by the hardware's exponential and
// reciprocal (a division and expf would take five times as long).
constexpr float kSiluFar = -87.0f;
template <bool NEAR>
__device__ __forceinline__ float silu_near_zero(float z) {
  return NEAR ? z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504f))
              : activate(z, TH_ACT_SILU);
}
__device__ __forceinline__ float silu_far(float z) {
  const float e = expf(0.5f * z);
  return z * e * e;
}
// The activation of a product of microscaled operands, F32: with an fp32 Y.
template <bool F32>
__device__ __forceinline__ float activate_mx(float z, int act) {
  if (act != TH_ACT_SILU) return activate(z, act);
  return z < kSiluFar ? silu_far(z) : silu_near_zero<!F32>(z);
}

// All of v, one decision for them.
template <bool MX, bool F32>
__device__ __forceinline__ void activate8(float (&v)[8], int act) {
  if (act == TH_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = activate(v[i], TH_ACT_RELU);
  } else if (act == TH_ACT_SILU) {
    if constexpr (MX) {  // far ones are rare
      float least = v[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) least = fminf(least, v[i]);
      if (__any(least < kSiluFar)) {
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          const float z = v[0], y = activate_mx<F32>(z, TH_ACT_SILU);
#pragma unroll
          for (int x = 0; x < 7; ++x) v[x] = v[x + 1];
          v[7] = y;
        }
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = MX ? silu_near_zero<!F32>(v[i]) : activate(v[i], TH_ACT_SILU);
  } else if (act == TH_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = activate(v[i], TH_ACT_GELU);
  }
}

// Residual and store of channel q of token t, its activation v.
__device__ __forceinline__ void put1(float v, int64_t t, int64_t q, const LinEpilogue& ep) {
  if (ep.y_f32) {
    if (ep.residual) v += ((const float*)ep.residual)[t * ep.ldr + q];
    ((float*)ep.y)[t * ep.ldy + q] = v;
  } else {
    if (ep.residual) v += bf16_to_f32(((const unsigned short*)ep.residual)[t * ep.ldr + q]);
    ((unsigned short*)ep.y)[t * ep.ldy + q] = f32_to_bf16_rne(v);
  }
}
// Channel q of token t.
template <bool MX = false>
__device__ __forceinline__ void finish1(float v, int64_t t, int64_t q, const LinEpilogue& ep) {
  if (ep.bias) v += bf16_to_f32(ep.bias[q]);
  if constexpr (MX)
    v = ep.y_f32 ? activate_mx<true>(v, ep.act) : activate_mx<false>(v, ep.act);
  else
    v = activate(v, ep.act);
  put1(v, t, q, ep);
}

// Residuals of eight consecutive channels as they are in memory, and their sum with v
// stored.
template <bool F32>
struct Out8;
template <>
struct Out8<false> {
  bf16_out_t r;
  __device__ __forceinline__ void load(const LinEpilogue& ep, int64_t t, int64_t q) {
    r = *(const bf16_out_t*)((const unsigned short*)ep.residual + t * ep.ldr + q);
  }
  template <bool MX = false>
  __device__ __forceinline__ void put(float (&v)[8], const LinEpilogue& ep, int64_t t, int64_t q) const {
    if (ep.residual) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] += __uint_as_float(r[i] << 16);
        v[2 * i + 1] += __uint_as_float(r[i] & 0xffff0000u);
      }
    }
    bf16x8_t y;
#pragma unroll
    for (int x = 0; x < 8; ++x) y[x] = (__bf16)v[x];
    bf16_out_t* to = (bf16_out_t*)((unsigned short*)ep.y + t * ep.ldy + q);
    if (MX && ep.past_cache)
      __builtin_nontemporal_store(__builtin_bit_cast(u32x4_t, y), to);
    else
      *to = __builtin_bit_cast(u32x4_t, y);
  }
};
template <>
struct Out8<true> {
  f32_out_t a, b;
  __device__ __forceinline__ void load(const LinEpilogue& ep, int64_t t, int64_t q) {
    const float* r = (const float*)ep.residual + t * ep.ldr + q;
    a = *(const f32_out_t*)r;
    b = *(const f32_out_t*)(r + 4);
  }
  template <bool MX = false>
  __device__ __forceinline__ void put(float (&v)[8], const LinEpilogue& ep, int64_t t, int64_t q) const {
    if (ep.residual) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] += a[i];
        v[4 + i] += b[i];
      }
    }
    float* y = (float*)ep.y + t * ep.ldy + q;
    *(f32_out_t*)y = f32x4_t{v[0], v[1], v[2], v[3]};
    *(f32_out_t*)(y + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
  }
};

// Epilogue of a wave's WM strips of 32 tokens, each kPass passes of the lanes' tokens:
// write_strip(i) puts strip i into LDS, values(p) is then the lane's eight channels from q of
// its token(i, p).
template <int WM, int kPass, bool MX = false, class Token, class Values, class Write>
__device__ __forceinline__ void finish_tile(const LinEpilogue& ep, int64_t n, int64_t c, int64_t q,
                                            Token&& token, Values&& values, Write&& write_strip) {
  const bool whole = q + 8 <= c;  // else fewer than eight channels, or none
  // The residuals of all strips, or as many as 64 registers hold, are on their way before the
  // first one is used: read strip by strip they cost 16 round trips to memory a tile.
  auto finish = [&](auto F32) __attribute__((always_inline)) {
    constexpr bool f32 = decltype(F32)::value;
    constexpr int kRoom = 16 / (kPass * (f32 ? 2 : 1)), kHeld = WM < kRoom ? WM : kRoom;
    Out8<f32> res[kHeld][kPass];
    float bias[8];  // once for all tokens: in the loop below every pass would wait for it
#pragma unroll
    for (int x = 0; x < 8; ++x) bias[x] = ep.bias && q + x < c ? bf16_to_f32(ep.bias[q + x]) : 0.f;
#pragma unroll
    for (int i0 = 0; i0 < WM; i0 += kHeld) {
      if (ep.residual) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
#pragma unroll
          for (int p = 0; p < kPass; ++p)
            if (token(i0 + i, p) < n && whole) res[i][p].load(ep, token(i0 + i, p), q);
      }
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        write_strip(i0 + i);
        if (ep.bias || ep.act != TH_ACT_NONE) {  // in place, by the lane that reads it next
#pragma unroll 1
          for (int p = 0; p < kPass; ++p) {
            float *at = values(p), v[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) v[x] = at[x];
            if (ep.bias) {
#pragma unroll
              for (int x = 0; x < 8; ++x) v[x] += bias[x];
            }
            activate8<MX, f32>(v, ep.act);
#pragma unroll
            for (int x = 0; x < 8; ++x) at[x] = v[x];
          }
        }
#pragma unroll
        for (int p = 0; p < kPass; ++p) {
          if (token(i0 + i, p) >= n || !whole) continue;
          const f32x4_t* vp = (const f32x4_t*)values(p);
          const f32x4_t lo = vp[0], hi = vp[1];
          float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
          res[i][p].template put<MX>(v, ep, token(i0 + i, p), q);
        }
        if (!whole) {  // the last channels of a row
#pragma unroll 1
          for (int p = 0; p < kPass; ++p) {
            if (token(i0 + i, p) >= n) break;
#pragma unroll 1
            for (int x = 0; q + x < c; ++x) put1(values(p)[x], token(i0 + i, p), q + x, ep);
          }
        }
        wave_sync();
      }
    }
  };
  if (ep.y_f32)
    finish(std::integral_constant<bool, true>{});
  else
    finish(std::integral_constant<bool, false>{});
}

// Sum of the splits' raw products in order, then the epilogue: 8 channels per thread,
// those of a row's end one by one.
template <bool MX>
__global__ __launch_bounds__(256) void linear_join_kernel(const float* __restrict__ part, int splits,
                                                          int64_t n, int64_t c, LinEpilogue ep) {
  const int64_t per_row = cdiv(c, 8), cp = per_row * 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n * per_row) return;
  const int64_t t = i / per_row, q = (i - t * per_row) * 8;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const f32x4_t* p = (const f32x4_t*)(part + t * cp + q);
#pragma unroll 4
  for (int s = 0; s < splits; ++s, p += n * cp / 4) {
    const f32x4_t lo = p[0], hi = p[1];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      v[x] += lo[x];
      v[4 + x] += hi[x];
    }
  }
  if (ep.bias) {
#pragma unroll
    for (int x = 0; x < 8; ++x) v[x] += q + x < c ? bf16_to_f32(ep.bias[q + x]) : 0.f;
  }
  if (ep.y_f32)
    activate8<MX, true>(v, ep.act);
  else
    activate8<MX, false>(v, ep.act);
  if (q + 8 > c) {
#pragma unroll
    for (int x = 0; x < 8; ++x)
      if (q + x < c) put1(v[x], t, q + x, ep);
    return;
  }
  auto put = [&](auto F32) {
    Out8<decltype(F32)::value> r;
    if (ep.residual) r.load(ep, t, q);
    r.put(v, ep, t, q);
  };
  if (ep.y_f32)
    put(std::integral_constant<bool, true>{});
  else
    put(std::integral_constant<bool, false>{});
}

}  // namespace th
