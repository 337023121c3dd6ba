// Linear layer with its epilogue, Y = act(X W^T + bias) + residual: X token-major
// [n, b], W [c, b] (row = output channel) in bf16, products exact in fp32 on the
// matrix cores, fp32 sums, epilogue in fp32, Y (bf16 or fp32) rounded once.
//
// "Pruning LLMs with Thanos", section "The compression target: linear layers": the
// layers a block consists of; section "The layer-reconstruction lens": the input of
// a layer is what its pruned predecessors produce.
//
// Tiles of (64 WM) tokens x (64 WN) channels on four waves (2 x 2, each
// 32 WM x 32 WN of v_mfma_f32_32x32x16_bf16 blocks). The contraction is contiguous
// in both operands, so an MFMA operand (8 consecutive k of a row per lane) is one
// 16-byte LDS read. Stages of 32 k (64-byte rows) are filled by direct global->LDS
// loads, four stages deep with the loads three ahead; the 16-byte pieces of a row
// are XOR-swizzled by (row / 4) & 3, so the operand reads (16 rows at one piece per
// 16 lanes) use all 64 banks. Fragments are double-buffered over the two 16-wide
// substeps of a stage. Tiles are walked in groups of 8 token tiles per channel
// tile, each XCD a contiguous range of that order, so that the workgroups of an
// XCD share X and W slices in its L2.
#include "common.h"
#include "lds_dma.h"

namespace th {

namespace {

constexpr int kLK = 32;  // contraction per stage
constexpr int kLThreads = 256;
constexpr int kLStages = 4;
constexpr int kLGroup = 8;  // token tiles per group in the walk order
constexpr int kLRow = kLK * 2;

__device__ __forceinline__ int lsw_off(int r, int piece) {
  return r * kLRow + ((piece ^ ((r >> 2) & 3)) << 4);
}

struct LinEpilogue {
  const unsigned short* bias;
  const void* residual;
  void* y;
  int64_t ldr, ldy;
  int act;       // th_activation
  int y_f32;     // Y and residual are fp32 (else bf16)
  int vec;       // 8 consecutive channels move as one or two 16-byte accesses
};

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case TH_ACT_RELU: return z > 0.0f || z != z ? z : 0.0f;
    case TH_ACT_SILU: return z / (1.0f + expf(-z));
    case TH_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    default: return z;
  }
}

// Eight consecutive channels q .. q+7 of token t (q + i < c and t < n hold where
// the caller passes `count` of them).
__device__ __forceinline__ void finish8(float (&v)[8], int64_t t, int64_t q, int count,
                                        const LinEpilogue& ep) {
  if (ep.bias) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < count) v[i] += bf16_to_f32(ep.bias[q + i]);
  }
  if (ep.act != TH_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = activate(v[i], ep.act);
  }
  if (ep.vec) {  // then count is 8
    if (ep.y_f32) {
      if (ep.residual) {
        const f32x4_t* r = (const f32x4_t*)((const float*)ep.residual + t * ep.ldr + q);
        const f32x4_t a = r[0], b = r[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] += a[i];
          v[4 + i] += b[i];
        }
      }
      f32x4_t* y = (f32x4_t*)((float*)ep.y + t * ep.ldy + q);
      y[0] = f32x4_t{v[0], v[1], v[2], v[3]};
      y[1] = f32x4_t{v[4], v[5], v[6], v[7]};
    } else {
      if (ep.residual) {
        const u32x4_t r = *(const u32x4_t*)((const unsigned short*)ep.residual + t * ep.ldr + q);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] += __uint_as_float(r[i] << 16);
          v[2 * i + 1] += __uint_as_float(r[i] & 0xffff0000u);
        }
      }
      u32x4_t o;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = (unsigned)f32_to_bf16_rne(v[2 * i]) | ((unsigned)f32_to_bf16_rne(v[2 * i + 1]) << 16);
      *(u32x4_t*)((unsigned short*)ep.y + t * ep.ldy + q) = o;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i >= count) break;
    if (ep.y_f32) {
      if (ep.residual) v[i] += ((const float*)ep.residual)[t * ep.ldr + q + i];
      ((float*)ep.y)[t * ep.ldy + q + i] = v[i];
    } else {
      if (ep.residual) v[i] += bf16_to_f32(((const unsigned short*)ep.residual)[t * ep.ldr + q + i]);
      ((unsigned short*)ep.y)[t * ep.ldy + q + i] = f32_to_bf16_rne(v[i]);
    }
  }
}

// Workgroup (x, split): tile x of the walk order, stages [split per, split per + per)
// of the contraction. With part set, the tile's raw sums go to part[split][n][c].
template <int WM, int WN>
__global__ __launch_bounds__(kLThreads) void linear_tile_kernel(
    const unsigned short* __restrict__ X, int64_t ldx, const unsigned short* __restrict__ W,
    int64_t n, int64_t b, int64_t c, int ntm, int ntn, int per_xcd, int stages_per_split,
    float* __restrict__ part, LinEpilogue ep) {
  constexpr int TM = 64 * WM, TN = 64 * WN;
  constexpr int kA = TM * kLRow, kB = TN * kLRow, kStage = kA + kB;
  constexpr int kLoads = WM + WN;  // 1 KB loads per wave and stage
  const int wg = blockIdx.x;
  const int lin = (wg % 8) * per_xcd + wg / 8;
  if (lin >= ntm * ntn) return;
  int tm, tn;
  {
    const int per_group = kLGroup * ntn;
    const int g = lin / per_group, in = lin - g * per_group;
    const int gs = min(kLGroup, ntm - g * kLGroup);
    tm = g * kLGroup + in % gs;
    tn = in / gs;
  }
  const int64_t M0 = (int64_t)tm * TM, N0 = (int64_t)tn * TN;
  const int nk_all = (int)cdiv(b, kLK);
  const int s_begin = blockIdx.y * stages_per_split;
  const int nk = min(stages_per_split, nk_all - s_begin);
  if (nk <= 0) return;  // no split of the launch is empty

  __shared__ __attribute__((aligned(1024))) unsigned char sm[kLStages * kStage];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;

  // Loader: chunks of 1 KB (16 rows of 64 bytes); wave w loads chunks w + 4 m of
  // either operand. Lane l fills row 16 chunk + l/4 at physical piece l%4.
  const int lrow = lane >> 2;
  const int lp = (lane & 3) ^ ((lrow >> 2) & 3);  // (row / 4) & 3 is the same in every chunk
  unsigned va[WM], vb[WN];
  int64_t ra, rb;
#pragma unroll
  for (int m = 0; m < WM; ++m) {
    ra = M0 + (wave + 4 * m) * 16 + lrow;
    ra = ra < n ? ra : n - 1;  // rows past the end feed outputs that are never stored
    va[m] = (unsigned)(((ra - M0) * ldx + lp * 8) * 2);
  }
#pragma unroll
  for (int m = 0; m < WN; ++m) {
    rb = N0 + (wave + 4 * m) * 16 + lrow;
    rb = rb < c ? rb : c - 1;
    vb[m] = (unsigned)(((rb - N0) * b + lp * 8) * 2);
  }
  const unsigned short* Xt = X + M0 * ldx;
  const unsigned short* Wt = W + N0 * b;
  // Stages past the last are loaded too (at most three, never read), so that every
  // stage has the same number of loads for the vmcnt waits; they re-read the last.
  auto issue_stage = [&](int it) {
    unsigned char* sbase = sm + (it % kLStages) * kStage;
    int st = s_begin + it;
    st = st < nk_all ? st : nk_all - 1;
    const int64_t k0 = (int64_t)st * kLK;
    if (k0 + kLK <= b) {
      lds_dma_s<WM>(va, Xt + k0, sbase + wave * 1024);
      lds_dma_s<WN>(vb, Wt + k0, sbase + kA + wave * 1024);
    } else {  // pieces past b re-read piece 0 of the stage; zero_tail clears them
      const unsigned back = k0 + lp * 8 < b ? 0u : (unsigned)(lp * 16);
      unsigned ta[WM], tb[WN];
#pragma unroll
      for (int m = 0; m < WM; ++m) ta[m] = va[m] - back;
#pragma unroll
      for (int m = 0; m < WN; ++m) tb[m] = vb[m] - back;
      lds_dma_s<WM>(ta, Xt + k0, sbase + wave * 1024);
      lds_dma_s<WN>(tb, Wt + k0, sbase + kA + wave * 1024);
    }
  };
  // zero this wave's pieces of stage it that lie past b (its own loads have landed)
  auto zero_tail = [&](int it) {
    const int64_t k0 = (int64_t)(s_begin + it) * kLK;
    if (k0 + kLK <= b || k0 + lp * 8 < b) return;
    unsigned char* sbase = sm + (it % kLStages) * kStage + wave * 1024 + lane * 16;
#pragma unroll
    for (int m = 0; m < WM; ++m) *(u32x4_t*)(sbase + m * 4096) = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
    for (int m = 0; m < WN; ++m) *(u32x4_t*)(sbase + kA + m * 4096) = u32x4_t{0u, 0u, 0u, 0u};
  };

  f32x16_t acc[WM][WN];
#pragma unroll
  for (int i = 0; i < WM; ++i)
#pragma unroll
    for (int j = 0; j < WN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
  const int r32 = lane & 31, half = lane >> 5;
  bf16x8_t a0[WM], b0[WN], a1[WM], b1[WN];
  auto read_frags = [&](const unsigned char* st, int sub, bf16x8_t (&a)[WM], bf16x8_t (&bb)[WN]) {
    const int pc = sub * 2 + half;  // piece of this lane's 8 k values
#pragma unroll
    for (int i = 0; i < WM; ++i)
      a[i] = *(const bf16x8_t*)(st + lsw_off(wm * 32 * WM + i * 32 + r32, pc));
#pragma unroll
    for (int j = 0; j < WN; ++j)
      bb[j] = *(const bf16x8_t*)(st + kA + lsw_off(wn * 32 * WN + j * 32 + r32, pc));
  };
  auto mfmas = [&](const bf16x8_t (&a)[WM], const bf16x8_t (&bb)[WN]) {
#pragma unroll
    for (int i = 0; i < WM; ++i)
#pragma unroll
      for (int j = 0; j < WN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], bb[j], acc[i][j], 0, 0, 0);
  };
  // all but the newest two stages of this wave's loads have landed
  auto wait_loads = [&] {
    if constexpr (kLoads == 8)
      __asm__ volatile("s_waitcnt vmcnt(16)" ::: "memory");
    else if constexpr (kLoads == 6)
      __asm__ volatile("s_waitcnt vmcnt(12)" ::: "memory");
    else
      __asm__ volatile("s_waitcnt vmcnt(8)" ::: "memory");
  };
  static_assert(kLoads == 8 || kLoads == 6 || kLoads == 4, "vmcnt immediates");

  issue_stage(0);
  issue_stage(1);
  issue_stage(2);
  wait_loads();
  zero_tail(0);
  __syncthreads();
  read_frags(sm, 0, a0, b0);
  for (int it0 = 0; it0 < nk; it0 += kLStages) {
    static_for<0, kLStages>([&](auto U) __attribute__((always_inline)) {
      constexpr int u = U;
      const int it = it0 + u;
      if (it < nk) {
        issue_stage(it0 + u + 3);  // its buffer was last read before the barrier of it-1
        read_frags(sm + u * kStage, 1, a1, b1);
        mfmas(a0, b0);
        wait_loads();
        zero_tail(it + 1);
        __syncthreads();
        read_frags(sm + ((u + 1) % kLStages) * kStage, 0, a0, b0);
        mfmas(a1, b1);
      }
    });
  }
  __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();  // every wave's loads have landed: the stages may be reused

  // Epilogue through LDS, one 32-token strip of the wave's block at a time: the lane
  // holds channel r32 of each 32 x 32 block and tokens 8 (e / 4) + 4 half + (e % 4);
  // read back, a lane has 8 consecutive channels of one token. The row pitch puts
  // the two halves of a write 128 bytes apart in the banks.
  constexpr int kCols = 32 * WN, kPitch = kCols + 8;
  static_assert(4 * 32 * kPitch * 4 <= kLStages * kStage, "strips fit the stages");
  float* strip = (float*)sm + wave * 32 * kPitch;
  constexpr int kLanes = kCols / 8;      // lanes per token
  constexpr int kTok = 64 / kLanes;      // tokens per pass
#pragma unroll
  for (int i = 0; i < WM; ++i) {
#pragma unroll
    for (int j = 0; j < WN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        strip[((e >> 2) * 8 + half * 4 + (e & 3)) * kPitch + j * 32 + r32] = acc[i][j][e];
    wave_sync();
#pragma unroll 1
    for (int t0 = 0; t0 < 32; t0 += kTok) {
      const int tr = t0 + lane / kLanes;
      const int64_t t = M0 + wm * 32 * WM + i * 32 + tr;
      const int64_t q = N0 + wn * kCols + (lane % kLanes) * 8;
      if (t < n && q < c) {
        const f32x4_t* p = (const f32x4_t*)(strip + tr * kPitch + (lane % kLanes) * 8);
        const f32x4_t lo = p[0], hi = p[1];
        float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        const int count = c - q < 8 ? (int)(c - q) : 8;
        if (part) {
          float* o = part + ((int64_t)blockIdx.y * n + t) * c + q;
#pragma unroll
          for (int x = 0; x < 8; ++x)
            if (x < count) o[x] = v[x];
        } else {
          finish8(v, t, q, count, ep);
        }
      }
    }
    wave_sync();
  }
}

// Sum of the splits' raw products in order, then the epilogue: 8 channels per thread.
__global__ __launch_bounds__(256) void linear_join_kernel(const float* __restrict__ part, int splits,
                                                          int64_t n, int64_t c, LinEpilogue ep) {
  const int64_t per_row = cdiv(c, 8);
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n * per_row) return;
  const int64_t t = i / per_row, q = (i - t * per_row) * 8;
  const int count = c - q < 8 ? (int)(c - q) : 8;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < splits; ++s) {
    const float* p = part + ((int64_t)s * n + t) * c + q;
#pragma unroll
    for (int x = 0; x < 8; ++x)
      if (x < count) v[x] += p[x];
  }
  finish8(v, t, q, count, ep);
}

struct LinPlan {
  int big;     // 256 x 256 tiles (else 128 x 128)
  int splits;  // pieces of the contraction
  int per;     // stages per piece
};

constexpr int kUnits = 256;  // compute units

LinPlan plan_of(int64_t n, int64_t b, int64_t c, bool can_split) {
  LinPlan p;
  const int64_t big_tiles = cdiv(n, 256) * cdiv(c, 256);
  p.big = big_tiles >= kUnits;
  const int64_t tiles = p.big ? big_tiles : cdiv(n, 128) * cdiv(c, 128);
  const int64_t stages = cdiv(b, kLK);
  int64_t splits = 1;
  if (can_split && tiles < 2 * kUnits) {
    splits = 2 * kUnits / tiles;
    if (splits > stages / 8) splits = stages / 8;
    if (splits < 1) splits = 1;
  }
  p.per = (int)cdiv(stages, splits);
  p.splits = (int)cdiv(stages, p.per);
  return p;
}

template <int WM, int WN>
hipError_t launch_tiles(const unsigned short* X, int64_t ldx, const unsigned short* W, int64_t n,
                        int64_t b, int64_t c, const LinPlan& p, float* part, const LinEpilogue& ep,
                        hipStream_t s) {
  const int ntm = (int)cdiv(n, 64 * WM), ntn = (int)cdiv(c, 64 * WN);
  const int per_xcd = (int)cdiv((int64_t)ntm * ntn, 8);
  hipLaunchKernelGGL((linear_tile_kernel<WM, WN>), dim3((unsigned)(8 * per_xcd), (unsigned)p.splits),
                     dim3(kLThreads), 0, s, X, ldx, W, n, b, c, ntm, ntn, per_xcd, p.per, part, ep);
  return hipGetLastError();
}

}  // namespace

size_t linear_workspace_floats(int64_t n, int64_t b, int64_t c) {
  const LinPlan p = plan_of(n, b, c, true);
  return p.splits > 1 ? (size_t)p.splits * (size_t)n * (size_t)c : 0;
}

hipError_t launch_linear(const unsigned short* X, int64_t ldx, const unsigned short* W, int64_t n,
                         int64_t b, int64_t c, const unsigned short* bias, int act,
                         const void* residual, int64_t ldr, void* Y, th_dtype ydt, int64_t ldy,
                         float* part, hipStream_t s) {
  LinEpilogue ep;
  ep.bias = bias;
  ep.residual = residual;
  ep.y = Y;
  ep.ldr = ldr;
  ep.ldy = ldy;
  ep.act = act;
  ep.y_f32 = ydt == TH_F32;
  const int64_t el = ep.y_f32 ? 4 : 8;
  ep.vec = c % 8 == 0 && ldy % el == 0 && (!residual || ldr % el == 0) &&
           (((uintptr_t)Y | (uintptr_t)residual) & 15) == 0;
  const LinPlan p = plan_of(n, b, c, part != nullptr);
  float* raw = p.splits > 1 ? part : nullptr;
  hipError_t e = p.big ? launch_tiles<4, 4>(X, ldx, W, n, b, c, p, raw, ep, s)
                       : launch_tiles<2, 2>(X, ldx, W, n, b, c, p, raw, ep, s);
  if (e != hipSuccess || !raw) return e;
  const int64_t items = n * cdiv(c, 8);
  hipLaunchKernelGGL(linear_join_kernel, dim3((unsigned)cdiv(items, 256)), dim3(256), 0, s, raw,
                     p.splits, n, c, ep);
  return hipGetLastError();
}

}  // namespace th
