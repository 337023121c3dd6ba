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
// 16-byte LDS read. Stages of 64 k (128-byte rows, whole cache lines) are filled by
// direct global->LDS loads, S stages deep; the 16-byte pieces of a row are
// XOR-swizzled by (row / 2) & 7, so the operand reads (16 rows at one piece per 16
// lanes) use all 64 banks. Fragments are double-buffered over the four 16-wide
// substeps of a stage. Tiles are walked in groups of 8 token tiles per channel tile,
// each XCD a contiguous range of that order, so that the workgroups of an XCD share
// X and W slices in its L2.
#include "common.h"
#include "lds_dma.h"

namespace th {

namespace {

constexpr int kLK = 64;  // contraction per stage
constexpr int kLThreads = 256;
constexpr int kLGroup = 8;  // token tiles per group in the walk order
constexpr int kLRow = kLK * 2;

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

// Channel q of token t.
__device__ __forceinline__ void finish1(float v, int64_t t, int64_t q, const LinEpilogue& ep) {
  if (ep.bias) v += bf16_to_f32(ep.bias[q]);
  v = activate(v, ep.act);
  if (ep.y_f32) {
    if (ep.residual) v += ((const float*)ep.residual)[t * ep.ldr + q];
    ((float*)ep.y)[t * ep.ldy + q] = v;
  } else {
    if (ep.residual) v += bf16_to_f32(((const unsigned short*)ep.residual)[t * ep.ldr + q]);
    ((unsigned short*)ep.y)[t * ep.ldy + q] = f32_to_bf16_rne(v);
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
// of the contraction. With part set, the tile's raw sums go to part[split][n][cp], cp
// being c rounded up to 8.
template <int WM, int WN, int S>
__global__ __launch_bounds__(kLThreads) void linear_tile_kernel(
    const unsigned short* __restrict__ X, int64_t ldx, const unsigned short* __restrict__ W,
    int64_t n, int64_t b, int64_t c, int ntm, int ntn, int per_xcd, int stages_per_split,
    float* __restrict__ part, LinEpilogue ep) {
  constexpr int TM = 64 * WM, TN = 64 * WN;
  constexpr int kA = TM * kLRow, kB = TN * kLRow, kStage = kA + kB;
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

  __shared__ __attribute__((aligned(1024))) unsigned char sm[S * kStage];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;

  // Loader: chunks of 1 KB (8 rows of 128 bytes); wave w loads chunks w + 4 m of
  // either operand, m < 2 WM (2 WN). Lane l fills row 8 chunk + l/8 at physical piece
  // l%8; (row / 2) & 7 is the same in each of its chunks.
  const int lrow = lane >> 3;
  const int lp = (lane & 7) ^ (((wave & 1) << 2) + (lane >> 4));
  unsigned va[2][WM], vb[2][WN];
#pragma unroll
  for (int m = 0; m < 2 * WM; ++m) {
    int64_t r = M0 + (wave + 4 * m) * 8 + lrow;
    r = r < n ? r : n - 1;  // rows past the end feed outputs that are never stored
    va[m / WM][m % WM] = (unsigned)(((r - M0) * ldx + lp * 8) * 2);
  }
#pragma unroll
  for (int m = 0; m < 2 * WN; ++m) {
    int64_t r = N0 + (wave + 4 * m) * 8 + lrow;
    r = r < c ? r : c - 1;
    vb[m / WN][m % WN] = (unsigned)(((r - N0) * b + lp * 8) * 2);
  }
  const unsigned short* Xt = X + M0 * ldx;
  const unsigned short* Wt = W + N0 * b;
  // Stages past the last are loaded too (at most S - 1, never read), so that every
  // stage has the same number of loads for the vmcnt waits; they re-read the last.
  // Pieces past b re-read piece 0 of the stage; zero_tail clears them.
  auto stage_k0 = [&](int it) {
    const int st = s_begin + it;
    return (int64_t)(st < nk_all ? st : nk_all - 1) * kLK;
  };
  auto issue_a = [&](int it) {
    unsigned char* sbase = sm + (it % S) * kStage + wave * 1024;
    const int64_t k0 = stage_k0(it);
    const unsigned back = k0 + lp * 8 < b ? 0u : (unsigned)(lp * 16);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      unsigned t[WM];
#pragma unroll
      for (int m = 0; m < WM; ++m) t[m] = va[h][m] - back;
      lds_dma_s<WM>(t, Xt + k0, sbase + h * WM * 4096);
    }
  };
  auto issue_b = [&](int it) {
    unsigned char* sbase = sm + (it % S) * kStage + kA + wave * 1024;
    const int64_t k0 = stage_k0(it);
    const unsigned back = k0 + lp * 8 < b ? 0u : (unsigned)(lp * 16);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      unsigned t[WN];
#pragma unroll
      for (int m = 0; m < WN; ++m) t[m] = vb[h][m] - back;
      lds_dma_s<WN>(t, Wt + k0, sbase + h * WN * 4096);
    }
  };
  // zero this wave's pieces of stage it that lie past b (its own loads have landed)
  auto zero_tail = [&](int it) {
    const int64_t k0 = (int64_t)(s_begin + it) * kLK;
    if (k0 + kLK <= b || k0 + lp * 8 < b) return;
    unsigned char* sbase = sm + (it % S) * kStage + wave * 1024 + lane * 16;
#pragma unroll
    for (int m = 0; m < 2 * WM; ++m) *(u32x4_t*)(sbase + m * 4096) = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
    for (int m = 0; m < 2 * WN; ++m) *(u32x4_t*)(sbase + kA + m * 4096) = u32x4_t{0u, 0u, 0u, 0u};
  };

  f32x16_t acc[WM][WN];
#pragma unroll
  for (int i = 0; i < WM; ++i)
#pragma unroll
    for (int j = 0; j < WN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
  const int r32 = lane & 31, half = lane >> 5;
  // operand address of a 32-row block: its row is a multiple of 32, so the swizzle is
  // the lane's own and a substep only XORs piece bits
  const int faddr = r32 * kLRow + ((half ^ ((r32 >> 1) & 7)) << 4);
  bf16x8_t a0[WM], b0[WN], a1[WM], b1[WN];
  auto read_frags = [&](int it, int sub, bf16x8_t (&a)[WM], bf16x8_t (&bb)[WN]) {
    const unsigned char* st = sm + (it % S) * kStage + (faddr ^ (sub << 5));
#pragma unroll
    for (int i = 0; i < WM; ++i) a[i] = *(const bf16x8_t*)(st + (wm * WM + i) * 32 * kLRow);
#pragma unroll
    for (int j = 0; j < WN; ++j) bb[j] = *(const bf16x8_t*)(st + kA + (wn * WN + j) * 32 * kLRow);
  };
  auto mfmas = [&](const bf16x8_t (&a)[WM], const bf16x8_t (&bb)[WN]) {
#pragma unroll
    for (int i = 0; i < WM; ++i)
#pragma unroll
      for (int j = 0; j < WN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], bb[j], acc[i][j], 0, 0, 0);
  };
  // all but the newest S - 2 stages of this wave's loads have landed
  auto wait_loads = [&] {
    constexpr int left = (S - 2) * 2 * (WM + WN);
    static_assert(left == 0 || left == 8 || left == 16, "vmcnt immediates");
    if constexpr (left == 0)
      __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
    else if constexpr (left == 8)
      __asm__ volatile("s_waitcnt vmcnt(8)" ::: "memory");
    else
      __asm__ volatile("s_waitcnt vmcnt(16)" ::: "memory");
  };

#pragma unroll
  for (int it = 0; it < S - 1; ++it) {
    issue_a(it);
    issue_b(it);
  }
  wait_loads();
  zero_tail(0);
  __syncthreads();
  read_frags(0, 0, a0, b0);
  for (int it = 0; it < nk; ++it) {
    issue_a(it + S - 1);  // its buffer was last read before the barrier of it-1
    read_frags(it, 1, a1, b1);
    mfmas(a0, b0);
    issue_b(it + S - 1);
    read_frags(it, 2, a0, b0);
    mfmas(a1, b1);
    read_frags(it, 3, a1, b1);
    mfmas(a0, b0);
    wait_loads();
    zero_tail(it + 1);
    __syncthreads();
    read_frags(it + 1, 0, a0, b0);
    mfmas(a1, b1);
  }
  __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();  // every wave's loads have landed: the stages may be reused

  // Epilogue through LDS, one 32-token strip of the wave's block at a time: the lane
  // holds channel r32 of each 32 x 32 block and tokens 8 (e / 4) + 4 half + (e % 4);
  // read back, a lane has 8 consecutive channels of one token. The row pitch puts
  // the two halves of a write 128 bytes apart in the banks.
  constexpr int kCols = 32 * WN, kPitch = kCols + 8;
  static_assert(4 * 32 * kPitch * 4 <= S * kStage, "strips fit the stages");
  float* strip = (float*)sm + wave * 32 * kPitch;
  constexpr int kLanes = kCols / 8;      // lanes per token
  constexpr int kTok = 64 / kLanes;      // tokens per pass
  const int64_t cp = (c + 7) & ~(int64_t)7;
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
        if (part) {
          f32x4_t* o = (f32x4_t*)(part + ((int64_t)blockIdx.y * n + t) * cp + q);
          o[0] = lo;
          o[1] = hi;
        } else {
          float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
          finish8(v, t, q, c - q < 8 ? (int)(c - q) : 8, ep);
        }
      }
    }
    wave_sync();
  }
}

// Sum of the splits' raw products in order, then the epilogue: 8 channels per thread.
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
  finish8(v, t, q, c - q < 8 ? (int)(c - q) : 8, ep);
}

// Skinny products, n <= 16 NT tokens: bound by reading W once. A workgroup takes 16
// channels, its eight waves an eighth of the contraction each; W goes straight from
// memory into the operands of v_mfma_f32_16x16x32_bf16 (W as the first one: lane l
// holds channel l % 16, k = 8 (l / 16) .. + 7), 8 steps of 1 KB in flight per wave, X
// comes from L2. The waves' sums meet in LDS and are added in the order of the waves.
constexpr int kSkWaves = 8;
constexpr int kSkSteps = 8;

template <int NT>
__global__ __launch_bounds__(64 * kSkWaves) void linear_skinny_kernel(
    const unsigned short* __restrict__ X, int64_t ldx, const unsigned short* __restrict__ W, int n,
    int64_t b, int64_t c, LinEpilogue ep) {
  __shared__ float red[kSkWaves][16 * NT][17];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r16 = lane & 15, kq = (lane >> 4) * 8;
  const int64_t f0 = (int64_t)blockIdx.x * 16;
  const int64_t fr = f0 + r16 < c ? f0 + r16 : c - 1;  // fills outputs that are not stored
  const unsigned short* wp = W + fr * b + kq;
  const unsigned short* xp[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int t = j * 16 + r16 < n ? j * 16 + r16 : n - 1;
    xp[j] = X + t * ldx + kq;
  }
  const int steps = (int)cdiv(b, 32), per = (int)cdiv(steps, kSkWaves);
  const int sb = wave * per, se = min(steps, sb + per);
  f32x4_t acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int s0 = sb; s0 < se; s0 += kSkSteps) {
    u32x4_t w[kSkSteps], x[kSkSteps][NT];
#pragma unroll
    for (int u = 0; u < kSkSteps; ++u) {
      const int64_t k = (int64_t)(s0 + u) * 32;
      const bool in = s0 + u < se && k + kq < b;
      const u32x4_t zero = u32x4_t{0u, 0u, 0u, 0u};
      w[u] = in ? __builtin_nontemporal_load((const u32x4_t*)(wp + k)) : zero;
#pragma unroll
      for (int j = 0; j < NT; ++j) x[u][j] = in ? *(const u32x4_t*)(xp[j] + k) : zero;
    }
#pragma unroll
    for (int u = 0; u < kSkSteps; ++u)
#pragma unroll
      for (int j = 0; j < NT; ++j)
        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w[u]),
                                                         __builtin_bit_cast(bf16x8_t, x[u][j]),
                                                         acc[j], 0, 0, 0);
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[wave][j * 16 + r16][(lane >> 4) * 4 + e] = acc[j][e];
  __syncthreads();
  for (int i = tid; i < 256 * NT; i += 64 * kSkWaves) {
    const int t = i >> 4, q = i & 15;
    if (t < n && f0 + q < c) {
      float v = red[0][t][q];
#pragma unroll
      for (int w = 1; w < kSkWaves; ++w) v += red[w][t][q];
      finish1(v, t, f0 + q, ep);
    }
  }
}

enum { kLinSkinny = 0, kLin64 = 1, kLin128 = 2, kLin256 = 4 };

struct LinPlan {
  int tile;    // one of the above
  int splits;  // pieces of the contraction
  int per;     // stages per piece
};

constexpr int kUnits = 256;  // compute units

LinPlan plan_of(int64_t n, int64_t b, int64_t c, bool can_split) {
  LinPlan p;
  p.per = (int)cdiv(b, kLK);
  p.splits = 1;
  if (n <= 64) {
    p.tile = kLinSkinny;
    return p;
  }
  const int64_t big = cdiv(n, 256) * cdiv(c, 256), mid = cdiv(n, 128) * cdiv(c, 128);
  p.tile = big >= kUnits ? kLin256 : (mid >= kUnits ? kLin128 : kLin64);
  const int64_t tiles = p.tile == kLin256 ? big : (p.tile == kLin128 ? mid : cdiv(n, 64) * cdiv(c, 64));
  const int64_t stages = p.per;
  if (can_split && tiles < kUnits) {
    int64_t splits = 2 * kUnits / tiles;
    if (splits > stages / 8) splits = stages / 8;
    if (splits < 1) splits = 1;
    p.per = (int)cdiv(stages, splits);
    p.splits = (int)cdiv(stages, p.per);
  }
  return p;
}

template <int WM, int WN, int S>
hipError_t launch_tiles(const unsigned short* X, int64_t ldx, const unsigned short* W, int64_t n,
                        int64_t b, int64_t c, const LinPlan& p, float* part, const LinEpilogue& ep,
                        hipStream_t s) {
  const int ntm = (int)cdiv(n, 64 * WM), ntn = (int)cdiv(c, 64 * WN);
  const int per_xcd = (int)cdiv((int64_t)ntm * ntn, 8);
  hipLaunchKernelGGL((linear_tile_kernel<WM, WN, S>),
                     dim3((unsigned)(8 * per_xcd), (unsigned)p.splits), dim3(kLThreads), 0, s, X,
                     ldx, W, n, b, c, ntm, ntn, per_xcd, p.per, part, ep);
  return hipGetLastError();
}

template <int NT>
hipError_t launch_skinny(const unsigned short* X, int64_t ldx, const unsigned short* W, int64_t n,
                         int64_t b, int64_t c, const LinEpilogue& ep, hipStream_t s) {
  hipLaunchKernelGGL((linear_skinny_kernel<NT>), dim3((unsigned)cdiv(c, 16)), dim3(64 * kSkWaves),
                     0, s, X, ldx, W, (int)n, b, c, ep);
  return hipGetLastError();
}

}  // namespace

size_t linear_workspace_floats(int64_t n, int64_t b, int64_t c) {
  const LinPlan p = plan_of(n, b, c, true);
  return p.splits > 1 ? (size_t)p.splits * (size_t)n * (size_t)(cdiv(c, 8) * 8) : 0;
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
  hipError_t e;
  switch (p.tile) {
    case kLinSkinny:
      e = n <= 16   ? launch_skinny<1>(X, ldx, W, n, b, c, ep, s)
          : n <= 32 ? launch_skinny<2>(X, ldx, W, n, b, c, ep, s)
                    : launch_skinny<4>(X, ldx, W, n, b, c, ep, s);
      break;
    case kLin64: e = launch_tiles<1, 1, 4>(X, ldx, W, n, b, c, p, raw, ep, s); break;
    case kLin128: e = launch_tiles<2, 2, 2>(X, ldx, W, n, b, c, p, raw, ep, s); break;
    default: e = launch_tiles<4, 4, 2>(X, ldx, W, n, b, c, p, raw, ep, s); break;
  }
  if (e != hipSuccess || !raw) return e;
  const int64_t items = n * cdiv(c, 8);
  hipLaunchKernelGGL(linear_join_kernel, dim3((unsigned)cdiv(items, 256)), dim3(256), 0, s, raw,
                     p.splits, n, c, ep);
  return hipGetLastError();
}

}  // namespace th
