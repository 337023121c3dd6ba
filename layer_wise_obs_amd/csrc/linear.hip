// Linear layer with its epilogue, Y = act(X W^T + bias) + residual: X token-major
// [n, b], W [c, b] (row = output channel) in bf16, products exact in fp32 on the
// matrix cores, fp32 sums, epilogue in fp32, Y (bf16 or fp32) rounded once.
//
// "Pruning LLMs with Thanos", section "The compression target: linear layers": the
// layers a block consists of; section "The layer-reconstruction lens": the input of
// a layer is what its pruned predecessors produce.
//
// Bound by the matrix cores at large n: tiles of (64 WM) tokens x (32 WN GN) channels
// on 2 x GN waves, each 32 WM x 32 WN of v_mfma_f32_16x16x32_bf16 blocks (by themselves,
// at this card's power limit, 1.88 PFLOP/s; the 32x32x16 form 1.69). The contraction
// is contiguous in both operands, so an MFMA operand (8 consecutive k of a row per
// lane) is one 16-byte LDS read. Stages of 64 k (128-byte rows, whole cache lines) are
// filled by direct global->LDS loads, SA stages of X and SB of W deep; the 16-byte
// pieces of a row are XOR-swizzled by (row / 2) & 7, so the operand reads (16 rows at
// one piece per 16 lanes) use all 64 banks. Fragments are double-buffered over the two
// 32-wide substeps of a stage. Tiles are walked in groups of 4 token tiles per channel
// tile, each XCD a contiguous range of that order, so that the workgroups of an XCD
// share X and W slices in its L2. 131072 tokens 4096 -> 4096: 3.33 ms (1319 TFLOP/s),
// 3.39-3.48 with a bf16 residual (66% of the cycles in products, 7.5 GB read past the L2s).
#include "common.h"
#include "lds_dma.h"
#include "linear_epilogue.h"

namespace th {

namespace {

constexpr int kLK = 64;  // contraction per stage
constexpr int kLGroup = 4;  // token tiles per group in the walk order
constexpr int kLRow = kLK * 2;

// Workgroup (x, split): tile x of the walk order, stages [split per, split per + per)
// of the contraction. With part set, the tile's raw sums go to part[split][n][cp], cp
// being c rounded up to 8.
template <int WM, int WN, int GN, int SA, int SB>
__global__ __launch_bounds__(128 * GN) void linear_tile_kernel(
    const unsigned short* __restrict__ X, int64_t ldx, const unsigned short* __restrict__ W,
    int64_t n, int64_t b, int64_t c, int ntm, int ntn, int per_xcd, int stages_per_split,
    float* __restrict__ part, LinEpilogue ep) {
  constexpr int TM = 64 * WM, TN = 32 * WN * GN;
  constexpr int kWaves = 2 * GN;
  constexpr int FM = 2 * WM, FN = 2 * WN;  // 16 x 16 blocks of a wave
  constexpr int LA = TM / 8 / kWaves, LB = TN / 8 / kWaves;  // 1 KB loads per wave and stage
  constexpr int kA = TM * kLRow, kB = TN * kLRow;  // one stage of either operand
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

  __shared__ __attribute__((aligned(1024))) unsigned char sm[SA * kA + SB * kB];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / GN, wn = wave % GN;
  const unsigned smb = lds_address(sm);

  // Loader: chunks of 1 KB (8 rows of 128 bytes); wave w loads chunks
  // w + kWaves m of either operand. Lane l fills row 8 chunk + l/8 at physical piece
  // l%8; (row / 2) & 7 is the same in each of its chunks.
  const int lrow = lane >> 3;
  const int lp = (lane & 7) ^ (((wave & 1) << 2) + (lane >> 4));
  unsigned va[LA], vb[LB];
#pragma unroll
  for (int m = 0; m < LA; ++m) {
    int64_t r = M0 + (wave + kWaves * m) * 8 + lrow;
    r = r < n ? r : n - 1;  // rows past the end feed outputs that are never stored
    va[m] = (unsigned)(((r - M0) * ldx + lp * 8) * 2);
  }
#pragma unroll
  for (int m = 0; m < LB; ++m) {
    int64_t r = N0 + (wave + kWaves * m) * 8 + lrow;
    r = r < c ? r : c - 1;
    vb[m] = (unsigned)(((r - N0) * b + lp * 8) * 2);
  }
  // Stages past the last are loaded too (never read), so that every stage has the same
  // number of loads for the vmcnt waits; they re-read the last. Pieces of the last
  // stage past b re-read its piece 0; zero_tail clears them.
  const int st_last = nk_all - 1;
  const bool past = (int64_t)st_last * kLK + lp * 8 >= b;
  const unsigned short *xs, *ws;  // the stages being issued
  unsigned abase = 0, bbase = 0;
  bool a_last = false, b_last = false;
  auto stage_a = [&](int it) {
    const int st = s_begin + it;
    xs = X + M0 * ldx + (int64_t)(st < st_last ? st : st_last) * kLK;
    abase = smb + (it % SA) * kA + wave * 1024;
    if (st >= st_last && !a_last) {  // from here on every stage issued is the last one
      a_last = true;
      if (past) {
#pragma unroll
        for (int m = 0; m < LA; ++m) va[m] -= lp * 16;
      }
    }
  };
  auto stage_b = [&](int it) {
    const int st = s_begin + it;
    ws = W + N0 * b + (int64_t)(st < st_last ? st : st_last) * kLK;
    bbase = smb + SA * kA + (it % SB) * kB + wave * 1024;
    if (st >= st_last && !b_last) {
      b_last = true;
      if (past) {
#pragma unroll
        for (int m = 0; m < LB; ++m) vb[m] -= lp * 16;
      }
    }
  };
  auto issue_a = [&](int m) { lds_dma1(va[m], xs, abase + m * kWaves * 1024); };
  auto issue_b = [&](int m) { lds_dma1(vb[m], ws, bbase + m * kWaves * 1024); };
  // zero this wave's pieces of stage it that lie past b (its own loads have landed)
  auto zero_tail = [&](int it) {
    const int64_t k0 = (int64_t)(s_begin + it) * kLK;
    if (k0 + kLK <= b || k0 + lp * 8 < b) return;
    unsigned char* za = sm + (it % SA) * kA + wave * 1024 + lane * 16;
    unsigned char* zb = sm + SA * kA + (it % SB) * kB + wave * 1024 + lane * 16;
#pragma unroll
    for (int m = 0; m < LA; ++m) *(u32x4_t*)(za + m * kWaves * 1024) = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
    for (int m = 0; m < LB; ++m) *(u32x4_t*)(zb + m * kWaves * 1024) = u32x4_t{0u, 0u, 0u, 0u};
  };

  f32x4_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int r16 = lane & 15, quad = lane >> 4;
  // operand address of a 16-row block: its row is a multiple of 16, so the swizzle is
  // the lane's own and a substep only XORs a piece bit
  const int faddr = r16 * kLRow + ((quad ^ ((r16 >> 1) & 7)) << 4);
  bf16x8_t a0[FM], b0[FN], a1[FM], b1[FN];
  // operand y of a substep: the FN blocks of W, then the FM of X
  auto read_one = [&](int it, int sub, int y, bf16x8_t (&a)[FM], bf16x8_t (&bb)[FN]) {
    if (y < FN)
      bb[y] = *(const bf16x8_t*)(sm + SA * kA + (it % SB) * kB + (faddr ^ (sub << 6)) +
                                 (wn * FN + y) * 16 * kLRow);
    else
      a[y - FN] = *(const bf16x8_t*)(sm + (it % SA) * kA + (faddr ^ (sub << 6)) +
                                     (wm * FM + y - FN) * 16 * kLRow);
  };
  // One substep's products, with the next substep's operand reads (of stage it2, substep
  // sub2) and a coming stage's loads between them. The order is pinned, products first:
  // after a barrier the matrix cores start at once.
  auto mfmas = [&](const bf16x8_t (&a)[FM], const bf16x8_t (&bb)[FN], int it2, int sub2,
                   bf16x8_t (&a2)[FM], bf16x8_t (&b2)[FN], auto&& load) {
    constexpr int per = (FM + FN + FM * FN - 1) / (FM * FN);  // reads after a product
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int x = 0; x < FM * FN; ++x) {
      const int i = x / FN, j = x % FN;
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], bb[j], acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int y = 0; y < per; ++y)
        if (x * per + y < FM + FN) read_one(it2, sub2, x * per + y, a2, b2);
      load(x);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // the loads of one operand's stage, spread evenly over a substep's products
  auto loads_a = [&](int x) {
    constexpr int gap = FM * FN / LA > 0 ? FM * FN / LA : 1, per = (LA + FM * FN - 1) / (FM * FN);
    if (x % gap == 0) {
#pragma unroll
      for (int m = 0; m < per; ++m)
        if (x / gap * per + m < LA) issue_a(x / gap * per + m);
    }
  };
  auto loads_b = [&](int x) {
    constexpr int gap = FM * FN / LB > 0 ? FM * FN / LB : 1, per = (LB + FM * FN - 1) / (FM * FN);
    if (x % gap == 0) {
#pragma unroll
      for (int m = 0; m < per; ++m)
        if (x / gap * per + m < LB) issue_b(x / gap * per + m);
    }
  };
  // Order of the loads: A(SA-1), B(SB), A(SA), B(SB+1), ... At the wait of stage it, A
  // and B of stage it + 1 have to have landed; newer are A(it + 2) .. A(it + SA - 1) and
  // B(it + 2) .. B(it + SB - 1).
  auto wait_loads = [&] {
    constexpr int left = (SA - 2) * LA + (SB - 2) * LB;
    static_assert(left == 4 || left == 6 || left == 8, "vmcnt immediates");
    if constexpr (left == 4)
      __asm__ volatile("s_waitcnt vmcnt(4)" ::: "memory");
    else if constexpr (left == 6)
      __asm__ volatile("s_waitcnt vmcnt(6)" ::: "memory");
    else
      __asm__ volatile("s_waitcnt vmcnt(8)" ::: "memory");
  };

  // prologue: B's stages 0 .. SB-2, A's 0 .. SA-2, waited for; then B(SB-1)
#pragma unroll
  for (int it = 0; it < SB - 1; ++it) {
    stage_b(it);
#pragma unroll
    for (int m = 0; m < LB; ++m) issue_b(m);
  }
#pragma unroll
  for (int it = 0; it < SA - 1; ++it) {
    stage_a(it);
#pragma unroll
    for (int m = 0; m < LA; ++m) issue_a(m);
  }
  __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
  zero_tail(0);
  __syncthreads();
  stage_b(SB - 1);
#pragma unroll
  for (int m = 0; m < LB; ++m) issue_b(m);
#pragma unroll
  for (int y = 0; y < FM + FN; ++y) read_one(0, 0, y, a0, b0);
  // A stage: half its products, then (its last operands read, the next stage landed,
  // the barrier) the other half. A's next stage goes into the buffer freed by the
  // barrier of stage it - 1 during the first half, B's into the one freed by this
  // stage's barrier during the second: a quarter of the address unit's rate, where all
  // loads in one half would take half of it in bursts.
  for (int it = 0; it < nk; ++it) {
    stage_a(it + SA - 1);
    mfmas(a0, b0, it, 1, a1, b1, loads_a);
    wait_loads();
    zero_tail(it + 1);
    __syncthreads();
    stage_b(it + SB);
    mfmas(a1, b1, it + 1, 0, a0, b0, loads_b);
  }
  __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();  // every wave's loads have landed: the stages may be reused

  // Epilogue through LDS, one 32-token strip of the wave's block at a time: the lane
  // holds channel l % 16 of each 16 x 16 block and tokens 4 (l / 16) + e; read back, a
  // lane has 8 consecutive channels of one token. The row pitch puts the four quarters
  // of a write 64 bytes apart in the banks.
  constexpr int kCols = 32 * WN, kPitch = kCols + 4;
  static_assert(kWaves * 32 * kPitch * 4 <= SA * kA + SB * kB, "strips fit the stages");
  float* strip = (float*)sm + wave * 32 * kPitch;
  constexpr int kLanes = kCols / 8;   // lanes per token
  constexpr int kTok = 64 / kLanes;   // tokens per pass
  constexpr int kPass = 32 / kTok;
  const int64_t cp = (c + 7) & ~(int64_t)7;
  const int tl = lane / kLanes, ql = (lane % kLanes) * 8;
  const int64_t q = N0 + wn * kCols + ql;
  auto token = [&](int i, int p) { return M0 + wm * 32 * WM + i * 32 + p * kTok + tl; };
  auto values = [&](int p) { return strip + (p * kTok + tl) * kPitch + ql; };
  auto write_strip = [&](int i) {
#pragma unroll
    for (int i2 = 0; i2 < 2; ++i2)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          strip[(i2 * 16 + quad * 4 + e) * kPitch + j * 16 + r16] = acc[2 * i + i2][j][e];
    wave_sync();
  };
  if (part) {
#pragma unroll
    for (int i = 0; i < WM; ++i) {
      write_strip(i);
#pragma unroll 1
      for (int p = 0; p < kPass; ++p) {
        if (token(i, p) < n && q < c) {
          const f32x4_t* v = (const f32x4_t*)values(p);
          f32x4_t* o = (f32x4_t*)(part + ((int64_t)blockIdx.y * n + token(i, p)) * cp + q);
          o[0] = v[0];
          o[1] = v[1];
        }
      }
      wave_sync();
    }
    return;
  }
  finish_tile<WM, kPass>(ep, n, c, q, token, values, write_strip);
}

// Skinny products, up to 16 tokens: bound by reading W once. A workgroup takes 16
// channels, its eight waves an eighth of the contraction each; W goes straight from
// memory into the operands of v_mfma_f32_16x16x32_bf16 (W as the first one: lane l
// holds channel l % 16, k = 8 (l / 16) .. + 7), kSkSteps steps of 1 KB in flight per
// wave, X comes from L2. The waves' sums meet in LDS and are added in the order of the
// waves. Workgroup x takes the channels from 16 (first + x). In a graph 7.2 us for one
// token 4096 -> 4096 (4.7 TB/s), 84 us for four 8192 -> 28672 (5.6 TB/s; nontemporal
// loads of W took a fifth longer). Few channels are few workgroups: one token
// 8192 -> 1024 takes 10.8 us (1.6 TB/s).
constexpr int kSkWaves = 8;
constexpr int kSkSteps = 8;

__global__ __launch_bounds__(64 * kSkWaves) void linear_skinny_kernel(
    const unsigned short* __restrict__ X, int64_t ldx, const unsigned short* __restrict__ W, int n,
    int64_t b, int64_t c, int64_t first, LinEpilogue ep) {
  __shared__ float red[kSkWaves][16][17];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r16 = lane & 15, kq = (lane >> 4) * 8;
  const int64_t f0 = (first + blockIdx.x) * 16;
  const int64_t fr = f0 + r16 < c ? f0 + r16 : c - 1;  // fills outputs that are not stored
  const unsigned short* wp = W + fr * b + kq;
  const unsigned short* xp = X + (r16 < n ? r16 : n - 1) * ldx + kq;
  const int steps = (int)cdiv(b, 32), per = (int)cdiv(steps, kSkWaves);
  const int sb = wave * per, se = min(steps, sb + per);
  f32x4_t acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int s0 = sb; s0 < se; s0 += kSkSteps) {
    u32x4_t w[kSkSteps], x[kSkSteps];
#pragma unroll
    for (int u = 0; u < kSkSteps; ++u) {
      const int64_t k = (int64_t)(s0 + u) * 32;
      const bool in = s0 + u < se && k + kq < b;
      const u32x4_t zero = u32x4_t{0u, 0u, 0u, 0u};
      w[u] = in ? *(const u32x4_t*)(wp + k) : zero;
      x[u] = in ? *(const u32x4_t*)(xp + k) : zero;
    }
#pragma unroll
    for (int u = 0; u < kSkSteps; ++u)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w[u]),
                                                    __builtin_bit_cast(bf16x8_t, x[u]), acc, 0, 0, 0);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) red[wave][r16][(lane >> 4) * 4 + e] = acc[e];
  __syncthreads();
  const int t = tid >> 4, q = tid & 15;
  if (t < n && f0 + q < c) {  // n <= 16
    float v = red[0][t][q];
#pragma unroll
    for (int w = 1; w < kSkWaves; ++w) v += red[w][t][q];
    finish1(v, t, f0 + q, ep);
  }
}

// The tile kernel's forms. Its time is modelled as rounds of `slots` workgroups, each
// taking fixed + stages * per_stage microseconds with every slot taken and half of the
// second part with few, and the join of splits as 3 us and its traffic at 4 TB/s. Measured
// in a graph, and modelled: 777 x 4096 -> 11008 on 172 tiles of 256 x 256 82-85 us, 96;
// 1024 x 4096 -> 4096 on 256 of 128 x 128 37-38, 41; 2048 x 4096 -> 4096 on 256 of
// 128 x 256 65-67, 66; 777 x 2056 -> 1023 on 208 of 64 x 64 14, 16. The cheapest form is
// taken: over 22 shapes of 13 tokens and more it came within 8% of the best of all forms
// and numbers of pieces, but for 256 x 4096 -> 4096 (11%: 22.2 us in pieces of 64 x 64
// tiles, 20.0 whole) and 64 x 4096 -> 11008 (17%: 22.4 on 128 x 128, 19.1 on 64 x 64).
struct LinTile {
  int tm, tn;
  int slots;  // workgroups that run at a time
  double per_stage, fixed;
};
enum { kLin64 = 0, kLin128 = 1, kLin128x256 = 2, kLin256 = 3, kLinTiles = 4, kLinSkinny = 4 };
constexpr LinTile kTiles[kLinTiles] = {
    {64, 64, 512, 0.53, 4.0},     // 4 waves of 32 x 32, two workgroups per compute unit
    {128, 128, 256, 0.55, 6.0},   // 8 waves of 64 x 32
    {128, 256, 256, 0.93, 7.0},   // 8 waves of 64 x 64
    {256, 256, 256, 1.54, 14.0},  // 8 waves of 128 x 64
};
// Up to 12 tokens the skinny kernel is ahead for thousands of channels (4096 -> 4096: 7.4 us
// for one token against 9.5 on tiles, 9.5 against 10.0 for twelve; 11008 -> 4096 20.9 against
// 19.8 for twelve). With few channels it is not: 12 tokens 8192 -> 1024 take 15.0 us, on 64 x 64
// tiles in sixteen pieces 9.3.
constexpr int64_t kSkinny = 12;

struct LinPlan {
  int tile;    // one of the above
  int splits;  // pieces of the contraction
  int per;     // stages per piece
};

LinPlan plan_of(int64_t n, int64_t b, int64_t c, bool can_split) {
  const int64_t stages = cdiv(b, kLK);
  LinPlan best = {kLinSkinny, 1, (int)stages};
  if (n <= kSkinny) return best;
  double least = 1e300;
  for (int t = 0; t < kLinTiles; ++t) {
    const LinTile& k = kTiles[t];
    const int64_t tiles = cdiv(n, k.tm) * cdiv(c, k.tn);
    for (int64_t want : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (want > 1 && (!can_split || stages < 2 * want || tiles * want > 4 * k.slots)) break;
      const int64_t per = cdiv(stages, want), splits = cdiv(stages, per);
      const int64_t full = tiles * splits / k.slots, rest = tiles * splits % k.slots;
      double us = (double)full * (k.fixed + (double)per * k.per_stage);
      if (rest)
        us += k.fixed + (double)per * k.per_stage * (0.5 + 0.5 * (double)rest / k.slots);
      if (splits > 1) us += 3.0 + 8.0 * (double)splits * (double)n * (double)c / 4e6;
      if (us < least) {
        least = us;
        best = {t, (int)splits, (int)per};
      }
    }
  }
  return best;
}

template <int WM, int WN, int GN, int SA, int SB>
hipError_t launch_tiles(const unsigned short* X, int64_t ldx, const unsigned short* W, int64_t n,
                        int64_t b, int64_t c, const LinPlan& p, float* part, const LinEpilogue& ep,
                        hipStream_t s) {
  const int ntm = (int)cdiv(n, 64 * WM), ntn = (int)cdiv(c, 32 * WN * GN);
  const int per_xcd = (int)cdiv((int64_t)ntm * ntn, 8);
  hipLaunchKernelGGL((linear_tile_kernel<WM, WN, GN, SA, SB>),
                     dim3((unsigned)(8 * per_xcd), (unsigned)p.splits), dim3(128 * GN), 0, s, X,
                     ldx, W, n, b, c, ntm, ntn, per_xcd, p.per, part, ep);
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
  ep.past_cache = 0;
  const LinPlan p = plan_of(n, b, c, part != nullptr);
  float* raw = p.splits > 1 ? part : nullptr;
  hipError_t e;
  switch (p.tile) {
    case kLinSkinny: {
      // a launch has less than 2^32 threads, 512 to a workgroup
      const int64_t groups = cdiv(c, 16), most = (int64_t)1 << 22;
      for (int64_t first = 0; first < groups; first += most)
        hipLaunchKernelGGL(linear_skinny_kernel,
                           dim3((unsigned)(groups - first < most ? groups - first : most)),
                           dim3(64 * kSkWaves), 0, s, X, ldx, W, (int)n, b, c, first, ep);
      e = hipGetLastError();
      break;
    }
    case kLin64: e = launch_tiles<1, 1, 2, 4, 4>(X, ldx, W, n, b, c, p, raw, ep, s); break;
    case kLin128: e = launch_tiles<2, 1, 4, 4, 4>(X, ldx, W, n, b, c, p, raw, ep, s); break;
    case kLin128x256: e = launch_tiles<2, 2, 4, 3, 3>(X, ldx, W, n, b, c, p, raw, ep, s); break;
    default: e = launch_tiles<4, 2, 4, 3, 2>(X, ldx, W, n, b, c, p, raw, ep, s); break;
  }
  if (e != hipSuccess || !raw) return e;
  const int64_t items = n * cdiv(c, 8);
  hipLaunchKernelGGL(linear_join_kernel<false>, dim3((unsigned)cdiv(items, 256)), dim3(256), 0, s, raw,
                     p.splits, n, c, ep);
  return hipGetLastError();
}

}  // namespace th
