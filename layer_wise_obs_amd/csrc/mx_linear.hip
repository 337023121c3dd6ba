// Linear layer on microscaled operands, Y = act(X W^T + bias) + residual: X [n, b] of e4m3 or
// e2m1, W [c, b] of e2m1, 32 consecutive k of a row sharing a power of two; fp32 sums, epilogue
// in fp32, Y (bf16 or fp32) rounded once. A pruned block's layers as they are served
// ("Pruning LLMs with Thanos", section "The compression target: linear layers").
//
// The matrix cores take both types and the scales: v_mfma_scale_f32_32x32x64_f8f6f4, whose
// lane holds 32 k of a row and their scale. By themselves, at this card's power limit, such
// products reach 4.4 PFLOP/s with an e4m3 X and 7.3 with an e2m1 one (in the 16x16x128 form
// 4.0 and 6.0). An operand's lane l holds row l % 32 and, of 64 k, of 4-bit elements k 32 (l / 32)
// .. + 31, of 8-bit ones k 16 (l / 32) .. + 15 and 32 further on; its scale is that of k block
// l / 32 either way.
//
// What the products add up: with an e2m1 X every sum of a step is exact to fp32. 8-bit
// elements span 2^-9 .. 2^8.8, and the cores align the products of eight consecutive k to the
// largest of them, dropping what is 13 places below it (measured with single products; over
// normal X and W 4.9e-6 of Y in root mean square). Rounding Y to bf16 costs 300 times that,
// so with a bf16 Y it stands. Where Y is fp32 (EXACT), and where the products cost nothing
// (few tokens), X enters in two parts, elements of 2 and more and the smaller ones (a bit of
// the byte tells): either part's products lie within 13 places, and two products give
// fp32's sum.
//
// A workgroup takes (32 FM GM) tokens x (32 FN GN) channels on GM x GN waves, each 32 FM x 32 FN,
// times KS: few tiles of 64 x 64 get twice the waves, which halve a step's k between them (777
// tokens 2080 -> 1023 with e4m3 and an fp32 Y 14.1 -> 11.7 us, 256 tokens 4096 -> 4096 20.8 ->
// 16.3; with e4m3 and a bf16 Y there is nothing to gain). Steps are of 256 k: a row of 4 bits is
// then one cache line of 128 bytes (with 64 bytes of a row at a time 872 us where this takes 840),
// one of 8 bits two, in halves. Direct global->LDS loads fill RX steps of X and RW of W; 16-byte
// pieces of a row are XOR-swizzled so that operand reads use all banks. Scales come 16 bytes
// (512 k) of a row at a time, two such every fourth step, into four slots of their own. But for
// them a step has no branch: behind one the compiler moved products, past the barrier (947 us).
// Operand reads and the next steps' loads stand between the products.
//
// Large products are bound by power: 32768 tokens 4096 -> 11008 with both of 4 bits take 810-890 us
// by card (3.6-3.3 PFLOP/s), at 1.5 GHz with the matrix cores half busy, and 1.96 GHz with the
// loads into LDS left out; with an e4m3 X and a bf16 Y 1085, with an fp32 Y 1960; 8192 tokens
// 11008 -> 4096 173, 244 and 444. Of 840 us the epilogue is 111, the stores of Y 62 of it. Waves
// of 64 x 128, eight to a tile: of 128 x 64 the same for 4 bits, 2234 against 2022 for the fp32 Y;
// four waves of 128 x 128 892 against 839.
#include "common.h"
#include "lds_dma.h"
#include "linear_epilogue.h"
#include "mx.h"

namespace th {

namespace {

constexpr int kMK = 256;         // contraction per step: whole cache lines of 4-bit rows
constexpr int kMScaleSlots = 4;  // buffers of 16 bytes (512 k) of scales a row
// Token tiles per group in the walk order: 32768 tokens 4096 -> 11008 in groups of 2, 4, 8, 16
// 853, 838, 878 and 901 us.
constexpr int kMGroup = 4;

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

struct MxOperand {
  const unsigned char *elements, *scales;
  int64_t ld, lds;
};

// Operand registers of 32 k of a row.
template <int TYPE>
struct MxFrag {
  i32x8_t v;
  __device__ __forceinline__ const i32x8_t& wide() const { return v; }
};
template <>
struct MxFrag<TH_MX_E2M1> {
  i32x4_t v;
  __device__ __forceinline__ i32x8_t wide() const {
    return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
  }
};

// The format codes of the instruction.
template <int TYPE>
constexpr int kMxCode = TYPE == TH_MX_E4M3 ? 0 : 4;

// The e4m3 elements of v of 2 and more (their exponent's first bit is set), the rest 0; and the
// others.
__device__ __forceinline__ void mx_part(const i32x8_t& v, i32x8_t& high, i32x8_t& low) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const unsigned u = (unsigned)v[i];
    // selectors 12 and 13 stand for bytes of zeros and of ones
    const unsigned mask = __builtin_amdgcn_perm(0u, 0u, ((u >> 6) & 0x01010101u) | 0x0c0c0c0cu);
    high[i] = (int)(u & mask);
    low[i] = (int)(u & ~mask);
  }
}

template <int XT, int FM, int FN, int GM, int GN, int KS, int RX, int RW, bool EXACT>
__global__ __launch_bounds__(64 * GM * GN * KS, 1) void mx_tile_kernel(MxOperand X, MxOperand W, int64_t n,
                                                                  int64_t b, int64_t c, int ntm, int ntn,
                                                                  int per_xcd, int steps_per_split,
                                                                  float* __restrict__ part,
                                                                  LinEpilogue ep) {
  constexpr bool kWide = XT == TH_MX_E4M3;  // X's rows of a step are two stages of 128 bytes
  constexpr int TM = 32 * FM * GM, TN = 32 * FN * GN;
  constexpr int kWaves = GM * GN * KS;
  constexpr int kXStage = TM * 128, kWStage = TN * 128;
  constexpr int kHalves = kWide ? 2 : 1;
  constexpr int kWAt = RX * kHalves * kXStage, kSAt = kWAt + RW * kWStage;  // in LDS
  constexpr int LX = TM / 8 / kWaves, LW = TN / 8 / kWaves;  // 1 KB loads per wave and stage
  constexpr int kScales = (TM + TN) * 16;                    // of 512 k
  constexpr int kLds = kSAt + kMScaleSlots * kScales;
  const int wg = blockIdx.x;
  const int lin = (wg % 8) * per_xcd + wg / 8;
  if (lin >= ntm * ntn) return;
  int tm, tn;
  {
    const int per_group = kMGroup * ntn;
    const int g = lin / per_group, in = lin - g * per_group;
    const int gs = min(kMGroup, ntm - g * kMGroup);
    tm = g * kMGroup + in % gs;
    tn = in / gs;
  }
  const int64_t M0 = (int64_t)tm * TM, N0 = (int64_t)tn * TN;
  const int steps = (int)cdiv(b, kMK);
  const int s_begin = blockIdx.y * steps_per_split;  // even
  const int nk = min(steps_per_split, steps - s_begin);
  if (nk <= 0) return;  // no split of the launch is empty

  __shared__ __attribute__((aligned(1024))) unsigned char sm[kLds];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kg = KS > 1 ? wave / (GM * GN) : 0;  // the wave's half of a step
  const int wm = wave % (GM * GN) / GN, wn = wave % GN;
  const unsigned smb = lds_address(sm);

  // Loader: chunks of 1 KB (8 rows of 128 bytes), wave w those w + kWaves m of either operand. Lane
  // l fills row 8 chunk + l / 8 at physical piece l % 8; (row / 2) & 7 is the same in each of its
  // chunks.
  const int lp = (lane & 7) ^ (((wave & 1) << 2) + (lane >> 4));
  unsigned vx[LX], vw[LW];
#pragma unroll
  for (int m = 0; m < LX; ++m) {
    int64_t r = M0 + (wave + kWaves * m) * 8 + (lane >> 3);
    r = r < n ? r : n - 1;  // rows past the end feed outputs that are never stored
    vx[m] = (unsigned)((r - M0) * X.ld + lp * 16);
  }
#pragma unroll
  for (int m = 0; m < LW; ++m) {
    int64_t r = N0 + (wave + kWaves * m) * 8 + (lane >> 3);
    r = r < c ? r : c - 1;
    vw[m] = (unsigned)((r - N0) * W.ld + lp * 16);
  }
  // Scales: 64 rows a load, X's rows first; a wave has those w + kWaves m, of X all or none.
  constexpr int kScaleLoads = (TM + TN) / 64, LS = (kScaleLoads + kWaves - 1) / kWaves;
  static_assert(LS == 1 || TM / 64 % kWaves == 0, "a load's rows are of one operand");
  unsigned vs[LS];
  const unsigned char* scale_base[LS];
#pragma unroll
  for (int m = 0; m < LS; ++m) {
    const int at = (wave + kWaves * m) * 64;
    const bool of_x = at < TM;
    int64_t r = of_x ? M0 + at + lane : N0 + at - TM + lane;
    const int64_t last = (of_x ? n : c) - 1;
    r = r < last ? r : last;
    vs[m] = (unsigned)(of_x ? (r - M0) * X.lds : (r - N0) * W.lds);
    scale_base[m] = of_x ? X.scales + M0 * X.lds : W.scales + N0 * W.lds;
  }
  const int super_last = (int)((b - 1) / 512);
  auto scale_slot = [&](int u) { return kSAt + u % kMScaleSlots * kScales; };
  auto load_scales = [&](int u) {  // those of steps 2 u and 2 u + 1
    const int64_t from = (int64_t)min(s_begin / 2 + u, super_last) * 16;
#pragma unroll
    for (int m = 0; m < LS; ++m)
      if (kWaves * (m + 1) <= kScaleLoads || wave + kWaves * m < kScaleLoads)
        lds_dma1(vs[m], scale_base[m] + from, smb + scale_slot(u) + (wave + kWaves * m) * 1024);
  };
  // Stages past the last are loaded too (never read), so that every step has the same number of
  // loads for the vmcnt waits; they re-read the last. Pieces of the last stage past b re-read
  // its piece 0. Loads of scales among them only make the waits stricter.
  const int x_last = (int)((b - 1) / (kMK / kHalves)), w_last = steps - 1;
  const unsigned x_back = (int64_t)x_last * (kMK / kHalves) + lp * (kWide ? 16 : 32) >= b ? lp * 16 : 0;
  const unsigned w_back = (int64_t)w_last * kMK + lp * 32 >= b ? lp * 16 : 0;
  const unsigned char *xs = X.elements, *ws = W.elements;
  unsigned xbase = 0, wbase = 0, x_cut = 0, w_cut = 0;
  auto stage_x = [&](int it, int half) {
    const int st = (s_begin + it) * kHalves + half;
    xs = X.elements + M0 * X.ld + (int64_t)min(st, x_last) * 128;
    xbase = smb + (it % RX * kHalves + half) * kXStage + wave * 1024;
    x_cut = st >= x_last ? x_back : 0;
  };
  auto stage_w = [&](int it) {
    const int st = s_begin + it;
    ws = W.elements + N0 * W.ld + (int64_t)min(st, w_last) * 128;
    wbase = smb + kWAt + it % RW * kWStage + wave * 1024;
    w_cut = st >= w_last ? w_back : 0;
  };
  auto issue_x = [&](int m) { lds_dma1(vx[m] - x_cut, xs, xbase + m * kWaves * 1024); };
  auto issue_w = [&](int m) { lds_dma1(vw[m] - w_cut, ws, wbase + m * kWaves * 1024); };
  // A load's 64 rows of scales, as they landed 16 bytes (512 k) of a row, are put in the order in
  // which the products want them, by the wave that loaded them: word 2 s + h of the rows one after
  // another, of a row the blocks 8 s + h, 2, 4 and 6 further on, that is the scales of half h of the
  // lanes in the four substeps of step s. (Read as they landed, a word of four blocks at a time,
  // 32 rows are in 8 banks: LDS is busy for 1.55 cycles where it is for one now. In time that is 1%
  // with an fp32 Y, and nothing where power is the limit.) Scales of blocks past b become 0 on either
  // side: whatever numbers the pieces re-read, their products are below 2^-242 and count nothing. (A
  // NaN among them is in its row already; as it is, such a scale might be 255.)
  auto arrange = [&](int u) {
    const int blocks = s_begin / 2 + u == super_last ? (int)(b / kMxBlock) - super_last * 16 : 16;
    for (int at = wave; at < kScaleLoads; at += kWaves) {
      unsigned char* chunk = sm + scale_slot(u) + at * 1024;
      u32x4_t z = *(const u32x4_t*)(chunk + lane * 16);
      if (blocks < 16) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int left = blocks - 4 * x;  // of this word's four
          if (left < 4) z[x] = left <= 0 ? 0u : z[x] & (0xffffffffu >> (32 - 8 * left));
        }
      }
      unsigned* to = (unsigned*)chunk + lane;
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        to[128 * st] = __builtin_amdgcn_perm(z[2 * st + 1], z[2 * st], 0x06040200u);
        to[128 * st + 64] = __builtin_amdgcn_perm(z[2 * st + 1], z[2 * st], 0x07050301u);
      }
    }
  };

  // the products of X's two parts have sums of their own where there are registers for them:
  // fewer wait for the one before
  constexpr bool kTwo = EXACT && kWide && FM * FN <= 2;
  f32x16_t acc[FM][FN], acc_low[kTwo ? FM : 1][kTwo ? FN : 1];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = acc_low[kTwo ? i : 0][kTwo ? j : 0][e] = 0.f;

  const int r32 = lane & 31, half = lane >> 5;
  const int faddr = r32 * 128 + ((half ^ ((r32 >> 1) & 7)) << 4);
  struct Frags {
    MxFrag<XT> a[FM];
    MxFrag<TH_MX_E2M1> b[FN];
  };
  Frags f0, f1;
  int sa[FM], sb[FN], sa_next[FM], sb_next[FN];  // scales of a step; byte x is substep x's
  // operand y of substep sub (64 k): the FN blocks of W, then the FM of X
  auto read_one = [&](int it, int sub, int y, Frags& f) __attribute__((always_inline)) {
    if (y < FN) {
      f.b[y].v = *(const i32x4_t*)(sm + kWAt + it % RW * kWStage + (wn * FN + y) * 4096 + (faddr ^ (sub << 5)));
    } else if constexpr (kWide) {
      const unsigned char* p = sm + (it % RX * 2 + sub / 2) * kXStage + (wm * FM + y - FN) * 4096;
      const i32x4_t lo = *(const i32x4_t*)(p + (faddr ^ (sub % 2 << 6)));
      const i32x4_t hi = *(const i32x4_t*)(p + (faddr ^ (sub % 2 << 6) ^ 32));
      f.a[y - FN].v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
      f.a[y - FN].v =
          *(const i32x4_t*)(sm + it % RX * kXStage + (wm * FM + y - FN) * 4096 + (faddr ^ (sub << 5)));
    }
  };
  auto read_scale = [&](int it, int y) {
    const unsigned char* p = sm + scale_slot(it / 2) + it % 2 * 512 + half * 256 + r32 * 4;
    const int row = y < FN ? TM + (wn * FN + y) * 32 : (wm * FM + y - FN) * 32;
    const int scale = *(const int*)(p + row / 64 * 1024 + row % 64 * 4);
    if (y < FN)
      sb_next[y] = scale;
    else
      sa_next[y - FN] = scale;
  };
  auto take_scales = [&](int shift) {
#pragma unroll
    for (int i = 0; i < FM; ++i) sa[i] = (int)((unsigned)sa_next[i] >> shift);
#pragma unroll
    for (int j = 0; j < FN; ++j) sb[j] = (int)((unsigned)sb_next[j] >> shift);
  };
  // One substep's products, with reads and loads between them; the order is pinned.
  auto products = [&](const Frags& f, auto SUB, auto&& between) __attribute__((always_inline)) {
    constexpr int byte = decltype(SUB)::value;
    auto product = [&](const i32x8_t& x, f32x16_t& to, int i, int j) __attribute__((always_inline)) {
      to = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          x, f.b[j].wide(), to, kMxCode<XT>, kMxCode<TH_MX_E2M1>, byte, sa[i], byte, sb[j]);
      __builtin_amdgcn_sched_barrier(0);
    };
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      if constexpr (EXACT && kWide) {
        i32x8_t high, low;
        mx_part(f.a[i].v, high, low);
#pragma unroll
        for (int j = 0; j < FN; ++j) product(low, kTwo ? acc_low[kTwo ? i : 0][kTwo ? j : 0] : acc[i][j], i, j);
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          product(high, acc[i][j], i, j);
          between(i * FN + j);
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          product(f.a[i].wide(), acc[i][j], i, j);
          between(i * FN + j);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  };
  constexpr int kProducts = FM * FN, kReads = (FM + FN + kProducts - 1) / kProducts;
  constexpr int kLoadsX = (LX + kProducts - 1) / kProducts, kLoadsW = (LW + kProducts - 1) / kProducts;
  constexpr int kGapX = kProducts / LX > 0 ? kProducts / LX : 1;
  constexpr int kGapW = kProducts / LW > 0 ? kProducts / LW : 1;
  auto reads = [&](int x, int it, int sub, Frags& f) __attribute__((always_inline)) {
#pragma unroll
    for (int y = 0; y < kReads; ++y)
      if (x * kReads + y < FM + FN) read_one(it, sub, x * kReads + y, f);
  };
  auto scales = [&](int x, int it) __attribute__((always_inline)) {
#pragma unroll
    for (int y = 0; y < kReads; ++y)
      if (x * kReads + y < FM + FN) read_scale(it, x * kReads + y);
  };
  auto loads_x = [&](int x) __attribute__((always_inline)) {
    if (x % kGapX == 0) {
#pragma unroll
      for (int m = 0; m < kLoadsX; ++m)
        if (x / kGapX * kLoadsX + m < LX) issue_x(x / kGapX * kLoadsX + m);
    }
  };
  auto loads_w = [&](int x) __attribute__((always_inline)) {
    if (x % kGapW == 0) {
#pragma unroll
      for (int m = 0; m < kLoadsW; ++m)
        if (x / kGapW * kLoadsW + m < LW) issue_w(x / kGapW * kLoadsW + m);
    }
  };
  // Loads not waited for before substep 3, where the next step's X (its first half) and W have to
  // have landed, and before substep 1, where this step's second half of X has to. They are issued
  // in the order: X (of 8 bits: its second half) of step it + RX in substep 3, W of it + RW in
  // the next step's substep 0, the first half of X of it + 1 + RX in its substep 1.
  constexpr int kStep = LX * kHalves + LW;
  constexpr int kLeft3 = kWide ? (RX == 1 ? 0 : LX + (RW - 2) * kStep) : (RW - 2) * kStep;
  constexpr int kLeft1 = LW + (RX - 1) * kStep;
  static_assert(RX == RW || (kWide && RX == 1 && RW == 2), "the order of the loads");
  static_assert(kLeft3 < 64 && kLeft1 < 64, "vmcnt immediates");

  if constexpr (KS == 1) {
    // prologue: the first scales, then steps 0 .. R-1 but for the last W, step 0 waited for
    load_scales(0);
    load_scales(1);
#pragma unroll
    for (int it = 0; it < RW; ++it) {
      if (it < RX) {
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
          stage_x(it, h);
#pragma unroll
          for (int m = 0; m < LX; ++m) issue_x(m);
        }
      }
      if (it < RW - 1) {
        stage_w(it);
#pragma unroll
        for (int m = 0; m < LW; ++m) issue_w(m);
      }
    }
    __asm__ volatile("s_waitcnt vmcnt(%0)" ::"n"((RW - 2) * LW + (RX - 1) * LX * kHalves) : "memory");
    arrange(0);
    arrange(1);
    __syncthreads();
#pragma unroll
    for (int y = 0; y < FM + FN; ++y) {
      read_one(0, 0, y, f0);
      read_scale(0, y);
    }
    // A step of 256 k: four substeps, each reading the next one's operands. Before the last one the
    // next step has landed, and the barrier frees this step's buffers (with 8 bits, another one
    // before the second frees the first half of X). But for the scales' at its beginning a step
    // has no branch: behind one the compiler puts the products before it, whose results nothing
    // needs yet.
    for (int it = 0; it < nk; ++it) {
      if (it % 4 == 0) {  // into the buffers whose last reads lie before the last barrier
        load_scales(it / 2 + 2);
        load_scales(it / 2 + 3);
      } else if (it % 4 == 3) {  // they have landed, and are read from this step's end on
        arrange(it / 2 + 1);
        arrange(it / 2 + 2);
      }
      take_scales(0);
      stage_w(it - 1 + RW);
      products(f0, std::integral_constant<int, 0>{}, [&](int x) __attribute__((always_inline)) {
        reads(x, it, 1, f1);
        loads_w(x);
      });
      if constexpr (kWide) {
        __asm__ volatile("s_waitcnt vmcnt(%0)" ::"n"(kLeft1) : "memory");
        __syncthreads();
        stage_x(it + RX, 0);
      }
      products(f1, std::integral_constant<int, 1>{}, [&](int x) __attribute__((always_inline)) {
        reads(x, it, 2, f0);
        if constexpr (kWide) loads_x(x);
      });
      products(f0, std::integral_constant<int, 2>{}, [&](int x) __attribute__((always_inline)) {
        reads(x, it, 3, f1);
      });
      __asm__ volatile("s_waitcnt vmcnt(%0)" ::"n"(kLeft3) : "memory");
      __syncthreads();
      stage_x(it + RX, kHalves - 1);
      products(f1, std::integral_constant<int, 3>{}, [&](int x) __attribute__((always_inline)) {
        reads(x, it + 1, 0, f0);
        scales(x, it + 1);
        loads_x(x);
      });
    }
  } else {
    // Two waves to a 32 x 32 block, either with half of a step's k: its two substeps, one barrier
    // between them, which the next step's X and W have landed before.
    static_assert(RX == RW && KS == 2, "one ring");
    load_scales(0);
    load_scales(1);
#pragma unroll
    for (int it = 0; it < RW; ++it) {
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        stage_x(it, h);
#pragma unroll
        for (int m = 0; m < LX; ++m) issue_x(m);
      }
      stage_w(it);
#pragma unroll
      for (int m = 0; m < LW; ++m) issue_w(m);
    }
    __asm__ volatile("s_waitcnt vmcnt(%0)" ::"n"((RW - 1) * kStep) : "memory");
    arrange(0);
    arrange(1);
    __syncthreads();
    auto read_all = [&](int it, int c, Frags& f) __attribute__((always_inline)) {
#pragma unroll
      for (int y = 0; y < FM + FN; ++y) read_one(it, 2 * kg + c, y, f);
    };
    auto read_scales = [&](int it) __attribute__((always_inline)) {
#pragma unroll
      for (int y = 0; y < FM + FN; ++y) read_scale(it, y);
    };
    read_all(0, 0, f0);
    read_scales(0);
    for (int it = 0; it < nk; ++it) {
      if (it % 4 == 0) {
        load_scales(it / 2 + 2);
        load_scales(it / 2 + 3);
      } else if (it % 4 == 3) {
        arrange(it / 2 + 1);
        arrange(it / 2 + 2);
      }
      take_scales(16 * kg);
      read_all(it, 1, f1);
      products(f0, std::integral_constant<int, 0>{}, [](int) {});
      __asm__ volatile("s_waitcnt vmcnt(%0)" ::"n"((RW - 2) * kStep) : "memory");
      __syncthreads();
      read_all(it + 1, 0, f0);
      read_scales(it + 1);
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        stage_x(it + RX, h);
#pragma unroll
        for (int m = 0; m < LX; ++m) issue_x(m);
      }
      stage_w(it + RW);
#pragma unroll
      for (int m = 0; m < LW; ++m) issue_w(m);
      products(f1, std::integral_constant<int, 1>{}, [](int) {});
    }
  }
  __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();  // every wave's loads have landed: the stages may be reused

  if constexpr (kTwo) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] += acc_low[i][j];
  }
  if constexpr (KS > 1) {  // the second halves' sums, added by the waves of the first
    static_assert(GM * GN * FM * FN * 4096 <= kLds, "sums fit the stages");
    float* sums = (float*)sm + (wave % (GM * GN)) * FM * FN * 1024 + lane;
    if (kg) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int e = 0; e < 16; ++e) sums[((i * FN + j) * 16 + e) * 64] = acc[i][j][e];
    }
    __syncthreads();
    if (kg) return;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] += sums[((i * FN + j) * 16 + e) * 64];
    wave_sync();  // read before the strips take their place
  }
  // Epilogue through LDS, one 32-token strip of the wave's block at a time: the lane holds
  // channel l % 32 of each block and tokens 8 (e / 4) + 4 (l / 32) + e % 4; read back, a lane has
  // 8 consecutive channels of one token.
  constexpr int kCols = 32 * FN, kPitch = kCols + 4;
  static_assert((KS > 1 ? GM * GN * FM * FN * 4096 : 0) + GM * GN * 32 * kPitch * 4 <= kLds,
                "strips fit the stages");
  // behind the sums of the second halves, which other waves may still read
  float* strip = (float*)sm + (KS > 1 ? GM * GN * FM * FN * 1024 : 0) + wave * 32 * kPitch;
  constexpr int kLanes = kCols / 8;   // lanes per token
  constexpr int kTok = 64 / kLanes;   // tokens per pass
  constexpr int kPass = 32 / kTok;
  const int64_t cp = (c + 7) & ~(int64_t)7;
  const int tl = lane / kLanes, ql = (lane % kLanes) * 8;
  const int64_t q = N0 + wn * kCols + ql;
  auto token = [&](int i, int p) { return M0 + wm * 32 * FM + i * 32 + p * kTok + tl; };
  auto values = [&](int p) { return strip + (p * kTok + tl) * kPitch + ql; };
  auto write_strip = [&](int i) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        strip[(8 * (e >> 2) + 4 * half + (e & 3)) * kPitch + j * 32 + r32] = acc[i][j][e];
    wave_sync();
  };
  if (part) {
#pragma unroll
    for (int i = 0; i < FM; ++i) {
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
  finish_tile<FM, kPass, true>(ep, n, c, q, token, values, write_strip);
}

// Up to 16 tokens: bound by reading W once. A workgroup takes 16 channels, its eight waves a
// share of the contraction each; W goes straight from memory into the operands of
// v_mfma_scale_f32_16x16x128_f8f6f4 (lane l: channel l % 16, k 32 (l / 16) .. + 31), with its
// scales 16 bytes (512 k) of a channel at a time; X comes from L2, in two parts where it is of
// e4m3. The waves' sums meet in LDS and are added in the order of the waves. Workgroup x takes
// the channels from 16 (first + x). One token 4096 -> 4096: 4.8-5.1 us, of which its 9 MB take
// 1.5; the rest is the launch and one chain of loads, products and joins. Longer contractions are
// several turns of 512 k in series: one token 11008 -> 4096 8.1-8.3, 4096 -> 11008 8.9 (their bytes 4.0),
// 16 tokens 12.2 and 12.7 (e2m1 X: 6.5 and 7.0, 8.5 and 9.6).
constexpr int kMsWaves = 8;

template <int XT>
__global__ __launch_bounds__(64 * kMsWaves) void mx_skinny_kernel(MxOperand X, MxOperand W, int n,
                                                                  int64_t b, int64_t c, int64_t first,
                                                                  LinEpilogue ep) {
  __shared__ float red[kMsWaves][16][17];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r16 = lane & 15, quad = lane >> 4;
  const int64_t f0 = (first + blockIdx.x) * 16;
  const int64_t fr = f0 + r16 < c ? f0 + r16 : c - 1;  // fills outputs that are not stored
  const int tr = r16 < n ? r16 : n - 1;
  const unsigned char *we = W.elements + fr * W.ld, *wsc = W.scales + fr * W.lds;
  const unsigned char *xe = X.elements + tr * X.ld, *xsc = X.scales + tr * X.lds;
  const int supers = (int)cdiv(b, 512), per = (int)cdiv(supers, kMsWaves);
  const int sb = wave * per, se = min(supers, sb + per);
  f32x4_t acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int u = sb; u < se; ++u) {
    u32x4_t w[4], x[4][XT == TH_MX_E4M3 ? 2 : 1];
    const u32x4_t ws4 = *(const u32x4_t*)(wsc + u * 16), xs4 = *(const u32x4_t*)(xsc + u * 16);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int64_t k = (int64_t)u * 512 + s * 128;
      const u32x4_t zero = u32x4_t{0u, 0u, 0u, 0u};
      w[s] = k + quad * 32 < b ? *(const u32x4_t*)(we + (k + quad * 32) / 2) : zero;
      if constexpr (XT == TH_MX_E4M3) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          x[s][h] = k + 64 * h + quad * 16 < b ? *(const u32x4_t*)(xe + k + 64 * h + quad * 16) : zero;
      } else {
        x[s][0] = k + quad * 32 < b ? *(const u32x4_t*)(xe + (k + quad * 32) / 2) : zero;
      }
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      // a block past the end has zeros for elements; 255 would make NaN of them
      const bool in = (int64_t)u * 512 + s * 128 + quad * 32 < b;
      const int ws = in ? (int)(ws4[s] >> (8 * quad)) : 0, xs = in ? (int)(xs4[s] >> (8 * quad)) : 0;
      MxFrag<TH_MX_E2M1> wf;
      wf.v = __builtin_bit_cast(i32x4_t, w[s]);
      if constexpr (XT == TH_MX_E4M3) {
        const i32x4_t lo = __builtin_bit_cast(i32x4_t, x[s][0]), hi = __builtin_bit_cast(i32x4_t, x[s][1]);
        i32x8_t high, low;
        mx_part(__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7), high, low);
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf.wide(), low, acc, 4, 0, 0, ws, 0, xs);
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf.wide(), high, acc, 4, 0, 0, ws, 0, xs);
      } else {
        MxFrag<TH_MX_E2M1> xf;
        xf.v = __builtin_bit_cast(i32x4_t, x[s][0]);
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf.wide(), xf.wide(), acc, 4, 4, 0, ws, 0,
                                                               xs);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) red[wave][r16][quad * 4 + e] = acc[e];
  __syncthreads();
  const int t = tid >> 4, q = tid & 15;
  if (t < n && f0 + q < c) {  // n <= 16
    float v = red[0][t][q];
#pragma unroll
    for (int w = 1; w < kMsWaves; ++w) v += red[w][t][q];
    finish1<true>(v, t, f0 + q, ep);
  }
}

// The tile kernel's forms. Its time is modelled as rounds of `slots` workgroups, each fixed +
// steps * (microseconds a step, by kind: e2m1, e4m3, e4m3 in two parts): `full` with all slots
// taken, and of forms with two workgroups per compute unit as soon as units are shared; between
// `lone` and that, by their number, in the other forms. The join of splits takes 1.7 us and its
// traffic at 4 TB/s. (Fitted to all forms' times, whole and in up to eight splits, at 17 to 6000
// tokens through 512 -> 2048, 2080 -> 1023, 4096 -> 4096, 4096 -> 11008 and 11008 -> 4096, in every
// kind: what it takes is as fast as the fastest in the mean, 5% slower at most.)
struct MxTile {
  int tm, tn;
  int slots;
  double lone[3], full[3], fixed;
};
enum { kMx64 = 0, kMx128 = 1, kMx128x256 = 2, kMx256 = 3, kMxTiles = 4, kMxSkinny = 4 };
constexpr int kMxUnits = 256;  // compute units
constexpr MxTile kMxForms[kMxTiles] = {
    {64, 64, 2 * kMxUnits, {0.27, 0.41, 0.63}, {0.48, 0.61, 1.16}, 5.2},    // 4 (or 4 times 2) waves of 32 x 32
    {128, 128, 2 * kMxUnits, {0.62, 0.76, 1.54}, {1.24, 1.62, 3.55}, 4.9},  // 8 waves of 32 x 64
    {128, 256, kMxUnits, {0.75, 1.18, 2.8}, {1.19, 1.49, 3.05}, 5.1},       // 8 waves of 64 x 64
    {256, 256, kMxUnits, {1.09, 1.88, 4.3}, {1.89, 2.5, 4.65}, 8.2},        // 8 waves of 64 x 128
};
constexpr int64_t kMxSkinnyTokens = 16;

struct MxPlan {
  int tile;
  int splits;  // pieces of the contraction
  int per;     // steps per piece, even where there are several
};

MxPlan plan_of(int xtype, int64_t n, int64_t b, int64_t c, bool exact, bool can_split) {
  const int64_t steps = cdiv(b, kMK);
  MxPlan best = {kMxSkinny, 1, (int)steps};
  if (n <= kMxSkinnyTokens) return best;
  const int kind = xtype == TH_MX_E2M1 ? 0 : (exact ? 2 : 1);
  double least = 1e300;
  for (int t = 0; t < kMxTiles; ++t) {
    const MxTile& k = kMxForms[t];
    const int64_t tiles = cdiv(n, k.tm) * cdiv(c, k.tn);
    if (tiles >= ((int64_t)1 << 23) - 8) continue;  // a launch has less than 2^32 threads
    for (int64_t want : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (want > 1 && (!can_split || tiles * want > 4 * k.slots)) break;
      const int64_t per = want == 1 ? steps : cdiv(cdiv(steps, 2), want) * 2;
      const int64_t splits = cdiv(steps, per);
      const int64_t full = tiles * splits / k.slots, rest = tiles * splits % k.slots;
      double us = (double)full * (k.fixed + (double)per * k.full[kind]);
      if (rest) {
        const double share = k.slots > kMxUnits ? (rest > kMxUnits ? 1.0 : 0.0) : (double)rest / k.slots;
        us += k.fixed + (double)per * (k.lone[kind] + (k.full[kind] - k.lone[kind]) * share);
      }
      if (splits > 1) us += 1.7 + 8.0 * (double)splits * (double)n * (double)c / 4e6;
      if (us < least) {
        least = us;
        best = {t, (int)splits, (int)per};
      }
      if (per <= 2) break;
    }
  }
  return best;
}

template <int XT, int FM, int FN, int GM, int GN, int KS, int RX, int RW, bool EXACT>
hipError_t launch_tiles(const MxOperand& X, const MxOperand& W, int64_t n, int64_t b, int64_t c,
                        const MxPlan& p, float* part, const LinEpilogue& ep, hipStream_t s) {
  const int ntm = (int)cdiv(n, 32 * FM * GM), ntn = (int)cdiv(c, 32 * FN * GN);
  const int per_xcd = (int)cdiv((int64_t)ntm * ntn, 8);
  hipLaunchKernelGGL((mx_tile_kernel<XT, FM, FN, GM, GN, KS, RX, RW, EXACT>),
                     dim3((unsigned)(8 * per_xcd), (unsigned)p.splits), dim3(64 * GM * GN * KS), 0, s, X, W, n, b,
                     c, ntm, ntn, per_xcd, p.per, part, ep);
  return hipGetLastError();
}

template <int XT, bool EXACT>
hipError_t launch_form(const MxOperand& X, const MxOperand& W, int64_t n, int64_t b, int64_t c,
                       const MxPlan& p, float* part, const LinEpilogue& ep, hipStream_t s) {
  constexpr bool wide = XT == TH_MX_E4M3;
  switch (p.tile) {
    case kMx64: return launch_tiles<XT, 1, 1, 2, 2, wide && !EXACT ? 1 : 2, wide ? 3 : 4, wide ? 3 : 4, EXACT>(X, W, n, b, c, p, part, ep, s);
    case kMx128: return launch_tiles<XT, 1, 2, 4, 2, 1, wide ? 1 : 2, 2, EXACT>(X, W, n, b, c, p, part, ep, s);
    case kMx128x256: return launch_tiles<XT, 2, 2, 2, 4, 1, 2, 2, EXACT>(X, W, n, b, c, p, part, ep, s);
    default: return launch_tiles<XT, 2, 4, 4, 2, 1, wide ? 1 : 2, 2, EXACT>(X, W, n, b, c, p, part, ep, s);
  }
}

}  // namespace

size_t mx_linear_workspace_floats(int xtype, int64_t n, int64_t b, int64_t c, th_dtype ydt) {
  const MxPlan p = plan_of(xtype, n, b, c, ydt == TH_F32, true);
  return p.splits > 1 ? (size_t)p.splits * (size_t)n * (size_t)(cdiv(c, 8) * 8) : 0;
}

void mx_linear_plan(int xtype, int64_t n, int64_t b, int64_t c, th_dtype ydt, bool can_split,
                    int32_t* tokens, int32_t* channels, int32_t* pieces) {
  const MxPlan p = plan_of(xtype, n, b, c, ydt == TH_F32, can_split);
  *tokens = p.tile == kMxSkinny ? (int32_t)kMxSkinnyTokens : kMxForms[p.tile].tm;
  *channels = p.tile == kMxSkinny ? 16 : kMxForms[p.tile].tn;
  *pieces = p.splits;
}

hipError_t launch_mx_linear(const th_mx& X, const th_mx& W, int64_t n, int64_t b, int64_t c,
                            const unsigned short* bias, int act, const void* residual, int64_t ldr,
                            void* Y, th_dtype ydt, int64_t ldy, float* part, hipStream_t s) {
  LinEpilogue ep;
  ep.bias = bias;
  ep.residual = residual;
  ep.y = Y;
  ep.ldr = ldr;
  ep.ldy = ldy;
  ep.act = act;
  ep.y_f32 = ydt == TH_F32;
  // bf16 Y of 2^27 and more outputs, 268 MB: the last level cache holds 256 MB. Past the caches and
  // through them, tokens 4096 -> 11008: 12192 tokens 327 and 334 us, 32768 806 and 810 (another card 810
  // and 835), 65536 1568 and 1582; below, 4096 to 16384 tokens, the same to 0.3%. An fp32 Y has no such form.
  ep.past_cache = n * c >= (int64_t)1 << 27;
  const MxOperand x = {(const unsigned char*)X.elements, (const unsigned char*)X.scales, X.ld, X.lds};
  const MxOperand w = {(const unsigned char*)W.elements, (const unsigned char*)W.scales, W.ld, W.lds};
  const bool wide = X.type == TH_MX_E4M3;
  const MxPlan p = plan_of(X.type, n, b, c, ep.y_f32, part != nullptr);
  if (p.tile == kMxSkinny) {
    // a launch has less than 2^32 threads, 512 to a workgroup
    const int64_t groups = cdiv(c, 16), most = (int64_t)1 << 22;
    for (int64_t first = 0; first < groups; first += most) {
      const dim3 grid((unsigned)(groups - first < most ? groups - first : most));
      if (wide)
        hipLaunchKernelGGL(mx_skinny_kernel<TH_MX_E4M3>, grid, dim3(64 * kMsWaves), 0, s, x, w, (int)n, b,
                           c, first, ep);
      else
        hipLaunchKernelGGL(mx_skinny_kernel<TH_MX_E2M1>, grid, dim3(64 * kMsWaves), 0, s, x, w, (int)n, b,
                           c, first, ep);
    }
    return hipGetLastError();
  }
  float* raw = p.splits > 1 ? part : nullptr;
  hipError_t e = !wide ? launch_form<TH_MX_E2M1, false>(x, w, n, b, c, p, raw, ep, s)
                 : ep.y_f32 ? launch_form<TH_MX_E4M3, true>(x, w, n, b, c, p, raw, ep, s)
                            : launch_form<TH_MX_E4M3, false>(x, w, n, b, c, p, raw, ep, s);
  if (e != hipSuccess || !raw) return e;
  const int64_t items = n * cdiv(c, 8);
  hipLaunchKernelGGL(linear_join_kernel<true>, dim3((unsigned)cdiv(items, 256)), dim3(256), 0, s, raw,
                     p.splits, n, c, ep);
  return hipGetLastError();
}

}  // namespace th
