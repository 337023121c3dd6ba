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
// Tiles as in linear.hip: (64 FM) tokens x (32 FN GN) channels on 2 x GN waves, each 32 FM x
// 32 FN. Stages of 128 k are filled by direct global->LDS loads, S deep; 16-byte pieces of a
// row are XOR-swizzled so that operand reads use all banks. Scales come 16 bytes (512 k) of a
// row at a time, every fourth stage, into two buffers of their own.
#include "common.h"
#include "lds_dma.h"
#include "linear_epilogue.h"
#include "mx.h"

namespace th {

namespace {

constexpr int kMK = 128;      // contraction per stage
constexpr int kMSuper = 4;    // stages per 16 bytes of scales
constexpr int kMGroup = 4;    // token tiles per group in the walk order

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
    const unsigned u = (unsigned)v[i], one = (u >> 6) & 0x01010101u;
    const unsigned mask = (one << 8) - one;  // bytes of ones: a byte's borrow is the next one's carry
    high[i] = (int)(u & mask);
    low[i] = (int)(u & ~mask);
  }
}

template <int XT, int FM, int FN, int GN, int S, bool EXACT>
__global__ __launch_bounds__(128 * GN) void mx_tile_kernel(MxOperand X, MxOperand W, int64_t n, int64_t b,
                                                           int64_t c, int ntm, int ntn, int per_xcd,
                                                           int stages_per_split,
                                                           float* __restrict__ part, LinEpilogue ep) {
  constexpr int TM = 64 * FM, TN = 32 * FN * GN;
  constexpr int kWaves = 2 * GN;
  constexpr int kXRow = XT == TH_MX_E4M3 ? kMK : kMK / 2, kWRow = kMK / 2;  // bytes of a stage's row
  constexpr int kA = TM * kXRow, kB = TN * kWRow;
  constexpr int LA = kA / 1024 / kWaves, LB = kB / 1024 / kWaves;  // 1 KB loads per wave and stage
  constexpr int kScales = (TM + TN) * 16;  // of 512 k
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
  const int nk_all = (int)cdiv(b, kMK);
  const int s_begin = blockIdx.y * stages_per_split;  // a multiple of kMSuper
  const int nk = min(stages_per_split, nk_all - s_begin);
  if (nk <= 0) return;  // no split of the launch is empty

  __shared__ __attribute__((aligned(1024))) unsigned char sm[S * (kA + kB) + 2 * kScales];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / GN, wn = wave % GN;
  const unsigned smb = lds_address(sm);

  // Loader: chunks of 1 KB, wave w those w + kWaves m of either operand. Rows of 64 bytes: lane l
  // fills row 16 chunk + l / 4 at physical piece l % 4, swizzled by (row / 4) & 3; of 128 bytes:
  // row 8 chunk + l / 8 at piece l % 8, by (row / 2) & 7. Either is the same in a lane's chunks.
  auto piece_of = [&](int row_bytes) {
    return row_bytes == 64 ? (lane & 3) ^ ((lane >> 4) & 3)
                           : (lane & 7) ^ (((wave & 1) << 2) + (lane >> 4));
  };
  const int la = piece_of(kXRow), lb = piece_of(kWRow);
  unsigned va[LA], vb[LB];
#pragma unroll
  for (int m = 0; m < LA; ++m) {
    int64_t r = M0 + (wave + kWaves * m) * (1024 / kXRow) + lane / (kXRow / 16);
    r = r < n ? r : n - 1;  // rows past the end feed outputs that are never stored
    va[m] = (unsigned)((r - M0) * X.ld + la * 16);
  }
#pragma unroll
  for (int m = 0; m < LB; ++m) {
    int64_t r = N0 + (wave + kWaves * m) * (1024 / kWRow) + lane / (kWRow / 16);
    r = r < c ? r : c - 1;
    vb[m] = (unsigned)((r - N0) * W.ld + lb * 16);
  }
  // Scales: 64 rows a load, X's rows first; the first waves have one each.
  constexpr int kScaleLoads = (TM + TN) / 64;
  static_assert(kScaleLoads <= kWaves, "one load of scales per wave");
  const bool scale_x = wave * 64 < TM;
  unsigned vs;
  {
    const int64_t first = scale_x ? M0 + wave * 64 : N0 + wave * 64 - TM;
    int64_t r = first + lane;
    const int64_t last = (scale_x ? n : c) - 1;
    r = r < last ? r : last;
    vs = (unsigned)(scale_x ? (r - M0) * X.lds : (r - N0) * W.lds);
  }
  const unsigned char* scale_base = scale_x ? X.scales + M0 * X.lds : W.scales + N0 * W.lds;
  const unsigned scale_lds = smb + S * (kA + kB) + wave * 1024;
  const int st_last = nk_all - 1, super_last = st_last / kMSuper;
  auto load_scales = [&](int it) {  // those of the stages from it on, a multiple of kMSuper
    if (wave >= kScaleLoads) return;
    const int u = (s_begin + it) / kMSuper;
    lds_dma1(vs, scale_base + (int64_t)min(u, super_last) * 16,
             scale_lds + (it / kMSuper % 2) * kScales);
  };
  // Stages past the last are loaded too (never read), so that every stage has the same number
  // of loads for the vmcnt waits; they re-read the last. Pieces of the last stage past b
  // re-read its piece 0; zero_tail clears them. Loads of scales among them only make the
  // waits stricter.
  const int64_t k_last = (int64_t)st_last * kMK;
  const bool a_past = k_last + la * (kMK / (kXRow / 16)) >= b;
  const bool b_past = k_last + lb * (kMK / (kWRow / 16)) >= b;
  const unsigned char *xs = X.elements, *ws = W.elements;
  unsigned abase = 0, bbase = 0;
  bool a_last = false, b_last = false;
  auto stage_a = [&](int it) {
    const int st = s_begin + it;
    xs = X.elements + M0 * X.ld + (int64_t)min(st, st_last) * kXRow;
    abase = smb + (it % S) * kA + wave * 1024;
    if (st >= st_last && !a_last) {  // from here on every stage issued is the last one
      a_last = true;
      if (a_past) {
#pragma unroll
        for (int m = 0; m < LA; ++m) va[m] -= la * 16;
      }
    }
  };
  auto stage_b = [&](int it) {
    const int st = s_begin + it;
    ws = W.elements + N0 * W.ld + (int64_t)min(st, st_last) * kWRow;
    bbase = smb + S * kA + (it % S) * kB + wave * 1024;
    if (st >= st_last && !b_last) {
      b_last = true;
      if (b_past) {
#pragma unroll
        for (int m = 0; m < LB; ++m) vb[m] -= lb * 16;
      }
    }
  };
  auto issue_a = [&](int m) { lds_dma1(va[m], xs, abase + m * kWaves * 1024); };
  auto issue_b = [&](int m) { lds_dma1(vb[m], ws, bbase + m * kWaves * 1024); };
  // Zero this wave's pieces of stage it that lie past b, and, where the stage is the first of
  // the last scales, the scales of blocks past it (255 there would make NaN of 0). Its own loads
  // have landed.
  auto zero_tail = [&](int it) {
    const int st = s_begin + it;
    if (it % kMSuper == 0 && st / kMSuper == super_last && wave < kScaleLoads) {
      const int blocks = (int)(b / kMxBlock) - super_last * 16;
      if (blocks < 16) {
        unsigned* z = (unsigned*)(sm + S * (kA + kB) + (it / kMSuper % 2) * kScales + wave * 1024 +
                                  lane * 16);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int left = blocks - 4 * x;  // of this word's four
          if (left < 4) z[x] = left <= 0 ? 0u : z[x] & (0xffffffffu >> (32 - 8 * left));
        }
      }
    }
    if (st != st_last) return;
    const u32x4_t zero = u32x4_t{0u, 0u, 0u, 0u};
    if (a_past) {
#pragma unroll
      for (int m = 0; m < LA; ++m)
        *(u32x4_t*)(sm + (it % S) * kA + (wave + m * kWaves) * 1024 + lane * 16) = zero;
    }
    if (b_past) {
#pragma unroll
      for (int m = 0; m < LB; ++m)
        *(u32x4_t*)(sm + S * kA + (it % S) * kB + (wave + m * kWaves) * 1024 + lane * 16) = zero;
    }
  };

  f32x16_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  const int r32 = lane & 31, half = lane >> 5;
  const int waddr = r32 * 64 + ((half ^ ((r32 >> 2) & 3)) << 4);   // rows of 64 bytes
  const int xaddr = XT == TH_MX_E4M3 ? r32 * 128 + ((half ^ ((r32 >> 1) & 7)) << 4) : waddr;
  struct Frags {
    MxFrag<XT> a[FM];
    MxFrag<TH_MX_E2M1> b[FN];
  };
  Frags f0, f1;
  int sa[FM], sb[FN], sa2[FM], sb2[FN];
  // operand y of substep sub (64 k): the FN blocks of W, then the FM of X
  auto read_one = [&](int it, int sub, int y, Frags& f) {
    if (y < FN) {
      f.b[y].v = *(const i32x4_t*)(sm + S * kA + (it % S) * kB + (wn * FN + y) * 32 * kWRow +
                                   (waddr ^ (sub << 5)));
    } else {
      const unsigned char* p = sm + (it % S) * kA + (wm * FM + y - FN) * 32 * kXRow;
      if constexpr (XT == TH_MX_E4M3) {
        const i32x4_t lo = *(const i32x4_t*)(p + (xaddr ^ (sub << 6)));
        const i32x4_t hi = *(const i32x4_t*)(p + (xaddr ^ (sub << 6) ^ 32));
        f.a[y - FN].v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      } else {
        f.a[y - FN].v = *(const i32x4_t*)(p + (xaddr ^ (sub << 5)));
      }
    }
  };
  // Scales of a stage's four blocks of 32 k, shifted so that substep sub's is byte 2 sub.
  auto read_scale = [&](int it, int y, int (&a)[FM], int (&bb)[FN]) {
    const unsigned char* p = sm + S * (kA + kB) + (it / kMSuper % 2) * kScales + (it % kMSuper) * 4;
    if (y < FN)
      bb[y] = *(const int*)(p + (TM + (wn * FN + y) * 32 + r32) * 16);
    else
      a[y - FN] = *(const int*)(p + ((wm * FM + y - FN) * 32 + r32) * 16);
  };
  auto shift_scales = [&](int (&a)[FM], int (&bb)[FN]) {
#pragma unroll
    for (int i = 0; i < FM; ++i) a[i] = (int)((unsigned)a[i] >> (8 * half));
#pragma unroll
    for (int j = 0; j < FN; ++j) bb[j] = (int)((unsigned)bb[j] >> (8 * half));
  };
  // One substep's products, with reads and loads between them; the order is pinned.
  auto mfmas = [&](const Frags& f, auto SUB, auto&& between) __attribute__((always_inline)) {
    constexpr int sub = decltype(SUB)::value;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      [[maybe_unused]] i32x8_t high, low;
      if constexpr (EXACT && XT == TH_MX_E4M3) mx_part(f.a[i].v, high, low);
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        if constexpr (EXACT && XT == TH_MX_E4M3) {
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              low, f.b[j].wide(), acc[i][j], kMxCode<XT>, kMxCode<TH_MX_E2M1>, 2 * sub, sa[i], 2 * sub,
              sb[j]);
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              high, f.b[j].wide(), acc[i][j], kMxCode<XT>, kMxCode<TH_MX_E2M1>, 2 * sub, sa[i],
              2 * sub, sb[j]);
        } else {
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              f.a[i].wide(), f.b[j].wide(), acc[i][j], kMxCode<XT>, kMxCode<TH_MX_E2M1>, 2 * sub,
              sa[i], 2 * sub, sb[j]);
        }
        __builtin_amdgcn_sched_barrier(0);
        between(i * FN + j);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  constexpr int kProducts = FM * FN, kReads = (FM + FN + kProducts - 1) / kProducts;
  constexpr int kLoadsA = (LA + kProducts - 1) / kProducts, kLoadsB = (LB + kProducts - 1) / kProducts;
  constexpr int kGapA = kProducts / LA > 0 ? kProducts / LA : 1;
  constexpr int kGapB = kProducts / LB > 0 ? kProducts / LB : 1;

  // prologue: the first two scales, W's and X's stages 0 .. S-2, waited for; then W's S-1
  load_scales(0);
  load_scales(kMSuper);
#pragma unroll
  for (int it = 0; it < S - 1; ++it) {
    stage_b(it);
#pragma unroll
    for (int m = 0; m < LB; ++m) issue_b(m);
    stage_a(it);
#pragma unroll
    for (int m = 0; m < LA; ++m) issue_a(m);
  }
  __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
  zero_tail(0);
  __syncthreads();
  stage_b(S - 1);
#pragma unroll
  for (int m = 0; m < LB; ++m) issue_b(m);
#pragma unroll
  for (int y = 0; y < FM + FN; ++y) {
    read_one(0, 0, y, f0);
    read_scale(0, y, sa, sb);
  }
  shift_scales(sa, sb);
  // A stage: half its products, then (its last operands read, the next stage landed, the
  // barrier) the other half. X's stage it + S - 1 goes into the buffer freed by the barrier of
  // stage it - 1 during the first half, W's stage it + S into the one freed by this stage's
  // during the second, every fourth stage's scales likewise.
  for (int it = 0; it < nk; ++it) {
    stage_a(it + S - 1);
    mfmas(f0, std::integral_constant<int, 0>{}, [&](int x) __attribute__((always_inline)) {
#pragma unroll
      for (int y = 0; y < kReads; ++y)
        if (x * kReads + y < FM + FN) read_one(it, 1, x * kReads + y, f1);
      if (x % kGapA == 0) {
#pragma unroll
        for (int m = 0; m < kLoadsA; ++m)
          if (x / kGapA * kLoadsA + m < LA) issue_a(x / kGapA * kLoadsA + m);
      }
    });
    __asm__ volatile("s_waitcnt vmcnt(%0)" ::"n"((S - 2) * (LA + LB)) : "memory");
    zero_tail(it + 1);
    __syncthreads();
    stage_b(it + S);
    if (it % kMSuper == kMSuper - 1) load_scales(it + 1 + kMSuper);
    mfmas(f1, std::integral_constant<int, 1>{}, [&](int x) __attribute__((always_inline)) {
#pragma unroll
      for (int y = 0; y < kReads; ++y)
        if (x * kReads + y < FM + FN) {
          read_one(it + 1, 0, x * kReads + y, f0);
          read_scale(it + 1, x * kReads + y, sa2, sb2);
        }
      if (x % kGapB == 0) {
#pragma unroll
        for (int m = 0; m < kLoadsB; ++m)
          if (x / kGapB * kLoadsB + m < LB) issue_b(x / kGapB * kLoadsB + m);
      }
    });
#pragma unroll
    for (int i = 0; i < FM; ++i) sa[i] = sa2[i];
#pragma unroll
    for (int j = 0; j < FN; ++j) sb[j] = sb2[j];
    shift_scales(sa, sb);
  }
  __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();  // every wave's loads have landed: the stages may be reused

  // Epilogue through LDS, one 32-token strip of the wave's block at a time: the lane holds
  // channel l % 32 of each block and tokens 8 (e / 4) + 4 (l / 32) + e % 4; read back, a lane has
  // 8 consecutive channels of one token.
  constexpr int kCols = 32 * FN, kPitch = kCols + 4;
  static_assert(kWaves * 32 * kPitch * 4 <= S * (kA + kB), "strips fit the stages");
  float* strip = (float*)sm + wave * 32 * kPitch;
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
  finish_tile<FM, kPass>(ep, n, c, q, token, values, write_strip);
}

// Up to 16 tokens: bound by reading W once. A workgroup takes 16 channels, its eight waves a
// share of the contraction each; W goes straight from memory into the operands of
// v_mfma_scale_f32_16x16x128_f8f6f4 (lane l: channel l % 16, k 32 (l / 16) .. + 31), with its
// scales 16 bytes (512 k) of a channel at a time; X comes from L2, in two parts where it is of
// e4m3. The waves' sums meet in LDS and are added in the order of the waves. Workgroup x takes
// the channels from 16 (first + x).
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
    finish1(v, t, f0 + q, ep);
  }
}

// The tile kernel's forms, their time modelled as in linear.hip: rounds of `slots` workgroups,
// each fixed + stages * per_stage microseconds with every slot taken and half of the second
// part with few, and the join of splits as 3 us and its traffic at 4 TB/s.
struct MxTile {
  int tm, tn;
  int slots;
  double per_stage[3], fixed;  // per stage: e2m1, e4m3, e4m3 in two parts
};
enum { kMx64 = 0, kMx128 = 1, kMx128x256 = 2, kMx256 = 3, kMxTiles = 4, kMxSkinny = 4 };
constexpr MxTile kMxForms[kMxTiles] = {
    {64, 64, 512, {0.4, 0.5, 0.6}, 4.0},
    {128, 128, 512, {0.5, 0.7, 0.9}, 6.0},
    {128, 256, 256, {0.6, 0.85, 1.1}, 7.0},
    {256, 256, 256, {1.0, 1.45, 2.2}, 12.0},
};
constexpr int64_t kMxSkinnyTokens = 16;

struct MxPlan {
  int tile;
  int splits;  // pieces of the contraction
  int per;     // stages per piece, a multiple of kMSuper
};

MxPlan plan_of(int xtype, int64_t n, int64_t b, int64_t c, bool exact, bool can_split) {
  const int64_t stages = cdiv(b, kMK);
  MxPlan best = {kMxSkinny, 1, (int)stages};
  if (n <= kMxSkinnyTokens) return best;
  const int kind = xtype == TH_MX_E2M1 ? 0 : (exact ? 2 : 1);
  double least = 1e300;
  for (int t = 0; t < kMxTiles; ++t) {
    const MxTile& k = kMxForms[t];
    const int64_t tiles = cdiv(n, k.tm) * cdiv(c, k.tn);
    for (int64_t want : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (want > 1 && (!can_split || stages < kMSuper * want || tiles * want > 4 * k.slots)) break;
      const int64_t per = want == 1 ? stages : cdiv(cdiv(stages, kMSuper), want) * kMSuper;
      const int64_t splits = cdiv(stages, per);
      const int64_t full = tiles * splits / k.slots, rest = tiles * splits % k.slots;
      double us = (double)full * (k.fixed + (double)per * k.per_stage[kind]);
      if (rest)
        us += k.fixed + (double)per * k.per_stage[kind] * (0.5 + 0.5 * (double)rest / k.slots);
      if (splits > 1) us += 3.0 + 8.0 * (double)splits * (double)n * (double)c / 4e6;
      if (us < least) {
        least = us;
        best = {t, (int)splits, (int)per};
      }
    }
  }
  return best;
}

template <int XT, int FM, int FN, int GN, int S, bool EXACT>
hipError_t launch_tiles(const MxOperand& X, const MxOperand& W, int64_t n, int64_t b, int64_t c,
                        const MxPlan& p, float* part, const LinEpilogue& ep, hipStream_t s) {
  const int ntm = (int)cdiv(n, 64 * FM), ntn = (int)cdiv(c, 32 * FN * GN);
  const int per_xcd = (int)cdiv((int64_t)ntm * ntn, 8);
  hipLaunchKernelGGL((mx_tile_kernel<XT, FM, FN, GN, S, EXACT>),
                     dim3((unsigned)(8 * per_xcd), (unsigned)p.splits), dim3(128 * GN), 0, s, X, W, n, b,
                     c, ntm, ntn, per_xcd, p.per, part, ep);
  return hipGetLastError();
}

template <int XT, bool EXACT>
hipError_t launch_form(const MxOperand& X, const MxOperand& W, int64_t n, int64_t b, int64_t c,
                       const MxPlan& p, float* part, const LinEpilogue& ep, hipStream_t s) {
  constexpr bool wide = XT == TH_MX_E4M3;
  switch (p.tile) {
    case kMx64: return launch_tiles<XT, 1, 1, 2, 4, EXACT>(X, W, n, b, c, p, part, ep, s);
    case kMx128: return launch_tiles<XT, 2, 1, 4, wide ? 3 : 4, EXACT>(X, W, n, b, c, p, part, ep, s);
    case kMx128x256: return launch_tiles<XT, 2, 2, 4, 4, EXACT>(X, W, n, b, c, p, part, ep, s);
    default: return launch_tiles<XT, 4, 2, 4, wide ? 3 : 4, EXACT>(X, W, n, b, c, p, part, ep, s);
  }
}

}  // namespace

size_t mx_linear_workspace_floats(int xtype, int64_t n, int64_t b, int64_t c, th_dtype ydt) {
  const MxPlan p = plan_of(xtype, n, b, c, ydt == TH_F32, true);
  return p.splits > 1 ? (size_t)p.splits * (size_t)n * (size_t)(cdiv(c, 8) * 8) : 0;
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
  hipLaunchKernelGGL(linear_join_kernel, dim3((unsigned)cdiv(items, 256)), dim3(256), 0, s, raw,
                     p.splits, n, c, ep);
  return hipGetLastError();
}

}  // namespace th
