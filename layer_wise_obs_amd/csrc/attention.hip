// Attention over packed sequences, O = softmax(scale Q K^T + mask) V, grouped heads
// (g = hq / hk query heads read one key head), causal to the end of the keys: the
// last query of a sequence sees its last key. What o_proj reads in a block whose
// q/k/v projections are pruned ("Pruning LLMs with Thanos", sections "The
// layer-reconstruction lens" and "The compression target: linear layers").
//
// One pass over the keys with a running reference m and sum l per query,
//   p_j = 2^(c s_j - m),  l += p_j,  O += p_j v_j,  c = scale log2(e),
// rescaled by 2^(m_old - m_new) when m moves. m only has to be near the maximum:
// it moves when a score passes it by more than 8 (p <= 2^8 then), so most tiles
// need no rescaling. m, l and O are fp32; p is rounded to bf16 for the matrix cores
// (off by at most 2^-8 of itself, like the output's own rounding: against 64 bits 2.0e-3
// rms instead of 1.65e-3). Products of what that rounding leaves, 2^-16 of p, too would
// take 673 -> 1079 us for 16 sequences of 2048 tokens, 32 heads of 128 (92 registers
// spill), 90 -> 104 for 24 prompts, heads of 80. The kernel for few rows below has them.
//
// A workgroup takes 128 rows of one sequence and key head, a row being a (token,
// query head of the group) pair, so K and V are read once for all g heads and
// single tokens fill g rows. Each of the four waves owns 32 rows. The products are
// formed transposed, S^T = K Q^T and O^T = V^T P^T with v_mfma_f32_16x16x32_bf16 (at
// this card's power limit 5% ahead of the 32x32x16 form): a lane then holds scores of
// two queries only (their softmax needs two exchanges with the other quarters of the
// wave), and its P values already are the operand of the second product -- the
// contraction order over keys is free, so V's transposing LDS reads
// (ds_read_b64_tr_b16, 4 keys each) follow the order P has in the registers.
// Tiles of 64 keys are copied into LDS by direct loads, double-buffered; the 16-byte
// pieces of a row are XOR-swizzled so that both kinds of operand reads use all banks.
//
// Bound by two waves per SIMD (their registers: 64 of O, 32 each of Q, scores, V and K
// operands; heads above 96 use all 256 and spill 1 to 13, reloaded outside the products)
// whose products and softmax overlap only in part: 16 sequences of 2048 tokens, 32 heads
// of 128, 645-695 us (790-850 TFLOP/s of the visible half), 38% of the cycles in
// products; one sequence of 16384, 8 heads on 2, 525-545 (1010-1050).
//
// Where there are few workgroups, the keys of each are split over several; the
// partial (m, l, O) are joined by a second kernel in a fixed order.
#include "common.h"
#include "lds_dma.h"

namespace th {

namespace {

constexpr int kAKT = 64;   // keys per tile
constexpr float kAMove = 8.0f;  // log2 of how far p may pass 1 before m moves

typedef short v4i16_t __attribute__((ext_vector_type(4)));
typedef short v8i16_t __attribute__((ext_vector_type(8)));
typedef unsigned short u16x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));

struct AttnArgs {
  const unsigned short *q, *k, *v;
  unsigned short* o;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head, o_token, o_head;
  const int32_t *q_start, *k_start;  // NULL: one sequence of all rows
  int64_t nq, nk;
  int nseq, hk, g, d, causal, splits;
  float c;        // scale * log2(e)
  float* part_o;  // [splits][nq][hq][d]
  float2* part_ml;
};

// Entry i of a start array, kept inside [0, n]: whatever it holds, no access leaves
// the tensors.
__device__ __forceinline__ int64_t start_at(const int32_t* s, int i, int64_t n) {
  if (!s) return i ? n : 0;
  const int64_t v = s[i];
  return v < 0 ? 0 : (v > n ? n : v);
}

struct Sequence {
  int index;              // -1: the slot belongs to none
  int64_t q0, q1, k0, k1;  // its rows of Q and K
};

// The slots of sequence s begin at floor(q_start[s] g / BM) + s: at least as many
// slots as the sequence has row blocks lie before the next one's. A slot belongs to
// the last sequence whose slots begin at or before it; up to 63 sequences are found
// with one load of either start array (a lane holds a start), more by looking at 64
// at a time.
template <int BM>
__device__ __forceinline__ Sequence sequence_of(const AttnArgs& a, int64_t slot, int lane) {
  Sequence r;
  r.index = -1;
  if (a.nseq < 64) {
    const int i = min(lane, a.nseq);
    const int q = (int)start_at(a.q_start, i, a.nq), k = (int)start_at(a.k_start, i, a.nk);
    const bool before = lane < a.nseq && (int64_t)q * a.g / BM + lane <= slot;
    const int cnt = __popcll(__ballot(before));
    if (cnt == 0) return r;
    r.index = cnt - 1;
    r.q0 = __builtin_amdgcn_readlane(q, cnt - 1);
    r.q1 = __builtin_amdgcn_readlane(q, cnt);
    r.k0 = __builtin_amdgcn_readlane(k, cnt - 1);
    r.k1 = __builtin_amdgcn_readlane(k, cnt);
    return r;
  }
  int lo = 0, len = a.nseq;
  for (;;) {
    const int step = (len + 63) >> 6;
    const int at = lane * step;
    const bool before =
        at < len && start_at(a.q_start, lo + at, a.nq) * a.g / BM + lo + at <= slot;
    const int cnt = __popcll(__ballot(before));
    if (cnt == 0) return r;
    lo += (cnt - 1) * step;
    if (step == 1) break;
    len = min(step, len - (cnt - 1) * step);
  }
  r.index = lo;
  r.q0 = start_at(a.q_start, lo, a.nq);
  r.q1 = start_at(a.q_start, lo + 1, a.nq);
  r.k0 = start_at(a.k_start, lo, a.nk);
  r.k1 = start_at(a.k_start, lo + 1, a.nk);
  return r;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Maximum over the two lanes (l, l + 32) that share a query.
__device__ __forceinline__ float half_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
// Maximum over the four lanes (l % 16 + 16 i) that share a query.
__device__ __forceinline__ float quad_max(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return half_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
// v_max3_f32: two maxima in one instruction, NaN operands ignored like fmaxf's (which
// the compiler precedes by a canonicalising maximum of either operand). The compiler
// does not know the instruction, so it puts no wait between a matrix product and it: a
// and the products of b and c must have been waited for by an ordinary operation that
// `a` depends on.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  __asm__("v_max3_f32 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "v"(c));
  return d;
}

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ bf16x2_t pack2(float a, float b) {
  return bf16x2_t{(__bf16)a, (__bf16)b};  // v_cvt_pk_bf16_f32, round to nearest even
}

// D elements per row in LDS, of which the first DC (the head rounded up to 16) make
// channels of O; PAD: the head is shorter than D.
template <int D, int DC, bool PAD>
__global__ __launch_bounds__(256, 2) void attention_kernel(AttnArgs a) {
  constexpr int NW = 4, ST = 2;              // waves of 32 rows; tiles of keys in LDS
  constexpr int kBM = 32 * NW;
  constexpr int kPieces = D / 8;             // 16-byte pieces per row
  constexpr int kRowB = D * 2;
  constexpr int kTile = kAKT * kRowB;        // one operand's tile
  constexpr int kLd = kTile / 1024 / NW;     // 1 KB loads per wave and operand
  constexpr int kRowsPer = 64 / kPieces;     // rows per 1 KB
  constexpr int kCB = DC / 16, kKS = (DC + 31) / 32;  // blocks of 16 channels, steps of 32
  __shared__ __attribute__((aligned(1024))) unsigned char sm[2 * ST * kTile];  // K tiles, V tiles

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int head = blockIdx.x % a.hk;
  // the last slots first: a causal sequence's longest rows are its last
  const int64_t slot = (int64_t)(gridDim.x / a.hk) - 1 - blockIdx.x / a.hk;
  const Sequence sq = sequence_of<kBM>(a, slot, lane);
  if (sq.index < 0) return;
  const int64_t q0 = sq.q0, q1 = sq.q1, k0 = sq.k0, k1 = sq.k1;
  const int lk = k1 > k0 ? (int)(k1 - k0) : 0;
  const int64_t rows = q1 > q0 ? (q1 - q0) * a.g : 0;
  const int64_t row0 = (slot - (q0 * a.g / kBM + sq.index)) * kBM;
  if (row0 < 0 || row0 >= rows) return;
  const int off = lk - (int)(q1 - q0);  // key of the same age as query 0

  // keys [0, limit) are visible to a row
  auto limit_of = [&](int64_t r) {
    if (!a.causal) return lk;
    const int64_t e = (int64_t)((unsigned)r / (unsigned)a.g) + off + 1;
    return (int)(e < 0 ? 0 : (e < lk ? e : lk));
  };
  const int64_t row_end = row0 + kBM < rows ? row0 + kBM : rows;
  const int keys = limit_of(row_end - 1);
  const int per = (int)cdiv(cdiv(keys, kAKT), a.splits) * kAKT;
  const int kbeg = min(keys, (int)blockIdx.y * per), kend = min(keys, kbeg + per);

  // this lane's rows: r16 of each block of 16
  const int64_t wrow = row0 + wave * 32;
  const bool wave_has = wrow < row_end;
  const int r16 = lane & 15, quad = lane >> 4;
  int64_t tok[2];
  int qh[2], visible[2], lim[2];
  bool valid[2];
#pragma unroll
  for (int rb = 0; rb < 2; ++rb) {
    const int64_t mine = wrow + rb * 16 + r16;
    valid[rb] = mine < row_end;
    const int64_t r = valid[rb] ? mine : row_end - 1;
    tok[rb] = (unsigned)r / (unsigned)a.g;  // nq g < 2^31
    qh[rb] = head * a.g + (int)(r - tok[rb] * a.g);
    visible[rb] = limit_of(r);
    lim[rb] = min(visible[rb], kend);
  }
  // rows ascend within a wave, and so do their limits
  const int lim_first = __builtin_amdgcn_readfirstlane(lim[0]);
  const int lim_last = wave_has ? __builtin_amdgcn_readlane(lim[1], 15) : 0;

  bf16x8_t qf[kKS][2];
#pragma unroll
  for (int rb = 0; rb < 2; ++rb) {
    const unsigned short* qp = a.q + (q0 + tok[rb]) * a.q_token + qh[rb] * a.q_head;
#pragma unroll
    for (int st = 0; st < kKS; ++st) {
      const int e = st * 32 + quad * 8;
      u32x4_t u = u32x4_t{0u, 0u, 0u, 0u};
      if (e < a.d) u = *(const u32x4_t*)(qp + e);
      qf[st][rb] = __builtin_bit_cast(bf16x8_t, u);
    }
  }

  f32x4_t o[kCB][2];
  float m[2], l[2];
  unsigned bad = 0;  // sign bits: V values met that are not finite, in tiles with hidden keys

  // Loader: chunk wave + NW i of a tile (1 KB, kRowsPer rows); lane l fills row
  // kRowsPer chunk + l / kPieces at physical piece l % kPieces. K pieces are
  // swizzled by the row so that 16 rows at one piece spread over all banks, V
  // pieces so that 8 rows x 32 bytes do; either is the same in a lane's chunks.
  const int lr = lane / kPieces, lpp = lane % kPieces;
  const int row_w = wave * kRowsPer + lr;  // + NW i kRowsPer
  const int swk = D == 128 ? (row_w & 15) : ((row_w >> 1) & 7);
  const int swv = D == 128 ? ((row_w & 7) << 1) : (((row_w >> 1) & 3) << 1);
  static_assert(D == 64 || NW * kRowsPer % 16 == 0, "one K swizzle per lane");
  const int ck = (lpp ^ swk) * 8;
  int cv = (lpp ^ swv) * 8;
  const unsigned short* kb = a.k + k0 * a.k_token + head * a.k_head;
  const unsigned short* vb = a.v + k0 * a.v_token + head * a.v_head;
  // K's pieces past the head are zero in every tile and never loaded; V's repeat its
  // first piece: they make channels that are not stored
  const bool in_k = !PAD || ck < a.d;
  if (PAD && cv >= a.d) cv = 0;
  if constexpr (PAD) {
    for (int i = tid; i < ST * kAKT * kPieces; i += 64 * NW) {
      const int row = i / kPieces, piece = i % kPieces;
      if (piece * 8 >= a.d)
        *(u32x4_t*)(sm + row * kRowB + ((piece ^ (D == 128 ? (row & 15) : ((row >> 1) & 7))) << 4)) =
            u32x4_t{0u, 0u, 0u, 0u};
    }
  }
  const unsigned smb = lds_address(sm);
  // byte offsets from the tile's first key (64 rows of less than 2^24 elements)
  unsigned vk[kLd], vv[kLd];
  auto offsets = [&](int last) {  // rows past `last` read that one: they are masked
#pragma unroll
    for (int i = 0; i < kLd; ++i) {
      const unsigned row = min(row_w + NW * i * kRowsPer, last);
      vk[i] = (row * (unsigned)a.k_token + ck) * 2;
      vv[i] = (row * (unsigned)a.v_token + cv) * 2;
    }
  };
  // The next tile's loads, one by one: i < kLd of K, then kLd of V.
  const unsigned short *gk = kb, *gv = vb;
  unsigned dk = 0;
  auto next_tile = [&](int kt, int buf) {
    if (kt + kAKT > lk) offsets(lk - 1 - kt);  // the sequence's last tile
    gk = kb + (int64_t)kt * a.k_token;
    gv = vb + (int64_t)kt * a.v_token;
    dk = smb + buf * kTile + wave * 1024;
  };
  auto load = [&](int i) {
    if (i < kLd) {
      if (in_k) lds_dma1(vk[i], gk, dk + i * NW * 1024);
    } else {
      lds_dma1(vv[i - kLd], gv, dk + ST * kTile + (i - kLd) * NW * 1024);
    }
  };

  // operand addresses inside a tile; the step's piece bits are XORed in
  const int kswz = D == 128 ? r16 : ((r16 >> 1) & 7);
  const int kaddr = r16 * kRowB + ((quad ^ kswz) << 4);
  const int vkey = 4 * quad + (r16 >> 2);
  const int vswz = D == 128 ? ((vkey & 7) << 1) : (((vkey >> 1) & 3) << 1);
  const int vaddr = vkey * kRowB + ((((r16 & 3) >> 1) ^ vswz) << 4) + (r16 & 1) * 8;

  const unsigned char *ks, *vs;  // the tile at hand
  // channels 16 cb + r16 of 32 keys from 32 kc: 4 quad + x, then 16 + 4 quad + x
  auto v_frag = [&](int kc, int cb) {
    const unsigned char* p = vs + kc * 32 * kRowB + (vaddr ^ (cb << 5));
    const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) v4i16_t*)p);
    const v4i16_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) v4i16_t*)(p + 16 * kRowB));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  // One tile of 64 keys from kt.
  auto tile = [&](int kt, bool more, auto CAREFUL) __attribute__((always_inline)) {
    constexpr bool careful = decltype(CAREFUL)::value;
    // Scores of four blocks of 16 keys: operands are read a step ahead, the next tile's
    // loads go between the products; the order is pinned.
    f32x4_t s[4][2];
    bf16x8_t kf[2][4];
    auto read_k = [&](int st, int kb16) {
      kf[st & 1][kb16] = *(const bf16x8_t*)(ks + kb16 * 16 * kRowB + (kaddr ^ (st << 6)));
    };
    auto scores = [&](auto LOADS) __attribute__((always_inline)) {
#pragma unroll
      for (int kb16 = 0; kb16 < 4; ++kb16) read_k(0, kb16);
#pragma unroll
      for (int st = 0; st < kKS; ++st) {
#pragma unroll
        for (int kb16 = 0; kb16 < 4; ++kb16) {
          if (st + 1 < kKS) read_k(st + 1, kb16);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int rb = 0; rb < 2; ++rb) {
            const f32x4_t zero = {};
            s[kb16][rb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                kf[st & 1][kb16], qf[st][rb], st ? s[kb16][rb] : zero, 0, 0, 0);
          }
          __builtin_amdgcn_sched_barrier(0);
          if constexpr (decltype(LOADS)::value) {
#pragma unroll
            for (int i = 0; i < 2 * kLd; ++i)
              if (i * 4 * kKS / (2 * kLd) == st * 4 + kb16) load(i);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
    };
    if (more)
      scores(std::integral_constant<bool, true>{});
    else
      scores(std::integral_constant<bool, false>{});
    const bool masked = kt + kAKT > lim_first;  // some row of the wave does not see every key
    if (masked) {
#pragma unroll
      for (int kb16 = 0; kb16 < 4; ++kb16)
#pragma unroll
        for (int rb = 0; rb < 2; ++rb)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[kb16][rb][e] =
                kt + kb16 * 16 + 4 * quad + e < lim[rb] ? s[kb16][rb][e] : -INFINITY;
      if constexpr (!careful) {
#pragma unroll 1
        for (int kc = 0; kc < 2; ++kc) {
          if (kt + 32 * kc + 32 <= lim_first) continue;  // every row sees these keys
#pragma unroll
          for (int cb = 0; cb < kCB; ++cb) {
            const u32x4_t u = __builtin_bit_cast(u32x4_t, v_frag(kc, cb));
            // an exponent of all ones, plus one in its last place, sets the sign bit
#pragma unroll
            for (int x = 0; x < 4; ++x) bad |= (u[x] & 0x7f807f80u) + 0x00800080u;
          }
        }
      }
    }
    // the first half of V is under way during the softmax
    v8i16_t vf[kCB];
#pragma unroll
    for (int cb = 0; cb < kCB; ++cb) vf[cb] = v_frag(0, cb);
    float top[2];
#pragma unroll
    for (int rb = 0; rb < 2; ++rb) top[rb] = fmaxf(s[2][rb][0], s[3][rb][0]);
    // the ordinary maxima above wait for the last products, which come after all others
#pragma unroll
    for (int rb = 0; rb < 2; ++rb) {
      top[rb] = max3(top[rb], s[0][rb][0], s[1][rb][0]);
#pragma unroll
      for (int e = 1; e < 4; ++e) {
        top[rb] = max3(top[rb], s[0][rb][e], s[1][rb][e]);
        top[rb] = max3(top[rb], s[2][rb][e], s[3][rb][e]);
      }
      top[rb] = quad_max(top[rb]) * a.c;
    }
    if (__any(top[0] > m[0] + kAMove || top[1] > m[1] + kAMove)) {  // also the first tile
#pragma unroll
      for (int rb = 0; rb < 2; ++rb) {
        const float mn = fmaxf(m[rb], top[rb]);
        const float f = exp2_fast(m[rb] - (mn == -INFINITY ? 0.f : mn));
        l[rb] *= f;
#pragma unroll
        for (int cb = 0; cb < kCB; ++cb)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[cb][rb][e] *= f;
        m[rb] = mn;
      }
    }
    bf16x8_t pf[2][2];
#pragma unroll
    for (int rb = 0; rb < 2; ++rb) {
      const float ref = m[rb] == -INFINITY ? 0.f : -m[rb];
#pragma unroll
      for (int kb16 = 0; kb16 < 4; ++kb16)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const bf16x2_t p = pack2(exp2_fast(fmaf(s[kb16][rb][2 * x], a.c, ref)),
                                   exp2_fast(fmaf(s[kb16][rb][2 * x + 1], a.c, ref)));
          // the sum takes the rounded weights, which are the ones that V meets
          l[rb] = __builtin_amdgcn_fdot2_f32_bf16(p, bf16x2_t{(__bf16)1.0f, (__bf16)1.0f}, l[rb],
                                                  false);
          pf[kb16 >> 1][rb][(kb16 & 1) * 4 + 2 * x] = p[0];
          pf[kb16 >> 1][rb][(kb16 & 1) * 4 + 2 * x + 1] = p[1];
        }
    }
    if constexpr (careful) {
      if (masked) {
#pragma unroll
        for (int kc = 0; kc < 2; ++kc)
#pragma unroll
          for (int cb = 0; cb < kCB; ++cb) {
            const v8i16_t vx = v_frag(kc, cb);
#pragma unroll 1
            for (int j = 0; j < 32; ++j) {  // element j % 8 of lanes 16 (j / 8) ..
              const int jq = j >> 3, jx = j & 7;
              const int key = kt + 32 * kc + 4 * jq + (jx & 3) + 16 * (jx >> 2);
              v8i16_t one;
#pragma unroll
              for (int x = 0; x < 8; ++x) one[x] = quad == jq && x == jx ? vx[x] : (short)0;
#pragma unroll
              for (int rb = 0; rb < 2; ++rb) {
                const f32x4_t zero = {};
                const f32x4_t z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf16x8_t, one), pf[kc][rb], zero, 0, 0, 0);
                if (key < lim[rb]) o[cb][rb] += z;
              }
            }
          }
        return;
      }
    }
#pragma unroll
    for (int kc = 0; kc < 2; ++kc)
#pragma unroll
      for (int cb = 0; cb < kCB; ++cb) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int rb = 0; rb < 2; ++rb)
          o[cb][rb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8_t, vf[cb]), pf[kc][rb], o[cb][rb], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
        if (kc == 0) vf[cb] = v_frag(1, cb);
      }
  };

  // One pass over the keys. A hidden key's p is 0, but 0 times an infinity or NaN in its
  // V row is not: the first pass looks through V in tiles with hidden keys, and where it
  // holds such a value the workgroup passes again, taking those tiles' products key by
  // key and keeping them for the rows that see the key.
  auto pass = [&](auto CAREFUL) __attribute__((always_inline)) {
#pragma unroll
    for (int rb = 0; rb < 2; ++rb) {
      m[rb] = -INFINITY;
      l[rb] = 0.f;
#pragma unroll
      for (int cb = 0; cb < kCB; ++cb) o[cb][rb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    offsets(kAKT - 1);
    if (kbeg < kend) {
      next_tile(kbeg, 0);
#pragma unroll
      for (int x = 0; x < 2 * kLd; ++x) load(x);
    }
    int buf = 0;
    for (int kt = kbeg; kt < kend; kt += kAKT) {
      __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this tile has landed
      __syncthreads();  // the buffer filled next was last read before this barrier
      const bool more = kt + kAKT < kend;
      if (more) next_tile(kt + kAKT, buf ^ 1);
      ks = sm + buf * kTile;
      vs = sm + (ST + buf) * kTile;
      buf ^= 1;
      if (kt < lim_last) {
        tile(kt, more, CAREFUL);
      } else if (more) {  // no row of this wave sees the tile
#pragma unroll
        for (int x = 0; x < 2 * kLd; ++x) load(x);
      }
    }
  };
  pass(std::integral_constant<bool, false>{});
  if (__syncthreads_or((bad & 0x80008000u) != 0)) {
    pass(std::integral_constant<bool, true>{});
    __syncthreads();  // a wave that is done puts its rows over tiles that others still read
  }

#pragma unroll
  for (int rb = 0; rb < 2; ++rb) {
    l[rb] += __shfl_xor(l[rb], 16);
    l[rb] += __shfl_xor(l[rb], 32);
  }
  // element 4 quad + e of each block of 16 is in register e
  if (a.splits > 1) {
#pragma unroll
    for (int rb = 0; rb < 2; ++rb) {
      if (!valid[rb]) continue;
      const int64_t at = ((int64_t)blockIdx.y * a.nq + q0 + tok[rb]) * (a.hk * a.g) + qh[rb];
      // l = -1 marks a piece that saw keys, all of them with scores of -inf
      if (quad == 0)
        a.part_ml[at] = make_float2(m[rb], lim[rb] > kbeg && l[rb] == 0.f ? -1.f : l[rb]);
      if (kbeg >= kend) continue;
#pragma unroll
      for (int cb = 0; cb < kCB; ++cb) {
        const int e = cb * 16 + 4 * quad;
        if (e < a.d) *(f32x4_t*)(a.part_o + at * a.d + e) = o[cb][rb];
      }
    }
    return;
  }
  // Through LDS (free: every pass ends at a barrier), so that a store instruction writes
  // whole rows: 4 elements per lane of 32 rows each took 4.5 us per round of workgroups.
  constexpr int kOutB = kRowB + 16;  // row pitch: rows 4 banks apart
  static_assert(NW * 32 * kOutB <= 2 * ST * kTile, "rows fit the tiles");
  unsigned char* ob = sm + wave * 32 * kOutB;
#pragma unroll
  for (int rb = 0; rb < 2; ++rb) {
    const bool any = visible[rb] > 0;
    const float inv = any ? 1.0f / l[rb] : 0.f;
#pragma unroll
    for (int cb = 0; cb < kCB; ++cb) {
      bf16x2_t w[2];
#pragma unroll
      for (int y = 0; y < 2; ++y)
        w[y] = any ? pack2(o[cb][rb][2 * y] * inv, o[cb][rb][2 * y + 1] * inv) : pack2(0.f, 0.f);
      *(bf16x4_t*)(ob + (rb * 16 + r16) * kOutB + (cb * 16 + 4 * quad) * 2) =
          __builtin_shufflevector(w[0], w[1], 0, 1, 2, 3);
    }
  }
  wave_sync();
  const int rows_here = (int)(row_end - wrow);  // of this wave's 32
#pragma unroll 1
  for (int r0 = 0; r0 < 32; r0 += kRowsPer) {
    const int rr = r0 + lr;  // of one block of 16: kRowsPer divides it
    const int64_t t = q0 + (unsigned)__shfl((int)(r0 < 16 ? tok[0] : tok[1]), rr & 15);
    const int hh = __shfl(r0 < 16 ? qh[0] : qh[1], rr & 15);
    if (rr < rows_here && lpp * 8 < a.d)
      *(u32x4_t*)(a.o + t * a.o_token + hh * a.o_head + lpp * 8) =
          *(const u32x4_t*)(ob + rr * kOutB + lpp * 16);
  }
}

// Few rows (single tokens over a cache): a workgroup takes 32 rows of one sequence and
// key head, and its four waves every fourth tile of 32 keys, each with two tiles of its
// own in LDS and no barrier in the loop; their (m, l, O) meet in LDS at the end. Bound
// by reading K and V; against 128-row workgroups, whose other three waves had no rows,
// a token over 300 keys of 32 heads went from 12.5 to 10.8 us (10.2 now). 16 tokens over
// 300001 keys, 64 heads on 8: 264 us (4.7 TB/s) and 6 for the join. Products of 32x32x16 (their lanes
// hold one query, so the softmax exchanges once). The weights enter the second product as
// a bf16 value and its rest, so 2^-16 of each is lost and not 2^-8 (error against 64 bits
// 1.65e-3 rms, the output's own rounding, instead of 2.14e-3; 3% more time, as the matrix
// cores are 9% busy). Everything else is as above.
template <int D, int DC, bool PAD>
__global__ __launch_bounds__(256, 1) void attention_few_kernel(AttnArgs a) {
  constexpr int kBM = 32, kKeys = 32, kWaves = 4;
  constexpr int kPieces = D / 8, kRowB = D * 2;
  constexpr int kTile = kKeys * kRowB;     // one operand's tile
  constexpr int kLd = kTile / 1024;        // 1 KB loads per operand
  constexpr int kRowsPer = 64 / kPieces;
  constexpr int kDB = DC / 32, kKS = DC / 16;
  constexpr int kOutW = D + 4;             // row pitch of the joined O, floats
  static_assert(32 * kOutW * 4 <= 4 * kTile, "O fits a wave's tiles");
  __shared__ __attribute__((aligned(1024))) unsigned char sm[kWaves * 4 * kTile];
  __shared__ float sm_m[kWaves][32], sm_l[kWaves][32];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int head = blockIdx.x % a.hk;
  const int64_t slot = (int64_t)(gridDim.x / a.hk) - 1 - blockIdx.x / a.hk;
  const Sequence sq = sequence_of<kBM>(a, slot, lane);
  if (sq.index < 0) return;
  const int64_t q0 = sq.q0, q1 = sq.q1, k0 = sq.k0, k1 = sq.k1;
  const int lk = k1 > k0 ? (int)(k1 - k0) : 0;
  const int64_t rows = q1 > q0 ? (q1 - q0) * a.g : 0;
  const int64_t row0 = (slot - (q0 * a.g / kBM + sq.index)) * kBM;
  if (row0 < 0 || row0 >= rows) return;
  const int off = lk - (int)(q1 - q0);
  auto limit_of = [&](int64_t r) {
    if (!a.causal) return lk;
    const int64_t e = (int64_t)((unsigned)r / (unsigned)a.g) + off + 1;
    return (int)(e < 0 ? 0 : (e < lk ? e : lk));
  };
  const int64_t row_end = row0 + kBM < rows ? row0 + kBM : rows;
  const int keys = limit_of(row_end - 1);
  const int per = (int)cdiv(cdiv(keys, kKeys), a.splits) * kKeys;
  const int kbeg = min(keys, (int)blockIdx.y * per), kend = min(keys, kbeg + per);
  const int64_t mine = row0 + (lane & 31);
  const int64_t r = mine < row_end ? mine : row_end - 1;
  const int64_t tok = (unsigned)r / (unsigned)a.g;
  const int qh = head * a.g + (int)(r - tok * a.g);
  const int lim = min(limit_of(r), kend);
  const int lim_first = __builtin_amdgcn_readfirstlane(lim);
  const int half = lane >> 5;

  bf16x8_t qf[kKS];
  {
    const unsigned short* qp = a.q + (q0 + tok) * a.q_token + qh * a.q_head;
#pragma unroll
    for (int st = 0; st < kKS; ++st) {
      const int e = st * 16 + half * 8;
      u32x4_t u = u32x4_t{0u, 0u, 0u, 0u};
      if (e < a.d) u = *(const u32x4_t*)(qp + e);
      qf[st] = __builtin_bit_cast(bf16x8_t, u);
    }
  }

  // Loader: load i fills rows kRowsPer i .. of the wave's own tile, pieces swizzled as
  // above.
  unsigned char* own = sm + wave * 4 * kTile;  // K0 V0 K1 V1
  auto k_swizzle = [](int row) { return D == 128 ? (row & 15) : ((row >> 1) & 7); };
  if constexpr (PAD) {
#pragma unroll
    for (int b = 0; b < 2; ++b)
      for (int i = lane; i < kKeys * kPieces; i += 64) {
        const int row = i / kPieces, piece = i % kPieces;
        if (piece * 8 >= a.d)
          *(u32x4_t*)(own + 2 * b * kTile + row * kRowB + ((piece ^ k_swizzle(row)) << 4)) =
              u32x4_t{0u, 0u, 0u, 0u};
      }
    wave_sync();
  }
  const int lr = lane / kPieces, lpp = lane % kPieces;
  auto k_piece = [&](int i) { return (lpp ^ k_swizzle(i * kRowsPer + lr)) * 8; };
  int cv = (lpp ^ (D == 128 ? ((lr & 3) << 2) : (((lr >> 1) & 1) << 2))) * 8;
  const unsigned short* kb = a.k + k0 * a.k_token + head * a.k_head;
  if (PAD && cv >= a.d) cv = 0;
  const unsigned short* vb = a.v + k0 * a.v_token + head * a.v_head;
  const unsigned ob = lds_address(sm) + wave * 4 * kTile;
  auto issue = [&](int kt, int buf) {
    const unsigned short* gk = kb + (int64_t)kt * a.k_token;
    const unsigned short* gv = vb + (int64_t)kt * a.v_token;
    const int last = min(kKeys, lk - kt) - 1;  // rows past the keys read the last: masked
#pragma unroll
    for (int i = 0; i < kLd; ++i) {
      const unsigned row = min(i * kRowsPer + lr, last);
      const int ck = k_piece(i);
      if (!PAD || ck < a.d)
        lds_dma1((row * (unsigned)a.k_token + ck) * 2, gk, ob + 2 * buf * kTile + i * 1024);
    }
#pragma unroll
    for (int i = 0; i < kLd; ++i) {
      const unsigned row = min(i * kRowsPer + lr, last);
      lds_dma1((row * (unsigned)a.v_token + cv) * 2, gv, ob + (2 * buf + 1) * kTile + i * 1024);
    }
  };
  const int krow = lane & 31;
  const int kswz = D == 128 ? (krow & 15) : ((krow >> 1) & 7);
  const int kaddr = krow * kRowB + ((half ^ kswz) << 4);
  const int s16 = lane & 15;
  const int vkey = 4 * half + (s16 >> 2);
  const int vswz = D == 128 ? ((vkey & 3) << 2) : (((vkey >> 1) & 1) << 2);
  const int vpiece = 2 * ((lane >> 4) & 1) + ((s16 & 3) >> 1);
  const int vaddr = vkey * kRowB + ((vpiece ^ vswz) << 4) + (s16 & 1) * 8;

  f32x16_t o[kDB];
  float m, l;
  unsigned bad = 0;
  auto tile = [&](int kt, int buf, auto CAREFUL) __attribute__((always_inline)) {
    constexpr bool careful = decltype(CAREFUL)::value;
    const unsigned char* ks = own + 2 * buf * kTile;
    const unsigned char* vs = ks + kTile;
    auto v_frag = [&](int ks16, int db) {
      const unsigned char* p = vs + ks16 * 16 * kRowB + (vaddr ^ (db << 6));
      const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) v4i16_t*)p);
      const v4i16_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) v4i16_t*)(p + 8 * kRowB));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    f32x16_t s2[2] = {{}, {}};  // two chains of products
#pragma unroll
    for (int st = 0; st < kKS; ++st) {
      const bf16x8_t kf = *(const bf16x8_t*)(ks + (kaddr ^ (st << 5)));
      s2[st & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[st], s2[st & 1], 0, 0, 0);
    }
    f32x16_t s;
#pragma unroll
    for (int e = 0; e < 16; ++e) s[e] = s2[0][e] + s2[1][e];
    const bool masked = kt + kKeys > lim_first;
    if (masked) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        s[e] = kt + 8 * (e >> 2) + 4 * half + (e & 3) < lim ? s[e] : -INFINITY;
      if constexpr (!careful) {
#pragma unroll
        for (int ks16 = 0; ks16 < 2; ++ks16)
#pragma unroll
          for (int db = 0; db < kDB; ++db) {
            const u32x4_t u = __builtin_bit_cast(u32x4_t, v_frag(ks16, db));
#pragma unroll
            for (int x = 0; x < 4; ++x) bad |= (u[x] & 0x7f807f80u) + 0x00800080u;
          }
      }
    }
    float top = s[0];
#pragma unroll
    for (int e = 1; e < 16; ++e) top = fmaxf(top, s[e]);
    top = half_max(top) * a.c;
    if (__any(top > m + kAMove)) {
      const float mn = fmaxf(m, top);
      const float f = exp2_fast(m - (mn == -INFINITY ? 0.f : mn));
      l *= f;
#pragma unroll
      for (int i = 0; i < kDB; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[i][e] *= f;
      m = mn;
    }
    const float ref = m == -INFINITY ? 0.f : -m;
    bf16x8_t pf[2], pr[2];  // the weights and what their rounding left
#pragma unroll
    for (int ks16 = 0; ks16 < 2; ++ks16) {
      u32x4_t wf, wr;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int e = ks16 * 8 + 2 * x;
        const float p0 = exp2_fast(fmaf(s[e], a.c, ref)), p1 = exp2_fast(fmaf(s[e + 1], a.c, ref));
        l += p0 + p1;
        wf[x] = __builtin_bit_cast(unsigned, pack2(p0, p1));
        wr[x] = __builtin_bit_cast(unsigned, pack2(p0 - __uint_as_float(wf[x] << 16),
                                                   p1 - __uint_as_float(wf[x] & 0xffff0000u)));
      }
      pf[ks16] = __builtin_bit_cast(bf16x8_t, wf);
      pr[ks16] = __builtin_bit_cast(bf16x8_t, wr);
    }
    if constexpr (careful) {
      if (masked) {
#pragma unroll
        for (int ks16 = 0; ks16 < 2; ++ks16)
#pragma unroll
          for (int db = 0; db < kDB; ++db) {
            const v8i16_t vx = v_frag(ks16, db);
#pragma unroll 1
            for (int j = 0; j < 16; ++j) {
              const int jh = (j >> 2) & 1, jx = (j & 3) + 4 * (j >> 3);
              v8i16_t one;
#pragma unroll
              for (int x = 0; x < 8; ++x) one[x] = half == jh && x == jx ? vx[x] : (short)0;
              const f32x16_t zero = {};
              const f32x16_t z = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                  __builtin_bit_cast(bf16x8_t, one), pf[ks16], zero, 0, 0, 0);
              const f32x16_t y = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                  __builtin_bit_cast(bf16x8_t, one), pr[ks16], zero, 0, 0, 0);
              if (kt + 16 * ks16 + j < lim) {
#pragma unroll
                for (int e = 0; e < 16; ++e) o[db][e] += z[e] + (isfinite(y[e]) ? y[e] : 0.f);
              }
            }
          }
        return;
      }
    }
#pragma unroll
    for (int ks16 = 0; ks16 < 2; ++ks16)
#pragma unroll
      for (int db = 0; db < kDB; ++db)
        {
          const bf16x8_t vf = __builtin_bit_cast(bf16x8_t, v_frag(ks16, db));
          o[db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pf[ks16], o[db], 0, 0, 0);
          if constexpr (careful) {
            const f32x16_t zero = {};
            const f32x16_t y = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pr[ks16], zero, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[db][e] += isfinite(y[e]) ? y[e] : 0.f;
          } else {
            o[db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pr[ks16], o[db], 0, 0, 0);
          }
        }
  };
  auto pass = [&](auto CAREFUL) __attribute__((always_inline)) {
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < kDB; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[i][e] = 0.f;
    constexpr int step = kWaves * kKeys;
    int kt = kbeg + wave * kKeys, buf = 0;
    if (kt < kend) issue(kt, 0);
    for (; kt < kend; kt += step, buf ^= 1) {
      if (kt + step < kend) {
        // the other buffer's reads are done before it is filled again
        __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        issue(kt + step, buf ^ 1);
        if constexpr (kLd == 8)
          __asm__ volatile("s_waitcnt vmcnt(16)" ::: "memory");
        else
          __asm__ volatile("s_waitcnt vmcnt(8)" ::: "memory");
      } else {
        __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
      }
      tile(kt, buf, CAREFUL);
    }
  };
  static_assert(kLd == 8 || kLd == 4, "vmcnt immediates");
  pass(std::integral_constant<bool, false>{});
  // An infinity that a row sees stays one times p, but is NaN times p's rest (0, or of the
  // other sign): where anything is not finite, the second pass leaves such products of the
  // rests out.
  float zeros[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kDB; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) zeros[e & 3] = fmaf(o[i][e], 0.f, zeros[e & 3]);
  const float zero = (zeros[0] + zeros[1]) + (zeros[2] + zeros[3]);
  if (__syncthreads_or((bad & 0x80008000u) != 0 || zero != 0.f)) {
    pass(std::integral_constant<bool, true>{});
    __syncthreads();
  }

  // Join of the waves: each puts its O (32 rows) over its own tiles.
  l += __shfl_xor(l, 32);
  float* po = (float*)own;
#pragma unroll
  for (int db = 0; db < kDB; ++db)
#pragma unroll
    for (int x = 0; x < 4; ++x)
      *(f32x4_t*)(po + (lane & 31) * kOutW + db * 32 + 8 * x + 4 * half) =
          f32x4_t{o[db][4 * x], o[db][4 * x + 1], o[db][4 * x + 2], o[db][4 * x + 3]};
  if (half == 0) {
    sm_m[wave][lane] = m;
    sm_l[wave][lane] = l;
  }
  __syncthreads();
  const int rr = tid >> 3;  // eight threads per row
  if (row0 + rr >= row_end) return;
  const int64_t rg = row0 + rr;
  const int64_t ot = (unsigned)rg / (unsigned)a.g;
  const int oh = head * a.g + (int)(rg - ot * a.g);
  const int vis = limit_of(rg);
  float mt = -INFINITY, lt = 0.f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) mt = fmaxf(mt, sm_m[w][rr]);
  const float rt = mt == -INFINITY ? 0.f : mt;
  float f[kWaves];
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    // a wave whose scores were all -inf (or that saw no key) weighs nothing, a NaN stays
    const float lw = sm_l[w][rr];
    f[w] = lw == 0.f ? 0.f : exp2_fast(sm_m[w][rr] - rt);
    lt += lw * f[w];
  }
  const int64_t at = ((int64_t)blockIdx.y * a.nq + q0 + ot) * (a.hk * a.g) + oh;
  if (a.splits > 1 && (tid & 7) == 0)
    a.part_ml[at] = make_float2(mt, min(vis, kend) > kbeg && lt == 0.f ? -1.f : lt);
  const float inv = vis > 0 ? 1.0f / lt : 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {  // elements 4 (tid % 8) + 32 i
    const int e = (tid & 7) * 4 + 32 * i;
    if (e >= a.d) break;
    f32x4_t v = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
      if (f[w] != 0.f)
        v += *(const f32x4_t*)((const float*)(sm + w * 4 * kTile) + rr * kOutW + e) * f[w];
    if (a.splits > 1) {
      *(f32x4_t*)(a.part_o + at * a.d + e) = v;
    } else {
      const bf16x2_t w0 = vis > 0 ? pack2(v[0] * inv, v[1] * inv) : pack2(0.f, 0.f);
      const bf16x2_t w1 = vis > 0 ? pack2(v[2] * inv, v[3] * inv) : pack2(0.f, 0.f);
      *(bf16x4_t*)(a.o + (q0 + ot) * a.o_token + oh * a.o_head + e) =
          __builtin_shufflevector(w0, w1, 0, 1, 2, 3);
    }
  }
}

// Joins the splits of the (token, query head) rows, groups of 32 lanes (4 elements
// each): a group per row for many rows of few splits, else eight groups to a row, each
// taking every eighth split; their sums are added in order. (Measured when they were
// built: 512 queries of 32 heads in two splits 19.4 us with a group per row, 29.6 with
// eight; 16 of 64 heads in eight, the other way round, 278 and 272.)
constexpr int kAJoinSplits = 8, kAJoinRows = 2048;

template <bool FEW>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a) {
  __shared__ float part[FEW ? 1 : 8][132];  // 128 elements, l, any
  const int grp = threadIdx.x / 32, lane = threadIdx.x & 31, e = lane * 4;
  const int hq = a.hk * a.g;
  const int64_t row = FEW ? (int64_t)blockIdx.x * 8 + grp : blockIdx.x;
  const int64_t tok = row / hq;
  const int qh = (int)(row - tok * hq);
  if (tok < start_at(a.q_start, 0, a.nq) || tok >= start_at(a.q_start, a.nseq, a.nq)) return;
  const int64_t step = a.nq * hq;
  float m = -INFINITY;
  for (int s = lane; s < a.splits; s += 32) m = fmaxf(m, a.part_ml[s * step + row].x);
#pragma unroll
  for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor(m, x, 32));
  const float ref = m == -INFINITY ? 0.f : m;
  f32x4_t o = f32x4_t{0.f, 0.f, 0.f, 0.f};
  float l = 0.f, any = 0.f;
  for (int s = FEW ? 0 : grp; s < a.splits; s += FEW ? 1 : 8) {
    const float2 ml = a.part_ml[s * step + row];
    if (ml.y != 0.f) any = 1.f;  // 0: the piece saw no key
    if (ml.y <= 0.f) continue;   // -1: only scores of -inf
    const float f = exp2_fast(ml.x - ref);
    l += ml.y * f;
    if (e < a.d) o += *(const f32x4_t*)(a.part_o + (s * step + row) * a.d + e) * f;
  }
  if constexpr (!FEW) {
#pragma unroll
    for (int y = 0; y < 4; ++y) part[grp][e + y] = o[y];
    if (lane == 0) {
      part[grp][128] = l;
      part[grp][129] = any;
    }
    __syncthreads();
    if (grp) return;
    for (int s = 1; s < 8; ++s) {
#pragma unroll
      for (int y = 0; y < 4; ++y) o[y] += part[s][e + y];
    }
    l = 0.f;
    any = 0.f;
    for (int s = 0; s < 8; ++s) {
      l += part[s][128];
      any += part[s][129];
    }
  }
  if (e >= a.d) return;
  // keys seen, but every score -inf: l is 0 and there is no softmax (NaN)
  u16x4_t w;
#pragma unroll
  for (int y = 0; y < 4; ++y) w[y] = any > 0.f ? f32_to_bf16_rne(o[y] / l) : (unsigned short)0;
  *(u16x4_t*)(a.o + tok * a.o_token + qh * a.o_head + e) = w;
}

template <int D, int DC, bool PAD>
void launch_kernel(const AttnArgs& a, hipStream_t s) {
  const int64_t slots = a.nq * a.g / 128 + a.nseq;
  hipLaunchKernelGGL((attention_kernel<D, DC, PAD>),
                     dim3((unsigned)(slots * a.hk), (unsigned)a.splits), dim3(256), 0, s, a);
}

template <int D, int DC, bool PAD>
void launch_few(const AttnArgs& a, hipStream_t s) {
  const int64_t slots = a.nq * a.g / 32 + a.nseq;
  hipLaunchKernelGGL((attention_few_kernel<D, DC, PAD>),
                     dim3((unsigned)(slots * a.hk), (unsigned)a.splits), dim3(256), 0, s, a);
}

constexpr int kAUnits = 256;  // compute units

struct AttnPlan {
  bool few;    // 32-row workgroups whose waves share the keys
  int splits;  // pieces of the keys
};

// By the sequences' average lengths, all that the host knows. Up to 32 rows a sequence
// the call is bound by reading the keys: the few-rows kernel (one workgroup per compute
// unit at a time), its keys in pieces of 320 or more while those do not fill the units,
// else of 512 or more up to four rounds, which even out the sequences' lengths. (16
// sequences over 300001 keys, lengths up to a factor of ten apart, 8 key heads: 286, 272,
// 294, 335 us in 4, 8, 16, 32 pieces, eight being taken; of equal lengths 215 in two, 236
// in eight. One over 512 keys, 32 heads: 11.7 us whole, as taken, 10.9 in eight; over
// 1024: 16.8 whole, 13.6 in three, as taken, 11.4 in eight; over 32768 keys, one head:
// 19 us in 64 pieces, 22 in 32.)
// With more rows the products bound it, and the pieces' results cost: the number of pieces
// with the least modelled time. A workgroup takes 7 us and 1.25 a tile of 64 keys where it
// has a compute unit for itself, 1.6 where two share it; more than two take turns, the
// longest or the average one (causal: half of the newest keys) setting the time; pieces are
// joined in 3 us and at 4 TB/s. (One sequence, whole and in pieces: 512 tokens, 32 heads of
// 64, 13.6 us and 18.9 in two; 1024, 32 of 128, 29 and 39; 2048, 8 of 128 on 2, 46 and 36 in
// four; 4096, 8 of 96 on 1, 77 and 62 in three; 300 over 20000 keys, 16 of 128 on 4, 388 and
// 73 in twelve. Of ten shapes, all came within 4% of the best of twelve numbers.)
// Batches that the averages misjudge take as long as their worst sequence, and are better
// called in parts: one token over 100000 keys among 63 over 100, 64 heads on 8: 662-677 us,
// 94 and 16 in two calls; over 20000 among 63 over 2000: 207-248, 37 and 118; a prompt of
// 4000 tokens among 255 single ones over 1000 keys, 32 heads: 1228-1279, 148 and 784-828
// (on 8 key heads 349, 144 and 213).
AttnPlan plan_of(const th_attention_params* p) {
  const int64_t g = p->hq / p->hk;
  const int64_t seqs = p->nseq < p->nq ? p->nseq : p->nq;
  const int64_t tokens = cdiv(p->nq, seqs), rows = tokens * g, keys = cdiv(p->nk, seqs);
  AttnPlan r;
  r.few = rows <= 32;
  const int64_t groups = seqs * cdiv(rows, r.few ? 32 : 128) * p->hk;
  if (r.few) {
    auto pieces = [&](int64_t workgroups, int64_t least) {
      const int64_t s = workgroups / groups < keys / least ? workgroups / groups : keys / least;
      return s < 1 ? (int64_t)1 : (s > 64 ? (int64_t)64 : s);
    };
    const int64_t one = pieces(kAUnits, 320), more = pieces(4 * kAUnits, 512);
    r.splits = (int)(one > more ? one : more);
    return r;
  }
  const int64_t tiles = cdiv(keys, kAKT);
  const double seen = p->causal ? (double)keys - 0.5 * (double)(tokens < keys ? tokens : keys)
                                : (double)keys;
  r.splits = 1;
  double least = 1e300;
  for (int s : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64}) {
    if (s > 1 && 3 * s > tiles) break;  // three tiles at least
    const double workgroups = (double)groups * s;
    const double longest = (double)cdiv(tiles, s);
    const double turns = seen / kAKT / s * workgroups / (2 * kAUnits);
    double us = 7.0 + (longest > turns ? longest : turns) * (workgroups <= kAUnits ? 1.25 : 1.6);
    if (s > 1) us += 3.0 + (double)s * (double)(p->nq * p->hq) * (double)(p->d + 2) * 8.0 / 4e6;
    if (us < least) {
      least = us;
      r.splits = s;
    }
  }
  return r;
}

// The pieces' (m, l) of `rows` rows, then their O, which is read and written 16 bytes at a
// time: an odd number of pairs is followed by 8 bytes of nothing.
size_t part_ml_bytes(int64_t rows) { return ((size_t)rows * sizeof(float2) + 15) & ~(size_t)15; }

}  // namespace

int64_t attention_workgroups(const th_attention_params* p) {
  if (p->nq == 0) return 0;
  return (p->nq * (p->hq / p->hk) / (plan_of(p).few ? 32 : 128) + p->nseq) * p->hk;
}

size_t attention_workspace_bytes(const th_attention_params* p) {
  if (p->nq == 0) return 0;
  const int s = plan_of(p).splits;
  if (s == 1) return 0;
  const int64_t rows = s * p->nq * p->hq;
  return part_ml_bytes(rows) + (size_t)rows * p->d * sizeof(float);
}

hipError_t launch_attention(const void* Q, const void* K, const void* V, const int32_t* q_start,
                            const int32_t* k_start, const th_attention_params* p, void* O,
                            void* workspace, hipStream_t s) {
  AttnArgs a;
  a.q = (const unsigned short*)Q;
  a.k = (const unsigned short*)K;
  a.v = (const unsigned short*)V;
  a.o = (unsigned short*)O;
  a.q_token = p->q_token;
  a.q_head = p->q_head;
  a.k_token = p->k_token;
  a.k_head = p->k_head;
  a.v_token = p->v_token;
  a.v_head = p->v_head;
  a.o_token = p->o_token;
  a.o_head = p->o_head;
  a.q_start = q_start;
  a.k_start = k_start;
  a.nq = p->nq;
  a.nk = p->nk;
  a.nseq = (int)p->nseq;
  a.hk = (int)p->hk;
  a.g = (int)(p->hq / p->hk);
  a.d = (int)p->d;
  a.causal = p->causal != 0;
  a.c = (float)(p->scale * 1.4426950408889634);
  const AttnPlan plan = plan_of(p);
  a.splits = workspace ? plan.splits : 1;
  a.part_ml = (float2*)workspace;
  a.part_o = workspace
                 ? (float*)((char*)workspace + part_ml_bytes(a.splits * p->nq * p->hq))
                 : nullptr;
  if (plan.few) {
    if (p->d < 64)
      launch_few<64, 64, true>(a, s);
    else if (p->d == 64)
      launch_few<64, 64, false>(a, s);
    else if (p->d < 128)
      launch_few<128, 128, true>(a, s);
    else
      launch_few<128, 128, false>(a, s);
  } else {
    switch (cdiv(p->d, 16)) {
      case 1:
      case 2: launch_kernel<64, 32, true>(a, s); break;
      case 3: launch_kernel<64, 48, true>(a, s); break;
      case 4:
        if (p->d < 64)
          launch_kernel<64, 64, true>(a, s);
        else
          launch_kernel<64, 64, false>(a, s);
        break;
      case 5: launch_kernel<128, 80, true>(a, s); break;
      case 6: launch_kernel<128, 96, true>(a, s); break;
      case 7: launch_kernel<128, 112, true>(a, s); break;
      default:
        if (p->d < 128)
          launch_kernel<128, 128, true>(a, s);
        else
          launch_kernel<128, 128, false>(a, s);
    }
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t rows = p->nq * p->hq;
  if (a.splits <= kAJoinSplits && rows > kAJoinRows)
    hipLaunchKernelGGL(attention_join_kernel<true>, dim3((unsigned)cdiv(rows, 8)), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL(attention_join_kernel<false>, dim3((unsigned)rows), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace th
