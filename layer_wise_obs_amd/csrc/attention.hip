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
// rms instead of 1.65e-3). Products of what that rounding leaves too would take 673 -> 1079 us
// for 16 sequences of 2048 tokens, 32 heads of 128 (92 registers spill), 90 -> 104 for 24
// prompts, heads of 80. The kernel for few rows below has them.
// Over pages every row has them: p enters as a bf16 value and its rest, also a bf16 value, so that
// 2^-16 of it is lost and not 2^-8 (error against 64 bits 1.66e-3 rms, the output's own rounding,
// instead of 2.2e-3), and a row's precision does not hang on the other sequences of its call.
// Half as many products again: 8 chunks of 4100 tokens over 65600 keys, 32 heads on 8, 636 -> 864 us,
// 4 prompts of 2048 tokens 177 -> 237, one of 512 tokens over 32768 keys 283 -> 383. The weights
// are kept in fp32 and made operands 32 keys at a time, the second 32's beside the last products of the
// first (beside the first ones, 0.5% more): for heads of 128 the loop over the tiles then spills m's
// two registers where they move, and three addresses for the last tile.
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

#include <algorithm>

namespace th {

namespace {

constexpr int kAKT = 64;   // keys per tile
constexpr float kAMove = 8.0f;  // log2 of how far p may pass 1 before m moves
constexpr int kAUnits = 256;  // compute units

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

// A paged cache: K and V are its pages, a key is found through its sequence's row of page
// numbers; k_start has lengths in the place of starts.
struct PagedArgs : AttnArgs {
  const int32_t* pages;
  int64_t pages_row, k_page, v_page, npages;
  int64_t keys_most;  // a sequence's pages hold as many keys
  int64_t each;       // rows of a sequence without q_start
  int shift;          // log2 of a page's keys
  int rows_from, rows_to;  // the kernel takes sequences of so many rows (tokens times the group)
  int slots;          // bound of the pieces' partial results per key head; 0: no keys are cut
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

// ---------------------------------------------------------------- paged: the work

constexpr int kAFewRows = 32;  // rows of a sequence that the few-rows kernel takes in one block

struct PagedWork {
  int sequence;            // -1: none
  int64_t q0, q1;          // its rows of Q
  int lk;                  // its keys
  int64_t row0;            // first row of the block
  int per, piece, pieces;  // keys of a piece, this one and how many there are
  int slot;                // of this piece's partial result, where there are several
};

// Rows, keys, row blocks of sequence s, as the kernel takes them (0 blocks: not its own).
template <int BM>
__device__ __forceinline__ void paged_sequence(const PagedArgs& a, int64_t s, int64_t& q0, int64_t& q1,
                                               int& lk, int& blocks) {
  if (a.q_start) {
    q0 = start_at(a.q_start, (int)s, a.nq);
    q1 = start_at(a.q_start, (int)s + 1, a.nq);
  } else {
    q0 = s * a.each;
    q1 = q0 + a.each;
  }
  const int64_t l = a.k_start[s];
  lk = (int)(l < 0 ? 0 : (l > a.keys_most ? a.keys_most : l));
  const int64_t rows = q1 > q0 ? (q1 - q0) * a.g : 0;
  blocks = rows >= a.rows_from && rows <= a.rows_to ? (int)cdiv(rows, BM) : 0;
}

// Tiles of a piece, from all sequences' real lengths: the tiles of all row blocks are shared out
// over the workgroups that run at a time, two to a compute unit, so that pieces are alike whatever
// the sequences are. (fp32 is off by less than 2^-17 of the sum; the bounds of the pieces' number
// want no fewer.) Few rows: pieces of 320 keys at least; (row block, key head) pairs that leave
// room are cut into as many pieces as run at a time, one short piece each counted; more pairs into
// twice as many, which evens out their lengths; so many that they even out by themselves, where
// one is longer than a workgroup's share. Others: pieces of a workgroup's share, three tiles at least.
// (Shares of a half, a third and a fifth of these were slower over the sequences tried: 64 tokens
// over 300001 keys, chunks of 4100 tokens over 40000, 256 tokens over 1000 each.)
template <int TILE, bool FEW>
__device__ __forceinline__ int paged_per(const PagedArgs& a, float tiles, float blocks) {
  if (a.slots == 0) return 1 << 26;  // more than any sequence has
  const float work = ceilf(tiles * (float)a.hk * (1.0f + 0x1p-16f)), pairs = blocks * (float)a.hk;
  float per;
  if constexpr (FEW) {
    const float at_once = pairs <= kAUnits ? 2 * kAUnits - pairs : (pairs < 6 * kAUnits ? 4 * kAUnits : 2 * kAUnits);
    per = fmaxf(ceilf(work / at_once * (1.0f + 0x1p-20f)), 320 / TILE);
  } else {
    per = fmaxf(ceilf(work * (0.5f / kAUnits)), 3.0f);
  }
  return (int)fminf(per, 0x1p26f);
}

// Inclusive sum over the lanes up to this one, of a full wave: within rows of 16 lanes, then the
// last lane of a row to the next one and of the first half to the second. (Without LDS,
// which shuffles take: 4 prompts of 2048 tokens 180 -> 175 us, 16 tokens over 1000 keys each 65.8 ->
// 63.2, one over 300 12.3 -> 12.1.)
template <class T>
__device__ __forceinline__ T lanes_scan(T v) {
  auto moved = [](T v, auto CONTROL, auto ROWS) __attribute__((always_inline)) {
    return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(CONTROL)::value,
                                                             decltype(ROWS)::value, 0xf, false));
  };
  v += moved(v, std::integral_constant<int, 0x111>{}, std::integral_constant<int, 0xf>{});  // one lane up
  v += moved(v, std::integral_constant<int, 0x112>{}, std::integral_constant<int, 0xf>{});  // two
  v += moved(v, std::integral_constant<int, 0x114>{}, std::integral_constant<int, 0xf>{});
  v += moved(v, std::integral_constant<int, 0x118>{}, std::integral_constant<int, 0xf>{});
  v += moved(v, std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xa>{});  // lane 15 of rows 0, 2
  v += moved(v, std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xc>{});  // lane 31
  return v;
}
__device__ __forceinline__ float lanes_sum(float v) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(lanes_scan(v)), 63));
}

// Piece `at` of the work: sequences in order, their row blocks, the blocks' pieces; BY_SLOT: of
// those only that leave partial results. A lane looks at a sequence.
template <int BM, int TILE, bool FEW, bool BY_SLOT>
__device__ __forceinline__ PagedWork paged_work(const PagedArgs& a, unsigned at, int lane) {
  PagedWork r;
  r.sequence = -1;
  int64_t q0 = 0, q1 = 0;
  int lk = 0, blocks = 0;
  int who = lane;  // the lane's sequence, from s0
  auto look = [&](int s0) {
    blocks = 0;
    if (s0 + lane < a.nseq) paged_sequence<BM>(a, s0 + lane, q0, q1, lk, blocks);
    who = lane;
    if (!FEW && a.nseq > 1 && a.nseq <= 64) {
      // the ones with most keys first: a long piece that begins last keeps the others waiting
      // (chunks of 4100 tokens with weights in one part, 708 -> 652 us; few rows have pieces that are
      // alike). More than 64 are taken as they come: a lane has room for one, and batches that large
      // gain little (called longest first: 65 chunks over 168447 keys, 32 heads on 8, 1671 -> 1632 us, 80
      // over 272687 3516 -> 3456, 120 over 390515 5104 -> 4933).
      const int all = a.nseq;
      int rank = 0;
      for (int j = 0; j < all; ++j) {
        const int other = __builtin_amdgcn_readlane(lk, j);
        rank += other > lk || (other == lk && j < lane) ? 1 : 0;
      }
      rank = lane < all ? rank : lane;
      auto move = [&](int v) { return __builtin_amdgcn_ds_permute(rank * 4, v); };
      q0 = move((int)q0);
      q1 = move((int)q1);
      lk = move(lk);
      blocks = move(blocks);
      who = move(lane);
    }
  };
  float tiles = 0.f, all = 0.f;
  if (a.slots || a.nseq <= 64) {
    for (int s0 = 0; s0 < a.nseq; s0 += 64) {
      look(s0);
      tiles += (float)blocks * (float)((unsigned)(lk + TILE - 1) / TILE);
      all += (float)blocks;
    }
  }
  if (a.slots) {
    tiles = lanes_sum(tiles);
    all = lanes_sum(all);
  }
  const int per = paged_per<TILE, FEW>(a, tiles, all);
  unsigned before = 0, cut = 0;  // pieces of the sequences before, and those among them with results
  for (int s0 = 0; s0 < a.nseq; s0 += 64) {
    if (a.nseq > 64) look(s0);
    const unsigned of = (unsigned)(lk + TILE - 1) / TILE;
    const unsigned pieces = blocks ? (of ? (of - 1) / (unsigned)per + 1 : 1u) : 0u;
    const unsigned count = (unsigned)blocks * pieces, part = pieces > 1 ? count : 0u;
    const unsigned upto = lanes_scan(count), parts = a.slots ? lanes_scan(part) : 0u;
    const unsigned long long found = __ballot(BY_SLOT ? cut + parts > at : before + upto > at);
    if (found) {
      const int f = __ffsll(found) - 1;
      const unsigned first = before + __builtin_amdgcn_readlane((int)(upto - count), f);
      const unsigned slot = cut + __builtin_amdgcn_readlane((int)(parts - part), f);
      r.sequence = s0 + __builtin_amdgcn_readlane(who, f);
      r.q0 = __builtin_amdgcn_readlane((int)q0, f);
      r.q1 = __builtin_amdgcn_readlane((int)q1, f);
      r.lk = __builtin_amdgcn_readlane(lk, f);
      const unsigned np = (unsigned)__builtin_amdgcn_readlane((int)pieces, f);
      const unsigned local = at - (BY_SLOT ? slot : first), block = local / np;
      r.pieces = (int)np;
      r.piece = (int)(local - block * np);
      // the last rows first: causal ones see most keys
      r.row0 = (int64_t)((unsigned)__builtin_amdgcn_readlane(blocks, f) - 1 - block) * BM;
      // a sequence's pieces are alike: 2^31 keys at most
      r.per = (int)(((unsigned)(r.lk + TILE - 1) / TILE + np - 1) / np) * TILE;
      r.slot = np > 1 ? (int)(slot + local) : -1;
      // starts that do not ascend can ask for more than there is room for
      if (np > 1 && slot + block * np + np > (unsigned)a.slots) r.sequence = -1;
      return r;
    }
    before += (unsigned)__builtin_amdgcn_readlane((int)upto, 63);
    cut += (unsigned)__builtin_amdgcn_readlane((int)parts, 63);
  }
  return r;
}

// Page of key `key` of a sequence (keys behind its last: of that one), inside the cache.
__device__ __forceinline__ int paged_number(const PagedArgs& a, const int32_t* row, int64_t key, int lk) {
  key = key < lk ? key : lk - 1;
  const int64_t p = row[key >> a.shift];
  return (int)(p < 0 ? 0 : (p >= a.npages ? a.npages - 1 : p));
}
// Where the 16 keys of `key` (a multiple of 16; behind the last: the last key's 16) begin in their
// page, in elements of K and V.
struct PagedPlace {
  int64_t k, v;
  __device__ __forceinline__ void set(const PagedArgs& a, int64_t page, int64_t key, int lk) {
    key = (key < lk ? key : lk - 1) & ~15;
    const int in = (int)key & ((1 << a.shift) - 1);
    k = page * a.k_page + (int64_t)in * a.k_token;
    v = page * a.v_page + (int64_t)in * a.v_token;
  }
};
__device__ __forceinline__ int64_t readlane64(int64_t v, int lane) {
  return (int64_t)((uint64_t)(unsigned)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 |
                   (unsigned)__builtin_amdgcn_readlane((int)v, lane));
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
template <int D, int DC, bool PAD, class Args>
__global__ __launch_bounds__(256, 2) void attention_kernel(Args a) {
  constexpr bool kPaged = std::is_same<Args, PagedArgs>::value;
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
  int64_t q0, q1, k0 = 0, row0;
  int lk;
  [[maybe_unused]] PagedWork work;
  if constexpr (kPaged) {
    work = paged_work<kBM, kAKT, false, false>(a, blockIdx.x / a.hk, lane);
    if (work.sequence < 0) return;
    q0 = work.q0;
    q1 = work.q1;
    lk = work.lk;
    row0 = work.row0;
  } else {
    // the last slots first: a causal sequence's longest rows are its last
    const int64_t slot = (int64_t)(gridDim.x / a.hk) - 1 - blockIdx.x / a.hk;
    const Sequence sq = sequence_of<kBM>(a, slot, lane);
    if (sq.index < 0) return;
    q0 = sq.q0;
    q1 = sq.q1;
    k0 = sq.k0;
    lk = sq.k1 > k0 ? (int)(sq.k1 - k0) : 0;
    row0 = (slot - (q0 * a.g / kBM + sq.index)) * kBM;
  }
  const int64_t rows = q1 > q0 ? (q1 - q0) * a.g : 0;
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
  int kbeg, kend;
  bool cut;
  if constexpr (kPaged) {
    kbeg = (int)min((int64_t)keys, (int64_t)work.piece * work.per);
    kend = keys - kbeg < work.per ? keys : kbeg + work.per;
    cut = work.pieces > 1;
  } else {
    const int per = (int)cdiv(cdiv(keys, kAKT), a.splits) * kAKT;
    kbeg = min(keys, (int)blockIdx.y * per), kend = min(keys, kbeg + per);
    cut = a.splits > 1;
  }

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
  const unsigned short* kb = a.k + (kPaged ? 0 : k0 * a.k_token) + head * a.k_head;
  const unsigned short* vb = a.v + (kPaged ? 0 : k0 * a.v_token) + head * a.v_head;
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
      unsigned row = min(row_w + NW * i * kRowsPer, last);
      if constexpr (kPaged) row &= 15;  // of its 16 keys
      vk[i] = (row * (unsigned)a.k_token + ck) * 2;
      vv[i] = (row * (unsigned)a.v_token + cv) * 2;
    }
  };
  // The next tile's loads, one by one: i < kLd of K, then kLd of V.
  const unsigned short *gk = kb, *gv = vb;
  unsigned dk = 0;
  // Paged: a load's rows lie in 16 consecutive keys, which are of one page. Lane x of `place` holds
  // where keys 16 x .. of the 1024 at hand are, `coming` the page of those of the next 1024.
  [[maybe_unused]] PagedPlace place = {0, 0};
  [[maybe_unused]] int coming = 0, first16 = 0;
  [[maybe_unused]] const int32_t* page_row = nullptr;
  if constexpr (kPaged) page_row = a.pages + work.sequence * a.pages_row;
  auto next_tile = [&](int kt, int buf) {
    if (kt + kAKT > lk) offsets(lk - 1 - kt);  // the sequence's last tile
    if constexpr (kPaged) {
      if ((kt & 1023) == 0 || kt == kbeg) {
        const int64_t from = (kt & ~1023) + 16 * lane;
        place.set(a, kt == kbeg ? paged_number(a, page_row, from, lk) : coming, from, lk);
        coming = paged_number(a, page_row, from + 1024, lk);
      }
      first16 = (kt >> 4) & 63;
    } else {
      gk = kb + (int64_t)kt * a.k_token;
      gv = vb + (int64_t)kt * a.v_token;
    }
    dk = smb + buf * kTile + wave * 1024;
  };
  auto load = [&](int i) {
    if constexpr (kPaged) {
      const int x = i < kLd ? i : i - kLd;
      const int at = first16 + ((wave + NW * x) * kRowsPer >> 4);
      if (i < kLd) {
        if (in_k) lds_dma1(vk[x], kb + readlane64(place.k, at), dk + x * NW * 1024);
      } else {
        lds_dma1(vv[x], vb + readlane64(place.v, at), dk + ST * kTile + x * NW * 1024);
      }
      return;
    }
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
          const float p0 = exp2_fast(fmaf(s[kb16][rb][2 * x], a.c, ref));
          const float p1 = exp2_fast(fmaf(s[kb16][rb][2 * x + 1], a.c, ref));
          if constexpr (kPaged) {  // s holds the weights as they are
            s[kb16][rb][2 * x] = p0;
            s[kb16][rb][2 * x + 1] = p1;
            l[rb] += p0 + p1;
          } else {
            const bf16x2_t p = pack2(p0, p1);
            // the sum takes the rounded weights, which are the ones that V meets
            l[rb] = __builtin_amdgcn_fdot2_f32_bf16(p, bf16x2_t{(__bf16)1.0f, (__bf16)1.0f}, l[rb],
                                                    false);
            pf[kb16 >> 1][rb][(kb16 & 1) * 4 + 2 * x] = p[0];
            pf[kb16 >> 1][rb][(kb16 & 1) * 4 + 2 * x + 1] = p[1];
          }
        }
    }
    // Paged: the weights of 32 keys from 32 kc as operands, and what their rounding leaves.
    [[maybe_unused]] bf16x8_t pr[2][2];
    [[maybe_unused]] auto operands = [&](int kc, int rb) __attribute__((always_inline)) {
      u32x4_t wf, wr;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const f32x4_t& w = s[2 * kc + (x >> 1)][rb];
        const float p0 = w[2 * (x & 1)], p1 = w[2 * (x & 1) + 1];
        wf[x] = __builtin_bit_cast(unsigned, pack2(p0, p1));
        wr[x] = __builtin_bit_cast(unsigned, pack2(p0 - __uint_as_float(wf[x] << 16),
                                                   p1 - __uint_as_float(wf[x] & 0xffff0000u)));
      }
      pf[kc][rb] = __builtin_bit_cast(bf16x8_t, wf);
      pr[kc][rb] = __builtin_bit_cast(bf16x8_t, wr);
    };
    if constexpr (careful) {
      // element j % 8 of lanes 16 (j / 8) .. of 32 keys' values alone, and which key that is
      auto alone = [&](const v8i16_t& v, int j) {
        v8i16_t one;
#pragma unroll
        for (int x = 0; x < 8; ++x) one[x] = quad == j >> 3 && x == (j & 7) ? v[x] : (short)0;
        return __builtin_bit_cast(bf16x8_t, one);
      };
      auto key_of = [&](int kc, int j) { return kt + 32 * kc + 4 * (j >> 3) + (j & 3) + 16 * (j >> 2 & 1); };
      if constexpr (kPaged) {
        // first the weights, then their rests, whose products with an infinity are left out
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
          auto add = [&](f32x4_t& to, const f32x4_t& z) {
#pragma unroll
            for (int e = 0; e < 4; ++e) to[e] += part == 0 || isfinite(z[e]) ? z[e] : 0.f;
          };
#pragma unroll
          for (int kc = 0; kc < 2; ++kc) {
            bf16x8_t w[2];
#pragma unroll
            for (int rb = 0; rb < 2; ++rb)
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                const float p = s[2 * kc + (x >> 2)][rb][x & 3];
                const __bf16 near = (__bf16)p;
                w[rb][x] = part == 0 ? near : (__bf16)(p - (float)near);
              }
#pragma unroll
            for (int cb = 0; cb < kCB; ++cb) {
              const v8i16_t v = v_frag(kc, cb);
              const f32x4_t zero = {};
              if (masked) {
#pragma unroll 1
                for (int j = 0; j < 32; ++j) {
                  const bf16x8_t one = alone(v, j);
#pragma unroll
                  for (int rb = 0; rb < 2; ++rb) {
                    const f32x4_t z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(one, w[rb], zero, 0, 0, 0);
                    if (key_of(kc, j) < lim[rb]) add(o[cb][rb], z);
                  }
                }
              } else {
#pragma unroll
                for (int rb = 0; rb < 2; ++rb)
                  add(o[cb][rb], __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                     __builtin_bit_cast(bf16x8_t, v), w[rb], zero, 0, 0, 0));
              }
            }
          }
        }
        return;
      } else if (masked) {
#pragma unroll
        for (int kc = 0; kc < 2; ++kc)
#pragma unroll
          for (int cb = 0; cb < kCB; ++cb) {
            const v8i16_t vx = v_frag(kc, cb);
#pragma unroll 1
            for (int j = 0; j < 32; ++j) {
              const bf16x8_t one = alone(vx, j);
#pragma unroll
              for (int rb = 0; rb < 2; ++rb) {
                const f32x4_t zero = {};
                const f32x4_t z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(one, pf[kc][rb], zero, 0, 0, 0);
                if (key_of(kc, j) < lim[rb]) o[cb][rb] += z;
              }
            }
          }
        return;
      }
    }
    if constexpr (kPaged) {
#pragma unroll
      for (int rb = 0; rb < 2; ++rb) operands(0, rb);
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
        if constexpr (kPaged) {
#pragma unroll
          for (int rb = 0; rb < 2; ++rb)
            o[cb][rb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8_t, vf[cb]), pr[kc][rb], o[cb][rb], 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (kc == 0) vf[cb] = v_frag(1, cb);
        if constexpr (kPaged) {
          if (kc == 0 && cb >= kCB - 2) operands(1, cb - (kCB - 2));
        }
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
  // Paged: an infinity that a row sees stays one times p, but is NaN times p's rest (0, or of the other
  // sign): where anything is not finite, the second pass leaves such products of the rests out.
  float zeros = 0.f;
  if constexpr (kPaged) {
#pragma unroll
    for (int rb = 0; rb < 2; ++rb)
#pragma unroll
      for (int cb = 0; cb < kCB; ++cb)
#pragma unroll
        for (int e = 0; e < 4; ++e) zeros = fmaf(o[cb][rb][e], 0.f, zeros);
  }
  if (__syncthreads_or((bad & 0x80008000u) != 0 || zeros != 0.f)) {
    pass(std::integral_constant<bool, true>{});
    __syncthreads();  // a wave that is done puts its rows over tiles that others still read
  }

#pragma unroll
  for (int rb = 0; rb < 2; ++rb) {
    l[rb] += __shfl_xor(l[rb], 16);
    l[rb] += __shfl_xor(l[rb], 32);
  }
  // element 4 quad + e of each block of 16 is in register e
  if (cut) {
#pragma unroll
    for (int rb = 0; rb < 2; ++rb) {
      if (!valid[rb]) continue;
      int64_t at;
      if constexpr (kPaged)
        at = ((int64_t)work.slot * a.hk + head) * kBM + wave * 32 + rb * 16 + r16;
      else
        at = ((int64_t)blockIdx.y * a.nq + q0 + tok[rb]) * (a.hk * a.g) + qh[rb];
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
// Paged, a workgroup has two waves where there are more than compute units, so that a unit holds
// two: the work before a workgroup's first and after its last tile (7 us and more) is beside the
// other's loads. 64 tokens over 300001 keys in pages, 64 heads on 8: 253-260 us (4.8 TB/s) and 7
// for the join; one token over 300 keys 12.0, the page numbers' loads before the keys' being the
// rest to 10.1; 16 tokens over 1000 keys each, 32 heads, 63 where packed keys take 54.
template <int D, int DC, bool PAD, int WAVES, class Args>
__global__ __launch_bounds__(64 * WAVES, 1) void attention_few_kernel(Args a) {
  constexpr bool kPaged = std::is_same<Args, PagedArgs>::value;
  constexpr int kBM = 32, kKeys = 32, kWaves = WAVES;
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
  int64_t q0, q1, k0 = 0, row0;
  int lk;
  [[maybe_unused]] PagedWork work;
  if constexpr (kPaged) {
    work = paged_work<kBM, kKeys, true, false>(a, blockIdx.x / a.hk, lane);
    if (work.sequence < 0) return;
    q0 = work.q0;
    q1 = work.q1;
    lk = work.lk;
    row0 = work.row0;
  } else {
    const int64_t slot = (int64_t)(gridDim.x / a.hk) - 1 - blockIdx.x / a.hk;
    const Sequence sq = sequence_of<kBM>(a, slot, lane);
    if (sq.index < 0) return;
    q0 = sq.q0;
    q1 = sq.q1;
    k0 = sq.k0;
    lk = sq.k1 > k0 ? (int)(sq.k1 - k0) : 0;
    row0 = (slot - (q0 * a.g / kBM + sq.index)) * kBM;
  }
  const int64_t rows = q1 > q0 ? (q1 - q0) * a.g : 0;
  if (row0 < 0 || row0 >= rows) return;
  const int off = lk - (int)(q1 - q0);
  auto limit_of = [&](int64_t r) {
    if (!a.causal) return lk;
    const int64_t e = (int64_t)((unsigned)r / (unsigned)a.g) + off + 1;
    return (int)(e < 0 ? 0 : (e < lk ? e : lk));
  };
  const int64_t row_end = row0 + kBM < rows ? row0 + kBM : rows;
  const int keys = limit_of(row_end - 1);
  int kbeg, kend;
  bool cut;
  if constexpr (kPaged) {
    kbeg = (int)min((int64_t)keys, (int64_t)work.piece * work.per);
    kend = keys - kbeg < work.per ? keys : kbeg + work.per;
    cut = work.pieces > 1;
  } else {
    const int per = (int)cdiv(cdiv(keys, kKeys), a.splits) * kKeys;
    kbeg = min(keys, (int)blockIdx.y * per), kend = min(keys, kbeg + per);
    cut = a.splits > 1;
  }
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
  const unsigned short* kb = a.k + (kPaged ? 0 : k0 * a.k_token) + head * a.k_head;
  if (PAD && cv >= a.d) cv = 0;
  const unsigned short* vb = a.v + (kPaged ? 0 : k0 * a.v_token) + head * a.v_head;
  const unsigned ob = lds_address(sm) + wave * 4 * kTile;
  // Paged: the wave's tiles are 32 kWaves keys apart and of two times 16 keys, each of one page. Lanes
  // 2x and 2x + 1 of `place` hold where those of tile x of the 32 at hand are, of `coming` the
  // pages of the next 32.
  [[maybe_unused]] PagedPlace place = {0, 0};
  [[maybe_unused]] int coming = 0;
  [[maybe_unused]] const int32_t* page_row = nullptr;
  if constexpr (kPaged) page_row = a.pages + work.sequence * a.pages_row;
  // One operand of a tile. K goes first: it finds the places of either.
  int64_t gk[2] = {0, 0}, gv[2] = {0, 0};  // of the last tile whose K was issued
  [[maybe_unused]] auto find_places = [&](int kt, const auto& a) __attribute__((always_inline)) {
    const int x = (kt - kbeg) / (kWaves * kKeys);
    if ((x & 31) == 0) {
      const int64_t key = (int64_t)kt + (lane >> 1) * (kWaves * kKeys) + (lane & 1) * 16;
      place.set(a, x == 0 ? paged_number(a, page_row, key, lk) : coming, key, lk);
      coming = paged_number(a, page_row, key + 32 * kWaves * kKeys, lk);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      gk[h] = readlane64(place.k, 2 * (x & 31) + h);
      gv[h] = readlane64(place.v, 2 * (x & 31) + h);
    }
  };
  auto issue = [&](int kt, int buf, bool of_k) __attribute__((always_inline)) {
    if constexpr (kPaged) {
      if (of_k) find_places(kt, a);
    } else {
      gk[0] = (int64_t)kt * a.k_token;
      gv[0] = (int64_t)kt * a.v_token;
    }
    const int last = min(kKeys, lk - kt) - 1;  // rows past the keys read the last: masked
#pragma unroll
    for (int i = 0; i < kLd; ++i) {
      unsigned row = min(i * kRowsPer + lr, last);
      if constexpr (kPaged) row &= 15;
      const int h = kPaged ? i * kRowsPer >> 4 : 0;  // the 16 keys that the load's rows are of
      if (of_k) {
        const int ck = k_piece(i);
        if (!PAD || ck < a.d)
          lds_dma1((row * (unsigned)a.k_token + ck) * 2, kb + gk[h], ob + 2 * buf * kTile + i * 1024);
      } else {
        lds_dma1((row * (unsigned)a.v_token + cv) * 2, vb + gv[h], ob + (2 * buf + 1) * kTile + i * 1024);
      }
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
  // Paged, two tiles are in flight, and the keys of a third as soon as this one's are read: at a
  // tile's beginning its K has landed and its V may not have. (64 tokens over 300001 keys, 64 heads
  // on 8: 294 -> 286 us. Packed keys go tile by tile: 2% slower there, 4% faster where one token
  // has 300 keys.) Loads that are newer than the ones waited for, in units of an operand's; the
  // pages' own loads among them only make the waits stricter.
  constexpr int kStep = kWaves * kKeys;
  auto wait_newer = [&](int units) __attribute__((always_inline)) {
    static_assert(kLd == 8 || kLd == 4, "vmcnt immediates");
    if (units == 3)
      __asm__ volatile("s_waitcnt vmcnt(%0)" ::"n"(3 * kLd) : "memory");
    else if (units == 2)
      __asm__ volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * kLd) : "memory");
    else if (units == 1)
      __asm__ volatile("s_waitcnt vmcnt(%0)" ::"n"(kLd) : "memory");
    else
      __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
  };
  auto keys_landed = [&](int kt) __attribute__((always_inline)) { wait_newer(kt + kStep < kend ? 3 : 1); };
  auto values_landed = [&](int kt) __attribute__((always_inline)) {
    if constexpr (!kPaged) return;
    wait_newer(kt + 2 * kStep < kend ? 3 : (kt + kStep < kend ? 2 : 0));
  };
  auto refill = [&](int kt, int buf, bool of_k) __attribute__((always_inline)) {
    if constexpr (!kPaged) return;
    if (kt + 2 * kStep < kend) {
      // the operand's reads are done before it is filled again
      __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      issue(kt + 2 * kStep, buf, of_k);
    }
  };
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
    refill(kt, buf, true);
    const bool masked = kt + kKeys > lim_first;
    if (masked) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        s[e] = kt + 8 * (e >> 2) + 4 * half + (e & 3) < lim ? s[e] : -INFINITY;
      if constexpr (!careful) {
        values_landed(kt);
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
    values_landed(kt);
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
    int kt = kbeg + wave * kKeys, buf = 0;
    auto issue_tile = [&](int at, int to) __attribute__((always_inline)) {
      issue(at, to, true);
      issue(at, to, false);
    };
    if (kt < kend) issue_tile(kt, 0);
    if (kPaged && kt + kStep < kend) issue_tile(kt + kStep, 1);
    for (; kt < kend; kt += kStep, buf ^= 1) {
      if constexpr (kPaged) {
        keys_landed(kt);
      } else if (kt + kStep < kend) {
        // the other buffer's reads are done before it is filled again
        __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        issue_tile(kt + kStep, buf ^ 1);
        wait_newer(2);
      } else {
        wait_newer(0);
      }
      tile(kt, buf, CAREFUL);
      refill(kt, buf, false);
    }
  };
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
  constexpr int kRowThreads = 64 * kWaves / 32;
  const int rr = tid / kRowThreads;
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
  int64_t at;
  if constexpr (kPaged)
    at = ((int64_t)work.slot * a.hk + head) * kBM + rr;
  else
    at = ((int64_t)blockIdx.y * a.nq + q0 + ot) * (a.hk * a.g) + oh;
  if (cut && tid % kRowThreads == 0)
    a.part_ml[at] = make_float2(mt, min(vis, kend) > kbeg && lt == 0.f ? -1.f : lt);
  const float inv = vis > 0 ? 1.0f / lt : 0.f;
#pragma unroll
  for (int i = 0; i < D / (4 * kRowThreads); ++i) {
    const int e = (tid % kRowThreads) * 4 + 4 * kRowThreads * i;
    if (e >= a.d) break;
    f32x4_t v = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
      if (f[w] != 0.f)
        v += *(const f32x4_t*)((const float*)(sm + w * 4 * kTile) + rr * kOutW + e) * f[w];
    if (cut) {
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

// Pieces 0 .. splits - 1 of one row, whose results are at ml + s * step and po + s * step * d,
// joined into o (d elements) by `groups` groups of 32 lanes (1, or the workgroup's 8), grp and
// lane being this thread's.
template <bool FEW>
__device__ __forceinline__ void join_row(const float2* ml, const float* po, int64_t step, int splits,
                                         int d, int grp, int lane, unsigned short* out) {
  __shared__ float part[FEW ? 1 : 8][132];  // 128 elements, l, any
  const int e = lane * 4;
  float m = -INFINITY;
  for (int s = lane; s < splits; s += 32) m = fmaxf(m, ml[s * step].x);
#pragma unroll
  for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor(m, x, 32));
  const float ref = m == -INFINITY ? 0.f : m;
  f32x4_t o = f32x4_t{0.f, 0.f, 0.f, 0.f};
  float l = 0.f, any = 0.f;
  constexpr int kApart = FEW ? 1 : 8, kAtOnce = 4;  // pieces whose results are on their way together
  for (int s0 = FEW ? 0 : grp; s0 < splits; s0 += kApart * kAtOnce) {
    float2 y[kAtOnce];
    f32x4_t v[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int64_t s = s0 + u * kApart;
      y[u] = make_float2(0.f, 0.f);
      v[u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      if (s < splits) {
        y[u] = ml[s * step];
        if (e < d) v[u] = *(const f32x4_t*)(po + s * step * d + e);  // anything, where no key was seen
      }
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      if (y[u].y != 0.f) any = 1.f;  // 0: the piece saw no key
      if (y[u].y <= 0.f) continue;   // -1: only scores of -inf
      const float f = exp2_fast(y[u].x - ref);
      l += y[u].y * f;
      o += v[u] * f;
    }
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
  if (e >= d) return;
  // keys seen, but every score -inf: l is 0 and there is no softmax (NaN)
  u16x4_t w;
#pragma unroll
  for (int y = 0; y < 4; ++y) w[y] = any > 0.f ? f32_to_bf16_rne(o[y] / l) : (unsigned short)0;
  *(u16x4_t*)(out + e) = w;
}

template <bool FEW>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a) {
  const int grp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int hq = a.hk * a.g;
  const int64_t row = FEW ? (int64_t)blockIdx.x * 8 + grp : blockIdx.x;
  const int64_t tok = row / hq;
  const int qh = (int)(row - tok * hq);
  if (tok < start_at(a.q_start, 0, a.nq) || tok >= start_at(a.q_start, a.nseq, a.nq)) return;
  join_row<FEW>(a.part_ml + row, a.part_o + row * a.d, a.nq * hq, a.splits, a.d, grp, lane,
                a.o + tok * a.o_token + qh * a.o_head);
}

// The same for a paged call: workgroup (slot, key head) joins a share of the rows of the row block
// that left a partial result there, each of its pieces another one: a group of 32 lanes per row,
// or, for few rows of many pieces, the eight groups to a row.
template <int BM, int TILE, bool FEW>
__global__ __launch_bounds__(256) void paged_join_kernel(PagedArgs a) {
  const int grp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int head = blockIdx.x % a.hk;
  const PagedWork w = paged_work<BM, TILE, FEW, true>(a, blockIdx.x / a.hk, threadIdx.x & 63);
  if (w.sequence < 0) return;
  const int64_t rows = (w.q1 - w.q0) * a.g - w.row0;
  const int block = (int)(rows < BM ? rows : BM), share = (int)cdiv(block, w.pieces);
  const int end = min(block, (w.piece + 1) * share);
  const int64_t first = ((int64_t)(w.slot - w.piece) * a.hk + head) * BM, step = (int64_t)a.hk * BM;
  auto join = [&](int r, auto ALONE) {
    const int64_t row = w.row0 + r, tok = w.q0 + (unsigned)row / (unsigned)a.g;
    const int qh = head * a.g + (int)((unsigned)row % (unsigned)a.g);
    join_row<decltype(ALONE)::value>(a.part_ml + first + r, a.part_o + (first + r) * a.d, step, w.pieces,
                                     a.d, grp, lane, a.o + tok * a.o_token + qh * a.o_head);
  };
  if (w.pieces <= 8 || share > 2) {
    for (int r = w.piece * share + grp; r < end; r += 8) join(r, std::integral_constant<bool, true>{});
    return;
  }
  for (int r = w.piece * share; r < end; ++r) {
    join(r, std::integral_constant<bool, false>{});
    __syncthreads();  // the groups' sums have been read
  }
}

template <int D, int DC, bool PAD, class Args>
void launch_kernel(const Args& a, dim3 groups, hipStream_t s) {
  hipLaunchKernelGGL((attention_kernel<D, DC, PAD, Args>), groups, dim3(256), 0, s, a);
}

template <int D, int DC, bool PAD, class Args>
void launch_few(const Args& a, dim3 groups, hipStream_t s) {
  if constexpr (std::is_same<Args, PagedArgs>::value) {
    if (groups.x > kAUnits) {
      hipLaunchKernelGGL((attention_few_kernel<D, DC, PAD, 2, Args>), groups, dim3(128), 0, s, a);
      return;
    }
  }
  hipLaunchKernelGGL((attention_few_kernel<D, DC, PAD, 4, Args>), groups, dim3(256), 0, s, a);
}

// The kernel for heads of a.d elements.
template <class Args>
void launch_by_head(const Args& a, bool few, dim3 groups, hipStream_t s) {
  if (few) {
    if (a.d < 64)
      launch_few<64, 64, true>(a, groups, s);
    else if (a.d == 64)
      launch_few<64, 64, false>(a, groups, s);
    else if (a.d < 128)
      launch_few<128, 128, true>(a, groups, s);
    else
      launch_few<128, 128, false>(a, groups, s);
    return;
  }
  switch (cdiv(a.d, 16)) {
    case 1:
    case 2: launch_kernel<64, 32, true>(a, groups, s); break;
    case 3: launch_kernel<64, 48, true>(a, groups, s); break;
    case 4:
      if (a.d < 64)
        launch_kernel<64, 64, true>(a, groups, s);
      else
        launch_kernel<64, 64, false>(a, groups, s);
      break;
    case 5: launch_kernel<128, 80, true>(a, groups, s); break;
    case 6: launch_kernel<128, 96, true>(a, groups, s); break;
    case 7: launch_kernel<128, 112, true>(a, groups, s); break;
    default:
      if (a.d < 128)
        launch_kernel<128, 128, true>(a, groups, s);
      else
        launch_kernel<128, 128, false>(a, groups, s);
  }
}

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
  const int64_t slots = a.nq * a.g / (plan.few ? 32 : 128) + a.nseq;
  launch_by_head(a, plan.few, dim3((unsigned)(slots * a.hk), (unsigned)a.splits), s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t rows = p->nq * p->hq;
  if (a.splits <= kAJoinSplits && rows > kAJoinRows)
    hipLaunchKernelGGL(attention_join_kernel<true>, dim3((unsigned)cdiv(rows, 8)), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL(attention_join_kernel<false>, dim3((unsigned)rows), dim3(256), 0, s, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------- paged: plan and launches

namespace {

struct PagedPlan {
  bool few, many;  // which of the two kernels run
  int few_to;      // rows of a sequence that the first takes; the second those above
  int64_t few_items, many_items;  // pieces a key head, at most
  int few_slots, many_slots;      // partial results a key head
};

// Which kernels: by the average rows, as in th_attention; but where they are few and some
// sequences may be longer all the same, either kernel takes its own. (A launch that finds nothing
// to do takes 3 to 10 us; a chunk of 1000 tokens in 32-row blocks takes twice as long as in
// 128-row ones.) The rest is what the device can find there, from sizes alone: sequences of r rows
// have r / BM row blocks, or part of one more; pieces are cut from T tiles so that
// T / per <= target / hk, and there are T / per + (row blocks) of them at most, those of cut row
// blocks no more than 2 T / per.
PagedPlan plan_of(const th_paged_cache* c, const th_paged_params* p) {
  PagedPlan r = {};
  if (p->nq == 0) return r;
  const int64_t g = p->hq / c->hk, nseq = c->nseq, most = c->width * c->page_tokens;
  const int64_t rows = p->nq * g, seqs = nseq < p->nq ? nseq : p->nq;
  r.few = rows <= kAFewRows * nseq;
  r.many = !r.few || (!p->even && p->nq > 2 * nseq && rows > kAFewRows);
  r.few_to = r.many ? kAFewRows : 0x7fffffff;
  auto bound = [&](int64_t blocks, int64_t target, int64_t least, int64_t& items, int& slots) {
    const int64_t pieces = cdiv(most, least);
    slots = pieces > 1 ? (int)(2 * target / c->hk) : 0;
    items = slots ? target / c->hk + blocks : blocks;
    if (slots && pieces < (1 << 20) && blocks * pieces < items) items = blocks * pieces;
    if (slots > items) slots = (int)items;
  };
  if (r.few) bound(r.many ? seqs : rows / 32 + seqs, 4 * kAUnits, 320, r.few_items, r.few_slots);
  if (r.many) {
    const int64_t longer = r.few ? std::min(seqs, rows / (kAFewRows + 1)) : seqs;
    bound(rows / 128 + longer, 2 * kAUnits, 3 * kAKT, r.many_items, r.many_slots);
  }
  return r;
}

size_t paged_rows(const PagedPlan& r, const th_paged_cache* c) {
  return ((size_t)r.few_slots * 32 + (size_t)r.many_slots * 128) * (size_t)c->hk;
}

}  // namespace

int64_t paged_attention_workgroups(const th_paged_cache* c, const th_paged_params* p) {
  if (p->nq == 0) return 0;
  const PagedPlan r = plan_of(c, p);
  return std::max(std::max(r.few_items, r.many_items), (int64_t)std::max(r.few_slots, r.many_slots)) *
         c->hk;
}

size_t paged_attention_workspace_bytes(const th_paged_cache* c, const th_paged_params* p) {
  if (p->nq == 0) return 0;
  const size_t rows = paged_rows(plan_of(c, p), c);
  return rows ? part_ml_bytes((int64_t)rows) + rows * (size_t)c->d * sizeof(float) : 0;
}

hipError_t launch_paged_attention(const void* Q, const int32_t* q_start, const th_paged_cache* c,
                                  const th_paged_params* p, void* O, void* workspace, hipStream_t s) {
  PagedArgs a = {};
  a.q = (const unsigned short*)Q;
  a.k = (const unsigned short*)c->k;
  a.v = (const unsigned short*)c->v;
  a.o = (unsigned short*)O;
  a.q_token = p->q_token;
  a.q_head = p->q_head;
  a.k_token = c->k_token;
  a.k_head = c->k_head;
  a.v_token = c->v_token;
  a.v_head = c->v_head;
  a.o_token = p->o_token;
  a.o_head = p->o_head;
  a.q_start = q_start;
  a.k_start = c->k_len;
  a.nq = p->nq;
  a.nseq = (int)c->nseq;
  a.hk = (int)c->hk;
  a.g = (int)(p->hq / c->hk);
  a.d = (int)c->d;
  a.causal = p->causal != 0;
  a.c = (float)(p->scale * 1.4426950408889634);
  a.pages = c->pages;
  a.pages_row = c->pages_row;
  a.k_page = c->k_page;
  a.v_page = c->v_page;
  a.npages = c->npages;
  a.keys_most = c->npages > 0 ? c->width * c->page_tokens : 0;
  a.each = p->nq / c->nseq;
  a.shift = __builtin_ctzll((unsigned long long)c->page_tokens);
  const PagedPlan plan = plan_of(c, p);
  const size_t rows = workspace ? paged_rows(plan, c) : 0;
  a.part_ml = (float2*)workspace;
  a.part_o = workspace ? (float*)((char*)workspace + part_ml_bytes((int64_t)rows)) : nullptr;
  if (plan.few) {
    a.rows_from = 1;
    a.rows_to = plan.few_to;
    a.slots = workspace ? plan.few_slots : 0;
    launch_by_head(a, true, dim3((unsigned)(plan.few_items * a.hk)), s);
    if (a.slots)
      hipLaunchKernelGGL((paged_join_kernel<32, 32, true>), dim3((unsigned)(a.slots * a.hk)), dim3(256),
                         0, s, a);
  }
  if (plan.many) {
    if (workspace) {  // behind the results of the few rows
      a.part_ml += (int64_t)plan.few_slots * 32 * a.hk;
      a.part_o += (int64_t)plan.few_slots * 32 * a.hk * a.d;
    }
    a.rows_from = plan.few ? plan.few_to + 1 : 1;
    a.rows_to = 0x7fffffff;
    a.slots = workspace ? plan.many_slots : 0;
    launch_by_head(a, false, dim3((unsigned)(plan.many_items * a.hk)), s);
    if (a.slots)
      hipLaunchKernelGGL((paged_join_kernel<128, kAKT, false>), dim3((unsigned)(a.slots * a.hk)),
                         dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace th
