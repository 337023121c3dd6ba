// New keys and values into the pages of a cache, which attention over it reads (attention.hip):
// row t of sequence s becomes key k_len[s] - (q_start[s+1] - t) of that sequence.
//
// A copy, bound by memory for many tokens and by its launch for few. Wave by wave: a token's
// sequence is found with one or two loads of the start array (a lane holds a start), then
// its lanes move the token's heads 16 bytes at a time, keys and values in turn. 12342 tokens of 32
// heads of 128: 71-79 us (5.1-5.7 TB/s); 16 tokens of 8 heads 3.1-3.4, of which a launch is 2.3.
#include "common.h"

namespace th {

namespace {

struct StoreArgs {
  const unsigned short *k, *v;
  int64_t k_token, k_head, v_token, v_head;
  th_paged_cache c;
  const int32_t* q_start;
  int64_t first, nq, each;  // first row of the launch; each: rows of a sequence without q_start
  int shift;         // log2 of page_tokens
  int pieces;        // of 16 bytes a head
};

__device__ __forceinline__ int64_t row_at(const int32_t* s, int64_t i, int64_t n) {
  const int64_t v = s[i];
  return v < 0 ? 0 : (v > n ? n : v);
}

// LANES (64, 128, 256) to a token, 256 / LANES tokens to a workgroup.
template <int LANES>
__global__ __launch_bounds__(256) void cache_store_kernel(StoreArgs a) {
  const int64_t t = a.first + (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  if (t >= a.nq) return;
  const int lane = threadIdx.x & 63;
  int64_t s, end;  // the sequence of the token, the row behind its last
  if (a.q_start) {
    // the last sequence that begins at or before the row
    int64_t lo = 0, len = a.c.nseq;
    for (;;) {
      const int64_t step = (len + 63) >> 6, at = lane * step;
      const bool before = at < len && row_at(a.q_start, lo + at, a.nq) <= t;
      const int count = __popcll(__ballot(before));
      if (count == 0) return;
      lo += (count - 1) * step;
      if (step == 1) break;
      len = min(step, len - (count - 1) * step);
    }
    s = lo;
    end = row_at(a.q_start, s + 1, a.nq);
    if (t >= end) return;
  } else {
    s = t / a.each;
    end = (s + 1) * a.each;
  }
  const int64_t most = a.c.width << a.shift;
  int64_t keys = a.c.k_len[s];
  keys = keys < 0 ? 0 : (keys > most ? most : keys);
  const int64_t key = keys - (end - t);
  if (key < 0) return;
  const int64_t page = a.c.pages[s * a.c.pages_row + (key >> a.shift)];
  if (page < 0 || page >= a.c.npages) return;
  const int64_t in = key & (a.c.page_tokens - 1);
  const unsigned short *k = a.k + t * a.k_token, *v = a.v + t * a.v_token;
  unsigned short* ko = (unsigned short*)a.c.k + page * a.c.k_page + in * a.c.k_token;
  unsigned short* vo = (unsigned short*)a.c.v + page * a.c.v_page + in * a.c.v_token;
  const int chunks = (int)a.c.hk * a.pieces;
  for (int i = threadIdx.x % LANES; i < chunks; i += LANES) {
    const int h = i / a.pieces, e = (i - h * a.pieces) * 8;
    *(u32x4_t*)(ko + h * a.c.k_head + e) = *(const u32x4_t*)(k + h * a.k_head + e);
    *(u32x4_t*)(vo + h * a.c.v_head + e) = *(const u32x4_t*)(v + h * a.v_head + e);
  }
}

template <int LANES>
void launch_store(StoreArgs a, hipStream_t s) {
  for (a.first = 0; a.first < a.nq; a.first += kMaxGroups * (256 / LANES)) {
    const int64_t groups = cdiv(a.nq - a.first, 256 / LANES);
    hipLaunchKernelGGL(cache_store_kernel<LANES>, dim3((unsigned)(groups < kMaxGroups ? groups : kMaxGroups)),
                       dim3(256), 0, s, a);
  }
}

}  // namespace

hipError_t launch_cache_store(const void* K, int64_t k_token, int64_t k_head, const void* V,
                              int64_t v_token, int64_t v_head, int64_t nq, const int32_t* q_start,
                              const th_paged_cache* c, hipStream_t s) {
  StoreArgs a;
  a.k = (const unsigned short*)K;
  a.v = (const unsigned short*)V;
  a.k_token = k_token;
  a.k_head = k_head;
  a.v_token = v_token;
  a.v_head = v_head;
  a.c = *c;
  a.q_start = q_start;
  a.nq = nq;
  a.each = nq / c->nseq;
  a.shift = __builtin_ctzll((unsigned long long)c->page_tokens);
  a.pieces = (int)(c->d / 8);
  const int64_t chunks = c->hk * a.pieces;
  if (chunks <= 64)
    launch_store<64>(a, s);
  else if (chunks <= 128)
    launch_store<128>(a, s);
  else
    launch_store<256>(a, s);
  return hipGetLastError();
}

}  // namespace th
