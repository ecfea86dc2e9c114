// Caches that are kept short: which tokens stay, by the attention weight that they have
// received, and moving those together in their pages.
//
// The choice.  Of n > budget tokens the first `sinks` and the last `recent` stay, and of
// those between as many of the heaviest as the budget leaves, equal ones in order.
// The least weight that stays is found digit by digit, from counts of the tokens by
// 11, 11 and 10 bits of their weight (as a whole number of the same order); then the
// tokens are walked through in order.  Up to 32768 tokens stay in registers, so they are read
// once.  What bounds it is the chain of barriers: a digit costs clearing, counting and
// ranking 2048 bins, some 1.5 us each.  8 rows of 1009 tokens: 6.5 us with a launch; 384 rows of
// up to 32768 tokens, 17 MB: 25 us (counted from memory at every digit 40; rows
// in order of their place instead of the longest first 31).  Longer rows are read from memory at
// every digit and twice more, still by one workgroup each: 8 rows of 131072 tokens 110 us.
//
// The move.  Slot i of a row gets token keep[i] >= i of the same row, so a row can be
// moved forward in place, part by part: what a part writes no later part reads.  A page
// that other rows hold too is not written; the row gets a free page in its place.  A row's
// parts follow each other, rows, heads and planes run side by side.  16 rows that keep
// 1024 of up to 2048 tokens of 2 KB in 16 planes, 1.07 GB read and written: 240 us, 4.5 TB/s, a
// plain copy's 4.9 less the parts that are as short as a head.

#include "tq.h"
#include "tq_attn_dev.h"
#include "tq_common.h"
#include "tq_decode.h"
#include "tq_kernels.h"
#include "tq_scan.h"

namespace tq {
namespace {

// ------------------------------------------------------------------ the choice

struct SelectParams {
  const float* scores;
  int64_t s_seq, s_head;
  const int32_t* lens;
  int32_t* keep;
  int32_t* counts;
  float* sums;
  int32_t S, B, H, budget, recent, sinks;
  int32_t sorted;  // rows are taken longest first
};

constexpr int kDigits = 3;
constexpr int kBins = 2048;
__device__ __forceinline__ constexpr int digit_shift(int d) { return d == 0 ? 21 : d == 1 ? 10 : 0; }
__device__ __forceinline__ constexpr int digit_bits(int d) { return d == 2 ? 10 : 11; }

// A weight as a whole number of the same order: -0 as 0, NaN as the least.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.f);
  if (x != x) return 0x007fffffu;  // -inf
  return u >> 31 ? ~u : u | 0x80000000u;
}

template <int WAVES>
struct SelectShared {
  int count[kBins];
  int sum[WAVES];
  int2 part[WAVES];
  uint32_t digit;
  int rest, same;
};

// The tokens of one row as whole numbers of the order in which they stay: kAlways for the
// first and the last ones, 0 past the end, no weight being either.  A workgroup of WAVES
// waves reads them, each wave a run of `steps` times 64.  KPT > 0: they stay in
// registers (steps <= KPT), otherwise every pass reads them again.
constexpr uint32_t kAlways = 0xffffffffu;
template <int WAVES, int KPT>
struct Tokens {
  const float* x;
  int n, lo, hi, first, steps;
  uint32_t held[KPT > 0 ? KPT : 1];
  __device__ __forceinline__ uint32_t key(int i, float v) const {
    return i >= n ? 0u : i < lo || i >= hi ? kAlways : order_of(v);
  }
  __device__ __forceinline__ Tokens(const SelectParams& p, const float* scores, int tokens) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    x = scores;
    n = tokens;
    lo = p.sinks;
    hi = n - p.recent;
    steps = (int)(((uint32_t)n + WAVES * kWave - 1) / (WAVES * kWave));
    first = wave * steps * kWave + lane;  // (up to 2^30 tokens: the last index stays below 2^31)
    if constexpr (KPT > 0) {
      float v[KPT];
#pragma unroll
      for (int j = 0; j < KPT; ++j) {
        const int i = first + j * kWave;
        v[j] = j < steps && i < n ? x[(uint32_t)i] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < KPT; ++j) held[j] = key(first + j * kWave, v[j]);
    }
  }
  // f(index, key) for this lane's tokens, in steps that the whole wave takes.
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    if constexpr (KPT > 0) {
#pragma unroll
      for (int j = 0; j < KPT; ++j)
        if (j < steps) f(first + j * kWave, held[j]);
    } else {
      for (int j0 = 0; j0 < steps; j0 += 4) {
        float v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int i = first + (j0 + u) * kWave;
          v[u] = j0 + u < steps && i < n ? x[i] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (j0 + u < steps) f(first + (j0 + u) * kWave, key(first + (j0 + u) * kWave, v[u]));
      }
    }
  }
};

// Chooses among the n > budget tokens of a row.
template <int WAVES, int KPT>
__device__ __forceinline__ void choose(const SelectParams& p, SelectShared<WAVES>& sh, const float* x,
                                       int n, int32_t* keep, float* sums) {
  constexpr int THREADS = WAVES * kWave;
  constexpr int BINS = kBins / THREADS;  // of a thread
  const int t = threadIdx.x, wave = t >> 6, lane = t & 63;
  const Tokens<WAVES, KPT> row(p, x, n);
  int want = p.budget - p.sinks - p.recent;  // of the tokens between
  // Those above `most` stay, and of those from `least` on the first `want`.
  uint32_t least = kAlways, most = kAlways - 1;
  if (want > 0) {
    least = 0;
    for (int d = 0; d < kDigits; ++d) {
      const int shift = digit_shift(d), bits = digit_bits(d), above = shift + bits;
#pragma unroll
      for (int k = 0; k < BINS; ++k) sh.count[k * THREADS + t] = 0;
      __syncthreads();
      row.each([&](int, uint32_t u) {
        if (d == 0 ? u - 1 < kAlways - 1 : u >> above == least >> above)
          atomicAdd(&sh.count[u >> shift & ((1u << bits) - 1)], 1);
      });
      __syncthreads();
      // from the heaviest bin down, BINS a thread
      int c[BINS], mine = 0;
#pragma unroll
      for (int k = 0; k < BINS; ++k) mine += c[k] = sh.count[kBins - 1 - (t * BINS + k)];
      int inc = mine;
#pragma unroll
      for (int off = 1; off < kWave; off <<= 1) {
        const int o = __shfl_up(inc, off, kWave);
        inc += lane >= off ? o : 0;
      }
      if (lane == 63) sh.sum[wave] = inc;
      __syncthreads();
      int before = inc - mine;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) before += w < wave ? sh.sum[w] : 0;
#pragma unroll
      for (int k = 0; k < BINS; ++k) {
        if (before < want && want <= before + c[k]) {
          sh.digit = kBins - 1 - (t * BINS + k);
          sh.rest = want - before;
          sh.same = c[k];
        }
        before += c[k];
      }
      __syncthreads();
      least |= sh.digit << shift;
      most = least | ((1u << shift) - 1);
      want = sh.rest;
      if (want == sh.same) break;  // all of this bin stay, whatever their further digits
    }
  } else {
    want = 0;
  }
  int more_before = 0, tie_before = 0;  // of this wave, then of those before it
  row.each([&](int, uint32_t u) {
    more_before += __popcll(__ballot(u > most));
    tie_before += __popcll(__ballot(u >= least));
  });
  if (lane == 0) sh.part[wave] = make_int2(more_before, tie_before - more_before);
  __syncthreads();
  more_before = tie_before = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    const int2 o = sh.part[w];
    more_before += w < wave ? o.x : 0;
    tie_before += w < wave ? o.y : 0;
  }
  auto rank = [](uint64_t mask) {  // lanes of it before this one
    return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                          __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
  };
  row.each([&](int i, uint32_t u) {
    const uint64_t m = __ballot(u > most), e = __ballot(u >= least) & ~m;
    if (!(m | e)) return;
    const int ties = tie_before + rank(e);
    const int at = more_before + rank(m) + (ties < want ? ties : want);
    if (u > most || (u >= least && ties < want)) {
      keep[at] = i;
      if (sums) sums[at] = x[i];
    }
    more_before += __popcll(m);
    tie_before += __popcll(e);
  });
}

// One workgroup per (sequence, head).  Four waves a SIMD: with eight the 32 tokens a lane do not
// fit its registers (66 us against 31 for 384 long rows).
template <int WAVES>
__global__ __launch_bounds__(WAVES * kWave, 4) void cache_select_kernel(SelectParams p) {
  constexpr int THREADS = WAVES * kWave;
  __shared__ SelectShared<WAVES> sh;
  const int t = threadIdx.x;
  int b = blockIdx.x / p.H;
  const int h = blockIdx.x - b * p.H;
  if (p.sorted) {
    // the longest sequences first: workgroup b of a head takes the one of rank b
    if (t < kWave) {
      const int mine = t < p.B ? p.lens[t] : INT32_MIN;
      int rank = 0;
      for (int i = 0; i < p.B; ++i) {
        const int other = __builtin_amdgcn_readlane(mine, i);
        rank += other > mine || (other == mine && i < t);
      }
      if (t < p.B && rank == b) sh.rest = t;
    }
    __syncthreads();
    b = sh.rest;
    __syncthreads();
  }
  const int row = b * p.H + h;
  const int len = p.lens[b];
  const int n = len < 0 ? 0 : len < p.S ? len : p.S;
  const float* x = p.scores + b * p.s_seq + h * p.s_head;
  int32_t* keep = p.keep + (int64_t)row * p.budget;
  float* sums = p.sums ? p.sums + (int64_t)row * p.budget : nullptr;
  if (h == 0 && t == 0) p.counts[b] = n < p.budget ? n : p.budget;
  if (n <= p.budget) {
    for (int i = t; i < p.budget; i += THREADS) {
      keep[i] = i < n ? i : -1;
      if (sums) sums[i] = i < n ? x[i] : 0.f;
    }
    return;
  }
  if constexpr (WAVES == 4) {
    if (n <= 4 * THREADS) choose<WAVES, 4>(p, sh, x, n, keep, sums);
    else choose<WAVES, 16>(p, sh, x, n, keep, sums);
  } else {
    if (n <= 8 * THREADS) choose<WAVES, 8>(p, sh, x, n, keep, sums);
    else if (n <= 32 * THREADS) choose<WAVES, 32>(p, sh, x, n, keep, sums);
    else choose<WAVES, 0>(p, sh, x, n, keep, sums);
  }
}

// How many tokens stay of each sequence, where there are no heads to choose for.
constexpr int kCountThreads = 256;
__global__ __launch_bounds__(kCountThreads) void cache_counts_kernel(SelectParams p) {
  const int b = blockIdx.x * kCountThreads + threadIdx.x;
  if (b >= p.B) return;
  const int most = p.S < p.budget ? p.S : p.budget, len = p.lens[b];
  p.counts[b] = len < 0 ? 0 : len < most ? len : most;
}

// ------------------------------------------------------------------ the move

struct Row;
struct KeepParams {
  unsigned char* pool;
  int64_t planes, page_bytes, n_pages;
  int64_t row_bytes, head_bytes;  // of a token, of one of its `heads` parts
  int32_t page_size, rows, width, groups, heads, n;
  FastDiv page;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* keep;
  const int32_t* counts;
  const int32_t* base;
  int32_t* table_out;
  int32_t* lens_out;
  int32_t* result;
  // workspace
  uint32_t* held;    // ceil(n_pages / 32): some row holds it
  uint32_t* shared;  // .. and another entry does too
  uint32_t* fresh;   // [rows][ceil(width / 32)]: entries that get a free page
  int32_t* need;     // [rows] how many
  int32_t* spare;    // [n_pages] free pages in ascending order
  Row* row;          // [rows] what becomes of it
};

__device__ __forceinline__ bool names_page(const KeepParams& p, int32_t id) {
  return (uint32_t)id < (uint32_t)p.n_pages;
}
__device__ __forceinline__ int entries(const KeepParams& p, int tokens) {
  return (int)(((uint32_t)tokens + (uint32_t)p.page_size - 1) / (uint32_t)p.page_size);
}
__device__ __forceinline__ int tokens_of(const KeepParams& p, int row) {
  const int64_t cap = (int64_t)p.width * p.page_size;
  const int n = p.lens[row];
  return n < 0 ? 0 : n < cap ? n : (int)cap;
}
// The tokens [0, first) of a row stay where they are; it has `total` after the move.
struct alignas(16) Row {
  int tokens, first, total;
  int moves;  // 0: refused, the row stays as it is
};
__device__ __forceinline__ Row row_of(const KeepParams& p, int r) {
  Row x;
  x.tokens = tokens_of(p, r);
  x.first = p.base ? p.base[r] : 0;
  x.first = x.first < 0 ? 0 : x.first < x.tokens ? x.first : x.tokens;
  int c = p.counts[r];
  c = c < 0 ? 0 : c < p.n ? c : p.n;
  x.total = c < x.tokens - x.first ? x.first + c : x.tokens;
  x.moves = 1;
  return x;
}
// The token that goes to slot i, -1 if the list names none from i on.
__device__ __forceinline__ int source_of(const KeepParams& p, const Row& x, int g, int r, int h, int i) {
  if (i < x.first) return i;
  const int t = p.keep[(((int64_t)g * p.rows + r) * p.heads + h) * p.n + (i - x.first)];
  return t >= i && t < x.tokens ? t : -1;
}

constexpr int kKeepThreads = 256;

__global__ __launch_bounds__(kKeepThreads) void keep_clear_kernel(KeepParams p) {
  const int64_t words = (p.n_pages + 31) / 32, marks = (int64_t)p.rows * ((p.width + 31) / 32);
  const int64_t step = (int64_t)gridDim.x * kKeepThreads;
  for (int64_t i = blockIdx.x * kKeepThreads + threadIdx.x; i < words; i += step)
    p.held[i] = p.shared[i] = 0;
  for (int64_t i = blockIdx.x * kKeepThreads + threadIdx.x; i < marks; i += step) p.fresh[i] = 0;
}

// Marks the pages of a row.
__device__ __forceinline__ bool mark_row(const KeepParams& p, int r, int tokens, int thread,
                                         int threads) {
  const int held = entries(p, tokens);
  bool any = false;  // page that another entry has marked before
  for (int e = thread; e < held; e += threads) {
    const int32_t id = p.table[(int64_t)r * p.width + e];
    if (!names_page(p, id)) continue;
    const uint32_t bit = 1u << (id & 31);
    if (atomicOr(&p.held[id >> 5], bit) & bit) {
      atomicOr(&p.shared[id >> 5], bit);
      any = true;
    }
  }
  return any;
}

// The entries of a row that need a page of their own, by a wave: shared ones with a slot that
// gets another token.  Returns their number.
__device__ __forceinline__ int mark_fresh(const KeepParams& p, int r, const Row& x, int lane) {
  const int64_t lists = (int64_t)p.groups * p.heads;
  const int held = entries(p, x.total);
  int need = 0;
  for (int e0 = x.first / p.page_size; e0 < held; e0 += kWave) {
    const int mine = e0 + lane;
    const int32_t id = mine < held ? p.table[(int64_t)r * p.width + mine] : -1;
    const bool shares = names_page(p, id) && p.shared[id >> 5] >> (id & 31) & 1;
    for (uint64_t todo = __ballot(shares); todo; todo &= todo - 1) {
      const int e = e0 + __builtin_ctzll(todo);
      const int64_t begin = (int64_t)e * p.page_size, end = begin + p.page_size;
      const int from = begin > x.first ? (int)begin : x.first;
      const int slots = (end < x.total ? (int)end : x.total) - from;
      // four of the lists' entries a lane at once, until one is found
      bool acts = false;
      for (int64_t k0 = lane; k0 - lane < lists * slots && !__any(acts); k0 += 4 * kWave) {
        int t[4], i[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int64_t k = k0 + u * kWave;
          const int list = (int)(k / slots);
          i[u] = from + (int)(k - (int64_t)list * slots);
          t[u] = k < lists * slots ? source_of(p, x, list / p.heads, r, list % p.heads, i[u]) : -1;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) acts |= t[u] >= 0 && t[u] != i[u];
      }
      if (__any(acts)) {
        if (lane == 0) p.fresh[(int64_t)r * ((p.width + 31) / 32) + e / 32] |= 1u << (e & 31);
        ++need;
      }
    }
  }
  return need;
}

__global__ __launch_bounds__(kKeepThreads) void keep_mark_kernel(KeepParams p) {
  (void)mark_row(p, blockIdx.x, tokens_of(p, blockIdx.x), threadIdx.x, kKeepThreads);
}
__global__ __launch_bounds__(kKeepThreads) void keep_need_kernel(KeepParams p) {
  const int r = (int)((blockIdx.x * kKeepThreads + threadIdx.x) / kWave);
  if (r >= p.rows) return;
  const Row x = row_of(p, r);
  const int n = mark_fresh(p, r, x, threadIdx.x & 63);
  if ((threadIdx.x & 63) == 0) p.row[r] = x;
  if ((threadIdx.x & 63) == 0) p.need[r] = n;
}

// Ranks the free pages and deals them out to the rows in order; the new state.
__device__ __forceinline__ void deal_pages(const KeepParams& p, int* red) {
  const int t = threadIdx.x;
  const int words = (int)((p.n_pages + 31) / 32);
  const int per = (words + kScanThreads - 1) / kScanThreads;
  const int w0 = t * per < words ? t * per : words, w1 = w0 + per < words ? w0 + per : words;
  auto open = [&](int w) {
    const int64_t left = p.n_pages - (int64_t)w * 32;
    return ~p.held[w] & (left >= 32 ? 0xffffffffu : (1u << left) - 1);
  };
  __shared__ int64_t red64[kScanThreads / kWave];  // wishes may add up past 32 bits
  int64_t wanted = 0;
  for (int r0 = 0; r0 < p.rows; r0 += kScanThreads) {
    int64_t total;
    (void)scan_block(r0 + t < p.rows ? (int64_t)p.need[r0 + t] : 0, red64, total);
    wanted += total;
  }
  int free_pages = 0;
  if (wanted > 0) {  // as many of the free pages as are wanted
    int mine = 0;
    for (int w = w0; w < w1; ++w) mine += __popc(open(w));
    int rank = scan_block(mine, red, free_pages);
    for (int w = w0; w < w1 && rank < wanted; ++w)
      for (uint32_t f = open(w); f && rank < wanted; f &= f - 1)
        p.spare[rank++] = w * 32 + __ffs(f) - 1;
  }
  __syncthreads();
  int64_t base = 0;
  int refused = 0;
  for (int r0 = 0; r0 < p.rows; r0 += kScanThreads) {
    const int r = r0 + t;
    const int64_t need = r < p.rows ? p.need[r] : 0;
    int64_t total;
    const int64_t before = base + scan_block(need, red64, total);
    base += total;
    if (r < p.rows) {
      const bool ok = need == 0 || before + need <= free_pages;
      p.row[r].moves = ok;
      p.need[r] = (int)(ok ? before : 0);  // from here on: its first free page
      refused += !ok;
    }
  }
  int total;
  (void)scan_block(refused, red, total);
  if (t == 0) *p.result = total;
}

__global__ __launch_bounds__(kScanThreads) void keep_deal_kernel(KeepParams p) {
  __shared__ int red[kScanThreads / kWave];
  deal_pages(p, red);
}

// A row's length and its part of the new table, by the threads of a wave or more.
__device__ __forceinline__ void write_row(const KeepParams& p, int r, int thread, int threads) {
  const Row x = p.row[r];
  const int tokens = x.moves ? x.total : x.tokens, held = entries(p, tokens);
  const uint32_t* fresh = p.fresh + (int64_t)r * ((p.width + 31) / 32);
  if (thread == 0) p.lens_out[r] = tokens;
  for (int e = thread; e < p.width; e += threads) {
    int32_t id = e < held ? p.table[(int64_t)r * p.width + e] : -1;
    if (e < held && x.moves && fresh[e / 32] >> (e & 31) & 1) {
      int k = p.need[r] + __popc(fresh[e / 32] & ((1u << (e & 31)) - 1));
      for (int w = 0; w < e / 32; ++w) k += __popc(fresh[w]);
      id = p.spare[k];
    }
    p.table_out[(int64_t)r * p.width + e] = id;
  }
}
__global__ __launch_bounds__(kKeepThreads) void keep_table_kernel(KeepParams p) {
  write_row(p, blockIdx.x, threadIdx.x, kKeepThreads);
}

// All of the bookkeeping by one workgroup, the bitmaps and rows in LDS: one launch instead
// of five.
constexpr int kOnePages = 64 * 1024, kOneRows = 256, kOneEntries = 48 * 1024;
constexpr int kOneMarks = kOneEntries / 32 + kOneRows;
__global__ __launch_bounds__(kScanThreads) void keep_one_kernel(KeepParams p) {
  __shared__ int red[kScanThreads / kWave];
  __shared__ uint32_t sHeld[kOnePages / 32], sShared[kOnePages / 32], sFresh[kOneMarks];
  __shared__ Row sRow[kOneRows];
  __shared__ int sNeed[kOneRows];
  const int t = threadIdx.x, wave = t >> 6, lane = t & 63;
  constexpr int kWaves = kScanThreads / kWave;
  uint32_t* const fresh = p.fresh;
  Row* const row = p.row;
  p.held = sHeld;
  p.shared = sShared;
  p.fresh = sFresh;
  p.row = sRow;
  p.need = sNeed;
  const int marks = p.rows * ((p.width + 31) / 32);
  if (t < p.rows) {
    sRow[t] = row_of(p, t);
    sNeed[t] = 0;
  }
  for (int i = t; i < (p.n_pages + 31) / 32; i += kScanThreads) sHeld[i] = sShared[i] = 0;
  for (int i = t; i < marks; i += kScanThreads) sFresh[i] = 0;
  __syncthreads();
  bool any = false;
  for (int r = wave; r < p.rows; r += kWaves) any |= mark_row(p, r, sRow[r].tokens, lane, kWave);
  if (__syncthreads_or(any)) {  // a page is shared
    for (int r = wave; r < p.rows; r += kWaves) {
      const int n = mark_fresh(p, r, sRow[r], lane);
      if (lane == 0) sNeed[r] = n;
    }
    __syncthreads();
    deal_pages(p, red);
    __syncthreads();
  } else if (t == 0) {
    *p.result = 0;
  }
  for (int r = wave; r < p.rows; r += kWaves) write_row(p, r, lane, kWave);
  for (int i = t; i < marks; i += kScanThreads) fresh[i] = sFresh[i];
  if (t < p.rows) row[t] = sRow[t];
}

// Bytes of a token's part that a workgroup moves, a column of the row's slots: the least and
// the most.
constexpr int64_t kColumn = 256, kMostColumn = 16 * kKeepThreads;
constexpr int kDepth = 4;  // loads of a thread under way
constexpr int64_t kMostBlocks = 1 << 20;  // of a launch

// A workgroup takes a column of a part of a row's tokens in one plane, slots in
// ascending order.
__device__ __forceinline__ void move_column(const KeepParams& p, const Row& x, int r, int h, int column,
                                            int plane, int64_t width) {
  const int g = plane / (int)(p.planes / p.groups);
  const int64_t at = (int64_t)h * p.head_bytes + column * width;
  const int64_t rest = p.head_bytes - column * width;
  const int lanes = (int)(rest < width ? rest : width) / 16, slots = kKeepThreads / lanes;
  const int sub = threadIdx.x / lanes, lane = threadIdx.x - sub * lanes;
  unsigned char* const pool = p.pool + (int64_t)plane * p.n_pages * p.page_bytes + at + lane * 16;
  const int32_t* const from = p.table + (int64_t)r * p.width;
  const int32_t* const to = p.table_out + (int64_t)r * p.width;
  const uint32_t* const fresh = p.fresh + (int64_t)r * ((p.width + 31) / 32);
  // One part: kDepth slots a thread.  src, dst: bytes from `pool`, -1 where nothing moves.
  struct Part {
    int64_t src[kDepth], dst[kDepth];
    u32x4 v[kDepth];
  };
  auto locate = [&](int64_t i0, Part& w) {
    int t[kDepth];
#pragma unroll
    for (int k = 0; k < kDepth; ++k) {
      const int64_t i = i0 + k * slots + sub;
      t[k] = sub < slots && i < x.total ? source_of(p, x, g, r, h, (int)i) : INT32_MIN;
    }
#pragma unroll
    for (int k = 0; k < kDepth; ++k) {
      w.src[k] = w.dst[k] = -1;
      const int i = (int)(i0 + k * slots + sub);
      if (t[k] == INT32_MIN) continue;
      const int e = (int)div_page(p.page, i);
      if (t[k] < 0 || t[k] == i) {  // the slot keeps its token
        if (!(fresh[e / 32] >> (e & 31) & 1)) continue;
        t[k] = i;
      }
      const int es = (int)div_page(p.page, t[k]);
      const int32_t sp = from[es], dp = to[e];
      if (!names_page(p, sp) || !names_page(p, dp)) continue;
      w.src[k] = sp * p.page_bytes + (t[k] - es * p.page_size) * p.row_bytes;
      w.dst[k] = dp * p.page_bytes + (i - e * p.page_size) * p.row_bytes;
    }
  };
  auto read = [&](Part& w) {
#pragma unroll
    for (int k = 0; k < kDepth; ++k)
      if (w.src[k] >= 0)
        w.v[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(pool + w.src[k]));
  };
  auto write = [&](Part& w) {
    // every thread's reads of this part have returned before any of its writes; those of
    // the next part, which are under way, lie behind all that this one writes
#pragma unroll
    for (int k = 0; k < kDepth; ++k) asm volatile("" : "+v"(w.v[k])::"memory");
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kDepth; ++k)
      if (w.dst[k] >= 0)
        __builtin_nontemporal_store(w.v[k], reinterpret_cast<u32x4*>(pool + w.dst[k]));
  };
  // tokens before the first list entry move only with their whole page
  const int64_t step = (int64_t)slots * kDepth;
  int64_t i0 = x.first / p.page_size * p.page_size;
  Part a, b;
  locate(i0, a);
  read(a);
  for (; i0 < x.total; i0 += 2 * step) {
    locate(i0 + step, b);
    read(b);
    write(a);
    if (i0 + step >= x.total) break;
    locate(i0 + 2 * step, a);
    read(a);
    write(b);
  }
}

__global__ __launch_bounds__(kKeepThreads) void keep_move_kernel(KeepParams p, int64_t width,
                                                                 int64_t items) {
  const int64_t columns = (p.head_bytes + width - 1) / width;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int plane = (int)(item % p.planes), column = (int)(item / p.planes % columns);
    const int64_t part = item / p.planes / columns;
    const int h = (int)(part % p.heads), r = (int)(part / p.heads);
    const Row x = p.row[r];
    if (x.moves) move_column(p, x, r, h, column, plane, width);
  }
}

int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

}  // namespace

hipError_t launch_cache_select(const SelectArgs& a, hipStream_t stream) {
  SelectParams p{};
  p.scores = a.scores;
  p.s_seq = a.s_seq;
  p.s_head = a.s_head;
  p.lens = a.lens;
  p.keep = a.keep;
  p.counts = a.counts;
  p.sums = a.sums;
  p.S = (int32_t)a.S;
  p.B = (int32_t)a.B;
  p.H = (int32_t)a.H;
  p.budget = (int32_t)a.budget;
  p.recent = (int32_t)a.recent;
  p.sinks = (int32_t)a.sinks;
  if (a.H == 0) {
    hipLaunchKernelGGL(cache_counts_kernel, dim3((uint32_t)((a.B + kCountThreads - 1) / kCountThreads)),
                       dim3(kCountThreads), 0, stream, p);
    return hipGetLastError();
  }
  const dim3 grid((uint32_t)(a.B * a.H));
  // More rows than are at work at once, long ones among them: the longest first, so that none
  // of those begins last.
  p.sorted = a.S > 4096 && a.B > 1 && a.B <= kWave && a.B * a.H > device_cus();
  // (four waves hold 4096 tokens in registers, and their barriers are shorter)
  if (a.S <= 4096)
    hipLaunchKernelGGL(cache_select_kernel<4>, grid, dim3(4 * kWave), 0, stream, p);
  else
    hipLaunchKernelGGL(cache_select_kernel<16>, grid, dim3(16 * kWave), 0, stream, p);
  return hipGetLastError();
}

int64_t keep_workspace_bytes(int64_t rows, int64_t width, int64_t n_pages) {
  return 2 * up16(4 * ((n_pages + 31) / 32)) + up16(4 * rows * ((width + 31) / 32)) +
         up16(4 * rows) + 16 * rows + up16(4 * n_pages);
}

hipError_t launch_pages_keep(const KeepArgs& a, hipStream_t s) {
  KeepParams p{};
  p.pool = a.pages.pool;
  p.planes = a.pages.planes;
  p.page_bytes = a.pages.page_bytes;
  p.n_pages = a.pages.n_pages;
  p.page_size = (int32_t)a.pages.page_size;
  p.page = fast_div(a.pages.page_size);
  p.row_bytes = a.pages.page_bytes / a.pages.page_size;
  p.head_bytes = p.row_bytes / a.heads;
  p.rows = (int32_t)a.pages.rows;
  p.width = (int32_t)a.pages.width;
  p.groups = (int32_t)a.groups;
  p.heads = (int32_t)a.heads;
  p.n = (int32_t)a.n;
  p.table = a.pages.table;
  p.lens = a.pages.lens;
  p.keep = a.keep;
  p.counts = a.counts;
  p.base = a.base;
  p.table_out = a.pages.table_out;
  p.lens_out = a.pages.lens_out;
  p.result = a.pages.result;
  unsigned char* w = static_cast<unsigned char*>(a.pages.workspace);
  auto take = [&](int64_t count) {
    unsigned char* q = w;
    w += up16(4 * count);
    return q;
  };
  p.held = reinterpret_cast<uint32_t*>(take((p.n_pages + 31) / 32));
  p.shared = reinterpret_cast<uint32_t*>(take((p.n_pages + 31) / 32));
  p.fresh = reinterpret_cast<uint32_t*>(take((int64_t)p.rows * ((p.width + 31) / 32)));
  p.need = reinterpret_cast<int32_t*>(take(p.rows));
  p.row = reinterpret_cast<Row*>(take(4 * (int64_t)p.rows));
  p.spare = reinterpret_cast<int32_t*>(take(p.n_pages));
  if (p.rows <= kOneRows && (int64_t)p.rows * p.width <= kOneEntries && p.n_pages <= kOnePages) {
    hipLaunchKernelGGL(keep_one_kernel, dim3(1), dim3(kScanThreads), 0, s, p);
  } else {
    const int64_t words = (p.n_pages + 31) / 32 + (int64_t)p.rows * ((p.width + 31) / 32);
    const int64_t blocks = (words + kKeepThreads - 1) / kKeepThreads;
    hipLaunchKernelGGL(keep_clear_kernel, dim3((uint32_t)(blocks < 1024 ? blocks : 1024)),
                       dim3(kKeepThreads), 0, s, p);
    constexpr int kRowWaves = kKeepThreads / kWave;
    if (p.rows > 0) {
      hipLaunchKernelGGL(keep_mark_kernel, dim3(p.rows), dim3(kKeepThreads), 0, s, p);
      hipLaunchKernelGGL(keep_need_kernel, dim3((p.rows + kRowWaves - 1) / kRowWaves),
                         dim3(kKeepThreads), 0, s, p);
    }
    hipLaunchKernelGGL(keep_deal_kernel, dim3(1), dim3(kScanThreads), 0, s, p);
    if (p.rows > 0)
      hipLaunchKernelGGL(keep_table_kernel, dim3(p.rows), dim3(kKeepThreads), 0, s, p);
  }
  if (p.rows > 0) {
    // Columns as wide as leaves two workgroups for a CU: with few tokens to move each
    // costs its chain of look-ups.  Measured (us on the GPU): 8 rows of up to 24 tokens of 2 KB
    // in 32 planes, columns of 256 bytes 12.5, of 1024 6.7.
    const int64_t parts = (int64_t)p.rows * p.heads * p.planes;
    int64_t width = kMostColumn, items;
    while (width > kColumn && (p.head_bytes + width - 1) / width * parts < 2 * device_cus()) width /= 2;
    items = (p.head_bytes + width - 1) / width * parts;
    if (items > 0)
      hipLaunchKernelGGL(keep_move_kernel, dim3((uint32_t)(items < kMostBlocks ? items : kMostBlocks)),
                         dim3(kKeepThreads), 0, s, p, width, items);
  }
  return hipGetLastError();
}

}  // namespace tq
