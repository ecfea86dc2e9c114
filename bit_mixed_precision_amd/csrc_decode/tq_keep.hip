// Caches that are kept short: which tokens stay, by the attention weight that they have
// received, and moving those together in their pages.
//
// The choice.  Of n > budget tokens the first `sinks` and the last `recent` stay, and of
// those between as many of the heaviest as the budget leaves, equal ones in order.
// The least weight that stays is found digit by digit, from counts of the tokens by
// 11, 11 and 10 bits of their weight (as a whole number of the same order); then the
// tokens are walked through in order.
//
// The move.  Slot i of a row gets token keep[i] >= i of the same row, so a row can be
// moved forward in place, part by part: what a part writes no later part reads.  A page
// that other rows hold too is not written; the row gets a free page in its place.

#include "tq.h"
#include "tq_common.h"
#include "tq_decode.h"
#include "tq_kernels.h"
#include "tq_scan.h"

namespace tq {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------ the choice

struct SelectParams {
  const float* scores;
  int64_t s_seq, s_head;
  const int32_t* lens;
  int32_t* keep;
  int32_t* counts;
  float* sums;
  int32_t S, B, H, budget, recent, sinks;
};

constexpr int kDigits = 3;
__device__ constexpr int kDigitShift[kDigits] = {21, 10, 0};
__device__ constexpr int kDigitBits[kDigits] = {11, 11, 10};
constexpr int kBins = 2048;

// A weight as a whole number of the same order: -0 as 0, NaN as the least.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.f);
  if (x != x) return 0x007fffffu;  // -inf
  return u >> 31 ? ~u : u | 0x80000000u;
}

// One workgroup per (sequence, head).
__global__ __launch_bounds__(kScanThreads) void cache_select_kernel(SelectParams p) {
  __shared__ int sCount[kBins];
  __shared__ int red[kScanThreads / kWave];
  __shared__ uint32_t sDigit;
  __shared__ int sRest;
  const int t = threadIdx.x;
  const int b = blockIdx.x / p.H, h = blockIdx.x - b * p.H;
  const int len = p.lens[b];
  const int n = len < 0 ? 0 : len < p.S ? len : p.S;
  const float* x = p.scores + b * p.s_seq + h * p.s_head;
  int32_t* keep = p.keep + (int64_t)blockIdx.x * p.budget;
  float* sums = p.sums ? p.sums + (int64_t)blockIdx.x * p.budget : nullptr;
  if (h == 0 && t == 0) p.counts[b] = n < p.budget ? n : p.budget;
  if (n <= p.budget) {
    for (int i = t; i < p.budget; i += kScanThreads) {
      keep[i] = i < n ? i : -1;
      if (sums) sums[i] = i < n ? x[i] : 0.f;
    }
    return;
  }
  const int lo = p.sinks, hi = n - p.recent;  // the tokens to choose from
  int want = p.budget - p.sinks - p.recent;   // fewer than hi - lo of them
  uint32_t least = 0;  // digits found so far: of the want-th heaviest
  if (want > 0) {
    for (int d = 0; d < kDigits; ++d) {
      const int shift = kDigitShift[d], bits = kDigitBits[d], above = shift + bits;
      for (int i = t; i < kBins; i += kScanThreads) sCount[i] = 0;
      __syncthreads();
      for (int i = lo + t; i < hi; i += kScanThreads) {
        const uint32_t u = order_of(x[i]);
        if (d == 0 || u >> above == least >> above)
          atomicAdd(&sCount[u >> shift & ((1u << bits) - 1)], 1);
      }
      __syncthreads();
      // from the heaviest bin down: two bins a thread
      const int b1 = kBins - 1 - 2 * t, c1 = sCount[b1], c0 = sCount[b1 - 1];
      int total;
      const int before = scan_block(c1 + c0, red, total);
      if (before < want && want <= before + c1) {
        sDigit = b1;
        sRest = want - before;
      } else if (before + c1 < want && want <= before + c1 + c0) {
        sDigit = b1 - 1;
        sRest = want - before - c1;
      }
      __syncthreads();
      least |= sDigit << shift;
      want = sRest;
      __syncthreads();
    }
  }
  // `want` of the tokens of just the least weight stay, the first ones
  int kept = 0, ties = 0;
  const bool any = p.budget > p.sinks + p.recent;
  for (int i0 = 0; i0 < n; i0 += kScanThreads) {
    const int i = i0 + t;
    bool stays = false, tie = false;
    float v = 0.f;
    if (i < n) {
      v = x[i];
      const uint32_t u = order_of(v);
      const bool choose = i >= lo && i < hi;
      stays = !choose || (any && u > least);
      tie = choose && any && u == least;
    }
    int total;
    const int tie_rank = ties + scan_block((int)tie, red, total);
    ties += total;
    stays |= tie && tie_rank < want;
    const int at = kept + scan_block((int)stays, red, total);
    kept += total;
    if (stays && at < p.budget) {
      keep[at] = i;
      if (sums) sums[at] = v;
    }
  }
}

// ------------------------------------------------------------------ the move

struct KeepParams {
  unsigned char* pool;
  int64_t planes, page_bytes, n_pages;
  int64_t row_bytes, head_bytes;  // of a token, of one of its `heads` parts
  int32_t page_size, rows, width, groups, heads, n;
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
  int32_t* moved;    // [rows] tokens after the move, -1: the row stays as it is
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
struct Row {
  int tokens, first, total;
};
__device__ __forceinline__ Row row_of(const KeepParams& p, int r) {
  Row x;
  x.tokens = tokens_of(p, r);
  x.first = p.base ? p.base[r] : 0;
  x.first = x.first < 0 ? 0 : x.first < x.tokens ? x.first : x.tokens;
  int c = p.counts[r];
  c = c < 0 ? 0 : c < p.n ? c : p.n;
  x.total = c < x.tokens - x.first ? x.first + c : x.tokens;
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
__device__ __forceinline__ void mark_row(const KeepParams& p, int r, int thread, int threads) {
  const int held = entries(p, tokens_of(p, r));
  for (int e = thread; e < held; e += threads) {
    const int32_t id = p.table[(int64_t)r * p.width + e];
    if (!names_page(p, id)) continue;
    const uint32_t bit = 1u << (id & 31);
    if (atomicOr(&p.held[id >> 5], bit) & bit) atomicOr(&p.shared[id >> 5], bit);
  }
}

// The entries of a row that need a page of their own, by a workgroup; returns their number.
__device__ __forceinline__ int mark_fresh(const KeepParams& p, int r, int* sNeed) {
  const Row x = row_of(p, r);
  if (threadIdx.x == 0) *sNeed = 0;
  __syncthreads();
  const int64_t lists = (int64_t)p.groups * p.heads;
  for (int e = x.first / p.page_size; e < entries(p, x.total); ++e) {
    const int32_t id = p.table[(int64_t)r * p.width + e];
    if (!names_page(p, id) || !(p.shared[id >> 5] >> (id & 31) & 1)) continue;
    const int from = e * p.page_size > x.first ? e * p.page_size : x.first;
    const int64_t end = (int64_t)(e + 1) * p.page_size;
    const int slots = (end < x.total ? (int)end : x.total) - from;
    bool acts = false;
    for (int64_t k = threadIdx.x; k < lists * slots && !acts; k += blockDim.x) {
      const int list = (int)(k / slots), i = from + (int)(k - (int64_t)list * slots);
      const int t = source_of(p, x, list / p.heads, r, list % p.heads, i);
      acts = t >= 0 && t != i;
    }
    if (__syncthreads_or(acts) && threadIdx.x == 0) {
      p.fresh[(int64_t)r * ((p.width + 31) / 32) + e / 32] |= 1u << (e & 31);
      ++*sNeed;
    }
  }
  __syncthreads();
  return *sNeed;
}

__global__ __launch_bounds__(kKeepThreads) void keep_mark_kernel(KeepParams p) {
  mark_row(p, blockIdx.x, threadIdx.x, kKeepThreads);
}
__global__ __launch_bounds__(kKeepThreads) void keep_need_kernel(KeepParams p) {
  __shared__ int sNeed;
  const int n = mark_fresh(p, blockIdx.x, &sNeed);
  if (threadIdx.x == 0) p.need[blockIdx.x] = n;
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
  int mine = 0, free_pages;
  for (int w = w0; w < w1; ++w) mine += __popc(open(w));
  int rank = scan_block(mine, red, free_pages);
  for (int w = w0; w < w1; ++w)
    for (uint32_t f = open(w); f; f &= f - 1) p.spare[rank++] = w * 32 + __ffs(f) - 1;
  __syncthreads();
  __shared__ int64_t red64[kScanThreads / kWave];  // wishes may add up past 32 bits
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
      const Row x = row_of(p, r);
      p.lens_out[r] = ok ? x.total : x.tokens;
      p.moved[r] = ok ? x.total : -1;
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

// A row of the new table, by the threads of a wave or more.
__device__ __forceinline__ void write_table(const KeepParams& p, int r, int thread, int threads) {
  const int held = entries(p, p.lens_out[r]);
  const uint32_t* fresh = p.fresh + (int64_t)r * ((p.width + 31) / 32);
  for (int e = thread; e < p.width; e += threads) {
    int32_t id = e < held ? p.table[(int64_t)r * p.width + e] : -1;
    if (e < held && p.moved[r] >= 0 && fresh[e / 32] >> (e & 31) & 1) {
      int k = p.need[r] + __popc(fresh[e / 32] & ((1u << (e & 31)) - 1));
      for (int w = 0; w < e / 32; ++w) k += __popc(fresh[w]);
      id = p.spare[k];
    }
    p.table_out[(int64_t)r * p.width + e] = id;
  }
}
__global__ __launch_bounds__(kKeepThreads) void keep_table_kernel(KeepParams p) {
  write_table(p, blockIdx.x, threadIdx.x, kKeepThreads);
}

// Bytes of a token's part that a workgroup moves: a column of the row's slots.
constexpr int kColumn = 256;
constexpr int kDepth = 4;  // loads of a thread under way
constexpr int64_t kMostBlocks = 1 << 20;  // of a launch

// A workgroup takes a column of a part of a row's tokens in one plane, slots in
// ascending order.
__device__ __forceinline__ void move_column(const KeepParams& p, int r, int h, int column, int plane) {
  const Row x = row_of(p, r);
  const int g = plane / (int)(p.planes / p.groups);
  const int64_t at = (int64_t)h * p.head_bytes + (int64_t)column * kColumn;
  const int64_t rest = p.head_bytes - (int64_t)column * kColumn;
  const int lanes = (int)(rest < kColumn ? rest : kColumn) / 16, slots = kKeepThreads / lanes;
  const int sub = threadIdx.x / lanes, lane = threadIdx.x - sub * lanes;
  unsigned char* const pool = p.pool + (int64_t)plane * p.n_pages * p.page_bytes + at + lane * 16;
  const int32_t* const from = p.table + (int64_t)r * p.width;
  const int32_t* const to = p.table_out + (int64_t)r * p.width;
  const uint32_t* const fresh = p.fresh + (int64_t)r * ((p.width + 31) / 32);
  // tokens before the first list entry move only with their whole page
  int64_t i0 = x.first / p.page_size * p.page_size;
  for (; i0 < x.total; i0 += slots * kDepth) {
    u32x4 v[kDepth];
    int64_t dst[kDepth];
#pragma unroll
    for (int k = 0; k < kDepth; ++k) {
      const int64_t slot = i0 + k * slots + sub;
      dst[k] = -1;
      if (sub >= slots || slot >= x.total) continue;
      const int i = (int)slot, e = i / p.page_size;
      const int t = source_of(p, x, g, r, h, i);
      if (t < 0 || (t == i && !(fresh[e / 32] >> (e & 31) & 1))) continue;
      const int es = t / p.page_size;
      const int32_t sp = from[es], dp = to[e];
      if (!names_page(p, sp) || !names_page(p, dp)) continue;
      v[k] = *reinterpret_cast<const u32x4*>(pool + sp * p.page_bytes +
                                             (t - es * p.page_size) * p.row_bytes);
      dst[k] = dp * p.page_bytes + (i - e * p.page_size) * p.row_bytes;
    }
    // every read of this part has returned before any of its writes
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kDepth; ++k)
      if (dst[k] >= 0) *reinterpret_cast<u32x4*>(pool + dst[k]) = v[k];
  }
}

__global__ __launch_bounds__(kKeepThreads) void keep_move_kernel(KeepParams p, int columns,
                                                                 int64_t items) {
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int plane = (int)(item % p.planes), column = (int)(item / p.planes % columns);
    const int64_t part = item / p.planes / columns;
    const int h = (int)(part % p.heads), r = (int)(part / p.heads);
    if (p.moved[r] >= 0) move_column(p, r, h, column, plane);
  }
}

int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

}  // namespace

int64_t select_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

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
  hipLaunchKernelGGL(cache_select_kernel, dim3((uint32_t)(a.B * a.H)), dim3(kScanThreads), 0,
                     stream, p);
  return hipGetLastError();
}

int64_t keep_workspace_bytes(int64_t rows, int64_t width, int64_t n_pages) {
  return 2 * up16(4 * ((n_pages + 31) / 32)) + up16(4 * rows * ((width + 31) / 32)) +
         2 * up16(4 * rows) + up16(4 * n_pages);
}

hipError_t launch_pages_keep(const KeepArgs& a, hipStream_t s) {
  KeepParams p{};
  p.pool = a.pages.pool;
  p.planes = a.pages.planes;
  p.page_bytes = a.pages.page_bytes;
  p.n_pages = a.pages.n_pages;
  p.page_size = (int32_t)a.pages.page_size;
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
  p.moved = reinterpret_cast<int32_t*>(take(p.rows));
  p.spare = reinterpret_cast<int32_t*>(take(p.n_pages));
  const int64_t words = (p.n_pages + 31) / 32 + (int64_t)p.rows * ((p.width + 31) / 32);
  const int64_t blocks = (words + kKeepThreads - 1) / kKeepThreads;
  hipLaunchKernelGGL(keep_clear_kernel, dim3((uint32_t)(blocks < 1024 ? blocks : 1024)),
                     dim3(kKeepThreads), 0, s, p);
  if (p.rows > 0) {
    hipLaunchKernelGGL(keep_mark_kernel, dim3(p.rows), dim3(kKeepThreads), 0, s, p);
    hipLaunchKernelGGL(keep_need_kernel, dim3(p.rows), dim3(kKeepThreads), 0, s, p);
  }
  hipLaunchKernelGGL(keep_deal_kernel, dim3(1), dim3(kScanThreads), 0, s, p);
  if (p.rows > 0) {
    hipLaunchKernelGGL(keep_table_kernel, dim3(p.rows), dim3(kKeepThreads), 0, s, p);
    const int columns = (int)((p.head_bytes + kColumn - 1) / kColumn);
    const int64_t items = (int64_t)p.rows * p.heads * columns * p.planes;
    if (items > 0)
      hipLaunchKernelGGL(keep_move_kernel, dim3((uint32_t)(items < kMostBlocks ? items : kMostBlocks)),
                         dim3(kKeepThreads), 0, s, p, columns, items);
  }
  return hipGetLastError();
}

}  // namespace tq
