// The pages of a key-value cache: forking, growing, compacting, copying.
//
// The page tables and lengths are the state.  Which pages are free follows from
// them: a bitmap with one bit per page is filled from the held table entries
// (bit-wise or and integer counts only, so the order of the atomics does not
// show), one workgroup ranks its free (or used) bits by popcounts and a prefix
// sum, and the data moves in a last launch that reads the list of pairs and
// their number from device memory: no call waits for the host.  Small states take
// fewer launches: the bookkeeping by one workgroup in LDS, or by every workgroup
// that copies, each for itself.
//
// Bound: the copied pages, read and written once per plane.  Measured: compacting a
// pool of 2048 pages in 16 planes, 500 moved, 524 MB: 114 us a call, of which the
// copies take 106 (5.0 TB/s through the caches; a plain copy reaches 4.9, the rotation
// with its stores past them 5.85); growing 64 rows of 43 entries 6.6 us, 256 of 256 13.8;
// forking 16 requests of 4 beams, 32 pages copied in 32 planes, 67 MB: 15 us on the GPU,
// 8 of them the copies; one request of 4 beams 6 us (8 us a call), the bookkeeping's
// chain of dependent reads.

#include "tq.h"
#include "tq_common.h"
#include "tq_decode.h"
#include "tq_kernels.h"
#include "tq_scan.h"

namespace tq {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kPagesThreads = 256;

struct PagesParams {
  unsigned char* pool;
  int64_t planes, page_bytes;
  int32_t n_pages, page_size, rows_in, rows, width;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* parent;
  const int32_t* add;
  int32_t* table_out;
  int32_t* lens_out;
  int32_t* refs;
  int32_t* result;
  // workspace
  uint32_t* bits;   // ceil(n_pages / 32)
  int32_t* need;    // [rows] pages wanted by a row
  int32_t* last;    // [rows] fork: the page a row copies
  const int32_t* tokens;  // [rows] fork: lengths of the new rows
  int32_t* src;     // [n_pages] copies: from
  int32_t* dst;     // [n_pages] copies: to
  int32_t* spare;   // [n_pages] free pages in ascending order
  int32_t* map;     // [n_pages] compact: where a page goes
  int32_t* pairs;   // [1] number of (src, dst)
  bool writes;      // this workgroup writes the outputs
};

__device__ __forceinline__ bool names_page(const PagesParams& p, int32_t id) {
  return (uint32_t)id < (uint32_t)p.n_pages;
}
// Tokens and table entries of an input row.
__device__ __forceinline__ int tokens_of(const PagesParams& p, int row) {
  const int64_t cap = (int64_t)p.width * p.page_size;
  const int n = p.lens[row];
  return n < 0 ? 0 : n < cap ? n : (int)cap;
}
__device__ __forceinline__ int entries(const PagesParams& p, int tokens) {
  return (int)(((uint32_t)tokens + (uint32_t)p.page_size - 1) / (uint32_t)p.page_size);
}

// Pages that growing row r asks for; -1 if its row of the table is too short.
__device__ __forceinline__ int wanted_pages(const PagesParams& p, int r, int tokens) {
  const int64_t want = (int64_t)tokens + (p.add[r] > 0 ? p.add[r] : 0);
  const int64_t cap = (int64_t)p.width * p.page_size;
  return want > cap ? -1 : entries(p, (int)want) - entries(p, tokens);
}

__global__ __launch_bounds__(kPagesThreads) void pages_clear_kernel(PagesParams p) {
  const int words = (p.n_pages + 31) / 32;
  for (int i = blockIdx.x * kPagesThreads + threadIdx.x; i < p.n_pages;
       i += gridDim.x * kPagesThreads) {
    if (i < words) p.bits[i] = 0;
    if (p.refs) p.refs[i] = 0;
  }
}

enum { kFork = 0, kGrow = 1, kCompact = 2 };

// One workgroup per output row: copies the row, marks the pages it holds and
// says how many pages it wants.
template <int OP>
__global__ __launch_bounds__(kPagesThreads) void pages_rows_kernel(PagesParams p) {
  const int r = blockIdx.x;
  int from = r;
  if constexpr (OP == kFork) {
    from = p.parent[r];
    if ((uint32_t)from >= (uint32_t)p.rows_in) from = -1;
  }
  const int tokens = from < 0 ? 0 : tokens_of(p, from);
  const int n = entries(p, tokens);
  const int32_t* row = p.table + (int64_t)(from < 0 ? 0 : from) * p.width;
  int32_t* out = p.table_out + (int64_t)r * p.width;
  int copied = -1;  // entry that this row does not share
  if constexpr (OP == kFork) {
    __shared__ int sLater;
    if (threadIdx.x == 0) sLater = 0;
    __syncthreads();
    if (from >= 0 && tokens % p.page_size != 0) {
      int later = 0;
      for (int i = threadIdx.x; i < r; i += kPagesThreads) later |= p.parent[i] == from;
      if (later) sLater = 1;  // every writer writes 1
    }
    __syncthreads();
    if (sLater && names_page(p, row[n - 1])) copied = n - 1;
    if (threadIdx.x == 0) {
      p.need[r] = copied >= 0;
      p.last[r] = copied >= 0 ? row[copied] : -1;
      p.lens_out[r] = tokens;
    }
  }
  if constexpr (OP == kGrow) {
    if (threadIdx.x == 0) p.need[r] = wanted_pages(p, r, tokens);
  }
  for (int i = threadIdx.x; i < p.width; i += kPagesThreads) {
    int32_t id = -1;
    if (i < n) {
      id = row[i];
      if (i != copied && names_page(p, id)) {
        atomicOr(&p.bits[id >> 5], 1u << (id & 31));
        if (p.refs) atomicAdd(&p.refs[id], 1);
      }
    }
    if constexpr (OP != kCompact) out[i] = id;
  }
}

__device__ __forceinline__ uint32_t valid_bits(const PagesParams& p, int word) {
  const int left = p.n_pages - word * 32;
  return left >= 32 ? 0xffffffffu : (1u << left) - 1;
}

// One workgroup: ranks the free pages, in ascending order, into spare[0 .. limit)
// and returns how many there are in all.
__device__ __forceinline__ int list_free(const PagesParams& p, int limit, int* red) {
  const int words = (p.n_pages + 31) / 32;
  const int per = (words + kScanThreads - 1) / kScanThreads;
  const int w0 = threadIdx.x * per, w1 = w0 + per < words ? w0 + per : words;
  int mine = 0;
  for (int w = w0; w < w1; ++w) mine += __popc(~p.bits[w] & valid_bits(p, w));
  int total;
  int rank = scan_block(mine, red, total);
  for (int w = w0; w < w1 && rank < limit; ++w) {
    uint32_t f = ~p.bits[w] & valid_bits(p, w);
    while (f && rank < limit) {
      p.spare[rank++] = w * 32 + __ffs(f) - 1;
      f &= f - 1;
    }
  }
  __syncthreads();  // the list is complete for this workgroup
  return total;
}

__device__ __forceinline__ void fork_assign(const PagesParams& p, int* red) {
  const int t = threadIdx.x;
  // wishes are 0 or 1; of the rows of the first round (mostly all) the rank is kept
  const bool first = t < p.rows && p.need[t];
  int wanted;
  const int first_rank = scan_block((int)first, red, wanted);
  const int first_total = wanted;
  for (int r0 = kScanThreads; r0 < p.rows; r0 += kScanThreads) {
    int total;
    (void)scan_block(r0 + t < p.rows ? p.need[r0 + t] : 0, red, total);
    wanted += total;
  }
  const int free_pages = list_free(p, wanted, red);
  int base = 0;
  for (int r0 = 0; r0 < p.rows; r0 += kScanThreads) {
    const int r = r0 + t;
    int need = first, rank = first_rank, total = first_total;
    if (r0 > 0) {
      need = r < p.rows ? p.need[r] : 0;
      rank = base + scan_block(need, red, total);
    }
    base += total;
    if (need) {
      const int tokens = p.tokens[r];
      int32_t* out = p.table_out + (int64_t)r * p.width + entries(p, tokens) - 1;
      if (rank < free_pages) {
        const int32_t id = p.spare[rank];
        p.src[rank] = p.last[r];
        p.dst[rank] = id;
        if (p.writes) *out = id;
        if (p.refs) p.refs[id] = 1;
      } else if (p.writes) {
        *out = -1;
        p.lens_out[r] = tokens / p.page_size * p.page_size;
      }
    }
  }
  if (t == 0) {
    const int kept = wanted < free_pages ? wanted : free_pages;
    *p.pairs = kept;
    *p.result = wanted - kept;
  }
}

__device__ __forceinline__ void grow_assign(const PagesParams& p, int* red) {
  __shared__ int64_t red64[kScanThreads / kWave];  // wishes add up past 32 bits
  const int t = threadIdx.x, lane = t & 63;
  auto wish = [&](int r) -> int64_t { return r < p.rows && p.need[r] > 0 ? p.need[r] : 0; };
  int64_t wanted;
  const int64_t first_rank = scan_block(wish(t), red64, wanted);
  const int64_t first_total = wanted;
  for (int r0 = kScanThreads; r0 < p.rows; r0 += kScanThreads) {
    int64_t total;
    (void)scan_block(wish(r0 + t), red64, total);
    wanted += total;
  }
  const int free_pages = list_free(p, wanted < p.n_pages ? (int)wanted : p.n_pages, red);
  int64_t base = 0;  // pages wanted by the rows before this round
  int refused = 0;
  for (int r0 = 0; r0 < p.rows; r0 += kScanThreads) {
    const int r = r0 + t;
    const int64_t need = wish(r);
    int64_t rank = first_rank, total = first_total;
    if (r0 > 0) rank = base + scan_block(need, red64, total);
    base += total;
    const bool ok = r < p.rows && p.need[r] >= 0 && (need == 0 || rank + need <= free_pages);
    int held = 0;
    if (r < p.rows) {
      const int tokens = tokens_of(p, r);
      held = entries(p, tokens);
      p.lens_out[r] = ok ? tokens + (p.add[r] > 0 ? p.add[r] : 0) : tokens;
      refused += !ok;
    }
    // a row's page by its own thread, the pages of a row that wants more by its wave
    const int cnt = ok ? (int)need : 0;
    if (cnt == 1) p.table_out[(int64_t)r * p.width + held] = p.spare[rank];
    for (uint64_t many = __ballot(cnt > 1); many; many &= many - 1) {
      const int k = __builtin_ctzll(many);
      const int n = __shfl(cnt, k, kWave), from = __shfl((int)rank, k, kWave);
      int32_t* out = p.table_out + (int64_t)(r0 + (t & ~63) + k) * p.width + __shfl(held, k, kWave);
      for (int i = lane; i < n; i += kWave) out[i] = p.spare[from + i];
    }
  }
  int total;
  (void)scan_block(refused, red, total);
  if (t == 0) *p.result = total;
}

__device__ __forceinline__ void compact_assign(const PagesParams& p, int* red) {
  const int words = (p.n_pages + 31) / 32;
  const int per = (words + kScanThreads - 1) / kScanThreads;
  const int w0 = threadIdx.x * per, w1 = w0 + per < words ? w0 + per : words;
  int mine = 0, used;
  for (int w = w0; w < w1; ++w) mine += __popc(p.bits[w]);
  (void)scan_block(mine, red, used);
  // bits at or above `used`, and free bits below it
  auto above = [&](int w) {
    const int left = used - w * 32;
    return left <= 0 ? p.bits[w] : left >= 32 ? 0u : p.bits[w] & ~((1u << left) - 1);
  };
  auto below = [&](int w) {
    const int left = used - w * 32;
    return left <= 0 ? 0u : left >= 32 ? ~p.bits[w] : ~p.bits[w] & ((1u << left) - 1);
  };
  int na = 0, nb = 0, moves, holes;
  for (int w = w0; w < w1; ++w) {
    na += __popc(above(w));
    nb += __popc(below(w));
  }
  int ra = scan_block(na, red, moves);
  int rb = scan_block(nb, red, holes);  // holes == moves
  for (int w = w0; w < w1; ++w) {
    for (uint32_t f = above(w); f; f &= f - 1) p.src[ra++] = w * 32 + __ffs(f) - 1;
    for (uint32_t f = below(w); f; f &= f - 1) p.dst[rb++] = w * 32 + __ffs(f) - 1;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < moves; i += kScanThreads) p.map[p.src[i]] = p.dst[i];
  if (threadIdx.x == 0) {
    *p.pairs = moves;
    *p.result = used;
  }
}

template <int OP>
__device__ __forceinline__ void assign(const PagesParams& p, int* red) {
  if constexpr (OP == kFork) fork_assign(p, red);
  if constexpr (OP == kGrow) grow_assign(p, red);
  if constexpr (OP == kCompact) compact_assign(p, red);
}

template <int OP>
__global__ __launch_bounds__(kScanThreads) void pages_assign_kernel(PagesParams p) {
  __shared__ int red[kScanThreads / kWave];
  assign<OP>(p, red);
}

// Bytes that a workgroup of T threads copies at a time, and such pieces of a page.
template <int T>
__host__ __device__ __forceinline__ int64_t pieces_of(int64_t page_bytes) {
  return (page_bytes + T * 64 - 1) / (T * 64);
}

// This workgroup's share of pairs x planes x pieces of a page, one in `blocks`.
// I: an unsigned type that holds their number; 64-bit divisions take longer than
// copying a piece.
template <int T, class I>
__device__ __forceinline__ void copy_share(const PagesParams& p, I pairs, I pieces, I first,
                                           I blocks) {
  const I planes = (I)p.planes, total = pairs * planes * pieces;
  for (I i = first; i < total; i += blocks) {
    const I rest = i / pieces, piece = i - rest * pieces;
    const I pair = rest / planes, plane = rest - pair * planes;
    const int32_t s = p.src[pair], d = p.dst[pair];
    if (!names_page(p, s) || !names_page(p, d)) continue;
    const unsigned char* from = p.pool + ((int64_t)plane * p.n_pages + s) * p.page_bytes;
    unsigned char* to = p.pool + ((int64_t)plane * p.n_pages + d) * p.page_bytes;
    const int64_t at = (int64_t)piece * (T * 64) + threadIdx.x * 16;
    u32x4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (at + k * T * 16 < p.page_bytes)
        v[k] = *reinterpret_cast<const u32x4*>(from + at + k * T * 16);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (at + k * T * 16 < p.page_bytes)
        *reinterpret_cast<u32x4*>(to + at + k * T * 16) = v[k];
  }
}

template <int T>
__device__ __forceinline__ void copy_turns(const PagesParams& p, int64_t pairs, uint32_t first,
                                           uint32_t blocks) {
  const int64_t pieces = pieces_of<T>(p.page_bytes);
  if (pairs * p.planes * pieces < INT32_MAX - (int64_t)blocks)
    copy_share<T, uint32_t>(p, (uint32_t)pairs, (uint32_t)pieces, first, blocks);
  else
    copy_share<T, uint64_t>(p, pairs, pieces, first, blocks);
}

// Row r of the table after compaction, by the threads of a workgroup.
__device__ __forceinline__ void retable_row(const PagesParams& p, int r, int held, int used,
                                            int thread, int threads) {
  const int64_t row = (int64_t)r * p.width;
  for (int i = thread; i < p.width; i += threads) {
    int32_t id = i < held ? p.table[row + i] : -1;
    if (names_page(p, id) && id >= used) id = p.map[id];
    p.table_out[row + i] = id;
  }
}

// All of the bookkeeping in one workgroup, with the bitmap and the rows' wishes in
// LDS: one launch instead of three, for states that one compute unit walks
// through in a few microseconds.  INSIDE (fork, compact): every workgroup does it
// for itself, the first writes the results and the others copy the pages, so that
// nothing else has to be launched.
constexpr int kOneRows = 256;
// Forking counts the holders of every page in LDS too (atomics on memory from one
// compute unit take 1.5 ns each: 256 x 128 entries 65 us).
template <int OP, bool INSIDE>
constexpr int one_pages() {
  return OP == kFork ? 8 * 1024 : INSIDE ? 4 * 1024 : 64 * 1024;
}

template <int OP, bool INSIDE>
__global__ __launch_bounds__(kScanThreads) void pages_one_kernel(PagesParams p) {
  constexpr int kPages = one_pages<OP, INSIDE>();
  constexpr int kPairs = !INSIDE ? 1 : OP == kFork ? kOneRows : kPages / 2;
  __shared__ int red[kScanThreads / kWave];
  __shared__ uint32_t sBits[kPages / 32];
  __shared__ int32_t sRefs[OP == kFork ? kPages : 1];
  __shared__ int sFrom[kOneRows], sHeld[kOneRows], sNeed[kOneRows], sLast[kOneRows];
  __shared__ int sSpare[kOneRows], sTokens[kOneRows];
  __shared__ int32_t sSrc[kPairs], sDst[kPairs], sMap[INSIDE && OP == kCompact ? kPages : 1];
  __shared__ int32_t sPairs, sResult;
  const int t = threadIdx.x;
  int32_t *const refs_out = p.refs, *const result_out = p.result;
  p.writes = !INSIDE || blockIdx.x == 0;
  p.bits = sBits;
  p.need = sNeed;
  p.last = sLast;
  p.tokens = sTokens;
  if (OP == kFork) p.spare = sSpare;  // a page a row at most
  if constexpr (INSIDE) {
    p.src = sSrc;
    p.dst = sDst;
    p.map = sMap;
    p.pairs = &sPairs;
    p.result = &sResult;
  }
  for (int i = t; i < (p.n_pages + 31) / 32; i += kScanThreads) sBits[i] = 0;
  if constexpr (OP == kFork) {
    for (int i = t; i < p.n_pages; i += kScanThreads) sRefs[i] = 0;
    p.refs = sRefs;
  }
  if (t < p.rows) {
    int from = t;
    if constexpr (OP == kFork) {
      from = p.parent[t];
      if ((uint32_t)from >= (uint32_t)p.rows_in) from = -1;
    }
    const int tokens = from < 0 ? 0 : tokens_of(p, from);
    sFrom[t] = from;
    sHeld[t] = entries(p, tokens);
    sNeed[t] = OP == kFork && from >= 0 && tokens % p.page_size != 0;  // may want a copy
    sTokens[t] = tokens;
    if (OP == kFork && p.writes) p.lens_out[t] = tokens;
    if constexpr (OP == kGrow) sNeed[t] = wanted_pages(p, t, tokens);
  }
  __syncthreads();
  // a wave takes every 16th row, the first entries of four rows at a time
  constexpr int kWaves = kScanThreads / kWave, kAtOnce = 4;
  const int lane = t & 63;
  for (int r0 = t >> 6; r0 < p.rows; r0 += kWaves * kAtOnce) {
    int32_t head[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int r = r0 + u * kWaves;
      const int held = r < p.rows ? sHeld[r] : 0;
      head[u] = lane < held ? p.table[(int64_t)sFrom[r] * p.width + lane] : -1;
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int r = r0 + u * kWaves;
      if (r >= p.rows) break;
      const int held = sHeld[r];
      bool wants = false;  // a copy of the last page: an earlier row continues the same one
      if (OP == kFork && sNeed[r]) {
        const int from = sFrom[r];
        int later = 0;
        for (int i = lane; i < r; i += kWave) later |= sFrom[i] == from;
        wants = __any(later);
        if (lane == 0) sNeed[r] = wants;
      }
      const int end = OP == kCompact || !p.writes ? held : p.width;
      for (int j = lane; j < end; j += kWave) {
        int32_t id = j < kWave ? head[u] : j < held ? p.table[(int64_t)sFrom[r] * p.width + j] : -1;
        if (j < held) {
          const bool names = names_page(p, id);
          if (wants && j == held - 1) {
            sLast[r] = id;
            if (!names) sNeed[r] = 0;
          } else if (names) {
            atomicOr(&sBits[id >> 5], 1u << (id & 31));
            if constexpr (OP == kFork) atomicAdd(&sRefs[id], 1);
          }
        }
        if (OP != kCompact && p.writes) p.table_out[(int64_t)r * p.width + j] = id;
      }
    }
  }
  __syncthreads();
  assign<OP>(p, red);
  __syncthreads();
  if (OP == kFork && p.writes && refs_out)
    for (int i = t; i < p.n_pages; i += kScanThreads) refs_out[i] = sRefs[i];
  if constexpr (INSIDE) {
    if (blockIdx.x > 0) {
      copy_turns<kScanThreads>(p, sPairs, blockIdx.x - 1, gridDim.x - 1);
      return;
    }
    if (t == 0) *result_out = sResult;
    if constexpr (OP == kCompact)
      for (int r = t >> 6; r < p.rows; r += kWaves)
        retable_row(p, r, sHeld[r], sResult, lane, kWave);
  }
}

// The copies, taken in turn by all but the first `table_blocks` workgroups; those
// rewrite the table's rows after compaction.
__global__ __launch_bounds__(kPagesThreads) void pages_move_kernel(PagesParams p, int64_t n,
                                                                   int table_blocks) {
  if ((int)blockIdx.x < table_blocks) {
    const int used = *p.result;
    for (int r = blockIdx.x; r < p.rows; r += table_blocks)
      retable_row(p, r, entries(p, tokens_of(p, r)), used, threadIdx.x, kPagesThreads);
    return;
  }
  copy_turns<kPagesThreads>(p, p.pairs ? (int64_t)*p.pairs : n, blockIdx.x - table_blocks,
                            gridDim.x - table_blocks);
}

int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

PagesParams params(const PagesArgs& a) {
  PagesParams p{};
  p.pool = a.pool;
  p.planes = a.planes;
  p.page_bytes = a.page_bytes;
  p.n_pages = (int32_t)a.n_pages;
  p.page_size = (int32_t)a.page_size;
  p.rows_in = (int32_t)a.rows_in;
  p.rows = (int32_t)a.rows;
  p.width = (int32_t)a.width;
  p.table = a.table;
  p.lens = a.lens;
  p.parent = a.parent;
  p.add = a.add;
  p.table_out = a.table_out;
  p.lens_out = a.lens_out;
  p.tokens = a.lens_out;
  p.refs = a.refs;
  p.result = a.result;
  unsigned char* w = static_cast<unsigned char*>(a.workspace);
  auto take = [&](int64_t count) {
    unsigned char* q = w;
    w += up16(4 * count);
    return q;
  };
  p.bits = reinterpret_cast<uint32_t*>(take((a.n_pages + 31) / 32));
  p.need = reinterpret_cast<int32_t*>(take(a.rows));
  p.last = reinterpret_cast<int32_t*>(take(a.rows));
  p.src = reinterpret_cast<int32_t*>(take(a.n_pages));
  p.dst = reinterpret_cast<int32_t*>(take(a.n_pages));
  p.spare = reinterpret_cast<int32_t*>(take(a.n_pages));
  p.map = reinterpret_cast<int32_t*>(take(a.n_pages));
  p.pairs = reinterpret_cast<int32_t*>(take(1));
  p.writes = true;
  return p;
}

// The copies, at most `most` of them, and the new table where `retable` is set.
hipError_t move(const PagesParams& p, int64_t most, bool retable, hipStream_t s) {
  const int64_t grid = 8 * device_cus();
  const int64_t items =
      most > grid && p.planes ? grid : most * p.planes * pieces_of<kPagesThreads>(p.page_bytes);
  const int table_blocks = !retable ? 0 : p.rows < 256 ? p.rows : 256;
  const int64_t blocks = table_blocks + (items < grid ? items : grid);
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL(pages_move_kernel, dim3((uint32_t)blocks), dim3(kPagesThreads), 0, s, p, most,
                     table_blocks);
  return hipGetLastError();
}

}  // namespace

int64_t pages_workspace_bytes(int64_t rows, int64_t n_pages) {
  return up16(4 * ((n_pages + 31) / 32)) + 2 * up16(4 * rows) + 4 * up16(4 * n_pages) + 16;
}

namespace {

// The bookkeeping of one operator: in one workgroup where the state is small.
// Measured (us on the GPU, one workgroup / separate launches), rows x width: fork
// 4 x 10 5.9 / 8.9, 64 x 43 7.4 / 13.2, 48 x 884 11.5 / 10.2, 256 x 128 19 / 25; grow
// 64 x 43 5.9 / 12.5, 256 x 256 21 / 16; compaction 4 x 10 7.9 / 10.4, 48 x 884
// 9.1 / 12.5, 256 x 256 19.2 / 17.9.  Each further launch costs the caller some 2 us.
constexpr int64_t kOneEntries = 48 * 1024;

template <int OP>
hipError_t launch_state(const PagesParams& p, hipStream_t s) {
  if (p.rows <= kOneRows && (int64_t)p.rows * p.width <= kOneEntries &&
      p.n_pages <= one_pages<OP, false>()) {
    hipLaunchKernelGGL((pages_one_kernel<OP, false>), dim3(1), dim3(kScanThreads), 0, s, p);
    return hipGetLastError();
  }
  const int64_t blocks = (p.n_pages + kPagesThreads - 1) / kPagesThreads;
  hipLaunchKernelGGL(pages_clear_kernel, dim3((uint32_t)(blocks < 1024 ? blocks : 1024)),
                     dim3(kPagesThreads), 0, s, p);
  if (p.rows > 0)
    hipLaunchKernelGGL(pages_rows_kernel<OP>, dim3(p.rows), dim3(kPagesThreads), 0, s, p);
  hipLaunchKernelGGL(pages_assign_kernel<OP>, dim3(1), dim3(kScanThreads), 0, s, p);
  return hipGetLastError();
}

// Bookkeeping and copies (`most` of them at most): in one launch where both are
// small, because every workgroup then does the bookkeeping.  Measured (us on the GPU,
// one launch / two; rows x width, planes): fork 4 x 10, 8 6.0 / 7.3, 64 x 128, 2 8.4 /
// 10.4, 32 x 16, 16 8.9 / 9.8; compaction 3 x 64, 4 7.6 / 8.5, 64 x 43, 8 23.6 / 24.4.
// Beyond the limits the bookkeeping of many workgroups gets in its own way: fork 64
// x 43, 32 23 / 18, 256 x 32, 2 40 / 18.
constexpr int64_t kInsideRows = 64, kInsideEntries = 8 * 1024, kInsideItems = 512;
constexpr int64_t kInsideBlocks = 128;

template <int OP>
hipError_t launch_pages(const PagesParams& p, int64_t most, hipStream_t s) {
  const int64_t pieces = pieces_of<kScanThreads>(p.page_bytes);
  if (p.rows <= kInsideRows && (int64_t)p.rows * p.width <= kInsideEntries &&
      p.n_pages <= one_pages<OP, true>() && most * p.planes * pieces <= kInsideItems) {
    const int64_t items = most * p.planes * pieces;
    hipLaunchKernelGGL((pages_one_kernel<OP, true>),
                       dim3((uint32_t)(1 + (items < kInsideBlocks ? items : kInsideBlocks))),
                       dim3(kScanThreads), 0, s, p);
    return hipGetLastError();
  }
  const hipError_t e = launch_state<OP>(p, s);
  return e != hipSuccess ? e : move(p, most, OP == kCompact, s);
}

}  // namespace

hipError_t launch_pages_fork(const PagesArgs& a, hipStream_t s) {
  return launch_pages<kFork>(params(a), a.rows < a.n_pages ? a.rows : a.n_pages, s);
}

hipError_t launch_pages_grow(const PagesArgs& a, hipStream_t s) {
  return launch_state<kGrow>(params(a), s);
}

hipError_t launch_pages_compact(const PagesArgs& a, hipStream_t s) {
  return launch_pages<kCompact>(params(a), a.n_pages / 2, s);
}

hipError_t launch_pages_copy(unsigned char* pool, int64_t planes, int64_t n_pages,
                             int64_t page_bytes, const int32_t* src, const int32_t* dst, int64_t n,
                             hipStream_t s) {
  PagesParams p{};
  p.pool = pool;
  p.planes = planes;
  p.n_pages = (int32_t)n_pages;
  p.page_bytes = page_bytes;
  p.src = const_cast<int32_t*>(src);  // read only
  p.dst = const_cast<int32_t*>(dst);
  return move(p, n, false, s);
}

}  // namespace tq
