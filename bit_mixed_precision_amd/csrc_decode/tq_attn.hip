// Attention of one new token per sequence over a paged key-value cache.
//
//     out[b][h] = sum_t softmax_t(scale * q[b][h] . k[t][h / G]) v[t][h / G]
//
// over the tokens t in [max(0, len - window), len) of sequence b, G = Hq / Hkv
// query heads sharing a key-value head; a row without tokens gives zeros and
// lse = -inf.  One pass over the cache with a running maximum and sum in fp32
// (base-2 exponents: the scale carries log2 e).
//
// Bound: reading K and V once from HBM; 2 * len * Hkv * D elements against
// 4 * len * Hq * D flops, i.e. at most 32 flops per byte at G = 16.
//
// MI355X design.  The unit of work is a tile of 32 tokens of one (sequence,
// key-value head), processed by one wave with no barrier:
//  * S^T = K Q^T by v_mfma_f32_16x16x32 with K as the A operand and up to 16
//    query heads as the columns; the matrix cores idle over 90% of the time even
//    so, which is why one kernel serves every G.
//  * K and V are loaded as whole rows (256 bytes by 16 lanes at D = 128).  A wave
//    turns half a tile of K into operand order in 4 KB of LDS (pieces XOR-swizzled:
//    no bank conflicts by the counters); loading K in operand order instead,
//    64 bytes of 16 rows at a time, costs 4-7%.
//  * The scores arrive with lane = head and 4 tokens of each half per lane,
//    which is the B operand order of the second product when V's tokens are
//    taken in the same order: lane group g contributes tokens 4 g .. 4 g + 3 of
//    both halves.  P never leaves its registers.
//  * O^T += V^T P^T: lane (li, g) holds 8 consecutive numbers (4 for D <= 64) of
//    its 8 tokens and turns them into A operands (8 tokens of one number) with 4
//    v_perm_b32 each.  O^T keeps lane = head, so rescaling and the final division
//    need no exchange.
//  * P enters the product as two 16-bit numbers, cut and remainder, the latter
//    rounded to nearest (to within 2^-22 of a weight in fp16, 2^-16 in bf16: one
//    number, 2^-12 and 2^-9, would add as much error as the output's own rounding; a
//    third would cost another product); fp16 exponents are shifted by 14 so that
//    weights down to 2^-28 of the largest keep all their bits.
//  * The next tile's K is loaded after this tile's scores, its V after this tile's
//    sums, also across the end of a row: the registers of one tile and the loads of
//    the next are the same, and a CU keeps some 100 KB in flight.
//  * Loads are buffer loads whose lane offset is pushed out of range where a
//    token is masked or a head ends, so what lies in unused places (NaN
//    included) reads as zero and no branch is needed.  Page sizes that are no
//    multiple of 16 find every token's address by itself.
//
// Work is split over the flattened list of (sequence, head, tile): every wave
// takes an equal contiguous run, computed on the device from the lengths, so one
// long sequence, or many ragged ones, fill the GPU alike and the host needs no
// lengths.  Rows that begin and end in a wave are written by it; what is left of
// the others, two parts a wave at most, joins in LDS at the end of the workgroup,
// and a row that spans workgroups leaves its sums in the workspace for the joining
// kernel (no atomics: the same bits on every run).  Where every row is short (by the
// table's width or the window) and they are not too many, each has a workgroup of
// its own instead and one launch does.
//
// Measured: 96 sequences of 2048 .. 8192 tokens, 64 query / 8 key-value heads of
// 128, pages of 16, 1.75 GB: 274 us, 6.4 TB/s (92% of what a plain read reaches on
// this card, 6.97 TB/s; HBM reads by the counters 1.00 of the algorithmic bytes);
// one sequence of 131072 tokens, 537 MB: 90 us, of which the join takes 5; 37
// ragged sequences of up to 4096 tokens, 24 heads of 64 in bf16, 116 MB: 31 us (25 in
// the first kernel, whose start and end weigh more); one of 97 tokens: 6.2 us, four
// dependent memory latencies and the launch.

#include <atomic>
#include <type_traits>

#include "tq.h"
#include "tq_attn_dev.h"
#include "tq_attn_slots.h"
#include "tq_common.h"
#include "tq_decode.h"
#include "tq_kernels.h"
#include "tq_mfma.h"

namespace tq {
namespace {

constexpr int kAttnThreads = kAttnWaves * kWave;
constexpr int kTileTokens = 32;
constexpr int kHeads = 16;                // query heads per workgroup
struct AttnParams {
  const unsigned char* Q;
  const unsigned char* K;
  const unsigned char* V;
  int64_t q_tok, q_head;                          // bytes
  int64_t page_stride, row_stride, head_stride;   // bytes
  const int32_t* table;
  const int32_t* lens;
  unsigned char* Out;
  float* lse;
  float* partial;  // [workgroups][2][slot_floats]
  int2* owner;     // [workgroups]: the row it began and left unfinished (or -1), its last workgroup
  FastDiv page;
  int32_t n_pages, width, B, Hq, Hkv, D, G, qtiles, window;
  int32_t direct;  // one workgroup per (sequence, head): nothing is split
  int32_t full;    // tiles of 16 KB or more in whole lines and pages of whole half tiles,
                   // two workgroups per CU
  float scale;
};

// Floats of one partial sum: heads x D numbers, maxima, sums.
__host__ __device__ __forceinline__ int64_t slot_floats(int heads, int D) {
  return heads * D + (2 * heads + 3) / 4 * 4;
}

template <bool BF>
__device__ __forceinline__ float4v mma(u32x4 a, u32x4 b, float4v c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a),
                                                   __builtin_bit_cast(bf8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a),
                                                  __builtin_bit_cast(half8, b), c, 0, 0, 0);
}


// NT: non-temporal, for lines that one wave reads once.  Measured (us, with /
// without): 96 sequences of 2048 .. 8192 tokens, 8 key heads of 128: 286 / 323;
// heads of 80, whose rows share 128-byte lines: 150 / 130; 64 query heads on one
// key head, read by four groups of heads: 45 / 41.
constexpr int kNonTemporal = 2;
template <bool NT>
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(
      u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, NT ? kNonTemporal : 0));
}
template <bool NT>
__device__ __forceinline__ u32x2 load8(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(
      u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, NT ? kNonTemporal : 0));
}
template <bool NT, class T>
__device__ __forceinline__ T load_at(const unsigned char* p) {
  if constexpr (NT)
    return __builtin_nontemporal_load(reinterpret_cast<const T*>(p));
  else
    return *reinterpret_cast<const T*>(p);
}

// Largest of the four lanes (li, g = 0..3) that hold one head.
__device__ __forceinline__ float max_over_groups(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, kWave));
  return fmaxf(v, __shfl_xor(v, 32, kWave));
}
__device__ __forceinline__ float sum_over_groups(float v) {
  v += __shfl_xor(v, 16, kWave);
  return v + __shfl_xor(v, 32, kWave);
}

// Tokens [lo, hi) of sequence b, clamped to what its table row can name, and
// the tiles [t0, t1) that hold them.
struct Range {
  int lo, hi, t0, t1;
};
__device__ __forceinline__ Range range_of_len(const AttnParams& p, int len) {
  const int cap = p.width * (int)p.page.d;
  const int n = len < 0 ? 0 : len;
  const int hi = n < cap ? n : cap;
  const int from = p.window > 0 && n > p.window ? n - p.window : 0;
  const int lo = from < hi ? from : hi;
  const int t0 = lo / kTileTokens;
  return {lo, hi, t0, lo < hi ? (hi + kTileTokens - 1) / kTileTokens : t0};
}
__device__ __forceinline__ Range range_of(const AttnParams& p, int b) {
  return range_of_len(p, read_const(p.lens, b));
}
// Tiles of sequence b, 0 where it is left out; the read does not wait for `in`.
__device__ __forceinline__ uint32_t tiles_of(const AttnParams& p, int b, bool in) {
  const Range r = range_of(p, b < p.B ? b : p.B - 1);
  return in && b < p.B ? r.t1 - r.t0 : 0;
}

// Sequences a lane, up to which a wave walks through them one by one.  Measured
// (us, walking / 64 at a time): 256 sequences of up to 32 tokens (4 a lane), 8 key
// heads of 128: 10.0 / 10.4, 4096 of one key head (64 a lane) 35.7 / 28.8.
constexpr int kFewLengths = 8;

// Every wave by itself: the number of tiles of all sequences, and those before
// this lane's; lane i looks after the sequences [i * per, (i + 1) * per).
__device__ __forceinline__ uint32_t scan_tiles(const AttnParams& p, int lane, int per,
                                               uint32_t& mine, uint32_t& total) {
  mine = tiles_of(p, lane * per, true);
  for (int i = 1; i < per; i += 8) {  // eight lengths at a time are under way
    uint32_t n[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) n[u] = tiles_of(p, lane * per + i + u, i + u < per);
#pragma unroll
    for (int u = 0; u < 8; ++u) mine += n[u];
  }
  const uint32_t inc = scan_wave(mine, lane);
  total = uni((int)__shfl(inc, 63, kWave));
  return inc - mine;
}

// A tile of the flattened list: head h (key-value head and group of 16 query
// heads) of sequence b, and the tile's place in its row.
struct Cursor {
  int b, h, tile;
  Range r;
};

// ln of the sum of exponentials, from the base-2 maximum and the scaled sum.
template <bool BF>
__device__ __forceinline__ float lse_of(float m, float sum) {
  return (m + __builtin_amdgcn_logf(sum) - (BF ? 0.f : 14.f)) / kLog2e;
}

// Divides by the sum and writes numbers d .. d + 7 of one head, and its lse.
template <bool BF>
__device__ __forceinline__ void finish(const AttnParams& p, int b, int head, int d, float m,
                                       float sum, const float* v) {
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  u32x4 u;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    u[e] = to16<BF>(v[2 * e] * inv) | ((uint32_t)to16<BF>(v[2 * e + 1] * inv) << 16);
  const int64_t at = (int64_t)b * p.Hq + head;
  *reinterpret_cast<u32x4*>(p.Out + (at * p.D + d) * 2) = u;
  if (p.lse && d == 0) p.lse[at] = lse_of<BF>(m, sum);
}

// Workgroups per CU, for which the registers are laid out: enough bytes in flight,
// and more only spill or crowd.  Measured (us): heads of 128, 96 sequences of 2048
// .. 8192 tokens, 8 key heads: 2 274, 3 314; heads of 64, 64 sequences of 1024 .. 4096,
// 24 key heads: 2 167, 3 173 (but 8 of 32768, 8 key heads: 104, 98); heads of 256, 8
// sequences of 32768, 2 key heads: 1 98, 2 124.
__host__ __device__ constexpr int blocks_per_cu(int64_t D) { return D > 128 ? 1 : 2; }

// Waves that share the tiles, of those that run: half of them, one workgroup per
// CU, where each has many tiles that are fetched without a detour (p.full: 16 KB a
// tile in whole lines, pages of whole half tiles), which keeps 64 KB of a CU in flight
// as it is.  Measured (us, half / all): one sequence of 131072 tokens, 8 key heads of
// 128: 93 / 102, 96 sequences of 2048 .. 8192: 285 / 294, 8 of 32768: 176 / 187 (but 64 of
// 4096, 24 key heads: 492 / 481); with fewer tiles a wave the other way round: 32
// sequences of up to 1024 tokens, if split (2.5 a wave) 26.2 / 24.4, 128 (10) 65.3 / 63.8;
// pages of 24 108 / 98.  Smaller heads keep less in flight, and those of 72 .. 120 share
// lines: the same 131072 tokens, heads of 64 75 / 54, 80 89 / 72, 96 93 / 84, 104 96 / 91,
// 112 98 / 103, 120 101 / 105; 32 sequences of 8192, 2 key heads of 80 84 / 62, 96 83 / 70,
// 104 104 / 74, 112 104 / 79, 120 113 / 84, 128 84 / 84; the 96 sequences, heads of 64 208 /
// 144, 80 280 / 276, 96 286 / 300, 104 352 / 376, 112 367 / 384, 120 399 / 411.
constexpr uint32_t kManyTiles = 12;
__device__ __forceinline__ uint32_t waves_for(const AttnParams& p, uint32_t units, uint32_t waves) {
  return p.full && units / kManyTiles >= waves ? waves / 2 : waves;
}

// DV: 64, 128 or 256, the head dimension rounded up (D <= DV, D % 8 == 0).
// UNI: the page size is a multiple of 16, so a half tile lies in one page and
// its base address is uniform.
// DIRECT: one workgroup per (sequence, head): nothing is split.  A wave then has part
// of one row, and its loads wait for no more than what they need: the next tile's
// are issued also where there is none (out of range), so that no branch makes the
// compiler wait for all.  Measured against one kernel for both forms (us): 8 key heads
// of 128, 4 sequences of 512 tokens 9.6 / 11.0, 32 of up to 256 7.3 / 8.0, 64 of up to
// 128 8.3 / 8.5; of 64, 64 of up to 512 10.9 / 12.6; of 256, 64 of up to 256 25.9 / 28.7.
template <bool BF, int DV, bool UNI, bool NT, bool DIRECT>
__global__ __launch_bounds__(kAttnThreads, blocks_per_cu(DV)) void paged_attention_kernel(
    AttnParams p) {
  constexpr int KS = DV / 32;             // MFMA steps of a score
  constexpr int NE = DV / 16;             // V operands (numbers per lane)
  constexpr int NV = DV == 256 ? 2 : 1;   // pieces of a head: LN numbers per lane each
  constexpr int LN = DV == 64 ? 4 : 8;
  constexpr int PW = LN * 16;             // numbers of a piece
  constexpr int KC = DV / 8;              // 16-byte pieces of a key
  constexpr int KR = kWave / KC;          // keys that one load covers
  // Keys are loaded as whole rows, like values, and turned in LDS; heads of more
  // than 128 numbers are loaded in operand order instead (64 bytes of 16 rows).
  constexpr bool LDSK = DV <= 128;
  // partial sums of this workgroup's waves: [wave][first, last][heads][D + 4], or,
  // direct, [wave][heads][D + 4]
  extern __shared__ __attribute__((aligned(16))) float sO[];
  // half a tile of keys on its way from load order to operand order, per wave
  __shared__ u32x4 sK[LDSK ? kAttnWaves * 16 * KC : 1];
  __shared__ float sM[kAttnSlots][kHeads], sL[kAttnSlots][kHeads];
  __shared__ int sRow[kAttnSlots], sEnds[kAttnSlots], sLast[kAttnSlots];

  const int tid = threadIdx.x;
  const int wave = uni(tid >> 6);
  const int lane = tid & 63, li = lane & 15, g = lane >> 4;
  const int H = p.Hkv * p.qtiles;
  const int slot_heads = p.G < kHeads ? p.G : kHeads;
  const int row_floats = p.D + 4;

  // this wave's run of tiles
  uint32_t left, run_end = 0;  // run_end: the unit after the run
  Cursor cur;
  Cut cut(0, 1);
  if constexpr (DIRECT) {
    cur.b = blockIdx.x / H;
    cur.h = blockIdx.x % H;
    cur.r = range_of(p, cur.b);
    const int n = cur.r.t1 - cur.r.t0;
    cur.tile = cur.r.t0 + n * wave / kAttnWaves;
    left = cur.r.t0 + n * (wave + 1) / kAttnWaves - cur.tile;
  } else {
    const int per = (p.B + kWave - 1) / kWave;
    uint32_t mine, total;
    const uint32_t before = scan_tiles(p, lane, per, mine, total);
    cut = Cut(total * H, waves_for(p, total * H, gridDim.x * kAttnWaves));
    const uint32_t part = blockIdx.x * kAttnWaves + wave;
    left = 0;
    if (part < cut.parts) {
      const uint32_t at = cut.start(part);
      run_end = cut.start(part + 1);
      left = run_end - at;
      const uint64_t has = __ballot(before * H <= at && at < (before + mine) * H);
      const int src = __builtin_ctzll(has);
      uint32_t in_row = at - (uint32_t)__builtin_amdgcn_readlane((int)before, src) * H;
      cur.b = src * per;
      // which of that lane's sequences: one by one, or, of many, 64 at a time
      for (int i = 0; per > kFewLengths && i < per; i += kWave) {
        const uint32_t n = tiles_of(p, src * per + i + lane, i + lane < per);
        const uint32_t inc = scan_wave(n, lane);
        const uint64_t hit = __ballot(in_row < inc * H);
        if (hit) {
          const int k = __builtin_ctzll(hit);
          cur.b = src * per + i + k;
          in_row -= (uint32_t)__builtin_amdgcn_readlane((int)(inc - n), k) * H;
          break;
        }
        in_row -= (uint32_t)__builtin_amdgcn_readlane((int)inc, kWave - 1) * H;
      }
      cur.r = range_of(p, cur.b);
      uint32_t n;
      // (the bounds on b hold whatever happens to the lengths meanwhile)
      while (in_row >= (n = (uint32_t)(cur.r.t1 - cur.r.t0)) * H && cur.b + 1 < p.B) {
        in_row -= n * H;
        cur.r = range_of(p, ++cur.b);
      }
      n = n > 0 ? n : 1;
      cur.h = in_row / n;
      cur.tile = cur.r.t0 + in_row % n;
    }
  }
  // its own slots are empty (written by the lane that fills them later: there is no
  // barrier in between)
  if (lane == 0)
#pragma unroll
    for (int part = 0; part < kAttnParts; ++part) sRow[attn_slot(wave, part)] = -1;

  auto advance = [&](Cursor& c) {  // only where another tile follows
    if (++c.tile < c.r.t1 || DIRECT) return;
    if (++c.h == H) {
      c.h = 0;
      while (c.b + 1 < p.B) {
        c.r = range_of(p, ++c.b);
        if (c.r.t1 > c.r.t0) break;
      }
    }
    c.tile = c.r.t0;
  };

  u32x4 kreg[2][KS];
  u32x4 vreg[8][NV];  // DV == 64 uses the first two dwords of each
  const uint32_t rs = (uint32_t)p.row_stride;
  // byte offsets of this lane's pieces in a half tile, out of range past the head's end
  const int kc = LDSK ? lane % KC : g, kr = LDSK ? lane / KC : li;  // its piece and its key
  const uint32_t koff = kc * 8 < p.D ? kr * rs + kc * 16 : kOut;
  uint32_t voff[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) voff[j] = li * LN < p.D ? (g * 4 + j) * rs + li * (LN * 2) : kOut;

  // where a tile's tokens lie
  struct Place {
    int id[2];         // UNI: the pages of its halves, -1 if absent
    int64_t off;       // else: byte offset of token lane % 32, -1 if masked
  };
  auto place_of = [&](const Cursor& c) {
    Place w;
    const int64_t row = (int64_t)c.b * p.width;
    const int t = c.tile * kTileTokens;
    if constexpr (UNI) {
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const int ta = t + 16 * a;
        const int id = read_const(p.table, row + (int)div_page(p.page, ta < c.r.hi ? ta : t));
        w.id[a] = (uint32_t)id < (uint32_t)p.n_pages ? id : -1;
      }
      w.off = 0;
    } else {
      const int tl = t + (lane & 31);
      const bool in = (uint32_t)(tl - c.r.lo) < (uint32_t)(c.r.hi - c.r.lo);
      const uint32_t pg = div_page(p.page, in ? tl : c.r.lo);
      const int id = p.table[row + pg];
      const bool ok = in & ((uint32_t)id < (uint32_t)p.n_pages);
      w.off = ok ? id * p.page_stride + (int64_t)(tl - (int)(pg * p.page.d)) * p.row_stride : -1;
      w.id[0] = w.id[1] = 0;
    }
    return w;
  };
  // tokens of half a that are present: [lo, lo + span) of the sequence
  auto span_of = [&](const Cursor& c, const Place& w, int a) {
    return !UNI || w.id[a] >= 0 ? (uint32_t)(c.r.hi - c.r.lo) : 0u;
  };
  auto base_of = [&](const unsigned char* pool, const Cursor& c, const Place& w, int a) {
    const int ta = c.tile * kTileTokens + 16 * a;
    const int slot = ta - (int)(div_page(p.page, ta) * p.page.d);
    const int id = w.id[a] < 0 ? 0 : w.id[a];
    return rsrc_at(pool + (c.h / p.qtiles) * p.head_stride + id * p.page_stride +
                   slot * p.row_stride);
  };
  auto shfl64 = [&](int64_t v, int src) {
    const int lo = __shfl((int)v, src, kWave), hi = __shfl((int)(v >> 32), src, kWave);
    return ((int64_t)hi << 32) | (uint32_t)lo;
  };
  auto load_k = [&](const Cursor& c, const Place& w) {
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      if constexpr (UNI) {
        const auto r = base_of(p.K, c, w, a);
        const int t = c.tile * kTileTokens + 16 * a + kr;
        const uint32_t span = span_of(c, w, a);
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          if constexpr (LDSK) {
            const bool in = (uint32_t)(t + i * KR - c.r.lo) < span;
            kreg[a][i] = load16<NT>(r, in ? koff + i * KR * rs : kOut);
          } else {
            const bool in = ((uint32_t)(t - c.r.lo) < span) & (i * 32 + g * 8 < p.D);
            kreg[a][i] = load16<NT>(r, in ? koff + i * 64 : kOut);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          const int64_t o = shfl64(w.off, 16 * a + (LDSK ? i * KR : 0) + kr);
          const int d = (LDSK ? 0 : i * 32) + kc * 8;
          const unsigned char* k = p.K + (c.h / p.qtiles) * p.head_stride + o + d * 2;
          kreg[a][i] = u32x4{0, 0, 0, 0};
          if (o >= 0 && d < p.D)
            kreg[a][i] = load_at<NT, u32x4>(k);
        }
      }
    }
  };
  auto load_v = [&](const Cursor& c, const Place& w) {
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      if constexpr (UNI) {
        const auto r = base_of(p.V, c, w, a);
        const int t = c.tile * kTileTokens + 16 * a + g * 4;
        const uint32_t span = span_of(c, w, a);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t off = (uint32_t)(t + j - c.r.lo) < span ? voff[j] : kOut;
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const uint32_t o = i == 0 || i * PW + li * LN < p.D ? off + i * PW * 2 : kOut;
            if constexpr (LN == 8) {
              vreg[4 * a + j][i] = load16<NT>(r, o);
            } else {
              const u32x2 x = load8<NT>(r, o);
              vreg[4 * a + j][i] = u32x4{x[0], x[1], 0, 0};
            }
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t o = shfl64(w.off, 16 * a + g * 4 + j);
          const unsigned char* v = p.V + (c.h / p.qtiles) * p.head_stride + o + li * (LN * 2);
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            vreg[4 * a + j][i] = u32x4{0, 0, 0, 0};
            if (o >= 0 && i * PW + li * LN < p.D) {
              if constexpr (LN == 8) {
                vreg[4 * a + j][i] = load_at<NT, u32x4>(v + i * PW * 2);
              } else {
                const u32x2 x = load_at<NT, u32x2>(v);
                vreg[4 * a + j][i] = u32x4{x[0], x[1], 0, 0};
              }
            }
          }
        }
      }
    }
  };

  u32x4 q[KS];
  float4v acc[NE];
  float m = -INFINITY, l = 0.f;
  int heads = 0, hq0 = 0;
  auto open_row = [&](const Cursor& c) {
    const int hk = c.h / p.qtiles, qt = c.h - hk * p.qtiles;
    heads = p.G - qt * kHeads < kHeads ? p.G - qt * kHeads : kHeads;
    hq0 = hk * p.G + qt * kHeads;
    // Q as the B operand: lane li holds head hq0 + li
    const unsigned char* qp = p.Q + c.b * p.q_tok + (int64_t)(hq0 + li) * p.q_head;
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      q[i] = u32x4{0, 0, 0, 0};
      if (li < heads && i * 32 + g * 8 < p.D)
        q[i] = *reinterpret_cast<const u32x4*>(qp + (i * 32 + g * 8) * 2);
    }
#pragma unroll
    for (int e = 0; e < NE; ++e) acc[e] = float4v{0, 0, 0, 0};
    m = -INFINITY;
    l = 0.f;
  };

  if (left > 0) {
    Place w_cur, w_next;
    Cursor next = cur;
    int first_tile = cur.tile;
    bool first_row = true;
    open_row(cur);  // queries do not wait for the page table
    w_cur = place_of(cur);
    load_k(cur, w_cur);
    load_v(cur, w_cur);
    const Place nowhere = {{-1, -1}, -1};
    if constexpr (DIRECT) w_next = nowhere;
    if (left > 1) {
      advance(next);
      w_next = place_of(next);
    }
    while (true) {
      const bool more = left > 1;
      float4v s[2];
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        s[a] = float4v{0, 0, 0, 0};
        if constexpr (LDSK) {
          // to operand order (lane li: key li, pieces 4 i + g); piece c of key t sits
          // at c ^ t, so that 16 keys' reads of one piece spread over the banks
          u32x4* turn = sK + wave * 16 * KC;
#pragma unroll
          for (int i = 0; i < KS; ++i)
            turn[(i * KR + kr) * KC + (kc ^ ((i * KR + kr) & (KC - 1)))] = kreg[a][i];
          __builtin_amdgcn_wave_barrier();
#pragma unroll
          for (int i = 0; i < KS; ++i)
            s[a] = mma<BF>(turn[li * KC + ((4 * i + g) ^ (li & (KC - 1)))], q[i], s[a]);
          __builtin_amdgcn_wave_barrier();
        } else {
#pragma unroll
          for (int i = 0; i < KS; ++i) s[a] = mma<BF>(kreg[a][i], q[i], s[a]);
        }
      }
      if (DIRECT || more) load_k(next, w_next);

      float x[8];
      float mt = -INFINITY;
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const int t = cur.tile * kTileTokens + 16 * a + g * 4;
        const uint32_t span = span_of(cur, w_cur, a);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          bool ok;
          if constexpr (UNI)
            ok = (uint32_t)(t + j - cur.r.lo) < span;
          else
            ok = __shfl((int)(w_cur.off >> 32), 16 * a + g * 4 + j, kWave) >= 0;
          const float v = ok ? s[a][j] * p.scale : -INFINITY;
          x[4 * a + j] = v;
          mt = fmaxf(mt, v);
        }
      }
      mt = max_over_groups(mt);
      if (!__all(mt <= m)) {
        const float mn = fmaxf(m, mt);
        const float alpha = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - mn);
        m = mn;
        l *= alpha;
#pragma unroll
        for (int e = 0; e < NE; ++e) acc[e] *= alpha;
      }
      // weights 2^(x - m); fp16 ones scaled by 2^14 (at most 2^14, 65504 being the limit)
      const float base = (m == -INFINITY ? 0.f : m) - (BF ? 0.f : 14.f);
      u32x4 hi, lo;
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        w[j] = __builtin_amdgcn_exp2f(x[j] - base);
        l += w[j];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t h2, l2;
        split2<BF>(w[2 * j], w[2 * j + 1], h2, l2);
        hi[j] = h2;
        lo[j] = l2;
      }
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        // numbers e of this lane's piece, tokens 0..7
        const int c = e / 8, d = (e % 8) / 2;
        const uint32_t sel = e & 1 ? 0x07060302u : 0x05040100u;
        u32x4 a;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          a[j] = __builtin_amdgcn_perm(vreg[2 * j + 1][c][d], vreg[2 * j][c][d], sel);
        acc[e] = mma<BF>(a, hi, acc[e]);
        acc[e] = mma<BF>(a, lo, acc[e]);
      }
      if (DIRECT || more) load_v(next, w_next);
      --left;

      const bool row_ends = cur.tile + 1 == cur.r.t1;
      if (!more || (!DIRECT && row_ends)) {
        // the row, or this wave's part of it, is done
        const bool begins = first_tile == cur.r.t0;
        const float lsum = sum_over_groups(l);
        if (begins && row_ends) {
          if (li < heads) {
#pragma unroll
            for (int c = 0; c < NV; ++c)
#pragma unroll
              for (int r = 0; r < 4; r += 8 / LN) {
                const int d = c * PW + (g * 4 + r) * LN;
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = acc[c * 8 + e % LN][r + e / LN];
                if (d < p.D) finish<BF>(p, cur.b, hq0 + li, d, m, lsum, o);
              }
          }
        } else {
          const int slot = attn_slot(wave, DIRECT || first_row ? 0 : 1);
          if (li < heads) {
            float* o = sO + (attn_sums_at(DIRECT, slot) * slot_heads + li) * row_floats;
#pragma unroll
            for (int c = 0; c < NV; ++c)
#pragma unroll
              for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int e = 0; e < LN; e += 4) {
                  const int d = c * PW + (g * 4 + r) * LN + e;
                  if (d < p.D)
                    *reinterpret_cast<float4v*>(o + d) =
                        float4v{acc[c * 8 + e][r], acc[c * 8 + e + 1][r], acc[c * 8 + e + 2][r],
                                acc[c * 8 + e + 3][r]};
                }
            if (g == 0) {
              sM[slot][li] = m;
              sL[slot][li] = lsum;
            }
          }
          if (lane == 0) {
            sRow[slot] = cur.b * H + cur.h;
            sEnds[slot] = (begins ? 1 : 0) | (row_ends ? 2 : 0);
            sLast[slot] = (int)(run_end - left) - 1 + (cur.r.t1 - cur.tile - 1);  // unit of the row's last tile
          }
        }
        first_row = false;
      }
      if (!more) break;
      cur = next;
      w_cur = w_next;
      if (!DIRECT && row_ends) {
        first_tile = cur.tile;
        open_row(cur);
      }
      if constexpr (DIRECT) w_next = nowhere;
      if (left > 1) {
        advance(next);
        w_next = place_of(next);
      }
    }
  }

  // Runs of slots of one row are joined: into the output where the row begins
  // and ends in this workgroup, else into the workspace (its first slot for a row
  // that began before, the second for one that goes on).
  __syncthreads();
  int owned = -1, last = 0;
  constexpr int kStep = DIRECT ? kAttnParts : 1;  // direct: no second parts
  const int row_of = lane < kAttnSlots ? sRow[lane] : -1;
  const int ends_of = sEnds[lane % kAttnSlots], last_of = sLast[lane % kAttnSlots];
  uint32_t todo = (uint32_t)__ballot(row_of >= 0);
  while (todo) {
    const int i = __builtin_ctz(todo);
    const int row = __builtin_amdgcn_readlane(row_of, i);
    const uint32_t members = (uint32_t)__ballot(row_of == row);
    todo &= ~members;
    const bool begins = __builtin_amdgcn_readlane(ends_of, i) & 1;
    const bool whole =
        begins && (__builtin_amdgcn_readlane(ends_of, 31 - __builtin_clz(members)) & 2);
    const int b = row / H, h = row - b * H;
    const int hk = h / p.qtiles, qt = h - hk * p.qtiles;
    const int nh = p.G - qt * kHeads < kHeads ? p.G - qt * kHeads : kHeads;
    float* part = p.partial + (2 * (int64_t)blockIdx.x + (begins ? 1 : 0)) * slot_floats(slot_heads, p.D);
    const int units = p.D / 8;
    for (int j = tid; j < nh * units; j += kAttnThreads) {
      const int hd = j / units, d = (j - hd * units) * 8;
      // every slot is read, so that the reads overlap; only members count
      float f[kAttnSlots], mm = -INFINITY, sum = 0.f;
#pragma unroll
      for (int k = 0; k < kAttnSlots; k += kStep) {
        f[k] = members >> k & 1 ? sM[k][hd] : -INFINITY;
        mm = fmaxf(mm, f[k]);
      }
      const float base = mm == -INFINITY ? 0.f : mm;
      float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < kAttnSlots; k += kStep) {
        f[k] = __builtin_amdgcn_exp2f(f[k] - base);
        const float lk = sL[k][hd];
        const float* o = sO + (attn_sums_at(DIRECT, k) * slot_heads + hd) * row_floats + d;
        const float4v x = *reinterpret_cast<const float4v*>(o);
        const float4v y = *reinterpret_cast<const float4v*>(o + 4);
        if (members >> k & 1) {
          sum += f[k] * lk;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] += f[k] * x[e];
            v[e + 4] += f[k] * y[e];
          }
        }
      }
      if (whole) {
        finish<BF>(p, b, hk * p.G + qt * kHeads + hd, d, mm, sum, v);
      } else {
        float* o = part + hd * p.D + d;
        *reinterpret_cast<float4v*>(o) = float4v{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<float4v*>(o + 4) = float4v{v[4], v[5], v[6], v[7]};
        if (d == 0) {
          part[slot_heads * p.D + hd] = mm;
          part[slot_heads * p.D + slot_heads + hd] = sum;
        }
      }
    }
    if (!DIRECT && begins && !whole) {  // goes on in the following workgroups
      owned = row;
      last = (int)(cut.part_of((uint32_t)__builtin_amdgcn_readlane(last_of, i)) / kAttnWaves);
    }
  }
  if (!DIRECT && tid == 0) p.owner[blockIdx.x] = make_int2(owned, last);

  // sequences without tokens: zeros and -inf
  auto clear = [&](int64_t b) {
    uint16_t* o = reinterpret_cast<uint16_t*>(p.Out) + b * p.Hq * p.D;
    for (int i = tid; i < p.Hq * p.D; i += kAttnThreads) o[i] = 0;
    if (p.lse)
      for (int i = tid; i < p.Hq; i += kAttnThreads) p.lse[b * p.Hq + i] = -INFINITY;
  };
  if constexpr (DIRECT) {
    if (cur.h == 0 && cur.r.hi <= cur.r.lo) clear(cur.b);
    return;
  }
  // spread over the workgroups and looked for 64 at a time
  for (int64_t b0 = blockIdx.x; b0 < p.B; b0 += (int64_t)gridDim.x * kWave) {
    const int64_t mine = b0 + (int64_t)gridDim.x * lane;
    const Range r = range_of(p, (int)(mine < p.B ? mine : b0));
    for (uint64_t none = __ballot(mine < p.B && r.hi <= r.lo); none; none &= none - 1)
      clear(b0 + (int64_t)gridDim.x * __builtin_ctzll(none));
  }
}

// Joins the partial sums of the rows that span workgroups of the first kernel:
// one workgroup per four query heads of the row that workgroup blockIdx.x began
// and left unfinished.  D / 4 lanes take a part, as many parts at once as that
// allows, and the waves take turns.
constexpr int kJoinHeads = 4;
constexpr int kMostBlocks = 1024;  // of the first kernel: parts of a row at most

template <bool BF>
__global__ __launch_bounds__(kAttnThreads) void paged_attention_join_kernel(AttnParams p) {
  __shared__ float sW[kMostBlocks * kJoinHeads];  // weight of each part
  __shared__ float sRed[2][kAttnWaves][kJoinHeads];
  __shared__ __attribute__((aligned(16))) float sV[kAttnWaves][kJoinHeads][256];
  const int2 own = p.owner[blockIdx.x];
  if (own.x < 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
  const int H = p.Hkv * p.qtiles;
  const int b = own.x / H, h = own.x - b * H;
  const int hk = h / p.qtiles, qt = h - hk * p.qtiles;
  const int slot_heads = p.G < kHeads ? p.G : kHeads;
  const int hd0 = blockIdx.y * kJoinHeads;
  const int rest = (p.G - qt * kHeads < kHeads ? p.G - qt * kHeads : kHeads) - hd0;
  if (rest <= 0) return;
  const int nh = rest < kJoinHeads ? rest : kJoinHeads;
  const int64_t size = slot_floats(slot_heads, p.D);
  const int n = own.y - (int)blockIdx.x + 1;
  // part 0 is this workgroup's second slot, the others the first slots that follow
  auto part = [&](int k) {
    return p.partial + (2 * ((int64_t)blockIdx.x + k) + (k == 0 ? 1 : 0)) * size;
  };
  // The first sums are under way while the weights are found: four parts of four
  // heads at once; past the end the last part, left out.
  const int L = p.D / 4, conc = kWave / L;
  const int sub = lane / L, col = lane - sub * L;
  const int step = kAttnWaves * conc;
  float4v x[4][kJoinHeads];
  auto fetch = [&](int k) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int ku = k + u * step;
      const float* o = part(ku < n ? ku : n - 1) + hd0 * p.D + col * 4;
#pragma unroll
      for (int i = 0; i < kJoinHeads; ++i)
        x[u][i] = *reinterpret_cast<const float4v*>(o + (i < nh ? i : 0) * p.D);
    }
  };
  // maxima and sums: thread (k, j) looks after head j of the parts k, k + 64, ..
  constexpr int kTurn = kAttnThreads / kJoinHeads;
  const int j = tid % kJoinHeads, k0 = tid / kJoinHeads;
  const int at_m = slot_heads * p.D + hd0 + (j < nh ? j : 0), at_l = at_m + slot_heads;
  const float* mine = part(k0 < n ? k0 : n - 1);
  const float m0 = mine[at_m], l0 = mine[at_l];
  int kx = wave * conc + sub;
  fetch(kx);
  float m = m0;
  for (int k = k0 + kTurn; k < n; k += kTurn) m = fmaxf(m, part(k)[at_m]);
#pragma unroll
  for (int off = kJoinHeads; off < kWave; off <<= 1) m = fmaxf(m, __shfl_xor(m, off, kWave));
  if (lane < kJoinHeads) sRed[0][wave][lane] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kAttnWaves; ++w) m = fmaxf(m, sRed[0][w][j]);
  const float base = m == -INFINITY ? 0.f : m;
  float sum = 0.f;
  for (int k = k0; k < n; k += kTurn) {
    const float w = __builtin_amdgcn_exp2f((k == k0 ? m0 : part(k)[at_m]) - base);
    sW[k * kJoinHeads + j] = w;
    sum += w * (k == k0 ? l0 : part(k)[at_l]);
  }
#pragma unroll
  for (int off = kJoinHeads; off < kWave; off <<= 1) sum += __shfl_xor(sum, off, kWave);
  if (lane < kJoinHeads) sRed[1][wave][lane] = sum;
  __syncthreads();
  float4v v[kJoinHeads];
#pragma unroll
  for (int i = 0; i < kJoinHeads; ++i) v[i] = float4v{0, 0, 0, 0};
  if (sub < conc) {
    while (kx < n) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int ku = kx + u * step;
        if (ku < n) {
#pragma unroll
          for (int i = 0; i < kJoinHeads; ++i) v[i] += sW[ku * kJoinHeads + i] * x[u][i];
        }
      }
      kx += 4 * step;
      if (kx < n) fetch(kx);
    }
  }
#pragma unroll
  for (int i = 0; i < kJoinHeads; ++i) {
    float4v t = v[i];
    for (int u = 1; u < conc; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) t[e] += __shfl(v[i][e], (col + u * L) & 63, kWave);
    if (sub == 0) *reinterpret_cast<float4v*>(&sV[wave][i][col * 4]) = t;
  }
  __syncthreads();
  if (wave < nh && lane < L) {
    float4v t = {0, 0, 0, 0};
    float total = 0.f, mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) {
      t += *reinterpret_cast<const float4v*>(&sV[w][wave][lane * 4]);
      total += sRed[1][w][wave];
      mx = fmaxf(mx, sRed[0][w][wave]);
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    const int64_t head = (int64_t)b * p.Hq + hk * p.G + qt * kHeads + hd0 + wave;
    u32x2 u;
#pragma unroll
    for (int e = 0; e < 2; ++e)
      u[e] = to16<BF>(t[2 * e] * inv) | ((uint32_t)to16<BF>(t[2 * e + 1] * inv) << 16);
    *reinterpret_cast<u32x2*>(p.Out + (head * p.D + lane * 4) * 2) = u;
    if (p.lse && lane == 0) p.lse[head] = lse_of<BF>(mx, total);
  }
}

constexpr int64_t kLdsBytes = 160 * 1024;
// What the kernel declares itself: the keys' turning buffer and small arrays.
int64_t static_lds(int64_t D) { return D > 128 ? 2048 : D > 64 ? 18 * 1024 : 10 * 1024; }
int64_t lds_bytes(int heads, int64_t D, bool direct) {
  return (attn_sums_at(direct, kAttnSlots - 1) + 1) * heads * (D + 4) * 4;
}

struct Grid {
  int64_t blocks, partials;  // workgroups; partial sums they may leave
  bool direct;
};

// Tiles a wave of the longest row, up to which a (sequence, head) has a workgroup of
// its own and nothing is left to join; more of them where the rows alone occupy half
// the CUs.  Measured (us on the GPU, own workgroup / split and joined; rows of up to
// 512, 768, 1024, 2048 tokens), 8 key heads of 128: 4 sequences 9.6 / 11.5, 12.1 /
// 11.4, 14.8 / 11.8, 26 / 14; 16 sequences 9.8 / 13.4, 13.3 / 15.7, 16.5 / 17.0, 29 /
// 25; 64 sequences 19 / 25, 26 / 30, 32 / 37, 63 / 63; of 64, 16 sequences 8.1 / 13.1,
// 9.8 / 13.7, 11.7 / 14.1, 20 / 18; of 256, up to 256 tokens 4 sequences 10.9 / 14.3, 64
// 26 / 28, up to 512 15.7 / 14.8, 42 / 40.
int64_t direct_tiles(int64_t rows, int64_t D) {
  return D > 128 ? 2 : 2 * rows >= device_cus() ? 8 : 4;
}

// Workgroups of their own per CU, up to which that holds: more of them come in
// rounds, each of which waits for memory from its start, where the split kernel
// fetches a row's first tile during the row before.  Measured (us, own / split; up to
// 32, 128, 256 tokens): 8 key heads of 64, 4 query heads each, 256 sequences (8 a CU) 8 /
// 9, 14 / 22, 22 / 28, 512 (16) 14 / 13, 26 / 31, 38 / 42, 1024 (32) 26 / 20, 44 / 46, 70 /
// 70; of 128, 128 sequences (4) 8 / 8, 14 / 19, 23 / 26, 256 (8) 15 / 10, 27 / 27, 41 / 40;
// of 256, 64 sequences (2) 10 / 10, 20 / 23, 28 / 28, 128 (4) 20 / 12, 35 / 30, 53 / 43.
// With one row a sequence the split kernel has a length and a page to find for each:
// 4096 sequences, one key head of 64 14 / 25, 24 / 42, 35 / 54, of 128 29 / 27, 49 / 54,
// 71 / 79; of 256 83 / 37, 139 / 89, 206 / 147.
bool direct_rows(int64_t B, int64_t H, int heads, int64_t D) {
  if (H == 1 && D <= 128) return true;
  const int64_t by_lds = kLdsBytes / (lds_bytes(heads, D, true) + static_lds(D));
  const int64_t by_regs = D > 128 ? 1 : D > 64 ? 2 : 4;  // at once
  const int64_t rounds = D > 64 ? 2 : 4;
  return B * H <= device_cus() * rounds * (by_lds < by_regs ? by_lds : by_regs);
}

// Workgroups of the first kernel: as many as the GPU holds at once, or one for
// each (sequence, head).
Grid attn_grid(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t capacity, int64_t window) {
  const int64_t G = Hq / Hkv, H = Hkv * ((G + kHeads - 1) / kHeads);
  const int heads = (int)(G < kHeads ? G : kHeads);
  // tiles of a row; a window may begin inside one
  int64_t tiles = (capacity + kTileTokens - 1) / kTileTokens;
  if (window > 0 && window < capacity) {
    const int64_t seen = (window + kTileTokens - 2) / kTileTokens + 1;
    if (seen < tiles) tiles = seen;
  }
  if (tiles <= direct_tiles(B * H, D) * kAttnWaves && direct_rows(B, H, heads, D))
    return {B * H, 0, true};
  const int64_t most = (B * H * tiles + kAttnWaves - 1) / kAttnWaves;
  const int64_t by_lds = kLdsBytes / (lds_bytes(heads, D, false) + static_lds(D));
  const int64_t by_regs = blocks_per_cu(D);
  int64_t grid = device_cus() * (by_lds < by_regs ? by_lds : by_regs);
  if (grid > kMostBlocks) grid = kMostBlocks;
  const int64_t blocks = most < grid ? most : grid;
  return {blocks, 2 * blocks, false};
}

template <bool BF, int DV, bool UNI, bool NT, bool DIRECT>
hipError_t launch_kernel(const AttnParams& p, int64_t grid, hipStream_t s) {
  const auto fn = paged_attention_kernel<BF, DV, UNI, NT, DIRECT>;
  const int lds = (int)lds_bytes(p.G < kHeads ? p.G : kHeads, p.D, DIRECT);
  if (lds + static_lds(p.D) > 64 * 1024) {  // above what every kernel may use
    static std::atomic<uint64_t> done{0};
    const hipError_t e = lds_limit_once(reinterpret_cast<const void*>(fn),
                                        (int)lds_bytes(kHeads, DV, DIRECT), done);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(fn, dim3((uint32_t)grid), dim3(kAttnThreads), lds, s, p);
  return hipGetLastError();
}

// Rows of whole 128-byte lines that no other head or group of query heads reads.
bool whole_lines(const AttnParams& p) {
  const uint64_t places = reinterpret_cast<uint64_t>(p.K) | reinterpret_cast<uint64_t>(p.V) |
                          (uint64_t)(p.page_stride | p.row_stride | p.head_stride) |
                          (uint64_t)p.D * 2;
  return p.qtiles == 1 && places % 128 == 0;
}

template <bool BF, int DV>
hipError_t launch_dv(const AttnParams& p, int64_t grid, hipStream_t s) {
  const bool nt = whole_lines(p);
  const auto form = [&](auto uni, auto lines) {
    return p.direct ? launch_kernel<BF, DV, uni, lines, true>(p, grid, s)
                    : launch_kernel<BF, DV, uni, lines, false>(p, grid, s);
  };
  using std::false_type, std::true_type;
  if (p.page.d % 16 == 0)
    return nt ? form(true_type{}, true_type{}) : form(true_type{}, false_type{});
  return nt ? form(false_type{}, true_type{}) : form(false_type{}, false_type{});
}

template <bool BF>
hipError_t launch_t(const AttnParams& p, int64_t grid, hipStream_t s) {
  const hipError_t e = p.D <= 64    ? launch_dv<BF, 64>(p, grid, s)
                       : p.D <= 128 ? launch_dv<BF, 128>(p, grid, s)
                                    : launch_dv<BF, 256>(p, grid, s);
  if (e != hipSuccess || p.direct) return e;
  const int heads = p.G < kHeads ? p.G : kHeads;
  hipLaunchKernelGGL((paged_attention_join_kernel<BF>),
                     dim3((uint32_t)grid, (heads + kJoinHeads - 1) / kJoinHeads),
                     dim3(kAttnThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace

int64_t attn_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t capacity) {
  const Grid g = attn_grid(B, Hq, Hkv, D, capacity, 0);  // a window takes no more
  const int64_t G = Hq / Hkv;
  if (g.direct) return 0;
  return g.partials * slot_floats((int)(G < kHeads ? G : kHeads), (int)D) * (int64_t)sizeof(float) +
         g.blocks * (int64_t)sizeof(int2);
}

hipError_t launch_paged_attention(int dtype, const AttnArgs& a, hipStream_t stream) {
  AttnParams p;
  p.Q = static_cast<const unsigned char*>(a.Q);
  p.K = static_cast<const unsigned char*>(a.k_pages);
  p.V = static_cast<const unsigned char*>(a.v_pages);
  p.q_tok = 2 * a.q_tok;
  p.q_head = 2 * a.q_head;
  p.page_stride = 2 * a.page_stride;
  p.row_stride = 2 * a.row_stride;
  p.head_stride = 2 * a.head_stride;
  p.table = a.page_table;
  p.lens = a.lens;
  p.Out = static_cast<unsigned char*>(a.Out);
  p.lse = a.lse;
  p.partial = static_cast<float*>(a.workspace);
  p.page = fast_div(a.page_size);
  p.n_pages = (int32_t)a.n_pages;
  p.width = (int32_t)a.width;
  p.B = (int32_t)a.B;
  p.Hq = (int32_t)a.Hq;
  p.Hkv = (int32_t)a.Hkv;
  p.D = (int32_t)a.D;
  p.G = (int32_t)(a.Hq / a.Hkv);
  p.qtiles = (p.G + kHeads - 1) / kHeads;
  p.window = (int32_t)a.window;
  p.scale = a.scale_log2;
  const Grid g = attn_grid(a.B, a.Hq, a.Hkv, a.D, a.width * a.page_size, a.window);
  p.direct = g.direct;
  p.full = a.D > 64 && whole_lines(p) && a.page_size % 16 == 0 && g.blocks >= 2 * device_cus();
  p.owner = reinterpret_cast<int2*>(
      p.partial + g.partials * slot_floats(p.G < kHeads ? p.G : kHeads, p.D));
  return dtype == TQ_BF16 ? launch_t<true>(p, g.blocks, stream)
                          : launch_t<false>(p, g.blocks, stream);
}

}  // namespace tq
