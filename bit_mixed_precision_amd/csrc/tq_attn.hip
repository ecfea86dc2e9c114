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
// key-value head), processed by one wave without LDS:
//  * S^T = K Q^T by v_mfma_f32_16x16x32 with K as the A operand: lane (li, g)
//    loads 16 bytes of token li, so a tile's two halves of 16 tokens come
//    straight from HBM in operand order.  Up to 16 query heads are the columns;
//    the matrix cores idle over 90% of the time even so, which is why one
//    kernel serves every G.
//  * The scores arrive with lane = head and 4 tokens of each half per lane,
//    which is the B operand order of the second product when V's tokens are
//    taken in the same order: lane group g contributes tokens 4 g .. 4 g + 3 of
//    both halves.  P never leaves its registers.
//  * O^T += V^T P^T: lane (li, g) loads 8 consecutive numbers (4 for D <= 64)
//    of its 8 tokens, whole 256-byte rows per 16 lanes, and turns them into A
//    operands (8 tokens of one number) with 4 v_perm_b32 per operand.  O^T keeps
//    lane = head, so rescaling and the final division need no exchange.
//  * P is split into two 16-bit numbers (high part and remainder), so rounding
//    it to the cache's type costs no accuracy; fp16 exponents are shifted by 14
//    so that weights down to 2^-28 of the largest keep all their bits.
//  * Loads are buffer loads whose lane offset is pushed out of range where a
//    token is masked or a head ends, so what lies in unused places (NaN
//    included) reads as zero and no branch is needed.
//
// Work is split over the flattened list of (sequence, head, tile): every
// workgroup takes an equal contiguous share, computed on the device from the
// lengths, so one long sequence, or many ragged ones, fill the GPU alike and the
// host needs no lengths.  Inside a workgroup the four waves take tiles in turn
// and join through LDS; a (sequence, head) that spans workgroups leaves partial
// sums in the workspace for the joining kernel.

#include "tq.h"
#include "tq_common.h"
#include "tq_decode.h"
#include "tq_kernels.h"
#include "tq_mfma.h"

namespace tq {
namespace {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));

constexpr int kAttnWaves = 4;
constexpr int kAttnThreads = kAttnWaves * kWave;
constexpr int kTileTokens = 32;
constexpr int kHeads = 16;                // query heads per workgroup
constexpr uint32_t kOut = 0x80000000u;    // a lane offset past every buffer
constexpr uint32_t kSpan = 0x7ffffffcu;   // bytes a buffer resource covers
constexpr float kLog2e = 1.4426950408889634f;

// t / d for 0 <= t < 2^30: exact with m = ceil(2^(30 + s) / d), s = ceil(log2 d).
struct FastDiv {
  uint32_t d, m, shift;
};

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
  float* partial;  // [2 * workgroups][kHeads * D + 2 * kHeads]
  FastDiv page;
  int32_t n_pages, width, B, Hq, Hkv, D, G, qtiles, window;
  int32_t direct;  // one workgroup per (sequence, head): nothing is split
  float scale;
};

template <bool BF>
__device__ __forceinline__ float4v mma(u32x4 a, u32x4 b, float4v c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a),
                                                   __builtin_bit_cast(bf8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a),
                                                  __builtin_bit_cast(half8, b), c, 0, 0, 0);
}

// Two floats as two 16-bit numbers (low half first) rounded toward zero, and
// what that left of them, rounded the same way: hi + lo is within 2^-20 (fp16,
// normal range) or 2^-14 (bf16) of the value.
template <bool BF>
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  if constexpr (BF) {
    const uint32_t xb = __builtin_bit_cast(uint32_t, x), yb = __builtin_bit_cast(uint32_t, y);
    hi = __builtin_amdgcn_perm(yb, xb, 0x07060302u);
    const float xr = x - __builtin_bit_cast(float, xb & 0xffff0000u);
    const float yr = y - __builtin_bit_cast(float, yb & 0xffff0000u);
    lo = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, yr), __builtin_bit_cast(uint32_t, xr),
                               0x07060302u);
  } else {
    const auto h = __builtin_amdgcn_cvt_pkrtz(x, y);
    hi = __builtin_bit_cast(uint32_t, h);
    lo = __builtin_bit_cast(uint32_t,
                            __builtin_amdgcn_cvt_pkrtz(x - (float)h[0], y - (float)h[1]));
  }
}

template <bool BF>
__device__ __forceinline__ uint16_t to16(float v) {
  if constexpr (BF) {
    const __bf16 h = (__bf16)v;
    return __builtin_bit_cast(uint16_t, h);
  } else {
    return f2h_bits(v);
  }
}

__device__ __forceinline__ uint32_t div_page(const FastDiv& f, uint32_t t) {
  return (uint32_t)(((uint64_t)t * f.m) >> f.shift);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_at(const unsigned char* p) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(((uint64_t)hi << 32) | lo),
                                           (short)0, (int)kSpan, kBufferWord3);
}

__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}
__device__ __forceinline__ u32x2 load8(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
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

// Tokens [lo, hi) of sequence b, clamped to what its table row can name.
struct Range {
  int lo, hi;
};
__device__ __forceinline__ Range range_of(const AttnParams& p, int b) {
  const int64_t cap = (int64_t)p.width * p.page.d;
  int n = p.lens[b];
  n = n < 0 ? 0 : n;
  const int hi = n < cap ? n : (int)cap;
  const int lo = p.window > 0 && n > p.window ? n - p.window : 0;
  return {lo < hi ? lo : hi, hi};
}
__device__ __forceinline__ int tiles_of(Range r) {
  return r.hi > r.lo ? (r.hi + kTileTokens - 1) / kTileTokens - r.lo / kTileTokens : 0;
}

// How the flattened tiles are cut: `total` tiles over `parts` workgroups, part
// w taking [w total / parts, (w + 1) total / parts).  A part has at least four
// tiles, one for each wave.
struct Cut {
  int64_t total;
  int64_t parts;
  __device__ __forceinline__ int64_t start(int64_t w) const { return w * total / parts; }
};
__device__ __forceinline__ Cut cut_of(int64_t total, int64_t grid) {
  const int64_t most = (total + kAttnWaves - 1) / kAttnWaves;
  return {total, most < grid ? most : grid};
}

// Sum of tiles over all sequences and over those before this thread's; thread
// i looks after the sequences [i * per, (i + 1) * per).
__device__ __forceinline__ int64_t scan_tiles(const AttnParams& p, int per, int64_t* red,
                                              int64_t& total) {
  const int t = threadIdx.x;
  int64_t mine = 0;
  for (int i = 0; i < per; ++i) {
    const int b = t * per + i;
    if (b < p.B) mine += tiles_of(range_of(p, b));
  }
  int64_t inc = mine;
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const int64_t o = __shfl_up(inc, off, kWave);
    if ((t & 63) >= off) inc += o;
  }
  if ((t & 63) == 63) red[t >> 6] = inc;
  __syncthreads();
  int64_t before = inc - mine;
  total = 0;
#pragma unroll
  for (int w = 0; w < kAttnWaves; ++w) {
    if (w < (t >> 6)) before += red[w];
    total += red[w];
  }
  return before;
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
  if (p.lse && d == 0) p.lse[at] = (m + __builtin_amdgcn_logf(sum) - (BF ? 0.f : 14.f)) / kLog2e;
}

// DV: 64, 128 or 256, the head dimension rounded up (D <= DV, D % 8 == 0).
// UNI: the page size is a multiple of 16, so a half tile lies in one page and
// its base address is uniform.
template <bool BF, int DV, bool UNI>
struct Tile {
  static constexpr int kSteps = DV / 32;              // MFMA steps of a score
  static constexpr int kOps = DV / 16;                // V operands (numbers per lane)
  static constexpr int kVecs = DV == 256 ? 2 : 1;     // 16-byte (8-byte) pieces per token and lane
  static constexpr int kLane = DV == 64 ? 4 : 8;      // consecutive numbers per piece
};

template <bool BF, int DV, bool UNI>
__global__ __launch_bounds__(kAttnThreads, DV == 256 ? 2 : 3) void paged_attention_kernel(
    AttnParams p) {
  using TT = Tile<BF, DV, UNI>;
  constexpr int KS = TT::kSteps, NE = TT::kOps, NV = TT::kVecs, LN = TT::kLane;
  constexpr int PW = LN * 16;   // numbers of one piece: the joining buffer's width
  constexpr int kRow = PW + 4;  // floats per head, 4 of padding
  __shared__ __attribute__((aligned(16))) float sO[kAttnWaves * kHeads * kRow];
  __shared__ float sM[kAttnWaves * kHeads], sL[kAttnWaves * kHeads];
  __shared__ int64_t sRed[kAttnWaves];
  __shared__ int64_t sStart;
  __shared__ int sSeq;

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63, li = lane & 15, g = lane >> 4;
  const int H = p.Hkv * p.qtiles;

  // rows without tokens: zeros and -inf, spread over the workgroups
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const Range r = range_of(p, b);
    if (r.hi > r.lo) continue;
    uint16_t* o = reinterpret_cast<uint16_t*>(p.Out) + (int64_t)b * p.Hq * p.D;
    for (int i = tid; i < p.Hq * p.D; i += kAttnThreads) o[i] = 0;
    if (p.lse)
      for (int i = tid; i < p.Hq; i += kAttnThreads) p.lse[(int64_t)b * p.Hq + i] = -INFINITY;
  }

  // this workgroup's share [at, end) of the flattened tiles and where it begins
  int64_t at, end;
  int b;
  uint32_t row_units;  // tiles x heads of sequence b
  uint32_t in_row;     // offset of `at` inside sequence b
  if (p.direct) {
    b = blockIdx.x / H;
    const int n = tiles_of(range_of(p, b));
    at = 0;
    end = n;
    in_row = (uint32_t)(blockIdx.x % H) * n;
    row_units = (uint32_t)n * H;
  } else {
    const int per = (p.B + kAttnThreads - 1) / kAttnThreads;
    int64_t total;
    int64_t before = scan_tiles(p, per, sRed, total);
    const Cut c = cut_of(total * H, gridDim.x);
    if ((int64_t)blockIdx.x >= c.parts) return;
    at = c.start(blockIdx.x);
    end = c.start((int64_t)blockIdx.x + 1);
    // the thread whose sequences hold unit `at` names the sequence
    for (int i = 0; i < per; ++i) {
      const int q = tid * per + i;
      if (q >= p.B) break;
      const int64_t n = tiles_of(range_of(p, q));
      if (before * H <= at && at < (before + n) * H) {
        sSeq = q;
        sStart = before * H;
      }
      before += n;
    }
    __syncthreads();
    b = __builtin_amdgcn_readfirstlane(sSeq);
    in_row = __builtin_amdgcn_readfirstlane((int)(at - sStart));
    row_units = (uint32_t)tiles_of(range_of(p, b)) * H;
  }
  const int64_t first_unit = at;

  while (at < end) {
    if (in_row >= row_units) {  // next sequence that has tiles
      in_row = 0;
      do {
        ++b;
        row_units = (uint32_t)tiles_of(range_of(p, b)) * H;
      } while (row_units == 0);
    }
    const Range rg = range_of(p, b);
    const int n = tiles_of(rg);
    const int h = (int)(in_row / (uint32_t)n);
    const int t_first = (int)(in_row % (uint32_t)n);
    const int64_t left = end - at;
    const int t_last = (int)(t_first + left < n ? t_first + left : n);  // past the last tile
    const int hk = h / p.qtiles, qt = h % p.qtiles;
    const int heads = p.G - qt * kHeads < kHeads ? p.G - qt * kHeads : kHeads;
    const int hq0 = hk * p.G + qt * kHeads;

    // Q as the B operand: lane li holds head hq0 + li
    u32x4 q[KS];
    {
      const unsigned char* qp = p.Q + b * p.q_tok + (int64_t)(hq0 + li) * p.q_head;
#pragma unroll
      for (int c = 0; c < KS; ++c) {
        q[c] = u32x4{0, 0, 0, 0};
        if (li < heads && c * 32 + g * 8 < p.D)
          q[c] = *reinterpret_cast<const u32x4*>(qp + (c * 32 + g * 8) * 2);
      }
    }

    float4v acc[NE];
#pragma unroll
    for (int e = 0; e < NE; ++e) acc[e] = float4v{0, 0, 0, 0};
    float m = -INFINITY, l = 0.f;

    const unsigned char* kh = p.K + hk * p.head_stride;
    const unsigned char* vh = p.V + hk * p.head_stride;
    const int32_t* row = p.table + (int64_t)b * p.width;
    const int tile0 = rg.lo / kTileTokens;
    const uint32_t rs = (uint32_t)p.row_stride;

    u32x4 kreg[2][KS];
    u32x4 vreg[8][NV];  // DV == 64 uses the first two dwords of each

    // page of the half tile at token t, or -1
    auto page_of = [&](int t) -> int {
      if (t >= rg.hi) return -1;
      const int id = row[div_page(p.page, (uint32_t)t)];
      return (uint32_t)id < (uint32_t)p.n_pages ? id : -1;
    };
    auto in_range = [&](int t) { return t >= rg.lo && t < rg.hi; };

    // byte offset of token t (per lane; pages that end inside a half tile), -1 if masked
    auto token_at = [&](int t) -> int64_t {
      if (!in_range(t)) return -1;
      const uint32_t pg = div_page(p.page, (uint32_t)t);
      const int id = row[pg];
      if ((uint32_t)id >= (uint32_t)p.n_pages) return -1;
      return id * p.page_stride + (int64_t)(t - (int)(pg * p.page.d)) * p.row_stride;
    };

    int id_next[2];  // pages of the tile whose loads come next (UNI)
    auto fetch_ids = [&](int tile) {
      if constexpr (UNI) {
        const int t0 = (tile0 + tile) * kTileTokens;
        id_next[0] = __builtin_amdgcn_readfirstlane(page_of(t0));
        id_next[1] = __builtin_amdgcn_readfirstlane(page_of(t0 + 16));
      }
    };
    int id_k[2], id_v[2];
    auto load_k = [&](int tile) {
      const int t0 = (tile0 + tile) * kTileTokens;
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const int t = t0 + 16 * a + li;
        if constexpr (UNI) {
          const int id = id_next[a];
          id_k[a] = id;
          const int ta = t0 + 16 * a;
          const int in_page = ta - (int)(div_page(p.page, (uint32_t)ta) * p.page.d);
          const auto r = rsrc_at(kh + (id < 0 ? 0 : id) * p.page_stride + in_page * p.row_stride);
          const bool ok = id >= 0 && in_range(t);
          const uint32_t off = ok ? li * rs + g * 16 : kOut;
#pragma unroll
          for (int c = 0; c < KS; ++c)
            kreg[a][c] = load16(r, c * 32 + g * 8 < p.D ? off + c * 64 : kOut);
        } else {
          const int64_t o = token_at(t);
#pragma unroll
          for (int c = 0; c < KS; ++c) {
            kreg[a][c] = u32x4{0, 0, 0, 0};
            if (o >= 0 && c * 32 + g * 8 < p.D)
              kreg[a][c] = *reinterpret_cast<const u32x4*>(kh + o + c * 64 + g * 16);
          }
        }
      }
    };
    auto load_v = [&](int tile) {
      const int t0 = (tile0 + tile) * kTileTokens;
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        if constexpr (UNI) {
          const int id = id_v[a];
          const int ta = t0 + 16 * a;
          const int in_page = ta - (int)(div_page(p.page, (uint32_t)ta) * p.page.d);
          const auto r = rsrc_at(vh + (id < 0 ? 0 : id) * p.page_stride + in_page * p.row_stride);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bool ok = id >= 0 && in_range(ta + g * 4 + j);
            const uint32_t off = ok ? (g * 4 + j) * rs + li * (LN * 2) : kOut;
#pragma unroll
            for (int c = 0; c < NV; ++c) {
              const uint32_t o = c * 128 + li * LN < p.D ? off + c * 256 : kOut;
              if constexpr (LN == 8) {
                vreg[4 * a + j][c] = load16(r, o);
              } else {
                const u32x2 x = load8(r, o);
                vreg[4 * a + j][c] = u32x4{x[0], x[1], 0, 0};
              }
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int64_t o = token_at(t0 + 16 * a + g * 4 + j);
#pragma unroll
            for (int c = 0; c < NV; ++c) {
              vreg[4 * a + j][c] = u32x4{0, 0, 0, 0};
              if (o >= 0 && c * 128 + li * LN < p.D) {
                const unsigned char* src = vh + o + c * 256 + li * (LN * 2);
                if constexpr (LN == 8) {
                  vreg[4 * a + j][c] = *reinterpret_cast<const u32x4*>(src);
                } else {
                  const u32x2 x = *reinterpret_cast<const u32x2*>(src);
                  vreg[4 * a + j][c] = u32x4{x[0], x[1], 0, 0};
                }
              }
            }
          }
        }
      }
    };

    int tile = t_first + wave;
    if (tile < t_last) {
      fetch_ids(tile);
      load_k(tile);
      id_v[0] = id_k[0];
      id_v[1] = id_k[1];
      load_v(tile);
      if (tile + kAttnWaves < t_last) fetch_ids(tile + kAttnWaves);
    }
    for (; tile < t_last; tile += kAttnWaves) {
      const bool more = tile + kAttnWaves < t_last;
      const int t0 = (tile0 + tile) * kTileTokens;
      float4v s[2];
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        s[a] = float4v{0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < KS; ++c) s[a] = mma<BF>(kreg[a][c], q[c], s[a]);
      }
      // masked tokens, by the page that the loads used
      bool page_ok[2] = {true, true};
      if constexpr (UNI) {
        page_ok[0] = id_k[0] >= 0;
        page_ok[1] = id_k[1] >= 0;
      }
      if (more) load_k(tile + kAttnWaves);

      float x[8];
      float mt = -INFINITY;
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = t0 + 16 * a + g * 4 + j;
          bool ok;
          if constexpr (UNI)
            ok = page_ok[a] && in_range(t);
          else
            ok = token_at(t) >= 0;
          const float v = ok ? s[a][j] * p.scale : -INFINITY;
          x[4 * a + j] = v;
          mt = fmaxf(mt, v);
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
      if (more) {
        id_v[0] = id_k[0];
        id_v[1] = id_k[1];
        load_v(tile + kAttnWaves);
        if (tile + 2 * kAttnWaves < t_last) fetch_ids(tile + 2 * kAttnWaves);
      }
    }
    l = sum_over_groups(l);

    // join the waves, one piece of the head at a time: sO[wave][head][number]
    const bool whole = t_first == 0 && t_last == n;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (at == first_unit ? 0 : 1);
    float* part = p.partial + slot * (kHeads * (p.D + 2));
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      __syncthreads();  // the previous readers are done
      if (li < heads) {
        float* o = sO + (wave * kHeads + li) * kRow;
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int e = 0; e < LN; e += 4)
            *reinterpret_cast<float4v*>(o + (g * 4 + r) * LN + e) =
                float4v{acc[c * 8 + e][r], acc[c * 8 + e + 1][r], acc[c * 8 + e + 2][r],
                        acc[c * 8 + e + 3][r]};
        if (g == 0) {
          sM[wave * kHeads + li] = m;
          sL[wave * kHeads + li] = l;
        }
      }
      __syncthreads();
      const int units = (p.D - c * PW < PW ? p.D - c * PW : PW) / 8;  // 8 numbers each
      for (int i = tid; i < heads * units; i += kAttnThreads) {
        const int hd = i / units, dl = (i % units) * 8, d = c * PW + dl;
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kAttnWaves; ++w) mm = fmaxf(mm, sM[w * kHeads + hd]);
        const float base = mm == -INFINITY ? 0.f : mm;
        float sum = 0.f, v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kAttnWaves; ++w) {
          const float f = __builtin_amdgcn_exp2f(sM[w * kHeads + hd] - base);
          sum += f * sL[w * kHeads + hd];
          const float* o = sO + (w * kHeads + hd) * kRow + dl;
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += f * o[e];
        }
        if (whole) {
          finish<BF>(p, b, hq0 + hd, d, mm, sum, v);
        } else {
          float* o = part + hd * p.D + d;
          *reinterpret_cast<float4v*>(o) = float4v{v[0], v[1], v[2], v[3]};
          *reinterpret_cast<float4v*>(o + 4) = float4v{v[4], v[5], v[6], v[7]};
          if (d == 0) {
            part[kHeads * p.D + hd] = mm;
            part[kHeads * p.D + kHeads + hd] = sum;
          }
        }
      }
    }
    at += t_last - t_first;
    in_row += t_last - t_first;
  }
}

// Joins the partial sums of every (sequence, head) that spans workgroups of the
// first kernel (grid `parts_grid`); one workgroup per (sequence, head).
template <bool BF>
__global__ __launch_bounds__(kAttnThreads) void paged_attention_join_kernel(AttnParams p,
                                                                            int parts_grid) {
  __shared__ int64_t sRed[kAttnWaves];
  __shared__ int64_t sBefore;
  const int tid = threadIdx.x;
  const int H = p.Hkv * p.qtiles;
  const int b = blockIdx.x / H, h = blockIdx.x % H;
  const int n = tiles_of(range_of(p, b));
  if (n == 0) return;
  const int per = (p.B + kAttnThreads - 1) / kAttnThreads;
  int64_t total;
  int64_t before = scan_tiles(p, per, sRed, total);
  for (int i = 0; i < per; ++i) {
    const int q = tid * per + i;
    if (q >= p.B) break;
    if (q == b) sBefore = before;
    before += tiles_of(range_of(p, q));
  }
  __syncthreads();
  const Cut c = cut_of(total * H, parts_grid);
  const int64_t u0 = sBefore * H + (int64_t)h * n, u1 = u0 + n;
  // the first part that reaches past u0, and the one that reaches u1
  int64_t w0 = u0 * c.parts / c.total;
  while (c.start(w0 + 1) <= u0) ++w0;
  while (c.start(w0) > u0) --w0;
  if (c.start(w0 + 1) >= u1) return;  // one part had it all
  const int hk = h / p.qtiles, qt = h % p.qtiles;
  const int heads = p.G - qt * kHeads < kHeads ? p.G - qt * kHeads : kHeads;
  const int hq0 = hk * p.G + qt * kHeads;
  const int64_t size = kHeads * (p.D + 2);
  const int per_head = p.D / 8;
  for (int i = tid; i < heads * per_head; i += kAttnThreads) {
    const int hd = i / per_head, d = (i % per_head) * 8;
    float m = -INFINITY, sum = 0.f, v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int64_t w = w0; c.start(w) < u1; ++w) {
      // a part's first fragment is in its even slot, its last one in the odd
      const int64_t slot = 2 * w + (c.start(w) >= u0 ? 0 : 1);
      const float* part = p.partial + slot * size;
      const float pm = part[kHeads * p.D + hd], pl = part[kHeads * p.D + kHeads + hd];
      const float mn = fmaxf(m, pm);
      const float base = mn == -INFINITY ? 0.f : mn;
      const float fa = __builtin_amdgcn_exp2f(m - base), fb = __builtin_amdgcn_exp2f(pm - base);
      m = mn;
      sum = sum * fa + pl * fb;
      const float* o = part + hd * p.D + d;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = v[e] * fa + o[e] * fb;
    }
    finish<BF>(p, b, hq0 + hd, d, m, sum, v);
  }
}

FastDiv fast_div(int64_t d) {
  uint32_t s = 0;
  while ((int64_t(1) << s) < d) ++s;
  const uint64_t m = ((uint64_t(1) << (30 + s)) + d - 1) / d;
  return {(uint32_t)d, (uint32_t)m, 30 + s};
}

int waves_grid(int64_t D) { return device_cus() * (D > 128 ? 2 : 3); }

// Workgroups of the first kernel, and whether each (sequence, head) has its own.
// With at most four tiles in a row every wave has one and a join would only
// cost its launch.
int64_t attn_grid(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t capacity, bool* direct) {
  const int64_t G = Hq / Hkv, H = Hkv * ((G + kHeads - 1) / kHeads);
  const int64_t tiles = capacity / kTileTokens + 2;  // a window may begin inside a tile
  *direct = capacity <= kAttnWaves * kTileTokens;
  if (*direct) return B * H;
  const int64_t most = (B * H * tiles + kAttnWaves - 1) / kAttnWaves;
  const int64_t grid = waves_grid(D);
  return most < grid ? most : grid;
}

template <bool BF, int DV>
hipError_t launch_dv(const AttnParams& p, int grid, hipStream_t s) {
  if (p.page.d % 16 == 0)
    hipLaunchKernelGGL((paged_attention_kernel<BF, DV, true>), dim3(grid), dim3(kAttnThreads), 0, s,
                       p);
  else
    hipLaunchKernelGGL((paged_attention_kernel<BF, DV, false>), dim3(grid), dim3(kAttnThreads), 0,
                       s, p);
  return hipGetLastError();
}

template <bool BF>
hipError_t launch_t(const AttnParams& p, int grid, hipStream_t s) {
  hipError_t e = p.D <= 64    ? launch_dv<BF, 64>(p, grid, s)
                 : p.D <= 128 ? launch_dv<BF, 128>(p, grid, s)
                              : launch_dv<BF, 256>(p, grid, s);
  if (e != hipSuccess || p.direct) return e;
  hipLaunchKernelGGL((paged_attention_join_kernel<BF>), dim3(p.B * p.Hkv * p.qtiles),
                     dim3(kAttnThreads), 0, s, p, grid);
  return hipGetLastError();
}

}  // namespace

int64_t attn_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t capacity) {
  bool direct;
  const int64_t grid = attn_grid(B, Hq, Hkv, D, capacity, &direct);
  return direct ? 0 : 2 * grid * kHeads * (D + 2) * (int64_t)sizeof(float);
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
  bool direct;
  const int64_t grid = attn_grid(a.B, a.Hq, a.Hkv, a.D, a.width * a.page_size, &direct);
  p.direct = direct;
  return dtype == TQ_BF16 ? launch_t<true>(p, (int)grid, stream)
                          : launch_t<false>(p, (int)grid, stream);
}

}  // namespace tq
