// The attention weight that every cached token receives, added to a running sum: what
// an eviction goes by.
//
//     w[b][h][t] = sum over nodes i and heads g of the group of
//                  exp(scale * q[b][i][hG + g] . k[t][h] - lse[b][i][hG + g])
//     scores[b][h][t] = decay * scores[b][h][t] + w   (cached tokens)
//                     = w                             (the nodes' own tokens)
//
// The normalizing sums are known (the attention before returned them), so tokens do not
// depend on each other and nothing is split or joined: a wave holds some tokens' keys in
// registers and walks through the rows (node, head of the group), whose queries lie in LDS.
//
// What bounds it: a token is 2 D bytes of a key-value head, and with R rows R exponentials at a
// quarter of the vector rate beside 2 R D operations.  16 sequences of up to 16384 tokens, 8 heads
// of 128, 128 rows each: 303 MB in 86 - 90 us (in turn 94 against 86 with each lane finding its own
// tokens), 3.4 TB/s; exponentials and the additions around them take 25 us, the matrix product
// 25, reading 44, and a unit of 128 tokens is too short to hide one behind the other.  Vector
// units are busy 56% of the time, twice what those exponentials and additions need; what
// the other half is has not been looked into.  Of one row each, 64 sequences of
// 1000 .. 8000 tokens: 458 MB in 105 us, 4.4 TB/s, waves waiting half their time.
// Two tiles of 16 tokens a wave: four need twice the registers, two workgroups a CU instead of
// three: 91 against 86, and one sequence of 2000 tokens 7.3 against 5.5.

#include <atomic>

#include "tq.h"
#include "tq_attn_dev.h"
#include "tq_common.h"
#include "tq_decode.h"
#include "tq_kernels.h"
#include "tq_mfma.h"

namespace tq {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kMaskWords = 4;
constexpr int kMaxNodes = 64 * kMaskWords;
constexpr int kQueryBytes = 48 * 1024;  // of LDS for queries
constexpr int kMostRows = 8192;         // (nodes times heads of a group)
constexpr int kCuLds = 160 * 1024;
// What the kernel declares itself: every node's bits and first token (and a flag).
constexpr int kFixedLds = kMaxNodes * (kMaskWords * 8 + 4) + 16;

struct WeightsParams {
  const unsigned char* Q;
  const unsigned char* K;
  int64_t q_seq, q_tok, q_head;                  // bytes
  int64_t page_stride, row_stride, head_stride;  // bytes
  const int32_t* table;
  const int32_t* lens;
  const int32_t* nodes;
  const uint64_t* mask;
  int64_t mask_seq;  // words
  const float* lse;  // [B][T][Hq]
  float* scores;
  int64_t s_seq, s_head;  // numbers
  FastDiv page, group;
  int32_t n_pages, width, B, T, words, Hq, Hkv, D, G, window, S;
  int32_t tiles;  // not 0: of the longest sequence; every tile has a workgroup
  int32_t chunk;  // rows whose queries lie in LDS at once, a multiple of 16
  float scale, decay;
};

template <bool BF>
__device__ __forceinline__ float4v mma16(u32x4 a, u32x4 b, float4v c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a),
                                                   __builtin_bit_cast(bf8, b), c, 0, 0, 0);
  else
    return mfma16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c);
}

// A sequence: n cached tokens, m nodes, tokens [lo, hi) that any node may see, the
// tiles [t0, t1) of UT tokens whose sums change.
struct Seq {
  int n, m, lo, hi, t0, t1;
};
template <int UT>
__device__ __forceinline__ Seq read_seq(const WeightsParams& p, int b) {
  Seq s;
  const int len = read_const(p.lens, b), nodes = p.nodes ? read_const(p.nodes, b) : p.T;
  const int cap = p.width * (int)p.page.d;
  s.n = len < 0 ? 0 : len < cap ? len : cap;
  s.m = nodes < 0 ? 0 : nodes < p.T ? nodes : p.T;
  s.hi = s.n + s.m < cap ? s.n + s.m : cap;
  s.lo = p.window > 0 && s.n > p.window ? s.n - p.window : 0;
  const int last = s.hi < p.S ? s.hi : p.S;
  s.t0 = p.decay == 1.f ? s.lo / UT : 0;
  s.t1 = s.m == 0 && p.decay == 1.f ? s.t0 : (last + UT - 1) / UT;
  if (s.t1 < s.t0) s.t1 = s.t0;
  return s;
}

// DV: 64, 128 or 256, the head dimension rounded up.  NT: 16-token tiles of a wave.  RUNS: 16
// tokens lie in one page, so that a wave finds them by scalar arithmetic; otherwise each lane
// finds its own.
template <bool BF, int DV, int NT, bool RUNS>
__global__ __launch_bounds__(kThreads, DV > 128 ? 2 : 3) void cache_weights_kernel(WeightsParams p) {
  constexpr int KS = DV / 32, UT = 16 * NT * kWaves, PC = DV / 8;
  // queries of `chunk` rows, a row's 16-byte pieces turned so that 16 rows' reads of one piece
  // spread over the banks; then lse of all rows, times log2 e, +inf: the row adds nothing
  extern __shared__ __attribute__((aligned(16))) unsigned char sQ[];
  const int chunk = p.chunk;
  float* const sLse = reinterpret_cast<float*>(sQ + chunk * DV * 2);
  __shared__ int sOut;  // some row adds nothing
  __shared__ uint64_t sBits[kMaxNodes][kMaskWords];
  __shared__ int sLow[kMaxNodes];

  const int tid = threadIdx.x;
  const int wave = uni(tid >> 6), lane = tid & 63, li = lane & 15, g = lane >> 4;

  int b = 0, h = 0, tile = 0;
  uint32_t left = 1;
  Seq s;
  if (p.tiles > 0) {
    const int row = blockIdx.x / p.tiles;
    tile = blockIdx.x - row * p.tiles;
    b = row / p.Hkv;
    h = row - b * p.Hkv;
    s = read_seq<UT>(p, b);
    tile += s.t0;
    if (tile >= s.t1) return;
  } else {
    const int per = (p.B + kWave - 1) / kWave;
    auto tiles_of = [&](int x, bool in) -> uint32_t {
      const Seq q = read_seq<UT>(p, x < p.B ? x : p.B - 1);
      return in && x < p.B ? q.t1 - q.t0 : 0;
    };
    uint32_t mine = 0;
    for (int i = 0; i < per; ++i) mine += tiles_of(lane * per + i, true);
    const uint32_t inc = scan_wave(mine, lane);
    const Cut cut((uint32_t)uni((int)__shfl(inc, 63, kWave)) * p.Hkv, gridDim.x);
    if (blockIdx.x >= cut.parts) return;
    uint32_t at = cut.start(blockIdx.x);
    left = cut.start(blockIdx.x + 1) - at;
    const uint64_t has = __ballot(at < inc * p.Hkv);
    const int src = has ? __builtin_ctzll(has) : 0;
    at -= (uint32_t)__builtin_amdgcn_readlane((int)(inc - mine), src) * p.Hkv;
    b = src * per;
    for (int i = 0; per > 1 && i < per; i += kWave) {
      const uint32_t n = tiles_of(src * per + i + lane, i + lane < per);
      const uint32_t run = scan_wave(n, lane);
      const uint64_t hit = __ballot(at < run * p.Hkv);
      if (hit) {
        const int k = __builtin_ctzll(hit);
        b = src * per + i + k;
        at -= (uint32_t)__builtin_amdgcn_readlane((int)(run - n), k) * p.Hkv;
        break;
      }
      at -= (uint32_t)__builtin_amdgcn_readlane((int)run, kWave - 1) * p.Hkv;
    }
    if (b >= p.B) b = p.B - 1;
    s = read_seq<UT>(p, b);
    const uint32_t n = s.t1 > s.t0 ? s.t1 - s.t0 : 1;
    h = at / n < (uint32_t)p.Hkv ? at / n : p.Hkv - 1;
    tile = s.t0 + at % n;
  }

  // Rows r0 .. of the queries to LDS, zeros past a head's end.  What stands behind the last row
  // is multiplied and gets a weight of 2^(-inf): the last row again, since zeros times
  // an infinite key would make NaN of that.
  auto stage = [&](int r0, int rows) {
    const int n = (rows - r0 < chunk ? rows - r0 : chunk) + 15 & ~15;
    for (int x = anew(threadIdx.x); x < n * PC; x += kThreads) {
      const int r = x / PC, piece = x - r * PC, row = r0 + r < rows ? r0 + r : rows - 1;
      u32x4 v = {0, 0, 0, 0};
      if (piece * 8 < p.D) {
        const int i = div_page(p.group, row);
        v = *reinterpret_cast<const u32x4*>(p.Q + b * p.q_seq + i * p.q_tok +
                                            (int64_t)(h * p.G + (row - i * p.G)) * p.q_head +
                                            piece * 16);
      }
      *reinterpret_cast<u32x4*>(sQ + (r * PC + (piece ^ (r & (PC < 16 ? PC - 1 : 15)))) * 16) = v;
    }
  };

  // Keys of a unit as the B operand, lane li holding token t0 + 16 n + li, and whether that
  // token is there.  They are under way while the unit before is computed, and the pages
  // of the unit after them, if it is of the same row, are looked up meanwhile.
  u32x4 k[NT][KS], k_next[NT][KS];
  bool there[NT], there_next[NT];
  int ids[NT];
  uint32_t k_off[KS];
#pragma unroll
  for (int x = 0; x < KS; ++x)
    k_off[x] = 32 * x + 8 * g < p.D ? li * (uint32_t)p.row_stride + 64 * x + 16 * g : kOut;
  auto look_up = [&](int bb, int tt, const Seq& q) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if constexpr (RUNS) {
        const int a = uni(tt * UT + wave * 16 * NT + 16 * n);
        const int t = a < q.lo ? q.lo : a;  // (a sequence of no tokens has no table entry to read)
        ids[n] = a + 16 > q.lo && a < q.hi
                     ? read_const(p.table, (int64_t)bb * p.width + uni(div_page(p.page, t))) : -1;
        continue;
      }
      const int t = tt * UT + wave * 16 * NT + 16 * n + li;
      const bool in = t >= q.lo && t < q.hi;
      ids[n] = in ? p.table[(int64_t)bb * p.width + div_page(p.page, t)] : -1;
    }
  };
  auto load = [&](int bb, int hh, int tt, const Seq& q) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if constexpr (RUNS) {
        const int a = uni(tt * UT + wave * 16 * NT + 16 * n);
        const bool page = (uint32_t)ids[n] < (uint32_t)p.n_pages;
        there_next[n] = page && a + li >= q.lo && a + li < q.hi;
        const int slot = a - (int)(uni(div_page(p.page, page ? a : 0)) * p.page.d);
        const auto r = rsrc_at(p.K + (page ? ids[n] * p.page_stride + slot * p.row_stride +
                                                 hh * p.head_stride : 0));
#pragma unroll
        for (int x = 0; x < KS; ++x)
          k_next[n][x] = __builtin_bit_cast(
              u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, there_next[n] ? k_off[x] : kOut, 0, 0));
        continue;
      }
      const int t = tt * UT + wave * 16 * NT + 16 * n + li;
      there_next[n] = (uint32_t)ids[n] < (uint32_t)p.n_pages;
      const int slot = t - (int)(div_page(p.page, there_next[n] ? t : 0) * p.page.d);
      const unsigned char* kp =
          p.K + ids[n] * p.page_stride + slot * p.row_stride + hh * p.head_stride;
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        const int d = 32 * x + 8 * g;
        k_next[n][x] = u32x4{0, 0, 0, 0};
        if (there_next[n] && d < p.D) k_next[n][x] = *reinterpret_cast<const u32x4*>(kp + d * 2);
      }
    }
  };
  look_up(b, tile, s);
  load(b, h, tile, s);
  if (left > 1 && tile + 1 < s.t1) look_up(b, tile + 1, s);

  int q_at[KS];  // where this lane's pieces of a row tile lie
#pragma unroll
  for (int x = 0; x < KS; ++x)
    q_at[x] = (li * PC + ((4 * x + g) ^ (li & (PC < 16 ? PC - 1 : 15)))) * 16;
  bool fresh = true;
  while (true) {
    const int rows = s.m * p.G;
    // the unit that follows
    int next_b = b, next_h = h, next_tile = tile + 1;
    Seq next_s = s;
    if (left > 1 && next_tile >= s.t1) {
      if (++next_h == p.Hkv) {
        next_h = 0;
        while (next_b + 1 < p.B) {
          next_s = read_seq<UT>(p, ++next_b);
          if (next_s.t1 > next_s.t0) break;
        }
      }
      next_tile = next_s.t0;
    }
    if (fresh) {
      const int tid = anew(threadIdx.x);
      __syncthreads();  // what the rows before needed has been read
      if (tid == 0) sOut = 0;
      if (rows <= chunk) stage(0, rows);
      __syncthreads();
      for (int r = tid; r < rows; r += kThreads) {
        const int i = div_page(p.group, r);
        const float l = p.lse[((int64_t)b * p.T + i) * p.Hq + h * p.G + (r - i * p.G)];
        const bool adds = fabsf(l) < INFINITY;
        sLse[r] = adds ? l * kLog2e : INFINITY;
        if (!adds) sOut = 1;  // every writer writes 1
      }
      for (int r = rows + tid; r < (rows + 15 & ~15); r += kThreads) sLse[r] = INFINITY;
      for (int i = tid; i < s.m; i += kThreads) {
        int seen = 0;
        for (int w = 0; w < kMaskWords; ++w) {
          const int valid = s.m - w * 64, upto = i + 1 - w * 64;
          const uint64_t some = valid >= 64 ? ~0ull : valid <= 0 ? 0ull : (1ull << valid) - 1;
          uint64_t bits = upto >= 64 ? ~0ull : upto <= 0 ? 0ull : (1ull << upto) - 1;
          if (p.mask) bits = w < p.words ? p.mask[b * p.mask_seq + (int64_t)i * p.words + w] : 0;
          sBits[i][w] = bits & some;
          seen += __popcll(bits & some);
        }
        const int low = p.window > 0 ? s.n + seen - p.window : 0;
        sLow[i] = low > 0 ? low : 0;
      }
      __syncthreads();
    }
    const int t0 = tile * UT + wave * 16 * NT;
    // the sums so far, for lane group g of the tiles g, g + 4, ..
    float old[(NT + 3) / 4];
#pragma unroll
    for (int n0 = 0; n0 < NT; n0 += 4) {
      const int t = t0 + 16 * (n0 + g) + li;
      old[n0 / 4] = n0 + g < NT && t < s.n && t < p.S
                        ? p.scores[b * p.s_seq + h * p.s_head + t] : 0.f;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      there[n] = there_next[n];
#pragma unroll
      for (int x = 0; x < KS; ++x) k[n][x] = k_next[n][x];
    }
    if (left > 1) {
      if (next_b != b || next_h != h) look_up(next_b, next_tile, next_s);
      load(next_b, next_h, next_tile, next_s);
      if (left > 2 && next_tile + 1 < next_s.t1) look_up(next_b, next_tile + 1, next_s);
    }
    float sum[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) sum[n] = 0.f;
    const bool edge = t0 + 16 * NT > s.n || (p.window > 0 && t0 < s.n + s.m - p.window) || sOut;
    for (int c0 = 0; c0 < rows; c0 += chunk) {
      const int n_rows = rows - c0 < chunk ? rows - c0 : chunk;
      if (rows > chunk) {
        __syncthreads();
        stage(c0, rows);
        __syncthreads();
      }
      // queries as the A operand: lane li holds row r + li of the chunk
      auto query = [&](int r, u32x4* q) {
#pragma unroll
        for (int x = 0; x < KS; ++x)
          q[x] = *reinterpret_cast<const u32x4*>(sQ + r * PC * 16 + q_at[x]);
        return *reinterpret_cast<const float4v*>(sLse + c0 + r + 4 * g);
      };
      auto score = [&](const u32x4* q, int n) {
        float4v c = {0, 0, 0, 0};
#pragma unroll
        for (int x = 0; x < KS; ++x) c = mma16<BF>(q[x], k[n][x], c);
        return c;
      };
      if (!edge) {
        for (int r = 0; r < n_rows; r += 16) {
          u32x4 q[KS];
          const float4v ls = query(r, q);
          float4v c[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) c[n] = score(q, n);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              sum[n] += __builtin_amdgcn_exp2f(fmaf(c[n][j], p.scale, -ls[j]));
        }
      } else {
        const int li = anew(lane & 15), g = anew(lane >> 4);
        for (int r = 0; r < n_rows; r += 16) {
          u32x4 q[KS];
          const float4v ls = query(r, q);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float4v c = score(q, n);
            const int t = t0 + 16 * n + li, at = t - s.n;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              bool ok = ls[j] < INFINITY;
              if (ok) {
                const int node = div_page(p.group, c0 + r + 4 * g + j);
                ok = at < 0 ? t >= sLow[node]
                            : at < kMaxNodes && (sBits[node][at >> 6] >> (at & 63) & 1);
              }
              const float w = __builtin_amdgcn_exp2f(fmaf(c[j], p.scale, -ls[j]));
              sum[n] += ok ? w : 0.f;
            }
          }
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) sum[n] = there[n] ? sum[n] : 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      sum[n] += __shfl_xor(sum[n], 16, kWave);
      sum[n] += __shfl_xor(sum[n], 32, kWave);
    }
    // lane group g writes the tiles g, g + 4, ..
#pragma unroll
    for (int n0 = 0; n0 < NT; n0 += 4) {
      float w = sum[n0];
#pragma unroll
      for (int n = 1; n < 4; ++n)
        if (n0 + n < NT) w = g == n ? sum[n0 + n] : w;
      const int t = t0 + 16 * (n0 + g) + li;
      if (n0 + g < NT && t < s.hi && t < p.S) {
        p.scores[b * p.s_seq + h * p.s_head + t] = t < s.n ? fmaf(p.decay, old[n0 / 4], w) : w;
      }
    }
    if (--left == 0) break;
    fresh = next_b != b || next_h != h;
    b = next_b;
    h = next_h;
    tile = next_tile;
    s = next_s;
  }
}

template <bool BF, int DV, int NT, bool RUNS>
hipError_t launch_nt(WeightsParams p, hipStream_t s) {
  constexpr int64_t UT = 16 * NT * kWaves;
  int64_t cap = (int64_t)p.width * p.page.d;
  if (cap > p.S) cap = p.S;
  const int64_t tiles = (cap + UT - 1) / UT, all = (int64_t)p.B * p.Hkv * tiles;
  if (all == 0) return hipSuccess;
  const int rows = (p.T * p.G + 15) / 16 * 16, most_rows = kQueryBytes / (DV * 2);
  p.chunk = rows < most_rows ? rows : most_rows;
  const int lds = p.chunk * DV * 2 + rows * 4;
  // What registers and LDS allow at once: with more, equal runs would be a full round and part
  // of another.  Measured (us, by registers alone / so), 16 sequences of 4096 .. 16384 tokens, 8 heads,
  // 176 rows, heads of 128 (two a CU instead of three) 159 / 130, 256 rows 333 / 287; 512 rows of heads
  // of 64 382 / 329.
  const int64_t by_lds = kCuLds / (lds + kFixedLds), by_registers = DV > 128 ? 2 : 3;
  const int64_t most = (by_lds < by_registers ? by_lds : by_registers) * device_cus();
  p.tiles = all <= 2 * most ? (int32_t)tiles : 0;
  if (lds > 48 * 1024) {
    static std::atomic<uint64_t> done{0};
    const hipError_t e =
        lds_limit_once(reinterpret_cast<const void*>(cache_weights_kernel<BF, DV, NT, RUNS>),
                       kQueryBytes + kMostRows * 4, done);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((cache_weights_kernel<BF, DV, NT, RUNS>),
                     dim3((uint32_t)(p.tiles || all < most ? all : most)), dim3(kThreads), lds, s, p);
  return hipGetLastError();
}

template <bool BF, bool RUNS>
hipError_t launch_weights(const WeightsParams& p, hipStream_t s) {
  return p.D <= 64    ? launch_nt<BF, 64, 2, RUNS>(p, s)
         : p.D <= 128 ? launch_nt<BF, 128, 2, RUNS>(p, s)
                      : launch_nt<BF, 256, 2, RUNS>(p, s);
}

}  // namespace

hipError_t launch_cache_weights(int dtype, const WeightsArgs& a, hipStream_t stream) {
  WeightsParams p{};
  const TreeArgs& t = a.tree;
  p.Q = static_cast<const unsigned char*>(t.Q);
  p.K = static_cast<const unsigned char*>(t.k_pages);
  p.q_seq = 2 * t.q_seq;
  p.q_tok = 2 * t.q_tok;
  p.q_head = 2 * t.q_head;
  p.page_stride = 2 * t.page_stride;
  p.row_stride = 2 * t.row_stride;
  p.head_stride = 2 * t.head_stride;
  p.table = t.page_table;
  p.lens = t.lens;
  p.nodes = t.nodes;
  p.mask = static_cast<const uint64_t*>(t.mask);
  p.mask_seq = t.mask_seq;
  p.lse = a.lse;
  p.scores = a.scores;
  p.s_seq = a.s_seq;
  p.s_head = a.s_head;
  p.page = fast_div(t.page_size);
  p.group = fast_div(t.Hq / t.Hkv);
  p.n_pages = (int32_t)t.n_pages;
  p.width = (int32_t)t.width;
  p.B = (int32_t)t.B;
  p.T = (int32_t)t.T;
  p.words = (int32_t)((t.T + 63) / 64);
  p.Hq = (int32_t)t.Hq;
  p.Hkv = (int32_t)t.Hkv;
  p.D = (int32_t)t.D;
  p.G = (int32_t)(t.Hq / t.Hkv);
  p.window = (int32_t)t.window;
  p.S = (int32_t)a.S;
  p.scale = t.scale_log2;
  p.decay = a.decay;
  const bool bf = dtype == TQ_BF16;
  if (t.page_size % 16 == 0)
    return bf ? launch_weights<true, true>(p, stream) : launch_weights<false, true>(p, stream);
  return bf ? launch_weights<true, false>(p, stream) : launch_weights<false, false>(p, stream);
}

}  // namespace tq
