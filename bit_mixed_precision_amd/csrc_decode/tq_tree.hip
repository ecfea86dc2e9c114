// Attention of the nodes of a drafted tree over a paged key-value cache, and the
// tree's ancestors as bits.
//
// A sequence b has n cached tokens and m nodes, whose keys and values lie in the slots
// n .. n + m - 1.  Node i sees the cached tokens and those nodes j whose bit is set
// in its mask (its ancestors and itself, as a rule):
//     out[b][i][h] = sum_t softmax_t(scale * q[b][i][h] . k[t][h / G]) v[t][h / G].
// One pass with a running maximum and sum in fp32 (base-2 exponents: the scale
// carries log2 e).
//
// The m * G queries that share a key-value head are the rows of one matrix product
// each with K and V; a row block of them and a run of tokens are a unit of work.

#include <atomic>
#include <type_traits>

#include "tq.h"
#include "tq_attn_dev.h"
#include "tq_common.h"
#include "tq_decode.h"
#include "tq_kernels.h"
#include "tq_mfma.h"

namespace tq {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kTreeThreads = 256;
constexpr int kTreeWaves = kTreeThreads / kWave;
constexpr int kTeamRows = 32;     // rows of a wave: columns of the matrix instruction
constexpr int kMaskWords = 4;     // of 64 nodes

struct TreeParams {
  const unsigned char* Q;
  const unsigned char* K;
  const unsigned char* V;
  int64_t q_seq, q_tok, q_head;                  // bytes
  int64_t page_stride, row_stride, head_stride;  // bytes
  const int32_t* table;
  const int32_t* lens;
  const int32_t* nodes;
  const uint64_t* mask;
  int64_t mask_seq;  // words
  unsigned char* Out;
  float* lse;
  float* partial;  // [workgroups][2][part_floats]
  int2* owner;     // [workgroups]: the row block it began and left unfinished (or -1), its last workgroup
  FastDiv page, group;
  int32_t n_pages, width, B, T, words, Hq, Hkv, D, G, window;
  int32_t direct;  // one workgroup per row block: nothing is split
  float scale;     // not negative
  uint32_t flip;   // sign bit where the caller's scale is negative
};

// Floats of one partial result: rows x D numbers, maxima, sums.
__host__ __device__ __forceinline__ int64_t part_floats(int rows, int D) {
  return (int64_t)rows * (D + 2);
}

template <bool BF>
__device__ __forceinline__ f32x16 mma32(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8, a),
                                                   __builtin_bit_cast(bf8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, a),
                                                  __builtin_bit_cast(half8, b), c, 0, 0, 0);
}

// Two floats as two 16-bit numbers, rounded to nearest.
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  using half2 = std::conditional_t<BF, bf2, half2v>;
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((float2v{x, y}), half2));
}

__device__ __forceinline__ int64_t shfl64(int64_t v, int src) {
  const int lo = __shfl((int)v, src, kWave), hi = __shfl((int)(v >> 32), src, kWave);
  return ((int64_t)hi << 32) | (uint32_t)lo;
}

// The low n bits, n of any value.
__device__ __forceinline__ uint32_t below(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1;
}

// The halves of x that are finite numbers, 0 in the place of the others.
template <bool BF>
__device__ __forceinline__ uint32_t finite_of(uint32_t x) {
  constexpr uint32_t exps = BF ? 0x7f80u : 0x7c00u;
  return ((x & exps) != exps ? x & 0xffffu : 0u) | ((x >> 16 & exps) != exps ? x & 0xffff0000u : 0u);
}
template <bool BF>
__device__ __forceinline__ float from16(uint32_t bits) {
  if constexpr (BF) return __builtin_bit_cast(float, bits << 16);
  else return h2f((uint16_t)bits);
}

// A sequence: n cached tokens, m nodes, tokens [lo, hi) that any node may see, the
// tiles [t0, t1) of UT tokens that hold them, and blocks of ROWS rows.
struct Seq {
  int n, m, lo, hi, t0, t1, blocks;
};
template <int UT, int ROWS>
__device__ __forceinline__ Seq seq_of(const TreeParams& p, int len, int nodes) {
  Seq s;
  const int cap = p.width * (int)p.page.d;
  s.n = len < 0 ? 0 : len < cap ? len : cap;
  s.m = nodes < 0 ? 0 : nodes < p.T ? nodes : p.T;
  s.hi = s.n + s.m < cap ? s.n + s.m : cap;
  s.lo = p.window > 0 && s.n > p.window ? s.n - p.window : 0;
  s.t0 = s.lo / UT;
  s.t1 = s.m > 0 ? (s.hi + UT - 1) / UT : s.t0;
  s.blocks = (s.m * p.G + ROWS - 1) / ROWS;
  return s;
}
template <int UT, int ROWS>
__device__ __forceinline__ Seq read_seq(const TreeParams& p, int b) {
  return seq_of<UT, ROWS>(p, read_const(p.lens, b), p.nodes ? read_const(p.nodes, b) : p.T);
}

// A unit: row block r, sequence b, key-value head h, tile.
struct Unit {
  int r, b, h, tile;
  Seq s;
};

// Weights are 2^(x - m + kShift): in fp16 the smaller ones then keep all their bits.
template <bool BF>
constexpr float kShift = BF ? 0.f : 14.f;

// Divides by the sum and writes numbers d .. d + 3 of one query, and its lse.
template <bool BF>
__device__ __forceinline__ void store_row(const TreeParams& p, int64_t at, int d, float m,
                                          float sum, float inv, float4v v) {
  u32x2 u;
  u[0] = pack2<BF>(v[0] * inv, v[1] * inv);
  u[1] = pack2<BF>(v[2] * inv, v[3] * inv);
  *reinterpret_cast<u32x2*>(p.Out + (at * p.D + d) * 2) = u;
  if (p.lse && d == 0) p.lse[at] = (m + __builtin_amdgcn_logf(sum) - kShift<BF>) / kLog2e;
}

// DP: the head dimension rounded up to what the kernel is built for.
// TEAM: waves that share a tile of tokens, each with 32 rows of its own; a workgroup
// has 4 / TEAM teams, which take turns at the tokens of the same rows.
template <int DP, int TEAM>
struct Shape {
  static constexpr int KS = DP / 16;               // steps of a score
  static constexpr int NE = DP / 32;               // blocks of 32 numbers of the output
  static constexpr int PC = DP / 8;                // 16-byte pieces of a row
  static constexpr int TT = TEAM == 4 ? 64 : 32;   // tokens of a tile
  static constexpr int SUB = TT / 32;
  static constexpr int TEAMS = kTreeWaves / TEAM;
  static constexpr int UT = TT * TEAMS;            // tokens of a unit
  static constexpr int ROWS = kTeamRows * TEAM;    // rows of a block
  static constexpr int PER = TT * PC / (kWave * TEAM);  // pieces of K (and of V) a thread loads
  static constexpr int TILE = TT * DP * 2;         // bytes of K (and of V)
  static constexpr int PAD = DP + 4;               // floats of a row of sums in LDS
  static constexpr int TILES = 2 * TILE * TEAMS;
  static constexpr int JOIN = TEAM == 4 ? 0 : kTreeWaves * kTeamRows * PAD * 4;
  static constexpr int LDS = TILES > JOIN ? TILES : JOIN;
  // A weight as two 16-bit numbers where memory sets the pace, as one with many rows,
  // where each costs a matrix product: rounding it to nearest then adds as much
  // error to the output as the output's own rounding.
  static constexpr bool SPLIT = TEAM == 1;
  // Where piece c of row t lies in its row: rows whose pieces would share banks are
  // turned against each other, for the reads of K (16 rows, one piece) and of V (4
  // rows, 4 pieces).
  __device__ static __forceinline__ int k_at(int t, int c) {
    if constexpr (PC % 16 == 0) return c ^ (t & 15);
    else if constexpr (PC % 8 == 0) return c ^ ((t >> 1) & 7);
    else return c ^ ((t >> 2) & 3);
  }
  __device__ static __forceinline__ int v_at(int t, int c) {
    if constexpr (PC % 16 == 0) return c ^ ((t & 3) << 2);
    else if constexpr (PC % 8 == 0) return c ^ (((t >> 1) & 1) << 2);
    else return c;
  }
};

template <bool BF, int DP, int TEAM>
__global__ __launch_bounds__(kTreeThreads, DP > 128 ? 1 : 2) void tree_attention_kernel(
    TreeParams p) {
  using S = Shape<DP, TEAM>;
  constexpr int KS = S::KS, NE = S::NE, PC = S::PC, TT = S::TT, SUB = S::SUB, UT = S::UT;
  constexpr int ROWS = S::ROWS, PER = S::PER;
  extern __shared__ __attribute__((aligned(16))) unsigned char sTiles[];
  // what a row sees of the nodes, and its first cached token
  __shared__ uint64_t sBits[kTreeWaves][kTeamRows][kMaskWords];
  __shared__ int sLow[kTreeWaves][kTeamRows];
  __shared__ float sM[kTreeWaves][kTeamRows], sL[kTreeWaves][kTeamRows];
  __shared__ int sOdd[S::TEAMS];  // values that are no finite numbers were left out of a tile

  const int tid = threadIdx.x;
  const int wave = uni(tid >> 6), lane = tid & 63, col = lane & 31, half = lane >> 5;
  const int team = wave / TEAM;
  const int tl = TEAM == 4 ? tid : lane;  // this thread in its team
  unsigned char* const sK = sTiles + team * 2 * S::TILE;
  unsigned char* const sV = sK + S::TILE;

  // this workgroup's run of units
  Unit cur{};
  uint32_t left = 0, run_end = 0;
  Cut cut(0, 1);
  if (p.direct) {
    const int per_block = p.B * p.Hkv;
    cur.r = blockIdx.x / per_block;
    const int rest = blockIdx.x - cur.r * per_block;
    cur.b = rest / p.Hkv;
    cur.h = rest - cur.b * p.Hkv;
    cur.s = read_seq<UT, ROWS>(p, cur.b);
    cur.tile = cur.s.t0;
    left = cur.r < cur.s.blocks ? cur.s.t1 - cur.s.t0 : 0;
  } else {
    const int per = (p.B + kWave - 1) / kWave;
    auto tiles_of = [&](int b, bool in, int r) -> uint32_t {  // of a head, 0 without block r
      const Seq s = read_seq<UT, ROWS>(p, b < p.B ? b : p.B - 1);
      return in && b < p.B && s.blocks > r ? s.t1 - s.t0 : 0;
    };
    uint32_t all = 0, most = 0;  // tiles x blocks, blocks
    for (int i = 0; i < per; ++i) {
      const int b = lane * per + i;
      const Seq s = read_seq<UT, ROWS>(p, b < p.B ? b : p.B - 1);
      if (b < p.B) {
        all += (uint32_t)(s.t1 - s.t0) * s.blocks;
        most = (uint32_t)s.blocks > most ? s.blocks : most;
      }
    }
    all = uni((int)__shfl(scan_wave(all, lane), 63, kWave));
    cut = Cut(all * p.Hkv, gridDim.x);
    if (blockIdx.x < cut.parts) {
      uint32_t at = cut.start(blockIdx.x);
      run_end = cut.start(blockIdx.x + 1);
      left = run_end - at;
      // the row block, the lane that looks after the sequence, the sequence
      const int lanes = (p.B + per - 1) / per;
      uint32_t mine = 0, inc = 0;
      for (cur.r = 0;; ++cur.r) {
        mine = 0;
        for (int i = 0; i < per; ++i) mine += tiles_of(lane * per + i, true, cur.r);
        inc = scan_wave(mine, lane);
        const uint32_t total = uni((int)__shfl(inc, 63, kWave)) * (uint32_t)p.Hkv;
        // (the bound holds whatever happens to the lengths meanwhile)
        if (at < total || cur.r >= p.T * p.G / ROWS) break;
        at -= total;
      }
      const uint64_t has = __ballot(at < inc * p.Hkv && lane < lanes);
      const int src = has ? __builtin_ctzll(has) : 0;
      at -= (uint32_t)__builtin_amdgcn_readlane((int)(inc - mine), src) * p.Hkv;
      cur.b = src * per;
      for (int i = 0; per > 1 && i < per; i += kWave) {
        const uint32_t n = tiles_of(src * per + i + lane, i + lane < per, cur.r);
        const uint32_t run = scan_wave(n, lane);
        const uint64_t hit = __ballot(at < run * p.Hkv);
        if (hit) {
          const int k = __builtin_ctzll(hit);
          cur.b = src * per + i + k;
          at -= (uint32_t)__builtin_amdgcn_readlane((int)(run - n), k) * p.Hkv;
          break;
        }
        at -= (uint32_t)__builtin_amdgcn_readlane((int)run, kWave - 1) * p.Hkv;
      }
      if (cur.b >= p.B) cur.b = p.B - 1;
      cur.s = read_seq<UT, ROWS>(p, cur.b);
      const uint32_t n = cur.s.t1 > cur.s.t0 ? cur.s.t1 - cur.s.t0 : 1;
      cur.h = at / n;
      cur.tile = cur.s.t0 + at % n;
      if (cur.h >= p.Hkv) cur.h = p.Hkv - 1;
    }
  }

  auto advance = [&](Unit& c) {  // only where another unit follows
    if (++c.tile < c.s.t1) return;
    if (++c.h == p.Hkv) {
      c.h = 0;
      while (true) {
        if (++c.b == p.B) {
          c.b = 0;
          if (++c.r > p.T * p.G / ROWS) break;  // past the end (the lengths have changed)
        }
        c.s = read_seq<UT, ROWS>(p, c.b);
        if (c.s.t1 > c.s.t0 && c.s.blocks > c.r) break;
      }
    }
    c.tile = c.s.t0;
  };

  // This lane's token of the team's tile: the page it lies in, as the table has it.
  auto first_token = [&](const Unit& c) { return c.tile * UT + team * TT; };
  auto page_id = [&](const Unit& c) {
    const int t = first_token(c) + (lane & (TT - 1));
    const bool in = t >= c.s.lo && t < c.s.hi;
    return p.table[(int64_t)c.b * p.width + div_page(p.page, in ? t : c.s.lo)];
  };
  u32x4 kreg[PER], vreg[PER];
  uint64_t present_next = 0;
  auto load = [&](const Unit& c, int id) {
    const int t = first_token(c) + (lane & (TT - 1));
    const bool ok = t >= c.s.lo && t < c.s.hi && (uint32_t)id < (uint32_t)p.n_pages;
    const int slot = t - (int)(div_page(p.page, ok ? t : 0) * p.page.d);
    const int64_t off = ok ? id * p.page_stride + slot * p.row_stride + c.h * p.head_stride : -1;
    present_next = __ballot(ok);
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int x = u * kWave * TEAM + tl, row = x / PC, piece = x - row * PC;
      const int64_t o = shfl64(off, row);
      kreg[u] = vreg[u] = u32x4{0, 0, 0, 0};
      if (o >= 0 && piece * 8 < p.D) {
        kreg[u] = *reinterpret_cast<const u32x4*>(p.K + o + piece * 16);
        vreg[u] = *reinterpret_cast<const u32x4*>(p.V + o + piece * 16);
      }
    }
  };
  // Whether some row may not see some present token of the tile.
  auto edge = [&](const Unit& c) {
    const int a = first_token(c);
    return a + TT > c.s.n || (p.window > 0 && a < c.s.n + c.s.m - p.window);
  };
  // Of such a tile only the finite values: a weight of zero times infinity would reach
  // rows that do not see the token.  close_row adds what is left out here.
  auto stage = [&](bool at_edge) {
    if (at_edge) {
      bool odd = false;
#pragma unroll
      for (int u = 0; u < PER; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t f = finite_of<BF>(vreg[u][i]);
          odd |= f != vreg[u][i];
          vreg[u][i] = f;
        }
      if (odd) sOdd[team] = 1;  // every writer writes 1
    }
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int x = u * kWave * TEAM + tl, row = x / PC, piece = x - row * PC;
      *reinterpret_cast<u32x4*>(sK + row * DP * 2 + S::k_at(row, piece) * 16) = kreg[u];
      *reinterpret_cast<u32x4*>(sV + row * DP * 2 + S::v_at(row, piece) * 16) = vreg[u];
    }
  };
  auto team_sync = [&] {
    if constexpr (TEAM == 4) __syncthreads();
    else __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  };

  u32x4 q[KS];
  f32x16 acc[NE];
  float m = -INFINITY, l = 0.f;
  int row0 = 0;  // of this wave
  auto open_row = [&](const Unit& c) {
    row0 = c.r * ROWS + (TEAM == 4 ? wave * kTeamRows : 0);
    const int row = row0 + col;
    const bool real = row < c.s.m * p.G;
    const int i = real ? div_page(p.group, row) : 0, g = real ? row - i * p.G : 0;
    const unsigned char* qp = p.Q + c.b * p.q_seq + i * p.q_tok + (int64_t)(c.h * p.G + g) * p.q_head;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const int d = k * 16 + half * 8;
      q[k] = u32x4{0, 0, 0, 0};
      if (real && d < p.D) q[k] = *reinterpret_cast<const u32x4*>(qp + d * 2);
    }
    int seen = 0;
    for (int w = 0; w < kMaskWords; ++w) {
      const int valid = c.s.m - w * 64;  // nodes of this word
      const uint64_t some = valid >= 64 ? ~0ull : valid <= 0 ? 0ull : (1ull << valid) - 1;
      uint64_t bits = 0;
      if (real && w < p.words) {
        if (p.mask) {
          bits = p.mask[c.b * p.mask_seq + (int64_t)i * p.words + w];
        } else {
          const int upto = i + 1 - w * 64;
          bits = upto >= 64 ? ~0ull : upto <= 0 ? 0ull : (1ull << upto) - 1;
        }
      }
      bits &= some;
      seen += __popcll(bits);
      if (half == 0) sBits[wave][col][w] = bits;
    }
    const int low = p.window > 0 ? c.s.n + seen - p.window : 0;
    if (half == 0) sLow[wave][col] = low > 0 ? low : 0;
#pragma unroll
    for (int e = 0; e < NE; ++e)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[e][r] = 0.f;
    m = -INFINITY;
    l = 0.f;
  };
  // Tokens a .. a + 31 that this lane's row sees, one bit each.
  auto sees = [&](const Unit& c, int a, uint32_t present) {
    const uint32_t cached = below(c.s.n - a) & ~below(sLow[wave][col] - a);
    const int j = a - c.s.n;  // the node of bit 0
    uint32_t drafted = 0;
    if (j > -32) {
      const int w = j >> 6, sh = j & 63;  // w = -1 where j < 0
      const uint64_t lo = w >= 0 && w < kMaskWords ? sBits[wave][col][w] : 0;
      const uint64_t hi = w + 1 >= 0 && w + 1 < kMaskWords ? sBits[wave][col][w + 1] : 0;
      drafted = (uint32_t)(lo >> sh) | (sh > 32 ? (uint32_t)(hi << (64 - sh)) : 0u);
    }
    return present & (cached | drafted);
  };
  // O^T += V^T P^T, from the A operands that `turn` makes of V's
  auto v_operand = [&](int e, int s, int u) {
    const int i = lane & 15;
    const int t = 32 * s + 16 * u + 4 * half + (i >> 2);
    const int piece = 4 * e + 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
    typedef __attribute__((address_space(3))) s16x4* lds4;
    const unsigned char* a = sV + t * DP * 2 + S::v_at(t, piece) * 16 + (i & 1) * 8;
    const unsigned char* b = sV + (t + 8) * DP * 2 + S::v_at(t + 8, piece) * 16 + (i & 1) * 8;
    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)a);
    const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)b);
    const u32x2 xu = __builtin_bit_cast(u32x2, x), yu = __builtin_bit_cast(u32x2, y);
    return u32x4{xu[0], xu[1], yu[0], yu[1]};
  };

  // Slots of the workspace: the end of a row that began before this run, the start of
  // one that goes on after it.
  auto part_of = [&](int which) {
    return p.partial + (2 * (int64_t)blockIdx.x + which) * part_floats(ROWS, p.D);
  };
  auto query_of = [&](const Unit& c, int row) {  // its place in [B][T][Hq]
    const int i = div_page(p.group, row), g = row - i * p.G;
    return ((int64_t)c.b * p.T + i) * p.Hq + c.h * p.G + g;
  };
  // The infinite values and NaN that stage has left out, of the tiles from `first` to
  // c's, for the rows that see their tokens.
  auto add_odd = [&](const Unit& c, int first) {
    Unit x = c;
    for (x.tile = first; x.tile <= c.tile; ++x.tile) {
      if (!edge(x)) continue;
      for (int k = 0; k < TT; ++k) {
        const int t = first_token(x) + k;
        if (t < c.s.lo || t >= c.s.hi) continue;
        const int pg = div_page(p.page, t);
        const int id = p.table[(int64_t)c.b * p.width + pg];
        if ((uint32_t)id >= (uint32_t)p.n_pages || !(sees(c, t, 1u) & 1)) continue;
        const unsigned char* v = p.V + id * p.page_stride + (t - pg * (int)p.page.d) * p.row_stride +
                                 c.h * p.head_stride;
#pragma unroll
        for (int e = 0; e < NE; ++e)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int d = 32 * e + 8 * r + 4 * half;
            if (d >= p.D) continue;
            const u32x2 u = *reinterpret_cast<const u32x2*>(v + d * 2);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float f = from16<BF>(u[i / 2] >> (16 * (i & 1)) & 0xffffu);
              if (!(fabsf(f) < INFINITY)) acc[e][4 * r + i] += f;
            }
          }
      }
    }
  };
  auto close_row = [&](const Unit& c, int first_tile, bool begins, bool ends) {
    if (sOdd[team]) add_odd(c, first_tile);
    const bool whole = begins && ends;
    float* const part = p.direct ? nullptr : part_of(begins ? 1 : 0);
    const int rows = c.s.m * p.G;
    const float sum = l + __shfl_xor(l, 32, kWave);
    if constexpr (TEAM == 4) {
      const int row = row0 + col;
      if (row < rows) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const float mm = m == -INFINITY ? -INFINITY : m * p.scale;
        const int64_t at = query_of(c, row);
        const int in_block = row - c.r * ROWS;
#pragma unroll
        for (int e = 0; e < NE; ++e)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int d = 32 * e + 8 * k + 4 * half;
            const float4v v = {acc[e][4 * k], acc[e][4 * k + 1], acc[e][4 * k + 2], acc[e][4 * k + 3]};
            if (d < p.D) {
              if (whole) store_row<BF>(p, at, d, mm, sum, inv, v);
              else *reinterpret_cast<float4v*>(part + in_block * p.D + d) = v;
            }
          }
        if (!whole && half == 0) {
          part[ROWS * p.D + in_block] = mm;
          part[ROWS * p.D + ROWS + in_block] = sum;
        }
      }
    } else {
      // the waves' sums meet in LDS
      float* const sO = reinterpret_cast<float*>(sTiles);
      __syncthreads();  // all tiles have been read
#pragma unroll
      for (int e = 0; e < NE; ++e)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<float4v*>(sO + (wave * kTeamRows + col) * S::PAD + 32 * e + 8 * k +
                                      4 * half) =
              float4v{acc[e][4 * k], acc[e][4 * k + 1], acc[e][4 * k + 2], acc[e][4 * k + 3]};
      if (half == 0) {
        sM[wave][col] = m == -INFINITY ? -INFINITY : m * p.scale;
        sL[wave][col] = sum;
      }
      __syncthreads();
      const int first = c.r * ROWS, n = rows - first < ROWS ? rows - first : ROWS;
      const int units = p.D / 4;
      for (int j = tid; j < n * units; j += kTreeThreads) {
        const int r = j / units, d = (j - r * units) * 4;
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kTreeWaves; ++w) mm = fmaxf(mm, sM[w][r]);
        const float base = mm == -INFINITY ? 0.f : mm;
        float total = 0.f;
        float4v v = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kTreeWaves; ++w) {
          const float f = __builtin_amdgcn_exp2f(sM[w][r] - base);
          total += f * sL[w][r];
          const float4v x = *reinterpret_cast<const float4v*>(sO + (w * kTeamRows + r) * S::PAD + d);
          // a wave without weight adds nothing, also where it has met NaN
          if (sL[w][r] != 0.f) v += f * x;
        }
        if (whole) {
          store_row<BF>(p, query_of(c, first + r), d, mm, total, total == 0.f ? 0.f : 1.f / total, v);
        } else {
          *reinterpret_cast<float4v*>(part + r * p.D + d) = v;
          if (d == 0) {
            part[ROWS * p.D + r] = mm;
            part[ROWS * p.D + ROWS + r] = total;
          }
        }
      }
      __syncthreads();  // the tiles may be written again
    }
  };

  int owned = -1, last = 0;
  if (tid < S::TEAMS) sOdd[tid] = 0;
  __syncthreads();
  if (left > 0) {
    int first_tile = cur.tile;
    Unit next = cur;
    open_row(cur);
    load(cur, page_id(cur));
    int id_next = 0;
    if (left > 1) {
      advance(next);
      id_next = page_id(next);
    }
    stage(edge(cur));
    uint64_t present = present_next;
    if (left > 1) load(next, id_next);
    team_sync();
    while (true) {
      const bool more = left > 1;
      const int a0 = first_token(cur);
      f32x16 s[SUB];
#pragma unroll
      for (int x = 0; x < SUB; ++x) {
#pragma unroll
        for (int r = 0; r < 16; ++r) s[x][r] = 0.f;
        const int t = 32 * x + col;
#pragma unroll
        for (int k = 0; k < KS; ++k)
          s[x] = mma32<BF>(*reinterpret_cast<const u32x4*>(sK + t * DP * 2 + S::k_at(t, 2 * k + half) * 16),
                           q[k], s[x]);
      }
      if (p.flip)
#pragma unroll
        for (int x = 0; x < SUB; ++x)
#pragma unroll
          for (int r = 0; r < 16; ++r) s[x][r] = -s[x][r];
      constexpr uint64_t kFull = TT == 64 ? ~0ull : 0xffffffffull;
      const uint64_t there = TT == 64 ? present : present & kFull;
      const bool masks = there != kFull || a0 + TT > cur.s.n ||
                         (p.window > 0 && a0 < cur.s.n + cur.s.m - p.window);
      if (masks) {
#pragma unroll
        for (int x = 0; x < SUB; ++x) {
          const uint32_t see = sees(cur, a0 + 32 * x, (uint32_t)(there >> (32 * x))) >> (4 * half);
#pragma unroll
          for (int r = 0; r < 16; ++r)
            s[x][r] = see >> (8 * (r >> 2) + (r & 3)) & 1 ? s[x][r] : -INFINITY;
        }
      }
      float top = s[0][0];
#pragma unroll
      for (int x = 0; x < SUB; ++x)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, s[x][r]);
      top = fmaxf(top, __shfl_xor(top, 32, kWave));
      if (!__all(top <= m)) {
        const float mn = fmaxf(m, top);
        const float alpha = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - mn) * p.scale);
        m = mn;
        l *= alpha;
#pragma unroll
        for (int e = 0; e < NE; ++e) acc[e] *= alpha;
      }
      const float base = (m == -INFINITY ? 0.f : m * p.scale) - kShift<BF>;
      u32x4 hi[SUB][2], lo[SUB][2];
#pragma unroll
      for (int x = 0; x < SUB; ++x)
#pragma unroll
        for (int r = 0; r < 16; r += 2) {
          const float w0 = __builtin_amdgcn_exp2f(fmaf(s[x][r], p.scale, -base));
          const float w1 = __builtin_amdgcn_exp2f(fmaf(s[x][r + 1], p.scale, -base));
          l += w0 + w1;
          uint32_t h2, l2 = 0;
          if constexpr (S::SPLIT) split2<BF>(w0, w1, h2, l2);
          else h2 = pack2<BF>(w0, w1);
          hi[x][r / 8][r % 8 / 2] = h2;
          lo[x][r / 8][r % 8 / 2] = l2;
        }
#pragma unroll
      for (int e = 0; e < NE; ++e)
#pragma unroll
        for (int x = 0; x < SUB; ++x)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const u32x4 v = v_operand(e, x, u);
            acc[e] = mma32<BF>(v, hi[x][u], acc[e]);
            if constexpr (S::SPLIT) acc[e] = mma32<BF>(v, lo[x][u], acc[e]);
          }
      --left;
      const bool ends = cur.tile + 1 == cur.s.t1;
      if (ends || !more) {
        const bool begins = first_tile == cur.s.t0;
        close_row(cur, first_tile, begins, ends);
        if (begins && !ends) {  // goes on in the following workgroups
          owned = (cur.r * p.B + cur.b) * p.Hkv + cur.h;
          last = (int)cut.part_of(run_end - left - 1 + (cur.s.t1 - cur.tile - 1));
        }
      }
      if (!more) break;
      team_sync();  // the tile has been read
      stage(edge(next));
      present = present_next;
      cur = next;
      if (ends) {
        first_tile = cur.tile;
        open_row(cur);
      }
      if (left > 1) {
        advance(next);
        load(next, page_id(next));
      }
      team_sync();
    }
  }
  if (!p.direct && tid == 0) p.owner[blockIdx.x] = make_int2(owned, last);

  // rows of nodes that are not there: zeros and -inf; looked for 64 at a time
  const int64_t all = (int64_t)p.B * p.T;
  for (int64_t x0 = blockIdx.x; x0 < all; x0 += (int64_t)gridDim.x * kWave) {
    const int64_t x = x0 + (int64_t)gridDim.x * lane;
    const int64_t xb = (x < all ? x : x0) / p.T;
    const int nodes = p.nodes ? p.nodes[xb] : p.T;
    for (uint64_t none = __ballot(x < all && x - xb * p.T >= nodes); none; none &= none - 1) {
      const int64_t at = (x0 + (int64_t)gridDim.x * __builtin_ctzll(none)) * p.Hq;
      u32x4* o = reinterpret_cast<u32x4*>(p.Out + at * p.D * 2);
      for (int i = tid; i < p.Hq * p.D / 8; i += kTreeThreads) o[i] = u32x4{0, 0, 0, 0};
      if (p.lse)
        for (int i = tid; i < p.Hq; i += kTreeThreads) p.lse[at + i] = -INFINITY;
    }
  }
}

// Joins the partial results of the row blocks that span workgroups: one workgroup for
// RPW rows of the block that workgroup blockIdx.x began and left unfinished, a wave's
// lanes over the numbers of a row and, as far as they reach, over its parts.
template <bool BF, int ROWS>
__global__ __launch_bounds__(kTreeThreads) void tree_join_kernel(TreeParams p) {
  __shared__ float sAcc[kTreeWaves][256], sMax[kTreeWaves], sSum[kTreeWaves];
  const int2 own = p.owner[blockIdx.x];
  if (own.x < 0) return;
  const int h = own.x % p.Hkv, rest = own.x / p.Hkv, b = rest % p.B, r = rest / p.B;
  const int nodes = p.nodes ? p.nodes[b] : p.T;
  const int m = nodes < p.T ? nodes : p.T;
  const int row = r * ROWS + blockIdx.y;
  if (row >= m * p.G) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
  const int64_t size = part_floats(ROWS, p.D);
  const int n = own.y - (int)blockIdx.x + 1;
  // part 0 is this workgroup's second slot, the others the first slots that follow
  auto part = [&](int k) {
    return p.partial + (2 * ((int64_t)blockIdx.x + k) + (k == 0 ? 1 : 0)) * size;
  };
  const int at_m = ROWS * p.D + blockIdx.y, at_l = at_m + ROWS;
  float mm = -INFINITY;
  for (int k = tid; k < n; k += kTreeThreads) mm = fmaxf(mm, part(k)[at_m]);
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) mm = fmaxf(mm, __shfl_xor(mm, off, kWave));
  if (lane == 0) sMax[wave] = mm;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kTreeWaves; ++w) mm = fmaxf(mm, sMax[w]);
  const float base = mm == -INFINITY ? 0.f : mm;
  float sum = 0.f;
  float4v v = {0, 0, 0, 0};
  for (int k = wave; k < n; k += kTreeWaves) {
    const float* o = part(k);
    const float f = __builtin_amdgcn_exp2f(o[at_m] - base), lk = o[at_l];
    sum += f * lk;
    if (lane * 4 < p.D) {
      const float4v x = *reinterpret_cast<const float4v*>(o + (int64_t)blockIdx.y * p.D + lane * 4);
      if (lk != 0.f) v += f * x;
    }
  }
  *reinterpret_cast<float4v*>(&sAcc[wave][lane * 4]) = v;
  if (lane == 0) sSum[wave] = sum;
  __syncthreads();
  if (wave != 0 || lane * 4 >= p.D) return;
  float total = 0.f;
  float4v t = {0, 0, 0, 0};
#pragma unroll
  for (int w = 0; w < kTreeWaves; ++w) {
    total += sSum[w];
    t += *reinterpret_cast<const float4v*>(&sAcc[w][lane * 4]);
  }
  const int i = div_page(p.group, row), g = row - i * p.G;
  store_row<BF>(p, ((int64_t)b * p.T + i) * p.Hq + h * p.G + g, lane * 4, mm, total,
                total == 0.f ? 0.f : 1.f / total, t);
}

// The path from the root to every node: bit j of word w of node i is set where node
// 64 w + j is i or one of the nodes above it.  One workgroup per tree; after k rounds
// a node has seen 2^k nodes of its path and points to the one above them.
__global__ __launch_bounds__(kTreeThreads) void tree_mask_kernel(const int32_t* parents, int T,
                                                                 int words, uint64_t* mask,
                                                                 int32_t* depth) {
  __shared__ uint64_t sSeen[2][kTreeThreads][kMaskWords];
  __shared__ int sUp[2][kTreeThreads];
  const int i = threadIdx.x;
  const int64_t tree = blockIdx.x;
  int up = -1;
  uint64_t seen[kMaskWords];
#pragma unroll
  for (int w = 0; w < kMaskWords; ++w) seen[w] = i >> 6 == w ? 1ull << (i & 63) : 0;
  if (i < T) {
    up = parents[tree * T + i];
    up = up >= 0 && up < i ? up : -1;
  }
  int from = 0;
  for (int reach = 1; reach < T; reach <<= 1, from ^= 1) {
#pragma unroll
    for (int w = 0; w < kMaskWords; ++w) sSeen[from][i][w] = seen[w];
    sUp[from][i] = up;
    __syncthreads();
    if (up >= 0) {
#pragma unroll
      for (int w = 0; w < kMaskWords; ++w) seen[w] |= sSeen[from][up][w];
      up = sUp[from][up];
    }
  }
  if (i >= T) return;
  int n = 0;
#pragma unroll
  for (int w = 0; w < kMaskWords; ++w) {
    n += __popcll(seen[w]);
    if (w < words) mask[(tree * T + i) * words + w] = seen[w];
  }
  if (depth) depth[tree * T + i] = n - 1;
}

constexpr int64_t kMostTreeBlocks = 1024;

struct TreeGrid {
  int64_t blocks;
  bool direct, wide;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

TreeGrid tree_grid(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t capacity) {
  const int64_t rows = T * (Hq / Hkv);
  const bool wide = rows > kTeamRows;
  const int64_t block_rows = wide ? 4 * kTeamRows : kTeamRows, unit = wide ? 64 : 128;
  const int64_t blocks = B * Hkv * ceil_div(rows, block_rows);
  const int64_t tiles = ceil_div(capacity, unit);
  if (tiles <= 4) return {blocks, true, wide};
  int64_t grid = device_cus() * (D > 128 ? 1 : 2);
  if (grid > kMostTreeBlocks) grid = kMostTreeBlocks;
  return {blocks * tiles < grid ? blocks * tiles : grid, false, wide};
}

template <bool BF, int DP, int TEAM>
hipError_t launch_tree(const TreeParams& p, int64_t grid, hipStream_t s) {
  using Sh = Shape<DP, TEAM>;
  const auto fn = tree_attention_kernel<BF, DP, TEAM>;
  if (Sh::LDS > 48 * 1024) {
    static std::atomic<uint64_t> done{0};
    const hipError_t e = lds_limit_once(reinterpret_cast<const void*>(fn), Sh::LDS, done);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(fn, dim3((uint32_t)grid), dim3(kTreeThreads), Sh::LDS, s, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.direct) return e;
  hipLaunchKernelGGL((tree_join_kernel<BF, Sh::ROWS>), dim3((uint32_t)grid, Sh::ROWS),
                     dim3(kTreeThreads), 0, s, p);
  return hipGetLastError();
}

template <bool BF, int TEAM>
hipError_t launch_tree_d(const TreeParams& p, int64_t grid, hipStream_t s) {
  return p.D <= 64    ? launch_tree<BF, 64, TEAM>(p, grid, s)
         : p.D <= 96  ? launch_tree<BF, 96, TEAM>(p, grid, s)
         : p.D <= 128 ? launch_tree<BF, 128, TEAM>(p, grid, s)
         : p.D <= 192 ? launch_tree<BF, 192, TEAM>(p, grid, s)
                      : launch_tree<BF, 256, TEAM>(p, grid, s);
}

}  // namespace

int64_t tree_workspace_bytes(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                             int64_t capacity) {
  const TreeGrid g = tree_grid(B, T, Hq, Hkv, D, capacity);
  if (g.direct) return 0;
  const int rows = g.wide ? 4 * kTeamRows : kTeamRows;
  return g.blocks * (2 * part_floats(rows, (int)D) * (int64_t)sizeof(float) + (int64_t)sizeof(int2));
}

hipError_t launch_tree_attention(int dtype, const TreeArgs& a, hipStream_t stream) {
  TreeParams p{};
  p.Q = static_cast<const unsigned char*>(a.Q);
  p.K = static_cast<const unsigned char*>(a.k_pages);
  p.V = static_cast<const unsigned char*>(a.v_pages);
  p.q_seq = 2 * a.q_seq;
  p.q_tok = 2 * a.q_tok;
  p.q_head = 2 * a.q_head;
  p.page_stride = 2 * a.page_stride;
  p.row_stride = 2 * a.row_stride;
  p.head_stride = 2 * a.head_stride;
  p.table = a.page_table;
  p.lens = a.lens;
  p.nodes = a.nodes;
  p.mask = static_cast<const uint64_t*>(a.mask);
  p.mask_seq = a.mask_seq;
  p.Out = static_cast<unsigned char*>(a.Out);
  p.lse = a.lse;
  p.partial = static_cast<float*>(a.workspace);
  p.page = fast_div(a.page_size);
  p.group = fast_div(a.Hq / a.Hkv);
  p.n_pages = (int32_t)a.n_pages;
  p.width = (int32_t)a.width;
  p.B = (int32_t)a.B;
  p.T = (int32_t)a.T;
  p.words = (int32_t)((a.T + 63) / 64);
  p.Hq = (int32_t)a.Hq;
  p.Hkv = (int32_t)a.Hkv;
  p.D = (int32_t)a.D;
  p.G = (int32_t)(a.Hq / a.Hkv);
  p.window = (int32_t)a.window;
  p.flip = a.scale_log2 < 0;
  // a scale of zero as the least normal number: the exponents of finite scores round to
  // zero all the same, and a masked score stays -inf
  const float scale = p.flip ? -a.scale_log2 : a.scale_log2;
  p.scale = scale < 0x1p-126f ? 0x1p-126f : scale;
  const TreeGrid g = tree_grid(a.B, a.T, a.Hq, a.Hkv, a.D, a.width * a.page_size);
  p.direct = g.direct;
  p.owner = reinterpret_cast<int2*>(
      p.partial + 2 * g.blocks * part_floats(g.wide ? 4 * kTeamRows : kTeamRows, p.D));
  const bool bf = dtype == TQ_BF16;
  if (g.wide)
    return bf ? launch_tree_d<true, 4>(p, g.blocks, stream)
              : launch_tree_d<false, 4>(p, g.blocks, stream);
  return bf ? launch_tree_d<true, 1>(p, g.blocks, stream)
            : launch_tree_d<false, 1>(p, g.blocks, stream);
}

hipError_t launch_tree_mask(const int32_t* parents, int64_t B, int64_t T, void* mask,
                            int32_t* depth, hipStream_t stream) {
  hipLaunchKernelGGL(tree_mask_kernel, dim3((uint32_t)B), dim3(kTreeThreads), 0, stream, parents,
                     (int)T, (int)((T + 63) / 64), static_cast<uint64_t*>(mask), depth);
  return hipGetLastError();
}

}  // namespace tq
