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
// each with K and V; a row block of them and a tile of tokens are a unit of work.
//
// What bounds it.  A token is 4 D bytes of a key-value head and 4 m G D operations: memory
// below some 200 rows, the matrix cores above.  Both forms compute S^T = K Q^T with the
// 32 x 32 x 16 instruction, so that a lane holds 16 scores of one row: the row's maximum and sum
// need one exchange between two lanes, and the weights are the second product's
// operand (O^T += V^T P^T) where they lie.  V is turned by the transposing read of LDS.
//   wide, for many rows: four waves of 32 rows each share tiles of 64 tokens, copied to LDS
//   past the registers, two tiles in turn.  131072 tokens, 64 nodes, 8 heads of 128 with 8
//   query heads each: 275 GFLOP in 370 us, 740 TFLOP/s, and 15 for the join (a plain product
//   of 8192^3 reaches 1330).  (Once the GPU has taken up the load: the calls 4 .. 40 after a
//   pause take up to 500.)  Matrix and other vector instructions take turns more than they
//   overlap: 39% and 42% of a SIMD's time, and waves wait a quarter of theirs; two waves a SIMD
//   are what the registers allow.  Four blocks of rows read the same tokens, and the L2s
//   catch half of that: 1.1 GB from memory of 0.54.  Mixing one tile's scores
//   with the product of the tile before inside a wave brought nothing (414 against 394).
//   thin, for up to 32 rows and short caches: the four waves share 128 tokens of the same
//   rows, each tile through registers to LDS that only its wave reads, and their sums meet
//   at the end.  37 ragged sequences of up to 4096 tokens, 24 heads of 64, 13 nodes: 122 MB in
//   37 us, 3.3 TB/s; half a tile's time goes to its chain page -> keys -> LDS -> scores, for
//   which three workgroups a CU do not make up.
// Row blocks are cut into equal runs over all workgroups; what spans several is joined by
// a second kernel in a fixed order (no atomics, the same bits on every run).

#include <math.h>

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
  int2* owner;     // [row blocks]: its first workgroup (-1 where that finished it), its last one
  FastDiv page, group;
  int32_t n_pages, width, B, T, words, Hq, Hkv, D, G, window;
  int32_t direct;  // one workgroup per row block: nothing is split
  int32_t runs;    // 16 tokens lie in one page
  int32_t lines;   // tokens are whole 128-byte lines
  float scale;     // not negative
  uint32_t flip;   // sign bits of two numbers where the caller's scale is negative: of the queries
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

// f of the values that the lanes l and l ^ 32 hold.
template <class F>
__device__ __forceinline__ float over_halves(float x, F f) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto both = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t low = both[0], high = both[1];
  return f(__builtin_bit_cast(float, low), __builtin_bit_cast(float, high));
}

__device__ __forceinline__ int64_t shfl64(int64_t v, int src) {
  const int lo = __shfl((int)v, src, kWave), hi = __shfl((int)(v >> 32), src, kWave);
  return ((int64_t)hi << 32) | (uint32_t)lo;
}

constexpr int kNonTemporal = 2;          // for lines that one wave reads once
constexpr int kNoLoads = 0x0f70;         // s_waitcnt: until no vector load is under way

template <int AUX>
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, AUX));
}
// 16 bytes at the resource's base + off to LDS: lane l writes the bytes dst + 16 l.  In
// assembly, because the compiler would otherwise wait for these copies before every
// transposing read of LDS, of whatever buffer; waited for by kNoLoads.  (Nothing is
// returned to a register.  A copy needs one state between the write of m0 and itself, and
// five after a vector instruction's write of its resource, which may be the one before: the
// compiler counts no states into assembly.)
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, int off, unsigned char* dst) {
  const uint32_t to = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)dst;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(to), "v"(off), "s"(r) : "memory", "m0");
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

// Weights are 2^(x - m + kShift): in fp16 the smaller ones then keep all their bits.  m follows
// the row's maximum only where that has risen by more than kSlack, so weights may reach
// 2^(kShift + kSlack) (fp16: 2^15): with many rows some maximum rises in most tiles, and
// every change multiplies all sums.
template <bool BF>
constexpr float kShift = BF ? 0.f : 9.f;
constexpr float kSlack = 6.f;
constexpr float kLn2 = 0.6931471805599453f;

// Divides by the sum and writes numbers d .. d + 3 of one query, and its lse.
template <bool BF>
__device__ __forceinline__ void store_row(const TreeParams& p, int64_t at, int d, float m,
                                          float sum, float inv, float4v v) {
  u32x2 u;
  u[0] = pack2<BF>(v[0] * inv, v[1] * inv);
  u[1] = pack2<BF>(v[2] * inv, v[3] * inv);
  *reinterpret_cast<u32x2*>(p.Out + (at * p.D + d) * 2) = u;
  if (p.lse && d == 0) p.lse[at] = (m + __builtin_amdgcn_logf(sum) - kShift<BF>) * kLn2;
}

// Workgroups per CU, for which the registers are laid out.
constexpr int tree_per_cu(int64_t D) { return D > 128 ? 1 : D > 64 ? 2 : 3; }

// DP: the head dimension rounded up to what the kernel is built for.
// TEAM: waves that share a tile of tokens, each with 32 rows of its own; a workgroup
// has 4 / TEAM teams, which take turns at the tokens of the same rows.
template <int DP, int TEAM, bool TWO>
struct Shape {
  static constexpr int KS = DP / 16;               // steps of a score
  static constexpr int NE = DP / 32;               // blocks of 32 numbers of the output
  static constexpr int PC = DP / 8;                // 16-byte pieces of a row
  static constexpr int TT = TEAM == 4 ? 64 : 32;   // tokens of a tile
  static constexpr int SUB = TT / 32;
  static constexpr int TEAMS = kTreeWaves / TEAM;
  static constexpr int UT = TT * TEAMS;            // tokens of a unit
  static constexpr int ROWS = kTeamRows * TEAM;    // rows of a block
  static constexpr int HALVES = TT / 16 / TEAM;         // runs of 16 tokens that a wave loads
  static constexpr int PH = 16 * PC / kWave;            // pieces of such a run, per thread
  static constexpr int PER = HALVES * PH;               // pieces of K (and of V) per thread
  static constexpr int TILE = TT * DP * 2;         // bytes of K (and of V)
  static constexpr int PAD = DP + 4;               // floats of a row of sums in LDS
  static constexpr int BUFFERS = TEAM == 4 ? 2 : 1;
  static constexpr int TILES = 2 * TILE * TEAMS * BUFFERS;
  static constexpr int JOIN = TEAM == 4 ? 0 : kTreeWaves * kTeamRows * PAD * 4;
  static constexpr int LDS = TILES > JOIN ? TILES : JOIN;
  // A weight as two 16-bit numbers where memory sets the pace, as one with many rows,
  // where each costs a matrix product: rounding it to nearest then adds as much
  // error to the output as the output's own rounding.
  static constexpr bool SPLIT = TWO;
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

template <bool BF, int DP, int TEAM, bool TWO>
__global__ __launch_bounds__(kTreeThreads, tree_per_cu(DP)) void tree_attention_kernel(
    TreeParams p) {
  using S = Shape<DP, TEAM, TWO>;
  constexpr int KS = S::KS, NE = S::NE, PC = S::PC, TT = S::TT, SUB = S::SUB, UT = S::UT;
  constexpr int ROWS = S::ROWS, PER = S::PER, PH = S::PH;
  extern __shared__ __attribute__((aligned(16))) unsigned char sTiles[];
  // what a row sees of the nodes, and its first cached token
  __shared__ uint64_t sBits[kTreeWaves][kTeamRows][kMaskWords];
  __shared__ int sLow[kTreeWaves][kTeamRows];
  __shared__ float sM[kTreeWaves][kTeamRows], sL[kTreeWaves][kTeamRows];
  __shared__ int sOdd[S::TEAMS];  // values that are no finite numbers were left out of a tile

  const int tid = threadIdx.x;
  const int wave = uni(tid >> 6), lane = tid & 63, col = lane & 31, half = lane >> 5;
  const int team = wave / TEAM;
  const int run16 = TEAM == 4 ? wave : 0;  // the first run of 16 tokens that this wave loads
  unsigned char* const sTeam = sTiles + team * 2 * S::TILE * S::BUFFERS;

  // This workgroup's run of units: every row block has a list (sequence, head, tile) of the
  // sequences that reach it, and workgroups by its length, which cut it into equal
  // runs.  Of equal lists workgroups i of all blocks then read the same tokens at the
  // same time on the same XCD (their number mostly being a multiple of 8), and all but
  // the first find them in its L2.
  Unit cur{};
  uint32_t left = 0, run_end = 0;
  Cut cut(0, 1);
  int part = 0;  // of the runs of its list
  if (p.direct) {
    const int rows = p.B * p.Hkv, rest = blockIdx.x % rows;
    cur.r = blockIdx.x / rows;
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
    // the first sequence that this lane looks after: mostly its only one
    const Seq own = read_seq<UT, ROWS>(p, lane * per < p.B ? lane * per : p.B - 1);
    const bool has_own = lane * per < p.B;
    uint32_t all = has_own ? (uint32_t)(own.t1 - own.t0) * own.blocks : 0;  // tiles x blocks
    int most = has_own ? own.blocks : 0;
    for (int i = 1; i < per; ++i) {
      const int b = lane * per + i;
      const Seq s = read_seq<UT, ROWS>(p, b < p.B ? b : p.B - 1);
      if (b < p.B) {
        all += (uint32_t)(s.t1 - s.t0) * s.blocks;
        most = s.blocks > most ? s.blocks : most;
      }
    }
    all = uni((int)__shfl(scan_wave(all, lane), 63, kWave));
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
      const int o = __shfl_xor(most, off, kWave);
      most = o > most ? o : most;
    }
    // one workgroup for each block, and of the others its share
    const uint32_t spare = gridDim.x - uni(most);
    uint32_t mine = 0, inc = 0, first = 0;
    for (; cur.r < uni(most); ++cur.r) {
      mine = has_own && own.blocks > cur.r ? own.t1 - own.t0 : 0;
      for (int i = 1; i < per; ++i) mine += tiles_of(lane * per + i, true, cur.r);
      inc = scan_wave(mine, lane);
      const uint32_t total = uni((int)__shfl(inc, 63, kWave));
      const uint32_t share = 1 + (uint32_t)((uint64_t)total * spare / (all ? all : 1));
      if (blockIdx.x < first + share) {
        cut = Cut(total * p.Hkv, share);
        part = blockIdx.x - first;
        break;
      }
      first += share;
    }
    if ((uint32_t)part < cut.parts) {
      uint32_t at = cut.start(part);
      run_end = cut.start(part + 1);
      left = run_end - at;
      // the lane that looks after the sequence, the sequence
      const uint64_t has = __ballot(at < inc * p.Hkv);
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
      // (the bounds hold whatever happens to the lengths meanwhile)
      if (cur.b >= p.B) cur.b = p.B - 1;
      cur.s = read_seq<UT, ROWS>(p, cur.b);
      const uint32_t n = cur.s.t1 > cur.s.t0 ? cur.s.t1 - cur.s.t0 : 1;
      cur.h = at / n;
      cur.tile = cur.s.t0 + at % n;
      if (cur.h >= p.Hkv) cur.h = p.Hkv - 1;
    }
  }
  // The first unit after c's row (of a sequence and head).
  auto next_row = [&](Unit& c) {
    if (++c.h == p.Hkv) {
      c.h = 0;
      do {
        if (++c.b >= p.B) {  // past the end (the lengths have changed)
          left = 0;
          return;
        }
        c.s = read_seq<UT, ROWS>(p, c.b);
      } while (c.s.t1 <= c.s.t0 || c.s.blocks <= c.r);
    }
    c.tile = c.s.t0;
  };

  auto first_token = [&](int tile) { return tile * UT + team * TT; };
  // The page of this lane's token of the team's tile, as the table has it.
  auto page_id = [&](const Unit& c, int tile) {
    const int t = first_token(tile) + (lane & (TT - 1));
    const bool in = t >= c.s.lo && t < c.s.hi;
    return p.table[(int64_t)c.b * p.width + div_page(p.page, in ? t : c.s.lo)];
  };
  // Whether some row may not see some present token of the tile.
  auto edge = [&](const Seq& s, int tile) {
    const int a = first_token(tile);
    return a + TT > s.n || (p.window > 0 && a < s.n + s.m - p.window);
  };
  // Of a tile at an edge only the finite values go to LDS: a weight of zero times infinity
  // would reach rows that do not see the token.  close_row adds what is left out here.
  u32x4 kreg[PER], vreg[PER];
  auto stage = [&](bool at_edge, unsigned char* buf) {
    if (at_edge) {
      // (single waves look first whether there are any: a number's exponent is all ones where
      // one more carries into its sign)
      constexpr uint32_t exps = BF ? 0x7f807f80u : 0x7c007c00u, one = BF ? 0x00800080u : 0x04000400u;
      uint32_t odd = TEAM == 4;
      if constexpr (TEAM == 1) {
#pragma unroll
        for (int u = 0; u < PER; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) odd |= (vreg[u][i] & exps) + one & 0x80008000u;
      }
      if (odd) {
        odd = 0;
#pragma unroll
        for (int u = 0; u < PER; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t f = finite_of<BF>(vreg[u][i]);
            odd |= f ^ vreg[u][i];
            vreg[u][i] = f;
          }
        if (odd) sOdd[team] = 1;  // every writer writes 1
      }
    }
    const int ln = TEAM == 1 ? lane : anew(lane);
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int x = u % PH * kWave + ln, row = 16 * (run16 + u / PH) + x / PC, piece = x % PC;
      *reinterpret_cast<u32x4*>(buf + (row * PC + S::k_at(row, piece)) * 16) = kreg[u];
      *reinterpret_cast<u32x4*>(buf + S::TILE + (row * PC + S::v_at(row, piece)) * 16) = vreg[u];
    }
  };
  // Fetches a tile.  A wave takes runs of 16 tokens, lane x their pieces x, x + 64, ..  Teams
  // of four copy straight to LDS where every token is there, none is at an edge and a
  // run lies in one page: where a piece lies in LDS is turned, so a lane fetches what
  // belongs to its place.  Other tiles, and those of single waves, go through registers,
  // where a run lies in one page by offsets that tokens that are not there send past
  // the buffer's end.
  uint64_t present = 0;  // tokens that are there, of the tile last fetched
  constexpr uint64_t kFull = TT == 64 ? ~0ull : 0xffffffffull;
  auto fetch = [&](const Unit& c, int tile, int id, unsigned char* buf) {
    const int a = first_token(tile);
    const int t = a + (lane & (TT - 1));
    const bool ok = t >= c.s.lo && t < c.s.hi && (uint32_t)id < (uint32_t)p.n_pages;
    const bool at_edge = edge(c.s, tile);
    present = __ballot(ok) & kFull;
    const int64_t head = c.h * p.head_stride;
    const int D = anew_uniform(p.D), ln = anew(lane);
    if (p.runs && (TEAM == 1 || (present == kFull && !at_edge))) {
#pragma unroll
      for (int r = 0; r < S::HALVES; ++r) {
        const int first = a + 16 * (run16 + r);
        const int slot = first - (int)(div_page(p.page, first) * p.page.d);
        // tokens [begin, begin + count) of the run are there
        int begin = 0, count = 16, page = __builtin_amdgcn_readlane(id, 16 * (run16 + r));
        if constexpr (TEAM == 1) {
          const uint32_t have = (uint32_t)(present >> (16 * r)) & 0xffff;  // no gaps: one page
          begin = have ? __builtin_ctz(have) : 0;
          count = __builtin_popcount(have);
          page = __builtin_amdgcn_readlane(id, 16 * r + begin);
          page = have ? page : 0;
        }
        const int64_t at = page * p.page_stride + slot * p.row_stride + head;
        const auto rk = rsrc_at(p.K + at), rv = rsrc_at(p.V + at);
#pragma unroll
        for (int u = 0; u < PH; ++u) {
          const int x = u * kWave + (TEAM == 4 ? lane : ln), row = x / PC, place = x - row * PC;
          if constexpr (TEAM == 4) {
            unsigned char* to = buf + (run16 * 16 * PC + u * kWave) * 16;
            const int kp = S::k_at(row, place), vp = S::v_at(row, place);
            if (kp * 8 < D) dma16(rk, row * (int)p.row_stride + kp * 16, to);
            if (vp * 8 < D) dma16(rv, row * (int)p.row_stride + vp * 16, to + S::TILE);
          } else {
            const bool in = (uint32_t)(row - begin) < (uint32_t)count && place * 8 < D;
            const uint32_t off = in ? row * (uint32_t)p.row_stride + place * 16 : kOut;
            if (p.lines) {
              kreg[r * PH + u] = load16<kNonTemporal>(rk, off);
              vreg[r * PH + u] = load16<kNonTemporal>(rv, off);
            } else {
              kreg[r * PH + u] = load16<0>(rk, off);
              vreg[r * PH + u] = load16<0>(rv, off);
            }
          }
        }
      }
      return;
    }
    const int slot = t - (int)(div_page(p.page, ok ? t : 0) * p.page.d);
    const int64_t off = ok ? id * p.page_stride + slot * p.row_stride + head : -1;
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int x = u % PH * kWave + ln, row = x / PC, piece = x - row * PC;
      const int64_t o = shfl64(off, 16 * (run16 + u / PH) + row);
      kreg[u] = vreg[u] = u32x4{0, 0, 0, 0};
      if (o >= 0 && piece * 8 < D) {
        kreg[u] = *reinterpret_cast<const u32x4*>(p.K + o + piece * 16);
        vreg[u] = *reinterpret_cast<const u32x4*>(p.V + o + piece * 16);
      }
    }
    if constexpr (TEAM == 4) stage(at_edge, buf);
  };

  u32x4 q[KS];
  f32x16 acc[NE];
  float m = -INFINITY, l = 0.f;
  int row0 = 0;  // of this wave
  auto open_row = [&](const Unit& c) {
    const int col = anew(lane & 31), half = anew(lane >> 5);
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
    if (p.flip)  // (without, nothing here waits for the queries)
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) q[k][i] ^= p.flip;
    int seen = 0;
#pragma unroll 1
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
    const int col = anew(lane & 31);
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
  auto v_operand = [&](const unsigned char* sV, int e, int s, int u) {
    const int i = lane & 15;
    const int t = 32 * s + 16 * u + 4 * half + (i >> 2);
    const int piece = 4 * e + 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
    typedef __attribute__((address_space(3))) s16x4* lds4;
    const unsigned char* a = sV + (t * PC + S::v_at(t, piece)) * 16 + (i & 1) * 8;
    const unsigned char* b = sV + ((t + 8) * PC + S::v_at(t + 8, piece)) * 16 + (i & 1) * 8;
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
    const int half = anew(lane >> 5);
    Unit x = c;
    for (x.tile = first; x.tile <= c.tile; ++x.tile) {
      if (!edge(c.s, x.tile)) continue;
      for (int k = 0; k < TT; ++k) {
        const int t = first_token(x.tile) + k;
        if (t < c.s.lo || t >= c.s.hi) continue;
        const int pg = div_page(p.page, t);
        const int id = p.table[(int64_t)c.b * p.width + pg];
        if ((uint32_t)id >= (uint32_t)p.n_pages || !(sees(c, t, 1u) & 1)) continue;
        const unsigned char* v = p.V + id * p.page_stride + (t - pg * (int)p.page.d) * p.row_stride +
                                 c.h * p.head_stride;
        const int D = anew_uniform(p.D);
#pragma unroll
        for (int e = 0; e < NE; ++e)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int d = 32 * e + 8 * r + 4 * half;
            if (d >= D) continue;
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
    const int col = anew(lane & 31), half = anew(lane >> 5), tid = anew(threadIdx.x);
    if (sOdd[team]) add_odd(c, first_tile);
    const bool whole = begins && ends;
    float* const part = p.direct ? nullptr : part_of(begins ? 1 : 0);
    const int rows = c.s.m * p.G;
    const float sum = over_halves(l, [](float x, float y) { return x + y; });
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
      // a thread has four numbers of rows r, r + EACH, ..
      constexpr int EACH = kTreeThreads / (DP / 4);
      const int r0 = tid / (DP / 4), d = (tid - r0 * (DP / 4)) * 4;
#pragma unroll 2
      for (int k = 0; k < (kTeamRows + EACH - 1) / EACH; ++k) {
        const int r = r0 + k * EACH;
        if (r0 >= EACH || r >= n || d >= p.D) continue;
        // (all of LDS is read before anything waits for it)
        float mw[kTreeWaves], lw[kTreeWaves], mm = -INFINITY, total = 0.f;
        float4v x[kTreeWaves], v = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kTreeWaves; ++w) {
          mw[w] = sM[w][r];
          lw[w] = sL[w][r];
          x[w] = *reinterpret_cast<const float4v*>(sO + (w * kTeamRows + r) * S::PAD + d);
        }
#pragma unroll
        for (int w = 0; w < kTreeWaves; ++w) mm = fmaxf(mm, mw[w]);
        const float base = mm == -INFINITY ? 0.f : mm;
#pragma unroll
        for (int w = 0; w < kTreeWaves; ++w) {
          const float f = __builtin_amdgcn_exp2f(mw[w] - base);
          total += f * lw[w];
          // a wave without weight adds nothing, also where it has met NaN
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] += lw[w] != 0.f ? f * x[w][i] : 0.f;
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

  // One tile: scores, weights, and their product with V.
  auto compute = [&](const Unit& c, int tile, uint64_t there, const unsigned char* sK) {
    const unsigned char* const sV = sK + S::TILE;
    const int a0 = first_token(tile);
    // Reads of LDS are issued well ahead of their use and kept there: a read that
    // is waited for takes longer than a matrix instruction.
    // (Of long heads half the keys at a time: more registers there are not.)
    constexpr int KH = KS <= 8 ? KS : KS / 2;
    f32x16 s[SUB];
#pragma unroll
    for (int x = 0; x < SUB; ++x)
#pragma unroll
      for (int r = 0; r < 16; ++r) s[x][r] = 0.f;
#pragma unroll
    for (int i0 = 0; i0 < KS; i0 += KH) {
      u32x4 k[KH][SUB];
#pragma unroll
      for (int i = 0; i < KH; ++i)
#pragma unroll
        for (int x = 0; x < SUB; ++x) {
          const int t = 32 * x + col;
          k[i][x] = *reinterpret_cast<const u32x4*>(
              sK + (t * PC + S::k_at(t, 2 * (i0 + i) + half)) * 16);
        }
      __builtin_amdgcn_sched_barrier(0);
      if (TEAM == 4) __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int i = 0; i < KH; ++i)
#pragma unroll
        for (int x = 0; x < SUB; ++x) s[x] = mma32<BF>(k[i][x], q[i0 + i], s[x]);
      if (TEAM == 4) __builtin_amdgcn_s_setprio(0);
      if (i0 + KH < KS) __builtin_amdgcn_sched_barrier(0);
    }
    u32x4 v[NE][SUB * 2];
    auto read_v = [&](int e) {
#pragma unroll
      for (int y = 0; y < SUB * 2; ++y) v[e][y] = v_operand(sV, e, y / 2, y % 2);
    };
    read_v(0);
    if constexpr (NE > 1) read_v(1);
    __builtin_amdgcn_sched_barrier(0);
    if (there != kFull || edge(c.s, tile)) {
#pragma unroll
      for (int x = 0; x < SUB; ++x) {
        const uint32_t see = sees(c, a0 + 32 * x, (uint32_t)(there >> (32 * x))) >> (4 * half);
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
    top = over_halves(top, [](float x, float y) { return fmaxf(x, y); });
    const bool stays = top <= m || (top - m) * p.scale <= kSlack;
    if (!__all(stays)) {
      // (every row by what it sees itself: a row beside it that rises changes none of its bits)
      const float mn = stays ? m : fmaxf(m, top);
      const float alpha = stays ? 1.f : __builtin_amdgcn_exp2f((m - mn) * p.scale);
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
    if (TEAM == 4) __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      __builtin_amdgcn_sched_barrier(0);
      if (e + 2 < NE) read_v(e + 2);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int y = 0; y < SUB * 2; ++y) {
        acc[e] = mma32<BF>(v[e][y], hi[y / 2][y % 2], acc[e]);
        if constexpr (S::SPLIT) acc[e] = mma32<BF>(v[e][y], lo[y / 2][y % 2], acc[e]);
      }
    }
    if (TEAM == 4) __builtin_amdgcn_s_setprio(0);
  };

  if (tid < S::TEAMS) sOdd[tid] = 0;
  if (S::BUFFERS == 2 && p.D < DP)  // direct copies leave the numbers past a head's end out
    for (int i = tid; i < S::TILES / 16; i += kTreeThreads)
      *reinterpret_cast<u32x4*>(sTiles + i * 16) = u32x4{0, 0, 0, 0};
  __syncthreads();
  if (left > 0) {
    unsigned char* buf = sTeam;
    int id = page_id(cur, cur.tile);
    if (TEAM == 4) open_row(cur);
    fetch(cur, cur.tile, id, buf);
    if (TEAM == 1) open_row(cur);  // its loads are waited for together with the tile's
    for (bool opened = true;; opened = false) {
      // the tiles [first, end) of one row
      const int first = cur.tile;
      const int end = (uint32_t)(cur.s.t1 - first) < left ? cur.s.t1 : first + (int)left;
      left -= end - first;
      const bool begins = first == cur.s.t0, ends = end == cur.s.t1;
      const uint32_t row_end = run_end - left + (cur.s.t1 - end);  // the unit after this row
      Unit next = cur;
      if (left > 0) next_row(next);
      id = end - first > 1 ? page_id(cur, first + 1) : left > 0 ? page_id(next, next.tile) : 0;
      if (!opened) open_row(cur);
      for (int tile = first; tile < end; ++tile) {
        const uint64_t there = present;
        if (TEAM == 4) {
          __builtin_amdgcn_s_waitcnt(kNoLoads);
          __syncthreads();  // this tile is there, and the one before it has been read
        } else {
          stage(edge(cur.s, tile), buf);
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
        unsigned char* const other = buf == sTeam ? sTeam + 2 * S::TILE : sTeam;
        unsigned char* const to = S::BUFFERS == 1 ? buf : other;
        const bool here = tile + 1 < end;  // the tile that follows is this row's
        if (here || left > 0) {
          fetch(here ? cur : next, here ? tile + 1 : next.tile, id, to);
          if (here)
            id = tile + 2 < end ? page_id(cur, tile + 2) : left > 0 ? page_id(next, next.tile) : 0;
        }
        compute(cur, tile, there, buf);
        buf = to;
      }
      cur.tile = end - 1;
      close_row(cur, first, begins, ends);
      if (begins && !p.direct && tid == 0)  // (where it does not end here, the following ones go on)
        p.owner[(cur.r * p.B + cur.b) * p.Hkv + cur.h] =
            make_int2(ends ? -1 : (int)blockIdx.x,
                      (int)blockIdx.x - part + (int)cut.part_of(row_end - 1));
      if (left == 0) break;
      cur = next;
    }
  }

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

// Joins the partial results of the row blocks that span workgroups.  A group of lanes, a power
// of two that holds D / 4, takes a row: each lane looks up the maximum and sum of one part, then
// all of them its numbers, part by part.  `share` groups, where rows are few and their
// parts many, take a row's parts in turns.
template <int DP>
constexpr int join_lanes() {
  return DP <= 64 ? 16 : DP <= 128 ? 32 : 64;
}
template <bool BF, int DP, int ROWS>
__global__ __launch_bounds__(kTreeThreads) void tree_join_kernel(TreeParams p, int blocks,
                                                                 int share) {
  constexpr int CL = join_lanes<DP>(), GROUPS = kTreeThreads / CL, U = 8;
  __shared__ __attribute__((aligned(16))) float sV[kTreeThreads * 4];
  const int tid = threadIdx.x, lane = tid % CL, col = lane * 4;
  const int turn = tid / CL % share, mine = tid / CL / share, step = GROUPS / share;
  const int base_lane = (tid & (kWave - 1)) - lane;
  const int64_t size = part_floats(ROWS, p.D);
  for (int block = blockIdx.x; block < blocks; block += gridDim.x) {
    const int2 own = p.owner[block];
    const int h = block % p.Hkv, rest = block / p.Hkv, b = rest % p.B, r = rest / p.B;
    const int nodes = p.nodes ? p.nodes[b] : p.T;
    int rows = (nodes < p.T ? nodes : p.T) * p.G - r * ROWS;
    if (rows <= 0 || own.x < 0) continue;  // (a block without rows has no owner)
    rows = rows < ROWS ? rows : ROWS;
    const int n = own.y - own.x + 1;
    // part 0 is the second slot of the workgroup that began the block, the others the first
    // slots of those that follow
    auto part = [&](int k) {
      return p.partial + (2 * ((int64_t)own.x + k) + (k == 0 ? 1 : 0)) * size;
    };
    for (int j0 = blockIdx.y * step; j0 < rows; j0 += gridDim.y * step) {
      const int j = j0 + mine;
      const bool real = j < rows;
      const int at_m = ROWS * p.D + (real ? j : 0), at_l = at_m + ROWS;
      float m = -INFINITY, total = 0.f;
      for (int k = lane; k < n; k += CL) m = fmaxf(m, part(k)[at_m]);
#pragma unroll
      for (int off = 1; off < CL; off <<= 1) m = fmaxf(m, __shfl_xor(m, off, kWave));
      const float base = m == -INFINITY ? 0.f : m;
      float4v v = {0, 0, 0, 0};
      for (int k0 = 0; k0 < n; k0 += CL) {
        const int k = k0 + lane < n ? k0 + lane : n - 1;
        float w = __builtin_amdgcn_exp2f(part(k)[at_m] - base);
        const float l = part(k)[at_l];
        // a part without weight adds nothing (-1), also where it has met NaN; one whose sum is NaN
        // has a weight of NaN, also where all its scores are, so that its maximum is -inf; and
        // one whose weight rounds to zero counts: an infinite value in it makes NaN
        if (k0 + lane >= n || l == 0.f) w = -1.f;
        else if (l != l) w = l;
        if (!(w < 0.f)) total += w * l;
        const int most = n - k0 < CL ? n - k0 : CL;
        for (int x0 = turn; x0 < most; x0 += U * share) {
          float4v x[U];
          float wx[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int i = x0 + u * share < most ? x0 + u * share : most - 1;
            wx[u] = __shfl(w, base_lane + i, kWave);
            if (x0 + u * share >= most) wx[u] = -1.f;
            x[u] = float4v{0, 0, 0, 0};
            if (!(wx[u] < 0.f) && real && col < p.D)
              x[u] = *reinterpret_cast<const float4v*>(part(k0 + i) + (int64_t)j * p.D + col);
          }
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (!(wx[u] < 0.f)) v += wx[u] * x[u];
        }
      }
#pragma unroll
      for (int off = 1; off < CL; off <<= 1) total += __shfl_xor(total, off, kWave);
      if (share > 1) {
        *reinterpret_cast<float4v*>(sV + tid * 4) = v;
        __syncthreads();
        if (turn == 0)
          for (int i = 1; i < share; ++i)
            v += *reinterpret_cast<const float4v*>(sV + (tid + i * CL) * 4);
        __syncthreads();
      }
      if (turn == 0 && real && col < p.D) {
        const int row = r * ROWS + j, i = div_page(p.group, row), g = row - i * p.G;
        store_row<BF>(p, ((int64_t)b * p.T + i) * p.Hq + h * p.G + g, col, m, total,
                      total == 0.f ? 0.f : 1.f / total, v);
      }
    }
  }
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

struct TreeGrid {
  int64_t grid, blocks;
  bool direct, wide;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Two forms.  Wide (heads of more than 128 numbers: always, the thin form's registers do not hold
// them): four waves share the tokens, each with 32 rows of its own, so that one reading of a
// tile serves 128 rows.  Thin: 32 rows, and the waves share the tokens: for
// up to 32 rows, and for short caches where the GPU has a CU for every 32 rows (heads of up to 64:
// for every 64), because four waves then walk through a row's tiles at once.  Measured (us,
// thin / wide), one tree of 24 nodes, 8 key heads of 128 and 8 query heads each, up to
// 32, 128, 256, 512 tokens: 9.6 / 10.2, 9.6 / 11.5, 11.7 / 14.9, 15.8 / 21.3; eight trees (384 thin
// workgroups) 12.8 / 10.8, 12.9 / 12.3, 16.1 / 15.7, 21.5 / 22.2; four of 64 nodes, 4 heads each of
// 64 7.2 / 8.7, 8.4 / 11.1, 10.9 / 16.0; ten of 100 nodes, 8 heads of 64 (320 thin workgroups), up to
// 204, 500 tokens 10.3 / 13.1, 13.6 / 17.4.  Either side of the limit, 192 and 512 tokens: heads of 64,
// 512 thin workgroups 11.8 / 11.2 and 15.8 / 18.3 (32 nodes, 8 / 1 heads), 12.7 / 12.1 and 16.9 / 19.4
// (100 nodes), 640 of them 14.7 / 11.2 and 19.5 / 18.4, 14.9 / 12.7 and 20.6 / 19.5; heads of 128, 256
// 13.8 / 14.4 and 19.2 / 23.3, 384 17.2 / 15.0 and 24.7 / 24.3.
constexpr int64_t kShort = 512;

TreeGrid tree_grid(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t capacity) {
  const int64_t rows = T * (Hq / Hkv), thin = B * Hkv * ceil_div(rows, kTeamRows);
  const int64_t room = device_cus() * (D > 64 ? 1 : 2);
  const bool wide = D > 128 || (rows > kTeamRows && !(capacity <= kShort && thin <= room));
  const int64_t blocks = wide ? B * Hkv * ceil_div(rows, 4 * kTeamRows) : thin;
  const int64_t tiles = ceil_div(capacity, wide ? 64 : 128) + 1;  // a window may begin inside one
  const int64_t at_once = device_cus() * tree_per_cu(D);
  // Nothing is split where a row has few tiles (splitting and joining cost some 10 us with
  // 32 rows, 20 with 128), or where there are so many rows that others are at work while a
  // workgroup takes a long one: four rounds, and no more than eight tiles of the longest row a
  // round, as the table has room for; or where there are more blocks of rows of a sequence
  // than the split could tell apart.
  // Measured (us, whole / split).  Few tiles, all rows equally long, heads of 128: thin, 8 blocks of
  // 512, 1024 tokens 16.6 / 15.3, 24.5 / 16.1; 128 blocks of 512, 1024, 1536 19.5 / 26.8, 29.6 / 31.6,
  // 40.4 / 36.7; 320 blocks of 1024, 2048 47.7 / 56.8, 83.0 / 86.8.  Wide, 16 blocks of 704
  // 27.7 / 22.4; 128 of 704, 1024, 1536 29.6 / 42.3, 37.9 / 38.2, 51.6 / 44.2; 384 of 704, 2048
  // 40.2 / 67.6, 92.1 / 110.9.  Equal rows would stay whole for longer where blocks are many; the
  // split is for those that are not equal.
  // Many rows, one of as many tokens as the table holds and the others of 400: 2048 thin blocks (four
  // rounds), 2048, 4096, 32768 tokens 143 / 123, 180 / 126, 709 / 158, without the long one 115 / 115;
  // 2048 wide ones 185 / 232, 236 / 199, 971 / 267, without 148 / 150; 4096 thin ones of heads of 64
  // (4096 sequences, whose lengths every workgroup reads) 115 / 156, 135 / 157, 418 / 159, without
  // 102 / 157.
  const int64_t few = wide ? 12 : blocks < device_cus() ? 5 : 9, rounds = blocks / at_once;
  if (tiles <= few || (rounds >= 4 && tiles <= 8 * rounds) || 4 * blocks >= at_once * B * Hkv)
    return {blocks, blocks, true, wide};
  return {blocks * tiles < at_once ? blocks * tiles : at_once, blocks, false, wide};
}

// Workgroups of a join: with one row of 16 lanes and more at a time, as many as keep every CU busy.
// Measured on the GPU (us): 32 blocks of 128 rows in 16 parts each 15.1 (a workgroup for each
// that began a block, most of them idle: 45), 384 blocks in some two parts 18.2, with 8192
// workgroups 14.2 and 20.5.  Whole calls of six shapes (1 .. 37 sequences of 2048 .. 32768 tokens,
// heads of 64 .. 256) differ by 3% at most between 1024, 2048 and 8192; with 512 24 sequences of
// 4096 tokens take 206 against 192.
constexpr int64_t kJoin = 2048;

template <bool BF, int DP, int TEAM, bool TWO>
hipError_t launch_tree(const TreeParams& p, const TreeGrid& g, hipStream_t s) {
  using Sh = Shape<DP, TEAM, TWO>;
  const auto fn = tree_attention_kernel<BF, DP, TEAM, TWO>;
  if (Sh::LDS > 48 * 1024) {
    static std::atomic<uint64_t> done{0};
    const hipError_t e = lds_limit_once(reinterpret_cast<const void*>(fn), Sh::LDS, done);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(fn, dim3((uint32_t)g.grid), dim3(kTreeThreads), Sh::LDS, s, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.direct) return e;
  constexpr int GROUPS = kTreeThreads / join_lanes<DP>();
  // groups share a row as long as each then has four parts or more, and a block's rows are
  // spread over workgroups as long as those are kJoin or fewer
  int share = 1;
  while (share < GROUPS && 8 * share * g.blocks <= g.grid) share *= 2;
  const int rows = p.T * p.G < Sh::ROWS ? p.T * p.G : Sh::ROWS;
  const int64_t across = g.blocks < kJoin ? g.blocks : kJoin;
  const int64_t slices = ceil_div((int64_t)rows * share, GROUPS), most = kJoin / across;
  hipLaunchKernelGGL((tree_join_kernel<BF, DP, Sh::ROWS>),
                     dim3((uint32_t)across, (uint32_t)(slices < most ? slices : most)),
                     dim3(kTreeThreads), 0, s, p, (int)g.blocks, share);
  return hipGetLastError();
}

template <bool BF>
hipError_t launch_tree_d(const TreeParams& p, const TreeGrid& g, hipStream_t s) {
  if (!g.wide)
    return p.D <= 64   ? launch_tree<BF, 64, 1, true>(p, g, s)
           : p.D <= 96 ? launch_tree<BF, 96, 1, true>(p, g, s)
                       : launch_tree<BF, 128, 1, true>(p, g, s);
  const bool two = p.T * p.G <= kTeamRows;  // of long heads
  return p.D <= 64    ? launch_tree<BF, 64, 4, false>(p, g, s)
         : p.D <= 96  ? launch_tree<BF, 96, 4, false>(p, g, s)
         : p.D <= 128 ? launch_tree<BF, 128, 4, false>(p, g, s)
         : p.D <= 192 ? two ? launch_tree<BF, 192, 4, true>(p, g, s)
                            : launch_tree<BF, 192, 4, false>(p, g, s)
         : two        ? launch_tree<BF, 256, 4, true>(p, g, s)
                      : launch_tree<BF, 256, 4, false>(p, g, s);
}

}  // namespace

int64_t tree_workspace_bytes(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                             int64_t capacity) {
  const TreeGrid g = tree_grid(B, T, Hq, Hkv, D, capacity);
  if (g.direct) return 0;
  const int rows = g.wide ? 4 * kTeamRows : kTeamRows;
  return g.grid * 2 * part_floats(rows, (int)D) * (int64_t)sizeof(float) +
         g.blocks * (int64_t)sizeof(int2);
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
  p.flip = a.scale_log2 < 0 ? 0x80008000u : 0u;
  p.runs = a.page_size % 16 == 0;
  const uint64_t places = reinterpret_cast<uint64_t>(p.K) | reinterpret_cast<uint64_t>(p.V) |
                          (uint64_t)(p.page_stride | p.row_stride | p.head_stride) | (uint64_t)p.D * 2;
  p.lines = places % 128 == 0;
  // a scale of zero as the least normal number: the exponents of finite scores round to
  // zero all the same, and a masked score stays -inf
  const float scale = fabsf(a.scale_log2);
  p.scale = scale < 0x1p-126f ? 0x1p-126f : scale;
  const TreeGrid g = tree_grid(a.B, a.T, a.Hq, a.Hkv, a.D, a.width * a.page_size);
  p.direct = g.direct;
  p.owner = reinterpret_cast<int2*>(
      p.partial + 2 * g.grid * part_floats(g.wide ? 4 * kTeamRows : kTeamRows, p.D));
  const bool bf = dtype == TQ_BF16;
  return bf ? launch_tree_d<true>(p, g, stream) : launch_tree_d<false>(p, g, stream);
}

hipError_t launch_tree_mask(const int32_t* parents, int64_t B, int64_t T, void* mask,
                            int32_t* depth, hipStream_t stream) {
  hipLaunchKernelGGL(tree_mask_kernel, dim3((uint32_t)B), dim3(kTreeThreads), 0, stream, parents,
                     (int)T, (int)((T + 63) / 64), static_cast<uint64_t*>(mask), depth);
  return hipGetLastError();
}

}  // namespace tq
