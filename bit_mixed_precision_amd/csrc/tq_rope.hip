// Rotary positions, and their use in a decode step: rotate queries and keys of
// the fused q/k/v product and write keys and values into the paged cache.
//
// A pair (a, b) of a head is turned by the angle of its token's position:
//     a' = a cos - b sin,   b' = b cos + a sin
// with cos and sin from a table of fp32 pairs, one row per position, computed
// in fp64 on the host: an angle of 10^5 turns keeps its full accuracy, which
// fp32 arithmetic on the device would not give.
//
// Bound: reading X and writing Y once (3 flops per number); the table row of a
// token (4 rot bytes) is shared by its heads and comes from the caches.
//
// Layout.  A head is cut into units: unit u < rot / 2V turns the two vectors of
// V numbers at u V and rot/2 + u V, which are the two sides of V pairs in the
// half layout and V/2 pairs each in the interleaved one; the units after that
// copy one vector of the rest.  With V = 8 (16-bit types) a lane moves 16 bytes
// per access and 8 lanes cover a 128-number head as two whole 128-byte lines.
// Heads of all tokens form one flattened list, so few heads or few tokens fill
// the lanes alike.

#include "tq.h"
#include "tq_common.h"
#include "tq_decode.h"
#include "tq_kernels.h"

namespace tq {
namespace {

constexpr int kRopeThreads = 256;

// n / d for 0 <= n < 2^31: exact with m = ceil(2^(31 + s) / d), s = ceil(log2 d).
struct Div31 {
  uint32_t d, m, shift;
  __host__ static Div31 of(int64_t d) {
    uint32_t s = 0;
    while ((int64_t(1) << s) < d) ++s;
    const uint64_t m = ((uint64_t(1) << (31 + s)) + d - 1) / d;
    return {(uint32_t)d, (uint32_t)m, 31 + s};
  }
  __device__ __forceinline__ uint32_t quot(uint32_t n) const {
    return (uint32_t)(((uint64_t)n * m) >> shift);
  }
};

struct RopeParams {
  const unsigned char* X;
  unsigned char* Y;
  int64_t x_tok, x_head, y_tok, y_head;  // elements
  const float2* table;
  const int32_t* pos;
  uint32_t n_pos, rows;  // rows = T * H
  int32_t rot, D;
  int32_t turn_units, units;  // per head: turning, all
  Div31 heads;
  // appending
  int32_t Hq, Hkv;
  unsigned char* K;
  unsigned char* Vp;
  int64_t page_stride, row_stride, head_stride;
  Div31 page;
  uint32_t n_pages, width, n_seqs;
  const int32_t* page_table;
  const int32_t* seqs;
};

// V numbers moved as one access (two or more of 16 bytes where they are longer).
template <class S, int V>
struct alignas(sizeof(S) * V < 16 ? sizeof(S) * V : 16) Pack {
  S v[V];
};

// One row (token, head) and unit of one thread.
template <class S, int V, bool INTER, bool INV, bool APPEND>
struct RopeItem {
  const S* x;
  S* y;  // nullptr: not written
  bool turn, zero;
  int u;
  uint32_t pos;
  Pack<S, V> a, b;

  __device__ __forceinline__ void locate(const RopeParams& p, uint32_t row, int unit) {
    u = unit;
    const uint32_t tok = p.heads.quot(row);
    const int head = (int)(row - tok * p.heads.d);
    const int32_t ps = p.pos[tok];
    pos = (uint32_t)ps;
    const bool ok = pos < p.n_pos;
    zero = !ok;
    turn = u < p.turn_units;
    x = reinterpret_cast<const S*>(p.X) + tok * p.x_tok + head * p.x_head;
    if constexpr (!APPEND) {
      y = reinterpret_cast<S*>(p.Y) + tok * p.y_tok + head * p.y_head;
    } else if (head < p.Hq) {
      y = reinterpret_cast<S*>(p.Y) + tok * p.y_tok + head * p.y_head;
    } else {
      const bool key = head < p.Hq + p.Hkv;
      if (!key) turn = false;
      y = nullptr;
      const uint32_t seq = p.seqs ? (uint32_t)p.seqs[tok] : tok;
      const uint32_t pg = p.page.quot(ok ? pos : 0);
      if (ok && seq < p.n_seqs && pg < p.width) {
        const uint32_t id = (uint32_t)p.page_table[(int64_t)seq * p.width + pg];
        if (id < p.n_pages)
          y = reinterpret_cast<S*>(key ? p.K : p.Vp) + id * p.page_stride +
              (pos - pg * p.page.d) * p.row_stride + (head - p.Hq - (key ? 0 : p.Hkv)) * p.head_stride;
      }
    }
  }
  // Numbers of the unit's two vectors (`second` also of units that copy, where
  // they lie inside rot), and whether there is a second one.
  __device__ __forceinline__ int first(const RopeParams& p) const {
    if (u >= p.turn_units) return p.rot + (u - p.turn_units) * V;
    return V == 1 && INTER ? 2 * u : u * V;
  }
  __device__ __forceinline__ int second(const RopeParams& p) const {
    return V == 1 && INTER ? 2 * u + 1 : p.rot / 2 + u * V;
  }
  __device__ __forceinline__ void load(const RopeParams& p) {
    a = *reinterpret_cast<const Pack<S, V>*>(x + first(p));
    if (u < p.turn_units) b = *reinterpret_cast<const Pack<S, V>*>(x + second(p));
  }
  __device__ __forceinline__ static void turn_pair(float2 cs, S& p, S& q) {
    const float sn = INV ? -cs.y : cs.y, fa = (float)p, fb = (float)q;
    p = (S)(fa * cs.x - fb * sn);
    q = (S)(fb * cs.x + fa * sn);
  }
  __device__ __forceinline__ void finish(const RopeParams& p) {
    if (turn && !zero) {
      const float2* t = p.table + (int64_t)pos * (p.rot / 2);
      if constexpr (INTER && V > 1) {
        const Pack<float2, V / 2> ca = *reinterpret_cast<const Pack<float2, V / 2>*>(t + u * (V / 2));
        const Pack<float2, V / 2> cb =
            *reinterpret_cast<const Pack<float2, V / 2>*>(t + p.rot / 4 + u * (V / 2));
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          turn_pair(ca.v[i], a.v[2 * i], a.v[2 * i + 1]);
          turn_pair(cb.v[i], b.v[2 * i], b.v[2 * i + 1]);
        }
      } else {
        const Pack<float2, V> c = *reinterpret_cast<const Pack<float2, V>*>(t + u * V);
#pragma unroll
        for (int i = 0; i < V; ++i) turn_pair(c.v[i], a.v[i], b.v[i]);
      }
    }
    if (zero) {
#pragma unroll
      for (int i = 0; i < V; ++i) a.v[i] = b.v[i] = (S)0.f;
    }
    if (!y) return;
    *reinterpret_cast<Pack<S, V>*>(y + first(p)) = a;
    if (u < p.turn_units) *reinterpret_cast<Pack<S, V>*>(y + second(p)) = b;
  }
};

// RPT rows per thread, their loads issued together.
template <class S, int V, bool INTER, bool INV, bool APPEND, int RPT>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeParams p) {
  const int slots = kRopeThreads / p.units > 0 ? kRopeThreads / p.units : 1;
  const int slot = threadIdx.x / p.units;
  for (int unit = threadIdx.x % p.units; unit < p.units; unit += kRopeThreads) {
    if (slot >= slots) break;
    RopeItem<S, V, INTER, INV, APPEND> it[RPT];
    const uint64_t row0 = (uint64_t)blockIdx.x * (slots * RPT) + slot;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const uint64_t row = row0 + (uint64_t)i * slots;
      if (row < p.rows) {
        it[i].locate(p, (uint32_t)row, unit);
        it[i].load(p);
      }
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i)
      if (row0 + (uint64_t)i * slots < p.rows) it[i].finish(p);
  }
}

template <class S, int V, bool INTER, bool INV, bool APPEND>
hipError_t launch_rows(const RopeParams& p, hipStream_t s) {
  const int slots = kRopeThreads / p.units > 0 ? kRopeThreads / p.units : 1;
  const int64_t one = ((int64_t)p.rows + slots - 1) / slots;
  if (one >= 8 * device_cus()) {
    hipLaunchKernelGGL((rope_kernel<S, V, INTER, INV, APPEND, 4>), dim3((uint32_t)((one + 3) / 4)),
                       dim3(kRopeThreads), 0, s, p);
  } else {
    hipLaunchKernelGGL((rope_kernel<S, V, INTER, INV, APPEND, 1>), dim3((uint32_t)one),
                       dim3(kRopeThreads), 0, s, p);
  }
  return hipGetLastError();
}

template <class S, int V>
hipError_t launch_kind(const RopeParams& p, bool inter, bool inv, bool append, hipStream_t s) {
  if (append) {
    if constexpr (sizeof(S) == 2)
      return inter ? launch_rows<S, V, true, false, true>(p, s)
                   : launch_rows<S, V, false, false, true>(p, s);
    return hipErrorInvalidValue;  // refused by the caller
  }
  if (inter)
    return inv ? launch_rows<S, V, true, true, false>(p, s)
               : launch_rows<S, V, true, false, false>(p, s);
  return inv ? launch_rows<S, V, false, true, false>(p, s)
             : launch_rows<S, V, false, false, false>(p, s);
}

// Whether vectors of V numbers of `size` bytes fit every address involved.
bool fits(const RopeArgs& a, int V, int size) {
  auto m = [&](int64_t n) { return n % V == 0; };
  auto al = [&](const void* q, int64_t bytes) {
    return reinterpret_cast<uintptr_t>(q) % bytes == 0;
  };
  if (!m(a.rot / 2) || !m(a.D - a.rot) || !m(a.x_tok) || !m(a.x_head) || !m(a.y_tok) ||
      !m(a.y_head) || !al(a.X, V * size) || !al(a.Y, V * size) || !al(a.table, 16))
    return false;
  return !a.k_pages || (m(a.page_stride) && m(a.row_stride) && m(a.head_stride) &&
                        al(a.k_pages, V * size) && al(a.v_pages, V * size));
}

}  // namespace

hipError_t launch_rope(int dtype, const RopeArgs& a, hipStream_t stream) {
  const int size = dtype == TQ_F32 ? 4 : 2;
  int V = 16 / size;
  while (V > 1 && !fits(a, V, size)) V = V == 8 ? 4 : 1;
  RopeParams p{};
  p.X = static_cast<const unsigned char*>(a.X);
  p.Y = static_cast<unsigned char*>(a.Y);
  p.x_tok = a.x_tok;
  p.x_head = a.x_head;
  p.y_tok = a.y_tok;
  p.y_head = a.y_head;
  p.table = reinterpret_cast<const float2*>(a.table);
  p.pos = a.pos;
  p.n_pos = (uint32_t)a.n_pos;
  p.rows = (uint32_t)(a.T * a.H);
  p.rot = (int32_t)a.rot;
  p.D = (int32_t)a.D;
  p.turn_units = (int32_t)(a.rot / 2 / V);
  p.units = p.turn_units + (int32_t)((a.D - a.rot) / V);
  p.heads = Div31::of(a.H);
  const bool append = a.k_pages != nullptr;
  if (append) {
    p.Hq = (int32_t)a.Hq;
    p.Hkv = (int32_t)a.Hkv;
    p.K = static_cast<unsigned char*>(a.k_pages);
    p.Vp = static_cast<unsigned char*>(a.v_pages);
    p.page_stride = a.page_stride;
    p.row_stride = a.row_stride;
    p.head_stride = a.head_stride;
    p.page = Div31::of(a.page_size);
    p.n_pages = (uint32_t)a.n_pages;
    p.width = (uint32_t)a.width;
    p.n_seqs = (uint32_t)a.n_seqs;
    p.page_table = a.page_table;
    p.seqs = a.seqs;
  }
  const bool inter = a.interleaved, inv = a.inverse;
  if (dtype == TQ_F32)
    return V == 4 ? launch_kind<float, 4>(p, inter, inv, append, stream)
                  : launch_kind<float, 1>(p, inter, inv, append, stream);
  if (dtype == TQ_BF16)
    return V == 8   ? launch_kind<__bf16, 8>(p, inter, inv, append, stream)
           : V == 4 ? launch_kind<__bf16, 4>(p, inter, inv, append, stream)
                    : launch_kind<__bf16, 1>(p, inter, inv, append, stream);
  return V == 8   ? launch_kind<_Float16, 8>(p, inter, inv, append, stream)
         : V == 4 ? launch_kind<_Float16, 4>(p, inter, inv, append, stream)
                  : launch_kind<_Float16, 1>(p, inter, inv, append, stream);
}

}  // namespace tq
