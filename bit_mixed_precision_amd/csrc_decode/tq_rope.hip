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
// Tokens and their heads form one flattened list, so few heads or few tokens fill
// the lanes alike; with enough of both a thread takes two heads of its token for
// one reading of the table.
//
// Measured: 8192 tokens x 72 heads of 128 inside the rows of a q/k/v product, fp16,
// 306 MB: 53 us a call, 5.7 TB/s (a plain copy of 2 GiB reaches 4.9); 4093 x 40 x 80 in
// fp32, 105 MB: 18 us; appending 8192 tokens of 64 + 2 x 8 heads of 128, 335 MB: 60 us;
// one token 5.2 us, 251 tokens 5.3 us, both the launch.

#include "tq.h"
#include "tq_common.h"
#include "tq_decode.h"
#include "tq_kernels.h"

namespace tq {
namespace {

constexpr int kRopeThreads = 256;
constexpr int64_t kMostBlocks = int64_t(1) << 23;  // of one launch; more than the heads of a token

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
  uint32_t n_pos, rows, tok0;  // rows of this launch: tokens from tok0 x slots
  int32_t rot, H;
  int32_t turn_units, units;  // per head: turning, all
  Div31 slots;                // threads that share a token's heads
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

// Large calls (RPT > 1) store 16-byte pieces past the caches: what they write does
// not stay there anyway.  Measured (us, with / without): 8192 tokens x 72 heads of
// 128 in fp16 53 / 55, 16384 x 24 x 64 19 / 25, 4093 x 40 x 80 in fp32 18 / 20;
// 8-byte pieces (20 pairs of 80 numbers) 52 / 44, which therefore go the usual way.
template <int RPT, class S, int V>
__device__ __forceinline__ void store(S* to, const Pack<S, V>& v) {
  if constexpr (RPT > 1 && sizeof(S) * V == 16) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), reinterpret_cast<u32x4*>(to));
  } else {
    *reinterpret_cast<Pack<S, V>*>(to) = v;
  }
}

// One unit of RPT heads of a token: heads slot, slot + head_slots, ...  The
// token's cosines and sines are read once for all of them, after the heads.
template <class S, int V, bool INTER, bool INV, bool APPEND, int RPT>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeParams p) {
  const int slots = kRopeThreads / p.units > 0 ? kRopeThreads / p.units : 1;
  const int slot = threadIdx.x / p.units;
  const uint64_t at = (uint64_t)blockIdx.x * slots + slot;
  if (slot >= slots || at >= p.rows) return;
  const uint32_t in_launch = p.slots.quot((uint32_t)at);
  const int head0 = (int)((uint32_t)at - in_launch * p.slots.d);
  const uint32_t tok = p.tok0 + in_launch;
  const uint32_t pos = (uint32_t)p.pos[tok];
  const bool known = pos < p.n_pos;
  const S* x = reinterpret_cast<const S*>(p.X) + tok * p.x_tok;
  S* y = reinterpret_cast<S*>(p.Y) + tok * p.y_tok;
  int64_t slot_at = -1;  // appending: where the token's slot is in the cache
  if constexpr (APPEND) {
    const uint32_t seq = p.seqs ? (uint32_t)p.seqs[tok] : tok;
    const uint32_t pg = p.page.quot(known ? pos : 0);
    if (known && seq < p.n_seqs && pg < p.width) {
      const uint32_t id = (uint32_t)p.page_table[(int64_t)seq * p.width + pg];
      if (id < p.n_pages) slot_at = id * p.page_stride + (pos - pg * p.page.d) * p.row_stride;
    }
  }
  // more units than threads: a thread takes every 256th
  for (int u = threadIdx.x - slot * p.units; u < p.units; u += kRopeThreads) {
    const bool turns = u < p.turn_units;
    // numbers of the unit's two vectors; a copying unit has the first only
    const int first = !turns ? p.rot + (u - p.turn_units) * V : V == 1 && INTER ? 2 * u : u * V;
    const int second = !turns ? first : V == 1 && INTER ? 2 * u + 1 : p.rot / 2 + u * V;
    Pack<S, V> a[RPT], b[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int head = head0 + i * (int)p.slots.d;
      if (head < p.H) {
        a[i] = *reinterpret_cast<const Pack<S, V>*>(x + head * p.x_head + first);
        if (turns) b[i] = *reinterpret_cast<const Pack<S, V>*>(x + head * p.x_head + second);
      }
    }
    Pack<float2, V> cs;
    if (turns && known) {
      const float2* t = p.table + (int64_t)pos * (p.rot / 2);
      if constexpr (INTER && V > 1) {
        const auto lo = *reinterpret_cast<const Pack<float2, V / 2>*>(t + u * (V / 2));
        const auto hi = *reinterpret_cast<const Pack<float2, V / 2>*>(t + p.rot / 4 + u * (V / 2));
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          cs.v[i] = lo.v[i];
          cs.v[V / 2 + i] = hi.v[i];
        }
      } else {
        cs = *reinterpret_cast<const Pack<float2, V>*>(t + u * V);
      }
    }
    auto turn = [&](float2 c, S& m, S& n) {
      const float sn = INV ? -c.y : c.y, fm = (float)m, fn = (float)n;
      // which product is fused is said here, and the results are kept in fp32 until
      // their one conversion: every variant gives the same bits
      float r0 = fmaf(fm, c.x, -(fn * sn)), r1 = fmaf(fn, c.x, fm * sn);
      asm("" : "+v"(r0), "+v"(r1));
      m = (S)r0;
      n = (S)r1;
    };
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int head = head0 + i * (int)p.slots.d;
      if (head >= p.H) continue;
      S* to = y + head * p.y_head;
      bool rotate = turns, write = true;
      if constexpr (APPEND) {
        if (head >= p.Hq) {  // a key or a value
          const int kv = head - p.Hq;
          const bool key = kv < p.Hkv;
          rotate = turns && key;
          write = slot_at >= 0;
          to = reinterpret_cast<S*>(key ? p.K : p.Vp) + slot_at +
               (key ? kv : kv - p.Hkv) * p.head_stride;
        }
      }
      if (!known) {
#pragma unroll
        for (int e = 0; e < V; ++e) a[i].v[e] = b[i].v[e] = (S)0.f;
      } else if (rotate) {
        if constexpr (INTER && V > 1) {
#pragma unroll
          for (int e = 0; e < V / 2; ++e) {
            turn(cs.v[e], a[i].v[2 * e], a[i].v[2 * e + 1]);
            turn(cs.v[V / 2 + e], b[i].v[2 * e], b[i].v[2 * e + 1]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) turn(cs.v[e], a[i].v[e], b[i].v[e]);
        }
      }
      if (write) {
        store<RPT, S, V>(to + first, a[i]);
        if (turns) store<RPT, S, V>(to + second, b[i]);
      }
    }
  }
}

template <class S, int V, bool INTER, bool INV, bool APPEND, int RPT>
hipError_t launch_heads(RopeParams p, int64_t T, hipStream_t s) {
  const int64_t head_slots = (p.H + RPT - 1) / RPT;
  p.slots = Div31::of(head_slots);
  const int slots = kRopeThreads / p.units > 0 ? kRopeThreads / p.units : 1;
  // a launch holds fewer than 2^32 threads
  const int64_t most = (kMostBlocks * slots) / head_slots;
  for (int64_t t = 0; t < T; t += most) {
    p.tok0 = (uint32_t)t;
    p.rows = (uint32_t)((T - t < most ? T - t : most) * head_slots);
    hipLaunchKernelGGL((rope_kernel<S, V, INTER, INV, APPEND, RPT>),
                       dim3((uint32_t)((p.rows + (int64_t)slots - 1) / slots)),
                       dim3(kRopeThreads), 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Two heads a thread where that leaves the GPU full of waves.  Measured (us, 1 / 2 /
// 3 / 4 heads): 8192 tokens x 72 heads of 128 in fp16 67 / 55 / 57 / 61.
template <class S, int V, bool INTER, bool INV, bool APPEND>
hipError_t launch_rows(const RopeParams& p, int64_t T, hipStream_t s) {
  const int64_t waves = T * p.H * p.units / kWave;
  if (waves >= 128 * device_cus())
    return launch_heads<S, V, INTER, INV, APPEND, 2>(p, T, s);
  return launch_heads<S, V, INTER, INV, APPEND, 1>(p, T, s);
}

template <class S, int V>
hipError_t launch_kind(const RopeParams& p, int64_t T, bool inter, bool inv, bool append,
                       hipStream_t s) {
  if (append) {
    if constexpr (sizeof(S) == 2)
      return inter ? launch_rows<S, V, true, false, true>(p, T, s)
                   : launch_rows<S, V, false, false, true>(p, T, s);
    return hipErrorInvalidValue;  // refused by the caller
  }
  if (inter)
    return inv ? launch_rows<S, V, true, true, false>(p, T, s)
               : launch_rows<S, V, true, false, false>(p, T, s);
  return inv ? launch_rows<S, V, false, true, false>(p, T, s)
             : launch_rows<S, V, false, false, false>(p, T, s);
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
  p.rot = (int32_t)a.rot;
  p.H = (int32_t)a.H;
  p.turn_units = (int32_t)(a.rot / 2 / V);
  p.units = p.turn_units + (int32_t)((a.D - a.rot) / V);
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
    return V == 4 ? launch_kind<float, 4>(p, a.T, inter, inv, append, stream)
                  : launch_kind<float, 1>(p, a.T, inter, inv, append, stream);
  if (dtype == TQ_BF16)
    return V == 8   ? launch_kind<__bf16, 8>(p, a.T, inter, inv, append, stream)
           : V == 4 ? launch_kind<__bf16, 4>(p, a.T, inter, inv, append, stream)
                    : launch_kind<__bf16, 1>(p, a.T, inter, inv, append, stream);
  return V == 8   ? launch_kind<_Float16, 8>(p, a.T, inter, inv, append, stream)
         : V == 4 ? launch_kind<_Float16, 4>(p, a.T, inter, inv, append, stream)
                  : launch_kind<_Float16, 1>(p, a.T, inter, inv, append, stream);
}

}  // namespace tq
