// What the kernels that read a paged key-value cache share: divisions by the page
// size, 16-bit weights, reads of what a call does not write, and the cut of a list of
// tiles into equal runs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "tq_common.h"
#include "tq_mfma.h"

namespace tq {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef float float2v __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f;

// t / d for 0 <= t < 2^30: exact with m = ceil(2^(30 + s) / d), s = ceil(log2 d).
struct FastDiv {
  uint32_t d, m, shift;
};

// Two floats x >= 0 as two 16-bit numbers each (low half first): x cut, and what
// that left of it, rounded to nearest, so that the errors of many weights do not add
// up to one side: hi + lo is within 2^-22 (fp16, normal range) or 2^-16 (bf16) of x.
// The first is cut, not rounded, for the second to have no sign, and the second is
// no less than `least` wherever x is not: an infinite value times them then stays
// infinite instead of becoming NaN.  Below that x has one number only, or none: a
// token without weight adds nothing, however large its value.  `least`: 2^-126 in
// bf16 (the least weight there is); in fp16 the type's own 2^-24, so that a weight that one
// number holds is off by as much: of a row's largest, which its caller scales to 2^14 (or to
// 2^9 at least), 2^-38 (2^-33).
template <bool BF>
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  constexpr float least = BF ? 0x1p-126f : 0x1p-24f;
  float xh, yh;
  if constexpr (BF) {
    const uint32_t xb = __builtin_bit_cast(uint32_t, x), yb = __builtin_bit_cast(uint32_t, y);
    hi = __builtin_amdgcn_perm(yb, xb, 0x07060302u);
    xh = __builtin_bit_cast(float, xb & 0xffff0000u);
    yh = __builtin_bit_cast(float, yb & 0xffff0000u);
  } else {
    const auto h = __builtin_amdgcn_cvt_pkrtz(x, y);
    hi = __builtin_bit_cast(uint32_t, h);
    xh = (float)h[0];
    yh = (float)h[1];
  }
  const float2v rest = {__builtin_amdgcn_fmed3f(x - xh, least, x),
                        __builtin_amdgcn_fmed3f(y - yh, least, y)};
  using half2 = std::conditional_t<BF, bf2, half2v>;
  lo = __builtin_bit_cast(uint32_t, __builtin_convertvector(rest, half2));
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

// A value that every lane holds, as the scalar it is.
__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A value that the compiler takes for a new one: what follows from it is computed where it
// stands, instead of being kept in registers through the whole loop.
__device__ __forceinline__ int anew(int v) {
  asm volatile("" : "+v"(v));
  return v;
}
__device__ __forceinline__ int anew_uniform(int v) {
  asm volatile("" : "+s"(v));
  return v;
}

// Reads of what no kernel of a call writes, through the scalar cache where the
// index is uniform.
typedef const __attribute__((address_space(4))) int32_t* const_i32;
__device__ __forceinline__ int32_t read_const(const int32_t* p, int64_t i) {
  return ((const_i32)(uint64_t)p)[i];
}

// The flattened list of `units` tiles (sequence, then head, then tile) cut into
// `parts` runs of q or, the first r of them, q + 1 tiles: one for each wave or workgroup.
struct Cut {
  uint32_t units, parts, q, r;
  __device__ __forceinline__ Cut(uint32_t n, uint32_t most) {
    units = n;
    parts = n < most ? n : most;
    q = parts ? n / parts : 0;
    r = n - parts * q;
  }
  __device__ __forceinline__ uint32_t start(uint32_t i) const { return i * q + (i < r ? i : r); }
  __device__ __forceinline__ uint32_t part_of(uint32_t unit) const {
    const uint32_t wide = r * (q + 1);
    return unit < wide ? unit / (q + 1) : r + (unit - wide) / q;
  }
};

// Sum over this lane and those before it.
__device__ __forceinline__ uint32_t scan_wave(uint32_t v, int lane) {
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const uint32_t o = __shfl_up(v, off, kWave);
    v += lane >= off ? o : 0;
  }
  return v;
}

inline FastDiv fast_div(int64_t d) {
  uint32_t s = 0;
  while ((int64_t(1) << s) < d) ++s;
  const uint64_t m = ((uint64_t(1) << (30 + s)) + d - 1) / d;
  return {(uint32_t)d, (uint32_t)m, 30 + s};
}

constexpr uint32_t kOut = 0x80000000u;   // a lane offset past every buffer
constexpr uint32_t kSpan = 0x7ffffffcu;  // bytes a buffer resource covers

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_at(const unsigned char* p) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(((uint64_t)hi << 32) | lo),
                                           (short)0, (int)kSpan, kBufferWord3);
}

}  // namespace tq
