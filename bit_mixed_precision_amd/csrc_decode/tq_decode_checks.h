// Argument checks that the decode-side entry points share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tq.h"

namespace tq {
namespace checks {

constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int64_t kMaxHeadDim = int64_t(1) << 16;
constexpr int64_t kMaxHeads = int64_t(1) << 16;
constexpr int64_t kMaxStride = int64_t(1) << 46;  // elements
// Elements that the steps of one dimension may span: the byte offsets of three
// dimensions of four-byte numbers add up to less than 2^62.
constexpr int64_t kMaxReach = int64_t(1) << 58;
constexpr int64_t kMaxAttnBatch = int64_t(1) << 20;
constexpr int64_t kMaxAttnHeads = int64_t(1) << 12;
constexpr int64_t kMaxRowStride = int64_t(1) << 24;  // 16 rows within 32-bit buffer offsets
constexpr int64_t kMaxPages = int64_t(1) << 24;
constexpr int64_t kMaxRows = int64_t(1) << 16;
constexpr int64_t kMaxPlanes = int64_t(1) << 16;
constexpr int64_t kMaxPageBytes = int64_t(1) << 30;

inline bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
// The stride of a dimension of one entry is never taken: whatever a caller has there
// (a view of a tensor may hold any number) stands for 0.
inline int64_t step(int64_t n, int64_t s) { return n == 1 ? 0 : s; }

// Stride s of a dimension of n >= 1 entries.
inline bool stride_ok(int64_t n, int64_t s) {
  return s >= 0 && s <= kMaxStride && s <= kMaxReach / n;
}

inline int device_ready() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) {
    (void)hipGetLastError();
    return TQ_ERR_DEVICE;
  }
  return TQ_OK;
}

inline int finish(hipError_t e) {
  if (e != hipSuccess) {
    (void)hipGetLastError();
    return TQ_ERR_DEVICE;
  }
  return TQ_OK;
}

// No two of n1 x n2 runs of `len` elements at strides s1, s2 (stride_ok) share an
// element.
inline bool distinct(int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t len) {
  if (n1 == 1) s1 = kMaxStride;  // a stride that is never taken
  if (n2 == 1) s2 = kMaxStride;
  const int64_t small = s1 < s2 ? s1 : s2, large = s1 < s2 ? s2 : s1;
  const int64_t n_small = s1 < s2 ? n1 : n2, n_large = s1 < s2 ? n2 : n1;
  if (n_small > 1 && small < len) return false;
  const int64_t run = n_small > 1 ? small * (n_small - 1) + len : len;
  return n_large == 1 || large >= run;
}

// The same for the heads of the slots of the pages of a cache, whose strides are
// nested in some order.
inline bool distinct_cache(int64_t n_pages, int64_t page, int64_t page_size, int64_t row,
                           int64_t heads, int64_t head, int64_t len) {
  struct Level {
    int64_t n, stride;
  } l[3] = {{n_pages, page}, {page_size, row}, {heads, head}};
  int64_t reach = len;  // elements from the first to past the last so far
  bool done[3] = {l[0].n == 1, l[1].n == 1, l[2].n == 1};
  for (int i = 0; i < 3; ++i) {
    int least = -1;
    for (int k = 0; k < 3; ++k)
      if (!done[k] && (least < 0 || l[k].stride < l[least].stride)) least = k;
    if (least < 0) break;
    if (l[least].stride < reach) return false;
    reach += l[least].stride * (l[least].n - 1);
    done[least] = true;
  }
  return true;
}

inline int rope_shapes(int64_t n_pos, int64_t rot, int64_t T, int64_t H, int64_t D) {
  if (n_pos < 0 || n_pos > kMaxTokens || D > kMaxHeadDim || rot < 2 || rot % 2 || rot > D ||
      T > kMaxTokens || H > kMaxHeads || T * H > INT32_MAX)
    return TQ_ERR_SHAPE;
  return TQ_OK;
}

inline int pages_shapes(int64_t n_pages, int64_t rows, int64_t width, int64_t page_size) {
  if (n_pages < 1 || n_pages > kMaxPages || rows < 0 || rows > kMaxRows || width < 1 ||
      page_size < 1 || width > kMaxTokens || page_size > kMaxTokens ||
      width * page_size > kMaxTokens)
    return TQ_ERR_SHAPE;
  return TQ_OK;
}

inline int pool_shapes(int64_t planes, int64_t page_bytes) {
  return planes < 0 || planes > kMaxPlanes || page_bytes < 16 || page_bytes % 16 ||
                 page_bytes > kMaxPageBytes
             ? TQ_ERR_SHAPE
             : TQ_OK;
}

inline int attn_shapes(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t page_size,
                       int64_t width) {
  if (B < 0 || B > kMaxAttnBatch || Hkv < 1 || Hq < 1 || Hq > kMaxAttnHeads || Hq % Hkv || D < 8 ||
      D > 256 || D % 8 || page_size < 1 || width < 1 || page_size > kMaxTokens ||
      width > kMaxTokens || width * page_size > kMaxTokens)
    return TQ_ERR_SHAPE;
  // the kernels count all tiles (32 tokens of one key-value head) in 32 bits
  const int64_t rows = B * Hkv * ((Hq / Hkv + 15) / 16);
  if (rows > INT32_MAX || rows * (width * page_size / 32 + 2) > INT32_MAX) return TQ_ERR_SHAPE;
  return TQ_OK;
}

}  // namespace checks
}  // namespace tq
