// Internal launchers of the decode-side kernels: rotary positions, attention
// over a paged cache, page bookkeeping.  Callers (tq_decode_api.hip) have
// already validated every argument.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tq {

// Strides in elements.
struct RopeArgs {
  const void* X;  // [T][H][D], H = Hq + Hkv rotated heads, then Hkv copied ones when appending
  int64_t x_tok, x_head;
  void* Y;  // rotated heads (appending: the query heads only)
  int64_t y_tok, y_head;
  const float* table;  // [n_pos][rot / 2][2]: cos, sin
  int64_t n_pos, rot;
  const int32_t* pos;  // [T]
  int64_t T, D;
  int interleaved, inverse;
  int64_t H;  // heads of X that this call touches
  // appending only (k_pages != nullptr)
  int64_t Hq, Hkv;
  void* k_pages;
  void* v_pages;
  int64_t n_pages, page_size, page_stride, row_stride, head_stride;
  const int32_t* page_table;  // [n_seqs][width]
  int64_t width, n_seqs;
  const int32_t* seqs;  // [T] or nullptr: token t belongs to sequence t
};
hipError_t launch_rope(int dtype, const RopeArgs& a, hipStream_t stream);

struct AttnArgs {
  const void* Q;
  int64_t q_tok, q_head;
  const void* k_pages;
  const void* v_pages;
  int64_t n_pages, page_size, page_stride, row_stride, head_stride;
  const int32_t* page_table;  // [B][width]
  int64_t width;
  const int32_t* lens;  // [B]
  int64_t B, Hq, Hkv, D;
  float scale_log2;  // score scale times log2(e)
  int64_t window;
  void* Out;   // [B][Hq][D]
  float* lse;  // [B][Hq] or nullptr
  void* workspace;
};
int64_t attn_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t capacity);
hipError_t launch_paged_attention(int dtype, const AttnArgs& a, hipStream_t stream);

// Page bookkeeping.  A sequence of `len` tokens holds the first
// ceil(len / page_size) entries of its row of the page table.
struct PagesArgs {
  unsigned char* pool;  // [planes][n_pages][page_bytes]
  int64_t planes, n_pages, page_bytes, page_size;
  const int32_t* table;  // [rows_in][width]
  const int32_t* lens;   // [rows_in]
  int64_t rows_in, rows, width;
  const int32_t* parent;  // fork: [rows]
  const int32_t* add;     // grow: [rows]
  int32_t* table_out;     // [rows][width]
  int32_t* lens_out;      // [rows]
  int32_t* refs;          // [n_pages] or nullptr
  int32_t* result;        // fork, grow: pages short; compact: pages in use
  void* workspace;
};
int64_t pages_workspace_bytes(int64_t rows, int64_t n_pages);
hipError_t launch_pages_fork(const PagesArgs& a, hipStream_t stream);
hipError_t launch_pages_grow(const PagesArgs& a, hipStream_t stream);
hipError_t launch_pages_compact(const PagesArgs& a, hipStream_t stream);
hipError_t launch_pages_copy(unsigned char* pool, int64_t planes, int64_t n_pages,
                             int64_t page_bytes, const int32_t* src, const int32_t* dst, int64_t n,
                             hipStream_t stream);

}  // namespace tq
