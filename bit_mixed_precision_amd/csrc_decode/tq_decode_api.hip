// C ABI of the decode-side operators (include/tq.h): argument checks.

#include <float.h>
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "tq.h"
#include "tq_decode.h"

namespace {

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

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
// The stride of a dimension of one entry is never taken: whatever a caller has there
// (a view of a tensor may hold any number) stands for 0.
int64_t step(int64_t n, int64_t s) { return n == 1 ? 0 : s; }

// Stride s of a dimension of n >= 1 entries.
bool stride_ok(int64_t n, int64_t s) { return s >= 0 && s <= kMaxStride && s <= kMaxReach / n; }

int device_ready() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) {
    (void)hipGetLastError();
    return TQ_ERR_DEVICE;
  }
  return TQ_OK;
}

int finish(hipError_t e) {
  if (e != hipSuccess) {
    (void)hipGetLastError();
    return TQ_ERR_DEVICE;
  }
  return TQ_OK;
}

// No two of n1 x n2 runs of `len` elements at strides s1, s2 (stride_ok) share an
// element.
bool distinct(int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t len) {
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
bool distinct_cache(int64_t n_pages, int64_t page, int64_t page_size, int64_t row, int64_t heads,
                    int64_t head, int64_t len) {
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

int rope_shapes(int64_t n_pos, int64_t rot, int64_t T, int64_t H, int64_t D) {
  if (n_pos < 0 || n_pos > kMaxTokens || D > kMaxHeadDim || rot < 2 || rot % 2 || rot > D ||
      T > kMaxTokens || H > kMaxHeads || T * H > INT32_MAX)
    return TQ_ERR_SHAPE;
  return TQ_OK;
}

int pages_shapes(int64_t n_pages, int64_t rows, int64_t width, int64_t page_size) {
  if (n_pages < 1 || n_pages > kMaxPages || rows < 0 || rows > kMaxRows || width < 1 ||
      page_size < 1 || width > kMaxTokens || page_size > kMaxTokens ||
      width * page_size > kMaxTokens)
    return TQ_ERR_SHAPE;
  return TQ_OK;
}

int pool_shapes(int64_t planes, int64_t page_bytes) {
  return planes < 0 || planes > kMaxPlanes || page_bytes < 16 || page_bytes % 16 ||
                 page_bytes > kMaxPageBytes
             ? TQ_ERR_SHAPE
             : TQ_OK;
}

int attn_shapes(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t page_size, int64_t width) {
  if (B < 0 || B > kMaxAttnBatch || Hkv < 1 || Hq < 1 || Hq > kMaxAttnHeads || Hq % Hkv || D < 8 ||
      D > 256 || D % 8 || page_size < 1 || width < 1 || page_size > kMaxTokens ||
      width > kMaxTokens || width * page_size > kMaxTokens)
    return TQ_ERR_SHAPE;
  // the kernels count all tiles (32 tokens of one key-value head) in 32 bits
  const int64_t rows = B * Hkv * ((Hq / Hkv + 15) / 16);
  if (rows > INT32_MAX || rows * (width * page_size / 32 + 2) > INT32_MAX) return TQ_ERR_SHAPE;
  return TQ_OK;
}

}  // namespace

extern "C" {

int tq_rope(int dtype, const void* X, int64_t x_tok, int64_t x_head, void* Y, int64_t y_tok,
            int64_t y_head, const float* table, int64_t n_pos, int64_t rot, const int32_t* pos,
            int64_t T, int64_t H, int64_t D, int interleaved, int inverse, void* stream) {
  if (T < 0 || H < 0) return TQ_ERR_SHAPE;
  if (T == 0 || H == 0) return TQ_OK;
  if (!X || !Y || (!table && n_pos != 0) || !pos) return TQ_ERR_NULL;
  int st = rope_shapes(n_pos, rot, T, H, D);
  if (st != TQ_OK) return st;
  x_tok = step(T, x_tok);
  x_head = step(H, x_head);
  y_tok = step(T, y_tok);
  y_head = step(H, y_head);
  if (!stride_ok(T, x_tok) || !stride_ok(H, x_head) || !stride_ok(T, y_tok) ||
      !stride_ok(H, y_head) || !distinct(T, y_tok, H, y_head, D))
    return TQ_ERR_SHAPE;
  if (X == Y && (x_tok != y_tok || x_head != y_head)) return TQ_ERR_SHAPE;
  const uintptr_t size = dtype == TQ_F32 ? 4 : 2;
  if (!aligned(X, size) || !aligned(Y, size) || !aligned(table, 8) || !aligned(pos, 4))
    return TQ_ERR_ALIGN;
  if (dtype < TQ_F16 || dtype > TQ_F32 || (interleaved & ~1) || (inverse & ~1))
    return TQ_ERR_VALUE;
  st = device_ready();
  if (st != TQ_OK) return st;
  tq::RopeArgs a{};
  a.X = X;
  a.x_tok = x_tok;
  a.x_head = x_head;
  a.Y = Y;
  a.y_tok = y_tok;
  a.y_head = y_head;
  a.table = table;
  a.n_pos = n_pos;
  a.rot = rot;
  a.pos = pos;
  a.T = T;
  a.H = H;
  a.D = D;
  a.interleaved = interleaved;
  a.inverse = inverse;
  return finish(tq::launch_rope(dtype, a, static_cast<hipStream_t>(stream)));
}

int tq_rope_append(int dtype, const void* QKV, int64_t qkv_tok, const float* table, int64_t n_pos,
                   int64_t rot, const int32_t* pos, const int32_t* seqs, const int32_t* page_table,
                   int64_t n_seqs, int64_t width, void* k_pages, void* v_pages, int64_t n_pages,
                   int64_t page_size, int64_t page_stride, int64_t row_stride,
                   int64_t head_stride, void* Q, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                   int interleaved, void* stream) {
  if (T < 0) return TQ_ERR_SHAPE;
  if (T == 0) return TQ_OK;
  if (!QKV || (!table && n_pos != 0) || !pos || !page_table || !k_pages || !v_pages || !Q) return TQ_ERR_NULL;
  if (Hq < 1 || Hkv < 1 || Hq > kMaxHeads || Hkv > kMaxHeads) return TQ_ERR_SHAPE;
  int st = rope_shapes(n_pos, rot, T, Hq + 2 * Hkv, D);
  if (st != TQ_OK) return st;
  qkv_tok = step(T, qkv_tok);
  page_stride = step(n_pages, page_stride);
  row_stride = step(page_size, row_stride);
  head_stride = step(Hkv, head_stride);
  if (n_pages < 1 || n_pages > INT32_MAX || n_seqs < 1 || n_seqs > INT32_MAX || width < 1 ||
      page_size < 1 || width > kMaxTokens || page_size > kMaxTokens ||
      width * page_size > kMaxTokens || !stride_ok(T, qkv_tok) ||
      !stride_ok(n_pages, page_stride) || !stride_ok(page_size, row_stride) ||
      !stride_ok(Hkv, head_stride) ||
      !distinct_cache(n_pages, page_stride, page_size, row_stride, Hkv, head_stride, D))
    return TQ_ERR_SHAPE;
  if (!aligned(QKV, 2) || !aligned(Q, 2) || !aligned(k_pages, 2) || !aligned(v_pages, 2) ||
      !aligned(table, 8) || !aligned(pos, 4) || !aligned(seqs, 4) || !aligned(page_table, 4))
    return TQ_ERR_ALIGN;
  if ((dtype != TQ_F16 && dtype != TQ_BF16) || (interleaved & ~1)) return TQ_ERR_VALUE;
  st = device_ready();
  if (st != TQ_OK) return st;
  tq::RopeArgs a{};
  a.X = QKV;
  a.x_tok = qkv_tok;
  a.x_head = D;
  a.Y = Q;
  a.y_tok = Hq * D;
  a.y_head = D;
  a.table = table;
  a.n_pos = n_pos;
  a.rot = rot;
  a.pos = pos;
  a.T = T;
  a.H = Hq + 2 * Hkv;
  a.D = D;
  a.interleaved = interleaved;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.n_pages = n_pages;
  a.page_size = page_size;
  a.page_stride = page_stride;
  a.row_stride = row_stride;
  a.head_stride = head_stride;
  a.page_table = page_table;
  a.width = width;
  a.n_seqs = n_seqs;
  a.seqs = seqs;
  return finish(tq::launch_rope(dtype, a, static_cast<hipStream_t>(stream)));
}

int64_t tq_paged_attention_workspace(int64_t B, int64_t Hq, int64_t Hkv, int64_t D,
                                     int64_t page_size, int64_t width) {
  if (attn_shapes(B, Hq, Hkv, D, page_size, width) != TQ_OK) return TQ_ERR_SHAPE;
  return B == 0 ? 0 : tq::attn_workspace_bytes(B, Hq, Hkv, D, width * page_size);
}

int tq_paged_attention(int dtype, const void* Q, int64_t q_tok, int64_t q_head,
                       const void* k_pages, const void* v_pages, int64_t n_pages,
                       int64_t page_size, int64_t page_stride, int64_t row_stride,
                       int64_t head_stride, const int32_t* page_table, int64_t width,
                       const int32_t* lens, int64_t B, int64_t Hq, int64_t Hkv, int64_t D,
                       double scale, int64_t window, void* Out, float* lse, void* workspace,
                       int64_t workspace_bytes, void* stream) {
  if (B < 0) return TQ_ERR_SHAPE;
  if (B == 0) return TQ_OK;
  if (!Q || !k_pages || !v_pages || !page_table || !lens || !Out) return TQ_ERR_NULL;
  int st = attn_shapes(B, Hq, Hkv, D, page_size, width);
  if (st != TQ_OK) return st;
  q_tok = step(B, q_tok);
  q_head = step(Hq, q_head);
  page_stride = step(n_pages, page_stride);
  row_stride = step(page_size, row_stride);
  head_stride = step(Hkv, head_stride);
  if (n_pages < 1 || n_pages > INT32_MAX || !stride_ok(B, q_tok) || !stride_ok(Hq, q_head) ||
      !stride_ok(n_pages, page_stride) || !stride_ok(page_size, row_stride) ||
      !stride_ok(Hkv, head_stride) || row_stride > kMaxRowStride || q_tok % 8 || q_head % 8 ||
      page_stride % 8 || row_stride % 8 || head_stride % 8)
    return TQ_ERR_SHAPE;
  const int64_t wants = tq::attn_workspace_bytes(B, Hq, Hkv, D, width * page_size);
  if (workspace_bytes < wants) return TQ_ERR_SHAPE;
  if (wants > 0 && !workspace) return TQ_ERR_NULL;
  if (!aligned(Q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(Out, 16) ||
      !aligned(workspace, 16) || !aligned(page_table, 4) || !aligned(lens, 4) || !aligned(lse, 4))
    return TQ_ERR_ALIGN;
  const double scale_log2 = scale * 1.4426950408889634;  // the kernels hold it in fp32
  if ((dtype != TQ_F16 && dtype != TQ_BF16) || !(fabs(scale_log2) <= FLT_MAX) || window < 0)
    return TQ_ERR_VALUE;
  st = device_ready();
  if (st != TQ_OK) return st;
  tq::AttnArgs a{};
  a.Q = Q;
  a.q_tok = q_tok;
  a.q_head = q_head;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.n_pages = n_pages;
  a.page_size = page_size;
  a.page_stride = page_stride;
  a.row_stride = row_stride;
  a.head_stride = head_stride;
  a.page_table = page_table;
  a.width = width;
  a.lens = lens;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  a.scale_log2 = (float)scale_log2;
  a.window = window > INT32_MAX ? 0 : window;  // longer than any sequence
  a.Out = Out;
  a.lse = lse;
  a.workspace = workspace;
  return finish(tq::launch_paged_attention(dtype, a, static_cast<hipStream_t>(stream)));
}

int64_t tq_pages_workspace(int64_t rows, int64_t n_pages) {
  if (pages_shapes(n_pages, rows, 1, 1) != TQ_OK) return TQ_ERR_SHAPE;
  return tq::pages_workspace_bytes(rows, n_pages);
}

int tq_pages_fork(void* pool, int64_t planes, int64_t n_pages, int64_t page_bytes,
                  const int32_t* table, const int32_t* lens, int64_t rows_in,
                  const int32_t* parent, int64_t rows, int64_t width, int64_t page_size,
                  int32_t* table_out, int32_t* lens_out, int32_t* refs, int32_t* short_out,
                  void* workspace, int64_t workspace_bytes, void* stream) {
  if (rows < 0 || rows_in < 0) return TQ_ERR_SHAPE;
  if ((rows > 0 && (!parent || !table_out || !lens_out)) || !short_out || !workspace ||
      (rows_in > 0 && (!table || !lens)) || (planes > 0 && !pool))
    return TQ_ERR_NULL;
  int st = pages_shapes(n_pages, rows, width, page_size);
  if (st != TQ_OK || (st = pool_shapes(planes, page_bytes)) != TQ_OK) return st;
  if (rows_in > kMaxRows || workspace_bytes < tq::pages_workspace_bytes(rows, n_pages))
    return TQ_ERR_SHAPE;
  if (!aligned(pool, 16) || !aligned(workspace, 16) || !aligned(table, 4) || !aligned(lens, 4) ||
      !aligned(parent, 4) || !aligned(table_out, 4) || !aligned(lens_out, 4) ||
      !aligned(refs, 4) || !aligned(short_out, 4))
    return TQ_ERR_ALIGN;
  st = device_ready();
  if (st != TQ_OK) return st;
  tq::PagesArgs a{};
  a.pool = static_cast<unsigned char*>(pool);
  a.planes = planes;
  a.n_pages = n_pages;
  a.page_bytes = page_bytes;
  a.page_size = page_size;
  a.table = table;
  a.lens = lens;
  a.rows_in = rows_in;
  a.rows = rows;
  a.width = width;
  a.parent = parent;
  a.table_out = table_out;
  a.lens_out = lens_out;
  a.refs = refs;
  a.result = short_out;
  a.workspace = workspace;
  return finish(tq::launch_pages_fork(a, static_cast<hipStream_t>(stream)));
}

int tq_pages_grow(const int32_t* table, const int32_t* lens, const int32_t* add, int64_t rows,
                  int64_t width, int64_t page_size, int64_t n_pages, int32_t* table_out,
                  int32_t* lens_out, int32_t* short_out, void* workspace,
                  int64_t workspace_bytes, void* stream) {
  if (rows < 0) return TQ_ERR_SHAPE;
  if ((rows > 0 && (!table || !lens || !add || !table_out || !lens_out)) || !short_out ||
      !workspace)
    return TQ_ERR_NULL;
  int st = pages_shapes(n_pages, rows, width, page_size);
  if (st != TQ_OK) return st;
  if (workspace_bytes < tq::pages_workspace_bytes(rows, n_pages)) return TQ_ERR_SHAPE;
  if (!aligned(workspace, 16) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(add, 4) ||
      !aligned(table_out, 4) || !aligned(lens_out, 4) || !aligned(short_out, 4))
    return TQ_ERR_ALIGN;
  st = device_ready();
  if (st != TQ_OK) return st;
  tq::PagesArgs a{};
  a.n_pages = n_pages;
  a.page_size = page_size;
  a.table = table;
  a.lens = lens;
  a.add = add;
  a.rows_in = a.rows = rows;
  a.width = width;
  a.table_out = table_out;
  a.lens_out = lens_out;
  a.result = short_out;
  a.workspace = workspace;
  return finish(tq::launch_pages_grow(a, static_cast<hipStream_t>(stream)));
}

int tq_pages_compact(void* pool, int64_t planes, int64_t n_pages, int64_t page_bytes,
                     const int32_t* table, const int32_t* lens, int64_t rows, int64_t width,
                     int64_t page_size, int32_t* table_out, int32_t* used_out, void* workspace,
                     int64_t workspace_bytes, void* stream) {
  if (rows < 0) return TQ_ERR_SHAPE;
  if ((rows > 0 && (!table || !lens || !table_out)) || !used_out || !workspace ||
      (planes > 0 && !pool))
    return TQ_ERR_NULL;
  int st = pages_shapes(n_pages, rows, width, page_size);
  if (st != TQ_OK || (st = pool_shapes(planes, page_bytes)) != TQ_OK) return st;
  if (workspace_bytes < tq::pages_workspace_bytes(rows, n_pages)) return TQ_ERR_SHAPE;
  if (!aligned(pool, 16) || !aligned(workspace, 16) || !aligned(table, 4) || !aligned(lens, 4) ||
      !aligned(table_out, 4) || !aligned(used_out, 4))
    return TQ_ERR_ALIGN;
  st = device_ready();
  if (st != TQ_OK) return st;
  tq::PagesArgs a{};
  a.pool = static_cast<unsigned char*>(pool);
  a.planes = planes;
  a.n_pages = n_pages;
  a.page_bytes = page_bytes;
  a.page_size = page_size;
  a.table = table;
  a.lens = lens;
  a.rows_in = a.rows = rows;
  a.width = width;
  a.table_out = table_out;
  a.result = used_out;
  a.workspace = workspace;
  return finish(tq::launch_pages_compact(a, static_cast<hipStream_t>(stream)));
}

int tq_pages_copy(void* pool, int64_t planes, int64_t n_pages, int64_t page_bytes,
                  const int32_t* src, const int32_t* dst, int64_t n, void* stream) {
  if (n < 0 || planes < 0) return TQ_ERR_SHAPE;
  if (n == 0 || planes == 0) return TQ_OK;
  if (!pool || !src || !dst) return TQ_ERR_NULL;
  int st = pages_shapes(n_pages, 0, 1, 1);
  if (st != TQ_OK || (st = pool_shapes(planes, page_bytes)) != TQ_OK) return st;
  if (n > kMaxPages) return TQ_ERR_SHAPE;
  if (!aligned(pool, 16) || !aligned(src, 4) || !aligned(dst, 4)) return TQ_ERR_ALIGN;
  st = device_ready();
  if (st != TQ_OK) return st;
  return finish(tq::launch_pages_copy(static_cast<unsigned char*>(pool), planes, n_pages,
                                      page_bytes, src, dst, n, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
