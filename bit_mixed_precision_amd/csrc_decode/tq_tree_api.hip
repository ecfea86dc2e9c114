// C ABI of the operators on several new tokens per sequence (include/tq.h): argument
// checks.

#include <float.h>
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "tq.h"
#include "tq_decode.h"
#include "tq_decode_checks.h"

using namespace tq::checks;

namespace {

constexpr int64_t kMaxNodes = 256;

int tree_shapes(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t page_size,
                int64_t width) {
  if (T < 1 || T > kMaxNodes) return TQ_ERR_SHAPE;
  const int st = attn_shapes(B, Hq, Hkv, D, page_size, width);
  if (st != TQ_OK) return st;
  // the kernels count all tiles (64 tokens of 32 rows at least) in 32 bits, and a launch holds
  // fewer than 2^24 workgroups of 256 threads
  const int64_t blocks = B * Hkv * ((T * (Hq / Hkv) + 31) / 32);
  if (blocks >= int64_t(1) << 24 || blocks * (width * page_size / 64 + 2) > INT32_MAX)
    return TQ_ERR_SHAPE;
  return TQ_OK;
}

// Queries [B][T][Hq][D] and pages that attention reads: strides and their multiples of 8.
bool tree_strides(const tq::TreeArgs& a) {
  return a.n_pages >= 1 && a.n_pages <= INT32_MAX && stride_ok(a.B, a.q_seq) &&
         stride_ok(a.T, a.q_tok) && stride_ok(a.Hq, a.q_head) &&
         stride_ok(a.n_pages, a.page_stride) && stride_ok(a.page_size, a.row_stride) &&
         stride_ok(a.Hkv, a.head_stride) && a.row_stride <= kMaxRowStride && a.q_seq % 8 == 0 &&
         a.q_tok % 8 == 0 && a.q_head % 8 == 0 && a.page_stride % 8 == 0 &&
         a.row_stride % 8 == 0 && a.head_stride % 8 == 0;
}

constexpr int64_t kMaxSelectRows = (int64_t(1) << 22) - 1;  // of 1024 threads: fewer than 2^32
constexpr int64_t kMostWeightRows = 8192;  // their sums lie in LDS

}  // namespace

extern "C" {

int tq_tree_mask(const int32_t* parents, int64_t B, int64_t T, int64_t* mask, int32_t* depth,
                 void* stream) {
  if (B < 0 || T < 0) return TQ_ERR_SHAPE;
  if (B == 0 || T == 0) return TQ_OK;
  if (!parents || !mask) return TQ_ERR_NULL;
  if (B > kMaxAttnBatch || T > kMaxNodes) return TQ_ERR_SHAPE;
  if (!aligned(parents, 4) || !aligned(mask, 8) || !aligned(depth, 4)) return TQ_ERR_ALIGN;
  const int st = device_ready();
  if (st != TQ_OK) return st;
  return finish(tq::launch_tree_mask(parents, B, T, mask, depth, static_cast<hipStream_t>(stream)));
}

int64_t tq_tree_attention_workspace(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                                    int64_t page_size, int64_t width) {
  if (T == 0 && B >= 0) return 0;
  if (tree_shapes(B, T, Hq, Hkv, D, page_size, width) != TQ_OK) return TQ_ERR_SHAPE;
  return B == 0 ? 0 : tq::tree_workspace_bytes(B, T, Hq, Hkv, D, width * page_size);
}

int tq_tree_attention(int dtype, const void* Q, int64_t q_seq, int64_t q_tok, int64_t q_head,
                      const void* k_pages, const void* v_pages, int64_t n_pages,
                      int64_t page_size, int64_t page_stride, int64_t row_stride,
                      int64_t head_stride, const int32_t* page_table, int64_t width,
                      const int32_t* lens, const int32_t* nodes, const int64_t* mask,
                      int64_t mask_seq, int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                      double scale, int64_t window, void* Out, float* lse, void* workspace,
                      int64_t workspace_bytes, void* stream) {
  if (B < 0 || T < 0) return TQ_ERR_SHAPE;
  if (B == 0 || T == 0) return TQ_OK;
  if (!Q || !k_pages || !v_pages || !page_table || !lens || !Out) return TQ_ERR_NULL;
  int st = tree_shapes(B, T, Hq, Hkv, D, page_size, width);
  if (st != TQ_OK) return st;
  tq::TreeArgs a{};
  a.Q = Q;
  a.q_seq = step(B, q_seq);
  a.q_tok = step(T, q_tok);
  a.q_head = step(Hq, q_head);
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.n_pages = n_pages;
  a.page_size = page_size;
  a.page_stride = step(n_pages, page_stride);
  a.row_stride = step(page_size, row_stride);
  a.head_stride = step(Hkv, head_stride);
  a.page_table = page_table;
  a.width = width;
  a.lens = lens;
  a.nodes = nodes;
  a.mask = mask;
  a.mask_seq = mask ? step(B, mask_seq) : 0;
  a.B = B;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  if (!tree_strides(a) || !stride_ok(B, a.mask_seq) || (window > 0 && window < T))
    return TQ_ERR_SHAPE;
  const int64_t wants = tq::tree_workspace_bytes(B, T, Hq, Hkv, D, width * page_size);
  if (workspace_bytes < wants) return TQ_ERR_SHAPE;
  if (wants > 0 && !workspace) return TQ_ERR_NULL;
  if (!aligned(Q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(Out, 16) ||
      !aligned(workspace, 16) || !aligned(page_table, 4) || !aligned(lens, 4) ||
      !aligned(nodes, 4) || !aligned(mask, 8) || !aligned(lse, 4))
    return TQ_ERR_ALIGN;
  const double scale_log2 = scale * 1.4426950408889634;  // the kernels hold it in fp32
  if ((dtype != TQ_F16 && dtype != TQ_BF16) || !(fabs(scale_log2) <= FLT_MAX) || window < 0)
    return TQ_ERR_VALUE;
  st = device_ready();
  if (st != TQ_OK) return st;
  a.scale_log2 = (float)scale_log2;
  a.window = window > INT32_MAX ? 0 : window;  // longer than any sequence
  a.Out = Out;
  a.lse = lse;
  a.workspace = workspace;
  return finish(tq::launch_tree_attention(dtype, a, static_cast<hipStream_t>(stream)));
}

int tq_cache_weights(int dtype, const void* Q, int64_t q_seq, int64_t q_tok, int64_t q_head,
                     const void* k_pages, int64_t n_pages, int64_t page_size, int64_t page_stride,
                     int64_t row_stride, int64_t head_stride, const int32_t* page_table,
                     int64_t width, const int32_t* lens, const int32_t* nodes, const int64_t* mask,
                     int64_t mask_seq, const float* lse, int64_t B, int64_t T, int64_t Hq,
                     int64_t Hkv, int64_t D, double scale, int64_t window, double decay,
                     float* scores, int64_t s_seq, int64_t s_head, int64_t S, void* stream) {
  if (B < 0 || T < 0 || S < 0) return TQ_ERR_SHAPE;
  if (B == 0 || T == 0 || S == 0) return TQ_OK;
  if (!Q || !k_pages || !page_table || !lens || !lse || !scores) return TQ_ERR_NULL;
  int st = tree_shapes(B, T, Hq, Hkv, D, page_size, width);
  if (st != TQ_OK) return st;
  if (S > kMaxTokens || T * (Hq / Hkv) > kMostWeightRows) return TQ_ERR_SHAPE;
  tq::WeightsArgs w{};
  tq::TreeArgs& a = w.tree;
  a.Q = Q;
  a.q_seq = step(B, q_seq);
  a.q_tok = step(T, q_tok);
  a.q_head = step(Hq, q_head);
  a.k_pages = k_pages;
  a.n_pages = n_pages;
  a.page_size = page_size;
  a.page_stride = step(n_pages, page_stride);
  a.row_stride = step(page_size, row_stride);
  a.head_stride = step(Hkv, head_stride);
  a.page_table = page_table;
  a.width = width;
  a.lens = lens;
  a.nodes = nodes;
  a.mask = mask;
  a.mask_seq = mask ? step(B, mask_seq) : 0;
  a.B = B;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  w.lse = lse;
  w.scores = scores;
  w.s_seq = step(B, s_seq);
  w.s_head = step(Hkv, s_head);
  w.S = S;
  if (!tree_strides(a) || !stride_ok(B, a.mask_seq) || (window > 0 && window < T) ||
      !stride_ok(B, w.s_seq) || !stride_ok(Hkv, w.s_head) ||
      !distinct(B, w.s_seq, Hkv, w.s_head, S))
    return TQ_ERR_SHAPE;
  if (!aligned(Q, 16) || !aligned(k_pages, 16) || !aligned(page_table, 4) || !aligned(lens, 4) ||
      !aligned(nodes, 4) || !aligned(mask, 8) || !aligned(lse, 4) || !aligned(scores, 4))
    return TQ_ERR_ALIGN;
  const double scale_log2 = scale * 1.4426950408889634;
  if ((dtype != TQ_F16 && dtype != TQ_BF16) || !(fabs(scale_log2) <= FLT_MAX) || window < 0 ||
      !(decay >= 0 && decay <= 1))
    return TQ_ERR_VALUE;
  st = device_ready();
  if (st != TQ_OK) return st;
  a.scale_log2 = (float)scale_log2;
  a.window = window > INT32_MAX ? 0 : window;
  w.decay = (float)decay;
  return finish(tq::launch_cache_weights(dtype, w, static_cast<hipStream_t>(stream)));
}

int tq_cache_select(const float* scores, int64_t s_seq, int64_t s_head, int64_t S,
                    const int32_t* lens, int64_t B, int64_t H, int64_t budget, int64_t recent,
                    int64_t sinks, int32_t* keep, int32_t* counts, float* sums, void* stream) {
  if (B < 0 || H < 0 || S < 0 || budget < 0 || recent < 0 || sinks < 0) return TQ_ERR_SHAPE;
  if (B == 0 || (H == 0 && !counts)) return TQ_OK;  // (without heads only counts are written)
  if ((S > 0 && H > 0 && !scores) || !lens || (budget > 0 && H > 0 && !keep) || !counts)
    return TQ_ERR_NULL;
  if (B > kMaxAttnBatch || H > kMaxAttnHeads || S > kMaxTokens || B * H > kMaxSelectRows ||
      budget > kMaxTokens || recent > budget || sinks > budget - recent)
    return TQ_ERR_SHAPE;
  s_seq = step(B, s_seq);
  s_head = step(H, s_head);
  if (H > 0 && (!stride_ok(B, s_seq) || !stride_ok(H, s_head))) return TQ_ERR_SHAPE;
  if (!aligned(scores, 4) || !aligned(lens, 4) || !aligned(keep, 4) || !aligned(counts, 4) ||
      !aligned(sums, 4))
    return TQ_ERR_ALIGN;
  const int st = device_ready();
  if (st != TQ_OK) return st;
  tq::SelectArgs a{};
  a.scores = scores;
  a.s_seq = s_seq;
  a.s_head = s_head;
  a.S = S;
  a.lens = lens;
  a.B = B;
  a.H = H;
  a.budget = budget;
  a.recent = recent;
  a.sinks = sinks;
  a.keep = keep;
  a.counts = counts;
  a.sums = sums;
  return finish(tq::launch_cache_select(a, static_cast<hipStream_t>(stream)));
}

int64_t tq_pages_keep_workspace(int64_t rows, int64_t width, int64_t n_pages) {
  if (pages_shapes(n_pages, rows, width, 1) != TQ_OK) return TQ_ERR_SHAPE;
  return tq::keep_workspace_bytes(rows, width, n_pages);
}

int tq_pages_keep(void* pool, int64_t planes, int64_t n_pages, int64_t page_bytes,
                  const int32_t* table, const int32_t* lens, int64_t rows, int64_t width,
                  int64_t page_size, const int32_t* keep, int64_t groups, int64_t heads, int64_t n,
                  const int32_t* counts, const int32_t* base, int32_t* table_out,
                  int32_t* lens_out, int32_t* short_out, void* workspace, int64_t workspace_bytes,
                  void* stream) {
  if (rows < 0 || n < 0) return TQ_ERR_SHAPE;
  if ((rows > 0 && (!table || !lens || !counts || !table_out || !lens_out || (n > 0 && !keep))) ||
      !short_out || !workspace || (planes > 0 && !pool))
    return TQ_ERR_NULL;
  int st = pages_shapes(n_pages, rows, width, page_size);
  if (st != TQ_OK || (st = pool_shapes(planes, page_bytes)) != TQ_OK) return st;
  // (a row's lists are counted in 32 bits)
  if (groups < 1 || groups > kMaxPlanes || planes % groups || heads < 1 || heads > kMaxHeads ||
      groups * heads > INT32_MAX || page_bytes % (page_size * heads) ||
      page_bytes / (page_size * heads) % 16 || n > kMaxTokens ||
      workspace_bytes < tq::keep_workspace_bytes(rows, width, n_pages))
    return TQ_ERR_SHAPE;
  if (!aligned(pool, 16) || !aligned(workspace, 16) || !aligned(table, 4) || !aligned(lens, 4) ||
      !aligned(keep, 4) || !aligned(counts, 4) || !aligned(base, 4) || !aligned(table_out, 4) ||
      !aligned(lens_out, 4) || !aligned(short_out, 4))
    return TQ_ERR_ALIGN;
  st = device_ready();
  if (st != TQ_OK) return st;
  tq::KeepArgs a{};
  a.pages.pool = static_cast<unsigned char*>(pool);
  a.pages.planes = planes;
  a.pages.n_pages = n_pages;
  a.pages.page_bytes = page_bytes;
  a.pages.page_size = page_size;
  a.pages.table = table;
  a.pages.lens = lens;
  a.pages.rows_in = a.pages.rows = rows;
  a.pages.width = width;
  a.pages.table_out = table_out;
  a.pages.lens_out = lens_out;
  a.pages.result = short_out;
  a.pages.workspace = workspace;
  a.keep = keep;
  a.groups = groups;
  a.heads = heads;
  a.n = n;
  a.counts = counts;
  a.base = base;
  return finish(tq::launch_pages_keep(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
