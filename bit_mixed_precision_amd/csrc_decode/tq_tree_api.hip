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
  // the kernels count all tiles (64 tokens of 32 rows at least) in 32 bits
  const int64_t blocks = B * Hkv * ((T * (Hq / Hkv) + 31) / 32);
  if (blocks > INT32_MAX || blocks * (width * page_size / 64 + 2) > INT32_MAX) return TQ_ERR_SHAPE;
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

}  // extern "C"
