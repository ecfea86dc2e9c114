/*
 * tq.h -- C ABI of the ternary-weight FP16 GEMM library (libtq.so), gfx950.
 *
 * The library computes Y = X (gamma T)^T, with FP16 activations X and ternary
 * weights T in {-1, 0, 1} stored in one of two lossless packings, as defined on
 * the project page "Scaling Laws and Efficient Inference for Ternary Language
 * Models":
 *   - "The model", steps 1-3: gamma = eps + mean|W| over the whole matrix,
 *     T = round(clip(W / gamma, -1, 1)), Y = X (gamma T)^T;
 *   - "Packing ternary weights" / "2 bits per weight" (TQ2): d' = d + 1 in a
 *     2-bit field, d' = (b >> 2j) & 3, four weights per byte;
 *   - "Packing ternary weights" / "1.6 bits per weight" (TQ1): five shifted
 *     digits read as a base-3 number N in [0, 242], stored as
 *     b = floor((256 N + 242) / 243);
 *   - "Fast inference on CPUs": one 16-bit scale per block of 256 weights;
 *   - "TriRun: ternary inference on GPUs": FP32 accumulation, FP16 output.
 *
 * Layouts (all row-major, no padding unless stated):
 *   X       fp16 [M][K]
 *   Y       fp16 [M][N]            Y[m][n] = sum_k X[m][k] * s[n][k/256] * T[n][k]
 *   T       int8 [N][K]            row n is output feature n (as nn.Linear)
 *   scales  fp16 [N][K/256]        s[n][b] scales weights k in [256 b, 256 b + 256)
 *   TQ2 qs  uint8 [N][K/4]         weight k = 4 i + j of a row: byte i, bits 2j..2j+1
 *   TQ1 qs  uint8 [N][ldq]         byte g of a row: weights 5 g .. 5 g + 4, the first
 *                                  one most significant; the last group of a row is
 *                                  padded with zero trits; bytes ceil(K/5) .. ldq-1
 *                                  are written as 0 and never read for values.
 *
 * Every function returns an int status (TQ_OK = 0, errors < 0).  No function
 * throws, aborts or prints.  Arguments are checked in this order: null
 * pointers, shapes, alignment, values; argument errors are reported before any
 * output is written or any kernel launched.  The caller owns every buffer.
 */
#ifndef TQ_H_
#define TQ_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum tq_status {
  TQ_OK = 0,
  TQ_ERR_NULL = -1,        /* a required pointer is NULL                         */
  TQ_ERR_SHAPE = -2,       /* negative or unsupported M, N, K, ldq               */
  TQ_ERR_VALUE = -3,       /* trit outside {-1,0,1}, NaN/Inf latent, gamma <= 0,  */
                           /* invalid packed byte                                 */
  TQ_ERR_ALIGN = -4,       /* a device pointer is not 16-byte aligned            */
  TQ_ERR_DEVICE = -5,      /* no usable HIP device, or a launch failed           */
  TQ_ERR_UNSUPPORTED = -6  /* an option this build does not provide              */
};

/* Source of the weights handed to the packers. */
typedef enum {
  TQ_SRC_TERNARY_I8 = 0, /* int8 [N][K] trits in {-1, 0, 1}                        */
  TQ_SRC_LATENT_F32 = 1  /* float [N][K] latent weights, ternarized with eps        */
} tq_src;

/* Kernel family for tq_gemm_*_ex.  AUTO picks, for TQ2, the skinny kernel for
 * M <= 16, and for M <= 32 when K <= 16384 and N >= 480 M, the tiled MFMA
 * kernel otherwise; for TQ1, the skinny kernel for M <= 16 and the tiled
 * (table-decode) kernel above (measured at K = 8192).  The others force one
 * family (used by the tests to cover both sides of the switch); the TQ2
 * skinny family serves M <= 32 and returns TQ_ERR_UNSUPPORTED above.  The
 * TQ1 tiled family takes ldq <= 2^22; a larger row stride runs the skinny
 * kernel instead. */
typedef enum {
  TQ_PATH_AUTO = 0,
  TQ_PATH_SKINNY = 1,
  TQ_PATH_TILED = 2,
  TQ_PATH_SIMPLE = 3 /* one wave per output row, VALU only: the plain GPU kernel */
} tq_path;

/* Human-readable name of a status code (static storage; never NULL). */
const char* tq_status_string(int status);

/* Version of this ABI; bumped on any incompatible change. */
int tq_abi_version(void);

/* Buffer sizes, in elements (bytes for qs).  Return -1 for invalid shapes. */
int64_t tq_tq2_bytes(int64_t N, int64_t K);  /* N * K / 4                           */
int64_t tq_tq1_ldq(int64_t K);               /* ceil(K / 5) rounded up to 16         */
int64_t tq_num_scales(int64_t N, int64_t K); /* N * K / 256                          */

/* ---------------------------------------------------------------------------
 * Host side (offline).  Thread-safe and stateless; uses several host threads
 * for large matrices.  All pointers are host memory.
 * ------------------------------------------------------------------------- */

/* "The model", steps 1-2.  W float [N][K], N, K >= 1.  gamma = eps + S / (N K),
 * where S is the exactly rounded fp64 sum of |W|; each trit is the fp64
 * quotient W / gamma clipped to [-1, 1] and rounded half to even.
 * T (int8 [N][K]) may be NULL to obtain gamma only; gamma_out may be NULL.
 * Errors: TQ_ERR_VALUE for a NaN/Inf weight, or a gamma that is not finite and
 * positive (e.g. eps = 0 and W = 0). */
int tq_ternarize_f32(const float* W, int64_t N, int64_t K, double eps,
                     int8_t* T, double* gamma_out);

/* TQ2 packing ("2 bits per weight").  K must be a positive multiple of 256.
 *   kind = TQ_SRC_LATENT_F32: W is float [N][K]; ternarize as tq_ternarize_f32,
 *     write qs, fill every entry of scales (fp16 bits [N][K/256]) with fp16(gamma)
 *     rounded to nearest even in one step from fp64, and store gamma in
 *     *gamma_out when non-NULL.  scales must not be NULL.
 *   kind = TQ_SRC_TERNARY_I8: W is int8 [N][K]; only qs is written; scales,
 *     gamma_out and eps are ignored (scales may be NULL).
 * qs is uint8 [N][K/4]. */
int tq_pack_tq2(int kind, const void* W, int64_t N, int64_t K, double eps,
                uint8_t* qs, uint16_t* scales_f16, double* gamma_out);

/* TQ1 packing ("1.6 bits per weight").  Same kinds and scales as tq_pack_tq2;
 * qs is uint8 [N][ldq] with ldq >= ceil(K/5).  K must be a positive multiple
 * of 256 (the scale block); the rows' last group is padded with zero trits. */
int tq_pack_tq1(int kind, const void* W, int64_t N, int64_t K, double eps, int64_t ldq,
                uint8_t* qs, uint16_t* scales_f16, double* gamma_out);

/* Inverse of the packers: T int8 [N][K].  K >= 1 (a multiple of 4 for TQ2).
 * TQ_ERR_VALUE for a 2-bit field equal to 3 (TQ2), for one of the 13 byte values
 * that no pattern produces, or for a non-zero padding trit (TQ1). */
int tq_unpack_tq2(const uint8_t* qs, int64_t N, int64_t K, int8_t* T);
int tq_unpack_tq1(const uint8_t* qs, int64_t N, int64_t K, int64_t ldq, int8_t* T);

/* ---------------------------------------------------------------------------
 * Device side.  Every pointer is device memory on the current HIP device.
 * The call only enqueues work on `stream` (a hipStream_t; NULL = the default
 * stream) and returns; it allocates nothing, never synchronizes and uses no
 * atomics, so Y is the same bit for bit on every run with the same inputs.
 *
 *   Y = X (s . T)^T :  X fp16 [M][K], Y fp16 [M][N], scales fp16 [N][K/256].
 *
 * Shapes: M, N >= 0 (M == 0 or N == 0 is a no-op that touches no pointer);
 * K a positive multiple of 256; M, N <= 2^24, K <= 2^20.  For TQ1,
 * ceil(K/5) <= ldq <= 2^24 and ldq % 16 == 0.  X, qs, scales and Y must be
 * 16-byte aligned.
 * Accumulation is fp32; Y is rounded to fp16 (nearest even) once, overflow
 * gives +-inf.  Trits are not validated on the device: a TQ2 field equal to 3
 * or an unused TQ1 byte gives unspecified (finite) values for that row.
 * Errors: TQ_ERR_DEVICE when no HIP device is usable or the launch fails.
 * ------------------------------------------------------------------------- */
int tq_gemm_tq2(const void* X, const void* qs, const void* scales_f16, void* Y,
                int64_t M, int64_t N, int64_t K, void* stream);
int tq_gemm_tq1(const void* X, const void* qs, int64_t ldq, const void* scales_f16, void* Y,
                int64_t M, int64_t N, int64_t K, void* stream);

/* Name of the kernel that tq_gemm_tq2_ex (format = 2) or tq_gemm_tq1_ex
 * (format = 1, with ldq <= 2^22) launches for this shape and path, as
 * profilers show it, copied NUL-terminated into name[cap].  TQ_ERR_SHAPE for an invalid shape,
 * TQ_ERR_VALUE for an unknown format or path, TQ_ERR_NULL for a NULL name,
 * TQ_ERR_UNSUPPORTED when the path is not available for the format.  Host
 * only; touches no device. */
int tq_kernel_name(int format, int64_t M, int64_t N, int64_t K, int path, char* name,
                   int64_t cap);

/* Same as above with an explicit kernel family (tq_path). */
int tq_gemm_tq2_ex(const void* X, const void* qs, const void* scales_f16, void* Y,
                   int64_t M, int64_t N, int64_t K, int path, void* stream);
int tq_gemm_tq1_ex(const void* X, const void* qs, int64_t ldq, const void* scales_f16, void* Y,
                   int64_t M, int64_t N, int64_t K, int path, void* stream);

/* ---------------------------------------------------------------------------
 * On-device ternarization and packing (the step before the product; project
 * page "The model" steps 1-2 and "Packing ternary weights").  The same
 * results as tq_pack_tq2 / tq_pack_tq1 with TQ_SRC_LATENT_F32, bit for bit:
 * gamma = eps + mean|W| with an exactly rounded fp64 sum of |W|, trits from
 * the fp64 quotient W / gamma with ties to even, fp16(gamma) in every scale.
 *
 * W float [N][K], qs, scales, gamma (one double), status (one int) and the
 * workspace are device memory on the current device; the call enqueues four
 * kernels on `stream` and returns (no host round trip, no allocation).
 * gamma and status may be NULL.  The workspace holds at least
 * tq_pack_dev_workspace_bytes(N, K) bytes (a few KB); its contents need no
 * initialization and are overwritten, so calls that may overlap need
 * separate workspaces.  The exact sum uses 64-bit integer atomics, whose
 * result does not depend on their order: every run gives the same bits.  W, qs, scales and the workspace must be
 * 16-byte aligned.  Shapes: N >= 1, 256 <= K <= 2^20, K % 256 == 0, N <=
 * 2^24; TQ1 ldq >= ceil(K/5).  Synchronous errors: TQ_ERR_NULL, TQ_ERR_SHAPE
 * (also a workspace that is too small), TQ_ERR_ALIGN, TQ_ERR_DEVICE.  A
 * non-finite latent or gamma is reported through *status (TQ_ERR_VALUE, else
 * TQ_OK) once the stream reaches it; qs and scales are then unspecified. */
int64_t tq_pack_dev_workspace_bytes(int64_t N, int64_t K); /* -1 for a bad shape */
int tq_pack_tq2_dev(const float* W, int64_t N, int64_t K, double eps, uint8_t* qs,
                    uint16_t* scales_f16, double* gamma, int* status, void* workspace,
                    int64_t workspace_bytes, void* stream);
int tq_pack_tq1_dev(const float* W, int64_t N, int64_t K, double eps, int64_t ldq, uint8_t* qs,
                    uint16_t* scales_f16, double* gamma, int* status, void* workspace,
                    int64_t workspace_bytes, void* stream);

/* tq_pack_tq2_dev without a workspace argument, for callers that cannot
 * allocate device memory (code under HIP graph capture, serving loops,
 * harnesses that forbid hipMalloc).  It runs the same four kernels with the
 * workspace in a fixed array of the library, tq_pack_dev_workspace_bytes()
 * bytes (4224) per device, reserved when the library is loaded and held until
 * the process ends; no call allocates or frees anything.  Every call on a
 * device uses that device's one array, so calls that overlap in time on one
 * device (other streams, other host threads) race and give unspecified qs,
 * scales and gamma; calls in one stream's order do not (each clears the
 * totals it needs at its start).  Arguments, results, status and errors as
 * tq_pack_tq2_dev (the same shape limits: N <= 2^24, K <= 2^20; a shape whose
 * workspace would exceed the array gives TQ_ERR_SHAPE); TQ_ERR_DEVICE also
 * when the array's device address cannot be obtained. */
int tq_pack_tq2_dev_noalloc(const float* W, int64_t N, int64_t K, double eps, uint8_t* qs,
                            uint16_t* scales_f16, double* gamma, int* status, void* stream);

/* TQ2 product on the tiled kernel with an explicit tile, for tuning and for
 * tests of every tile: 16 mt activation rows x 64 ng weight rows (32 ng when
 * mt = 8) per workgroup of ng x kg waves (kg of them split K).  Compiled
 * tiles: mt in {2, 4} with (ng, kg) in {(4, 2), (2, 4), (2, 2), (1, 4)},
 * mt = 2 with (1, 8), and mt = 8 with (4, 2); any other tile gives
 * TQ_ERR_UNSUPPORTED.  Everything
 * else is as tq_gemm_tq2. */
int tq_gemm_tq2_tiled(const void* X, const void* qs, const void* scales_f16, void* Y,
                      int64_t M, int64_t N, int64_t K, int mt, int ng, int kg, void* stream);

/* Fused gate / up product of the decode step's gated MLP (SwiGLU, named in
 * the architecture section of the project page "Scaling Laws and Efficient
 * Inference for Ternary Language Models"; each product as in "The model"):
 *   Y[m][n] = silu(g) * u,  g = sum_k X[m][k] s_g[n][k/256] T_g[n][k],
 *                           u = sum_k X[m][k] s_u[n][k/256] T_u[n][k],
 * silu(g) = g / (1 + exp(-g)), g, u and the product in fp32, one fp16
 * rounding.  Gate and up matrices are TQ2 packed as for tq_gemm_tq2 (qs
 * [N][K/4], scales [N][K/256] fp16), both N x K; X [M][K] and Y [M][N] fp16,
 * all device pointers, 16-byte aligned, owned by the caller.  For decode
 * sizes: 1 <= M <= 16 (larger M gives TQ_ERR_UNSUPPORTED); one launch streams
 * both matrices, the skinny kernel's offset rounding applies to g and u.
 * Errors as tq_gemm_tq2 (M = 0 or N = 0 is a no-op returning TQ_OK). */
int tq_gemm_tq2_swiglu(const void* X, const void* qs_gate, const void* scales_gate_f16,
                       const void* qs_up, const void* scales_up_f16, void* Y, int64_t M,
                       int64_t N, int64_t K, void* stream);

/* Input gradient of the ternary product for quantization-aware training
 * (the backward pass through "The model", step 3, on the project page
 * "Scaling Laws and Efficient Inference for Ternary Language Models"):
 *   dX[m][k] = sum_n dY[m][n] * scales[n][k/256] * T[n][k],
 * i.e. dY (s . T) with the TQ2 matrix of tq_gemm_tq2 (qs [N][K/4], scales
 * [N][K/256] fp16) read the other way round; dY [M][N] and dX [M][K] fp16,
 * device pointers, 16-byte aligned, owned by the caller; FP32 accumulation,
 * one fp16 rounding.  N must be a positive multiple of 8 and at most 2^20, K
 * a multiple of 256 (TQ_ERR_SHAPE otherwise); M = 0 is a no-op returning
 * TQ_OK.  Block scales must satisfy |s| < 1024: the kernel carries a column's
 * field position as an exact factor of up to 64 on the decoded s.  The weight
 * gradient under the straight-through estimator is tq_ste_grad_w. */
int tq_gemm_tq2_bwd_x(const void* dY, const void* qs, const void* scales_f16, void* dX,
                      int64_t M, int64_t N, int64_t K, void* stream);

/* Gradient that reaches the latent weights of a ternary linear under the
 * straight-through estimator (project page "Scaling Laws and Efficient
 * Inference for Ternary Language Models", "The model": gradients pass to the
 * latent weights with a straight-through estimator; Spectra page,
 * "Architecture of TriLM and FloatLM").  The quantizer W -> gamma T is taken
 * as the identity in the backward pass, so the latent weights receive the
 * gradient with respect to the effective weights of Y = X (gamma T)^T:
 *   dW[n][k] = sum_m dY[m][n] * X[m][k]            (accumulate = 0)
 *   dW[n][k] = dW[n][k] + sum_m dY[m][n] X[m][k]   (accumulate = 1)
 * gamma is not differentiated and no weight is masked (e.g. outside the clip
 * window |W / gamma| <= 1); the result does not depend on W, gamma or T.
 * dY fp16 [M][N] (the output gradient), X fp16 [M][K] (the layer input), dW
 * fp32 [N][K] (the latent weights' layout), all row-major device pointers,
 * 16-byte aligned, owned by the caller; FP32 accumulation, FP32 output, the
 * same bits on every run.  Shapes: M >= 0 (M = 0 writes zeros and reads
 * neither input, which may then be NULL, or is a no-op with accumulate = 1);
 * N = 0 or K = 0 is a no-op; N and K multiples of 8 and
 * at most 2^24; M N and M K at most 2^30 (split larger batches and
 * accumulate).  Errors: TQ_ERR_SHAPE, TQ_ERR_NULL, TQ_ERR_ALIGN,
 * TQ_ERR_VALUE (accumulate not 0 or 1), TQ_ERR_DEVICE. */
int tq_ste_grad_w(const void* dY, const void* X, float* dW, int64_t M, int64_t N, int64_t K,
                  int accumulate, void* stream);

/* Re-pack TQ1 weights as TQ2 on the device: the trits of qs1 ([N][ldq],
 * "1.6 bits per weight" on the project page "Scaling Laws and Efficient
 * Inference for Ternary Language Models") written as the 2-bit fields of qs2
 * ([N][K/4], "2 bits per weight"), bit for bit what tq_pack_tq2 writes for
 * the same trits; the block scales are shared unchanged.  Device pointers,
 * 16-byte aligned, owned by the caller; qs2 holds tq_tq2_bytes(N, K) bytes.
 * K a multiple of 256, ceil(K/5) <= ldq <= 2^24 and ldq a multiple of 16
 * (TQ_ERR_SHAPE otherwise); N = 0 is a no-op.  Byte values that no trit group encodes are
 * not detected. */
int tq_transcode_tq1_tq2(const void* qs1, int64_t ldq, int64_t N, int64_t K, void* qs2,
                         void* stream);

/* Activation rows from which tq_gemm_tq1_ws transcodes for an N x K matrix
 * (the measured crossover against the table-decode tiled kernel: 96 for
 * N <= 16384, else 33); TQ_ERR_SHAPE for
 * N < 1 or K not a positive multiple of 256. */
int64_t tq_tq1_transcode_min_m(int64_t N, int64_t K);

/* TQ1 product with a caller workspace, for batch and prefill sizes: with
 * M >= tq_tq1_transcode_min_m(N, K) and workspace_bytes >= tq_tq2_bytes(N, K),
 * the weights are first re-packed into the workspace as by
 * tq_transcode_tq1_tq2 and the TQ2 kernels of tq_gemm_tq2 run on it (the
 * TQ1 tiled kernel decodes every weight through LDS table lookups once per
 * activation tile; this decodes it once per call, at the cost of writing and
 * reading a 2-bit copy), so Y equals tq_gemm_tq2's on the same trits bit for
 * bit.
 * Otherwise (smaller M, no or too small a workspace) it is tq_gemm_tq1.
 * The workspace is device memory owned by the caller, 16-byte aligned when
 * given (TQ_ERR_ALIGN otherwise), overwritten by the call, and must not
 * overlap X, qs, scales or Y; calls that overlap on one workspace race.
 * Everything else is as tq_gemm_tq1. */
int tq_gemm_tq1_ws(const void* X, const void* qs, int64_t ldq, const void* scales_f16, void* Y,
                   int64_t M, int64_t N, int64_t K, void* workspace, int64_t workspace_bytes,
                   void* stream);

/* Measurement aid: the practical read ceiling for the weight-streaming
 * kernels.  Small-batch ternary inference is bound by reading the packed
 * weights ("TriRun: ternary inference on GPUs" on the project page "Scaling
 * Laws and Efficient Inference for Ternary Language Models"); this reads
 * `bytes` bytes at `src` once, with the loads the GEMV kernels use, and
 * computes nothing, so its time at a given size is what a launch that only
 * streams those bytes costs on this GPU.  src and sink are device pointers,
 * 16-byte aligned, owned by the caller; sink (4 bytes) is written only when
 * the XOR of the data equals one fixed 32-bit value.  bytes must be a
 * non-negative multiple of 16 (TQ_ERR_SHAPE otherwise); 0 is a no-op. */
int tq_stream_read(const void* src, int64_t bytes, void* sink, void* stream);

/* As tq_gemm_tq2_tiled with the weight rows per wave explicit: 16 mt
 * activation rows x 16 nr ng weight rows per workgroup of ng x kg waves.
 * Compiled tiles (mt, nr, ng, kg): mt in {2, 4} with (4, 4, 2), (4, 2, 4),
 * (4, 2, 2), (4, 1, 4), (2, 1, 4), (2, 2, 4), and (2, 2, 1, 8), (2, 4, 1, 8),
 * (8, 2, 4, 2);
 * any other gives TQ_ERR_UNSUPPORTED.  Everything else is as tq_gemm_tq2. */
int tq_gemm_tq2_tile(const void* X, const void* qs, const void* scales_f16, void* Y, int64_t M,
                     int64_t N, int64_t K, int mt, int nr, int ng, int kg, void* stream);

/* TQ2 product on the wide-tile kernel (v_mfma_f32_32x32x16_f16) with an
 * explicit tile, for tuning and for tests of every tile: 32 mt activation rows
 * x 32 nt ng weight rows per workgroup of ng x kg = 4 waves (kg of them split
 * K).  Compiled tiles: mt in {1, 2, 4}, nt in {1, 2}, (ng, kg) in {(2, 2),
 * (1, 4)}, except mt = 4 with kg = 4; any other gives TQ_ERR_UNSUPPORTED.
 * M K and N K / 4 must stay below 2^31 bytes (TQ_ERR_SHAPE otherwise).
 * Everything else is as tq_gemm_tq2. */
int tq_gemm_tq2_wide(const void* X, const void* qs, const void* scales_f16, void* Y, int64_t M,
                     int64_t N, int64_t K, int mt, int nt, int ng, int kg, void* stream);

/* TQ1 product on the table-decode tiled kernel with an explicit tile, for
 * tuning and for tests of every tile.  The tiles and their meaning are
 * tq_gemm_tq2_tile's; the weights are the 1.6-bit rows of tq_gemm_tq1 ("1.6
 * bits per weight" on the project page "Scaling Laws and Efficient Inference
 * for Ternary Language Models"), read once from HBM with no 2-bit copy:
 * each block's bytes are copied to LDS and every byte's five trits come from
 * a 256-entry table built with the pages' multiply-by-3 decoder.  ldq above
 * 2^22 or a tile not compiled gives TQ_ERR_UNSUPPORTED.  Everything else is as
 * tq_gemm_tq1. */
int tq_gemm_tq1_tile(const void* X, const void* qs, int64_t ldq, const void* scales_f16, void* Y,
                     int64_t M, int64_t N, int64_t K, int mt, int nr, int ng, int kg,
                     void* stream);

/* ---------------------------------------------------------------------------
 * Between the products of a decoder layer: rotary positions, attention of one
 * new token over a paged key-value cache, and the pages of that cache.  The
 * architecture section of the project page names rotary positions (base 5e5)
 * and LLaMA-style attention; the operators are the standard ones, stated below.
 *
 * Types: fp16, bfloat16 and, for tq_rope, fp32 (tq_dtype).  Strides are in
 * elements, 0 to 2^46, and a stride times the entries of its dimension is at most
 * 2^58; the stride of a dimension of one entry is not looked at.  Device entry points enqueue on `stream` and return; they never
 * allocate, synchronize or use memory that is not an argument, and can be
 * captured in a HIP graph.
 *
 * A paged cache.  Keys and values live in pages of page_size tokens; number
 * d of head h of slot i of page p is at
 *   pages[p * page_stride + i * row_stride + h * head_stride + d].
 * A page table int32 [rows][width] names, for every sequence, the pages of its
 * tokens in order: token t is in slot t % page_size of page
 * table[row][t / page_size].  A sequence of len tokens holds the first
 * ceil(len / page_size) entries of its row; entries past them are not read.
 * ------------------------------------------------------------------------- */

typedef enum { TQ_F16 = 0, TQ_BF16 = 1, TQ_F32 = 2 } tq_dtype;

/* How the rotation frequencies f_i = theta^(-2 i / rot), i < rot / 2, are
 * changed for contexts `factor` times longer than the trained one. */
typedef enum {
  TQ_ROPE_NONE = 0,   /* not at all                                             */
  TQ_ROPE_LINEAR = 1, /* f_i / factor: positions interpolated                   */
  TQ_ROPE_BASE = 2,   /* theta * factor^(rot / (rot - 2)): the base raised      */
  TQ_ROPE_PARTS = 3   /* f_i k_i + f_i / factor (1 - k_i), k_i = (r_i - slow) / */
                      /* (fast - slow) clipped to [0, 1], r_i = trained f_i /   */
                      /* (2 pi) the turns pair i makes in the trained context   */
} tq_rope_scaling;

/* Host function: the table [n_pos][rot / 2][2] of (cos, sin) of p f_i for
 * positions p < n_pos, both times `gain`, computed in fp64 and rounded once to
 * fp32.  factor is ignored for TQ_ROPE_NONE; trained, fast and slow are used by
 * TQ_ROPE_PARTS only.  Errors: TQ_ERR_NULL; TQ_ERR_SHAPE (n_pos outside
 * [0, 2^30], rot odd or outside [2, 2^16], rot = 2 with TQ_ROPE_BASE);
 * TQ_ERR_VALUE (unknown scaling; theta, factor, gain, trained not finite and
 * positive; fast <= slow). */
int tq_rope_table(int64_t n_pos, int64_t rot, double theta, int scaling, double factor,
                  double trained, double fast, double slow, double gain, float* table);

/* Rotary positions.  The first rot numbers of every head of X [T][H][D] are
 * rot / 2 pairs -- (x_i, x_{i + rot/2}), or (x_{2i}, x_{2i+1}) with interleaved
 * -- and pair i of token t is turned by the angle that row pos[t] of `table`
 * holds:
 *   y_a = x_a cos - x_b sin,   y_b = x_b cos + x_a sin;
 * numbers rot .. D - 1 are copied.  inverse = 1 turns back by the same angles:
 * with the same table this is the gradient dX of dY (the rotation's transpose,
 * table gain included).  Computed in fp32, rounded once to X's type.
 * X and Y: device pointers, number d of head h of token t at
 * x_tok t + x_head h + d; heads and tokens may lie in any order and X may
 * repeat (stride 0), but no two elements of Y may share an address
 * (TQ_ERR_SHAPE).  Y = X with equal strides is allowed, any other overlap not.
 * pos int32 [T], device; a token whose position is outside [0, n_pos) comes
 * out as zeros.  table: fp32 [n_pos][rot / 2][2], device, 8-byte aligned (NULL
 * when n_pos = 0).
 * T = 0 or H = 0 is a no-op.  D <= 2^16, rot even, 2 <= rot <= D, H <= 2^16,
 * T <= 2^30, T H < 2^31.  Errors: TQ_ERR_NULL, TQ_ERR_SHAPE, TQ_ERR_ALIGN (X or Y not
 * aligned to an element), TQ_ERR_VALUE (dtype, interleaved, inverse). */
int tq_rope(int dtype, const void* X, int64_t x_tok, int64_t x_head, void* Y, int64_t y_tok,
            int64_t y_head, const float* table, int64_t n_pos, int64_t rot, const int32_t* pos,
            int64_t T, int64_t H, int64_t D, int interleaved, int inverse, void* stream);

/* The decode step's use of tq_rope in one launch: QKV holds, for each of T
 * tokens, Hq query, Hkv key and Hkv value heads of D numbers (the row of a
 * fused q/k/v product), token t at QKV + qkv_tok t.  Turned queries are written
 * to Q [T][Hq][D]; turned keys and the values go to the slot of position pos[t]
 * in the paged cache (as above), in the row seqs[t] of the page table, or row t
 * when seqs is NULL.  fp16 or bfloat16.
 * A token whose position is outside [0, n_pos) gets zeros in Q, and nothing of
 * it is written to the cache; nor is it where the row is outside
 * [0, n_seqs), the position is past the table's width, or the page is outside
 * [0, n_pages).  Two tokens of one call must not name the same slot.
 * Limits as tq_rope's with H = Hq + 2 Hkv, and Hq, Hkv >= 1.
 * Errors as tq_rope's, and TQ_ERR_SHAPE for page geometry (page_size < 1,
 * negative strides, width * page_size > 2^30, strides that let two numbers of a
 * cache share an address). */
int tq_rope_append(int dtype, const void* QKV, int64_t qkv_tok, const float* table, int64_t n_pos,
                   int64_t rot, const int32_t* pos, const int32_t* seqs, const int32_t* page_table,
                   int64_t n_seqs, int64_t width, void* k_pages, void* v_pages, int64_t n_pages,
                   int64_t page_size, int64_t page_stride, int64_t row_stride,
                   int64_t head_stride, void* Q, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                   int interleaved, void* stream);

/* tq_rope_append where a token's slot is not its position: the drafted nodes of a tree,
 * whose positions go by their depth, and caches that have lost tokens.  slots int32 [T],
 * device, or NULL: positions.  Keys and values of token t go to slot slots[t] of its row;
 * queries and keys are turned by position pos[t].  A slot outside the table's width, or
 * negative, is not written.  Everything else as tq_rope_append. */
int tq_rope_append_at(int dtype, const void* QKV, int64_t qkv_tok, const float* table,
                      int64_t n_pos, int64_t rot, const int32_t* pos, const int32_t* slots,
                      const int32_t* seqs, const int32_t* page_table, int64_t n_seqs,
                      int64_t width, void* k_pages, void* v_pages, int64_t n_pages,
                      int64_t page_size, int64_t page_stride, int64_t row_stride,
                      int64_t head_stride, void* Q, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                      int interleaved, void* stream);

/* Attention of one new token per sequence over the paged cache:
 *   out[b][h] = sum_t w_t v[t][h / G],  w = softmax_t(scale q[b][h] . k[t][h / G])
 * over the tokens t in [max(0, len - window), len) of sequence b (window = 0:
 * all), G = Hq / Hkv.  Q: number d of head h of sequence b at q_tok b +
 * q_head h + d; Out [B][Hq][D]; lse fp32 [B][Hq] or NULL: ln of the sum of the
 * exponentials, for joining with other parts of the same softmax.  lens int32
 * [B]: negative counts as 0, and at most width * page_size tokens are read.
 * A sequence with no token gives zeros and lse = -inf.  A page outside
 * [0, n_pages) counts as absent: its tokens are left out.  What the cache holds
 * in other slots, NaN included, has no influence.
 * fp16 or bfloat16 in and out, fp32 scores, weights and sums; each weight enters
 * the product with v as two 16-bit numbers, rounded to within 2^-22 (fp16; 2^-16
 * bfloat16) of itself, in fp16 or within 2^-38 of the row's largest.  A weight of
 * zero adds nothing, however large its (finite) value; in fp16 one below 2^-39 of the
 * row's largest may add nothing.  An infinite value gives an infinite result, or NaN
 * where its weight is zero, and in fp16 it may where it is below 2^-38 of the largest.
 * The same bits on every run.  Outputs and workspace must not overlap the inputs.
 * D a multiple of 8, 8 <= D <= 256; Hq a multiple of Hkv, Hq <= 2^12; B <=
 * 2^20; width * page_size <= 2^30; B * Hkv * ceil(Hq / Hkv / 16) * (width *
 * page_size / 32 + 2) < 2^31; strides multiples of 8, row_stride <= 2^24;
 * pointers 16-byte aligned.  workspace: tq_paged_attention_workspace(...)
 * bytes, 16-byte aligned, contents irrelevant; calls that overlap on one
 * workspace race.
 * Errors: TQ_ERR_NULL, TQ_ERR_SHAPE (a workspace that is too small included),
 * TQ_ERR_ALIGN, TQ_ERR_VALUE (dtype, scale log2(e) not finite in fp32, window < 0),
 * TQ_ERR_DEVICE.  B = 0 is a no-op. */
int tq_paged_attention(int dtype, const void* Q, int64_t q_tok, int64_t q_head,
                       const void* k_pages, const void* v_pages, int64_t n_pages,
                       int64_t page_size, int64_t page_stride, int64_t row_stride,
                       int64_t head_stride, const int32_t* page_table, int64_t width,
                       const int32_t* lens, int64_t B, int64_t Hq, int64_t Hkv, int64_t D,
                       double scale, int64_t window, void* Out, float* lse, void* workspace,
                       int64_t workspace_bytes, void* stream);

/* Workspace bytes of tq_paged_attention for tables of `width` pages;
 * TQ_ERR_SHAPE for shapes it refuses. */
int64_t tq_paged_attention_workspace(int64_t B, int64_t Hq, int64_t Hkv, int64_t D,
                                     int64_t page_size, int64_t width);

/* The paths of drafted trees: parents int32 [B][T], node i hanging on node parents[i]
 * < i of its tree, or on the last cached token where parents[i] is anything else.  mask: 64-bit
 * words [B][T][ceil(T / 64)]; bit j % 64 of word j / 64 of node i is set where j is i
 * or a node above it, all other bits are clear.  depth int32 [B][T] or NULL: the number
 * of nodes above i, which with the sequence's length is the node's position.
 * All device pointers.  T <= 256, B <= 2^20; B = 0 or T = 0 is a no-op.  Errors:
 * TQ_ERR_NULL, TQ_ERR_SHAPE, TQ_ERR_ALIGN (mask to 8 bytes), TQ_ERR_DEVICE. */
int tq_tree_mask(const int32_t* parents, int64_t B, int64_t T, int64_t* mask, int32_t* depth,
                 void* stream);

/* Attention of several new tokens per sequence over the paged cache: sequence b has
 * lens[b] cached tokens (negative counts as 0) and the first nodes[b] of T nodes
 * (NULL: all; below 0 none), whose keys and values lie in the slots lens[b],
 * lens[b] + 1, ... after them.
 *   out[b][i][h] = sum_t w_t v[t][h / G],  w = softmax_t(scale q[b][i][h] . k[t][h / G])
 * over the cached tokens and the tokens lens[b] + j of the nodes j < nodes[b] whose bit
 * is set for node i in mask (words as tq_tree_mask writes them, sequence b's at mask +
 * mask_seq b, mask_seq = 0: one tree for all; any bits will do, also none; NULL: a
 * chain, j <= i).  With a window (0: none, otherwise at least T) a node that sees s
 * nodes sees only the last window - s cached tokens.  At most width * page_size tokens
 * are read, and an absent page's tokens are left out, as by tq_paged_attention.
 * Rows of nodes that are not there, and of nodes that see no token, are zeros with
 * lse = -inf.  Q: number d of head h of node i of sequence b at q_seq b + q_tok i +
 * q_head h + d; Out [B][T][Hq][D]; lse fp32 [B][T][Hq] or NULL.
 * fp16 or bfloat16 in and out, fp32 scores, weights and sums.  Up to 32 rows (T G <= 32) a
 * weight enters the product with v as two 16-bit numbers, rounded to within 2^-22 (fp16;
 * 2^-16 bfloat16) of itself; with more rows as two or as one, rounded to nearest (2^-11 of
 * itself in fp16, 2^-8 in bfloat16).  Which it is goes by all sizes of the call, the batch and
 * the table's width among them, and the order of the sums by these and all lengths: a sequence
 * may have other last bits beside other sequences.  In fp16 a weight may also be off by 2^-33 of the row's
 * largest, and one below 2^-34 of it may add nothing.  An infinite value gives an infinite
 * result, or NaN where its weight is zero or, in fp16, may add nothing.  A token that a
 * node does not see has no influence on it, whatever its key and value hold.  The same
 * bits on every run.  Outputs and workspace must not overlap the inputs.
 * Limits as tq_paged_attention's, and T <= 256; B * Hkv * ceil(T G / 32) < 2^24, and times
 * (width * page_size / 64 + 2) < 2^31.  workspace: tq_tree_attention_workspace(...) bytes,
 * 16-byte aligned, contents irrelevant; calls that overlap on one workspace race.
 * Errors: as tq_paged_attention's; TQ_ERR_SHAPE for a window below T.  B = 0 or T = 0
 * is a no-op. */
int tq_tree_attention(int dtype, const void* Q, int64_t q_seq, int64_t q_tok, int64_t q_head,
                      const void* k_pages, const void* v_pages, int64_t n_pages,
                      int64_t page_size, int64_t page_stride, int64_t row_stride,
                      int64_t head_stride, const int32_t* page_table, int64_t width,
                      const int32_t* lens, const int32_t* nodes, const int64_t* mask,
                      int64_t mask_seq, int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                      double scale, int64_t window, void* Out, float* lse, void* workspace,
                      int64_t workspace_bytes, void* stream);

/* Workspace bytes of tq_tree_attention for tables of `width` pages; TQ_ERR_SHAPE for
 * shapes it refuses. */
int64_t tq_tree_attention_workspace(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                                    int64_t page_size, int64_t width);

/* What an eviction goes by: the attention weight that every cached token receives,
 * added to a running sum.  Arguments as tq_tree_attention's (T = 1: one new token per
 * sequence, lens not counting it); lse fp32 [B][T][Hq] is what that call returned.
 *   w[b][h][t] = sum over nodes i and query heads j of head h's group of
 *                exp(scale q[b][i][j] . k[t][h] - lse[b][i][j]) over the tokens i sees
 *   scores[b][h][t] = decay scores[b][h][t] + w   for the lens[b] cached tokens,
 *                   = w                           for the nodes' own tokens,
 * in place; numbers of tokens past those, and of tokens from S on, stay as they are.  A
 * row whose lse is infinite or no number adds nothing (tokens that a verification has
 * rejected: lse = -inf).  scores fp32, number t of head h of sequence b at s_seq b +
 * s_head h + t, none of which may share an address.  fp32 sums, in an order that does
 * not change from run to run.
 * Limits as tq_tree_attention's, T G <= 8192, S <= 2^30.  Errors likewise; TQ_ERR_VALUE
 * for a decay outside [0, 1].  B, T or S = 0 is a no-op. */
int tq_cache_weights(int dtype, const void* Q, int64_t q_seq, int64_t q_tok, int64_t q_head,
                     const void* k_pages, int64_t n_pages, int64_t page_size, int64_t page_stride,
                     int64_t row_stride, int64_t head_stride, const int32_t* page_table,
                     int64_t width, const int32_t* lens, const int32_t* nodes, const int64_t* mask,
                     int64_t mask_seq, const float* lse, int64_t B, int64_t T, int64_t Hq,
                     int64_t Hkv, int64_t D, double scale, int64_t window, double decay,
                     float* scores, int64_t s_seq, int64_t s_head, int64_t S, void* stream);

/* Which tokens stay: of each sequence and head, with n = lens[b] tokens (negative counts
 * as 0, and S at most) all, where n <= budget, else `budget` of them: the first `sinks`,
 * the last `recent`, and of the others those of the largest scores (equal ones by the
 * lowest index; NaN counts as -inf, -0 as 0).  scores fp32, number t of head h of
 * sequence b at s_seq b + s_head h + t, t < S.
 * keep int32 [B][H][budget]: their indexes, ascending, then -1; counts int32 [B]:
 * min(n, budget); sums fp32 [B][H][budget] or NULL: their scores, then 0.
 * All device pointers.  sinks + recent <= budget <= 2^30, S <= 2^30, B <= 2^20, H <= 2^12,
 * B H < 2^22.  Outputs must not overlap the inputs.  Errors: TQ_ERR_NULL, TQ_ERR_SHAPE,
 * TQ_ERR_ALIGN, TQ_ERR_DEVICE.  B = 0 is a no-op; H = 0 writes counts alone, unless that is NULL. */
int tq_cache_select(const float* scores, int64_t s_seq, int64_t s_head, int64_t S,
                    const int32_t* lens, int64_t B, int64_t H, int64_t budget, int64_t recent,
                    int64_t sinks, int32_t* keep, int32_t* counts, float* sums, void* stream);

/* The pages of a cache.  The page table and the lengths are the whole state: a
 * page is free when no row holds it, and a page held by several rows is shared.
 * The functions read one state and write another, so a step can be repeated and
 * captured; outputs must not overlap inputs.  Tables are int32 [rows][width],
 * lengths int32 [rows] (negative counts as 0; at most width * page_size tokens
 * are looked at).  Output rows are written whole, -1 past the held entries.
 * The pool holds `planes` planes (the keys and the values of every layer, say)
 * of n_pages pages of page_bytes contiguous bytes each; a page's copy is made
 * in every plane.  page_bytes a multiple of 16, pool 16-byte aligned.
 * Entries outside [0, n_pages) name no page: they are kept and never followed.
 * Two rows may share the pages that both have filled.  A caller that cuts a length
 * back into such a page has to give that row a page of its own (tq_pages_copy) before
 * it appends there: neither forking nor growing looks for it.
 * workspace: tq_pages_workspace(rows, n_pages) bytes, 16-byte aligned.
 * Limits: rows <= 2^16, width * page_size <= 2^30, n_pages <= 2^24, planes <=
 * 2^16, page_bytes <= 2^30.  Free pages are taken in ascending order for rows
 * in ascending order, so results do not depend on timing. */

/* Forking: row r of the output continues input row parent[r] (no row, an empty
 * sequence, when parent[r] is outside [0, rows_in)).  Pages are shared, except
 * the last one where it is partly filled: the first row that continues a parent
 * keeps it, every further row gets a free page and a copy.  Input rows that no
 * output row continues release their pages, also for these copies.
 * refs int32 [n_pages] or NULL: how many output entries hold each page.
 * short_out int32 [1]: rows for which no free page was left; such a row is cut
 * to its full pages.  This is also how sequences are freed (parent = -1). */
int tq_pages_fork(void* pool, int64_t planes, int64_t n_pages, int64_t page_bytes,
                  const int32_t* table, const int32_t* lens, int64_t rows_in,
                  const int32_t* parent, int64_t rows, int64_t width, int64_t page_size,
                  int32_t* table_out, int32_t* lens_out, int32_t* refs, int32_t* short_out,
                  void* workspace, int64_t workspace_bytes, void* stream);

/* Growing: row r gets add[r] more tokens (negative counts as 0), with free
 * pages for those that its last page cannot hold; nothing is copied.  Where the
 * table's width does not suffice, or the row and those before it need more pages
 * together than are free, the row keeps its length and pages, and short_out
 * int32 [1] counts such rows. */
int tq_pages_grow(const int32_t* table, const int32_t* lens, const int32_t* add, int64_t rows,
                  int64_t width, int64_t page_size, int64_t n_pages, int32_t* table_out,
                  int32_t* lens_out, int32_t* short_out, void* workspace,
                  int64_t workspace_bytes, void* stream);

/* Compacting: with n pages in use, the i-th used page at or above n (in
 * ascending order) moves to the i-th free page below n and the tables follow,
 * so that pages 0 .. n - 1 are used and the rest of the pool can be given back.
 * used_out int32 [1]: n.  Lengths do not change. */
int tq_pages_compact(void* pool, int64_t planes, int64_t n_pages, int64_t page_bytes,
                     const int32_t* table, const int32_t* lens, int64_t rows, int64_t width,
                     int64_t page_size, int32_t* table_out, int32_t* used_out, void* workspace,
                     int64_t workspace_bytes, void* stream);

/* Copying: page src[i] over page dst[i] in every plane, i < n; pairs with
 * either outside [0, n_pages) are left out.  src, dst int32 [n], device.  A
 * page must not be a destination twice, nor both a source and a destination. */
int tq_pages_copy(void* pool, int64_t planes, int64_t n_pages, int64_t page_bytes,
                  const int32_t* src, const int32_t* dst, int64_t n, void* stream);

/* Keeping some tokens: row r keeps its first base[r] tokens (base NULL: 0; clipped to its
 * length) and then the counts[r] tokens that keep lists (clipped to n and to what
 * the row has after base[r]); they move together, and pages past the last one are
 * released.  What an eviction leaves (tq_cache_select's indexes), or the accepted path of
 * a tree: base the length before the nodes, keep base + the path's nodes.
 * A token is `heads` parts of page_bytes / page_size / heads bytes, each with a list of
 * its own, and every run of planes / groups planes likewise: keep int32
 * [groups][rows][heads][n].  Slot base[r] + i gets token keep[..][i].  Lists ascend, so
 * that entry i is base[r] + i at least; for an entry below that, or past the row's length,
 * the slot keeps its token.  Slots past the last token, and those of pages that a row
 * releases, stay as they are.
 * A page that is held by more than one table entry is not written: where a token in it
 * would change, the row gets a free page in its place, with its kept tokens.  A row that
 * needs pages, and together with those before it more than are free, keeps its tokens, length
 * and pages, and short_out int32 [1] counts such rows; one that needs none never does.  lens_out int32 [rows]: base +
 * counts.  page_bytes a multiple of page_size * heads * 16, planes one of groups; heads
 * <= 2^16, groups * heads < 2^31.  workspace: tq_pages_keep_workspace(rows, width, n_pages)
 * bytes. */
int tq_pages_keep(void* pool, int64_t planes, int64_t n_pages, int64_t page_bytes,
                  const int32_t* table, const int32_t* lens, int64_t rows, int64_t width,
                  int64_t page_size, const int32_t* keep, int64_t groups, int64_t heads, int64_t n,
                  const int32_t* counts, const int32_t* base, int32_t* table_out,
                  int32_t* lens_out, int32_t* short_out, void* workspace, int64_t workspace_bytes,
                  void* stream);

/* Workspace bytes of tq_pages_keep; TQ_ERR_SHAPE for sizes that it refuses. */
int64_t tq_pages_keep_workspace(int64_t rows, int64_t width, int64_t n_pages);

/* Workspace bytes of fork, grow and compact; TQ_ERR_SHAPE for sizes that they
 * refuse. */
int64_t tq_pages_workspace(int64_t rows, int64_t n_pages);

#ifdef __cplusplus
}
#endif

#endif /* TQ_H_ */
