/*
 * pql.h -- C ABI of libpql, the quantized-linear hot path for AMD MI355X (gfx950).
 *
 * Two steps, as the pages describe the online-quantized linear layer:
 *   1. quantize bf16 activations (every call) and weights (once, at load) into
 *      block-scaled low-precision codes plus scales;
 *   2. a scaled GEMM on those codes, C = A * W^T, returning bf16.
 * ("vLLM-Omni Online Quantization complete guide", section "How online
 *  quantization works underneath", steps 1-3; "[vLLM] Other quantization: FP8,
 *  ModelOpt, INC, TorchAO, Quark", section "FP8"; "vLLM-Omni accelerates
 *  inference with AutoRound quantization", section "Usage".)
 *
 * Conventions for every call:
 *   - Operands: A is [M, K] (tokens x input channels), W is [N, K] (output x
 *     input channels, a linear layer's own layout), C is [M, N].  K is the
 *     contraction axis and is contiguous in every operand.
 *   - All pointers except the size outputs are DEVICE pointers on the current
 *     HIP device.  The caller allocates and owns every buffer, including
 *     workspace; the library allocates no device memory and keeps no state
 *     besides a per-device property cache, a thread-local error message and
 *     the static device buffer of pql_qlinear_noalloc (see there).
 *   - Work is enqueued on `stream` (a hipStream_t; NULL is the null stream)
 *     and the call returns without synchronizing.  Calls are re-entrant.
 *   - Every argument check runs before anything is enqueued; on any error
 *     nothing is enqueued and pql_last_error() describes the problem.
 *   - Launch log: with the environment variable PQL_LOG set to anything but
 *     "" or "0" (read once, at the first call), pql_quantize,
 *     pql_quantize_static, pql_dequantize, pql_qgemm(_ex), pql_qlinear(_ex),
 *     pql_qlinear_noalloc, pql_repack, the expert calls (pql_moe_*,
 *     pql_swiglu_quantize) and those of the cache (pql_rope, pql_kv_*) each
 *     write one line to stderr: the
 *     call, scheme, role and shape, then the kernel enqueued (the name
 *     pql_kernel_name gives) and the stream, "nothing to do" for an empty
 *     operand, or "rejected (status S)" with the pql_last_error() text.
 *   - Element sizes: bf16 = 2 bytes, fp32 = 4 bytes.  Leading dimensions
 *     (ldx, ldy, lda, ldc) are in elements.  Device pointers must be 16-byte
 *     aligned and leading dimensions multiples of 8 elements (ldc: any value
 *     >= N).  The span a leading dimension addresses, (rows - 1) * ld + cols,
 *     must stay within 2^40 elements (INVALID_ARGUMENT otherwise).
 *
 * Packed layouts: what every call below except pql_repack produces and
 * consumes, laid out for the GEMM kernels (per scheme; rows = M for
 * activations, N for weights, cols = K):
 *   FP8_TENSOR    codes u8 e4m3fn [rows, cols]          scales f32 [1]
 *   FP8_ROW       codes u8 e4m3fn [rows, cols]          scales f32 [rows]
 *   FP8_BLOCK128  codes u8 e4m3fn [rows, cols]          scales f32 [rows, cols/128] (activation)
 *                                                       scales f32 [rows/128, cols/128] (weight)
 *   MXFP8         codes u8 e4m3fn [rows, cols]          scales u8 e8m0, packed [G, rows, 4]
 *   MXFP4         codes u8 [rows, cols/2], two e2m1,    scales u8 e8m0, packed [G, rows, 8]
 *                 element 2j in the low nibble
 *   W4A16_ASYM    codes u32 [rows, cols/8], element k   scales bf16 [cols/128, rows]
 *                 at bits 4*(k mod 8)                   zeros u8 [cols/128, rows] (0..15)
 *   W4A16_SYM     as W4A16_ASYM with every zero-point 8
 *   INT8_ROW      codes i8 [rows, cols] (two's         scales f32 [rows]
 *                 complement)
 *   MXFP4_DUAL    codes as MXFP4                       scales: fine e8m0 packed [G, rows, 8], then
 *                                                       from the next 256-byte boundary coarse
 *                                                       f32 [cols/512, rows] (group-major)
 * All codes are K-contiguous, which is the operand order the matrix cores
 * consume, so weights need no re-layout after quantization.
 * W4A16 scales and zero-points are group-major ([group, row]): one K-group's
 * values for consecutive weight rows are consecutive, which is how the GEMM
 * stages them.
 * MX scales are packed for the GEMM's staging: with c = 4 (MXFP8) or 8
 * (MXFP4) and G = ceil(cols / (32 c)), byte [g, r, b] is the exponent of row
 * r's 32-element block c g + b (K-elements 32 (c g + b) .. + 31); bytes past
 * the row's last block are 127.  A chunk covers 128 bytes of codes, so the
 * exponents one GEMM step needs for consecutive rows are consecutive bytes.
 *
 * Canonical layouts (PQL_LAYOUT_CANONICAL): the same codes, with the scales
 * and zero-points of every row together: MX exponents u8 [rows, cols/32],
 * W4A16 scales bf16 [rows, cols/128] and zero-points u8 [rows, cols/128],
 * MXFP4_DUAL fine exponents u8 [rows, cols/32] then (from the next 256-byte
 * boundary, as packed) coarse f32 [rows, cols/512]; for every other scheme the
 * canonical and packed layouts are the same bytes.
 * pql_repack converts between the two on the device.
 */
#ifndef PQL_H
#define PQL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define PQL_VERSION 2

typedef enum pql_status {
  PQL_OK = 0,
  PQL_ERR_INVALID_ARGUMENT = 1, /* null pointer, bad size, stride or alignment */
  PQL_ERR_UNSUPPORTED = 2,      /* scheme x role not defined, or device is not gfx950 */
  PQL_ERR_WORKSPACE = 3,        /* workspace missing or smaller than pql_workspace_size() */
  PQL_ERR_HIP = 4               /* HIP runtime error (no device, launch failure) */
} pql_status;

/* Quantization schemes.
 *   FP8_TENSOR / FP8_ROW / FP8_BLOCK128: dynamic symmetric FP8 e4m3fn with an
 *     fp32 scale per tensor, per row (per token for activations, per output
 *     channel for weights) or per block (1x128 for activations, 128x128 for
 *     weights) ("[vLLM] Other quantization...", section "FP8").
 *     s = fp32(amax / 448) (1 if that is 0); code = e4m3fn(fp32(x / s)),
 *     round to nearest even, saturating at +-448, sign of zero kept.
 *   MXFP8 / MXFP4: OCP MX, one e8m0 exponent per 32 consecutive K-elements
 *     ("vLLM-Omni Online Quantization complete guide", section "How online
 *     quantization works underneath", steps 2-3).
 *     X = clamp(floor(log2 amax) - emax, -127, 127) (emax 8 for e4m3, 2 for
 *     e2m1; amax = 0 gives -127), scale code X + 127, code = RNE_sat(x * 2^-X).
 *   W4A16_ASYM / W4A16_SYM: int4 weights, group 128 along K, bf16 scale and
 *     4-bit zero-point per group; activations stay bf16 ("vLLM-Omni
 *     accelerates inference with AutoRound quantization", section "Usage").
 *     Weight quantization is round-to-nearest:
 *       asym: s = bf16(fp32(fp32(max(0,max x) - min(0,min x)) / 15)),
 *             z = clamp(rne(fp32(-min(0,min x) / s)), 0, 15)
 *       sym:  s = bf16(fp32(max|x| / 7)), z = 8
 *       q = clamp(rne(fp32(x / s)) + z, 0, 15); s = 0 is replaced by 1 (z = 0 asym).
 *   INT8_ROW: int8 W8A8, symmetric, one fp32 scale per row (per token for
 *     activations, per output channel for weights), dynamic only ("vLLM-Omni
 *     Online Quantization complete guide", sections "Key parameters in
 *     detail" and "How online quantization works underneath": the int8
 *     online path quantizes weights with weight scales; its activation
 *     scales are dynamic, a static activation scheme is an error).
 *     s = fp32(amax / 127) (1 if that is 0); code = clamp(rne(fp32(x / s)), -128, 127).
 *   MXFP4_DUAL: MXFP4 with two online scale levels, a coarse fp32 scale per
 *     512 K-elements and a fine e8m0 exponent per 32 ("vLLM-Omni Online
 *     Quantization complete guide", section "How online quantization works
 *     underneath", MXFP4 paragraph; the calibrated multiplier of offline
 *     checkpoints is all ones online and leaves x unchanged).  K % 512 == 0.
 *     s_c = fp32(amax_512 / 6) (1 if 0); v = fp32(x / s_c) (correctly
 *     rounded); X = clamp(floor(log2 max|v|) - 2, -127, 127) per 32-block;
 *     code = RNE_sat_e2m1(v * 2^-X).  Dequantized: fp32(decode * 2^X) * s_c.
 *     No fused alpha / bias epilogue.
 */
typedef enum pql_scheme {
  PQL_FP8_TENSOR = 0,
  PQL_FP8_ROW = 1,
  PQL_FP8_BLOCK128 = 2,
  PQL_MXFP8 = 3,
  PQL_MXFP4 = 4,
  PQL_W4A16_ASYM = 5,
  PQL_W4A16_SYM = 6,
  PQL_INT8_ROW = 7,
  PQL_MXFP4_DUAL = 8
} pql_scheme;

typedef enum pql_role { PQL_ACTIVATION = 0, PQL_WEIGHT = 1 } pql_role;

typedef enum pql_layout { PQL_LAYOUT_CANONICAL = 0, PQL_LAYOUT_PACKED = 1 } pql_layout;

typedef enum pql_op {
  PQL_OP_QUANTIZE = 0,
  PQL_OP_DEQUANTIZE = 1,
  PQL_OP_QGEMM = 2,
  PQL_OP_QLINEAR = 3
} pql_op;

/* Library version (PQL_VERSION). */
int pql_version(void);

/* Text of the last error on the calling thread ("" if none).  The pointer
 * stays valid until the thread's next pql call. */
const char* pql_last_error(void);

/* Byte sizes of the codes, scales and zero-point buffers of a quantized
 * [rows, cols] tensor in the packed layout (zeros_bytes is 0 except for
 * W4A16).  Size outputs are host pointers; any may be NULL.
 * Errors: INVALID_ARGUMENT for negative sizes or cols / rows that the scheme
 * cannot block (cols % 32 for FP8 tensor/row, INT8_ROW and MX, cols % 128 for
 * FP8_BLOCK128 and W4A16, rows % 128 for FP8_BLOCK128 weights), and for
 * cols > 2^20, rows > 2^31 - 1 or rows * cols > 2^40 (the same limits hold for
 * every quantize and dequantize call; GEMMs take K <= 2^20, M, N <= 2^30 and
 * at most 2^31 - 1 output tiles of 64 x 64);
 * UNSUPPORTED for W4A16 activations or an unknown scheme / role. */
pql_status pql_quantized_sizes(int scheme, int role, int64_t rows, int64_t cols,
                               size_t* codes_bytes, size_t* scales_bytes,
                               size_t* zeros_bytes);

/* pql_quantized_sizes for either layout (PQL_LAYOUT_PACKED gives the same
 * sizes as pql_quantized_sizes; canonical MX scales take rows * cols / 32
 * bytes, without the packed layout's padding).  Same errors, plus
 * INVALID_ARGUMENT for an unknown layout. */
pql_status pql_layout_sizes(int scheme, int role, int layout, int64_t rows, int64_t cols, size_t* codes_bytes,
                            size_t* scales_bytes, size_t* zeros_bytes);

/* Convert a quantized tensor's scales (and W4A16 zero-points) from one layout
 * to the other on the device ("vLLM-Omni Online Quantization complete
 * guide", section "How online quantization works underneath", step 2: online
 * weights are brought into the layout the GEMM consumes, with the scales
 * rearranged to match).  Codes are the same bytes in both layouts and are not
 * touched.  scales_in / zeros_in are in `from_layout`, scales_out /
 * zeros_out (caller-allocated, pql_layout_sizes(to_layout) bytes) receive
 * `to_layout`; zeros are required for W4A16 and ignored otherwise.  When the
 * two layouts are the same bytes (the layouts are equal, or the scheme has
 * one layout) this is a device copy, nothing if input and output coincide;
 * otherwise input and output must be distinct buffers.  Errors: as
 * pql_quantize's shape checks, INVALID_ARGUMENT for an unknown layout, NULL
 * buffers or overlapping buffers of a transposing repack. */
pql_status pql_repack(int scheme, int role, int from_layout, int to_layout, const void* scales_in,
                      const void* zeros_in, void* scales_out, void* zeros_out, int64_t rows, int64_t cols,
                      void* stream);

/* Workspace bytes a call needs (host output).  op = PQL_OP_QUANTIZE: the
 * per-tensor scheme needs a small partial-maximum buffer, the others 0.
 * op = PQL_OP_QLINEAR: room for the activation's codes and scales (0 for
 * W4A16).  Other ops need none.  `role` matters for QUANTIZE only. */
pql_status pql_workspace_size(int op, int scheme, int role, int64_t M, int64_t N,
                              int64_t K, size_t* bytes);

/* Quantize a bf16 tensor x[rows, cols] (row stride ldx elements) into the
 * packed layout.  Activation role: rows = M; weight role: rows = N.
 * `zeros` is written for W4A16 only (may be NULL otherwise).  The scales are
 * dynamic (computed from x).  FP8_TENSOR needs `workspace` of at least
 * pql_workspace_size(PQL_OP_QUANTIZE, ...) bytes; other schemes ignore it.
 * rows = 0 is a no-op. */
pql_status pql_quantize(int scheme, int role, const void* x, int64_t rows, int64_t cols,
                        int64_t ldx, void* codes, void* scales, void* zeros,
                        void* workspace, size_t workspace_bytes, void* stream);

/* y[rows, cols] (bf16, row stride ldy) = bf16_RNE(fp32(decode(code) * scale))
 * (W4A16: bf16_RNE((q - z) * s)).  Inputs in the packed layout. */
pql_status pql_dequantize(int scheme, int role, const void* codes, const void* scales,
                          const void* zeros, int64_t rows, int64_t cols, void* y,
                          int64_t ldy, void* stream);

/* C[M, N] (bf16, row stride ldc) = A_hat * W_hat^T on already-quantized
 * operands, fp32 accumulation, bf16 round-to-nearest-even output.
 *   FP8 / MX schemes: a = activation codes [M, K], a_scales its scales
 *   (packed activation layout); w_codes / w_scales the weight's.
 *   W4A16: a = bf16 activation [M, K] (contiguous), a_scales unused (NULL),
 *   w_zeros required.
 * K must be a multiple of 128; M, N >= 1 may be ragged (tails are masked);
 * FP8_BLOCK128 needs N % 128 == 0 (the weight's 128-row blocks). */
pql_status pql_qgemm(int scheme, const void* a, const void* a_scales, const void* w_codes,
                     const void* w_scales, const void* w_zeros, int64_t M, int64_t N,
                     int64_t K, void* c, int64_t ldc, void* stream);

/* The linear layer's forward: quantize the bf16 activation a[M, K] (row
 * stride lda) with the scheme's activation rule into `workspace`, then
 * qgemm against the quantized weight.  W4A16 uses a as-is (lda must equal K)
 * and needs no workspace.  C as for pql_qgemm.
 * A few tokens (1 <= M <= 16) under FP8_TENSOR, FP8_ROW, FP8_BLOCK128 or
 * INT8_ROW take one fused launch instead ("vLLM-Omni Online Quantization
 * complete guide", section "How online quantization works underneath": the
 * activation quantize fused into the GEMM): each workgroup recomputes the
 * activation's scales and codes on chip, with the same rule and the same
 * codes as pql_quantize, and the workspace is neither needed nor touched
 * (pql_workspace_size gives 0 for these shapes).  The result differs from
 * quantize + qgemm only in the order of the fp32 partial sums. */
pql_status pql_qlinear(int scheme, const void* a, int64_t M, int64_t K, int64_t lda,
                       const void* w_codes, const void* w_scales, const void* w_zeros,
                       int64_t N, void* c, int64_t ldc, void* workspace,
                       size_t workspace_bytes, void* stream);

/* Static-scale FP8 quantization (FP8_TENSOR and FP8_BLOCK128 only): the
 * scale is supplied instead of computed from x ("[vLLM] Other quantization:
 * FP8, ModelOpt, INC, TorchAO, Quark", section "FP8": the static tensor-wise
 * and static 128-block symmetric scheme keys).  `scales` (device, read only)
 * is in the scheme's scale layout for `role` (f32 [1]; f32
 * [rows, cols/128] for activations, f32 [rows/128, cols/128] for weights) and
 * must hold finite positive values (not checked on the device: a zero, NaN or
 * infinite scale gives meaningless codes).  codes = e4m3fn(fp32(x / s)),
 * round to nearest even, saturating at +-448: values beyond 448 s clamp,
 * which a calibrated scale makes possible.  Same shape rules as
 * pql_quantize; rows = 0 is a no-op.  UNSUPPORTED for other schemes
 * (INT8_ROW has no static scheme). */
pql_status pql_quantize_static(int scheme, int role, const void* x, int64_t rows, int64_t cols, int64_t ldx,
                               const void* scales, void* codes, void* stream);

/* pql_qgemm with the fused epilogue ("vLLM-Omni Online Quantization complete
 * guide", section "How online quantization works underneath": the FP8 path's
 * alpha * (A @ B) + bias):
 *   C[m, n] = bf16_RNE(alpha * (A_hat W_hat^T)[m, n] + bias[n])
 * computed in fp32 with one rounding to bf16.  alpha is a finite host fp32;
 * bias is a device bf16 [N] vector (16-byte aligned, N even) or NULL.
 * Defined for FP8_TENSOR, FP8_ROW, FP8_BLOCK128 and INT8_ROW; other schemes
 * are UNSUPPORTED unless alpha == 1 and bias == NULL (then identical to
 * pql_qgemm).  INT8_ROW sums in int32, then scales in fp32.  Other arguments
 * and errors as pql_qgemm. */
pql_status pql_qgemm_ex(int scheme, const void* a, const void* a_scales, const void* w_codes, const void* w_scales,
                        const void* w_zeros, int64_t M, int64_t N, int64_t K, float alpha, const void* bias,
                        void* c, int64_t ldc, void* stream);

/* pql_qlinear with the fused epilogue (alpha, bias as pql_qgemm_ex) and,
 * optionally, static activation scales: with `a_static_scales` non-NULL
 * (FP8_TENSOR: f32 [1]; FP8_BLOCK128: f32 [M, K/128]; device, read only,
 * finite and positive) the activation is quantized with those scales as
 * pql_quantize_static does, and the GEMM reads them in place; NULL means
 * dynamic scales, as pql_qlinear.  Static scales for any other scheme are
 * UNSUPPORTED.  The workspace is the one pql_workspace_size(PQL_OP_QLINEAR)
 * gives, in both cases. */
pql_status pql_qlinear_ex(int scheme, const void* a, int64_t M, int64_t K, int64_t lda, const void* a_static_scales,
                          const void* w_codes, const void* w_scales, const void* w_zeros, int64_t N, float alpha,
                          const void* bias, void* c, int64_t ldc, void* workspace, size_t workspace_bytes,
                          void* stream);

/* pql_qlinear_ex for callers that cannot allocate device memory at call
 * time -- code being captured into a HIP graph, tight serving loops, harnesses
 * that forbid allocation -- and so cannot hand over a workspace.  Arguments,
 * results and errors are those of pql_qlinear_ex without the workspace: the
 * activation's codes and scales go to a static device buffer of the library
 * (pql_noalloc_scratch_bytes(), 64 MiB, held on every device the library runs
 * on until the process ends).  Nothing is allocated or freed, by the library
 * or anything it calls.  An activation whose codes and scales need more than
 * that (pql_workspace_size(PQL_OP_QLINEAR, ...) > pql_noalloc_scratch_bytes())
 * is rejected with PQL_ERR_WORKSPACE before anything is enqueued.  Every call
 * on one device shares that device's buffer and leaves its contents behind
 * (nothing in it needs to start at zero): calls that overlap in time on one
 * device -- on different streams, or from different threads without ordering
 * -- race and give undefined results.  W4A16 uses no buffer. */
pql_status pql_qlinear_noalloc(int scheme, const void* a, int64_t M, int64_t K, int64_t lda, const void* a_static_scales,
                               const void* w_codes, const void* w_scales, const void* w_zeros, int64_t N, float alpha,
                               const void* bias, void* c, int64_t ldc, void* stream);

/* Size in bytes of pql_qlinear_noalloc's static device buffer. */
size_t pql_noalloc_scratch_bytes(void);

/* Name of the kernel that `op` would launch for these sizes (for "no silent
 * fallback" checks); "" if the combination is invalid.  Static string. */
const char* pql_kernel_name(int op, int scheme, int role, int64_t M, int64_t N, int64_t K);

/* ------------------------------------------------------------------ experts
 * The layer of experts around the quantized linear: a router picks k of E
 * experts for each of T tokens, the P = T * k assignments are grouped by
 * expert, every expert's rows are multiplied with its own quantized weight,
 * and the results are summed back to tokens.  One pass, in order:
 *   pql_moe_route -> pql_moe_plan -> pql_quantize (T rows) -> pql_moe_qgemm
 *   (gather) -> pql_swiglu_quantize -> pql_moe_qgemm -> pql_moe_combine
 * Nothing is read back to the host in between: the group sizes stay on the
 * device, so the whole pass can be captured into a HIP graph.
 * Limits: 1 <= E <= 1024, 1 <= k <= 32, T * k <= 2^24 - 1. */

/* Element types of router logits. */
typedef enum pql_dtype { PQL_F32 = 0, PQL_BF16 = 1, PQL_F16 = 2 } pql_dtype;

/* Scores of the experts from the logits x[t, :]: softmax over all E, or a
 * sigmoid of each. */
typedef enum pql_moe_score { PQL_MOE_SOFTMAX = 0, PQL_MOE_SIGMOID = 1 } pql_moe_score;

/* Score of a group of experts: its highest choice, or the sum of its two
 * highest (of the one, where only one is available). */
typedef enum pql_moe_group { PQL_MOE_GROUP_MAX = 0, PQL_MOE_GROUP_TOP2 = 1 } pql_moe_group;

/* The k experts of each token and their weights.
 *   s = softmax(x) or sigmoid(x);  the choice is s + bias[e] with a bias (fp32
 *   [E], for balance; it decides who is chosen, not the weight), formed in
 *   64 bits, and the order of the logits themselves without one.
 *   With groups > 1 (E / groups consecutive experts each) only the experts of
 *   the top_groups groups with the highest group scores take part.
 *   ids[t, 0..k-1]: the experts of highest choice, best first; equal choices
 *   go to the lowest index (experts and groups alike).
 *   weights[t, j] = s of ids[t, j], divided by the sum over the k if
 *   `renormalize` (0 where that sum is 0), times `scale`.
 * A logit of -inf (or a bias of -inf or NaN) makes an expert unavailable;
 * slots for which no expert is left get id -1 and weight 0.  A row that holds
 * a NaN or +inf gets id -1 and weight NaN in every slot, and
 * pql_moe_combine then gives NaN for that token.
 * logits: [T, E], row stride ldl >= E, aligned to its element type.  ids
 * (int32) and weights (fp32): [T, k], contiguous.  T = 0 is a no-op. */
pql_status pql_moe_route(int score, int dtype, const void* logits, int64_t T, int64_t E, int64_t ldl,
                         const float* bias, int64_t k, int64_t groups, int64_t top_groups, int group_score,
                         int renormalize, float scale, int32_t* ids, float* weights, void* stream);

/* Workspace bytes of pql_moe_plan (host output; may be 0). */
pql_status pql_moe_plan_workspace(int64_t T, int64_t k, int64_t E, size_t* bytes);

/* Group the assignments i = t * k + j (ids[i], [T, k] contiguous) by expert,
 * in order of i within an expert.  An id outside 0 .. E - 1 (an expert held
 * elsewhere, or none) takes no part.
 *   offsets int32 [E + 1]: expert e has positions offsets[e] .. offsets[e+1]-1
 *   order   int32 [P]: order[p] = i for the position p; -1 from offsets[E] on
 *   slots   int32 [P]: slots[i] = p, or -1 where the id takes no part
 * T = 0 writes zero offsets.  The result is the same on every run. */
pql_status pql_moe_plan(const int32_t* ids, int64_t T, int64_t k, int64_t E, int32_t* offsets, int32_t* order,
                        int32_t* slots, void* workspace, size_t workspace_bytes, void* stream);

/* The experts' products, FP8_ROW and FP8_BLOCK128:
 *   C[p, n] = bf16( sum_k a_hat[row(p), k] w_hat[e * N + n, k] )
 * for every position p < offsets[E], e the expert whose range holds p,
 * fp32 accumulation as in pql_qgemm.  gather != 0: row(p) = order[p] / k, the
 * assignment's token (the activation has T rows); gather = 0: row(p) = p (T * k
 * rows, order may be NULL).  w_codes / w_scales: the E weights [N, K] stacked,
 * i.e. what pql_quantize writes for the [E * N, K] weight (FP8_BLOCK128 needs
 * N % 128 == 0).  Rows of C from offsets[E] on are left as they were.  offsets
 * and order are pql_moe_plan's; values outside their ranges are clamped, never
 * followed.  K % 128 == 0, N <= 2^20. */
pql_status pql_moe_qgemm(int scheme, const void* a, const void* a_scales, int64_t a_rows, int gather,
                         const void* w_codes, const void* w_scales, const int32_t* offsets, const int32_t* order,
                         int64_t T, int64_t k, int64_t E, int64_t N, int64_t K, void* c, int64_t ldc, void* stream);

/* Gated activation and quantization in one pass, FP8_ROW and FP8_BLOCK128:
 *   h[r, c] = silu(x[r, c]) * x[r, cols + c],  silu(g) = g / (1 + exp(-g)),
 * from a bf16 [rows, 2 * cols] tensor (gate half, then up half; row stride ldx),
 * kept in fp32, then quantized by the scheme's activation rule into codes (saturating,
 * also where a scale is subnormal) and scales as pql_quantize lays them out.  row_count (device int32, or NULL): rows
 * from *row_count on are left as they were -- offsets + E of a plan, so that
 * positions of experts held elsewhere cost nothing.  h must be finite.  rows <= 2^24 - 1;
 * rows = 0 is a no-op. */
pql_status pql_swiglu_quantize(int scheme, const void* x, int64_t rows, int64_t cols, int64_t ldx,
                               const int32_t* row_count, void* codes, void* scales, void* stream);

/* out[t, n] = bf16( add[t, n] + sum_j weights[t, j] * y[slots[t * k + j], n] )
 * in fp32, j ascending, `add` (bf16 [T, N], a shared expert's output or a
 * residual; may be `out` itself) last, one rounding.  A slot outside
 * 0 .. y_rows - 1 contributes weights[t, j] * 0.  Row strides in elements, any
 * value >= N; rows that all start on 16 bytes with N % 8 == 0 run fastest. */
pql_status pql_moe_combine(const void* y, int64_t y_rows, int64_t ldy, const int32_t* slots, const float* weights,
                           int64_t T, int64_t k, int64_t N, const void* add, int64_t ldadd, void* out, int64_t ldo,
                           void* stream);

/* Name of the kernel pql_moe_qgemm would launch; "" if the combination is invalid. */
const char* pql_moe_kernel_name(int scheme, int gather, int64_t T, int64_t k, int64_t E, int64_t N, int64_t K);

/* -------------------------------------------------- cache of keys and values
 * The attention of a layer beside its quantized linears: q and k are turned by
 * their positions, k and v go into a paged cache, quantized as they are written
 * ("[vLLM] Other quantization: FP8, ModelOpt, INC, TorchAO, Quark", section
 * "ModelOpt": KV-cache quantization), and the new tokens attend over the pages.
 * Per layer and step:
 *   pql_rope (q) -> pql_kv_append (k, v) -> pql_kv_attention
 * with pql_kv_slots once per step.  Nothing is read back to the host, so a
 * step can be captured into a HIP graph.
 *
 * A cache holds n_pages pages of page_size tokens (a power of two, 16 .. 2^16;
 * n_pages * page_size <= 2^31 - 1) for Hk heads of D values, D one of 64, 128,
 * 192, 256, a page of all heads below 2^31 bytes:
 *   KV_BF16        k, v bf16 [n_pages, Hk, page_size, D]            no scales
 *   KV_FP8_TENSOR  k, v e4m3fn codes of the same shape              scales f32 [1] each,
 *                                                                   given by the caller
 *   KV_FP8_ROW     k, v e4m3fn codes of the same shape              scales f32 [n_pages, Hk, page_size]
 * (FP8: the rules of the schemes of that name, a row being one token's head.)
 * Token slot s is place s % page_size of page s / page_size.  Nothing in a
 * cache needs to be initialised: a slot that no token was written to is never
 * part of an answer.
 *
 * A batch is B sequences: the new tokens of sequence b are the rows
 * starts[b] .. starts[b + 1] - 1 of q, k and v (starts int32 [B + 1], not
 * decreasing), lens[b] (int32) is its number of tokens in the cache with the
 * new ones, and pages[b, p] (int32 [B, width], row stride ldp >= width) the
 * page of its tokens p * page_size on.  The i-th of n new tokens is at
 * position lens[b] - n + i.  Values outside their ranges are never followed:
 * starts are cut to 0 .. T, negative lens to 0, and tokens past the width pages
 * or on a page outside 0 .. n_pages - 1 are absent.
 * Row strides ld*t (token) and ld*h (head) are in elements, any multiples of 8;
 * the D values of a head are contiguous and start on 16 bytes.
 * Limits: T * H * D <= 2^34 (T * Hk * D where keys and values are appended,
 * n * Hk * D where they are read; T <= 2^31 - 1 for pql_kv_slots), B <= 2^20,
 * width * page_size <= 2^30, (B - 1) * ldp <= 2^40, 2^40 values in a half of a
 * cache or from the first to the last of an operand.  pql_kv_attention:
 * H <= 65535, and fewer than 2^24 workgroups, T * H / r + min(B, T) * Hk of which
 * are its tiles of r = 16, 32 or 128 rows (a single token for each of 2^20
 * sequences with 15 heads of the cache is within, with 16 not);
 * pql_kv_attention_workspace refuses what is past it. */

typedef enum pql_kv_scheme { PQL_KV_BF16 = 0, PQL_KV_FP8_TENSOR = 1, PQL_KV_FP8_ROW = 2 } pql_kv_scheme;

/* Which values of a head form the pairs that are turned: (i, i + rotary / 2),
 * or (2 i, 2 i + 1). */
typedef enum pql_rope_layout { PQL_ROPE_HALF = 0, PQL_ROPE_INTERLEAVED = 1 } pql_rope_layout;

/* Rotary positions: the first `rotary` values of every head of x[T, H, D] are
 * turned pair by pair,
 *   (x1, x2) -> scale * (x1 cos a - x2 sin a, x2 cos a + x1 sin a),
 *   a = positions[t] * freqs[i] radians,
 * the others copied.  freqs: device fp64 [rotary / 2]; the angle is formed and
 * reduced in fp64, so positions far out keep theirs, the rest is fp32 with one
 * rounding to bf16.  out may be x itself with the same strides (no other
 * overlap).  rotary: a multiple of 16 up to D, D a multiple of 8, 16 to 1024;
 * positions int32.  T = 0 is a no-op. */
pql_status pql_rope(int layout, const void* x, int64_t T, int64_t H, int64_t D, int64_t ldxt, int64_t ldxh,
                    const int32_t* positions, const double* freqs, int64_t rotary, float scale, void* out,
                    int64_t ldot, int64_t ldoh, void* stream);

/* Byte sizes of each of a cache's two codes buffers and of its two scales
 * buffers (host outputs, either may be NULL). */
pql_status pql_kv_sizes(int scheme, int64_t n_pages, int64_t page_size, int64_t Hk, int64_t D, size_t* codes_bytes,
                        size_t* scales_bytes);

/* slots[t] and positions[t] (int32 [T]) of a batch's new tokens.  Rows of no
 * sequence get slot -1 and position 0, as does a token before the start of its
 * sequence (more new tokens than lens[b]); a token past its row of pages or on a
 * negative page gets slot -1. */
pql_status pql_kv_slots(const int32_t* starts, const int32_t* lens, const int32_t* pages, int64_t B, int64_t width,
                        int64_t ldp, int64_t page_size, int64_t T, int32_t* slots, int32_t* positions, void* stream);

/* Write T tokens' keys and values into the slots[t] of a cache.  A slot
 * outside 0 .. n_pages * page_size - 1 writes nothing (padding); a slot named
 * twice holds one of its two tokens' values in each byte, which is not said.
 * With positions (int32 [T]; NULL: none) the keys are turned first, as pql_rope
 * does, and quantized from fp32 without a rounding in between; layout, freqs,
 * rotary and rope_scale as there.
 * KV_FP8_TENSOR reads its scales (finite and positive), KV_FP8_ROW writes them:
 * s = fp32(amax / 448) over the head (1 if 0), code = e4m3fn(fp32(x / s)),
 * saturating.  A NaN stays a NaN (and an infinity makes its row NaN under
 * KV_FP8_ROW). */
pql_status pql_kv_append(int scheme, const void* k, int64_t ldkt, int64_t ldkh, const void* v, int64_t ldvt,
                         int64_t ldvh, int64_t T, const int32_t* slots, int layout, const int32_t* positions,
                         const double* freqs, int64_t rotary, float rope_scale, void* k_codes, void* v_codes,
                         float* k_scales, float* v_scales, int64_t n_pages, int64_t page_size, int64_t Hk, int64_t D,
                         void* stream);

/* The keys and values of n slots back in bf16, bf16_RNE(fp32(decode(code) * s)),
 * as k_out and v_out [n, Hk, D].  A slot outside the cache reads as zeros. */
pql_status pql_kv_read(int scheme, const void* k_codes, const void* v_codes, const float* k_scales,
                       const float* v_scales, int64_t n_pages, int64_t page_size, int64_t Hk, int64_t D,
                       const int32_t* slots, int64_t n, void* k_out, int64_t ldkt, int64_t ldkh, void* v_out,
                       int64_t ldvt, int64_t ldvh, void* stream);

/* Workspace bytes of pql_kv_attention (host output; may be 0). */
pql_status pql_kv_attention_workspace(int scheme, int64_t T, int64_t H, int64_t Hk, int64_t D, int64_t B,
                                      int64_t width, int64_t page_size, size_t* bytes);

/* Attention of a batch's new tokens over its pages, H query heads of which
 * H / Hk consecutive ones share a head of the cache:
 *   out[t, h] = sum_j p_j v_j,  p = softmax over the visible j of scale * q[t, h] . k_j
 * j runs over the sequence's tokens; with causal != 0 a token at position i
 * sees j <= i, with window > 0 only j > i - window.  q: bf16 [T, H, D]; scores,
 * sums and the joining of a split context are fp32, the weights p enter the
 * matrix cores in 16 bits (fp16 for FP8 caches, where one that is, with its value's
 * scale, below 2^-21 of its row's largest is exact to 2^-32 of that; bf16 for
 * KV_BF16), one rounding to bf16 at the end.  lse (fp32 [T, H], contiguous, or
 * NULL) receives log sum_j exp(scale q . k_j).
 * A token that sees nothing gets zeros and an lse of -inf.  Rows of no sequence
 * are left as they were.  out and q do not overlap.  A NaN or an infinity in
 * the cache reaches only the tokens that see it, possibly all of their D values.
 * KV_FP8_ROW: values whose scale is below 2^-90 are exact to 2^-113 (a negative
 * scale counts as 0), and a token's weight is lost beside one whose value scale is
 * 2^100 times its own, unless its own is below 2^-90 or its values are all zero.
 * Calls that overlap in time need workspaces of their own. */
pql_status pql_kv_attention(int scheme, const void* q, int64_t ldqt, int64_t ldqh, int64_t T, int64_t H,
                            const void* k_codes, const void* v_codes, const float* k_scales, const float* v_scales,
                            int64_t n_pages, int64_t page_size, int64_t Hk, int64_t D, const int32_t* starts,
                            const int32_t* lens, const int32_t* pages, int64_t B, int64_t width, int64_t ldp,
                            int causal, int64_t window, float scale, void* out, int64_t ldot, int64_t ldoh, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream);

/* Name of the kernel pql_kv_attention would launch; "" if the combination is invalid. */
const char* pql_kv_kernel_name(int scheme, int64_t T, int64_t H, int64_t Hk, int64_t D, int64_t B, int64_t width,
                               int64_t page_size);

#ifdef __cplusplus
}
#endif

#endif /* PQL_H */
