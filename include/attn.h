/*
 * attn.h: C ABI of the GB300 (sm_103a) exact multi-head attention library.
 *
 * The operation comes from "Self-attention, CUDA kernels and FlashAttention" (2026-11-15):
 *   section 1 "How self-attention works mathematically in a Vision Transformer":
 *       Scores = Q K^T / sqrt(d_k); a softmax along each row (each row sums to one);
 *       Attention(Q, K, V) = softmax(Q K^T / sqrt(d_k)) V; the same computation runs
 *       independently for every head.
 *   section 3 "FlashAttention: solving the Transformer memory bottleneck":
 *       tiled, fused evaluation that never stores the N x N matrix in HBM ("Tiling"), an
 *       online softmax ("The online softmax trick"), and a backward pass that keeps only
 *       small per-row normalisation statistics and recomputes the attention tiles on chip
 *       ("Recomputation in backpropagation").
 *
 * Conventions shared by every entry point:
 *   - Tensors are dense, contiguous, row-major [B, H, N, d_k] bf16 (`const void *` / `void *`
 *     here, so that the header needs no CUDA half-precision types).  Row (b, h, i) starts at
 *     element ((b * H + h) * N + i) * d_k.  `lse` and the other per-row vectors are [B, H, N]
 *     fp32.  All pointers are device pointers, 16-byte aligned.
 *   - `scale` multiplies Q K^T before the softmax; pass 1/sqrt(d_k) for the article's
 *     formula.  It must be finite and > 0.
 *   - Supported: d_k in {64, 128}; B, H, N >= 1; B*H*N*d_k < 2^40 elements; N < 2^31.
 *   - Ownership: the caller allocates and owns every buffer, including the forward and
 *     backward workspaces.  The library allocates no device memory on these paths.
 *   - Calls enqueue work on `stream` and return without waiting; only
 *     attn_get_device_status() synchronises (that stream).  Outputs must not overlap inputs.
 *   - The compute calls allocate nothing and never synchronise, so they may be captured in a
 *     CUDA graph on `stream` and replayed (the captured pointers, sizes and scale are fixed).
 *   - Errors: every argument check runs before any launch; on failure the call returns a
 *     non-zero attn_status and launches nothing.  A kernel that cannot make progress does not
 *     hang the GPU: each of its waits gives up after a bounded time and records
 *     ATTN_ERR_TIMEOUT in a per-device status word, read by attn_get_device_status().
 */
#ifndef ATTN_GB300_H
#define ATTN_GB300_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    ATTN_OK = 0,
    ATTN_ERR_INVALID_ARG = 1,     /* null pointer, size < 1, bad scale, overlapping buffers */
    ATTN_ERR_UNSUPPORTED_DK = 2,  /* d_k not in {64, 128} */
    ATTN_ERR_MISALIGNED = 3,      /* a pointer not 16-byte aligned */
    ATTN_ERR_LAUNCH = 4,          /* the CUDA runtime refused a launch or a query */
    ATTN_ERR_TIMEOUT = 5,         /* a kernel wait gave up (reported by attn_get_device_status) */
    ATTN_ERR_WORKSPACE = 6,       /* workspace null, misaligned or smaller than required */
    ATTN_ERR_DEVICE = 7,          /* the current device is not an sm_103 GPU */
    ATTN_ERR_TOO_LARGE = 8        /* attn_bwd_noalloc: sizes need more than its fixed scratch */
} attn_status;

/*
 * Forward pass (section 1's Attention(Q,K,V); section 3's tiling and online softmax).
 *   q, k, v : [B,H,N,d_k] bf16 inputs.
 *   o       : [B,H,N,d_k] bf16 output, O = softmax(scale * Q K^T) V, rounded to nearest.
 *   lse     : [B,H,N] fp32 output, lse[b,h,i] = log(sum_j exp(scale * q_i . k_j)) (natural
 *             log): the per-row statistic the backward pass recomputes the tiles from.
 * Arithmetic: scores in fp32 (tensor cores), softmax statistics in fp32, and the product of
 * the weights with V on fp16 tensor cores: each weight is rounded to fp16 (relative error at
 * most 2^-11) and V is rounded to fp16, which is exact for |v| in [2^-14, 65504]; smaller
 * entries keep an absolute precision of 2^-25, and an entry of V above 65504 in magnitude
 * makes the O rows it contributes to non-finite.  O is normalised by the unrounded row sum.
 */
attn_status attn_fwd(const void *q, const void *k, const void *v, void *o, float *lse, int B,
                     int H, int N, int d_k, float scale, cudaStream_t stream);

/*
 * Diagnostic forward: attn_fwd() (same o and lse, bitwise) that also writes O before it is
 * rounded to bf16, so that the arithmetic's own error can be told apart from the output
 * rounding (section 1's Attention(Q,K,V); the bf16 o is exactly o32 rounded to nearest).
 *   o32 : [B,H,N,d_k] fp32 device output, 16-byte aligned, written with per-row stores (slow:
 *         for tests and measurements, not for training).
 * Errors: as attn_fwd; ATTN_ERR_INVALID_ARG for a null o32 or one overlapping another buffer,
 * ATTN_ERR_MISALIGNED for a misaligned one.
 */
attn_status attn_fwd_diagnostic(const void *q, const void *k, const void *v, void *o, float *lse,
                                float *o32, int B, int H, int N, int d_k, float scale,
                                cudaStream_t stream);

/*
 * Bytes of device workspace attn_fwd_with_workspace() uses for these sizes: an fp16 copy of V
 * (B*H*N*d_k*2 bytes rounded up to a multiple of 256) where the sequence is long enough for
 * one rounding pass over V ahead of the forward kernel to cost less than rounding every V tile
 * in the shared memory of each CTA that reads it (d_k = 64: N >= 2048; d_k = 128: N >= 8192),
 * else 0.  Also 0 for sizes attn_fwd rejects.
 */
size_t attn_fwd_workspace_size(int B, int H, int N, int d_k);

/*
 * The forward pass of attn_fwd() with a caller workspace (section 3's tiled forward; the
 * operation, arguments, layouts, arithmetic and results are attn_fwd's, bitwise: V is rounded
 * to fp16 the same way, only in one pass over HBM into the workspace instead of in shared
 * memory).  Where attn_fwd_workspace_size() is 0 the call is attn_fwd() and `workspace` may
 * be null.
 *   workspace : caller-owned device memory of at least attn_fwd_workspace_size(B,H,N,d_k)
 *               bytes, 256-byte aligned, overwritten; it must not overlap q, k, v, o or lse.
 * Errors: as attn_fwd, plus ATTN_ERR_WORKSPACE (null, misaligned or too small where a
 * workspace is needed) and ATTN_ERR_INVALID_ARG for a workspace overlapping another buffer.
 */
attn_status attn_fwd_with_workspace(const void *q, const void *k, const void *v, void *o, float *lse,
                                    void *workspace, size_t workspace_bytes, int B, int H, int N,
                                    int d_k, float scale, cudaStream_t stream);

/*
 * Bytes of device workspace attn_bwd() needs for these sizes: two fp32 statistics per row
 * (-lse * log2(e) and -rowsum(dO o O), [B,H] x N rounded up to 128, stored interleaved per
 * pair of rows) and an fp32 dQ accumulator ([B,H,N,d_k]), each region 256-byte aligned.
 * Returns 0 if the sizes are unsupported.
 */
size_t attn_bwd_workspace_size(int B, int H, int N, int d_k);

/*
 * Backward pass (section 3, "Recomputation in backpropagation": only the per-row statistic
 * `lse` from attn_fwd is kept; the probabilities are recomputed on chip).  With
 * P = exp(scale * Q K^T - lse) and D_i = sum_c dO_ic O_ic:
 *   dV = P^T dO;   dP = dO V^T;   dS = P o (dP - D);   dQ = scale * dS K;   dK = scale * dS^T Q.
 *   q, k, v, o, dout : [B,H,N,d_k] bf16 inputs (o is attn_fwd's output, dout = dL/dO).
 *   lse              : [B,H,N] fp32 from attn_fwd for the same q, k, scale.
 *   dq, dk, dv       : [B,H,N,d_k] bf16 outputs.
 *   workspace        : device memory of at least attn_bwd_workspace_size(B,H,N,d_k) bytes,
 *                      256-byte aligned, owned by the caller; its contents on entry do not
 *                      matter and on return are unspecified.
 * dQ is accumulated across key tiles with fp32 atomic additions, so its low-order bits may
 * differ from run to run; dK and dV are deterministic.  Exception: for d_k = 64 and N <= 256
 * over at most one head per SM (and N <= 128 or more heads than half the SMs) one kernel takes
 * each head whole and accumulates dQ on chip, without atomics: all three gradients are then
 * bitwise reproducible, and the workspace is not touched.
 */
attn_status attn_bwd(const void *q, const void *k, const void *v, const void *o,
                     const void *dout, const float *lse, void *dq, void *dk, void *dv,
                     void *workspace, size_t workspace_bytes, int B, int H, int N, int d_k,
                     float scale, cudaStream_t stream);

/*
 * The same backward pass with dQ computed without atomics, so that dQ, dK and dV are bitwise
 * reproducible from run to run (the article leaves the scheduling of the recomputation open;
 * this is the alternative to accumulating dQ with fp32 atomics).  Arguments, layouts, workspace
 * and errors are those of attn_bwd().  It runs the preprocess, the key-stationary kernel for dK
 * and dV alone, then a query-stationary pass that recomputes S = scale Q K^T and dP = dO V^T
 * tile by tile and accumulates dQ = scale * dS K in order, one CTA per 128 query rows.  It does
 * 14 instead of 10 B*H*N^2*d_k flops.  Where attn_bwd() takes heads whole (d_k = 64, short
 * sequences, few heads; see there) it runs that same kernel, which needs no atomics.
 */
attn_status attn_bwd_deterministic(const void *q, const void *k, const void *v, const void *o,
                                   const void *dout, const float *lse, void *dq, void *dk,
                                   void *dv, void *workspace, size_t workspace_bytes, int B,
                                   int H, int N, int d_k, float scale, cudaStream_t stream);

/*
 * The three stream-ordered phases attn_bwd() runs, for callers that schedule or time them
 * separately.  Run on one stream, in this order, with the same sizes, scale and workspace,
 * they produce exactly what attn_bwd() produces.
 *
 * attn_bwd_preprocess: reads o, dout and lse; writes into the workspace -D_i, with
 *   D_i = sum_c dO_ic O_ic, and -lse_i * log2(e) (rows padded to a multiple of 128; padding rows
 *   get 0 and -inf, i.e. zero probability), and zeroes the workspace's fp32 dQ accumulator.
 * attn_bwd_main: for every 128-key tile, recomputes P = 2^(scale log2(e) q.k - lse log2(e))
 *   from q, k and the workspace, writes dk (= scale * dS^T Q) and dv (= P^T dO), and adds
 *   dS K into the dQ accumulator.  Reads q, k, v, dout and the workspace.
 * attn_bwd_dq_convert: dq = bf16(scale * accumulator).
 */
attn_status attn_bwd_preprocess(const void *o, const void *dout, const float *lse,
                                void *workspace, size_t workspace_bytes, int B, int H, int N,
                                int d_k, cudaStream_t stream);
attn_status attn_bwd_main(const void *q, const void *k, const void *v, const void *dout,
                          void *dk, void *dv, void *workspace, size_t workspace_bytes, int B,
                          int H, int N, int d_k, float scale, cudaStream_t stream);
attn_status attn_bwd_dq_convert(void *workspace, size_t workspace_bytes, void *dq, int B, int H,
                                int N, int d_k, float scale, cudaStream_t stream);

/*
 * Reads and clears the current device's status word after synchronising `stream`.
 * Returns ATTN_OK, ATTN_ERR_TIMEOUT if a kernel wait gave up since the last call, or
 * ATTN_ERR_LAUNCH if the stream reports a CUDA error.
 */
attn_status attn_get_device_status(cudaStream_t stream);

/* A static, human-readable name for a status code. */
const char *attn_status_string(attn_status status);

/*
 * The CUDA call behind the most recent ATTN_ERR_LAUNCH returned on the calling host thread,
 * with the runtime's error name and text ("no error" if there was none).  The string belongs
 * to the library and stays valid until the thread's next failing call.
 */
const char *attn_last_error_string(void);

/*
 * Diagnostics: launches one tiny kernel that waits, with the library's bounded-wait
 * routine, on a barrier nothing ever signals, giving up after `limit_us` microseconds
 * (1 ... 10^6).  The following attn_get_device_status() must then return ATTN_ERR_TIMEOUT.
 * Used to test the failure path without hanging or faulting the GPU.
 */
attn_status attn_debug_wait_timeout(unsigned limit_us, cudaStream_t stream);

/*
 * Query / key / value projection (section 1, "Generating queries, keys and values":
 * Q = X W_Q, K = X W_K, V = X W_V, each W in R^(D x d_k) per head): the step that feeds
 * attn_fwd.  The heads' weights side by side form one D x D matrix per projection; head h
 * takes its columns [h d_k, (h+1) d_k), and the outputs are written directly in the
 * [B, H, N, d_k] layout attn_fwd reads.
 *   x             : [B, N, D] bf16 (token rows).
 *   w_q, w_k, w_v : [D, D] bf16 row-major (input dimension x output columns).
 *   q, k, v       : [B, H, N, d_k] bf16 outputs (fp32 accumulation, rounded to nearest).
 * Requirements: D = H * d_k, D a multiple of 128, d_k in {64, 128}; pointers 16-byte aligned;
 * outputs overlap neither each other nor the inputs.
 */
attn_status attn_qkv_proj(const void *x, const void *w_q, const void *w_k, const void *w_v,
                          void *q, void *k, void *v, int B, int N, int D, int H, int d_k,
                          cudaStream_t stream);

/*
 * Backward of attn_qkv_proj for the gradients dq, dk, dv ([B, H, N, d_k] bf16, e.g. from
 * attn_bwd): dX = sum_t dY_t W_t^T ([B, N, D] bf16 output) and dW_t = X^T dY_t summed over all
 * B*N tokens ([D, D] fp32 outputs, written from zero).  Where too few dW tiles exist to fill
 * the GPU, the token rows are split across CTAs and their partial sums added with fp32 atomics,
 * so the last bits of dW may then vary between runs.
 * Same size rules as attn_qkv_proj.
 */
attn_status attn_qkv_proj_bwd(const void *x, const void *w_q, const void *w_k, const void *w_v,
                              const void *dq, const void *dk, const void *dv, void *dx,
                              float *dw_q, float *dw_k, float *dw_v, int B, int N, int D, int H,
                              int d_k, cudaStream_t stream);

/*
 * The rest of a transformer block around the attention: the linear layers with their epilogue,
 * the root-mean-square norm, and the 8-bit forms of both.  Shared rules:
 *   - Matrices are dense, row-major bf16 (or e4m3 with fp32 scales where a name ends in _q8);
 *     vectors (bias, norm weight, scales, 1/rms) are fp32.  M counts rows (tokens), 0 <= M < 2^31
 *     (the linear layers: M <= 2^31 - 256, and with several sequences and heads (attn_out_proj) the
 *     sequences, each padded to a multiple of 32 rows, together that many; more are refused with
 *     ATTN_ERR_INVALID_ARG, and their workspace sizes are 0).  With M = 0 the forward calls do nothing
 *     and the backward calls write zeros to the gradients of the parameters.
 *   - Widths (K, N_out, D) are multiples of 8 (K of e4m3 operands: 16) and below 2^20; no operand holds
 *     2^40 elements or more.  Other widths are refused with ATTN_ERR_INVALID_ARG.
 *   - Pointers are 16-byte aligned, and outputs overlap no input and no other output, except
 *     where an entry point allows it by name.
 */
typedef enum {
    ATTN_ACT_NONE = 0,
    ATTN_ACT_RELU = 1,
    ATTN_ACT_GELU = 2,       /* z Phi(z), with the normal distribution function (erf form) */
    ATTN_ACT_GELU_TANH = 3,  /* z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2 */
    ATTN_ACT_SILU = 4        /* z / (1 + exp(-z)) */
} attn_activation;

/*
 * Linear layer: z = x w + bias, y = act(z) + residual, in one kernel.
 *   x : [M, K] bf16.   w : [K, N_out] bf16 (input dimension x output columns, as w_q above).
 *   bias : [N_out] fp32 or null.   residual : [M, N_out] bf16 or null.
 *   y : [M, N_out] bf16 output; it may be `residual` itself.
 *   z : [M, N_out] bf16 output or null: the pre-activation, kept for attn_linear_bwd().
 * Arithmetic: bf16 products summed in fp32, bias, activation and residual in fp32, y and z each
 * rounded once.  The activation is off by at most 2^-20 (1 + |z|) before that, and by 2^-12 of its own
 * value where that is 2^-119 or more in magnitude (left of zero, smaller values may come out as zero).
 */
attn_status attn_linear(const void *x, const void *w, const float *bias, const void *residual,
                        void *y, void *z, int M, int K, int N_out, attn_activation act,
                        cudaStream_t stream);

/*
 * Output projection: attn_linear() without an activation, reading attention's output in the
 * layout attn_fwd() writes it, so that the heads need no copy to be put side by side:
 *   y[b, i, :] = sum_h o[b, h, i, :] w[h d_k : (h+1) d_k, :] + bias + residual[b, i, :].
 * As in attn_fwd(), B, H and N are at least 1: an empty batch is refused here and in the backward
 * (ATTN_ERR_INVALID_ARG), not a call that does nothing.
 *   o : [B, H, N, d_k] bf16.   w : [H * d_k, N_out] bf16.   residual, y : [B, N, N_out] bf16.
 */
attn_status attn_out_proj(const void *o, const void *w, const float *bias, const void *residual,
                          void *y, int B, int H, int N, int d_k, int N_out, cudaStream_t stream);

/*
 * Bytes of device workspace attn_linear_bwd() (with these sizes; act selects whether dz is kept)
 * and attn_out_proj_bwd() need.  Both return 0 for sizes the calls reject.
 */
size_t attn_linear_bwd_workspace_size(int M, int K, int N_out, attn_activation act);
size_t attn_out_proj_bwd_workspace_size(int B, int H, int N, int d_k, int N_out);

/*
 * Backward of attn_linear().  With dz = dy * act'(z) (dz = dy for ATTN_ACT_NONE):
 *   dx = dz w^T;  dw = x^T dz;  dbias = sum over rows of dz.  (The residual's gradient is dy.)
 *   dy : [M, N_out] bf16.   z : [M, N_out] bf16 from attn_linear (null for ATTN_ACT_NONE).
 *   dx : [M, K] bf16, dw : [K, N_out] bf16, dbias : [N_out] fp32; each may be null (not computed).
 *   workspace : caller-owned, 256-byte aligned, at least the size above, overwritten.
 * dz is rounded to bf16 for the two products (the tensor cores' operands are bf16) and summed unrounded
 * for dbias; without an activation it is dy and nothing is rounded before the outputs.  All sums are
 * in fp32 in a fixed order: results are bitwise reproducible.  dw has the weights' type; gradients of
 * many micro-batches are best added up in fp32 by the caller.
 */
attn_status attn_linear_bwd(const void *x, const void *w, const void *dy, const void *z, void *dx,
                            void *dw, float *dbias, void *workspace, size_t workspace_bytes, int M,
                            int K, int N_out, attn_activation act, cudaStream_t stream);

/* Backward of attn_out_proj(): d_o [B, H, N, d_k], dw [H * d_k, N_out], dbias; as above. */
attn_status attn_out_proj_bwd(const void *o, const void *w, const void *dy, void *d_o, void *dw,
                              float *dbias, void *workspace, size_t workspace_bytes, int B, int H,
                              int N, int d_k, int N_out, cudaStream_t stream);

/*
 * Root-mean-square norm with the residual's addition:
 *   h = x + residual (h = x without one);  rstd = 1 / sqrt(mean(h^2) + eps);
 *   y = h * rstd * weight.
 *   x, residual : [M, D] bf16 (residual may be null).   weight : [D] fp32.   0 <= eps, finite.
 *   y : [M, D] bf16 output.   rstd : [M] fp32 output or null, kept for attn_rms_norm_bwd().
 *   h : [M, D] bf16 output or null; may be x or residual itself.  Without a residual it is not
 *       written and must be null.
 * The statistics and y are taken from the unrounded fp32 sum; h and y are each rounded once.  The
 * sum of a row's squares has to fit fp32.
 */
attn_status attn_rms_norm(const void *x, const void *residual, const float *weight, void *y, void *h,
                          float *rstd, int M, int D, float eps, cudaStream_t stream);

/* Bytes of device workspace attn_rms_norm_bwd() needs (0 for sizes it rejects). */
size_t attn_rms_norm_bwd_workspace_size(int M, int D);

/*
 * Backward of attn_rms_norm().  With g = dy * weight and n = h * rstd:
 *   dx = rstd * (g - n * mean(g * n)) + dh;   dweight = sum over rows of dy * n.
 * dx is the gradient of x and of the residual alike.
 *   dy, h : [M, D] bf16.   rstd : [M] fp32.   dh : [M, D] bf16 or null, the gradient that reaches
 *   h by its other uses.   dx : [M, D] bf16 output, may be dh itself.   dweight : [D] fp32 output.
 *   workspace : caller-owned, 256-byte aligned, overwritten.  Bitwise reproducible.
 */
attn_status attn_rms_norm_bwd(const void *dy, const void *h, const float *weight, const float *rstd,
                              const void *dh, void *dx, float *dweight, void *workspace,
                              size_t workspace_bytes, int M, int D, cudaStream_t stream);

/*
 * attn_rms_norm() with y in e4m3 and one fp32 scale a row:
 *   scale = max(max |y|, 1e-30) / 448;  yq = y / scale rounded to nearest e4m3.
 * A row that holds an infinity or a NaN gets a NaN scale: nothing it stands for is finite.
 *   yq : [M, D] e4m3 output.   scale : [M] fp32 output.   Others as attn_rms_norm.
 */
attn_status attn_rms_norm_q8(const void *x, const void *residual, const float *weight, void *yq,
                             float *scale, void *h, int M, int D, float eps, cudaStream_t stream);

/*
 * Rows of x [M, D] bf16 as e4m3 with one fp32 scale each, by the rule of attn_rms_norm_q8(): the
 * activations between two 8-bit products, and (as [N_out, K] rows) the weights of attn_linear_q8().
 */
attn_status attn_quantize_q8(const void *x, void *xq, float *scale, int M, int D, cudaStream_t stream);

/*
 * attn_linear() in 8 bits: z = x_scale[m] w_scale[n] (xq wq^T) + bias, y = act(z) + residual.
 *   xq : [M, K] e4m3, x_scale : [M] fp32.   wq : [N_out, K] e4m3 (one row an output column),
 *   w_scale : [N_out] fp32.   bias, residual, y as attn_linear.   K % 16 = 0, N_out % 8 = 0.
 * e4m3 products (exact) summed in fp32.  The product of the two scales is formed first and has to be a
 * normal fp32 number.
 */
attn_status attn_linear_q8(const void *xq, const float *x_scale, const void *wq, const float *w_scale,
                           const float *bias, const void *residual, void *y, int M, int K, int N_out,
                           attn_activation act, cudaStream_t stream);

/*
 * Diagnostics: the kernels that a call of the linear layers runs, a function of the sizes alone that is
 * decided on the host (no GPU is needed).  kind: 0 attn_linear() / attn_out_proj(), 1 attn_linear_q8(),
 * 2 attn_linear_bwd() / attn_out_proj_bwd() asked for all gradients.  x is [B, H, N, d_k] as in
 * attn_out_proj(), or with B = H = 1 the plain [N, d_k] matrix.  Writes five ints:
 *   plan[0]  rows of a tile of the few-row kernel (16 ... 128) where that makes y (kind 2: dx), else 0
 *   plan[1]  its splits of the sum (1, 2, 4 or 8), else 0
 *   plan[2]  columns of a tile of the pair kernel (128 or 256), 0 where it does not run
 *   plan[3]  kind 2: ways in which dw's sum over the rows is split, else 0
 *   plan[4]  kind 2: dbias from 0 a pass of its own, 1 whole columns or 2 slices of rows beside the products
 * For tests, which assert that they reach every kernel.
 */
attn_status attn_debug_linear_plan(int kind, int B, int H, int N, int d_k, int N_out, attn_activation act,
                                   int *plan);

/*
 * Bytes of device workspace attn_fwd_unfused() needs: the fp32 score matrix S [B,H,N,N] and the
 * bf16 probabilities P [B,H,N,N], each region 256-byte aligned (6 B H N^2 bytes and padding).
 * Returns 0 if the sizes are unsupported.
 */
size_t attn_fwd_unfused_workspace_size(int B, int H, int N, int d_k);

/*
 * Standard attention, the comparison point of section 3 ("memory bandwidth bottleneck"): the
 * same O and LSE as attn_fwd, computed the way the article says frameworks compute it before
 * FlashAttention: S = scale * Q K^T is written to HBM (fp32, by a batched cuBLAS GEMM), a softmax
 * pass reads S and writes P = softmax(S) to HBM (bf16, rounded after normalisation) and LSE, and
 * a second batched cuBLAS GEMM reads P back for O = P V (fp32 accumulation, bf16 output).
 * Memory grows as N^2 per head; the fused attn_fwd needs none.
 *   q, k, v, o, lse : as attn_fwd.  workspace : caller-owned device memory of at least
 *   attn_fwd_unfused_workspace_size() bytes, 256-byte aligned, overwritten.
 * Errors: as attn_fwd, plus ATTN_ERR_WORKSPACE; B*H*N must fit an int and B*H*N^2 stay below
 * 2^40 (ATTN_ERR_INVALID_ARG).  cuBLAS is loaded at the first call; if it cannot be loaded or
 * created the call returns ATTN_ERR_LAUNCH and attn_last_error_string() says why.  Calls are
 * serialised by a lock (one cuBLAS handle per device).
 */
attn_status attn_fwd_unfused(const void *q, const void *k, const void *v, void *o, float *lse,
                             void *workspace, size_t workspace_bytes, int B, int H, int N, int d_k,
                             float scale, cudaStream_t stream);

/*
 * Element-wise fp32 addition c[i] = a[i] + b[i], 0 <= i < n: the vector_add_cuda kernel of
 * section 2 ("Practical code comparison: raw CUDA C++ vs OpenAI Triton", the raw CUDA C++
 * version: one element per index, guarded by i < n), used here as the library's HBM bandwidth
 * probe (16-byte vector accesses, grid-stride over whole waves of the SMs).
 *   a, b : n fp32 device inputs;  c : n fp32 device output (may be a or b itself; no other
 *   overlap).  All 16-byte aligned.  n = 0 is a no-op; n < 0 is ATTN_ERR_INVALID_ARG.
 * Each c[i] is the correctly rounded fp32 sum, bit for bit what one fp32 addition gives.
 */
attn_status vector_add(const float *a, const float *b, float *c, long long n, cudaStream_t stream);

/*
 * attn_bwd_noalloc: the backward pass without any workspace argument, for callers that cannot
 * allocate device memory at the point where they run the backward: code that must not call
 * cudaMalloc (or an allocator built on it) there, for example because it runs under a memory
 * budget fixed up front or inside a framework that owns all device allocations.  The article
 * has no counterpart; this is a convenience of this library.
 *
 * Arguments and results are those of attn_bwd() without `workspace` / `workspace_bytes`.  The
 * scratch attn_bwd keeps in the workspace (attn_bwd_workspace_size(B,H,N,d_k) bytes) comes
 * instead from one array of 64 MiB compiled into the library; every GPU that loads the library
 * holds it until the process exits.  Sizes whose scratch exceeds 64 MiB are refused with
 * ATTN_ERR_TOO_LARGE before anything is launched.  The call allocates no device memory.
 *
 * The first call on a device looks up the array's device address (cudaGetSymbolAddress) and
 * caches it; make that first call before any stream capture.  All calls share the one array:
 * calls whose work can overlap on the GPU (different streams, or different host threads without
 * ordering) race on it and produce wrong gradients; order them on one stream.  Each call
 * rewrites everything it reads from the array, so earlier contents do not matter.
 */
attn_status attn_bwd_noalloc(const void *q, const void *k, const void *v, const void *o,
                             const void *dout, const float *lse, void *dq, void *dk, void *dv,
                             int B, int H, int N, int d_k, float scale, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_GB300_H */
