/*
 * kda_layer.h -- the operators of libkda that stand around and beside the KDA
 * recurrence in a model's layers:
 *
 *   kda_rmsnorm_*  RMS normalisation with the residual's addition, with a bf16
 *                  output or an 8-bit (e4m3) output with scales, and its gradient;
 *   kda_conv_*     the short causal depthwise convolution ahead of a recurrence
 *                  (prompts, one token per sequence, gradient);
 *   kda_ssm_*      the selective state-space scan (prompts, one token per
 *                  sequence, gradient).
 *
 * The conventions are those of kda.h: device pointers on the current HIP
 * device, work enqueued on `stream` without synchronising, status codes
 * returned before anything is enqueued, caller-owned workspaces (or, when NULL,
 * one taken and released with hipMallocAsync / hipFreeAsync on the stream), no
 * global mutable state, packed batches described by a device int64 cu_seqlens.
 *
 * Strides.  Activations are read with strides, in elements: the last dimensions
 * (stated at each call) are contiguous, tokens are `*_stride_t` apart and batch
 * rows `*_stride_b` apart, so that slices of a wider projection need no copy.
 * Inputs may overlap or be broadcast (stride 0).  Every tensor that a call
 * writes is contiguous and lies apart from everything else that the call
 * touches (KDA_ERR_OVERLAP), but for the pairs that may be one tensor, as
 * stated at the calls.  The norm and the convolution take any stride and any
 * address that is a multiple of the type's size; the scan reads x, B, C and d_out
 * 16 bytes at a time, at addresses that are multiples of 16 bytes, with strides that
 * are multiples of 8 elements (KDA_ERR_ALIGN otherwise), and its other tensors of
 * more than one dimension, dt and ddt aside, begin at such addresses too.  Strides of
 * more than 2^40 elements, more than 2^40 rows or tokens, more than 2^22 columns or
 * channels, and scans of more than 2^31 - 128 tokens, 65535 heads or 2^31 - 1
 * sequences, pieces or chunks are refused (KDA_ERR_SHAPE).
 *
 * Packed batches.  With cu_seqlens (int64 [num_seqs + 1], cu[0] = 0, never
 * falling, cu[num_seqs] <= T), B is 1 and sequence n holds the tokens
 * cu[n] .. cu[n + 1] - 1.  Sequences may be empty (their final state is their
 * initial state).  Rows from cu[num_seqs] on belong to no sequence: no call
 * reads them into a result, and the rows of an output there are left as they
 * were.  The contents are clamped to 0 .. T on the device, so that wrong ones
 * give wrong results but no access outside the tensors; KDA_VALIDATE=1 in the
 * environment checks them on the host as kda_fwd does (except that
 * cu[num_seqs] < T is allowed).
 */
#ifndef KDA_LAYER_H_
#define KDA_LAYER_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- RMS normalisation ------------------------------------------------------
 * For every row r of D values, in fp32:
 *   h = x + residual (h = x without residual),   n = h / sqrt(mean(h^2) + eps),
 *   y = n * weight;
 * y is rounded once, from fp32, to the output's type.  residual_out takes h,
 * rounded to the residual's type. */
typedef struct {
    int64_t rows, D;
    int64_t x_stride, residual_stride;      /* elements between rows (>= 0) */
    int32_t residual_dtype, weight_dtype;   /* kda_dtype_t; residual_dtype also of residual_out (and, in the
                                               gradient, of h and d_residual_out) */
    float eps;                              /* finite, >= 2^-126 */
    int64_t group;                          /* quantised output: columns per scale (128), or 0: one scale per row */
    int64_t d_out_stride, d_residual_stride;/* the gradient's inputs */
    void *workspace;                        /* gradient only: >= kda_rmsnorm_bwd_workspace_size(), 256-byte aligned */
    size_t workspace_bytes;
} kda_rmsnorm_desc_t;

/* x: bf16 [rows, D]; residual: [rows, D] of residual_dtype, or NULL; weight: [D];
 * residual_out: [rows, D] or NULL (NULL without residual), it may be `residual`
 * itself when that is contiguous; out: bf16 [rows, D], it may be `x` likewise. */
kda_status_t kda_rmsnorm_fwd(const void *x, const void *residual, const void *weight, void *residual_out,
                             void *out, const kda_rmsnorm_desc_t *desc, hipStream_t stream);

/* The same with an 8-bit output: out_q, e4m3 (OCP, largest finite value 448)
 * [rows, D], and scales, fp32 [rows, ceil(D / group)] ([rows, 1] with group 0):
 * the value an entry stands for is out_q * scale, with
 *   scale = max(max |y| over the group / 448, 2^-126)
 * taken from the unrounded y.  A NaN in a group makes its scale and its entries
 * NaN. */
kda_status_t kda_rmsnorm_quant(const void *x, const void *residual, const void *weight, void *residual_out,
                               void *out_q, float *scales, const kda_rmsnorm_desc_t *desc, hipStream_t stream);

/* The gradient of <d_out, y> + <d_residual_out, h>: with h (what residual_out
 * took, or x where there was no residual; its stride is x_stride, its type
 * residual_dtype), n = h rstd and d_out bf16,
 *   dh = rstd (weight d_out - n mean(weight d_out n)) + d_residual_out,
 *   dweight = sum over rows of d_out n.
 * d_residual_out: of residual_dtype, or NULL for zeros.  dx: bf16 [rows, D],
 * the gradient of x (and of a bf16 residual).  dresidual: fp32 [rows, D], the
 * unrounded gradient for an fp32 residual, or NULL.  dweight: fp32 [D]. */
kda_status_t kda_rmsnorm_bwd(const void *h, const void *weight, const void *d_out, const void *d_residual_out,
                             void *dx, float *dresidual, float *dweight, const kda_rmsnorm_desc_t *desc,
                             hipStream_t stream);
/* Bytes of workspace kda_rmsnorm_bwd needs (0 if the shapes are invalid). */
size_t kda_rmsnorm_bwd_workspace_size(const kda_rmsnorm_desc_t *desc);

/* ---- short causal convolution --------------------------------------------------
 * For every sequence and channel d, with the W - 1 inputs before its first
 * token taken from the initial state (or zero):
 *   pre_t = bias + sum_k weight[d, k] x_{t - (W - 1) + k},
 *   out_t = pre_t, or with silu: pre_t / (1 + exp(-pre_t)).
 * The state of a sequence is its last W - 1 inputs, oldest first: [num_seqs,
 * W - 1, D]. */
typedef struct {
    int64_t B, T, D, W;                     /* W is 2, 3 or 4 */
    int64_t num_seqs;                       /* B, or the packed batch's sequences */
    int64_t x_stride_b, x_stride_t;         /* x [B, T, D] */
    int64_t d_out_stride_b, d_out_stride_t; /* gradient only: d_out [B, T, D] */
    int32_t silu;                           /* 0 or 1 */
    int32_t weight_dtype;                   /* of weight and bias */
    int32_t initial_state_dtype, final_state_dtype;
    void *workspace;                        /* gradient only */
    size_t workspace_bytes;
} kda_conv_desc_t;

/* x: bf16; weight: [D, W]; bias: [D] or NULL; initial_state, final_state: or
 * NULL, final_state may be initial_state when the types match; out: bf16
 * [B, T, D], not x. */
kda_status_t kda_conv_fwd(const void *x, const void *weight, const void *bias, const void *initial_state,
                          void *final_state, const int64_t *cu_seqlens, void *out, const kda_conv_desc_t *desc,
                          hipStream_t stream);
/* One token per sequence (T = 1, num_seqs = B): the same in one launch, with
 * final_state required.  It may be initial_state. */
kda_status_t kda_conv_decode(const void *x, const void *weight, const void *bias, const void *initial_state,
                             void *final_state, void *out, const kda_conv_desc_t *desc, hipStream_t stream);
/* The gradient of <d_out, out> + <d_final_state, final_state>.  d_out: bf16;
 * d_final_state: of final_state_dtype, or NULL for zeros; dx: bf16 [B, T, D];
 * dweight: fp32 [D, W]; dbias: fp32 [D] or NULL; d_initial_state: fp32
 * [num_seqs, W - 1, D] or NULL. */
kda_status_t kda_conv_bwd(const void *x, const void *weight, const void *bias, const void *initial_state,
                          const int64_t *cu_seqlens, const void *d_out, const void *d_final_state, void *dx,
                          float *dweight, float *dbias, float *d_initial_state, const kda_conv_desc_t *desc,
                          hipStream_t stream);
/* Bytes of workspace kda_conv_bwd needs (0 if the shapes are invalid). */
size_t kda_conv_bwd_workspace_size(const kda_conv_desc_t *desc);

/* ---- selective state-space scan --------------------------------------------------
 * For every sequence and head h (with the G groups of B and C shared by H / G
 * consecutive heads each), with a P x N fp32 state S:
 *   dt_t = softplus(dt_t + dt_bias[h]),   a_t = -exp(A_log[h]) dt_t,
 *   S_t = exp(a_t) S_{t-1} + dt_t x_t B_t^T,
 *   y_t = S_t C_t + D[h] x_t. */
typedef struct {
    int64_t B, T, H, P, G, N;               /* P and N are 64 or 128; H is a multiple of G */
    int64_t num_seqs;
    int64_t x_stride_b, x_stride_t;         /* x [B, T, H, P]; token strides are below 2^24 here */
    int64_t dt_stride_b, dt_stride_t;       /* dt [B, T, H] */
    int64_t b_stride_b, b_stride_t;         /* B [B, T, G, N] */
    int64_t c_stride_b, c_stride_t;         /* C [B, T, G, N] */
    int64_t d_out_stride_b, d_out_stride_t; /* gradient only: d_out [B, T, H, P] */
    int32_t initial_state_dtype, final_state_dtype;
    void *workspace;
    size_t workspace_bytes;
    /* 64-token chunks per piece of a state chain: 0 for the library's rule
     * (kda_ssm_piece_chunks), n > 0 for n (at most n in a packed batch, whose
     * sequences are cut evenly).  A piece is what one workgroup walks
     * through in order; shorter pieces make more of them, and where a sequence
     * has several, its tokens are read twice (once for the pieces' states). */
    int64_t piece_chunks;
    int64_t launch_piece;                   /* most workgroups of one launch, rounded up to a multiple of 8; 0: the
                                               library's (2^23, so that only very large batches take several) */
} kda_ssm_desc_t;

/* Bytes of workspace kda_ssm_fwd and kda_ssm_bwd need for these shapes (0 if they
 * are invalid; with B = 1 enough for a packed batch too), and the chunks per piece
 * they use (at most, in a packed batch of several sequences; -1 if the shapes are
 * invalid).  Host arithmetic. */
size_t kda_ssm_fwd_workspace_size(const kda_ssm_desc_t *desc);
size_t kda_ssm_bwd_workspace_size(const kda_ssm_desc_t *desc);
int64_t kda_ssm_piece_chunks(const kda_ssm_desc_t *desc);

/* x, dt, B, C: bf16; A_log: fp32 [H]; dt_bias: fp32 [H] or NULL (zeros); D: fp32
 * [H] or NULL (no skip term); initial_state, final_state: [num_seqs, H, P, N] or
 * NULL, final_state may be initial_state when the types match; out: bf16
 * [B, T, H, P].  A NaN or infinity in a token reaches its sequence's outputs from
 * that token on, and no other sequence. */
kda_status_t kda_ssm_fwd(const void *x, const void *dt, const void *Bm, const void *Cm, const float *A_log,
                         const float *dt_bias, const float *D, const void *initial_state, void *final_state,
                         const int64_t *cu_seqlens, void *out, const kda_ssm_desc_t *desc, hipStream_t stream);
/* One token per sequence (T = 1, num_seqs = B), in one launch and without a
 * workspace; final_state (required) may be initial_state. */
kda_status_t kda_ssm_decode(const void *x, const void *dt, const void *Bm, const void *Cm, const float *A_log,
                            const float *dt_bias, const float *D, const void *initial_state, void *final_state,
                            void *out, const kda_ssm_desc_t *desc, hipStream_t stream);
/* The gradient of <d_out, out> + <d_final_state, final_state>.  d_out: bf16;
 * d_final_state: of final_state_dtype, or NULL for zeros.  dx [B, T, H, P], ddt
 * [B, T, H], dB and dC [B, T, G, N]: bf16; dA_log, ddt_bias, dD: fp32 [H]
 * (ddt_bias and dD may be NULL); d_initial_state: fp32 [num_seqs, H, P, N] or
 * NULL.  The forward's states are computed again, and the state entering every
 * chunk and the gradient of the one leaving it are held in the workspace (2 x 4 P N
 * bytes per chunk and head).  A NaN or infinity in a token reaches all gradients of
 * its 64-token chunk, those of its sequence that depend on the chunk's and the
 * parameters'. */
kda_status_t kda_ssm_bwd(const void *x, const void *dt, const void *Bm, const void *Cm, const float *A_log,
                         const float *dt_bias, const float *D, const void *initial_state,
                         const int64_t *cu_seqlens, const void *d_out, const void *d_final_state, void *dx,
                         void *ddt, void *dB, void *dC, float *dA_log, float *ddt_bias, float *dD,
                         float *d_initial_state, const kda_ssm_desc_t *desc, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* KDA_LAYER_H_ */
