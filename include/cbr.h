/*
 * cbr.h -- C ABI of libcbr.so: the fused Conv2D -> BatchNorm -> ReLU (CBR) operator
 * on AMD Instinct MI355X (gfx950), training forward, folded-BN inference and backward.
 *
 * Pages the operations follow (cited by title and section):
 *   [CBR]  Tech-Renaissance blog, "(20) CBR fused operator: Conv + BatchNorm + ReLU"
 *   [BN]   "CUDA implementation of batch normalization (BatchNorm)" (dpshk.com)
 *   [TL]   "TileLang operator-fusion case: Conv2D+ReLU"
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Layouts ([CBR] section 8): activations NHWC, filters KRSC (K = output channels),
 * conv outputs N x P x Q x K, all dense.  P = (H + 2*pad_h - R)/stride_h + 1 and
 * Q = (W + 2*pad_w - S)/stride_w + 1 (floor); the convolution is a cross-correlation
 * with zero padding, dilation 1, one group.  M = N*P*Q is the number of output pixels.
 *
 * Types: tensors marked bf16 are bfloat16 bit patterns (uint16_t); statistics,
 * gamma/beta, the weight gradient and conv bias are float32.
 *
 * Pointers: every tensor pointer is a DEVICE pointer, 16-byte aligned, owned by the
 * caller; no call allocates or frees device memory.  The library keeps two things per
 * device for the life of the process: the scratch array of cbr_forward_train_noalloc
 * (module memory, loaded with the library) and, once cbr_backward has run with a dx
 * there, a second stream with three events (created on that first call).  The cbr_shape
 * pointer is a host pointer read during the call only.  `workspace` is caller-owned
 * device scratch of at least cbr_workspace_bytes(shape, op) bytes (256-byte aligned);
 * its contents are undefined between calls and it must not be shared by calls that
 * may run concurrently.  `stream` is a hipStream_t (NULL = the null stream).
 *
 * Execution: each call validates its arguments on the host, then enqueues its
 * kernels on `stream` and returns without synchronising.  Faults during kernel
 * execution surface at the caller's next synchronisation, as HIP reports them.
 * Results are bitwise reproducible run to run (no floating-point atomics).
 *
 * Errors: a non-zero return means nothing was enqueued and no output was written,
 * except CBR_E_HIP, which reports a failed launch (outputs then undefined).  No call
 * aborts or exits the process.
 *
 * Limits (CBR_E_UNSUPPORTED): K % 8 != 0 ([CBR] section 8: output channels a multiple
 * of 8); K > 2048; any tensor with 2^30 elements or more; pad >= filter size;
 * dx requested with a stride other than 1.
 */
#ifndef CBR_H
#define CBR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct cbr_shape {
    int32_t n, h, w, c;                     /* input, NHWC                         */
    int32_t k, r, s;                        /* filter, KRSC (k = output channels)  */
    int32_t stride_h, stride_w, pad_h, pad_w;
} cbr_shape;

enum cbr_status {
    CBR_OK = 0,
    CBR_E_NULL = 1,         /* a required pointer is NULL                            */
    CBR_E_SHAPE = 2,        /* non-positive size, stride < 1, negative pad, empty out,
                               or M < 2 in training (no batch variance from one value) */
    CBR_E_UNSUPPORTED = 3,  /* valid but outside the limits listed above             */
    CBR_E_ALIGN = 4,        /* a tensor pointer is not 16-byte aligned               */
    CBR_E_WORKSPACE = 5,    /* workspace NULL or smaller than cbr_workspace_bytes    */
    CBR_E_HIP = 6,          /* a kernel launch failed                                */
    CBR_E_VALUE = 7         /* eps < 0, momentum outside [0,1], or not finite; an unknown
                               type or kind, or an argument that does not fit the others */
};

enum cbr_op { CBR_OP_TRAIN = 0, CBR_OP_INFER = 1, CBR_OP_BWD = 2 };

/* Human-readable name of a status code (static string, never NULL). */
const char *cbr_status_str(int status);

/* Checks the shape alone; writes P and Q when they are non-NULL.  Returns a status. */
int cbr_output_hw(const cbr_shape *shape, int32_t *p, int32_t *q);

/* Number of uint32 words of the packed ReLU mask: ceil(M*K / 32). */
size_t cbr_mask_words(const cbr_shape *shape);

/* Workspace bytes that op (enum cbr_op) needs for this shape; 0 for an invalid shape.
 * For CBR_OP_BWD the figure includes room for dz, used when the caller passes dz = NULL. */
size_t cbr_workspace_bytes(const cbr_shape *shape, int op);

/*
 * Training-mode forward ([CBR] sections 2 and 4.1-4.3; [BN] 2.1, 2.4):
 *   z        = conv(x, w)                                   bf16 [N,P,Q,K]  (out)
 *   mean_k   = (1/M) sum z,  var_k = (1/M) sum (z - mean_k)^2   (biased; from the
 *              fp32 accumulators, before z is rounded to bf16)
 *   invstd_k = 1/sqrt(var_k + eps)
 *   u        = gamma_k * (z - mean_k) * invstd_k + beta_k  (computed from stored z)
 *   y        = max(u, 0)                                    bf16 [N,P,Q,K]  (out)
 *   relu_mask: bit (i % 32) of word (i / 32) is (u_i > 0) for the NHWC linear index i
 *              of y; cbr_mask_words() words, bits past M*K are zero        (out)
 *   saved_mean = mean, saved_invstd = invstd                   float [K]   (out)
 *   run_mean_out = (1-momentum)*run_mean_in + momentum*mean    float [K]   (out)
 *   run_var_out  = (1-momentum)*run_var_in  + momentum*var     float [K]   (out)
 * x: bf16 NHWC [N,H,W,C]; w: bf16 KRSC [K,R,S,C]; gamma, beta, run_*_in: float [K].
 * Needs M >= 2 (CBR_E_SHAPE otherwise).  u normalises the stored bf16 z with statistics
 * of the unrounded values, so a channel whose batch variance is below the bf16 rounding
 * error of its values (var << (2^-8 |z|)^2, e.g. a constant non-zero channel) gets u
 * dominated by that rounding error.
 * run_mean_out/run_var_out may alias run_mean_in/run_var_in (in-place update); no other
 * output may alias an input.  There is no conv bias: batch normalisation cancels it.
 */
int cbr_forward_train(const cbr_shape *shape,
                      const uint16_t *x, const uint16_t *w,
                      const float *gamma, const float *beta,
                      const float *run_mean_in, const float *run_var_in,
                      float eps, float momentum,
                      uint16_t *z, uint16_t *y, uint32_t *relu_mask,
                      float *saved_mean, float *saved_invstd,
                      float *run_mean_out, float *run_var_out,
                      void *workspace, size_t ws_bytes, void *stream);

/*
 * Folded-BN inference forward ([CBR] sections 2 and 6; [BN] 4.4; [TL] fused ReLU
 * epilogue):
 *   s_k      = gamma_k / sqrt(run_var_k + eps)
 *   w_fold   = w * s_k (per output channel, rounded to bf16),
 *   b_fold_k = (b_k - run_mean_k) * s_k + beta_k   (float)
 *   y        = max(conv(x, w_fold) + b_fold, 0)                   bf16 [N,P,Q,K] (out)
 * conv_bias may be NULL (read as zero).  All other pointers as in training.
 */
int cbr_forward_infer(const cbr_shape *shape,
                      const uint16_t *x, const uint16_t *w, const float *conv_bias,
                      const float *gamma, const float *beta,
                      const float *run_mean, const float *run_var, float eps,
                      uint16_t *y, void *workspace, size_t ws_bytes, void *stream);

/*
 * Backward of the training forward ([CBR] section 5; [BN] 3.1-3.3):
 *   g      = dy * mask                      (never written to memory)
 *   xhat   = (z - saved_mean) * saved_invstd (recomputed from the stored bf16 z)
 *   dbeta  = sum_m g,  dgamma = sum_m g * xhat                       float [K] (out)
 *   dz     = gamma * saved_invstd * (g - dbeta/M - xhat * dgamma/M)  bf16 [N,P,Q,K]
 *   dw[k,r,s,c] = sum_{n,p,q} dz[n,p,q,k] * x[n, p*sh-ph+r, q*sw-pw+s, c]  float KRSC
 *   dx[n,h,v,c] = sum_{k,r,s} dz[n,p,q,k] * w[k,r,s,c] over the (p,q) that read
 *                 x[n,h,v] through tap (r,s)                           bf16 NHWC
 *   dw and dx are computed from the bf16 dz above (as the CBR page's WGrad and DGrad
 *   read dL/d(conv_out) from a half-precision buffer), accumulated in fp32.
 * Needs M >= 2 (CBR_E_SHAPE otherwise).
 * Inputs: x, w, z (bf16), relu_mask, dy (bf16 [N,P,Q,K]), gamma, saved_mean,
 * saved_invstd (float [K]) -- the training forward's inputs and outputs.
 * dz may be NULL (then it lives in the workspace).  dx may be NULL: the first-layer
 * form of [CBR] 5.3, which skips the data gradient.  dx may alias x: the weight
 * gradient finishes reading x before the data gradient writes dx ([CBR] 5.2).
 * A non-NULL dx needs stride 1 in both directions.
 * With a dx, the data gradient's filter flip (it reads only w) runs on a second stream
 * that the library keeps per device, beside the BN backward; when dx does not overlap x
 * the weight gradient may run there too (see CBR_STAGE_BWD).  Both are forked from and
 * joined back to `stream` with events: the call's work is still complete when `stream`
 * reaches its end.  Calls on one device from several host threads serialise their
 * enqueueing around that stream.
 */
int cbr_backward(const cbr_shape *shape,
                 const uint16_t *x, const uint16_t *w, const uint16_t *z,
                 const uint32_t *relu_mask, const uint16_t *dy,
                 const float *gamma, const float *saved_mean, const float *saved_invstd,
                 uint16_t *dz, float *dgamma, float *dbeta, float *dw, uint16_t *dx,
                 void *workspace, size_t ws_bytes, void *stream);

/*
 * The training forward for callers that cannot allocate device memory: code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc.  Same arguments
 * and results as cbr_forward_train without the workspace: the kernels' scratch is a
 * CBR_NOALLOC_SCRATCH_BYTES array that the library holds on each device from the first
 * call made with that device current until the process ends (its address is looked up
 * then, with hipGetSymbolAddress).  The call itself allocates nothing.
 * Limit: shapes whose cbr_workspace_bytes(shape, CBR_OP_TRAIN) exceeds
 * CBR_NOALLOC_SCRATCH_BYTES return CBR_E_WORKSPACE (the 256 x 56 x 56 x 64 workload needs
 * about 133 KB, the 224 x 224 first layer at N = 64 also about 133 KB).
 * All calls on one device share that device's array: calls that may overlap on one
 * device (different streams, different host threads) race, and must be serialised by
 * the caller.  A call leaves the array's contents undefined; no call depends on them.
 */
#define CBR_NOALLOC_SCRATCH_BYTES (4u << 20)

int cbr_forward_train_noalloc(const cbr_shape *shape,
                              const uint16_t *x, const uint16_t *w,
                              const float *gamma, const float *beta,
                              const float *run_mean_in, const float *run_var_in,
                              float eps, float momentum,
                              uint16_t *z, uint16_t *y, uint32_t *relu_mask,
                              float *saved_mean, float *saved_invstd,
                              float *run_mean_out, float *run_var_out, void *stream);

/*
 * Conv2D + bias + ReLU without batch normalisation ([TL] "fused ReLU" section: the ReLU
 * applied in the convolution's epilogue, before the result leaves the chip):
 *   y = max(conv(x, w) + bias, 0)                                  bf16 [N,P,Q,K] (out)
 * x: bf16 NHWC [N,H,W,C]; w: bf16 KRSC [K,R,S,C]; bias: float [K], may be NULL (read as
 * zero).  No workspace.  Shape limits and errors as for the other calls.
 */
int cbr_conv2d_bias_relu(const cbr_shape *shape, const uint16_t *x, const uint16_t *w, const float *bias,
                         uint16_t *y, void *stream);

/*
 * Conv2D + bias without activation ([TL] basic convolution with a bias epilogue; the
 * convolution of [CBR] section 2, y = conv(x, W, b)):
 *   y = conv(x, w) + bias                                          bf16 [N,P,Q,K] (out)
 * Arguments as for cbr_conv2d_bias_relu.
 */
int cbr_conv2d_bias(const cbr_shape *shape, const uint16_t *x, const uint16_t *w, const float *bias,
                    uint16_t *y, void *stream);

/*
 * Norms before and after a block, with its gate and residual scale
 * ----------------------------------------------------------------
 * A block (convolutions, a product, ...) maps activations to a branch f; the residual
 * stream x takes it in.  Rows are pixels (or tokens): rows x channels, dense, NHWC order,
 * so N*H*W rows.  Row m belongs to gate row i = m / rows_per_gate (H*W: a gate an image;
 * 1: a gate of its own for every row).  One pass over x and f computes
 *   n    = post(f)                       norm after the block, per row, or f itself
 *   y    = x + alpha * r_c * g_ic * n    gated and scaled residual add      stream (out)
 *   h    = pre(y)                        norm before the next block, per row  branch (out)
 * with the norms
 *   CBR_NORM_LAYER: (v - mean) / sqrt(var + eps) * w + b   (var biased, over the channels)
 *   CBR_NORM_RMS:    v / sqrt(mean of v^2 + eps) * w + b
 *   CBR_NORM_NONE:  n = f;  as `pre`: there is no h.
 * Everything is computed in fp32 and rounded once per output; h uses y before its rounding.
 * Types: x, y, dx, dy have stream_type; f, h, gate and their gradients branch_type; both
 * are CBR_BF16, CBR_F16 or CBR_F32, and they are equal or stream_type is CBR_F32.
 * w, b, r, their gradients and the statistics are float.
 *
 * Limits: rows < 2^31, channels <= 8192 (any, odd ones too), rows a multiple of
 * rows_per_gate.  channels % 8 == 0 takes 16-byte accesses.  Rows and channels must be
 * positive (CBR_E_SHAPE).
 */
enum cbr_dtype { CBR_BF16 = 0, CBR_F16 = 1, CBR_F32 = 2, CBR_E4M3 = 3, CBR_E5M2 = 4 };
enum cbr_norm { CBR_NORM_NONE = 0, CBR_NORM_RMS = 1, CBR_NORM_LAYER = 2 };

typedef struct cbr_block_shape {
    int64_t rows;
    int64_t rows_per_gate;          /* read only where a gate is given                */
    int32_t channels;
    int32_t post, pre;              /* enum cbr_norm                                  */
    int32_t stream_type, branch_type;   /* enum cbr_dtype                             */
    float alpha;                    /* constant factor of the branch (1: none)        */
    float eps_post, eps_pre;
} cbr_block_shape;

/* Workspace bytes of cbr_block_norm_backward, never 0 for a valid shape; 0 for an invalid
 * one.  The forward needs none.  Calls under way at the same time need one each. */
size_t cbr_block_norm_workspace_bytes(const cbr_block_shape *shape);

/*
 * Forward.  f may be NULL: then post is CBR_NORM_NONE, gate, res_scale and y are NULL and
 * h = pre(x) (a first block's norm).  pre CBR_NORM_NONE: pre_w, pre_b, h and pre_stats are
 * NULL (a last block's residual add).  post_w, post_b, pre_w, pre_b [channels], gate
 * [rows / rows_per_gate][channels] and res_scale [channels] may each be NULL (1, or 0 for
 * the biases); weights without their norm are refused (CBR_E_VALUE), as is a call with
 * neither f nor pre.  post_stats, pre_stats: float [rows][2], (mean, 1/std) of each row
 * (mean 0 for RMS), for the backward; NULL skips them (inference).
 * y may alias x and h may alias f (same type and place); no other output may alias an input.
 */
int cbr_block_norm_forward(const cbr_block_shape *shape, const void *x, const void *f,
                           const float *post_w, const float *post_b, const void *gate,
                           const float *res_scale, const float *pre_w, const float *pre_b,
                           void *y, void *h, float *post_stats, float *pre_stats, void *stream);

/*
 * Backward.  dy: gradient to y from everything after it but h (NULL: zero; with pre
 * CBR_NORM_NONE it is needed); dh: gradient to h.  With vhat the normalised values,
 *   D  = dy + (pre norm's backward of dh at y):  dx = D                    stream (out)
 *   dg_ic = alpha r_c sum_{rows of i} D n,   dr_c = alpha sum D g n
 *   df = post norm's backward of alpha r g D,                               branch (out)
 *   dpost_w = sum alpha r g D nhat,  dpost_b = sum alpha r g D,
 *   dpre_w = sum dh yhat,            dpre_b = sum dh
 * y, f, post_stats, pre_stats as the forward left them (y: x where f is NULL; y and
 * pre_stats are read only for a pre norm, post_stats only for a post norm).  Without f
 * the branch outputs are NULL and dx is the gradient to x.
 * dpost_w, dpost_b, dgate, dres_scale, dpre_w, dpre_b may each be NULL (not wanted); a
 * gradient of something that has no value here is refused (CBR_E_VALUE), but dpost_b and
 * dpre_b need no bias, dpost_w and dpre_w no weight and dres_scale no res_scale: where the
 * forward read 1 or 0 the gradient exists all the same.
 * The sums over rows run in a fixed order: fp32 over a workgroup's rows, then fp64.
 * dx may alias dy and df may alias f or dh (same type and place); no other output may alias
 * an input.
 */
int cbr_block_norm_backward(const cbr_block_shape *shape, const void *dy, const void *dh,
                            const void *y, const void *f,
                            const float *post_w, const float *post_b, const void *gate,
                            const float *res_scale, const float *pre_w,
                            const float *post_stats, const float *pre_stats,
                            void *dx, void *df, float *dpost_w, float *dpost_b, void *dgate,
                            float *dres_scale, float *dpre_w, float *dpre_b,
                            void *workspace, size_t ws_bytes, void *stream);

/*
 * 8-bit floating point: operands with a scale for each block of 128
 * ------------------------------------------------------------------
 * src [rows][cols], dense, of CBR_BF16, CBR_F16 or CBR_F32; v is src, or its transpose
 * where `transpose` is non-zero, with v_rows rows of v_cols values.  v is written in
 * q_type (CBR_E4M3: finite values up to 448; CBR_E5M2: up to 57344) with one scale for
 * each group of `block` rows by 128 columns of v (block 1 or 128), groups at the edges
 * being smaller:
 *   a = max(largest |v| of the group, fmax * 2^-126),  scale = a / fmax,
 *   q = v * fmax / a, rounded to nearest, ties to even: v = q * scale up to rounding.
 * q [v_rows][ldq] bytes, ldq >= v_cols a multiple of 16; bytes past v_cols of a row are
 * left as they are.  scale: float [ceil(v_cols / 128)][ceil(v_rows / block)], the blocks
 * of 128 columns outermost.  A NaN becomes NaN and does not touch the rest of its group;
 * an infinity makes its group's scale infinite, and the group stands for NaN.
 * rows and cols positive, < 2^31, and ceil(rows / 64) * ceil(cols / 128) < 2^24
 * (CBR_E_UNSUPPORTED beyond that).  q and scale may not overlap src or each other.
 */
typedef struct cbr_quant_shape {
    int64_t rows, cols;             /* of src                                         */
    int64_t ldq;                    /* bytes from a row of q to the next              */
    int32_t src_type, q_type;       /* enum cbr_dtype                                 */
    int32_t transpose, block;
} cbr_quant_shape;

int cbr_fp8_quantize(const cbr_quant_shape *shape, const void *src, void *q, float *scale, void *stream);

/*
 * Matrix product of such operands (a 1x1 convolution's forward, data gradient or weight
 * gradient over N*H*W pixels):
 *   d[i][j] = act( sum_t a_scale[t][i] * b_scale[t][j / b_block]
 *                        * sum_{k in block t} a[i][k] * b[j][k]  + bias[j] )
 * a [m][lda], b [n][ldb] bytes in a_type, b_type (CBR_E4M3 or CBR_E5M2), row strides
 * multiples of 16 and at least k; what lies past k in a row is not used.  a_scale
 * [ceil(k/128)][m] (block 1), b_scale [ceil(k/128)][ceil(n / b_block)], b_block 1 or 128.
 * d [m][n] dense, d_type CBR_BF16, CBR_F16 or CBR_F32; bias float [n] or NULL; act is
 * max(v, 0) where relu is non-zero (a NaN stays one), else v.  Scales may have any size: a
 * sum is not lost where a_scale * b_scale, or the sum times one of them, leaves fp32 and the
 * result does not.  All sums are fp32, and the
 * result is rounded once, unless short_sums is non-zero: then each eight consecutive products
 * (k = 8i .. 8i + 7) may be summed with 13 bits below the leading one of the largest, by the
 * 8-bit matrix instruction at twice the rate, and everything beyond the eight in fp32.  An
 * eight then loses less than 8 * 2^-13 of its largest product, however little its sum is.
 * Measured for any k: 1.4e-5 of the result's norm on normally distributed operands, 2.5e-6
 * (always towards zero) on their absolute values, 2.2e-5 with magnitudes spread over some
 * e^6.  short_sums is for 16-bit outputs (with CBR_F32: CBR_E_VALUE).
 *   forward:          a = activations [pixels][C], b = filter [K][C] with b_block 128
 *   data gradient:    a = dy [pixels][K],          b = filter transposed [C][K], b_block 128
 *   weight gradient:  a = dy transposed [K][pixels], b = activations transposed, b_block 1
 * m, n, k positive; m < 2^31, n, lda, ldb <= 2^23 and ceil(m / 64) * ceil(n / 64) <
 * 2^24 - 1 (CBR_E_UNSUPPORTED beyond that); a stride that is too small or no multiple of
 * 16 is CBR_E_SHAPE.  d and the workspace may not overlap an operand or each other.
 * The workspace (cbr_gemm_fp8_workspace_bytes, 0 where the shape needs none or is
 * invalid) holds the parts of a long sum that several workgroups share; they are added in
 * a fixed order.  Calls under way at the same time need one each.
 */
typedef struct cbr_gemm_shape {
    int64_t m;
    int64_t n, k;
    int64_t lda, ldb;               /* bytes from a row to the next                   */
    int32_t a_type, b_type, d_type; /* enum cbr_dtype                                 */
    int32_t b_block;                /* 1 or 128                                       */
    int32_t relu;
    int32_t short_sums;             /* 0: fp32 sums                                   */
} cbr_gemm_shape;

size_t cbr_gemm_fp8_workspace_bytes(const cbr_gemm_shape *shape);

int cbr_gemm_fp8(const cbr_gemm_shape *shape, const void *a, const float *a_scale, const void *b,
                 const float *b_scale, const float *bias, void *d,
                 void *workspace, size_t ws_bytes, void *stream);

/*
 * Group norm with an activation
 * -----------------------------
 * For maps that a convolution or a product left, where batches are too small for batch
 * statistics: x [images][pixels][channels], dense (NHWC: pixels = H*W).  The channels are
 * `groups` groups of channels / groups neighbouring ones; of each image's group
 *   mean = mean of x, var = mean of (x - mean)^2 over pixels and channels (biased),
 *   xhat = (x - mean) / sqrt(var + eps),  u = xhat * w_c + b_c,  y = act(u)
 *   CBR_ACT_NONE: u;  CBR_ACT_RELU: max(u, 0), a NaN stays one;  CBR_ACT_SILU: u / (1 + e^-u).
 * SiLU: |u| up to 2^127; values of y and of the slope below 2^-119 may become 0.
 * x, y, dx, dy have `type` (CBR_BF16, CBR_F16 or CBR_F32); w, b, their gradients and the
 * statistics are float.  Everything is computed in fp32 and rounded once.
 *
 * Limits: channels a multiple of groups (CBR_E_SHAPE); channels / groups <= 8192, channels < 2^24, images and
 * pixels < 2^31, at most 2^46 values, and not so many small groups or images that a launch
 * would need 2^32 threads (CBR_E_UNSUPPORTED): 2^31 values are always fewer.
 */
enum cbr_act { CBR_ACT_NONE = 0, CBR_ACT_RELU = 1, CBR_ACT_SILU = 2 };

typedef struct cbr_group_norm_shape {
    int64_t images, pixels;
    int32_t channels, groups;
    int32_t type;                   /* enum cbr_dtype                                 */
    int32_t act;                    /* enum cbr_act                                   */
    float eps;
} cbr_group_norm_shape;

/* Workspace bytes of the forward (backward 0) or the backward (non-zero): 0 where the shape
 * needs none, or is invalid.  Calls under way at the same time need one each. */
size_t cbr_group_norm_workspace_bytes(const cbr_group_norm_shape *shape, int backward);

/*
 * Forward.  w, b [channels] may each be NULL (1, 0).  stats: float [images][groups][2], (mean,
 * 1/sqrt(var + eps)), for the backward; NULL skips them (inference).  y may be x itself (in place);
 * no other output may overlap an input.
 */
int cbr_group_norm_forward(const cbr_group_norm_shape *shape, const void *x, const float *w, const float *b,
                           void *y, float *stats, void *workspace, size_t ws_bytes, void *stream);

/*
 * Backward.  dy: gradient to y; x, w, b and stats as the forward had and left them.  With
 * g = dy * act'(u) (ReLU: 0 for u <= 0), over an image's pixels S1_c = sum g xhat, S0_c = sum g, and
 * over a group of M = pixels * channels / groups values
 *   dx = (w g - sum_c w S0 / M - xhat sum_c w S1 / M) / sqrt(var + eps),
 *   dw = sum of S1 over the images,  db = sum of S0.
 * dx, dw, db may each be NULL (not wanted), not all three.  dw needs no w, db no b.  The sums run in a fixed
 * order, in fp32; dw and db add up the parts of images, and of large images' tiles, in fp64.  dx may be dy itself,
 * or x (in place); no other output may overlap an input.
 */
int cbr_group_norm_backward(const cbr_group_norm_shape *shape, const void *dy, const void *x, const float *w,
                            const float *b, const float *stats, void *dx, float *dw, float *db,
                            void *workspace, size_t ws_bytes, void *stream);

/*
 * 4-bit floating point: operands with an exponent for each group of 32
 * ---------------------------------------------------------------------
 * src [rows][cols], dense, of CBR_BF16, CBR_F16 or CBR_F32; v is src, or its transpose
 * where `transpose` is non-zero, with v_rows rows of v_cols values.  Each group of 32
 * consecutive values of a row of v (fewer in a row's last one) has a scale, a power of two, and
 * 4-bit values (sign, two bits of exponent, one of mantissa: 0, 1/2, 1, 3/2, 2, 3, 4, 6):
 *   a = largest |v| of the group,  scale = 2^(floor(log2 a) - 2), at least 2^-127 (also a = 0),
 *   q = v / scale, rounded to nearest, ties to even (0, 1, 2, 4), above 6 to 6.
 * q [v_rows][ldq] bytes, two values a byte, the first in the lower four bits; ldq a
 * multiple of 16, at least 16 * ceil(v_cols / 32): a group takes 16 bytes, zeros behind v_cols;
 * bytes past the last group are left as they are.  scale: one byte a group, the exponent plus
 * 127, [ceil(v_cols / 128)][v_rows][4]: the four groups of 128 values together; 127 (1) where
 * there is no group.  A NaN or infinity makes its group's scale 255 (NaN) and its values 0: the
 * group stands for NaN.  rows and cols positive, < 2^31, and
 * ceil(v_rows / 16) * ceil(v_cols / 128) < 2^24 (CBR_E_UNSUPPORTED beyond that).  q and scale may
 * not overlap src or each other.
 */
typedef struct cbr_fp4_shape {
    int64_t rows, cols;             /* of src                                         */
    int64_t ldq;                    /* bytes from a row of q to the next              */
    int32_t type;                   /* of src: enum cbr_dtype                         */
    int32_t transpose;
} cbr_fp4_shape;

int cbr_fp4_quantize(const cbr_fp4_shape *shape, const void *src, void *q, void *scale, void *stream);

/* What q and scale stand for, in `type`: v [v_rows][v_cols], dense (of a transposed shape the transpose;
 * it is not turned back).  Rounded to nearest where the type does not hold a value (CBR_F16).  v may not
 * overlap q or scale. */
int cbr_fp4_dequantize(const cbr_fp4_shape *shape, const void *q, const void *scale, void *v, void *stream);

/*
 * Matrix product of such operands:
 *   d[i][j] = act( sum_t a_scale[i][t] * b_scale[j][t] * sum_{k in group t} a[i][k] * b[j][k]  + bias[j] )
 * a [m][lda], b [n][ldb] bytes and scales [ceil(k / 128)][m or n][4] as cbr_fp4_quantize leaves them: the
 * values behind k in the last group are part of the sum and have to be zeros (in one of the operands at
 * least), what lies past the groups is not used.  lda, ldb multiples of 16, at least 16 * ceil(k / 32).
 * d [m][n] dense, d_type CBR_BF16, CBR_F16 or CBR_F32; bias float [n] or NULL; act is max(v, 0) where relu
 * is non-zero (a NaN stays one), else v.  All sums are fp32: a group of 32 is exact, each one added moves the sum
 * by at most 2^-22 of the magnitudes so far, and the result is rounded once.  A scaled sum that passes fp32's
 * largest value within a group is an infinity, one below its smallest normal value may become 0.
 * Forward, data and weight gradient of a 1x1 convolution as for cbr_gemm_fp8.
 * m, n, k positive; m < 2^31, n, lda, ldb <= 2^22, k <= 2^23 and ceil(m / 64) * ceil(n / 64) <
 * 2^24 - 1 (CBR_E_UNSUPPORTED beyond that).  d and the workspace may not overlap an operand or each other.
 * The workspace (cbr_gemm_fp4_workspace_bytes, 0 where the shape needs none or is invalid) holds the parts
 * of a long sum that several workgroups share; they are added in a fixed order.  Calls under way at the
 * same time need one each.
 */
typedef struct cbr_gemm_fp4_shape {
    int64_t m;
    int64_t n, k;
    int64_t lda, ldb;               /* bytes from a row to the next                   */
    int32_t d_type;                 /* enum cbr_dtype                                 */
    int32_t relu;
} cbr_gemm_fp4_shape;

size_t cbr_gemm_fp4_workspace_bytes(const cbr_gemm_fp4_shape *shape);

int cbr_gemm_fp4(const cbr_gemm_fp4_shape *shape, const void *a, const void *a_scale, const void *b,
                 const void *b_scale, const float *bias, void *d,
                 void *workspace, size_t ws_bytes, void *stream);

/*
 * Kernel plans (tuning interface).  Each convolution stage of a call runs one kernel and
 * tile shape, its "plan", chosen per shape like the per-shape engine choice of [CBR]
 * section 7 (empirical search, winner per shape) and [TL]'s autotuned tile
 * configurations: a compiled-in table of plans measured offline (tune.py), else a
 * default rule.  Stages: CBR_STAGE_TRAIN_CONV (the conv + statistics of
 * cbr_forward_train), CBR_STAGE_INFER_CONV (the conv of cbr_forward_infer and of the
 * conv + bias calls), CBR_STAGE_DGRAD (the data gradient's conv), CBR_STAGE_WGRAD (the
 * weight gradient), CBR_STAGE_BWD (how cbr_backward schedules its gradients).  Plans:
 * 1 persistent 3x3/64-channel conv, 2 first-layer conv, 3 large-tile 224x256,
 * 4 large-tile 448x128, 5 generic 128x128, 6 generic 128x64, 7 weight gradient with
 * transposed reads, 8 generic weight gradient, 9 backward on one stream (weight gradient,
 * then data gradient), 10 backward with the weight gradient on a second stream beside the
 * data gradient ([CBR] section 5.2's WGrad stream; used only when dx does not overlap x,
 * else the call falls back to 9), 11 backward with no dz tensor: both gradients form dz
 * from dy, z and the mask while staging their operands ([CBR] section 5.1 keeps the
 * masked gradient on chip; K <= 256 and C % 8 == 0; used only when dz is NULL, else
 * the call falls back to 9), 12 weight gradient with transposed reads on 256 x 256 tiles
 * (C % 256 == 0 and K % 256 == 0).
 *
 * cbr_plan_of: the plan the stage will run for this layer shape (> 0), or minus a status.
 * cbr_plan_eligible: 1 if the plan can run the stage for this shape, 0 if not, or minus
 *   a status for an invalid shape or stage.
 * cbr_plan_name: a static name of a plan id.
 * cbr_set_plan_override: makes the stage run `plan` wherever it is eligible (plan 0
 *   clears it); process-wide, for the tuner and tests only.  cbr_workspace_bytes follows
 *   the override, so query it after setting one.  CBR_E_VALUE for a bad stage or plan.
 */
enum cbr_stage { CBR_STAGE_TRAIN_CONV = 0, CBR_STAGE_INFER_CONV = 1, CBR_STAGE_DGRAD = 2, CBR_STAGE_WGRAD = 3,
                 CBR_STAGE_BWD = 4 };

int cbr_plan_of(const cbr_shape *shape, int stage);
int cbr_plan_eligible(const cbr_shape *shape, int stage, int plan);
const char *cbr_plan_name(int plan);
int cbr_set_plan_override(int stage, int plan);

/*
 * Timed variants for profiling: identical to the calls above, and in addition record
 * caller-created hipEvent_t handles (passed as void*) at the start of the first kernel
 * and the end of the last kernel of each stage (taken from the kernels' own dispatch
 * timestamps, so no marker packets are added to the stream).  `events` may be NULL
 * (then the call is exactly the untimed one).  Event pairs (start, end):
 *   train:  [0,1] convolution + channel sums, [2,3] statistics finalize,
 *           [4,5] normalise + ReLU + mask                                  (6 events)
 *   infer:  [0,1] fold, [2,3] convolution + bias + ReLU                     (4 events)
 *   bwd:    [0,1] BN backward (reduce, finalize, dz), [2,3] weight gradient,
 *           [4,5] data gradient (recorded back to back when dx is NULL)    (6 events)
 *   conv2d_bias(_relu): [0,1] the convolution                             (2 events)
 */
int cbr_forward_train_ev(const cbr_shape *shape,
                         const uint16_t *x, const uint16_t *w,
                         const float *gamma, const float *beta,
                         const float *run_mean_in, const float *run_var_in,
                         float eps, float momentum,
                         uint16_t *z, uint16_t *y, uint32_t *relu_mask,
                         float *saved_mean, float *saved_invstd,
                         float *run_mean_out, float *run_var_out,
                         void *workspace, size_t ws_bytes, void *stream, void *const *events);

int cbr_forward_infer_ev(const cbr_shape *shape,
                         const uint16_t *x, const uint16_t *w, const float *conv_bias,
                         const float *gamma, const float *beta,
                         const float *run_mean, const float *run_var, float eps,
                         uint16_t *y, void *workspace, size_t ws_bytes, void *stream,
                         void *const *events);

int cbr_backward_ev(const cbr_shape *shape,
                    const uint16_t *x, const uint16_t *w, const uint16_t *z,
                    const uint32_t *relu_mask, const uint16_t *dy,
                    const float *gamma, const float *saved_mean, const float *saved_invstd,
                    uint16_t *dz, float *dgamma, float *dbeta, float *dw, uint16_t *dx,
                    void *workspace, size_t ws_bytes, void *stream, void *const *events);

int cbr_conv2d_bias_relu_ev(const cbr_shape *shape, const uint16_t *x, const uint16_t *w, const float *bias,
                            uint16_t *y, void *stream, void *const *events);

int cbr_conv2d_bias_ev(const cbr_shape *shape, const uint16_t *x, const uint16_t *w, const float *bias,
                       uint16_t *y, void *stream, void *const *events);

#ifdef __cplusplus
}
#endif

#endif /* CBR_H */
