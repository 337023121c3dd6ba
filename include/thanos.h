/*
 * thanos.h -- C ABI of libthanos: block-wise multi-constraint pruning of one
 * linear layer (Thanos-style) on AMD Instinct MI355X (gfx950).
 *
 * Method sources (page titles and sections):
 *   [BLOG]  "Pruning LLMs with Thanos" (project blog post):
 *           "The layer-reconstruction lens" (objective ||WX - What X||_F^2,
 *           decomposition over rows), "One deletion with compensation: the OBS
 *           view" (damped Hessian, OBS update and cost), "Contribution one: solve
 *           a selected set directly" (joint update delta = -u Rhat^-1 R),
 *           "Contribution two: keep the budget global and the execution local"
 *           (dynamic residual budget), "Making irregular row masks batchable".
 *   [EXPL]  "Weight Pruning in Large Language Models: How SparseGPT, Wanda, and
 *           Semi-Structured 2:4 Sparsity ..." (explainer): "SparseGPT:
 *           Second-Order Reconstruction at Scale" (H = 2XX^T + lambda*I, one
 *           Cholesky of H^-1 per layer), "Wanda: Pruning by Weights and
 *           Activations", "N:M Semi-Structured Sparsity (2:4 Pattern)".
 *   [REPO]  "Thanos - Method of Pruning LLMs" (repository README), "Usage":
 *           --sparsity_ratio and --sparsity_type {unstructured, 2:4, 4:8}.
 *
 * Conventions for every entry point:
 *   - Pointers are DEVICE pointers unless the comment says "host".
 *   - Matrices are row-major. W is c x b (row = output channel, contiguous over
 *     the b inputs). X is b x n with tokens as columns; it is passed token-major
 *     as X^T [n, b] (the same bytes as column-major X), row pitch ldx elements.
 *   - The caller owns every buffer, including the workspace. The library never
 *     allocates device memory; the one entry point without a workspace argument
 *     (th_prune_layer_noalloc) uses a fixed array the library holds from load.
 *   - Work is enqueued on `stream` (a hipStream_t; NULL = the default stream).
 *     The factorisation of the Hessian also runs part of its work on a stream
 *     the library creates once per device and host thread (default priority);
 *     that work is joined back into `stream` with events, so everything the
 *     caller enqueues on `stream` afterwards sees the results.
 *     Entry points that return host values or a status that depends on device
 *     results synchronise that stream before returning.
 *   - Argument errors are reported before anything is launched. No C++
 *     exception crosses this interface. th_last_error() gives a message for the
 *     last non-OK status of the calling thread.
 *   - Calls that share a workspace or output buffers must not overlap.
 */
#ifndef THANOS_H_
#define THANOS_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct ihipStream_t;
typedef struct ihipStream_t* th_stream_t; /* identical to hipStream_t */

typedef enum {
  TH_OK = 0,
  TH_ERR_INVALID_ARG = 1, /* bad size, null pointer, unsupported combination */
  TH_ERR_NOT_SPD = 2,     /* the damped Hessian has a non-positive pivot */
  TH_ERR_NONFINITE = 3,   /* NaN/Inf in W or in the Hessian's diagonal */
  TH_ERR_WORKSPACE = 4,   /* workspace smaller than the size query returned */
  TH_ERR_HIP = 5          /* a HIP runtime call failed */
} th_status;

typedef enum { TH_F32 = 0, TH_BF16 = 1 } th_dtype;
typedef enum { TH_UNSTRUCTURED = 0, TH_NM = 1 } th_pattern_kind;
typedef enum { TH_SCORE_OBS = 0, TH_SCORE_WANDA = 1 } th_score;

typedef struct {
  int32_t kind; /* th_pattern_kind */
  int32_t n;    /* N:M: keep n of every m consecutive weights of a row */
  int32_t m;
} th_pattern;

typedef struct {
  /* Unstructured: fraction p in [0,1]; the layer loses
   * k_total = round-half-even(p*c*b) weights in total [BLOG, "Contribution two"].
   * N:M: ignored (the pattern fixes 1 - n/m), as with [REPO]'s --sparsity_ratio. */
  double sparsity;
  th_pattern pattern;
  /* Column block size B, 1 <= B <= 128. Blocks run left to right; finished
   * blocks are frozen [BLOG, "The scaling problem, and what SparseGPT changes"].
   * N:M needs m | B and m | b. */
  int64_t block;
  /* Damping: absolute lambda if lambda_is_relative == 0, else
   * lambda = lambda * mean(diag(2G)) (typical: 0.01, relative). */
  double lambda;
  int32_t lambda_is_relative;
  /* Score g_q in S_kq = W_kq^2 g_q: OBS g_q = 1/[(H_F)^-1]_qq over the active
   * columns F [BLOG, "One deletion with compensation"]; Wanda g_q = G_qq
   * ([EXPL, "Wanda"]; same ordering as |W| ||X_q||). */
  int32_t score;
} th_prune_params;

typedef struct {
  double lambda_used;    /* absolute damping that was applied (or derived, see below) */
  int64_t total_pruned;  /* number of weights set to zero */
  int64_t nblocks;       /* number of column blocks */
} th_stats;

/* H += 2 * X_chunk^T X_chunk on the lower triangle (entries with row >= column).
 * [EXPL, "SparseGPT: Second-Order Reconstruction at Scale"]: H = 2XX^T (+ lambda I
 * later). X_chunk: [t, b] token-major, dtype xdt (TH_BF16: products are exact in
 * fp32 and accumulate in fp32 on the matrix cores; TH_F32: fp32 FMA). ldx >= b
 * and, for TH_BF16, b % 8 == 0, ldx % 8 == 0 and a 16-byte aligned X. H: b x b fp32, zeroed by
 * the caller before the first chunk; the strict upper triangle is not touched.
 * workspace (optional, may be NULL with workspace_bytes 0; 16-byte aligned) lets
 * small b split the token range over more workgroups and large b run 384 x 256
 * tiles with the last round's tiles cut into token pieces; size from
 * th_hessian_workspace_size. The summation order is fixed, so repeated calls give
 * bit-identical H. Asynchronous. */
th_status th_hessian_accumulate(float* H, const void* X_chunk, th_dtype xdt, int64_t t,
                                int64_t b, int64_t ldx, void* workspace,
                                size_t workspace_bytes, th_stream_t stream);
th_status th_hessian_workspace_size(int64_t t, int64_t b, size_t* bytes /* host */);

/* Damping and symmetrisation of an accumulated H (= 2G on the lower triangle):
 * lambda = lambda_rel * mean(diag(H)) if lambda_is_relative else lambda;
 * H_qq += lambda; the upper triangle is overwritten by the mirror of the lower
 * [BLOG, "One deletion with compensation"]. *lambda_out (host, optional) gets the
 * absolute lambda. Synchronises the stream. */
th_status th_hessian_finalize(float* H, int64_t b, double lambda, int32_t lambda_is_relative,
                              double* lambda_out, th_stream_t stream);

/* Prune one layer [BLOG, "Contribution one" and "Contribution two"; N:M masks per
 * "The semi-structured N:M variant" paragraph of "Contribution two"].
 *   W [c,b] dtype wdt (TH_BF16 or TH_F32): read, then overwritten with What
 *     rounded to wdt (round-to-nearest-even for bf16).
 *   Exactly one of X / H is non-NULL:
 *     X [n,b] token-major (ldx = b), dtype xdt: H = 2XX^T + lambda*I is built
 *       inside (p->lambda, p->lambda_is_relative);
 *     H [b,b] fp32, full symmetric and already damped. If p->score is Wanda,
 *       G_qq is taken as (H_qq - lambda)/2 with lambda = p->lambda (absolute) or
 *       lambda_rel/(1+lambda_rel) * mean(diag H) (relative; exact for an H that
 *       th_hessian_finalize produced with the same lambda_rel).
 *   W_out_f32 [c,b] fp32 (optional): What in fp32.
 *   mask_out [c,b] uint8 (optional): 1 = pruned.
 *   workspace: >= th_prune_layer_workspace_size bytes, 256-byte aligned.
 *   stats_out (host, optional); block_counts (host, optional, nblocks entries):
 *     weights pruned in each block.
 * Returns TH_ERR_NOT_SPD if the Cholesky factorisation of the damped Hessian
 * meets a non-positive pivot, TH_ERR_NONFINITE for NaN/Inf in W or diag(H).
 * Synchronises the stream once, at the end. */
th_status th_prune_layer(void* W, th_dtype wdt, int64_t c, int64_t b, const void* X,
                         th_dtype xdt, int64_t n, const float* H, const th_prune_params* p,
                         float* W_out_f32, uint8_t* mask_out, void* workspace,
                         size_t workspace_bytes, th_stats* stats_out,
                         int64_t* block_counts, th_stream_t stream);
th_status th_prune_layer_workspace_size(int64_t c, int64_t b, int64_t n, int32_t have_x,
                                        const th_prune_params* p, size_t* bytes /* host */);

/* th_prune_layer without a workspace argument and without allocating, for callers
 * that cannot allocate device memory (code under HIP graph capture, tight serving
 * loops, harnesses that forbid allocation). Its device memory is one file-scope
 * array of TH_NOALLOC_SCRATCH_BYTES bytes that every GPU the library runs on holds
 * from the library's load until the process ends. th_prune_layer_workspace_size
 * bounds what a call needs (less when the caller passes W_out_f32 and mask_out):
 * square layers up to b = 1024 fit with X given, up to about b = 2000 with a
 * given H. Arguments,
 * results, synchronisation and errors as th_prune_layer; a layer that needs more
 * scratch returns TH_ERR_WORKSPACE before anything is launched. The first call on
 * a device (per host thread) looks up the array's address and creates the
 * factorisation's side stream and events; no call allocates memory. All calls on
 * one GPU share its array and every call clears what must start at zero: calls
 * that overlap on one GPU (other host threads, other streams) race and must not
 * be made. */
#define TH_NOALLOC_SCRATCH_BYTES (64u << 20)
th_status th_prune_layer_noalloc(void* W, th_dtype wdt, int64_t c, int64_t b, const void* X,
                                 th_dtype xdt, int64_t n, const float* H, const th_prune_params* p,
                                 float* W_out_f32, uint8_t* mask_out, th_stats* stats_out,
                                 int64_t* block_counts, th_stream_t stream);

/* Inverse factor of a damped Hessian, for layers that share one input (q/k/v,
 * gate/up): H^-1 = U^T U with U upper [EXPL, "SparseGPT: Second-Order
 * Reconstruction at Scale": one factorisation of the inverse Hessian per layer;
 * here per shared input]. Exactly one of X ([n,b] token-major, dtype xdt: H =
 * 2XX^T + lambda*I is built inside) / H ([b,b] fp32, full symmetric, already
 * damped) is non-NULL; lambda and lambda_is_relative as in th_prune_params.
 * U [b,b] fp32 (device, caller-owned): receives U, zero below the diagonal (with
 * X it also serves as the Hessian's scratch). *lambda_out (host, optional): the
 * absolute lambda, added (X given) or taken to be in a given H (lambda when
 * absolute, lambda/(1+lambda) * mean(diag H) when relative). workspace: >=
 * th_factor_workspace_size bytes, 256-byte aligned. Synchronises once.
 * TH_ERR_NOT_SPD / TH_ERR_NONFINITE as th_prune_layer. */
th_status th_factor(const void* X, th_dtype xdt, int64_t n, const float* H, int64_t b,
                    double lambda, int32_t lambda_is_relative, float* U, double* lambda_out,
                    void* workspace, size_t workspace_bytes, th_stream_t stream);
th_status th_factor_workspace_size(int64_t b, int64_t n, int32_t have_x, size_t* bytes /* host */);

/* th_prune_layer from a given factor U (th_factor's output; read only, copied
 * into the workspace): the same block loop, so the result is identical to
 * th_prune_layer on the H that U came from [BLOG, "Contribution one" and
 * "Contribution two"]. p->score must be TH_SCORE_OBS (the Wanda score needs
 * diag(H)); p->lambda is not used and stats_out->lambda_used is 0. Other
 * arguments, synchronisation and errors as th_prune_layer. workspace: >=
 * th_prune_layer_factored_workspace_size bytes. */
th_status th_prune_layer_factored(void* W, th_dtype wdt, int64_t c, int64_t b, const float* U,
                                  const th_prune_params* p, float* W_out_f32, uint8_t* mask_out,
                                  void* workspace, size_t workspace_bytes, th_stats* stats_out,
                                  int64_t* block_counts, th_stream_t stream);
th_status th_prune_layer_factored_workspace_size(int64_t c, int64_t b, const th_prune_params* p,
                                                 size_t* bytes /* host */);

/* The alpha variant: round-half-even(alpha*c) rows of W stay dense, the other
 * rows are pruned as a layer of their own [BLOG, "What the experiments show":
 * the alpha = 0.1 variant keeps 10% of the rows as outliers, so 50% becomes 45%].
 * Which rows is not on the pages; here the rows of largest output energy
 * s_k = sum_q W_kq^2 G_qq (fp64 sums, ranked by their fp32 value, ties to the
 * higher row index), with G_qq from X's column norms (th_column_sq_norms) or
 * from a given damped H as (H_qq - lambda)/2. Arguments as th_prune_layer, plus
 * alpha in [0, 1] and dense_rows_out [c] uint8 (device, optional): 1 = kept
 * dense. Dense rows are left unchanged (mask 0); block_counts and stats count
 * the pruned rows only. workspace: >= th_prune_layer_alpha_workspace_size
 * bytes. Synchronisation and errors as th_prune_layer (a non-finite weight in
 * any row gives TH_ERR_NONFINITE). */
th_status th_prune_layer_alpha(void* W, th_dtype wdt, int64_t c, int64_t b, const void* X,
                               th_dtype xdt, int64_t n, const float* H, const th_prune_params* p,
                               double alpha, float* W_out_f32, uint8_t* mask_out,
                               uint8_t* dense_rows_out, void* workspace, size_t workspace_bytes,
                               th_stats* stats_out, int64_t* block_counts, th_stream_t stream);
th_status th_prune_layer_alpha_workspace_size(int64_t c, int64_t b, int64_t n, int32_t have_x,
                                              const th_prune_params* p, double alpha,
                                              size_t* bytes /* host */);

/* Input of down_proj from a gated feed-forward: Y = silu(X W_gate^T) * (X W_up^T)
 * with silu(z) = z/(1+e^-z) [BLOG, "The compression target: linear layers":
 * feed-forward projections joined by a nonlinearity; gate/up/down as in LLaMA].
 * X [n,d] token-major, W_gate and W_up [f,d] row-major, Y [n,f]; all bf16 (dt
 * must be TH_BF16), device, caller-owned. Products on the bf16 matrix cores with
 * fp32 sums, silu and the product in fp32, Y rounded to nearest even. Needs
 * d % 8 == 0 and 16-byte aligned X, W_gate, W_up. Asynchronous on the stream. */
th_status th_gated_ffn_input(const void* X, const void* W_gate, const void* W_up, th_dtype dt,
                             int64_t n, int64_t d, int64_t f, void* Y, th_stream_t stream);

/* Linear layer with its epilogue: Y = act(X W^T + bias) + residual, what a block's
 * (pruned) projections hand to the next layer [BLOG, "The compression target:
 * linear layers"; "The layer-reconstruction lens"]. X [n,b] token-major (row pitch
 * ldx), W [c,b], bias [c] or NULL, all bf16 (dt must be TH_BF16); residual [n,c]
 * (row pitch ldr) or NULL and Y [n,c] (row pitch ldy) in ydt (bf16 or fp32).
 * Products on the bf16 matrix cores with fp32 sums, epilogue in fp32, Y rounded
 * once. gelu(z) = z Phi(z), with the error function; silu(z) = z / (1 + e^-z). Y may
 * be the residual (same pitch); it must not overlap X, W or bias. Needs
 * b % 8 == 0, b >= 8, ldx % 8 == 0, b and ldx < 2^22, and 16-byte aligned X and W;
 * n < 2^31, c < 2^27 and at most 2^24 - 16 blocks of 64 x 64 outputs; n = 0 is allowed. workspace (optional, may be NULL with workspace_bytes 0;
 * 16-byte aligned) lets launches of few tiles split the contraction; size from
 * th_linear_workspace_size (0 where it does not help). The pieces are summed in a
 * fixed order, so repeated calls give identical bits. Asynchronous. */
typedef enum { TH_ACT_NONE = 0, TH_ACT_RELU = 1, TH_ACT_SILU = 2, TH_ACT_GELU = 3 } th_activation;
th_status th_linear_workspace_size(int64_t n, int64_t b, int64_t c, size_t* bytes /* host */);
th_status th_linear(const void* X, int64_t ldx, const void* W, th_dtype dt, int64_t n, int64_t b,
                    int64_t c, const void* bias, th_activation act, const void* residual,
                    int64_t ldr, void* Y, th_dtype ydt, int64_t ldy, void* workspace,
                    size_t workspace_bytes, th_stream_t stream);

/* Microscaled matrices, the form in which the pruned layers of a block are served [BLOG,
 * "The compression target: linear layers"]: [n, b] in blocks of 32 consecutive elements of
 * a row; a value is its element times 2^(scale - 127) of its block. Elements are e4m3 (a
 * byte: sign, 4 bits of exponent, 3 of mantissa, up to 448) or e2m1 (4 bits, up to 6;
 * element 2i of a row in the low half of byte i). Scales are a byte a block; 255: none of
 * the block's values is a number. */
typedef enum { TH_MX_E4M3 = 0, TH_MX_E2M1 = 1 } th_mx_type;
typedef struct {
  void* elements; /* element bytes of row t from elements + t * ld */
  void* scales;   /* scales of row t from scales + t * lds, b / 32 bytes */
  int64_t ld, lds; /* row pitches in BYTES */
  int32_t type;   /* th_mx_type */
} th_mx;

/* X [n,b] (row pitch ldx elements, dtype xdt) in the form of Y (host struct; its buffers are
 * written): a block's scale is the smallest power at which none of its elements, rounded to
 * nearest even, passes the type's largest number, so an element is off by at most half a
 * step; below 2^-127 elements become 0 or what is left of them, past 2^119 (e4m3) and 2^125
 * (e2m1) they saturate. A block that holds a NaN or an infinity gets scale 255 and
 * elements 0. b % 32 == 0; any row pitch and alignment; n = 0 is allowed, n < 2^31. Buffers
 * must not overlap. Asynchronous. */
th_status th_mx_quantize(const void* X, th_dtype xdt, int64_t n, int64_t b, int64_t ldx,
                         const th_mx* Y, th_stream_t stream);
/* The values of X [n,b] as Y (row pitch ldy elements, dtype ydt), rounded once. Arguments as
 * above. Asynchronous. */
th_status th_mx_dequantize(const th_mx* X, int64_t n, int64_t b, void* Y, th_dtype ydt,
                           int64_t ldy, th_stream_t stream);

/* th_linear on microscaled operands, Y = act(X W^T + bias) + residual: X [n,b] in either
 * type, W [c,b] of TH_MX_E2M1. Elements 16-byte aligned with row pitches that are multiples
 * of 16; scales likewise, and the bytes behind a row's last scale up to the next multiple of
 * 16, the last row's included, may be read (they are never used). bias [c] bf16 or NULL, act,
 * residual and Y (bf16 or fp32: ydt) as in th_linear, any pitch and alignment. Products are
 * exact and sums fp32 where X is e2m1, where Y is fp32 and where n <= 16; with an e4m3 X and a
 * bf16 Y the matrix cores align the products of eight consecutive elements to the largest and
 * drop what lies 13 binary places below it (over normal data 5e-6 of Y in root mean square,
 * 1/300 of Y's own rounding; where large products cancel, up to 2^-13 of the largest each).
 * Who needs fp32's sums there asks for an fp32 Y.
 * n >= 0, c >= 1, 32 <= b < 2^22, b % 32 == 0, pitches < 2^22 bytes. workspace (optional, may
 * be NULL with workspace_bytes 0; 16-byte aligned) lets launches with few tiles split the
 * contraction; size from th_mx_linear_workspace_size (xtype: th_mx_type of X; 0 where it does
 * not help). The order of all sums is fixed, so repeated calls give identical bits.
 * Asynchronous. */
th_status th_mx_linear_workspace_size(int32_t xtype, int64_t n, int64_t b, int64_t c, th_dtype ydt,
                                      size_t* bytes /* host */);
th_status th_mx_linear(const th_mx* X, const th_mx* W, int64_t n, int64_t b, int64_t c,
                       const void* bias, th_activation act, const void* residual, int64_t ldr,
                       void* Y, th_dtype ydt, int64_t ldy, void* workspace, size_t workspace_bytes,
                       th_stream_t stream);

/* What a product of these sizes runs on (host only): the tokens and channels of a workgroup's
 * tile and the pieces of its contraction, with the workspace of
 * th_mx_linear_workspace_size or without one. */
th_status th_debug_mx_linear_plan(int32_t xtype, int64_t n, int64_t b, int64_t c, th_dtype ydt,
                                  int32_t workspace, int32_t* tokens, int32_t* channels,
                                  int32_t* pieces);

/* Root-mean-square norm of the rows of a residual stream, what the q/k/v and the
 * gate/up projections of a block read [BLOG, "The compression target: linear
 * layers"]: Y_tq = X_tq / sqrt(mean_q X_tq^2 + eps) * weight_q. X [n,b] (row pitch
 * ldx, dtype xdt), weight [b] in xdt, Y [n,b] (row pitch ldy, dtype ydt); sums and
 * products in fp32, Y rounded once. Y may be X (same dtype and pitch); otherwise
 * they must not overlap. n = 0 is allowed; n < 2^31; eps 0 or a positive normal
 * fp32 number. A row whose sum of squares passes fp32's range gives zeros. Any width,
 * row pitch and alignment of whole elements. Asynchronous on the stream. */
th_status th_rms_norm(const void* X, th_dtype xdt, int64_t n, int64_t b, int64_t ldx,
                      const void* weight, double eps, void* Y, th_dtype ydt, int64_t ldy,
                      th_stream_t stream);

/* The norm behind an addition to the residual stream: h = X + R rounded to xdt, stored in sum
 * (optional), and h / sqrt(mean h^2 + eps) * weight in Y (dtype ydt) or, with Y NULL,
 * microscaled in Y_mx (host struct), what th_mx_linear reads. R NULL: h = X, and sum has to be
 * NULL. X, R, sum [n,b] in xdt with their own row pitches in elements, weight [b] in xdt.
 * Sums, root and products in fp64, every output rounded once (Y_mx: scales and roundings as
 * in th_mx_quantize of the unrounded values; b % 32 == 0). sum may be X or R (same pitch); Y
 * and Y_mx must not overlap other buffers. n, eps, widths, pitches and alignments as in
 * th_rms_norm. Asynchronous. */
th_status th_add_rms_norm(const void* X, int64_t ldx, const void* R, int64_t ldr, th_dtype xdt,
                          int64_t n, int64_t b, const void* weight, double eps, void* sum,
                          int64_t ldsum, void* Y, th_dtype ydt, int64_t ldy, const th_mx* Y_mx,
                          th_stream_t stream);

/* Rotary positions of the queries and keys of n tokens, with an optional norm of
 * each head in the same pass. Element e of head h of token t is at
 * x[t * x_token + h * x_head + e] (strides in elements); y likewise. norm: [d]
 * weights in the same dtype, or NULL for none. y may be x with the same strides;
 * otherwise they must not overlap. */
typedef struct {
  const void* x;
  void* y;
  const void* norm;
  int64_t heads;
  int64_t x_token, x_head, y_token, y_head;
} th_heads;
typedef enum { TH_ROTARY_HALF = 0, TH_ROTARY_INTERLEAVED = 1 } th_rotary_layout;

/* q and k (host structs; k may be NULL): heads of d elements, 1 <= d <= 256, dtype
 * dt. A head with a norm becomes x / sqrt(mean x^2 + eps) * norm first (eps as in
 * th_rms_norm, norms alike in fp32). Then the
 * pairs of its first rot elements (even, 0 <= rot <= d), (x_i, x_{i+rot/2}) for
 * TH_ROTARY_HALF or (x_2i, x_2i+1) for TH_ROTARY_INTERLEAVED, i < rot/2, turn by
 * the angle positions[t] * freqs[i]: (a, b) -> amplitude (a cos - b sin,
 * b cos + a sin). The elements past rot keep their (normed) value. positions [n]
 * int32 (device; any order and sign), or NULL for 0 .. n-1; freqs [rot/2] double
 * (device), see th_rotary_freqs. Angles, their sines and cosines are fp64,
 * rounded once; the rest is fp32, outputs rounded once. amplitude: 0 or a normal
 * fp32 number. Neither side's y may overlap the other side's x or y. n = 0 is
 * allowed; n * heads < 2^31. Asynchronous. */
th_status th_rotary(const th_heads* q, const th_heads* k, th_dtype dt, int64_t n, int64_t d,
                    int64_t rot, th_rotary_layout layout, const int32_t* positions,
                    const double* freqs, double amplitude, double eps, th_stream_t stream);

/* Frequencies for th_rotary, f_i = base^(-2i/rot) radians a position for i < rot/2,
 * scaled for long contexts: with by_bands == 0 all of them are divided by `divide`
 * (1 = unscaled); with by_bands != 0 a pair that makes r = original_length f_i /
 * (2 pi) turns over the original length keeps its frequency for r >= fast_turns,
 * has it divided by `divide` for r <= slow_turns, and between them is multiplied by
 * keep + (1 - keep) / divide, keep = (r - slow_turns) / (fast_turns - slow_turns).
 * scaling NULL: unscaled with base 10000. freqs: HOST, rot/2 doubles. Host only. */
typedef struct {
  double base;
  double divide;
  double original_length, slow_turns, fast_turns;
  int32_t by_bands;
} th_rotary_scaling;
th_status th_rotary_freqs(int64_t rot, const th_rotary_scaling* scaling, double* freqs /* host */);

/* Attention over packed sequences, what o_proj reads [BLOG, "The compression target:
 * linear layers"; "The layer-reconstruction lens"]: per query and head
 * O = softmax(scale Q K^T) V over the visible keys. Element e of head h of row t of
 * Q is at Q[t * q_token + h * q_head + e] (strides in elements); K, V and O alike.
 * Query head h reads key head h / (hq / hk).
 *   Sequence s owns rows q_start[s] .. q_start[s+1]-1 of Q and O and rows
 *   k_start[s] .. k_start[s+1]-1 of K and V (nseq + 1 ascending int32, device).
 *   k_start NULL: the same as q_start. q_start NULL (then k_start NULL, nseq 1):
 *   all rows are one sequence. With causal != 0 the last query of a sequence sees
 *   its last key, the one before it one key fewer, and so on (a sequence may have
 *   more keys than queries: single tokens over a cache; or fewer: its first queries
 *   see none). Lengths of 0 are allowed.
 * A query that sees no key gets zeros. What hidden keys and values hold never enters,
 * infinities and NaN included. Rows of O before q_start[0] or from q_start[nseq] on
 * are left as they are. Start values outside the tensors are moved to their ends, so
 * a bad one never reads or writes outside them; where starts do not ascend, the rows
 * concerned are unspecified. */
typedef struct {
  int64_t nq, nk;     /* rows of Q and O; rows of K and V */
  int64_t hq, hk, d;  /* heads of Q and O; of K and V; elements per head */
  int64_t q_token, q_head, k_token, k_head, v_token, v_head, o_token, o_head;
  int64_t nseq;
  int32_t causal;
  double scale;       /* > 0, typically 1 / sqrt(d); scale log2(e) a normal fp32 number */
} th_attention_params;

/* dt must be TH_BF16; 8 <= d <= 128, d % 8 == 0; hk divides hq; strides are multiples
 * of 8 (k_token, v_token < 2^24) and Q, K, V, O 16-byte aligned; nq * hq / hk,
 * nk < 2^31 - 2^16; hk times the row blocks (of 32 rows where the sequences average
 * no more, else of 128), plus hk nseq, < 2^24. O must not overlap the inputs. Scores,
 * maxima, sums and O accumulate in fp32. The weights enter the second product rounded to
 * bf16; where the sequences average no more than 32 rows (tokens times hq / hk), as a
 * bf16 value and its rest. workspace (optional, may be NULL with workspace_bytes 0;
 * 16-byte aligned) lets launches of few queries split the keys; size from
 * th_attention_workspace_size (0 where it does not help). The order of all sums is
 * fixed, so repeated calls give identical bits. How the work is cut follows the average
 * lengths, all that the host knows: sequences that differ by more than a factor of about
 * ten, or a prompt among many single tokens, are faster in a call of their own.
 * Asynchronous. */
th_status th_attention_workspace_size(const th_attention_params* p, size_t* bytes /* host */);
th_status th_attention(const void* Q, const void* K, const void* V, th_dtype dt,
                       const int32_t* q_start, const int32_t* k_start,
                       const th_attention_params* p, void* O, void* workspace,
                       size_t workspace_bytes, th_stream_t stream);

/* A paged cache of the keys and values of nseq sequences (host struct; pointers to the
 * device). Element e of head h of token j of page p is at k[p * k_page + j * k_token +
 * h * k_head + e] (strides in elements); v likewise. Key x of sequence s is token
 * x % page_tokens of page pages[s * pages_row + x / page_tokens]; the sequence has k_len[s]
 * keys, the newest tokens' included. Lengths outside [0, width * page_tokens] are taken as
 * the nearest end of it. Sequences may share pages. */
typedef struct {
  void *k, *v;
  int64_t npages, page_tokens; /* page_tokens: a power of two, 16 .. 65536 */
  int64_t hk, d;               /* key heads; elements per head */
  int64_t k_page, k_token, k_head, v_page, v_token, v_head;
  const int32_t* pages;        /* [nseq][width], row pitch pages_row */
  const int32_t* k_len;        /* [nseq] */
  int64_t nseq, width, pages_row;
} th_paged_cache;

/* The keys and values of nq new tokens, K and V [nq, hk, d] (strides in elements), into the
 * cache's pages. q_start as in th_attention (nseq + 1 ascending int32, device): rows
 * q_start[s] .. q_start[s+1]-1 are the last keys of sequence s, the last row its key
 * k_len[s]-1. q_start NULL: every sequence has nq / nseq rows. A row whose key is before the
 * sequence's first, or whose page is not in [0, npages), is not stored, nor are rows before
 * q_start[0] and from q_start[nseq] on; start values outside [0, nq] are moved to its ends.
 * Where two rows have one place (sequences that share a page), each element there is one of
 * theirs. dt must be TH_BF16; d and alignment as in th_paged_attention, also of K and V.
 * Asynchronous. */
th_status th_cache_store(const void* K, int64_t k_token, int64_t k_head, const void* V,
                         int64_t v_token, int64_t v_head, th_dtype dt, int64_t nq,
                         const int32_t* q_start, const th_paged_cache* cache,
                         th_stream_t stream);

/* th_attention of nq new tokens over a paged cache that holds their keys already: rows
 * q_start[s] .. q_start[s+1]-1 of Q and O (NULL: nq / nseq rows each) over the k_len[s] keys
 * of sequence s. With causal != 0 the last row sees the sequence's last key, the one before
 * it one key fewer, and so on. A row that sees no key gets zeros; what hidden keys and
 * values, and page places past k_len, hold never enters; rows of no sequence are left as they
 * are. Pages outside [0, npages) are read as the nearest end of it. */
typedef struct {
  int64_t nq, hq;  /* rows and heads of Q and O */
  int64_t q_token, q_head, o_token, o_head;
  int32_t causal;
  int32_t even;    /* != 0: q_start is NULL */
  double scale;    /* as in th_attention */
} th_paged_params;

/* dt must be TH_BF16; 8 <= d <= 128, d % 8 == 0; hk divides hq; strides are multiples of 8
 * (k_token, v_token < 2^24), all >= 0, and Q, O, k, v 16-byte aligned; nq * hq / hk and
 * width * page_tokens < 2^31 - 2^16, npages < 2^31, nseq < 2^24; row blocks and pieces of
 * keys in one launch < 2^24. O must not overlap the inputs. Scores, maxima, sums and O
 * accumulate in fp32; the weights enter the second product as a bf16 value and its rest, also a
 * bf16 value, so that 2^-16 of a weight is lost whatever the lengths of its sequence and of the
 * others (th_attention loses 2^-8 where sequences average more than 32 rows). The host needs no
 * lengths: how the keys are cut into pieces is found on the device from the real ones,
 * sequences of up to 32 rows (tokens times hq / hk) apart from longer ones, so that batches of
 * unlike sequences keep every compute unit busy, and a captured call follows the lengths of each
 * replay. workspace (optional, may be NULL with workspace_bytes 0; 16-byte aligned) lets the
 * keys be cut; size from th_paged_attention_workspace_size. The order of all sums is fixed by
 * the lengths, so repeated calls give identical bits. Asynchronous. */
th_status th_paged_attention_workspace_size(const th_paged_cache* cache, const th_paged_params* p,
                                            size_t* bytes /* host */);
th_status th_paged_attention(const void* Q, th_dtype dt, const int32_t* q_start,
                             const th_paged_cache* cache, const th_paged_params* p, void* O,
                             void* workspace, size_t workspace_bytes, th_stream_t stream);

/* Comparator: the column-sequential schedule of SparseGPT on the same Hessian and
 * factor [BLOG, "The scaling problem, and what SparseGPT changes": left to right,
 * every row at once, finished columns frozen, compensation only into active
 * columns, masks refreshed per block; EXPL, "SparseGPT: Second-Order
 * Reconstruction at Scale": pruning w_kq subtracts (w_kq/[H^-1]_qq) times row q
 * of H^-1 over the active columns from the rest of row k]. With H^-1 = U^T U that
 * update is (w_kq/U_qq) U_{q,q:}. Mask of block J chosen at block start from the
 * score w_kq^2/U_qq^2 (the cost of deleting w_kq alone when column q is
 * processed): unstructured, the block's round-half-even(p*c*|J|) lowest
 * (score, flat index k*b+q) — an equal quota per block, unlike th_prune_layer's
 * global budget; N:M, the m-n lowest (score, column) of every aligned group.
 * Arguments, layout, ownership, synchronisation and errors as th_prune_layer;
 * p->score must be TH_SCORE_OBS (else TH_ERR_INVALID_ARG). workspace: >=
 * th_prune_sparsegpt_workspace_size bytes, 256-byte aligned. block_counts get
 * the weights pruned in each block. */
th_status th_prune_sparsegpt(void* W, th_dtype wdt, int64_t c, int64_t b, const void* X,
                             th_dtype xdt, int64_t n, const float* H, const th_prune_params* p,
                             float* W_out_f32, uint8_t* mask_out, void* workspace,
                             size_t workspace_bytes, th_stats* stats_out,
                             int64_t* block_counts, th_stream_t stream);
th_status th_prune_sparsegpt_workspace_size(int64_t c, int64_t b, int64_t n, int32_t have_x,
                                            const th_prune_params* p, size_t* bytes /* host */);

/* E = ||(W - What) X||_F^2 = sum_k D_k G D_k^T and E / ||W X||_F^2
 * [BLOG, "The layer-reconstruction lens"]. W and What: [c,b] dtype wdt. Exactly
 * one of X ([n,b] token-major, dtype xdt) or G ([b,b] fp32, full symmetric,
 * undamped XX^T) is non-NULL. Products on the fp32 matrix cores, sums in fp64.
 * err_out, rel_err_out: host. Synchronises the stream. */
th_status th_reconstruction_error(const void* W, const void* What, th_dtype wdt, int64_t c,
                                  int64_t b, const void* X, th_dtype xdt, int64_t n,
                                  const float* G, void* workspace, size_t workspace_bytes,
                                  double* err_out, double* rel_err_out, th_stream_t stream);
th_status th_reconstruction_error_workspace_size(int64_t c, int64_t b, int32_t have_x,
                                                 size_t* bytes /* host */);

/* ---- Entry points for parity tests: one step of the path on given inputs ---- */

/* N:M selection on given scores [c, blk] fp32: in every aligned group of m
 * columns, mark the m-n lowest (score, column) pairs (ties: lower column first)
 * [BLOG, "The compression target: linear layers"; EXPL, "N:M ..."].
 * mask_blk [c, blk] uint8, 1 = pruned. Asynchronous. */
th_status th_debug_select_nm(const float* scores, int64_t c, int64_t blk, int32_t n, int32_t m,
                             uint8_t* mask_blk, th_stream_t stream);

/* Global residual-budget selection on given scores [c, f] fp32 (f = b_full - j0
 * active columns, row pitch f): the r lowest keys (score, k*b_full + j0 + q)
 * form the candidate set; mask_blk [c, blk] (uint8, row pitch blk) gets the
 * candidates in the first blk columns, s_k [c] (int32, optional) their count per
 * row [BLOG, "Contribution two"]. workspace: >= 64 KiB. Synchronises. */
th_status th_debug_select_global(const float* scores, int64_t c, int64_t f, int64_t b_full,
                                 int64_t j0, int64_t blk, int64_t r, uint8_t* mask_blk,
                                 int32_t* s_k, void* workspace, size_t workspace_bytes,
                                 th_stream_t stream);

/* ---- Comparators without compensation ------------------------------------
 * [EXPL, "Wanda: Pruning by Weights and Activations"]: score |W_kq| * ||X_q||_2,
 * thresholds computed per output row, no update of the remaining weights.
 * [EXPL, "The Failure of Magnitude Pruning in Large Transformers"]: rank by
 * |W_kq| and remove the smallest (compared here per output row, like Wanda).
 * [BLOG, "Why magnitude alone misses important weights"]: W_kq^2 G_qq (G = X X^T)
 * orders like the Wanda score. [EXPL, "N:M Semi-Structured Sparsity (2:4
 * Pattern)"]: both enforce the pattern within every aligned group of m. */
typedef enum { TH_BASE_MAGNITUDE = 0, TH_BASE_WANDA = 1 } th_baseline;

/* gdiag[q] = G_qq = sum_t X_tq^2 (fp64 accumulation in a fixed order, rounded to
 * fp32). X token-major [n, b] (row pitch ldx >= b), bf16 or fp32; gdiag: b floats.
 * workspace (device) >= th_column_sq_norms_workspace_size bytes. Asynchronous. */
th_status th_column_sq_norms_workspace_size(int64_t n, int64_t b, size_t* bytes /* host */);
th_status th_column_sq_norms(const void* X, th_dtype xdt, int64_t n, int64_t b, int64_t ldx,
                             float* gdiag, void* workspace, size_t workspace_bytes,
                             th_stream_t stream);

/* Prune W (c x b, bf16 or fp32) in place: the pruned entries become exactly 0,
 * every other entry is left unchanged. Key of (k, q): w^2 rounded to fp32, times
 * gdiag[q] (Wanda; gdiag required, device, b floats) or times 1 (magnitude;
 * gdiag ignored), rounded to fp32; among equal keys the lower column is pruned
 * first. Unstructured (p->pattern.kind): every row loses its round-half-even(
 * p->sparsity * b) smallest keys. N:M: in every aligned group of m along a row,
 * the m-n smallest (1 <= m <= 128, m | b). p->block, lambda and score are not
 * used. mask_out (optional, device, c x b uint8): 1 = pruned. Asynchronous. */
th_status th_prune_baseline(void* W, th_dtype wdt, int64_t c, int64_t b, th_baseline method,
                            const float* gdiag, const th_prune_params* p, uint8_t* mask_out,
                            th_stream_t stream);

/* U = upper-triangular factor with H^-1 = U^T U (U = chol_upper(H^-1), the factor
 * [EXPL, "SparseGPT"] computes once per layer), from a damped, full symmetric H
 * [b,b] fp32. U [b,b] fp32 (strict lower triangle zero). workspace: >= b*b*4 +
 * 2*ceil(b/128)*128*256*4 + 2*2*3*256*ceil(b/256)*256 + 65536 bytes
 * (TH_ERR_WORKSPACE if smaller). Returns
 * TH_ERR_NOT_SPD on a non-positive pivot.
 * Synchronises. */
th_status th_debug_factor(const float* H, int64_t b, float* U, void* workspace,
                          size_t workspace_bytes, th_stream_t stream);

/* H += 2 X^T X on the lower triangle through the 384 x 256 rectangles that
 * th_hessian_accumulate takes for large layers (bf16 X, [EXPL, "SparseGPT:
 * Second-Order Reconstruction at Scale"]), with the work split fixed here
 * instead of by the device: whole tiles in rounds of P workgroups, each remaining
 * tile cut into m pieces of consecutive 32-token stages whose sums are added in a
 * fixed order (m = 0: chosen as for the device's compute units; m = 1: those
 * tiles whole as well). Arguments as th_hessian_accumulate with t >= 32 and
 * ldx < 2^25; 1 <= P <= 4096, 0 <= m <= t / 32; workspace: >= (number of cut
 * tiles) * (m * 98304 + 1) * 4 bytes (TH_ERR_WORKSPACE if smaller;
 * ceil(b/384) * ceil(b/256) * (m * 98304 + 1) * 4 always suffices), 16-byte
 * aligned. Asynchronous. */
th_status th_debug_syrk_rect(float* H, const void* X_chunk, int64_t t, int64_t b, int64_t ldx,
                             int32_t P, int32_t m, void* workspace, size_t workspace_bytes,
                             th_stream_t stream);

/* W[:, col0:col_end] -= Z[:, 0:K] R[r0:r0+K, col0:col_end] on operands split once into
 * three bf16 planes and 256 x 256 tiles, the update the N:M block loop applies to
 * the columns past each group of eight blocks ["Pruning LLMs with Thanos", section
 * "Contribution one: solve a selected set directly": every block's compensation
 * reaches all still-active columns]. W [c, b] fp32 (pitch b), Z [c, ldz] fp32,
 * R [>= r0+K, b] fp32, all device. K % 16 == 0, 0 <= col0 < col_end <= b, ldz >= K.
 * The tiles of a last, partial round of one workgroup per compute unit run in
 * pieces of consecutive k stages whose sums are subtracted in a fixed order.
 * workspace: the split planes, Y = 3 * ceil(K/64)*64 * (ceil(c/256) +
 * ceil((col_end-col0)/256)) * 256 * 2 bytes rounded up to a multiple of 256, then
 * 256 piece slots of 256 KB: >= Y + 67108864 bytes (TH_ERR_WORKSPACE if smaller),
 * 16-byte aligned. Asynchronous. */
th_status th_debug_far_update(float* W, int64_t c, int64_t b, const float* Z, int64_t ldz,
                              const float* R, int64_t r0, int64_t K, int64_t col0,
                              int64_t col_end, void* workspace, size_t workspace_bytes,
                              th_stream_t stream);

/* Message for the last non-OK status on this thread (never NULL). */
const char* th_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* THANOS_H_ */
