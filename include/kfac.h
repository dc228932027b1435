/*
 * kfac.h -- C ABI of the GB300 (sm_103a) K-FAC curvature-step library
 * (libkfac_gb300.so).
 *
 * The library implements the per-layer Kronecker-factored curvature step of
 * Osawa et al., "Large-Scale Distributed Second-Order Optimization Using
 * Kronecker-Factored Approximate Curvature for Deep Convolutional Neural
 * Networks" (section 3.2, Eq. 4-7, and the diagonal BatchNorm Fisher of
 * section 1):
 *   kfac_factor_update   builds A = E[a a^T] / G = E[g g^T] and folds it into a
 *                        running average                      (Eq. 5)
 *   kfac_damp_invert     damps both factors of a layer (pi-split Tikhonov) and
 *                        inverts them                           (Eq. 6)
 *   kfac_precondition    G^-1 grad A^-1                         (Eq. 7)
 *   kfac_bn_diag_fisher  diagonal Fisher of BatchNorm parameters and the
 *                        damped diagonal preconditioned gradient
 * and the operators next to that step when the layer set is a language
 * model's or a policy's: the losses that make the output gradients, and the
 * bound on the step:
 *   kfac_token_logprob, kfac_token_logprob_grad
 *                        log-probabilities of chosen tokens from logits
 *   kfac_policy_loss     clipped policy loss with a KL term, and its gradient
 *   kfac_preference_loss loss over pairs of sequences, and its gradient
 *   kfac_clip_norm       norm over many tensors, clipping, weight step
 *   kfac_verify_draft    drafted tokens accepted or replaced under the policy's
 *                        probabilities
 *   kfac_checkpoint_store, kfac_checkpoint_load, kfac_weight_grad
 *                        layer inputs kept in 8 bits, and the weight gradient
 *                        from them (kfac_factor_update takes them too)
 *
 * Conventions shared by every entry point:
 *   - Every buffer pointer inside a descriptor is a DEVICE pointer on the
 *     current CUDA device, owned by the caller; descriptor arrays themselves
 *     are HOST memory and may be freed when the call returns.
 *   - The library allocates no device memory.  Calls that need scratch take a
 *     caller-owned device `workspace` of at least the size the matching
 *     *_workspace_size query returns (256-byte aligned); its contents need no
 *     initialisation and are clobbered.
 *   - All work is enqueued on `stream` (a cudaStream_t; NULL = legacy default
 *     stream) and is asynchronous: results are ready once the stream has
 *     reached that point.  The library keeps no global state beyond the
 *     per-device streams and events of kfac_damp_invert (below); concurrent
 *     calls on different streams with disjoint buffers and workspaces are
 *     allowed.
 *   - KFAC_ERR_INVALID / KFAC_ERR_UNSUPPORTED / KFAC_ERR_WORKSPACE are
 *     returned BEFORE anything is enqueued (outputs untouched).  Every
 *     operand must be memory of the current device (or managed memory):
 *     host memory or another GPU's memory gives KFAC_ERR_INVALID (checked
 *     last, right before the call enqueues its work).
 *     KFAC_ERR_CUDA reports a launch failure (cudaGetLastError after a
 *     launch); the stream may then hold part of the work.
 *   - Matrices are row-major with an explicit leading dimension (elements).
 *     bf16 values are passed as uint16_t bit patterns.
 *   - Device error word: the first int32 of the workspace of
 *     kfac_factor_update, kfac_damp_invert and kfac_precondition.  Each call
 *     sets it to 0 on its stream before its kernels; its kernels OR bits into
 *     it, which the caller reads after synchronising the stream (the call's
 *     return status cannot report them: the kernels run after it returns):
 *       KFAC_ERRW_NONFINITE (16): a value the call wrote to an output (a
 *         factor, an inverse or one of the inversion's intermediate blocks,
 *         a preconditioned gradient, an updated weight) is NaN or infinite --
 *         e.g. the input held NaN/Inf or the statistic overflowed fp32 --
 *         or an entry of the upper triangle of a factor that
 *         kfac_damp_invert reads is.  The values are written as computed
 *         (NaN stays NaN); nothing is clamped.  Layers of the same call whose
 *         inputs are finite are not affected, but the bit does not say which
 *         layer it was (kfac_damp_invert's info does, per factor).
 *       1, 2, 4 (KFAC_ERRW_TIMEOUT_*): a wait of the tensor-core engine on a
 *         shared-memory barrier (operand stage, free stage, accumulator) ran
 *         past its limit (about 2 s; never expected in a healthy run).  The
 *         CTA then stops issuing work, waits (bounded) for the copies and
 *         products it already issued, releases its tensor memory and exits
 *         without trapping; 8 is set when that drain wait ran out too.  The
 *         call's outputs are then undefined.
 *     A word of 0 means no kernel of the call saw either condition.
 *     kfac_policy_loss, kfac_preference_loss, kfac_clip_norm,
 *     kfac_verify_draft and kfac_weight_grad write the word too (with the
 *     bits that their sections name).
 */
#ifndef KFAC_GB300_H
#define KFAC_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    KFAC_OK = 0,
    KFAC_ERR_INVALID = 1,      /* null pointer, non-positive size, ld < width, ... */
    KFAC_ERR_UNSUPPORTED = 2,  /* valid but not implemented (dtype, shape limit)  */
    KFAC_ERR_NOT_PD = 3,       /* reserved for host-side reporting of info[]      */
    KFAC_ERR_CUDA = 4,         /* a CUDA launch or runtime call failed             */
    KFAC_ERR_WORKSPACE = 5     /* workspace missing, misaligned or too small      */
} kfac_status;

typedef enum {
    KFAC_BF16 = 0,
    KFAC_F32 = 1,
    KFAC_F16 = 2,
    KFAC_E4M3 = 3   /* a checkpoint (kfac_checkpoint_store): sources of kfac_factor_update only */
} kfac_dtype;

/* Storage of a symmetric fp32 factor (only its upper triangle is stored or
 * read):
 *   KFAC_LAYOUT_FULL          row-major [d][ld], entry (i, j) at F[i*ld + j];
 *   KFAC_LAYOUT_PACKED_UPPER  the upper triangle row after row, d(d+1)/2
 *                             floats: entry (i, j), i <= j, at
 *                             F[i*d - i*(i+1)/2 + j]  (row i holds j = i..d-1);
 *                             the ld argument is ignored.
 * The packed form halves a factor's footprint (Osawa et al. section 1: the
 * symmetry of the Kronecker factors is exploited to reduce overhead). */
typedef enum { KFAC_LAYOUT_FULL = 0, KFAC_LAYOUT_PACKED_UPPER = 1 } kfac_layout;

/* Bits of the device error word (see above). */
enum {
    KFAC_ERRW_TIMEOUT_OPERAND = 1,
    KFAC_ERRW_TIMEOUT_STAGE = 2,
    KFAC_ERRW_TIMEOUT_ACCUM = 4,
    KFAC_ERRW_TIMEOUT_DRAIN = 8,
    KFAC_ERRW_NONFINITE = 16,
    KFAC_ERRW_TARGET = 32      /* a target that is not below the vocabulary's size */
};

/* Human-readable name of a status code (static string, never NULL). */
const char *kfac_status_string(int status);

/* Library version as major*10000 + minor*100 + patch: KFAC_VERSION of the header that the
 * library was built with.  Where a caller's KFAC_VERSION has another minor or major number
 * its descriptors may have another size (an array of them another stride): it must not call.
 *   300: kfac_factor_desc ends with scales and ldx. */
#define KFAC_VERSION 300
int kfac_version(void);

/* Number of kernel launches this library has enqueued in this process so far
 * (a diagnostic counter; every entry point adds the launches it makes). */
long long kfac_launch_count(void);

/* Optional per-kernel timing (diagnostic, off by default).  While enabled,
 * every kernel launch the library makes is bracketed by CUDA events recorded
 * on its launch stream (up to 65536 launches).  kfac_timing_read waits for
 * those events, writes for each kernel kind k < n the total device time in
 * milliseconds (ms[k]) and the number of launches (launches[k]), and clears
 * the record; it returns KFAC_OK or KFAC_ERR_CUDA.  kfac_timing_enable
 * returns the previous setting.  Kind names: kfac_timing_kind_name(k) ("" past
 * the last kind).  Launches enqueued during stream capture are recorded as
 * external event nodes of the graph: read the record after the graph has run. */
int kfac_timing_enable(int on);
int kfac_timing_read(double *ms, long long *launches, int n);
const char *kfac_timing_kind_name(int k);
/* The same record launch by launch, in enqueue order: for the first n launches
 * the start (ms after the first recorded launch's start), the duration (ms),
 * the kernel kind and the launch stream's handle (a value that tells streams
 * apart, nothing more); any output may be NULL.  Clears the record and
 * returns the number of launches it held (-1 if an event query failed). */
int kfac_timing_read_launches(double *start_ms, double *dur_ms, int *kind, unsigned long long *stream, int n);

/* ======================================================================
 * kfac_factor_update -- Kronecker factor statistic + running average.
 *
 * Osawa et al. section 3.2, Eq. 5: A_{l-1} is built from the layer's input
 * activations, G_l from the gradients of the layer's output.  For each
 * descriptor the call forms the patch matrix P [M x d] of the source tensor
 * and updates the UPPER triangle (i <= j) of the fp32 factor F in place:
 *
 *     F[i][j] <- beta * F[i][j] + alpha * sum_m P[m][i] * P[m][j]
 *
 * The running average F <- xi F + (1 - xi) P^T P / M is alpha = (1 - xi)/M,
 * beta = xi; accumulating one statistic over several chunks of rows uses
 * beta = xi on the first chunk and beta = 1 afterwards with alpha = (1-xi)/M_total.
 * Entries strictly below the diagonal are neither read nor written.
 *
 * Patch matrix (im2col; row m = (img*Ho + ho)*Wo + wo):
 *   P[m][(r*kw + s)*c + ch] = x[img][ho*stride_h - pad_h + r][wo*stride_w - pad_w + s][ch]
 *   (zero outside the image), Ho = (h + 2*pad_h - kh)/stride_h + 1 (same for Wo),
 *   and when append_one != 0 a last column of ones (an FC bias), so
 *   d = kh*kw*c + (append_one ? 1 : 0).
 * A fully connected layer or an output-gradient source [M x C] is
 * h = w = kh = kw = stride = 1, pad = 0, n = M rows.
 *
 * Fields:
 *   dtype   KFAC_BF16 or KFAC_F16 (tensor cores, fp32 accumulation; the
 *           paper computes in half precision), KFAC_F32 (fp32 CUDA cores), or
 *           KFAC_E4M3: a checkpoint of n rows, c columns (its column of ones
 *           included) of a fully connected source, x its elements with the
 *           pitch ldx and `scales` its exponents (tensor cores, the exact values
 *           that the checkpoint stands for, fp32 accumulation)
 *   x       device, dense NHWC [n][h][w][c] of dtype (channel stride 1)
 *   F, ldf  device fp32 factor in `layout`: KFAC_LAYOUT_FULL [d][ldf] with
 *           ldf >= d, or KFAC_LAYOUT_PACKED_UPPER (d(d+1)/2 floats, ldf
 *           ignored); its upper triangle is updated
 *   layout  kfac_layout of F (a trailing field: zero-initialised = FULL)
 * Errors: INVALID for null x/F, n,h,w,c,kh,kw,stride < 1, pad < 0, Ho/Wo < 1,
 *   ldf < d (full layout), an unknown dtype or layout; for a checkpoint also
 *   null scales and ldx < c; UNSUPPORTED for
 *   d > 65536 or more than 2^31 rows; for a checkpoint also for anything but
 *   h = w = kh = kw = stride = 1, pad = 0, append_one = 0, and for x, scales
 *   or ldx that are not multiples of 16 bytes.
 * Workspace: kfac_factor_update_workspace_size(descs, count) bytes.
 * ==================================================================== */
typedef struct {
    int32_t dtype;
    const void *x;
    int32_t n, h, w, c;
    int32_t kh, kw, stride_h, stride_w, pad_h, pad_w;
    int32_t append_one;
    float *F;
    int64_t ldf;
    float alpha, beta;
    int32_t layout;
    const uint8_t *scales;   /* KFAC_E4M3: the checkpoint's exponents (else ignored) */
    int64_t ldx;             /* KFAC_E4M3: its elements' pitch (else ignored) */
} kfac_factor_desc;

size_t kfac_factor_update_workspace_size(const kfac_factor_desc *descs, int count);
kfac_status kfac_factor_update(const kfac_factor_desc *descs, int count,
                               void *workspace, size_t workspace_bytes, void *stream);

/* ======================================================================
 * kfac_damp_invert -- damped inverses of both factors of each layer.
 *
 * Osawa et al. section 3.2, Eq. 6: (G (x) A)^-1 = G^-1 (x) A^-1.  Damping
 * (the paper states none; Tikhonov split by pi as in the K-FAC paper it
 * cites):
 *     pi = sqrt((tr A / dA) / (tr G / dG)),
 *     damp_A = pi * sqrt(gamma),  damp_G = sqrt(gamma) / pi      (pi_split != 0)
 *     damp_A = damp_G = sqrt(gamma)                              (pi_split == 0)
 * and writes the FULL symmetric fp32 inverses (both triangles, exactly
 * symmetric)
 *     A_inv = (A + damp_A I)^-1,  G_inv = (G + damp_G I)^-1
 * computed in fp32 through a Cholesky factorisation X = L L^T (left-looking,
 * 128-wide block columns; each 128 x 128 diagonal block factored and
 * inverted by one CTA), the triangular inverse W = L^-1 (recursive 2 x 2
 * blocking) and X^-1 = W^T W.  The block products run on tensor cores as
 * three tf32 products per slice on (hi, lo) splits of the fp32 operands with
 * fp32 accumulation.  Only the upper triangles of A and G are read.
 *
 * Streams: the call is ordered on `stream` as a whole.  Its middle part forks
 * onto library-owned streams of the current device (the longest chains at
 * high priority, the rest at low priority; created with their events on the
 * first call on a device) and joins back into `stream`, so stream capture
 * records a graph with parallel branches.  Make the first call on a device
 * outside stream capture.  Optional 16-bit copies of the inverses (bf16, or
 * fp16 when copy_dtype is KFAC_F16) are written when the *_bf16 pointers are
 * non-NULL (their ld must be a multiple of 8 elements and their base 16-byte
 * aligned, for the tensor-core preconditioner).  A and G may be stored in
 * either kfac_layout (layout_A, layout_G; the lda/ldg of a packed factor are
 * ignored); the inverses are always full row-major.
 *
 * Device outputs besides the inverses:
 *   info   int32 [2*count] (may be NULL): info[2l] for A of layer l,
 *          info[2l+1] for its G; 0 = success, k+1 = the k-th pivot was not
 *          positive or not finite (matrix not positive definite); the
 *          corresponding inverse is then undefined.  The call itself still
 *          returns KFAC_OK: read info after synchronising the stream.
 *   damp   float [2*count] (may be NULL): the damp_A, damp_G applied.
 * Errors: INVALID for null A/G/A_inv/G_inv, dA/dG < 1, ld < d (full layouts
 *   and the outputs), gamma < 0, an unknown layout or copy_dtype;
 *   UNSUPPORTED for d > 16384 or a 16-bit copy's ld not a multiple of 8.
 * Workspace: kfac_damp_invert_workspace_size(descs, count) bytes.
 * ==================================================================== */
typedef struct {
    const float *A; int32_t dA; int64_t lda;
    const float *G; int32_t dG; int64_t ldg;
    float *A_inv; int64_t ld_ainv;
    float *G_inv; int64_t ld_ginv;
    uint16_t *A_inv_bf16; int64_t ld_ainv_bf16;   /* optional 16-bit copy */
    uint16_t *G_inv_bf16; int64_t ld_ginv_bf16;   /* optional 16-bit copy */
    int32_t layout_A, layout_G;                   /* kfac_layout of A and G */
    int32_t copy_dtype;                           /* KFAC_BF16 (0) or KFAC_F16 */
} kfac_invert_desc;

size_t kfac_damp_invert_workspace_size(const kfac_invert_desc *descs, int count);
kfac_status kfac_damp_invert(const kfac_invert_desc *descs, int count, float gamma,
                             int pi_split, int32_t *info, float *damp,
                             void *workspace, size_t workspace_bytes, void *stream);

/* ======================================================================
 * kfac_precondition -- preconditioned gradient of each layer.
 *
 * Osawa et al. section 3.2, Eq. 7 in row-major form: for grad [dG x dA],
 *     out = G_inv * grad * A_inv            (out fp32 [dG][ld_out])
 * i.e. (G (x) A)^-1 vec(grad) with symmetric inverses.  A_inv and G_inv are
 * read as FULL matrices (kfac_damp_invert writes both triangles).
 * dtype KFAC_BF16: G_inv, A_inv, grad are bf16 (tensor cores, fp32
 *   accumulation; the intermediate grad*A_inv is rounded to bf16); each ld
 *   must be a multiple of 8 and each base 16-byte aligned.  Rows that start
 *   on 128-byte boundaries (ld a multiple of 64) are read in whole 128-byte
 *   segments and run faster (FC 4096: 0.36 against 0.31 ms); fp32 outputs
 *   whose rows start on 16-byte boundaries are stored 16 bytes at a time.
 * dtype KFAC_F16: the same with fp16 operands (the intermediate is rounded
 *   to fp16).
 * dtype KFAC_F32: all operands fp32 (CUDA cores).
 * Fused step on the weights (Osawa et al. section 3.2, Eq. 8): when w is not
 *   NULL, the epilogue of the second product also applies
 *       w <- w - eta * out               (w fp32 [dG][ld_w], in place)
 *   with the fp32 value of out before it is stored; out may then be NULL
 *   (the preconditioned gradient is not kept).  w must not overlap any other
 *   operand.  Zero-initialised trailing fields (w = NULL) leave w alone.
 * Errors: INVALID for null G_inv/A_inv/grad, both out and w NULL, d < 1,
 *   ld < width; UNSUPPORTED for a bf16 ld/alignment violation or d > 65536.
 * Workspace: kfac_precondition_workspace_size(descs, count, dtype) bytes.
 * ==================================================================== */
typedef struct {
    int32_t dG, dA;
    const void *G_inv; int64_t ld_ginv;
    const void *A_inv; int64_t ld_ainv;
    const void *grad;  int64_t ld_grad;
    float *out;        int64_t ld_out;    /* may be NULL when w is set */
    float *w;          int64_t ld_w;      /* optional: the layer's weights */
    float eta;                            /* learning rate of the step on w */
} kfac_precond_desc;

size_t kfac_precondition_workspace_size(const kfac_precond_desc *descs, int count, int dtype);
kfac_status kfac_precondition(const kfac_precond_desc *descs, int count, int dtype,
                              void *workspace, size_t workspace_bytes, void *stream);

/* ======================================================================
 * kfac_precondition_noalloc -- kfac_precondition without a caller workspace.
 *
 * The paper has no counterpart: this is a service for callers that cannot
 * allocate device memory -- host frameworks that own all device memory
 * through their own pool and do not let a library call cudaMalloc, step
 * loops in which cudaMalloc's implicit device-wide synchronisation would
 * stall the pipeline, and embedded callers whose device-memory budget is
 * fixed at start-up.  Same arguments, results and errors as
 * kfac_precondition (bitwise the same outputs), but the scratch comes from a
 * fixed array in the library's own device memory, kfac_noalloc_scratch_bytes()
 * bytes (32 MiB), held by every GPU that loads the library until the process
 * exits.  The call allocates nothing (no cudaMalloc, cudaFree or allocating
 * library routine).
 *   - KFAC_ERR_WORKSPACE when kfac_precondition_workspace_size() of the
 *     arguments exceeds kfac_noalloc_scratch_bytes() (split the layers over
 *     several calls, or use kfac_precondition with a workspace).
 *   - Set-up: the first call on a device (and the first call after that
 *     device's context was re-created, e.g. by cudaDeviceReset) looks up the
 *     array's device address with that device current (a runtime query, no
 *     allocation).  Make that first call before any stream capture begins.
 *   - All calls on a device share the one array and its contents persist
 *     from call to call (each call clears the parts that must start at zero:
 *     the error word, which is the array's first int32, and the split-K
 *     counters).  Calls whose GPU work overlaps (e.g. on two streams without
 *     ordering between them) race on the array: order them on one stream.
 * ==================================================================== */
size_t kfac_noalloc_scratch_bytes(void);
kfac_status kfac_precondition_noalloc(const kfac_precond_desc *descs, int count, int dtype,
                                      void *stream);

/* ======================================================================
 * kfac_bn_diag_fisher -- diagonal Fisher of BatchNorm parameters.
 *
 * Osawa et al. section 1 (contributions): the Fisher of BatchNormalization
 * layers is approximated as diagonal.  For each descriptor, from per-sample
 * gradients x [n_samples][C] (fp32, row-major, dense):
 *     F_c       <- xi * F_c + (1 - xi) * (1/n) sum_i x_ic^2   (xi = 0: plain)
 *     grad_mean_c = (1/n) sum_i x_ic
 *     precond_c   = grad_mean_c / (F_c + gamma)
 * F is read only when xi != 0.  grad_mean may be NULL.  The reduction order
 * is fixed, so results are bitwise reproducible run to run.
 * Errors: INVALID for null x/F/precond, C < 1, n_samples < 1, gamma < 0.
 * No workspace.
 * ==================================================================== */
typedef struct {
    const float *x;
    int32_t C;
    float *F;
    float *grad_mean;
    float *precond;
} kfac_bn_desc;

kfac_status kfac_bn_diag_fisher(const kfac_bn_desc *descs, int count, int n_samples,
                                float gamma, float xi, void *stream);

/* ======================================================================
 * Losses on logits.
 *
 * The rows of `logits` [rows][ld] (dtype KFAC_BF16, KFAC_F16 or KFAC_F32,
 * `vocab` wide) are scores z of one token each; with the temperature tau,
 *     lse  = ln sum_j exp(z_j / tau),   p_j = exp(z_j / tau - lse),
 *     logp = z_target / tau - lse,      H = - sum_j p_j ln p_j,
 *     d logp / d z_j = (1[j = target] - p_j) / tau,
 *     d H / d z_j    = - p_j (ln p_j + H) / tau.
 * Sums, statistics and coefficients are fp32 or wider; a gradient is rounded
 * once to the logits' dtype.
 *   - target [rows], int64 or (target_i32 != 0) int32.  A row whose target is
 *     negative is ignored: its logits are not read, its gradient is zeros and
 *     its other outputs are 0.  A target >= vocab is ignored too, and sets
 *     KFAC_ERRW_TARGET in the error word of the calls that have one
 *     (kfac_token_logprob writes NaN as its logp).
 *   - Logits of -inf are tokens that cannot be chosen: p = 0, gradient 0.  A
 *     row whose logits are all -inf has no distribution: logp = lse = -inf,
 *     H = 0, gradient 0, and the losses leave it out.  NaN or +inf logits of a
 *     row that is not ignored give NaN for the row, as computed.
 *   - Rows may start at any element boundary and ld may be any value >= vocab.
 *     Rows of logits and dlogits whose starts agree modulo 16 bytes (equal ld
 *     and bases on 16-byte boundaries, for one) are the fastest.
 *   - dlogits must not overlap logits.  Every element [row][j < vocab] is
 *     written; elements past the vocabulary are neither read nor written.
 *   - vocab is at most 2^24 and rows at most 2^31 - 1 (UNSUPPORTED beyond).
 *   - tau must be positive and finite, and so must log2(e) / tau in fp32 (tau at
 *     least 4.3e-39).
 * Results are bitwise reproducible run to run.
 * ==================================================================== */

/* kfac_token_logprob -- log-probabilities of the targets (and, where not NULL,
 * lse and H) of every row.  `saved` [rows][2] (NULL: not wanted) receives the
 * row's maximum m = max_j z_j and sum_j exp((z_j - m) / tau) for the gradient (0,
 * 0 for an ignored row); m and the sum stay apart because lse loses the sum's
 * bits where |m| is large, as in a row masked with the lowest value.
 * Errors: INVALID for null logits/target/logp, rows < 0, vocab < 1, ld < vocab,
 * a bad dtype or tau, saved not on an 8-byte boundary.
 * No workspace, no error word.  rows = 0 does nothing. */
typedef struct {
    int32_t dtype;
    const void *logits; int64_t ld;
    int64_t rows; int32_t vocab;
    const void *target; int32_t target_i32;
    float temperature;
    float *logp;                /* [rows] */
    float *lse;                 /* [rows], may be NULL */
    float *entropy;             /* [rows], may be NULL */
    float *saved;               /* [rows][2], may be NULL */
} kfac_logprob_desc;

kfac_status kfac_token_logprob(const kfac_logprob_desc *desc, void *stream);

/* kfac_token_logprob_grad -- the logits' gradient from the gradients of logp
 * and (optionally) H, with the saved values and H that kfac_token_logprob gave:
 *     dlogits_j = dlogp (1[j = target] - p_j) / tau - dentropy p_j (ln p_j + H) / tau.
 * A row with dlogp = 0 (and dentropy = 0) is not read and gets zeros.  Errors:
 * as above, null saved/dlogp/dlogits, dentropy without entropy.  No workspace,
 * no error word. */
typedef struct {
    int32_t dtype;
    const void *logits; int64_t ld;
    int64_t rows; int32_t vocab;
    const void *target; int32_t target_i32;
    float temperature;
    const float *saved;         /* [rows][2] */
    const float *entropy;       /* [rows]; needed with dentropy */
    const float *dlogp;         /* [rows] */
    const float *dentropy;      /* [rows], may be NULL */
    void *dlogits; int64_t ld_d;
} kfac_logprob_grad_desc;

kfac_status kfac_token_logprob_grad(const kfac_logprob_grad_desc *desc, void *stream);

/* kfac_policy_loss -- clipped policy loss with a KL term and an entropy bonus,
 * and the gradient of its logits in the same call.  Per row that is not
 * ignored, with the advantage A, the log-probability `old` under the policy
 * that drew the token and `ref` under the reference policy:
 *     r = exp(logp - old),  c = min(max(r, 1 - clip_low), 1 + clip_high),
 *     pg = - min(r A, c A),
 *     kl = exp(ref - logp) - (ref - logp) - 1      (0 without ref_logp),
 *     l  = pg + kl_coef kl - entropy_coef H,
 *     loss = sum over rows of w l,
 *     dl / dlogp = - r A [r A <= c A] + kl_coef (1 - exp(ref - logp)),
 *     dlogits = grad_scale * dloss / dz.
 *   - w is `weight` [rows] where given (a row with w = 0 is ignored), else 1 / N, N
 *     the number of rows with a valid target; with seq_mean != 0, 1 / (seqs n_s),
 *     n_s the number of such rows of the row's sequence.
 *   - advantage is [rows], or [seqs] when seq_offsets (device int32 [seqs + 1],
 *     non-decreasing) is given: sequence s holds rows seq_offsets[s] ..
 *     seq_offsets[s + 1] - 1, and rows of no sequence are ignored.  Offsets
 *     outside 0 .. rows are read as the nearest of the two.
 *   - stats [5] receives the sums over rows of w l, w pg, w kl, w H and
 *     w [the clipped branch was taken].  H is computed when entropy_coef != 0
 *     or `entropy` is not NULL (else stats[3] = 0).
 *   - logp, kl, entropy: [rows], optional.  dlogits NULL: the loss only.
 * Error word (first int32 of the workspace): KFAC_ERRW_TARGET, 1, 2 or 4
 * (KFAC_ERRW_TIMEOUT_*: a wait on the rows kept in shared memory ran past about
 * 2 s; the outputs are then undefined), and KFAC_ERRW_NONFINITE when a counted row's logp, loss term or gradient
 * coefficient (with grad_scale / tau, where dlogits is given), or the loss, is
 * NaN or infinite (a gradient that overflows fp16 as it is rounded does not set
 * it).
 * Errors: INVALID for null logits/target/advantage/old_logp/stats, rows < 0, vocab < 1,
 *   ld or ld_d < vocab, clip_low or clip_high negative or NaN, a coefficient that is not
 *   finite, seqs < 1 with seq_offsets, seq_mean without seq_offsets or with weight,
 *   kl_coef != 0 or kl without ref_logp, a bad dtype or tau.
 * Workspace: kfac_policy_loss_workspace_size(desc) bytes. */
typedef struct {
    int32_t dtype;
    const void *logits; int64_t ld;
    int64_t rows; int32_t vocab;
    const void *target; int32_t target_i32;
    float temperature;
    const float *advantage;
    const float *old_logp;      /* [rows] */
    const float *ref_logp;      /* [rows], may be NULL */
    const float *weight;        /* [rows], may be NULL */
    const int32_t *seq_offsets; int32_t seqs; int32_t seq_mean;
    float clip_low, clip_high, kl_coef, entropy_coef, grad_scale;
    float *stats;               /* [5] */
    float *logp, *kl, *entropy; /* [rows] each, may be NULL */
    void *dlogits; int64_t ld_d;
} kfac_policy_desc;

size_t kfac_policy_loss_workspace_size(const kfac_policy_desc *desc);
kfac_status kfac_policy_loss(const kfac_policy_desc *desc, void *workspace, size_t workspace_bytes, void *stream);

/* kfac_preference_loss -- loss over pairs of sequences (paired log ratios
 * against a reference), and the gradient of its logits.  Sequence k holds rows
 * seq_offsets[k] .. seq_offsets[k + 1] - 1; sequences 2 b and 2 b + 1 are the
 * preferred and the other one of pair b.  With l_k the sum (average != 0: the
 * mean) of logp over the rows of sequence k with a valid target (0 when it
 * has none) and the reference's same quantity ref_k,
 *     h = (l_2b - ref_2b) - (l_2b+1 - ref_2b+1),
 *     KFAC_PREF_SIGMOID  f = - (1 - e) ln sigma(beta h) - e ln sigma(-beta h)
 *     KFAC_PREF_HINGE    f = max(0, 1 - beta h)
 *     KFAC_PREF_IPO      f = (h - 1 / (2 beta))^2
 *     loss = sum over pairs of v f,   dlogits = grad_scale * dloss / dz,
 * e the label_smoothing (SIGMOID only), v `pair_weight` [pairs] or 1 / pairs.
 * The sums over a sequence are formed in pairs of fp32 words, h in fp64.  Rows
 * of no sequence are ignored; offsets as in kfac_policy_loss.
 *   - ref_logp [2 pairs], may be NULL (0: no reference).
 *   - loss [1]; pair_loss [pairs] (f), seq_logp [2 pairs] (l) and
 *     token_logp [rows] are optional.  dlogits NULL: the loss only.
 * Error word: as kfac_policy_loss (logp of a counted row, l, f, the loss, and
 * where dlogits is given the gradient coefficients of sequences with counted
 * rows).
 * Errors: INVALID for null logits/target/seq_offsets/loss, rows < 0, pairs < 1,
 *   vocab < 1, ld or ld_d < vocab, an unknown kind, beta not positive and
 *   finite, label_smoothing outside [0, 1) or with another kind, a grad_scale
 *   that is not finite, a bad dtype or tau.
 * Workspace: kfac_preference_loss_workspace_size(desc) bytes. */
typedef enum { KFAC_PREF_SIGMOID = 0, KFAC_PREF_HINGE = 1, KFAC_PREF_IPO = 2 } kfac_pref_kind;

typedef struct {
    int32_t dtype;
    const void *logits; int64_t ld;
    int64_t rows; int32_t vocab;
    const void *target; int32_t target_i32;
    float temperature;
    const int32_t *seq_offsets; int32_t pairs;   /* [2 pairs + 1] */
    const float *ref_logp;
    const float *pair_weight;
    int32_t kind; int32_t average;
    float beta, label_smoothing, grad_scale;
    float *loss;
    float *pair_loss, *seq_logp, *token_logp;
    void *dlogits; int64_t ld_d;
} kfac_preference_desc;

size_t kfac_preference_loss_workspace_size(const kfac_preference_desc *desc);
kfac_status kfac_preference_loss(const kfac_preference_desc *desc, void *workspace, size_t workspace_bytes,
                                 void *stream);

/* ======================================================================
 * kfac_clip_norm -- norm over many tensors, clipping, and the weight step.
 *
 * Over all descriptors, with y = x where y is NULL,
 *     norm  = sqrt(sum x y)     (0 where the sum is negative),
 *     scale = max_norm / norm if norm > max_norm, else 1,
 *     out   = scale x                         (where out is not NULL)
 *     w    <- w - eta scale x                 (fp32, where w is not NULL).
 * With y = NULL this is clipping by the global Euclidean norm.  With x the
 * preconditioned gradients and y the gradients, sum x y = g^T F^-1 g is the
 * squared length of the natural gradient step in the Fisher metric, and
 * max_norm = sqrt(kappa) / eta bounds the step's second-order KL change by
 * kappa / 2.
 *   - x: [rows][ld] of dtype (KFAC_BF16, KFAC_F16, KFAC_F32), cols wide; a vector is
 *     one row.  y: [rows][ld_y] of y_dtype, which is dtype or, with x in fp32,
 *     any of the three (fp32 steps and the 16-bit gradients that they come
 *     from).  out: [rows][ld_out] of out_dtype; w: [rows][ld_w] fp32.
 *     Any ld >= cols and any element-aligned base.  A tensor is read 16 bytes at
 *     a time where all its operands run on without a gap (ld = cols), or where
 *     the pitches of all of them (x, y, out and w) are multiples of 8 elements;
 *     else element by element.  Dense tensors are the fastest.  rows or
 *     cols = 0: the tensor adds nothing.
 *   - out may be x itself (same dtype and ld); then nothing is rewritten when
 *     scale = 1.  Otherwise no output may overlap an input or another output.
 *   - max_norm > 0; +inf never clips.
 *   - norm [1], scale [1]: device, optional.
 * Finite inputs give the right norm as long as it fits fp32 itself: sums whose
 * fp32 squares overflow or vanish are formed again from scaled values, and
 * partial sums are added in fp64 in a fixed order (bitwise reproducible).
 * Non-finite inputs propagate as computed (an infinite norm gives scale 0, a
 * NaN norm scale NaN) and set KFAC_ERRW_NONFINITE in the error word, which a
 * caller that skips such steps reads.
 * Errors: INVALID for count < 0, null x of a tensor that is not empty, negative
 *   sizes, ld < cols, a bad dtype (or pair of them), out = x with another dtype or ld, a base that
 *   is not element-aligned, max_norm not positive or NaN, eta not finite.
 * Workspace: kfac_clip_norm_workspace_size(descs, count) bytes.
 * ==================================================================== */
typedef struct {
    const void *x; int64_t ld;
    const void *y; int64_t ld_y;       /* may be NULL */
    void *out;     int64_t ld_out;     /* may be NULL */
    float *w;      int64_t ld_w;       /* may be NULL */
    int64_t rows, cols;
    int32_t dtype, y_dtype, out_dtype;
} kfac_clip_desc;

size_t kfac_clip_norm_workspace_size(const kfac_clip_desc *descs, int count);
kfac_status kfac_clip_norm(const kfac_clip_desc *descs, int count, float max_norm, float eta, float *norm,
                           float *scale, void *workspace, size_t workspace_bytes, void *stream);

/* ======================================================================
 * Checkpoints: matrices kept in 8 bits until the backward pass.
 *
 * A layer's input a [rows][cols] is needed again for its weight gradient and for
 * its factor A.  Kept as a checkpoint it takes 1.03 bytes a value:
 *   - elements q [rows][ldq], e4m3 (1 sign, 4 exponent, 3 mantissa bits);
 *   - one exponent for every block of 32 consecutive rows of one column (rows
 *     32 t .. 32 t + 31; the last block may be shorter), a byte holding e + 127.
 *   A value is q 2^e, with e the smallest integer >= -127 for which the block's
 *   largest finite magnitude is at most 448 2^e (-127 for a block of zeros), and
 *   q = x 2^-e rounded to the nearest e4m3 (ties to even; where e = 120, at
 *   most 240).  So a value is off by at most 2^-4 of itself or 2^(e - 10),
 *   whichever is more.  An infinity or NaN is kept as NaN in its own place.
 *   - Blocks run along the rows because every use sums over rows: a block is one
 *     step of the tensor cores' block-scaled product, which takes the values
 *     exactly as they are kept.
 *   - append_one != 0: the checkpoint has one more column, all ones (exactly
 *     kept): the input [a, 1] of a layer with a bias.  Its width is then
 *     cols + 1.
 *   - scales: kfac_checkpoint_scale_bytes(rows, width) bytes.  The exponent of
 *     block t of column c is byte
 *         ((c / 128) ceil(rows / 128) + t / 4) 512 + (c mod 32) 16
 *             + (c mod 128) / 32 * 4 + t mod 4;
 *     bytes of no block are 0.
 *   - q and scales start on 16-byte boundaries and ldq is a multiple of 16 (of
 *     32 is better: a factor of 8192 x 4097 takes 95 us then, and 102 if not);
 *     elements of q past the width are not written, and what they hold does not
 *     matter.
 * ==================================================================== */

/* kfac_checkpoint_store -- checkpoints of x (KFAC_BF16, KFAC_F16 or KFAC_F32),
 * any ld >= cols and any element-aligned base.
 * kfac_checkpoint_load -- the values of checkpoints, rounded to x's type (fp32 and
 * in general bf16 hold them exactly; fp16 rounds below 2^-14, and a value above 65504 becomes
 * infinite there.  Finite fp16 values from 63488 on have such a value, 65536: a matrix that may
 * hold them is restored to bf16 or fp32).
 * One launch for each 64 matrices.  rows = 0: nothing to do.  No workspace, no
 * error word.  What a call writes must not overlap anything else that it reads or writes.
 * Errors: INVALID for count < 0, rows < 0, cols < 1, ld < cols, ldq < width,
 *   null x, q or scales of a matrix with rows, a base of x that is not
 *   element-aligned, a bad dtype; UNSUPPORTED for q, scales or ldq that are
 *   not multiples of 16 bytes, width > 2^20, more than 2^31 - 1 rows or
 *   tiles of 128 x 128. */
typedef struct {
    int32_t dtype;
    void *x; int64_t ld;          /* store: read; load: written */
    int64_t rows; int32_t cols;
    int32_t append_one;
    uint8_t *q; int64_t ldq;
    uint8_t *scales;
} kfac_checkpoint_desc;

size_t kfac_checkpoint_scale_bytes(int64_t rows, int32_t width);
kfac_status kfac_checkpoint_store(const kfac_checkpoint_desc *descs, int count, void *stream);
kfac_status kfac_checkpoint_load(const kfac_checkpoint_desc *descs, int count, void *stream);

/* kfac_weight_grad -- weight gradients of fully connected layers from checkpoints
 * of their inputs a [rows][dA] and of their output gradients g [rows][dG]:
 *     out[i][j] <- beta out[i][j] + alpha sum_m g[m][i] a[m][j]
 * with the values that the checkpoints stand for (their products are exact), fp32
 * accumulation, one rounding to out's type (KFAC_F32, KFAC_BF16 or KFAC_F16).
 * out is read only where beta != 0; rows = 0 leaves beta out.  Results are
 * bitwise reproducible run to run.  No out may overlap another one of the call (sums over
 * parts of a batch: one call for each, with beta = 1) or an input.
 * Error word (first int32 of the workspace): KFAC_ERRW_NONFINITE when a value of
 * out (before its rounding) is NaN or infinite, 1, 2, 4, 8 (KFAC_ERRW_TIMEOUT_*).
 * Errors: INVALID for count < 0, rows < 0, dA or dG < 1, ld < dA, ldq_a < dA,
 *   ldq_g < dG, null buffers (those of a and g where rows > 0), a base of out
 *   that is not element-aligned, a bad out_dtype, alpha or beta not finite;
 *   UNSUPPORTED as kfac_checkpoint_store.
 * Workspace: kfac_weight_grad_workspace_size(descs, count) bytes. */
typedef struct {
    const uint8_t *q_a; int64_t ldq_a; const uint8_t *scales_a;
    const uint8_t *q_g; int64_t ldq_g; const uint8_t *scales_g;
    int64_t rows; int32_t dA, dG;
    void *out; int64_t ld;        /* [dG][ld] */
    int32_t out_dtype;
    float alpha, beta;
} kfac_weight_grad_desc;

size_t kfac_weight_grad_workspace_size(const kfac_weight_grad_desc *descs, int count);
kfac_status kfac_weight_grad(const kfac_weight_grad_desc *descs, int count, void *workspace,
                             size_t workspace_bytes, void *stream);

/* ======================================================================
 * kfac_verify_draft -- drafted tokens accepted or replaced, so that what comes out
 * is distributed as if every token had been drawn from the policy.
 *
 * Sequence b holds rows seq_offsets[b] .. seq_offsets[b + 1] - 1 of `logits`, the
 * policy's scores at the position of each drafted token and, in the last row, at
 * the position behind them (so n rows verify n - 1 drafted tokens).  With p =
 * softmax(z / tau) of a row of logits and q = softmax(zd / tau_d) of the same row
 * of `draft`, the scores that the drafted token x was drawn from:
 *   - x is accepted if u q(x) < p(x), u = uniform[row];
 *   - at the first row whose token is not accepted, or at the last row, the
 *     sequence gets a new token, argmax_j r_j / E_j, with r = max(p - q, 0) at a
 *     token that was not accepted (p itself where that leaves nothing), r = p
 *     at the last row, and E = noise[b][j].  With E drawn from the exponential
 *     distribution that is a draw from r.  Equal quotients: the lowest j.
 * draft NULL: the token was not drawn but looked up (q is 1 at x).
 * greedy != 0: x is accepted if it is the lowest j that maximises z, and the new
 * token is that j; draft, uniform and noise are not read.
 *   - accepted [seqs] receives the number of accepted tokens, out_tokens [rows] (the
 *     type of tokens) the accepted tokens and the new one, and -1 in the rows
 *     behind it; logp [rows] (may be NULL) ln p of the token, 0 behind it.  As
 *     target and old_logp these serve kfac_policy_loss.  out_tokens may be tokens.
 *   - A sequence without rows accepts 0 tokens and writes nothing else.  Rows of
 *     no sequence are left as they were.  Offsets outside 0 .. rows are read as
 *     the nearest of the two; sequences must not share rows.
 *   - tokens int64 or (token_i32 != 0) int32; the one of a last row is not read. A
 *     token outside 0 .. vocab - 1 is not accepted, and replaced by a draw from
 *     p; one >= vocab sets KFAC_ERRW_TARGET.
 *   - p and q are formed in fp32: each is off by about 1e-6 of itself, and r by as much of the
 *     larger of the two.
 *   - Logits of -inf have probability 0.  A row of the policy with NaN, +inf or
 *     nothing but -inf has no distribution: its token is -1, its logp NaN, the sequence ends
 *     there, and KFAC_ERRW_NONFINITE is set.  A row of the draft that has none:
 *     its token is replaced by a draw from p, and the bit is set too.
 *   - draft_saved [rows][2] (may be NULL): the maximum and the sum of
 *     exp((z - m) / tau_d) of the draft's rows, as kfac_token_logprob's `saved`
 *     gives them; then the draft's rows are read only where a token is replaced.
 *   - noise [seqs][ld_noise]: positive; what is not (NaN, too) is read as 2^-126.  u is in [0, 1).
 *   - Rows of logits and draft may start at any element boundary, any ld.
 * Error word (first int32 of the workspace): the two bits named above.
 * Errors: INVALID for null seq_offsets/accepted, with rows also for null logits/tokens/
 *   out_tokens and unless greedy null uniform/noise and ld_noise < vocab (rows = 0: none
 *   of these is read); rows < 0, seqs < 1, vocab < 1, ld or ld_draft < vocab, a pointer
 *   that is not on its elements' boundary, draft_saved without draft or not on an 8-byte
 *   boundary, a bad dtype, tau or tau_d; UNSUPPORTED for vocab > 2^24, rows > 2^31 - 1,
 *   seqs > 2^20.
 * Workspace: kfac_verify_draft_workspace_size(desc) bytes. */
typedef struct {
    int32_t dtype;
    const void *logits; int64_t ld;
    int64_t rows; int32_t vocab;
    const void *tokens; int32_t token_i32;
    float temperature;
    const int32_t *seq_offsets; int32_t seqs;    /* [seqs + 1] */
    const void *draft; int64_t ld_draft;         /* dtype; may be NULL */
    const float *draft_saved;                    /* [rows][2], may be NULL */
    float draft_temperature;
    const float *uniform;                        /* [rows] */
    const float *noise; int64_t ld_noise;
    int32_t greedy;
    int32_t *accepted;                           /* [seqs] */
    void *out_tokens;                            /* [rows] */
    float *logp;                                 /* [rows], may be NULL */
} kfac_verify_desc;

size_t kfac_verify_draft_workspace_size(const kfac_verify_desc *desc);
kfac_status kfac_verify_draft(const kfac_verify_desc *desc, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* KFAC_GB300_H */
