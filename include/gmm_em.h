/*
 * gmm_em.h - C ABI of the fused diagonal-covariance GMM EM library for
 * AMD Instinct MI355X (gfx950).
 *
 * The method is one expectation-maximization (EM) iteration of a Gaussian
 * mixture with diagonal covariances, fused so that the N x K responsibility
 * matrix is never written to device memory: statistics are formed per data
 * tile and accumulated globally into O(K*D) buffers ("Flash-GMM: A
 * Memory-Efficient Kernel for Scalable Soft Clustering", section 1 for the
 * responsibility matrix, section 3 for the tiled EM with globally accumulated
 * per-tile statistics; the abstract for the use of responsibilities to assign
 * border vectors to several clusters).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Data X: device pointer, row-major, n rows of d values with a leading
 *   dimension ldx >= d (in elements, at most 2^24 - 1: GMM_E_UNSUPPORTED
 *   above), fp32 or bf16 (x_dtype). Values between d and ldx are never
 *   used (they may be read, never past the last row's d-th value).
 * Parameters: device pointers, fp32, row-major:
 *   weights[k] (mixture weights, >= 0, not all 0),
 *   means[k*d], variances[k*d] (> 0).
 * Workspace: a device buffer of at least gmm_workspace_bytes(d, k) bytes,
 *   owned by the caller. Its size does not depend on n. Calls that share a
 *   workspace must not overlap in time (use one stream, or separate
 *   workspaces).
 * Stream: a hipStream_t passed as void* (NULL = the null stream). All work is
 *   enqueued asynchronously on it; results are valid once the stream has
 *   reached them. Nothing synchronises except gmm_device_status and
 *   gmm_fit with tol > 0.
 * Errors: every function returns a gmm_status. Argument errors found on the
 *   host are returned before anything is enqueued (buffers are untouched).
 *   Invalid parameter values (non-finite, variance <= 0, negative weight,
 *   all weights zero) are detected on the device: the call still returns
 *   GMM_OK, outputs are NaN, and gmm_device_status reports GMM_E_PARAMS.
 *   No function throws or aborts.
 * Determinism: for a given device, inputs and (d, k) every output is
 *   bitwise reproducible; no floating-point atomics are used.
 * Ownership: the library allocates no device memory and keeps no state
 *   between calls besides cached device properties.
 */
#ifndef GMM_EM_H
#define GMM_EM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GMM_OK = 0,
    GMM_E_INVALID = 1,   /* bad size, pointer, stride or option */
    GMM_E_DTYPE = 2,     /* unsupported data type */
    GMM_E_WORKSPACE = 3, /* workspace missing or too small */
    GMM_E_PARAMS = 4,    /* invalid parameter values (reported by gmm_device_status) */
    GMM_E_HIP = 5,       /* a HIP runtime call failed */
    GMM_E_UNSUPPORTED = 6  /* shape outside what this build supports */
} gmm_status;

typedef enum { GMM_F32 = 0, GMM_BF16 = 1 } gmm_dtype;

/* Arithmetic of the E-step and M-step contractions (see gmm_estep_arithmetic). */
typedef enum {
    GMM_ESTEP_FP64 = 0,              /* both passes' E-step in fp64 */
    GMM_ESTEP_INT8_SLICES = 1,       /* normaliser pass on int8 slices, statistics pass fp64 */
    GMM_ESTEP_INT8_SLICES_BOTH = 2,  /* both passes' E-step on int8 slices, M-step fp64 */
    GMM_ESTEP_INT8_SLICES_MSTEP = 3, /* as 2, and the M-step on int8 slices too */
    GMM_ESTEP_BF16_SPLIT = 4         /* bf16 data: E-step and M-step on split bf16 */
} gmm_estep_kind;

/* Bytes of device workspace needed for data of dimension d and k components.
 * Independent of the number of rows. Returns 0 for unsupported shapes:
 * d <= 768 and k <= 2^22 are supported (d <= 128 uses register-tiled
 * kernels; wider rows use kernels that split the dimension over the waves of
 * a workgroup and process rows in chunks of 4096). */
size_t gmm_workspace_bytes(int32_t d, int32_t k);

/* One EM iteration (E-step, responsibilities, M-step) in place.
 *
 * Computes, for the input parameters theta = (weights, means, variances):
 *   l[n][k]  = log w[k] + log N(x_n | mu_k, diag(var_k))      (log-density)
 *   lse[n]   = log sum_k exp(l[n][k])                          (normaliser)
 *   r[n][k]  = exp(l[n][k] - lse[n])                          (responsibility)
 *   N[k] = sum_n r[n][k], S1[k] = sum_n r[n][k] x_n, S2 = sum_n r[n][k] x_n^2
 * and overwrites theta with the M-step update
 *   w'[k] = N[k]/n, mu'[k] = S1[k]/N[k], var'[k] = max(S2[k]/N[k] - mu'[k]^2, var_floor)
 * (a component with N[k] == 0 keeps its mean and variance and gets weight 0).
 * r is never stored: it lives in registers between the two contractions.
 * Schedule: two passes over the rows (normalisers, then statistics); the
 * second recomputes the log-densities instead of storing them.
 * Arithmetic: the E-step contraction sum_d (w b a - w a^2 / 2) (a = x - s,
 * b = mu - s, w = 1/var, s a per-dimension shift) runs either in fp64 or
 * exactly on int8 slices (the features and coefficients written as 7-bit
 * digits with power-of-two scales; integer products and sums are exact and
 * the digit levels are added in fp64), which differs from the fp64
 * contraction by at most 2^-20 nats per log-density plus fp64 rounding. The
 * call picks the int8 form on the device whenever its error bound holds for
 * the data and parameters at hand (always, for integer-valued data within
 * the supported range); gmm_estep_arithmetic reports which one ran. When
 * both passes use it they compute bitwise identical log-densities. The M-step
 * contraction is fp64, except where every feature is exact in its digits
 * (integer-valued data, or data on a grid of 2^-m, within the range): then
 * it runs on int8 slices as well, on responsibilities cut per 64-row block
 * and component to 42 bits below the block's largest one (fp32 precision
 * for every row within 2^-18 of it); N[k], S1[k] and S2[k] are then exact for
 * those weights up to fp64 rounding, so the variance keeps full accuracy.
 * Responsibilities keep the fp64 exponent range: a component whose
 * responsibilities are all below fp32's smallest value but above fp64's
 * still gets a nonzero N[k].
 * bf16 data (d <= 128) that the int8 form does not cover runs both passes on
 * the bf16 matrix units instead when its checks hold: a = x - s exact in
 * bf16, and 2^-23 * max_k sum_d (|w/2| amax_d^2 + |w b| amax_d) <= 2^-7
 * (amax_d the largest |a| in dimension d). Features [a^2 hi, a^2 lo, a] are
 * exact in bf16, coefficients are split in three bf16 parts, each 32-dim
 * slice accumulates in fp32 and the slices add in fp64: the log-densities
 * differ from the fp64 contraction by about 2^-24 of the slices' magnitude
 * (that estimate is what the check bounds). The M-step contracts fp32
 * responsibilities (exact as three bf16 parts; those below 2^-100 count as
 * 0) in fp32 per 32-row tile and fp64 across tiles.
 * loglik_dev (device, 1 double, may be NULL) receives sum_n lse[n] for the
 * INPUT parameters. var_floor must be finite and >= 0. n >= 1. */
int gmm_em_step(const void* x, int64_t n, int32_t d, int64_t ldx, int32_t x_dtype,
                float* weights, float* means, float* variances, int32_t k, float var_floor,
                double* loglik_dev, void* workspace, size_t workspace_bytes, void* stream);

/* gmm_em_step for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * the same EM step with the same arguments and results, but no workspace
 * argument. It uses a device array of 128 MiB that the library holds in its
 * code object (one copy per GPU, kept until the process ends); the call
 * itself allocates nothing. The array is shared by every call on a GPU:
 * calls that overlap in time on one GPU (several streams or host threads)
 * race and give undefined results. It holds no state that a call depends on
 * (each call rewrites what it reads). Shapes whose workspace does not fit
 * 128 MiB (with its 262,144-row chunks and the statistics pass's row groups
 * reduced to fit) return GMM_E_UNSUPPORTED: d = 96 with k = 1024 fits, d = 768
 * with k = 16384 does not. The reduction order differs from gmm_em_step's,
 * so results agree to rounding, not bitwise. */
int gmm_em_step_noalloc(const void* x, int64_t n, int32_t d, int64_t ldx, int32_t x_dtype,
                        float* weights, float* means, float* variances, int32_t k,
                        float var_floor, double* loglik_dev, void* stream);

/* max_iter EM iterations (gmm_em_step repeated). loglik_hist_dev (device,
 * max_iter doubles, may be NULL) receives L(theta_t) for t = 0, 1, ...
 * When tol > 0 the host reads each L after its step (one synchronisation per
 * iteration) and stops once L_t - L_{t-1} < tol * |L_t|. iters_done (host
 * pointer, may be NULL) receives the number of steps taken. */
int gmm_fit(const void* x, int64_t n, int32_t d, int64_t ldx, int32_t x_dtype,
            float* weights, float* means, float* variances, int32_t k, float var_floor,
            int32_t max_iter, double tol, double* loglik_hist_dev, int32_t* iters_done,
            void* workspace, size_t workspace_bytes, void* stream);

/* Log-likelihood of the data under the parameters (the E-step half only).
 * total_dev (device, 1 double) receives sum_n lse[n]; per_row_dev (device,
 * n doubles, may be NULL) receives lse[n]. n may be 0 (total = 0). */
int gmm_loglik(const void* x, int64_t n, int32_t d, int64_t ldx, int32_t x_dtype,
               const float* weights, const float* means, const float* variances, int32_t k,
               double* total_dev, double* per_row_dev, void* workspace, size_t workspace_bytes,
               void* stream);

/* Soft multi-assignment: the m components of highest responsibility for each
 * row, most responsible first (ties: smaller component index first), with
 * their responsibilities r[n][k]. idx_dev (device, n*m int32) and resp_dev
 * (device, n*m floats) are row-major n x m. 1 <= m <= min(k, 4). n may be 0.
 * The log-densities run on int8 slices for fp32 rows where gmm_em_step's
 * conditions for them hold, else in fp64 (bf16 rows: fp64).
 * Parameter errors are reported by gmm_device_status; the outputs are then
 * unspecified. */
int gmm_assign_topm(const void* x, int64_t n, int32_t d, int64_t ldx, int32_t x_dtype,
                    const float* weights, const float* means, const float* variances, int32_t k,
                    int32_t m, int32_t* idx_dev, float* resp_dev, void* workspace,
                    size_t workspace_bytes, void* stream);

/* One Lloyd (k-means) step, the hard-assignment quantizer that the Flash-GMM
 * pages compare the GMM against in the IVF coarse quantizer ("Flash-GMM: A
 * Memory-Efficient Kernel for Scalable Soft Clustering", section 3). It is
 * the EM step's limit for equal weights and equal spherical variances
 * shrinking to zero, and runs on the same two passes:
 *   z[n]  = argmin_k |x_n - c_k|^2       (ties: smaller k)
 *   c'_k  = mean of the rows with z = k  (c_k kept when no row has z = k)
 * centroids (device, k x d floats, row-major) is read and overwritten with c'.
 * assign_dev (device, n int32, may be NULL) receives z. inertia_dev (device,
 * 1 double, may be NULL) receives sum_n |x_n - c_z[n]|^2 for the INPUT
 * centroids. The distances use the expanded form 2 a.b - a.a - b.b about a
 * per-dimension shift, in fp64 or, where the data and centroids allow it (as
 * for gmm_em_step: the int8 slices' error bound holds), on exact int8 slices
 * (exact up to fp64 rounding either way), so rows whose two nearest
 * centroids are within rounding of each other may be assigned either one.
 * The workspace is the one for (d, k). n >= 1; d <= 768 (GMM_E_UNSUPPORTED
 * otherwise). A non-finite centroid is reported by gmm_device_status and
 * turns the outputs into NaN. */
int gmm_kmeans_step(const void* x, int64_t n, int32_t d, int64_t ldx, int32_t x_dtype,
                    float* centroids, int32_t k, int32_t* assign_dev, double* inertia_dev,
                    void* workspace, size_t workspace_bytes, void* stream);

/* Inverted lists of an IVF coarse quantizer from top-m soft assignments: the
 * GMM responsibilities put border vectors in several lists ("Flash-GMM: A
 * Memory-Efficient Kernel for Scalable Soft Clustering", abstract; the
 * review page, section 1, for the IVF index). idx_dev and resp_dev (device,
 * n*m int32 and floats, row-major n x m, most responsible first, as
 * gmm_assign_topm writes them). Row r goes to list idx[r][0] and, for
 * j >= 1, to list idx[r][j] when resp[r][j] >= min_resp; ids outside [0, k)
 * are skipped. resp_dev may be NULL: then every entry is kept and the
 * stored values are 1. Output (device): offsets_dev (k+1 int64; list c is
 * entries offsets[c] .. offsets[c+1]-1, offsets[k] = entries stored),
 * rows_dev (int32 row ids, capacity n*m; each list in increasing row order)
 * and values_dev (the entries' responsibilities, capacity n*m, may be NULL).
 * The result does not depend on scheduling (a stable counting sort).
 * 1 <= k <= 16384 and n*m < 2^31 (GMM_E_UNSUPPORTED otherwise); min_resp
 * must not be NaN. The workspace (device, 256-byte aligned) has
 * gmm_ivf_workspace_bytes(n, m, k) bytes; it depends on n. */
size_t gmm_ivf_workspace_bytes(int64_t n, int32_t m, int32_t k);
int gmm_ivf_build(const int32_t* idx_dev, const float* resp_dev, int64_t n, int32_t m, int32_t k,
                  float min_resp, int64_t* offsets_dev, int32_t* rows_dev, float* values_dev,
                  void* workspace, size_t workspace_bytes, void* stream);

/* max_iter Lloyd steps (gmm_kmeans_step repeated) on the centroids in place.
 * inertia_hist_dev (device, max_iter doubles, may be NULL) receives the
 * inertia of the centroids entering step t, t = 0, 1, ... When tol > 0 the
 * host reads each inertia after its step (one synchronisation per step) and
 * stops once I_{t-1} - I_t < tol * I_t. iters_done (host pointer, may be
 * NULL) receives the number of steps taken. */
int gmm_kmeans_fit(const void* x, int64_t n, int32_t d, int64_t ldx, int32_t x_dtype,
                   float* centroids, int32_t k, int32_t max_iter, double tol,
                   double* inertia_hist_dev, int32_t* iters_done, void* workspace,
                   size_t workspace_bytes, void* stream);

/* Scores of given codes under a softmax over v codes, from its logits.
 * The log-likelihood of a learned softmax over components in place of a
 * mixture's: with l = scale * x (rounded to fp32) for row x of the logits,
 *   norm[2r], norm[2r+1] = max l, log sum exp(l - max l)
 *   logprob[r]  = l[t] - norm[2r] - norm[2r+1]        for t = targets[r]
 *   entropy[r]  = -sum p log p                         with p = softmax(l)
 *   top_idx[r][j], top_logprob[r][j], j < m: the m most probable codes, most
 *     probable first (ties: smaller index first), and their log p.
 * logits (device): n rows of v values with leading dimension ldl >= v (in
 * elements; any alignment of an element), fp32 or bf16; offsets are 64-bit.
 * targets (device, n int32, may be NULL: then logprob is not used): a
 * negative target gives no code, its logprob is 0; one of v or more gives
 * NaN. scale (an inverse temperature) must be finite and > 0. entropy (n floats)
 * and norm (2n floats) may be NULL. 0 <= m <= min(v, GMM_TOP_MAX); top_idx and
 * top_logprob (n*m, row-major) are unused when m = 0, and top_idx with the
 * exponentials of top_logprob is what gmm_ivf_build reads.
 * Masks: a logit of -inf (or one whose l is) has probability 0 and is never an
 * alternative: places left over hold -1 and -inf. A row with nothing left has
 * norm (-inf, 0), entropy 0 and logprob -inf. A row with a NaN or +inf (or one
 * whose l is) has NaN in logprob, entropy and norm; NaN is never an alternative.
 * Rows whose largest l is the lowest finite value are ordinary rows.
 * Sums are fp32 in a fixed order (bitwise reproducible). n may be 0; n <= 2^40,
 * v <= 2^30. The workspace (device, 256-byte aligned) has
 * gmm_logits_score_workspace_bytes(n, v, m) bytes (0: invalid sizes). */
#define GMM_TOP_MAX 16
size_t gmm_logits_score_workspace_bytes(int64_t n, int32_t v, int32_t m);
int gmm_logits_score(const void* logits, int64_t n, int32_t v, int64_t ldl, int32_t dtype,
                     const int32_t* targets, int32_t m, float scale, float* logprob,
                     float* entropy, float* norm, int32_t* top_idx, float* top_logprob,
                     void* workspace, size_t workspace_bytes, void* stream);

/* Gradient of gmm_logits_score's logprob and entropy with respect to the
 * logits: for the gradients g_logprob and g_entropy (device, n floats each; each
 * may be NULL: 0) that arrive at them,
 *   dlogits[r][v] = scale * (g_logprob ([v = t] - p) - g_entropy p (log p + entropy))
 * norm and entropy are what gmm_logits_score wrote for the same logits, targets
 * and scale; targets may be NULL without g_logprob, entropy without g_entropy.
 * dlogits (device, type of the logits, leading dimension lddl >= v) may be the
 * logits themselves with the same leading dimension. Rows with nothing left get
 * 0, rows without a target 0 from g_logprob, rows with a target of v or more or
 * a NaN get NaN. Needs no workspace. */
int gmm_logits_score_backward(const void* logits, int64_t n, int32_t v, int64_t ldl, int32_t dtype,
                              const int32_t* targets, const float* norm, const float* entropy,
                              const float* g_logprob, const float* g_entropy, float scale,
                              void* dlogits, int64_t lddl, void* stream);

/* gmm_logits_score fused with the product that makes the logits: x = h W^T for
 * n rows h of d values (hidden, leading dimension ldh >= d) and the codes' v rows
 * of d values (weight, ldw >= d), both fp32 or both bf16 (device, any alignment
 * of an element). targets, m, scale and the outputs are gmm_logits_score's; the
 * n x v matrix of logits is not formed when m = 0, and a chunk of rows at a
 * time lies in the workspace as fp32 when m > 0. bf16 products are exact and
 * added in fp32; fp32 operands are cut into three bf16 planes and multiplied to
 * 2^-24 of each product, so both types give fp32 logits. A logit of -inf (of a
 * bf16 weight of -inf, or of a product beyond fp32) is a masked code, one of +inf or
 * NaN gives its row NaN; an infinity in an fp32 operand counts as NaN, and a product of
 * fp32 operands beyond 2^135 may. 1 <= d <= 2^20, v <= 2^22 (GMM_E_UNSUPPORTED beyond). The workspace (device, 256-byte aligned)
 * has gmm_head_score_workspace_bytes bytes (0: invalid or unsupported sizes); it
 * is bounded in n. Rows of bf16 that are 16-byte aligned with d a multiple of 64
 * are read in place, others are laid out in the workspace first. */
size_t gmm_head_score_workspace_bytes(int64_t n, int32_t d, int32_t v, int32_t dtype, int32_t m);
int gmm_head_score(const void* hidden, int64_t n, int32_t d, int64_t ldh, const void* weight,
                   int32_t v, int64_t ldw, int32_t dtype, const int32_t* targets, int32_t m,
                   float scale, float* logprob, float* entropy, float* norm, int32_t* top_idx,
                   float* top_logprob, void* workspace, size_t workspace_bytes, void* stream);

/* Gradient of gmm_head_score's logprob and entropy with respect to hidden and
 * weight: with dx of gmm_logits_score_backward for the same arguments,
 *   d_hidden = dx W (n x d),   d_weight = dx^T h (v x d),
 * in the operands' type, rounded once from fp32 sums (leading dimensions lddh,
 * lddw >= d). Either may be NULL (not computed), not both. They must not overlap
 * hidden or weight. dx is computed a chunk of rows at a time into the
 * workspace: exactly for fp32 operands. For bf16 the two products have fp16 operands,
 * each multiplied by a power of two that is taken out of the sums again: dx by one for
 * each row, W by one for each dim, and for d_weight h by one for each dim after its rows
 * are divided by dx's. They have 11 significant bits (all of W's and h's 8) down to
 * 2^-29 of the most that a row's dx can reach, of a dim's largest |W| and of a dim's
 * largest |h| times what its row's dx can reach, and nothing below 2^-39 of it. Rows
 * without a gradient add 0 whatever finite values they hold; an infinity or NaN in W or
 * h gives NaN in its dim of d_hidden or d_weight.
 * n = 0 sets d_weight to 0. Sizes as for gmm_head_score; the workspace grows with n by 4
 * bytes a row for bf16. */
size_t gmm_head_score_backward_workspace_bytes(int64_t n, int32_t d, int32_t v, int32_t dtype);
int gmm_head_score_backward(const void* hidden, int64_t n, int32_t d, int64_t ldh,
                            const void* weight, int32_t v, int64_t ldw, int32_t dtype,
                            const int32_t* targets, const float* norm, const float* entropy,
                            const float* g_logprob, const float* g_entropy, float scale,
                            void* d_hidden, int64_t lddh, void* d_weight, int64_t lddw,
                            void* workspace, size_t workspace_bytes, void* stream);

/* A mixture-of-experts layer for a few rows. For row x of n rows of d values
 * (leading dimension ldx >= d), with e experts of f features:
 *   z = x G^T (gate: e x d, row-major); the m experts of largest z, largest
 *   first (ties: smaller index first; NaN ranks last), go to idx[r][0..m) and
 *   their shares to resp[r][0..m): the softmax of z over the picked experts, or
 *   over all experts when share_all is not 0;
 *   y = sum_j resp[r][j] W_out[c] (silu(W_a[c] x) * (W_b[c] x)),  c = idx[r][j].
 * w_in (e x 2f x d, row-major) holds f rows W_a and then f rows W_b for each
 * expert, w_out (e x d x f) the rows W_out. gate may be NULL: then idx and resp
 * (device, n*m, as gmm_assign_topm writes them: a mixture as the router) are
 * read instead of written; picks outside [0, e) are skipped, an expert picked
 * twice by a row counts twice. x, gate, weights and y (leading dimension
 * ldy >= d) are all fp32 or all bf16, at any alignment of an element. y must
 * not overlap x.
 * Products of bf16 are exact; every sum is fp32 in a fixed order (bitwise
 * reproducible); the features between the two products keep 16 significant bits
 * for bf16 data and 24 for fp32; y is rounded once. Each expert's weights are
 * read once for every 64 rows that picked it, unpicked experts' not at all; with
 * many rows per expert the layer is bound by its products instead.
 * 1 <= m <= min(e, GMM_TOP_MAX); n may be 0; e <= 4096, n*m <= 2^20, d and f <= 2^20
 * (GMM_E_UNSUPPORTED beyond). The workspace (device, 256-byte aligned) has
 * gmm_moe_layer_workspace_bytes bytes (0: invalid or unsupported sizes). */
size_t gmm_moe_layer_workspace_bytes(int64_t n, int32_t d, int32_t f, int32_t e, int32_t dtype,
                                     int32_t m);
int gmm_moe_layer(const void* x, int64_t n, int32_t d, int64_t ldx, const void* gate, int32_t e,
                  const void* w_in, const void* w_out, int32_t f, int32_t dtype, int32_t m,
                  int32_t share_all, int32_t* idx, float* resp, void* y, int64_t ldy,
                  void* workspace, size_t workspace_bytes, void* stream);

/* Embedding of codes: out[r] = scale * table[codes[r]], rounded once to the table's type. The
 * input end of a model over codes, as gmm_head_score is its output end. table (device): v rows of d
 * values with leading dimension ldt >= d, fp32 or bf16; codes (device, n int32): a negative one is
 * no code and gives a row of 0, one of v or more a row of NaN. out (n x d, type of the table, leading
 * dimension ldo >= d) must not overlap the table. Any alignment of an element; offsets are 64-bit.
 * scale must be finite. n may be 0; n <= 2^40, d <= 2^20, v <= 2^22 (GMM_E_UNSUPPORTED beyond
 * for d and v). Needs no workspace. */
int gmm_embed(const void* table, int32_t v, int32_t d, int64_t ldt, int32_t dtype,
              const int32_t* codes, int64_t n, float scale, void* out, int64_t ldo, void* stream);

/* Gradient of gmm_embed with respect to its table: for the gradient grad (device, n x d, leading
 * dimension ldg >= d) that arrives at out,
 *   d_table[c] = scale * sum of grad[r] over the rows r with codes[r] = c
 * in grad's type, rounded once from fp32 sums; a code that no row has gets 0, rows whose code is
 * not in [0, v) add nothing. The rows are sorted by code, so every sum has one order (bitwise
 * reproducible) and the work is cut evenly however often a code occurs. d_table (v x d, leading
 * dimension ldt >= d) must not overlap grad. n = 0 sets d_table to 0. n < 2^31, d and v as for
 * gmm_embed (GMM_E_UNSUPPORTED beyond). The workspace (device, 256-byte aligned) has
 * gmm_embed_backward_workspace_bytes(n, d, v) bytes (0: invalid or unsupported sizes). */
size_t gmm_embed_backward_workspace_bytes(int64_t n, int32_t d, int32_t v);
int gmm_embed_backward(const void* grad, int64_t n, int32_t d, int64_t ldg, int32_t dtype,
                       const int32_t* codes, int32_t v, float scale, void* d_table, int64_t ldt,
                       void* workspace, size_t workspace_bytes, void* stream);

/* Rows in 8-bit integers: for each row of x (device, n rows of d values, leading dimension
 * ldx >= d, fp32 or bf16)
 *   scale[r] = max |x_r| / 127 (rounded to fp32),  q[r][k] = the integer nearest x_r[k] / scale[r]
 * (ties to the even one, within +-127). A row of zeros (or one whose scale is below fp32's smallest
 * value) has scale 0 and q 0; a row with an infinity or NaN has scale NaN and q 0, so that its
 * products are NaN. q: n x d with leading dimension ldq >= d (values between d and ldq are left as
 * they are). n may be 0; n <= 2^40, d < 2^17 (GMM_E_UNSUPPORTED beyond). Needs no workspace. */
int gmm_quantize_rows(const void* x, int64_t n, int32_t d, int64_t ldx, int32_t dtype, int8_t* q,
                      int64_t ldq, float* scale, void* stream);

/* Product of rows in 8-bit integers with a scale for each row and each code (or output channel):
 *   y[r][c] = (sum_k q[r][k] w[c][k]) * q_scale[r] * w_scale[c]
 * q: n x d (leading dimension ldq >= d), w: v x d (ldw >= d), as gmm_quantize_rows writes them (all
 * 256 values are allowed); q_scale n floats, w_scale v floats. The sums are exact; the sum, its
 * product with q_scale and then with w_scale are rounded to fp32 and y (n x v, ldy >= v) to dtype
 * (fp32 or bf16). y must not overlap the operands. With w the codes' quantised rows this is the
 * head's logits in 8 bits, read by gmm_logits_score and gmm_beam_step. Any alignment; offsets are
 * 64-bit. n may be 0; n <= 2^40, d < 2^17, v <= 2^22 (GMM_E_UNSUPPORTED beyond). The workspace
 * (device, 256-byte aligned) has gmm_quantized_product_workspace_bytes bytes, enough for any operands,
 * or gmm_quantized_product_call_workspace_bytes bytes, what these operands need (nothing for those that
 * are read in place); 0: invalid or unsupported sizes. Both are bounded in n. Operands that are 16-byte
 * aligned with a leading dimension that is a multiple of 16 and d a multiple of 128 are read in place;
 * others too where few rows or codes make that faster, and are laid out in the workspace first where
 * it is not. Rows that are not 4-byte aligned are read by the aligned words that hold their bytes. */
size_t gmm_quantized_product_workspace_bytes(int64_t n, int32_t d, int32_t v);
size_t gmm_quantized_product_call_workspace_bytes(const int8_t* q, int64_t n, int32_t d, int64_t ldq,
                                                  const int8_t* w, int32_t v, int64_t ldw);
int gmm_quantized_product(const int8_t* q, int64_t n, int32_t d, int64_t ldq, const float* q_scale,
                          const int8_t* w, int32_t v, int64_t ldw, const float* w_scale, void* y,
                          int64_t ldy, int32_t dtype, void* workspace, size_t workspace_bytes,
                          void* stream);

/* A step of beam search over the logits of b searches with w beams each (device, b w rows of v
 * values, leading dimension ldl >= v, fp32 or bf16; row s w + k is beam k of search s). With
 * l = scale * x as in gmm_logits_score, the continuations of a search are
 *   score(k, c) = scores[s][k] + ((l_c - max l) - log sum exp(l - max l))
 * and the m best, best first, go to parent[s][j] = k, code[s][j] = c and score[s][j] (b x m each).
 * Equal scores: the smaller k first, then the larger l, then the smaller c. A beam whose last code
 * (last, b x w int32, may be NULL) equals end >= 0 has ended: its one continuation is itself, with
 * code end and its score unchanged. A beam whose score is not finite is dead and has none; the
 * rows of ended and dead beams are not read. A code whose logit is -inf or NaN, or whose score is -inf
 * or NaN (every code of a row with a NaN or +inf), is no continuation; places left over hold
 * -1, -1 and -inf. 1 <= w, m <= GMM_TOP_MAX, which may differ (a first step has w = 1); v <= 2^30.
 * b may be 0. parent, code and score must not overlap scores and last. The workspace (device,
 * 256-byte aligned) has gmm_beam_step_workspace_bytes bytes (0: invalid sizes). */
size_t gmm_beam_step_workspace_bytes(int64_t b, int32_t w, int32_t v, int32_t m);
int gmm_beam_step(const void* logits, int64_t b, int32_t w, int32_t v, int64_t ldl, int32_t dtype,
                  const float* scores, const int32_t* last, int32_t end, int32_t m, float scale,
                  int32_t* parent, int32_t* code, float* score, void* workspace,
                  size_t workspace_bytes, void* stream);

/* Moves the states that belong to beams after gmm_beam_step: for o < outer (layers, for example),
 *   out[o][s m + j] = state[o][s w + parent[s][j]]      (0 where parent is not in [0, w))
 * with rows of row_bytes bytes (of any type and alignment), strides in bytes: out's rows must not
 * overlap, state's may be the same row (stride 0). out may be state itself (w = m, the same
 * strides): then rows that stay are not touched and each other one is read and written once; else it
 * must not overlap state. parent: b x m int32. outer and b may be 0. */
int gmm_beam_reorder(const void* state, int64_t outer, int64_t stride_outer, int64_t b, int32_t w,
                     int64_t stride_row, int64_t row_bytes, const int32_t* parent, int32_t m,
                     void* out, int64_t out_stride_outer, int64_t out_stride_row, void* stream);

/* Balance of a router over e experts (or of the codes of an assignment over their lists). For gate
 * logits (device, n rows of e values, leading dimension ldz >= e, fp32 or bf16), p = softmax of a
 * row, and picks idx (n x m int32, as gmm_moe_layer and gmm_assign_topm write them):
 *   counts[c] = picks of c,  totals[0] = rows with a pick,  totals[1] = picks
 *   prob[c] = the mean of p_c over the rows with a pick
 *   loss = e * sum_c counts[c] / totals[1] * prob[c]        (1 when balanced)
 * Picks outside [0, e) are none; a row without a pick (padding) is left out altogether. No such row:
 * loss and prob 0. norm[r] = (max z, log sum exp(z - max z)) for the gradient: (+inf, 0) for a row
 * left out, (-inf, 0) for a row whose logits are all -inf (its p counts as 0), NaN for a row with a
 * NaN or +inf, which makes loss and prob NaN. Sums are fp32 in a fixed order (bitwise reproducible).
 * 1 <= m <= GMM_TOP_MAX; n may be 0; e <= 4096 and n m < 2^31 (GMM_E_UNSUPPORTED beyond). The
 * workspace (device, 256-byte aligned) has gmm_balance_loss_workspace_bytes bytes (0: invalid
 * or unsupported sizes). */
size_t gmm_balance_loss_workspace_bytes(int64_t n, int32_t e, int32_t m);
int gmm_balance_loss(const void* logits, int64_t n, int32_t e, int64_t ldz, int32_t dtype,
                     const int32_t* idx, int32_t m, float* loss, int32_t* counts, int64_t* totals,
                     float* prob, float* norm, void* workspace, size_t workspace_bytes, void* stream);

/* Gradient of gmm_balance_loss's loss with respect to the logits (counts have none), in their type:
 *   dlogits[r][c] = g e / totals[0] * p_c (f_c - sum_c' f_c' p_c'),  f_c = counts[c] / totals[1]
 * counts, totals and norm are what gmm_balance_loss wrote; g_loss (device, 1 float, may be NULL: 1)
 * is the gradient that arrives at loss. Rows left out or with no logit above -inf get 0, rows with
 * a NaN or +inf NaN. dlogits (leading dimension lddz >= e) may be the logits themselves with the same
 * leading dimension. Needs no workspace. */
int gmm_balance_loss_backward(const void* logits, int64_t n, int32_t e, int64_t ldz, int32_t dtype,
                              const int32_t* counts, const int64_t* totals, const float* norm,
                              const float* g_loss, void* dlogits, int64_t lddz, void* stream);

/* Synchronises the stream and returns GMM_E_PARAMS if the last call that used
 * this workspace found invalid parameter values, GMM_OK otherwise, or
 * GMM_E_HIP if the synchronisation failed. */
int gmm_device_status(const void* workspace, void* stream);

/* Synchronises the stream and returns the gmm_estep_kind of the last call
 * that used this workspace: of the E-step of gmm_em_step / gmm_fit /
 * gmm_loglik, of the distance pass of gmm_kmeans_step / gmm_kmeans_fit, or of
 * the log-densities of gmm_assign_topm (the last two report
 * GMM_ESTEP_INT8_SLICES when they ran on int8 slices, else GMM_ESTEP_FP64;
 * rows wider than 128 always run in fp64), or -1 if the workspace is NULL or
 * the synchronisation failed. */
int gmm_estep_arithmetic(const void* workspace, void* stream);

/* Static description of a status code. */
const char* gmm_status_string(int status);

/* Measurement hook (not part of the method). gmm_profile_begin(max_launches)
 * creates 4 * max_launches HIP events (host objects; no device memory) and
 * starts recording them on the calling entry point's stream around every
 * normaliser-pass (pass 1) and statistics-pass (pass 2) launch of the calls
 * that follow, up to max_launches of each. gmm_profile_end() synchronises
 * those events, returns the summed milliseconds and launch counts of each
 * pass, stops recording and destroys the events (GMM_E_INVALID if no
 * recording is active). This recording is the library's only process-wide
 * state: it is guarded by a mutex, but it is outside the re-entrancy promise
 * above (calls on several streams between begin and end are all recorded
 * into the same totals). Meant for benchmarks. */
int gmm_profile_begin(int32_t max_launches);
int gmm_profile_end(double* ms_pass1, int32_t* launches_pass1, double* ms_pass2,
                    int32_t* launches_pass2);

/* Library version as major*10000 + minor*100 + patch. */
int32_t gmm_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GMM_EM_H */
