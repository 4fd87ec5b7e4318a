/*
 * cat.h — C ABI of the GB300 CAT library (libcat.so): the forward pass, its
 * backward pass, and the 2-D (BCCB) circulant attention of a second page.
 *
 * CAT (circular-convolutional attention), as defined on the notes page
 * "CAT: Circular-Convolutional Attention for Sub-Quadratic Transformers",
 * section 方法详解 (method):
 *   - 整体框架 (overall framework): CAT replaces multi-head self-attention;
 *     its parameters are W_A (attention projection, one column per head) and
 *     W_V (value projection).  V = X·W_V is an INPUT here: the value
 *     projection is an ordinary dense GEMM and is not part of this library.
 *   - 关键设计, "circulant attention matrix construction": per head h,
 *     Z = X·W_A[:, h], Z* = softmax over the N tokens, and circ(Z*) is the
 *     N x N circulant whose rows are successive cyclic shifts.
 *   - 关键设计, "FFT acceleration": circ(Z*)·V = IFFT(FFT(Z*) ⊙ FFT(V)),
 *     exact, O(N log N); this orientation gives circ(Z*)[i,j] = Z*[(i-j) mod N].
 *
 * Data layout (all dense, row-major, caller-owned device memory unless a
 * function says otherwise):
 *   X   [B, N, D]   tokens
 *   W_A [D, H]      one score column per head
 *   V   [B, N, D]   projected values; head h owns columns [h·D/H, (h+1)·D/H)
 *   O   [B, N, D]   output, same layout as V
 *   z*  [B, H, N]   fp32 softmax weights (only from cat_forward_zstar)
 * X, W_A, V and O all have the plan's dtype.  All arithmetic is fp32:
 * bf16 inputs are widened exactly, bf16 outputs are rounded to nearest-even.
 *
 * Every function returns a cat_status (0 = CAT_OK, negative = error) and
 * never aborts, exits or traps.  GPU work is enqueued asynchronously on the
 * plan's stream; errors raised by kernels are reported by cat_plan_sync.
 */
#ifndef CAT_H_
#define CAT_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Opaque plan: shape, dtype, stream, device workspace, twiddle tables. */
typedef struct cat_plan_s *cat_plan_t;

/* Storage type of X, W_A, V and O. */
typedef enum { CAT_F32 = 0, CAT_BF16 = 1 } cat_dtype_t;

/* Type of token ids and targets. */
typedef enum { CAT_I32 = 2, CAT_I64 = 3 } cat_id_type_t;

/* Status codes. */
enum {
  CAT_OK = 0,
  CAT_ERR_INVALID_ARG = -1,   /* bad shape, null pointer, D % H != 0, ...   */
  CAT_ERR_UNSUPPORTED_N = -2, /* N has a prime factor > 7 or exceeds limits */
  CAT_ERR_MISALIGNED = -3,    /* a device pointer is not 16-byte aligned    */
  CAT_ERR_PLAN_MISMATCH = -4, /* call shape/dtype differs from the plan's   */
  CAT_ERR_ALLOC = -5,         /* device or host allocation failed           */
  CAT_ERR_CUDA = -6,          /* a CUDA runtime call or launch failed       */
  CAT_ERR_DEVICE_STATUS = -7, /* a kernel reported an internal check failure*/
  CAT_ERR_ALIAS = -8,         /* O overlaps X, W_A or V                     */
  CAT_ERR_TOO_LARGE = -9      /* beyond cat_forward_noalloc's fixed workspace */
};

/* Size limits of the library. */
#define CAT_MAX_N (1 << 22)   /* longest sequence                          */
#define CAT_MAX_D 8192        /* widest model dimension                    */

/*
 * cat_plan_create — validate a problem shape and build everything the
 * forward pass needs: the execution path (single-CTA shared-memory FFT for
 * N up to 16384, four-step multi-CTA FFT above), fp32 twiddle tables
 * computed in fp64 on the host, and the device workspace (scores, softmax
 * weights, their spectra, four-step scratch).  The plan owns that memory.
 *
 *   out    : receives the plan (set to NULL on failure)
 *   B      : batch size, >= 0 (B = 0 makes cat_forward a no-op)
 *   N      : sequence length, 1 <= N <= CAT_MAX_N, 7-smooth (only prime
 *            factors 2, 3, 5, 7)
 *   D, H   : model width and head count, 1 <= H <= D <= CAT_MAX_D, D % H == 0
 *   dtype  : CAT_F32 or CAT_BF16
 *   stream : cudaStream_t to enqueue on (NULL = legacy default stream); the
 *            caller keeps ownership and must keep it alive while the plan
 *            uses it.
 * Errors: CAT_ERR_INVALID_ARG, CAT_ERR_UNSUPPORTED_N, CAT_ERR_ALLOC,
 * CAT_ERR_CUDA.  Uses the CUDA device current at the call.
 */
int cat_plan_create(cat_plan_t *out, int B, int N, int D, int H, int dtype,
                    void *stream);

/*
 * cat_plan_query — the plan cat_plan_create would build for this shape,
 * without touching the device or allocating: *workspace_bytes (may be
 * NULL) receives the device workspace it would allocate, and desc (may be
 * NULL; capacity len bytes, NUL-terminated, truncated if needed) the same
 * one-line description cat_plan_describe gives (path, factorisation,
 * launch shapes).  The backward workspace, allocated at a plan's first
 * backward call, is not included.  Errors: those of cat_plan_create's
 * shape validation (CAT_ERR_INVALID_ARG, CAT_ERR_UNSUPPORTED_N).
 */
int cat_plan_query(int B, int N, int D, int H, int dtype,
                   size_t *workspace_bytes, char *desc, int len);

/* Release a plan and its device memory.  NULL is accepted (no-op).
 * Synchronises the plan's stream first.  Destroying twice is undefined. */
int cat_plan_destroy(cat_plan_t plan);

/* Change the stream later calls enqueue on. */
int cat_plan_set_stream(cat_plan_t plan, void *stream);

/*
 * cat_forward — O = CAT(X, W_A, V) for every batch and head (both designs
 * of the notes page cited above): scores, softmax over tokens, spectrum of
 * z* once per (b, h), then per value column IFFT(FFT(z*) ⊙ FFT(v)).
 *
 * X, W_A, V: device pointers, read only.  O: device pointer, written.
 * All four must be 16-byte aligned and O must not overlap the others.
 * B, N, D, H, dtype must equal the plan's (CAT_ERR_PLAN_MISMATCH).
 * Asynchronous on the plan's stream: work that the fast long-sequence path
 * (head width 64, N = 512·N2 with N2 in 32..256) spreads over the plan's two
 * internal streams forks from and joins back into the plan's stream, so the
 * call is ordered like a single kernel on it.  The plan's workspace is
 * reused, so two calls on one plan must not run concurrently on different
 * streams.
 */
int cat_forward(cat_plan_t plan, const void *X, const void *W_A, const void *V,
                void *O, int B, int N, int D, int H, int dtype);

/*
 * cat_forward_fused — the value projection and the scores from one pass
 * over X, then the forward: V = X·W_V (written to V) and z = X·W_A from the
 * same tensor-core GEMM [V | z] = X·[W_V | W_A] (the notes page cited
 * above, 整体框架 overall framework: a CAT layer projects X with W_V for
 * the values and W_A for the scores), then O = CAT(X, W_A, V) exactly as
 * cat_forward computes it from those V and z.
 *
 * X [B, N, D], W_V [D, D] (row-major, V[b, n, :] = X[b, n, :]·W_V) and
 * W_A [D, H]: device pointers, read only.  V and O [B, N, D]: device
 * pointers, written.  bf16 only (CAT_ERR_INVALID_ARG otherwise), D a
 * multiple of 64, H <= 16; products of bf16 values are exact, accumulation
 * fp32; V is rounded to bf16 (nearest even); the scores are kept as
 * double-float sums of 64-wide fp32 slices.  All pointers 16-byte aligned;
 * V and O must not overlap the inputs or each other (CAT_ERR_ALIAS).  The
 * first call allocates the plan's transposed-weight workspace (2·D·(D+16)
 * bytes; CAT_ERR_ALLOC).  Asynchronous on the plan's stream.
 */
int cat_forward_fused(cat_plan_t plan, const void *X, const void *W_V,
                      const void *W_A, void *V, void *O, int B, int N, int D,
                      int H, int dtype);

/*
 * cat_project — the fused projection alone: V = X·W_V (written to V) and
 * z* = softmax over the tokens of X·W_A (fp32 [B, H, N], written to the
 * device pointer zstar), from the same one-pass tensor-core GEMM as
 * cat_forward_fused.  Arguments, limits and errors as cat_forward_fused;
 * zstar must not overlap X or V (CAT_ERR_ALIAS).
 */
int cat_project(cat_plan_t plan, const void *X, const void *W_V, const void *W_A,
                void *V, float *zstar, int B, int N, int D, int H, int dtype);

/*
 * cat_forward_zstar — only the first two steps (score projection and
 * softmax over the N tokens, "circulant attention matrix construction"):
 * writes z* as fp32 [B, H, N] to the device pointer zstar (16-byte aligned).
 */
int cat_forward_zstar(cat_plan_t plan, const void *X, const void *W_A,
                      float *zstar, int B, int N, int D, int H, int dtype);

/*
 * cat_forward_host — the same forward on HOST buffers, copies included: X,
 * W_A, V are read from host memory and O is written to host memory before
 * the call returns (it synchronises).  With B >= 2 the call runs one batch
 * per step and overlaps the copies with the compute: batch b's inputs copy
 * in on one internal stream while batch b - 1 computes on the plan's stream
 * and batch b - 2's output copies out on another.  The first call sets up
 * plan-owned device staging (two batches' worth, or the whole problem when
 * B = 1), two internal one-batch plans and the copy streams, which the plan
 * keeps; CAT_ERR_ALLOC if that fails.  Pinned (page-locked) host memory is
 * needed for the copies to overlap; pageable memory works but serialises.
 * Kernel status of the internal plans is reported by cat_plan_sync.
 */
int cat_forward_host(cat_plan_t plan, const void *X, const void *W_A,
                     const void *V, void *O, int B, int N, int D, int H,
                     int dtype);

/*
 * cat_backward — gradients of a loss L through the forward pass, given the
 * upstream gradient dO = dL/dO.  The notes page cited above trains CAT
 * layers with the usual losses and optimisers (section 损失函数 / 训练策略,
 * loss and training strategy) but prints no gradients; these follow from
 * the forward definitions by the chain rule, per (b, h):
 *   dV   = circ(z*)^T dO          dV[j, c] = sum_i z*[(i - j) mod N] dO[i, c]
 *   dz*[k] = sum_{c in h} sum_i dO[i, c] V[(i - k) mod N, c]
 *          = Re IFFT( sum_c FFT(dO[:, c]) ⊙ conj(FFT(V[:, c])) )
 *   dz   = z* ⊙ (dz* - <z*, dz*>)  (softmax Jacobian)
 *   dW_A[d, h] = sum_{b, n} X[b, n, d] dz[b, h, n]
 *   dX[b, n, d] = sum_h dz[b, h, n] W_A[d, h]
 * z* is recomputed from X and W_A (nothing is kept from a forward call).
 *
 * X, W_A, V, dO: device pointers, read only ([B,N,D], [D,H], [B,N,D],
 * [B,N,D]).  dX [B,N,D], dW_A [D,H], dV [B,N,D]: device pointers, written;
 * dW_A is overwritten, not accumulated into.  All seven have the plan's
 * dtype (bf16 gradients are rounded to nearest-even from fp32), must be
 * 16-byte aligned (CAT_ERR_MISALIGNED), and no output may overlap an input
 * or another output (CAT_ERR_ALIAS).  Shape arguments must equal the plan's.
 * The first call configures and allocates the plan's backward workspace
 * (correlation scratch, dz*, dz, dW_A partial sums), which the plan keeps;
 * CAT_ERR_ALLOC if that fails.  Asynchronous on the plan's stream; the
 * plan's forward workspace is reused, so a backward and a forward on one
 * plan must not run concurrently on different streams.
 */
int cat_backward(cat_plan_t plan, const void *X, const void *W_A, const void *V,
                 const void *dO, void *dX, void *dW_A, void *dV, int B, int N,
                 int D, int H, int dtype);

/*
 * cat_backward_dz — only the score-side gradients of cat_backward: writes
 * dz* = dL/dz* and dz = dL/dz (the softmax backward of dz*), each fp32
 * [B, H, N], to the device pointers dzstar and dz (16-byte aligned, not
 * overlapping the inputs or each other: CAT_ERR_ALIAS).  Inputs and errors
 * as for cat_backward.
 */
int cat_backward_dz(cat_plan_t plan, const void *X, const void *W_A,
                    const void *V, const void *dO, float *dzstar, float *dz,
                    int B, int N, int D, int H, int dtype);

/*
 * 2-D circulant attention — the page "Vision Transformers are Circulant
 * Attention Learners": for tokens on an h x w grid (token n = y·w + x) the
 * attention map is modelled as a BCCB matrix (block circulant with
 * circulant blocks) with generator σ(a), so that O = σ(a) ⊛ V, a 2-D
 * circular convolution, computed with 2-D FFTs; a comes from Q and K by
 * FFTs and an element-wise product.  The page prints no formula for a; the
 * reading taken is the channel-averaged 2-D circular cross-correlation
 *     a[b, hd, k] = (1/dh) Σ_{c in head hd} Σ_i Q[b, i, c] · K[b, i ⊖ k, c]
 * (i ⊖ k: grid-wise difference mod (h, w)), σ the softmax over the N = h·w
 * lags, and O[b, i, c] = Σ_j σ(a)[b, hd(c), i ⊖ j] · V[b, j, c].
 *
 * cat_plan_create_2d — a plan for B batches on an h x w grid (1 <= h, w <=
 * 16384, each 7-smooth, h·w <= CAT_MAX_N), model width D, H heads, dtype,
 * stream; errors as cat_plan_create.  A 2-D plan serves only the cat2d_*
 * calls (the 1-D calls return CAT_ERR_PLAN_MISMATCH), and the cat2d_* calls
 * take only 2-D plans.  It allocates its whole workspace at creation.
 */
int cat_plan_create_2d(cat_plan_t *out, int B, int h, int w, int D, int H,
                       int dtype, void *stream);

/*
 * cat2d_forward — O = σ(a) ⊛ V for every batch and head.  Q, K, V: device
 * pointers [B, h·w, D], read only; O: device pointer [B, h·w, D], written;
 * all in the plan's dtype, 16-byte aligned, O not overlapping Q, K or V.
 * Asynchronous on the plan's stream.
 */
int cat2d_forward(cat_plan_t plan, const void *Q, const void *K, const void *V,
                  void *O, int B, int h, int w, int D, int H, int dtype);

/*
 * cat2d_scores — only the scores a (before the softmax), fp32 [B, H, h·w],
 * to the device pointer a (16-byte aligned, not overlapping Q or K:
 * CAT_ERR_ALIAS).
 */
int cat2d_scores(cat_plan_t plan, const void *Q, const void *K, float *a,
                 int B, int h, int w, int D, int H, int dtype);

/*
 * Operators around a CAT layer in a training step: the notes page cited
 * above alternates CAT layers with ordinary softmax attention (CAT-Alter) in
 * pre-norm ViT and GPT-2 stacks trained by a clipped optimiser.  Their plans
 * are cat_plan_t too: cat_plan_sync, cat_plan_describe, cat_plan_set_stream
 * and cat_plan_destroy serve them, every other plan call returns
 * CAT_ERR_PLAN_MISMATCH for them.  Calls are asynchronous on the plan's
 * stream, may be captured into a CUDA graph, and run on the plan's device
 * whichever device is current.  A plan's workspace is reused by every call
 * (and by every graph captured from it), so the calls and replays of one
 * plan must not run concurrently.  Results repeat bit for bit.
 */

/* Widest head and most token rows of the softmax attention. */
#define CAT_ATTN_MAX_DH 128
#define CAT_ATTN_MAX_TOKENS (1 << 30)

/*
 * cat_plan_create_attn — softmax attention over packed sequences: T token
 * rows hold S sequences of different lengths one after another, sequence s
 * in rows cu_seqlens[s] .. cu_seqlens[s+1] - 1, each attending to itself
 * only.  Hq query heads share Hkv key heads, query head h reads key head
 * h / (Hq / Hkv).
 *
 *   max_tokens, max_seqs : the largest T and S of a call, >= 0 (max_tokens <=
 *            CAT_ATTN_MAX_TOKENS; their blocks, (max_tokens / 64 +
 *            max_seqs)·Hq, and max_tokens·Hq within 2^31)
 *   Hq, Hkv, dh : heads and head width, Hq % Hkv == 0, 1 <= dh <=
 *            CAT_ATTN_MAX_DH, Hq·dh <= 2^20
 *   dtype  : of Q, K, V, O and the gradients; products accumulate in fp32,
 *            lse is fp32
 *   causal : 1: row i of a sequence sees rows 0 .. i of it; 0: all of it
 *   scale  : factor of the scores, > 0; 0 means 1/sqrt(dh)
 *   stream : as for cat_plan_create
 * Errors: CAT_ERR_INVALID_ARG, CAT_ERR_ALLOC, CAT_ERR_CUDA.
 */
int cat_plan_create_attn(cat_plan_t *out, int max_tokens, int max_seqs, int Hq,
                         int Hkv, int dh, int dtype, int causal, float scale,
                         void *stream);

/*
 * cat_attn_forward — per sequence and head, with its rows i, j:
 *   s_ij = scale·q_i·k_j (j <= i if causal), lse_i = log Σ_j exp(s_ij),
 *   o_i  = Σ_j exp(s_ij - lse_i) v_j.
 *
 * Q [T, Hq, dh], K and V [T, Hkv, dh]: token rows ldq, ldk, ldv elements
 * apart (>= the row's own width; heads dense in a row), so that they may be
 * columns of one projection's output.  O [T, Hq, dh] and lse [Hq, T] (fp32,
 * for the backward): dense, written.  cu_seqlens: device array of S + 1
 * ascending int values within 0 .. T.  Rows that no sequence holds (before
 * cu_seqlens[0], from cu_seqlens[S] on) are neither read into any result nor
 * written; a sequence may be empty.  Pointers need the alignment of their
 * element type.  bf16 data whose rows and heads all start on 16-byte
 * boundaries, and fp32 data (its backward up to dh = 64), take the tensor
 * cores; the rest takes the FP32 pipe, an order of magnitude slower.  On the
 * tensor cores the probabilities of bf16 data are rounded to bf16 (a half step
 * of 2^-8 of each, in O and in the backward's dV), its ds_ij are two bf16 terms
 * (2^-16), and fp32 operands are split into three (errors of fp32's own size).
 * A pair the mask excludes contributes nothing, whatever its rows hold; fp32
 * rows that meet an infinity or NaN are computed one by one, which takes far
 * longer (a NaN in 8192 causal tokens: 50 ms).  If cu_seqlens is not ascending
 * within 0 .. T, the sequences concerned are skipped and cat_plan_sync returns
 * CAT_ERR_DEVICE_STATUS.
 * Errors: CAT_ERR_PLAN_MISMATCH (not an attention plan, T or S above the
 * plan's), CAT_ERR_INVALID_ARG, CAT_ERR_MISALIGNED, CAT_ERR_ALIAS (an output
 * meets an input or another output), CAT_ERR_CUDA.  T = 0 or S = 0: no-op.
 */
int cat_attn_forward(cat_plan_t plan, const void *Q, const void *K,
                     const void *V, void *O, float *lse, const int *cu_seqlens,
                     int T, int S, long long ldq, long long ldk, long long ldv);

/*
 * cat_attn_backward — gradients for the upstream gradient dO = dL/dO, from
 * the forward's inputs and its O and lse:
 *   p_ij = exp(s_ij - lse_i), ds_ij = p_ij (dO_i·v_j - dO_i·o_i),
 *   dQ_i = scale Σ_j ds_ij k_j, dK_j = scale Σ_i ds_ij q_i, dV_j = Σ_i p_ij dO_i,
 * dK and dV summed over the query heads that share the key head.  O and dO
 * dense; dQ, dK, dV with token strides lddq, lddk, lddv (they may be columns
 * of one buffer), overwritten, not accumulated into.  Other arguments and
 * errors as for cat_attn_forward.
 */
int cat_attn_backward(cat_plan_t plan, const void *Q, const void *K,
                      const void *V, const void *O, const float *lse,
                      const void *dO, void *dQ, void *dK, void *dV,
                      const int *cu_seqlens, int T, int S, long long ldq,
                      long long ldk, long long ldv, long long lddq,
                      long long lddk, long long lddv);

/* Most rows of one layer-norm call. */
#define CAT_NORM_MAX_ROWS (1 << 30)

/*
 * cat_plan_create_layernorm — layer norm over rows of D elements
 * (1 <= D <= CAT_MAX_D), at most max_rows of them a call (0 ..
 * CAT_NORM_MAX_ROWS); eps >= 0.
 * Errors: CAT_ERR_INVALID_ARG, CAT_ERR_ALLOC, CAT_ERR_CUDA.
 */
int cat_plan_create_layernorm(cat_plan_t *out, int max_rows, int D, int dtype,
                              float eps, void *stream);

/*
 * cat_layernorm_forward — per row of X [rows, D], with its mean and
 * rstd = 1/sqrt(variance + eps) (the variance over D, not D - 1):
 *   Y = (X - mean)·rstd·gamma + beta.
 * gamma and beta [D] may be NULL (1 and 0).  mean and rstd [rows] (fp32) are
 * written for the backward.  X, gamma, beta, Y: the plan's dtype, dense,
 * 16-byte aligned; outputs must not overlap inputs or each other
 * (CAT_ERR_ALIAS).  rows above the plan's: CAT_ERR_PLAN_MISMATCH.
 */
int cat_layernorm_forward(cat_plan_t plan, const void *X, const void *gamma,
                          const void *beta, void *Y, float *mean, float *rstd,
                          int rows);

/*
 * cat_layernorm_backward — with x̂ = (X - mean)·rstd and g = dY·gamma:
 *   dX = rstd (g - mean_D(g) - x̂·mean_D(g·x̂)),
 *   dgamma = Σ_rows dY·x̂, dbeta = Σ_rows dY (fp32 sums, rounded once).
 * dgamma and dbeta may each be NULL (not wanted) and are overwritten.
 * rows = 0 writes zeros to them.  Other arguments and errors as above.
 */
int cat_layernorm_backward(cat_plan_t plan, const void *X, const void *gamma,
                           const float *mean, const float *rstd, const void *dY,
                           void *dX, void *dgamma, void *dbeta, int rows);

/* Most tensors of one clipping plan. */
#define CAT_CLIP_MAX_TENSORS (1 << 20)

/*
 * cat_plan_create_clip — the global norm of a list of gradients, and clipping
 * by it.  count >= 0 tensors, tensor i of sizes[i] >= 0 elements (dense) and
 * type dtypes[i] (host arrays, copied).  Errors: CAT_ERR_INVALID_ARG,
 * CAT_ERR_ALLOC, CAT_ERR_CUDA.
 */
int cat_plan_create_clip(cat_plan_t *out, int count, const long long *sizes,
                         const int *dtypes, void *stream);

/*
 * cat_grad_norm — *norm (device, fp32) = sqrt(Σ_i Σ_k grads[i][k]²).  grads:
 * host array of the plan's count device pointers (read during the call), each
 * aligned to its element type; tensors of size 0 may be NULL.  norm must not
 * lie in a gradient (CAT_ERR_ALIAS).  Sums keep values from 1e-30 to 1e30 apart
 * from fp32's limits.
 */
int cat_grad_norm(cat_plan_t plan, const void *const *grads, float *norm);

/*
 * cat_grad_clip — *norm as above, then outs[i] = c·grads[i] with
 * c = max_norm / norm where norm > max_norm, else 1.  outs[i] may be grads[i]
 * (in place); apart from that no output may overlap a gradient, another
 * output or norm (CAT_ERR_ALIAS: the same tensor twice in place, too).
 * max_norm >= 0, infinity allowed.  If a gradient holds an infinity or NaN,
 * *norm is not finite and c = 1: the caller sees it and the gradients keep
 * their values.
 */
int cat_grad_clip(cat_plan_t plan, const void *const *grads, void *const *outs,
                  float max_norm, float *norm);

/*
 * The rest of a language model's training step: the embedding at its start, the
 * residual stream between its layers, the cross entropy over the vocabulary at
 * its end.  The conventions of the operators above hold.  Ids and targets are
 * device arrays of 32- or 64-bit integers (id_type CAT_I32 or CAT_I64, aligned
 * to their size); a negative one marks a token that has none (padding, no
 * target), one of V or more is treated the same way and cat_plan_sync returns
 * CAT_ERR_DEVICE_STATUS.  Arrays of the plan's dtype are dense and 16-byte
 * aligned (CAT_ERR_MISALIGNED); outputs overlap neither inputs nor each other
 * (CAT_ERR_ALIAS); T or rows above the plan's: CAT_ERR_PLAN_MISMATCH.
 */

/* Largest vocabulary, most tokens of an embedding and of a cross entropy call. */
#define CAT_MAX_VOCAB (1 << 20)
#define CAT_STEP_MAX_TOKENS (1 << 24)
#define CAT_XENT_MAX_TOKENS (1 << 20)

/*
 * cat_plan_create_embed — rows of a table W [V, D], looked up by token, for at
 * most max_tokens tokens a call (0 .. CAT_STEP_MAX_TOKENS); 1 <= V <=
 * CAT_MAX_VOCAB, 1 <= D <= CAT_MAX_D, scale finite.
 * Errors: CAT_ERR_INVALID_ARG, CAT_ERR_ALLOC, CAT_ERR_CUDA.
 */
int cat_plan_create_embed(cat_plan_t *out, int max_tokens, int V, int D,
                          int dtype, float scale, void *stream);

/*
 * cat_embed_forward — Y[i] = scale·W[ids[i]] for T tokens (Y [T, D]); a row of
 * zeros where the token has no id.  T = 0: no-op.
 */
int cat_embed_forward(cat_plan_t plan, const void *ids, int id_type,
                      const void *W, void *Y, int T);

/*
 * cat_embed_backward — dW[v] = scale·Σ dY[i] over the tokens i with ids[i] = v
 * (fp32 sums in a fixed order, rounded once); dY [T, D], dW [V, D].
 * accumulate = 1: the sums are added to dW (which may hold the gradient of
 * output weights tied to the table), rows of ids that no token has keep their
 * bits; 0: dW is overwritten, those rows with zeros.  Rows of dY whose token
 * has no id are not read.
 */
int cat_embed_backward(cat_plan_t plan, const void *ids, int id_type,
                       const void *dY, void *dW, int accumulate, int T);

/*
 * cat_plan_create_resnorm — what lies between two blocks of a residual stream:
 * the block's output B, with a norm of its own (post = 1) or without (0), a
 * gate and a scale, is added to the stream R, and the sum is normed for the next
 * block.  At most max_rows rows a call (0 .. CAT_NORM_MAX_ROWS) of 1 <= D <=
 * CAT_MAX_D elements; eps >= 0 (both norms'), scale finite.
 * Errors: CAT_ERR_INVALID_ARG, CAT_ERR_ALLOC, CAT_ERR_CUDA.
 */
int cat_plan_create_resnorm(cat_plan_t *out, int max_rows, int D, int dtype,
                            int post, float eps, float scale, void *stream);

/*
 * cat_resnorm_forward — per row, with the layer norm LN of cat_layernorm_forward:
 *   u = post ? LN(B; post_gamma, post_beta) : B,
 *   H = R + scale·gate·u,   Y = LN(H; gamma, beta).
 * gate: NULL (1), [D] (gate_rows = 0) or [rows, D] (gate_rows = 1).  The weights
 * of the norms ([D] each) may be NULL (1 and 0); without post, post_gamma and
 * post_beta must be.  stats (fp32, for the backward): [2][rows], or [4][rows]
 * with post: mean and rstd of H, mean and rstd of B.  Y and stats are those of H
 * before its rounding to the plan's dtype.
 */
int cat_resnorm_forward(cat_plan_t plan, const void *R, const void *B,
                        const void *gate, int gate_rows, const void *post_gamma,
                        const void *post_beta, const void *gamma,
                        const void *beta, void *H, void *Y, float *stats,
                        int rows);

/*
 * cat_resnorm_backward — from the forward's inputs, its H and stats, and the
 * upstream gradients dH (NULL: zero) and dY of its outputs:
 *   dh = dH + (gradient of LN at H for dY),  dR = dh,
 *   dgate = scale·u·dh (summed over the rows where the gate is [D]),
 *   du = scale·gate·dh,  dB = post ? (gradient of LN at B for du) : du,
 * and the weights' gradients (fp32 sums over the rows, rounded once).  H enters as
 * stored: in dgamma a bf16 H is half a step off the one whose norm Y is.  dgate and
 * the weights' gradients may each be NULL (not wanted), all are overwritten.
 * rows = 0 writes zeros to the sums over the rows.
 */
int cat_resnorm_backward(cat_plan_t plan, const void *H, const void *B,
                         const void *gate, int gate_rows,
                         const void *post_gamma, const void *post_beta,
                         const void *gamma, const float *stats, const void *dH,
                         const void *dY, void *dR, void *dB, void *dgate,
                         void *dpost_gamma, void *dpost_beta, void *dgamma,
                         void *dbeta, int rows);

/*
 * cat_plan_create_xent — softmax cross entropy over a vocabulary of V, from
 * hidden states of width D (1 <= V <= CAT_MAX_VOCAB, 1 <= D <= CAT_MAX_D) and
 * the output weights, for at most max_tokens tokens a call (0 ..
 * CAT_XENT_MAX_TOKENS).  grad = 0: a plan for the forward alone, which needs
 * far less workspace.
 * Errors: CAT_ERR_INVALID_ARG, CAT_ERR_ALLOC, CAT_ERR_CUDA.
 */
int cat_plan_create_xent(cat_plan_t *out, int max_tokens, int V, int D,
                         int dtype, int grad, void *stream);

/*
 * cat_xent_forward — for T tokens, X [T, D], W [V, D] and targets [T]:
 *   l_iv = X_i·W_v,  lse[i] = log Σ_v exp(l_iv),  loss[i] = lse[i] - l_{i,targets[i]}
 * (fp32).  Tokens without a target: both are 0, their rows of X are not read.
 * The logits are not kept.  Products run on the tensor cores with fp32 sums, fp32
 * operands as three bf16 terms (errors of fp32's own size); an fp32 logit that is
 * not finite is computed again by its definition.  So weights of minus infinity
 * rule ids out, a logit of plus infinity makes lse that.  loss is (the largest
 * logit - the target's) + log of the sum of exponentials of the differences to the
 * largest: never negative, and no worse for large logits; lse is rounded to fp32
 * once.  T = 0: no-op.
 */
int cat_xent_forward(cat_plan_t plan, const void *X, const void *W,
                     const void *targets, int id_type, float *loss, float *lse,
                     int T);

/*
 * cat_xent_backward — from the forward's inputs and its lse, for the upstream
 * gradient dloss of the losses (fp32: one value for all tokens, dloss_each = 0,
 * or [T], dloss_each = 1):
 *   d_iv = dloss_i (exp(l_iv - lse_i) - [v = targets_i]),  dX = d·W,  dW = dᵀ·X.
 * The logits are made again, a piece of the vocabulary at a time; the
 * probabilities of a row share the rounding of its lse (half a step, 2^-24 |lse|,
 * relative).  dX [T, D] and dW [V, D] are overwritten; either may be NULL (not
 * wanted).  Tokens without a target have a zero row in dX and no part in dW; their
 * dloss and lse are not read.  For bf16 data d_iv is rounded to bf16 as an operand
 * of the products (a half step of 2^-8 of each; one dloss for all tokens is applied
 * to the results instead), for fp32 data it is three bf16 terms.  Sums over tokens
 * and ids are fp32; of bf16 summands of one sign a run of 65536 loses 0.0004 (tensor
 * core accumulators cut instead of rounding), longer sums no more.  Gradients that
 * a value takes part in that is not finite are not finite.
 * CAT_ERR_PLAN_MISMATCH too for a plan with grad = 0.
 */
int cat_xent_backward(cat_plan_t plan, const void *X, const void *W,
                      const void *targets, int id_type, const float *lse,
                      const float *dloss, int dloss_each, void *dX, void *dW,
                      int T);

/*
 * cat_plan_sync — wait for the plan's stream, then read the device status
 * word the kernels set when an internal check fails (a bad index that was
 * skipped instead of accessed).  Returns CAT_OK, CAT_ERR_DEVICE_STATUS
 * (the word is cleared after reporting) or CAT_ERR_CUDA.
 */
int cat_plan_sync(cat_plan_t plan);

/*
 * cat_plan_describe — copy a one-line, NUL-terminated description of the
 * plan (path, factorisation, launch shapes, workspace bytes) into buf
 * (capacity len bytes, truncated if needed).
 */
int cat_plan_describe(cat_plan_t plan, char *buf, int len);

/*
 * cat_plan_timing — stage timing for profiling.  max_calls > 0 arms the plan
 * to record CUDA events around its three stages (score; softmax and, on the
 * shared-memory and fast paths, the spectrum of z*; the circulant product,
 * which on the general long-sequence path includes the spectrum of z*) on
 * its stream for the next max_calls cat_forward calls, discarding earlier
 * records; max_calls = 0 turns recording off.  On the fast path an event is
 * also recorded after each of passes A, B and C of every chunk.  While
 * recording, a forward runs its kernels one after another on the plan's
 * stream (the fast path otherwise replays a graph that overlaps chunks on
 * two internal streams), so each stage's and each pass's time is its own.
 * Synchronises the plan's stream.  The plan owns the events.
 * Errors: CAT_ERR_INVALID_ARG, CAT_ERR_ALLOC, CAT_ERR_CUDA.
 */
int cat_plan_timing(cat_plan_t plan, int max_calls);

/*
 * cat_plan_stage_times — wait for the plan's stream and write into ms[0..2]
 * (host array, cap >= 3) the milliseconds each stage took, summed over the
 * calls recorded since cat_plan_timing; *ncalls (may be NULL) receives how
 * many calls that was.  Errors: CAT_ERR_INVALID_ARG, CAT_ERR_CUDA.
 */
int cat_plan_stage_times(cat_plan_t plan, float *ms, int cap, int *ncalls);

/*
 * cat_plan_pass_times — fast path only: wait for the plan's stream and write
 * into ms[0..2] (host array, cap >= 3) the milliseconds that passes A, B and
 * C took, each summed over all chunks of the calls recorded since
 * cat_plan_timing; *launches (may be NULL) receives how many launches of
 * each pass that was (chunks per call times calls), so ms[i] / *launches is
 * one launch's average duration.  Errors: CAT_ERR_INVALID_ARG (no plan, cap
 * < 3, or not the fast path), CAT_ERR_CUDA.
 */
int cat_plan_pass_times(cat_plan_t plan, float *ms, int cap, int *launches);

/* Limits of cat_forward_noalloc's fixed device workspace. */
#define CAT_NOALLOC_MAX_ROWS (1 << 18) /* B·H·N                                 */
#define CAT_NOALLOC_MAX_N 16384        /* sequence length                       */

/*
 * cat_forward_noalloc — the same forward as cat_forward (short-sequence
 * shared-memory path), for callers that cannot allocate device memory: a
 * process whose device memory has been handed to a caching or pooled
 * allocator (where cudaMalloc would fail or fragment the pool), or a
 * latency-critical caller that cannot absorb the device-wide
 * synchronisation cudaMalloc and cudaFree imply.  It needs no plan and
 * never calls cudaMalloc, cudaFree or any allocating routine.  The notes
 * page has no counterpart to this entry point; it only changes where the
 * workspace lives.
 *
 * The workspace (scores, z*, spectra, twiddles, status word; about 5 MiB)
 * is one fixed array in the library's device image, which every GPU that
 * loads the library holds until the process exits.  Its size bounds the
 * problem: B·H·N <= CAT_NOALLOC_MAX_ROWS and N <= CAT_NOALLOC_MAX_N, else
 * CAT_ERR_TOO_LARGE.  Other shape rules and host-side errors are those of
 * cat_plan_create and cat_forward.  The kernels' own status word (a failed
 * internal check, which cat_plan_sync reports for plan calls) has no reader
 * here: it is cleared at every call and not reported, so only the returned
 * status (argument and launch errors) tells the caller of a failure.
 *
 * X, W_A, V (read) and O (written): device pointers as for cat_forward.
 * stream: cudaStream_t to enqueue on (NULL = legacy default stream).
 * The call is asynchronous.  The first call on each device also does a
 * one-time set-up on the host (it looks up the array's device address and
 * raises the kernels' shared-memory limits), so make that first call before
 * any stream capture.  All calls share the one array and it keeps the last
 * call's contents: calls whose GPU work overlaps (on different streams, or
 * from different host threads) race on it and must be ordered by the
 * caller.
 */
int cat_forward_noalloc(const void *X, const void *W_A, const void *V, void *O, int B,
                        int N, int D, int H, int dtype, void *stream);

/*
 * cat_probe_dft32 — measurement only, not part of the forward or backward:
 * applies one length-32 DFT stage `rounds` times (each scaled by
 * 1/sqrt(32)) to `nsig` complex fp32 signals (device pointers x, y,
 * [nsig][32] interleaved re/im), keeping each signal on chip, so that the
 * time is the stage's own cost.  mode 0: the register DFT-32 on the FP32
 * pipe (one signal per thread); mode 1 / 2: the stage as a dense 64 x 64 real
 * contraction on the tensor cores (tcgen05, 128 signals per CTA) with the
 * operands split into 2 / 3 bf16 terms (about 16 / 24 significant bits).
 * For the choice of where the small-DFT stages of the circulant product
 * run (the notes page's "FFT acceleration" design fixes the transform, not
 * the unit).  Asynchronous on `stream`.  Errors: CAT_ERR_INVALID_ARG,
 * CAT_ERR_ALLOC, CAT_ERR_CUDA.
 */
int cat_probe_dft32(const void *x, void *y, int nsig, int mode, int rounds, void *stream);

/* Static string for a status code ("CAT_OK", "CAT_ERR_INVALID_ARG", ...). */
const char *cat_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* CAT_H_ */
