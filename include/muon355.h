/*
 * muon355.h - C ABI of libmuon355, the Muon optimizer step on AMD Instinct
 * MI355X (gfx950).
 *
 * One Muon step for a hidden 2-D weight W (m x n) with gradient G is three
 * calls, in this order, all asynchronous on one HIP stream:
 *
 *   muon_momentum       M <- beta*M + (1-beta)*G, the Nesterov blend N, and
 *                       the sum of squares of N.
 *   muon_orthogonalize  O = K Newton-Schulz steps on N / (||N||_F + eps),
 *                       run on the smaller side (transposed when m > n).
 *   muon_apply          W <- (1 - lr*wd)*W - lr*s*O with the shape factor s.
 *
 * Sources ("the pages") cited below:
 *   [NOTES]  "Reading notes on SOAP, Muon and higher-order optimizers",
 *            section 1 "AdamW vs. SOAP vs. Muon" (moving-average momentum).
 *   [GUIDE]  "LLM Optimizers: From SGD and AdamW to SOAP, Muon, and Scalable
 *            Training", sections 11.3 (momentum, Nesterov), 11.4
 *            (Newton-Schulz equations, epsilon, tall transpose) and 11.5
 *            (shape factors, decoupled weight decay).
 *   [LESSON] "Matrix optimizers: K-FAC, Shampoo and Muon" (Lesson 12),
 *            subsection "Newton-Schulz: UV^T with matrix products only"
 *            (Lemma 3 and the three-step algorithm) and subsection "Muon"
 *            (steps 1-4, update size).
 *   [PREPRINT] "SOAP, Muon, and Beyond: Pushing LLM Pretraining Scales"
 *            (epsilon 1e-7 for Muon).
 *   [ZH]     "初探优化器（一）：从SGD到SOAP-Muon", section 6.2 (the SOAP
 *            step; one power-iteration step plus QR for the bases).
 *
 * Beside the Muon step, muon_adamw updates the parameters Muon leaves to
 * AdamW ([GUIDE] sections 5 and 6), and the soap_* calls run SOAP, Adam in
 * the eigenbasis of Shampoo's statistics ([GUIDE] 11.1-11.2).
 *
 * Beside the optimizers stand the operators of the expert layers whose weights
 * they step: muon_block_* (8-bit block codes and their products), muon_route_*
 * (tokens to experts) and muon_expert_* (each token's sum over its experts).
 *
 * Conventions shared by every entry point:
 *   - All matrix memory and all workspaces are caller-owned DEVICE memory.
 *     The library never allocates, frees or synchronizes; every call only
 *     enqueues kernels on `stream` (a hipStream_t; NULL = the null stream)
 *     and returns.  Debugging aid: with MUON355_DEBUG_SYNC=1 in
 *     the environment every call waits for the work it enqueued and reports
 *     a failed kernel as MUON_ERR_LAUNCH naming the call.
 *   - Matrices are row-major with a leading dimension `ld` (elements between
 *     consecutive rows, ld >= cols).  A batch holds `count` matrices of one
 *     shape and dtype: matrix i lives at ptrs[i] when `ptrs` is non-NULL (a
 *     DEVICE array of count pointers) and at base + i*stride elements
 *     otherwise.  All pointers must be 16-byte aligned.
 *   - Arguments are validated before anything is enqueued.  A non-OK status
 *     means nothing was enqueued (except MUON_ERR_LAUNCH, which reports a
 *     failed launch); muon_last_error() then gives a thread-local message.
 *     No C++ exception crosses this boundary.
 *   - Non-finite values in G or M propagate to sumsq and to the outputs; the
 *     caller may test sumsq and skip muon_apply (the library never skips).
 *   - Calls on one stream are ordered; calls that share a workspace must not
 *     run concurrently on different streams.
 */
#ifndef MUON355_H
#define MUON355_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MUON355_ABI_VERSION 1

typedef enum muon_status {
  MUON_OK = 0,
  MUON_ERR_INVALID_VALUE = 1, /* a NULL required pointer, a bad size or a bad hyperparameter */
  MUON_ERR_UNSUPPORTED = 2,   /* a dtype or mode combination that is not built */
  MUON_ERR_WORKSPACE = 3,     /* workspace missing or smaller than the *_workspace() query */
  MUON_ERR_LAUNCH = 4         /* a kernel launch failed (hipGetLastError) */
} muon_status_t;

typedef enum muon_dtype {
  MUON_F32 = 0,  /* IEEE binary32 */
  MUON_BF16 = 1  /* bfloat16 (upper half of binary32), round-to-nearest-even on store */
} muon_dtype_t;

typedef enum muon_scale {
  MUON_SCALE_MATCH_RMS = 0, /* s = coeff * sqrt(max(m, n)); coeff = 0.2 matches AdamW's update RMS
                               ([GUIDE] 11.5, [LESSON] "Muon" step 4 and "Update size") */
  MUON_SCALE_ORIGINAL = 1,  /* s = sqrt(max(1, m / n)) ([GUIDE] 11.5, [LESSON] "Muon" step 4) */
  MUON_SCALE_NONE = 2       /* s = 1 */
} muon_scale_t;

typedef struct muon_batch {
  void* const* ptrs; /* device array of `count` matrix pointers, or NULL to use base/stride */
  void* base;        /* matrix i at base + i*stride elements when ptrs == NULL */
  int64_t stride;    /* elements between consecutive matrices (strided batch) */
  int64_t count;     /* number of matrices, 1 .. 65535 (split larger batches) */
  int64_t rows;      /* m >= 1; rows * cols <= 2^31 - 1 */
  int64_t cols;      /* n >= 1 */
  int64_t ld;        /* leading dimension in elements, >= cols */
  int32_t dtype;     /* muon_dtype_t */
  int32_t reserved;  /* must be 0 */
} muon_batch_t;

/* Bytes of device workspace muon_momentum needs for `count` matrices of
 * rows x cols (per-block partial sums of the Frobenius reduction). */
size_t muon_momentum_workspace(int64_t count, int64_t rows, int64_t cols);

/*
 * Momentum, Nesterov blend and the sum of squares of the Newton-Schulz input.
 *
 *   M <- beta*M + (1-beta)*G                          ([NOTES] section 1)
 *   N  = (1-beta)*G + beta*M   if nesterov, else N = M
 *   sumsq[i] = sum of N_i^2 over all entries          ([GUIDE] 11.4, X_0)
 *
 * The pages write the accumulating form B <- beta*B + G, N = G + beta*B
 * ([GUIDE] 11.3, [LESSON] "Muon" steps 1-2); the moving average here is
 * (1-beta) times it, which Newton-Schulz's normalization removes.
 *
 * grad : G, BF16 or F32, read only.
 * mom  : M, F32, read and written in place.
 * nout : N, BF16 or F32, written; may be NULL only when nesterov == 0, in
 *        which case M itself is the Newton-Schulz input.
 * sumsq: device float[count], written (sum of squares of N as computed in
 *        fp32, before any bf16 rounding of N; partials are added in fp64).
 * beta : in [0, 1).  nesterov: 0 or 1.
 * Arithmetic is fp32.  Shapes of grad, mom and nout must match.
 */
muon_status_t muon_momentum(const muon_batch_t* grad, const muon_batch_t* mom,
                            const muon_batch_t* nout, float* sumsq, float beta,
                            int nesterov, void* workspace, size_t ws_bytes,
                            void* stream);

/* Bytes of device workspace muon_momentum_grouped needs: the sum of
 * muon_momentum_workspace over the groups; 0 for invalid arguments. */
size_t muon_momentum_grouped_workspace(int ngroups, const int64_t* counts,
                                       const int64_t* rows, const int64_t* cols);

/*
 * muon_momentum for several shape classes in one launch (plus one launch of
 * the sum-of-squares finalization): group g is the batch grads[g], moms[g],
 * nouts[g] with its own device float[count] sumsqs[g], all with the meaning,
 * layout and rules of muon_momentum; beta and nesterov are shared.  The
 * pages' per-layer and per-expert matrices come in a few shape classes
 * ([NOTES] section 1 and 3), so one step's momentum is one grid here.
 *
 * ngroups: 1..8.  grads, moms: host arrays of ngroups descriptors.  nouts:
 * host array of ngroups descriptors, or NULL (only without Nesterov: M is
 * then the Newton-Schulz input of every group).  sumsqs: host array of
 * ngroups device pointers.  workspace: at least
 * muon_momentum_grouped_workspace bytes, 16-byte aligned.  Every group is
 * validated before anything is enqueued; muon_last_error() names the
 * failing group.  Results equal separate muon_momentum calls bit for bit.
 */
muon_status_t muon_momentum_grouped(int ngroups, const muon_batch_t* grads,
                                    const muon_batch_t* moms,
                                    const muon_batch_t* nouts,
                                    float* const* sumsqs, float beta,
                                    int nesterov, void* workspace,
                                    size_t ws_bytes, void* stream);

/*
 * Allocation-free form of muon_momentum_grouped, for callers that cannot
 * allocate device memory or hand the library a workspace: code under HIP
 * graph capture, tight serving loops, harnesses that forbid allocation.
 *
 * Same arguments, meaning, validation and results (bit for bit) as
 * muon_momentum_grouped, without `workspace` and `ws_bytes`: the per-block
 * partial sums go to a static device array of MUON_NOALLOC_SCRATCH_BYTES
 * that the library holds on each GPU it runs on until the process ends (its
 * address is looked up on the first call on a device).  The call allocates
 * and frees nothing.
 *
 * Limit: muon_momentum_grouped_workspace(...) of the call must not exceed
 * MUON_NOALLOC_SCRATCH_BYTES (8 MiB: about two million partial sums, i.e.
 * up to about 1.7e10 matrix elements per call); larger calls return
 * MUON_ERR_WORKSPACE before anything is enqueued.
 * Every call on one GPU uses that GPU's one array: calls that may overlap
 * on a GPU (unordered streams, several host threads) race on it and must be
 * serialized by the caller.  Nothing in the array needs to start at zero:
 * each call writes every partial it reads.
 */
#define MUON_NOALLOC_SCRATCH_BYTES ((size_t)8 << 20)

muon_status_t muon_momentum_grouped_noalloc(int ngroups, const muon_batch_t* grads,
                                            const muon_batch_t* moms,
                                            const muon_batch_t* nouts,
                                            float* const* sumsqs, float beta,
                                            int nesterov, void* stream);

/* Bytes of device workspace muon_orthogonalize needs for `count` matrices
 * of stored shape rows x cols computed in `compute` (MUON_BF16 or MUON_F32).
 * Returns 0 for invalid arguments. */
size_t muon_orthogonalize_workspace(int64_t count, int64_t rows, int64_t cols,
                                    int32_t compute);

/*
 * Newton-Schulz orthogonalization ([GUIDE] 11.4; [LESSON] Lemma 3 and the
 * algorithm after it):
 *   X_0 = N / (sqrt(sumsq) + eps), transposed when rows > cols;
 *   K times: A = X X^T;  B = b*A + c*A*A;  X <- a*X + B*X;
 *   O = X_K in the stored orientation.
 *
 * in     : N, BF16 or F32 (the momentum output), read only.
 * sumsq  : device float[count] from muon_momentum, or NULL to have it
 *          computed here from `in`.
 * out    : O, BF16 or F32, same rows/cols as `in`, written.  May alias
 *          `in` (the iteration runs in the workspace).
 * steps  : K >= 0 (5 in Muon).  a, b, c: finite coefficients, the same at
 *          every step ((3.4445, -4.7750, 2.0315) in Muon).
 * eps    : finite, >= 0 (1e-7 in Muon, [PREPRINT]); added to the norm.
 * compute: MUON_BF16 = bf16 MFMA operands with fp32 accumulation; X is
 *          carried between steps as a bf16 high part (the MFMA operand)
 *          plus its rounding residual as 8-bit codes with an exponent shared
 *          by 16 values, about 16 significant bits together, for the a*X
 *          term (the fast path);
 *          MUON_F32   = fp32 MFMA throughout (the parity path).
 *          With MUON_BF16 an F32 `in` is preferred: the high/low copy of X
 *          starts from it, while a BF16 `in` starts the iteration from
 *          bf16-rounded values, an error the iteration amplifies on
 *          ill-conditioned inputs (about 10x larger output error at
 *          condition number 1e4).
 * The Gram and polynomial GEMMs compute only upper-triangle tiles and
 * mirror them.  The Newton-Schulz shape padded to the tile size (128 or
 * 256) may hold at most 2^30 elements; larger shapes return
 * MUON_ERR_UNSUPPORTED.
 */
muon_status_t muon_orthogonalize(const muon_batch_t* in, const float* sumsq,
                                 const muon_batch_t* out, int steps, float a,
                                 float b, float c, float eps, int32_t compute,
                                 void* workspace, size_t ws_bytes,
                                 void* stream);

/* Grouped form: `ngroups` batches of different shapes orthogonalized with
 * one kernel launch per stage (every group's tiles packed into one grid).
 * ins[g], outs[g] and sumsqs[g] are as in muon_orthogonalize (sumsqs may be
 * NULL, or hold NULL entries, to compute them here).  1 <= ngroups <= 8.
 * The workspace query takes the same per-group arrays. */
size_t muon_orthogonalize_grouped_workspace(int ngroups, const int64_t* counts,
                                            const int64_t* rows,
                                            const int64_t* cols,
                                            int32_t compute);
muon_status_t muon_orthogonalize_grouped(int ngroups, const muon_batch_t* ins,
                                         const float* const* sumsqs,
                                         const muon_batch_t* outs, int steps,
                                         float a, float b, float c, float eps,
                                         int32_t compute, void* workspace,
                                         size_t ws_bytes, void* stream);

/*
 * The momentum and the Newton-Schulz input in one pass ("packed" pair).
 *
 * muon_momentum_packed_grouped does what muon_momentum_grouped does for M and
 * the sums of squares (same arithmetic: M is bit-identical; the sums of
 * squares are added per 64 x 64 tile instead of per block, then in fp64 in
 * a fixed order), but instead of writing the Nesterov blend N to a caller
 * buffer it writes N straight into `workspace` in the layout the
 * Newton-Schulz kernels read (bf16 high part and 8-bit residual with
 * MUON_BF16; fp32 with MUON_F32; padded, and transposed when rows > cols).
 * muon_orthogonalize_packed_grouped then runs the iteration of
 * muon_orthogonalize_grouped from that workspace, dividing by
 * sqrt(sumsq) + eps inside its first step ([GUIDE] 11.4, X_0 equation: the
 * Gram of step 0 is scaled by 1/(||N||+eps)^2 and its update by
 * 1/(||N||+eps)), so N never makes a round trip through memory.
 *
 * Contract: both calls take the same groups (the shapes of grads[g] in the
 * first are the shapes of outs[g] in the second), the same compute and the
 * same workspace of at least muon_packed_grouped_workspace bytes (16-byte
 * aligned), in this order on one stream; the workspace carries the packed
 * input from the first call to the second.  sumsqs[g]: device float[count]
 * written by the first call, read by the second.  steps >= 1 (steps == 0
 * takes the separate calls).  Arguments, hyperparameters, outputs and
 * errors otherwise as muon_momentum_grouped and muon_orthogonalize_grouped.
 * The result differs from the separate calls only by rounding (the input is
 * scaled after its bf16 rounding instead of before).
 */
size_t muon_packed_grouped_workspace(int ngroups, const int64_t* counts,
                                     const int64_t* rows, const int64_t* cols,
                                     int32_t compute);
muon_status_t muon_momentum_packed_grouped(int ngroups, const muon_batch_t* grads,
                                           const muon_batch_t* moms,
                                           float* const* sumsqs, float beta,
                                           int nesterov, int32_t compute,
                                           void* workspace, size_t ws_bytes,
                                           void* stream);
muon_status_t muon_orthogonalize_packed_grouped(int ngroups, const float* const* sumsqs,
                                                const muon_batch_t* outs, int steps,
                                                float a, float b, float c, float eps,
                                                int32_t compute, void* workspace,
                                                size_t ws_bytes, void* stream);

/*
 * The second call of the packed pair with the parameter update folded into
 * its last step ([GUIDE] 11.5 update equation; [LESSON] "Muon" step 4):
 * instead of writing O it updates each weight in place,
 *   W <- (1 - lr*weight_decay) * W - lr * s * O,
 * s from `mode` and `coeff` and (m, n) = (rows, cols) of W, as
 * muon_apply_grouped does for an O of the same shape.  O is never stored:
 * each value goes from the last GEMM's fp32 accumulator into the update, so
 * the result differs from muon_orthogonalize_packed_grouped followed by
 * muon_apply_grouped only by O's rounding to the dtype of a caller buffer
 * (none for fp32 O).  weights[g] takes the place of outs[g] (same shapes,
 * bf16 or fp32, read and written in place); every other argument, the
 * workspace and the errors are those of muon_orthogonalize_packed_grouped,
 * and lr, weight_decay, mode and coeff are checked as in muon_apply.
 */
muon_status_t muon_orthogonalize_apply_packed_grouped(int ngroups, const float* const* sumsqs,
                                                      const muon_batch_t* weights, int steps,
                                                      float a, float b, float c, float eps,
                                                      float lr, float weight_decay, int32_t mode,
                                                      float coeff, int32_t compute,
                                                      void* workspace, size_t ws_bytes,
                                                      void* stream);

/*
 * Parameter update ([GUIDE] 11.5 update equation; [LESSON] "Muon" step 4):
 *   W <- (1 - lr*weight_decay) * W - lr * s * O
 * with s from `mode` and `coeff` (see muon_scale_t) and (m, n) = (rows,
 * cols) of W.  Both terms read the old W.  Arithmetic is fp32; a BF16 W is
 * rounded once to nearest even.
 *
 * weight: W, BF16 or F32, in place.  ortho: O, BF16 or F32, same shape.
 * lr, weight_decay, coeff: finite.
 */
muon_status_t muon_apply(const muon_batch_t* weight, const muon_batch_t* ortho,
                         float lr, float weight_decay, int32_t mode,
                         float coeff, void* stream);

/*
 * muon_apply for several shape classes in one launch: group g updates
 * weights[g] from orthos[g] with the meaning and rules of muon_apply, its
 * scale s taken from its own (rows, cols); lr, weight_decay, mode and coeff
 * are shared.  ngroups: 1..8; weights, orthos: host arrays of ngroups
 * descriptors.  Every group is validated before the launch; results equal
 * separate muon_apply calls bit for bit.
 */
muon_status_t muon_apply_grouped(int ngroups, const muon_batch_t* weights,
                                 const muon_batch_t* orthos, float lr,
                                 float weight_decay, int32_t mode, float coeff,
                                 void* stream);

/*
 * AdamW for the parameters Muon does not take (embeddings, output head, norms,
 * biases), many tensors in one launch ([GUIDE] section 5 "Adam, line by
 * line" and section 6, decoupled weight decay):
 *   m <- beta1*m + (1-beta1)*g;   v <- beta2*v + (1-beta2)*g^2
 *   m_hat = m / (1 - beta1^t);    v_hat = v / (1 - beta2^t)
 *   theta <- (1 - lr*weight_decay)*theta - lr * m_hat / (sqrt(v_hat) + eps)
 * Epsilon is added outside the square root.  Arithmetic is fp32 (bias
 * corrections in double on the host); a BF16 theta is rounded once to
 * nearest even.
 *
 * Every tensor is a contiguous run of numels[i] elements (any shape),
 * 16-byte aligned.  The tensor list lives in DEVICE memory and is only
 * read by the kernel: params[i] (theta, in/out, param_dtype), grads[i]
 * (read, grad_dtype), exp_avg[i] and exp_avg_sq[i] (F32 state, in/out,
 * zero before step 1), numels[i], and chunk_offsets[0..count] = prefix sums
 * of ceil(numels[i] / MUON_ADAMW_CHUNK) with chunk_offsets[0] = 0;
 * total_chunks = chunk_offsets[count] is passed by value (the library does
 * not read device memory on the host).  Each kernel access is bounded by
 * its tensor's numel, so an inconsistent chunk table leaves elements
 * un-updated but never reads or writes outside a tensor.
 *
 * step : t >= 1, the number of this update for every tensor in the list
 *        (one list per parameter group; a tensor whose gradient is absent
 *        is left out of the call, [GUIDE] 6.2).
 * beta1, beta2 in [0, 1); eps finite >= 0; lr, weight_decay finite.
 */
#define MUON_ADAMW_CHUNK 4096

typedef struct muon_tensor_list {
  int64_t count;                 /* tensors, >= 1 */
  int64_t total_chunks;          /* chunk_offsets[count]; 1 .. 2^31-1 */
  void* const* params;           /* device array [count] */
  const void* const* grads;      /* device array [count] */
  float* const* exp_avg;         /* device array [count] */
  float* const* exp_avg_sq;      /* device array [count] */
  const int64_t* numels;         /* device array [count] */
  const int64_t* chunk_offsets;  /* device array [count + 1] */
  int32_t param_dtype;           /* muon_dtype_t of every theta */
  int32_t grad_dtype;            /* muon_dtype_t of every gradient */
} muon_tensor_list_t;

muon_status_t muon_adamw(const muon_tensor_list_t* tensors, int64_t step, float lr, float beta1,
                         float beta2, float eps, float weight_decay, void* stream);

/*
 * One step's control block, in DEVICE memory (64 bytes, 16-byte aligned,
 * owned by the caller): muon_grad_norm writes it, and the calls that take a
 * `control` argument read it when they RUN, not when they are enqueued.  A
 * captured step that replays therefore clips by its own gradients' norm and
 * counts its own steps.  Before the first use: lr_factor = 1, the rest 0.
 * Calls that share a block must be ordered, as calls that share a workspace.
 */
typedef struct muon_step_control {
  float norm;          /* global 2-norm of the gradients */
  float scale;         /* factor of every gradient: min(1, max_norm / norm) */
  float lr_factor;     /* factor of lr; written by the caller only */
  int32_t skip;        /* nonzero: this step changes no parameter and no state */
  int64_t step;        /* t: steps begun and not skipped */
  int64_t skipped;     /* steps skipped */
  int32_t reserved[8]; /* the library's; back at zero after every call */
} muon_step_control_t;

/* A gradient of a muon_grad_list: numel elements in one contiguous run,
 * aligned to its element size (16-byte aligned runs are read fastest). */
typedef struct muon_grad {
  const void* data;
  int64_t numel;       /* >= 0 */
  int64_t first_chunk; /* chunks of the tensors before it in the list */
  int32_t dtype;       /* muon_dtype_t; the types of a list may differ, another value adds nothing */
  int32_t reserved;    /* 0 */
} muon_grad_t;

#define MUON_GRAD_CHUNK 16384

/* Gradients of any number and types.  Both arrays lie in DEVICE memory and
 * are only read.  Tensor i takes ceil(numel / MUON_GRAD_CHUNK) chunks, and
 * chunk_tensor[c] names the tensor of chunk c.  An entry outside [0, count)
 * or a chunk outside its tensor is passed over, so a wrong table reads
 * nothing outside the tensors. */
typedef struct muon_grad_list {
  int64_t count;               /* tensors, >= 1 */
  int64_t total_chunks;        /* 0 .. 2^31-1 (0: every tensor is empty) */
  const muon_grad_t* grads;    /* device array [count] */
  const int32_t* chunk_tensor; /* device array [total_chunks] */
} muon_grad_list_t;

/*
 * Global gradient norm, clip factor and step count:
 *   norm  = sqrt(sum of g^2 over every element of every tensor)
 *   scale = min(1, max_norm / norm)   (NaN when norm is NaN)
 *   skip  = (flags & MUON_SKIP_NONFINITE) and norm is not finite
 *   step += 1, or skipped += 1 when skip
 * The gradients are only read: the calls that take `control` multiply by
 * `scale` as they read them.  Squares and sums are fp64 in an order that
 * depends on the list alone: none overflows, and equal inputs give equal bits.
 * The norm itself is a float: finite gradients whose norm is past the largest
 * float have an infinite one, and scale 0 (1 when max_norm is infinite).
 *
 * max_norm : > 0; infinity never clips.  flags: 0 or MUON_SKIP_NONFINITE.
 * workspace: at least muon_grad_norm_workspace bytes, 16-byte aligned; holds
 *            temporaries of this call alone.
 */
#define MUON_SKIP_NONFINITE 1

size_t muon_grad_norm_workspace(int64_t total_chunks);
muon_status_t muon_grad_norm(const muon_grad_list_t* grads, float max_norm, int flags,
                             muon_step_control_t* control, void* workspace, size_t ws_bytes, void* stream);

/*
 * AdamW ([GUIDE] sections 5 and 6) over many tensors in one launch, whatever
 * their types, each with its own weight decay and learning-rate factor, and
 * with its moments in 32 bits or in 8.
 *
 * The update, in fp32:
 *   g <- scale * g
 *   m <- beta1*m + (1-beta1)*g;   v <- beta2*v + (1-beta2)*g^2
 *   theta <- (1 - l*weight_decay)*theta - l*(m / (1-beta1^t)) / (sqrt(v / (1-beta2^t)) + eps)
 * with l = lr * lr_factor of the tensor.  A BF16 theta is rounded once to
 * nearest even.
 *
 * 32-bit state: m and v are floats, zero before step 1.
 *
 * 8-bit state: m and r = sqrt(v) are e4m3 codes (OCP: 4 exponent and 3
 * mantissa bits, largest value 448), one scale each for every 256
 * consecutive elements: m = scales[2b]*code, r = scales[2b+1]*code for the
 * elements of block b.  All codes and scales are zero before step 1.  After
 * the update a block's scale is its largest |m| (or r) / 448, and
 * y = m / scale (or r / scale) becomes floor(|y|/q + u)*q with y's sign,
 * where q = 2^(max(floor(log2|y|), -6) - 3) is the code step at |y| and u in
 * [0, 1) has 20 random bits, so a code's expected value is y.  (Rounded to
 * nearest, an average with beta2 near 1 would never move: a step changes r by
 * far less than half a code step.)  The mean of y is kept, not that of
 * y^2: v comes out high by r's variance, 5 to 6 % of it with Gaussian
 * gradients.  A positive r keeps at least the smallest
 * code 2^-9: with r = 0 beside m > 0 the next update would be m / eps.  A block
 * whose largest value is below 2^-100 holds zeros.  A gradient that is not
 * finite, or whose square is not, makes its block's scales non-finite, and
 * with them every moment of the block.
 *   The random bits of an element come from `seed`, t and its position
 * counter + i alone: a = mix(floor(position / 16) ^ mix(mix(t) ^ seed)),
 * b = mix(a + 0x6A09E667), s = a + (position mod 16) * b mod 2^32; m takes the
 * bits 31..12 of s, r the bits 31..12 of s rotated by 16.  mix(x):
 * x ^= x >> 16; x *= 0xBB67AE85; x ^= x >> 15; x *= 0x9E3779B9; x ^= x >> 16.
 * 16 elements draw from one arithmetic progression with a random step: any two
 * of them have independent bits for m, and for r independent leading 13 bits
 * (of the bits 4 to 6 of r's 20, the first k are equal in elements whose
 * distance 2^k divides).  m and r of one element have independent leading 16
 * bits (the leading four of each are the last four of the other).
 * Equal inputs give equal bits on every run.
 *
 * State arrays hold numel rounded up to a multiple of MUON_STATE_BLOCK
 * elements; those past numel are zero before step 1 and stay zero.  theta
 * and the gradients end at numel: nothing past it is read or written.
 */
typedef struct muon_param {
  void* param;          /* theta, in/out */
  const void* grad;
  void* m;              /* m as float, or its e4m3 codes, in/out, 16-byte aligned */
  void* v;              /* v as float, or the codes of r, in/out, 16-byte aligned */
  float* scales;        /* 8-bit: float[2 * ceil(numel / 256)], 8-byte aligned; 32-bit: NULL */
  int64_t numel;        /* >= 0; theta and grad are contiguous, aligned to their element size */
  int64_t counter;      /* 8-bit: position of element 0, a multiple of 256 */
  int64_t first_chunk;  /* chunks of the tensors before it in the list */
  float weight_decay;
  float lr_factor;
  int32_t param_dtype;  /* muon_dtype_t; a tensor with another value here or below is left alone */
  int32_t grad_dtype;   /* muon_dtype_t */
  int32_t state_bits;   /* 32 or 8 */
  int32_t reserved;     /* 0 */
} muon_param_t;

#define MUON_PARAM_CHUNK 4096
#define MUON_STATE_BLOCK 256

/* As muon_grad_list, with chunks of MUON_PARAM_CHUNK elements. */
typedef struct muon_param_list {
  int64_t count;
  int64_t total_chunks;        /* 0 .. 2^24-1 */
  const muon_param_t* params;  /* device array [count] */
  const int32_t* chunk_tensor; /* device array [total_chunks] */
} muon_param_list_t;

typedef struct muon_adamw_hyper {
  double lr, beta1, beta2, eps;
  uint32_t seed;     /* of the 8-bit states' rounding */
  uint32_t reserved; /* 0 */
} muon_adamw_hyper_t;

/* step   : t >= 1, and scale = 1 and nothing is skipped, when control is NULL.
 * control: with a control block (DEVICE memory), t, the gradients' scale, the
 *          skip and a further factor of lr are read from it when the kernel
 *          runs, and `step` is not used; a block whose step is below 1 counts
 *          as t = 1.
 * lr finite; beta1, beta2 in [0, 1); eps 0 or in [2^-126, 2^125] (with eps 0
 * an element that has had no gradient yet becomes 0 / 0).
 * No tensor may appear twice or overlap another in the list. */
muon_status_t muon_adamw_multi(const muon_param_list_t* params, const muon_adamw_hyper_t* hyper, int64_t step,
                               const muon_step_control_t* control, void* stream);

/* muon_momentum_packed_grouped and muon_apply_grouped under a control block
 * (DEVICE memory, not NULL): the momentum reads scale * G in place of G, and
 * with skip set the momentum leaves M and the apply leaves W as they are (sumsqs
 * and the Newton-Schulz call between them then come from whatever the workspace
 * held, and nothing takes their results).  Without skip and with scale = 1 the results
 * are those of the plain calls bit for bit.  lr is multiplied by the block's
 * lr_factor. */
muon_status_t muon_momentum_packed_grouped_controlled(int ngroups, const muon_batch_t* grads,
                                                      const muon_batch_t* moms, float* const* sumsqs, float beta,
                                                      int nesterov, int32_t compute, void* workspace,
                                                      size_t ws_bytes, const muon_step_control_t* control,
                                                      void* stream);
muon_status_t muon_apply_grouped_controlled(int ngroups, const muon_batch_t* weights, const muon_batch_t* orthos,
                                            float lr, float weight_decay, int32_t mode, float coeff,
                                            const muon_step_control_t* control, void* stream);

/*
 * SOAP: Adam run in the eigenbasis of Shampoo's row and column statistics
 * ([GUIDE] section 11.1 "SOAP: Adam in Shampoo's eigenbasis" and 11.2;
 * [ZH] section 6.2), for `count` same-shape
 * m x n matrices.  All SOAP state is caller-owned F32 device memory, one
 * muon_batch_t each, with the gradient's count:
 *   L (m x m), R (n x n)   row and column statistics, zero before step 1;
 *   QL (m x m), QR (n x n) their bases, the identity before step 1;
 *   mbar, vbar (m x n)     Adam's moments in the rotated basis, zero before
 *                          step 1.
 * A side passed as NULL (statistic and basis together) keeps the identity
 * basis: an axis too long to precondition ([GUIDE] 11.2).  One update at
 * step t = 1, 2, ... with refresh interval f:
 *   soap_statistics(G, L, R, beta_s);
 *   if ((t - 1) % f == 0) soap_refresh(L, R, QL, QR, mbar, ...);
 *   soap_precondition(G, QL, QR, mbar, vbar, D, t, beta1, beta2, eps, ...);
 *   muon_apply(W, D, lr, weight_decay, MUON_SCALE_NONE, 1, stream);
 * the last line being W <- (1 - lr*wd) W - lr D.  All arithmetic is fp32
 * (the products on the fp32 matrix cores).  The calls enqueue on `stream`
 * and never allocate or synchronize; a workspace (16-byte aligned, of the
 * size its query returns, 0 for arguments out of range) holds temporaries
 * and is free again when the stream reaches the end of the call.
 * Errors: as for the Muon calls (NULL or mismatched descriptors, BF16 where
 * F32 is required, betas outside [0, 1), step < 1, eps not finite or < 0,
 * a short workspace), checked before anything is enqueued.
 */

/* L <- beta_s L + (1-beta_s) G G^T and R <- beta_s R + (1-beta_s) G^T G
 * ([GUIDE] 11.1 first display).  grad: F32 or BF16, m x n.  L or R may be
 * NULL.  Only the upper triangle of the old statistic is read and both
 * triangles are written, so a statistic stays exactly symmetric. */
muon_status_t soap_statistics(const muon_batch_t* grad, const muon_batch_t* L, const muon_batch_t* R,
                              float beta_s, void* stream);

/* soap_statistics for up to 8 groups (shape classes) at once: grads[g] is
 * group g's gradient descriptor and Ls[g], Rs[g] point to its statistics or
 * are NULL.  The products
 * of all groups share launches (one per operand layout, longest reduction
 * first), so small groups fill the chip beside large ones; every statistic
 * is bit-identical to soap_statistics on its group.  The three arrays are
 * host arrays of ngroups entries.  Errors name the group; nothing is
 * enqueued unless every group is valid. */
muon_status_t soap_statistics_grouped(int ngroups, const muon_batch_t* grads, const muon_batch_t* const* Ls,
                                      const muon_batch_t* const* Rs, float beta_s, void* stream);

/* Q factor of a QR factorization, the triangular factor's diagonal made
 * non-negative (unique for a full-rank input): Householder reflections
 * in 16-column panels with blocked trailing updates.  a (read only) and q:
 * F32, n x n, n <= 32768. */
size_t soap_qr_workspace(int64_t count, int64_t n);
muon_status_t soap_qr(const muon_batch_t* a, const muon_batch_t* q, void* workspace, size_t ws_bytes,
                      void* stream);

/* Basis refresh by one power-iteration step plus QR ([GUIDE] 11.2, [ZH]
 * 6.2 step 2): QL <- qr(L QL), QR <- qr(R QR) as soap_qr, and the first
 * moment carried exactly into the new bases ([GUIDE] 11.1 third display):
 * mbar <- QL_new^T QL_old mbar QR_old^T QR_new.  mbar (m x n) gives the
 * shape; a NULL side is left out. */
size_t soap_refresh_workspace(int64_t count, int64_t rows, int64_t cols, int with_l, int with_r);
muon_status_t soap_refresh(const muon_batch_t* L, const muon_batch_t* R, const muon_batch_t* QL,
                           const muon_batch_t* QR, const muon_batch_t* mbar, void* workspace, size_t ws_bytes,
                           void* stream);

/* soap_refresh for up to 8 groups (shape classes) at once: Ls[g], Rs[g],
 * QLs[g], QRs[g] point to group g's descriptors or are NULL for a side
 * without statistic; mbars[g] is group g's first moment.  All QRs of one
 * order, over every group and side, run as one batched factorization. */
size_t soap_refresh_grouped_workspace(int ngroups, const int64_t* counts, const int64_t* rows,
                                      const int64_t* cols, const int* with_l, const int* with_r);
muon_status_t soap_refresh_grouped(int ngroups, const muon_batch_t* const* Ls, const muon_batch_t* const* Rs,
                                   const muon_batch_t* const* QLs, const muon_batch_t* const* QRs,
                                   const muon_batch_t* mbars, void* workspace, size_t ws_bytes, void* stream);

/* [GUIDE] 11.1 between refreshes:
 *   Gbar = QL^T G QR;  mbar <- beta1 mbar + (1-beta1) Gbar;
 *   vbar <- beta2 vbar + (1-beta2) Gbar^2;
 *   D = QL [ (mbar / (1-beta1^t)) / (sqrt(vbar / (1-beta2^t)) + eps) ] QR^T
 * with epsilon after the square root.  grad: F32 or BF16, m x n; QL, QR
 * as above or NULL (identity); mbar, vbar in/out; dir (D, out): F32 m x n,
 * not aliasing the others. */
size_t soap_precondition_workspace(int64_t count, int64_t rows, int64_t cols);
muon_status_t soap_precondition(const muon_batch_t* grad, const muon_batch_t* QL, const muon_batch_t* QR,
                                const muon_batch_t* mbar, const muon_batch_t* vbar, const muon_batch_t* dir,
                                int64_t step, float beta1, float beta2, float eps, void* workspace,
                                size_t ws_bytes, void* stream);

/* soap_precondition for up to 8 groups (shape classes) at once, with one
 * step count and one set of hyperparameters: grads, mbars, vbars and dirs
 * are host arrays of ngroups descriptors, QLs and QRs host arrays of
 * ngroups pointers (NULL: identity).  Each rotation stage launches the
 * products of all groups together; every direction is bit-identical to
 * soap_precondition on its group.  The workspace holds two m x n
 * temporaries per group (the sum of the groups' soap_precondition
 * workspaces).  Errors name the group; nothing is enqueued unless every
 * group is valid. */
size_t soap_precondition_grouped_workspace(int ngroups, const int64_t* counts, const int64_t* rows,
                                           const int64_t* cols);
muon_status_t soap_precondition_grouped(int ngroups, const muon_batch_t* grads, const muon_batch_t* const* QLs,
                                        const muon_batch_t* const* QRs, const muon_batch_t* mbars,
                                        const muon_batch_t* vbars, const muon_batch_t* dirs, int64_t step,
                                        float beta1, float beta2, float eps, void* workspace, size_t ws_bytes,
                                        void* stream);

/* Static text for a status code. */
const char* muon_status_string(muon_status_t status);
/* Thread-local detail of the last non-OK return on this thread ("" if none). */
const char* muon_last_error(void);
/* MUON355_ABI_VERSION of the loaded library. */
int muon_abi_version(void);

/* ------------------------------------------------------------------------
 * Expert layers in 8-bit floating point.
 *
 * What the layers whose matrices the step updates are run with, forward and
 * backward: a weight or an activation as 8-bit codes, the products of such
 * codes (of one matrix, of every expert's, and of the experts' weight
 * gradients, added to the buffers that the step reads), the routing of tokens
 * to experts with the bias that balances it, and the tokens' sums over their
 * experts.
 * ------------------------------------------------------------------------ */

/*
 * A matrix of e4m3 codes (OCP: 4 exponent and 3 mantissa bits, largest value
 * 448) with an fp32 scale for each block of 128 columns of one row
 * (block_rows 1) or of 128 rows (block_rows 128):
 *
 *   value(r, c) = code(r, c) * scales[(c / 128) * scale_ld + r / block_rows]
 *
 * The scales of one block column lie together, as a product reads them.
 * Rows are padded to whole blocks: ld >= cols rounded up to 128, and the codes
 * behind a row's last column, up to the end of its last block, are zero.
 * Everything that writes codes here writes these zeros; products read them.
 */
#define MUON_CODE_BLOCK 128

typedef struct muon_codes {
  void* codes;          /* matrix i at codes + i*stride bytes, 16-byte aligned */
  float* scales;        /* matrix i at scales + i*scale_stride floats */
  int64_t stride;       /* bytes between matrices, a multiple of 16 */
  int64_t scale_stride; /* floats between matrices */
  int64_t count;        /* number of matrices, 1 .. 65535 */
  int64_t rows;         /* 1 .. 2^31 - 128 */
  int64_t cols;         /* 1 .. 2^31 - 128 */
  int64_t ld;           /* bytes between rows, a multiple of 16, below 2^31 */
  int64_t scale_ld;     /* floats between block columns, >= rows / block_rows rounded up */
  int32_t block_rows;   /* 1 or MUON_CODE_BLOCK */
  int32_t reserved;     /* must be 0 */
} muon_codes_t;

/*
 * A matrix, or a batch of them, as codes in its own order (q), as codes of its
 * transpose (qt), or both from one pass over it:
 *
 *   scale = max|x| / 448,   code = round(448 * x / max|x|)   over a block,
 *
 * to nearest, ties to even.  A quotient that fp32 holds is exact before that
 * rounding (so ties are ties), another within its last place.  A block whose
 * largest magnitude is below 2^-100 gets scale 0 and codes 0.  A block that
 * holds a NaN or an infinity gets a scale that is not finite, and every value
 * of it is NaN: products pass it on.
 *
 * x     : BF16 or F32, any alignment of its elements; read only.
 * pairs : NULL, or device int32[n]: row i of the codes is row pairs[i] / k of x,
 *         times weights[pairs[i]] when `weights` is not NULL, and zeros where
 *         pairs[i] < 0 (rows sent to experts, as muon_route lists them).
 *         x->count must be 1, block_rows 1; q has n rows and qt n columns.
 *         A pair behind x's last row gives zeros too, and x may have no rows
 *         at all (0, base NULL).  Without pairs, k is 1 and weights NULL.
 *         A row's weight falls out of the quotients of its own blocks (q); the
 *         scales and the blocks of qt are those of products rounded to fp32.
 * q, qt : either may be NULL; equal counts and block_rows.
 */
muon_status_t muon_block_quantize(const muon_batch_t* x, const int32_t* pairs, const float* weights, int64_t k,
                                  const muon_codes_t* q, const muon_codes_t* qt, void* stream);

/*
 * Products C = A * B^T over codes: A has M rows, B has N, both K columns; C is
 * M x N, row-major, BF16 or F32.  A's blocks have one row, B's one or 128.
 * Sums over a block of 128 are fp32, each is multiplied by the two scales in
 * fp32 and added to an fp32 sum, in an order that depends on the shapes alone:
 * the same call gives the same bits.
 *   BF16 results come from the matrix instruction for 8-bit floats, which drops
 *     what lies 13 bits below the largest of eight neighbouring products: less
 *     than 2^-10 of it in all.  Where the products' signs are mixed at random
 *     that is about 5e-5 of a result's size, a fortieth of its rounding to BF16;
 *     a result that is small because its products cancel may lose more of its
 *     own size (take F32 where that matters).
 *   F32 results (gradients that batches add to) come from the one for BF16, on
 *     codes that BF16 holds exactly: products are exact, sums fp32.
 *
 * MUON_PRODUCT_BATCH : count products; a, b and c have equal counts; offsets
 *   is NULL.
 * MUON_PRODUCT_ROWS  : b holds E matrices, a and c one.  Rows offsets[e] ..
 *   offsets[e+1]-1 of C are those rows of A times B[e]^T.  Rows behind
 *   offsets[E] are left as they were.
 * MUON_PRODUCT_REDUCE: c holds E matrices, a and b one.  C[e] is the product
 *   over columns offsets[e] .. offsets[e+1]-1 alone.  An expert without columns
 *   gets zeros.  Offsets that are multiples of 128 are best: an expert that
 *   starts or ends inside a block of columns shares that block's scales with
 *   its neighbour, its NaN among them, and the block is read for both.
 *   A and B are codes of transposes here: C is a gradient of weights,
 *   rows(A) = outputs, rows(B) = inputs, columns = rows of activations.
 *
 * offsets   : device int32[E+1], ascending, in [0, M] or [0, K].  Values
 *             outside are taken as the nearest bound.
 * accumulate: 1: C += the product (F32 only); an expert without columns is
 *             left as it was.
 * C must not overlap A or B.
 */
typedef enum muon_product {
  MUON_PRODUCT_BATCH = 0,
  MUON_PRODUCT_ROWS = 1,
  MUON_PRODUCT_REDUCE = 2
} muon_product_t;

muon_status_t muon_block_matmul(const muon_codes_t* a, const muon_codes_t* b, const muon_batch_t* c,
                                const int32_t* offsets, int32_t product, int32_t accumulate, void* stream);

/*
 * Routing of tokens to experts.  With the logits z of a token:
 *
 *   s = softmax(z) or sigmoid(z) over the experts;  key = s + bias
 *   the experts are `groups` runs of equal length; a group's mark is the sum of
 *   its group_best (1 or 2) largest keys; the top_groups best groups stay
 *   chosen = the k largest keys of the groups that stay, best first
 *   w_j = scale * s_j, over the sum of the chosen ones' s if `renormalize`
 *         (0 where that sum is 0)
 *
 * The bias chooses and does not weigh.  Of equal keys or marks the lower index
 * comes first.  Keys are compared as if computed exactly, to fp64's rounding;
 * without a bias, in one group or with group_best 1, they are the logits.
 * A logit of -inf takes its expert out; where fewer than k are left the rest
 * of chosen is -1 with weight 0, and so is a token whose mask is 0.  A token
 * with a NaN (or +inf under softmax, or with a NaN bias) goes nowhere: -1, and
 * its weights are NaN, which muon_expert_sum passes on.
 *
 * The order of the (token, j) pairs by expert: expert e's rows are
 * offsets[e] .. offsets[e+1]-1, in the order of the tokens, each expert's rounded up
 * to a multiple of `align` rows (MUON_CODE_BLOCK where weight gradients are
 * taken over them).  slots[t*k+j] is the pair's row or -1, pairs[row] is t*k+j
 * or -1: between an expert's last pair and the next one's first row, and
 * behind offsets[experts].  pairs has muon_route_capacity() elements.
 */
#define MUON_MAX_EXPERTS 512
#define MUON_MAX_CHOSEN 16
#define MUON_MAX_EXPERT_GROUPS 32
#define MUON_MAX_ORDERED_TOKENS 4194304 /* of a call that writes the order or the loads */

typedef enum muon_score { MUON_SCORE_SOFTMAX = 0, MUON_SCORE_SIGMOID = 1 } muon_score_t;

typedef struct muon_route {
  const void* logits;   /* [tokens, experts], aligned to its element size */
  int64_t ld;           /* elements between tokens, >= experts */
  int64_t tokens;       /* >= 1; tokens * k < 2^31 */
  int64_t experts;      /* 1 .. MUON_MAX_EXPERTS */
  int64_t k;            /* 1 .. MUON_MAX_CHOSEN, <= experts of top_groups groups */
  int32_t dtype;        /* muon_dtype_t of the logits */
  int32_t score;        /* muon_score_t */
  int32_t renormalize;  /* 0 or 1 */
  int32_t groups;       /* 1 .. MUON_MAX_EXPERT_GROUPS, divides experts */
  int32_t top_groups;   /* 1 .. groups */
  int32_t group_best;   /* 1 or 2 */
  int32_t align;        /* 1 .. 65536 */
  float scale;          /* finite */
} muon_route_t;

/* Rows of the order: tokens*k + experts*(align-1), rounded up to a multiple of
 * align; 0 for arguments that muon_route refuses. */
int64_t muon_route_capacity(int64_t tokens, int64_t experts, int64_t k, int64_t align);
/* Bytes of device workspace of muon_route; enough for fewer tokens or experts too. */
size_t muon_route_workspace(int64_t tokens, int64_t experts);

/*
 * bias   : device float[experts] or NULL.  mask: device uint8[tokens] or NULL.
 * chosen : int32[tokens*k], weights: float[tokens*k], written.
 * slots  : int32[tokens*k], pairs: int32[capacity], offsets: int32[experts+1],
 *          written; all three or none (NULL).
 * loads  : int32[experts] or NULL: each expert's pairs are added (micro-batches
 *          of a step add up; the caller keeps the sums below 2^31).
 * workspace: at least muon_route_workspace bytes, 16-byte aligned; holds
 *          temporaries of this call alone.
 */
muon_status_t muon_route(const muon_route_t* r, const float* bias, const uint8_t* mask, int32_t* chosen,
                         float* weights, int32_t* slots, int32_t* pairs, int32_t* offsets, int32_t* loads,
                         void* workspace, size_t ws_bytes, void* stream);

/*
 * Gradient of the logits from the gradient of the weights, with chosen and
 * weights as muon_route wrote them for the same description (its groups, bias
 * and mask only chose).  grad_logits: [tokens, experts] of the logits' type,
 * ld_grad elements between tokens, written whole.  A NaN in a token's weights,
 * or in the gradient of one that has an expert, makes its row NaN.  A token
 * without experts and with weights 0 gets zeros, whatever its logits are.
 */
muon_status_t muon_route_backward(const muon_route_t* r, const int32_t* chosen, const float* weights,
                                  const float* grad_weights, void* grad_logits, int64_t ld_grad, void* stream);

/*
 * The bias's own step, once an optimizer step: bias[e] += rate where the
 * expert's load lies below the mean, -= rate where it lies above (compared in
 * integers), and the loads start again from 0.  With several GPUs the loads
 * are summed over them before.  With `control` a step that skips leaves the
 * bias as it is (the loads start again all the same).  rate: finite, >= 0.
 */
muon_status_t muon_balance_update(float* bias, int32_t* loads, int64_t experts, float rate,
                                  const muon_step_control_t* control, void* stream);

/*
 * Each token's sum over its experts' rows: out[t] = sum over j, in its order,
 * of weights[t*k+j] * y[slots[t*k+j]], in fp32, rounded once (BF16 or F32,
 * whichever y has).  A slot that is negative or behind y's last row counts as
 * a row of zeros.  weights may be NULL (ones).  y and out: one matrix each,
 * equal cols; out has a row for each token and must not overlap y.
 * k: 1 .. MUON_MAX_CHOSEN.
 */
muon_status_t muon_expert_sum(const muon_batch_t* y, const int32_t* slots, const float* weights, int64_t k,
                              const muon_batch_t* out, void* stream);

/*
 * The gradient of those weights: dots[t*k+j] = <grad[t], y[slots[t*k+j]]> in
 * fp32, 0 where the slot has no row.  (The gradient of y is grad's rows in the
 * order of the pairs, times the weights: muon_block_quantize makes its codes.)
 */
muon_status_t muon_expert_dot(const muon_batch_t* grad, const muon_batch_t* y, const int32_t* slots, int64_t k,
                              float* dots, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MUON355_H */
