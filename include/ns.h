/*
 * ns.h -- C ABI of libns, batched quintic Newton-Schulz orthogonalization on
 * one GB300 (sm_103a).
 *
 * The operation. For every matrix X (M x N, row-major) of a batch:
 *     X <- X / (||X||_F + eps)
 *     work on W = X^T when M > N (W is m x n, m = min(M,N), n = max(M,N))
 *     repeat `steps` times:  A = W W^T;  B = b*A + c*A*A;  W = a*W + B*W
 *     write W back into X (transposed back when M > N).
 * The three pages this library follows -- "Fix megabatch_orthogonalize_async
 * hang on empty FSDP2 shards" (microsoft/dion), "Balance LayerWise optimizer
 * shards by Newton-Schulz cost, not parameter size" (Megatron-LM) and the
 * xtuner Muon remainder-strategy PR -- run this iteration on stacks of
 * same-shape 2-D momentum matrices but never print it; the form and the
 * default coefficients (a,b,c) = (3.4445, -4.7750, 2.0315), 5 steps and
 * eps = 1e-7 are Muon's standard quintic Newton-Schulz. The megabatch layout
 * (a stack of same-shape matrices, per-rank zero padding) is the first page's
 * "Concrete repro" and "Fix" sections; its "Fix" section also states the
 * invariant that zero rows stay zero, which lets the library skip padded rows
 * and columns instead of computing them. The cost model is the second page's
 * "Changes" item 1.
 *
 * Conventions for every call:
 *  - Pointers named X / X_host are caller-owned. Device pointers must be on
 *    the current CUDA device. Nothing is retained after the call returns,
 *    except the library's internal workspace cache (see ns_release_workspace).
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream). All device work is stream-ordered on it; calls do not
 *    synchronise unless stated. The workspace cache goes by the handle (for
 *    cudaStreamPerThread, by the thread's stream): before a stream with work
 *    of this library in flight is destroyed, wait for it, as another stream
 *    may get the same handle.
 *  - Return value: NS_OK (0) or a negative NS_E* code. Arguments are
 *    validated before anything is launched; on a validation error nothing
 *    runs and the matrices are untouched. No C++ exception crosses the ABI.
 *  - CUDA graphs: once ns_orthogonalize_batched (or _sched) has run with the
 *    same matrices, shapes, steps, coefficients and stream, a repeat call
 *    allocates nothing and uploads nothing, so it may be captured into a
 *    graph on that stream and replayed. The library keeps the descriptor
 *    tables of the last 8 distinct batches per stream on the device, so a
 *    caller alternating between a few batches (e.g. remainder batches) also
 *    uploads nothing after the first call of each. What a captured call uses
 *    of the workspace cache stays allocated for its graph until
 *    ns_release_workspace, whatever later calls on that stream need. All
 *    calls on one stream share that scratch, the captured ones among them:
 *    replays of graphs captured on a stream must not run at the same time as
 *    one another or as later calls on that stream (replay them on it, or order
 *    them otherwise).
 */
#ifndef NS_H_
#define NS_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* element types of X */
#define NS_F32 0  /* float32 in, float32 out, fp32-accurate arithmetic throughout (see ns_set_f32_gemm) */
#define NS_BF16 1 /* bfloat16 in/out; bf16 tensor-core operands, fp32 accumulation */

/* status codes */
#define NS_OK 0
#define NS_EINVAL (-1)   /* null pointer, negative dims/count/steps, bad dtype, a side above
                            2^30 - 1 or a matrix above 2^40 elements (training operators: the
                            limits they state), overlapping matrices */
#define NS_EALIGN (-2)   /* a pointer is not aligned to its element size (8-bit checkpoints: 16 bytes) */
#define NS_ENOMEM (-3)   /* workspace allocation failed / caller workspace too small */
#define NS_ECUDA (-4)    /* a CUDA runtime or driver call failed */
#define NS_ETIMEOUT (-5) /* a bounded device-side wait gave up (reported by ns_get_status) */
#define NS_ENODEV (-6)   /* no CUDA driver or device, or the current device is not sm_100-family */
#define NS_ETOOBIG (-7)  /* batch needs more scratch than ns_orthogonalize_batched_noalloc holds */
#define NS_EBOUNDS (-8)  /* a debug build's bounds check caught a store (reported by ns_get_status) */

/*
 * ns_orthogonalize_batched -- Newton-Schulz of `count` matrices, in place.
 *   X       host array of `count` device pointers; X[i] points at a
 *           contiguous row-major matrix of shapes[2i] x shapes[2i+1]
 *           elements of `dtype`. Matrices may differ in shape; a zero
 *           dimension makes that matrix a no-op. Matrices must not overlap
 *           (checked: overlapping ranges give NS_EINVAL).
 *   shapes  host array of 2*count int64 (M, N) pairs, read before return.
 *   count   number of matrices (0 is valid and does nothing).
 *   steps   number of iterations (>= 0; 0 = normalisation only).
 *   coeffs  NULL for (3.4445, -4.7750, 2.0315), else a host array of three
 *           floats (a, b, c) used by every step.
 *   dtype   NS_F32 or NS_BF16.
 *   stream  cudaStream_t.
 * eps is 1e-7. Work is scheduled largest ns_cost first. Scratch memory comes
 * from an internal per-(device, stream) workspace that grows on demand with
 * stream-ordered allocation.
 */
int ns_orthogonalize_batched(void *const *X, const int64_t *shapes, int count, int steps,
                             const float *coeffs, int dtype, void *stream);

/*
 * ns_orthogonalize_batched_ex -- as above, with an explicit eps and an
 * explicit caller-owned device workspace of at least
 * ns_workspace_bytes(shapes, count, dtype) bytes (256-byte aligned). The
 * workspace must not be used by anything else until the stream has passed
 * this call's work. Returns NS_ENOMEM if it is too small.
 */
int ns_orthogonalize_batched_ex(void *const *X, const int64_t *shapes, int count, int steps,
                                const float *coeffs, float eps, int dtype, void *workspace,
                                size_t workspace_bytes, void *stream);

/*
 * ns_orthogonalize_batched_sched -- as ns_orthogonalize_batched, but step s
 * uses its own coefficients: coeff_table is a host array of steps x 3 floats,
 * row s = (a, b, c) of step s, read before return; 1 <= steps <= 32 (0 steps
 * is normalisation only and reads no table). The pages print no schedule;
 * this serves coefficient schedules that change from step to step.
 * Returns NS_EINVAL for a NULL table or more than 32 steps.
 */
int ns_orthogonalize_batched_sched(void *const *X, const int64_t *shapes, int count, int steps,
                                   const float *coeff_table, int dtype, void *stream);

/* Device workspace bytes the _ex call needs for this batch (0 on bad input). */
size_t ns_workspace_bytes(const int64_t *shapes, int count, int dtype);

/*
 * ns_orthogonalize_batched_host -- the same operation on HOST matrices:
 * copies each X_host[i] to the device, runs the method, copies the results
 * back into X_host[i] and returns once they are there. The batch is split into
 * up to 8 contiguous groups of about equal bytes, each of at least 32 MiB
 * (a smaller batch is one group); the copies in of group g+1,
 * the Newton-Schulz of group g and the copies out of group g-1 overlap on
 * library-owned streams ordered by events (even groups compute on `stream`,
 * odd groups on a second library stream, so one group's last partial wave of
 * tiles overlaps the next group's first; under NS_SCHED_SINGLE every group
 * computes on `stream`). Host buffers may be
 * pageable or pinned (only pinned buffers let the copies overlap). Device
 * copies and workspaces are part of the internal per-(device, stream) cache.
 */
int ns_orthogonalize_batched_host(void *const *X_host, const int64_t *shapes, int count,
                                  int steps, const float *coeffs, int dtype, void *stream);

/*
 * ns_orthogonalize_batched_noalloc -- the same operation as
 * ns_orthogonalize_batched (same arguments, eps = 1e-7) for callers that
 * cannot allocate device memory: processes whose framework allocator has
 * already reserved nearly all of HBM, optimizer steps that cannot absorb an
 * allocator's synchronisation, runtimes that forbid allocation after
 * start-up. It calls no cudaMalloc, cudaFree or other allocating routine; its
 * scratch is one fixed 256 MiB device array inside the library, reserved on
 * every device that loads the library until the process exits.
 *   - A batch whose ns_workspace_bytes exceeds 256 MiB is rejected with
 *     NS_ETOOBIG before anything runs (e.g. one 4096 x 4096 bf16 matrix
 *     fits; one 8192 x 6144 does not).
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current; make that first call
 *     before any stream capture.
 *   - Every call shares the one array and leaves its contents behind; each
 *     call clears what must start at zero itself. Calls that overlap on the
 *     GPU (other streams, other host threads) race on the array: serialise
 *     them.
 * The pages have no counterpart of this entry point; it exists for callers
 * of this library that cannot allocate.
 */
int ns_orthogonalize_batched_noalloc(void *const *X, const int64_t *shapes, int count, int steps,
                                     const float *coeffs, int dtype, void *stream);

/*
 * ns_muon_update_batched -- one optimizer step around the orthogonalization,
 * for `count` matrices: the momentum step, Newton-Schulz and a scaled write
 * of the result. The dion page's "Summary" names Muon, NorMuon and Dion2 as
 * the optimizers that run the megabatch Newton-Schulz on momentum matrices;
 * the pages do not print their updates, so every constant here is a
 * parameter. For each matrix i, with every buffer M x N row-major of `dtype`
 * on the current device:
 *     Mom[i] <- mu * Mom[i] + G[i]                       (stored in Mom[i])
 *     X      <- G[i] + mu * Mom[i]   if nesterov, else Mom[i]
 *     Out[i] <- scale * NS(X)         (NS as ns_orthogonalize_batched, eps 1e-7)
 *   G       host array of count device pointers: gradients, read only
 *   Mom     host array of count device pointers: momentum buffers, updated
 *   Out     host array of count device pointers: where the update is written;
 *           Out[i] may be G[i] itself (the gradient buffer is overwritten)
 *   shapes, count, steps, coeffs, dtype, stream: as ns_orthogonalize_batched
 *   mu, scale  finite floats; nesterov 0 or 1.
 * One element-wise kernel does the momentum step and writes X into Out (bf16:
 * Mom and X rounded to nearest even, arithmetic in fp32); the Newton-Schulz
 * call then works on Out in place, and `scale` is applied inside its last
 * step before the final rounding. Buffers of the batch must not overlap,
 * except Out[i] == G[i] (NS_EINVAL otherwise, before anything runs). Other
 * returns as ns_orthogonalize_batched.
 */
int ns_muon_update_batched(void *const *G, void *const *Mom, void *const *Out, const int64_t *shapes,
                           int count, int steps, const float *coeffs, float mu, int nesterov,
                           float scale, int dtype, void *stream);

/* ------------------------------------------------------------------------
 * Operators of the training step around the optimizer: the token embedding
 * and its gradient, the clipped policy loss on logits, activations held for
 * the backward pass in 8 bits, and the weight gradients formed from them
 * (the matrices ns_muon_update_batched takes as G).
 *
 * The conventions at the top of this file hold: device pointers on the
 * current device, stream-ordered, no synchronisation, validated before
 * anything is launched. Matrices are row-major with a row pitch ld_* in
 * elements (at least the row's length; no other requirement: rows and bases
 * need only their element's alignment, 16-byte aligned ones are faster).
 * dtype NS_F32 or NS_BF16; arithmetic and every sum in fp32, each output
 * rounded once. Results are the same bits from call to call: no sum's order
 * depends on the schedule. Outputs must not overlap inputs or each other
 * unless stated (NS_EINVAL); column ranges of one buffer, with its pitch, do
 * not. Scratch comes from the internal per-(device,
 * stream) workspace cache, one block per operator that grows to the largest
 * call: ns_embed_grad of more than 1024 ids 16 bytes an id and 8 bytes a column
 * for every 16 to 64 ids, ns_policy_loss 4 bytes a row, ns_ckpt_wgrad 2 bytes
 * per value of X, 2 (bf16 that TMA cannot address) or 6 (fp32) per value of
 * dY, and 4 per value of G and part when the rows are split between CTAs; the
 * others none. Once a call of the same sizes has run on a stream, a repeat
 * allocates nothing and may be captured into a CUDA graph, on the terms at the
 * top of this file.
 */

/* types of token ids and targets */
#define NS_I32 0
#define NS_I64 1

/*
 * ns_embed_lookup -- Out[t, :] = scale * Table[ids[t], :] for `count` ids.
 *   table  vocab x dim of dtype; ids: count integers of id_type on the device;
 *   out    count x dim of dtype.
 * An id outside [0, vocab) is padding: its row of Out is zero. dim < 2^30;
 * here and below, other sides and pitches are at most 2^31 - 1 and 2^31 unless
 * stated, and a matrix spans at most 2^46 elements.
 */
int ns_embed_lookup(const void *table, int64_t ld_table, int64_t vocab, int64_t dim, const void *ids, int id_type,
                    int64_t count, float scale, void *out, int64_t ld_out, int dtype, void *stream);

/*
 * ns_embed_grad -- gradient of ns_embed_lookup with respect to the table:
 *     S[v, :] = scale * sum over t with ids[t] == v of dOut[t, :]
 *     Grad    = S                 accumulate 0: every row written, zero where no id points
 *     Grad   += S                 accumulate 1: only the rows that an id points to are touched
 *   dout   count x dim of dtype;  grad  vocab x dim of grad_dtype (NS_F32 or
 *   NS_BF16, whatever dtype is).
 * Sums run in fp32 over the positions in a fixed order and are rounded once.
 * Ids outside [0, vocab) have no gradient; their rows of dOut are not read.
 * count <= 2^30, vocab < 2^31 - 1, dim <= 2^24, (count / 16 + 1) *
 * (dim / 128 + 1) < 2^31 (count * dim up to about 2^42).
 */
int ns_embed_grad(const void *dout, int64_t ld_dout, const void *ids, int id_type, int64_t count, float scale,
                  void *grad, int64_t ld_grad, int64_t vocab, int64_t dim, int dtype, int grad_dtype, int accumulate,
                  void *stream);

/*
 * ns_token_logprobs -- logp[t] = z[y] - log sum_j exp z[j] with z =
 * Logits[t, :] * inv_temperature and y = targets[t], for `rows` rows of
 * `vocab` logits. A row whose target is outside [0, vocab) is masked: its
 * logits are not read and its logp is 0. A row of logits that are all
 * -infinity holds no distribution and gives 0 as well. logp: rows floats.
 * vocab < 2^30 (ns_policy_loss too).
 */
int ns_token_logprobs(const void *logits, int64_t ld_logits, int64_t rows, int64_t vocab, const void *targets,
                      int id_type, float inv_temperature, float *logp, int dtype, void *stream);

/*
 * ns_policy_loss -- clipped policy loss with a KL term, and its gradient with
 * respect to the logits. With logp as ns_token_logprobs, per row t:
 *     r    = exp(logp - old_logp)                (1 when old_logp is NULL)
 *     gain = min(r A, clip(r, 1 - clip_low, 1 + clip_high) A),  A = advantage
 *     k    = exp(ref_logp - logp) - (ref_logp - logp) - 1   (0 when ref_logp is NULL)
 *     loss = sum over rows of weight * (kl_coef * k - gain)
 *     g    = weight * inv_temperature *
 *            ((r A <= clipped r A ? -r A : 0) + kl_coef * (1 - exp(ref_logp - logp)))
 *     dLogits[t, j] = g * ((j == y) - softmax(z)[j])
 *   targets    rows integers of id_type; old_logp, ref_logp (either may be
 *              NULL), advantage, weight: rows floats
 *   loss       one float; logp, kl: rows floats (kl[t] = k)
 *   dlogits    rows x vocab of dtype; NULL for no gradient; may be logits
 *              itself (same pointer and pitch: the gradient written over them)
 * A row is masked when its target is outside [0, vocab), its weight is 0 or its
 * logits are all -infinity: it adds nothing to the loss, its logp and kl are
 * 0, its gradient row is zero, and (but for the last case) its logits and its
 * other inputs are not looked at, whatever they hold. A NaN in any input of
 * another row makes the loss and the row's gradient NaN; but with kl_coef 0 the
 * KL term has no part in them, whatever k is, and is only written. kl_coef,
 * clip_low, clip_high finite and >= 0, inv_temperature finite and > 0.
 */
int ns_policy_loss(const void *logits, int64_t ld_logits, int64_t rows, int64_t vocab, const void *targets,
                   int id_type, const float *old_logp, const float *ref_logp, const float *advantage,
                   const float *weight, float inv_temperature, float clip_low, float clip_high, float kl_coef,
                   float *loss, float *logp, float *kl, void *dlogits, int64_t ld_dlogits, int dtype, void *stream);

/*
 * Activations held in 8 bits ("checkpoints"). A rows x cols matrix is held
 * as int8 values and one scale byte per block of 32 consecutive values of a
 * row (the last block of a row may be shorter):
 *     E     = exponent field of the block's largest magnitude as a float32, at least 7
 *     q     = x * 2^(133 - E) rounded half to even, at most 127 in magnitude
 *     value = q * 2^(E - 133)
 * The scale is a power of two, so q comes without a division and every value
 * is exact in bf16 (7 magnitude bits): the backward pass can feed it to the
 * tensor cores as it is. The error is at most half a unit, 1/128 of the
 * block's largest magnitude, (for magnitudes that round to 128 units: one
 * unit). A block that holds an infinity or NaN has E = 255 and reads back as
 * NaN throughout.
 *   q       rows x ns_ckpt_pitch(cols) bytes; bytes beyond cols are 0
 *   scales  rows x ns_ckpt_scale_pitch(cols) bytes; beyond the last block 0
 * Both 16-byte aligned (NS_EALIGN). cols <= 2^30.
 */
int64_t ns_ckpt_pitch(int64_t cols);       /* cols rounded up to a multiple of 16; -1 if negative */
int64_t ns_ckpt_scale_pitch(int64_t cols); /* ceil(cols / 32) rounded up to a multiple of 4 */

/* ns_ckpt_store -- hold X in 8 bits.  ns_ckpt_load -- Out = the values held. */
int ns_ckpt_store(const void *x, int64_t ld_x, int64_t rows, int64_t cols, void *q, void *scales, int dtype,
                  void *stream);
int ns_ckpt_load(const void *q, const void *scales, int64_t rows, int64_t cols, void *out, int64_t ld_out, int dtype,
                 void *stream);

/*
 * ns_gated_forward -- H = silu(Gate) * Up, silu(x) = x / (1 + exp(-x)), and
 * Gate and Up held in 8 bits for the backward pass, in one pass over both.
 * All rows x cols; gate and up share the pitch ld_in, so they may be the two
 * halves of one rows x 2 cols matrix.
 */
int ns_gated_forward(const void *gate, const void *up, int64_t ld_in, int64_t rows, int64_t cols, void *h, int64_t ld_h,
                     void *q_gate, void *s_gate, void *q_up, void *s_up, int dtype, void *stream);

/*
 * ns_gated_backward -- from dH and the values g, u that the two checkpoints
 * hold: dGate = dH u s (1 + g (1 - s)), dUp = dH g s, with s = 1 / (1 +
 * exp(-g)); and, unless h is NULL, H = g s u again (the input of the next
 * layer's weight gradient). dgate and dup share the pitch ld_d.
 */
int ns_gated_backward(const void *dh, int64_t ld_dh, const void *q_gate, const void *s_gate, const void *q_up,
                      const void *s_up, int64_t rows, int64_t cols, void *dgate, void *dup, int64_t ld_d, void *h,
                      int64_t ld_h, int dtype, void *stream);

/*
 * ns_ckpt_wgrad -- weight gradients from an input held in 8 bits. With X the
 * rows x n_in values of the checkpoint and dY rows x n_out:
 *     G[e] (+)= sum over rows t of group e of dY[t, :]^T X[t, :]      (n_out x n_in)
 *   offsets  groups + 1 ascending int32 on the device: group e is rows
 *            [offsets[e], offsets[e+1]) (values are clamped to [0, rows]);
 *            NULL with groups = 1 for all rows. A group without rows gives 0.
 *   grad     groups x n_out x n_in of grad_dtype, contiguous: a stack of
 *            matrices as ns_muon_update_batched takes them
 *   accumulate  0: G is overwritten; 1: the sum is added to it
 * dY of dtype: bf16, or fp32 (held as three bf16 slices inside, so products
 * are exact to 2^-24). Rows of other groups never reach a group's sum,
 * whatever they hold. Sums in fp32: the tensor cores' accumulators are added
 * to fp32 registers every 512 rows (their own sum loses up to a unit in the
 * last place per instruction). rows, n_out and n_in <= 2^30, groups * n_out *
 * n_in <= 2^42.
 */
int ns_ckpt_wgrad(const void *dy, int64_t ld_dy, int64_t rows, int64_t n_out, const void *q, const void *scales,
                  int64_t n_in, const int32_t *offsets, int groups, void *grad, int dtype, int grad_dtype,
                  int accumulate, void *stream);

/*
 * Operators of an expert layer. As the operators above: the checks come before
 * any launch, work is ordered on `stream`, nothing synchronises. Scratch, where
 * a call needs some, is the caller's (device memory, no initial values needed),
 * so calls captured into different graphs share none; nothing is allocated.
 */

/*
 * ns_route -- the router: for each of `rows` rows of `experts` logits l (pitch
 * ld_logits) the top_k experts of largest l, ties to the lower index, with the
 * weights softmax(l) (renormalise = 1: divided by the sum of the chosen ones).
 *   live       NULL, or rows bytes: a row with 0 is padding, it is not read
 *   ids        rows x top_k experts, largest logit first; -1 where none is left
 *              (logits of -infinity are never chosen) and in rows of padding; a
 *              row of -infinity alone counts as padding
 *   weights    rows x top_k floats, 0 where the id is -1
 *   logz       rows floats, log sum exp l (0 for padding)
 *   counts     experts: slots of each;  offsets: experts + 1, their running sum
 *   order      rows x top_k: the slots (row * top_k + place) in the experts'
 *              order, ascending within an expert, then -1
 *   live_rows  one int: T, the rows that are not padding
 *   loss       one float: balance_coef * experts / (top_k T^2) * sum_e counts[e] *
 *              (sum over rows of softmax(l)[e]) + z_coef / T * sum of logz^2 (T = 0: 0;
 *              squares in fp32, infinite from |logz| = 1.8e19 on; z_coef = 0 leaves them out)
 * A NaN orders above every number; a NaN or +infinity in a row makes its
 * weights, its logz and the loss NaN. offsets is what ns_blocks_matmul and
 * ns_ckpt_wgrad take, order what ns_blocks_store_rows takes (per = top_k).
 * experts <= 1024, top_k <= 32 and <= experts, rows * top_k <= 2^30. workspace:
 * ns_route_workspace(rows, experts) bytes, 4-byte aligned (less: NS_ENOMEM).
 */
int64_t ns_route_workspace(int64_t rows, int experts); /* -1 for bad sizes */
int ns_route(const void *logits, int64_t ld_logits, int64_t rows, int experts, int top_k, const uint8_t *live,
             int renormalise, float balance_coef, float z_coef, int32_t *ids, float *weights, float *logz,
             int32_t *counts, int32_t *offsets, int32_t *order, int32_t *live_rows, float *loss, void *workspace,
             size_t workspace_bytes, int dtype, void *stream);

/*
 * ns_route_backward -- the logits' gradient of the loss (its own gradient 1)
 * and of the weights, dweights (rows x top_k, NULL: none; without effect where the
 * id is -1). ids, weights, logz, counts, live_rows and the coefficients as ns_route
 * gave and got them; counts are taken as constants. With p = softmax(l) and s[e] =
 * balance_coef * experts * counts[e] / (top_k T^2):
 *     dl = p (s - sum p s + 2 z_coef logz / T) + the weights' part:
 *     renormalise 1: w (dw - sum w dw) at the chosen; 0: dw joins s at the chosen
 * Rows of padding get zeros. dlogits may be logits itself (same pitch).
 */
int ns_route_backward(const void *logits, int64_t ld_logits, int64_t rows, int experts, int top_k, const int32_t *ids,
                      const float *weights, const float *dweights, const float *logz, const int32_t *counts,
                      const int32_t *live_rows, int renormalise, float balance_coef, float z_coef, void *dlogits,
                      int64_t ld_dlogits, int dtype, void *stream);

/*
 * Matrices held in 8-bit floating point ("blocks"): e4m3 values q with one scale
 * byte s per block of 128 values of a row ("rows") or of 128 x 128 values
 * ("tiles"; blocks at a matrix's ends are smaller):
 *     value = q * 2^(s - 127)
 *     s     = smallest >= 1 with (largest magnitude of the block) <= 448 * 2^(s - 127)
 *     q     = x * 2^(127 - s) rounded to e4m3, half to even
 * A block that holds an infinity or NaN has s = 255 and reads back as NaN
 * throughout. The scale is a power of two, so x is rounded once; a magnitude
 * that rounds to 2^128 (from 1.9375 * 2^127 on) reads back as infinity.
 *   q       rows x ns_blocks_pitch(cols) bytes; bytes beyond cols are 0
 *   scales  rows x ns_blocks_scale_pitch(cols) bytes; for tiles one such row for
 *           every 128 rows of a matrix, counted anew for each of a stack; 0 beyond
 * Both 16-byte aligned (NS_EALIGN). cols < 2^30.
 */
int64_t ns_blocks_pitch(int64_t cols);       /* cols rounded up to a multiple of 16; -1 if negative */
int64_t ns_blocks_scale_pitch(int64_t cols); /* ceil(cols / 128) rounded up to a multiple of 4 */

/* ns_blocks_store_rows -- rows of X with a scale per 128 values. With index
 * (`rows` int32 on the device) row r holds X[index[r] / per], a row of zeros where
 * index[r] is negative or beyond x_rows; without, rows = x_rows and per = 1. */
int ns_blocks_store_rows(const void *x, int64_t ld_x, int64_t x_rows, const int32_t *index, int per, int64_t rows,
                         int64_t cols, void *q, void *scales, int dtype, void *stream);
/* ns_blocks_store_tiles -- a stack of `groups` matrices of rows x cols (one
 * behind the other, all rows ld_x apart) with a scale per 128 x 128 values. */
int ns_blocks_store_tiles(const void *x, int64_t ld_x, int groups, int64_t rows, int64_t cols, void *q, void *scales,
                          int dtype, void *stream);
/* ns_blocks_load -- Out = the values held (groups * rows rows; groups = 1 unless tiles). */
int ns_blocks_load(const void *q, const void *scales, int tiles, int groups, int64_t rows, int64_t cols, void *out,
                   int64_t ld_out, int dtype, void *stream);

/*
 * ns_blocks_matmul -- the product of such matrices, A (rows x k, rows form) and
 * a stack of W (tiles form):
 *     back = 0: Out[t] = A[t] W[e]^T, W[e] n x k      (a layer, forward)
 *     back = 1: Out[t] = A[t] W[e],   W[e] k x n      (its input's gradient)
 * for the rows t of group e.
 *   offsets  groups + 1 ascending int32 on the device, as for ns_ckpt_wgrad:
 *            group e is rows [offsets[e], offsets[e+1]); rows of no group become
 *            zeros. NULL with groups = 1 for all rows.
 *   out      rows x n of dtype
 * The tensor cores apply the scales and add up to 1024 products along k in their
 * fp32 accumulators, which may lose a unit in the last place for every 32 products:
 * less than 2^-17 of the sum of the products' magnitudes for k <= 32768 (2^-21
 * measured, products of one sign). Accumulators are added in fp32 registers, the
 * result is rounded once.
 * rows, n and k <= 2^30, groups <= 2^20, groups * n * k <= 2^42.
 */
int ns_blocks_matmul(const void *qa, const void *sa, int64_t rows, int64_t k, const void *qw, const void *sw, int64_t n,
                     int back, const int32_t *offsets, int groups, void *out, int64_t ld_out, int dtype, void *stream);

/*
 * ns_block_norm -- the norms after and before a block, with the block's gate
 * and the residual scale, in one pass. Per row, with mean over cols:
 *     u = Y * rsqrt(mean Y^2 + eps) * post   (post NULL: u = Y)
 *     R = a X + b gate u                     (Y NULL: R = a X)
 *     Z = R * rsqrt(mean R^2 + eps) * pre    (pre NULL: no Z), from R before it is rounded
 *   x, r   rows x cols of dtype, the residual stream
 *   y, z   rows x cols of block_dtype: the block's output, the next block's input;
 *          block_dtype may be bf16 beside an fp32 dtype, not the other way round
 *   gate   gate_dtype; gate_form NS_GATE_NONE (NULL, 1), NS_GATE_COLS (cols values),
 *          NS_GATE_ROWS (one value a row, ld_gate apart), NS_GATE_FULL (rows x cols)
 *   post, pre   cols values of weight_dtype
 *   post_rstd, pre_rstd   rows floats for the backward pass (where post / pre)
 * r may be x and z may be y (same pitch). cols <= 16384. Y or pre must be given.
 * Squares are summed in fp32: a row whose sum is beyond it (magnitudes from about
 * 1.8e19 / sqrt(cols) on) counts as infinitely long, and its norm is 0.
 */
#define NS_GATE_NONE 0
#define NS_GATE_COLS 1
#define NS_GATE_ROWS 2
#define NS_GATE_FULL 3
int ns_block_norm(const void *x, int64_t ld_x, const void *y, int64_t ld_y, const void *gate, int gate_form,
                  int64_t ld_gate, const void *post, const void *pre, int64_t rows, int64_t cols, float a, float b,
                  float eps, void *r, int64_t ld_r, void *z, int64_t ld_z, float *post_rstd, float *pre_rstd, int dtype,
                  int block_dtype, int weight_dtype, int gate_dtype, void *stream);

/*
 * ns_block_norm_backward -- from dR (NULL: zero, only with pre) and dZ: dX, dY, the
 * gate's gradient in the gate's form, and dpost, dpre (weight_dtype). X, Y, gate, post,
 * pre, a and b as given to ns_block_norm (copies of X and Y where that wrote over
 * them), whose rstd's it takes; R is formed again from them, and without pre X is
 * not read. dx may be dR and dy may be dZ (same type and pitch). Sums over rows
 * are taken in fp32 in a fixed order. workspace: ns_block_norm_workspace(rows, cols)
 * bytes, 4-byte aligned (less: NS_ENOMEM).
 */
int64_t ns_block_norm_workspace(int64_t rows, int64_t cols); /* -1 for bad sizes */
int ns_block_norm_backward(const void *dr, int64_t ld_dr, const void *dz, int64_t ld_dz, const void *x, int64_t ld_x,
                           const void *y, int64_t ld_y, const void *gate, int gate_form, int64_t ld_gate,
                           const void *post, const void *pre, const float *post_rstd, const float *pre_rstd,
                           int64_t rows, int64_t cols, float a, float b, void *dx, int64_t ld_dx, void *dy,
                           int64_t ld_dy, void *dgate, int64_t ld_dgate, void *dpost, void *dpre, void *workspace,
                           size_t workspace_bytes, int dtype, int block_dtype, int weight_dtype, int gate_dtype,
                           void *stream);

/*
 * ns_dropout -- Out = [residual +] X with a share `prob` of its elements dropped
 * and the others divided by the share that stays. The mask is drawn, not
 * stored: the same call on the gradient is the backward pass.
 * Eight consecutive columns of a row share a counter n = offset + row *
 * ceil(cols / 8) + column / 8 (mod 2^64). Philox4x32-10 with the key `seed` and the
 * counter words (n mod 2^32, n / 2^32, 0, 0) gives eight 16-bit numbers h, a word's
 * low half first; with (.., .., 1, 0) eight more, l. An element is dropped when
 * h * 65536 + l < limit = round(prob * 2^32), the others are multiplied by 2^32 /
 * (2^32 - limit), rounded to fp32; with a residual the product and the sum take one
 * rounding in fp32. A call uses rows * ceil(cols / 8) counters.
 *   state     NULL, or {seed, offset} on the device (two 64-bit numbers, 8-byte
 *             aligned) added to the arguments: a captured call draws anew when
 *             they change
 *   residual  NULL, or rows x cols of out_dtype
 *   out       rows x cols of out_dtype: dtype, or fp32 with a residual; may be x
 *             or residual (same type and pitch)
 * A dropped element has no part in the result, whatever it holds. prob in [0, 1].
 */
int ns_dropout(const void *x, int64_t ld_x, const void *residual, int64_t ld_residual, int64_t rows, int64_t cols,
               double prob, uint64_t seed, uint64_t offset, const void *state, void *out, int64_t ld_out, int dtype,
               int out_dtype, void *stream);

/*
 * ns_cost -- Newton-Schulz cost of an M x N matrix, max(M,N) * min(M,N)^2
 * (second page, "Changes" item 1: the dominant term of the orthogonalization).
 * Returns -1 if M or N is negative.
 */
int64_t ns_cost(int64_t M, int64_t N);

/*
 * ns_plan_shards -- host-only planner that assigns whole matrices to
 * `nshards` shards (GPUs, streams or ranks) so that Newton-Schulz work is
 * balanced. It follows the second page's "Changes" items 1-3: matrices are
 * taken largest first and each goes to the least-loaded shard; with
 * order = NS_PLAN_COST "size" and "load" are the ns_cost of the matrices,
 * with order = NS_PLAN_NUMEL they are element counts (the numel heuristic that
 * page replaces, kept for comparison).
 *   shapes     host array of 2*count (M, N) of the matrices Newton-Schulz runs
 *              on; a 1-D parameter of n elements is passed as (1, n), whose
 *              cost equals its numel.
 *   numels     NULL (element counts are M*N), or count element counts a shard
 *              stores, when they differ from the shape Newton-Schulz sees
 *              (a tensor-parallel shard is stored locally but orthogonalised
 *              after an all-gather: the second page's GTP case).
 *   numel_eps  per-call numel cap: when >= 0, a shard is a candidate for a
 *              matrix only while the elements placed on it by this call plus
 *              the matrix's stay within ceil((1 + numel_eps) * total / nshards);
 *              if no shard qualifies the matrix goes to the shard with the
 *              fewest elements placed by this call (least-numel fallback).
 *              The page uses 0.3. A negative value disables the cap.
 *   loads      NULL, or nshards int64 loads that persist across calls (one
 *              call per bucket); read as the starting loads and updated.
 *   assign     out: count shard indices.
 * Ties go to the shard with fewer elements placed by this call, then to the
 * lower index. Returns NS_OK or NS_EINVAL. Touches no GPU.
 */
#define NS_PLAN_COST 0
#define NS_PLAN_NUMEL 1
int ns_plan_shards(const int64_t *shapes, const int64_t *numels, int count, int nshards, double numel_eps,
                   int order, int64_t *loads, int *assign);

/*
 * ns_get_status -- synchronise `stream`, then return and clear the device
 * status word of the current device: NS_OK, or NS_ETIMEOUT if a kernel's
 * bounded wait gave up (its outputs are then unspecified), NS_EBOUNDS if a
 * debug build's bounds check caught a store outside its buffer (the store was
 * not made; outputs unspecified), or NS_ECUDA if the synchronisation itself
 * failed or a CTA pair's tensor-memory allocations disagreed.
 */
int ns_get_status(void *stream);

/*
 * Debug builds. Compiled with NS_DEBUG_BOUNDS (e.g. NS_BUILD_TAG=debug
 * NS_EXTRA_NVCC_FLAGS=-DNS_DEBUG_BOUNDS with the package's build script),
 * every store of the library's kernels is checked against the buffer it
 * belongs to; a store outside it is not made and the device status word
 * records NS_EBOUNDS. Release builds compile the checks away.
 * ns_selftest_bounds_check exercises the mechanism without touching memory:
 * one thread asks whether a store one past the end of a 4-byte buffer is in
 * bounds. Synchronises `stream`. Returns NS_OK in a debug build (the status
 * word then reads NS_EBOUNDS), NS_EINVAL in a release build.
 */
int ns_selftest_bounds_check(void *stream);

/* ns_strerror -- static description of a status code. */
const char *ns_strerror(int code);

/*
 * ns_release_workspace -- synchronise the device and free the internal
 * workspace cache of the current device, which ends the use of every graph
 * that holds captured calls. Returns NS_OK or NS_ECUDA.
 */
int ns_release_workspace(void);

/* ns_num_kernel_launches -- kernels this library launched on this process
 * since load (for launch accounting in benchmarks). */
int64_t ns_num_kernel_launches(void);

/*
 * ns_set_workspace_limit -- cap, in bytes, on any one workspace the library's
 * internal cache allocates (per device, stream and use); 0 removes the cap
 * (the default). A call whose batch needs a larger workspace than the cap and
 * than the cache already holds returns NS_ENOMEM before anything is allocated
 * or launched, exactly as when the device allocation itself fails. Calls with
 * a caller workspace (_ex) and ns_orthogonalize_batched_noalloc are not
 * affected. Process-wide; returns NS_OK.
 */
int ns_set_workspace_limit(size_t bytes);

/* ns_set_nvtx -- NVTX ranges for profilers' timelines: with enable != 0 every
 * call is bracketed by a range "ns call" and every kernel launch by a range
 * naming its class ("ns gram", "ns apply", ...). Off by default, unless the
 * environment variable NS_NVTX=1 was set when the library first looked.
 * Process-wide; returns NS_OK. */
int ns_set_nvtx(int enable);

/* ns_num_workspace_allocations -- device allocations (workspace cache growth)
 * this library has requested in this process since load; calls that reuse the
 * cached workspace, calls given a caller workspace and
 * ns_orthogonalize_batched_noalloc leave it unchanged. */
int64_t ns_num_workspace_allocations(void);

/*
 * Per-kernel timing for measurement tools. While enabled, every kernel
 * launch of later calls is bracketed by a pair of CUDA events recorded on the
 * caller's stream (a few microseconds of overhead per launch).
 * ns_set_kernel_timing(1) enables and clears the record, (0) disables it.
 * ns_get_kernel_times synchronises on the recorded events and writes, for the
 * kernel classes 0 norm pass (the one read of the caller's matrices: bf16 tile
 * sums of squares and extents, plus a copy where the first step cannot read
 * them in place; fp32 the sums and extents), 1 norm finish (bf16: the
 * per-matrix scale from the tile sums), 2 gram, 3 square, 4 apply,
 * 5 resident, 6 gemm (the tensor-core kernel running every step and phase of
 * a call in one launch), 7 prep (fp32: the normalising copy, or its bf16
 * slices on the tensor cores), 8 momentum
 * (ns_muon_update_batched's element-wise step), 9 embedding lookup, 10 sort of
 * the ids, 11 embedding gradient, 12 log probabilities and policy loss, 13
 * 8-bit checkpoints and the gated activation, 14 weight gradient (with its
 * preparation), 15 router, 16 matrices held in blocks, 17 their product, 18
 * block norms, 19 dropout, the total milliseconds into
 * ms[k] and the launch count into launches[k] for k < n (n <= 20). Returns
 * NS_OK or NS_EINVAL / NS_ECUDA.
 */
int ns_set_kernel_timing(int enable);
int ns_get_kernel_times(double *ms, int64_t *launches, int n);

/*
 * ns_set_gemm_schedule -- how later calls launch the bf16 tensor-core GEMMs
 * (process-wide):
 *   NS_SCHED_PHASE   one persistent launch per step and phase (default);
 *   NS_SCHED_SINGLE  one persistent, cooperative launch per call running every
 *                    step and phase; an item waits, on a per-matrix completion
 *                    counter, until the earlier phases of its matrix are done,
 *                    so phases of different matrices overlap. On GB300 it
 *                    measured 0-3% slower than NS_SCHED_PHASE on the
 *                    8 x 8192x6144, 76 x 2048x6144 and mixed 120-matrix
 *                    batches, so it is not the default.
 * Results are the same in both. The fp32 tensor-core path (ns_set_f32_gemm)
 * always uses NS_SCHED_PHASE. Returns NS_OK or NS_EINVAL.
 */
#define NS_SCHED_PHASE 0
#define NS_SCHED_SINGLE 1
int ns_set_gemm_schedule(int mode);

/*
 * ns_set_f32_gemm -- how later calls compute the GEMMs of large fp32 matrices
 * (those not on the shared-memory resident path), process-wide:
 *   NS_F32_TENSOR  tcgen05 tensor cores (default): every fp32 tensor (the
 *                  iterate, A and B) is held as three bf16 slices
 *                  x = h + m + l, h = bf16(x), m = bf16(x - h),
 *                  l = bf16(x - h - m) (x to 2^-27 relative), and each
 *                  product is the fp32-accumulated sum of the six slice
 *                  products of weight 2^-18 or more, smallest first:
 *                  (h,l), (l,h), (m,m), (h,m), (m,h), (h,h). The dropped
 *                  products weigh 2^-27 or less. The tensor cores' fp32
 *                  accumulation loses up to about a unit in the last place
 *                  per instruction, so the error grows with the contraction
 *                  length: measured 2.2e-5 relative after 5 steps for
 *                  2048 x 6144 (fp32 CUDA cores: 5.0e-6). A call whose
 *                  largest fp32 matrix has max(M, N) > 16384 therefore runs
 *                  on the CUDA cores, keeping every result within fp32's
 *                  1e-4 bar.
 *   NS_F32_SIMT    CUDA-core fp32 FMA GEMMs.
 * Both follow the same definition (the quintic iteration in fp32 between
 * phases); their rounding differs, so their results differ in the last
 * bits. The workspace size (ns_workspace_bytes) depends on the mode in effect
 * when it is computed. Returns NS_OK or NS_EINVAL.
 */
#define NS_F32_TENSOR 0
#define NS_F32_SIMT 1
int ns_set_f32_gemm(int mode);

/*
 * ns_selftest_wait_timeout -- failure-detection self-test. Launches one CTA
 * that waits, with the library's bounded wait and a limit of `limit_us`
 * microseconds (1 .. 10^7), on an mbarrier nothing will ever arrive on. The
 * wait gives up, records NS_ETIMEOUT in the device status word (read it with
 * ns_get_status) and the kernel exits normally: no fault, no trap, no hang,
 * and the CUDA context stays usable. Synchronises `stream`. Returns NS_OK if
 * the wait gave up as designed, NS_EINVAL for a bad limit, NS_ECUDA otherwise.
 */
int ns_selftest_wait_timeout(int limit_us, void *stream);

/*
 * ns_selftest_dependency_timeout -- failure-detection self-test of the
 * tensor-core kernel's dependency waits (the per-matrix completion counters of
 * the NS_SCHED_SINGLE schedule). Runs a two-step call on two 512 x 768 bf16
 * matrices (allocated, filled and released by the call itself) in one
 * cooperative launch whose completion signals are held back, with every
 * bounded wait limited to `limit_us` microseconds (1 .. 10^7): the items that
 * depend on earlier phases wait on counters that never advance, give up,
 * record NS_ETIMEOUT in the device status word (read it with ns_get_status),
 * drain their in-flight copies and MMAs, free their TMEM and exit. No fault,
 * no trap, no hang; the context stays usable. Synchronises `stream`. Returns
 * NS_OK if the waits gave up as designed, NS_EINVAL for a bad limit, NS_ENOMEM
 * if the buffers could not be allocated, NS_ECUDA otherwise.
 */
int ns_selftest_dependency_timeout(int limit_us, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* NS_H_ */
