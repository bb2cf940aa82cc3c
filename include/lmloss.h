/*
 * lmloss: fused LM-head loss forward + backward over a [T, V] logit matrix,
 * for one NVIDIA GB300 GPU (sm_103a).
 *
 * One call computes, sharing one softmax pass per row:
 *   - cross-entropy in the collapse-free form NLL = softplus(lse_{j!=t} z_j - z_t)
 *       [torchtitan PR 5661 "fix softmax collapse with improved CE perf",
 *        commit message, "Numerics (TP > 1 only)"];
 *   - z-loss alpha * lse^2
 *       [xtuner PR 1963 "[FSDP][Loss] Switch gradient reduction to SUM", z-loss diff];
 *   - optional forward-KL distillation against teacher logits, and
 *   - optional GSPO sequence-level clipped aggregation over packed segments
 *       [Fast-LLM PR 552 "Fuse GSPO into the monolithic compiled loss (#507)",
 *        "Why it needed special handling" and "Approach"],
 * reduced either as a token mean or as a SUM over the caller's global
 * denominator [xtuner PR 1963, description], and writes the gradient
 * d(total)/d(logits) once, optionally over the logits in place.
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE memory owned by the caller, row-major.
 *     The library never frees or retains them past the call.
 *   - Calls are asynchronous on the given stream; no entry point synchronises
 *     the device except lmloss_get_device_error and lmloss_get_timing.
 *   - Argument errors are detected on the host and returned synchronously
 *     before anything is launched.  Data errors found on the device (a target
 *     outside [0, V) that is not -100, a segment id >= num_segments, a GSPO
 *     log-ratio sum out of range, a bounded wait that expired) are recorded in
 *     the handle's device error word; the affected rows' losses and gradients
 *     are NaN.  Read the word with lmloss_get_device_error after syncing.
 *   - One handle per stream: two calls on one handle must not overlap.
 */
#ifndef LMLOSS_H
#define LMLOSS_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    LMLOSS_OK = 0,
    LMLOSS_ERR_INVALID_ARG = 1,   /* null/misaligned pointer, bad size, ld < V, ...        */
    LMLOSS_ERR_UNSUPPORTED = 2,   /* valid but not served: a launch shape that does not fit, */
                                  /* a row too long to stage (see lmloss_forward_backward),  */
                                  /* T >= 2^30, a shard call with a teacher or policy term    */
    LMLOSS_ERR_CUDA = 3,          /* a CUDA runtime call failed                            */
    LMLOSS_ERR_BAD_TARGET = 4,    /* device: target not in [0, V) and not -100             */
    LMLOSS_ERR_BAD_SEGMENT = 5,   /* device: segment id >= num_segments                    */
    LMLOSS_ERR_RANGE = 6,         /* device: GSPO log-ratio sum beyond +-2^31; a 4-bit     */
                                  /* table's weight or scale that is not finite            */
    LMLOSS_ERR_TIMEOUT = 7,       /* device: a bounded wait on a copy expired              */
    LMLOSS_ERR_BAD_PARENT = 8     /* device: a beam's parent outside [0, K)                */
} lmloss_status;

/* FP16 is taken by the vocabulary operators below only. */
typedef enum { LMLOSS_BF16 = 0, LMLOSS_FP32 = 1, LMLOSS_FP16 = 2 } lmloss_dtype;

typedef enum {
    LMLOSS_REDUCE_SUM = 0,        /* every term scaled by 1 / denominator                  */
    LMLOSS_REDUCE_TOKEN_MEAN = 1  /* token terms / #active tokens, GSPO / #non-empty segs   */
} lmloss_reduction;

#define LMLOSS_IGNORE_INDEX (-100)

typedef struct lmloss_ctx* lmloss_handle;

/*
 * Arguments of one call.  Zero-initialise, then fill what is used.
 *
 * Layout: logits, teacher_logits and grad_out are [T, ld] row-major arrays of
 * `dtype` (bf16 or fp32) whose first V columns are used; all three share ld.
 * Elements must be naturally aligned, and teacher_logits / grad_out must sit at
 * the same address modulo 16 bytes as logits (true for any two buffers from
 * one allocator with the same ld).
 *
 * Row r is ACTIVE iff targets[r] != -100 and (loss_mask == NULL or
 * loss_mask[r] != 0).  Inactive rows add nothing and get an all-zero gradient
 * [torchtitan PR 5661, "Numerics": ignored labels are zeroed by the mask].
 */
typedef struct {
    const void* logits;          /* [T, ld] dtype                                          */
    int64_t T;                   /* rows (tokens), >= 0                                    */
    int64_t V;                   /* vocabulary columns, >= 1                               */
    int64_t ld;                  /* row stride in elements, >= V                           */
    int32_t dtype;               /* lmloss_dtype                                           */
    int32_t reduction;           /* lmloss_reduction                                       */
    const int64_t* targets;      /* [T] target column, or -100 to ignore the row           */
    const uint8_t* loss_mask;    /* [T] or NULL                                            */

    float ce_weight;             /* weight of the CE term (0 for pure GSPO)                */
    float z_alpha;               /* z-loss alpha; 0 disables                               */

    const void* teacher_logits;  /* [T, ld] dtype, or NULL to disable distillation         */
    float kl_weight;             /* weight of KL(q || p^tau), q = softmax(teacher / tau),   */
                                 /*     p^tau = softmax(logits / tau)                      */
    float temperature;           /* distillation temperature tau: finite and > 0 with a    */
                                 /*     teacher (ignored without one)                      */

    const int32_t* segment_ids;  /* [T] GSPO segment of each row, -1 = none; NULL disables */
    int32_t num_segments;        /* segments in this call, <= the handle's max_segments    */
    const float* advantages;     /* [num_segments] per-segment advantage A_i               */
    const float* old_logprobs;   /* [T] behaviour-policy log-prob of each target           */
    float clip_eps_low;          /* ratio clipped to [1 - clip_eps_low, 1 + clip_eps_high] */
    float clip_eps_high;

    double denominator;          /* SUM reduction: every term is divided by this (> 0)     */

    void* grad_out;              /* [T, ld] dtype; == logits writes in place; NULL = none  */
    float* loss_out;             /* [5] total, ce, z, kl, policy (GSPO or GRPO), each      */
                                 /*     after its scale                                    */
    float* logp_out;             /* optional [T]: log p_target = -NLL (0 on inactive rows) */
    float* lse_out;              /* optional [T]: logsumexp of the row (0 on inactive)     */
    float* kl_out;               /* optional [T]: per-row KL (0 on inactive / no teacher)  */
    int64_t* count_out;          /* optional [2]: active rows, non-empty GSPO segments     */
    int32_t* seg_count_out;      /* optional [num_segments]: active tokens per segment     */
    float* seg_ratio_out;        /* optional [num_segments]: s_i = exp(mean log-ratio)     */
    uint8_t* seg_flag_out;       /* optional [num_segments]: 1 iff gradient flows via s_i  */
    float* seg_loss_out;         /* optional [num_segments]: L_i before the GSPO scale     */

    const float* token_advantages; /* [T] GRPO per-token advantages, or NULL: token-level  */
                                 /* clipped surrogate -min(rho A, clamp(rho) A) with        */
                                 /* rho = exp(logp - old_logprobs), clip_eps_low/high,     */
                                 /* scaled like the CE term; exclusive with segment_ids    */
    float* entropy_out;          /* optional [T]: entropy of softmax(logits) (0 inactive)  */
} lmloss_args;

/* What the last call launched (for tuning and for benchmark bookkeeping). */
typedef struct {
    int32_t launches;            /* kernels launched by the call                           */
    int32_t path;                /* 0 fused single-read, 1 stats-only, 2 GSPO three-phase  */
    int32_t cluster;             /* CTAs per row in the fused kernel                       */
    int32_t threads;             /* threads per CTA of the main kernel                     */
    int32_t nbuf;                /* staging buffers per CTA in the fused kernel (1 or 2)   */
    int32_t grid;                /* CTAs of the main kernel                                */
    int32_t smem_bytes;          /* dynamic shared memory per CTA of the main kernel       */
    int32_t reserved;
} lmloss_call_info;

/* Create a handle on `device`: allocates the workspace for calls with up to
 * max_T rows and max_segments GSPO segments (40 B per row plus about 40 B per
 * segment) and the device error word.  The caller owns the handle. */
lmloss_status lmloss_create(lmloss_handle* handle, int device, int64_t max_T, int32_t max_segments);

/* Free the handle and its workspace.  Synchronises the handle's device. */
lmloss_status lmloss_destroy(lmloss_handle handle);

/* Host-only validation of `args` (no CUDA call).  Returns what
 * lmloss_forward_backward would return before launching anything, except
 * for the handle's capacity limits. */
lmloss_status lmloss_check_args(const lmloss_args* args);

/*
 * Loss and gradient for one batch, asynchronous on `stream`.  The call makes
 * no host synchronisation and no allocation, so it may be captured into a CUDA
 * graph and replayed (the graph then reads whatever the captured buffers hold).
 *
 * Paths:
 *   - no GSPO, grad_out != NULL: one fused kernel reads every active row once
 *     (staged in shared memory across a thread-block cluster), reduces its
 *     max / non-target sum / teacher statistics through distributed shared
 *     memory, and writes the gradient once;
 *   - no GSPO, grad_out == NULL: forward statistics only;
 *   - GSPO: statistics pass, segment seam, gradient pass (the seam must see
 *     every row of a segment before any gradient, so the logits are read twice)
 *     [Fast-LLM PR 552, "Approach": GSPO's backward follows its eager seam].
 * A teacher combines with every other term, GSPO included (its gradient pass
 * reads the teacher's row statistics back from the workspace).
 * Row length: a row is staged across at most 16 CTAs, each slice in one CTA's
 * shared memory (227 KB on GB300), so V is at most 1,835,008 for bf16 logits
 * (917,504 with a teacher) and half that for fp32; a longer row returns
 * LMLOSS_ERR_UNSUPPORTED before anything is launched.  Vocabularies beyond that
 * go through the vocabulary-shard calls below.
 * loss_out is written on every path.  The gradient is
 *   s * (ce_weight (p - onehot) + 2 z_alpha lse p + kl_weight (p^tau - q) / tau)
 *     + c_r (p - onehot)
 * with s the token scale, c_r the row's GSPO (or GRPO) coefficient, and the
 * distillation term the derivative of kl_weight KL(q || p^tau) (Fast-LLM PR 552,
 * the list of combinable losses, names distillation; read as the forward KL at
 * temperature tau with no tau^2 factor, so tau = 1 gives kl_weight (p - q)); it
 * is rounded to nearest-even into dtype.
 */
lmloss_status lmloss_forward_backward(lmloss_handle handle, const lmloss_args* args, cudaStream_t stream);

/*
 * lmloss_forward_backward for logits that are in host memory: the call copies
 * them into the device buffer args->logits (and the teacher's into
 * args->teacher_logits) itself, in chunks of chunk_rows rows (0: T / 8, at
 * most 64 chunks), on a stream of the handle's own, and launches each chunk's
 * staged-row kernel on `stream` as soon as that chunk has landed, so the
 * kernels run under the copies of the chunks after them and the call takes
 * little more than the copies.
 *
 * host_logits (host_teacher) hold the same [T, ld] rows as the device buffer;
 * host_teacher is non-NULL exactly when args->teacher_logits is.  The copies
 * overlap only from pinned memory (cudaHostAlloc / cudaHostRegister).  Every
 * other pointer in args is device memory as for lmloss_forward_backward; the
 * gradient may be written in place into args->logits.  The copies start after
 * the work already queued on `stream`; the whole call is complete when `stream`
 * reaches its end.  Results are bitwise those of lmloss_forward_backward on the
 * same data (each row's computation does not depend on the chunking, and the
 * token-mean count and the loss reduction run once over all rows).
 *
 * With GSPO (segment_ids) the chunks run the statistics pass; the segment step
 * and the gradient pass, which need every row's log-prob, follow once all rows
 * are in.  The first call creates the copy stream and 65 events (freed by
 * lmloss_destroy), so it belongs before any stream capture; later calls can be
 * captured in a CUDA graph (the copy stream joins the capture through the
 * events, and a replay copies whatever the host buffers hold then).
 * lmloss_set_timing records nothing for this call.
 */
lmloss_status lmloss_forward_backward_host(lmloss_handle handle, const lmloss_args* args, const void* host_logits,
                                           const void* host_teacher, int64_t chunk_rows, cudaStream_t stream);

/* Read and clear the device error word.  Synchronises the handle's device.
 * Returns LMLOSS_OK when no device-side data error occurred since the last read. */
lmloss_status lmloss_get_device_error(lmloss_handle handle);

/* Human-readable name of a status. */
const char* lmloss_status_string(lmloss_status status);

/* Override the fused kernel's launch shape: cluster size (1..16), threads per
 * CTA (128, 256, 512 or 1024) and rows staged per CTA (1 or 2); other values are
 * LMLOSS_ERR_INVALID_ARG, and 0 keeps the automatic choice.  Shapes that do not
 * fit are rejected at the next call with LMLOSS_ERR_UNSUPPORTED. */
lmloss_status lmloss_set_launch_config(lmloss_handle handle, int cluster, int threads, int nbuf);

/* When enabled (which also resets the record), each call records a pair of
 * CUDA events on its stream around its main kernel(s), up to 4096 calls.
 * lmloss_get_timing waits for the last pair and returns the summed elapsed
 * time of every recorded call and how many calls were recorded. */
lmloss_status lmloss_set_timing(lmloss_handle handle, int enable);
lmloss_status lmloss_get_timing(lmloss_handle handle, float* total_ms, int32_t* calls);

/* Failure-detection self-test (diagnostic; synchronises the device): runs the
 * bounded wait that guards every copy in the kernels on a barrier that nothing
 * arrives at, giving up after limit_cycles SM clock cycles.  Returns
 * LMLOSS_ERR_TIMEOUT when the wait gave up as it should (LMLOSS_OK if it
 * somehow completed), with the device still usable. */
lmloss_status lmloss_selftest_bounded_wait(lmloss_handle handle, long long limit_cycles);

/* Launch shape and kernel count of the last call on this handle. */
lmloss_status lmloss_get_call_info(lmloss_handle handle, lmloss_call_info* info);

/*
 * Allocation-free variant of lmloss_forward_backward.  The pages have no
 * counterpart: it is for callers that may not allocate device memory once they
 * are running, such as an inference-engine plugin whose enqueue step must not
 * allocate, or a service that plans all of its device memory at start-up,
 * because cudaMalloc can synchronise the device and can fail under memory
 * pressure.
 *
 * Same arguments, results and asynchrony as lmloss_forward_backward, on the
 * current device, without a handle.  It allocates nothing: its workspace is a
 * fixed array of about 2.8 MB inside this library, which every GPU that loads
 * the library holds until the process exits.  Limits: T <= LMLOSS_NOALLOC_MAX_T
 * rows and, with GSPO, num_segments <= LMLOSS_NOALLOC_MAX_SEGMENTS; a larger
 * call returns LMLOSS_ERR_INVALID_ARG before anything is launched.
 *
 * The first call on a device looks up the array's device address and the
 * device's SM limits, and clears the array (no allocation; it synchronises
 * that device once); make that first call before any stream capture.  The
 * address is kept for the life of the process: after cudaDeviceReset on a
 * device the module is reloaded elsewhere, so do not call this entry point on
 * that device again.  Every call on a device shares the one array, which keeps the last
 * call's contents, so calls that overlap on the GPU (other streams, other host
 * threads) race and must be serialised by the caller.  Device-side data errors
 * show up only as NaN losses and gradients: there is no handle to read them from.
 */
#define LMLOSS_NOALLOC_MAX_T 65536
#define LMLOSS_NOALLOC_MAX_SEGMENTS 4096
lmloss_status lmloss_forward_backward_noalloc(const lmloss_args* args, cudaStream_t stream);

/* ---- Vocabulary-split rows (the vocabulary of each row spread over K shards)
 *
 * torchtitan PR 5661, "Numerics (TP > 1 only)": with the vocabulary split over
 * devices, each shard drops the target from its own sum of exponentials and
 * only per-row statistics are combined.  Here the K shards are K separate
 * [T, V_k] logit matrices on one GPU, holding the columns [v0_k, v0_k + V_k)
 * of a V_total-wide vocabulary.  Three steps, in order, on one handle, with no
 * other call on that handle in between (the merge leaves the rows' statistics
 * in its workspace for the gradient step); cross-entropy and z-loss only (a
 * teacher, GSPO, GRPO, the entropy or per-row KL: LMLOSS_ERR_UNSUPPORTED).
 *
 * lmloss_shard_stats: for each active row, the shard's maximum over its
 *   non-target columns, the sum of e^(z - max) over them, the target logit if
 *   the shard holds the target column and 1.0 / 0.0 for "holds it", into
 *   part_out[4 T] (device, fp32, caller-owned).  `args` describes the shard:
 *   logits [T, ld] with V = V_k columns, targets in global column numbers
 *   [0, V_total).  grad_out and loss_out are ignored.
 * lmloss_shard_merge: merges the K shards' partials (parts: host array of K
 *   <= 16 device pointers) in shard order into each row's NLL and lse; writes
 *   loss_out (CE and z-loss with the call's reduction; the KL and policy slots
 *   are 0), logp_out / lse_out / count_out if given.  `args`: T, V = V_total,
 *   targets, loss_mask, ce_weight, z_alpha, reduction, denominator; logits are
 *   not read.  A row whose target no shard holds sets LMLOSS_ERR_BAD_TARGET.
 * lmloss_shard_grad: writes the shard's gradient (grad_out, [T, ld], may alias
 *   the shard's logits) from the merged statistics: the same bits as a
 *   whole-row call would give each column, up to the order of the merge. */
lmloss_status lmloss_shard_stats(lmloss_handle handle, const lmloss_args* args, int64_t v0, int64_t V_total,
                                 float* part_out, cudaStream_t stream);
lmloss_status lmloss_shard_merge(lmloss_handle handle, const lmloss_args* args, const float* const* parts,
                                 int32_t K, cudaStream_t stream);
lmloss_status lmloss_shard_grad(lmloss_handle handle, const lmloss_args* args, int64_t v0, int64_t V_total,
                                cudaStream_t stream);

/* ---- Vocabulary operators: the two ends of the vocabulary around the loss
 *
 * Embedding lookup and its gradient (the table the tokens come in through, often
 * the same matrix as the LM head), and beam search's step over [rows, V] logits
 * with the reordering of the beams' states (what the LM head answers with).
 *
 * They share a handle of their own: a workspace of the caller's size and a
 * device error word.  The conventions at the top of this header hold: caller-owned
 * device memory, asynchronous on the given stream, no allocation and no host
 * synchronisation per call (so a call can be captured in a CUDA graph), argument
 * errors returned before anything is launched, data errors in the error word, one
 * handle per stream.  Results do not depend on the timing of the GPU's blocks:
 * the same inputs give the same bits.
 */
typedef struct lmloss_vocab_ctx* lmloss_vocab_handle;

/* A handle on `device` with `workspace_bytes` of workspace: the most that any of
 * its calls needs by lmloss_embedding_workspace / lmloss_beam_workspace /
 * lmloss_logprobs_workspace / lmloss_table4_logits_workspace (0 serves the lookups, the
 * reordering, gradients of up to 1024 positions and of log-probabilities, and the making of
 * 4-bit tables, which need none). */
lmloss_status lmloss_vocab_create(lmloss_vocab_handle* handle, int device, size_t workspace_bytes);

/* At least `workspace_bytes` of workspace for the calls that follow.  Allocates where the handle has
 * less; what it had lives as long as the handle, so that graphs captured with it can be replayed.
 * Allowed while a stream is captured, and not part of the graph. */
lmloss_status lmloss_vocab_reserve(lmloss_vocab_handle handle, size_t workspace_bytes);

/* Free the handle and its workspace.  Synchronises the handle's device. */
lmloss_status lmloss_vocab_destroy(lmloss_vocab_handle handle);

/* Read and clear the handle's device error word.  Synchronises the device. */
lmloss_status lmloss_vocab_get_device_error(lmloss_vocab_handle handle);

typedef enum { LMLOSS_INT64 = 0, LMLOSS_INT32 = 1 } lmloss_id_dtype;

/*
 * Arguments of an embedding call.  `table` is [V, ld_table], `rows` is
 * [T, ld_rows], the first D columns of each used; elements naturally aligned.
 * An id of LMLOSS_IGNORE_INDEX marks a position without a token.
 */
typedef struct {
    const void* ids;             /* [T] token of each position                             */
    int64_t T;                   /* positions, >= 0 and < 2^30                             */
    int64_t V;                   /* rows of the table, >= 1 and < 2^31 - 1                 */
    int64_t D;                   /* columns, >= 1 and <= 2^30                              */
    void* table;                 /* forward: the weights (read);                           */
                                 /* backward: the weights' gradient (written)              */
    int64_t ld_table;            /* row stride in elements, >= D                           */
    void* rows;                  /* forward: the embeddings (written);                     */
                                 /* backward: the embeddings' gradient (read)              */
    int64_t ld_rows;             /* row stride in elements, >= D                           */
    int32_t ids_dtype;           /* lmloss_id_dtype                                        */
    int32_t table_dtype;         /* lmloss_dtype, each of the three with each              */
    int32_t rows_dtype;          /* lmloss_dtype                                           */
    float scale;                 /* finite                                                 */
    int32_t accumulate;          /* backward: 0 writes the whole gradient (zeros where no  */
                                 /* position holds the token), 1 adds to what is there     */
                                 /* and leaves the other rows alone                        */
} lmloss_embedding_args;

/* Host-only validation of `args` (no CUDA call). */
lmloss_status lmloss_embedding_check_args(const lmloss_embedding_args* args);

/* The workspace that lmloss_embedding_backward needs for `args` (pointers are
 * not looked at) and for any call of no more positions and columns, whatever its
 * types: it grows with T and D and depends on nothing else. */
lmloss_status lmloss_embedding_workspace(const lmloss_embedding_args* args, size_t* bytes);

/*
 * rows[t] = scale * table[ids[t]], rounded once to the rows' type; zeros where
 * ids[t] is LMLOSS_IGNORE_INDEX.  Any other id outside [0, V) sets
 * LMLOSS_ERR_BAD_TARGET and gives a row of NaN.
 */
lmloss_status lmloss_embedding_forward(lmloss_vocab_handle handle, const lmloss_embedding_args* args,
                                       cudaStream_t stream);

/*
 * table[v] (+)= scale * sum of rows[t] over the positions t with ids[t] = v.
 * The positions are sorted by token; each token's rows are added in fp32, in an
 * order that the ids alone fix, and the result is rounded once to a 16-bit table.
 * Added to an fp32 table, the product with the scale is rounded and then its sum with
 * the old value (most additions are the memory's own, which takes subnormals as 0:
 * the old value, the product and the sum alike; the others are fused and keep them).  An id outside
 * [0, V) that is not LMLOSS_IGNORE_INDEX sets LMLOSS_ERR_BAD_TARGET and adds
 * nothing.
 */
lmloss_status lmloss_embedding_backward(lmloss_vocab_handle handle, const lmloss_embedding_args* args,
                                        cudaStream_t stream);

#define LMLOSS_MAX_BEAMS 64      /* beams of a sequence, and candidates of a beam step     */

/*
 * Arguments of a beam step over B sequences of K beams: logits is
 * [B * K, ld], row b * K + k for beam k of sequence b.
 */
typedef struct {
    const void* logits;          /* [B * K, ld] dtype, first V columns used                */
    int64_t B;                   /* sequences, >= 0                                        */
    int64_t V;                   /* vocabulary columns, >= 1 and <= 2^31 - 2^16            */
    int64_t ld;                  /* row stride in elements, >= V                           */
    int32_t K;                   /* beams of a sequence, 1 .. LMLOSS_MAX_BEAMS             */
    int32_t M;                   /* candidates wanted, 1 .. LMLOSS_MAX_BEAMS               */
    int32_t dtype;               /* lmloss_dtype, any of the three                         */
    double length_penalty;       /* alpha >= 0 (0 without lengths): candidates are ranked  */
                                 /* by score / length^alpha                                */
    int64_t eos_token;           /* the end token, -1 = none (not with `finished`)         */
    const float* scores;         /* [B, K] summed log-probability of each beam             */
    const uint8_t* finished;     /* [B, K] or NULL: 1 = the beam has ended                 */
    const int32_t* lengths;      /* [B, K] or NULL: tokens of each beam so far             */
    const int32_t* token_mask;   /* NULL, or rows of ceil(V / 32) words: bit v % 32 of     */
                                 /* word v / 32 is set where token v may follow            */
    int64_t mask_stride;         /* words between rows of the mask; 0 = one row for all    */
    float* scores_out;           /* [B, M]                                                 */
    int32_t* parents_out;        /* [B, M] beam of the sequence that the candidate goes on */
    int64_t* tokens_out;         /* [B, M]                                                 */
    float* lse_out;              /* optional [B, K]: logsumexp of each row (0 if finished) */
    uint8_t* finished_out;       /* optional [B, M]                                        */
    int32_t* lengths_out;        /* optional [B, M], only with lengths                     */
} lmloss_beam_args;

/* Host-only validation of `args` (no CUDA call). */
lmloss_status lmloss_beam_check_args(const lmloss_beam_args* args);

/* The workspace that lmloss_beam_step needs for `args` (pointers are not looked at). */
lmloss_status lmloss_beam_workspace(const lmloss_beam_args* args, size_t* bytes);

/*
 * For each sequence, the M best candidates (k, v) by score
 *   scores[k] + logits[k][v] - lse_k,   lse_k = logsumexp of the whole row,
 * (divided by length^alpha for the ranking, or by the largest double where that
 * passes it), best first, equal ones by k, then by v.  The candidates of a row are in
 * the exact order of their logits.  Rows are ranked against one another by a score and a
 * division in fp64, from a sum of exponentials in fp32 (an lse_k about as close as
 * lse_out's own rounding brings it) and a power within 3e-9 (1 + alpha) of itself.
 * scores_out holds the score before the division, rounded to fp32.
 *   - A finished beam's row is not read: its one candidate is (k, eos_token) with
 *     its score as it is, and its length does not grow.
 *   - A token whose mask bit is 0 is no candidate; the row's logsumexp still
 *     covers it.
 *   - A candidate whose score is not finite is none (a masked token, a -inf logit,
 *     a beam at -inf; NaN or +inf in a row take the whole row out).
 *   - Where fewer than M are left, the rest gets score -inf, token
 *     LMLOSS_IGNORE_INDEX, parent m % K, finished 0 and that parent's length.
 * finished_out: the parent had ended, or the token is eos_token.
 */
lmloss_status lmloss_beam_step(lmloss_vocab_handle handle, const lmloss_beam_args* args, cudaStream_t stream);

/*
 * One state of the beams, as bytes: for each outer index (o0, o1, o2) and each row
 * r = b * K + k a run of `inner` bytes at
 *   base + r * row_stride + o0 * outer_stride[0] + o1 * outer_stride[1] + o2 * outer_stride[2].
 * dst == src reorders in place (then with the same strides and K_out == K);
 * otherwise the two must not overlap (halves of a double buffer may lie
 * interleaved, at any dimension; sides entangled in other ways are refused).
 * Strides are in bytes and not negative; no two runs of dst may overlap.
 */
typedef struct {
    const void* src;
    void* dst;
    int64_t inner;               /* bytes of a run, >= 0                                   */
    int64_t src_row_stride;
    int64_t dst_row_stride;
    int64_t outer[3];            /* outer counts, >= 0; 1 where unused                     */
    int64_t src_outer_stride[3];
    int64_t dst_outer_stride[3];
} lmloss_beam_state;

/* Host-only validation of a reordering (no CUDA call). */
lmloss_status lmloss_beam_check_states(const lmloss_beam_state* states, int32_t num_states, int64_t B, int32_t K,
                                       int32_t K_out);

/*
 * Every state's row b * K_out + m becomes its row b * K + parents[b, m]
 * (parents: [B, K_out] int32, device).  `states` is a host array, read during the
 * call.  The states move side by side, in no order: no state's dst may overlap
 * another's src or dst (two that begin at the same byte are refused, so a swap
 * of two buffers, or one state given twice in place).  A parent outside [0, K) sets LMLOSS_ERR_BAD_PARENT and leaves that row of
 * dst as it is.
 */
lmloss_status lmloss_beam_reorder(lmloss_vocab_handle handle, const lmloss_beam_state* states, int32_t num_states,
                                  const int32_t* parents, int64_t B, int32_t K, int32_t K_out, cudaStream_t stream);

/* ---- Log-probabilities of given tokens
 *
 * Over rows of [T, V] logits, at a temperature tau and over the columns that a mask allows
 * (y = logits / tau; columns that are not allowed count as -inf):
 *   lse = ln sum_v e^y_v,   logp_j = y_{t_j} - lse,   H = -sum_v p_v ln p_v,  p = e^(y - lse)
 * and the M largest log-probabilities with their tokens.  The handle, the conventions and the
 * error word are those of the vocabulary operators.
 */
#define LMLOSS_MAX_ALTERNATIVES 64
#define LMLOSS_MAX_GIVEN 1024    /* given tokens a row of a gradient                       */

typedef struct {
    const void* logits;          /* [T, ld] dtype, first V columns used                    */
    int64_t T;                   /* rows, >= 0 and < 2^30                                  */
    int64_t V;                   /* vocabulary columns, >= 1 and <= 2^31 - 2^16            */
    int64_t ld;                  /* row stride in elements, >= V                           */
    int32_t dtype;               /* lmloss_dtype, any of the three                         */
    int32_t ids_dtype;           /* lmloss_id_dtype of tokens                              */
    const void* tokens;          /* [T, n] given tokens, LMLOSS_IGNORE_INDEX = none;       */
                                 /* NULL with n = 0                                        */
    int64_t n;                   /* given tokens a row, 0 .. 2^20                          */
    float temperature;           /* 2^-20 .. 2^20                                          */
    int32_t M;                   /* alternatives, 0 .. LMLOSS_MAX_ALTERNATIVES             */
    const int32_t* token_mask;   /* NULL, or rows of ceil(V / 32) words: bit v % 32 of     */
                                 /* word v / 32 is set where token v is allowed            */
    int64_t mask_stride;         /* words between rows of the mask; 0 = one row for all    */
    float* logp_out;             /* [T, n]                                                 */
    float* lse_out;              /* optional [T]                                           */
    float* entropy_out;          /* optional [T]                                           */
    float* top_logp_out;         /* [T, M]                                                 */
    int64_t* top_tokens_out;     /* [T, M]                                                 */
    float* row_max_out;          /* optional [T]: the row's largest allowed logit          */
    float* log_sum_out;          /* optional [T]: lse - row_max / tau                      */
} lmloss_logprobs_args;

/* Host-only validation of `args` (no CUDA call). */
lmloss_status lmloss_logprobs_check_args(const lmloss_logprobs_args* args);

/* The workspace that lmloss_logprobs_forward needs for `args` (pointers are not
 * looked at); it grows with M and T and has a bound of about 2.2 MB. */
lmloss_status lmloss_logprobs_workspace(const lmloss_logprobs_args* args, size_t* bytes);

/*
 * One read of the logits.  Sums of exponentials in fp32 (an lse and an entropy
 * within a few fp32 steps of the exact ones), log-probabilities from their difference in fp64,
 * rounded to fp32.
 *   - LMLOSS_IGNORE_INDEX gives a log-probability of 0; another token outside [0, V)
 *     NaN and LMLOSS_ERR_BAD_TARGET; one that is not allowed, or whose logit is -inf, -inf.
 *   - Alternatives come in the exact order of their logits, equal ones by token.  Where
 *     fewer than M have a finite logit and are allowed, the rest gets -inf and
 *     LMLOSS_IGNORE_INDEX.
 *   - A row in which nothing is allowed (or every allowed logit is -inf): lse, row_max and
 *     log_sum -inf, entropy 0, log-probabilities -inf.
 *   - NaN or +inf in an allowed column: lse, log_sum, entropy and log-probabilities are NaN, and
 *     the row has no alternatives.  What stands in columns that are not allowed has no effect.
 */
lmloss_status lmloss_logprobs_forward(lmloss_vocab_handle handle, const lmloss_logprobs_args* args,
                                      cudaStream_t stream);

typedef struct {
    const void* logits;          /* as for the forward call, up to the mask                */
    int64_t T;
    int64_t V;
    int64_t ld;
    int32_t dtype;
    int32_t ids_dtype;
    const void* tokens;          /* [T, n] or NULL with n = 0                              */
    int64_t n;                   /* 0 .. LMLOSS_MAX_GIVEN                                  */
    float temperature;
    const int32_t* token_mask;
    int64_t mask_stride;
    const float* lse;            /* [T] of the forward call; not looked at beside log_sum  */
    const float* grad_logp;      /* [T, n] or NULL with n = 0                              */
    const float* entropy;        /* [T] of the forward call, with grad_entropy             */
    const float* grad_entropy;   /* optional [T]                                           */
    void* grad_out;              /* [T, ld_grad] dtype, written whole; == logits with the  */
                                 /* same ld writes in place, otherwise no overlap          */
    int64_t ld_grad;             /* row stride in elements, >= V                           */
    const float* row_max;        /* optional [T] of the forward call, both or neither      */
    const float* log_sum;        /* optional [T]                                           */
} lmloss_logprobs_grad_args;

/* Host-only validation of `args` (no CUDA call). */
lmloss_status lmloss_logprobs_check_grad_args(const lmloss_logprobs_grad_args* args);

/*
 * grad_out[r][v] = ( sum_{j: t_j = v} g_j - p_v (sum_j g_j + gH (ln p_v + H)) ) / tau
 * in fp32, rounded once; 0 in columns that are not allowed, and in a whole row whose log_sum
 * (without it: lse) is -inf.  With row_max and log_sum, ln p_v = (z_v - row_max) / tau - log_sum,
 * as good at every temperature.  With lse alone, ln p_v = y_v - lse: p is off by a factor of
 * e to what fp32 leaves of lse (2^-24 of it: 1e-6 for an lse of 15, 1e-3 for 15000), and a row
 * whose lse passes fp32's range gets 0.  A token given twice counts twice; one that is not
 * allowed still takes its -g p from the others, as its logp = -inf - lse does.  Tokens outside
 * [0, V) that are not LMLOSS_IGNORE_INDEX set LMLOSS_ERR_BAD_TARGET and add nothing.  No
 * workspace.
 */
lmloss_status lmloss_logprobs_backward(lmloss_vocab_handle handle, const lmloss_logprobs_grad_args* args,
                                       cudaStream_t stream);

/* ---- A vocabulary table in 4 bits
 *
 * A [V, D] table with one scale, and on request one zero point, for each row and group of
 * `group` columns:  w[v][c] = scales[g][v] * (q[v][c] - zeros[g][v]),  g = c / group, q in 0 .. 15,
 * and 8 in the zeros' place where there are none.  It is made from float weights, looked up
 * (an embedding) and multiplied with hidden rows (an LM head); a tied model uses one for both.
 */
typedef struct {
    uint8_t* values;             /* [V, ld_values]: column c in the low (c even) or high   */
                                 /* half of byte c / 2; 16-byte aligned                    */
    int64_t ld_values;           /* row stride in bytes, >= (D + 1) / 2, a multiple of 16  */
    void* scales;                /* [ceil(D / group), ld_scales] scale_dtype, 16-byte      */
                                 /* aligned                                                */
    int64_t ld_scales;           /* elements, >= V; as bytes a multiple of 16              */
    uint8_t* zeros;              /* [ceil(D / group), ld_zeros] or NULL; 16-byte aligned   */
    int64_t ld_zeros;            /* >= V, a multiple of 16 (not looked at without zeros)   */
    int64_t V;                   /* rows, 1 .. 2^31 - 2^16                                 */
    int64_t D;                   /* columns, 1 .. 2^20                                     */
    int32_t group;               /* 32, 64 or 128                                          */
    int32_t scale_dtype;         /* lmloss_dtype                                           */
} lmloss_table4;

/* Host-only validation of a table (no CUDA call). */
lmloss_status lmloss_table4_check(const lmloss_table4* table);

typedef struct {
    lmloss_table4 table;         /* written                                                */
    const void* weight;          /* [V, ld_weight] weight_dtype                            */
    int64_t ld_weight;           /* row stride in elements, >= D                           */
    int32_t weight_dtype;        /* lmloss_dtype                                           */
} lmloss_table4_quantize_args;

/*
 * The table nearest to float weights, group by group (R rounds to the scales' type, quotients
 * w / s are rounded to the nearest whole number, halves to the even one):
 *   without zeros  s = R(max |w| / 7),          q = clamp(w / s, -8, 7) + 8
 *   with zeros     s = R((hi - lo) / 15),       z = clamp(-lo / s, 0, 15),  q = clamp(w / s + z, 0, 15)
 *                  lo = min(0, w), hi = max(0, w)
 * the quotient before R in fp32.  A group of s = 0 holds zeros.  A group with a weight that is
 * not finite, or whose scale leaves its type's range, gets a scale of NaN, and
 * LMLOSS_ERR_RANGE is set.  In the last byte of a row of odd D the high half is 0; bytes past it
 * are left alone.
 */
lmloss_status lmloss_table4_quantize(lmloss_vocab_handle handle, const lmloss_table4_quantize_args* args,
                                     cudaStream_t stream);

typedef struct {
    lmloss_table4 table;         /* read                                                   */
    const void* ids;             /* [T]                                                    */
    int64_t T;                   /* >= 0 and < 2^30                                        */
    void* rows;                  /* [T, ld_rows] rows_dtype, written                       */
    int64_t ld_rows;             /* >= D                                                   */
    int32_t ids_dtype;           /* lmloss_id_dtype                                        */
    int32_t rows_dtype;          /* lmloss_dtype                                           */
    float scale;                 /* finite                                                 */
} lmloss_table4_lookup_args;

/* rows[t] = scale * w[ids[t]], computed in fp32 and rounded once more; ids as for
 * lmloss_embedding_forward. */
lmloss_status lmloss_table4_lookup(lmloss_vocab_handle handle, const lmloss_table4_lookup_args* args,
                                   cudaStream_t stream);

typedef struct {
    lmloss_table4 table;         /* read                                                   */
    const void* hidden;          /* [T, ld_hidden] hidden_dtype, first D columns used      */
    int64_t T;                   /* rows, >= 0 and < 2^24                                  */
    int64_t ld_hidden;           /* >= D                                                   */
    void* logits;                /* [T, ld_logits] logits_dtype, written                   */
    int64_t ld_logits;           /* >= V                                                   */
    int32_t hidden_dtype;        /* lmloss_dtype                                           */
    int32_t logits_dtype;        /* lmloss_dtype                                           */
    float scale;                 /* finite                                                 */
} lmloss_table4_logits_args;

/* Host-only validation (no CUDA call). */
lmloss_status lmloss_table4_check_quantize_args(const lmloss_table4_quantize_args* args);
lmloss_status lmloss_table4_check_lookup_args(const lmloss_table4_lookup_args* args);
lmloss_status lmloss_table4_check_logits_args(const lmloss_table4_logits_args* args);

/* The workspace that lmloss_table4_logits needs for `args` (pointers are not looked at)
 * and for any call of no more rows and columns, whatever its types.  (Calls of up to 8 rows, 4
 * where hidden values or logits are fp32, need none up to 6144 columns, and some beyond.) */
lmloss_status lmloss_table4_logits_workspace(const lmloss_table4_logits_args* args, size_t* bytes);

/*
 * logits[t][v] = scale * sum_c hidden[t][c] * w[v][c]: from one row (a decoding step) to a
 * prompt's.  Within a group the products with the whole numbers q - z are summed, and the sum
 * is scaled by the group's scale: no weight is rounded.  Sums in fp32, one rounding at the end.
 * fp32 hidden values count with an error of at most 2^-23 of the largest in their group of
 * columns plus 2^-46 of the largest in their row (two fp16 hold one: beside a column 2^11 times as
 * large a value keeps 11 bits), 16-bit ones of at most 2^-35 of the largest in their row.  A row with an
 * infinity or NaN gives what the formula gives, slowly, and does not disturb the others.  A
 * row's logits depend on that row, its index, the table and T alone.  `logits` overlaps neither
 * `hidden` nor the table.  A wait inside that expires sets LMLOSS_ERR_TIMEOUT; the logits mean nothing then.
 */
lmloss_status lmloss_table4_logits(lmloss_vocab_handle handle, const lmloss_table4_logits_args* args,
                                   cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LMLOSS_H */
