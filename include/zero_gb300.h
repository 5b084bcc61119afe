/*
 * zero_gb300.h -- C ABI of the ZeRO sharded mixed-precision optimizer step
 * (Adam; also SGD with momentum and SGD) on one GB300 (sm_103a).
 *
 * What the library computes
 * -------------------------
 * ZeRO-DP partitions a data-parallel job's model states -- optimizer state
 * (stage 1, P_os), gradients (stage 2, P_os+g) and parameters (stage 3,
 * P_os+g+p) -- across the N_d data-parallel ranks, each rank keeping 1/N_d
 * ("ZeRO：大模型训练的内存优化革命" 3.1.1-3.1.3; ZeRO visual reading, stage
 * list).  In mixed precision each parameter carries a 16-bit copy, a 16-bit
 * gradient and 12 bytes of fp32 optimizer state (master weight, momentum,
 * variance) ("AI论文陪读·ZeRO" section 01; ZeRO visual reading, 16Ψ account).
 * One optimizer step of a stage-2 rank is: reduce-scatter the gradients of
 * each constant-size bucket to their owners, update the owned fp32 shard with
 * Adam, cast it to 16 bits and all-gather the new parameters to every rank
 * (ZeRO visual reading, communication accounting; SC-2020 ZeRO notes, "Deep
 * Dive into ZeRO-R / C_B" for the fixed-size fusion buffers).
 *
 * Here the N_d ranks are simulated: each rank's buffers are separate regions
 * of one GPU's memory, and each collective is the memory traffic of the fused
 * kernels.  Per bucket, one kernel reads the N_d ranks' 16-bit gradients,
 * sums them in rank order in fp32, rounds once to 16 bits, checks for inf/NaN
 * (loss-scale overflow), unscales by 1/(S*N_d), applies the optimizer --
 * Adam (Kingma & Ba, Algorithm 1: bias correction, eps outside the square
 * root, no weight decay), or SGD with momentum, or SGD -- to the owned fp32
 * state and writes the 16-bit cast to every rank (stages 0-2) or to the
 * owner's shard (stage 3).  The partition does not change the
 * step's result: every stage gives the same numbers as one unpartitioned step.
 *
 * Layout
 * ------
 *   Psi  = n_params; N = n_ranks; A = align_elems (default 2048).
 *   P    = ceil(Psi / N) rounded up to a multiple of A; rank r owns flat
 *          indices [r*P, (r+1)*P).  padded = N*P.
 *   Buckets are consecutive windows of bucket_elems elements over [0, Psi),
 *   in parameter order; the last one may be shorter.  Padding elements
 *   [Psi, padded) are never read or written by a step (keep them zero).
 *   16-bit buffers hold IEEE binary16 or bfloat16 bit patterns (dtype).
 *   With dtype ZERO_FP32 (fp32 training) the gradient, parameter and
 *   reduced buffers hold binary32 values instead -- 4 bytes per element,
 *   the same element counts -- and the "16-bit" cast is the identity.
 *   Per rank r (device memory, caller-owned):
 *     grads[r]    16-bit gradient, grad16_elems = padded elements, flat index
 *                 order (loss-scaled).  Stages 0 and 1 overwrite it with the
 *                 reduced gradient (the all-reduce result).
 *     params16[r] 16-bit parameters: the full vector (padded elements) in
 *                 stages 0-2; only rank r's shard (P elements) in stage 3.
 *   fp32 state w, m, v: state_elems floats each (the arrays the optimizer
 *   uses; see zero_optimizer_t).  Stages 1-3: the N shards
 *   concatenated, i.e. flat index order (padded elements).  Stage 0: N full
 *   replicas, replica r at offset r*padded.  Two copies of each may be given:
 *   [cur] holds the current state; [1-cur] is the shadow that a fused step
 *   writes the new state into (the step is speculative until the global
 *   overflow flag is known; a clean step then flips cur).
 *   reduced: 16-bit reduced gradient, padded elements in flat order (each
 *   owner's shard), needed by the two-pass path in stages 2 and 3.
 *   workspace: workspace_bytes of device memory, 16-byte aligned; contents
 *   are scratch owned by the library during a step.
 *
 * Paths
 * -----
 *   fused     (no clipping and shadow state given): one kernel per bucket,
 *             state read from [cur] and written to [1-cur].  On overflow the
 *             step is discarded and each written 16-bit parameter is restored
 *             to the cast of the unchanged master weights.  In stages 2 and 3
 *             a bucket kernel that starts after the step's flag is raised
 *             writes nothing, and only the window the others wrote is
 *             restored (hbm_bytes counts what really moved); so the 16-bit
 *             parameters must hold the cast of the current master weights
 *             when a step starts, as every step leaves them.
 *   two-pass  (clipping, or no shadow): pass 1 per bucket reduces and checks
 *             the gradient, materialises it (grads[] in stages 0/1, reduced
 *             in stages 2/3) and accumulates the exact sum of squares; a
 *             one-thread kernel forms the global norm and clip coefficient
 *             (16-bit types only);
 *             pass 2 per bucket updates the state in place, or does nothing
 *             when the flag is set.
 *
 *   Inside zero_step / zero_step_stageK (and the update pass of
 *   zero_step_end) consecutive bucket kernels use programmatic dependent
 *   launch: a bucket kernel may start while its predecessor drains; kernels
 *   still complete in stream order.  Kernels launched by zero_step_bucket
 *   follow plain stream order.
 *
 * Conventions
 * -----------
 *   The caller owns all memory; the library allocates nothing and never
 *   throws.  Between calls it keeps only: per process, the resident-block
 *   count of each kernel on each device (behind a lock) and which devices a
 *   kernel's shared-memory limit was raised on; per thread, the
 *   error text, the profiling events, and whether each pointer it was given
 *   for a replicated output is device memory of the current device (asked
 *   of the driver on every call outside stream capture, so a freed address
 *   that later holds host or managed memory is seen as such; while a stream
 *   is captured no query is made and the answer last seen on the thread
 *   stands, an unknown pointer counting as not device memory).  A fetcher's state lives in caller memory.  Several threads
 *   may call at once on different jobs and streams.  Every
 *   function returns a zero_status_t; on failure zero_last_error() gives a
 *   message (thread-local).  Kernels run asynchronously on the caller's stream
 *   (a cudaStream_t passed as void*; NULL = legacy default stream).  The
 *   end of a step synchronises that stream once to read the overflow flag
 *   (zero_step_async, below, keeps the step state on the device instead).
 *   Device pointers must be 16-byte aligned (ZERO_EALIGN otherwise).  Any
 *   pointer the GPU can load from and store to is accepted: on GB300 the
 *   gradients or the fp32 optimizer state may live in pinned host memory,
 *   which the kernels then reach over NVLink-C2C.
 *   Pointer arrays (grads, params16, dst) are host arrays of device
 *   pointers, read during the call only.
 */
#ifndef ZERO_GB300_H
#define ZERO_GB300_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define ZERO_GB300_VERSION 1
#define ZERO_MAX_RANKS 64
#define ZERO_DEFAULT_ALIGN 2048

typedef enum {
    ZERO_OK = 0,
    ZERO_EINVAL = 1,         /* bad argument, inconsistent plan or call order */
    ZERO_EALIGN = 2,         /* a device pointer is not 16-byte aligned */
    ZERO_ENOMEM = 3,         /* a caller-provided buffer is missing or too small */
    ZERO_ECUDA = 4,          /* a CUDA runtime call failed (message has the CUDA error) */
    ZERO_ETIMEOUT = 5,       /* a kernel's bounded wait on its own copies ran out (seconds); the step was not applied */
    ZERO_EUNSUPPORTED = 6    /* n_ranks outside 1..64, or another unsupported size */
} zero_status_t;

/* Model precision of gradients and parameters.  ZERO_FP16 / ZERO_BF16:
 * mixed precision (b = 2 bytes, fp32 master state).  ZERO_FP32: fp32
 * training as in the pages' fp32 SGD and SGD-with-momentum examples (b = 4;
 * ZeRO visual reading, worked examples C): the reduced gradient is the fp32
 * rank-order sum itself and the parameters equal the fp32 master weights
 * bit for bit.  The library still keeps the master shard w apart from the
 * parameter copies (a step can then be discarded), so its state holds 4
 * bytes per parameter more than the pages' K; gradient clipping is not
 * available with ZERO_FP32 (ZERO_EUNSUPPORTED).  The no-allocation stage-2
 * entry point takes 16-bit types only. */
typedef enum { ZERO_FP16 = 0, ZERO_BF16 = 1, ZERO_FP32 = 2 } zero_dtype_t;

/* Optimizer on the fp32 master weights ("ZeRO visual reading", accounting
 * with b and K: mixed-precision Adam K = 12, SGD with momentum K = 8, SGD
 * K = 4, each counting the 4-byte fp32 master copy).  State arrays used:
 * Adam w, m, v; SGD with momentum w, m; SGD w (the others may be NULL). */
typedef enum { ZERO_ADAM = 0, ZERO_SGD_MOMENTUM = 1, ZERO_SGD = 2 } zero_optimizer_t;

/* Job description.  56 bytes. */
typedef struct zero_config {
    int64_t n_params;            /* Psi >= 0 */
    int64_t bucket_elems;        /* B > 0, multiple of 8 (gradient bucket, C_B) */
    int64_t align_elems;         /* A: shard alignment in elements; 0 -> 2048; multiple of 8 */
    const int64_t* layer_sizes;  /* stage-3 gather units in parameter order (sum = Psi); NULL -> one */
    int32_t n_layers;            /* entries in layer_sizes (0 when NULL) */
    int32_t stage;               /* ZeRO-DP stage 0..3 */
    int32_t n_ranks;             /* N_d, 1..64 */
    int32_t dtype;               /* zero_dtype_t of parameters and gradients */
    int32_t optimizer;           /* zero_optimizer_t (0: Adam) */
    int32_t reserved;            /* 0 */
} zero_config_t;

/* Partition and sizes derived from a config by zero_plan.  128 bytes. */
typedef struct zero_plan {
    int64_t shard_elems;         /* P */
    int64_t padded_elems;        /* N*P */
    int64_t n_buckets;           /* ceil(Psi / B) */
    int64_t n_layers;
    int64_t max_layer_elems;     /* capacity of a stage-3 gather destination */
    int64_t state_elems;         /* floats in each of w, m, v: N*P, or N*N*P in stage 0 */
    int64_t param16_elems;       /* per rank: N*P in stages 0-2, P in stage 3 */
    int64_t grad16_elems;        /* per rank: N*P */
    int64_t reduced_elems;       /* N*P in stages 2-3 (two-pass path), else 0 */
    int64_t workspace_bytes;
    int64_t hbm_bytes_fused;     /* algorithmic HBM bytes of one fused step (each array access once) */
    int64_t hbm_bytes_two_pass;  /* algorithmic HBM bytes of one two-pass step */
    int64_t comm_counted_bytes;  /* bytes crossing simulated rank boundaries per step, all ranks */
    double comm_paper_bytes;     /* per rank per step: 2*Psi*b (stages 0-2), 3*Psi*b (stage 3) */
    double mem_total_bytes;      /* per rank, paper formula (b = 2, or 4 for ZERO_FP32; K = the fp32
                                    state bytes kept), see zero_model_state_bytes */
    double reserved;
} zero_plan_t;

/* Optimizer hyper-parameters.  Adam (Kingma & Ba, Algorithm 1) uses lr,
 * beta1, beta2, eps; SGD with momentum (PyTorch's rule without dampening:
 * m' = momentum*m + g, w' = w - lr*m') uses lr and momentum; SGD
 * (w' = w - lr*g) uses lr.  24 bytes. */
typedef struct zero_adam {
    float lr, beta1, beta2, eps;
    float max_grad_norm;         /* > 0: clip the global L2 norm of the unscaled gradient; <= 0: off */
    float momentum;              /* SGD with momentum only */
} zero_adam_t;

/* Host-side step state, read and updated by a step.  32 bytes. */
typedef struct zero_state {
    int64_t t;                   /* Adam steps applied so far; a clean step applies t+1 */
    float loss_scale;            /* S: gradients arrive multiplied by S */
    float min_loss_scale;        /* dynamic scaling never halves below this */
    int32_t dynamic;             /* 0 static scale; 1 halve on overflow, double after growth_interval clean steps */
    int32_t growth_interval;     /* 0: never grow */
    int32_t good_steps;          /* consecutive clean steps (dynamic scaling) */
    int32_t reserved;
} zero_state_t;

/* Caller-owned device buffers (layout above).  88 bytes. */
typedef struct zero_buffers {
    void* const* grads;          /* [N] */
    void* const* params16;       /* [N] */
    float* w[2];
    float* m[2];
    float* v[2];
    void* reduced;
    void* workspace;
    int32_t cur;                 /* 0 or 1; the fused path flips it after a clean step */
    int32_t reserved;
} zero_buffers_t;

/* Outcome of one step.  64 bytes. */
typedef struct zero_step_result {
    int64_t t;                   /* step count after the step */
    int64_t hbm_bytes;           /* algorithmic HBM bytes moved */
    int64_t comm_counted_bytes;  /* bytes crossing simulated rank boundaries */
    double grad_norm;            /* clipping on: ||g||_2 (+inf on overflow); off: -1 */
    uint32_t overflow;           /* 1 if any reduced gradient element was inf or NaN */
    int32_t skipped;             /* 1 if the update was discarded (overflow) */
    float clip_coef;             /* min(1, max_grad_norm/(||g||+1e-6)); 1 when off or skipped */
    float loss_scale_used;
    float new_loss_scale;
    int32_t kernel_launches;     /* kernels this step launched */
    int32_t path;                /* 0 fused, 1 two-pass */
    int32_t reserved;
} zero_step_result_t;

/* ---- planning (host only, no CUDA calls) ------------------------------ */

/* Partition, bucket table sizes, buffer sizes and the paper's accounting for
 * cfg.  Source: the shard rule -- each of the N_d ranks keeps one contiguous
 * 1/N_d of the flattened states, per stage (ZeRO visual reading, stage list;
 * "ZeRO：大模型训练的内存优化革命" 3.1.1-3.1.3) -- the constant-size gradient
 * buckets (same page, 3.2.2, C_B; SC-2020 ZeRO notes, "Deep Dive into
 * ZeRO-R") and the per-stage memory and communication formulas (ZeRO visual
 * reading, stage formulas and communication accounting).  The shard is padded
 * to align_elems (a layout choice the pages leave open).  cfg and out are
 * caller memory; nothing is kept.  Errors: ZERO_EINVAL (bad field or NULL),
 * ZERO_EUNSUPPORTED (n_ranks outside 1..64, n_params above 2^40). */
zero_status_t zero_plan(const zero_config_t* cfg, zero_plan_t* out);

/* Segments of bucket b: for each rank owning part of it, in rank order,
 * seg[3k] = rank, seg[3k+1] = offset inside that rank's shard, seg[3k+2] =
 * length -- where the reduce-scatter of one fusion bucket sends its
 * elements ("ZeRO：大模型训练的内存优化革命" 3.1.2 and 3.2.2; ZeRO visual
 * reading, stage list: the owner of a gradient shard reduces it).  seg must
 * hold 3*n_ranks entries; *n_seg receives the count.  Errors: ZERO_EINVAL
 * (b outside 0..n_buckets-1, NULL output), as zero_plan for cfg. */
zero_status_t zero_plan_bucket(const zero_config_t* cfg, int64_t b, int64_t* seg, int32_t* n_seg);

/* Flat start and length of stage-3 layer `layer`: the unit that stage 3
 * gathers before the layer runs and releases after it
 * ("ZeRO：大模型训练的内存优化革命" 3.1.3; ZeRO visual reading, stage-3
 * section).  Errors: ZERO_EINVAL (layer out of range, NULL output). */
zero_status_t zero_plan_layer(const zero_config_t* cfg, int32_t layer, int64_t* start, int64_t* len);

/* Per-rank model-state bytes of the paper's accounting (ZeRO visual reading,
 * stage formulas; Table 1): out[0] parameters, out[1] gradients, out[2]
 * optimizer state, out[3] total.  param_bytes b (2 mixed precision, 4 fp32),
 * optim_K K (12 mixed-precision Adam; the page's calculator also uses 4 for
 * fp32 SGD with momentum, 0 for SGD).  Stage 0: (2b+K)Psi; 1: 2b*Psi +
 * K*Psi/N; 2: b*Psi + (b+K)*Psi/N; 3: (2b+K)*Psi/N. */
zero_status_t zero_model_state_bytes(int64_t n_params, int32_t n_ranks, int32_t stage,
                                     int32_t param_bytes, int32_t optim_K, double out[4]);

/* Communication per step.  *paper_per_rank: the paper's volume, 2*Psi*b for
 * stages 0-2 and 3*Psi*b for stage 3 ("AI论文陪读·ZeRO" section 04; ZeRO
 * visual reading, communication accounting).  *counted_all_ranks: bytes that
 * cross simulated rank boundaries, k*(N-1)*Psi*b with k = 2 (stages 0, 2),
 * 3 (stage 1, counting its end-of-step parameter all-gather; stage 3, two
 * parameter all-gathers and one reduce-scatter). */
zero_status_t zero_comm_bytes(int64_t n_params, int32_t n_ranks, int32_t stage, int32_t param_bytes,
                              double* paper_per_rank, int64_t* counted_all_ranks);

/* ---- the step (device) --------------------------------------------------- */

/* One complete optimizer step over all buckets: begin, every bucket, end.
 * zero_step dispatches on cfg->stage; zero_step_stageK requires stage K
 * (ZERO_EINVAL otherwise).  Sources, per stage: stage 0 is plain data
 * parallelism (every rank keeps every state, gradients all-reduced); stage 1
 * partitions the optimizer state (P_os), stage 2 also the gradients
 * (P_os+g), stage 3 also the parameters (P_os+g+p)
 * ("ZeRO：大模型训练的内存优化革命" 3.1.1-3.1.3; ZeRO visual reading, stage
 * list and communication accounting: reduce-scatter, update of the owned
 * shard, all-gather).  The update itself is the mixed-precision one: fp32
 * master weights and optimizer state updated from the 16-bit gradient, then
 * cast back to 16 bits (SC-2020 ZeRO notes, "Where Did All the Memory Go? /
 * Model States"; "AI论文陪读·ZeRO" section 01).  Adam is Kingma & Ba,
 * Algorithm 1 (the pages name Adam but do not print it).  The buffers are the
 * caller's (layout above); the call returns after reading the step's
 * overflow flag (one synchronisation of `stream`).  Errors: ZERO_EINVAL,
 * ZERO_EALIGN, ZERO_ENOMEM (missing buffer), ZERO_ECUDA (a launch or the
 * synchronisation failed; the message has the CUDA error), ZERO_EUNSUPPORTED.
 * On any error before the first launch nothing on the device has changed. */
zero_status_t zero_step(const zero_config_t* cfg, const zero_plan_t* plan, zero_buffers_t* bufs,
                        const zero_adam_t* adam, zero_state_t* state, void* stream,
                        zero_step_result_t* out);
zero_status_t zero_step_stage0(const zero_config_t* cfg, const zero_plan_t* plan, zero_buffers_t* bufs,
                               const zero_adam_t* adam, zero_state_t* state, void* stream,
                               zero_step_result_t* out);
zero_status_t zero_step_stage1(const zero_config_t* cfg, const zero_plan_t* plan, zero_buffers_t* bufs,
                               const zero_adam_t* adam, zero_state_t* state, void* stream,
                               zero_step_result_t* out);
zero_status_t zero_step_stage2(const zero_config_t* cfg, const zero_plan_t* plan, zero_buffers_t* bufs,
                               const zero_adam_t* adam, zero_state_t* state, void* stream,
                               zero_step_result_t* out);
zero_status_t zero_step_stage3(const zero_config_t* cfg, const zero_plan_t* plan, zero_buffers_t* bufs,
                               const zero_adam_t* adam, zero_state_t* state, void* stream,
                               zero_step_result_t* out);

/* The same step, bucket by bucket, for gradients that arrive one bucket at a
 * time (backward hooks filling a constant-size bucket: the fused buffer of
 * "ZeRO：大模型训练的内存优化革命" 3.2.2 and the SC-2020 ZeRO notes, "Deep
 * Dive into ZeRO-R", C_B).  Call begin, then
 * zero_step_bucket exactly once for every bucket b in any order, then end,
 * all on one stream with unchanged arguments.
 * bucket_grads: NULL to read bufs->grads, or (stages 2 and 3 only) a host
 * array of N device pointers, each to this bucket's gradient window (bucket
 * length, element 0 = the bucket's first flat index); it may be reused for
 * the next bucket once this bucket's kernel has run on the stream. */
zero_status_t zero_step_begin(const zero_config_t* cfg, const zero_plan_t* plan, zero_buffers_t* bufs,
                              const zero_adam_t* adam, const zero_state_t* state, void* stream);
zero_status_t zero_step_bucket(const zero_config_t* cfg, const zero_plan_t* plan, zero_buffers_t* bufs,
                               const zero_adam_t* adam, const zero_state_t* state, int64_t bucket,
                               void* const* bucket_grads, void* stream);
zero_status_t zero_step_end(const zero_config_t* cfg, const zero_plan_t* plan, zero_buffers_t* bufs,
                            const zero_adam_t* adam, zero_state_t* state, void* stream,
                            zero_step_result_t* out);
/* Several buckets of the same step in one call: buckets[0..count), in that
 * order, each exactly once in the step as for zero_step_bucket.
 * bucket_grads: NULL, or (stages 2 and 3) count*N device pointers, bucket k's
 * N windows at bucket_grads[k*N .. k*N+N).  The first kernel follows plain
 * stream order; each later one is a programmatic dependent of the one before
 * (it may start while its predecessor drains, as inside zero_step), so every
 * window must hold its gradients before the call's first kernel runs.  Same
 * errors as zero_step_bucket (ZERO_EINVAL for an index out of range). */
zero_status_t zero_step_buckets(const zero_config_t* cfg, const zero_plan_t* plan, zero_buffers_t* bufs,
                                const zero_adam_t* adam, const zero_state_t* state, const int64_t* buckets,
                                int32_t count, void* const* bucket_grads, void* stream);

/* Stage 3: copy layer `layer`'s 16-bit parameters from the owners' shards
 * (param_shards[r], P elements each) into each of the n_dst destination
 * buffers dst[d] (capacity max_layer_elems; element j = flat index
 * layer_start + j).  The parameter all-gather that runs before a layer's
 * forward and again before its backward (ZeRO visual reading, communication
 * accounting; "ZeRO：大模型训练的内存优化革命" 3.1.3).  n_dst 1..64.  With the
 * destinations and the layer's shards in device memory the layer is written
 * 2 MB chunk by chunk, destination by destination (the chunk's source stays
 * in L2); otherwise each value is read once and stored to every
 * destination. */
zero_status_t zero_gather_layer(const zero_config_t* cfg, const zero_plan_t* plan, int32_t layer,
                                void* const* param_shards, void* const* dst, int32_t n_dst, void* stream);

/* ---- steps without host synchronisation ------------------------------------
 * The step state (t, the beta powers of the bias correction, the loss scale
 * and its scaler) can live in device memory instead: zero_step_async then
 * enqueues the whole step and returns without waiting, so steps pipeline
 * back to back and a step can be captured in a CUDA graph.  A prepare
 * kernel clears the workspace head and derives the step's scalars from the
 * state block; after the bucket kernels a commit writes the outcome back (t
 * and the beta powers advance on a clean step; the scaler halves on
 * overflow and grows after growth_interval clean steps) together with the
 * last step's flag, norm and clip coefficient, which zero_dev_state_read
 * brings to the host.  Results equal the synchronised step's bit for bit.
 * Fused path: the host does not learn the flag, so bufs->cur flips on every
 * call; after an overflow the restore (which also runs the commit) copies
 * the unchanged state into the copy the next step reads and restores the
 * parameters.  A graph captured from one call therefore serves every other
 * step: capture one call per value of bufs->cur and replay them alternately.
 * The step's kernels are launched as one chain of programmatic dependent
 * launches (each small kernel, and the first bucket kernel, waits for its
 * predecessor before it touches memory).  A two-pass step (clipping, or no
 * shadow state) of a model that is one bucket, in stages 2-3, moving at
 * most 64 MiB (n x (2 N e + 2 e + 24) bytes, e the value size) is two
 * kernels after a memset of the workspace head: pass 1, whose last block
 * derives the scalars and finishes the norm, and pass 2, whose last block
 * commits.
 * The device state block is 64 bytes, 16-byte aligned, caller-owned. */
typedef struct zero_dev_state { int64_t opaque[8]; } zero_dev_state_t;   /* 64 bytes */

/* Initialise the block from a host state (synchronises `stream`); `adam`
 * must carry the betas the steps will use (both in [0, 1)). */
zero_status_t zero_dev_state_init(void* dev_state, const zero_adam_t* adam, const zero_state_t* state, void* stream);
/* Enqueue one step (all buckets); never synchronises.  *kernel_launches
 * (may be NULL) receives the kernels it launched. */
zero_status_t zero_step_async(const zero_config_t* cfg, const zero_plan_t* plan, zero_buffers_t* bufs,
                              const zero_adam_t* adam, void* dev_state, void* stream, int32_t* kernel_launches);
/* The same step one bucket at a time (for buckets that become ready during
 * the backward pass), with the step state on the device: begin (the prepare
 * kernel), then zero_step_bucket_async for every bucket in any order --
 * bucket_grads as for zero_step_bucket (stages 2/3 only) -- then end (the
 * two-pass path's finalize and update kernels, and the commit; on the fused
 * path bufs->cur flips).  None of them synchronises; the sequence can be
 * captured in a graph. */
zero_status_t zero_step_begin_async(const zero_config_t* cfg, const zero_plan_t* plan, zero_buffers_t* bufs,
                                    const zero_adam_t* adam, void* dev_state, void* stream);
zero_status_t zero_step_bucket_async(const zero_config_t* cfg, const zero_plan_t* plan, zero_buffers_t* bufs,
                                     const zero_adam_t* adam, int64_t bucket, void* const* bucket_grads,
                                     void* stream);
/* zero_step_buckets for the device-state protocol (between begin_async and
 * end_async). */
zero_status_t zero_step_buckets_async(const zero_config_t* cfg, const zero_plan_t* plan, zero_buffers_t* bufs,
                                      const zero_adam_t* adam, const int64_t* buckets, int32_t count,
                                      void* const* bucket_grads, void* stream);
zero_status_t zero_step_end_async(const zero_config_t* cfg, const zero_plan_t* plan, zero_buffers_t* bufs,
                                  const zero_adam_t* adam, void* dev_state, void* stream, int32_t* kernel_launches);
/* Copy the block to the host (synchronises `stream`): the current step state
 * and the last step's outcome (t, overflow, skipped, grad_norm, clip_coef,
 * new_loss_scale; path -1).  Returns ZERO_ETIMEOUT (outputs still filled) if
 * a bounded wait inside the last step's kernels ran out; that step was not
 * applied and the loss scaler was left as it was. */
zero_status_t zero_dev_state_read(const void* dev_state, zero_state_t* state, zero_step_result_t* last, void* stream);

/* ---- stage 3: gathers ahead of use under a live-parameter budget ---------
 * A fetcher gathers the layers of one pass (an order of layers: forward
 * 0..L-1, backward L-1..0, any sequence) into a caller-owned pool of
 * `capacity` 16-bit elements per destination, placing them as a ring in
 * fetch order, so the layers resident at once never exceed the capacity
 * (DeepSpeed's stage3_max_live_parameters; ZeRO visual reading, stage-3
 * section: gather the next layers ahead of time, release after use).  Up to
 * `depth` layers ahead are gathered on `side_stream`; a fetch makes the
 * caller's stream wait for that layer only; a release makes the side stream
 * wait before reusing the space.  Protocol, per position pos = 0, 1, ...:
 * zero_fetch_layer(pos) -> use the layer at *offset in every pool buffer on
 * `stream` -> zero_release_layer(pos).  The caller keeps `order`, the pool,
 * the shards and the 2*(depth+1) events (cudaEvent_t, created by the caller)
 * alive while the fetcher is used; zero_fetcher_t is caller memory holding
 * the fetcher's state (no allocation).  Layer sizes are rounded up to 8
 * elements in the pool; capacity must hold the largest layer. */
#define ZERO_FETCH_MAX_DEPTH 32
#define ZERO_FETCH_MAX_RESIDENT 128
typedef struct zero_fetcher { int64_t opaque[1024]; } zero_fetcher_t;   /* 8 KB */

zero_status_t zero_fetcher_init(zero_fetcher_t* f, const zero_config_t* cfg, const zero_plan_t* plan,
                                void* const* param_shards, void* const* pool, int32_t n_dst, int64_t capacity,
                                const int32_t* order, int32_t n_order, int32_t depth, void* side_stream,
                                void* const* events, int32_t n_events);
/* Make layer order[pos] resident and ordered before later work on `stream`;
 * *offset receives its element offset in each pool buffer. */
zero_status_t zero_fetch_layer(zero_fetcher_t* f, int32_t pos, void* stream, int64_t* offset);
/* Done with order[pos] (after the work already enqueued on `stream`). */
zero_status_t zero_release_layer(zero_fetcher_t* f, int32_t pos, void* stream);
/* Largest resident element count reached, gathers issued. */
zero_status_t zero_fetcher_stats(const zero_fetcher_t* f, int64_t* max_live, int32_t* gathers);
/* The fetcher's decisions without a GPU: for each position q, issue_at[q] is
 * the position at whose fetch its gather is issued and offsets[q] its pool
 * offset; *max_live the largest resident element count.  ZERO_ENOMEM if a
 * layer cannot fit; ZERO_EINVAL if capacity is below the largest layer. */
zero_status_t zero_fetch_schedule(const int64_t* layer_sizes, int32_t n_layers, const int32_t* order, int32_t n_order,
                                  int64_t capacity, int32_t depth, int32_t* issue_at, int64_t* offsets,
                                  int64_t* max_live);

/* Stage-2 step that allocates nothing and needs no scratch from the caller.
 * The paper has no counterpart: this exists for callers that cannot obtain
 * device memory for the workspace and the reduced-gradient buffer -- code
 * running inside another runtime that owns the device's memory pool, or code
 * that must not allocate after start-up.  The scratch lives in one static
 * device array inside the library (4 KB + 16 MiB, held by every GPU that
 * loads the library until the process exits), so the plan's padded_elems
 * must be at most 8,388,608 (ZERO_EUNSUPPORTED otherwise, with a message).
 * Same arguments and results as zero_step_stage2, except: bufs->workspace,
 * bufs->reduced and the shadow copies bufs->w/m/v[1-cur] are ignored; the
 * step always takes the two-pass path and updates the [cur] state in place
 * (clipping allowed).  The caller still passes the gradients, parameters and
 * fp32 state.  The array used is the current device's, so `stream` must
 * belong to the current device (ZERO_EINVAL otherwise; NULL is the current
 * device's legacy default stream).  The first call on each device looks up the array's device
 * address (cudaGetSymbolAddress, with that device current); make that first
 * call before any stream capture.  Each call clears the array's workspace
 * part before use; the rest keeps the last call's contents.  All calls share
 * the array: calls whose kernels overlap on the GPU (other streams or host
 * threads) race on it. */
zero_status_t zero_step_stage2_noalloc(const zero_config_t* cfg, const zero_plan_t* plan, zero_buffers_t* bufs,
                                       const zero_adam_t* adam, zero_state_t* state, void* stream,
                                       zero_step_result_t* out);

/* ---- P_a: partitioned activation checkpoints (ZeRO-R) --------------------
 * Under model parallelism the input of a layer -- the activation checkpoint
 * that backward recomputes the layer from -- is replicated on all N_m
 * model-parallel ranks.  P_a keeps a 1/N_m slice per rank after the forward
 * pass and rebuilds the checkpoint with an all-gather when backward needs
 * it; P_a+cpu keeps the slices in host memory ("ZeRO：大模型训练的内存优化
 * 革命" 3.2.1; SC-2020 ZeRO notes, "P_a: Partitioned Activation
 * Checkpointing").  The N_m ranks are simulated as buffers, like the
 * data-parallel ranks.  Slice of rank r: values [r*P, min((r+1)*P, act_elems)),
 * P = ceil(act_elems / N_m) rounded up to align_elems.  72 bytes. */
typedef struct zero_pa_plan {
    int64_t act_elems;              /* values in one checkpoint, >= 0 */
    int64_t shard_elems;            /* P */
    int64_t align_elems;            /* 0 -> 2048; a multiple of 8 */
    int32_t n_mp;                   /* N_m, 1..64 */
    int32_t dtype;                  /* zero_dtype_t of the activations (2 or 4 bytes) */
    int64_t mem_per_rank_bytes;     /* without P_a: the whole checkpoint on every rank */
    int64_t mem_per_rank_pa_bytes;  /* with P_a: one slice (P_a+cpu: none on the GPU) */
    int64_t gather_bytes;           /* bytes crossing simulated rank boundaries in one all-gather, all ranks */
    int64_t reserved[2];
} zero_pa_plan_t;

zero_status_t zero_pa_plan(int64_t act_elems, int32_t n_mp, int32_t dtype, int64_t align_elems,
                           zero_pa_plan_t* out);
/* After the forward pass: rank r copies its slice of replicas[r] (the
 * checkpoint as rank r holds it: act_elems values) to shards[r] (room for
 * shard_elems values; device or pinned host memory -- P_a+cpu).  Arrays of
 * n_mp pointers, 16-byte aligned.  One kernel launch, asynchronous. */
zero_status_t zero_pa_partition(const zero_pa_plan_t* plan, const void* const* replicas, void* const* shards,
                                void* stream);
/* Before the layer's recomputation: the all-gather -- the checkpoint rebuilt
 * from the n_mp slices into each of dst[0..n_dst) (act_elems values each;
 * n_dst 1..64).  One kernel launch, asynchronous. */
zero_status_t zero_pa_gather(const zero_pa_plan_t* plan, const void* const* shards, void* const* dst, int32_t n_dst,
                             void* stream);

/* ---- layer norm -----------------------------------------------------------
 * The norm in front of a transformer block or the vocabulary projection, and
 * its gradient, on rows of `dim` values:
 *   y  = (x - mean) * rstd * weight + bias,  rstd = 1/sqrt(var + eps)
 *   dx = rstd * (g - avg(g) - xhat * avg(g * xhat)),  g = dy * weight,
 *        xhat = (x - mean) * rstd,  avg over the row
 *   dweight = sum over rows of dy * xhat,  dbias = sum over rows of dy
 * Every sum is a binary32 sum in an order fixed by the plan; each output is
 * rounded once to its type.  All of x, weight, bias, y, dy, dx, dweight,
 * dbias have the plan's dtype; mean and rstd are binary32, one per row.
 * Rows may lie further apart than dim (strides, in values); what is between
 * them is neither read nor written.  Outputs must not overlap inputs.
 * Pointers need the alignment of their type only: rows that start on 16-byte
 * boundaries take 16-byte accesses, 16-bit ones on 4-byte boundaries 4-byte
 * accesses (1.6 times slower), others single-value ones (two to two and a half
 * times slower in 16-bit types).  72 bytes. */
typedef struct zero_ln_plan {
    int64_t rows, dim;
    int64_t x_stride;            /* values between rows of x and dx */
    int64_t y_stride;            /* values between rows of y and dy */
    int64_t workspace_bytes;     /* zero_ln_backward's workspace */
    int64_t hbm_bytes_forward;   /* algorithmic HBM bytes (each array access once) */
    int64_t hbm_bytes_backward;
    int32_t dtype;               /* zero_dtype_t */
    int32_t blocks;              /* backward: row groups summed apart */
    int64_t reserved;
} zero_ln_plan_t;

/* Host only.  strides 0: dim.  rows >= 0, 1 <= dim <= 2^20, strides >= dim.
 * Errors: ZERO_EINVAL, ZERO_EUNSUPPORTED (rows or dim too large). */
zero_status_t zero_ln_plan(int64_t rows, int64_t dim, int32_t dtype, int64_t x_stride, int64_t y_stride,
                           zero_ln_plan_t* out);
/* weight NULL: ones; bias NULL: zeros; mean, rstd NULL: not written.
 * Asynchronous on `stream`.  Errors: ZERO_EINVAL (plan not made by
 * zero_ln_plan, eps < 0 or NaN), ZERO_ENOMEM (x or y NULL), ZERO_EALIGN,
 * ZERO_ECUDA. */
zero_status_t zero_ln_forward(const zero_ln_plan_t* plan, const void* x, const void* weight, const void* bias,
                              float eps, void* y, float* mean, float* rstd, void* stream);
/* mean and rstd as the forward pass wrote them.  dx, dweight, dbias NULL:
 * not computed.  dweight and dbias are overwritten, with zeros when there are no rows.  workspace:
 * plan->workspace_bytes, 16-byte aligned (may be NULL when neither dweight
 * nor dbias is wanted). */
zero_status_t zero_ln_backward(const zero_ln_plan_t* plan, const void* dy, const void* x, const void* weight,
                               const float* mean, const float* rstd, void* dx, void* dweight, void* dbias,
                               void* workspace, void* stream);

/* ---- root-mean-square norm -------------------------------------------------
 * The norm of a block that adds its output x to a residual stream, and its
 * gradient, on rows of `dim` values (Zhang & Sennrich, "Root Mean Square Layer
 * Normalization"):
 *   h  = x + residual, rounded to the dtype (h = x without a residual)
 *   y  = h * rstd * weight,  rstd = 1/sqrt(avg(h^2) + eps), avg over the row
 *   dx = rstd * (g - xhat * avg(g * xhat)) + dh,  g = dy * weight, xhat = h * rstd
 *   dweight = sum over rows of dy * xhat
 * dh is the gradient that reaches h by the stream itself; dx is that of x and of
 * the residual alike.  All of x, residual, h, weight, y, dy, dh, dx, dweight
 * have the plan's dtype; rstd is binary32, one per row.  Sums are binary32 in
 * an order fixed by the plan and the pointers' alignment; each output is rounded
 * once.  Squares are summed as they are: a row with values over 2^63 or so in
 * bfloat16 or binary32 has an infinite sum, and y 0; with eps 0 one whose values are
 * all under 2^-75 or so has a sum of 0, and y as h * infinity.
 * y may also be (or be as well) q, one byte per value with a scale byte for every
 * `block` (32 or 128) values of a row, the last block of a row maybe shorter:
 *   q = e4m3 (1 sign, 4 exponent, 3 fraction bits, 448 the largest) of
 *   y * 2^(127 - e), rounded to nearest even once, from binary32;
 *   e: the least byte >= 0 with the block's largest |y| <= 448 * 2^(e - 127);
 *   a block with an infinity or a NaN: e = 255, codes 0x7f or 0xff (NaN).
 * Rows may lie further apart than dim (strides, in values; x_stride: rows of x,
 * residual, h, dh and dx; y_stride: of y, dy, q and values); what is between them is
 * neither read nor written.  q_scale rows are scale_cols bytes apart.  Pointers need
 * the alignment of their type only: rows that all start on 16-byte boundaries (the
 * weight too) take 16-byte accesses, up to 65536 bytes a row forward and 32768 backward;
 * others single-value ones, up to 2.2 times slower.  zero_rms_values takes 16 codes at
 * once where q, values and their rows start on 16 bytes and dim is a multiple of 16,
 * else one (up to 3 times slower).  Outputs must not overlap inputs, but h may be x or
 * residual itself and dx may be dh itself.  88 bytes. */
typedef struct zero_rms_plan {
    int64_t rows, dim;
    int64_t x_stride, y_stride;
    int64_t scale_cols;          /* ceil(dim / block); 0 without 8-bit results */
    int64_t workspace_bytes;     /* zero_rms_backward's workspace */
    int64_t hbm_bytes_forward;   /* algorithmic HBM bytes, with a residual; with a block: q, else y */
    int64_t hbm_bytes_backward;
    int32_t dtype;               /* zero_dtype_t */
    int32_t block;               /* 0: no 8-bit results */
    int32_t blocks;              /* backward: row groups summed apart */
    int32_t reserved;
    int64_t reserved2;
} zero_rms_plan_t;

/* Host only.  strides 0: dim.  rows >= 0, 1 <= dim <= 2^20, strides >= dim.
 * Errors: ZERO_EINVAL, ZERO_EUNSUPPORTED (rows or dim too large, another block). */
zero_status_t zero_rms_plan(int64_t rows, int64_t dim, int32_t dtype, int64_t x_stride, int64_t y_stride, int32_t block,
                            zero_rms_plan_t* out);
/* residual NULL: h = x, and h must be NULL; else h is written.  weight NULL:
 * ones.  y NULL or q NULL: not written (not both).  rstd NULL: not written.
 * Asynchronous on `stream`.  Errors: ZERO_EINVAL (plan not made by
 * zero_rms_plan, eps < 0 or NaN, q without a block), ZERO_ENOMEM, ZERO_EALIGN,
 * ZERO_ECUDA. */
zero_status_t zero_rms_forward(const zero_rms_plan_t* plan, const void* x, const void* residual, const void* weight,
                               float eps, void* h, void* y, void* q, uint8_t* q_scale, float* rstd, void* stream);
/* 8-bit results as bfloat16 values, exact (under 2^-133 cut to its subnormals). */
zero_status_t zero_rms_values(const zero_rms_plan_t* plan, const void* q, const uint8_t* q_scale, void* values,
                              void* stream);
/* h and rstd as the forward pass had them.  dh NULL: 0.  dx, dweight NULL: not
 * computed; dweight is overwritten, with zeros when there are no rows.
 * workspace: plan->workspace_bytes, 16-byte aligned (may be NULL without
 * dweight). */
zero_status_t zero_rms_backward(const zero_rms_plan_t* plan, const void* dy, const void* dh, const void* h,
                                const void* weight, const float* rstd, void* dx, void* dweight, void* workspace,
                                void* stream);

/* ---- softmax cross entropy over a large vocabulary ---------------------------
 * The loss of tokens' last hidden states x [tokens, hidden] against a weight
 * w [vocab, hidden] (a vocabulary projection, or a tied embedding), without
 * the [tokens, vocab] logits in memory:
 *   z = x w^T;  lse_i = log sum_v exp z_iv;  loss_i = lse_i - z_i,t(i)
 *   G_iv = s_i (exp(z_iv - lse_i) - [v = t(i)]);  dx = G w;  dw = G^T x
 * The forward pass keeps one running maximum and sum per token and strip of
 * 128 vocabulary entries.  The backward pass computes z again, a piece of the
 * vocabulary at a time, and holds G of one piece in 16 bits.
 * x, w, dx and dw have the plan's dtype (ZERO_FP16 or ZERO_BF16; ZERO_FP32 is
 * ZERO_EUNSUPPORTED); products are accumulated in binary32 (1024 values at a
 * time on the tensor cores, which round toward zero, those sums to nearest;
 * the loss of more than 3 tokens and G use the same z, up to 3 tokens' loss is
 * summed by plain multiply-adds and G's z in steps of 512), softmax
 * statistics and loss are binary32, dx and dw are rounded once, and G is
 * rounded once, to the dtype (the operand type of the products that use it),
 * scaled so that its largest row factor is 1 (binary16: 2^14, so its absolute
 * spacing, 2^-38 of the largest |s_i|, cuts small probabilities of tokens whose
 * factors are some 10^6 times below it).
 * A token whose target is outside 0..vocab-1 (such as -100) has no loss: its
 * loss is 0 and its row of dx is 0, whatever x and w hold (its row of x still
 * enters dw's product, times 0: an infinity or NaN there makes dw NaN).  Rows
 * may lie further apart than hidden (strides in values, multiples of 8).  All
 * pointers 16-byte aligned but targets, loss, lse, total and dloss (alignment
 * of their type).  Results do not depend on timing: equal calls give equal
 * bits.  96 bytes. */
typedef struct zero_ce_plan {
    int64_t tokens, vocab, hidden;
    int64_t x_stride, w_stride;  /* values between rows of x and dx, of w and dw */
    int64_t piece;               /* vocabulary entries per piece of the backward pass, a multiple of 256 */
    int64_t workspace_bytes;
    int64_t flops_forward;       /* 2 tokens vocab hidden */
    int64_t flops_backward;      /* 6 tokens vocab hidden: z again, dx, dw */
    int32_t dtype;
    int32_t splits;              /* parts of the vocabulary that dx's product sums apart */
    int64_t reserved[2];
} zero_ce_plan_t;

/* Host only.  strides 0: hidden (then a multiple of 8); piece 0: chosen so
 * that G takes about 512 MiB, else rounded up to a multiple of 256.  tokens
 * >= 0, vocab >= 1, hidden >= 1.  Errors: ZERO_EINVAL, ZERO_EALIGN (a stride
 * that is not a multiple of 8), ZERO_EUNSUPPORTED (tokens or vocab over 2^24,
 * hidden over 2^20, their product about 2^58 or more). */
zero_status_t zero_ce_plan(int64_t tokens, int64_t vocab, int64_t hidden, int32_t dtype, int64_t x_stride,
                           int64_t w_stride, int64_t piece, zero_ce_plan_t* out);
/* loss, lse: binary32, one per token.  total (may be NULL): {mean loss of the
 * tokens that have one (0 when none has), their number}.  workspace:
 * plan->workspace_bytes, contents scratch.  Asynchronous. */
zero_status_t zero_ce_forward(const zero_ce_plan_t* plan, const void* x, const void* w, const int64_t* targets,
                              float* loss, float* lse, float* total, void* workspace, void* stream);
/* lse as the forward pass wrote it.  s_i = dloss[i] * grad_scale, or with
 * dloss NULL grad_scale / (number of tokens that have a loss): the gradient
 * of the mean, times grad_scale (the loss scale).  An s_i that is not finite
 * makes its token's dx NaN, and dw, and no other token's dx.  dx, dw NULL: not
 * computed; they are overwritten otherwise (with zeros where there are no
 * tokens). */
zero_status_t zero_ce_backward(const zero_ce_plan_t* plan, const void* x, const void* w, const int64_t* targets,
                               const float* lse, const float* dloss, float grad_scale, void* dx, void* dw,
                               void* workspace, void* stream);
/* Synchronises `stream`; ZERO_ETIMEOUT if a bounded wait inside the last
 * forward or backward call with this workspace ran out (a call that computes
 * nothing has none).  Losses of tokens that have one, dx and dw are then NaN, so
 * zero_adamw_check sees them too. */
zero_status_t zero_ce_status(const zero_ce_plan_t* plan, const void* workspace, void* stream);

/* ---- log probabilities over a large vocabulary ---------------------------------
 * What a policy's update and a scored answer need of the last hidden states x
 * [tokens, hidden] against a weight w [vocab, hidden], without the logits in
 * memory unless alternatives are asked for (the products are cross entropy's):
 *   z = x w^T * scale (scale: the inverse temperature);  lse_i = log sum_v exp z_iv
 *   logp_i = z_i,t(i) - lse_i;  p = exp(z - lse);  entropy_i = -sum_v p_iv log p_iv
 *   the `top` most likely entries, in falling order of their logits, the lower
 *   index first where they are equal
 *   G_iv = a_i ([v = t(i)] - p_iv) - b_i p_iv (log p_iv + entropy_i)
 *   dx = scale * G w;  dw = scale * G^T x
 * with a = dlogp * grad_scale and b = dentropy * grad_scale.  Types, strides,
 * alignment, sums, statistics and the 16-bit G are as for cross entropy (G's rows
 * are scaled by the largest |a_i| + 4 |b_i|); top_index has 8-byte alignment, other
 * binary32 arrays 4-byte.  A token whose target is outside 0..vocab-1 has logp 0
 * and no dlogp; its entropy, alternatives and dentropy are like any other's.
 * Alternatives are logits above -infinity that are numbers; where there are fewer
 * than `top`, log probability -infinity and index -1.  The order is that of the
 * logits as computed: those closer than their binary32 sums' rounding may
 * change places.  A row with a logit that is NaN or +infinity, or with none above
 * -infinity, has NaN logp and entropy; a -infinity beside others adds nothing to
 * either.  With alternatives the workspace has room for the logits of `rows` tokens
 * at a time while they are sought (binary32, 2 GiB at most unless 256 rows need more),
 * of which large batches write a part only.
 * Results do not depend on timing: equal calls give equal bits.  104 bytes. */
typedef struct zero_lp_plan {
    int64_t tokens, vocab, hidden;
    int64_t x_stride, w_stride;  /* values between rows of x and dx, of w and dw */
    int64_t piece;               /* vocabulary entries per piece of the backward pass, a multiple of 256 */
    int64_t rows;                /* tokens per piece of the forward pass, a multiple of 256 */
    int64_t workspace_bytes;
    int64_t flops_forward;       /* 2 tokens vocab hidden */
    int64_t flops_backward;      /* 6 tokens vocab hidden: z again, dx, dw */
    int32_t dtype;
    int32_t splits;              /* parts of the vocabulary that dx's product sums apart */
    int32_t top;
    int32_t reserved;
    int64_t reserved2;
} zero_lp_plan_t;

/* Host only.  As zero_ce_plan; 0 <= top <= 32 alternatives (more:
 * ZERO_EUNSUPPORTED). */
zero_status_t zero_lp_plan(int64_t tokens, int64_t vocab, int64_t hidden, int32_t dtype, int64_t x_stride, int64_t w_stride,
                           int64_t piece, int32_t top, zero_lp_plan_t* out);
/* scale > 0.  logp, lse, entropy (may be NULL): binary32, one per token.
 * top_logp, top_index: [tokens, top] (NULL where top is 0).  workspace:
 * plan->workspace_bytes, contents scratch.  Asynchronous. */
zero_status_t zero_lp_forward(const zero_lp_plan_t* plan, const void* x, const void* w, const int64_t* targets, float scale,
                              float* logp, float* lse, float* entropy, float* top_logp, int64_t* top_index, void* workspace,
                              void* stream);
/* lse and entropy as the forward pass wrote them with the same scale.  dlogp,
 * dentropy: binary32, one per token, NULL: 0 (entropy may be NULL without
 * dentropy).  A factor that is not finite makes its token's dx NaN, and dw, and
 * no other token's dx.  dx, dw NULL: not computed; they are overwritten otherwise
 * (dw with zeros where there are no tokens). */
zero_status_t zero_lp_backward(const zero_lp_plan_t* plan, const void* x, const void* w, const int64_t* targets, float scale,
                               const float* lse, const float* entropy, const float* dlogp, const float* dentropy,
                               float grad_scale, void* dx, void* dw, void* workspace, void* stream);
/* As zero_ce_status; after ZERO_ETIMEOUT the forward pass' results and the
 * gradients are NaN, but logp of tokens without a target, which is 0, and
 * top_index, which is -1. */
zero_status_t zero_lp_status(const zero_lp_plan_t* plan, const void* workspace, void* stream);

/* ---- AdamW over a list of tensors -------------------------------------------
 * One optimizer step of every tensor of a list in one kernel launch, for
 * parameters that are not laid out as one flat partitioned vector (a head or
 * an adapter beside the sharded model).  Adam as in the sharded step
 * (Kingma & Ba, Algorithm 1) with decoupled weight decay (Loshchilov &
 * Hutter, "Decoupled Weight Decay Regularization"), g = grad * grad_scale:
 *   w = w * (1 - lr * weight_decay)
 *   m = b1*m + (1-b1)*g;  v = b2*v + (1-b2)*(g*g)
 *   w = w - lr * (m/bc1) / (sqrt(v/bc2) + eps),  bc = 1 - b^t
 * state_bits 32: m, v binary32, one IEEE rounding per operation in the
 * sharded step's order (weight_decay 0 gives its results bit for bit, where
 * the bias corrections agree).
 * state_bits 8: m and r = sqrt(v) are kept in one byte per value, in blocks
 * of 256 values of a tensor with one scale byte each:
 *   scale byte e: the block's values are stored relative to 2^(e-127), e the
 *     exponent field of the largest one plus 2^-4 of its binade (at most 253;
 *     0: the block is zero), so relative magnitudes lie below 31/16, the
 *     largest code, and the largest too can be rounded up;
 *   m: sign bit 7, exponent E = bits 6..4, fraction f = bits 3..0: (16+f)/16 *
 *     2^(E-7), or f/16 * 2^-6 when E = 0;
 *   r: exponent E = bits 7..4, fraction f: (16+f)/16 * 2^(E-15), or f/16 *
 *     2^-14 when E = 0.
 *   A value is rounded down or up to a code at random, up with the chance of
 *   its distance from the lower one (an EMA with b2 = 0.999 moves by 0.1 % a
 *   step, far below a code's spacing, and rounding to nearest would hold it
 *   still.)  A nonzero r is never stored as 0, so no later step divides by
 *   eps alone.  The 16 random bits of value i (its place in the plan's flat
 *   order) come from i, t and seed alone: h = (lo32(i/2) * 0x9E3779B1 +
 *   (i/2 >> 32) * 0x6A09E667 + seed + t * 0x510E527F), h = (h ^ h>>15) *
 *   0xBB67AE85, h = (h ^ h>>15) * 0xA54FF53B, h ^= h>>16 (all mod 2^32); even
 *   i takes the low half, odd i the high half.
 *   The update uses m and r before they are rounded:
 *     r = sqrt(b2*(r*r) + (1-b2)*(g*g));
 *     w = w - (m * (lr/bc1)) / (r * (1/sqrt(bc2)) + eps)
 * master is the binary32 weight; param (may be NULL) receives its cast to
 * the plan's dtype, the type of grad.  A non-finite gradient that is not
 * checked for (zero_adamw_check) makes its weight non-finite too, and 8-bit
 * moments of its whole block useless: scale 253, the largest codes there, 0 and
 * the least nonzero root beside it.  With eps 0 a weight whose
 * gradients were all zero becomes 0/0, as the formula says.  72 bytes. */
typedef struct zero_adamw_tensor {
    const void* grad;
    void* param;                 /* NULL: not written */
    float* master;
    void* m;                     /* float, or one byte per value */
    void* v;
    uint8_t* m_scale;            /* 8-bit states: ceil(numel / 256) bytes (else NULL) */
    uint8_t* v_scale;
    int64_t numel;               /* >= 0 */
    float weight_decay;
    int32_t reserved;            /* 0 */
} zero_adamw_tensor_t;

/* 64 bytes. */
typedef struct zero_adamw_plan {
    int64_t n_tensors;
    int64_t numel;               /* values in all tensors */
    int64_t flat_elems;          /* the flat order: tensor after tensor, each from a multiple of 256 */
    int64_t n_chunks;
    int64_t table_bytes;         /* device memory of the list */
    int64_t hbm_bytes;           /* algorithmic HBM bytes of one step */
    int32_t dtype, state_bits;   /* zero_dtype_t; 8 or 32 */
    int64_t mark;                /* of the fields above: a plan is used as zero_adamw_plan made it */
} zero_adamw_plan_t;

/* Hyper-parameters of one step.  32 bytes. */
typedef struct zero_adamw {
    int64_t t;                   /* the step's number, from 1 */
    float lr, beta1, beta2, eps;
    float grad_scale;            /* multiplies every gradient: 1/(S*N) */
    uint32_t seed;               /* 8-bit states: of the random rounding */
} zero_adamw_t;

/* Host only.  Errors: ZERO_EINVAL (bad field), ZERO_EUNSUPPORTED (state_bits
 * neither 8 nor 32, over 2^20 tensors or 2^40 values). */
zero_status_t zero_adamw_plan(const zero_adamw_tensor_t* tensors, int64_t n_tensors, int32_t dtype,
                              int32_t state_bits, zero_adamw_plan_t* out);
/* Write the list into `table` (plan->table_bytes of device memory, 16-byte
 * aligned, kept by the caller); synchronises `stream`.  The pointers are
 * taken as they are now: a list whose gradients move needs its table written
 * again.  Pointers need the alignment of their type; tensors whose buffers
 * all start on 16-byte boundaries take 16-byte accesses, others single-value
 * ones.  Tensors must not overlap.  Errors: ZERO_EINVAL, ZERO_ENOMEM (a NULL
 * buffer), ZERO_EALIGN, ZERO_ECUDA. */
zero_status_t zero_adamw_table_init(const zero_adamw_plan_t* plan, const zero_adamw_tensor_t* tensors, void* table,
                                    void* stream);
/* *flag = 1 if any gradient is inf or NaN, else 0 (device memory, 4-byte aligned). */
zero_status_t zero_adamw_check(const zero_adamw_plan_t* plan, const void* table, uint32_t* flag, void* stream);
/* One step; asynchronous.  skip: NULL, or a device flag -- nothing changes
 * when it is nonzero. */
zero_status_t zero_adamw_step(const zero_adamw_plan_t* plan, const void* table, const zero_adamw_t* hp,
                              const uint32_t* skip, void* stream);
/* The global norm of the list's gradients, norm = |grad_scale| sqrt(sum g^2),
 * and the factor that clips them, as in the sharded step: min(1, max_norm /
 * (norm + 1e-6)); where max_norm <= 0 or infinite nothing is clipped and the
 * factor is 1, whatever the norm.  norm: device memory, {norm, factor}.
 * flag (may be NULL): what zero_adamw_check gives, in the same pass.  An infinite
 * gradient makes norm +inf and the factor, where it clips, 0; a NaN makes both NaN
 * (with grad_scale 0 either does): pass flag to the step.  Squares are summed in
 * binary32 32 (binary32 gradients: 16) at a time, those sums in binary64; where
 * binary32 overflows or underflows, all in binary64.  Equal lists give equal bits.
 * workspace: zero_adamw_norm_workspace bytes of device memory, 16-byte aligned,
 * contents scratch.  Asynchronous.
 * Errors: ZERO_EINVAL (grad_scale not finite, max_norm NaN), ZERO_ENOMEM,
 * ZERO_EALIGN, ZERO_ECUDA. */
zero_status_t zero_adamw_norm(const zero_adamw_plan_t* plan, const void* table, float grad_scale, float max_norm,
                              float* norm, uint32_t* flag, void* workspace, void* stream);
/* Host only. */
zero_status_t zero_adamw_norm_workspace(const zero_adamw_plan_t* plan, int64_t* bytes);
/* zero_adamw_step with every gradient times norm[1] besides, as zero_adamw_norm
 * wrote it: g = grad * (norm[1] * grad_scale), the factors' product rounded once. */
zero_status_t zero_adamw_step_clipped(const zero_adamw_plan_t* plan, const void* table, const zero_adamw_t* hp,
                                      const float* norm, const uint32_t* skip, void* stream);
/* The gradients themselves times norm[1], each rounded to the list's dtype, in
 * place (norm[1] = 1 leaves them): for an optimizer that is not this one.  The
 * list's grad pointers must be writable then. */
zero_status_t zero_adamw_clip(const zero_adamw_plan_t* plan, const void* table, const float* norm, void* stream);
/* 8-bit states: the stored m and r = sqrt(v) as bfloat16 values, exact (m of
 * scale bytes below 4, under 2^-122, cut to bfloat16's subnormals), in
 * the plan's flat order (flat_elems each, 16-byte aligned; the gaps between
 * tensors are not written): for a checkpoint. */
zero_status_t zero_adamw_states(const zero_adamw_plan_t* plan, const void* table, void* m, void* root_v,
                                void* stream);

/* Profiling: for the step calls made afterwards on this thread, record
 * start_event (a cudaEvent_t) on the step's stream right after the workspace
 * clear, before the first kernel, and end_event after the step's last kernel,
 * before the overflow flag is read (zero_step_async: after its prepare
 * kernel, and after the last bucket or update kernel, before the restore and
 * commit; those two kernel edges then do not overlap).  The caller creates
 * the events and keeps
 * them valid; (NULL, NULL) turns recording off.  Bucket kernels launched
 * back to back inside one call overlap their edges, so the events give the
 * step's kernel span, not per-kernel durations. */
zero_status_t zero_set_profile_events(void* start_event, void* end_event);

/* Thread-local message of the last failed call ("" if none).  No
 * counterpart on the pages: error reporting of this C ABI.  The string is
 * owned by the library and stays valid until the thread's next failing
 * call. */
const char* zero_last_error(void);
/* ZERO_GB300_VERSION of the loaded library (no counterpart on the pages). */
int32_t zero_version(void);

#ifdef __cplusplus
}
#endif
#endif
