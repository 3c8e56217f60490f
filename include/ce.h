/*
 * ce.h -- C ABI of libgbce, the fused vocabulary cross-entropy pass for
 * NVIDIA GB300 (sm_103a).
 *
 * One call runs, on one GPU and on the caller's stream, the whole pass the
 * TENPU "Parallel Cross Entropy (Triton)" issue (Ascend/TransformerEngineNPU
 * #29) describes in its section 1 "Interface":
 *
 *     loss = parallel_cross_entropy(inp, target, label_smoothing, reduce_loss,
 *                                   dist_process_group, ignore_idx)
 *
 *   - inp: logits (B,SQ,V) or (SQ,B,V), FP32 / BF16 (FP16 also accepted);
 *   - target: (B,SQ) or (SQ,B), global vocabulary indices (int64 here);
 *   - softmax and loss accumulate in FP32, the loss is FP32, the gradient is
 *     written back in the input dtype (same section), in place over the
 *     logits (section 6 "Memory": in-place gradient staging);
 *   - loss of a row = logsumexp(x) - x[target] (CSDN "Ascend CANN ops-nn
 *     cross-entropy fusion: from three kernel launches to one", section
 *     "Fusion scheme: log_softmax + NLL"), with PyTorch-style label smoothing
 *     (1-a)*nll + a*mean_j(-log_softmax_j);
 *   - gradient of a row = (softmax - (1-a)*onehot(target) - a/V) * dloss
 *     (same article, section "Backward" and pitfall 3, with the smoothing mass
 *     spread over all V classes as torch F.cross_entropy does);
 *   - rows whose target equals ignore_idx (default -100) get loss 0 and a
 *     zero gradient and are left out of the mean (TENPU #29 section 1;
 *     mindspore/hyper-parallel #269 section 3.1);
 *   - reduce_loss: the mean over kept rows, produced on the device by a
 *     fixed-order reduction (TENPU #29 counts n_non_ignore on the host,
 *     section 7 "Known limitations"; here the count runs on the device).
 *
 * dist_process_group has no counterpart: the vocabulary-parallel combine of
 * (max, sum-exp, target logit) that hyper-parallel #269 section 3.1 runs as
 * MAX/SUM all-reduces plus a gather runs here between vocabulary chunks of
 * one GPU (thread-block clusters over distributed shared memory, or a second
 * kernel).
 *
 * Conventions for every entry point:
 *   - every pointer argument is a DEVICE pointer unless it says "host";
 *   - the caller owns all memory; the library allocates nothing, keeps no
 *     pointer after the call returns and never synchronises the stream
 *     (ce_get_error excepted);
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream); all work is enqueued on it in order;
 *   - dims: the logits have shape (dim0, dim1, V); (B,SQ,V) and (SQ,B,V)
 *     differ only in which of dim0/dim1 is the batch; row (i, j) is the
 *     flattened row r = i*dim1 + j; element (i, j, v) sits at
 *     logits + (i*strides[0] + j*strides[1] + v*strides[2]) elements;
 *     strides[2] must be 1 (non-unit vocabulary stride: make the tensor
 *     contiguous first, as TENPU #29 "Problems and solutions" does);
 *   - targets: int64, target of row (i, j) at targets[i*target_strides[0] +
 *     j*target_strides[1]];
 *   - logits (and a separate gradient) must sit on a multiple of their element
 *     size (CE_ERR_INVALID_ARG otherwise); rows need no further alignment:
 *     rows on the 16-byte grid take the TMA kernels, others 16-byte loads
 *     between a scalar head and tail (CE_PATH_VECROW, the two-stage kernels,
 *     ce_bwd, ce_vp_partials);
 *   - logits may be masked by any value below the others, -inf included where
 *     there is no smoothing; a row whose every logit is below -2^30 has no
 *     finite loss from ce_fwd_bwd and its kin;
 *   - errors found on the host are returned before anything is launched;
 *     a target outside [0, V) that is not ignore_idx is found on the device:
 *     that row gets loss NaN and a zero gradient, and the device error word
 *     in the workspace gets CE_DEVERR_TARGET_RANGE (read it with
 *     ce_get_error).  Kernels never trap.
 */
#ifndef GBCE_CE_H
#define GBCE_CE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { CE_F32 = 0, CE_BF16 = 1, CE_F16 = 2 } ce_dtype;

/* (B,SQ,V): dim0 = B, dim1 = SQ.  (SQ,B,V): dim0 = SQ, dim1 = B. */
typedef enum { CE_LAYOUT_BSV = 0, CE_LAYOUT_SBV = 1 } ce_layout;

typedef enum {
    CE_OK = 0,
    CE_ERR_INVALID_ARG = 1,        /* null pointer, bad size, smoothing outside [0,1],
                                      logits off their element size, ... */
    CE_ERR_UNSUPPORTED_DTYPE = 2,
    CE_ERR_BAD_STRIDE = 3,         /* strides[2] != 1, a negative stride, or (ce_fwd_bwd)
                                      rows that share memory */
    CE_ERR_WORKSPACE_TOO_SMALL = 4,
    CE_ERR_LAUNCH = 5,             /* a CUDA launch or attribute call failed */
    CE_ERR_TARGET_RANGE = 6,       /* reported by ce_get_error only */
    CE_ERR_DEVICE_TIMEOUT = 7,     /* reported by ce_get_error only */
    CE_ERR_UNSUPPORTED_PATH = 8    /* a forced path cannot run this shape */
} ce_status;

/* Bits of the device error word (ce_get_error). */
#define CE_DEVERR_TARGET_RANGE 0x1u
#define CE_DEVERR_TIMEOUT 0x2u     /* a bounded wait inside a kernel gave up */

typedef enum {
    CE_PATH_AUTO = 0,
    CE_PATH_ROW = 1,       /* one CTA holds a whole row in shared memory and registers */
    CE_PATH_CLUSTER = 2,   /* a thread-block cluster splits each row; combine over DSMEM */
    CE_PATH_TWO_STAGE = 3, /* per-chunk statistics kernel, then combine + gradient kernel */
    CE_PATH_STREAM = 4,    /* one CTA streams whole rows twice through a TMA ring (rows
                              claimed from a counter in the workspace); the second read
                              of a row is served by L2, or for rows of at least twice
                              the ring by the ring's last tiles still in shared memory.
                              Default shape: rows up to 128 KB 16 KB tiles, 6 deep, two
                              CTAs per SM; wider rows 32 KB tiles, 6 deep, one CTA.
                              Rows off the 16-byte grid (the default for such rows over
                              32 KB): the ring takes each row's aligned body, and the at
                              most 2 (16/sizeof(T) - 1) elements before and after it are
                              read and written one per thread (256 consuming threads).
                              A vocabulary split (num_vocab_chunks = K, the default path
                              for a split of aligned rows into at most 32 non-empty
                              chunks; 16 KB tiles, two CTAs per SM): each chunk streams
                              as its own run of tiles with the warps' running max shared,
                              the
                              chunks' (max, sum-exp, sum, target logit) partials are
                              combined in chunk order (256 consuming threads) */
    CE_PATH_WARP = 5,      /* one warp per row, the row held in one shared-memory tile
                              (rows up to 32 KB) */
    CE_PATH_VECROW = 6     /* rows off the 16-byte grid (any alignment): a persistent
                              grid, two passes of plain 16-byte loads per row between a
                              scalar head and tail, the second served by L2; a warp per
                              row up to 32 KB, else a CTA per row (512 threads two per
                              SM, rows over 320 KB 1024 threads one per SM); no
                              vocabulary split, no class weights */
} ce_path;

typedef struct {
    int force_path;         /* ce_path; CE_PATH_AUTO lets the planner choose */
    int num_vocab_chunks;   /* 0: planner chooses; K > 0: cut V into K contiguous
                               chunks of ceil(V/K) (rounded up to 16 bytes on the
                               row, cluster and stream paths, so fewer chunks may be
                               non-empty) whose partials are combined on the device:
                               the stream path for aligned rows cut into up to 32
                               non-empty chunks, else the two-stage path (the
                               cluster path when forced, up to 16 chunks) */
    void* event_begin;      /* cudaEvent_t or NULL: recorded on `stream` right
                               before the main kernel of the pass */
    void* event_end;        /* cudaEvent_t or NULL: recorded right after it */
    int tune_threads;       /* 0 = default; otherwise CTA size (256 or 512; on the stream
                               path the number of consuming threads); CE_PATH_VECROW
                               also takes 1024 (one CTA per SM) and 32 (a row per warp),
                               which the stream, row and cluster paths refuse */
    int tune_stages;        /* 0 = default; otherwise TMA pipeline depth (2..4 rows on the
                               row/cluster paths, 2..12 tiles on the stream path, 6 or 12
                               tiles on the warp path: 12 = two tiles per consumer warp,
                               the default for 16 KB tiles from 8192 rows on) */
    int tune_ctas_per_sm;   /* 0 = as many as fit; otherwise a cap */
    int tune_l2_keep;       /* stream path: 0 = default (1), 1 = the first read asks L2 to
                               keep the row for the second (evict-last), 2 = evict-first */
    int tune_tile_kb;       /* stream and warp paths: 0 = default, else the ring tile size
                               (16 or 32 KB) */
    const float* class_weights; /* NULL, or device float32[V]: per-class weights as in
                               torch F.cross_entropy(weight=...): the smoothed target's
                               class j term is weighted by w_j and the mean divides by
                               the summed weight of the kept rows' targets.  Runs on the
                               stream path when the rows and this vector are 16-byte
                               aligned and no vocabulary split is asked for (256
                               consuming threads), else on the two-stage path;
                               CE_PATH_ROW, CE_PATH_CLUSTER and CE_PATH_WARP are refused
                               with CE_ERR_UNSUPPORTED_PATH (ce_fwd_bwd, ce_fwd_only;
                               not ce_bwd) */
    int reserved[2];        /* must be zero */
} ce_options;

/* Bytes of device workspace a call with these sizes needs (either entry
 * point, any path, reduce_loss or not).  Host only; returns 0 for invalid
 * sizes.  opts may be NULL. */
size_t ce_workspace_bytes(int64_t dim0, int64_t dim1, int64_t V, ce_dtype dtype,
                          const ce_options* opts);

/* Forward and backward in one pass.
 *   logits          (dim0, dim1, V) in `dtype`; read, then overwritten with the
 *                   gradient (grad_inplace must equal logits).
 *   label_smoothing a in [0, 1].
 *   ignore_idx      target value that marks a row as ignored (usually -100).
 *   reduce_loss     0: per-row losses; 1: mean over rows whose target is not
 *                   ignore_idx.
 *   dloss           float32 upstream gradient: one value (reduce_loss = 1; the
 *                   gradient of the mean, each kept row is scaled by dloss/n)
 *                   or one value per flattened row (reduce_loss = 0); NULL
 *                   means 1.
 *   loss_out        float32: one value (reduce_loss = 1; NaN when every row is
 *                   ignored) or dim0*dim1 values in flattened row order.
 *   n_non_ignore_out  int64 count of rows whose target != ignore_idx, or NULL.
 *   workspace       at least ce_workspace_bytes(...) bytes, 256-byte aligned;
 *                   its contents need no initialisation and must not be
 *                   shared by calls that may run concurrently.
 *   opts            NULL for defaults.
 * Returns CE_OK once every kernel is enqueued. */
ce_status ce_fwd_bwd(void* logits, ce_dtype dtype, ce_layout layout, int64_t dim0, int64_t dim1,
                     int64_t V, const int64_t strides[3], const int64_t* targets,
                     const int64_t target_strides[2], float label_smoothing, int64_t ignore_idx,
                     int reduce_loss, const float* dloss, float* loss_out, void* grad_inplace,
                     int64_t* n_non_ignore_out, void* workspace, size_t workspace_bytes,
                     const ce_options* opts, void* stream);

/* Forward only: the logits are read, never written.  Same arguments as
 * ce_fwd_bwd minus dloss and the gradient, plus
 *   lse_out   float32 logsumexp of every row (NaN for ignored or out-of-range
 *             rows), or NULL. */
ce_status ce_fwd_only(const void* logits, ce_dtype dtype, ce_layout layout, int64_t dim0,
                      int64_t dim1, int64_t V, const int64_t strides[3], const int64_t* targets,
                      const int64_t target_strides[2], float label_smoothing, int64_t ignore_idx,
                      int reduce_loss, float* loss_out, float* lse_out, int64_t* n_non_ignore_out,
                      void* workspace, size_t workspace_bytes, const ce_options* opts,
                      void* stream);

/* Backward only, from the logsumexp a forward-only pass saved: for callers
 * that learn the upstream gradient after the forward (autograd).  Writes
 *   grad_j = g * (exp(x_j - lse) - a/V) - g * (1-a) * [j == target]
 * for every kept row (CSDN "Ascend CANN ops-nn cross-entropy fusion",
 * section "Backward", pitfall 3; smoothing over all V classes) and zeros for
 * ignored or out-of-range rows; g = dloss[0] / n_non_ignore (reduce_loss) or
 * dloss[row] (otherwise; NULL means 1).
 *   logits, targets, sizes, strides, label_smoothing, ignore_idx: as given to
 *                  ce_fwd_only; the logits must be unchanged since then.
 *   lse            float32 per flattened row, from ce_fwd_only's lse_out.
 *   n_non_ignore   int64 count from ce_fwd_only's n_non_ignore_out; required
 *                  when reduce_loss.
 *   grad           gradient in the logits dtype with its own strides
 *                  (grad_strides[2] == 1): either the logits themselves (same
 *                  strides; the TENPU in-place staging) or memory that does
 *                  not overlap them.
 * One read of the logits and one write of the gradient per element; no
 * workspace.  Returns CE_OK once the kernel is enqueued on `stream`. */
ce_status ce_bwd(const void* logits, ce_dtype dtype, ce_layout layout, int64_t dim0, int64_t dim1,
                 int64_t V, const int64_t strides[3], const int64_t* targets,
                 const int64_t target_strides[2], const float* lse, float label_smoothing,
                 int64_t ignore_idx, int reduce_loss, const float* dloss,
                 const int64_t* n_non_ignore, void* grad, const int64_t grad_strides[3],
                 void* stream);

/* Vocabulary-parallel cross-entropy (mindspore/hyper-parallel #269, section
 * 3.1: each tensor-parallel rank holds a ceil(V/tp) slice of the vocabulary;
 * per-row (max, sum-exp) statistics of the slice, a MAX all-reduce and a SUM
 * all-reduce of the rescaled sums and a gather of the target logit -- TENPU
 * #29 section 6's m_d_Xy gather -- then a backward without collectives).  The
 * three calls below are the three steps; a caller with one GPU runs them over
 * vocabulary shards held as separate tensors, a caller with several ranks
 * would all-gather the partials between steps 1 and 2.
 *
 * Step 1: statistics of one shard.
 *   shard_logits   (dim0, dim1, V_shard) columns [vocab_offset, vocab_offset +
 *                  V_shard) of the vocabulary; strides as for ce_fwd_bwd.
 *   targets        global vocabulary indices, as for ce_fwd_bwd.
 *   partials       float32 [dim0*dim1][4], 16-byte aligned: per flattened row
 *                  {max, sum of exp(x - max), sum of x, target logit if the
 *                  target lies in this shard else 0}; ignored rows get
 *                  {-inf, 0, 0, 0}. */
ce_status ce_vp_partials(const void* shard_logits, ce_dtype dtype, int64_t dim0, int64_t dim1,
                         int64_t V_shard, const int64_t strides[3], const int64_t* targets,
                         const int64_t target_strides[2], int64_t vocab_offset, int64_t ignore_idx,
                         float* partials, void* stream);

/* Step 2: combine the partials of all shards, in shard order.
 *   partials       num_shards consecutive blocks of [dim0*dim1][4] (shard k's
 *                  block k), 1 <= num_shards <= 64.
 *   shard_offsets  HOST array of num_shards + 1 increasing column offsets:
 *                  shard k covers [shard_offsets[k], shard_offsets[k+1]);
 *                  shard_offsets[0] = 0, shard_offsets[num_shards] = V.
 *   loss_out, reduce_loss, n_non_ignore_out, workspace: as for ce_fwd_bwd
 *                  (workspace of ce_workspace_bytes(dim0, dim1, V, dtype, NULL)).
 *   lse_out        float32 logsumexp per flattened row (required: step 3 needs
 *                  it); NaN for ignored or out-of-range rows.
 * Out-of-range targets set CE_DEVERR_TARGET_RANGE in the workspace. */
ce_status ce_vp_combine(const float* partials, int num_shards, const int64_t* shard_offsets,
                        int64_t dim0, int64_t dim1, const int64_t* targets,
                        const int64_t target_strides[2], float label_smoothing, int64_t ignore_idx,
                        int reduce_loss, float* loss_out, float* lse_out,
                        int64_t* n_non_ignore_out, void* workspace, size_t workspace_bytes,
                        void* stream);

/* Step 3: the gradient of one shard from the combined lse -- ce_bwd for the
 * columns [vocab_offset, vocab_offset + V_shard) of a V_total vocabulary (the
 * smoothing share is a / V_total; the one-hot term lands in the shard that
 * holds the target).  Other arguments as for ce_bwd. */
ce_status ce_vp_bwd(const void* shard_logits, ce_dtype dtype, int64_t dim0, int64_t dim1,
                    int64_t V_shard, const int64_t strides[3], const int64_t* targets,
                    const int64_t target_strides[2], int64_t vocab_offset, int64_t V_total,
                    const float* lse, float label_smoothing, int64_t ignore_idx, int reduce_loss,
                    const float* dloss, const int64_t* n_non_ignore, void* grad,
                    const int64_t grad_strides[3], void* stream);

/* lm_head + cross-entropy, chunked over token rows (the sequence-chunked
 * lm_head + loss of the TorchTitan ChunkedLossWrapper that hyper-parallel
 * #269 describes: the full (N, V) logits never exist).  For each chunk of
 * chunk_rows rows: logits = hidden . weight^T into the workspace -- for
 * bf16 / fp16 with H a multiple of 8 and 16-byte aligned hidden and weight,
 * this library's tcgen05 GEMM, whose epilogue also folds every (row,
 * 256-column tile) into softmax statistics that a per-row combine turns into
 * lse and the loss, then the backward from lse writes the gradient in place;
 * otherwise a cuBLAS GEMM and this library's fused pass -- scaled with the
 * kept-row count of the whole batch; then grad_hidden = dlogits . weight and
 * grad_weight += dlogits^T . hidden (cuBLAS GEMMs, fp32 accumulation).
 * GBCE_LINEAR_GEMM=library in the environment (read once, at the first
 * call) takes the cuBLAS branch for every dtype and shape, for comparison.
 *   hidden       (N, H) row-major, dtype; weight (V, H) row-major, dtype.
 *   targets      int64 [N], contiguous.
 *   loss_out     one value (reduce_loss) or N values.
 *   grad_hidden  (N, H) row-major, dtype, written; or NULL.
 *   grad_weight  (V, H) row-major float32, ACCUMULATED into (zero it first for
 *                a fresh gradient); or NULL.
 *   workspace    ce_linear_workspace_bytes(N, H, V, dtype, chunk_rows) bytes,
 *                256-byte aligned; it holds one chunk of logits (rows padded
 *                to a multiple of 8 elements), their statistics and cuBLAS's
 *                workspace.  cuBLAS creates one handle per host thread and
 *                device on first use (its own small allocation).
 * Returns CE_OK once every kernel and GEMM is enqueued on `stream`. */
size_t ce_linear_workspace_bytes(int64_t N, int64_t H, int64_t V, ce_dtype dtype,
                                 int64_t chunk_rows);
ce_status ce_linear_fwd_bwd(const void* hidden, const void* weight, ce_dtype dtype, int64_t N,
                            int64_t H, int64_t V, const int64_t* targets, float label_smoothing,
                            int64_t ignore_idx, int reduce_loss, const float* dloss,
                            float* loss_out, void* grad_hidden, float* grad_weight,
                            int64_t* n_non_ignore_out, int64_t chunk_rows, void* workspace,
                            size_t workspace_bytes, void* stream);

/* ce_fwd_bwd without a workspace argument: the pass keeps its scratch in a
 * fixed 2 MiB array of device memory that the library itself reserves on
 * every GPU where it is loaded (held until the process exits).  The pages have
 * no counterpart of this entry point; it exists for callers that must not
 * allocate device memory for a call: runtimes that plan every byte of device
 * memory before they start and give custom operators no workspace, and
 * latency-critical loops where cudaMalloc (which may synchronise the device or
 * fail on a fragmented heap) is not acceptable.  The caller still passes the
 * logits, targets and outputs, as for ce_fwd_bwd; this call allocates nothing.
 *
 * Limit: the scratch must hold 256 bytes + 4*dim0*dim1 bytes rounded up to
 * 256 (per-row losses), plus 16*dim0*dim1*K bytes rounded up to 256 when the
 * planner takes the two-stage path with K chunks.  Larger problems are
 * rejected with CE_ERR_WORKSPACE_TOO_SMALL before anything is launched
 * (about 520,000 rows on the row, cluster, stream, warp and plain-load
 * paths).
 *
 * Set-up: the first call on a device looks up the scratch's device address
 * with that device current (the caller's current device); make that first
 * call before any stream capture.  No part of the scratch needs clearing:
 * every pass writes what it later reads.  All calls on a device share the one
 * array and it keeps the last call's contents, so calls that may overlap on
 * the GPU (different streams, or threads enqueuing at once) race on it:
 * serialise them.  The error word lives in that internal scratch, so
 * ce_get_error cannot read it; ce_noalloc_get_error (below) reads it
 * instead.  Out-of-range targets also show as NaN row losses; a bounded wait
 * inside a kernel that gave up (CE_DEVERR_TIMEOUT, see ce_wait_timeout_probe)
 * shows only there: the call has already returned CE_OK, and some loss and
 * gradient rows may be left unwritten. */
ce_status ce_fwd_bwd_noalloc(void* logits, ce_dtype dtype, ce_layout layout, int64_t dim0,
                             int64_t dim1, int64_t V, const int64_t strides[3],
                             const int64_t* targets, const int64_t target_strides[2],
                             float label_smoothing, int64_t ignore_idx, int reduce_loss,
                             const float* dloss, float* loss_out, void* grad_inplace,
                             int64_t* n_non_ignore_out, const ce_options* opts, void* stream);

/* ce_get_error for ce_fwd_bwd_noalloc: waits for `stream`, then copies the
 * error word of the last no-alloc pass on the current device (the one its
 * fixed scratch array holds) into *host_err (host pointer) and decodes it as
 * ce_get_error does.  Serialise it with the no-alloc passes like they are
 * serialised with each other: a pass enqueued on another stream meanwhile
 * rewrites the word.  Returns CE_ERR_INVALID_ARG if host_err is NULL,
 * CE_ERR_LAUNCH if the scratch's address cannot be looked up or the copy
 * fails. */
ce_status ce_noalloc_get_error(void* stream, uint32_t* host_err);

/* ---------------------------------------------------------------------------
 * The operators around the pass at the two ends of the vocabulary: the
 * embedding rows of the (tied) vocabulary matrix, the norm in front of the
 * lm_head, and what is applied to the logits before a token is taken from
 * them.  The conventions above hold; rows of activations are N rows of H
 * elements, unit stride within a row and one stride (in elements) between
 * rows.  Any base that is a multiple of the element size and any row stride
 * work; bases and strides on the 16-byte grid move 16 bytes per load.  All
 * sums are float32 and taken in an order fixed by the sizes, so results are
 * the same on every run.
 */

/* out_i = scale * weight[token_i], computed in float32 and rounded once.
 *   tokens       int64 (dim0, dim1), token (i, j) at tokens[i*token_strides[0] +
 *                j*token_strides[1]]; output row i*dim1 + j.  A token equal to
 *                ignore_idx gives a row of zeros; any other token outside
 *                [0, V) a row of NaN.
 *   weight       (V, H) rows weight_stride elements apart, in `dtype`.
 *   out          rows out_stride elements apart, in `dtype`; no overlap with
 *                the weight.
 *   workspace    NULL, or >= 256 bytes, 16-byte aligned: its error word is
 *                cleared, then gets CE_DEVERR_TARGET_RANGE for an out-of-range
 *                token (ce_get_error). */
ce_status ce_embed_fwd(const int64_t* tokens, int64_t dim0, int64_t dim1,
                       const int64_t token_strides[2], const void* weight, ce_dtype dtype,
                       int64_t V, int64_t H, int64_t weight_stride, float scale,
                       int64_t ignore_idx, void* out, int64_t out_stride, void* workspace,
                       size_t workspace_bytes, void* stream);

/* Gradient of ce_embed_fwd:  dW_v = scale * (sum of grad_out_i over tokens
 * i = v, in float32, in an order fixed by the tokens and the sizes).
 * Ignored and out-of-range tokens give nothing; the latter set
 * CE_DEVERR_TARGET_RANGE in the workspace.
 *   grad_out     N = dim0*dim1 rows in `dtype`, grad_out_stride apart (0 for
 *                one row that all tokens share).
 *   grad_weight  (V, H) rows grad_weight_stride apart, in grad_dtype: CE_F32, or
 *                `dtype`.
 *   accumulate   0: every element is written (zeros for tokens that do not
 *                occur).  1 (CE_F32 only): added to what is there, rows of
 *                tokens that do not occur are not touched -- the tied matrix's
 *                float32 gradient that ce_linear_fwd_bwd has added to.  Values
 *                below 2^-126, there or in a sum, are taken as zeros.
 *   workspace    ce_embed_bwd_workspace_bytes(N, H, V) bytes, 16-byte aligned,
 *                no initialisation; not shared by calls that may overlap. */
size_t ce_embed_bwd_workspace_bytes(int64_t N, int64_t H, int64_t V);
ce_status ce_embed_bwd(const void* grad_out, ce_dtype dtype, int64_t grad_out_stride,
                       const int64_t* tokens, int64_t dim0, int64_t dim1,
                       const int64_t token_strides[2], int64_t V, int64_t H, float scale,
                       int64_t ignore_idx, void* grad_weight, ce_dtype grad_dtype,
                       int64_t grad_weight_stride, int accumulate, void* workspace,
                       size_t workspace_bytes, void* stream);

/* 8-bit outputs of ce_rmsnorm_fwd. */
typedef enum { CE_QUANT_NONE = 0, CE_QUANT_E4M3 = 1, CE_QUANT_E5M2 = 2 } ce_quant;

/* The residual's addition and the root-mean-square norm:
 *   h = x + residual,  y_j = h_j * weight_j / sqrt(mean_j h_j^2 + eps)
 * in float32; h and y are each rounded once, y from the unrounded h.
 *   residual     NULL (h = x; residual_out is then optional) or N rows.
 *   weight       H contiguous elements in weight_dtype: `dtype` or CE_F32.
 *   out          y: N rows in `dtype`, or with quant N rows of H bytes
 *                (out_stride in bytes): y_j / scale rounded to nearest even and
 *                saturated, scale = max(max |y_j| / top, 2^-126) over each run of
 *                group_size columns (32, 64 or 128; 0: the row), top = 448
 *                (e4m3) or 57344 (e5m2).  The quotient takes one rounding to
 *                float32, from h_j weight_j and its group's maximum, before that to
 *                8 bits; the scale's last bits go with the order of the row's sum
 *                (its width and alignment).  A group that holds an infinity or a NaN
 *                has no finite values to give.
 *   scales       with quant: float32 (N, ceil(H / group)) contiguous.
 *   residual_out h: N rows in `dtype`.  It may replace x or residual, and out (without
 *                quant) x or residual, with the same strides; other overlaps
 *                are not allowed.
 * H up to 2^20. */
ce_status ce_rmsnorm_fwd(const void* x, const void* residual, const void* weight, ce_dtype dtype,
                         ce_dtype weight_dtype, int64_t N, int64_t H, int64_t x_stride,
                         int64_t residual_stride, float eps, void* out, int64_t out_stride,
                         ce_quant quant, int group_size, float* scales, void* residual_out,
                         int64_t residual_out_stride, void* stream);

/* Gradients of ce_rmsnorm_fwd (without quant) from the stored h: with
 * n_j = h_j / sqrt(mean h^2 + eps) and c = mean_j(g_j w_j n_j),
 *   grad_x_j = (g_j w_j - n_j c) / sqrt(mean h^2 + eps) + grad_h_j
 *   grad_weight_j = sum over rows of g_j n_j          (float32, written)
 *   grad_h       the gradient that reaches h from the residual stream, or NULL.
 *   grad_x       the gradient of x and of the residual alike, rounded once;
 *                may replace grad_out, h or grad_h with the same strides.
 *   grad_weight  NULL to skip (no workspace needed then).
 *   workspace    ce_rmsnorm_bwd_workspace_bytes(N, H) bytes, 16-byte aligned, no
 *                initialisation; not shared by calls that may overlap.  Its error
 *                word gets CE_DEVERR_TIMEOUT if a bounded wait inside the kernel
 *                gave up (ce_get_error). */
size_t ce_rmsnorm_bwd_workspace_bytes(int64_t N, int64_t H);
ce_status ce_rmsnorm_bwd(const void* grad_out, const void* h, const void* weight,
                         const void* grad_h, ce_dtype dtype, ce_dtype weight_dtype, int64_t N,
                         int64_t H, int64_t grad_out_stride, int64_t h_stride,
                         int64_t grad_h_stride, float eps, void* grad_x, int64_t grad_x_stride,
                         float* grad_weight, void* workspace, size_t workspace_bytes,
                         void* stream);

/* What is applied to the logits of a row before a token is taken from them.
 * Every pointer may be NULL (that step is left out); rows are flattened, r =
 * i*dim1 + j. */
typedef struct {
    const int64_t* history;         /* token k of row r at history[r*history_stride + k];
                                       tokens outside [0, V) count nowhere */
    int64_t history_stride;
    int64_t history_max;            /* tokens a row has room for, below 2^30 */
    const int64_t* history_lengths; /* [N] tokens in use (clamped to [0, history_max]);
                                       NULL: all */
    const int64_t* prompt_lengths;  /* [N] the first ones are the prompt: they count for
                                       the repetition penalty only; NULL: 0 */
    const float* repetition_penalty; /* [N] > 0 */
    const float* frequency_penalty; /* [N] */
    const float* presence_penalty;  /* [N] */
    const int64_t* bias_tokens;     /* bias k of row r for token bias_tokens[r*stride + k]
                                       (outside [0, V): none); equal tokens add up in order */
    const float* bias_values;
    int64_t bias_tokens_stride, bias_values_stride;
    int64_t bias_max;               /* biases per row */
    const int32_t* mask;            /* bit v % 32 of word v / 32: token v is allowed */
    int64_t mask_stride;            /* words between rows, 0: one mask for all */
    const float* temperature;       /* [N] > 0 */
    float mask_value;               /* output of a token that is not allowed */
    int reserved[2];                /* must be zero */
} ce_logits_params;

/* Per row, in float32, rounded once, with s_j: token j is in the history, c_j:
 * its count after the prompt, b_j: its summed biases,
 *   z_j = s_j ? (x_j > 0 ? x_j / repetition : x_j * repetition) : x_j
 *   y_j = (z_j - frequency * c_j - presence * [c_j > 0] + b_j) / temperature
 *   out_j = allowed_j ? y_j : mask_value
 * In CE_F32 a quotient is rounded once; in the 16-bit types it is a product with
 * the rounded reciprocal (at most 2^-23 of the value more, before the rounding to
 * the type).  A token that is not allowed gives mask_value whatever its logit (NaN
 * included); a row that allows none is mask_value throughout.  ce_fwd_bwd with
 * smoothing needs a finite mask_value (say -3e4: its smoothing term sums the
 * logits).  out may be the logits themselves (same strides).
 *   workspace    at least ce_logits_workspace_bytes(dim0*dim1, V, dtype, history_max,
 *                bias_max) bytes, 16-byte aligned, no initialisation; not shared
 *                by calls that may overlap.  NULL where that is 0 (no
 *                lists, or few columns in all). */
size_t ce_logits_workspace_bytes(int64_t N, int64_t V, ce_dtype dtype, int64_t history_max,
                                 int64_t bias_max);
ce_status ce_logits_process(const void* logits, ce_dtype dtype, int64_t dim0, int64_t dim1,
                            int64_t V, const int64_t strides[3], const ce_logits_params* params,
                            void* out, const int64_t out_strides[3], void* workspace,
                            size_t workspace_bytes, void* stream);

/* Gradient of ce_logits_process with respect to the logits:
 *   grad_j = allowed_j ? grad_out_j / temperature * (s_j ? (x_j > 0 ? 1 / repetition
 *                        : repetition) : 1) : 0
 * with quotients as above.  The logits are read where the history holds their
 * token; the biases, the counts and mask_value play no part.  grad may be grad_out
 * (same strides), not the logits.  workspace as for ce_logits_process. */
ce_status ce_logits_process_bwd(const void* grad_out, const int64_t grad_out_strides[3],
                                const void* logits, ce_dtype dtype, int64_t dim0, int64_t dim1,
                                int64_t V, const int64_t strides[3],
                                const ce_logits_params* params, void* grad,
                                const int64_t grad_strides[3], void* workspace,
                                size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * A row's log-probabilities: given tokens', the entropy, the likeliest tokens';
 * and the divergence from a teacher's.  The conventions above hold; rows are rows
 * of logits as for ce_fwd_bwd, flattened r = i*dim1 + j (dim0*dim1 below 2^31).
 * Lists of tokens are int64 (dim0, dim1, n), element (i, j, k) at
 * tokens[i*strides[0] + j*strides[1] + k*strides[2]], strides not negative.
 * Arithmetic is float32 on differences from the row's maximum; sums are taken in
 * an order fixed by the sizes.
 */

/* With lp_j = x_j - logsumexp(x):
 *   logprobs       float32 [N][given]: lp of the given tokens (at most 1024 a row).
 *                  A token equal to ignore_idx gives 0; any other outside [0, V) NaN
 *                  and CE_DEVERR_TARGET_RANGE in the workspace's error word.
 *   entropy        float32 [N] or NULL: -sum_j exp(lp_j) lp_j.
 *   top_k          0 to min(256, V): the k largest logits, in falling order, equal
 *                  ones the lower column first (-0 is 0):
 *   top_tokens     int64 [N][top_k], top_logprobs float32 [N][top_k].
 *   stats          float32 [N][4], 16-byte aligned, or NULL: {max, log sum exp(x - max),
 *                  entropy, 0} for ce_logprobs_bwd.
 *   workspace      ce_logprobs_workspace_bytes(dim0*dim1, V, dtype, top_k) bytes, 16-byte
 *                  aligned, no initialisation; not shared by calls that may overlap.  0 bytes,
 *                  and CE_ERR_INVALID_ARG from the call: sizes out of range, or top_k with
 *                  rows of more than 256 MiB (V times the type's size).
 * A row whose given tokens (one at least) are all ignore_idx is not read: zeros, and
 * ignore_idx for its top tokens.  A row of -inf throughout (a mask that allows
 * nothing) has log-probabilities of -inf, entropy 0 and top tokens 0, 1, 2, ...  A NaN
 * or +inf in a row makes its log-probabilities and its entropy NaN; a NaN is never
 * among the top tokens (-1 where no others are left). */
size_t ce_logprobs_workspace_bytes(int64_t N, int64_t V, ce_dtype dtype, int top_k);
ce_status ce_logprobs_fwd(const void* logits, ce_dtype dtype, int64_t dim0, int64_t dim1, int64_t V,
                          const int64_t strides[3], const int64_t* tokens,
                          const int64_t token_strides[3], int64_t given, int64_t ignore_idx,
                          float* logprobs, float* entropy, int top_k, int64_t* top_tokens,
                          float* top_logprobs, float* stats, void* workspace,
                          size_t workspace_bytes, void* stream);

/* Gradient of ce_logprobs_fwd's log-probabilities and entropy H with respect to the
 * logits, from the stats it left (p_j = exp(lp_j)):
 *   grad_j = sum_k g_k [t_k = j] - p_j sum_k g_k - h p_j (lp_j + H)
 *   grad_logprobs  float32 [N][given] g, or NULL;  grad_entropy  float32 [N] h, or NULL.
 *   grad           in the logits' dtype with its own strides: the logits themselves
 *                  (same strides) or memory that does not overlap them.
 * Zeros for a row that was not read and for one of -inf throughout; ignored and
 * out-of-range tokens give nothing; a token given twice gets both. */
ce_status ce_logprobs_bwd(const void* logits, ce_dtype dtype, int64_t dim0, int64_t dim1, int64_t V,
                          const int64_t strides[3], const int64_t* tokens,
                          const int64_t token_strides[3], int64_t given, int64_t ignore_idx,
                          const float* stats, const float* grad_logprobs,
                          const float* grad_entropy, void* grad, const int64_t grad_strides[3],
                          void* stream);

/* Distillation from a teacher's top logits, forward and backward in one pass.  With
 * s = 1/temperature, p = softmax(s x) over the vocabulary and q_k the teacher's
 * probability of its token t_k (k < K, 1 <= K <= 1024),
 *   q_k = exp(s z_k) / sum_k exp(s z_k)  (normalize), or exp(s z_k) as it is
 *   loss = temperature^2 sum_k q_k (log q_k - log p_{t_k})
 *   grad_j = dloss temperature (p_j sum_k q_k - sum_k q_k [t_k = j])
 *   teacher_tokens  int64 (dim0, dim1, K).  A row whose first token is ignore_idx is
 *                   ignored: loss 0, zero gradient, not counted.  A later ignore_idx
 *                   leaves that entry out, whatever its logit.  Any other token
 *                   outside [0, V): loss NaN, zero gradient, CE_DEVERR_TARGET_RANGE.
 *   teacher_logits  (dim0, dim1, K) z in teacher_dtype with strides not negative; -inf
 *                   gives q_k = 0.  Without normalize: log-probabilities, those of
 *                   ce_logprobs_fwd, say (temperature 1); the tokens that are not
 *                   listed then take no part.
 *   temperature     1e-4 to 1e4.
 *   dloss, reduce_loss, loss_out, n_non_ignore_out: as for ce_fwd_bwd.
 *   grad            as for ce_logprobs_bwd.
 *   workspace       ce_distill_workspace_bytes(dim0*dim1, V, dtype) bytes, 16-byte
 *                   aligned, no initialisation; not shared by calls that may overlap.
 * Tokens listed twice are two entries.  A row of logits of -inf throughout has p = 0:
 * loss +inf where some q_k > 0, zero gradient. */
size_t ce_distill_workspace_bytes(int64_t N, int64_t V, ce_dtype dtype);
ce_status ce_distill_fwd_bwd(const void* logits, ce_dtype dtype, int64_t dim0, int64_t dim1,
                             int64_t V, const int64_t strides[3], const int64_t* teacher_tokens,
                             const int64_t teacher_token_strides[3], const void* teacher_logits,
                             ce_dtype teacher_dtype, const int64_t teacher_strides[3], int64_t K,
                             float temperature, int normalize, int64_t ignore_idx, int reduce_loss,
                             const float* dloss, float* loss_out, void* grad,
                             const int64_t grad_strides[3], int64_t* n_non_ignore_out,
                             void* workspace, size_t workspace_bytes, void* stream);

/* Forward only.  stats: float32 [N][4], 16-byte aligned, or NULL: {max of the logits, log sum
 * exp(s (x - max)), max of the teacher's logits, log sum exp(s (z - max))} for
 * ce_distill_bwd; an ignored row's are {-inf, 0, -inf, 0}. */
ce_status ce_distill_fwd(const void* logits, ce_dtype dtype, int64_t dim0, int64_t dim1, int64_t V,
                         const int64_t strides[3], const int64_t* teacher_tokens,
                         const int64_t teacher_token_strides[3], const void* teacher_logits,
                         ce_dtype teacher_dtype, const int64_t teacher_strides[3], int64_t K,
                         float temperature, int normalize, int64_t ignore_idx, int reduce_loss,
                         float* loss_out, float* stats, int64_t* n_non_ignore_out, void* workspace,
                         size_t workspace_bytes, void* stream);

/* Backward only, from ce_distill_fwd's stats (and its n_non_ignore_out with
 * reduce_loss); no workspace. */
ce_status ce_distill_bwd(const void* logits, ce_dtype dtype, int64_t dim0, int64_t dim1, int64_t V,
                         const int64_t strides[3], const int64_t* teacher_tokens,
                         const int64_t teacher_token_strides[3], const void* teacher_logits,
                         ce_dtype teacher_dtype, const int64_t teacher_strides[3], int64_t K,
                         float temperature, int normalize, int64_t ignore_idx, int reduce_loss,
                         const float* stats, const float* dloss, const int64_t* n_non_ignore,
                         void* grad, const int64_t grad_strides[3], void* stream);

/* Waits for `stream`, then copies the device error word of the last pass that
 * used `workspace` into *host_err (host pointer).  Returns CE_OK,
 * CE_ERR_TARGET_RANGE or CE_ERR_DEVICE_TIMEOUT from its bits, CE_ERR_LAUNCH if
 * the copy fails.  Diagnostic use: this is the only call that synchronises. */
ce_status ce_get_error(const void* workspace, void* stream, uint32_t* host_err);

/* Failure detection check (no counterpart on the pages).  Every wait inside
 * this library's kernels -- on a TMA copy landing, on a ring slot, on a row
 * handed between warps -- is bounded: after ~1.5 s it gives up, sets
 * CE_DEVERR_TIMEOUT in the workspace error word and lets the kernel return,
 * so a lost copy is reported instead of hanging the GPU.  This call runs that
 * same bounded wait once, in a one-thread kernel, on an mbarrier that nothing
 * arrives on, and writes the result as the error word of `workspace`
 * (>= 256 bytes, 16-byte aligned): ce_get_error then returns
 * CE_ERR_DEVICE_TIMEOUT after ~1.5 s, and the stream stays usable.  Returns
 * CE_OK once the kernel is enqueued, CE_ERR_INVALID_ARG for a bad workspace. */
ce_status ce_wait_timeout_probe(void* workspace, size_t workspace_bytes, void* stream);

/* Static English description of a status code. */
const char* ce_status_string(ce_status status);

/* Path the planner would take for these arguments (host only): CE_PATH_ROW,
 * CE_PATH_CLUSTER, CE_PATH_TWO_STAGE, CE_PATH_STREAM, CE_PATH_WARP or
 * CE_PATH_VECROW, with the vocabulary chunk count in *chunks_out (host
 * pointer, may be NULL).  Returns -1 for arguments
 * ce_fwd_bwd would reject, -2 for a forced path that cannot run them. */
int ce_plan_path(const void* logits, ce_dtype dtype, int64_t dim0, int64_t dim1, int64_t V,
                 const int64_t strides[3], const ce_options* opts, int* chunks_out);

#ifdef __cplusplus
}
#endif

#endif /* GBCE_CE_H */
