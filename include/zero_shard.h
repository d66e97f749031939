/* zero_shard.h -- C ABI of the ZeRO per-rank shard step on AMD Instinct MI355X (gfx950).
 *
 * One data-parallel rank owns a contiguous slice ("shard") of a flat buffer of
 * Psi parameters.  After the gradient reduce-scatter, the rank holds the N
 * ranks' 16-bit gradient contributions for its slice.  The shard step
 *   1. sums them in fp32, removes the loss scale and averages,
 *   2. checks for inf/NaN and computes the global L2 norm (with optional
 *      clipping and loss-scale-driven skipping),
 *   3. runs mixed-precision Adam(W) on the fp32 master weights, momentum and
 *      variance of the slice,
 *   4. casts the new master weights to fp16/bf16 into the rank's slot of the
 *      full parameter buffer that the all-gather fills.
 * Sources (page titles and sections):
 *   "CMU 11-868 L18: How ZeRO Cuts Data-Parallel Memory", Mechanism 1, steps 3-6
 *     (reduce-scatter to fp32, update own slice of variance/momentum/params,
 *     copy to fp16, all-gather);
 *   "ZeRO: Memory Optimizations Toward Training Trillion Parameter Models"
 *     (paper-graph summary), 3.4: model-state analysis (16 Psi bill), Stage 1
 *     (Pos) and Stage 2 (Pos+g), and the residual-state note on gradient-norm
 *     buffers;
 *   "zero-stages-simulation" README, partitioning paragraph: the flattened
 *     buffer is cut into N contiguous pieces of (almost) the same length and
 *     rank r holds piece r;
 *   "ZeRO: Memory Optimization for Large Models" (lesson), Stage 1 and 2;
 *   "ZeRO Stage 1/2/3" guide, section 5 (AdamW with weight decay, the
 *     reduce bucket size);
 *   "CMU 11-868 L18", Other memory optimizations (ZeRO++ block-quantised
 *     payloads); paper summary 3.4, Stage 2 bucketization (gradients reduced
 *     bucket by bucket during the backward pass).
 *
 * Conventions for every call below.
 *   - Pointers named *_dev are device pointers (hipMalloc'd or torch tensors);
 *     all other pointers are host pointers.  Every buffer is owned by the
 *     caller.  The library never allocates or frees device memory.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).
 *     Calls that touch device memory only enqueue work on `stream` and return;
 *     they never synchronise.  Results are visible after the caller syncs.
 *   - Arguments are validated before anything is enqueued: on an argument
 *     error (EINVAL, EALIGN, ERANGE, ESPACE) nothing was enqueued and nothing
 *     was written.  EHIP (the runtime refused a launch) can follow earlier
 *     launches of the same call (a pass is issued as several launches, see
 *     ZERO_LAUNCH_TILES).  zero_last_error() describes the problem.  Faults
 *     inside kernels surface at the next sync.
 *   - 16-bit data is passed as raw storage (uint16 bit patterns); `dtype`
 *     selects ZERO_F16 (IEEE binary16) or ZERO_BF16 (bfloat16).
 *   - Element counts and offsets are int64 (Psi reaches 1.3e10 elements).
 *   - Alignment: contribution buffers, their row stride (a multiple of 8
 *     elements), g and the fp32 state arrays must be 16-byte aligned; rows of
 *     a row table need 8 bytes.  The gather slot needs only 2-byte alignment.
 *   - valid_len == 0 (an empty tail rank) is legal: nothing is enqueued except
 *     where the call says otherwise.
 *   - Calls on different streams are independent as long as they use
 *     different ctrl blocks and workspaces.
 *   - Sizes the library cannot see are the caller's to guarantee: a gather
 *     buffer holds at least offset + valid_len elements; contribution rows
 *     hold valid_len elements (and a [N, stride] buffer N * stride); g and
 *     flat state arrays valid_len floats; a paired state's buffer
 *     zero_pair_elems;
 *     workspaces ws_bytes (checked against zero_workspace_bytes); quantised
 *     codes zero_qcode_bytes and block records zero_qblock_count entries.
 *     A buffer shorter than that is read or written out of bounds.
 */
#ifndef ZERO_SHARD_H
#define ZERO_SHARD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum { ZERO_F16 = 1, ZERO_BF16 = 2 };

enum {
    ZERO_OK = 0,
    ZERO_EINVAL = -1, /* bad argument (null pointer, count, dtype, ...) */
    ZERO_EALIGN = -2, /* misaligned pointer or stride */
    ZERO_ERANGE = -3, /* size or offset out of the supported range */
    ZERO_ESPACE = -4, /* workspace too small */
    ZERO_EHIP = -5    /* the HIP runtime refused a launch */
};

enum { ZERO_SCALER_NONE = 0, ZERO_SCALER_STATIC = 1, ZERO_SCALER_DYNAMIC = 2 };

#define ZERO_MAX_CONTRIB 1024 /* largest N accepted by the reduce */
#define ZERO_MAX_RANKS 64     /* most ctrl blocks combined in one call; most rows in a row table */
#define ZERO_QBLOCK 2048      /* elements per quantisation block (one tile) */

/* Parameters of one quantisation block: value = scale * (code - zero).  A
 * block that held a non-finite value has scale NaN and zero 0. */
typedef struct {
    float scale;
    int32_t zero;
} zero_qblock;

/* Optimizer, clipping and loss-scale settings, passed by host pointer and
 * copied into the kernel arguments.  The pages name Adam (Kingma and Ba) and
 * AdamW with weight_decay but print no update; the library applies
 * bias-corrected Adam with epsilon outside the square root and decoupled
 * weight decay:  m = b1 m + (1-b1) g;  v = b2 v + (1-b2) g*g;
 * p = p - lr ((m / (1-b1^t)) / (sqrt(v / (1-b2^t)) + eps) + wd p),
 * every operation rounded to fp32, b^t a running fp64 product.
 * max_grad_norm > 0 turns clipping on: g is multiplied by
 * min(1, max_grad_norm / (norm + 1e-6)), the coefficient formed in fp64 and
 * rounded to fp32 (the rule of torch.nn.utils.clip_grad_norm_ given an fp64
 * norm).
 * scaler: NONE keeps S = 1; STATIC keeps the initial S; DYNAMIC halves S
 * (not below min_scale) on a skipped step and doubles it after
 * growth_interval consecutive applied steps, unless the doubled value is
 * not finite, when S stays (torch._amp_update_scale_'s schedule, plus the
 * min_scale floor).  A step whose reduced gradient holds inf or NaN is
 * always skipped. */
typedef struct zero_hparams {
    float lr, beta1, beta2, eps, weight_decay, max_grad_norm;
    int32_t scaler;
    float min_scale;
    int32_t growth_interval;
} zero_hparams;

/* Control block: 128 bytes in DEVICE memory, one per rank, written only by the
 * library's kernels.  Host code may copy it back to read the decisions.
 * It carries the step-to-step scalars so that no step needs a host sync. */
typedef struct zero_ctrl {
    double sumsq;       /* last step: global sum of g^2 over all ranks (fp64) */
    double norm;        /* last step: sqrt(sumsq) (inf/NaN when the gradient was) */
    double beta1_pow;   /* beta1^t */
    double beta2_pow;   /* beta2^t */
    float loss_scale;   /* S that the next step's contributions carry */
    float scale_used;   /* S of the last step */
    float clip;         /* clip factor applied by the last step (1 when none) */
    int32_t nonfinite;  /* last step: 1 if any reduced element was inf/NaN */
    int32_t skip;       /* last step was skipped (state, slot and t unchanged) */
    int32_t t;          /* applied optimizer steps */
    int32_t good_steps; /* applied steps since the last skip or doubling point */
    int32_t cur;        /* fused path: which set of the paired state is current */
    uint32_t arrive;    /* internal: arrival counter of the norm reduction, 0 between calls */
    uint32_t reserved[15];
} zero_ctrl;

/* Elements per workgroup tile of every streaming pass.  The fused path's
 * double-buffered state interleaves its two sets tile by tile. */
#define ZERO_TILE 2048

/* Launch sizes: a streaming pass (reduce, fused step, Adam) over valid_len
 * elements is issued as ceil(ceil(valid_len / ZERO_TILE) / T) consecutive
 * launches of at most T tiles on the caller's stream, which a profiler lists
 * one by one; the results are those of one launch.  T = ZERO_LAUNCH_TILES
 * for the Adam passes and for a pass that reads N <= 8 contribution rows;
 * over N > 8 rows (reduce and fused step, every source) T =
 * max(ZERO_LAUNCH_MIN_TILES, ZERO_LAUNCH_ROW_TILES / N) (zero_launch_tiles).
 * The fused step that also writes the quantised all-gather payload takes at
 * most ZERO_LAUNCH_PAYLOAD_TILES of those. */
#define ZERO_LAUNCH_TILES 32768
#define ZERO_LAUNCH_ROW_TILES 131072
#define ZERO_LAUNCH_MIN_TILES 2048
#define ZERO_LAUNCH_PAYLOAD_TILES 16384

/* One rank's fp32 optimizer state: master weights, Adam m, Adam v.
 * Flat form (two-pass path, pack/unpack): three arrays of valid_len
 * contiguous floats.
 * Paired form (fused path): ONE buffer of zero_pair_elems(valid_len) floats
 * holding two copies (sets) of the whole state, interleaved per tile of
 * ZERO_TILE elements as [tile][set][master | m | v][ZERO_TILE]: array q
 * (0 master, 1 m, 2 v) of set s for element i lives at buffer
 * [(i / ZERO_TILE) * 6 * ZERO_TILE + s * 3 * ZERO_TILE + q * ZERO_TILE
 * + i % ZERO_TILE].  Its zero_state is {buffer, buffer + ZERO_TILE,
 * buffer + 2 * ZERO_TILE}; the paired calls check that and return EINVAL
 * otherwise.  A tile's whole state (both sets, all three arrays, 48 KiB) is
 * one contiguous block, so the fused pass reads one set and writes the other
 * in one region of memory; with the launch configuration of the passes this
 * measured 1-2% faster than three separately allocated arrays. */
typedef struct zero_state {
    float *master;
    float *m;
    float *v;
} zero_state;

/* Partition ("zero-stages-simulation" README, flat partitioning paragraph;
 * lesson "ZeRO: Memory Optimization for Large Models", Stage 1 step 3):
 * the flat buffer is split into N contiguous shards of ceil(Psi/N) elements,
 * rank r owns [r*shard, r*shard + valid) with valid = clamp(Psi - r*shard, 0,
 * shard); tail ranks are short or empty.  Pure host arithmetic.
 * Returns ZERO_EINVAL for psi < 1, nranks < 1, rank outside [0, nranks) or a
 * null output pointer. */
int zero_partition(int64_t psi, int32_t nranks, int32_t rank, int64_t *shard_len,
                   int64_t *offset, int64_t *valid_len);

/* Bytes of the device workspace per tile of ZERO_TILE elements: the first
 * level of the norm and overflow reduction keeps one partial per tile. */
#define ZERO_PARTIAL_BYTES 16

/* Buckets (paper summary 3.4, Stage 2, bucketization: gradients are reduced
 * bucket by bucket as the backward pass produces them; "ZeRO Stage 1/2/3"
 * guide, section 5: reduce_bucket_size).  The per-element calls
 * (zero_reduce_grads and its _rows/_q forms, zero_fused_step and its
 * _rows/_q/_qgather forms) may be issued as several calls over consecutive
 * pieces of one shard, each piece [b0, b0 + len) starting at a multiple of
 * ZERO_TILE, as the pieces arrive.  The call for a piece takes every
 * per-element pointer advanced by b0 elements (contribution rows, g, the
 * 16-bit slot's offset; the paired state's pointers by 6 * b0 floats; INT8 codes
 * by b0 bytes, INT4 codes by b0 / 2, block records by b0 / ZERO_TILE), and
 * the workspace advanced by (b0 / ZERO_TILE) * ZERO_PARTIAL_BYTES bytes with
 * ws_bytes reduced by as much; ctrl, hparams and the row stride stay the
 * same.  After the last piece, zero_grad_norm_overflow over the whole
 * workspace and valid_len, then the rest of the step over the whole shard
 * (zero_adam_step or zero_adam_step_qgather; zero_fused_restore or
 * zero_fused_restore_q), complete the step: the results equal those of one
 * call over the whole shard, bit for bit.  On the fused path each piece's
 * Adam update can therefore run as soon as its gradient has arrived; the
 * skip decision still waits for the last piece. */

/* sizeof(zero_ctrl); allocate that many bytes of device memory per rank. */
size_t zero_ctrl_bytes(void);

/* Device workspace (bytes) needed by zero_reduce_grads and zero_fused_step
 * for a shard of valid_len elements: one 16-byte partial (fp64 sum of
 * squares, non-finite flag) per tile of ZERO_TILE elements, plus 256 slots
 * for the second level of the reduction (about 0.8% of the shard's fp16
 * size). */
size_t zero_workspace_bytes(int64_t valid_len);

/* Most tiles per launch T of a pass that reads nranks contribution rows, as
 * defined with ZERO_LAUNCH_TILES; nranks <= 0 gives the Adam passes' T. */
int64_t zero_launch_tiles(int32_t nranks);

/* Floats of the one buffer of a paired (fused-path) state for valid_len
 * elements: 6 * ceil(valid_len / ZERO_TILE) * ZERO_TILE. */
size_t zero_pair_elems(int64_t valid_len);

/* Initialise a ctrl block on `stream`: t = 0, beta powers 1, loss scale S
 * (must be finite and > 0; use 1 without a scaler), cur = 0, arrive = 0. */
int zero_ctrl_init(zero_ctrl *ctrl_dev, float loss_scale, void *stream);

/* Reduce ("CMU 11-868 L18", Mechanism 1 step 3: the reduce-scatter leaves each
 * rank the fp32 mean of all ranks' gradients over its own slice only; paper
 * summary 3.4 Stage 2, reduce-scatter of gradients):
 *   g[i] = fl32( sum_{k=0..N-1} C[k][i] ) * fl32(1 / (N * S)),   i < valid_len,
 * summed in fp32 in rank order k = 0..N-1; S is ctrl->loss_scale.
 * contrib_dev: N rows of `stride` elements (16-bit, dtype), row k at
 * contrib_dev + k*stride; only columns < valid_len are read.
 * g_dev: valid_len floats, written.
 * The same pass writes the first level of the norm and overflow reduction,
 * one partial per workgroup, into ws_dev (ws_bytes >= zero_workspace_bytes).
 * Errors: EINVAL (null, dtype, nranks outside [1, ZERO_MAX_CONTRIB],
 * stride < valid_len), EALIGN, ESPACE. */
int zero_reduce_grads(const void *contrib_dev, int32_t dtype, int32_t nranks, int64_t stride,
                      int64_t valid_len, const zero_ctrl *ctrl_dev, float *g_dev, void *ws_dev,
                      size_t ws_bytes, void *stream);

/* zero_reduce_grads with the N contribution rows in separate places: row k
 * starts at rows_dev[k] (valid_len 16-bit values; element i of the shard at
 * rows_dev[k][i]).  This is the form a reduce-scatter takes when every rank
 * reads its slice of the N ranks' gradient buffers directly, each slice
 * mapped into this process from its owner's memory ("CMU 11-868 L18",
 * Mechanism 1 step 3; paper summary 3.4 Stage 2): no staging copy into one
 * [N, stride] buffer.  The result is bit-identical to zero_reduce_grads on
 * the same rows (same order k = 0..N-1).  rows_dev is a host array of nranks
 * device pointers, copied into the launch (reusable on return); each pointer
 * must be non-NULL and 8-byte aligned, rows may alias (they are only read).
 * Errors: EINVAL (null table or row, dtype, nranks outside
 * [1, ZERO_MAX_RANKS]), EALIGN (a row not 8-byte aligned, g), ESPACE. */
int zero_reduce_grads_rows(const void *const *rows_dev, int32_t dtype, int32_t nranks,
                           int64_t valid_len, const zero_ctrl *ctrl_dev, float *g_dev,
                           void *ws_dev, size_t ws_bytes, void *stream);

/* Norm, overflow and step decisions (paper summary 3.4, residual states:
 * gradient-norm computation over all gradients; "CMU 11-868 L18", The memory
 * bill, same note).  Combines the per-tile partials that the previous
 * zero_reduce_grads or zero_fused_step left in each ws_dev[r] (valid_len[r]
 * elements) into the global sum of squares and the global non-finite flag of
 * the `nranks` ranks given (nranks > 1 stands in for the scalar all-reduce
 * between data-parallel ranks; with one rank they are its own).  The
 * reduction is deterministic: contiguous ranges of the concatenated partials
 * are summed in order, then the ranges in index order.  Then, in every ctrl
 * block: norm = sqrt(sumsq); skip = nonfinite; loss-scale update; clip
 * factor; if applied: t += 1, beta powers advance and, when `pingpong` is
 * nonzero, cur flips to the state set the fused step just wrote.  Enqueued
 * even when every valid_len is 0.
 * ws_dev, valid_len and ctrl_dev are host arrays of nranks entries (ws_dev and
 * ctrl_dev entries are device pointers).  Each ws_dev[r] must be the whole
 * workspace of zero_workspace_bytes(valid_len[r]) bytes that the step used
 * (the reduction keeps its second level behind rank 0's partials).  All ctrl
 * blocks must hold the same scalars (they do when they are always updated
 * together), and calls sharing ctrl_dev[0] must not overlap.
 * Errors: EINVAL (null, nranks outside [1, ZERO_MAX_RANKS], bad hparams),
 * EALIGN, ERANGE. */
int zero_grad_norm_overflow(int32_t nranks, void *const *ws_dev, const int64_t *valid_len,
                            zero_ctrl *const *ctrl_dev, const zero_hparams *hp,
                            int32_t pingpong, void *stream);

/* Adam on the owned slice ("CMU 11-868 L18", Mechanism 1 step 4: the rank's
 * fp32 master weights and both Adam moments are the only optimizer state it
 * touches; paper summary 3.4 Stage 1), fused with the cast into the gather
 * slot (Mechanism 1 step 5: the new master weights, rounded to the 16-bit
 * format).
 * Two-pass path: runs after zero_reduce_grads and zero_grad_norm_overflow
 * (pingpong = 0), reads g_dev and ctrl (skip, clip, t, beta powers), updates
 * state in place.  When gather_dev is not NULL, writes
 * RNE_dtype(master[i]) to gather_dev[offset + i].  A skipped step returns
 * from every workgroup without writing.
 * Errors: EINVAL, EALIGN, ERANGE (offset < 0). */
int zero_adam_step(const zero_state *state, const float *g_dev, int64_t valid_len,
                   const zero_hparams *hp, const zero_ctrl *ctrl_dev, void *gather_dev,
                   int32_t gather_dtype, int64_t offset, void *stream);

/* zero_adam_step that also writes the quantised all-gather payload of the
 * new parameters (ZeRO++, "CMU 11-868 L18", Other memory optimizations; see
 * zero_fused_step_qgather): codes_dev and blocks_dev equal, bit for bit,
 * what zero_quantize_blocks(gather_dtype, bits) would write from the 16-bit
 * slot after the step.  gather_dev may be NULL (no 16-bit slot written);
 * gather_dtype always names the 16-bit format that is quantised.  A skipped
 * step writes nothing, so slot and payload keep the previous step's values;
 * the caller initialises the payload with the slot (zero_quantize_blocks
 * over the initial slot), since the first step may be skipped.
 * Errors: as zero_adam_step, plus EINVAL (bits not 8 or 4, null codes or
 * blocks, gather dtype) and EALIGN (codes or blocks not 8-byte aligned). */
int zero_adam_step_qgather(const zero_state *state, const float *g_dev, int64_t valid_len,
                           const zero_hparams *hp, const zero_ctrl *ctrl_dev, void *gather_dev,
                           int32_t gather_dtype, int64_t offset, int32_t bits, void *codes_dev,
                           zero_qblock *blocks_dev, void *stream);

/* Cast ("CMU 11-868 L18", Mechanism 1 steps 5-6; lesson Stage 1 step 4):
 * gather_dev[offset + i] = RNE_dtype(master_dev[i]) for i < valid_len,
 * unconditionally (also used to fill the initial parameters). */
int zero_cast_to_gather(const float *master_dev, int64_t valid_len, void *gather_dev,
                        int32_t dtype, int64_t offset, void *stream);

/* Fused single pass (clipping off): reduce + norm/overflow partials + Adam +
 * cast, reading each contribution and each state word once.  Because the
 * skip decision is only known after every element has been summed, the
 * state is double-buffered in the paired layout (zero_state above): the
 * kernel reads the set ctrl->cur names and writes the other one;
 * zero_grad_norm_overflow with pingpong = 1 then makes the written set
 * current, or keeps the old one on a skipped step, and zero_fused_restore
 * rewrites the gather slot from the kept master on a skipped step.  Bias
 * correction uses t+1.  pair: a paired state (one 16-byte aligned buffer of
 * zero_pair_elems(valid_len) floats, see zero_state).  Requires hp->max_grad_norm <= 0
 * (EINVAL otherwise).  Other arguments as in zero_reduce_grads and
 * zero_adam_step; gather_dev must not be NULL. */
int zero_fused_step(const void *contrib_dev, int32_t contrib_dtype, int32_t nranks,
                    int64_t stride, const zero_state *pair, int64_t valid_len, void *gather_dev,
                    int32_t gather_dtype, int64_t offset, const zero_hparams *hp,
                    const zero_ctrl *ctrl_dev, void *ws_dev, size_t ws_bytes, void *stream);

/* zero_fused_step with the contribution rows given as a table of row
 * pointers, as in zero_reduce_grads_rows (same requirements on rows_dev and
 * nranks <= ZERO_MAX_RANKS): the one-pass reduce-scatter + Adam + cast of a
 * rank that reads the N ranks' slices where they lie.  Bit-identical to
 * zero_fused_step on the same rows.  Speed depends on where the rows lie:
 * on the 13B shard, rows that start at the same offset in their pages (N
 * separate, equally aligned allocations) ran about 4% slower than rows in
 * one [N, stride] buffer, and row k started k * 4 KiB into its allocation
 * recovered about half of that; the table itself costs 0.3%. */
int zero_fused_step_rows(const void *const *rows_dev, int32_t contrib_dtype, int32_t nranks,
                         const zero_state *pair, int64_t valid_len, void *gather_dev,
                         int32_t gather_dtype, int64_t offset, const zero_hparams *hp,
                         const zero_ctrl *ctrl_dev, void *ws_dev, size_t ws_bytes, void *stream);

/* After a fused step's zero_grad_norm_overflow: if ctrl->skip, rewrite
 * gather_dev[offset + i] from the current master of the paired state;
 * otherwise every workgroup returns at once. */
int zero_fused_restore(const zero_state *pair, int64_t valid_len, void *gather_dev,
                       int32_t dtype, int64_t offset, const zero_ctrl *ctrl_dev, void *stream);

/* Copies a flat state (valid_len floats per array) into the current set of a
 * paired state (set ctrl->cur), e.g. to load initial or checkpointed weights. */
int zero_pair_store(const zero_state *flat, const zero_state *pair, int64_t valid_len,
                    const zero_ctrl *ctrl_dev, void *stream);

/* Copies the current set of a paired state out to a flat state. */
int zero_pair_load(const zero_state *pair, const zero_state *flat, int64_t valid_len,
                   const zero_ctrl *ctrl_dev, void *stream);

/* ---- Several ranks' shards on one GPU ---------------------------------------
 * "zero-stages-simulation" README (riteshverma), the per-stage data-flow
 * table: its toy runs every rank of the data-parallel group in one process,
 * each rank owning one shard.  When several ranks' shards share a GPU and
 * each is small (the toy's 32 shards have ten tiles each), one launch per
 * shard leaves the chip idle between launches.  The calls below are
 * zero_fused_step and zero_fused_restore (fused path), and zero_reduce_grads
 * and zero_adam_step (two-pass path), for up to ZERO_MAX_RANKS shards at
 * once, as one launch per ZERO_BATCH_SHARDS shards: every shard's results are
 * bit-identical to its own calls'.  Between the two launches of a step,
 * zero_grad_norm_overflow over the shards' workspaces and ctrl blocks takes
 * the shared decision. */

/* One shard of a batched call: what the single-shard calls take for it.  Each
 * call reads only the fields it needs (see below). */
typedef struct zero_shard {
    const void *contrib_dev; /* [nranks, stride] 16-bit rows, 16-byte aligned */
    int64_t stride;          /* elements between rows: >= valid_len, a multiple of 8 */
    float *pair_dev;         /* fused path: paired state, zero_pair_elems(valid_len) floats,
                                16-byte aligned (the buffer zero_state's master points to) */
    int64_t valid_len;       /* at most one launch of tiles (see the calls) */
    int64_t offset;          /* the shard's slot in the gather buffer, in elements */
    zero_ctrl *ctrl_dev;     /* the shard's (rank's) ctrl block */
    void *ws_dev;            /* zero_workspace_bytes(valid_len) bytes, 16-byte aligned */
    size_t ws_bytes;
    zero_state state;        /* two-pass path: flat master, m, v of valid_len floats */
    float *g_dev;            /* two-pass path: the reduced gradient, valid_len floats,
                                16-byte aligned */
} zero_shard;

#define ZERO_BATCH_SHARDS 32 /* most shards in one launch of a batched call */

/* zero_fused_step for each of the nshards (1..ZERO_MAX_RANKS) shards in the
 * host array `shards` (contrib_dev, stride, pair_dev, valid_len, offset,
 * ctrl_dev, ws_dev and ws_bytes are read), which share contrib_dtype, nranks,
 * the gather buffer and its dtype, and hp (no clipping).  The shards' states,
 * slots, ctrl blocks and workspaces must not overlap.  Every shard is checked
 * before anything is enqueued, with the errors of zero_fused_step; a shard of
 * more than zero_launch_tiles(nranks) tiles returns ERANGE (step it with its
 * own calls).  Shards with valid_len 0 launch nothing; so in the calls below. */
int zero_fused_step_shards(const zero_shard *shards, int32_t nshards, int32_t contrib_dtype,
                           int32_t nranks, void *gather_dev, int32_t gather_dtype,
                           const zero_hparams *hp, void *stream);

/* zero_fused_restore for each shard after the decision (only pair_dev,
 * valid_len, offset and ctrl_dev are read; at most ZERO_LAUNCH_TILES tiles
 * per shard). */
int zero_fused_restore_shards(const zero_shard *shards, int32_t nshards, void *gather_dev,
                              int32_t gather_dtype, void *stream);

/* zero_reduce_grads for each shard (contrib_dev, stride, valid_len, ctrl_dev,
 * ws_dev, ws_bytes and g_dev are read; at most zero_launch_tiles(nranks)
 * tiles per shard, ERANGE otherwise). */
int zero_reduce_grads_shards(const zero_shard *shards, int32_t nshards, int32_t contrib_dtype,
                             int32_t nranks, void *stream);

/* zero_adam_step for each shard after the decision (state, g_dev, valid_len,
 * offset and ctrl_dev are read; at most ZERO_LAUNCH_TILES tiles per shard);
 * gather_dev NULL writes no slot.  Clipping as in zero_adam_step. */
int zero_adam_step_shards(const zero_shard *shards, int32_t nshards, const zero_hparams *hp,
                          void *gather_dev, int32_t gather_dtype, void *stream);

/* ---- Block-quantised payloads (ZeRO++) --------------------------------------
 * "CMU 11-868 L18", Other memory optimizations: ZeRO++ quantises the
 * parameters of the forward all-gather block-wise from 16 bits to INT8 with a
 * zero point, and the gradient reduce-scatter to INT8 or INT4.  The page
 * gives neither block size nor rounding; this library's reading:
 *   blocks of ZERO_QBLOCK consecutive elements from the start of the buffer
 *   (the last may be short), Q = 2^bits - 1, and per block
 *     lo = min(0, min x), hi = max(0, max x),
 *     scale = (hi - lo) / Q (1 when that is 0),
 *     zero  = clamp(rint(-lo / scale), 0, Q),
 *     code  = clamp(rint(x * (1 / scale)) + zero, 0, Q),
 *   each operation one fp32 rounding, rint half to even: per block, the
 *   affine quantisation of PyTorch (MinMaxObserver's scale and zero point,
 *   quantize_per_tensor's codes, quint4x2's nibble order), which floors the
 *   scale at fp32 epsilon instead.  Real 0 is exact; |x - value| <= scale / 2
 *   up to the roundings.  A block holding inf or
 *   NaN, or whose scale overflows, gets scale NaN, zero 0 and codes 0, so it
 *   dequantises to NaN and a downstream overflow check still fires.
 *   Codes: bits = 8, one byte per element; bits = 4, two per byte, the
 *   even-indexed element in the low nibble.
 * codes and blocks must be 8-byte aligned; a 16-bit src or dst needs only
 * 2-byte alignment (a parameter slot at any offset), with vector accesses
 * where its alignment allows. */

/* Blocks of a quantised buffer of len elements: ceil(len / ZERO_QBLOCK). */
size_t zero_qblock_count(int64_t len);

/* Code bytes of a quantised buffer of len elements: len (8 bits) or
 * ceil(len / 2) (4 bits); 0 for len <= 0. */
size_t zero_qcode_bytes(int64_t len, int32_t bits);

/* Quantises len 16-bit values (dtype) at src_dev into codes_dev
 * (zero_qcode_bytes) and blocks_dev (zero_qblock_count entries): a sender's
 * gradient slice for a quantised reduce-scatter, or a rank's parameter slot
 * for a quantised all-gather.  Deterministic (no atomics).
 * Errors: EINVAL (null, dtype, bits not 8 or 4), EALIGN, ERANGE. */
int zero_quantize_blocks(const void *src_dev, int32_t dtype, int64_t len, int32_t bits,
                         void *codes_dev, zero_qblock *blocks_dev, void *stream);

/* dst_dev[i] = RNE_dtype(scale_b * (code_i - zero_b)), b = i / ZERO_QBLOCK:
 * the receiving side of a quantised all-gather. */
int zero_dequantize_blocks(const void *codes_dev, const zero_qblock *blocks_dev, int32_t bits,
                           int64_t len, void *dst_dev, int32_t dtype, void *stream);

/* zero_reduce_grads over quantised contributions: row k is codes_dev[k] with
 * blocks_dev[k], each quantised from the start of this rank's slice (the
 * sender quantises every destination's slice on its own), so block b covers
 * shard elements [b * ZERO_QBLOCK, ...).  Each value is dequantised as above
 * (one fp32 rounding) and the N values are summed in fp32 in rank order;
 * overflow flag, 1/(N*S) and the norm partials are as in zero_reduce_grads.
 * codes_dev and blocks_dev are host arrays of nranks device pointers
 * (nranks <= ZERO_MAX_RANKS), copied into the launch.
 * Errors: EINVAL (null table or row, bits, nranks), EALIGN, ESPACE, ERANGE. */
int zero_reduce_grads_q(const void *const *codes_dev, const zero_qblock *const *blocks_dev,
                        int32_t bits, int32_t nranks, int64_t valid_len,
                        const zero_ctrl *ctrl_dev, float *g_dev, void *ws_dev, size_t ws_bytes,
                        void *stream);

/* zero_fused_step over quantised contributions (rows as in
 * zero_reduce_grads_q): the one-pass step of a rank whose gradient
 * reduce-scatter arrives as INT8 or INT4 blocks. */
int zero_fused_step_q(const void *const *codes_dev, const zero_qblock *const *blocks_dev,
                      int32_t bits, int32_t nranks, const zero_state *pair, int64_t valid_len,
                      void *gather_dev, int32_t gather_dtype, int64_t offset,
                      const zero_hparams *hp, const zero_ctrl *ctrl_dev, void *ws_dev,
                      size_t ws_bytes, void *stream);

/* zero_fused_step (strided rows) that also writes the quantised all-gather
 * payload of the rank's new parameters ("CMU 11-868 L18", Other memory
 * optimizations: ZeRO++ quantises the parameters block-wise to INT8 with a
 * zero point for the forward all-gather).  Block b covers shard elements
 * [b * ZERO_QBLOCK, ...), which is exactly one tile of the pass, so the
 * block's range, record and codes come out of the same pass as the new
 * parameters: codes_dev (zero_qcode_bytes(valid_len, bits)) and blocks_dev
 * (zero_qblock_count(valid_len) records) equal, bit for bit, what
 * zero_quantize_blocks(gather_dtype, bits) would write from the 16-bit slot
 * after the step.  gather_dev may be NULL: then no 16-bit slot is written
 * (every rank rebuilds the parameters from the gathered payload with
 * zero_dequantize_blocks, this one included); gather_dtype still names the
 * 16-bit format that is quantised.  bits is 8 (the page's choice) or 4.
 * On a skipped step, zero_fused_restore_q (not zero_fused_restore) rewrites
 * the slot and the payload.  Other arguments and errors as in zero_fused_step
 * and zero_quantize_blocks (codes_dev and blocks_dev 8-byte aligned). */
int zero_fused_step_qgather(const void *contrib_dev, int32_t contrib_dtype, int32_t nranks,
                            int64_t stride, const zero_state *pair, int64_t valid_len,
                            void *gather_dev, int32_t gather_dtype, int64_t offset, int32_t bits,
                            void *codes_dev, zero_qblock *blocks_dev, const zero_hparams *hp,
                            const zero_ctrl *ctrl_dev, void *ws_dev, size_t ws_bytes,
                            void *stream);

/* zero_fused_step_qgather with the contribution rows given as a table of row
 * pointers (rows_dev as in zero_reduce_grads_rows, nranks <= ZERO_MAX_RANKS).
 * Bit-identical to zero_fused_step_qgather on the same rows.  Errors: those
 * of zero_fused_step_rows for the table, then those of
 * zero_fused_step_qgather for the rest. */
int zero_fused_step_rows_qgather(const void *const *rows_dev, int32_t contrib_dtype,
                                 int32_t nranks, const zero_state *pair, int64_t valid_len,
                                 void *gather_dev, int32_t gather_dtype, int64_t offset,
                                 int32_t bits, void *codes_dev, zero_qblock *blocks_dev,
                                 const zero_hparams *hp, const zero_ctrl *ctrl_dev, void *ws_dev,
                                 size_t ws_bytes, void *stream);

/* zero_fused_step_qgather over quantised contributions (qcodes_dev,
 * qblocks_dev and qbits as codes_dev, blocks_dev and bits of
 * zero_reduce_grads_q): ZeRO++ end to end in one pass, with the gradient
 * reduce-scatter arriving as INT8 or INT4 blocks and the parameters leaving
 * as the bits-bit all-gather payload (codes_dev, blocks_dev).  The two widths
 * are independent.  Errors: those of zero_fused_step_q for the quantised
 * rows (qbits, tables, 8-byte alignment), then those of
 * zero_fused_step_qgather for the rest. */
int zero_fused_step_q_qgather(const void *const *qcodes_dev, const zero_qblock *const *qblocks_dev,
                              int32_t qbits, int32_t nranks, const zero_state *pair,
                              int64_t valid_len, void *gather_dev, int32_t gather_dtype,
                              int64_t offset, int32_t bits, void *codes_dev,
                              zero_qblock *blocks_dev, const zero_hparams *hp,
                              const zero_ctrl *ctrl_dev, void *ws_dev, size_t ws_bytes,
                              void *stream);

/* After a zero_fused_step_qgather's (or its _rows/_q form's)
 * zero_grad_norm_overflow: if ctrl->skip,
 * rewrite the slot (when gather_dev is not NULL) and the payload from the
 * current master of the paired state, as the step would have written them;
 * otherwise every workgroup returns at once. */
int zero_fused_restore_q(const zero_state *pair, int64_t valid_len, void *gather_dev,
                         int32_t dtype, int64_t offset, int32_t bits, void *codes_dev,
                         zero_qblock *blocks_dev, const zero_ctrl *ctrl_dev, void *stream);

/* ---- Allocation-free step ---------------------------------------------------
 * For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation): one rank's
 * whole fused step without a workspace argument.  It is zero_fused_step
 * followed by zero_grad_norm_overflow (this rank alone, pingpong = 1) and
 * zero_fused_restore, with the per-tile norm and overflow partials kept in
 * a static device array inside the library (ZERO_NOALLOC_MAX_LEN /
 * ZERO_TILE + 256 partials of ZERO_PARTIAL_BYTES, about 16 MiB, held by every
 * GPU the library runs on until the process ends); the results equal those
 * three calls' bit for bit.  The caller passes inputs, state, slot and ctrl
 * as for zero_fused_step; the call allocates nothing.  All calls on one GPU
 * share that array: calls that overlap on one GPU (on different streams, or
 * from different threads without ordering) race, so they must be ordered.
 * Errors: those of zero_fused_step, ERANGE for valid_len above
 * ZERO_NOALLOC_MAX_LEN (nothing enqueued), EHIP if the array's device
 * address cannot be obtained (first call on each device). */
#define ZERO_NOALLOC_MAX_LEN 2147483648LL
int zero_fused_step_noalloc(const void *contrib_dev, int32_t contrib_dtype, int32_t nranks,
                            int64_t stride, const zero_state *pair, int64_t valid_len,
                            void *gather_dev, int32_t gather_dtype, int64_t offset,
                            const zero_hparams *hp, zero_ctrl *ctrl_dev, void *stream);

/* ---- Matrices: orthogonalised updates ---------------------------------------
 * For parameters that are whole matrices inside a shard.  A stack is `count`
 * row-major matrices of rows x cols elements.  In this part and the next one no
 * output may share memory with what its call still reads (EINVAL), except
 * where it says so; outputs and workspaces of one call lie apart.
 *
 * The orthogonalisation of G is k steps of an odd quintic iteration on the
 * normalised matrix, on whichever side is smaller:
 *     X <- G / (||G||_F + eps)
 *     X <- (a I + b S + c S^2) X,  S = X X^T      (rows <= cols)
 *     X <- X (a I + b S + c S^2),  S = X^T X      (rows >  cols)
 * which drives every singular value of X towards 1 and keeps the singular
 * vectors.  A zero matrix gives zeros; a matrix holding inf or NaN gives NaN.
 * Between steps X is fp32; the products take fp16 operands (scaled, fp32 sums)
 * whose diagonals are kept apart in fp32.  Results in fp16, and all of matrices
 * whose smaller side is at most 128, take every operand in two fp16 parts: before
 * their own rounding they are within 1e-5 of the iteration in 64 bits (relative,
 * Frobenius norm; for rank one see below).  Results in bf16 and the optimizer's
 * update take one part above 128: within about 1e-3, up to 1.8e-3 where the rank
 * is low or the elements are equal, beside bf16's own 1.7e-3, in 0.4 of the time.
 * Sums of equal terms round alike, so that matrices of rank one may be off by up to 5e-7 times
 * their smaller side more (constant ones; with normal factors 4e-5 to 3e-4). */
#define ZERO_F32 3 /* a dtype of the matrix calls below, where they say so */

#define ZERO_NS_REACH 3.5 /* singular values between steps, at most: the fp16 operands' range */

typedef struct zero_newton_schulz {
    /* The polynomial's coefficients, finite.  Singular values of X start in [0, 1]; a
     * step takes those up to r to at most the largest |a s + b s^3 + c s^5|, s in [0, r].
     * That bound, from step to step, may not exceed ZERO_NS_REACH before the last step
     * (EINVAL).  The usual coefficients stay below 1.3. */
    float a, b, c;
    float eps;     /* added to the Frobenius norm, >= 0 */
    int32_t steps; /* k, 0..64 */
} zero_newton_schulz;

/* Bytes of device workspace for zero_orthogonalize and zero_muon_step over
 * such a stack (16-byte aligned; 0 where a workgroup holds a whole matrix, among
 * them all with both sides up to 128).  0 for sizes the calls refuse.
 * zero_muon_step, and zero_orthogonalize with a result in bf16, need only
 * zero_muon_workspace_bytes, which is never more. */
size_t zero_ns_workspace_bytes(int32_t count, int64_t rows, int64_t cols);
size_t zero_muon_workspace_bytes(int32_t count, int64_t rows, int64_t cols);

/* dst[b] = orthogonalisation of src[b].  src: src_dtype ZERO_F16, ZERO_BF16
 * or ZERO_F32; row r of matrix b starts at element b * src_stride + r * src_ld.
 * dst: dst_dtype ZERO_F16 or ZERO_BF16, laid out likewise; it may be src when
 * the elements' size and the layout agree.  count, rows or cols of 0: nothing is enqueued.
 * Errors: EINVAL (null pointer, dtype, coefficients, steps, eps), EALIGN (a
 * pointer not aligned to its elements, workspace not to 16 bytes), ERANGE
 * (rows or cols above 65536, negative sizes, count above 65535, ld below
 * cols, stride below the matrix), ESPACE (workspace too small). */
int zero_orthogonalize(const void *src_dev, int32_t src_dtype, int32_t count, int64_t rows,
                       int64_t cols, int64_t src_ld, int64_t src_stride, void *dst_dev,
                       int32_t dst_dtype, int64_t dst_ld, int64_t dst_stride,
                       const zero_newton_schulz *ns, void *ws_dev, size_t ws_bytes, void *stream);

/* How the orthogonalised update is scaled before it meets lr. */
enum {
    ZERO_MUON_SCALE_SHAPE = 0, /* sqrt(max(1, rows / cols)) */
    ZERO_MUON_SCALE_RMS = 1    /* 0.2 sqrt(max(rows, cols)): the root mean square of an AdamW update */
};

typedef struct zero_muon_hparams {
    float lr, momentum, weight_decay;
    int32_t nesterov; /* 0 or 1 */
    int32_t scale;    /* ZERO_MUON_SCALE_* */
    zero_newton_schulz ns;
} zero_muon_hparams;

/* One optimizer step for a stack of matrices of a shard, in place, beside
 * zero_adam_step for the shard's other parameters (two-pass path: g comes from
 * zero_reduce_grads, the decisions from zero_grad_norm_overflow):
 *     g' = clip g;  mom = mu mom + (1 - mu) g'
 *     u = nesterov ? (1 - mu) g' + mu mom : mom
 *     p = (p - lr wd p) - lr s NS(u);  slot = RNE16(p)
 * momentum, the decay and the final update round each operation to fp32 in
 * that order.  master_dev, mom_dev, g_dev: fp32; matrix b is the rows * cols
 * elements from b * stride.  ctrl_dev may be NULL (no clipping, no skip); on a
 * skipped step nothing is written.  gather_dev may be NULL (no slot), else
 * element i of master goes to gather[offset + i].  Errors: as
 * zero_orthogonalize's, and EINVAL for lr, momentum (0 <= mu < 1),
 * weight_decay or scale out of range. */
int zero_muon_step(float *master_dev, float *mom_dev, const float *g_dev, int32_t count,
                   int64_t rows, int64_t cols, int64_t stride, const zero_muon_hparams *hp,
                   const zero_ctrl *ctrl_dev, void *gather_dev, int32_t gather_dtype,
                   int64_t offset, void *ws_dev, size_t ws_bytes, void *stream);

/* The same with every operand in two fp16 parts, as for results in fp16: the update is
 * as exact as those above a smaller side of 128 too, in 2.4 times the time (the same
 * call up to 128).  ws: zero_ns_workspace_bytes. */
int zero_muon_step_exact(float *master_dev, float *mom_dev, const float *g_dev, int32_t count,
                         int64_t rows, int64_t cols, int64_t stride, const zero_muon_hparams *hp,
                         const zero_ctrl *ctrl_dev, void *gather_dev, int32_t gather_dtype,
                         int64_t offset, void *ws_dev, size_t ws_bytes, void *stream);

/* ---- Matrices: MXFP4 (OCP microscaling) operands -----------------------------
 * A matrix quantised along its rows: every 32 consecutive elements of a row
 * share a scale 2^(s - 127) (one byte s, E8M0) and hold 4-bit codes (E2M1:
 * 0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives; sign in bit 3).  For a
 * block whose largest magnitude is x, s - 127 = floor(log2 x) - 2 (not below
 * -127; x = 0: -127), each element is rounded to the nearest code, ties to
 * the even code, and saturates at 6.  A block holding inf or NaN has s = 255
 * (NaN) and codes 0.  Columns are padded with zeros to P = a multiple of 128.
 * codes: [rows][P / 2] bytes, the even element in the low four bits;
 * scales: [rows][P / 32] bytes; both 16-byte aligned. */
int64_t zero_mx4_padded(int64_t cols);
size_t zero_mx4_code_bytes(int64_t rows, int64_t cols);
size_t zero_mx4_scale_bytes(int64_t rows, int64_t cols);

/* Quantises src (rows x cols, row stride ld elements; ZERO_F16, ZERO_BF16 or
 * ZERO_F32) along its rows into codes/scales and, from the same read, along its
 * columns into codes_t/scales_t: the quantisation of the transposed matrix
 * (cols x rows).  Either pair may be NULL, not both.  Errors: EINVAL, EALIGN
 * (src to its elements, outputs to 16 bytes), ERANGE (negative sizes, rows or
 * cols above 2^24, ld below cols). */
int zero_mx4_quantize(const void *src_dev, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                      void *codes_dev, void *scales_dev, void *codes_t_dev, void *scales_t_dev,
                      void *stream);

/* The values: dst (rows x cols, row stride ld; ZERO_F16, ZERO_BF16 or
 * ZERO_F32, rounded to nearest even from the exact product). */
int zero_mx4_dequantize(const void *codes_dev, const void *scales_dev, int64_t rows, int64_t cols,
                        void *dst_dev, int32_t dtype, int64_t ld, void *stream);

/* c[i][j] = sum over k of A[i][k] B[j][k] (+ c[i][j] when accumulate is 1 and
 * c is ZERO_F32), A m x k and B n x k quantised along k, sums in fp32; c is
 * m x n, row stride ldc, ZERO_F16, ZERO_BF16 or ZERO_F32.  k = 0 gives zeros
 * (or c unchanged).  No product needs a workspace: zero_mx4_matmul_workspace_bytes
 * is 0 for all sizes, and ws is not looked at. */
size_t zero_mx4_matmul_workspace_bytes(int64_t m, int64_t n, int64_t k);
int zero_mx4_matmul(const void *a_codes_dev, const void *a_scales_dev, const void *b_codes_dev,
                    const void *b_scales_dev, int64_t m, int64_t n, int64_t k, void *c_dev,
                    int32_t c_dtype, int64_t ldc, int32_t accumulate, void *ws_dev,
                    size_t ws_bytes, void *stream);

/* zero_mx4_matmul with A given as values (ZERO_F16, ZERO_BF16 or ZERO_F32, row
 * stride lda) and quantised on the way in, for the few rows of single tokens: the codes
 * and scales of zero_mx4_quantize and the product of zero_mx4_matmul, whose fp32
 * sums may be added in another order (9 to 32 rows with n above 8192).  m is at most
 * ZERO_MX4_ROWS_MAX.  No workspace is needed up to m = 32 where m times the padded
 * k is at most 16384. */
#define ZERO_MX4_ROWS_MAX 64
size_t zero_mx4_matmul_rows_workspace_bytes(int64_t m, int64_t n, int64_t k);
int zero_mx4_matmul_rows(const void *a_dev, int32_t a_dtype, int64_t lda, const void *b_codes_dev,
                         const void *b_scales_dev, int64_t m, int64_t n, int64_t k, void *c_dev,
                         int32_t c_dtype, int64_t ldc, void *ws_dev, size_t ws_bytes,
                         void *stream);

/* A linear layer whose three products take MXFP4 operands, each quantised along the
 * dimension that the product sums over:
 *     y = x w^T,  dx = dy w,  dw = dy^T x
 * x is tokens x k, w n x k, y and dy tokens x n; all of one dtype (ZERO_F16,
 * ZERO_BF16 or ZERO_F32), each with its row stride in elements.  The forward
 * call reads x and w once and also leaves what the gradients need: x_t and w_t,
 * the operands of x^T and w^T (k x tokens and k x n), each one buffer of
 * zero_mx4_operand_bytes; either may be NULL.  dx needs w_t and dw x_t; either
 * gradient may be NULL.  The rounding to 4 bits is passed through.  Sizes are
 * at least 1.  Errors: EINVAL, EALIGN (matrices to their elements, the rest to
 * 16 bytes), ERANGE, ESPACE. */
size_t zero_mx4_operand_bytes(int64_t rows, int64_t cols);
size_t zero_mx4_linear_workspace_bytes(int64_t tokens, int64_t n, int64_t k);
int zero_mx4_linear(const void *x_dev, int64_t ldx, const void *w_dev, int64_t ldw, int32_t dtype,
                    int64_t tokens, int64_t n, int64_t k, void *y_dev, int64_t ldy, void *x_t_dev,
                    void *w_t_dev, void *ws_dev, size_t ws_bytes, void *stream);
size_t zero_mx4_linear_grad_workspace_bytes(int64_t tokens, int64_t n);
int zero_mx4_linear_grad(const void *dy_dev, int64_t lddy, int32_t dtype, int64_t tokens, int64_t n,
                         int64_t k, const void *x_t_dev, const void *w_t_dev, void *dx_dev,
                         int64_t lddx, void *dw_dev, int64_t lddw, void *ws_dev, size_t ws_bytes,
                         void *stream);

/* ---- Rows of tokens -----------------------------------------------------------
 * What a training step or a served token does between the linear layers.  Rows
 * are given by their first element and a row stride in elements; dtypes are
 * ZERO_F16, ZERO_BF16 or ZERO_F32; rows and columns go up to 2^24 unless a call
 * says otherwise.  What would take a launch of 2^32 threads or more is refused
 * (ERANGE): the norm has one for 8 or 16 columns of a row, the lookup 256 for a token
 * of 2048 columns or more.  Sums are fp32 or wider, in an order that depends on sizes
 * alone, but for rows that a call computes in 64 bits: those come last.
 *
 * MXFP8 rows: blocks of 32 along a row as in the part above, with 8-bit codes
 * (E4M3, largest 448).  A block's scale 2^(s - 127) is the smallest power of two
 * (s >= 0) that leaves its largest magnitude at 448 or below, so that nothing
 * saturates; each element is rounded to the nearest code, ties to even.  A block
 * holding inf or NaN has s = 255 (NaN) and codes 0.  codes: [rows][P] bytes, P as
 * above; scales: [rows][P / 32] (zero_mx4_scale_bytes); both 16-byte aligned.
 * Errors of all calls: EINVAL, EALIGN (rows to their elements, codes, scales and
 * workspaces to 16 bytes), ERANGE, ESPACE.  Results share no memory with inputs, with one
 * another or with the workspace (EINVAL) but where a call allows it. */
size_t zero_mx8_code_bytes(int64_t rows, int64_t cols);
int zero_mx8_quantize(const void *src_dev, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                      void *codes_dev, void *scales_dev, void *stream);
int zero_mx8_dequantize(const void *codes_dev, const void *scales_dev, int64_t rows, int64_t cols,
                        void *dst_dev, int32_t dtype, int64_t ld, void *stream);

/* c[i][j] = sum over k of A[i][k] B[j][k] (+ c[i][j] when accumulate is 1 and c is
 * ZERO_F32): A m x k in MXFP8, B n x k in MXFP4, both along k.  The _rows form takes
 * A as values (a_dtype, row stride lda) and quantises them on the way in; up to m = 32
 * with m times the padded k up to 8192 in the product's own kernel, without a
 * workspace.  k = 0 gives zeros (or c unchanged).  Results are sums in fp32, rounded once
 * to c's type. */
int zero_mx8_matmul(const void *a_codes_dev, const void *a_scales_dev, const void *b_codes_dev,
                    const void *b_scales_dev, int64_t m, int64_t n, int64_t k, void *c_dev,
                    int32_t c_dtype, int64_t ldc, int32_t accumulate, void *stream);
size_t zero_mx8_matmul_rows_workspace_bytes(int64_t m, int64_t n, int64_t k);
int zero_mx8_matmul_rows(const void *a_dev, int32_t a_dtype, int64_t lda, const void *b_codes_dev,
                         const void *b_scales_dev, int64_t m, int64_t n, int64_t k, void *c_dev,
                         int32_t c_dtype, int64_t ldc, int32_t accumulate, void *ws_dev,
                         size_t ws_bytes, void *stream);

/* Root-mean-square norm of every row, with the residual's addition:
 *     h = x + residual, rounded to the residual's type (h = x without one)
 *     y = h / sqrt(mean(h^2) + eps) * w
 * x, w and y are of one dtype; the residual and h of the same or ZERO_F32.
 * residual and h come together or are both NULL.  h may be the residual's place and
 * y x's (same row stride).  Squares that leave fp32's range are summed scaled.  The _mx8
 * form leaves y as MXFP8 rows.  eps >= 0. */
int zero_rms_norm(const void *x_dev, int32_t dtype, int64_t ldx, const void *residual_dev,
                  int32_t residual_dtype, int64_t ldr, const void *w_dev, int64_t tokens,
                  int64_t cols, float eps, void *y_dev, int64_t ldy, void *h_dev, int64_t ldh,
                  void *stream);
int zero_rms_norm_mx8(const void *x_dev, int32_t dtype, int64_t ldx, const void *residual_dev,
                      int32_t residual_dtype, int64_t ldr, const void *w_dev, int64_t tokens,
                      int64_t cols, float eps, void *codes_dev, void *scales_dev, void *h_dev,
                      int64_t ldh, void *stream);

/* Its gradients, from dy (dtype), h (h_dtype: dtype or ZERO_F32) and, where h went on
 * too, its gradient dh (h_dtype; may be NULL).  With u = h / sqrt(mean(h^2) + eps), g = dy w:
 *     dr = (g - u mean(g u)) / sqrt(mean(h^2) + eps) + dh    the residual's, h_dtype
 *     dx = dr rounded to dtype;   dw = sum over tokens of dy u, dtype
 * Each of dx, dr and dw may be NULL; the workspace is for dw.  Rows whose sums or
 * products leave fp32's range are computed in 64 bits. */
size_t zero_rms_norm_grad_workspace_bytes(int64_t tokens, int64_t cols);
int zero_rms_norm_grad(const void *dy_dev, int64_t lddy, const void *h_dev, int32_t h_dtype,
                       int64_t ldh, const void *w_dev, int32_t dtype, const void *dh_dev,
                       int64_t lddh, int64_t tokens, int64_t cols, float eps, void *dx_dev,
                       int64_t lddx, void *dr_dev, int64_t lddr, void *dw_dev, void *ws_dev,
                       size_t ws_bytes, void *stream);

/* y = x 65536 / (65536 - T) where element (r, c) stays, else 0; plus the residual
 * where there is one.  T = p 65536 rounded to a whole number (p in [0, 1]).  An element stays when its 16 bits are T or
 * more: word c % 8 / 2 (low half for even c) of Philox4x32-10 under the key seed (low
 * word first) at the counter {c / 8, r, low and high word of the offset}.  The offset is `offset` plus,
 * where offset_dev is not NULL, the number there when the kernel runs: a captured
 * graph draws anew when the program moves it between replays.  The mask depends on
 * r, c, seed and offset alone and is stored nowhere; the gradient is the same call
 * on dy without a residual.  y may be x's or the residual's place (same row stride).
 * rows up to 2^32, cols up to 2^34, rows times cols up to 2^40. */
int zero_dropout(const void *x_dev, int32_t dtype, int64_t ldx, const void *residual_dev,
                 int64_t ldr, int64_t rows, int64_t cols, double p, uint64_t seed,
                 uint64_t offset, const uint64_t *offset_dev, void *y_dev, int64_t ldy,
                 void *stream);

/* out[t] = table[ids[t]] * scale, rounded once; ids: `tokens` contiguous numbers of
 * id_bytes 4 or 8 (signed).  An id outside [0, vocab) gives zeros and takes no part in
 * the gradient (padding; the other ranks' part of a table that is split by rows).  The
 * gradient writes every row of the table's: scale times the sum of dy over the
 * row's tokens, in their order, in fp32, rounded once. */
int zero_embedding(const void *ids_dev, int32_t id_bytes, int64_t tokens, const void *table_dev,
                   int32_t dtype, int64_t ldt, int64_t vocab, int64_t cols, float scale,
                   void *out_dev, int64_t ldo, void *stream);
size_t zero_embedding_grad_workspace_bytes(int64_t tokens, int64_t vocab, int64_t cols);
int zero_embedding_grad(const void *ids_dev, int32_t id_bytes, int64_t tokens, const void *dy_dev,
                        int32_t dtype, int64_t lddy, int64_t vocab, int64_t cols, float scale,
                        void *dtable_dev, int64_t ldo, void *ws_dev, size_t ws_bytes,
                        void *stream);

/* Tokens by expert.  Slot t * k + j is token t's j-th assignment, ids its expert.
 * zero_expert_sort: order[i] = the slot at place i when the slots are sorted by expert
 * (equal ones in the order of slots; those outside [0, experts) last), place its
 * inverse, offsets[e] = the first place of expert e, offsets[experts] = the number of
 * slots that have one.  slots = tokens k up to 2^24. */
size_t zero_expert_sort_workspace_bytes(int64_t slots, int64_t experts);
int zero_expert_sort(const void *ids_dev, int32_t id_bytes, int64_t slots, int64_t experts,
                     int32_t *order_dev, int32_t *place_dev, int32_t *offsets_dev, void *ws_dev,
                     size_t ws_bytes, void *stream);

/* rows[place[slot]] = x[slot / k]; zeros at places from *used_dev on (used_dev =
 * offsets + experts).  rows: tokens k of them.  In this call and the next two a place
 * outside [0, tokens k) is left out. */
int zero_expert_rows(const void *x_dev, int32_t dtype, int64_t ldx, const int32_t *place_dev,
                     const int32_t *used_dev, int64_t tokens, int64_t k, int64_t cols,
                     void *rows_dev, int64_t ldr, void *stream);

/* y[t] = sum over j of weights[t][j] rows[place[t k + j]], slots without an expert left
 * out; in fp32, rounded once.  weights: [tokens][k], dtype or ZERO_F32; NULL: ones, which
 * is the gradient of zero_expert_rows.  The gradients: drows[place] = weight * dy[t], zeros
 * from *used_dev on; dweights[t][j] = rows[place] . dy[t], 0 without an expert.  Either
 * may be NULL (without dweights rows may be too). */
int zero_expert_combine(const void *rows_dev, int32_t dtype, int64_t ldr, const int32_t *place_dev,
                        const int32_t *used_dev, const void *weights_dev, int32_t weights_dtype,
                        int64_t tokens, int64_t k, int64_t cols, void *y_dev, int64_t ldy,
                        void *stream);
int zero_expert_combine_grad(const void *dy_dev, int64_t lddy, const void *rows_dev, int32_t dtype,
                             int64_t ldr, const int32_t *place_dev, const int32_t *used_dev,
                             const void *weights_dev, int32_t weights_dtype, int64_t tokens,
                             int64_t k, int64_t cols, void *drows_dev, int64_t lddr,
                             void *dweights_dev, void *stream);

/* Message for the last nonzero return on the calling thread ("" if none). */
const char *zero_last_error(void);

#ifdef __cplusplus
}
#endif

#endif
