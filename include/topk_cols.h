/*
 * topk_cols: column-wise top-k over a speculative drafter's vocabulary logits,
 * for AMD Instinct MI355X (gfx950).
 *
 * What it computes (ignis docs, page "DFlash2", section "How it works"):
 * for every column of a V-row logit matrix, select the k largest values and
 * their row ids, largest first, with ties broken toward the smaller row id.
 * The result is bit-identical to a plain per-column sort, so draft acceptance
 * cannot move.  A column is one draft position; the page's drafter proposes 7
 * per lane over a 248,046-token vocabulary (56 columns at eight lanes).
 *
 * The page leaves three points open.  This library reads them as follows.
 *   - Values compare as real numbers, so -0 equals +0 and a tie between them
 *     goes to the smaller row.  Subnormals compare exactly; nothing is flushed.
 *   - NaN of any sign or payload ranks above +Inf, and all NaNs tie with each
 *     other (the smaller row wins).
 *   - out_values holds the stored bit pattern of the selected element, so -0
 *     stays -0 and a NaN keeps its payload.
 *
 * Lifecycle: create a handle once per shape, run it any number of times,
 * destroy it.  All functions return a topk_status; none aborts or throws.
 */
#ifndef TOPK_COLS_H
#define TOPK_COLS_H

#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    TOPK_OK = 0,
    TOPK_ERR_INVALID_ARG = -1,  /* an argument is out of range, NULL or misaligned */
    TOPK_ERR_UNSUPPORTED = -2,  /* valid, but beyond this build's limits (k > TOPK_MAX_K, V > TOPK_MAX_V) */
    TOPK_ERR_HIP = -3,          /* a HIP runtime call failed (no device, launch error, ...) */
    TOPK_ERR_OUT_OF_MEMORY = -4, /* the workspace could not be allocated */
    TOPK_ERR_TIMEOUT = -5       /* reported by topk_cols_check: a run's cross-workgroup wait gave up */
} topk_status;

typedef enum {
    TOPK_BF16 = 0, /* bfloat16 stored as 16-bit patterns */
    TOPK_F32 = 1   /* IEEE binary32 */
} topk_dtype;

typedef enum {
    TOPK_COL_CONTIG = 0,     /* element (row r, column c) at x[c*ld + r], ld >= V */
    TOPK_ROW_INTERLEAVED = 1 /* element (row r, column c) at x[r*ld + c], ld >= C */
} topk_layout;

/* Largest k accepted. */
#define TOPK_MAX_K 64
/* Largest V accepted (row ids must fit in 24 bits). */
#define TOPK_MAX_V ((int64_t)((1 << 24) - 1))

typedef struct topk_cols *topk_cols_t;

/*
 * Create a handle for one shape on the current HIP device.
 *
 * V: rows (the vocabulary), 1 <= V <= TOPK_MAX_V.
 * C: columns (draft positions), >= 1.
 * k: 1 <= k <= V and k <= TOPK_MAX_K.
 * dtype, layout: see the enums.
 * ld: leading dimension in elements, ld >= V (column-contiguous) or ld >= C
 *     (row-interleaved).  Elements in the padding are never read.
 *
 * The handle owns a small device workspace: one partial list of k 8-byte
 * keys per column and vocabulary segment (C * segments * k keys), an error
 * word and, for the column-contiguous layout, one 128-byte line per column
 * holding a counter and the run count modulo 255, or, for the
 * row-interleaved layout, 32 4-byte bound words per column (C rounded up to
 * a multiple of 64) that the segments of a column share during a run.  Create allocates it on the
 * current device with hipMalloc, zeroes it and waits for the zeroing to
 * finish; create is not meant for the hot loop.  Every run leaves the
 * workspace ready for the next one; nothing is reset from the host.
 *
 * On any failure *out is set to NULL, and nothing stays allocated.
 * Returns TOPK_ERR_INVALID_ARG for a bad argument or a NULL out.
 * Returns TOPK_ERR_UNSUPPORTED when k > TOPK_MAX_K or V > TOPK_MAX_V, or
 * for the row-interleaved layout when C > 134,217,664.
 * Returns TOPK_ERR_HIP when there is no usable device.
 * Returns TOPK_ERR_OUT_OF_MEMORY when the allocation fails.
 */
int topk_cols_create(topk_cols_t *out, int64_t V, int64_t C, int32_t k, int32_t dtype,
                     int32_t layout, int64_t ld);

/*
 * Select the top k of every column.
 *
 * logits: device pointer to the matrix described at create.  It must be
 *         aligned to the element size.
 * out_values: device, C*k elements of the input dtype, aligned to the element
 *         size.  out_values[c*k + j] is the j-th largest of column c; j = 0 is
 *         the largest.
 * out_ids: device, C*k int32, 4-byte aligned.  out_ids[c*k + j] is the 0-based
 *         row of out_values[c*k + j].
 * stream: the HIP stream to enqueue on (0 = the null stream).
 *
 * Asynchronous: run only enqueues kernels.  It does not synchronize and does
 * not allocate.  The outputs are valid once the stream reaches this point.
 * The caller keeps ownership of all three buffers.  Runs on one handle must be
 * ordered on a single stream: the workspace serves one run at a time.  Use a
 * separate handle for each stream that runs concurrently.
 *
 * Graph capture: a run's enqueued work depends only on the handle's shape
 * and the arguments; the state that changes from run to run (the run count
 * that tags the column-contiguous layout's cross-workgroup lists) lives in
 * the workspace and is advanced by the kernels.  A run may therefore be
 * captured into a HIP graph and replayed (each replay is a run: replays
 * must not overlap each other or other runs on the handle).
 *
 * Cross-workgroup wait (column-contiguous layout): each column is merged by
 * the last of its workgroups to finish, which reads the others' lists and
 * waits, with a bound of tens of milliseconds, for any that has not landed
 * yet.  Every list was stored before its workgroup finished, so the wait
 * only covers stores still in flight and the bound is never reached in
 * normal operation.  If it were, that workgroup writes no output for the
 * column and sets the workspace's error word; topk_cols_check reports it.
 *
 * Returns TOPK_ERR_INVALID_ARG for a NULL or misaligned pointer, or a NULL
 * handle.  Returns TOPK_ERR_HIP when the launch fails.
 */
int topk_cols_run(topk_cols_t h, const void *logits, void *out_values, int32_t *out_ids,
                  hipStream_t stream);

/* Free the handle and its workspace.  NULL is accepted and returns TOPK_OK.
 * The caller must ensure no run on the handle is still in flight. */
int topk_cols_destroy(topk_cols_t h);

/*
 * Like topk_cols_run, over the first n_cols columns only (0 <= n_cols <= C):
 * a round in which fewer drafts are active than the handle was created for
 * (the "DFlash2" page, "How it works": the drafter proposes up to
 * spec.draft_tokens tokens per lane, so a round may carry fewer columns).
 * Lay the active columns out first; with a per-lane draft count, pack each
 * lane's active columns one after another and pass their total.
 *
 * Columns n_cols..C-1 of the matrix are not read, and out_values/out_ids are
 * written only in their first n_cols*k entries (same layout as
 * topk_cols_run).  n_cols = 0 enqueues nothing and returns TOPK_OK.  The
 * handle's launch decomposition (segments per column) stays the one chosen
 * at create, and the results are the same as a run on a matrix of n_cols
 * columns.  Ownership, ordering and capture rules are those of topk_cols_run.
 *
 * Returns TOPK_ERR_INVALID_ARG for n_cols < 0 or n_cols > C, and otherwise
 * as topk_cols_run.
 */
int topk_cols_run_n(topk_cols_t h, int64_t n_cols, const void *logits, void *out_values,
                    int32_t *out_ids, hipStream_t stream);

/*
 * Like topk_cols_run_n, with the row ids translated through a table: the
 * "DFlash2" page ("How it works") describes a "shortlist" head that scores
 * only the 131,072 most frequent tokens, so its row r stands for vocabulary
 * token row_to_id[r].  Selection is unchanged: values compare as for
 * topk_cols_run and ties go to the smaller ROW (shortlist position), not to
 * the smaller token id.  Only the reported id changes:
 * out_ids[c*k + j] = row_to_id[row of the j-th largest of column c].
 *
 * row_to_id: device, V int32 entries, 4-byte aligned, read-only, owned by
 *            the caller; any values (the table need not be a permutation).
 *
 * Returns TOPK_ERR_INVALID_ARG for a NULL or misaligned row_to_id, and
 * otherwise as topk_cols_run_n.
 */
int topk_cols_run_mapped(topk_cols_t h, int64_t n_cols, const void *logits, const int32_t *row_to_id,
                         void *out_values, int32_t *out_ids, hipStream_t stream);

/*
 * Sample one draft per column from its top-k list (the step after the
 * selection when the drafter samples: the "DFlash2" page measures sampled
 * drafting at temperature 1.0, top_p 0.95 and top_k 20, section "Greedy
 * coding is the best case" and the last row of "The numbers").  The page does
 * not spell out the sampler; this is the standard reading.  For column c with
 * top-k values v_0 >= ... >= v_{k-1} (values[c*k + j], largest first, as a
 * topk_cols run writes them):
 *   w_j = exp((v_j - v_0) / temperature),  S_m = w_0 + ... + w_{m-1},
 *   n   = the smallest m with S_m >= top_p * S_k   (the nucleus),
 *   u   = uniform in [0, 1) from Philox4x32-10 with counter
 *         (offset & 0xFFFFFFFF, offset >> 32, c, 0) and key
 *         (seed & 0xFFFFFFFF, seed >> 32): u = ((out0 << 32 | out1) >> 11) * 2^-53,
 *   j*  = the smallest j < n with S_{j+1} > u * S_n,
 * then out_ids[c] = ids[c*k + j*] and, if out_pos is not NULL,
 * out_pos[c] = j*.  A column whose v_0 is not finite (NaN, +Inf, -Inf) takes
 * j* = 0.  All arithmetic is IEEE double in the order written, with exp
 * evaluated by a fixed method (Cody-Waite reduction, degree-13 Taylor
 * polynomial by fused multiply-adds, ldexp), so the draw is reproducible
 * bit for bit by any implementation of these steps.  The same (seed,
 * offset, c) always gives the same u: advance offset between rounds.
 *
 * values: device, C*k elements of dtype (TOPK_BF16 or TOPK_F32), aligned to
 *         the element size; each row sorted largest first.
 * ids:    device, C*k int32 (rows, or token ids from topk_cols_run_mapped).
 * out_ids: device, C int32.  out_pos: device, C int32, or NULL.
 * All buffers are owned by the caller.  Asynchronous on stream; no
 * allocation, no synchronization, no handle.
 *
 * Returns TOPK_ERR_INVALID_ARG for a NULL or misaligned pointer, C < 1,
 * k < 1 or k > TOPK_MAX_K, an unknown dtype, temperature not finite and
 * positive, or top_p outside (0, 1]; TOPK_ERR_HIP when the launch fails.
 */
int topk_cols_sample(const void *values, const int32_t *ids, int64_t C, int32_t k, int32_t dtype,
                     double temperature, double top_p, uint64_t seed, uint64_t offset, int32_t *out_ids,
                     int32_t *out_pos, hipStream_t stream);

/*
 * The steps around the top-k in a round of speculative decoding.
 *
 * A round's matrix has one column per position.  Lane l owns the contiguous
 * columns col_start[l] .. col_start[l+1]-1 ("pack each lane's active columns
 * one after another", topk_cols_run_n); a lane with d drafts has d columns
 * of the drafter's logits, or d + 1 of the target's (column j of the lane
 * follows its first j drafts).  Where an entry point takes col_start NULL,
 * every lane has the same number of columns: C / lanes, and C must be a
 * multiple of lanes.  draft_start packs the drafts of the lanes in the same
 * way; NULL means n_drafts / lanes each.
 *
 *   topk_cols_plan     lays the round out: col_start, each column's lane,
 *                      position and cache slot, and the blocks it needs;
 *   topk_cols_adjust   applies penalties, biases and grammar masks to logits;
 *   topk_cols_verify   accepts or refuses drafts against the target's lists;
 *   topk_cols_count    adds the tokens a lane gained to its history, which
 *                      topk_cols_adjust reads.
 *
 * All of them are asynchronous on the stream, take no handle, allocate
 * nothing, keep nothing between calls and may be captured and replayed.
 * Buffers belong to the caller.  Index arrays are read on the device and
 * cannot be checked by the call: offsets outside their array are cut to it, a
 * lane that ends before it starts is empty, ids outside [0, V) are ignored, and
 * lanes must not overlap.  The argument structures are read before the call
 * returns.
 */

/* Most lanes of a call of these entry points (each of them looks at every
 * lane, whether it has columns or not). */
#define TOPK_MAX_LANES ((int64_t)1 << 20)

/* The rules of topk_cols_adjust.  Zero (NULL) leaves a rule out. */
typedef struct {
    int64_t V;                /* rows, 1 <= V <= TOPK_MAX_V */
    int64_t C;                /* columns of the matrix, >= 1 */
    int64_t lanes;            /* >= 1 */
    int32_t dtype;            /* topk_dtype */
    int32_t layout;           /* topk_layout */
    int64_t ld;               /* leading dimension of the logits, as for topk_cols_create */
    int64_t out_ld;           /* leading dimension of the result */
    const int32_t *col_start; /* device, lanes + 1, or NULL */
    /* The lanes' histories (written by topk_cols_count), both or neither:
     * counts[l*counts_ld + r]: bit 31 set if token r occurs in lane l's
     * prompt, the lower bits how often it occurs in its output;
     * seen[l*seen_ld + r/32]: bit r % 32 set where that word is not zero. */
    const int32_t *counts;
    int64_t counts_ld;        /* >= V */
    const uint32_t *seen;
    int64_t seen_ld;          /* >= ceil(V / 32) */
    const float *repetition;  /* device, lanes values > 0, or NULL: 1 */
    const float *presence;    /* device, lanes values, or NULL: 0 */
    const float *frequency;   /* device, lanes values, or NULL: 0 */
    /* Drafts that precede the columns, both or neither: column j of lane l
     * takes the lane's first j drafts as further output tokens. */
    const int32_t *drafts;    /* device, n_drafts token ids */
    const int32_t *draft_start; /* device, lanes + 1, or NULL: n_drafts / lanes each */
    int64_t n_drafts;
    /* Biases, all or none: entries bias_start[l] .. bias_start[l+1]-1 add
     * bias_values[e] to row bias_ids[e].  Of several entries for one row the
     * last counts.  Meant for lists of up to a few thousand entries: each
     * workgroup reads its lane's whole list. */
    const int32_t *bias_start; /* device, lanes + 1 */
    const int32_t *bias_ids;   /* device, n_bias */
    const float *bias_values;  /* device, n_bias */
    int64_t n_bias;
    /* Masks: row r of column c is allowed if bit r % 32 of
     * mask[m*mask_ld + r/32] is set, m = mask_index[c]; a column whose m is
     * outside [0, mask_count) has no mask.  mask_index NULL: m = c. */
    const uint32_t *mask;      /* device, mask_count rows of words, or NULL */
    int64_t mask_ld;           /* >= ceil(V / 32) */
    int64_t mask_count;        /* >= 1; >= C when mask_index is NULL */
    const int32_t *mask_index; /* device, C, or NULL */
} topk_adjust_rules;

/*
 * Apply penalties, biases and masks to logits.  With x the stored value of
 * row r in column c (column j of lane l), n the token's count in the lane's
 * output and the first j drafts, in that order:
 *   1. r occurs in the prompt or n > 0: x = x > 0 ? x / repetition : x * repetition
 *   2. n > 0:  x = x - (frequency * n + presence)
 *   3. r has a bias:  x = x + bias
 *   4. the mask forbids r:  x = -Inf
 * Steps 1 to 3 are carried out in binary64 and rounded once to binary32 and,
 * for TOPK_BF16, from there to bfloat16 (to nearest, ties to even).  An
 * element that no step applies to keeps its stored bits.  A mask may leave a
 * column empty: every row is then -Inf, and a top-k of it gives rows 0 to
 * k-1.
 *
 * logits, out: device, aligned to the element size.  out may be logits
 *   itself (then out_ld must be ld) and must not overlap it otherwise.
 *   Columns that belong to no lane, and the padding, are not written.
 *
 * Returns TOPK_ERR_INVALID_ARG for a NULL or misaligned pointer, a size or
 * leading dimension out of range, an incomplete group, lanes that do not
 * divide C (col_start NULL) or n_drafts (draft_start NULL);
 * TOPK_ERR_UNSUPPORTED for V > TOPK_MAX_V, lanes > TOPK_MAX_LANES, or C,
 * n_drafts, n_bias or mask_count beyond 2^31 - 1; TOPK_ERR_HIP when a launch
 * fails.
 */
int topk_cols_adjust(const topk_adjust_rules *rules, const void *logits, void *out, hipStream_t stream);

/*
 * Add tokens to the lanes' histories (see topk_adjust_rules).
 *
 * ids: device, n_ids token ids; lane l's are ids[start[l]] ..
 *   ids[start[l+1]-1].  Ids outside [0, V) (the -1 behind a lane's tokens in
 *   topk_cols_verify's output) are skipped.  May be NULL when n_ids is 0.
 * start: device, lanes + 1, or NULL: n_ids / lanes tokens each.
 * prompt_len: device, lanes, or NULL.  The first prompt_len[l] of a lane's
 *   tokens are prompt, the others output.  NULL: all are output.
 * fresh: device, lanes, or NULL.  A lane with fresh[l] != 0 starts anew: its
 *   history is cleared first.
 * counts, seen: device, updated; counts_ld >= V, seen_ld >= ceil(V / 32).
 *   A count must stay below 2^31.  Words beyond V are left as they are.
 * The result does not depend on the order of a lane's tokens.  Calls on the
 * same history must be ordered on a stream.
 *
 * Returns TOPK_ERR_INVALID_ARG for a NULL or misaligned pointer, V < 1,
 * lanes < 1, n_ids < 0, a leading dimension that is too small, or lanes that
 * do not divide n_ids (start NULL); TOPK_ERR_UNSUPPORTED for V > TOPK_MAX_V,
 * lanes > TOPK_MAX_LANES or n_ids beyond 2^31 - 1; TOPK_ERR_HIP when a launch
 * fails.
 */
int topk_cols_count(int64_t V, int64_t lanes, const int32_t *ids, int64_t n_ids, const int32_t *start,
                    const int32_t *prompt_len, const int32_t *fresh, int32_t *counts, int64_t counts_ld,
                    uint32_t *seen, int64_t seen_ld, hipStream_t stream);

typedef struct {
    int64_t lanes;               /* >= 1 */
    int32_t dtype;               /* topk_dtype of both lists' values */
    int32_t k;                   /* entries of a target list, 1 .. TOPK_MAX_K */
    int32_t kq;                  /* entries of a draft list, 1 .. TOPK_MAX_K (unused without draft lists) */
    int64_t C;                   /* target columns, >= 1 */
    const int32_t *col_start;    /* device, lanes + 1, or NULL */
    const void *target_values;   /* device, C*k, as a topk_cols run on the target's logits wrote them */
    const int32_t *target_ids;   /* device, C*k */
    int64_t n_drafts;            /* drafts in the buffers, >= 0 */
    const int32_t *draft_start;  /* device, lanes + 1, or NULL: n_drafts / lanes each */
    const int32_t *drafts;       /* device, n_drafts token ids (may be NULL when n_drafts is 0) */
    const void *draft_values;    /* device, n_drafts*kq, the lists the drafts were sampled from, or NULL */
    const int32_t *draft_ids;    /* device, n_drafts*kq, or NULL together with draft_values */
    double temperature;          /* >= 0, finite */
    double top_p;                /* in (0, 1] */
    uint64_t seed, offset;       /* as for topk_cols_sample */
    int64_t max_tokens;          /* >= 1: entries of a lane in out_tokens */
    int32_t *out_tokens;         /* device, lanes*max_tokens */
    int32_t *out_count;          /* device, lanes */
} topk_verify_args;

/*
 * Verify a round's drafts against the target's top-k lists and draw the
 * token that follows the last accepted one, so that the tokens are
 * distributed as samples of the target ("one target verify pass, commit the
 * longest agreeing run plus one token", the "DFlash2" page, "How it works";
 * the rule is the published acceptance test of speculative sampling:
 * Leviathan, Kalman and Matias, 2023).
 *
 * A list of values v_0 >= v_1 >= ... stands for the distribution
 * topk_cols_sample draws from: w_j = exp((v_j - v_0) / temperature), S_m =
 * w_0 + ... + w_{m-1}, n the smallest m with S_m >= top_p * S_k, and
 * probability w_j / S_n for j < n, 0 beyond.  With temperature 0, or where
 * v_0 is not finite, entry 0 has probability 1.  A token's probability is
 * that of the first entry with its id, 0 if there is none.  Without draft
 * lists a draft has probability 1 (it was not sampled).
 *
 * For lane l let m be the smallest of its draft count, its columns - 1 and
 * max_tokens - 1.  With p_j the distribution of its column j, d_j its j-th
 * draft, q_j that draft's list and u, u' two uniforms in [0, 1) of the
 * column:
 *   draft j < m is accepted if u * q_j(d_j) < p_j(d_j);
 *   t is the number of drafts accepted before the first refused one;
 *   the next token is entry i of column t, the smallest i of positive weight
 *   with R_{i+1} > u' * R_k, where R_i sums the first i of the weights
 *   max(p_t(i) - q_t(id_i), 0) if t < m, or p_t(i) if t = m or those are
 *   all 0 (the last entry of positive weight where rounding leaves none).
 * out_tokens[l*max_tokens ..] = the t drafts, the token, then -1;
 * out_count[l] = t + 1.  A lane without columns gets only -1, and count 0.
 *
 * u and u' come from Philox4x32-10 as in topk_cols_sample, with counter
 * (offset & 0xFFFFFFFF, offset >> 32, column, 1) for u and (.., 2) for u',
 * the column being the target column's index.  (topk_cols_sample uses 0, so
 * one offset can serve a round.)  Arithmetic is IEEE double in the order
 * written, exp as in topk_cols_sample, and a running sum is a scan: within
 * each 16 entries in steps of 1, 2, 4 and 8, then the sums of entries 0-15
 * and 32-47 onto the 16 that follow, then that of the first 32 onto the rest.
 * The result is reproducible bit for bit.
 *
 * Returns TOPK_ERR_INVALID_ARG for a NULL or misaligned pointer, a value out
 * of the ranges above, or lanes that do not divide C (col_start NULL) or
 * n_drafts (draft_start NULL); TOPK_ERR_UNSUPPORTED for lanes >
 * TOPK_MAX_LANES, or C, n_drafts or max_tokens beyond 2^31 - 1;
 * TOPK_ERR_HIP when the launch fails.
 */
int topk_cols_verify(const topk_verify_args *args, hipStream_t stream);

typedef struct {
    int64_t lanes;              /* >= 1 */
    int64_t capacity;           /* columns the outputs hold, >= 1 */
    int32_t block_size;         /* tokens of a cache block, >= 1 */
    const int32_t *lens;        /* device, lanes: tokens of each lane in the cache */
    const int32_t *add;         /* device, lanes: columns wanted this round; <= 0 for none */
    const int32_t *held;        /* device, lanes: blocks in the lane's table row */
    int32_t *table;             /* device, lanes rows of table_ld block ids; new ids are written */
    int64_t table_ld;           /* >= 1: the most blocks a lane can have */
    const int32_t *free_ids;    /* device, n_free_ids: a stack of free blocks, its top at the end */
    int64_t n_free_ids;         /* >= 0 */
    const int32_t *free_count;  /* device, 1: entries of free_ids that are free */
    int32_t *out_held;          /* device, lanes; not held itself */
    int32_t *out_free_count;    /* device, 1; not free_count itself */
    int32_t *out_refused;       /* device, 1: lanes that wanted columns and got none */
    int32_t *out_col_start;     /* device, lanes + 1 */
    int32_t *out_col_lane;      /* device, capacity: the column's lane, or -1 */
    int32_t *out_col_pos;       /* device, capacity: its token's position in the lane, or -1 */
    int64_t *out_slots;         /* device, capacity: where its keys go, or -1 */
} topk_plan_args;

/*
 * Plan a round: give every lane its columns, and the cache blocks its new
 * tokens need.
 *
 * Lane l's new tokens have positions lens[l] .. lens[l] + add[l] - 1; a
 * position p lies in entry p / block_size of the lane's table row and in
 * slot table[..] * block_size + p % block_size.  The lane needs
 *   need = max(0, ceil((lens + add) / block_size) - held)
 * further blocks (blocks left over from refused drafts count as held).
 * Lanes are served in order.  A lane with add > 0 is refused when its blocks
 * do not fit its table row or its tokens exceed 2^31 - 1, when the needs of the lanes up to and including
 * it (those refused for the former apart) exceed the free blocks and its own
 * need is not 0, or when the columns of the lanes up to and including it
 * (those refused for blocks apart) exceed the capacity.  A refused lane gets
 * no columns and no blocks.
 *
 * Served lane l takes free_ids[free_count - 1 - i], free_ids[free_count - 2
 * - i], ..., i being the blocks taken by the lanes before it, and they are
 * written to its table row from entry held[l] on.  out_held and
 * out_free_count state what holds afterwards: pass them as the next round's
 * held and free_count.  Blocks are given back by writing them to free_ids
 * behind the free ones and raising the count.  Columns from
 * out_col_start[lanes] on get lane, position and slot -1, so a round padded
 * to its capacity can be replayed from a captured graph.
 * lens < 0 counts as 0, held as cut to [0, table_ld], free_count to [0,
 * n_free_ids].  Outputs must not overlap the inputs or each other.
 *
 * Returns TOPK_ERR_INVALID_ARG for a NULL or misaligned pointer, a size out
 * of range, out_held == held or out_free_count == free_count;
 * TOPK_ERR_UNSUPPORTED for lanes > TOPK_MAX_LANES, or capacity, table_ld or
 * n_free_ids beyond 2^31 - 1; TOPK_ERR_HIP when the launch fails.
 */
int topk_cols_plan(const topk_plan_args *args, hipStream_t stream);

/*
 * Rounds whose drafts form a tree, and the cache that their keys go to.
 *
 * Column 0 of a lane is its anchor, the last committed token; the others are
 * drafts, and parents[c] gives for column c, the lane's column j, the column
 * of the lane that its token follows: parents[c] < j.  (A chain of drafts has
 * parents -1, 0, 1, ...; a column whose entry is outside [0, j) follows none.)
 * All arrays are packed like the columns (col_start, C).
 *
 *   topk_cols_tree         each column's ancestors, as a mask, and its position;
 *   topk_cols_cache_write  the columns' keys and values into the slots of
 *                          topk_cols_plan, which reserves them in column order:
 *                          column j of lane l lies behind the lane's lens[l]
 *                          tokens, at place lens[l] + j;
 *   topk_cols_attend       attention of the columns over cache and ancestors;
 *   topk_cols_verify_tree  the drafts that the target accepts: a path;
 *   topk_cols_cache_move   the path's keys and values close up behind the
 *                          lane's tokens.
 *
 * What is said above of the steps around the top-k holds for these too.
 * Lengths below 0 count as 0; a lane has at most 2^31 - 1 places, and no more
 * than its row of the table has slots for.
 */

/*
 * The tree of a round.
 *
 * parents: device, C.  lens: device, lanes, or NULL: 0.
 * mask: device, C rows of mask_ld >= 1 words.  Bit i % 32 of word i / 32 of
 *   column j's row is set if i == j or column i is an ancestor of j; all other
 *   bits of the row are 0.  (Columns from 32*mask_ld on have no bit.)
 * positions: device, C: lens[l] plus the number of the column's ancestors, the
 *   place its token has in the text.
 * Rows and positions of columns that belong to no lane are not written.
 *
 * Returns TOPK_ERR_INVALID_ARG for a NULL or misaligned pointer, C < 1, lanes
 * < 1, mask_ld < 1 or lanes that do not divide C (col_start NULL);
 * TOPK_ERR_UNSUPPORTED for lanes > TOPK_MAX_LANES or C or mask_ld beyond 2^31
 * - 1; TOPK_ERR_HIP when the launch fails.
 */
int topk_cols_tree(int64_t lanes, int64_t C, const int32_t *col_start, const int32_t *parents, const int32_t *lens,
                   uint32_t *mask, int64_t mask_ld, int32_t *positions, hipStream_t stream);

typedef enum {
    TOPK_CACHE_BF16 = 0, /* bfloat16 */
    TOPK_CACHE_FP8 = 1   /* 8-bit floating point, e4m3 (no infinities), with a power of two for each row */
} topk_cache_format;

/* Largest head dimension of a cache. */
#define TOPK_MAX_DIM 256

/*
 * A cache of keys and values in blocks, described by the caller (who owns its
 * buffers): element d of head h of slot s in layer y is at
 *   y*layer_stride + (s / block_size)*block_stride + (s % block_size)*slot_stride + h*head_stride + d
 * of keys, or of values; in a TOPK_CACHE_FP8 cache a row (a slot's head) stands
 * for its elements times 2^(b - 127), b being the byte at
 *   y*scale_layer_stride + (s / block_size)*scale_block_stride + (s % block_size)*scale_slot_stride
 *   + h*scale_head_stride
 * of key_scales, or of value_scales.  (b = 255 stands for NaN in all of the row;
 * topk_cols_cache_write never writes it.)
 */
typedef struct {
    int64_t layers;      /* >= 1 */
    int64_t blocks;      /* of a layer, >= 1 */
    int32_t block_size;  /* slots of a block, >= 1 */
    int32_t heads;       /* key heads, >= 1 */
    int32_t dim;         /* a multiple of 16, at most TOPK_MAX_DIM */
    int32_t format;      /* topk_cache_format */
    void *keys, *values; /* device, 16-byte aligned */
    /* strides in elements, >= 0 and multiples of 16 bytes */
    int64_t layer_stride, block_stride, slot_stride, head_stride;
    uint8_t *key_scales, *value_scales; /* device; unused with TOPK_CACHE_BF16 */
    int64_t scale_layer_stride, scale_block_stride, scale_slot_stride, scale_head_stride; /* in bytes, >= 0 */
} topk_cache;

typedef struct {
    int64_t C;              /* columns, >= 1 */
    int64_t layer;          /* of the cache, 0 .. layers - 1 */
    int32_t dtype;          /* topk_dtype of keys and values */
    const void *keys;       /* device, 16-byte aligned: element d of head h of column c at c*key_stride + h*key_head_stride + d */
    const void *values;
    int64_t key_stride, key_head_stride;     /* in elements, >= 0 and multiples of 16 bytes */
    int64_t value_stride, value_head_stride;
    const int64_t *slots;   /* device, C: where each column goes; outside the cache: nowhere */
} topk_cache_write_args;

/*
 * Write keys and values into a layer of the cache.
 *
 * TOPK_CACHE_BF16: elements are rounded to bfloat16 (to nearest, ties to even).
 * TOPK_CACHE_FP8: with a the largest finite |x_i| of a row (one head of one
 * column, keys and values apart), e is the smallest whole number with a <=
 * 448 * 2^e, at least -126; the row keeps x_i * 2^-e rounded to e4m3 (to
 * nearest, ties to even) and the byte e + 127.  448 is the largest value of
 * e4m3, so nothing overflows; infinities and NaN become NaN.  Multiplying by a
 * power of two is exact: reading back rounds no further.
 *
 * Slots must differ from each other.
 *
 * Returns TOPK_ERR_INVALID_ARG for a NULL or misaligned pointer, or a value or
 * stride out of the ranges above; TOPK_ERR_UNSUPPORTED for dim >
 * TOPK_MAX_DIM, blocks*block_size beyond 2^31 - 1, a layer whose last slot ends
 * more than 64 GiB (its scale: 4 GiB) from the layer's start, layers*heads beyond
 * 2^20 or C*heads beyond 2^26;
 * TOPK_ERR_HIP when the launch fails.
 */
int topk_cols_cache_write(const topk_cache *cache, const topk_cache_write_args *args, hipStream_t stream);

typedef struct {
    int64_t lanes;            /* >= 1 */
    int64_t C;                /* columns, >= 1 */
    int64_t layer;            /* of the cache, 0 .. layers - 1 */
    int32_t heads;            /* query heads, a multiple of the cache's heads: query head h reads head h / (heads / cache heads) */
    int32_t window;           /* >= 0; 0: none */
    float scale;              /* at most 2^127 in magnitude */
    const void *q;            /* device, 16-byte aligned, bfloat16: element d of head h of column c at c*q_stride + h*q_head_stride + d */
    int64_t q_stride, q_head_stride;     /* in elements, >= 0 and multiples of 8 */
    const int32_t *col_start; /* device, lanes + 1, or NULL */
    const int32_t *lens;      /* device, lanes: tokens of each lane before its columns */
    const int32_t *table;     /* device, lanes rows of table_ld block ids */
    int64_t table_ld;         /* >= 1 */
    const uint32_t *mask;     /* device, C rows of mask_ld words (topk_cols_tree), or NULL: a chain */
    int64_t mask_ld;          /* >= 1 with a mask */
    const int32_t *positions; /* device, C, or NULL: lens[l] + j */
    void *out;                /* device, 16-byte aligned, bfloat16, laid out like q by the strides below */
    int64_t out_stride, out_head_stride;
    void *workspace;          /* device, 256-byte aligned */
    int64_t workspace_bytes;  /* at least what topk_cols_attend_workspace says */
} topk_attend_args;

/*
 * Attention of a round's columns over the cache.
 *
 * For column c, column j of lane l (of n columns), and query head h:
 *   out = sum_p w_p v_p / sum_p w_p,  w_p = exp(s_p - max s),  s_p = scale * (q . k_p)
 * over the visible places p of the lane, k_p and v_p being the key and value
 * in slot table[l][p / block_size]*block_size + p % block_size:
 *   p < lens[l]:               visible, with a window if p > positions[c] - window
 *                              (positions below lens[l] count as lens[l]);
 *   lens[l] <= p < lens[l]+n:  visible if bit p - lens[l] of the column's mask is
 *                              set (columns from 32*mask_ld on are not), whatever
 *                              the window; without a mask if p - lens[l] <= j,
 *                              with a window also j - (p - lens[l]) < window.
 * A column with nothing visible, or whose scores are all -Inf, gets zeros.
 * What lies in places that are not visible does not matter, NaN and infinities
 * included.  Places beyond the table's row are not visible; block ids are cut
 * to the cache's.  Columns that belong to no lane are not written.
 *
 * Products are of bfloat16 elements (an e4m3 element times its power of two is
 * one, except that results below 2^-126 may be 0), sums are binary32; the
 * weights are rounded to bfloat16 before the sum over values, and the result
 * once to bfloat16.  The same call gives the same bits.  What other lanes'
 * columns hold does not matter; how many they have, and how long those lanes
 * are, decides how a lane's places are shared out among workgroups, so its sums
 * may be rounded differently next to other lanes.
 *
 * The workspace holds partial results of places that several workgroups share;
 * nothing in it is kept between calls.  Calls that may overlap need one each.
 * out must not overlap q or the cache.
 *
 * Returns TOPK_ERR_INVALID_ARG for a NULL or misaligned pointer, a value or
 * stride out of the ranges above, lanes that do not divide C (col_start NULL)
 * or a workspace that is too small; TOPK_ERR_UNSUPPORTED for lanes >
 * TOPK_MAX_LANES, dim > TOPK_MAX_DIM, table_ld, mask_ld or blocks*block_size
 * beyond 2^31 - 1, a layer larger than topk_cols_cache_write takes, layers*heads
 * beyond 2^20 or C*heads beyond 2^26; TOPK_ERR_HIP when a launch fails.
 */
int topk_cols_attend(const topk_cache *cache, const topk_attend_args *args, hipStream_t stream);

/* The bytes of workspace that topk_cols_attend needs for these arguments
 * (whose pointers are not looked at): they depend on sizes only, not on the
 * lanes' lengths.  Errors as for topk_cols_attend, bytes is then 0. */
int topk_cols_attend_workspace(const topk_cache *cache, const topk_attend_args *args, int64_t *bytes);

/*
 * Close up an accepted path: for i = 0, 1, ..., width - 1 in this order, the
 * keys and values of place lens[l] + columns[l*width + i] of lane l, in all
 * layers, go to place lens[l] + i (as topk_cols_attend counts places; rows and
 * scales are copied as they are).  Entries that are not larger than i, -1
 * behind the path among them, are left out, and so are places outside the
 * table's row and blocks outside the cache.  The entries of a lane that are
 * carried out must increase (a path's do: a parent comes before its child).
 *
 * lens: device, lanes.  table: device, lanes rows of table_ld block ids.
 * columns: device, lanes*width (topk_cols_verify_tree's out_columns).
 *
 * Returns TOPK_ERR_INVALID_ARG for a NULL or misaligned pointer, or a value or
 * stride out of range; TOPK_ERR_UNSUPPORTED for lanes > TOPK_MAX_LANES, dim >
 * TOPK_MAX_DIM, table_ld, width or blocks*block_size beyond 2^31 - 1, a layer
 * larger than topk_cols_cache_write takes, or layers*heads beyond 2^20;
 * TOPK_ERR_HIP when a launch fails.
 */
int topk_cols_cache_move(const topk_cache *cache, int64_t lanes, const int32_t *lens, const int32_t *table,
                         int64_t table_ld, const int32_t *columns, int64_t width, hipStream_t stream);

typedef struct {
    int64_t lanes;               /* >= 1 */
    int32_t dtype;               /* topk_dtype of both lists' values */
    int32_t k;                   /* entries of a target list, 1 .. TOPK_MAX_K */
    int32_t kq;                  /* entries of a draft list, 1 .. TOPK_MAX_K (unused without draft lists) */
    int64_t C;                   /* columns, >= 1 */
    const int32_t *col_start;    /* device, lanes + 1, or NULL */
    const void *target_values;   /* device, C*k, as a topk_cols run on the target's logits wrote them */
    const int32_t *target_ids;   /* device, C*k */
    const int32_t *tokens;       /* device, C: each column's token (the anchors' are not looked at) */
    const int32_t *parents;      /* device, C */
    const void *draft_values;    /* device, C*kq, or NULL: row c is the list that column c's children were sampled from */
    const int32_t *draft_ids;    /* device, C*kq, or NULL together with draft_values */
    const float *uniforms;       /* device, C*2, in [0, 1): u judges draft c, u' draws the token that follows column c */
    double temperature;          /* >= 0, finite */
    double top_p;                /* in (0, 1] */
    int64_t max_tokens;          /* >= 1: entries of a lane in out_tokens and out_columns */
    int32_t *out_tokens;         /* device, lanes*max_tokens */
    int32_t *out_columns;        /* device, lanes*max_tokens */
    int32_t *out_count;          /* device, lanes */
} topk_verify_tree_args;

/*
 * Verify a tree of drafts against the target's top-k lists, from given random
 * numbers, so that the tokens are distributed as samples of the target: the
 * acceptance test of topk_cols_verify, with the siblings of a refused draft
 * judged against what is left of the target's distribution (each of them
 * sampled on its own from the same list; Miao and others, 2024).
 *
 * Distributions, and a token's probability in them, are those of
 * topk_cols_verify.  Lane l starts at its column 0.  At column c, with w = p_c
 * and W = 1, its children x are judged in the order of their columns:
 *   x is accepted if u_x * q(x) * W < w(x), where q(x) is the probability of
 *   x's token in column c's draft list (1 without lists) and w(x) the weight of
 *   the first entry with that token, 0 if there is none; the lane goes on at x;
 *   otherwise each w_i becomes max(w_i - W * q_i, 0), q_i being the probability
 *   of entry i's token (without lists 1 for x's token, 0 for others), and W the
 *   sum of them; if that is 0, w is p_c and W is 1 again.
 * Where no child is accepted, or max_tokens - 1 are (no further one is judged
 * then: w = p_c), the lane ends with entry i of column c, the smallest i of
 * positive weight with R_{i+1} > u'_c * R_k, R_i being the sum of the first i
 * weights (the last entry of positive weight where rounding leaves none).
 * out_tokens[l*max_tokens ..] = the t accepted tokens, the last one, then -1;
 * out_columns[l*max_tokens ..] = column 0, the t accepted columns, then -1;
 * out_count[l] = t + 1.  A lane without columns gets only -1, and count 0.
 *
 * Arithmetic is IEEE double in the order written, exp and running sums as in
 * topk_cols_verify.  The result is reproducible bit for bit.
 *
 * Returns TOPK_ERR_INVALID_ARG for a NULL or misaligned pointer, a value out of
 * the ranges above, or lanes that do not divide C (col_start NULL);
 * TOPK_ERR_UNSUPPORTED for lanes > TOPK_MAX_LANES, or C or max_tokens beyond
 * 2^31 - 1; TOPK_ERR_HIP when the launch fails.
 */
int topk_cols_verify_tree(const topk_verify_tree_args *args, hipStream_t stream);

/* A static, human-readable name for a status code.  Never NULL. */
const char *topk_cols_status_string(int status);

/*
 * For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the run of
 * topk_cols_run for the shape (V, C, k, dtype, layout, ld) of
 * topk_cols_create, with no handle.  Nothing is allocated: the workspace is
 * a static array of 8 MiB that each GPU the library runs on holds until the
 * process ends.  The first call on a device looks the array's address up
 * (hipGetSymbolAddress); later calls only launch kernels.
 *
 * Arguments as for topk_cols_create and topk_cols_run (all pointers device
 * pointers owned by the caller).  The launch decomposition is the one
 * topk_cols_create would choose; results are identical to a handle's.
 * Asynchronous on stream; no synchronization, no allocation.
 *
 * Every call on a GPU shares that GPU's array, which keeps what the last
 * call left: each call that completes leaves the parts that must start at
 * zero at zero, so calls of any shape and layout may follow each other on
 * one stream, or be captured and replayed.  Calls that overlap on one GPU
 * (unordered streams, overlapping replays) race: order them.  A
 * cross-workgroup wait that gives up (never in normal operation) leaves an
 * error in the array; topk_cols_check(NULL) reports it and clears the array.
 *
 * Returns the errors of topk_cols_create for a bad shape, and
 * TOPK_ERR_UNSUPPORTED when C > 4096 or the shape's workspace exceeds the
 * array (for example 248,046 x 448 bf16 rows with k = 16 needs 7.0 MiB and
 * fits); TOPK_ERR_INVALID_ARG for a NULL or misaligned pointer;
 * TOPK_ERR_HIP when there is no device or the launch fails.
 */
int topk_cols_run_noalloc(int64_t V, int64_t C, int32_t k, int32_t dtype, int32_t layout, int64_t ld,
                          const void *logits, void *out_values, int32_t *out_ids, hipStream_t stream);

/*
 * Report whether any run on the handle since the last check had a
 * cross-workgroup wait give up (see topk_cols_run).  Waits for all work on
 * the handle's device to finish (hipDeviceSynchronize) and reads the
 * handle's error word: not meant for the hot loop.  With h = NULL it checks
 * the workspace of topk_cols_run_noalloc on the current device instead.
 *
 * Returns TOPK_OK when no wait gave up.  Returns TOPK_ERR_TIMEOUT when one
 * did: the outputs of the runs since the last check are not valid, and the
 * workspace has been reset (zeroed, synchronously), so later runs are valid
 * again.  Returns TOPK_ERR_HIP when a HIP call fails (for h = NULL: also
 * when there is no device).
 */
int topk_cols_check(topk_cols_t h);

/*
 * For tests of the error path only: with on != 0, every later column-
 * contiguous run of the handle (with more than one segment per column) has
 * its merging workgroups treat every other list as not yet written and give
 * up after a few re-reads, as if a list never arrived.  Every kernel still
 * runs to completion.  topk_cols_check then returns TOPK_ERR_TIMEOUT and
 * resets the workspace.  on = 0 restores normal runs.  Returns
 * TOPK_ERR_INVALID_ARG for a NULL handle.
 */
int topk_cols_debug_fail_waits(topk_cols_t h, int32_t on);

/*
 * Like topk_cols_create, but with the vocabulary-axis split fixed to
 * `segments` workgroups per column (row segments for the interleaved layout)
 * instead of the automatic choice; 0 means automatic.  For tests and tuning:
 * the result is the same for every split.  For the column-contiguous
 * layout segments above 64, and for the row-interleaved layout segments * k
 * above 2048, return TOPK_ERR_UNSUPPORTED; negative values return
 * TOPK_ERR_INVALID_ARG.
 */
int topk_cols_create_with_segments(topk_cols_t *out, int64_t V, int64_t C, int32_t k,
                                   int32_t dtype, int32_t layout, int64_t ld, int64_t segments);

/* Kernel families of the column-contiguous layout (topk_cols_create_tuned). */
typedef enum {
    TOPK_ALGO_AUTO = 0,       /* chosen from the shape */
    TOPK_ALGO_WORKGROUP = 1,  /* a workgroup per vocabulary segment */
    TOPK_ALGO_ONE_WAVE = 3    /* one wave per column and no vocabulary split: the design that the
                                 "DFlash2" page ("How it works") replaced, kept as a baseline;
                                 never chosen automatically */
} topk_algo;

/*
 * Like topk_cols_create_with_segments, with the kernel family fixed as well
 * (column-contiguous layout; the row-interleaved layout accepts only
 * TOPK_ALGO_AUTO).  For tests and tuning: every family gives the same result.
 * TOPK_ALGO_ONE_WAVE accepts segments 0 or 1 only (else
 * TOPK_ERR_UNSUPPORTED).  An unknown algo returns TOPK_ERR_INVALID_ARG.
 */
int topk_cols_create_tuned(topk_cols_t *out, int64_t V, int64_t C, int32_t k, int32_t dtype,
                           int32_t layout, int64_t ld, int64_t segments, int32_t algo);

/*
 * Introspection for tests and benchmarks.  Writes the launch decomposition
 * chosen at create.
 * segments: workgroups per column (vocabulary-axis split) for the
 *           column-contiguous kernels, or row segments for the interleaved one.
 * blocks: total workgroups of the scan kernel (the row-interleaved layout
 *         adds a merge kernel of ceil(C / 4) workgroups).
 * workspace_bytes: device bytes owned by the handle.
 * algo: the topk_algo in use (TOPK_ALGO_AUTO for the row-interleaved layout).
 * Any output pointer may be NULL.
 */
int topk_cols_query(topk_cols_t h, int64_t *segments, int64_t *blocks, int64_t *workspace_bytes,
                    int32_t *algo);

#ifdef __cplusplus
}
#endif

#endif /* TOPK_COLS_H */
