/*
 * dsatopk.h - C ABI of the dsatopk library: per-row windowed top-k selection
 * over fp32 indexer scores with a fused RAGGED or PAGED emit, for AMD
 * Instinct MI355X (gfx950).
 *
 * The operation (DeepSeek-V4 DSA indexer top-k transform, as described in
 * the sglang PR digests on prhub.com.cn):
 *
 *   For each row b, with L = max(seq_lens[b], 0) and s = row_starts[b]
 *   (0 when row_starts is NULL), select the k largest scores among
 *   scores[b * score_stride + s + j] for window positions j in [0, L).
 *   Equal scores (IEEE ==, so -0.0 equals +0.0) are ordered by lower
 *   position first. Rows with L <= k select every position 0 .. L-1 and do
 *   not read their scores. Each selected position j is emitted as
 *     RAGGED: j + out_offsets[b]
 *     PAGED:  page_table[b * page_table_stride + j / page_size] * page_size
 *             + j % page_size
 *   into row b of out ([num_rows, k] int32). The first min(k, L) slots of a
 *   row hold the selection in an unspecified order; slots min(k, L) .. k-1
 *   hold -1.
 *   Sources: PR #35175 digest ("RAGGED prefill top-k moved to the v2 JIT
 *   kernel"), section "Key source excerpts": topk_ragged_kernel (window,
 *   trivial path, -1 padding, output = position + out_offsets[b]) and
 *   TopKProblem (emit adds the bias; transform_output maps through the page
 *   table with page_bits = log2(page_size)). PR #26788 digest ("faster top-k
 *   + page-table transform (runtime k <= 2048)"), "Key source excerpts":
 *   plan_topk_v2 / topk_transform_512_v2 signatures, runtime k.
 *
 * Conventions for every call below:
 *   - Pointers named scores, seq_lens, row_starts, out_offsets, page_table,
 *     plan and out are DEVICE pointers. `stream` is a hipStream_t (NULL is
 *     the default stream).
 *   - Calls are asynchronous on `stream`, allocate nothing, never
 *     synchronize the host, and only launch kernels (no memset or copy
 *     nodes), so they may be captured in a HIP graph.
 *   - The caller owns every buffer. `scores` is only read; it is never
 *     written, not even outside the window.
 *   - Host-checkable preconditions are checked before anything is launched;
 *     on error nothing is written and a status other than DSATOPK_OK is
 *     returned. No call aborts or throws.
 *   - The library holds no global state and is safe to call from several
 *     host threads.
 */
#ifndef DSATOPK_H_
#define DSATOPK_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes (every call returns one of these as an int). */
enum {
    DSATOPK_OK = 0,
    /* k outside [1, DSATOPK_MAX_K]; num_rows < 0; a required pointer is NULL;
       score_stride < 1; page_size not a power of two in [1, 2^20];
       page_table_stride < 1. */
    DSATOPK_ERR_INVALID_ARG = 1,
    /* scores or plan not 16-byte aligned, or score_stride not a multiple of 4. */
    DSATOPK_ERR_ALIGNMENT = 2,
    /* plan_bytes smaller than dsatopk_plan_bytes(num_rows). */
    DSATOPK_ERR_PLAN_TOO_SMALL = 3,
    /* the HIP runtime reported an error (no device, launch failure). */
    DSATOPK_ERR_HIP = 4,
    /* dsatopk_paged_noalloc: num_rows above DSATOPK_NOALLOC_MAX_ROWS. */
    DSATOPK_ERR_TOO_LARGE = 5,
    /* workspace missing or smaller than dsatopk_attend_bytes(...),
       dsatopk_shared_bytes(...), dsatopk_expanded_bytes(...) or
       dsatopk_expanded_shared_bytes(...). */
    DSATOPK_ERR_WORKSPACE_TOO_SMALL = 6
};

/* Largest k (runtime value; one build serves every k). The pages bound the
   v2 kernel to 0 < topk <= 2048 (PR #35175 digest, backend dispatch
   condition; PR #26788 digest title). */
#define DSATOPK_MAX_K 2048

/* Longest supported window. Longer windows are a device-side precondition
   violation (see dsatopk_paged). */
#define DSATOPK_MAX_SEQ_LEN 131072

/* Element types of the serving operators' inputs. */
enum {
    DSATOPK_BF16 = 0, /* bfloat16 */
    DSATOPK_FP16 = 1, /* IEEE half */
    DSATOPK_FP8 = 2   /* e4m3 without infinities (OCP), the indexer only */
};

/* Human-readable name of a status code (static string, never NULL). */
const char* dsatopk_status_string(int status);

/* Size in bytes of the plan buffer for `num_rows` rows (0 if num_rows < 0). */
size_t dsatopk_plan_bytes(int32_t num_rows);

/*
 * dsatopk_plan - build the device-side schedule for a batch.
 *
 * Reads seq_lens[num_rows] and row_starts[num_rows] (int32, device;
 * row_starts may be NULL, meaning every window starts at column 0) and
 * writes the plan buffer (device, plan_bytes >= dsatopk_plan_bytes(num_rows),
 * 16-byte aligned): each row's length class (trivial or up to 8192 aligned
 * floats, up to 16384, up to 32768, longer) with the rows of each class
 * listed, and, when the batch has at most 256 rows longer than 32768, a cut
 * of each of them into segments of 8192 floats (4096 when that would give
 * fewer segments than the GPU's 256 CUs), served by one workgroup each,
 * with a zeroed exchange area per row through which the segments merge
 * their histograms. Longer rows of batches with more of them are read
 * whole by one workgroup each. Everything is computed on the device;
 * nothing is read back. The transform calls read the split schedule, and
 * in batches of up to 1024 rows at score strides above 40960 floats the
 * class lists, whose order (longest class first) sets which rows start
 * first; rows go to their kernel by their own length.
 *
 * The plan only schedules: a call given a plan built from different
 * seq_lens / row_starts / k, or no plan at all (NULL), returns the same
 * outputs (every kernel recomputes each row's class and segment count, and
 * a long row that does not match its planned segments is read whole). A
 * plan must come from a dsatopk_plan call with the same num_rows. A plan
 * may be reused by any number of later transform calls (one per layer,
 * say): each call leaves the exchange areas and its work counters zeroed
 * again. Calls that share one plan must not run concurrently.
 *
 * Split rows wait for each other with bounded polls. A wait that gives up
 * (which a correct launch never sees: it takes a segment that cannot run
 * for about a second) sets the plan's error word (dsatopk_plan_error) and
 * leaves that row's outputs all -1 instead of a partial selection; build
 * the plan again before its next use. Plan word 15 (the int32 at byte
 * offset 60) holds the number of polls after which such a wait gives up;
 * dsatopk_plan writes 0, meaning about 2^20. It is exposed for tests that
 * force a wait to give up.
 *
 * Source: PR #26788 digest, "Key source excerpts", plan_topk_v2 (a device
 * plan built from seq_lens and reused by the transform); the layout here is
 * this library's own.
 *
 * Errors: DSATOPK_ERR_INVALID_ARG (num_rows < 0, k outside [1, 2048],
 * NULL seq_lens or plan with num_rows > 0), DSATOPK_ERR_ALIGNMENT (plan not
 * 16-byte aligned), DSATOPK_ERR_PLAN_TOO_SMALL, DSATOPK_ERR_HIP (a launch
 * failed; its own status is checked, not an earlier one).
 * num_rows == 0 is a no-op.
 */
int dsatopk_plan(const int32_t* seq_lens, const int32_t* row_starts, int32_t num_rows, int32_t k,
                 void* plan, size_t plan_bytes, void* stream);

/*
 * dsatopk_plan_error - read a plan's error word.
 *
 * Copies the plan's error word into *error (host memory) after the work
 * already queued on `stream` and synchronizes `stream`: 0 when no split-row
 * wait of the transform calls since the plan was built gave up, 1 when one
 * did (those rows' outputs are all -1; see dsatopk_plan). Unlike the other
 * calls this one waits for the device and must not be captured in a graph.
 * plan is a device pointer from dsatopk_plan, plan_bytes its size.
 *
 * Errors: DSATOPK_ERR_INVALID_ARG (NULL plan or error),
 * DSATOPK_ERR_PLAN_TOO_SMALL (plan_bytes below the 256-byte header),
 * DSATOPK_ERR_HIP (the copy or the synchronization failed).
 */
int dsatopk_plan_error(const void* plan, size_t plan_bytes, int32_t* error, void* stream);

/*
 * dsatopk_paged - top-k with the PAGED emit.
 *
 * Source: PR #26788 digest ("faster top-k + page-table transform (runtime
 * k <= 2048)"), "Key source excerpts": topk_transform_512_v2 takes the
 * scores, seq_lens, the page tables, page_size and the plan and writes the
 * page-mapped indices; PR #35175 digest, TopKProblem::transform_output (the
 * map page_table[j >> page_bits] << page_bits | (j & (page_size - 1)), and
 * -1 for padding).
 *
 *   scores            fp32 [num_rows, score_stride], row-major, 16-B aligned
 *                     base, score_stride % 4 == 0. Read only.
 *   seq_lens          int32 [num_rows]; negative values are read as 0.
 *   row_starts        int32 [num_rows] or NULL (every window starts at
 *                     column 0). Any residue modulo 4 is allowed.
 *   page_table        int32 [num_rows, page_table_stride]; entry
 *                     j / page_size of row b is the physical page of window
 *                     position j.
 *   page_size         power of two in [1, 2^20].
 *   num_rows, k       0 <= num_rows; 1 <= k <= 2048.
 *   plan, plan_bytes  from dsatopk_plan, or NULL / 0. Its exchange areas are
 *                     written during the call and left zeroed.
 *   out               int32 [num_rows, k], written (all of it).
 *
 * Device-side preconditions (not checkable without reading device memory,
 * so not checked): 0 <= row_starts[b]; row_starts[b] + seq_len_b <=
 * score_stride; seq_len_b <= 131072; page_table_stride >= ceil(seq_len_b /
 * page_size); every emitted value < 2^31. NaN scores are outside the
 * contract (the selection stays inside the window, but which NaNs are
 * picked is unspecified).
 *
 * Errors: DSATOPK_ERR_INVALID_ARG, DSATOPK_ERR_ALIGNMENT,
 * DSATOPK_ERR_PLAN_TOO_SMALL, DSATOPK_ERR_HIP. num_rows == 0 is a no-op.
 */
int dsatopk_paged(const float* scores, int64_t score_stride, const int32_t* seq_lens,
                  const int32_t* row_starts, const int32_t* page_table,
                  int64_t page_table_stride, int32_t page_size, int32_t num_rows, int32_t k,
                  void* plan, size_t plan_bytes, int32_t* out, void* stream);

/*
 * dsatopk_paged_packed - dsatopk_paged for packed rows, with raw positions
 * beside the paged ones.
 *
 * Packed rows: query rows of one request share that request's page-table
 * row, while their score windows sit at batch-wide columns of the score
 * buffer (sglang/FlashInfer packed PAGED digest, "fix(dsa): use FlashInfer
 * fused top-k for packed PAGED rows": the page table's start for a row is
 * its score window start minus the request's KV start, and a row-to-batch
 * map picks the table row). Raw positions: the transform's optional raw
 * index output (PR #26788 digest, out_raw_indices).
 *
 * Arguments as for dsatopk_paged, plus:
 *   table_rows    int32 [num_rows] (device) or NULL: row b reads page-table
 *                 row table_rows[b] (row b when NULL). The page table may
 *                 then hold fewer rows than num_rows.
 *   table_starts  int32 [num_rows] (device) or NULL: window position j of
 *                 row b is table position table_starts[b] + j (j when
 *                 NULL); out = table[q / page_size] * page_size +
 *                 q % page_size with q that table position.
 *   out_raw       int32 [num_rows, k] or NULL: when given, also written
 *                 (all of it) with the selected window positions j, slot
 *                 for slot with out, and -1 where out holds -1.
 *
 * With table_rows, table_starts and out_raw all NULL this is dsatopk_paged.
 * Device-side preconditions (not checked): table_rows[b] names a row of the
 * page table; 0 <= table_starts[b]; the row's table positions
 * table_starts[b] .. table_starts[b] + seq_len_b - 1 lie inside that row
 * (page_table_stride >= ceil((table_starts[b] + seq_len_b) / page_size)).
 *
 * Errors: as dsatopk_paged.
 */
int dsatopk_paged_packed(const float* scores, int64_t score_stride, const int32_t* seq_lens,
                         const int32_t* row_starts, const int32_t* page_table,
                         int64_t page_table_stride, int32_t page_size,
                         const int32_t* table_rows, const int32_t* table_starts,
                         int32_t num_rows, int32_t k, void* plan, size_t plan_bytes,
                         int32_t* out, int32_t* out_raw, void* stream);

/*
 * dsatopk_ragged - top-k with the RAGGED emit: out = j + out_offsets[b].
 *
 * Arguments as for dsatopk_paged, with out_offsets int32 [num_rows]
 * (device) in place of the page table. With out_offsets == row_starts the
 * outputs are absolute columns of the score row (PR #35175 digest,
 * "Impact": the output is then the token's position in the flattened KV).
 *
 * Errors: as dsatopk_paged.
 */
int dsatopk_ragged(const float* scores, int64_t score_stride, const int32_t* seq_lens,
                   const int32_t* row_starts, const int32_t* out_offsets, int32_t num_rows,
                   int32_t k, void* plan, size_t plan_bytes, int32_t* out, void* stream);

/* Largest batch of dsatopk_paged_noalloc (its plan fits 16 MiB). */
#define DSATOPK_NOALLOC_MAX_ROWS 262144

/*
 * dsatopk_paged_noalloc - dsatopk_paged with its plan in the library's own
 * static device memory, for callers that cannot allocate (code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc).
 *
 * Arguments as for dsatopk_paged, without the plan: each call builds the
 * batch's plan (dsatopk_plan) in a 16 MiB device array of the library, then
 * runs the PAGED transform with it. Nothing is allocated or freed, by this
 * call or by anything it calls; the caller passes the inputs and out.
 *
 * The array is one per GPU, held by every GPU the library runs on until the
 * process ends, and shared by every call on that GPU: calls that overlap on
 * one GPU (several streams or host threads at once) race on it and must be
 * ordered by the caller. Each call writes the parts of the plan that must
 * start at zero itself. The first call on a device looks the array's
 * address up (hipGetSymbolAddress) with that device current; later calls
 * reuse it.
 *
 * Errors: DSATOPK_ERR_TOO_LARGE (num_rows > DSATOPK_NOALLOC_MAX_ROWS,
 * returned before any HIP call), then as dsatopk_paged. num_rows == 0 is a
 * no-op.
 */
int dsatopk_paged_noalloc(const float* scores, int64_t score_stride, const int32_t* seq_lens,
                          const int32_t* row_starts, const int32_t* page_table,
                          int64_t page_table_stride, int32_t page_size, int32_t num_rows,
                          int32_t k, int32_t* out, void* stream);

/* ------------------------------------------------------------------------
 * The serving operators around the selection: page maps, cache writes, indexer
 * scores and latent attention. The conventions above hold for them too (device
 * pointers, asynchronous, no allocation, only kernel launches). Strides are
 * in elements; a tensor's last dimension is contiguous. Every call reads
 * inputs at its stated bounds only: page numbers and slots outside a cache
 * are treated as absent.
 * ------------------------------------------------------------------------ */

/*
 * dsatopk_page_maps - the pages, cache slots and top-k row arguments of a
 * serving step, from its request lengths.
 *
 *   seq_lens      int32 [num_requests]: tokens of each request after the
 *                 step; negative values are read as 0.
 *   new_lens      int32 [num_requests]: those of them that the step adds,
 *                 clamped to [0, seq_len]. NULL: min(1, seq_len).
 *   page_table    int32 [num_requests, page_table_width], rows
 *                 page_table_stride apart. Request r's entries below
 *                 ceil((seq_len - new_len) / page_size) are the pages that
 *                 it holds. The following ones, up to ceil(seq_len /
 *                 page_size), are WRITTEN with pages of the free list: the
 *                 list's pages go to the requests in order, each request's
 *                 in order.
 *   page_size     power of two in [1, 2^20].
 *   free_pages    int32 [num_free].
 *   num_tokens    rows of the outputs below, at most 2^30. A step of fewer tokens leaves
 *                 empty rows behind them; tokens past num_tokens get neither
 *                 a row nor a page.
 *
 * Written, all of them, tokens of request 0 first, each request's in order:
 *   token_starts  int32 [num_requests + 1]: first token of each request.
 *   slots         int32 [num_tokens]: page * page_size + offset, where the
 *                 token's cache entry goes; -1 for an empty row, a page
 *                 past the table's width, one that the free list did not have
 *                 (its table entry is then -1), or a slot past 2^31 - 1.
 *   table_rows    int32 [num_tokens]: the token's request (0 for empty rows).
 *   row_lens      int32 [num_tokens]: the token's position + 1, which is its
 *                 causal window (0 for empty rows). With table_rows these
 *                 are the row arguments of dsatopk_paged_packed,
 *                 dsatopk_scores_paged and dsatopk_attend_paged.
 *   counts        int32 [2]: tokens of the step, pages that they open. More
 *                 tokens than num_tokens, or more pages than num_free: the
 *                 step did not fit.
 *
 * Device-side precondition: the step's tokens and pages, over all requests,
 * are below 2^31.
 * Errors: DSATOPK_ERR_INVALID_ARG, DSATOPK_ERR_HIP.
 */
int dsatopk_page_maps(const int32_t* seq_lens, const int32_t* new_lens, int32_t num_requests,
                      int32_t* page_table, int64_t page_table_stride, int32_t page_table_width,
                      int32_t page_size, const int32_t* free_pages, int32_t num_free,
                      int32_t num_tokens, int32_t* token_starts, int32_t* slots,
                      int32_t* table_rows, int32_t* row_lens, int32_t* counts, void* stream);

/*
 * dsatopk_append_latent - a step's new latent vectors into the paged cache,
 * their rotary part turned by their positions, and the queries' rotary parts
 * with them:
 *
 *   y[t][0 : latent_dim] = x[t] * weight / sqrt(mean(x[t]^2) + eps)  (over the
 *                          latent part; weight NULL: as it is)
 *   y[t][latent_dim :]   = the pairs (a, b) of x[t][latent_dim :], each as
 *                          (a cos - b sin, a sin + b cos)
 *
 * with the cosines and sines of position row_lens[t] - 1. Slots and windows
 * are dsatopk_page_maps' slots and row_lens.
 *
 *   latent        type [num_tokens, latent_dim + rope_dim], rows latent_stride
 *                 apart.
 *   slots         int32 [num_tokens]: page * page_size + offset, none twice (a
 *                 slot of two tokens holds parts of either).
 *   row_lens      int32 [num_tokens]: the token's position + 1.
 *                 A token whose slot is outside the cache, or whose position
 *                 is outside [0, num_positions), is not cached; without a
 *                 position its rotary parts are not turned.
 *   num_tokens    at most 2^30.
 *   cos_sin       float [num_positions, rope_dim], rows cos_sin_stride apart:
 *                 a position's rope_dim / 2 cosines, then as many sines.
 *   interleaved   pair i is elements 2i and 2i + 1 of the rotary part if not
 *                 0, i and i + rope_dim / 2 if 0.
 *   weight        float [latent_dim] or NULL; eps finite, not negative.
 *   type          DSATOPK_BF16 or DSATOPK_FP16.
 *   latent_dim    256 or 512; rope_dim 64.
 *   cache         type [num_pages, page_size, latent_dim + rope_dim], strides
 *                 page_stride, token_stride, as dsatopk_attend_paged reads it.
 *   out           type [num_tokens, latent_dim + rope_dim] or NULL: also
 *                 receives y, of every token (for a prompt's keys and values).
 *                 May be latent itself (with its stride), and must not overlap
 *                 it otherwise.
 *   q_rope        type [num_tokens, num_heads, rope_dim], the rotary parts of
 *                 the queries, strides q_row_stride, q_head_stride;
 *   q_out         type, of the same shape, receives them turned. May be q_rope
 *                 itself (with its strides), and must not overlap it otherwise.
 *   num_heads     0 (no queries: q_rope and q_out are not looked at) .. 1024.
 *
 * Computed in fp32 and rounded once. Errors: DSATOPK_ERR_INVALID_ARG,
 * DSATOPK_ERR_ALIGNMENT (a pointer not 16-byte aligned, a stride no multiple
 * of 16 bytes), DSATOPK_ERR_HIP. num_tokens == 0 is a no-op.
 */
int dsatopk_append_latent(const void* latent, int64_t latent_stride, const int32_t* slots,
                          const int32_t* row_lens, int32_t num_tokens, const float* cos_sin,
                          int64_t cos_sin_stride, int32_t num_positions, int32_t interleaved,
                          const float* weight, float eps, int32_t type, int32_t latent_dim,
                          int32_t rope_dim, void* cache, int64_t num_pages, int64_t page_stride,
                          int64_t token_stride, int32_t page_size, void* out, int64_t out_stride,
                          const void* q_rope, int64_t q_row_stride, int64_t q_head_stride,
                          void* q_out, int64_t q_out_row_stride, int64_t q_out_head_stride,
                          int32_t num_heads, void* stream);

/*
 * dsatopk_append_index - a step's new indexer keys into their cache, as
 * dsatopk_scores_paged reads it, and the indexer's queries made ready with
 * them:
 *
 *   y = (x - mean x) / sqrt(var x + eps) * weight + bias   (keys only; weight
 *       and bias NULL: as it is), then the first rope_dim elements turned as
 *       by dsatopk_append_latent.
 *   index_type = type:         y, rounded.
 *   index_type = DSATOPK_FP8:  s = max |y| / 448 (of at least 2^-100), and
 *       y / s, taken as y * (448 / max |y|), rounded to e4m3. A key's s goes to
 *       its place of key_scales; a query's into its head's weight, weights_out =
 *       weights * s.
 *
 *   keys          type [num_tokens, head_dim], rows key_stride apart.
 *   slots, row_lens, num_tokens, cos_sin, num_positions, interleaved
 *                 as for dsatopk_append_latent; rope_dim 64.
 *   weight, bias  float [head_dim], both or neither.
 *   type          DSATOPK_BF16 or DSATOPK_FP16 (keys and q).
 *   head_dim      64 or 128.
 *   index_keys    index_type [num_pages, page_size, head_dim], strides
 *                 page_stride, token_stride.
 *   key_scales    float [num_pages, page_size], pages scale_page_stride apart
 *                 (DSATOPK_FP8 only).
 *   q             type [num_tokens, num_heads, head_dim];
 *   q_out         index_type, of the same shape. With 16 bits it may be q
 *                 itself (with its strides), and must not overlap it otherwise.
 *   weights       float [num_tokens, num_heads], rows weight_stride apart;
 *   weights_out   the same, rows weight_out_stride apart, may be weights itself
 *                 (both DSATOPK_FP8 only).
 *   num_heads     0 (no queries) .. 128.
 *
 * What becomes 8 bits has to be finite. Computed in fp32 and rounded once.
 * Errors: DSATOPK_ERR_INVALID_ARG, DSATOPK_ERR_ALIGNMENT (a pointer not 16-byte
 * aligned, key_scales and weights not 4-byte; a stride no multiple of 16
 * bytes), DSATOPK_ERR_HIP. num_tokens == 0 is a no-op.
 */
int dsatopk_append_index(const void* keys, int64_t key_stride, const int32_t* slots,
                         const int32_t* row_lens, int32_t num_tokens, const float* cos_sin,
                         int64_t cos_sin_stride, int32_t num_positions, int32_t rope_dim,
                         int32_t interleaved, const float* weight, const float* bias, float eps,
                         int32_t type, int32_t head_dim, void* index_keys, int32_t index_type,
                         int64_t num_pages, int64_t page_stride, int64_t token_stride,
                         int32_t page_size, float* key_scales, int64_t scale_page_stride,
                         const void* q, int64_t q_row_stride, int64_t q_head_stride, void* q_out,
                         int64_t q_out_row_stride, int64_t q_out_head_stride, const float* weights,
                         int64_t weight_stride, float* weights_out, int64_t weight_out_stride,
                         int32_t num_heads, void* stream);

/*
 * dsatopk_scores_paged - the indexer's scores over a paged key cache:
 *
 *   out[b, j] = key_scale[j] * sum_h weights[b, h] * max(0, q[b, h] . key[j])
 *
 * for j in [0, min(seq_lens[b], columns, page_table_width * page_size)),
 * with key[j] the key at page_table[table_rows[b]][j / page_size], offset
 * j % page_size. Other columns of out are not written.
 *
 *   q             type [num_rows, num_heads, head_dim], strides
 *                 q_row_stride, q_head_stride.
 *   weights       float [num_rows, num_heads], rows weight_stride apart.
 *   keys          type [num_pages, page_size, head_dim], strides
 *                 key_page_stride, key_token_stride.
 *   key_scales    float [num_pages, page_size], pages scale_page_stride
 *                 apart, or NULL (ones).
 *   type          DSATOPK_BF16, DSATOPK_FP16 or DSATOPK_FP8 (q and keys).
 *   num_heads     1 .. 128; head_dim 64 or 128.
 *   seq_lens      int32 [num_rows]; negative values are read as 0.
 *   table_rows    int32 [num_rows] or NULL (row b reads table row b).
 *   out           float [num_rows, >= columns], rows out_stride apart; a
 *                 top-k's score buffer (for it: 16-byte aligned, out_stride
 *                 a multiple of 4).
 *   columns       at most 2^30. The work is shared out by columns (and the
 *                 table's positions, if fewer), not by seq_lens: a call on a
 *                 table or buffer much wider than its longest row is slower
 *                 than on their first columns.
 *
 * A page outside [0, num_pages) reads as keys of score 0. Products are
 * exact, sums are fp32.
 * Errors: DSATOPK_ERR_INVALID_ARG, DSATOPK_ERR_ALIGNMENT (q or keys not
 * 16-byte aligned, or one of their strides no multiple of 16 bytes),
 * DSATOPK_ERR_HIP. num_rows == 0 is a no-op.
 */
int dsatopk_scores_paged(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                         const float* weights, int64_t weight_stride, const void* keys,
                         int64_t num_pages, int64_t key_page_stride, int64_t key_token_stride,
                         const float* key_scales, int64_t scale_page_stride, int32_t type,
                         int32_t num_heads, int32_t head_dim, const int32_t* seq_lens,
                         const int32_t* page_table, int64_t page_table_stride,
                         int32_t page_table_width, int32_t page_size, const int32_t* table_rows,
                         int32_t num_rows, float* out, int64_t out_stride, int64_t columns,
                         void* stream);

/*
 * dsatopk_scores_ragged - the same over flattened keys [num_keys, head_dim]
 * (rows key_stride apart; key_scales float [num_keys] or NULL): out[b, c] for
 * the columns c of row b's window [row_starts[b], row_starts[b] +
 * seq_lens[b]), as dsatopk_ragged reads them, cut at columns and num_keys.
 */
int dsatopk_scores_ragged(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                          const float* weights, int64_t weight_stride, const void* keys,
                          int64_t num_keys, int64_t key_stride, const float* key_scales,
                          int32_t type, int32_t num_heads, int32_t head_dim,
                          const int32_t* seq_lens, const int32_t* row_starts, int32_t num_rows,
                          float* out, int64_t out_stride, int64_t columns, void* stream);

/*
 * dsatopk_attend_selected, dsatopk_attend_paged - latent attention in its
 * absorbed form: all heads of a query row read one cached vector per token,
 *
 *   s[b, h, j] = scale * sum over latent_dim + rope_dim of q[b, h] * c[j]
 *   out[b, h]  = sum_j softmax_j(s[b, h, j]) * c[j][0 : latent_dim]
 *   lse[b, h]  = log(sum_j exp(s[b, h, j]))        (natural logarithm)
 *
 * over the tokens j that row b reads:
 *   selected   the slots of row b of `slots` (page * page_size + offset, as
 *              dsatopk_paged and dsatopk_paged_packed emit them; in any
 *              order; slots outside the cache, -1 among them, are skipped);
 *   paged      positions 0 .. min(seq_lens[b], page_table_width * page_size)
 *              - 1 of page table row table_rows[b] (row b when NULL); tokens
 *              of a page outside the cache are skipped.
 * A row that reads no token gets zeros and lse -inf.
 *
 *   q             type [num_rows, num_heads, latent_dim + rope_dim], strides
 *                 q_row_stride, q_head_stride.
 *   cache         type [num_pages, page_size, latent_dim + rope_dim], strides
 *                 page_stride, token_stride; latent part first.
 *   page_size     power of two in [1, 2^20].
 *   type          DSATOPK_BF16 or DSATOPK_FP16.
 *   num_heads     1 .. 1024; latent_dim 256 or 512; rope_dim 64.
 *   scale         finite and above 0.
 *   slots         int32 [num_rows, k], rows slot_stride apart.
 *   max_seq_len   an upper bound on seq_lens, at most 2^31 - 65 (rows of a
 *                 larger table are cut there). It sets how the tokens are
 *                 split over workgroups (and the workspace's size); longer
 *                 rows are read whole all the same.
 *   out           type [num_rows, num_heads, latent_dim], contiguous.
 *   lse           float [num_rows, num_heads] or NULL.
 *   workspace     at least dsatopk_attend_bytes(num_rows, num_heads,
 *                 latent_dim, k or max_seq_len) bytes, 16-byte aligned
 *                 (NULL where that is 0). Calls that overlap must not share
 *                 one.
 *
 * Scores, softmax and sums are fp32; the softmax's weights are rounded to
 * `type` before the second product: off by at most half a step, for
 * DSATOPK_FP16 at least 2^-35 of the row's largest weight. The order of the
 * sums is fixed: the same inputs give the same bits.
 *
 * Errors: DSATOPK_ERR_INVALID_ARG, DSATOPK_ERR_ALIGNMENT (q, cache or
 * workspace not 16-byte aligned, out not 8-byte aligned, a stride of q or
 * cache no multiple of 8 elements), DSATOPK_ERR_WORKSPACE_TOO_SMALL,
 * DSATOPK_ERR_HIP. num_rows == 0 is a no-op.
 */
size_t dsatopk_attend_bytes(int32_t num_rows, int32_t num_heads, int32_t latent_dim,
                            int64_t max_tokens);

int dsatopk_attend_selected(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                            const void* cache, int64_t num_pages, int64_t page_stride,
                            int64_t token_stride, int32_t page_size, int32_t type,
                            int32_t num_heads, int32_t latent_dim, int32_t rope_dim, float scale,
                            const int32_t* slots, int64_t slot_stride, int32_t k,
                            int32_t num_rows, void* out, float* lse, void* workspace,
                            size_t workspace_bytes, void* stream);

int dsatopk_attend_paged(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                         const void* cache, int64_t num_pages, int64_t page_stride,
                         int64_t token_stride, int32_t page_size, int32_t type, int32_t num_heads,
                         int32_t latent_dim, int32_t rope_dim, float scale,
                         const int32_t* seq_lens, const int32_t* page_table,
                         int64_t page_table_stride, int32_t page_table_width,
                         const int32_t* table_rows, int64_t max_seq_len, int32_t num_rows,
                         void* out, float* lse, void* workspace, size_t workspace_bytes,
                         void* stream);

/*
 * dsatopk_attend_shared - dsatopk_attend_paged for rows in groups whose first
 * tokens are the same cached ones (requests behind one prompt, samples of one
 * context, drafted tokens of one request): these are read once for all rows of
 * a group. It pays where groups are large and share much; rows by themselves,
 * and groups of less than about 300000 rows times shared tokens (16 heads), are
 * faster in dsatopk_attend_paged, by 4 to 10 us a call.
 *
 *   group_starts  int32 [num_groups + 1], rising: group g is rows
 *                 group_starts[g] .. group_starts[g + 1] - 1. The first entry is
 *                 taken as 0 and the last as num_rows, so that every row is in a
 *                 group. A group may be a single row, or empty.
 *                 (Where they do not rise, results of the rows concerned mean
 *                 nothing; no memory but the arguments' is touched.)
 *   shared_lens   int32 [num_groups]: positions 0 .. shared_lens[g] - 1 of a
 *                 group's rows are those of its first row's page table (what
 *                 other rows' tables have there is not looked at). Row b reads
 *                 the first min(seq_lens[b], shared_lens[g]) there, and the
 *                 following ones, up to seq_lens[b], in its own table.
 *                 Negative values are read as 0, those past the table are cut.
 *   max_shared_len, max_own_len  upper bounds on shared_lens and on the tokens
 *                 that a row reads by itself, at most 2^31 - 65. They set how
 *                 many workgroups are started at most (and the workspace's
 *                 size); longer ones are read whole all the same, but a bound of 0
 *                 is taken at its word: with max_shared_len 0 rows read all
 *                 of their tokens by themselves, with max_own_len 0 (and the
 *                 other not 0) none past their group's shared ones.
 *   workspace     at least dsatopk_shared_bytes(num_rows, num_heads,
 *                 latent_dim, num_groups, max_shared_len, max_own_len) bytes,
 *                 16-byte aligned. Calls that overlap must not share one.
 *
 * The other arguments are those of dsatopk_attend_paged, as are the rounding
 * and the errors. A shared position that some but not all rows of its group see
 * has to hold finite values (its weight is 0 in the others, which infinities
 * and NaN turn into NaN; rows that see nothing at all get zeros all the same);
 * what no row sees may hold anything. num_groups 0 is refused unless num_rows
 * is 0.
 */
size_t dsatopk_shared_bytes(int32_t num_rows, int32_t num_heads, int32_t latent_dim,
                            int32_t num_groups, int64_t max_shared_len, int64_t max_own_len);

int dsatopk_attend_shared(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                          const void* cache, int64_t num_pages, int64_t page_stride,
                          int64_t token_stride, int32_t page_size, int32_t type, int32_t num_heads,
                          int32_t latent_dim, int32_t rope_dim, float scale,
                          const int32_t* seq_lens, const int32_t* page_table,
                          int64_t page_table_stride, int32_t page_table_width,
                          const int32_t* table_rows, const int32_t* group_starts,
                          const int32_t* shared_lens, int32_t num_groups, int64_t max_shared_len,
                          int64_t max_own_len, int32_t num_rows, void* out, float* lse,
                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * dsatopk_attend_expanded - latent attention in its expanded form, for
 * prompts: keys and values of each head (the latent vectors' projections),
 * one rotary key for all heads,
 *
 *   s[i, h, j] = scale * (q[i, h][0 : nope_dim] . k[j, h] + q[i, h][nope_dim :] . k_rope[j])
 *   out[i, h]  = sum_j softmax_j(s[i, h, j]) * v[j, h]
 *   lse[i, h]  = log(sum_j exp(s[i, h, j]))
 *
 * over a ragged batch: request r has the queries q_starts[r] .. q_starts[r +
 * 1] - 1 and the keys k_starts[r] .. k_starts[r + 1] - 1. With `causal`,
 * query i of a request's n sees its first (keys - n + i + 1) keys: the
 * queries are the request's last tokens. A query that sees no key gets zeros
 * and lse -inf.
 *
 *   q             type [num_queries, num_heads, nope_dim + rope_dim]
 *   k             type [num_keys, num_heads, nope_dim]
 *   v             type [num_keys, num_heads, value_dim]
 *   k_rope        type [num_keys, rope_dim]
 *                 (each with its row and head strides, those of keys and
 *                 values at most 2^27; k and v may be parts of one tensor)
 *   type          DSATOPK_BF16 or DSATOPK_FP16.
 *   num_heads     1 .. 1024; nope_dim 128, rope_dim 64, value_dim 128.
 *   scale         finite and above 0.
 *   q_starts, k_starts  int32 [num_requests + 1], rising; parts past
 *                 num_queries and num_keys are cut off.
 *   max_queries   an upper bound on a request's queries (rows past it are
 *                 not computed).
 *   out           type [num_queries, num_heads, value_dim], contiguous. Rows
 *                 of no request are not written.
 *   lse           float [num_queries, num_heads] or NULL.
 *   workspace     at least dsatopk_expanded_bytes(num_requests, num_heads,
 *                 num_queries, num_keys, max_queries) bytes, 16-byte aligned
 *                 (NULL where that is 0: batches that fill the card are not
 *                 split). Calls that overlap must not share one.
 *
 * Values must be finite, also those of keys that causality hides from some
 * queries (their weight is 0, which infinities and NaN turn into NaN). Hidden
 * keys may hold anything. Rounding as for dsatopk_attend_selected.
 *
 * Errors: DSATOPK_ERR_INVALID_ARG, DSATOPK_ERR_ALIGNMENT (an input not
 * 16-byte aligned or a stride no multiple of 8 elements; out not 8-byte
 * aligned), DSATOPK_ERR_WORKSPACE_TOO_SMALL, DSATOPK_ERR_HIP. No queries: a
 * no-op.
 */
size_t dsatopk_expanded_bytes(int32_t num_requests, int32_t num_heads, int32_t num_queries,
                              int32_t num_keys, int32_t max_queries);

int dsatopk_attend_expanded(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                            const void* k, int64_t k_row_stride, int64_t k_head_stride,
                            const void* v, int64_t v_row_stride, int64_t v_head_stride,
                            const void* k_rope, int64_t rope_row_stride, int32_t type,
                            int32_t num_heads, int32_t nope_dim, int32_t rope_dim,
                            int32_t value_dim, float scale, int32_t causal,
                            const int32_t* q_starts, const int32_t* k_starts,
                            int32_t num_requests, int32_t num_queries, int32_t num_keys,
                            int32_t max_queries, void* out, float* lse, void* workspace,
                            size_t workspace_bytes, void* stream);

/*
 * dsatopk_attend_expanded_shared - dsatopk_attend_expanded for prompts behind
 * keys that several of them share, which are there once: request r has the
 * keys shared_starts[r] .. shared_starts[r] + shared_lens[r] - 1, all of which
 * every query of it sees, and behind them its own, k_starts[r] .. k_starts[r +
 * 1] - 1, which it sees as in dsatopk_attend_expanded.
 *
 *   shared_starts, shared_lens  int32 [num_requests], negative values read as
 *                 0, lengths cut at num_keys. Neighbouring requests with the
 *                 same two values share the work on these keys, too; equal
 *                 values further apart do not. Length 0: none are shared.
 *   num_queries, num_keys  at most 2^30.
 *   max_keys      an upper bound on a request's keys, shared and own; it sets how
 *                 few rows of many keys are split (and the workspace's size),
 *                 and nothing else.
 *   workspace     at least dsatopk_expanded_shared_bytes(num_heads,
 *                 num_queries, max_keys) bytes, 16-byte aligned (NULL where
 *                 that is 0).
 *
 * The other arguments, the rounding and the errors are those of
 * dsatopk_attend_expanded, but there is no max_queries: all rows are
 * computed. Values must be finite here, too, those of a request's own keys
 * and of the shared ones. Other requests' keys may hold anything: where queries
 * of several requests stand in a tile (of up to 256) and a result is not
 * finite, the tile is computed once more, each query from its own keys only.
 */
size_t dsatopk_expanded_shared_bytes(int32_t num_heads, int32_t num_queries, int32_t max_keys);

int dsatopk_attend_expanded_shared(
    const void* q, int64_t q_row_stride, int64_t q_head_stride, const void* k,
    int64_t k_row_stride, int64_t k_head_stride, const void* v, int64_t v_row_stride,
    int64_t v_head_stride, const void* k_rope, int64_t rope_row_stride, int32_t type,
    int32_t num_heads, int32_t nope_dim, int32_t rope_dim, int32_t value_dim, float scale,
    int32_t causal, const int32_t* q_starts, const int32_t* k_starts, const int32_t* shared_starts,
    const int32_t* shared_lens, int32_t num_requests, int32_t num_queries, int32_t num_keys,
    int32_t max_keys, void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DSATOPK_H_ */
