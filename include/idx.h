/*
 * idx.h - C ABI of the GB300 decode indexer library (libidx.so).
 *
 * The indexer of the sglang PR 48224 page (sgl-amd-mono #86): every decode row is
 * scored against every key its request has cached, and the row's exact top-2048
 * is selected (section Motivation, first paragraph).  It reads an FP8 E4M3 or
 * bf16 paged key cache (section Accuracy Tests), leaves out positions from a
 * row's bound on (section Modifications, commit 2), and selects by radix digits whose first digit is radix_key >> 26
 * over 64 bins (section Modifications, commit 4).  The score of the key at
 * logical position t for row r is
 *
 *     score[r][t] = sum_{h<64} w[r][h] * ReLU(scale_t * <q[r][h][:], k_t>)
 *
 * with 64 heads of 128 dimensions; scale_t is the key's fp32 scale (E4M3 cache)
 * or 1 (bf16 cache).
 *
 * Conventions for every call below:
 *   - Pointers named "device" are caller-owned device memory; the library never
 *     allocates, frees or keeps them.  Pointers named "host" are host memory.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Every call
 *     is asynchronous on it unless its comment says otherwise.
 *   - Arguments are validated on the host before anything is launched; a bad
 *     argument returns IDX_EINVAL (or IDX_EUNSUPPORTED for a shape the library
 *     does not handle) and launches nothing.  A failed launch returns IDX_ECUDA.
 *   - Errors found on the device (a page id outside [0, P), a row bound above
 *     max_bound or pt_stride * 64, a request id outside [0, Q), a pipeline wait
 *     that ran out of time) never trap: the kernel records them in a status word
 *     inside the workspace, clamps the bound or skips the page or the row, and
 *     finishes; read the word with idx_last_device_status().
 *   - Key positions are logical positions within the row's request: position t
 *     lives in physical page page_table[req * pt_stride + t / 64], slot t % 64.
 *   - Host threads: any call may be made from several host threads at once, on
 *     the same or different devices, as long as concurrent calls use different
 *     workspaces (the library's one-time per-device setup is serialised inside
 *     it).  idx_topk_noalloc is the exception: its scratch is one per device.
 *     idx_debug_set and idx_profile_events change process-wide state that the
 *     next call from any thread picks up.
 */
#ifndef IDX_H
#define IDX_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define IDX_HEADS 64      /* query heads per row */
#define IDX_DIM 128       /* dimensions per head and per key */
#define IDX_PAGE 64       /* tokens per cache page */
#define IDX_MAX_K 2048    /* largest top-k */
#define IDX_MAX_ROWS 65535

typedef enum {
    IDX_OK = 0,
    IDX_EINVAL = 1,       /* bad argument (null pointer, negative size, small workspace ...) */
    IDX_EUNSUPPORTED = 2, /* valid but outside what this build handles */
    IDX_ECUDA = 3,        /* a CUDA runtime call or launch failed */
    IDX_ETIMEOUT = 4,     /* a device-side wait ran out of time (device status only) */
    IDX_EDEVICE = 5       /* bad data seen on the device: page id, bound or request id out of range */
} idx_status;

typedef enum {
    IDX_KV_E4M3 = 0,      /* keys are OCP E4M3 bytes with one fp32 scale per token */
    IDX_KV_BF16 = 1       /* keys are bf16, scale 1 */
} idx_kv_dtype;

/* One indexer problem.  All array pointers are device memory owned by the caller. */
typedef struct {
    const void *q;             /* bf16 [R][64][128], contiguous, 16-byte aligned */
    const float *w;            /* fp32 [R][64], contiguous, 16-byte aligned */
    const void *k_cache;       /* [P][64][128]: E4M3 bytes or bf16, contiguous, 16-byte aligned */
    const float *k_scale;      /* fp32 [P][64] for IDX_KV_E4M3, 16-byte aligned, every value >= 0;
                                  must be NULL for IDX_KV_BF16 */
    const int32_t *page_table; /* int32 [Q][pt_stride]: page ids in [0, P) for every page a row reads */
    const int32_t *row_req;    /* int32 [R]: request of each row, in [0, Q) */
    const int32_t *row_bound;  /* int32 [R]: row r scores positions 0 .. row_bound[r]-1 */
    int32_t R;                 /* rows, 1 .. IDX_MAX_ROWS */
    int32_t Q;                 /* requests, >= 1 */
    int64_t P;                 /* pages in the cache, >= 1 */
    int32_t pt_stride;         /* page-table row length, >= 1 */
    int32_t max_bound;         /* host upper bound on every row_bound[r]; sizes scratch, so no
                                  device-to-host read is needed; 0 <= max_bound <= pt_stride*64 */
    int32_t kv_dtype;          /* idx_kv_dtype */
    int32_t rows_hint;         /* host hint, like max_bound: 0 if unknown, else an upper bound on the
                                  rows of any one request in this problem.  1 or 2 (a lone live row,
                                  or a row and its pad row) lets the scan batch 4 / rows tiles into
                                  one accumulator so that every epilogue warp has work.  The result
                                  never depends on it: a hint below the true count only costs
                                  speed.  Negative: IDX_EINVAL. */
} idx_problem;

/* Bytes of device workspace that idx_score / idx_topk / idx_launch need for this
 * problem and top-k (the largest of the three; every call accepts more).  The
 * workspace is caller-owned, needs no initialisation and may be reused by later
 * calls on the same stream; two calls that overlap in time need two workspaces.
 * Returns 0 if the problem is invalid. */
size_t idx_workspace_size(const idx_problem *problem, int32_t K);

/* Scores only (the scan and contraction; section Motivation, first paragraph).
 *   scores  device fp32 [R][ld], ld >= max_bound: scores[r][t] written for t < row_bound[r],
 *           other entries untouched.
 *   hist    device uint32 [R][64] or NULL: when given, hist[r][d] = number of t < row_bound[r]
 *           with radix_key(scores[r][t]) >> 26 == d (the fused first-digit histogram of
 *           section Modifications, commit 4).  radix_key maps the fp32 bits to an unsigned key
 *           that orders like the value, with -0.0 read as +0.0.
 *   ws      device workspace of ws_bytes >= idx_workspace_size(problem, 1). */
idx_status idx_score(const idx_problem *problem, float *scores, int64_t ld, uint32_t *hist,
                     void *ws, size_t ws_bytes, void *stream);

/* Exact top-K of given scores (section Motivation: exact top-2048; section
 * Modifications, commit 4: radix selection with a 64-bin first digit).
 *   scores     device fp32 [R][ld]; only t < row_bound[r] is read; values must not be NaN.
 *   row_bound  device int32 [R]; max_bound (host) >= every row_bound[r], ld >= max_bound.
 *   K          1 .. IDX_MAX_K.
 *   hist       device uint32 [R][64] first-digit histogram of these scores (as idx_score
 *              writes it) or NULL.  Accepted for callers that hold one; this build
 *              counts the finer 12-bit prefix of the radix keys in one pass over the
 *              scores and does not need it.
 *   out_idx    device int32 [R][K]: positions ordered by score descending, then position
 *              ascending; entries past min(K, row_bound[r]) are -1.  Scores compare by value
 *              (-0.0 == +0.0).
 *   ws         device workspace of ws_bytes >= idx_workspace_size() of a problem with these
 *              R and max_bound. */
idx_status idx_topk(const float *scores, int64_t ld, const int32_t *row_bound, int32_t R,
                    int32_t max_bound, int32_t K, const uint32_t *hist, int32_t *out_idx,
                    void *ws, size_t ws_bytes, void *stream);

/* The fused indexer launch: idx_score into workspace scratch, the fused first-digit
 * histogram, then idx_topk; out_idx as for idx_topk. */
idx_status idx_launch(const idx_problem *problem, int32_t K, int32_t *out_idx, void *ws,
                      size_t ws_bytes, void *stream);

/* idx_launch that also returns the selected keys' scores (the first half of a
 * key-sharded indexer: each shard ranks the keys it holds; see idx_merge_topk).
 *   out_score  device fp32 [R][K]: out_score[r][j] is the score of position
 *              out_idx[r][j] (-0.0 comes back as +0.0); -inf where out_idx is -1.
 * Other arguments and errors as for idx_launch; a NULL out_score is IDX_EINVAL. */
idx_status idx_launch_scored(const idx_problem *problem, int32_t K, int32_t *out_idx, float *out_score,
                             void *ws, size_t ws_bytes, void *stream);

/* Exact top-K of the union of S ranked parts: the merge of a key-sharded indexer.
 * The "Release Test Suite - GLM-5.2-EXL3" page (section Config change) runs decode
 * context parallelism with a top-k owner merge: every GPU ranks the keys of its
 * shard of the cache and one owner merges the lists.  The union of the shards'
 * top-K lists holds the global top-K, so the merge reproduces the unsharded
 * selection exactly.
 *   part_idx     device int32 [S][R][Kin]: part s's positions in its own numbering,
 *                ordered by score descending then position ascending, -1 padded
 *                (as idx_launch_scored writes them).
 *   part_score   device fp32 [S][R][Kin]: their scores (no NaN).
 *   part_offset  HOST int32 [S], >= 0: added to part s's positions; the parts must
 *                cover disjoint position ranges (a position of the request is in
 *                exactly one part).
 *   S            1 .. IDX_MERGE_MAX_PARTS; Kin, K in 1 .. IDX_MAX_K.
 *   out_idx      device int32 [R][K]: the merged positions, same order, -1 padded.
 *   out_score    device fp32 [R][K] or NULL: their scores, -inf where out_idx is -1.
 * Returns IDX_EINVAL for a bad argument and IDX_EUNSUPPORTED for S or R above the
 * limits; launches nothing then.
 * Asynchronous on `stream`; allocates nothing. */
#define IDX_MERGE_MAX_PARTS 8
idx_status idx_merge_topk(const int32_t *part_idx, const float *part_score, const int32_t *part_offset,
                          int32_t S, int32_t R, int32_t Kin, int32_t K, int32_t *out_idx, float *out_score,
                          void *stream);

/* Bytes of device arena idx_launch_host needs: the inputs' device copies, the
 * output and the workspace. */
size_t idx_host_arena_size(const idx_problem *host_problem, int32_t K);

/* idx_launch on HOST inputs.  host_problem's array pointers are host memory (pinned
 * memory makes the copies asynchronous; pageable memory makes them synchronous).
 * A rows_hint of 0 is replaced by the most rows of any request, counted from the
 * host row map.
 * Copies every input into `arena` (device, arena_bytes >= idx_host_arena_size()),
 * runs idx_launch and copies the [R][K] result back into host_out (host).  All
 * copies are issued on `stream`; the caller synchronises the stream before reading
 * host_out. */
idx_status idx_launch_host(const idx_problem *host_problem, int32_t K, int32_t *host_out,
                           void *arena, size_t arena_bytes, void *stream);

/* Synchronises `stream`, then reads and clears the device status word of workspace
 * `ws` (of the last call that used it): IDX_OK, IDX_ETIMEOUT or IDX_EDEVICE, or
 * IDX_ECUDA if the stream reports an error. */
idx_status idx_last_device_status(void *ws, void *stream);

/* Static description of a status code. */
const char *idx_status_string(idx_status status);

/* Library version, major * 10000 + minor * 100 + patch. */
int32_t idx_version(void);

/* Test hooks.  IDX_DEBUG_WAIT_LIMIT_NS sets the time limit of every device-side wait
 * (default 1e9 ns); IDX_DEBUG_STALL_SCORE_MMA > 0 makes the next scoring launch hold
 * back its first accumulator hand-off, so that its waits run out and it reports
 * IDX_ETIMEOUT.  Process-wide; returns the previous value.  Not for production use. */
#define IDX_DEBUG_WAIT_LIMIT_NS 1
#define IDX_DEBUG_STALL_SCORE_MMA 2
int64_t idx_debug_set(int32_t what, int64_t value);

/* Measurement hook.  When `start` and `stop` (cudaEvent_t) are non-NULL, the next
 * idx_score or idx_launch records `start` on its stream just before the scoring
 * kernel and `stop` just after it, so the scoring kernel alone can be timed with
 * cudaEventElapsedTime.  Applies to one call, then clears itself.  Process-wide. */
void idx_profile_events(void *start, void *stop);

/* Writes every row's new key into the paged cache, ahead of idx_launch (the sglang
 * PR 48224 page, section Reviewer notes, "New keys": a key the launch writes is
 * scored for every row of its request in the launch).  Row r's key goes to logical
 * position row_bound[r] - 1 of request row_req[r], so the scan that follows reads it
 * for every row whose bound covers it.
 *   problem  as for idx_launch; problem->k_cache and problem->k_scale are WRITTEN
 *            (device memory the caller owns and may write).
 *   k_new    device bf16 [R][128], 16-byte aligned: each row's new key.
 * E4M3 cache: scale = amax / 448 in fp32 (1 for a zero key) goes to k_scale, and
 * each value divided by it in fp32 goes to the nearest E4M3 code (ties to even),
 * saturating at +-448.  bf16 cache: the values as given.  Rows with bound 0 write
 * nothing; a row whose page id is outside [0, P) writes nothing (idx_launch then
 * reports the page).  Rows of one request must have different bounds (each writes
 * its own position).  Asynchronous on `stream`; allocates nothing. */
idx_status idx_patch_new_keys(const idx_problem *problem, const void *k_new, void *stream);

/* idx_launch with the rows' new keys written first, inside the launch (the same
 * page section, "New keys": a key the launch writes is scored by every row of its
 * request whose bound covers it).  The launch's first kernel writes row r's key
 * at position row_bound[r] - 1 exactly as idx_patch_new_keys does, before the
 * scan reads the cache; the result equals idx_patch_new_keys followed by
 * idx_launch, in one launch sequence instead of two.
 *   problem  as for idx_launch; problem->k_cache and problem->k_scale are WRITTEN.
 *   k_new    device bf16 [R][128], 16-byte aligned (NULL or misaligned: IDX_EINVAL).
 * Other arguments, outputs and errors as for idx_launch; rows of one request must
 * have different bounds. */
idx_status idx_launch_new_keys(const idx_problem *problem, const void *k_new, int32_t K, int32_t *out_idx,
                               void *ws, size_t ws_bytes, void *stream);

/* Top-1 of each row of logits in one launch: the later "draft_topk1_postprocess"
 * commit on the sglang PR 48224 page.  Each split of a row folds its (value,
 * lowest index) into a per-row 64-bit key with an atomic maximum; the split that
 * arrives last writes the row's results and resets the row's state.  Ties go to
 * the lowest index; a NaN reads as -1e30; -0.0 and +0.0 compare equal.
 *   logits     device fp32 [R][ld], columns 0 .. V-1 read; ld >= V >= 1.
 *   out_idx    device int32 [R]: the index of each row's largest value.
 *   out_val    device fp32 [R] or NULL: that value (after the NaN reading; a zero
 *              maximum is written as +0.0).
 *   tokens     device int32 [R][tokens_ld] or NULL: tokens[r * tokens_ld + token_col]
 *              gets out_idx[r] (the draft token column); 0 <= token_col < tokens_ld.
 *   positions  device int32 [R] or NULL: positions[r] += 1.
 *   state      device buffer of state_bytes >= idx_top1_state_size(R), 16-byte
 *              aligned, all zero before its first use; every call leaves it zero
 *              again.  Calls that share a state must not overlap in time.
 * Returns IDX_EINVAL for a bad argument and IDX_EUNSUPPORTED for V > INT32_MAX, in
 * both cases launching nothing. */
size_t idx_top1_state_size(int32_t R);
idx_status idx_top1(const float *logits, int64_t ld, int32_t R, int64_t V, int32_t *out_idx,
                    float *out_val, int32_t *tokens, int64_t tokens_ld, int32_t token_col,
                    int32_t *positions, void *state, size_t state_bytes, void *stream);

/* Exact top-K of given scores with no caller workspace.  The page has no
 * counterpart: this is idx_topk run on scratch that lives in the library itself,
 * a file-scope device array of IDX_NOALLOC_SCRATCH_BYTES (enough for up to
 * IDX_NOALLOC_MAX_ROWS rows at any K up to IDX_MAX_K and any max_bound).  It is
 * for callers that cannot allocate device memory on their decode path: a host
 * program that links only this library and has no device allocator of its own,
 * or a serving loop that reserves all its memory up front because an allocation
 * between steps can synchronise the device or fail under memory pressure.  The
 * call allocates nothing.
 *   scores, ld, row_bound, R, max_bound, K, out_idx: as for idx_topk (no hist).
 *   R > IDX_NOALLOC_MAX_ROWS returns IDX_EUNSUPPORTED and launches nothing; the
 *   other argument checks are those of idx_topk (IDX_EINVAL).
 *   Setup: the first call on a device looks up the scratch's device address
 *   (cudaGetSymbolAddress) and keeps it for later calls; make that first call on
 *   each device before any stream capture begins.  A failed lookup returns
 *   IDX_ECUDA.  The kept address belongs to the device's context as it was at
 *   that first call: after a cudaDeviceReset (or anything else that destroys and
 *   recreates the device's primary context) the process must be restarted before
 *   this call is used on that device again.
 *   Nothing in the scratch has to start at zero: every call clears the selection
 *   state it uses before its kernels read it.
 *   The scratch is one per device and process: two calls whose work can overlap
 *   in time (different streams, or different host threads) race on it, and the
 *   caller must order them (e.g. one stream).  Device-detected errors (a row bound
 *   outside [0, max_bound], clamped as idx_topk does) have no readback here. */
#define IDX_NOALLOC_MAX_ROWS 8
#define IDX_NOALLOC_SCRATCH_BYTES (1280 * 1024)
idx_status idx_topk_noalloc(const float *scores, int64_t ld, const int32_t *row_bound, int32_t R,
                            int32_t max_bound, int32_t K, int32_t *out_idx, void *stream);

/* ---------------------------------------------------------------------------
 * The tree-verify decode step around the indexer: page tables and slot maps for a
 * step's new tokens (idx_tree_tables), their keys and values into the paged cache
 * (idx_write_kv), and the attention of each request's drafted tokens over that
 * cache, whole (idx_tree_attention) or at the positions that idx_launch selected
 * (idx_tree_attention_selected).
 *
 * A step gives request i new_len[i] tokens at logical positions ctx_len[i] ..
 * ctx_len[i] + new_len[i] - 1 of its pages; they are the rows row_start[i] ..
 * row_start[i + 1] - 1 of every per-row array.  In a tree of drafted tokens, token
 * t stands at the storage position ctx_len[i] + t whatever its depth.
 *
 * The state buffer of these calls is device memory, 1024-byte aligned, all zero
 * before its first use.  Its first word is a status word that errors found on the
 * device are or-ed into; idx_last_device_status reads and clears it.  Calls that
 * overlap in time need a state each, and after IDX_ETIMEOUT a state is zeroed anew.
 * Arrays are aligned to their elements at least (IDX_EINVAL otherwise). */
#define IDX_MAX_REQS 4096     /* requests of a step */
#define IDX_MAX_TREE 64       /* drafted tokens of one request (bits of a mask) */

/* Page tables, slot maps and tree masks of a step, from request lengths.
 * Request i holds ceil(ctx_len[i] / 64) pages already and gets the pages that its
 * new tokens need, in request order, from the top of the free stack:
 * free_pages[free_count - 1], free_pages[free_count - 2], ...  A prompt is a
 * request with ctx_len 0. */
typedef struct {
    const int32_t *ctx_len;    /* device int32 [Q]: tokens each request has cached (< 0 reads as 0,
                                  lengths above 2^30 - 64 as that) */
    const int32_t *new_len;    /* device int32 [Q]: new tokens of each request (< 0 reads as 0) */
    const int32_t *parent;     /* device int32 [cap] or NULL (a chain): the parent of row r as a token number
                                  of its request, below the row's own number; -1 for a root */
    const int32_t *free_pages; /* device int32 [free_count]: page ids in [0, P) */
    const int32_t *free_count; /* device int32 [1] */
    int32_t *page_table;       /* device int32 [Q][pt_stride]: held pages are read, new entries written */
    int32_t *row_start;        /* out, device int32 [Q + 1]: exclusive prefix sums of new_len, at most cap
                                  (INT32_MAX where cap is 0) */
    int32_t *free_left;        /* out, device int32 [1]: pages left on the free stack (not free_count itself) */
    int32_t *row_req;          /* out, device int32 [cap]: the row's request */
    int32_t *row_bound;        /* out, device int32 [cap]: its storage position + 1 (idx_patch_new_keys's bound) */
    int32_t *row_pos;          /* out, device int32 [cap]: ctx_len + depth in the tree (the rotary position) */
    int32_t *slot;             /* out, device int32 [cap]: page * 64 + position % 64, or -1 without a page */
    uint64_t *mask;            /* out, device [cap] or NULL: bit u set iff token u is the row's token or one of
                                  its ancestors */
    int64_t P;                 /* pages of the cache, 1 .. INT32_MAX / 64 */
    int32_t Q;                 /* requests, 1 .. IDX_MAX_REQS */
    int32_t pt_stride;         /* page-table row length, >= 1 */
    int32_t cap;               /* rows that the per-row arrays hold, 0 .. INT32_MAX - 3 (0: only tables and
                                  row_start) */
} idx_tree_tables_args;

/* Bytes of state that idx_tree_tables needs. */
size_t idx_tree_tables_state_size(void);

/* One launch.  Rows from row_start[Q] to cap - 1 are padding: request 0, bound 0,
 * position 0, slot -1, mask 0.  Found on the device and recorded as IDX_EDEVICE:
 * fewer free pages than needed or a table row too short (the rows without a page
 * get slot -1, their table entries -1), more new tokens than cap (the rest have no
 * row; for cap 0: more than INT32_MAX), a page id outside [0, P) (slot -1), a parent
 * that is not an earlier token (read as a root), a request of more than IDX_MAX_TREE
 * new tokens with parents or masks asked for (those past the 64th: mask 0, depth
 * counted as in a chain).  IDX_EINVAL for a NULL or bad argument, IDX_EUNSUPPORTED for
 * Q, P or cap above the limits; launches nothing then. */
idx_status idx_tree_tables(const idx_tree_tables_args *args, void *state, size_t state_bytes, void *stream);

/* A paged key/value cache.  Element (page p, token s, head h, dim d) of K and of V
 * is at p * page_stride + s * token_stride + h * head_stride + d elements: any order
 * of tokens and heads, and K and V interleaved in one allocation. */
typedef struct {
    void *k, *v;               /* device, E4M3 bytes or bf16, 16-byte aligned */
    float *k_scale, *v_scale;  /* device fp32 [P][Hkv][64] for E4M3, 16-byte aligned; NULL for bf16 */
    int64_t P;                 /* pages, 1 .. INT32_MAX / 64 */
    int64_t page_stride, token_stride, head_stride;  /* elements; multiples of 16 bytes, positive */
    int32_t Hkv;               /* key/value heads, 1 .. 1024 */
    int32_t D;                 /* dimensions per head: 64 or 128 */
    int32_t kv_dtype;          /* idx_kv_dtype */
} idx_kv_cache;

/* Writes R tokens' keys and values into the cache.
 *   k_new, v_new  device bf16: row r's head h at r * row_stride + h * D elements, 16-byte
 *                 aligned, row_stride >= Hkv * D and a multiple of 8 (a slice of a fused
 *                 projection's output fits).
 *   slot          device int32 [R]: page * 64 + token (idx_tree_tables writes it); a
 *                 slot outside [0, P * 64) writes nothing.  Slots >= 0 must differ.
 * bf16 cache: the values as given.  E4M3 cache: per token and head scale = amax / 448
 * in fp32 (1 for an all-zero vector), each value divided by it in fp32 and rounded to
 * the nearest E4M3 code (ties to even), saturating at +-448.  A NaN is left out of
 * amax and becomes a NaN code (a vector of NaN only: scale 1); an infinity makes the
 * scale infinite, itself a NaN code and the vector's other codes zeros.  R = 0 does
 * nothing.
 * Asynchronous on `stream`; allocates nothing. */
idx_status idx_write_kv(const idx_kv_cache *cache, const void *k_new, const void *v_new, int64_t row_stride,
                        const int32_t *slot, int64_t R, void *stream);

/* The drafted tokens of Q requests and the cache they attend to. */
typedef struct {
    const void *q;             /* device bf16: row r's head h at r * q_row_stride + h * D elements, 16-byte aligned */
    int64_t q_row_stride;      /* elements, >= Hq * D, a multiple of 8 */
    idx_kv_cache cache;        /* read only here */
    const int32_t *page_table; /* device int32 [Q][pt_stride] */
    const int32_t *ctx_len;    /* device int32 [Q] */
    const int32_t *row_start;  /* device int32 [Q + 1]: ascending, within 0 .. R */
    const uint64_t *mask;      /* device [R]: bit u set iff the row sees its request's drafted token u;
                                  NULL: a chain (token t sees 0 .. t) */
    int32_t R;                 /* rows that q and the outputs hold, 1 .. IDX_MAX_ROWS */
    int32_t Q;                 /* requests, 1 .. IDX_MAX_REQS */
    int32_t pt_stride;
    int32_t max_ctx;           /* host upper bound on every ctx_len, 0 .. pt_stride * 64, at most 2^30 */
    int32_t max_new;           /* host upper bound on every request's rows, 1 .. IDX_MAX_TREE */
    int32_t Hq;                /* query heads, a multiple of cache.Hkv; head h reads key/value head h / (Hq / Hkv);
                                  Hq / Hkv at most 128 */
    float scale;               /* of the scores, finite and >= 0 */
} idx_tree_problem;

/* Bytes of state for the attention calls on this problem; sel_k: 0 for
 * idx_tree_attention, the selection's K for idx_tree_attention_selected.  0 if the
 * problem is invalid. */
size_t idx_tree_state_size(const idx_tree_problem *problem, int32_t sel_k);

/* Attention of every drafted token over its request's cached tokens and the drafted
 * tokens that its mask shows (their K and V already in the cache, see idx_write_kv).
 * For row r of request i and head h, with k_j and v_j the cache's values (code times
 * scale) at logical position j,
 *     V(r)  = { j < ctx_len[i] } + { ctx_len[i] + u : u < rows of i, bit u of mask[r] }
 *     s_j   = scale * <q[r][h], k_j>
 *     out   = sum_j exp(s_j) v_j / sum_j exp(s_j),   lse = log sum_j exp(s_j)   over j in V(r);
 * a row that sees nothing, or only scores of -inf, gets zeros and lse -inf.  Masked
 * positions contribute nothing, whatever the cache holds there (NaN and infinities
 * included).
 *   out  device bf16 [R][Hq][D], 16-byte aligned.
 *   lse  device fp32 [R][Hq] or NULL.
 * Rows outside every request are not written.  Sums and softmax statistics are fp32;
 * the probabilities are rounded to bf16 for the product with V (to two bf16 terms in
 * tiles of 64 or 128 positions that are not visible as a whole to every row), which
 * leaves an error nearly as large as the rounding of out to bf16; beside an
 * E4M3 cache q is used as the sum of two E4M3 terms, exact for elements down to 2^-9 of
 * its row's largest and to 2^-17 of that below.  Equal calls give equal bits.
 * The launch is cooperative: its CTAs, at most one per SM, run at the same time.
 * Device-detected (IDX_EDEVICE): a page id outside [0, P) (its tokens are left out),
 * ctx_len outside 0 .. max_ctx, more rows than max_new or positions past the page
 * table (clamped), row_start outside 0 .. R or descending, so many keys over requests that
 * share rows that tiles pass 31 bits (nothing is written).  IDX_ETIMEOUT: a wait ran out.
 * Asynchronous on `stream`; allocates nothing. */
idx_status idx_tree_attention(const idx_tree_problem *problem, void *out, float *lse, void *state,
                              size_t state_bytes, void *stream);

/* The same over selected positions: V(r) = { sel[r][n] : 0 <= sel[r][n] < ctx_len[i] } +
 * { ctx_len[i] + u : bit u of mask[r] }.
 *   sel    device int32 [R][sel_k]: idx_launch's out_idx on rows bounded by ctx_len (any
 *          order; entries outside 0 .. ctx_len - 1, such as its -1 padding, are skipped).
 *          A row's entries must differ.
 *   sel_k  1 .. IDX_MAX_K.
 * Other arguments, outputs and errors as for idx_tree_attention. */
idx_status idx_tree_attention_selected(const idx_tree_problem *problem, const int32_t *sel, int32_t sel_k, void *out,
                                       float *lse, void *state, size_t state_bytes, void *stream);

/* ---------------------------------------------------------------------------
 * The two ends of the verify step: from a projection's output to q and the cache
 * (idx_norm_rope), and from the logits to the next step's lengths (idx_sample,
 * idx_tree_accept, idx_tree_commit). */
typedef enum {
    IDX_NORM_NONE = 0,    /* y = x */
    IDX_NORM_RMS = 1,     /* y = x / sqrt(mean(x^2) + eps) * weight */
    IDX_NORM_LAYER = 2    /* y = (x - mean(x)) / sqrt(mean((x - mean(x))^2) + eps) * weight + bias */
} idx_norm;

#define IDX_MAX_AXES 4

/* Queries, keys and values of R rows as a fused projection leaves them. */
typedef struct {
    const void *q, *k, *v;     /* device bf16: row r's head h at r * stride + h * D elements, 16-byte aligned; q NULL for
                                  Hq = 0, k NULL for Hkv = 0, v given with a cache that has values, else NULL */
    int64_t q_stride, k_stride, v_stride;     /* elements, at least the row's heads, multiples of 8 */
    void *q_out, *k_out;       /* device bf16, laid out as q and k; each may be its input itself (with its stride), else
                                  they overlap no input.  k_out NULL: the keys go to the cache alone */
    int64_t q_out_stride, k_out_stride;
    const float *q_weight, *q_bias, *k_weight, *k_bias;   /* device fp32 [D], 16-byte aligned, or NULL (1 and 0).
                                  Weights with a norm only, biases with IDX_NORM_LAYER only */
    const int32_t *pos;        /* device int32: row r's position on axis a at a * pos_stride + r (any int32 value) */
    int64_t pos_stride;        /* >= R (>= 0 for one axis) */
    const float *inv_freq;     /* device fp32 [rot / 2]: radians per position (not finite: NaN) */
    const int32_t *slot;       /* device int32 [R] with a cache (as idx_write_kv's), else NULL */
    const int32_t *rows;       /* device int32 [1] or NULL: rows from *rows on are left as they were */
    int64_t R;
    int32_t Hq, Hkv;           /* heads, 0 .. 1024, not both 0 */
    int32_t D;                 /* 64, 128 or 256 (64 or 128 with a cache) */
    int32_t rot;               /* rotated dimensions 0 .. rot - 1: a multiple of 16 within 0 .. D */
    int32_t interleaved;       /* 0: dimension i turns with i + rot / 2; 1: 2 i turns with 2 i + 1 */
    int32_t q_norm, k_norm;    /* idx_norm */
    float eps;                 /* 2^-60 .. 1 */
    int32_t axes;              /* 1 .. IDX_MAX_AXES */
    uint8_t axis[128];         /* HOST: frequency i turns by the position on axis axis[i], i < rot / 2 */
} idx_norm_rope_args;

/* Norm of every head of q and k, then its rotation: with y the normed head and
 * angle_i = pos[axis[i]][r] * inv_freq[i] in real numbers, for any position (off by 2^-32 of a
 * turn at most while |inv_freq| <= 1, and by an fp32 rounding of what is left of it beside the
 * nearest quarter turn), for the pair (a, b) of frequency i
 *     z_a = y_a cos angle_i - y_b sin angle_i,   z_b = y_b cos angle_i + y_a sin angle_i.
 * All of it in fp32, rounded once: q to q_out; k to k_out (bf16) where given, and to the
 * cache where given, at its rows' slots: bf16, or E4M3 with scale = amax / 448 of the fp32
 * values (1 where they are all zero, else 2^-149 at least), saturating; v to the cache exactly
 * as idx_write_kv.
 * NaN and infinity in a normed or quantised head act as idx_write_kv and the formulas say;
 * a head whose squares pass fp32's range is normed all the same.  A slot outside
 * [0, P * 64) writes nothing to the cache; slots >= 0 must differ.
 * cache  NULL, or a cache of Hkv heads of D dimensions; one without values (v and v_scale
 *        NULL, the indexer's key cache among them: Hkv = 1, D = 128, token_stride 128)
 *        takes the keys alone.
 * R = 0 does nothing.  Asynchronous on `stream`; allocates nothing. */
idx_status idx_norm_rope(const idx_norm_rope_args *args, const idx_kv_cache *cache, void *stream);

typedef enum {
    IDX_LOGITS_F32 = 0,
    IDX_LOGITS_BF16 = 1
} idx_logits_dtype;

#define IDX_MAX_VOCAB 360448   /* logits of a row that the sampler takes */

/* Logits of R rows and how a token of each is drawn.  Every parameter is a value per row. */
typedef struct {
    const void *logits;        /* device fp32 or bf16 [R][ld], aligned to its elements; columns 0 .. V-1 are read */
    const float *u;            /* device fp32 [R]: a random number in [0, 1) (below it or NaN: 0, above it, 1 among
                                  that: fp32's last number below 1, 1 - 2^-24) */
    const float *temperature;  /* device fp32 [R] or NULL (1): 0 or less, or NaN: the largest logit's token; else used
                                  within 2^-60 .. 2^60 */
    const int32_t *top_k;      /* device int32 [R] or NULL: 0 or less, or V or more: off */
    const float *top_p;        /* device fp32 [R] or NULL: 1 or more, or NaN: off; 0 or less: the largest logit's token */
    const float *min_p;        /* device fp32 [R] or NULL: 0 or less, or NaN: off; used as at most 1 */
    const int32_t *rows;       /* device int32 [1] or NULL: rows from *rows on are left as they were */
    int64_t ld;                /* elements, >= V */
    int32_t R;                 /* 1 .. IDX_MAX_ROWS */
    int32_t V;                 /* 1 .. IDX_MAX_VOCAB */
    int32_t logits_dtype;      /* idx_logits_dtype */
} idx_sample_args;

/* Draws a token of every row, in one launch.  With w_i = exp((l_i - max l) / T) and the
 * tokens ordered by logit descending, then index ascending:
 *   top-k keeps the first k; top-p of those the ones before which there is less than
 *   p times their weight; min-p of those the ones with w_i >= min_p.
 * The token is the first kept one, in order of index, up to and with which there is more
 * than u times the kept weight: its probability is w_i over that weight.
 *   token    device int32 [R]; -1 for a row without a logit above -inf.
 *   logprob  device fp32 [R] or NULL: the log of the token's probability among the kept
 *            (-inf beside token -1).
 * A NaN counts as -inf; with logits of +inf those alone have weight.  Weights are held to
 * about 2^-38 of themselves as integers, one unit 2^-44 of the power of two at or above the
 * largest (0 below a unit), and summed exactly: where 64-bit sums put a token, so does this,
 * but for numbers u that close to a border.  Equal calls give equal results, and a row the
 * same in any batch.
 * Asynchronous on `stream`; allocates nothing and needs no workspace. */
idx_status idx_sample(const idx_sample_args *args, int32_t *token, float *logprob, void *stream);

/* The drafted trees of a step and the token sampled (or ranked first) at every row. */
typedef struct {
    const int32_t *row_start;  /* device int32 [Q + 1]: ascending, within 0 .. cap (idx_tree_tables writes it) */
    const int32_t *parent;     /* device int32 [cap] or NULL (a chain), as idx_tree_tables reads it */
    const int32_t *draft;      /* device int32 [cap]: every row's own token; a request's token 0 is the one that was
                                  known before the step */
    const int32_t *target;     /* device int32 [cap]: the token drawn from every row's logits */
    const int32_t *ctx_len;    /* device int32 [Q]: tokens cached before the step (as idx_tree_tables reads them) */
    const int32_t *page_table; /* device int32 [Q][pt_stride], with the step's pages */
    int32_t *free_pages;       /* device int32 [free_cap]: the free stack; pages given back are written from free_count on */
    const int32_t *free_count; /* device int32 [1]: its height (idx_tree_tables's free_left) */
    int32_t *free_left;        /* out, device int32 [1]: its height afterwards; may be free_count itself */
    int32_t *new_ctx;          /* out, device int32 [Q]: ctx_len + accept_len; may be ctx_len itself */
    int32_t *accept_len;       /* out, device int32 [Q]: accepted tokens, token 0 among them; 0 for a request without rows */
    int32_t *last;             /* out, device int32 [Q]: the sampled token behind the last accepted one: the next step's
                                  token 0 (-1 for a request without rows) */
    int32_t *path;             /* out, device int32 [cap]: path[row_start[i] + a] is the token number of request i's a-th
                                  accepted token, -1 from accept_len[i] on */
    int32_t *token;            /* out, device int32 [cap]: the request's new tokens, token[row_start[i] + a] =
                                  target[row_start[i] + path[row_start[i] + a]], -1 from accept_len[i] on */
    int64_t P;                 /* pages of the cache, 1 .. INT32_MAX / 64 */
    int32_t Q;                 /* requests, 1 .. IDX_MAX_REQS */
    int32_t pt_stride;         /* page-table row length, >= 1 */
    int32_t cap;               /* rows that the per-row arrays hold, 1 .. INT32_MAX - 3 */
    int32_t free_cap;          /* entries of free_pages, >= 0 */
} idx_tree_accept_args;

/* Bytes of state that idx_tree_accept needs: as for idx_tree_tables, all zero before its
 * first use; calls that overlap in time need one each. */
size_t idx_tree_accept_state_size(void);

/* One launch.  A request's token 0 is accepted; behind an accepted token n the first child c
 * (parent[c] == n) with draft[c] == target[n] is, and so on.  Where target is drawn by
 * idx_sample, the accepted tokens and `last` are distributed as the model alone would draw
 * them, whatever was drafted.  Pages of the step's tokens that hold none of the first
 * ctx_len + accept_len positions go back to the stack, in order of requests and positions;
 * their table entries are left as they were, behind the request's length.  The accepted
 * tokens' keys and values still lie at their slots in the tree: idx_tree_commit moves them.
 * Rows from row_start[Q] on are not written.
 * Outputs may not overlap inputs or each other, but for the two that say so.
 * Found on the device and recorded as IDX_EDEVICE: row_start outside 0 .. cap or descending
 * (cut), a request of more than IDX_MAX_TREE rows (those past the 64th are not accepted), a
 * parent that is not an earlier token (nobody's child), a page to give back without an id in
 * [0, P) or without room on the stack (left out). */
idx_status idx_tree_accept(const idx_tree_accept_args *args, void *state, size_t state_bytes, void *stream);

/* Moves the accepted tokens' keys and values, scales with them, to consecutive positions:
 * for a = 1 .. accept_len[i] - 1 from the slot of row row_start[i] + path[row_start[i] + a] to
 * that of row row_start[i] + a, bit for bit, as if all were read before any is written.
 *   cache       any; one without values moves keys alone (see idx_norm_rope).
 *   row_start, accept_len, path   as idx_tree_accept reads and writes them.
 *   slot        device int32 [cap], as idx_tree_tables writes it: page * 64 + token.
 * Rows with path <= a or outside the request, and slots outside [0, P * 64), move nothing;
 * slots >= 0 must differ.  Asynchronous on `stream`; allocates nothing. */
idx_status idx_tree_commit(const idx_kv_cache *cache, const int32_t *row_start, const int32_t *accept_len,
                           const int32_t *path, const int32_t *slot, int32_t Q, int32_t cap, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* IDX_H */
