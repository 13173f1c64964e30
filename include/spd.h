/*
 * spd.h -- sparse paged decode attention for GB300 (sm_103a): the C ABI.
 *
 * The library computes the attention hot path of sparse rollouts over a paged
 * bf16 KV cache: per-page key summaries, query-aware page scoring with a
 * per-sequence page budget, attention over only the selected pages (split-K
 * with a log-sum-exp merge), and dense causal verification of k+1 drafted
 * positions over the whole cache.
 *
 * Sources.  Block-sparse (page) attention during rollouts with a KV budget and
 * a page size, and a Top-k over pages: the Sparrow project page, "Insights" and
 * "Control Study 2" (cost model; block size 16 and above; page size 16).  A
 * budget that grows with generation length: Sparrow, "Control Study 1"
 * (sparsity scheduling).  Sparse drafting of k = 6 tokens and dense
 * verification over the complete KV cache: the S3R abstract, Figure 6 and
 * Table 7.  The page score is a Quest-style upper bound from per-page,
 * per-channel key minima and maxima (Quest is in Sparrow's reference list;
 * the pages print no scoring rule of their own).
 *
 * Conventions shared by every call.
 *  - All tensor pointers are DEVICE pointers owned by the caller; the library
 *    never allocates, frees or synchronises (except spd_device_status).  Every
 *    call is asynchronous on `stream` (a cudaStream_t; NULL = legacy default).
 *  - bf16 values are passed as raw 16-bit patterns (spd_bf16).  K, V, q, the
 *    summaries and o must be 16-byte aligned; the KV cache base additionally
 *    must allow 16-byte row strides (D * 2 bytes, always true for D = 64, 128).
 *  - Paged KV cache: K and V are [num_phys_pages][H_kv][page_size][D] bf16, so
 *    one (physical page, KV head) tile is contiguous.  page_table is
 *    [B][max_pages_per_seq] int32 of physical page ids; seq_lens is [B] int32
 *    token counts (including the current token, or all T draft tokens).
 *    Sequence b uses logical pages 0 .. ceil(seq_lens[b] / page_size) - 1; the
 *    cache slots past seq_lens[b] in its last page are never used for a result
 *    (their contents may be anything, including NaN).
 *  - GQA: query head hq reads KV head hq / G, G = H_q / H_kv.
 *  - Softmax: logits z = softmax_scale * q.k; lse is the natural-log
 *    log-sum-exp of the scaled logits.  A row that sees no token gets o = 0,
 *    lse = -inf.
 *  - Workspace: `ws` is caller-owned device scratch of at least the size the
 *    matching *_workspace_size function returns.  The counters and flags some
 *    calls keep in it (unit queue, split tickets, the step's chain) MUST be
 *    zero before the first call that uses the buffer (zero the whole buffer
 *    once); every successful call leaves them zero again.  The queue and the tickets
 *    of every call lie in the buffer's first bytes, where no call writes anything
 *    else, so a buffer can be reused by any later call, whatever its kind and
 *    dims, on the same stream.  Two calls keep more, and want the whole buffer
 *    zeroed again if it has served other calls, or themselves with other sizes:
 *    sparse_decode_step (its chain lies behind its scores), and sparse_decode_attn
 *    or dense_verify_attn told to split (num_splits > 1) more than 16,384 rows
 *    B * H_kv.  Calls that overlap on the GPU must use different workspaces.
 *  - Errors: argument problems are reported synchronously by the returned
 *    status (nothing is launched); spd_last_error() gives a message.  Problems
 *    only the GPU can see (a page id outside [0, num_phys_pages), a selection
 *    entry out of range, a bounded wait that ran out) set bits in a device
 *    status word read by spd_device_status(); the affected rows are skipped or
 *    zeroed, and no kernel traps, asserts or spins without a bound.
 */
#ifndef SPD_H
#define SPD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef uint16_t spd_bf16; /* bfloat16 bit pattern */

typedef enum {
    SPD_OK = 0,
    SPD_ERR_INVALID_ARG = 1, /* null pointer, bad size, misaligned pointer, inconsistent shapes */
    SPD_ERR_UNSUPPORTED = 2, /* a shape outside the supported set (see spd_dims) */
    SPD_ERR_CUDA = 3,        /* a CUDA runtime or launch error; see spd_last_error() */
    SPD_ERR_WORKSPACE = 4    /* ws is NULL or ws_bytes is below the required size */
} spd_status;

/* Device status bits (spd_device_status). */
#define SPD_DEV_BAD_PAGE 0x1u  /* a page-table entry outside [0, num_phys_pages) */
#define SPD_DEV_BAD_SEL 0x2u   /* a selected page id outside the sequence, or nsel > k_max */
#define SPD_DEV_TIMEOUT 0x4u   /* a bounded wait on an asynchronous copy ran out */
#define SPD_DEV_BAD_LEN 0x8u   /* seq_lens[b] outside [0, max_pages_per_seq * page_size] (the row is
                                * then treated as empty: nothing selected, o = 0, lse = -inf), or
                                * too short for the tokens being appended */
#define SPD_DEV_BAD_TOKEN 0x10u /* spec_accept: a drafted token outside [0, n_vocab);
                                 * token_logprobs: a target outside [-1, n_vocab) */
#define SPD_DEV_BAD_POS 0x20u   /* a position outside the rotation's table */
#define SPD_DEV_BAD_TREE 0x40u  /* a parent that is not before its node, a path entry outside [0, T) or a
                                 * path length outside [0, T] */

/*
 * Problem shape.  Supported: D in {64, 128}; page_size in {16, 32, 64};
 * H_kv >= 1, H_q % H_kv == 0, G = H_q / H_kv <= 8; max_pages_per_seq >= 1;
 * num_phys_pages * H_kv * page_size < 2^31.  B = 0 is a valid no-op.
 */
typedef struct {
    int32_t B;                 /* sequences */
    int32_t H_q;               /* query heads */
    int32_t H_kv;              /* KV heads */
    int32_t D;                 /* head dimension */
    int32_t page_size;         /* tokens per page */
    int32_t max_pages_per_seq; /* row length of page_table */
    int64_t num_phys_pages;    /* pages in the K / V / summary arrays */
} spd_dims;

typedef enum {
    SPD_BUDGET_FIXED_PAGES = 0,   /* budget = fixed_pages */
    SPD_BUDGET_LINEAR_TOKENS = 1, /* ceil(max(min_tokens, ceil(len*slope_num/slope_den) + intercept) / page_size) */
    SPD_BUDGET_FRACTION = 2,      /* ceil(len * frac_num / (frac_den * page_size)) */
    SPD_BUDGET_TOP_P = 3          /* the smallest set holding top_p of the page weight (below) */
} spd_budget_mode;

/*
 * Per-sequence page budget (the sparsity schedule), evaluated on the device in
 * exact 64-bit integer arithmetic from len = seq_lens[b].  The first
 * sink_pages pages (the attention sink) and the last local_pages pages (the
 * local window) are always selected and count toward the budget.  The number
 * of pages selected for a (sequence, KV head) is
 *   k_eff = min(P, max(min(budget, k_max), |mandatory|)),  P = ceil(len / page_size).
 *
 * SPD_BUDGET_TOP_P makes the budget query-dependent (the pages stress that the
 * budget a query needs varies strongly: S3R abstract, Sparrow "Control Study
 * 1").  Each page gets the weight w(p) = exp(score_scale * (score(p) - max
 * score)), a softmax over pages of the bound logits; after the mandatory
 * pages, the best-scoring pages are added until the selected weight reaches
 * top_p of the total, at most k_max pages in all.  On the device the weights
 * are fp32 exponentials rounded to multiples of 2^-31 and summed as exact
 * integers, so the count is deterministic; it can differ from a real-number
 * evaluation only where the selected weight lands within that rounding of
 * the top_p share.
 */
typedef struct {
    int32_t mode; /* spd_budget_mode */
    int32_t fixed_pages;
    int64_t min_tokens, slope_num, slope_den, intercept; /* LINEAR_TOKENS (slope_den > 0) */
    int64_t frac_num, frac_den;                          /* FRACTION (frac_den > 0) */
    int32_t sink_pages, local_pages;                     /* >= 0 */
    float top_p;       /* TOP_P: share of the page weight to hold, in [0, 1] */
    float score_scale; /* TOP_P: logit scale of the scores (> 0), e.g. 1 / sqrt(D) */
} spd_budget_policy;

/* Library ABI version (major * 100 + minor). */
int32_t spd_version(void);

/* Message for the last non-OK status returned on this host thread ("" if none). */
const char *spd_last_error(void);

/*
 * Reads (and with clear != 0, resets) the device status word of the current
 * device.  Synchronises the device.  Returns SPD_ERR_CUDA if the read fails.
 */
spd_status spd_device_status(uint32_t *out, int32_t clear);

/*
 * Limit, in nanoseconds of the GPU's global timer, of every bounded wait in the
 * kernels launched after this call, from any host thread (2 s by default): an
 * mbarrier wait on an asynchronous copy, and in sparse_decode_step's chain a
 * selection waiting for its row's scores or an attention unit waiting for its
 * row's selection.  A wait that runs out sets SPD_DEV_TIMEOUT, the kernel
 * skips the rest of the affected rows and returns; the workspace of such a
 * call must be zeroed again before it is reused.  Graphs keep the limit they
 * were captured with.  ns = 0 is rejected (SPD_ERR_INVALID_ARG).
 */
spd_status spd_set_wait_limit_ns(uint64_t ns);
uint64_t spd_wait_limit_ns(void);

/* Workspace sizes in bytes (0 on invalid arguments; see spd_last_error). */
size_t spd_score_select_workspace_size(const spd_dims *dims);
size_t spd_sparse_decode_workspace_size(const spd_dims *dims, int32_t k_max, int32_t num_splits);
size_t spd_dense_verify_workspace_size(const spd_dims *dims, int32_t T, int32_t num_splits);

/*
 * pages_summarize -- per-page key summaries (Quest-style page metadata that the
 * scoring rule reads; the pages' cost model charges one scoring read per
 * generated page: Sparrow, "Control Study 2", scoring term).
 *
 * For each listed (sequence b, logical page p) and each KV head h, writes the
 * channel-wise minimum and maximum of the keys of the page's valid tokens
 * (positions < seq_lens[b]), phys = page_table[b][p]:
 *   summ[b][h][p][0][d] = min_t K[phys][h][t][d],  summ[b][h][p][1][d] = max_t ...
 * summ is bf16 [B][H_kv][max_pages_per_seq][2][D], sequence-major so that
 * scoring a (sequence, KV head) row reads one contiguous stream; bf16 min/max
 * is exact.  Sequences that share physical pages (the rollouts of one prompt
 * sharing its prefix pages) each keep their own copy of a shared page's
 * summary: the scoring reads each sharer's copy once per step either way, but
 * the copies cost memory (4 * D bytes per page and KV head per sharer) and a
 * rewritten shared page must be summarised again for every sharer (one
 * only_pages entry per (sequence, page) slot).
 * only_pages: NULL = every logical page of every sequence; otherwise n_only
 * entries, each b * max_pages_per_seq + p (a slot of page_table), e.g. the
 * page the newest token was written to.  Entries whose p is past the
 * sequence's last page are skipped.  Pages not listed are left untouched.
 */
spd_status pages_summarize(const spd_dims *dims, const spd_bf16 *K, const int32_t *page_table,
                           const int32_t *seq_lens, const int32_t *only_pages, int32_t n_only,
                           spd_bf16 *summ, void *stream);

/*
 * kv_append_refresh -- appends the T newest tokens of every sequence to the
 * paged cache and rewrites the summaries of the pages they land in, in one
 * kernel (the per-step cache update before scoring: one token per decode
 * step; after verification, the T drafted positions rewritten with the
 * target's keys and values).  KV pages: S3R Figure 1(c); the per-step scoring
 * read of the summaries: Sparrow, "Control Study 2".
 *
 * seq_lens[b] already counts the new tokens: token t (0 <= t < T) goes to
 * position pos = seq_lens[b] - T + t, i.e. slot pos % page_size of physical
 * page page_table[b][pos / page_size], for every KV head:
 *   K[phys][h][slot][:] = k_new[b][t][h][:],  V[...] = v_new[b][t][h][:]
 * (k_new, v_new bf16 [B][T][H_kv][D], copied bit for bit).  Every page that
 * receives a token gets summ[b][h][p] = min / max over all its valid tokens
 * after the write -- the same bits pages_summarize would write -- whatever
 * the summary held before.  Other pages and cache slots are untouched.
 * Supported: 1 <= T <= 4096.  A sequence with seq_lens[b] < T or
 * seq_lens[b] > max_pages_per_seq * page_size is skipped and sets
 * SPD_DEV_BAD_LEN; a page id outside [0, num_phys_pages) sets SPD_DEV_BAD_PAGE.
 * K, V, k_new, v_new and summ must be 16-byte aligned.  Sequences must not
 * share the physical pages they append to.
 */
spd_status kv_append_refresh(const spd_dims *dims, int32_t T, spd_bf16 *K, spd_bf16 *V,
                             const int32_t *page_table, const int32_t *seq_lens,
                             const spd_bf16 *k_new, const spd_bf16 *v_new, spd_bf16 *summ,
                             void *stream);

/*
 * pages_score_select -- query-aware page scoring plus budgeted top-k
 * (Sparrow, "Control Study 2": KV budget B, page size, Top-k over pages;
 * "Control Study 1": length-scheduled budget).
 *
 * q is bf16 [B][H_q][D] (the decode query); summ is the [B][H_kv][max_pages][2][D]
 * array pages_summarize maintains.  For every sequence b, KV head h and page
 * p < P_b, the score is
 *   score(p) = max_{g < G} sum_d max(q[b][hG+g][d] * kmin[d], q[b][hG+g][d] * kmax[d])
 * (an upper bound of q.k over the page's keys), accumulated in fp32 from the
 * bf16 summaries.  Then the mandatory pages plus the best-scoring remaining
 * pages (score descending, ties to the lower page id) up to k_eff are
 * selected and written in ascending page order:
 *   sel [B][H_kv][k_max] int32 logical page ids (entries past nsel untouched),
 *   nsel[B][H_kv] int32 = k_eff.
 * scores: optional fp32 [B][H_kv][max_pages_per_seq] output of the raw scores
 * (slots past P_b untouched); NULL keeps them in the workspace.
 * Requires k_max >= sink_pages + local_pages.
 */
spd_status pages_score_select(const spd_dims *dims, const spd_bf16 *q, const spd_bf16 *summ,
                              const int32_t *seq_lens,
                              const spd_budget_policy *policy, int32_t *sel, int32_t *nsel,
                              int32_t k_max, float *scores, void *ws, size_t ws_bytes,
                              void *stream);

/*
 * pages_append_score_select -- kv_append_refresh with T = 1 and
 * pages_score_select in one pass over the summaries: the warp that scores the
 * tile holding a row's last page first writes the step's token (position
 * seq_lens[b] - 1) into K and V, rebuilds that page's summary (stored to summ
 * and used for the score), then scores the tile.  Results (K, V, summ, sel,
 * nsel, scores) are bit-identical to kv_append_refresh(T = 1) followed by
 * pages_score_select; one kernel launch and one pass over the cache update
 * fewer.  k_new, v_new: bf16 [B][H_kv][D].  A sequence with seq_lens[b] = 0
 * sets SPD_DEV_BAD_LEN and is skipped; a page id outside [0, num_phys_pages)
 * sets SPD_DEV_BAD_PAGE.  Other arguments and errors as the two calls.
 */
spd_status pages_append_score_select(const spd_dims *dims, spd_bf16 *K, spd_bf16 *V,
                                     const int32_t *page_table, const int32_t *seq_lens,
                                     const spd_bf16 *k_new, const spd_bf16 *v_new, const spd_bf16 *q,
                                     spd_bf16 *summ, const spd_budget_policy *policy, int32_t *sel,
                                     int32_t *nsel, int32_t k_max, float *scores, void *ws,
                                     size_t ws_bytes, void *stream);

/*
 * sparse_decode_attn -- attention of the decode query over the selected pages
 * only (block-sparse page attention: Sparrow, "Insights" and "Control Study
 * 2"; the S3R sparse drafter of Table 7).
 *
 * For each sequence b and query head hq (KV head h = hq / G): exact softmax
 * attention over the valid tokens of pages sel[b][h][0 .. nsel[b][h]):
 *   o[b][hq][d] (bf16), lse[b][hq] (fp32, natural log; may be NULL).
 * num_splits: 0 = automatic; otherwise the selected list of each (b, h) is cut
 * into that many contiguous parts processed in parallel and merged with the
 * log-sum-exp rule of lse_merge.  The workspace must hold
 * spd_sparse_decode_workspace_size(dims, k_max, num_splits) bytes.
 */
spd_status sparse_decode_attn(const spd_dims *dims, const spd_bf16 *q, const spd_bf16 *K,
                              const spd_bf16 *V, const int32_t *page_table,
                              const int32_t *seq_lens, const int32_t *sel, const int32_t *nsel,
                              int32_t k_max, int32_t num_splits, float softmax_scale,
                              spd_bf16 *o, float *lse, void *ws, size_t ws_bytes, void *stream);

/*
 * sparse_decode_step -- one whole sparse decode step in one call: the step's
 * token appended (as kv_append_refresh with T = 1; skipped when k_new and
 * v_new are NULL), every page scored and the budgeted selection made (as
 * pages_score_select), and attention over the selected pages (as
 * sparse_decode_attn with automatic splits).  Results -- K, V, summ, sel,
 * nsel, o, lse -- are those of the separate calls.
 *
 * The three kernels are chained row by row instead of grid by grid: scoring
 * hands out its tiles in row order and counts the finished tiles of each row,
 * the selection of a row starts as soon as its count is complete, and the
 * attention units of a row (one, or several and a merge when there are few
 * rows) as soon as its selection is published (release / acquire flags in the
 * workspace; every wait is bounded and reports SPD_DEV_TIMEOUT).  The
 * workspace (spd_sparse_decode_step_workspace_size bytes) must be zero before
 * its first use, and before a step with other dims or k_max or behind other calls
 * that used it; a step leaves it as it needs it, and other calls may follow one.
 * Calls that overlap on the GPU need separate workspaces.  Errors as the separate
 * calls.
 */
size_t spd_sparse_decode_step_workspace_size(const spd_dims *dims, int32_t k_max);
spd_status sparse_decode_step(const spd_dims *dims, spd_bf16 *K, spd_bf16 *V, const int32_t *page_table,
                              const int32_t *seq_lens, const spd_bf16 *k_new, const spd_bf16 *v_new,
                              const spd_bf16 *q, spd_bf16 *summ, const spd_budget_policy *policy,
                              int32_t *sel, int32_t *nsel, int32_t k_max, float softmax_scale,
                              spd_bf16 *o, float *lse, void *ws, size_t ws_bytes, void *stream);

/*
 * sparse_decode_attn_noalloc -- sparse_decode_attn for callers that cannot
 * allocate device memory.  It has no counterpart on the pages: it is the same
 * computation, with the same arguments and results as sparse_decode_attn,
 * minus the workspace.
 *
 * Who needs it: code that runs where a cudaMalloc is not allowed or not
 * wanted -- an inference engine that owns all device memory through a fixed
 * arena and gives plug-ins no workspace argument, or a latency-critical decode
 * loop that must not call cudaMalloc because it can synchronise the device
 * and stall every stream.  Such a caller still passes q, K, V, the page table,
 * the selection and the outputs; the scratch this call needs (the unit queue,
 * the split tickets and the split partials) lives in a fixed array compiled
 * into the library, SPD_NOALLOC_SCRATCH_BYTES (8 MiB) per GPU, which every GPU
 * that loads the library holds until the process exits.
 *
 * Behaviour: the first call on a device looks up that array's device address
 * (once per device, with that device current); make that first call before
 * any stream capture.  Each call clears the array's counters on `stream`
 * (cudaMemsetAsync) and never calls cudaMalloc, cudaFree or any allocating
 * library routine.  The split count is num_splits, or with num_splits = 0 the
 * automatic count lowered until the partials fit the array; if the requested
 * split count (or even one split) needs more scratch than the array holds, the
 * call returns SPD_ERR_UNSUPPORTED and launches nothing.  All calls share the
 * one array: calls that overlap on the GPU (different streams, or different
 * host threads without ordering) race and give wrong results.
 */
#define SPD_NOALLOC_SCRATCH_BYTES ((size_t)8 << 20)
spd_status sparse_decode_attn_noalloc(const spd_dims *dims, const spd_bf16 *q, const spd_bf16 *K,
                                      const spd_bf16 *V, const int32_t *page_table,
                                      const int32_t *seq_lens, const int32_t *sel,
                                      const int32_t *nsel, int32_t k_max, int32_t num_splits,
                                      float softmax_scale, spd_bf16 *o, float *lse, void *stream);

/*
 * dense_verify_attn -- dense causal verification of T drafted positions over
 * the complete KV cache (S3R abstract; Table 7 "Verify (TV)", k = 6 so T = 7).
 *
 * q is bf16 [B][T][H_q][D]; the drafted tokens' K/V are already the last T
 * tokens of each sequence.  Row t (absolute position seq_lens[b] - T + t)
 * attends over tokens 0 .. seq_lens[b] - T + t.  Outputs o bf16 [B][T][H_q][D]
 * and lse fp32 [B][T][H_q] (may be NULL).  T = 1 is dense decode attention.
 * Supported: 1 <= T and T * G <= 64.  num_splits: 0 = automatic.
 */
spd_status dense_verify_attn(const spd_dims *dims, int32_t T, const spd_bf16 *q,
                             const spd_bf16 *K, const spd_bf16 *V, const int32_t *page_table,
                             const int32_t *seq_lens, int32_t num_splits, float softmax_scale,
                             spd_bf16 *o, float *lse, void *ws, size_t ws_bytes, void *stream);

/*
 * spec_accept -- exact speculative sampling over k drafted tokens per sequence
 * (S3R abstract: responses come from full-attention verification and exact
 * speculative sampling, so they follow the dense policy; k = 6 in Table 7).
 *
 * p_draft fp32 [B][k][n_vocab]: the drafter's distribution at each drafted
 * position; q_target fp32 [B][k+1][n_vocab]: the target's distribution at the
 * same positions plus the one after the last draft (from dense_verify_attn's
 * pass); draft int32 [B][k]; u_acc fp32 [B][k] and u_res fp32 [B]: uniform
 * numbers in [0, 1) drawn by the caller.  Rows need not be normalised.
 * For each sequence: draft x at position i is accepted iff
 * u_acc[b][i] * p_i(x) < q_i(x) (product formed exactly in fp64), in order,
 * until the first rejection j.  The emitted token is a draw from integer
 * weights on a 2^-40 grid, W(x) = max(0, F(q_j(x)) - F(p_j(x))) with
 * F(v) = floor(2^40 * min(v, 1)) (0 for v <= 0 or NaN), or W(x) = F(q_j(x))
 * when that residual is zero everywhere; after k acceptances W(x) = F(q_k(x))
 * (the bonus token).  The draw is the smallest x whose running sum of W
 * exceeds floor(u_res[b] * sum(W)); all sums are exact integers, so the
 * result does not depend on summation order.  W zero everywhere: -1.  (Mass
 * below 2^-40 per token is never drawn: at most n_vocab * 2^-40 of total
 * variation from the real-number rule.)
 * Outputs: n_accepted int32 [B]; tokens int32 [B][k+1] = the accepted drafts,
 * the emitted token, then -1.  A draft outside [0, n_vocab) at or before the
 * first rejection sets SPD_DEV_BAD_TOKEN and gives that sequence
 * n_accepted = 0, tokens = -1.
 * Supported: 1 <= k <= 32, 1 <= n_vocab <= 2^21; p_draft and q_target 16-byte
 * aligned.
 */
spd_status spec_accept(int32_t B, int32_t k, int32_t n_vocab, const float *p_draft,
                       const float *q_target, const int32_t *draft, const float *u_acc,
                       const float *u_res, int32_t *n_accepted, int32_t *tokens, void *stream);

/*
 * lse_merge -- combine S partial attention results computed over disjoint
 * token sets (split-K FlashDecoding):
 *   lse = log sum_s exp(part_lse[s]),  o = sum_s exp(part_lse[s] - lse) * part_o[s].
 * part_o fp32 [S][rows][D] (each partial already normalised), part_lse fp32
 * [S][rows] (natural log; -inf marks an empty partial).  Writes o bf16
 * [rows][D] and lse fp32 [rows] (lse may be NULL).  All partials empty:
 * o = 0, lse = -inf.  Supported: S >= 1, D in {64, 128}.
 */
spd_status lse_merge(int32_t S, int32_t rows, int32_t D, const float *part_o,
                     const float *part_lse, spd_bf16 *o, float *lse, void *stream);

/*
 * spd_rope -- norm of each head's row and position rotation of queries and keys
 * (what the Qwen3 shapes of the rollout studies do between the projection and the
 * attention).  A head row x of D channels becomes
 *   y = x / sqrt(mean(x^2) + eps) * weight          (no norm where weight is NULL)
 * and then, for i < rot_dim / 2 and the angle of the row's position and of i,
 *   (y[a], y[b]) -> (y[a] cos - y[b] sin, y[b] cos + y[a] sin),
 * (a, b) = (i, i + rot_dim / 2), or (2i, 2i + 1) with interleaved != 0; channels
 * from rot_dim on are not rotated.  Everything is fp32, rounded to bf16 once.
 * Supported: rot_dim a multiple of 8 in [0, D]; table fp32 [n_pos][2][rot_dim / 2],
 * the cosines of a position and then its sines, 16-byte aligned (rot_dim = 0: not
 * read, may be NULL); weights bf16 [D], 8-byte aligned; eps >= 0 and finite.
 */
typedef struct {
    const float *table;
    int32_t n_pos;
    int32_t rot_dim;
    int32_t interleaved;
    float eps;
    const spd_bf16 *q_weight; /* NULL: queries without a norm */
    const spd_bf16 *k_weight; /* NULL: keys without a norm */
} spd_rope;

/*
 * qk_norm_rope -- norm and rotation of the queries and keys of `rows` tokens in one
 * pass: q_out[row][h] and k_out[row][h] from q and k at positions[row] (int32).
 *
 * q: rows of H_q * D contiguous bf16, q_stride elements apart (k likewise, H_kv and
 * k_stride), so both may be views of one fused projection; strides multiples of 8,
 * at least the row's length.  q or k may be NULL: that side is skipped.  q_out bf16
 * [rows][H_q][D], k_out bf16 [rows][H_kv][D]; an output may be its own input where
 * that is contiguous, and must not overlap an input otherwise.  Pointers 16-byte
 * aligned.  A position outside [0, n_pos) sets SPD_DEV_BAD_POS and gives zero rows
 * (with rot_dim = 0 the positions are not read and may be NULL).
 * Supported: D in {64, 128}; any H_q, H_kv >= 1; rows >= 0 (0: no-op).
 */
spd_status qk_norm_rope(int64_t rows, int32_t H_q, int32_t H_kv, int32_t D, const spd_rope *rope,
                        const spd_bf16 *q, int64_t q_stride, const spd_bf16 *k, int64_t k_stride,
                        const int32_t *positions, spd_bf16 *q_out, spd_bf16 *k_out, void *stream);

/*
 * kv_append_rope -- kv_append_refresh of the normalised and rotated keys, and the
 * queries of the same tokens, in one kernel: what a layer does between its projection
 * and pages_score_select or dense_verify_attn.
 *
 * Token t (0 <= t < T) of sequence b is row b * T + t of q, k and v (strided rows as
 * in qk_norm_rope; v_stride elements apart) and has position seq_lens[b] - T + t.
 * K, V and summ afterwards, and q_out bf16 [B][T][H_q][D], are bit for bit what
 * qk_norm_rope at those positions and kv_append_refresh give.  q and q_out may both
 * be NULL (keys and values only).
 * Supported: 1 <= T <= 4096.  A sequence with seq_lens[b] < T or seq_lens[b] >
 * max_pages_per_seq * page_size sets SPD_DEV_BAD_LEN, one with seq_lens[b] > n_pos
 * (where rot_dim > 0) sets SPD_DEV_BAD_POS: its cache is left as it was and its q_out
 * rows are zeros.  A page id outside [0, num_phys_pages) sets SPD_DEV_BAD_PAGE and
 * skips that page's tokens.  Sequences must not share the pages they append to.
 */
spd_status kv_append_rope(const spd_dims *dims, int32_t T, const spd_rope *rope, spd_bf16 *K,
                          spd_bf16 *V, const int32_t *page_table, const int32_t *seq_lens,
                          const spd_bf16 *q, int64_t q_stride, const spd_bf16 *k, int64_t k_stride,
                          const spd_bf16 *v, int64_t v_stride, spd_bf16 *q_out, spd_bf16 *summ,
                          void *stream);

/*
 * The 4-bit paged cache.  kv4 is bytes [num_phys_pages][H_kv][2][page_size * D * 9 / 16],
 * 16-byte aligned: for each page and KV head the keys (0) and the values (1), each
 * page_size rows of D / 2 code bytes (row-major, channel 2j in the low and channel
 * 2j + 1 in the high four bits of byte j) and then page_size rows of D / 16 scale
 * bytes, one for each group of 16 channels.  4.5 bits an element.
 *
 * A code is an e2m1 number (sign, 2 exponent bits, 1 mantissa bit: 0, 0.5, 1, 1.5, 2,
 * 3, 4, 6), a scale an e4m3 number, and the value is code * scale * 2^exp, exp being
 * k_exp for keys and v_exp for values: exact in bf16.  exp is the caller's, one for
 * the whole cache, -64 <= exp <= 64; it should bring the values' largest magnitudes
 * near 2^exp * 100, well inside the scales' range [2^-9, 448] (0 suits keys and values
 * of unit size; a cache of small values wants a negative v_exp).
 * Page tables, seq_lens and the summaries are those of the bf16 cache, so
 * pages_score_select serves both.
 */

/*
 * kv4_append -- quantises the T newest tokens of every sequence into the cache and
 * rewrites the summaries of the pages they land in (min / max of the values as held,
 * so the scores bound the logits of the 4-bit attention).
 *
 * k_new, v_new: bf16 [B][T][H_kv][D], contiguous; positions, errors and limits as
 * kv_append_refresh.  A group's scale is amax / (6 * 2^exp) rounded to the nearest
 * e4m3 number, at most 448; codes are x / (scale * 2^exp) rounded to the nearest e2m1
 * number (ties to the even code), at most 6 in magnitude; a zero scale gives zeros.
 * Infinities saturate; NaN counts as zero.
 */
spd_status kv4_append(const spd_dims *dims, int32_t T, uint8_t *kv4, int32_t k_exp, int32_t v_exp,
                      const int32_t *page_table, const int32_t *seq_lens, const spd_bf16 *k_new,
                      const spd_bf16 *v_new, spd_bf16 *summ, void *stream);

/*
 * kv4_read -- the T newest tokens of every sequence as the values that the cache
 * holds: k_out, v_out bf16 [B][T][H_kv][D], exact.  For checks against the unquantised
 * rows and for moving a cache to bf16.  Limits as kv4_append; the rows of a sequence
 * or page that is skipped there are zeros.
 */
spd_status kv4_read(const spd_dims *dims, int32_t T, const uint8_t *kv4, int32_t k_exp, int32_t v_exp,
                    const int32_t *page_table, const int32_t *seq_lens, spd_bf16 *k_out,
                    spd_bf16 *v_out, void *stream);

/*
 * kv4_sparse_decode_attn / kv4_dense_verify_attn -- sparse_decode_attn and
 * dense_verify_attn over the 4-bit cache: arguments, limits, errors and results as
 * there, over the values that the cache stands for; softmax_scale * 2^k_exp finite in
 * fp32, num_splits ignored where B * H_kv > 16384 (no row is split then).  Workspaces
 * by the sizes below (tickets zero before the first use, left zero).
 * As over the bf16 cache, a unit (a split of a row) is summed in fp32 by the tensor
 * cores, which cut what lies some 2^-25 below a sum: a row of more than 2^17 tokens should
 * not be kept in one split (values of one sign, mean error of o: 0.1 % at 2^17 tokens in
 * one unit, 0.7 % at 2^20; with automatic splits none).
 */
size_t spd_kv4_sparse_decode_workspace_size(const spd_dims *dims, int32_t k_max, int32_t num_splits);
size_t spd_kv4_dense_verify_workspace_size(const spd_dims *dims, int32_t T, int32_t num_splits);
spd_status kv4_sparse_decode_attn(const spd_dims *dims, const spd_bf16 *q, const uint8_t *kv4,
                                  int32_t k_exp, int32_t v_exp, const int32_t *page_table,
                                  const int32_t *seq_lens, const int32_t *sel, const int32_t *nsel,
                                  int32_t k_max, int32_t num_splits, float softmax_scale, spd_bf16 *o,
                                  float *lse, void *ws, size_t ws_bytes, void *stream);
spd_status kv4_dense_verify_attn(const spd_dims *dims, int32_t T, const spd_bf16 *q,
                                 const uint8_t *kv4, int32_t k_exp, int32_t v_exp,
                                 const int32_t *page_table, const int32_t *seq_lens,
                                 int32_t num_splits, float softmax_scale, spd_bf16 *o, float *lse,
                                 void *ws, size_t ws_bytes, void *stream);

/*
 * token_logprobs -- log probabilities of given tokens, one pass over their logits: the
 * sampled tokens' behaviour probabilities of a rollout, or those of spec_accept's
 * output (tokens [B][k+1] against the target's logits [B][k+1][n_vocab]).
 *
 * logits: `rows` rows of n_vocab numbers (fp32, or bf16 with logits_bf16 != 0),
 * row_stride elements apart, row_stride >= n_vocab.  With z = inv_temperature * logits:
 *   lse[row] = log sum_x exp z(x),   logprob[row] = z(targets[row]) - lse[row],
 *   entropy[row] = -sum_x p(x) log p(x),  p = exp(z - lse),
 * and the top_k largest logits (ties: the lower token first) as top_ids int32
 * [rows][top_k] with top_logprobs fp32 [rows][top_k], in descending order.
 * logprob, entropy and lse are fp32 and may each be NULL; top_ids and top_logprobs go
 * together and are NULL with top_k = 0.
 * targets int32: -1 (no token, as behind spec_accept's last one) gives logprob 0; any
 * other target outside [0, n_vocab) gives 0 too and sets SPD_DEV_BAD_TOKEN.  targets
 * may be NULL with logprob.
 * A logit of -inf (a masked token) has probability 0, logprob -inf and is never an
 * alternative: where fewer than top_k logits are above -inf the rest is id -1, logprob
 * -inf.  A row with no logit above -inf has lse = -inf, logprob = -inf, entropy = 0.
 * A NaN makes its row's lse, logprob and entropy NaN and is never an alternative.  So does
 * +inf (it leaves no distribution), which is the first alternative with logprob NaN.
 * Supported: 1 <= n_vocab <= 2^21, 0 <= top_k <= 32, inv_temperature > 0 and
 * finite, times log2(e) too (up to 2.35e38), 0 <= rows < 2^31 (0: no-op); logits aligned
 * to their type.
 */
size_t spd_token_logprobs_workspace_size(int64_t rows, int32_t n_vocab, int32_t top_k);
spd_status token_logprobs(int64_t rows, int32_t n_vocab, const void *logits, int32_t logits_bf16,
                          int64_t row_stride, const int32_t *targets, float inv_temperature,
                          float *logprob, float *entropy, float *lse, int32_t top_k, int32_t *top_ids,
                          float *top_logprobs, void *ws, size_t ws_bytes, void *stream);

/*
 * Trees of drafted tokens.  A tree of T <= 64 nodes is parents int32 [B][T]: node 0 is
 * the root (the last token of the sequence, whose keys and values are not in the cache
 * yet), parents[b][v] the node that v follows, smaller than v, and -1 for a root; a node
 * with parent -2, or one below such a node, is no node (trees of fewer than T nodes).  Any
 * other parent sets SPD_DEV_BAD_TREE and makes v no node.  A chain of drafted tokens is
 * parents = -1, 0, 1, 2, ...
 * seq_lens counts the cache alone: the nodes' keys and values are rows of their own, and
 * only an accepted path reaches the cache (kv_append_path), so no page holds a rejected
 * token and no summary has to be taken back.
 */

/*
 * tree_verify_attn -- attention of every node of a tree of drafted tokens over the whole
 * cache, its ancestors and itself (dense_verify_attn for drafts with alternatives).
 *
 * q: bf16 rows of H_q * D, node v of sequence b at row b * T + v, q_stride elements apart;
 * k_tree, v_tree likewise (H_kv * D), so all three may be views of one projection: strides
 * multiples of 8, at least the row's length.  Row (b, v) attends over cache tokens
 * 0 .. seq_lens[b] - 1 and over tree rows u for u = v and v's ancestors.  Outputs o bf16
 * [B][T][H_q][D] and lse fp32 [B][T][H_q] (may be NULL); the rows of what is no node are
 * o = 0, lse = -inf.  seq_lens[b] = 0 (a tree on an empty cache) is valid; a length that the
 * page table has no room for sets SPD_DEV_BAD_LEN and gives such rows to the whole sequence.  A page
 * id outside [0, num_phys_pages) sets SPD_DEV_BAD_PAGE and its tokens are not seen.
 * What is no node may hold anything in its rows of q, k_tree and v_tree, and what lies in a page behind the length
 * may too; a node's infinities and NaN reach only the rows that see it, those of a cached value every row of its
 * sequence and head.
 * The sums of values of one sign come out low by up to 0.01 % where a sequence is long, whatever its length.
 * Supported: 1 <= T <= 64, B * H_kv <= 16384, max_pages_per_seq * page_size <= 2^30.  The workspace needs no zeros.
 */
size_t spd_tree_verify_workspace_size(const spd_dims *dims, int32_t T);
spd_status tree_verify_attn(const spd_dims *dims, int32_t T, const spd_bf16 *q, int64_t q_stride,
                            const spd_bf16 *K, const spd_bf16 *V, const int32_t *page_table,
                            const int32_t *seq_lens, const spd_bf16 *k_tree, int64_t k_stride,
                            const spd_bf16 *v_tree, int64_t v_stride, const int32_t *parents,
                            float softmax_scale, spd_bf16 *o, float *lse, void *ws, size_t ws_bytes,
                            void *stream);

/*
 * spec_accept_tree -- a path through a tree of drafted tokens, accepted from given random
 * numbers so that the tokens follow the target's distribution whatever the tree proposes
 * (spec_accept for drafts with alternatives that were picked, not drawn: the most likely
 * tokens of a drafter, as many at a node as one likes).
 *
 * q_target fp32 [B][T][n_vocab]: the target's distribution behind each node (rows need not
 * be normalised); draft int32 [B][T]: the nodes' tokens (the root's is not read);
 * u_acc fp32 [B][T] and u_res fp32 [B]: uniform numbers in [0, 1).
 * The walk starts at node 0.  At a node with row q, weights are whole numbers on a 2^-40
 * grid, W(x) = floor(2^40 * min(q(x), 1)) (0 for q(x) <= 0 or NaN), R = sum W.  Its children c
 * are tried in ascending order, with token x = draft[c]: c is taken iff
 * floor(u_acc[c] * R) < W(x); otherwise R -= W(x) and W(x) = 0.  The walk goes on from the
 * taken child; where none is taken, the last token is the smallest x whose running sum of W
 * exceeds floor(u_res * R) (-1 where R = 0; u_res >= 1 draws the last x of positive
 * weight).  Every sum is exact, so results do not depend on any order.
 * Outputs: n_path int32 [B], the nodes walked, the root among them; path int32 [B][T], these
 * nodes, then -1; tokens int32 [B][T], what follows each of them (the next one's draft, at last
 * the drawn token), then -1.  Where node 0 is not a root, n_path = 0 and all else is -1.
 * A draft outside [0, n_vocab) that is tried is not taken and sets SPD_DEV_BAD_TOKEN.
 * A sequence with a copy that does not come within the limit keeps its n_path, path and tokens as they were (SPD_DEV_TIMEOUT);
 * waits of a sequence's CTAs for one another have the default limit at least.
 * Supported: 1 <= T <= 64, 1 <= n_vocab <= 2^21, B * 16 < 2^31; q_target 16-byte aligned.
 */
spd_status spec_accept_tree(int32_t B, int32_t T, int32_t n_vocab, const float *q_target,
                            const int32_t *draft, const int32_t *parents, const float *u_acc,
                            const float *u_res, int32_t *n_path, int32_t *path, int32_t *tokens,
                            void *stream);

/*
 * kv_append_path -- appends the accepted path's keys and values to the paged cache and
 * rebuilds the summaries of the pages they land in, in one kernel.
 *
 * For i < n_path[b]: row path[b][i] of k_tree and v_tree (rows as in tree_verify_attn) goes to
 * position seq_lens[b] + i, bit for bit; summ as kv_append_refresh leaves it; new_lens[b] =
 * seq_lens[b] + n_path[b] (new_lens int32 [B], not seq_lens itself).  A sequence with a path length
 * outside [0, T] or an entry outside [0, T) sets SPD_DEV_BAD_TREE, one with a length below 0 or no room
 * in the page table SPD_DEV_BAD_LEN: its cache is left as it was and new_lens[b] = seq_lens[b].  A page
 * id outside [0, num_phys_pages) sets SPD_DEV_BAD_PAGE and skips that page's tokens.
 * Supported: 1 <= T <= 64.  Sequences must not share the pages they append to.
 */
spd_status kv_append_path(const spd_dims *dims, int32_t T, spd_bf16 *K, spd_bf16 *V,
                          const int32_t *page_table, const int32_t *seq_lens, const spd_bf16 *k_tree,
                          int64_t k_stride, const spd_bf16 *v_tree, int64_t v_stride,
                          const int32_t *path, const int32_t *n_path, spd_bf16 *summ,
                          int32_t *new_lens, void *stream);

/*
 * kv_weights_update -- adds to every cached token the attention weight that the newest
 * queries gave it: what kv_evict goes by.
 *
 * w_in, w_out: fp32 [B][H_kv][max_pages_per_seq * page_size], one weight for a token of a KV
 * head.  q bf16 [B][T][H_q][D] and lse fp32 [B][T][H_q] are the inputs and the output of the
 * attention of the newest tokens (dense_verify_attn, sparse_decode_attn with T = 1, or
 * tree_verify_attn: then path and n_path tell which rows were accepted, and the cache
 * holds them already).  Sequence b has N = n_path[b] query rows path[b][0 .. N) (without path and n_path:
 * N = T rows in order), the i-th at position seq_lens[b] - N + i.  For t < seq_lens[b]:
 *   w_out[b][h][t] = (t < seq_lens[b] - N ? decay * w_in[b][h][t] : 0)
 *                  + sum over i, g with t <= position i of exp(softmax_scale * q . K[t] - lse)
 * (hq = h * G + g); other places of w_out are left as they were.  w_in may be w_out, or NULL (all
 * weights start from 0).  Rows with lse = -inf add nothing.
 * sel, nsel (both or neither; [B][H_kv][k_max] and [B][H_kv] as pages_score_select writes them): only
 * tokens of the selected pages get the sum, and only these pages are read.
 * A length outside the page table's room, or below N, sets SPD_DEV_BAD_LEN, a path entry or length
 * outside its range SPD_DEV_BAD_TREE: that sequence's weights are left as they were.  A page id outside
 * [0, num_phys_pages) sets SPD_DEV_BAD_PAGE and its tokens get no sum; a selection entry outside the
 * sequence's pages, or nsel outside [0, k_max], sets SPD_DEV_BAD_SEL and is passed over (nsel clamped).
 * Supported: 1 <= T <= 64; path and n_path go together; decay and softmax_scale finite; max_pages_per_seq *
 * page_size <= 2^30.
 */
spd_status kv_weights_update(const spd_dims *dims, int32_t T, const spd_bf16 *q, const float *lse,
                             const spd_bf16 *K, const int32_t *page_table, const int32_t *seq_lens,
                             const int32_t *path, const int32_t *n_path, const int32_t *sel,
                             const int32_t *nsel, int32_t k_max, float decay, float softmax_scale,
                             const float *w_in, float *w_out, void *stream);

/*
 * kv_evict -- shortens every sequence to `budget` tokens of each KV head: the first n_sink, the newest
 * n_recent, and of the others those of the largest weights.
 *
 * new_lens[b] = min(seq_lens[b], budget).  Each KV head keeps that many tokens of its own choice (weights fp32
 * [B][H_kv][max_pages_per_seq * page_size], compared as numbers, NaN below all; the lower position among
 * equals), in the order of their positions: the j-th kept one, kept[b][h][j] (int32 [B][H_kv][budget], its
 * old position), has its key and value copied from its page to slot j % page_size of page
 * dst_table[b][j / page_size], its weight to weights_out[b][h][j], and summ gets the new pages' minima and
 * maxima.  Places behind new_lens[b] are left as they were, and the old pages too: with dst_table as the
 * page table and new_lens as the lengths every call goes on over the shortened cache (rotated keys
 * keep their rotation), and the old pages are free.
 * dst_table is int32 [B][max_pages_per_seq]; its first ceil(new_lens[b] / page_size) pages must be pages that no
 * sequence of the call reads or writes otherwise (old pages may be shared by sequences).  weights_out is not
 * weights, new_lens not seq_lens.  A length that the page table has no room for sets SPD_DEV_BAD_LEN: nothing is
 * written for it but new_lens[b] = 0.  A page id outside [0, num_phys_pages) sets SPD_DEV_BAD_PAGE: tokens
 * read from it become zeros, a new page is skipped.
 * Supported: 1 <= budget, 0 <= n_sink, n_recent, n_sink + n_recent <= budget, max_pages_per_seq * page_size
 * <= 2^30, B * H_kv * max_pages_per_seq < 2^31.
 */
spd_status kv_evict(const spd_dims *dims, int32_t budget, int32_t n_sink, int32_t n_recent, spd_bf16 *K,
                    spd_bf16 *V, const int32_t *page_table, const int32_t *seq_lens,
                    const float *weights, const int32_t *dst_table, int32_t *kept, float *weights_out,
                    spd_bf16 *summ, int32_t *new_lens, void *stream);

/*
 * spd_round -- one S3R round captured as CUDA graphs: k sparse draft steps,
 * then dense verification of the k + 1 positions and exact speculative
 * sampling, replayed with one graph launch per part (S3R Table 7: drafting
 * runs under CUDA Graphs; "Draft (6Tq)" and "Verify (TV)" are its two parts).
 *
 * Draft step s (0 <= s < k), on lengths seq_lens[s][:] (which count the token
 * the step appends):
 *   kv_append_refresh(T = 1, k_draft[s], v_draft[s]);
 *   pages_score_select(q_draft[s]) into sel / nsel (reused by every step);
 *   sparse_decode_attn(q_draft[s]) -> o_draft[s], lse_draft[s].
 * Verification, on lengths seq_lens[k][:]:
 *   kv_append_refresh(T = k + 1, k_verify, v_verify)   (rewrites the positions);
 *   dense_verify_attn(T = k + 1, q_verify) -> o_verify, lse_verify;
 *   spec_accept(...) -> n_accepted, tokens            (skipped when n_vocab = 0).
 * Layouts: seq_lens int32 [k + 1][B]; q_draft bf16 [k][B][H_q][D]; k_draft,
 * v_draft bf16 [k][B][H_kv][D]; q_verify bf16 [B][k+1][H_q][D]; k_verify,
 * v_verify bf16 [B][k+1][H_kv][D]; o_draft [k][B][H_q][D]; lse_draft
 * [k][B][H_q] (may be NULL); o_verify / lse_verify as dense_verify_attn; the
 * sampling buffers as spec_accept.  The three workspaces are sized by the
 * matching *_workspace_size calls; the split counts and softmax_scale mean
 * what they mean in those calls.
 *
 * spd_round_create validates the descriptor, makes each call once on a
 * private stream under capture (so every argument error surfaces here, with
 * nothing launched) and instantiates the graphs; the buffers must stay valid
 * and keep their addresses for the life of the round.  spd_round_launch
 * replays part 0 (draft steps), 1 (verification) or 2 (both, in order) on
 * `stream`; replaying is the same computation as making the calls.  Make one
 * ordinary call of the library on the device before the first create.
 */
typedef struct {
    spd_dims dims;
    int32_t k; /* draft steps per round, 1 <= k <= 32 */
    spd_bf16 *K, *V, *summ;
    const int32_t *page_table;
    const int32_t *seq_lens;
    const spd_bf16 *q_draft, *k_draft, *v_draft;
    const spd_bf16 *q_verify, *k_verify, *v_verify;
    spd_budget_policy policy;
    int32_t k_max;
    int32_t *sel, *nsel;
    spd_bf16 *o_draft;
    float *lse_draft;
    spd_bf16 *o_verify;
    float *lse_verify;
    int32_t n_vocab;
    const float *p_draft, *q_target;
    const int32_t *draft_tokens;
    const float *u_acc, *u_res;
    int32_t *n_accepted, *tokens;
    void *ws_select;
    size_t ws_select_bytes;
    void *ws_sparse;
    size_t ws_sparse_bytes;
    void *ws_verify;
    size_t ws_verify_bytes;
    int32_t sparse_splits, verify_splits;
    float softmax_scale;
} spd_round_desc;

typedef struct spd_round_s spd_round;

spd_status spd_round_create(const spd_round_desc *desc, spd_round **out);
spd_status spd_round_launch(spd_round *round, int32_t part, void *stream);
void spd_round_destroy(spd_round *round);

#ifdef __cplusplus
}
#endif

#endif /* SPD_H */
