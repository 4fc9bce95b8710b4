/*
 * sfi.h - C ABI of libsfi: Slow-Fast Inference (SFI) decode attention over a
 * sparse, recallable KV memory, for NVIDIA GB300 (sm_103a).
 *
 * Method: "Slow-Fast Inference: Training-Free Inference Acceleration via
 * Within-Sentence Support Stability" (Xie et al., 2026).
 *   Figure 2 caption: fast steps attend to a managed sparse state
 *     (sink + selected + recent); a slow step performs dense attention, collects
 *     masked attention logits over the allowed candidate set and invokes the
 *     Selector to refresh the selected memory for the next segment.
 *   Figure 3 caption: (A) the Selector and cache reorganisation of layer i run on
 *     an aux stream while the main stream computes layer i+1's attention;
 *     (B) sink and selected tokens are packed into a contiguous compact buffer and
 *     recent tokens are read in place from paged KV.
 *   Table 1: kernel-level sparse/dense speedup at KV length 16K, batch 16, bf16.
 * The same per-KV-head logit statistics are what "A Sparse Glimpse of the Whole:
 * Train-Free Self-Speculative Decoding" (SparseSpec-L, abstract) recycles as its
 * importance signal.
 *
 * Notation: B requests, Hq query heads, Hkv KV heads, G = Hq / Hkv, D head_dim,
 * P page size, L the current length of a request (the current token included),
 * S sink size, W recent-window size, k selected tokens per KV head.
 * Query head h reads KV head h / G. Softmax scale defaults to 1/sqrt(D).
 *
 * Sparse state of a request at length L (the fast step attends to exactly this):
 *   sink     positions [0, min(S, L))              compact rows [0, min(S, L))
 *   selected positions idx[0 .. count)             compact rows [S, S + count)
 *   recent   positions [max(S, L - W), L)          read in place from the pages
 * Candidates of a slow step at length L: C = [S, L - W) (empty when L <= S + W).
 *
 * Conventions for every entry point:
 *   - The caller owns every buffer. The library allocates nothing, frees nothing,
 *     never synchronises and never changes the current device. Device pointers
 *     must belong to the current device.
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL = legacy default stream)
 *     and runs asynchronously.
 *   - Host-side errors (a NULL pointer, an unsupported shape, a short workspace)
 *     are returned before anything is launched. A failed launch returns
 *     SFI_ERR_CUDA.
 *   - Device-side errors never trap: the kernel ORs an SFI_DEV_* bit into
 *     *dev_status (optional; may be NULL) and skips the offending unit's writes.
 *     In the attention calls the unit is a (request, KV head), or what the call says:
 *     when any of its page ids is out of range, or one of its waits runs out, none of
 *     its outputs, log-sum-exps or score entries is written (the caller's values stay),
 *     in every split plan; other units are unaffected.
 *   - Per-request arrays (q, out, lse, scores, seq_lens, page_table rows,
 *     k_per_req, counts, compact rows) are indexed by the request id r. An entry
 *     point processes `batch` requests: r = req_ids[b] when req_ids is non-NULL
 *     (a subset of a larger batch, e.g. the slow subset of a mixed step), else
 *     r = b. req_ids must not repeat an id within one call. A call that is not told how
 *     many requests there are takes the ids as they are.
 *   - Supported: head_dim 64 or 128, page_size 16, G in {1, 2, 4, 8}. Q/K/V are
 *     bf16; outputs, LSE and scores are fp32 unless the call says otherwise; positions
 *     are int32.
 *   - LSE is the natural log of sum_j exp(scale * q . k_j) over the attended
 *     positions.
 */
#ifndef SFI_H
#define SFI_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SFI_VERSION 1

#if defined(__GNUC__)
#define SFI_API __attribute__((visibility("default")))
#else
#define SFI_API
#endif

typedef enum {
    SFI_OK = 0,
    SFI_ERR_INVALID_ARG = 1, /* NULL pointer, negative size, inconsistent shape */
    SFI_ERR_UNSUPPORTED = 2, /* head_dim, page_size or group size not supported */
    SFI_ERR_WORKSPACE = 3,   /* workspace missing or smaller than sfi_workspace_size() */
    SFI_ERR_CUDA = 4         /* a CUDA call or launch failed */
} sfi_status;

/* Bits ORed into *dev_status by the kernels (0 = no error). */
#define SFI_DEV_BAD_PAGE 1u     /* a page-table entry outside [0, num_pages) */
#define SFI_DEV_BAD_LEN 2u      /* seq_len < 1 or beyond the page table */
#define SFI_DEV_K_OVERFLOW 4u   /* k_r < 0, k_r > k_cap, or sink + count > capacity */
#define SFI_DEV_BAD_INDEX 8u    /* a selected position outside [0, L) */
#define SFI_DEV_TIMEOUT 16u     /* an in-kernel pipeline wait ran past its bound */
#define SFI_DEV_BAD_COMPACT 32u /* compact rows of a request fall outside the buffer */
#define SFI_DEV_NO_PAGE 64u     /* fewer free pages than a reservation needs */
#define SFI_DEV_BAD_PROB 128u   /* no probability above zero to sample from */

/* Launch flags of the attention entry points (bitwise OR). */
/* SFI_ATTN_EARLY_KV_PREFETCH: the kernel that precedes this call on the stream does
 * not write this call's paged KV pools, compact buffer, page table, lengths or
 * request ids, nor the compact counts and capacities. The
 * kernel may then start streaming them (programmatic dependent launch) before that
 * preceding kernel has finished; q, k_new and v_new are still read, and every output
 * written, only after it has finished. Without the flag nothing is read before then. */
#define SFI_ATTN_EARLY_KV_PREFETCH 1u
/* SFI_ATTN_RAGGED (sfi_fast_decode_attn and sfi_slow_dense_attn_with_scores): the
 * requests' lengths differ widely (a ragged batch). The launch is then planned in
 * fixed-size chunks, as sfi_mixed_decode_attn does (each (request, KV head) gets
 * splits in proportion to its real length, found on the device), instead of the same
 * number of splits for every request; num_splits is ignored and the workspace must
 * hold sfi_mixed_workspace_size(shape, batch, 0, max_tokens, 0) bytes for the fast
 * call and sfi_mixed_workspace_size(shape, 0, batch, 0, max_tokens) for the dense one. */
#define SFI_ATTN_RAGGED 2u
/* SFI_ATTN_TEST_WITHHOLD (the same two calls; diagnostic, for testing the bounded
 * in-kernel waits): the TMA producer of every CTA withholds the copies of its second
 * stage, so the consumers' wait for it runs out (after about 2 s) and the launch
 * reports SFI_DEV_TIMEOUT; the affected units write no output, the workspace is
 * left zeroed as after any launch, and the context stays usable. Units shorter than
 * two stages are unaffected. Not for production use. */
#define SFI_ATTN_TEST_WITHHOLD 4u

/* Most query tokens per request in the multi-token calls (tokens x G must also be
 * <= 16: G = 2 allows 8 tokens, G = 4 four, G = 8 two). */
#define SFI_MAX_QUERY_TOKENS 16
/* Largest vocabulary of sfi_verify_tokens. */
#define SFI_MAX_VOCAB 1048576
/* Most requests in one sfi_page_reserve call. */
#define SFI_MAX_PAGE_REQS 1024
/* Most pages of a map in sfi_page_compact (its plan counts past the last one in 32 bits). */
#define SFI_MAX_COMPACT_PAGES 2147475456

/* Attention geometry shared by all calls. */
typedef struct {
    int32_t num_q_heads;  /* Hq */
    int32_t num_kv_heads; /* Hkv */
    int32_t head_dim;     /* D: 64 or 128 */
    int32_t page_size;    /* P: 16 */
    float softmax_scale;  /* <= 0 selects 1/sqrt(D) */
} sfi_attn_shape;

/* Paged bf16 KV cache (Figure 3: the dense KV is kept in pages and never discarded). */
typedef struct {
    void *k_pool;               /* bf16 [num_pages][Hkv][P][D], 16-byte aligned */
    void *v_pool;               /* bf16 [num_pages][Hkv][P][D], 16-byte aligned */
    int32_t num_pages;          /* pages in each pool */
    int32_t max_pages_per_req;  /* row stride of page_table */
    const int32_t *page_table;  /* int32 [B][max_pages_per_req]: page of positions [16p, 16p+16) */
    const int32_t *seq_lens;    /* int32 [B]: L of each request, current token included */
} sfi_paged_kv;

/* Compact buffer (Figure 3B: sink + selected packed contiguously), one per layer.
 * Row i of KV head h of request r is buffer row  row_offset[r] + h * capacity[r] + i,
 * each row D bf16 values. Rows [0, min(S, L)) hold the sink, rows [S, S + count[r])
 * the selection in ascending position order. */
typedef struct {
    void *k;                   /* bf16 [total_rows][D], 16-byte aligned */
    void *v;                   /* bf16 [total_rows][D], 16-byte aligned */
    int64_t total_rows;        /* rows in each of k and v */
    const int64_t *row_offset; /* int64 [B] */
    const int32_t *capacity;   /* int32 [B] rows per KV head, >= S + k_r */
    const int32_t *count;      /* int32 [B] selected rows per KV head (written by sfi_select_topk) */
} sfi_compact_kv;

/*
 * sfi_paged_kv_append - write the current token's K and V into the paged cache.
 * Figure 3 caption (paged KV). For each request r, position L_r - 1 (L_r =
 * seq_lens[r], which already counts the new token) receives k_new[r] and v_new[r]:
 * slot (L_r - 1) % P of page page_table[r][(L_r - 1) / P].
 *   k_new, v_new : bf16 [B][Hkv][D], indexed by request id like q
 * Device errors: SFI_DEV_BAD_LEN, SFI_DEV_BAD_PAGE (that request is skipped).
 */
SFI_API sfi_status sfi_paged_kv_append(const sfi_attn_shape *shape, const sfi_paged_kv *kv, const void *k_new,
                               const void *v_new, const int32_t *req_ids, int32_t batch, int32_t *dev_status,
                               void *stream);

/*
 * sfi_fast_decode_attn - the fast step (Figure 2: attention over sink + selected +
 * recent; Figure 3B: the compact segment is streamed contiguously, the recent
 * segment is gathered page by page in place).
 * Each query head h of request r attends, with one softmax, to compact rows
 * [0, min(S, L) + count[r]) of KV head h / G followed by paged positions
 * [max(S, L - W), L). The compact buffer must have been filled by
 * sfi_compact_gather at a length >= min(S, L) (the sink is complete).
 *   q       : bf16 [B][Hq][D]
 *   k_new, v_new : bf16 [B][Hkv][D] or both NULL. When given, the call first does
 *                what sfi_paged_kv_append does (the current token goes to position
 *                L - 1 of the pages) and attends to the cache after that append;
 *                when L <= S the token is a sink row and is used in place of compact
 *                row L - 1 (the compact buffer itself is not written).
 *   out     : fp32 [B][Hq][D], 8-byte aligned
 *   lse     : fp32 [B][Hq] or NULL
 *   max_tokens : an upper bound on S + max count + W + P over the batch, used to
 *                plan split-KV; 0 lets the library assume the compact capacity
 *                is small. It affects speed only, never results.
 *   num_splits : 0 = automatic; otherwise the number of KV splits per
 *                (request, KV head) (clamped to the plan's maximum).
 *   flags      : 0, SFI_ATTN_EARLY_KV_PREFETCH and/or SFI_ATTN_RAGGED (and the diagnostic
 *                SFI_ATTN_TEST_WITHHOLD).
 *   workspace  : at least sfi_workspace_size(shape, batch, max_tokens, num_splits)
 *                bytes of device memory, zero-filled before its first use. The
 *                kernels leave its split counters zero-filled again when they
 *                finish, device errors and timed-out waits included (every split
 *                of a unit reaches the counter). Launches that share one
 *                workspace must not overlap in time.
 * Device errors: SFI_DEV_BAD_LEN, SFI_DEV_BAD_PAGE, SFI_DEV_K_OVERFLOW,
 * SFI_DEV_BAD_COMPACT, SFI_DEV_TIMEOUT.
 */
SFI_API sfi_status sfi_fast_decode_attn(const sfi_attn_shape *shape, const sfi_paged_kv *kv, const sfi_compact_kv *compact,
                                int32_t sink, int32_t recent, const void *q, const void *k_new, const void *v_new,
                                float *out, float *lse,
                                const int32_t *req_ids, int32_t batch, int32_t max_tokens, int32_t num_splits, uint32_t flags,
                                void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream);

/*
 * sfi_slow_dense_attn_with_scores - the slow step (Figure 2 caption: dense
 * attention plus the masked attention logits over the candidate set).
 * Each query head attends to all positions [0, L) of its KV head through the page
 * table. When scores is non-NULL it also writes, for every KV head kv,
 *   scores[r][kv][j] = sum_{g < G} scale * q_{kv*G+g} . k_{kv,j}   for j in [S, L - W)
 *   scores[r][kv][j] = -inf                                        for other j < L
 * in fp32; entries j >= L are not written. With scores == NULL this is the dense
 * full-KV decode attention (the denominator of Table 1).
 *   k_new, v_new : bf16 [B][Hkv][D] or both NULL: the current token, appended at
 *                  position L - 1 before the attention (as sfi_paged_kv_append)
 *   scores       : fp32 [B][Hkv][score_stride], score_stride >= max L, or NULL
 *   max_tokens   : an upper bound on L + P over the batch (split planning only)
 *   num_splits, flags, workspace, workspace_bytes : as for sfi_fast_decode_attn
 * Device errors: SFI_DEV_BAD_LEN (also when L > score_stride: the scores of that
 * request are then not written), SFI_DEV_BAD_PAGE, SFI_DEV_TIMEOUT.
 */
SFI_API sfi_status sfi_slow_dense_attn_with_scores(const sfi_attn_shape *shape, const sfi_paged_kv *kv, int32_t sink,
                                           int32_t recent, const void *q, const void *k_new, const void *v_new,
                                           float *out, float *lse, float *scores,
                                           int64_t score_stride, const int32_t *req_ids, int32_t batch,
                                           int32_t max_tokens, int32_t num_splits, uint32_t flags, void *workspace,
                                           size_t workspace_bytes, int32_t *dev_status, void *stream);

/*
 * sfi_mixed_decode_attn - one launch for a batch whose requests are at different
 * steps: the requests fast_ids[0 .. n_fast) do the fast step of
 * sfi_fast_decode_attn, the requests slow_ids[0 .. n_slow) the slow step of
 * sfi_slow_dense_attn_with_scores (dense attention, plus the masked scores when
 * scores is non-NULL). "ASPIRE: Asynchronous Batched Self-Speculative Decoding for
 * Long-Context LLM Inference" (abstract): drafting and verifying requests coexist in
 * the same batched forward pass; SFI (Figure 2 caption): each request takes fast steps
 * and, at its own boundaries, slow steps. A request id must appear in at most one of
 * the two lists.
 *   q, k_new, v_new, out, lse, scores, score_stride : as for the two calls above
 *   compact          : required when n_fast > 0
 *   max_fast_tokens  : an upper bound on S + max count + W + P over the fast requests
 *   max_dense_tokens : an upper bound on L + P over the slow requests
 *   flags            : 0 or SFI_ATTN_EARLY_KV_PREFETCH
 *   workspace        : at least sfi_mixed_workspace_size(...) bytes, zero-filled before
 *                      its first use (left zero-filled after each launch without
 *                      device error); launches sharing it must not overlap.
 * Device errors: those of sfi_fast_decode_attn and sfi_slow_dense_attn_with_scores.
 */
SFI_API sfi_status sfi_mixed_decode_attn(const sfi_attn_shape *shape, const sfi_paged_kv *kv,
                                         const sfi_compact_kv *compact, int32_t sink, int32_t recent, const void *q,
                                         const void *k_new, const void *v_new, float *out, float *lse, float *scores,
                                         int64_t score_stride, const int32_t *fast_ids, int32_t n_fast,
                                         const int32_t *slow_ids, int32_t n_slow, int32_t max_fast_tokens,
                                         int32_t max_dense_tokens, uint32_t flags, void *workspace,
                                         size_t workspace_bytes, int32_t *dev_status, void *stream);

/* Workspace bytes sfi_mixed_decode_attn needs for these arguments on the current
 * device (0 when it needs none). With one of n_fast, n_slow zero (the SFI_ATTN_RAGGED
 * plans of the single-mode calls) the size is valid for every batch size up to the
 * other, as for sfi_workspace_size. */
SFI_API size_t sfi_mixed_workspace_size(const sfi_attn_shape *shape, int32_t n_fast, int32_t n_slow,
                                        int32_t max_fast_tokens, int32_t max_dense_tokens);

/*
 * Multi-token calls. "A Sparse Glimpse of the Whole: Train-Free Self-Speculative
 * Decoding" (abstract): drafts come from the target model itself over the sparse,
 * recallable KV state; a full-context verification checks them and its per-head
 * attention statistics are recycled as the importance signal, with no extra forward.
 * Here a request carries T = num_tokens query tokens at positions L - T .. L - 1
 * (L = seq_lens[r] counts them). Query token t sees the context as it stands at length
 * L_t = L - T + t + 1 (causal).
 *   q   : bf16 [B][T][Hq][D], indexed by request id
 *   k_new, v_new : bf16 [B][T][Hkv][D] or both NULL. When given, the call first does
 *         what sfi_paged_kv_append_tokens does (the T tokens go to their page slots)
 *         and attends to the cache after that append; otherwise their K/V must already
 *         be in the pages. In the draft call the T positions must lie past the sink
 *         (L - T >= S): the compact buffer is not written.
 *   out : fp32 [B][T][Hq][D], 8-byte aligned;  lse : fp32 [B][T][Hq] or NULL
 * T x G > 16 returns SFI_ERR_UNSUPPORTED.
 */

/*
 * sfi_paged_kv_append_tokens - sfi_paged_kv_append for the T newest tokens: token t
 * of request r goes to position L_r - T + t.
 *   k_new, v_new : bf16 [B][T][Hkv][D], indexed by request id
 * Device errors: SFI_DEV_BAD_LEN (L < T), SFI_DEV_BAD_PAGE (that row is skipped).
 */
SFI_API sfi_status sfi_paged_kv_append_tokens(const sfi_attn_shape *shape, const sfi_paged_kv *kv, const void *k_new,
                                              const void *v_new, int32_t num_tokens, const int32_t *req_ids,
                                              int32_t batch, int32_t *dev_status, void *stream);

/*
 * sfi_dense_verify_attn - verification: token t of each request attends densely to
 * positions [0, L_t). When scores is non-NULL it writes the recycled statistic, for
 * every KV head kv:
 *   scores[r][kv][j] = sum over tokens t with j < L_t, sum_{g < G} of
 *                      scale * q_{t, kv*G+g} . k_{kv,j}          for j in [S, L - W)
 *   scores[r][kv][j] = -inf                                      for other j < L
 * (with T = 1 this is sfi_slow_dense_attn_with_scores). The Selector
 * (sfi_select_topk) then refreshes the selection from it; run it with the accepted
 * length, whose candidate set [S, L' - W) lies inside the scored one.
 *   scores, score_stride : as for sfi_slow_dense_attn_with_scores
 *   max_tokens : an upper bound on L + P over the batch (split planning only)
 *   num_splits, flags : as for sfi_fast_decode_attn (with k_new/v_new the append is
 *                part of the call, so SFI_ATTN_EARLY_KV_PREFETCH remains valid)
 *   workspace  : at least sfi_multi_workspace_size(shape, batch, T, max_tokens,
 *                num_splits) bytes, zero-filled before first use (kept so).
 * Device errors: SFI_DEV_BAD_LEN (also L < T, or L > score_stride), SFI_DEV_BAD_PAGE,
 * SFI_DEV_TIMEOUT.
 */
SFI_API sfi_status sfi_dense_verify_attn(const sfi_attn_shape *shape, const sfi_paged_kv *kv, int32_t sink,
                                         int32_t recent, const void *q, int32_t num_tokens, const void *k_new,
                                         const void *v_new, float *out, float *lse,
                                         float *scores, int64_t score_stride, const int32_t *req_ids, int32_t batch,
                                         int32_t max_tokens, int32_t num_splits, uint32_t flags, void *workspace,
                                         size_t workspace_bytes, int32_t *dev_status, void *stream);

/*
 * sfi_sparse_draft_attn - T draft tokens over the sparse state in one pass: token t
 * sees exactly what sfi_fast_decode_attn at length L_t sees, compact rows
 * [0, min(S, L_t) + count[r]) and the recent window [max(S, L_t - W), L_t); so the
 * result equals T single-token fast steps. A non-empty selection (count[r] > 0)
 * needs L - T + 1 >= S (else SFI_DEV_K_OVERFLOW). With T = 1 the call is
 * sfi_fast_decode_attn (same kernel; flags other than SFI_ATTN_EARLY_KV_PREFETCH are
 * ignored, and the token may also lie in the sink).
 *   max_tokens : an upper bound on S + max count + W + T + P (split planning only)
 *   num_splits, flags, workspace : as for sfi_dense_verify_attn
 * Device errors: those of sfi_fast_decode_attn.
 */
SFI_API sfi_status sfi_sparse_draft_attn(const sfi_attn_shape *shape, const sfi_paged_kv *kv,
                                         const sfi_compact_kv *compact, int32_t sink, int32_t recent, const void *q,
                                         int32_t num_tokens, const void *k_new, const void *v_new, float *out,
                                         float *lse, const int32_t *req_ids,
                                         int32_t batch, int32_t max_tokens, int32_t num_splits, uint32_t flags,
                                         void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream);

/* Workspace bytes the two multi-token attention calls need on the current device,
 * valid for every batch size 1..batch as for sfi_workspace_size (0 when none; 0 also
 * on invalid input). */
SFI_API size_t sfi_multi_workspace_size(const sfi_attn_shape *shape, int32_t batch, int32_t num_tokens,
                                        int32_t max_tokens, int32_t num_splits);

/*
 * sfi_select_topk - the Selector (Figure 2 caption): for every (request r, KV
 * head kv) keep the k_eff = min(k_per_req[r], |C|) candidates of C = [S, L - W)
 * with the largest score; equal scores go to the lower position; -0 equals +0;
 * NaN ranks below every number. The result is written in ascending position
 * order, and k_eff to count_out[r].
 *   scores    : fp32 [B][Hkv][score_stride] (as written by the slow step)
 *   seq_lens  : int32 [B] (L at the slow step)
 *   k_per_req : int32 [B], 0 <= k_r <= k_cap
 *   idx_out   : int32 [B][Hkv][k_cap]; entries past k_eff are not written
 *   count_out : int32 [B]
 * Limits: |C| <= 262144 candidates per request.
 * Device errors: SFI_DEV_K_OVERFLOW (also when |C| is past the limit),
 * SFI_DEV_BAD_LEN (L > score_stride); that request's outputs are not written.
 */
SFI_API sfi_status sfi_select_topk(const float *scores, int64_t score_stride, int32_t num_kv_heads, const int32_t *seq_lens,
                           int32_t sink, int32_t recent, const int32_t *k_per_req, int32_t k_cap, int32_t *idx_out,
                           int32_t *count_out, const int32_t *req_ids, int32_t batch, int32_t *dev_status,
                           void *stream);

/*
 * sfi_compact_gather - cache reorganisation (Figure 3: sink and selected tokens
 * packed into the contiguous compact buffer). For every (request, KV head):
 *   compact row i          <- paged position i          for i < min(S, L)
 *   compact row S + t      <- paged position idx[t]     for t < count[r]
 * for both K and V, copied bit for bit. `count` is the Selector's count_out and
 * normally the same array as compact->count.
 *   idx   : int32 [B][Hkv][k_cap] ascending positions (from sfi_select_topk)
 *   count : int32 [B]
 * Device errors: SFI_DEV_BAD_LEN, SFI_DEV_BAD_PAGE, SFI_DEV_BAD_INDEX,
 * SFI_DEV_K_OVERFLOW, SFI_DEV_BAD_COMPACT (offending rows are skipped).
 */
SFI_API sfi_status sfi_compact_gather(const sfi_attn_shape *shape, const sfi_paged_kv *kv, const int32_t *idx,
                              const int32_t *count, int32_t k_cap, int32_t sink, const sfi_compact_kv *compact,
                              const int32_t *req_ids, int32_t batch, int32_t *dev_status, void *stream);

/*
 * sfi_select_compact - sfi_select_topk followed by sfi_compact_gather in one call
 * (Figure 2 caption: the Selector refreshes the selected memory; Figure 3: cache
 * reorganisation into the contiguous compact buffer): the two kernels are launched in
 * sequence on the stream, with count = count_out.
 *   scores, score_stride, k_per_req, k_cap, idx_out : as for sfi_select_topk
 *   count_out : int32 [B], normally the same array as compact->count
 *   kv->seq_lens gives L (as for both calls)
 * Device errors: those of the two calls (a request with an invalid compact layout
 * keeps its selection but is not packed).
 */
SFI_API sfi_status sfi_select_compact(const sfi_attn_shape *shape, const sfi_paged_kv *kv, const float *scores,
                                      int64_t score_stride, int32_t sink, int32_t recent, const int32_t *k_per_req,
                                      int32_t k_cap, int32_t *idx_out, int32_t *count_out,
                                      const sfi_compact_kv *compact, const int32_t *req_ids, int32_t batch,
                                      int32_t *dev_status, void *stream);

/*
 * sfi_fast_decode_attn_noalloc - the fast step of sfi_fast_decode_attn for callers
 * that cannot allocate device memory. The paper has no counterpart to this call; it
 * exists for users of this library.
 * Who needs it: sfi_fast_decode_attn wants a caller-provided device workspace for
 * its split-KV partial results. A plugin running inside a host application that owns
 * every device allocation, or a latency-critical path that must not call cudaMalloc
 * (which can synchronise the whole device), has no way to provide one. This call
 * takes the same inputs and outputs, minus the workspace, and uses instead a fixed
 * array of SFI_NOALLOC_SCRATCH_BYTES inside the library's device memory. Every GPU
 * that loads the library holds that array until the process exits.
 *   - It calls no cudaMalloc, cudaFree or other allocating routine.
 *   - Its first call on a device looks up the array's device address on that device
 *     (cudaGetSymbolAddress, with that device current); make that first call before
 *     any stream capture.
 *   - The looked-up address is kept for the life of the process: a device reset
 *     (cudaDeviceReset) after the first call on a device is not supported.
 *   - Returns SFI_ERR_WORKSPACE when the split plan for these arguments needs more
 *     than SFI_NOALLOC_SCRATCH_BYTES (sfi_workspace_size tells the need, or
 *     sfi_mixed_workspace_size(shape, batch, 0, max_tokens, 0) with SFI_ATTN_RAGGED);
 *     reduce num_splits or the batch per call.
 *   - All calls on a device share the one array, which keeps what the last call left
 *     in it. A call whose plan uses the array (more than 8 splits, or any chunked
 *     plan of more than one chunk under SFI_ATTN_RAGGED) first zeroes its split
 *     counters with an async memset on `stream`; a plan that merges inside a
 *     thread-block cluster uses no scratch and issues no memset. Calls whose work can
 *     overlap on the GPU (for example on two streams) race on the array: order them
 *     on one stream.
 * Arguments, results and device errors are those of sfi_fast_decode_attn.
 */
#define SFI_NOALLOC_SCRATCH_BYTES (4u << 20)
SFI_API sfi_status sfi_fast_decode_attn_noalloc(const sfi_attn_shape *shape, const sfi_paged_kv *kv,
                                                const sfi_compact_kv *compact, int32_t sink, int32_t recent,
                                                const void *q, const void *k_new, const void *v_new, float *out,
                                                float *lse, const int32_t *req_ids,
                                                int32_t batch, int32_t max_tokens, int32_t num_splits, uint32_t flags,
                                                int32_t *dev_status, void *stream);

/*
 * sfi_workspace_size - bytes of workspace the attention entry points need for this
 * batch, token bound and split request on the current device, valid for every batch
 * size 1..batch (calls on a subset of the requests plan their splits for the subset):
 * one split counter per (request, KV head) at the start of the buffer, and the largest
 * block of split-KV partial states of those plans, which each call places at the end
 * of the buffer it is given. So calls with different batch sizes may share one buffer
 * (one at a time) when it holds the size for the largest of them. Returns 0 when no
 * plan needs any (at most 8 splits: the splits of a unit merge inside a thread-block
 * cluster) and on invalid input.
 */
SFI_API size_t sfi_workspace_size(const sfi_attn_shape *shape, int32_t batch, int32_t max_tokens, int32_t num_splits);

/*
 * sfi_plan_splits - the split count the attention entry points will use for these
 * arguments on the current device (for reports and tests). 0 on invalid input.
 * Automatic plans (num_splits = 0) give the (request, KV head) units about 85% of one
 * wave of two CTAs per SM; a count between 8 and 16 becomes 8. Every split keeps at
 * least four stages of 64 tokens, or three while the plan stays at most 8 splits (the
 * splits of a unit then merge inside a thread-block cluster). A plan of 2..8 splits
 * also leaves a ninth of the SM slots free in whole clusters, by the count of
 * sfi_attn_cluster_capacity, one split fewer at a time until it does. An explicit
 * num_splits is honoured down to two stages per split.
 */
SFI_API int32_t sfi_plan_splits(const sfi_attn_shape *shape, int32_t batch, int32_t max_tokens, int32_t num_splits);

/*
 * sfi_attn_cluster_capacity - how many thread-block clusters of cluster_size attention
 * CTAs (1..8) the current device holds at once (its occupancy query for the attention
 * kernel, cached per device). A cluster is placed whole on one GPC, so this can be
 * below the SM slots divided by cluster_size. 0 on invalid input, when there is no
 * device, or when the query fails.
 */
SFI_API int32_t sfi_attn_cluster_capacity(int32_t cluster_size);

/*
 * Head norm and position rotation, into the cache. The attention calls above take Q
 * after, and keep K after, the norm of each head and the rotation by position; this
 * call makes both from the projections' output, in one pass.
 *
 * sfi_rope describes the rotation. Pair i of the rot_dim / 2 rotated pairs of a head
 * turns by pos * turns[i] / 2^64 whole turns, where pos is the token's position on axis
 * axis[i]: the product wraps modulo one turn exactly, so angles are as good at position
 * 2^31 as at 0. turns[i] = round(inv_freq[i] / (2 pi) * 2^64) modulo 2^64.
 */
typedef struct {
    const uint64_t *turns; /* [rot_dim / 2] */
    const uint8_t *axis;   /* [rot_dim / 2], each < num_axes; NULL: axis 0 */
    int32_t rot_dim;       /* rotated dims, the first of each head: a multiple of 16 up to D */
    int32_t num_axes;      /* position axes (1; or e.g. 3: time, height, width), 1..8 */
    int32_t interleaved;   /* 0: pair i is dims (i, i + rot_dim / 2); 1: dims (2i, 2i + 1) */
} sfi_rope;

/*
 * sfi_qk_norm_rope - for every new token and head: y = rotate(x * w / sqrt(mean(x^2) + eps)),
 * in fp32, rounded once to bf16. Token t < n_r of request r (n_r = new_lens[r], or T when
 * new_lens is NULL) has slot L_r - n_r + t; tokens t >= n_r are neither read nor written.
 *   q, k, v   : bf16; token t of request r starts at element (r T + t) * stride of each,
 *               its heads are contiguous ([Hq][D], [Hkv][D], [Hkv][D]), so the three may be
 *               parts of one fused projection. Strides (in elements) are multiples of 8,
 *               pointers 16-byte aligned. v may be NULL when kv is.
 *   rope      : NULL: no rotation
 *   q_weight, k_weight : bf16 [D], 16-byte aligned, or NULL: no norm for q (for k)
 *   positions : int32, axis a of token t of request r at a * axis_stride + r T + t; or NULL:
 *               the slot is the position on every axis. Positions may be negative.
 *   seq_lens  : int32 [B], the lengths L_r when kv is NULL (with kv its own are used), or NULL
 *   q_out     : bf16 [B][T][Hq][D]
 *   k_out     : bf16 [B][T][Hkv][D], or NULL
 *   kv        : the pages that receive K and V at the tokens' slots, or NULL (then rope
 *               needs positions or seq_lens)
 * Outputs must not overlap inputs. At least one of k_out and kv must be given. An attention
 * call that follows on the stream and reads the pages written here must not be given
 * SFI_ATTN_EARLY_KV_PREFETCH.
 * Device errors: SFI_DEV_BAD_LEN (n_r < 0, n_r > T, L_r < n_r, or L_r beyond the page
 * table: nothing of that request is written), SFI_DEV_BAD_PAGE (that token's K and V
 * are not written to the pages), SFI_DEV_BAD_INDEX (an axis[i] >= num_axes: pair i does
 * not turn).
 */
SFI_API sfi_status sfi_qk_norm_rope(const sfi_attn_shape *shape, const sfi_rope *rope, const void *q, int64_t q_stride,
                                    const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                                    const void *q_weight, const void *k_weight, float eps, const int32_t *positions,
                                    int64_t axis_stride, int32_t num_tokens, const int32_t *new_lens,
                                    const int32_t *seq_lens, void *q_out, void *k_out, const sfi_paged_kv *kv, const int32_t *req_ids, int32_t batch,
                                    int32_t *dev_status, void *stream);

/*
 * The cache held in 4 bits. A token's K (and V) row of one head is held in groups of 16
 * values along D: a scale s in e4m3 and 16 codes in e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and
 * their negatives); value = code * s * g, with one power of two g for all K (k_scale) and
 * one for all V (v_scale) of a cache. 4.5 bits a value. Quantisation: s = e4m3(min(amax /
 * (6 g), 448)), code = e2m1(x / (s g)), both to nearest with ties to even; s = 0 gives
 * zeros; a group with a NaN or an infinity gets the scale NaN and reads back as NaN.
 *
 * The block of one (page, KV head) has 18 D bytes (16-byte aligned, K and V together, so
 * that one contiguous read brings what 16 positions need):
 *   [0, 8D)    K codes: byte token * D/2 + d/2, the even d in the low four bits
 *   [8D, 9D)   K scales: byte token * D/16 + d/16
 *   [9D, 17D)  V codes, in the order the matrix instruction's lanes take them: for
 *              d = 64 a + 16 b + 8 c + 2 e + f and token = 4 t + 2 h + l the byte
 *              512 a + 128 e + 32 t + 16 f + 4 b + 2 h + c, l = 0 in the low four bits
 *   [17D, 18D) V scales: byte t * D/4 + 4 * (d/16) + token % 4, t = token / 4
 */
typedef struct {
    void *pool;                /* [num_pages][Hkv][18 D] bytes, 16-byte aligned */
    int32_t num_pages;
    int32_t max_pages_per_req; /* row stride of page_table */
    const int32_t *page_table; /* int32 [B][max_pages_per_req] */
    const int32_t *seq_lens;   /* int32 [B]: L of each request */
    float k_scale, v_scale;    /* powers of two */
} sfi_paged_kv4;

/* Sink and selected rows of one layer, packed into 4-bit blocks: block i of KV head h of
 * request r is block  page_offset[r] + h * capacity[r] + i;  its 16 rows are the compact
 * rows [16 i, 16 i + 16) (sink rows [0, min(S, L)), selection from row S on). */
typedef struct {
    void *pool;                 /* [total_pages][18 D] bytes, 16-byte aligned */
    int64_t total_pages;
    const int64_t *page_offset; /* int64 [B] */
    const int32_t *capacity;    /* int32 [B] blocks per KV head, >= (S + k_r + 15) / 16 */
    const int32_t *count;       /* int32 [B] selected rows per KV head */
} sfi_compact_kv4;

/*
 * sfi_kv4_append - quantise the n_r newest tokens of each request (n_r = new_lens[r], or
 * num_tokens when new_lens is NULL) into the pages: token t < n_r goes to position
 * L_r - n_r + t. Other positions of a page keep their bits. The requests of one call must
 * not share the pages they write.
 *   k_new, v_new : bf16, 16-byte aligned; token t of request r starts at element
 *                  (r num_tokens + t) * k_stride (v_stride), its heads are contiguous [Hkv][D];
 *                  strides are multiples of 8
 * Device errors: SFI_DEV_BAD_LEN (n_r < 0, n_r > num_tokens, L_r < n_r or L_r beyond the page
 * table: that request is skipped), SFI_DEV_BAD_PAGE (that page's tokens are skipped).
 */
SFI_API sfi_status sfi_kv4_append(const sfi_attn_shape *shape, const sfi_paged_kv4 *kv, const void *k_new,
                                  int64_t k_stride, const void *v_new, int64_t v_stride, int32_t num_tokens, const int32_t *new_lens,
                                  const int32_t *req_ids, int32_t batch, int32_t *dev_status, void *stream);

/*
 * sfi_kv4_read - the values the cache holds, e.g. for the attention of a prompt's next
 * chunk: row t of request r receives position first[r] + t (first NULL: position t), in
 * bf16 (exact unless out of bf16's range). Rows at positions >= L_r keep their contents.
 *   k_out, v_out : bf16 [B][num_tokens][Hkv][D], 16-byte aligned
 * Device errors: SFI_DEV_BAD_LEN (L_r < 0 or beyond the page table, or first[r] < 0: that
 * request is skipped), SFI_DEV_BAD_PAGE (that page's rows are skipped).
 */
SFI_API sfi_status sfi_kv4_read(const sfi_attn_shape *shape, const sfi_paged_kv4 *kv, void *k_out, void *v_out,
                                int32_t num_tokens, const int32_t *first, const int32_t *req_ids, int32_t batch,
                                int32_t *dev_status, void *stream);

/*
 * sfi_kv4_compact_gather - sfi_compact_gather for the 4-bit cache: the codes and scales of
 * sink and selected rows move as they are (nothing is quantised again). Every block up to
 * (rows + 15) / 16 is written whole; rows that hold nothing become zeros.
 *   idx   : int32 [B][Hkv][k_cap] ascending positions;  count : int32 [B]
 * Device errors: SFI_DEV_BAD_LEN, SFI_DEV_K_OVERFLOW, SFI_DEV_BAD_COMPACT (that request is
 * skipped), SFI_DEV_BAD_INDEX, SFI_DEV_BAD_PAGE (that row becomes zeros).
 */
SFI_API sfi_status sfi_kv4_compact_gather(const sfi_attn_shape *shape, const sfi_paged_kv4 *kv, const int32_t *idx,
                                          const int32_t *count, int32_t k_cap, int32_t sink,
                                          const sfi_compact_kv4 *compact, const int32_t *req_ids, int32_t batch,
                                          int32_t *dev_status, void *stream);

/*
 * sfi_kv4_dense_attn - sfi_dense_verify_attn (num_tokens query tokens, causal; with one
 * token sfi_slow_dense_attn_with_scores) over the 4-bit cache, whose newest tokens are in
 * the pages already. The work is split over the GPU by the requests' real lengths (few
 * requests with narrow page tables: by KV head), so the call takes no bound on them.
 * num_tokens x G <= 16.
 *   q : bf16 [B][num_tokens][Hq][D];  out : fp32 of that shape, 8-byte aligned
 *   lse : fp32 [B][num_tokens][Hq] or NULL;  scores, score_stride : as there, or NULL
 *   workspace : sfi_kv4_workspace_size(shape, batch, num_tokens) bytes, 256-byte aligned,
 *               zero-filled before its first use (its counters are left zero); calls of
 *               other shapes may use it too, when it holds their size; launches sharing it
 *               must not overlap, those of captured graphs included
 * Device errors: SFI_DEV_BAD_LEN (also L < num_tokens, or L > score_stride), SFI_DEV_BAD_PAGE.
 */
SFI_API sfi_status sfi_kv4_dense_attn(const sfi_attn_shape *shape, const sfi_paged_kv4 *kv, int32_t sink,
                                      int32_t recent, const void *q, int32_t num_tokens, float *out, float *lse,
                                      float *scores, int64_t score_stride, const int32_t *req_ids, int32_t batch,
                                      void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream);

/*
 * sfi_kv4_fast_attn - sfi_sparse_draft_attn (with one token sfi_fast_decode_attn) over the
 * 4-bit compact blocks and the recent window of the 4-bit pages. A query token that sees
 * nothing (no sink, no selection, recent = 0) gets out = 0 and lse = -inf.
 *   other arguments : as for sfi_kv4_dense_attn
 * Device errors: SFI_DEV_BAD_LEN, SFI_DEV_BAD_PAGE, SFI_DEV_K_OVERFLOW, SFI_DEV_BAD_COMPACT.
 */
SFI_API sfi_status sfi_kv4_fast_attn(const sfi_attn_shape *shape, const sfi_paged_kv4 *kv,
                                     const sfi_compact_kv4 *compact, int32_t sink, int32_t recent, const void *q,
                                     int32_t num_tokens, float *out, float *lse, const int32_t *req_ids,
                                     int32_t batch, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                                     void *stream);

/* Workspace bytes of the two 4-bit attention calls on the current device, valid for every
 * batch size 1..batch and every num_tokens up to the given one (0 on invalid input). */
SFI_API size_t sfi_kv4_workspace_size(const sfi_attn_shape *shape, int32_t batch, int32_t num_tokens);

/*
 * Pages shared between requests. A page id names the same page in every pool of a cache
 * (each layer's K and V, or the 4-bit pools). ref_count[p] says how many requests hold
 * page p (0: free); request r holds the pages page_table[r][0 .. (seq_lens[r] + 15) / 16).
 * The calls keep all state on the device, and their results do not depend on the order in
 * which the GPU runs them: free pages are handed out lowest id first.
 */
typedef struct {
    int32_t *page_table;       /* int32 [num_reqs][max_pages_per_req] */
    int32_t *seq_lens;         /* int32 [num_reqs] */
    int32_t *ref_count;        /* int32 [num_pages] */
    int32_t num_reqs;
    int32_t max_pages_per_req;
    int32_t num_pages;
    int32_t page_size;         /* 16 */
} sfi_page_map;

typedef struct {
    void *const *pools;  /* device array of num_pools device pointers, each 16-byte aligned */
    int32_t num_pools;
    int64_t page_bytes;  /* bytes of a page in each pool, a multiple of 16 */
    int32_t num_pages;   /* pages of each pool */
} sfi_page_pools;

/*
 * sfi_page_copy - page src[i] -> page dst[i] in every pool, i < n. No page may be a
 * destination twice, or both a source and a destination.
 * Device errors: SFI_DEV_BAD_PAGE (that pair is skipped).
 */
SFI_API sfi_status sfi_page_copy(const sfi_page_pools *pools, const int32_t *src, const int32_t *dst, int32_t n,
                                 int32_t *dev_status, void *stream);

/*
 * sfi_page_fork - request dst[i] becomes a branch of request src[i]: it holds the pages of
 * the first fork_lens[i] tokens (NULL: all of them), and its length is that. No page is
 * copied; sfi_page_reserve copies what a branch is about to write. What dst[i] held before
 * is not released: free it first. A request may be the source of many branches, but the
 * destination of one, and not both.
 * Device errors: SFI_DEV_BAD_INDEX (a request id out of range, or src[i] == dst[i]),
 * SFI_DEV_BAD_LEN (a length out of range), SFI_DEV_BAD_PAGE (the source holds an id out of
 * range): that branch is skipped.
 */
SFI_API sfi_status sfi_page_fork(const sfi_page_map *map, const int32_t *src, const int32_t *dst,
                                 const int32_t *fork_lens, int32_t n, int32_t *dev_status, void *stream);

/*
 * sfi_page_reserve - room for the next append: request reqs[i] (reqs NULL: request i) grows
 * to new_lens[i] >= its length, its part-filled last page becomes its own (when others hold
 * it too, it is copied in every pool to a free page; of the holders in one call the last
 * in the list keeps the original if nobody else holds it), and free pages are taken for the
 * rest. Pages are handed out in the order of the list, then of positions, lowest id first.
 *   pools     : may be NULL when no request's last page is shared
 *   workspace : sfi_page_workspace_size(map) bytes, 16-byte aligned; no initial contents;
 *               launches sharing it must not overlap
 * n <= SFI_MAX_PAGE_REQS; a request may appear once. All or nothing: when a request is
 * refused or the free pages do not suffice, nothing changes.
 * Device errors: SFI_DEV_BAD_INDEX, SFI_DEV_BAD_LEN, SFI_DEV_BAD_PAGE, SFI_DEV_NO_PAGE.
 */
SFI_API sfi_status sfi_page_reserve(const sfi_page_map *map, const sfi_page_pools *pools, const int32_t *new_lens,
                                    const int32_t *reqs, int32_t n, void *workspace, size_t workspace_bytes,
                                    int32_t *dev_status, void *stream);

/*
 * sfi_page_free - request reqs[i] lets go of its pages (pages nobody holds are free again)
 * and has length 0. A request named twice lets go of them once.
 * Device errors: SFI_DEV_BAD_INDEX, SFI_DEV_BAD_LEN (that request is skipped),
 * SFI_DEV_BAD_PAGE (an id out of range, or a page with no holder left: that page is
 * skipped).
 */
SFI_API sfi_status sfi_page_free(const sfi_page_map *map, const int32_t *reqs, int32_t n, int32_t *dev_status,
                                 void *stream);

/*
 * sfi_page_compact - the live pages move to the front of the pools: with N pages held, the
 * j-th held page with an id >= N moves to the j-th free id below N, in every pool. The new
 * table and counts are written beside the old ones, which stay valid for reads already on
 * their way (only free pages are overwritten) until the caller changes over; whoever takes
 * pages in between must use the new ones. Table entries behind a request's length are
 * copied as they are.
 *   table_out : int32 [num_reqs][max_pages_per_req];  ref_out : int32 [num_pages]
 *   live_out  : int32 [1], N
 *   workspace : sfi_page_workspace_size(map) bytes, 16-byte aligned; no initial contents;
 *               launches sharing it must not overlap
 * table_out and ref_out must not be the map's own arrays.
 * num_pages <= SFI_MAX_COMPACT_PAGES.
 * Device errors: SFI_DEV_BAD_LEN, SFI_DEV_BAD_PAGE (entries that are out of range are copied
 * as they are).
 */
SFI_API sfi_status sfi_page_compact(const sfi_page_map *map, const sfi_page_pools *pools, int32_t *table_out,
                                    int32_t *ref_out, int32_t *live_out, void *workspace, size_t workspace_bytes,
                                    int32_t *dev_status, void *stream);

/*
 * sfi_page_trim - request reqs[i] (reqs NULL: request i) keeps its first new_lens[i] tokens: its
 * length becomes that, and the pages behind it are let go (pages nobody holds are free again).
 * The counterpart of sfi_page_reserve, for drafts that were refused and evicted caches. A request
 * may appear once.
 * Device errors: SFI_DEV_BAD_INDEX, SFI_DEV_BAD_LEN (a length below zero, above the request's or
 * beyond the table: that request is skipped), SFI_DEV_BAD_PAGE (an id out of range, or a page
 * with no holder left: that page is skipped).
 */
SFI_API sfi_status sfi_page_trim(const sfi_page_map *map, const int32_t *new_lens, const int32_t *reqs, int32_t n,
                                 int32_t *dev_status, void *stream);

/* Workspace bytes of sfi_page_reserve and sfi_page_compact (0 on invalid input). */
SFI_API size_t sfi_page_workspace_size(const sfi_page_map *map);

/*
 * Prompts, caches of a fixed size, drafts. A request's cache is written by its prompt, cut back to
 * the positions that attention has used most, and extended by drafts that the target verifies.
 */

/*
 * sfi_window_attn - attention of the n_r newest tokens of each request (n_r = new_lens[r], or
 * num_tokens when new_lens is NULL), whose K and V are in the pages already, through a sliding
 * window with sinks: the token at position p sees every j <= p with j < S or j > p - W (W >= L:
 * causal attention; the newest token of a request sees what sfi_fast_decode_attn sees with no
 * selection). Any number of tokens: a whole prompt, a chunk behind cached context, one step.
 *   q   : bf16, 16-byte aligned; token t of request r starts at element (r num_tokens + t) *
 *         q_stride, its heads are contiguous [Hq][D]; q_stride is a multiple of 8. q has num_reqs
 *         requests (request ids are below that). Token t < n_r is at position L_r - n_r + t.
 *   out : bf16 [B][num_tokens][Hq][D], 16-byte aligned (sums in fp32, rounded at the end). The weights
 *         that meet V have two bf16 terms in calls of up to 16 query rows per KV head (num_tokens G),
 *         one in longer calls (off by 2^-8 of sum w |v| at most).
 *   lse : fp32 [B][num_tokens][Hq] or NULL. Rows of tokens t >= n_r are not written. A token that
 *         sees nothing (S = 0, W = 0) gets out = 0 and lse = -inf.
 * What a token does not see has no influence on it, NaN and infinities included. Outputs must not
 * overlap inputs.
 * Device errors: SFI_DEV_BAD_INDEX (a request id outside [0, num_reqs)), SFI_DEV_BAD_LEN (n_r < 0,
 * n_r > num_tokens, L_r < n_r or L_r beyond the page table): that request is skipped.
 * SFI_DEV_BAD_PAGE, SFI_DEV_TIMEOUT (the tokens whose block reads that page are not written: up to
 * 256 / G tokens of a KV head's query heads; of up to 16 query rows per KV head, all of them).
 */
SFI_API sfi_status sfi_window_attn(const sfi_attn_shape *shape, const sfi_paged_kv *kv, int32_t sink, int32_t recent,
                                   const void *q, int64_t q_stride, int32_t num_reqs, int32_t num_tokens,
                                   const int32_t *new_lens, void *out, float *lse, const int32_t *req_ids,
                                   int32_t batch, int32_t *dev_status, void *stream);

/*
 * sfi_attn_mass - the attention weight that the new tokens gave to each position, summed over them
 * and over the query heads of each KV head:
 *   mass[r][kv][j] = decay * mass[r][kv][j] + sum over t, g of exp(scale q_{t, kv G + g} . k_j - lse_{t, kv G + g})
 * over the tokens that see j as in sfi_window_attn, for j < L_r. At the new positions (j >= L_r - n_r)
 * what mass held before does not count; with decay = 0 it does not anywhere. Entries j >= L_r are not
 * written. sfi_select_topk takes the result as scores; sfi_kv_evict keeps the heaviest positions.
 *   q, q_stride, num_reqs, num_tokens, new_lens : as for sfi_window_attn
 *   lse  : fp32 [B][num_tokens][Hq], of the attention of these tokens
 *   mass : fp32 [B][Hkv][mass_stride], mass_stride >= max L
 * The result does not depend on the order in which the GPU runs the call. A request may appear once in it.
 * Device errors: SFI_DEV_BAD_INDEX, SFI_DEV_BAD_LEN (as for sfi_window_attn, or L_r > mass_stride):
 * that request is skipped. SFI_DEV_BAD_PAGE, SFI_DEV_TIMEOUT (the block of positions that holds the page
 * is not written: 128 in calls of up to 128 query rows per KV head, else 256).
 */
SFI_API sfi_status sfi_attn_mass(const sfi_attn_shape *shape, const sfi_paged_kv *kv, int32_t sink, int32_t recent,
                                 const void *q, int64_t q_stride, int32_t num_reqs, int32_t num_tokens,
                                 const int32_t *new_lens, const float *lse, float *mass, int64_t mass_stride, float decay,
                                 const int32_t *req_ids, int32_t batch, int32_t *dev_status, void *stream);

/*
 * sfi_kv_evict - cut each request's cache, per KV head, to the sink [0, S), the recent window
 * [L - W, L) and the k_r = k_per_req[r] candidates between them with the largest mass (chosen as
 * sfi_select_topk does: equal ones go to the lower position). The kept rows of K and V move to the
 * front of the request's pages in place, in the order of their positions, bit for bit. All KV heads
 * keep equally many rows; seq_lens and the page table are not changed (they serve all layers): when
 * every layer is cut, sfi_page_trim takes the lengths over. The requests of one call must not share
 * the pages they hold (sfi_page_reserve gives a branch its last page only: do not evict from pages
 * with other holders).
 *   mass      : fp32 [B][Hkv][mass_stride], mass_stride >= max L
 *   k_per_req : int32 [B], 0 <= k_r <= k_cap
 *   idx_out   : int32 [B][Hkv][k_cap] (NULL when k_cap is 0), the kept candidates' former positions,
 *               ascending; entries past the count are not written
 *   count_out : int32 [B], min(k_r, candidates)
 *   mass_out  : fp32 [B][Hkv][mass_stride] or NULL: the kept rows' mass, in their new order; not mass
 *   new_lens  : int32 [B], the rows that are left; not seq_lens
 * A request may appear once in a call.
 * Limits: as for sfi_select_topk.
 * Device errors: SFI_DEV_BAD_LEN (L_r < 0, beyond the page table or > mass_stride), SFI_DEV_K_OVERFLOW:
 * nothing of that request is written. SFI_DEV_BAD_PAGE (that row stays as it was).
 */
SFI_API sfi_status sfi_kv_evict(const sfi_attn_shape *shape, const sfi_paged_kv *kv, const float *mass,
                                int64_t mass_stride, int32_t sink, int32_t recent, const int32_t *k_per_req,
                                int32_t k_cap, int32_t *idx_out, int32_t *count_out, float *mass_out,
                                int32_t *new_lens, const int32_t *req_ids, int32_t batch, int32_t *dev_status,
                                void *stream);

/*
 * sfi_verify_tokens - which drafted tokens the target keeps, and the token behind them, from given
 * random numbers. Request r has n_r = draft_lens[r] drafts x_t (num_drafts when draft_lens is NULL),
 * drawn from q_t; p_t is the target's distribution after t of them.
 *   Draft t is accepted while u_t q_t(x_t) < p_t(x_t); a is the number accepted.
 *   The next token is the first i with w_0 + ... + w_i > u_T (w_0 + ... + w_{V-1}), where w =
 *   max(p_a - q_a, 0) when a < n_r, else p_{n_r}; should that be zero everywhere, w = p_a.
 * With draft NULL the drafts were chosen, not drawn: q_t(x_t) = 1, and 0 elsewhere. The sums are
 * exact in units of 2^-56, so the result does not depend on any order.
 *   target : fp32, row t <= n_r of request r at element (r (num_drafts + 1) + t) * target_stride
 *   draft  : fp32, row t < n_r of request r at element (r num_drafts + t) * draft_stride, or NULL
 *            (values count as at least 0 and at most 1, a NaN as 0; a row's sum must stay below 64)
 *   tokens : int32 [B][num_drafts];  u : fp32 [B][num_drafts + 1] in [0, 1), u_T the last of a row
 *   out_tokens : int32 [B][num_drafts + 1]: the accepted drafts, the next token, then -1
 *   accepted   : int32 [B]: a
 *   seq_lens, new_lens : int32 [B] or both NULL: new_lens[r] = seq_lens[r] - n_r + a, the cache
 *            without the refused drafts (for sfi_page_trim)
 * vocab <= SFI_MAX_VOCAB.
 * Device errors: SFI_DEV_BAD_LEN (n_r < 0 or > num_drafts), SFI_DEV_BAD_INDEX (a draft outside the
 * vocabulary): that request is skipped. SFI_DEV_BAD_PROB (nothing to sample from: the next token is -1).
 */
SFI_API sfi_status sfi_verify_tokens(const float *target, int64_t target_stride, const float *draft,
                                     int64_t draft_stride, const int32_t *tokens, const float *u, int32_t vocab,
                                     int32_t num_drafts, const int32_t *draft_lens, const int32_t *seq_lens,
                                     int32_t *out_tokens, int32_t *accepted, int32_t *new_lens, const int32_t *req_ids,
                                     int32_t batch, int32_t *dev_status, void *stream);

/* Human-readable name of a status code (static string). */
SFI_API const char *sfi_status_string(sfi_status status);

/* SFI_VERSION of the built library. */
SFI_API int32_t sfi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SFI_H */
