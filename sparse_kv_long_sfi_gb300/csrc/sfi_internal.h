// Internal interface between the C ABI layer (sfi_api.cu) and the kernel files.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/sfi.h"

namespace sfi {

// Tokens per sub-block: one page of the paged pool, one unit of TMA work, one
// mma.sync n-extent pair for a consumer warp.
constexpr int kSubTokens = 16;
// Consumer warps per attention CTA (each owns one sub-block of every stage).
constexpr int kConsumerWarps = 4;
// Rows of the query tile handled per (request, KV head): G <= 8 query heads share a KV head.
constexpr int kMaxGroup = 8;
// Query rows of one (request, KV head) unit in the multi-token kernels: tokens x G <= 16
// fill the whole M = 16 tile.
constexpr int kMaxRows = 16;
// Attention CTAs resident per SM (shared memory sized for this).
constexpr int kAttnCtasPerSm = 2;
// Splits of one unit that merge inside a thread-block cluster (portable cluster size);
// more splits merge through the global workspace.
constexpr int kMaxClusterSplits = 8;

// kModeMixed: one launch where each request is either fast (fast_ids) or slow
// (slow_ids: dense attention with scores); 1-D grid of work items.
enum AttnMode : int { kModeFast = 0, kModeDense = 1, kModeMixed = 2 };

struct AttnParams {
    const __nv_bfloat16 *q;  // [B][tokens][Hq][D]
    float *out;              // [B][tokens][Hq][D]
    float *lse;              // [B][tokens][Hq] or null
    float *scores;           // [B][Hkv][score_stride] or null
    int64_t score_stride;
    const int32_t *page_table;
    int32_t max_pages;
    int32_t num_pages;
    const int32_t *seq_lens;
    const int64_t *c_row_offset;
    const int32_t *c_capacity;
    const int32_t *c_count;
    int64_t c_total_rows;
    const int32_t *req_ids;
    int32_t hq, hkv, group;
    int32_t sink, recent;
    float scale;       // softmax scale
    float scale_log2;  // scale * log2(e)
    int32_t splits;
    // query tokens per request (positions L - tokens .. L - 1) and tile rows tokens x group
    int32_t tokens, rows;
    // mixed mode: request lists and per-mode split counts
    const int32_t *fast_ids;
    const int32_t *slow_ids;
    int32_t n_fast, n_slow, fast_splits, slow_splits;
    // sub-blocks per split in mixed mode (0: the mode's units split evenly into *_splits)
    int32_t fast_chunk_sb, slow_chunk_sb;
    int32_t early_prefetch;  // SFI_ATTN_EARLY_KV_PREFETCH: stream KV before the dependency wait
    int32_t withhold;        // SFI_ATTN_TEST_WITHHOLD: 1 + the stage whose copies are never issued (0 = none)
    // fused append of the current token (position L - 1), or null
    const __nv_bfloat16 *k_new;  // [B][Hkv][D]
    const __nv_bfloat16 *v_new;
    __nv_bfloat16 *k_pool_w;     // the paged pools, for the append's writes
    __nv_bfloat16 *v_pool_w;
    int32_t *ws_count;  // [units]
    float *ws_ml;       // [units][splits][rows per slot][2]
    float *ws_part;     // [units][splits][rows per slot][D]
    int32_t *dev_status;
};

struct AttnMaps {
    CUtensorMap pool_k, pool_v;  // rows = (page * Hkv + kv) * P + slot
    CUtensorMap comp_k, comp_v;  // rows = compact buffer rows (dummy copies of pool maps in dense mode)
};

// Workspace layout for `units` (request, KV head) pairs and `splits` splits: the split
// counters at the start, the partial states (data_bytes) at the end of a buffer of
// `bytes` bytes (0: exactly `total`).
struct WorkspaceLayout {
    size_t count_off, ml_off, part_off, data_bytes, total;
};
// Single-token launches keep kMaxGroup rows per partial slot, multi-token ones kMaxRows.
WorkspaceLayout workspace_layout(int64_t units, int splits, int head_dim, int rows = kMaxGroup, size_t bytes = 0);
WorkspaceLayout workspace_layout_slots(int64_t units, int64_t slots, int head_dim, int rows = kMaxGroup,
                                       size_t bytes = 0);

// Clusters of `size` attention CTAs (1..kMaxClusterSplits) the current device holds at
// once (the occupancy query of the head-dim-128 kernel, cached per device); 0 when the
// query fails or there is no device.
int attn_cluster_capacity(int size);

cudaError_t launch_attention(int head_dim, int mode, bool with_scores, const AttnMaps &maps, const AttnParams &p,
                             int batch, cudaStream_t stream);
// Multi-token launch: mode kModeFast (draft over the sparse state) or kModeDense
// (verification; scores written when p.scores is set).
cudaError_t launch_attention_multi(int head_dim, int mode, const AttnMaps &maps, const AttnParams &p, int batch,
                                   cudaStream_t stream);

struct TopkParams {
    const float *scores;
    int64_t score_stride;
    int32_t hkv;
    const int32_t *seq_lens;
    int32_t sink, recent;
    const int32_t *k_per_req;
    int32_t k_cap;
    int32_t *idx_out;
    int32_t *count_out;
    const int32_t *req_ids;
    int32_t *dev_status;
};
cudaError_t launch_select_topk(const TopkParams &p, int batch, cudaStream_t stream);

struct CopyParams {
    const __nv_bfloat16 *k_pool_src;
    const __nv_bfloat16 *v_pool_src;
    __nv_bfloat16 *k_pool_dst;
    __nv_bfloat16 *v_pool_dst;
    int32_t num_pages, max_pages;
    const int32_t *page_table;
    const int32_t *seq_lens;
    int32_t hkv, head_dim;
    const int32_t *req_ids;
    int32_t *dev_status;
    // append of the `tokens` newest tokens
    int32_t tokens;
    const __nv_bfloat16 *k_new;
    const __nv_bfloat16 *v_new;
    // compaction
    const int32_t *idx;
    const int32_t *count;
    int32_t k_cap, sink;
    __nv_bfloat16 *ck;
    __nv_bfloat16 *cv;
    int64_t c_total_rows;
    const int64_t *c_row_offset;
    const int32_t *c_capacity;
};
cudaError_t launch_paged_append(const CopyParams &p, int batch, cudaStream_t stream);
cudaError_t launch_compact_gather(const CopyParams &p, int batch, int max_rows, cudaStream_t stream);

// Helpers of the entry points (sfi_api.cu).
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned8(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
int sm_count_current_device();
float resolve_scale(const sfi_attn_shape *s);
sfi_status check_shape(const sfi_attn_shape *s);
sfi_status check_paged(const sfi_attn_shape *s, const sfi_paged_kv *kv);

struct NormRopeParams {
    const __nv_bfloat16 *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // elements between tokens
    const __nv_bfloat16 *q_weight, *k_weight;
    float eps;
    const uint64_t *turns;
    const uint8_t *axis;
    int32_t rot_dim, num_axes, interleaved;
    const int32_t *positions;  // [num_axes][all requests][tokens], or null
    int64_t axis_stride;       // entries of one axis
    int32_t tokens;
    const int32_t *new_lens;
    __nv_bfloat16 *q_out, *k_out, *k_pool, *v_pool;
    const int32_t *page_table, *seq_lens;
    int32_t max_pages, num_pages;
    int32_t hq, hkv;
    const int32_t *req_ids;
    int32_t *dev_status;
};
cudaError_t launch_qk_norm_rope(const NormRopeParams &p, int head_dim, int batch, cudaStream_t stream);

// The calls that copy to and from the 4-bit cache.
struct Kv4CopyParams {
    uint8_t *pool;
    float k_scale, v_scale;
    const int32_t *page_table, *seq_lens;
    int32_t max_pages, num_pages, hkv;
    const int32_t *req_ids;
    int32_t *dev_status;
    // append and read of `tokens` positions
    int32_t tokens;
    const int32_t *new_lens, *first;
    const __nv_bfloat16 *k_new, *v_new;
    int64_t k_stride, v_stride;  // elements between tokens of k_new, v_new
    __nv_bfloat16 *k_out, *v_out;
    // compaction
    const int32_t *idx, *count;
    int32_t k_cap, sink;
    uint8_t *c_pool;
    int64_t c_total_pages;
    const int64_t *c_page_offset;
    const int32_t *c_capacity;
};
cudaError_t launch_kv4_append(const Kv4CopyParams &p, int head_dim, int batch, cudaStream_t stream);
cudaError_t launch_kv4_read(const Kv4CopyParams &p, int head_dim, int batch, cudaStream_t stream);
cudaError_t launch_kv4_compact(const Kv4CopyParams &p, int head_dim, int batch, cudaStream_t stream);

struct Kv4AttnParams {
    const __nv_bfloat16 *q;
    float *out, *lse, *scores;
    int64_t score_stride;
    const uint8_t *pool;
    const int32_t *page_table, *seq_lens;
    int32_t max_pages, num_pages;
    const uint8_t *c_pool;  // compact blocks (fast step), or null
    int64_t c_total_pages;
    const int64_t *c_page_offset;
    const int32_t *c_capacity, *c_count;
    const int32_t *req_ids;
    int32_t first, batch;  // this launch takes the requests first .. first + batch - 1 of the call
    int32_t hq, hkv, group;
    int32_t tokens, rows;
    int32_t sink, recent;
    float k_mul;    // softmax scale * k_scale
    float v_scale;
    int32_t *ws_count;  // [CTAs], zero between launches: that of the CTA which a shared unit begins in
    float *ws_ml;       // [CTAs][2][16 rows][2]
    float *ws_part;     // [CTAs][2][16 rows][D]
    int32_t *dev_status;
};
// Requests of one launch (their page counts' prefix lies in shared memory), and CTAs of one.
constexpr int kKv4MaxBatch = 512;
constexpr int kKv4CtasPerSm = 2;
constexpr int kKv4MaxCtas = 512;
cudaError_t launch_kv4_attn(const Kv4AttnParams &p, int head_dim, cudaStream_t stream);

// Page operators.
struct PageMapParams {
    int32_t *page_table, *seq_lens, *ref_count;
    int32_t num_reqs, max_pages, num_pages;
};
struct PagePoolParams {
    void *const *pools;
    int32_t num_pools;
    int64_t page_bytes;
    int32_t num_pages;
};
size_t page_workspace_bytes(int32_t num_pages);
cudaError_t launch_page_copy(const PagePoolParams &q, const int32_t *src, const int32_t *dst, int n,
                             int32_t *dev_status, cudaStream_t stream);
cudaError_t launch_page_fork(const PageMapParams &m, const int32_t *src, const int32_t *dst, const int32_t *fork_lens,
                             int n, int32_t *dev_status, cudaStream_t stream);
cudaError_t launch_page_free(const PageMapParams &m, const int32_t *reqs, int n, int32_t *dev_status,
                             cudaStream_t stream);
cudaError_t launch_page_reserve(const PageMapParams &m, const PagePoolParams *q, const int32_t *new_lens,
                                const int32_t *reqs, int n, void *ws, int32_t *dev_status, cudaStream_t stream);
cudaError_t launch_page_compact(const PageMapParams &m, const PagePoolParams &q, int32_t *table_out, int32_t *ref_out,
                                int32_t *live_out, void *ws, int32_t *dev_status, cudaStream_t stream);

}  // namespace sfi
