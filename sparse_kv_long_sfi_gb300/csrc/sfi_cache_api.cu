// C ABI of the cache-side operators (declared in include/sfi.h): argument validation and
// kernel dispatch. Allocates nothing.
#include <algorithm>
#include <cmath>

#include "sfi_internal.h"

namespace {

using sfi::aligned16;
using sfi::aligned8;

sfi_status launched(cudaError_t e) { return e == cudaSuccess ? SFI_OK : SFI_ERR_CUDA; }

// A power of two well inside fp32's range (so that 6 g, s g and the softmax scale times g stay normal).
bool power_of_two(float g) {
    int e = 0;
    return std::isfinite(g) && std::frexp(g, &e) == 0.5f && e >= -63 && e <= 64;
}

sfi_status check_kv4(const sfi_attn_shape *s, const sfi_paged_kv4 *kv) {
    const sfi_status st = sfi::check_shape(s);
    if (st != SFI_OK) return st;
    if (!kv || !kv->pool || !kv->page_table || !kv->seq_lens) return SFI_ERR_INVALID_ARG;
    if (kv->num_pages <= 0 || kv->max_pages_per_req <= 0 || !aligned16(kv->pool)) return SFI_ERR_INVALID_ARG;
    if (!power_of_two(kv->k_scale) || !power_of_two(kv->v_scale)) return SFI_ERR_INVALID_ARG;
    if ((int64_t)kv->max_pages_per_req * s->page_size >= (int64_t(1) << 31)) return SFI_ERR_UNSUPPORTED;
    return SFI_OK;
}

sfi_status check_compact4(const sfi_compact_kv4 *c) {
    if (!c || !c->pool || !c->page_offset || !c->capacity || !c->count) return SFI_ERR_INVALID_ARG;
    return c->total_pages > 0 && aligned16(c->pool) ? SFI_OK : SFI_ERR_INVALID_ARG;
}

sfi::Kv4CopyParams copy_params(const sfi_attn_shape *shape, const sfi_paged_kv4 *kv, const int32_t *req_ids,
                               int32_t *dev_status) {
    sfi::Kv4CopyParams p{};
    p.pool = static_cast<uint8_t *>(kv->pool);
    p.k_scale = kv->k_scale;
    p.v_scale = kv->v_scale;
    p.page_table = kv->page_table;
    p.seq_lens = kv->seq_lens;
    p.max_pages = kv->max_pages_per_req;
    p.num_pages = kv->num_pages;
    p.hkv = shape->num_kv_heads;
    p.req_ids = req_ids;
    p.dev_status = dev_status;
    return p;
}

// Workspace of the 4-bit attention: a counter per CTA, then the partial states (m, l) and O of
// up to two units per CTA, sixteen rows each. The counters, which launches leave zero for the
// next one, take the same first 16 KB whatever the shape, so that calls of several shapes may
// share a workspace: no shape's partial states lie on another's counters.
struct Kv4Workspace {
    size_t ml, part, total;
};

Kv4Workspace kv4_workspace(const sfi_attn_shape *shape) {
    const int ctas = std::min(sfi::sm_count_current_device() * sfi::kKv4CtasPerSm, sfi::kKv4MaxCtas);
    const size_t slots = (size_t)ctas * 2 * sfi::kMaxRows;
    Kv4Workspace w{};
    w.ml = 16384;
    static_assert(sfi::kKv4MaxCtas * sizeof(int32_t) <= 16384, "a counter per CTA");
    w.part = w.ml + slots * 2 * 4;
    w.total = w.part + slots * shape->head_dim * 4;
    return w;
}

sfi_status kv4_attention(const sfi_attn_shape *shape, const sfi_paged_kv4 *kv, const sfi_compact_kv4 *compact,
                         int32_t sink, int32_t recent, const void *q, int32_t num_tokens, float *out, float *lse,
                         float *scores, int64_t score_stride, const int32_t *req_ids, int32_t batch, void *workspace,
                         size_t workspace_bytes, int32_t *dev_status, void *stream) {
    const sfi_status st = check_kv4(shape, kv);
    if (st != SFI_OK) return st;
    if (batch < 0 || sink < 0 || recent < 0 || !q || !out || !aligned16(q) || !aligned8(out))
        return SFI_ERR_INVALID_ARG;
    if (num_tokens < 1 || num_tokens > SFI_MAX_QUERY_TOKENS || (scores && score_stride <= 0))
        return SFI_ERR_INVALID_ARG;
    const int group = shape->num_q_heads / shape->num_kv_heads;
    if (num_tokens * group > sfi::kMaxRows) return SFI_ERR_UNSUPPORTED;
    // a warp counts its blocks in 32 bits
    if ((int64_t)shape->num_kv_heads * kv->max_pages_per_req >= (int64_t(1) << 31)) return SFI_ERR_UNSUPPORTED;
    if (batch == 0) return SFI_OK;
    const Kv4Workspace w = kv4_workspace(shape);
    if (!workspace || workspace_bytes < w.total || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return SFI_ERR_WORKSPACE;
    char *ws = static_cast<char *>(workspace);
    sfi::Kv4AttnParams p{};
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.out = out;
    p.lse = lse;
    p.scores = scores;
    p.score_stride = score_stride;
    p.pool = static_cast<const uint8_t *>(kv->pool);
    p.page_table = kv->page_table;
    p.seq_lens = kv->seq_lens;
    p.max_pages = kv->max_pages_per_req;
    p.num_pages = kv->num_pages;
    if (compact) {
        p.c_pool = static_cast<const uint8_t *>(compact->pool);
        p.c_total_pages = compact->total_pages;
        p.c_page_offset = compact->page_offset;
        p.c_capacity = compact->capacity;
        p.c_count = compact->count;
    }
    p.hq = shape->num_q_heads;
    p.hkv = shape->num_kv_heads;
    p.group = group;
    p.tokens = num_tokens;
    p.rows = num_tokens * group;
    p.sink = sink;
    p.recent = recent;
    p.k_mul = sfi::resolve_scale(shape) * kv->k_scale;
    p.v_scale = kv->v_scale;
    p.ws_count = reinterpret_cast<int32_t *>(ws);
    p.ws_ml = reinterpret_cast<float *>(ws + w.ml);
    p.ws_part = reinterpret_cast<float *>(ws + w.part);
    p.dev_status = dev_status;
    // more requests than one launch takes: launches in turn on the stream
    for (int32_t b = 0; b < batch; b += sfi::kKv4MaxBatch) {
        p.first = b;
        p.req_ids = req_ids;
        p.batch = batch - b < sfi::kKv4MaxBatch ? batch - b : sfi::kKv4MaxBatch;
        if (sfi::launch_kv4_attn(p, shape->head_dim, static_cast<cudaStream_t>(stream)) != cudaSuccess)
            return SFI_ERR_CUDA;
    }
    return SFI_OK;
}

sfi_status check_map(const sfi_page_map *m) {
    if (!m || !m->page_table || !m->seq_lens || !m->ref_count) return SFI_ERR_INVALID_ARG;
    if (m->num_reqs <= 0 || m->max_pages_per_req <= 0 || m->num_pages <= 0) return SFI_ERR_INVALID_ARG;
    if (m->page_size != sfi::kSubTokens) return SFI_ERR_UNSUPPORTED;
    if ((int64_t)m->max_pages_per_req * m->page_size >= (int64_t(1) << 31)) return SFI_ERR_UNSUPPORTED;
    return SFI_OK;
}

sfi_status check_pools(const sfi_page_pools *q) {
    if (!q || !q->pools || q->num_pools <= 0 || q->num_pages <= 0) return SFI_ERR_INVALID_ARG;
    return q->page_bytes > 0 && q->page_bytes % 16 == 0 ? SFI_OK : SFI_ERR_INVALID_ARG;
}

sfi::PageMapParams map_params(const sfi_page_map *m) {
    return {m->page_table, m->seq_lens, m->ref_count, m->num_reqs, m->max_pages_per_req, m->num_pages};
}

sfi::PagePoolParams pool_params(const sfi_page_pools *q) {
    return {q->pools, q->num_pools, q->page_bytes, q->num_pages};
}

}  // namespace

extern "C" {

sfi_status sfi_qk_norm_rope(const sfi_attn_shape *shape, const sfi_rope *rope, const void *q, int64_t q_stride,
                            const void *k, int64_t k_stride, const void *v, int64_t v_stride, const void *q_weight,
                            const void *k_weight, float eps, const int32_t *positions, int64_t axis_stride,
                            int32_t num_tokens, const int32_t *new_lens, const int32_t *seq_lens, void *q_out,
                            void *k_out, const sfi_paged_kv *kv, const int32_t *req_ids, int32_t batch, int32_t *dev_status,
                            void *stream) {
    sfi_status st = sfi::check_shape(shape);
    if (st != SFI_OK) return st;
    if (kv && (st = sfi::check_paged(shape, kv)) != SFI_OK) return st;
    if (!q || !k || !q_out || (!k_out && !kv) || (kv && !v)) return SFI_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_out) ||
        !aligned16(q_weight) || !aligned16(k_weight))
        return SFI_ERR_INVALID_ARG;
    const int64_t d = shape->head_dim;
    if (q_stride < shape->num_q_heads * d || k_stride < shape->num_kv_heads * d ||
        (v && v_stride < shape->num_kv_heads * d) || q_stride % 8 || k_stride % 8 || (v && v_stride % 8))
        return SFI_ERR_INVALID_ARG;
    if (batch < 0 || num_tokens < 1 || !std::isfinite(eps) || eps < 0.f) return SFI_ERR_INVALID_ARG;
    if (rope) {
        if (rope->rot_dim < 0 || rope->rot_dim > d || rope->rot_dim % 16) return SFI_ERR_UNSUPPORTED;
        if (!rope->turns || rope->num_axes < 1 || rope->num_axes > 8 || (rope->interleaved & ~1))
            return SFI_ERR_INVALID_ARG;
        if (!positions && !kv && !seq_lens) return SFI_ERR_INVALID_ARG;
        if (positions && rope->num_axes > 1 && axis_stride < num_tokens) return SFI_ERR_INVALID_ARG;
    }
    if (batch == 0) return SFI_OK;
    sfi::NormRopeParams p{};
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.v = kv ? static_cast<const __nv_bfloat16 *>(v) : nullptr;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_weight = static_cast<const __nv_bfloat16 *>(q_weight);
    p.k_weight = static_cast<const __nv_bfloat16 *>(k_weight);
    p.eps = eps;
    p.num_axes = 1;
    if (rope) {
        p.turns = rope->turns;
        p.axis = rope->axis;
        p.rot_dim = rope->rot_dim;
        p.num_axes = rope->num_axes;
        p.interleaved = rope->interleaved;
    }
    p.positions = positions;
    p.axis_stride = axis_stride;
    p.tokens = num_tokens;
    p.new_lens = new_lens;
    p.seq_lens = seq_lens;
    p.q_out = static_cast<__nv_bfloat16 *>(q_out);
    p.k_out = static_cast<__nv_bfloat16 *>(k_out);
    if (kv) {
        p.k_pool = static_cast<__nv_bfloat16 *>(kv->k_pool);
        p.v_pool = static_cast<__nv_bfloat16 *>(kv->v_pool);
        p.page_table = kv->page_table;
        p.seq_lens = kv->seq_lens;
        p.max_pages = kv->max_pages_per_req;
        p.num_pages = kv->num_pages;
    }
    p.hq = shape->num_q_heads;
    p.hkv = shape->num_kv_heads;
    p.req_ids = req_ids;
    p.dev_status = dev_status;
    return launched(sfi::launch_qk_norm_rope(p, shape->head_dim, batch, static_cast<cudaStream_t>(stream)));
}

sfi_status sfi_kv4_append(const sfi_attn_shape *shape, const sfi_paged_kv4 *kv, const void *k_new, int64_t k_stride,
                          const void *v_new, int64_t v_stride, int32_t num_tokens, const int32_t *new_lens, const int32_t *req_ids, int32_t batch,
                          int32_t *dev_status, void *stream) {
    const sfi_status st = check_kv4(shape, kv);
    if (st != SFI_OK) return st;
    if (!k_new || !v_new || !aligned16(k_new) || !aligned16(v_new) || num_tokens < 1 || batch < 0)
        return SFI_ERR_INVALID_ARG;
    const int64_t row = (int64_t)shape->num_kv_heads * shape->head_dim;
    if (k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8) return SFI_ERR_INVALID_ARG;
    if (batch == 0) return SFI_OK;
    sfi::Kv4CopyParams p = copy_params(shape, kv, req_ids, dev_status);
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.tokens = num_tokens;
    p.new_lens = new_lens;
    p.k_new = static_cast<const __nv_bfloat16 *>(k_new);
    p.v_new = static_cast<const __nv_bfloat16 *>(v_new);
    return launched(sfi::launch_kv4_append(p, shape->head_dim, batch, static_cast<cudaStream_t>(stream)));
}

sfi_status sfi_kv4_read(const sfi_attn_shape *shape, const sfi_paged_kv4 *kv, void *k_out, void *v_out,
                        int32_t num_tokens, const int32_t *first, const int32_t *req_ids, int32_t batch,
                        int32_t *dev_status, void *stream) {
    const sfi_status st = check_kv4(shape, kv);
    if (st != SFI_OK) return st;
    if (!k_out || !v_out || !aligned16(k_out) || !aligned16(v_out) || num_tokens < 1 || batch < 0)
        return SFI_ERR_INVALID_ARG;
    if (batch == 0) return SFI_OK;
    sfi::Kv4CopyParams p = copy_params(shape, kv, req_ids, dev_status);
    p.tokens = num_tokens;
    p.first = first;
    p.k_out = static_cast<__nv_bfloat16 *>(k_out);
    p.v_out = static_cast<__nv_bfloat16 *>(v_out);
    return launched(sfi::launch_kv4_read(p, shape->head_dim, batch, static_cast<cudaStream_t>(stream)));
}

sfi_status sfi_kv4_compact_gather(const sfi_attn_shape *shape, const sfi_paged_kv4 *kv, const int32_t *idx,
                                  const int32_t *count, int32_t k_cap, int32_t sink, const sfi_compact_kv4 *compact,
                                  const int32_t *req_ids, int32_t batch, int32_t *dev_status, void *stream) {
    sfi_status st = check_kv4(shape, kv);
    if (st != SFI_OK) return st;
    if ((st = check_compact4(compact)) != SFI_OK) return st;
    if (!idx || !count || k_cap < 0 || sink < 0 || batch < 0) return SFI_ERR_INVALID_ARG;
    if (batch == 0 || (int64_t)sink + k_cap == 0) return SFI_OK;
    if ((int64_t)sink + k_cap + 15 >= (int64_t(1) << 31)) return SFI_ERR_INVALID_ARG;
    sfi::Kv4CopyParams p = copy_params(shape, kv, req_ids, dev_status);
    p.idx = idx;
    p.count = count;
    p.k_cap = k_cap;
    p.sink = sink;
    p.c_pool = static_cast<uint8_t *>(compact->pool);
    p.c_total_pages = compact->total_pages;
    p.c_page_offset = compact->page_offset;
    p.c_capacity = compact->capacity;
    return launched(sfi::launch_kv4_compact(p, shape->head_dim, batch, static_cast<cudaStream_t>(stream)));
}

sfi_status sfi_kv4_dense_attn(const sfi_attn_shape *shape, const sfi_paged_kv4 *kv, int32_t sink, int32_t recent,
                              const void *q, int32_t num_tokens, float *out, float *lse, float *scores,
                              int64_t score_stride, const int32_t *req_ids, int32_t batch, void *workspace,
                              size_t workspace_bytes, int32_t *dev_status, void *stream) {
    return kv4_attention(shape, kv, nullptr, sink, recent, q, num_tokens, out, lse, scores, score_stride, req_ids,
                         batch, workspace, workspace_bytes, dev_status, stream);
}

sfi_status sfi_kv4_fast_attn(const sfi_attn_shape *shape, const sfi_paged_kv4 *kv, const sfi_compact_kv4 *compact,
                             int32_t sink, int32_t recent, const void *q, int32_t num_tokens, float *out, float *lse,
                             const int32_t *req_ids, int32_t batch, void *workspace, size_t workspace_bytes,
                             int32_t *dev_status, void *stream) {
    const sfi_status st = check_compact4(compact);
    if (st != SFI_OK) return st;
    return kv4_attention(shape, kv, compact, sink, recent, q, num_tokens, out, lse, nullptr, 0, req_ids, batch,
                         workspace, workspace_bytes, dev_status, stream);
}

size_t sfi_kv4_workspace_size(const sfi_attn_shape *shape, int32_t batch, int32_t num_tokens) {
    if (sfi::check_shape(shape) != SFI_OK || batch < 0 || num_tokens < 1 || num_tokens > SFI_MAX_QUERY_TOKENS) return 0;
    if (num_tokens * (shape->num_q_heads / shape->num_kv_heads) > sfi::kMaxRows) return 0;
    return kv4_workspace(shape).total;
}

sfi_status sfi_page_copy(const sfi_page_pools *pools, const int32_t *src, const int32_t *dst, int32_t n,
                         int32_t *dev_status, void *stream) {
    const sfi_status st = check_pools(pools);
    if (st != SFI_OK) return st;
    if (!src || !dst || n < 0) return SFI_ERR_INVALID_ARG;
    if (n == 0) return SFI_OK;
    return launched(
        sfi::launch_page_copy(pool_params(pools), src, dst, n, dev_status, static_cast<cudaStream_t>(stream)));
}

sfi_status sfi_page_fork(const sfi_page_map *map, const int32_t *src, const int32_t *dst, const int32_t *fork_lens,
                         int32_t n, int32_t *dev_status, void *stream) {
    const sfi_status st = check_map(map);
    if (st != SFI_OK) return st;
    if (!src || !dst || n < 0) return SFI_ERR_INVALID_ARG;
    if (n == 0) return SFI_OK;
    return launched(
        sfi::launch_page_fork(map_params(map), src, dst, fork_lens, n, dev_status, static_cast<cudaStream_t>(stream)));
}

sfi_status sfi_page_reserve(const sfi_page_map *map, const sfi_page_pools *pools, const int32_t *new_lens,
                            const int32_t *reqs, int32_t n, void *workspace, size_t workspace_bytes,
                            int32_t *dev_status, void *stream) {
    sfi_status st = check_map(map);
    if (st != SFI_OK) return st;
    if (pools && (st = check_pools(pools)) != SFI_OK) return st;
    if (!new_lens || n < 0 || (pools && pools->num_pages < map->num_pages)) return SFI_ERR_INVALID_ARG;
    if (!reqs && n > map->num_reqs) return SFI_ERR_INVALID_ARG;
    if (n > SFI_MAX_PAGE_REQS) return SFI_ERR_UNSUPPORTED;
    if (n == 0) return SFI_OK;
    if (!workspace || !aligned16(workspace) || workspace_bytes < sfi::page_workspace_bytes(map->num_pages))
        return SFI_ERR_WORKSPACE;
    sfi::PagePoolParams q{};
    if (pools) q = pool_params(pools);
    return launched(sfi::launch_page_reserve(map_params(map), pools ? &q : nullptr, new_lens, reqs, n, workspace,
                                             dev_status, static_cast<cudaStream_t>(stream)));
}

sfi_status sfi_page_free(const sfi_page_map *map, const int32_t *reqs, int32_t n, int32_t *dev_status, void *stream) {
    const sfi_status st = check_map(map);
    if (st != SFI_OK) return st;
    if (!reqs || n < 0) return SFI_ERR_INVALID_ARG;
    if (n == 0) return SFI_OK;
    return launched(sfi::launch_page_free(map_params(map), reqs, n, dev_status, static_cast<cudaStream_t>(stream)));
}

sfi_status sfi_page_compact(const sfi_page_map *map, const sfi_page_pools *pools, int32_t *table_out, int32_t *ref_out,
                            int32_t *live_out, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                            void *stream) {
    sfi_status st = check_map(map);
    if (st != SFI_OK) return st;
    if ((st = check_pools(pools)) != SFI_OK) return st;
    if (!table_out || !ref_out || !live_out || pools->num_pages < map->num_pages) return SFI_ERR_INVALID_ARG;
    if (table_out == map->page_table || ref_out == map->ref_count) return SFI_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace) || workspace_bytes < sfi::page_workspace_bytes(map->num_pages))
        return SFI_ERR_WORKSPACE;
    return launched(sfi::launch_page_compact(map_params(map), pool_params(pools), table_out, ref_out, live_out,
                                             workspace, dev_status, static_cast<cudaStream_t>(stream)));
}

size_t sfi_page_workspace_size(const sfi_page_map *map) {
    return check_map(map) == SFI_OK ? sfi::page_workspace_bytes(map->num_pages) : 0;
}

}  // extern "C"
