// C ABI of the operators around prompts, caches of a fixed size and drafts (declared in include/sfi.h):
// argument validation and kernel dispatch. Allocates nothing.
#include <algorithm>
#include <cmath>

#include "sfi_internal.h"

namespace {

using sfi::aligned16;

sfi_status launched(cudaError_t e) { return e == cudaSuccess ? SFI_OK : SFI_ERR_CUDA; }

// What sfi_window_attn and sfi_attn_mass have in common.
sfi_status window_params(const sfi_attn_shape *shape, const sfi_paged_kv *kv, int32_t sink, int32_t recent,
                         const void *q, int64_t q_stride, int32_t num_reqs, int32_t num_tokens, const int32_t *new_lens,
                         const int32_t *req_ids, int32_t batch, int32_t *dev_status, sfi::WindowParams &p) {
    sfi_status st = sfi::check_shape(shape);
    if (st != SFI_OK) return st;
    if ((st = sfi::check_paged(shape, kv)) != SFI_OK) return st;
    if (!q || !aligned16(q) || sink < 0 || recent < 0 || num_tokens < 1 || num_reqs < 0 || batch < 0)
        return SFI_ERR_INVALID_ARG;
    if (q_stride < (int64_t)shape->num_q_heads * shape->head_dim || q_stride % 8) return SFI_ERR_INVALID_ARG;
    // a grid's second and third dimension; TMA coordinates and strides
    if (shape->num_kv_heads > 65535 || batch > 65535) return SFI_ERR_UNSUPPORTED;
    if ((int64_t)num_reqs * num_tokens >= (int64_t(1) << 31) || q_stride >= (int64_t(1) << 38)) return SFI_ERR_UNSUPPORTED;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.q_stride = q_stride;
    p.k_pool = static_cast<const __nv_bfloat16 *>(kv->k_pool);
    p.v_pool = static_cast<const __nv_bfloat16 *>(kv->v_pool);
    p.page_table = kv->page_table;
    p.seq_lens = kv->seq_lens;
    p.new_lens = new_lens;
    p.req_ids = req_ids;
    p.max_pages = kv->max_pages_per_req;
    p.num_pages = kv->num_pages;
    p.reqs = num_reqs;
    p.hq = shape->num_q_heads;
    p.hkv = shape->num_kv_heads;
    p.group = p.hq / p.hkv;
    p.tokens = num_tokens;
    p.sink = sink;
    p.recent = recent;
    p.scale_log2 = sfi::resolve_scale(shape) * 1.4426950408889634f;
    p.dev_status = dev_status;
    return SFI_OK;
}

// The maps of K and V, and of the queries in boxes of `rows` rows (0: none).
bool window_maps(const sfi_attn_shape *shape, const sfi_paged_kv *kv, const sfi::WindowParams &p, int rows,
                 sfi::WindowMaps &maps) {
    const int64_t pool_rows = (int64_t)kv->num_pages * p.hkv * sfi::kSubTokens;
    return sfi::encode_rows(&maps.k, kv->k_pool, pool_rows, shape->head_dim) &&
           sfi::encode_rows(&maps.v, kv->v_pool, pool_rows, shape->head_dim) &&
           (rows == 0 || sfi::encode_queries(&maps.q, p.q, (int64_t)p.reqs * p.tokens, p.q_stride, p.hq,
                                             shape->head_dim, p.group, rows / p.group));
}

}  // namespace

extern "C" {

sfi_status sfi_window_attn(const sfi_attn_shape *shape, const sfi_paged_kv *kv, int32_t sink, int32_t recent,
                           const void *q, int64_t q_stride, int32_t num_reqs, int32_t num_tokens,
                           const int32_t *new_lens, void *out, float *lse, const int32_t *req_ids, int32_t batch,
                           int32_t *dev_status, void *stream) {
    sfi::WindowParams p{};
    const sfi_status st = window_params(shape, kv, sink, recent, q, q_stride, num_reqs, num_tokens, new_lens, req_ids,
                                        batch, dev_status, p);
    if (st != SFI_OK) return st;
    if (!out || !aligned16(out)) return SFI_ERR_INVALID_ARG;
    if (batch == 0 || num_reqs == 0) return SFI_OK;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.lse = lse;
    const bool step = (int64_t)num_tokens * p.group <= sfi::kMaxRows;
    // (a CTA for each 256 query rows of a KV head)
    if ((int64_t)batch * p.hkv * (((int64_t)num_tokens * p.group + 255) / 256) >= (int64_t(1) << 31)) return SFI_ERR_UNSUPPORTED;
    sfi::WindowMaps maps{};
    if (!window_maps(shape, kv, p, step ? 0 : sfi::kPromptBoxRows, maps)) return SFI_ERR_CUDA;
    const auto launch = step ? sfi::launch_window_step : sfi::launch_window_prompt;
    return launched(launch(maps, p, shape->head_dim, batch, static_cast<cudaStream_t>(stream)));
}

sfi_status sfi_attn_mass(const sfi_attn_shape *shape, const sfi_paged_kv *kv, int32_t sink, int32_t recent,
                         const void *q, int64_t q_stride, int32_t num_reqs, int32_t num_tokens,
                         const int32_t *new_lens, const float *lse, float *mass, int64_t mass_stride, float decay,
                         const int32_t *req_ids, int32_t batch, int32_t *dev_status, void *stream) {
    sfi::WindowParams p{};
    const sfi_status st = window_params(shape, kv, sink, recent, q, q_stride, num_reqs, num_tokens, new_lens, req_ids,
                                        batch, dev_status, p);
    if (st != SFI_OK) return st;
    if (!lse || !mass || mass_stride < 1 || !std::isfinite(decay)) return SFI_ERR_INVALID_ARG;
    if (batch == 0 || num_reqs == 0) return SFI_OK;
    // (a CTA for each 128 positions of a KV head at most)
    const int64_t most = std::min<int64_t>((int64_t)kv->max_pages_per_req * sfi::kSubTokens, mass_stride);
    if ((int64_t)batch * p.hkv * ((most + 127) / 128) >= (int64_t(1) << 31)) return SFI_ERR_UNSUPPORTED;
    sfi::WindowMaps maps{};
    if (!window_maps(shape, kv, p, sfi::mass_rows((int64_t)num_tokens * p.group), maps)) return SFI_ERR_CUDA;
    const sfi::MassParams w{lse, mass, mass_stride, decay};
    return launched(sfi::launch_attn_mass(maps, p, w, shape->head_dim, batch, static_cast<cudaStream_t>(stream)));
}

sfi_status sfi_kv_evict(const sfi_attn_shape *shape, const sfi_paged_kv *kv, const float *mass, int64_t mass_stride,
                        int32_t sink, int32_t recent, const int32_t *k_per_req, int32_t k_cap, int32_t *idx_out,
                        int32_t *count_out, float *mass_out, int32_t *new_lens, const int32_t *req_ids, int32_t batch,
                        int32_t *dev_status, void *stream) {
    sfi_status st = sfi::check_shape(shape);
    if (st != SFI_OK) return st;
    if ((st = sfi::check_paged(shape, kv)) != SFI_OK) return st;
    if (!mass || !k_per_req || (!idx_out && k_cap > 0) || !count_out || !new_lens || mass == mass_out || new_lens == kv->seq_lens)
        return SFI_ERR_INVALID_ARG;
    if (mass_stride < 1 || sink < 0 || recent < 0 || k_cap < 0 || batch < 0) return SFI_ERR_INVALID_ARG;
    if (shape->num_kv_heads > 65535 || batch > 65535) return SFI_ERR_UNSUPPORTED;
    if (batch == 0) return SFI_OK;
    // (no request is that long; their sum with a length stays within 32 bits)
    sink = std::min(sink, 1 << 30);
    recent = std::min(recent, 1 << 30);
    sfi::TopkParams t{};
    t.scores = mass;
    t.score_stride = mass_stride;
    t.max_len = std::min<int64_t>(mass_stride, (int64_t)kv->max_pages_per_req * sfi::kSubTokens);
    t.hkv = shape->num_kv_heads;
    t.seq_lens = kv->seq_lens;
    t.sink = sink;
    t.recent = recent;
    t.k_per_req = k_per_req;
    t.k_cap = k_cap;
    t.idx_out = idx_out;
    t.count_out = count_out;
    t.req_ids = req_ids;
    t.dev_status = dev_status;
    sfi::EvictParams p{};
    p.k_pool = static_cast<__nv_bfloat16 *>(kv->k_pool);
    p.v_pool = static_cast<__nv_bfloat16 *>(kv->v_pool);
    p.page_table = kv->page_table;
    p.seq_lens = kv->seq_lens;
    p.req_ids = req_ids;
    p.max_pages = kv->max_pages_per_req;
    p.num_pages = kv->num_pages;
    p.hkv = shape->num_kv_heads;
    p.head_dim = shape->head_dim;
    p.mass = mass;
    p.mass_out = mass_out;
    p.mass_stride = mass_stride;
    p.sink = sink;
    p.recent = recent;
    p.k_per_req = k_per_req;
    p.idx = idx_out;
    p.k_cap = k_cap;
    p.new_lens = new_lens;
    p.dev_status = dev_status;
    return launched(sfi::launch_kv_evict(p, t, batch, static_cast<cudaStream_t>(stream)));
}

sfi_status sfi_verify_tokens(const float *target, int64_t target_stride, const float *draft, int64_t draft_stride,
                             const int32_t *tokens, const float *u, int32_t vocab, int32_t num_drafts,
                             const int32_t *draft_lens, const int32_t *seq_lens, int32_t *out_tokens,
                             int32_t *accepted, int32_t *new_lens, const int32_t *req_ids, int32_t batch,
                             int32_t *dev_status, void *stream) {
    if (!target || !tokens || !u || !out_tokens || !accepted || (seq_lens == nullptr) != (new_lens == nullptr))
        return SFI_ERR_INVALID_ARG;
    if (vocab < 1 || num_drafts < 1 || batch < 0 || target_stride < vocab || (draft && draft_stride < vocab))
        return SFI_ERR_INVALID_ARG;
    if (vocab > SFI_MAX_VOCAB || batch > (1 << 24)) return SFI_ERR_UNSUPPORTED;
    if (batch == 0) return SFI_OK;
    sfi::VerifyParams p{};
    p.target = target;
    p.target_stride = target_stride;
    p.draft = draft;
    p.draft_stride = draft_stride;
    p.tokens = tokens;
    p.u = u;
    p.vocab = vocab;
    p.drafts = num_drafts;
    p.draft_lens = draft_lens;
    p.seq_lens = seq_lens;
    p.req_ids = req_ids;
    p.out_tokens = out_tokens;
    p.accepted = accepted;
    p.new_lens = new_lens;
    p.dev_status = dev_status;
    return launched(sfi::launch_verify_tokens(p, batch, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
