// C ABI of the cache-side operators (declared in include/sfi.h): argument validation and
// kernel dispatch. Allocates nothing.
#include <cmath>

#include "sfi_internal.h"

namespace {

using sfi::aligned16;
using sfi::aligned8;

sfi_status launched(cudaError_t e) { return e == cudaSuccess ? SFI_OK : SFI_ERR_CUDA; }

}  // namespace

extern "C" {

sfi_status sfi_qk_norm_rope(const sfi_attn_shape *shape, const sfi_rope *rope, const void *q, int64_t q_stride,
                            const void *k, int64_t k_stride, const void *v, int64_t v_stride, const void *q_weight,
                            const void *k_weight, float eps, const int32_t *positions, int64_t axis_stride,
                            int32_t num_tokens, const int32_t *new_lens, void *q_out, void *k_out,
                            const sfi_paged_kv *kv, const int32_t *req_ids, int32_t batch, int32_t *dev_status,
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
        if (!positions && !kv) return SFI_ERR_INVALID_ARG;
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

}  // extern "C"
