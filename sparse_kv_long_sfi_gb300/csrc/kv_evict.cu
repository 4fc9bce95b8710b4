// Eviction's second half: the kept rows of K and V move to the front of a request's pages.
//
// The Selector (select_topk.cu) has chosen, per (request, KV head), the candidates of [S, L - W) with
// the largest weights, in ascending positions. Row i of what remains comes from position
//   src(i) = i for i < min(S, L),  idx[i - S] for the chosen ones,  L - W + (i - S - count) behind them,
// and src(i) >= i ascends. So rows are moved in place, chunk after chunk: a chunk's rows may be read
// any number of chunks ahead (its sources lie at or behind its own destinations, behind all earlier
// ones), and may be written once all chunks up to it have been read.
//
// Bound by HBM: every moved row is read and written once. The order along a row of work allows no
// second CTA in it, but K, V and parts of the head dimension are independent, so a unit is cut into
// 64- to 256-byte columns until there are enough CTAs; a ring of kEvictStages chunks by cp.async
// keeps their reads in flight, and positions and page ids are fetched one and two chunks further ahead.
// Weights go to a second buffer (they are also the Selector's input), in the same launch.
// 16 requests of 8 x 2112 rows cut to 2048 (128-dim heads): 54.9 us with the Selector (264 MB, 38.9 us).
//
// It writes bf16 pages, so it does not release its dependents early (see page_ops.cu).
#include <algorithm>

#include "sfi_device.cuh"
#include "sfi_internal.h"

namespace sfi {

namespace {

constexpr int kEvictThreads = 256;
constexpr int kEvictStages = 4;
constexpr int kEvictLoads = 2;  // 16-byte pieces of a thread in a chunk

}  // namespace

__global__ void __launch_bounds__(kEvictThreads) kv_evict_kernel(const EvictParams p, int parts) {
    __shared__ __align__(16) int4 s_ring[kEvictStages][kEvictLoads][kEvictThreads];
    const int tid = threadIdx.x;
    grid_dependency_wait();
    const int r = p.req_ids ? p.req_ids[blockIdx.z] : (int)blockIdx.z;
    const int kvh = blockIdx.y;
    const bool weights = (int)blockIdx.x == 2 * parts;
    const bool lead = tid == 0 && blockIdx.x == 0 && kvh == 0;
    const int L = p.seq_lens[r];
    const int k = p.k_per_req[r];
    // (the Selector has refused what is refused here for its own reasons; lengths are checked against the table here)
    const int64_t cand = (int64_t)L - p.recent - p.sink;
    if (L < 0 || L > p.max_pages * kSubTokens || L > p.mass_stride) {
        if (lead) report(p.dev_status, SFI_DEV_BAD_LEN);
        return;
    }
    if (k < 0 || k > p.k_cap || cand > kTopkMaxCandidates) {
        if (lead) report(p.dev_status, SFI_DEV_K_OVERFLOW);
        return;
    }
    const int count = (int)max((int64_t)0, min((int64_t)k, cand));
    const bool all = count >= cand;  // nothing is evicted
    const int kept = all ? L : L - (int)(cand - count);
    if (lead) p.new_lens[r] = kept;
    const int32_t *idx = p.idx + ((int64_t)r * p.hkv + kvh) * p.k_cap;
    auto source = [&](int i) -> int {
        if (all || i < p.sink) return i;
        const int c = i - p.sink;
        return c < count ? idx[c] : i + (L - kept);
    };
    if (weights) {
        if (!p.mass_out) return;
        const int64_t row = ((int64_t)r * p.hkv + kvh) * p.mass_stride;
        for (int i = tid; i < kept; i += kEvictThreads) {
            const int s = source(i);
            if ((uint32_t)s < (uint32_t)L) p.mass_out[row + i] = p.mass[row + s];
        }
        return;
    }
    if (all) return;
    const bool is_v = (int)blockIdx.x >= parts;
    const int part = (int)blockIdx.x - (is_v ? parts : 0);
    const int per_row = p.head_dim * 2 / parts / 16;  // 16-byte pieces of a row's part: a power of two
    const int rows = kEvictThreads / per_row;         // rows of one load; a chunk has kEvictLoads times as many
    const int mine = tid / per_row;
    char *pool = reinterpret_cast<char *>(is_v ? p.v_pool : p.k_pool) + part * (p.head_dim * 2 / parts) + (tid % per_row) * 16;
    const int32_t *ptab = p.page_table + (int64_t)r * p.max_pages;
    const int first = min(p.sink, L);  // sink rows stay where they are
    const int chunk_rows = rows * kEvictLoads;
    const int chunks = (kept - first + chunk_rows - 1) / chunk_rows;
    uint32_t err = 0;
    // the row behind (page, position), or null
    auto at = [&](int page, int pos) -> char * {
        if (page < 0 || page >= p.num_pages) {
            err |= SFI_DEV_BAD_PAGE;
            return nullptr;
        }
        return pool + (((int64_t)page * p.hkv + kvh) * kSubTokens + pos % kSubTokens) * p.head_dim * 2;
    };
    int src_pos[kEvictLoads], src_page[kEvictLoads], next_pos[kEvictLoads];
    auto fetch_pos = [&](int c, int (&pos)[kEvictLoads]) {
#pragma unroll
        for (int j = 0; j < kEvictLoads; ++j) {
            const int i = first + c * chunk_rows + j * rows + mine;
            const int s = c < chunks && i < kept ? source(i) : -1;
            // (a selection that is not the Selector's could lead anywhere)
            if (s >= L || (s >= 0 && s < i)) err |= SFI_DEV_BAD_INDEX;
            pos[j] = s >= L || s <= i ? -1 : s;  // rows that stay are not moved
        }
    };
    auto fetch_page = [&](const int (&pos)[kEvictLoads], int (&page)[kEvictLoads]) {
#pragma unroll
        for (int j = 0; j < kEvictLoads; ++j) page[j] = pos[j] >= 0 ? ptab[pos[j] / kSubTokens] : -1;
    };
    // Which rows of the chunks in the ring are moved: bit stage * kEvictLoads + j.
    uint32_t moved = 0;
    auto issue = [&](int c, const int (&pos)[kEvictLoads], const int (&page)[kEvictLoads]) {
        const int st = c % kEvictStages;
#pragma unroll
        for (int j = 0; j < kEvictLoads; ++j) {
            const uint32_t bit = 1u << (st * kEvictLoads + j);
            moved &= ~bit;
            if (pos[j] >= 0) {
                const char *from = at(page[j], pos[j]);
                if (from) {
                    moved |= bit;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(&s_ring[st][j][tid])),
                                 "l"(from)
                                 : "memory");
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch_pos(0, src_pos);
    fetch_pos(1, next_pos);
    fetch_page(src_pos, src_page);
    int dst_page[kEvictLoads];
    auto fetch_dst = [&](int c) {
#pragma unroll
        for (int j = 0; j < kEvictLoads; ++j) {
            const int i = first + c * chunk_rows + j * rows + mine;
            dst_page[j] = c < chunks && i < kept ? ptab[i / kSubTokens] : -1;
        }
    };
    fetch_dst(0);
    for (int c = 0; c < chunks + kEvictStages - 1; ++c) {
        // chunk c is requested, chunk c - (stages - 1) is written
        int pos[kEvictLoads], page[kEvictLoads];
#pragma unroll
        for (int j = 0; j < kEvictLoads; ++j) pos[j] = src_pos[j], page[j] = src_page[j], src_pos[j] = next_pos[j];
        fetch_page(src_pos, src_page);
        fetch_pos(c + 2, next_pos);
        issue(c, pos, page);
        const int done = c - (kEvictStages - 1);
        if (done < 0) continue;
        asm volatile("cp.async.wait_group %0;" ::"n"(kEvictStages - 1) : "memory");
        __syncthreads();  // every thread's reads up to this chunk have arrived
        const int st = done % kEvictStages;
        int to_page[kEvictLoads];
#pragma unroll
        for (int j = 0; j < kEvictLoads; ++j) to_page[j] = dst_page[j];
        fetch_dst(done + 1);
#pragma unroll
        for (int j = 0; j < kEvictLoads; ++j) {
            if (!((moved >> (st * kEvictLoads + j)) & 1u)) continue;
            const int i = first + done * chunk_rows + j * rows + mine;
            char *to = at(to_page[j], i);
            if (to) st_v4(to, s_ring[st][j][tid]);
        }
    }
    if (err) report(p.dev_status, err);
}

cudaError_t launch_kv_evict(const EvictParams &p, int batch, cudaStream_t stream) {
    const int sms = sm_count_current_device();
    if (sms <= 0) return cudaErrorInvalidDevice;
    // Four CTAs per SM, as far as columns of 64 bytes allow.
    const int64_t units = (int64_t)batch * p.hkv * 2;
    int parts = 1;
    while (parts < p.head_dim / 32 && units * parts < (int64_t)sms * 4) parts *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * parts + 1), (unsigned)p.hkv, (unsigned)batch);
    cfg.blockDim = dim3(kEvictThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_evict_kernel, p, parts);
}

}  // namespace sfi
