// Eviction: per (request, KV head) the candidates of [S, L - W) with the largest weights are chosen, and
// the kept rows of K and V move to the front of the request's pages.
//
// The choice is that of the Selector (select_topk.cu), which serves rows of more than 16384 candidates
// here too. Its passes are laid out for long rows; the caches that are evicted from are short, so up to
// that length one CTA keeps all keys in registers and counts them in one small histogram per pass of
// 8 bits (16 x 8 units of 1792 candidates: 18 us there, 10 here, each alone).
//
// Row i of what remains comes from position
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
// 16 requests of 8 x 2112 rows cut to 2048 (128-dim heads): 31 us, the move alone 28 (264 MB, 38.9 us of HBM
// time, but most of it stays in L2); 8 of 7001 to 16384 cut to about 1100: 30 us, the choice alone 14.5 and the move
// 19.5 (76 MB, 11.3 us). Which kernel chooses follows the width of the weights, not the rows' lengths: the first of
// these takes 40 us in weights of 131072.
//
// It writes bf16 pages, so it does not release its dependents early (see page_ops.cu).
#include <algorithm>
#include <atomic>

#include "sfi_device.cuh"
#include "sfi_internal.h"

namespace sfi {

namespace {

constexpr int kEvictThreads = 256;
constexpr int kEvictStages = 3, kEvictTables = 5;
constexpr int kEvictLoads = 4;  // 16-byte pieces of a thread in a chunk

constexpr int kSelectEach = 16;        // keys of a thread
constexpr uint32_t kNoCandidate = 0u;  // below every key

// Ascending keys: -0 as +0, NaN below all.
__device__ __forceinline__ uint32_t weight_key(float x) {
    uint32_t u = __float_as_uint(x);
    if ((u & 0x7fffffffu) > 0x7f800000u) return 1u;
    if (u == 0x80000000u) u = 0u;
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

}  // namespace

// One CTA per unit, 16 candidates of a thread. What is refused here is reported by kv_evict_kernel.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) evict_select_kernel(const EvictParams p, int32_t *idx_out, int32_t *count_out) {
    constexpr int kWarps = THREADS / 32;
    // Long rows have four counters for each bin, so that fewer of a warp's atomics meet in one (8 requests of up to 16384
    // rows, the whole call: 30.2 us; with 8, 16 and 32 counters, which have to be added up, 30.8, 31.6 and 31.9).
    constexpr int kCopies = THREADS == 1024 ? 4 : 1;
    __shared__ uint32_t s_hist[256 * kCopies];
    __shared__ uint32_t s_bin[256];
    __shared__ uint32_t s_prefix, s_rem, s_in;
    __shared__ int2 s_count[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    const int kvh = blockIdx.x;
    const int r = p.req_ids ? p.req_ids[blockIdx.y] : (int)blockIdx.y;
    const int L = p.seq_lens[r], k = p.k_per_req[r];
    if (L < 0 || L > p.max_pages * kSubTokens || L > p.mass_stride || k < 0 || k > p.k_cap) return;
    const int n = (int)max((int64_t)0, (int64_t)L - p.recent - p.sink);  // at most THREADS * 16: the row's stride says so
    const int keep = min(k, n);
    if (kvh == 0 && tid == 0) count_out[r] = keep;
    int32_t *out = idx_out + ((int64_t)r * p.hkv + kvh) * p.k_cap;
    if (keep == n) {
        for (int i = tid; i < n; i += THREADS) out[i] = p.sink + i;
        return;
    }
    if (keep == 0) return;
    // a warp's candidates lie in a row: 32 j + lane behind its first
    const int first = warp * 32 * kSelectEach;
    const float *row = p.mass + ((int64_t)r * p.hkv + kvh) * p.mass_stride + p.sink;
    uint32_t key[kSelectEach];
#pragma unroll
    for (int j = 0; j < kSelectEach; ++j) {
        const int i = first + 32 * j + lane;
        key[j] = i < n ? __float_as_uint(row[i]) : 0u;
    }
#pragma unroll
    for (int j = 0; j < kSelectEach; ++j)
        key[j] = first + 32 * j + lane < n ? weight_key(__uint_as_float(key[j])) : kNoCandidate;
    // The bits of the smallest kept key, from the top: the keys that share them are those in [low, high], `rem` of
    // them are kept.
    uint32_t low = 1u, high = 0xffffffffu, rem = (uint32_t)keep;
    uint32_t prefix = 0;
    bool whole = false;  // all of them are
    for (int i = tid; i < 256 * kCopies; i += THREADS) s_hist[i] = 0;
    __syncthreads();
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
#pragma unroll
        for (int j = 0; j < kSelectEach; ++j) {
            if (key[j] >= low && key[j] <= high) atomicAdd(&s_hist[((key[j] >> shift) & 255u) * kCopies + (lane & (kCopies - 1))], 1u);
        }
        __syncthreads();
        {
            // a bin's counters, cleared for the next pass (in an order without bank conflicts)
            constexpr int kParts = THREADS / 256, kSpan = kCopies / kParts;
            const int bin = tid / kParts, part = tid % kParts;
            uint32_t sum = 0;
#pragma unroll 8
            for (int i = 0; i < kSpan; ++i) {
                uint32_t *at = &s_hist[bin * kCopies + part * kSpan + ((i + bin) & (kSpan - 1))];
                sum += *at;
                *at = 0;
            }
#pragma unroll
            for (int off = 1; off < kParts; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            if (part == 0) s_bin[bin] = sum;
        }
        __syncthreads();
        if (warp == 0) {
            // lane i: bins 255 - 8 i down to 248 - 8 i
            uint32_t h[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += h[i] = s_bin[255 - 8 * lane - i];
            uint32_t above = sum;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, above, off);
                if (lane >= off) above += o;
            }
            above -= sum;  // keys in higher bins than this lane's
            if (above < rem && rem <= above + sum) {
                uint32_t at = above;
                int i = 0;
                for (; at + h[i] < rem; ++i) at += h[i];
                s_prefix = (uint32_t)(255 - 8 * lane - i) << shift;
                s_rem = rem - at;
                s_in = h[i];
            }
        }
        __syncthreads();
        // (bits above this digit are the same in low and high)
        prefix |= s_prefix;
        rem = s_rem;
        low = max(prefix, 1u);
        high = prefix | ((1u << shift) - 1u);
        whole = s_in == rem;
        if (whole) break;
    }
    // ranks in the order of positions: kept ones are above `high`, or in [low, high] and among its first `rem`
    const uint32_t lower = (1u << lane) - 1u;
    if (whole) {
        int mine = 0;
#pragma unroll
        for (int j = 0; j < kSelectEach; ++j) mine += key[j] >= low;
        mine = __reduce_add_sync(0xffffffffu, mine);
        if (lane == 0) s_count[warp].x = mine;
        __syncthreads();
        int at = __reduce_add_sync(0xffffffffu, lane < warp ? s_count[lane].x : 0);
#pragma unroll
        for (int j = 0; j < kSelectEach; ++j) {
            const bool take = key[j] >= low;
            const uint32_t taken = __ballot_sync(0xffffffffu, take);
            if (take) out[at + __popc(taken & lower)] = p.sink + first + 32 * j + lane;
            at += __popc(taken);
        }
        return;
    }
    int above = 0, equal = 0;
#pragma unroll
    for (int j = 0; j < kSelectEach; ++j) {
        above += key[j] > high;
        equal += key[j] >= low && key[j] <= high;
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) s_count[warp] = make_int2(above, equal);
    __syncthreads();
    const int2 before = lane < warp ? s_count[lane] : make_int2(0, 0);
    int seen = __reduce_add_sync(0xffffffffu, before.y);
    int at = __reduce_add_sync(0xffffffffu, before.x) + min(seen, (int)rem);
#pragma unroll
    for (int j = 0; j < kSelectEach; ++j) {
        const bool same = key[j] >= low && key[j] <= high;
        const uint32_t same_all = __ballot_sync(0xffffffffu, same);
        const bool take = key[j] > high || (same && seen + __popc(same_all & lower) < (int)rem);
        const uint32_t taken = __ballot_sync(0xffffffffu, take);
        if (take) out[at + __popc(taken & lower)] = p.sink + first + 32 * j + lane;
        at += __popc(taken);
        seen += __popc(same_all);
    }
}

__global__ void __launch_bounds__(kEvictThreads) kv_evict_kernel(const EvictParams p, int parts) {
    extern __shared__ __align__(16) int4 s_dyn[];
    int4(*ring)[kEvictLoads][kEvictThreads] = reinterpret_cast<int4(*)[kEvictLoads][kEvictThreads]>(s_dyn);
    // A chunk's rows: where each comes from (or -1: it is not moved) and goes to, as rows of the pool. A thread
    // works out one row, not each of the 16 pieces that the threads move (61% of issue slots then: 37 us for
    // 16 x 8 x 2048 rows that lie in L2, 26 now).
    int2(*table)[kEvictThreads] = reinterpret_cast<int2(*)[kEvictThreads]>(s_dyn + kEvictStages * kEvictLoads * kEvictThreads);
    const int tid = threadIdx.x;
    grid_dependency_wait();
    const int r = p.req_ids ? p.req_ids[blockIdx.z] : (int)blockIdx.z;
    const int kvh = blockIdx.y;
    const bool weights = (int)blockIdx.x == 2 * parts;
    const bool lead = tid == 0 && blockIdx.x == 0 && kvh == 0;
    const int L = p.seq_lens[r];
    const int k = p.k_per_req[r];
    // (the choice has refused the same requests: nothing of theirs is written)
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
#pragma unroll 4
        for (int i = tid; i < kept; i += kEvictThreads) {
            const int s = source(i);
            if ((uint32_t)s < (uint32_t)L) p.mass_out[row + i] = p.mass[row + s];
        }
        return;
    }
    if (all) return;
    const bool is_v = (int)blockIdx.x >= parts;
    const int part = (int)blockIdx.x - (is_v ? parts : 0);
    const int per_row = p.head_dim * 2 / parts / 16;  // 16-byte pieces of a row's part: a power of two, 4 to 16
    const int shift = __ffs(per_row) - 1;
    const int rows = kEvictThreads >> shift;          // rows of one load; a chunk has kEvictLoads times as many
    const int mine = tid >> shift;
    const int row_bytes = p.head_dim * 2;
    char *pool = reinterpret_cast<char *>(is_v ? p.v_pool : p.k_pool) + part * (row_bytes / parts) + (tid & (per_row - 1)) * 16;
    const int32_t *ptab = p.page_table + (int64_t)r * p.max_pages;
    const int first = min(p.sink, L);  // sink rows stay where they are
    const int chunk_rows = rows * kEvictLoads;  // (at most a row for each thread)
    const int chunks = (kept - first + chunk_rows - 1) / chunk_rows;
    uint32_t err = 0;
    // this thread's row of a chunk: its place, where it comes from (-1: it stays, or there is none), and their pages
    int src = -1, src_page = 0, dst_page = 0, next = -1;
    auto fetch_pos = [&](int c) -> int {
        const int i = first + c * chunk_rows + tid;
        if (c >= chunks || tid >= chunk_rows || i >= kept) return -1;
        return source(i);
    };
    auto fetch_pages = [&](int c) {  // of chunk c, whose source is in `src`
        const int i = first + c * chunk_rows + tid;
        // (a selection that is not the Selector's could lead anywhere)
        if (src >= L || (src >= 0 && src < i)) err |= SFI_DEV_BAD_INDEX;
        if (src >= L || src <= i) src = -1;  // (rows that stay are not moved)
        if (src >= 0) {
            src_page = ptab[src / kSubTokens];
            dst_page = ptab[i / kSubTokens];
        }
    };
    auto write_table = [&](int c) {
        int2 e = make_int2(-1, -1);
        if (src >= 0) {
            const int i = first + c * chunk_rows + tid;
            if ((uint32_t)src_page >= (uint32_t)p.num_pages || (uint32_t)dst_page >= (uint32_t)p.num_pages)
                err |= SFI_DEV_BAD_PAGE;
            else
                e = make_int2((src_page * p.hkv + kvh) * kSubTokens + src % kSubTokens,
                              (dst_page * p.hkv + kvh) * kSubTokens + i % kSubTokens);
        }
        table[c % kEvictTables][tid] = e;
    };
    // chunk 0's rows, the pages of chunk 1 and the positions of chunk 2 before the loop
    src = fetch_pos(0);
    next = fetch_pos(1);
    fetch_pages(0);
    write_table(0);
    src = next;
    next = fetch_pos(2);
    fetch_pages(1);
    __syncthreads();
    for (int c = 0; c < chunks + kEvictStages - 1; ++c) {
        // chunk c is requested, chunk c - (stages - 1) is written; the rows of chunk c + 1 are put down, the pages of
        // c + 2 and the positions of c + 3 are on their way
        write_table(c + 1);
        src = next;
        next = fetch_pos(c + 3);
        fetch_pages(c + 2);
        if (c < chunks) {
#pragma unroll
            for (int j = 0; j < kEvictLoads; ++j) {
                const int from = table[c % kEvictTables][j * rows + mine].x;
                if (from >= 0)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(&ring[c % kEvictStages][j][tid])),
                                 "l"(pool + (int64_t)from * row_bytes)
                                 : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        const int done = c - (kEvictStages - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kEvictStages - 1) : "memory");
        __syncthreads();  // every thread's reads up to chunk `done` have arrived; the rows of chunk c + 1 are there
        if (done < 0) continue;
#pragma unroll
        for (int j = 0; j < kEvictLoads; ++j) {
            const int to = table[done % kEvictTables][j * rows + mine].y;
            if (to >= 0) st_v4(pool + (int64_t)to * row_bytes, ring[done % kEvictStages][j][tid]);
        }
    }
    if (err) report(p.dev_status, err);
}

namespace {

template <int THREADS>
cudaError_t launch_select(const EvictParams &p, const TopkParams &select, int batch, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.hkv, (unsigned)batch);
    cfg.blockDim = dim3(THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_select_kernel<THREADS>, p, select.idx_out, select.count_out);
}

}  // namespace

cudaError_t launch_kv_evict(const EvictParams &p, const TopkParams &select, int batch, cudaStream_t stream) {
    const int sms = sm_count_current_device();
    if (sms <= 0) return cudaErrorInvalidDevice;
    // No row has more candidates than the weights' stride leaves.
    const int64_t most = p.mass_stride - p.sink - p.recent;
    constexpr int kSmem = kEvictThreads * (kEvictStages * kEvictLoads * 16 + kEvictTables * 8);
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kv_evict_kernel), kSmem, configured);
    if (e != cudaSuccess) return e;
    if (most <= 256 * kSelectEach)
        e = launch_select<256>(p, select, batch, stream);
    else if (most <= 1024 * kSelectEach)
        e = launch_select<1024>(p, select, batch, stream);
    else
        e = launch_select_topk(select, batch, stream);
    if (e != cudaSuccess) return e;
    // Four CTAs per SM, as far as columns of 64 bytes allow. (Sharing the rows that come from behind the end of what
    // remains between CTAs of a cluster, where most of a cache goes, was slower: 32 us without, 38 with 2 or 4.)
    const int64_t units = (int64_t)batch * p.hkv * 2;
    int parts = 1;
    while (parts < p.head_dim / 32 && units * parts < (int64_t)sms * 4) parts *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * parts + 1), (unsigned)p.hkv, (unsigned)batch);
    cfg.blockDim = dim3(kEvictThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_evict_kernel, p, parts);
}

}  // namespace sfi
