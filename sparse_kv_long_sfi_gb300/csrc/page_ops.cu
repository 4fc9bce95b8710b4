// Pages shared between requests: copying, forking, reserving (copy on write), freeing and
// compacting. All state (page table, lengths, a holder count per page) is on the device.
//
// Planning is integer work on small arrays and is done where its result cannot depend on
// the order of threads: counts change by atomic additions alone, free pages are found by
// one CTA that scans the counts in page order (ranks by prefix sums), and lists are
// written at those ranks. The bytes move in a second launch that reads the list's length
// on the device; it is bound by HBM (a page is read and written once per pool).
//
// The kernels wait for the stream's previous kernel as dependent launches, but none releases
// its own dependents early: they write page tables, lengths and pages, which an attention
// launch may be allowed to read ahead of its wait (SFI_ATTN_EARLY_KV_PREFETCH). (Nor would any
// kernel do so before its own wait: see launch_dependent_clusters.)
#include <algorithm>

#include "sfi_device.cuh"
#include "sfi_internal.h"

namespace sfi {

namespace {

constexpr int kPageThreads = 256;
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kCopyChunk = 16384;  // bytes of a pool's page that a CTA moves at once

// Workspace (int32): [0] moves, [1] unused .. [3], then the moves' sources, their
// destinations (num_pages each), and the free or new page ids (num_pages).
struct PageLists {
    int32_t *moves, *src, *dst, *ids;
    __host__ __device__ PageLists(void *ws, int32_t num_pages)
        : moves(static_cast<int32_t *>(ws)), src(moves + 4), dst(src + num_pages), ids(dst + num_pages) {}
};

// Exclusive sum over the CTA's threads; *total receives the whole.
__device__ __forceinline__ int block_scan(int v, int *s_warp, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
    }
    __syncthreads();  // the last round's sums have been read
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int w = lane < kPlanWarps ? s_warp[lane] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, w, off);
        if (lane >= off) w += o;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
    return (warp ? before : 0) + incl - v;
}

// Adds v >= 0 of all of the CTA's threads to *sum in 64 bits (complete after the next barrier).
__device__ __forceinline__ void block_sum(int v, unsigned long long *sum) {
    const uint32_t lo = __reduce_add_sync(0xffffffffu, (uint32_t)v & 0xffffu);
    const uint32_t hi = __reduce_add_sync(0xffffffffu, (uint32_t)v >> 16);
    if ((threadIdx.x & 31) == 0) atomicAdd(sum, ((unsigned long long)hi << 16) + lo);
}

// Pages that len >= 0 tokens take. (No sum that a length near 2^31 could carry past it: every
// length, those that only device data can say too, compares with the table's width.)
__device__ __forceinline__ int pages_of(int len) { return len / kSubTokens + (len % kSubTokens != 0); }

}  // namespace

// Row r of the table by the new page ids (entries out of range, and those behind the
// request's length, as they are).
__device__ void renumber_row(const PageMapParams &m, int r, const int32_t *new_ids, int32_t *table_out,
                             int32_t *dev_status) {
    const int L = m.seq_lens[r];
    const bool fine = L >= 0 && pages_of(L) <= m.max_pages;
    if (!fine && threadIdx.x == 0) report(dev_status, SFI_DEV_BAD_LEN);
    const int held = fine ? pages_of(L) : 0;
    for (int i = threadIdx.x; i < m.max_pages; i += kPageThreads) {
        int page = m.page_table[(int64_t)r * m.max_pages + i];
        if (i < held) {
            if (page < 0 || page >= m.num_pages)
                report(dev_status, SFI_DEV_BAD_PAGE);
            else
                page = new_ids[page];
        }
        table_out[(int64_t)r * m.max_pages + i] = page;
    }
}

// ---- copy: page src[i] -> dst[i] of every pool, in chunks ------------------------------
// (TABLE: with table_out, a compaction's new table is written in the same launch)
//
// That part takes registers: 48 against 32, five CTAs per SM against eight. Pages of up to half a
// chunk leave threads idle and want the eight (2000 pages of 8 x 4608 bytes: 25.3 us, 33.3 with
// five; 4000 of 8 x 8192: 86.7 and 92.2). Larger ones stream better from the five (4000 of
// 8 x 12288 bytes: 124 us, 128 with eight; 3500 of 8 x 32768: 281 and 293), so they take the same
// kernel as a compaction, without a table.
template <bool TABLE>
__global__ void __launch_bounds__(kPageThreads) page_copy_kernel(void *const *pools, int num_pools, int64_t page_bytes,
                                                                 int num_pages, const int32_t *src, const int32_t *dst,
                                                                 int n_host, const int32_t *n_dev, const PageMapParams m,
                                                                 const int32_t *new_ids, int32_t *table_out,
                                                                 int32_t *dev_status) {
    constexpr int kLoads = kCopyChunk / 16 / kPageThreads;
    grid_dependency_wait();
    if (TABLE && table_out)
        for (int r = blockIdx.x; r < m.num_reqs; r += gridDim.x) renumber_row(m, r, new_ids, table_out, dev_status);
    const int n = n_dev ? *n_dev : n_host;
    const int chunks = (int)((page_bytes + kCopyChunk - 1) / kCopyChunk);
    const int64_t items = (int64_t)n * num_pools * chunks;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int chunk = (int)(item % chunks);
        const int64_t at = item / chunks;
        const int pool = (int)(at % num_pools), i = (int)(at / num_pools);
        const int a = src[i], z = dst[i];
        if (a < 0 || a >= num_pages || z < 0 || z >= num_pages) {
            if (threadIdx.x == 0) report(dev_status, SFI_DEV_BAD_PAGE);
            continue;
        }
        uint8_t *base = static_cast<uint8_t *>(pools[pool]);
        const int64_t off = (int64_t)chunk * kCopyChunk + threadIdx.x * 16;
        const uint8_t *from = base + a * page_bytes;
        uint8_t *to = base + z * page_bytes;
        int4 v[kLoads];
#pragma unroll
        for (int k = 0; k < kLoads; ++k)
            if (off + k * kPageThreads * 16 < page_bytes) v[k] = ld_stream_v4(from + off + k * kPageThreads * 16);
#pragma unroll
        for (int k = 0; k < kLoads; ++k)
            if (off + k * kPageThreads * 16 < page_bytes) st_v4(to + off + k * kPageThreads * 16, v[k]);
    }
}

// ---- fork and free: one CTA per request -------------------------------------------------
__global__ void __launch_bounds__(kPageThreads) page_fork_kernel(const PageMapParams m, const int32_t *src,
                                                                 const int32_t *dst, const int32_t *fork_lens,
                                                                 int32_t *dev_status) {
    grid_dependency_wait();
    const int a = src[blockIdx.x], z = dst[blockIdx.x];
    uint32_t err = 0;
    int len = 0;
    if (a < 0 || a >= m.num_reqs || z < 0 || z >= m.num_reqs || a == z) {
        err = SFI_DEV_BAD_INDEX;
    } else {
        const int L = m.seq_lens[a];
        len = fork_lens ? fork_lens[blockIdx.x] : L;
        if (L < 0 || pages_of(L) > m.max_pages || len < 0 || len > L) err = SFI_DEV_BAD_LEN;
    }
    const int held = err ? 0 : pages_of(len);
    const int32_t *from = m.page_table + (int64_t)a * m.max_pages;
    bool out = false;
    for (int i = threadIdx.x; i < held; i += kPageThreads) out |= (uint32_t)from[i] >= (uint32_t)m.num_pages;
    if (__syncthreads_or(out)) err = SFI_DEV_BAD_PAGE;
    if (err) {
        if (threadIdx.x == 0) report(dev_status, err);
        return;
    }
    int32_t *to = m.page_table + (int64_t)z * m.max_pages;
    for (int i = threadIdx.x; i < held; i += kPageThreads) {
        const int page = from[i];
        to[i] = page;
        atomicAdd(m.ref_count + page, 1);
    }
    if (threadIdx.x == 0) m.seq_lens[z] = len;
}

__global__ void __launch_bounds__(kPageThreads) page_free_kernel(const PageMapParams m, const int32_t *reqs,
                                                                 int32_t *dev_status) {
    grid_dependency_wait();
    const int r = reqs[blockIdx.x];
    if (r < 0 || r >= m.num_reqs) {
        if (threadIdx.x == 0) report(dev_status, SFI_DEV_BAD_INDEX);
        return;
    }
    // the length is taken, so that a request named twice lets go of its pages once
    __shared__ int s_len;
    if (threadIdx.x == 0) {
        s_len = atomicExch(m.seq_lens + r, 0);
        if (s_len < 0 || pages_of(s_len) > m.max_pages) {
            m.seq_lens[r] = s_len;
            report(dev_status, SFI_DEV_BAD_LEN);
            s_len = 0;
        }
    }
    __syncthreads();
    const int L = s_len;
    const int32_t *row = m.page_table + (int64_t)r * m.max_pages;
    const int held = pages_of(L);
    for (int i = threadIdx.x; i < held; i += kPageThreads) {
        const int page = row[i];
        if (page < 0 || page >= m.num_pages) {
            report(dev_status, SFI_DEV_BAD_PAGE);
        } else if (atomicSub(m.ref_count + page, 1) <= 0) {
            atomicAdd(m.ref_count + page, 1);  // nobody held it: as it was
            report(dev_status, SFI_DEV_BAD_PAGE);
        }
    }
}

// ---- reserve: one CTA plans for all requests --------------------------------------------
// Three passes: what each request needs (and whether its last page is its own), the lowest
// free pages, and their distribution; then the copies of shared last pages are launched.
__global__ void __launch_bounds__(kPlanThreads) page_reserve_kernel(const PageMapParams m, const int32_t *new_lens,
                                                                    const int32_t *reqs, int n, int can_copy, void *ws,
                                                                    int32_t *dev_status) {
    __shared__ int s_warp[kPlanWarps];
    __shared__ int2 s_entry[kPlanThreads];  // request and part-filled last page (or -1) of list entry i
    __shared__ int s_first[kPlanThreads];   // rank of its first page among those handed out
    __shared__ unsigned long long s_need;   // pages that all of them need
    grid_dependency_wait();
    const PageLists lists(ws, m.num_pages);
    const int tid = threadIdx.x;
    uint32_t err = 0;
    int r = -1, len = 0, want = 0, last = -1, fresh = 0;
    if (tid < n) {
        r = reqs ? reqs[tid] : tid;
        if (r < 0 || r >= m.num_reqs) {
            err = SFI_DEV_BAD_INDEX;
        } else {
            len = m.seq_lens[r];
            want = new_lens[tid];
            if (len < 0 || want < len || (int64_t)want > (int64_t)m.max_pages * kSubTokens) {
                err = SFI_DEV_BAD_LEN;
            } else {
                fresh = pages_of(want) - pages_of(len);
                if (want > len && len % kSubTokens) {
                    last = m.page_table[(int64_t)r * m.max_pages + len / kSubTokens];
                    if (last < 0 || last >= m.num_pages) {
                        err = SFI_DEV_BAD_PAGE;
                        last = -1;
                    }
                }
            }
        }
    }
    s_entry[tid] = make_int2(r, last);
    if (tid == 0) {
        lists.moves[0] = 0;
        s_need = 0;
    }
    __syncthreads();
    int before = 0;  // holders of the same last page that come earlier in the list
    bool twice = false;
#pragma unroll 8
    for (int i = 0; i < min(tid & ~31, n); ++i) {  // the warps before this one, then its own lanes
        const int2 e = s_entry[i];
        before += e.y == last;
        twice |= e.x == r;
    }
    const uint32_t lower = (1u << (tid & 31)) - 1u;
    before += __popc(__match_any_sync(0xffffffffu, last) & lower);
    twice |= (__match_any_sync(0xffffffffu, r) & lower) != 0;
    if (tid < n && r >= 0 && twice) err = SFI_DEV_BAD_INDEX;  // named twice
    if (__syncthreads_or(err != 0)) {
        if (err) report(dev_status, err);
        return;
    }
    // a shared last page is copied, except by the last of its holders in the list when they
    // are all there are
    const bool copy = last >= 0 && m.ref_count[last] - before > 1;
    // (a row of the table may have 2^27 pages, so 1024 requests may ask for more than 32 bits count;
    // the scan's sums hold when there are that many pages at all)
    block_sum(fresh + copy, &s_need);
    int total = 0, copies = 0;
    const int first = block_scan(fresh + copy, s_warp, &total);
    const int move = block_scan(copy, s_warp, &copies);
    s_first[tid] = first;
    if (copies && !can_copy) {
        if (tid == 0) report(dev_status, SFI_DEV_BAD_PAGE);
        return;
    }
    if (s_need > (unsigned long long)m.num_pages) {
        if (tid == 0) report(dev_status, SFI_DEV_NO_PAGE);
        return;
    }
    // the `total` lowest free pages
    int found = 0;
    for (int base = 0; base < m.num_pages && found < total; base += kPlanThreads * 4) {
        const int p0 = base + tid * 4;
        int c[4], k = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[i] = p0 + i < m.num_pages ? m.ref_count[p0 + i] : 1;
            k += c[i] == 0;
        }
        int here = 0;
        int at = found + block_scan(k, s_warp, &here);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c[i] == 0) {
                if (at < total) lists.ids[at] = p0 + i;
                ++at;
            }
        found += here;
    }
    if (found < total) {
        if (tid == 0) report(dev_status, SFI_DEV_NO_PAGE);
        return;
    }
    __syncthreads();  // ids are written, counts are read
    for (int i = tid; i < total; i += kPlanThreads) m.ref_count[lists.ids[i]] = 1;
    if (tid < n) {
        if (copy) {
            lists.src[move] = last;
            lists.dst[move] = lists.ids[first];
            atomicSub(m.ref_count + last, 1);
        }
        m.seq_lens[r] = want;
    }
    if (tid == 0) lists.moves[0] = copies;
    // table entries: a warp per request (entries [full pages, pages wanted) take the next ids)
    for (int e = tid >> 5; e < n; e += kPlanWarps) {
        const int rr = reqs ? reqs[e] : e;
        const int before = e + 1 < n ? s_first[e + 1] : total;
        const int have = before - s_first[e];
        const int end = pages_of(new_lens[e]);
        for (int i = tid & 31; i < have; i += 32)
            m.page_table[(int64_t)rr * m.max_pages + end - have + i] = lists.ids[s_first[e] + i];
    }
}

// ---- compact: one CTA pairs the live pages behind the first N with the holes before it ---
__global__ void __launch_bounds__(kPlanThreads) page_compact_plan_kernel(const PageMapParams m, int32_t *ref_out,
                                                                         int32_t *live_out, void *ws) {
    __shared__ int s_warp[kPlanWarps];
    grid_dependency_wait();
    const PageLists lists(ws, m.num_pages);
    const int tid = threadIdx.x;
    int mine = 0;
#pragma unroll 8
    for (int i = tid; i < m.num_pages; i += kPlanThreads) mine += m.ref_count[i] > 0;
    int live = 0;
    block_scan(mine, s_warp, &live);
    // below N: holes in order; from N on: movers in order; there are as many of each. A warp
    // takes 32 kEach pages in a row; its ranks come from ballots, and one scan over the warps
    // serves both lists (holes in the lower half).
    constexpr int kEach = 8;
    const int lane = tid & 31;
    const uint32_t lower = (1u << lane) - 1u;
    int holes = 0, movers = 0;
    for (int base = 0; base < m.num_pages; base += kPlanThreads * kEach) {
        const int p0 = base + (tid >> 5) * (32 * kEach) + lane;
        int c[kEach], count = 0;
        uint32_t hole[kEach], mover[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) c[k] = p0 + 32 * k < m.num_pages ? m.ref_count[p0 + 32 * k] : 0;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = p0 + 32 * k;
            hole[k] = __ballot_sync(0xffffffffu, i < live && c[k] <= 0);
            mover[k] = __ballot_sync(0xffffffffu, i >= live && i < m.num_pages && c[k] > 0);
            count += __popc(hole[k]) | __popc(mover[k]) << 16;
        }
        int both = 0;
        // the warp's count enters the scan through its first lane; every lane gets what came before
        const int before = __shfl_sync(0xffffffffu, block_scan(lane == 0 ? count : 0, s_warp, &both), 0);
        int h = holes + (before & 0xffff), v = movers + (before >> 16);
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = p0 + 32 * k;
            if (i < m.num_pages) {
                const bool moves = (mover[k] >> lane) & 1u;
                if ((hole[k] >> lane) & 1u) lists.dst[h + __popc(hole[k] & lower)] = i;
                if (moves) lists.src[v + __popc(mover[k] & lower)] = i;
                lists.ids[i] = i;
                ref_out[i] = moves ? 0 : c[k];
            }
            h += __popc(hole[k]);
            v += __popc(mover[k]);
        }
        holes += both & 0xffff;
        movers += both >> 16;
    }
    __syncthreads();
    constexpr int kMoves = 4;  // moves of a thread whose loads are in flight together
    for (int i0 = tid; i0 < movers; i0 += kPlanThreads * kMoves) {
        int from[kMoves], to[kMoves], held[kMoves];
#pragma unroll
        for (int k = 0; k < kMoves; ++k) {
            const int i = i0 + k * kPlanThreads;
            from[k] = i < movers ? lists.src[i] : -1;
            to[k] = i < movers ? lists.dst[i] : 0;
        }
#pragma unroll
        for (int k = 0; k < kMoves; ++k) held[k] = from[k] >= 0 ? m.ref_count[from[k]] : 0;
#pragma unroll
        for (int k = 0; k < kMoves; ++k)
            if (from[k] >= 0) {
                lists.ids[from[k]] = to[k];
                ref_out[to[k]] = held[k];
            }
    }
    if (tid == 0) {
        lists.moves[0] = movers;
        *live_out = live;
    }
}

namespace {

cudaError_t launch_copy(const PagePoolParams &q, const int32_t *src, const int32_t *dst, int n, int most,
                        const int32_t *n_dev, const PageMapParams &m, const int32_t *new_ids, int32_t *table_out,
                        int32_t *dev_status, cudaStream_t stream) {
    const int sms = sm_count_current_device();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const int64_t chunks = (q.page_bytes + kCopyChunk - 1) / kCopyChunk;
    const int64_t items = std::max<int64_t>((int64_t)most * q.num_pools * chunks, table_out ? m.num_reqs : 0);
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(items, (int64_t)sms * 8));
    const bool small = !table_out && q.page_bytes <= kCopyChunk / 2;
    return launch_dependent(small ? page_copy_kernel<false> : page_copy_kernel<true>, grid, kPageThreads, 0, stream, q.pools, q.num_pools, q.page_bytes,
                            q.num_pages, src, dst, n, n_dev, m, new_ids, table_out, dev_status);
}

}  // namespace

size_t page_workspace_bytes(int32_t num_pages) { return ((size_t)num_pages * 3 + 4) * 4; }

cudaError_t launch_page_copy(const PagePoolParams &q, const int32_t *src, const int32_t *dst, int n,
                             int32_t *dev_status, cudaStream_t stream) {
    return launch_copy(q, src, dst, n, n, nullptr, PageMapParams{}, nullptr, nullptr, dev_status, stream);
}

cudaError_t launch_page_fork(const PageMapParams &m, const int32_t *src, const int32_t *dst, const int32_t *fork_lens,
                             int n, int32_t *dev_status, cudaStream_t stream) {
    return launch_dependent(page_fork_kernel, n, kPageThreads, 0, stream, m, src, dst, fork_lens, dev_status);
}

cudaError_t launch_page_free(const PageMapParams &m, const int32_t *reqs, int n, int32_t *dev_status,
                             cudaStream_t stream) {
    return launch_dependent(page_free_kernel, n, kPageThreads, 0, stream, m, reqs, dev_status);
}

cudaError_t launch_page_reserve(const PageMapParams &m, const PagePoolParams *q, const int32_t *new_lens,
                                const int32_t *reqs, int n, void *ws, int32_t *dev_status, cudaStream_t stream) {
    const cudaError_t e = launch_dependent(page_reserve_kernel, 1, kPlanThreads, 0, stream, m, new_lens, reqs, n,
                                           q != nullptr ? 1 : 0, ws, dev_status);
    if (e != cudaSuccess || !q) return e;
    const PageLists lists(ws, m.num_pages);
    return launch_copy(*q, lists.src, lists.dst, 0, n, lists.moves, PageMapParams{}, nullptr, nullptr, dev_status, stream);
}

cudaError_t launch_page_compact(const PageMapParams &m, const PagePoolParams &q, int32_t *table_out, int32_t *ref_out,
                                int32_t *live_out, void *ws, int32_t *dev_status, cudaStream_t stream) {
    const cudaError_t e = launch_dependent(page_compact_plan_kernel, 1, kPlanThreads, 0, stream, m, ref_out, live_out, ws);
    if (e != cudaSuccess) return e;
    const PageLists lists(ws, m.num_pages);
    return launch_copy(q, lists.src, lists.dst, 0, m.num_pages / 2, lists.moves, m, lists.ids, table_out, dev_status,
                       stream);
}

}  // namespace sfi
