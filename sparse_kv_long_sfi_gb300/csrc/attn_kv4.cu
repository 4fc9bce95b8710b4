// Attention over the 4-bit cache: dense (with the Selector's scores) and over the sparse
// state, one to sixteen query rows per KV head.
//
//   o = sum_j softmax_j(scale q . k_j) v_j,  lse,  scores_j = sum over rows of scale q . k_j
//
// The work is the blocks of all (request, KV head) units in one row; every warp of the
// grid takes an equal run of it, so a ragged batch, one long request and many short ones
// are all spread evenly, and the launch needs no bound on the lengths. Runs of one unit
// meet by log-sum-exp: within a CTA through shared memory, across CTAs through the
// workspace, where the last CTA of a unit adds the parts in order (the result does not
// depend on which one that is).
//
// Few units of few blocks are latency: there, a unit belongs to a cluster of CTAs, which finds
// its blocks without the others' lengths and adds up its parts in shared memory (cluster_of).
//
// Per block (16 tokens): S^T = K Q^T and O^T += V^T P^T with mma.m16n8k16, the tokens (or
// dims) as the M side, so that eight query rows take one N tile. Codes become fp16 by
// conversion and one multiplication by their scale: a product of an e2m1 and an e4m3
// value is exact in fp16. So is Q in fp16, each row scaled by a power of two to just below 2^15:
// a value below 2^-31 of its row's largest loses bits, at most 2^-39 of that largest one. P goes in as two fp16 terms (22 bits; times 2^7 to keep small
// probabilities off the subnormals), so the output is as good as fp32's. The running
// maximum moves only when a score passes it by 2^8.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kv4_format.cuh"

namespace sfi {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.f;   // the maximum may lag by this (in powers of two)
constexpr float kLift = 7.f;   // P is computed times 2^7
constexpr int kKv4MaxCluster = 8;  // CTAs of a cluster

enum Kv4Mode : int { kKv4Dense = 0, kKv4Scores = 1, kKv4Fast = 2 };

// ROWS: the query rows of a KV head that a variant takes. Up to four, P's two terms share
// the N tile (columns 0..3 the first, 4..7 the second, over the same rows); up to eight,
// they take an instruction each; up to sixteen, there are two N tiles, whose accumulators leave
// room for one CTA per SM. Two rows (the slow step of 16 x 16K tokens, 16/8/128 heads) take
// 65.2 us in the first variant, 73.0 in the second, 99.9 in the third; eight rows (refresh and
// fast step of 32 x 1792 rows, 2 tokens x 4 heads, as runs of the row) 97.8 us in the second and 108 in the third.
template <int D, int ROWS>
struct Tile {
    static constexpr int kNt = ROWS > 8 ? 2 : 1;
    static constexpr bool kShared = ROWS <= 4;
    static constexpr int kWarps = 8;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kParts = 2 * kWarps;  // partials of a CTA: the first and the last run of each warp
    static constexpr int kDepth = 4;           // blocks in flight per warp
    static constexpr int kRing = kDepth * Kv4<D>::kBlock;
    static constexpr int kPart = ROWS * D * 4;  // a partial O
    static constexpr int kFirst = kWarps * kRing;  // partials of first runs
    static constexpr int kSmem = kFirst + kWarps * kPart;
    // in clusters, behind that: a CTA's share of all CTAs' sums (D / 4 items of 24 bytes a row, rounded up)
    static constexpr int kClusterSmem = kSmem + (ROWS * (D / 4) + kKv4MaxCluster) * 24;
    static_assert(ROWS * (D / 4) <= 2 * kThreads, "a thread takes one item of a CTA's share");
    static_assert(kRing >= kPart, "a warp's ring holds its last partial");
    static_assert(kSmem >= kThreads * 24, "the merge's arrays lie where the rings were");
};

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// The stream is read once: it must not push what stays (code, queries, partials) out of L2.
__device__ __forceinline__ void cp_async16(void *dst, const void *src, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint.L2::256B [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
                 "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// What a request's units consist of: compact blocks [0, ncomp), then pages [page0, page0 + n - ncomp).
struct ReqPlan {
    int L, n, ncomp, page0, nvis;  // nvis: selected rows
    int64_t cblock;
    int cap;
};

__device__ __forceinline__ int request_id(const Kv4AttnParams &p, int b) {
    return p.req_ids ? p.req_ids[p.first + b] : p.first + b;
}

template <int MODE>
__device__ __forceinline__ ReqPlan plan_request(const Kv4AttnParams &p, int b, uint32_t *err) {
    const int r = request_id(p, b);
    ReqPlan q{};
    q.L = p.seq_lens[r];
    int cnt = 0, cap = 0;
    int64_t off = 0;
    if (MODE == kKv4Fast) {  // all on their way before the first is looked at
        cnt = p.c_count[r];
        cap = p.c_capacity[r];
        off = p.c_page_offset[r];
    }
    if (q.L < p.tokens || q.L > p.max_pages * kSubTokens || (MODE == kKv4Scores && q.L > p.score_stride)) {
        *err |= SFI_DEV_BAD_LEN;
        return q;
    }
    if (MODE != kKv4Fast) {
        q.n = (q.L + 15) / 16;
        return q;
    }
    const int64_t rows = (int64_t)min(p.sink, q.L) + cnt;
    const int ncomp = (int)((rows + 15) / 16);
    if (cnt < 0 || cap < 0 || ncomp > cap || (cnt > 0 && q.L - p.tokens + 1 < p.sink)) {
        *err |= SFI_DEV_K_OVERFLOW;
        return q;
    }
    if (off < 0 || off + (int64_t)p.hkv * cap > p.c_total_pages) {
        *err |= SFI_DEV_BAD_COMPACT;
        return q;
    }
    q.nvis = cnt;
    q.ncomp = ncomp;
    q.cblock = off;
    q.cap = cap;
    const int lo = max(p.sink, q.L - p.tokens + 1 - p.recent);
    q.page0 = lo / 16;
    const int last = (q.L - 1) / 16;
    q.n = ncomp + (lo < q.L ? last - q.page0 + 1 : 0);
    if (q.n == 0) {  // nothing to see: one page, masked
        q.page0 = last;
        q.n = 1;
    }
    return q;
}

// A place in the row of work: block `pg` of KV head h of request b.
struct Place {
    int b, h, pg;
};

__device__ __forceinline__ Place locate(const int64_t *prefix, int batch, int hkv, int64_t f) {
    int lo = 0, hi = batch - 1;
    while (lo < hi) {  // the last request that starts at or before f (empty ones start where the next does)
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] * hkv <= f) lo = mid; else hi = mid - 1;
    }
    const int64_t n = prefix[lo + 1] - prefix[lo], in = f - prefix[lo] * hkv;
    Place at;
    at.b = lo;
    at.h = (int)quotient(in, n);
    at.pg = (int)(in - at.h * n);
    return at;
}

// Four dims of a row, gathered from partial states by log-sum-exp.
struct Gathered {
    float mx = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    // N parts (m = -inf, l = 0, x = 0 where there is none)
    template <int N>
    __device__ __forceinline__ void add(const float2 (&ml)[N], const float4 (&x)[N]) {
        float now = mx;
#pragma unroll
        for (int i = 0; i < N; ++i) now = fmaxf(now, ml[i].x);
        const float keep = mx == now ? 1.f : fast_exp2(mx - now);
        mx = now;
        sum *= keep;
        acc.x *= keep;
        acc.y *= keep;
        acc.z *= keep;
        acc.w *= keep;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float w = ml[i].x == now ? 1.f : fast_exp2(ml[i].x - now);
            sum = fmaf(w, ml[i].y, sum);
            acc.x = fmaf(w, x[i].x, acc.x);
            acc.y = fmaf(w, x[i].y, acc.y);
            acc.z = fmaf(w, x[i].z, acc.z);
            acc.w = fmaf(w, x[i].w, acc.w);
        }
    }
};

// Four values of an output row (at `at`); lse_at >= 0: its log-sum-exp too.
__device__ __forceinline__ void write_row(const Kv4AttnParams &p, int64_t at, const Gathered &g, int64_t lse_at) {
    const float w = g.sum == 0.f ? 0.f : p.v_scale / g.sum;
    float2 *out = reinterpret_cast<float2 *>(p.out + at);
    out[0] = make_float2(g.acc.x * w, g.acc.y * w);
    out[1] = make_float2(g.acc.z * w, g.acc.w * w);
    if (p.lse && lse_at >= 0) p.lse[lse_at] = g.sum == 0.f ? -INFINITY : (g.mx - kLift + log2f(g.sum)) * kLn2;
}

// Run w of `parts` nearly equal runs of [0, total): the first total % parts are one longer.
struct Runs {
    int64_t parts, q, r;
    __device__ __forceinline__ Runs(int64_t total, int64_t n) : parts(n), q(quotient(total, n)), r(total - q * n) {}
    __device__ __forceinline__ int64_t start(int64_t w) const { return w * q + min(w, r); }
    __device__ __forceinline__ int64_t owner(int64_t f) const {
        return f < r * (q + 1) ? quotient(f, q + 1) : r + quotient(f - r * (q + 1), q);
    }
};

// The warps' runs over as many CTAs as there is work for. Where a full grid would get less than
// one or two blocks per warp, fewer warps take that many (figures of page tables too wide for
// clusters): one is the shortest chain (1K tokens of one request: 9.4 us, 10.9 with two at least). Up to four, long units are better cut into whole
// pairs (one request of 16K tokens: 16.7 us with four blocks, 18.3 with 3.3 on average; 4 tokens of
// one request of 8K: 24.9 and 27.7), while short ones, with their many edges, are better spread
// (64 requests of 200 tokens: 22.4 us with 2.7 blocks on average, 25.0 with four).
template <int kWarps>
__device__ __forceinline__ Runs runs_of(const Kv4AttnParams &p, const int64_t *prefix) {
    const int64_t total = prefix[p.batch] * p.hkv, grid = (int64_t)gridDim.x * kWarps;
    const bool long_units = prefix[p.batch] >= 128 * (int64_t)p.batch;  // 2K tokens on average
    const int least = total <= grid ? 1 : (total > 2 * grid && total <= 4 * grid && long_units ? 4 : 2);
    const int64_t ctas = min((int64_t)gridDim.x, (total + kWarps * least - 1) / (kWarps * least));
    return Runs(total, max(ctas * kWarps, (int64_t)1));
}

}  // namespace

// CLUSTER: a cluster of CTAs takes one unit, see cluster_of; otherwise a warp takes a run of the row.
template <int D, int ROWS, int MODE, bool CLUSTER>
__global__ void __launch_bounds__(Tile<D, ROWS>::kThreads, ROWS <= 8 ? 2 : 1) kv4_attn_kernel(const Kv4AttnParams p) {
    using F = Kv4<D>;
    using T = Tile<D, ROWS>;
    constexpr int NT = T::kNt, kWarps = T::kWarps, kThreads = T::kThreads, kParts = T::kParts;
    constexpr int kKs = D / 16;  // k steps of S, and m tiles of O
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_prefix[kKv4MaxBatch + 1];
    __shared__ int64_t s_unit0[kParts];             // first block of a partial's unit
    __shared__ int s_unit[kParts];                  // its unit, or -1
    __shared__ int s_bad[kParts];                   // its run met a bad page id
    __shared__ float s_ml[kParts][ROWS][2];
    __shared__ int s_last[2], s_open[2], s_lead[kParts];
    __shared__ int64_t s_open0[2];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;

    grid_dependency_wait();
    grid_launch_dependents();  // not before the wait: see launch_dependent_clusters
    uint32_t none = 0;  // (a request's errors are reported once, where its blocks are counted)
    Place at{};
    ReqPlan aplan{};
    int run;  // blocks of this warp
    int64_t f0 = 0;
    const int gshift = __ffs(p.group) - 1;  // the group size is a power of two
    // a unit's query rows as they lie (lane (g, t): dims t D/4 .. of row g)
    auto load_query = [&](const Place &x, int4 (&raw_q)[NT][D / 32]) {
        const int64_t tok0 = (int64_t)request_id(p, x.b) * p.tokens;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = T::kShared ? g & 3 : nt * 8 + g;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) raw_q[nt][i] = make_int4(0, 0, 0, 0);
            if (row < p.rows) {
                const int head = x.h * p.group + (row & (p.group - 1));
                const __nv_bfloat16 *src = p.q + ((tok0 + (row >> gshift)) * p.hq + head) * D + t * (D / 4);
#pragma unroll
                for (int i = 0; i < D / 32; ++i) raw_q[nt][i] = *reinterpret_cast<const int4 *>(src + i * 8);
            }
        }
    };
    int4 raw_query[NT][D / 32];
    if constexpr (CLUSTER) {
        // ---- this cluster's unit, in equal runs over its warps ----
        const int unit = blockIdx.x / cluster_nctarank(), rank = cluster_ctarank();
        const int parts = kWarps * cluster_nctarank(), part = rank * kWarps + warp;
        at.b = unit / p.hkv;
        at.h = unit - at.b * p.hkv;
        if (cluster_nctarank() > 1) cluster_arrive_relaxed();  // (waited for before the first remote store)
        load_query(at, raw_query);  // on their way while the plan and the blocks are fetched
        uint32_t err = 0;
        aplan = plan_request<MODE>(p, at.b, &err);
        if (err && tid == 0 && rank == 0 && at.h == 0) report(p.dev_status, err);
        if (aplan.n == 0) {  // every CTA of the cluster
            if (cluster_nctarank() > 1) cluster_wait();
            return;
        }
        const int q = aplan.n / parts, r = aplan.n - q * parts;
        at.pg = part * q + min(part, r);
        run = q + (part < r);
    } else {
        // ---- the row of work: blocks of each request, summed up (every warp for itself) ----
        uint32_t err = 0;
        int64_t carry = 0;
        for (int base = 0; base < p.batch; base += 32) {
            const int b = base + lane;
            const int64_t v = b < p.batch ? plan_request<MODE>(p, b, &err).n : 0;
            int64_t incl = v;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int64_t o = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += o;
            }
            if (b < p.batch) s_prefix[b] = carry + incl - v;
            carry += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) s_prefix[p.batch] = carry;
        if (err && blockIdx.x == 0 && warp == 0) report(p.dev_status, err);
        if (lane < 2) s_unit[2 * warp + lane] = -1;
        if (tid < 2) s_open[tid] = -1;
        __syncwarp();
        const Runs runs = runs_of<kWarps>(p, s_prefix);
        if (s_prefix[p.batch] == 0 || (int64_t)blockIdx.x * kWarps >= runs.parts) return;
        f0 = runs.start((int64_t)blockIdx.x * kWarps + warp);
        run = (int)(runs.start((int64_t)blockIdx.x * kWarps + warp + 1) - f0);
        if (run > 0) {
            at = locate(s_prefix, p.batch, p.hkv, f0);
            load_query(at, raw_query);  // on their way while page ids and blocks are fetched
            aplan = plan_request<MODE>(p, at.b, &none);
        }
    }

    // ---- copies: this warp's blocks, kDepth of them in flight ----
    uint8_t *ring = smem + warp * T::kRing;
    const uint64_t policy = l2_policy_evict_first();
    Place ahead = at;
    int ids = 0, ids_base = 0;     // page ids of the unit, 32 at a time (lane i: number ids_base + i)
    const int32_t *id_row = nullptr;
    int left = run;                  // those still to be copied
    uint32_t bad_units = 0;        // bit (number of the unit in this run) % 32: it has a bad page id
    int unit_ahead = 0, unit_here = 0;
    bool unchecked = false;        // ids are on their way (a cluster's first copies do not wait for them)
    auto load_ids = [&](int first) {
        ids_base = first;
        ids = first + lane < aplan.n - aplan.ncomp ? id_row[first + lane] : 0;
    };
    auto check_ids = [&]() {
        const bool out = (uint32_t)ids >= (uint32_t)p.num_pages;
        if (out) ids = 0;  // any page: the unit writes nothing
        if (__any_sync(0xffffffffu, out)) {
            bad_units |= 1u << (unit_ahead & 31);
            if (lane == 0) report(p.dev_status, SFI_DEV_BAD_PAGE);
        }
    };
    auto enter_ahead = [&]() {
        id_row = p.page_table + (int64_t)request_id(p, ahead.b) * p.max_pages + aplan.page0;
        bad_units &= ~(1u << (unit_ahead & 31));
        load_ids(max(0, ahead.pg - aplan.ncomp));
        if constexpr (CLUSTER) unchecked = true;
        else check_ids();
    };
    auto issue = [&](int slot) {
        if (left > 0) {
            const uint8_t *src;
            if (MODE == kKv4Fast && ahead.pg < aplan.ncomp) {
                src = p.c_pool + (aplan.cblock + (int64_t)ahead.h * aplan.cap + ahead.pg) * F::kBlock;
            } else {
                const int i = ahead.pg - aplan.ncomp;
                if (i >= ids_base + 32) {
                    load_ids(i);
                    check_ids();
                } else if (CLUSTER && unchecked) {
                    check_ids();
                }
                unchecked = false;
                const int page = __shfl_sync(0xffffffffu, ids, i - ids_base);
                src = p.pool + ((int64_t)page * p.hkv + ahead.h) * F::kBlock;
            }
            src += lane * 16;
            uint8_t *dst = ring + slot * F::kBlock + lane * 16;
#pragma unroll
            for (int c = 0; c < F::kBlock / 16; c += 32)
                if (c + 32 <= F::kBlock / 16 || lane < F::kBlock / 16 - c) cp_async16(dst + c * 16, src + c * 16, policy);
            --left;
            if (++ahead.pg == aplan.n && left > 0) {  // (not in a cluster, whose warps have one unit)
                ahead.pg = 0;
                if (++ahead.h == p.hkv) {
                    ahead.h = 0;
                    do ++ahead.b; while (s_prefix[ahead.b + 1] == s_prefix[ahead.b]);
                }
                ++unit_ahead;
                aplan = plan_request<MODE>(p, ahead.b, &none);
                enter_ahead();
            }
        }
        cp_async_commit();
    };
    if (run > 0) enter_ahead();
#pragma unroll
    for (int i = 0; i < T::kDepth; ++i) issue(i);

    // ---- this warp's units ----
    uint32_t bq[NT][kKs][2];     // Q as B fragments
    float mul[NT][2];            // fp16 product -> score in powers of two
    float o[NT][kKs][4];
    float base[NT][2], l[NT][2];  // kLift - running maximum (+inf: nothing seen), sum of 2^(score + base)
    ReqPlan plan{};
    int f = 0, unit0 = 0;        // this block, and the first of its unit, counted from the warp's first
    int slot = 0;
    bool drop = false;   // scores mode: the request has a bad page id
    int looked_at = -1;  // the request that this says
    const bool multi = p.tokens > 1;
    // blocks that every row sees whole: [0, in_comp) and [in_from, in_to)
    int in_comp = 0, in_from = 0, in_to = 0;
    float *score_row = nullptr;

    // positions (or compact rows) [lo, hi) that query token i sees
    auto span = [&](bool comp, int i, int &lo, int &hi) {
        const int Lt = plan.L - p.tokens + 1 + i;
        if (MODE == kKv4Fast) {
            lo = comp ? 0 : max(p.sink, Lt - p.recent);
            hi = comp ? min(p.sink, Lt) + plan.nvis : Lt;
        } else {
            lo = 0;
            hi = Lt;
        }
    };

    auto token_of = [&](int row) { return min(row >> gshift, p.tokens - 1); };
    auto row_of = [&](int nt, int c) { return T::kShared ? (2 * t + c) & 3 : nt * 8 + 2 * t + c; };
    const float second = T::kShared && t >= 2 ? -1.f : 0.f;  // this lane's columns take P's second term

    auto enter_unit = [&](const int4 (&raw_q)[NT][D / 32]) {
        if constexpr (CLUSTER) plan = aplan;
        else plan = plan_request<MODE>(p, at.b, &none);
        unit0 = f - at.pg;
        const int r = request_id(p, at.b);
        if (MODE == kKv4Scores && looked_at != at.b) {
            // scores are written on the way, so all page ids of the request are looked at before
            looked_at = at.b;
            const int32_t *row = p.page_table + (int64_t)r * p.max_pages;
            bool out = false;
            auto look = [&](int id) { out |= (uint32_t)id >= (uint32_t)p.num_pages; };
            int done = 0;
            if ((reinterpret_cast<uintptr_t>(row) & 15u) == 0) {  // four ids at a time
                done = plan.n & ~3;
#pragma unroll 8
                for (int i = lane * 4; i < done; i += 128) {
                    const int4 id = *reinterpret_cast<const int4 *>(row + i);
                    look(id.x);
                    look(id.y);
                    look(id.z);
                    look(id.w);
                }
            }
#pragma unroll 4
            for (int i = done + lane; i < plan.n; i += 32) look(row[i]);
            drop = __any_sync(0xffffffffu, out);
        }
        {
            int lo_a, hi_a, lo_z, hi_z;
            span(false, 0, lo_a, hi_a);
            span(false, p.tokens - 1, lo_z, hi_z);
            // pages from ceil(lo_z / 16) to floor(hi_a / 16), counted in blocks of the unit
            in_from = (lo_z + 15) / 16 - plan.page0 + plan.ncomp;
            in_to = hi_a / 16 - plan.page0 + plan.ncomp;
            in_from = max(in_from, plan.ncomp);
            if (MODE == kKv4Fast) {
                span(true, 0, lo_a, hi_a);
                in_comp = hi_a / 16;
            }
        }
        if (MODE == kKv4Scores) score_row = p.scores + ((int64_t)r * p.hkv + at.h) * p.score_stride;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int4(&raw)[D / 32] = raw_q[nt];
            // the row's largest magnitude, as bits; 2^shift takes it to [2^14, 2^15)
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint32_t w[4] = {(uint32_t)raw[i].x, (uint32_t)raw[i].y, (uint32_t)raw[i].z, (uint32_t)raw[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) top = max(top, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int e = (int)(top >> 7);  // biased exponent; 255: the row holds an infinity or NaN
            // up and down both stay in fp32's normal range (a subnormal row counts as exponent 1)
            const int shift = e == 255 ? 0 : min(14 + 127 - max(e, 1), 126);
            const float up = __uint_as_float((uint32_t)(127 + shift) << 23);
            const float down = __uint_as_float((uint32_t)(127 - shift) << 23);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {  // k steps 2 i and 2 i + 1: four dims each of these eight
                float x[8];
                bf16x8_to_f32(raw[i], x);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    bq[nt][2 * i + k][0] = pack_f16x2(x[4 * k] * up, x[4 * k + 1] * up);
                    bq[nt][2 * i + k][1] = pack_f16x2(x[4 * k + 2] * up, x[4 * k + 3] * up);
                }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {  // S^T's columns 2t, 2t + 1 are this lane's
                mul[nt][c] = __shfl_sync(0xffffffffu, down, (2 * t + c) * 4) * p.k_mul * kLog2e;
                base[nt][c] = INFINITY;
                l[nt][c] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < kKs; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[nt][j][c] = 0.f;
        }
    };

    // S^T of PB blocks: rows g -> tokens tu and (g + 8) tu + 2, columns 2t, 2t + 1
    const int tu = 4 * (g >> 1) + (g & 1);
    auto products = [&](auto pb_tag, const uint8_t *blk0, const uint8_t *blk1, auto &s) {
        constexpr int PB = decltype(pb_tag)::value;
        uint32_t ka[PB][D / 32], kb[PB][D / 32];  // codes of the two tokens, dims t D/4 ...
        uint32_t sa[PB][D / 64], sb[PB][D / 64];  // their scales, twice in a register
#pragma unroll
        for (int b = 0; b < PB; ++b) {
            const uint8_t *blk = b ? blk1 : blk0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c) s[b][nt][c] = 0.f;
            if constexpr (D == 128) {
                const uint4 x = *reinterpret_cast<const uint4 *>(blk + tu * F::kKRow + t * 16);
                const uint4 y = *reinterpret_cast<const uint4 *>(blk + (tu + 2) * F::kKRow + t * 16);
                ka[b][0] = x.x; ka[b][1] = x.y; ka[b][2] = x.z; ka[b][3] = x.w;
                kb[b][0] = y.x; kb[b][1] = y.y; kb[b][2] = y.z; kb[b][3] = y.w;
                const uint32_t ha = e4m3x2_to_f16(*reinterpret_cast<const uint16_t *>(blk + F::kKScale + tu * 8 + t * 2));
                const uint32_t hb =
                    e4m3x2_to_f16(*reinterpret_cast<const uint16_t *>(blk + F::kKScale + (tu + 2) * 8 + t * 2));
                sa[b][0] = __byte_perm(ha, 0, 0x1010); sa[b][1] = __byte_perm(ha, 0, 0x3232);
                sb[b][0] = __byte_perm(hb, 0, 0x1010); sb[b][1] = __byte_perm(hb, 0, 0x3232);
            } else {
                const uint2 x = *reinterpret_cast<const uint2 *>(blk + tu * F::kKRow + t * 8);
                const uint2 y = *reinterpret_cast<const uint2 *>(blk + (tu + 2) * F::kKRow + t * 8);
                ka[b][0] = x.x; ka[b][1] = x.y;
                kb[b][0] = y.x; kb[b][1] = y.y;
                sa[b][0] = __byte_perm(e4m3x2_to_f16(blk[F::kKScale + tu * 4 + t]), 0, 0x1010);
                sb[b][0] = __byte_perm(e4m3x2_to_f16(blk[F::kKScale + (tu + 2) * 4 + t]), 0, 0x1010);
            }
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
#pragma unroll
            for (int b = 0; b < PB; ++b) {
                uint32_t xa[4], xb[4];
                e2m1x8_to_f16(ka[b][w], xa);
                e2m1x8_to_f16(kb[b][w], xb);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t a[4] = {hmul2(xa[2 * k], sa[b][w / 2]), hmul2(xb[2 * k], sb[b][w / 2]),
                                           hmul2(xa[2 * k + 1], sa[b][w / 2]), hmul2(xb[2 * k + 1], sb[b][w / 2])};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16_16816(s[b][nt], a, bq[nt][2 * w + k][0], bq[nt][2 * w + k][1]);
                }
            }
        }
    };

    // PB blocks from blk on (EDGE: one block, some of whose tokens some rows do not see).
    auto consume = [&](auto pb_tag, auto edge_tag, uint8_t *blk0, uint8_t *blk1) {
        constexpr int PB = decltype(pb_tag)::value;
        constexpr bool EDGE = decltype(edge_tag)::value;
        const bool comp = EDGE && MODE == kKv4Fast && at.pg < plan.ncomp;
        const int pos0 = 16 * (comp ? at.pg : plan.page0 + at.pg - plan.ncomp);
        float s[PB][NT][4];
        products(pb_tag, blk0, blk1, s);
        if constexpr (!EDGE) {
            // V scales in fp16 for the whole warp, where the K codes were: lane w converts word w
            // (four tokens of one group)
            __syncwarp();
#pragma unroll
            for (int b = 0; b < PB; ++b) {
                uint8_t *blk = b ? blk1 : blk0;
                if (D == 128 || lane < D / 4) {
                    const uint32_t w = *reinterpret_cast<const uint32_t *>(blk + F::kVScale + lane * 4);
                    *reinterpret_cast<uint2 *>(blk + lane * 8) =
                        make_uint2(e4m3x2_to_f16((uint16_t)w), e4m3x2_to_f16((uint16_t)(w >> 16)));
                }
            }
            __syncwarp();
        }
        // ---- scores (natural units), masks, exponents ----
        uint32_t hide = 0;  // bits 4 nt + c: not seen
        if (EDGE) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    int lo, hi;
                    span(comp, token_of(row_of(nt, c & 1)), lo, hi);
                    const int pos = pos0 + tu + (c & 2);
                    if (pos < lo || pos >= hi) hide |= 1u << (4 * nt + c);
                }
        }
        if (MODE == kKv4Scores) {
            // The rows' sum of each token (rows that are not there hold zeros). Over the four lanes
            // of a token group the sums end up one in each: lane t has token tu + 2 (t & 1) of block
            // t / 2. With shared columns lanes t and t + 2 hold the same rows.
            float one[PB];
#pragma unroll
            for (int b = 0; b < PB; ++b) {
                float sum[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    sum[k] = 0.f;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            if (!EDGE || !((hide >> (4 * nt + 2 * k + c)) & 1u))
                                sum[k] = fmaf(s[b][nt][2 * k + c], mul[nt][c], sum[k]);
                }
                const float give = (t & 1) ? sum[0] : sum[1];
                one[b] = ((t & 1) ? sum[1] : sum[0]) + __shfl_xor_sync(0xffffffffu, give, 1);
            }
            float all = one[0];
            if constexpr (PB == 2) {
                all = (t & 2) ? one[1] : one[0];
                if (!T::kShared) all += __shfl_xor_sync(0xffffffffu, (t & 2) ? one[0] : one[1], 2);
            } else if (!T::kShared) {
                all += __shfl_xor_sync(0xffffffffu, one[0], 2);
            }
            const int pos = pos0 + tu + 2 * (t & 1) + (PB == 2 ? 8 * (t & 2) : 0);
            if ((PB == 2 || t < 2) && (!EDGE || pos < plan.L))
                score_row[pos] = pos >= p.sink && pos < plan.L - p.recent ? all * kLn2 : -INFINITY;
        }
        // y = score in powers of two above the running maximum, plus kLift
        float y[PB][NT][4];
        float top = -INFINITY;
#pragma unroll
        for (int b = 0; b < PB; ++b)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    y[b][nt][c] = fmaf(s[b][nt][c], mul[nt][c & 1], base[nt][c & 1]);
                    if (EDGE && ((hide >> (4 * nt + c)) & 1u)) y[b][nt][c] = -INFINITY;
                    top = fmaxf(top, y[b][nt][c]);
                }
        if (__any_sync(0xffffffffu, top > kLift + kLazy)) {  // the maximum has fallen far behind: move it
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float x = -INFINITY;
#pragma unroll
                    for (int b = 0; b < PB; ++b)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            if (!EDGE || !((hide >> (4 * nt + c + 2 * k)) & 1u))
                                x = fmaxf(x, s[b][nt][c + 2 * k] * mul[nt][c]);
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                    const float was = kLift - base[nt][c], now = fmaxf(was, x);
                    const float a = was == now ? 1.f : fast_exp2(was - now);
                    base[nt][c] = kLift - now;
                    l[nt][c] *= a;
#pragma unroll
                    for (int j = 0; j < kKs; ++j) {
                        o[nt][j][c] *= a;
                        o[nt][j][c + 2] *= a;
                    }
#pragma unroll
                    for (int b = 0; b < PB; ++b)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float &z = y[b][nt][c + 2 * k];
                            z = fmaf(s[b][nt][c + 2 * k], mul[nt][c], base[nt][c]);
                            if (EDGE && ((hide >> (4 * nt + c + 2 * k)) & 1u)) z = -INFINITY;
                        }
                }
        }
        // ---- P^T as two fp16 terms ----
        uint32_t ph[PB][NT][2];
        [[maybe_unused]] uint32_t pl[PB][NT][2];
#pragma unroll
        for (int b = 0; b < PB; ++b)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float x[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) x[c] = fast_exp2(y[b][nt][c]);
                l[nt][0] += x[0] + x[2];
                l[nt][1] += x[1] + x[3];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t h = pack_f16x2(x[2 * k], x[2 * k + 1]);
                    const float2 hf = __half22float2(*reinterpret_cast<const __half2 *>(&h));
                    if constexpr (T::kShared) {
                        ph[b][nt][k] = transpose_8x8(pack_f16x2(fmaf(hf.x, second, x[2 * k]), fmaf(hf.y, second, x[2 * k + 1])));
                    } else {
                        ph[b][nt][k] = transpose_8x8(h);
                        pl[b][nt][k] = transpose_8x8(pack_f16x2(x[2 * k] - hf.x, x[2 * k + 1] - hf.y));
                    }
                }
            }
        // ---- O^T += V^T P^T: rows g, g + 8 -> dims 16 j + g, 16 j + g + 8; k -> tokens 4t .. 4t + 3 ----
        uint32_t keep = 0, part = 0;  // scale bytes of tokens seen by some row; by some but not all
        if (EDGE) {
            int lo_a, hi_a, lo_z, hi_z;
            span(comp, 0, lo_a, hi_a);
            span(comp, p.tokens - 1, lo_z, hi_z);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int pos = pos0 + 4 * t + i;
                if (pos >= lo_a && pos < hi_z) {
                    keep |= 0xffu << (8 * i);
                    if (multi && !(pos >= lo_z && pos < hi_a)) part |= 0xffu << (8 * i);
                }
            }
        }
#pragma unroll
        for (int q = 0; q < F::kQuads; ++q) {
            uint32_t cv[PB][4], sv[4], sh[PB][4][2];
#pragma unroll
            for (int b = 0; b < PB; ++b) {
                const uint8_t *blk = b ? blk1 : blk0;
                const uint4 cw = *reinterpret_cast<const uint4 *>(blk + F::kVCode + q * 512 + (g >> 1) * 128 + t * 32 +
                                                                  (g & 1) * 16);
                cv[b][0] = cw.x; cv[b][1] = cw.y; cv[b][2] = cw.z; cv[b][3] = cw.w;
                if constexpr (EDGE) {
                    const uint4 sw = *reinterpret_cast<const uint4 *>(blk + F::kVScale + t * F::kVScaleT + q * 16);
                    sv[0] = sw.x; sv[1] = sw.y; sv[2] = sw.z; sv[3] = sw.w;
                } else {
                    const uint4 *sw = reinterpret_cast<const uint4 *>(blk + t * (D / 2) + q * 32);
                    const uint4 x = sw[0], y4 = sw[1];
                    sh[b][0][0] = x.x; sh[b][0][1] = x.y; sh[b][1][0] = x.z; sh[b][1][1] = x.w;
                    sh[b][2][0] = y4.x; sh[b][2][1] = y4.y; sh[b][3][0] = y4.z; sh[b][3][1] = y4.w;
                }
            }
#pragma unroll
            for (int jr = 0; jr < 4; ++jr) {
                const int j = q * 4 + jr;
                if (EDGE) {
                    sv[jr] &= keep;
                    if (multi) {
                        // A NaN of a token that only some rows see must not reach the others through
                        // 0 * NaN: it is taken out here and given to the rows that see it.
                        uint32_t nan = 0;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if ((part >> (8 * i) & 1u) && ((sv[jr] >> (8 * i)) & 0x7fu) == 0x7fu) {
                                nan |= 1u << (4 * t + i);
                                sv[jr] &= ~(0xffu << (8 * i));
                            }
                        if (__any_sync(0xffffffffu, nan != 0)) {
                            nan |= __shfl_xor_sync(0xffffffffu, nan, 1);
                            nan |= __shfl_xor_sync(0xffffffffu, nan, 2);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int c = 0; c < 2; ++c) {
                                    int lo, hi;
                                    span(comp, token_of(row_of(nt, c)), lo, hi);
                                    uint32_t mine = 0;
                                    for (int i = 0; i < 16; ++i)
                                        if (pos0 + i >= lo && pos0 + i < hi) mine |= 1u << i;
                                    if (nan & mine) o[nt][j][c] = o[nt][j][c + 2] = NAN;
                                }
                        }
                    }
                }
                // the blocks' own sum first, then one rounded addition: the matrix instruction
                // truncates, which over a long run would bias O
                float sum[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) sum[nt][c] = 0.f;
#pragma unroll
                for (int b = 0; b < PB; ++b) {
                    uint32_t x[4];
                    e2m1x8_to_f16(cv[b][jr], x);
                    uint32_t s01, s23;
                    if constexpr (EDGE) {
                        s01 = e4m3x2_to_f16((uint16_t)sv[jr]);
                        s23 = e4m3x2_to_f16((uint16_t)(sv[jr] >> 16));
                    } else {
                        s01 = sh[b][jr][0];
                        s23 = sh[b][jr][1];
                    }
                    const uint32_t a[4] = {hmul2(x[0], s01), hmul2(x[1], s01), hmul2(x[2], s23), hmul2(x[3], s23)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if constexpr (!T::kShared) mma_f16_16816(sum[nt], a, pl[b][nt][0], pl[b][nt][1]);
                        mma_f16_16816(sum[nt], a, ph[b][nt][0], ph[b][nt][1]);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[nt][j][c] += sum[nt][c];
            }
        }
    };

    // the end of this warp's run of a unit: its output when the run is the whole unit, else a partial
    auto leave_unit = [&](int run0, int run1) {
        const bool whole = !CLUSTER && run0 == unit0 && run1 == unit0 + plan.n;
        const bool bad = drop || ((bad_units >> (unit_here & 31)) & 1u);
        const bool last = !CLUSTER && run1 == run;
        const int part = CLUSTER ? warp : warp * 2 + (last ? 1 : 0);
        if constexpr (CLUSTER) {
            if (bad && lane < ROWS) s_ml[part][lane][0] = NAN;
        } else if (lane == 0 && !whole) {
            s_unit[part] = at.b * p.hkv + at.h;
            s_unit0[part] = runs_of<kWarps>(p, s_prefix).start((int64_t)blockIdx.x * kWarps + warp) + unit0;
            s_bad[part] = bad;
        }
        if (bad) return;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], 4);
                l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], 8);
                l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], 16);
                if (T::kShared) {  // O of P's second term, two lanes on
#pragma unroll
                    for (int j = 0; j < kKs; ++j) {
                        o[nt][j][c] += __shfl_xor_sync(0xffffffffu, o[nt][j][c], 2);
                        o[nt][j][c + 2] += __shfl_xor_sync(0xffffffffu, o[nt][j][c + 2], 2);
                    }
                }
            }
        const int r = request_id(p, at.b);
        float *dst = reinterpret_cast<float *>(last ? ring : smem + T::kFirst + warp * T::kPart);
        if (!whole && last) {  // the ring is done with once every copy has landed
            cp_async_wait<0>();
            __syncwarp();
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int row = row_of(nt, c);
                if (row >= p.rows || (T::kShared && t >= 2)) continue;
                if (whole) {
                    const int64_t to = ((int64_t)r * p.tokens + row / p.group) * p.hq + at.h * p.group + row % p.group;
                    const float w = l[nt][c] == 0.f ? 0.f : p.v_scale / l[nt][c];
#pragma unroll
                    for (int j = 0; j < kKs; ++j) {
                        p.out[to * D + 16 * j + g] = o[nt][j][c] * w;
                        p.out[to * D + 16 * j + g + 8] = o[nt][j][c + 2] * w;
                    }
                    if (p.lse && g == 0)
                        p.lse[to] = l[nt][c] == 0.f ? -INFINITY : (log2f(l[nt][c]) - base[nt][c]) * kLn2;
                } else {
#pragma unroll
                    for (int j = 0; j < kKs; ++j) {
                        dst[row * D + 16 * j + g] = o[nt][j][c];
                        dst[row * D + 16 * j + g + 8] = o[nt][j][c + 2];
                    }
                    if (g == 0) {
                        s_ml[part][row][0] = kLift - base[nt][c];
                        s_ml[part][row][1] = l[nt][c];
                    }
                }
            }
    };

    int run0 = 0;
    if (run > 0) enter_unit(raw_query);
    while (f < run) {
        // two blocks at once where every row sees both whole
        int pairs = 0;
        if (!drop) {
            int inside = at.pg >= in_from ? in_to - at.pg : 0;
            if (MODE == kKv4Fast) inside = max(inside, in_comp - at.pg);
            pairs = min(inside, run - f) / 2;
        }
        if (pairs > 0) {
            for (int i = 0; i < pairs; ++i) {
                const int slot1 = slot + 1 == T::kDepth ? 0 : slot + 1;
                cp_async_wait<T::kDepth - 2>();
                __syncwarp();
                consume(std::integral_constant<int, 2>{}, std::false_type{}, ring + slot * F::kBlock,
                        ring + slot1 * F::kBlock);
                __syncwarp();  // every lane is done with the blocks that the next copies replace
                issue(slot);
                issue(slot1);
                slot = slot1 + 1 == T::kDepth ? 0 : slot1 + 1;
                at.pg += 2;
            }
            f += 2 * pairs;
        } else {
            cp_async_wait<T::kDepth - 1>();
            __syncwarp();
            if (!drop) consume(std::integral_constant<int, 1>{}, std::true_type{}, ring + slot * F::kBlock, ring);
            __syncwarp();
            issue(slot);
            slot = slot + 1 == T::kDepth ? 0 : slot + 1;
            ++f;
            ++at.pg;
        }
        if ((!CLUSTER && at.pg == plan.n) || f == run) {
            leave_unit(run0, f);
            run0 = f;
            if (f < run) {
                at.pg = 0;
                if (++at.h == p.hkv) {
                    at.h = 0;
                    do ++at.b; while (s_prefix[at.b + 1] == s_prefix[at.b]);
                }
                ++unit_here;
                load_query(at, raw_query);
                enter_unit(raw_query);
            }
        }
    }
    cp_async_wait<0>();
    if constexpr (CLUSTER) {
        // ---- the CTA's eight partials are added up, `ways` lanes to four dims of a row; the sums go to
        // the CTA of the cluster that writes these dims (`share` items of the unit each) ----
        const int ctas = cluster_nctarank(), rank = cluster_ctarank();
        const int items = p.rows * (D / 4), share = (items + ctas - 1) / ctas;
        float4 *got_x = reinterpret_cast<float4 *>(smem + T::kSmem);  // [CTA][share]
        float2 *got_ml = reinterpret_cast<float2 *>(got_x + ctas * share);
        int ways = 1;
        while (ways < kWarps && 2 * ways * items <= kThreads) ways *= 2;
        const int wide = 32 / ways, way = lane / wide;
        const int64_t row0 = (int64_t)request_id(p, at.b) * p.tokens;
        auto write = [&](int e, const Gathered &got) {
            const int row = e / (D / 4), d = e % (D / 4) * 4;
            const int64_t to = (row0 + (row >> gshift)) * p.hq + at.h * p.group + (row & (p.group - 1));
            write_row(p, to * D + d, got, d == 0 ? to : -1);
        };
        if (run == 0 && lane < ROWS) {
            s_ml[warp][lane][0] = -INFINITY;
            s_ml[warp][lane][1] = 0.f;
        }
        __syncthreads();
        if (ctas > 1) cluster_wait();  // the others have begun: their shared memory is there
        for (int e0 = warp * wide; e0 < items; e0 += kWarps * wide) {
            const int e = min(e0 + lane % wide, items - 1);
            const int row = e / (D / 4), d = e % (D / 4) * 4;
            Gathered got;
            bool bad = false;
#pragma unroll 1
            for (int c = way; c < kWarps; c += ways * 4) {
                float2 ml[4];
                float4 x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = c + i * ways;
                    ml[i] = make_float2(-INFINITY, 0.f);
                    x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (k < kWarps) {
                        ml[i] = make_float2(s_ml[k][row][0], s_ml[k][row][1]);
                        if (ml[i].x > -INFINITY)  // (a warp without blocks has written no sums)
                            x[i] = *reinterpret_cast<const float4 *>(smem + T::kFirst + k * T::kPart + (row * D + d) * 4);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) bad |= isnan(ml[i].x);
                got.add(ml, x);
            }
            // the lanes' sums, brought to one maximum first
            float top = got.mx;
            for (int off = wide; off < 32; off *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float w = got.mx == top ? 1.f : fast_exp2(got.mx - top);
            got.mx = top;
            got.sum *= w;
            got.acc.x *= w;
            got.acc.y *= w;
            got.acc.z *= w;
            got.acc.w *= w;
            for (int off = wide; off < 32; off *= 2) {
                got.sum += __shfl_xor_sync(0xffffffffu, got.sum, off);
                got.acc.x += __shfl_xor_sync(0xffffffffu, got.acc.x, off);
                got.acc.y += __shfl_xor_sync(0xffffffffu, got.acc.y, off);
                got.acc.z += __shfl_xor_sync(0xffffffffu, got.acc.z, off);
                got.acc.w += __shfl_xor_sync(0xffffffffu, got.acc.w, off);
            }
            bad = __any_sync(0xffffffffu, bad);  // any part of the unit: nothing of it is written
            if (way == 0 && e0 + lane < items) {
                if (ctas > 1) {
                    const int owner = e / share, to = rank * share + e - owner * share;
                    st_cluster_f32x4(cluster_map(smem_u32(got_x + to), owner), got.acc);
                    st_cluster_f32x2(cluster_map(smem_u32(got_ml + to), owner), bad ? NAN : got.mx, got.sum);
                } else if (!bad) {
                    write(e, got);
                }
            }
        }
        if (ctas == 1) return;
        __syncwarp();
        cluster_sync();
        // ---- this CTA's share of the unit: a part from each CTA ----
        const int e = rank * share + tid;
        if (tid < share && e < items) {
            float2 ml[kKv4MaxCluster];
            float4 x[kKv4MaxCluster];
            bool bad = false;
#pragma unroll
            for (int k = 0; k < kKv4MaxCluster; ++k) {
                ml[k] = make_float2(-INFINITY, 0.f);
                x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k < ctas) {
                    ml[k] = got_ml[k * share + tid];
                    x[k] = got_x[k * share + tid];
                }
                bad |= isnan(ml[k].x);
            }
            Gathered got;
            got.add(ml, x);
            if (!bad) write(e, got);
        }
        return;
    }
    __syncthreads();

    // ---- the CTA's partials, unit by unit: the unit's output where the CTA holds all of it, else
    // the CTA's part of it (s_open: units begun before this CTA, or going on after it) ----
    const Runs runs = runs_of<kWarps>(p, s_prefix);
    const int64_t cta0 = runs.start((int64_t)blockIdx.x * kWarps), cta1 = runs.start((int64_t)(blockIdx.x + 1) * kWarps);
    const int my_unit = lane < kParts ? s_unit[lane] : -1;
    const uint32_t mine = __match_any_sync(0xffffffffu, my_unit);
    const uint32_t bads = __ballot_sync(0xffffffffu, lane < kParts && my_unit >= 0 && s_bad[min(lane, kParts - 1)]);
    // the units in order of their first part; all items of all of them are spread over the threads
    const bool leads = my_unit >= 0 && __ffs(mine) - 1 == lane;
    const uint32_t leaders = __ballot_sync(0xffffffffu, leads);
    if (leads) s_lead[__popc(leaders & ((1u << lane) - 1u))] = lane;  // the same from every warp
    __syncwarp();
    const int items = p.rows * (D / 4), all_items = __popc(leaders) * items;
    for (int e0 = warp * 32; e0 < all_items; e0 += kThreads) {
        const int i = min(e0 + lane, all_items - 1), e = i % items;
        const int first = s_lead[i / items];
        const int u = __shfl_sync(0xffffffffu, my_unit, first);
        const uint32_t parts = __shfl_sync(0xffffffffu, mine, first);
        const bool bad = bads & parts;
        const int b = u / p.hkv, h = u - b * p.hkv;
        const int r = request_id(p, b);
        const int64_t u0 = s_unit0[first], u1 = u0 + (s_prefix[b + 1] - s_prefix[b]);
        const bool complete = u0 >= cta0 && u1 <= cta1;
        const int side = u0 < cta0 ? 0 : 1;  // this CTA's slot for it in the workspace
        const int64_t ws_row = ((int64_t)blockIdx.x * 2 + side) * kMaxRows;
        if (!complete && e == 0) {
            s_open[side] = u;
            s_open0[side] = u0;
        }
        if (e0 + lane < all_items && !(complete && bad)) {
            const int row = e / (D / 4), d = e % (D / 4) * 4;
            Gathered got;
            // four parts at a time, rolled: most of this code's time is its own fetching
#pragma unroll 1
            for (uint32_t left = parts; left;) {
                float2 ml[4];
                float4 x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = __ffs(left) - 1;
                    ml[i] = make_float2(-INFINITY, 0.f);
                    x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (k >= 0) {
                        ml[i] = make_float2(s_ml[k][row][0], s_ml[k][row][1]);
                        x[i] = *reinterpret_cast<const float4 *>(
                            smem + ((k & 1) ? (k >> 1) * T::kRing : T::kFirst + (k >> 1) * T::kPart) + (row * D + d) * 4);
                    }
                    left &= left - 1;  // 0 stays 0
                }
                got.add(ml, x);
            }
            if (complete) {
                const int64_t to = ((int64_t)r * p.tokens + row / p.group) * p.hq + h * p.group + row % p.group;
                write_row(p, to * D + d, got, d == 0 ? to : -1);
            } else {
                __stcg(reinterpret_cast<float4 *>(p.ws_part + (ws_row + row) * D + d), got.acc);
                // a maximum of NaN: the part met a bad page id (its sums are not read)
                if (d == 0) __stcg(reinterpret_cast<float2 *>(p.ws_ml) + ws_row + row, make_float2(bad ? NAN : got.mx, got.sum));
            }
        }
    }

    // ---- units shared with other CTAs: the last of them to come here adds the parts up ----
    __syncthreads();
    if (tid < 2) {
        const int u = s_open[tid];
        int last = 0;
        if (u >= 0) {
            const int64_t u0 = s_open0[tid], u1 = u0 + (s_prefix[u / p.hkv + 1] - s_prefix[u / p.hkv]);
            // a unit that others share begins in one CTA, whose last unit it is: its counter counts
            // them (an index that does not depend on the shape, as the workspace's parts do not)
            const int c0 = (int)(runs.owner(u0) / kWarps), others = (int)(runs.owner(u1 - 1) / kWarps) - c0;
            // releases the CTA's part (ordered before it by the barrier) and acquires the others'
            int old;
            asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(old) : "l"(p.ws_count + c0) : "memory");
            last = old == others;
            if (last) p.ws_count[c0] = 0;
        }
        s_last[tid] = last;
    }
    __syncthreads();
    if (!s_last[0] && !s_last[1]) return;
    {
        // where the CTA is the last for both of its units, half of the threads take each
        const bool both = s_last[0] && s_last[1];
        const int threads = both ? kThreads / 2 : kThreads;
        const int side = both ? tid / threads : (s_last[0] ? 0 : 1), me = tid % threads;
        const int u = s_open[side];
        const int b = u / p.hkv, h = u - b * p.hkv;
        const int r = request_id(p, b);
        const int64_t u0 = s_open0[side], u1 = u0 + (s_prefix[b + 1] - s_prefix[b]);
        const int c0 = (int)(runs.owner(u0) / kWarps), c1 = (int)(runs.owner(u1 - 1) / kWarps);
        const int parts = c1 - c0 + 1;
        // slot of part c: a unit lies in the second slot of the CTA it begins in, else in the first
        auto row_at = [&](int c, int row) { return ((int64_t)(c0 + c) * 2 + (c == 0)) * kMaxRows + row; };
        // a thread takes four dims of a row, eight parts at a time; where there are more parts and
        // threads to spare, `ways` threads share an item, each with every ways-th part (as many as
        // half of the CTA has to spare, in both cases: the order of the sums may not depend on
        // which CTA came last)
        constexpr int kBatch = 8;
        const int ways = max(1, min(kThreads / 2 / items, (parts + kBatch - 1) / kBatch)), wide = min(items, threads);
        float2 *red_ml = reinterpret_cast<float2 *>(smem);
        float4 *red = reinterpret_cast<float4 *>(smem + kThreads * 8);
        for (int e0 = 0; e0 < items; e0 += threads) {
            const int e = e0 + me % wide, way = me / wide;
            const int row = e / (D / 4), d = e % (D / 4) * 4;
            const bool busy = e < items && way < ways;
            Gathered got;
            bool bad = false;
#pragma unroll 1
            for (int c = way; c < parts && busy; c += ways * kBatch) {
                float2 ml[kBatch];
                float4 x[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int k = c + i * ways;
                    ml[i] = make_float2(-INFINITY, 0.f);
                    x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (k < parts) {
                        ml[i] = __ldcg(reinterpret_cast<const float2 *>(p.ws_ml) + row_at(k, row));
                        x[i] = __ldcg(reinterpret_cast<const float4 *>(p.ws_part + row_at(k, row) * D + d));
                    }
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) bad |= isnan(ml[i].x);
                got.add(ml, x);
            }
            if (__syncthreads_or(ways > 1)) {  // (either half may need it)
                red_ml[tid] = make_float2(bad ? NAN : got.mx, got.sum);
                red[tid] = got.acc;
                __syncthreads();
                if (way == 0 && busy)
                    for (int k = 1; k < ways; ++k) {
                        const float2 ml[1] = {red_ml[tid + k * wide]};
                        const float4 x[1] = {red[tid + k * wide]};
                        bad |= isnan(ml[0].x);
                        got.add(ml, x);
                    }
            }
            if (busy && way == 0 && !bad) {
                const int64_t to = ((int64_t)r * p.tokens + row / p.group) * p.hq + h * p.group + row % p.group;
                write_row(p, to * D + d, got, d == 0 ? to : -1);
            }
        }
    }
}

namespace {

template <int D, int ROWS, bool CLUSTER>
constexpr int smem_of = CLUSTER ? Tile<D, ROWS>::kClusterSmem : Tile<D, ROWS>::kSmem;

// The shared-memory opt-in is a per-device function attribute: set it once per device.
template <int D, int ROWS, int MODE, bool CLUSTER>
cudaError_t configure(int dev) {
    static std::atomic<uint64_t> configured{0};
    const uint64_t bit = (dev >= 0 && dev < 64) ? (uint64_t(1) << dev) : 0;
    if (bit && (configured.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kv4_attn_kernel<D, ROWS, MODE, CLUSTER>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem_of<D, ROWS, CLUSTER>);
    if (e == cudaSuccess) configured.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

// cluster: CTAs per unit, or 0 for runs of the row of work.
template <int D, int ROWS, int MODE, bool CLUSTER>
cudaError_t launch_one(const Kv4AttnParams &p, int ctas, int cluster, cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = configure<D, ROWS, MODE, CLUSTER>(dev);
    if (e != cudaSuccess) return e;
    return launch_dependent_clusters(kv4_attn_kernel<D, ROWS, MODE, CLUSTER>, ctas, cluster, Tile<D, ROWS>::kThreads,
                                     smem_of<D, ROWS, CLUSTER>, stream, p);
}

// How many clusters of `size` CTAs the device holds at once (0: not known).
template <int D, int ROWS, int MODE>
int resident_clusters(int size) {
    static std::atomic<int> cache[64][kKv4MaxCluster + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    const int known = cache[dev][size].load(std::memory_order_relaxed);
    if (known > 0) return known;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)size);
    cfg.blockDim = dim3(Tile<D, ROWS>::kThreads);
    cfg.dynamicSmemBytes = smem_of<D, ROWS, true>;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)size;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (configure<D, ROWS, MODE, true>(dev) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kv4_attn_kernel<D, ROWS, MODE, true>, &cfg) != cudaSuccess) {
        cudaGetLastError();  // leave no error behind for the next launch's check
        return 0;
    }
    if (n > 0) cache[dev][size].store(n, std::memory_order_relaxed);
    return n;
}

// The CTAs that each unit gets as a cluster of its own, or 0 for the row of work.
// Clusters need no prefix over the requests and meet through shared memory, so they begin and end
// about 6 us sooner: 16 requests of 64 + 704 + 256 rows, 16/8/128 heads, take 10.1 us and 15.9 with
// the row of work, one request 6.8 and 11.4, four tokens of 32/8/128 heads 16.4 and 29.3. So it is
// clusters of as many CTAs as are all resident at once, where that is possible (64 of these requests
// would take several waves: 26.4 us in the row), except for units so long that the CTAs left idle
// cost more: a warp gets blocks / (8 size) of them instead of blocks units / (8 slots). With 160
// units of 304 slots, 110 blocks of D = 128 each take about as long either way, 88 take 15.5 us and
// 18.0 in the row, 183 take 25.5 and 22.8; with 240 units 128 blocks take 19.9 and 23.2, 270 blocks
// 34.9 and 32.5. At D = 64 a block takes half as long (160 units, 128 blocks: 14.1 and 16.3, 270:
// 24.1 and 20.5), and sixteen rows gain more (88 units of 152 slots, 128 blocks: 21.1 and 29.8, 270:
// 36.8 and 35.4; D = 64: 14.2 and 19.4, 24.4 and 23.1).
// The lengths are known on the device alone: the compact pool's size stands for them, so a batch of
// very unequal selections may get clusters where the row would be better (one of 8000 rows among
// fifteen of 300: 32 us and 17; 32 to 8192 rows over eight requests: 20.9 and 17.5). Both in one
// kernel, chosen by the real lengths, cost every fast step 0.5 us and the row 3 us more.
//
// Dense attention: lengths differ more, and the page table's width bounds them. Clusters take what they
// take in sixteen blocks a warp at most: 1000 tokens of one request, 8/2/64 heads with scores, take
// 5.8 us and 9.7 in the row; 16 requests of 4000 tokens, 16/8/128 heads with scores 22.7 and 29.3
// (lengths of 60 to 4000: 20.1 and 17.4); 4 tokens of 4 requests of 4000, 32/8/128 heads 14.4 and 26.7.
template <int D, int ROWS, int MODE>
int cluster_of(const Kv4AttnParams &p, int64_t slots) {
    const int64_t units = (int64_t)p.batch * p.hkv;
    int64_t size = std::min<int64_t>(kKv4MaxCluster, slots / units);
    while (size > 0 && resident_clusters<D, ROWS, MODE>((int)size) < units) --size;
    if (MODE != kKv4Fast) return p.max_pages <= 16 * Tile<D, ROWS>::kWarps * size ? (int)size : 0;
    const int64_t blocks = p.c_total_pages / units + p.recent / 16 + 1;
    constexpr int64_t kEven = ROWS > 8 || D == 64 ? 96 : 48;  // the blocks that a CTA may have more than in the row
    return blocks * (slots - units * size) > kEven * size * slots ? 0 : (int)size;
}

template <int D, int ROWS, int MODE>
cudaError_t launch_choice(const Kv4AttnParams &p, int ctas, cudaStream_t stream) {
    const int size = cluster_of<D, ROWS, MODE>(p, ctas);
    if (size > 0) return launch_one<D, ROWS, MODE, true>(p, p.batch * p.hkv * size, size, stream);
    return launch_one<D, ROWS, MODE, false>(p, ctas, 0, stream);
}

template <int D, int ROWS>
cudaError_t launch_mode(const Kv4AttnParams &p, int ctas, cudaStream_t stream) {
    if (p.c_pool) return launch_choice<D, ROWS, kKv4Fast>(p, ctas, stream);
    return p.scores ? launch_choice<D, ROWS, kKv4Scores>(p, ctas, stream)
                    : launch_choice<D, ROWS, kKv4Dense>(p, ctas, stream);
}

template <int D>
cudaError_t launch_rows(const Kv4AttnParams &p, int sms, cudaStream_t stream) {
    // one wave: two CTAs per SM for up to eight rows, one for up to sixteen (registers)
    const int two = std::min(sms * kKv4CtasPerSm, kKv4MaxCtas), one = std::min(sms, kKv4MaxCtas);
    if (p.rows <= 4) return launch_mode<D, 4>(p, two, stream);
    return p.rows <= 8 ? launch_mode<D, 8>(p, two, stream) : launch_mode<D, 16>(p, one, stream);
}

}  // namespace

cudaError_t launch_kv4_attn(const Kv4AttnParams &p, int head_dim, cudaStream_t stream) {
    const int sms = sm_count_current_device();
    if (sms <= 0) return cudaErrorInvalidDevice;
    return head_dim == 128 ? launch_rows<128>(p, sms, stream) : launch_rows<64>(p, sms, stream);
}

}  // namespace sfi
