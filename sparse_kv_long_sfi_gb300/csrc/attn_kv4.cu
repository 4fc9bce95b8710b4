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
// Per block (16 tokens): S^T = K Q^T and O^T += V^T P^T with mma.m16n8k16, the tokens (or
// dims) as the M side, so that eight query rows take one N tile. Codes become fp16 by
// conversion and one multiplication by their scale: a product of an e2m1 and an e4m3
// value is exact in fp16. Q in fp16 is exact, too: each row is scaled by a power of two to
// just below 2^15. P goes in as two fp16 terms (22 bits; times 2^7 to keep small
// probabilities off the subnormals), so the output is as good as fp32's. The running
// maximum moves only when a score passes it by 2^8.
#include <algorithm>
#include <type_traits>

#include "kv4_format.cuh"

namespace sfi {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.f;   // the maximum may lag by this (in powers of two)
constexpr float kLift = 7.f;   // P is computed times 2^7
constexpr int kMinPages = 2;   // blocks per warp at least, before fewer CTAs work

enum Kv4Mode : int { kKv4Dense = 0, kKv4Scores = 1, kKv4Fast = 2 };

template <int D, int NT>
struct Tile {
    static constexpr int kDepth = NT == 1 ? 4 : 6;  // blocks in flight per warp
    static constexpr int kRing = kDepth * Kv4<D>::kBlock;
    static constexpr int kRowsPad = 8 * NT;
    static constexpr int kPart = kRowsPad * D * 4;  // a partial O
    static constexpr int kFirst = kWarps * kRing;
    static constexpr int kSmem = kFirst + kWarps * kPart;
    static_assert(kRing >= kPart, "a warp's ring holds its last partial");
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

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
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
    if (q.L < p.tokens || q.L > p.max_pages * kSubTokens || (MODE == kKv4Scores && q.L > p.score_stride)) {
        *err |= SFI_DEV_BAD_LEN;
        return q;
    }
    if (MODE != kKv4Fast) {
        q.n = (q.L + 15) / 16;
        return q;
    }
    const int cnt = p.c_count[r], cap = p.c_capacity[r];
    const int64_t off = p.c_page_offset[r];
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
    at.h = (int)(in / n);
    at.pg = (int)(in - at.h * n);
    return at;
}

// Page ids of a unit, 32 at a time (lane i: number base + i).
struct PageIds {
    int ids, base;
};

}  // namespace

template <int D, int NT, int MODE>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) kv4_attn_kernel(const Kv4AttnParams p) {
    using F = Kv4<D>;
    using T = Tile<D, NT>;
    constexpr int kKs = D / 16;  // k steps of S, and m tiles of O
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_prefix[kKv4MaxBatch + 1];
    __shared__ uint32_t s_bad[kKv4MaxBatch / 32];
    __shared__ int64_t s_carry[kWarps];
    __shared__ int64_t s_unit0[2 * kWarps];            // first block of a partial's unit
    __shared__ int s_unit[2 * kWarps];                 // its unit, or -1
    __shared__ float s_ml[2 * kWarps][T::kRowsPad][2];
    __shared__ int s_last;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;

    // ---- the row of work: blocks of each request, summed up ----
    uint32_t err = 0;
    {
        int64_t carry = 0;
        for (int base = 0; base < p.batch; base += kThreads) {
            const int b = base + tid;
            int64_t v = b < p.batch ? plan_request<MODE>(p, b, &err).n : 0;
            int64_t incl = v;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int64_t o = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += o;
            }
            if (lane == 31) s_carry[warp] = incl;
            __syncthreads();
            int64_t before = carry, all = carry;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) before += s_carry[w];
                all += s_carry[w];
            }
            if (b < p.batch) s_prefix[b] = before + incl - v;
            carry = all;
            __syncthreads();
        }
        if (tid == 0) s_prefix[p.batch] = carry;
        if (tid < kKv4MaxBatch / 32) s_bad[tid] = 0;
        if (tid < 2 * kWarps) s_unit[tid] = -1;
        if (err && blockIdx.x == 0) report(p.dev_status, err);
    }
    __syncthreads();
    const int64_t total = s_prefix[p.batch] * p.hkv;
    const int64_t ctas = min((int64_t)gridDim.x, (total + kWarps * kMinPages - 1) / (kWarps * kMinPages));
    if ((int64_t)blockIdx.x >= ctas) return;
    const int64_t warps = ctas * kWarps;
    const int64_t f0 = ((int64_t)blockIdx.x * kWarps + warp) * total / warps;
    const int64_t f1 = ((int64_t)blockIdx.x * kWarps + warp + 1) * total / warps;
    const int64_t cta0 = (int64_t)blockIdx.x * kWarps * total / warps;
    const int64_t cta1 = ((int64_t)blockIdx.x + 1) * kWarps * total / warps;

    // ---- copies: this warp's blocks, kDepth of them in flight ----
    uint8_t *ring = smem + warp * T::kRing;
    Place ahead{};
    ReqPlan aplan{};
    PageIds ids{0, 0};
    int64_t fa = f0;  // next block to copy
    auto load_ids = [&](int first) {  // page ids [first, first + 32) of the unit's pages
        ids.base = first;
        const int r = request_id(p, ahead.b);
        const int i = first + lane;
        ids.ids = i < aplan.n - aplan.ncomp ? p.page_table[(int64_t)r * p.max_pages + aplan.page0 + i] : 0;
    };
    uint32_t none = 0;
    auto enter_ahead = [&]() {
        aplan = plan_request<MODE>(p, ahead.b, &none);
        load_ids(max(0, ahead.pg - aplan.ncomp));
    };
    auto issue = [&](int slot) {
        if (fa < f1) {
            const uint8_t *src;
            if (MODE == kKv4Fast && ahead.pg < aplan.ncomp) {
                src = p.c_pool + (aplan.cblock + (int64_t)ahead.h * aplan.cap + ahead.pg) * F::kBlock;
            } else {
                const int i = ahead.pg - aplan.ncomp;
                if (i >= ids.base + 32) load_ids(i);
                int page = __shfl_sync(0xffffffffu, ids.ids, i - ids.base);
                if (page < 0 || page >= p.num_pages) page = 0;  // the unit is dropped below
                src = p.pool + ((int64_t)page * p.hkv + ahead.h) * F::kBlock;
            }
            uint8_t *dst = ring + slot * F::kBlock;
#pragma unroll
            for (int c = lane; c < F::kBlock / 16; c += 32) cp_async16(dst + c * 16, src + c * 16);
            ++fa;
            if (++ahead.pg == aplan.n && fa < f1) {
                ahead.pg = 0;
                if (++ahead.h == p.hkv) {
                    ahead.h = 0;
                    do ++ahead.b; while (s_prefix[ahead.b + 1] == s_prefix[ahead.b]);
                }
                enter_ahead();
            }
        }
        cp_async_commit();
    };
    Place at{};
    if (f0 < f1) {
        at = locate(s_prefix, p.batch, p.hkv, f0);
        ahead = at;
        enter_ahead();
    }
#pragma unroll
    for (int i = 0; i < T::kDepth; ++i) issue(i);

    // ---- page ids of every request this CTA touches: one bad id drops the request ----
    {
        const int b0 = locate(s_prefix, p.batch, p.hkv, cta0).b, b1 = locate(s_prefix, p.batch, p.hkv, cta1 - 1).b;
        for (int b = b0; b <= b1; ++b) {
            const ReqPlan q = plan_request<MODE>(p, b, &none);
            const int r = request_id(p, b);
            const int32_t *row = p.page_table + (int64_t)r * p.max_pages + q.page0;
            bool bad = false;
#pragma unroll 8
            for (int i = tid; i < q.n - q.ncomp; i += kThreads) bad |= (uint32_t)__ldg(row + i) >= (uint32_t)p.num_pages;
            if (bad) atomicOr(&s_bad[b >> 5], 1u << (b & 31));
        }
    }
    __syncthreads();

    // ---- this warp's units ----
    uint32_t bq[NT][kKs][2];     // Q as B fragments
    float mul[NT][2];            // fp16 product -> score in powers of two
    float nat[NT][2];            // ... -> score (scores mode; 0 in rows that are not there)
    int rtok[NT][2];             // query token of this lane's rows
    float o[NT][kKs][4];
    float base[NT][2], l[NT][2];  // kLift - running maximum (+inf: nothing seen), sum of 2^(score + base)
    ReqPlan plan{};
    int64_t f = f0, unit0 = 0;
    int slot = 0;
    bool bad = false;
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

    auto enter_unit = [&]() {
        plan = plan_request<MODE>(p, at.b, &none);
        unit0 = f - at.pg;
        bad = (s_bad[at.b >> 5] >> (at.b & 31)) & 1u;
        const int r = request_id(p, at.b);
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
            const int row = nt * 8 + g;
            int4 raw[D / 32];
#pragma unroll
            for (int i = 0; i < D / 32; ++i) raw[i] = make_int4(0, 0, 0, 0);
            if (row < p.rows) {
                const int tok = row / p.group, head = at.h * p.group + row % p.group;
                const __nv_bfloat16 *src = p.q + (((int64_t)r * p.tokens + tok) * p.hq + head) * D + t * (D / 4);
#pragma unroll
                for (int i = 0; i < D / 32; ++i) raw[i] = *reinterpret_cast<const int4 *>(src + i * 8);
            }
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
            for (int i = 0; i < D / 32; ++i) {
                float x[8];
                bf16x8_to_f32(raw[i], x);
#pragma unroll
                for (int k = 0; k < 2; ++k) {  // k step 2 i + k: dims 4 k .. 4 k + 3 of these eight
                    bq[nt][2 * i + k][0] = pack_f16x2(x[4 * k] * up, x[4 * k + 1] * up);
                    bq[nt][2 * i + k][1] = pack_f16x2(x[4 * k + 2] * up, x[4 * k + 3] * up);
                }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {  // S^T's columns of this lane are rows 2t, 2t + 1
                const int col = nt * 8 + 2 * t + c;
                const float x = __shfl_sync(0xffffffffu, down, (2 * t + c) * 4) * p.k_mul;
                mul[nt][c] = x * kLog2e;
                nat[nt][c] = col < p.rows ? x : 0.f;
                rtok[nt][c] = min(col / p.group, p.tokens - 1);
                base[nt][c] = INFINITY;
                l[nt][c] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < kKs; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[nt][j][c] = 0.f;
        }
    };

    // S^T of one block: rows g -> tokens tu and (g + 8) tu + 2, columns 2t, 2t + 1
    const int tu = 4 * (g >> 1) + (g & 1);
    auto products = [&](const uint8_t *blk, float (&s)[NT][4]) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) s[nt][c] = 0.f;
        uint32_t ka[D / 32], kb[D / 32];  // codes of the two tokens, dims t D/4 ...
        uint32_t sa[D / 64], sb[D / 64];  // their scales, twice in a register
        if constexpr (D == 128) {
            const uint4 a = *reinterpret_cast<const uint4 *>(blk + tu * F::kKRow + t * 16);
            const uint4 b = *reinterpret_cast<const uint4 *>(blk + (tu + 2) * F::kKRow + t * 16);
            ka[0] = a.x; ka[1] = a.y; ka[2] = a.z; ka[3] = a.w;
            kb[0] = b.x; kb[1] = b.y; kb[2] = b.z; kb[3] = b.w;
            const uint32_t ha = e4m3x2_to_f16(*reinterpret_cast<const uint16_t *>(blk + F::kKScale + tu * 8 + t * 2));
            const uint32_t hb = e4m3x2_to_f16(*reinterpret_cast<const uint16_t *>(blk + F::kKScale + (tu + 2) * 8 + t * 2));
            sa[0] = __byte_perm(ha, 0, 0x1010); sa[1] = __byte_perm(ha, 0, 0x3232);
            sb[0] = __byte_perm(hb, 0, 0x1010); sb[1] = __byte_perm(hb, 0, 0x3232);
        } else {
            const uint2 a = *reinterpret_cast<const uint2 *>(blk + tu * F::kKRow + t * 8);
            const uint2 b = *reinterpret_cast<const uint2 *>(blk + (tu + 2) * F::kKRow + t * 8);
            ka[0] = a.x; ka[1] = a.y;
            kb[0] = b.x; kb[1] = b.y;
            sa[0] = __byte_perm(e4m3x2_to_f16(blk[F::kKScale + tu * 4 + t]), 0, 0x1010);
            sb[0] = __byte_perm(e4m3x2_to_f16(blk[F::kKScale + (tu + 2) * 4 + t]), 0, 0x1010);
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
            uint32_t xa[4], xb[4];
            e2m1x8_to_f16(ka[w], xa);
            e2m1x8_to_f16(kb[w], xb);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t a[4] = {hmul2(xa[2 * k], sa[w / 2]), hmul2(xb[2 * k], sb[w / 2]),
                                       hmul2(xa[2 * k + 1], sa[w / 2]), hmul2(xb[2 * k + 1], sb[w / 2])};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma_f16_16816(s[nt], a, bq[nt][2 * w + k][0], bq[nt][2 * w + k][1]);
            }
        }
    };

    // PB blocks from blk on (EDGE: one block, some of whose tokens some rows do not see).
    auto consume = [&](auto pb_tag, auto edge_tag, const uint8_t *blk0, const uint8_t *blk1) {
        constexpr int PB = decltype(pb_tag)::value;
        constexpr bool EDGE = decltype(edge_tag)::value;
        const bool comp = EDGE && MODE == kKv4Fast && at.pg < plan.ncomp;
        const int pos0 = 16 * (comp ? at.pg : plan.page0 + at.pg - plan.ncomp);
        float s[PB][NT][4];
#pragma unroll
        for (int b = 0; b < PB; ++b) products(b ? blk1 : blk0, s[b]);
        // ---- scores (natural units), masks, exponents ----
        uint32_t hide = 0;  // bits 4 nt + c: not seen
        if (EDGE) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    int lo, hi;
                    span(comp, rtok[nt][c & 1], lo, hi);
                    const int pos = pos0 + tu + (c & 2);
                    if (pos < lo || pos >= hi) hide |= 1u << (4 * nt + c);
                }
        }
        if (MODE == kKv4Scores) {
            // the rows' sum of each token; lane t of four ends up with token tu + 2 (t & 1) of block t / 2
            float sum[PB][2];
#pragma unroll
            for (int b = 0; b < PB; ++b)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float x = 0.f;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float y = s[b][nt][2 * k + c] * nat[nt][c];
                            x += EDGE && ((hide >> (4 * nt + 2 * k + c)) & 1u) ? 0.f : y;
                        }
                    sum[b][k] = x;
                }
            float one[PB];
#pragma unroll
            for (int b = 0; b < PB; ++b) {
                const float give = (t & 1) ? sum[b][0] : sum[b][1];
                one[b] = ((t & 1) ? sum[b][1] : sum[b][0]) + __shfl_xor_sync(0xffffffffu, give, 1);
            }
            float all;
            if constexpr (PB == 2) {
                const float give = (t & 2) ? one[0] : one[1];
                all = ((t & 2) ? one[1] : one[0]) + __shfl_xor_sync(0xffffffffu, give, 2);
            } else {
                all = one[0] + __shfl_xor_sync(0xffffffffu, one[0], 2);
            }
            const int pos = pos0 + tu + 2 * (t & 1) + (PB == 2 ? 8 * (t & 2) : 0);
            if ((PB == 2 || t < 2) && (!EDGE || pos < plan.L))
                score_row[pos] = pos >= p.sink && pos < plan.L - p.recent ? all : -INFINITY;
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
        uint32_t ph[PB][NT][2], pl[PB][NT][2];
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
                    ph[b][nt][k] = transpose_8x8(h);
                    pl[b][nt][k] = transpose_8x8(pack_f16x2(x[2 * k] - hf.x, x[2 * k + 1] - hf.y));
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
            uint32_t cv[PB][4], sv[PB][4];
#pragma unroll
            for (int b = 0; b < PB; ++b) {
                const uint8_t *blk = b ? blk1 : blk0;
                const uint4 cw = *reinterpret_cast<const uint4 *>(blk + F::kVCode + q * 512 + (g >> 1) * 128 + t * 32 +
                                                                  (g & 1) * 16);
                const uint4 sw = *reinterpret_cast<const uint4 *>(blk + F::kVScale + t * F::kVScaleT + q * 16);
                cv[b][0] = cw.x; cv[b][1] = cw.y; cv[b][2] = cw.z; cv[b][3] = cw.w;
                sv[b][0] = sw.x; sv[b][1] = sw.y; sv[b][2] = sw.z; sv[b][3] = sw.w;
            }
#pragma unroll
            for (int jr = 0; jr < 4; ++jr) {
                const int j = q * 4 + jr;
                if (EDGE) {
                    sv[0][jr] &= keep;
                    if (multi) {
                        // A NaN of a token that only some rows see must not reach the others through
                        // 0 * NaN: it is taken out here and given to the rows that see it.
                        uint32_t nan = 0;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if ((part >> (8 * i) & 1u) && ((sv[0][jr] >> (8 * i)) & 0x7fu) == 0x7fu) {
                                nan |= 1u << (4 * t + i);
                                sv[0][jr] &= ~(0xffu << (8 * i));
                            }
                        if (__any_sync(0xffffffffu, nan != 0)) {
                            nan |= __shfl_xor_sync(0xffffffffu, nan, 1);
                            nan |= __shfl_xor_sync(0xffffffffu, nan, 2);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int c = 0; c < 2; ++c) {
                                    int lo, hi;
                                    span(comp, rtok[nt][c], lo, hi);
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
                    const uint32_t s01 = e4m3x2_to_f16((uint16_t)sv[b][jr]),
                                   s23 = e4m3x2_to_f16((uint16_t)(sv[b][jr] >> 16));
                    const uint32_t a[4] = {hmul2(x[0], s01), hmul2(x[1], s01), hmul2(x[2], s23), hmul2(x[3], s23)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_f16_16816(sum[nt], a, pl[b][nt][0], pl[b][nt][1]);
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

    const int r_rows = p.rows;
    // the end of this warp's run of a unit: its output when the run is the whole unit, else a partial
    auto leave_unit = [&](int64_t run0, int64_t run1) {
        const bool whole = run0 == unit0 && run1 == unit0 + plan.n;
        if (bad) {
            if (lane == 0 && run0 == unit0) report(p.dev_status, SFI_DEV_BAD_PAGE);
            return;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], 4);
                l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], 8);
                l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], 16);
            }
        const int r = request_id(p, at.b);
        const bool last = run1 == f1;
        const int part = warp * 2 + (last ? 1 : 0);
        float *dst = last ? reinterpret_cast<float *>(ring)
                          : reinterpret_cast<float *>(smem + T::kFirst + warp * T::kPart);
        if (!whole && last) {  // the ring is done with once every copy has landed
            cp_async_wait<0>();
            __syncwarp();
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int row = nt * 8 + 2 * t + c;
                if (whole) {
                    if (row < r_rows) {
                        const int64_t to = ((int64_t)r * p.tokens + row / p.group) * p.hq + at.h * p.group + row % p.group;
                        const float w = l[nt][c] == 0.f ? 0.f : p.v_scale / l[nt][c];
#pragma unroll
                        for (int j = 0; j < kKs; ++j) {
                            p.out[to * D + 16 * j + g] = o[nt][j][c] * w;
                            p.out[to * D + 16 * j + g + 8] = o[nt][j][c + 2] * w;
                        }
                        if (p.lse && g == 0)
                            p.lse[to] = l[nt][c] == 0.f ? -INFINITY : (log2f(l[nt][c]) - base[nt][c]) * kLn2;
                    }
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
        if (!whole && lane == 0) {
            s_unit[part] = at.b * p.hkv + at.h;
            s_unit0[part] = unit0;
        }
    };

    int64_t run0 = f0;
    if (f < f1) enter_unit();
    while (f < f1) {
        const uint8_t *blk0 = ring + slot * F::kBlock;
        const int slot1 = slot + 1 == T::kDepth ? 0 : slot + 1;
        // two blocks at once where every row sees both whole
        const bool pair = !bad && f + 2 <= f1 && ((at.pg >= in_from && at.pg + 2 <= in_to) ||
                                                  (MODE == kKv4Fast && at.pg + 2 <= in_comp));
        if (pair) {
            cp_async_wait<T::kDepth - 2>();
            __syncwarp();
            consume(std::integral_constant<int, 2>{}, std::false_type{}, blk0, ring + slot1 * F::kBlock);
        } else {
            cp_async_wait<T::kDepth - 1>();
            __syncwarp();
            if (!bad) consume(std::integral_constant<int, 1>{}, std::true_type{}, blk0, blk0);
        }
        __syncwarp();  // every lane is done with the blocks that the next copies replace
        issue(slot);
        if (pair) issue(slot1);
        const int step = pair ? 2 : 1;
        slot = pair ? (slot1 + 1 == T::kDepth ? 0 : slot1 + 1) : slot1;
        f += step;
        at.pg += step;
        if (at.pg == plan.n || f == f1) {
            leave_unit(run0, f);
            run0 = f;
            if (f < f1) {
                at.pg = 0;
                if (++at.h == p.hkv) {
                    at.h = 0;
                    do ++at.b; while (s_prefix[at.b + 1] == s_prefix[at.b]);
                }
                enter_unit();
            }
        }
    }
    cp_async_wait<0>();
    __syncthreads();

    // ---- partials of the CTA, unit by unit (in order) ----
    auto part_ptr = [&](int i) {
        return (i & 1) ? reinterpret_cast<const float *>(smem + (i >> 1) * T::kRing)
                       : reinterpret_cast<const float *>(smem + T::kFirst + (i >> 1) * T::kPart);
    };
    for (int i = 0; i < 2 * kWarps;) {
        const int u = s_unit[i];
        if (u < 0) {
            ++i;
            continue;
        }
        int end = i + 1;
        for (int k = i + 1; k < 2 * kWarps; ++k)
            if (s_unit[k] == u) end = k + 1;
        const int b = u / p.hkv, h = u - b * p.hkv;
        const int r = request_id(p, b);
        const int64_t u0 = s_unit0[i], u1 = u0 + (s_prefix[b + 1] - s_prefix[b]);
        const bool complete = u0 >= cta0 && u1 <= cta1;
        // this CTA's slot: 0 when the unit began before it, else 1
        const int64_t ws_slot = (int64_t)blockIdx.x * 2 + (u0 < cta0 ? 0 : 1);
        for (int e = tid; e < r_rows * D; e += kThreads) {
            const int row = e / D, d = e % D;
            float mx = -INFINITY, sum = 0.f, acc = 0.f;
            for (int k = i; k < end; ++k)
                if (s_unit[k] == u) mx = fmaxf(mx, s_ml[k][row][0]);
            for (int k = i; k < end; ++k)
                if (s_unit[k] == u) {
                    const float mk = s_ml[k][row][0];
                    const float w = mk == mx ? 1.f : fast_exp2(mk - mx);
                    sum = fmaf(w, s_ml[k][row][1], sum);
                    acc = fmaf(w, part_ptr(k)[row * D + d], acc);
                }
            if (complete) {
                const int64_t to = ((int64_t)r * p.tokens + row / p.group) * p.hq + h * p.group + row % p.group;
                p.out[to * D + d] = sum == 0.f ? 0.f : acc * (p.v_scale / sum);
                if (p.lse && d == 0) p.lse[to] = sum == 0.f ? -INFINITY : (mx - kLift + log2f(sum)) * kLn2;
            } else {
                p.ws_part[(ws_slot * 16 + row) * D + d] = acc;
                if (d == 0) {
                    p.ws_ml[(ws_slot * 16 + row) * 2] = mx;
                    p.ws_ml[(ws_slot * 16 + row) * 2 + 1] = sum;
                }
            }
        }
        if (!complete) {
            const int c0 = (int)(((u0 + 1) * ctas - 1) / total), c1 = (int)((u1 * ctas - 1) / total);
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const int old = atomicAdd(p.ws_count + u, 1);
                s_last = old == c1 - c0;
                if (s_last) p.ws_count[u] = 0;
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                for (int e = tid; e < r_rows * D; e += kThreads) {
                    const int row = e / D, d = e % D;
                    float mx = -INFINITY, sum = 0.f, acc = 0.f;
#pragma unroll 8
                    for (int c = c0; c <= c1; ++c)
                        mx = fmaxf(mx, __ldcg(p.ws_ml + (((int64_t)c * 2 + (c == c0)) * 16 + row) * 2));
#pragma unroll 8
                    for (int c = c0; c <= c1; ++c) {
                        const int64_t at_row = ((int64_t)c * 2 + (c == c0)) * 16 + row;
                        const float mk = __ldcg(p.ws_ml + at_row * 2);
                        const float w = mk == mx ? 1.f : fast_exp2(mk - mx);
                        sum = fmaf(w, __ldcg(p.ws_ml + at_row * 2 + 1), sum);
                        acc = fmaf(w, __ldcg(p.ws_part + at_row * D + d), acc);
                    }
                    const int64_t to = ((int64_t)r * p.tokens + row / p.group) * p.hq + h * p.group + row % p.group;
                    p.out[to * D + d] = sum == 0.f ? 0.f : acc * (p.v_scale / sum);
                    if (p.lse && d == 0) p.lse[to] = sum == 0.f ? -INFINITY : (mx - kLift + log2f(sum)) * kLn2;
                }
            }
            __syncthreads();
        }
        i = end;
    }
}

namespace {

template <int D, int NT, int MODE>
cudaError_t launch_one(const Kv4AttnParams &p, int ctas, cudaStream_t stream) {
    auto kernel = kv4_attn_kernel<D, NT, MODE>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Tile<D, NT>::kSmem);
    if (e != cudaSuccess) return e;
    kernel<<<ctas, kThreads, Tile<D, NT>::kSmem, stream>>>(p);
    return cudaGetLastError();
}

template <int D, int NT>
cudaError_t launch_mode(const Kv4AttnParams &p, int ctas, cudaStream_t stream) {
    if (p.c_pool) return launch_one<D, NT, kKv4Fast>(p, ctas, stream);
    return p.scores ? launch_one<D, NT, kKv4Scores>(p, ctas, stream) : launch_one<D, NT, kKv4Dense>(p, ctas, stream);
}

}  // namespace

cudaError_t launch_kv4_attn(const Kv4AttnParams &p, int head_dim, cudaStream_t stream) {
    const int sms = sm_count_current_device();
    if (sms <= 0) return cudaErrorInvalidDevice;
    // one wave: two CTAs per SM for up to eight rows, one for up to sixteen (registers)
    if (p.rows <= 8)
        return head_dim == 128 ? launch_mode<128, 1>(p, sms * kKv4CtasPerSm, stream)
                               : launch_mode<64, 1>(p, sms * kKv4CtasPerSm, stream);
    return head_dim == 128 ? launch_mode<128, 2>(p, sms, stream) : launch_mode<64, 2>(p, sms, stream);
}

}  // namespace sfi
