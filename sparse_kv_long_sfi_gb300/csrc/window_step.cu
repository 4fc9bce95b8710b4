// Attention of a decode step (up to 16 query rows per KV head: one token, or a few drafted ones) over
// the paged cache, through a sliding window with sinks.
//
// Bound by HBM, or by latency for short windows: every visible K and V row is read once and the
// arithmetic is small. So a unit (request, KV head) is spread over a cluster of up to eight CTAs of four
// warps; each warp takes an equal run of the unit's pages and streams it through its own ring of pages
// by TMA, with no barrier between warps. S = Q K^T and O += P V are mma.sync.m16n8k16 (tcgen05 would
// want 64 rows at least, and its hand-overs between warps cost a short step more than they save). P has two
// bf16 terms (as in the decode attention), which costs nothing up to eight rows, which leave half of a fragment free,
// and 1% above.
// Parts meet once: within a CTA through shared memory, then every CTA pushes each share of the rows to
// the CTA that writes it, through distributed shared memory, behind one cluster barrier.
// 32 requests, 32/8/128 heads, window 4096: 85 us (94% of the measured copy bandwidth); 16 requests, 16/8/128
// heads, window 256: 6.7 us (latency).
#include <algorithm>
#include <atomic>

#include "window_span.cuh"

namespace sfi {

namespace {

constexpr int kStepWarps = 4;
constexpr int kStepThreads = kStepWarps * 32;
constexpr int kStepMaxCluster = 8;

template <int D>
struct StepTile {
    static constexpr int kHalves = D / 64;
    static constexpr int kPageBytes = kSubTokens * D * 2;  // K (or V) of a page
    static constexpr int kStages = D == 128 ? 3 : 6;       // pages in flight per warp: two CTAs on an SM
    static constexpr int kWarpBytes = kStages * 2 * kPageBytes;
    static constexpr int kRecvFloats = kMaxRows * D + kStepMaxCluster * 16;  // shares, each padded to 16 floats
    static constexpr int kSmem = kStepWarps * kWarpBytes + kRecvFloats * 4 + 1024;
};

}  // namespace

// EIGHT: at most eight query rows per unit (the other half of a fragment's rows holds the low parts of P).
template <int D, bool EIGHT>
__global__ void __launch_bounds__(kStepThreads, 2)
    window_step_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ WindowParams p) {
    using T = StepTile<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float *recv = reinterpret_cast<float *>(smem + kStepWarps * T::kWarpBytes);  // [CTAs][floats of a share]
    __shared__ __align__(8) uint64_t full[kStepWarps][T::kStages];
    __shared__ float s_m[kStepWarps][kMaxRows], s_l[kStepWarps][kMaxRows];  // per warp
    __shared__ float s_pm[kStepMaxCluster][kMaxRows], s_pl[kStepMaxCluster][kMaxRows];  // per CTA of the cluster
    __shared__ float s_scale[kMaxRows], s_top[kMaxRows], s_sum[kMaxRows];
    __shared__ float s_weight[kStepMaxCluster][kMaxRows];
    __shared__ uint32_t s_odd;  // rows of this CTA's share that are not finite
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ctas = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
    cluster_arrive_relaxed();
    if (lane == 0) {
        for (int i = 0; i < T::kStages; ++i) mbar_init(&full[warp][i], 1);
        fence_barrier_init();
    }
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    __syncwarp();
    grid_dependency_wait();
    grid_launch_dependents();
    const int kvh = blockIdx.y;
    const int r = p.req_ids ? p.req_ids[blockIdx.z] : (int)blockIdx.z;
    if (r < 0 || r >= p.reqs) {
        if (threadIdx.x == 0 && rank == 0 && kvh == 0) report(p.dev_status, SFI_DEV_BAD_INDEX);
        cluster_wait();
        return;
    }
    const int L = p.seq_lens[r];
    const int n = p.new_lens ? p.new_lens[r] : p.tokens;
    if (n <= 0 || n > p.tokens || L < n || L > p.max_pages * kSubTokens) {  // alike in the whole cluster
        if (threadIdx.x == 0 && rank == 0 && kvh == 0 && (n < 0 || n > p.tokens || L < n || L > p.max_pages * kSubTokens))
            report(p.dev_status, SFI_DEV_BAD_LEN);
        cluster_wait();
        return;
    }
    const int G = p.group, rows = n * G;
    const WindowSpan span(L - n, L - 1, p.sink, p.recent);
    // this warp's run of pages
    const int workers = ctas * kStepWarps, me = rank * kStepWarps + warp;
    const int page0 = (int)((int64_t)span.pages * me / workers), page1 = (int)((int64_t)span.pages * (me + 1) / workers);
    const int32_t *ptab = p.page_table + (int64_t)r * p.max_pages;
    uint8_t *ring = smem + warp * T::kWarpBytes;
    bool bad = false;
    int ids = page0 + lane < page1 ? ptab[span.page(page0 + lane)] : 0;  // of the next 32 pages
    const int g = lane >> 2, t = lane & 3, mi = lane >> 3, r8 = lane & 7;
    // Q's fragments: rows g and g + 8 (row = token * G + head)
    uint32_t qa[D / 16][4];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int row = g + 8 * half, tok = row / G;
        const __nv_bfloat16 *q = p.q + ((int64_t)r * p.tokens + tok) * p.q_stride + ((int64_t)kvh * G + row % G) * D + 2 * t;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            qa[ks][half] = row < rows ? *reinterpret_cast<const uint32_t *>(q + ks * 16) : 0u;
            qa[ks][2 + half] = row < rows ? *reinterpret_cast<const uint32_t *>(q + ks * 16 + 8) : 0u;
        }
    }
    // requests page v of this run (warp-collective)
    auto request = [&](int v) {
        const int i = v - page0;
        if (i > 0 && (i & 31) == 0) ids = v + lane < page1 ? ptab[span.page(v + lane)] : 0;
        const int page = __shfl_sync(0xffffffffu, ids, i & 31);
        const bool ok = page >= 0 && page < p.num_pages;
        bad |= !ok;
        if (lane == 0) {
            const int st = i % T::kStages;
            uint8_t *to = ring + st * 2 * T::kPageBytes;
            if (ok) {
                mbar_arrive_expect_tx(&full[warp][st], 2 * T::kPageBytes);
                const uint64_t policy = l2_policy_evict_first();
                const int y = (page * p.hkv + kvh) * kSubTokens;
#pragma unroll
                for (int h = 0; h < T::kHalves; ++h) {
                    tma_load_2d(to + h * (kSubTokens * 128), &tm_k, h * 64, y, &full[warp][st], policy);
                    tma_load_2d(to + T::kPageBytes + h * (kSubTokens * 128), &tm_v, h * 64, y, &full[warp][st], policy);
                }
            } else {
                mbar_arrive(&full[warp][st]);
            }
        }
        __syncwarp();
    };
    for (int v = page0; v < min(page1, page0 + T::kStages); ++v) request(v);

    const RowWindow first(L - n, p.sink, p.recent, span), last(L - 1, p.sink, p.recent, span);
    const RowWindow wa(L - n + min(g, rows - 1) / G, p.sink, p.recent, span);
    const RowWindow wb(L - n + min(g + 8, rows - 1) / G, p.sink, p.recent, span);
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    bool late = false;
    for (int v = page0; v < page1; ++v) {
        const int st = (v - page0) % T::kStages;
        if (!mbar_wait_warp(&full[warp][st], ((v - page0) / T::kStages) & 1)) {
            late = true;
            // (the ring has another use below: what is on its way lands first, within the same limits)
            for (int u = v - page0; u < min(page1, v + T::kStages) - page0; ++u)
                mbar_wait_warp(&full[warp][u % T::kStages], (u / T::kStages) & 1);
            break;
        }
        const uint32_t ka = smem_u32(ring + st * 2 * T::kPageBytes), va = ka + T::kPageBytes;
        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t b0, b1, b2, b3;
            ldsm_x4(ka + (ks >> 2) * (kSubTokens * 128) + (((mi >> 1) << 3) + r8) * 128 +
                        ((((ks & 3) * 2 + (mi & 1)) ^ r8) << 4),
                    b0, b1, b2, b3);
            mma_bf16_16816(s[0], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], b0, b1);
            mma_bf16_16816(s[1], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], b2, b3);
        }
        // this lane's slots of rows g (x[0]) and g + 8 (x[1])
        float x[2][4] = {{s[0][0], s[0][1], s[1][0], s[1][1]}, {s[0][2], s[0][3], s[1][2], s[1][3]}};
        const int v0 = v * kSubTokens;
        const bool whole = all_see(v0, kSubTokens, first, last);
        uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
        if (!whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = v0 + (i >> 1) * 8 + 2 * t + (i & 1);
                if (!wa.sees(at)) x[0][i] = -INFINITY;
                if (!wb.sees(at)) x[1][i] = -INFINITY;
                // V rows that no row sees may hold anything, NaN among it
                if (!(at < last.sink || (at < last.hi && (first.hi == 0 || at >= first.lo))))
                    keep[i >> 1] &= (i & 1) ? 0x0000ffffu : 0xffff0000u;
            }
        }
        // P of rows g, g + 8: slots 0-7 and 8-15. As two bf16 terms (2^-16 of a weight at most is lost): the low ones
        // are rows 8 to 15 of the same product where those are free, else a product of their own.
        uint32_t pa[2][2], pb[2][2];
        bool moved = false;
        float alpha[2];
#pragma unroll
        for (int h = 0; h < (EIGHT ? 1 : 2); ++h) {
            float top = fmaxf(fmaxf(x[h][0], x[h][1]), fmaxf(x[h][2], x[h][3]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float now = fmaxf(m[h], top * p.scale_log2);
            const float base = now == -INFINITY ? 0.f : now;
            alpha[h] = fast_exp2(m[h] - base);
            moved |= alpha[h] != 1.f;
            m[h] = now;
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = fast_exp2(fmaf(x[h][i], p.scale_log2, -base));
            l[h] = l[h] * alpha[h] + ((w[0] + w[1]) + (w[2] + w[3]));
#pragma unroll
            for (int i = 0; i < 2; ++i) split_bf16x2(w[2 * i], w[2 * i + 1], pa[h][i], pb[h][i]);
        }
        if (EIGHT) {
            alpha[1] = alpha[0];
            pa[1][0] = pb[0][0];
            pa[1][1] = pb[0][1];
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                o[i][0] *= alpha[0];
                o[i][1] *= alpha[0];
                o[i][2] *= alpha[1];
                o[i][3] *= alpha[1];
            }
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            uint32_t b0, b1, b2, b3;
            ldsm_x4_trans(va + (j >> 2) * (kSubTokens * 128) + (((mi & 1) << 3) + r8) * 128 +
                              ((((j & 3) * 2 + (mi >> 1)) ^ r8) << 4),
                          b0, b1, b2, b3);
            if (!whole) {
                b0 &= keep[0];
                b1 &= keep[1];
                b2 &= keep[0];
                b3 &= keep[1];
            }
            mma_bf16_16816(o[2 * j], pa[0][0], pa[1][0], pa[0][1], pa[1][1], b0, b1);
            mma_bf16_16816(o[2 * j + 1], pa[0][0], pa[1][0], pa[0][1], pa[1][1], b2, b3);
            if (!EIGHT) {
                mma_bf16_16816(o[2 * j], pb[0][0], pb[1][0], pb[0][1], pb[1][1], b0, b1);
                mma_bf16_16816(o[2 * j + 1], pb[0][0], pb[1][0], pb[0][1], pb[1][1], b2, b3);
            }
        }
        __syncwarp();  // the page has been read
        if (v + T::kStages < page1) request(v + T::kStages);
    }
    if (bad && lane == 0) report(p.dev_status, SFI_DEV_BAD_PAGE);
    if (late && lane == 0) report(p.dev_status, SFI_DEV_TIMEOUT);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    // ---- the CTA's warps, through each warp's own ring ----
    float *mine = reinterpret_cast<float *>(ring);  // [16][D]
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        float *to = mine + g * D + ((i * 8 + 2 * t) ^ ((g & 3) << 3));
        if (EIGHT) {
            *reinterpret_cast<float2 *>(to) = make_float2(o[i][0] + o[i][2], o[i][1] + o[i][3]);
        } else {
            *reinterpret_cast<float2 *>(to) = make_float2(o[i][0], o[i][1]);
            *reinterpret_cast<float2 *>(to + 8 * D) = make_float2(o[i][2], o[i][3]);
        }
    }
    if (t == 0) {
        s_m[warp][g] = m[0];
        s_m[warp][g + 8] = m[1];
        s_l[warp][g] = l[0];
        s_l[warp][g + 8] = l[1];
    }
    if (threadIdx.x == 0) s_odd = 0;
    cluster_wait();  // every CTA of the cluster has begun
    const bool failed = __syncthreads_or(bad || late);
    // this CTA's part of each share goes to the CTA that writes it
    const int pieces = rows * (D / 4), share = (pieces + ctas - 1) / ctas;  // in units of four values
    for (int i = threadIdx.x; i < pieces; i += kStepThreads) {
        const int row = i / (D / 4), d = (i % (D / 4)) * 4;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kStepWarps; ++w) top = fmaxf(top, s_m[w][row]);
        const float base = top == -INFINITY ? 0.f : top;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kStepWarps; ++w) {
            const float f = fast_exp2(s_m[w][row] - base);
            const float4 v = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(smem + w * T::kWarpBytes) +
                                                               row * D + (d ^ ((row & 3) << 3)));
            sum.x += v.x * f;
            sum.y += v.y * f;
            sum.z += v.z * f;
            sum.w += v.w * f;
        }
        const int owner = i / share;
        st_cluster_f32x4(cluster_map(smem_u32(recv + (rank * share + i - owner * share) * 4), (uint32_t)owner), sum);
    }
    for (int i = threadIdx.x; i < rows * ctas; i += kStepThreads) {
        const int row = i % rows, to = i / rows;
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kStepWarps; ++w) top = fmaxf(top, s_m[w][row]);
        const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int w = 0; w < kStepWarps; ++w) sum += s_l[w][row] * fast_exp2(s_m[w][row] - base);
        st_cluster_f32(cluster_map(smem_u32(&s_pm[rank][row]), (uint32_t)to), top);
        st_cluster_f32(cluster_map(smem_u32(&s_pl[rank][row]), (uint32_t)to), failed ? -1.f : sum);
    }
    cluster_sync();
    // ---- this CTA's share of the output ----
    if (threadIdx.x < rows) {
        const int row = threadIdx.x;
        float top = -INFINITY, sum = 0.f;
        bool miss = false;
        for (int c = 0; c < ctas; ++c) {
            top = fmaxf(top, s_pm[c][row]);
            miss |= s_pl[c][row] < 0.f;
        }
        const float base = top == -INFINITY ? 0.f : top;
        for (int c = 0; c < ctas; ++c) {
            const float f = fast_exp2(s_pm[c][row] - base);
            s_weight[c][row] = f;
            sum += s_pl[c][row] * f;
        }
        s_top[row] = base;
        s_sum[row] = sum;
        s_scale[row] = miss ? -1.f : sum == 0.f ? 0.f : 1.f / sum;
        if (!miss && p.lse && rank == 0) {
            const int64_t at = ((int64_t)r * p.tokens + row / G) * p.hq + (int64_t)kvh * G + row % G;
            p.lse[at] = sum == 0.f ? -INFINITY : (base + log2f(sum)) * 0.6931471805599453f;
        }
    }
    __syncthreads();
    const int piece1 = min(pieces, (rank + 1) * share);
    for (int i = rank * share + (int)threadIdx.x; i < piece1; i += kStepThreads) {
        const int row = i / (D / 4), d = (i % (D / 4)) * 4;
        const float scale = s_scale[row];
        if (scale < 0.f) continue;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < ctas; ++c) {
            const float f = s_weight[c][row];
            const float4 v = *reinterpret_cast<const float4 *>(recv + (c * share + i - rank * share) * 4);
            sum.x += v.x * f;
            sum.y += v.y * f;
            sum.z += v.z * f;
            sum.w += v.w * f;
        }
        if (n > 1 && !(fabsf(sum.x) + fabsf(sum.y) + fabsf(sum.z) + fabsf(sum.w) < INFINITY)) atomicOr(&s_odd, 1u << row);
        const int64_t at = ((int64_t)r * p.tokens + row / G) * p.hq + (int64_t)kvh * G + row % G;
        *reinterpret_cast<uint2 *>(p.out + at * D + d) =
            make_uint2(pack_bf16x2(sum.x * scale, sum.y * scale), pack_bf16x2(sum.z * scale, sum.w * scale));
    }
    if (n == 1) return;
    // (with several tokens a row may have met the NaN of a position that only later tokens see)
    __syncthreads();
    if (warp > 0 || s_odd == 0) return;
    const int row = min(lane, rows - 1);
    mend_rows<D, true>(p, r, kvh, L, n, L - n, L - 1, 0, lane < rows && (s_odd >> row & 1u), s_top[row], s_sum[row],
                       rank * share, piece1);
}

namespace {

// CTAs of a unit: while all of them fit the SMs (two each) and every warp has two pages at least; of long units two at
// least, whose second wave evens out the first. (256 units of 4160 rows: 88 us in 256 CTAs, 84 in 512, 91 in 1024; 128
// units of 320 rows: 6.7 us in 256 CTAs, 15 in 512.)
int step_cluster(int64_t units, int pages, int sms) {
    int c = 1;
    while (c < kStepMaxCluster && units * 2 * c <= 2 * (int64_t)sms && pages >= 4 * c * kStepWarps) c *= 2;
    return c == 1 && pages >= 32 * kStepWarps ? 2 : c;
}

template <int D, bool EIGHT>
cudaError_t launch_step(const WindowMaps &maps, const WindowParams &p, int batch, cudaStream_t stream) {
    auto kernel = window_step_kernel<D, EIGHT>;
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kernel), StepTile<D>::kSmem, configured);
    if (e != cudaSuccess) return e;
    const int sms = sm_count_current_device();
    if (sms <= 0) return cudaErrorInvalidDevice;
    // the most pages that a unit can read
    const int64_t seen = (int64_t)p.sink + p.recent + p.tokens + 2 * kSubTokens;
    const int pages = (int)std::min<int64_t>(p.max_pages, seen / kSubTokens);
    const int ctas = step_cluster((int64_t)batch * p.hkv, pages, sms);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, (unsigned)p.hkv, (unsigned)batch);
    cfg.blockDim = dim3(kStepThreads);
    cfg.dynamicSmemBytes = StepTile<D>::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, maps.k, maps.v, p);
}

}  // namespace

cudaError_t launch_window_step(const WindowMaps &maps, const WindowParams &p, int head_dim, int batch,
                               cudaStream_t stream) {
    const bool eight = (int64_t)p.tokens * p.group <= 8;
    const auto launch = head_dim == 128 ? (eight ? launch_step<128, true> : launch_step<128, false>)
                                        : (eight ? launch_step<64, true> : launch_step<64, false>);
    return launch(maps, p, batch, stream);
}

}  // namespace sfi
