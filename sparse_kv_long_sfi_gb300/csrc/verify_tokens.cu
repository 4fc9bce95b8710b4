// Verification of drafted tokens against the target's probabilities, from given random numbers.
//
// Draft t of a request is accepted while u_t q_t(x_t) < p_t(x_t), which keeps it with probability
// min(1, p / q). Behind a accepted drafts one more token comes from w = max(p_a - q_a, 0), or from
// w = p_a when all were accepted: the first i with w_0 + ... + w_i > u sum(w). Accepted and sampled
// tokens together are distributed as the target's own.
//
// A sample must not depend on the order of a sum, and in a vocabulary's long tail the steps of the
// cumulated weights are smaller than fp32 can tell apart. So weights are whole multiples of 2^-56 in
// 64 bits: p - q is exact there, sums are too (in any order), and the step that holds the sample is
// found among them without rounding. (fp64 sums would do nearly as well, but the fp64 pipe of this GPU
// needs longer for one addition per weight than memory for the weights.)
//
// Bound by HBM for large batches: of 2 T + 1 rows of V values only the row of p (and of q) where the
// drafts end is read whole. A cluster of eight CTAs shares a request's row, so that one request fills
// eight SMs and the row is read once; every CTA keeps the sum of each run of 128 weights, the CTAs
// exchange their totals, and the one that holds the sample reads that run again.
// 64 requests of 150001 tokens with 7 drafts: 26 us (77 MB, 11.3 us of HBM time; clusters of seven, three CTAs on every
// SM, take 29); one of 32000: 5.7 us (latency).
#include "sfi_device.cuh"
#include "sfi_internal.h"

namespace sfi {

namespace {

constexpr int kVerifyCluster = 8;
constexpr int kVerifyThreads = 256;                    // (with 512, 64 requests come in two waves: 33 us)
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyRun = 128;                        // weights of a warp's run, four of each lane
constexpr int kVerifyBatch = 4;                        // runs of a warp whose loads are in flight together
constexpr int kVerifyRuns = SFI_MAX_VOCAB / kVerifyCluster / kVerifyRun + kVerifyWarps;

// What a given value counts as: NaN and values below zero are nothing, values above one are one.
__device__ __forceinline__ float probability(float p) { return fminf(fmaxf(p, 0.f), 1.f); }

// A probability in units of 2^-56, by shifts of its significand (the conversion instruction to 64 bits made the call
// 65 us instead of 33).
__device__ __forceinline__ int64_t fixed(float p) {
    const uint32_t u = __float_as_uint(probability(p));
    const uint64_t one = (uint64_t)((u & 0x7fffffu) | 0x800000u) << 33;  // as for [1, 2)
    return (int64_t)(one >> min(127u - (u >> 23), 63u));
}

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

__device__ __forceinline__ int64_t warp_scan(int64_t v, int lane) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += o;
    }
    return v;
}

}  // namespace

__global__ void __launch_bounds__(kVerifyThreads) verify_tokens_kernel(const VerifyParams p) {
    __shared__ int64_t s_run[kVerifyRuns];
    __shared__ int64_t s_total[kVerifyCluster];
    __shared__ int64_t s_warp[kVerifyWarps];
    __shared__ int s_accepted, s_err;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cluster_ctarank();
    cluster_arrive_relaxed();
    grid_dependency_wait();
    grid_launch_dependents();
    const int b = blockIdx.x / kVerifyCluster;
    const int r = p.req_ids ? p.req_ids[b] : b;
    const int T = p.drafts, V = p.vocab;
    const int n = p.draft_lens ? p.draft_lens[r] : T;
    const int32_t *tok = p.tokens + (int64_t)r * T;
    // accepted drafts: every CTA of the cluster looks at them itself
    if (warp == 0) {
        uint32_t err = n < 0 || n > T ? SFI_DEV_BAD_LEN : 0;
        int a = 0;
        bool more = !err;
        for (int t0 = 0; t0 < n && !err; t0 += 32) {
            const int t = t0 + lane;
            bool ok = true, bad = false;
            if (t < n) {
                const int x = tok[t];
                bad = x < 0 || x >= V;
                if (!bad) {
                    const float pt = probability(p.target[((int64_t)r * (T + 1) + t) * p.target_stride + x]);
                    const float qt = p.draft ? probability(p.draft[((int64_t)r * T + t) * p.draft_stride + x]) : 1.f;
                    // 24 by 24 bits: exact in fp64
                    ok = (double)p.u[(int64_t)r * (T + 1) + t] * (double)qt < (double)pt;
                }
            }
            if (__any_sync(0xffffffffu, bad)) err = SFI_DEV_BAD_INDEX;
            const uint32_t miss = __ballot_sync(0xffffffffu, !ok);
            if (more) a = miss ? t0 + __ffs(miss) - 1 : min(n, t0 + 32);
            more = more && !miss;
        }
        if (lane == 0) {
            s_accepted = a;
            s_err = (int)err;
            if (err && rank == 0) report(p.dev_status, err);
        }
    }
    cluster_wait();  // every CTA has begun: its shared memory may be written
    __syncthreads();
    if (s_err) return;  // the same in every CTA of the cluster
    const int a = s_accepted;
    const bool rejected = a < n;
    const float *prow = p.target + ((int64_t)r * (T + 1) + a) * p.target_stride;
    const float *qrow = rejected && p.draft ? p.draft + ((int64_t)r * T + a) * p.draft_stride : nullptr;
    // with drafts that were no sample but one token's choice, q is 1 there and 0 elsewhere
    int gone = rejected && !p.draft ? tok[a] : -1;

    // this CTA's part of the row, in whole runs
    const int runs = (V + kVerifyRun - 1) / kVerifyRun;
    const int per = (runs + kVerifyCluster - 1) / kVerifyCluster;
    const int run0 = min(rank * per, runs), run1 = min(run0 + per, runs);
    int64_t total = 0, before = 0;
    for (int pass = 0; pass < 2; ++pass) {
        int64_t mine = 0;
        for (int run = run0 + warp; run < run1; run += kVerifyBatch * kVerifyWarps) {
            // all loads of a few runs before the first use
            float pv[kVerifyBatch][4], qv[kVerifyBatch][4];
#pragma unroll
            for (int k = 0; k < kVerifyBatch; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i = (run + k * kVerifyWarps) * kVerifyRun + 32 * j + lane;
                    const bool in = run + k * kVerifyWarps < run1 && i < V && i != gone;
                    pv[k][j] = in ? prow[i] : 0.f;
                    qv[k][j] = in && qrow ? qrow[i] : 0.f;
                }
#pragma unroll
            for (int k = 0; k < kVerifyBatch; ++k) {
                int64_t w = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) w += max(fixed(pv[k][j]) - fixed(qv[k][j]), (int64_t)0);
                w = warp_sum(w);
                const int at = run + k * kVerifyWarps;
                if (lane == 0 && at < run1) s_run[at - run0] = w;
                mine += w;
            }
        }
        if (lane == 0) s_warp[warp] = mine;
        __syncthreads();
        if (warp == 0) {
            const int64_t cta = warp_sum(lane < kVerifyWarps ? s_warp[lane] : 0);
            if (lane < kVerifyCluster) {
                const uint32_t to = cluster_map(smem_u32(&s_total[rank]), (uint32_t)lane);
                asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(to), "l"(cta) : "memory");
            }
        }
        cluster_sync();
        total = before = 0;
#pragma unroll
        for (int i = 0; i < kVerifyCluster; ++i) {
            if (i < rank) before += s_total[i];
            total += s_total[i];
        }
        // p nowhere above q, although a draft was refused (a difference of roundings): p itself
        if (total > 0 || !rejected || pass == 1) break;
        qrow = nullptr;
        gone = -1;
        cluster_sync();  // every CTA has read the totals
    }
    if (total <= 0 && rank == 0 && tid == 0) report(p.dev_status, SFI_DEV_BAD_PROB);
    // u in [0, 1) as a fraction of 2^64 (a NaN is 0): target = floor(u total), and the sample is the
    // first step that lies above it
    const float u = fminf(fmaxf(p.u[(int64_t)r * (T + 1) + T], 0.f), 0.99999994f);
    const int64_t target = (int64_t)__umul64hi((uint64_t)total, __float2ull_rz(u * 18446744073709551616.f));
    const bool here = total > 0 ? target >= before && target < before + s_total[rank] : rank == 0;
    if (here && warp == 0) {
        int next = -1;
        if (total > 0) {
            // the run, then the weight in it
            int64_t sum = before;
            int run = run0;
            for (; run < run1; run += 32) {
                const int64_t v = run + lane < run1 ? s_run[run + lane - run0] : 0;
                const int64_t incl = warp_scan(v, lane);
                const uint32_t above = __ballot_sync(0xffffffffu, sum + incl > target);
                if (above) {
                    const int at = __ffs(above) - 1;
                    sum += __shfl_sync(0xffffffffu, incl - v, at);
                    run += at;
                    break;
                }
                sum += __shfl_sync(0xffffffffu, incl, 31);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = run * kVerifyRun + 32 * j + lane;
                const bool in = i < V && i != gone;
                const float pi = in ? prow[i] : 0.f, qi = in && qrow ? qrow[i] : 0.f;
                const int64_t incl = warp_scan(max(fixed(pi) - fixed(qi), (int64_t)0), lane);
                const uint32_t above = __ballot_sync(0xffffffffu, sum + incl > target);
                if (above && next < 0) next = run * kVerifyRun + 32 * j + __ffs(above) - 1;
                sum += __shfl_sync(0xffffffffu, incl, 31);
            }
        }
        for (int t = lane; t <= T; t += 32)
            p.out_tokens[(int64_t)r * (T + 1) + t] = t < a ? tok[t] : t == a ? next : -1;
        if (lane == 0) {
            p.accepted[r] = a;
            if (p.new_lens) p.new_lens[r] = p.seq_lens[r] - n + a;
        }
    }
    cluster_sync();  // no CTA ends while another may still write its totals
}

cudaError_t launch_verify_tokens(const VerifyParams &p, int batch, cudaStream_t stream) {
    return launch_dependent_clusters(verify_tokens_kernel, batch * kVerifyCluster, kVerifyCluster, kVerifyThreads, 0,
                                     stream, p);
}

}  // namespace sfi
