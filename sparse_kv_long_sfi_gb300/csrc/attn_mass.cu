// Accumulated attention weights: what the queries of new tokens gave to each cached position,
//   mass[h][j] = decay mass[h][j] + sum over tokens t that see j and heads g of exp(x_{t,g,j} - lse_{t,g}).
//
// The attention call has left the log-sum-exps, so a weight needs no second pass over its row. With many
// tokens it is bound by the tensor cores and the exponentials (2 D flops and one exp per pair), with few
// by HBM (K is read once). S^T = K Q^T puts positions on the M side: a thread owns a position, and the sum
// over the query rows is a sum over the columns it reads, with no exchange between threads and one writer
// per position (no atomics: the order of additions, and so the result, is the same in every run).
//
// Two kernels:
//  * Long calls (over 128 query rows): an item is 256 positions of one KV head, as two tiles of 128, and the query rows
//    that see any of them (row = token * G + head) in tiles of 128. The K rows lie in tensor memory as the A operand
//    (they come by TMA, and each thread moves half of its own position's row), so the products read the query rows
//    alone from shared memory, at the rate of the tensor cores; with K in shared memory too they took 82 cycles instead
//    of 64. Three buffers of S^T are used in turn, and free again as soon as a thread has its 64 columns in registers;
//    sums are fp32, eight of them per position and tile. A CTA that is done takes over one that has not begun (cluster
//    launch control), when the loads of its last item are under way: started anew for each item, it spent 8 us on its
//    own beginning and end (16 chunks of 512 tokens behind 4096, 8 steps each: 225 us then, 162 now), and taken
//    earlier, long items had others behind them (one prompt of 8192: 193 us).
//    Where items are few, a cluster shares the query rows of each (see mass_parts).
//  * Short calls: the query rows (16, 32, 64 or 128 of them) stay in shared memory, and a CTA walks a run of
//    tiles of 128 positions through a ring; two warpgroups take the tiles in turn.
// A prompt of 8192 tokens, 16/8/128 heads: 131 us (56% of the measured bf16 rate); two of 32/8/128: 467 us (63%). A step
// of 256 positions x 128 query rows takes 1850 cycles, of which the exponentials need 1090 and the products 1024: reads of
// tensor memory (480 cycles of a warp beside the products) and waits are not hidden by four warps per scheduler. Slower:
// half of a step's columns read while half of the last are summed (317 us where this takes 256), both tiles' positions in
// each thread (304, with half of the reads of shared memory).
// The last 64 tokens of 8 x 16384, 16/8/128 heads: 52 us (79% of the measured copy
// bandwidth). A CTA's run follows the table's and the weights' width: 123 us where these are 131072 positions wide.
#include <algorithm>
#include <atomic>

#include "tensor_core.cuh"
#include "window_span.cuh"

namespace sfi {

namespace {

constexpr int kLongThreads = 640;   // four warpgroups of sums; in the fifth a copy warp and two matrix warps
constexpr int kLongWarps = 16;
// Registers of a thread: the launch gives 96 (640 x 96 = 61440); 512 x 104 + 128 x 64 = 61440. (The sums hold 64 columns
// each; every spilled value in their loop shows.)
constexpr int kLongSumRegs = 104, kLongOtherRegs = 64;
constexpr int kShortThreads = 320;  // two warpgroups of sums, a copy warp, a matrix warp
constexpr int kShortWarps = 8;
constexpr int kMassKeys = 256;     // positions of a CTA
constexpr int kKeyTile = 128;
constexpr int kMassMaxParts = 8;   // CTAs that share a long call's positions, each with a part of the query rows

template <int D, int ROWS>
struct MassTile {
    static constexpr int kHalves = D / 64;
    static constexpr int kKeyHalf = kKeyTile * 128;
    static constexpr int kKeyBytes = kHalves * kKeyHalf;  // K of 128 positions
    static constexpr int kRowHalf = ROWS * 128;
    static constexpr int kRowBytes = kHalves * kRowHalf;  // a tile of query rows
    static constexpr uint32_t kScores = mma_desc(kKeyTile, ROWS, false);
};
template <int D>
struct LongTile : MassTile<D, 128> {
    static constexpr int kRows = 128;
    static constexpr int kStages = 6;   // of query rows and K
    static constexpr int kBuffers = 3;  // of S^T
    static constexpr int kScoresAt = 128;  // tensor memory: K of the two tiles (at 0 and 64), then S^T
    static constexpr int kColumns = 512;
    static constexpr int kSmem = kStages * MassTile<D, 128>::kRowBytes + 1024;
};
template <int D, int ROWS>
struct ShortTile : MassTile<D, ROWS> {
    static constexpr int kStages = (ROWS <= 32 ? 3 : 2) * (128 / D);  // of keys: two CTAs on an SM
    static constexpr int kColumns = 2 * ROWS;                        // two buffers of S^T
    static constexpr int kSmem = MassTile<D, ROWS>::kRowBytes + kStages * MassTile<D, ROWS>::kKeyBytes + 1024;
};

// Weights of one position, summed over COLS columns (query rows) of its lane of S^T: all of them, or [lo, hi).
// lse: the columns' -lse in log2 units.
template <int COLS, bool WHOLE>
__device__ __forceinline__ void add_columns(const uint32_t (&s)[COLS], const float *lse, uint64_t scale, int lo, int hi,
                                            uint64_t (&sum)[4]) {
#pragma unroll
    for (int i = 0; i < COLS; i += 4) {
        const float4 e = *reinterpret_cast<const float4 *>(&lse[i]);
        const float2 x = unpair(fma2(pair(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), scale, pair(e.x, e.y)));
        const float2 y = unpair(fma2(pair(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])), scale, pair(e.z, e.w)));
        float v[4] = {fast_exp2(x.x), fast_exp2(x.y), fast_exp2(y.x), fast_exp2(y.y)};
        if (!WHOLE) {
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = i + k >= lo && i + k < hi ? v[k] : 0.f;
        }
        sum[(i >> 1) & 3] = add2(sum[(i >> 1) & 3], pair(v[0], v[1]));
        sum[((i >> 1) & 3) + 1] = add2(sum[((i >> 1) & 3) + 1], pair(v[2], v[3]));
    }
}

__device__ __forceinline__ float total(const uint64_t (&sum)[4]) {
    const float2 both = unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
    return both.x + both.y;
}

// The same from tensor memory; while some columns are summed, the next are on their way.
template <int COLS, bool WHOLE>
__device__ __forceinline__ float sum_columns(uint32_t addr, const float *lse, float scale_log2, int lo, int hi) {
    constexpr int kLoad = COLS < 32 ? 16 : 32;  // columns of one read of tensor memory
    uint32_t s[2][kLoad];
    auto load = [&](int c, uint32_t (&v)[kLoad]) {
        if constexpr (kLoad == 32) tmem_load32(addr + c, v);
        else tmem_load16(addr + c, v);
    };
    const uint64_t scale = pair(scale_log2, scale_log2);
    uint64_t sum[4] = {0, 0, 0, 0};
    load(0, s[0]);
#pragma unroll
    for (int c = 0; c < COLS; c += kLoad) {
        tmem_wait_load();
        if (c + kLoad < COLS) load(c + kLoad, s[(c / kLoad & 1) ^ 1]);
        add_columns<kLoad, WHOLE>(s[c / kLoad & 1], lse + c, scale, lo - c, hi - c, sum);
    }
    return total(sum);
}

// 256 positions of one (request, KV head), from k0 on. kvh < 0: there is none left.
struct MassItem {
    int kvh, r, L, n, k0;
};

// What all roles derive of an item: its last position, and this CTA's share of the tiles of query rows, from position
// `from` on (tokens that see any of its positions, in whole tiles).
struct MassWork {
    int k1, from, steps;
    __device__ __forceinline__ MassWork(const MassItem &it, const WindowParams &p, int per_tile, int rank, int parts) {
        k1 = min(it.k0 + kMassKeys, it.L) - 1;
        const int seen = max(it.L - it.n, it.k0);
        const int to = it.k0 < p.sink ? it.L - 1 : (int)min((int64_t)it.L - 1, (int64_t)k1 + p.recent - 1);
        const int all = it.n > 0 && to >= seen ? (to - seen) / per_tile + 1 : 0;
        const int step0 = (int)((int64_t)all * rank / parts);
        steps = (int)((int64_t)all * (rank + 1) / parts) - step0;
        from = seen + step0 * per_tile;
    }
};

}  // namespace

template <int D>
__global__ void __launch_bounds__(kLongThreads, 1)
    mass_long_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const WindowParams p, const MassParams w, int units) {
    using T = LongTile<D>;
    constexpr int ROWS = T::kRows;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ __align__(16) uint4 s_answer;
    __shared__ __align__(8) uint64_t answered, item_full[2], item_read[2];
    __shared__ __align__(8) uint64_t k_full[2], part_full[2], full[T::kStages], empty[T::kStages];
    __shared__ __align__(8) uint64_t s_full[2][4], s_empty[2][4], products_end[2];  // of a tile's products, in turn
    __shared__ MassItem s_item[2];
    __shared__ __align__(16) float s_lse[T::kStages][ROWS];  // -lse in log2 units
    __shared__ int s_bad[T::kStages];                        // a tile of K: a page of the item is out of range
    __shared__ float s_part[kMassKeys];                      // sums over the second half of the columns
    __shared__ float s_recv[kMassMaxParts - 1][kMassKeys];   // (the first CTA's) sums of the other CTAs of a cluster
    __shared__ float s_failed[kMassMaxParts - 1];            // whether they failed
    __shared__ uint32_t s_tmem;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int parts = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        mbar_init(&answered, 1);
        for (int i = 0; i < T::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kLongWarps);
        }
        for (int i = 0; i < 2; ++i) {
            for (int k = 0; k < 4; ++k) {
                mbar_init(&s_full[i][k], 1);
                mbar_init(&s_empty[i][k], kLongWarps / 2);
            }
            mbar_init(&item_full[i], 1);
            mbar_init(&item_read[i], kLongWarps + 2);
            mbar_init(&k_full[i], kLongWarps / 2 * 32);
            mbar_init(&part_full[i], kLongWarps / 4);
            mbar_init(&products_end[i], 1);
        }
        fence_barrier_init();
    }
    if (warp == kLongWarps + 1) tmem_alloc(&s_tmem, T::kColumns);
    cluster_arrive_relaxed();
    grid_dependency_wait();
    grid_launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const int G = p.group, shift = __ffs(G) - 1, per_tile = ROWS >> shift;
    bool fine = true, spoiled = false;  // (spoiled: a bad page)
    float acc = 0.f, old = 0.f;  // of this thread's position, in a cluster still here at the end
    float *to = nullptr;

    if (warp >= kLongWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLongOtherRegs));
        if (warp == kLongWarps) {
            // ---- the items: K of the positions, then the query rows tile by tile. The next is taken when all loads of
            // the last are under way, shortly before its sums end, so that the longest have none behind them. ----
            uint32_t x = blockIdx.x / parts;
            bool left = true;
            int taken = 0;
            auto next_item = [&]() {  // one thread
                MassItem it{-1, 0, 0, 0, 0};
                while (left && it.kvh < 0) {
                    if (taken > 0) {
                        bool late = false;
                        left = parts == 1 && take_next_cta(&s_answer, &answered, (taken - 1) & 1, x, late);
                        if (late) report(p.dev_status, SFI_DEV_TIMEOUT);
                        if (!left) break;
                    }
                    ++taken;
                    // (the blocks with the most query rows, the first of every request and head, first)
                    const int block = (int)x / units, unit = (int)x - block * units;
                    const int b = unit / p.hkv, kvh = unit - b * p.hkv;
                    const int r = p.req_ids ? p.req_ids[b] : b;
                    const bool lead = block == 0 && kvh == 0 && rank == 0;
                    if (r < 0 || r >= p.reqs) {
                        if (lead) report(p.dev_status, SFI_DEV_BAD_INDEX);
                        continue;
                    }
                    const int L = p.seq_lens[r], n = p.new_lens ? p.new_lens[r] : p.tokens;
                    if (n < 0 || n > p.tokens || L < n || L > p.max_pages * kSubTokens || L > w.stride) {
                        if (lead) report(p.dev_status, SFI_DEV_BAD_LEN);
                        continue;
                    }
                    if ((int64_t)block * kMassKeys < L) it = MassItem{kvh, r, L, n, block * kMassKeys};
                }
                return it;
            };
            int use = 0;
            auto next_slot = [&]() {
                const int slot = use % T::kStages;
                fine = use < T::kStages || tc_wait(&empty[slot], (use / T::kStages - 1) & 1);
                use += fine;
                return slot;
            };
            for (int i = 0; fine; ++i) {
                fine = i < 2 || tc_wait(&item_read[i & 1], ((i >> 1) - 1) & 1);
                if (!fine) break;
                if (lane == 0) {
                    s_item[i & 1] = next_item();
                    mbar_arrive(&item_full[i & 1]);
                }
                __syncwarp();
                const MassItem it = s_item[i & 1];
                if (it.kvh < 0) break;
                const MassWork work(it, p, per_tile, rank, parts);
                if (work.steps == 0) continue;
                // page ids: a lane each; this lane's rows of the next tile: their log-sum-exps are fetched a step ahead
                const bool listed = lane < kMassKeys / kSubTokens && it.k0 + lane * kSubTokens <= work.k1;
                const int page = listed ? p.page_table[(int64_t)it.r * p.max_pages + it.k0 / kSubTokens + lane] : -1;
                const float *lse = w.lse + (int64_t)it.r * p.tokens * p.hq + (it.kvh << shift);
                float next[ROWS / 32];
                auto fetch = [&](int j) {
#pragma unroll
                    for (int k = 0; k < ROWS / 32; ++k) {
                        const int row = k * 32 + lane, tok = work.from - (it.L - it.n) + j * per_tile + (row >> shift);
                        next[k] = j < work.steps && tok < it.n
                                      ? lse[(int64_t)tok * p.hq + (row & (G - 1))] * -1.4426950408889634f
                                      : 0.f;
                    }
                };
                fetch(0);
                const bool ok = page >= 0 && page < p.num_pages;
                const uint32_t take = __ballot_sync(0xffffffffu, ok);
                const bool bad = __any_sync(0xffffffffu, listed && !ok);
                if (bad && lane == 0) report(p.dev_status, SFI_DEV_BAD_PAGE);
                for (int t = 0; t < 2 && fine; ++t) {
                    const int slot = next_slot();
                    if (!fine) break;
                    const uint32_t pages = take >> (t * 8) & 0xffu;
                    if (lane == 0) {
                        s_bad[slot] = bad;  // nothing of the item's positions is written
                        if (pages) mbar_arrive_expect_tx(&full[slot], __popc(pages) * kSubTokens * D * 2);
                        else mbar_arrive(&full[slot]);
                    }
                    const int half = lane >> 3, at = lane & 7, mine = __shfl_sync(0xffffffffu, page, t * 8 + at);
                    __syncwarp();
                    if (half < T::kHalves && (pages >> at & 1u))
                        tma_tile_2d(ring + slot * T::kRowBytes + half * T::kKeyHalf + at * kSubTokens * 128, &tm_k,
                                    half * 64, (mine * p.hkv + it.kvh) * kSubTokens, &full[slot]);
                }
                for (int j = 0; j < work.steps && fine; ++j) {
                    const int slot = next_slot();
                    if (!fine) break;
#pragma unroll
                    for (int k = 0; k < ROWS / 32; ++k) s_lse[slot][k * 32 + lane] = next[k];
                    fetch(j + 1);
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&full[slot], T::kRowBytes);
#pragma unroll
                        for (int h = 0; h < T::kHalves; ++h)
                            tma_tile_3d(ring + slot * T::kRowBytes + h * T::kRowHalf, &tm_q, h * 64, it.kvh << shift,
                                        it.r * p.tokens + work.from - (it.L - it.n) + j * per_tile, &full[slot]);
                    }
                    __syncwarp();
                }
            }
            drain_ring(full, use);
        } else if (warp < kLongWarps + 3) {
            // ---- one thread for each of the two tiles (see tc_wait_one) ----
            const int t = warp - kLongWarps - 1;
            if (lane == 0) {
                const uint32_t ra = smem_u32(ring);
                int use = 0, product = t, mine = 0;  // of the ring, of the buffers, and items with any so far
                for (int i = 0; fine; ++i) {
                    fine = tc_wait_one(&item_full[i & 1], (i >> 1) & 1);
                    if (!fine) break;
                    const MassItem it = s_item[i & 1];
                    mbar_arrive(&item_read[i & 1]);
                    if (it.kvh < 0) break;
                    const MassWork work(it, p, per_tile, rank, parts);
                    if (work.steps == 0) continue;
                    use += 2;
                    fine = tc_wait_one(&k_full[t], mine++ & 1);
                    for (int j = 0; j < work.steps && fine; ++j, ++use, product += 2) {
                        const int slot = use % T::kStages, buf = product % T::kBuffers, own = product >> 1;
                        const int before = product - T::kBuffers;  // the other tile's, which had the buffer
                        fine = tc_wait_one(&full[slot], (use / T::kStages) & 1) &&
                               (before < 0 || tc_wait_one(&s_empty[t ^ 1][before >> 1 & 3], (before >> 3) & 1));
                        if (!fine) break;
                        tc_fence_after();
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks)
                            mma_ts(tmem + T::kScoresAt + buf * ROWS, tmem + t * 64 + ks * 8,
                                   smem_desc(ra + slot * T::kRowBytes + (ks >> 2) * T::kRowHalf + (ks & 3) * 32, 16), T::kScores,
                                   ks > 0);
                        mma_commit(&s_full[t][own & 3]);
                    }
                }
                drain_products(&products_end[t]);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kLongSumRegs));
        // ---- one position per thread, half of the columns each: four warps of every scheduler hide what the
        // reads of tensor memory, exponentials and hand-overs of one leave open ----
        constexpr int kCols = ROWS / 2;
        const int t = (warp >> 2) & 1, half = warp >> 3, row = (int)threadIdx.x & (kKeyTile - 1);
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
        int use = 0, product = t, mine = 0;  // of the ring, of the buffers, and items with any so far
        for (int i = 0; fine; ++i) {
            fine = tc_wait(&item_full[i & 1], (i >> 1) & 1);
            if (!fine) break;
            // (what a step needs of it now and then is read again: the loop has no registers to spare)
            const MassItem &it = s_item[i & 1];
            if (it.kvh < 0) break;
            int from, steps, whole0, whole1;  // steps [whole0, whole1): all tokens see all positions of the tile
            acc = old = 0.f;
            {
                const MassWork work(it, p, per_tile, rank, parts);
                from = work.from;
                steps = work.steps;
                const int tile0 = it.k0 + t * kKeyTile, tile1 = min(tile0 + kKeyTile - 1, work.k1);
                whole0 = max(0, (tile1 - from + per_tile - 1) / per_tile);
                // the last position whose token sees all of the tile
                const int64_t last = tile1 < p.sink ? it.L - 1 : min((int64_t)it.L - 1, (int64_t)tile0 + p.recent - 1);
                whole1 = last + 1 < from + per_tile ? 0 : (int)((last + 1 - from) / per_tile);
                const int key = tile0 + row;
                if (half == 0 && rank == 0 && key < it.L - it.n && w.decay != 0.f)
                    old = w.decay * w.mass[((int64_t)it.r * p.hkv + it.kvh) * w.stride + key];
            }
            bool bad = false;
            if (steps > 0) {
                // half of this position's K row goes to tensor memory (the products of the last item are done). Every
                // warp waits for all of the ring in order: a phase of a slot that it had left out could be taken for
                // the next but one. (A second tile without positions is gone through all the same.)
#pragma unroll
                for (int e = 0; e < 2; ++e, ++use) {
                    const int slot = use % T::kStages;
                    fine = fine && tc_wait(&full[slot], (use / T::kStages) & 1);
                    if (fine && e == t) {
                        spoiled |= bad = s_bad[slot] != 0;
                        const uint8_t *k = ring + slot * T::kRowBytes + (D == 128 ? half * T::kKeyHalf : 0) + row * 128;
                        uint32_t x[D / 4];
#pragma unroll
                        for (int c = 0; c < D / 16; ++c) {
                            const int at = D == 128 ? c : half * 4 + c;
                            const uint4 v = *reinterpret_cast<const uint4 *>(k + ((at ^ (row & 7)) << 4));
                            x[4 * c] = v.x;
                            x[4 * c + 1] = v.y;
                            x[4 * c + 2] = v.z;
                            x[4 * c + 3] = v.w;
                        }
                        if constexpr (D == 128) tmem_store32(lanes + t * 64 + half * 32, x);
                        else tmem_store16(lanes + t * 64 + half * 16, x);
                        tmem_wait_store();
                        tc_fence_before();
                        mbar_arrive(&k_full[t]);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&empty[slot]);
                }
                if (!fine) break;
                for (int j = 0; j < steps; ++j, ++use, product += 2) {
                    const int slot = use % T::kStages, buf = product % T::kBuffers, own = product >> 1;
                    fine = tc_wait(&full[slot], (use / T::kStages) & 1) && tc_wait(&s_full[t][own & 3], (own >> 2) & 1);
                    if (!fine) break;
                    tc_fence_after();
                    // all of this thread's columns, so that the buffer is free for another product while they are summed
                    const uint32_t addr = lanes + T::kScoresAt + buf * ROWS + half * kCols;
                    const float *lse = s_lse[slot] + half * kCols;
                    uint32_t s[kCols];
                    tmem_load32(addr, reinterpret_cast<uint32_t(&)[32]>(s[0]));
                    tmem_load32(addr + 32, reinterpret_cast<uint32_t(&)[32]>(s[32]));
                    tmem_wait_load();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s_empty[t][own & 3]);
                    const uint64_t scale = pair(p.scale_log2, p.scale_log2);
                    uint64_t sum[4] = {0, 0, 0, 0};
                    bool all = j >= whole0 && j < whole1, any = true;  // of this warp's positions
                    int lo = 0, hi = 0;
                    if (!all) {
                        // columns whose tokens see this position
                        const int key = it.k0 + t * kKeyTile + row, q0 = from + j * per_tile, L = it.L;
                        lo = min(ROWS, max(0, key - q0) << shift) - half * kCols;
                        const int64_t end = key < p.sink ? (int64_t)L : min((int64_t)L, (int64_t)key + p.recent);
                        hi = ((int)max((int64_t)0, min((int64_t)per_tile, end - q0)) << shift) - half * kCols;
                        all = __all_sync(0xffffffffu, lo <= 0 && hi >= kCols);
                        any = __any_sync(0xffffffffu, max(lo, 0) < min(hi, kCols));
                    }
                    if (all) add_columns<kCols, true>(s, lse, scale, 0, 0, sum);
                    else if (any) add_columns<kCols, false>(s, lse, scale, lo, hi, sum);
                    acc += total(sum);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&empty[slot]);
                }
                if (!fine) break;
                // (the next item's sums cannot come before this one's have been read: its products need K of all warps)
                if (half == 1) {
                    s_part[t * kKeyTile + row] = acc;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&part_full[t]);
                } else {
                    fine = tc_wait(&part_full[t], mine & 1);
                    if (!fine) break;
                    acc += s_part[t * kKeyTile + row];
                }
                ++mine;
            }
            const int key = it.k0 + t * kKeyTile + row;
            if (half == 0 && key < min(it.k0 + kMassKeys, it.L) && !bad) {
                float *mass = w.mass + ((int64_t)it.r * p.hkv + it.kvh) * w.stride + key;
                if (parts == 1) *mass = old + acc;
                else to = mass;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_read[i & 1]);
        }
    }
    if (!fine && lane == 0) report(p.dev_status, SFI_DEV_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == kLongWarps + 1) tmem_free(tmem, T::kColumns);
    cluster_wait();  // every CTA of the cluster has begun
    if (parts > 1) {
        // the first CTA adds the others' sums to its own, in their order
        const int i = (int)threadIdx.x & (kMassKeys - 1);
        if (rank > 0 && warp < kLongWarps / 2) st_cluster_f32(cluster_map(smem_u32(&s_recv[rank - 1][i]), 0u), acc);
        const bool failed = __syncthreads_or(!fine || spoiled);
        if (rank > 0 && threadIdx.x == 0)
            st_cluster_f32(cluster_map(smem_u32(&s_failed[rank - 1]), 0u), failed ? 1.f : 0.f);
        cluster_sync();
        if (rank > 0 || failed || to == nullptr) return;
        for (int c = 0; c < parts - 1; ++c) {
            if (s_failed[c] != 0.f) return;
            acc += s_recv[c][i];
        }
        *to = old + acc;
    }
}

// ---- short calls ---------------------------------------------------------------------------------
template <int D, int ROWS>
__global__ void __launch_bounds__(kShortThreads, 2)
    mass_short_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const WindowParams p, const MassParams w, int per_cta) {
    using T = ShortTile<D, ROWS>;
    constexpr int kStages = T::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *ring = smem + T::kRowBytes;
    __shared__ __align__(8) uint64_t q_full, full[kStages], empty[kStages];
    __shared__ __align__(8) uint64_t s_full[2], s_empty[2], products_end;
    __shared__ __align__(16) float s_lse[ROWS];  // -lse in log2 units
    __shared__ int s_bad[kStages];               // a page of the slot's tile is out of range
    __shared__ uint32_t s_tmem;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();
    grid_launch_dependents();
    const int kvh = blockIdx.y;
    const int r = p.req_ids ? p.req_ids[blockIdx.z] : (int)blockIdx.z;
    if (r < 0 || r >= p.reqs) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && kvh == 0) report(p.dev_status, SFI_DEV_BAD_INDEX);
        return;
    }
    const int L = p.seq_lens[r];
    const int n = p.new_lens ? p.new_lens[r] : p.tokens;
    if (n < 0 || n > p.tokens || L < n || L > p.max_pages * kSubTokens || L > w.stride) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && kvh == 0) report(p.dev_status, SFI_DEV_BAD_LEN);
        return;
    }
    const int tile0 = blockIdx.x * per_cta, tile1 = min((L + kKeyTile - 1) / kKeyTile, tile0 + per_cta);
    if (tile0 >= tile1) return;
    const int G = p.group, shift = __ffs(G) - 1;
    const int q0 = L - n;  // position of the first query token
    // whether any token sees any position of a tile
    auto seen = [&](int tile) {
        const int k0 = tile * kKeyTile, k1 = min(k0 + kKeyTile, L) - 1;
        const int64_t to = k0 < p.sink ? L - 1 : min((int64_t)L - 1, (int64_t)k1 + p.recent - 1);
        return n > 0 && to >= max(q0, k0);
    };
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        mbar_init(&q_full, 1);
        mbar_init(&products_end, 1);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], 4);
        }
        fence_barrier_init();
    }
    if (threadIdx.x < ROWS) {
        const int tok = threadIdx.x >> shift;
        s_lse[threadIdx.x] = tok < n ? w.lse[((int64_t)r * p.tokens + tok) * p.hq + (kvh << shift) + (threadIdx.x & (G - 1))] *
                                           -1.4426950408889634f
                                     : 0.f;
    }
    if (warp == kShortWarps + 1) tmem_alloc(&s_tmem, T::kColumns);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    bool fine = true;

    if (warp == kShortWarps) {
        if (lane == 0) {
            mbar_arrive_expect_tx(&q_full, T::kRowBytes);
#pragma unroll
            for (int h = 0; h < T::kHalves; ++h)
                tma_tile_3d(smem + h * T::kRowHalf, &tm_q, h * 64, kvh << shift, r * p.tokens, &q_full);
        }
        const int32_t *ptab = p.page_table + (int64_t)r * p.max_pages;
        const int last_page = (L - 1) / kSubTokens;
        auto page_of = [&](int tile) -> int {
            const int v = tile * (kKeyTile / kSubTokens) + (lane & 7);
            return tile < tile1 && v <= last_page ? ptab[v] : -1;
        };
        int next = page_of(tile0), use = 0;
        for (int tile = tile0; tile < tile1; ++tile) {
            const int page = next;
            next = page_of(tile + 1);
            if (!seen(tile)) continue;
            const int slot = use % kStages;
            if (use >= kStages && !tc_wait(&empty[slot], (use / kStages - 1) & 1)) {
                fine = false;
                break;
            }
            ++use;
            const bool listed = tile * (kKeyTile / kSubTokens) + (lane & 7) <= last_page;
            const bool ok = page >= 0 && page < p.num_pages;
            const bool bad = __any_sync(0xffffffffu, listed && !ok);
            const uint32_t take = __ballot_sync(0xffffffffu, ok && lane < 8);
            if (lane == 0) {
                s_bad[slot] = bad;
                if (bad) report(p.dev_status, SFI_DEV_BAD_PAGE);
                if (take) mbar_arrive_expect_tx(&full[slot], __popc(take) * kSubTokens * D * 2);
                else mbar_arrive(&full[slot]);
            }
            __syncwarp();
            if (ok && lane < 8 * T::kHalves) {
                const int half = lane >> 3, at = lane & 7;
                tma_tile_2d(ring + slot * T::kKeyBytes + half * T::kKeyHalf + at * kSubTokens * 128, &tm_k, half * 64,
                            (page * p.hkv + kvh) * kSubTokens, &full[slot]);
            }
        }
        drain_ring(full, use);
        tc_wait(&q_full, 0);
    } else if (warp == kShortWarps + 1) {
        const uint32_t qa = smem_u32(smem), ra = smem_u32(ring);
        fine = tc_wait(&q_full, 0);
        int use = 0;
        for (int tile = tile0; tile < tile1 && fine; ++tile) {
            if (!seen(tile)) continue;
            const int slot = use % kStages, buf = use & 1;
            fine = tc_wait(&full[slot], (use / kStages) & 1) && (use < 2 || tc_wait(&s_empty[buf], (use / 2 - 1) & 1));
            if (!fine) break;
            tc_fence_after();
            if (lane == 0) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    mma_ss(tmem + buf * ROWS,
                           smem_desc(ra + slot * T::kKeyBytes + (ks >> 2) * T::kKeyHalf + (ks & 3) * 32, 16),
                           smem_desc(qa + (ks >> 2) * T::kRowHalf + (ks & 3) * 32, 16), T::kScores, ks > 0);
                mma_commit(&s_full[buf]);
            }
            __syncwarp();
            ++use;
        }
        if (lane == 0) drain_products(&products_end);
    } else {
        // ---- one position per thread; the warpgroups take the seen tiles in turn ----
        const int group = warp >> 2;
        const uint32_t addr = tmem + ((uint32_t)(warp & 3) << 21) + group * ROWS;
        float *mass = w.mass + ((int64_t)r * p.hkv + kvh) * w.stride;
        int use = 0;
        for (int tile = tile0; tile < tile1; ++tile) {
            const int k0 = tile * kKeyTile, k1 = min(k0 + kKeyTile, L) - 1;
            const int key = k0 + ((int)threadIdx.x & (kKeyTile - 1));
            const bool any = seen(tile);
            // (tiles that nobody sees are the first warpgroup's: they only decay)
            if (any ? (use++ & 1) != group : group != 0) continue;
            float old = 0.f;
            if (key < q0 && w.decay != 0.f) old = w.decay * mass[key];
            float sum = 0.f;
            bool bad = false;
            if (any) {
                const int at = use - 1, slot = at % kStages;
                fine = tc_wait(&full[slot], (at / kStages) & 1);
                if (!fine) break;
                bad = s_bad[slot] != 0;
                fine = tc_wait(&s_full[group], (at / 2) & 1);
                if (!fine) break;
                tc_fence_after();
                if (lane == 0) mbar_arrive(&empty[slot]);  // the tile has been multiplied
                const bool whole = (n << shift) == ROWS && k1 <= q0 && (k1 < p.sink || (int64_t)k0 > (int64_t)L - 1 - p.recent);
                if (whole) {
                    sum = sum_columns<ROWS, true>(addr, s_lse, p.scale_log2, 0, 0);
                } else {
                    const int64_t end = key < p.sink ? (int64_t)L : min((int64_t)L, (int64_t)key + p.recent);
                    const int lo = min(n, max(0, key - q0)) << shift;
                    const int hi = (int)max((int64_t)0, min((int64_t)n, end - q0)) << shift;
                    sum = sum_columns<ROWS, false>(addr, s_lse, p.scale_log2, lo, hi);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_empty[group]);
            }
            if (key <= k1 && !bad) mass[key] = old + sum;
        }
    }
    if (!fine && lane == 0) report(p.dev_status, SFI_DEV_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == kShortWarps + 1) tmem_free(tmem, T::kColumns);
}

namespace {

template <typename... Params, typename... Args>
cudaError_t launch_mass(void (*kernel)(Params...), int threads, int smem, std::atomic<uint64_t> &configured, dim3 grid,
                        int cluster, cudaStream_t stream, const Args &...args) {
    const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kernel), smem, configured);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// CTAs that share the query rows of 256 positions of a long call: more while the longest item would take well longer than
// an SM's part of all work, and a CTA has four steps at least. (One prompt of 4096 tokens, 2 KV heads: 256 us with one,
// 62 with eight; of 1024, 8 heads: 24 and 12 with four; four of 4096, 8/2/64 heads: 123 and 65 with two. But one of 8192
// with 8 heads, 32 x 8 items, the longest 1.2 times an SM's part: 131 and 152 with two, which begin anew for each item.)
int mass_parts(const WindowParams &p, int64_t units, int64_t blocks, int sms) {
    const int64_t per_tile = 128 / p.group;
    const int64_t longest = (std::min<int64_t>(p.tokens, p.sink > 0 ? p.tokens : (int64_t)p.recent + kMassKeys) + per_tile - 1) / per_tile;
    // (half of the longest for the blocks that hold new tokens)
    const int64_t steps = units * (blocks - std::min(blocks, ((int64_t)p.tokens + kMassKeys - 1) / kMassKeys) / 2) * longest;
    int parts = 1;
    while (parts < kMassMaxParts && longest >= 8 * parts && 2 * longest * sms > 3 * steps * parts) parts *= 2;
    return parts;
}

template <int D>
cudaError_t launch_long(const WindowMaps &maps, const WindowParams &p, const MassParams &w, int64_t most, int batch,
                        cudaStream_t stream) {
    static std::atomic<uint64_t> configured{0};
    const int sms = sm_count_current_device();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const int64_t units = (int64_t)batch * p.hkv, blocks = (most + kMassKeys - 1) / kMassKeys;
    const int parts = mass_parts(p, units, blocks, sms);
    return launch_mass(mass_long_kernel<D>, kLongThreads, LongTile<D>::kSmem, configured,
                       dim3((unsigned)(units * blocks * parts)), parts, stream, maps.q, maps.k, p, w, (int)units);
}

template <int D, int ROWS>
cudaError_t launch_short(const WindowMaps &maps, const WindowParams &p, const MassParams &w, int64_t most, int batch,
                         cudaStream_t stream) {
    static std::atomic<uint64_t> configured{0};
    const int sms = sm_count_current_device();
    if (sms <= 0) return cudaErrorInvalidDevice;
    // Runs of tiles: two CTAs for each place (two on an SM), so that ragged lengths even out; a run pays for its
    // CTA's start from a few tiles on (64 units of 128 tiles: 62 us with one, 52 with two, 56 with three, 58 with six).
    const int64_t tiles = (most + kKeyTile - 1) / kKeyTile, units = (int64_t)batch * p.hkv;
    const int64_t places = (int64_t)sms * 2 * 2;
    const int64_t per = std::max<int64_t>(1, (tiles * units + places - 1) / places);
    return launch_mass(mass_short_kernel<D, ROWS>, kShortThreads, ShortTile<D, ROWS>::kSmem, configured,
                       dim3((unsigned)((tiles + per - 1) / per), (unsigned)p.hkv, (unsigned)batch), 1,
                       stream, maps.q, maps.k, p, w, (int)per);
}

template <int D>
cudaError_t launch_rows(const WindowMaps &maps, const WindowParams &p, const MassParams &w, int64_t rows, int64_t most,
                        int batch, cudaStream_t stream) {
    if (rows > 128) return launch_long<D>(maps, p, w, most, batch, stream);
    switch (mass_rows(rows)) {
        case 16: return launch_short<D, 16>(maps, p, w, most, batch, stream);
        case 32: return launch_short<D, 32>(maps, p, w, most, batch, stream);
        case 64: return launch_short<D, 64>(maps, p, w, most, batch, stream);
        default: return launch_short<D, 128>(maps, p, w, most, batch, stream);
    }
}

}  // namespace

// Query rows of a tile: all of a short call's (16, 32, 64 or 128), or 128.
int mass_rows(int64_t rows) {
    int n = 16;
    while (n < 128 && n < rows) n *= 2;
    return n;
}

cudaError_t launch_attn_mass(const WindowMaps &maps, const WindowParams &p, const MassParams &w, int head_dim, int batch,
                             cudaStream_t stream) {
    const int64_t rows = (int64_t)p.tokens * p.group;
    const int64_t most = std::min<int64_t>((int64_t)p.max_pages * kSubTokens, w.stride);  // positions of a request
    return head_dim == 128 ? launch_rows<128>(maps, p, w, rows, most, batch, stream)
                           : launch_rows<64>(maps, p, w, rows, most, batch, stream);
}

}  // namespace sfi
