// Attention of prompts (and of any chunk of more than 16 query rows per KV head) over the paged cache,
// through a sliding window with sinks.
//
// x = scale q . k over the positions that a token sees, out = sum exp(x - max) v / sum exp(x - max), in
// one pass over the keys with a running maximum and sum per row.
//
// Bound by the tensor cores: 4 D flops for each pair of a query row and a position. A CTA takes 256
// query rows of one KV head (row = token * G + head, so a group's heads share every key) as two tiles
// of 128, and walks the visible keys in tiles of 128:
//  * S = Q K^T and O += P V are tcgen05.mma with M = 128. S and O of both tiles live in tensor memory
//    (4 x 128 columns); P goes back there in bf16 over its own S and is the A operand of the second
//    product, so neither passes through shared memory.
//  * Four warps per tile hold one row per thread: maxima and sums need no shuffle. While one tile's
//    softmax runs, the tensor cores work for the other tile.
//  * The running maximum moves only when a score passes it by 2^8 (weights up to 2^8 lose nothing in
//    bf16 or fp32), so O is hardly ever rescaled; that is done by the softmax threads themselves.
//  * One warp fetches Q, K and V, page by page, by TMA with the 128-byte swizzle, K and V into a ring of
//    tiles; a thread per tile issues its matrix instructions.
//  * A CTA that is nearly done takes over one that has not begun (cluster launch control), so that the next
//    item's Q and first keys are on their way, and its first scores formed, while the last rows are written.
//    (Taken when an item begins, the longest had others behind them: ragged chunks 267 us instead of 245.)
// P is rounded to bf16 for the second product (2^-8 of each weight at most, which averages out over
// the keys); sums of P are taken before that, in fp32.
//
// A zero weight times a NaN is a NaN in a matrix product, so V's rows behind the last position (stale
// bytes of a page's tail) are zeroed in shared memory, and a row whose output is not finite, because of what
// it does not see, is computed again from the positions it sees alone (mend_rows).
// 16/8/128 heads: two prompts of 8192 tokens with window 1024 139 us (53% of the measured bf16 rate: 1280 keys are
// multiplied for 1088 that are seen, and a CTA's first and last steps are masked), one causal prompt of 8192 206 us (71%);
// 32/8/128 heads, 16384 tokens: 1.47 ms (80%). In the loop a step of 256 rows x 128 keys takes 3080 cycles, its 32
// products nominally 2048 of them. A NaN of V that all rows of a prompt of 8192 see: 230 us; one that all but its last
// token do not see: 6.1 ms, for the rows of that one block.
#include <algorithm>
#include <atomic>

#include "tensor_core.cuh"
#include "window_span.cuh"

namespace sfi {

namespace {

constexpr int kPromptThreads = 384;  // two softmax warpgroups; in the third:
constexpr int kCopyWarp = 8, kMmaWarp = 9, kItemWarp = 11;  // (a matrix warp for each tile: 9 and 10)
// Registers of a thread: the launch gives 168 (384 x 168 = 64512 of the SM's 65536), the softmax threads take what
// the third warpgroup gives back: 256 x 208 + 128 x 80 = 63488. (With 168 the softmax spills.)
constexpr int kSoftmaxRegs = 208, kOtherRegs = 80;
constexpr int kTileRows = 128;       // query rows of a tile, keys of a step
constexpr int kTilePages = kTileRows / kSubTokens;
constexpr float kGrowth = 8.f;       // the running maximum moves when a score passes it by this (log2)
constexpr uint32_t kTmemColumns = 512;
constexpr int64_t kTogether = 16 << 20, kTailTogether = 48 << 20;
constexpr int kTailWaves = 3;
constexpr int kAhead = 2;  // steps of an item that are left to load when the next is taken
constexpr int kItemReaders = 8 + 3;  // softmax warps, the copy warp, the matrix threads

template <int D>
struct PromptTile {
    static constexpr int kHalves = D / 64;               // 128-byte columns of a row
    static constexpr int kHalfBytes = kTileRows * 128;
    static constexpr int kBytes = kHalves * kHalfBytes;  // a tile of 128 rows
    static constexpr int kStages = D == 128 ? 5 : 8;     // what shared memory holds beside Q
    static constexpr int kSmem = (2 + kStages) * kBytes + 1024;
    static constexpr uint32_t kScores = mma_desc(kTileRows, kTileRows, false);
    static constexpr uint32_t kValues = mma_desc(kTileRows, D, true);
};

// 256 query rows of one (request, KV head): tokens tok0 .. of its n new ones. kvh < 0: there is none left.
struct PromptItem {
    int kvh, r, L, n, tok0;
};

// What all roles derive of an item.
struct PromptWork {
    int p0, p1, tiles;  // positions of the first and last token; tiles of query rows
    WindowSpan span;
    int steps;
    __device__ __forceinline__ PromptWork(const PromptItem &it, const WindowParams &p, int per_tile)
        : p0(it.L - it.n + it.tok0), p1(it.L - it.n + min(it.n, it.tok0 + 2 * per_tile) - 1),
          tiles(min(it.n, it.tok0 + 2 * per_tile) - it.tok0 > per_tile ? 2 : 1), span(p0, p1, p.sink, p.recent),
          steps((span.pages + kTilePages - 1) / kTilePages) {}
};

// The order of the items: units (request, KV head) in groups of `group`, and the units from `tail` on in one; in a group
// the tiles with the most keys of every unit first.
struct PromptOrder {
    int units, group, tail, tiles;
};

}  // namespace

template <int D>
__global__ void __launch_bounds__(kPromptThreads, 1)
    window_prompt_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ WindowParams p,
                         const PromptOrder order) {
    using T = PromptTile<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *ring = smem + 2 * T::kBytes;
    __shared__ __align__(16) uint4 s_answer;
    __shared__ __align__(8) uint64_t answered, item_full[2], item_read[2];
    __shared__ __align__(8) uint64_t q_full[2], q_free, loads_done, near_end, tail_ready, tail_done[2];
    __shared__ __align__(8) uint64_t full[T::kStages], empty[T::kStages];
    __shared__ __align__(8) uint64_t s_full[2], p_ready[2][2], o_done[2], turn[2], products_end[2];
    __shared__ PromptItem s_item[2], s_mine[8];  // s_mine: of each softmax warp, for what hardly ever happens at its end
    __shared__ uint32_t s_tmem;
    __shared__ int s_bad[2];  // of an item (even, odd): it writes no output
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        mbar_init(&answered, 1);
        mbar_init(&q_free, 8);
        mbar_init(&loads_done, 1);
        mbar_init(&near_end, 1);
        mbar_init(&tail_ready, 1);
        for (int i = 0; i < T::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&item_full[i], 1);
            mbar_init(&item_read[i], kItemReaders);
            mbar_init(&q_full[i], 1);
            mbar_init(&tail_done[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_ready[i][0], kTileRows);
            mbar_init(&p_ready[i][1], kTileRows);
            mbar_init(&o_done[i], 1);
            mbar_init(&turn[i], 1);
            mbar_init(&products_end[i], 1);
        }
        fence_barrier_init();
    }
    if (warp == kMmaWarp) tmem_alloc(&s_tmem, kTmemColumns);
    grid_dependency_wait();
    grid_launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const int G = p.group, shift = __ffs(G) - 1, per_tile = kTileRows >> shift;  // G is a power of two

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kCopyWarp) {
            // ---- Q, then K and V tile by tile ----
            int use = 0, loaded = 0, pairs = 0;  // tiles of K and V, items with any, and with two tiles of Q
            bool fine = true;
            for (int i = 0; fine; ++i) {
                fine = tc_wait(&item_full[i & 1], (i >> 1) & 1);
                if (!fine) break;
                const PromptItem it = s_item[i & 1];
                __syncwarp();
                if (lane == 0) mbar_arrive(&item_read[i & 1]);
                if (it.kvh < 0) break;
                const PromptWork w(it, p, per_tile);
                if (w.steps == 0) continue;
                // (an item's scores are all formed then, and its page errors read)
                fine = loaded == 0 || tc_wait(&q_free, (loaded - 1) & 1);
                if (!fine) break;
                pairs += w.tiles == 2;
                if (lane == 0) {
                    s_bad[loaded & 1] = 0;
                    for (int t = 0; t < w.tiles; ++t) {
                        mbar_arrive_expect_tx(&q_full[t], T::kBytes);
                        for (int h = 0; h < T::kHalves; ++h)
                            tma_tile_3d(smem + t * T::kBytes + h * T::kHalfBytes, &tm_q, h * 64, it.kvh * G,
                                        it.r * p.tokens + it.tok0 + t * per_tile, &q_full[t]);
                    }
                }
                __syncwarp();
                ++loaded;
                const int32_t *ptab = p.page_table + (int64_t)it.r * p.max_pages;
                auto page_of = [&](int step) -> int {
                    const int v = step * kTilePages + (lane & 7);
                    return v < w.span.pages ? ptab[w.span.page(v)] : -1;
                };
                int next = page_of(0);
                for (int j = 0; j < w.steps && fine; ++j) {
                    if (lane == 0 && j == max(0, w.steps - kAhead)) mbar_arrive(&near_end);
                    const int page = next;
                    next = j + 1 < w.steps ? page_of(j + 1) : -1;
                    const bool listed = j * kTilePages + (lane & 7) < w.span.pages;
                    const bool ok = page >= 0 && page < p.num_pages;
                    const uint32_t take = __ballot_sync(0xffffffffu, ok && lane < kTilePages);
                    if (listed && !ok && lane < kTilePages) {
                        report(p.dev_status, SFI_DEV_BAD_PAGE);
                        s_bad[(loaded - 1) & 1] = 1;
                    }
                    for (int kv = 0; kv < 2; ++kv, ++use) {
                        const int slot = use % T::kStages;
                        fine = use < T::kStages || tc_wait(&empty[slot], (use / T::kStages - 1) & 1);
                        if (!fine) break;
                        if (lane == 0) {
                            const uint32_t bytes = __popc(take) * kSubTokens * D * 2;
                            if (bytes) mbar_arrive_expect_tx(&full[slot], bytes);
                            else mbar_arrive(&full[slot]);
                        }
                        __syncwarp();
                        if (ok && lane < kTilePages * T::kHalves) {
                            const int half = lane / kTilePages, at = lane % kTilePages;
                            tma_tile_2d(ring + slot * T::kBytes + half * T::kHalfBytes + at * kSubTokens * 128,
                                        kv ? &tm_v : &tm_k, half * 64, (page * p.hkv + it.kvh) * kSubTokens, &full[slot]);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0 && fine) mbar_arrive(&loads_done);  // s_bad of this item is final
            }
            if (!fine && lane == 0) report(p.dev_status, SFI_DEV_TIMEOUT);
            drain_ring(full, use);
            if (loaded > 0) tc_wait(&q_full[0], (loaded - 1) & 1);
            if (pairs > 0) tc_wait(&q_full[1], (pairs - 1) & 1);
        } else if ((warp == kMmaWarp || warp == kMmaWarp + 1) && lane == 0) {
            // ---- a tile's matrix instructions: S(0), then PV(j) and S(j + 1) ----
            // A thread issues 8 of them in the time that they take, so what it waits for and signals in between has to
            // run beside the other tile's: hence a thread for each, and one signal (commit) per step. That of S(j + 1)
            // says that PV(j) is done too, since they run in the order of their issue.
            const int t = warp - kMmaWarp;
            const uint32_t qa = smem_u32(smem) + t * T::kBytes, ra = smem_u32(ring);
            auto scores = [&](int slot) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t off = (ks >> 2) * T::kHalfBytes + (ks & 3) * 32;
                    mma_ss(tmem + t * kTileRows, smem_desc(qa + off, 16), smem_desc(ra + slot * T::kBytes + off, 16),
                           T::kScores, ks > 0);
                }
                mma_commit(&s_full[t]);
            };
            auto arrived = [&](int use) { return tc_wait_one(&full[use % T::kStages], (use / T::kStages) & 1); };
            // uses of the ring, and this tile's items, steps and turns so far
            int base = 0, mine = 0, step = 0, phase = 0;
            bool fine = true;
            for (int i = 0; fine; ++i) {
                fine = tc_wait_one(&item_full[i & 1], (i >> 1) & 1);
                if (!fine) break;
                const PromptItem it = s_item[i & 1];
                mbar_arrive(&item_read[i & 1]);
                if (it.kvh < 0) break;
                const PromptWork w(it, p, per_tile);
                if (w.steps == 0) continue;
                const int first = base;
                base += 2 * w.steps;
                if (t >= w.tiles) continue;
                const int own = mine++;
                // With two tiles the threads take turns: interleaved, both tiles' instructions would end together, and
                // both softmaxes would run while the tensor cores wait (a step then took 4400 cycles instead of 3000).
                auto my_turn = [&]() {
                    if (w.tiles == 1) return true;
                    const int k = phase++;
                    return (t == 0 && k == 0) || tc_wait_one(&turn[t], (k - (t == 0)) & 1);
                };
                auto hand_over = [&]() {
                    if (w.tiles == 2) mbar_arrive(&turn[t ^ 1]);
                };
                // K of step j is use first + 2 j of the ring, V the one behind it
                fine = tc_wait_one(&q_full[t], own & 1) && arrived(first) && my_turn();
                if (!fine) break;
                tc_fence_after();
                scores(first % T::kStages);
                hand_over();
                fine = arrived(first + 1);
                for (int j = 0; j < w.steps && fine; ++j, ++step) {
                    const int slot_v = (first + 2 * j + 1) % T::kStages;
                    const bool more = j + 1 < w.steps;
                    if (more) {
                        fine = arrived(first + 2 * j + 2);
                    } else {
                        if (t == 0) mbar_arrive(&tail_ready);  // V's last tile is there
                        // (a barrier for each tile: an item of one tile could go by meanwhile, and a phase of a common
                        // one with it, whose parity this thread would then wait for in vain)
                        fine = tc_wait_one(&tail_done[t], own & 1);
                    }
                    fine = fine && tc_wait_one(&p_ready[t][0], step & 1) && my_turn();
                    if (!fine) break;
                    tc_fence_after();
                    auto values = [&](int ks0) {
#pragma unroll
                        for (int ks = ks0; ks < ks0 + kTileRows / 32; ++ks)
                            mma_ts(tmem + 2 * kTileRows + t * D, tmem + t * kTileRows + ks * 8,
                                   smem_desc(ra + slot_v * T::kBytes + ks * 16 * 128, T::kHalfBytes), T::kValues,
                                   j + ks > 0);
                    };
                    values(0);
                    fine = tc_wait_one(&p_ready[t][1], step & 1);
                    if (!fine) break;
                    tc_fence_after();
                    values(kTileRows / 32);
                    if (more) {
                        scores((first + 2 * j + 2) % T::kStages);
                        hand_over();
                        fine = arrived(first + 2 * j + 3);
                    } else {
                        mma_commit(&o_done[t]);
                        hand_over();
                    }
                }
            }
            if (!fine) report(p.dev_status, SFI_DEV_TIMEOUT);
            drain_products(&products_end[t]);
        } else if (warp == kItemWarp) {
            // ---- the items, and the tails of V ----
            bool fine = true, left = true;
            uint32_t x = blockIdx.x;
            int taken = 0, loaded = 0, tail_use = 0;
            // the item of CTA x, or of the next that has any work
            auto publish = [&](int i) {
                if (lane == 0) {
                    PromptItem it{-1, 0, 0, 0, 0};
                    while (left && it.kvh < 0) {
                        if (taken > 0) {
                            bool late = false;
                            left = take_next_cta(&s_answer, &answered, (taken - 1) & 1, x, late);
                            fine &= !late;
                            if (!left) break;
                        }
                        ++taken;
                        const bool in_tail = (int)x >= order.tail * order.tiles;
                        // units of earlier groups, and of this one
                        const int before = in_tail ? order.tail : (int)x / (order.group * order.tiles) * order.group;
                        const int size = in_tail ? order.units - before : min(order.group, order.tail - before);
                        const int at = (int)x - before * order.tiles, unit = before + at % size, tile = at / size;
                        const int b = unit / p.hkv, kvh = unit - b * p.hkv;
                        const int r = p.req_ids ? p.req_ids[b] : b;
                        const bool lead = kvh == 0 && tile == 0;
                        if (r < 0 || r >= p.reqs) {
                            if (lead) report(p.dev_status, SFI_DEV_BAD_INDEX);
                            continue;
                        }
                        const int L = p.seq_lens[r], n = p.new_lens ? p.new_lens[r] : p.tokens;
                        if (n < 0 || n > p.tokens || L < n || L > p.max_pages * kSubTokens) {
                            if (lead) report(p.dev_status, SFI_DEV_BAD_LEN);
                            continue;
                        }
                        const int tok0 = (order.tiles - 1 - tile) * 2 * per_tile;
                        if (tok0 < n) it = PromptItem{kvh, r, L, n, tok0};
                    }
                    if (i >= 2) fine &= tc_wait_one(&item_read[i & 1], ((i >> 1) - 1) & 1);
                    s_item[i & 1] = it;
                    mbar_arrive(&item_full[i & 1]);
                }
                __syncwarp();
                const PromptItem it = s_item[i & 1];
                return it;
            };
            PromptItem it = publish(0);
            for (int i = 0; it.kvh >= 0; ++i) {
                const PromptWork w(it, p, per_tile);
                // (not before this one is near its end: the longest should have none behind them)
                if (w.steps > 0) fine = tc_wait(&near_end, loaded & 1);
                if (!fine) break;
                const PromptItem next = publish(i + 1);
                if (__any_sync(0xffffffffu, !fine)) break;
                it = next;
                if (w.steps == 0) continue;
                // what lies behind the last position must not meet a zero weight as a NaN
                fine = tc_wait(&tail_ready, loaded & 1);
                if (!fine) break;
                ++loaded;
                // (the matrix threads are in step: this is the slot of the item's last V)
                tail_use += 2 * w.steps;
                const int slot = (tail_use - 1) % T::kStages;
                const int rows = max(0, w.span.slots - (w.steps - 1) * kTileRows);
                for (int c = rows * 8 + lane; c < kTileRows * 8; c += 32)
#pragma unroll
                    for (int h = 0; h < T::kHalves; ++h)
                        *reinterpret_cast<int4 *>(ring + slot * T::kBytes + h * T::kHalfBytes + c * 16) = make_int4(0, 0, 0, 0);
                fence_async_shared();
                __syncwarp();
                if (lane < w.tiles) mbar_arrive(&tail_done[lane]);
            }
            if (!fine) report(p.dev_status, SFI_DEV_TIMEOUT);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        // ---- softmax: one query row per thread ----
        const int t = warp >> 2;  // tile
        const int row = threadIdx.x & (kTileRows - 1);
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's 32 lanes
        const uint32_t s_addr = lanes + t * kTileRows, o_addr = lanes + 2 * kTileRows + t * D;
        const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
        int base = 0, loaded = 0, step = 0, outs = 0;  // uses of the ring, items with keys, steps, outputs so far
        bool fine = true;
        for (int i = 0; fine; ++i) {
            fine = tc_wait(&item_full[i & 1], (i >> 1) & 1);
            if (!fine) break;
            const PromptItem it = s_item[i & 1];
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&item_read[i & 1]);
                s_mine[warp] = it;
            }
            if (it.kvh < 0) break;
            const PromptWork w(it, p, per_tile);
            const int use0 = base, item = loaded;
            base += 2 * w.steps;
            loaded += w.steps > 0;
            if (t >= w.tiles) continue;
            const int token = it.tok0 + t * per_tile + (row >> shift), head = it.kvh * G + (row & (G - 1));
            const bool mine = token < it.n;  // rows behind the request's tokens are not written
            const int pos = it.L - it.n + token;
            const RowWindow win(mine ? pos : w.p1, p.sink, p.recent, w.span);
            // the first and the last token of this warp's rows: what both see needs no mask
            const int warp_tok = it.tok0 + t * per_tile + ((warp & 3) * 32 >> shift);
            const RowWindow first(min(it.L - it.n + warp_tok, w.p1), p.sink, p.recent, w.span);
            const RowWindow last(min(it.L - it.n + warp_tok + (31 >> shift), w.p1), p.sink, p.recent, w.span);
            // a slot of the ring is free for the copies when both tiles are done with it
            auto release = [&](uint64_t *bar) {
                if (row == 0) {
                    mbar_arrive(bar);
                    if (w.tiles == 1) mbar_arrive(bar);
                }
            };
            float m = -INFINITY, l = 0.f;
            bool bad = false;
            for (int j = 0; j < w.steps; ++j, ++step) {
                fine = tc_wait(&s_full[t], step & 1);
                if (!fine) break;
                tc_fence_after();
                release(&empty[(use0 + 2 * j) % T::kStages]);
                if (j > 0) release(&empty[(use0 + 2 * j - 1) % T::kStages]);
                if (j + 1 == w.steps) {
                    // all warps see the item's page errors before the copies go on to the next one
                    fine = tc_wait(&loads_done, item & 1);
                    if (!fine) break;
                    bad = s_bad[item & 1] != 0;
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&q_free);
                        if (w.tiles == 1) mbar_arrive(&q_free);
                    }
                }
                uint32_t s[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_load32(s_addr + c * 32, s[c]);
                tmem_wait_load();
                const int v0 = j * kTileRows;
                if (!all_see(v0, kTileRows, first, last)) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t see = win.sees32(v0 + c * 32);
                        if (!__all_sync(0xffffffffu, see == 0xffffffffu)) {
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (!((see >> k) & 1u)) s[c][k] = 0xff800000u;
                        }
                    }
                }
                float top[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    top[c] = fmaxf(__uint_as_float(s[c][0]), __uint_as_float(s[c][1]));
#pragma unroll
                    for (int k = 2; k < 32; k += 2)
                        top[c] = max3(top[c], __uint_as_float(s[c][k]), __uint_as_float(s[c][k + 1]));
                }
                const float now = fmaxf(max3(top[0], top[1], top[2]), top[3]) * p.scale_log2;
                const bool grow = now > m + kGrowth;
                float alpha = 1.f;
                if (grow) {
                    alpha = fast_exp2(m - now);
                    m = now;
                    l *= alpha;
                }
                if (j > 0 && __any_sync(0xffffffffu, grow)) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        tmem_load32(o_addr + c, o);
                        tmem_wait_load();
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                        tmem_store32(o_addr + c, o);
                    }
                }
                const float zero = m == -INFINITY ? 0.f : m;
                const uint64_t scale2 = pair(p.scale_log2, p.scale_log2), zero2 = pair(-zero, -zero);
                uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t e[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const uint32_t(&x)[32] = s[2 * c + k / 16];
                        const float2 d = unpair(fma2(
                            pair(__uint_as_float(x[2 * (k % 16)]), __uint_as_float(x[2 * (k % 16) + 1])), scale2, zero2));
                        const float a = fast_exp2(d.x), b = fast_exp2(d.y);
                        sum[k & 3] = add2(sum[k & 3], pair(a, b));
                        e[k] = pack_bf16x2(a, b);
                    }
                    tmem_store32(s_addr + c * 32, e);
                    tmem_wait_store();
                    tc_fence_before();
                    mbar_arrive(&p_ready[t][c]);
                }
                const float2 both = unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
                l += both.x + both.y;
            }
            // ---- the rows' output ----
            if (fine && w.steps > 0) {
                fine = tc_wait(&o_done[t], outs++ & 1);
                if (fine) release(&empty[(use0 + 2 * w.steps - 1) % T::kStages]);
            }
            if (!fine) break;
            tc_fence_after();
            const bool write = mine && !bad;
            const int64_t at = ((int64_t)it.r * p.tokens + token) * p.hq + head;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            // Straight from registers, 32 bytes of a row at a time (whole sectors): staged in shared memory whole lines
            // would leave together, but that room is worth more to the ring (a fifth tile: 321 -> 300 us for ragged
            // chunks, 226 -> 212 us for a prompt of 8192).
            __nv_bfloat16 *out = p.out + at * D;
            bool odd = false;
#pragma unroll 1
            for (int half = 0; half < T::kHalves; ++half) {
                uint32_t o[2][32];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (w.steps > 0) {
                        tmem_load32(o_addr + half * 64 + c * 32, o[c]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[c][k] = 0u;
                    }
                }
                tmem_wait_load();
                uint32_t big = 0;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) big = max(big, o[c][k] & 0x7fffffffu);
#pragma unroll
                    for (int k = 0; k < 32; k += 16) {
                        uint32_t v[8];
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            v[q] = pack_bf16x2(__uint_as_float(o[c][k + 2 * q]) * inv, __uint_as_float(o[c][k + 2 * q + 1]) * inv);
                        __nv_bfloat16 *to = out + half * 64 + c * 32 + k;
                        if (write && wide) {
                            st_v8(to, v);
                        } else if (write) {
                            st_v4(to, make_int4((int)v[0], (int)v[1], (int)v[2], (int)v[3]));
                            st_v4(to + 8, make_int4((int)v[4], (int)v[5], (int)v[6], (int)v[7]));
                        }
                    }
                }
                odd |= big >= 0x7f800000u;
            }
            if (write && p.lse) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
            if (__any_sync(0xffffffffu, odd && write)) {
                __syncwarp();
                const PromptItem own = s_mine[warp];
                const PromptWork all(own, p, per_tile);
                mend_rows<D, false>(p, own.r, own.kvh, own.L, own.n, all.p0, all.p1,
                             (own.tok0 << shift) + t * kTileRows + (warp & 3) * 32, odd && write, m, l, 0, 32 * (D / 4));
            }
            tc_fence_before();  // O has been read: the next item's first weights let it be overwritten
        }
        if (!fine && lane == 0) report(p.dev_status, SFI_DEV_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) tmem_free(tmem, kTmemColumns);
}

namespace {

template <int D>
cudaError_t launch_prompt(const WindowMaps &maps, const WindowParams &p, int batch, cudaStream_t stream) {
    auto kernel = window_prompt_kernel<D>;
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kernel), PromptTile<D>::kSmem, configured);
    if (e != cudaSuccess) return e;
    const int per_cta = 2 * kTileRows / p.group;
    const int tiles = (p.tokens + per_cta - 1) / per_cta;
    const int64_t units = (int64_t)batch * p.hkv, items = units * tiles;
    // A few units at a time keep their K and V in L2 (kTogether bytes at their longest), but the last of them would leave
    // long tiles to the end: the units with the last kTailWaves CTAs per SM (if L2 holds them) are one group.
    // As items are taken late this matters little: between groups of 1 and 64 MB and one and six waves a prompt of 8192
    // takes 204 to 210 us and ragged chunks 245 to 254; but 4 x 4096 tokens of 8/2/64 heads take 114 with one wave, 103
    // with two and 99 with three.
    const int64_t bytes = (int64_t)p.max_pages * kSubTokens * D * 4;
    const int sms = sm_count_current_device();
    const int group = (int)std::max<int64_t>(1, std::min(units, kTogether / bytes));
    const int64_t last = std::min<int64_t>((kTailWaves * sms + tiles - 1) / tiles, std::max<int64_t>(1, kTailTogether / bytes));
    const int tail = (int)std::max<int64_t>(0, units - last);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)items);
    cfg.blockDim = dim3(kPromptThreads);
    cfg.dynamicSmemBytes = PromptTile<D>::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, maps.q, maps.k, maps.v, p, PromptOrder{(int)units, group, tail, tiles});
}

}  // namespace

cudaError_t launch_window_prompt(const WindowMaps &maps, const WindowParams &p, int head_dim, int batch,
                                 cudaStream_t stream) {
    return head_dim == 128 ? launch_prompt<128>(maps, p, batch, stream) : launch_prompt<64>(maps, p, batch, stream);
}

}  // namespace sfi
