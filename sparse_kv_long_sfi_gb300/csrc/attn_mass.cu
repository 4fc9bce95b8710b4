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
//  * Long calls (over 128 query rows): a CTA takes 256 positions of one KV head as two tiles of 128 and walks
//    the query rows that see any of them (row = token * G + head) in tiles of 128. The K rows stay in tensor
//    memory as the A operand (each thread brings half of its own position's row there), so the products read
//    the query rows alone from shared memory, at the rate of the tensor cores; with K in shared memory too
//    they took 82 cycles instead of 64. Three buffers of S^T are used in turn; sums are fp32, eight of them
//    per position and tile.
//  * Short calls: the query rows (16, 32, 64 or 128 of them) stay in shared memory, and a CTA walks a run of
//    tiles of 128 positions through a ring; two warpgroups take the tiles in turn.
// A prompt of 8192 tokens, 16/8/128 heads: 135 us (54% of the measured bf16 rate).
// The last 64 tokens of 8 x 16384, 16/8/128 heads: 52 us (80% of the measured copy
// bandwidth).
#include <algorithm>
#include <atomic>

#include "tensor_core.cuh"
#include "window_span.cuh"

namespace sfi {

namespace {

constexpr int kLongThreads = 608;   // four warpgroups of sums, a copy warp, two matrix warps
constexpr int kLongWarps = 16;
constexpr int kShortThreads = 320;  // two warpgroups of sums, a copy warp, a matrix warp
constexpr int kShortWarps = 8;
constexpr int kMassKeys = 256;     // positions of a CTA
constexpr int kKeyTile = 128;

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
    static constexpr int kStages = 4;   // of query rows
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
        const int at = c / kLoad & 1;
        tmem_wait_load();
        if (c + kLoad < COLS) load(c + kLoad, s[at ^ 1]);  // on their way while these are summed
#pragma unroll
        for (int i = 0; i < kLoad; i += 4) {
            const float4 e = *reinterpret_cast<const float4 *>(&lse[c + i]);
            const float2 x = unpair(fma2(pair(__uint_as_float(s[at][i]), __uint_as_float(s[at][i + 1])), scale, pair(e.x, e.y)));
            const float2 y = unpair(fma2(pair(__uint_as_float(s[at][i + 2]), __uint_as_float(s[at][i + 3])), scale, pair(e.z, e.w)));
            float v[4] = {fast_exp2(x.x), fast_exp2(x.y), fast_exp2(y.x), fast_exp2(y.y)};
            if (!WHOLE) {
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = c + i + k >= lo && c + i + k < hi ? v[k] : 0.f;
            }
            sum[(i >> 1) & 3] = add2(sum[(i >> 1) & 3], pair(v[0], v[1]));
            sum[((i >> 1) & 3) + 1] = add2(sum[((i >> 1) & 3) + 1], pair(v[2], v[3]));
        }
    }
    const float2 both = unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
    return both.x + both.y;
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kLongThreads, 1)
    mass_long_kernel(const __grid_constant__ CUtensorMap tm_q, const WindowParams p, const MassParams w,
                     int units) {
    using T = LongTile<D>;
    constexpr int ROWS = T::kRows;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ __align__(8) uint64_t k_full, full[T::kStages], empty[T::kStages];
    __shared__ __align__(8) uint64_t s_full[T::kBuffers], s_empty[T::kBuffers];
    __shared__ __align__(16) float s_lse[T::kStages][ROWS];  // -lse in log2 units
    __shared__ float s_part[kMassKeys];                      // sums over the second half of the columns
    __shared__ uint32_t s_tmem;
    __shared__ int s_bad;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();
    grid_launch_dependents();
    // (the blocks with the most query rows, the first of every request and head, first)
    const int block = (int)blockIdx.x / units, unit = (int)blockIdx.x - block * units;
    const int b = unit / p.hkv, kvh = unit - b * p.hkv;
    const int r = p.req_ids ? p.req_ids[b] : b;
    if (r < 0 || r >= p.reqs) {
        if (threadIdx.x == 0 && block == 0 && kvh == 0) report(p.dev_status, SFI_DEV_BAD_INDEX);
        return;
    }
    const int L = p.seq_lens[r];
    const int n = p.new_lens ? p.new_lens[r] : p.tokens;
    if (n < 0 || n > p.tokens || L < n || L > p.max_pages * kSubTokens || L > w.stride) {
        if (threadIdx.x == 0 && block == 0 && kvh == 0) report(p.dev_status, SFI_DEV_BAD_LEN);
        return;
    }
    const int k0 = block * kMassKeys;
    if (k0 >= L) return;
    const int k1 = min(k0 + kMassKeys, L) - 1;
    const int G = p.group, shift = __ffs(G) - 1, per_tile = ROWS >> shift;
    // tokens that see any of these positions, in whole tiles counted from the first of them
    const int from = max(L - n, k0);
    const int to = k0 < p.sink ? L - 1 : (int)min((int64_t)L - 1, (int64_t)k1 + p.recent - 1);
    const int steps = n > 0 && to >= from ? (to - from) / per_tile + 1 : 0;
    const int tiles = k1 - k0 >= kKeyTile ? 2 : 1;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tm_q);
        mbar_init(&k_full, kLongWarps * 32);
        for (int i = 0; i < T::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], tiles * kLongWarps / 2);
        }
        for (int i = 0; i < T::kBuffers; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], kLongWarps / 2);
        }
        s_bad = 0;
        fence_barrier_init();
    }
    if (warp == kLongWarps + 1) tmem_alloc(&s_tmem, T::kColumns);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    bool fine = true;
    float acc = 0.f, old = 0.f;
    const int key = k0 + ((int)threadIdx.x & (kMassKeys - 1));  // of the first 512 threads
    float *mass = w.mass + ((int64_t)r * p.hkv + kvh) * w.stride;

    if (warp == kLongWarps) {
        if (steps > 0) {
            // this lane's rows of the next tile: their log-sum-exps are fetched a step ahead
            const float *lse = w.lse + (int64_t)r * p.tokens * p.hq + (kvh << shift);
            float next[ROWS / 32];
            auto fetch = [&](int j) {
#pragma unroll
                for (int k = 0; k < ROWS / 32; ++k) {
                    const int i = k * 32 + lane, tok = from - (L - n) + j * per_tile + (i >> shift);
                    next[k] = j < steps && tok < n ? lse[(int64_t)tok * p.hq + (i & (G - 1))] * -1.4426950408889634f : 0.f;
                }
            };
            fetch(0);
            for (int j = 0; j < steps; ++j) {
                const int slot = j % T::kStages;
                if (j >= T::kStages && !tc_wait(&empty[slot], (j / T::kStages - 1) & 1)) {
                    fine = false;
                    break;
                }
                const int tok0 = from - (L - n) + j * per_tile;
#pragma unroll
                for (int k = 0; k < ROWS / 32; ++k) s_lse[slot][k * 32 + lane] = next[k];
                fetch(j + 1);
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full[slot], T::kRowBytes);
#pragma unroll
                    for (int h = 0; h < T::kHalves; ++h)
                        tma_tile_3d(ring + slot * T::kRowBytes + h * T::kRowHalf, &tm_q, h * 64, kvh << shift,
                                    r * p.tokens + tok0, &full[slot]);
                }
                __syncwarp();
            }
        }
    } else if (warp > kLongWarps) {
        // one thread for each of the two tiles (see tc_wait_one)
        const int t = warp - kLongWarps - 1;
        if (lane == 0 && t < tiles && steps > 0) {
            const uint32_t ra = smem_u32(ring);
            fine = tc_wait_one(&k_full, 0);
            for (int j = 0; j < steps && fine; ++j) {
                const int slot = j % T::kStages, use = j * tiles + t, buf = use % T::kBuffers;
                fine = tc_wait_one(&full[slot], (j / T::kStages) & 1) &&
                       (use < T::kBuffers || tc_wait_one(&s_empty[buf], (use / T::kBuffers - 1) & 1));
                if (!fine) break;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    mma_ts(tmem + T::kScoresAt + buf * ROWS, tmem + t * 64 + ks * 8,
                           smem_desc(ra + slot * T::kRowBytes + (ks >> 2) * T::kRowHalf + (ks & 3) * 32, 16), T::kScores,
                           ks > 0);
                mma_commit(&s_full[buf]);
            }
        }
    } else {
        // ---- one position per thread, half of the columns each: four warps of every scheduler hide what the
        // reads of tensor memory, exponentials and hand-overs of one leave open ----
        constexpr int kCols = ROWS / 2;
        const int t = (warp >> 2) & 1, half = warp >> 3;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
        if (steps > 0) {
            // half of this position's K row
            const int page = key <= k1 ? p.page_table[(int64_t)r * p.max_pages + key / kSubTokens] : 0;
            const bool ok = page >= 0 && page < p.num_pages;
            if (!ok) {
                if (key % kSubTokens == 0 && half == 0) report(p.dev_status, SFI_DEV_BAD_PAGE);
                s_bad = 1;  // nothing of this CTA's positions is written
            }
            const __nv_bfloat16 *row = p.k_pool + (((int64_t)page * p.hkv + kvh) * kSubTokens + key % kSubTokens) * D + half * (D / 2);
            uint32_t x[D / 4];
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const int4 v = ok && key <= k1 ? ld_stream_v4(row + i * 8) : make_int4(0, 0, 0, 0);
                x[4 * i] = (uint32_t)v.x;
                x[4 * i + 1] = (uint32_t)v.y;
                x[4 * i + 2] = (uint32_t)v.z;
                x[4 * i + 3] = (uint32_t)v.w;
            }
            if constexpr (D == 128) tmem_store32(lanes + t * 64 + half * 32, x);
            else tmem_store16(lanes + t * 64 + half * 16, x);
            tmem_wait_store();
            tc_fence_before();
            mbar_arrive(&k_full);
        }
        if (half == 0 && key < L - n && w.decay != 0.f) old = w.decay * mass[key];
        const int tile0 = k0 + t * kKeyTile, tile1 = min(tile0 + kKeyTile - 1, k1);
        for (int j = 0; j < (t < tiles ? steps : 0); ++j) {
            const int slot = j % T::kStages, use = j * tiles + t, buf = use % T::kBuffers;
            fine = tc_wait(&full[slot], (j / T::kStages) & 1) && tc_wait(&s_full[buf], (use / T::kBuffers) & 1);
            if (!fine) break;
            tc_fence_after();
            const int q0 = from + j * per_tile, q1 = q0 + per_tile - 1;  // positions of the tile's tokens
            const bool whole = q1 < L && tile1 <= q0 && (tile1 < p.sink || (int64_t)tile0 > (int64_t)q1 - p.recent);
            // columns whose tokens see this position
            int lo = 0, hi = ROWS;
            if (!whole) {
                lo = min(ROWS, max(0, key - q0) << shift);
                const int64_t end = key < p.sink ? (int64_t)L : min((int64_t)L, (int64_t)key + p.recent);
                hi = (int)max((int64_t)0, min((int64_t)per_tile, end - q0)) << shift;
            }
            const uint32_t addr = lanes + T::kScoresAt + buf * ROWS + half * kCols;
            const float *lse = s_lse[slot] + half * kCols;
            if (whole) acc += sum_columns<kCols, true>(addr, lse, p.scale_log2, 0, 0);
            else acc += sum_columns<kCols, false>(addr, lse, p.scale_log2, lo - half * kCols, hi - half * kCols);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&s_empty[buf]);
                mbar_arrive(&empty[slot]);
            }
        }
    }
    if (!fine && lane == 0) {
        report(p.dev_status, SFI_DEV_TIMEOUT);
        s_bad = 1;
    }
    if (warp >= kLongWarps / 2 && warp < kLongWarps) s_part[key - k0] = acc;
    tc_fence_before();
    __syncthreads();
    if (warp == kLongWarps + 1) tmem_free(tmem, T::kColumns);
    if (warp < kLongWarps / 2 && key <= k1 && s_bad == 0) mass[key] = old + (acc + s_part[key - k0]);
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
    __shared__ __align__(8) uint64_t s_full[2], s_empty[2];
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
                        cudaStream_t stream, const Args &...args) {
    const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kernel), smem, configured);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D>
cudaError_t launch_long(const WindowMaps &maps, const WindowParams &p, const MassParams &w, int64_t most, int batch,
                        cudaStream_t stream) {
    static std::atomic<uint64_t> configured{0};
    const int64_t units = (int64_t)batch * p.hkv;
    return launch_mass(mass_long_kernel<D>, kLongThreads, LongTile<D>::kSmem, configured,
                       dim3((unsigned)(units * ((most + kMassKeys - 1) / kMassKeys))), stream, maps.q, p, w, (int)units);
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
                       dim3((unsigned)((tiles + per - 1) / per), (unsigned)p.hkv, (unsigned)batch), stream, maps.q,
                       maps.k, p, w, (int)per);
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
