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
//  * One warp fetches K and V, page by page, by TMA with the 128-byte swizzle into a ring of tiles; one
//    thread issues all matrix instructions.
// P is rounded to bf16 for the second product (2^-9 of each weight at most, which averages out over
// the keys); sums of P are taken before that, in fp32.
//
// A zero weight times a NaN is a NaN in a matrix product, so V's rows behind the last position (stale
// bytes of a page's tail) are zeroed in shared memory, and a row whose output is not finite is computed
// again key by key, from the positions it sees alone.
// Two prompts of 8192 tokens, 16/8/128 heads, window 1024: 164 us (44% of the measured bf16 rate); in the loop a step of
// 256 rows x 128 keys takes 3080 cycles (84%), of 32000 of a CTA's 47000.
#include <atomic>

#include "tensor_core.cuh"
#include "window_span.cuh"

namespace sfi {

namespace {

constexpr int kPromptThreads = 384;  // two softmax warpgroups; a copy warp and a matrix warp in the third
constexpr int kCopyWarp = 8, kMmaWarp = 9, kTailWarp = 11;  // (a matrix warp for each tile: 9 and 10)
// Registers of a thread: the launch gives 168 (384 x 168 = 64512 of the SM's 65536), the softmax threads take what
// the third warpgroup gives back: 256 x 208 + 128 x 80 = 63488. (With 168 the softmax spills.)
constexpr int kSoftmaxRegs = 208, kOtherRegs = 80;
constexpr int kTileRows = 128;       // query rows of a tile, keys of a step
constexpr int kTilePages = kTileRows / kSubTokens;
constexpr float kGrowth = 8.f;       // the running maximum moves when a score passes it by this (log2)
constexpr uint32_t kTmemColumns = 512;

template <int D>
struct PromptTile {
    static constexpr int kHalves = D / 64;                 // 128-byte columns of a row
    static constexpr int kHalfBytes = kTileRows * 128;
    static constexpr int kBytes = kHalves * kHalfBytes;    // a tile of 128 rows
    static constexpr int kStages = D == 128 ? 5 : 8;       // what shared memory holds beside Q
    static constexpr int kSmem = (2 + kStages) * kBytes + 1024;
    static constexpr uint32_t kScores = mma_desc(kTileRows, kTileRows, false);
    static constexpr uint32_t kValues = mma_desc(kTileRows, D, true);
};

}  // namespace

template <int D>
__global__ void __launch_bounds__(kPromptThreads, 1)
    window_prompt_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ WindowParams p) {
    using T = PromptTile<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *ring = smem + 2 * T::kBytes;
    __shared__ __align__(8) uint64_t q_full, loads_done, tail_ready, tail_done;
    __shared__ __align__(8) uint64_t full[T::kStages], empty[T::kStages];
    __shared__ __align__(8) uint64_t s_full[2], p_ready[2][2], o_done[2], turn[2];
    __shared__ uint32_t s_tmem;
    __shared__ int s_bad;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();
    grid_launch_dependents();
    const int kvh = blockIdx.x;
    const int r = p.req_ids ? p.req_ids[blockIdx.y] : (int)blockIdx.y;
    if (r < 0 || r >= p.reqs) {
        if (threadIdx.x == 0 && blockIdx.z == 0 && kvh == 0) report(p.dev_status, SFI_DEV_BAD_INDEX);
        return;
    }
    const int L = p.seq_lens[r];
    const int n = p.new_lens ? p.new_lens[r] : p.tokens;
    if (n < 0 || n > p.tokens || L < n || L > p.max_pages * kSubTokens) {
        if (threadIdx.x == 0 && blockIdx.z == 0 && kvh == 0) report(p.dev_status, SFI_DEV_BAD_LEN);
        return;
    }
    // the tokens with the most keys first, those of every request and head
    const int G = p.group, shift = __ffs(G) - 1, per_tile = kTileRows >> shift;  // G is a power of two
    const int tok0 = ((int)gridDim.z - 1 - (int)blockIdx.z) * 2 * per_tile;
    if (tok0 >= n) return;
    const int tok1 = min(n, tok0 + 2 * per_tile) - 1;
    const int tiles_q = tok1 - tok0 >= per_tile ? 2 : 1;
    const int p0 = L - n + tok0, p1 = L - n + tok1;
    const WindowSpan span(p0, p1, p.sink, p.recent);
    const int steps = (span.pages + kTilePages - 1) / kTilePages;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        mbar_init(&q_full, 1);
        mbar_init(&loads_done, 1);
        mbar_init(&tail_ready, 1);
        mbar_init(&tail_done, 1);
        for (int i = 0; i < T::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], tiles_q);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_ready[i][0], kTileRows);
            mbar_init(&p_ready[i][1], kTileRows);
            mbar_init(&turn[i], 1);
            mbar_init(&o_done[i], 1);
        }
        s_bad = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) tmem_alloc(&s_tmem, kTmemColumns);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kCopyWarp) {
            // ---- Q, then K and V tile by tile ----
            if (lane == 0) {
                mbar_arrive_expect_tx(&q_full, tiles_q * T::kBytes);
                for (int t = 0; t < tiles_q; ++t)
                    for (int h = 0; h < T::kHalves; ++h)
                        tma_tile_3d(smem + t * T::kBytes + h * T::kHalfBytes, &tm_q, h * 64, kvh * G,
                                    r * p.tokens + tok0 + t * per_tile, &q_full);
            }
            const int32_t *ptab = p.page_table + (int64_t)r * p.max_pages;
            auto page_of = [&](int step) -> int {
                const int v = step * kTilePages + (lane & 7);
                return v < span.pages ? ptab[span.page(v)] : -1;
            };
            int next = page_of(0);
            bool late = false;
            for (int j = 0; j < steps && !late; ++j) {
                const int page = next;
                next = j + 1 < steps ? page_of(j + 1) : -1;
                const bool in_list = j * kTilePages + (lane & 7) < span.pages;
                const bool ok = page >= 0 && page < p.num_pages;
                const uint32_t take = __ballot_sync(0xffffffffu, ok && lane < kTilePages);
                if (in_list && !ok && lane < kTilePages) {
                    report(p.dev_status, SFI_DEV_BAD_PAGE);
                    s_bad = 1;  // the CTA writes no output
                }
                for (int kv = 0; kv < 2; ++kv) {
                    const int use = 2 * j + kv, slot = use % T::kStages;
                    if (use >= T::kStages && !tc_wait(&empty[slot], (use / T::kStages - 1) & 1)) {
                        late = true;
                        break;
                    }
                    if (lane == 0) {
                        const uint32_t bytes = __popc(take) * kSubTokens * D * 2;
                        if (bytes) mbar_arrive_expect_tx(&full[slot], bytes);
                        else mbar_arrive(&full[slot]);
                    }
                    __syncwarp();
                    if (ok && lane < kTilePages * T::kHalves) {
                        const int half = lane / kTilePages, at = lane % kTilePages;
                        tma_tile_2d(ring + slot * T::kBytes + half * T::kHalfBytes + at * kSubTokens * 128,
                                    kv ? &tm_v : &tm_k, half * 64, (page * p.hkv + kvh) * kSubTokens, &full[slot]);
                    }
                }
            }
            if (late && lane == 0) {
                report(p.dev_status, SFI_DEV_TIMEOUT);
                s_bad = 1;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&loads_done);  // s_bad is final
        } else if ((warp == kMmaWarp || warp == kMmaWarp + 1) && lane == 0 && warp - kMmaWarp < tiles_q && steps > 0) {
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
            // K of step j is use 2 j of the ring, V use 2 j + 1
            auto arrived = [&](int use) { return tc_wait_one(&full[use % T::kStages], (use / T::kStages) & 1); };
            // With two tiles the threads take turns: interleaved, both tiles' instructions would end together, and
            // both softmaxes would run while the tensor cores wait (a step then took 4400 cycles instead of 3000).
            auto my_turn = [&](int phase) {
                return tiles_q == 1 || (t == 0 && phase == 0) || tc_wait_one(&turn[t], (phase - (t == 0)) & 1);
            };
            bool fine = tc_wait_one(&q_full, 0) && arrived(0) && my_turn(0);
            if (fine) {
                tc_fence_after();
                scores(0);
                if (tiles_q == 2) mbar_arrive(&turn[t ^ 1]);
                fine = arrived(1);
            }
            for (int j = 0; j < steps && fine; ++j) {
                const int slot_v = (2 * j + 1) % T::kStages;
                const bool more = j + 1 < steps;
                if (more) {
                    fine = arrived(2 * j + 2);
                } else {
                    if (t == 0) mbar_arrive(&tail_ready);  // V's last tile is there
                    fine = tc_wait_one(&tail_done, 0);
                }
                fine = fine && tc_wait_one(&p_ready[t][0], j & 1) && my_turn(j + 1);
                if (!fine) break;
                tc_fence_after();
                auto values = [&](int ks0) {
#pragma unroll
                    for (int ks = ks0; ks < ks0 + kTileRows / 32; ++ks)
                        mma_ts(tmem + 2 * kTileRows + t * D, tmem + t * kTileRows + ks * 8,
                               smem_desc(ra + slot_v * T::kBytes + ks * 16 * 128, T::kHalfBytes), T::kValues, j + ks > 0);
                };
                values(0);
                fine = tc_wait_one(&p_ready[t][1], j & 1);
                if (!fine) break;
                tc_fence_after();
                values(kTileRows / 32);
                if (more) {
                    scores((2 * j + 2) % T::kStages);
                    if (tiles_q == 2) mbar_arrive(&turn[t ^ 1]);
                    fine = arrived(2 * j + 3);
                } else {
                    mma_commit(&o_done[t]);
                    if (tiles_q == 2 && t == 0) mbar_arrive(&turn[1]);
                }
            }
            if (!fine) report(p.dev_status, SFI_DEV_TIMEOUT);
        } else if (warp == kTailWarp && steps > 0) {
            // ---- what lies behind the last position must not meet a zero weight as a NaN ----
            const int slot = (2 * steps - 1) % T::kStages;
            if (tc_wait(&tail_ready, 0)) {
                const int rows = max(0, span.slots - (steps - 1) * kTileRows);
                for (int i = rows * 8 + lane; i < kTileRows * 8; i += 32)
#pragma unroll
                    for (int h = 0; h < T::kHalves; ++h)
                        *reinterpret_cast<int4 *>(ring + slot * T::kBytes + h * T::kHalfBytes + i * 16) = make_int4(0, 0, 0, 0);
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(&tail_done);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        // ---- softmax: one query row per thread ----
        const int t = warp >> 2;                      // tile
        const int row = threadIdx.x & (kTileRows - 1);
        const int token = tok0 + t * per_tile + (row >> shift), head = kvh * G + (row & (G - 1));
        const bool mine = token < n;                  // rows behind the request's tokens are not written
        const int pos = L - n + token;
        const RowWindow win(mine ? pos : p1, p.sink, p.recent, span);
        // the first and the last token of this warp's rows: what both see needs no mask
        const int warp_tok = tok0 + t * per_tile + ((warp & 3) * 32 >> shift);
        const RowWindow first(min(L - n + warp_tok, p1), p.sink, p.recent, span);
        const RowWindow last(min(L - n + warp_tok + (31 >> shift), p1), p.sink, p.recent, span);
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's 32 lanes
        const uint32_t s_addr = lanes + t * kTileRows, o_addr = lanes + 2 * kTileRows + t * D;
        float m = -INFINITY, l = 0.f;
        bool fine = true;
        const int my_steps = t < tiles_q ? steps : 0;
        for (int j = 0; j < my_steps; ++j) {
            fine = tc_wait(&s_full[t], j & 1);
            if (!fine) break;
            tc_fence_after();
            if ((threadIdx.x & (kTileRows - 1)) == 0) {  // this tile is done with K of this step and V of the last
                mbar_arrive(&empty[(2 * j) % T::kStages]);
                if (j > 0) mbar_arrive(&empty[(2 * j - 1) % T::kStages]);
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
                        for (int i = 0; i < 32; ++i)
                            if (!((see >> i) & 1u)) s[c][i] = 0xff800000u;
                    }
                }
            }
            float top[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                top[c] = fmaxf(__uint_as_float(s[c][0]), __uint_as_float(s[c][1]));
#pragma unroll
                for (int i = 2; i < 32; i += 2) top[c] = max3(top[c], __uint_as_float(s[c][i]), __uint_as_float(s[c][i + 1]));
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
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                    tmem_store32(o_addr + c, o);
                }
            }
            const float base = m == -INFINITY ? 0.f : m;
            const uint64_t scale2 = pair(p.scale_log2, p.scale_log2), base2 = pair(-base, -base);
            uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t w[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const uint32_t(&x)[32] = s[2 * c + i / 16];
                    const float2 e = unpair(fma2(pair(__uint_as_float(x[2 * (i % 16)]), __uint_as_float(x[2 * (i % 16) + 1])),
                                                 scale2, base2));
                    const float a = fast_exp2(e.x), b = fast_exp2(e.y);
                    sum[i & 3] = add2(sum[i & 3], pair(a, b));
                    w[i] = pack_bf16x2(a, b);
                }
                tmem_store32(s_addr + c * 32, w);
                tmem_wait_store();
                tc_fence_before();
                mbar_arrive(&p_ready[t][c]);
            }
            const float2 both = unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
            l += both.x + both.y;
        }
        // ---- the row's output ----
        bool odd = false;
        fine = fine && tc_wait(&loads_done, 0);
        if (fine && my_steps > 0) fine = tc_wait(&o_done[t], 0);
        if (!fine && lane == 0) report(p.dev_status, SFI_DEV_TIMEOUT);
        const bool write = fine && t < tiles_q && mine && s_bad == 0;
        if (fine && t < tiles_q) {
            tc_fence_after();
            const int64_t at = ((int64_t)r * p.tokens + token) * p.hq + head;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            // through the warp's part of Q's tile (nothing reads it any more), so that whole rows leave together:
            // 16-byte stores to 32 rows at a time took 6000 cycles
            constexpr int kChunks = D / 8;  // 16-byte pieces of a row
            uint8_t *stage = smem + t * T::kBytes + (warp & 3) * 32 * D * 2;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                if (my_steps > 0) {
                    tmem_load32(o_addr + c, o);
                    tmem_wait_load();
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0u;
                }
                uint32_t big = 0;
#pragma unroll
                for (int i = 0; i < 32; ++i) big = max(big, o[i] & 0x7fffffffu);
                odd |= big >= 0x7f800000u;
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                    int4 v;
                    v.x = (int)pack_bf16x2(__uint_as_float(o[i]) * inv, __uint_as_float(o[i + 1]) * inv);
                    v.y = (int)pack_bf16x2(__uint_as_float(o[i + 2]) * inv, __uint_as_float(o[i + 3]) * inv);
                    v.z = (int)pack_bf16x2(__uint_as_float(o[i + 4]) * inv, __uint_as_float(o[i + 5]) * inv);
                    v.w = (int)pack_bf16x2(__uint_as_float(o[i + 6]) * inv, __uint_as_float(o[i + 7]) * inv);
                    *reinterpret_cast<int4 *>(stage + lane * D * 2 + ((((c + i) / 8) ^ (lane & 7)) << 4)) = v;
                }
            }
            __syncwarp();
            const uint32_t rows = __ballot_sync(0xffffffffu, write);
            const int row0 = (warp & 3) * 32, chunk = lane % kChunks;
            __nv_bfloat16 *out = p.out + (((int64_t)r * p.tokens + tok0 + t * per_tile) * p.hq + kvh * G) * D + chunk * 8;
#pragma unroll 4
            for (int i = lane / kChunks; i < 32; i += 32 / kChunks) {
                const int tok = (row0 + i) >> shift, h = (row0 + i) & (G - 1);
                const int4 v = *reinterpret_cast<const int4 *>(stage + i * D * 2 + ((chunk ^ (i & 7)) << 4));
                if ((rows >> i) & 1u) st_v4(out + ((int64_t)tok * p.hq + h) * D, v);
            }
            __syncwarp();
            if (write && p.lse) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
            uint32_t again = __ballot_sync(0xffffffffu, odd && write);
            while (again) {
                const int from = __ffs(again) - 1;
                again &= again - 1;
                window_row<D>(p, r, __shfl_sync(0xffffffffu, token, from), __shfl_sync(0xffffffffu, head, from),
                              __shfl_sync(0xffffffffu, pos, from), __shfl_sync(0xffffffffu, m, from),
                              __shfl_sync(0xffffffffu, l, from), 0, D);
            }
        }
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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.hkv, (unsigned)batch, (unsigned)((p.tokens + per_cta - 1) / per_cta));
    cfg.blockDim = dim3(kPromptThreads);
    cfg.dynamicSmemBytes = PromptTile<D>::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, maps.q, maps.k, maps.v, p);
}

}  // namespace

cudaError_t launch_window_prompt(const WindowMaps &maps, const WindowParams &p, int head_dim, int batch,
                                 cudaStream_t stream) {
    return head_dim == 128 ? launch_prompt<128>(maps, p, batch, stream) : launch_prompt<64>(maps, p, batch, stream);
}

}  // namespace sfi
