// Accumulated attention weights: what the queries of new tokens gave to each cached position,
//   mass[h][j] = decay mass[h][j] + sum over tokens t that see j and heads g of exp(x_{t,g,j} - lse_{t,g}).
//
// The attention call has left the log-sum-exps, so a weight needs no second pass over its row. With many
// tokens it is bound by the tensor cores and the exponentials (2 D flops and one exp per pair), with few
// by HBM (K is read once). S^T = K Q^T puts positions on the M side: a thread owns a position, and the sum
// over the query rows is a sum over the columns it reads, with no exchange between threads and one writer
// per position (no atomics: the order of additions, and so the result, is the same in every run).
//
// A CTA takes 256 positions of one KV head as two tiles of 128, whose K rows stay in shared memory, and
// walks the query rows that see any of them (row = token * G + head) in tiles of kRows: 128, or as few as
// the call has when it is short, so that several CTAs share an SM and K streams. S^T is double-buffered in
// tensor memory; weights are summed in fp32, four sums per thread and tile.
// A prompt of 8192 tokens, 16/8/128 heads: 252 us (29% of the measured bf16 rate).
#include <algorithm>
#include <atomic>

#include "tensor_core.cuh"
#include "window_span.cuh"

namespace sfi {

namespace {

constexpr int kMassThreads = 320;  // two warpgroups of sums, a copy warp, a matrix warp
constexpr int kMassCopyWarp = 8, kMassMmaWarp = 9;
constexpr int kMassKeys = 256;     // positions of a CTA
constexpr int kKeyTile = 128;

template <int D, int ROWS>
struct MassTile {
    static constexpr int kHalves = D / 64;
    static constexpr int kKeyHalf = kKeyTile * 128;
    static constexpr int kKeyBytes = kHalves * kKeyHalf;       // K of 128 positions
    static constexpr int kRowHalf = ROWS * 128;
    static constexpr int kRowBytes = kHalves * kRowHalf;       // a tile of query rows
    static constexpr int kStages = ROWS == 128 ? 4 : 1;        // (fewer rows: one tile has them all)
    static constexpr int kBuffers = ROWS == 128 ? 2 : 1;       // of S^T
    static constexpr int kColumns = 2 * ROWS * kBuffers;
    static constexpr int kSmem = 2 * kKeyBytes + kStages * kRowBytes + 1024;
    static constexpr int kPerSm = ROWS == 128 ? 1 : ROWS == 64 ? 2 : 3;
    static constexpr uint32_t kScores = mma_desc(kKeyTile, ROWS, false);
};

// Weights of one position, summed over the columns (query rows) of its lane of S^T: all, or [lo, hi).
template <int ROWS, bool WHOLE>
__device__ __forceinline__ void sum_columns(uint32_t addr, const float *lse, float scale_log2, int lo, int hi,
                                            float (&sum)[4]) {
    constexpr int kLoad = ROWS < 32 ? 16 : 32;  // columns of one read of tensor memory
    uint32_t s[2][kLoad];
    auto load = [&](int c, uint32_t (&v)[kLoad]) {
        if constexpr (kLoad == 32) tmem_load32(addr + c, v);
        else tmem_load16(addr + c, v);
    };
    load(0, s[0]);
#pragma unroll
    for (int c = 0; c < ROWS; c += kLoad) {
        const int at = c / kLoad & 1;
        tmem_wait_load();
        if (c + kLoad < ROWS) load(c + kLoad, s[at ^ 1]);  // on their way while these are summed
#pragma unroll
        for (int i = 0; i < kLoad; i += 4) {
            const float4 e = *reinterpret_cast<const float4 *>(&lse[c + i]);
            const float x[4] = {fast_exp2(fmaf(__uint_as_float(s[at][i]), scale_log2, e.x)),
                                fast_exp2(fmaf(__uint_as_float(s[at][i + 1]), scale_log2, e.y)),
                                fast_exp2(fmaf(__uint_as_float(s[at][i + 2]), scale_log2, e.z)),
                                fast_exp2(fmaf(__uint_as_float(s[at][i + 3]), scale_log2, e.w))};
#pragma unroll
            for (int k = 0; k < 4; ++k) sum[k] += WHOLE || (c + i + k >= lo && c + i + k < hi) ? x[k] : 0.f;
        }
    }
}

}  // namespace

template <int D, int ROWS>
__global__ void __launch_bounds__(kMassThreads, MassTile<D, ROWS>::kPerSm)
    attn_mass_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const WindowParams p, const MassParams w) {
    using T = MassTile<D, ROWS>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *ring = smem + 2 * T::kKeyBytes;
    __shared__ __align__(8) uint64_t k_full, full[T::kStages], empty[T::kStages];
    __shared__ __align__(8) uint64_t s_full[T::kBuffers], s_empty[T::kBuffers];
    __shared__ __align__(16) float s_lse[T::kStages][ROWS];  // -lse in log2 units
    __shared__ uint32_t s_tmem;
    __shared__ int s_bad;
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
    const int k0 = blockIdx.x * kMassKeys;
    if (k0 >= L) return;
    const int k1 = min(k0 + kMassKeys, L) - 1;
    const int G = p.group, shift = __ffs(G) - 1, per_tile = ROWS >> shift;
    // tokens that see any of these positions, in whole tiles counted from the first of them
    const int from = max(L - n, k0);
    const int to = k0 < p.sink ? L - 1 : (int)min((int64_t)L - 1, (int64_t)k1 + p.recent - 1);
    const int steps = n > 0 && to >= from ? (to - from) / per_tile + 1 : 0;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        mbar_init(&k_full, 1);
        for (int i = 0; i < T::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1 + 8);
        }
        for (int i = 0; i < T::kBuffers; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], 8);
        }
        s_bad = 0;
        fence_barrier_init();
    }
    if (warp == kMassMmaWarp) tmem_alloc(&s_tmem, T::kColumns);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    bool fine = true;
    float acc = 0.f, old = 0.f;
    const int key = k0 + (int)threadIdx.x;  // of the first 256 threads
    float *mass = w.mass + ((int64_t)r * p.hkv + kvh) * w.stride;

    if (warp == kMassCopyWarp) {
        if (steps > 0) {
            // K: sixteen pages
            const int v = (k0 / kSubTokens) + (lane & 15);
            const bool listed = v <= k1 / kSubTokens;
            const int page = listed ? p.page_table[(int64_t)r * p.max_pages + v] : -1;
            const bool ok = page >= 0 && page < p.num_pages;
            if (listed && !ok) {
                if (lane < 16) report(p.dev_status, SFI_DEV_BAD_PAGE);
                s_bad = 1;  // nothing of this CTA's positions is written
            }
            const uint32_t take = __ballot_sync(0xffffffffu, ok && lane < 16);
            if (lane == 0) {
                if (take) mbar_arrive_expect_tx(&k_full, __popc(take) * kSubTokens * D * 2);
                else mbar_arrive(&k_full);
            }
            __syncwarp();
            if (ok && lane < 16 * T::kHalves) {
                const int half = lane >> 4, at = lane & 15;
                tma_tile_2d(smem + (at >> 3) * T::kKeyBytes + half * T::kKeyHalf + (at & 7) * kSubTokens * 128, &tm_k,
                            half * 64, (page * p.hkv + kvh) * kSubTokens, &k_full);
            }
            for (int j = 0; j < steps; ++j) {
                const int slot = j % T::kStages;
                if (j >= T::kStages && !tc_wait(&empty[slot], (j / T::kStages - 1) & 1)) {
                    fine = false;
                    break;
                }
                const int tok0 = from - (L - n) + j * per_tile;
                for (int i = lane; i < ROWS; i += 32) {
                    const int tok = tok0 + (i >> shift);
                    s_lse[slot][i] =
                        tok < n ? w.lse[((int64_t)r * p.tokens + tok) * p.hq + (kvh << shift) + (i & (G - 1))] * -1.4426950408889634f
                                : 0.f;
                }
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
    } else if (warp == kMassMmaWarp) {
        const uint32_t ka = smem_u32(smem), ra = smem_u32(ring);
        const int tiles = k1 - k0 >= kKeyTile ? 2 : 1;
        if (steps > 0) fine = tc_wait(&k_full, 0);
        for (int j = 0; j < steps && fine; ++j) {
            const int slot = j % T::kStages, buf = j % T::kBuffers;
            fine = tc_wait(&full[slot], (j / T::kStages) & 1);
            if (fine && j >= T::kBuffers) fine = tc_wait(&s_empty[buf], (j / T::kBuffers - 1) & 1);
            if (!fine) break;
            tc_fence_after();
            if (lane == 0) {
                for (int t = 0; t < tiles; ++t)
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        mma_ss(tmem + (buf * 2 + t) * ROWS,
                               smem_desc(ka + t * T::kKeyBytes + (ks >> 2) * T::kKeyHalf + (ks & 3) * 32, 16),
                               smem_desc(ra + slot * T::kRowBytes + (ks >> 2) * T::kRowHalf + (ks & 3) * 32, 16),
                               T::kScores, ks > 0);
                mma_commit(&s_full[buf]);
                mma_commit(&empty[slot]);
            }
            __syncwarp();
        }
    } else {
        // ---- one position per thread ----
        const int t = warp >> 2;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21) + t * ROWS;
        if (key < L - n && w.decay != 0.f) old = w.decay * mass[key];
        const int tile0 = k0 + t * kKeyTile, tile1 = min(tile0 + kKeyTile - 1, k1);
        const bool any = tile0 <= k1;
        for (int j = 0; j < steps; ++j) {
            const int slot = j % T::kStages, buf = j % T::kBuffers;
            fine = tc_wait(&full[slot], (j / T::kStages) & 1) &&
                   tc_wait(&s_full[buf], (j / T::kBuffers) & 1);
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
            const uint32_t addr = lanes + buf * 2 * ROWS;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
            if (any && whole) sum_columns<ROWS, true>(addr, s_lse[slot], p.scale_log2, lo, hi, sum);
            else if (any) sum_columns<ROWS, false>(addr, s_lse[slot], p.scale_log2, lo, hi, sum);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&s_empty[buf]);
                mbar_arrive(&empty[slot]);
            }
            acc += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        }
    }
    if (!fine && lane == 0) {
        report(p.dev_status, SFI_DEV_TIMEOUT);
        s_bad = 1;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMassMmaWarp) tmem_free(tmem, T::kColumns);
    if (warp < 8 && key <= k1 && s_bad == 0) mass[key] = old + acc;
}

namespace {

template <int D, int ROWS>
cudaError_t launch_mass(const WindowMaps &maps, const WindowParams &p, const MassParams &w, int batch,
                        cudaStream_t stream) {
    auto kernel = attn_mass_kernel<D, ROWS>;
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kernel), MassTile<D, ROWS>::kSmem, configured);
    if (e != cudaSuccess) return e;
    const int64_t most = std::min<int64_t>((int64_t)p.max_pages * kSubTokens, w.stride);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((most + kMassKeys - 1) / kMassKeys), (unsigned)p.hkv, (unsigned)batch);
    cfg.blockDim = dim3(kMassThreads);
    cfg.dynamicSmemBytes = MassTile<D, ROWS>::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, maps.q, maps.k, p, w);
}

template <int D>
cudaError_t launch_mass_rows(const WindowMaps &maps, const WindowParams &p, const MassParams &w, int rows, int batch,
                             cudaStream_t stream) {
    switch (rows) {
        case 16: return launch_mass<D, 16>(maps, p, w, batch, stream);
        case 32: return launch_mass<D, 32>(maps, p, w, batch, stream);
        case 64: return launch_mass<D, 64>(maps, p, w, batch, stream);
        default: return launch_mass<D, 128>(maps, p, w, batch, stream);
    }
}

}  // namespace

// Query rows of a tile: all of a short call's (16, 32 or 64), or 128.
int mass_rows(int64_t rows) {
    int n = 16;
    while (n < 128 && n < rows) n *= 2;
    return n;
}

cudaError_t launch_attn_mass(const WindowMaps &maps, const WindowParams &p, const MassParams &w, int head_dim, int batch,
                             cudaStream_t stream) {
    const int rows = mass_rows((int64_t)p.tokens * p.group);
    return head_dim == 128 ? launch_mass_rows<128>(maps, p, w, rows, batch, stream)
                           : launch_mass_rows<64>(maps, p, w, rows, batch, stream);
}

}  // namespace sfi
