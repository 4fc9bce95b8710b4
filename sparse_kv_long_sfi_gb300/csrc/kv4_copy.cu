// The calls that fill, read back and compact the 4-bit cache.
//
// One warp owns K or V of one (page, KV head) block at a time, so the half-byte updates of a
// partly written page race with nobody. K rows are contiguous in a block; V codes lie in the
// order of the matrix instruction's lanes, so rows of V pass through shared memory.
// All three are copies with a conversion: bound by HBM when there are many tokens, by
// launch latency in a decode step.
#include <algorithm>

#include "kv4_format.cuh"

namespace sfi {

constexpr int kKv4Warps = 8;

// Shared memory of a warp: a page's V codes and scales by token.
template <int D>
struct Kv4Tile {
    uint2 code[16][D / 16];  // sixteen codes of a token
    uint8_t scale[16][D / 16];
};

// The larger magnitudes of two pairs of bf16.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a & 0x7fff7fffu), "r"(b & 0x7fff7fffu));
    return r;
}

// Codes and scale of eight values (a lane's part of a row; the lane beside it holds the
// other half of the group of 16).
__device__ __forceinline__ uint32_t quantise8(int4 raw, float inv6g, float g, uint32_t *scale) {
    const uint32_t w[4] = {(uint32_t)raw.x, (uint32_t)raw.y, (uint32_t)raw.z, (uint32_t)raw.w};
    // the largest magnitude; a NaN wins
    uint32_t top2 = max_abs_bf16x2(max_abs_bf16x2(w[0], w[1]), max_abs_bf16x2(w[2], w[3]));
    top2 = max_abs_bf16x2(top2, __shfl_xor_sync(0xffffffffu, top2, 1));
    const uint32_t top = max(top2 & 0xffffu, top2 >> 16);
    const bool fine = top < 0x7f80u;
    const uint32_t s = fine ? group_scale(__uint_as_float(top << 16), inv6g) : kE4m3Nan;
    *scale = s;
    float x[8];
    bf16x8_to_f32(raw, x);
    const float step = e4m3_to_f32(s) * g;
    const float inv = reciprocal(step);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= inv;
    return fine && step > 0.f ? f32x8_to_e2m1(x) : 0u;
}

// An item of the append and the read: K or V of one page of one KV head of one request.
struct Kv4Item {
    int is_v, h, slot, entry;
    __device__ __forceinline__ Kv4Item(int64_t item, int hkv, int slots) {
        is_v = (int)(item & 1);
        const int64_t at = item >> 1, page = quotient(at, hkv);
        h = (int)(at - page * hkv);
        entry = (int)quotient(page, slots);
        slot = (int)(page - (int64_t)entry * slots);
    }
};

// Rows [a, b) of the block's K or V (row tok from src + (tok - a) * stride).
template <int D>
__device__ void write_block(uint8_t *block, Kv4Tile<D> &tile, const __nv_bfloat16 *src, int64_t stride, int a, int b,
                            bool is_v, float g, int lane) {
    using F = Kv4<D>;
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kIters = 16 / kRows;
    const int sub = lane / kLanes, l = lane % kLanes;
    const float inv6g = reciprocal(6.f * g);
    int4 raw[kIters];
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
        const int row = i * kRows + sub;
        raw[i] = make_int4(0, 0, 0, 0);
        if (row >= a && row < b) raw[i] = ld_stream_v4(src + (int64_t)(row - a) * stride + l * 8);
    }
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
        const int row = i * kRows + sub;
        if ((i + 1) * kRows <= a || i * kRows >= b) continue;  // no row of this load (the same in all lanes)
        uint32_t s;
        const uint32_t code = quantise8(raw[i], inv6g, g, &s);
        if (row < a || row >= b) continue;
        if (is_v) {
            reinterpret_cast<uint32_t *>(tile.code[row])[l] = code;
            if ((l & 1) == 0) tile.scale[row][l / 2] = (uint8_t)s;
        } else {
            *reinterpret_cast<uint32_t *>(block + row * F::kKRow + l * 4) = code;
            if ((l & 1) == 0) block[F::kKScale + row * F::kGroups + l / 2] = (uint8_t)s;
        }
    }
    if (!is_v) return;
    __syncwarp();
    // a lane per (four tokens, sixteen dims): their codes as the eight words they make in the
    // block, their scales as the word of the four
    if (lane < 4 * F::kGroups) {
        const int t = lane / F::kGroups, j = lane % F::kGroups;
        uint32_t keep = 0, keep_scale = 0;  // bits of a word that belong to tokens outside [a, b)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (4 * t + i < a || 4 * t + i >= b) {
                keep |= 0x0f0fu << (16 * (i >> 1) + 4 * (i & 1));
                keep_scale |= 0xffu << (8 * i);
            }
        if (keep != 0xffffffffu) {
            uint32_t in[4][2], out[8], sc = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint2 c = tile.code[4 * t + i][j];
                in[i][0] = c.x;
                in[i][1] = c.y;
                sc |= (uint32_t)tile.scale[4 * t + i][j] << (8 * i);
            }
            v_pack(in, out);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                uint32_t *dst = reinterpret_cast<uint32_t *>(block + F::kVCode + v_word(j, k, t));
                *dst = keep ? (*dst & keep) | (out[k] & ~keep) : out[k];
            }
            uint32_t *dst = reinterpret_cast<uint32_t *>(block + F::kVScale + lane * 4);
            *dst = keep_scale ? (*dst & keep_scale) | (sc & ~keep_scale) : sc;
        }
    }
    __syncwarp();
}

template <int D>
__global__ void __launch_bounds__(kKv4Warps * 32, 4) kv4_append_kernel(const Kv4CopyParams p, int batch, int page_slots) {
    __shared__ Kv4Tile<D> s_tile[kKv4Warps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t items = (int64_t)batch * page_slots * p.hkv * 2;
    grid_dependency_wait();
    grid_launch_dependents();  // not before the wait: see launch_dependent_clusters
    for (int64_t item = (int64_t)blockIdx.x * kKv4Warps + warp; item < items;
         item += (int64_t)gridDim.x * kKv4Warps) {
        const Kv4Item x(item, p.hkv, page_slots);
        const int r = p.req_ids ? p.req_ids[x.entry] : x.entry;
        const int L = p.seq_lens[r];
        const int n = p.new_lens ? p.new_lens[r] : p.tokens;
        if (n < 0 || n > p.tokens || L < n || L > p.max_pages * kSubTokens) {
            if (lane == 0 && x.h == 0 && x.slot == 0) report(p.dev_status, SFI_DEV_BAD_LEN);
            continue;
        }
        const int first = L - n;
        const int pg = first / kSubTokens + x.slot;
        if (pg > (L - 1) / kSubTokens) continue;  // (before its position, which may pass 32 bits)
        const int pos0 = pg * kSubTokens;
        const int a = max(first - pos0, 0), b = min(L - pos0, kSubTokens);
        if (a >= b) continue;
        const int page = p.page_table[(int64_t)r * p.max_pages + pg];
        if (page < 0 || page >= p.num_pages) {
            if (lane == 0) report(p.dev_status, SFI_DEV_BAD_PAGE);
            continue;
        }
        const int64_t stride = x.is_v ? p.v_stride : p.k_stride;
        const __nv_bfloat16 *src = (x.is_v ? p.v_new : p.k_new) +
                                   ((int64_t)r * p.tokens + (pos0 + a - first)) * stride + (int64_t)x.h * D;
        write_block<D>(p.pool + ((int64_t)page * p.hkv + x.h) * Kv4<D>::kBlock, s_tile[warp], src, stride, a, b, x.is_v,
                       x.is_v ? p.v_scale : p.k_scale, lane);
    }
}

// Rows [a, b) of a block's K or V as bf16 rows (row tok to dst + (tok - a) * stride).
template <int D>
__device__ void read_block(const uint8_t *block, Kv4Tile<D> &tile, __nv_bfloat16 *dst, int64_t stride, int a, int b,
                           bool is_v, float g, int lane) {
    using F = Kv4<D>;
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kIters = 16 / kRows;
    const int sub = lane / kLanes, l = lane % kLanes;
    uint32_t code[kIters], scale[kIters];
    if (is_v) {
        // a lane per (four tokens, sixteen dims) brings V's codes into rows
        if (lane < 4 * F::kGroups) {
            const int t = lane / F::kGroups, j = lane % F::kGroups;
            uint32_t in[4][2], out[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) out[k] = *reinterpret_cast<const uint32_t *>(block + F::kVCode + v_word(j, k, t));
            const uint32_t sc = *reinterpret_cast<const uint32_t *>(block + F::kVScale + lane * 4);
            v_unpack(out, in);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                tile.code[4 * t + i][j] = make_uint2(in[i][0], in[i][1]);
                tile.scale[4 * t + i][j] = (uint8_t)(sc >> (8 * i));
            }
        }
        __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
        const int row = i * kRows + sub;
        if (is_v) {
            code[i] = reinterpret_cast<const uint32_t *>(tile.code[row])[l];
            scale[i] = tile.scale[row][l / 2];
        } else {
            code[i] = *reinterpret_cast<const uint32_t *>(block + row * F::kKRow + l * 4);
            scale[i] = block[F::kKScale + row * F::kGroups + l / 2];
        }
    }
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
        const int row = i * kRows + sub;
        if (row < a || row >= b) continue;
        uint32_t h[4];
        float x[8];
        e2m1x8_to_f16(code[i], h);
        const float s = e4m3_to_f32(scale[i]) * g;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h[k]));
            x[2 * k] = v.x * s;
            x[2 * k + 1] = v.y * s;
        }
        st_v4(dst + (int64_t)(row - a) * stride + l * 8, f32x8_to_bf16(x));
    }
    __syncwarp();
}

template <int D>
__global__ void __launch_bounds__(kKv4Warps * 32) kv4_read_kernel(const Kv4CopyParams p, int batch, int page_slots) {
    __shared__ Kv4Tile<D> s_tile[kKv4Warps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t items = (int64_t)batch * page_slots * p.hkv * 2;
    grid_dependency_wait();
    grid_launch_dependents();  // not before the wait: see launch_dependent_clusters
    for (int64_t item = (int64_t)blockIdx.x * kKv4Warps + warp; item < items;
         item += (int64_t)gridDim.x * kKv4Warps) {
        const Kv4Item x(item, p.hkv, page_slots);
        const int r = p.req_ids ? p.req_ids[x.entry] : x.entry;
        const int L = p.seq_lens[r];
        const int first = p.first ? p.first[r] : 0;
        if (L < 0 || L > p.max_pages * kSubTokens || first < 0) {
            if (lane == 0 && x.h == 0 && x.slot == 0) report(p.dev_status, SFI_DEV_BAD_LEN);
            continue;
        }
        const int end = (int)min((int64_t)L, (int64_t)first + p.tokens);
        const int64_t pos0 = ((int64_t)first / kSubTokens + x.slot) * kSubTokens;
        const int a = (int)max(first - pos0, (int64_t)0), b = (int)min(end - pos0, (int64_t)kSubTokens);
        if (a >= b) continue;
        const int page = p.page_table[(int64_t)r * p.max_pages + pos0 / kSubTokens];
        if (page < 0 || page >= p.num_pages) {
            if (lane == 0) report(p.dev_status, SFI_DEV_BAD_PAGE);
            continue;
        }
        const int64_t row = ((int64_t)r * p.tokens + (pos0 + a - first)) * p.hkv + x.h;
        read_block<D>(p.pool + ((int64_t)page * p.hkv + x.h) * Kv4<D>::kBlock, s_tile[warp],
                      (x.is_v ? p.v_out : p.k_out) + row * D, (int64_t)p.hkv * D, a, b, x.is_v,
                      x.is_v ? p.v_scale : p.k_scale, lane);
    }
}

// Compact blocks: each warp writes one block whole. Row i of it comes from one position's
// page; the codes and scales move unchanged. A token's V codes are a quarter of the 32-byte
// sectors they lie in, so a row's gather reads 64 + 32 + 2 D + 32 bytes (D = 128).
template <int D>
__global__ void __launch_bounds__(kKv4Warps * 32) kv4_compact_kernel(const Kv4CopyParams p, int batch, int slots) {
    using F = Kv4<D>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t items = (int64_t)batch * slots * p.hkv;
    grid_launch_dependents();  // (an ordinary launch: everything before it on the stream has finished)
    for (int64_t item = (int64_t)blockIdx.x * kKv4Warps + warp; item < items;
         item += (int64_t)gridDim.x * kKv4Warps) {
        const int h = (int)(item % p.hkv);
        const int64_t at = item / p.hkv;
        const int ps = (int)(at % slots), bi = (int)(at / slots);
        const int r = p.req_ids ? p.req_ids[bi] : bi;
        const int L = p.seq_lens[r], cnt = p.count[r], cap = p.c_capacity[r];
        const int64_t off = p.c_page_offset[r];
        uint32_t err = 0;
        if (L < 1 || L > p.max_pages * kSubTokens) err = SFI_DEV_BAD_LEN;
        else if (cnt < 0 || cnt > p.k_cap || cap < 0 || ((int64_t)p.sink + cnt + 15) / 16 > cap || (cnt > 0 && L < p.sink))
            err = SFI_DEV_K_OVERFLOW;
        else if (off < 0 || off + (int64_t)p.hkv * cap > p.c_total_pages) err = SFI_DEV_BAD_COMPACT;
        if (err) {
            if (lane == 0 && h == 0 && ps == 0) report(p.dev_status, err);
            continue;
        }
        const int ns = min(p.sink, L);
        const int rows = ns + cnt;  // cnt > 0 only with ns == sink
        if (ps * 16 >= rows) continue;
        // lane i (and i + 16) looks up row i: its page's block and its slot there
        const int i = ps * 16 + (lane & 15);
        int64_t src = -1;
        int slot = 0;
        if (i < rows) {
            const int pos = i < ns ? i : p.idx[((int64_t)r * p.hkv + h) * p.k_cap + (i - p.sink)];
            if (pos < 0 || pos >= L) {
                err = SFI_DEV_BAD_INDEX;
            } else {
                const int page = p.page_table[(int64_t)r * p.max_pages + pos / kSubTokens];
                if (page < 0 || page >= p.num_pages) err = SFI_DEV_BAD_PAGE;
                else src = ((int64_t)page * p.hkv + h) * F::kBlock;
                slot = pos % kSubTokens;
            }
        }
        if (err && lane < 16) report(p.dev_status, err);
        uint8_t *dst = p.c_pool + (off + (int64_t)h * cap + ps) * F::kBlock;
        // Every load of the block is on its way before the first store; a row that holds nothing
        // reads the pool's first block and is cleared.
        const bool none = src < 0;
        if (none) src = 0;
        const uint32_t empty = __ballot_sync(0xffffffffu, none);  // bit i: row i
        constexpr int kLanes = F::kKRow / 16;      // 16-byte pieces of a K row
        constexpr int kKIters = 16 * kLanes / 32;  // two, or one at D = 64
        constexpr int kVIters = D / 64;
        int4 kv[kKIters];
#pragma unroll
        for (int i = 0; i < kKIters; ++i) {
            const int row = (i * 32 + lane) / kLanes, piece = lane % kLanes;
            const int64_t s = __shfl_sync(0xffffffffu, src, row);
            const int sl = __shfl_sync(0xffffffffu, slot, row);
            kv[i] = ld_stream_v4(p.pool + s + sl * F::kKRow + piece * 16);
            if ((empty >> row) & 1u) kv[i] = make_int4(0, 0, 0, 0);
        }
        uint32_t ksc;  // two lanes per row: half of its K scales each
        constexpr int kHalf = F::kGroups / 2;  // 4 or 2 bytes
        {
            const int row = lane >> 1;
            const int64_t s = __shfl_sync(0xffffffffu, src, row);
            const int sl = __shfl_sync(0xffffffffu, slot, row);
            const uint8_t *at = p.pool + s + F::kKScale + sl * F::kGroups + (lane & 1) * kHalf;
            if constexpr (kHalf == 4) ksc = *reinterpret_cast<const uint32_t *>(at);
            else ksc = *reinterpret_cast<const uint16_t *>(at);
            if ((empty >> row) & 1u) ksc = 0;
        }
        int4 vv[kVIters][4];  // V codes: the units of the four tokens that this lane's unit joins
        int from[4];          // where a token's half bytes lie in them
        const VUnit x(lane);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t s = __shfl_sync(0xffffffffu, src, 4 * x.t + q);
            const int sl = __shfl_sync(0xffffffffu, slot, 4 * x.t + q);
            from[q] = 16 * ((sl >> 1) & 1) + 4 * (sl & 1);
            // the same dims of the source token's group of four
            const uint8_t *at = p.pool + s + F::kVCode + (lane - 2 * x.t + 2 * (sl >> 2)) * 16;
#pragma unroll
            for (int i = 0; i < kVIters; ++i) vv[i][q] = ld_stream_v4(at + i * 512);
        }
        uint32_t vsc = 0;  // lane w: the word of four tokens' V scales (16 words at D = 64)
        {
            const int w = lane % (4 * F::kGroups);
            const int t = w / F::kGroups, grp = w % F::kGroups;
            uint32_t byte[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t s = __shfl_sync(0xffffffffu, src, 4 * t + q);
                const int sl = __shfl_sync(0xffffffffu, slot, 4 * t + q);
                byte[q] = p.pool[s + F::kVScale + (sl >> 2) * F::kVScaleT + grp * 4 + (sl & 3)];
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (!((empty >> (4 * t + q)) & 1u)) vsc |= byte[q] << (8 * q);
        }
#pragma unroll
        for (int i = 0; i < kKIters; ++i) st_v4(dst + (i * 32 + lane) * 16, kv[i]);
        if constexpr (kHalf == 4) *reinterpret_cast<uint32_t *>(dst + F::kKScale + lane * 4) = ksc;
        else *reinterpret_cast<uint16_t *>(dst + F::kKScale + lane * 2) = (uint16_t)ksc;
#pragma unroll
        for (int i = 0; i < kVIters; ++i) {
            uint32_t res[4] = {0, 0, 0, 0};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t w[4] = {(uint32_t)vv[i][q].x, (uint32_t)vv[i][q].y, (uint32_t)vv[i][q].z, (uint32_t)vv[i][q].w};
                const uint32_t keep = (empty >> (4 * x.t + q)) & 1u ? 0u : 0x0f0fu;
#pragma unroll
                for (int jr = 0; jr < 4; ++jr) res[jr] |= ((w[jr] >> from[q]) & keep) << (16 * (q >> 1) + 4 * (q & 1));
            }
            st_v4(dst + F::kVCode + i * 512 + lane * 16, make_int4((int)res[0], (int)res[1], (int)res[2], (int)res[3]));
        }
        if (lane < 4 * F::kGroups) *reinterpret_cast<uint32_t *>(dst + F::kVScale + lane * 4) = vsc;
    }
}

namespace {

// One warp per item, as many CTAs as there are items up to several waves.
int copy_grid(int64_t items) {
    const int sms = sm_count_current_device();
    return (int)std::max<int64_t>(1, std::min<int64_t>((items + kKv4Warps - 1) / kKv4Warps, (int64_t)sms * 32));
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4CopyParams &p, int head_dim, int batch, cudaStream_t stream) {
    const int slots = (int)(((int64_t)p.tokens + 30) / 16);  // pages that `tokens` positions can touch
    const int grid = copy_grid((int64_t)batch * slots * p.hkv * 2);
    return launch_dependent(head_dim == 128 ? kv4_append_kernel<128> : kv4_append_kernel<64>, grid, kKv4Warps * 32, 0, stream,
                            p, batch, slots);
}

cudaError_t launch_kv4_read(const Kv4CopyParams &p, int head_dim, int batch, cudaStream_t stream) {
    const int slots = (int)(((int64_t)p.tokens + 30) / 16);
    const int grid = copy_grid((int64_t)batch * slots * p.hkv * 2);
    return launch_dependent(head_dim == 128 ? kv4_read_kernel<128> : kv4_read_kernel<64>, grid, kKv4Warps * 32, 0, stream,
                            p, batch, slots);
}

cudaError_t launch_kv4_compact(const Kv4CopyParams &p, int head_dim, int batch, cudaStream_t stream) {
    const int slots = (p.sink + p.k_cap + 15) / 16;
    const int grid = copy_grid((int64_t)batch * slots * p.hkv);
    // Not a dependent launch: behind an attention launch it would run with the shared-memory
    // split of that kernel, whose L1 is too small for it (32 requests of 1792 rows and the
    // attention after them: 134 us a pair against 106 us).
    auto kernel = head_dim == 128 ? kv4_compact_kernel<128> : kv4_compact_kernel<64>;
    kernel<<<grid, kKv4Warps * 32, 0, stream>>>(p, batch, slots);
    return cudaGetLastError();
}

}  // namespace sfi
