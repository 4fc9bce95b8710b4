// Head norm and position rotation of the new tokens' Q and K, written (with V) to where
// the attention calls read them: one pass over the projections' output.
//
// y = rotate(x * w / sqrt(mean(x^2) + eps)) per head row x of D values, in fp32, rounded
// once to bf16. Pair i turns by pos * turns[i] / 2^64 whole turns: the 64-bit product
// wraps modulo one turn by itself, so nothing of the angle is lost at far positions and
// no table of cosines is read; the upper 32 bits give the fraction of the turn to 2^-32.
//
// Bound by HBM: each row is read and written once. A row is held by D / 8 lanes (16 bytes
// each), a warp takes one token's rows two (four at D = 64) at a time, with four such
// loads in flight; its lanes compute the token's rot_dim / 2 cosines and sines once and
// keep the eight pairs of their own dims in registers for all rows.
#include <algorithm>

#include "sfi_device.cuh"
#include "sfi_internal.h"

namespace sfi {

constexpr int kNormWarps = 8;
constexpr int kNormBatch = 4;  // row loads in flight per lane

__device__ __forceinline__ void unpack8(int4 v, float (&x)[8]) {
    const uint32_t w[4] = {(uint32_t)v.x, (uint32_t)v.y, (uint32_t)v.z, (uint32_t)v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ int4 pack8(const float (&x)[8]) {
    return make_int4((int)pack_bf16x2(x[0], x[1]), (int)pack_bf16x2(x[2], x[3]), (int)pack_bf16x2(x[4], x[5]),
                     (int)pack_bf16x2(x[6], x[7]));
}

// One warp takes rows [chunk * rows_per_item, ...) of one token's q, k and v rows.
template <int D>
__global__ void __launch_bounds__(kNormWarps * 32) qk_norm_rope_kernel(const NormRopeParams p, int batch,
                                                                       int rows_per_item, int chunks) {
    constexpr int kLanes = D / 8;          // lanes per row
    constexpr int kRows = 32 / kLanes;     // rows per load
    __shared__ float2 s_cs[kNormWarps][D / 2];  // (cos, sin) of the token's pairs
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / kLanes, l = lane % kLanes;
    const int64_t items = (int64_t)batch * p.tokens * chunks;
    const int rows_all = p.hq + p.hkv + (p.v ? p.hkv : 0);
    const int half = p.rot_dim / 2;
    const bool rotated = l * 8 < p.rot_dim;
    // the lane that holds the other member of this lane's pairs (split halves)
    const int mate = p.interleaved || !rotated ? lane : (l * 8 < half ? lane + half / 8 : lane - half / 8);
    const bool second = l * 8 >= half;
    grid_launch_dependents();
    grid_dependency_wait();

    for (int64_t item = (int64_t)blockIdx.x * kNormWarps + warp; item < items; item += (int64_t)gridDim.x * kNormWarps) {
        const int64_t tok = item / chunks;
        const int chunk = (int)(item - tok * chunks);
        const int b = (int)(tok / p.tokens), t = (int)(tok - (int64_t)b * p.tokens);
        const int r = p.req_ids ? p.req_ids[b] : b;
        const int n = p.new_lens ? p.new_lens[r] : p.tokens;
        int slot = 0, page = -1;
        bool bad = n < 0 || n > p.tokens;
        if (p.seq_lens) {
            const int L = p.seq_lens[r];
            bad = bad || L < n || L > p.max_pages * kSubTokens;
            slot = L - n + t;
        }
        if (bad) {
            if (lane == 0 && t == 0 && chunk == 0) report(p.dev_status, SFI_DEV_BAD_LEN);
            continue;
        }
        if (t >= n) continue;
        const int64_t row_tok = (int64_t)r * p.tokens + t;
        if (p.seq_lens) {
            page = p.page_table[(int64_t)r * p.max_pages + slot / kSubTokens];
            if (page < 0 || page >= p.num_pages) {
                page = -1;
                if (lane == 0 && chunk == 0) report(p.dev_status, SFI_DEV_BAD_PAGE);
            }
        }
        // the token's rotations
        float cs[8], sn[8];
        if (p.rot_dim > 0) {
            __syncwarp();
            for (int i = lane; i < half; i += 32) {
                const int a = p.axis ? p.axis[i] : 0;
                int64_t pos = slot;
                if (p.positions) pos = a < p.num_axes ? p.positions[(int64_t)a * p.axis_stride + row_tok] : 0;
                if (a >= p.num_axes) {
                    pos = 0;
                    report(p.dev_status, SFI_DEV_BAD_INDEX);
                }
                const uint64_t turn = (uint64_t)pos * p.turns[i];
                const float x = (float)(int32_t)(turn >> 32) * 4.656612873077393e-10f;  // half turns in [-1, 1)
                float s, c;
                sincospif(x, &s, &c);
                s_cs[warp][i] = make_float2(c, s);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = l * 8 + i;
                const int pair = p.interleaved ? e / 2 : (second ? e - half : e);
                const float2 v = rotated ? s_cs[warp][pair] : make_float2(1.f, 0.f);
                cs[i] = v.x;
                // the sign of the mate's share: minus for the first member of a pair
                sn[i] = (p.interleaved ? (i & 1) == 0 : !second) ? -v.y : v.y;
            }
        }
        const int row_end = min(rows_all, (chunk + 1) * rows_per_item);
        for (int row0 = chunk * rows_per_item; row0 < row_end; row0 += kRows * kNormBatch) {
            int4 raw[kNormBatch];
#pragma unroll
            for (int u = 0; u < kNormBatch; ++u) {
                const int row = row0 + u * kRows + sub;
                if (row < row_end) {
                    const __nv_bfloat16 *src;
                    if (row < p.hq)
                        src = p.q + row_tok * p.q_stride + (int64_t)row * D;
                    else if (row < p.hq + p.hkv)
                        src = p.k + row_tok * p.k_stride + (int64_t)(row - p.hq) * D;
                    else
                        src = p.v + row_tok * p.v_stride + (int64_t)(row - p.hq - p.hkv) * D;
                    raw[u] = *reinterpret_cast<const int4 *>(src + l * 8);
                } else {
                    raw[u] = make_int4(0, 0, 0, 0);
                }
            }
#pragma unroll
            for (int u = 0; u < kNormBatch; ++u) {
                if (row0 + u * kRows >= row_end) break;
                const int row = row0 + u * kRows + sub;
                const bool is_q = row < p.hq, is_v = row >= p.hq + p.hkv;
                const __nv_bfloat16 *w = is_q ? p.q_weight : p.k_weight;
                int4 res = raw[u];
                float x[8];
                unpack8(raw[u], x);
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
                for (int off = kLanes / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
                if (w) {
                    const float rs = rsqrtf(ss * (1.f / D) + p.eps);
                    float wf[8];
                    unpack8(*reinterpret_cast<const int4 *>(w + l * 8), wf);
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = x[i] * rs * wf[i];
                }
                if (p.rot_dim > 0) {
                    float y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], mate);
                    if (rotated) {
                        if (p.interleaved) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) y[i] = x[i ^ 1];
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] = fmaf(y[i], sn[i], x[i] * cs[i]);
                    }
                }
                if (row >= row_end) continue;
                if (!is_v) res = pack8(x);
                if (is_q) {
                    *reinterpret_cast<int4 *>(p.q_out + (row_tok * p.hq + row) * D + l * 8) = res;
                } else {
                    const int h = row - p.hq - (is_v ? p.hkv : 0);
                    if (p.k_out && !is_v) *reinterpret_cast<int4 *>(p.k_out + (row_tok * p.hkv + h) * D + l * 8) = res;
                    if (page >= 0)
                        *reinterpret_cast<int4 *>((is_v ? p.v_pool : p.k_pool) +
                                                  (((int64_t)page * p.hkv + h) * kSubTokens + slot % kSubTokens) * D +
                                                  l * 8) = res;
                }
            }
        }
    }
}

cudaError_t launch_qk_norm_rope(const NormRopeParams &p, int head_dim, int batch, cudaStream_t stream) {
    const int sms = sm_count_current_device();
    if (sms <= 0) return cudaErrorInvalidDevice;
    // Few tokens are spread over warps by their rows (one load each: 16 tokens of 32 rows
    // take 64 warps); many tokens keep a warp per token, which computes its cosines once.
    const int rows = p.hq + p.hkv + (p.v ? p.hkv : 0);
    const int step = (head_dim == 128 ? 2 : 4) * kNormBatch;
    const int64_t tokens = (int64_t)batch * p.tokens;
    const int64_t warps = (int64_t)sms * 4 * kNormWarps;
    const int steps = (rows + step - 1) / step;
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(steps, warps / tokens));
    const int rows_per_item = (int)((steps + want - 1) / want) * step;
    const int chunks = (rows + rows_per_item - 1) / rows_per_item;
    const int64_t ctas = (tokens * chunks + kNormWarps - 1) / kNormWarps;
    const int grid = (int)std::min<int64_t>(ctas, (int64_t)sms * 64);
    return launch_dependent(head_dim == 128 ? qk_norm_rope_kernel<128> : qk_norm_rope_kernel<64>, grid, kNormWarps * 32,
                            0, stream, p, batch, rows_per_item, chunks);
}

}  // namespace sfi
