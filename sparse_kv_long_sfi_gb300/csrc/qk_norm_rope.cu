// Head norm and position rotation of the new tokens' Q and K, written (with V) to where
// the attention calls read them: one pass over the projections' output.
//
// y = rotate(x * w / sqrt(mean(x^2) + eps)) per head row x of D values, in fp32, rounded
// once to bf16. Pair i turns by pos * turns[i] / 2^64 whole turns: the 64-bit product
// wraps modulo one turn by itself, so nothing of the angle is lost at far positions and
// no table of cosines is read; the upper 32 bits give the fraction of the turn to 2^-32.
//
// Bound by HBM: each row is read and written once. A row is held by D / 8 lanes, a warp takes
// one token's rows two (four at D = 64) at a time with four such loads in flight. Norm weight
// and rotation of a token become two factors per dim, once for its Q and once for its K rows:
// y = (x A + x' B) / rms, x' the other member of the pair. Where whole heads turn in split
// halves a lane holds both members (dims 4 l .. and D/2 + 4 l ..); otherwise it holds eight
// dims in a row and fetches x' from its mate lane. Three CTAs per SM (80 registers) keep enough
// loads in flight: 2 x 8192 tokens of 32/8/128 heads take 73 us (5.5 TB/s; two CTAs 12 us longer,
// four, which spill, 4 us). The variant for the other rotations has two CTAs per SM: 95 us for half
// of each head in split halves, 91 for adjacent pairs, whose members lie in one lane.
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

// A lane's eight values of a row: in a row, or four of each half.
template <int D, bool HALVES>
__device__ __forceinline__ int4 load_row(const __nv_bfloat16 *row, int l) {
    if constexpr (!HALVES) return *reinterpret_cast<const int4 *>(row + l * 8);
    const int2 a = *reinterpret_cast<const int2 *>(row + l * 4), b = *reinterpret_cast<const int2 *>(row + D / 2 + l * 4);
    return make_int4(a.x, a.y, b.x, b.y);
}
template <int D, bool HALVES>
__device__ __forceinline__ void store_row(__nv_bfloat16 *row, int l, int4 v) {
    if constexpr (!HALVES) {
        *reinterpret_cast<int4 *>(row + l * 8) = v;
    } else {
        *reinterpret_cast<int2 *>(row + l * 4) = make_int2(v.x, v.y);
        *reinterpret_cast<int2 *>(row + D / 2 + l * 4) = make_int2(v.z, v.w);
    }
}

// One warp takes rows [chunk * rows_per_item, ...) of one token's q, k and v rows.
template <int D, bool HALVES>
__global__ void __launch_bounds__(kNormWarps * 32, HALVES ? 3 : 2) qk_norm_rope_kernel(const NormRopeParams p, int batch,
                                                                       int rows_per_item, int chunks) {
    constexpr int kLanes = D / 8;          // lanes per row
    constexpr int kRows = 32 / kLanes;     // rows per load
    __shared__ float2 s_cs[kNormWarps][D / 2];  // (cos, sin) of the token's pairs
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / kLanes, l = lane % kLanes;
    const int64_t items = (int64_t)batch * p.tokens * chunks;
    const int half = p.rot_dim / 2;
    const bool rotated = HALVES || l * 8 < p.rot_dim;
    const bool second = l * 8 >= half;  // this lane's dims are the second members (split halves)
    // the lane that holds the other members of this lane's pairs (split halves)
    const int mate = p.interleaved || !rotated ? lane : (second ? lane - half / 8 : lane + half / 8);
    // (no early release of dependents: an attention launch may be allowed to read the pages ahead)
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
            bad = bad || L < n || (p.page_table && L > p.max_pages * kSubTokens);
            slot = L - n + t;
        }
        if (bad) {
            if (lane == 0 && t == 0 && chunk == 0) report(p.dev_status, SFI_DEV_BAD_LEN);
            continue;
        }
        if (t >= n) continue;
        const int64_t row_tok = (int64_t)r * p.tokens + t;
        if (p.page_table) {
            page = p.page_table[(int64_t)r * p.max_pages + slot / kSubTokens];
            if (page < 0 || page >= p.num_pages) {
                page = -1;
                if (lane == 0 && chunk == 0) report(p.dev_status, SFI_DEV_BAD_PAGE);
            }
        }
        // the token's rotations
        float cs[8], sn[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
        if (HALVES || p.rot_dim > 0) {
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
                const int pair = HALVES ? l * 4 + (i & 3) : (p.interleaved ? e / 2 : (second ? e - half : e));
                if (rotated) {
                    const float2 v = s_cs[warp][pair];
                    cs[i] = v.x;
                    // the sign of the mate's share: minus for the first member of a pair
                    sn[i] = (HALVES ? i < 4 : (p.interleaved ? (i & 1) == 0 : !second)) ? -v.y : v.y;
                }
            }
        }
        // rows [first, last) of the item within a group of `heads` rows that starts at row `from`
        const int lo = chunk * rows_per_item, hi = lo + rows_per_item;
        auto rows_of = [&](int from, int heads, int &first, int &last) {
            first = min(max(lo - from, 0), heads);
            last = min(max(hi - from, 0), heads);
        };
        // norm and rotation of rows [first, last); put(head, value) stores one
        auto turn_rows = [&](const __nv_bfloat16 *src, const __nv_bfloat16 *weight, int first, int last, auto put) {
            if (first >= last) return;
            float A[8], B[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) A[i] = 1.f;
            if (weight) unpack8(load_row<D, HALVES>(weight, l), A);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float w = HALVES ? A[i ^ 4] : (p.interleaved ? A[i ^ 1] : __shfl_sync(0xffffffffu, A[i], mate));
                B[i] = w * sn[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) A[i] *= cs[i];
            for (int row0 = first; row0 < last; row0 += kRows * kNormBatch) {
                int4 raw[kNormBatch];
#pragma unroll
                for (int u = 0; u < kNormBatch; ++u) {
                    const int row = row0 + u * kRows + sub;
                    raw[u] = make_int4(0, 0, 0, 0);
                    if (row < last) raw[u] = load_row<D, HALVES>(src + (int64_t)row * D, l);
                }
#pragma unroll
                for (int u = 0; u < kNormBatch; ++u) {
                    if (row0 + u * kRows >= last) break;
                    const int row = row0 + u * kRows + sub;
                    float x[8], y[8];
                    unpack8(raw[u], x);
                    float rs = 1.f;
                    if (weight) {
                        float ss = 0.f;
#pragma unroll
                        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
                        for (int off = kLanes / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
                        rs = rsqrtf(ss * (1.f / D) + p.eps);
                    }
                    if (HALVES || p.interleaved) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) y[i] = x[HALVES ? i ^ 4 : i ^ 1];
                    } else if (p.rot_dim > 0) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], mate);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (rotated && (HALVES || p.rot_dim > 0))
                            x[i] = fmaf(y[i], B[i], x[i] * A[i]) * rs;
                        else
                            x[i] = x[i] * A[i] * rs;
                    }
                    if (row < last) put(row, pack8(x));
                }
            }
        };
        int first, last;
        rows_of(0, p.hq, first, last);
        turn_rows(p.q + row_tok * p.q_stride, p.q_weight, first, last, [&](int h, int4 v) {
            store_row<D, HALVES>(p.q_out + (row_tok * p.hq + h) * D, l, v);
        });
        const int64_t page_row = ((int64_t)page * p.hkv * kSubTokens + slot % kSubTokens) * D;
        rows_of(p.hq, p.hkv, first, last);
        turn_rows(p.k + row_tok * p.k_stride, p.k_weight, first, last, [&](int h, int4 v) {
            if (p.k_out) store_row<D, HALVES>(p.k_out + (row_tok * p.hkv + h) * D, l, v);
            if (page >= 0) store_row<D, HALVES>(p.k_pool + page_row + (int64_t)h * kSubTokens * D, l, v);
        });
        if (p.v && page >= 0) {
            rows_of(p.hq + p.hkv, p.hkv, first, last);
            const __nv_bfloat16 *src = p.v + row_tok * p.v_stride + l * 8;
            __nv_bfloat16 *dst = p.v_pool + page_row + l * 8;
            for (int row0 = first + sub; row0 < last; row0 += kRows * kNormBatch) {
                int4 raw[kNormBatch];
#pragma unroll
                for (int u = 0; u < kNormBatch; ++u)
                    if (row0 + u * kRows < last) raw[u] = *reinterpret_cast<const int4 *>(src + (int64_t)(row0 + u * kRows) * D);
#pragma unroll
                for (int u = 0; u < kNormBatch; ++u)
                    if (row0 + u * kRows < last)
                        *reinterpret_cast<int4 *>(dst + (int64_t)(row0 + u * kRows) * kSubTokens * D) = raw[u];
            }
        }
    }
}

cudaError_t launch_qk_norm_rope(const NormRopeParams &p, int head_dim, int batch, cudaStream_t stream) {
    const int sms = sm_count_current_device();
    if (sms <= 0) return cudaErrorInvalidDevice;
    // Few tokens are spread over warps by their rows (one round of loads each: 16 tokens of 32
    // rows take 64 warps and 4.2 us, 6.7 us with a warp per token); many tokens keep a warp per
    // token, which computes its cosines once.
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
    // both members of a pair in a lane: 73 us for 2 x 8192 tokens of 32/8/128 heads, 96 by shuffles
    const bool halves = p.rot_dim == head_dim && !p.interleaved;
    auto kernel = head_dim == 128 ? (halves ? qk_norm_rope_kernel<128, true> : qk_norm_rope_kernel<128, false>)
                                  : (halves ? qk_norm_rope_kernel<64, true> : qk_norm_rope_kernel<64, false>);
    return launch_dependent(kernel, grid, kNormWarps * 32, 0, stream, p, batch, rows_per_item, chunks);
}

}  // namespace sfi
