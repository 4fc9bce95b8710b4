// Which positions a block of new tokens sees through a sink and a sliding window, and the list of
// pages that holds them: the sink's pages, then those of the window, without what lies between.
#pragma once

#include "sfi_device.cuh"
#include "sfi_internal.h"

namespace sfi {

// Tokens at positions p0 .. p1 see j <= p with j < S or j > p - W. A slot v of the list holds position
// v in the sink's pages (v < 16 sink_pages) and v + skip behind them; the positions that are between a
// sink that ends inside a page and the window count as sink slots, and no row sees them.
struct WindowSpan {
    int sink_pages;  // pages of the sink (those that any of the tokens sees)
    int skip;        // positions left out between the two parts, whole pages
    int pages;       // pages of the list
    int slots;       // slots up to the last position seen

    __device__ __forceinline__ WindowSpan(int p0, int p1, int sink, int recent) {
        sink_pages = (min(sink, p1 + 1) + kSubTokens - 1) / kSubTokens;
        const int lo = max(sink, p0 + 1 - recent);  // lowest window position of any row
        pages = sink_pages;
        skip = 0;
        slots = min(sink, p1 + 1);
        if (lo <= p1) {
            const int first = max(sink_pages, lo / kSubTokens);
            pages += p1 / kSubTokens + 1 - first;
            skip = (first - sink_pages) * kSubTokens;
            slots = p1 + 1 - skip;
        }
    }
    // The page (index in the request's row of the table) behind page v of the list.
    __device__ __forceinline__ int page(int v) const { return v < sink_pages ? v : v + skip / kSubTokens; }
};

// The slots that the token at position p sees: [0, sink) and [lo, hi).
struct RowWindow {
    int sink, lo, hi;
    __device__ __forceinline__ RowWindow(int p, int s, int w, const WindowSpan &span) {
        sink = min(s, p + 1);
        const int first = max(s, p + 1 - w);
        const bool any = first <= p;
        lo = any ? first - span.skip : 0;
        hi = any ? p + 1 - span.skip : 0;
    }
    __device__ __forceinline__ bool sees(int v) const { return v < sink || (v >= lo && v < hi); }
    // The same of the slots v .. v + 31, a bit for each.
    __device__ __forceinline__ uint32_t sees32(int v) const {
        return below32(sink - v) | (below32(hi - v) & ~below32(lo - v));
    }
    static __device__ __forceinline__ uint32_t below32(int n) {
        return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
    }
};

// Whether every token of p0 .. p1 sees all of the slots [v, v + n): they end before the first token's
// last one, and begin in the sink, or behind the start of the last token's window (or that window
// begins where the sink ends).
__device__ __forceinline__ bool all_see(int v, int n, const RowWindow &first, const RowWindow &last) {
    return v + n <= first.sink || (v + n <= first.hi && (v >= last.lo || last.lo <= first.sink));
}

// ---- rows whose output is not finite ------------------------------------------------------------------------
// A matrix product makes NaN of a masked weight (zero) and a NaN or infinity of V. So a row that came out so is looked
// at again: where nothing that it does not see can have spoiled it, its output is what the arithmetic gives, and stays
// (a NaN early in a prompt is seen by all later rows); the others are computed again from what they see. What rows of a
// block do not see, but were multiplied with, lies at the edges of their windows: a few hundred positions at most,
// however long the context is.

// Weights as two bf16 terms each. The first is the weight cut off, so that the second, with 2^-23 of the weight added,
// is above zero when the weight is: an infinity of V stays one in both products.
__device__ __forceinline__ void split_bf16x2(float a, float b, uint32_t &hi, uint32_t &lo) {
    constexpr float kMore = 1.f + 0x1p-23f;
    const uint32_t x = __float_as_uint(a) & 0xffff0000u, y = __float_as_uint(b) & 0xffff0000u;
    hi = x >> 16 | y;
    lo = pack_bf16x2(fmaf(a, kMore, -__uint_as_float(x)), fmaf(b, kMore, -__uint_as_float(y)));
}

// A pair of bf16 values with a NaN or infinity among them.
__device__ __forceinline__ bool nonfinite_pair(uint32_t v) {
    return (v & 0x7f80u) == 0x7f80u || (v & 0x7f800000u) == 0x7f800000u;
}

// Whether V holds a NaN or infinity in one of the slots [from, to) that the row of this lane does not see (by a whole
// warp, a row in each lane).
template <int D>
__device__ __forceinline__ bool hidden_nonfinite(const WindowParams &p, int r, int kvh, const WindowSpan &span, int from,
                                                 int to, const RowWindow &win) {
    const int lane = threadIdx.x & 31;
    bool hit = false;
    for (int v0 = from / kSubTokens * kSubTokens; v0 < to; v0 += kSubTokens) {
        const int page = p.page_table[(int64_t)r * p.max_pages + span.page(v0 / kSubTokens)];
        if (page < 0 || page >= p.num_pages) continue;
        const int64_t row = ((int64_t)page * p.hkv + kvh) * kSubTokens;
        const uint32_t *v = reinterpret_cast<const uint32_t *>(p.v_pool + row * D) + lane;
        uint32_t odd = 0;
#pragma unroll
        for (int j = 0; j < kSubTokens; ++j)
#pragma unroll
            for (int k = 0; k < D / 64; ++k) odd |= nonfinite_pair(v[j * (D / 2) + 32 * k]) ? 1u << j : 0u;
        odd = __reduce_or_sync(0xffffffffu, odd);
        for (; odd; odd &= odd - 1) {
            const int at = v0 + __ffs(odd) - 1;
            hit |= at >= from && at < to && !win.sees(at);
        }
    }
    return hit;
}

// The rows `need` (a bit each) of the 16 rows from row0 on (row = token * G + head of one KV head) computed again from
// the positions that each sees, by a whole warp, with weights of one or two bf16 terms. Lane i < 16 has row i's maximum
// m (log2 units) and sum l. Values that are not finite stay out of the product and are added to the rows that see them.
// Writes the values 4 piece0 .. 4 piece1 - 1 of the 16 x D. Fragments come straight from memory: 16 rows of 131072
// positions take 30 ms, 256 rows of eight warps 120 (the prompt kernel's other roles wait two seconds for them, some two
// million positions).
template <int D, bool TWO_TERMS>
__device__ __forceinline__ void window_rows(const WindowParams &p, int r, int kvh, int L, int n, int row0, uint32_t need,
                                            float m, float l, int piece0, int piece1) {
    constexpr int kDims = 64, kTiles = kDims / 8;  // dims of a pass (few registers: the caller keeps its own)
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, G = p.group;
    int pos[2];  // of rows g and g + 8
    float base[2], inv[2];
    const __nv_bfloat16 *q[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int i = g + 8 * half, row = row0 + i, tok = row / G;
        const bool wanted = need >> i & 1u;
        pos[half] = wanted ? L - n + tok : -1;
        const float top = __shfl_sync(0xffffffffu, m, i), sum = __shfl_sync(0xffffffffu, l, i);
        base[half] = top == -INFINITY ? 0.f : top;
        inv[half] = sum == 0.f ? 0.f : 1.f / sum;
        const int64_t head = (int64_t)kvh * G + row % G;
        q[half] = p.q + ((int64_t)r * p.tokens + tok) * p.q_stride + head * D + 2 * t;
    }
    const int high = __reduce_max_sync(0xffffffffu, max(pos[0], pos[1]));
    const int low = __reduce_min_sync(0xffffffffu, min(pos[0] < 0 ? high : pos[0], pos[1] < 0 ? high : pos[1]));
    const int sink = min(p.sink, high + 1), window = max(sink, low + 1 - p.recent);
#pragma unroll 1
    for (int d0 = 0; d0 < D; d0 += kDims) {
        float o[kTiles][4];
#pragma unroll
        for (int i = 0; i < kTiles; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
#pragma unroll 1
        for (int k0 = 0; k0 <= high; k0 += kSubTokens) {
            if (k0 >= sink && k0 + kSubTokens <= window) k0 = window / kSubTokens * kSubTokens;
            if (k0 > high) break;
            const int page = p.page_table[(int64_t)r * p.max_pages + k0 / kSubTokens];
            if (page < 0 || page >= p.num_pages) continue;
            const int64_t at = ((int64_t)page * p.hkv + kvh) * kSubTokens * D;
            float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            const __nv_bfloat16 *k = p.k_pool + at + g * D + 2 * t;
#pragma unroll
            for (int ks = 0; ks < D; ks += 16) {
                uint32_t qa[4];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    qa[half] = pos[half] < 0 ? 0u : *reinterpret_cast<const uint32_t *>(q[half] + ks);
                    qa[2 + half] = pos[half] < 0 ? 0u : *reinterpret_cast<const uint32_t *>(q[half] + ks + 8);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    mma_bf16_16816(s[h], qa[0], qa[1], qa[2], qa[3],
                                   *reinterpret_cast<const uint32_t *>(k + h * 8 * D + ks),
                                   *reinterpret_cast<const uint32_t *>(k + h * 8 * D + ks + 8));
            }
            uint32_t see[2], pa[2][2], pb[2][2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int end = pos[half] + 1;
                see[half] = RowWindow::below32(min(p.sink, end) - k0) |
                            (RowWindow::below32(end - k0) & ~RowWindow::below32(max(0, end - p.recent) - k0));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float w[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        w[e] = see[half] >> (8 * h + 2 * t + e) & 1u
                                   ? fast_exp2(fmaf(s[h][2 * half + e], p.scale_log2, -base[half]))
                                   : 0.f;
                    if (TWO_TERMS) split_bf16x2(w[0], w[1], pa[half][h], pb[half][h]);
                    else pa[half][h] = pack_bf16x2(w[0], w[1]);
                }
            }
            const uint16_t *v = reinterpret_cast<const uint16_t *>(p.v_pool + at) + 2 * t * D + d0 + g;
            bool odd = false;
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
                uint32_t b[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t x = v[h * 8 * D + i * 8], y = v[(h * 8 + 1) * D + i * 8];
                    if ((x & 0x7f80u) == 0x7f80u) odd = true, x = 0;
                    if ((y & 0x7f80u) == 0x7f80u) odd = true, y = 0;
                    b[h] = x | y << 16;
                }
                mma_bf16_16816(o[i], pa[0][0], pa[1][0], pa[0][1], pa[1][1], b[0], b[1]);
                if (TWO_TERMS) mma_bf16_16816(o[i], pb[0][0], pb[1][0], pb[0][1], pb[1][1], b[0], b[1]);
            }
            if (!__any_sync(0xffffffffu, odd)) continue;
#pragma unroll 1
            for (int j = 0; j < kSubTokens; ++j)
#pragma unroll
                for (int i = 0; i < kTiles; ++i) {
                    const uint32_t x = *reinterpret_cast<const uint32_t *>(p.v_pool + at + j * D + d0 + i * 8 + 2 * t);
                    if (!nonfinite_pair(x)) continue;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float f = __uint_as_float(e ? x & 0xffff0000u : x << 16);
                        if (fabsf(f) < INFINITY) continue;
                        if (see[0] >> j & 1u) o[i][e] += f;
                        if (see[1] >> j & 1u) o[i][2 + e] += f;
                    }
                }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int i = g + 8 * half, row = row0 + i;
            if (pos[half] < 0) continue;
            __nv_bfloat16 *out = p.out + (((int64_t)r * p.tokens + row / G) * p.hq + (int64_t)kvh * G + row % G) * D;
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
                const int d = d0 + j * 8 + 2 * t, piece = i * (D / 4) + d / 4;
                if (piece >= piece0 && piece < piece1)
                    *reinterpret_cast<uint32_t *>(out + d) =
                        pack_bf16x2(o[j][2 * half] * inv[half], o[j][2 * half + 1] * inv[half]);
            }
        }
    }
}

// What a warp does about rows of a block (tokens at p0 .. p1) that came out not finite: those of row0 + lane where `odd`
// is set, with their maxima and sums. Writes the values 4 piece0 .. 4 piece1 - 1 of the 32 x D. (Not inline, and in
// passes of 64 dims: inline, or with all dims at once, it cost the prompt kernel registers and 1 to 6% of its speed.)
template <int D, bool TWO_TERMS>
__device__ __noinline__ void mend_rows(const WindowParams &p, int r, int kvh, int L, int n, int p0, int p1, int row0,
                                       bool odd, float m, float l, int piece0, int piece1) {
    const int lane = threadIdx.x & 31, G = p.group;
    const WindowSpan span(p0, p1, p.sink, p.recent);
    const RowWindow first(min(L - n + row0 / G, p1), p.sink, p.recent, span);
    const RowWindow last(min(L - n + (row0 + 31) / G, p1), p.sink, p.recent, span);
    const RowWindow win(min(L - n + (row0 + lane) / G, p1), p.sink, p.recent, span);
    // slots that not all of the rows see: [first.sink, last.lo) and [first.hi, slots)
    const int to = first.hi > 0 ? min(max(first.sink, last.lo), span.slots) : span.slots;
    const bool hit = hidden_nonfinite<D>(p, r, kvh, span, first.sink, to, win) |
                     hidden_nonfinite<D>(p, r, kvh, span, max(to, first.hi), span.slots, win);
    // (a score that is not finite leaves nothing finite)
    const uint32_t need = __ballot_sync(0xffffffffu, odd && hit && l < INFINITY);
    for (int half = 0; half < 32; half += 16) {
        const float top = __shfl_sync(0xffffffffu, m, half | (lane & 15));
        const float sum = __shfl_sync(0xffffffffu, l, half | (lane & 15));
        if (need >> half & 0xffffu)
            window_rows<D, TWO_TERMS>(p, r, kvh, L, n, row0 + half, need >> half & 0xffffu, top, sum,
                                      piece0 - half * (D / 4), piece1 - half * (D / 4));
    }
}

}  // namespace sfi
