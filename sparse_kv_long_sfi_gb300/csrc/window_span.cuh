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

// One output row computed again key by key, by a whole warp (D / 32 values per lane): a matrix product
// makes NaN of a masked weight (zero) and a NaN or infinity of V, here hidden positions are not read.
// m: the row's running maximum in log2 units, l: its sum. Writes the dims [d0, d1).
template <int D>
__device__ __forceinline__ void window_row(const WindowParams &p, int r, int token, int head, int pos, float m, float l,
                                        int d0, int d1) {
    constexpr int kEach = D / 32;
    const int lane = threadIdx.x & 31, kvh = head / p.group;
    const int64_t row = (int64_t)r * p.tokens + token;
    float q[kEach], acc[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        q[i] = __bfloat162float(p.q[row * p.q_stride + (int64_t)head * D + lane * kEach + i]);
        acc[i] = 0.f;
    }
    const int sink = min(p.sink, pos + 1);
    for (int j = 0; j <= pos; ++j) {
        if (j == sink) j = max(j, pos + 1 - p.recent);
        if (j > pos) break;
        const int page = p.page_table[(int64_t)r * p.max_pages + j / kSubTokens];
        if (page < 0 || page >= p.num_pages) continue;
        const int64_t at = (((int64_t)page * p.hkv + kvh) * kSubTokens + j % kSubTokens) * D + lane * kEach;
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < kEach; ++i) x += q[i] * __bfloat162float(p.k_pool[at + i]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        const float w = fast_exp2(x * p.scale_log2 - m);
#pragma unroll
        for (int i = 0; i < kEach; ++i) acc[i] += w * __bfloat162float(p.v_pool[at + i]);
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int d = lane * kEach + i;
        if (d >= d0 && d < d1) p.out[(row * p.hq + head) * D + d] = __float2bfloat16(acc[i] / l);
    }
}

}  // namespace sfi
