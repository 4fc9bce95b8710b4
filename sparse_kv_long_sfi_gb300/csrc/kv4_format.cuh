// The 4-bit block format of one (page, KV head) (documented at sfi_paged_kv4): offsets,
// conversions between codes and values, and the group quantisation.
#pragma once

#include <cuda_fp16.h>

#include "sfi_device.cuh"
#include "sfi_internal.h"

namespace sfi {

template <int D>
struct Kv4 {
    static constexpr int kBlock = 18 * D;       // bytes of a block
    static constexpr int kKRow = D / 2;         // bytes of a K row's codes
    static constexpr int kGroups = D / 16;      // scales of a row
    static constexpr int kKScale = 8 * D;       // offsets within the block
    static constexpr int kVCode = 9 * D;
    static constexpr int kVScale = 17 * D;
    static constexpr int kVScaleT = D / 4;      // bytes of the V scales of four tokens
    static constexpr int kQuads = D / 64;       // 512-byte runs of V codes (64 dims each)
};

// Eight e2m1 codes -> four pairs of fp16 (byte i: low four bits in the lower half of h[i]).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// Two e4m3 scales (low byte first) -> a pair of fp16.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint16_t s) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(s));
    return h;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// v rounded to 16 significant bits. A bf16 value over a step of a few bits is either exactly
// halfway between two codes (or two e4m3 scales) or at least 2^-8.4 of itself away from there:
// with x = X 2^a (X < 256), the step S 2^b (S < 16, or 3 for the scale itself) and the halfway
// point T 2^c (T < 32), |X 2^k - T S| is a whole number in the unit where both sides are, hence
// at least 1 of at most 480. So the value times the step's fp32 reciprocal (off by 2^-21)
// decides every rounding like the exact quotient once its last bits are rounded away.
__device__ __forceinline__ float round16(float v) {
    return __uint_as_float((__float_as_uint(v) + 0x80u) & 0xffffff00u);
}

// 1 / v to 2^-23 of itself.
__device__ __forceinline__ float reciprocal(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// The e4m3 scale of a group whose largest magnitude is amax (inv6g: 1 / (6 g)); nearest even,
// at most 448.
__device__ __forceinline__ uint32_t group_scale(float amax, float inv6g) {
    uint16_t s;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s) : "f"(0.f), "f"(round16(amax * inv6g)));
    return s & 0xffu;
}

constexpr uint32_t kE4m3Nan = 0x7fu;

__device__ __forceinline__ float e4m3_to_f32(uint32_t s) {
    const uint32_t h = e4m3x2_to_f16((uint16_t)s);
    return __low2float(*reinterpret_cast<const __half2 *>(&h));
}

// Eight values over the group's step -> eight e2m1 codes (value i in bits 4i..4i+3), by way
// of fp16: its 11 bits do for the codes what round16 does for the scale.
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float (&y)[8]) {
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t.reg .b32 h0, h1, h2, h3;\n\t"
        "cvt.rn.f16x2.f32 h0, %2, %1;\n\t"
        "cvt.rn.f16x2.f32 h1, %4, %3;\n\t"
        "cvt.rn.f16x2.f32 h2, %6, %5;\n\t"
        "cvt.rn.f16x2.f32 h3, %8, %7;\n\t"
        "cvt.rn.satfinite.e2m1x2.f16x2 b0, h0;\n\t"
        "cvt.rn.satfinite.e2m1x2.f16x2 b1, h1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f16x2 b2, h2;\n\t"
        "cvt.rn.satfinite.e2m1x2.f16x2 b3, h3;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(w)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return w;
}

__device__ __forceinline__ void bf16x8_to_f32(int4 v, float (&x)[8]) {
    const uint32_t w[4] = {(uint32_t)v.x, (uint32_t)v.y, (uint32_t)v.z, (uint32_t)v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ int4 f32x8_to_bf16(const float (&x)[8]) {
    return make_int4((int)pack_bf16x2(x[0], x[1]), (int)pack_bf16x2(x[2], x[3]), (int)pack_bf16x2(x[4], x[5]),
                     (int)pack_bf16x2(x[6], x[7]));
}

// 16-byte unit u of the V codes of a block (memory order) holds, for tokens 4t..4t+3 and
// j = 4 * quad .. 4 * quad + 3, the dims 16 j + g (bytes 0 and 2 of word j) and 16 j + g + 8
// (bytes 1 and 3); bytes 0 and 1 are tokens 4t, 4t+1, bytes 2 and 3 tokens 4t+2, 4t+3.
struct VUnit {
    int quad, g, t;
    __device__ __forceinline__ explicit VUnit(int u)
        : quad(u >> 5), g(((u >> 3) & 3) * 2 + (u & 1)), t((u >> 1) & 3) {}
};

// Codes of four tokens' dims 16 j .. 16 j + 15 (in[i][c]: token 4t + i, dims 16 j + 8 c ..,
// one code in four bits) <-> the words of j in the units g = 0 .. 7 of t.
__device__ __forceinline__ void v_pack(const uint32_t (&in)[4][2], uint32_t (&out)[8]) {
    uint32_t even[2][2], odd[2][2];  // [pair of tokens][c]: byte k holds dim 2k (2k + 1) of both
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint32_t a = in[2 * h][c], b = in[2 * h + 1][c];
            even[h][c] = (a & 0x0f0f0f0fu) | ((b & 0x0f0f0f0fu) << 4);
            odd[h][c] = ((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);
        }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t sel = k | (4 + k) << 4;
        out[2 * k] = __byte_perm(__byte_perm(even[0][0], even[0][1], sel), __byte_perm(even[1][0], even[1][1], sel), 0x5410);
        out[2 * k + 1] = __byte_perm(__byte_perm(odd[0][0], odd[0][1], sel), __byte_perm(odd[1][0], odd[1][1], sel), 0x5410);
    }
}
__device__ __forceinline__ void v_unpack(const uint32_t (&out)[8], uint32_t (&in)[4][2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int byte = 2 * h + c;
            const uint32_t sel = byte | (4 + byte) << 4;
            const uint32_t even = __byte_perm(__byte_perm(out[0], out[2], sel), __byte_perm(out[4], out[6], sel), 0x5410);
            const uint32_t odd = __byte_perm(__byte_perm(out[1], out[3], sel), __byte_perm(out[5], out[7], sel), 0x5410);
            in[2 * h][c] = (even & 0x0f0f0f0fu) | ((odd & 0x0f0f0f0fu) << 4);
            in[2 * h + 1][c] = ((even >> 4) & 0x0f0f0f0fu) | (odd & 0xf0f0f0f0u);
        }
}

// Byte offset, within a block's V codes, of word j of unit g of t.
__device__ __forceinline__ int v_word(int j, int g, int t) {
    return (j >> 2) * 512 + (g >> 1) * 128 + t * 32 + (g & 1) * 16 + (j & 3) * 4;
}

}  // namespace sfi
