// fp4_quant.cuh -- microscaled 4-bit quantisation of 32 columns in a thread's registers,
// shared by the quantiser and by the product that quantises its own tokens, so that both take
// every decision with the same operations.
#pragma once

#include <type_traits>

#include "fp4.cuh"
#include "sm100.cuh"

namespace mx {
namespace fp4 {

// 8 values to 8 E2M1 codes, the first in the lowest nibble
__device__ __forceinline__ uint32_t pack8(const float2* v) {
    uint32_t o;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(o)
        : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y));
    return o;
}

__device__ __forceinline__ uint32_t e4m3_bits(float v) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
    return r & 0xFFu;
}
__device__ __forceinline__ float e4m3_value(uint32_t b) {
    uint32_t h;
    const uint16_t in = uint16_t(b);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(in));
    return __half2float(__ushort_as_half(uint16_t(h & 0xFFFFu)));
}
__device__ __forceinline__ float e8m0_value(uint32_t b) {
    if (b == 0xFFu) return __uint_as_float(0x7FC00000u);
    return __uint_as_float(b == 0 ? 0x00400000u : b << 23);     // 2^(b - 127); 2^-127 is subnormal
}

constexpr uint32_t kInfBits = 0x7F800000u;

// The 16-column format.  fl(x / d) by the published reciprocal-and-correct division
// (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990): r = fl(1/d), q = fl(x r), e = x - q d exactly by one fma, then
// fl(q + e r).  What is needed of the quotient is only the side of the seven E2M1
// boundaries on which it lies; over all 2^23 significands of d and the x next to
// each boundary, the corrected quotient and the IEEE division agree on that; the same
// holds for a / (6 g) and the boundaries of E4M3.  e is a multiple of the unit of q d and has to
// stay one of 2^-149: next to the smallest boundary (1/4) that takes d >= 2^-101, and s may be 2^-9.
// So below g = 2^-90 the whole division is done with x and g 2^32 times as large, which
// leaves every quotient as it is (no bit is lost: s g is normal).  That is a path of its own (SMALL),
// since a factor in the usual one costs it registers (fp32, 4096 x 8192: 26.4 to 29.4 us).
// Where a scale saturated, values beyond 16 d are brought to 16 d first: their codes are 6 either way, and
// x r cannot overflow.
constexpr float kSmallScale = 0x1p-90f, kSmallUp = 0x1p32f;
struct MatrixScale {
    float g, g6, r6;                               // g, fl(6 g), fl(1 / fl(6 g)); of the scaled matrix if small
    bool small;
};
__device__ __forceinline__ MatrixScale matrix_scale(float g) {
    const bool small = g < kSmallScale;
    if (small) g = __fmul_rn(g, kSmallUp);
    const float g6 = __fmul_rn(6.0f, g);
    return {g, g6, __frcp_rn(g6), small};
}

__device__ __forceinline__ float quick_div(float x, float d, float r) {
    const float q = __fmul_rn(x, r);
    return __fmaf_rn(__fmaf_rn(-q, d, x), r, q);
}

// s as its byte; d and r of the values, or of the scaled ones
template <bool SMALL>
__device__ __forceinline__ uint32_t scale16(uint32_t amax, const MatrixScale& m, float& d, float& r, bool& beyond) {
    if (amax >= kInfBits) {
        d = r = __uint_as_float(0x7FC00000u);
        beyond = false;
        return 0x7Fu;
    }
    // beyond 1024 (6 g) the scale saturates however the quotient is rounded
    const float a = SMALL ? __fmul_rn(__uint_as_float(amax), kSmallUp) : __uint_as_float(amax);
    const uint32_t s = e4m3_bits(a < __fmul_rn(1024.0f, m.g6) ? quick_div(a, m.g6, m.r6) : 1024.0f);
    d = __fmul_rn(e4m3_value(s), m.g);
    r = d > 0.0f ? __frcp_rn(d) : 0.0f;
    beyond = __fmul_rn(a, r) > 16.0f;
    return s;
}

// codes of the 16 values of a block with maximum amax; returns the scale's byte
template <bool SMALL>
__device__ __forceinline__ uint32_t quant_block(float2 (&v)[8], uint32_t amax, const MatrixScale& m, uint32_t* codes) {
    float d, r;
    bool beyond;
    const uint32_t s = scale16<SMALL>(amax, m, d, r, beyond);
    if constexpr (SMALL) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = make_float2(__fmul_rn(v[i].x, kSmallUp), __fmul_rn(v[i].y, kSmallUp));
    }
    if (beyond) {
        const float lim = __fmul_rn(16.0f, d);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = make_float2(fminf(fmaxf(v[i].x, -lim), lim), fminf(fmaxf(v[i].y, -lim), lim));
    }
    const float2 r2 = make_float2(r, r), nd = make_float2(-d, -d), z = make_float2(-0.0f, -0.0f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 q = sm100::fma2(v[i], r2, z);             // x r + (-0) = fl(x r)
        v[i] = sm100::fma2(sm100::fma2(q, nd, v[i]), r2, q);
    }
    codes[0] = pack8(v);
    codes[1] = pack8(v + 4);
    return s;
}

// The 32-column format: the scale is a power of two, so x 2^-e is exact (or so small
// that its code is zero).  Returns the biased exponent and sets inv = 2^-e.
__device__ __forceinline__ uint32_t scale32(uint32_t amax, float& inv) {
    if (amax >= kInfBits) {
        inv = 0.0f;
        return 0xFFu;
    }
    const int be = int(amax >> 23);               // floor(log2 a) + 127, 0 for subnormals and zero
    const int sb = max(be - 2, 0);                // e + 127
    inv = __uint_as_float(uint32_t(254 - sb) << 23);
    return uint32_t(sb);
}

// 32 columns [c0, c0 + 32) of a row as they lie in memory, zero past K; half j of them as fp32
// pairs, and its largest size as fp32 bits (NaN > infinity > finite, as integers).  16-bit types
// stay packed until a half is used, and take the maximum on packed pairs.
template <typename T> struct Columns {
    static constexpr bool kPacked = sizeof(T) == 2;
    alignas(16) uint32_t w[kPacked ? 16 : 32];   // moved as uint4

    template <bool ALIGNED> __device__ __forceinline__ void load(const T* row, int c0, int K) {
        if (ALIGNED && c0 + 32 <= K) {
#pragma unroll
            for (int i = 0; i < int(sizeof(T)) * 2; ++i)
                reinterpret_cast<uint4*>(w)[i] = reinterpret_cast<const uint4*>(row + c0)[i];
        } else if constexpr (kPacked) {
            const uint16_t* h = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int c = c0 + 2 * i;
                w[i] = (c < K ? uint32_t(h[c]) : 0u) | (c + 1 < K ? uint32_t(h[c + 1]) << 16 : 0u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = c0 + i < K ? __float_as_uint(row[c0 + i]) : 0u;
        }
    }
    __device__ __forceinline__ uint32_t amax(int j) const {
        uint32_t m = 0;
        if constexpr (kPacked) {
#pragma unroll
            for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[8 * j + i] & 0x7FFF7FFFu);
            const uint16_t h = uint16_t(max(m & 0xFFFFu, m >> 16));
            return __float_as_uint(to_f32(*reinterpret_cast<const T*>(&h))) & 0x7FFFFFFFu;
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) m = max(m, w[16 * j + i] & 0x7FFFFFFFu);
            return m;
        }
    }
    __device__ __forceinline__ void values(int j, float2 (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (!kPacked)
                v[i] = make_float2(__uint_as_float(w[16 * j + 2 * i]), __uint_as_float(w[16 * j + 2 * i + 1]));
            else if constexpr (std::is_same_v<T, __half>)
                v[i] = __half22float2(*reinterpret_cast<const __half2*>(&w[8 * j + i]));
            else
                v[i] = make_float2(__uint_as_float(w[8 * j + i] << 16), __uint_as_float(w[8 * j + i] & 0xFFFF0000u));
        }
    }
};

template <bool SMALL, typename T>
__device__ __forceinline__ uint32_t quant_two_blocks(const Columns<T>& x, const MatrixScale& m, uint32_t (&codes)[4]) {
    float2 v[8];
    x.values(0, v);
    const uint32_t s = quant_block<SMALL>(v, x.amax(0), m, codes);
    x.values(1, v);
    return s | (quant_block<SMALL>(v, x.amax(1), m, codes + 2) << 8);
}

// the codes of 32 columns and their scale bytes: two blocks' (16-column format, the second in
// bits 8..15) or one block's
template <int FMT, typename T>
__device__ __forceinline__ uint32_t quant_columns(const Columns<T>& x, const MatrixScale& m, uint32_t (&codes)[4]) {
    if constexpr (FMT == MX_FP4_E4M3_16) {
        return m.small ? quant_two_blocks<true>(x, m, codes) : quant_two_blocks<false>(x, m, codes);
    } else {
        float2 v[8];
        float inv;
        const uint32_t s = scale32(max(x.amax(0), x.amax(1)), inv);
        const float2 i2 = make_float2(inv, inv), z = make_float2(-0.0f, -0.0f);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            x.values(j, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = sm100::fma2(v[i], i2, z);
            codes[2 * j] = pack8(v);
            codes[2 * j + 1] = pack8(v + 4);
        }
        return s;
    }
}

}  // namespace fp4
}  // namespace mx
