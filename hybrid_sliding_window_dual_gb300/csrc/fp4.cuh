// The 4-bit element format of FP4 pools: device helpers.
//
// A row's 16-element blocks share a scale. An element is an E2M1 code (sign, 2
// exponent bits, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), element 2 i in the
// lower half of byte i. A scale is a byte E5M3: an f16 without its sign and
// its last 7 bits (values up to 10240 are written). A code has at most 2
// significant bits and a scale 4, so code * scale has at most 6 and lies
// between 2^-18 and 61440: it is an f16, and a bf16, exactly.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <stdint.h>

#include "common.cuh"

namespace hswa {

constexpr int kFp4Block = 16;
constexpr float kFp4MaxScale = 10240.f;  // 6 times it is an f16; the next scale's would not be
constexpr uint32_t kFp4MaxScaleByte = 0xe2;

// The 8 codes of a word as f16 pairs: elements (0, 1), (2, 3), (4, 5), (6, 7).
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t &p0, uint32_t &p1, uint32_t &p2, uint32_t &p3) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(p0), "=r"(p1), "=r"(p2), "=r"(p3)
        : "r"(w));
}

__device__ __forceinline__ uint32_t hmul2_bits(uint32_t a, uint32_t b) {
    uint32_t c;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
    return c;
}

// A scale byte as an f16 in both halves.
__device__ __forceinline__ uint32_t scale_f16x2(uint32_t byte) { return byte * 0x00800080u; }

__device__ __forceinline__ float scale_value(uint8_t byte) {
    return __half2float(__ushort_as_half((unsigned short)((unsigned)byte << 7)));
}

// Value of element i of a row of codes.
__device__ __forceinline__ float fp4_value(const uint8_t *codes, const uint8_t *scales, int64_t i) {
    const uint32_t c = codes[i >> 1] >> (4 * (i & 1)) & 15, e = c >> 1 & 3, m = c & 1;
    const float x = e ? (float)((2 + m) << (e - 1)) * 0.5f : (float)m * 0.5f;
    return (c & 8 ? -x : x) * scale_value(scales[i / kFp4Block]);
}

// The scale byte of a block whose largest magnitude is amax: the nearest E5M3
// value to the fp32 quotient amax / 6 (ties to the even one), at most 10240.
__device__ __forceinline__ uint32_t fp4_scale(float amax) {
    const float x = fminf(__fdiv_rn(amax, 6.f), kFp4MaxScale);
    if (x < 0x1p-14f) return __float2uint_rn(x * 0x1p17f);  // steps of 2^-17; 8 of them make the first normal value
    uint32_t u = __float_as_uint(x);
    u += 0x7ffff + (u >> 20 & 1);
    return (u >> 20) - ((127 - 15) << 3);
}

// x / scale for a code: the nearest E2M1 value to it is that of the exact
// quotient. q - (s q - x) / s is x / s to far less than a step of fp32, so that
// it rounds to a border between codes only if x / s is on one: such borders
// times a scale have at most 7 significant bits, and no other fp32 x is nearer
// to that product than half a step of the quotient's. A -0 keeps its sign. x
// is finite, and no more than a few scales unless the scale is the largest.
struct Fp4Divider {
    float s, r;
    __device__ __forceinline__ explicit Fp4Divider(uint32_t scale) : s(scale_value((uint8_t)scale)) {
        r = __frcp_rn(s);
    }
    __device__ __forceinline__ float operator()(float x) const {
        const float q = x * r;
        return fmaf(-fmaf(s, q, -x), r, q);
    }
};

// Under the largest scale values past 6 of it, infinities among them, become
// 6 of it. (The conversion saturates, but the remainder of an infinity is none.)
__device__ __forceinline__ float fp4_clamp(float x) { return fminf(fmaxf(x, -6.f * kFp4MaxScale), 6.f * kFp4MaxScale); }

// 8 values as codes under a scale byte: the nearest E2M1 value to x / scale
// (ties to the even code), at most 6; all codes 0 under scale 0.
__device__ __forceinline__ uint32_t fp4_codes8(const float *in, uint32_t scale) {
    if (scale == 0) return 0;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = in[i];
    if (__builtin_expect(scale == kFp4MaxScaleByte, 0)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fp4_clamp(x[i]);
    }
    const Fp4Divider div(scale);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w |= (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(div(x[2 * i]), div(x[2 * i + 1])), __NV_E2M1, cudaRoundNearest) << (8 * i);
    return w;
}

__device__ __forceinline__ uint2 fp4_codes(const float (&x)[16], uint32_t scale) {
    return make_uint2(fp4_codes8(x, scale), fp4_codes8(x + 8, scale));
}

// One value's code.
__device__ __forceinline__ uint32_t fp4_code(float x, uint32_t scale) {
    if (scale == 0) return 0;
    return __nv_cvt_float2_to_fp4x2(make_float2(Fp4Divider(scale)(scale == kFp4MaxScaleByte ? fp4_clamp(x) : x), 0.f), __NV_E2M1, cudaRoundNearest) & 15;
}

__device__ __forceinline__ float amax16(const float (&x)[16]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(x[i]));
    return m;
}

}  // namespace hswa
