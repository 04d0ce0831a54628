// kv4.cuh - the 4-bit cache: its layout and its conversions.
//
// 16 neighbouring channels of a head share a scale s (e4m3); a value is u c with u = s ts (ts the head's own scale, 1
// without one) and a code c of e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives.  s c has at most six significant bits
// and lies between 2^-10 and 2880: exact in fp16, which is what the tensor cores are fed.
//
// The block of a (page, key-value head) holds the codes of its tokens, [page_size][D / 2] bytes with the even channel in the
// low half, then their scales, [page_size][D / 16] bytes.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace gdn {

// Eight codes to four pairs of fp16: d[i] = values of the codes in byte i, the low half first.
__device__ __forceinline__ void kv4_codes(uint32_t w, uint32_t (&d)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(w));
}
// Two scales (bytes 0 and 1) to fp16.  The byte that e4m3 has for NaN counts as the 480 that would follow 448: stale
// bytes behind a sequence stay finite, and P = 0 takes them away.
__device__ __forceinline__ uint32_t kv4_scales(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\tmin.f16x2 %0, %0, %2;\n\t}"
        : "=r"(r)
        : "r"(two), "r"(0x5f805f80u));
    return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2 *>(&x)); }

// The scale's byte and the unit u of 16 values with the largest magnitude amax.
__device__ __forceinline__ uint32_t kv4_unit(float amax, float ts, float &unit) {
    const float s = fminf(__fdiv_rn(amax, 6.f * ts), 448.f);
    uint16_t b;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(0.f), "f"(s));
    unit = f16x2_to_f32(kv4_scales(b)).x * ts;
    return b & 0xffu;
}
// Codes of eight values in units of u, the first in the lowest bits; halfway goes to the even code.
__device__ __forceinline__ uint32_t kv4_encode(const float (&t)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(t[0]), "f"(t[1]), "f"(t[2]), "f"(t[3]), "f"(t[4]), "f"(t[5]), "f"(t[6]), "f"(t[7]));
    return r;
}

// The power of two that brings a row's largest magnitude into [1, 2), and its inverse (both normal numbers; for rows below
// 2^-126, nothing but zeros among them, 2^126).  With an infinity in the row the power is NaN, which makes all of its scores
// NaN, as the definition has it: each is infinite or NaN, and a softmax over those has no value.
__device__ __forceinline__ float kv4_row_power(float amax, float &inverse) {
    const int e = max(1, min((int)(__float_as_uint(amax) >> 23 & 255u), 253));  // (biased)
    inverse = __uint_as_float((uint32_t)e << 23);
    return fmaf(amax, 0.f, __uint_as_float((uint32_t)(254 - e) << 23));  // (infinity times 0)
}

// A row's softmax factor c inverse ks, in an order that leaves the range only if the product does, and then kept
// from 0 and infinity: a masked score stays -inf and a difference of 0 stays 0 under it.
__device__ __forceinline__ float kv4_row_factor(float c, float inverse, float ks) {
    const float lo = fminf(fminf(c, inverse), ks), hi = fmaxf(fmaxf(c, inverse), ks);
    const float mid = fmaxf(fminf(fmaxf(c, inverse), ks), fminf(c, inverse));
    return fminf(fmaxf(lo * hi * mid, 1e-30f), 1e30f);
}

}  // namespace gdn
