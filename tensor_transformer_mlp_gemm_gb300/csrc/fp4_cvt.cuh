// fp4_cvt.cuh -- the arithmetic of quantisation to 4 bits (see fp4_quant.cuh for the
// definition), shared by the kernels that quantise.
//
// Magnitudes are compared as integers once they are the largest: the 15 low bits of a bf16
// grow with |x|, with infinities and NaN on top.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "fp4_quant.cuh"
#include "fp8_cvt.cuh"

namespace tpmlp {
namespace q4 {

// The larger magnitude of two pairs of bf16, with some sign; NaN (0x7FFF) where either is.
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// the largest magnitude's bits among a pair, among 8 values
__device__ __forceinline__ uint32_t fold(uint32_t w) { return larger(w, w >> 16) & 0x7FFFu; }
__device__ __forceinline__ uint32_t largest(const uint4& v) {
    return fold(larger(larger(v.x, v.y), larger(v.z, v.w)));
}

// A group's scale: its byte, and what its values are multiplied by (0: not finite).
struct Scale4 {
    uint32_t byte;
    float inv;
};

// e4m3 without a sign, in fp32
__device__ __forceinline__ float e4m3_f(uint32_t b) {
    return b >= 8 ? __uint_as_float((b << 20) + (120u << 23)) : static_cast<float>(b) * 0.001953125f;
}

// Magnitude bits of a bf16 group's largest value -> its scale.  inv_g: 1 / g, 0 if g is not
// one; not used by mx.
template <int FMT>
__device__ __forceinline__ Scale4 scale_of(uint32_t amax, float inv_g) {
    Scale4 r;
    if constexpr (FMT == FP4_MX) {
        // |x| = 2^(e - 127) (1 + m / 128); 6 = 1.5 * 2^2
        const int e = static_cast<int>(amax >> 7), m = static_cast<int>(amax & 0x7Fu);
        const int k = max(e - 129 + (m > 64 ? 1 : 0), -126);
        r.byte = static_cast<uint32_t>(k + 127);
        r.inv = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
        if (amax >= 0x7F80u) {
            r.byte = 0xFFu;
            r.inv = 0.0f;
        }
    } else {
        // amax / 6 as a product with a rounded 1 / 6, then rounded to 12 significant bits
        // (Veltkamp's splitting): a border between two e4m3 values has 5, and a quotient that
        // is not on it is 2^-9 of it away.  (4096 / 6 is past the largest scale.)
        const float v = fminf(__uint_as_float(amax << 16) * inv_g, 4096.0f) * (1.0f / 6.0f);
        const float t = __fmul_rn(v, 4097.0f), w = __fsub_rn(t, __fsub_rn(t, v));
        uint16_t b;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(0.0f), "f"(w));
        r.byte = max(static_cast<uint32_t>(b), 1u);
        float inv_s;  // (off by 2^-23 at most)
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv_s) : "f"(e4m3_f(r.byte)));
        r.inv = inv_s * inv_g;
        if (amax >= 0x7F80u || inv_g == 0.0f) {
            r.byte = 0x7Fu;
            r.inv = 0.0f;
        }
    }
    return r;
}

// The reciprocal of a tensor's scale, 0 for what is none.
__device__ __forceinline__ float inverse_of(const float* g) {
    const uint32_t b = __float_as_uint(__ldg(g)), e = b >> 23;
    return (b & 0x807FFFFFu) == 0 && e >= 127 - 110 && e <= 127 + 117 ? __uint_as_float((254u - e) << 23) : 0.0f;
}

// x * inv in both halves.  Of nv, inv is a rounded reciprocal, so the product of an x on a
// border may miss it by a few 2^-22: it is rounded to multiples of 2^-16, which borders are,
// and which no other quotient (2^-9 of a border away) reaches a border by.
template <int FMT>
__device__ __forceinline__ float2 scaled(float2 x, float inv) {
    if constexpr (FMT == FP4_MX) return __fmul2_rn(x, make_float2(inv, inv));
    const float2 big = make_float2(192.0f, 192.0f), neg = make_float2(-192.0f, -192.0f);
    return __fadd2_rn(__ffma2_rn(x, make_float2(inv, inv), big), neg);
}

// four pairs as 4-bit values, the first in the lowest half byte
__device__ __forceinline__ uint32_t cvt8(float2 a, float2 b, float2 c, float2 d) {
    uint32_t r;
    asm("{\n\t.reg .b8 p, q, r, s;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 p, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 q, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 r, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 s, %8, %7;\n\t"
        "mov.b32 %0, {p, q, r, s};\n\t}"
        : "=r"(r)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
    return r;
}

}  // namespace q4
}  // namespace tpmlp
