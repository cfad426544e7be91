// fp8_cvt.cuh -- the arithmetic of quantisation to 8 bits (see fp8_quant.cuh for
// the definition), shared by the kernels that quantise.
//
// Magnitudes are compared as integers: the 15 low bits of a bf16 grow with |x|,
// with infinities and NaN on top, so a packed 16-bit maximum compares two values
// at once and a group that is not finite shows as a maximum of at least 0x7F80.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "fp8_quant.cuh"

namespace tpmlp {
namespace q8 {

constexpr uint32_t kMagnitudes = 0x7FFF7FFFu;

// the larger of two packed 16-bit halves
__device__ __forceinline__ uint32_t fold(uint32_t w) { return max(w & 0xFFFFu, w >> 16); }

// the largest magnitude's bits among 8 bf16 values
__device__ __forceinline__ uint32_t largest(const uint4& v) {
    return fold(__vmaxu2(__vmaxu2(v.x & kMagnitudes, v.y & kMagnitudes),
                         __vmaxu2(v.z & kMagnitudes, v.w & kMagnitudes)));
}

// Magnitude bits of a group's largest value -> the scale and its reciprocal.
struct Scale {
    float s, inv;
    bool fine;
};

__device__ __forceinline__ Scale scale_of(uint32_t amax, int fmt) {
    // |x| = 2^(e - 127) (1 + m / 128); top = 1.75 * 2^8 or 1.75 * 2^15
    const int e = static_cast<int>(amax >> 7), m = static_cast<int>(amax & 0x7Fu);
    int k = e - 127 - (fmt == FP8_E4M3 ? 8 : 15) + (m > 96 ? 1 : 0);
    if (e == 0 || k < -119) k = -119;
    Scale r;
    r.fine = amax < 0x7F80u;
    r.s = r.fine ? __uint_as_float(static_cast<uint32_t>(k + 127) << 23)
                 : __uint_as_float(0x7FC00000u);
    r.inv = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
    return r;
}

// lo and hi rounded to 8 bits, hi in the upper byte
__device__ __forceinline__ uint32_t cvt2(float lo, float hi, int fmt) {
    uint16_t r;
    if (fmt == FP8_E4M3)
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// the two bf16 values of a word
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// 8 bf16 values of one group in 8 bits
__device__ __forceinline__ uint2 cvt8(const uint4& v, const Scale& sc, int fmt) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f =
            __fmul2_rn(make_float2(lo_f(w[j]), hi_f(w[j])), make_float2(sc.inv, sc.inv));
        o[j] = cvt2(f.x, f.y, fmt);
    }
    return sc.fine ? make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16)) : make_uint2(0u, 0u);
}

}  // namespace q8
}  // namespace tpmlp
