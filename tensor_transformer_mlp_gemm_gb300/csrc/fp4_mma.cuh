// fp4_mma.cuh -- device pieces of the 4-bit products: the tcgen05 instructions for 4-bit
// operands with block scales, and the scales' way into tensor memory.  (Bounded waits and
// what else the 8-bit products have: fp8_mma.cuh.)
//
// tcgen05.mma.kind::mxf4 multiplies groups of 32 along K by powers of two given as 8-bit
// exponents (scale_vec::2X), kind::mxf4nvf4 groups of 16 by e4m3 scales (scale_vec::4X); both
// take 64 of K at a time and accumulate in fp32.  A word of tensor memory holds four scales
// of a row: 64 of K of nv, 128 of mx, of which an instruction takes the lower or the upper
// two.  The words of 128 rows take 4 columns: row r in lane r % 32, column r / 32, and the
// same in each quarter of the lanes, which is how tcgen05.cp lays down a 512-byte block of
// scales (fp4_quant.cuh).
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "fp4_gemm.cuh"
#include "fp8_mma.cuh"
#include "two_sum.cuh"

namespace tpmlp {
namespace f4 {

// D[tmem] (+)= (A x scale_A) x (B x scale_B), on a CTA pair (issued by the even CTA: each
// CTA's own rows of A, half the rows of B from each; both hold all scales of B) or on one CTA.
template <int FMT, int CTAS>
__device__ __forceinline__ void mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                    uint32_t sa_tmem, uint32_t sb_tmem, uint32_t accumulate) {
#define F4_MMA(GROUP, KIND)                                                                      \
    asm volatile("{\n\t.reg .pred p;\n\t"                                                        \
                 "setp.ne.b32 p, %6, 0;\n\t"                                                     \
                 "tcgen05.mma.cta_group::" GROUP ".kind::" KIND                                  \
                 " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),                         \
                 "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate) \
                 : "memory")
    if constexpr (FMT == FP4_MX) {
        if constexpr (CTAS == 2)
            F4_MMA("2", "mxf4.block_scale.scale_vec::2X");
        else
            F4_MMA("1", "mxf4.block_scale.scale_vec::2X");
    } else {
        if constexpr (CTAS == 2)
            F4_MMA("2", "mxf4nvf4.block_scale.scale_vec::4X");
        else
            F4_MMA("1", "mxf4nvf4.block_scale.scale_vec::4X");
    }
#undef F4_MMA
}

// Instruction descriptor: 4-bit operands, K-major, fp32 accumulator.
//   bits 4-5, 29-30 which of a scale word's bytes B's and A's scales start at (mx: 0 or 2);
//   7-9 A format, 10-11 B format (1 = the 4-bit one); 17-22 N >> 3; bit 23 the scales are
//   8-bit exponents (else e4m3); 27-28 M >> 7.
template <int FMT>
__host__ __device__ constexpr uint32_t idesc(int M, int N) {
    return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
           (FMT == FP4_MX ? 1u << 23 : 0u) | (static_cast<uint32_t>(M >> 7) << 27);
}
// The same with scales from byte 2 of their words.
constexpr uint32_t UPPER_SCALES = (2u << 4) | (2u << 29);

// A 512-byte block of scales from shared memory into 4 columns of tensor memory (of both
// CTAs of a pair, each from its own).
template <int CTAS>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
    if constexpr (CTAS == 2)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// Its descriptor: rows of 16 bytes, 8 of them next to each other, no swizzle.
__device__ __forceinline__ uint64_t scales_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128 >> 4) << 16) |
           (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}

// gA gB of nv as two factors whose product it is: multiplied by one after the other, a sum
// leaves fp32's range only where the result does.  NaN unless both are powers of two within
// what quantising takes.
struct Alpha {
    float first, second;
};
__device__ __forceinline__ Alpha alpha_of(const float* ga, const float* gb) {
    const uint32_t a = __float_as_uint(__ldg(ga)), b = __float_as_uint(__ldg(gb));
    const int ea = static_cast<int>(a >> 23) - 127, eb = static_cast<int>(b >> 23) - 127;
    Alpha r;
    if ((a & 0x807FFFFFu) || (b & 0x807FFFFFu) || min(ea, eb) < -110 || max(ea, eb) > 117) {
        r.first = r.second = __uint_as_float(0x7FC00000u);
    } else {
        const int e = ea + eb, h = e >> 1;
        r.first = __uint_as_float(static_cast<uint32_t>(h + 127) << 23);
        r.second = __uint_as_float(static_cast<uint32_t>(e - h + 127) << 23);
    }
    return r;
}

// Column sums from their partial rows, in order: a warp of each CTA takes 32 columns at a time.
__device__ __forceinline__ void column_sums(const Fp4GemmParams& p, int cta, int ctas, int lane) {
    // (unsigned: a step may pass 2^31)
    const unsigned cols = p.sum_cols, step = ctas * 32;
    for (unsigned c = cta * 32 + lane; c < cols; c += step) {
        const float* from = p.sums + c;
        Sum s = {0.0f, 0.0f};
        long long r = 0;
        for (; r + 8 <= p.sum_rows; r += 8) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __ldg(from + (r + i) * p.sum_cols);
#pragma unroll
            for (int i = 0; i < 8; ++i) s.add(x[i]);
        }
        for (; r < p.sum_rows; ++r) s.add(__ldg(from + r * p.sum_cols));
        // (of infinities the second part is NaN)
        p.db[c] = isfinite(s.hi) ? s.hi + s.lo : s.hi;
    }
}

__device__ __forceinline__ int pick(int part, int g, int s) {
    return part == F4_GROUP ? g : part == F4_KSEG ? s : 0;
}

}  // namespace f4
}  // namespace tpmlp
