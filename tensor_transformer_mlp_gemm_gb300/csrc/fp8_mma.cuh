// fp8_mma.cuh -- device pieces of the 8-bit products: the tcgen05 instructions
// for 8-bit operands, bounded waits, and the promotion of a K block's partial
// sums from tensor memory into scaled fp32 sums.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "fp8_gemm.cuh"
#include "gemm_params.h"
#include "ptx.cuh"

namespace tpmlp {
namespace f8 {

// D[tmem] (+)= A[smem] x B[smem], 8-bit floating-point operands, fp32 sums; the
// pair form is issued by the even CTA.
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor of kind::f8f6f4 with an fp32 accumulator.
//   bits 4-5 D format (1 = f32); 7-9 A format, 10-12 B format (0 = e4m3, 1 = e5m2);
//   bit 15 A is MN-major; bit 16 B is MN-major; 17-22 N >> 3; 24-28 M >> 4.
__host__ __device__ constexpr uint32_t idesc(int M, int N, int a_mn, int b_mn) {
    return (1u << 4) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Descriptor of the 32-wide K slice kk (0..3) of a 128 x 128-byte operand box.
//   K-major:  rows of 128 bytes, 8-row swizzle atoms every 1024 bytes; the slice
//             starts 32 bytes further along the row.
//   MN-major: 128 K rows of 128 bytes, 8-row atoms every 1024 bytes; the slice
//             starts 32 rows (4096 bytes) further down.
__device__ __forceinline__ uint64_t operand_desc(uint32_t tile, int kk, int mn) {
    return ptx::smem_desc_sw128(tile + (mn ? kk * 4096 : kk * 32), mn ? F8_BOX_BYTES : 16, 1024);
}

// Waits for phase `parity` of `bar`; gives up (false) when another role has, or
// after the limit (then this one aborts the CTA and sets `code` in the error word).
template <bool CLUSTER>
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                     unsigned long long timeout_ns, unsigned* err, unsigned code) {
    auto done = [&] {
        return CLUSTER ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity);
    };
    if (done()) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
    while (true) {
        if (done()) return true;
        if (*abort_flag) return false;
        if (ptx::globaltimer_ns() - t0 > timeout_ns) {
            *abort_flag = 1;
            atomicOr(err, code);
            return false;
        }
    }
}

// Teardown wait: ignores the abort flag, still bounded.
__device__ __forceinline__ bool drain(uint32_t bar, uint32_t parity, unsigned long long timeout_ns,
                                      unsigned* err) {
    const uint64_t t0 = ptx::globaltimer_ns();
    while (!ptx::mbar_try_wait(bar, parity)) {
        if (ptx::globaltimer_ns() - t0 > timeout_ns) {
            atomicOr(err, ERR_DRAIN);
            return false;
        }
    }
    return true;
}

// Registers per thread of the calling warpgroup (all of its warps call it).
template <int N>
__device__ __forceinline__ void reg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// ---- packed fp32 pairs -----------------------------------------------------------
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// acc[0..C) += scale * (C columns of this thread's tensor-memory lane), C a
// multiple of 32 (acc holds pairs).  VEC: times column factors too, read from
// shared memory as pairs (every lane reads the same ones).
template <int C, bool VEC>
__device__ __forceinline__ void promote(uint32_t taddr, float scale, const uint64_t* col,
                                        uint64_t (&acc)[C / 2]) {
    const uint64_t s2 = pack2(scale, scale);
#pragma unroll
    for (int c = 0; c < C / 32; ++c) {
        uint32_t v[32];
        ptx::tmem_ld_32x32b_x32(taddr + c * 32, v);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint64_t x = pack2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
            if constexpr (VEC) {
                acc[c * 16 + i] = fma2(x, mul2(col[c * 16 + i], s2), acc[c * 16 + i]);
            } else {
                acc[c * 16 + i] = fma2(x, s2, acc[c * 16 + i]);
            }
        }
    }
}

}  // namespace f8
}  // namespace tpmlp
