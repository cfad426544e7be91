// norm_device.cuh -- device pieces shared by the norms' forward and backward kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "gemm_params.h"
#include "ptx.cuh"

namespace tpmlp {
namespace nr {

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

__device__ __forceinline__ void unpack(const uint4& u, float2 (&f)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

__device__ __forceinline__ uint4 pack(const float2 (&f)[4]) {
    return make_uint4(pack2(f[0].x, f[0].y), pack2(f[1].x, f[1].y), pack2(f[2].x, f[2].y),
                      pack2(f[3].x, f[3].y));
}

__device__ __forceinline__ uint4 zero4() { return make_uint4(0, 0, 0, 0); }

// Quotient and remainder of start, start + stride, start + 2 stride, ... by n, all of
// them below 2^31: divided once, then stepped.
struct Stepper {
    uint32_t q, r, dq, dr, n;  // (r + dr may pass 2^31)
    __device__ __forceinline__ Stepper(long long start, long long stride, long long by) {
        n = static_cast<uint32_t>(by);
        q = static_cast<uint32_t>(start) / n;
        r = static_cast<uint32_t>(start) - q * n;
        dq = static_cast<uint32_t>(stride) / n;
        dr = static_cast<uint32_t>(stride) - dq * n;
    }
    __device__ __forceinline__ void step() {
        q += dq;
        r += dr;
        if (r >= n) {
            r -= n;
            ++q;
        }
    }
};

// Waits for phase `parity` of `bar`; after the limit, false, and the error word says so.
__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, unsigned long long timeout_ns,
                                        unsigned* err, unsigned code = ERR_EPILOGUE) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
    while (!ptx::mbar_try_wait(bar, parity)) {
        if (ptx::globaltimer_ns() - t0 > timeout_ns) {
            atomicOr(err, code);
            return false;
        }
    }
    return true;
}

// The same for copies of its own, before a CTA goes on without them.  They end by
// themselves: the limit is not the caller's where that is short.
__device__ __forceinline__ void drain_on(uint32_t bar, uint32_t parity, unsigned long long timeout_ns,
                                         unsigned* err) {
    wait_on(bar, parity, max(timeout_ns, 1000000000ULL), err, ERR_DRAIN);
}

// The sum of v over the warp, the same in every lane and every run.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace nr
}  // namespace tpmlp
