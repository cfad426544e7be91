// two_sum.cuh -- a sum in two fp32 parts (Knuth's two-sum), which hold it nearly as well as 64
// bits would: those run at 1/64 of the rate here.
#pragma once

#include <cuda_runtime.h>

namespace tpmlp {

struct Sum {
    float hi, lo;
    __device__ __forceinline__ void add(float x) {
        const float t = __fadd_rn(hi, x), z = __fsub_rn(t, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(t, z)), __fsub_rn(x, z)));
        hi = t;
    }
    // over the lanes of a warp, FIRST apart at most
    template <int FIRST>
    __device__ __forceinline__ void over_lanes() {
#pragma unroll
        for (int o = FIRST; o > 0; o >>= 1) {
            const float h = __shfl_xor_sync(0xffffffffu, hi, o), l = __shfl_xor_sync(0xffffffffu, lo, o);
            add(h);
            lo = __fadd_rn(lo, l);
        }
    }
};

}  // namespace tpmlp
