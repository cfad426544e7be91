// fp8_internal.h -- host-side helpers of the 8-bit calls: checks of scale pointers, and
// tensor maps of 8-bit operands, kept by shape in the library's map cache.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "abi_internal.h"
#include "map_cache.h"

namespace tpmlp {
namespace abi {

// defined beside the tensor maps of the bf16 GEMM
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
extern EncodeTiledFn g_encode;
extern MapCache g_maps;
extern unsigned long long g_timeout_ns;
extern thread_local int g_stall;  // failure-detection self-test (tpmlp_selftest_stall_loads)

// Scales are read and written one at a time: a part of a larger array may start anywhere.
inline tpmlp_status check_scale(const void* p) {
    if (!p) return TPMLP_ERR_INVALID_ARG;
    return reinterpret_cast<uintptr_t>(p) % 4 ? TPMLP_ERR_UNSUPPORTED : TPMLP_OK;
}

inline tpmlp_status check_scales(const void* const* p, int n) {
    if (!p) return TPMLP_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i) {
        const tpmlp_status s = check_scale(p[i]);
        if (s != TPMLP_OK) return s;
    }
    return TPMLP_OK;
}

typedef CUresult (*ReplaceAddressFn)(CUtensorMap*, void*);
inline ReplaceAddressFn replace_address() {
    static const ReplaceAddressFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapReplaceAddress", &f, 12000,
                                                         cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return reinterpret_cast<ReplaceAddressFn>(ok ? f : nullptr);
    }();
    return fn;
}

inline bool set_address(CUtensorMap* m, const void* ptr) {
    const ReplaceAddressFn replace = replace_address();
    return replace && replace(m, const_cast<void*>(ptr)) == CUDA_SUCCESS;
}

// Row-major 8-bit matrix [outer, inner] (inner a multiple of 16), fetched as
// boxes of 128 bytes x `box_outer` rows with the 128-byte swizzle; what lies
// outside the matrix reads as zeros.  One map is kept for each shape (activations
// come at new addresses all the time), and its copy gets the address.
inline bool encode_bytes(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t outer,
                         uint32_t box_outer) {
    const cuuint64_t dims[2] = {inner, outer};
    const cuuint64_t strides[1] = {inner};
    const cuuint32_t box[2] = {128, box_outer};
    const MapKey key =
        make_map_key(CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, nullptr, dims, strides, box,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
    const bool ok = g_maps.get(key, m, [&](CUtensorMap* out) {
        const cuuint32_t estr[2] = {1, 1};
        return g_encode(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides,
                        box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    });
    return ok && set_address(m, ptr);
}

}  // namespace abi
}  // namespace tpmlp
