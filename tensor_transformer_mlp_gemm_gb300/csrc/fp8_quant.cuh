// fp8_quant.cuh -- quantisation of bf16 matrices to 8-bit floating point with
// one scale for each group of 128.
//
// A group G of values x gets the scale s and the 8-bit values q with
//     s = the smallest power of two with max |x| <= s * top, at least 2^-119
//     q = round-to-nearest-even_8bit(x / s)
// where top is the format's largest value (448 for e4m3, 57344 for e5m2).  A
// power of two makes x / s exact, so q is one rounding of x and the same on
// every machine; the floor keeps 1 / s finite.  A group that holds an infinity
// or a NaN gets s = NaN and q = 0: what is computed from it is NaN, not a
// saturated number.
//
// Groups:  rows   128 consecutive columns of one row    scales [ceil(C/128)][ld]
//          cols   128 consecutive rows of one column    scales [ceil(R/128)][C]
//          block  128 x 128                             scales [ceil(R/128)][ceil(C/128)]
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

namespace tpmlp {

constexpr int FP8_GROUP = 128;
constexpr int FP8_MAX_PARTS = 8;

enum Fp8Format : int { FP8_E4M3 = 0, FP8_E5M2 = 1 };

// One launch over `parts` matrices of the same shape.
struct Fp8QuantParams {
    const void* src[FP8_MAX_PARTS];    // bf16 [R, C]
    void* q_rows[FP8_MAX_PARTS];       // 8-bit [R, C]
    float* s_rows[FP8_MAX_PARTS];      // [ceil(C/128)][ld]
    void* q_cols[FP8_MAX_PARTS];       // 8-bit [R, C] (blocks: q)
    float* s_cols[FP8_MAX_PARTS];      // [ceil(R/128)][C] (blocks: s)
    float* sums[FP8_MAX_PARTS];        // fp32 column sums of each 128 rows, [ceil(R/128)][sums_ld]
    long long rows, cols, ld, sums_ld;
    int parts;
    int fmt_rows, fmt_cols;
};

// Which outputs a launch makes.
enum Fp8QuantMode : int {
    FP8_Q_ROWS = 1,
    FP8_Q_COLS = 2,
    FP8_Q_SUMS = 4,   // with ROWS | COLS only
    FP8_Q_BLOCK = 8   // alone
};

// cudaErrorInvalidValue for a mode that is not built or a grid past the limit.
cudaError_t launch_fp8_quant(const Fp8QuantParams& p, int mode, cudaStream_t st);

}  // namespace tpmlp
