// fp8_gemm.cuh -- host-visible description of one launch of the 8-bit matrix
// product with scales per block of 128, and its launchers.
//
//     C_g[m, n] = sum_s sum_kb sa[kb, m] * sb[kb, n] * sum_{k in kb} A[m, k] B[n, k]   (+ bias[n])
//
// over K blocks of 128, with A's scale per row and K block and B's either per
// 128 columns and K block (weights) or per column and K block (activations);
// the scales are powers of two (any other reads as NaN).
// Groups g share a launch (column-parallel shards), segments s are summed into
// the same output (row-parallel shards), as in the bf16 GEMM.  Operands are
// 8-bit matrices, K-major (row-major [rows, K]) or MN-major (row-major
// [K, rows]); both are fetched as 128 x 128-byte boxes.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace tpmlp {

constexpr int F8_MAX_MAPS = 8;
constexpr int F8_BK = 128;                  // K per stage: one scale block, one 128-byte swizzle row
constexpr int F8_BOX_BYTES = 128 * 128;     // one operand box

// How an operand's maps and scale arrays are indexed.
enum Fp8Part : int { F8_SINGLE = 0, F8_GROUP = 1, F8_KSEG = 2 };
// Which variant: outputs and the kind of B's scale.
enum Fp8Out : int {
    F8_BF16_BLOCK = 0,  // bf16 output, B scaled per 128 x 128 block
    F8_F32_VECTOR = 1   // fp32 output, B scaled per column and K block
};

struct Fp8GemmParams {
    CUtensorMap a_map[F8_MAX_MAPS];
    CUtensorMap b_map[F8_MAX_MAPS];
    void* out[F8_MAX_MAPS];            // [M, N] per group, or [chunk_rows, N] per token chunk
    const float* sa[F8_MAX_MAPS];      // A's scales: [kb * sa_kb + m]
    const float* sb[F8_MAX_MAPS];      // B's: [kb * sb_kb + (n / 128) * sb_n] or [kb * sb_kb + n]
    long long sa_kb, sb_kb, sb_n;
    int M, N, K;                       // per group; K per segment
    int groups, ksegs;
    int a_part, b_part;
    int a_mn, b_mn;                    // MN-major operands
    int mtiles, ntiles, total_tiles, band;
    int chunk_rows;                    // > 0: output i holds rows [i * chunk_rows, ...), else output g
    const void* bias;                  // bf16 [groups * N] or null
    uint32_t ab_format;                // instruction descriptor bits of the operands' 8-bit formats
    unsigned int* err;                 // the device error word and the limit of any one wait
    unsigned long long timeout_ns;
    int stall;                         // failure-detection self-test: the loader of a cluster's last
                                       // CTA issues this many of its copies; < 0: all
};

// The whole product on CTA pairs with 256 x 256 output tiles; A's maps have boxes of
// 128 rows.
cudaError_t launch_fp8_gemm(const Fp8GemmParams& p, int out, cudaStream_t st);

// The same (bf16 output, B scaled per block) for few rows of A: tiles of 128 columns
// by `rows` rows of A, which is also the box of A's maps, with K cut over up to 8 CTAs
// of a cluster.
cudaError_t launch_fp8_small(const Fp8GemmParams& p, int rows, cudaStream_t st);
// Those rows for a product of this shape on the current device; 0: it has rows and
// columns enough for the pairs.
cudaError_t fp8_small_rows(int M, int N, int groups, int& rows);

}  // namespace tpmlp
