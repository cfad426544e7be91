// fp4_gemm.cuh -- host-visible description of one launch of the matrix product on 4-bit
// operands, and its launchers.
//
//     C_g[m, n] = gA gB sum_s sum_k A_s[m, k] B_s[n, k]   (+ bias[n])
//
// A and B are the values that 4-bit numbers and their groups' scales stand for
// (fp4_quant.cuh); gA and gB the tensors' scales (nv).  Groups g share a launch
// (column-parallel shards), segments s are summed into the same output (row-parallel
// shards).  Both operands are K-major: a product over tokens takes its operands
// transposed, as quantising along tokens writes them.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "fp4_quant.cuh"

namespace tpmlp {

constexpr int F4_MAX_MAPS = 8;
constexpr int F4_BK = 256;               // K per stage: a 128-byte swizzle row
constexpr int F4_BOX_BYTES = 128 * 128;  // 128 rows of an operand for it

// How an operand's maps are indexed.
enum Fp4Part : int { F4_SINGLE = 0, F4_GROUP = 1, F4_KSEG = 2 };

struct Fp4GemmParams {
    // [bytes of K, rows, matrices]: one map for all of an operand's matrices where they lie at
    // equal steps (a_z, b_z: the matrix is the third coordinate), else one for each
    CUtensorMap a_map[F4_MAX_MAPS];      // values, boxes of 128 bytes x 128 rows
    CUtensorMap b_map[F4_MAX_MAPS];
    CUtensorMap as_map[F4_MAX_MAPS];     // scales, 128 rows of one stage (of B, 256 rows)
    CUtensorMap bs_map[F4_MAX_MAPS];
    const uint8_t* sa[F4_MAX_MAPS];      // the same scales, for the few-rows kernel
    const uint8_t* sb[F4_MAX_MAPS];
    void* out[F4_MAX_MAPS];              // [M, N] per group, or [chunk_rows, N] per token chunk
    const void* x[F4_MAX_MAPS];          // few rows only: A in bf16 [M, K], quantised on the way
    const float* ga;                     // the tensors' scales (nv)
    const float* gb;
    int early;                           // B may be read before the grids ahead have ended
    int M, N, K;                         // per group; K per segment
    int groups, ksegs;
    int a_part, b_part;
    int a_z, b_z;
    int a_seg;                           // K blocks from a segment to the next in one matrix A, or 0
    int mtiles, ntiles, total_tiles, band;
    int chunk_rows;                      // > 0: output i holds rows [i * chunk_rows, ...), else output g
    const void* bias;                    // bf16 [groups * N] or null
    const float* sums;                   // rows of partial column sums [sum_rows, sum_cols] that are
    float* db;                           // added up into db on the way, or null
    long long sum_rows;
    int sum_cols;
    int apart;                           // takes nothing from the grid ahead and runs beside it, but
                                         // ends after it (pairs only)
    unsigned int* err;                   // the device error word and the limit of any one wait
    unsigned long long timeout_ns;
    int stall;                           // failure-detection self-test: the loader of a cluster's last
                                         // CTA issues this many of its copies; < 0: all
};

// The whole product on CTA pairs with 256 x 256 output tiles; f32: fp32 outputs (no bias),
// else bf16.
cudaError_t launch_fp4_gemm(const Fp4GemmParams& p, int fmt, bool f32, cudaStream_t st);

// The same (bf16 output) for few rows of A: tiles of 128 columns by `rows` rows of A, which
// is also the box of A's maps, with K cut over up to 8 CTAs of a cluster.
// A comes in 4 bits, or (quantise: up to FP4_QUANT_ROWS rows) in bf16.
constexpr int FP4_QUANT_ROWS = 32;
cudaError_t launch_fp4_small(const Fp4GemmParams& p, int fmt, int rows, bool quantise, cudaStream_t st);
// Those rows for a product of this shape on the current device; 0: it has rows and
// columns enough for the pairs.
cudaError_t fp4_small_rows(int M, int N, int K, int groups, int ksegs, int fmt, int& rows);
// Whether few rows are quantised faster by the product itself than by a launch ahead of it.
cudaError_t fp4_small_quantises(int M, int N, int K, int groups, int ksegs, bool& quantises);

}  // namespace tpmlp
