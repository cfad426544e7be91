// fp4_quant.cuh -- quantisation of bf16 matrices to 4-bit floating point (a sign, two
// exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) with a scale for each
// group along the axis that a product sums over.
//
//   mx   groups of 32, s = the smallest power of two with max |x| <= 6 s, at least 2^-126,
//        kept as an 8-bit exponent (biased by 127)
//   nv   groups of 16 and a power of two g for the tensor: s = max |x| / (6 g) rounded to
//        e4m3 (at most 448, at least 2^-9); g is the smallest with which the tensor's
//        largest finite magnitude is at most 6 * 448 g, at least 2^-110, or a caller's
//   q = round-to-nearest-even_4bit(x / s), of nv x / (s g), at most 6
//
// A group that holds an infinity or a NaN gets the scale NaN (0xFF, of e4m3 0x7F) and
// q = 0.  A g that is not a power of two of 2^-110 .. 2^117 makes every scale NaN.
//
// Powers of two keep every comparison exact: a bf16 x has 8 significant bits and s of nv
// 4, so x / (s g) is either on a border between two 4-bit values or 2^-9 of it away, and
// q is the same on every machine.
//
// Layouts.  A 4-bit matrix [R, K] summed over K ("K-major") lies in rows of up32(K) / 2
// bytes, element 2i in the low half of byte i, zeros behind K.  "Rows" quantises a bf16
// matrix [T, C] to [T, C], "cols" to the transposed [C, T].  Scales lie as the tensor cores
// take them: blocks of 128 rows by 4 groups, 512 bytes each, row r's group j at byte
// 16 (r % 32) + 4 (r / 32) + j; blocks along K next to each other, filled up to multiples
// of 256 of K (2 blocks of mx, 4 of nv), then the next 128 rows.  What fills up is zeros
// with the smallest scale.
#pragma once

#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace tpmlp {

constexpr int FP4_MAX_PARTS = 8;
enum Fp4Format : int { FP4_MX = 0, FP4_NV = 1 };

__host__ __device__ constexpr int fp4_group(int fmt) { return fmt == FP4_NV ? 16 : 32; }
// bytes of scales of 128 rows for each 256 of K
__host__ __device__ constexpr int fp4_scale_step(int fmt) { return fmt == FP4_NV ? 2048 : 1024; }
__host__ __device__ constexpr long long fp4_ld(long long K) { return (K + 31) / 32 * 16; }
__host__ __device__ constexpr long long fp4_packed_bytes(long long R, long long K) { return R * fp4_ld(K); }
__host__ __device__ constexpr long long fp4_scale_bytes(long long R, long long K, int fmt) {
    return (R + 127) / 128 * ((K + 255) / 256) * fp4_scale_step(fmt);
}

// One launch over `parts` matrices [rows, cols] of the same shape, each with outputs of its
// own; or (gather) over one matrix whose row chunks of `rows` (a multiple of 128) are the
// parts, with outputs 0.
struct Fp4QuantParams {
    const void* src[FP4_MAX_PARTS];   // bf16
    uint8_t* q_rows[FP4_MAX_PARTS];
    uint8_t* s_rows[FP4_MAX_PARTS];
    uint8_t* q_cols[FP4_MAX_PARTS];
    uint8_t* s_cols[FP4_MAX_PARTS];
    float* sums[FP4_MAX_PARTS];       // column sums of each 128 rows, [ceil(R/128)][sums_ld]
    const float* scale;               // g (nv)
    long long rows, cols, sums_ld;
    long long rows_k;                 // K of q_rows and s_rows, of which a part is `cols`; 0: cols
    int parts, gather;
    unsigned int* err;                // the device error word and the limit of any one wait
    unsigned long long timeout_ns;
    int stall;                        // failure-detection self-test: the last CTA loads this many tiles; < 0: all
};

enum Fp4QuantMode : int { FP4_Q_ROWS = 1, FP4_Q_COLS = 2, FP4_Q_SUMS = 4 };  // SUMS with both

// cudaErrorInvalidValue for a mode that is not built or a grid past the limit.
cudaError_t launch_fp4_quant(const Fp4QuantParams& p, int fmt, int mode, cudaStream_t st);
// g of all parts together into *scale (src, rows, cols and parts of p are read), by one kernel or
// two.
int fp4_tensor_scale_kernels(const Fp4QuantParams& p);
cudaError_t launch_fp4_tensor_scale(const Fp4QuantParams& p, float* scale, cudaStream_t st);
// The values of a 4-bit matrix [R, K] (K-major) in bf16 [R, K].
cudaError_t launch_fp4_dequant(long long R, long long K, int fmt, const void* q, const void* s,
                               const float* scale, void* out, cudaStream_t st);

}  // namespace tpmlp
