// fp8_quant.cu -- quantisation to 8-bit floating point (see fp8_quant.cuh for
// the definition).
//
// What bounds it: HBM traffic, 2 bytes read and 1 byte written per element and
// grouping.  So both groupings of an activation, and the column sums of a
// gradient (the bias gradient), come from one read.
//
// A CTA takes a 128 x 128 tile, which is 128 whole row groups, 128 whole
// column groups and one whole block, so no group crosses CTAs and nothing is
// read twice.  A thread holds 8 rows x 8 columns as eight 16-byte loads, all
// in flight before the first use; the arithmetic is fp8_cvt.cuh's.
//
// The formats are template constants and non-finite columns a path of their own: with
// both looked at in every conversion, both groupings of 16384 x 4096 took 68 us, now
// 54 (5.0 TB/s); a weight of 12288 x 4608 takes 31 us (5.5 TB/s).
#include "fp8_quant.cuh"

#include "fp8_cvt.cuh"
#include "ptx.cuh"

namespace tpmlp {
namespace {

using namespace q8;

constexpr int QT = 256;          // threads
constexpr int QV = 8;            // rows (and columns) per thread
constexpr int QWARPS = QT / 32;

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// CTAs of an SM: a thread's 64 values leave room for three, and for four where there is
// one grouping (asked for none, the compiler left two of the bias gradient's kind: 70 us
// instead of 63 at 16384 x 4096).
constexpr int per_sm(int mode) { return mode == FP8_Q_BLOCK || mode == FP8_Q_ROWS || mode == FP8_Q_COLS ? 4 : 3; }

template <int MODE, int RF, int CF>
__global__ void __launch_bounds__(QT, per_sm(MODE))
    fp8_quant_kernel(const __grid_constant__ Fp8QuantParams p, int col_tiles) {
    constexpr bool ROWS = MODE & FP8_Q_ROWS, COLS = MODE & FP8_Q_COLS, SUMS = MODE & FP8_Q_SUMS,
                   BLOCK = MODE & FP8_Q_BLOCK;
    __shared__ uint4 s_max[QWARPS][16];       // column magnitudes of each warp's rows
    __shared__ alignas(8) float s_inv[FP8_GROUP];  // reciprocal column scales (0: not finite)
    __shared__ float s_row[FP8_GROUP];        // row scales
    __shared__ alignas(8) float s_sum[SUMS ? QWARPS : 1][FP8_GROUP];
    __shared__ uint32_t s_blk[QWARPS];

    const int part = blockIdx.y;
    const long long rt = blockIdx.x / col_tiles, ct = blockIdx.x % col_tiles;
    const long long r0 = rt * FP8_GROUP, c0 = ct * FP8_GROUP;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cv = lane & 15;                 // this thread's 8 columns
    const int slot = warp * 2 + (lane >> 4);  // its rows: slot + 16 i
    const long long c = c0 + cv * QV;
    const bool col_in = c < p.cols;

    // the dependent launch may be scheduled as soon as there is room for it; it
    // waits for this grid's results itself
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();

    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.src[part]) + c);
    const long long vstep = p.cols / 8;
    uint4 v[QV];
#pragma unroll
    for (int i = 0; i < QV; ++i) {
        const long long r = r0 + slot + 16 * i;
        v[i] = (col_in && r < p.rows) ? __ldg(src + r * vstep) : make_uint4(0, 0, 0, 0);
    }

    uint32_t row_max[QV];
    uint32_t cm[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < QV; ++i) {
        if (ROWS) row_max[i] = largest(v[i]);
        if (COLS || BLOCK) {
#pragma unroll
            for (int j = 0; j < 4; ++j) cm[j] = __vmaxu2(cm[j], word(v[i], j) & kMagnitudes);
        }
    }

    if constexpr (BLOCK) {
        uint32_t m = fold(__vmaxu2(__vmaxu2(cm[0], cm[1]), __vmaxu2(cm[2], cm[3])));
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) s_blk[warp] = m;
        __syncthreads();
        m = s_blk[0];
#pragma unroll
        for (int w = 1; w < QWARPS; ++w) m = max(m, s_blk[w]);
        const Scale sc = scale_of(m, CF);
        if (threadIdx.x == 0) p.s_cols[part][rt * col_tiles + ct] = sc.s;
        if (col_in) {
            uint8_t* q = static_cast<uint8_t*>(p.q_cols[part]);
#pragma unroll
            for (int i = 0; i < QV; ++i) {
                const long long r = r0 + slot + 16 * i;
                if (r >= p.rows) break;
                *reinterpret_cast<uint2*>(q + r * p.cols + c) = cvt8(v[i], sc, CF);
            }
        }
        return;
    }

    if constexpr (COLS) {
        // both row slots of the warp, then the warps
#pragma unroll
        for (int j = 0; j < 4; ++j) cm[j] = __vmaxu2(cm[j], __shfl_xor_sync(0xffffffffu, cm[j], 16));
        if (lane < 16) s_max[warp][cv] = make_uint4(cm[0], cm[1], cm[2], cm[3]);
    }
    if constexpr (SUMS) {
        // this thread's 8 rows in order, then the other row slot, then the warps
        float2 cs[QV / 2] = {};
#pragma unroll
        for (int i = 0; i < QV; ++i)
#pragma unroll
            for (int j = 0; j < QV / 2; ++j) {
                const uint32_t w = word(v[i], j);
                cs[j] = __fadd2_rn(cs[j], make_float2(lo_f(w), hi_f(w)));
            }
#pragma unroll
        for (int j = 0; j < QV / 2; ++j) {
            cs[j].x += __shfl_xor_sync(0xffffffffu, cs[j].x, 16);
            cs[j].y += __shfl_xor_sync(0xffffffffu, cs[j].y, 16);
            if (lane < 16) *reinterpret_cast<float2*>(&s_sum[warp][cv * QV + 2 * j]) = cs[j];
        }
    }

    if constexpr (ROWS) {
        uint8_t* q = static_cast<uint8_t*>(p.q_rows[part]);
        // two rows' maxima share a word
        uint32_t rm[QV / 2];
#pragma unroll
        for (int i = 0; i < QV / 2; ++i) rm[i] = row_max[2 * i] | row_max[2 * i + 1] << 16;
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1)
#pragma unroll
            for (int i = 0; i < QV / 2; ++i)
                rm[i] = __vmaxu2(rm[i], __shfl_xor_sync(0xffffffffu, rm[i], o));
#pragma unroll
        for (int i = 0; i < QV; ++i) {
            const Scale sc = scale_of(i & 1 ? rm[i / 2] >> 16 : rm[i / 2] & 0xFFFFu, RF);
            const long long r = r0 + slot + 16 * i;
            if (cv == 0) s_row[slot + 16 * i] = sc.s;
            if (col_in && r < p.rows) {
                *reinterpret_cast<uint2*>(q + r * p.cols + c) = cvt8(v[i], sc, RF);
            }
        }
    }
    __syncthreads();

    bool fine = true;
    if (threadIdx.x < FP8_GROUP) {
        const int k = threadIdx.x;
        if (ROWS && r0 + k < p.rows) p.s_rows[part][ct * p.ld + r0 + k] = s_row[k];
        if constexpr (COLS) {
            const uint16_t* mags = reinterpret_cast<const uint16_t*>(&s_max[0][0]);
            uint32_t m = 0;
#pragma unroll
            for (int w = 0; w < QWARPS; ++w) m = max(m, static_cast<uint32_t>(mags[w * 128 + k]));
            const Scale sc = scale_of(m, CF);
            s_inv[k] = sc.fine ? sc.inv : 0.0f;
            fine = sc.fine;
            if (c0 + k < p.cols) p.s_cols[part][rt * p.cols + c0 + k] = sc.s;
        }
        if constexpr (SUMS) {
            float t = s_sum[0][k];
#pragma unroll
            for (int w = 1; w < QWARPS; ++w) t += s_sum[w][k];
            if (c0 + k < p.cols) p.sums[part][rt * p.sums_ld + c0 + k] = t;
        }
    }
    if constexpr (COLS) {
        const bool all_fine = __syncthreads_and(fine);
        if (!col_in) return;
        float2 inv[QV / 2];
#pragma unroll
        for (int j = 0; j < QV / 2; ++j) inv[j] = *reinterpret_cast<const float2*>(&s_inv[cv * QV + 2 * j]);
        uint8_t* q = static_cast<uint8_t*>(p.q_cols[part]);
#pragma unroll
        for (int i = 0; i < QV; ++i) {
            const long long r = r0 + slot + 16 * i;
            if (r >= p.rows) break;
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t w = word(v[i], j);
                float2 f = make_float2(lo_f(w), hi_f(w));
                if (!all_fine) {  // a column that is not finite: 0 * inf would be NaN
                    f.x = inv[j].x > 0.0f ? f.x : 0.0f;
                    f.y = inv[j].y > 0.0f ? f.y : 0.0f;
                }
                f = __fmul2_rn(f, inv[j]);
                o[j] = cvt2(f.x, f.y, CF);
            }
            *reinterpret_cast<uint2*>(q + r * p.cols + c) =
                make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
        }
    }
}

template <int MODE, int RF, int CF>
cudaError_t launch_formats(const Fp8QuantParams& p, cudaStream_t st) {
    const long long rt = (p.rows + FP8_GROUP - 1) / FP8_GROUP;
    const long long ct = (p.cols + FP8_GROUP - 1) / FP8_GROUP;
    if (ct > 0x7FFFFFFFLL || rt > 0x7FFFFFFFLL / ct) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(rt * ct), static_cast<unsigned>(p.parts), 1);
    cfg.blockDim = dim3(QT, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fp8_quant_kernel<MODE, RF, CF>, p, static_cast<int>(ct));
}

// the formats are the kernel's own constants; a grouping that is not asked for has none
template <int MODE>
cudaError_t launch(const Fp8QuantParams& p, cudaStream_t st) {
    constexpr bool ROWS = MODE & FP8_Q_ROWS, COLS = MODE & (FP8_Q_COLS | FP8_Q_BLOCK);
    constexpr int R5 = ROWS ? FP8_E5M2 : FP8_E4M3, C5 = COLS ? FP8_E5M2 : FP8_E4M3;
    if (ROWS && p.fmt_rows == FP8_E5M2)
        return COLS && p.fmt_cols == FP8_E5M2 ? launch_formats<MODE, R5, C5>(p, st)
                                              : launch_formats<MODE, R5, FP8_E4M3>(p, st);
    return COLS && p.fmt_cols == FP8_E5M2 ? launch_formats<MODE, FP8_E4M3, C5>(p, st)
                                          : launch_formats<MODE, FP8_E4M3, FP8_E4M3>(p, st);
}

}  // namespace

cudaError_t launch_fp8_quant(const Fp8QuantParams& p, int mode, cudaStream_t st) {
    switch (mode) {
        case FP8_Q_ROWS: return launch<FP8_Q_ROWS>(p, st);
        case FP8_Q_COLS: return launch<FP8_Q_COLS>(p, st);
        case FP8_Q_ROWS | FP8_Q_COLS: return launch<FP8_Q_ROWS | FP8_Q_COLS>(p, st);
        case FP8_Q_ROWS | FP8_Q_COLS | FP8_Q_SUMS:
            return launch<FP8_Q_ROWS | FP8_Q_COLS | FP8_Q_SUMS>(p, st);
        case FP8_Q_BLOCK: return launch<FP8_Q_BLOCK>(p, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace tpmlp
