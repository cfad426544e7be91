// fp4_quant.cu -- quantisation to 4-bit floating point and back (see fp4_quant.cuh for
// the definition).
//
// What bounds it: HBM traffic, 2 bytes read and 0.53 (mx) or 0.56 (nv) written for each
// element and grouping.  So both groupings of a matrix, and the column sums of a gradient
// (the bias gradient), come from one read.
//
// A CTA takes a 128 x 128 tile: whole groups, and whole blocks of scales, both ways.  For
// the rows a thread holds 8 rows x 8 columns as eight 16-byte loads, all in flight before
// the first use.  For the columns the tile goes through shared memory, and a thread takes
// 32 rows of two columns, which is 16 bytes of each column's output.
#include <cuda_fp16.h>

#include "fp4_cvt.cuh"
#include "fp4_quant.cuh"
#include "ptx.cuh"

namespace tpmlp {
namespace {

using namespace q4;
using q8::hi_f;
using q8::kMagnitudes;
using q8::lo_f;

constexpr int QT = 256;  // threads
constexpr int TILE = 128;

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// where the scale of group j (0..7) of row r (0..127) lies in a tile's block or two
__device__ __forceinline__ uint32_t scale_at(uint32_t r, uint32_t j) {
    return (j >> 2) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (j & 3);
}

constexpr int per_sm(int mode) { return mode & FP4_Q_COLS ? 3 : 4; }

template <int FMT, int MODE>
__global__ void __launch_bounds__(QT, per_sm(MODE))
    fp4_quant_kernel(const __grid_constant__ Fp4QuantParams p, int col_tiles) {
    constexpr bool ROWS = MODE & FP4_Q_ROWS, COLS = MODE & FP4_Q_COLS, SUMS = MODE & FP4_Q_SUMS;
    constexpr int SB = fp4_scale_step(FMT) / 2;  // bytes of a tile's scales
    constexpr int PER = FMT == FP4_NV ? 2 : 1;   // groups of 32 elements
    __shared__ uint4 s_tile[COLS ? TILE * TILE / 8 : 1];  // [row][column / 8], columns as below
    __shared__ alignas(16) uint8_t s_rows[ROWS ? SB : 16];
    __shared__ alignas(16) uint8_t s_cols[COLS ? SB : 16];

    const int part = p.gather ? 0 : blockIdx.y;
    const long long rt = blockIdx.x / col_tiles, ct = blockIdx.x % col_tiles;
    const long long r0 = rt * TILE, c0 = ct * TILE;
    const long long total = p.gather ? p.rows * p.parts : p.rows;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cv = lane & 15;                 // this thread's 8 columns
    const int slot = warp * 2 + (lane >> 4);  // its rows: slot + 16 i
    const long long c = c0 + cv * 8;
    const bool col_in = c < p.cols;

    // The dependent launch after the wait: what came before this grid has ended when it starts,
    // so that it may read weights before this grid ends.
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    float inv_g = 0.0f;
    if constexpr (FMT == FP4_NV) inv_g = inverse_of(p.scale);
    int from = part;
    long long before = 0;  // rows of the parts before this one
    if (p.gather && r0 < total) {
        from = static_cast<int>(r0 / p.rows);
        before = from * p.rows;
    }
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.src[from]) + c);
    const long long vstep = p.cols / 8;
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const long long r = r0 + slot + 16 * i;
        v[i] = (col_in && r < total) ? __ldg(src + (r - before) * vstep) : make_uint4(0, 0, 0, 0);
    }

    if constexpr (COLS) {
        // 16-byte vector cv of a row lies at cv ^ 2 (row / 32), so that a warp's reads below
        // meet 32 banks
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = slot + 16 * i;
            s_tile[r * 16 + (cv ^ ((r >> 5) << 1))] = v[i];
        }
    }
    if constexpr (ROWS) {
        // largest magnitudes of each row's groups, two rows in a word
        uint32_t rm[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) rm[i] = largest(v[2 * i]) | largest(v[2 * i + 1]) << 16;
#pragma unroll
        for (int o = 1; o < 4 / PER; o <<= 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) rm[i] = larger(rm[i], __shfl_xor_sync(0xffffffffu, rm[i], o));
        const uint32_t group = PER == 2 ? cv >> 1 : cv >> 2;
        uint8_t* q = p.q_rows[part];
        const long long ld = fp4_ld(p.cols);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const Scale4 sc = scale_of<FMT>((i & 1 ? rm[i / 2] >> 16 : rm[i / 2]) & 0x7FFFu, inv_g);
            const int r = slot + 16 * i;
            if (cv % (4 / PER) == 0) s_rows[scale_at(r, group)] = static_cast<uint8_t>(sc.byte);
            if (col_in && r0 + r < total) {
                float2 f[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t w = word(v[i], j);
                    f[j] = scaled<FMT>(make_float2(lo_f(w), hi_f(w)), sc.inv);
                }
                const uint32_t u = cvt8(f[0], f[1], f[2], f[3]);
                *reinterpret_cast<uint32_t*>(q + (r0 + r) * ld + c / 2) = sc.inv > 0.0f ? u : 0u;
            }
        }
    }
    __syncthreads();

    if constexpr (COLS) {
        const int g = lane & 3, cp = warp * 8 + (lane >> 2);  // 32 rows, two columns
        const uint32_t* tile = reinterpret_cast<const uint32_t*>(s_tile) + g * 32 * 64 + (cp ^ (g << 3));
        uint32_t w[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) w[k] = tile[k * 64];
        const long long cc = c0 + 2 * cp;
        if constexpr (SUMS) {
            // 32 rows in order, then the four groups of them
            float2 t = make_float2(lo_f(w[0]), hi_f(w[0]));
#pragma unroll
            for (int k = 1; k < 32; ++k) t = __fadd2_rn(t, make_float2(lo_f(w[k]), hi_f(w[k])));
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                t.x += __shfl_xor_sync(0xffffffffu, t.x, o);
                t.y += __shfl_xor_sync(0xffffffffu, t.y, o);
            }
            if (g == 0 && cc < p.cols && r0 < total)
                *reinterpret_cast<float2*>(p.sums[part] + rt * p.sums_ld + cc) = t;
        }
        const long long ld = fp4_ld(total);
        const bool in = cc < p.cols && r0 + 32 * g < total;
        uint8_t* q = p.q_cols[part] + cc * ld + r0 / 2 + g * 16;
        uint32_t m[PER];
#pragma unroll
        for (int h = 0; h < PER; ++h) {
            m[h] = w[h * (32 / PER)];
#pragma unroll
            for (int k = 1; k < 32 / PER; ++k) m[h] = larger(m[h], w[h * (32 / PER) + k]);
        }
#pragma unroll
        for (int side = 0; side < 2; ++side) {  // the even column, the odd one
            uint32_t o[4];
            Scale4 sc[PER];
#pragma unroll
            for (int h = 0; h < PER; ++h) {
                sc[h] = scale_of<FMT>((side ? m[h] >> 16 : m[h]) & 0x7FFFu, inv_g);
                s_cols[scale_at(2 * cp + side, g * PER + h)] = static_cast<uint8_t>(sc[h].byte);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const Scale4& s = sc[j * PER / 4];
                float2 f[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a = w[8 * j + 2 * i], b = w[8 * j + 2 * i + 1];
                    f[i] = scaled<FMT>(side ? make_float2(hi_f(a), hi_f(b)) : make_float2(lo_f(a), lo_f(b)),
                                       s.inv);
                }
                o[j] = cvt8(f[0], f[1], f[2], f[3]);
                if (!(s.inv > 0.0f)) o[j] = 0;
            }
            if (in) *reinterpret_cast<uint4*>(q + side * ld) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        __syncthreads();
    }

    // the tile's scales, as they lie
    if (threadIdx.x < SB / 16) {
        const int i = threadIdx.x * 16;
        if (ROWS && r0 < total) {
            uint8_t* s = p.s_rows[part] + rt * ((p.cols + 255) / 256) * (2 * SB) + ct * SB + i;
            *reinterpret_cast<uint4*>(s) = *reinterpret_cast<const uint4*>(s_rows + i);
        }
        if (COLS && c0 < p.cols) {
            uint8_t* s = p.s_cols[part] + ct * ((total + 255) / 256) * (2 * SB) + rt * SB + i;
            *reinterpret_cast<uint4*>(s) = *reinterpret_cast<const uint4*>(s_cols + i);
        }
    }
}

template <int FMT, int MODE>
cudaError_t launch(const Fp4QuantParams& p, cudaStream_t st) {
    const long long total = p.gather ? p.rows * p.parts : p.rows;
    long long rt = (total + TILE - 1) / TILE, ct = (p.cols + TILE - 1) / TILE;
    // scales are filled up to 256 along the grouped axis
    if (MODE & FP4_Q_ROWS) ct += ct & 1;
    if (MODE & FP4_Q_COLS) rt += rt & 1;
    if (ct > 0x7FFFFFFFLL || rt > 0x7FFFFFFFLL / ct) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(rt * ct), static_cast<unsigned>(p.gather ? 1 : p.parts), 1);
    cfg.blockDim = dim3(QT, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fp4_quant_kernel<FMT, MODE>, p, static_cast<int>(ct));
}

template <int FMT>
cudaError_t launch_mode(const Fp4QuantParams& p, int mode, cudaStream_t st) {
    switch (mode) {
        case FP4_Q_ROWS: return launch<FMT, FP4_Q_ROWS>(p, st);
        case FP4_Q_COLS: return launch<FMT, FP4_Q_COLS>(p, st);
        case FP4_Q_ROWS | FP4_Q_COLS: return launch<FMT, FP4_Q_ROWS | FP4_Q_COLS>(p, st);
        case FP4_Q_ROWS | FP4_Q_COLS | FP4_Q_SUMS:
            return launch<FMT, FP4_Q_ROWS | FP4_Q_COLS | FP4_Q_SUMS>(p, st);
    }
    return cudaErrorInvalidValue;
}

// ---- the scale of a tensor ---------------------------------------------------------

constexpr int MT = 512, M_PER_SM = 3, M_UNROLL = 4;

// g grows with the largest magnitude, and positive floats compare as integers: each CTA
// raises *scale, which starts at 0, to that of its own values.
__global__ void __launch_bounds__(MT, M_PER_SM)
    fp4_tensor_scale_kernel(const __grid_constant__ Fp4QuantParams p, long long vecs, unsigned* scale) {
    __shared__ uint32_t s_max[MT / 32];
    const uint4* src = static_cast<const uint4*>(p.src[blockIdx.y]);
    const long long step = static_cast<long long>(gridDim.x) * MT;
    uint32_t m = 0;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    for (long long i = static_cast<long long>(blockIdx.x) * MT + threadIdx.x; i < vecs; i += M_UNROLL * step) {
        uint4 v[M_UNROLL];
#pragma unroll
        for (int u = 0; u < M_UNROLL; ++u)
            v[u] = i + u * step < vecs ? __ldg(src + i + u * step) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int u = 0; u < M_UNROLL; ++u) {
            uint32_t x = largest(v[u]);
            if (x >= 0x7F80u) {  // what is not finite does not count
                x = 0;
                for (int j = 0; j < 4; ++j) {
                    const uint32_t w = word(v[u], j) & kMagnitudes;
                    if ((w & 0xFFFFu) < 0x7F80u) x = max(x, w & 0xFFFFu);
                    if ((w >> 16) < 0x7F80u) x = max(x, w >> 16);
                }
            }
            m = max(m, x);
        }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 1; w < MT / 32; ++w) m = max(m, s_max[w]);
        // 6 * 448 = 1.3125 * 2^11
        const int e = static_cast<int>(m >> 7), f = static_cast<int>(m & 0x7Fu);
        const int k = max(e - 127 - 11 + (f > 40 ? 1 : 0), -110);
        atomicMax(scale, static_cast<unsigned>(k + 127) << 23);
    }
}

// ---- back ----------------------------------------------------------------------------

// A CTA takes 128 rows by 256 of K, whose scales lie next to each other; a warp a row at a
// time, 8 values a lane, sixteen rows' values under way before the first use.
constexpr int DT = 256, D_ROWS = 128 / (DT / 32);

template <int FMT>
__global__ void __launch_bounds__(DT, 4)
    fp4_dequant_kernel(long long R, long long K, int kblocks, const uint8_t* __restrict__ q,
                       const uint8_t* __restrict__ s, const float* __restrict__ scale,
                       uint16_t* __restrict__ out) {
    __shared__ uint4 s_scales[fp4_scale_step(FMT) / 16];
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long rt = blockIdx.x / kblocks;
    const int kb = static_cast<int>(blockIdx.x % kblocks);
    const long long r0 = rt * 128 + warp, k = kb * 256LL + lane * 8;
    const long long ld = fp4_ld(K);
    const bool in = k < K;
    const uint8_t* from = q + r0 * ld + k / 2;
    uint32_t u[D_ROWS];
#pragma unroll
    for (int i = 0; i < D_ROWS; ++i)
        u[i] = in && r0 + 8 * i < R ? __ldg(reinterpret_cast<const uint32_t*>(from + 8 * i * ld)) : 0u;
    if (threadIdx.x < fp4_scale_step(FMT) / 16)
        s_scales[threadIdx.x] = __ldg(reinterpret_cast<const uint4*>(s) +
                                      static_cast<long long>(blockIdx.x) * (fp4_scale_step(FMT) / 16) + threadIdx.x);
    float g = 1.0f;
    if constexpr (FMT == FP4_NV) g = inverse_of(scale) == 0.0f ? __uint_as_float(0x7FC00000u) : __ldg(scale);
    __syncthreads();
    if (!in) return;
    const uint8_t* scales = reinterpret_cast<const uint8_t*>(s_scales);
    const uint32_t group = lane * 8 / fp4_group(FMT);
    const bool whole = k + 8 <= K && K % 8 == 0;
    uint16_t* to = out + r0 * K + k;
#pragma unroll
    for (int i = 0; i < D_ROWS; ++i) {
        if (r0 + 8 * i >= R) break;
        const uint32_t byte = scales[scale_at(warp + 8 * i, group)];
        float f;
        if constexpr (FMT == FP4_MX)
            f = __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : byte << 23);
        else
            f = byte >= 0x7F ? __uint_as_float(0x7FC00000u) : e4m3_f(byte) * g;
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t h;
            asm("{\n\t.reg .b8 a, b, c, d;\n\t"
                "mov.b32 {a, b, c, d}, %1;\n\t"
                "cvt.rn.f16x2.e2m1x2 %0, a;\n\t}"
                : "=r"(h)
                : "r"(u[i] >> (8 * j)));
            const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
            const float2 y = __fmul2_rn(x, make_float2(f, f));
            // (exact: 6 significant bits)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[j]) : "f"(y.y), "f"(y.x));
        }
        uint16_t* row = to + 8 * i * K;
        if (whole) {
            *reinterpret_cast<uint4*>(row) = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (k + j < K) row[j] = static_cast<uint16_t>(j & 1 ? o[j / 2] >> 16 : o[j / 2]);
        }
    }
}

}  // namespace

cudaError_t launch_fp4_quant(const Fp4QuantParams& p, int fmt, int mode, cudaStream_t st) {
    return fmt == FP4_NV ? launch_mode<FP4_NV>(p, mode, st) : launch_mode<FP4_MX>(p, mode, st);
}

cudaError_t launch_fp4_tensor_scale(const Fp4QuantParams& p, float* scale, cudaStream_t st) {
    cudaError_t e = cudaMemsetAsync(scale, 0, sizeof(float), st);
    if (e != cudaSuccess) return e;
    const long long vecs = p.rows * p.cols / 8;
    int sms = 0, dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    const long long most = max(1LL, static_cast<long long>(sms) * M_PER_SM / p.parts);
    const long long ctas = min((vecs + MT * M_UNROLL - 1) / (MT * M_UNROLL), most);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(max(ctas, 1LL)), static_cast<unsigned>(p.parts), 1);
    cfg.blockDim = dim3(MT, 1, 1);
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, fp4_tensor_scale_kernel, p, vecs, reinterpret_cast<unsigned*>(scale));
}

cudaError_t launch_fp4_dequant(long long R, long long K, int fmt, const void* q, const void* s,
                               const float* scale, void* out, cudaStream_t st) {
    const long long kb = (K + 255) / 256, rt = (R + 127) / 128;
    if (rt > 0x7FFFFFFFLL / kb) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(rt * kb), 1, 1);
    cfg.blockDim = dim3(DT, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    auto kern = fmt == FP4_NV ? fp4_dequant_kernel<FP4_NV> : fp4_dequant_kernel<FP4_MX>;
    return cudaLaunchKernelEx(&cfg, kern, R, K, static_cast<int>(kb), static_cast<const uint8_t*>(q),
                              static_cast<const uint8_t*>(s), scale, static_cast<uint16_t*>(out));
}

}  // namespace tpmlp
