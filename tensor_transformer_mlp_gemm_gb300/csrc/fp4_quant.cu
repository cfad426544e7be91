// fp4_quant.cu -- quantisation to 4-bit floating point and back (see fp4_quant.cuh for
// the definition).
//
// What bounds it: HBM traffic, 2 bytes read and 0.53 (mx) or 0.56 (nv) written for each
// element and grouping.  So both groupings of a matrix, and the column sums of a gradient
// (the bias gradient), come from one read.
//
// A CTA takes 128 x 128 tiles, whole groups and whole blocks of scales both ways, and copies the
// next into shared memory under the arithmetic of one.  A thread takes 32 columns of two rows,
// then 32 rows of two columns: whole groups, 16 bytes of each output.  (Tiles loaded into
// registers, 8 rows x 8 columns a thread, had every lane of a group work out its scale and
// nothing on the way meanwhile: both groupings of 16384 x 4096 43 us, now 40, with the sums 46,
// now 42; threads of 16 rows or columns, 512 in a CTA, took 45 us.)  No unit is full: it issues in
// 65 (mx) and 71 % (nv) of the cycles, two and 2.5 instructions a value and grouping for the
// conversion alone, has the ALU busy for 70 % and DRAM for 55 and 44 %; with six warps for each
// scheduler most of what waits does so for the barrier behind a tile.
#include <cuda_fp16.h>

#include "fp4_cvt.cuh"
#include "fp4_quant.cuh"
#include "fp8_mma.cuh"
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

constexpr int Q_PER_SM = 3;
// A row of a tile in shared memory takes 17 times 16 bytes, and every 32 rows 32 bytes more: the
// eight rows that a quarter of a warp reads 16 bytes of, and the four runs of 32 rows that a
// warp reads words of, meet different banks.
constexpr int Q_PITCH = 272;
constexpr int Q_STAGE = 35072;
__device__ __forceinline__ uint32_t row_at(int r) { return r * Q_PITCH + (r >> 5) * 32; }
static_assert(127 * Q_PITCH + 3 * 32 + 256 <= Q_STAGE && Q_STAGE % 128 == 0, "a tile's rows");
constexpr int Q_SMEM = 2 * Q_STAGE;
static_assert(Q_PER_SM * (Q_SMEM + 4 * 1024 + 1024) <= 228 * 1024, "shared memory of an SM");

// The pair of largest magnitudes among 8 values.
__device__ __forceinline__ uint32_t largest2(const uint4& v) {
    return larger(larger(v.x, v.y), larger(v.z, v.w));
}

// Copies `bytes` (a multiple of 16) to shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

template <int FMT, int MODE>
__global__ void __launch_bounds__(QT, Q_PER_SM)
    fp4_quant_kernel(const __grid_constant__ Fp4QuantParams p, unsigned row_tiles, unsigned col_tiles,
                     unsigned tiles) {
    constexpr bool ROWS = MODE & FP4_Q_ROWS, COLS = MODE & FP4_Q_COLS, SUMS = MODE & FP4_Q_SUMS;
    constexpr int SB = fp4_scale_step(FMT) / 2;  // bytes of a tile's scales
    constexpr int PER = FMT == FP4_NV ? 2 : 1;   // groups of 32 elements
    extern __shared__ __align__(128) uint8_t s_tiles[];
    __shared__ alignas(16) uint8_t s_rows[2][ROWS ? SB : 16];
    __shared__ alignas(16) uint8_t s_cols[2][COLS ? SB : 16];
    __shared__ alignas(8) uint64_t s_bar[2];
    __shared__ volatile int s_abort;

    const long long total = p.gather ? p.rows * p.parts : p.rows;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t tile0 = ptx::smem_u32(s_tiles), bar0 = ptx::smem_u32(s_bar);

    // Tiles part by part, row by row from the last on (which whoever wrote or read the matrix left
    // in L2: a weight of 12288 x 4608 behind its tensor's scale 2 us), each CTA every
    // gridDim.x-th; stepped, not divided out.
    struct Tile {
        unsigned part, rt, ct;
    };
    const unsigned each = row_tiles * col_tiles;
    auto tile_of = [&](unsigned t) { return Tile{t / each, t % each / col_tiles, t % col_tiles}; };
    const Tile step = tile_of(gridDim.x);
    auto next_of = [&](Tile x) {
        x.ct += step.ct;
        x.rt += step.rt;
        x.part += step.part;
        if (x.ct >= col_tiles) {
            x.ct -= col_tiles;
            ++x.rt;
        }
        if (x.rt >= row_tiles) {
            x.rt -= row_tiles;
            ++x.part;
        }
        return x;
    };
    // Starts a tile's way into buffer b: thread r copies row r, and zeroes what the matrix does
    // not have of it.
    int loads = 0;
    auto load = [&](const Tile& x, int b) {
        if (blockIdx.x == gridDim.x - 1 && loads == p.stall) return;
        ++loads;
        const long long r0 = static_cast<long long>(row_tiles - 1 - x.rt) * TILE, c0 = static_cast<long long>(x.ct) * TILE;
        const int rows = total - r0 < TILE ? static_cast<int>(max(0LL, total - r0)) : TILE;
        const int bytes = 2 * (p.cols - c0 < TILE ? static_cast<int>(max(0LL, p.cols - c0)) : TILE);
        if (threadIdx.x == 0) ptx::mbar_arrive_expect_tx(bar0 + 8 * b, rows * bytes);
        if (threadIdx.x < TILE) {
            const int r = threadIdx.x;
            const int here = r < rows ? bytes : 0;
            if (here > 0) {
                unsigned from = x.part;
                long long row = r0 + r;
                if (p.gather && p.parts > 1) {  // (chunks of whole tiles)
                    const unsigned chunk = static_cast<unsigned>(p.rows / TILE);
                    from = (row_tiles - 1 - x.rt) / chunk;
                    row -= static_cast<long long>(from) * p.rows;
                }
                bulk_load(tile0 + b * Q_STAGE + row_at(r),
                          static_cast<const uint16_t*>(p.src[from]) + row * p.cols + c0, here, bar0 + 8 * b);
            }
            if (here < 2 * TILE) {
                uint4* to = reinterpret_cast<uint4*>(s_tiles + b * Q_STAGE + row_at(r));
                for (int i = here / 16; i < TILE / 8; ++i) to[i] = make_uint4(0, 0, 0, 0);
            }
        }
    };

    if (threadIdx.x == 0) {
        ptx::mbar_init(bar0, 1);
        ptx::mbar_init(bar0 + 8, 1);
        s_abort = 0;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    __syncthreads();
    // The dependent launch after the wait: what came before this grid has ended when it starts,
    // so that it may read weights before this grid ends.
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    float inv_g = 0.0f;
    if constexpr (FMT == FP4_NV) inv_g = inverse_of(p.scale);
    int b = 0;
    uint32_t phase = 0;
    Tile x = tile_of(blockIdx.x);
    load(x, 0);
    __syncthreads();  // (zeroes)
    int done = 0;
    for (unsigned t = blockIdx.x; t < tiles; t += gridDim.x, ++done) {
        const Tile next = next_of(x);
        if (t + gridDim.x < tiles) load(next, b ^ 1);
        const bool ok = f8::wait(bar0 + 8 * b, phase, &s_abort, p.timeout_ns, p.err, ERR_EPILOGUE);
        const unsigned rt = row_tiles - 1 - x.rt;
        const long long r0 = static_cast<long long>(rt) * TILE, c0 = static_cast<long long>(x.ct) * TILE;
        const uint8_t* tile = s_tiles + b * Q_STAGE;
        if (ROWS && ok) {
            const int run = lane >> 3;  // a thread takes 32 columns of two rows
            const long long c = c0 + run * 32;
            uint8_t* q = p.q_rows[x.part];
            const long long ld = fp4_ld(p.rows_k);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = warp * 16 + (lane & 7) + 8 * i;
                const uint4* src = reinterpret_cast<const uint4*>(tile + row_at(r) + run * 64);
                const uint4 v[4] = {src[0], src[1], src[2], src[3]};
                uint32_t o[4];
#pragma unroll
                for (int h = 0; h < PER; ++h) {
                    uint32_t m = larger(largest2(v[h * 2]), largest2(v[h * 2 + 1]));
                    if constexpr (PER == 1) m = larger(m, larger(largest2(v[2]), largest2(v[3])));
                    const Scale4 sc = scale_of<FMT>(fold(m), inv_g);
                    s_rows[b][scale_at(r, run * PER + h)] = static_cast<uint8_t>(sc.byte);
#pragma unroll
                    for (int j = h * (4 / PER); j < (h + 1) * (4 / PER); ++j) {
                        float2 f[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t w = word(v[j], e);
                            f[e] = scaled<FMT>(make_float2(lo_f(w), hi_f(w)), sc.inv);
                        }
                        o[j] = cvt8(f[0], f[1], f[2], f[3]);
                        if (!(sc.inv > 0.0f)) o[j] = 0;
                    }
                }
                if (c < p.cols && r0 + r < total)
                    *reinterpret_cast<uint4*>(q + (r0 + r) * ld + c / 2) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
        if (COLS && ok) {
            const int g = lane & 3, cp = warp * 8 + (lane >> 2);  // 32 rows, two columns
            const uint32_t* src = reinterpret_cast<const uint32_t*>(tile + row_at(32 * g)) + cp;
            uint32_t w[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) w[k] = src[k * (Q_PITCH / 4)];
            const long long cc = c0 + 2 * cp;
            const long long ld = fp4_ld(total);
            const bool in = cc < p.cols && r0 + 32 * g < total;
            uint8_t* q = p.q_cols[x.part] + cc * ld + r0 / 2 + g * 16;
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
                    s_cols[b][scale_at(2 * cp + side, g * PER + h)] = static_cast<uint8_t>(sc[h].byte);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const Scale4& s = sc[j * PER / 4];
                    float2 f[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t u = w[8 * j + 2 * i], y = w[8 * j + 2 * i + 1];
                        f[i] = scaled<FMT>(side ? make_float2(hi_f(u), hi_f(y)) : make_float2(lo_f(u), lo_f(y)),
                                           s.inv);
                    }
                    o[j] = cvt8(f[0], f[1], f[2], f[3]);
                    if (!(s.inv > 0.0f)) o[j] = 0;
                }
                if (in) *reinterpret_cast<uint4*>(q + side * ld) = make_uint4(o[0], o[1], o[2], o[3]);
            }
            if constexpr (SUMS) {
                // 32 rows in order, then the four groups of them; read again, which takes fewer
                // registers than they have until here
                asm volatile("" ::: "memory");
                float2 s = make_float2(0.0f, 0.0f);
#pragma unroll 8
                for (int k = 0; k < 32; ++k) {
                    const uint32_t u = src[k * (Q_PITCH / 4)];
                    s = __fadd2_rn(s, make_float2(lo_f(u), hi_f(u)));
                }
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
                    s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
                }
                if (g == 0 && cc < p.cols && r0 < total)
                    *reinterpret_cast<float2*>(p.sums[x.part] + rt * p.sums_ld + cc) = s;
            }
        }
        // the buffer has been read and the scales are there; who gave up takes the others along
        ptx::fence_proxy_async_smem();
        if (__syncthreads_or(!ok)) {
            // what is still on its way lands before the CTA leaves
            if (threadIdx.x == 0) {
                if (loads > done) f8::drain(bar0 + 8 * b, phase, p.timeout_ns, p.err);
                if (loads > done + 1) f8::drain(bar0 + 8 * (b ^ 1), phase ^ b, p.timeout_ns, p.err);
            }
            return;
        }
        if (threadIdx.x < SB / 16) {
            const int i = threadIdx.x * 16;
            // (tiles times bytes pass 2^32 from 2^29 of K on)
            if (ROWS && r0 < total) {
                uint8_t* s = p.s_rows[x.part] + rt * ((p.rows_k + 255) / 256) * (2 * SB) + static_cast<long long>(x.ct) * SB + i;
                *reinterpret_cast<uint4*>(s) = *reinterpret_cast<const uint4*>(&s_rows[b][i]);
            }
            if (COLS && c0 < p.cols) {
                uint8_t* s = p.s_cols[x.part] + x.ct * ((total + 255) / 256) * (2 * SB) + static_cast<long long>(rt) * SB + i;
                *reinterpret_cast<uint4*>(s) = *reinterpret_cast<const uint4*>(&s_cols[b][i]);
            }
        }
        phase ^= b;
        b ^= 1;
        x = next;
    }
}

template <int FMT, int MODE>
cudaError_t launch(const Fp4QuantParams& p, cudaStream_t st) {
    constexpr int kDevices = 64;
    static int sms[kDevices] = {};  // asked once a device, with the kernel's attribute
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    int n = __atomic_load_n(&sms[dev], __ATOMIC_ACQUIRE);
    if (n == 0) {
        e = cudaFuncSetAttribute(fp4_quant_kernel<FMT, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, Q_SMEM);
        if (e != cudaSuccess) return e;
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        __atomic_store_n(&sms[dev], n, __ATOMIC_RELEASE);
    }
    const long long total = p.gather ? p.rows * p.parts : p.rows;
    long long rt = (total + TILE - 1) / TILE, ct = (p.cols + TILE - 1) / TILE;
    // scales are filled up to 256 along the grouped axis
    if (MODE & FP4_Q_ROWS) ct += ct & 1;
    if (MODE & FP4_Q_COLS) rt += rt & 1;
    const long long parts = p.gather ? 1 : p.parts;
    if (rt > 0x7FFFFFFFLL / ct / parts) return cudaErrorInvalidValue;
    const long long tiles = rt * ct * parts, most = static_cast<long long>(n) * Q_PER_SM;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles < most ? tiles : most), 1, 1);
    cfg.blockDim = dim3(QT, 1, 1);
    cfg.dynamicSmemBytes = Q_SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fp4_quant_kernel<FMT, MODE>, p, static_cast<unsigned>(rt),
                              static_cast<unsigned>(ct), static_cast<unsigned>(tiles));
}

// ---- few rows, by rows alone -------------------------------------------------------
// A thread takes 32 columns of a row, straight from and to global memory.  For up to FEW values:
// the product waits for this launch, and without shared memory in use its CTAs find room beside
// these (whole calls with this and with the tiles: 48 tokens, 12288 -> 12288 features in eight
// row shards 20.7 us, 24.3; 256 x 4096 tokens 11.0, 12.5; but 777 x 2080 19.0, 17.1).

constexpr long long FEW = 1 << 20;
constexpr int RT = 128;

template <int FMT>
__global__ void __launch_bounds__(RT)
    fp4_quant_few_kernel(const __grid_constant__ Fp4QuantParams p, int row_tiles, int runs) {
    constexpr int PER = FMT == FP4_NV ? 2 : 1;  // groups of 32
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const long long i = static_cast<long long>(blockIdx.x) * RT + threadIdx.x;
    const long long row = i / runs;
    const int run = static_cast<int>(i - row * runs), part = blockIdx.y;
    if (row >= row_tiles * 128LL) return;
    float inv_g = 0.0f;
    if constexpr (FMT == FP4_NV) inv_g = inverse_of(p.scale);
    const bool in = row < p.rows && run * 32LL < p.cols;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.src[part]) +
                                                      (in ? row * p.cols + run * 32LL : 0));
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = in ? __ldg(src + j) : make_uint4(0, 0, 0, 0);
    uint8_t* scales = p.s_rows[part] + (row >> 7) * ((p.rows_k + 255) / 256) * fp4_scale_step(FMT);
    uint32_t o[4];
#pragma unroll
    for (int h = 0; h < PER; ++h) {
        uint32_t m = larger(largest2(v[h * 2]), largest2(v[h * 2 + 1]));
        if constexpr (PER == 1) m = larger(m, larger(largest2(v[2]), largest2(v[3])));
        const Scale4 sc = scale_of<FMT>(fold(m), inv_g);
        const int group = run * PER + h;
        scales[(group >> 2) * 512LL + scale_at(row & 127, group & 3)] = static_cast<uint8_t>(sc.byte);
#pragma unroll
        for (int j = h * (4 / PER); j < (h + 1) * (4 / PER); ++j) {
            float2 f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t w = word(v[j], e);
                f[e] = scaled<FMT>(make_float2(lo_f(w), hi_f(w)), sc.inv);
            }
            o[j] = cvt8(f[0], f[1], f[2], f[3]);
            if (!(sc.inv > 0.0f)) o[j] = 0;
        }
    }
    if (in)
        *reinterpret_cast<uint4*>(p.q_rows[part] + row * fp4_ld(p.rows_k) + run * 16LL) =
            make_uint4(o[0], o[1], o[2], o[3]);
}

template <int FMT>
cudaError_t launch_few(const Fp4QuantParams& p, cudaStream_t st) {
    const long long rt = (p.rows + 127) / 128, runs = (p.cols + 255) / 256 * 8;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(rt * runs), static_cast<unsigned>(p.parts), 1);  // 128 rows each
    cfg.blockDim = dim3(RT, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fp4_quant_few_kernel<FMT>, p, static_cast<int>(rt), static_cast<int>(runs));
}

template <int FMT>
cudaError_t launch_mode(const Fp4QuantParams& p, int mode, cudaStream_t st) {
    switch (mode) {
        case FP4_Q_ROWS:
            return p.rows * p.cols * p.parts <= FEW && (!p.gather || p.parts == 1) ? launch_few<FMT>(p, st)
                                                                     : launch<FMT, FP4_Q_ROWS>(p, st);
        case FP4_Q_COLS: return launch<FMT, FP4_Q_COLS>(p, st);
        case FP4_Q_ROWS | FP4_Q_COLS: return launch<FMT, FP4_Q_ROWS | FP4_Q_COLS>(p, st);
        case FP4_Q_ROWS | FP4_Q_COLS | FP4_Q_SUMS:
            return launch<FMT, FP4_Q_ROWS | FP4_Q_COLS | FP4_Q_SUMS>(p, st);
    }
    return cudaErrorInvalidValue;
}

// ---- the scale of a tensor ---------------------------------------------------------

// The largest finite magnitude (as bits) of eight values and m.
__device__ __forceinline__ uint32_t largest_finite(const uint4& v, uint32_t m) {
    uint32_t x = largest(v);
    if (x >= 0x7F80u) {  // what is not finite does not count
        x = 0;
        for (int j = 0; j < 4; ++j) {
            const uint32_t w = word(v, j) & kMagnitudes;
            if ((w & 0xFFFFu) < 0x7F80u) x = max(x, w & 0xFFFFu);
            if ((w >> 16) < 0x7F80u) x = max(x, w >> 16);
        }
    }
    return max(m, x);
}

// The largest of a CTA's threads, in its first warp.
template <int THREADS>
__device__ __forceinline__ uint32_t largest_of_cta(uint32_t m) {
    __shared__ uint32_t s_max[THREADS / 32];
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x < 32) m = __reduce_max_sync(0xffffffffu, s_max[threadIdx.x % (THREADS / 32)]);
    return m;
}

// g for this largest magnitude, as bits: 6 * 448 = 1.3125 * 2^11
__device__ __forceinline__ uint32_t tensor_scale_of(uint32_t m) {
    const int e = static_cast<int>(m >> 7), f = static_cast<int>(m & 0x7Fu);
    return static_cast<uint32_t>(max(e - 127 - 11 + (f > 40 ? 1 : 0), -110) + 127) << 23;
}

// Bound by the read alone: 12288 x 4608 20 us, 5.7 TB/s, 4 vectors a thread under way.
constexpr int MT = 512, M_PER_SM = 3, M_UNROLL = 4;

// *scale = 0, by a kernel: behind a memset the next kernel would start only when it has ended.
__global__ void fp4_zero_kernel(unsigned* scale) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    *scale = 0;
}

// g grows with the largest magnitude, and positive floats compare as integers: each CTA
// raises *scale, which starts at 0, to that of its own values.  What came before has ended when
// this starts (fp4_zero_kernel lets it), so only *scale is waited for.
__global__ void __launch_bounds__(MT, M_PER_SM)
    fp4_tensor_scale_kernel(const __grid_constant__ Fp4QuantParams p, long long vecs, unsigned* scale) {
    const uint4* src = static_cast<const uint4*>(p.src[blockIdx.y]);
    const long long step = static_cast<long long>(gridDim.x) * MT;
    uint32_t m = 0;
    ptx::griddep_launch_dependents();
    for (long long i = static_cast<long long>(blockIdx.x) * MT + threadIdx.x; i < vecs; i += M_UNROLL * step) {
        uint4 v[M_UNROLL];
#pragma unroll
        for (int u = 0; u < M_UNROLL; ++u)
            v[u] = i + u * step < vecs ? __ldg(src + i + u * step) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int u = 0; u < M_UNROLL; ++u) m = largest_finite(v[u], m);
    }
    m = largest_of_cta<MT>(m);
    if (threadIdx.x == 0) {
        ptx::griddep_wait();
        atomicMax(scale, tensor_scale_of(m));
    }
}

// Small tensors in one launch, by one cluster whose CTAs hand their largest to the first: as many
// vectors in all parts as its threads have on the way at once.  (By this and by two launches, us of
// the device one behind the other, of the host: 1 x 4096 1.65, 1.8 and 2.9, 4.6; 16 x 12288 2.3, 1.95
// and 2.9, 4.5; but 128 x 4096 3.7, 2.2.  The wait for the cluster's start takes 0.04 to 0.1 of it.)
constexpr int CT = 1024, C_CTAS = 8;
constexpr unsigned ONE = C_CTAS * CT * M_UNROLL;

__global__ void __cluster_dims__(C_CTAS, 1, 1) __launch_bounds__(CT, 1)
    fp4_small_scale_kernel(const __grid_constant__ Fp4QuantParams p, unsigned vecs, unsigned* scale) {
    __shared__ uint32_t s_all[C_CTAS];
    // (the first CTA's shared memory is there once it has started: all have by the wait below)
    ptx::cluster_arrive_relaxed();
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const unsigned all = vecs * p.parts;
    uint4 v[M_UNROLL];
#pragma unroll
    for (int u = 0; u < M_UNROLL; ++u) {
        const unsigned at = (u * C_CTAS + blockIdx.x) * CT + threadIdx.x, part = at < all ? at / vecs : 0;
        v[u] = at < all ? __ldg(static_cast<const uint4*>(p.src[part]) + (at - part * vecs))
                        : make_uint4(0, 0, 0, 0);
    }
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < M_UNROLL; ++u) m = largest_finite(v[u], m);
    m = largest_of_cta<CT>(m);
    __syncwarp();
    ptx::cluster_wait();
    if (threadIdx.x == 0)
        f8::store_cluster(ptx::mapa_shared(ptx::smem_u32(&s_all[blockIdx.x]), 0), static_cast<int>(m));
    __syncwarp();
    ptx::cluster_sync();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        for (int i = 0; i < C_CTAS; ++i) m = max(m, s_all[i]);
        *scale = tensor_scale_of(m);
    }
}

// ---- back ----------------------------------------------------------------------------

// A CTA takes 128 rows by 256 of K, whose scales lie next to each other; a warp a row at a
// time, 8 values a lane, sixteen rows' values under way before the first use.  Bound by HBM, most
// of it the bf16 result: 16384 x 4096 27 us, 6.3 TB/s.
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

cudaError_t launch_fp4_quant(const Fp4QuantParams& params, int fmt, int mode, cudaStream_t st) {
    Fp4QuantParams p = params;
    if (p.rows_k == 0) p.rows_k = p.cols;
    return fmt == FP4_NV ? launch_mode<FP4_NV>(p, mode, st) : launch_mode<FP4_MX>(p, mode, st);
}

int fp4_tensor_scale_kernels(const Fp4QuantParams& p) { return p.rows * p.cols / 8 <= ONE / p.parts ? 1 : 2; }

cudaError_t launch_fp4_tensor_scale(const Fp4QuantParams& p, float* scale, cudaStream_t st) {
    cudaError_t e;
    const long long vecs = p.rows * p.cols / 8;
    if (fp4_tensor_scale_kernels(p) == 1) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(C_CTAS, 1, 1);
        cfg.blockDim = dim3(CT, 1, 1);
        cfg.stream = st;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, fp4_small_scale_kernel, p, static_cast<unsigned>(vecs),
                                  reinterpret_cast<unsigned*>(scale));
    }
    int sms = 0, dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    const long long most = max(1LL, static_cast<long long>(sms) * M_PER_SM / p.parts);
    const long long ctas = min((vecs + MT * M_UNROLL - 1) / (MT * M_UNROLL), most);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1, 1, 1);
    cfg.blockDim = dim3(1, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, fp4_zero_kernel, reinterpret_cast<unsigned*>(scale));
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(max(ctas, 1LL)), static_cast<unsigned>(p.parts), 1);
    cfg.blockDim = dim3(MT, 1, 1);
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
