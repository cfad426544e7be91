// fp8_gemm.cu -- the 8-bit product with scales per block of 128 on tcgen05 CTA
// pairs (see fp8_gemm.cuh for the mathematics).
//
// A scale changes every 128 of K, so the sum over K cannot stay in tensor
// memory: each K block's 256 x 256 partial sums go to one of two accumulators
// there, and the epilogue warps read them back, multiply by the block's scales
// and add them up in fp32 registers while the tensor cores fill the other
// accumulator.
//
// CTA layout (384 threads, persistent over tiles; both CTAs of a pair):
//   warp 0       TMA producer: this CTA's 128 rows of A and of B for each K block
//   warp 1       owns the tensor memory; in the even CTA issues the pair's MMAs,
//                four K slices of 32 for each K block
//   warps 2, 3   idle (registers move between whole warpgroups)
//   warps 4..11  promotion and output: warp w reads lanes 32 (w % 4) .. of the
//                accumulator, columns 128 ((w - 4) / 4) .., so a thread keeps 128
//                sums of one row in registers, and the 128 columns share one
//                weight block
// 128 sums, the 32 values read and the addresses do not fit the 168 registers a
// thread of 384 can launch with (measured: 450 bytes of spills): the first
// warpgroup gives most of its registers to the other two.
// What bounds it: the tensor cores at 512 clocks for a K block of a pair's tile
// if the promotion of 128 x 256 sums per CTA (half the fp32 rate with single
// multiply-adds, a quarter with the packed ones used here) stays below that.
//
// Every wait is bounded as in the bf16 GEMM: a wait that expires sets a flag
// that ends the CTA's roles, copies and MMAs in flight are drained (bounded),
// tensor memory is freed, and the error word tells the host.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fp8_gemm.cuh"
#include "fp8_mma.cuh"

namespace tpmlp {
namespace {

using namespace f8;

constexpr int F_THREADS = 384;
// 128 x 56 + 256 x 216 = 62464 of the 384 x 168 = 64512 registers at launch
constexpr int F_FEW_REGS = 56, F_MANY_REGS = 216;
constexpr int F_EPI_WARPS = 8;
constexpr int F_TILE = 256;        // pair tile rows and columns
constexpr int F_STAGE_BYTES = 2 * F8_BOX_BYTES;
constexpr int F_STORE_BYTES = F_EPI_WARPS * 4096;  // per warp: 2 bf16 boxes or 1 fp32 box
constexpr int F_TMEM_COLS = 512;

template <int OUT>
struct Cfg {
    static constexpr bool kVec = OUT == F8_F32_VECTOR;
    static constexpr int kStages = kVec ? 5 : 6;
    // column factors: two K blocks of 128 floats per warp
    static constexpr int kColBytes = kVec ? F_EPI_WARPS * 2 * 512 : 0;
    static constexpr int kSmem = 1024 + kStages * F_STAGE_BYTES + F_STORE_BYTES + kColBytes + 256;
};
static_assert(Cfg<F8_BF16_BLOCK>::kSmem <= 232448 && Cfg<F8_F32_VECTOR>::kSmem <= 232448, "fits a CTA");

__device__ __forceinline__ void decode(const Fp8GemmParams& p, int tile, int& g, int& m0, int& n0) {
    // bands of `band` M-tiles, M fastest: the pairs running together share B
    const int nt = p.ntiles * p.groups;
    const int b = tile / (p.band * nt);
    const int r = tile - b * p.band * nt;
    const int rows = min(p.band, p.mtiles - b * p.band);
    const int ntg = r / rows;
    g = ntg / p.ntiles;
    m0 = (b * p.band + r % rows) * F_TILE;
    n0 = (ntg - g * p.ntiles) * F_TILE;
}

__device__ __forceinline__ int pick(int part, int g, int s) {
    return part == F8_GROUP ? g : part == F8_KSEG ? s : 0;
}

// 128 x 128-byte box of an operand: rows from `row`, K from k0
__device__ __forceinline__ void load_box(const CUtensorMap* m, int mn, int row, int k0, uint32_t dst,
                                         uint32_t bar) {
    ptx::tma_load_2d_pair(dst, m, mn ? row : k0, mn ? k0 : row, bar);
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

template <int OUT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(F_THREADS, 1)
    fp8_gemm_kernel(const __grid_constant__ Fp8GemmParams p) {
    using C = Cfg<OUT>;
    constexpr int NST = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t store0 = base + NST * F_STAGE_BYTES;
    uint8_t* col_area = gbase + NST * F_STAGE_BYTES + F_STORE_BYTES;
    const uint32_t bar0 = store0 + F_STORE_BYTES + C::kColBytes;
    uint8_t* bar_area = col_area + C::kColBytes;
    const uint32_t bar_full = bar0;              // [NST] used in the even CTA
    const uint32_t bar_empty = bar0 + 8 * NST;   // [NST] both CTAs
    const uint32_t bar_tfull = bar0 + 16 * NST;  // [2] both CTAs
    const uint32_t bar_tempty = bar_tfull + 16;  // [2] used in the even CTA
    const uint32_t bar_drain = bar_tempty + 16;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_area + 16 * NST + 40);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bar_area + 16 * NST + 44);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(ptx::cluster_ctarank());
    const int cluster = blockIdx.x / 2, nclusters = gridDim.x / 2;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NST; ++s) {
            ptx::mbar_init(bar_full + 8 * s, 1);
            ptx::mbar_init(bar_empty + 8 * s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(bar_tfull + 8 * a, 1);
            ptx::mbar_init(bar_tempty + 8 * a, 2 * F_EPI_WARPS);
        }
        ptx::mbar_init(bar_drain, 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(ptx::smem_u32(tmem_slot), F_TMEM_COLS);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    __syncwarp();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    ptx::griddep_wait();

    const int kblocks = (p.K + F8_BK - 1) / F8_BK;
    const int nk = kblocks * p.ksegs;

    if (warp < 4) {
        reg_dec<F_FEW_REGS>();
        if (warp == 0 && lane == 0) {
            const uint32_t even_full = ptx::mapa_shared(bar_full, 0);
            int stage = 0;
            uint32_t phase = 0;
            long long fills = 0;
            bool ok = true;
            for (int tile = cluster; ok && tile < p.total_tiles; tile += nclusters) {
                if (tile + nclusters >= p.total_tiles) ptx::griddep_launch_dependents();
                int g, m0, n0;
                decode(p, tile, g, m0, n0);
                const int arow = m0 + rank * 128, brow = n0 + rank * 128;
                for (int s = 0; ok && s < p.ksegs; ++s) {
                    const CUtensorMap* am = p.a_map + pick(p.a_part, g, s);
                    const CUtensorMap* bm = p.b_map + pick(p.b_part, g, s);
                    for (int kb = 0; kb < kblocks; ++kb) {
                        if (!wait<false>(bar_empty + 8 * stage, phase ^ 1u, abort_flag, p.timeout_ns,
                                         p.err, ERR_PRODUCER)) {
                            ok = false;
                            break;
                        }
                        const uint32_t sa = base + stage * F_STAGE_BYTES;
                        if (rank == 0)
                            ptx::mbar_arrive_expect_tx(bar_full + 8 * stage, 2 * F_STAGE_BYTES);
                        load_box(am, p.a_mn, arow, kb * F8_BK, sa, even_full + 8 * stage);
                        load_box(bm, p.b_mn, brow, kb * F8_BK, sa + F8_BOX_BYTES,
                                 even_full + 8 * stage);
                        ++fills;
                        if (++stage == NST) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                }
            }
            if (ok) {
                // no release of a stage may arrive after this CTA has left
                for (int i = 0; i < NST; ++i) {
                    if (!drain(bar_empty + 8 * stage, phase ^ 1u, p.timeout_ns, p.err)) break;
                    if (++stage == NST) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            } else if (rank == 0) {
                for (long long f = (fills > NST ? fills - NST : 0); f < fills; ++f) {
                    const int st = static_cast<int>(f % NST);
                    if (!drain(bar_full + 8 * st, static_cast<uint32_t>((f / NST) & 1), p.timeout_ns,
                               p.err))
                        break;
                }
            }
        } else if (warp == 1 && lane == 0 && rank == 0) {
            const uint32_t id = idesc(F_TILE, F_TILE, p.a_mn, p.b_mn) | p.ab_format;
            int stage = 0;
            uint32_t phase = 0;
            long long blk = 0;  // K blocks issued
            bool ok = true;
            for (int tile = cluster; ok && tile < p.total_tiles; tile += nclusters) {
                for (int kk = 0; kk < nk; ++kk, ++blk) {
                    const int acc = static_cast<int>(blk & 1);
                    if (!wait<true>(bar_tempty + 8 * acc, static_cast<uint32_t>((blk >> 1) & 1) ^ 1u,
                                    abort_flag, p.timeout_ns, p.err, ERR_MMA) ||
                        !wait<false>(bar_full + 8 * stage, phase, abort_flag, p.timeout_ns, p.err,
                                     ERR_MMA)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint32_t sa = base + stage * F_STAGE_BYTES;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_pair(tmem + acc * 256, operand_desc(sa, k, p.a_mn),
                                 operand_desc(sa + F8_BOX_BYTES, k, p.b_mn), id, k > 0 ? 1u : 0u);
                    ptx::mma_commit_pair_multicast(bar_empty + 8 * stage, 0x3);
                    ptx::mma_commit_pair_multicast(bar_tfull + 8 * acc, 0x3);
                    if (++stage == NST) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            ptx::mma_commit_pair(bar_drain);
            drain(bar_drain, 0, p.timeout_ns, p.err);
            if (ok) {
                // the last releases of both accumulators arrive on this CTA
                for (long long j = (blk > 2 ? blk - 2 : 0); j < blk; ++j)
                    if (!drain(bar_tempty + 8 * (j & 1), static_cast<uint32_t>((j >> 1) & 1),
                               p.timeout_ns, p.err))
                        break;
            }
        }
    } else {
        reg_inc<F_MANY_REGS>();
        const int quarter = warp & 3;         // the accumulator lanes this warp may read
        const int half = (warp - 4) >> 2;     // its 128 columns
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * 128;
        const uint32_t even_tempty = ptx::mapa_shared(bar_tempty, 0);
        uint8_t* store = gbase + NST * F_STAGE_BYTES + (warp - 4) * 4096;
        const uint32_t store_u32 = store0 + (warp - 4) * 4096;
        float* colbuf = reinterpret_cast<float*>(col_area + (warp - 4) * 1024);
        long long blk = 0;
        bool ok = true;
        for (int tile = cluster; ok && tile < p.total_tiles; tile += nclusters) {
            int g, m0, n0;
            decode(p, tile, g, m0, n0);
            const int row0 = m0 + rank * 128 + quarter * 32;
            const int m = row0 + lane, n = n0 + half * 128;
            const bool row_in = m < p.M, col_in = n < p.N;
            uint64_t acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0;
            // scales of K block (s, kb), fetched one block ahead
            auto scales = [&](int s, int kb, float& a, float& b, float4& bv) {
                a = row_in ? __ldg(p.sa[pick(p.a_part, g, s)] + kb * p.sa_kb + m) : 0.0f;
                const float* sb = p.sb[pick(p.b_part, g, s)] + kb * p.sb_kb;
                if constexpr (C::kVec) {
                    const int nn = n + lane * 4;
                    bv = nn < p.N ? __ldg(reinterpret_cast<const float4*>(sb + nn))
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
                } else {
                    b = col_in ? __ldg(sb + (n >> 7) * p.sb_n) : 0.0f;
                }
            };
            float a = 0.0f, b = 1.0f;
            float4 bv = make_float4(0.f, 0.f, 0.f, 0.f);
            if (nk > 0) scales(0, 0, a, b, bv);
            int s = 0, kb = 0;
            for (int kk = 0; kk < nk; ++kk, ++blk) {
                const float scale = a * b;
                float* cb = colbuf + (blk & 1) * 128;
                if constexpr (C::kVec) {
                    // two buffers: the lanes that still read the other one are at most a block behind
                    *reinterpret_cast<float4*>(cb + lane * 4) = bv;
                    __syncwarp();
                }
                if (++kb == kblocks) {
                    kb = 0;
                    ++s;
                }
                if (kk + 1 < nk) scales(s, kb, a, b, bv);
                const int ab = static_cast<int>(blk & 1);
                ok = wait<false>(bar_tfull + 8 * ab, static_cast<uint32_t>((blk >> 1) & 1),
                                 abort_flag, p.timeout_ns, p.err, ERR_EPILOGUE);
                ok = __all_sync(0xffffffffu, ok);  // the warp gives up together
                if (!ok) break;
                ptx::tc_fence_after();
                promote<128, C::kVec>(lanes + ab * 256, scale,
                                      reinterpret_cast<const uint64_t*>(cb), acc);
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_cluster(even_tempty + 8 * ab);
            }
            if (!ok) break;
            // output: 32 columns at a time through this warp's staging box
            if (!col_in || row0 >= p.M) continue;
            int part = g, y0 = row0;
            if (p.chunk_rows > 0) {
                part = row0 / p.chunk_rows;
                y0 -= part * p.chunk_rows;
            }
            const __nv_bfloat16* bias =
                p.bias ? static_cast<const __nv_bfloat16*>(p.bias) + static_cast<long long>(g) * p.N
                       : nullptr;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int nn = n + c * 32;
                if (nn < p.N) {
                    float x[32];
#pragma unroll
                    for (int i = 0; i < 16; ++i) unpack2(acc[c * 16 + i], x[2 * i], x[2 * i + 1]);
                    uint8_t* box = C::kVec ? store : store + (c & 1) * 2048;
                    const uint32_t box_u32 = C::kVec ? store_u32 : store_u32 + (c & 1) * 2048;
                    if (lane == 0) {
                        if (C::kVec) ptx::bulk_wait_group_read<0>();
                        else ptx::bulk_wait_group_read<1>();
                    }
                    __syncwarp();
                    if constexpr (C::kVec) {
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            *reinterpret_cast<float4*>(box + lane * 128 + ((q ^ (lane & 7)) << 4)) =
                                make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
                    } else {
                        if (bias) {
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                if (nn + 8 * q < p.N) {
                                    const uint4 u = __ldg(reinterpret_cast<const uint4*>(bias + nn + 8 * q));
                                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                                    for (int j = 0; j < 4; ++j) {
                                        x[8 * q + 2 * j] += __uint_as_float(w[j] << 16);
                                        x[8 * q + 2 * j + 1] += __uint_as_float(w[j] & 0xFFFF0000u);
                                    }
                                }
                            }
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float* f = x + 8 * q;
                            *reinterpret_cast<uint4*>(box + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) =
                                make_uint4(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]),
                                           bf16x2(f[4], f[5]), bf16x2(f[6], f[7]));
                        }
                    }
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        ptx::tma_store_2d(&p.out_map[part], box_u32, nn, y0);
                        ptx::bulk_commit_group();
                    }
                }
            }
        }
        if (lane == 0) ptx::bulk_wait_group<0>();
        __syncwarp();
    }

    ptx::tc_fence_before();
    __syncwarp();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        ptx::tmem_dealloc_pair(tmem, F_TMEM_COLS);
    }
}

// CTA pairs that fit on the current device at once (queried once per device and variant).
template <int OUT>
cudaError_t max_clusters(int& out) {
    constexpr int kDevices = 64;
    static int known[kDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    int n = __atomic_load_n(&known[dev], __ATOMIC_ACQUIRE);
    if (n == 0) {
        auto kern = fp8_gemm_kernel<OUT>;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<OUT>::kSmem);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2, 1, 1);
        cfg.blockDim = dim3(F_THREADS, 1, 1);
        cfg.dynamicSmemBytes = Cfg<OUT>::kSmem;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 2;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorInvalidConfiguration;
        __atomic_store_n(&known[dev], n, __ATOMIC_RELEASE);
    }
    out = n;
    return cudaSuccess;
}

template <int OUT>
cudaError_t launch(const Fp8GemmParams& p, cudaStream_t st) {
    int pairs = 0;
    cudaError_t e = max_clusters<OUT>(pairs);
    if (e != cudaSuccess) return e;
    const int clusters = p.total_tiles < pairs ? p.total_tiles : pairs;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * clusters, 1, 1);
    cfg.blockDim = dim3(F_THREADS, 1, 1);
    cfg.dynamicSmemBytes = Cfg<OUT>::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fp8_gemm_kernel<OUT>, p);
}

}  // namespace

cudaError_t launch_fp8_gemm(const Fp8GemmParams& p, int out, cudaStream_t st) {
    return out == F8_F32_VECTOR ? launch<F8_F32_VECTOR>(p, st) : launch<F8_BF16_BLOCK>(p, st);
}

}  // namespace tpmlp
