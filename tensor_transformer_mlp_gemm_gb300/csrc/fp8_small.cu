// fp8_small.cu -- the 8-bit product with scales per block of 128 for few rows of A
// (tokens): decoding, where every weight is read once for a handful of tokens.
//
// What bounds it: the weights' bytes.  256 x 256 tiles leave most SMs without work
// then (a 12288-wide layer has 48), so here the tensor cores' 128 rows are 128
// features of the weight and their columns are the tokens (16 to 256 of them), and
// the K axis is cut over the CTAs of a cluster: two CTAs for an SM up to 64 tokens,
// with about 100 KB of weights on the way each.  The parts meet in distributed
// shared memory: each CTA leaves its sums in its own, and adds a share of the
// tokens over all of them, in the order of the CTAs.
// Measured with cold caches, launch included: one token, 12288 -> 12288 features in 39 us
// (151 MB; 22 us at the copy rate), 4096 -> 12288 in 18 us; 48 tokens 39 and 20 us.  Without
// the launch, by the profiler: 48 tokens, 12288 -> 12288 29 us; one token, 4096 -> 12288
// 13.5 us.  Back to back, where 50 MB of weights stay in L2: 29 and 8.9 us.
//
// CTA layout (256 threads):
//   warp 0       TMA producer: 128 features and the tile's tokens for each K block
//   warp 1       owns the tensor memory, issues the MMAs
//   warps 4..7   the scales of each K block into tensor memory (each its quarter of
//                the lanes), then the output
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fp8_gemm.cuh"
#include "fp8_mma.cuh"

namespace tpmlp {
namespace {

using namespace f8;

constexpr int S_THREADS = 256;
constexpr int S_WARPS = 4;       // scale and output warps
constexpr int S_MAX_SPLIT = 8;   // the portable cluster size
constexpr int S_AHEAD = 4;       // K blocks whose scales are under way

// Up to 64 tokens two CTAs take an SM, at 256 one.  At 128 either: one with a ring as
// deep as two have together, or two.  One is faster while K can be cut in two with it
// (12288 -> 4608 features 22 us, two 25), two for wider layers (12288 -> 12288 43 us,
// one 53).
template <int TN, int PER_SM>
struct Small {
    static constexpr int kStages = TN == 16 ? 6 : TN == 32 ? 5 : TN == 64 ? 4 : TN == 256 ? 4 : PER_SM == 2 ? 3 : 6;
    static constexpr int kStageBytes = F8_BOX_BYTES + TN * 128;
    static constexpr int kSmem = 1024 + kStages * kStageBytes + 256;
    static constexpr int kSums = TN < 32 ? 32 : TN;      // columns of sums
    static constexpr int kScaleB = 4;                    // a slot: 4 columns for A, then B's
    static constexpr int kColsB = TN < 32 ? 1 : TN / 32;
    static constexpr int kSlot = kColsB <= 4 ? 8 : 16;   // columns of a slot
    static constexpr int kTmemCols = kSums + kStages * kSlot <= 128   ? 128
                                     : kSums + kStages * kSlot <= 256 ? 256
                                                                      : 512;
    static constexpr int kPerSm = PER_SM;
    static_assert(kSums + kStages * kSlot <= 512 / kPerSm, "tensor memory");
    static_assert(TN * 128 * 4 <= kStages * kStageBytes, "the sums fit where the operands were");
    static_assert(kPerSm * (kSmem + 1024) <= 228 * 1024, "shared memory of an SM");
};

__device__ __forceinline__ int pick(int part, int g, int s) {
    return part == F8_GROUP ? g : part == F8_KSEG ? s : 0;
}

__device__ __forceinline__ float4 load_cluster(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

template <int TN, int PER_SM>
__global__ void __launch_bounds__(S_THREADS, Small<TN, PER_SM>::kPerSm)
    fp8_small_kernel(const __grid_constant__ Fp8GemmParams p, int splits) {
    using C = Small<TN, PER_SM>;
    constexpr int NST = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t bar0 = base + NST * C::kStageBytes;
    uint8_t* bar_area = gbase + NST * C::kStageBytes;
    const uint32_t bar_full = bar0;            // [NST] operands (1 + bytes) and scales (4 warps)
    const uint32_t bar_empty = bar0 + 8 * NST; // [NST]
    const uint32_t bar_done = bar0 + 16 * NST; // all MMAs
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_area + 16 * NST + 8);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bar_area + 16 * NST + 12);
    // K blocks copied, and those with each warp's scales (a role that has given up says so)
    volatile int* copied = abort_flag + 1;
    volatile int* scaled = abort_flag + 2;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(blockIdx.x % splits);
    const int tile = static_cast<int>(blockIdx.x / splits);
    const int ntiles = (p.N + 127) / 128;
    const int g = tile / ntiles, f0 = (tile - g * ntiles) * 128;  // group, first feature
    const int t0 = static_cast<int>(blockIdx.y) * TN;             // first token

    if (threadIdx.x == 0) {
        for (int s = 0; s < NST; ++s) {
            ptx::mbar_init(bar_full + 8 * s, 1 + S_WARPS);
            ptx::mbar_init(bar_empty + 8 * s, 1);
        }
        ptx::mbar_init(bar_done, 1);
        *abort_flag = 0;
        scaled[0] = scaled[1] = scaled[2] = scaled[3] = 0x7FFFFFFF;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), C::kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();

    const int kblocks = (p.K + F8_BK - 1) / F8_BK;
    const int nk = kblocks * p.ksegs;
    const int first = static_cast<int>(static_cast<long long>(rank) * nk / splits);
    const int last = static_cast<int>(static_cast<long long>(rank + 1) * nk / splits);

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int s = first / kblocks, kb = first - s * kblocks, fills = 0;
            const int stop = p.stall >= 0 && rank == splits - 1 ? min(last, first + p.stall) : last;
            for (int k = first; k < stop; ++k) {
                if (!wait(bar_empty + 8 * stage, phase ^ 1u, abort_flag, p.timeout_ns, p.err,
                          ERR_PRODUCER))
                    break;
                const uint32_t sw = base + stage * C::kStageBytes, full = bar_full + 8 * stage;
                const int k0 = kb * F8_BK;
                ptx::mbar_arrive_expect_tx(full, C::kStageBytes);
                ptx::tma_load_2d(sw, p.b_map + pick(p.b_part, g, s), p.b_mn ? f0 : k0,
                                 p.b_mn ? k0 : f0, full);
                ptx::tma_load_2d(sw + F8_BOX_BYTES, p.a_map + pick(p.a_part, g, s), k0, t0, full);
                ++fills;
                if (++kb == kblocks) {
                    kb = 0;
                    ++s;
                }
                if (++stage == NST) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            *copied = fills;
        }
        __syncwarp();
    } else if (warp == 1) {
        const uint32_t id = idesc(128, TN, p.b_mn, 0) | p.ab_format;
        const uint64_t da = operand_desc(base, 0, p.b_mn), db = operand_desc(base + F8_BOX_BYTES, 0, 0);
        const uint32_t ka = (p.b_mn ? 4096 : 32) >> 4, kbs = 32 >> 4;
        int stage = 0;
        uint32_t phase = 0;
        for (int k = first; k < last; ++k) {
            const bool ok = __all_sync(0xffffffffu, wait(bar_full + 8 * stage, phase, abort_flag,
                                                         p.timeout_ns, p.err, ERR_MMA));
            if (!ok) break;
            ptx::tc_fence_after();
            const uint32_t step = stage * (C::kStageBytes >> 4);
            const uint32_t sf = tmem + C::kSums + stage * C::kSlot;
            if (elect_one()) {
#pragma unroll
                for (uint32_t i = 0; i < 4; ++i)
                    mma_one(tmem, da + step + i * ka, db + step + i * kbs, id, sf, sf + C::kScaleB,
                            (k > first || i > 0) ? 1u : 0u);
                ptx::mma_commit(bar_empty + 8 * stage);
            }
            __syncwarp();
            if (++stage == NST) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (elect_one()) ptx::mma_commit(bar_done);
        __syncwarp();
    } else if (warp >= 4) {
        const int q = warp & 3;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
        {
            // scales: the weight block's one for all 128 features, the tokens' own
            float v[S_AHEAD][1 + C::kColsB];
            int s = first / kblocks, kb = first - s * kblocks;
            auto fetch = [&](float (&d)[1 + C::kColsB]) {
                const float* sa = p.sa[pick(p.a_part, g, s)] + kb * p.sa_kb;
                d[0] = __ldg(p.sb[pick(p.b_part, g, s)] + kb * p.sb_kb + (f0 >> 7) * p.sb_n);
#pragma unroll
                for (int c = 0; c < C::kColsB; ++c) {
                    const int t = t0 + 32 * c + lane;
                    d[1 + c] = t < p.M ? __ldg(sa + t) : 1.0f;
                }
                if (++kb == kblocks) {
                    kb = 0;
                    ++s;
                }
            };
#pragma unroll
            for (int u = 0; u < S_AHEAD; ++u)
                if (first + u < last) fetch(v[u]);
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int k0 = first; ok && k0 < last; k0 += S_AHEAD) {
#pragma unroll
                for (int u = 0; u < S_AHEAD; ++u) {
                    if (!ok || k0 + u >= last) break;
                    uint32_t w[4], x[C::kColsB];
                    w[0] = w[1] = w[2] = w[3] = scale_word(__float_as_uint(v[u][0]));
#pragma unroll
                    for (int c = 0; c < C::kColsB; ++c) x[c] = scale_word(__float_as_uint(v[u][1 + c]));
                    if (k0 + u + S_AHEAD < last) fetch(v[u]);
                    ok = __all_sync(0xffffffffu, wait(bar_empty + 8 * stage, phase ^ 1u, abort_flag,
                                                      p.timeout_ns, p.err, ERR_PRODUCER));
                    if (!ok) {
                        if (lane == 0) scaled[q] = k0 + u - first;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint32_t t = lanes + C::kSums + stage * C::kSlot;
                    store_cols4(t, w);
                    if constexpr (C::kColsB == 8) {
                        store_cols8(t + C::kScaleB, x);
                    } else if constexpr (C::kColsB == 4) {
                        store_cols4(t + C::kScaleB, x);
                    } else {
#pragma unroll
                        for (int c = 0; c < C::kColsB; ++c) store_col(t + C::kScaleB + c, x[c]);
                    }
                    store_wait();
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_relaxed(bar_full + 8 * stage);
                    if (++stage == NST) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
        // this CTA's sums, feature by feature of each token, where the operands were
        // (not of a CTA that has given up: copies and MMAs may still be under way there)
        if (__all_sync(0xffffffffu, wait(bar_done, 0, abort_flag, p.timeout_ns, p.err, ERR_EPILOGUE))) {
            ptx::tc_fence_after();
            float* sums = reinterpret_cast<float*>(gbase);
            const int f = q * 32 + lane;
#pragma unroll
            for (int c = 0; c < TN / 16; ++c) {
                float x[16];
                load_cols16(lanes + c * 16, x);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    asm volatile("" : "+f"(x[i]));  // used after the wait
                    sums[(c * 16 + i) * 128 + f] = x[i];
                }
            }
            ptx::tc_fence_before();
        }
    }

    // every CTA's sums are in place
    __syncwarp();
    ptx::cluster_sync();
    if (threadIdx.x == 0 && *abort_flag) {
        // What this CTA has under way ends before it does.  A stage counts the scale warps
        // too: those that gave up before they came to it are stood in for.
        const int n = *copied;
        for (int k = max(0, n - NST); k < n; ++k) {
            const uint32_t full = bar_full + 8 * (k % NST);
            for (int w = 0; w < S_WARPS; ++w)
                if (scaled[w] <= k) arrive_relaxed(full);
            drain(full, static_cast<uint32_t>((k / NST) & 1), p.timeout_ns, p.err);
        }
        drain(bar_done, 0, p.timeout_ns, p.err);
    }
    {
        // tokens rank, rank + splits, ... of the tile: a warp a token, four features a lane
        const int col = f0 + lane * 4;
        float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.bias && col < p.N) {
            const uint2 u = __ldg(reinterpret_cast<const uint2*>(
                static_cast<const __nv_bfloat16*>(p.bias) + static_cast<long long>(g) * p.N + col));
            b = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                            __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
        }
        const int here = min(TN, p.M - t0);
        for (int t = rank + warp * splits; t < here; t += (S_THREADS / 32) * splits) {
            const uint32_t at = base + (t * 128 + lane * 4) * 4;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int r = 0; r < splits; ++r) {
                const float4 x = load_cluster(ptx::mapa_shared(at, static_cast<uint32_t>(r)));
                s.x += x.x;
                s.y += x.y;
                s.z += x.z;
                s.w += x.w;
            }
            if (col < p.N) {
                int part = g;
                long long y = t0 + t;
                if (p.chunk_rows > 0) {
                    part = static_cast<int>(y / p.chunk_rows);
                    y -= static_cast<long long>(part) * p.chunk_rows;
                }
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out[part]) + y * p.N + col) =
                    make_uint2(bf16x2(s.x + b.x, s.y + b.y), bf16x2(s.z + b.z, s.w + b.w));
            }
        }
    }
    // nobody leaves while its sums are read
    __syncwarp();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        ptx::tmem_dealloc(tmem, C::kTmemCols);
    }
}

// attr: two of them, the cluster's first
template <int TN, int PER_SM>
void configure(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, int splits) {
    cfg.gridDim = dim3(static_cast<unsigned>(splits), 1, 1);
    cfg.blockDim = dim3(S_THREADS, 1, 1);
    cfg.dynamicSmemBytes = Small<TN, PER_SM>::kSmem;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
}

// Stands in for the kernel where the runtime is asked how many of its clusters run at
// once: of a kernel that allocates tensor memory it counts one CTA on an SM, whatever it
// allocates.  (Never launched; as many registers as two CTAs may have.)
template <int TN, int PER_SM>
__global__ void __launch_bounds__(S_THREADS, Small<TN, PER_SM>::kPerSm) fp8_small_stand_in() {}

// Clusters of each size that a device runs at once (a cluster lies in one group of SMs:
// with two CTAs on an SM 97 of 3, 74 of 4 and 36 of 8 on 152 SMs).
template <int TN, int PER_SM>
cudaError_t resident(const int*& clusters) {
    constexpr int kDevices = 64;
    static int known[kDevices][S_MAX_SPLIT + 1] = {};
    static int ready[kDevices] = {};  // asked once a device, with the kernel's attribute
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    if (!__atomic_load_n(&ready[dev], __ATOMIC_ACQUIRE)) {
        e = cudaFuncSetAttribute(fp8_small_kernel<TN, PER_SM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Small<TN, PER_SM>::kSmem);
        if (e != cudaSuccess) return e;
        e = cudaFuncSetAttribute(fp8_small_stand_in<TN, PER_SM>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, Small<TN, PER_SM>::kSmem);
        if (e != cudaSuccess) return e;
        for (int c = 1; c <= S_MAX_SPLIT; ++c) {
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute attr[2];
            configure<TN, PER_SM>(cfg, attr, c);
            cfg.numAttrs = 1;
            int n = 0;
            e = cudaOccupancyMaxActiveClusters(&n, fp8_small_stand_in<TN, PER_SM>, &cfg);
            if (e != cudaSuccess) return e;
            __atomic_store_n(&known[dev][c], n, __ATOMIC_RELAXED);
        }
        __atomic_store_n(&ready[dev], 1, __ATOMIC_RELEASE);
    }
    clusters = known[dev];
    return cudaSuccess;
}

template <int TN, int PER_SM>
cudaError_t launch(const Fp8GemmParams& p, cudaStream_t st) {
    const int* clusters = nullptr;
    const cudaError_t e = resident<TN, PER_SM>(clusters);
    if (e != cudaSuccess) return e;
    const long long tiles = static_cast<long long>((p.N + 127) / 128) * p.groups;
    const long long rows = (p.M + TN - 1) / TN;
    const long long nk = static_cast<long long>((p.K + F8_BK - 1) / F8_BK) * p.ksegs;
    // The widest split whose CTAs all run at once and still have a K block each.  128
    // tokens, 12288 -> 4608 features (36 tiles): 4 parts 22 us, 3 or 5 parts 25 or 33;
    // 48 tokens, 12288 -> 12288 (96 tiles): 3 parts 39 us, 2 or 4 parts 43 or 47.
    int splits = static_cast<int>(nk < S_MAX_SPLIT ? nk : S_MAX_SPLIT);
    while (splits > 1 && tiles * rows > clusters[splits]) --splits;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    configure<TN, PER_SM>(cfg, attr, splits);
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * splits), static_cast<unsigned>(rows), 1);
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, fp8_small_kernel<TN, PER_SM>, p, splits);
}

}  // namespace

cudaError_t fp8_small_rows(int M, int N, int groups, int& rows) {
    rows = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
    if (M <= 128) return cudaSuccess;
    const int* clusters = nullptr;
    const cudaError_t e = resident<256, 1>(clusters);
    if (e != cudaSuccess) return e;
    // Pairs on 256 x 256 tiles are faster unless so few tiles that K can be cut in four
    // here.  256 tokens: 12288 -> 4096 features (32 tiles) 29 us here and 37 on pairs,
    // 4096 -> 4096 18 and 20; 2064 -> 8240 (65 tiles, cut in two) 22 and 16.
    const long long tiles = static_cast<long long>((N + 127) / 128) * groups;
    rows = tiles * ((M + 255LL) / 256) <= clusters[4] ? 256 : 0;
    return cudaSuccess;
}

cudaError_t launch_fp8_small(const Fp8GemmParams& p, int rows, cudaStream_t st) {
    switch (rows) {
        case 16: return launch<16, 2>(p, st);
        case 32: return launch<32, 2>(p, st);
        case 64: return launch<64, 2>(p, st);
        case 128: {
            const int* clusters = nullptr;
            const cudaError_t e = resident<128, 1>(clusters);
            if (e != cudaSuccess) return e;
            const long long tiles = static_cast<long long>((p.N + 127) / 128) * p.groups;
            return tiles <= clusters[2] ? launch<128, 1>(p, st) : launch<128, 2>(p, st);
        }
        case 256: return launch<256, 1>(p, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace tpmlp
