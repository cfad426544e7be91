// fp4_small.cu -- the 4-bit product for few rows of A (tokens): decoding, where every
// weight is read once for a handful of tokens.
//
// What bounds it: the weights' bytes.  As in the 8-bit form the tensor cores' 128 rows are
// 128 features of the weight, their columns the tokens (16 to 256 of them), and the K axis
// is cut over the CTAs of a cluster, whose parts meet in distributed shared memory: each
// leaves its sums in its own, and adds a share of the tokens over all of them, in the order
// of the CTAs.
//
// Measured, weights not in L2: 1 token, 12288 -> 36864 features 40 us (6.4 TB/s of weights and
// scales); 48 tokens, 12288 -> 12288 21 us; 1 token, 4096 -> 12288 8 us, of which 4 are the
// weights' and the rest a launch, the first stage's way and the join of the sums.
//
// CTA layout (256 threads):
//   warp 0       producer: 128 features and the tile's tokens for each 256 of K, and
//                their scales
//   warp 1       owns the tensor memory, copies the scales into it, issues the MMAs
//   warp 2       adds up column sums
//   warps 4..7   quantise the tokens where they come in bf16; the output
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fp4_cvt.cuh"
#include "fp4_gemm.cuh"
#include "fp4_mma.cuh"

namespace tpmlp {
namespace {

using namespace f8;

constexpr int S_THREADS = 256;
constexpr int S_WARPS = 4;       // of the output, and of quantising
constexpr int S_MAX_SPLIT = 8;   // the portable cluster size

// Up to 64 tokens two CTAs take an SM, at 256 one.  At 128 either: one with a ring as
// deep as two have together, or two.
template <int FMT, int TN, int PER_SM>
struct Small {
    static constexpr int kScales = fp4_scale_step(FMT);  // of 128 rows for a stage
    static constexpr int kBlocks = kScales / 512;        // in blocks of 512 bytes
    static constexpr int kTiles = TN > 128 ? 2 : 1;      // times 128 tokens with scales
    static constexpr int kStageBytes = F4_BOX_BYTES + TN * 128 + (1 + kTiles) * kScales;
    static constexpr int kTail = 256;                    // barriers
    static constexpr int kFit = (PER_SM == 2 ? 114 * 1024 - 1024 : 227 * 1024) - 1024 - kTail;
    static constexpr int kStages = kFit / kStageBytes < 6 ? kFit / kStageBytes : 6;
    static constexpr int kSmem = 1024 + kStages * kStageBytes + kTail;
    static constexpr int kSums = TN < 32 ? 32 : TN;      // columns of sums
    static constexpr int kSlot = 4 * kBlocks * (1 + kTiles);  // of scales: A's, then B's
    static constexpr int kTmemCols = kSums + kStages * kSlot <= 128   ? 128
                                     : kSums + kStages * kSlot <= 256 ? 256
                                                                      : 512;
    static constexpr int kPerSm = PER_SM;
    static constexpr int kSharing = TN <= 16 ? 1 : 2;    // warps that quantise a stage
    static_assert(kStages >= 3 && kStageBytes % 1024 == 0, "stages");
    static_assert(kSums + kStages * kSlot <= 512 / kPerSm, "tensor memory");
    static_assert(TN * 128 * 4 <= kStages * kStageBytes, "the sums fit where the operands were");
    static_assert(kPerSm * (kSmem + 1024) <= 228 * 1024, "shared memory of an SM");
};

// 1-D copy of `bytes` (a multiple of 16) into this CTA's shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
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

template <int FMT, int TN, int PER_SM, bool QUANT>
__global__ void __launch_bounds__(S_THREADS, Small<FMT, TN, PER_SM>::kPerSm)
    fp4_small_kernel(const __grid_constant__ Fp4GemmParams p, int splits) {
    using C = Small<FMT, TN, PER_SM>;
    constexpr int NST = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t bar0 = base + NST * C::kStageBytes;
    uint8_t* bar_area = gbase + NST * C::kStageBytes;
    const uint32_t bar_full = bar0;            // [NST] operands and scales
    const uint32_t bar_empty = bar0 + 8 * NST; // [NST]
    const uint32_t bar_done = bar0 + 16 * NST; // all MMAs
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_area + 16 * NST + 8);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bar_area + 16 * NST + 12);
    // stages copied, and those with each warp's values (a role that has given up says so)
    volatile int* copied = abort_flag + 1;
    volatile int* quantised = abort_flag + 2;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(blockIdx.x % splits);
    const int tile = static_cast<int>(blockIdx.x / splits);
    const int ntiles = (p.N + 127) / 128;
    const int g = tile / ntiles, f0 = (tile - g * ntiles) * 128;  // group, first feature
    const int t0 = static_cast<int>(blockIdx.y) * TN;             // first token

    if (threadIdx.x == 0) {
        for (int s = 0; s < NST; ++s) {
            ptx::mbar_init(bar_full + 8 * s, QUANT ? 1 + C::kSharing : 1);
            ptx::mbar_init(bar_empty + 8 * s, 1);
        }
        ptx::mbar_init(bar_done, 1);
        *abort_flag = 0;
        for (int w = 0; w < S_WARPS; ++w) quantised[w] = 0x7FFFFFFF;
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

    const int kblocks = (p.K + F4_BK - 1) / F4_BK;
    const int nk = kblocks * p.ksegs;
    const int first = static_cast<int>(static_cast<long long>(rank) * nk / splits);
    const int last = static_cast<int>(static_cast<long long>(rank + 1) * nk / splits);

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int s = first / kblocks, kb = first - s * kblocks, fills = 0;
            const int stop = p.stall >= 0 && rank == splits - 1 ? min(last, first + p.stall) : last;
            // B's part of stage `stage`; scales of 128 rows lie next to each other along K
            constexpr uint32_t X_BYTES = QUANT ? TN * 128 + C::kScales : 0;  // written here, not copied
            // (of long K their offsets pass 2^31)
            const long long along = static_cast<long long>(kblocks) * C::kScales;
            const long long along_a = p.a_seg ? along * p.ksegs : along;
            auto load_b = [&](int st, int seg, int block) {
                const uint32_t sw = base + st * C::kStageBytes, full = bar_full + 8 * st;
                const int wi = f4::pick(p.b_part, g, seg);
                ptx::mbar_arrive_expect_tx(full, C::kStageBytes - X_BYTES);
                // (a byte holds two of K)
                ptx::tma_load_3d(sw, p.b_map + (p.b_z ? 0 : wi), block * 128, f0, p.b_z ? wi : 0, full);
                bulk_load(sw + F4_BOX_BYTES + TN * 128,
                          p.sb[wi] + (f0 >> 7) * along + static_cast<long long>(block) * C::kScales, C::kScales, full);
            };
            // what the ring takes of B, if that may be read already
            int ahead = 0;
            for (int es = s, eb = kb; p.early && ahead < NST && first + ahead < stop; ++ahead) {
                load_b(ahead, es, eb);
                if (++eb == kblocks) {
                    eb = 0;
                    ++es;
                }
            }
            ptx::griddep_wait();
            for (int k = first; k < stop; ++k) {
                if (k - first >= ahead) {
                    if (!wait(bar_empty + 8 * stage, phase ^ 1u, abort_flag, p.timeout_ns, p.err,
                              ERR_PRODUCER))
                        break;
                    load_b(stage, s, kb);
                }
                if constexpr (!QUANT) {
                    const uint32_t sw = base + stage * C::kStageBytes, full = bar_full + 8 * stage;
                    const int xi = f4::pick(p.a_part, g, s);
                    const int ka = s * p.a_seg + kb;
                    ptx::tma_load_3d(sw + F4_BOX_BYTES, p.a_map + (p.a_z ? 0 : xi), ka * 128, t0, p.a_z ? xi : 0, full);
#pragma unroll
                    for (int i = 0; i < C::kTiles; ++i) {
                        // (behind the last token any: nobody reads those sums)
                        const int at = t0 + 128 * i < p.M ? (t0 >> 7) + i : 0;
                        bulk_load(sw + F4_BOX_BYTES + TN * 128 + (1 + i) * C::kScales,
                                  p.sa[xi] + at * along_a + static_cast<long long>(ka) * C::kScales, C::kScales, full);
                    }
                }
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
        const uint32_t id = f4::idesc<FMT>(128, TN);
        const uint64_t da = operand_desc(base, 0, 0), db = operand_desc(base + F4_BOX_BYTES, 0, 0);
        const uint64_t ds = f4::scales_desc(base + F4_BOX_BYTES + TN * 128);
        int stage = 0;
        uint32_t phase = 0;
        for (int k = first; k < last; ++k) {
            const bool ok = __all_sync(0xffffffffu, wait(bar_full + 8 * stage, phase, abort_flag,
                                                         p.timeout_ns, p.err, ERR_MMA));
            if (!ok) break;
            ptx::tc_fence_after();
            const uint32_t step = stage * (C::kStageBytes >> 4);
            const uint32_t sfa = tmem + C::kSums + stage * C::kSlot, sfb = sfa + 4 * C::kBlocks;
            if (elect_one()) {
#pragma unroll
                for (uint32_t j = 0; j < C::kBlocks; ++j) {
                    const uint64_t d = ds + step + j * (512 >> 4);
                    f4::copy_scales<1>(sfa + 4 * j, d);
#pragma unroll
                    for (uint32_t i = 0; i < C::kTiles; ++i)
                        f4::copy_scales<1>(sfb + 4 * (C::kTiles * j + i), d + (1 + i) * (C::kScales >> 4));
                }
#pragma unroll
                for (uint32_t i = 0; i < 4; ++i) {
                    const uint32_t j = FMT == FP4_NV ? i : i >> 1;
                    f4::mma<FMT, 1>(tmem, da + step + i * (32 >> 4), db + step + i * (32 >> 4),
                                    FMT == FP4_MX && (i & 1) ? id | f4::UPPER_SCALES : id, sfa + 4 * j,
                                    sfb + 4 * C::kTiles * j, (k > first || i > 0) ? 1u : 0u);
                }
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
    } else if (warp == 2) {
        // what came before this grid has ended when the next starts
        ptx::griddep_wait();
        ptx::griddep_launch_dependents();
        if (p.sums)
            f4::column_sums(p, blockIdx.y * gridDim.x + blockIdx.x, gridDim.x * gridDim.y, lane);
    } else if (warp >= 4) {
        const int q = warp & 3;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
        ptx::griddep_wait();
        if constexpr (QUANT) {
            // A: a warp takes 16 rows of every stage that is its own, each lane 32 of every fourth
            // of them, 16 bytes of a 128-byte swizzle row.  What lies behind the last token is
            // left: nobody reads those sums.  (With all four warps at each stage a stage took
            // 1.2 us from one wait to the next: 12288 -> 36864 features, 48 stages a CTA, 8 tokens
            // 63 us, now 42.)
            constexpr int PER = FMT == FP4_NV ? 2 : 1;  // groups of 32
            constexpr int N = 4;                        // rows of a lane
            constexpr int SHARE = C::kSharing, TURN = S_WARPS / SHARE;
            const int row0 = (q % SHARE) * 16 + (lane >> 3), run = lane & 7;
            float inv_g = 0.0f;
            if constexpr (FMT == FP4_NV) inv_g = q4::inverse_of(p.ga);
            auto fetch = [&](int stage_k, uint4 (&v)[N][4]) {
                const int s = stage_k / kblocks, kb = stage_k - s * kblocks;
                const int k = kb * F4_BK + run * 32;
                const uint16_t* src = static_cast<const uint16_t*>(p.x[f4::pick(p.a_part, g, s)]) + k;
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const int row = row0 + 4 * n;
                    const bool in = row < p.M && k < p.K;
                    const uint4* at = reinterpret_cast<const uint4*>(src + static_cast<long long>(row) * p.K);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[n][j] = in ? __ldg(at + j) : make_uint4(0, 0, 0, 0);
                }
            };
            uint4 next[N][4];
            int k = first + q / SHARE;
            if (k < last) fetch(k, next);
            for (; k < last; k += TURN) {
                uint4 o[N];
                uint32_t byte[N][PER];
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const uint4* v = next[n];
                    uint32_t w4[4];
#pragma unroll
                    for (int h = 0; h < PER; ++h) {
                        uint32_t m = q4::larger(q4::largest(v[2 * h]), q4::largest(v[2 * h + 1]));
                        if constexpr (PER == 1)
                            m = q4::larger(m, q4::larger(q4::largest(v[2]), q4::largest(v[3])));
                        const q4::Scale4 sc = q4::scale_of<FMT>(m & 0x7FFFu, inv_g);
                        byte[n][h] = sc.byte;
#pragma unroll
                        for (int j = h * (4 / PER); j < (h + 1) * (4 / PER); ++j) {
                            const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
                            float2 f[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                f[e] = q4::scaled<FMT>(make_float2(q8::lo_f(w[e]), q8::hi_f(w[e])), sc.inv);
                            w4[j] = sc.inv > 0.0f ? q4::cvt8(f[0], f[1], f[2], f[3]) : 0u;
                        }
                    }
                    o[n] = make_uint4(w4[0], w4[1], w4[2], w4[3]);
                    if ((q % SHARE) * 16 + 4 * (n + 1) >= p.M) break;  // (the rest behind the last token)
                }
                if (k + TURN < last) fetch(k + TURN, next);
                const int stage = (k - first) % NST;
                const uint32_t phase = static_cast<uint32_t>((k - first) / NST) & 1u;
                const bool ok = __all_sync(0xffffffffu, wait(bar_empty + 8 * stage, phase ^ 1u, abort_flag,
                                                             p.timeout_ns, p.err, ERR_PRODUCER));
                if (!ok) {
                    if (lane == 0) quantised[q] = k - first;
                    break;
                }
                uint8_t* to = gbase + stage * C::kStageBytes + F4_BOX_BYTES;
                uint8_t* scales = to + TN * 128 + C::kScales;
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const int row = row0 + 4 * n;
                    if (row >= p.M) break;
                    *reinterpret_cast<uint4*>(to + row * 128 + ((run ^ (row & 7)) << 4)) = o[n];
#pragma unroll
                    for (int h = 0; h < PER; ++h) {
                        const int j = run * PER + h;  // the stage's group
                        scales[row * 16 + (j >> 2) * 512 + (j & 3)] = static_cast<uint8_t>(byte[n][h]);
                    }
                }
                // for the tensor cores, which read shared memory another way
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar_full + 8 * stage);
            }
        }
        // this CTA's sums, feature by feature of each token, where the operands were
        // (not of a CTA that has given up: copies and MMAs may still be under way there)
        if (__all_sync(0xffffffffu, wait(bar_done, 0, abort_flag, p.timeout_ns, p.err, ERR_EPILOGUE))) {
            ptx::tc_fence_after();
            float* sums = reinterpret_cast<float*>(gbase) + q * 32 + lane;  // a feature, token by token
            constexpr int AT = TN < 64 ? TN : TN > 128 ? 16 : 64;  // columns on the way at a time
#pragma unroll
            for (int c = 0; c < TN; c += AT) {
                float x[AT];
#pragma unroll
                for (int i = 0; i < AT; i += 16) load_cols16(lanes + c + i, x + i);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < AT; ++i) {
                    asm volatile("" : "+f"(x[i]));  // used after the wait
                    sums[(c + i) * 128] = x[i];
                }
            }
            ptx::tc_fence_before();
        }
    }

    // every CTA's sums are in place
    ptx::griddep_wait();
    __syncwarp();
    ptx::cluster_sync();
    if (threadIdx.x == 0 && *abort_flag) {
        // What this CTA has under way ends before it does.  A stage counts the quantising warps
        // too: those that gave up before they came to it are stood in for.
        const int n = *copied;
        for (int k = max(0, n - NST); k < n; ++k) {
            const uint32_t full = bar_full + 8 * (k % NST);
            for (int w = 0; QUANT && w < S_WARPS; ++w)
                if (w / C::kSharing == k % (S_WARPS / C::kSharing) && quantised[w] <= k) arrive_relaxed(full);
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
        f4::Alpha alpha = {1.0f, 1.0f};
        if constexpr (FMT == FP4_NV) alpha = f4::alpha_of(p.ga, p.gb);
        const int here = min(TN, p.M - t0);
        for (int t = rank + warp * splits; t < here; t += (S_THREADS / 32) * splits) {
            const uint32_t at = base + (t * 128 + lane * 4) * 4;
            // (all parts on the way before the first is added)
            float4 x[S_MAX_SPLIT];
#pragma unroll
            for (int r = 0; r < S_MAX_SPLIT; ++r)
                if (r < splits) x[r] = load_cluster(ptx::mapa_shared(at, static_cast<uint32_t>(r)));
            float4 s = x[0];
#pragma unroll
            for (int r = 1; r < S_MAX_SPLIT; ++r) {
                if (r < splits) {
                    s.x += x[r].x;
                    s.y += x[r].y;
                    s.z += x[r].z;
                    s.w += x[r].w;
                }
            }
            if constexpr (FMT == FP4_NV) {
                s.x = s.x * alpha.first * alpha.second;
                s.y = s.y * alpha.first * alpha.second;
                s.z = s.z * alpha.first * alpha.second;
                s.w = s.w * alpha.first * alpha.second;
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
template <int FMT, int TN, int PER_SM, bool QUANT>
void configure(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, int splits) {
    cfg.gridDim = dim3(static_cast<unsigned>(splits), 1, 1);
    cfg.blockDim = dim3(S_THREADS, 1, 1);
    cfg.dynamicSmemBytes = Small<FMT, TN, PER_SM>::kSmem;
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
template <int FMT, int TN, int PER_SM, bool QUANT>
__global__ void __launch_bounds__(S_THREADS, Small<FMT, TN, PER_SM>::kPerSm) fp4_small_stand_in() {}

// Clusters of each size that a device runs at once (a cluster lies in one group of SMs:
// with two CTAs on an SM 97 of 3, 74 of 4 and 36 of 8 on 152 SMs).
template <int FMT, int TN, int PER_SM, bool QUANT>
cudaError_t resident(const int*& clusters) {
    constexpr int kDevices = 64;
    static int known[kDevices][S_MAX_SPLIT + 1] = {};
    static int ready[kDevices] = {};  // asked once a device, with the kernel's attribute
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    if (!__atomic_load_n(&ready[dev], __ATOMIC_ACQUIRE)) {
        e = cudaFuncSetAttribute(fp4_small_kernel<FMT, TN, PER_SM, QUANT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Small<FMT, TN, PER_SM>::kSmem);
        if (e != cudaSuccess) return e;
        e = cudaFuncSetAttribute(fp4_small_stand_in<FMT, TN, PER_SM, QUANT>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, Small<FMT, TN, PER_SM>::kSmem);
        if (e != cudaSuccess) return e;
        for (int c = 1; c <= S_MAX_SPLIT; ++c) {
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute attr[2];
            configure<FMT, TN, PER_SM, QUANT>(cfg, attr, c);
            cfg.numAttrs = 1;
            int n = 0;
            e = cudaOccupancyMaxActiveClusters(&n, fp4_small_stand_in<FMT, TN, PER_SM, QUANT>, &cfg);
            if (e != cudaSuccess) return e;
            __atomic_store_n(&known[dev][c], n, __ATOMIC_RELAXED);
        }
        __atomic_store_n(&ready[dev], 1, __ATOMIC_RELEASE);
    }
    clusters = known[dev];
    return cudaSuccess;
}

template <int FMT, int TN, int PER_SM, bool QUANT>
cudaError_t launch(const Fp4GemmParams& p, cudaStream_t st) {
    const int* clusters = nullptr;
    const cudaError_t e = resident<FMT, TN, PER_SM, QUANT>(clusters);
    if (e != cudaSuccess) return e;
    const long long tiles = static_cast<long long>((p.N + 127) / 128) * p.groups;
    const long long rows = (p.M + TN - 1) / TN;
    const long long nk = static_cast<long long>((p.K + F4_BK - 1) / F4_BK) * p.ksegs;
    // The widest split whose CTAs all run at once and still have a K block each.  Whole calls
    // of mx (nv up to 4 us more): 128 tokens, 12288 -> 4608 features (36 tiles) 4 parts 14.2 us,
    // 3 or 5 parts 14.9 or 21.0; 1 token, the same, 8 parts 8.4, 4 parts 7.7, 2 parts 10.2; 48
    // tokens, 12288 -> 12288 in eight row shards (96 tiles) 3 parts 20.3, 2 or 4 parts 19.3 or
    // 24.8; 4096 -> 4096 (32 tiles) 8 parts 8.4, 4 parts 7.4.  (More parts than run at once cost up
    // to half; fewer than this rule's would save up to 12 % of the shortest calls.)
    int splits = static_cast<int>(nk < S_MAX_SPLIT ? nk : S_MAX_SPLIT);
    while (splits > 1 && tiles * rows > clusters[splits]) --splits;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    configure<FMT, TN, PER_SM, QUANT>(cfg, attr, splits);
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * splits), static_cast<unsigned>(rows), 1);
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, fp4_small_kernel<FMT, TN, PER_SM, QUANT>, p, splits);
}

}  // namespace

cudaError_t fp4_small_rows(int M, int N, int K, int groups, int ksegs, int fmt, int& rows) {
    rows = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
    if (M <= 64) return cudaSuccess;
    const int* clusters = nullptr;  // (of one CTA on an SM)
    const cudaError_t e = fmt == FP4_NV ? resident<FP4_NV, 256, 1, false>(clusters) : resident<FP4_MX, 256, 1, false>(clusters);
    if (e != cudaSuccess) return e;
    const long long tiles = static_cast<long long>((N + 127) / 128) * groups;
    const long long nk = static_cast<long long>((K + F4_BK - 1) / F4_BK) * ksegs;
    if (M <= 128) {
        // Pairs on 256 x 256 tiles where K is short and cannot be cut in two, but the tiles are
        // one for each pair (us here, on pairs: 128 tokens, 4096 -> 12288 features 15.0, 13.4;
        // 6144 -> 12288 16.6, 16.1; but 2080 -> 8224 10.4, 11.5, 4096 -> 24576 20.7, 24.8,
        // 12288 -> 36864 51.1, 53.2).
        if (tiles > clusters[2] && tiles <= 2 * clusters[2] && nk <= 24) rows = 0;
        return cudaSuccess;
    }
    // Pairs are faster unless so few tiles that K can be cut in four here, and above 256
    // tokens unless K is long too (us here, on pairs: 333 tokens, 1056 -> 2080 features 11.8, 9.9;
    // 4096 -> 1024 11.5, 12.6; 512 tokens, 8192 -> 2048 15.5, 18.3).
    rows = tiles * ((M + 255LL) / 256) <= clusters[4] && (M <= 256 || nk >= 16) ? 256 : 0;
    // Up to 256 tokens tiles of 128 read weights twice, but from L2, and have half the sums to
    // hand on: faster where K is cut in as many or is short (256 tokens, by 128 and by 256:
    // 1024 -> 1024 8.0, 10.1; 8192 -> 2048 12.6, 13.9; 4096 -> 4096 12.0, 12.9; but 12288 -> 4096
    // 19.4, 17.9).
    if (rows == 256 && M <= 256 && (2 * tiles <= clusters[4] || nk <= 16)) rows = 128;
    return cudaSuccess;
}

cudaError_t fp4_small_quantises(int M, int N, int K, int groups, int ksegs, bool& quantises) {
    // Every CTA quantises what it takes of the tokens.  Up to 16 that is less than a launch; up
    // to 32 where a CTA has four stages or fewer (24 tokens, 4096 -> 4096 features 6.9 us, 8.3
    // with a launch ahead; 32 tokens, 12288 -> 12288, sixteen stages, 26.7 and 23.4).
    quantises = M <= 16;
    if (M <= 16 || M > FP4_QUANT_ROWS) return cudaSuccess;
    const int* clusters = nullptr;
    const cudaError_t e = resident<FP4_MX, 32, 2, true>(clusters);
    if (e != cudaSuccess) return e;
    const long long tiles = static_cast<long long>((N + 127) / 128) * groups;
    const long long nk = static_cast<long long>((K + F4_BK - 1) / F4_BK) * ksegs;
    quantises = tiles * nk <= 4LL * clusters[1];
    return cudaSuccess;
}

template <int FMT>
static cudaError_t launch_rows(const Fp4GemmParams& p, int rows, bool quantise, cudaStream_t st) {
    if (quantise && p.M > FP4_QUANT_ROWS) return cudaErrorInvalidValue;
    switch (rows) {
        case 16: return quantise ? launch<FMT, 16, 2, true>(p, st) : launch<FMT, 16, 2, false>(p, st);
        case 32: return quantise ? launch<FMT, 32, 2, true>(p, st) : launch<FMT, 32, 2, false>(p, st);
        case 64: return launch<FMT, 64, 2, false>(p, st);
        case 128: {
            const int* clusters = nullptr;
            const cudaError_t e = resident<FMT, 128, 1, false>(clusters);
            if (e != cudaSuccess) return e;
            const long long tiles =
                static_cast<long long>((p.N + 127) / 128) * p.groups * ((p.M + 127LL) / 128);
            return tiles <= clusters[2] ? launch<FMT, 128, 1, false>(p, st) : launch<FMT, 128, 2, false>(p, st);
        }
        case 256: return launch<FMT, 256, 1, false>(p, st);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_fp4_small(const Fp4GemmParams& p, int fmt, int rows, bool quantise, cudaStream_t st) {
    return fmt == FP4_NV ? launch_rows<FP4_NV>(p, rows, quantise, st)
                         : launch_rows<FP4_MX>(p, rows, quantise, st);
}

}  // namespace tpmlp
