// fp4_gemm.cu -- the 4-bit product on tcgen05 CTA pairs (see fp4_gemm.cuh for the
// mathematics).
//
// CTA layout (384 threads, persistent over tiles; both CTAs of a pair compute one
// 256 x 256 tile, 128 rows each):
//   warps 0, 2   TMA producers for each 256 of K: of this CTA's 128 rows of A and their
//                scales; of its 128 rows of B and the scales of all 256.  (One thread for
//                all four copies took longer than the MMAs where a segment of K is two
//                stages: forward of 16384 x 4096 x 4096 in eight segments 101 us, now 90.)
//   warp 1       owns the tensor memory; in the even CTA copies the pair's scales into it and
//                issues the MMAs, four K slices of 64 for each stage
//   warp 3       waits for the grid ahead where the product need not; adds up column sums
//   warps 4..11  output: warp w reads lanes 32 (w % 4) .. of the accumulator and columns
//                128 ((w - 4) / 4) .. into registers, frees the accumulator for the next
//                tile's MMAs, and writes from there
// What bounds it: the tensor cores, at 256 x 256 x 256 33.5 MFLOP for 64 KB of operands and 6 to
// 12 KB of scales from L2.  Measured: 2048 tokens, 12288 -> 36864 features nv 254 us, 7.3 PFLOP/s;
// 16384 x 4096 x 4096 mx 86 us, 6.4 PFLOP/s, where a tile has 16 stages: of these the scales'
// copies take 3 (nv 6), and the accumulator's hand-over and the outputs beside the loads 10 each.
//
// Tensor memory: 256 columns of sums, then a slot of scales for each stage (24 columns of mx,
// 48 of nv): a stage that is free has a slot that no MMA reads.
//
// Every wait is bounded as in the 8-bit product: a wait that expires sets a flag that ends
// the roles of both CTAs, copies and MMAs in flight are drained (bounded), tensor memory is
// freed, and the error word tells the host.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fp4_gemm.cuh"
#include "fp4_mma.cuh"

namespace tpmlp {
namespace {

using namespace f8;

constexpr int F_THREADS = 384;
// registers per thread: 128 x 72 + 256 x 216 = 64512, as at launch (384 x 168)
constexpr int F_FEW_REGS = 72, F_MANY_REGS = 216;
constexpr int F_OUT_WARPS = 8;
constexpr int F_TILE = 256;        // pair tile rows and columns
constexpr int F_TMEM_COLS = 512;
constexpr int F_SCALE_COL = 256;   // first column of the scale slots
constexpr int F_BIAS = F_OUT_WARPS * 512;   // each output warp's 128 columns, fp32
constexpr int F_TURN = F_OUT_WARPS * 2048;  // and 32 rows of 64 output bytes
constexpr int F_BARS = 256;

template <int FMT>
struct Shape {
    static constexpr int kStages = 5;
    static constexpr int kScales = fp4_scale_step(FMT);       // of 128 rows for a stage
    static constexpr int kBlocks = kScales / 512;             // in blocks of 512 bytes
    static constexpr int kStageBytes = 2 * F4_BOX_BYTES + 3 * kScales;
    static constexpr int kSlot = 12 * kBlocks;                // columns: A's 4 a block, then B's 8
    static constexpr int kSmem = 1024 + kStages * kStageBytes + F_BIAS + F_TURN + F_BARS;
    static_assert(kStageBytes % 1024 == 0, "swizzled boxes start on 1024 bytes");
    static_assert(kSmem <= 232448, "fits a CTA");
    static_assert(F_SCALE_COL + kStages * kSlot <= F_TMEM_COLS, "tensor memory");
};

__device__ __forceinline__ void decode(const Fp4GemmParams& p, int tile, int& g, int& m0, int& n0) {
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

// How many stages a role that gave up has done (one that did not: all), 64-bit counts in
// shared memory: in the even CTA those copied, A's and B's by it and by the odd one; in both
// those issued.
constexpr int F_COPIED = 0, F_ISSUED = 4, F_COUNTS = 5;

// After a wait has expired and every role has left its loop: what a CTA has under way ends.
// (Not inlined: its values would take registers from the roles.)
template <int FMT>
__device__ __noinline__ void settle(uint32_t bar0, int nk, int tiles, unsigned long long timeout_ns,
                                    unsigned* err) {
    constexpr int NST = Shape<FMT>::kStages;
    constexpr uint32_t STAGE = Shape<FMT>::kStageBytes;
    const uint32_t bar_full = bar0, bar_empty = bar0 + 8 * NST, bar_done = bar0 + 16 * NST;
    const long long* counts =
        static_cast<const long long*>(__cvta_shared_to_generic(bar0 + 16 * NST + 32));
    auto stages = [&](int i) { return min(counts[i], static_cast<long long>(tiles) * nk); };
    if (ptx::cluster_ctarank() == 0) {
        // The copies of both CTAs.  A stage's barrier counts the bytes of all four producers, as
        // its first arms it; what will not come is taken off, or it is armed with what comes.
        long long n = 0;
        for (int i = 0; i < 4; ++i) n = max(n, stages(F_COPIED + i));
        for (long long k = max(0LL, n - NST); k < n; ++k) {
            const uint32_t full = bar_full + 8 * static_cast<uint32_t>(k % NST);
            uint32_t coming = 0;
            for (int i = 0; i < 4; ++i)
                if (k < stages(F_COPIED + i)) coming += F4_BOX_BYTES + (1 + (i & 1)) * Shape<FMT>::kScales;
            if (k >= stages(F_COPIED))
                ptx::mbar_arrive_expect_tx(full, coming);
            else if (coming < 2 * STAGE)
                complete_tx(full, 2 * STAGE - coming);
            drain(full, static_cast<uint32_t>((k / NST) & 1), timeout_ns, err);
        }
    }
    // the MMAs' arrivals on this CTA (the MMAs themselves have ended)
    const long long n = stages(F_ISSUED), whole = n / nk;
    for (long long k = max(0LL, n - NST); k < n; ++k)
        drain(bar_empty + 8 * static_cast<uint32_t>(k % NST), static_cast<uint32_t>((k / NST) & 1),
              timeout_ns, err);
    if (whole > 0) drain(bar_done, static_cast<uint32_t>((whole - 1) & 1), timeout_ns, err);
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

template <int FMT, bool F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(F_THREADS, 1)
    fp4_gemm_kernel(const __grid_constant__ Fp4GemmParams p) {
    using S = Shape<FMT>;
    constexpr int NST = S::kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* after = smem_raw + (base - raw) + NST * S::kStageBytes;
    const uint32_t bar0 = base + NST * S::kStageBytes + F_BIAS + F_TURN;
    uint8_t* bar_area = after + F_BIAS + F_TURN;
    const uint32_t bar_full = bar0;              // [NST] even CTA: both CTAs' operands and scales
    const uint32_t bar_empty = bar0 + 8 * NST;   // [NST] both CTAs
    const uint32_t bar_done = bar0 + 16 * NST;   // both CTAs: the tile is in the accumulator
    const uint32_t bar_free = bar_done + 8;      // even CTA: both CTAs have read it
    const uint32_t bar_drain = bar_free + 8;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_area + 16 * NST + 24);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bar_area + 16 * NST + 28);
    const uint32_t stages_done = bar0 + 16 * NST + 32;
    static_assert(16 * NST + 32 + 8 * F_COUNTS <= F_BARS, "barriers and counts");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(ptx::cluster_ctarank());
    const int cluster = blockIdx.x / 2, nclusters = gridDim.x / 2;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NST; ++s) {
            ptx::mbar_init(bar_full + 8 * s, 1);
            ptx::mbar_init(bar_empty + 8 * s, 1);
        }
        ptx::mbar_init(bar_done, 1);
        ptx::mbar_init(bar_free, 2 * F_OUT_WARPS);
        ptx::mbar_init(bar_drain, 1);
        *abort_flag = 0;
        for (int i = 0; i < F_COUNTS; ++i)
            reinterpret_cast<long long*>(bar_area + 16 * NST + 32)[i] = 0x7FFFFFFFFFFFFFFFLL;
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
    // (B may be there before the grids ahead have ended, or everything.  Warp 3 waits below, once its
    // registers are free: two of the output warps need them, and waited with it.  Backward of 333
    // tokens, 1056 -> 2080 features, in a graph 19.0 us, now 16.1; 256 tokens, 19712 -> 8192 137, now
    // 134; but 200 tokens, 12288 -> 12288 in eight shards 146, now 148.)
    if (warp != 3 && !(p.apart || (p.early && warp == 2))) ptx::griddep_wait();

    const int kblocks = (p.K + F4_BK - 1) / F4_BK;
    const int nk = kblocks * p.ksegs;
    // a wait of this kernel; who gives up takes the other CTA along
    auto wait_for = [&](uint32_t bar, uint32_t parity, unsigned code) {
        if (wait(bar, parity, abort_flag, p.timeout_ns, p.err, code)) return true;
        store_cluster(ptx::mapa_shared(bar0 + 16 * NST + 28, static_cast<uint32_t>(rank ^ 1)), 1);
        return false;
    };

    if (warp < 4) {
        reg_dec<F_FEW_REGS>();
        if ((warp == 0 || warp == 2) && lane == 0) {
            // ---------------- TMA producers ----------------
            const bool of_b = warp == 2;
            const CUtensorMap *maps = of_b ? p.b_map : p.a_map, *smaps = of_b ? p.bs_map : p.as_map;
            const int part = of_b ? p.b_part : p.a_part, has_z = of_b ? p.b_z : p.a_z;
            const int seg = of_b ? 0 : p.a_seg;
            const uint32_t even_full = ptx::mapa_shared(bar_full, 0);
            const uint32_t to = base + (of_b ? F4_BOX_BYTES : 0);
            const uint32_t sto = base + 2 * F4_BOX_BYTES + (of_b ? S::kScales : 0);
            int stage = 0;
            uint32_t phase = 0;
            long long fills = 0;
            bool ok = true;
            for (int tile = cluster; ok && tile < p.total_tiles; tile += nclusters) {
                if (!p.apart && !of_b && tile + nclusters >= p.total_tiles) ptx::griddep_launch_dependents();
                int g, m0, n0;
                decode(p, tile, g, m0, n0);
                const int row = (of_b ? n0 : m0) + rank * 128, srow = (of_b ? n0 : row) >> 7;
                for (int s = 0; ok && s < p.ksegs; ++s) {
                    const int i = f4::pick(part, g, s), at = has_z ? 0 : i, z = i - at;
                    const CUtensorMap *map = maps + at, *smap = smaps + at;
                    for (int kb = s * seg, end = kb + kblocks; kb < end; ++kb) {
                        if ((fills == p.stall && rank == 1) ||
                            !wait_for(bar_empty + 8 * stage, phase ^ 1u, ERR_PRODUCER)) {
                            ok = false;
                            break;
                        }
                        const uint32_t off = stage * S::kStageBytes, full = even_full + 8 * stage;
                        if (rank == 0 && !of_b)  // counts everybody's bytes
                            ptx::mbar_arrive_expect_tx(bar_full + 8 * stage, 2 * S::kStageBytes);
                        // (a byte holds two of K, an element of the scales' maps eight bytes)
                        ptx::tma_load_3d_pair(to + off, map, kb * 128, row, z, full);
                        ptx::tma_load_3d_pair(sto + off, smap, kb * (S::kScales / 8), srow, z, full);
                        ++fills;
                        if (++stage == NST) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                }
            }
            // no release of a stage may arrive after this CTA has left
            for (int i = 0; ok && i < NST; ++i) {
                ok = wait_for(bar_empty + 8 * stage, phase ^ 1u, ERR_PRODUCER);
                if (++stage == NST) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok)
                store_cluster64(ptx::mapa_shared(stages_done + 8 * (F_COPIED + 2 * rank + of_b), 0), fills);
        } else if (warp == 3) {
            ptx::griddep_wait();
            if (p.apart) ptx::griddep_launch_dependents();  // (the grid ahead has ended)
            if (p.sums) f4::column_sums(p, blockIdx.x, gridDim.x, lane);
        } else if (warp == 1 && rank == 0) {
            // ---------------- MMA issuer ----------------
            // The whole warp walks the loop and one lane issues, so the descriptors
            // stay in uniform registers.
            const uint32_t id = f4::idesc<FMT>(F_TILE, F_TILE);
            const uint64_t da = operand_desc(base, 0, 0), db = operand_desc(base + F4_BOX_BYTES, 0, 0);
            const uint64_t ds = f4::scales_desc(base + 2 * F4_BOX_BYTES);
            int stage = 0;
            uint32_t phase = 0, tiles = 0;
            long long issued = 0;
            bool ok = true;
            for (int tile = cluster; ok && tile < p.total_tiles; tile += nclusters, ++tiles) {
                ok = __all_sync(0xffffffffu, wait_for(bar_free, (tiles & 1) ^ 1u, ERR_MMA));
                if (!ok) break;
                for (int kk = 0; kk < nk; ++kk) {
                    ok = __all_sync(0xffffffffu, wait_for(bar_full + 8 * stage, phase, ERR_MMA));
                    if (!ok) break;
                    ptx::tc_fence_after();
                    const uint32_t step = stage * (S::kStageBytes >> 4);
                    const uint32_t sfa = tmem + F_SCALE_COL + stage * S::kSlot, sfb = sfa + 4 * S::kBlocks;
                    if (elect_one()) {
#pragma unroll
                        for (uint32_t j = 0; j < S::kBlocks; ++j) {
                            // block j of A's 128 rows and of B's two times 128
                            const uint64_t d = ds + step + j * (512 >> 4);
                            f4::copy_scales<2>(sfa + 4 * j, d);
                            f4::copy_scales<2>(sfb + 8 * j, d + (S::kScales >> 4));
                            f4::copy_scales<2>(sfb + 8 * j + 4, d + 2 * (S::kScales >> 4));
                        }
#pragma unroll
                        for (uint32_t k = 0; k < 4; ++k) {
                            const uint32_t j = FMT == FP4_NV ? k : k >> 1;
                            f4::mma<FMT, 2>(tmem, da + step + k * (32 >> 4), db + step + k * (32 >> 4),
                                            FMT == FP4_MX && (k & 1) ? id | f4::UPPER_SCALES : id,
                                            sfa + 4 * j, sfb + 8 * j, (kk > 0 || k > 0) ? 1u : 0u);
                        }
                        ptx::mma_commit_pair_multicast(bar_empty + 8 * stage, 0x3);
                        if (kk + 1 == nk) ptx::mma_commit_pair_multicast(bar_done, 0x3);
                    }
                    __syncwarp();
                    ++issued;
                    if (++stage == NST) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (elect_one()) {
                ptx::mma_commit_pair(bar_drain);
                drain(bar_drain, 0, p.timeout_ns, p.err);
                // the last release of the accumulator arrives on this CTA
                if (ok && tiles > 0) wait_for(bar_free, (tiles - 1) & 1, ERR_MMA);
                for (uint32_t r = 0; !ok && r < 2; ++r)
                    store_cluster64(ptx::mapa_shared(stages_done + 8 * F_ISSUED, r), issued);
            }
            __syncwarp();
        }
    } else {
        // ---------------- output ----------------
        reg_inc<F_MANY_REGS>();
        const int quarter = warp & 3;         // the accumulator lanes this warp may read
        const int side = (warp - 4) >> 2;     // its 128 columns
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + side * 128;
        const uint32_t even_free = ptx::mapa_shared(bar_free, 0);
        float* bias_buf = reinterpret_cast<float*>(after) + (warp - 4) * 128;
        uint8_t* turn = after + F_BIAS + (warp - 4) * 2048;
        f4::Alpha alpha = {1.0f, 1.0f};
        if constexpr (FMT == FP4_NV) alpha = f4::alpha_of(p.ga, p.gb);
        uint32_t tiles = 0;
        for (int tile = cluster; tile < p.total_tiles; tile += nclusters, ++tiles) {
            int g, m0, n0;
            decode(p, tile, g, m0, n0);
            const int row0 = m0 + rank * 128 + quarter * 32;
            const int n = n0 + side * 128;
            if constexpr (!F32) {
                // four columns of the bias per lane, under the MMAs
                uint2 u = make_uint2(0, 0);
                if (p.bias && n + lane * 4 < p.N)
                    u = __ldg(reinterpret_cast<const uint2*>(
                        static_cast<const __nv_bfloat16*>(p.bias) + static_cast<long long>(g) * p.N +
                        n + lane * 4));
                __syncwarp();
                *reinterpret_cast<float4*>(bias_buf + lane * 4) =
                    make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                                __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
                __syncwarp();
            }
            bool ok = wait_for(bar_done, tiles & 1, ERR_EPILOGUE);
            ok = __all_sync(0xffffffffu, ok);  // the warp gives up together
            if (!ok) break;
            ptx::tc_fence_after();
            float acc[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) load_cols(lanes + c * 32, acc + c * 32);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 128; ++i) asm volatile("" : "+f"(acc[i]));  // used after the wait
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_relaxed_cluster(even_free);

            // The warp's rows are turned round in shared memory and leave as whole sectors:
            // 64 bytes of all 32 rows at a time, 8 rows to a store instruction, or of fp32
            // outputs 128 bytes of 16 rows, 4 rows to an instruction.
            if (n >= p.N || row0 >= p.M) continue;
            int part = g, y0 = row0;
            if (p.chunk_rows > 0) {
                part = row0 / p.chunk_rows;
                y0 -= part * p.chunk_rows;
            }
            constexpr int ELEM = F32 ? 4 : 2;
            constexpr int SEG = F32 ? 128 : 64;       // bytes of a row at a time
            constexpr int ROWS = 2048 / SEG;          // rows that the buffer takes
            constexpr int W = SEG / ELEM, V = 16 / ELEM, VECS = SEG / 16;
            auto swizzle = [](int r) { return F32 ? r & 7 : (r >> 1) & 3; };
            uint8_t* out = static_cast<uint8_t*>(p.out[part]) +
                           (static_cast<long long>(y0) * p.N + n) * ELEM;
            const int lr = lane % ROWS, rr = lane / VECS, rv = lane % VECS;
#pragma unroll
            for (int c = 0; c < 128 / W; ++c) {
                if (n + c * W >= p.N) break;  // (the same for the whole warp)
#pragma unroll
                for (int h = 0; h < 32; h += ROWS) {
                    __syncwarp();
                    if (lane - lr == h) {
#pragma unroll
                        for (int q = 0; q < VECS; ++q) {
                            float x[V];
#pragma unroll
                            for (int i = 0; i < V; ++i) {
                                x[i] = acc[c * W + q * V + i];
                                if constexpr (FMT == FP4_NV) x[i] = x[i] * alpha.first * alpha.second;
                            }
                            uint4 u;
                            if constexpr (F32) {
                                u = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]),
                                               __float_as_uint(x[2]), __float_as_uint(x[3]));
                            } else {
                                const float4* b =
                                    reinterpret_cast<const float4*>(bias_buf + c * W + q * V);
                                const float4 b0 = b[0], b1 = b[1];
                                u = make_uint4(bf16x2(x[0] + b0.x, x[1] + b0.y),
                                               bf16x2(x[2] + b0.z, x[3] + b0.w),
                                               bf16x2(x[4] + b1.x, x[5] + b1.y),
                                               bf16x2(x[6] + b1.z, x[7] + b1.w));
                            }
                            *reinterpret_cast<uint4*>(turn + lr * SEG + ((q ^ swizzle(lr)) << 4)) = u;
                        }
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = rr + (32 / VECS) * i;
                        const uint4 u = *reinterpret_cast<const uint4*>(
                            turn + r * SEG + ((rv ^ swizzle(r)) << 4));
                        if (row0 + h + r < p.M && n + c * W + rv * V < p.N)
                            *reinterpret_cast<uint4*>(out + static_cast<long long>(h + r) * p.N * ELEM +
                                                      c * SEG + rv * 16) = u;
                    }
                }
            }
        }
    }

    ptx::tc_fence_before();
    __syncwarp();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    if (*abort_flag) {  // (both CTAs' flag, or neither's)
        // (a warp with registers enough)
        if (warp == 4 && lane == 0)
            settle<FMT>(bar0, nk, (p.total_tiles - cluster - 1) / nclusters + 1, p.timeout_ns, p.err);
        __syncwarp();
        ptx::cluster_sync();
    }
    if (warp == 1) {
        __syncwarp();
        ptx::tmem_dealloc_pair(tmem, F_TMEM_COLS);
    }
}

// CTA pairs that fit on the current device at once (queried once per device and variant).
template <int FMT, bool F32>
cudaError_t max_clusters(int& out) {
    constexpr int kDevices = 64;
    static int known[kDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    int n = __atomic_load_n(&known[dev], __ATOMIC_ACQUIRE);
    if (n == 0) {
        auto kern = fp4_gemm_kernel<FMT, F32>;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<FMT>::kSmem);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2, 1, 1);
        cfg.blockDim = dim3(F_THREADS, 1, 1);
        cfg.dynamicSmemBytes = Shape<FMT>::kSmem;
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

template <int FMT, bool F32>
cudaError_t launch(const Fp4GemmParams& p, cudaStream_t st) {
    int pairs = 0;
    cudaError_t e = max_clusters<FMT, F32>(pairs);
    if (e != cudaSuccess) return e;
    const int clusters = p.total_tiles < pairs ? p.total_tiles : pairs;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * clusters, 1, 1);
    cfg.blockDim = dim3(F_THREADS, 1, 1);
    cfg.dynamicSmemBytes = Shape<FMT>::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fp4_gemm_kernel<FMT, F32>, p);
}

}  // namespace

cudaError_t launch_fp4_gemm(const Fp4GemmParams& p, int fmt, bool f32, cudaStream_t st) {
    if (fmt == FP4_NV) return f32 ? launch<FP4_NV, true>(p, st) : launch<FP4_NV, false>(p, st);
    return f32 ? launch<FP4_MX, true>(p, st) : launch<FP4_MX, false>(p, st);
}

}  // namespace tpmlp
