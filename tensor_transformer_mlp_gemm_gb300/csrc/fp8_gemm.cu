// fp8_gemm.cu -- the 8-bit product with scales per block of 128 on tcgen05 CTA
// pairs (see fp8_gemm.cuh for the mathematics).
//
// The tensor cores apply the scales (fp8_mma.cuh), so the sum over all of K stays
// in tensor memory.  An earlier form kept each K block's sums apart and scaled
// and added them in registers: reading 128 x 256 sums back for every K block
// and the way from there to the next MMAs took 880 clocks a block where the MMAs
// take 512, and that form spent 1050 on scales per column of B.
//
// CTA layout (512 threads, persistent over tiles; both CTAs of a pair compute one
// 256 x 256 tile, 128 rows each):
//   warp 0       TMA producer: this CTA's 128 rows of A and of B for each K block
//   warp 1       owns the tensor memory; in the even CTA issues the pair's MMAs,
//                four K slices of 32 for each K block
//   warps 4..7   scales: the exponents of this CTA's 128 rows of A and of all 256
//                rows of B for each K block, into tensor memory, a slot per stage.
//                Each warp copies a quarter of them to a ring in shared memory, six
//                to nine K blocks ahead, turns them into exponents there, and
//                writes all of them to its quarter of the lanes, three K blocks at
//                a time (one at a time, loaded into registers, took 750 to 1100
//                clocks a block; each warp turning all of them, 840)
//   warps 8..15  output: warp w reads lanes 32 (w % 4) .. of the accumulator and
//                columns 128 ((w - 8) / 4) .. into registers, frees the accumulator
//                for the next tile's MMAs, and writes from there
// Tensor memory: 256 columns of sums, then 6 x 16 columns of scales.  Two
// accumulators of 256 columns leave none for the scales; with one, the MMAs wait for it
// to be read.
// What bounds it: the tensor cores, 512 clocks for each K block of a tile, and nearly as
// much the 32 KB that each CTA takes from L2 for it: with MMAs of 64 columns instead of
// 256 and the same copies, 19456 x 8192 x 1024 took 77 us instead of 94.  (So MMAs of
// fewer columns for a last, narrow tile gained nothing.)  Short K pays for the hand-over
// of the accumulator and the output, about 3000 clocks a tile.  Measured: 2048 x 12288 x
// 36864 in 525 us (3.5 PFLOP/s, the tensor pipe busy in 86 % of the cycles), 16384 x 4096
// x 4096 in 163 us; fp32 outputs of 512 x 4096 each, K = 16384, in 180 us (256 tiles for
// 76 pairs: the fourth wave is a third full), of 1536 x 12288, K = 2048, in 227 us.
//
// Every wait is bounded as in the bf16 GEMM: a wait that expires sets a flag that ends
// the roles of both CTAs, copies and MMAs in flight are drained (bounded), tensor memory
// is freed, and the error word tells the host.  For that each role leaves behind how far
// it came: what counts on a stage's barrier is stood in for where a role stopped before
// it, so that the barrier's phase says when the copies have landed.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fp8_gemm.cuh"
#include "fp8_mma.cuh"

namespace tpmlp {
namespace {

using namespace f8;

constexpr int F_THREADS = 512;
// registers per thread: 128 x 56 + 128 x 72 + 256 x 192 = 65536, as at launch (512 x 128)
constexpr int F_FEW_REGS = 56, F_SCALE_REGS = 72, F_MANY_REGS = 192;
constexpr int F_SCALE_WARPS = 4, F_OUT_WARPS = 8;
constexpr int F_TILE = 256;        // pair tile rows and columns
constexpr int F_STAGES = 6;
constexpr int F_STAGE_BYTES = 2 * F8_BOX_BYTES;
constexpr int F_TMEM_COLS = 512;
constexpr int F_SCALE_COL = 256;   // first column of the scale slots, 16 columns each:
constexpr int F_SCALE_B = 4;       // A's 4, then B's 8
constexpr int F_BIAS = F_OUT_WARPS * 512;   // each output warp's 128 columns, fp32
constexpr int F_TURN = F_OUT_WARPS * 2048;  // and 32 rows of 64 output bytes
constexpr int F_BATCH = 3;       // K blocks the scale warps take at a time
constexpr int F_RING = 3;        // batches in their ring
static_assert(F_STAGES % F_BATCH == 0, "a batch's stages are consecutive");
constexpr int F_SLOT = 32 * 12 * 4;  // scales of a K block: [c][lane], c as below
constexpr int F_SWAP = F_RING * F_BATCH * F_SLOT;
constexpr int F_SMEM = 1024 + F_STAGES * F_STAGE_BYTES + F_BIAS + F_TURN + F_SWAP + 256;
static_assert(F_SMEM <= 232448, "fits a CTA");

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

// How many K blocks a role that gave up has done (one that did not: all), 64-bit counts in
// shared memory: in the even CTA those copied and those with scales, by it and by the odd
// one; in both those issued.
constexpr int F_BLOCKS_DONE = 16 * F_STAGES + 32;  // from the barriers on
constexpr int F_COPIED = 0, F_SCALED = 2, F_ISSUED = 4, F_COUNTS = 5;

// After a wait has expired and every role has left its loop: what a CTA has under way ends.
// (Not inlined: its values would take registers from the roles.)
__device__ __noinline__ void settle(uint32_t bar0, int nk, int tiles, unsigned long long timeout_ns,
                                    unsigned* err) {
    constexpr int NST = F_STAGES;
    const uint32_t bar_full = bar0, bar_empty = bar0 + 8 * NST, bar_done = bar0 + 16 * NST;
    const long long* counts = static_cast<const long long*>(__cvta_shared_to_generic(bar0 + F_BLOCKS_DONE));
    auto blocks = [&](int i) { return min(counts[i], static_cast<long long>(tiles) * nk); };
    if (ptx::cluster_ctarank() == 0) {
        // the copies of both CTAs
        const long long even = blocks(F_COPIED), odd = blocks(F_COPIED + 1), n = max(even, odd);
        for (long long k = max(0LL, n - NST); k < n; ++k) {
            const uint32_t full = bar_full + 8 * static_cast<uint32_t>(k % NST);
            if (k >= even)
                ptx::mbar_arrive_expect_tx(full, F_STAGE_BYTES);  // the odd CTA's only
            else if (k >= odd)
                complete_tx(full, F_STAGE_BYTES);  // which will not come
            for (int r = 0; r < 2; ++r)
                for (int w = 0; w < F_SCALE_WARPS; ++w)
                    if (k >= blocks(F_SCALED + r)) arrive_relaxed(full);
            drain(full, static_cast<uint32_t>((k / NST) & 1), timeout_ns, err);
        }
    }
    // the MMAs' arrivals on this CTA (the MMAs themselves have ended)
    const long long n = blocks(F_ISSUED), whole = n / nk;
    for (long long k = max(0LL, n - NST); k < n; ++k)
        drain(bar_empty + 8 * static_cast<uint32_t>(k % NST), static_cast<uint32_t>((k / NST) & 1),
              timeout_ns, err);
    if (whole > 0) drain(bar_done, static_cast<uint32_t>((whole - 1) & 1), timeout_ns, err);
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

template <int OUT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(F_THREADS, 1)
    fp8_gemm_kernel(const __grid_constant__ Fp8GemmParams p) {
    constexpr bool F32 = OUT == F8_F32_VECTOR;
    constexpr int NST = F_STAGES;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* after = smem_raw + (base - raw) + NST * F_STAGE_BYTES;
    const uint32_t bar0 = base + NST * F_STAGE_BYTES + F_BIAS + F_TURN + F_SWAP;
    uint8_t* bar_area = after + F_BIAS + F_TURN + F_SWAP;
    const uint32_t bar_full = bar0;              // [NST] even CTA: both CTAs' operands and scales
    const uint32_t bar_empty = bar0 + 8 * NST;   // [NST] both CTAs
    const uint32_t bar_done = bar0 + 16 * NST;   // both CTAs: the tile is in the accumulator
    const uint32_t bar_free = bar_done + 8;      // even CTA: both CTAs have read it
    const uint32_t bar_drain = bar_free + 8;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_area + 16 * NST + 24);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bar_area + 16 * NST + 28);
    const uint32_t blocks_done = bar0 + F_BLOCKS_DONE;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(ptx::cluster_ctarank());
    const int cluster = blockIdx.x / 2, nclusters = gridDim.x / 2;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NST; ++s) {
            ptx::mbar_init(bar_full + 8 * s, 1 + 2 * F_SCALE_WARPS);
            ptx::mbar_init(bar_empty + 8 * s, 1);
        }
        ptx::mbar_init(bar_done, 1);
        ptx::mbar_init(bar_free, 2 * F_OUT_WARPS);
        ptx::mbar_init(bar_drain, 1);
        *abort_flag = 0;
        for (int i = 0; i < F_COUNTS; ++i)
            reinterpret_cast<long long*>(bar_area + F_BLOCKS_DONE)[i] = 0x7FFFFFFFFFFFFFFFLL;
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
    // a wait of this kernel; who gives up takes the other CTA along
    auto wait_for = [&](uint32_t bar, uint32_t parity, unsigned code) {
        if (wait(bar, parity, abort_flag, p.timeout_ns, p.err, code)) return true;
        store_cluster(ptx::mapa_shared(bar0 + 16 * NST + 28, static_cast<uint32_t>(rank ^ 1)), 1);
        return false;
    };

    if (warp < 4) {
        reg_dec<F_FEW_REGS>();
        if (warp == 0 && lane == 0) {
            // ---------------- TMA producer ----------------
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
                        if ((fills == p.stall && rank == 1) ||
                            !wait_for(bar_empty + 8 * stage, phase ^ 1u, ERR_PRODUCER)) {
                            ok = false;
                            break;
                        }
                        const uint32_t sa = base + stage * F_STAGE_BYTES, full = even_full + 8 * stage;
                        const int k0 = kb * F8_BK;
                        if (rank == 0)  // counts both CTAs' bytes
                            ptx::mbar_arrive_expect_tx(bar_full + 8 * stage, 2 * F_STAGE_BYTES);
                        ptx::tma_load_2d_pair(sa, am, p.a_mn ? arow : k0, p.a_mn ? k0 : arow, full);
                        ptx::tma_load_2d_pair(sa + F8_BOX_BYTES, bm, p.b_mn ? brow : k0,
                                              p.b_mn ? k0 : brow, full);
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
            if (!ok) store_cluster64(ptx::mapa_shared(blocks_done + 8 * (F_COPIED + rank), 0), fills);
        } else if (warp == 1 && rank == 0) {
            // ---------------- MMA issuer ----------------
            // The whole warp walks the loop and one lane issues, so the descriptors
            // stay in uniform registers.
            const uint32_t id = idesc(F_TILE, F_TILE, p.a_mn, p.b_mn) | p.ab_format;
            const uint64_t da = operand_desc(base, 0, p.a_mn);
            const uint64_t db = operand_desc(base + F8_BOX_BYTES, 0, p.b_mn);
            const uint32_t ka = (p.a_mn ? 4096 : 32) >> 4, kb = (p.b_mn ? 4096 : 32) >> 4;
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
                    const uint32_t step = stage * (F_STAGE_BYTES >> 4);
                    const uint32_t sf = tmem + F_SCALE_COL + stage * 16;
                    if (elect_one()) {
#pragma unroll
                        for (uint32_t k = 0; k < 4; ++k)
                            mma_pair(tmem, da + step + k * ka, db + step + k * kb, id, sf,
                                     sf + F_SCALE_B, (kk > 0 || k > 0) ? 1u : 0u);
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
                    store_cluster64(ptx::mapa_shared(blocks_done + 8 * F_ISSUED, r), issued);
            }
            __syncwarp();
        }
    } else if (warp < 8) {
        // ---------------- scales ----------------
        reg_dec<F_SCALE_REGS>();
        const int q = warp & 3;  // its quarter of the lanes
        const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16) + F_SCALE_COL;
        const uint32_t even_full = ptx::mapa_shared(bar_full, 0);
        uint8_t* ring = after + F_BIAS + F_TURN;
        const uint32_t ring_u32 = base + NST * F_STAGE_BYTES + F_BIAS + F_TURN;
        // Scales 0..3 of a lane are A's rows lane + 32 c, 4..11 B's rows lane + 32 (c - 4).
        // This warp fetches A's c = q and B's 4 + 2q, 5 + 2q; of a weight, whose 128 rows
        // have one scale, two lanes of warp 0 fetch two.
        struct {
            int tile, seg, kb, m, n, g;
            const float *a, *b;
        } f;
        f.tile = cluster;
        auto start_segment = [&] {
            f.a = p.sa[pick(p.a_part, f.g, f.seg)] + f.m;
            f.b = p.sb[pick(p.b_part, f.g, f.seg)] + (F32 ? f.n : (f.n >> 7) * p.sb_n);
        };
        auto start_tile = [&] {
            int m0, n0;
            decode(p, f.tile, f.g, m0, n0);
            f.m = m0 + rank * 128 + lane + 32 * q;
            f.n = F32 ? n0 + lane + 64 * q : n0 + 128 * (lane & 1);
            f.seg = f.kb = 0;
            start_segment();
        };
        if (f.tile < p.total_tiles) start_tile();
        auto fetch = [&](uint32_t slot) {
            if (f.tile >= p.total_tiles) return;
            const uint32_t dst = ring_u32 + slot * F_SLOT + lane * 4;
            copy4(dst + q * 128, f.m < p.M ? f.a : p.sa[0], f.m < p.M);
            if constexpr (F32) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bool in = f.n + 32 * i < p.N;
                    copy4(dst + (4 + 2 * q + i) * 128, in ? f.b + 32 * i : p.sb[0], in);
                }
            } else if (q == 0 && lane < 2) {
                copy4(dst + 4 * 128, f.n < p.N ? f.b : p.sb[0], f.n < p.N);
            }
            f.a += p.sa_kb;
            f.b += p.sb_kb;
            if (++f.kb == kblocks) {
                f.kb = 0;
                if (++f.seg == p.ksegs) {
                    f.tile += nclusters;
                    if (f.tile < p.total_tiles) start_tile();
                } else {
                    start_segment();
                }
            }
        };
        auto fetch_batch = [&](uint32_t batch) {
#pragma unroll
            for (int u = 0; u < F_BATCH; ++u) fetch((batch % F_RING) * F_BATCH + u);
            copy_commit();
        };
#pragma unroll
        for (int i = 0; i < F_RING - 1; ++i) fetch_batch(i);
        const int tiles = cluster < p.total_tiles ? (p.total_tiles - cluster - 1) / nclusters + 1 : 0;
        const long long blocks = static_cast<long long>(tiles) * nk;
        int stage = 0;
        uint32_t phase = 0;
        uint32_t slot = 0, batch = 0;
        long long done = 0;
        for (; done < blocks; done += F_BATCH, ++batch) {
            const int here = blocks - done < F_BATCH ? static_cast<int>(blocks - done) : F_BATCH;
            // the stages' last MMAs have read their scales (they end in order)
            const bool ok = wait_for(bar_empty + 8 * (stage + here - 1), phase ^ 1u, ERR_PRODUCER);
            copy_wait<F_RING - 2>();
            // what this thread copied, as exponents
            uint32_t* words = reinterpret_cast<uint32_t*>(ring + slot * (F_BATCH * F_SLOT)) + lane;
            if (++slot == F_RING) slot = 0;
#pragma unroll
            for (int u = 0; u < F_BATCH; ++u) {
                uint32_t* x = words + u * (F_SLOT / 4);
                x[32 * q] = scale_word(x[32 * q]);
                if constexpr (F32) {
                    uint32_t* y = x + 32 * (4 + 2 * q);
                    y[0] = scale_word(y[0]);
                    y[32] = scale_word(y[32]);
                } else if (q == 0 && lane < 2) {
                    x[32 * 4] = scale_word(x[32 * 4]);
                }
            }
            // this batch is ready and the one before it has been read by all four warps,
            // which also give up together
            if (barrier_any<F_SCALE_WARPS * 32>(!ok)) break;
            ptx::tc_fence_after();
#pragma unroll
            for (int u = 0; u < F_BATCH; ++u) {
                if (u < here) {
                    const uint32_t* x = words + u * (F_SLOT / 4);
                    uint32_t w[12];
#pragma unroll
                    for (int c = 0; c < 4; ++c) w[c] = x[32 * c];
                    if constexpr (F32) {
#pragma unroll
                        for (int c = 4; c < 12; ++c) w[c] = x[32 * c];
                    } else {
                        const uint2 y = *reinterpret_cast<const uint2*>(x - lane + 32 * 4);
                        w[4] = w[5] = w[6] = w[7] = y.x;
                        w[8] = w[9] = w[10] = w[11] = y.y;
                    }
                    const uint32_t t = lanes + (stage + u) * 16;
                    store_cols4(t, w);
                    store_cols8(t + F_SCALE_B, w + 4);
                }
            }
            store_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
#pragma unroll
                for (int u = 0; u < F_BATCH; ++u)
                    if (u < here) arrive_relaxed_cluster(even_full + 8 * (stage + u));
            }
            // into the batch before this one, which all four have read
            fetch_batch(batch + F_RING - 1);
            stage += F_BATCH;
            if (stage == NST) {
                stage = 0;
                phase ^= 1u;
            }
        }
        copy_wait<0>();
        // (the four warps go on and give up together)
        if (done < blocks && warp == 4 && lane == 0)
            store_cluster64(ptx::mapa_shared(blocks_done + 8 * (F_SCALED + rank), 0), done);
    } else {
        // ---------------- output ----------------
        reg_inc<F_MANY_REGS>();
        const int quarter = warp & 3;         // the accumulator lanes this warp may read
        const int side = (warp - 8) >> 2;     // its 128 columns
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + side * 128;
        const uint32_t even_free = ptx::mapa_shared(bar_free, 0);
        float* bias_buf = reinterpret_cast<float*>(after) + (warp - 8) * 128;
        uint8_t* turn = after + F_BIAS + (warp - 8) * 2048;
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

            // The warp's rows are turned round in shared memory and leave as whole
            // sectors: 64 bytes of all 32 rows at a time, 8 rows to a store instruction,
            // or of fp32 outputs, where the stores count, 128 bytes of 16 rows, 4 rows to
            // an instruction (1 K block a tile, 4432 x 7744: 35 us instead of 39; bf16
            // outputs so 8 % slower).  (Bulk stores waited for each other's staging, 8600
            // clocks a tile; each thread storing along its own row, 32 rows to an
            // instruction, took 9800; this takes about 6500.)
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
                            const float* x = acc + c * W + q * V;
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
        if (warp == 8 && lane == 0)
            settle(bar0, nk, (p.total_tiles - cluster - 1) / nclusters + 1, p.timeout_ns, p.err);
        __syncwarp();
        ptx::cluster_sync();
    }
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
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, F_SMEM);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2, 1, 1);
        cfg.blockDim = dim3(F_THREADS, 1, 1);
        cfg.dynamicSmemBytes = F_SMEM;
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
    cfg.dynamicSmemBytes = F_SMEM;
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
