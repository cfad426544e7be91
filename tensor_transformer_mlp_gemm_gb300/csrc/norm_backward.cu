// norm_backward.cu -- backward pass of the norms around a block (see
// norm_residual.cuh for the mathematics).
//
// What bounds it: HBM traffic, dOut, dXn, Z and Out read and dX and dZ written once
// (12 bytes an element).  So everything a row gives, its two data gradients and its
// share of up to five column sums, comes from one pass: a thread keeps the sums of
// its 8 columns in registers over all of its rows.
//
// A row has two sums over its columns, one after the other (dZ needs dX's first), and
// one row at a time spent 2800 clocks on them whatever its width, where 4096 columns
// are worth 2100 of HBM time.  So a group of threads takes two rows at a time, narrow
// rows are spread over up to 6 groups of a CTA's threads, and one thread of a group
// keeps bulk copies of its next rows under way into a ring in shared memory.
// Rows of more than 4096 columns take a cluster of 2 to 4 CTAs side by side, whose row
// sums meet in each other's shared memory: each warp sends its part to every CTA,
// counted on that CTA's mbarrier, and every warp adds all parts in the same order.  (A
// cluster barrier instead waits for the row's own loads and stores too: 6600 clocks a
// row, measured at 917 x 9000.)  As many clusters are launched as run at once (46 of 3
// and 36 of 4 on 152 SMs): two more made a second wave and doubled the time.
// A CTA has 384 threads where those hold the row or rows: they have registers for
// everything.  With 512 instead, rms and layer norms at 16384 x 2560 took 131 and 166 us,
// now 115 and 136; 16384 x 1536 90 and 115, now 70 and 80; 16384 x 1024, as 3 groups
// instead of 4, 55 and 71, now 51 and 59; 917 x 9000 layer 53, now 43; 2048 x 12288 layer
// 111 as 3 x 512, 105 as 4 x 384.
// The column sums of a block of rows go to a partial row, and a second kernel adds the
// blocks in order; a gate whose rows lie in one group is finished there.  No atomics.
// Measured, rms norms and 8 gates, back to back, both launches: 16384 x 4096 in 137 us (5.9
// TB/s), layer norms 159; 8192 x 8192 165 and 190; 2048 x 12288 76; 16384 x 2048 80; 16384 x
// 1024 46; 917 x 9000 and 7 gates, layer, 37.  (Figures above: cold caches, up to 6 us more.)
#include <algorithm>

#include "gemm_params.h"
#include "norm_device.cuh"
#include "norm_residual.cuh"
#include "ptx.cuh"

namespace tpmlp {
namespace {

using namespace nr;

constexpr int NB_THREADS = 512;          // of a CTA
constexpr int NB_FEWER = 384;            // where they hold the row
constexpr int NB_COLS = NB_THREADS * 8;  // columns of one CTA
constexpr int NB_WARPS = NB_THREADS / 32;
constexpr int NB_MAX_CLUSTER = 4;
constexpr int NB_MAX_GROUPS = 6;
constexpr int NB_ROWS = 2;               // rows a group takes at a time
constexpr int NB_ARRAYS = 5;             // dOut, dXn, Out, Z, gate
constexpr int NB_STAGES = 2;             // row pairs in the ring
constexpr int NB_RING = NB_STAGES * NB_ROWS * NB_ARRAYS * NB_COLS * 2;
static_assert(NB_COLS * NB_MAX_CLUSTER >= NR_MAX_H, "a cluster holds the widest row");

// CTAs side by side for a row, groups of a CTA's threads that take rows of their own, and
// the CTA's threads: 384 unless only 512 hold one or two rows.  Every CTA of a cluster has
// columns of the row.
int cluster_of(long long h) {
    return h <= NB_COLS ? 1 : h <= 2 * NB_COLS ? 2 : h <= 3 * NB_FEWER * 8 ? 3 : 4;
}
int groups_of(long long h) {
    if (h > NB_COLS / 2) return 1;
    for (int g : {6, 4, 3})
        if (h * g <= NB_FEWER * 8) return g;
    return 2;
}
int threads_of(long long h) {
    return h * groups_of(h) <= static_cast<long long>(cluster_of(h)) * NB_FEWER * 8 ? NB_FEWER
                                                                                    : NB_THREADS;
}

// A float into a CTA of the cluster, its four bytes counted on that CTA's mbarrier.
__device__ __forceinline__ void send(uint32_t addr, float v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(
                     addr),
                 "r"(__float_as_uint(v)), "r"(bar)
                 : "memory");
}

// What the sums of a CTA need: the parts [group][buf][value][slot], a slot for each warp
// of the row, mbarriers (the cluster's sums, the ring), and the limit of a wait.
constexpr int NB_VALUES = 2 * NB_ROWS;
struct Shared {
    float part[2][NB_VALUES * NB_MAX_CLUSTER * NB_WARPS];  // groups side by side
    alignas(8) uint64_t sum_bar[2];
    uint64_t ring_bar[NB_MAX_GROUPS][NB_STAGES];
    // What the end after an expired wait needs.  It is not in registers: the row loop has
    // none left (there it spilled: layer norms of 16384 x 4096 221 us, not 159).
    volatile int gave_up;                       // a wait of the CTA has expired
    volatile uint32_t copy_end[NB_MAX_GROUPS];  // rows of a group below this are copied,
    volatile uint32_t row0[NB_MAX_GROUPS];      // from this one on
    // copies not waited for: two pairs of rows from this one on, below that one
    volatile uint32_t under_way[NB_MAX_GROUPS], under_way_end[NB_MAX_GROUPS];
};
// A CTA with a wait that has expired waits no more, sends no more and copies no more, but
// goes through the rows that are left, so that no barrier misses a thread.
struct Waits {
    unsigned long long timeout_ns;
    unsigned* err;
};

template <typename F>
__device__ __forceinline__ void wait_on(uint32_t bar, uint32_t parity, const Waits& w, Shared& sm,
                                        F&& expired) {
    if (ptx::mbar_try_wait(bar, parity)) return;
    const uint64_t t0 = ptx::globaltimer_ns();
    while (!ptx::mbar_try_wait(bar, parity)) {
        if (sm.gave_up || ptx::globaltimer_ns() - t0 > w.timeout_ns) {
            atomicOr(w.err, ERR_EPILOGUE);
            expired();
            return;
        }
    }
}

// Sums of N (1, 2 or 4) values over the warp: value n's is left in the 32 / N lanes from
// n * 32 / N on.  Halving the values at each of the first steps takes 5 or 6 shuffles.
template <int N>
__device__ __forceinline__ float warp_sums(const float (&v)[N], int lane) {
    float x;
    if constexpr (N == 4) {
        const bool up = lane & 16, odd = lane & 8;
        float a = up ? v[2] : v[0], b = up ? v[3] : v[1];
        a += __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 16);
        b += __shfl_xor_sync(0xffffffffu, up ? v[1] : v[3], 16);
        x = odd ? b : a;
        x += __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
    } else if constexpr (N == 2) {
        const bool up = lane & 16;
        x = up ? v[1] : v[0];
        x += __shfl_xor_sync(0xffffffffu, up ? v[0] : v[1], 16);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
    } else {
        x = v[0];
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
    }
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Sums of N values over a row: the group's warps, and the cluster's CTAs.  The buffers
// alternate: a part of the next but one sum can only come once every warp has given its
// part of the next, and so has read this one.
template <int CL, int WG, int N, typename F>
__device__ __forceinline__ void row_sums(float (&v)[N], Shared& sm, int& buf, uint32_t (&phase)[2],
                                         int group, int rank, const Waits& w, F&& expired) {
    constexpr int SLOTS = CL * WG, LP = 32 / N;
    const int warp = (threadIdx.x >> 5) % WG, lane = threadIdx.x & 31;
    float* part = sm.part[buf] + group * (NB_VALUES * WG);
    const float x = warp_sums<N>(v, lane);
    const int n = lane / LP, slot = rank * WG + warp;
    if constexpr (CL == 1) {
        if (lane % LP == 0) part[n * SLOTS + slot] = x;
        asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + group), "n"(WG * 32) : "memory");
    } else {
        const uint32_t bar = ptx::smem_u32(&sm.sum_bar[buf]);
        const bool alive = !sm.gave_up;
        if (threadIdx.x == 0 && alive) ptx::mbar_arrive_expect_tx(bar, SLOTS * N * 4);
        // lane n * LP + i sends value n to CTA i
        if (lane % LP < CL && alive) {
            const uint32_t to = static_cast<uint32_t>(lane % LP);
            send(ptx::mapa_shared(ptx::smem_u32(part + n * SLOTS + slot), to), x,
                 ptx::mapa_shared(bar, to));
        }
        __syncwarp();
        wait_on(bar, phase[buf], w, sm, expired);
        phase[buf] ^= 1u;
    }
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < (SLOTS + LP - 1) / LP; ++i)
        if (i * LP + lane % LP < SLOTS) t += part[n * SLOTS + i * LP + lane % LP];
#pragma unroll
    for (int o = LP / 2; o >= 1; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, t, i * LP);
    buf ^= 1;
}

template <int POST, int PRE, int CL, int G, int THREADS>
__global__ void __launch_bounds__(THREADS, 1)
    nr_backward_kernel(const __grid_constant__ NrBackwardParams p) {
    constexpr bool Z = POST != NR_ABSENT, POST_NORM = POST >= NR_POST_RMS, BEFORE = PRE != NR_NONE;
    constexpr bool POST_LAYER = POST == NR_POST_LAYER, PRE_LAYER = PRE == NR_PRE_LAYER;
    constexpr int R = NB_ROWS, GT = THREADS / G, WG = GT / 32, ROW = GT * 16;  // a row's bytes in the ring
    static_assert(CL == 1 || G == 1, "wide rows take whole CTAs");
    static_assert(WG > 1, "a group's warps meet at a barrier");
    // Z and the gate are read from the ring when they are needed, not held from the start:
    // that spilled (layer norms, 16384 x 4096 182 us instead of 168; rms norms, 16384 x
    // 2048 94 instead of 85).  Where they fit they are held, and the stage is free sooner
    // (rms norms, 16384 x 4096 139 us, not 147).
    constexpr bool HOLD = THREADS == NB_THREADS && G == 1 && !POST_LAYER && !PRE_LAYER;
    extern __shared__ __align__(128) uint8_t ring_all[];
    __shared__ Shared sm;
    const int rank = CL == 1 ? 0 : static_cast<int>(ptx::cluster_ctarank());
    const int group = threadIdx.x / GT, tid = threadIdx.x % GT, lane = threadIdx.x & 31;
    const long long block = blockIdx.x / CL;
    const float inv_h = 1.0f / static_cast<float>(p.h);
    const int c0 = rank * (THREADS * 8), c = c0 + tid * 8;
    const bool in = c < p.h;
    const Waits waits = {p.timeout_ns, p.err};
    const bool gate = Z && p.gate != nullptr, dout = p.dout.p[0] != nullptr;
    uint8_t* ring = ring_all + group * (NB_STAGES * R * NB_ARRAYS * ROW);
    int buf = 0;
    uint32_t phase[2] = {0, 0};

    if (threadIdx.x == 0) {
        ptx::mbar_init(ptx::smem_u32(&sm.sum_bar[0]), 1);
        ptx::mbar_init(ptx::smem_u32(&sm.sum_bar[1]), 1);
        sm.gave_up = 0;
        for (int g = 0; g < G; ++g)
            for (int s = 0; s < NB_STAGES; ++s) ptx::mbar_init(ptx::smem_u32(&sm.ring_bar[g][s]), 1);
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    __syncthreads();
    if constexpr (CL > 1) ptx::cluster_sync();  // all of the cluster's barriers exist
    ptx::griddep_wait();

    auto weight = [&](const void* w) {
        return in ? __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + c)) : zero4();
    };
    const uint4 w1 = POST_NORM ? weight(p.post_gamma) : zero4();
    const uint4 b1 = POST_LAYER ? weight(p.post_beta) : zero4();
    const uint4 w2 = BEFORE ? weight(p.pre_gamma) : zero4();

    // this group's rows: a part of a cut gate's, or whole gates
    const bool cut = p.blocks_per_seq > 0;
    long long row, last;
    if (cut) {
        const long long seq = block / p.blocks_per_seq, first = seq * p.gate_rows;
        const long long b0 = first + (block - seq * p.blocks_per_seq) * p.rows_per_block;
        const long long b1r = min(b0 + p.rows_per_block, first + p.gate_rows);
        const long long per = (p.rows_per_block + G - 1) / G;
        row = min(b0 + group * per, b1r);
        last = min(row + per, b1r);
    } else {
        const long long per = p.seqs_per_group * p.gate_rows;
        row = min((block * G + group) * per, p.T);
        last = min(row + per, p.T);
    }

    // the ring: one thread of the group has the copies of a row pair under way
    const int cols = min(GT * 8, p.h - c0);
    const uint32_t bytes = static_cast<uint32_t>(cols) * 2;
    // (a row's token chunk and gate are stepped, not divided out: the divisions were
    // half of all instructions)
    Stepper copy_chunk(row, 1, p.rows_per_chunk), copy_gate(row, 1, p.gate_rows);
    auto copy_rows = [&](long long r0, int stage) {
        const uint32_t bar = ptx::smem_u32(&sm.ring_bar[group][stage]);
        const int n = r0 + 1 < last ? 2 : 1;
        const int arrays = (dout ? 1 : 0) + (BEFORE ? 2 : 0) + (Z ? 1 : 0) + (gate ? 1 : 0);
        ptx::mbar_arrive_expect_tx(bar, bytes * static_cast<uint32_t>(n * arrays));
        for (int i = 0; i < n; ++i) {
            const uint32_t k = copy_chunk.q;
            const long long off = static_cast<long long>(copy_chunk.r) * p.h + c0;
            const uint32_t dst = ptx::smem_u32(ring) + (stage * R + i) * (NB_ARRAYS * ROW);
            auto get = [&](int a, const void* base, long long o) {
                asm volatile(
                    "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                        dst + a * ROW),
                    "l"(static_cast<const __nv_bfloat16*>(base) + o), "r"(bytes), "r"(bar)
                    : "memory");
            };
            if (dout) get(0, p.dout.p[k], off);
            if (BEFORE) {
                get(1, p.dxn.p[k], off);
                get(2, p.out.p[k], off);
            }
            if (Z) get(3, p.z.p[k], off);
            if (gate) get(4, p.gate, static_cast<long long>(copy_gate.q) * p.h + c0);
            copy_chunk.step();
            copy_gate.step();
        }
    };
    if (tid == 0) {
#pragma unroll
        for (int s = 0; s < NB_STAGES; ++s)
            if (row + s * R < last && (p.stall < 0 || rank + 1 < CL || s < p.stall))
                copy_rows(row + s * R, s);
        sm.row0[group] = static_cast<uint32_t>(row);
        sm.copy_end[group] = static_cast<uint32_t>(
            p.stall < 0 || rank + 1 < CL ? last : min(last, row + static_cast<long long>(p.stall) * R));
        sm.under_way_end[group] = 0;
    }
    // lane 4 i + k has statistic k of the pair's row i
    auto load_stats = [&](long long r0) {
        const long long r = r0 + (lane >> 2);
        return lane < 4 * R && r < last && (POST_NORM || BEFORE)
                   ? __ldg(p.stats + (lane & 3) * p.T + r)
                   : 0.0f;
    };
    float stat = load_stats(row);

    float2 s_pre[4] = {}, s_pre_b[4] = {}, s_post[4] = {}, s_post_b[4] = {}, s_gate[4] = {};
    int stage = 0;
    uint32_t ring_phase = 0;
    Stepper chunk(row, 1, p.rows_per_chunk), seq(row, 1, p.gate_rows);
    // a wait has expired: under way may be the pair from row r on and the next one
    auto expired = [&](long long r) {
        sm.gave_up = 1;
        if (tid == 0 && sm.copy_end[group] > 0) {
            sm.under_way[group] = static_cast<uint32_t>(r);
            sm.under_way_end[group] = sm.copy_end[group];
            sm.copy_end[group] = 0;
        }
    };
    for (; row < last; row += R) {
        wait_on(ptx::smem_u32(&sm.ring_bar[group][stage]), ring_phase, waits, sm, [&] { expired(row); });
        uint4 q_dout[R], q_dxn[R], q_out[R], q_z[R], q_gate[R];
        float m1[R], r1[R], m2[R], r2[R];
        const uint8_t* src = ring + stage * (R * NB_ARRAYS * ROW) + tid * 16;
        auto get = [&](int i, int a) {
            return in && row + i < last
                       ? *reinterpret_cast<const uint4*>(src + (i * NB_ARRAYS + a) * ROW)
                       : zero4();
        };
        // (one CTA's sums wait on no mbarrier, so what follows the pair is known here, if
        // there are registers to keep it in)
        constexpr bool EARLY = CL == 1 && THREADS == NB_FEWER;
        const bool more = EARLY && tid == 0 && row + NB_STAGES * R < sm.copy_end[group];
        // every thread of the group has read this stage
        auto release = [&] {
            if (EARLY ? more : tid == 0 && row + NB_STAGES * R < sm.copy_end[group])
                copy_rows(row + NB_STAGES * R, stage);
            if (++stage == NB_STAGES) {
                stage = 0;
                ring_phase ^= 1u;
            }
        };
        auto group_sync = [&] {
            asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + group), "n"(GT) : "memory");
        };
#pragma unroll
        for (int i = 0; i < R; ++i) {
            q_dout[i] = dout ? get(i, 0) : zero4();
            if (BEFORE) {
                q_dxn[i] = get(i, 1);
                q_out[i] = get(i, 2);
            }
            if (Z && HOLD) {
                q_z[i] = get(i, 3);
                q_gate[i] = gate ? get(i, 4) : zero4();
            }
            // (a row that is not there has statistics 0: nothing comes of it)
            m1[i] = POST_LAYER ? __shfl_sync(0xffffffffu, stat, 4 * i) : 0.0f;
            r1[i] = POST_NORM ? __shfl_sync(0xffffffffu, stat, 4 * i + 1) : 0.0f;
            m2[i] = PRE_LAYER ? __shfl_sync(0xffffffffu, stat, 4 * i + 2) : 0.0f;
            r2[i] = BEFORE ? __shfl_sync(0xffffffffu, stat, 4 * i + 3) : 0.0f;
            // (nor of columns outside the row, which hold zeros)
            if (POST_LAYER && !in) m1[i] = 0.0f;
            if (PRE_LAYER && !in) m2[i] = 0.0f;
        }
        stat = load_stats(row + R);

        float2 g[R][4];
        if constexpr (BEFORE) {
            constexpr int N = PRE_LAYER ? 2 * R : R;
            float sums[N];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float2 d[4], v[4], w[4];
                unpack(q_dxn[i], d);
                unpack(q_out[i], v);
                unpack(w2, w);
                const float2 m = both(-m2[i]), r = both(r2[i]);
                float2 sv = both(0.0f), sw = both(0.0f);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 hat = __fmul2_rn(PRE_LAYER ? __fadd2_rn(v[e], m) : v[e], r);
                    s_pre[e] = __ffma2_rn(d[e], hat, s_pre[e]);
                    if (PRE_LAYER) s_pre_b[e] = __fadd2_rn(s_pre_b[e], d[e]);
                    const float2 wd = __fmul2_rn(w[e], d[e]);
                    sv = __ffma2_rn(wd, hat, sv);
                    if (PRE_LAYER) sw = __fadd2_rn(sw, wd);
                }
                sums[i] = sv.x + sv.y;
                if (PRE_LAYER) sums[R + i] = sw.x + sw.y;
            }
            row_sums<CL, WG, N>(sums, sm, buf, phase, group, rank, waits, [&] { expired(row); });
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float2 d[4], v[4], w[4];
                unpack(q_dxn[i], d);
                unpack(q_out[i], v);
                unpack(w2, w);
                unpack(q_dout[i], g[i]);
                const float2 m = both(-m2[i]), r = both(r2[i]), mv = both(-sums[i] * inv_h),
                             mw = both(PRE_LAYER ? -sums[R + i] * inv_h : 0.0f);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 hat = __fmul2_rn(PRE_LAYER ? __fadd2_rn(v[e], m) : v[e], r);
                    const float2 wd = PRE_LAYER ? __ffma2_rn(w[e], d[e], mw) : __fmul2_rn(w[e], d[e]);
                    g[i][e] = __ffma2_rn(r, __ffma2_rn(hat, mv, wd), g[i][e]);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i) unpack(q_dout[i], g[i]);
        }
        if constexpr (!Z || HOLD) {
            // (else the group met at its sums; over a cluster they meet at an mbarrier, which
            // does not order what a thread has read and not yet used)
            if constexpr (!BEFORE || CL > 1) group_sync();
            release();
        }
        uint32_t k[R];
        long long off[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            k[i] = chunk.q;
            off[i] = static_cast<long long>(chunk.r) * p.h + c;
            chunk.step();
            if (in && row + i < last) {
                float2 o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = Z ? __fmul2_rn(both(p.alpha), g[i][e]) : g[i][e];
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.dx[k[i]]) + off[i]) = pack(o);
            }
        }
        if constexpr (Z) {
            constexpr int N = POST_LAYER ? 2 * R : R;
            float sums[N];
            float2 w[4], b[4];
            unpack(w1, w);
            unpack(b1, b);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float2 z[4], t[4];
                if (!HOLD) {
                    q_z[i] = get(i, 3);
                    q_gate[i] = gate ? get(i, 4) : zero4();
                }
                unpack(q_z[i], z);
                unpack(q_gate[i], t);
                const float2 m = both(-m1[i]), r = both(r1[i]);
                float2 sv = both(0.0f), sw = both(0.0f);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 hat =
                        POST_NORM ? __fmul2_rn(POST_LAYER ? __fadd2_rn(z[e], m) : z[e], r) : z[e];
                    if (gate) {
                        const float2 u = POST_LAYER  ? __ffma2_rn(hat, w[e], b[e])
                                         : POST_NORM ? __fmul2_rn(hat, w[e])
                                                     : hat;
                        s_gate[e] = __ffma2_rn(g[i][e], u, s_gate[e]);
                        g[i][e] = __fmul2_rn(g[i][e], t[e]);
                    }
                    if (POST_NORM) {
                        s_post[e] = __ffma2_rn(g[i][e], hat, s_post[e]);
                        if (POST_LAYER) s_post_b[e] = __fadd2_rn(s_post_b[e], g[i][e]);
                        const float2 wd = __fmul2_rn(w[e], g[i][e]);
                        sv = __ffma2_rn(wd, hat, sv);
                        if (POST_LAYER) sw = __fadd2_rn(sw, wd);
                    }
                }
                if (POST_NORM) {
                    sums[i] = sv.x + sv.y;
                    if (POST_LAYER) sums[R + i] = sw.x + sw.y;
                }
                const uint32_t seq_q = seq.q;
                const bool seq_end = seq.r + 1 == seq.n;
                seq.step();
                if (gate && !cut && row + i < last && seq_end) {
                    // the gate's last row: its sum is complete
                    if (in) {
                        float4* dst = reinterpret_cast<float4*>(
                            p.dgate + static_cast<long long>(seq_q) * p.h + c);
                        dst[0] = make_float4(s_gate[0].x, s_gate[0].y, s_gate[1].x, s_gate[1].y);
                        dst[1] = make_float4(s_gate[2].x, s_gate[2].y, s_gate[3].x, s_gate[3].y);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) s_gate[e] = both(0.0f);
                }
            }
            if constexpr (POST_NORM) {
                row_sums<CL, WG, N>(sums, sm, buf, phase, group, rank, waits,
                                    [&] { expired(HOLD ? row + R : row); });  // (the stage is free)
                if (!HOLD) release();
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    float2 z[4];
                    unpack(q_z[i], z);
                    const float2 m = both(-m1[i]), r = both(r1[i]), mv = both(-sums[i] * inv_h),
                                 mw = both(POST_LAYER ? -sums[R + i] * inv_h : 0.0f);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 hat = __fmul2_rn(POST_LAYER ? __fadd2_rn(z[e], m) : z[e], r);
                        const float2 wd =
                            POST_LAYER ? __ffma2_rn(w[e], g[i][e], mw) : __fmul2_rn(w[e], g[i][e]);
                        g[i][e] = __fmul2_rn(r, __ffma2_rn(hat, mv, wd));
                    }
                }
            } else if constexpr (!HOLD) {
                group_sync();
                release();
            }
#pragma unroll
            for (int i = 0; i < R; ++i)
                if (in && row + i < last)
                    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.dz[k[i]]) + off[i]) = pack(g[i]);
        }
    }

    if (tid == 0) {
        // copies that were not waited for land before the CTA leaves
        const uint32_t end = sm.under_way_end[group];
        for (uint32_t i = 0; i < NB_STAGES && end > 0; ++i) {
            const uint32_t r = sm.under_way[group] + i * R, pair = (r - sm.row0[group]) / R;
            if (r < end)
                drain_on(ptx::smem_u32(&sm.ring_bar[group][pair % NB_STAGES]), pair / NB_STAGES & 1u,
                     p.timeout_ns, p.err);
        }
    }
    __syncwarp();
    if constexpr (CL > 1) ptx::cluster_arrive_relaxed();

    // the block's column sums, the groups' added in order: one partial row for each vector
    ptx::griddep_launch_dependents();
    int v = 0;
    const int nv = (BEFORE ? 1 : 0) + (PRE_LAYER ? 1 : 0) + (POST_NORM ? 1 : 0) + (POST_LAYER ? 1 : 0);
    float* part = p.part + block * (nv + (gate && cut ? 1 : 0)) * p.h;
    float* meet = reinterpret_cast<float*>(ring_all);  // [group][columns]: the ring is done with
    auto put = [&](const float2 (&s)[4]) {
        float t[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = e & 1 ? s[e / 2].y : s[e / 2].x;
        if constexpr (G > 1) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; ++e) meet[group * (GT * 8) + e * GT + tid] = t[e];
            __syncthreads();
            if (group == 0) {
#pragma unroll
                for (int q = 1; q < G; ++q)
#pragma unroll
                    for (int e = 0; e < 8; ++e) t[e] += meet[q * (GT * 8) + e * GT + tid];
            }
        }
        if (in && group == 0) {
            float4* d = reinterpret_cast<float4*>(part + static_cast<long long>(v) * p.h + c);
            d[0] = make_float4(t[0], t[1], t[2], t[3]);
            d[1] = make_float4(t[4], t[5], t[6], t[7]);
        }
        ++v;
    };
    if constexpr (BEFORE) put(s_pre);
    if constexpr (PRE_LAYER) put(s_pre_b);
    if constexpr (POST_NORM) put(s_post);
    if constexpr (POST_LAYER) put(s_post_b);
    if constexpr (Z) {
        if (gate && cut) put(s_gate);
    }
    // No part may be on its way to a CTA that has left.  The last sums have all been waited
    // for, so none is; but a CTA that gave up is done before the others, which send until
    // their own wait for the same sum has run out.
    __syncwarp();
    if constexpr (CL > 1) ptx::cluster_wait();
}

// out[c] = sum over the blocks of a vector's partial rows, in block order within
// each of 8 row lanes, then the lanes in order.  blockIdx.y: the vector, then each
// gate whose rows are cut.
struct FinishParams {
    const float* part;
    float* out[5];               // the vectors' outputs; the last one dgate's
    long long h, ld, blocks;
    int vectors, blocks_per_seq;
};

__global__ void __launch_bounds__(256) nr_finish_kernel(const __grid_constant__ FinishParams p) {
    __shared__ float4 s[8][32];
    const int lane = threadIdx.x & 31, slot = threadIdx.x >> 5;
    const long long c = (static_cast<long long>(blockIdx.x) * 32 + lane) * 4;
    long long first = 0, n = p.blocks;
    int v = static_cast<int>(blockIdx.y);
    float* out;
    ptx::griddep_wait();
    if (v < p.vectors) {
        out = p.out[v];
    } else {
        const long long seq = v - p.vectors;
        first = seq * p.blocks_per_seq;
        n = p.blocks_per_seq;
        out = p.out[4] + seq * p.h;
        v = p.vectors;
    }
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < p.h) {
        const float* src = p.part + first * p.ld + v * p.h + c;
#pragma unroll 4
        for (long long b = slot; b < n; b += 8) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(src + b * p.ld));
            t.x += x.x;
            t.y += x.y;
            t.z += x.z;
            t.w += x.w;
        }
    }
    s[slot][lane] = t;
    __syncthreads();
    if (slot == 0 && c < p.h) {
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            const float4 x = s[i][lane];
            t.x += x.x;
            t.y += x.y;
            t.z += x.z;
            t.w += x.w;
        }
        *reinterpret_cast<float4*>(out + c) = t;
    }
}

constexpr int kDevices = 64;

// The kernel's attribute, set once a device.
template <int POST, int PRE, int CL, int G, int THREADS>
cudaError_t prepare(int& dev) {
    static int ready[kDevices] = {};
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    if (!__atomic_load_n(&ready[dev], __ATOMIC_ACQUIRE)) {
        e = cudaFuncSetAttribute(nr_backward_kernel<POST, PRE, CL, G, THREADS>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, NB_RING);
        if (e != cudaSuccess) return e;
        __atomic_store_n(&ready[dev], 1, __ATOMIC_RELEASE);
    }
    return cudaSuccess;
}

// attr: two of them, the cluster's first
void configure(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, long long blocks, int cl,
               int threads) {
    cfg.gridDim = dim3(static_cast<unsigned>(blocks * cl), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = NB_RING;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cl);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
}

template <int POST, int PRE, int CL, int G, int THREADS = NB_THREADS>
cudaError_t launch_rows(const NrBackwardParams& p, cudaStream_t st) {
    int dev = 0;
    const cudaError_t e = prepare<POST, PRE, CL, G, THREADS>(dev);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    configure(cfg, attr, p.blocks, CL, THREADS);
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, nr_backward_kernel<POST, PRE, CL, G, THREADS>, p);
}

// Clusters of CL CTAs that run at once (asked once a device; every variant of the kernel
// takes an SM for itself).
template <int CL>
cudaError_t resident(long long& clusters) {
    static int known[kDevices] = {};
    int dev = 0;
    cudaError_t e = prepare<NR_ABSENT, NR_PRE_RMS, CL, 1, NB_FEWER>(dev);
    if (e != cudaSuccess) return e;
    int n = __atomic_load_n(&known[dev], __ATOMIC_ACQUIRE);
    if (n == 0) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[2];
        configure(cfg, attr, 1, CL, NB_FEWER);
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&n, nr_backward_kernel<NR_ABSENT, NR_PRE_RMS, CL, 1, NB_FEWER>, &cfg);
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorInvalidConfiguration;
        __atomic_store_n(&known[dev], n, __ATOMIC_RELEASE);
    }
    clusters = n;
    return cudaSuccess;
}

template <int POST, int PRE>
cudaError_t launch(const NrBackwardParams& p, cudaStream_t st) {
    const int cl = cluster_of(p.h), g = groups_of(p.h);
    if (threads_of(p.h) == NB_FEWER) {
        if (cl == 2) return launch_rows<POST, PRE, 2, 1, NB_FEWER>(p, st);
        if (cl == 3) return launch_rows<POST, PRE, 3, 1, NB_FEWER>(p, st);
        if (cl == 4) return launch_rows<POST, PRE, 4, 1, NB_FEWER>(p, st);
        if (g == 1) return launch_rows<POST, PRE, 1, 1, NB_FEWER>(p, st);
        if (g == 2) return launch_rows<POST, PRE, 1, 2, NB_FEWER>(p, st);
        if (g == 3) return launch_rows<POST, PRE, 1, 3, NB_FEWER>(p, st);
        if (g == 4) return launch_rows<POST, PRE, 1, 4, NB_FEWER>(p, st);
        return launch_rows<POST, PRE, 1, 6, NB_FEWER>(p, st);
    }
    if (cl == 2) return launch_rows<POST, PRE, 2, 1>(p, st);
    if (cl == 4) return launch_rows<POST, PRE, 4, 1>(p, st);
    return g == 1 ? launch_rows<POST, PRE, 1, 1>(p, st) : launch_rows<POST, PRE, 1, 2>(p, st);
}

template <int POST>
cudaError_t launch_pre(const NrBackwardParams& p, int pre, cudaStream_t st) {
    if (pre == NR_PRE_RMS) return launch<POST, NR_PRE_RMS>(p, st);
    if (pre == NR_PRE_LAYER) return launch<POST, NR_PRE_LAYER>(p, st);
    if constexpr (POST != NR_ABSENT) return launch<POST, NR_NONE>(p, st);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t nr_plan(NrBackwardParams& p, int sm_count) {
    const int cl = cluster_of(p.h);
    long long blocks = sm_count;
    cudaError_t e = cudaSuccess;
    if (cl == 2) e = resident<2>(blocks);
    if (cl == 3) e = resident<3>(blocks);
    if (cl == 4) e = resident<4>(blocks);
    if (e != cudaSuccess) return e;
    blocks = std::max(1LL, std::min(blocks, static_cast<long long>(NR_MAX_UNITS / cl)));
    const long long groups = groups_of(p.h);
    p.seqs = p.T / p.gate_rows;
    p.blocks_per_seq = 0;
    p.rows_per_block = p.seqs_per_group = 0;
    if (p.seqs >= blocks * groups) {
        p.seqs_per_group = (p.seqs + blocks * groups - 1) / (blocks * groups);
        const long long used = (p.seqs + p.seqs_per_group - 1) / p.seqs_per_group;
        p.blocks = (used + groups - 1) / groups;
    } else {
        // at least a row pair for each group
        const long long most = std::max(1LL, p.gate_rows / (2 * groups));
        long long per = std::max(1LL, std::min(blocks / p.seqs, most));
        p.rows_per_block = (p.gate_rows + per - 1) / per;
        per = (p.gate_rows + p.rows_per_block - 1) / p.rows_per_block;
        p.blocks_per_seq = static_cast<int>(per);
        p.blocks = p.seqs * per;
    }
    return cudaSuccess;
}

size_t nr_partial_bytes(long long h) {
    // (gates that are cut may be more than the blocks that run at once, but fewer than
    // their groups)
    return static_cast<size_t>(NR_MAX_UNITS / cluster_of(h)) * groups_of(h) * 5 *
           static_cast<size_t>(h) * sizeof(float);
}

cudaError_t launch_nr_backward(const NrBackwardParams& p, int post, int pre, cudaStream_t st) {
    cudaError_t e = cudaErrorInvalidValue;
    switch (post) {
        case NR_ABSENT: e = launch_pre<NR_ABSENT>(p, pre, st); break;
        case NR_IDENTITY: e = launch_pre<NR_IDENTITY>(p, pre, st); break;
        case NR_POST_RMS: e = launch_pre<NR_POST_RMS>(p, pre, st); break;
        case NR_POST_LAYER: e = launch_pre<NR_POST_LAYER>(p, pre, st); break;
    }
    if (e != cudaSuccess) return e;
    const bool cut = post != NR_ABSENT && p.gate && p.blocks_per_seq > 0;
    FinishParams f = {};
    f.part = p.part;
    f.h = p.h;
    f.blocks = p.blocks;
    f.blocks_per_seq = p.blocks_per_seq;
    int v = 0;
    if (pre != NR_NONE) f.out[v++] = p.dpre_gamma;
    if (pre == NR_PRE_LAYER) f.out[v++] = p.dpre_beta;
    if (post >= NR_POST_RMS) f.out[v++] = p.dpost_gamma;
    if (post == NR_POST_LAYER) f.out[v++] = p.dpost_beta;
    f.vectors = v;
    f.out[4] = p.dgate;
    f.ld = static_cast<long long>(v + (cut ? 1 : 0)) * p.h;
    const long long rows = v + (cut ? p.seqs : 0);
    if (rows == 0) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.h / 4 + 31) / 32), static_cast<unsigned>(rows), 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, nr_finish_kernel, f);
}

}  // namespace tpmlp
