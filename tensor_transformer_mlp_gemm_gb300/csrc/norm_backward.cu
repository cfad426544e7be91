// norm_backward.cu -- backward pass of the norms around a block (see
// norm_residual.cuh for the mathematics).
//
// What bounds it: HBM traffic, dOut, dXn, Z and Out read and dX and dZ written once
// (12 bytes an element).  So everything a row gives, its two data gradients and its
// share of up to five column sums, comes from one pass: a thread keeps the sums of
// its 8 columns in registers over all rows of its block, and the next row's vectors
// are loaded while this one is worked on.
//
// 512 threads hold 4096 columns.  Wider rows take a cluster of 2 or 4 CTAs side by
// side, whose row sums meet in each other's shared memory: each warp sends its part
// to every CTA, counted on that CTA's mbarrier, and every warp adds all parts in the
// same order.  (A cluster barrier instead waits for the row's own loads and stores
// too: 6600 clocks a row, measured at 917 x 9000.)  A row has two such sums, as dZ
// needs dX's row sum first.
// The column sums of a block go to a partial row, and a second kernel adds the blocks
// in order; a gate whose rows lie in one block is finished there and then.  No atomics.
#include <algorithm>

#include "gemm_params.h"
#include "norm_device.cuh"
#include "norm_residual.cuh"
#include "ptx.cuh"

namespace tpmlp {
namespace {

using namespace nr;

constexpr int NB_THREADS = 512;
constexpr int NB_COLS = NB_THREADS * 8;  // columns of one CTA
constexpr int NB_WARPS = NB_THREADS / 32;
constexpr int NB_MAX_CLUSTER = 4;
static_assert(NB_COLS * NB_MAX_CLUSTER >= NR_MAX_H, "a cluster holds the widest row");

int cluster_of(long long h) { return h <= NB_COLS ? 1 : h <= 2 * NB_COLS ? 2 : 4; }

// A float into a CTA of the cluster, its four bytes counted on that CTA's mbarrier.
__device__ __forceinline__ void send(uint32_t addr, float v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(
                     addr),
                 "r"(__float_as_uint(v)), "r"(bar)
                 : "memory");
}

// What the row sums of a CTA need: the parts [buf][value][CTA * 16 + warp], two
// mbarriers, and the limit of a wait.
struct Sums {
    float part[2][2][NB_MAX_CLUSTER * NB_WARPS];
    alignas(8) uint64_t bar[2];
};
struct SumState {
    int buf;
    uint32_t phase[2];
    int rank;
    unsigned long long timeout_ns;
    unsigned* err;
};

// Sums of one or two values over the row (all CTAs of the cluster), in a fixed order.
// The buffers alternate: a part of the next but one sum can only be sent once every
// warp has sent its part of the next, and so has read this one.
template <int CL, bool TWO>
__device__ __forceinline__ void row_sum(float& a, float& b, Sums& sm, SumState& st) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, buf = st.buf;
    a = warp_sum(a);
    if (TWO) b = warp_sum(b);
    if constexpr (CL == 1) {
        if (lane == 0) {
            sm.part[buf][0][warp] = a;
            if (TWO) sm.part[buf][1][warp] = b;
        }
        __syncthreads();
    } else {
        const uint32_t bar = ptx::smem_u32(&sm.bar[buf]);
        if (threadIdx.x == 0)
            ptx::mbar_arrive_expect_tx(bar, CL * NB_WARPS * (TWO ? 8 : 4));
        if (lane < CL) {
            const uint32_t to = static_cast<uint32_t>(lane);
            const uint32_t rbar = ptx::mapa_shared(bar, to);
            send(ptx::mapa_shared(ptx::smem_u32(&sm.part[buf][0][st.rank * NB_WARPS + warp]), to), a, rbar);
            if (TWO)
                send(ptx::mapa_shared(ptx::smem_u32(&sm.part[buf][1][st.rank * NB_WARPS + warp]), to), b,
                     rbar);
        }
        __syncwarp();
        if (!ptx::mbar_try_wait(bar, st.phase[buf])) {
            const uint64_t t0 = ptx::globaltimer_ns();
            while (!ptx::mbar_try_wait(bar, st.phase[buf])) {
                if (ptx::globaltimer_ns() - t0 > st.timeout_ns) {
                    atomicOr(st.err, ERR_EPILOGUE);
                    break;
                }
            }
        }
        st.phase[buf] ^= 1u;
    }
    float s = 0.0f, t = 0.0f;
#pragma unroll
    for (int i = 0; i < (CL * NB_WARPS + 31) / 32; ++i) {
        if (i * 32 + lane < CL * NB_WARPS) {
            s += sm.part[buf][0][i * 32 + lane];
            if (TWO) t += sm.part[buf][1][i * 32 + lane];
        }
    }
    a = warp_sum(s);
    if (TWO) b = warp_sum(t);
    st.buf ^= 1;
}

template <int POST, int PRE, int CL>
__global__ void __launch_bounds__(NB_THREADS, 1)
    nr_backward_kernel(const __grid_constant__ NrBackwardParams p) {
    constexpr bool Z = POST != NR_ABSENT, POST_NORM = POST >= NR_POST_RMS;
    constexpr bool POST_LAYER = POST == NR_POST_LAYER, PRE_LAYER = PRE == NR_PRE_LAYER;
    __shared__ Sums sm;
    const int rank = CL == 1 ? 0 : static_cast<int>(ptx::cluster_ctarank());
    SumState ss = {0, {0, 0}, rank, p.timeout_ns, p.err};
    const long long block = blockIdx.x / CL;
    const float inv_h = 1.0f / static_cast<float>(p.h);
    const int c = (rank * NB_THREADS + threadIdx.x) * 8;
    const bool in = c < p.h;
    if constexpr (CL > 1) {
        if (threadIdx.x == 0) {
            ptx::mbar_init(ptx::smem_u32(&sm.bar[0]), 1);
            ptx::mbar_init(ptx::smem_u32(&sm.bar[1]), 1);
            ptx::fence_mbar_init();
        }
        __syncwarp();
        ptx::cluster_sync();  // all of the cluster's barriers exist
    }
    ptx::griddep_wait();

    auto weight = [&](const void* w) {
        return in ? __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + c)) : zero4();
    };
    const uint4 w1 = POST_NORM ? weight(p.post_gamma) : zero4();
    const uint4 b1 = POST_LAYER ? weight(p.post_beta) : zero4();
    const uint4 w2 = PRE != NR_NONE ? weight(p.pre_gamma) : zero4();

    // this block's rows
    long long row, last, next_gate;
    if (p.blocks_per_seq > 0) {
        const long long seq = block / p.blocks_per_seq;
        const long long first = seq * p.gate_rows;
        row = first + (block - seq * p.blocks_per_seq) * p.rows_per_block;
        next_gate = first + p.gate_rows;  // the whole block lies before it
        last = min(row + p.rows_per_block, next_gate);
    } else {
        row = block * p.seqs_per_block * p.gate_rows;
        next_gate = row + p.gate_rows;
        last = min(row + p.seqs_per_block * p.gate_rows, p.T);
    }
    const bool gate = Z && p.gate != nullptr;

    float s_pre[PRE != NR_NONE ? 8 : 1] = {}, s_pre_b[PRE_LAYER ? 8 : 1] = {};
    float s_post[POST_NORM ? 8 : 1] = {}, s_post_b[POST_LAYER ? 8 : 1] = {};
    float s_gate[Z ? 8 : 1] = {};
    uint4 gate_v = zero4();

    struct Row {
        uint4 dout, dxn, z, out;
        float m1, r1, m2, r2;
    };
    auto load = [&](long long r, Row& d) {
        const int k = static_cast<int>(r / p.rows_per_chunk);
        const long long off = (r - k * p.rows_per_chunk) * p.h + c;
        auto get = [&](const void* base) {
            return in ? __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + off))
                      : zero4();
        };
        d.dout = p.dout.p[0] ? get(p.dout.p[k]) : zero4();
        if (PRE != NR_NONE) {
            d.dxn = get(p.dxn.p[k]);
            d.out = get(p.out.p[k]);
            d.m2 = PRE_LAYER ? __ldg(p.stats + 2 * p.T + r) : 0.0f;
            d.r2 = __ldg(p.stats + 3 * p.T + r);
        }
        if (Z) d.z = get(p.z.p[k]);
        if (POST_NORM) {
            d.m1 = POST_LAYER ? __ldg(p.stats + r) : 0.0f;
            d.r1 = __ldg(p.stats + p.T + r);
        }
    };
    auto load_gate = [&](long long r) {
        if (gate)
            gate_v = in ? __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.gate) +
                                                               r / p.gate_rows * p.h + c))
                        : zero4();
    };
    auto finish_gate = [&](float* dst) {
        if (in) {
            reinterpret_cast<float4*>(dst + c)[0] = make_float4(s_gate[0], s_gate[1], s_gate[2], s_gate[3]);
            reinterpret_cast<float4*>(dst + c)[1] = make_float4(s_gate[4], s_gate[5], s_gate[6], s_gate[7]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s_gate[i] = 0.0f;
    };

    Row cur;
    if (row < last) {
        load(row, cur);
        if constexpr (Z) load_gate(row);
    }
    while (row < last) {
        Row nxt;
        if (row + 1 < last) load(row + 1, nxt);
        const int k = static_cast<int>(row / p.rows_per_chunk);
        const long long off = (row - k * p.rows_per_chunk) * p.h + c;
        float g[8];
        unpack(cur.dout, g);
        if constexpr (PRE != NR_NONE) {
            float d[8], v[8], w[8];
            unpack(cur.dxn, d);
            unpack(cur.out, v);
            unpack(w2, w);
            float sv = 0.0f, sw = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = in ? (v[i] - cur.m2) * cur.r2 : 0.0f;
                s_pre[i] = fmaf(d[i], v[i], s_pre[i]);
                if (PRE_LAYER) s_pre_b[i] += d[i];
                w[i] *= d[i];
                sv = fmaf(w[i], v[i], sv);
                if (PRE_LAYER) sw += w[i];
            }
            row_sum<CL, PRE_LAYER>(sv, sw, sm, ss);
            const float mv = sv * inv_h, mw = PRE_LAYER ? sw * inv_h : 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = fmaf(cur.r2, w[i] - mw - v[i] * mv, g[i]);
        }
        {
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = Z ? p.alpha * g[i] : g[i];
            if (in) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.dx[k]) + off) = pack(o);
        }
        if constexpr (Z) {
            float z[8], w[8], b[8], t[8];
            unpack(cur.z, z);
            unpack(w1, w);
            unpack(b1, b);
            if (POST_NORM) {
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] = in ? (z[i] - cur.m1) * cur.r1 : 0.0f;
            }
            if (gate) {
                unpack(gate_v, t);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float u = POST_NORM ? (POST_LAYER ? fmaf(z[i], w[i], b[i]) : z[i] * w[i]) : z[i];
                    s_gate[i] = fmaf(g[i], u, s_gate[i]);
                    g[i] *= t[i];
                }
            }
            if constexpr (POST_NORM) {
                float sv = 0.0f, sw = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s_post[i] = fmaf(g[i], z[i], s_post[i]);
                    if (POST_LAYER) s_post_b[i] += g[i];
                    w[i] *= g[i];
                    sv = fmaf(w[i], z[i], sv);
                    if (POST_LAYER) sw += w[i];
                }
                row_sum<CL, POST_LAYER>(sv, sw, sm, ss);
                const float mv = sv * inv_h, mw = POST_LAYER ? sw * inv_h : 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) g[i] = cur.r1 * (w[i] - mw - z[i] * mv);
            }
            if (in) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.dz[k]) + off) = pack(g);
        }
        ++row;
        cur = nxt;
        if constexpr (Z) {
            if (gate && p.blocks_per_seq == 0 && row == next_gate) {
                // the gate's last row: its sum is complete
                finish_gate(p.dgate + (row - 1) / p.gate_rows * p.h);
                next_gate += p.gate_rows;
                if (row < last) load_gate(row);
            }
        }
    }

    // this block's column sums: one partial row for each vector
    int v = 0;
    const int nv = (PRE != NR_NONE) + PRE_LAYER + POST_NORM + POST_LAYER;
    float* part = p.part + block * (nv + (gate && p.blocks_per_seq > 0)) * p.h;
    auto put = [&](const float* s) {
        if (in) {
            float4* d = reinterpret_cast<float4*>(part + static_cast<long long>(v) * p.h + c);
            d[0] = make_float4(s[0], s[1], s[2], s[3]);
            d[1] = make_float4(s[4], s[5], s[6], s[7]);
        }
        ++v;
    };
    if constexpr (PRE != NR_NONE) put(s_pre);
    if constexpr (PRE_LAYER) put(s_pre_b);
    if constexpr (POST_NORM) put(s_post);
    if constexpr (POST_LAYER) put(s_post_b);
    if constexpr (Z) {
        if (gate && p.blocks_per_seq > 0) put(s_gate);
    }
    ptx::griddep_launch_dependents();
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

template <int POST, int PRE, int CL>
cudaError_t launch_rows(const NrBackwardParams& p, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.blocks * CL), 1, 1);
    cfg.blockDim = dim3(NB_THREADS, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CL;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CL > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, nr_backward_kernel<POST, PRE, CL>, p);
}

template <int POST, int PRE>
cudaError_t launch(const NrBackwardParams& p, cudaStream_t st) {
    const int cl = cluster_of(p.h);
    return cl == 1 ? launch_rows<POST, PRE, 1>(p, st)
           : cl == 2 ? launch_rows<POST, PRE, 2>(p, st)
                     : launch_rows<POST, PRE, 4>(p, st);
}

template <int POST>
cudaError_t launch_pre(const NrBackwardParams& p, int pre, cudaStream_t st) {
    if (pre == NR_PRE_RMS) return launch<POST, NR_PRE_RMS>(p, st);
    if (pre == NR_PRE_LAYER) return launch<POST, NR_PRE_LAYER>(p, st);
    if constexpr (POST != NR_ABSENT) return launch<POST, NR_NONE>(p, st);
    return cudaErrorInvalidValue;
}

}  // namespace

void nr_plan(NrBackwardParams& p, int sm_count) {
    const long long units = std::max(1, std::min(sm_count, NR_MAX_UNITS) / cluster_of(p.h));
    p.seqs = p.T / p.gate_rows;
    if (p.seqs >= units) {
        p.blocks_per_seq = 0;
        p.seqs_per_block = (p.seqs + units - 1) / units;
        p.blocks = (p.seqs + p.seqs_per_block - 1) / p.seqs_per_block;
        p.rows_per_block = 0;
    } else {
        long long per = std::min(units / p.seqs, p.gate_rows);
        p.rows_per_block = (p.gate_rows + per - 1) / per;
        per = (p.gate_rows + p.rows_per_block - 1) / p.rows_per_block;
        p.blocks_per_seq = static_cast<int>(per);
        p.blocks = p.seqs * per;
        p.seqs_per_block = 0;
    }
}

size_t nr_partial_bytes(long long h) {
    return static_cast<size_t>(NR_MAX_UNITS / cluster_of(h)) * 5 * static_cast<size_t>(h) *
           sizeof(float);
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
