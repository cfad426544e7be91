// norm_forward.cu -- forward pass of the norms around a block (see
// norm_residual.cuh for the mathematics).
//
// What bounds it: HBM traffic, X and Z read and Out and Xn written once (8 bytes
// an element, 7 where Xn is 8-bit).  So both norms run in one pass over a row
// that stays in registers: a CTA takes a row at a time, a thread one or two
// 16-byte vectors of it, and a row costs one block sum for each rms and two for
// each layer norm (mean, then the squares of what is left: no cancellation).
// A CTA walks rows a grid apart; its columns' weights come from L1 at each row
// (kept in registers they spill or halve the rows in flight), and the row's token
// chunk and gate are stepped, not divided out: three 64-bit divisions a row and
// thread were 40 % of the instructions.
#include "fp8_cvt.cuh"
#include "norm_device.cuh"
#include "norm_residual.cuh"
#include "ptx.cuh"

namespace tpmlp {
namespace {

using namespace nr;

// Sum of v over the CTA, in a fixed order; `buf` alternates from call to call,
// so one barrier is enough.
__device__ __forceinline__ float block_sum(float v, float (*smem)[32], int& buf) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    v = warp_sum(v);
    if (lane == 0) smem[buf][warp] = v;
    __syncthreads();
    const float t = warp_sum(lane < warps ? smem[buf][lane] : 0.0f);
    buf ^= 1;
    return t;
}

// rms and layer statistics of the CTA's row (columns outside it hold zeros)
template <bool LAYER, int V>
__device__ __forceinline__ void row_stats(const float (&x)[V][8], const bool (&in)[V], float inv_h,
                                          float eps, float& mean, float& rstd, float (*smem)[32],
                                          int& buf) {
    mean = 0.0f;
    if (LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) s += x[j][i];
        mean = block_sum(s, smem, buf) * inv_h;
    }
    float q = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (in[j]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = x[j][i] - mean;
                q = fmaf(d, d, q);
            }
        }
    }
    rstd = rsqrtf(block_sum(q, smem, buf) * inv_h + eps);
}

template <int POST, int PRE, int V>
__global__ void __launch_bounds__(1024) nr_forward_kernel(const __grid_constant__ NrForwardParams p) {
    __shared__ float smem[2][32];
    int buf = 0;
    const float inv_h = 1.0f / static_cast<float>(p.h);
    int c[V];
    bool in[V];
    ptx::griddep_wait();
#pragma unroll
    for (int j = 0; j < V; ++j) {
        c[j] = (j * blockDim.x + threadIdx.x) * 8;
        in[j] = c[j] < p.h;
    }
    Stepper chunk(blockIdx.x, gridDim.x, p.rows_per_chunk), gate(blockIdx.x, gridDim.x, p.gate_rows);
    for (long long row = blockIdx.x; row < p.T; row += gridDim.x, chunk.step(), gate.step()) {
        const int k = chunk.q;
        const long long off = static_cast<long long>(chunk.r) * p.h;
        auto at = [&](const void* base, int j) {
            return reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + off + c[j]);
        };
        auto weight = [&](const void* w, int j, float (&f)[8]) {
            unpack(in[j] ? __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + c[j]))
                         : zero4(),
                   f);
        };
        uint4 xv[V], zv[V], gv[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            xv[j] = in[j] ? __ldg(at(p.x.p[k], j)) : zero4();
            if (POST != NR_ABSENT) zv[j] = in[j] ? __ldg(at(p.z.p[k], j)) : zero4();
            if (POST != NR_ABSENT && p.gate)
                gv[j] = in[j] ? __ldg(reinterpret_cast<const uint4*>(
                                    static_cast<const __nv_bfloat16*>(p.gate) +
                                    static_cast<long long>(gate.q) * p.h + c[j]))
                              : zero4();
        }
        float v[V][8];
        if constexpr (POST == NR_ABSENT) {
#pragma unroll
            for (int j = 0; j < V; ++j) unpack(xv[j], v[j]);
        } else {
            float mean = 0.0f, rstd = 1.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) unpack(zv[j], v[j]);
            if constexpr (POST >= NR_POST_RMS) {
                row_stats<POST == NR_POST_LAYER, V>(v, in, inv_h, p.eps, mean, rstd, smem, buf);
                if (threadIdx.x == 0 && p.stats) {
                    p.stats[row] = mean;
                    p.stats[p.T + row] = rstd;
                }
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float x[8], w[8], b[8];
                unpack(xv[j], x);
                if (POST >= NR_POST_RMS) {
                    weight(p.post_gamma, j, w);
                    if (POST == NR_POST_LAYER) weight(p.post_beta, j, b);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        v[j][i] = POST == NR_POST_LAYER ? fmaf((v[j][i] - mean) * rstd, w[i], b[i])
                                                        : v[j][i] * rstd * w[i];
                }
                if (p.gate) {
                    unpack(gv[j], w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[j][i] *= w[i];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] = fmaf(p.alpha, x[i], v[j][i]);
                const uint4 o = pack(v[j]);
                if (in[j]) *const_cast<uint4*>(at(p.out[k], j)) = o;
                unpack(o, v[j]);  // N_pre reads what was stored
            }
        }
        if constexpr (PRE != NR_NONE) {
            float mean, rstd;
            row_stats<PRE == NR_PRE_LAYER, V>(v, in, inv_h, p.eps, mean, rstd, smem, buf);
            if (threadIdx.x == 0 && p.stats) {
                p.stats[2 * p.T + row] = mean;
                p.stats[3 * p.T + row] = rstd;
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float w[8], b[8];
                weight(p.pre_gamma, j, w);
                if (PRE == NR_PRE_LAYER) weight(p.pre_beta, j, b);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[j][i] = PRE == NR_PRE_LAYER ? fmaf((v[j][i] - mean) * rstd, w[i], b[i])
                                                  : v[j][i] * rstd * w[i];
                const uint4 o = in[j] ? pack(v[j]) : zero4();
                if (in[j] && p.xn[0]) *const_cast<uint4*>(at(p.xn[k], j)) = o;
                if (p.q) {
                    // 16 threads hold a group of 128
                    uint32_t m = q8::largest(o);
#pragma unroll
                    for (int s = 8; s >= 1; s >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, s));
                    const q8::Scale sc = q8::scale_of(m, p.q_format);
                    if (in[j]) {
                        *reinterpret_cast<uint2*>(p.q + row * p.h + c[j]) = q8::cvt8(o, sc, p.q_format);
                        if ((threadIdx.x & 15) == 0) p.q_scale[(c[j] >> 7) * p.T + row] = sc.s;
                    }
                }
            }
        }
    }
    ptx::griddep_launch_dependents();
}

template <int POST, int PRE>
cudaError_t launch(const NrForwardParams& p, int sm_count, cudaStream_t st) {
    const long long vectors = p.h / 8;
    // two vectors a thread from 2048 columns on (256 threads), at most 1024 threads
    const int V = vectors <= 256 ? 1 : 2;
    int threads = 128;
    while (threads * V < vectors) threads *= 2;
    const long long resident = static_cast<long long>(sm_count) * (1024 / threads);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.T < resident ? p.T : resident), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return V == 1 ? cudaLaunchKernelEx(&cfg, nr_forward_kernel<POST, PRE, 1>, p)
                  : cudaLaunchKernelEx(&cfg, nr_forward_kernel<POST, PRE, 2>, p);
}

template <int POST>
cudaError_t launch_pre(const NrForwardParams& p, int pre, int sm_count, cudaStream_t st) {
    if (pre == NR_PRE_RMS) return launch<POST, NR_PRE_RMS>(p, sm_count, st);
    if (pre == NR_PRE_LAYER) return launch<POST, NR_PRE_LAYER>(p, sm_count, st);
    if constexpr (POST != NR_ABSENT) return launch<POST, NR_NONE>(p, sm_count, st);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_nr_forward(const NrForwardParams& p, int post, int pre, int sm_count,
                              cudaStream_t st) {
    switch (post) {
        case NR_ABSENT: return launch_pre<NR_ABSENT>(p, pre, sm_count, st);
        case NR_IDENTITY: return launch_pre<NR_IDENTITY>(p, pre, sm_count, st);
        case NR_POST_RMS: return launch_pre<NR_POST_RMS>(p, pre, sm_count, st);
        case NR_POST_LAYER: return launch_pre<NR_POST_LAYER>(p, pre, sm_count, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace tpmlp
