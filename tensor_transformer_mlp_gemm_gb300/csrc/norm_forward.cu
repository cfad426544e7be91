// norm_forward.cu -- forward pass of the norms around a block (see
// norm_residual.cuh for the mathematics).
//
// What bounds it: HBM traffic, X and Z read and Out and Xn written once (8 bytes
// an element, 7 where Xn is 8-bit).  So both norms run in one pass over a row
// that stays in registers: a CTA takes a row at a time, a thread one or two
// 16-byte vectors of it, and a row costs one block sum for each rms and two for
// each layer norm (mean, then the squares of what is left: no cancellation).
// One thread keeps bulk copies of the CTA's next two rows (X, Z, gate) under way into
// shared memory: loaded when they were needed, rows spent half their time waiting.
// What is left is bound by instructions, issued in 71 % of all cycles (ncu), so fp32
// values go two at a time (packed fma, 16384 x 4096 with 8-bit Xn 113 -> 98 us).
// A CTA walks rows a grid apart; its columns' weights come from L1 at each row (in
// registers they spill: layer norms 106 -> 139 us), and the row's token chunk and gate
// are stepped, not divided out: three 64-bit divisions a row and thread were 40 % of
// the instructions.
// A thread whose wait has expired waits no more and copies no more, but goes through the
// rows that are left with the others, so that no barrier misses it; what it has under way
// lands first.
// Measured, rms norms and a gate, cold caches, launch included: 16384 x 4096 in 88 us
// (6.1 TB/s), with 8-bit Xn 96; 8192 x 8192 88; 2048 x 12288 43; 16384 x 1024 29.  Back to back 16384 x 4096 84 (8-bit 86), 2048 x 12288 36, 16384 x 1024 24.
#include "fp8_cvt.cuh"
#include "norm_device.cuh"
#include "norm_residual.cuh"
#include "ptx.cuh"

namespace tpmlp {
namespace {

using namespace nr;

constexpr int NF_STAGES = 2;  // rows in the ring
static_assert(NF_STAGES == 2, "the other stage is the next row's");

// Sum of v over the CTA, in a fixed order; `buf` alternates from call to call,
// so one barrier is enough.
__device__ __forceinline__ float block_sum(float v, float (*smem)[32], int& buf) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    v = warp_sum(v);
    if (lane == 0) smem[buf][warp] = v;
    __syncthreads();
    float t = 0.0f;
    for (int w = 0; w < warps; w += 4) {
        const float4 f = *reinterpret_cast<const float4*>(&smem[buf][w]);
        t += (f.x + f.y) + (f.z + f.w);
    }
    buf ^= 1;
    return t;
}

// rms and layer statistics of the CTA's row (columns outside it hold zeros)
template <bool LAYER, int V>
__device__ __forceinline__ void row_stats(const float2 (&x)[V][4], const bool (&in)[V], float inv_h,
                                          float eps, float& mean, float& rstd, float (*smem)[32],
                                          int& buf) {
    mean = 0.0f;
    if (LAYER) {
        float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) s = __fadd2_rn(s, x[j][i]);
        mean = block_sum(s.x + s.y, smem, buf) * inv_h;
    }
    float2 q = make_float2(0.0f, 0.0f);
    const float2 m = make_float2(-mean, -mean);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (!LAYER || in[j]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 d = LAYER ? __fadd2_rn(x[j][i], m) : x[j][i];
                q = __ffma2_rn(d, d, q);
            }
        }
    }
    rstd = rsqrtf(block_sum(q.x + q.y, smem, buf) * inv_h + eps);
}

template <int POST, int PRE, int V, bool FULL>
__global__ void __launch_bounds__(1024) nr_forward_kernel(const __grid_constant__ NrForwardParams p) {
    extern __shared__ __align__(128) uint8_t ring[];  // [stage][X, Z, gate][row]
    __shared__ alignas(16) float smem[2][32];
    __shared__ alignas(8) uint64_t bar[NF_STAGES];
    int buf = 0;
    const uint32_t bytes = static_cast<uint32_t>(p.h) * 2;
    const uint32_t slot = (bytes + 127u) & ~127u;
    constexpr bool Z = POST != NR_ABSENT;
    const bool gated = Z && p.gate != nullptr;
    const uint32_t arrays = 1 + (Z ? 1 : 0) + (gated ? 1 : 0);
    if (threadIdx.x == 0) {
        for (int i = 0; i < NF_STAGES; ++i) ptx::mbar_init(ptx::smem_u32(&bar[i]), 1);
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    __syncthreads();
    const float inv_h = 1.0f / static_cast<float>(p.h);
    int c[V];
    bool in[V];
    ptx::griddep_wait();
#pragma unroll
    for (int j = 0; j < V; ++j) {
        c[j] = (j * blockDim.x + threadIdx.x) * 8;
        in[j] = FULL || c[j] < p.h;
    }
    Stepper chunk(blockIdx.x, gridDim.x, p.rows_per_chunk);
    Stepper copy_chunk(blockIdx.x, gridDim.x, p.rows_per_chunk), copy_gate(blockIdx.x, gridDim.x, p.gate_rows);
    // rows below this are copied; -1 once a wait of this thread has expired
    long long copy_end = p.stall < 0 ? p.T : min(p.T, blockIdx.x + static_cast<long long>(p.stall) * gridDim.x);
    // (thread 0, row after row of this CTA)
    auto copy_row = [&](int stage) {
        const uint32_t b = ptx::smem_u32(&bar[stage]);
        const uint32_t dst = ptx::smem_u32(ring) + static_cast<uint32_t>(stage) * 3 * slot;
        ptx::mbar_arrive_expect_tx(b, bytes * arrays);
        auto get = [&](uint32_t a, const void* base, long long row) {
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                    dst + a * slot),
                "l"(static_cast<const __nv_bfloat16*>(base) + row * p.h), "r"(bytes), "r"(b)
                : "memory");
        };
        get(0, p.x.p[copy_chunk.q], copy_chunk.r);
        if (Z) get(1, p.z.p[copy_chunk.q], copy_chunk.r);
        if (gated) get(2, p.gate, copy_gate.q);
        copy_chunk.step();
        copy_gate.step();
    };
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 0; i < NF_STAGES; ++i)
            if (blockIdx.x + static_cast<long long>(i) * gridDim.x < copy_end) copy_row(i);
    }
    int stage = 0;
    uint32_t phase = 0;
    for (long long row = blockIdx.x; row < p.T; row += gridDim.x, chunk.step()) {
        const uint32_t k = chunk.q;
        const long long off = static_cast<long long>(chunk.r) * p.h;
        auto at = [&](const void* base, int j) {
            return reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + off + c[j]);
        };
        auto bits = [&](const void* w, int j) {
            return in[j] ? __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + c[j]))
                         : zero4();
        };
        auto weight = [&](const void* w, int j, float2 (&f)[4]) { unpack(bits(w, j), f); };
        // With no block before there are registers to load the weights under the wait (layer
        // norms of 16384 x 4096 49 us, now 43; rms norms 43.5, now 42.3).
        uint4 early[V], early_b[V];
        if constexpr (POST == NR_ABSENT) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                early[j] = bits(p.pre_gamma, j);
                if (PRE == NR_PRE_LAYER) early_b[j] = bits(p.pre_beta, j);
            }
        }
        const uint8_t* src = ring + stage * 3 * slot;
        auto here = [&](int a, int j, float2 (&f)[4]) {
            unpack(in[j] ? *reinterpret_cast<const uint4*>(src + a * slot + c[j] * 2) : zero4(), f);
        };
        // the stage is read for the last time: the copy of the row NF_STAGES rows on
        auto next = [&] {
            if (threadIdx.x == 0 && row + static_cast<long long>(NF_STAGES) * gridDim.x < copy_end)
                copy_row(stage);
            if (++stage == NF_STAGES) {
                stage = 0;
                phase ^= 1u;
            }
        };
        {
            const uint32_t b = ptx::smem_u32(&bar[stage]);
            if (!ptx::mbar_try_wait(b, phase) && copy_end >= 0 &&
                !wait_on(b, phase, p.timeout_ns, p.err)) {
                if (threadIdx.x == 0) {
                    // what is under way: this row and the next one
                    const int other = stage ^ 1;
                    if (row < copy_end) drain_on(b, phase, p.timeout_ns, p.err);
                    if (row + gridDim.x < copy_end)
                        drain_on(ptx::smem_u32(&bar[other]), other ? phase : phase ^ 1u, p.timeout_ns, p.err);
                }
                copy_end = -1;
            }
        }
        float2 v[V][4];
        if constexpr (POST == NR_ABSENT) {
#pragma unroll
            for (int j = 0; j < V; ++j) here(0, j, v[j]);
        } else {
            float mean = 0.0f, rstd = 1.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) here(1, j, v[j]);
            if constexpr (POST >= NR_POST_RMS) {
                row_stats<POST == NR_POST_LAYER, V>(v, in, inv_h, p.eps, mean, rstd, smem, buf);
                if (threadIdx.x == 0 && p.stats) {
                    p.stats[row] = mean;
                    p.stats[p.T + row] = rstd;
                }
            }
            const float2 m2 = make_float2(-mean, -mean), r2 = make_float2(rstd, rstd);
            const float2 a2 = make_float2(p.alpha, p.alpha);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float2 x[4], w[4], b[4];
                here(0, j, x);
                if (POST >= NR_POST_RMS) {
                    weight(p.post_gamma, j, w);
                    if (POST == NR_POST_LAYER) weight(p.post_beta, j, b);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        v[j][i] = POST == NR_POST_LAYER
                                      ? __ffma2_rn(__fmul2_rn(__fadd2_rn(v[j][i], m2), r2), w[i], b[i])
                                      : __fmul2_rn(__fmul2_rn(v[j][i], r2), w[i]);
                }
                if (gated) {
                    here(2, j, w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[j][i] = __fmul2_rn(v[j][i], w[i]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) v[j][i] = __ffma2_rn(a2, x[i], v[j][i]);
                const uint4 o = pack(v[j]);
                if (in[j]) *const_cast<uint4*>(at(p.out[k], j)) = o;
                unpack(o, v[j]);  // N_pre reads what was stored
            }
        }
        if constexpr (PRE != NR_NONE) {
            float mean, rstd;
            row_stats<PRE == NR_PRE_LAYER, V>(v, in, inv_h, p.eps, mean, rstd, smem, buf);
            next();
            if (threadIdx.x == 0 && p.stats) {
                p.stats[2 * p.T + row] = mean;
                p.stats[3 * p.T + row] = rstd;
            }
            const float2 m2 = make_float2(-mean, -mean), r2 = make_float2(rstd, rstd);
            uint4 o[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float2 w[4], b[4];
                unpack(POST == NR_ABSENT ? early[j] : bits(p.pre_gamma, j), w);
                if (PRE == NR_PRE_LAYER) unpack(POST == NR_ABSENT ? early_b[j] : bits(p.pre_beta, j), b);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[j][i] = PRE == NR_PRE_LAYER
                                  ? __ffma2_rn(__fmul2_rn(__fadd2_rn(v[j][i], m2), r2), w[i], b[i])
                                  : __fmul2_rn(__fmul2_rn(v[j][i], r2), w[i]);
                o[j] = in[j] ? pack(v[j]) : zero4();
                if (in[j] && p.xn[0]) *const_cast<uint4*>(at(p.xn[k], j)) = o[j];
            }
            if (p.q) {
                // 16 threads hold a group of 128; two groups' maxima share a word
                uint32_t m[(V + 1) / 2];
#pragma unroll
                for (int j = 0; j < V; j += 2)
                    m[j / 2] = q8::largest(o[j]) | (j + 1 < V ? q8::largest(o[j + 1 < V ? j + 1 : j]) << 16 : 0u);
#pragma unroll
                for (int s = 8; s >= 1; s >>= 1)
#pragma unroll
                    for (int j = 0; j < (V + 1) / 2; ++j)
                        m[j] = __vmaxu2(m[j], __shfl_xor_sync(0xffffffffu, m[j], s));
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const q8::Scale sc = q8::scale_of(j & 1 ? m[j / 2] >> 16 : m[j / 2] & 0xFFFFu, p.q_format);
                    if (in[j]) {
                        *reinterpret_cast<uint2*>(p.q + row * p.h + c[j]) = q8::cvt8(o[j], sc, p.q_format);
                        if ((threadIdx.x & 15) == 0) p.q_scale[(c[j] >> 7) * p.T + row] = sc.s;
                    }
                }
            }
        } else {
            __syncthreads();
            next();
        }
    }
    ptx::griddep_launch_dependents();
}

template <int POST, int PRE>
cudaError_t launch(const NrForwardParams& p, int sm_count, cudaStream_t st) {
    const long long vectors = p.h / 8;
    // Two vectors a thread as soon as they fill four warps (a 2048-wide row of 16384 in
    // 49 us; with one vector a thread 59), whole warps in fours, at most 1024 threads.
    const int V = vectors <= 128 ? 1 : 2;
    const int threads = static_cast<int>((vectors + 128 * V - 1) / (128 * V)) * 128;
    const int smem = NF_STAGES * 3 * ((p.h * 2 + 127) / 128 * 128);
    // 64 registers a thread let 1024 threads onto an SM; their rings always fit
    const long long resident = static_cast<long long>(sm_count) * (1024 / threads);
    // a row that fills every thread needs no test of its columns (layer norms at 16384 x
    // 4096 113 -> 106 us)
    const bool full = static_cast<long long>(threads) * V * 8 == p.h;
    auto kernel = V == 1 ? (full ? nr_forward_kernel<POST, PRE, 1, true> : nr_forward_kernel<POST, PRE, 1, false>)
                         : (full ? nr_forward_kernel<POST, PRE, 2, true> : nr_forward_kernel<POST, PRE, 2, false>);
    const int variant = (V - 1) * 2 + (full ? 1 : 0);
    constexpr int kDevices = 64;
    static int ready[kDevices][4] = {};  // the kernel's attribute is set, per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    if (!__atomic_load_n(&ready[dev][variant], __ATOMIC_ACQUIRE)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 NF_STAGES * 3 * NR_MAX_H * 2);
        if (e != cudaSuccess) return e;
        __atomic_store_n(&ready[dev][variant], 1, __ATOMIC_RELEASE);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.T < resident ? p.T : resident), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
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
