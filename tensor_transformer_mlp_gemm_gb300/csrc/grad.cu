// grad.cu -- the global norm of many gradients, and clipping by it (declared in
// include/tpmlp.h).
//
//   norm = sqrt(sum over all tensors of g^2)
//   out  = g * min(1, max_norm / (norm + 1e-6))
//
// What bounds it: HBM traffic.  Clipping reads every gradient twice and writes it once: the
// norm is not known before all have been read.  The second pass takes the tensors from the
// other end, so that what the first read last, which L2 (129 MB) still holds, comes first.
// Measured, fp32: 4096 x 16384 block (537 MB) the norm 79 us, 6.8 TB/s, all 249 us; 256 x 1024
// block (2 MB) 5.2 us, the latency of two launches.  In place and below the limit nothing is
// written, but everything is read twice all the same.
//
// Each tensor is cut into chunks, numbered over all tensors of a launch, at multiples of 16
// bytes of its address; CTA b takes chunks b, b + grid, ...  Which thread sums what, and in
// which order, depends on sizes and alignment alone, so the norm is the same in every run.  A
// thread adds the squares of up to 8 vectors of 16 bytes in fp32 where none can overflow or
// vanish against their sum, else in 64 bits; these sums are added in two fp32 parts (in 64 bits
// the smallest calls took twice as long), those of the CTAs in 64 bits.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "abi_internal.h"
#include "fp8_internal.h"
#include "ptx.cuh"
#include "tpmlp.h"
#include "two_sum.cuh"

#define TPMLP_API extern "C" __attribute__((visibility("default")))

namespace tpmlp {
namespace {

using namespace abi;

constexpr int GT = 512;          // threads
constexpr int G_PER_SM = 2;
constexpr int G_VECS = 8;        // vectors of a thread in the largest chunk
constexpr int G_CTAS = 1024;     // at most (partial sums of a launch)
constexpr int G_FEW = 32, G_MANY = 512;  // tensors in a launch's arguments
constexpr int64_t G_TENSORS = 65536;     // in a call
// Bytes at the end that the first pass leaves in L2 like any others; what lies before them is
// marked as the first to go.  (4096 x 16384 block in fp32: 87 us, all alike 93.)
constexpr unsigned G_KEEP = 50u << 20;
constexpr double G_EPS = 1e-6;

// The tensors of one launch.
template <int N>
struct Tensors {
    const void* in[N];
    void* out[N];
    long long count[N];
    unsigned first[N];     // chunks before it
    uint8_t type[N];
    int n, vecs;           // tensors; vectors of a thread in a chunk
    unsigned chunks;
};

__device__ __forceinline__ int element_bytes(int type) { return type == TPMLP_GRAD_F32 ? 4 : 2; }

// Chunk c of a launch: its tensor's bytes [begin, end) that lie in it, and where the tensor
// starts.  `base`, the address that vectors count from, is a multiple of 16.
struct Chunk {
    uintptr_t base, begin, end;
    int i, type;
};

template <int N>
__device__ __forceinline__ Chunk chunk_of(const Tensors<N>& p, unsigned c) {
    int lo = 0, hi = p.n - 1;  // the last tensor with first <= c
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.first[mid] <= c)
            lo = mid;
        else
            hi = mid - 1;
    }
    Chunk k;
    k.i = lo;
    k.type = p.type[lo];
    k.begin = reinterpret_cast<uintptr_t>(p.in[lo]);
    k.end = k.begin + static_cast<uintptr_t>(p.count[lo]) * element_bytes(k.type);
    k.base = (k.begin & ~static_cast<uintptr_t>(15)) +
             static_cast<uintptr_t>(c - p.first[lo]) * (static_cast<uintptr_t>(p.vecs) * GT * 16);
    return k;
}

// The vector at `a` of a chunk's tensor; what lies outside the tensor is zero and not read.
__device__ __forceinline__ uint4 load_vector(const Chunk& k, uintptr_t a) {
    if (a >= k.begin && a + 16 <= k.end) return __ldg(reinterpret_cast<const uint4*>(a));
    uint32_t w[4] = {0, 0, 0, 0};
    if (a + 16 > k.begin && a < k.end) {
        if (k.type == TPMLP_GRAD_F32) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (a + 4 * i >= k.begin && a + 4 * i < k.end) w[i] = __ldg(reinterpret_cast<const uint32_t*>(a) + i);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (a + 2 * i >= k.begin && a + 2 * i < k.end)
                    w[i / 2] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(a) + i)) << (16 * (i & 1));
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A load whose line is the first to leave L2.
__device__ __forceinline__ uint4 load_once(const uint4* a) {
    uint64_t policy;
    uint4 v;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    asm volatile("ld.global.nc.L1::no_allocate.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(a), "l"(policy));
    return v;
}

// This thread's vectors of a chunk.  In one that its tensor fills they are loaded without a
// test between them, all in flight before the first use.
template <int N>
__device__ __forceinline__ void load_chunk(const Tensors<N>& p, const Chunk& k, uint4 (&v)[G_VECS], bool keep) {
    const uintptr_t a = k.base + threadIdx.x * 16;
    const bool whole = k.base >= k.begin && k.base + static_cast<uintptr_t>(p.vecs) * (GT * 16) <= k.end;
    if (whole && p.vecs == G_VECS) {
        const uint4* src = reinterpret_cast<const uint4*>(a);
        if (keep) {
#pragma unroll
            for (int u = 0; u < G_VECS; ++u) v[u] = __ldg(src + u * GT);
        } else {
#pragma unroll
            for (int u = 0; u < G_VECS; ++u) v[u] = load_once(src + u * GT);
        }
        return;
    }
#pragma unroll
    for (int u = 0; u < G_VECS; ++u)
        v[u] = u < p.vecs ? load_vector(k, a + u * (GT * 16)) : make_uint4(0, 0, 0, 0);
}

// the two values of a word of bf16 or fp16
__device__ __forceinline__ float2 halves(uint32_t w, int type) {
    if (type == TPMLP_GRAD_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

__device__ __forceinline__ float squares(const uint4& v, int type) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (type == TPMLP_GRAD_F32) {
            const float x = __uint_as_float(w[j]);
            s = fmaf(x, x, s);
        } else {
            const float2 x = halves(w[j], type);
            s = fmaf(x.x, x.x, s);
            s = fmaf(x.y, x.y, s);
        }
    }
    return s;
}

__device__ __noinline__ double squares64(uint4 v, int type) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    double s = 0.0;
    for (int j = 0; j < 4; ++j) {
        float2 x = make_float2(__uint_as_float(w[j]), 0.0f);
        if (type != TPMLP_GRAD_F32) x = halves(w[j], type);
        s = fma(static_cast<double>(x.x), static_cast<double>(x.x), s);
        s = fma(static_cast<double>(x.y), static_cast<double>(x.y), s);
    }
    return s;
}

// Each value of a vector times f e.
__device__ __forceinline__ void scale(uint32_t (&w)[4], int type, float f, float e) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (type == TPMLP_GRAD_F32) {
            w[j] = __float_as_uint(__uint_as_float(w[j]) * f * e);
            continue;
        }
        const float2 y = halves(w[j], type);
        if (type == TPMLP_GRAD_BF16) {
            const __nv_bfloat162 z = __floats2bfloat162_rn(y.x * f * e, y.y * f * e);
            w[j] = *reinterpret_cast<const uint32_t*>(&z);
        } else {
            const __half2 z = __floats2half2_rn(y.x * f * e, y.y * f * e);
            w[j] = *reinterpret_cast<const uint32_t*>(&z);
        }
    }
}

template <int N>
__global__ void __launch_bounds__(GT, G_PER_SM)
    grad_squares_kernel(const __grid_constant__ Tensors<N> p, unsigned keep, double* __restrict__ partial) {
    __shared__ Sum s_sum[GT / 32];
    __shared__ double s_wide[GT / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    ptx::griddep_wait();
    // (after the wait: the kernel that clips may then read the gradients before its own)
    ptx::griddep_launch_dependents();
    Sum acc = {0.0f, 0.0f};
    double wide = 0.0;
    for (unsigned c = blockIdx.x; c < p.chunks; c += gridDim.x) {
        const Chunk k = chunk_of(p, c);
        uint4 v[G_VECS];
        load_chunk(p, k, v, c + keep >= p.chunks);
        float s = 0.0f;
        if (k.type == TPMLP_GRAD_F32) {
#pragma unroll
            for (int u = 0; u < G_VECS; ++u) s += squares(v[u], TPMLP_GRAD_F32);
        } else {
#pragma unroll
            for (int u = 0; u < G_VECS; ++u) s += squares(v[u], k.type);
        }
        // At most 64 squares: below 2^-126 each is off by at most 2^-150, 2^-34 of a sum of
        // 2^-110; and no number of sums up to 2^90 overflows.
        if (s >= 0x1p-110f && s <= 0x1p90f) {
            acc.add(s);
        } else {
            uint32_t any = 0;
#pragma unroll
            for (int u = 0; u < G_VECS; ++u) any |= v[u].x | v[u].y | v[u].z | v[u].w;
            if (any)
#pragma unroll
                for (int u = 0; u < G_VECS; ++u) wide += squares64(v[u], k.type);
        }
    }
    acc.over_lanes<16>();
    if (lane == 0) s_sum[warp] = acc;
    const bool any_wide = __syncthreads_or(wide != 0.0);  // (NaN too)
    if (any_wide) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) wide += __shfl_xor_sync(0xffffffffu, wide, o);
        if (lane == 0) s_wide[warp] = wide;
        __syncthreads();
    }
    if (warp == 0) {
        acc = s_sum[lane % (GT / 32)];
        acc.over_lanes<GT / 64>();
        if (lane == 0) {
            double sum = static_cast<double>(acc.hi) + static_cast<double>(acc.lo);
            if (any_wide)
                for (int w = 0; w < GT / 32; ++w) sum += s_wide[w];
            partial[blockIdx.x] = sum;
        }
    }
}

// The norm of all partial sums, and min(1, max_norm / (norm + 1e-6)) as f e, in every thread.  (In
// two factors where fp32 would lose digits: f stays normal down to quotients of 2^-266, where no
// product is.  A NaN stays.)
struct Norm {
    float norm, f, e;
};
__device__ __forceinline__ Norm norm_of(const double* partial, int n, float max_norm, Norm* s_norm) {
    if (threadIdx.x < 32) {
        double x = 0.0;
        for (int i = threadIdx.x; i < n; i += 32) x += partial[i];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (threadIdx.x == 0) {
            // (roots and quotients in 64 bits take a microsecond)
            const bool plain = x >= 1e-30 && x <= 1e30;
            float r = sqrtf(static_cast<float>(x)), f = max_norm / (r + static_cast<float>(G_EPS)), e = 1.0f;
            if (plain && (f >= 0x1p-100f || max_norm == 0.0f)) {
                f = fminf(f, 1.0f);
            } else {
                const double root = sqrt(x), q = max_norm / (root + G_EPS);
                const bool tiny = q < 0x1p-100, least = q < 0x1p-200;
                if (!plain) r = static_cast<float>(root);
                f = q >= 1.0 ? 1.0f : static_cast<float>(least ? q * 0x1p140 : tiny ? q * 0x1p64 : q);
                e = least ? 0x1p-140f : tiny ? 0x1p-64f : 1.0f;
            }
            *s_norm = Norm{r, f, e};
        }
    }
    __syncthreads();
    return *s_norm;
}

__global__ void __launch_bounds__(GT) grad_norm_kernel(const double* partial, int n, float* norm) {
    __shared__ Norm s_norm;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const Norm x = norm_of(partial, n, 0.0f, &s_norm);
    if (threadIdx.x == 0) *norm = x.norm;
}

template <int N>
__global__ void __launch_bounds__(GT, G_PER_SM)
    grad_scale_kernel(const __grid_constant__ Tensors<N> p, const double* __restrict__ partial, int n,
                      float max_norm, float* norm) {
    __shared__ Norm s_norm;
    ptx::griddep_launch_dependents();
    // the first chunk is on its way while the sums of squares end
    Chunk k = chunk_of(p, p.chunks - 1 - blockIdx.x);
    uint4 v[G_VECS];
    load_chunk(p, k, v, true);
    ptx::griddep_wait();
    const Norm x = norm_of(partial, n, max_norm, &s_norm);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = x.norm;
    const float f = x.f, e = x.e;
    for (unsigned r = blockIdx.x; r < p.chunks; r += gridDim.x) {
        if (r != blockIdx.x) {
            k = chunk_of(p, p.chunks - 1 - r);
            load_chunk(p, k, v, true);
        }
        const uintptr_t to = reinterpret_cast<uintptr_t>(p.out[k.i]) - k.begin;  // (wraps)
        if (to == 0 && f == 1.0f) continue;  // in place, and nothing changes
        const bool plain = to % 16 == 0 && k.base >= k.begin &&
                           k.base + static_cast<uintptr_t>(p.vecs) * (GT * 16) <= k.end;
#pragma unroll
        for (int u = 0; u < G_VECS; ++u) {
            const uintptr_t a = k.base + (u * GT + threadIdx.x) * 16;
            uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
            scale(w, k.type, f, e);
            if (u >= p.vecs) break;
            if (plain) {
                __stcs(reinterpret_cast<uint4*>(a + to), make_uint4(w[0], w[1], w[2], w[3]));
                continue;
            }
            if (a + 16 <= k.begin || a >= k.end) continue;
            if (a >= k.begin && a + 16 <= k.end && to % 16 == 0) {
                __stcs(reinterpret_cast<uint4*>(a + to), make_uint4(w[0], w[1], w[2], w[3]));
            } else if (k.type == TPMLP_GRAD_F32) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (a + 4 * i >= k.begin && a + 4 * i < k.end) reinterpret_cast<uint32_t*>(a + to)[i] = w[i];
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (a + 2 * i >= k.begin && a + 2 * i < k.end)
                        reinterpret_cast<uint16_t*>(a + to)[i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
            }
        }
    }
}

inline int host_bytes(int type) { return type == TPMLP_GRAD_F32 ? 4 : 2; }

tpmlp_status check_tensors(const tpmlp_grad_tensor* t, int64_t n, bool out) {
    if (n < 0 || (n > 0 && !t)) return TPMLP_ERR_INVALID_ARG;
    if (n > G_TENSORS) return TPMLP_ERR_UNSUPPORTED;
    for (int64_t i = 0; i < n; ++i) {
        if (t[i].count < 0 || t[i].type < TPMLP_GRAD_F32 || t[i].type > TPMLP_GRAD_F16)
            return TPMLP_ERR_INVALID_ARG;
        if (t[i].count == 0) continue;
        if (!t[i].grad || (out && !t[i].out)) return TPMLP_ERR_INVALID_ARG;
        if (t[i].count > (int64_t(1) << 40)) return TPMLP_ERR_UNSUPPORTED;
        const uintptr_t mask = host_bytes(t[i].type) - 1;
        if ((reinterpret_cast<uintptr_t>(t[i].grad) & mask) ||
            (out && (reinterpret_cast<uintptr_t>(t[i].out) & mask)))
            return TPMLP_ERR_UNSUPPORTED;
    }
    return TPMLP_OK;
}

template <typename K, typename... A>
cudaError_t launch(K kern, unsigned grid, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(GT, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Fills a launch's arguments with the tensors from *at on; false (and nothing changes): there
// are none left.
template <int N>
bool fill(Tensors<N>& p, const tpmlp_grad_tensor* t, int64_t n, int64_t* at, int vecs) {
    while (*at < n && t[*at].count == 0) ++*at;
    if (*at == n) return false;
    p.n = 0;
    p.vecs = vecs;
    unsigned long long chunks = 0;
    for (; *at < n && p.n < N; ++*at) {
        const tpmlp_grad_tensor& x = t[*at];
        if (x.count == 0) continue;
        const uint64_t bytes = (reinterpret_cast<uintptr_t>(x.grad) & 15) +
                               static_cast<uint64_t>(x.count) * host_bytes(x.type);
        const uint64_t chunk = static_cast<uint64_t>(vecs) * GT * 16, need = (bytes + chunk - 1) / chunk;
        if (chunks + need > 0x7FFFFFFFull) break;
        p.in[p.n] = x.grad;
        p.out[p.n] = x.out;
        p.count[p.n] = x.count;
        p.type[p.n] = static_cast<uint8_t>(x.type);
        p.first[p.n] = static_cast<unsigned>(chunks);
        chunks += need;
        ++p.n;
    }
    p.chunks = static_cast<unsigned>(chunks);
    return true;
}

// Tensors in a launch's arguments, vectors of a thread in a chunk, CTAs.
struct Plan {
    int per_launch, vecs, ctas;
};

Plan plan_of(const DeviceInfo& dev, const tpmlp_grad_tensor* t, int64_t n) {
    Plan p;
    int64_t filled = 0;
    uint64_t bytes = 0;
    for (int64_t i = 0; i < n; ++i) {
        filled += t[i].count > 0;
        bytes += static_cast<uint64_t>(t[i].count) * host_bytes(t[i].type);
    }
    p.per_launch = filled <= G_FEW ? G_FEW : G_MANY;
    p.ctas = dev.sm_count * G_PER_SM < G_CTAS ? dev.sm_count * G_PER_SM : G_CTAS;
    // chunks small enough that every CTA has one
    p.vecs = G_VECS;
    while (p.vecs > 1 && bytes < static_cast<uint64_t>(p.ctas) * p.vecs * GT * 16) p.vecs /= 2;
    return p;
}

template <int N>
tpmlp_status run(const Plan& plan, const tpmlp_grad_tensor* t, int64_t n, bool clip, float max_norm,
                 float* norm, double* partial, cudaStream_t st) {
    // where each launch's tensors start
    constexpr int kMost = static_cast<int>(G_TENSORS / G_MANY) + 1;
    int64_t start[kMost];
    int launches = 0;
    Tensors<N> p;
    for (int64_t at = 0;;) {
        const int64_t from = at;
        if (!fill(p, t, n, &at, plan.vecs)) break;
        if (launches == kMost) return TPMLP_ERR_UNSUPPORTED;
        start[launches++] = from;
    }
    const unsigned keep = clip ? G_KEEP / (static_cast<unsigned>(plan.vecs) * GT * 16) : 0;
    int sums = 0;
    for (int l = 0; l < launches; ++l) {
        int64_t at = start[l];
        if (launches > 1) fill(p, t, n, &at, plan.vecs);
        const unsigned grid = p.chunks < static_cast<unsigned>(plan.ctas) ? p.chunks : plan.ctas;
        TPMLP_CUDA(timed(TPMLP_KERNEL_BIAS_GRAD, 1, st,
                         [&] { return launch(grad_squares_kernel<N>, grid, st, p, keep, partial + sums); }));
        sums += static_cast<int>(grid);
    }
    const double* all = partial;
    if (!clip || launches == 0) {
        TPMLP_CUDA(timed(TPMLP_KERNEL_BIAS_GRAD, 1, st,
                         [&] { return launch(grad_norm_kernel, 1u, st, all, sums, norm); }));
        return TPMLP_OK;
    }
    // from the last launch back: `p` still holds its tensors
    for (int l = launches - 1; l >= 0; --l) {
        int64_t at = start[l];
        if (l < launches - 1) fill(p, t, n, &at, plan.vecs);
        const unsigned grid = p.chunks < static_cast<unsigned>(plan.ctas) ? p.chunks : plan.ctas;
        TPMLP_CUDA(timed(TPMLP_KERNEL_BIAS_GRAD, 1, st, [&] {
            return launch(grad_scale_kernel<N>, grid, st, p, all, sums, max_norm,
                          l == launches - 1 ? norm : static_cast<float*>(nullptr));
        }));
    }
    return TPMLP_OK;
}

tpmlp_status norm_and_clip(const tpmlp_grad_tensor* t, int64_t n, bool clip, float max_norm, void* norm,
                           void* workspace, cudaStream_t st) {
    TPMLP_TRY(check_tensors(t, n, clip));
    if (clip && !(max_norm >= 0.0f && std::isfinite(max_norm))) return TPMLP_ERR_INVALID_ARG;
    TPMLP_TRY(check_scale(norm));
    TPMLP_TRY(check_ptr(workspace));
    DeviceInfo* dev = nullptr;
    TPMLP_TRY(device_info(&dev));
    const Plan plan = plan_of(*dev, t, n);
    float* out = static_cast<float*>(norm);
    double* partial = static_cast<double*>(workspace);
    return plan.per_launch == G_FEW ? run<G_FEW>(plan, t, n, clip, max_norm, out, partial, st)
                                    : run<G_MANY>(plan, t, n, clip, max_norm, out, partial, st);
}

}  // namespace
}  // namespace tpmlp

using namespace tpmlp;
using namespace tpmlp::abi;

TPMLP_API size_t tpmlp_grad_workspace_bytes(int64_t tensors) {
    if (tensors < 0 || tensors > G_TENSORS) return 0;
    return (static_cast<size_t>(tensors) / G_MANY + 1) * G_CTAS * sizeof(double);
}

TPMLP_API tpmlp_status tpmlp_grad_norm(const tpmlp_grad_tensor* tensors, int64_t n, void* norm,
                                       void* workspace, void* stream) {
    return norm_and_clip(tensors, n, false, 0.0f, norm, workspace, static_cast<cudaStream_t>(stream));
}

TPMLP_API tpmlp_status tpmlp_grad_clip(const tpmlp_grad_tensor* tensors, int64_t n, float max_norm,
                                       void* norm, void* workspace, void* stream) {
    return norm_and_clip(tensors, n, true, max_norm, norm, workspace, static_cast<cudaStream_t>(stream));
}
