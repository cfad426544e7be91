// norm_abi.cu -- the C ABI of the norms around a block (declared in
// include/tpmlp.h; the kernels are norm_forward.cu and norm_backward.cu).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "abi_internal.h"
#include "fp8_internal.h"
#include "norm_residual.cuh"
#include "tpmlp.h"

#define TPMLP_API extern "C" __attribute__((visibility("default")))

namespace tpmlp {
namespace {

using namespace abi;

inline bool kind_ok(int k) { return k == TPMLP_NORM_NONE || k == TPMLP_NORM_RMS || k == TPMLP_NORM_LAYER; }

tpmlp_status check_norm(const tpmlp_norm_params* d) {
    if (!d || d->tokens < 0 || d->hidden <= 0 || d->seq_chunks <= 0 || d->gate_rows < 0)
        return TPMLP_ERR_INVALID_ARG;
    if (!kind_ok(d->post) || !kind_ok(d->pre)) return TPMLP_ERR_INVALID_ARG;
    if (d->tokens % d->seq_chunks != 0) return TPMLP_ERR_INVALID_ARG;
    if (d->gate_rows > 0 && d->tokens % d->gate_rows != 0) return TPMLP_ERR_INVALID_ARG;
    if (!(d->eps >= 0.0f) || !std::isfinite(d->eps) || !std::isfinite(d->residual_scale))
        return TPMLP_ERR_INVALID_ARG;
    if (d->seq_chunks > NR_MAX_CHUNKS || d->hidden % 8 != 0 || d->hidden > NR_MAX_H ||
        d->tokens > (int64_t(1) << 31) - 1)
        return TPMLP_ERR_UNSUPPORTED;
    return TPMLP_OK;
}

// A weight that the kind uses, or does not: then it must be null.
tpmlp_status check_weight(const void* p, bool used) {
    if (used) return check_ptr(p);
    return p ? TPMLP_ERR_INVALID_ARG : TPMLP_OK;
}

// The same for an array of token chunks (`tokens` = 0: its entries are not looked at).
tpmlp_status check_chunks(const void* const* p, bool used, int64_t tokens, int n) {
    if (!used) return p ? TPMLP_ERR_INVALID_ARG : TPMLP_OK;
    if (!p) return TPMLP_ERR_INVALID_ARG;
    return tokens > 0 ? check_ptrs(p, n) : TPMLP_OK;
}

inline const void* const* in(void* const* p) { return reinterpret_cast<const void* const*>(p); }

int post_of(const tpmlp_norm_params& d, bool z) {
    if (!z) return NR_ABSENT;
    return d.post == TPMLP_NORM_RMS ? NR_POST_RMS : d.post == TPMLP_NORM_LAYER ? NR_POST_LAYER : NR_IDENTITY;
}

int pre_of(const tpmlp_norm_params& d) {
    return d.pre == TPMLP_NORM_RMS ? NR_PRE_RMS : d.pre == TPMLP_NORM_LAYER ? NR_PRE_LAYER : NR_NONE;
}

template <typename P>
void copy_chunks(P& dst, const void* const* src, int n) {
    if (src)
        for (int i = 0; i < n; ++i) dst.p[i] = src[i];
}

void copy_chunks(void** dst, void* const* src, int n) {
    if (src)
        for (int i = 0; i < n; ++i) dst[i] = src[i];
}

}  // namespace
}  // namespace tpmlp

using namespace tpmlp;
using namespace tpmlp::abi;

TPMLP_API size_t tpmlp_norm_workspace_bytes(const tpmlp_norm_params* params) {
    if (check_norm(params) != TPMLP_OK) return 0;
    return align256(nr_partial_bytes(params->hidden));
}

TPMLP_API tpmlp_status tpmlp_norm_forward(const tpmlp_norm_params* params, const void* const* X,
                                          const void* const* Z, const void* post_gamma,
                                          const void* post_beta, const void* gate,
                                          const void* pre_gamma, const void* pre_beta,
                                          void* const* Out, void* const* Xn, void* Xq, void* Xs,
                                          void* stats, void* stream) {
    TPMLP_TRY(check_norm(params));
    const tpmlp_norm_params& d = *params;
    const bool z = Z != nullptr, pre = d.pre != TPMLP_NORM_NONE;
    // without Z there is only the norm before
    if (!z && (d.post != TPMLP_NORM_NONE || !pre)) return TPMLP_ERR_INVALID_ARG;
    // (arrays of no tokens may be null: whether they are there is not looked at)
    if (d.tokens > 0) {
        if ((gate != nullptr) != (d.gate_rows > 0) || (gate && !z)) return TPMLP_ERR_INVALID_ARG;
        if ((Xq != nullptr) != (Xs != nullptr)) return TPMLP_ERR_INVALID_ARG;
        if (pre != (Xn != nullptr || Xq != nullptr)) return TPMLP_ERR_INVALID_ARG;
    }
    if (Xq && d.q_format != TPMLP_FP8_E4M3 && d.q_format != TPMLP_FP8_E5M2) return TPMLP_ERR_INVALID_ARG;
    if (Xq && d.hidden % 16 != 0) return TPMLP_ERR_UNSUPPORTED;
    const int n = d.seq_chunks;
    TPMLP_TRY(check_chunks(X, true, d.tokens, n));
    TPMLP_TRY(check_chunks(Z, z, d.tokens, n));
    TPMLP_TRY(check_chunks(in(Out), z, d.tokens, n));
    TPMLP_TRY(check_chunks(in(Xn), Xn != nullptr, d.tokens, n));
    TPMLP_TRY(check_weight(post_gamma, d.post != TPMLP_NORM_NONE));
    TPMLP_TRY(check_weight(post_beta, d.post == TPMLP_NORM_LAYER));
    TPMLP_TRY(check_weight(pre_gamma, pre));
    TPMLP_TRY(check_weight(pre_beta, d.pre == TPMLP_NORM_LAYER));
    if (d.tokens > 0) {
        if (gate) TPMLP_TRY(check_ptr(gate));
        if (Xq) {
            TPMLP_TRY(check_ptr(Xq));
            TPMLP_TRY(check_scale(Xs));
        }
        if (stats) TPMLP_TRY(check_scale(stats));
    }
    DeviceInfo* dev = nullptr;
    TPMLP_TRY(device_info(&dev));
    if (d.tokens == 0) return TPMLP_OK;
    NrForwardParams p;
    std::memset(&p, 0, sizeof(p));
    copy_chunks(p.x, X, n);
    copy_chunks(p.z, Z, n);
    copy_chunks(p.out, Out, n);
    copy_chunks(p.xn, Xn, n);
    p.post_gamma = post_gamma;
    p.post_beta = post_beta;
    p.pre_gamma = pre_gamma;
    p.pre_beta = pre_beta;
    p.gate = gate;
    p.q = static_cast<uint8_t*>(Xq);
    p.q_scale = static_cast<float*>(Xs);
    p.stats = static_cast<float*>(stats);
    p.T = d.tokens;
    p.rows_per_chunk = d.tokens / n;
    p.gate_rows = d.gate_rows > 0 ? d.gate_rows : d.tokens;
    p.h = static_cast<int>(d.hidden);
    p.q_format = d.q_format;
    p.eps = d.eps;
    p.alpha = d.residual_scale;
    p.err = dev->err;
    p.timeout_ns = g_timeout_ns;
    p.stall = g_stall;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    TPMLP_CUDA(timed(TPMLP_KERNEL_LAYERNORM_FWD, 1, st, [&] {
        return launch_nr_forward(p, post_of(d, z), pre_of(d), dev->sm_count, st);
    }));
    return TPMLP_OK;
}

TPMLP_API tpmlp_status tpmlp_norm_backward(const tpmlp_norm_params* params, const void* const* dOut,
                                           const void* const* dXn, const void* const* Z,
                                           const void* const* Out, const void* post_gamma,
                                           const void* post_beta, const void* gate,
                                           const void* pre_gamma, const void* stats,
                                           void* const* dX, void* const* dZ, void* dpost_gamma,
                                           void* dpost_beta, void* dgate, void* dpre_gamma,
                                           void* dpre_beta, void* workspace, void* stream) {
    TPMLP_TRY(check_norm(params));
    const tpmlp_norm_params& d = *params;
    const bool z = Z != nullptr, pre = d.pre != TPMLP_NORM_NONE;
    const bool post = d.post != TPMLP_NORM_NONE;
    if (!z && (post || !pre)) return TPMLP_ERR_INVALID_ARG;
    if (d.tokens > 0 && ((gate != nullptr) != (d.gate_rows > 0) || (gate && !z)))
        return TPMLP_ERR_INVALID_ARG;
    if (!pre && !dOut) return TPMLP_ERR_INVALID_ARG;
    const int n = d.seq_chunks;
    TPMLP_TRY(check_chunks(dOut, dOut != nullptr, d.tokens, n));
    TPMLP_TRY(check_chunks(dXn, pre, d.tokens, n));
    TPMLP_TRY(check_chunks(Z, z, d.tokens, n));
    TPMLP_TRY(check_chunks(Out, pre, d.tokens, n));
    TPMLP_TRY(check_chunks(in(dX), true, d.tokens, n));
    TPMLP_TRY(check_chunks(in(dZ), z, d.tokens, n));
    TPMLP_TRY(check_weight(post_gamma, post));
    TPMLP_TRY(check_weight(post_beta, d.post == TPMLP_NORM_LAYER));
    TPMLP_TRY(check_weight(pre_gamma, pre));
    TPMLP_TRY(check_weight(dpost_gamma, post));
    TPMLP_TRY(check_weight(dpost_beta, d.post == TPMLP_NORM_LAYER));
    TPMLP_TRY(check_weight(dpre_gamma, pre));
    TPMLP_TRY(check_weight(dpre_beta, d.pre == TPMLP_NORM_LAYER));
    if (d.tokens > 0) {
        TPMLP_TRY(check_weight(gate, gate != nullptr));
        TPMLP_TRY(check_weight(dgate, gate != nullptr));
        if (post || pre) TPMLP_TRY(check_scale(stats));
        TPMLP_TRY(check_ptr(workspace));
    }
    DeviceInfo* dev = nullptr;
    TPMLP_TRY(device_info(&dev));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (d.tokens == 0) {
        const size_t bytes = static_cast<size_t>(d.hidden) * sizeof(float);
        for (void* g : {dpost_gamma, dpost_beta, dpre_gamma, dpre_beta})
            if (g) TPMLP_CUDA(cudaMemsetAsync(g, 0, bytes, st));
        return TPMLP_OK;
    }
    NrBackwardParams p;
    std::memset(&p, 0, sizeof(p));
    copy_chunks(p.dout, dOut, n);
    copy_chunks(p.dxn, dXn, n);
    copy_chunks(p.z, Z, n);
    copy_chunks(p.out, Out, n);
    copy_chunks(p.dx, dX, n);
    copy_chunks(p.dz, dZ, n);
    p.post_gamma = post_gamma;
    p.post_beta = post_beta;
    p.pre_gamma = pre_gamma;
    p.gate = gate;
    p.stats = static_cast<const float*>(stats);
    p.part = static_cast<float*>(workspace);
    p.dpost_gamma = static_cast<float*>(dpost_gamma);
    p.dpost_beta = static_cast<float*>(dpost_beta);
    p.dpre_gamma = static_cast<float*>(dpre_gamma);
    p.dpre_beta = static_cast<float*>(dpre_beta);
    p.dgate = static_cast<float*>(dgate);
    p.T = d.tokens;
    p.rows_per_chunk = d.tokens / n;
    p.gate_rows = d.gate_rows > 0 ? d.gate_rows : d.tokens;
    p.h = static_cast<int>(d.hidden);
    p.alpha = d.residual_scale;
    p.err = dev->err;
    p.timeout_ns = g_timeout_ns;
    p.stall = g_stall;
    TPMLP_CUDA(nr_plan(p, dev->sm_count));
    // the second launch adds up what the row blocks left, if anything
    const bool sums = post || pre || (gate && p.blocks_per_seq > 0);
    TPMLP_CUDA(timed(TPMLP_KERNEL_LAYERNORM_BWD, sums ? 2 : 1, st, [&] {
        return launch_nr_backward(p, post_of(d, z), pre_of(d), st);
    }));
    return TPMLP_OK;
}
