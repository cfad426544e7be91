// fp8_linear.cu -- the C ABI of the 8-bit calls (declared in include/tpmlp.h):
// quantisation with a scale for each group of 128, and the tensor-parallel
// linear layers on 8-bit operands.
//
//   column parallel  forward   Y_i = X.W_i + b_i      X row groups, W_i blocks; t groups
//                    backward  dX = sum_i dY_i.W_i^T  dY_i row groups, W_i blocks; t k-segments
//                              dW_i = X^T.dY_i        X and dY_i column groups; t groups
//                              db = column sums of dY
//   row parallel     forward   Z = sum_i X_i.W_i + b  t k-segments
//                    backward  dX_i = dZ.W_i^T        t groups
//                              dW_i = X_i^T.dZ        t groups
//
// A weight is read as it lies, [in, out]: MN-major by the forward pass, K-major
// by the backward pass, with its block scales indexed one way or the other.
// Contractions over tokens need groups along tokens, so the backward pass makes
// both groupings of dY (and the bias gradient's partial sums) in one read.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "abi_internal.h"
#include "colsum.cuh"
#include "fp8_gemm.cuh"
#include "fp8_internal.h"
#include "fp8_quant.cuh"
#include "tpmlp.h"

#define TPMLP_API extern "C" __attribute__((visibility("default")))

namespace tpmlp {
namespace {

using namespace abi;

static_assert(TPMLP_FP8_E4M3 == FP8_E4M3 && TPMLP_FP8_E5M2 == FP8_E5M2, "format codes");

enum class Split { Column, Row };

struct Lin {
    int T, in, out, t, chunks, Tc, shard;
};

inline long long up128(long long n) { return (n + FP8_GROUP - 1) / FP8_GROUP; }

tpmlp_status check_fp8_dims(const tpmlp_linear_dims* d, Split k) {
    if (!d) return TPMLP_ERR_INVALID_ARG;
    if (d->tokens < 0 || d->in_features <= 0 || d->out_features <= 0 || d->t <= 0 ||
        d->seq_chunks <= 0)
        return TPMLP_ERR_INVALID_ARG;
    const int64_t split = k == Split::Column ? d->out_features : d->in_features;
    const int64_t other = k == Split::Column ? d->in_features : d->out_features;
    if (split % d->t != 0 || d->tokens % d->seq_chunks != 0) return TPMLP_ERR_INVALID_ARG;
    if (d->t > kMaxShards || d->seq_chunks > kMaxShards) return TPMLP_ERR_UNSUPPORTED;
    if ((split / d->t) % 16 != 0 || other % 16 != 0) return TPMLP_ERR_UNSUPPORTED;
    // the products round each up to tiles of 256 in 32 bits
    const int64_t lim = (int64_t(1) << 31) - 256;
    if (d->tokens > lim || d->in_features > lim || d->out_features > lim)
        return TPMLP_ERR_UNSUPPORTED;
    if (d->seq_chunks > 1 && (d->tokens / d->seq_chunks) % FP8_GROUP != 0)
        return TPMLP_ERR_UNSUPPORTED;
    return TPMLP_OK;
}

inline bool format_ok(int f) { return f == TPMLP_FP8_E4M3 || f == TPMLP_FP8_E5M2; }

tpmlp_status check_formats(const tpmlp_fp8_formats* f) {
    if (!f || !format_ok(f->x) || !format_ok(f->w) || !format_ok(f->dy)) return TPMLP_ERR_INVALID_ARG;
    return TPMLP_OK;
}

Lin lin_of(const tpmlp_linear_dims& d, Split k) {
    Lin s;
    s.T = static_cast<int>(d.tokens);
    s.in = static_cast<int>(d.in_features);
    s.out = static_cast<int>(d.out_features);
    s.t = d.t;
    s.chunks = d.seq_chunks;
    s.Tc = s.T / s.chunks;
    s.shard = (k == Split::Column ? s.out : s.in) / s.t;
    return s;
}

// Backward scratch: dY by rows and by columns (8-bit and scales) and the
// bias gradient's partial sums.  Sized for either split.
struct Scratch {
    size_t q_rows, s_rows, q_cols, s_cols, sums, total;
};

Scratch scratch_layout(const tpmlp_linear_dims& d) {
    const size_t T = static_cast<size_t>(d.tokens), out = static_cast<size_t>(d.out_features);
    // a column shard has its own row groups: up to one more for each shard
    const size_t row_groups = static_cast<size_t>(up128(d.out_features)) + d.t;
    const size_t col_groups = static_cast<size_t>(up128(d.tokens));
    Scratch s;
    s.q_rows = 0;
    s.s_rows = s.q_rows + align256(T * out);
    s.q_cols = s.s_rows + align256(row_groups * align256(T * sizeof(float)));
    s.s_cols = s.q_cols + align256(T * out);
    s.sums = s.s_cols + align256(col_groups * out * sizeof(float));
    s.total = s.sums + align256(col_groups * out * sizeof(float)) + 256;
    return s;
}

// One operand of a product: its matrices (one, or one per group or K segment),
// each [outer, inner] row-major, and their scales.
struct Operand {
    const void* const* q;
    const void* const* s;
    int n;
    int part;
    int mn;        // MN-major: [K, rows]
};

struct Product {
    int M, N, K, groups, ksegs;
    Operand a, b;
    long long sa_kb, sb_kb, sb_n;
    int a_format, b_format;
    const void* bias;
    int out_kind;
    void* const* out;
    int nout;          // outputs: one per group, or one per token chunk
    int chunk_rows;    // > 0: rows per token chunk
};

bool encode_operand(CUtensorMap* m, const Operand& o, int K, int rows, int box) {
    if (!(o.mn ? encode_bytes(m, o.q[0], rows, K, 128) : encode_bytes(m, o.q[0], K, rows, box)))
        return false;
    for (int i = 1; i < o.n; ++i) {
        m[i] = m[0];
        if (!set_address(&m[i], o.q[i])) return false;
    }
    return true;
}

tpmlp_status run_product(const DeviceInfo* dev, const Product& d, int kind, cudaStream_t st) {
    Fp8GemmParams p;
    std::memset(&p, 0, sizeof(p));
    int few = 0;  // rows of a tile of the few-rows kernel
    if (d.out_kind == F8_BF16_BLOCK) TPMLP_CUDA(fp8_small_rows(d.M, d.N, d.groups, few));
    if (!encode_operand(p.a_map, d.a, d.K, d.M, few ? few : 128) ||
        !encode_operand(p.b_map, d.b, d.K, d.N, 128))
        return TPMLP_ERR_UNSUPPORTED;
    for (int i = 0; i < d.a.n; ++i) p.sa[i] = static_cast<const float*>(d.a.s[i]);
    for (int i = 0; i < d.b.n; ++i) p.sb[i] = static_cast<const float*>(d.b.s[i]);
    for (int i = 0; i < d.nout; ++i) p.out[i] = d.out[i];
    p.sa_kb = d.sa_kb;
    p.sb_kb = d.sb_kb;
    p.sb_n = d.sb_n;
    p.M = d.M;
    p.N = d.N;
    p.K = d.K;
    p.groups = d.groups;
    p.ksegs = d.ksegs;
    p.a_part = d.a.part;
    p.b_part = d.b.part;
    p.a_mn = d.a.mn;
    p.b_mn = d.b.mn;
    const long long mt = (static_cast<long long>(d.M) + 255) / 256;
    const long long nt = (static_cast<long long>(d.N) + 255) / 256;
    if (mt * nt > 0x7FFFFFFFLL / d.groups) return TPMLP_ERR_UNSUPPORTED;
    p.mtiles = static_cast<int>(mt);
    p.ntiles = static_cast<int>(nt);
    p.total_tiles = static_cast<int>(mt * nt * d.groups);
    p.band = p.mtiles < kBand ? p.mtiles : kBand;
    p.chunk_rows = d.chunk_rows;
    p.bias = d.bias;
    // the few-rows kernel has the weights for the instruction's A
    const int fa = few ? d.b_format : d.a_format, fb = few ? d.a_format : d.b_format;
    p.ab_format = (static_cast<uint32_t>(fa) << 7) | (static_cast<uint32_t>(fb) << 10);
    p.err = dev->err;
    p.timeout_ns = g_timeout_ns;
    p.stall = g_stall;
    TPMLP_CUDA(timed(kind, 1, st, [&] {
        return few ? launch_fp8_small(p, few, st) : launch_fp8_gemm(p, d.out_kind, st);
    }));
    return TPMLP_OK;
}

// dY [n parts] quantised both ways into the workspace, with the bias gradient.
struct QuantGrad {
    void* q_rows[kMaxShards];
    void* s_rows[kMaxShards];
    void* q_cols[kMaxShards];
    void* s_cols[kMaxShards];
};

tpmlp_status quantize_grad(const Lin& s, Split k, int format, const void* const* dY,
                           const tpmlp_linear_dims& dims, uint8_t* ws, void* db, QuantGrad* o,
                           cudaStream_t st) {
    const Scratch L = scratch_layout(dims);
    const size_t T = static_cast<size_t>(s.T);
    Fp8QuantParams q;
    std::memset(&q, 0, sizeof(q));
    q.fmt_rows = q.fmt_cols = format;
    float* sums = reinterpret_cast<float*>(ws + L.sums);
    q.sums_ld = s.out;
    q.ld = s.T;
    if (k == Split::Column) {
        // t matrices [T, oi], side by side in db
        q.parts = s.t;
        q.rows = s.T;
        q.cols = s.shard;
        const size_t groups = static_cast<size_t>(up128(s.shard));
        for (int i = 0; i < s.t; ++i) {
            q.q_rows[i] = ws + L.q_rows + i * T * s.shard;
            q.q_cols[i] = ws + L.q_cols + i * T * s.shard;
            q.s_rows[i] = reinterpret_cast<float*>(ws + L.s_rows + i * groups * align256(T * 4));
            q.s_cols[i] = reinterpret_cast<float*>(ws + L.s_cols) +
                          i * static_cast<size_t>(up128(s.T)) * s.shard;
            q.sums[i] = sums + static_cast<size_t>(i) * s.shard;
        }
    } else {
        // token chunks of one matrix [T, out]
        q.parts = s.chunks;
        q.rows = s.Tc;
        q.cols = s.out;
        for (int j = 0; j < s.chunks; ++j) {
            const size_t r0 = static_cast<size_t>(j) * s.Tc, g0 = r0 / FP8_GROUP;
            q.q_rows[j] = ws + L.q_rows + r0 * s.out;
            q.q_cols[j] = ws + L.q_cols + r0 * s.out;
            q.s_rows[j] = reinterpret_cast<float*>(ws + L.s_rows) + r0;
            q.s_cols[j] = reinterpret_cast<float*>(ws + L.s_cols) + g0 * s.out;
            q.sums[j] = sums + g0 * s.out;
        }
    }
    for (int i = 0; i < q.parts; ++i) q.src[i] = dY[i];
    TPMLP_CUDA(timed(TPMLP_KERNEL_SP_COPY, 1, st, [&] {
        return launch_fp8_quant(q, FP8_Q_ROWS | FP8_Q_COLS | FP8_Q_SUMS, st);
    }));
    TPMLP_CUDA(timed(TPMLP_KERNEL_BIAS_GRAD, 1, st, [&] {
        return launch_colsum_f32(sums, up128(s.T), s.out, s.out, static_cast<float*>(db), st);
    }));
    for (int i = 0; i < q.parts; ++i) {
        o->q_rows[i] = q.q_rows[i];
        o->s_rows[i] = q.s_rows[i];
        o->q_cols[i] = q.q_cols[i];
        o->s_cols[i] = q.s_cols[i];
    }
    return TPMLP_OK;
}

tpmlp_status zero_grads(const Lin& s, Split k, void* const* dW, void* db, cudaStream_t st) {
    const size_t other = static_cast<size_t>(k == Split::Column ? s.in : s.out);
    for (int i = 0; i < s.t; ++i)
        TPMLP_CUDA(cudaMemsetAsync(dW[i], 0, other * s.shard * sizeof(float), st));
    TPMLP_CUDA(cudaMemsetAsync(db, 0, static_cast<size_t>(s.out) * sizeof(float), st));
    return TPMLP_OK;
}

tpmlp_status forward(Split k, const tpmlp_linear_dims* dims, const tpmlp_fp8_formats* f,
                     const void* const* Xq, const void* const* Xs, const void* const* Wq,
                     const void* const* Ws, const void* b, void* const* Y, void* workspace,
                     cudaStream_t st) {
    TPMLP_TRY(check_fp8_dims(dims, k));
    TPMLP_TRY(check_formats(f));
    const Lin s = lin_of(*dims, k);
    const bool col = k == Split::Column;
    const int nx = col ? 1 : s.t, ny = col ? s.t : s.chunks;
    TPMLP_TRY(check_ptr(b));
    TPMLP_TRY(check_ptrs(Wq, s.t));
    TPMLP_TRY(check_scales(Ws, s.t));
    if (s.T > 0) {
        TPMLP_TRY(check_ptrs(Xq, nx));
        TPMLP_TRY(check_scales(Xs, nx));
        TPMLP_TRY(check_ptrs(reinterpret_cast<const void* const*>(Y), ny));
        TPMLP_TRY(check_ptr(workspace));
    }
    DeviceInfo* dev = nullptr;
    TPMLP_TRY(device_info(&dev));
    if (s.T == 0) return TPMLP_OK;
    Product p;
    p.M = s.T;
    p.N = col ? s.shard : s.out;
    p.K = col ? s.in : s.shard;
    p.groups = col ? s.t : 1;
    p.ksegs = col ? 1 : s.t;
    p.a = Operand{Xq, Xs, nx, col ? F8_SINGLE : F8_KSEG, 0};
    p.b = Operand{Wq, Ws, s.t, col ? F8_GROUP : F8_KSEG, 1};
    p.sa_kb = s.T;
    p.sb_kb = up128(p.N);
    p.sb_n = 1;
    p.a_format = f->x;
    p.b_format = f->w;
    p.bias = b;
    p.out_kind = F8_BF16_BLOCK;
    p.out = Y;
    p.nout = ny;
    p.chunk_rows = col ? 0 : s.Tc;
    return run_product(dev, p, TPMLP_KERNEL_LINEAR_FWD, st);
}

tpmlp_status backward(Split k, const tpmlp_linear_dims* dims, const tpmlp_fp8_formats* f,
                      const void* const* dY, const void* const* Xq, const void* const* Xs,
                      const void* const* Wq, const void* const* Ws, void* const* dX,
                      void* const* dW, void* db, void* workspace, cudaStream_t st) {
    TPMLP_TRY(check_fp8_dims(dims, k));
    TPMLP_TRY(check_formats(f));
    const Lin s = lin_of(*dims, k);
    const bool col = k == Split::Column;
    const int nx = col ? 1 : s.t, ndy = col ? s.t : s.chunks, ndx = col ? s.chunks : s.t;
    TPMLP_TRY(check_ptrs(Wq, s.t));
    TPMLP_TRY(check_scales(Ws, s.t));
    TPMLP_TRY(check_ptrs(reinterpret_cast<const void* const*>(dW), s.t));
    TPMLP_TRY(check_ptr(db));
    if (s.T > 0) {
        TPMLP_TRY(check_ptrs(dY, ndy));
        TPMLP_TRY(check_ptrs(Xq, nx));
        TPMLP_TRY(check_scales(Xs, nx));
        TPMLP_TRY(check_ptrs(reinterpret_cast<const void* const*>(dX), ndx));
        TPMLP_TRY(check_ptr(workspace));
    }
    DeviceInfo* dev = nullptr;
    TPMLP_TRY(device_info(&dev));
    if (s.T == 0) return zero_grads(s, k, dW, db, st);
    QuantGrad g;
    TPMLP_TRY(quantize_grad(s, k, f->dy, dY, *dims, static_cast<uint8_t*>(workspace), db, &g, st));
    const int ng = col ? s.t : 1;  // quantised gradients: per shard, or one
    {
        // dX: M = T, N = in (or ii per group), K = oi per segment (or out)
        Product p;
        p.M = s.T;
        p.N = col ? s.in : s.shard;
        p.K = col ? s.shard : s.out;
        p.groups = col ? 1 : s.t;
        p.ksegs = col ? s.t : 1;
        p.a = Operand{g.q_rows, g.s_rows, ng, col ? F8_KSEG : F8_SINGLE, 0};
        p.b = Operand{Wq, Ws, s.t, col ? F8_KSEG : F8_GROUP, 0};
        p.sa_kb = s.T;
        p.sb_kb = 1;
        p.sb_n = up128(p.K);
        p.a_format = f->dy;
        p.b_format = f->w;
        p.bias = nullptr;
        p.out_kind = F8_BF16_BLOCK;
        p.out = dX;
        p.nout = ndx;
        p.chunk_rows = col ? s.Tc : 0;
        TPMLP_TRY(run_product(dev, p, TPMLP_KERNEL_LINEAR_DGRAD, st));
    }
    {
        // dW_i: M = in (or ii), N = oi (or out), K = T
        Product p;
        p.M = col ? s.in : s.shard;
        p.N = col ? s.shard : s.out;
        p.K = s.T;
        p.groups = s.t;
        p.ksegs = 1;
        p.a = Operand{Xq, Xs, nx, col ? F8_SINGLE : F8_GROUP, 1};
        p.b = Operand{g.q_cols, g.s_cols, ng, col ? F8_GROUP : F8_SINGLE, 1};
        p.sa_kb = p.M;
        p.sb_kb = p.N;
        p.sb_n = 0;
        p.a_format = f->x;
        p.b_format = f->dy;
        p.bias = nullptr;
        p.out_kind = F8_F32_VECTOR;
        p.out = dW;
        p.nout = s.t;
        p.chunk_rows = 0;
        TPMLP_TRY(run_product(dev, p, TPMLP_KERNEL_LINEAR_WGRAD, st));
    }
    return TPMLP_OK;
}

}  // namespace
}  // namespace tpmlp

using namespace tpmlp;
using namespace tpmlp::abi;

TPMLP_API tpmlp_status tpmlp_fp8_quantize(const tpmlp_fp8_quant* d, const void* const* src,
                                          void* const* q_rows, void* const* s_rows,
                                          void* const* q_cols, void* const* s_cols, void* stream) {
    if (!d || d->rows < 0 || d->cols <= 0 || d->parts <= 0) return TPMLP_ERR_INVALID_ARG;
    if (!format_ok(d->rows_format) || !format_ok(d->cols_format)) return TPMLP_ERR_INVALID_ARG;
    const bool rows = q_rows || s_rows, cols = q_cols || s_cols;
    if (!rows && !cols) return TPMLP_ERR_INVALID_ARG;
    if (rows && d->scale_ld < d->rows) return TPMLP_ERR_INVALID_ARG;
    const int64_t lim = (int64_t(1) << 31) - 1;
    if (d->parts > FP8_MAX_PARTS || d->cols % 16 != 0 || d->rows > lim || d->cols > lim)
        return TPMLP_ERR_UNSUPPORTED;
    const int n = d->parts;
    if (d->rows > 0) {
        TPMLP_TRY(check_ptrs(src, n));
        if (rows) {
            TPMLP_TRY(check_ptrs(reinterpret_cast<const void* const*>(q_rows), n));
            TPMLP_TRY(check_scales(reinterpret_cast<const void* const*>(s_rows), n));
        }
        if (cols) {
            TPMLP_TRY(check_ptrs(reinterpret_cast<const void* const*>(q_cols), n));
            TPMLP_TRY(check_scales(reinterpret_cast<const void* const*>(s_cols), n));
        }
    }
    DeviceInfo* dev = nullptr;
    TPMLP_TRY(device_info(&dev));
    if (d->rows == 0) return TPMLP_OK;
    Fp8QuantParams p;
    std::memset(&p, 0, sizeof(p));
    for (int i = 0; i < n; ++i) {
        p.src[i] = src[i];
        if (rows) {
            p.q_rows[i] = q_rows[i];
            p.s_rows[i] = static_cast<float*>(s_rows[i]);
        }
        if (cols) {
            p.q_cols[i] = q_cols[i];
            p.s_cols[i] = static_cast<float*>(s_cols[i]);
        }
    }
    p.rows = d->rows;
    p.cols = d->cols;
    p.ld = d->scale_ld;
    p.parts = n;
    p.fmt_rows = d->rows_format;
    p.fmt_cols = d->cols_format;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int mode = (rows ? FP8_Q_ROWS : 0) | (cols ? FP8_Q_COLS : 0);
    TPMLP_CUDA(timed(TPMLP_KERNEL_SP_COPY, 1, st, [&] { return launch_fp8_quant(p, mode, st); }));
    return TPMLP_OK;
}

TPMLP_API tpmlp_status tpmlp_fp8_quantize_weight(const void* W, int64_t in, int64_t out, int format,
                                                 void* q, void* s, void* stream) {
    if (in <= 0 || out <= 0 || !format_ok(format)) return TPMLP_ERR_INVALID_ARG;
    const int64_t lim = (int64_t(1) << 31) - 1;
    if (out % 16 != 0 || in > lim || out > lim) return TPMLP_ERR_UNSUPPORTED;
    TPMLP_TRY(check_ptr(W));
    TPMLP_TRY(check_ptr(q));
    TPMLP_TRY(check_scale(s));
    DeviceInfo* dev = nullptr;
    TPMLP_TRY(device_info(&dev));
    Fp8QuantParams p;
    std::memset(&p, 0, sizeof(p));
    p.src[0] = W;
    p.q_cols[0] = q;
    p.s_cols[0] = static_cast<float*>(s);
    p.rows = in;
    p.cols = out;
    p.parts = 1;
    p.fmt_cols = format;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    TPMLP_CUDA(timed(TPMLP_KERNEL_SP_COPY, 1, st,
                     [&] { return launch_fp8_quant(p, FP8_Q_BLOCK, st); }));
    return TPMLP_OK;
}

TPMLP_API size_t tpmlp_fp8_linear_workspace_bytes(const tpmlp_linear_dims* dims) {
    if (check_fp8_dims(dims, Split::Column) != TPMLP_OK && check_fp8_dims(dims, Split::Row) != TPMLP_OK)
        return 0;
    return scratch_layout(*dims).total;
}

TPMLP_API tpmlp_status tpmlp_fp8_column_linear_forward(
    const tpmlp_linear_dims* dims, const tpmlp_fp8_formats* formats, const void* Xq, const void* Xs,
    const void* const* Wq_shards, const void* const* Ws_shards, const void* b, void* const* Y_shards,
    void* workspace, void* stream) {
    return forward(Split::Column, dims, formats, &Xq, &Xs, Wq_shards, Ws_shards, b, Y_shards,
                   workspace, static_cast<cudaStream_t>(stream));
}

TPMLP_API tpmlp_status tpmlp_fp8_row_linear_forward(
    const tpmlp_linear_dims* dims, const tpmlp_fp8_formats* formats, const void* const* Xq_shards,
    const void* const* Xs_shards, const void* const* Wq_shards, const void* const* Ws_shards,
    const void* b, void* const* Z, void* workspace, void* stream) {
    return forward(Split::Row, dims, formats, Xq_shards, Xs_shards, Wq_shards, Ws_shards, b, Z,
                   workspace, static_cast<cudaStream_t>(stream));
}

TPMLP_API tpmlp_status tpmlp_fp8_column_linear_backward(
    const tpmlp_linear_dims* dims, const tpmlp_fp8_formats* formats, const void* const* dY_shards,
    const void* Xq, const void* Xs, const void* const* Wq_shards, const void* const* Ws_shards,
    void* const* dX, void* const* dW_shards, void* db, void* workspace, void* stream) {
    return backward(Split::Column, dims, formats, dY_shards, &Xq, &Xs, Wq_shards, Ws_shards, dX,
                    dW_shards, db, workspace, static_cast<cudaStream_t>(stream));
}

TPMLP_API tpmlp_status tpmlp_fp8_row_linear_backward(
    const tpmlp_linear_dims* dims, const tpmlp_fp8_formats* formats, const void* const* dZ,
    const void* const* Xq_shards, const void* const* Xs_shards, const void* const* Wq_shards,
    const void* const* Ws_shards, void* const* dX_shards, void* const* dW_shards, void* db,
    void* workspace, void* stream) {
    return backward(Split::Row, dims, formats, dZ, Xq_shards, Xs_shards, Wq_shards, Ws_shards,
                    dX_shards, dW_shards, db, workspace, static_cast<cudaStream_t>(stream));
}
