// fp4_linear.cu -- the C ABI of the 4-bit calls (declared in include/tpmlp.h):
// quantisation and back, and the tensor-parallel linear layers on 4-bit operands.
//
//   column parallel  forward   Y_i = X.W_i + b_i      X rows, W_i cols; t groups
//                    backward  dX = sum_i dY_i.W_i^T  dY_i rows, W_i rows; t k-segments
//                              dW_i = X^T.dY_i        X cols, dY_i cols; t groups
//                              db = column sums of dY
//   row parallel     forward   Z = sum_i X_i.W_i + b  t k-segments
//                    backward  dX_i = dZ.W_i^T        t groups
//                              dW_i = X_i^T.dZ        t groups
//
// "rows" is a matrix quantised along its features, "cols" one quantised along its rows and
// transposed: each product's operands are grouped along the axis that it sums over and lie
// along it.  X and dY come in bf16 and are quantised on the way, X both ways in one read
// where the caller keeps it for the backward pass, dY with the bias gradient's sums.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "abi_internal.h"
#include "fp4_gemm.cuh"
#include "fp8_internal.h"
#include "tpmlp.h"

#define TPMLP_API extern "C" __attribute__((visibility("default")))

namespace tpmlp {
namespace {

using namespace abi;

static_assert(static_cast<int>(TPMLP_FP4_MX) == FP4_MX && static_cast<int>(TPMLP_FP4_NV) == FP4_NV, "format codes");

enum class Split { Column, Row };

struct Lin {
    int T, in, out, t, chunks, Tc, shard;
};

inline long long up128(long long n) { return (n + 127) / 128; }

tpmlp_status check_fp4_dims(const tpmlp_linear_dims* d, Split k) {
    if (!d) return TPMLP_ERR_INVALID_ARG;
    if (d->tokens < 0 || d->in_features <= 0 || d->out_features <= 0 || d->t <= 0 ||
        d->seq_chunks <= 0)
        return TPMLP_ERR_INVALID_ARG;
    const int64_t split = k == Split::Column ? d->out_features : d->in_features;
    const int64_t other = k == Split::Column ? d->in_features : d->out_features;
    if (split % d->t != 0 || d->tokens % d->seq_chunks != 0) return TPMLP_ERR_INVALID_ARG;
    if (d->t > kMaxShards || d->seq_chunks > kMaxShards) return TPMLP_ERR_UNSUPPORTED;
    if ((split / d->t) % 32 != 0 || other % 32 != 0) return TPMLP_ERR_UNSUPPORTED;
    // the products round each up to tiles of 256 in 32 bits
    const int64_t lim = (int64_t(1) << 31) - 256;
    if (d->tokens > lim || d->in_features > lim || d->out_features > lim)
        return TPMLP_ERR_UNSUPPORTED;
    if (d->seq_chunks > 1 && (d->tokens / d->seq_chunks) % 128 != 0) return TPMLP_ERR_UNSUPPORTED;
    return TPMLP_OK;
}

inline bool format_ok(int f) { return f == TPMLP_FP4_MX || f == TPMLP_FP4_NV; }

// A tensor's scale: nv has one, mx none.
tpmlp_status check_tensor_scale(const void* s, int format) {
    if (format == TPMLP_FP4_MX) return s ? TPMLP_ERR_INVALID_ARG : TPMLP_OK;
    return check_scale(s);
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

// `n` matrices [R, K] in 4 bits, side by side.
struct Packed {
    uint8_t* q[kMaxShards];
    uint8_t* s[kMaxShards];
    long long k;  // of rows that the parts share (joined), else 0
};

inline size_t packed_bytes(int n, long long R, long long K, int format) {
    return align256(static_cast<size_t>(n) * fp4_packed_bytes(R, K)) +
           static_cast<size_t>(n) * fp4_scale_bytes(R, K, format);
}

// Lays them out at `at`, which moves on.
Packed place(uint8_t*& at, int n, long long R, long long K, int format) {
    Packed o = {};
    uint8_t* s = at + align256(static_cast<size_t>(n) * fp4_packed_bytes(R, K));
    for (int i = 0; i < n; ++i) {
        o.q[i] = at + i * fp4_packed_bytes(R, K);
        o.s[i] = s + i * fp4_scale_bytes(R, K, format);
    }
    at += packed_bytes(n, R, K, format);
    return o;
}

// The same for segments of K that a product sums: where each is whole stages of K, as one
// matrix [R, n K], which takes one tensor map in the place of n (no slower, no faster).
Packed place_segments(uint8_t*& at, int n, long long R, long long K, int format) {
    if (n == 1 || K % F4_BK != 0) return place(at, n, R, K, format);
    Packed o = place(at, 1, R, n * K, format);
    for (int i = 1; i < n; ++i) {
        o.q[i] = o.q[0] + i * (K / 2);
        o.s[i] = o.s[0] + i * (K / F4_BK) * fp4_scale_step(format);
    }
    o.k = n * K;
    return o;
}

// Scratch of a forward call: X by rows; of a backward call: dY by rows and by columns, the
// bias gradient's partial sums, and dY's scale.
size_t forward_bytes(const tpmlp_linear_dims& d, Split k, int format) {
    const bool col = k == Split::Column;
    return packed_bytes(col ? 1 : d.t, d.tokens, col ? d.in_features : d.in_features / d.t, format) + 256;
}
size_t backward_bytes(const tpmlp_linear_dims& d, Split k, int format) {
    const int n = k == Split::Column ? d.t : 1;
    const long long cols = d.out_features / n;
    return packed_bytes(n, d.tokens, cols, format) + packed_bytes(n, cols, d.tokens, format) +
           align256(static_cast<size_t>(up128(d.tokens)) * d.out_features * sizeof(float)) + 256;
}

// The step between matrices [outer, inner bytes] that lie at equal, ascending ones which a tensor
// map takes beside its rows' (whole rows of them, of at least a matrix), else 0.
uint64_t equal_steps(const void* const* p, int n, uint64_t inner, uint64_t outer) {
    const uint64_t first = reinterpret_cast<uint64_t>(p[0]);
    const uint64_t step = n > 1 ? reinterpret_cast<uint64_t>(p[1]) - first : 0;
    for (int i = 2; i < n; ++i)
        if (reinterpret_cast<uint64_t>(p[i]) - first != i * step) return 0;
    return step < (uint64_t(1) << 40) && step >= inner * outer && step % inner == 0 ? step : 0;
}

// Matrices [outer, inner bytes], `n` of them `step` bytes apart, in elements of `elem` bytes and
// boxes of box_inner elements x box_outer rows.  Kept by shape and step, as maps of 8-bit operands
// are by shape.
bool encode3(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t outer, uint64_t n, uint64_t step,
             int elem, uint32_t box_inner, uint32_t box_outer) {
    const CUtensorMapDataType type = elem == 8 ? CU_TENSOR_MAP_DATA_TYPE_INT64 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const CUtensorMapSwizzle swizzle = elem == 8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B;
    const cuuint64_t dims[3] = {inner / elem, outer, n};
    const cuuint64_t strides[2] = {inner, n > 1 ? step : inner * outer};
    const cuuint32_t box[3] = {box_inner, box_outer, 1};
    const MapKey key =
        make_map_key(type, 3, nullptr, dims, strides, box, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
    const bool ok = g_maps.get(key, m, [&](CUtensorMap* out) {
        const cuuint32_t estr[3] = {1, 1, 1};
        return g_encode(out, type, 3, const_cast<void*>(ptr), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    });
    return ok && set_address(m, ptr);
}

// One operand of a product: its matrices (one, or one per group or K segment), each
// [rows, K], and their scales.
struct Operand {
    const void* const* q;
    const void* const* s;
    int n;
    int part;
    const void* scale;  // of the tensor (nv)
    long long k;        // > 0: all segments are one matrix with this K
};

struct Product {
    int M, N, K, groups, ksegs;
    Operand a, b;
    const void* bias;
    bool f32;
    void* const* out;
    int nout;          // outputs: one per group, or one per token chunk
    int chunk_rows;    // > 0: rows per token chunk
    const void* const* x;  // A in bf16, for the few-rows kernel to quantise, or null
    // B was there before this call: it may be read before the grids ahead have ended, which
    // wait for what came before the call and only then let others start.  (Not where they write
    // B, as of a weight gradient, nor without one ahead.)
    bool early;
    bool apart;        // takes nothing from the grid ahead
    const float* sums; // partial rows of the bias gradient that are added up on the way, or null
    float* db;
    long long sum_rows;
    int sum_cols;
};

// The maps of an operand's values, and (box_tiles > 0) of its scales, that many times 128 rows a
// box; *z: one map for all its matrices.
bool encode_operand(CUtensorMap* m, CUtensorMap* sm, const Operand& o, int K, int rows, int box,
                    int format, uint32_t box_tiles, int* z) {
    const uint64_t inner = static_cast<uint64_t>(fp4_scale_bytes(1, K, format));
    const uint64_t step = equal_steps(o.q, o.n, fp4_ld(K), rows);
    const uint64_t sstep = equal_steps(o.s, o.n, inner, up128(rows));
    *z = o.n > 1 && step && sstep;
    const uint64_t n = *z ? o.n : 1;
    if (!encode3(m, o.q[0], fp4_ld(K), rows, n, step, 1, 128, box)) return false;
    const uint32_t width = static_cast<uint32_t>(fp4_scale_step(format) / 8);
    if (box_tiles && !encode3(sm, o.s[0], inner, up128(rows), n, sstep, 8, width, box_tiles)) return false;
    for (int i = 1; !*z && i < o.n; ++i) {
        m[i] = m[0];
        if (!set_address(&m[i], o.q[i])) return false;
        if (!box_tiles) continue;
        sm[i] = sm[0];
        if (!set_address(&sm[i], o.s[i])) return false;
    }
    return true;
}

tpmlp_status run_product(const DeviceInfo* dev, const Product& d, int format, int kind, cudaStream_t st) {
    Fp4GemmParams p;
    std::memset(&p, 0, sizeof(p));
    int few = 0;  // rows of a tile of the few-rows kernel
    if (!d.f32) TPMLP_CUDA(fp4_small_rows(d.M, d.N, d.K, d.groups, d.ksegs, format, few));
    if ((!d.x && !encode_operand(p.a_map, p.as_map, d.a, d.a.k > 0 ? static_cast<int>(d.a.k) : d.K, d.M,
                               few ? few : 128, format, few ? 0 : 1, &p.a_z)) ||
        !encode_operand(p.b_map, p.bs_map, d.b, d.K, d.N, 128, format, few ? 0 : 2, &p.b_z))
        return TPMLP_ERR_UNSUPPORTED;
    for (int i = 0; i < d.a.n; ++i) {
        if (d.x)
            p.x[i] = d.x[i];
        else
            p.sa[i] = static_cast<const uint8_t*>(d.a.s[i]);
    }
    p.early = d.early;
    p.apart = d.apart;
    p.sums = d.sums;
    p.db = d.db;
    p.sum_rows = d.sum_rows;
    p.sum_cols = d.sum_cols;
    for (int i = 0; i < d.b.n; ++i) p.sb[i] = static_cast<const uint8_t*>(d.b.s[i]);
    for (int i = 0; i < d.nout; ++i) p.out[i] = d.out[i];
    p.ga = static_cast<const float*>(d.a.scale);
    p.gb = static_cast<const float*>(d.b.scale);
    p.M = d.M;
    p.N = d.N;
    p.K = d.K;
    p.groups = d.groups;
    p.ksegs = d.ksegs;
    p.a_part = d.a.part;
    p.a_seg = d.a.k > 0 ? d.K / F4_BK : 0;
    p.b_part = d.b.part;
    const long long mt = (static_cast<long long>(d.M) + 255) / 256;
    const long long nt = (static_cast<long long>(d.N) + 255) / 256;
    if (mt * nt > 0x7FFFFFFFLL / d.groups) return TPMLP_ERR_UNSUPPORTED;
    p.mtiles = static_cast<int>(mt);
    p.ntiles = static_cast<int>(nt);
    p.total_tiles = static_cast<int>(mt * nt * d.groups);
    p.band = p.mtiles < kBand ? p.mtiles : kBand;
    p.chunk_rows = d.chunk_rows;
    p.bias = d.bias;
    p.err = dev->err;
    p.timeout_ns = g_timeout_ns;
    p.stall = g_stall;
    TPMLP_CUDA(timed(kind, 1, st, [&] {
        return few ? launch_fp4_small(p, format, few, d.x != nullptr, st) : launch_fp4_gemm(p, format, d.f32, st);
    }));
    return TPMLP_OK;
}

// Quantises an activation or gradient: token chunks of one matrix [T, cols], or `parts`
// matrices.  calibrated: *scale is given; else (nv) it is computed here.  Neither by rows nor by
// columns: only that.
tpmlp_status quantize(const DeviceInfo* dev, const void* const* src, int parts, bool gather, long long rows, long long cols,
                      int format, void* scale, bool calibrated, const Packed* by_rows,
                      const Packed* by_cols, float* sums, long long sums_ld, cudaStream_t st) {
    Fp4QuantParams p;
    std::memset(&p, 0, sizeof(p));
    p.parts = parts;
    p.gather = gather;
    p.rows = rows;
    p.cols = cols;
    p.scale = static_cast<const float*>(scale);
    p.sums_ld = sums_ld;
    p.err = dev->err;
    p.timeout_ns = g_timeout_ns;
    p.stall = g_stall;
    const int outs = gather ? 1 : parts;
    for (int i = 0; i < parts; ++i) p.src[i] = src[i];
    for (int i = 0; i < outs; ++i) {
        if (by_rows) p.rows_k = by_rows->k;
        if (by_rows) p.q_rows[i] = by_rows->q[i], p.s_rows[i] = by_rows->s[i];
        if (by_cols) p.q_cols[i] = by_cols->q[i], p.s_cols[i] = by_cols->s[i];
        if (sums) p.sums[i] = sums + i * cols;
    }
    if (format == FP4_NV && !calibrated)
        TPMLP_CUDA(timed(TPMLP_KERNEL_SP_COPY, fp4_tensor_scale_kernels(p), st,
                         [&] { return launch_fp4_tensor_scale(p, static_cast<float*>(scale), st); }));
    if (!by_rows && !by_cols) return TPMLP_OK;
    const int mode = (by_rows ? FP4_Q_ROWS : 0) | (by_cols ? FP4_Q_COLS : 0) | (sums ? FP4_Q_SUMS : 0);
    TPMLP_CUDA(timed(TPMLP_KERNEL_SP_COPY, 1, st, [&] { return launch_fp4_quant(p, format, mode, st); }));
    return TPMLP_OK;
}

tpmlp_status zero_grads(const Lin& s, Split k, void* const* dW, void* db, cudaStream_t st) {
    const size_t other = static_cast<size_t>(k == Split::Column ? s.in : s.out);
    for (int i = 0; i < s.t; ++i)
        TPMLP_CUDA(cudaMemsetAsync(dW[i], 0, other * s.shard * sizeof(float), st));
    TPMLP_CUDA(cudaMemsetAsync(db, 0, static_cast<size_t>(s.out) * sizeof(float), st));
    return TPMLP_OK;
}

// Whether one of m buffers lies over one of n.
bool any_overlap(const void* const* a, int m, int64_t abytes, void* const* b, int n, int64_t bbytes) {
    for (int i = 0; i < m; ++i) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(a[i]);
        for (int j = 0; j < n; ++j) {
            const uintptr_t y = reinterpret_cast<uintptr_t>(b[j]);
            if (x < y + bbytes && y < x + abytes) return true;
        }
    }
    return false;
}

inline const void* const* as_const(void* const* p) { return reinterpret_cast<const void* const*>(p); }

tpmlp_status forward(Split k, const tpmlp_linear_dims* dims, int format, const void* const* X,
                     void* x_scale, int x_calibrated, void* const* Xq, void* const* Xs,
                     const void* const* Wq, const void* const* Ws, const void* w_scale, const void* b,
                     void* const* Y, void* workspace, cudaStream_t st) {
    TPMLP_TRY(check_fp4_dims(dims, k));
    if (!format_ok(format)) return TPMLP_ERR_INVALID_ARG;
    const Lin s = lin_of(*dims, k);
    const bool col = k == Split::Column, save = Xq || Xs;
    // X: token chunks, or shards; kept by columns: one matrix, or shards
    const int nx = col ? s.chunks : s.t, nq = col ? 1 : s.t, ny = col ? s.t : s.chunks;
    TPMLP_TRY(check_ptr(b));
    TPMLP_TRY(check_ptrs(Wq, s.t));
    TPMLP_TRY(check_ptrs(Ws, s.t));
    TPMLP_TRY(check_tensor_scale(w_scale, format));
    TPMLP_TRY(check_tensor_scale(x_scale, format));
    if (s.T > 0) {
        TPMLP_TRY(check_ptrs(X, nx));
        TPMLP_TRY(check_ptrs(as_const(Y), ny));
        TPMLP_TRY(check_ptr(workspace));
        if (save) {
            TPMLP_TRY(check_ptrs(as_const(Xq), nq));
            TPMLP_TRY(check_ptrs(as_const(Xs), nq));
        }
    }
    DeviceInfo* dev = nullptr;
    TPMLP_TRY(device_info(&dev));
    if (s.T == 0) return TPMLP_OK;
    const int K = col ? s.in : s.shard;
    uint8_t* at = static_cast<uint8_t*>(workspace);
    const Packed rows = place_segments(at, nq, s.T, K, format);
    Packed cols = {};
    for (int i = 0; save && i < nq; ++i) {
        cols.q[i] = static_cast<uint8_t*>(Xq[i]);
        cols.s[i] = static_cast<uint8_t*>(Xs[i]);
    }
    Product p = {};
    p.M = s.T;
    p.N = col ? s.shard : s.out;
    p.K = K;
    p.groups = col ? s.t : 1;
    p.ksegs = col ? 1 : s.t;
    // (to keep X by columns takes the launch anyway; and CTAs that quantise X read it while others
    // write Y)
    bool quantises = false;
    if (!save && !any_overlap(X, nx, 2LL * (col ? s.Tc : s.T) * K, Y, ny, 2LL * (col ? s.T : s.Tc) * p.N))
        TPMLP_CUDA(fp4_small_quantises(p.M, p.N, p.K, p.groups, p.ksegs, quantises));
    p.x = quantises ? X : nullptr;
    p.early = !p.x;
    TPMLP_TRY(quantize(dev, X, nx, col, col ? s.Tc : s.T, K, format, x_scale, x_calibrated != 0,
                       p.x ? nullptr : &rows, save ? &cols : nullptr, nullptr, 0, st));
    p.a = Operand{reinterpret_cast<const void* const*>(rows.q), reinterpret_cast<const void* const*>(rows.s),
                  rows.k > 0 ? 1 : nq, rows.k > 0 || col ? F4_SINGLE : F4_KSEG, x_scale, rows.k};
    if (p.x) p.a = Operand{nullptr, nullptr, nq, col ? F4_SINGLE : F4_KSEG, x_scale, 0};
    p.b = Operand{Wq, Ws, s.t, col ? F4_GROUP : F4_KSEG, w_scale, 0};
    p.bias = b;
    p.f32 = false;
    p.out = Y;
    p.nout = ny;
    p.chunk_rows = col ? 0 : s.Tc;
    return run_product(dev, p, format, TPMLP_KERNEL_LINEAR_FWD, st);
}

tpmlp_status backward(Split k, const tpmlp_linear_dims* dims, int format, const void* const* dY,
                      const void* const* Xq, const void* const* Xs, const void* x_scale,
                      const void* const* Wq, const void* const* Ws, const void* w_scale,
                      void* const* dX, void* const* dW, void* db, void* workspace, cudaStream_t st) {
    TPMLP_TRY(check_fp4_dims(dims, k));
    if (!format_ok(format)) return TPMLP_ERR_INVALID_ARG;
    const Lin s = lin_of(*dims, k);
    const bool col = k == Split::Column;
    const int nx = col ? 1 : s.t, ndy = col ? s.t : s.chunks, ndx = col ? s.chunks : s.t;
    const int ng = col ? s.t : 1;  // quantised gradients: per shard, or one
    TPMLP_TRY(check_ptrs(Wq, s.t));
    TPMLP_TRY(check_ptrs(Ws, s.t));
    TPMLP_TRY(check_tensor_scale(w_scale, format));
    TPMLP_TRY(check_tensor_scale(x_scale, format));
    TPMLP_TRY(check_ptrs(as_const(dW), s.t));
    TPMLP_TRY(check_ptr(db));
    if (s.T > 0) {
        TPMLP_TRY(check_ptrs(dY, ndy));
        TPMLP_TRY(check_ptrs(Xq, nx));
        TPMLP_TRY(check_ptrs(Xs, nx));
        TPMLP_TRY(check_ptrs(as_const(dX), ndx));
        TPMLP_TRY(check_ptr(workspace));
    }
    DeviceInfo* dev = nullptr;
    TPMLP_TRY(device_info(&dev));
    if (s.T == 0) return zero_grads(s, k, dW, db, st);
    const int width = s.out / ng;  // columns of a gradient
    uint8_t* at = static_cast<uint8_t*>(workspace);
    const Packed rows = place_segments(at, ng, s.T, width, format), cols = place(at, ng, width, s.T, format);
    float* sums = reinterpret_cast<float*>(at);
    at += align256(static_cast<size_t>(up128(s.T)) * s.out * sizeof(float));
    void* dy_scale = format == FP4_NV ? at : nullptr;
    TPMLP_TRY(quantize(dev, dY, ndy, !col, col ? s.T : s.Tc, width, format, dy_scale, false, &rows, &cols, sums,
                       s.out, st));
    {
        // dX: M = T, N = in (or ii per group), K = oi per segment (or out); and db
        Product p = {};
        p.sums = sums;
        p.db = static_cast<float*>(db);
        p.sum_rows = up128(s.T);
        p.sum_cols = s.out;
        p.M = s.T;
        p.N = col ? s.in : s.shard;
        p.K = width;
        p.groups = col ? 1 : s.t;
        p.ksegs = col ? s.t : 1;
        p.a = Operand{reinterpret_cast<const void* const*>(rows.q),
                      reinterpret_cast<const void* const*>(rows.s), rows.k > 0 ? 1 : ng,
                      col && rows.k == 0 ? F4_KSEG : F4_SINGLE, dy_scale, rows.k};
        p.b = Operand{Wq, Ws, s.t, col ? F4_KSEG : F4_GROUP, w_scale, 0};
        p.f32 = false;
        p.out = dX;
        p.nout = ndx;
        p.chunk_rows = col ? s.Tc : 0;
        p.early = true;
        TPMLP_TRY(run_product(dev, p, format, TPMLP_KERNEL_LINEAR_DGRAD, st));
    }
    {
        // dW_i: M = in (or ii), N = oi (or out), K = T.  Its operands were there when dX's
        // product began: it runs beside the last of that, and ends after it (with db added up on
        // the way: backward of 16384 x 4096 x 4096 in eight shards 222 us, now 210; of 4096 x 4096
        // x 4096 95, now 85; of 40 tokens 40, now 36).
        Product p = {};
        p.apart = true;
        p.M = col ? s.in : s.shard;
        p.N = width;
        p.K = s.T;
        p.groups = s.t;
        p.ksegs = 1;
        p.a = Operand{Xq, Xs, nx, col ? F4_SINGLE : F4_GROUP, x_scale, 0};
        p.b = Operand{reinterpret_cast<const void* const*>(cols.q),
                      reinterpret_cast<const void* const*>(cols.s), ng, col ? F4_GROUP : F4_SINGLE, dy_scale, 0};
        p.f32 = true;
        p.out = dW;
        p.nout = s.t;
        TPMLP_TRY(run_product(dev, p, format, TPMLP_KERNEL_LINEAR_WGRAD, st));
    }
    return TPMLP_OK;
}

// What the two quantising calls have in common.
tpmlp_status check_quant(const tpmlp_fp4_quant* d) {
    if (!d || d->rows < 0 || d->cols <= 0 || d->parts <= 0 || !format_ok(d->format))
        return TPMLP_ERR_INVALID_ARG;
    const int64_t lim = (int64_t(1) << 31) - 1;
    if (d->parts > FP4_MAX_PARTS || d->cols % 32 != 0 || d->rows > lim || d->cols > lim)
        return TPMLP_ERR_UNSUPPORTED;
    if (d->gather && d->parts > 1 && (d->rows % 128 != 0 || d->rows * d->parts > lim))
        return TPMLP_ERR_UNSUPPORTED;
    return TPMLP_OK;
}

Fp4QuantParams quant_params(const tpmlp_fp4_quant& d, const void* const* src) {
    Fp4QuantParams p;
    std::memset(&p, 0, sizeof(p));
    for (int i = 0; i < d.parts && d.rows > 0; ++i) p.src[i] = src[i];
    p.rows = d.rows;
    p.cols = d.cols;
    p.parts = d.parts;
    p.gather = d.gather != 0;
    return p;
}

}  // namespace
}  // namespace tpmlp

using namespace tpmlp;
using namespace tpmlp::abi;

TPMLP_API size_t tpmlp_fp4_packed_bytes(int64_t rows, int64_t k) {
    return rows < 0 || k < 0 ? 0 : static_cast<size_t>(fp4_packed_bytes(rows, k));
}

TPMLP_API size_t tpmlp_fp4_scale_bytes(int64_t rows, int64_t k, int format) {
    return rows < 0 || k < 0 || !format_ok(format) ? 0 : static_cast<size_t>(fp4_scale_bytes(rows, k, format));
}

TPMLP_API tpmlp_status tpmlp_fp4_tensor_scale(const tpmlp_fp4_quant* d, const void* const* src, void* scale,
                                              void* stream) {
    TPMLP_TRY(check_quant(d));
    if (d->format != TPMLP_FP4_NV) return TPMLP_ERR_INVALID_ARG;
    TPMLP_TRY(check_scale(scale));
    if (d->rows > 0) TPMLP_TRY(check_ptrs(src, d->parts));
    DeviceInfo* dev = nullptr;
    TPMLP_TRY(device_info(&dev));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const Fp4QuantParams p = quant_params(*d, src);
    TPMLP_CUDA(timed(TPMLP_KERNEL_SP_COPY, fp4_tensor_scale_kernels(p), st,
                     [&] { return launch_fp4_tensor_scale(p, static_cast<float*>(scale), st); }));
    return TPMLP_OK;
}

TPMLP_API tpmlp_status tpmlp_fp4_quantize(const tpmlp_fp4_quant* d, const void* const* src,
                                          const void* scale, void* const* q_rows, void* const* s_rows,
                                          void* const* q_cols, void* const* s_cols, void* stream) {
    TPMLP_TRY(check_quant(d));
    const bool rows = q_rows || s_rows, cols = q_cols || s_cols;
    if (!rows && !cols) return TPMLP_ERR_INVALID_ARG;
    TPMLP_TRY(check_tensor_scale(scale, d->format));
    const int n = d->parts, outs = d->gather ? 1 : n;
    if (d->rows > 0) {
        TPMLP_TRY(check_ptrs(src, n));
        if (rows) {
            TPMLP_TRY(check_ptrs(as_const(q_rows), outs));
            TPMLP_TRY(check_ptrs(as_const(s_rows), outs));
        }
        if (cols) {
            TPMLP_TRY(check_ptrs(as_const(q_cols), outs));
            TPMLP_TRY(check_ptrs(as_const(s_cols), outs));
        }
    }
    DeviceInfo* dev = nullptr;
    TPMLP_TRY(device_info(&dev));
    if (d->rows == 0) return TPMLP_OK;
    Fp4QuantParams p = quant_params(*d, src);
    for (int i = 0; i < outs; ++i) {
        if (rows) p.q_rows[i] = static_cast<uint8_t*>(q_rows[i]), p.s_rows[i] = static_cast<uint8_t*>(s_rows[i]);
        if (cols) p.q_cols[i] = static_cast<uint8_t*>(q_cols[i]), p.s_cols[i] = static_cast<uint8_t*>(s_cols[i]);
    }
    p.scale = static_cast<const float*>(scale);
    p.err = dev->err;
    p.timeout_ns = g_timeout_ns;
    p.stall = g_stall;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int mode = (rows ? FP4_Q_ROWS : 0) | (cols ? FP4_Q_COLS : 0);
    TPMLP_CUDA(timed(TPMLP_KERNEL_SP_COPY, 1, st, [&] { return launch_fp4_quant(p, d->format, mode, st); }));
    return TPMLP_OK;
}

TPMLP_API tpmlp_status tpmlp_fp4_dequantize(int64_t rows, int64_t k, int format, const void* q,
                                            const void* s, const void* scale, void* out, void* stream) {
    if (rows < 0 || k < 0 || !format_ok(format)) return TPMLP_ERR_INVALID_ARG;
    const int64_t lim = (int64_t(1) << 31) - 1;
    if (rows > lim || k > lim) return TPMLP_ERR_UNSUPPORTED;
    TPMLP_TRY(check_tensor_scale(scale, format));
    if (rows > 0 && k > 0) {
        TPMLP_TRY(check_ptr(q));
        TPMLP_TRY(check_ptr(s));
        TPMLP_TRY(check_ptr(out));
    }
    DeviceInfo* dev = nullptr;
    TPMLP_TRY(device_info(&dev));
    if (rows == 0 || k == 0) return TPMLP_OK;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    TPMLP_CUDA(timed(TPMLP_KERNEL_SP_COPY, 1, st, [&] {
        return launch_fp4_dequant(rows, k, format, q, s, static_cast<const float*>(scale), out, st);
    }));
    return TPMLP_OK;
}

TPMLP_API size_t tpmlp_fp4_linear_workspace_bytes(const tpmlp_linear_dims* dims, int format, int backward) {
    if (!format_ok(format)) return 0;
    size_t most = 0;
    for (const Split k : {Split::Column, Split::Row}) {
        if (check_fp4_dims(dims, k) != TPMLP_OK) continue;
        const size_t f = forward_bytes(*dims, k, format), b = backward ? backward_bytes(*dims, k, format) : 0;
        if (f > most) most = f;
        if (b > most) most = b;
    }
    return most;
}

TPMLP_API tpmlp_status tpmlp_fp4_column_linear_forward(
    const tpmlp_linear_dims* dims, int format, const void* const* X, void* x_scale, int x_calibrated,
    void* Xq, void* Xs, const void* const* Wq_shards, const void* const* Ws_shards, const void* w_scale,
    const void* b, void* const* Y_shards, void* workspace, void* stream) {
    return forward(Split::Column, dims, format, X, x_scale, x_calibrated, Xq ? &Xq : nullptr,
                   Xs ? &Xs : nullptr, Wq_shards, Ws_shards, w_scale, b, Y_shards, workspace,
                   static_cast<cudaStream_t>(stream));
}

TPMLP_API tpmlp_status tpmlp_fp4_row_linear_forward(
    const tpmlp_linear_dims* dims, int format, const void* const* X_shards, void* x_scale,
    int x_calibrated, void* const* Xq_shards, void* const* Xs_shards, const void* const* Wq_shards,
    const void* const* Ws_shards, const void* w_scale, const void* b, void* const* Z, void* workspace,
    void* stream) {
    return forward(Split::Row, dims, format, X_shards, x_scale, x_calibrated, Xq_shards, Xs_shards,
                   Wq_shards, Ws_shards, w_scale, b, Z, workspace, static_cast<cudaStream_t>(stream));
}

TPMLP_API tpmlp_status tpmlp_fp4_column_linear_backward(
    const tpmlp_linear_dims* dims, int format, const void* const* dY_shards, const void* Xq,
    const void* Xs, const void* x_scale, const void* const* Wq_shards, const void* const* Ws_shards,
    const void* w_scale, void* const* dX, void* const* dW_shards, void* db, void* workspace, void* stream) {
    return backward(Split::Column, dims, format, dY_shards, &Xq, &Xs, x_scale, Wq_shards, Ws_shards,
                    w_scale, dX, dW_shards, db, workspace, static_cast<cudaStream_t>(stream));
}

TPMLP_API tpmlp_status tpmlp_fp4_row_linear_backward(
    const tpmlp_linear_dims* dims, int format, const void* const* dZ, const void* const* Xq_shards,
    const void* const* Xs_shards, const void* x_scale, const void* const* Wq_shards,
    const void* const* Ws_shards, const void* w_scale, void* const* dX_shards, void* const* dW_shards,
    void* db, void* workspace, void* stream) {
    return backward(Split::Row, dims, format, dZ, Xq_shards, Xs_shards, x_scale, Wq_shards, Ws_shards,
                    w_scale, dX_shards, dW_shards, db, workspace, static_cast<cudaStream_t>(stream));
}
