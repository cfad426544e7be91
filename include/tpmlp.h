/*
 * tpmlp.h -- C ABI of libtpmlp: the tensor-parallel Transformer MLP block,
 * forward and backward, on one sm_103 GPU, and the column- and row-parallel
 * linear layers it is made of (the attention projections).
 *
 *     Z = GeLU(X.A + b1).B + b2
 *
 * Sources (page title, section):
 *   [FGO]    "Megatron-LM：NVIDIA 的大规模并行训练方案", section
 *            "Megatron-LM 核心架构 / 张量并行原理": Y = XA; A split by
 *            columns [A_1, A_2] gives Y_i = X.A_i (column parallel); A split
 *            by rows with X split by columns gives Y = sum_i X_i.A_i summed by
 *            an AllReduce (row parallel); the MLP's first linear is column
 *            parallel and its second row parallel.
 *   [FGO-F]  same page, "融合优化技术": Bias + GeLU fused into one kernel.
 *   [FGO-SP] same page, "并行训练范式 / 序列并行": sequence parallelism on
 *            top of tensor parallelism, along the sequence dimension.
 *   [CH2]    "2、分布式训练基础：数据并行、模型并行、流水线并行的基本概念与区别",
 *            "2.2 模型并行 —— 张量并行 / 核心原理": column-parallel split
 *            [W1, W2], row-parallel split [W1; W2] with X = [X1, X2] and an
 *            AllReduce sum.
 *
 * All t shards live on the one GPU; the row-parallel AllReduce of the
 * forward pass (and its conjugate in the backward pass) becomes an on-chip
 * split-K accumulation over the shards.  In the sequence-parallel variant X
 * and dZ arrive as seq_chunks token chunks and Z and dX leave in the same
 * chunking: the gather before the column-parallel GEMM is done by addressing
 * the chunks directly, the reduce-scatter after the row-parallel GEMM by the
 * split-K accumulation plus a row-to-chunk mapping in the GEMM's epilogue.
 *
 * Conventions for every call:
 *   - All matrices are dense, row-major, with the shapes given below.
 *     Notation: T = tokens, h = hidden, f = ffn, fi = f / t, Tc = T / seq_chunks.
 *   - All buffer pointers are DEVICE pointers on the current CUDA device,
 *     owned by the caller, 16-byte aligned.  The library never allocates
 *     or frees device memory during a forward/backward call.
 *   - Pointer-array arguments ("const void* const*") are HOST arrays of
 *     device pointers (one per shard or per chunk); the library copies the
 *     pointers during the call and does not keep the host array.
 *   - Calls are asynchronous on the given stream (a cudaStream_t passed as
 *     void*; NULL = the legacy default stream).  A returned TPMLP_OK means the
 *     work was validated and enqueued; device-side failures (a bounded wait
 *     that expired) are reported by tpmlp_sync_check().
 *   - Validation failures return an error before anything is launched and
 *     leave every output untouched.  Nothing crosses the ABI as an exception.
 *   - Results are bitwise reproducible run to run (no atomics in any sum).
 *   - Thread-compatible: concurrent calls from several host threads are
 *     allowed on different streams with different workspaces.
 *
 * Requirements (else TPMLP_ERR_UNSUPPORTED): an sm_103 device; h and fi
 * multiples of 8; 1 <= t <= 8; 1 <= seq_chunks <= 8 dividing T, and, when
 * seq_chunks > 1, Tc a multiple of 128; T, h, f below 2^31.
 */
#ifndef TPMLP_H
#define TPMLP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    TPMLP_OK = 0,
    TPMLP_ERR_INVALID_ARG = 1,  /* null pointer, bad dims, t mismatch */
    TPMLP_ERR_UNSUPPORTED = 2,  /* shape/alignment/device outside the requirements */
    TPMLP_ERR_CUDA = 3,         /* a CUDA runtime/driver call failed */
    TPMLP_ERR_TIMEOUT = 4       /* a bounded device wait expired (see tpmlp_sync_check) */
} tpmlp_status;

typedef struct {
    int64_t tokens;      /* T: micro-batch x sequence rows, sequence-major */
    int64_t hidden;      /* h */
    int64_t ffn;         /* f */
    int32_t t;           /* tensor-parallel shards (1..8) */
    int32_t seq_chunks;  /* 1, or the sequence-parallel degree (normally t) */
} tpmlp_dims;

/* Bytes of device workspace a forward/backward pair needs: the saved
 * pre-activation Y and activation H (written by tpmlp_forward, read by
 * tpmlp_backward), the gradient dY (written and read by tpmlp_backward) and
 * the bias-gradient partial sums.  The caller allocates it (256-byte aligned
 * is best) and keeps it alive from the forward to the matching backward. */
size_t tpmlp_workspace_bytes(const tpmlp_dims* dims);

/* Byte offsets inside the workspace of Y, H and dY, each stored shard-major
 * as t blocks [T, fi] bf16 (shard i at offset + i*T*fi*2).  Any output may be
 * NULL.  Lets a caller inspect the saved activations. */
tpmlp_status tpmlp_workspace_layout(const tpmlp_dims* dims, size_t* y_offset,
                                    size_t* h_offset, size_t* dy_offset);

/* Forward pass ([FGO] 张量并行原理, [CH2] 2.2, [FGO-F] 融合优化技术):
 *   for each shard i:  Y_i = X.A_i + b1[i*fi:(i+1)*fi],  H_i = GeLU(Y_i)
 *   Z = (sum_i H_i.B_i) + b2          (b2 added once, after the shard sum)
 * GeLU is the tanh form 0.5 y (1 + tanh(sqrt(2/pi) (y + 0.044715 y^3))).
 *   X        [seq_chunks] chunks of [Tc, h] bf16 (chunk j = token rows j*Tc..)
 *   A_shards [t] shards of [h, fi] bf16   (column block i of A)
 *   b1       [f] bf16
 *   B_shards [t] shards of [fi, h] bf16   (row block i of B)
 *   b2       [h] bf16
 *   t        must equal dims->t
 *   Z        [seq_chunks] chunks of [Tc, h] bf16 (output)
 *   workspace  >= tpmlp_workspace_bytes(dims) bytes; Y and H are saved there
 * Products accumulate in fp32 on the tensor cores; bias and GeLU are applied
 * in fp32 in the GEMM epilogue; Y, H and Z are rounded to bf16 once. */
tpmlp_status tpmlp_forward(const tpmlp_dims* dims,
                           const void* const* X,
                           const void* const* A_shards, const void* b1,
                           const void* const* B_shards, const void* b2,
                           int t,
                           void* const* Z,
                           void* workspace, void* stream);

/* Backward pass: the chain rule of tpmlp_forward for upstream gradient dZ.
 *   dY_i = (dZ.B_i^T) * GeLU'(Y_i)   (kept in the workspace, bf16)
 *   dX   = sum_i dY_i.A_i^T          (the backward AllReduce, on chip)
 *   dA_i = X^T.dY_i,  dB_i = H_i^T.dZ,
 *   db1  = column sums of dY, db2 = column sums of dZ.
 *   dZ        [seq_chunks] chunks of [Tc, h] bf16
 *   X, A_shards, B_shards   as passed to tpmlp_forward
 *   workspace the workspace of the matching tpmlp_forward (Y, H read; dY written)
 *   dX        [seq_chunks] chunks of [Tc, h] bf16 (output)
 *   dA_shards [t] of [h, fi] fp32 (output, overwritten)
 *   db1       [f] fp32 (output, overwritten)
 *   dB_shards [t] of [fi, h] fp32 (output, overwritten)
 *   db2       [h] fp32 (output, overwritten)
 * With T = 0 the weight and bias gradients are set to zero. */
tpmlp_status tpmlp_backward(const tpmlp_dims* dims,
                            const void* const* dZ,
                            const void* const* X,
                            const void* const* A_shards,
                            const void* const* B_shards,
                            void* workspace,
                            void* const* dX,
                            void* const* dA_shards, void* db1,
                            void* const* dB_shards, void* db2,
                            void* stream);

/* Selective recompute ("融合优化技术" and "高级特性 / 选择性激活重计算" on
 * "Megatron-LM：NVIDIA 的大规模并行训练方案": keep part of the activations,
 * recompute the rest in the backward pass).  Same block, same results for
 * Z, dX, dA, db1 and db2 (bitwise); dB is computed from H = GeLU(Y) rebuilt
 * from the saved bf16 Y, so it may differ from tpmlp_backward's in the last
 * bits.  Only Y (T x f bf16) is kept between the forward and the backward
 * pass ("saved", per layer); H, dY and the partial sums live in "scratch",
 * which holds nothing between calls and can be shared by all layers that run
 * on one stream.  The dH GEMM's epilogue rebuilds H from Y as it computes dY.
 *   saved   >= *saved_bytes device bytes: written by the forward, read by the backward
 *   scratch >= *scratch_bytes device bytes: used during either call only
 * Other arguments, layouts and errors as tpmlp_forward / tpmlp_backward. */
tpmlp_status tpmlp_recompute_workspace_bytes(const tpmlp_dims* dims, size_t* saved_bytes,
                                             size_t* scratch_bytes);
tpmlp_status tpmlp_forward_recompute(const tpmlp_dims* dims,
                                     const void* const* X,
                                     const void* const* A_shards, const void* b1,
                                     const void* const* B_shards, const void* b2,
                                     int t,
                                     void* const* Z,
                                     void* saved, void* scratch, void* stream);
tpmlp_status tpmlp_backward_recompute(const tpmlp_dims* dims,
                                      const void* const* dZ,
                                      const void* const* X,
                                      const void* const* A_shards,
                                      const void* const* B_shards,
                                      void* saved, void* scratch,
                                      void* const* dX,
                                      void* const* dA_shards, void* db1,
                                      void* const* dB_shards, void* db2,
                                      void* stream);

/* ---- Tensor-parallel linear layers ------------------------------------------
 * The two halves of the block without the GeLU, as the attention projections
 * use them ([CH2] 2.2: the QKV projection is column parallel, the output
 * projection row parallel; [FGO] 张量并行原理).  Same kernels, conventions,
 * sequence-parallel chunking and error behaviour as tpmlp_forward /
 * tpmlp_backward.  Notation: T = tokens, in = in_features, out =
 * out_features, Tc = T / seq_chunks.
 *
 * Requirements (else TPMLP_ERR_UNSUPPORTED) as for the block, with:
 *   column parallel: t divides out (else TPMLP_ERR_INVALID_ARG); in and
 *                    oi = out / t multiples of 8;
 *   row parallel:    t divides in (else TPMLP_ERR_INVALID_ARG); ii = in / t
 *                    and out multiples of 8.
 * The workspace holds only scratch (tail-split partial tiles, bias-gradient
 * partial sums); nothing in it lives from one call to the next, so one
 * workspace may serve every linear layer that runs on one stream. */
typedef struct {
    int64_t tokens;        /* T */
    int64_t in_features;   /* in: K of the forward product */
    int64_t out_features;  /* out: N of the forward product */
    int32_t t;             /* shards (1..8): of out (column) or of in (row) */
    int32_t seq_chunks;    /* 1, or the sequence-parallel degree */
} tpmlp_linear_dims;

/* Bytes of scratch workspace any linear-layer call with these dims needs. */
size_t tpmlp_linear_workspace_bytes(const tpmlp_linear_dims* dims);

/* Column-parallel forward:  Y_i = X.W_i + b[i*oi:(i+1)*oi]
 *   X        [seq_chunks] chunks of [Tc, in] bf16 (gathered on the fly)
 *   W_shards [t] of [in, oi] bf16 (column block i of W)
 *   b        [out] bf16
 *   Y_shards [t] of [T, oi] bf16 (output)
 * Backward for upstream dY_i:
 *   dX = sum_i dY_i.W_i^T  (on-chip shard sum; written back in chunks)
 *   dW_i = X^T.dY_i,  db = column sums of [dY_1 .. dY_t]
 *   dY_shards [t] of [T, oi] bf16;  X, W_shards as in the forward
 *   dX        [seq_chunks] chunks of [Tc, in] bf16 (output)
 *   dW_shards [t] of [in, oi] fp32 (output, overwritten)
 *   db        [out] fp32 (output, overwritten)
 * With T = 0 the forward does nothing and the backward zeroes dW and db. */
tpmlp_status tpmlp_column_linear_forward(const tpmlp_linear_dims* dims,
                                         const void* const* X,
                                         const void* const* W_shards, const void* b,
                                         void* const* Y_shards,
                                         void* workspace, void* stream);
tpmlp_status tpmlp_column_linear_backward(const tpmlp_linear_dims* dims,
                                          const void* const* dY_shards,
                                          const void* const* X,
                                          const void* const* W_shards,
                                          void* const* dX,
                                          void* const* dW_shards, void* db,
                                          void* workspace, void* stream);

/* Row-parallel forward:  Z = (sum_i X_i.W_i) + b   (b added once, after the
 * shard sum -- the AllReduce of [CH2] 2.2 done on chip)
 *   X_shards [t] of [T, ii] bf16 (column block i of the input)
 *   W_shards [t] of [ii, out] bf16 (row block i of W)
 *   b        [out] bf16
 *   Z        [seq_chunks] chunks of [Tc, out] bf16 (output, reduce-scattered)
 * Backward for upstream dZ:
 *   dX_i = dZ.W_i^T,  dW_i = X_i^T.dZ,  db = column sums of dZ
 *   dZ        [seq_chunks] chunks of [Tc, out] bf16;  X_shards, W_shards as in the forward
 *   dX_shards [t] of [T, ii] bf16 (output)
 *   dW_shards [t] of [ii, out] fp32 (output, overwritten)
 *   db        [out] fp32 (output, overwritten)
 * With T = 0 the forward does nothing and the backward zeroes dW and db. */
tpmlp_status tpmlp_row_linear_forward(const tpmlp_linear_dims* dims,
                                      const void* const* X_shards,
                                      const void* const* W_shards, const void* b,
                                      void* const* Z,
                                      void* workspace, void* stream);
tpmlp_status tpmlp_row_linear_backward(const tpmlp_linear_dims* dims,
                                       const void* const* dZ,
                                       const void* const* X_shards,
                                       const void* const* W_shards,
                                       void* const* dX_shards,
                                       void* const* dW_shards, void* db,
                                       void* workspace, void* stream);

/* ---- Sequence-parallel LayerNorm / Dropout sublayer ---------------------------
 * "Megatron-LM：NVIDIA 的大规模并行训练方案", "并行训练范式 / 序列并行": on top
 * of tensor parallelism, LayerNorm and Dropout are distributed along the
 * sequence dimension, each rank working on its token chunk.  The sublayer
 * around the block is the pre-LayerNorm residual block
 *
 *   Out = X + Dropout(MLP(LN(X)))
 *   LN(X) = (X - mean) * rstd * gamma + beta per token row over h,
 *           mean and var the row's mean and (biased) variance, rstd = 1/sqrt(var + eps)
 *   Dropout(z) = keep ? z / (1 - p) : 0
 *
 * keep for element (r, n) of the [T, h] output, e = r * h + n (r the token
 * row over all chunks): Philox4x32-10 (Salmon, Moraes, Dror and Shaw,
 * "Parallel random numbers: as easy as 1, 2, 3", SC'11) with key
 * (seed_lo, seed_hi) and counter (lo, hi, 0, 0) of offset + e / 4; word e % 4
 * of its output is compared with floor((1 - p) * 2^32) (keep iff below).
 * The same element keeps the same mask in the forward and the backward call.
 *
 * The forward pass runs LN per token chunk, then the block on LN(X) with the
 * dropout and the residual add fused into the row GEMM's epilogue, which also
 * stores the mask as bits in the workspace; the backward pass undoes the
 * dropout on dOut from those bits (summing dZ's columns into db2 on the way),
 * runs the block's backward pass, then LN's backward with the residual
 * gradient dOut added:
 *   dX = LN'(dXn) + dOut,  dgamma = sum_r dXn * xhat,  dbeta = sum_r dXn
 * Layouts, chunking, conventions and errors as tpmlp_forward / tpmlp_backward,
 * with h <= 16384 (else TPMLP_ERR_UNSUPPORTED), eps >= 0 and 0 <= p < 1
 * (else TPMLP_ERR_INVALID_ARG).  gamma, beta [h] bf16; dgamma, dbeta [h] fp32.
 * The workspace (tpmlp_sp_workspace_bytes) holds the block's workspace plus
 * LN(X), the row statistics, the dropout mask's bits (T x ceil(h / 32) 32-bit
 * words), dZ and the gradient of LN(X); it must be kept from the forward call
 * to the matching backward call. */
typedef struct {
    float eps;           /* LayerNorm epsilon (e.g. 1e-5) */
    double dropout_p;    /* probability of dropping an element, 0 <= p < 1 */
    uint64_t seed;       /* Philox key */
    uint64_t offset;     /* Philox counter offset, in blocks of 4 elements */
} tpmlp_sp_params;

size_t tpmlp_sp_workspace_bytes(const tpmlp_dims* dims);
/* Byte offsets in that workspace of LN(X) and of dZ (= dOut with the dropout
 * undone, written by tpmlp_sp_backward), each a [T, h] bf16 tensor stored
 * chunk after chunk.  Either output may be NULL. */
tpmlp_status tpmlp_sp_workspace_layout(const tpmlp_dims* dims, size_t* xn_offset,
                                       size_t* dz_offset);
tpmlp_status tpmlp_sp_forward(const tpmlp_dims* dims, const tpmlp_sp_params* sp,
                              const void* const* X, const void* gamma, const void* beta,
                              const void* const* A_shards, const void* b1,
                              const void* const* B_shards, const void* b2, int t,
                              void* const* Out, void* workspace, void* stream);
tpmlp_status tpmlp_sp_backward(const tpmlp_dims* dims, const tpmlp_sp_params* sp,
                               const void* const* dOut, const void* const* X,
                               const void* gamma, const void* const* A_shards,
                               const void* const* B_shards, void* workspace,
                               void* const* dX, void* dgamma, void* dbeta,
                               void* const* dA_shards, void* db1,
                               void* const* dB_shards, void* db2, void* stream);

/* ---- 8-bit linear layers ------------------------------------------------------
 * The tensor-parallel linear layers on 8-bit floating-point operands with one
 * fp32 scale for each group of 128 values ("blocks of 128"), sums in fp32:
 *
 *   Y[m, n] = b[n] + sum_kb sx[kb, m] sw[kb, n / 128] sum_{k in kb} xq[m, k] wq[k, n]
 *
 * over K blocks kb of 128 input features.  Half the weight bytes of bf16 when
 * few tokens are decoded, twice its tensor rate when there are many.
 *
 * Quantisation of a group G of bf16 values x:
 *   s = the smallest power of two with max |x| <= s * top, at least 2^-119
 *   q = x / s (exact) rounded to nearest even
 * top = 448 for e4m3, 57344 for e5m2.  A group that holds an infinity or a NaN
 * gets s = NaN and q = 0, so what is computed from it is NaN.  The tensor cores
 * apply the scales as 8-bit exponents: a matrix quantised elsewhere may be used
 * if its scales are powers of two, 2^-126 .. 2^127; any other scale reads as NaN.
 *
 * Layouts, for a matrix [R, C] row-major (R tokens or input features):
 *   q         8-bit [R, C], C a multiple of 16
 *   rows      groups of 128 along a row:    s fp32 [ceil(C/128), ld], ld >= R
 *   columns   groups of 128 along a column: s fp32 [ceil(R/128), C]
 *   weight    blocks of 128 x 128:          s fp32 [ceil(R/128), ceil(C/128)]
 * Conventions, chunking, errors and workspace rules as for the bf16 linear
 * layers, with features and shards multiples of 16 and no more than 2^31 - 256
 * tokens or features (else TPMLP_ERR_UNSUPPORTED); scales (s) may start at any
 * multiple of 4 bytes. */
typedef enum {
    TPMLP_FP8_E4M3 = 0, /* 4 exponent bits, 3 mantissa bits, no infinities */
    TPMLP_FP8_E5M2 = 1  /* 5 exponent bits, 2 mantissa bits */
} tpmlp_fp8_format;

/* `parts` matrices [rows, cols] of the same shape, quantised in one launch. */
typedef struct {
    int64_t rows, cols;   /* of each part */
    int64_t scale_ld;     /* leading dimension (floats) of the row scales, >= rows */
    int32_t parts;        /* 1..8 */
    int32_t rows_format;  /* tpmlp_fp8_format of q_rows */
    int32_t cols_format;  /* and of q_cols */
} tpmlp_fp8_quant;

/* Formats of a linear layer's operands. */
typedef struct {
    int32_t x, w, dy;
} tpmlp_fp8_formats;

/* Quantise activations by rows, by columns, or both in one read of src (bf16).
 * src, q_rows, s_rows, q_cols, s_cols: host arrays of `parts` device pointers;
 * the row pair or the column pair may be NULL, not both.  Parts may be the
 * shards of a tensor (each with outputs of its own) or the token chunks of one
 * [T, cols] matrix: then part j of Tc = T / parts rows writes
 *   q + j Tc cols,  s_rows + j Tc (scale_ld = T),  s_cols + j (Tc / 128) cols,
 * which gathers the chunks; Tc must then be a multiple of 128. */
tpmlp_status tpmlp_fp8_quantize(const tpmlp_fp8_quant* quant, const void* const* src,
                                void* const* q_rows, void* const* s_rows, void* const* q_cols,
                                void* const* s_cols, void* stream);

/* Quantise one weight shard W [in, out] bf16 in 128 x 128 blocks. */
tpmlp_status tpmlp_fp8_quantize_weight(const void* W, int64_t in, int64_t out, int format, void* q,
                                       void* s, void* stream);

/* Bytes of scratch workspace any 8-bit linear call with these dims needs. */
size_t tpmlp_fp8_linear_workspace_bytes(const tpmlp_linear_dims* dims);

/* Column parallel.  Forward:  Y_i = X.W_i + b[i*oi:(i+1)*oi]
 *   Xq, Xs     X [T, in] by rows (one matrix; quantising gathered the chunks)
 *   Wq, Ws     [t] shards [in, oi] in blocks
 *   b          [out] bf16;  Y_shards [t] of [T, oi] bf16 (output)
 * Backward for upstream dY_i (bf16, quantised here by rows and by columns in
 * the format formats->dy):
 *   dX = sum_i dY_i.W_i^T (bf16, seq_chunks chunks), dW_i = X^T.dY_i (fp32),
 *   db = column sums of the bf16 dY (fp32)
 *   Xq, Xs     X [T, in] by columns, kept from the forward pass
 * With T = 0 the forward does nothing and the backward zeroes dW and db. */
tpmlp_status tpmlp_fp8_column_linear_forward(const tpmlp_linear_dims* dims,
                                             const tpmlp_fp8_formats* formats, const void* Xq,
                                             const void* Xs, const void* const* Wq_shards,
                                             const void* const* Ws_shards, const void* b,
                                             void* const* Y_shards, void* workspace, void* stream);
tpmlp_status tpmlp_fp8_column_linear_backward(const tpmlp_linear_dims* dims,
                                              const tpmlp_fp8_formats* formats,
                                              const void* const* dY_shards, const void* Xq,
                                              const void* Xs, const void* const* Wq_shards,
                                              const void* const* Ws_shards, void* const* dX,
                                              void* const* dW_shards, void* db, void* workspace,
                                              void* stream);

/* Row parallel.  Forward:  Z = (sum_i X_i.W_i) + b
 *   Xq, Xs     [t] shards X_i [T, ii] by rows;  Wq, Ws [t] shards [ii, out]
 *   b          [out] bf16;  Z seq_chunks chunks of [Tc, out] bf16 (output)
 * Backward for upstream dZ (seq_chunks chunks, bf16):
 *   dX_i = dZ.W_i^T (bf16 [T, ii]), dW_i = X_i^T.dZ (fp32 [ii, out]), db (fp32)
 *   Xq, Xs     [t] shards X_i [T, ii] by columns, kept from the forward pass */
tpmlp_status tpmlp_fp8_row_linear_forward(const tpmlp_linear_dims* dims,
                                          const tpmlp_fp8_formats* formats,
                                          const void* const* Xq_shards,
                                          const void* const* Xs_shards,
                                          const void* const* Wq_shards,
                                          const void* const* Ws_shards, const void* b,
                                          void* const* Z, void* workspace, void* stream);
tpmlp_status tpmlp_fp8_row_linear_backward(const tpmlp_linear_dims* dims,
                                           const tpmlp_fp8_formats* formats,
                                           const void* const* dZ, const void* const* Xq_shards,
                                           const void* const* Xs_shards,
                                           const void* const* Wq_shards,
                                           const void* const* Ws_shards, void* const* dX_shards,
                                           void* const* dW_shards, void* db, void* workspace,
                                           void* stream);

/* ---- Linear layers on 4-bit operands ------------------------------------------------
 * The same layers with X, W and dY in 4-bit floating point (a sign, two exponent bits, one
 * mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) and a scale for each group along the axis that
 * a product sums over, on the tensor cores' 4-bit instructions:
 *
 *   mx   groups of 32; s = the smallest power of two with max |x| <= 6 s, at least 2^-126,
 *        stored as an 8-bit exponent (biased by 127)
 *   nv   groups of 16 and a scale g (fp32, on the device) for the tensor, which all its
 *        shards share: s = max |x| / (6 g) rounded to e4m3, at most 448, at least 2^-9;
 *        tpmlp_fp4_tensor_scale makes g the smallest power of two, at least 2^-110, with
 *        which the largest finite magnitude is at most 6 * 448 g.  A given g has to be a
 *        power of two of 2^-110 .. 2^117 (else every result is NaN); what it leaves out of
 *        range becomes the largest value
 *   q  = round-to-nearest-even(x / s), of nv x / (s g)
 *
 * Two things differ from what else goes under these names.  mx elsewhere often takes for s the
 * power of two of max |x| over that of 4 and cuts off what lies above 6 s: bytes differ for a
 * group whose largest is between 6 and 8 times a power of two.  nv elsewhere takes any fp32 for
 * g: tensors quantised with one are not taken here.
 *
 * The same on every machine: powers of two leave every comparison exact.  A group with an
 * infinity or a NaN has the scale NaN, and so have the results that take part of it.
 *
 * A 4-bit matrix [R, K] is summed over K: R rows of (K rounded up to 32) / 2 bytes, element
 * 2i in the low half of byte i.  Its scales: for each 128 rows and each 256 of K 1024 bytes
 * (mx) or 2048 (nv) of one byte a scale, in blocks of 128 rows by 4 groups, row r's group j
 * at byte 16 (r % 32) + 4 (r / 32) + j of its block.  Quantising "by rows" makes [T, C] of a
 * bf16 [T, C], "by columns" the transposed [C, T].  tpmlp_fp4_packed_bytes and
 * tpmlp_fp4_scale_bytes are the sizes of the two arrays, which start on 16 bytes.
 * Conventions, chunking, errors and workspace rules as for the bf16 linear layers, with
 * features and shards multiples of 32 and no more than 2^31 - 256 tokens or features (else
 * TPMLP_ERR_UNSUPPORTED). */
typedef enum {
    TPMLP_FP4_MX = 0,
    TPMLP_FP4_NV = 1
} tpmlp_fp4_format;

/* `parts` bf16 matrices [rows, cols] of the same shape, quantised in one launch: each with
 * outputs of its own (gather = 0), or row chunks of one matrix [parts * rows, cols] with one
 * output (gather = 1; rows then a multiple of 128 unless parts = 1). */
typedef struct {
    int64_t rows, cols; /* of each part; cols a multiple of 32 */
    int32_t parts;      /* 1..8 */
    int32_t gather;
    int32_t format;     /* tpmlp_fp4_format */
} tpmlp_fp4_quant;

size_t tpmlp_fp4_packed_bytes(int64_t rows, int64_t k);
size_t tpmlp_fp4_scale_bytes(int64_t rows, int64_t k, int format);

/* g of all parts together (nv) into scale[0], fp32 on the device. */
tpmlp_status tpmlp_fp4_tensor_scale(const tpmlp_fp4_quant* quant, const void* const* src, void* scale,
                                    void* stream);

/* Quantise by rows, by columns, or both in one read of src.  scale: g (nv), NULL (mx).
 * q_rows, s_rows, q_cols, s_cols: host arrays of `parts` device pointers (one with gather);
 * the row pair or the column pair may be NULL, not both. */
tpmlp_status tpmlp_fp4_quantize(const tpmlp_fp4_quant* quant, const void* const* src, const void* scale,
                                void* const* q_rows, void* const* s_rows, void* const* q_cols,
                                void* const* s_cols, void* stream);

/* The values of a 4-bit matrix [rows, k] in bf16, which holds them exactly (but those that
 * rounding took past its largest value, which become infinite). */
tpmlp_status tpmlp_fp4_dequantize(int64_t rows, int64_t k, int format, const void* q, const void* s,
                                  const void* scale, void* out, void* stream);

/* Bytes of scratch workspace a call with these dims needs: forward calls, or (backward != 0)
 * forward and backward calls.  0 for unsupported dims. */
size_t tpmlp_fp4_linear_workspace_bytes(const tpmlp_linear_dims* dims, int format, int backward);

/* Column parallel.  Forward:  Y_i = X.W_i + b[i*oi:(i+1)*oi], X quantised here by rows
 *   X          seq_chunks chunks of [Tc, in] bf16
 *   x_scale    g of X (nv; NULL for mx): read if x_calibrated, else computed and written
 *   Xq, Xs     X by columns (output, for the backward pass), or both NULL
 *   Wq, Ws     [t] shards W_i by columns ([oi, in]);  w_scale their g
 *   b          [out] bf16;  Y_shards [t] of [T, oi] bf16 (output)
 * Backward for upstream dY_i (bf16, quantised here both ways, g computed):
 *   dX = sum_i dY_i.W_i^T (bf16, seq_chunks chunks), dW_i = X^T.dY_i (fp32),
 *   db = column sums of the bf16 dY (fp32)
 *   Xq, Xs, x_scale  as the forward call left them
 *   Wq, Ws     [t] shards W_i by rows ([in, oi])
 * With T = 0 the forward does nothing and the backward zeroes dW and db.  Y may lie over X, and
 * dX over dY; nothing else that is written over anything else of the call. */
tpmlp_status tpmlp_fp4_column_linear_forward(const tpmlp_linear_dims* dims, int format,
                                             const void* const* X, void* x_scale, int x_calibrated,
                                             void* Xq, void* Xs, const void* const* Wq_shards,
                                             const void* const* Ws_shards, const void* w_scale,
                                             const void* b, void* const* Y_shards, void* workspace,
                                             void* stream);
tpmlp_status tpmlp_fp4_column_linear_backward(const tpmlp_linear_dims* dims, int format,
                                              const void* const* dY_shards, const void* Xq,
                                              const void* Xs, const void* x_scale,
                                              const void* const* Wq_shards, const void* const* Ws_shards,
                                              const void* w_scale, void* const* dX,
                                              void* const* dW_shards, void* db, void* workspace,
                                              void* stream);

/* Row parallel.  Forward:  Z = (sum_i X_i.W_i) + b
 *   X          [t] shards X_i [T, ii] bf16, with one x_scale
 *   Xq, Xs     [t] shards by columns (output), or both NULL
 *   Wq, Ws     [t] shards W_i by columns ([out, ii]);  Z seq_chunks chunks of [Tc, out] bf16
 * Backward for upstream dZ (seq_chunks chunks, bf16):
 *   dX_i = dZ.W_i^T (bf16 [T, ii]), dW_i = X_i^T.dZ (fp32 [ii, out]), db (fp32)
 *   Wq, Ws     [t] shards W_i by rows ([ii, out]) */
tpmlp_status tpmlp_fp4_row_linear_forward(const tpmlp_linear_dims* dims, int format,
                                          const void* const* X_shards, void* x_scale, int x_calibrated,
                                          void* const* Xq_shards, void* const* Xs_shards,
                                          const void* const* Wq_shards, const void* const* Ws_shards,
                                          const void* w_scale, const void* b, void* const* Z,
                                          void* workspace, void* stream);
tpmlp_status tpmlp_fp4_row_linear_backward(const tpmlp_linear_dims* dims, int format,
                                           const void* const* dZ, const void* const* Xq_shards,
                                           const void* const* Xs_shards, const void* x_scale,
                                           const void* const* Wq_shards, const void* const* Ws_shards,
                                           const void* w_scale, void* const* dX_shards,
                                           void* const* dW_shards, void* db, void* workspace,
                                           void* stream);

/* ---- Norms before and after a block, with its gate and residual scale ------------
 * What surrounds a block f in a residual stream X with a norm on both sides of it:
 *
 *   u   = N_post(Z)                                  Z = f(...), per token row over h
 *   Out = residual_scale * X + gate[row / gate_rows] * u      (bf16)
 *   Xn  = N_pre(Out)                                 the next block's input
 *
 *   rms    N(v) = v rstd gamma,                rstd = 1 / sqrt(mean(v^2) + eps)
 *   layer  N(v) = (v - mean) rstd gamma + beta, rstd = 1 / sqrt(var + eps), var biased
 *   none   post: u = Z;  pre: no Xn
 *
 * in one pass over the rows.  Xn is written in bf16, in 8 bits by rows (as the
 * 8-bit linear layers take it: the bf16 rounding of Xn, quantised), or both.
 * With Z = NULL there is no block before: Xn = N_pre(X), Out is X and not written
 * (post none, no gate, Out NULL; residual_scale is not used).
 *
 *   gate   bf16 [tokens / gate_rows, h]: one row for each run of gate_rows tokens (a
 *          sequence, or all tokens: gate_rows = tokens).  gate_rows = 0: no gate.
 *   stats  fp32 [4][tokens]: mean and rstd of Z's rows, mean and rstd of Out's (means
 *          of rms norms are 0; rows of kind none are not written).  Kept for the
 *          backward pass; NULL in the forward call: not wanted.
 *
 * Backward, for the gradients dOut of Out (NULL: none) and dXn of Xn:
 *   g = dOut + N_pre'(dXn),  dX = residual_scale * g,  dgate = sum of g * u over the
 *   gate's rows,  dZ = N_post'(gate * g),  and the weights' gradients.
 *   With Z = NULL:  dX = dOut + N_pre'(dXn), Out being X.
 * gamma, beta, gate bf16; their gradients fp32 (overwritten).  Pointers of what a
 * kind does not have must be NULL.  Statistics and sums are fp32, in a fixed order.
 * X, Z, Out, Xn and their gradients come in seq_chunks token chunks of tokens /
 * seq_chunks rows; Xq and Xs are whole.  hidden: a multiple of 8 (16 with Xq), at most
 * 16384; else TPMLP_ERR_UNSUPPORTED.  gate_rows divides tokens, eps >= 0, else
 * TPMLP_ERR_INVALID_ARG.  With tokens = 0 the forward does nothing and the backward
 * zeroes the gammas' and betas' gradients.  stats and Xs may start at any multiple of 4
 * bytes.  The workspace is scratch of one call. */
typedef enum {
    TPMLP_NORM_NONE = 0,
    TPMLP_NORM_RMS = 1,
    TPMLP_NORM_LAYER = 2
} tpmlp_norm_kind;

typedef struct {
    int64_t tokens, hidden;
    int64_t gate_rows;     /* tokens that share a row of the gate; 0 = no gate */
    int32_t seq_chunks;
    int32_t post, pre;     /* tpmlp_norm_kind */
    int32_t q_format;      /* tpmlp_fp8_format of Xq */
    float eps;
    float residual_scale;
} tpmlp_norm_params;

/* Bytes of workspace the backward call needs (0 for invalid params). */
size_t tpmlp_norm_workspace_bytes(const tpmlp_norm_params* params);

tpmlp_status tpmlp_norm_forward(const tpmlp_norm_params* params, const void* const* X,
                                const void* const* Z, const void* post_gamma,
                                const void* post_beta, const void* gate, const void* pre_gamma,
                                const void* pre_beta, void* const* Out, void* const* Xn, void* Xq,
                                void* Xs, void* stats, void* stream);

tpmlp_status tpmlp_norm_backward(const tpmlp_norm_params* params, const void* const* dOut,
                                 const void* const* dXn, const void* const* Z,
                                 const void* const* Out, const void* post_gamma,
                                 const void* post_beta, const void* gate, const void* pre_gamma,
                                 const void* stats, void* const* dX, void* const* dZ,
                                 void* dpost_gamma, void* dpost_beta, void* dgate,
                                 void* dpre_gamma, void* dpre_beta, void* workspace,
                                 void* stream);

/* ---- Norm of all gradients, and clipping by it -------------------------------------
 * Before an optimiser's step: the Euclidean norm of a list of gradients together, and
 *
 *   out = grad * min(1, max_norm / (norm + 1e-6))
 *
 * for each of them, in the gradient's own type (the product in fp32, rounded once).  out may
 * be grad itself; it may not lie over any other tensor of the list, nor may a tensor be in
 * the list twice.  Tensors are contiguous, of any size (0 too, and then any pointer), and start
 * on a multiple of their element's size.  Squares are summed in fp32 over at most 64 elements,
 * from there in two fp32 parts and in 64 bits (in 64 bits at once where fp32 would overflow or
 * lose them), in an order that depends on sizes and alignment alone.  A NaN makes the norm and everything clipped
 * NaN; an infinity makes the norm infinite and what is clipped 0 (infinities NaN).  In place,
 * gradients whose factor is 1 are not written.
 *   norm       fp32 [1] on the device (output; infinite where the norm is past fp32's range,
 *              which clipping is not bound to)
 *   max_norm   finite, >= 0
 *   workspace  tpmlp_grad_workspace_bytes(n) bytes of scratch of one call
 * At most 65536 tensors of at most 2^40 elements (else TPMLP_ERR_UNSUPPORTED). */
typedef enum {
    TPMLP_GRAD_F32 = 0,
    TPMLP_GRAD_BF16 = 1,
    TPMLP_GRAD_F16 = 2
} tpmlp_grad_type;

typedef struct {
    const void* grad;
    void* out;      /* read by tpmlp_grad_clip only */
    int64_t count;  /* elements */
    int32_t type;   /* tpmlp_grad_type */
} tpmlp_grad_tensor;

size_t tpmlp_grad_workspace_bytes(int64_t tensors);
tpmlp_status tpmlp_grad_norm(const tpmlp_grad_tensor* tensors, int64_t n, void* norm, void* workspace,
                             void* stream);
tpmlp_status tpmlp_grad_clip(const tpmlp_grad_tensor* tensors, int64_t n, float max_norm, void* norm,
                             void* workspace, void* stream);

/* Human-readable name of a status code (static storage, never NULL). */
const char* tpmlp_status_string(tpmlp_status s);

/* Synchronises the stream, then reports: TPMLP_ERR_CUDA if a CUDA error is
 * pending, TPMLP_ERR_TIMEOUT if a kernel of this library gave up on a bounded
 * wait since the last check (the device error word is then cleared), else
 * TPMLP_OK.  Kernels that time out stop early, leave their outputs
 * incomplete, release their tensor memory and return; the context stays
 * usable. */
tpmlp_status tpmlp_sync_check(void* stream);

/* Tail split of the GEMMs.  When a GEMM's output tiles do not fill the last
 * wave of CTA pairs, the K ranges of the leftover tiles are split across the
 * pairs that would otherwise idle; each part writes an fp32 partial tile into
 * the workspace and the last part to finish sums them in a fixed order (the
 * result stays bitwise reproducible) before the fused epilogue.  This is done
 * only for tiles at least `kblocks` 64-deep K steps long (default 128); 0
 * turns it off.  Affects launches enqueued after the call. */
tpmlp_status tpmlp_set_split_min_kblocks(int kblocks);

/* Head prefetch of the GEMMs: when a CTA pair starts a tile, it asks L2 for
 * the first `kblocks` 64-deep K steps of its next tile's operands, a whole
 * tile ahead of the loads that use them.  Helps GEMMs with short K ranges per
 * tile (the weight gradients, K = tokens), whose tile starts otherwise wait for
 * data fetched from DRAM; costs one extra TMA instruction per prefetched box.
 * 0 turns it off; 0..64, else TPMLP_ERR_INVALID_ARG.  Results do not depend on
 * it.  Affects launches enqueued after the call. */
tpmlp_status tpmlp_set_head_prefetch(int kblocks);

/* Tile width of the GEMMs with bf16 outputs (every GEMM but the weight
 * gradients).  A CTA pair computes either 256 x 256 output tiles (two
 * accumulators in tensor memory: a tile's epilogue runs under the next
 * tile's MMAs) or 256 x 512 tiles (one accumulator in two halves, K steps in
 * three phases so each half drains under MMAs on the other), which move a
 * quarter fewer operand bytes from L2 per FLOP.  mode 0 always 256; 1 picks
 * 512 where its tiles fill the GPU's waves at least as well as 256-wide ones;
 * 2 always 512; 3 (default) picks 512 for GEMMs of at least 256 K steps of 64
 * (summed over the row-parallel shards), where the one-half phases are a
 * small share and the lower operand traffic lowers the power drawn.  0 to 3,
 * else TPMLP_ERR_INVALID_ARG.  Half 0 of a wide tile sums K in the narrow
 * tile's order (bitwise equal columns); half 1 starts its sum further along K
 * (equal within rounding).  Affects launches enqueued after the call. */
tpmlp_status tpmlp_set_wide_tiles(int mode);

/* TMA tensor-map cache.  Every call encodes one tensor map per operand shard,
 * token chunk and output of each GEMM it launches; the library keeps the
 * encoded maps in a cache keyed by every argument of the encoding (base
 * address, element type, extents, strides, box, swizzle), so a repeated call
 * on the same buffers encodes nothing.  A buffer at a new address is a new key
 * (a stale entry is never used for another address); the operands of the 8-bit
 * and 4-bit layers share one map for each shape (4-bit shards that lie at equal steps, of whole
 * rows, one for each shape and step), and each call sets the address in its own copy.  At most
 * 4096 maps are kept; when the cache is full it is emptied.  Thread-safe (one mutex).
 * tpmlp_map_cache_stats reports the hits, misses (encodings) and entries so
 * far; any pointer may be NULL.  Always TPMLP_OK. */
tpmlp_status tpmlp_map_cache_stats(uint64_t* hits, uint64_t* misses, uint64_t* entries);

/* Self-test of the cache logic on the host (no GPU, no driver): runs a fixed
 * sequence against a private cache of capacity 4 with a stand-in encoder and
 * writes out[0..7] = hits, misses, encoder calls, final entries, 1 if a hit
 * returned the bytes of the first encoding, 1 if a new address gave another
 * map, the capacity, and the key size in bytes.  n >= 8, else
 * TPMLP_ERR_INVALID_ARG. */
tpmlp_status tpmlp_selftest_map_cache(uint64_t* out, int n);

/* Upper bound, in nanoseconds, on any single wait inside a kernel of this
 * library (default 2e9).  Affects launches enqueued after the call. */
tpmlp_status tpmlp_set_wait_timeout_ns(uint64_t ns);

/* Failure-detection self-test.  Runs one 128 x 256 x 64 GEMM tile whose
 * loader deliberately issues no loads, so the tensor-core issuer's wait on
 * its first stage can only end by the bounded-wait limit; the kernel then
 * records the timeout, drains, frees its tensor memory and returns.
 *   a  [128, 64] bf16 device buffer, b [256, 64] bf16, c [128, 256] bf16
 *   (valid buffers of at least those sizes; c may be partially written).
 * Synchronises the stream and returns what tpmlp_sync_check returns:
 * TPMLP_ERR_TIMEOUT when the failure was detected as designed. */
tpmlp_status tpmlp_selftest_stalled_gemm(const void* a, const void* b, void* c,
                                         uint64_t timeout_ns, void* stream);

/* The same for the products of the 8-bit and 4-bit linear layers, the quantisation to 4 bits in
 * tiles and the norms around a block:
 * after this call, those that the calling thread launches stop loading in the last
 * CTA of each cluster after `copies` (>= 0) steps (K blocks, or rows), so that what
 * waits for the rest gives up at the limit
 * (tpmlp_set_wait_timeout_ns) and tpmlp_sync_check returns TPMLP_ERR_TIMEOUT.
 * -1: they load everything again (default). */
tpmlp_status tpmlp_selftest_stall_loads(int copies);

/* Explicit sequence-parallel gather and scatter ("Megatron-LM：NVIDIA 的大规模
 * 并行训练方案", 并行训练范式 / 序列并行: the tensor-parallel block gathers the
 * sequence chunks before its column-parallel GEMM and reduce-scatters its
 * output to them after the row-parallel GEMM).  tpmlp_forward / tpmlp_backward
 * do both without copies, through one tensor map per chunk and an epilogue that
 * writes each row into its chunk; these calls make the copies explicit.
 *   tpmlp_sp_gather:  out[T, cols] = concatenation along tokens of the
 *                     dims->seq_chunks chunks [T / seq_chunks, cols]
 *   tpmlp_sp_scatter: chunk j = rows [j T / seq_chunks, (j + 1) T / seq_chunks)
 *                     of in[T, cols]
 * bf16 (any 2-byte element), row-major, cols a multiple of 8 (else
 * TPMLP_ERR_UNSUPPORTED), 16-byte-aligned device pointers, at most 8 chunks;
 * dims->tokens and dims->seq_chunks are read, the rest of dims is not.  One
 * kernel on `stream`, asynchronous; nothing is allocated. */
tpmlp_status tpmlp_sp_gather(const tpmlp_dims* dims, const void* const* chunks, int64_t cols,
                             void* out, void* stream);
tpmlp_status tpmlp_sp_scatter(const tpmlp_dims* dims, const void* in, int64_t cols,
                              void* const* chunks, void* stream);

/* Column sums of one bf16 matrix [rows, cols] into fp32 out[cols] -- the
 * reduction tpmlp_backward uses for its bias gradients (db2 is the column
 * sums of dZ) -- for callers that cannot allocate device memory.  The pages
 * have no counterpart to this call; it exists for the library's users.
 *
 * Who needs it: tpmlp_backward takes its scratch from a caller-allocated
 * workspace.  A caller embedded in another runtime whose device memory is
 * owned by that runtime's pool cannot add a cudaMalloc of its own (it would
 * escape the pool's budget, and cudaFree synchronises the whole device); a
 * latency-critical loop may forbid allocation after start-up.  This call
 * allocates nothing: it keeps its partial sums in a static 4 MiB device
 * array (1,048,576 floats) inside the library, which every GPU that loads the
 * library holds until the process exits.
 *   src   device bf16 [rows, cols], row-major, 16-byte aligned
 *   rows  >= 0 (rows = 0 writes zeros), below 2^31
 *   cols  multiple of 8, at most 1,048,576; larger returns TPMLP_ERR_UNSUPPORTED
 *   out   device fp32 [cols], 16-byte aligned, overwritten
 * The first call on a device does a one-time set-up (looks up the array's
 * device address); make that first call before any stream capture.  All
 * calls on a device share the array and the last call's contents stay in it;
 * nothing in it needs clearing, but calls that overlap on the GPU (unordered
 * streams) race on it.  Asynchronous on `stream`, like every other call. */
tpmlp_status tpmlp_column_sums_noalloc(const void* src, int64_t rows, int64_t cols, void* out,
                                       void* stream);

/* Kernel-level timing.  Between tpmlp_profile_begin and tpmlp_profile_end
 * the library records a CUDA event pair on the launch stream around each of
 * its kernel launches (at most `capacity` launches).  tpmlp_profile_end
 * synchronises on those events and writes, for each kernel kind k <
 * nkinds, the summed milliseconds ms[k] and the launch count launches[k];
 * it returns the number of launches recorded, or -1 on error. */
enum {
    TPMLP_KERNEL_COLUMN_FWD = 0,  /* Y_i = X.A_i + b1, H_i = GeLU(Y_i) */
    TPMLP_KERNEL_ROW_FWD = 1,     /* Z = sum_i H_i.B_i + b2 */
    TPMLP_KERNEL_DGRAD_H = 2,     /* dY_i = (dZ.B_i^T) * GeLU'(Y_i) */
    TPMLP_KERNEL_DGRAD_X = 3,     /* dX = sum_i dY_i.A_i^T */
    TPMLP_KERNEL_WGRAD_B = 4,     /* dB_i = H_i^T.dZ */
    TPMLP_KERNEL_WGRAD_A = 5,     /* dA_i = X^T.dY_i */
    TPMLP_KERNEL_BIAS_GRAD = 6,   /* db1, db2, linear db column sums; gradient norm and clipping (all launches) */
    TPMLP_KERNEL_LINEAR_FWD = 7,  /* linear layers (bf16, 8-bit, 4-bit): Y_i = X.W_i + b, Z = sum_i X_i.W_i + b */
    TPMLP_KERNEL_LINEAR_DGRAD = 8,  /* linear layers (bf16, 8-bit, 4-bit): dX = sum_i dY_i.W_i^T, dX_i = dZ.W_i^T (4-bit: and db) */
    TPMLP_KERNEL_LINEAR_WGRAD = 9,  /* linear layers (bf16, 8-bit, 4-bit): dW_i */
    TPMLP_KERNEL_LAYERNORM_FWD = 10,  /* sequence-parallel sublayer: LN(X) and row statistics; tpmlp_norm_forward */
    TPMLP_KERNEL_LAYERNORM_BWD = 11,  /* sequence-parallel sublayer: dX, dgamma, dbeta (2 launches; 3 for h > 4096); tpmlp_norm_backward (2; 1 with no norm and no gate to add up) */
    TPMLP_KERNEL_DROPOUT_BWD = 12,    /* sequence-parallel sublayer: dZ from dOut and the mask, db2 (2 launches) */
    TPMLP_KERNEL_SP_COPY = 13,        /* tpmlp_sp_gather / tpmlp_sp_scatter, 8-bit and 4-bit quantisation and back */
    TPMLP_KERNEL_KINDS = 14
};
tpmlp_status tpmlp_profile_begin(int capacity);
/* The same, with event pairs only around the launches of the kernel kinds
 * whose bits are set in `kinds` (bit k = kind k): timing one kind costs the
 * others no event records.  TPMLP_ERR_INVALID_ARG for capacity <= 0, kinds
 * == 0 or a bit at or above TPMLP_KERNEL_KINDS. */
tpmlp_status tpmlp_profile_begin_kinds(int capacity, uint32_t kinds);
int tpmlp_profile_end(double* ms, int* launches, int nkinds);
const char* tpmlp_kernel_name(int kind);

#ifdef __cplusplus
}
#endif

#endif /* TPMLP_H */
