// norm_residual.cuh -- norms before and after a block, fused with its gate and
// residual scale:
//
//   u   = N_post(Z)                      the block's output, normalised per token row
//   Out = alpha X + gate[row / gate_rows] * u     (bf16)
//   Xn  = N_pre(Out)                     the next block's input (bf16, and / or 8-bit
//                                        with a scale for each 128 of a row)
//   rms    N(v) = v rstd gamma                    rstd = 1 / sqrt(mean(v^2) + eps)
//   layer  N(v) = (v - mean) rstd gamma + beta    rstd = 1 / sqrt(var + eps), var biased
//
// and the gradients
//
//   g      = dOut + N_pre'(dXn)          dX = alpha g
//   dgate  = sum over the gate's rows of g * u
//   dZ     = N_post'(gate * g)
//   N'(dy) = rstd (w - vhat mean(w vhat) [- mean(w), layer]),  w = dy gamma,
//            vhat = (v - mean) rstd,  dgamma = sum dy vhat,  dbeta = sum dy
//
// Statistics, products and sums are fp32; Out is rounded to bf16 before N_pre
// reads it, so that its statistics are those of the stored rows.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

namespace tpmlp {

constexpr int NR_MAX_CHUNKS = 8;
constexpr int NR_MAX_H = 16384;
constexpr int NR_MAX_UNITS = 192;  // most CTAs of the backward pass that run at once: one on an SM

// N_post: no Z at all (Out is X, not written), identity, rms, layer;  N_pre: none, rms, layer
enum NrPost : int { NR_ABSENT = 0, NR_IDENTITY = 1, NR_POST_RMS = 2, NR_POST_LAYER = 3 };
enum NrPre : int { NR_NONE = 0, NR_PRE_RMS = 1, NR_PRE_LAYER = 2 };

struct NrChunks {
    const void* p[NR_MAX_CHUNKS];
};

struct NrForwardParams {
    NrChunks x, z;
    void* out[NR_MAX_CHUNKS];
    void* xn[NR_MAX_CHUNKS];     // [0] null: not wanted
    const void *post_gamma, *post_beta, *pre_gamma, *pre_beta;  // bf16 [h]
    const void* gate;            // bf16 [T / gate_rows, h] or null
    uint8_t* q;                  // 8-bit [T, h] or null
    float* q_scale;              // [ceil(h / 128)][T]
    float* stats;                // [4][T]: mean and rstd of Z, mean and rstd of Out; or null
    long long T, rows_per_chunk, gate_rows;
    int h, q_format;
    float eps, alpha;
    unsigned int* err;           // the device error word and the limit of any one wait
    unsigned long long timeout_ns;
    int stall;                   // failure-detection self-test: rows that a CTA copies; < 0: all
};

struct NrBackwardParams {
    NrChunks dout, dxn, z, out;  // dout.p[0] null: zero
    void* dx[NR_MAX_CHUNKS];
    void* dz[NR_MAX_CHUNKS];
    const void *post_gamma, *post_beta, *pre_gamma, *gate;
    const float* stats;
    float* part;                 // partial sums [blocks][vectors][h]
    float *dpost_gamma, *dpost_beta, *dpre_gamma, *dpre_beta, *dgate;
    long long T, rows_per_chunk, gate_rows;
    int h;
    float alpha;
    // rows of a block: see nr_plan
    long long seqs, blocks, rows_per_block, seqs_per_group;
    int blocks_per_seq;
    unsigned int* err;           // the device error word and the limit of any one wait
    unsigned long long timeout_ns;
    int stall;                   // failure-detection self-test: row pairs that each group of a cluster's
                                 // last CTA copies; < 0: all
};

cudaError_t launch_nr_forward(const NrForwardParams& p, int post, int pre, int sm_count,
                              cudaStream_t st);
// The rows, and, if there are any, the sums over the row blocks: up to two launches.
cudaError_t launch_nr_backward(const NrBackwardParams& p, int post, int pre, cudaStream_t st);

// Row blocks of the backward pass.  A block never holds part of one gate's rows
// and part of another's: with few gates each gate's rows are cut into
// blocks_per_seq blocks, with many each group of a block's threads takes
// seqs_per_group whole gates (blocks_per_seq = 0).
cudaError_t nr_plan(NrBackwardParams& p, int sm_count);
// The most bytes of partial sums a backward pass of this width needs.
size_t nr_partial_bytes(long long h);

}  // namespace tpmlp
