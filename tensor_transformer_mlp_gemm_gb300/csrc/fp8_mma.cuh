// fp8_mma.cuh -- device pieces of the 8-bit products: the tcgen05 instructions
// for 8-bit operands with block scales, the scales' way into tensor memory, and
// bounded waits.
//
// tcgen05.mma.kind::mxf8f6f4.block_scale multiplies every 32 elements of K of a
// row of A and of B by a power of two each, given as 8-bit exponents (biased by
// 127, 255 = NaN) in tensor memory, and accumulates in fp32.  A scale of 128
// elements is that of its four slices of 32.
//
// Scales of 128 rows take 4 columns of tensor memory: row r in lane r % 32,
// column r / 32, and the 32 lanes' words again in each of the other three
// quarters of the lanes.  A word holds four exponents, of which the instruction
// picks one; here all four are the same.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "fp8_gemm.cuh"
#include "gemm_params.h"
#include "ptx.cuh"

namespace tpmlp {
namespace f8 {

// D[tmem] (+)= (A x scale_A) x (B x scale_B); the pair form is issued by the even
// CTA and takes each CTA's own rows of A with their scales, and from each CTA half
// the rows of B, whose scales both CTAs hold in full.
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, uint32_t sa_tmem, uint32_t sb_tmem,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate)
        : "memory");
}

// The same on one CTA (its own 128 rows of A, all rows of B).
__device__ __forceinline__ void mma_one(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t sa_tmem, uint32_t sb_tmem,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate)
        : "memory");
}

// Instruction descriptor of kind::mxf8f6f4 with an fp32 accumulator.
//   bits 4-5, 29-30 which exponent of a scale word is B's, A's (the first);
//   7-9 A format, 10-12 B format (0 = e4m3, 1 = e5m2); bit 15 A is MN-major, 16 B;
//   17-22 N >> 3; bit 23 the scales are 8-bit exponents; 27-28 M >> 7.
__host__ __device__ constexpr uint32_t idesc(int M, int N, int a_mn, int b_mn) {
    return (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
           (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(M >> 7) << 27);
}

// Descriptor of the 32-wide K slice kk (0..3) of a 128 x 128-byte operand box.
//   K-major:  rows of 128 bytes, 8-row swizzle atoms every 1024 bytes; the slice
//             starts 32 bytes further along the row.
//   MN-major: 128 K rows of 128 bytes, 8-row atoms every 1024 bytes; the slice
//             starts 32 rows (4096 bytes) further down.
__device__ __forceinline__ uint64_t operand_desc(uint32_t tile, int kk, int mn) {
    return ptx::smem_desc_sw128(tile + (mn ? kk * 4096 : kk * 32), mn ? F8_BOX_BYTES : 16, 1024);
}

// A scale's word: its exponent four times; NaN (255) for anything but a positive
// power of two of 2^-126 .. 2^127.
__device__ __forceinline__ uint32_t scale_word(uint32_t bits) {
    const uint32_t e = (bits & 0x807FFFFFu) == 0 && bits != 0 ? bits >> 23 : 255u;
    return __byte_perm(e, 0, 0);
}

// This thread's lane of its warp's quarter: 1, 4 and 8 consecutive columns.
__device__ __forceinline__ void store_col(uint32_t taddr, uint32_t v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(v) : "memory");
}
__device__ __forceinline__ void store_cols4(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                 : "memory");
}
__device__ __forceinline__ void store_cols8(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
        : "memory");
}
__device__ __forceinline__ void store_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// The same on this CTA's own mbarrier.
__device__ __forceinline__ void arrive_relaxed(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// One lane of the (converged) warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

// Waits for phase `parity` of `bar`; gives up (false) when another role has, or
// after the limit (then this one aborts the CTA and sets `code` in the error word).
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                     unsigned long long timeout_ns, unsigned* err, unsigned code) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
    while (true) {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (ptx::globaltimer_ns() - t0 > timeout_ns) {
            *abort_flag = 1;
            atomicOr(err, code);
            return false;
        }
    }
}

// Teardown wait for what this CTA has under way itself: ignores the abort flag.  Copies and
// MMAs end by themselves, so its limit is not the caller's where that is short.
constexpr unsigned long long DRAIN_NS = 1000000000ULL;
__device__ __forceinline__ bool drain(uint32_t bar, uint32_t parity, unsigned long long timeout_ns,
                                      unsigned* err) {
    const uint64_t t0 = ptx::globaltimer_ns();
    while (!ptx::mbar_try_wait(bar, parity)) {
        if (ptx::globaltimer_ns() - t0 > max(timeout_ns, DRAIN_NS)) {
            atomicOr(err, ERR_DRAIN);
            return false;
        }
    }
    return true;
}

// Arrive on an mbarrier of either CTA of the pair without ordering this thread's
// memory accesses: it only says that tensor memory has been read or written,
// which the waits and the fence before it order.  (A release at cluster scope
// waits for the thread's outstanding global loads too: 2000 clocks, measured.)
__device__ __forceinline__ void arrive_relaxed_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
                 : "memory");
}

// A word or two into shared memory of either CTA of the pair.
__device__ __forceinline__ void store_cluster(uint32_t cluster_addr, int v) {
    asm volatile("st.relaxed.cluster.shared::cluster.b32 [%0], %1;" ::"r"(cluster_addr), "r"(v)
                 : "memory");
}
__device__ __forceinline__ void store_cluster64(uint32_t cluster_addr, long long v) {
    asm volatile("st.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(cluster_addr), "l"(v)
                 : "memory");
}

// Takes bytes that no copy will bring off what the mbarrier's phase waits for.
__device__ __forceinline__ void complete_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

// Barrier 1 of `threads` threads of the CTA; whether any of them came with `fail`.
template <int THREADS>
__device__ __forceinline__ bool barrier_any(bool fail) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred q, r;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "barrier.cta.red.or.pred r, 1, %2, q;\n\t"
        "selp.u32 %0, 1, 0, r;\n\t}"
        : "=r"(r)
        : "r"(fail ? 1u : 0u), "n"(THREADS)
        : "memory");
    return r != 0;
}

// ---- asynchronous 4-byte copies into shared memory (zero where !in) ------------------
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
                 "r"(in ? 4 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Registers per thread of the calling warpgroup (all of its warps call it).
template <int N>
__device__ __forceinline__ void reg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// 32 columns of this thread's tensor-memory lane into v (usable after load_wait).
__device__ __forceinline__ void load_cols(uint32_t taddr, float* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
          "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
          "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]),
          "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]),
          "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr));
}

// 16 columns of this thread's tensor-memory lane into v (usable after load_wait).
__device__ __forceinline__ void load_cols16(uint32_t taddr, float* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
          "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
          "=f"(v[14]), "=f"(v[15])
        : "r"(taddr));
}

}  // namespace f8
}  // namespace tpmlp
