// attn_common.cuh -- what the attention kernels share: paired fp32 arithmetic,
// operand offsets, tensor-memory stores, MMAs whose A operand lies in tensor
// memory, and the forward kernels' layout.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"

namespace tpmlp {
namespace {

constexpr int kRowBytes = 128;  // one 64-column bf16 box row (the swizzle width)

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 values in one 64-bit register, for the paired fp32 instructions
// (one issue slot for two FMAs or two adds).
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f32x2_split(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Byte offset of UMMA k-step kk (16 elements) inside a K-major operand tile
// of R rows stored as 64-column boxes (R x 128 B each): box kk/4, 32 B a step.
template <int R>
__device__ __forceinline__ uint32_t kmajor_step(int kk) {
    return static_cast<uint32_t>((kk >> 2) * (R * kRowBytes) + (kk & 3) * 32);
}

// Byte offset of UMMA k-step kk of an MN-major operand whose K runs along the
// box rows: 16 rows of 128 B.
__device__ __forceinline__ uint32_t mnmajor_step(int kk) {
    return static_cast<uint32_t>(kk * 16 * kRowBytes);
}

__device__ __forceinline__ uint64_t desc_add(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }

// Stores 32 consecutive 32-bit TMEM columns of this thread's lane (same
// lane quadrant rule as tmem_ld32).
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0],"
        " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16,"
        " %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}


// D[tmem] (+)= A[tmem] * B[smem]^T, bf16 x bf16 -> f32: the A operand (128
// rows = TMEM lanes, 16 k values packed two bf16 to a 32-bit column, low
// half first) is read from tensor memory.
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 16 consecutive 32-bit TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0],"
        " {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
}

// tcgen05 MMA chain D (+)= A B^T with A in tensor memory (k-step kk reads the
// 8 columns a_tmem + 8 kk) and B MN-major along d in shared memory (the value
// or query/key tile as the N operand, N = d): the N extent is issued as a
// multiple of 64 (whole swizzle atoms, `box_bytes` apart) plus a 32-wide
// tail, so that no MMA spans part of an atom.  The tail (d % 64 == 32) goes
// to columns d_tail (d_tmem + the whole atoms' width unless given).
template <int D, int KSTEPS>
__device__ __forceinline__ void mma_ts_n_is_d(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                              uint32_t box_bytes, bool accumulate_first,
                                              uint32_t d_tail = 0xFFFFFFFFu) {
    constexpr int N1 = (D / 64) * 64;
    constexpr int N2 = D - N1;
    constexpr uint32_t id1 = idesc_bf16_f32(128, N1 > 0 ? N1 : 64, false, true);
    constexpr uint32_t id2 = idesc_bf16_f32(128, N2 > 0 ? N2 : 32, false, true);
#pragma unroll
    for (int kk = 0; kk < KSTEPS; ++kk) {
        const uint32_t acc = (accumulate_first || kk > 0) ? 1u : 0u;
        const uint64_t bd = desc_add(b_desc, mnmajor_step(kk));
        if constexpr (N1 > 0) tc_mma_f16_ts(d_tmem, a_tmem + 8 * kk, bd, id1, acc);
        if constexpr (N2 > 0)
            tc_mma_f16_ts(d_tail == 0xFFFFFFFFu ? d_tmem + N1 : d_tail, a_tmem + 8 * kk,
                          desc_add(bd, (N1 / 64) * box_bytes), id2, acc);
    }
}

// The forward kernels (two query tiles A and B in ping-pong).
constexpr int kFwdThreads = 320;  // 8 softmax warps, producer, MMA
constexpr float kRescaleLog2 = 8.0f;  // keep a stale row max while it is within 2^8

template <int D>
struct FwdCfg {
    static constexpr int NB = (D + 63) / 64;            // 64-column boxes per row
    static constexpr int BKV = D <= 128 ? 128 : 64;     // keys per K/V tile
    static constexpr int QTILE = NB * 128 * kRowBytes;  // 128 query rows x D (box-padded)
    static constexpr int KVTILE = NB * BKV * kRowBytes;
    static constexpr int FIXED = 2 * QTILE;
    static constexpr int STAGES_FIT = (225 * 1024 - FIXED) / KVTILE;
    static constexpr int STAGES = STAGES_FIT > 6 ? 6 : STAGES_FIT;
    static constexpr int SMEM = 1024 + FIXED + STAGES * KVTILE + 256;
    // TMEM columns of tile x.  d <= 128: S at 256 x, O at 256 x + 128 (its
    // 32-wide tail, d = 96, right after).  d = 160: S at 64 x, the 128-column
    // part of O at 128 + 128 x and its 32-column tail at 384 + 32 x, so that
    // every N >= 128 accumulator part starts on a multiple of 128.
    static constexpr uint32_t s_col(int x) { return D <= 128 ? 256u * x : 64u * x; }
    static constexpr uint32_t o_col(int x) { return D <= 128 ? 256u * x + 128u : 128u + 128u * x; }
    static constexpr uint32_t o_tail(int x) {
        return D <= 128 ? o_col(x) + (D / 64) * 64 : 384u + 32u * x;
    }
    // column of 32-column chunk c of O_x
    static constexpr uint32_t o_chunk(int x, int c) {
        return c < (D / 64) * 2 ? o_col(x) + 32u * c : o_tail(x) + 32u * (c - (D / 64) * 2);
    }
};

}  // namespace
}  // namespace tpmlp
