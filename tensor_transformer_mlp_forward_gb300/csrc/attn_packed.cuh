// attn_packed.cuh -- work items of the packed attention kernels.
//
// A packed batch is a [T, heads, d] matrix of tokens in which sequence i owns
// rows cu_seqlens[i] .. cu_seqlens[i + 1] - 1.  The kernels' work is cut into
// tiles of `tile` tokens of one sequence; the list of tiles is made on the
// device, because the offsets live there: a sequence of n tiles has entries of
// rank 1 .. n (rank = how many of the sequence's tiles a causal forward tile
// sees, or how many see a key tile), and the list holds the highest ranks
// first, so that the persistent kernels take the heaviest items first.
#pragma once

#include <atomic>

#include "attn_common.cuh"

namespace tpmlp {
namespace {

constexpr int kPlanShared = 4096;  // ranks that one CTA counts in shared memory
constexpr int kStatusShape = 2;    // TPMLP_ERR_SHAPE

// The header words of a plan: item counters of the kernels that take its
// items, and the number of entries.
enum { kPlanWork0 = 0, kPlanWork1 = 1, kPlanCount = 2 };

// Inclusive prefix sum over the CTA's threads; *total is the sum of all.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();  // the last call's sums have been read
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < warps; ++w) {
        const int s = warp_sums[w];
        before += w < warp ? s : 0;
        all += s;
    }
    *total = all;
    return v + before;
}

// One CTA (whole warps).  entries: {first row, length, rank - 1, tiles of the
// sequence}, packed_attn_entries(nb, T, tile) at most; `ranks` holds
// packed_attn_ranks(T) words, used beyond kPlanShared ranks.
// Offsets that leave [0, T] or fall make an empty list and set the device
// status word.
__device__ __forceinline__ void plan_block(const int* __restrict__ cu, int nb, int T, int tile,
                                           int4* __restrict__ entries, unsigned* __restrict__ head,
                                           int* __restrict__ ranks, int* status) {
    __shared__ int s_count[kPlanShared + 1];
    __shared__ int s_sums[32];
    __shared__ int s_most, s_bad;
    const int tid = threadIdx.x, nt = blockDim.x;
    const int most = T / tile + 1;  // a sequence has at most this many tiles
    int* count = most <= kPlanShared ? s_count : ranks;
    for (int r = tid; r <= most; r += nt) count[r] = 0;
    if (tid == 0) s_most = s_bad = 0;
    __syncthreads();
    for (int i = tid; i < nb; i += nt) {
        const int a = cu[i], b = cu[i + 1];
        if (a < 0 || b < a || b > T) {
            s_bad = 1;
        } else if (b > a) {
            const int n = (b - a + tile - 1) / tile;
            atomicAdd(&count[n], 1);
            atomicMax(&s_most, n);
        }
    }
    __syncthreads();
    if (s_bad) {
        if (tid == 0) {
            head[kPlanWork0] = head[kPlanWork1] = head[kPlanCount] = 0u;
            atomicCAS(status, 0, kStatusShape);  // a timeout that nobody has read yet stays
        }
        return;
    }
    // first[r]: entries of higher rank, i.e. over r' > r of sequences with >= r' tiles
    int longer = 0, above = 0;
    for (int top = s_most; top >= 1; top -= nt) {
        const int r = top - tid;
        int all;
        const int c = longer + block_scan(r >= 1 ? count[r] : 0, s_sums, &all);
        longer += all;
        const int mine = r >= 1 ? c : 0;
        const int upto = above + block_scan(mine, s_sums, &all);
        above += all;
        if (r >= 1) count[r] = upto - mine;
    }
    __syncthreads();
    if (tid == 0) {
        head[kPlanWork0] = head[kPlanWork1] = 0u;
        head[kPlanCount] = static_cast<unsigned>(above);
    }
    // a warp per sequence, or the whole CTA where there are fewer sequences
    const int team = nb < nt / 32 ? nt : 32;
    for (int i = tid / team; i < nb; i += nt / team) {
        const int a = cu[i], len = cu[i + 1] - a, n = (len + tile - 1) / tile;
        for (int r = 1 + tid % team; r <= n; r += team)
            entries[atomicAdd(&count[r], 1)] = make_int4(a, len, r - 1, n);
    }
}

// Waits of these kernels' roles, by polls (a failing one sleeps 4 us, so the limit is
// that of the timed waits).  The roles run different code on one SM and push each
// other's out of the instruction caches: a wait that inlines the timed loops took
// 250 clocks when its phase was complete, this one takes 64.
__device__ __noinline__ void give_up(volatile uint32_t* abort, int* status, int site) {
    *abort = 1u;
    atomicExch(status, kStatusTimeout);
    atomicCAS(status + 1, 0, site);
}

// One thread.
__device__ __forceinline__ bool thread_wait(uint64_t* bar, uint32_t parity, volatile uint32_t* abort, int* status,
                                            int site) {
#pragma unroll 1
    for (int i = 0; !mbar_try_wait(bar, parity); ++i) {
        if (*abort) return false;
        if (i >= kPollLimit) {
            give_up(abort, status, site);
            return false;
        }
    }
    return true;
}

// Whether both phases are complete (or sleeps on one of them): the two polls are on
// their way together, so that a wait for two costs little more than a wait for one.
__device__ __forceinline__ bool mbar_try_wait_both(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
        "and.pred p, p, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(a)), "r"(pa), "r"(smem_u32(b)), "r"(pb)
        : "memory");
    return ok != 0;
}

// A whole warp, whose lanes poll and leave together.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile uint32_t* abort, int* status,
                                          int site) {
#pragma unroll 1
    for (int i = 0; !__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity)); ++i) {
        if (__any_sync(0xFFFFFFFFu, *abort != 0u || i >= kPollLimit)) {
            if (i >= kPollLimit) give_up(abort, status, site);
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ bool warp_wait_both(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb,
                                               volatile uint32_t* abort, int* status, int site) {
#pragma unroll 1
    for (int i = 0; !__all_sync(0xFFFFFFFFu, mbar_try_wait_both(a, pa, b, pb)); ++i) {
        if (__any_sync(0xFFFFFFFFu, *abort != 0u || i >= kPollLimit)) {
            if (i >= kPollLimit) give_up(abort, status, site);
            return false;
        }
    }
    return true;
}

// MMAs and commits issued by a converged warp, one elected lane doing it (the same one
// each time, so that they run in order).  Operands of an MMA live in uniform registers:
// in a branch that a single lane takes the compiler moves each of them there one by
// one, 63 to 67 clocks an MMA, more than the 64 that a 128 x 128 x 16 one runs; a warp
// that stays together spends 40.
// Descriptors: low word {address, leading offset}, high word as below (rows of 128
// bytes, swizzled, 8 rows = 1024 bytes apart).
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);

__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t lbo) {
    return ((saddr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}

__device__ __forceinline__ void warp_mma_ss(uint32_t d_tmem, uint32_t a_low, uint32_t b_low, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
        "elect.sync _|e, 0xFFFFFFFF;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 da, {%1, %4};\n\t"
        "mov.b64 db, {%2, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_low), "r"(b_low), "r"(idesc), "n"(kDescHigh), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void warp_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_low, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 db;\n\t"
        "elect.sync _|e, 0xFFFFFFFF;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 db, {%2, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_low), "r"(idesc), "n"(kDescHigh), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void warp_commit(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xFFFFFFFF;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xFFFFFFFF;\n\t"
        "@e mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}

// D = A B^T over the head dim: A 128 rows, B N rows, both K-major boxes.
template <int D, int N>
__device__ __forceinline__ void warp_mma_scores(uint32_t d_tmem, uint32_t a_low, uint32_t b_low) {
    constexpr uint32_t id = idesc_bf16_f32(128, N, false, false);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
        warp_mma_ss(d_tmem, a_low + (kmajor_step<128>(kk) >> 4), b_low + (kmajor_step<N>(kk) >> 4), id, kk > 0 ? 1u : 0u);
}

// D (+)= A B^T with A packed bf16 in tensor memory (K columns; k-steps of 8 columns,
// those of the second half of K from a_tmem + HALF on) and B a tile of K rows, MN-major
// along the head dim: N in whole 64-wide swizzle atoms, then a 32-wide tail.
template <int D, int K, int HALF>
__device__ __forceinline__ void warp_mma_values(uint32_t acc, uint32_t tail, uint32_t a_tmem, uint32_t b_low,
                                                bool accumulate) {
    constexpr int N1 = (D / 64) * 64, N2 = D - N1, STEPS = K / 16;
    constexpr uint32_t id1 = idesc_bf16_f32(128, N1, false, true);
    constexpr uint32_t id2 = idesc_bf16_f32(128, N2 > 0 ? N2 : 32, false, true);
#pragma unroll
    for (int kk = 0; kk < STEPS; ++kk) {
        const uint32_t on = (accumulate || kk > 0) ? 1u : 0u;
        const uint32_t at = a_tmem + (kk / (STEPS / 2)) * HALF + (kk % (STEPS / 2)) * 8;
        const uint32_t bl = b_low + (mnmajor_step(kk) >> 4);
        warp_mma_ts(acc, at, bl, id1, on);
        if constexpr (N2 > 0) warp_mma_ts(tail, at, bl + (N1 / 64) * (K * kRowBytes >> 4), id2, on);
    }
}

// Tensor-memory loads and stores are instructions of the whole warp, and the compiler may
// leave lanes apart after a branch by lane (a causal mask, a row behind the end): they are
// brought together first.
__device__ __forceinline__ void warp_tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    __syncwarp();
    tmem_ld32(taddr, r);
}
__device__ __forceinline__ void warp_tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    __syncwarp();
    tmem_st32(taddr, r);
}
__device__ __forceinline__ void warp_tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    __syncwarp();
    tmem_st16(taddr, r);
}

// The end of a wait for tensor-memory loads, with their registers passing through it: what
// is computed from them cannot be moved in front of the wait.
__device__ __forceinline__ void tmem_loaded(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                   "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                   "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
                 :
                 : "memory");
}

// Zeroes rows first .. rows - 1 of an operand tile of NB 64-column boxes in
// shared memory (a box row is 128 bytes whatever the swizzle does within it),
// by `threads` threads, and makes the zeros visible to the tensor cores.
// Rows behind a sequence's end belong to the next sequence: their weights are
// exact zeros, but zero times an infinity or NaN of theirs would be NaN.
template <int NB>
__device__ __forceinline__ void zero_rows(uint32_t tile, int rows, int first, int tid, int threads) {
    const int chunks = (rows - first) * 8;  // 16-byte chunks of a box
    for (int c = tid; c < chunks; c += threads)
#pragma unroll
        for (int b = 0; b < NB; ++b)
            st_shared_v4(tile + static_cast<uint32_t>((b * rows + first) * kRowBytes + c * 16), 0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
}

// The rounding of a pair of fp32 values times `f` to packed bf16.
__device__ __forceinline__ uint32_t pack_scaled(uint32_t lo, uint32_t hi, float f) {
    return pack_bf16x2(__uint_as_float(lo) * f, __uint_as_float(hi) * f);
}

// 32 bytes, to an address on a 32-byte boundary (wide) or a 16-byte one.
__device__ __forceinline__ void store_32(void* p, const uint32_t (&w)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// Where a warp's 32 accumulator rows go: rows of a matrix one after another, `ld`
// values apart, the first `valid` of them.
struct RowsOut {
    __nv_bfloat16* row;  // this lane's
    long long ld;
    int valid;           // rows from this warp's first row on
    bool wide;           // rows start on 32-byte boundaries

    __device__ __forceinline__ RowsOut(__nv_bfloat16* base, long long ld_, long long first_row, int col, int valid_)
        : row(base + (first_row + (threadIdx.x & 31)) * ld_ + col), ld(ld_), valid(valid_),
          wide(((reinterpret_cast<uintptr_t>(base) | static_cast<uintptr_t>(ld_ * 2)) & 31u) == 0) {}

    // Columns [32 c, 32 c + 32) of this lane's row, 16 packed words.  A lane's stores
    // to its own row alone would touch 32 lines an instruction (a read-out of 128
    // columns took 3600 clocks): neighbours exchange half a chunk, so that two lanes
    // write 64 bytes of one row, in 32-byte stores.
    __device__ __forceinline__ void store(int c, const uint32_t (&w)[16]) const {
        const int lane = threadIdx.x & 31;
        const bool odd = lane & 1;
        uint32_t even_row[8], odd_row[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, odd ? w[i] : w[8 + i], 1);
            even_row[i] = odd ? got : w[i];
            odd_row[i] = odd ? w[8 + i] : got;
        }
        const int even = lane & ~1;
        __nv_bfloat16* at = row + 32 * c + (odd ? 16 : 0);
        if (even < valid) store_32(odd ? at - ld : at, even_row, wide);
        if (even + 1 < valid) store_32(odd ? at : at + ld, odd_row, wide);
    }
};

// Scales and rounds accumulator chunk c (32 columns from `addr` on) and stores it.
__device__ __forceinline__ void read_out(const RowsOut& out, int c, uint32_t addr, float f) {
    uint32_t v[32], w[16];
    warp_tmem_ld32(addr, v);  // warp-collective: every lane loads
    tmem_loaded(v);
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack_scaled(v[2 * i], v[2 * i + 1], f);
    out.store(c, w);
}

// Lets a kernel have its dynamic shared memory, once per device.
template <auto KERNEL>
cudaError_t allow_shared(int bytes) {
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

}  // namespace
}  // namespace tpmlp
