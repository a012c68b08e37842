// layernorm_plain.cu -- LayerNorm without a residual (the final norm in front
// of the output head), forward and backward, in bf16, fp16 and fp32.
//
// Per row of h values:
//   mu = mean(x) ; var = mean((x - mu)^2) ; rstd = 1/sqrt(var + eps)
//   y = (x - mu) rstd gamma + beta
// and its backward pass:
//   xhat = (x - mu) rstd ; g = dy gamma
//   dx = rstd (g - mean(g) - xhat mean(g xhat))
//   dgamma = sum_rows dy xhat ; dbeta = sum_rows dy
// All sums and statistics are fp32.  A few operations per value: bound by HBM.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <type_traits>

#include "../../include/tpmlp.h"
#include "kernels.h"

namespace tpmlp {
namespace {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

constexpr int kNormMaxStages = 6;
constexpr int kNormMaxCluster = 8;
constexpr int kNormMaxPerSm = 4;  // CTAs of the backward kernel
// Rows that a thread of the backward kernel takes together, and the blocks
// that it begins before the one that it finishes.  The ring needs twice as
// many stages as the latter.
template <int VEC>
constexpr int norm_rows() { return VEC == 8 ? 2 : 1; }
template <int VEC>
constexpr int norm_ahead(int elem) { return VEC == 1 && elem == 2 ? 2 : 1; }

// A piece of a row held by one thread: VEC > 1 consecutive values, 16 bytes,
// or (VEC 1, rows that do not start on 16-byte boundaries) two single values
// a row's thread count apart.  The arithmetic runs on pairs of fp32 values
// (one packed instruction for two), and these kernels are close to the
// issue rate: 37 instructions a value of the backward pass when written one
// by one, 14 with pairs.
template <typename T, int VEC>
struct Piece {
    static constexpr int N = VEC == 1 ? 2 : VEC;
    static constexpr int WORDS = N * static_cast<int>(sizeof(T)) / 4;
    uint32_t w[WORDS];
};

// Column of value j of piece k for thread `sub` of `group`.
template <int VEC>
__device__ __forceinline__ int piece_col(int k, int j, int group, int sub) {
    return VEC == 1 ? (2 * k + j) * group + sub : (k * group + sub) * VEC + j;
}

// Piece k of the row at p (columns at and beyond h read 0).
template <typename T, int VEC>
__device__ __forceinline__ Piece<T, VEC> load_piece(const T* p, int k, int group, int sub, int h) {
    Piece<T, VEC> r;
    const int c = piece_col<VEC>(k, 0, group, sub);
    if constexpr (VEC > 1) {
        static_assert(sizeof(r) == 16, "a 16-byte piece");
        uint4 u = make_uint4(0u, 0u, 0u, 0u);
        if (c < h) u = *reinterpret_cast<const uint4*>(p + c);
        r.w[0] = u.x; r.w[1] = u.y; r.w[2] = u.z; r.w[3] = u.w;
    } else if constexpr (sizeof(T) == 4) {
        r.w[0] = c < h ? reinterpret_cast<const uint32_t*>(p)[c] : 0u;
        r.w[1] = c + group < h ? reinterpret_cast<const uint32_t*>(p)[c + group] : 0u;
    } else {
        const uint32_t lo = c < h ? reinterpret_cast<const uint16_t*>(p)[c] : 0u;
        const uint32_t hi = c + group < h ? reinterpret_cast<const uint16_t*>(p)[c + group] : 0u;
        r.w[0] = lo | (hi << 16);
    }
    return r;
}

// The same without a branch: columns behind the row read some value of it.
template <typename T, int VEC>
__device__ __forceinline__ Piece<T, VEC> load_piece_any(const T* p, int k, int group, int sub, int h) {
    Piece<T, VEC> r;
    const int c = piece_col<VEC>(k, 0, group, sub);
    if constexpr (VEC > 1) {
        const uint4 u = *reinterpret_cast<const uint4*>(p + min(c, h - VEC));
        r.w[0] = u.x; r.w[1] = u.y; r.w[2] = u.z; r.w[3] = u.w;
    } else if constexpr (sizeof(T) == 4) {
        r.w[0] = reinterpret_cast<const uint32_t*>(p)[min(c, h - 1)];
        r.w[1] = reinterpret_cast<const uint32_t*>(p)[min(c + group, h - 1)];
    } else {
        const uint32_t lo = reinterpret_cast<const uint16_t*>(p)[min(c, h - 1)];
        const uint32_t hi = reinterpret_cast<const uint16_t*>(p)[min(c + group, h - 1)];
        r.w[0] = lo | (hi << 16);
    }
    return r;
}

template <typename T, int VEC>
__device__ __forceinline__ void store_piece(T* p, const Piece<T, VEC>& r, int k, int group, int sub, int h) {
    const int c = piece_col<VEC>(k, 0, group, sub);
    if constexpr (VEC > 1) {
        if (c < h) *reinterpret_cast<uint4*>(p + c) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    } else if constexpr (sizeof(T) == 4) {
        if (c < h) reinterpret_cast<uint32_t*>(p)[c] = r.w[0];
        if (c + group < h) reinterpret_cast<uint32_t*>(p)[c + group] = r.w[1];
    } else {
        if (c < h) reinterpret_cast<uint16_t*>(p)[c] = static_cast<uint16_t>(r.w[0]);
        if (c + group < h) reinterpret_cast<uint16_t*>(p)[c + group] = static_cast<uint16_t>(r.w[0] >> 16);
    }
}

// Pair i of a piece as fp32, and back (rounded once).
template <typename T, int VEC>
__device__ __forceinline__ float2 pair_of(const Piece<T, VEC>& r, int i) {
    if constexpr (sizeof(T) == 4) {
        return make_float2(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
    } else if constexpr (std::is_same_v<T, __half>) {
        return __half22float2(*reinterpret_cast<const __half2*>(&r.w[i]));
    } else {
        return make_float2(__uint_as_float(r.w[i] << 16), __uint_as_float(r.w[i] & 0xFFFF0000u));
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void set_pair(Piece<T, VEC>& r, int i, float2 v) {
    if constexpr (sizeof(T) == 4) {
        r.w[2 * i] = __float_as_uint(v.x);
        r.w[2 * i + 1] = __float_as_uint(v.y);
    } else if constexpr (std::is_same_v<T, __half>) {
        const __half2 p = __floats2half2_rn(v.x, v.y);
        r.w[i] = *reinterpret_cast<const uint32_t*>(&p);
    } else {
        r.w[i] = pack_bf16x2(v.x, v.y);
    }
}

// Packed fp32 arithmetic: each half rounded as the scalar operation.
__device__ __forceinline__ unsigned long long bits(float2 v) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
    return r;
}
__device__ __forceinline__ float2 halves(unsigned long long b) {
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(b));
    return v;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
    return halves(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
    return halves(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
    return halves(r);
}
// g = dy gamma.  The packed product may be fused with the subtraction of
// mean(g) behind it; a row of one value (VEC 1) needs it rounded as it was
// summed, so that g - mean(g) is 0.
template <int VEC>
__device__ __forceinline__ float2 product(float2 a, float2 b) {
    if constexpr (VEC == 1) return make_float2(__fmul_rn(a.x, b.x), __fmul_rn(a.y, b.y));
    return mul2(a, b);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// The pairs of piece k as fp32 values of a row at p.
template <int VEC>
__device__ __forceinline__ void store_pairs(float* p, const float2* v, int k, int group, int sub, int h) {
    const int c = piece_col<VEC>(k, 0, group, sub);
    if constexpr (VEC == 1) {
        if (c < h) p[c] = v[0].x;
        if (c + group < h) p[c + group] = v[0].y;
    } else if (c < h) {
#pragma unroll
        for (int j = 0; j < VEC / 2; j += 2)
            *reinterpret_cast<float4*>(p + c + 2 * j) = make_float4(v[j].x, v[j].y, v[j + 1].x, v[j + 1].y);
    }
}

__device__ __forceinline__ float2 warp_sum(float2 x) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        x.x += __shfl_xor_sync(0xFFFFFFFFu, x.x, off);
        x.y += __shfl_xor_sync(0xFFFFFFFFu, x.y, off);
    }
    return x;
}

// Sums over the warp of the U pairs' 2 U values: 32 / (2 U) lanes after one
// another receive each.  A lane gives away half of its values at each of the
// first steps: 6 exchanges for four values instead of 20.
template <int U>
__device__ __forceinline__ float warp_sums(const float2 (&v)[U]) {
    static_assert(U == 1 || U == 2, "");
    const int lane = threadIdx.x & 31;
    float2 k = v[0];
    if constexpr (U == 2) {
        const bool second = lane & 16;
        const float2 away = second ? v[0] : v[1];
        if (second) k = v[1];
        k.x += __shfl_xor_sync(0xFFFFFFFFu, away.x, 16);
        k.y += __shfl_xor_sync(0xFFFFFFFFu, away.y, 16);
    }
    constexpr int HALF = 16 / U;
    const bool other = lane & HALF;
    float x = other ? k.y : k.x;
    x += __shfl_xor_sync(0xFFFFFFFFu, other ? k.x : k.y, HALF);
#pragma unroll
    for (int off = HALF / 2; off >= 1; off >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
    return x;
}

// Sum over the W warps of a row's group (`first` and the W - 1 behind it);
// every thread receives the total, added in the same order in every thread.
// `scratch` holds one entry a warp.  All threads of the CTA call it.
__device__ __forceinline__ float2 group_sum(float2 x, int W, int first, float2* scratch) {
    x = warp_sum(x);
    if (W == 1) return x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) scratch[warp] = x;
    __syncthreads();
    const int lanes = 1 << (32 - __clz(W - 1)), i = lane & (lanes - 1);  // W up to a power of two
    x = i < W ? scratch[first + i] : both(0.0f);
    for (int off = lanes >> 1; off >= 1; off >>= 1) {
        x.x += __shfl_xor_sync(0xFFFFFFFFu, x.x, off);
        x.y += __shfl_xor_sync(0xFFFFFFFFu, x.y, off);
    }
    return x;
}

// Forward: W warps a row, the row in registers (NV pieces a thread), so all
// of its loads are in flight at once and x is read once.  The variance is
// taken from x - mu.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(1024)
    norm_forward_reg_kernel(const T* __restrict__ x, const T* __restrict__ gamma,
                            const T* __restrict__ beta, int rows, int h, int W, float eps,
                            T* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd) {
    pdl_launch_dependents();  // the next kernel may begin its launch
    pdl_wait();               // its inputs may come from the kernel before it
    __shared__ float2 scratch[2][32];
    const int group = 32 * W;  // threads a row
    const int g = threadIdx.x / group, sub = threadIdx.x - g * group, first = g * W;
    const int row = blockIdx.x * (blockDim.x / group) + g;
    const bool ok = row < rows;
    const long long base = static_cast<long long>(row) * h;
    constexpr int PAIRS = Piece<T, VEC>::N / 2;
    Piece<T, VEC> in[NV];
    float2 acc = both(0.0f);
#pragma unroll
    for (int k = 0; k < NV; ++k) in[k] = load_piece<T, VEC>(x + base, k, group, sub, ok ? h : 0);
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) acc = add2(acc, pair_of(in[k], i));
    const float mu = group_sum(make_float2(acc.x + acc.y, 0.0f), W, first, scratch[0]).x / static_cast<float>(h);
    acc = both(0.0f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        // the zeros behind the row are not its values
        if (piece_col<VEC>(k, 0, group, sub) >= h) continue;
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            float2 c = add2(pair_of(in[k], i), both(-mu));
            if (VEC == 1 && piece_col<VEC>(k, 1, group, sub) >= h) c.y = 0.0f;
            acc = fma2(c, c, acc);
        }
    }
    const float var = group_sum(make_float2(acc.x + acc.y, 0.0f), W, first, scratch[1]).x / static_cast<float>(h);
    const float rs = 1.0f / sqrtf(var + eps);
    if (!ok) return;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const Piece<T, VEC> g = load_piece<T, VEC>(gamma, k, group, sub, h);
        const Piece<T, VEC> b = load_piece<T, VEC>(beta, k, group, sub, h);
        Piece<T, VEC> o;
#pragma unroll
        for (int i = 0; i < PAIRS; ++i)
            set_pair(o, i, fma2(mul2(add2(pair_of(in[k], i), both(-mu)), both(rs)), pair_of(g, i), pair_of(b, i)));
        store_piece<T, VEC>(y + base, o, k, group, sub, h);
    }
    if (sub == 0) {
        mean[row] = mu;
        rstd[row] = rs;
    }
}

// Backward in one pass over x and dy.  Blocks of R rows (R = NT / 32 / W, W
// warps a row) stream through a ring of `stages` buffers in shared memory,
// one bulk copy a tensor and block (the rows of a block are one contiguous
// range), so that the loads in flight do not depend on the registers; block
// b goes to CTA (or cluster) b mod their number.  Every thread keeps the
// same columns in every row and adds its part of dgamma and dbeta in
// registers; at the end the CTA's groups meet in shared memory, in group
// order, and the sums go to part[0 / 1][CTA or cluster][column].
// Rows wider than a CTA's registers are cut over the `cl` CTAs of a cluster
// (one row at a time, `cols` columns each).
// Measured in bf16: 8192 x 1024 in 18.9 us with the sum of the parts (2.7 TB/s;
// start, end and the sum's launch are half of it), 40960 x 1024 in 47 us (5.4
// TB/s), 8192 x 8192 in 70 us (5.8 TB/s), 2048 x 20480 in 55 us (4.6 TB/s);
// the longest are bound by HBM reading and writing at once.
// There is no barrier in the loop.  A warp begins block i + AHEAD (its part of
// the row sums, which go to the shared memory of every CTA of the row and are
// counted on an mbarrier there) before it finishes block i
// (dx, from the sums of all warps, which have long arrived): with a barrier a
// block, a cluster's exchange of about a microsecond stands in every row.
struct NormBackwardArgs {
    int rows, h, W, stages;
    int cl, cols;   // CTAs a row, columns of one
    int buf_bytes;  // one tensor's block in the ring, 16-byte multiple
    int* status;
};

template <typename T, int VEC, int NV, int NT, int MIN_CTAS, bool CLUSTER>
__global__ void __launch_bounds__(NT, MIN_CTAS)
    norm_backward_ring_kernel(const T* __restrict__ dy, const T* __restrict__ x,
                              const T* __restrict__ gamma, const float* __restrict__ mean,
                              const float* __restrict__ rstd, const NormBackwardArgs p,
                              T* __restrict__ dx, float* __restrict__ part_g,
                              float* __restrict__ part_b) {
    // rows of a block that one thread takes together: two share the loop's
    // overhead and gamma (one where the ring has no room for two, or rows are
    // misaligned)
    constexpr int U = norm_rows<VEC>();
    constexpr int AHEAD = norm_ahead<VEC>(sizeof(T)), SLOTS = 2 * AHEAD;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t full[kNormMaxStages];
    __shared__ uint64_t sums[SLOTS];  // a block's sums of all warps have arrived
    __shared__ float2 slots[SLOTS][(CLUSTER ? kNormMaxCluster : 1) * (NT / 32)][U];
    __shared__ uint32_t abort_flag;
    pdl_launch_dependents();  // the next kernel may begin its launch
    constexpr long long E = sizeof(T);
    const int warps = blockDim.x >> 5;  // NT / 32 at most
    const int group = 32 * p.W, R = warps / p.W;
    const int g = CLUSTER ? 0 : threadIdx.x / group, sub = threadIdx.x - g * group;
    const int cl = CLUSTER ? p.cl : 1;
    const int rank = CLUSTER ? static_cast<int>(cluster_ctarank()) : 0;
    const uint32_t unit = CLUSTER ? blockIdx.x / cl : blockIdx.x;
    const uint32_t step = CLUSTER ? gridDim.x / cl : gridDim.x;
    const int c0 = rank * p.cols;              // this CTA's columns of a row
    const int h = CLUSTER ? min(p.cols, p.h - c0) : p.h;
    const uint32_t rows = p.rows, block_rows = R * U;
    const uint32_t blocks = (rows + block_rows - 1) / block_rows;
    const long long total = E * p.rows * p.h;  // bytes of a tensor
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) mbar_init(&full[s], 1);
        // a cluster counts the bytes that its warps send, one CTA its warps
        for (int s = 0; s < SLOTS; ++s) mbar_init(&sums[s], CLUSTER ? 1 : warps);
        abort_flag = 0u;
        fence_mbar_init();
    }
    pdl_wait();  // dy may come from the kernel before this one
    if constexpr (CLUSTER)
        cluster_sync();  // the peers run: their shared memory may be written
    else
        __syncthreads();

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // which of a block's 2 U sums a lane holds, and which of its holders it is
    constexpr int HOLDERS = 16 / U;
    static_assert(HOLDERS >= kNormMaxCluster, "a holder for each CTA");
    const int value = lane / HOLDERS, part = lane % HOLDERS;
    // where it sends it: its place of slot 0, and that slot's barrier
    uint32_t peer_slot = 0, peer_bar = 0;
    if constexpr (CLUSTER) {
        if (part < cl) {
            peer_slot = map_to_cta(smem_u32(slots[0][rank * warps + warp]) + 4 * value, part);
            peer_bar = map_to_cta(smem_u32(&sums[0]), part);
        }
    }

    // This CTA's blocks are unit, unit + step, ..., n of them.  Everything a
    // block needs advances by additions: with divisions and 64-bit addresses
    // in the loop the overhead was 490 instructions a warp and block against
    // 200 of arithmetic.
    const int n = blocks > unit ? static_cast<int>((blocks - unit + step - 1) / step) : 0;
    const uint32_t row_step = step * block_rows;
    const uint32_t stage_bytes = 2u * p.buf_bytes;
    const int row_bytes = static_cast<int>(E) * h;

    // Warp 0: copies of the next block not yet issued into the next stage, one a
    // lane.
    // One CTA a row: the block's rows are one contiguous range, of which whole
    // 16-byte granules of the tensor are copied (all but its last few bytes).
    // A cluster: each row's columns are copied by themselves.
    const long long first_b0 = E * (static_cast<long long>(unit) * block_rows * p.h + c0);
    const long long issue_step = E * row_step * p.h;
    long long issue_b0 = first_b0;
    int issue_left = n, issue_stage = 0;
    uint32_t issue_row = unit * block_rows;
    auto copied = [&](long long b0, int bytes, long long& a0) {  // first byte, and their number
        a0 = b0 & ~15LL;
        const long long a1 = min((min(b0 + bytes, total) + 15) & ~15LL, total & ~15LL);
        return a1 > a0 ? static_cast<uint32_t>(a1 - a0) : 0u;
    };
    auto issue = [&]() {
        if (issue_left <= 0) return;
        const uint32_t dst = smem_u32(ring) + issue_stage * stage_bytes;
        uint64_t* bar = &full[issue_stage];
        const uint8_t *px = reinterpret_cast<const uint8_t*>(x), *pd = reinterpret_cast<const uint8_t*>(dy);
        if (CLUSTER && U > 1) {
            const int k = min(static_cast<uint32_t>(U), rows - issue_row), u = lane & (U - 1), t = lane / U;
            if (lane == 0) mbar_arrive_expect_tx(bar, 2 * k * row_bytes);
            if (t < 2 && u < k)
                bulk_load(dst + u * row_bytes + t * p.buf_bytes, (t ? pd : px) + issue_b0 + u * E * p.h, row_bytes, bar);
        } else {
            long long a0;
            const uint32_t bytes = copied(issue_b0, CLUSTER ? row_bytes : static_cast<int>(block_rows) * row_bytes, a0);
            if (lane == 0) mbar_arrive_expect_tx(bar, 2 * bytes);
            if (lane < 2 && bytes) bulk_load(dst + lane * p.buf_bytes, (lane ? pd : px) + a0, bytes, bar);
        }
        issue_b0 += issue_step;
        issue_row += row_step;
        --issue_left;
        if (++issue_stage == p.stages) issue_stage = 0;
    };
    if (warp == 0)
        for (int s = 0; s < p.stages; ++s) issue();

    constexpr int PAIRS = Piece<T, VEC>::N / 2;
    float2 acc_g[NV * PAIRS], acc_b[NV * PAIRS];
    Piece<T, VEC> kg[NV];  // gamma, 0 behind the row: what is read there counts nothing
#pragma unroll
    for (int i = 0; i < NV * PAIRS; ++i) acc_g[i] = acc_b[i] = both(0.0f);
#pragma unroll
    for (int k = 0; k < NV; ++k) kg[k] = load_piece<T, VEC>(gamma + c0, k, group, sub, h);
    const float inv_h = 1.0f / static_cast<float>(p.h);
    struct Stats {
        float2 v[U];
    };
    // the statistics of this thread's rows (0 behind the last)
    auto row_stats = [&](uint32_t row) {
        Stats s;
#pragma unroll
        for (int u = 0; u < U; ++u)
            s.v[u] = row + u < rows ? make_float2(__ldg(mean + row + u), __ldg(rstd + row + u)) : both(0.0f);
        return s;
    };
    // This thread's first row of a block in a stage's buffers; `skip`: where the
    // block starts in its first 16-byte granule (rows of VEC 1 only).
    const uint32_t group_off = static_cast<uint32_t>(row_bytes) * (g * U);
    const uint32_t skip0 = VEC == 1 ? static_cast<uint32_t>(first_b0 & 15) : 0u;
    const uint32_t skip_step = VEC == 1 ? static_cast<uint32_t>(issue_step & 15) : 0u;
    auto row_at = [&](int stage, uint32_t skip) {
        return reinterpret_cast<const T*>(ring + (stage * stage_bytes + skip + group_off));
    };
    auto dy_of = [&](const T* sx) {
        return reinterpret_cast<const T*>(reinterpret_cast<const uint8_t*>(sx) + p.buf_bytes);
    };
    // A wait that gives up: the copies issued so far (the last of each stage; the
    // earlier ones were waited for) land, and so does what peers have sent,
    // before the CTA is gone.
    auto give_up = [&] {
        if (threadIdx.x == 0) {
            const int issued = n - issue_left;
            for (int s = 0; s < p.stages && s < issued; ++s)
                wait_drain(&full[s], static_cast<uint32_t>((issued - 1 - s) / p.stages) & 1u, p.status);
        }
        if constexpr (CLUSTER) {
            for (int i = 0; i < 100; ++i) __nanosleep(10000);
            cluster_sync_thread();
        }
        exit_thread();
    };
    // Begins the CTA's i-th block: waits for its copies and sends this warp's
    // part of its rows' sums of g and g (x - mu) to every CTA of the row.
    int b_stage = 0, b_slot = 0;
    uint32_t b_phase = 0, b_skip = skip0, b_row = unit * block_rows + g * U;
    auto begin = [&](int i, const Stats& st) {
        warp_wait_polls(&full[b_stage], b_phase, &abort_flag, p.status, give_up);
        if constexpr (VEC == 1) {
            if (i == n - 1) {  // the tensor's last few bytes, if they are here: plain loads
                const long long b0 = first_b0 + i * issue_step;
                const int block_bytes = CLUSTER ? row_bytes : static_cast<int>(block_rows) * row_bytes;
                long long a0;
                const uint32_t bytes = copied(b0, block_bytes, a0);
                const long long e = max(a0 + bytes, b0) / E + threadIdx.x;
                if (e < min(b0 + block_bytes, total) / E) {
                    uint8_t* d = ring + b_stage * stage_bytes + (e * E - a0);
                    *reinterpret_cast<T*>(d) = x[e];
                    *reinterpret_cast<T*>(d + p.buf_bytes) = dy[e];
                }
                __syncthreads();
            }
        }
        float2 m[U], mx[U];
#pragma unroll
        for (int u = 0; u < U; ++u) m[u] = mx[u] = both(0.0f);
        if (b_row < rows) {  // (a second row behind the last reads stale values: its sums go nowhere)
            const T* sx = row_at(b_stage, b_skip);
            const T* sdy = dy_of(sx);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const Piece<T, VEC> px = load_piece_any<T, VEC>(sx + u * h, k, group, sub, h);
                    const Piece<T, VEC> pd = load_piece_any<T, VEC>(sdy + u * h, k, group, sub, h);
#pragma unroll
                    for (int j = 0; j < PAIRS; ++j) {
                        const float2 gj = product<VEC>(pair_of(pd, j), pair_of(kg[k], j));
                        m[u] = add2(m[u], gj);
                        mx[u] = fma2(gj, add2(pair_of(px, j), both(-st.v[u].x)), mx[u]);
                    }
                }
            }
        }
        uint64_t* bar = &sums[b_slot];
        float2* slot = slots[b_slot][rank * warps + warp];
#pragma unroll
        for (int u = 0; u < U; ++u) m[u] = make_float2(m[u].x + m[u].y, mx[u].x + mx[u].y);
        const float v = warp_sums<U>(m);
        if constexpr (!CLUSTER) {
            if (part == 0) reinterpret_cast<float*>(slot)[value] = v;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);  // releases the slot to the waiting warps
        } else {
            if (threadIdx.x == 0) mbar_arrive_expect_tx(bar, cl * warps * U * sizeof(float2));
            if (part < cl)
                st_async_f32(peer_slot + b_slot * sizeof(slots[0]), v, peer_bar + b_slot * sizeof(sums[0]));
        }
        __syncwarp();
        if (++b_stage == p.stages) {
            b_stage = 0;
            b_phase ^= 1u;
        }
        b_slot = b_slot + 1 == SLOTS ? 0 : b_slot + 1;
        b_skip = (b_skip + skip_step) & 15;
        b_row += row_step;
    };

    // Slots and stages.  A warp sends block i + AHEAD behind its finish of
    // block i, for which it had the sums of block i: every warp of the row had
    // begun block i, so had finished block i - AHEAD and read its slots.  So 2
    // AHEAD slots are enough; and the buffers of block i - AHEAD are free.
    uint32_t row = b_row;
    Stats st[AHEAD], st_next;
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
        st[a] = row_stats(row + a * row_step);
        if (a < n) begin(a, st[a]);
    }
    st_next = row_stats(row + AHEAD * row_step);
    int stage = 0, slot = 0;
    uint32_t phase = 0, skip = skip0;
    T* out = dx + static_cast<long long>(row) * p.h + c0;
    const long long out_step = static_cast<long long>(row_step) * p.h;
    for (int i = 0; i < n; ++i) {
        const Stats st_after = row_stats(row + (AHEAD + 1) * row_step);
        warp_wait_polls(&sums[slot], phase, &abort_flag, p.status, give_up);
        if (warp == 0 && i >= AHEAD) issue();  // block i - AHEAD is read
        float2 m[U];
        if constexpr (CLUSTER) {
            const float* f = reinterpret_cast<const float*>(slots[slot]);
            float v = 0.0f;
            for (int j = part; j < cl * warps; j += HOLDERS) v += f[2 * U * j + value];
#pragma unroll
            for (int off = HOLDERS / 2; off >= 1; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
#pragma unroll
            for (int u = 0; u < U; ++u)
                m[u] = make_float2(__shfl_sync(0xFFFFFFFFu, v, 2 * u * HOLDERS),
                                   __shfl_sync(0xFFFFFFFFu, v, (2 * u + 1) * HOLDERS));
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                m[u] = both(0.0f);
#pragma unroll 4
                for (int j = 0; j < p.W; ++j) m[u] = add2(m[u], slots[slot][g * p.W + j][u]);
            }
        }
        if (row < rows) {
            const bool second = U == 1 || row + 1 < rows;
            float mg[U], mgx[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                mg[u] = m[u].x * inv_h;                  // mean(g)
                mgx[u] = m[u].y * inv_h * st[0].v[u].y;  // mean(g xhat)
            }
            const T* sx = row_at(stage, skip);
            const T* sdy = dy_of(sx);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (u > 0 && !second) break;
                    const float mu = st[0].v[u].x, rs = st[0].v[u].y;
                    const Piece<T, VEC> px = load_piece_any<T, VEC>(sx + u * h, k, group, sub, h);
                    const Piece<T, VEC> pd = load_piece_any<T, VEC>(sdy + u * h, k, group, sub, h);
                    Piece<T, VEC> o;
#pragma unroll
                    for (int j = 0; j < PAIRS; ++j) {
                        const float2 d = pair_of(pd, j);
                        // one rstd a factor: its powers leave the range of fp32 (rows of
                        // 1e13, or eps below 1e-25) where the products do not
                        const float2 xhat = mul2(add2(pair_of(px, j), both(-mu)), both(rs));
                        const float2 gj = product<VEC>(d, pair_of(kg[k], j));
                        set_pair(o, j, mul2(both(rs), fma2(xhat, both(-mgx[u]), add2(gj, both(-mg[u])))));
                        acc_g[k * PAIRS + j] = fma2(d, xhat, acc_g[k * PAIRS + j]);
                        acc_b[k * PAIRS + j] = add2(acc_b[k * PAIRS + j], d);
                    }
                    store_piece<T, VEC>(out + u * p.h, o, k, group, sub, h);
                }
            }
        }
        if (i + AHEAD < n) begin(i + AHEAD, st_next);
#pragma unroll
        for (int a = 0; a + 1 < AHEAD; ++a) st[a] = st[a + 1];
        st[AHEAD - 1] = st_next;
        st_next = st_after;
        if (++stage == p.stages) stage = 0;
        if (++slot == SLOTS) {
            slot = 0;
            phase ^= 1u;
        }
        skip = (skip + skip_step) & 15;
        row += row_step;
        out += out_step;
    }

    // No CTA leaves while a value that it has sent is on its way to a peer:
    // it has itself waited for the last block's sums, to which the peers'
    // own values of every block belong, but not for their receipt.
    if constexpr (CLUSTER) cluster_sync();
    float* out_g = part_g + static_cast<long long>(unit) * p.h + c0;
    float* out_b = part_b + static_cast<long long>(unit) * p.h + c0;
    if (R == 1) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            store_pairs<VEC>(out_g, &acc_g[k * PAIRS], k, group, sub, h);
            store_pairs<VEC>(out_b, &acc_b[k * PAIRS], k, group, sub, h);
        }
        return;
    }
    // The ring's buffers are free: every copy has been waited for and read.
    // Pair i of a thread sits at i group + sub, so that a warp's accesses are
    // consecutive.
    float2* sg = reinterpret_cast<float2*>(ring);
    float2* sb = sg + NV * PAIRS * group;
    for (int r = 0; r < R; ++r) {
        __syncthreads();
        if (g == r) {
#pragma unroll
            for (int i = 0; i < NV * PAIRS; ++i) {
                const int o = i * group + sub;
                sg[o] = r ? add2(sg[o], acc_g[i]) : acc_g[i];
                sb[o] = r ? add2(sb[o], acc_b[i]) : acc_b[i];
            }
        }
    }
    __syncthreads();
    if (g == 0) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
#pragma unroll
            for (int i = 0; i < PAIRS; ++i) {
                acc_g[k * PAIRS + i] = sg[(k * PAIRS + i) * group + sub];
                acc_b[k * PAIRS + i] = sb[(k * PAIRS + i) * group + sub];
            }
            store_pairs<VEC>(out_g, &acc_g[k * PAIRS], k, group, sub, h);
            store_pairs<VEC>(out_b, &acc_b[k * PAIRS], k, group, sub, h);
        }
    }
}

// dgamma[c] = sum_i part_g[i][c], dbeta likewise: CHAINS interleaved chains (a
// warp each) over i, then the chains in order.
template <int CHAINS>
__global__ void __launch_bounds__(32 * CHAINS)
    norm_param_reduce_kernel(const float* __restrict__ part_g, const float* __restrict__ part_b,
                             int n, int h, float* __restrict__ dgamma, float* __restrict__ dbeta) {
    pdl_launch_dependents();  // the next kernel may begin its launch
    pdl_wait();               // the parts come from the kernel before this one
    __shared__ float chain[CHAINS][32];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane;
    const float* part = blockIdx.y ? part_b : part_g;
    float s = 0.0f;
    if (c < h) {
#pragma unroll 10
        for (int i = w; i < n; i += CHAINS) s += __ldg(part + static_cast<long long>(i) * h + c);
    }
    chain[w][lane] = s;
    __syncthreads();
    if (w == 0 && c < h) {
        s = 0.0f;
#pragma unroll
        for (int j = 0; j < CHAINS; ++j) s += chain[j][lane];
        (blockIdx.y ? dbeta : dgamma)[c] = s;
    }
}

cudaError_t param_reduce(const float* pg, const float* pb, int n, int h, float* dgamma, float* dbeta,
                         cudaStream_t st, int* launches) {
    ++*launches;
    const dim3 grid((h + 31) / 32, 2);
    // few columns: many warps a column block, so that each adds few rows; many:
    // the column blocks fill the GPU by themselves
    if (h <= 4096)
        return launch_dependent(norm_param_reduce_kernel<32>, grid, dim3(1024), 0, st, pg, pb, n, h, dgamma, dbeta);
    return launch_dependent(norm_param_reduce_kernel<8>, grid, dim3(256), 0, st, pg, pb, n, h, dgamma, dbeta);
}

// ---------------------------------------------------------- any row width
// Rows beyond what the kernels above hold: one CTA a row, the row read from
// memory (L2) again for each step.

constexpr int kRowThreads = 256;

// Sum over the CTA; every thread receives the total.
__device__ __forceinline__ float cta_sum(float x, float* scratch) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
    __syncthreads();  // scratch may still be read by a previous call
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = x;
    __syncthreads();
    float t = (threadIdx.x & 31) < kRowThreads / 32 ? scratch[threadIdx.x & 31] : 0.0f;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, off);
    return t;
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads)
    norm_forward_kernel(const T* __restrict__ x, const T* __restrict__ gamma,
                        const T* __restrict__ beta, int h, float eps, T* __restrict__ y,
                        float* __restrict__ mean, float* __restrict__ rstd) {
    pdl_launch_dependents();  // the next kernel may begin its launch
    pdl_wait();               // its inputs may come from the kernel before it
    __shared__ float scratch[32];
    const long long base = static_cast<long long>(blockIdx.x) * h;
    float sum = 0.0f;
    for (int i = threadIdx.x; i < h; i += kRowThreads) sum += to_f32(x[base + i]);
    const float mu = cta_sum(sum, scratch) / static_cast<float>(h);
    float sq = 0.0f;
    for (int i = threadIdx.x; i < h; i += kRowThreads) {
        const float c = to_f32(x[base + i]) - mu;
        sq = fmaf(c, c, sq);
    }
    const float rs = 1.0f / sqrtf(cta_sum(sq, scratch) / static_cast<float>(h) + eps);
    for (int i = threadIdx.x; i < h; i += kRowThreads)
        y[base + i] = from_f32<T>((to_f32(x[base + i]) - mu) * rs * to_f32(gamma[i]) + to_f32(beta[i]));
    if (threadIdx.x == 0) {
        mean[blockIdx.x] = mu;
        rstd[blockIdx.x] = rs;
    }
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads)
    norm_backward_kernel(const T* __restrict__ dy, const T* __restrict__ x,
                         const T* __restrict__ gamma, const float* __restrict__ mean,
                         const float* __restrict__ rstd, int h, T* __restrict__ dx) {
    pdl_launch_dependents();  // the next kernel may begin its launch
    pdl_wait();               // its inputs may come from the kernel before it
    __shared__ float scratch[32];
    const long long base = static_cast<long long>(blockIdx.x) * h;
    const float mu = mean[blockIdx.x], rs = rstd[blockIdx.x];
    float mg = 0.0f, mgx = 0.0f;
    for (int i = threadIdx.x; i < h; i += kRowThreads) {
        const float g = to_f32(dy[base + i]) * to_f32(gamma[i]);
        mg += g;
        mgx = fmaf(g, (to_f32(x[base + i]) - mu) * rs, mgx);
    }
    mg = cta_sum(mg, scratch) / static_cast<float>(h);
    mgx = cta_sum(mgx, scratch) / static_cast<float>(h);
    for (int i = threadIdx.x; i < h; i += kRowThreads) {
        // the product is rounded as it was summed: a row of one value gives 0
        const float g = __fmul_rn(to_f32(dy[base + i]), to_f32(gamma[i]));
        const float xhat = (to_f32(x[base + i]) - mu) * rs;
        dx[base + i] = from_f32<T>(rs * (g - mg - xhat * mgx));
    }
}

// Column sums of dy xhat and dy over one chunk of rows: a CTA of 32 x 8
// threads takes 32 columns, thread row k the rows k, k + 8, ... of its chunk;
// the eight sums are added in order.  Writes part[0 / 1][chunk][column].
template <typename T>
__global__ void __launch_bounds__(256)
    norm_param_grad_kernel(const T* __restrict__ dy, const T* __restrict__ x,
                           const float* __restrict__ mean, const float* __restrict__ rstd, int T_,
                           int h, int rows_per_chunk, float* __restrict__ part) {
    pdl_launch_dependents();  // the next kernel may begin its launch
    pdl_wait();               // its inputs may come from the kernel before it
    __shared__ float sg[8][32], sb[8][32];
    const int c = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + c;
    const int r0 = blockIdx.y * rows_per_chunk, r1 = min(T_, r0 + rows_per_chunk);
    float g = 0.0f, b = 0.0f;
    if (col < h) {
        for (int r = r0 + k; r < r1; r += 8) {
            const long long i = static_cast<long long>(r) * h + col;
            const float d = to_f32(dy[i]);
            g = fmaf(d, (to_f32(x[i]) - mean[r]) * rstd[r], g);
            b += d;
        }
    }
    sg[k][c] = g;
    sb[k][c] = b;
    __syncthreads();
    if (k == 0 && col < h) {
        for (int j = 1; j < 8; ++j) {
            g += sg[j][c];
            b += sb[j][c];
        }
        part[static_cast<long long>(blockIdx.y) * h + col] = g;
        part[static_cast<long long>(gridDim.y + blockIdx.y) * h + col] = b;
    }
}

int ceil_div(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

constexpr int kSms = 152;

int ceil_pow2(int x) {
    int p = 1;
    while (p < x) p *= 2;
    return p;
}

template <typename T, int VEC, int NV>
cudaError_t forward_reg(const T* x, const T* gamma, const T* beta, int T_, int h, int W, float eps, T* y,
                        float* mean, float* rstd, cudaStream_t st) {
    const int rows = std::max(1, 8 / W), threads = rows * 32 * W;
    return launch_dependent(norm_forward_reg_kernel<T, VEC, NV>, dim3(ceil_div(T_, rows)), dim3(threads), 0,
                            st, x, gamma, beta, T_, h, W, eps, y, mean, rstd);
}

// W warps a row.  Measured in bf16: 8192 x 1024 in 7.9 us (4.3 TB/s: launch
// and first loads are a quarter of it), 8192 x 8192 in 50 us (5.4 TB/s), 2048 x
// 20480 in 37 us (4.5 TB/s), 1280 x 32768 in 40 us.
template <typename T, int VEC>
cudaError_t forward_rows(const T* x, const T* gamma, const T* beta, int T_, int h, float eps, T* y,
                         float* mean, float* rstd, cudaStream_t st) {
    // 32 values a thread keep the most loads in flight an SM; with few rows
    // more threads a row, down to 8 values each, fill the SMs instead.
    // (Single values want more registers each than pieces: 16 a thread.)
    int per = VEC == 1 && h <= 16 * 1024 ? 16 : 32;
    while (per > 8 && h <= 32 * per / 2) per /= 2;  // one warp holds the row with fewer
    while (per > 8 && static_cast<long long>(T_) * ceil_div(h, 32 * per) < 16LL * kSms &&
           ceil_div(h, 32 * per / 2) <= 32)
        per /= 2;
    // rows beyond 16 warps of that: 40 values a thread, so that two rows (two
    // CTAs of 512 threads) share an SM and one's sums overlap the other's loads
    if (per == 32 && h > 16 * 1024 && h <= 20 * 1024)
        return forward_reg<T, VEC, 40 / Piece<T, VEC>::N>(x, gamma, beta, T_, h, ceil_div(h, 32 * 40), eps, y, mean, rstd, st);
    // the same with 48 and 64 values where a register holds two (1706 x 24576
    // bf16: 36 us, with 32 values 48; 1024 x 40960: 48 us, row read again from
    // memory 78)
    if constexpr (VEC == 8) {
        if (h > 20 * 1024 && h <= 24 * 1024)
            return forward_reg<T, VEC, 6>(x, gamma, beta, T_, h, ceil_div(h, 32 * 48), eps, y, mean, rstd, st);
        if (h > 24 * 1024)
            return forward_reg<T, VEC, 8>(x, gamma, beta, T_, h, ceil_div(h, 32 * 64), eps, y, mean, rstd, st);
    }
    const int W = ceil_div(h, 32 * per);
    if (per == 32) return forward_reg<T, VEC, 32 / Piece<T, VEC>::N>(x, gamma, beta, T_, h, W, eps, y, mean, rstd, st);
    if (per == 16) return forward_reg<T, VEC, 16 / Piece<T, VEC>::N>(x, gamma, beta, T_, h, W, eps, y, mean, rstd, st);
    return forward_reg<T, VEC, 8 / Piece<T, VEC>::N>(x, gamma, beta, T_, h, W, eps, y, mean, rstd, st);
}

template <typename T>
cudaError_t forward(const void* x_, const void* gamma_, const void* beta_, int T_, int h, float eps,
                    void* y_, float* mean, float* rstd, cudaStream_t st, int* launches) {
    const T *x = static_cast<const T*>(x_), *gamma = static_cast<const T*>(gamma_),
            *beta = static_cast<const T*>(beta_);
    T* y = static_cast<T*>(y_);
    ++*launches;
    constexpr int VEC = 16 / sizeof(T);
    if (h <= 32 * 32 * (VEC == 8 && h % VEC == 0 ? 64 : 32)) {
        if (h % VEC == 0) return forward_rows<T, VEC>(x, gamma, beta, T_, h, eps, y, mean, rstd, st);
        return forward_rows<T, 1>(x, gamma, beta, T_, h, eps, y, mean, rstd, st);
    }
    return launch_dependent(norm_forward_kernel<T>, dim3(T_), dim3(kRowThreads), 0, st, x, gamma, beta, h, eps,
                            y, mean, rstd);
}

// How a backward call runs: the ring kernel with W warps and `cl` CTAs a
// row, 16 values a thread, or, units = 0, the kernels for any width.
struct NormPlan {
    int units;  // CTAs, or clusters of `cl` CTAs
    int W, cl, cols, stages, buf_bytes, threads, smem;
    int room;  // the most shared memory that a plan of this many CTAs an SM takes
};

// A CTA's share of an SM's shared memory beside the static arrays.
constexpr int norm_room(int per_sm) { return 227 * 1024 / per_sm - (per_sm == 1 ? 5 : 4) * 1024; }

NormPlan norm_plan(int T, int h, int elem) {
    NormPlan p{};
    // 16 values a thread (128 registers): 16 warps an SM.  Rows beyond 8 warps
    // take a cluster, of an even number of CTAs: SMs come in pairs, and an odd
    // number leaves places empty (2048 x 20480 bf16: 73 us with five).  Of
    // those the number whose CTAs fill the SMs' warps best (63 us with six of
    // seven warps, two an SM; 60, now 55, with eight of five, three an SM), the
    // smaller where the difference is small.
    // Rows beyond eight CTAs of 8 warps take eight of up to 16.
    const int warps = h <= kNormMaxCluster * 16 * 256 ? 8 : 16;
    int most = 0;
    for (int cl = 1; cl <= kNormMaxCluster; cl += cl == 1 ? 1 : 2) {
        const int cols = cl == 1 ? h : ceil_div(ceil_div(h, cl), 8) * 8, W = ceil_div(cols, 32 * 16);
        if (W > warps) continue;
        const int live = std::min(kNormMaxPerSm, 16 / W) * cols;  // columns at work on an SM
        if (live <= most + most / 16) continue;
        most = live;
        p.cl = cl;
        p.cols = cols;
        p.W = W;
        if (cl == 1) break;
    }
    if (p.cl == 0) return NormPlan{};
    if (p.W < 4 && p.cl == 1) p.W = ceil_pow2(p.W);  // groups that fill 8 warps
    const int R = p.cl == 1 ? std::max(1, 8 / p.W) : 1, U = elem == 2 && h % 8 == 0 ? norm_rows<8>() : norm_rows<1>();
    p.threads = 32 * R * p.W;
    // a block of rows and what its first and last granule hold besides
    p.buf_bytes = (static_cast<int>((static_cast<long long>(R) * U * p.cols * elem + 15) / 16) + 1) * 16;
    const int per_sm = std::min(kNormMaxPerSm, 16 / (R * p.W));
    p.room = norm_room(per_sm);
    const int blocks = ceil_div(T, R * U), units = kSms * per_sm / p.cl;
    p.stages = std::min(kNormMaxStages, p.room / (2 * p.buf_bytes));
    // the meeting place of the groups' sums: 16 values a thread and tensor
    p.smem = std::max(p.stages * 2 * p.buf_bytes, R > 1 ? 2 * 16 * 4 * 32 * p.W : 0);
    p.units = std::min(blocks, units);
    return p;
}

// Launches the ring kernel and sets *units to the CTAs or clusters it ran
// with: no more clusters than can be resident at once (the GPU's parts hold a
// number of SMs that clusters need not divide; one cluster too many would
// run alone behind all others).
template <typename T, int VEC, int NV, int NT, int MIN_CTAS>
cudaError_t backward_ring(const NormPlan& p, const T* dy, const T* x, const T* gamma, const float* mean,
                          const float* rstd, int T_, int h, T* dx, float* pg, float* pb, int* status,
                          cudaStream_t st, int* units) {
    auto kern = norm_backward_ring_kernel<T, VEC, NV, NT, MIN_CTAS, false>;
    if constexpr (NV * Piece<T, VEC>::N == 16)
        if (p.cl > 1) kern = norm_backward_ring_kernel<T, VEC, NV, NT, MIN_CTAS, true>;
    // The attribute is the kernel's, not the launch's: the same from every call (the
    // most that any plan of this kernel takes), so that a call of another
    // width in another thread takes nothing from this one.
    static_assert(MIN_CTAS * (NT / 32) == 16, "a plan has at least MIN_CTAS of these CTAs an SM");
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, norm_room(MIN_CTAS));
    if (e != cudaSuccess) return e;
    const NormBackwardArgs a{T_, h, p.W, p.stages, p.cl, p.cols, p.buf_bytes, status};
    if (p.cl == 1) {
        *units = p.units;
        return launch_dependent(kern, dim3(p.units), dim3(p.threads), p.smem, st, dy, x, gamma, mean, rstd, a, dx, pg,
                                pb);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(p.threads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.cl;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    // clusters of this size that fit with the most shared memory a plan takes
    static std::atomic<int> fit[kNormMaxCluster + 1][NT / 32 + 1];  // the same for every device of this build's target
    int n = fit[p.cl][p.W].load(std::memory_order_relaxed);
    if (n == 0) {
        cfg.gridDim = dim3(p.cl);
        cfg.dynamicSmemBytes = p.room;
        cfg.numAttrs = 1;
        if ((e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg)) != cudaSuccess) return e;
        n = std::max(n, 1);
        fit[p.cl][p.W].store(n, std::memory_order_relaxed);
    }
    *units = std::min(p.units, n);
    cfg.gridDim = dim3(*units * p.cl);
    cfg.dynamicSmemBytes = p.smem;
    cfg.numAttrs = dependent_launch() ? 2 : 1;
    if ((e = cudaLaunchKernelEx(&cfg, kern, dy, x, gamma, mean, rstd, a, dx, pg, pb)) != cudaSuccess) return e;
    return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t backward_rows(const NormPlan& p, const T* dy, const T* x, const T* gamma, const float* mean,
                          const float* rstd, int T_, int h, T* dx, float* pg, float* pb, int* status,
                          cudaStream_t st, int* units) {
    constexpr int N = Piece<T, VEC>::N;
    // rows that a warp holds with 8 values a lane (16384 x 256 bf16: 17.6 -> 14.0 us)
    if (h <= 256)
        return backward_ring<T, VEC, 8 / N, 256, 2>(p, dy, x, gamma, mean, rstd, T_, h, dx, pg, pb, status, st, units);
    if (p.threads > 256)
        return backward_ring<T, VEC, 16 / N, 512, 1>(p, dy, x, gamma, mean, rstd, T_, h, dx, pg, pb, status, st, units);
    return backward_ring<T, VEC, 16 / N, 256, 2>(p, dy, x, gamma, mean, rstd, T_, h, dx, pg, pb, status, st, units);
}

template <typename T>
cudaError_t backward(const void* dy_, const void* x_, const void* gamma_, const float* mean,
                     const float* rstd, int T_, int h, void* dx_, float* dgamma, float* dbeta,
                     float* partial, int* status, cudaStream_t st, int* launches) {
    const T *dy = static_cast<const T*>(dy_), *x = static_cast<const T*>(x_),
            *gamma = static_cast<const T*>(gamma_);
    T* dx = static_cast<T*>(dx_);
    cudaError_t e;
    const NormPlan p = norm_plan(T_, h, sizeof(T));
    if (p.units > 0) {
        constexpr int VEC = 16 / sizeof(T);
        // one CTA or cluster: its sums are the result
        float* pg = p.units == 1 ? dgamma : partial;
        float* pb = p.units == 1 ? dbeta : partial + static_cast<size_t>(p.units) * h;
        int units = 0;
        if (h % VEC == 0)
            e = backward_rows<T, VEC>(p, dy, x, gamma, mean, rstd, T_, h, dx, pg, pb, status, st, &units);
        else
            e = backward_rows<T, 1>(p, dy, x, gamma, mean, rstd, T_, h, dx, pg, pb, status, st, &units);
        if (e != cudaSuccess) return e;
        ++*launches;
        if (p.units == 1) return cudaSuccess;
        return param_reduce(pg, pb, units, h, dgamma, dbeta, st, launches);
    }
    e = launch_dependent(norm_backward_kernel<T>, dim3(T_), dim3(kRowThreads), 0, st, dy, x, gamma, mean, rstd,
                         h, dx);
    if (e != cudaSuccess) return e;
    const int chunks = norm_param_parts(T_, h, sizeof(T));
    float* pb = partial + static_cast<size_t>(chunks) * h;
    e = launch_dependent(norm_param_grad_kernel<T>, dim3(ceil_div(h, 32), chunks), dim3(256), 0, st, dy, x,
                         mean, rstd, T_, h, ceil_div(T_, chunks), partial);
    if (e != cudaSuccess) return e;
    *launches += 2;
    return param_reduce(partial, pb, chunks, h, dgamma, dbeta, st, launches);
}

}  // namespace

int norm_param_parts(int T, int h, int elem) {
    const NormPlan p = norm_plan(T, h, elem);
    if (p.units > 0) return p.units;
    const long long col_blocks = (h + 31) / 32;
    return static_cast<int>(std::max(1LL, std::min<long long>((1216 + col_blocks - 1) / col_blocks, (T + 31) / 32)));
}

cudaError_t launch_norm_forward(int dtype, const void* x, const void* gamma, const void* beta, int T,
                                int h, float eps, void* y, float* mean, float* rstd,
                                cudaStream_t st, int* launches) {
    switch (dtype) {
        case TPMLP_BF16: return forward<__nv_bfloat16>(x, gamma, beta, T, h, eps, y, mean, rstd, st, launches);
        case TPMLP_FP16: return forward<__half>(x, gamma, beta, T, h, eps, y, mean, rstd, st, launches);
        default: return forward<float>(x, gamma, beta, T, h, eps, y, mean, rstd, st, launches);
    }
}

cudaError_t launch_norm_backward(int dtype, const void* dy, const void* x, const void* gamma,
                                 const float* mean, const float* rstd, int T, int h, void* dx,
                                 float* dgamma, float* dbeta, float* partial, int* status, cudaStream_t st,
                                 int* launches) {
    auto run = [&](auto* t) {
        return backward<std::remove_pointer_t<decltype(t)>>(dy, x, gamma, mean, rstd, T, h, dx, dgamma, dbeta,
                                                            partial, status, st, launches);
    };
    switch (dtype) {
        case TPMLP_BF16: return run(static_cast<__nv_bfloat16*>(nullptr));
        case TPMLP_FP16: return run(static_cast<__half*>(nullptr));
        default: return run(static_cast<float*>(nullptr));
    }
}

}  // namespace tpmlp
