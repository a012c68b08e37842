// head_loss.cu -- the row kernels of the output head's softmax cross entropy
// (the GEMMs that make the logits and their gradient are in
// gemm_head_loss.cu).
//
// Per token t with logits z_v = X_t . W_v and target y:
//   others = log sum_{v != y} exp(z_v)
//   loss   = log(1 + exp(others - z_y))        lse = z_y + loss
// which is lse - z_y, but keeps its relative precision where the model is
// sure of the target and lse and z_y are near equals.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "kernels.h"

namespace tpmlp {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float dot8(const uint4 a, const uint4 b) {
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        s = fmaf(__uint_as_float(x[j] << 16), __uint_as_float(y[j] << 16), s);
        s = fmaf(__uint_as_float(x[j] & 0xFFFF0000u), __uint_as_float(y[j] & 0xFFFF0000u), s);
    }
    return s;
}

// Thread `sub` of `group`'s share of the dot product of two rows of n pieces of
// 8 values, loads in batches.
__device__ __forceinline__ float dot_rows(const __nv_bfloat16* a_row, const __nv_bfloat16* b_row, int n, int sub,
                                          int group) {
    const uint4* x = reinterpret_cast<const uint4*>(a_row);
    const uint4* w = reinterpret_cast<const uint4*>(b_row);
    float dot = 0.0f;
    for (int i = sub; i < n; i += 4 * group) {
        uint4 a[4], b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool in = i + j * group < n;
            a[j] = in ? __ldg(x + i + j * group) : make_uint4(0u, 0u, 0u, 0u);
            b[j] = in ? __ldg(w + i + j * group) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) dot += dot8(a[j], b[j]);
    }
    return dot;
}

// {m, s} stands for s 2^(m log2(e)); m = -inf: nothing.
__device__ __forceinline__ float2 join(float2 a, float2 b) {
    const float m = fmaxf(a.x, b.x);
    const float shift = m == -INFINITY ? 0.0f : m;
    return make_float2(m, a.y * ex2_approx((a.x - shift) * kLog2e) + b.y * ex2_approx((b.x - shift) * kLog2e));
}

// A number as the sum of two floats, the second below half a step of the
// first: twice a float's precision for the few values that need it (double
// precision instructions are rare and slow on this part).  `add` takes the exact
// error of the upper sum by Knuth's two-sum (The Art of Computer Programming 2,
// 4.2.2).
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two add(Two a, Two b) {
    const float s = __fadd_rn(a.hi, b.hi), t = __fsub_rn(s, a.hi);
    const float e = __fadd_rn(__fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(b.hi, t)), __fadd_rn(a.lo, b.lo));
    const float hi = __fadd_rn(s, e);
    return Two{hi, __fsub_rn(e, __fsub_rn(hi, s))};
}

// m + log(s), s >= 0: the exponent of s apart, so that the float logarithm is of
// a number near 1.  ln 2 is cut to 12 bits and a rest (Cody and Waite's
// reduction): k times the former is exact.
__device__ __forceinline__ Two log_sum(float m, float s) {
    if (!(s > 0.0f && s < INFINITY)) return Two{m + logf(s), 0.0f};
    const int k = ((__float_as_int(s) >> 23) & 0xFF) - 127;  // s is a sum of powers of two near 1: normal
    const float f = __int_as_float(__float_as_int(s) - (k << 23));
    constexpr float kLn2Hi = 0.693115234375f, kLn2Lo = 3.194618498e-05f;
    return add(add(Two{m, 0.0f}, Two{k * kLn2Hi, 0.0f}), Two{fmaf(static_cast<float>(k), kLn2Lo, logf(f)), 0.0f});
}

// What the loss and lse of a row come from: {m, s} of the classes beside the
// target, the target's logit, and what to do with them.
struct Row {
    float2 others;
    Two logit;
    int y;  // the target, V for one outside the vocabulary
};

__device__ __forceinline__ void finish_row(const Row& r, Two log_others, int V, float* loss, float* lse) {
    if (r.y < 0) {  // ignored token
        *loss = 0.0f;
        *lse = log_others.hi;
    } else if (r.y >= V) {  // no such class: never silent
        *loss = __int_as_float(0x7FC00000);
        *lse = log_others.hi;
    } else {
        const Two d = log_others.hi == -INFINITY ? log_others : add(log_others, Two{-r.logit.hi, -r.logit.lo});
        float e = expf(-fabsf(d.hi));
        if (fabsf(d.hi) < 100.0f) e = fmaf(e, d.hi > 0.0f ? -d.lo : d.lo, e);
        const float l = d.hi != d.hi ? d.hi : fmaxf(d.hi, 0.0f) + log1pf(e);
        *loss = l;
        *lse = r.logit.hi + (r.logit.lo + l);
    }
}

// A class whose share of a row's sum is w / s (w: its term beside the
// largest's, s: the sum, log s: near enough `log_others`) puts that share of its
// logit's error into lse.  A tensor-core logit is off by about h |z| 2^-30:
// whether that is more than 2^-20 of lse.
__device__ __forceinline__ bool too_coarse(float z, float w, float s, float log_others, int h) {
    return static_cast<float>(h) * fabsf(z) * w > 1024.0f * s * fmaxf(1.0f, fabsf(log_others));
}

// A CTA takes `rows` rows (a power of two up to 32), kThreads / rows threads
// a row: they join the row's column parts and take the dot product of the
// target's logit in fp32.  (A tensor-core accumulator is cut toward zero at
// every step of 16: a logit of 20 from a row of 20480 values comes out 5e-4
// small.)  Where other classes make much of a row's sum -- a model sure of
// the wrong token or torn between a few, or a token that does not count --
// their logits are taken again like that, the largest of each column part that
// has one: the GEMM says which 16 columns hold it.  (A second large class in
// the same part keeps its accumulator's error, that share of h |z| 2^-30.)
__global__ void __launch_bounds__(kThreads)
    head_combine_kernel(const float2* __restrict__ parts, const uint8_t* __restrict__ where, int n_parts,
                        int part_cols, const __nv_bfloat16* __restrict__ X, const __nv_bfloat16* __restrict__ W,
                        const long long* __restrict__ targets, int T, int h, int V, int rows,
                        float* __restrict__ loss, float* __restrict__ lse) {
    pdl_launch_dependents();  // the next kernel may begin its launch
    pdl_wait();               // the parts come from the kernel before this one
    __shared__ float2 warp_part[kThreads / 32];
    __shared__ Two warp_dot[kThreads / 32];
    __shared__ Row again[32];  // rows whose largest logits are taken again
    __shared__ bool is_again[32];
    const int group = kThreads / rows;  // threads a row, 8..256
    const int r = threadIdx.x / group, sub = threadIdx.x % group;
    const int row = blockIdx.x * rows + r;
    const bool ok = row < T;
    const long long y = ok ? __ldg(targets + row) : -1;
    const float2 none = make_float2(-INFINITY, 0.0f);
    float2 acc = none;
    float dot = 0.0f;
    // The loads come in batches, the first parts' before the dot product, whose
    // addresses wait for the target: one latency after the other was 21 us at
    // 8192 tokens.
    constexpr int kBatch = 8;
    float2 batch[kBatch];
    auto load_parts = [&](int first) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = first + j * group;
            batch[j] = ok && i < n_parts ? __ldg(parts + static_cast<long long>(i) * T + row) : none;
        }
    };
    load_parts(sub);
    if (ok && y >= 0 && y < V)
        dot = dot_rows(X + static_cast<long long>(row) * h, W + y * h, h >> 3, sub, group);
    for (int i = sub;;) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) acc = join(acc, batch[j]);
        i += kBatch * group;
        if (i >= n_parts) break;
        load_parts(i);
    }
    // The threads' shares of the dot product meet as two floats: one holds a
    // logit of 20 to 1e-6, which would be the relative error of a small loss.
    Two logit{dot, 0.0f};
    const int width = min(group, 32);
    for (int off = width >> 1; off >= 1; off >>= 1) {
        float2 o;
        o.x = __shfl_xor_sync(0xFFFFFFFFu, acc.x, off);
        o.y = __shfl_xor_sync(0xFFFFFFFFu, acc.y, off);
        acc = join(acc, o);
        Two l;
        l.hi = __shfl_xor_sync(0xFFFFFFFFu, logit.hi, off);
        l.lo = __shfl_xor_sync(0xFFFFFFFFu, logit.lo, off);
        logit = add(logit, l);
    }
    if (group > 32) {
        if ((threadIdx.x & 31) == 0) {
            warp_part[threadIdx.x >> 5] = acc;
            warp_dot[threadIdx.x >> 5] = logit;
        }
        __syncthreads();
        if (sub == 0) {
            for (int w = 1; w < group / 32; ++w) {
                acc = join(acc, warp_part[(threadIdx.x >> 5) + w]);
                logit = add(logit, warp_dot[(threadIdx.x >> 5) + w]);
            }
        }
    }
    bool redo = false;
    if (sub == 0 && ok) {
        const Row mine{acc, logit, y < 0 ? -1 : static_cast<int>(min(y, static_cast<long long>(V)))};
        const Two others = log_sum(acc.x, acc.y);
        // (Not where the target outweighs the sum, so that it does not matter; nor
        // where 64 classes' worth share the sum, which up to h = 65536 the test itself
        // excludes: beyond, it would be a second product of the row with most of W.)
        const bool outweighed = y >= 0 && y < V && logit.hi > others.hi + 20.0f;
        redo = where != nullptr && !outweighed && acc.y < 64.0f && too_coarse(acc.x, 1.0f, acc.y, others.hi, h);
        if (redo)
            again[r] = mine;
        else
            finish_row(mine, others, V, loss + row, lse + row);
    }
    if (sub == 0) is_again[r] = redo;
    if (!__syncthreads_or(redo)) return;
    __shared__ Two z[16];
    __shared__ unsigned coarse[kThreads / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int k = 0; k < rows; ++k) {
        if (!is_again[k]) continue;  // the same in all threads
        const int at = blockIdx.x * rows + k;
        const Row q = again[k];
        const Two log_others = log_sum(q.others.x, q.others.y);
        const uint4* x = reinterpret_cast<const uint4*>(X + static_cast<long long>(at) * h);
        float more = 0.0f;  // thread 0: what the sum lacks, part by part
        for (int first = 0; first < n_parts; first += kThreads) {
            const int mine = first + threadIdx.x;
            const float m = mine < n_parts ? __ldg(parts + static_cast<long long>(mine) * T + at).x : -INFINITY;
            const float w = ex2_approx((m - q.others.x) * kLog2e);
            const bool again_here = m > -INFINITY && too_coarse(m, w, q.others.y, log_others.hi, h);
            const unsigned bits = __ballot_sync(0xFFFFFFFFu, again_here);
            if (lane == 0) coarse[warp] = bits;
            __syncthreads();
            for (int i = 0; i < kThreads / 32; ++i) {
                for (unsigned left = coarse[i]; left != 0; left &= left - 1) {
                    const int part = first + 32 * i + __ffs(left) - 1;
                    const long long p = static_cast<long long>(part) * T + at;
                    const float was = __ldg(parts + p).x;
                    const int col = part * part_cols + 16 * __ldg(where + p);
                    for (int c = warp; c < 16; c += kThreads / 32) {
                        const int v = col + c;
                        const bool in = v < V && v != q.y;
                        const uint4* w8 = reinterpret_cast<const uint4*>(W + static_cast<long long>(in ? v : 0) * h);
                        float d = 0.0f;
#pragma unroll 4
                        for (int j = lane; j < (h >> 3); j += 32) d += dot8(__ldg(x + j), __ldg(w8 + j));
                        Two sum{d, 0.0f};
#pragma unroll
                        for (int off = 16; off >= 1; off >>= 1) {
                            Two o;
                            o.hi = __shfl_xor_sync(0xFFFFFFFFu, sum.hi, off);
                            o.lo = __shfl_xor_sync(0xFFFFFFFFu, sum.lo, off);
                            sum = add(sum, o);
                        }
                        if (lane == 0) z[c] = in ? sum : Two{-INFINITY, 0.0f};
                    }
                    __syncthreads();
                    if (threadIdx.x == 0) {
                        Two best = z[0];
                        for (int c = 1; c < 16; ++c)
                            if (z[c].hi > best.hi) best = z[c];
                        more += ex2_approx((was - q.others.x) * kLog2e) * expm1f((best.hi - was) + best.lo);
                    }
                    __syncthreads();
                }
            }
            __syncthreads();  // coarse[] is read
        }
        if (threadIdx.x == 0)
            finish_row(q, log_sum(q.others.x, q.others.y + more), V, loss + at, lse + at);
    }
}

// The largest |dloss| of the tokens that count (1 where that is 0 or not
// finite), taken by one CTA over all of them.  The logits' gradients are
// divided by it, so that in the usual case, one weight for all counted tokens,
// the weights are exactly 1 and the bf16 gradient rounds p - [v == y] itself,
// not its product with an arbitrary factor; it multiplies the fp32 sums of dX
// and dW.
__device__ __forceinline__ float dloss_scale(const float* __restrict__ dloss, const long long* __restrict__ targets,
                                             int T) {
    __shared__ float most[kThreads / 32];
    constexpr int kBatch = 8;  // a thread's loads in flight
    float s = 0.0f;
    for (long long t0 = threadIdx.x; t0 < T; t0 += kBatch * kThreads) {
        float d[kBatch];
        int sign[kBatch];  // the targets' upper halves
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const long long t = t0 + j * kThreads;
            d[j] = t < T ? __ldg(dloss + t) : 0.0f;
            sign[j] = t < T ? __ldg(reinterpret_cast<const int*>(targets) + 2 * t + 1) : -1;
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (sign[j] >= 0) s = fmaxf(s, fabsf(d[j]));  // (a NaN counts as 0)
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s = fmaxf(s, __shfl_xor_sync(0xFFFFFFFFu, s, off));
    if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = s;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) s = fmaxf(s, most[w]);
    return s > 0.0f && s < INFINITY ? s : 1.0f;
}

// q[t] = exp(z - lse[t]) - 1 for the logit z of token t's target, 0 where there
// is none: what the backward pass has of it beside the other classes'
// probabilities.  With the model sure of the target, z and lse are near equals,
// and z as the GEMM has it -- cut toward zero at every step, 5e-4 small at a
// logit of 20 from 20480 products -- would leave nothing of their difference
// (the gradient of such a token came out some hundred times too large).  So z
// is taken in fp32, as forward, and only the difference is rounded.
// `rows` rows a CTA as in head_combine_kernel; CTA 0 takes the largest |dloss|.
// 3 to 5 us a call up to 1024 tokens, of which 2 are the launch; 10 us for 8192
// x 1024 (X and the targets' rows of W, 34 MB, 3.4 TB/s).
__global__ void __launch_bounds__(kThreads)
    head_target_kernel(const float* __restrict__ dloss, const __nv_bfloat16* __restrict__ X,
                       const __nv_bfloat16* __restrict__ W, const long long* __restrict__ targets,
                       const float* __restrict__ lse, int T, int h, int V, int rows, float* __restrict__ q,
                       float* __restrict__ scale) {
    pdl_launch_dependents();  // the next kernel may begin its launch
    pdl_wait();               // X comes from the kernel before this one
    if (blockIdx.x == 0) {
        const float s = dloss_scale(dloss, targets, T);
        if (threadIdx.x == 0) *scale = s;
        return;
    }
    __shared__ Two warp_dot[kThreads / 32];
    const int group = kThreads / rows;  // threads a row, 8..256
    const int r = threadIdx.x / group, sub = threadIdx.x % group;
    const int row = (blockIdx.x - 1) * rows + r;
    const bool ok = row < T;
    const long long y = ok ? __ldg(targets + row) : -1;
    const bool in = y >= 0 && y < V;
    const float l = ok ? __ldg(lse + row) : 0.0f;
    Two z{in ? dot_rows(X + static_cast<long long>(row) * h, W + y * h, h >> 3, sub, group) : 0.0f, 0.0f};
    for (int off = min(group, 32) >> 1; off >= 1; off >>= 1) {
        Two o;
        o.hi = __shfl_xor_sync(0xFFFFFFFFu, z.hi, off);
        o.lo = __shfl_xor_sync(0xFFFFFFFFu, z.lo, off);
        z = add(z, o);
    }
    if (group > 32) {
        if ((threadIdx.x & 31) == 0) warp_dot[threadIdx.x >> 5] = z;
        __syncthreads();
        if (sub == 0)
            for (int w = 1; w < group / 32; ++w) z = add(z, warp_dot[(threadIdx.x >> 5) + w]);
    }
    if (sub == 0 && ok) q[row] = in ? expm1f((z.hi - l) + z.lo) : 0.0f;
}

// out[i] = bf16(s sum_k P[k][i]): a CTA takes 256 / chains pieces of 8 values,
// `chains` threads a piece (1, or 16 or 32 for many planes of few values),
// each adding planes c, c + chains, ... in order; then the chains in order.
// `mend`, called before the planes are read, returns what adds the rest that
// the sum lacks to the 8 values at i.
template <typename Mend>
__device__ __forceinline__ void reduce_planes(const float* __restrict__ P, int planes, long long count,
                                              int chains, float s, __nv_bfloat16* __restrict__ out,
                                              Mend&& mend) {
    __shared__ float part[kThreads][9];
    const int pieces = kThreads / chains;
    const int chain = threadIdx.x / pieces, piece = threadIdx.x % pieces;
    const long long i = (static_cast<long long>(blockIdx.x) * pieces + piece) * 8;
    const bool ok = i < count;
    float a[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = 0.0f;
    const auto rest = mend(i, chain == 0 && ok);
    if (ok) {
#pragma unroll 4
        for (int k = chain; k < planes; k += chains) {
            const float4* q = reinterpret_cast<const float4*>(P + k * count + i);
            const float4 x = __ldg(q), y = __ldg(q + 1);
            a[0] += x.x; a[1] += x.y; a[2] += x.z; a[3] += x.w;
            a[4] += y.x; a[5] += y.y; a[6] += y.z; a[7] += y.w;
        }
    }
    if (chains > 1) {
#pragma unroll
        for (int j = 0; j < 8; ++j) part[threadIdx.x][j] = a[j];
        __syncthreads();
        if (chain == 0) {
            for (int k = 1; k < chains; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) a[j] += part[k * pieces + piece][j];
        }
    }
    if (chain != 0 || !ok) return;
    rest(a);
    uint4 o;
    o.x = pack_bf16x2(s * a[0], s * a[1]);
    o.y = pack_bf16x2(s * a[2], s * a[3]);
    o.z = pack_bf16x2(s * a[4], s * a[5]);
    o.w = pack_bf16x2(s * a[6], s * a[7]);
    *reinterpret_cast<uint4*>(out + i) = o;
}

__global__ void __launch_bounds__(kThreads)
    head_reduce_kernel(const float* __restrict__ P, int planes, long long count, int chains,
                       const float* __restrict__ scale, __nv_bfloat16* __restrict__ out) {
    pdl_launch_dependents();  // the next kernel may begin its launch
    pdl_wait();               // its inputs come from the kernel before it
    reduce_planes(P, planes, count, chains, __ldg(scale), out, [](long long, bool) { return [](float(&)[8]) {}; });
}

__device__ __forceinline__ void add_scaled8(float (&x)[8], float e, const uint4 u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = fmaf(e, __uint_as_float(w[i] << 16), x[2 * i]);
        x[2 * i + 1] = fmaf(e, __uint_as_float(w[i] & 0xFFFF0000u), x[2 * i + 1]);
    }
}

// The end of the few-token backward pass (T <= 16).  A target's dz is most of
// its token's gradient, and with few tokens its one rounding to bf16 would be
// most of the error: up to half a step of 2^-8, where many tokens average it
// out.  So CTAs 0 .. reduce_ctas - 1 sum dX's planes and add err[t] W[y_t], what
// that rounding lost; and CTA reduce_ctas + k computes dW's row of token k's
// target once more, from fp32 dz: the T logits of that row are dot products of
// a few rows.  (Mending both where the target's row passes by made the large
// kernel a fifth slower.)
__global__ void __launch_bounds__(kThreads)
    head_few_finish_kernel(const float* __restrict__ P, int planes, int chains, int reduce_ctas,
                           const float* __restrict__ scale, const float* __restrict__ err,
                           const float* __restrict__ dloss, const float* __restrict__ lse,
                           const long long* __restrict__ targets, const __nv_bfloat16* __restrict__ X,
                           const __nv_bfloat16* __restrict__ W, int T, int h, int V,
                           __nv_bfloat16* __restrict__ dX, __nv_bfloat16* __restrict__ dW) {
    pdl_launch_dependents();  // the next kernel may begin its launch
    pdl_wait();               // its inputs come from the kernel before it
    const float s = __ldg(scale);
    if (static_cast<int>(blockIdx.x) < reduce_ctas) {
        reduce_planes(P, planes, static_cast<long long>(T) * h, chains, s, dX, [&](long long i, bool here) {
            const int t = here ? static_cast<int>(i / h) : 0;
            const long long y = __ldg(targets + t);
            const bool in = here && y >= 0 && y < V;
            const uint4 w = in ? __ldg(reinterpret_cast<const uint4*>(W + y * h + (i - static_cast<long long>(t) * h)))
                               : make_uint4(0u, 0u, 0u, 0u);
            const float e = in ? __ldg(err + t) : 0.0f;
            return [=](float(&a)[8]) {
                if (in) add_scaled8(a, e, w);
            };
        });
        return;
    }
    __shared__ float sums[kThreads / 32][16];
    __shared__ float dz[16];
    const int own = static_cast<int>(blockIdx.x) - reduce_ctas;
    // A token a lane, all loads at once: one after the other their latencies
    // would be most of this kernel's time.
    const int n = h >> 3, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool token = lane < T;
    const long long yt = token ? __ldg(targets + lane) : -1;
    const float gt = token ? __ldg(dloss + lane) : 0.0f, lse_t = token ? __ldg(lse + lane) : 0.0f;
    const long long y = __shfl_sync(0xFFFFFFFFu, yt, own);
    if (y < 0 || y >= V) return;
    if (__any_sync(0xFFFFFFFFu, lane < own && yt == y)) return;  // an earlier token's CTA does the row
    const uint4* w = reinterpret_cast<const uint4*>(W + y * h);
    float dot[16];
#pragma unroll
    for (int t = 0; t < 16; ++t) dot[t] = 0.0f;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint4 u = __ldg(w + i);
#pragma unroll
        for (int t = 0; t < 16; ++t)
            if (t < T) dot[t] += dot8(__ldg(reinterpret_cast<const uint4*>(X + static_cast<long long>(t) * h) + i), u);
    }
#pragma unroll
    for (int t = 0; t < 16; ++t) {
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) dot[t] += __shfl_xor_sync(0xFFFFFFFFu, dot[t], off);
        if (lane == 0) sums[warp][t] = dot[t];
    }
    __syncthreads();
    if (threadIdx.x < 16) {
        const int t = threadIdx.x;
        float z = 0.0f, d = 0.0f;
#pragma unroll
        for (int k = 0; k < kThreads / 32; ++k) z += sums[k][t];
        if (yt >= 0) {
            const float g = yt < V ? gt / s : __int_as_float(0x7FC00000);
            d = g * ex2_approx(fmaf(z, kLog2e, -lse_t * kLog2e)) - (yt == y ? g : 0.0f);
        }
        dz[t] = d;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
        float a[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = 0.0f;
#pragma unroll
        for (int t = 0; t < 16; ++t)
            if (t < T) add_scaled8(a, dz[t], __ldg(reinterpret_cast<const uint4*>(X + static_cast<long long>(t) * h) + i));
        uint4 o;
        o.x = pack_bf16x2(s * a[0], s * a[1]);
        o.y = pack_bf16x2(s * a[2], s * a[3]);
        o.z = pack_bf16x2(s * a[4], s * a[5]);
        o.w = pack_bf16x2(s * a[6], s * a[7]);
        reinterpret_cast<uint4*>(dW + y * h)[i] = o;
    }
}

int chains_for(int planes) { return planes >= 64 ? 32 : planes >= 8 ? 16 : 1; }

unsigned blocks_of(long long n, long long per) { return static_cast<unsigned>((n + per - 1) / per); }

// As many rows a CTA of the row kernels as let all run at once, five an SM: few
// rows get many threads (1000 rows with 256 each need a second wave: 9 us more).
int rows_a_cta(int T) {
    int rows = 1;
    while (rows < 32 && T > 5 * 152LL * rows) rows *= 2;
    return rows;
}

}  // namespace

cudaError_t launch_head_combine(const float2* parts, const uint8_t* where, int n_parts, int part_cols,
                                const __nv_bfloat16* X, const __nv_bfloat16* W, const long long* targets, int T,
                                int h, int V, float* loss, float* lse, cudaStream_t st, int* launches) {
    const int rows = rows_a_cta(T);
    ++*launches;
    return launch_dependent(head_combine_kernel, dim3(blocks_of(T, rows)), dim3(kThreads), 0, st, parts,
                            where, n_parts, part_cols, X, W, targets, T, h, V, rows, loss, lse);
}

cudaError_t launch_head_target(const float* dloss, const __nv_bfloat16* X, const __nv_bfloat16* W,
                               const long long* targets, const float* lse, int T, int h, int V, float* q,
                               float* scale, cudaStream_t st, int* launches) {
    const int rows = rows_a_cta(T);
    ++*launches;
    return launch_dependent(head_target_kernel, dim3(1 + blocks_of(T, rows)), dim3(kThreads), 0, st, dloss, X, W,
                            targets, lse, T, h, V, rows, q, scale);
}

cudaError_t launch_head_reduce(const float* P, int planes, long long count, const float* scale,
                               __nv_bfloat16* out, cudaStream_t st, int* launches) {
    ++*launches;
    const int chains = chains_for(planes);
    return launch_dependent(head_reduce_kernel, dim3(blocks_of(count / 8, kThreads / chains)), dim3(kThreads), 0, st,
                            P, planes, count, chains, scale, out);
}

cudaError_t launch_head_few_finish(const float* P, int planes, const float* scale, const float* err,
                                   const float* dloss, const float* lse, const long long* targets,
                                   const __nv_bfloat16* X, const __nv_bfloat16* W, int T, int h, int V,
                                   __nv_bfloat16* dX, __nv_bfloat16* dW, cudaStream_t st, int* launches) {
    ++*launches;
    const int chains = chains_for(planes);
    const int ctas = static_cast<int>(blocks_of(static_cast<long long>(T) * h / 8, kThreads / chains));
    return launch_dependent(head_few_finish_kernel, dim3(ctas + T), dim3(kThreads), 0, st, P, planes, chains, ctas,
                            scale, err, dloss, lse, targets, X, W, T, h, V, dX, dW);
}

}  // namespace tpmlp
