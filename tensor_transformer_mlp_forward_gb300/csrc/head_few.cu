// head_few.cu -- the output head for at most 16 tokens.
//
// With so few tokens the vocabulary matrix W [V, h] is everything: the
// forward pass reads it once (103 MB at 50257 x 1024: 15.4 us at the measured
// 6.67 TB/s), the backward pass reads it and writes a dW of its size.  A
// tcgen05 tile has 128 rows, so here nearly all of its rows would be padding
// loaded and multiplied for nothing (one token took 41 us that way).  These
// kernels stream W through registers into warp-level matrix instructions,
// m16n8k16, bf16 in, fp32 sums.
//
// A matrix instruction sums over k in any order as long as both operands use
// the same one.  So a lane takes 16 consecutive bytes of a row (8 values) as
// its share of two k16 steps, for W and for X alike, and nothing is staged
// in shared memory or transposed: a warp's load of 8 rows fills whole
// sectors.  A matrix instruction takes 32 clocks or so of a quarter of an SM
// whatever it multiplies, so the tokens are its columns, eight at a time, and
// the vocabulary or the columns of W its 16 rows.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "kernels.h"

namespace tpmlp {
namespace {

constexpr int kTokens = 16;   // at most
constexpr int kWarps = 4;     // of a CTA
constexpr int kRows = 32;     // vocabulary rows of a task: two m16 tiles, loaded eight rows at a time
constexpr int kTiles = kRows / 8;
constexpr int kKStep = 64;    // columns of a step: 128 bytes of a row
constexpr int kCtasPerSm = 4;  // of the logits kernel
constexpr int kGradCtas = 4;   // of the gradient kernel
constexpr int kSms = 152;
constexpr int kColumns = 64;  // columns of W that a warp of the gradient kernel owns

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma1688(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(b0));
}

// A read that nothing will ask for again soon (W is larger than L1).
__device__ __forceinline__ uint4 load_stream(const void* p) {
    uint4 u;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "l"(p));
    return u;
}

// The largest |dloss| of the tokens that count, which scales the gradients (1
// where it is 0 or not finite).  A token a lane: one after the other their
// loads' latencies added up to some microseconds.  Called by whole warps.
__device__ __forceinline__ float dloss_scale(const float* dloss, const long long* targets, int T) {
    const int lane = threadIdx.x & 31;
    const long long y = lane < T ? __ldg(targets + lane) : -1;
    const float d = lane < T ? fabsf(__ldg(dloss + lane)) : 0.0f;
    float s = fmaxf(y >= 0 ? d : 0.0f, 0.0f);  // (a NaN counts as 0)
#pragma unroll
    for (int off = kTokens / 2; off >= 1; off >>= 1) s = fmaxf(s, __shfl_xor_sync(0xFFFFFFFFu, s, off));
    s = __shfl_sync(0xFFFFFFFFu, s, 0);
    return s > 0.0f && s < INFINITY ? s : 1.0f;
}

struct FewArgs {
    const __nv_bfloat16 *X, *W;
    const long long* targets;
    int T, h, V;
    float2* parts;  // forward: {max, sum of exponentials}, [CTA][T]
    // backward
    const float *dloss, *lse;
    __nv_bfloat16 *dz, *dzt;  // [16][ldz] and [ldz][16]
    int ldz;
    float* scale;
    float* err;  // [16]: what each target's dz lost in its rounding (mended at the end)
};

// Logits of the 16 tokens against tasks of 32 vocabulary rows, CTA b taking
// tasks b, b + grid, ... (neighbours in memory at the same time).  The four
// warps split k (64 columns each in turn, so that together they read 512
// consecutive bytes of a row) and their sums meet in shared memory.  Then
// thread (token, 4 rows): forward, the running maximum and sum of
// exponentials; backward, the logits' gradient.  The loads run one step ahead,
// across the tasks too: a task has few steps (four a warp at h = 1024), and
// starting each anew left the memory idle a third of the time.
template <bool GRAD, int TT>
__global__ void __launch_bounds__(32 * kWarps, kCtasPerSm) head_few_logits_kernel(const FewArgs p) {
    pdl_launch_dependents();  // the next kernel may begin its launch
    __shared__ __align__(16) float red[2][kWarps][8 * TT][kRows + 4];
    __shared__ __align__(16) __nv_bfloat16 tr[2][kRows][kTokens];
    pdl_wait();  // X comes from the kernel before this one
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int steps = (p.h + kKStep - 1) / kKStep;
    const __nv_bfloat16* x[TT];
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) x[tt] = p.X + static_cast<long long>(g + 8 * tt < p.T ? g + 8 * tt : 0) * p.h + q * 8;

    // this thread's token and rows of a task behind the meeting of the sums
    const int t = threadIdx.x / (kRows / 4), vq = threadIdx.x % (kRows / 4) * 4;
    long long y = -1;
    float mx = -INFINITY, sum = 0.0f, lse2 = INFINITY, weight = 0.0f;
    if (t < p.T) y = __ldg(p.targets + t);
    if constexpr (GRAD) {
        const float s = dloss_scale(p.dloss, p.targets, p.T);
        if (blockIdx.x == 0 && threadIdx.x == 0) *p.scale = s;
        if (t < p.T && y >= 0) {
            lse2 = __ldg(p.lse + t) * kLog2e;
            weight = y < p.V ? __ldg(p.dloss + t) / s : __int_as_float(0x7FC00000);
        }
    }

    const int row0 = blockIdx.x * kRows, row_step = gridDim.x * kRows;
    uint4 wb[2][kTiles][2];
    // One step's loads of W: columns 64 step .. of the task at v0.  Rows behind
    // the vocabulary read its last.
    auto load = [&](int v0, int step, int b) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int k = step * kKStep + s * 32;  // + q * 8 .. + 7
            const bool ok = k + q * 8 < p.h;
            const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int i = 0; i < kTiles; ++i)
                wb[b][i][s] = ok ? load_stream(p.W + static_cast<long long>(min(v0 + i * 8 + g, p.V - 1)) * p.h + q * 8 + k)
                                 : z;
        }
    };
    float acc[kTiles / 2][TT][4];
    // X's share of the step comes from L1 when it is needed: the registers go
    // to W's loads in flight.
    auto multiply = [&](int step, int b) {
        uint4 xa[TT][2];
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k = step * kKStep + s * 32;
                xa[tt][s] = k + q * 8 < p.h && g + 8 * tt < p.T ? __ldg(reinterpret_cast<const uint4*>(x[tt] + k))
                                                                 : make_uint4(0u, 0u, 0u, 0u);
            }
        }
        // A step's products are summed by themselves and then added: a matrix
        // instruction cuts its sum towards zero, which over a long row's hundreds
        // of steps would shrink every logit by some 2^-18.
#pragma unroll
        for (int i = 0; i < kTiles / 2; ++i) {
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) {
                float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const uint4 lo = wb[b][2 * i][s], hi = wb[b][2 * i + 1][s];  // rows g, g + 8 of 16
                    mma16816(z, lo.x, hi.x, lo.y, hi.y, xa[tt][s].x, xa[tt][s].y);
                    mma16816(z, lo.z, hi.z, lo.w, hi.w, xa[tt][s].z, xa[tt][s].w);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][tt][e] += z[e];
            }
        }
    };
    int parity = 0;
    int next_v = row0, next_step = warp;  // what the next load takes
    auto load_next = [&](int b) {
        if (next_step >= steps) {
            next_v += row_step;
            next_step = warp;
        }
        if (next_v < p.V && next_step < steps) load(next_v, next_step, b);
        next_step += kWarps;
    };
    const int mine = warp < steps ? (steps - warp + kWarps - 1) / kWarps : 0;  // steps of this warp
    int buf = 0;
    if (mine) load_next(0);
    for (int v0 = row0; v0 < p.V; v0 += row_step, parity ^= 1) {
#pragma unroll
        for (int i = 0; i < kTiles / 2; ++i)
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) acc[i][tt][0] = acc[i][tt][1] = acc[i][tt][2] = acc[i][tt][3] = 0.0f;
        int left = mine, step = warp;
        // the buffers are named by constants: an odd step first, then pairs
        auto one = [&](int b) {
            if (b) {
                load_next(0);
                multiply(step, 1);
            } else {
                load_next(1);
                multiply(step, 0);
            }
            step += kWarps;
        };
        if (left & 1) {
            one(buf);
            buf ^= 1;
            --left;
        }
        if (buf == 0) {
            for (; left > 0; left -= 2) {
                one(0);
                one(1);
            }
        } else {
            for (; left > 0; left -= 2) {
                one(1);
                one(0);
            }
        }
#pragma unroll
        for (int i = 0; i < kTiles / 2; ++i)
#pragma unroll
            for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    red[parity][warp][8 * tt + 2 * q + (e & 1)][16 * i + g + 8 * (e >> 1)] = acc[i][tt][e];
        __syncthreads();
        float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            if (t >= 8 * TT) break;
            const float4 r = *reinterpret_cast<const float4*>(&red[parity][k][t][vq]);
            z[0] += r.x; z[1] += r.y; z[2] += r.z; z[3] += r.w;
        }
        const int v = v0 + vq;
        if constexpr (!GRAD) {
            float bm = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (v + j >= p.V || v + j == y) z[j] = -INFINITY;  // the target is left out (head_loss.cu)
                bm = fmaxf(bm, z[j]);
            }
            const float nm = fmaxf(mx, bm);
            const float shift = nm == -INFINITY ? 0.0f : nm * kLog2e;
            sum *= ex2_approx(fmaf(mx, kLog2e, -shift));
#pragma unroll
            for (int j = 0; j < 4; ++j) sum += ex2_approx(fmaf(z[j], kLog2e, -shift));
            mx = nm;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                z[j] = weight * ex2_approx(fmaf(z[j], kLog2e, -lse2));
                if (v + j == y) z[j] -= weight;
                if (v + j >= p.V) z[j] = 0.0f;
            }
            const uint2 d = make_uint2(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]));
            if (y >= v && y < v + 4) {
                const float own = y == v ? z[0] : y == v + 1 ? z[1] : y == v + 2 ? z[2] : z[3];
                p.err[t] = own - __bfloat162float(__float2bfloat16_rn(own));
            }
            *reinterpret_cast<uint2*>(p.dz + static_cast<long long>(t) * p.ldz + v) = d;
            tr[parity][vq][t] = __ushort_as_bfloat16(static_cast<unsigned short>(d.x));
            tr[parity][vq + 1][t] = __ushort_as_bfloat16(static_cast<unsigned short>(d.x >> 16));
            tr[parity][vq + 2][t] = __ushort_as_bfloat16(static_cast<unsigned short>(d.y));
            tr[parity][vq + 3][t] = __ushort_as_bfloat16(static_cast<unsigned short>(d.y >> 16));
            __syncthreads();
            if (threadIdx.x < kRows * kTokens / 8)
                reinterpret_cast<uint4*>(p.dzt + static_cast<long long>(v0) * kTokens)[threadIdx.x] =
                    reinterpret_cast<const uint4*>(&tr[parity][0][0])[threadIdx.x];
        }
        // the other parity's buffers come next: a warp reaches this one's again
        // only behind the barrier of the task between
    }
    if constexpr (!GRAD) {
#pragma unroll
        for (int off = kRows / 8; off >= 1; off >>= 1) {
            const float om = __shfl_xor_sync(0xFFFFFFFFu, mx, off);
            const float os = __shfl_xor_sync(0xFFFFFFFFu, sum, off);
            const float nm = fmaxf(mx, om);
            const float shift = nm == -INFINITY ? 0.0f : nm;
            sum = sum * ex2_approx((mx - shift) * kLog2e) + os * ex2_approx((om - shift) * kLog2e);
            mx = nm;
        }
        if (vq == 0 && t < p.T) p.parts[static_cast<long long>(blockIdx.x) * p.T + t] = make_float2(mx, sum);
    }
}

// Eight pairs along k from two rows' 8 values.
__device__ __forceinline__ void pairs_of(const uint4 a, const uint4 b, uint32_t (&o)[8]) {
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[2 * i] = __byte_perm(x[i], y[i], 0x5410);
        o[2 * i + 1] = __byte_perm(x[i], y[i], 0x7632);
    }
}

// Rows of more than 1024 values: dX and dW from dz, W read a second time.  A
// warp owns 64 columns and a range of vocabulary rows, 16 of them at a time.
// dX's sums over the range go to plane[range][T][h]; dW = s dz^T X.  Reading W
// and writing dW in one kernel is what HBM serves best: it fills at 3.9 TB/s
// and copies at 6.8 (read and write together), and a kernel that only wrote
// dW took 29 us for 103 MB.  A lane loads 8 columns of rows 2q, 2q + 1, 2q + 8
// and 2q + 9 and byte-permutes them into pairs along the rows: no
// transposition through shared memory.  The warp's 64 columns of X stay in
// registers.  Column n of dW's instruction j is column 8 n + j of the 64, so
// that a lane ends with 16 consecutive columns and whole 128-byte lines leave.
// kDepth steps' loads of W are in flight (one token, 51200 x 20480, both
// kernels: 1158 us with four CTAs an SM and two steps, 1254 with three and
// three, 1317 with four and three.  Four CTAs leave 128 registers: this form
// spills 16 bytes a thread with up to eight tokens, 64 with more).
template <int TT>
__global__ void __launch_bounds__(32 * kWarps, kGradCtas)
    head_few_grad_kernel(const __nv_bfloat16* __restrict__ X, const __nv_bfloat16* __restrict__ W,
                         const __nv_bfloat16* __restrict__ dz, const __nv_bfloat16* __restrict__ dzt,
                         int ldz, const float* __restrict__ scale, int T, int h, int V,
                         int range_rows, __nv_bfloat16* __restrict__ dW, float* __restrict__ plane) {
    constexpr int kDepth = 2;
    pdl_launch_dependents();  // the next kernel may begin its launch
    pdl_wait();               // dz comes from the kernel before this one
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int col0 = (blockIdx.x * kWarps + warp) * kColumns;
    if (col0 >= h) return;
    const int c = min(col0 + g * 8, h - 8);  // columns behind the row are not stored
    uint32_t xb[TT][8];
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
        uint4 r[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int tok = 2 * q + k + 8 * tt;
            r[k] = tok < T ? __ldg(reinterpret_cast<const uint4*>(X + static_cast<long long>(tok) * h + c))
                           : make_uint4(0u, 0u, 0u, 0u);
        }
        pairs_of(r[0], r[1], xb[tt]);
    }
    const float s = __ldg(scale);
    float acc[TT][4][4];  // [.][m]: columns 8 g + 2 m, + 1 of tokens 2 q, 2 q + 1
#pragma unroll
    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
        for (int m = 0; m < 4; ++m) acc[tt][m][0] = acc[tt][m][1] = acc[tt][m][2] = acc[tt][m][3] = 0.0f;
    const int r0 = blockIdx.y * range_rows, r1 = min(r0 + range_rows, V);
    uint4 w[kDepth][4];
    uint32_t d[2][2 * TT], t[2][2 * TT];
    auto load_w = [&](int vb, int b) {
        if (vb >= r1) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // rows behind the vocabulary read its last; dz is 0 there
            const int v = vb + 2 * q + (i & 1) + (i >> 1) * 8;
            w[b][i] = load_stream(W + static_cast<long long>(min(v, V - 1)) * h + c);
        }
    };
    auto load_dz = [&](int vb, int b) {
        if (vb >= r1) return;
#pragma unroll
        for (int i = 0; i < 2 * TT; ++i) {
            d[b][i] = __ldg(reinterpret_cast<const uint32_t*>(dz + static_cast<long long>(g + (i >> 1) * 8) * ldz + vb +
                                                              2 * q + (i & 1) * 8));
            t[b][i] = __ldg(reinterpret_cast<const uint32_t*>(dzt + static_cast<long long>(vb + g + (i & 1) * 8) * kTokens +
                                                              2 * q + (i >> 1) * 8));
        }
    };
#pragma unroll
    for (int b = 0; b < kDepth; ++b) load_w(r0 + 16 * b, b);
    load_dz(r0, 0);
    for (int vb = r0; vb < r1; vb += 32 * kDepth) {
#pragma unroll
        for (int u = 0; u < 2 * kDepth; ++u) {
            const int vr = vb + 16 * u;
            if (vr >= r1) break;
            const int b = u % kDepth, e = u & 1;
            load_dz(vr + 16, e ^ 1);
            {
                uint32_t lo[8], hi[8];
                pairs_of(w[b][0], w[b][1], lo);
                pairs_of(w[b][2], w[b][3], hi);
                load_w(vr + 16 * kDepth, b);
#pragma unroll
                for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                    for (int m = 0; m < 4; ++m)
                        mma16816(acc[tt][m], lo[2 * m], lo[2 * m + 1], hi[2 * m], hi[2 * m + 1], d[e][2 * tt], d[e][2 * tt + 1]);
            }
            float o[8][4];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
                if constexpr (TT == 1)
                    mma1688(o[j], t[e][0], t[e][1], xb[0][j]);
                else
                    mma16816(o[j], t[e][0], t[e][1], t[e][2], t[e][3], xb[0][j], xb[1][j]);
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {  // rows g, g + 8
                const int v = vr + g + 8 * r;
#pragma unroll
                for (int half = 0; half < 2; ++half) {  // columns 16 q .., 16 q + 8 ..
                    const int n = col0 + 16 * q + 8 * half, k = 2 * r + half;
                    if (v < V && n < h)
                        __stcs(reinterpret_cast<uint4*>(dW + static_cast<long long>(v) * h + n),
                               make_uint4(pack_bf16x2(s * o[0][k], s * o[1][k]), pack_bf16x2(s * o[2][k], s * o[3][k]),
                                          pack_bf16x2(s * o[4][k], s * o[5][k]), pack_bf16x2(s * o[6][k], s * o[7][k])));
                }
            }
        }
    }
    if (col0 + g * 8 >= h) return;
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int tok = 2 * q + e + 8 * tt;
            if (tok < T) {
                float4* o = reinterpret_cast<float4*>(plane + (static_cast<long long>(blockIdx.y) * T + tok) * h + c);
                o[0] = make_float4(acc[tt][0][e], acc[tt][0][2 + e], acc[tt][1][e], acc[tt][1][2 + e]);
                o[1] = make_float4(acc[tt][2][e], acc[tt][2][2 + e], acc[tt][3][e], acc[tt][3][2 + e]);
            }
        }
    }
}

// The whole backward pass in one reading of W, for rows of up to 1024 values:
// a CTA takes blocks of 16 vocabulary rows, which the tensor memory
// accelerator brings to shared memory (boxes of 64 columns, 128-byte swizzle,
// a ring of blocks).  A warp owns one or two boxes of every block: its share
// of the logits' sums, then (dz of the block known) its columns of dX and of
// the block's dW.  X stays in registers in both operand forms, dX's sums too.
// The logits of block i + 1 are begun before block i is finished,
// so that one pair of barriers a block serves both.
// The warp-level matrix instructions are what bounds this kernel (with 16
// tokens in their rows: 58 us of which the memory alone needs 22 to read and
// 14 more to write).  So the tokens are their columns, in TT tiles of eight:
// up to eight tokens take half the instructions.
constexpr int kFusedColumns = 1024;
constexpr int kFusedRows = 16;
constexpr int kBoxBytes = kFusedRows * 128;
constexpr int kFusedStageBytes = kFusedColumns / 64 * kBoxBytes;

// Up to eight tokens: two CTAs an SM of eight warps with two boxes each, so
// that one's barriers overlap the other's arithmetic (7 tokens: 57 us with
// one CTA of 16 warps, 47 with two).  Up to 16: the registers of two boxes
// would spill (71 us against 66).
template <int TT>
struct Fused {
    static constexpr int BOXES = TT == 1 ? 2 : 1;  // of a warp
    static constexpr int WARPS = kFusedColumns / 64 / BOXES;
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int CTAS = BOXES;  // an SM
    static constexpr int STAGES = 6 / CTAS;
    static constexpr int SMEM = 1024 + STAGES * kFusedStageBytes;
};

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 u;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(addr));
    return u;
}

template <int TT>
__global__ void __launch_bounds__(Fused<TT>::THREADS, Fused<TT>::CTAS)
    head_few_fused_kernel(const __grid_constant__ CUtensorMap tmW, const FewArgs p,
                          __nv_bfloat16* __restrict__ dW, float* __restrict__ plane, int* status) {
    constexpr int WARPS = Fused<TT>::WARPS, BOXES = Fused<TT>::BOXES, STAGES = Fused<TT>::STAGES;
    pdl_launch_dependents();  // the next kernel may begin its launch
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[STAGES];
    __shared__ float red[WARPS][kFusedRows][8 * TT + 4];
    __shared__ __align__(16) __nv_bfloat16 dzs[8 * TT][kFusedRows], dzts[kFusedRows][8 * TT];
    __shared__ uint32_t abort_flag;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;  // swizzle atoms repeat every 1024 bytes
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int boxes = (p.h + 63) / 64;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) mbar_init(&full[s], 1);
        abort_flag = 0u;
        fence_mbar_init();
        prefetch_tmap(&tmW);
    }
    __syncthreads();
    pdl_wait();  // X comes from the kernel before this one
    const int first = static_cast<int>(blockIdx.x), step = static_cast<int>(gridDim.x);
    const int blocks = (p.V + kFusedRows - 1) / kFusedRows;
    const int n = blocks > first ? (blocks - 1 - first) / step + 1 : 0;
    // Blocks that are copied: all n, or those issued when a wait gave up (the
    // status word is set; the loop goes on, on whatever the buffers hold).
    int to_issue = n;
    auto issue = [&](int i) {  // thread 0: the CTA's i-th block
        if (i >= to_issue) return;
        const int s = i % STAGES;
        mbar_arrive_expect_tx(&full[s], boxes * kBoxBytes);
        for (int b = 0; b < boxes; ++b)
            tma_load_3d(&tmW, smem_u32(&full[s]), ring + s * kFusedStageBytes + b * kBoxBytes, 64 * b, 0,
                        (first + i * step) * kFusedRows);
    };
    if (threadIdx.x == 0)
        for (int i = 0; i < STAGES; ++i) issue(i);

    // X as columns (tokens) x k for the logits, as k (tokens) x columns for dW
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    uint4 xa[BOXES][TT][2];
    uint32_t xb[BOXES][TT][8];
#pragma unroll
    for (int b = 0; b < BOXES; ++b) {
        const int col0 = (warp + b * WARPS) * 64;
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int c = col0 + k * 32 + q * 8, tok = g + 8 * tt;
                xa[b][tt][k] = c < p.h && tok < p.T ? __ldg(reinterpret_cast<const uint4*>(p.X + static_cast<long long>(tok) * p.h + c)) : zero;
            }
            uint4 r[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int c = col0 + g * 8, tok = 2 * q + k + 8 * tt;
                r[k] = c < p.h && tok < p.T ? __ldg(reinterpret_cast<const uint4*>(p.X + static_cast<long long>(tok) * p.h + c)) : zero;
            }
            pairs_of(r[0], r[1], xb[b][tt]);
        }
    }
    // thread (row of the block, token) of the logits' meeting
    const int vr = threadIdx.x / (8 * TT), t = threadIdx.x % (8 * TT);
    long long y = -1;
    float lse2 = INFINITY, weight = 0.0f;
    const float s = dloss_scale(p.dloss, p.targets, p.T);
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.scale = s;
    if (t < p.T) {
        y = __ldg(p.targets + t);
        if (y >= 0) {
            lse2 = __ldg(p.lse + t) * kLog2e;
            weight = y < p.V ? __ldg(p.dloss + t) / s : __int_as_float(0x7FC00000);
        }
    }
    float acc[BOXES][TT][4][4];  // [.][.][m]: columns 8 g + 2 m, + 1 of tokens 2 q, 2 q + 1
#pragma unroll
    for (int b = 0; b < BOXES; ++b)
#pragma unroll
        for (int tt = 0; tt < TT; ++tt)
#pragma unroll
            for (int m = 0; m < 4; ++m)
                acc[b][tt][m][0] = acc[b][tt][m][1] = acc[b][tt][m][2] = acc[b][tt][m][3] = 0.0f;

    // The warp's share of block i's logits, to red.  16-byte piece c of row r
    // sits at position c ^ (r mod 8) of its 128 bytes.
    auto logits = [&](int i) {
        const int st = i % STAGES;
        warp_wait_polls(&full[st], static_cast<uint32_t>(i / STAGES) & 1u, &abort_flag, status,
                        [&] { to_issue = min(to_issue, max(i - 1, 0) + STAGES); });
        float z[TT][4];
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) z[tt][0] = z[tt][1] = z[tt][2] = z[tt][3] = 0.0f;
#pragma unroll
        for (int b = 0; b < BOXES; ++b) {
            if (warp + b * WARPS >= boxes) break;
            const uint32_t box = ring + st * kFusedStageBytes + (warp + b * WARPS) * kBoxBytes + g * 128;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t at = box + (((q + 4 * k) ^ g) << 4);
                const uint4 lo = ld_shared_v4(at), hi = ld_shared_v4(at + 8 * 128);  // rows g, g + 8
#pragma unroll
                for (int tt = 0; tt < TT; ++tt) {
                    mma16816(z[tt], lo.x, hi.x, lo.y, hi.y, xa[b][tt][k].x, xa[b][tt][k].y);
                    mma16816(z[tt], lo.z, hi.z, lo.w, hi.w, xa[b][tt][k].z, xa[b][tt][k].w);
                }
            }
        }
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
            *reinterpret_cast<float2*>(&red[warp][g][8 * tt + 2 * q]) = make_float2(z[tt][0], z[tt][1]);
            *reinterpret_cast<float2*>(&red[warp][g + 8][8 * tt + 2 * q]) = make_float2(z[tt][2], z[tt][3]);
        }
    };
    // dz of block i from the warps' shares, in both operand forms.
    auto gradient = [&](int i) {
        if (vr >= kFusedRows) return;
        const int v = (first + i * step) * kFusedRows + vr;
        float z = 0.0f;
#pragma unroll 4
        for (int w = 0; w < min(boxes, WARPS); ++w) z += red[w][vr][t];
        float d = weight * ex2_approx(fmaf(z, kLog2e, -lse2));
        if (v == y) d -= weight;
        if (v >= p.V) d = 0.0f;
        const __nv_bfloat16 b = __float2bfloat16_rn(d);
        if (v == y) p.err[t] = d - __bfloat162float(b);
        dzs[t][vr] = b;
        dzts[vr][t] = b;
    };
    // dX's sums and dW of block i.
    auto finish = [&](int i) {
        const int v0 = (first + i * step) * kFusedRows;
        uint32_t a[2 * TT], d[TT][2];
#pragma unroll
        for (int k = 0; k < 2 * TT; ++k)
            a[k] = *reinterpret_cast<const uint32_t*>(&dzts[g + (k & 1) * 8][2 * q + (k >> 1) * 8]);
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
            d[tt][0] = *reinterpret_cast<const uint32_t*>(&dzs[g + 8 * tt][2 * q]);
            d[tt][1] = *reinterpret_cast<const uint32_t*>(&dzs[g + 8 * tt][2 * q + 8]);
        }
#pragma unroll
        for (int b = 0; b < BOXES; ++b) {
            if (warp + b * WARPS >= boxes) break;
            const uint32_t box = ring + (i % STAGES) * kFusedStageBytes + (warp + b * WARPS) * kBoxBytes;
            const int col0 = (warp + b * WARPS) * 64;
            {
                uint4 w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = 2 * q + (k & 1) + (k >> 1) * 8;
                    w[k] = ld_shared_v4(box + r * 128 + ((g ^ (r & 7)) << 4));
                }
                uint32_t lo[8], hi[8];
                pairs_of(w[0], w[1], lo);
                pairs_of(w[2], w[3], hi);
#pragma unroll
                for (int tt = 0; tt < TT; ++tt) {
#pragma unroll
                    for (int m = 0; m < 4; ++m)
                        mma16816(acc[b][tt][m], lo[2 * m], lo[2 * m + 1], hi[2 * m], hi[2 * m + 1], d[tt][0], d[tt][1]);
                }
            }
            float o[8][4];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
                if constexpr (TT == 1)
                    mma1688(o[j], a[0], a[1], xb[b][0][j]);
                else
                    mma16816(o[j], a[0], a[1], a[2], a[3], xb[b][0][j], xb[b][1][j]);
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {  // rows g, g + 8
                const int v = v0 + g + 8 * r;
#pragma unroll
                for (int half = 0; half < 2; ++half) {  // columns 16 q .., 16 q + 8 ..
                    const int c = col0 + 16 * q + 8 * half, e = 2 * r + half;
                    if (v < p.V && c < p.h)
                        __stcs(reinterpret_cast<uint4*>(dW + static_cast<long long>(v) * p.h + c),
                               make_uint4(pack_bf16x2(s * o[0][e], s * o[1][e]), pack_bf16x2(s * o[2][e], s * o[3][e]),
                                          pack_bf16x2(s * o[4][e], s * o[5][e]), pack_bf16x2(s * o[6][e], s * o[7][e])));
                }
            }
        }
    };

    if (n > 0) {
        logits(0);
        __syncthreads();
        gradient(0);
        __syncthreads();
    }
    for (int i = 0; i < n; ++i) {
        if (i + 1 < n) logits(i + 1);
        finish(i);
        __syncthreads();  // block i is read, block i + 1's shares are there
        if (threadIdx.x == 0) issue(i + STAGES);
        if (i + 1 < n) gradient(i + 1);
        __syncthreads();
    }
    // copies that a wait has given up on land before the CTA may leave
    if (threadIdx.x == 0 && *static_cast<volatile uint32_t*>(&abort_flag))
        for (int s = 0; s < min(STAGES, to_issue); ++s)
            wait_drain(&full[s], static_cast<uint32_t>((to_issue - 1 - s) / STAGES) & 1u, status);
#pragma unroll
    for (int b = 0; b < BOXES; ++b) {
        const int c = (warp + b * WARPS) * 64 + 8 * g;
        if (c >= p.h) break;
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int tok = 2 * q + e + 8 * tt;
                if (tok < p.T) {
                    const float(&r)[4][4] = acc[b][tt];
                    float4* o = reinterpret_cast<float4*>(plane + (static_cast<long long>(blockIdx.x) * p.T + tok) * p.h + c);
                    o[0] = make_float4(r[0][e], r[0][2 + e], r[1][e], r[1][2 + e]);
                    o[1] = make_float4(r[2][e], r[2][2 + e], r[3][e], r[3][2 + e]);
                }
            }
        }
    }
}

template <int TT>
cudaError_t launch_fused(const CUtensorMap& tm, const FewArgs& a, int ctas, __nv_bfloat16* dW, float* plane,
                         int* status, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(head_few_fused_kernel<TT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Fused<TT>::SMEM);
    if (e != cudaSuccess) return e;
    return launch_dependent(head_few_fused_kernel<TT>, dim3(ctas), dim3(Fused<TT>::THREADS), Fused<TT>::SMEM, st, tm, a, dW,
                            plane, status);
}

int ceil_div(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

}  // namespace

bool head_few(int T) { return T <= kTokens; }

int head_few_parts(int V) { return std::min(ceil_div(V, kRows), kSms * kCtasPerSm); }

int head_few_ldz(int V) { return ceil_div(V, kRows) * kRows; }

// Rows of W that a fused block brings (0: h is too wide for the fused form).
int head_few_box_rows(int h) { return h <= kFusedColumns ? kFusedRows : 0; }

// Planes of dX: the fused form's CTAs, or the ranges of vocabulary rows, as many
// as fill the GPU with CTAs of 256 columns.
int head_few_planes(int T, int h, int V) {
    if (head_few_box_rows(h)) return std::min((T <= 8 ? Fused<1>::CTAS : Fused<2>::CTAS) * kSms, ceil_div(V, kFusedRows));
    const int col_ctas = ceil_div(h, kColumns * kWarps);
    return std::max(1, std::min(kSms * kGradCtas / col_ctas, ceil_div(V, 16)));
}

cudaError_t launch_head_few_lse(const __nv_bfloat16* X, const __nv_bfloat16* W, const long long* targets,
                                int T, int h, int V, float2* parts, cudaStream_t st, int* launches) {
    FewArgs a = {};
    a.X = X; a.W = W; a.targets = targets; a.T = T; a.h = h; a.V = V;
    a.parts = parts;
    ++*launches;
    auto kern = T <= 8 ? head_few_logits_kernel<false, 1> : head_few_logits_kernel<false, 2>;
    return launch_dependent(kern, dim3(head_few_parts(V)), dim3(32 * kWarps), 0, st, a);
}

cudaError_t launch_head_few_backward(const float* dloss, const __nv_bfloat16* X, const __nv_bfloat16* W,
                                     const long long* targets, const float* lse, int T, int h, int V,
                                     __nv_bfloat16* dz, __nv_bfloat16* dzt, float* scale, float* err, float* plane,
                                     __nv_bfloat16* dW, const CUtensorMap* tm, int* status, cudaStream_t st,
                                     int* launches) {
    FewArgs a = {};
    a.X = X; a.W = W; a.targets = targets; a.T = T; a.h = h; a.V = V;
    a.dloss = dloss; a.lse = lse; a.dz = dz; a.dzt = dzt; a.ldz = head_few_ldz(V); a.scale = scale; a.err = err;
    ++*launches;
    cudaError_t e;
    if (head_few_box_rows(h)) {
        const int ctas = head_few_planes(T, h, V);
        return T <= 8 ? launch_fused<1>(*tm, a, ctas, dW, plane, status, st)
                      : launch_fused<2>(*tm, a, ctas, dW, plane, status, st);
    }
    auto kern = T <= 8 ? head_few_logits_kernel<true, 1> : head_few_logits_kernel<true, 2>;
    e = launch_dependent(kern, dim3(head_few_parts(V)), dim3(32 * kWarps), 0,
                                     st, a);
    if (e != cudaSuccess) return e;
    const int planes = head_few_planes(T, h, V);
    const int range_rows = ceil_div(ceil_div(V, planes), 16) * 16;
    ++*launches;
    auto grad = T <= 8 ? head_few_grad_kernel<1> : head_few_grad_kernel<2>;
    return launch_dependent(grad, dim3(ceil_div(h, kColumns * kWarps), planes), dim3(32 * kWarps), 0,
                            st, X, W, static_cast<const __nv_bfloat16*>(dz), static_cast<const __nv_bfloat16*>(dzt),
                            a.ldz, static_cast<const float*>(scale), T, h, V, range_rows, dW, plane);
}

}  // namespace tpmlp
