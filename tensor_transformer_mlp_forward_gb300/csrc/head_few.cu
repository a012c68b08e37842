// head_few.cu -- the output head for at most 16 tokens.
//
// With so few tokens the vocabulary matrix W [V, h] is everything: the
// forward pass reads it once (103 MB at 50257 x 1024: 15.4 us at the measured
// 6.67 TB/s), the backward pass reads it and writes a dW of its size.  A
// tcgen05 tile has 128 rows, so here nearly all of its rows would be padding
// loaded and multiplied for nothing (one token took 41 us that way).  These
// kernels stream W through registers into warp-level matrix instructions,
// whose 16 rows are the tokens: m16n8k16, bf16 in, fp32 sums.
//
// A matrix instruction sums over k in any order as long as both operands use
// the same one.  So a lane takes 16 consecutive bytes of a row (8 values) as
// its share of two k16 steps, for W and for X alike, and nothing is staged
// in shared memory or transposed: a warp's load of 8 rows fills whole
// sectors.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "kernels.h"

namespace tpmlp {
namespace {

constexpr int kTokens = 16;   // rows of a matrix instruction
constexpr int kWarps = 4;     // of a CTA
constexpr int kRows = 32;     // vocabulary rows of a task: four n8 tiles
constexpr int kTiles = kRows / 8;
constexpr int kKStep = 64;    // columns of a step: 128 bytes of a row
constexpr int kCtasPerSm = 4;
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

// A read that nothing will ask for again soon (W is larger than L1).
__device__ __forceinline__ uint4 load_stream(const void* p) {
    uint4 u;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "l"(p));
    return u;
}

struct FewArgs {
    const __nv_bfloat16 *X, *W;
    const long long* targets;
    int T, h, V, tasks;
    float2* parts;  // forward: {max, sum of exponentials}, [CTA][T]
    // backward
    const float *dloss, *lse;
    __nv_bfloat16 *dz, *dzt;  // [16][ldz] and [ldz][16]
    int ldz;
    float* scale;
};

// Logits of the 16 tokens against tasks of 32 vocabulary rows, CTA b taking
// tasks b, b + grid, ...  The four warps split k (64 columns each in turn, so
// that together they read 512 consecutive bytes of a row) and their sums
// meet in shared memory.  Then thread (token, 4 rows): forward, the running
// maximum and sum of exponentials; backward, the logits' gradient.
template <bool GRAD>
__global__ void __launch_bounds__(32 * kWarps, kCtasPerSm) head_few_logits_kernel(const FewArgs p) {
    pdl_launch_dependents();  // the next kernel may begin its launch
    __shared__ __align__(16) float red[2][kWarps][kTokens][kRows + 4];
    __shared__ __align__(16) __nv_bfloat16 tr[2][kRows][kTokens];
    pdl_wait();  // X comes from the kernel before this one
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int steps = (p.h + kKStep - 1) / kKStep;
    const bool lo_ok = g < p.T, hi_ok = g + 8 < p.T;
    const __nv_bfloat16* xlo = p.X + static_cast<long long>(lo_ok ? g : 0) * p.h + q * 8;
    const __nv_bfloat16* xhi = p.X + static_cast<long long>(hi_ok ? g + 8 : 0) * p.h + q * 8;
    const bool two = p.T > 8;

    // this thread's token and rows of a task behind the meeting of the sums
    const int t = threadIdx.x / (kRows / 4), vq = threadIdx.x % (kRows / 4) * 4;
    long long y = -1;
    float mx = -INFINITY, sum = 0.0f, lse2 = INFINITY, weight = 0.0f;
    if (t < p.T) y = __ldg(p.targets + t);
    if constexpr (GRAD) {
        float s = 0.0f;
        for (int i = 0; i < p.T; ++i)
            if (__ldg(p.targets + i) >= 0) s = fmaxf(s, fabsf(__ldg(p.dloss + i)));
        if (!(s > 0.0f && s < INFINITY)) s = 1.0f;
        if (blockIdx.x == 0 && threadIdx.x == 0) *p.scale = s;
        if (t < p.T && y >= 0) {
            lse2 = __ldg(p.lse + t) * kLog2e;
            weight = y < p.V ? __ldg(p.dloss + t) / s : __int_as_float(0x7FC00000);
        }
    }

    int parity = 0;
    for (int task = blockIdx.x; task < p.tasks; task += gridDim.x, parity ^= 1) {
        const int v0 = task * kRows;
        const __nv_bfloat16* w[kTiles];
#pragma unroll
        for (int i = 0; i < kTiles; ++i)  // rows behind the vocabulary read its last
            w[i] = p.W + static_cast<long long>(min(v0 + i * 8 + g, p.V - 1)) * p.h + q * 8;
        float acc[kTiles][4];
#pragma unroll
        for (int i = 0; i < kTiles; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
        uint4 wb[2][kTiles][2], xa[2][2][2];
        auto load = [&](int step, int b) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k = step * kKStep + s * 32;  // + q * 8 .. + 7
                const bool ok = k + q * 8 < p.h;
                const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int i = 0; i < kTiles; ++i) wb[b][i][s] = ok ? load_stream(w[i] + k) : z;
                xa[b][0][s] = ok && lo_ok ? __ldg(reinterpret_cast<const uint4*>(xlo + k)) : z;
                xa[b][1][s] = two && ok && hi_ok ? __ldg(reinterpret_cast<const uint4*>(xhi + k)) : z;
            }
        };
        auto multiply = [&](int b) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const uint4 a = xa[b][0][s], c = xa[b][1][s];
#pragma unroll
                for (int i = 0; i < kTiles; ++i) {
                    const uint4 u = wb[b][i][s];
                    mma16816(acc[i], a.x, c.x, a.y, c.y, u.x, u.y);
                    mma16816(acc[i], a.z, c.z, a.w, c.w, u.z, u.w);
                }
            }
        };
        if (warp < steps) load(warp, 0);
        for (int step = warp; step < steps; step += 2 * kWarps) {  // one step's loads ahead
            if (step + kWarps < steps) load(step + kWarps, 1);
            multiply(0);
            if (step + kWarps < steps) {
                if (step + 2 * kWarps < steps) load(step + 2 * kWarps, 0);
                multiply(1);
            }
        }
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
            *reinterpret_cast<float2*>(&red[parity][warp][g][i * 8 + 2 * q]) = make_float2(acc[i][0], acc[i][1]);
            *reinterpret_cast<float2*>(&red[parity][warp][g + 8][i * 8 + 2 * q]) = make_float2(acc[i][2], acc[i][3]);
        }
        __syncthreads();
        float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
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

// dX and dW from dz: a warp owns 64 columns and a range of vocabulary rows.
// Per 16 rows it loads its 16 x 64 block of W once (a lane: 8 columns of
// rows 2q, 2q + 1, 2q + 8, 2q + 9, byte-permuted into pairs along the rows),
// adds dz W to its 16 x 64 sums of dX, and multiplies dz^T by its 64 columns
// of X, which stay in registers, into that block of dW.  Column n of
// instruction j is column 8 n + j of the 64, so that a lane's eight
// instructions give it 16 consecutive columns of dW: whole lines are stored.
// dX's sums of each range go to plane[range][T][h].
__global__ void __launch_bounds__(32 * kWarps, kCtasPerSm)
    head_few_grad_kernel(const __nv_bfloat16* __restrict__ X, const __nv_bfloat16* __restrict__ W,
                         const __nv_bfloat16* __restrict__ dz, const __nv_bfloat16* __restrict__ dzt,
                         int ldz, const float* __restrict__ scale, int T, int h, int V,
                         int range_rows, __nv_bfloat16* __restrict__ dW, float* __restrict__ plane) {
    pdl_launch_dependents();  // the next kernel may begin its launch
    pdl_wait();               // dz comes from the kernel before this one
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int col0 = (blockIdx.x * kWarps + warp) * kColumns;
    if (col0 >= h) return;
    const int c = col0 + g * 8;  // columns this lane loads
    const bool c_ok = c < h;
    const int row_off[4] = {2 * q, 2 * q + 1, 2 * q + 8, 2 * q + 9};
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    // eight pairs along k from two rows' 8 values
    auto pairs = [](const uint4 a, const uint4 b, uint32_t (&o)[8]) {
        const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[2 * i] = __byte_perm(x[i], y[i], 0x5410);
            o[2 * i + 1] = __byte_perm(x[i], y[i], 0x7632);
        }
    };
    uint32_t xb[2][8];
    {
        uint4 r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r[i] = c_ok && row_off[i] < T
                       ? __ldg(reinterpret_cast<const uint4*>(X + static_cast<long long>(row_off[i]) * h + c))
                       : zero;
        pairs(r[0], r[1], xb[0]);
        pairs(r[2], r[3], xb[1]);
    }
    const float s = __ldg(scale);
    float ax[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j) ax[j][0] = ax[j][1] = ax[j][2] = ax[j][3] = 0.0f;

    const int r0 = blockIdx.y * range_rows, r1 = min(r0 + range_rows, V);
    uint4 wn[4];
    uint32_t an[4], tn[4];
    auto load = [&](int vb) {
#pragma unroll
        for (int i = 0; i < 4; ++i)  // rows behind the vocabulary read its last; dz is 0 there
            wn[i] = c_ok ? load_stream(W + static_cast<long long>(min(vb + row_off[i], V - 1)) * h + c) : zero;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            an[i] = __ldg(reinterpret_cast<const uint32_t*>(dz + static_cast<long long>(g + (i & 1) * 8) * ldz + vb +
                                                            2 * q + (i >> 1) * 8));
            tn[i] = __ldg(reinterpret_cast<const uint32_t*>(dzt + static_cast<long long>(vb + g + (i & 1) * 8) * kTokens +
                                                            2 * q + (i >> 1) * 8));
        }
    };
    if (r0 < r1) load(r0);
    for (int vb = r0; vb < r1; vb += 16) {
        uint32_t wb[2][8], a[4], t[4];
        pairs(wn[0], wn[1], wb[0]);
        pairs(wn[2], wn[3], wb[1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = an[i];
            t[i] = tn[i];
        }
        if (vb + 16 < r1) load(vb + 16);
        float o[8][4];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            mma16816(ax[j], a[0], a[1], a[2], a[3], wb[0][j], wb[1][j]);
            o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
            mma16816(o[j], t[0], t[1], t[2], t[3], xb[0][j], xb[1][j]);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {  // rows g, g + 8
            const int v = vb + g + 8 * r;
#pragma unroll
            for (int half = 0; half < 2; ++half) {  // columns 16 q .., 16 q + 8 ..
                const int n = col0 + 16 * q + 8 * half, e = 2 * r + half;
                if (v < V && n < h)
                    *reinterpret_cast<uint4*>(dW + static_cast<long long>(v) * h + n) =
                        make_uint4(pack_bf16x2(s * o[0][e], s * o[1][e]), pack_bf16x2(s * o[2][e], s * o[3][e]),
                                   pack_bf16x2(s * o[4][e], s * o[5][e]), pack_bf16x2(s * o[6][e], s * o[7][e]));
            }
        }
    }
    float* out = plane + static_cast<long long>(blockIdx.y) * T * h;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int tok = g + 8 * r;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int n = col0 + 16 * q + 8 * half, e = 2 * r + half;
            if (tok < T && n < h) {
                float4* d = reinterpret_cast<float4*>(out + static_cast<long long>(tok) * h + n);
                d[0] = make_float4(ax[0][e], ax[1][e], ax[2][e], ax[3][e]);
                d[1] = make_float4(ax[4][e], ax[5][e], ax[6][e], ax[7][e]);
            }
        }
    }
}

int ceil_div(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

}  // namespace

bool head_few(int T) { return T <= kTokens; }

int head_few_parts(int V) { return std::min(ceil_div(V, kRows), kSms * kCtasPerSm); }

int head_few_ldz(int V) { return ceil_div(V, kRows) * kRows; }

// Ranges of vocabulary rows, as many as fill the GPU with CTAs of 256 columns.
int head_few_planes(int h, int V) {
    const int col_ctas = ceil_div(h, kColumns * kWarps);
    return std::max(1, std::min(kSms * kCtasPerSm / col_ctas, ceil_div(V, 16)));
}

cudaError_t launch_head_few_lse(const __nv_bfloat16* X, const __nv_bfloat16* W, const long long* targets,
                                int T, int h, int V, float2* parts, cudaStream_t st, int* launches) {
    FewArgs a = {};
    a.X = X; a.W = W; a.targets = targets; a.T = T; a.h = h; a.V = V;
    a.tasks = ceil_div(V, kRows);
    a.parts = parts;
    ++*launches;
    return launch_dependent(head_few_logits_kernel<false>, dim3(head_few_parts(V)), dim3(32 * kWarps), 0, st, a);
}

cudaError_t launch_head_few_backward(const float* dloss, const __nv_bfloat16* X, const __nv_bfloat16* W,
                                     const long long* targets, const float* lse, int T, int h, int V,
                                     __nv_bfloat16* dz, __nv_bfloat16* dzt, float* scale, float* plane,
                                     __nv_bfloat16* dW, cudaStream_t st, int* launches) {
    FewArgs a = {};
    a.X = X; a.W = W; a.targets = targets; a.T = T; a.h = h; a.V = V;
    a.tasks = ceil_div(V, kRows);
    a.dloss = dloss; a.lse = lse; a.dz = dz; a.dzt = dzt; a.ldz = head_few_ldz(V); a.scale = scale;
    ++*launches;
    cudaError_t e = launch_dependent(head_few_logits_kernel<true>, dim3(head_few_parts(V)), dim3(32 * kWarps), 0,
                                     st, a);
    if (e != cudaSuccess) return e;
    const int planes = head_few_planes(h, V);
    const int range_rows = ceil_div(ceil_div(V, planes), 16) * 16;
    ++*launches;
    return launch_dependent(head_few_grad_kernel, dim3(ceil_div(h, kColumns * kWarps), planes), dim3(32 * kWarps), 0,
                            st, X, W, static_cast<const __nv_bfloat16*>(dz), static_cast<const __nv_bfloat16*>(dzt),
                            a.ldz, static_cast<const float*>(scale), T, h, V, range_rows, dW, plane);
}

}  // namespace tpmlp
