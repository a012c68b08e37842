// qk_norm_rope.cu -- norms of queries and keys for each head with the rotary
// position rotation in the same pass, forward and backward, in bf16, fp16 and fp32.
//
// Per token t and head, x the head's d values, p = positions[t]:
//   rstd = 1 / sqrt(mean(x^2) + eps) ; u = x rstd gamma
//   y_i          = u_i cos(a_i) - u_{i + rot/2} sin(a_i)
//   y_{i + rot/2} = u_{i + rot/2} cos(a_i) + u_i sin(a_i)     i < rot / 2
//   y_j = u_j                                                 j >= rot
//   a_i = p theta^(-2 i / rot)
// and, R(-p) turning back, its backward pass:
//   g = R(-p) dy ; xhat = x rstd ; dgamma = sum over tokens and heads of g xhat
//   dx = rstd (g gamma - xhat mean(g gamma xhat))
//
// Angles: theta^(-2i/rot) / 2 pi turns a position as a 64-bit fixed-point fraction
// f; p f modulo 2^64 is the angle's fraction of a turn, exact but for f's rounding
// (2^-53 relative), so far positions lose nothing to the size of p.  The nearest
// quarter turn comes off as an integer, and the rest (at most an eighth of a turn)
// is rounded to fp32 once.
//
// A few operations per value: bound by HBM.  A thread holds two pieces of 8 values
// of a head, the two that the rotation mixes, so the rotation is its own business
// and the head's sums cross d / 16 lanes.  A CTA takes a run of (token, head) pairs
// and computes the sines and cosines of its few tokens once, in shared memory, while
// its loads are on their way; every thread has UNITS heads in flight.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/tpmlp.h"
#include "kernels.h"

namespace tpmlp {
namespace {

constexpr int kQkThreads = 256;

struct QkTurns {
    unsigned long long f[128];  // per pair: turns a position, times 2^64
};

struct QkArgs {
    const void *q, *k;       // [T, nh, d], [T, nkv, d], tokens ldq, ldk values apart
    const void *dy_q, *dy_k;
    void *out_q, *out_k;     // y or dx
    const void *gamma_q, *gamma_k;  // [d]
    const int* positions;    // [T]
    float* rstd;             // [T, nh + nkv]: forward output, backward input
    float* partial;          // backward: [CTA][2][d] of dgamma_q, dgamma_k
    long long ldq, ldk, ldyq, ldyk, ldoq, ldok;
    long long total;         // T (nh + nkv)
    int T, nh, heads, d, rot;
    float eps, inv_d;
};

// Eight values as fp32 pairs of a 16-byte piece (two for fp32).
template <typename T>
struct Raw {
    uint4 w[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Raw<T> load8(const T* p) {
    Raw<T> r;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) r.w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
    return r;
}

template <typename T>
__device__ __forceinline__ Raw<T> zero8() {
    Raw<T> r;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) r.w[i] = make_uint4(0u, 0u, 0u, 0u);
    return r;
}

__device__ __forceinline__ float2 widen(uint32_t w, __nv_bfloat16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 widen(uint32_t w, __half) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t narrow(float a, float b, __nv_bfloat16) { return pack_bf16x2(a, b); }
__device__ __forceinline__ uint32_t narrow(float a, float b, __half) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T>
__device__ __forceinline__ void unpack8(const Raw<T>& r, float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        const uint32_t w[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    } else {
        const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = widen(w[i], T{});
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(narrow(v[0], v[1], T{}), narrow(v[2], v[3], T{}),
                                                  narrow(v[4], v[5], T{}), narrow(v[6], v[7], T{}));
    }
}

// cos and sin of 2 pi (p f / 2^64 mod 1).
__device__ __forceinline__ float2 turn(int p, unsigned long long f) {
    const unsigned long long a = static_cast<unsigned long long>(static_cast<long long>(p)) * f;
    const unsigned long long quarter = (a + (1ull << 61)) >> 62;  // nearest quarter turn, modulo 4
    const long long rest = static_cast<long long>(a - (quarter << 62));  // +- 2^61
    // in half turns, for cospi and sinpi
    const float x = static_cast<float>(static_cast<int>(rest >> 31)) * 4.656612873077393e-10f * 0.5f;
    float s, c;
    sincospif(x, &s, &c);
    const bool swap = quarter & 1ull;
    const float cc = swap ? s : c, ss = swap ? c : s;
    const unsigned q = static_cast<unsigned>(quarter) & 3u;
    return make_float2(q == 1u || q == 2u ? -cc : cc, q >= 2u ? -ss : ss);
}

// Values of a head's two pieces held by lane `u` of its group.
struct Place {
    int a, b;    // columns of the pieces
    bool on;     // this lane has values
    bool turns;  // and rotates them
};
__device__ __forceinline__ Place place_of(int u, int d, int rot) {
    Place p;
    p.on = 16 * u < d;
    p.turns = 16 * u < rot;
    p.a = p.turns ? 8 * u : 16 * u;
    p.b = p.turns ? 8 * u + rot / 2 : 16 * u + 8;
    return p;
}

// cos and sin of the tokens [t0, t0 + tokens) into shared memory, [token][2][rot / 2].
__device__ __forceinline__ void fill_turns(float* table, const QkArgs& a, const QkTurns& turns, long long t0,
                                           int tokens) {
    const int half = a.rot / 2;
    for (int i = threadIdx.x; i < tokens * half; i += kQkThreads) {
        const int t = i / half, j = i - t * half;
        const float2 cs = turn(__ldg(a.positions + t0 + t), turns.f[j]);
        table[(2 * t) * half + j] = cs.x;
        table[(2 * t + 1) * half + j] = cs.y;
    }
}

__device__ __forceinline__ void load_f8(const float* p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// (a, b) turned by the angle whose cos and sin are given; sign -1 turns back.
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const float* table, int half, int u, float sign) {
    float c[8], s[8];
    load_f8(table + 8 * u, c);
    load_f8(table + half + 8 * u, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float si = sign * s[i], x = a[i], y = b[i];
        a[i] = x * c[i] - y * si;
        b[i] = y * c[i] + x * si;
    }
}

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// A run of UNITS x kQkThreads / LANES (token, head) pairs.
template <typename T, int LANES, int UNITS>
__global__ void __launch_bounds__(kQkThreads)
    qk_forward_kernel(const __grid_constant__ QkArgs a, const __grid_constant__ QkTurns turns) {
    pdl_launch_dependents();
    pdl_wait();
    extern __shared__ float table[];
    constexpr int GROUPS = kQkThreads / LANES;
    const long long first = static_cast<long long>(blockIdx.x) * (GROUPS * UNITS);
    const int count = static_cast<int>(a.total - first < GROUPS * UNITS ? a.total - first : GROUPS * UNITS);
    const long long t0 = first / a.heads;
    const int h0 = static_cast<int>(first - t0 * a.heads);
    const int u = threadIdx.x % LANES, grp = threadIdx.x / LANES;
    const Place pl = place_of(u, a.d, a.rot);
    Raw<T> xa[UNITS], xb[UNITS];
    int tok[UNITS], head[UNITS];
#pragma unroll
    for (int n = 0; n < UNITS; ++n) {
        const int i = n * GROUPS + grp;
        tok[n] = (h0 + i) / a.heads;
        head[n] = h0 + i - tok[n] * a.heads;
        xa[n] = zero8<T>();
        xb[n] = zero8<T>();
        if (i < count && pl.on) {
            const long long t = t0 + tok[n];
            const T* x = head[n] < a.nh ? static_cast<const T*>(a.q) + t * a.ldq + head[n] * a.d
                                        : static_cast<const T*>(a.k) + t * a.ldk + (head[n] - a.nh) * a.d;
            xa[n] = load8(x + pl.a);
            xb[n] = load8(x + pl.b);
        }
    }
    fill_turns(table, a, turns, t0, (h0 + count - 1) / a.heads + 1);
    __syncthreads();
#pragma unroll
    for (int n = 0; n < UNITS; ++n) {
        const int i = n * GROUPS + grp;
        float va[8], vb[8];
        unpack8(xa[n], va);
        unpack8(xb[n], vb);
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(va[e], va[e], fmaf(vb[e], vb[e], sum));
        const float r = __frsqrt_rn(group_sum<LANES>(sum) * a.inv_d + a.eps);
        if (i >= count || !pl.on) continue;
        const bool isq = head[n] < a.nh;
        const T* gamma = static_cast<const T*>(isq ? a.gamma_q : a.gamma_k);
        float ga[8], gb[8];
        unpack8(load8(gamma + pl.a), ga);
        unpack8(load8(gamma + pl.b), gb);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            va[e] = va[e] * r * ga[e];
            vb[e] = vb[e] * r * gb[e];
        }
        if (pl.turns) rotate(va, vb, table + tok[n] * a.rot, a.rot / 2, u, 1.0f);
        const long long t = t0 + tok[n];
        T* y = isq ? static_cast<T*>(a.out_q) + t * a.ldoq + head[n] * a.d
                   : static_cast<T*>(a.out_k) + t * a.ldok + (head[n] - a.nh) * a.d;
        store8(y + pl.a, va);
        store8(y + pl.b, vb);
        if (u == 0) a.rstd[t * a.heads + head[n]] = r;
    }
}

// Runs of pairs, CTA by CTA in a fixed order: each thread keeps its 16 columns' sums
// of dgamma_q and dgamma_k, which the CTA adds up at the end.
template <typename T, int LANES, int UNITS>
__global__ void __launch_bounds__(kQkThreads)
    qk_backward_kernel(const __grid_constant__ QkArgs a, const __grid_constant__ QkTurns turns) {
    pdl_launch_dependents();
    pdl_wait();
    extern __shared__ float table[];
    constexpr int GROUPS = kQkThreads / LANES, RUN = GROUPS * UNITS, WARPS = kQkThreads / 32;
    const int u = threadIdx.x % LANES, grp = threadIdx.x / LANES;
    const Place pl = place_of(u, a.d, a.rot);
    float acc[2][16];
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[0][e] = acc[1][e] = 0.0f;
    for (long long first = static_cast<long long>(blockIdx.x) * RUN; first < a.total;
         first += static_cast<long long>(gridDim.x) * RUN) {
        const int count = static_cast<int>(a.total - first < RUN ? a.total - first : RUN);
        const long long t0 = first / a.heads;
        const int h0 = static_cast<int>(first - t0 * a.heads);
        Raw<T> xa[UNITS], xb[UNITS], ya[UNITS], yb[UNITS];
        int tok[UNITS], head[UNITS];
        float rstd[UNITS];
#pragma unroll
        for (int n = 0; n < UNITS; ++n) {
            const int i = n * GROUPS + grp;
            tok[n] = (h0 + i) / a.heads;
            head[n] = h0 + i - tok[n] * a.heads;
            xa[n] = xb[n] = ya[n] = yb[n] = zero8<T>();
            rstd[n] = 0.0f;
            if (i < count && pl.on) {
                const long long t = t0 + tok[n];
                const bool isq = head[n] < a.nh;
                const int col = (isq ? head[n] : head[n] - a.nh) * a.d;
                const T* x = (isq ? static_cast<const T*>(a.q) + t * a.ldq : static_cast<const T*>(a.k) + t * a.ldk) + col;
                const T* y =
                    (isq ? static_cast<const T*>(a.dy_q) + t * a.ldyq : static_cast<const T*>(a.dy_k) + t * a.ldyk) + col;
                xa[n] = load8(x + pl.a);
                xb[n] = load8(x + pl.b);
                ya[n] = load8(y + pl.a);
                yb[n] = load8(y + pl.b);
                rstd[n] = __ldg(a.rstd + t * a.heads + head[n]);
            }
        }
        __syncthreads();  // the last run's sines have been read
        fill_turns(table, a, turns, t0, (h0 + count - 1) / a.heads + 1);
        __syncthreads();
#pragma unroll
        for (int n = 0; n < UNITS; ++n) {
            const int i = n * GROUPS + grp;
            const bool on = i < count && pl.on, isq = head[n] < a.nh;
            float va[8], vb[8], ga[8], gb[8];
            unpack8(xa[n], va);
            unpack8(xb[n], vb);
            unpack8(ya[n], ga);
            unpack8(yb[n], gb);
            if (on && pl.turns) rotate(ga, gb, table + tok[n] * a.rot, a.rot / 2, u, -1.0f);
            float wa[8], wb[8];
            float sum = 0.0f;
            if (on) {
                const T* gamma = static_cast<const T*>(isq ? a.gamma_q : a.gamma_k);
                unpack8(load8(gamma + pl.a), wa);
                unpack8(load8(gamma + pl.b), wb);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    va[e] *= rstd[n];
                    vb[e] *= rstd[n];
                    const float pa = ga[e] * va[e], pb = gb[e] * vb[e];
                    if (isq) {
                        acc[0][e] += pa;
                        acc[0][8 + e] += pb;
                    } else {
                        acc[1][e] += pa;
                        acc[1][8 + e] += pb;
                    }
                    sum = fmaf(pa, wa[e], fmaf(pb, wb[e], sum));
                }
            }
            const float m = group_sum<LANES>(sum) * a.inv_d;
            if (!on) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                va[e] = rstd[n] * (ga[e] * wa[e] - va[e] * m);
                vb[e] = rstd[n] * (gb[e] * wb[e] - vb[e] * m);
            }
            const long long t = t0 + tok[n];
            T* dx = isq ? static_cast<T*>(a.out_q) + t * a.ldoq + head[n] * a.d
                        : static_cast<T*>(a.out_k) + t * a.ldok + (head[n] - a.nh) * a.d;
            store8(dx + pl.a, va);
            store8(dx + pl.b, vb);
        }
    }
    // lanes of the same columns, then the warps, in a fixed order
    __syncthreads();
    float* rows = table;  // [warp][2][d]
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            float v = acc[s][e];
#pragma unroll
            for (int o = 16; o >= LANES; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
            if (threadIdx.x % 32 < LANES && pl.on)
                rows[((threadIdx.x / 32) * 2 + s) * a.d + (e < 8 ? pl.a + e : pl.b + e - 8)] = v;
        }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.d; c += kQkThreads) {
        float v = 0.0f;
        for (int w = 0; w < WARPS; ++w) v += rows[w * 2 * a.d + c];
        a.partial[static_cast<long long>(blockIdx.x) * 2 * a.d + c] = v;
    }
}

// dgamma = the CTAs' parts added up: 32 columns a CTA, 32 threads a column.
__global__ void __launch_bounds__(1024) qk_dgamma_kernel(const float* partial, int parts, int d, float* dgamma_q,
                                                         float* dgamma_k) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ float s[32][33];
    const int x = threadIdx.x % 32, y = threadIdx.x / 32, c = blockIdx.x * 32 + x;
    float v = 0.0f;
    if (c < 2 * d)
        for (int i = y; i < parts; i += 32) v += partial[static_cast<long long>(i) * 2 * d + c];
    s[y][x] = v;
    __syncthreads();
    v = s[x][y];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    const int col = blockIdx.x * 32 + y;
    if (x == 0 && col < 2 * d) (col < d ? dgamma_q[col] : dgamma_k[col - d]) = v;
}

constexpr int kUnitsForward = 4, kUnitsBackward = 2;

int lanes_of(int d) { return d <= 32 ? 2 : d <= 64 ? 4 : d <= 128 ? 8 : 16; }

// Tokens that a run of pairs can touch.
int most_tokens(int run, int heads) { return (run + heads - 2) / heads + 1; }

QkArgs make_args(const QkNormRope& p) {
    QkArgs a{};
    a.q = p.q; a.k = p.k;
    a.dy_q = p.dy_q; a.dy_k = p.dy_k;
    a.out_q = p.out_q; a.out_k = p.out_k;
    a.gamma_q = p.gamma_q; a.gamma_k = p.gamma_k;
    a.positions = p.positions;
    a.rstd = p.rstd;
    a.partial = p.partial;
    a.ldq = p.ldq; a.ldk = p.ldk; a.ldyq = p.ldyq; a.ldyk = p.ldyk; a.ldoq = p.ldoq; a.ldok = p.ldok;
    a.heads = p.nh + p.nkv;
    a.total = static_cast<long long>(p.T) * a.heads;
    a.T = p.T; a.nh = p.nh; a.d = p.d; a.rot = p.rot;
    a.eps = p.eps;
    a.inv_d = 1.0f / static_cast<float>(p.d);
    return a;
}

QkTurns make_turns(double theta, int rot) {
    QkTurns t{};
    for (int i = 0; i < rot / 2; ++i) {
        double f = std::pow(theta, -2.0 * i / rot) * 0.15915494309189535;  // 1 / (2 pi)
        f -= std::floor(f);
        t.f[i] = static_cast<unsigned long long>(f * 18446744073709551616.0);  // f < 1
    }
    return t;
}

template <typename T, int LANES>
cudaError_t forward(const QkArgs& a, const QkTurns& turns, cudaStream_t st) {
    constexpr int run = kUnitsForward * kQkThreads / LANES;
    const size_t smem = sizeof(float) * static_cast<size_t>(most_tokens(run, a.heads)) * a.rot;
    return launch_dependent(qk_forward_kernel<T, LANES, kUnitsForward>,
                            dim3(static_cast<unsigned>((a.total + run - 1) / run)), dim3(kQkThreads), smem, st, a, turns);
}

template <typename T, int LANES>
cudaError_t backward(const QkArgs& a, const QkTurns& turns, int parts, cudaStream_t st) {
    constexpr int run = kUnitsBackward * kQkThreads / LANES;
    const size_t table = static_cast<size_t>(most_tokens(run, a.heads)) * a.rot;
    const size_t rows = static_cast<size_t>(kQkThreads / 32) * 2 * a.d;
    return launch_dependent(qk_backward_kernel<T, LANES, kUnitsBackward>, dim3(static_cast<unsigned>(parts)),
                            dim3(kQkThreads), sizeof(float) * (table > rows ? table : rows), st, a, turns);
}

template <typename T>
cudaError_t by_lanes(const QkArgs& a, const QkTurns& t, int parts, cudaStream_t st) {
    switch (lanes_of(a.d)) {
        case 2: return parts ? backward<T, 2>(a, t, parts, st) : forward<T, 2>(a, t, st);
        case 4: return parts ? backward<T, 4>(a, t, parts, st) : forward<T, 4>(a, t, st);
        case 8: return parts ? backward<T, 8>(a, t, parts, st) : forward<T, 8>(a, t, st);
        default: return parts ? backward<T, 16>(a, t, parts, st) : forward<T, 16>(a, t, st);
    }
}

cudaError_t launch(const QkNormRope& p, int parts, cudaStream_t st) {
    const QkArgs a = make_args(p);
    const QkTurns t = make_turns(p.theta, p.rot);
    if (p.dtype == TPMLP_BF16) return by_lanes<__nv_bfloat16>(a, t, parts, st);
    if (p.dtype == TPMLP_FP16) return by_lanes<__half>(a, t, parts, st);
    return by_lanes<float>(a, t, parts, st);
}

}  // namespace

int qk_norm_parts(int T, int heads, int d) {
    const long long run = kUnitsBackward * kQkThreads / lanes_of(d);
    const long long runs = (static_cast<long long>(T) * heads + run - 1) / run;
    return static_cast<int>(runs < kQkMaxParts ? runs : kQkMaxParts);
}

cudaError_t launch_qk_norm_rope_forward(const QkNormRope& p, cudaStream_t st, int* launches) {
    const cudaError_t e = launch(p, 0, st);
    if (e == cudaSuccess) ++*launches;
    return e;
}

cudaError_t launch_qk_norm_rope_backward(const QkNormRope& p, float* dgamma_q, float* dgamma_k, cudaStream_t st,
                                         int* launches) {
    const int parts = qk_norm_parts(p.T, p.nh + p.nkv, p.d);
    cudaError_t e = launch(p, parts, st);
    if (e != cudaSuccess) return e;
    ++*launches;
    e = launch_dependent(qk_dgamma_kernel, dim3((2 * p.d + 31) / 32), dim3(1024), 0, st, p.partial, parts, p.d, dgamma_q,
                         dgamma_k);
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace tpmlp
