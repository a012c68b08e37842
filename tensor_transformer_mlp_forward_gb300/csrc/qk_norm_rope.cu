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
// f, right to 2^-64; p f modulo 2^64 is the angle's fraction of a turn, right to
// 2^-64 |p| <= 2^-33, well below fp32's last bit of an eighth of a turn.  The nearest
// quarter turn comes off as an integer, and the rest (at most an eighth of a turn)
// is rounded to fp32 once.
//
// A few operations per value: bound by HBM, and not far from the issue rate, so the
// arithmetic runs on pairs of fp32 values.  A thread holds two pieces of 8 values of a
// head, the two that the rotation mixes, so the rotation is its own business and the
// head's sums cross d / 16 lanes.  A CTA takes runs of (token, head) pairs, and computes
// the sines and cosines of a run's few tokens once, in shared memory, while its values are
// on their way.  Forward, a CTA takes one run: CTAs that come and go keep more loads in
// flight than resident ones that fetch a run ahead.  Backward, resident CTAs on queries or
// on keys carry the sums of one dgamma from run to run, the next run's values on their way
// while one is computed.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/tpmlp.h"
#include "kernels.h"

namespace tpmlp {
namespace {

// Small CTAs wait less at the barrier between a run's sines and their use: 32 and 58 us
// (forward and backward, 8192 tokens of 40 heads of 128) against 34 and 61 with 256
// threads.  At least one for each of a token's pairs (rot / 2 <= 128).
constexpr int kQkThreads = 128;

struct QkTurns {
    unsigned long long f[128];  // per pair: turns a position, times 2^64
};

// Queries or keys.
struct QkJob {
    const void *x, *dy;      // [T, heads, d], tokens ldx, lddy values apart
    void* out;               // y or dx
    const void* gamma;       // [d]
    int ldx, lddy, ldo;
    int heads, first;        // first: the matrix's first column of rstd
    int step_t, step_h;      // (tokens, heads) from one run of a CTA to its next
    int group_t, group_h;    // and from one unit of a thread to the next
};

struct QkArgs {
    QkJob job[2];            // queries, keys
    int ctas[2];             // CTAs of each
    const int* positions;    // [T]
    float* rstd;             // [T, all heads]: forward output, backward input
    float* partial;          // backward: [CTA][d] of dgamma
    int T, all_heads, d, rot;
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

// Pairs of fp32 values, one instruction for two.
__device__ __forceinline__ uint64_t two(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 apart(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint64_t widen(uint32_t w, __nv_bfloat16) {
    return two(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint64_t widen(uint32_t w, __half) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return two(f.x, f.y);
}
__device__ __forceinline__ uint32_t narrow(uint64_t v, __nv_bfloat16) {
    const float2 f = apart(v);
    return pack_bf16x2(f.x, f.y);
}
__device__ __forceinline__ uint32_t narrow(uint64_t v, __half) {
    const float2 f = apart(v);
    const __half2 h = __floats2half2_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T>
__device__ __forceinline__ void unpack8(const Raw<T>& r, uint64_t (&v)[4]) {
    if constexpr (sizeof(T) == 4) {
        const uint32_t w[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = two(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    } else {
        const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = widen(w[i], T{});
    }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const uint64_t (&v)[4]) {
    if constexpr (sizeof(T) == 4) {
        const float2 a = apart(v[0]), b = apart(v[1]), c = apart(v[2]), d = apart(v[3]);
        reinterpret_cast<float4*>(p)[0] = make_float4(a.x, a.y, b.x, b.y);
        reinterpret_cast<float4*>(p)[1] = make_float4(c.x, c.y, d.x, d.y);
    } else {
        *reinterpret_cast<uint4*>(p) =
            make_uint4(narrow(v[0], T{}), narrow(v[1], T{}), narrow(v[2], T{}), narrow(v[3], T{}));
    }
}

// cos and sin of 2 pi (p f / 2^64 mod 1), the rest behind the nearest quarter turn
// rounded to fp32 once, whatever its size.  For the 16-bit types by Taylor's series, whose
// first missing terms are below 2^-21 and 2^-25 at an eighth of a turn and fall with the
// angle, so small sines keep all of their digits: backward, 58 us where sincospi takes 60
// (8192 tokens of 40 heads of 128).
template <bool SERIES>
__device__ __forceinline__ float2 turn(int p, unsigned long long f) {
    const unsigned long long a = static_cast<unsigned long long>(static_cast<long long>(p)) * f;
    const unsigned long long quarter = (a + (1ull << 61)) >> 62;  // nearest quarter turn, modulo 4
    const long long rest = static_cast<long long>(a - (quarter << 62));  // +- 2^61
    float s, c;
    if constexpr (SERIES) {
        const float r = __ll2float_rn(rest) * (3.14159265358979f * 0x1p-63f), r2 = r * r;
        s = fmaf(r * r2, fmaf(r2, fmaf(r2, -1.0f / 5040.0f, 1.0f / 120.0f), -1.0f / 6.0f), r);
        c = fmaf(r2, fmaf(r2, fmaf(r2, fmaf(r2, 1.0f / 40320.0f, -1.0f / 720.0f), 1.0f / 24.0f), -0.5f), 1.0f);
    } else {
        sincospif(__ll2float_rn(rest) * 0x1p-63f, &s, &c);  // half turns
    }
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

// A thread's share of the sines and cosines: pair j of every per'th token of a run.
struct TurnsOf {
    int tok, j, per;
    unsigned long long f;
    __device__ __forceinline__ TurnsOf(const QkTurns& turns, int half) {
        per = half > 0 ? kQkThreads / half : 0;
        tok = half > 0 ? threadIdx.x / half : 0;
        j = half > 0 ? threadIdx.x - tok * half : 0;
        f = half > 0 ? turns.f[j] : 0ull;
        if (tok >= per) tok = 1 << 30;  // beyond every run
    }
    // cos and sin of the tokens [t0, t0 + tokens) into shared memory, [token][2][rot / 2]
    template <bool SERIES>
    __device__ __forceinline__ void fill(float* table, const int* positions, int t0, int tokens, int rot) const {
        for (int t = tok; t < tokens; t += per) {
            const float2 cs = turn<SERIES>(__ldg(positions + t0 + t), f);
            table[t * rot + j] = cs.x;
            table[t * rot + rot / 2 + j] = cs.y;
        }
    }
};

// (a, b) turned by the angle whose cos and sin are given, or (sign -1) back.
__device__ __forceinline__ void rotate(uint64_t (&a)[4], uint64_t (&b)[4], const float* table, int half, int u,
                                       float sign) {
    const ulonglong2* c = reinterpret_cast<const ulonglong2*>(table + 8 * u);
    const ulonglong2* s = reinterpret_cast<const ulonglong2*>(table + half + 8 * u);
    const uint64_t plus = two(sign, sign), minus = two(-sign, -sign);
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const ulonglong2 cc = c[i / 2], ss = s[i / 2];
        const uint64_t c2[2] = {cc.x, cc.y}, s2[2] = {ss.x, ss.y};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint64_t x = a[i + k], y = b[i + k];
            a[i + k] = fma2(y, mul2(s2[k], minus), mul2(x, c2[k]));
            b[i + k] = fma2(x, mul2(s2[k], plus), mul2(y, c2[k]));
        }
    }
}

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

__device__ __forceinline__ float sum4(const uint64_t (&v)[2]) {
    const float2 f = apart(add2(v[0], v[1]));
    return f.x + f.y;
}

// A (token, head) pair, moved without a division.
struct Pair {
    int t, h;
    __device__ __forceinline__ void move(int dt, int dh, int heads) {
        t += dt;
        h += dh;
        if (h >= heads) {
            h -= heads;
            ++t;
        }
    }
};

template <typename T>
__device__ __forceinline__ const T* row_of(const void* p, int ld, Pair at, int d) {
    return static_cast<const T*>(p) + (static_cast<long long>(at.t) * ld + at.h * d);
}

// One run: pairs of a token's queries and keys, queries first.
template <typename T, int LANES, int UNITS, int PER_SM>
__global__ void __launch_bounds__(kQkThreads, PER_SM)
    qk_forward_kernel(const __grid_constant__ QkArgs a, const __grid_constant__ QkTurns turns) {
    pdl_launch_dependents();
    pdl_wait();
    extern __shared__ __align__(16) float table[];
    constexpr int GROUPS = kQkThreads / LANES, RUN = GROUPS * UNITS;
    constexpr bool SERIES = sizeof(T) == 2;
    const int heads = a.all_heads, nh = a.job[0].heads, d = a.d;
    const int u = threadIdx.x % LANES, grp = threadIdx.x / LANES;
    const Place pl = place_of(u, d, a.rot);
    const TurnsOf mine(turns, a.rot / 2);
    const long long first = static_cast<long long>(blockIdx.x) * RUN, whole = first / heads;
    const int t0 = static_cast<int>(whole), h0 = static_cast<int>(first - whole * heads);
    Pair at;
    at.t = t0 + (h0 + grp) / heads;
    at.h = (h0 + grp) % heads;
    const int group_t = GROUPS / heads, group_h = GROUPS % heads;
    Raw<T> xa[UNITS], xb[UNITS];
    Pair from = at;
#pragma unroll
    for (int n = 0; n < UNITS; ++n) {
        xa[n] = xb[n] = zero8<T>();
        if (from.t < a.T && pl.on) {
            const T* x = from.h < nh ? row_of<T>(a.job[0].x, a.job[0].ldx, from, d)
                                     : row_of<T>(a.job[1].x, a.job[1].ldx, Pair{from.t, from.h - nh}, d);
            xa[n] = load8(x + pl.a);
            xb[n] = load8(x + pl.b);
        }
        from.move(group_t, group_h, heads);
    }
    mine.fill<SERIES>(table, a.positions, t0, min(t0 + (h0 + RUN - 1) / heads, a.T - 1) - t0 + 1, a.rot);
    __syncthreads();
#pragma unroll
    for (int n = 0; n < UNITS; ++n) {
        const bool on = at.t < a.T && pl.on, isq = at.h < nh;
        uint64_t va[4], vb[4], sum[2] = {0ull, 0ull};
        unpack8(xa[n], va);
        unpack8(xb[n], vb);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e & 1] = fma2(va[e], va[e], fma2(vb[e], vb[e], sum[e & 1]));
        const float r = rsqrtf(group_sum<LANES>(sum4(sum)) * a.inv_d + a.eps);
        if (on) {
            const T* gamma = static_cast<const T*>(isq ? a.job[0].gamma : a.job[1].gamma);
            const uint64_t rr = two(r, r);
            uint64_t wa[4], wb[4];
            unpack8(load8(gamma + pl.a), wa);
            unpack8(load8(gamma + pl.b), wb);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                va[e] = mul2(mul2(va[e], rr), wa[e]);
                vb[e] = mul2(mul2(vb[e], rr), wb[e]);
            }
            if (pl.turns) rotate(va, vb, table + (at.t - t0) * a.rot, a.rot / 2, u, 1.0f);
            T* out = const_cast<T*>(isq ? row_of<T>(a.job[0].out, a.job[0].ldo, at, d)
                                        : row_of<T>(a.job[1].out, a.job[1].ldo, Pair{at.t, at.h - nh}, d));
            store8(out + pl.a, va);
            store8(out + pl.b, vb);
            if (u == 0) a.rstd[static_cast<long long>(at.t) * heads + at.h] = r;
        }
        at.move(group_t, group_h, heads);
    }
}

// CTAs [0, ctas[0]) take the queries' runs in turn, the others the keys'.
template <typename T, int LANES, int UNITS, int PER_SM>
__global__ void __launch_bounds__(kQkThreads, PER_SM)
    qk_backward_kernel(const __grid_constant__ QkArgs a, const __grid_constant__ QkTurns turns, int table_floats) {
    pdl_launch_dependents();
    pdl_wait();
    extern __shared__ __align__(16) float tables[];
    constexpr int GROUPS = kQkThreads / LANES, RUN = GROUPS * UNITS;
    constexpr bool SERIES = sizeof(T) == 2;
    const bool keys = static_cast<int>(blockIdx.x) >= a.ctas[0];
    const QkJob& j = a.job[keys];
    const int heads = j.heads, d = a.d;
    const int u = threadIdx.x % LANES, grp = threadIdx.x / LANES;
    const Place pl = place_of(u, d, a.rot);
    const TurnsOf mine(turns, a.rot / 2);
    // gamma's two pieces, for every run
    uint64_t wa[4], wb[4];
    {
        const T* gamma = static_cast<const T*>(j.gamma);
        unpack8(pl.on ? load8(gamma + pl.a) : zero8<T>(), wa);
        unpack8(pl.on ? load8(gamma + pl.b) : zero8<T>(), wb);
    }
    uint64_t acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0ull;
    // the run's first pair, its last one's token, and this thread's first pair
    Pair at0, last, at;
    {
        const long long first = static_cast<long long>(blockIdx.x - (keys ? a.ctas[0] : 0)) * RUN;
        const long long t0 = first / heads;
        at0.t = static_cast<int>(t0);
        at0.h = static_cast<int>(first - t0 * heads);
        last.t = at0.t + (at0.h + RUN - 1) / heads;
        last.h = (at0.h + RUN - 1) % heads;
        at.t = at0.t + (at0.h + grp) / heads;
        at.h = (at0.h + grp) % heads;
    }
    Raw<T> xa[UNITS], xb[UNITS], ya[UNITS], yb[UNITS];
    float rstd[UNITS];
    auto load = [&](Pair from) {
#pragma unroll
        for (int n = 0; n < UNITS; ++n) {
            xa[n] = xb[n] = ya[n] = yb[n] = zero8<T>();
            rstd[n] = 0.0f;
            if (from.t < a.T && pl.on) {
                const T* x = row_of<T>(j.x, j.ldx, from, d);
                xa[n] = load8(x + pl.a);
                xb[n] = load8(x + pl.b);
                const T* y = row_of<T>(j.dy, j.lddy, from, d);
                ya[n] = load8(y + pl.a);
                yb[n] = load8(y + pl.b);
                rstd[n] = __ldg(a.rstd + static_cast<long long>(from.t) * a.all_heads + j.first + from.h);
            }
            from.move(j.group_t, j.group_h, heads);
        }
    };
    auto fill = [&](int k) {
        mine.fill<SERIES>(tables + (k & 1) * table_floats, a.positions, at0.t, min(last.t, a.T - 1) - at0.t + 1, a.rot);
    };
    load(at);
    fill(0);
    __syncthreads();
    for (int k = 0; at0.t < a.T; ++k) {
        const float* table = tables + (k & 1) * table_floats;
        const int t0 = at0.t;
        uint64_t va[UNITS][4], vb[UNITS][4], ga[UNITS][4], gb[UNITS][4];
        float r[UNITS];
#pragma unroll
        for (int n = 0; n < UNITS; ++n) {
            unpack8(xa[n], va[n]);
            unpack8(xb[n], vb[n]);
            unpack8(ya[n], ga[n]);
            unpack8(yb[n], gb[n]);
            r[n] = rstd[n];
        }
        // the next run's values, and its tokens' turns, while this one is computed
        Pair here = at;
        at0.move(j.step_t, j.step_h, heads);
        last.move(j.step_t, j.step_h, heads);
        at.move(j.step_t, j.step_h, heads);
        load(at);
        fill(k + 1);
#pragma unroll
        for (int n = 0; n < UNITS; ++n) {
            const bool on = here.t < a.T && pl.on;
            const float* turned = table + (here.t - t0) * a.rot;
            uint64_t sum[2] = {0ull, 0ull};
            if (on && pl.turns) rotate(ga[n], gb[n], turned, a.rot / 2, u, -1.0f);
            const uint64_t rr = two(r[n], r[n]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // (a pair beyond the end is all zeros)
                va[n][e] = mul2(va[n][e], rr);
                vb[n][e] = mul2(vb[n][e], rr);
                const uint64_t pa = mul2(ga[n][e], va[n][e]), pb = mul2(gb[n][e], vb[n][e]);
                acc[e] = add2(acc[e], pa);
                acc[4 + e] = add2(acc[4 + e], pb);
                sum[e & 1] = fma2(pa, wa[e], fma2(pb, wb[e], sum[e & 1]));
            }
            const float m = -group_sum<LANES>(sum4(sum)) * a.inv_d;
            const uint64_t mm = two(m, m);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                va[n][e] = mul2(rr, fma2(va[n][e], mm, mul2(ga[n][e], wa[e])));
                vb[n][e] = mul2(rr, fma2(vb[n][e], mm, mul2(gb[n][e], wb[e])));
            }
            if (on) {
                T* out = const_cast<T*>(row_of<T>(j.out, j.ldo, here, d));
                store8(out + pl.a, va[n]);
                store8(out + pl.b, vb[n]);
            }
            here.move(j.group_t, j.group_h, heads);
        }
        __syncthreads();  // this run's sines have been read, the next one's are there
    }
    {
        // lanes of the same columns, then the warps, in a fixed order
        float* rows = tables;  // [warp][d]
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 f = apart(acc[e]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v = h ? f.y : f.x;
#pragma unroll
                for (int o = 16; o >= LANES; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
                if (threadIdx.x % 32 < LANES && pl.on)
                    rows[threadIdx.x / 32 * d + (e < 4 ? pl.a + 2 * e : pl.b + 2 * e - 8) + h] = v;
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < d; c += kQkThreads) {
            float v = 0.0f;
            for (int w = 0; w < kQkThreads / 32; ++w) v += rows[w * d + c];
            a.partial[static_cast<long long>(blockIdx.x) * d + c] = v;
        }
    }
}

// dgamma = the CTAs' parts added up: 32 columns a CTA, 32 threads a column.  Columns
// [0, d) are the queries', whose parts come first, [d, 2 d) the keys'.
__global__ void __launch_bounds__(1024)
    qk_dgamma_kernel(const float* partial, int parts_q, int parts, int d, float* dgamma_q, float* dgamma_k) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ float s[32][33];
    const int x = threadIdx.x % 32, y = threadIdx.x / 32, c = blockIdx.x * 32 + x;
    float v = 0.0f;
    if (c < 2 * d) {
        const float* column = partial + (c < d ? c : c - d);
        const int end = c < d ? parts_q : parts;
        // eight parts on their way at a time
        for (int i = y + (c < d ? 0 : parts_q); i < end; i += 8 * 32) {
            float w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = i + 32 * k < end ? column[static_cast<long long>(i + 32 * k) * d] : 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) v += w[k];
        }
    }
    s[y][x] = v;
    __syncthreads();
    v = s[x][y];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    const int col = blockIdx.x * 32 + y;
    if (x == 0 && col < 2 * d) (col < d ? dgamma_q[col] : dgamma_k[col - d]) = v;
}

// Pairs a thread holds, and CTAs an SM: what the registers allow with enough loads in
// flight (backward: two pairs 64 us, five CTAs, which spill, 62).
template <typename T>
constexpr int kUnitsForward = sizeof(T) == 4 ? 2 : 4;
constexpr int kUnitsBackward = 1, kPerSmForward = 8, kPerSmBackward = 4;

int lanes_of(int d) { return d <= 32 ? 2 : d <= 64 ? 4 : d <= 128 ? 8 : 16; }

// CTAs for the queries and the keys: in proportion to their runs, one run each at least.
void deal_ctas(int T, int nh, int nkv, long long run, int most, int (&ctas)[2]) {
    const long long q = (1LL * T * nh + run - 1) / run, k = (1LL * T * nkv + run - 1) / run;
    if (q + k <= most) {
        ctas[0] = static_cast<int>(q);
        ctas[1] = static_cast<int>(k);
        return;
    }
    long long c = (q * most + (q + k) / 2) / (q + k);
    c = c < 1 ? 1 : c > most - 1 ? most - 1 : c;
    ctas[0] = static_cast<int>(c < q ? c : q);
    ctas[1] = static_cast<int>(most - c < k ? most - c : k);
}

// Numbers of some 106 bits as sums of two doubles: products and sums whose rounding is
// caught exactly (Dekker 1971, with a fused multiply-add).
struct Wide {
    double hi, lo;
};
Wide fast_sum(double a, double b) {  // |a| >= |b|
    const double s = a + b;
    return {s, b - (s - a)};
}
Wide times(Wide a, Wide b) {
    const double p = a.hi * b.hi;
    return fast_sum(p, std::fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}

// |x| modulo 1, times 2^64
unsigned long long fraction(double x) {
    return static_cast<unsigned long long>(std::nearbyint((x - std::floor(x)) * 0x1p64));
}

// theta^(-2 i / rot) / 2 pi modulo 1, as powers of r = theta^(-1 / n), n = rot / 2, in 106
// bits: from pow's r by one Newton step towards theta r^n = 1.
QkTurns make_turns(double theta, int rot) {
    QkTurns t{};
    const int n = rot / 2;
    if (n == 0) return t;
    const double r0 = std::pow(theta, -1.0 / n);
    Wide all{theta, 0.0}, square{r0, 0.0};
    for (int m = n; m > 0; m >>= 1) {
        if (m & 1) all = times(all, square);
        if (m > 1) square = times(square, square);
    }
    const Wide r = fast_sum(r0, -r0 * (((all.hi - 1.0) + all.lo) / n));
    // 16 + 8 powers, then products of two
    Wide low[9], high{0.15915494309189535, -9.839338337591243e-18};  // 1 / (2 pi)
    low[0] = {1.0, 0.0};
    for (int i = 1; i < 9; ++i) low[i] = times(low[i - 1], r);
    for (int i = 0; i < n; ++i) {
        const Wide f = times(high, low[i % 8]);
        t.f[i] = fraction(f.hi) + (f.lo < 0.0 ? 0ull - fraction(-f.lo) : fraction(f.lo));
        if (i % 8 == 7) high = times(high, low[8]);
    }
    return t;
}

QkJob make_job(const void* x, const void* dy, void* out, const void* gamma, long long ldx, long long lddy, long long ldo,
               int heads, int first, int ctas, int run, int groups) {
    QkJob j{x, dy, out, gamma, static_cast<int>(ldx), static_cast<int>(lddy), static_cast<int>(ldo), heads, first};
    const long long step = 1LL * ctas * run;
    j.step_t = static_cast<int>(step / heads);
    j.step_h = static_cast<int>(step % heads);
    j.group_t = groups / heads;
    j.group_h = groups % heads;
    return j;
}

QkArgs make_args(const QkNormRope& p) {
    QkArgs a{};
    const int groups = kQkThreads / lanes_of(p.d), run = kUnitsBackward * groups;
    deal_ctas(p.T, p.nh, p.nkv, run, kQkSms * kPerSmBackward, a.ctas);
    a.job[0] = make_job(p.q, p.dy_q, p.out_q, p.gamma_q, p.ldq, p.ldyq, p.ldoq, p.nh, 0, a.ctas[0], run, groups);
    a.job[1] = make_job(p.k, p.dy_k, p.out_k, p.gamma_k, p.ldk, p.ldyk, p.ldok, p.nkv, p.nh, a.ctas[1], run, groups);
    a.positions = p.positions;
    a.rstd = p.rstd;
    a.partial = p.partial;
    a.T = p.T;
    a.all_heads = p.nh + p.nkv;
    a.d = p.d;
    a.rot = p.rot;
    a.eps = p.eps;
    a.inv_d = 1.0f / static_cast<float>(p.d);
    return a;
}

// Shared memory of `tables` tables of sines and cosines: as many tokens as a run can touch
// (18 KB at most).
size_t table_bytes(int run, int heads, int rot, int tables) {
    return sizeof(float) * static_cast<size_t>((run + heads - 2) / heads + 1) * rot * tables;
}

template <typename T, int LANES>
cudaError_t forward_as(const QkArgs& a, const QkTurns& turns, cudaStream_t st) {
    constexpr int run = kUnitsForward<T> * kQkThreads / LANES;
    const long long pairs = 1LL * a.T * a.all_heads;
    return launch_dependent(qk_forward_kernel<T, LANES, kUnitsForward<T>, kPerSmForward>,
                            dim3(static_cast<unsigned>((pairs + run - 1) / run)), dim3(kQkThreads),
                            table_bytes(run, a.all_heads, a.rot, 1), st, a, turns);
}

template <typename T, int LANES>
cudaError_t backward_as(const QkArgs& a, const QkTurns& turns, cudaStream_t st) {
    constexpr int run = kUnitsBackward * kQkThreads / LANES;
    const int heads = a.job[0].heads < a.job[1].heads ? a.job[0].heads : a.job[1].heads;
    const size_t tables = table_bytes(run, heads, a.rot, 2), rows = sizeof(float) * (kQkThreads / 32) * a.d;
    return launch_dependent(qk_backward_kernel<T, LANES, kUnitsBackward, kPerSmBackward>,
                            dim3(static_cast<unsigned>(a.ctas[0] + a.ctas[1])), dim3(kQkThreads),
                            tables > rows ? tables : rows, st, a, turns, static_cast<int>(tables / (2 * sizeof(float))));
}

template <typename T>
cudaError_t by_lanes(const QkArgs& a, const QkTurns& t, bool back, cudaStream_t st) {
    switch (lanes_of(a.d)) {
        case 2: return back ? backward_as<T, 2>(a, t, st) : forward_as<T, 2>(a, t, st);
        case 4: return back ? backward_as<T, 4>(a, t, st) : forward_as<T, 4>(a, t, st);
        case 8: return back ? backward_as<T, 8>(a, t, st) : forward_as<T, 8>(a, t, st);
        default: return back ? backward_as<T, 16>(a, t, st) : forward_as<T, 16>(a, t, st);
    }
}

cudaError_t launch(const QkNormRope& p, const QkArgs& a, bool back, cudaStream_t st) {
    const QkTurns t = make_turns(p.theta, p.rot);
    if (p.dtype == TPMLP_BF16) return by_lanes<__nv_bfloat16>(a, t, back, st);
    if (p.dtype == TPMLP_FP16) return by_lanes<__half>(a, t, back, st);
    return by_lanes<float>(a, t, back, st);
}

}  // namespace

int qk_norm_parts(int T, int nh, int nkv, int d) {
    int ctas[2];
    deal_ctas(T, nh, nkv, kUnitsBackward * kQkThreads / lanes_of(d), kQkSms * kPerSmBackward, ctas);
    return ctas[0] + ctas[1];
}

cudaError_t launch_qk_norm_rope_forward(const QkNormRope& p, cudaStream_t st, int* launches) {
    const cudaError_t e = launch(p, make_args(p), false, st);
    if (e == cudaSuccess) ++*launches;
    return e;
}

cudaError_t launch_qk_norm_rope_backward(const QkNormRope& p, float* dgamma_q, float* dgamma_k, cudaStream_t st,
                                         int* launches) {
    const QkArgs a = make_args(p);
    cudaError_t e = launch(p, a, true, st);
    if (e != cudaSuccess) return e;
    ++*launches;
    e = launch_dependent(qk_dgamma_kernel, dim3((2 * p.d + 31) / 32), dim3(1024), 0, st,
                         static_cast<const float*>(p.partial), a.ctas[0], a.ctas[0] + a.ctas[1], p.d, dgamma_q, dgamma_k);
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace tpmlp
