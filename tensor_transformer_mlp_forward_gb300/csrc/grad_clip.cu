// grad_clip.cu -- the global norm of many gradient tensors, and clipping.
//
//   norm = sqrt(sum over all tensors and values of g^2)
//   out  = g min(1, max_norm / (norm + 1e-6))
//
// Tensors are bf16, fp16 or fp32, each of any size and of any alignment.  Bound by
// HBM: the gradients are read for the norm, read again and written.  The tensors are
// cut into pieces of kPieceBytes, dealt out to a fixed grid, each CTA leaving one
// partial sum, so that the order of the additions depends on the sizes alone.  The
// table of tensors travels in the kernels' parameters: nothing is copied to the
// device, and a captured call holds its own table.
//
// A square above 2^63 overflows fp32, one below 2^-75 is lost, although the norm need
// not be: beside the sum of the squares run those of the values times 2^-64 and times
// 2^100, of which a CTA takes the one that its sum calls for.  (A batch whose squares
// stay in range adds its own sum times 2^-128 and 2^200 to them, so only a batch outside
// is gone through again.)  The CTAs' sums are added in 64 bits.
//
// The clipping pass walks the pieces backwards: the norm's pass has left the last
// ones in L2.
//
// 550 M values (1.1 GB): 184 us reading (6.1 TB/s), 341 us reading and writing (6.4 TB/s).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "../../include/tpmlp.h"
#include "kernels.h"

namespace tpmlp {
namespace {

constexpr int kClipThreads = 256;
constexpr int kPieceBytes = 32768;  // eight 16-byte words a thread
constexpr int kWords = kPieceBytes / 16 / kClipThreads;
constexpr float kDown = 5.421010862427522e-20f;   // 2^-64
constexpr float kUp = 1.2676506002282294e30f;      // 2^100
constexpr float kDownSquared = 2.938735877055719e-39f;  // 2^-128
constexpr float kLow = 7.888609052210118e-31f;     // 2^-100: a batch's sum below it goes through again
constexpr float kLowSum = 8.271806125530277e-25f;  // 2^-80: a CTA's

template <int MOST>
struct Table {
    const void* in[MOST];
    void* out[MOST];
    long long size[MOST];      // values
    unsigned first[MOST + 1];  // pieces before the tensor
    unsigned char dtype[MOST];
    int count;
};

template <int MOST>
__device__ __forceinline__ int find_tensor(const Table<MOST>& t, unsigned piece) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= piece)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ float wide(float x) { return x; }
__device__ __forceinline__ float wide(__half x) { return __half2float(x); }
__device__ __forceinline__ float wide(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__half* p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ float2 word_pair(uint32_t w, __nv_bfloat16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 word_pair(uint32_t w, __half) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

__device__ __forceinline__ uint64_t pair_of_word(uint32_t w, __nv_bfloat16) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(w << 16), "r"(w & 0xFFFF0000u));
    return r;
}
__device__ __forceinline__ uint64_t pair_of_word(uint32_t w, __half) {
    const float2 f = word_pair(w, __half{});
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(f.x), "f"(f.y));
    return r;
}

enum Scale { kAsIs, kScaleDown, kScaleUp };

struct Sums {
    float plain, down, up;
    // a batch's sum of squares, and it or what `squares` gives for the scaled values
    template <typename F>
    __device__ __forceinline__ void add(F&& squares) {
        const float batch = squares(std::integral_constant<Scale, kAsIs>{});
        plain += batch;
        down += batch < INFINITY ? batch * kDownSquared : squares(std::integral_constant<Scale, kScaleDown>{});
        up += batch < kLow ? squares(std::integral_constant<Scale, kScaleUp>{}) : batch * kUp * kUp;
    }
};

// The sum of the squares of a 16-byte word's (scaled) values in pairs.
template <typename T, Scale SCALE>
__device__ __forceinline__ void add_squares(uint64_t (&acc)[2], const uint4& w) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
    uint64_t factor;
    asm("mov.b64 %0, {%1, %1};" : "=l"(factor) : "f"(SCALE == kScaleDown ? kDown : kUp));
#pragma unroll
    for (int i = 0; i < (sizeof(T) == 4 ? 2 : 4); ++i) {
        uint64_t x;
        if constexpr (sizeof(T) == 4)
            asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "r"(v[2 * i]), "r"(v[2 * i + 1]));
        else
            x = pair_of_word(v[i], T{});
        if (SCALE != kAsIs) asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(x) : "l"(factor));
        asm("fma.rn.f32x2 %0, %1, %1, %0;" : "+l"(acc[i & 1]) : "l"(x));
    }
}

__device__ __forceinline__ float sum_of(const uint64_t (&acc)[2]) {
    float a, b, c, d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(acc[0]));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(c), "=f"(d) : "l"(acc[1]));
    return (a + b) + (c + d);
}

template <typename T, Scale SCALE>
__device__ __forceinline__ float squares_of(const uint4 (&w)[kWords]) {
    uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
    for (int i = 0; i < kWords; ++i) add_squares<T, SCALE>(acc, w[i]);
    return sum_of(acc);
}

template <Scale SCALE>
__device__ __forceinline__ float squares_of(const float (&v)[8]) {
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float x = SCALE == kAsIs ? v[k] : v[k] * (SCALE == kScaleDown ? kDown : kUp);
        sum = fmaf(x, x, sum);
    }
    return sum;
}

template <typename T>
__device__ __forceinline__ void sum_piece(Sums& s, const T* p, long long n) {
    constexpr int PER = kPieceBytes / static_cast<int>(sizeof(T));
    constexpr int VEC = 16 / static_cast<int>(sizeof(T));
    const int here = static_cast<int>(n < PER ? n : PER);
    if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
        const uint4* q = reinterpret_cast<const uint4*>(p) + threadIdx.x;
        uint4 w[kWords];
        if (here == PER) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = __ldg(q + i * kClipThreads);
        } else {
            const int words = here / VEC;
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                w[i] = i * kClipThreads + static_cast<int>(threadIdx.x) < words ? __ldg(q + i * kClipThreads)
                                                                               : make_uint4(0u, 0u, 0u, 0u);
            const int at = words * VEC + threadIdx.x;  // the last, incomplete word
            float v[8] = {at < here ? wide(p[at]) : 0.0f};
            s.add([&](auto scale) { return squares_of<decltype(scale)::value>(v); });
        }
        s.add([&](auto scale) { return squares_of<T, decltype(scale)::value>(w); });
    } else {
        for (int i = threadIdx.x; i < here; i += 8 * kClipThreads) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = i + k * kClipThreads < here ? wide(p[i + k * kClipThreads]) : 0.0f;
            s.add([&](auto scale) { return squares_of<decltype(scale)::value>(v); });
        }
    }
}

template <typename T>
__device__ __forceinline__ uint32_t scale_word(uint32_t w, float f) {
    if constexpr (sizeof(T) == 4) {
        return __float_as_uint(__uint_as_float(w) * f);
    } else {
        const float2 v = word_pair(w, T{});
        if constexpr (std::is_same<T, __half>::value) {
            const __half2 h = __floats2half2_rn(v.x * f, v.y * f);
            return *reinterpret_cast<const uint32_t*>(&h);
        } else {
            return pack_bf16x2(v.x * f, v.y * f);
        }
    }
}

template <typename T>
__device__ __forceinline__ void scale_piece(const T* p, T* o, long long n, float f) {
    constexpr int PER = kPieceBytes / static_cast<int>(sizeof(T));
    constexpr int VEC = 16 / static_cast<int>(sizeof(T));
    const int here = static_cast<int>(n < PER ? n : PER);
    if (((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(o)) & 15u) == 0) {
        const int words = here / VEC;
        uint4 w[kWords];
        if (here == PER) {
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                w[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i * kClipThreads + threadIdx.x);
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                __stcs(reinterpret_cast<uint4*>(o) + i * kClipThreads + threadIdx.x,
                       make_uint4(scale_word<T>(w[i].x, f), scale_word<T>(w[i].y, f), scale_word<T>(w[i].z, f),
                                  scale_word<T>(w[i].w, f)));
            return;
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const int at = i * kClipThreads + threadIdx.x;
            if (at < words) w[i] = __ldcs(reinterpret_cast<const uint4*>(p) + at);
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const int at = i * kClipThreads + threadIdx.x;
            if (at < words)
                __stcs(reinterpret_cast<uint4*>(o) + at,
                       make_uint4(scale_word<T>(w[i].x, f), scale_word<T>(w[i].y, f), scale_word<T>(w[i].z, f),
                                  scale_word<T>(w[i].w, f)));
        }
        const int at = words * VEC + threadIdx.x;
        if (at < here) put(o + at, wide(p[at]) * f);
    } else {
        for (int i = threadIdx.x; i < here; i += 8 * kClipThreads) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = i + k * kClipThreads < here ? wide(p[i + k * kClipThreads]) : 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (i + k * kClipThreads < here) put(o + i + k * kClipThreads, v[k] * f);
        }
    }
}

__device__ __forceinline__ float cta_sum(float v, float* s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    __syncthreads();
    if (threadIdx.x % 32 == 0) s[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < kClipThreads / 32; ++w) v += s[w];
    return v;
}

template <int MOST>
__global__ void __launch_bounds__(kClipThreads, 4)
    grad_squares_kernel(const __grid_constant__ Table<MOST> t, double* partial) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ float scratch[kClipThreads / 32];
    Sums s{0.0f, 0.0f, 0.0f};
    const unsigned pieces = t.first[t.count];
    for (unsigned c = blockIdx.x; c < pieces; c += gridDim.x) {
        const int i = find_tensor(t, c);
        const long long at = static_cast<long long>(c - t.first[i]);
        if (t.dtype[i] == TPMLP_FP32) {
            constexpr int per = kPieceBytes / 4;
            sum_piece(s, static_cast<const float*>(t.in[i]) + at * per, t.size[i] - at * per);
        } else if (t.dtype[i] == TPMLP_FP16) {
            constexpr int per = kPieceBytes / 2;
            sum_piece(s, static_cast<const __half*>(t.in[i]) + at * per, t.size[i] - at * per);
        } else {
            constexpr int per = kPieceBytes / 2;
            sum_piece(s, static_cast<const __nv_bfloat16*>(t.in[i]) + at * per, t.size[i] - at * per);
        }
    }
    const float plain = cta_sum(s.plain, scratch);
    const float down = cta_sum(s.down, scratch);
    const float up = cta_sum(s.up, scratch);
    if (threadIdx.x == 0)
        partial[blockIdx.x] = isinf(plain) ? down * 0x1p128 : plain < kLowSum ? up * 0x1p-200 : plain;
}

// The norm from the partial sums, the same bits in every CTA that computes it.
__device__ __forceinline__ float norm_of(const double* partial, int parts) {
    __shared__ double sums[kClipThreads / 32];
    double p = 0.0;
    for (int i = threadIdx.x; i < parts; i += kClipThreads) p += partial[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) p += __shfl_xor_sync(0xFFFFFFFFu, p, o);
    if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = p;
    __syncthreads();
    p = 0.0;
#pragma unroll
    for (int w = 0; w < kClipThreads / 32; ++w) p += sums[w];
    return static_cast<float>(sqrt(p));
}

__global__ void __launch_bounds__(kClipThreads) grad_norm_kernel(const double* partial, int parts, float* norm) {
    pdl_launch_dependents();
    pdl_wait();
    const float n = norm_of(partial, parts);
    if (threadIdx.x == 0) *norm = n;
}

template <int MOST>
__global__ void __launch_bounds__(kClipThreads, 3)
    grad_scale_kernel(const __grid_constant__ Table<MOST> t, const double* partial, int parts, float max_norm,
                      float* norm) {
    pdl_launch_dependents();
    pdl_wait();
    const float n = norm_of(partial, parts);
    if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
    const float ratio = max_norm / (n + 1e-6f);
    const float f = ratio < 1.0f || isnan(ratio) ? ratio : 1.0f;
    const unsigned pieces = t.first[t.count];
    for (unsigned c = blockIdx.x; c < pieces; c += gridDim.x) {
        const unsigned piece = pieces - 1 - c;
        const int i = find_tensor(t, piece);
        if (f == 1.0f && t.out[i] == t.in[i]) continue;  // in place: the values stay
        const long long at = static_cast<long long>(piece - t.first[i]);
        if (t.dtype[i] == TPMLP_FP32) {
            constexpr int per = kPieceBytes / 4;
            scale_piece(static_cast<const float*>(t.in[i]) + at * per, static_cast<float*>(t.out[i]) + at * per,
                        t.size[i] - at * per, f);
        } else if (t.dtype[i] == TPMLP_FP16) {
            constexpr int per = kPieceBytes / 2;
            scale_piece(static_cast<const __half*>(t.in[i]) + at * per, static_cast<__half*>(t.out[i]) + at * per,
                        t.size[i] - at * per, f);
        } else {
            constexpr int per = kPieceBytes / 2;
            scale_piece(static_cast<const __nv_bfloat16*>(t.in[i]) + at * per,
                        static_cast<__nv_bfloat16*>(t.out[i]) + at * per, t.size[i] - at * per, f);
        }
    }
}

// A launch takes at most this many tensors (its table is a kernel parameter): the
// small table where it is enough, because the driver copies all of it.
constexpr int kSmallTable = 64, kLargeTable = 768;

struct Part {
    int first, count;   // tensors
    unsigned pieces;
    int grid, partial;  // CTAs, and the first one's partial sum
};

// The part of the list that starts at tensor `i`: up to kLargeTable tensors (their
// pieces fit 32 bits: the caller has checked the values of all).
Part part_at(const long long* sizes, const int* dtypes, int n, int i, int partial) {
    Part p{i, 0, 0u, 0, partial};
    long long pieces = 0;
    for (; i < n && p.count < kLargeTable; ++i, ++p.count) {
        const long long bytes = sizes[i] * (dtypes[i] == TPMLP_FP32 ? 4 : 2);
        pieces += (bytes + kPieceBytes - 1) / kPieceBytes;
    }
    p.pieces = static_cast<unsigned>(pieces);
    p.grid = static_cast<int>(pieces < kClipCtas ? pieces : kClipCtas);
    return p;
}

template <int MOST>
Table<MOST> make_table(const void* const* in, void* const* out, const long long* sizes, const int* dtypes,
                       const Part& p) {
    Table<MOST> t;
    unsigned pieces = 0;
    for (int k = 0; k < p.count; ++k) {
        const int i = p.first + k;
        t.in[k] = in[i];
        t.out[k] = out ? out[i] : nullptr;
        t.size[k] = sizes[i];
        t.dtype[k] = static_cast<unsigned char>(dtypes[i]);
        t.first[k] = pieces;
        const long long bytes = sizes[i] * (dtypes[i] == TPMLP_FP32 ? 4 : 2);
        pieces += static_cast<unsigned>((bytes + kPieceBytes - 1) / kPieceBytes);
    }
    t.first[p.count] = pieces;
    t.count = p.count;
    return t;
}

template <int MOST>
cudaError_t squares(const void* const* in, const long long* sizes, const int* dtypes, const Part& p, double* partial,
                    cudaStream_t st) {
    return launch_dependent(grad_squares_kernel<MOST>, dim3(p.grid), dim3(kClipThreads), 0, st,
                            make_table<MOST>(in, nullptr, sizes, dtypes, p), partial + p.partial);
}

template <int MOST>
cudaError_t scale(const void* const* in, void* const* out, const long long* sizes, const int* dtypes, const Part& p,
                  const double* partial, int parts, float max_norm, float* norm, cudaStream_t st) {
    return launch_dependent(grad_scale_kernel<MOST>, dim3(p.grid), dim3(kClipThreads), 0, st,
                            make_table<MOST>(in, out, sizes, dtypes, p), partial, parts, max_norm, norm);
}

}  // namespace

long long grad_partials(int n) {
    const long long parts = (static_cast<long long>(n) + kLargeTable - 1) / kLargeTable;
    return (parts > 0 ? parts : 1) * kClipCtas;
}

cudaError_t launch_grad_clip(const void* const* in, void* const* out, const long long* sizes, const int* dtypes, int n,
                             float max_norm, float* norm, double* partial, cudaStream_t st, int* launches) {
    int parts = 0;
    cudaError_t e;
    for (int i = 0; i < n;) {
        const Part p = part_at(sizes, dtypes, n, i, parts);
        i = p.first + p.count;
        if (p.pieces == 0) continue;
        e = p.count <= kSmallTable ? squares<kSmallTable>(in, sizes, dtypes, p, partial, st)
                                   : squares<kLargeTable>(in, sizes, dtypes, p, partial, st);
        if (e != cudaSuccess) return e;
        ++*launches;
        parts += p.grid;
    }
    if (out == nullptr || parts == 0) {
        e = launch_dependent(grad_norm_kernel, dim3(1), dim3(kClipThreads), 0, st, static_cast<const double*>(partial),
                             parts, norm);
        if (e == cudaSuccess) ++*launches;
        return e;
    }
    int at = 0;
    for (int i = 0; i < n;) {
        const Part p = part_at(sizes, dtypes, n, i, at);
        i = p.first + p.count;
        if (p.pieces == 0) continue;
        float* put_norm = at == 0 ? norm : nullptr;
        e = p.count <= kSmallTable
                ? scale<kSmallTable>(in, out, sizes, dtypes, p, partial, parts, max_norm, put_norm, st)
                : scale<kLargeTable>(in, out, sizes, dtypes, p, partial, parts, max_norm, put_norm, st);
        if (e != cudaSuccess) return e;
        ++*launches;
        at += p.grid;
    }
    return cudaSuccess;
}

}  // namespace tpmlp
