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
#include <cstdint>

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

template <typename T>
cudaError_t forward(const void* x, const void* gamma, const void* beta, int T_, int h, float eps,
                    void* y, float* mean, float* rstd, cudaStream_t st, int* launches) {
    ++*launches;
    return launch_dependent(norm_forward_kernel<T>, dim3(T_), dim3(kRowThreads), 0, st,
                            static_cast<const T*>(x), static_cast<const T*>(gamma),
                            static_cast<const T*>(beta), h, eps, static_cast<T*>(y), mean, rstd);
}

template <typename T>
cudaError_t backward(const void* dy, const void* x, const void* gamma, const float* mean,
                     const float* rstd, int T_, int h, void* dx, float* dgamma, float* dbeta,
                     float* partial, cudaStream_t st, int* launches) {
    cudaError_t e = launch_dependent(norm_backward_kernel<T>, dim3(T_), dim3(kRowThreads), 0, st,
                                     static_cast<const T*>(dy), static_cast<const T*>(x),
                                     static_cast<const T*>(gamma), mean, rstd, h, static_cast<T*>(dx));
    if (e != cudaSuccess) return e;
    ++*launches;
    const int chunks = norm_param_chunks(T_, h);
    e = launch_dependent(norm_param_grad_kernel<T>, dim3(ceil_div(h, 32), chunks), dim3(256), 0, st,
                         static_cast<const T*>(dy), static_cast<const T*>(x), mean, rstd, T_, h,
                         ceil_div(T_, chunks), partial);
    if (e != cudaSuccess) return e;
    ++*launches;
    if ((e = launch_rowsum_f32(partial, chunks, h, dgamma, st, launches)) != cudaSuccess) return e;
    return launch_rowsum_f32(partial + static_cast<size_t>(chunks) * h, chunks, h, dbeta, st, launches);
}

}  // namespace

int norm_param_chunks(int T, int h) {
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
                                 float* dgamma, float* dbeta, float* partial, cudaStream_t st,
                                 int* launches) {
    switch (dtype) {
        case TPMLP_BF16:
            return backward<__nv_bfloat16>(dy, x, gamma, mean, rstd, T, h, dx, dgamma, dbeta, partial, st, launches);
        case TPMLP_FP16:
            return backward<__half>(dy, x, gamma, mean, rstd, T, h, dx, dgamma, dbeta, partial, st, launches);
        default:
            return backward<float>(dy, x, gamma, mean, rstd, T, h, dx, dgamma, dbeta, partial, st, launches);
    }
}

}  // namespace tpmlp
