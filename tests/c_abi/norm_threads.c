/* norm_threads.c -- two host threads that call tp_ln_backward (or
 * tp_ln_residual_forward) at once, each on a stream of its own, with row
 * widths of their own: every call must be accepted and give what the same
 * call gave before the threads began.
 *
 *   norm_threads backward|residual calls h1 h2
 *
 * Exit status: 0 on success; 2 bad arguments; 4 a CUDA runtime call failed;
 * 5 the library refused a call or an output differs. */
#include <pthread.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <cuda_runtime_api.h>

#include "tpmlp.h"

enum { ROWS = 64 };

struct job {
    int residual, h, calls, status;
    void *x, *gamma, *dx, *sum;
    float *mean, *rstd, *dgamma, *dbeta, *partial;
    cudaStream_t stream;
    uint16_t *want, *got;
};

static int call(const struct job* j) {
    const int s = j->residual
                      ? tp_ln_residual_forward(j->x, j->x, j->gamma, j->gamma, ROWS, j->h, 1e-5f, j->dx, j->sum,
                                               j->mean, j->rstd, j->stream)
                      : tp_ln_backward(j->x, j->x, j->gamma, j->mean, j->rstd, ROWS, j->h, TPMLP_BF16, j->dx,
                                       j->dgamma, j->dbeta, j->partial, j->stream);
    if (s != TPMLP_OK) {
        fprintf(stderr, "%s, h = %d: %s (CUDA error %d)\n",
                j->residual ? "tp_ln_residual_forward" : "tp_ln_backward", j->h, tp_mlp_status_string(s),
                tpmlp_last_cuda_error());
        return 5;
    }
    return 0;
}

static int fetch(const struct job* j, uint16_t* to) {
    if (cudaMemcpyAsync(to, j->dx, sizeof(uint16_t) * ROWS * (size_t)j->h, cudaMemcpyDeviceToHost, j->stream) !=
            cudaSuccess ||
        cudaStreamSynchronize(j->stream) != cudaSuccess)
        return 4;
    return 0;
}

static int set_up(struct job* j) {
    const size_t n = ROWS * (size_t)j->h, floats = tp_ln_backward_workspace_floats(ROWS, j->h, TPMLP_BF16);
    j->want = malloc(sizeof(uint16_t) * n);
    j->got = malloc(sizeof(uint16_t) * n);
    if (!j->want || !j->got) return 4;
    uint32_t seed = 12345u + (uint32_t)j->h;
    for (size_t i = 0; i < n; ++i) { /* bf16 of about +-1: exponent 126 or 127 */
        seed = seed * 1664525u + 1013904223u;
        j->got[i] = (uint16_t)(((seed >> 16) & 0x80FFu) | 0x3F00u);
    }
    if (cudaMalloc(&j->x, 2 * n) || cudaMalloc(&j->gamma, 2 * (size_t)j->h) || cudaMalloc(&j->dx, 2 * n) || cudaMalloc(&j->sum, 2 * n) ||
        cudaMalloc((void**)&j->mean, 4 * ROWS) || cudaMalloc((void**)&j->rstd, 4 * ROWS) ||
        cudaMalloc((void**)&j->dgamma, 4 * (size_t)j->h) || cudaMalloc((void**)&j->dbeta, 4 * (size_t)j->h) ||
        cudaMalloc((void**)&j->partial, 4 * floats) || cudaStreamCreateWithFlags(&j->stream, cudaStreamNonBlocking) ||
        cudaMemcpy(j->x, j->got, 2 * n, cudaMemcpyHostToDevice) ||
        cudaMemcpy(j->gamma, j->got, 2 * (size_t)j->h, cudaMemcpyHostToDevice))
        return 4;
    if (tp_ln_forward(j->x, j->gamma, j->gamma, ROWS, j->h, TPMLP_BF16, 1e-5f, j->dx, j->mean, j->rstd, j->stream) !=
        TPMLP_OK)
        return 5;
    const int s = call(j);
    return s ? s : fetch(j, j->want);
}

static void* work(void* arg) {
    struct job* j = arg;
    for (int i = 0; i < j->calls && j->status == 0; ++i) {
        j->status = call(j);
        if (j->status == 0 && i % 1000 == 999) {
            j->status = fetch(j, j->got);
            if (j->status == 0 && memcmp(j->got, j->want, sizeof(uint16_t) * ROWS * (size_t)j->h) != 0) {
                fprintf(stderr, "h = %d: the output differs\n", j->h);
                j->status = 5;
            }
        }
    }
    return NULL;
}

int main(int argc, char** argv) {
    if (argc != 5 || (strcmp(argv[1], "backward") != 0 && strcmp(argv[1], "residual") != 0)) {
        fprintf(stderr, "usage: %s backward|residual calls h1 h2\n", argv[0]);
        return 2;
    }
    struct job jobs[2];
    pthread_t threads[2];
    memset(jobs, 0, sizeof jobs);
    for (int k = 0; k < 2; ++k) {
        jobs[k].residual = strcmp(argv[1], "residual") == 0;
        jobs[k].calls = atoi(argv[2]);
        jobs[k].h = atoi(argv[3 + k]);
        if (jobs[k].calls < 1 || jobs[k].h < 1) return 2;
        const int s = set_up(&jobs[k]);
        if (s) return s;
    }
    for (int k = 0; k < 2; ++k)
        if (pthread_create(&threads[k], NULL, work, &jobs[k])) return 4;
    for (int k = 0; k < 2; ++k) pthread_join(threads[k], NULL);
    return jobs[0].status ? jobs[0].status : jobs[1].status;
}
