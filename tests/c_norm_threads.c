/* Two host threads norm rows of different widths, whose launches share a kernel and
 * differ in its shared memory.  Every call has to be accepted.  Prints "threads ok". */
#include <cuda_runtime.h>
#include <pthread.h>
#include <stdint.h>
#include <stdio.h>

#include "vlmce.h"

enum { kRows = 2000, kCalls = 20000 };

typedef struct {
    int64_t H;
    void *x, *w, *y, *dx, *ws;
    float *rstd;
    size_t ws_bytes;
    cudaStream_t stream;
    pthread_barrier_t *start;
    int refused;
} Job;

static int prepare(Job *j, int64_t H) {
    j->H = H;
    j->ws_bytes = vlmce_rmsnorm_bwd_workspace_bytes(kRows, H);
    return cudaStreamCreateWithFlags(&j->stream, cudaStreamNonBlocking) ||
           cudaMalloc(&j->x, kRows * H * 2) || cudaMalloc(&j->y, kRows * H * 2) ||
           cudaMalloc(&j->dx, kRows * H * 2) || cudaMalloc(&j->w, H * 2) ||
           cudaMalloc((void **)&j->rstd, kRows * 4) || cudaMalloc(&j->ws, j->ws_bytes) ||
           cudaMemset(j->x, 0, kRows * H * 2) || cudaMemset(j->w, 0, H * 2) ||
           cudaMemset(j->rstd, 0, kRows * 4);
}

static void *run(void *p) {
    Job *j = p;
    pthread_barrier_wait(j->start);
    for (int i = 0; i < kCalls; ++i) {
        vlmce_status st = rmsnorm_fwd(j->x, j->H, NULL, j->H, j->w, VLMCE_BF16, VLMCE_BF16, kRows,
                                      j->H, 1e-6f, 0.f, j->y, j->H, VLMCE_BF16, NULL, j->H,
                                      j->rstd, NULL, (vlmce_stream_t)j->stream);
        if (st == VLMCE_OK && i % 4 == 0)
            st = rmsnorm_bwd(j->y, j->H, j->x, j->H, j->w, VLMCE_BF16, j->rstd, NULL, j->H,
                             VLMCE_BF16, kRows, j->H, 0.f, j->dx, j->H, NULL, 0, j->ws,
                             j->ws_bytes, (vlmce_stream_t)j->stream);
        if (st != VLMCE_OK && j->refused++ == 0)
            printf("H %lld, call %d: %s [%s]\n", (long long)j->H, i, vlmce_status_string(st),
                   vlmce_last_error());
    }
    return NULL;
}

int main(void) {
    pthread_barrier_t start;
    Job job[2] = {{0}, {0}};
    pthread_t t[2];
    pthread_barrier_init(&start, NULL, 2);
    for (int i = 0; i < 2; ++i) {
        job[i].start = &start;
        if (prepare(&job[i], i ? 4096 : 8192)) return 2;
    }
    for (int i = 0; i < 2; ++i) pthread_create(&t[i], NULL, run, &job[i]);
    for (int i = 0; i < 2; ++i) pthread_join(t[i], NULL);
    if (cudaDeviceSynchronize() != cudaSuccess) return 3;
    if (job[0].refused || job[1].refused) {
        printf("refused: %d and %d of %d\n", job[0].refused, job[1].refused, kCalls);
        return 1;
    }
    printf("threads ok\n");
    return 0;
}
