// ops_sum.cu -- column sums of partial rows, the last step of every gradient that sums over tokens.
#include "ops.cuh"

namespace falcon {

namespace {

constexpr int kSumCols = 32, kChains = 8;

struct SumJobs {
    SumJob job[4];
};

// 32 columns a block (one 128-byte line of each row), kChains sums over every kChains-th row, joined in a
// fixed order. Bound by the latency of the loads: eight rows of a chain are in flight together. 33000 columns of 128
// rows take 16.5 us, 128 columns of 296 rows 6 us (with 32 chains and blocks of 1024 threads 52 and 6.7 us).
__global__ void __launch_bounds__(kSumCols * kChains) column_sum_kernel(SumJobs jobs, int nparts) {
    __shared__ float acc[kChains][kSumCols + 1];
    const SumJob j = jobs.job[blockIdx.y];
    if ((long long)blockIdx.x * kSumCols >= j.n) return;
    const long long e = (long long)blockIdx.x * kSumCols + threadIdx.x;
    float s = 0.f;
    if (e < j.n) {
        constexpr int U = 8;
        const float *p = j.part + threadIdx.y * j.stride + e;
        const long long step = kChains * j.stride;
        int i = threadIdx.y;
        for (; i + (U - 1) * kChains < nparts; i += U * kChains) {
            float x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) x[u] = p[u * step];
#pragma unroll
            for (int u = 0; u < U; ++u) s += x[u];
            p += U * step;
        }
        float x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = i + u * kChains < nparts ? p[u * step] : 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) s += x[u];
    }
    acc[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && e < j.n) {
        float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kChains; ++i) t[i % 4] += acc[i][threadIdx.x];
        j.out[e] = (t[0] + t[1]) + (t[2] + t[3]);
    }
}

}  // namespace

cudaError_t launch_column_sums(const SumJob *jobs, int njobs, long long nparts, cudaStream_t s) {
    SumJobs js{};
    long long most = 0;
    int n = 0;
    for (int i = 0; i < njobs; ++i) {
        if (!jobs[i].out || jobs[i].n == 0) continue;
        js.job[n++] = jobs[i];
        most = jobs[i].n > most ? jobs[i].n : most;
    }
    if (n == 0) return cudaSuccess;
    if (nparts > 0x7fffffff / 16) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)((most + kSumCols - 1) / kSumCols), (unsigned)n);
    column_sum_kernel<<<grid, dim3(kSumCols, kChains), 0, s>>>(js, (int)nparts);
    return cudaGetLastError();
}

}  // namespace falcon
