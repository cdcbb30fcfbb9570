// ops_sum.cu -- column sums of partial rows, the last step of every gradient that sums over tokens.
#include "ops.cuh"

namespace falcon {

namespace {

constexpr int kSumCols = 32, kSumChains = 32;

struct SumJobs {
    SumJob job[4];
};

// 32 columns a block (one 128-byte line of each row), 32 chains over the rows joined in a fixed order.
__global__ void __launch_bounds__(kSumCols * kSumChains) column_sum_kernel(SumJobs jobs, long long nparts) {
    __shared__ float acc[kSumChains][kSumCols + 1];
    const SumJob j = jobs.job[blockIdx.y];
    const long long e = (long long)blockIdx.x * kSumCols + threadIdx.x;
    if ((long long)blockIdx.x * kSumCols >= j.n) return;
    float s = 0.f;
    if (e < j.n) {
#pragma unroll 8
        for (long long p = threadIdx.y; p < nparts; p += kSumChains) s += j.part[p * j.stride + e];
    }
    acc[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && e < j.n) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < kSumChains; ++i) t += acc[i][threadIdx.x];
        j.out[e] = t;
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
    const dim3 grid((unsigned)((most + kSumCols - 1) / kSumCols), (unsigned)n);
    column_sum_kernel<<<grid, dim3(kSumCols, kSumChains), 0, s>>>(js, nparts);
    return cudaGetLastError();
}

}  // namespace falcon
