// ops_sum.cu -- column sums of partial rows, the last step of every gradient that sums over tokens.
#include "ops.cuh"

namespace falcon {

namespace {

constexpr int kSumCols = 32, kChains = 8;

struct SumJobs {
    SumJob job[4];
    unsigned first[4];   // blocks of the jobs before
    int count;
};

// 32 columns a block (one 128-byte line of each row), kChains sums over every kChains-th row, joined in a fixed order.
// Bound by the latency of the loads: eight rows of a chain are in flight together. 36900 columns of 26 rows take 4.1 us,
// 10240 of 108 rows 4.7 us, 256 of 296 rows 5.7 us (one chain and 128 columns a block: 5.1, 9.1 and 18 us; 32 chains:
// slower by a tenth to threefold). Blocks are numbered through the jobs: a grid of the widest job for each of them
// took 16 us for the first of these.
// LONG: more rows than kLong (one for each of very many short sequences). A chain then hands its sum over after each kRun
// batches, so that it loses no more than a short one. On its own, since that costs the short sums up to a microsecond.
constexpr int kBatch = 8, kRun = 1024, kLong = kRun * kBatch * kChains;

template <bool LONG>
__global__ void __launch_bounds__(kSumCols * kChains) column_sum_kernel(SumJobs jobs, int nparts, long long runs) {
    __shared__ float acc[kChains][kSumCols + 1];
    int which = 0;
#pragma unroll
    for (int i = 1; i < 4; ++i)
        if (i < jobs.count && blockIdx.x >= jobs.first[i]) which = i;
    const SumJob j = jobs.job[which];
    const long long e = (long long)(blockIdx.x - jobs.first[which]) * kSumCols + threadIdx.x;
    float s = 0.f;
    if (e < j.n) {
        constexpr int U = kBatch;
        const float *p = j.part + threadIdx.y * j.stride + e;
        const long long step = kChains * j.stride;
        float done = 0.f;
        if (LONG) {
            for (long long r = 0; r < runs; ++r) {
#pragma unroll 4
                for (int k = 0; k < kRun; ++k) {
                    float x[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) x[u] = p[u * step];
#pragma unroll
                    for (int u = 0; u < U; ++u) s += x[u];
                    p += U * step;
                }
                done += s;
                s = 0.f;
            }
        }
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
        if (LONG) s += done;
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
    long long blocks = 0;
    for (int i = 0; i < njobs; ++i) {
        if (!jobs[i].out || jobs[i].n == 0) continue;
        js.job[js.count] = jobs[i];
        js.first[js.count++] = (unsigned)blocks;
        blocks += (jobs[i].n + kSumCols - 1) / kSumCols;
    }
    if (js.count == 0) return cudaSuccess;
    if (blocks > kMaxGrid) return cudaErrorInvalidConfiguration;
    const dim3 block(kSumCols, kChains);
    if (nparts > kLong) column_sum_kernel<true><<<(unsigned)blocks, block, 0, s>>>(js, (int)(nparts % kLong), nparts / kLong);
    else column_sum_kernel<false><<<(unsigned)blocks, block, 0, s>>>(js, (int)nparts, 0);
    return cudaGetLastError();
}

}  // namespace falcon
