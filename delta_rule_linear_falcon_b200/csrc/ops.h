// ops.h -- internal launch interface of the operators around the memory (convolution, q/k norm,
// selective scan): what api_ops.cu checks and hands to the kernel translation units.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

#include "../../include/falcon.h"

namespace falcon {

constexpr long long kMaxGrid = 0x7fffffffLL;

// Column sums of partial rows: out[e] = sum_p part[p * stride + e] for e < n, in a fixed order. Up to
// four arrays in one launch; a job without an output is left out.
struct SumJob {
    const float *part = nullptr;
    long long n = 0, stride = 0;
    float *out = nullptr;
};
cudaError_t launch_column_sums(const SumJob *jobs, int njobs, long long nparts, cudaStream_t s);

// convolution (conv.cu)
cudaError_t launch_conv_fwd(const falcon_conv_args_t &a, int num_sms, cudaStream_t s);
cudaError_t launch_conv_step(const falcon_conv_args_t &a, int num_sms, cudaStream_t s);
size_t conv_bwd_workspace(const falcon_conv_args_t &a);
cudaError_t launch_conv_bwd(const falcon_conv_args_t &a, const falcon_conv_grads_t &g, float *ws, cudaStream_t s);

// selective scan (scan.cu, scan_bwd.cu)
struct ScanPlan {
    int seg = 0;        // tokens of a segment (T when the sequence is not split)
    int nseg = 1;
    size_t bytes = 0;   // workspace: states and sums of steps between the segments
};
ScanPlan scan_plan(const falcon_scan_args_t &a, int num_sms);
cudaError_t launch_scan_fwd(const falcon_scan_args_t &a, const ScanPlan &plan, float *ws, cudaStream_t s);
cudaError_t launch_scan_step(const falcon_scan_args_t &a, int num_sms, cudaStream_t s);
size_t scan_bwd_workspace(const falcon_scan_args_t &a);
bool scan_bwd_fits(const falcon_scan_args_t &a);   // its grids
cudaError_t launch_scan_bwd(const falcon_scan_args_t &a, const falcon_scan_grads_t &g, float *ws, cudaStream_t s);

// norm of queries and keys (qknorm.cu)
size_t qknorm_bwd_workspace(const falcon_qknorm_args_t &a);
cudaError_t launch_qknorm_fwd(const falcon_qknorm_args_t &a, cudaStream_t s);
cudaError_t launch_qknorm_bwd(const falcon_qknorm_args_t &a, const falcon_qknorm_grads_t &g, float *ws, cudaStream_t s);

}  // namespace falcon
