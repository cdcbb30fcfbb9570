// scan.cuh -- what the forward and backward kernels of the selective scan share.
#pragma once

#include "ops.cuh"

namespace falcon {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

constexpr int kScanThreads = 128;
constexpr int kScanChunk = 8;   // tokens whose inputs are loaded together

enum ScanMode : int {
    kScanFull = 0,   // outputs, from the given or joined start state
    kScanEnds = 1,   // each segment's end state from a zero state, and its sum of steps
    kScanBoth = 2    // the same, and the gradient that its outputs send to the state before it
};

struct ScanWork {
    int seg, nseg;     // tokens of a segment, segments
    float *ends;       // [nseg][B,H,dv,dk]
    float *grads;      // [nseg][B,H,dv,dk] (kScanBoth)
    float *steps;      // [nseg][B,H,dv]
    falcon_view_t dO;  // kScanBoth
};

// One pass over segments (scan.cu).
cudaError_t launch_scan_pass(int mode, const falcon_scan_args_t &a, const ScanWork &w, cudaStream_t s);

}  // namespace falcon
