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

// States between segments: [B,H,dv][nseg][cols], cols = dk rounded up to scan_cols (16-byte rows); the
// segments of a channel lie together, so that the walk along them reads consecutive lines.
struct ScanWork {
    int seg, nseg;     // tokens of a segment (a multiple of kScanChunk), segments
    int run;           // segments that a block of kScanBoth walks
    float *ends;       // end states (kScanEnds: the last segment's place keeps the initial state)
    float *grads;      // kScanBoth
    float *steps;      // [B,H,dv][nseg] sums of steps
    falcon_view_t dO;  // kScanBoth
};

inline int scan_cols(int dk) { return dk <= 4 ? 4 : dk <= 8 ? 8 : dk <= 16 ? 16 : dk <= 32 ? 32 : dk <= 64 ? 64 : 128; }

// One pass over segments (scan.cu).
cudaError_t launch_scan_pass(int mode, const falcon_scan_args_t &a, const ScanWork &w, cudaStream_t s);

}  // namespace falcon
