// scan.cuh -- what the forward and backward kernels of the selective scan share.
#pragma once

#include <float.h>

#include "ops.cuh"

namespace falcon {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// A in units of log2 e, a decay being 2^(dt x). An infinite A, or one that overflows here, is the largest finite value of
// its sign: a step of 0, as behind a sequence's end, times infinity would be NaN, and so would the sums of steps of 0
// between segments. Decays over steps above 2^-120 are 0 all the same.
__device__ __forceinline__ float decay_rate(float a) {
    const float x = a * kLog2e;
    return x < -FLT_MAX ? -FLT_MAX : x > FLT_MAX ? FLT_MAX : x;   // NaN stays
}

constexpr int kScanThreads = 128;
constexpr int kScanChunk = 8;   // tokens whose inputs are loaded together

enum ScanMode : int {
    kScanFull = 0,   // outputs, from the given or joined start state
    kScanEnds = 1,   // each segment's end state from a zero state, and its sum of steps
    kScanBoth = 2    // for the backward pass: walks of several segments, each from a zero state: the state before each
                     // segment, the walk's end state, and the gradient that its outputs send to the state before it
};

// States between segments: [B,H,dv][number][cols], cols = dk rounded up to scan_cols (16-byte rows); those of a
// channel lie together, so that the walk along them reads consecutive lines.
struct ScanWork {
    int seg, nseg;     // tokens of a segment (a multiple of kScanChunk), segments
    float *ends;       // kScanEnds: [nseg] end states (the last segment's place keeps the initial state);
                       // kScanBoth: [nseg] states before the segments
    float *steps;      // [B,H,dv][nseg] sums of steps: of the segment; kScanBoth: of its walk before it
    // kScanBoth
    int walk, nwalk;   // segments of a walk, walks
    int block;         // walks of a block
    float *wends;      // [nwalk] end states of the walks
    float *wgrads;     // [nwalk] gradients with respect to the states before them
    float *wsteps;     // [B,H,dv][nwalk] sums of steps
    falcon_view_t dO;
};

inline int scan_cols(int dk) { return dk <= 4 ? 4 : dk <= 8 ? 8 : dk <= 16 ? 16 : dk <= 32 ? 32 : dk <= 64 ? 64 : 128; }

// One pass over segments (scan.cu).
cudaError_t launch_scan_pass(int mode, const falcon_scan_args_t &a, const ScanWork &w, cudaStream_t s);

}  // namespace falcon
