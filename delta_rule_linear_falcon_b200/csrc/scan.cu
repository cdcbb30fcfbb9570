// scan.cu -- falcon_scan_fwd and falcon_scan_step: the selective scan
//   S_t[i,c] = exp(dt_t[i] A[i,c]) S_{t-1}[i,c] + dt_t[i] v_t[i] k_t[c],
//   o_t[i]   = (sum_c S_t[i,c] q_t[c] + D[i] v_t[i]) silu(z_t[i]).
//
// Each entry of the state takes one exponential and four fp32 operations a token, so at dk = 16 the
// exponential unit (16 a clock and SM) bounds the pass, well above HBM: 16 exponentials against about
// eight bytes of v, delta, z and o. No product is shared between channels, so there is no matrix
// instruction to use. A thread owns a channel and ST <= 16 columns of its state in registers (SL lanes
// share a channel when dk > 16 and join their parts of o); neighbouring lanes own neighbouring channels,
// so v, delta, z and o move as whole lines whatever their alignment. q_t and k_t are the same for all
// channels of a head: the block stages kScanChunk tokens of them in shared memory (double buffered) and
// reads them as broadcasts. The next chunk's loads are issued before this chunk's arithmetic.
// The step size (softplus) is computed once per channel and token, 1 / 16 of the state's exponentials.
//
// Split: B H dv channels are the only parallel axis of the recurrence; with few of them the sequence is
// cut into segments (scan_plan). A first launch runs every segment from a zero state and leaves its end
// state E and the sum of its steps sd, from which the decay over the segment is exp(A sd); in the second
// each segment joins the states before it, S <- exp(A sd_j) S + E_j, and runs with outputs.
#include "scan.cuh"

namespace falcon {

namespace {

template <typename IO, int ST, int SL, int MODE>
__global__ void __launch_bounds__(kScanThreads) scan_kernel(falcon_scan_args_t a, ScanWork w, int ngrp) {
    constexpr int DKP = ST * SL;                     // padded columns
    constexpr int CPB = kScanThreads / SL;           // channels of a block
    constexpr int ROW = 2 * DKP;                     // k and q of a token
    constexpr int NKQ = (kScanChunk * ROW + kScanThreads - 1) / kScanThreads;
    typedef Pack<IO, 1> P;
    __shared__ __align__(16) float kq[2][kScanChunk * ROW];

    unsigned bid = blockIdx.x;
    const int grp = (int)(bid % (unsigned)ngrp);
    bid /= (unsigned)ngrp;
    const int bh = (int)(bid % (unsigned)(a.B * a.H));
    const int seg = (int)(bid / (unsigned)(a.B * a.H));
    const int b = bh / a.H, h = bh % a.H;
    const int tid = threadIdx.x;
    const int sl = tid % SL, ch = grp * CPB + tid / SL;
    const bool ok = ch < a.dv;
    const int n = seq_length(a.lengths, b, a.T);
    const long long first = (long long)seg * w.seg;
    const int t0 = (int)(first < n ? first : n);
    const int t1 = (int)(first + w.seg < n ? first + w.seg : n);

    const long long hc = (long long)h * a.dv + ch;               // (H,dv)
    const long long bhc = (long long)bh * a.dv + ch;             // (B,H,dv)
    const long long plane = (long long)a.B * a.H * a.dv * a.dk;  // one segment's states
    const long long rows = (long long)a.B * a.H * a.dv;

    if (MODE == kScanEnds && seg == w.nseg - 1) {
        // the last segment's end is not needed: its place keeps the initial state for the second launch,
        // which may write S_out over S0
        if (ok)
#pragma unroll
            for (int s = 0; s < ST; ++s)
                if (sl * ST + s < a.dk)
                    w.ends[seg * plane + bhc * a.dk + sl * ST + s] = a.S0 ? a.S0[bhc * a.dk + sl * ST + s] : 0.f;
        return;
    }

    float A2[ST], S[ST], Pr[MODE == kScanBoth ? ST : 1], G[MODE == kScanBoth ? ST : 1];
#pragma unroll
    for (int s = 0; s < ST; ++s) {
        const int c = sl * ST + s;
        A2[s] = ok && c < a.dk ? a.A[hc * a.dk + c] * kLog2e : 0.f;
        S[s] = 0.f;
        if (MODE == kScanBoth) { Pr[s] = 1.f; G[s] = 0.f; }
    }
    const float bias = ok && a.delta_bias ? a.delta_bias[hc] : 0.f;
    const float skip = ok && MODE == kScanFull && a.D ? a.D[hc] : 0.f;
    const bool soft = (a.flags & FALCON_SCAN_SOFTPLUS) != 0;
    if (MODE == kScanFull && ok) {
        const float *from = w.nseg > 1 ? w.ends + (long long)(w.nseg - 1) * plane : a.S0;
#pragma unroll
        for (int s = 0; s < ST; ++s)
            if (from && sl * ST + s < a.dk) S[s] = from[bhc * a.dk + sl * ST + s];
        for (int j = 0; j < seg; ++j) {
            const float sd = w.steps[j * rows + bhc];
            const float *e = w.ends + j * plane + bhc * a.dk + sl * ST;
#pragma unroll
            for (int s = 0; s < ST; ++s)
                if (sl * ST + s < a.dk) S[s] = fmaf(fast_ex2(A2[s] * sd), S[s], e[s]);
        }
    }

    const IO *pv = row_of<IO>(a.v, b, h, 0) + ch;
    const IO *pd = row_of<IO>(a.delta, b, h, 0) + ch;
    const IO *pz = a.z.p ? row_of<IO>(a.z, b, h, 0) + ch : nullptr;
    const IO *pk = row_of<IO>(a.k, b, h, 0);
    const IO *pq = row_of<IO>(a.q, b, h, 0);
    const float *pg = MODE == kScanBoth ? row_of<float>(w.dO, b, h, 0) + ch : nullptr;
    IO *po = MODE == kScanFull ? row_of<IO>(a.o, b, h, 0) + ch : nullptr;

    typename P::raw rv[kScanChunk], rd[kScanChunk], rz[kScanChunk], rkq[NKQ];
    float rg[MODE == kScanBoth ? kScanChunk : 1];
    auto fetch = [&](int t) {
#pragma unroll
        for (int j = 0; j < kScanChunk; ++j) {
            const bool in = ok && t + j < t1;
            rv[j] = in ? P::ld(pv + (t + j) * a.v.st) : P::zero();
            rd[j] = in ? P::ld(pd + (t + j) * a.delta.st) : P::zero();
            if (MODE != kScanEnds) rz[j] = in && pz ? P::ld(pz + (t + j) * a.z.st) : P::zero();
            if (MODE == kScanBoth) rg[j] = in ? pg[(t + j) * w.dO.st] : 0.f;
        }
#pragma unroll
        for (int m = 0; m < NKQ; ++m) {
            const int e = tid + m * kScanThreads, j = e / ROW, c = e % DKP;
            const bool isq = e % ROW >= DKP;
            rkq[m] = P::zero();
            if (e < kScanChunk * ROW && t + j < t1 && c < a.dk && !(MODE == kScanEnds && isq))
                rkq[m] = isq ? P::ld(pq + (t + j) * a.q.st + c) : P::ld(pk + (t + j) * a.k.st + c);
        }
    };

    float sum = 0.f;
    fetch(t0);
    int buf = 0;
    for (int t = t0; t < t1; t += kScanChunk, buf ^= 1) {
        float dt[kScanChunk], dtv[kScanChunk], v[kScanChunk], z[kScanChunk], g[kScanChunk];
#pragma unroll
        for (int m = 0; m < NKQ; ++m) {
            const int e = tid + m * kScanThreads;
            float x[1];
            P::cvt(rkq[m], x);
            if (e < kScanChunk * ROW) kq[buf][e] = x[0];
        }
#pragma unroll
        for (int j = 0; j < kScanChunk; ++j) {
            float x[1];
            P::cvt(rv[j], x);
            v[j] = x[0];
            P::cvt(rd[j], x);
            const float raw = x[0] + bias;
            dt[j] = ok && t + j < t1 ? (soft ? softplus(raw) : raw) : 0.f;   // 0 behind the end: the state stays
            dtv[j] = dt[j] * v[j];
            if (MODE != kScanEnds) {
                P::cvt(rz[j], x);
                z[j] = x[0];
            }
            if (MODE == kScanBoth) g[j] = pz ? rg[j] * silu(z[j]) : rg[j];
            if (MODE != kScanFull) sum += dt[j];
        }
        if (t + kScanChunk < t1) fetch(t + kScanChunk);
        __syncthreads();   // the chunk is staged; the other buffer was last read before this barrier
#pragma unroll
        for (int j = 0; j < kScanChunk; ++j) {
            const float4 *k4 = reinterpret_cast<const float4 *>(&kq[buf][j * ROW + sl * ST]);
            const float4 *q4 = reinterpret_cast<const float4 *>(&kq[buf][j * ROW + DKP + sl * ST]);
            float y = 0.f;
#pragma unroll
            for (int s4 = 0; s4 < ST / 4; ++s4) {
                const float4 kk = k4[s4];
                float4 qq = make_float4(0.f, 0.f, 0.f, 0.f);
                if (MODE != kScanEnds) qq = q4[s4];
                const float kx[4] = {kk.x, kk.y, kk.z, kk.w}, qx[4] = {qq.x, qq.y, qq.z, qq.w};
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int s = s4 * 4 + r;
                    const float e = fast_ex2(dt[j] * A2[s]);
                    S[s] = fmaf(e, S[s], dtv[j] * kx[r]);
                    if (MODE == kScanFull) y = fmaf(S[s], qx[r], y);
                    if (MODE == kScanBoth) {
                        Pr[s] *= e;
                        G[s] = fmaf(Pr[s], g[j] * qx[r], G[s]);
                    }
                }
            }
            if (MODE == kScanFull) {
#pragma unroll
                for (int m = 1; m < SL; m <<= 1) y += __shfl_xor_sync(0xffffffffu, y, m);
                y = fmaf(skip, v[j], y);
                if (pz) y *= silu(z[j]);
                if (ok && sl == 0 && t + j < t1) {
                    const float out[1] = {y};
                    P::st(po + (t + j) * a.o.st, out);
                }
            }
        }
    }
    if (!ok) return;
    float *to = MODE == kScanFull ? (seg == w.nseg - 1 ? a.S_out : nullptr) : w.ends + seg * plane;
#pragma unroll
    for (int s = 0; s < ST; ++s) {
        const int c = sl * ST + s;
        if (c >= a.dk) continue;
        if (to) to[bhc * a.dk + c] = S[s];
        if (MODE == kScanBoth) w.grads[seg * plane + bhc * a.dk + c] = G[s];
    }
    if (MODE != kScanFull && sl == 0) w.steps[seg * rows + bhc] = sum;
}

// One token. A channel's row of the state is read and written by G lanes, four columns each, so the
// state moves in whole lines; each thread has kStepRows channels' rows in flight.
constexpr int kStepThreads = 128, kStepRows = 4;

template <typename IO, int G, bool V4>
__global__ void __launch_bounds__(kStepThreads) scan_step_kernel(falcon_scan_args_t a, int ngrp) {
    constexpr int CPP = kStepThreads / G;   // channels of a pass
    const int grp = blockIdx.x % (unsigned)ngrp;
    const int bh = blockIdx.x / (unsigned)ngrp;
    const int b = bh / a.H, h = bh % a.H;
    const int sl = threadIdx.x % G, c0 = sl * 4;
    const int ch0 = grp * CPP * kStepRows + threadIdx.x / G;
    const IO *pq = row_of<IO>(a.q, b, h, 0), *pk = row_of<IO>(a.k, b, h, 0);
    const IO *pv = row_of<IO>(a.v, b, h, 0), *pd = row_of<IO>(a.delta, b, h, 0);
    const IO *pz = a.z.p ? row_of<IO>(a.z, b, h, 0) : nullptr;
    IO *po = row_of<IO>(a.o, b, h, 0);
    const bool soft = (a.flags & FALCON_SCAN_SOFTPLUS) != 0;

    auto row4 = [&](const float *p, float (&x)[4]) {
        if (V4) {
            const float4 f = *reinterpret_cast<const float4 *>(p + c0);
            x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = c0 + r < a.dk ? p[c0 + r] : 0.f;
        }
    };
    float S[kStepRows][4], A[kStepRows][4], q[4], k[4];
    const bool cols = c0 < a.dk;
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) {
        const int ch = ch0 + i * CPP;
#pragma unroll
        for (int r = 0; r < 4; ++r) { S[i][r] = 0.f; A[i][r] = 0.f; }
        if (ch < a.dv && cols) {
            row4(a.S0 + ((long long)bh * a.dv + ch) * a.dk, S[i]);
            row4(a.A + ((long long)h * a.dv + ch) * a.dk, A[i]);
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const bool in = c0 + r < a.dk;
        q[r] = in ? Io<IO>::ld(pq, c0 + r) : 0.f;
        k[r] = in ? Io<IO>::ld(pk, c0 + r) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) {
        const int ch = ch0 + i * CPP;
        const bool ok = ch < a.dv;
        const long long hc = (long long)h * a.dv + ch;
        float dt = 0.f, v = 0.f;
        if (ok) {
            v = Io<IO>::ld(pv, ch);
            dt = Io<IO>::ld(pd, ch) + (a.delta_bias ? a.delta_bias[hc] : 0.f);
            if (soft) dt = softplus(dt);
        }
        float y = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            S[i][r] = fmaf(fast_ex2(dt * (A[i][r] * kLog2e)), S[i][r], dt * v * k[r]);
            y = fmaf(S[i][r], q[r], y);
        }
#pragma unroll
        for (int m = 1; m < G; m <<= 1) y += __shfl_xor_sync(0xffffffffu, y, m);
        if (ok && cols) {
            float *to = a.S_out + ((long long)bh * a.dv + ch) * a.dk + c0;
            if (V4) *reinterpret_cast<float4 *>(to) = make_float4(S[i][0], S[i][1], S[i][2], S[i][3]);
            else
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (c0 + r < a.dk) to[r] = S[i][r];
        }
        if (ok && sl == 0) {
            if (a.D) y = fmaf(a.D[hc], v, y);
            if (pz) y *= silu(Io<IO>::ld(pz, ch));
            Io<IO>::st(po, ch, y);
        }
    }
}

template <typename IO, int ST, int SL>
cudaError_t scan_pass_t(int mode, const falcon_scan_args_t &a, const ScanWork &w, cudaStream_t s) {
    const int cpb = kScanThreads / SL;
    const int ngrp = (a.dv + cpb - 1) / cpb;
    const long long blocks = (long long)ngrp * a.B * a.H * w.nseg;
    if (blocks > kMaxGrid) return cudaErrorInvalidConfiguration;
    if (mode == kScanFull) scan_kernel<IO, ST, SL, kScanFull><<<(unsigned)blocks, kScanThreads, 0, s>>>(a, w, ngrp);
    else if (mode == kScanEnds) scan_kernel<IO, ST, SL, kScanEnds><<<(unsigned)blocks, kScanThreads, 0, s>>>(a, w, ngrp);
    else scan_kernel<IO, ST, SL, kScanBoth><<<(unsigned)blocks, kScanThreads, 0, s>>>(a, w, ngrp);
    return cudaGetLastError();
}

template <typename IO>
cudaError_t scan_pass_io(int mode, const falcon_scan_args_t &a, const ScanWork &w, cudaStream_t s) {
    if (a.dk <= 4) return scan_pass_t<IO, 4, 1>(mode, a, w, s);
    if (a.dk <= 8) return scan_pass_t<IO, 8, 1>(mode, a, w, s);
    if (a.dk <= 16) return scan_pass_t<IO, 16, 1>(mode, a, w, s);
    if (a.dk <= 32) return scan_pass_t<IO, 16, 2>(mode, a, w, s);
    if (a.dk <= 64) return scan_pass_t<IO, 16, 4>(mode, a, w, s);
    return scan_pass_t<IO, 16, 8>(mode, a, w, s);
}

template <typename IO, int G>
cudaError_t scan_step_t(const falcon_scan_args_t &a, cudaStream_t s) {
    const int per = kStepThreads / G * kStepRows;
    const int ngrp = (a.dv + per - 1) / per;
    const long long blocks = (long long)ngrp * a.B * a.H;
    if (blocks > kMaxGrid) return cudaErrorInvalidConfiguration;
    const uintptr_t any = reinterpret_cast<uintptr_t>(a.S0) | reinterpret_cast<uintptr_t>(a.S_out) | reinterpret_cast<uintptr_t>(a.A);
    if (a.dk % 4 == 0 && any % 16 == 0) scan_step_kernel<IO, G, true><<<(unsigned)blocks, kStepThreads, 0, s>>>(a, ngrp);
    else scan_step_kernel<IO, G, false><<<(unsigned)blocks, kStepThreads, 0, s>>>(a, ngrp);
    return cudaGetLastError();
}

template <typename IO>
cudaError_t scan_step_io(const falcon_scan_args_t &a, cudaStream_t s) {
    if (a.dk <= 4) return scan_step_t<IO, 1>(a, s);
    if (a.dk <= 8) return scan_step_t<IO, 2>(a, s);
    if (a.dk <= 16) return scan_step_t<IO, 4>(a, s);
    if (a.dk <= 32) return scan_step_t<IO, 8>(a, s);
    if (a.dk <= 64) return scan_step_t<IO, 16>(a, s);
    return scan_step_t<IO, 32>(a, s);
}

}  // namespace

cudaError_t launch_scan_pass(int mode, const falcon_scan_args_t &a, const ScanWork &w, cudaStream_t s) {
    return a.io_dtype == FALCON_BF16 ? scan_pass_io<__nv_bfloat16>(mode, a, w, s) : scan_pass_io<float>(mode, a, w, s);
}

// Segments: as many as fill the SMs with kWarpsWanted warps each, of at least kMinSeg tokens, and only
// where the unsplit grid has less than half of that (the split costs the exponentials twice).
ScanPlan scan_plan(const falcon_scan_args_t &a, int num_sms) {
    constexpr long long kWarpsWanted = 12, kMinSeg = 64;
    ScanPlan p;
    p.seg = a.T;
    const int sl = a.dk <= 16 ? 1 : a.dk <= 32 ? 2 : a.dk <= 64 ? 4 : 8;
    const long long bh = (long long)a.B * a.H;
    const long long warps = bh * ((a.dv * (long long)sl + kScanThreads - 1) / kScanThreads) * (kScanThreads / 32);
    const long long want = kWarpsWanted * num_sms;
    if (warps == 0 || warps * 2 > want) return p;
    long long nseg = want / warps;
    const long long most = a.T / kMinSeg;
    if (nseg > most) nseg = most;
    if (nseg < 3) return p;
    long long seg = (a.T + nseg - 1) / nseg;
    seg = (seg + kScanChunk - 1) / kScanChunk * kScanChunk;
    p.seg = (int)seg;
    p.nseg = (int)((a.T + seg - 1) / seg);
    p.bytes = (size_t)p.nseg * bh * a.dv * (a.dk + 1) * sizeof(float);
    return p;
}

cudaError_t launch_scan_fwd(const falcon_scan_args_t &a, const ScanPlan &plan, float *ws, cudaStream_t s) {
    if ((long long)a.B * a.H == 0) return cudaSuccess;
    ScanWork w{};
    w.seg = plan.seg;
    w.nseg = plan.nseg;
    if (plan.nseg > 1) {
        w.ends = ws;
        w.steps = ws + (size_t)plan.nseg * a.B * a.H * a.dv * a.dk;
        const cudaError_t e = launch_scan_pass(kScanEnds, a, w, s);
        if (e != cudaSuccess) return e;
    }
    return launch_scan_pass(kScanFull, a, w, s);
}

cudaError_t launch_scan_step(const falcon_scan_args_t &a, cudaStream_t s) {
    if ((long long)a.B * a.H == 0) return cudaSuccess;
    return a.io_dtype == FALCON_BF16 ? scan_step_io<__nv_bfloat16>(a, s) : scan_step_io<float>(a, s);
}

}  // namespace falcon
