// scan_bwd.cu -- falcon_scan_bwd: gradients of the selective scan. With a_t = exp(dt_t A) and
// dy_t = dO_t silu(z_t), G_t = dL/dS_t runs backwards, G_t = dy_t q_t^T + a_{t+1} G_{t+1}, and
//   dq_t = sum_i dy S_t;  dk_t = sum_i G_t dt v;  sum_c G_t k -> dv, ddelta;
//   W_t = G_t a_t S_{t-1}:  ddt += sum_c A W;  dA += dt W.
// Both chains are linear, so the sequence is cut into segments of kSeg tokens that need nothing from each
// other but S before and G behind them:
//   1. every segment's end state from zero, its sum of steps, and the gradient that its outputs send to
//      the state before it (sum_t prod_{s<=t} a_s dy_t q_t, one exponential for both directions);
//   2. the joins along the segments, S ascending and G descending, in place;
//   3. every segment on its own: S forward (dq, the output for dz, the states of kSub tokens kept in
//      shared memory), G backward;
//   4. sums of partial rows: dA, dD, ddelta_bias over segments and sequences, dq and dk over the blocks of
//      a head's channels, in a fixed order.
// Step 3 sums over channels (dq, dk) and over columns (dv, ddelta, dz) of the same products. A thread owns
// 4 channels x 4 columns, SL = dk / 4 lanes side by side: the first additions of either sum are fused
// multiply-adds in registers, the rest 3 to 6 shuffles (lanes_sum) for 16 entries.
#include "scan.cuh"

namespace falcon {

namespace {

constexpr int kSub = 8;              // tokens whose states are kept
constexpr int kNSub = 2;
constexpr int kSeg = kSub * kNSub;   // tokens of a segment

template <int SL> struct BwdShape {
    static constexpr int kWarps = SL == 1 ? 1 : (SL == 2 ? 2 : 4);
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kChWarp = 32 / SL * 4;          // channels of a warp
    static constexpr int kCh = kChWarp * kWarps;         // channels of a block
    static constexpr int kCols = SL * 4;                 // padded columns
    // shared memory, in floats
    static constexpr int kChan = kSeg * kCh;             // one array over (token, channel)
    static constexpr int kKq = kSeg * kCols;             // k or q
    static constexpr int kRed = kWarps * kSeg * kCols;   // a warp's part of dq or dk
    static constexpr int kHist = kSub * 16 * kThreads;
    static constexpr int kStart = (kNSub - 1) * 16 * kThreads;
    static constexpr size_t kBytes = sizeof(float) * (4 * kChan + 2 * kKq + 2 * kRed + kHist + kStart);
};

struct ScanBwdWork {
    int nseg;
    float *ends, *grads, *steps;   // as in ScanWork; ends takes the segment's part of dA in step 3
    float *dd, *db;                // [nseg][B,H,dv] parts of dD and ddelta_bias
    float *qk;                     // [2][ngrp][B,H,T,dk] parts of dq and dk (where a head has several blocks)
};

// Step 2. Thread e of (B,H,dv,dk): y = 0 walks the end states upwards and leaves the state before each
// segment, y = 1 walks the gradients downwards and leaves the gradient behind each segment.
__global__ void __launch_bounds__(256) scan_join_kernel(falcon_scan_args_t a, ScanBwdWork w, const float *dS_T, float *dS0) {
    const long long plane = (long long)a.B * a.H * a.dv * a.dk, rows = (long long)a.B * a.H * a.dv;
    const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
    if (e >= plane) return;
    const long long row = e / a.dk;
    const float A2 = a.A[e % ((long long)a.H * a.dv * a.dk)] * kLog2e;
    constexpr int U = 8;   // segments in flight
    if (blockIdx.y == 0) {
        float S = a.S0 ? a.S0[e] : 0.f;
        for (int j0 = 0; j0 < w.nseg; j0 += U) {
            float x[U], d[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (j0 + u < w.nseg) {
                    x[u] = w.ends[(j0 + u) * plane + e];
                    d[u] = w.steps[(j0 + u) * rows + row];
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (j0 + u < w.nseg) {
                    w.ends[(j0 + u) * plane + e] = S;
                    S = fmaf(fast_ex2(A2 * d[u]), S, x[u]);
                }
        }
    } else {
        float G = dS_T ? dS_T[e] : 0.f;
        for (int j0 = w.nseg - 1; j0 >= 0; j0 -= U) {
            float x[U], d[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (j0 - u >= 0) {
                    x[u] = w.grads[(j0 - u) * plane + e];
                    d[u] = w.steps[(j0 - u) * rows + row];
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (j0 - u >= 0) {
                    w.grads[(j0 - u) * plane + e] = G;
                    G = fmaf(fast_ex2(A2 * d[u]), G, x[u]);
                }
        }
        if (dS0) dS0[e] = G;
    }
}

template <typename IO, int SL>
__global__ void __launch_bounds__(BwdShape<SL>::kThreads) scan_bwd_kernel(falcon_scan_args_t a, falcon_scan_grads_t g,
                                                                          ScanBwdWork w, int ngrp) {
    typedef BwdShape<SL> Sh;
    constexpr int NT = Sh::kThreads, CH = Sh::kCh, COLS = Sh::kCols, CL = 32 / SL;
    extern __shared__ __align__(16) float sm[];
    float *sDt = sm;                    // [token][channel]: dt;  after its token: sum_c G k
    float *sDv = sDt + Sh::kChan;       // dt v;                  after its token: sum_c A W
    float *sDy = sDv + Sh::kChan;       // dy
    float *sY = sDy + Sh::kChan;        // sum_c S q
    float *sK = sY + Sh::kChan, *sQ = sK + Sh::kKq;
    float *sDq = sQ + Sh::kKq, *sDk = sDq + Sh::kRed;   // [warp][token][column]
    float *hist = sDk + Sh::kRed;       // [slot][4][thread] float4: the state before each token
    float *start = hist + Sh::kHist;    // [sub][4][thread] float4: the state before a sub-segment

    unsigned bid = blockIdx.x;
    const int grp = (int)(bid % (unsigned)ngrp);
    bid /= (unsigned)ngrp;
    const int bh = (int)(bid % (unsigned)(a.B * a.H));
    const int seg = (int)(bid / (unsigned)(a.B * a.H));
    const int b = bh / a.H, h = bh % a.H;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int sl = lane % SL, cl = lane / SL;
    const int n = seq_length(a.lengths, b, a.T);
    const int t0 = seg * kSeg, c00 = grp * CH;
    const bool soft = (a.flags & FALCON_SCAN_SOFTPLUS) != 0;
    const long long plane = (long long)a.B * a.H * a.dv * a.dk, rows = (long long)a.B * a.H * a.dv;

    const IO *pv = row_of<IO>(a.v, b, h, 0), *pd = row_of<IO>(a.delta, b, h, 0);
    const IO *pz = a.z.p ? row_of<IO>(a.z, b, h, 0) : nullptr;
    const IO *pk = row_of<IO>(a.k, b, h, 0), *pq = row_of<IO>(a.q, b, h, 0);
    const float *pg = row_of<float>(g.dO, b, h, 0);

    // ---- the segment's inputs
    for (int idx = tid; idx < Sh::kChan; idx += NT) {
        const int t = t0 + idx / CH, ch = c00 + idx % CH;
        float dt = 0.f, dtv = 0.f, dy = 0.f;
        if (t < n && ch < a.dv) {
            dt = Io<IO>::ld(pd, t * a.delta.st + ch) + (a.delta_bias ? a.delta_bias[(long long)h * a.dv + ch] : 0.f);
            if (soft) dt = softplus(dt);
            dtv = dt * Io<IO>::ld(pv, t * a.v.st + ch);
            dy = pg[t * g.dO.st + ch];
            if (pz) dy *= silu(Io<IO>::ld(pz, t * a.z.st + ch));
        }
        sDt[idx] = dt;
        sDv[idx] = dtv;
        sDy[idx] = dy;
    }
    for (int idx = tid; idx < Sh::kKq; idx += NT) {
        const int t = t0 + idx / COLS, c = idx % COLS;
        const bool in = t < n && c < a.dk;
        sK[idx] = in ? Io<IO>::ld(pk, t * a.k.st + c) : 0.f;
        sQ[idx] = in ? Io<IO>::ld(pq, t * a.q.st + c) : 0.f;
    }

    // ---- this thread's 4 channels x 4 columns
    const int lc = warp * Sh::kChWarp + cl * 4;   // first channel in the block
    float A2[4][4], S[4][4], G[4][4], dA[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int ch = c00 + lc + i, c = sl * 4 + s;
            const bool ok = ch < a.dv && c < a.dk;
            const long long at = ((long long)bh * a.dv + ch) * a.dk + c;
            A2[i][s] = ok ? a.A[((long long)h * a.dv + ch) * a.dk + c] * kLog2e : 0.f;
            S[i][s] = ok ? w.ends[seg * plane + at] : 0.f;
            G[i][s] = ok ? w.grads[seg * plane + at] : 0.f;
            dA[i][s] = 0.f;
        }
    __syncthreads();

    auto keep = [&](float *to, int slot) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            reinterpret_cast<float4 *>(to)[(slot * 4 + i) * NT + tid] = make_float4(S[i][0], S[i][1], S[i][2], S[i][3]);
    };
    auto four = [](const float *p, float (&x)[4]) {
        const float4 f = *reinterpret_cast<const float4 *>(p);
        x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
    };
    auto advance = [&](int t) {   // S_{t-1} -> S_t
        float dt[4], dtv[4], k[4];
        four(sDt + t * CH + lc, dt);
        four(sDv + t * CH + lc, dtv);
        four(sK + t * COLS + sl * 4, k);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int s = 0; s < 4; ++s) S[i][s] = fmaf(fast_ex2(dt[i] * A2[i][s]), S[i][s], dtv[i] * k[s]);
    };
    bool write;

    // ---- forward
#pragma unroll 1
    for (int t = 0; t < kSeg; ++t) {
        if (t % kSub == 0 && t / kSub < kNSub - 1) keep(start, t / kSub);
        if (t >= kSeg - kSub) keep(hist, t - (kSeg - kSub));
        advance(t);
        float q[4], dy[4], y[4], dq[4];
        four(sQ + t * COLS + sl * 4, q);
        four(sDy + t * CH + lc, dy);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[i] = 0.f;
            dq[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                y[i] = fmaf(S[i][s], q[s], y[i]);
                dq[s] = fmaf(S[i][s], dy[i], dq[s]);
            }
        const int iy = lanes_sum<4, SL, 1>(y, lane, write);
        if (write)
#pragma unroll
            for (int i = 0; i < (SL >= 4 ? 1 : 4 / SL); ++i) sY[t * CH + lc + iy + i] = y[i];
        const int iq = lanes_sum<4, CL, SL>(dq, lane, write);
        if (write)
#pragma unroll
            for (int s = 0; s < (CL >= 4 ? 1 : 4 / CL); ++s) sDq[(warp * kSeg + t) * COLS + sl * 4 + iq + s] = dq[s];
    }

    // ---- backward
#pragma unroll 1
    for (int sub = kNSub - 1; sub >= 0; --sub) {
        if (sub < kNSub - 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 f = reinterpret_cast<const float4 *>(start)[(sub * 4 + i) * NT + tid];
                S[i][0] = f.x; S[i][1] = f.y; S[i][2] = f.z; S[i][3] = f.w;
            }
#pragma unroll 1
            for (int j = 0; j < kSub; ++j) {
                keep(hist, j);
                if (j < kSub - 1) advance(sub * kSub + j);
            }
        }
#pragma unroll 1
        for (int j = kSub - 1; j >= 0; --j) {
            const int t = sub * kSub + j;
            float dt[4], dtv[4], dy[4], k[4], q[4], dk[4], ch[8];
            four(sDt + t * CH + lc, dt);
            four(sDv + t * CH + lc, dtv);
            four(sDy + t * CH + lc, dy);
            four(sK + t * COLS + sl * 4, k);
            four(sQ + t * COLS + sl * 4, q);
#pragma unroll
            for (int i = 0; i < 4; ++i) dk[i] = ch[i] = ch[4 + i] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float p[4];
                four(hist + 4 * ((j * 4 + i) * NT + tid), p);
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const float gs = fmaf(dy[i], q[s], G[i][s]);
                    ch[i] = fmaf(gs, k[s], ch[i]);
                    dk[s] = fmaf(gs, dtv[i], dk[s]);
                    G[i][s] = gs * fast_ex2(dt[i] * A2[i][s]);
                    const float W = G[i][s] * p[s];
                    ch[4 + i] = fmaf(A2[i][s], W, ch[4 + i]);
                    dA[i][s] = fmaf(dt[i], W, dA[i][s]);
                }
            }
            const int ik = lanes_sum<4, CL, SL>(dk, lane, write);
            if (write)
#pragma unroll
                for (int s = 0; s < (CL >= 4 ? 1 : 4 / CL); ++s) sDk[(warp * kSeg + t) * COLS + sl * 4 + ik + s] = dk[s];
            const int ic = lanes_sum<8, SL, 1>(ch, lane, write);   // the shuffles follow every lane's reads of this token
            __syncwarp();
            if (write)
#pragma unroll
                for (int i = 0; i < (SL >= 8 ? 1 : 8 / SL); ++i) {
                    const int m = ic + i;   // 0..3: sum G k, 4..7: sum A W (in units of log2 e)
                    if (m < 4) sDt[t * CH + lc + m] = ch[i];
                    else sDv[t * CH + lc + m - 4] = ch[i] * kLn2;
                }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int ch = c00 + lc + i, c = sl * 4 + s;
            if (ch < a.dv && c < a.dk) w.ends[seg * plane + ((long long)bh * a.dv + ch) * a.dk + c] = dA[i][s];
        }
    __syncthreads();

    // ---- gradients of the channels; thread tid keeps the channels tid, tid + NT, ..
    for (int cc = tid; cc < CH; cc += NT) {
        const int ch = c00 + cc;
        if (ch >= a.dv) continue;
        const long long hc = (long long)h * a.dv + ch;
        const float skip = a.D ? a.D[hc] : 0.f, bias = a.delta_bias ? a.delta_bias[hc] : 0.f;
        float dd = 0.f, db = 0.f;
#pragma unroll 4
        for (int j = 0; j < kSeg; ++j) {
            const int t = t0 + j;
            if (t >= a.T) break;
            float dv = 0.f, ddl = 0.f, dz = 0.f;
            if (t < n) {
                const float gk = sDt[j * CH + cc], aw = sDv[j * CH + cc], dy = sDy[j * CH + cc];
                const float raw = Io<IO>::ld(pd, t * a.delta.st + ch) + bias;
                const float v = Io<IO>::ld(pv, t * a.v.st + ch);
                const float dt = soft ? softplus(raw) : raw;
                dv = fmaf(dt, gk, skip * dy);
                ddl = fmaf(v, gk, aw);
                if (soft) ddl *= sigmoid(raw);
                if (pz) {
                    const float z = Io<IO>::ld(pz, t * a.z.st + ch);
                    dz = pg[t * g.dO.st + ch] * fmaf(skip, v, sY[j * CH + cc]) * silu_grad(z);
                }
                dd = fmaf(dy, v, dd);
                db += ddl;
            }
            row_of<float>(g.dv, b, h, t)[ch] = dv;
            row_of<float>(g.ddelta, b, h, t)[ch] = ddl;
            if (pz && g.dz.p) row_of<float>(g.dz, b, h, t)[ch] = dz;
        }
        w.dd[seg * rows + (long long)bh * a.dv + ch] = dd;
        w.db[seg * rows + (long long)bh * a.dv + ch] = db;
    }
    // ---- dq and dk: the warps' parts
    for (int idx = tid; idx < Sh::kKq; idx += NT) {
        const int j = idx / COLS, c = idx % COLS, t = t0 + j;
        if (t >= a.T || c >= a.dk) continue;
        float dq = 0.f, dk = 0.f;
#pragma unroll
        for (int x = 0; x < Sh::kWarps; ++x) {
            dq += sDq[(x * kSeg + j) * COLS + c];
            dk += sDk[(x * kSeg + j) * COLS + c];
        }
        if (ngrp == 1) {
            row_of<float>(g.dq, b, h, t)[c] = dq;
            row_of<float>(g.dk, b, h, t)[c] = dk;
        } else {
            const long long part = (long long)a.B * a.H * a.T * a.dk;
            const long long at = grp * part + ((long long)bh * a.T + t) * a.dk + c;
            w.qk[at] = dq;
            w.qk[ngrp * part + at] = dk;
        }
    }
}

// dq and dk of a head whose channels are in several blocks.
__global__ void __launch_bounds__(256) scan_qk_sum_kernel(falcon_scan_args_t a, falcon_scan_grads_t g, const float *qk, int ngrp) {
    const long long part = (long long)a.B * a.H * a.T * a.dk;
    const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
    if (e >= part) return;
    float s = 0.f;
    const float *p = qk + blockIdx.y * ngrp * part + e;
#pragma unroll 4
    for (int i = 0; i < ngrp; ++i) s += p[i * part];
    const int c = (int)(e % a.dk);
    const long long r = e / a.dk;
    const int t = (int)(r % a.T);
    const long long bh = r / a.T;
    const falcon_view_t &to = blockIdx.y ? g.dk : g.dq;
    row_of<float>(to, bh / a.H, bh % a.H, t)[c] = s;
}

int bwd_lanes(int dk) {
    int sl = 1;
    while (sl * 4 < dk) sl *= 2;
    return sl;
}

int bwd_channels(int sl) {
    switch (sl) {
        case 1: return BwdShape<1>::kCh;
        case 2: return BwdShape<2>::kCh;
        case 4: return BwdShape<4>::kCh;
        case 8: return BwdShape<8>::kCh;
        case 16: return BwdShape<16>::kCh;
        default: return BwdShape<32>::kCh;
    }
}

struct BwdSizes {
    int nseg, ngrp;
    long long plane, rows, qk;   // floats of one segment's states, of its channels, of all parts of dq and dk
};

BwdSizes bwd_sizes(const falcon_scan_args_t &a) {
    BwdSizes z;
    z.nseg = (a.T + kSeg - 1) / kSeg;
    const int ch = bwd_channels(bwd_lanes(a.dk));
    z.ngrp = (a.dv + ch - 1) / ch;
    z.rows = (long long)a.B * a.H * a.dv;
    z.plane = z.rows * a.dk;
    z.qk = z.ngrp > 1 ? 2LL * z.ngrp * a.B * a.H * a.T * a.dk : 0;
    return z;
}

template <typename IO, int SL>
cudaError_t scan_bwd_t(const falcon_scan_args_t &a, const falcon_scan_grads_t &g, const ScanBwdWork &w, int ngrp, cudaStream_t s) {
    const long long blocks = (long long)ngrp * a.B * a.H * w.nseg;
    if (blocks > kMaxGrid) return cudaErrorInvalidConfiguration;
    const size_t smem = BwdShape<SL>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(scan_bwd_kernel<IO, SL>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    scan_bwd_kernel<IO, SL><<<(unsigned)blocks, BwdShape<SL>::kThreads, smem, s>>>(a, g, w, ngrp);
    return cudaGetLastError();
}

template <typename IO>
cudaError_t scan_bwd_io(const falcon_scan_args_t &a, const falcon_scan_grads_t &g, const ScanBwdWork &w, int ngrp, cudaStream_t s) {
    switch (bwd_lanes(a.dk)) {
        case 1: return scan_bwd_t<IO, 1>(a, g, w, ngrp, s);
        case 2: return scan_bwd_t<IO, 2>(a, g, w, ngrp, s);
        case 4: return scan_bwd_t<IO, 4>(a, g, w, ngrp, s);
        case 8: return scan_bwd_t<IO, 8>(a, g, w, ngrp, s);
        case 16: return scan_bwd_t<IO, 16>(a, g, w, ngrp, s);
        default: return scan_bwd_t<IO, 32>(a, g, w, ngrp, s);
    }
}

}  // namespace

size_t scan_bwd_workspace(const falcon_scan_args_t &a) {
    const BwdSizes z = bwd_sizes(a);
    return sizeof(float) * (size_t)(z.nseg * (2 * z.plane + 3 * z.rows) + z.qk);
}

cudaError_t launch_scan_bwd(const falcon_scan_args_t &a, const falcon_scan_grads_t &g, float *ws, cudaStream_t s) {
    if (a.H == 0) return cudaSuccess;
    const BwdSizes z = bwd_sizes(a);
    ScanBwdWork w{};
    w.nseg = z.nseg;
    w.ends = ws;
    w.grads = w.ends + z.nseg * z.plane;
    w.steps = w.grads + z.nseg * z.plane;
    w.dd = w.steps + z.nseg * z.rows;
    w.db = w.dd + z.nseg * z.rows;
    w.qk = w.db + z.nseg * z.rows;
    cudaError_t e;
    if (a.B > 0) {
        if (z.nseg > 0) {
            ScanWork p{};
            p.seg = kSeg;
            p.nseg = z.nseg;
            p.ends = w.ends;
            p.grads = w.grads;
            p.steps = w.steps;
            p.dO = g.dO;
            e = launch_scan_pass(kScanBoth, a, p, s);
            if (e != cudaSuccess) return e;
        }
        const long long jb = (z.plane + 255) / 256;
        if (jb > kMaxGrid) return cudaErrorInvalidConfiguration;
        scan_join_kernel<<<dim3((unsigned)jb, 2), 256, 0, s>>>(a, w, g.dS_T, g.dS0);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        if (z.nseg > 0) {
            e = a.io_dtype == FALCON_BF16 ? scan_bwd_io<__nv_bfloat16>(a, g, w, z.ngrp, s) : scan_bwd_io<float>(a, g, w, z.ngrp, s);
            if (e != cudaSuccess) return e;
            if (z.ngrp > 1) {
                const long long blocks = ((long long)a.B * a.H * a.T * a.dk + 255) / 256;
                if (blocks > kMaxGrid) return cudaErrorInvalidConfiguration;
                scan_qk_sum_kernel<<<dim3((unsigned)blocks, 2), 256, 0, s>>>(a, g, w.qk, z.ngrp);
                e = cudaGetLastError();
                if (e != cudaSuccess) return e;
            }
        }
    }
    const long long hrows = (long long)a.H * a.dv, hplane = hrows * a.dk;
    const SumJob jobs[3] = {{w.ends, hplane, hplane, g.dA}, {w.dd, hrows, hrows, g.dD}, {w.db, hrows, hrows, g.ddelta_bias}};
    return launch_column_sums(jobs, 3, (long long)z.nseg * a.B, s);
}

}  // namespace falcon
