// scan_bwd.cu -- falcon_scan_bwd: gradients of the selective scan. With a_t = exp(dt_t A) and
// dy_t = dO_t silu(z_t), G_t = dL/dS_t runs backwards, G_t = dy_t q_t^T + a_{t+1} G_{t+1}, and
//   dq_t = sum_i dy S_t;  dk_t = sum_i G_t dt v;  sum_c G_t k -> dv, ddelta;
//   W_t = G_t a_t S_{t-1}:  ddt += sum_c A W;  dA += dt W.
// Both chains are linear, so the sequence is cut into walks of a few segments of kSeg tokens, and walks need nothing
// from each other but S before and G behind them:
//   1. from a zero state before each walk: the state before each of its segments, its end state and sum of steps, and
//      the gradient that its outputs send to the state before it (sum_t prod_{s<=t} a_s dy_t q_t, one exponential for
//      both directions);
//   2. the joins along the walks, S ascending and G descending, in place;
//   3. every walk on its own, its segments from the last to the first, G handed down: S forward from the segment's
//      state (dq, the output for dz, the state at every kSub-th token kept in shared memory), then, kSub tokens at a
//      time, their states again into registers and G backward;
//   4. sums of partial rows: dA, dD, ddelta_bias over walks and sequences, dq and dk over the blocks of a head's
//      channels, in a fixed order.
// A sequence that is one walk needs no joins, one that is one segment no step 1 either.
// Step 3 sums over channels (dq, dk) and over columns (dv, ddelta, dz) of the same products. A thread owns
// 4 channels x 4 columns, SL = dk / 4 lanes side by side: the first additions of either sum are fused
// multiply-adds in registers, the rest 3 to 6 shuffles (lanes_sum) for 16 entries.
// B2 H16 T2048 dv128 dk16, bf16, 332 us. One launch at a time, each from cold caches: 77 us for step 1, 12 for the joins,
// 261 for step 3, 6 for the sums (356 in all). Step 3 is bound by latency at 11 warps an SM (168 registers, half of them
// states, 100 bytes spilled; 70 KB of shared memory): its instruction slots are at half, the exponential unit at 39%.
// dk 4, 8 and 64 of the same tensors: 463, 309 and 1826 us (blocks of one and two warps, and 128 channels' products over
// 64 columns). Taken out one at a time, the channels' gradients at a segment's end were 55 us of it
// (45 since they are formed two tokens an instruction), the shuffled sums 28, the exponentials 19.
#include "scan.cuh"

namespace falcon {

namespace {

constexpr int kSub = 4;              // tokens whose states are kept in registers
constexpr int kNSub = 4;
constexpr int kSeg = kSub * kNSub;   // tokens of a segment

template <int SL> struct BwdShape {
    static constexpr int kWarps = SL == 1 ? 1 : (SL == 2 ? 2 : 4);
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kChWarp = 32 / SL * 4;          // channels of a warp
    static constexpr int kCh = kChWarp * kWarps;         // channels of a block
    static constexpr int kPer = kCh / kThreads > 0 ? kCh / kThreads : 1;   // channels whose gradients a thread forms
    static constexpr int kCols = SL * 4;                 // padded columns
    // shared memory, in floats
    static constexpr int kChan = kSeg * kCh;             // one array over (token, channel)
    static constexpr int kKq = kSeg * kCols;             // k or q
    static constexpr int kRed = kWarps * kSeg * kCols;   // a warp's part of dq or dk
    static constexpr int kStart = (kNSub - 1) * 16 * kThreads;
    static constexpr size_t kBytes = sizeof(float) * (4 * kChan + 4 * kKq + 2 * kRed + kStart);
};

struct ScanBwdWork {
    ScanWork s;                    // seg = kSeg; wends and wgrads hold the joined states after step 2
    float *dA;                     // [nwalk][B][H,dv,dk] parts
    float *dd, *db;                // [nwalk][B][H,dv] parts of dD and ddelta_bias
    float *qk;                     // [2][ngrp][B,H,T,dk] parts of dq and dk (where a head has several blocks)
};

// Step 2. A thread per column of a channel's state: y = 0 walks the end states upwards and leaves the state
// before each walk, y = 1 goes over the gradients downwards and leaves the gradient behind each walk.
__global__ void __launch_bounds__(256) scan_join_kernel(falcon_scan_args_t a, ScanWork w, int cols, const float *dS_T, float *dS0) {
    const long long rows = (long long)a.B * a.H * a.dv;
    const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long row = e / cols;
    const int c = (int)(e % cols);
    if (row >= rows || c >= a.dk) return;
    const float A2 = decay_rate(a.A[row % ((long long)a.H * a.dv) * a.dk + c]);
    const float *steps = w.wsteps + row * w.nwalk;
    constexpr int U = 16;   // walks in flight
    if (blockIdx.y == 0) {
        float *x = w.wends + row * w.nwalk * cols + c;
        float S = a.S0 ? a.S0[row * a.dk + c] : 0.f;
        for (int j0 = 0; j0 < w.nwalk; j0 += U) {
            float y[U], d[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (j0 + u < w.nwalk) {
                    y[u] = x[(long long)(j0 + u) * cols];
                    d[u] = steps[j0 + u];
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (j0 + u < w.nwalk) {
                    x[(long long)(j0 + u) * cols] = S;
                    S = fmaf(fast_ex2(A2 * d[u]), S, y[u]);
                }
        }
    } else {
        float *x = w.wgrads + row * w.nwalk * cols + c;
        float G = dS_T ? dS_T[row * a.dk + c] : 0.f;
        for (int j0 = w.nwalk - 1; j0 >= 0; j0 -= U) {
            float y[U], d[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (j0 - u >= 0) {
                    y[u] = x[(long long)(j0 - u) * cols];
                    d[u] = steps[j0 - u];
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (j0 - u >= 0) {
                    x[(long long)(j0 - u) * cols] = G;
                    G = fmaf(fast_ex2(A2 * d[u]), G, y[u]);
                }
        }
        if (dS0) dS0[row * a.dk + c] = G;
    }
}

// ONE: the sequence is a single walk, so that its states are the given ones and its gradient of the initial state the
// answer, and a segment's sub-segments without tokens are passed over (B3 H16 T5 dk32 dv2048: 117 us in all against 373).
// Compiled on its own, because the registers it takes cost the other 355 us instead of 332 for the case above.
template <typename IO, int SL, bool ONE>
__global__ void __launch_bounds__(BwdShape<SL>::kThreads, BwdShape<SL>::kWarps == 4 ? 3 : 1)
scan_bwd_kernel(falcon_scan_args_t a, falcon_scan_grads_t g, ScanBwdWork w, int ngrp) {
    typedef BwdShape<SL> Sh;
    typedef Pack<IO, 1> P;
    constexpr int NT = Sh::kThreads, CH = Sh::kCh, COLS = Sh::kCols, CL = 32 / SL;
    constexpr int EU = 16;   // tokens whose loads are in flight at a segment's end
    extern __shared__ __align__(16) float sm[];
    float *sDt = sm;                    // [token][channel]: dt;  after its token: sum_c G k
    float *sDv = sDt + Sh::kChan;       // dt v;                  after its token: sum_c A W
    float *sDy = sDv + Sh::kChan;       // dy
    float *sY = sDy + Sh::kChan;        // sum_c S q
    float *sK = sY + Sh::kChan, *sQ = sK + 2 * Sh::kKq;     // [token][column], every value twice: a pair's factor
    float *sDq = sQ + 2 * Sh::kKq, *sDk = sDq + Sh::kRed;   // [warp][token][column]
    float *start = sDk + Sh::kRed;      // [sub][4][thread] float4: the state before a sub-segment

    unsigned bid = blockIdx.x;
    const int grp = (int)(bid % (unsigned)ngrp);
    bid /= (unsigned)ngrp;
    const int bh = (int)(bid % (unsigned)(a.B * a.H));
    const int walk = (int)(bid / (unsigned)(a.B * a.H));
    const int b = bh / a.H, h = bh % a.H;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int sl = lane % SL, cl = lane / SL;
    const int n = seq_length(a.lengths, b, a.T);
    const int c00 = grp * CH;
    const bool soft = (a.flags & FALCON_SCAN_SOFTPLUS) != 0;

    // this thread's 4 channels x 4 columns, as pairs of channels: factors of a channel (dt, dt v, dy) are pairs as
    // they lie, factors of a column (k, q) pairs of one value, and sums over columns need no last addition
    const int lc = warp * Sh::kChWarp + cl * 4;   // first channel in the block
    f32x2 A2[2][4], S[2][4], G[2][4], dA[2][4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int c = sl * 4 + s;
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int ch = c00 + lc + i;
            x[i] = ch < a.dv && c < a.dk ? decay_rate(a.A[((long long)h * a.dv + ch) * a.dk + c]) : 0.f;
        }
        A2[0][s] = pack2(x[0], x[1]);
        A2[1][s] = pack2(x[2], x[3]);
        dA[0][s] = dA[1][s] = 0ull;
    }
    float dd[Sh::kPer], db[Sh::kPer], skip[Sh::kPer], bias[Sh::kPer];   // of the channels tid, tid + NT, ..
#pragma unroll
    for (int m = 0; m < Sh::kPer; ++m) {
        const int ch = c00 + tid + m * NT;
        const bool ok = tid + m * NT < CH && ch < a.dv;
        dd[m] = db[m] = 0.f;
        skip[m] = ok && a.D ? a.D[(long long)h * a.dv + ch] : 0.f;
        bias[m] = ok && a.delta_bias ? a.delta_bias[(long long)h * a.dv + ch] : 0.f;
    }

    auto advance = [&](int t) {   // S_{t-1} -> S_t
        f32x2 dt[2], dtv[2], k[4];
        load_pairs(sDt + t * CH + lc, dt[0], dt[1]);
        load_pairs(sDv + t * CH + lc, dtv[0], dtv[1]);
        load_pairs(sK + (t * COLS + sl * 4) * 2, k[0], k[1]);
        load_pairs(sK + (t * COLS + sl * 4) * 2 + 4, k[2], k[3]);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int s = 0; s < 4; ++s) S[i][s] = fma2(ex2_2(mul2(dt[i], A2[i][s])), S[i][s], mul2(dtv[i], k[s]));
    };

    // a row of (B,H,dv,dk): this thread's columns
    auto given = [&](const float *s, long long row, f32x2 (&o)[2]) {
        float v[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = s && sl * 4 + c < a.dk ? s[row * a.dk + sl * 4 + c] : 0.f;
        o[0] = pack2(v[0], v[1]);
        o[1] = pack2(v[2], v[3]);
    };
    const int seg0 = walk * w.s.walk, seg1 = min(seg0 + w.s.walk, w.s.nseg);
#pragma unroll 1
    for (int seg = seg1 - 1; seg >= seg0; --seg) {
        const int t0 = seg * kSeg;
        const int here = min(max(n - t0, 0), kSeg), rows = min(a.T - t0, kSeg);   // tokens of the sequence; of the arrays
        const int subs = ONE ? max((here + kSub - 1) / kSub, 1) : kNSub;   // sub-segments to go through
        // ---- the segment's states (a row of each channel), then its inputs
        {
            f32x2 x[4][2], y[4][2], u[4][2];
            float pre[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int ch = c00 + lc + i;
                x[i][0] = x[i][1] = y[i][0] = y[i][1] = u[i][0] = u[i][1] = 0ull;
                pre[i] = 0.f;
                if (ch < a.dv) {
                    const long long row = (long long)bh * a.dv + ch;
                    if (!ONE || w.s.nseg > 1) {   // a single one starts its walk
                        load_pairs(w.s.ends + (row * w.s.nseg + seg) * COLS + sl * 4, x[i][0], x[i][1]);
                        pre[i] = w.s.steps[row * w.s.nseg + seg];
                    }
                    if (ONE) {
                        given(a.S0, row, y[i]);
                        if (seg == seg1 - 1) given(g.dS_T, row, u[i]);
                    } else {
                        load_pairs(w.s.wends + (row * w.s.nwalk + walk) * COLS + sl * 4, y[i][0], y[i][1]);
                        if (seg == seg1 - 1) load_pairs(w.s.wgrads + (row * w.s.nwalk + walk) * COLS + sl * 4, u[i][0], u[i][1]);
                    }
                }
            }
            const IO *pk = row_of<IO>(a.k, b, h, t0), *pq = row_of<IO>(a.q, b, h, t0);
            for (int idx = tid; idx < Sh::kKq; idx += NT) {
                const int j = idx / COLS, c = idx % COLS;
                const bool in = j < here && c < a.dk;
                const float kk = in ? Io<IO>::ld(pk, j * a.k.st + c) : 0.f;
                const float qq = in ? Io<IO>::ld(pq, j * a.q.st + c) : 0.f;
                reinterpret_cast<float2 *>(sK)[idx] = make_float2(kk, kk);
                reinterpret_cast<float2 *>(sQ)[idx] = make_float2(qq, qq);
            }
            // thread tid stages the channels whose gradients it forms
#pragma unroll
            for (int m = 0; m < Sh::kPer; ++m) {
                const int cc = tid + m * NT, ch = c00 + cc;
                if (cc >= CH) continue;
                const bool ok = ch < a.dv;
                const IO *pv = row_of<IO>(a.v, b, h, t0) + ch, *pd = row_of<IO>(a.delta, b, h, t0) + ch;
                const IO *pz = a.z.p ? row_of<IO>(a.z, b, h, t0) + ch : nullptr;
                const float *pg = row_of<float>(g.dO, b, h, t0) + ch;
                constexpr int U = 8;
#pragma unroll 1
                for (int j0 = 0; j0 < kSeg; j0 += U) {
                    typename P::raw rv[U], rd[U], rz[U];
                    float rg[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const bool in = ok && j0 + u < here;
                        rv[u] = rd[u] = rz[u] = P::zero();
                        rg[u] = 0.f;
                        if (in) {
                            rv[u] = P::ld(pv);
                            rd[u] = P::ld(pd);
                            if (pz) rz[u] = P::ld(pz);
                            rg[u] = *pg;
                        }
                        pv += a.v.st;
                        pd += a.delta.st;
                        if (pz) pz += a.z.st;
                        pg += g.dO.st;
                    }
#pragma unroll
                    for (int u = 0; u < U; u += 2) {
                        float *to = sDt + (j0 + u) * CH + cc;   // the arrays lie kChan apart
                        float d0 = Io<IO>::cvt(rd[u]) + bias[m], d1 = Io<IO>::cvt(rd[u + 1]) + bias[m];
                        if (soft) unpack2(softplus2(pack2(d0, d1)), d0, d1);
                        if (!(ok && j0 + u < here)) d0 = 0.f;
                        if (!(ok && j0 + u + 1 < here)) d1 = 0.f;
                        float g0 = rg[u], g1 = rg[u + 1];
                        if (pz) unpack2(mul2(pack2(g0, g1), silu2(pack2(Io<IO>::cvt(rz[u]), Io<IO>::cvt(rz[u + 1])))), g0, g1);
                        to[0] = d0;
                        to[CH] = d1;
                        to[Sh::kChan] = d0 * Io<IO>::cvt(rv[u]);
                        to[Sh::kChan + CH] = d1 * Io<IO>::cvt(rv[u + 1]);
                        to[2 * Sh::kChan] = g0;
                        to[2 * Sh::kChan + CH] = g1;
                    }
                }
            }
            // rows of channels to pairs of channels; S = the walk's own part + the decayed state before the walk
            auto turned = [](const f32x2 (&r)[4][2], f32x2 (&o)[2][4]) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        float p0, p1, r0, r1;
                        unpack2(r[2 * i][s], p0, p1);
                        unpack2(r[2 * i + 1][s], r0, r1);
                        o[i][2 * s] = pack2(p0, r0);
                        o[i][2 * s + 1] = pack2(p1, r1);
                    }
            };
            f32x2 before[2][4];
            turned(x, S);
            turned(y, before);
            if (seg == seg1 - 1) turned(u, G);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const f32x2 p2 = pack2(pre[2 * i], pre[2 * i + 1]);
#pragma unroll
                for (int s = 0; s < 4; ++s) S[i][s] = fma2(ex2_2(mul2(p2, A2[i][s])), before[i][s], S[i][s]);
            }
        }
        __syncthreads();

        // ---- forward, all but the last sub-segment
        auto outputs = [&](int t) {   // y_t and this warp's part of dq_t from S_t
            f32x2 q[4], dy[2];
            float y[4], dq[4];
            load_pairs(sQ + (t * COLS + sl * 4) * 2, q[0], q[1]);
            load_pairs(sQ + (t * COLS + sl * 4) * 2 + 4, q[2], q[3]);
            load_pairs(sDy + t * CH + lc, dy[0], dy[1]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f32x2 y2 = mul2(S[i][0], q[0]);
#pragma unroll
                for (int s = 1; s < 4; ++s) y2 = fma2(S[i][s], q[s], y2);
                unpack2(y2, y[2 * i], y[2 * i + 1]);
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) dq[s] = sum2(fma2(S[1][s], dy[1], mul2(S[0][s], dy[0])));
            bool write;
            const int iy = lanes_sum<4, SL, 1>(y, lane, write);
            if (write)
#pragma unroll
                for (int i = 0; i < (SL >= 4 ? 1 : 4 / SL); ++i) sY[t * CH + lc + iy + i] = y[i];
            const int iq = lanes_sum<4, CL, SL>(dq, lane, write);
            if (write)
#pragma unroll
                for (int s = 0; s < (CL >= 4 ? 1 : 4 / CL); ++s) sDq[(warp * kSeg + t) * COLS + sl * 4 + iq + s] = dq[s];
        };
#pragma unroll 1
        for (int t = 0; t < (subs - 1) * kSub; ++t) {
            if (t % kSub == 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    store_pairs(start + ((t / kSub * 4 + i) * NT + tid) * 4, S[i / 2][i % 2 * 2], S[i / 2][i % 2 * 2 + 1]);
            }
            advance(t);
            outputs(t);
        }

        // ---- sub-segment by sub-segment from the end: the states before its tokens, then backward
#pragma unroll 1
        for (int sub = subs - 1; sub >= 0; --sub) {
            f32x2 before[kSub][2][4];
            const bool last = sub == subs - 1;    // its forward pass is still to come
            if (!last) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    load_pairs(start + ((sub * 4 + i) * NT + tid) * 4, S[i / 2][i % 2 * 2], S[i / 2][i % 2 * 2 + 1]);
            }
#pragma unroll
            for (int j = 0; j < kSub; ++j) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int s = 0; s < 4; ++s) before[j][i][s] = S[i][s];
                if (j < kSub - 1 || last) advance(sub * kSub + j);
                if (last) outputs(sub * kSub + j);
            }
#pragma unroll
            for (int j = kSub - 1; j >= 0; --j) {
                const int t = sub * kSub + j;
                f32x2 dt[2], dtv[2], dy[2], k[4], q[4];
                float dk[4], ch[8];
                bool write;
                load_pairs(sDt + t * CH + lc, dt[0], dt[1]);
                load_pairs(sDv + t * CH + lc, dtv[0], dtv[1]);
                load_pairs(sDy + t * CH + lc, dy[0], dy[1]);
                load_pairs(sK + (t * COLS + sl * 4) * 2, k[0], k[1]);
                load_pairs(sK + (t * COLS + sl * 4) * 2 + 4, k[2], k[3]);
                load_pairs(sQ + (t * COLS + sl * 4) * 2, q[0], q[1]);
                load_pairs(sQ + (t * COLS + sl * 4) * 2 + 4, q[2], q[3]);
                f32x2 gk[2] = {0ull, 0ull}, aw[2] = {0ull, 0ull};
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    f32x2 dk2 = 0ull;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const f32x2 gs = fma2(dy[i], q[s], G[i][s]);
                        gk[i] = fma2(gs, k[s], gk[i]);
                        dk2 = fma2(gs, dtv[i], dk2);
                        G[i][s] = mul2(gs, ex2_2(mul2(dt[i], A2[i][s])));
                        const f32x2 W = mul2(G[i][s], before[j][i][s]);
                        aw[i] = fma2(A2[i][s], W, aw[i]);
                        dA[i][s] = fma2(dt[i], W, dA[i][s]);
                    }
                    dk[s] = sum2(dk2);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    unpack2(gk[i], ch[2 * i], ch[2 * i + 1]);
                    unpack2(aw[i], ch[4 + 2 * i], ch[5 + 2 * i]);
                }
                const int ik = lanes_sum<4, CL, SL>(dk, lane, write);
                if (write)
#pragma unroll
                    for (int s = 0; s < (CL >= 4 ? 1 : 4 / CL); ++s) sDk[(warp * kSeg + t) * COLS + sl * 4 + ik + s] = dk[s];
                const int ic = lanes_sum<8, SL, 1>(ch, lane, write);
                __syncwarp();   // every lane has read this token's dt and dt v
                if (write)
#pragma unroll
                    for (int i = 0; i < (SL >= 8 ? 1 : 8 / SL); ++i) {
                        const int m = ic + i;   // 0..3: sum G k, 4..7: sum A W (in units of log2 e)
                        if (m < 4) sDt[t * CH + lc + m] = ch[i];
                        else sDv[t * CH + lc + m - 4] = ch[i] * kLn2;
                    }
            }
        }
        __syncthreads();

        // ---- gradients of the channels, two tokens an instruction; the loads of all tokens are in flight together
#pragma unroll
        for (int m = 0; m < Sh::kPer; ++m) {
            const int cc = tid + m * NT, ch = c00 + cc;
            if (cc >= CH || ch >= a.dv) continue;
            const IO *pv = row_of<IO>(a.v, b, h, t0) + ch, *pd = row_of<IO>(a.delta, b, h, t0) + ch;
            float *ov = row_of<float>(g.dv, b, h, t0) + ch, *od = row_of<float>(g.ddelta, b, h, t0) + ch;
            const bool has_dz = a.z.p && g.dz.p;
            const IO *pz = has_dz ? row_of<IO>(a.z, b, h, t0) + ch : nullptr;
            const float *pg = row_of<float>(g.dO, b, h, t0) + ch;
            float *oz = has_dz ? row_of<float>(g.dz, b, h, t0) + ch : nullptr;
            typename P::raw rv[EU], rd[EU], rz[EU];
            float rg[EU];
#pragma unroll 1
            for (int j0 = 0; j0 < rows; j0 += EU) {
#pragma unroll
                for (int u = 0; u < EU; ++u) {
                    rv[u] = rd[u] = rz[u] = P::zero();
                    rg[u] = 0.f;
                    if (j0 + u < here) {
                        rv[u] = P::ld(pv);
                        rd[u] = P::ld(pd);
                        if (has_dz) {
                            rz[u] = P::ld(pz);
                            rg[u] = *pg;
                        }
                    }
                    pv += a.v.st;
                    pd += a.delta.st;
                    pz += a.z.st;
                    pg += g.dO.st;
                }
                const f32x2 bias2 = pack2(bias[m], bias[m]), skip2 = pack2(skip[m], skip[m]);
                f32x2 dd2 = 0ull, db2 = 0ull;
#pragma unroll
                for (int u = 0; u < EU; u += 2) {
                    const float *at = sDt + (j0 + u) * CH + cc;   // the four arrays lie kChan apart
                    auto both = [&](int which) { return pack2(at[which * Sh::kChan], at[which * Sh::kChan + CH]); };
                    const f32x2 gk = both(0), aw = both(1), dy = both(2);
                    const f32x2 v = pack2(Io<IO>::cvt(rv[u]), Io<IO>::cvt(rv[u + 1]));
                    const f32x2 raw = add2(pack2(Io<IO>::cvt(rd[u]), Io<IO>::cvt(rd[u + 1])), bias2);
                    f32x2 ddl = fma2(v, gk, aw), dt = raw;
                    if (soft) {
                        dt = softplus2(raw);
                        ddl = mul2(ddl, sigmoid2(raw));
                    }
                    const f32x2 dv = fma2(dt, gk, mul2(skip2, dy));
                    float d0, d1, l0, l1, z0 = 0.f, z1 = 0.f;
                    unpack2(dv, d0, d1);
                    unpack2(ddl, l0, l1);
                    if (has_dz) {
                        const f32x2 z = pack2(Io<IO>::cvt(rz[u]), Io<IO>::cvt(rz[u + 1])), sg = sigmoid2(z);
                        const f32x2 slope = mul2(sg, fma2(z, fma2(sg, pack2(-1.f, -1.f), pack2(1.f, 1.f)), pack2(1.f, 1.f)));
                        unpack2(mul2(mul2(pack2(rg[u], rg[u + 1]), fma2(skip2, v, both(3))), slope), z0, z1);
                    }
                    const bool in0 = j0 + u < here, in1 = j0 + u + 1 < here;   // rows behind the end are 0
                    l0 = in0 ? l0 : 0.f;
                    l1 = in1 ? l1 : 0.f;
                    dd2 = fma2(dy, v, dd2);     // dy and v are 0 there
                    db2 = add2(db2, pack2(l0, l1));
                    if (j0 + u < rows) {
                        *ov = in0 ? d0 : 0.f;
                        *od = l0;
                        if (has_dz) *oz = in0 ? z0 : 0.f;
                    }
                    if (j0 + u + 1 < rows) {
                        ov[g.dv.st] = in1 ? d1 : 0.f;
                        od[g.ddelta.st] = l1;
                        if (has_dz) oz[g.dz.st] = in1 ? z1 : 0.f;
                    }
                    ov += 2 * g.dv.st;
                    od += 2 * g.ddelta.st;
                    oz += 2 * g.dz.st;
                }
                dd[m] += sum2(dd2);
                db[m] += sum2(db2);
            }
        }
        // ---- dq and dk: the warps' parts
        for (int idx = tid; idx < Sh::kKq; idx += NT) {
            const int j = idx / COLS, c = idx % COLS;
            if (j >= rows || c >= a.dk) continue;
            float dq = 0.f, dk = 0.f;
            if (j < here) {
#pragma unroll
                for (int x = 0; x < Sh::kWarps; ++x) {
                    dq += sDq[(x * kSeg + j) * COLS + c];
                    dk += sDk[(x * kSeg + j) * COLS + c];
                }
            }
            if (ngrp == 1) {
                row_of<float>(g.dq, b, h, t0 + j)[c] = dq;
                row_of<float>(g.dk, b, h, t0 + j)[c] = dk;
            } else {
                const long long part = (long long)a.B * a.H * a.T * a.dk;
                const long long at = grp * part + ((long long)bh * a.T + t0 + j) * a.dk + c;
                w.qk[at] = dq;
                w.qk[ngrp * part + at] = dk;
            }
        }
        __syncthreads();   // the next segment's inputs take these places
    }
    // ---- this block's parts of the parameters' gradients
    const long long part = (long long)walk * a.B + b, HV = (long long)a.H * a.dv;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int ch = c00 + lc + 2 * i, c = sl * 4 + s;
            float lo, hi;
            unpack2(dA[i][s], lo, hi);
            float *to = w.dA + (part * HV + (long long)h * a.dv + ch) * a.dk + c;
            if (ch < a.dv && c < a.dk) to[0] = lo;
            if (ch + 1 < a.dv && c < a.dk) to[a.dk] = hi;
            if (ONE && g.dS0) {   // G has come down to the initial state
                float *to_s = g.dS0 + ((long long)bh * a.dv + ch) * a.dk + c;
                unpack2(G[i][s], lo, hi);
                if (ch < a.dv && c < a.dk) to_s[0] = lo;
                if (ch + 1 < a.dv && c < a.dk) to_s[a.dk] = hi;
            }
        }
#pragma unroll
    for (int m = 0; m < Sh::kPer; ++m) {
        const int cc = tid + m * NT, ch = c00 + cc;
        if (cc >= CH || ch >= a.dv) continue;
        w.dd[part * HV + (long long)h * a.dv + ch] = dd[m];
        w.db[part * HV + (long long)h * a.dv + ch] = db[m];
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
    int nseg, walk, nwalk, ngrp, cols;
    int block;          // walks of a block of step 1
    long long groups1;  // blocks of step 1 for each of its stretches of walks
    long long rows;     // channels of all sequences
    long long qk;       // floats of all parts of dq and dk
    long long floats;   // the workspace
};

// Turns that `blocks` blocks take at three an SM: what registers and shared memory allow steps 1 and 3 for dk from 9 to
// 32. (Shared memory leaves five blocks an SM for dk <= 4, four for dk <= 8, two for dk <= 64 and one above; they are
// planned the same way.)
long long turns(long long blocks) { return (blocks + 148 * 3 - 1) / (148 * 3); }

// Segments of a walk: those with the shortest estimate in tokens' work of a block of step 3: its turns times a walk and
// its prologue, and 0.4 for each walk's joins and parts of dA (as large as the state). For the case above that is ten
// segments, one turn of 416 blocks (with two, four and eight segments 385, 382 and 470 us in all where this took 344).
BwdSizes bwd_sizes(const falcon_scan_args_t &a) {
    BwdSizes z;
    z.nseg = (a.T + kSeg - 1) / kSeg;
    const int ch = bwd_channels(bwd_lanes(a.dk));
    z.ngrp = (a.dv + ch - 1) / ch;
    z.cols = scan_cols(a.dk);
    z.rows = (long long)a.B * a.H * a.dv;
    const long long groups = (long long)z.ngrp * a.B * a.H;
    double best = 0.0;
    z.walk = 1;
    for (int walk = 1; walk <= 32; ++walk) {
        const long long n = (z.nseg + walk - 1) / walk;
        const double cost = (double)turns(groups * n) * (walk * kSeg + 4) + 0.4 * n;
        if (walk == 1 || cost < best) {
            best = cost;
            z.walk = walk;
        }
    }
    z.nwalk = (z.nseg + z.walk - 1) / z.walk;
    // step 1: blocks of as many walks as fill the SMs best, with a prologue of about 24 tokens' time
    const int cpb = kScanThreads / (a.dk <= 16 ? 1 : a.dk <= 32 ? 2 : a.dk <= 64 ? 4 : 8);
    z.groups1 = (long long)a.B * a.H * ((a.dv + cpb - 1) / cpb);
    z.block = 1;
    for (int n = 1; n <= 16; ++n) {
        const double cost = (double)turns(z.groups1 * ((z.nwalk + n - 1) / n)) * (n * z.walk * kSeg + 24);
        if (n == 1 || cost < best) {
            best = cost;
            z.block = n;
        }
    }
    z.qk = z.ngrp > 1 ? 2LL * z.ngrp * a.B * a.H * a.T * a.dk : 0;
    z.floats = z.rows * (z.nseg * (z.cols + 1LL) + z.nwalk * (2LL * z.cols + 1 + a.dk + 2)) + z.qk;
    return z;
}

template <typename IO, int SL>
cudaError_t scan_bwd_t(const falcon_scan_args_t &a, const falcon_scan_grads_t &g, const ScanBwdWork &w, int ngrp, cudaStream_t s) {
    const long long blocks = (long long)ngrp * a.B * a.H * w.s.nwalk;
    const size_t smem = BwdShape<SL>::kBytes;
    const auto kern = w.s.nwalk == 1 ? scan_bwd_kernel<IO, SL, true> : scan_bwd_kernel<IO, SL, false>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)blocks, BwdShape<SL>::kThreads, smem, s>>>(a, g, w, ngrp);
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

// Every launch's grid, so that a call that one of them would refuse writes nothing.
bool scan_bwd_fits(const falcon_scan_args_t &a) {
    const BwdSizes z = bwd_sizes(a);
    const long long bh = (long long)a.B * a.H, walks = (z.nwalk + z.block - 1) / z.block;
    const auto fits = [](long long n, long long times) { return times == 0 || n <= kMaxGrid / times; };
    return fits(z.groups1, walks) && fits(z.ngrp * bh, z.nwalk) && (z.rows * z.cols + 255) / 256 <= kMaxGrid &&
           (z.ngrp <= 1 || (bh * a.T * a.dk + 255) / 256 <= kMaxGrid) && ((long long)a.H * a.dv * (a.dk + 2LL)) / 32 + 3 <= kMaxGrid;
}

size_t scan_bwd_workspace(const falcon_scan_args_t &a) { return sizeof(float) * (size_t)bwd_sizes(a).floats; }

cudaError_t launch_scan_bwd(const falcon_scan_args_t &a, const falcon_scan_grads_t &g, float *ws, cudaStream_t s) {
    if (a.H == 0) return cudaSuccess;
    const BwdSizes z = bwd_sizes(a);
    ScanBwdWork w{};
    w.s.seg = kSeg;
    w.s.nseg = z.nseg;
    w.s.walk = z.walk;
    w.s.nwalk = z.nwalk;
    w.s.block = z.block;
    w.s.dO = g.dO;
    w.s.ends = ws;   // the rows of states first: they are read as 16-byte pairs
    w.s.wends = w.s.ends + z.nseg * z.rows * z.cols;
    w.s.wgrads = w.s.wends + z.nwalk * z.rows * z.cols;
    w.s.steps = w.s.wgrads + z.nwalk * z.rows * z.cols;
    w.s.wsteps = w.s.steps + z.nseg * z.rows;
    w.dA = w.s.wsteps + z.nwalk * z.rows;
    w.dd = w.dA + z.nwalk * z.rows * a.dk;
    w.db = w.dd + z.nwalk * z.rows;
    w.qk = w.db + z.nwalk * z.rows;
    const bool single = z.nwalk == 1 && a.B == 1;   // one part of each parameter's gradient: it is the gradient
    if (single) {
        w.dA = g.dA;
        if (g.dD) w.dd = g.dD;
        if (g.ddelta_bias) w.db = g.ddelta_bias;
    }
    cudaError_t e;
    if (a.B > 0) {
        if (z.nseg > 1) {
            e = launch_scan_pass(kScanBoth, a, w.s, s);
            if (e != cudaSuccess) return e;
        }
        if (z.nwalk != 1) {
            const long long jb = (z.rows * z.cols + 255) / 256;
            scan_join_kernel<<<dim3((unsigned)jb, 2), 256, 0, s>>>(a, w.s, z.cols, g.dS_T, g.dS0);
            e = cudaGetLastError();
            if (e != cudaSuccess) return e;
        }
        if (z.nseg > 0) {
            e = a.io_dtype == FALCON_BF16 ? scan_bwd_io<__nv_bfloat16>(a, g, w, z.ngrp, s) : scan_bwd_io<float>(a, g, w, z.ngrp, s);
            if (e != cudaSuccess) return e;
            if (z.ngrp > 1) {
                const long long blocks = ((long long)a.B * a.H * a.T * a.dk + 255) / 256;
                scan_qk_sum_kernel<<<dim3((unsigned)blocks, 2), 256, 0, s>>>(a, g, w.qk, z.ngrp);
                e = cudaGetLastError();
                if (e != cudaSuccess) return e;
            }
        }
    }
    if (single) return cudaSuccess;
    const long long hrows = (long long)a.H * a.dv, hplane = hrows * a.dk;
    const SumJob jobs[3] = {{w.dA, hplane, hplane, g.dA}, {w.dd, hrows, hrows, g.dD}, {w.db, hrows, hrows, g.ddelta_bias}};
    return launch_column_sums(jobs, 3, (long long)z.nwalk * a.B, s);
}

}  // namespace falcon
