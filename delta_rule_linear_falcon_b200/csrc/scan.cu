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
    constexpr int NP = ST / 2;                       // pairs of columns of a thread
    typedef Pack<IO, 1> P;
    __shared__ __align__(16) float kq[2][kScanChunk * ROW];

    unsigned bid = blockIdx.x;
    const int grp = (int)(bid % (unsigned)ngrp);
    bid /= (unsigned)ngrp;
    const int bh = (int)(bid % (unsigned)(a.B * a.H));
    const int seg0 = (int)(bid / (unsigned)(a.B * a.H)) * (MODE == kScanBoth ? w.run : 1);
    const int b = bh / a.H, h = bh % a.H;
    const int tid = threadIdx.x;
    const int sl = tid % SL, ch = grp * CPB + tid / SL;
    const bool ok = ch < a.dv;
    const int n = seq_length(a.lengths, b, a.T);
    // tokens [t0, t1), of which those below n are there
    const long long first = (long long)seg0 * w.seg;
    const long long last = MODE == kScanBoth ? first + (long long)w.run * w.seg : first + w.seg;
    const int t0 = (int)(first < a.T ? first : a.T);
    const int t1 = (int)(last < a.T ? last : a.T);
    const int te = n < t1 ? n : t1;

    const long long hc = (long long)h * a.dv + (ok ? ch : 0);      // (H,dv)
    const long long bhc = (long long)bh * a.dv + (ok ? ch : 0);    // (B,H,dv)
    const float *S0 = a.S0 ? a.S0 + bhc * a.dk : nullptr;
    float *const ends = w.ends + bhc * w.nseg * DKP + sl * ST;     // this thread's columns, segment by segment
    float *const steps = w.steps + bhc * w.nseg;

    if (MODE == kScanEnds && seg0 == w.nseg - 1) {
        // the last segment's end is not needed: its place keeps the initial state for the second launch,
        // which may write S_out over S0
        if (ok)
#pragma unroll
            for (int s = 0; s < ST; ++s)
                ends[(long long)seg0 * DKP + s] = S0 && sl * ST + s < a.dk ? S0[sl * ST + s] : 0.f;
        return;
    }

    f32x2 A2[NP], S[NP], Pr[MODE == kScanBoth ? NP : 1], G[MODE == kScanBoth ? NP : 1];
    auto column = [&](const float *row, int s) { return ok && row && sl * ST + s < a.dk ? row[sl * ST + s] : 0.f; };
#pragma unroll
    for (int s = 0; s < NP; ++s) {
        A2[s] = pack2(column(a.A + hc * a.dk, 2 * s) * kLog2e, column(a.A + hc * a.dk, 2 * s + 1) * kLog2e);
        S[s] = 0ull;
        if (MODE == kScanBoth) { Pr[s] = pack2(1.f, 1.f); G[s] = 0ull; }
    }
    const float bias = ok && a.delta_bias ? a.delta_bias[hc] : 0.f;
    const float skip = ok && MODE == kScanFull && a.D ? a.D[hc] : 0.f;
    const bool soft = (a.flags & FALCON_SCAN_SOFTPLUS) != 0;
    if (MODE == kScanFull) {
        if (w.nseg == 1) {
#pragma unroll
            for (int s = 0; s < NP; ++s) S[s] = pack2(column(S0, 2 * s), column(S0, 2 * s + 1));
        } else if (ok) {
#pragma unroll
            for (int s = 0; s < NP; s += 2) load_pairs(ends + (long long)(w.nseg - 1) * DKP + 2 * s, S[s], S[s + 1]);
#pragma unroll 2
            for (int j = 0; j < seg0; ++j) {
                const float sd = steps[j];
                const f32x2 sd2 = pack2(sd, sd);
#pragma unroll
                for (int s = 0; s < NP; s += 2) {
                    f32x2 e0, e1;
                    load_pairs(ends + (long long)j * DKP + 2 * s, e0, e1);
                    S[s] = fma2(ex2_2(mul2(A2[s], sd2)), S[s], e0);
                    S[s + 1] = fma2(ex2_2(mul2(A2[s + 1], sd2)), S[s + 1], e1);
                }
            }
        }
    }

    const unsigned cu = ok ? (unsigned)ch : 0u;
    const IO *pv = row_of<IO>(a.v, b, h, t0), *pd = row_of<IO>(a.delta, b, h, t0);
    const IO *pz = a.z.p ? row_of<IO>(a.z, b, h, t0) : nullptr;
    const IO *pk = row_of<IO>(a.k, b, h, 0), *pq = row_of<IO>(a.q, b, h, 0);
    const float *pg = MODE == kScanBoth ? row_of<float>(w.dO, b, h, t0) : nullptr;
    IO *po = MODE == kScanFull ? row_of<IO>(a.o, b, h, t0) : nullptr;

    typename P::raw rv[kScanChunk], rd[kScanChunk], rz[kScanChunk], rkq[NKQ];
    float rg[MODE == kScanBoth ? kScanChunk : 1];
    // loads of the chunk at t, and the row pointers on to the next one
    auto fetch = [&](int t) {
        const bool whole = t + kScanChunk <= te;
#pragma unroll
        for (int j = 0; j < kScanChunk; ++j) {
            const bool in = whole || t + j < te;
            rv[j] = P::zero();
            rd[j] = P::zero();
            if (MODE != kScanEnds) rz[j] = P::zero();
            if (MODE == kScanBoth) rg[j] = 0.f;
            if (in) {
                rv[j] = P::ld(pv + cu);
                rd[j] = P::ld(pd + cu);
                if (MODE != kScanEnds && pz) rz[j] = P::ld(pz + cu);
                if (MODE == kScanBoth) rg[j] = pg[cu];
            }
            pv += a.v.st;
            pd += a.delta.st;
            if (MODE != kScanEnds && pz) pz += a.z.st;
            if (MODE == kScanBoth) pg += w.dO.st;
        }
#pragma unroll
        for (int m = 0; m < NKQ; ++m) {
            const int e = tid + m * kScanThreads, j = e / ROW, c = e % DKP;
            const bool isq = e % ROW >= DKP;
            rkq[m] = P::zero();
            if (e < kScanChunk * ROW && t + j < te && c < a.dk && !(MODE == kScanEnds && isq))
                rkq[m] = isq ? P::ld(pq + (t + j) * a.q.st + c) : P::ld(pk + (t + j) * a.k.st + c);
        }
    };

    float sum = 0.f;
    int seg = seg0, left = w.seg;   // kScanBoth: the segment being walked and its tokens to come
    fetch(t0);
    int buf = 0;
    for (int t = t0; t < (MODE == kScanBoth ? t1 : te); t += kScanChunk, buf ^= 1) {
        float dt[kScanChunk], v[kScanChunk], z[kScanChunk], g[kScanChunk];
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
            dt[j] = soft ? softplus(raw) : raw;
            if (MODE != kScanEnds) {
                P::cvt(rz[j], x);
                z[j] = x[0];
            }
            g[j] = MODE == kScanBoth ? (pz ? rg[j] * silu(z[j]) : rg[j]) : 0.f;
        }
        if (t + kScanChunk > te) {   // behind the end the step is 0, the state stays, and nothing flows back
#pragma unroll
            for (int j = 0; j < kScanChunk; ++j)
                if (t + j >= te) dt[j] = v[j] = g[j] = 0.f;
        }
        if (t + kScanChunk < te) fetch(t + kScanChunk);
        __syncthreads();   // the chunk is staged; the other buffer was last read before this barrier
        const bool whole = t + kScanChunk <= te;
#pragma unroll
        for (int j = 0; j < kScanChunk; ++j) {
            const float *k4 = &kq[buf][j * ROW + sl * ST];
            const float *q4 = &kq[buf][j * ROW + DKP + sl * ST];
            const f32x2 dt2 = pack2(dt[j], dt[j]);
            const float b1 = dt[j] * v[j];
            const f32x2 b2 = pack2(b1, b1);
            f32x2 y2 = 0ull, g2 = 0ull;
            if (MODE == kScanBoth) g2 = pack2(g[j], g[j]);
            if (MODE != kScanFull) sum += dt[j];
#pragma unroll
            for (int s = 0; s < NP; s += 2) {
                f32x2 kk[2], qq[2];
                load_pairs(k4 + 2 * s, kk[0], kk[1]);
                if (MODE != kScanEnds) load_pairs(q4 + 2 * s, qq[0], qq[1]);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const f32x2 e = ex2_2(mul2(dt2, A2[s + r]));
                    S[s + r] = fma2(e, S[s + r], mul2(b2, kk[r]));
                    if (MODE == kScanFull) y2 = fma2(S[s + r], qq[r], y2);
                    if (MODE == kScanBoth) {
                        Pr[s + r] = mul2(Pr[s + r], e);
                        G[s + r] = fma2(Pr[s + r], mul2(g2, qq[r]), G[s + r]);
                    }
                }
            }
            if (MODE == kScanFull) {
                float y = sum2(y2);
#pragma unroll
                for (int m = 1; m < SL; m <<= 1) y += __shfl_xor_sync(0xffffffffu, y, m);
                y = fmaf(skip, v[j], y);
                if (pz) y *= silu(z[j]);
                if (ok && sl == 0 && (whole || t + j < te)) {
                    const float out[1] = {y};
                    P::st(po + cu, out);
                }
                po += a.o.st;
            }
        }
        if (MODE == kScanBoth) {
            left -= kScanChunk;
            if (left == 0 || t + kScanChunk >= t1) {   // the segment's end: hand it over, start the next from zero
                if (ok) {
                    float *const to = ends + (long long)seg * DKP, *const tg = w.grads + (bhc * w.nseg + seg) * DKP + sl * ST;
#pragma unroll
                    for (int s = 0; s < NP; s += 2) {
                        store_pairs(to + 2 * s, S[s], S[s + 1]);
                        store_pairs(tg + 2 * s, G[s], G[s + 1]);
                    }
                    if (sl == 0) steps[seg] = sum;
                }
                ++seg;
                left = w.seg;
                sum = 0.f;
#pragma unroll
                for (int s = 0; s < NP; ++s) {
                    S[s] = 0ull;
                    G[s] = 0ull;
                    Pr[s] = pack2(1.f, 1.f);
                }
            }
        }
    }
    if (MODE == kScanBoth || !ok) return;
    if (MODE == kScanEnds) {
#pragma unroll
        for (int s = 0; s < NP; s += 2) store_pairs(ends + (long long)seg0 * DKP + 2 * s, S[s], S[s + 1]);
        if (sl == 0) steps[seg0] = sum;
    } else if (a.S_out && seg0 == w.nseg - 1) {
        float *to = a.S_out + bhc * a.dk;
#pragma unroll
        for (int s = 0; s < NP; ++s) {
            float lo, hi;
            unpack2(S[s], lo, hi);
            if (sl * ST + 2 * s < a.dk) to[sl * ST + 2 * s] = lo;
            if (sl * ST + 2 * s + 1 < a.dk) to[sl * ST + 2 * s + 1] = hi;
        }
    }
}

// One token. A channel's row of the state is read and written by G lanes, four columns each, so the state
// moves in whole lines; each thread has the rows of kStepRows channels in flight, and those of the next sequence
// while it works on this one's. A block takes the same channels of several sequences: A, as large as a sequence's
// state, is read once for them. A channel's scalars (step, dt v, output) belong to one of its lanes.
constexpr int kStepThreads = 128, kStepRows = 4;

template <typename IO, int G, bool V4>
__global__ void __launch_bounds__(kStepThreads) scan_step_kernel(falcon_scan_args_t a, int ngrp, int chunk) {
    constexpr int CPP = kStepThreads / G;                          // channels of a pass
    constexpr int OWN = G >= kStepRows ? 1 : kStepRows / G;        // rows whose scalars this lane keeps
    const int grp = blockIdx.x % (unsigned)ngrp;
    const unsigned rest = blockIdx.x / (unsigned)ngrp;
    const int h = rest % (unsigned)a.H;
    const int b0 = (int)(rest / (unsigned)a.H) * chunk, b1 = min(b0 + chunk, a.B);
    const int lane = threadIdx.x & 31, sl = threadIdx.x % G, c0 = sl * 4;
    const int ch0 = grp * CPP * kStepRows + threadIdx.x / G;
    const bool soft = (a.flags & FALCON_SCAN_SOFTPLUS) != 0, cols = c0 < a.dk;
    // the row whose total lanes_sum leaves in this lane, and the lane of the group that keeps row i
    const int own = G >= kStepRows ? sl / (G / kStepRows > 0 ? G / kStepRows : 1) : sl * OWN;
    const bool writes = G < kStepRows || sl % (G / kStepRows > 0 ? G / kStepRows : 1) == 0;
    auto keeper = [](int i) { return G >= kStepRows ? i * (G / kStepRows) : i / OWN; };

    auto row4 = [&](const float *p, float (&x)[4]) {
        if (V4) {
            const float4 f = __ldcs(reinterpret_cast<const float4 *>(p + c0));
            x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = c0 + r < a.dk ? __ldcs(p + c0 + r) : 0.f;
        }
    };
    float S[kStepRows][4], A2[kStepRows][4], q[4], k[4], raw[OWN], v[OWN], z[OWN], bias[OWN], skip[OWN];
    auto fetch = [&](int b) {
#pragma unroll
        for (int i = 0; i < kStepRows; ++i) {
            const int ch = ch0 + i * CPP;
#pragma unroll
            for (int r = 0; r < 4; ++r) S[i][r] = 0.f;
            if (ch < a.dv && cols) row4(a.S0 + (((long long)b * a.H + h) * a.dv + ch) * a.dk, S[i]);
        }
        const IO *pq = row_of<IO>(a.q, b, h, 0), *pk = row_of<IO>(a.k, b, h, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            q[r] = c0 + r < a.dk ? Io<IO>::ld(pq, c0 + r) : 0.f;
            k[r] = c0 + r < a.dk ? Io<IO>::ld(pk, c0 + r) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < OWN; ++j) {
            const int ch = ch0 + (own + j) * CPP;
            raw[j] = v[j] = z[j] = 0.f;
            if (ch < a.dv) {
                raw[j] = Io<IO>::ld(row_of<IO>(a.delta, b, h, 0), ch);
                v[j] = Io<IO>::ld(row_of<IO>(a.v, b, h, 0), ch);
                if (a.z.p) z[j] = Io<IO>::ld(row_of<IO>(a.z, b, h, 0), ch);
            }
        }
    };
    fetch(b0);
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) {
        const int ch = ch0 + i * CPP;
        const float *row = a.A + ((long long)h * a.dv + ch) * a.dk + c0;
#pragma unroll
        for (int r = 0; r < 4; ++r) A2[i][r] = 0.f;
        if (ch < a.dv && cols) {
            if (V4) {
                const float4 f = *reinterpret_cast<const float4 *>(row);
                A2[i][0] = f.x * kLog2e; A2[i][1] = f.y * kLog2e; A2[i][2] = f.z * kLog2e; A2[i][3] = f.w * kLog2e;
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (c0 + r < a.dk) A2[i][r] = row[r] * kLog2e;
            }
        }
    }
#pragma unroll
    for (int j = 0; j < OWN; ++j) {
        const int ch = ch0 + (own + j) * CPP;
        bias[j] = ch < a.dv && a.delta_bias ? a.delta_bias[(long long)h * a.dv + ch] : 0.f;
        skip[j] = ch < a.dv && a.D ? a.D[(long long)h * a.dv + ch] : 0.f;
    }
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        float dt[OWN], dtv[OWN], vv[OWN], zz[OWN], y[kStepRows], T[kStepRows][4];
#pragma unroll
        for (int j = 0; j < OWN; ++j) {
            const float x = raw[j] + bias[j];
            dt[j] = soft ? softplus(x) : x;
            dtv[j] = dt[j] * v[j];
            vv[j] = v[j];
            zz[j] = z[j];
        }
#pragma unroll
        for (int i = 0; i < kStepRows; ++i) {
            const float d = __shfl_sync(0xffffffffu, dt[i % OWN], keeper(i), G), x = __shfl_sync(0xffffffffu, dtv[i % OWN], keeper(i), G);
            y[i] = 0.f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                T[i][r] = fmaf(fast_ex2(d * A2[i][r]), S[i][r], x * k[r]);
                y[i] = fmaf(T[i][r], q[r], y[i]);
            }
        }
        if (b + 1 < b1) fetch(b + 1);
        const long long bh = (long long)b * a.H + h;
#pragma unroll
        for (int i = 0; i < kStepRows; ++i) {
            const int ch = ch0 + i * CPP;
            if (ch < a.dv && cols) {
                float *to = a.S_out + (bh * a.dv + ch) * a.dk + c0;
                if (V4) __stcs(reinterpret_cast<float4 *>(to), make_float4(T[i][0], T[i][1], T[i][2], T[i][3]));
                else
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (c0 + r < a.dk) __stcs(to + r, T[i][r]);
            }
        }
        bool first;
        lanes_sum<kStepRows, G, 1>(y, lane, first);
        if (writes) {
            IO *po = row_of<IO>(a.o, b, h, 0);
#pragma unroll
            for (int j = 0; j < OWN; ++j) {
                const int ch = ch0 + (own + j) * CPP;
                float o = fmaf(skip[j], vv[j], y[j]);
                if (a.z.p) o *= silu(zz[j]);
                if (ch < a.dv) Io<IO>::st(po, ch, o);
            }
        }
    }
}

template <typename IO, int ST, int SL>
cudaError_t scan_pass_t(int mode, const falcon_scan_args_t &a, const ScanWork &w, cudaStream_t s) {
    const int cpb = kScanThreads / SL;
    const int ngrp = (a.dv + cpb - 1) / cpb;
    const int runs = mode == kScanBoth ? (w.nseg + w.run - 1) / w.run : w.nseg;
    const long long blocks = (long long)ngrp * a.B * a.H * runs;
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
    int chunk = 8;   // sequences of a block, while two blocks a place on the GPU are left
    while (chunk > 1 && (long long)ngrp * a.H * ((a.B + chunk - 1) / chunk) < 148 * 8) chunk /= 2;
    const long long blocks = (long long)ngrp * a.H * ((a.B + chunk - 1) / chunk);
    if (blocks > kMaxGrid) return cudaErrorInvalidConfiguration;
    const uintptr_t any = reinterpret_cast<uintptr_t>(a.S0) | reinterpret_cast<uintptr_t>(a.S_out) | reinterpret_cast<uintptr_t>(a.A);
    if (a.dk % 4 == 0 && any % 16 == 0) scan_step_kernel<IO, G, true><<<(unsigned)blocks, kStepThreads, 0, s>>>(a, ngrp, chunk);
    else scan_step_kernel<IO, G, false><<<(unsigned)blocks, kStepThreads, 0, s>>>(a, ngrp, chunk);
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
    p.bytes = (size_t)p.nseg * bh * a.dv * (scan_cols(a.dk) + 1) * sizeof(float);
    return p;
}

cudaError_t launch_scan_fwd(const falcon_scan_args_t &a, const ScanPlan &plan, float *ws, cudaStream_t s) {
    if ((long long)a.B * a.H == 0) return cudaSuccess;
    ScanWork w{};
    w.seg = plan.seg;
    w.nseg = plan.nseg;
    if (plan.nseg > 1) {
        w.ends = ws;
        w.steps = ws + (size_t)plan.nseg * a.B * a.H * a.dv * scan_cols(a.dk);
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
