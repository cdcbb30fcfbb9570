// scan.cu -- falcon_scan_fwd and falcon_scan_step: the selective scan
//   S_t[i,c] = exp(dt_t[i] A[i,c]) S_{t-1}[i,c] + dt_t[i] v_t[i] k_t[c],
//   o_t[i]   = (sum_c S_t[i,c] q_t[c] + D[i] v_t[i]) silu(z_t[i]).
//
// Each entry of the state takes one exponential and four fp32 operations a token, so at dk = 16 the
// exponential unit (16 a clock and SM) bounds the pass, well above HBM: 16 exponentials against about
// eight bytes of v, delta, z and o. No product is shared between channels, so there is no matrix
// instruction to use. A thread owns a channel and ST <= 16 columns of its state in registers, two columns an
// instruction (SL lanes share a channel when dk > 16 and join their parts of o). Everything else is kept short,
// because it competes with those exponentials for the instruction slots: v, delta and z of kScanChunk tokens come
// as 16-byte asynchronous copies into a ring in shared memory, one copy a thread and tensor, and are read there at
// fixed offsets; o goes back the same way, in the place of z (or v) (loads and stores of single elements, with
// their addresses, took a fifth of the pass). Where rows are not 16-byte multiples, elements are copied one by one
// (B1 T16384 dv2048 off alignment: 503 us against 352).
// q_t and k_t, the same for all channels of a head, are staged in fp32 and read as broadcasts. Step sizes (softplus)
// are computed two tokens an instruction, once per channel and token.
//
// Split: B H dv channels are the only parallel axis of the recurrence; with few of them the sequence is
// cut into segments (scan_plan). A first launch runs every segment from a zero state and leaves its end
// state E and the sum of its steps sd, from which the decay over the segment is exp(A sd); in the second
// each segment joins the states before it, S <- exp(A sd_j) S + E_j, and runs with outputs.
// Measured, bf16, dk = 16: B4 H16 T2048 dv128 (64 blocks unsplit) 183 us in 9 segments, 383 us unsplit. B1 T16384
// dv2048: 352 us in 37 segments. 512 blocks unsplit (B32 H16 T1024 dv128): 439 us, 110 us for each 2^28 entries, whose
// exponentials alone are 58 us. No unit is full: in the launches of the split passes the exponential unit is at 66 to 69%
// (a quarter of its work moved to the multiply-add pipes) and 71%, the instruction slots at 61 to 63% and 48%, the
// multiply-add pipes at 60 to 63% and 40%, with 11 to 13 warps an SM (124 and 128 registers): too few of them to cover
// each other's latencies. Two passes and four exponentials for three are the other half of the distance.
#include "scan.cuh"

namespace falcon {

namespace {

// Rows of CHUNK tokens x CPB channels of E, brought into shared memory by the block's threads. WIDE: asynchronous
// copies of 16 bytes; otherwise a thread holds its elements in registers between load() and store().
template <typename E, int CPB, bool WIDE> struct Tile {
    static constexpr int kPer = 16 / (int)sizeof(E);                       // elements of a copy
    static constexpr int kPieces = kScanChunk * CPB / kPer;
    static constexpr int kCopies = (kPieces + kScanThreads - 1) / kScanThreads;
    static constexpr int kElems = (kScanChunk * CPB + kScanThreads - 1) / kScanThreads;
    E raw[WIDE ? 1 : kElems];
    // the rows t.. of `view` from channel c0 on, te tokens and dv channels being there
    __device__ __forceinline__ void load(E *to, const E *rows, long long st, int left, int channels) {
        if (WIDE) {
#pragma unroll
            for (int m = 0; m < kCopies; ++m) {
                const int p = threadIdx.x + m * kScanThreads, j = p / (CPB / kPer), c = p % (CPB / kPer) * kPer;
                if (p < kPieces && j < left && c < channels) copy_async<16>(to + j * CPB + c, rows + j * st + c);
            }
        } else {
#pragma unroll
            for (int m = 0; m < kElems; ++m) {
                const int p = threadIdx.x + m * kScanThreads, j = p / CPB, c = p % CPB;
                if (p < kScanChunk * CPB && j < left && c < channels) raw[m] = rows[j * st + c];
            }
        }
    }
    __device__ __forceinline__ void store(E *to) const {
        if (!WIDE) {
#pragma unroll
            for (int m = 0; m < kElems; ++m) {
                const int p = threadIdx.x + m * kScanThreads;
                if (p < kScanChunk * CPB) to[p] = raw[m];
            }
        }
    }
};

// CHUNK tokens' outputs from shared memory to their rows, by the threads that copied those places in.
template <typename E, int CPB, bool WIDE>
__device__ __forceinline__ void put_rows(const E *from, E *rows, long long st, int left, int channels) {
    typedef Tile<E, CPB, WIDE> T;
    if (WIDE) {
#pragma unroll
        for (int m = 0; m < T::kCopies; ++m) {
            const int p = threadIdx.x + m * kScanThreads, j = p / (CPB / T::kPer), c = p % (CPB / T::kPer) * T::kPer;
            if (p < T::kPieces && j < left && c < channels)
                *reinterpret_cast<uint4 *>(rows + j * st + c) = *reinterpret_cast<const uint4 *>(from + j * CPB + c);
        }
    } else {
#pragma unroll
        for (int m = 0; m < T::kElems; ++m) {
            const int p = threadIdx.x + m * kScanThreads, j = p / CPB, c = p % CPB;
            if (p < kScanChunk * CPB && j < left && c < channels) rows[j * st + c] = from[p];
        }
    }
}

template <typename IO, int ST, int SL, int MODE, bool WIDE>
__global__ void __launch_bounds__(kScanThreads, MODE == kScanBoth ? 3 : 4) scan_kernel(falcon_scan_args_t a, ScanWork w, int ngrp) {
    constexpr int C = kScanChunk;
    constexpr int DKP = ST * SL;                     // padded columns
    constexpr int CPB = kScanThreads / SL;           // channels of a block
    constexpr int ROW = 2 * DKP;                     // k and q of a token
    constexpr int NKQ = (C * ROW + kScanThreads - 1) / kScanThreads;
    constexpr int NP = ST / 2;                       // pairs of columns of a thread
    // of the segments' ends pass, every fourth pair's exponentials go to the multiply-add pipes (3% of the whole split
    // pass; with outputs, or more of them, the instruction slots are worth more)
    constexpr int POLY = MODE == kScanEnds ? 4 : 0;
    constexpr int RING = WIDE ? (sizeof(IO) == 4 ? 2 : 3) : 2;   // chunks in shared memory
    typedef Pack<IO, 1> P;
    __shared__ __align__(16) float kq[2][C * ROW];
    __shared__ __align__(16) IO tv[RING][C * CPB], td[RING][C * CPB], tz[RING][MODE == kScanEnds ? 1 : C * CPB];
    __shared__ __align__(16) float tg[RING][MODE == kScanBoth ? C * CPB : 1];

    unsigned bid = blockIdx.x;
    const int grp = (int)(bid % (unsigned)ngrp);
    bid /= (unsigned)ngrp;
    const int bh = (int)(bid % (unsigned)(a.B * a.H));
    const int seg0 = (int)(bid / (unsigned)(a.B * a.H)) * (MODE == kScanBoth ? w.walk * w.block : 1);
    const int b = bh / a.H, h = bh % a.H;
    const int tid = threadIdx.x;
    const int sl = tid % SL, lc = tid / SL, ch = grp * CPB + lc;
    const int channels = min(CPB, a.dv - grp * CPB);
    const bool ok = ch < a.dv;
    const int n = seq_length(a.lengths, b, a.T);
    // tokens [t0, t1), of which those below n are there
    const long long first = (long long)seg0 * w.seg;
    const long long last = MODE == kScanBoth ? first + (long long)w.walk * w.block * w.seg : first + w.seg;
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

    // ---- the ring: one tile for each tensor and chunk
    const bool has_z = MODE != kScanEnds && a.z.p;
    const long long c0 = (long long)grp * CPB;
    const IO *pv = row_of<IO>(a.v, b, h, t0) + c0, *pd = row_of<IO>(a.delta, b, h, t0) + c0;
    const IO *pz = has_z ? row_of<IO>(a.z, b, h, t0) + c0 : nullptr;
    const float *pg = MODE == kScanBoth ? row_of<float>(w.dO, b, h, t0) + c0 : nullptr;
    const IO *pk = row_of<IO>(a.k, b, h, 0), *pq = row_of<IO>(a.q, b, h, 0);
    Tile<IO, CPB, WIDE> xv, xd, xz;
    Tile<float, CPB, WIDE> xg;
    auto ask = [&](int t, int place) {   // the chunk at t; the row pointers go on to the next
        if (t < te) {
            xv.load(tv[place], pv, a.v.st, te - t, channels);
            xd.load(td[place], pd, a.delta.st, te - t, channels);
            if (has_z) xz.load(tz[place], pz, a.z.st, te - t, channels);
            if (MODE == kScanBoth) xg.load(tg[place], pg, w.dO.st, te - t, channels);
        }
        pv += C * a.v.st;
        pd += C * a.delta.st;
        if (has_z) pz += C * a.z.st;
        if (MODE == kScanBoth) pg += C * w.dO.st;
        if (WIDE) copy_commit();
    };
    auto settle = [&](int place) {       // !WIDE: what ask() holds in registers
        xv.store(tv[place]);
        xd.store(td[place]);
        if (has_z) xz.store(tz[place]);
        if (MODE == kScanBoth) xg.store(tg[place]);
    };
    typename P::raw rkq[NKQ];
    auto load_kq = [&](int t) {
#pragma unroll
        for (int m = 0; m < NKQ; ++m) {
            const int e = tid + m * kScanThreads, j = e / ROW, c = e % DKP;
            const bool isq = e % ROW >= DKP;
            rkq[m] = P::zero();
            if (e < C * ROW && t + j < te && c < a.dk && !(MODE == kScanEnds && isq))
                rkq[m] = isq ? P::ld(pq + (t + j) * a.q.st + c) : P::ld(pk + (t + j) * a.k.st + c);
        }
    };
    auto stage_kq = [&](float *to) {
#pragma unroll
        for (int m = 0; m < NKQ; ++m) {
            const int e = tid + m * kScanThreads;
            float x[1];
            P::cvt(rkq[m], x);
            if (e < C * ROW) to[e] = x[0];
        }
    };
    load_kq(t0);
#pragma unroll
    for (int i = 0; i < RING - 1; ++i) ask(t0 + i * C, i);
    if (!WIDE) settle(0);

    // ---- this thread's state
    f32x2 A2[NP], S[NP], Pr[MODE == kScanBoth ? NP : 1], G[MODE == kScanBoth ? NP : 1];
    auto column = [&](const float *row, int s) { return ok && row && sl * ST + s < a.dk ? row[sl * ST + s] : 0.f; };
#pragma unroll
    for (int s = 0; s < NP; ++s) {
        A2[s] = pack2(decay_rate(column(a.A + hc * a.dk, 2 * s)), decay_rate(column(a.A + hc * a.dk, 2 * s + 1)));
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

    IO *po = MODE == kScanFull ? row_of<IO>(a.o, b, h, t0) + c0 : nullptr;
    float sum = 0.f;
    int seg = seg0, left = 0;   // kScanBoth: the next segment, and the tokens before it
    const int tend = MODE == kScanBoth ? t1 : te;
    int place = 0, before = RING - 1, buf = 0;
    for (int t = t0; t < tend; t += C, buf ^= 1) {
        if (MODE == kScanBoth && left == 0) {   // the state before the segment that starts here
            if (ok) {
                float *const to = ends + (long long)seg * DKP;
#pragma unroll
                for (int s = 0; s < NP; s += 2) store_pairs(to + 2 * s, S[s], S[s + 1]);
                if (sl == 0) steps[seg] = sum;
            }
            ++seg;
            left = w.seg;
        }
        stage_kq(kq[buf]);
        if (WIDE) copy_wait<RING - 2>();
        __syncthreads();   // the chunk is there, and the one before is through
        if (MODE == kScanFull && t > t0) {
            put_rows<IO, CPB, WIDE>(has_z ? tz[before] : tv[before], po, a.o.st, C, channels);
            po += C * a.o.st;
            if (!WIDE) __syncthreads();   // other threads' elements
        }
        load_kq(t + C);
        ask(t + (RING - 1) * C, before);

        float dt[C], g[C];
        const IO *const vs = tv[place] + lc, *const ds = td[place] + lc;
        IO *const zs = tz[place] + (MODE == kScanEnds ? 0 : lc);
#pragma unroll
        for (int j = 0; j < C; j += 2) {
            const float x0 = Io<IO>::ld(ds, j * CPB) + bias, x1 = Io<IO>::ld(ds, (j + 1) * CPB) + bias;
            dt[j] = x0;
            dt[j + 1] = x1;
            if (soft) unpack2(softplus2(pack2(x0, x1)), dt[j], dt[j + 1]);
            g[j] = g[j + 1] = 0.f;
            if (MODE == kScanBoth) {
                const float *const gs = tg[place] + lc;
                g[j] = gs[j * CPB];
                g[j + 1] = gs[(j + 1) * CPB];
                if (has_z)
                    unpack2(mul2(pack2(g[j], g[j + 1]), silu2(pack2(Io<IO>::ld(zs, j * CPB), Io<IO>::ld(zs, (j + 1) * CPB)))), g[j], g[j + 1]);
            }
        }
        const bool whole = t + C <= te;
        if (!whole) {   // behind the end the step is 0, the state stays, and nothing flows back
#pragma unroll
            for (int j = 0; j < C; ++j)
                if (t + j >= te) dt[j] = g[j] = 0.f;
        }
        float y[C];
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const float *k4 = &kq[buf][j * ROW + sl * ST];
            const float *q4 = &kq[buf][j * ROW + DKP + sl * ST];
            const f32x2 dt2 = pack2(dt[j], dt[j]);
            float v = Io<IO>::ld(vs, j * CPB);
            if (!whole && t + j >= te) v = 0.f;   // the ring holds anything there
            const float b1 = dt[j] * v;
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
                    const f32x2 x = mul2(dt2, A2[s + r]);
                    const f32x2 e = POLY > 0 && (s + r) % (POLY > 0 ? POLY : 1) == 0 ? ex2_poly2(x) : ex2_2(x);
                    S[s + r] = fma2(e, S[s + r], mul2(b2, kk[r]));
                    if (MODE == kScanFull) y2 = fma2(S[s + r], qq[r], y2);
                    if (MODE == kScanBoth) {
                        Pr[s + r] = mul2(Pr[s + r], e);
                        G[s + r] = fma2(Pr[s + r], mul2(g2, qq[r]), G[s + r]);
                    }
                }
            }
            if (MODE == kScanFull) {
                y[j] = sum2(y2);
#pragma unroll
                for (int m = 1; m < SL; m <<= 1) y[j] += __shfl_xor_sync(0xffffffffu, y[j], m);
                y[j] = fmaf(skip, v, y[j]);
            }
        }
        if (MODE == kScanFull && sl == 0) {   // outputs in the place of z, or of v
            IO *const os = has_z ? zs : tv[place] + lc;
#pragma unroll
            for (int j = 0; j < C; j += 2) {
                if (has_z)
                    unpack2(mul2(pack2(y[j], y[j + 1]), silu2(pack2(Io<IO>::ld(zs, j * CPB), Io<IO>::ld(zs, (j + 1) * CPB)))), y[j], y[j + 1]);
                Io<IO>::st(os, j * CPB, y[j]);
                Io<IO>::st(os, (j + 1) * CPB, y[j + 1]);
            }
        }
        before = place;
        place = place + 1 < RING ? place + 1 : 0;
        if (!WIDE) settle(place);
        if (MODE == kScanBoth) {
            left -= C;
            if (t + C >= t1 || (left == 0 && seg % w.walk == 0)) {   // the walk's end: hand it over, start the next from zero
                if (ok) {
                    const long long at = bhc * w.nwalk + (seg - 1) / w.walk;
                    float *const to = w.wends + at * DKP + sl * ST, *const to_g = w.wgrads + at * DKP + sl * ST;
#pragma unroll
                    for (int s = 0; s < NP; s += 2) {
                        store_pairs(to + 2 * s, S[s], S[s + 1]);
                        store_pairs(to_g + 2 * s, G[s], G[s + 1]);
                    }
                    if (sl == 0) w.wsteps[at] = sum;
                }
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
    if (WIDE) copy_wait<0>();
    if (MODE == kScanFull && tend > t0) {   // the last chunk's outputs
        __syncthreads();
        put_rows<IO, CPB, WIDE>(has_z ? tz[before] : tv[before], po, a.o.st, (te - t0 - 1) % C + 1, channels);
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
// moves in whole lines. A thread has the rows of kStepRows channels and works through several sequences: A, as large
// as a sequence's state, is read once for them, and the states come through a ring of asynchronous copies into places
// that only the copying thread reads (no barrier; bytes in flight cost no registers). A channel's scalars (step, dt v,
// output) belong to one of its lanes and are loaded one sequence ahead. HBM bounds it: bf16, dk = 16, 256 sequences of
// H32 dv128 28 us, 5.2 TB/s; 1024 of H32 dv64 dk64 173 us, 6.2 TB/s (38 and 260 us with the next sequence's rows in
// registers, which left five blocks an SM). Blocks an SM and places of the ring, for these two: six and three 28 and 173
// us, eight and three (64 registers) 30 and 180, six and four 29 and 173, ten and two 32 and 198. dk = 15, whose rows
// are not 16-byte aligned and go by four bytes: 40 us against the 28.
constexpr int kStepThreads = 128, kStepRows = 4, kStepRing = 3, kStepBlocks = 6;

template <typename IO, int G, bool V4>
__global__ void __launch_bounds__(kStepThreads, kStepBlocks) scan_step_kernel(falcon_scan_args_t a, int ngrp, int chunk) {
    constexpr int CPP = kStepThreads / G;                          // channels of a pass
    constexpr int OWN = G >= kStepRows ? 1 : kStepRows / G;        // rows whose scalars this lane keeps
    typedef Pack<IO, V4 ? 4 : 1> P;
    constexpr int NK = V4 ? 1 : 4;
    __shared__ __align__(16) float ring[kStepRing][kStepRows][kStepThreads][4];
    const int grp = blockIdx.x % (unsigned)ngrp;
    const unsigned rest = blockIdx.x / (unsigned)ngrp;
    const int h = rest % (unsigned)a.H;
    const int b0 = (int)(rest / (unsigned)a.H) * chunk, b1 = b0 + min(chunk, a.B - b0);
    const int tid = threadIdx.x, lane = tid & 31, sl = tid % G, c0 = sl * 4;
    const int ch0 = grp * CPP * kStepRows + tid / G;
    const bool soft = (a.flags & FALCON_SCAN_SOFTPLUS) != 0;
    // the row whose total lanes_sum leaves in this lane, and the lane of the group that keeps row i
    const int own = G >= kStepRows ? sl / (G / kStepRows > 0 ? G / kStepRows : 1) : sl * OWN;
    const bool writes = G < kStepRows || sl % (G / kStepRows > 0 ? G / kStepRows : 1) == 0;
    auto keeper = [](int i) { return G >= kStepRows ? i * (G / kStepRows) : i / OWN; };
    // element r of row i is one of the state's (V4: all four or none)
    auto there = [&](int i, int r) { return ch0 + i * CPP < a.dv && c0 + (V4 ? 0 : r) < a.dk; };

    // ---- the states: this thread's part of sequence b, `per` elements from one sequence's to the next
    const long long per = (long long)a.H * a.dv * a.dk, first = ((long long)b0 * a.H + h) * a.dv * a.dk + (long long)ch0 * a.dk + c0;
    const float *from = a.S0 + first;
    float *to = a.S_out + first;
    auto ask = [&](int place, bool any) {
        if (any) {
#pragma unroll
            for (int i = 0; i < kStepRows; ++i) {
                if (V4) {
                    if (there(i, 0)) copy_async<16>(ring[place][i][tid], from + i * CPP * a.dk);
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (there(i, r)) copy_async<4>(&ring[place][i][tid][r], from + i * CPP * a.dk + r);
                }
            }
        }
        from += per;
        copy_commit();
    };
#pragma unroll
    for (int j = 0; j < kStepRing - 1; ++j) ask(j, j < b1 - b0);
#pragma unroll
    for (int i = 0; i < kStepRows; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (!there(i, r))
#pragma unroll
                for (int j = 0; j < kStepRing; ++j) ring[j][i][tid][r] = 0.f;

    typename P::raw rq[NK], rk[NK];
    float raw[OWN], v[OWN], z[OWN], bias[OWN], skip[OWN];
    auto fetch = [&](int b) {
        const IO *pq = row_of<IO>(a.q, b, h, 0), *pk = row_of<IO>(a.k, b, h, 0);
#pragma unroll
        for (int r = 0; r < NK; ++r) {
            rq[r] = c0 + r < a.dk ? P::ld(pq + c0 + r) : P::zero();
            rk[r] = c0 + r < a.dk ? P::ld(pk + c0 + r) : P::zero();
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
    auto columns = [&](const typename P::raw (&x)[NK], f32x2 (&to2)[2]) {
        float f[4];
        if constexpr (V4) {
            P::cvt(x[0], f);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float one[1];
                P::cvt(x[r], one);
                f[r] = one[0];
            }
        }
        to2[0] = pack2(f[0], f[1]);
        to2[1] = pack2(f[2], f[3]);
    };
    fetch(b0);
    f32x2 A2[kStepRows][2];
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) {
        const float *row = a.A + ((long long)h * a.dv + ch0 + i * CPP) * a.dk + c0;
        float f[4] = {0.f, 0.f, 0.f, 0.f};
        if (V4) {
            if (there(i, 0)) Pack<float, 4>::cvt(Pack<float, 4>::ld(row), f);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (there(i, r)) f[r] = row[r];
        }
        A2[i][0] = pack2(decay_rate(f[0]), decay_rate(f[1]));
        A2[i][1] = pack2(decay_rate(f[2]), decay_rate(f[3]));
    }
#pragma unroll
    for (int j = 0; j < OWN; ++j) {
        const int ch = ch0 + (own + j) * CPP;
        bias[j] = ch < a.dv && a.delta_bias ? a.delta_bias[(long long)h * a.dv + ch] : 0.f;
        skip[j] = ch < a.dv && a.D ? a.D[(long long)h * a.dv + ch] : 0.f;
    }
    int place = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        float dt[OWN], dtv[OWN], vv[OWN], zz[OWN], y[kStepRows];
        f32x2 q[2], k[2];
#pragma unroll
        for (int j = 0; j < OWN; ++j) {
            const float x = raw[j] + bias[j];
            dt[j] = soft ? softplus(x) : x;
            dtv[j] = dt[j] * v[j];
            vv[j] = v[j];
            zz[j] = z[j];
        }
        columns(rq, q);
        columns(rk, k);
        if (b + 1 < b1) fetch(b + 1);
        // the place that is filled now was read a sequence ago
        ask(place == 0 ? kStepRing - 1 : place - 1, b1 - b > kStepRing - 1);
        copy_wait<kStepRing - 1>();
#pragma unroll
        for (int i = 0; i < kStepRows; ++i) {
            const float d = __shfl_sync(0xffffffffu, dt[i % OWN], keeper(i), G), x = __shfl_sync(0xffffffffu, dtv[i % OWN], keeper(i), G);
            const f32x2 d2 = pack2(d, d), x2 = pack2(x, x);
            f32x2 S[2];
            load_pairs(ring[place][i][tid], S[0], S[1]);
            S[0] = fma2(ex2_2(mul2(d2, A2[i][0])), S[0], mul2(x2, k[0]));
            S[1] = fma2(ex2_2(mul2(d2, A2[i][1])), S[1], mul2(x2, k[1]));
            y[i] = sum2(fma2(S[1], q[1], mul2(S[0], q[0])));
            float f[4];
            unpack2(S[0], f[0], f[1]);
            unpack2(S[1], f[2], f[3]);
            if (V4) {
                if (there(i, 0)) __stcs(reinterpret_cast<float4 *>(to + i * CPP * a.dk), make_float4(f[0], f[1], f[2], f[3]));
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (there(i, r)) __stcs(to + i * CPP * a.dk + r, f[r]);
            }
        }
        to += per;
        place = place + 1 == kStepRing ? 0 : place + 1;
        bool alone;
        lanes_sum<kStepRows, G, 1>(y, lane, alone);
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

template <typename IO, int ST, int SL, int MODE>
cudaError_t scan_pass_t(const falcon_scan_args_t &a, const ScanWork &w, cudaStream_t s) {
    const int cpb = kScanThreads / SL;
    const int ngrp = (a.dv + cpb - 1) / cpb;
    const int runs = MODE == kScanBoth ? (w.nwalk + w.block - 1) / w.block : w.nseg;
    const long long blocks = (long long)ngrp * a.B * a.H * runs;
    if (blocks > kMaxGrid) return cudaErrorInvalidConfiguration;
    const int es = sizeof(IO), V = 16 / es;
    bool wide = a.dv % V == 0 && view_packs(a.v, V, es) && view_packs(a.delta, V, es) && view_packs(a.z, V, es);
    if (MODE == kScanFull) wide = wide && view_packs(a.o, V, es);
    if (MODE == kScanBoth) wide = wide && view_packs(w.dO, 4, 4);
    if (wide) scan_kernel<IO, ST, SL, MODE, true><<<(unsigned)blocks, kScanThreads, 0, s>>>(a, w, ngrp);
    else scan_kernel<IO, ST, SL, MODE, false><<<(unsigned)blocks, kScanThreads, 0, s>>>(a, w, ngrp);
    return cudaGetLastError();
}

template <typename IO, int ST, int SL>
cudaError_t scan_pass_mode(int mode, const falcon_scan_args_t &a, const ScanWork &w, cudaStream_t s) {
    if (mode == kScanFull) return scan_pass_t<IO, ST, SL, kScanFull>(a, w, s);
    if (mode == kScanEnds) return scan_pass_t<IO, ST, SL, kScanEnds>(a, w, s);
    return scan_pass_t<IO, ST, SL, kScanBoth>(a, w, s);
}

template <typename IO>
cudaError_t scan_pass_io(int mode, const falcon_scan_args_t &a, const ScanWork &w, cudaStream_t s) {
    if (a.dk <= 4) return scan_pass_mode<IO, 4, 1>(mode, a, w, s);
    if (a.dk <= 8) return scan_pass_mode<IO, 8, 1>(mode, a, w, s);
    if (a.dk <= 16) return scan_pass_mode<IO, 16, 1>(mode, a, w, s);
    if (a.dk <= 32) return scan_pass_mode<IO, 16, 2>(mode, a, w, s);
    if (a.dk <= 64) return scan_pass_mode<IO, 16, 4>(mode, a, w, s);
    return scan_pass_mode<IO, 16, 8>(mode, a, w, s);
}

template <typename IO, int G>
cudaError_t scan_step_t(const falcon_scan_args_t &a, int num_sms, cudaStream_t s) {
    const int per = kStepThreads / G * kStepRows;
    const int ngrp = (a.dv + per - 1) / per;
    // sequences of a block: the number with the shortest estimate, in turns of the blocks that the SMs hold at once
    // (a block's start, with its rows of A, costs about one sequence). 256 sequences of H32 dv128: 10 to a block and
    // one turn 28 us; 8 and 1.2 turns 34, 4 and 2.3 turns 31, one and 9.2 turns 38.
    auto blocks_of = [&](int chunk) { return (long long)ngrp * a.H * ((a.B - 1LL + chunk) / chunk); };
    int chunk = 1;
    long long best = 0;
    for (int c = 1; c <= 32 && c <= a.B; ++c) {
        const long long cost = (blocks_of(c) + num_sms * kStepBlocks - 1) / (num_sms * kStepBlocks) * (c + 1);
        if (c == 1 || cost < best) {
            best = cost;
            chunk = c;
        }
    }
    const long long blocks = blocks_of(chunk);
    if (blocks > kMaxGrid) return cudaErrorInvalidConfiguration;
    const uintptr_t any = reinterpret_cast<uintptr_t>(a.S0) | reinterpret_cast<uintptr_t>(a.S_out) | reinterpret_cast<uintptr_t>(a.A);
    const bool v4 = a.dk % 4 == 0 && any % 16 == 0 && view_packs(a.q, 4, sizeof(IO)) && view_packs(a.k, 4, sizeof(IO));
    if (v4) scan_step_kernel<IO, G, true><<<(unsigned)blocks, kStepThreads, 0, s>>>(a, ngrp, chunk);
    else scan_step_kernel<IO, G, false><<<(unsigned)blocks, kStepThreads, 0, s>>>(a, ngrp, chunk);
    return cudaGetLastError();
}

template <typename IO>
cudaError_t scan_step_io(const falcon_scan_args_t &a, int num_sms, cudaStream_t s) {
    if (a.dk <= 4) return scan_step_t<IO, 1>(a, num_sms, s);
    if (a.dk <= 8) return scan_step_t<IO, 2>(a, num_sms, s);
    if (a.dk <= 16) return scan_step_t<IO, 4>(a, num_sms, s);
    if (a.dk <= 32) return scan_step_t<IO, 8>(a, num_sms, s);
    if (a.dk <= 64) return scan_step_t<IO, 16>(a, num_sms, s);
    return scan_step_t<IO, 32>(a, num_sms, s);
}

}  // namespace

cudaError_t launch_scan_pass(int mode, const falcon_scan_args_t &a, const ScanWork &w, cudaStream_t s) {
    return a.io_dtype == FALCON_BF16 ? scan_pass_io<__nv_bfloat16>(mode, a, w, s) : scan_pass_io<float>(mode, a, w, s);
}

// Segments: the number with the shortest estimate. A token takes a block alone on its SM 1.75 times what it takes
// one of several (measured at dk = 16: 380 cycles against 219 for each), so k blocks on an SM take max(1.75, k) a token.
// Both passes over a segment of L tokens are 1.8 L tokens' work (the first forms no outputs) and each join of a
// state before it about one. Unsplit, the pass is T tokens' work. Other widths go by the same numbers: bf16 B2 H16 T2048
// dk64 dv128 517 us as it splits it, 592 unsplit.
ScanPlan scan_plan(const falcon_scan_args_t &a, int num_sms) {
    constexpr long long kMinSeg = 32;
    ScanPlan p;
    p.seg = a.T;
    const int sl = a.dk <= 16 ? 1 : a.dk <= 32 ? 2 : a.dk <= 64 ? 4 : 8;
    const long long bh = (long long)a.B * a.H, cpb = kScanThreads / sl;
    const long long groups = bh * ((a.dv + cpb - 1) / cpb);
    if (groups == 0 || a.T < 2 * kMinSeg) return p;
    auto token = [&](long long blocks) {
        const long long k = (blocks + num_sms - 1) / num_sms;
        return k <= 1 ? 1.75 : (double)k;
    };
    double best = (double)a.T * token(groups);
    long long nseg = 1;
    for (int k = 1; k <= 8; ++k) {
        long long n = (long long)num_sms * k / groups;
        if (n > a.T / kMinSeg) n = a.T / kMinSeg;
        if (n < 2) continue;
        const double cost = (1.8 * (double)a.T / n + 0.5 * n) * token(groups * n);
        if (cost < best) {
            best = cost;
            nseg = n;
        }
    }
    if (nseg == 1) return p;
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

cudaError_t launch_scan_step(const falcon_scan_args_t &a, int num_sms, cudaStream_t s) {
    if ((long long)a.B * a.H == 0) return cudaSuccess;
    return a.io_dtype == FALCON_BF16 ? scan_step_io<__nv_bfloat16>(a, num_sms, s) : scan_step_io<float>(a, num_sms, s);
}

}  // namespace falcon
