// qknorm.cu -- falcon_qknorm_fwd / falcon_qknorm_bwd: the norm of every head's query and key rows with
// the rotation by position in the same pass.
//
// A row is read once and written once for a few flops an element: bound by HBM. A row of d channels
// belongs to LANES neighbouring lanes with NV packs of V channels each (16 bytes, or 8 of bf16), so a warp
// moves whole rows; the sum of squares comes from shuffles. Both channels of a rotated pair are in one lane: a
// pack of FALCON_ROT_HALF is V / 2 channels of the lower half and the V / 2 that turn with them (two 8-byte
// accesses; exchanging packs between lanes took a shuffle for every channel: 98 us instead of 94 for B8 H16+16
// T4096 d128 in bf16; with the weights folded into the rotation and two channels an instruction it is 90, 6 TB/s).
// A group of LANES lanes takes one token and walks its heads, kRows of them in flight: the
// token's sines and cosines, the same for every head, are formed once by the block (the angle's whole turns
// taken off in fp64), kept in registers over the walk, and the row addresses advance by one addition.
// Where pointers, strides, d or rot are not multiples of a pack, V = 1: lane l owns channels l, l + 32, ..
// and partners come through shared memory (the same case with rows off alignment: 182 us in all against 97).
// Few heads a token pay badly for its angles: B4 H4+1 T8192 d128 32 us against 13 at the copy rate, B1 H8+2 18 against 6.
// Backward: the same walk with the row turned back; dwq and dwk are summed per lane over the tokens of a
// block, then over blocks by a second launch. B4 H16+4 T2048 d128: 44 us and 6 us of kernels for
// 210 MB (32 us at the copy rate), 82 us in all off alignment; bound by instruction latency, 16 warps an SM (the registers of two rows and their prefetch).
#include "ops.cuh"

namespace falcon {

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormWarps = kNormThreads / 32;
constexpr int kMaxWidth = 256;
constexpr double kTwoOverPi = 0.63661977236758134308;

struct NormShape {
    long long groups;   // ceil(B T / tokens of a block): one token for each group of lanes
    // forward: a block takes `heads` heads of its tokens, blockIdx.y of them
    int heads, parts;
    // backward: the list of (group of tokens, head), heads fastest, cut into equal stretches, one for each of the
    // blocks that the SMs hold at once (so the parts of dwq and dwk are few, and no block is left with half a
    // turn; forward, where blocks carry nothing over, blocks in plenty took 90 us against 117 for this)
    long long units;
    int blocks;
};

// Where pair p's (cos, sin) lies. V > 1: V / 2 pairs a pack, two of them in 16 bytes, [two pairs of the
// pack][pack], so that the lanes of a row read neighbouring words.
template <int V>
__device__ __forceinline__ int turn_slot(const falcon_qknorm_args_t &a, int p) {
    if (V == 1) return p;
    constexpr int H = V > 1 ? V / 2 : 1;
    const int packs = (a.rot + V - 1) / V;
    return ((p % H) / 2 * packs + p / H) * 2 + (p & 1);
}
// Slots of a token (the last pack may be padded).
__host__ __device__ inline int turn_slots(const falcon_qknorm_args_t &a, int V) {
    return V == 1 ? a.rot / 2 : (a.rot + V - 1) / V * (V / 2);
}

// (cos, sin) of t quarter turns: whole ones are taken off in fp64, and the rest f, |f| <= 1/2, goes into polynomials in
// f^2 for sin(f pi/2) / f and cos(f pi/2) (least-squares fits on [0, 1/4], good to 3e-9). The library's sine and
// cosine in its place: 34.4 us against 32.8 for a case of 5 heads with d 256, whose angles few rows share.
__device__ __forceinline__ float2 turned(double t) {
    const double whole = rint(t);
    const float f = (float)(t - whole), u = f * f;
    float s = fmaf(u, -0.0046016579f, 0.079680033f);
    s = fmaf(u, s, -0.64596349f);
    s = f * fmaf(u, s, 1.5707964f);
    float c = fmaf(u, 0.00090402167f, -0.020860288f);
    c = fmaf(u, c, 0.25366923f);
    c = fmaf(u, c, -1.2337005f);
    c = fmaf(u, c, 1.f);
    const int q = (int)__double2ll_rn(whole) & 3;
    const float x = q & 1 ? -s : c, y = q & 1 ? c : s;
    return q & 2 ? make_float2(-x, -y) : make_float2(x, y);
}

// Sines and cosines of `tokens` tokens from tok0 on. Padded pairs turn by nothing.
template <int V>
__device__ __forceinline__ void angles(const falcon_qknorm_args_t &a, long long tok0, int tokens, float2 *cs) {
    const int slots = turn_slots(a, V), half = a.rot / 2;
    const long long all = (long long)a.B * a.T;
    for (int i = threadIdx.x; i < tokens * slots; i += kNormThreads) {
        const int j = i / slots, p = i % slots;
        const long long tok = tok0 + j;
        float2 r = make_float2(1.f, 0.f);
        if (tok < all && p < half) {
            const double pos = a.positions ? (double)a.positions[tok] : (double)(tok % a.T);
            r = turned(pos * (double)a.freq[p] * kTwoOverPi);
        }
        cs[j * slots + turn_slot<V>(a, p)] = r;
    }
}

// 1 / root of a row with sum of squares ss; scale is 1 / d for FALCON_NORM_RMS, else 1.
__device__ __forceinline__ float root_inverse(const falcon_qknorm_args_t &a, float ss, float scale) {
    if (a.norm == FALCON_NORM_NONE) return 1.f;
    const float m = fmaf(ss, scale, a.eps);
    return m == 0.f ? 0.f : rsqrtf(m);
}

template <int LANES>
__device__ __forceinline__ float lanes_total(float x) {
#pragma unroll
    for (int m = 1; m < LANES; m <<= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// A pack of a row in registers: the first channels of its pairs, then the second ones. `row` points at the row's
// first channel.
template <typename E, int V, bool HALF> struct Row {
    static constexpr int H = V / 2;
    typedef Pack<E, H> P;
    struct raw { typename P::raw a, b; };
    static __device__ __forceinline__ int first(int p, int rot) { return HALF && p * V < rot ? p * H : p * V; }
    static __device__ __forceinline__ int second(int p, int rot) { return HALF && p * V < rot ? rot / 2 + p * H : p * V + H; }
    static __device__ __forceinline__ int channel(int p, int i, int rot) {
        if (!HALF) return p * V + (i < H ? 2 * i : 2 * (i - H) + 1);
        return i < H ? first(p, rot) + i : second(p, rot) + i - H;
    }
    // where a pack's halves lie, formed once for all rows
    struct Place {
        int a, b;
        __device__ __forceinline__ Place(int p, int rot) : a(first(p, rot)), b(second(p, rot)) {}
    };
    static __device__ __forceinline__ raw zero() { return raw{P::zero(), P::zero()}; }
    static __device__ __forceinline__ raw ld(const E *row, Place at) { return raw{P::ld(row + at.a), P::ld(row + at.b)}; }
    static __device__ __forceinline__ void cvt(const raw &r, float (&x)[V]) {
        float u[H], v[H];
        P::cvt(r.a, u);
        P::cvt(r.b, v);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float y = HALF ? (i < H ? u[i % H] : v[i % H]) : (channel(0, i, 0) < H ? u[channel(0, i, 0) % H] : v[channel(0, i, 0) % H]);
            x[i] = y;
        }
    }
    static __device__ __forceinline__ void st(E *row, Place at, const float (&x)[V]) {
        float u[H], v[H];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int j = HALF ? i : channel(0, i, 0);
            if (j < H) u[j % H] = x[i];
            else v[j % H] = x[i];
        }
        P::st(row + at.a, u);
        P::st(row + at.b, v);
    }
};
template <typename E, bool HALF> struct Row<E, 1, HALF> {
    typedef Pack<E, 1> P;
    typedef typename P::raw raw;
    struct Place {
        int a;
        __device__ __forceinline__ Place(int p, int) : a(p) {}
    };
    static __device__ __forceinline__ int channel(int p, int, int) { return p; }
    static __device__ __forceinline__ raw zero() { return P::zero(); }
    static __device__ __forceinline__ raw ld(const E *row, Place at) { return P::ld(row + at.a); }
    static __device__ __forceinline__ void cvt(raw r, float (&x)[1]) { P::cvt(r, x); }
    static __device__ __forceinline__ void st(E *row, Place at, const float (&x)[1]) { P::st(row + at.a, x); }
};

// Pairs 2 i and 2 i + 1 of pack p where they turn, 0 where they do not: there a sine of 0 times a partner that is not
// finite would be NaN. (FALCON_ROT_HALF: all of a pack's pairs turn, or none.)
template <int V>
__device__ __forceinline__ f32x2 turning(f32x2 x, int p, int i, int rot) {
    float lo, hi;
    unpack2(x, lo, hi);
    const int first = p * V + 4 * i;
    return pack2(first < rot ? lo : 0.f, first + 2 < rot ? hi : 0.f);
}

// A lane's part of a token's rotation: the factors of its pairs.
template <int V, int LANES, int NV, bool HALF, bool SOME> struct Turn {
    static constexpr int H = V / 2;
    float c[NV][H], s[NV][H];
    __device__ __forceinline__ void load(const falcon_qknorm_args_t &a, int lane, const float2 *cs, float sign) {
        const int packs = (a.rot + V - 1) / V;
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int p = lane + m * LANES;
#pragma unroll
            for (int i = 0; i < H; i += 2) {
                float4 r = make_float4(1.f, 0.f, 1.f, 0.f);
                if (p < packs) r = reinterpret_cast<const float4 *>(cs)[i / 2 * packs + p];
                c[m][i] = r.x;
                s[m][i] = sign * r.y;
                c[m][i + 1 < H ? i + 1 : i] = r.z;
                s[m][i + 1 < H ? i + 1 : i] = sign * r.w;
            }
        }
    }
    __device__ __forceinline__ void apply(float (&n)[NV][V], int, float *) const {
#pragma unroll
        for (int m = 0; m < NV; ++m)
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const float x1 = n[m][i], x2 = n[m][H + i];
                n[m][i] = fmaf(x1, c[m][i], -x2 * s[m][i]);
                n[m][H + i] = fmaf(x2, c[m][i], x1 * s[m][i]);
            }
    }
};
// One channel a pack: the factor of the channel itself, its partner, and the partner's factor with its sign. SOME:
// channels that do not turn have the 0 behind the row for a partner.
template <int LANES, int NV, bool HALF, bool SOME> struct Turn<1, LANES, NV, HALF, SOME> {
    float c[NV], s[NV];
    int from[NV];
    __device__ __forceinline__ void load(const falcon_qknorm_args_t &a, int lane, const float2 *cs, float sign) {
        const int half = a.rot / 2;
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int p = lane + m * LANES;
            c[m] = 1.f;
            s[m] = 0.f;
            from[m] = SOME ? kMaxWidth : p;
            if (p < a.rot) {
                const bool hi = HALF ? p >= half : (p & 1) != 0;
                from[m] = HALF ? (hi ? p - half : p + half) : p ^ 1;
                const float2 r = cs[HALF ? (hi ? p - half : p) : p / 2];
                c[m] = r.x;
                s[m] = (hi ? sign : -sign) * r.y;
            }
        }
    }
    __device__ __forceinline__ void apply(float (&n)[NV][1], int lane, float *stage) const {   // stage: the warp's row
        __syncwarp();
#pragma unroll
        for (int m = 0; m < NV; ++m) stage[lane + m * LANES] = n[m][0];
        __syncwarp();
#pragma unroll
        for (int m = 0; m < NV; ++m) n[m][0] = fmaf(n[m][0], c[m], stage[from[m]] * s[m]);
    }
};

// Which channels turn: none, each one, those of whole packs (as in halves they always are), or some. A pair that does not
// turn must not see its partner (a sine of 0 times infinity is NaN), and choosing costs registers, so each is compiled on
// its own; of single channels only the first two and the last.
enum TurnKind : int { kTurnNone, kTurnAll, kTurnPacks, kTurnSome };

// Blocks an SM that the last two are held to (0: as it comes), measured on bf16 B8 H16+16 T4096. Some of a pack's pairs:
// d64 with 6 turned, in packs of four, six 51 us, as it comes 58; in packs of eight four 95, as it comes (three) 103. Whole
// packs: as it comes 94, four 102; fp32 B8 H8+8 in pairs five 88, as it comes (four) 90; in halves it comes with five.
// One channel a pack, d 199 fp32: four 93, as it comes 101.
constexpr int fwd_blocks(int es, int V, int NV, bool half, int turn) {
    if (turn < kTurnPacks) return 0;
    if (V == 1) return NV == 8 ? 4 : 0;
    if (NV > 1) return 0;
    if (turn == kTurnPacks) return es == 4 && !half ? 5 : 0;
    return V == 8 ? 4 : es == 2 ? 6 : 5;
}

template <typename IO, int V, int LANES, int NV, bool HALF, int TURN>
__global__ void __launch_bounds__(kNormThreads, fwd_blocks(sizeof(IO), V, NV, HALF, TURN)) qknorm_fwd_kernel(falcon_qknorm_args_t a, NormShape s) {
    typedef Row<IO, V, HALF> R;
    constexpr int G = kNormThreads / LANES;       // groups of lanes, tokens of a block
    constexpr int kRows = NV >= 4 ? 1 : 4 / NV;   // rows in flight
    extern __shared__ __align__(16) float2 cs[];
    __shared__ float stage_all[V == 1 ? kNormWarps : 1][V == 1 ? kMaxWidth + (TURN == kTurnSome) : 1];
    float *stage = stage_all[V == 1 ? threadIdx.x >> 5 : 0];
    if (V == 1 && TURN == kTurnSome && threadIdx.x % 32 == 0) stage[kMaxWidth] = 0.f;   // read behind a row's barriers
    const long long tok0 = (long long)blockIdx.x * G;
    const int lane = threadIdx.x % LANES, slot = threadIdx.x / LANES;
    Turn<V, LANES, NV, HALF, TURN == kTurnSome> turn;
    if (a.rot > 0) {
        angles<V>(a, tok0, G, cs);
        __syncthreads();
        turn.load(a, lane, cs + slot * turn_slots(a, V), 1.f);
    }
    const long long tok = tok0 + slot;
    bool live = tok < (long long)a.B * a.T;
    const int b = live ? (int)(tok / a.T) : 0, t = live ? (int)(tok - (long long)b * a.T) : 0;
    live = live && t < seq_length(a.lengths, b, a.T);
    const int h0 = blockIdx.y * s.heads, h1 = min(h0 + s.heads, a.Hq + a.Hk);
    const float scale = a.norm == FALCON_NORM_RMS ? 1.f / (float)a.d : 1.f;
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {      // queries, then keys
        const falcon_view_t &in = which ? a.k : a.q, &out = which ? a.k_out : a.q_out;
        const float *weight = which ? a.wk : a.wq;
        const int first = which ? max(h0 - a.Hq, 0) : h0, last = which ? h1 - a.Hq : min(h1, a.Hq);
        if (first >= last) continue;
        float w[NV][V];
#pragma unroll
        for (int m = 0; m < NV; ++m)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int p = lane + m * LANES;
                w[m][i] = weight && p * V < a.d ? weight[R::channel(p, i, a.rot)] : 1.f;
            }
        // the weights go into the rotation: a pair (x1, x2) becomes (x1 c1 - x2 s2, x2 c2 + x1 s1) / root
        constexpr int Q = V > 1 ? V / 4 : 1;
        f32x2 c1[NV][Q], s1[NV][Q], c2[NV][Q], s2[NV][Q];
        if constexpr (V > 1) {
#pragma unroll
            for (int m = 0; m < NV; ++m)
#pragma unroll
                for (int i = 0; i < Q; ++i) {
                    constexpr int H = V / 2;
                    const int j = 2 * i;
                    const float ca = a.rot > 0 ? turn.c[m][j] : 1.f, cb = a.rot > 0 ? turn.c[m][j + 1] : 1.f;
                    const float sa = a.rot > 0 ? turn.s[m][j] : 0.f, sb = a.rot > 0 ? turn.s[m][j + 1] : 0.f;
                    c1[m][i] = pack2(w[m][j] * ca, w[m][j + 1] * cb);
                    s1[m][i] = pack2(w[m][j] * sa, w[m][j + 1] * sb);
                    c2[m][i] = pack2(w[m][H + j] * ca, w[m][H + j + 1] * cb);
                    s2[m][i] = pack2(-w[m][H + j] * sa, -w[m][H + j + 1] * sb);
                }
        }
        const IO *px = row_of<IO>(in, b, first, t);
        IO *po = row_of<IO>(out, b, first, t);
        for (int h = first; h < last; h += kRows) {
            typename R::raw raw[kRows][NV];
#pragma unroll
            for (int r = 0; r < kRows; ++r)
#pragma unroll
                for (int m = 0; m < NV; ++m) {
                    raw[r][m] = R::zero();
                    if (live && h + r < last && (lane + m * LANES) * V < a.d)
                        raw[r][m] = R::ld(px + r * in.sh, typename R::Place(lane + m * LANES, a.rot));
                }
            px += kRows * in.sh;
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                float x[NV][V];
#pragma unroll
                for (int m = 0; m < NV; ++m) R::cvt(raw[r][m], x[m]);
                if constexpr (V > 1) {
                    constexpr int H = V / 2;
                    f32x2 x1[NV][Q], x2[NV][Q], sq = 0ull;
#pragma unroll
                    for (int m = 0; m < NV; ++m)
#pragma unroll
                        for (int i = 0; i < Q; ++i) {
                            x1[m][i] = pack2(x[m][2 * i], x[m][2 * i + 1]);
                            x2[m][i] = pack2(x[m][H + 2 * i], x[m][H + 2 * i + 1]);
                            sq = fma2(x1[m][i], x1[m][i], sq);
                            sq = fma2(x2[m][i], x2[m][i], sq);
                        }
                    const float ri = root_inverse(a, a.norm == FALCON_NORM_NONE ? 0.f : lanes_total<LANES>(sum2(sq)), scale);
                    const f32x2 ri2 = pack2(ri, ri);
#pragma unroll
                    for (int m = 0; m < NV; ++m)
#pragma unroll
                        for (int i = 0; i < Q; ++i) {
                            f32x2 y1, y2;
                            if (TURN == kTurnNone) {
                                y1 = mul2(ri2, mul2(x1[m][i], c1[m][i]));
                                y2 = mul2(ri2, mul2(x2[m][i], c2[m][i]));
                            } else {
                                f32x2 z1 = 0ull, z2 = 0ull;
                                if (TURN == kTurnAll || (lane + m * LANES) * V < a.rot) {
                                    z1 = mul2(x2[m][i], s2[m][i]);
                                    z2 = mul2(x1[m][i], s1[m][i]);
                                    if (TURN == kTurnSome) {   // the last pack's pairs may turn in part
                                        z1 = turning<V>(z1, lane + m * LANES, i, a.rot);
                                        z2 = turning<V>(z2, lane + m * LANES, i, a.rot);
                                    }
                                }
                                y1 = mul2(ri2, fma2(x1[m][i], c1[m][i], z1));
                                y2 = mul2(ri2, fma2(x2[m][i], c2[m][i], z2));
                            }
                            unpack2(y1, x[m][2 * i], x[m][2 * i + 1]);
                            unpack2(y2, x[m][H + 2 * i], x[m][H + 2 * i + 1]);
                        }
                } else {
                    float ss = 0.f;
#pragma unroll
                    for (int m = 0; m < NV; ++m) ss = fmaf(x[m][0], x[m][0], ss);
                    const float ri = root_inverse(a, a.norm == FALCON_NORM_NONE ? 0.f : lanes_total<LANES>(ss), scale);
#pragma unroll
                    for (int m = 0; m < NV; ++m) x[m][0] = x[m][0] * ri * w[m][0];
                    if (a.rot > 0) turn.apply(x, lane, stage);
                }
                if (live && h + r < last) {
#pragma unroll
                    for (int m = 0; m < NV; ++m)
                        if ((lane + m * LANES) * V < a.d) R::st(po + r * out.sh, typename R::Place(lane + m * LANES, a.rot), x[m]);
                }
            }
            po += kRows * out.sh;
        }
    }
}

template <typename IO, int V, int LANES, int NV, bool HALF, int TURN>
__global__ void __launch_bounds__(kNormThreads, NV == 1 ? 2 : 1) qknorm_bwd_kernel(falcon_qknorm_args_t a, falcon_qknorm_grads_t g, NormShape s,
                                                                  float *part) {
    typedef Row<IO, V, HALF> R;
    typedef Row<float, V, HALF> F;
    constexpr int G = kNormThreads / LANES;
    constexpr int kRows = NV > 1 ? 1 : 2;   // rows worked on together, as many more on their way
    extern __shared__ __align__(16) float2 cs[];
    __shared__ float stage_all[V == 1 ? kNormWarps : 1][V == 1 ? kMaxWidth + (TURN == kTurnSome) : 1];
    __shared__ float sw[2][kMaxWidth];
    float *stage = stage_all[V == 1 ? threadIdx.x >> 5 : 0];
    if (V == 1 && TURN == kTurnSome && threadIdx.x % 32 == 0) stage[kMaxWidth] = 0.f;   // read behind a row's barriers
    const int lane = threadIdx.x % LANES, slot = threadIdx.x / LANES;
    const int heads = a.Hq + a.Hk;
    const bool plain = TURN != kTurnAll && a.norm == FALCON_NORM_NONE;   // dx is u then, whatever x is
    const float scale = a.norm == FALCON_NORM_RMS ? 1.f / (float)a.d : 1.f;
    constexpr int NP = V > 1 ? V / 2 : 1;
    f32x2 dw2[2][NV][NP];   // V > 1: the first channels of the pairs, then the second
    float dw[2][NV];        // V = 1
#pragma unroll
    for (int m = 0; m < NV; ++m) {
        dw[0][m] = dw[1][m] = 0.f;
#pragma unroll
        for (int i = 0; i < NP; ++i) dw2[0][m][i] = dw2[1][m][i] = 0ull;
    }
    const long long u_end = s.units * (blockIdx.x + 1) / s.blocks;
    int h0 = 0, h1 = 0;
    for (long long at = s.units * blockIdx.x / s.blocks; at < u_end; at += h1 - h0) {
        const long long tok0 = at / heads * G;
        h0 = (int)(at % heads);
        h1 = (int)(u_end - at < heads - h0 ? h0 + (u_end - at) : heads);
        const long long tok = tok0 + slot;
        const bool there = tok < (long long)a.B * a.T;
        const int b = there ? (int)(tok / a.T) : 0, t = there ? (int)(tok - (long long)b * a.T) : 0;
        const bool live = there && t < seq_length(a.lengths, b, a.T);

        Turn<V, LANES, NV, HALF, TURN == kTurnSome> turn;
        if (a.rot > 0) {
            __syncthreads();
            angles<V>(a, tok0, G, cs);
            __syncthreads();
            turn.load(a, lane, cs + slot * turn_slots(a, V), -1.f);
        }
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const falcon_view_t &in = which ? a.k : a.q, &up = which ? g.dk_out : g.dq_out, &to = which ? g.dk : g.dq;
            const float *weight = which ? a.wk : a.wq;
            const int first = which ? max(h0 - a.Hq, 0) : h0, last = which ? h1 - a.Hq : min(h1, a.Hq);
            if (first >= last) continue;
            float w[NV][V];
#pragma unroll
            for (int m = 0; m < NV; ++m)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int p = lane + m * LANES;
                    w[m][i] = weight && p * V < a.d ? weight[R::channel(p, i, a.rot)] : 1.f;
                }
            const IO *px = row_of<IO>(in, b, first, t);
            const float *pu = row_of<float>(up, b, first, t);
            float *po = row_of<float>(to, b, first, t);
            typename R::raw rx[kRows][NV];
            typename F::raw ru[kRows][NV];
            auto fetch = [&](int h) {
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
#pragma unroll
                    for (int m = 0; m < NV; ++m) {
                        const int p = lane + m * LANES;
                        rx[r][m] = R::zero();
                        ru[r][m] = F::zero();
                        if (live && h + r < last && p * V < a.d) {
                            rx[r][m] = R::ld(px, typename R::Place(p, a.rot));
                            ru[r][m] = F::ld(pu, typename F::Place(p, a.rot));
                        }
                    }
                    px += in.sh;
                    pu += up.sh;
                }
            };
            fetch(first);
            for (int h = first; h < last; h += kRows) {
                typename R::raw cx[kRows][NV];
                typename F::raw cu[kRows][NV];
#pragma unroll
                for (int r = 0; r < kRows; ++r)
#pragma unroll
                    for (int m = 0; m < NV; ++m) {
                        cx[r][m] = rx[r][m];
                        cu[r][m] = ru[r][m];
                    }
                if (h + kRows < last) fetch(h + kRows);
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    float x[NV][V], u[NV][V];
#pragma unroll
                    for (int m = 0; m < NV; ++m) {
                        R::cvt(cx[r][m], x[m]);
                        F::cvt(cu[r][m], u[m]);
                    }
                    if constexpr (V > 1) {   // two channels an instruction
                        constexpr int H = V / 2, Q = V / 4;
                        f32x2 x1[NV][Q], x2[NV][Q], u1[NV][Q], u2[NV][Q], sum = 0ull;
#pragma unroll
                        for (int m = 0; m < NV; ++m)
#pragma unroll
                            for (int i = 0; i < Q; ++i) {
                                x1[m][i] = pack2(x[m][2 * i], x[m][2 * i + 1]);
                                x2[m][i] = pack2(x[m][H + 2 * i], x[m][H + 2 * i + 1]);
                                sum = fma2(x1[m][i], x1[m][i], sum);
                                sum = fma2(x2[m][i], x2[m][i], sum);
                            }
                        const float ri = root_inverse(a, a.norm == FALCON_NORM_NONE ? 0.f : lanes_total<LANES>(sum2(sum)), scale);
                        const f32x2 ri2 = pack2(ri, ri);
                        sum = 0ull;
#pragma unroll
                        for (int m = 0; m < NV; ++m)
#pragma unroll
                            for (int i = 0; i < Q; ++i) {
                                u1[m][i] = pack2(u[m][2 * i], u[m][2 * i + 1]);
                                u2[m][i] = pack2(u[m][H + 2 * i], u[m][H + 2 * i + 1]);
                                if (TURN == kTurnAll || (TURN != kTurnNone && (lane + m * LANES) * V < a.rot)) {
                                    const f32x2 c = pack2(turn.c[m][2 * i], turn.c[m][2 * i + 1]);
                                    const f32x2 sn = pack2(turn.s[m][2 * i], turn.s[m][2 * i + 1]);
                                    const f32x2 ns = pack2(-turn.s[m][2 * i], -turn.s[m][2 * i + 1]);
                                    f32x2 z1 = mul2(u2[m][i], ns), z2 = mul2(u1[m][i], sn);
                                    if (TURN == kTurnSome) {   // the last pack's pairs may turn in part
                                        z1 = turning<V>(z1, lane + m * LANES, i, a.rot);
                                        z2 = turning<V>(z2, lane + m * LANES, i, a.rot);
                                    }
                                    u1[m][i] = fma2(u1[m][i], c, z1);
                                    u2[m][i] = fma2(u2[m][i], c, z2);
                                }
                                x1[m][i] = mul2(x1[m][i], ri2);
                                x2[m][i] = mul2(x2[m][i], ri2);
                                if (part) {      // rows that are not there are zero
                                    dw2[which][m][i] = fma2(u1[m][i], x1[m][i], dw2[which][m][i]);
                                    dw2[which][m][Q + i] = fma2(u2[m][i], x2[m][i], dw2[which][m][Q + i]);
                                }
                                u1[m][i] = mul2(u1[m][i], pack2(w[m][2 * i], w[m][2 * i + 1]));
                                u2[m][i] = mul2(u2[m][i], pack2(w[m][H + 2 * i], w[m][H + 2 * i + 1]));
                                sum = fma2(u1[m][i], x1[m][i], sum);
                                sum = fma2(u2[m][i], x2[m][i], sum);
                            }
                        const float dot = a.norm == FALCON_NORM_NONE ? 0.f : -lanes_total<LANES>(sum2(sum)) * scale;
                        const f32x2 dot2 = pack2(dot, dot);
#pragma unroll
                        for (int m = 0; m < NV; ++m)
#pragma unroll
                            for (int i = 0; i < Q; ++i) {
                                const f32x2 xa = plain ? 0ull : x1[m][i], xb = plain ? 0ull : x2[m][i];
                                unpack2(mul2(ri2, fma2(xa, dot2, u1[m][i])), u[m][2 * i], u[m][2 * i + 1]);
                                unpack2(mul2(ri2, fma2(xb, dot2, u2[m][i])), u[m][H + 2 * i], u[m][H + 2 * i + 1]);
                            }
                    } else {
                        float ss = 0.f, dot = 0.f;
#pragma unroll
                        for (int m = 0; m < NV; ++m) ss = fmaf(x[m][0], x[m][0], ss);
                        const float ri = root_inverse(a, a.norm == FALCON_NORM_NONE ? 0.f : lanes_total<LANES>(ss), scale);
                        if (a.rot > 0) turn.apply(u, lane, stage);
#pragma unroll
                        for (int m = 0; m < NV; ++m) {
                            x[m][0] *= ri;
                            dw[which][m] = fmaf(u[m][0], x[m][0], dw[which][m]);
                            u[m][0] *= w[m][0];
                            dot = fmaf(u[m][0], x[m][0], dot);
                        }
                        dot = a.norm == FALCON_NORM_NONE ? 0.f : -lanes_total<LANES>(dot) * scale;
#pragma unroll
                        for (int m = 0; m < NV; ++m) u[m][0] = ri * fmaf(plain ? 0.f : x[m][0], dot, u[m][0]);
                    }
                    if (there && h + r < last) {
#pragma unroll
                        for (int m = 0; m < NV; ++m) {
                            if (!live)
#pragma unroll
                                for (int i = 0; i < V; ++i) u[m][i] = 0.f;
                            if ((lane + m * LANES) * V < a.d) F::st(po, typename F::Place(lane + m * LANES, a.rot), u[m]);
                        }
                    }
                    po += to.sh;
                }
            }
        }
    }
    if (!part) return;
    // the block's sums, lane group by lane group in order
    for (int i = threadIdx.x; i < 2 * kMaxWidth; i += kNormThreads) sw[i / kMaxWidth][i % kMaxWidth] = 0.f;
    for (int k = 0; k < G; ++k) {
        __syncthreads();
        if (slot == k) {
#pragma unroll
            for (int m = 0; m < NV; ++m) {
                const int p = lane + m * LANES;
                if (p * V < a.d)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const int e = R::channel(p, i, a.rot);
                        float lo[2], hi[2];
                        unpack2(dw2[0][m][i / 2 % NP], lo[0], hi[0]);
                        unpack2(dw2[1][m][i / 2 % NP], lo[1], hi[1]);
                        sw[0][e] += V == 1 ? dw[0][m] : i & 1 ? hi[0] : lo[0];
                        sw[1][e] += V == 1 ? dw[1][m] : i & 1 ? hi[1] : lo[1];
                    }
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.d; i += kNormThreads)
        part[(long long)blockIdx.x * 2 * a.d + i] = sw[i / a.d][i % a.d];
}

// The pack's width: 16 bytes of the io type where every row and the rotation allow it (accesses are of half a pack), for
// bf16 also 8; else one channel (d 28, all of it rotated, backward: 34 us in packs of 8 bytes, 159 in single channels;
// d 64 with 6 rotated, forward: 33 us against 58).
int norm_pack(const falcon_qknorm_args_t &a, const falcon_qknorm_grads_t *g) {
    const int es = a.io_dtype == FALCON_BF16 ? 2 : 4;
    for (int V = 16 / es; V >= 4; V /= 2) {
        const int H = V / 2;
        bool ok = a.d % V == 0 && view_packs(a.q, H, es) && view_packs(a.k, H, es);
        if (a.rot_layout == FALCON_ROT_HALF) ok = ok && a.rot % V == 0;
        if (!g) ok = ok && view_packs(a.q_out, H, es) && view_packs(a.k_out, H, es);
        else ok = ok && view_packs(g->dq_out, H, 4) && view_packs(g->dk_out, H, 4) && view_packs(g->dq, H, 4) && view_packs(g->dk, H, 4);
        if (ok) return V;
    }
    return 1;
}

int norm_lanes(const falcon_qknorm_args_t &a, int V) {
    const int packs = a.d / V;
    return V == 1 || packs > 16 ? 32 : packs > 8 ? 16 : packs > 4 ? 8 : 4;
}

constexpr int kBwdBlocks = 148 * 2;

// Forward, a token's heads go to several blocks while there are fewer than kWanted threads (three quarters of what
// the GPU holds).
NormShape norm_shape(const falcon_qknorm_args_t &a, int lanes) {
    constexpr long long kWanted = 148LL * 1536;
    constexpr int kMaxParts = 65535;   // of a grid's second axis
    NormShape s;
    const int heads = a.Hq + a.Hk, per = kNormThreads / lanes;
    const long long all = (long long)a.B * a.T;
    s.groups = (all + per - 1) / per;
    s.heads = heads;
    s.parts = 1;
    while (s.heads > 1 && all * lanes * s.parts < kWanted) {
        const int fewer = (s.heads + 1) / 2, parts = (heads + fewer - 1) / fewer;
        if (parts > kMaxParts) break;
        s.heads = fewer;
        s.parts = parts;
    }
    s.units = s.groups * heads;
    s.blocks = (int)(s.units < kBwdBlocks ? s.units : kBwdBlocks);
    return s;
}

template <typename IO, int V, int LANES, int NV, bool HALF, int TURN>
cudaError_t norm_launch(const falcon_qknorm_args_t &a, const falcon_qknorm_grads_t *g, float *part, cudaStream_t st) {
    const NormShape s = norm_shape(a, LANES);
    const size_t smem = (size_t)(kNormThreads / LANES) * turn_slots(a, V) * sizeof(float2);
    if (g) {
        qknorm_bwd_kernel<IO, V, LANES, NV, HALF, TURN><<<s.blocks, kNormThreads, smem, st>>>(a, *g, s, part);
    } else {
        if (s.groups > kMaxGrid) return cudaErrorInvalidConfiguration;
        qknorm_fwd_kernel<IO, V, LANES, NV, HALF, TURN><<<dim3((unsigned)s.groups, (unsigned)s.parts), kNormThreads, smem, st>>>(a, s);
    }
    return cudaGetLastError();
}

template <typename IO, int V, int LANES, int NV, bool HALF>
cudaError_t norm_run(const falcon_qknorm_args_t &a, const falcon_qknorm_grads_t *g, float *part, cudaStream_t st) {
    if (a.rot == 0) {   // halves then, see norm_any
        if constexpr (HALF) return norm_launch<IO, V, LANES, NV, HALF, kTurnNone>(a, g, part, st);
    } else if (a.rot == a.d && !(g && a.norm == FALCON_NORM_NONE)) {   // (without a norm the gradient has to choose as well)
        return norm_launch<IO, V, LANES, NV, HALF, kTurnAll>(a, g, part, st);
    }
    if constexpr (V > 1 && !HALF) {
        if (a.rot % V == 0) return norm_launch<IO, V, LANES, NV, HALF, kTurnPacks>(a, g, part, st);
    }
    return norm_launch<IO, V, LANES, NV, HALF, (V > 1 && HALF) ? kTurnPacks : kTurnSome>(a, g, part, st);
}

template <typename IO, int V, bool HALF>
cudaError_t norm_packed(const falcon_qknorm_args_t &a, const falcon_qknorm_grads_t *g, float *part, cudaStream_t st) {
    if constexpr (V < 8) {   // 256 channels of 8 are 32 packs
        if (a.d / V > 32) return norm_run<IO, V, 32, 2, HALF>(a, g, part, st);
    }
    switch (norm_lanes(a, V)) {
        case 4: return norm_run<IO, V, 4, 1, HALF>(a, g, part, st);
        case 8: return norm_run<IO, V, 8, 1, HALF>(a, g, part, st);
        case 16: return norm_run<IO, V, 16, 1, HALF>(a, g, part, st);
        default: return norm_run<IO, V, 32, 1, HALF>(a, g, part, st);
    }
}

template <typename IO, int W, bool HALF>
cudaError_t norm_io(const falcon_qknorm_args_t &a, const falcon_qknorm_grads_t *g, float *part, cudaStream_t st) {
    const int V = norm_pack(a, g);
    if (V == W) return norm_packed<IO, W, HALF>(a, g, part, st);
    if constexpr (W == 8) {
        if (V == 4) return norm_packed<IO, 4, HALF>(a, g, part, st);
    }
    if (a.d <= 32) return norm_run<IO, 1, 32, 1, HALF>(a, g, part, st);
    if (a.d <= 64) return norm_run<IO, 1, 32, 2, HALF>(a, g, part, st);
    if (a.d <= 128) return norm_run<IO, 1, 32, 4, HALF>(a, g, part, st);
    return norm_run<IO, 1, 32, 8, HALF>(a, g, part, st);
}

cudaError_t norm_any(const falcon_qknorm_args_t &a, const falcon_qknorm_grads_t *g, float *part, cudaStream_t st) {
    const bool half = a.rot_layout == FALCON_ROT_HALF || a.rot == 0;   // the layouts differ where something turns
    if (a.io_dtype == FALCON_BF16) return half ? norm_io<__nv_bfloat16, 8, true>(a, g, part, st) : norm_io<__nv_bfloat16, 8, false>(a, g, part, st);
    return half ? norm_io<float, 4, true>(a, g, part, st) : norm_io<float, 4, false>(a, g, part, st);
}

bool nothing(const falcon_qknorm_args_t &a) { return (long long)a.B * a.T * (a.Hq + a.Hk) == 0; }

}  // namespace

// Enough for any alignment of the views.
size_t qknorm_bwd_workspace(const falcon_qknorm_args_t &a) {
    return nothing(a) ? 0 : (size_t)kBwdBlocks * 2 * a.d * sizeof(float);
}

cudaError_t launch_qknorm_fwd(const falcon_qknorm_args_t &a, cudaStream_t st) {
    return nothing(a) ? cudaSuccess : norm_any(a, nullptr, nullptr, st);
}

cudaError_t launch_qknorm_bwd(const falcon_qknorm_args_t &a, const falcon_qknorm_grads_t &g, float *ws, cudaStream_t st) {
    long long parts = 0;
    if (!nothing(a)) {
        const cudaError_t e = norm_any(a, &g, g.dwq || g.dwk ? ws : nullptr, st);
        if (e != cudaSuccess) return e;
        parts = norm_shape(a, norm_lanes(a, norm_pack(a, &g))).blocks;
    }
    const SumJob jobs[2] = {{ws, a.d, 2LL * a.d, g.dwq}, {ws + a.d, a.d, 2LL * a.d, g.dwk}};
    return launch_column_sums(jobs, 2, parts, st);
}

}  // namespace falcon
