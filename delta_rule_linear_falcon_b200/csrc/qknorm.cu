// qknorm.cu -- falcon_qknorm_fwd / falcon_qknorm_bwd: the norm of every head's query and key rows with
// the rotation by position in the same pass.
//
// A row is read once and written once for a few flops an element: bound by HBM. A row of d channels
// belongs to LANES neighbouring lanes with NV packs of 16 bytes each (of the io type), so a warp moves
// whole rows; the sum of squares and the partner of a rotated pair come from shuffles (the partner of
// FALCON_ROT_HALF is rot / 2 channels away, a whole number of packs). A group of LANES lanes takes one token
// and walks its heads, kRows of them in flight: the token's sines and cosines, the same for every head, are
// formed once by the block (the angle's whole turns taken off in fp64), kept in registers over the walk, and
// the row addresses advance by one addition. With few tokens the heads are cut over more groups.
// Where pointers, strides, d or rot / 2 are not multiples of a pack, V = 1: lane l owns channels l, l + 32, ..
// and partners come through shared memory.
// Backward: the same walk with the row turned back; dwq and dwk are summed per lane over the tokens of a
// block, then over blocks by a second launch.
#include "ops.cuh"

namespace falcon {

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormWarps = kNormThreads / 32;
constexpr int kMaxWidth = 256;
constexpr double kInvTwoPi = 0.15915494309189533577;

struct NormShape {
    long long groups;   // blocks along the tokens: one token for each group of lanes
    int heads;          // heads of a walk
    int parts;          // walks of a token
};

// Where pair p's (cos, sin) lies: V > 1 as 16-byte pairs of pairs, [pair of the pack][pack], so that the lanes
// of a row read neighbouring words.
template <int V>
__device__ __forceinline__ int turn_slot(const falcon_qknorm_args_t &a, int p) {
    if (V == 1) return p;
    const int per = a.rot_layout == FALCON_ROT_HALF ? V : V / 2;   // pairs of a pack
    const int packs = (a.rot / 2 + per - 1) / per;
    return ((p % per) / 2 * packs + p / per) * 2 + (p & 1);
}
// Slots of a token (the last pack may be padded).
__host__ __device__ inline int turn_slots(const falcon_qknorm_args_t &a, int V) {
    if (V == 1) return a.rot / 2;
    const int per = a.rot_layout == FALCON_ROT_HALF ? V : V / 2;
    return (a.rot / 2 + per - 1) / per * per;
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
            const double turns = pos * (double)a.freq[p] * kInvTwoPi;
            sincospif(2.f * (float)(turns - rint(turns)), &r.y, &r.x);
        }
        cs[j * slots + turn_slot<V>(a, p)] = r;
    }
}

// 1 / root of a row with sum of squares ss.
__device__ __forceinline__ float root_inverse(const falcon_qknorm_args_t &a, float ss) {
    if (a.norm == FALCON_NORM_NONE) return 1.f;
    const float m = (a.norm == FALCON_NORM_RMS ? ss / (float)a.d : ss) + a.eps;
    return m == 0.f ? 0.f : rsqrtf(m);
}

template <int LANES>
__device__ __forceinline__ float lanes_total(float x) {
#pragma unroll
    for (int m = 1; m < LANES; m <<= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// A lane's part of a token's rotation: for each of its packs' channels the factors of the channel itself (c) and of
// its partner (s, with the partner's sign).
template <int V, int LANES, int NV, bool HALF> struct Turn {
    float c[NV][V], s[NV][V];
    int froms[NV];   // HALF: the pack of each pack's partners (V = 1: the partner's channel)

    __device__ __forceinline__ void load(const falcon_qknorm_args_t &a, int lane, const float2 *cs, float sign) {
        const int half = a.rot / 2;
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int p = lane + m * LANES;
            froms[m] = p;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                c[m][i] = 1.f;
                s[m][i] = 0.f;
            }
            if (V == 1) {
                if (p < a.rot) {
                    const bool hi = HALF ? p >= half : (p & 1) != 0;
                    froms[m] = HALF ? (hi ? p - half : p + half) : p ^ 1;
                    const float2 r = cs[HALF ? (hi ? p - half : p) : p / 2];
                    c[m][0] = r.x;
                    s[m][0] = (hi ? sign : -sign) * r.y;
                }
            } else if (HALF) {
                const int hp = half / V;
                if (p < 2 * hp) {
                    const bool hi = p >= hp;
                    froms[m] = hi ? p - hp : p + hp;
                    const float f = hi ? sign : -sign;
#pragma unroll
                    for (int i = 0; i < V; i += 2) {
                        const float4 r = reinterpret_cast<const float4 *>(cs)[i / 2 * hp + (hi ? p - hp : p)];
                        c[m][i] = r.x;
                        s[m][i] = f * r.y;
                        c[m][i + 1 < V ? i + 1 : i] = r.z;
                        s[m][i + 1 < V ? i + 1 : i] = f * r.w;
                    }
                }
            } else {
                const int packs = (half + V / 2 - 1) / (V > 1 ? V / 2 : 1);
                if (p < packs) {
#pragma unroll
                    for (int i = 0; i + 3 < V; i += 4) {
                        const float4 r = reinterpret_cast<const float4 *>(cs)[i / 4 * packs + p];
                        c[m][i] = c[m][i + 1] = r.x;
                        s[m][i] = -sign * r.y;
                        s[m][i + 1] = sign * r.y;
                        c[m][i + 2] = c[m][i + 3] = r.z;
                        s[m][i + 2] = -sign * r.w;
                        s[m][i + 3] = sign * r.w;
                    }
                }
            }
        }
    }

    // n <- the row turned; stage: the warp's shared row (V = 1).
    __device__ __forceinline__ void apply(float (&n)[NV][V], int lane, float *stage) const {
        float o[NV][V];
        if (V == 1) {
            __syncwarp();
#pragma unroll
            for (int m = 0; m < NV; ++m) stage[lane + m * LANES] = n[m][0];
            __syncwarp();
#pragma unroll
            for (int m = 0; m < NV; ++m) o[m][0] = stage[froms[m]];
        } else if (HALF) {
#pragma unroll
            for (int m = 0; m < NV; ++m)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float x = 0.f;
#pragma unroll
                    for (int mm = 0; mm < NV; ++mm) {
                        const float y = __shfl_sync(0xffffffffu, n[mm][i], froms[m] % LANES, LANES);
                        if (NV == 1 || froms[m] / LANES == mm) x = y;
                    }
                    o[m][i] = x;
                }
        } else {
#pragma unroll
            for (int m = 0; m < NV; ++m)
#pragma unroll
                for (int i = 0; i < V; ++i) o[m][i] = n[m][V > 1 ? i ^ 1 : i];
        }
#pragma unroll
        for (int m = 0; m < NV; ++m)
#pragma unroll
            for (int i = 0; i < V; ++i) n[m][i] = fmaf(n[m][i], c[m][i], o[m][i] * s[m][i]);
    }
};

template <typename IO, int V, int LANES, int NV, bool HALF>
__global__ void __launch_bounds__(kNormThreads) qknorm_fwd_kernel(falcon_qknorm_args_t a, NormShape s) {
    typedef Pack<IO, V> P;
    constexpr int G = kNormThreads / LANES;       // groups of lanes, tokens of a block
    constexpr int kRows = V == 1 ? 1 : 4 / NV;    // rows in flight
    extern __shared__ __align__(16) float2 cs[];
    __shared__ float stage_all[V == 1 ? kNormWarps : 1][V == 1 ? kMaxWidth : 1];
    float *stage = stage_all[V == 1 ? threadIdx.x >> 5 : 0];
    const long long tok0 = (long long)blockIdx.x * G;
    const int lane = threadIdx.x % LANES, slot = threadIdx.x / LANES;
    Turn<V, LANES, NV, HALF> turn;
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
                const int e = (lane + m * LANES) * V + i;
                w[m][i] = weight && e < a.d ? weight[e] : 1.f;
            }
        const IO *px = row_of<IO>(in, b, first, t) + lane * V;
        IO *po = row_of<IO>(out, b, first, t) + lane * V;
        for (int h = first; h < last; h += kRows) {
            typename P::raw raw[kRows][NV];
#pragma unroll
            for (int r = 0; r < kRows; ++r)
#pragma unroll
                for (int m = 0; m < NV; ++m) {
                    raw[r][m] = P::zero();
                    if (live && h + r < last && (lane + m * LANES) * V < a.d) raw[r][m] = P::ld(px + r * in.sh + m * LANES * V);
                }
            px += kRows * in.sh;
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                float x[NV][V], ss = 0.f;
#pragma unroll
                for (int m = 0; m < NV; ++m) {
                    P::cvt(raw[r][m], x[m]);
#pragma unroll
                    for (int i = 0; i < V; ++i) ss = fmaf(x[m][i], x[m][i], ss);
                }
                const float ri = root_inverse(a, a.norm == FALCON_NORM_NONE ? 0.f : lanes_total<LANES>(ss));
#pragma unroll
                for (int m = 0; m < NV; ++m)
#pragma unroll
                    for (int i = 0; i < V; ++i) x[m][i] = x[m][i] * ri * w[m][i];
                if (a.rot > 0) turn.apply(x, lane, stage);
                if (live && h + r < last) {
#pragma unroll
                    for (int m = 0; m < NV; ++m)
                        if ((lane + m * LANES) * V < a.d) P::st(po + r * out.sh + m * LANES * V, x[m]);
                }
            }
            po += kRows * out.sh;
        }
    }
}

template <typename IO, int V, int LANES, int NV, bool HALF>
__global__ void __launch_bounds__(kNormThreads) qknorm_bwd_kernel(falcon_qknorm_args_t a, falcon_qknorm_grads_t g, NormShape s,
                                                                  float *part) {
    typedef Pack<IO, V> P;
    typedef Pack<float, V> F;
    constexpr int G = kNormThreads / LANES;
    constexpr int kRows = V == 1 || NV > 1 ? 1 : 2;
    extern __shared__ __align__(16) float2 cs[];
    __shared__ float stage_all[V == 1 ? kNormWarps : 1][V == 1 ? kMaxWidth : 1];
    __shared__ float sw[2][kMaxWidth];
    float *stage = stage_all[V == 1 ? threadIdx.x >> 5 : 0];
    const int lane = threadIdx.x % LANES, slot = threadIdx.x / LANES;
    const long long walks = s.groups * s.parts;
    float dw[2][NV][V];
#pragma unroll
    for (int m = 0; m < NV; ++m)
#pragma unroll
        for (int i = 0; i < V; ++i) dw[0][m][i] = dw[1][m][i] = 0.f;
    for (long long walk = blockIdx.x; walk < walks; walk += gridDim.x) {
        const long long tok0 = walk / s.parts * G;
        const int h0 = (int)(walk % s.parts) * s.heads, h1 = min(h0 + s.heads, a.Hq + a.Hk);
        Turn<V, LANES, NV, HALF> turn;
        if (a.rot > 0) {
            __syncthreads();
            angles<V>(a, tok0, G, cs);
            __syncthreads();
            turn.load(a, lane, cs + slot * turn_slots(a, V), -1.f);
        }
        const long long tok = tok0 + slot;
        const bool there = tok < (long long)a.B * a.T;
        const int b = there ? (int)(tok / a.T) : 0, t = there ? (int)(tok - (long long)b * a.T) : 0;
        const bool live = there && t < seq_length(a.lengths, b, a.T);
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
                    const int e = (lane + m * LANES) * V + i;
                    w[m][i] = weight && e < a.d ? weight[e] : 1.f;
                }
            const IO *px = row_of<IO>(in, b, first, t) + lane * V;
            const float *pu = row_of<float>(up, b, first, t) + lane * V;
            float *po = row_of<float>(to, b, first, t) + lane * V;
            for (int h = first; h < last; h += kRows) {
                typename P::raw rx[kRows][NV];
                typename F::raw ru[kRows][NV];
#pragma unroll
                for (int r = 0; r < kRows; ++r)
#pragma unroll
                    for (int m = 0; m < NV; ++m) {
                        rx[r][m] = P::zero();
                        ru[r][m] = F::zero();
                        if (live && h + r < last && (lane + m * LANES) * V < a.d) {
                            rx[r][m] = P::ld(px + r * in.sh + m * LANES * V);
                            ru[r][m] = F::ld(pu + r * up.sh + m * LANES * V);
                        }
                    }
                px += kRows * in.sh;
                pu += kRows * up.sh;
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    float x[NV][V], u[NV][V], ss = 0.f, dot = 0.f;
#pragma unroll
                    for (int m = 0; m < NV; ++m) {
                        P::cvt(rx[r][m], x[m]);
                        F::cvt(ru[r][m], u[m]);
#pragma unroll
                        for (int i = 0; i < V; ++i) ss = fmaf(x[m][i], x[m][i], ss);
                    }
                    const float ri = root_inverse(a, a.norm == FALCON_NORM_NONE ? 0.f : lanes_total<LANES>(ss));
                    if (a.rot > 0) turn.apply(u, lane, stage);
#pragma unroll
                    for (int m = 0; m < NV; ++m)
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            x[m][i] *= ri;
                            if (live && h + r < last) dw[which][m][i] = fmaf(u[m][i], x[m][i], dw[which][m][i]);
                            u[m][i] *= w[m][i];
                            dot = fmaf(u[m][i], x[m][i], dot);
                        }
                    if (a.norm != FALCON_NORM_NONE) {
                        dot = lanes_total<LANES>(dot);
                        if (a.norm == FALCON_NORM_RMS) dot /= (float)a.d;
#pragma unroll
                        for (int m = 0; m < NV; ++m)
#pragma unroll
                            for (int i = 0; i < V; ++i) u[m][i] = ri * fmaf(-x[m][i], dot, u[m][i]);
                    }
                    if (there && h + r < last) {
#pragma unroll
                        for (int m = 0; m < NV; ++m) {
                            if (!live)
#pragma unroll
                                for (int i = 0; i < V; ++i) u[m][i] = 0.f;
                            if ((lane + m * LANES) * V < a.d) F::st(po + r * to.sh + m * LANES * V, u[m]);
                        }
                    }
                }
                po += kRows * to.sh;
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
                const int e = (lane + m * LANES) * V;
                if (e < a.d)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        sw[0][e + i] += dw[0][m][i];
                        sw[1][e + i] += dw[1][m][i];
                    }
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.d; i += kNormThreads)
        part[(long long)blockIdx.x * 2 * a.d + i] = sw[i / a.d][i % a.d];
}

// The pack's width: 16 bytes of the io type where every row and the rotation allow it.
int norm_pack(const falcon_qknorm_args_t &a, const falcon_qknorm_grads_t *g) {
    const int es = a.io_dtype == FALCON_BF16 ? 2 : 4, V = 16 / es;
    bool ok = a.d % V == 0 && view_packs(a.q, V, es) && view_packs(a.k, V, es);
    if (a.rot_layout == FALCON_ROT_HALF) ok = ok && (a.rot / 2) % V == 0;
    if (!g) ok = ok && view_packs(a.q_out, V, es) && view_packs(a.k_out, V, es);
    else ok = ok && view_packs(g->dq_out, 4, 4) && view_packs(g->dk_out, 4, 4) && view_packs(g->dq, 4, 4) && view_packs(g->dk, 4, 4);
    return ok ? V : 1;
}

int norm_lanes(const falcon_qknorm_args_t &a, int V) {
    const int packs = a.d / V;
    return V == 1 || packs > 16 ? 32 : packs > 8 ? 16 : packs > 4 ? 8 : 4;
}

// One token for each group of lanes; its heads over several groups while those are fewer than kWanted
// threads (three quarters of what the GPU holds).
NormShape norm_shape(const falcon_qknorm_args_t &a, int lanes) {
    constexpr long long kWanted = 148LL * 1536;   // threads
    NormShape s;
    const int heads = a.Hq + a.Hk, per = kNormThreads / lanes;
    const long long all = (long long)a.B * a.T;
    s.groups = (all + per - 1) / per;
    s.heads = heads;
    s.parts = 1;
    while (s.heads > 1 && all * lanes * s.parts < kWanted) {
        s.heads = (s.heads + 1) / 2;
        s.parts = (heads + s.heads - 1) / s.heads;
    }
    return s;
}

constexpr long long kBwdBlocks = 148 * 4;
long long bwd_blocks(const NormShape &s) { return s.groups * s.parts < kBwdBlocks ? s.groups * s.parts : kBwdBlocks; }

template <typename IO, int V, int LANES, int NV, bool HALF>
cudaError_t norm_run(const falcon_qknorm_args_t &a, const falcon_qknorm_grads_t *g, float *part, cudaStream_t st) {
    const NormShape s = norm_shape(a, LANES);
    const size_t smem = (size_t)(kNormThreads / LANES) * turn_slots(a, V) * sizeof(float2);
    if (g) {
        qknorm_bwd_kernel<IO, V, LANES, NV, HALF><<<(unsigned)bwd_blocks(s), kNormThreads, smem, st>>>(a, *g, s, part);
    } else {
        if (s.groups > kMaxGrid || s.parts > 65535) return cudaErrorInvalidConfiguration;
        qknorm_fwd_kernel<IO, V, LANES, NV, HALF><<<dim3((unsigned)s.groups, (unsigned)s.parts), kNormThreads, smem, st>>>(a, s);
    }
    return cudaGetLastError();
}

template <typename IO, int W, bool HALF>
cudaError_t norm_io(const falcon_qknorm_args_t &a, const falcon_qknorm_grads_t *g, float *part, cudaStream_t st) {
    const int V = norm_pack(a, g);
    if (V == 1) return norm_run<IO, 1, 32, 8, HALF>(a, g, part, st);
    if (a.d / V > 32) return norm_run<IO, W, 32, 2, HALF>(a, g, part, st);
    switch (norm_lanes(a, V)) {
        case 4: return norm_run<IO, W, 4, 1, HALF>(a, g, part, st);
        case 8: return norm_run<IO, W, 8, 1, HALF>(a, g, part, st);
        case 16: return norm_run<IO, W, 16, 1, HALF>(a, g, part, st);
        default: return norm_run<IO, W, 32, 1, HALF>(a, g, part, st);
    }
}

cudaError_t norm_any(const falcon_qknorm_args_t &a, const falcon_qknorm_grads_t *g, float *part, cudaStream_t st) {
    const bool half = a.rot_layout == FALCON_ROT_HALF;
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
        parts = bwd_blocks(norm_shape(a, norm_lanes(a, norm_pack(a, &g))));
    }
    const SumJob jobs[2] = {{ws, a.d, 2LL * a.d, g.dwq}, {ws + a.d, a.d, 2LL * a.d, g.dwk}};
    return launch_column_sums(jobs, 2, parts, st);
}

}  // namespace falcon
