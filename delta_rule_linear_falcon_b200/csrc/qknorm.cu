// qknorm.cu -- falcon_qknorm_fwd / falcon_qknorm_bwd: the norm of every head's query and key rows with
// the rotation by position in the same pass.
//
// A row is read once and written once for a few flops an element: bound by HBM. A row of d channels
// belongs to LANES neighbouring lanes with NV packs of 16 bytes each (of the io type), so a warp moves
// whole rows; the sum of squares and the partner of a rotated pair come from shuffles (the partner of
// FALCON_ROT_HALF is rot / 2 channels away, a whole number of packs). Where pointers, strides, d or rot / 2
// are not multiples of a pack, V = 1: lane l owns channels l, l + 32, .. and partners come through shared
// memory. The angles of a token are the same for all its heads: a block takes one or more tokens with all
// heads and forms each token's sines and cosines once, the angle's whole turns taken off in fp64.
// Backward: the same walk with the row turned back; dwq and dwk are summed per lane over the rows of a
// block, then over blocks by a second launch.
#include "ops.cuh"

namespace falcon {

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormWarps = kNormThreads / 32;
constexpr int kMaxWidth = 256;
constexpr double kInvTwoPi = 0.15915494309189533577;

struct NormShape {
    int tokens;         // tokens of a group
    long long groups;   // groups of all sequences together: ceil(B T / tokens)
    int heads;          // heads a block takes (grid.y parts)
    int parts;
};

// Sines and cosines of `tokens` tokens, [token][rot / 2] (cos, sin).
__device__ __forceinline__ void angles(const falcon_qknorm_args_t &a, long long tok0, int tokens, float2 *cs) {
    const int half = a.rot / 2;
    const long long all = (long long)a.B * a.T;
    for (int i = threadIdx.x; i < tokens * half; i += kNormThreads) {
        const long long tok = tok0 + i / half;
        float2 r = make_float2(1.f, 0.f);
        if (tok < all) {
            const double pos = a.positions ? (double)a.positions[tok] : (double)(tok % a.T);
            const double turns = pos * (double)a.freq[i % half] * kInvTwoPi;
            sincospif(2.f * (float)(turns - rint(turns)), &r.y, &r.x);
        }
        cs[i] = r;
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

// One thread's part of a row: packs lane, lane + LANES, .. (V > 1) or channels lane, lane + 32, .. (V = 1).
// Turns n by +angle (sign = 1) or -angle (sign = -1).
template <int V, int LANES, int NV>
__device__ __forceinline__ void turn(const falcon_qknorm_args_t &a, float (&n)[NV][V], int lane, const float2 *cs,
                                     float sign, float *stage) {
    if (a.rot == 0) return;
    const int half = a.rot / 2;
    if (V == 1) {
        __syncwarp();
#pragma unroll
        for (int m = 0; m < NV; ++m)
            if (lane + m * LANES < a.rot) stage[lane + m * LANES] = n[m][0];
        __syncwarp();
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int e = lane + m * LANES;
            if (e >= a.rot) continue;
            const bool hi = a.rot_layout == FALCON_ROT_HALF ? e >= half : (e & 1) != 0;
            const int pair = a.rot_layout == FALCON_ROT_HALF ? (hi ? e - half : e) : e / 2;
            const float other = stage[a.rot_layout == FALCON_ROT_HALF ? (hi ? e - half : e + half) : (e ^ 1)];
            const float2 c = cs[pair];
            n[m][0] = fmaf(n[m][0], c.x, (hi ? other : -other) * (sign * c.y));
        }
    } else if (a.rot_layout == FALCON_ROT_PAIRS) {
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int e = (lane + m * LANES) * V;
            if (e >= a.rot) continue;   // rot is a multiple of 2; pairs do not cross a pack
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                if (e + i >= a.rot) break;
                const float2 c = cs[(e + i) / 2];
                const float x1 = n[m][i], x2 = n[m][i + 1], sn = sign * c.y;
                n[m][i] = fmaf(x1, c.x, -x2 * sn);
                n[m][i + 1 < V ? i + 1 : i] = fmaf(x2, c.x, x1 * sn);
            }
        }
    } else {
        const int hp = half / V;   // the partner's distance in packs
        float o[NV][V];
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int p = lane + m * LANES;
            const bool hi = p >= hp;
            const int from = p < 2 * hp ? (hi ? p - hp : p + hp) : p;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float x = 0.f;
#pragma unroll
                for (int mm = 0; mm < NV; ++mm) {
                    const float y = __shfl_sync(0xffffffffu, n[mm][i], from % LANES, LANES);
                    if (from / LANES == mm) x = y;
                }
                o[m][i] = hi ? x : -x;
            }
        }
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int p = lane + m * LANES;
            if (p >= 2 * hp) continue;
            const int e = (p >= hp ? p - hp : p) * V;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float2 c = cs[e + i];
                n[m][i] = fmaf(n[m][i], c.x, o[m][i] * (sign * c.y));
            }
        }
    }
}

template <typename IO, int V, int LANES, int NV>
__global__ void __launch_bounds__(kNormThreads) qknorm_fwd_kernel(falcon_qknorm_args_t a, NormShape s) {
    typedef Pack<IO, V> P;
    constexpr int RPW = 32 / LANES;   // rows of a warp
    extern __shared__ __align__(16) float2 cs[];
    __shared__ float stage_all[V == 1 ? kNormWarps : 1][V == 1 ? kMaxWidth : 1];
    float *stage = stage_all[V == 1 ? threadIdx.x >> 5 : 0];
    const long long tok0 = (long long)blockIdx.x * s.tokens;
    angles(a, tok0, s.tokens, cs);
    __syncthreads();
    const int lane = threadIdx.x % LANES;
    const int slot = threadIdx.x / LANES;              // this group of lanes among the block's
    const int h0 = blockIdx.y * s.heads;
    const int hn = min(s.heads, a.Hq + a.Hk - h0);
    const long long all = (long long)a.B * a.T;
    const int rows = s.tokens * hn;
    for (int r0 = 0; r0 < rows; r0 += kNormWarps * RPW) {
        const int r = r0 + slot;
        const int j = r / hn, hh = h0 + r % hn;
        const long long tok = tok0 + j;
        bool live = r < rows && tok < all;
        const int b = live ? (int)(tok / a.T) : 0, t = live ? (int)(tok % a.T) : 0;
        live = live && t < seq_length(a.lengths, b, a.T);
        const bool isq = hh < a.Hq;
        const int h = isq ? hh : hh - a.Hq;
        const falcon_view_t &in = isq ? a.q : a.k, &out = isq ? a.q_out : a.k_out;
        const float *w = isq ? a.wq : a.wk;
        float x[NV][V];
        float ss = 0.f;
        const IO *px = live ? row_of<IO>(in, b, h, t) : nullptr;
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int e = (lane + m * LANES) * V;
            P::cvt(live && e < a.d ? P::ld(px + e) : P::zero(), x[m]);
#pragma unroll
            for (int i = 0; i < V; ++i) ss = fmaf(x[m][i], x[m][i], ss);
        }
        const float ri = root_inverse(a, a.norm == FALCON_NORM_NONE ? 0.f : lanes_total<LANES>(ss));
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int e = (lane + m * LANES) * V;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                x[m][i] *= ri;
                if (w && e < a.d) x[m][i] *= w[e + i];
            }
        }
        turn<V, LANES, NV>(a, x, lane, cs + (r < rows ? j : 0) * (a.rot / 2), 1.f, stage);
        if (live) {
            IO *po = row_of<IO>(out, b, h, t);
#pragma unroll
            for (int m = 0; m < NV; ++m) {
                const int e = (lane + m * LANES) * V;
                if (e < a.d) P::st(po + e, x[m]);
            }
        }
    }
}

template <typename IO, int V, int LANES, int NV>
__global__ void __launch_bounds__(kNormThreads) qknorm_bwd_kernel(falcon_qknorm_args_t a, falcon_qknorm_grads_t g, NormShape s,
                                                                  float *part) {
    typedef Pack<IO, V> P;
    typedef Pack<float, V> F;
    constexpr int RPW = 32 / LANES;
    extern __shared__ __align__(16) float2 cs[];
    __shared__ float stage_all[V == 1 ? kNormWarps : 1][V == 1 ? kMaxWidth : 1];
    __shared__ float sw[2][kMaxWidth];
    float *stage = stage_all[V == 1 ? threadIdx.x >> 5 : 0];
    const int lane = threadIdx.x % LANES, slot = threadIdx.x / LANES;
    const int heads = a.Hq + a.Hk;
    const long long all = (long long)a.B * a.T;
    float dw[2][NV][V];
#pragma unroll
    for (int m = 0; m < NV; ++m)
#pragma unroll
        for (int i = 0; i < V; ++i) dw[0][m][i] = dw[1][m][i] = 0.f;
    for (long long grp = blockIdx.x; grp < s.groups; grp += gridDim.x) {
        const long long tok0 = grp * s.tokens;
        __syncthreads();
        angles(a, tok0, s.tokens, cs);
        __syncthreads();
        const int rows = s.tokens * heads;
        for (int r0 = 0; r0 < rows; r0 += kNormWarps * RPW) {
            const int r = r0 + slot;
            const int j = r / heads, hh = r % heads;
            const long long tok = tok0 + j;
            const bool there = r < rows && tok < all;
            const int b = there ? (int)(tok / a.T) : 0, t = there ? (int)(tok % a.T) : 0;
            const bool live = there && t < seq_length(a.lengths, b, a.T);
            const bool isq = hh < a.Hq;
            const int h = isq ? hh : hh - a.Hq;
            const falcon_view_t &in = isq ? a.q : a.k, &up = isq ? g.dq_out : g.dk_out, &to = isq ? g.dq : g.dk;
            const float *w = isq ? a.wq : a.wk;
            float x[NV][V], u[NV][V];
            float ss = 0.f;
            const IO *px = live ? row_of<IO>(in, b, h, t) : nullptr;
            const float *pu = live ? row_of<float>(up, b, h, t) : nullptr;
#pragma unroll
            for (int m = 0; m < NV; ++m) {
                const int e = (lane + m * LANES) * V;
                const bool ok = live && e < a.d;
                P::cvt(ok ? P::ld(px + e) : P::zero(), x[m]);
                F::cvt(ok ? F::ld(pu + e) : F::zero(), u[m]);
#pragma unroll
                for (int i = 0; i < V; ++i) ss = fmaf(x[m][i], x[m][i], ss);
            }
            const float ri = root_inverse(a, a.norm == FALCON_NORM_NONE ? 0.f : lanes_total<LANES>(ss));
            turn<V, LANES, NV>(a, u, lane, cs + (r < rows ? j : 0) * (a.rot / 2), -1.f, stage);
            float dot = 0.f;
#pragma unroll
            for (int m = 0; m < NV; ++m) {
                const int e = (lane + m * LANES) * V;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    x[m][i] *= ri;
                    const float d = u[m][i] * x[m][i];
                    if (live) {
                        if (isq) dw[0][m][i] += d;
                        else dw[1][m][i] += d;
                    }
                    if (w && e < a.d) u[m][i] *= w[e + i];
                    dot = fmaf(u[m][i], x[m][i], dot);
                }
            }
            if (a.norm != FALCON_NORM_NONE) {
                dot = lanes_total<LANES>(dot);
                if (a.norm == FALCON_NORM_RMS) dot /= (float)a.d;
#pragma unroll
                for (int m = 0; m < NV; ++m)
#pragma unroll
                    for (int i = 0; i < V; ++i) u[m][i] = ri * fmaf(-x[m][i], dot, u[m][i]);
            }
            if (there) {
                float *po = row_of<float>(to, b, h, t);
#pragma unroll
                for (int m = 0; m < NV; ++m) {
                    const int e = (lane + m * LANES) * V;
                    if (!live)
#pragma unroll
                        for (int i = 0; i < V; ++i) u[m][i] = 0.f;
                    if (e < a.d) F::st(po + e, u[m]);
                }
            }
        }
    }
    if (!part) return;
    // the block's sums, lane group by lane group in order
    for (int i = threadIdx.x; i < 2 * kMaxWidth; i += kNormThreads) sw[i / kMaxWidth][i % kMaxWidth] = 0.f;
    for (int k = 0; k < kNormThreads / LANES; ++k) {
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

// Tokens of a group: about 64 rows, so that every warp has several and the angles are shared by them.
NormShape norm_shape(const falcon_qknorm_args_t &a, int num_sms) {
    NormShape s;
    const int heads = a.Hq + a.Hk;
    s.tokens = 1;
    while (s.tokens < 16 && s.tokens * heads < 64) s.tokens *= 2;
    const long long all = (long long)a.B * a.T;
    s.groups = (all + s.tokens - 1) / s.tokens;
    s.heads = heads;
    s.parts = 1;
    // few tokens: their heads over several blocks
    while (s.heads > 8 && s.groups * s.parts < 2LL * num_sms) {
        s.heads = (s.heads + 1) / 2;
        s.parts = (heads + s.heads - 1) / s.heads;
    }
    return s;
}

long long bwd_blocks(const NormShape &s) { return s.groups < 148 * 6 ? s.groups : 148 * 6; }

template <typename IO, int V, int LANES, int NV>
cudaError_t norm_run(const falcon_qknorm_args_t &a, const falcon_qknorm_grads_t *g, const NormShape &s, float *part, cudaStream_t st) {
    const size_t smem = (size_t)s.tokens * (a.rot / 2) * sizeof(float2);
    if (g) {
        qknorm_bwd_kernel<IO, V, LANES, NV><<<(unsigned)bwd_blocks(s), kNormThreads, smem, st>>>(a, *g, s, part);
    } else {
        if (s.groups > kMaxGrid || s.parts > 65535) return cudaErrorInvalidConfiguration;
        qknorm_fwd_kernel<IO, V, LANES, NV><<<dim3((unsigned)s.groups, (unsigned)s.parts), kNormThreads, smem, st>>>(a, s);
    }
    return cudaGetLastError();
}

template <typename IO, int W>
cudaError_t norm_io(const falcon_qknorm_args_t &a, const falcon_qknorm_grads_t *g, const NormShape &s, float *part, cudaStream_t st) {
    const int V = norm_pack(a, g);
    if (V == 1) return norm_run<IO, 1, 32, 8>(a, g, s, part, st);
    const int packs = a.d / V;
    if (packs <= 4) return norm_run<IO, W, 4, 1>(a, g, s, part, st);
    if (packs <= 8) return norm_run<IO, W, 8, 1>(a, g, s, part, st);
    if (packs <= 16) return norm_run<IO, W, 16, 1>(a, g, s, part, st);
    if (packs <= 32) return norm_run<IO, W, 32, 1>(a, g, s, part, st);
    return norm_run<IO, W, 32, 2>(a, g, s, part, st);
}

bool nothing(const falcon_qknorm_args_t &a) { return (long long)a.B * a.T * (a.Hq + a.Hk) == 0; }

}  // namespace

size_t qknorm_bwd_workspace(const falcon_qknorm_args_t &a) {
    if (nothing(a)) return 0;
    return (size_t)bwd_blocks(norm_shape(a, 1)) * 2 * a.d * sizeof(float);
}

cudaError_t launch_qknorm_fwd(const falcon_qknorm_args_t &a, int num_sms, cudaStream_t st) {
    if (nothing(a)) return cudaSuccess;
    const NormShape s = norm_shape(a, num_sms);
    return a.io_dtype == FALCON_BF16 ? norm_io<__nv_bfloat16, 8>(a, nullptr, s, nullptr, st) : norm_io<float, 4>(a, nullptr, s, nullptr, st);
}

cudaError_t launch_qknorm_bwd(const falcon_qknorm_args_t &a, const falcon_qknorm_grads_t &g, float *ws, int num_sms, cudaStream_t st) {
    (void)num_sms;
    long long parts = 0;
    if (!nothing(a)) {
        const NormShape s = norm_shape(a, 1);
        parts = bwd_blocks(s);
        float *part = g.dwq || g.dwk ? ws : nullptr;
        const cudaError_t e = a.io_dtype == FALCON_BF16 ? norm_io<__nv_bfloat16, 8>(a, &g, s, part, st) : norm_io<float, 4>(a, &g, s, part, st);
        if (e != cudaSuccess) return e;
    }
    const SumJob jobs[2] = {{ws, a.d, 2LL * a.d, g.dwq}, {ws + a.d, a.d, 2LL * a.d, g.dwk}};
    return launch_column_sums(jobs, 2, parts, st);
}

}  // namespace falcon
