// conv.cu -- falcon_conv_fwd / falcon_conv_step / falcon_conv_bwd: the short causal depthwise
// convolution p_t = bias + sum_{j<K} w_j x_{t-K+1+j}, y = act(p).
//
// Forward: 2 K flops for an element read once and written once, so the kernel is bound by HBM. A thread
// owns V channels (16 bytes of them where pointers, strides and d allow it, else one channel) and walks
// a run of tokens with the last K - 1 inputs in registers; four tokens' loads are in flight at a time.
// Neighbouring threads own neighbouring channels, so every access of a warp is whole lines, whichever of
// token-major and head-major the two views are. A run re-reads its K - 1 first inputs (from L2).
// Backward: the same walk with a second window, of dp: step t needs x_{t-K+1..t} for p_t and act', adds
// dp_t x to dw, and emits dx_{t-K+1} = sum_j w_j dp_{t-j}. The walk goes K - 1 tokens past the run
// (dp there is formed again by the next run). dw and dbias: registers, then the block's shared memory,
// then one row of partial sums for each block, summed in a fixed order by a second launch.
#include "ops.cuh"

namespace falcon {

namespace {

constexpr int kConvThreads = 256;
constexpr int kConvBatch = 4;     // tokens whose loads are in flight together

// Threads of a block: bx over the packs of one token's channels, by over runs of tokens.
struct ConvShape {
    int nv;          // packs of V channels of a head
    int bx, by;
    int run;         // tokens a thread walks
    long long ncb;   // blocks along the channels
    long long ntb;   // blocks along the tokens
};

ConvShape conv_shape(const falcon_conv_args_t &a, int V, int run, int first) {
    ConvShape s;
    s.nv = (a.d + V - 1) / V;
    const long long packs = (long long)a.H * s.nv;
    s.bx = 32;
    while (s.bx < kConvThreads && s.bx < packs) s.bx *= 2;
    s.by = kConvThreads / s.bx;
    s.run = run;
    s.ncb = (packs + s.bx - 1) / s.bx;
    const long long tokens = (long long)a.T + first;
    s.ntb = (tokens + (long long)run * s.by - 1) / ((long long)run * s.by);
    if (s.ntb < 1) s.ntb = 1;
    return s;
}

template <int K> struct Taps {
    static constexpr int kPast = K > 1 ? K - 1 : 1;   // rows kept of the past (one unused row for K = 1)
};

// Row r of the cached tail of (b, h): (B,H,K-1,d).
template <typename IO, int K>
__device__ __forceinline__ IO *tail_row(const void *p, int b, int h, int H, int r, int d) {
    return reinterpret_cast<IO *>(const_cast<void *>(p)) + (((long long)b * H + h) * (K - 1) + r) * d;
}

template <int K, int V>
__device__ __forceinline__ void load_weights(const falcon_conv_args_t &a, int h, int c0, float (&w)[K][V], float (&bias)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const long long c = (long long)h * a.d + c0 + i;
#pragma unroll
        for (int j = 0; j < K; ++j) w[j][i] = a.w[c * K + j];
        bias[i] = a.bias ? a.bias[c] : 0.f;
    }
}

template <typename IO, int K, int V, bool SILU>
__global__ void __launch_bounds__(kConvThreads) conv_fwd_kernel(falcon_conv_args_t a, ConvShape s) {
    typedef Pack<IO, V> P;
    constexpr int kPast = Taps<K>::kPast;
    unsigned bid = blockIdx.x;
    const unsigned cb = bid % (unsigned)s.ncb;
    bid /= (unsigned)s.ncb;
    const unsigned tb = bid % (unsigned)s.ntb;
    const int b = (int)(bid / (unsigned)s.ntb);
    const long long pack = (long long)cb * s.bx + threadIdx.x;
    if (pack >= (long long)a.H * s.nv) return;
    const int h = (int)(pack / s.nv), c0 = (int)(pack % s.nv) * V;
    const int n = seq_length(a.lengths, b, a.T);
    const long long tile = (long long)tb * s.by + threadIdx.y;
    const long long t0 = tile * s.run;
    const long long t1 = t0 + s.run < n ? t0 + s.run : n;

    float w[K][V], bias[V];
    load_weights<K, V>(a, h, c0, w, bias);
    const IO *x = row_of<IO>(a.x, b, h, 0) + c0;
    IO *y = row_of<IO>(a.y, b, h, 0) + c0;

    float past[kPast][V];   // x_{t-K+1} .. x_{t-1}, oldest first
    auto extended = [&](long long t, float (&o)[V]) {   // input t, or the cached tail, or zero
        if (t >= 0) P::cvt(P::ld(x + t * a.x.st), o);
        else if (a.state) P::cvt(P::ld(tail_row<IO, K>(a.state, b, h, a.H, (int)(t + K - 1), a.d) + c0), o);
        else
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = 0.f;
    };
    if (t0 < t1) {
        if (K > 1) {
#pragma unroll
            for (int j = 0; j < K - 1; ++j) extended(t0 - (K - 1) + j, past[j]);
        }
        for (long long t = t0; t < t1; t += kConvBatch) {
            typename P::raw in[kConvBatch];
#pragma unroll
            for (int u = 0; u < kConvBatch; ++u) in[u] = t + u < t1 ? P::ld(x + (t + u) * a.x.st) : P::zero();
#pragma unroll
            for (int u = 0; u < kConvBatch; ++u) {
                float cur[V], out[V];
                P::cvt(in[u], cur);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float p = bias[i];
#pragma unroll
                    for (int j = 0; j < K - 1; ++j) p = fmaf(w[j][i], past[j][i], p);
                    p = fmaf(w[K - 1][i], cur[i], p);
                    out[i] = SILU ? silu(p) : p;
#pragma unroll
                    for (int j = 0; j + 1 < K - 1; ++j) past[j][i] = past[j + 1][i];
                    if (K > 1) past[kPast - 1][i] = cur[i];
                }
                if (t + u < t1) P::st(y + (t + u) * a.y.st, out);
            }
        }
    }
    // the tail behind the last token; the thread that read `state` writes it, rows ascending, so that
    // both may be the same memory
    if (K > 1 && a.state_out && tile == 0) {
        for (int r = 0; r < K - 1; ++r) {
            float o[V];
            extended((long long)n - (K - 1) + r, o);
            P::st(tail_row<IO, K>(a.state_out, b, h, a.H, r, a.d) + c0, o);
        }
    }
}

// One token: the tail and the token are read once, the output and the shifted tail written once.
template <typename IO, int K, int V, bool SILU>
__global__ void __launch_bounds__(128) conv_step_kernel(falcon_conv_args_t a, int nv) {
    typedef Pack<IO, V> P;
    const long long packs = (long long)a.H * nv;
    const long long g = (long long)blockIdx.x * 128 + threadIdx.x;
    if (g >= packs * a.B) return;
    const int b = (int)(g / packs);
    const int pack = (int)(g - b * packs);
    const int h = pack / nv, c0 = (pack % nv) * V;
    float past[Taps<K>::kPast][V], cur[V], out[V], w[K][V], bias[V];
    P::cvt(P::ld(row_of<IO>(a.x, b, h, 0) + c0), cur);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) P::cvt(P::ld(tail_row<IO, K>(a.state, b, h, a.H, j, a.d) + c0), past[j]);
    load_weights<K, V>(a, h, c0, w, bias);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float p = bias[i];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) p = fmaf(w[j][i], past[j][i], p);
        p = fmaf(w[K - 1][i], cur[i], p);
        out[i] = SILU ? silu(p) : p;
    }
    P::st(row_of<IO>(a.y, b, h, 0) + c0, out);
#pragma unroll
    for (int j = 0; j + 1 < K; ++j)
        P::st(tail_row<IO, K>(a.state_out, b, h, a.H, j, a.d) + c0, j + 1 < K - 1 ? past[j + 1 < Taps<K>::kPast ? j + 1 : 0] : cur);
}

template <typename IO, int K, int V, bool SILU>
__global__ void __launch_bounds__(kConvThreads) conv_bwd_kernel(falcon_conv_args_t a, falcon_conv_grads_t g, ConvShape s,
                                                                float *part) {
    typedef Pack<IO, V> P;
    typedef Pack<float, V> F;
    constexpr int kPast = Taps<K>::kPast;
    extern __shared__ float sums[];   // kConvThreads x (K + 1) V
    unsigned bid = blockIdx.x;
    const unsigned cb = bid % (unsigned)s.ncb;
    bid /= (unsigned)s.ncb;
    const unsigned tb = bid % (unsigned)s.ntb;
    const int b = (int)(bid / (unsigned)s.ntb);
    const long long pack = (long long)cb * s.bx + threadIdx.x;
    const bool in = pack < (long long)a.H * s.nv;
    const int h = in ? (int)(pack / s.nv) : 0, c0 = in ? (int)(pack % s.nv) * V : 0;
    const int n = seq_length(a.lengths, b, a.T);
    // the walk starts at the oldest cached token, -(K-1)
    const long long t0 = -(K - 1) + ((long long)tb * s.by + threadIdx.y) * s.run;
    const long long t1 = t0 + s.run < a.T ? t0 + s.run : a.T;

    float dw[K][V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        db[i] = 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) dw[j][i] = 0.f;
    }
    if (in && t0 < t1) {
        float w[K][V], bias[V];
        load_weights<K, V>(a, h, c0, w, bias);
        const IO *x = row_of<IO>(a.x, b, h, 0) + c0;
        const float *dy = row_of<float>(g.dy, b, h, 0) + c0;
        float *dx = row_of<float>(g.dx, b, h, 0) + c0;
        float past[kPast][V], dp[K][V];   // inputs before t; dp_{t-K+1} .. dp_t
        auto extended = [&](long long t) {
            if (t >= 0) return t < n ? P::ld(x + t * a.x.st) : P::zero();
            if (t >= -(K - 1) && a.state) return P::ld(tail_row<IO, K>(a.state, b, h, a.H, (int)(t + K - 1), a.d) + c0);
            return P::zero();
        };
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int j = 0; j < K; ++j) dp[j][i] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < K - 1; ++j) P::cvt(extended(t0 - (K - 1) + j), past[j]);
        for (long long tt = t0; tt < t1 + K - 1; tt += kConvBatch) {
            typename P::raw xin[kConvBatch];
            typename F::raw gin[kConvBatch];
#pragma unroll
            for (int u = 0; u < kConvBatch; ++u) {
                const long long t = tt + u;
                const bool live = t >= 0 && t < n && t < t1 + K - 1;
                xin[u] = t < t1 + K - 1 ? extended(t) : P::zero();
                gin[u] = live ? F::ld(dy + t * g.dy.st) : F::zero();
            }
#pragma unroll
            for (int u = 0; u < kConvBatch; ++u) {
                const long long t = tt + u;
                const bool own = t < t1;          // this run's dw
                const bool live = t >= 0 && t < n;
                float cur[V], gy[V], out[V];
                P::cvt(xin[u], cur);
                F::cvt(gin[u], gy);
#pragma unroll
                for (int i = 0; i < V; ++i) {
#pragma unroll
                    for (int j = 0; j + 1 < K; ++j) dp[j][i] = dp[j + 1][i];
                    float d = gy[i];
                    if (SILU) {
                        float p = bias[i];
#pragma unroll
                        for (int j = 0; j < K - 1; ++j) p = fmaf(w[j][i], past[j][i], p);
                        p = fmaf(w[K - 1][i], cur[i], p);
                        d *= silu_grad(p);
                    }
                    d = live ? d : 0.f;           // also where p or act'(p) is not finite
                    dp[K - 1][i] = d;
                    if (own && live) {
#pragma unroll
                        for (int j = 0; j < K - 1; ++j) dw[j][i] = fmaf(d, past[j][i], dw[j][i]);
                        dw[K - 1][i] = fmaf(d, cur[i], dw[K - 1][i]);
                        db[i] += d;
                    }
                    float o = 0.f;
#pragma unroll
                    for (int j = 0; j < K; ++j) o = fmaf(w[j][i], dp[K - 1 - j][i], o);
                    out[i] = o;
#pragma unroll
                    for (int j = 0; j + 1 < K - 1; ++j) past[j][i] = past[j + 1][i];
                    if (K > 1) past[kPast - 1][i] = cur[i];
                }
                const long long r = t - (K - 1);   // the input whose gradient is complete
                if (r < t0 || r >= t1) continue;
                // the tail that state_out copied: extended rows n .. n + K - 2, inputs n - K + 1 .. n - 1
                const long long tail = r + (K - 1) - n;
                if (g.dstate_out && tail >= 0 && tail < K - 1) {
                    const float *q = tail_row<float, K>(g.dstate_out, b, h, a.H, (int)tail, a.d) + c0;
#pragma unroll
                    for (int i = 0; i < V; ++i) out[i] += q[i];
                }
                if (r >= 0) {
                    if (r >= n)
#pragma unroll
                        for (int i = 0; i < V; ++i) out[i] = 0.f;
                    F::st(dx + r * g.dx.st, out);
                } else if (g.dstate) {
                    float *q = tail_row<float, K>(g.dstate, b, h, a.H, (int)(r + K - 1), a.d) + c0;
#pragma unroll
                    for (int i = 0; i < V; ++i) q[i] = out[i];
                }
            }
        }
    }
    // the block's sums over its runs, then one partial row: (H,d,K) of dw, (H,d) of dbias
    constexpr int M = (K + 1) * V;
    float *mine = sums + (threadIdx.y * s.bx + threadIdx.x) * M;
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < K; ++j) mine[i * K + j] = dw[j][i];
        mine[K * V + i] = db[i];
    }
    __syncthreads();
    const long long HD = (long long)a.H * a.d;
    float *row = part + ((long long)b * s.ntb + tb) * HD * (K + 1);
    for (int e = threadIdx.y * s.bx + threadIdx.x; e < s.bx * M; e += kConvThreads) {
        float acc = 0.f;
        for (int y = 0; y < s.by; ++y) acc += sums[(long long)y * s.bx * M + e];
        const long long pk = (long long)cb * s.bx + e / M;
        if (pk >= (long long)a.H * s.nv) continue;
        const int m = e % M;
        const long long c = pk / s.nv * a.d + pk % s.nv * V;
        if (m < K * V) row[c * K + m] = acc;
        else row[(long long)HD * K + c + (m - K * V)] = acc;
    }
}

// Whether V channels go as one access: d and both the io and fp32 views.
int conv_pack(const falcon_conv_args_t &a, const falcon_view_t *f32a, const falcon_view_t *f32b) {
    const int es = a.io_dtype == FALCON_BF16 ? 2 : 4;
    const int V = f32a ? 4 : 16 / es;
    bool ok = a.d % V == 0 && view_packs(a.x, V, es);
    if (!f32a) ok = ok && view_packs(a.y, V, es);
    else ok = ok && view_packs(*f32a, V, 4) && view_packs(*f32b, V, 4);
    ok = ok && reinterpret_cast<uintptr_t>(a.state) % (V * es) == 0;
    if (!f32a) ok = ok && reinterpret_cast<uintptr_t>(a.state_out) % (V * es) == 0;
    return ok ? V : 1;
}

// Tokens of a thread's run: long runs re-read less of the past, short ones give more threads.
int conv_run(const falcon_conv_args_t &a, int V, long long want_threads) {
    const long long packs = (long long)a.H * ((a.d + V - 1) / V) * a.B;
    int run = 64;
    while (run > 8 && packs * ((a.T + run - 1) / run) < want_threads) run /= 2;
    return run;
}

#define FALCON_CONV_TAPS(M)                                                            \
    switch (a.K) {                                                                     \
        case 1: M(1); break;                                                           \
        case 2: M(2); break;                                                           \
        case 3: M(3); break;                                                           \
        case 4: M(4); break;                                                           \
        case 5: M(5); break;                                                           \
        case 6: M(6); break;                                                           \
        case 7: M(7); break;                                                           \
        case 8: M(8); break;                                                           \
        default: return cudaErrorInvalidValue;                                         \
    }

template <typename IO, int V>
cudaError_t conv_fwd_io(const falcon_conv_args_t &a, const ConvShape &s, cudaStream_t st) {
    const long long blocks = s.ncb * s.ntb * a.B;
    if (blocks > kMaxGrid) return cudaErrorInvalidConfiguration;
    const dim3 block(s.bx, s.by);
#define FALCON_RUN(K)                                                                             \
    if (a.act == FALCON_ACT_SILU) conv_fwd_kernel<IO, K, V, true><<<(unsigned)blocks, block, 0, st>>>(a, s); \
    else conv_fwd_kernel<IO, K, V, false><<<(unsigned)blocks, block, 0, st>>>(a, s)
    FALCON_CONV_TAPS(FALCON_RUN)
#undef FALCON_RUN
    return cudaGetLastError();
}

template <typename IO, int V>
cudaError_t conv_step_io(const falcon_conv_args_t &a, cudaStream_t st) {
    const int nv = (a.d + V - 1) / V;
    const long long blocks = ((long long)a.H * nv * a.B + 127) / 128;
    if (blocks > kMaxGrid) return cudaErrorInvalidConfiguration;
#define FALCON_RUN(K)                                                                             \
    if (a.act == FALCON_ACT_SILU) conv_step_kernel<IO, K, V, true><<<(unsigned)blocks, 128, 0, st>>>(a, nv); \
    else conv_step_kernel<IO, K, V, false><<<(unsigned)blocks, 128, 0, st>>>(a, nv)
    FALCON_CONV_TAPS(FALCON_RUN)
#undef FALCON_RUN
    return cudaGetLastError();
}

template <typename IO, int V>
cudaError_t conv_bwd_io(const falcon_conv_args_t &a, const falcon_conv_grads_t &g, const ConvShape &s, float *ws, cudaStream_t st) {
    const long long blocks = s.ncb * s.ntb * a.B;
    if (blocks > kMaxGrid) return cudaErrorInvalidConfiguration;
    const dim3 block(s.bx, s.by);
    const size_t smem = (size_t)kConvThreads * (a.K + 1) * V * sizeof(float);
#define FALCON_RUN(K)                                                                             \
    if (a.act == FALCON_ACT_SILU) conv_bwd_kernel<IO, K, V, true><<<(unsigned)blocks, block, smem, st>>>(a, g, s, ws); \
    else conv_bwd_kernel<IO, K, V, false><<<(unsigned)blocks, block, smem, st>>>(a, g, s, ws)
    FALCON_CONV_TAPS(FALCON_RUN)
#undef FALCON_RUN
    return cudaGetLastError();
}

ConvShape conv_bwd_shape(const falcon_conv_args_t &a, int V) {
    return conv_shape(a, V, conv_run(a, V, 148 * 1024), a.K - 1);
}

}  // namespace

cudaError_t launch_conv_fwd(const falcon_conv_args_t &a, int num_sms, cudaStream_t st) {
    if ((long long)a.B * a.H == 0) return cudaSuccess;
    const int V = conv_pack(a, nullptr, nullptr);
    const ConvShape s = conv_shape(a, V, conv_run(a, V, (long long)num_sms * 2048), 0);
    if (a.io_dtype == FALCON_BF16)
        return V == 8 ? conv_fwd_io<__nv_bfloat16, 8>(a, s, st) : conv_fwd_io<__nv_bfloat16, 1>(a, s, st);
    return V == 4 ? conv_fwd_io<float, 4>(a, s, st) : conv_fwd_io<float, 1>(a, s, st);
}

cudaError_t launch_conv_step(const falcon_conv_args_t &a, cudaStream_t st) {
    if ((long long)a.B * a.H == 0) return cudaSuccess;
    const int V = conv_pack(a, nullptr, nullptr);
    if (a.io_dtype == FALCON_BF16) return V == 8 ? conv_step_io<__nv_bfloat16, 8>(a, st) : conv_step_io<__nv_bfloat16, 1>(a, st);
    return V == 4 ? conv_step_io<float, 4>(a, st) : conv_step_io<float, 1>(a, st);
}

// The workspace does not depend on the alignment of the views, so it is the larger of both packings'.
size_t conv_bwd_workspace(const falcon_conv_args_t &a) {
    size_t most = 0;
    for (int V = 1; V <= 4; V += 3) {
        const ConvShape s = conv_bwd_shape(a, V);
        const size_t bytes = (size_t)a.B * s.ntb * a.H * a.d * (a.K + 1) * sizeof(float);
        most = bytes > most ? bytes : most;
    }
    return most;
}

cudaError_t launch_conv_bwd(const falcon_conv_args_t &a, const falcon_conv_grads_t &g, float *ws, cudaStream_t st) {
    if (a.H == 0) return cudaSuccess;
    const int V = conv_pack(a, &g.dy, &g.dx);
    const ConvShape s = conv_bwd_shape(a, V);
    if (a.B > 0) {
        cudaError_t e;
        if (a.io_dtype == FALCON_BF16) e = V == 4 ? conv_bwd_io<__nv_bfloat16, 4>(a, g, s, ws, st) : conv_bwd_io<__nv_bfloat16, 1>(a, g, s, ws, st);
        else e = V == 4 ? conv_bwd_io<float, 4>(a, g, s, ws, st) : conv_bwd_io<float, 1>(a, g, s, ws, st);
        if (e != cudaSuccess) return e;
    }
    const long long HD = (long long)a.H * a.d, row = HD * (a.K + 1);   // dw (H,d,K), then dbias (H,d)
    const SumJob jobs[2] = {{ws, HD * a.K, row, g.dw}, {ws + HD * a.K, HD, row, g.dbias}};
    return launch_column_sums(jobs, 2, (long long)a.B * s.ntb, st);
}

}  // namespace falcon
