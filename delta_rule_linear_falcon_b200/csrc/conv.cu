// conv.cu -- falcon_conv_fwd / falcon_conv_step / falcon_conv_bwd: the short causal depthwise
// convolution p_t = bias + sum_{j<K} w_j x_{t-K+1+j}, y = act(p).
//
// Forward: 2 K flops for an element read once and written once, so the kernel is bound by HBM. A thread
// owns V channels (8 bytes of them where pointers, strides and d allow it, else one channel) and walks
// a run of tokens with the last K - 1 inputs in registers. Neighbouring threads own neighbouring channels,
// so every access of a warp is whole lines, whichever of token-major and head-major the two views are.
// The inputs come ahead of their use through a ring in shared memory (kStages batches of kConvBatch tokens,
// asynchronous copies into places that only the copying thread reads, so no barrier): bytes in flight cost no
// registers. Eight bytes a thread rather than 16 leave registers for four blocks an SM (B8 H16 T4096 d128 bf16: 57 us
// against 72 before the runs were fitted to the SMs, 55 since). One channel a thread (V = 1): a batch's loads are in
// flight together (the same case off alignment: 123 us). A run re-reads its K - 1 first inputs (from L2). 53 us of kernel
// there, 5.1 TB/s: the exponential unit (two of its operations for each silu) is at 64% and the instruction slots at
// 65%. K = 8, whose window and weights leave two blocks an SM: 75 us.
// Backward: the same walk with a second window, of dp: step t needs x_{t-K+1..t} for p_t and act', adds
// dp_t x to dw, and emits dx_{t-K+1} = sum_j w_j dp_{t-j}. The walk goes K - 1 tokens past the run
// (dp there is formed again by the next run). dw and dbias: registers, then the block's shared memory,
// then one row of partial sums for each block, summed in a fixed order by a second launch. B4 H16 T4096 d128 bf16:
// 73 us and 6 us of kernels for 336 MB (51 us at the copy rate), 140 us in all off alignment. Eighty registers and 21
// warps an SM, instruction slots at 57%: bound by latency. K = 5 82 us in all, K = 8 111 us, two blocks an SM. Short
// sequences have a row of partial sums each, and blocks that T does not fill: B512 H16 T16 79 us against 25 at the
// copy rate.
#include "ops.cuh"

namespace falcon {

namespace {

constexpr int kConvThreads = 256;
constexpr int kConvBatch = 4;     // tokens of a batch
constexpr int kStages = 3;        // batches of the ring

// Threads of a block: bx over the packs of one token's channels, by over runs of tokens.
struct ConvShape {
    int nv;          // packs of V channels of a head
    int bx, by;
    int run;         // tokens a thread walks
    long long ncb;   // blocks along the channels
    long long ntb;   // blocks along the tokens
};

// Runs: so long that the blocks fill the `slots` that the SMs hold once, twice, .. (long runs re-read less of the past
// and leave fewer partial rows; a part-filled last turn costs as much as a full one: 55 us against 57 forward and 84
// against 89 backward with runs of 128), and at most kLongest tokens.
ConvShape conv_shape(const falcon_conv_args_t &a, int V, long long slots) {
    constexpr long long kLongest = 160, kShortest = 8;
    ConvShape s;
    s.nv = (a.d - 1) / V + 1;
    const long long packs = (long long)a.H * s.nv;
    s.bx = 32;
    while (s.bx < kConvThreads && s.bx < packs) s.bx *= 2;
    s.by = kConvThreads / s.bx;
    s.ncb = (packs + s.bx - 1) / s.bx;
    long long run = kLongest;
    for (int turns = 1; turns <= 8; ++turns) {
        const long long all = s.ncb * a.B, rows = all > 0 ? all : 1, tiles = slots * turns > rows ? slots * turns / rows : 1;
        run = (a.T + tiles * s.by - 1) / (tiles * s.by);
        if (run <= kLongest) break;
    }
    s.run = (int)(run > kLongest ? kLongest : run < kShortest ? kShortest : run);
    s.ntb = ((long long)a.T + (long long)s.run * s.by - 1) / ((long long)s.run * s.by);
    if (s.ntb < 1) s.ntb = 1;
    return s;
}

template <int K> struct Taps {
    static constexpr int kPast = K > 1 ? K - 1 : 1;   // rows kept of the past (one unused row for K = 1)
};

// A thread's V channels as pairs (the upper half of the only pair is unused for V = 1).
template <int V> struct Pairs {
    static constexpr int N = V > 1 ? V / 2 : 1;
};
template <typename IO, int V>
__device__ __forceinline__ void to_pairs(typename Pack<IO, V>::raw r, f32x2 (&o)[Pairs<V>::N]) {
    float x[V];
    Pack<IO, V>::cvt(r, x);
#pragma unroll
    for (int i = 0; i < Pairs<V>::N; ++i) o[i] = pack2(x[2 * i], x[V > 1 ? 2 * i + 1 : 0]);
}
template <int V>
__device__ __forceinline__ void from_pairs(const f32x2 (&p)[Pairs<V>::N], float (&x)[V]) {
#pragma unroll
    for (int i = 0; i < Pairs<V>::N; ++i) {
        float lo, hi;
        unpack2(p[i], lo, hi);
        x[2 * i] = lo;
        if (V > 1) x[V > 1 ? 2 * i + 1 : 0] = hi;
    }
}

// Row r of the cached tail of (b, h): (B,H,K-1,d).
template <typename IO, int K>
__device__ __forceinline__ IO *tail_row(const void *p, int b, int h, int H, int r, int d) {
    return reinterpret_cast<IO *>(const_cast<void *>(p)) + (((long long)b * H + h) * (K - 1) + r) * d;
}

template <int K, int V>
__device__ __forceinline__ void load_weights(const falcon_conv_args_t &a, int h, int c0, float (&w)[K][V], float (&bias)[V]) {
    const float *p = a.w + ((long long)h * a.d + c0) * K;
    float f[K * V];   // (V channels, K taps) as they lie
    if (V > 1 && V * K % 4 == 0 && (reinterpret_cast<uintptr_t>(a.w) & 15) == 0) {   // V K floats from c0 K: whole 16-byte words
#pragma unroll
        for (int i = 0; i + 3 < K * V; i += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(p + i);
            f[i] = x.x; f[i + 1] = x.y; f[i + 2] = x.z; f[i + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < K * V; ++i) f[i] = p[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < K; ++j) w[j][i] = f[i * K + j];
        bias[i] = a.bias ? a.bias[(long long)h * a.d + c0 + i] : 0.f;
    }
}
template <int K, int V>
__device__ __forceinline__ void load_weights(const falcon_conv_args_t &a, int h, int c0, f32x2 (&w)[K][Pairs<V>::N],
                                             f32x2 (&bias)[Pairs<V>::N]) {
    float f[K][V], g[V];
    load_weights<K, V>(a, h, c0, f, g);
#pragma unroll
    for (int i = 0; i < Pairs<V>::N; ++i) {
        const int i1 = V > 1 ? 2 * i + 1 : 0;
        bias[i] = pack2(g[2 * i], g[i1]);
#pragma unroll
        for (int j = 0; j < K; ++j) w[j][i] = pack2(f[j][2 * i], f[j][i1]);
    }
}

// p = bias + sum_j w_j (window), oldest input first.
template <int K, int N>
__device__ __forceinline__ f32x2 taps(const f32x2 (&w)[K][N], const f32x2 (&past)[Taps<K>::kPast][N], f32x2 cur, f32x2 bias, int i) {
    f32x2 p = bias;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) p = fma2(w[j][i], past[j][i], p);
    return fma2(w[K - 1][i], cur, p);
}

template <typename IO, int K, int V, bool SILU>
__global__ void __launch_bounds__(kConvThreads, K <= 4 ? 4 : 2) conv_fwd_kernel(falcon_conv_args_t a, ConvShape s) {
    typedef Pack<IO, V> P;
    constexpr int kPast = Taps<K>::kPast, N = Pairs<V>::N;
    __shared__ __align__(16) typename P::raw ring[V > 1 ? kStages : 1][V > 1 ? kConvBatch : 1][V > 1 ? kConvThreads : 1];
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
    const int t0 = (int)(tile * s.run < n ? tile * s.run : n);
    const int t1 = t0 + s.run < n ? t0 + s.run : n;
    const int me = threadIdx.y * s.bx + threadIdx.x;

    const IO *x = row_of<IO>(a.x, b, h, 0) + c0;
    auto extended = [&](int t) {   // input t, or the cached tail, or zero
        if (t >= 0) return P::ld(x + t * a.x.st);
        if (a.state) return P::ld(tail_row<IO, K>(a.state, b, h, a.H, t + K - 1, a.d) + c0);
        return P::zero();
    };
    if (t0 < t1) {
        const IO *ahead = x + t0 * a.x.st;   // the next token to be asked for
        int ta = t0;
        auto ask = [&](int stage) {
            if (V > 1) {
#pragma unroll
                for (int u = 0; u < kConvBatch; ++u) {
                    if (ta + u < t1) copy_async<(int)sizeof(typename P::raw)>(&ring[stage][u][me], ahead);
                    ahead += a.x.st;
                }
                ta += kConvBatch;
                copy_commit();
            }
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) ask(i);
        f32x2 w[K][N], bias[N], past[kPast][N];   // past: x_{t-K+1} .. x_{t-1}
        load_weights<K, V>(a, h, c0, w, bias);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) to_pairs<IO, V>(extended(t0 - (K - 1) + j), past[j]);
        IO *y = row_of<IO>(a.y, b, h, t0) + c0;
        int stage = 0, free_stage = kStages - 1;
        for (int t = t0; t < t1; t += kConvBatch) {
            typename P::raw in[kConvBatch];
            if (V > 1) {
                ask(free_stage);
                free_stage = free_stage + 1 < kStages ? free_stage + 1 : 0;
                copy_wait<kStages - 1>();
#pragma unroll
                for (int u = 0; u < kConvBatch; ++u) in[u] = ring[stage][u][me];
                stage = stage + 1 < kStages ? stage + 1 : 0;
            } else {
#pragma unroll
                for (int u = 0; u < kConvBatch; ++u) in[u] = t + u < t1 ? P::ld(x + (t + u) * a.x.st) : P::zero();
            }
#pragma unroll
            for (int u = 0; u < kConvBatch; ++u) {
                if (t + u >= t1) break;
                f32x2 cur[N], p[N];
                float out[V];
                to_pairs<IO, V>(in[u], cur);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    p[i] = taps<K, N>(w, past, cur[i], bias[i], i);
#pragma unroll
                    for (int j = 0; j + 1 < K - 1; ++j) past[j][i] = past[j + 1][i];
                    if (K > 1) past[kPast - 1][i] = cur[i];
                }
                if (SILU) {
#pragma unroll
                    for (int i = 0; i < N; ++i) p[i] = silu2(p[i]);
                }
                from_pairs<V>(p, out);
                P::st(y, out);
                y += a.y.st;
            }
        }
    }
    // the tail behind the last token; the thread that read `state` writes it, rows ascending, so that
    // both may be the same memory
    if (K > 1 && a.state_out && tile == 0) {
        for (int r = 0; r < K - 1; ++r) {
            float o[V];
            P::cvt(extended(n - (K - 1) + r), o);
            P::st(tail_row<IO, K>(a.state_out, b, h, a.H, r, a.d) + c0, o);
        }
    }
}

// One token: the tail and the token are read once, the output and the shifted tail written once. A thread takes its pack
// in several sequences, the next one's rows under way: the weights, for bf16 twice as many bytes as the sequence's rows,
// are read once for them (4096 sequences of H32 d128 K4: 48 us, 5.6 TB/s; 61 with a thread for each pack and sequence).
// Blocks an SM of K <= 4: eight 48 us, six 54; of K = 8 (512 of H24 d128): six 15 us, eight 17.
constexpr int kStepThreads = 128;
__host__ __device__ constexpr int step_blocks(int K) { return K <= 4 ? 8 : 6; }

template <typename IO, int K, int V, bool SILU>
__global__ void __launch_bounds__(kStepThreads, step_blocks(K)) conv_step_kernel(falcon_conv_args_t a, int nv, int chunk) {
    typedef Pack<IO, V> P;
    const long long packs = (long long)a.H * nv;
    const long long g = (long long)blockIdx.x * kStepThreads + threadIdx.x;
    const long long start = g / packs * chunk;   // behind the last sequence in threads that the last block has left over
    if (start >= a.B) return;
    const int b0 = (int)start, b1 = b0 + min(chunk, a.B - b0);
    const int pack = (int)(g % packs);
    const int h = pack / nv, c0 = (pack % nv) * V;
    typename P::raw next[K];   // the tail, then the token
    auto fetch = [&](int b) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) next[j] = P::ld(tail_row<IO, K>(a.state, b, h, a.H, j, a.d) + c0);
        next[K - 1] = P::ld(row_of<IO>(a.x, b, h, 0) + c0);
    };
    fetch(b0);
    float w[K][V], bias[V];
    load_weights<K, V>(a, h, c0, w, bias);
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        typename P::raw row[K];
        float p[V];
#pragma unroll
        for (int j = 0; j < K; ++j) row[j] = next[j];
        if (b + 1 < b1) fetch(b + 1);
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = bias[i];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            float x[V];
            P::cvt(row[j], x);
#pragma unroll
            for (int i = 0; i < V; ++i) p[i] = fmaf(w[j][i], x[i], p[i]);
        }
        if (SILU) {
#pragma unroll
            for (int i = 0; i < V; ++i) p[i] = silu(p[i]);
        }
        P::st(row_of<IO>(a.y, b, h, 0) + c0, p);
#pragma unroll
        for (int j = 0; j + 1 < K; ++j)
            *reinterpret_cast<typename P::raw *>(tail_row<IO, K>(a.state_out, b, h, a.H, j, a.d) + c0) = row[j + 1];
    }
}

struct True { static constexpr bool value = true; };
struct False { static constexpr bool value = false; };

template <typename IO, int K, int V, bool SILU>
__global__ void __launch_bounds__(kConvThreads, K <= 4 ? 3 : 2) conv_bwd_kernel(falcon_conv_args_t a, falcon_conv_grads_t g, ConvShape s,
                                                                   float *part_w, float *part_b) {
    typedef Pack<IO, V> P;
    typedef Pack<float, V> F;
    constexpr int kPast = Taps<K>::kPast, N = Pairs<V>::N;
    extern __shared__ __align__(16) char smem[];   // the rings of dy and x, then the block's sums
    typedef typename F::raw RingG[kConvBatch][kConvThreads];
    typedef typename P::raw RingX[kConvBatch][kConvThreads];
    RingG *ring_g = reinterpret_cast<RingG *>(smem);
    RingX *ring_x = reinterpret_cast<RingX *>(smem + kStages * sizeof(RingG));
    unsigned bid = blockIdx.x;
    const unsigned cb = bid % (unsigned)s.ncb;
    bid /= (unsigned)s.ncb;
    const unsigned tb = bid % (unsigned)s.ntb;
    const int b = (int)(bid / (unsigned)s.ntb);
    const long long pack = (long long)cb * s.bx + threadIdx.x;
    const bool in = pack < (long long)a.H * s.nv;
    const int h = in ? (int)(pack / s.nv) : 0, c0 = in ? (int)(pack % s.nv) * V : 0;
    const int n = seq_length(a.lengths, b, a.T);
    const long long tile = (long long)tb * s.by + threadIdx.y;
    const int t0 = (int)(tile * s.run < a.T ? tile * s.run : a.T);
    const int t1 = t0 + s.run < a.T ? t0 + s.run : a.T;
    const int r0 = tile == 0 ? -(K - 1) : t0;   // inputs [r0, t1) get their gradient here
    const int tend = t1 + K - 1;                // the walk's end
    const int me = threadIdx.y * s.bx + threadIdx.x;

    f32x2 dw[K][N], db[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        db[i] = 0ull;
#pragma unroll
        for (int j = 0; j < K; ++j) dw[j][i] = 0ull;
    }
    if (in && (t0 < t1 || tile == 0)) {
        const IO *x = row_of<IO>(a.x, b, h, 0) + c0;
        const float *dy = row_of<float>(g.dy, b, h, 0) + c0;
        auto extended = [&](int t) {
            if (t >= 0) return t < n ? P::ld(x + t * a.x.st) : P::zero();
            if (t >= -(K - 1) && a.state) return P::ld(tail_row<IO, K>(a.state, b, h, a.H, t + K - 1, a.d) + c0);
            return P::zero();
        };
        const int te = tend < n ? tend : n;     // tokens that are there
        const IO *ahead_x = x + t0 * a.x.st;
        const float *ahead_g = dy + t0 * g.dy.st;
        int ta = t0;
        auto ask = [&](int stage) {
            if (V > 1) {
#pragma unroll
                for (int u = 0; u < kConvBatch; ++u) {
                    if (ta + u < te) {
                        copy_async<(int)sizeof(typename P::raw)>(&ring_x[stage][u][me], ahead_x);
                        copy_async<(int)sizeof(typename F::raw)>(&ring_g[stage][u][me], ahead_g);
                    }
                    ahead_x += a.x.st;
                    ahead_g += g.dy.st;
                }
                ta += kConvBatch;
                copy_commit();
            }
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) ask(i);
        f32x2 w[K][N], bias[N], past[kPast][N], dp[K][N];   // inputs before t; dp_{t-K+1} .. dp_t
        load_weights<K, V>(a, h, c0, w, bias);
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < K; ++j) dp[j][i] = 0ull;
#pragma unroll
        for (int j = 0; j < K - 1; ++j) to_pairs<IO, V>(extended(t0 - (K - 1) + j), past[j]);
        float *dx = row_of<float>(g.dx, b, h, 0) + c0 + (t0 - (K - 1)) * g.dx.st;   // the row that the walk emits next

        // One token. WHOLE: it is there, its dw is this run's, and an input of this run is complete.
        auto token = [&](auto whole, int t, typename P::raw rx, typename F::raw rg) {
            constexpr bool WHOLE = decltype(whole)::value;
            const bool live = WHOLE || t < n;
            f32x2 cur[N], d2[N], out[N];
            to_pairs<IO, V>(rx, cur);
            to_pairs<float, V>(rg, d2);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (SILU) {   // silu'(p) = s (1 + p (1 - s)), s the sigmoid
                    const f32x2 one = pack2(1.f, 1.f), p = taps<K, N>(w, past, cur[i], bias[i], i), sg = sigmoid2(p);
                    d2[i] = mul2(d2[i], mul2(sg, fma2(p, fma2(sg, pack2(-1.f, -1.f), one), one)));
                }
                if (!live) d2[i] = 0ull;          // also where p or act'(p) is not finite
#pragma unroll
                for (int j = 0; j + 1 < K; ++j) dp[j][i] = dp[j + 1][i];
                dp[K - 1][i] = d2[i];
                if (WHOLE || (live && t < t1)) {
#pragma unroll
                    for (int j = 0; j < K - 1; ++j) dw[j][i] = fma2(d2[i], past[j][i], dw[j][i]);
                    dw[K - 1][i] = fma2(d2[i], cur[i], dw[K - 1][i]);
                    db[i] = add2(db[i], d2[i]);
                }
                out[i] = mul2(w[0][i], dp[K - 1][i]);
#pragma unroll
                for (int j = 1; j < K; ++j) out[i] = fma2(w[j][i], dp[K - 1 - j][i], out[i]);
#pragma unroll
                for (int j = 0; j + 1 < K - 1; ++j) past[j][i] = past[j + 1][i];
                if (K > 1) past[kPast - 1][i] = cur[i];
            }
            float o[V];
            from_pairs<V>(out, o);
            if (WHOLE) {
                F::st(dx, o);
            } else {
                const int r = t - (K - 1);        // the input whose gradient is complete
                if (r >= r0 && r < t1) {
                    // the tail that state_out copied: extended rows n .. n + K - 2, inputs n - K + 1 .. n - 1
                    const int tail = t - n;
                    if (g.dstate_out && tail >= 0 && tail < K - 1) {
                        const float *q = tail_row<float, K>(g.dstate_out, b, h, a.H, tail, a.d) + c0;
#pragma unroll
                        for (int i = 0; i < V; ++i) o[i] += q[i];
                    }
                    if (r >= 0) {
                        if (r >= n)
#pragma unroll
                            for (int i = 0; i < V; ++i) o[i] = 0.f;
                        F::st(dx, o);
                    } else if (g.dstate) {
                        float *q = tail_row<float, K>(g.dstate, b, h, a.H, r + K - 1, a.d) + c0;
#pragma unroll
                        for (int i = 0; i < V; ++i) q[i] = o[i];
                    }
                }
            }
            dx += g.dx.st;
        };

        const int whole0 = r0 + K - 1, whole1 = t1 < n ? t1 : n;
        int stage = 0, free_stage = kStages - 1;
        for (int t = t0; t < tend; t += kConvBatch) {
            typename P::raw rx[kConvBatch];
            typename F::raw rg[kConvBatch];
            if (V > 1) {
                ask(free_stage);
                free_stage = free_stage + 1 < kStages ? free_stage + 1 : 0;
                copy_wait<kStages - 1>();
#pragma unroll
                for (int u = 0; u < kConvBatch; ++u) {
                    rx[u] = ring_x[stage][u][me];
                    rg[u] = ring_g[stage][u][me];
                }
                stage = stage + 1 < kStages ? stage + 1 : 0;
            } else {
#pragma unroll
                for (int u = 0; u < kConvBatch; ++u) {
                    rx[u] = t + u < te ? P::ld(x + (t + u) * a.x.st) : P::zero();
                    rg[u] = t + u < te ? F::ld(dy + (t + u) * g.dy.st) : F::zero();
                }
            }
            if (t >= whole0 + (tile == 0 ? K - 1 : 0) && t + kConvBatch <= whole1) {
#pragma unroll
                for (int u = 0; u < kConvBatch; ++u) token(True{}, t + u, rx[u], rg[u]);
            } else {
#pragma unroll
                for (int u = 0; u < kConvBatch; ++u) {
                    if (t + u >= tend) break;
                    const bool there = t + u < te;   // a place of the ring that was not asked for holds anything
                    token(False{}, t + u, there ? rx[u] : P::zero(), there ? rg[u] : F::zero());
                }
            }
        }
        copy_wait<0>();
    }
    __syncthreads();   // the rings' places are free
    // the block's sums over its runs, then one partial row of dw (H,d,K) and of dbias (H,d)
    constexpr int M = (K + 1) * V;
    float *sums = reinterpret_cast<float *>(smem);
    float *mine = sums + me * M;
    {
        float f[V];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            from_pairs<V>(dw[j], f);
#pragma unroll
            for (int i = 0; i < V; ++i) mine[i * K + j] = f[i];
        }
        from_pairs<V>(db, f);
#pragma unroll
        for (int i = 0; i < V; ++i) mine[K * V + i] = f[i];
    }
    __syncthreads();
    const long long HD = (long long)a.H * a.d;
    const long long row = (long long)b * s.ntb + tb;
    for (int e = me; e < s.bx * M; e += kConvThreads) {
        float acc = 0.f;
        for (int y = 0; y < s.by; ++y) acc += sums[(long long)y * s.bx * M + e];
        const long long pk = (long long)cb * s.bx + e / M;
        if (pk >= (long long)a.H * s.nv) continue;
        const int m = e % M;
        const long long c = pk / s.nv * a.d + pk % s.nv * V;
        if (m < K * V) part_w[(row * HD + c) * K + m] = acc;
        else part_b[row * HD + c + (m - K * V)] = acc;
    }
}

// Whether V channels go as one access: d and both the io and fp32 views.
int conv_pack(const falcon_conv_args_t &a, const falcon_view_t *f32a, const falcon_view_t *f32b) {
    const int es = a.io_dtype == FALCON_BF16 ? 2 : 4;
    const int V = f32a ? 2 : 8 / es;
    bool ok = a.d % V == 0 && view_packs(a.x, V, es);
    if (!f32a) ok = ok && view_packs(a.y, V, es);
    else ok = ok && view_packs(*f32a, V, 4) && view_packs(*f32b, V, 4);
    ok = ok && reinterpret_cast<uintptr_t>(a.state) % (V * es) == 0;
    if (!f32a) ok = ok && reinterpret_cast<uintptr_t>(a.state_out) % (V * es) == 0;
    return ok ? V : 1;
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
cudaError_t conv_step_io(const falcon_conv_args_t &a, int num_sms, cudaStream_t st) {
    const int nv = (a.d - 1) / V + 1;
    const long long packs = (long long)a.H * nv, threads = (long long)num_sms * step_blocks(a.K) * kStepThreads;
    // sequences of a thread: the number with the shortest estimate, in turns of the threads that the SMs hold at once
    // (a thread's start, with its weights, costs about one sequence). For fp32, whose weights weigh half as much, up to two:
    // 4096 sequences of H32 d128 K4 take 87 us with two, 90 with seven, 93 with one.
    auto all = [&](int chunk) { return packs * ((a.B - 1LL + chunk) / chunk); };
    int chunk = 1;
    long long best = 0;
    for (int c = 1; c <= (sizeof(IO) == 2 ? 32 : 2) && c <= a.B; ++c) {
        const long long cost = (all(c) + threads - 1) / threads * (c + 1);
        if (c == 1 || cost < best) {
            best = cost;
            chunk = c;
        }
    }
    const long long blocks = (all(chunk) + kStepThreads - 1) / kStepThreads;
    if (blocks > kMaxGrid) return cudaErrorInvalidConfiguration;
#define FALCON_RUN(K)                                                                             \
    if (a.act == FALCON_ACT_SILU) conv_step_kernel<IO, K, V, true><<<(unsigned)blocks, kStepThreads, 0, st>>>(a, nv, chunk); \
    else conv_step_kernel<IO, K, V, false><<<(unsigned)blocks, kStepThreads, 0, st>>>(a, nv, chunk)
    FALCON_CONV_TAPS(FALCON_RUN)
#undef FALCON_RUN
    return cudaGetLastError();
}

template <typename IO, int V>
cudaError_t conv_bwd_io(const falcon_conv_args_t &a, const falcon_conv_grads_t &g, const ConvShape &s, float *pw, float *pb, cudaStream_t st) {
    const long long blocks = s.ncb * s.ntb * a.B;
    if (blocks > kMaxGrid) return cudaErrorInvalidConfiguration;
    const dim3 block(s.bx, s.by);
    const size_t ring = V > 1 ? (size_t)kStages * kConvBatch * kConvThreads * V * (sizeof(float) + sizeof(IO)) : 0;
    const size_t sums = (size_t)kConvThreads * (a.K + 1) * V * sizeof(float);
    const size_t smem = ring > sums ? ring : sums;
#define FALCON_RUN(K)                                                                             \
    {                                                                                             \
        const auto kern = a.act == FALCON_ACT_SILU ? conv_bwd_kernel<IO, K, V, true> : conv_bwd_kernel<IO, K, V, false>; \
        if (smem > 48 * 1024) {                                                                   \
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem); \
            if (e != cudaSuccess) return e;                                                       \
        }                                                                                         \
        kern<<<(unsigned)blocks, block, smem, st>>>(a, g, s, pw, pb);                                 \
    }
    FALCON_CONV_TAPS(FALCON_RUN)
#undef FALCON_RUN
    return cudaGetLastError();
}

ConvShape conv_bwd_shape(const falcon_conv_args_t &a, int V) {
    return conv_shape(a, V, 148 * (a.K <= 4 ? 3 : 2));
}

}  // namespace

cudaError_t launch_conv_fwd(const falcon_conv_args_t &a, int num_sms, cudaStream_t st) {
    if ((long long)a.B * a.H == 0) return cudaSuccess;
    const int V = conv_pack(a, nullptr, nullptr);
    const ConvShape s = conv_shape(a, V, (long long)num_sms * (a.K <= 4 ? 4 : 2));
    if (a.io_dtype == FALCON_BF16)
        return V == 4 ? conv_fwd_io<__nv_bfloat16, 4>(a, s, st) : conv_fwd_io<__nv_bfloat16, 1>(a, s, st);
    return V == 2 ? conv_fwd_io<float, 2>(a, s, st) : conv_fwd_io<float, 1>(a, s, st);
}

cudaError_t launch_conv_step(const falcon_conv_args_t &a, int num_sms, cudaStream_t st) {
    if ((long long)a.B * a.H == 0) return cudaSuccess;
    const int V = conv_pack(a, nullptr, nullptr);
    if (a.io_dtype == FALCON_BF16) return V == 4 ? conv_step_io<__nv_bfloat16, 4>(a, num_sms, st) : conv_step_io<__nv_bfloat16, 1>(a, num_sms, st);
    return V == 2 ? conv_step_io<float, 2>(a, num_sms, st) : conv_step_io<float, 1>(a, num_sms, st);
}

// The workspace does not depend on the alignment of the views, so it is the larger of both packings'.
size_t conv_bwd_workspace(const falcon_conv_args_t &a) {
    size_t most = 0;
    for (int V = 1; V <= 2; ++V) {
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
    // partial rows of dw, then of dbias; a single one is the gradient
    const long long HD = (long long)a.H * a.d, rows = (long long)a.B * s.ntb;
    float *pw = rows == 1 ? g.dw : ws, *pb = rows == 1 && g.dbias ? g.dbias : ws + rows * HD * a.K;
    if (a.B > 0) {
        cudaError_t e;
        if (a.io_dtype == FALCON_BF16) e = V == 2 ? conv_bwd_io<__nv_bfloat16, 2>(a, g, s, pw, pb, st) : conv_bwd_io<__nv_bfloat16, 1>(a, g, s, pw, pb, st);
        else e = V == 2 ? conv_bwd_io<float, 2>(a, g, s, pw, pb, st) : conv_bwd_io<float, 1>(a, g, s, pw, pb, st);
        if (e != cudaSuccess) return e;
    }
    if (rows == 1) return cudaSuccess;
    const SumJob jobs[2] = {{pw, HD * a.K, HD * a.K, g.dw}, {pb, HD, HD, g.dbias}};
    return launch_column_sums(jobs, 2, rows, st);
}

}  // namespace falcon
