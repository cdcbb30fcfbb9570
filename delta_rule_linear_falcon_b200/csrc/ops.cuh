// ops.cuh -- device helpers of the operators around the memory.
#pragma once

#include "common.cuh"
#include "ops.h"

namespace falcon {

// V consecutive elements as one access: `raw` is what a load leaves in registers, so that a
// prefetched value costs no conversion before it is used.
template <typename IO, int V> struct Pack;

template <> struct Pack<float, 1> {
    typedef float raw;
    static __device__ __forceinline__ raw ld(const float *p) { return *p; }
    static __device__ __forceinline__ raw zero() { return 0.f; }
    static __device__ __forceinline__ void cvt(raw r, float (&x)[1]) { x[0] = r; }
    static __device__ __forceinline__ void st(float *p, const float (&x)[1]) { *p = x[0]; }
};
template <> struct Pack<float, 2> {
    typedef float2 raw;
    static __device__ __forceinline__ raw ld(const float *p) { return *reinterpret_cast<const float2 *>(p); }
    static __device__ __forceinline__ raw zero() { return make_float2(0.f, 0.f); }
    static __device__ __forceinline__ void cvt(raw r, float (&x)[2]) { x[0] = r.x; x[1] = r.y; }
    static __device__ __forceinline__ void st(float *p, const float (&x)[2]) { *reinterpret_cast<float2 *>(p) = make_float2(x[0], x[1]); }
};
template <> struct Pack<float, 4> {
    typedef float4 raw;
    static __device__ __forceinline__ raw ld(const float *p) { return *reinterpret_cast<const float4 *>(p); }
    static __device__ __forceinline__ raw zero() { return make_float4(0.f, 0.f, 0.f, 0.f); }
    static __device__ __forceinline__ void cvt(raw r, float (&x)[4]) { x[0] = r.x; x[1] = r.y; x[2] = r.z; x[3] = r.w; }
    static __device__ __forceinline__ void st(float *p, const float (&x)[4]) {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    }
};
template <> struct Pack<__nv_bfloat16, 1> {
    typedef __nv_bfloat16 raw;
    static __device__ __forceinline__ raw ld(const __nv_bfloat16 *p) { return *p; }
    static __device__ __forceinline__ raw zero() { return __float2bfloat16(0.f); }
    static __device__ __forceinline__ void cvt(raw r, float (&x)[1]) { x[0] = __bfloat162float(r); }
    static __device__ __forceinline__ void st(__nv_bfloat16 *p, const float (&x)[1]) { *p = __float2bfloat16_rn(x[0]); }
};
__device__ __forceinline__ void unpack_bf16x2(uint32_t u, float &lo, float &hi) {
    lo = __uint_as_float(u << 16);
    hi = __uint_as_float(u & 0xffff0000u);
}
template <> struct Pack<__nv_bfloat16, 2> {
    typedef uint32_t raw;
    static __device__ __forceinline__ raw ld(const __nv_bfloat16 *p) { return *reinterpret_cast<const uint32_t *>(p); }
    static __device__ __forceinline__ raw zero() { return 0u; }
    static __device__ __forceinline__ void cvt(raw r, float (&x)[2]) { unpack_bf16x2(r, x[0], x[1]); }
    static __device__ __forceinline__ void st(__nv_bfloat16 *p, const float (&x)[2]) {
        *reinterpret_cast<uint32_t *>(p) = pack_bf16x2(x[0], x[1]);
    }
};
template <> struct Pack<__nv_bfloat16, 4> {
    typedef uint2 raw;
    static __device__ __forceinline__ raw ld(const __nv_bfloat16 *p) { return *reinterpret_cast<const uint2 *>(p); }
    static __device__ __forceinline__ raw zero() { return make_uint2(0u, 0u); }
    static __device__ __forceinline__ void cvt(raw r, float (&x)[4]) {
        unpack_bf16x2(r.x, x[0], x[1]);
        unpack_bf16x2(r.y, x[2], x[3]);
    }
    static __device__ __forceinline__ void st(__nv_bfloat16 *p, const float (&x)[4]) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    }
};
// Asynchronous copy of 4, 8 or 16 bytes into the thread's own place in shared memory, and the wait for all but the
// newest N groups of them.
template <int BYTES>
__device__ __forceinline__ void copy_async(void *smem, const void *global) {
    const unsigned s = (unsigned)__cvta_generic_to_shared(smem);
    if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(global) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(s), "l"(global), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <typename E>
__device__ __forceinline__ E *row_of(const falcon_view_t &v, long long b, long long h, long long t) {
    return reinterpret_cast<E *>(v.p) + b * v.sb + h * v.sh + t * v.st;
}

// Tokens of sequence b: lengths[b] clamped to [0, T].
__device__ __forceinline__ int seq_length(const int *lengths, int b, int T) {
    return lengths ? min(max(lengths[b], 0), T) : T;
}

__device__ __forceinline__ float fast_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float silu(float x) { return x / (1.f + __expf(-x)); }
// log(1 + e^x) = max(x, 0) + log(1 + e), e = e^-|x| <= 1, and log(1 + e) / e on [0, 1] by a polynomial whose constant is
// 1 and whose other eight coefficients are a least-squares fit reweighted towards equal errors (3e-8 of the value, 2e-7
// with its roundings). As exact for very negative x, where the result is e^x, as for others; one operation of the
// exponential unit (a quotient in place of half of the polynomial takes another).
#define FALCON_LOG1P(F, S) \
    F(F(F(F(F(F(F(F(S(0.005364812f), S(-0.030065743f)), S(0.079204455f)), S(-0.13753796f)), S(0.19153652f)), S(-0.24857163f)), \
          S(0.33321324f)), S(-0.49999648f)), S(1.f))
__device__ __forceinline__ float softplus(float x) {
    const float e = fast_ex2(-1.4426950408889634f * fabsf(x));
    const auto f = [e](float p, float c) { return fmaf(p, e, c); };
    const auto s = [](float c) { return c; };
    return fmaf(e, FALCON_LOG1P(f, s), fmaxf(x, 0.f));
}

// Two fp32 values in a 64-bit register pair; one instruction works on both (sm_100).
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.ftz.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.ftz.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.ftz.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 ex2_2(f32x2 a) {
    float lo, hi;
    unpack2(a, lo, hi);
    return pack2(fast_ex2(lo), fast_ex2(hi));
}
// The same on the multiply-add pipes, for kernels that the exponential unit bounds: x = n + f with n the nearest
// whole number (the low bits of x + 1.5 2^23), 2^f by a polynomial of degree 5 on [-1/2, 1/2] with constant 1 (a
// least-squares fit reweighted towards equal errors: 2e-7 of the value with its roundings, as good as the unit's, and
// exact towards f = 0), n added to the exponent. For x <= 0; below -125 the value is 2^-125.
__device__ __forceinline__ f32x2 ex2_poly2(f32x2 a) {
    float lo, hi;
    unpack2(a, lo, hi);
    const f32x2 x = pack2(fmaxf(lo, -125.f), fmaxf(hi, -125.f));
    const f32x2 t = add2(x, pack2(12582912.f, 12582912.f));
    const f32x2 f = fma2(add2(t, pack2(-12582912.f, -12582912.f)), pack2(-1.f, -1.f), x);
    f32x2 p = fma2(f, pack2(0.0013264726f, 0.0013264726f), pack2(0.009671513f, 0.009671513f));
    p = fma2(f, p, pack2(0.055507336f, 0.055507336f));
    p = fma2(f, p, pack2(0.24022242f, 0.24022242f));
    p = fma2(f, p, pack2(0.693147f, 0.693147f));
    p = fma2(f, p, pack2(1.f, 1.f));
    float pl, ph, tl, th;
    unpack2(p, pl, ph);
    unpack2(t, tl, th);
    return pack2(__int_as_float(__float_as_int(pl) + (__float_as_int(tl) << 23)),
                 __int_as_float(__float_as_int(ph) + (__float_as_int(th) << 23)));
}
__device__ __forceinline__ float sum2(f32x2 a) {
    float lo, hi;
    unpack2(a, lo, hi);
    return lo + hi;
}
__device__ __forceinline__ float fast_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// softplus, 1 / (1 + e^-x) and x / (1 + e^-x) of two values.
__device__ __forceinline__ f32x2 softplus2(f32x2 x) {
    float a, b;
    unpack2(x, a, b);
    const f32x2 e = pack2(fast_ex2(-1.4426950408889634f * fabsf(a)), fast_ex2(-1.4426950408889634f * fabsf(b)));
    const auto f = [e](f32x2 p, f32x2 c) { return fma2(p, e, c); };
    const auto s = [](float c) { return pack2(c, c); };
    return fma2(e, FALCON_LOG1P(f, s), pack2(fmaxf(a, 0.f), fmaxf(b, 0.f)));
}
__device__ __forceinline__ f32x2 sigmoid2(f32x2 x) {
    float a, b;
    unpack2(add2(ex2_2(mul2(x, pack2(-1.4426950408889634f, -1.4426950408889634f))), pack2(1.f, 1.f)), a, b);
    return pack2(fast_rcp(a), fast_rcp(b));
}
__device__ __forceinline__ f32x2 silu2(f32x2 x) { return mul2(x, sigmoid2(x)); }
// Four floats of a 16-byte aligned row as two pairs.
__device__ __forceinline__ void load_pairs(const float *p, f32x2 &a, f32x2 &b) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(p);
    a = v.x;
    b = v.y;
}
__device__ __forceinline__ void store_pairs(float *p, f32x2 a, f32x2 b) {
    *reinterpret_cast<ulonglong2 *>(p) = make_ulonglong2(a, b);
}

// Host: whether a view takes accesses of `bytes` bytes (pointer and strides), V elements of es bytes.
inline bool view_packs(const falcon_view_t &v, int V, int es) {
    if (!v.p) return true;
    return reinterpret_cast<uintptr_t>(v.p) % (size_t)(V * es) == 0 && v.sb % V == 0 && v.sh % V == 0 && v.st % V == 0;
}

// Sums v[0..N) over NL lanes whose numbers differ by multiples of STRIDE (a power of two): as long as
// a lane holds more than one value each step hands half of them to the partner and keeps the rest
// (N + N/2 + ... shuffles instead of N log NL). Leaves max(1, N / NL) totals in v[0..]; returns the
// index of the first. Where NL > N, lanes with equal index hold the same totals; `first` says which writes.
template <int N, int NL, int STRIDE>
__device__ __forceinline__ int lanes_sum(float (&v)[N], int lane, bool &first) {
    int idx = 0;
    first = true;
    int n = N;
#pragma unroll
    for (int m = NL / 2; m >= 1; m >>= 1) {
        const bool hi = (lane & (m * STRIDE)) != 0;
        if (n > 1) {
            n >>= 1;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                if (i < n) {
                    const float send = hi ? v[i] : v[i + n];
                    const float keep = hi ? v[i + n] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, send, m * STRIDE);
                }
            }
            if (hi) idx += n;
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], m * STRIDE);
            if (hi) first = false;
        }
    }
    return idx;
}

}  // namespace falcon
