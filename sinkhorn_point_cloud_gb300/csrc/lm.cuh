// lm.cuh -- device helpers of the language-model loss kernels: 16-byte
// vectors of logits in three types, (max, sum) pairs of a softmax, and a
// logarithm that keeps more than 24 bits.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "common.cuh"
#include "sot.h"

namespace sot {

template <int DT>
struct Elem;
template <>
struct Elem<SOT_F32> {
    using T = float;
    static constexpr int N = 4;  // elements of 16 bytes
    __device__ static float get(T v) { return v; }
    __device__ static T put(float v) { return v; }
};
template <>
struct Elem<SOT_F16> {
    using T = __half;
    static constexpr int N = 8;
    __device__ static float get(T v) { return __half2float(v); }
    __device__ static T put(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<SOT_BF16> {
    using T = __nv_bfloat16;
    static constexpr int N = 8;
    __device__ static float get(T v) { return __bfloat162float(v); }
    __device__ static T put(float v) { return __float2bfloat16_rn(v); }
};

// 16 bytes <-> N floats, in pairs.
template <int DT>
__device__ __forceinline__ void unpack(const uint4& v, float2 (&f)[Elem<DT>::N / 2]) {
    if constexpr (DT == SOT_F32) {
        f[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
        f[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
    } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == SOT_BF16)
                f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
            else {
                __half2 h;
                *reinterpret_cast<uint32_t*>(&h) = w[i];
                f[i] = __half22float2(h);
            }
        }
    }
}
template <int DT>
__device__ __forceinline__ uint4 pack(const float2 (&f)[Elem<DT>::N / 2]) {
    uint4 v;
    if constexpr (DT == SOT_F32) {
        v = make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                       __float_as_uint(f[1].y));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == SOT_BF16) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[i].x, f[i].y);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __half2 h = __floats2half2_rn(f[i].x, f[i].y);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return v;
}

__device__ __forceinline__ float load_float(const void* p, int type, long long i) {
    if (type == SOT_F32) return static_cast<const float*>(p)[i];
    if (type == SOT_F16) return __half2float(static_cast<const __half*>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
// An index in [0, n), or -1.
__device__ __forceinline__ int load_index(const void* p, int type, long long i, int n) {
    const long long v = type == SOT_I64 ? static_cast<const long long*>(p)[i] : static_cast<const int*>(p)[i];
    return v >= 0 && v < n ? (int)v : -1;
}

// Softmax statistics of a set of logits: m = max x, s = sum exp2((x - m) sc)
// with sc = log2(e) / temperature.  The difference is taken before the
// scaling, so logits near the type's largest and lowest values neither
// overflow nor lose a row of equal lowest values.  A set whose largest value
// is -inf has s = 0: its stabiliser is taken as 0.
struct MS {
    float m, s;
};
__device__ __forceinline__ float stab(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ MS ms_combine(MS a, MS b, float sc) {
    const float M = fmaxf(a.m, b.m), u = stab(M);
    return MS{M, a.s * ex2f((a.m - u) * sc) + b.s * ex2f((b.m - u) * sc)};
}
__device__ __forceinline__ MS ms_warp(MS v, float sc) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        MS w;
        w.m = __shfl_xor_sync(0xffffffffu, v.m, o);
        w.s = __shfl_xor_sync(0xffffffffu, v.s, o);
        v = ms_combine(v, w, sc);
    }
    return v;
}

// Adds N logits to a thread's running statistics.
template <int DT>
__device__ __forceinline__ void ms_add(MS& r, const float2 (&f)[Elem<DT>::N / 2], float sc) {
    constexpr int P = Elem<DT>::N / 2;
    float mx = fmaxf(f[0].x, f[0].y);
#pragma unroll
    for (int i = 1; i < P; ++i) mx = fmaxf(mx, fmaxf(f[i].x, f[i].y));
    if (mx > r.m) {
        r.s *= ex2f((r.m - mx) * sc);
        r.m = mx;
    }
    const float u = stab(r.m);
    float2 t = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const float2 d = fadd2(f[i], make_float2(-u, -u));
        t = fadd2(t, make_float2(ex2f(d.x * sc), ex2f(d.y * sc)));
    }
    r.s += t.x + t.y;
}

// log s for s > 0 with an absolute error near 2^-25: the exponent's part is
// exact in 64 bits, the rest is the logarithm of a number in [0.75, 1.5).
// +-0, infinities and NaN go to logf.
__device__ __forceinline__ double log_wide(float s) {
    if (!(s >= 1.17549435e-38f && s < INFINITY)) return (double)logf(s);
    const uint32_t b = __float_as_uint(s) - 0x3f400000u;
    const int e = (int)b >> 23;
    const float f = __uint_as_float(__float_as_uint(s) - ((uint32_t)e << 23));
    return (double)e * 0.69314718055994530942 + (double)logf(f);
}

// exp(u) - u - 1 without the cancellation of small u (Taylor series to u^9).
__device__ __forceinline__ float exp_minus_linear(float u) {
    if (fabsf(u) < 0.5f) {
        float p = 1.f / 362880.f;
        p = fmaf(p, u, 1.f / 40320.f);
        p = fmaf(p, u, 1.f / 5040.f);
        p = fmaf(p, u, 1.f / 720.f);
        p = fmaf(p, u, 1.f / 120.f);
        p = fmaf(p, u, 1.f / 24.f);
        p = fmaf(p, u, 1.f / 6.f);
        p = fmaf(p, u, 0.5f);
        return u * u * p;
    }
    return expm1f(u) - u;
}

__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Cluster-wide barrier with release / acquire semantics for shared memory.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Store to the same shared-memory location in CTA `rank` of the cluster.
__device__ __forceinline__ void cluster_store(const float* local_ptr, uint32_t rank, float v) {
    const uint32_t la = (uint32_t)__cvta_generic_to_shared(local_ptr);
    uint32_t ra;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(la), "r"(rank));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(ra), "f"(v) : "memory");
}

}  // namespace sot
