// lm.cuh -- device helpers of the language-model loss kernels: 16-byte granules of
// logits in three types, softmax statistics, float-pair sums and logarithms,
// clusters.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "common.cuh"
#include "sot.h"
#include "tc_ptx.cuh"

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
    using T2 = __half2;
    static constexpr int N = 8;
    __device__ static float get(T v) { return __half2float(v); }
    __device__ static T put(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<SOT_BF16> {
    using T = __nv_bfloat16;
    using T2 = __nv_bfloat162;
    static constexpr int N = 8;
    __device__ static float get(T v) { return __bfloat162float(v); }
    __device__ static T put(float v) { return __float2bfloat16_rn(v); }
};

// Packed product of two floats by two (one instruction, each lane rounded as the scalar product).
__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2,%3};\n\tmov.b64 rb, {%4,%5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0,%1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

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
// Largest of the N elements (packed maxima for the 16-bit types; NaN is passed over).
template <int DT>
__device__ __forceinline__ float max_of(const uint4& v) {
    if constexpr (DT == SOT_F32) {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    } else if constexpr (DT == SOT_BF16) {
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
        const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return __bfloat162float(__hmax(m.x, m.y));
    } else {
        const __half2* h = reinterpret_cast<const __half2*>(&v);
        const __half2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return __half2float(__hmax(__low2half(m), __high2half(m)));
    }
}
// L2 eviction policies of 16-byte accesses: what is read again soon stays longest,
// what is read for the last time or written goes first.
__device__ __forceinline__ uint64_t policy_keep() {
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ uint64_t policy_drop() {
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
// (Not volatile: no kernel reads an address again after it has written it.)
__device__ __forceinline__ uint4 load16(const uint4* p, uint64_t policy) {
    uint4 v;
    asm("ld.global.L2::cache_hint.v4.u32 {%0,%1,%2,%3}, [%4], %5;"
        : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
        : "l"(p), "l"(policy));
    return v;
}
__device__ __forceinline__ void store16(uint4* p, const uint4& v, uint64_t policy) {
    asm volatile("st.global.L2::cache_hint.v4.u32 [%0], {%1,%2,%3,%4}, %5;" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w), "l"(policy)
                 : "memory");
}

// One element at p, copied to shared memory behind the thread's back as the 32-bit word
// around it; element_of gives it after async_wait.
template <class T>
__device__ __forceinline__ void fetch_element(float* to, const T* p) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to)), "l"((unsigned long long)p & ~3ull) : "memory");
}
__device__ __forceinline__ void async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
template <int DT>
__device__ __forceinline__ float element_of(float word, const typename Elem<DT>::T* p) {
    if constexpr (sizeof(*p) == 4) return word;
    else {
        const uint32_t b = __float_as_uint(word);
        const unsigned short h = (unsigned short)((unsigned long long)p & 2ull ? b >> 16 : b);
        typename Elem<DT>::T e;
        memcpy(&e, &h, sizeof(e));
        return Elem<DT>::get(e);
    }
}

template <int DT>
__device__ __forceinline__ uint4 nothing() {  // N times -inf
    constexpr unsigned w = DT == SOT_F32 ? 0xff800000u : DT == SOT_F16 ? 0xfc00fc00u : 0xff80ff80u;
    return make_uint4(w, w, w, w);
}
// Largest elements of two vectors, element by element.
template <int DT>
__device__ __forceinline__ uint4 max2(const uint4& a, const uint4& b) {
    uint4 r;
    if constexpr (DT == SOT_F32) {
        r.x = __float_as_uint(fmaxf(__uint_as_float(a.x), __uint_as_float(b.x)));
        r.y = __float_as_uint(fmaxf(__uint_as_float(a.y), __uint_as_float(b.y)));
        r.z = __float_as_uint(fmaxf(__uint_as_float(a.z), __uint_as_float(b.z)));
        r.w = __float_as_uint(fmaxf(__uint_as_float(a.w), __uint_as_float(b.w)));
    } else {
        using H = typename Elem<DT>::T2;
        const H *p = reinterpret_cast<const H*>(&a), *q = reinterpret_cast<const H*>(&b);
        H* o = reinterpret_cast<H*>(&r);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = __hmax2(p[i], q[i]);
    }
    return r;
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

// Writes N elements at columns e .. e + N - 1 of a row (those of them that exist).
template <int DT>
__device__ __forceinline__ void store_cols(typename Elem<DT>::T* row, int e, int V,
                                           const float2 (&f)[Elem<DT>::N / 2], bool aligned) {
    constexpr int N = Elem<DT>::N;
    if (aligned && e >= 0 && e + N <= V) {
        *reinterpret_cast<uint4*>(row + e) = pack<DT>(f);
        return;
    }
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        if (e + 2 * i >= 0 && e + 2 * i < V) row[e + 2 * i] = Elem<DT>::put(f[i].x);
        if (e + 2 * i + 1 >= 0 && e + 2 * i + 1 < V) row[e + 2 * i + 1] = Elem<DT>::put(f[i].y);
    }
}

// Replaces the elements at columns outside [0, V).
template <int DT>
__device__ __forceinline__ void mask_cols(float2 (&f)[Elem<DT>::N / 2], int e, int V, float fill) {
#pragma unroll
    for (int i = 0; i < Elem<DT>::N / 2; ++i) {
        if (e + 2 * i < 0 || e + 2 * i >= V) f[i].x = fill;
        if (e + 2 * i + 1 < 0 || e + 2 * i + 1 >= V) f[i].y = fill;
    }
}

// Whether two rows start at the same place of a granule.
template <class T>
__device__ __forceinline__ bool same_granules(const T* x, const T* g) {
    return ((uint32_t)((unsigned long long)x ^ (unsigned long long)g) & 15u) == 0;
}

// Softmax statistics of a set of logits with sc = log2(e) / temperature: its
// stabiliser m (its largest value, or one near enough for the sums' range) and
// s = sum exp2(x sc - m2), m2 = m sc rounded to 32 bits.
// Taking the rounded m2 everywhere (sums, joins, probabilities) makes its
// rounding cancel; only the fused x sc - m2 is rounded, at the size of the
// result.  Where m2 overflows (m near the type's lowest or largest value) the
// neighbouring numbers are so far apart that only logits equal to m have any
// weight: s counts those.  A set of nothing but -inf has s = 0.
struct MS {
    float m, s;
};
// Whether a stabiliser is so far from 0 (m2 its rounded product with sc) that floats next to
// it lie 2^6 or more apart in the exponent: then only the logits equal to it count.
// Below that, m2 is off by 2^5 at most, which all weights share.
__device__ __forceinline__ bool is_far(float m2) { return !(fabsf(m2) < 0x1p30f); }
// (infinite x and m are not equal here: such a row has no sum)
__device__ __forceinline__ float equal_weight(float x, float m) { return x - m == 0.f ? 1.f : x != x ? x : 0.f; }
// Weight of a logit x against stabiliser m.
__device__ __forceinline__ float weight_of(float x, float m, float sc) {
    const float m2 = __fmul_rn(m, sc);
    if (!is_far(m2)) return ex2f(fmaf(x, sc, -m2));
    return equal_weight(x, m);
}
// Factor that takes sums against stabiliser m to stabiliser M >= m.
__device__ __forceinline__ float rescale(float m, float M, float sc) {
    const float M2 = __fmul_rn(M, sc);
    if (!is_far(M2)) return ex2f(__fsub_rn(__fmul_rn(m, sc), M2));  // not fused: the rounded products
    return m - M == 0.f ? 1.f : 0.f;
}
__device__ __forceinline__ MS ms_combine(MS a, MS b, float sc) {
    const float M = fmaxf(a.m, b.m);
    return MS{M, a.s * rescale(a.m, M, sc) + b.s * rescale(b.m, M, sc)};
}
// Largest value of a warp, in every lane: one reduction instruction.
__device__ __forceinline__ float warp_max1(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ MS ms_warp(MS v, float sc) {
    const float M = warp_max1(v.m);
    return MS{M, warp_sum(v.s * rescale(v.m, M, sc))};
}

// exp2(x sc - u) of a pair.
__device__ __forceinline__ float2 ex2_pair(float2 x, float u, float sc) {
    const float2 t = ffma2(x, make_float2(sc, sc), make_float2(-u, -u));
    return make_float2(ex2f(t.x), ex2f(t.y));
}

// A thread's running statistics: s (in two halves) against stabiliser m, u = m sc
// rounded; where that is far from 0, s counts the logits equal to m.  Nothing needs m to be the largest value, only the sums to stay clear of
// overflow and underflow, and logits seldom leave the range where the first
// guess, 0, does that.  So a batch is summed against the m at hand, with no
// maximum to wait for, and only a batch whose sum comes out beyond 2^24 or
// below 2^-40 is looked at again.
struct Running {
    float m, u;
    float2 s;
    bool far;
    __device__ __forceinline__ Running() : m(0.f), u(0.f), s(make_float2(0.f, 0.f)), far(false) {}

    template <int DT>
    __device__ __forceinline__ float2 sum(const uint4& v, float sc) const {
        float2 f[Elem<DT>::N / 2], t = make_float2(0.f, 0.f);
        unpack<DT>(v, f);
        if (!far) {
#pragma unroll
            for (int i = 0; i < Elem<DT>::N / 2; ++i) t = fadd2(t, ex2_pair(f[i], u, sc));
        } else {
#pragma unroll
            for (int i = 0; i < Elem<DT>::N / 2; ++i)
                t = fadd2(t, make_float2(equal_weight(f[i].x, m), equal_weight(f[i].y, m)));
        }
        return t;
    }
    // A batch with largest value mx whose sum is out of range: m moves to mx if
    // that is larger, or if nothing has been summed yet.
    __device__ __forceinline__ void move(float mx, float sc) {
        const bool none = s.x == 0.f && s.y == 0.f;
        if ((none && mx > -INFINITY) || mx > m) {
            const float k = none ? 0.f : rescale(m, mx, sc), v = __fmul_rn(mx, sc);
            s = fmul2(s, make_float2(k, k));
            m = mx;
            far = is_far(v);
            u = far ? 0.f : v;
            if (mx == INFINITY) s = make_float2(NAN, 0.f);  // and stays
        }
    }
    template <int DT, int P>
    __device__ __forceinline__ void add(const uint4 (&v)[P], float sc) {
        float2 t = make_float2(0.f, 0.f);
        if (!far) {
            float2 f[Elem<DT>::N / 2];
#pragma unroll
            for (int j = 0; j < P; ++j) {
                unpack<DT>(v[j], f);
                float2 w = ex2_pair(f[0], u, sc);
#pragma unroll
                for (int i = 1; i < Elem<DT>::N / 2; ++i) w = fadd2(w, ex2_pair(f[i], u, sc));
                t = fadd2(t, w);
            }
        }
        const float both = t.x + t.y;
        if (!(both > 0x1p-40f && both < 0x1p24f)) {
            uint4 top = v[0];
#pragma unroll
            for (int j = 1; j < P; ++j) top = max2<DT>(top, v[j]);
            move(max_of<DT>(top), sc);
            t = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < P; ++j) t = fadd2(t, sum<DT>(v[j], sc));
        }
        s = fadd2(s, t);
    }
    __device__ __forceinline__ MS result() const {
        const float both = s.x + s.y;
        return MS{both == 0.f ? -INFINITY : m, both};
    }
};

// log s for s > 0 as an unevaluated sum, absolute error near 2^-25: s = 2^e f with
// f in [0.75, 1.5), e times a 12-bit head of ln 2 is exact, the rest is rounded
// at the size of log f.  +-0, infinities and NaN go to logf.
__device__ __forceinline__ float2 log_ff(float s) {
    if (!(s >= 1.17549435e-38f && s < INFINITY)) return make_float2(logf(s), 0.f);
    constexpr float head = 2839.f / 4096.f, rest = (float)(0.69314718055994530942 - 2839.0 / 4096.0);
    const int e = (int)(__float_as_uint(s) - 0x3f400000u) >> 23;
    const float f = __uint_as_float(__float_as_uint(s) - ((uint32_t)e << 23));
    const float2 r = two_sum(__fmul_rn((float)e, head), fmaf((float)e, rest, logf(f)));
    return r;
}
__device__ __forceinline__ double to_double(float2 v) { return (double)v.x + (double)v.y; }
__device__ __forceinline__ float2 ff_warp_sum(float2 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float2 w = make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o));
        v = ff_add(v, w);
    }
    return v;
}

// exp(u) - u - 1 without the cancellation of small u (Taylor series to u^9); +inf at both ends.
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
    return u == INFINITY ? u : expm1f(u) - u;
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
// Its two halves, without ordering memory: this CTA has started; all have.
__device__ __forceinline__ void cluster_arrive_started() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait_started() {
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
// The address in CTA `rank` of the cluster of a shared-memory address of this one.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
    uint32_t ra;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(addr), "r"(rank));
    return ra;
}
__device__ __forceinline__ void cluster_store(uint32_t ra, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(ra), "f"(v) : "memory");
}

}  // namespace sot
