// k_routed.cu -- a routed layer for a few tokens: scores, choice, experts, joined output.
//
//   r_te = x_t . router_e + bias_e,   the K largest of a token are its experts (lower ones first among equal),
//   w    = their softmax weights (over all experts, or over the chosen ones),
//   out_t = sum_k w_k down_e (silu(gate_e x_t) * up_e x_t),   e = the k-th expert of t.
// A few tokens read far more weights than they compute with: the chosen experts' 3 F H weights bound it.
// Here are the scores (64 tokens of 64 experts, H = 2048: 9 us, beside which the next kernel comes up) and, for fp32 and for
// sizes that the tensor cores' copies do not take, a kernel of warps for each step (k_routed_tc.cu has the others): a warp an
// output, an expert's row read again for each of its tokens (H = 2048, F = 1024, 8 of 64 experts, 1 / 8 / 64 tokens: bf16 with
// rows of x off their 16 bytes 73 / 311 / 1850 us, where the tensor cores take 31 / 97 / 150; fp32 78 / 364 / 2410).
#include <cuda_runtime.h>

#include "kernels.h"
#include "routed.cuh"

namespace sot {

namespace {

constexpr int NT = 256, NW = NT / 32;

// Scores.  Two experts' scores may lie closer than a 32-bit sum tells them apart, and which is chosen must not
// depend on the order of a sum: products of 16-bit types are exact in 32 bits, and sums go in pairs of floats.
// A CTA takes an expert and up to eight tokens; with fewer, each token's sum is split over several warps.
template <int DT>
__device__ __forceinline__ void add_product(float2& s, float2& low, float2 x, float2 r) {
    const float2 minus = make_float2(-1.f, -1.f), p = fmul2(x, r), t = fadd2(s, p), z = ffma2(s, minus, t);
    // what t has lost of s + p, lane by lane
    const float2 e = fadd2(ffma2(ffma2(z, minus, t), minus, s), ffma2(z, minus, p));
    if constexpr (DT == SOT_F32) low = fadd2(low, ffma2(x, r, make_float2(-p.x, -p.y)));
    low = fadd2(low, e);
    s = t;
}
template <int DT>
__global__ void __launch_bounds__(NT) routed_scores_kernel(const RoutedArgs a, int tokens, bool whole, unsigned* zero, int zeros) {
    using T = typename Elem<DT>::T;
    constexpr int N = Elem<DT>::N;
    __shared__ float2 part[NW];
    __shared__ float plain[NW];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int i = blockIdx.x * NT + threadIdx.x; i < zeros; i += gridDim.x * NT) zero[i] = 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, splits = NW / tokens;
    const int e = blockIdx.x % a.E, t = blockIdx.x / a.E * tokens + warp / splits, split = warp % splits;
    float2 s = make_float2(0.f, 0.f), low = s;
    if (t < a.T) {
        const T* const x = static_cast<const T*>(a.x) + t * a.ldx;
        const T* const r = static_cast<const T*>(a.router) + (long long)e * a.H;
        if (whole) {
#pragma unroll 4
            for (int i = (split * 32 + lane) * N; i < a.H; i += splits * 32 * N) {
                float2 f[N / 2], g[N / 2];
                unpack<DT>(*reinterpret_cast<const uint4*>(x + i), f);
                unpack<DT>(*reinterpret_cast<const uint4*>(r + i), g);
#pragma unroll
                for (int j = 0; j < N / 2; ++j) add_product<DT>(s, low, f[j], g[j]);
            }
        } else
            for (int i = split * 32 + lane; i < a.H; i += splits * 32)
                add_product<DT>(s, low, make_float2(Elem<DT>::get(x[i]), 0.f), make_float2(Elem<DT>::get(r[i]), 0.f));
    }
    const float far = warp_sum(s.x + s.y);
    const float2 both = ff_warp_sum(ff_add(ff_renorm(s.x, low.x), ff_renorm(s.y, low.y)));
    if (lane == 0) {
        part[warp] = both;
        plain[warp] = far;
    }
    __syncthreads();
    if (split || lane || t >= a.T) return;
    const float bias = a.bias ? a.bias[e] : 0.f;
    float2 sum = make_float2(bias, 0.f);
    float all = bias;
    for (int w = warp; w < warp + splits; ++w) {
        sum = ff_add(sum, part[w]);
        all += plain[w];
    }
    // (an infinity or NaN goes without the low parts, which would make a NaN of either)
    a.logits[(long long)t * a.E + e] = fabsf(all) < INFINITY ? sum.x + sum.y : all;
}
template <int DT>
cudaError_t launch_scores(const RoutedArgs& a, unsigned* zero, int zeros, cudaStream_t st) {
    int tokens = 1;
    while (tokens < NW && tokens < a.T) tokens *= 2;
    const bool whole = a.H % Elem<DT>::N == 0 && a.ldx % Elem<DT>::N == 0 && (unsigned long long)a.x % 16 == 0 &&
                       (unsigned long long)a.router % 16 == 0;
    count_launches(1);
    routed_scores_kernel<DT><<<a.E * ((a.T + tokens - 1) / tokens), NT, 0, st>>>(a, tokens, whole, zero, zeros);
    return cudaGetLastError();
}

// Choice: a warp a token.
__global__ void __launch_bounds__(NT) routed_choose_kernel(const RoutedArgs a) {
    const int lane = threadIdx.x & 31, t = blockIdx.x * NW + (threadIdx.x >> 5);
    if (t >= a.T) return;
    int id;
    float w;
    routed_choose(a.logits + (long long)t * a.E, a.E, a.K, a.renorm, a.scale, id, w);
    if (lane < a.K) {
        a.ids[t * a.K + lane] = id;
        a.weights[t * a.K + lane] = w;
    }
}

// h[p][f] = silu(gate x) * up x for the pairs p = (token, choice) of an expert: a warp a column f.
template <int DT>
__global__ void __launch_bounds__(NT) routed_up_kernel(const RoutedArgs a, int blocks) {
    using T = typename Elem<DT>::T;
    const int lane = threadIdx.x & 31, e = blockIdx.x / blocks, f = blockIdx.x % blocks * NW + (threadIdx.x >> 5);
    if (f >= a.F) return;
    const T* const g = static_cast<const T*>(a.gate_up) + ((long long)e * 2 * a.F + f) * a.H;
    const T* const u = g + (long long)a.F * a.H;
    for (int p0 = 0; p0 < a.T * a.K; p0 += 32) {
        unsigned hit = __ballot_sync(0xffffffffu, p0 + lane < a.T * a.K && a.ids[p0 + lane] == e);
        for (; hit; hit &= hit - 1) {
            const int p = p0 + __ffs(hit) - 1;
            const T* const x = static_cast<const T*>(a.x) + (long long)(p / a.K) * a.ldx;
            float sg = 0.f, su = 0.f;
            for (int i = lane; i < a.H; i += 32) {
                const float v = Elem<DT>::get(x[i]);
                sg = fmaf(v, Elem<DT>::get(g[i]), sg);
                su = fmaf(v, Elem<DT>::get(u[i]), su);
            }
            sg = warp_sum(sg);
            su = warp_sum(su);
            if (lane == 0) a.h[(long long)p * a.F + f] = sg / (1.f + expf(-sg)) * su;
        }
    }
}

// y[p][i] = down h[p]: a warp a row i of the expert.
template <int DT>
__global__ void __launch_bounds__(NT) routed_down_kernel(const RoutedArgs a, int blocks) {
    using T = typename Elem<DT>::T;
    const int lane = threadIdx.x & 31, e = blockIdx.x / blocks, i = blockIdx.x % blocks * NW + (threadIdx.x >> 5);
    if (i >= a.H) return;
    const T* const d = static_cast<const T*>(a.down) + ((long long)e * a.H + i) * a.F;
    for (int p0 = 0; p0 < a.T * a.K; p0 += 32) {
        unsigned hit = __ballot_sync(0xffffffffu, p0 + lane < a.T * a.K && a.ids[p0 + lane] == e);
        for (; hit; hit &= hit - 1) {
            const int p = p0 + __ffs(hit) - 1;
            float s = 0.f;
            for (int f = lane; f < a.F; f += 32) s = fmaf(a.h[(long long)p * a.F + f], Elem<DT>::get(d[f]), s);
            s = warp_sum(s);
            if (lane == 0) a.y[(long long)p * a.H + i] = s;
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(NT) routed_join_kernel(const RoutedArgs a) {
    const long long at = (long long)blockIdx.x * NT + threadIdx.x;
    if (at >= (long long)a.T * a.H) return;
    const int t = (int)(at / a.H), i = (int)(at % a.H);
    float s = 0.f;
    for (int k = 0; k < a.K; ++k) {
        const int p = t * a.K + k;
        if (a.ids[p] >= 0) s = fmaf(a.weights[p], a.y[(long long)p * a.H + i], s);
        else s += a.weights[p];  // 0, or NaN
    }
    static_cast<typename Elem<DT>::T*>(a.out)[t * a.ldo + i] = Elem<DT>::put(s);
}

template <int DT>
cudaError_t launch_plain(const RoutedArgs& a, cudaStream_t st) {
    const int up = (a.F + NW - 1) / NW, down = (a.H + NW - 1) / NW;
    const cudaError_t e = launch_scores<DT>(a, nullptr, 0, st);
    if (e != cudaSuccess) return e;
    count_launches(4);
    routed_choose_kernel<<<(a.T + NW - 1) / NW, NT, 0, st>>>(a);
    routed_up_kernel<DT><<<a.E * up, NT, 0, st>>>(a, up);
    routed_down_kernel<DT><<<a.E * down, NT, 0, st>>>(a, down);
    routed_join_kernel<DT><<<(unsigned)(((long long)a.T * a.H + NT - 1) / NT), NT, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

// The tensor cores need whole granules; the other form takes any size, stride and type, with a warp an output.
RoutedPlan routed_plan(const RoutedArgs& a, int sms) {
    RoutedPlan p = {};
    p.tc = routed_tc_fits(a);
    if (p.tc) {
        p.on_tc = routed_tc_plan(a, sms);
        p.scratch = p.on_tc.scratch;
        return p;
    }
    p.y_at = (sizeof(float) * (size_t)a.T * a.K * a.F + 255) & ~(size_t)255;
    p.scratch = p.y_at + sizeof(float) * (size_t)a.T * a.K * a.H;
    return p;
}

cudaError_t launch_routed(RoutedArgs a, const RoutedPlan& p, unsigned char* scratch, int sms, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    if (p.tc) {
        unsigned* const zero = reinterpret_cast<unsigned*>(scratch + p.on_tc.barrier_at);
        const int zeros = p.on_tc.zeros;
        const cudaError_t e = a.dtype == SOT_BF16 ? launch_scores<SOT_BF16>(a, zero, zeros, st) : launch_scores<SOT_F16>(a, zero, zeros, st);
        return e != cudaSuccess ? e : launch_routed_tc(a, p.on_tc, scratch, sms, st);
    }
    a.h = reinterpret_cast<float*>(scratch + p.h_at);
    a.y = reinterpret_cast<float*>(scratch + p.y_at);
    switch (a.dtype) {
        case SOT_F32: return launch_plain<SOT_F32>(a, st);
        case SOT_F16: return launch_plain<SOT_F16>(a, st);
        default: return launch_plain<SOT_BF16>(a, st);
    }
}

}  // namespace sot
