// k_routed.cu -- a routed layer for a few tokens: scores, choice, experts, joined output.
//
//   r_te = x_t . router_e + bias_e,   the K largest of a token are its experts (lower ones first among equal),
//   w    = their softmax weights (over all experts, or over the chosen ones),
//   out_t = sum_k w_k down_e (silu(gate_e x_t) * up_e x_t),   e = the k-th expert of t.
// A few tokens read far more weights than they compute with: the chosen experts' 3 F H weights bound it.
#include <cuda_runtime.h>

#include "kernels.h"
#include "lm.cuh"
#include "routed.h"

namespace sot {

namespace {

constexpr int NT = 256, NW = NT / 32;

// Scores.  Two experts' scores may lie closer than a 32-bit sum tells them apart, and which is chosen must not
// depend on the order of a sum: products of 16-bit types are exact in 32 bits, and sums go in pairs of floats.
template <int DT>
__global__ void __launch_bounds__(NT) routed_scores_kernel(const RoutedArgs a) {
    using T = typename Elem<DT>::T;
    const int lane = threadIdx.x & 31, w = blockIdx.x * NW + (threadIdx.x >> 5);
    if (w >= a.T * a.E) return;
    const int t = w / a.E, e = w % a.E;
    const T* const x = static_cast<const T*>(a.x) + t * a.ldx;
    const T* const r = static_cast<const T*>(a.router) + (long long)e * a.H;
    float2 s = make_float2(0.f, 0.f);
    for (int i = lane; i < a.H; i += 32) {
        const float2 p = two_prod(Elem<DT>::get(x[i]), Elem<DT>::get(r[i])), q = two_sum(s.x, p.x);
        s = make_float2(q.x, s.y + (q.y + p.y));
    }
    const float far = warp_sum(s.x);
    s = ff_warp_sum(ff_renorm(s.x, s.y));
    if (a.bias) s = ff_add(s, make_float2(a.bias[e], 0.f));
    // (an infinity or NaN goes without the low parts, which would make a NaN of either)
    if (lane == 0) a.logits[w] = fabsf(far) < INFINITY && !(a.bias && !(fabsf(a.bias[e]) < INFINITY)) ? s.x + s.y
                                                                        : far + (a.bias ? a.bias[e] : 0.f);
}

// Choice: a warp a token.
__global__ void __launch_bounds__(NT) routed_choose_kernel(const RoutedArgs a) {
    const int lane = threadIdx.x & 31, t = blockIdx.x * NW + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const float* const r = a.logits + (long long)t * a.E;
    constexpr int R = ROUTED_MAX_E / 32;
    unsigned key[R];  // 0: -inf, or no expert
    float m = -INFINITY, bad = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int e = i * 32 + lane;
        const float v = e < a.E ? r[e] : -INFINITY;
        if (!(v < INFINITY)) bad = 1.f;
        m = fmaxf(m, v);
        key[i] = v > -INFINITY ? ord_encode(v + 0.f) : 0u;
    }
    m = warp_max(m);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (key[i]) sum += expf(ord_decode(key[i]) - m);
    sum = warp_sum(sum);
    bad = warp_max(bad);
    float chosen = 0.f, mine = 0.f;
    int id = -1;  // lane k: the k-th choice
    for (int k = 0; k < a.K; ++k) {
        unsigned best = 0;
#pragma unroll
        for (int i = 0; i < R; ++i) best = max(best, key[i]);
        best = __reduce_max_sync(0xffffffffu, best);
        if (best == 0 || bad != 0.f) break;
        int at = 0x7fffffff;
#pragma unroll
        for (int i = R - 1; i >= 0; --i)
            if (key[i] == best) at = i * 32 + lane;
        at = __reduce_min_sync(0xffffffffu, at);
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (i * 32 + lane == at) key[i] = 0;
        const float v = expf(ord_decode(best) - m);
        chosen += v;
        if (lane == k) {
            id = at;
            mine = v;
        }
    }
    if (lane < a.K) {
        a.ids[t * a.K + lane] = id;
        a.weights[t * a.K + lane] = bad != 0.f ? NAN : id < 0 ? 0.f : mine / (a.renorm ? chosen : sum) * a.scale;
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
    count_launches(5);
    routed_scores_kernel<DT><<<(a.T * a.E + NW - 1) / NW, NT, 0, st>>>(a);
    routed_choose_kernel<<<(a.T + NW - 1) / NW, NT, 0, st>>>(a);
    routed_up_kernel<DT><<<a.E * up, NT, 0, st>>>(a, up);
    routed_down_kernel<DT><<<a.E * down, NT, 0, st>>>(a, down);
    routed_join_kernel<DT><<<(unsigned)(((long long)a.T * a.H + NT - 1) / NT), NT, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

RoutedPlan routed_plan(const RoutedArgs& a, int) {
    RoutedPlan p = {};
    p.y_at = (sizeof(float) * (size_t)a.T * a.K * a.F + 255) & ~(size_t)255;
    p.scratch = p.y_at + sizeof(float) * (size_t)a.T * a.K * a.H;
    return p;
}

cudaError_t launch_routed(RoutedArgs a, const RoutedPlan& p, unsigned char* scratch, int, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    a.h = reinterpret_cast<float*>(scratch + p.h_at);
    a.y = reinterpret_cast<float*>(scratch + p.y_at);
    switch (a.dtype) {
        case SOT_F32: return launch_plain<SOT_F32>(a, st);
        case SOT_F16: return launch_plain<SOT_F16>(a, st);
        default: return launch_plain<SOT_BF16>(a, st);
    }
}

}  // namespace sot
