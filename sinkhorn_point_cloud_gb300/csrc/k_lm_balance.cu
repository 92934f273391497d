// k_lm_balance.cu -- the router's balance loss, its per-expert counts and its
// gradient.
//
// With N kept tokens, c_e the number of their choices of expert e and
// f_e = E c_e / (K N):
//   loss[0] = coef / N sum_t sum_e f_e p_te,   loss[1] = z_coef / N sum_t lse_t^2,
//   dx_te = 1/N ( coef p_te (f_e - sum_j f_j p_tj) + 2 z_coef lse_t p_te ).
// The counts come first (a small pass over the choices); then one warp takes a
// token, holds its E logits in registers and writes the gradient from them, so
// each logit is read once and each gradient written once.
#include <cuda_runtime.h>

#include "kernels.h"
#include "lm.cuh"
#include "lm.h"

namespace sot {

namespace {

constexpr int BAL_NT = 256;
constexpr int BAL_PARTS = 304;

__global__ void __launch_bounds__(BAL_NT) lm_count_kernel(LmBalanceArgs a) {
    __shared__ int hist[LM_MAX_E];
    __shared__ int kept;
    for (int e = threadIdx.x; e < a.E; e += BAL_NT) hist[e] = 0;
    if (threadIdx.x == 0) kept = 0;
    __syncthreads();
    int n = 0;
    for (long long t = (long long)blockIdx.x * BAL_NT + threadIdx.x; t < a.T; t += (long long)gridDim.x * BAL_NT) {
        if (a.mask && !a.mask[t]) continue;
        ++n;
        for (int k = 0; k < a.K; ++k) {
            const int id = load_index(a.ids, a.ids_type, t * a.K + k, a.E);
            if (id >= 0) atomicAdd(&hist[id], 1);
        }
    }
    if (n) atomicAdd(&kept, n);
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += BAL_NT)
        if (hist[e]) atomicAdd(&a.counts[e], hist[e]);
    if (threadIdx.x == 0 && kept) atomicAdd(a.kept, kept);
}

// One warp per token; lane l holds experts l, l + 32, ...
template <int DT, int R>
__global__ void __launch_bounds__(BAL_NT) lm_balance_kernel(LmBalanceArgs a) {
    using T = typename Elem<DT>::T;
    __shared__ float f[LM_MAX_E];
    __shared__ double red[2][BAL_NT / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int kept = *a.kept;
    const float inv_n = kept > 0 ? 1.f / (float)kept : 0.f;
    for (int e = threadIdx.x; e < a.E; e += BAL_NT)
        f[e] = (float)a.counts[e] * (float)((double)a.E / ((double)a.K * (double)(kept > 0 ? kept : 1)));
    __syncthreads();
    double sum_dot = 0.0, sum_z = 0.0;
    for (long long t = (long long)blockIdx.x * (BAL_NT / 32) + warp; t < a.T; t += (long long)gridDim.x * (BAL_NT / 32)) {
        T* const g = a.grad ? static_cast<T*>(a.grad) + t * a.ldg : nullptr;
        if (a.mask && !a.mask[t]) {
            if (g)
                for (int e = lane; e < a.E; e += 32) g[e] = Elem<DT>::put(0.f);
            continue;
        }
        const T* const x = static_cast<const T*>(a.x) + t * a.ld;
        float v[R], m = -INFINITY;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int e = lane + 32 * i;
            v[i] = e < a.E ? Elem<DT>::get(x[e]) : -INFINITY;
            m = fmaxf(m, v[i]);
        }
        m = warp_max(m);
        const float u = m == -INFINITY ? 0.f : m;
        float s = 0.f, d = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int e = lane + 32 * i;
            v[i] = ex2f((v[i] - u) * SOT_LOG2E);
            s += v[i];
            d = fmaf(v[i], e < a.E ? f[e] : 0.f, d);
        }
        s = warp_sum(s);
        d = warp_sum(d) / s;
        const float lse = m + logf(s);
        sum_dot += d;
        sum_z += (double)lse * lse;
        if (g) {
            const float base = 2.f * a.z_coef * lse - a.coef * d, k = inv_n / s;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int e = lane + 32 * i;
                if (e < a.E) g[e] = Elem<DT>::put(v[i] * k * fmaf(a.coef, f[e], base));
            }
        }
    }
    if (lane == 0) {
        red[0][warp] = sum_dot;
        red[1][warp] = sum_z;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        double v = 0.0;
        for (int w = 0; w < BAL_NT / 32; ++w) v += red[threadIdx.x][w];
        a.part[2 * blockIdx.x + threadIdx.x] = (float)v;
    }
}

__global__ void lm_balance_sum_kernel(LmBalanceArgs a, int parts) {
    const int i = threadIdx.x >> 5, lane = threadIdx.x & 31;
    double v = 0.0;
    for (int p = lane; p < parts; p += 32) v += (double)a.part[2 * p + i];
    v = warp_sum_d(v);
    const int kept = *a.kept;
    if (lane == 0) a.loss[i] = kept > 0 ? (float)(v * (double)(i ? a.z_coef : a.coef) / (double)kept) : 0.f;
}

template <int DT>
void launch_main(const LmBalanceArgs& a, int blocks, cudaStream_t st) {
    const int r = (a.E + 31) / 32;
    if (r <= 1) lm_balance_kernel<DT, 1><<<blocks, BAL_NT, 0, st>>>(a);
    else if (r <= 2) lm_balance_kernel<DT, 2><<<blocks, BAL_NT, 0, st>>>(a);
    else if (r <= 4) lm_balance_kernel<DT, 4><<<blocks, BAL_NT, 0, st>>>(a);
    else if (r <= 8) lm_balance_kernel<DT, 8><<<blocks, BAL_NT, 0, st>>>(a);
    else if (r <= 16) lm_balance_kernel<DT, 16><<<blocks, BAL_NT, 0, st>>>(a);
    else lm_balance_kernel<DT, 32><<<blocks, BAL_NT, 0, st>>>(a);
}

}  // namespace

int lm_balance_parts() { return BAL_PARTS; }

cudaError_t launch_lm_balance(const LmBalanceArgs& a, cudaStream_t st) {
    cudaError_t e = cudaMemsetAsync(a.counts, 0, sizeof(int) * a.E, st);
    if (e != cudaSuccess) return e;
    e = cudaMemsetAsync(a.kept, 0, sizeof(int), st);
    if (e != cudaSuccess) return e;
    const long long want = (a.T + BAL_NT / 32 - 1) / (BAL_NT / 32);
    const int blocks = (int)(want < 1 ? 1 : want < BAL_PARTS ? want : BAL_PARTS);
    const long long cw = (a.T + BAL_NT - 1) / BAL_NT;
    const int cblocks = (int)(cw < 1 ? 1 : cw < BAL_PARTS ? cw : BAL_PARTS);
    count_launches(3);
    lm_count_kernel<<<cblocks, BAL_NT, 0, st>>>(a);
    switch (a.dtype) {
        case SOT_F32: launch_main<SOT_F32>(a, blocks, st); break;
        case SOT_F16: launch_main<SOT_F16>(a, blocks, st); break;
        default: launch_main<SOT_BF16>(a, blocks, st); break;
    }
    lm_balance_sum_kernel<<<1, 64, 0, st>>>(a, blocks);
    return cudaGetLastError();
}

}  // namespace sot
