// k_lm.cu -- the plan of the row kernels (lm_row.cuh), the gradient of token
// log-probabilities from a known log-sum-exp, and the paired preference loss.
#include <cuda_runtime.h>

#include "kernels.h"
#include "lm_row.cuh"
#include "tc.h"

namespace sot {

namespace {

// Gradient of the token log-probabilities from a known log-sum-exp:
// dx_v = (g / tau) (1[v = target] - p_v).  No statistic is missing, so every
// granule stands alone: one read and one write per logit.
constexpr int GRAD_NT = 256;

template <int DT>
__global__ void __launch_bounds__(GRAD_NT) lm_grad_kernel(LmGradArgs a, int G, int chunks) {
    using T = typename Elem<DT>::T;
    constexpr int N = Elem<DT>::N;
    const long long row = blockIdx.x / chunks;
    const int part = (int)(blockIdx.x % chunks);
    const Slice s = slice_of<DT>(a.x, row, a.ld, a.V, G, part);
    T* const grow = static_cast<T*>(a.grad) + row * a.ldg;
    const bool aligned = (((unsigned long long)grow ^ (unsigned long long)(static_cast<const T*>(a.x) + row * a.ld)) & 15) == 0;
    const int tgt = load_index(a.target, a.target_type, row, a.V);
    const float g = tgt >= 0 ? a.g[row] / a.tau : 0.f;
    const float sc = SOT_LOG2E / a.tau;
    const float lse = a.lse[row];
    const float u = lse * a.tau;  // (x - u) / tau = log p
    for (int i = threadIdx.x; i < s.ng; i += GRAD_NT) {
        const int e = s.e0 + i * N;
        float2 f[N / 2];
        if (g != 0.f) {
            unpack<DT>(s.src[i], f);
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                const int c = e + 2 * j;
                f[j].x = g * ((c == tgt ? 1.f : 0.f) - ex2f((f[j].x - u) * sc));
                f[j].y = g * ((c + 1 == tgt ? 1.f : 0.f) - ex2f((f[j].y - u) * sc));
            }
        } else {
#pragma unroll
            for (int j = 0; j < N / 2; ++j) f[j] = make_float2(0.f, 0.f);
        }
        store_cols<DT>(grow, e, a.V, f, aligned);
    }
}

// Paired preference loss.  One CTA per pair: the two sequences' sums of
// (logp - ref) in 64 bits (they cancel in the margin), then the token
// gradients.  Offsets are clamped to [0, T], so wrong ones touch nothing else.
constexpr int PREF_NT = 256;

__global__ void __launch_bounds__(PREF_NT) lm_preference_kernel(LmPrefArgs a) {
    __shared__ double red[4][PREF_NT / 32];
    const int p = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long off[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const long long o = a.offsets[2 * (long long)p + i];
        off[i] = o < 0 ? 0 : (o > a.T ? a.T : o);
    }
    double v[4] = {0.0, 0.0, 0.0, 0.0};  // sums and counts of the chosen and the rejected
#pragma unroll
    for (int h = 0; h < 2; ++h)
        for (long long t = off[h] + tid; t < off[h + 1]; t += PREF_NT) {
            if (a.target && load_index(a.target, a.target_type, t, 0x7fffffff) < 0) continue;
            v[2 * h] += (double)a.logp[t] - (a.ref_logp ? (double)a.ref_logp[t] : 0.0);
            v[2 * h + 1] += 1.0;
        }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = warp_sum_d(v[i]);
        if (lane == 0) red[i][warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = 0.0;
        for (int k = 0; k < PREF_NT / 32; ++k) v[i] += red[i][k];
    }
    const double nc = a.average ? fmax(v[1], 1.0) : 1.0, nr = a.average ? fmax(v[3], 1.0) : 1.0;
    const float margin = (float)(v[0] / nc - v[2] / nr);
    const float z = a.beta * margin;
    const float e = expf(-fabsf(z)), l = log1pf(e);
    const float sp = (z >= 0.f ? 1.f : e) / (1.f + e), sn = (z >= 0.f ? e : 1.f) / (1.f + e);  // sigma(z), sigma(-z)
    const float lp = fmaxf(-z, 0.f) + l, ln = fmaxf(z, 0.f) + l;                              // -log of the two
    if (tid == 0) {
        const float loss = (1.f - a.smoothing) * lp + (a.smoothing != 0.f ? a.smoothing * ln : 0.f);
        if (a.loss) a.loss[p] = z != z ? z : loss;
        if (a.margin) a.margin[p] = margin;
    }
    if (!a.grad) return;
    const float d = a.scale * a.beta * (a.smoothing * sp - (1.f - a.smoothing) * sn);
    const float gc = (float)(d / nc), gr = (float)(-d / nr);
#pragma unroll
    for (int h = 0; h < 2; ++h)
        for (long long t = off[h] + tid; t < off[h + 1]; t += PREF_NT) {
            const bool out = a.target && load_index(a.target, a.target_type, t, 0x7fffffff) < 0;
            a.grad[t] = out ? 0.f : (h ? gr : gc);
        }
    // tokens before the first and after the last sequence belong to no pair
    if (p == 0)
        for (long long t = tid; t < off[0]; t += PREF_NT) a.grad[t] = 0.f;
    if (p == a.P - 1)
        for (long long t = off[2] + tid; t < a.T; t += PREF_NT) a.grad[t] = 0.f;
}

int row_granule(int dtype) { return dtype == SOT_F32 ? 4 : 8; }

// How a row is cut and who works on it.
void row_plan(bool grads, long long T, int dtype, int V, int K, bool tail, int sms, LmRowPlan* p) {
    const int N = row_granule(dtype);
    const long long total = ((long long)V + 2 * N - 2) / N;  // granules, whatever the row's alignment
    const auto plan = [&](int NW, int CL) {
        const long long G = (total + CL - 1) / CL;
        const size_t smem = NW == 1 ? ((size_t)G * 32 + (size_t)K * 12) * WARP_ROWS
                                    : (size_t)K * 12 + (tail ? ((size_t)G + 3) / 4 * 4 : 0);
        *p = LmRowPlan{NW, CL, (int)G, smem, sms};
    };
    const auto warps = [](long long G, int per) { return G <= per * 128ll ? 4 : G <= per * 256ll ? 8 : 16; };
    // Up to 8 KB a warp takes the row alone: 16384 rows of 4096 bf16 with gradient take
    // 57 us, with a CTA each 81 us; at 6144 a CTA is as fast (95 us both).
    if (total <= 528) {
        plan(1, 1);
    } else if (T < sms) {
        // Few rows: cut a row further, down to 512 granules a CTA, while the SMs have
        // room, and give it enough warps for eight granules a thread.
        int CL = 1;
        while (CL < ROW_MAX_CL && T * CL * 2 <= sms && total / (2 * CL) >= 512) CL *= 2;
        plan(warps((total + CL - 1) / CL, 8), CL);
    } else if (!grads) {
        // Read once: small CTAs, many on an SM (2048 rows of 131072 bf16: 80 us, with
        // 16 warps 86 us).
        plan(4, 1);
    } else {
        // Read twice: a thread takes up to 26 granules.  Smaller CTAs spend more on
        // starting (16384 rows of 16384 bf16: 4 warps 175 us, 8 warps 189 us); larger
        // shares keep more rows under way than L2 holds until their second pass (8192
        // rows of 65536, a third left out: 16 warps 284 us, 8 warps 320 us).
        int CL = 1;
        while (CL < ROW_MAX_CL && total > CL * 26ll * 512) CL *= 2;
        plan(warps((total + CL - 1) / CL, 26), CL);
    }
}

}  // namespace

bool lm_tail_fits(int dtype, int V, int K) {
    LmRowPlan p;
    row_plan(true, 1ll << 31, dtype, V, K, true, 1, &p);
    return p.smem <= 200 * 1024;
}

cudaError_t launch_lm_row(LmOp op, const LmRowArgs& a, int sms, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    LmRowPlan p;
    row_plan(op != LM_LOGPROB, a.T, a.dtype, a.V, a.K, a.tail != 0, sms, &p);
    if (a.T * p.CL > 0x7fffffffll) return cudaErrorInvalidValue;
    LmRowLaunch L = {};
    tc_test_hold(&L.hold, &L.wait_ns);
    cudaError_t e = async_status_address(&L.status);
    if (e != cudaSuccess) return e;
    count_launches(1);
    switch (a.dtype) {
        case SOT_F32: return launch_row_f32(op, a, p, L, st);
        case SOT_F16: return launch_row_f16(op, a, p, L, st);
        default: return launch_row_bf16(op, a, p, L, st);
    }
}

cudaError_t launch_lm_grad(const LmGradArgs& a, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    const int N = row_granule(a.dtype);
    const long long total = ((long long)a.V + 2 * N - 2) / N;
    // blocks of at least 2048 granules (32 KB), fewer blocks where the grid's limit asks for it
    long long G = 2048;
    while ((total + G - 1) / G * a.T > 0x7fffffffll) G *= 2;
    const int chunks = (int)((total + G - 1) / G);
    const dim3 grid((unsigned)(chunks * a.T));
    count_launches(1);
    switch (a.dtype) {
        case SOT_F32: lm_grad_kernel<SOT_F32><<<grid, GRAD_NT, 0, st>>>(a, (int)G, chunks); break;
        case SOT_F16: lm_grad_kernel<SOT_F16><<<grid, GRAD_NT, 0, st>>>(a, (int)G, chunks); break;
        default: lm_grad_kernel<SOT_BF16><<<grid, GRAD_NT, 0, st>>>(a, (int)G, chunks); break;
    }
    return cudaGetLastError();
}

cudaError_t launch_lm_preference(const LmPrefArgs& a, cudaStream_t st) {
    if (a.P == 0) return a.grad && a.T ? cudaMemsetAsync(a.grad, 0, sizeof(float) * a.T, st) : cudaSuccess;
    count_launches(1);
    lm_preference_kernel<<<a.P, PREF_NT, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace sot
