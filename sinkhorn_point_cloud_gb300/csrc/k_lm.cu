// k_lm.cu -- the plan of the row kernels (lm_row.cuh), the gradient of token
// log-probabilities from a known log-sum-exp, and the paired preference loss.
#include <cuda_runtime.h>

#include "kernels.h"
#include "lm_row.cuh"

namespace sot {

namespace {

// Gradient of the token log-probabilities from a known log-sum-exp:
// dx_v = (g / tau) (1[v = target] - p_v).  No statistic is missing, so every
// granule stands alone: one read and one write per logit, memory-bound.  A
// thread's loads go in batches of four, eight granules a thread; only the granule
// that holds the target looks at its columns (one at a time in all of them takes 6 us more).
// 10388 x 32768 bf16: 198 us, the copy bandwidth (1.02).  With the log-probabilities' pass before
// it and the paired loss between, three launches that each run over the whole batch and so
// read the logits twice, 308 us, 0.98 of the copy bandwidth for the 2.04 GB this moves.
constexpr int GRAD_NT = 256;

template <int DT>
__global__ void __launch_bounds__(GRAD_NT) lm_grad_kernel(const LmGradArgs a, int G, int chunks) {
    using T = typename Elem<DT>::T;
    constexpr int N = Elem<DT>::N, U = 4;
    const long long row = blockIdx.x / chunks;
    const T* const x = static_cast<const T*>(a.x) + row * a.ld;
    T* const grow = static_cast<T*>(a.grad) + row * a.ldg;
    const Slice s = slice_at<DT>(x, a.V, G, blockIdx.x % chunks);
    const bool aligned = same_granules<T>(x, grow);
    const int tgt = load_index(a.target, a.target_type, row, a.V);
    const float g = tgt >= 0 ? a.g[row] / a.tau : 0.f;
    const float sc = SOT_LOG2E / a.tau;
    const float lse = a.lse[row], u = lse * SOT_LOG2E;  // log2 p = x sc - u
    // Far from 0 the rounding of u would show: the difference comes first there.  What
    // lse itself has lost (2^-24 of it) can leave p too large, but not above 1.
    const bool far = !(fabsf(u) < 0x1p10f);
    const auto prob = [&](float x) {
        const float d = (x - lse * a.tau) / a.tau;
        return expf(d > 0.f ? 0.f : d);
    };
    const uint64_t policy = policy_drop();
    const auto finish = [&](float2 (&f)[N / 2], int c) {  // columns c ..
        const bool here = (unsigned)(tgt - c) < (unsigned)N;
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
            float2 p;
            if (!far) p = ex2_pair(f[j], u, sc);
            else p = make_float2(prob(f[j].x), prob(f[j].y));
            f[j] = p;
        }
        if (here) {
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                f[j].x -= c + 2 * j == tgt ? 1.f : 0.f;
                f[j].y -= c + 2 * j + 1 == tgt ? 1.f : 0.f;
            }
        }
#pragma unroll
        for (int j = 0; j < N / 2; ++j) f[j] = fmul2(f[j], make_float2(-g, -g));
    };
    if (g == 0.f) {  // not read
        slice_zero<DT>(s, grow, a.V, aligned, threadIdx.x, GRAD_NT);
        return;
    }
    if (!aligned) {
        for (int i = threadIdx.x; i < s.ng; i += GRAD_NT) {
            float2 f[N / 2];
            unpack<DT>(s.src[i], f);
            finish(f, s.e0 + i * N);
            store_cols<DT>(grow, s.e0 + i * N, a.V, f, false);
        }
        return;
    }
    uint4* const dst = reinterpret_cast<uint4*>(grow + s.e0);
    for (int i = s.lo + threadIdx.x; i < s.hi; i += U * GRAD_NT) {
        uint4 v[U];
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (i + j * GRAD_NT < s.hi) v[j] = load16(s.src + i + j * GRAD_NT, policy);
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (i + j * GRAD_NT < s.hi) {
                float2 f[N / 2];
                unpack<DT>(v[j], f);
                finish(f, s.e0 + (i + j * GRAD_NT) * N);
                store16(dst + i + j * GRAD_NT, pack<DT>(f), policy);
            }
    }
    const int e = edge_granule(s, threadIdx.x, GRAD_NT);
    if (e >= 0) {
        float2 f[N / 2];
        unpack<DT>(s.src[e], f);
        finish(f, s.e0 + e * N);
        store_cols<DT>(grow, s.e0 + e * N, a.V, f, false);
    }
}

// Paired preference loss.  One CTA per pair: the two sequences' sums of
// (logp - ref) to about 48 bits (they cancel in the margin), then the token
// gradients.  Offsets are clamped to [0, T], so wrong ones touch nothing else.
// A few KB a pair: the chain of loads, reductions and stores, about 4 us, is all it costs.
constexpr int PREF_NT = 256;

__global__ void __launch_bounds__(PREF_NT) lm_preference_kernel(const LmPrefArgs a) {
    constexpr int NW = PREF_NT / 32;
    __shared__ float2 red[2][NW];
    __shared__ int count[2][NW];
    const int p = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long off[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) off[i] = min(max(a.offsets[2 * (long long)p + i], 0ll), a.T);
    float2 v[2];
    int n[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        v[h] = make_float2(0.f, 0.f);
        n[h] = 0;
        for (long long t = off[h] + tid; t < off[h + 1]; t += PREF_NT) {
            if (a.target && load_index(a.target, a.target_type, t, 0x7fffffff) < 0) continue;
            v[h] = ff_add_or_far(v[h], two_sum(a.logp[t], a.ref_logp ? -a.ref_logp[t] : 0.f));
            ++n[h];
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        v[h] = ff_sum_or_far(v[h]);
        n[h] = __reduce_add_sync(0xffffffffu, n[h]);
        if (lane == 0) {
            red[h][warp] = v[h];
            count[h][warp] = n[h];
        }
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        v[h] = ff_sum_or_far(lane < NW ? red[h][lane] : make_float2(0.f, 0.f));
        n[h] = __reduce_add_sync(0xffffffffu, lane < NW ? count[h][lane] : 0);
    }
    const float nc = a.average ? (float)max(n[0], 1) : 1.f, nr = a.average ? (float)max(n[1], 1) : 1.f;
    float margin;
    if (a.average) {
        margin = (float)(to_double(v[0]) / nc - to_double(v[1]) / nr);
    } else {
        const float2 d = ff_add(v[0], make_float2(-v[1].x, -v[1].y));
        const float f = v[0].x - v[1].x;
        margin = fabsf(f) < INFINITY ? d.x + d.y : f;
    }
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
    const float gc = d / nc, gr = -d / nr;
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
void row_plan(bool grads, bool whole, long long T, int dtype, int V, int K, bool tail, int sms, LmRowPlan* p) {
    const int N = row_granule(dtype);
    // granules of a row: `whole` where every row starts with one, otherwise whatever its alignment
    const long long total = ((long long)V + (whole ? N - 1 : 2 * N - 2)) / N;
    const auto plan = [&](int NW, int CL) {
        const long long G = (total + CL - 1) / CL;
        const size_t smem = NW == 0 ? (size_t)K * 12 * SHORT_NW
                                    : (size_t)K * 12 + (tail ? cut_bytes((int)G) + cut_batches((int)G, NW * 32) : 0);
        *p = LmRowPlan{NW, CL, (int)G, smem};
    };
    const auto warps = [](long long G, int per) { return G <= per * 128ll ? 4 : G <= per * 256ll ? 8 : 16; };
    // Up to 8 KB a warp takes the row alone: 16384 rows of 4096 bf16 with gradient take 58
    // us, with a CTA each 81 us.
    if (total <= 512 && K <= SHORT_MAX_K) {
        plan(0, 1);
    } else if (T < sms) {
        // Few rows: cut a row further, down to 512 granules a CTA, up to two CTAs an SM,
        // and give it enough warps for eight granules a thread.
        int CL = 1;
        while (CL < ROW_MAX_CL && T * CL <= sms && total / (2 * CL) >= 512) CL *= 2;
        while (CL < ROW_MAX_CL && tail && total > CL * 65536ll) CL *= 2;  // the tail's marks, a byte a granule
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
    row_plan(true, false, 1ll << 31, dtype, V, K, true, 1, &p);
    return p.smem <= MAX_SMEM;
}

cudaError_t launch_lm_row(LmOp op, const LmRowArgs& a, int sms, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    LmRowPlan p;
    const bool whole = (unsigned long long)a.x % 16 == 0 && a.ld % row_granule(a.dtype) == 0;
    // (Losses alone are cut as they are with their gradient: the same sums, so the same bits.)
    row_plan(op != LM_LOGPROB, whole, a.T, a.dtype, a.V, a.K, a.tail != 0, sms, &p);
    if (a.T * p.CL > 0x7fffffffll) return cudaErrorInvalidValue;
    const LmRowLaunch L = {p.CL, p.G};
    count_launches(1);
    switch (a.dtype) {
        case SOT_F32: return launch_row_f32(op, a, p, L, st);
        case SOT_F16: return launch_row_f16(op, a, p, L, st);
        default: return launch_row_bf16(op, a, p, L, st);
    }
}

cudaError_t launch_lm_grad(const LmGradArgs& a, int sms, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    const int N = row_granule(a.dtype);
    const long long total = ((long long)a.V + 2 * N - 2) / N;
    // Eight granules a thread, or four where that leaves SMs without work; more where
    // the grid's limit asks for it.
    long long G = (total + 2047) / 2048 * a.T < 2ll * sms ? 1024 : 2048;
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
