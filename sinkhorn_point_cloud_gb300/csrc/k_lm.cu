// k_lm.cu -- losses over rows of logits, with their gradients.
//
// A row x of V logits at temperature tau has p = softmax(x / tau).  Every loss
// here depends on the row through log p at a few columns, so its gradient is
//   dx_v = c p_v   at every column, corrected at those few columns,
// with c known once the row's log-sum-exp is.  One thread-block cluster takes a
// row: each CTA keeps a slice of it in shared memory, the slices' (max, sum)
// pairs are exchanged through distributed shared memory, and the gradient is
// written from the kept slice.  So a row is read from memory once and its
// gradient written once, which is the least any form can do; memory traffic
// bounds the kernel.
#include <cuda_runtime.h>

#include "kernels.h"
#include "lm.cuh"
#include "lm.h"

namespace sot {

namespace {

constexpr int ROW_NT = 512;
constexpr int ROW_MAX_CL = 8;
constexpr int NREC = 6;  // a CTA's record: (m, s), the entries' (m, s), a 64-bit sum

// What the row's threads need once its statistics are known.
struct RowCoef {
    float u, c;        // dx_v = c exp2((x_v - u) sc)
    float M, inv_S;    // p_v = exp2((x_v - M) sc) inv_S
    float fa, fb;      // a corrected column: fa p_v - fb q_v
};

__device__ __forceinline__ void put_double(const float* rec, uint32_t rank, double v) {
    const long long b = __double_as_longlong(v);
    cluster_store(rec, rank, __int_as_float((int)(b & 0xffffffffll)));
    cluster_store(rec + 1, rank, __int_as_float((int)(b >> 32)));
}
__device__ __forceinline__ double get_double(const float* rec) {
    return __longlong_as_double((long long)(unsigned)__float_as_int(rec[0]) |
                                ((long long)__float_as_int(rec[1]) << 32));
}

// The slice of row `row` that CTA `rank` of its cluster takes, in 16-byte
// granules of memory.  A row that starts or ends inside a granule is read with
// the whole granule: memory is allocated in larger aligned pieces, so the
// other bytes are readable; they are masked.
struct Slice {
    const uint4* src;
    long long e0;  // column of the first element of the slice (may be negative)
    int ng;        // granules
};
template <int DT>
__device__ __forceinline__ Slice slice_of(const void* x, long long row, long long ld, int V, int G, uint32_t rank) {
    using T = typename Elem<DT>::T;
    constexpr int N = Elem<DT>::N;
    const unsigned long long A = (unsigned long long)(static_cast<const T*>(x) + row * ld);
    const int head = (int)(A & 15) / (int)sizeof(T);
    const long long total = ((long long)head + V + N - 1) / N;
    long long first = (long long)rank * G, last = first + G;
    if (last > total) last = total;
    Slice s;
    s.src = reinterpret_cast<const uint4*>(A & ~15ull) + first;
    s.e0 = first * N - head;
    s.ng = last > first ? (int)(last - first) : 0;
    return s;
}

// Writes N elements at columns e .. e + N - 1 of a row.
template <int DT>
__device__ __forceinline__ void store_cols(typename Elem<DT>::T* row, long long e, int V,
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

template <int DT>
__device__ __forceinline__ void mask_cols(float2 (&f)[Elem<DT>::N / 2], long long e, int V, float fill) {
#pragma unroll
    for (int i = 0; i < Elem<DT>::N / 2; ++i) {
        if (e + 2 * i < 0 || e + 2 * i >= V) f[i].x = fill;
        if (e + 2 * i + 1 < 0 || e + 2 * i + 1 >= V) f[i].y = fill;
    }
}

template <int DT, int OP>
__global__ void __launch_bounds__(ROW_NT) lm_row_kernel(LmRowArgs a, int CL, int G) {
    using T = typename Elem<DT>::T;
    constexpr int N = Elem<DT>::N;
    extern __shared__ uint4 sm[];
    T* const se = reinterpret_cast<T*>(sm);
    float* const ex = reinterpret_cast<float*>(sm + G);  // entries: logit, weight q, column
    float* const eq = ex + a.K;
    int* const eid = reinterpret_cast<int*>(eq + a.K);
    __shared__ MS red[ROW_NT / 32];
    __shared__ float rec[2][ROW_MAX_CL][NREC];
    __shared__ RowCoef coef;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();
    const float sc = SOT_LOG2E / a.tau;
    int par = 0;
    for (long long row = blockIdx.x / CL; row < a.T; row += gridDim.x / CL) {
        const float w = a.weight ? a.weight[row] : 1.f / (float)a.T;
        const int tgt = OP == LM_DISTILL ? 0 : load_index(a.target, a.target_type, row, a.V);
        const bool keep = tgt >= 0 && (OP == LM_LOGPROB || w != 0.f);
        const Slice s = slice_of<DT>(a.x, row, a.ld, a.V, G, rank);
        T* const grow = a.grad ? static_cast<T*>(a.grad) + row * a.ldg : nullptr;
        const bool aligned = (((unsigned long long)grow ^ (unsigned long long)(static_cast<const T*>(a.x) + row * a.ld)) & 15) == 0;
        if (!keep) {
            if (grow) {
                float2 z[N / 2];
#pragma unroll
                for (int i = 0; i < N / 2; ++i) z[i] = make_float2(0.f, 0.f);
                for (int i = tid; i < s.ng; i += ROW_NT) store_cols<DT>(grow, s.e0 + (long long)i * N, a.V, z, aligned);
            }
            if (rank == 0 && tid == 0) {
                if (a.loss) a.loss[row] = 0.f;
                if (a.logp) a.logp[row] = 0.f;
                if (a.lse) a.lse[row] = 0.f;
                if (a.kl) a.kl[row] = 0.f;
            }
            continue;
        }
        for (int i = tid; i < s.ng; i += ROW_NT) sm[i] = s.src[i];
        __syncthreads();
        const long long e_end = s.e0 + (long long)s.ng * N;
        // Teacher side: q, its sums, and the entries' logits in this slice.
        double Q = 0.0, B = 0.0, D = 0.0;
        float qr = 0.f;
        MS top{-INFINITY, 0.f};
        if (OP == LM_DISTILL) {
            if (warp == 0) {
                float zmax = -INFINITY;
                for (int k = lane; k < a.K; k += 32) {
                    const int id = load_index(a.ids, a.ids_type, row * a.K + k, a.V);
                    const float z = load_float(a.teacher, a.teacher_type, row * a.K + k);
                    eid[k] = id;
                    eq[k] = id >= 0 ? z : -INFINITY;
                    if (id >= 0) zmax = fmaxf(zmax, z);
                }
                zmax = warp_max(zmax);
                const float z0 = a.tail ? 0.f : stab(zmax);
                for (int k = lane; k < a.K; k += 32) {
                    const float dz = (eq[k] - z0) / a.tau;
                    const float q = expf(dz);
                    eq[k] = q;
                    Q += q;
                    if (q != 0.f) B += (double)q * dz;
                }
                Q = warp_sum_d(Q);
                B = warp_sum_d(B);
                if (!a.tail && Q > 0.0) {  // normalise: q / Q, sum q log q
                    const float inv = (float)(1.0 / Q);
                    const double logZ = log(Q);
                    B = B / Q - logZ;
                    for (int k = lane; k < a.K; k += 32) eq[k] *= inv;
                    Q = 1.0;
                }
                for (int k = lane; k < a.K; k += 32) {
                    const int id = eid[k];
                    float v = -INFINITY;
                    if (id >= 0 && id >= s.e0 && id < e_end) {
                        v = Elem<DT>::get(se[id - s.e0]);
                        if (eq[k] != 0.f) D += (double)eq[k] * (double)v;
                        if (a.tail) {
                            se[id - s.e0] = Elem<DT>::put(-INFINITY);
                            MS one{v, v == -INFINITY ? 0.f : 1.f};
                            top = ms_combine(top, one, sc);
                        }
                    } else
                        eid[k] = -1;  // not this CTA's
                    ex[k] = v;
                }
                D = warp_sum_d(D);
                if (a.tail) top = ms_warp(top, sc);
            }
            __syncthreads();
        } else if (warp == 0 && tgt >= s.e0 && tgt < e_end)
            D = (double)Elem<DT>::get(se[tgt - s.e0]);
        // Row statistics of the slice.
        MS r{-INFINITY, 0.f};
        for (int i = tid; i < s.ng; i += ROW_NT) {
            float2 f[N / 2];
            unpack<DT>(sm[i], f);
            const long long e = s.e0 + (long long)i * N;
            if (e < 0 || e + N > a.V) mask_cols<DT>(f, e, a.V, -INFINITY);
            ms_add<DT>(r, f, sc);
        }
        r = ms_warp(r, sc);
        if (lane == 0) red[warp] = r;
        __syncthreads();
        if (warp == 0) {
            r = lane < ROW_NT / 32 ? red[lane] : MS{-INFINITY, 0.f};
            r = ms_warp(r, sc);
            if (lane < CL) {
                const float* p = rec[par][rank];
                cluster_store(p, lane, r.m);
                cluster_store(p + 1, lane, r.s);
                cluster_store(p + 2, lane, top.m);
                cluster_store(p + 3, lane, top.s);
                put_double(p + 4, lane, D);
            }
        }
        cluster_sync();
        if (warp == 0) {
            r = MS{-INFINITY, 0.f};
            top = r;
            D = 0.0;
            if (lane < CL) {
                const float* p = rec[par][lane];
                r = MS{p[0], p[1]};
                top = MS{p[2], p[3]};
                D = get_double(p + 4);
            }
            r = ms_warp(r, sc);
            top = ms_warp(top, sc);
            D = warp_sum_d(D);
            if (lane == 0) {
                const MS all = ms_combine(r, top, sc);
                const double logS = log_wide(all.s), it = 1.0 / (double)a.tau;
                RowCoef c;
                c.M = stab(all.m);
                c.inv_S = 1.f / all.s;
                c.u = c.M;
                if (OP == LM_DISTILL) {
                    const float wt = w * a.tau;
                    double loss = 0.0;
                    if (Q > 0.0) loss = B - (D - Q * (double)all.m) * it + Q * logS;
                    c.fa = wt * (float)Q;
                    c.fb = wt;
                    c.c = c.fa * c.inv_S;
                    if (a.tail) {
                        qr = (float)fmax(0.0, 1.0 - Q);
                        if (!(r.s > 0.f)) qr = r.s == 0.f ? 0.f : r.s;  // no column outside the entries: no tail outcome
                        if (qr > 0.f)
                            loss += (double)qr * (log_wide(qr) - (((double)r.m - (double)all.m) + log_wide(r.s) - logS));
                        c.fa = wt * (float)(Q + qr);
                        c.u = stab(r.m);
                        c.c = r.s == 0.f ? 0.f : wt * ((float)(Q + qr) * ex2f((r.m - c.M) * sc) * c.inv_S - qr / r.s);
                    }
                    if (rank == 0 && a.loss) a.loss[row] = (float)(loss * (double)w * (double)a.tau * (double)a.tau);
                } else {
                    const double logp = (D - (double)all.m) * it - logS;
                    float g = 0.f;
                    if (OP == LM_POLICY) {
                        const float A = a.adv[row];
                        const float ratio = expf((float)(logp - (double)a.old_logp[row]));
                        const float free = ratio * A, held = fminf(fmaxf(ratio, a.clip_lo), a.clip_hi) * A;
                        float loss = -fminf(free, held), kl = 0.f;
                        g = free <= held ? -free : 0.f;
                        if (free != free) loss = g = free;
                        if (a.ref_logp) {
                            const float d = (float)((double)a.ref_logp[row] - logp);
                            kl = exp_minus_linear(d);
                            loss += a.kl_coef * kl;
                            g -= a.kl_coef * expm1f(d);
                        }
                        g *= w;
                        if (rank == 0) {
                            if (a.loss) a.loss[row] = w * loss;
                            if (a.kl) a.kl[row] = kl;
                        }
                    }
                    c.fa = -g / a.tau;
                    c.fb = c.fa;
                    c.c = c.fa * c.inv_S;
                    if (rank == 0) {
                        if (a.logp) a.logp[row] = (float)logp;
                        if (a.lse) a.lse[row] = (float)((double)all.m * it + logS);
                    }
                }
                coef = c;
            }
        }
        par ^= 1;
        if (!grow) {
            __syncthreads();  // the slice and the sums are free for the next row
            continue;
        }
        __syncthreads();
        const RowCoef c = coef;
        for (int i = tid; i < s.ng; i += ROW_NT) {
            float2 f[N / 2];
            unpack<DT>(sm[i], f);
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                f[j].x = c.c * ex2f((f[j].x - c.u) * sc);
                f[j].y = c.c * ex2f((f[j].y - c.u) * sc);
            }
            store_cols<DT>(grow, s.e0 + (long long)i * N, a.V, f, aligned);
        }
        __syncthreads();  // the corrections come after the columns they replace
        if (OP == LM_DISTILL) {
            for (int k = tid; k < a.K; k += ROW_NT)
                if (eid[k] >= 0)
                    grow[eid[k]] = Elem<DT>::put(c.fa * (ex2f((ex[k] - c.M) * sc) * c.inv_S) - c.fb * eq[k]);
            __syncthreads();
        } else if (tid == 0 && tgt >= s.e0 && tgt < e_end)
            grow[tgt] = Elem<DT>::put(c.fa * (ex2f((Elem<DT>::get(se[tgt - s.e0]) - c.M) * sc) * c.inv_S) - c.fb);
        if (OP != LM_DISTILL) __syncthreads();
    }
    cluster_sync();  // no CTA leaves while a peer may still store to it
}

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
        const long long e = s.e0 + (long long)i * N;
        float2 f[N / 2];
        if (g != 0.f) {
            unpack<DT>(s.src[i], f);
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                const long long c = e + 2 * j;
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

struct RowPlan {
    int CL, G;
    size_t smem;
};
// The fewest CTAs a row can be cut into with a slice within shared memory.
bool row_plan(int dtype, int V, int K, RowPlan* p) {
    const int N = dtype == SOT_F32 ? 4 : 8;
    const long long total = ((long long)V + 2 * N - 2) / N;  // granules, whatever the row's alignment
    const size_t entries = (size_t)K * 12;
    for (int CL = 1; CL <= ROW_MAX_CL; CL *= 2) {
        const long long G = (total + CL - 1) / CL;
        const size_t smem = (size_t)G * 16 + entries;
        if (smem <= (CL == ROW_MAX_CL ? 200u : 64u) * 1024) {
            *p = RowPlan{CL, (int)G, smem};
            return true;
        }
    }
    return false;
}

template <int DT, int OP>
cudaError_t launch_row_t(const LmRowArgs& a, const RowPlan& p, cudaStream_t st) {
    auto kern = lm_row_kernel<DT, OP>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)p.smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.CL, 1, 1);
    cfg.blockDim = dim3(ROW_NT, 1, 1);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.CL;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    e = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg);
    if (e != cudaSuccess) return e;
    if (clusters < 1) return cudaErrorInvalidConfiguration;
    const long long n = a.T < clusters ? a.T : clusters;
    cfg.gridDim = dim3((unsigned)(n * p.CL), 1, 1);
    count_launches(1);
    e = cudaLaunchKernelEx(&cfg, kern, a, p.CL, p.G);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int DT>
cudaError_t launch_row_d(LmOp op, const LmRowArgs& a, const RowPlan& p, cudaStream_t st) {
    switch (op) {
        case LM_LOGPROB: return launch_row_t<DT, LM_LOGPROB>(a, p, st);
        case LM_POLICY: return launch_row_t<DT, LM_POLICY>(a, p, st);
        default: return launch_row_t<DT, LM_DISTILL>(a, p, st);
    }
}

}  // namespace

bool lm_row_fits(int dtype, int V, int K) {
    RowPlan p;
    return row_plan(dtype, V, K, &p);
}

cudaError_t launch_lm_row(LmOp op, const LmRowArgs& a, int, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    RowPlan p;
    if (!row_plan(a.dtype, a.V, a.K, &p)) return cudaErrorInvalidValue;
    switch (a.dtype) {
        case SOT_F32: return launch_row_d<SOT_F32>(op, a, p, st);
        case SOT_F16: return launch_row_d<SOT_F16>(op, a, p, st);
        default: return launch_row_d<SOT_BF16>(op, a, p, st);
    }
}

cudaError_t launch_lm_grad(const LmGradArgs& a, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    const int N = a.dtype == SOT_F32 ? 4 : 8;
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
