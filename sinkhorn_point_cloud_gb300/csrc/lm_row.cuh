// lm_row.cuh -- losses over rows of logits, with their gradients.
//
// A row x of V logits at temperature tau has p = softmax(x / tau).  Every loss
// here depends on the row through log p at a few columns, so its gradient is
//   dx_v = c p_v   at every column, corrected at those few columns,
// with c known once the row's log-sum-exp is.  The row stays in shared memory
// between the two, so it is read from memory once and its gradient written
// once, the least any form can do; memory traffic is what bounds the kernel.
//
// One thread-block cluster takes a row, each CTA a slice of it, and the grid
// stays resident and walks the rows through a ring of stages.  A stage has a
// warp of its own for everything about its row but the row itself: it starts
// the row's bulk copy, prepares the teacher's side while the copy is under way,
// joins the slice's statistics, exchanges them with the other CTAs through
// distributed shared memory, forms the loss and the gradient's coefficients,
// corrects the few columns at the end and starts the next copy.  The consumer
// warps only stream: statistics of row i, then the gradient of row i - lag, so
// the stage warps' latencies pass while the consumers have other rows to work on.
// Every wait is bounded; one that runs out ends the CTA's loops, leaves NaN
// losses and reports through sot_async_status.
#pragma once
#include <cuda_runtime.h>

#include "lm.cuh"
#include "lm.h"

namespace sot {

constexpr int ROW_MAX_CL = 8;
constexpr int ROW_MAX_ST = 4;
constexpr int NREC = 6;  // a CTA's record: (m, s), the entries' (m, s), a 64-bit sum

struct LmRowLaunch {
    int CL, G, ST, lag;          // CTAs a row, granules a slice, stages, rows between statistics and gradient
    int hold;                    // testing hook: no copy from this row of a cluster on (-1: off)
    unsigned long long wait_ns;  // limit of every wait
    unsigned* status;            // the device's status word of asynchronous calls
};

// What the row's threads need once its statistics are known.
struct RowCoef {
    float u, c;      // dx_v = c exp2(x_v sc - u)
    float far;       // not 0: u overflows, and dx_v = c where x_v = m, 0 elsewhere
    float m;
    float M, inv_S;  // p_v = weight of x_v against M times inv_S
    float fa, fb;    // a corrected column: fa p_v - fb q_v
    __device__ __forceinline__ void set(float v, float sc) {
        const float v2 = __fmul_rn(v, sc);
        m = v;
        far = fabsf(v2) < INFINITY ? 0.f : 1.f;
        u = far != 0.f ? 0.f : v2;
    }
};

// The slice of row `row` that CTA `rank` of its cluster takes, in 16-byte
// granules of memory.  A row that starts or ends inside a granule is read with
// the whole granule: memory is allocated in larger aligned pieces, so the
// other bytes are readable; they are masked.
struct Slice {
    const uint4* src;
    int e0;      // column of the first element of the slice (may be negative)
    int ng;      // granules
    int lo, hi;  // those that lie within the row: [lo, hi)
};
template <int DT>
__device__ __forceinline__ Slice slice_at(const typename Elem<DT>::T* row, int V, int G, uint32_t rank) {
    constexpr int N = Elem<DT>::N;
    const unsigned long long A = (unsigned long long)row;
    const int head = (int)((uint32_t)A & 15u) / (int)sizeof(*row);
    const int total = (int)(((unsigned)head + (unsigned)V + N - 1) / N), first = (int)rank * G;
    Slice s;
    s.src = reinterpret_cast<const uint4*>(A & ~15ull) + first;
    s.e0 = first * N - head;
    s.ng = max(0, min(total - first, G));
    s.lo = s.e0 < 0 ? 1 : 0;
    s.hi = s.ng - (s.e0 + s.ng * N > V ? 1 : 0);
    return s;
}
template <int DT>
__device__ __forceinline__ Slice slice_of(const void* x, long long row, long long ld, int V, int G, uint32_t rank) {
    return slice_at<DT>(static_cast<const typename Elem<DT>::T*>(x) + row * ld, V, G, rank);
}

// Writes N elements at columns e .. e + N - 1 of a row.
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

template <int DT>
__device__ __forceinline__ void mask_cols(float2 (&f)[Elem<DT>::N / 2], int e, int V, float fill) {
#pragma unroll
    for (int i = 0; i < Elem<DT>::N / 2; ++i) {
        if (e + 2 * i < 0 || e + 2 * i >= V) f[i].x = fill;
        if (e + 2 * i + 1 < 0 || e + 2 * i + 1 >= V) f[i].y = fill;
    }
}

// Barriers of a stage: its copy has landed; (tail) the entries are taken out of
// the slice; the slice's statistics, the coefficients, the gradient are done;
// the other CTAs' records have arrived (two, used in turn).
enum { RB_FULL = 0, RB_CUT, RB_REC, RB_COEF, RB_GRAD, RB_MAIL, RB_COUNT = RB_MAIL + 2 };

template <int NW>
struct RowShared {
    uint64_t bar[ROW_MAX_ST][RB_COUNT];
    MS rec[ROW_MAX_ST][NW];
    RowCoef coef[ROW_MAX_ST];
    float mail[ROW_MAX_ST][2][ROW_MAX_CL][NREC];
    int keep[ROW_MAX_ST];
    int abort;
};

// The teacher's entries of a row (one warp): weights q in eq, columns in eid
// (-1: unused), and the sums Q = sum q and B = sum q log q.
__device__ __forceinline__ void teacher_side(const LmRowArgs& a, long long row, float* eq, int* eid, float2& Q, float2& B) {
    const int lane = threadIdx.x & 31;
    float zmax = -INFINITY;
    for (int k0 = 0; k0 < a.K; k0 += 128) {  // four loads in flight a lane
        int id[4];
        float z[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = k0 + 32 * j + lane;
            id[j] = k < a.K ? load_index(a.ids, a.ids_type, row * a.K + k, a.V) : -1;
            z[j] = k < a.K ? load_float(a.teacher, a.teacher_type, row * a.K + k) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = k0 + 32 * j + lane;
            if (id[j] < 0) z[j] = -INFINITY;
            zmax = fmaxf(zmax, z[j]);
            if (k < a.K) {
                eid[k] = id[j];
                eq[k] = z[j];
            }
        }
    }
    zmax = warp_max1(zmax);
    const float z0 = a.tail || zmax == -INFINITY ? 0.f : zmax, inv_tau = (float)a.inv_tau;
    Q = B = make_float2(0.f, 0.f);
    for (int k = lane; k < a.K; k += 32) {
        const float dz = (eq[k] - z0) * inv_tau, q = expf(dz);
        eq[k] = q;
        Q = ff_add(Q, make_float2(q, 0.f));
        if (q != 0.f) B = ff_add(B, two_prod(q, dz));
    }
    Q = ff_warp_sum(Q);
    B = ff_warp_sum(B);
    if (!a.tail && Q.x > 0.f) {  // q / Q and sum q log q
        const float inv = __frcp_rn(Q.x);
        const float low = -fmaf(Q.x, inv, fmaf(Q.y, inv, -1.f)) * inv;  // 1 / Q = inv + low
        float2 logZ = log_ff(Q.x);
        logZ.y = fmaf(Q.y, inv, logZ.y);
        B = ff_add(ff_mul(B, make_float2(inv, low)), make_float2(-logZ.x, -logZ.y));
        Q = make_float2(1.f, 0.f);
        for (int k = lane; k < a.K; k += 32) eq[k] *= inv;
    }
}

// Sum over a warp; a sum that is not finite goes without its low parts.
__device__ __forceinline__ float2 ff_sum_or_far(float2 v) {
    const float2 s = ff_warp_sum(v);
    const float f = warp_sum(v.x);
    return fabsf(f) < INFINITY ? s : make_float2(f, 0.f);
}

// The entries' logits in this slice: ex, D = sum q x, and for the tail their
// statistics, with the entries themselves taken out of the slice.
template <int DT>
__device__ __forceinline__ void student_side(const LmRowArgs& a, const Slice& s, typename Elem<DT>::T* se, float* ex,
                                             const float* eq, int* eid, float sc, float2& D, MS& top) {
    const int lane = threadIdx.x & 31;
    const int e_end = s.e0 + s.ng * Elem<DT>::N;
    D = make_float2(0.f, 0.f);
    top = MS{-INFINITY, 0.f};
    for (int k = lane; k < a.K; k += 32) {
        const int id = eid[k];
        float v = -INFINITY;
        if (id >= 0 && id >= s.e0 && id < e_end) {
            v = Elem<DT>::get(se[id - s.e0]);
            if (eq[k] != 0.f) D = fabsf(v) < INFINITY ? ff_add(D, two_prod(eq[k], v)) : make_float2(D.x + v, 0.f);
            if (a.tail) {
                se[id - s.e0] = Elem<DT>::put(-INFINITY);
                top.m = fmaxf(top.m, v);
            }
        } else
            eid[k] = -1;  // not this CTA's
        ex[k] = v;
    }
    D = ff_sum_or_far(D);
    if (a.tail) {
        top.m = warp_max1(top.m);
        for (int k = lane; k < a.K; k += 32) top.s += weight_of(ex[k], top.m, sc);
        top.s = top.m == -INFINITY ? 0.f : warp_sum(top.s);
        fence_proxy_async_smem();  // the removals come before the stage's next copy
        __syncwarp();
    }
}

// What a row's stage warp knows of the row before its copy starts.
struct RowMeta {
    int tgt;
    float w, old, ref, adv;
    bool keep;
};
template <int OP>
__device__ __forceinline__ RowMeta row_meta(const LmRowArgs& a, long long row) {
    RowMeta m;
    m.tgt = OP == LM_DISTILL ? 0 : load_index(a.target, a.target_type, row, a.V);
    m.w = OP == LM_LOGPROB ? 1.f : a.weight ? a.weight[row] : 1.f / (float)a.T;
    m.old = m.ref = m.adv = 0.f;
    if (OP == LM_POLICY) {
        m.old = a.old_logp[row];
        m.adv = a.adv[row];
        if (a.ref_logp) m.ref = a.ref_logp[row];
    }
    m.keep = m.tgt >= 0 && m.w != 0.f;
    return m;
}

// The row's loss and the gradient's coefficients from its joined statistics
// (one lane): r without and top with the entries of a tail, D = sum q x or the
// target's logit.  `publish` hands the coefficients on before the losses, which
// nothing waits for, are finished.
template <int OP, class Publish>
__device__ __forceinline__ RowCoef row_finish(const LmRowArgs& a, long long row, const RowMeta& m, MS r, MS top, float2 Q,
                                              float2 B, float2 D, float sc, bool write, Publish publish) {
    const MS all = OP == LM_DISTILL && a.tail ? ms_combine(r, top, sc) : r;
    // log(sum exp(x / tau)) = m2 ln 2 + log s with the rounded m2 that the sums
    // were formed with; where m2 overflows, m / tau + log s
    const float m2 = __fmul_rn(all.m, sc);
    const bool far = !(fabsf(m2) < INFINITY);
    const float2 ln2 = make_float2(0.693147182f, -1.904654212e-9f);
    RowCoef c;
    c.M = all.m;
    c.inv_S = __frcp_rn(all.s);
    c.set(all.m, sc);
    if (OP == LM_DISTILL) {
        const float wt = m.w * a.tau;
        float qr = 0.f;
        c.fa = wt * Q.x;
        c.fb = wt;
        c.c = c.fa * c.inv_S;
        if (a.tail) {
            // no column outside the entries: no tail outcome
            qr = r.s == 0.f ? 0.f : r.s > 0.f ? fmaxf(0.f, (1.f - Q.x) - Q.y) : r.s;
            c.fa = wt * (Q.x + qr);
            c.set(r.m, sc);
            c.c = r.s == 0.f ? 0.f : wt * ((Q.x + qr) * rescale(r.m, c.M, sc) * c.inv_S - qr / r.s);
        }
        publish(c);
        if (write && a.loss) {
            const double logS = to_double(log_ff(all.s)), q = to_double(Q), k = 0.69314718055994530942;
            double loss = 0.0;
            if (q > 0.0)
                loss = to_double(B) + q * logS -
                       (far ? (to_double(D) - q * (double)all.m) * a.inv_tau : (to_double(D) * (double)sc - q * (double)m2) * k);
            if (a.tail && !(qr <= 0.f)) {
                const double apart = far ? ((double)r.m - (double)all.m) * a.inv_tau
                                         : ((double)__fmul_rn(r.m, sc) - (double)m2) * k;
                loss += (double)qr * (to_double(log_ff(qr)) - (apart + to_double(log_ff(r.s)) - logS));
            }
            a.loss[row] = (float)(loss * (double)m.w * (double)a.tau * (double)a.tau);
        }
        return c;
    }
    // logp = (x sc - m2) ln 2 - log s, kept to more than 24 bits until it is compared
    const float2 logS = log_ff(all.s), minus = make_float2(-logS.x, -logS.y);
    const float2 t = two_prod(D.x, sc), ts = two_sum(t.x, -m2);
    float2 logp = ff_add(ff_mul(ff_renorm(ts.x, ts.y + t.y), ln2), minus);
    if (!(fabsf(logp.x) < INFINITY)) logp = make_float2((float)(((double)D.x - (double)all.m) * a.inv_tau) - logS.x, 0.f);
    float g = 0.f, loss = 0.f, kl = 0.f;
    if (OP == LM_POLICY) {
        const float2 d0 = two_sum(logp.x, -m.old);
        const float ratio = expf(fabsf(d0.x) < INFINITY ? d0.x + (d0.y + logp.y) : d0.x);
        const float free = ratio * m.adv, held = fminf(fmaxf(ratio, a.clip_lo), a.clip_hi) * m.adv;
        loss = -fminf(free, held);
        g = free <= held ? -free : 0.f;
        if (free != free) loss = g = free;
        if (a.ref_logp) {
            const float2 d1 = two_sum(m.ref, -logp.x);
            const float d = fabsf(d1.x) < INFINITY ? d1.x + (d1.y - logp.y) : d1.x;
            kl = exp_minus_linear(d);
            loss += a.kl_coef * kl;
            g -= a.kl_coef * (kl + d);
        }
        g *= m.w;
    }
    c.fa = c.fb = -g * (float)a.inv_tau;
    c.c = c.fa * c.inv_S;
    publish(c);
    if (write) {
        if (a.loss) a.loss[row] = m.w * loss;
        if (a.kl) a.kl[row] = kl;
        if (a.logp) a.logp[row] = logp.x + logp.y;
        if (a.lse) {
            const float2 l = ff_add(ff_mul(make_float2(m2, 0.f), ln2), logS);
            a.lse[row] = far ? (float)((double)all.m * a.inv_tau) + logS.x : l.x + l.y;
        }
    }
    return c;
}

__device__ __forceinline__ void row_outputs(const LmRowArgs& a, long long row, float v) {
    if (a.loss) a.loss[row] = v;
    if (a.logp) a.logp[row] = v;
    if (a.lse) a.lse[row] = v;
    if (a.kl) a.kl[row] = v;
}

// ---- what the consumers do with a slice (threads tid = 0 .. NT - 1).  Granules inside
// the row go in batches of four a thread, so that their loads are under way
// together and one comparison serves 4 N logits; the granule the row starts in
// and the one it ends in belong to two lanes of the first warp.
__device__ __forceinline__ int edge_granule(const Slice& s, int tid) {
    if (tid == 0 && s.ng > 0 && s.lo > 0) return 0;
    if (tid == 1 && s.ng > 0 && s.hi < s.ng && (s.ng > 1 || s.lo == 0)) return s.ng - 1;
    return -1;
}
template <int DT, int NT>
__device__ __forceinline__ MS slice_stats(const Slice& s, const uint4* src, int V, float sc, int tid) {
    constexpr int N = Elem<DT>::N;
    Running r;
    int g = s.lo + tid;
    for (; g + 3 * NT < s.hi; g += 4 * NT) {
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = src[g + j * NT];
        r.raise(max_of<DT>(max2<DT>(max2<DT>(v[0], v[1]), max2<DT>(v[2], v[3]))), sc);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float2 f[N / 2];
            unpack<DT>(v[j], f);
            r.add(f, sc);
        }
    }
    for (; g < s.hi; g += NT) {
        const uint4 v = src[g];
        float2 f[N / 2];
        unpack<DT>(v, f);
        r.raise(max_of<DT>(v), sc);
        r.add(f, sc);
    }
    const int e = edge_granule(s, tid);
    if (e >= 0) {
        float2 f[N / 2];
        unpack<DT>(src[e], f);
        mask_cols<DT>(f, s.e0 + e * N, V, -INFINITY);
        r.raise(max_of<DT>(f), sc);
        r.add(f, sc);
    }
    return MS{r.m, r.s.x + r.s.y};
}

template <int DT>
__device__ __forceinline__ void grad_of(float2 (&f)[Elem<DT>::N / 2], const RowCoef& c, float sc) {
    if (c.far == 0.f) {
#pragma unroll
        for (int k = 0; k < Elem<DT>::N / 2; ++k) f[k] = fmul2(ex2_pair(f[k], c.u, sc), make_float2(c.c, c.c));
    } else {
#pragma unroll
        for (int k = 0; k < Elem<DT>::N / 2; ++k) {
            f[k].x = c.c * (f[k].x - c.m == 0.f ? 1.f : 0.f);
            f[k].y = c.c * (f[k].y - c.m == 0.f ? 1.f : 0.f);
        }
    }
}

template <int DT, int NT>
__device__ __forceinline__ void slice_grad(const Slice& s, const uint4* src, const RowCoef& coef,
                                           typename Elem<DT>::T* grow, int V, float sc, bool aligned, int tid) {
    constexpr int N = Elem<DT>::N;
    const RowCoef c = coef;
    if (aligned) {
        uint4* const dst = reinterpret_cast<uint4*>(grow + s.e0);
        int g = s.lo + tid;
        for (; g + 3 * NT < s.hi; g += 4 * NT) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = src[g + j * NT];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float2 f[N / 2];
                unpack<DT>(v[j], f);
                grad_of<DT>(f, c, sc);
                dst[g + j * NT] = pack<DT>(f);
            }
        }
        for (; g < s.hi; g += NT) {
            float2 f[N / 2];
            unpack<DT>(src[g], f);
            grad_of<DT>(f, c, sc);
            dst[g] = pack<DT>(f);
        }
        const int e = edge_granule(s, tid);
        if (e >= 0) {
            float2 f[N / 2];
            unpack<DT>(src[e], f);
            grad_of<DT>(f, c, sc);
            store_cols<DT>(grow, s.e0 + e * N, V, f, false);
        }
    } else {
        for (int g = tid; g < s.ng; g += NT) {
            float2 f[N / 2];
            unpack<DT>(src[g], f);
            grad_of<DT>(f, c, sc);
            store_cols<DT>(grow, s.e0 + g * N, V, f, false);
        }
    }
}

template <int DT, int NT>
__device__ __forceinline__ void slice_zero(const Slice& s, typename Elem<DT>::T* grow, int V, bool aligned, int tid) {
    constexpr int N = Elem<DT>::N;
    float2 z[N / 2];
#pragma unroll
    for (int k = 0; k < N / 2; ++k) z[k] = make_float2(0.f, 0.f);
    for (int g = tid; g < s.ng; g += NT) store_cols<DT>(grow, s.e0 + g * N, V, z, aligned);
}

template <int DT, int OP, int NW>
__global__ void __launch_bounds__((NW + ROW_MAX_ST) * 32, NW == 4 ? 5 : NW == 8 ? 3 : 2)
    lm_row_kernel(const LmRowArgs a, const LmRowLaunch L) {
    using T = typename Elem<DT>::T;
    constexpr int N = Elem<DT>::N, NT = NW * 32;
    extern __shared__ __align__(128) uint4 sm[];
    __shared__ RowShared<NW> S;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();
    const float sc = SOT_LOG2E / a.tau;
    const int ST = L.ST, lag = L.lag;
    const long long first = blockIdx.x / L.CL, step = gridDim.x / L.CL;
    const long long n = (a.T - first + step - 1) / step;  // rows of this cluster
    volatile int* const abort = &S.abort;
    auto bar = [&](int st, int k) { return smem_u32(&S.bar[st][k]); };

    if (tid == 0) {
        for (int st = 0; st < ST; ++st) {
            mbar_init(bar(st, RB_FULL), 1);
            mbar_init(bar(st, RB_CUT), 1);
            mbar_init(bar(st, RB_REC), NW);
            mbar_init(bar(st, RB_COEF), 1);
            mbar_init(bar(st, RB_GRAD), NW);
            mbar_init(bar(st, RB_MAIL), L.CL);
            mbar_init(bar(st, RB_MAIL + 1), L.CL);
        }
        S.abort = 0;
        fence_mbar_init();
    }
    if (L.CL > 1) cluster_sync();  // the barriers exist before a peer arrives on them
    else __syncthreads();

    if (warp < NW) {
        // ---- consumers: statistics of row i, gradient of row i - lag
        const uint32_t ready = OP == LM_DISTILL && a.tail ? RB_CUT : RB_FULL;
        const long long end = n + (a.grad ? lag : 0);
        const T *x = static_cast<const T*>(a.x) + first * a.ld, *gx = x;  // rows i and i - lag
        T* grow = static_cast<T*>(a.grad) + (a.grad ? first * a.ldg : 0);
        const long long x_step = step * a.ld, g_step = step * a.ldg;
        int st = 0, gst = 0;         // their stages
        uint32_t ph = 0u, gph = 0u;  // and these stages' phases
        for (long long i = 0; i < end; ++i) {
            if (i < n) {
                if (!mbar_wait_bounded(bar(st, ready), ph, abort, L.wait_ns)) break;
                if (S.keep[st]) {
                    const MS r = ms_warp(slice_stats<DT, NT>(slice_at<DT>(x, a.V, L.G, rank), sm + (size_t)st * L.G, a.V, sc, tid), sc);
                    if (lane == 0) S.rec[st][warp] = r;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(st, RB_REC));
                x += x_step;
                if (++st == ST) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            if (a.grad && i >= lag) {
                const Slice s = slice_at<DT>(gx, a.V, L.G, rank);
                const bool aligned = ((uint32_t)((unsigned long long)grow ^ (unsigned long long)gx) & 15u) == 0;
                if (!mbar_wait_bounded(bar(gst, RB_COEF), gph, abort, L.wait_ns)) break;
                if (S.keep[gst])
                    slice_grad<DT, NT>(s, sm + (size_t)gst * L.G, S.coef[gst], grow, a.V, sc, aligned, tid);
                else
                    slice_zero<DT, NT>(s, grow, a.V, aligned, tid);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(gst, RB_GRAD));
                gx += x_step;
                grow += g_step;
                if (++gst == ST) {
                    gst = 0;
                    gph ^= 1u;
                }
            }
        }
    } else {
        // ---- stage warps: stage st has rows st, st + ST, ...
        const int st = warp - NW;
        T* const se = reinterpret_cast<T*>(sm + (size_t)st * L.G);
        float* const ex = reinterpret_cast<float*>(sm + (size_t)ST * L.G) + (size_t)st * 3 * a.K;
        float* const eq = ex + a.K;
        int* const eid = reinterpret_cast<int*>(eq + a.K);
        uint32_t ph = 0u, kept = 0u;  // phase of the stage's barriers; kept rows (phase of the mail)
        bool fine = true, copying = false;
        uint32_t cph = 1u;  // phase of the copy under way
        auto start = [&](long long i, const RowMeta& m) {  // row i's copy
            const Slice s = slice_of<DT>(a.x, first + i * step, a.ld, a.V, L.G, rank);
            copying = false;
            if (i == L.hold) return;
            copying = true;
            cph ^= 1u;
            if (lane == 0) {
                S.keep[st] = m.keep;
                if (m.keep && s.ng > 0) {
                    mbar_arrive_expect_tx(bar(st, RB_FULL), (uint32_t)s.ng * 16);
                    bulk_g2s(smem_u32(se), s.src, (uint32_t)s.ng * 16, bar(st, RB_FULL));
                } else
                    mbar_arrive(bar(st, RB_FULL));
            }
        };
        long long i = st;
        RowMeta next;
        if (i < n) {
            next = row_meta<OP>(a, first + i * step);
            start(i, next);
        }
        for (; i < n; i += ST) {
            const long long row = first + i * step;
            const RowMeta m = next;
            if (i + ST < n) next = row_meta<OP>(a, first + (i + ST) * step);  // used when this row is done
            const Slice s = slice_of<DT>(a.x, row, a.ld, a.V, L.G, rank);
            MS r{-INFINITY, 0.f}, top{-INFINITY, 0.f};
            float2 Q = make_float2(0.f, 0.f), B = Q, D = Q;
            if (OP == LM_DISTILL && m.keep) teacher_side(a, row, eq, eid, Q, B);
            if (!(fine = mbar_wait_bounded(bar(st, RB_FULL), ph, abort, L.wait_ns))) break;
            copying = false;
            if (m.keep) {
                if (OP == LM_DISTILL)
                    student_side<DT>(a, s, se, ex, eq, eid, sc, D, top);
                else if (m.tgt >= s.e0 && m.tgt < s.e0 + s.ng * N)
                    D.x = Elem<DT>::get(se[m.tgt - s.e0]);
            }
            const float xt = D.x;  // the target's logit, where this slice has it
            if (OP == LM_DISTILL && a.tail && lane == 0) mbar_arrive(bar(st, RB_CUT));
            if (!(fine = mbar_wait_bounded(bar(st, RB_REC), ph, abort, L.wait_ns))) break;
            if (m.keep) {
                if (lane < NW) r = S.rec[st][lane];
                r = ms_warp(r, sc);
            }
            if (!a.grad && i + ST < n) {  // the slice is done with
                __syncwarp();
                start(i + ST, next);
            }
            if (m.keep && L.CL > 1) {
                const uint32_t par = kept & 1u;
                if (lane < L.CL) {
                    const uint32_t to = cluster_addr(smem_u32(S.mail[st][par][rank]), lane);
                    cluster_store(to, r.m);
                    cluster_store(to + 4, r.s);
                    cluster_store(to + 8, top.m);
                    cluster_store(to + 12, top.s);
                    cluster_store(to + 16, D.x);
                    cluster_store(to + 20, D.y);
                    cluster_arrive(cluster_addr(bar(st, RB_MAIL + par), lane));
                }
                if (!(fine = mbar_wait_cluster(bar(st, RB_MAIL + par), (kept >> 1) & 1u, abort, L.wait_ns))) break;
                r = top = MS{-INFINITY, 0.f};
                D = make_float2(0.f, 0.f);
                if (lane < L.CL) {
                    const float* p = S.mail[st][par][lane];
                    r = MS{p[0], p[1]};
                    top = MS{p[2], p[3]};
                    D = make_float2(p[4], p[5]);
                }
                r = ms_warp(r, sc);
                if (OP == LM_DISTILL) {
                    if (a.tail) top = ms_warp(top, sc);
                    D = ff_sum_or_far(D);
                } else
                    D.x = warp_sum(D.x);  // the one slice that has the target gave its logit
                ++kept;
            }
            RowCoef c;
            if (m.keep) {
                c = row_finish<OP>(a, row, m, r, top, Q, B, D, sc, rank == 0 && lane == 0, [&](const RowCoef& k) {
                    if (a.grad && lane == 0) {
                        S.coef[st] = k;
                        mbar_arrive(bar(st, RB_COEF));
                    }
                });
            } else if (lane == 0) {
                if (a.grad) mbar_arrive(bar(st, RB_COEF));
                if (rank == 0) row_outputs(a, row, 0.f);
            }
            if (a.grad) {
                // the corrections come after the columns they replace
                if (!(fine = mbar_wait_bounded(bar(st, RB_GRAD), ph, abort, L.wait_ns))) break;
                T* const grow = static_cast<T*>(a.grad) + row * a.ldg;
                if (m.keep) {
                    if (OP == LM_DISTILL) {
                        for (int k = lane; k < a.K; k += 32)
                            if (eid[k] >= 0)
                                grow[eid[k]] = Elem<DT>::put(c.fa * (weight_of(ex[k], c.M, sc) * c.inv_S) - c.fb * eq[k]);
                    } else if (lane == 0 && m.tgt >= s.e0 && m.tgt < s.e0 + s.ng * N)
                        grow[m.tgt] = Elem<DT>::put(c.fa * (weight_of(xt, c.M, sc) * c.inv_S) - c.fb);
                }
                __syncwarp();
                if (i + ST < n) start(i + ST, next);
            }
            ph ^= 1u;
        }
        if (!fine) {
            if (copying) {  // no copy may be in flight when the CTA ends
                int dummy = 0;
                mbar_wait_bounded(bar(st, RB_FULL), cph, &dummy, L.wait_ns);
            }
            if (lane == 0) atomicOr(L.status, SOT_DEV_TIMEOUT);
            if (rank == 0 && lane == 0)
                for (; i < n; i += ST) row_outputs(a, first + i * step, NAN);
        }
    }
    __syncwarp();
    if (L.CL > 1) cluster_sync();  // no CTA leaves while a peer may still store to it
}

// Short rows: one warp takes a row from its copy to its corrections, so nothing is
// handed from warp to warp and a row costs one warp's instructions.  Two buffers
// a warp: the next row's copy is under way while this one is worked on.
constexpr int WARP_ROWS = 4;  // warps of a CTA

template <int DT, int OP>
__global__ void __launch_bounds__(WARP_ROWS * 32, 6) lm_warp_kernel(const LmRowArgs a, const LmRowLaunch L) {
    using T = typename Elem<DT>::T;
    extern __shared__ __align__(128) uint4 sm[];
    __shared__ uint64_t full[WARP_ROWS][2];
    __shared__ int timed_out[WARP_ROWS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float sc = SOT_LOG2E / a.tau;
    uint4* const buf = sm + (size_t)warp * 2 * L.G;
    float* const ex = reinterpret_cast<float*>(sm + (size_t)WARP_ROWS * 2 * L.G) + (size_t)warp * 3 * a.K;
    float* const eq = ex + a.K;
    int* const eid = reinterpret_cast<int*>(eq + a.K);
    const uint32_t bar0 = smem_u32(&full[warp][0]);
    volatile int* const abort = &timed_out[warp];
    if (lane == 0) {
        mbar_init(bar0, 1);
        mbar_init(bar0 + 8, 1);
        *abort = 0;
        fence_mbar_init();
    }
    __syncwarp();
    const long long first = (long long)blockIdx.x * WARP_ROWS + warp, step = (long long)gridDim.x * WARP_ROWS;
    bool copying[2] = {false, false};
    auto start = [&](long long row, const RowMeta& m, int b) {
        copying[b] = row / step != L.hold;
        if (lane == 0 && copying[b]) {
            const Slice s = slice_of<DT>(a.x, row, a.ld, a.V, L.G, 0);
            if (m.keep) {
                mbar_arrive_expect_tx(bar0 + 8 * b, (uint32_t)s.ng * 16);
                bulk_g2s(smem_u32(buf + (size_t)b * L.G), s.src, (uint32_t)s.ng * 16, bar0 + 8 * b);
            } else
                mbar_arrive(bar0 + 8 * b);
        }
    };
    long long row = first;
    RowMeta m, next;
    if (row < a.T) {
        m = row_meta<OP>(a, row);
        start(row, m, 0);
        if (row + step < a.T) next = row_meta<OP>(a, row + step);
    }
    uint32_t ph = 0u;
    int b = 0;
    for (; row < a.T; row += step) {
        RowMeta after;
        if (row + step < a.T) {
            start(row + step, next, b ^ 1);  // that buffer's row is done
            if (row + 2 * step < a.T) after = row_meta<OP>(a, row + 2 * step);
        }
        float2 Q = make_float2(0.f, 0.f), B = Q, D = Q;
        if (OP == LM_DISTILL && m.keep) teacher_side(a, row, eq, eid, Q, B);
        if (!mbar_wait_bounded(bar0 + 8 * b, ph, abort, L.wait_ns)) break;
        copying[b] = false;
        const Slice s = slice_of<DT>(a.x, row, a.ld, a.V, L.G, 0);
        uint4* const src = buf + (size_t)b * L.G;
        T* const se = reinterpret_cast<T*>(src);
        T* const grow = a.grad ? static_cast<T*>(a.grad) + row * a.ldg : nullptr;
        const bool aligned =
            ((uint32_t)((unsigned long long)grow ^ (unsigned long long)(static_cast<const T*>(a.x) + row * a.ld)) & 15u) == 0;
        if (m.keep) {
            MS top{-INFINITY, 0.f};
            if (OP == LM_DISTILL) student_side<DT>(a, s, se, ex, eq, eid, sc, D, top);
            else D.x = Elem<DT>::get(se[m.tgt - s.e0]);
            const MS r = ms_warp(slice_stats<DT, 32>(s, src, a.V, sc, lane), sc);
            const RowCoef c = row_finish<OP>(a, row, m, r, top, Q, B, D, sc, lane == 0, [](const RowCoef&) {});
            if (grow) {
                slice_grad<DT, 32>(s, src, c, grow, a.V, sc, aligned, lane);
                __syncwarp();  // the corrections come after the columns they replace
                if (OP == LM_DISTILL) {
                    for (int k = lane; k < a.K; k += 32)
                        if (eid[k] >= 0)
                            grow[eid[k]] = Elem<DT>::put(c.fa * (weight_of(ex[k], c.M, sc) * c.inv_S) - c.fb * eq[k]);
                } else if (lane == 0)
                    grow[m.tgt] = Elem<DT>::put(c.fa * (weight_of(D.x, c.M, sc) * c.inv_S) - c.fb);
            }
        } else {
            if (grow) slice_zero<DT, 32>(s, grow, a.V, aligned, lane);
            if (lane == 0) row_outputs(a, row, 0.f);
        }
        __syncwarp();
        m = next;
        next = after;
        b ^= 1;
        if (b == 0) ph ^= 1u;
    }
    if (row < a.T) {  // a wait ran out: no copy may be in flight when the CTA ends
        int dummy = 0;
        if (copying[b]) mbar_wait_bounded(bar0 + 8 * b, ph, &dummy, L.wait_ns);
        if (copying[b ^ 1]) mbar_wait_bounded(bar0 + 8 * (b ^ 1), b ? ph ^ 1u : ph, &dummy, L.wait_ns);
        if (lane == 0) {
            atomicOr(L.status, SOT_DEV_TIMEOUT);
            for (; row < a.T; row += step) row_outputs(a, row, NAN);
        }
    }
}

struct LmRowPlan {
    int NW, CL, G, ST, lag;  // NW = 1: the short-row kernel
    size_t smem;
    int sms;
};

template <int DT, int OP, int NW>
cudaError_t launch_row_n(const LmRowArgs& a, const LmRowPlan& p, LmRowLaunch L, cudaStream_t st) {
    auto kern = lm_row_kernel<DT, OP, NW>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)p.smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.CL, 1, 1);
    cfg.blockDim = dim3((NW + p.ST) * 32, 1, 1);
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
    L.CL = p.CL;
    L.G = p.G;
    L.ST = p.ST;
    L.lag = p.lag;
    e = cudaLaunchKernelEx(&cfg, kern, a, L);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int DT, int OP>
cudaError_t launch_row_w(const LmRowArgs& a, const LmRowPlan& p, LmRowLaunch L, cudaStream_t st) {
    auto kern = lm_warp_kernel<DT, OP>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)p.smem);
    if (e != cudaSuccess) return e;
    int per_sm = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, WARP_ROWS * 32, p.smem);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    const long long want = (a.T + WARP_ROWS - 1) / WARP_ROWS, most = (long long)per_sm * p.sms;
    L.CL = 1;
    L.G = p.G;
    kern<<<(unsigned)(want < most ? want : most), WARP_ROWS * 32, p.smem, st>>>(a, L);
    return cudaGetLastError();
}

template <int DT, int OP>
cudaError_t launch_row_o(const LmRowArgs& a, const LmRowPlan& p, const LmRowLaunch& L, cudaStream_t st) {
    switch (p.NW) {
        case 1: return launch_row_w<DT, OP>(a, p, L, st);
        case 4: return launch_row_n<DT, OP, 4>(a, p, L, st);
        case 8: return launch_row_n<DT, OP, 8>(a, p, L, st);
        default: return launch_row_n<DT, OP, 16>(a, p, L, st);
    }
}

template <int DT>
cudaError_t launch_row_t(LmOp op, const LmRowArgs& a, const LmRowPlan& p, const LmRowLaunch& L, cudaStream_t st) {
    switch (op) {
        case LM_LOGPROB: return launch_row_o<DT, LM_LOGPROB>(a, p, L, st);
        case LM_POLICY: return launch_row_o<DT, LM_POLICY>(a, p, L, st);
        default: return launch_row_o<DT, LM_DISTILL>(a, p, L, st);
    }
}

// One translation unit per type (k_lm_f32.cu, k_lm_f16.cu, k_lm_bf16.cu).
cudaError_t launch_row_f32(LmOp op, const LmRowArgs& a, const LmRowPlan& p, const LmRowLaunch& L, cudaStream_t st);
cudaError_t launch_row_f16(LmOp op, const LmRowArgs& a, const LmRowPlan& p, const LmRowLaunch& L, cudaStream_t st);
cudaError_t launch_row_bf16(LmOp op, const LmRowArgs& a, const LmRowPlan& p, const LmRowLaunch& L, cudaStream_t st);

}  // namespace sot
