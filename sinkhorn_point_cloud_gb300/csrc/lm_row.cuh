// lm_row.cuh -- losses over rows of logits, with their gradients.
//
// A row x of V logits at temperature tau has p = softmax(x / tau).  Every loss
// here depends on the row through log p at a few columns, so its gradient is
//   dx_v = c p_v   at every column, corrected at those few columns,
// with c known once the row's log-sum-exp is.  Memory traffic bounds all of it:
// the least is one read of the row and one write of the gradient.
//
// lm_row_kernel: a CTA takes a row, or a cluster of CTAs a slice of it each, in
// two passes: statistics, then the gradient.  The second pass reads the row
// again, from L2, where it still is: the rows under way at one time take 40 to 60
// of the 129 MB, and the first pass asks L2 to keep them while the stores and the
// second pass ask for nothing to be kept (counted: DRAM reads are the logits
// once, 0.2697 GB for 0.2684 GB).  Several CTAs share an SM and are in different
// phases, so loads, reductions and stores of different rows overlap without any
// hand-over inside a CTA.  A warp of its own prepares the teacher's side during
// the first pass, joins the statistics (with the cluster's other CTAs through
// distributed shared memory) and forms the loss and the gradient's coefficients.
//   Measured on the GPU, of 6779 GB/s of copy bandwidth: log-probabilities of 16384 x
//   32000 bf16 in 155 us (1.00); policy loss of 8192 x 65536, a third of the rows left
//   out, in 276 us (0.95); distillation of 4096 x 131072 in 340 us (0.93).  Batches of a
//   few waves of CTAs lose part of the last one: 3001 x 50021 fp16 in 103 us (0.82),
//   1001 x 50021 fp32 with the tail in 72 us (0.72).  Few rows: 4 to 6 us, the
//   latency of one launch, one load, a reduction across the cluster and one store.
//   Also tried (347 us for the distillation then): slices resident in shared memory, copied in bulk by warps of their
//   own (465 us for the distillation: a row's slices wait for one another), a ring
//   of chunks (519 us: 0.4 us of hand-overs a chunk), a resident grid that walks the
//   rows (442 us).
//
// lm_short_kernel: short rows, a warp each, kept in registers between the passes.
//   16384 rows of 2048 bf16: policy loss 28 us with gradient (0.71), 18 us without; with a
//   CTA a row it was 73 and 46 us.  Distillation with 8 entries 44 us, with the tail 50
//   us: the chain of the entries' loads and sums is what a row waits for.
#pragma once
#include <cuda_runtime.h>

#include "lm.cuh"
#include "lm.h"

namespace sot {

constexpr int ROW_MAX_CL = 8;
constexpr int NREC = 8;  // a CTA's record: (m, s), the entries' (m, s), its part of their distance or the target's logit

struct LmRowLaunch {
    int CL, G;  // CTAs a row, granules a slice
};

// Sums against the guessed stabiliser 0 may be as small as 2^-40, and weights that are
// formed against it again would vanish where probabilities are still 2^-86.  For such a sum,
// k = floor(log2 s) is the better stabiliser, and an exact one; returns 2^k.
__device__ __forceinline__ float small_sum(float m, float s, float& k) {
    const bool small = m == 0.f && s > 0.f && s < 1.f;
    const uint32_t e = __float_as_uint(s) & 0x7f800000u;
    k = small ? (float)((int)(e >> 23) - 127) : 0.f;
    return small ? __uint_as_float(e) : 1.f;
}

// What the row's threads need once its statistics are known.
struct RowCoef {
    float u, c;      // dx_v = c exp2(x_v sc - u)
    float far;       // not 0: dx_v = c where x_v = m, 0 elsewhere
    float m;
    float M, inv_S;  // p_v = weight of x_v against M times inv_S;
    float k;         // k < 0: weight of x_v is exp2(x_v sc - k) instead
    float fa, fb;    // a corrected column: fa p_v - fb q_v
    __device__ __forceinline__ void set(float v, float sc) {
        const float v2 = __fmul_rn(v, sc);
        m = v;
        far = is_far(v2) ? 1.f : 0.f;
        u = far != 0.f ? 0.f : v2;
    }
    __device__ __forceinline__ float prob(float x, float sc) const {
        return (k < 0.f ? ex2f(fmaf(x, sc, -k)) : weight_of(x, M, sc)) * inv_S;
    }
};

// The slice of a row that CTA `rank` of its cluster takes, in 16-byte
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

// The teacher's entries of a row (one warp), in two steps.  First the entries as
// they are: values in eq (-inf: unused), columns in eid (-1: unused); returns the
// largest value.  The student's logits in columns [c0, c1) of the row at x are on
// their way to ex meanwhile.  U loads in flight: 4096 x 32000 with 256 entries take
// 121 us with four and the logits fetched after the weights, 115 with the logits
// fetched here, 106 with eight; short rows have no registers for eight (57 and 65 us).
template <int DT, int U>
__device__ __forceinline__ float teacher_entries(const LmRowArgs& a, long long row, int c0, int c1,
                                                 const typename Elem<DT>::T* x, float* ex, float* eq, int* eid) {
    const int lane = threadIdx.x & 31;
    float zmax = -INFINITY;
    for (int k0 = 0; k0 < a.K; k0 += 32 * U) {  // U loads in flight a lane
        int id[U];
        float z[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int k = k0 + 32 * j + lane;
            id[j] = k < a.K ? load_index(a.ids, a.ids_type, row * a.K + k, a.V) : -1;
            z[j] = k < a.K ? load_float(a.teacher, a.teacher_type, row * a.K + k) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int k = k0 + 32 * j + lane;
            if (id[j] < 0) z[j] = -INFINITY;
            zmax = fmaxf(zmax, z[j]);
            if (id[j] >= 0 && id[j] >= c0 && id[j] < c1) fetch_element(ex + k, x + id[j]);
            if (k < a.K) {
                eid[k] = id[j];
                eq[k] = z[j];
            }
        }
    }
    return warp_max1(zmax);
}
// Then the weights q in eq, and the sums Q = sum q and B = sum q log q.
__device__ __forceinline__ void teacher_weights(const LmRowArgs& a, float zmax, float* eq, float2& Q, float2& B) {
    const int lane = threadIdx.x & 31;
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

// s + v; a sum that is not finite goes without its low part (which would be NaN), so that an
// infinity stays one whatever is added after it.
__device__ __forceinline__ float2 ff_add_or_far(float2 s, float2 v) {
    const float f = s.x + v.x;
    return fabsf(f) < INFINITY ? ff_add(s, v) : make_float2(f, 0.f);
}
// Sum over a warp, with the same exception.
__device__ __forceinline__ float2 ff_sum_or_far(float2 v) {
    const float2 s = ff_warp_sum(v);
    const float f = warp_sum(v.x);
    return fabsf(f) < INFINITY ? s : make_float2(f, 0.f);
}

// A sum whose low parts are summed apart (y), so that the chain from term to term is one addition.
__device__ __forceinline__ void sum_apart(float2& s, float2 v) {
    const float2 t = two_sum(s.x, v.x);
    s = make_float2(t.x, s.y + (t.y + v.y));
}
__device__ __forceinline__ float2 warp_sum_apart(float2 s) {
    return ff_sum_or_far(fabsf(s.x) < INFINITY ? ff_renorm(s.x, s.y) : make_float2(s.x, 0.f));
}
// sum q (x - m) over the entries (one warp): what a row's loss needs of the student's logits.
// Against m the terms have one sign, or are small, so nothing is lost where the logits lie far from 0.
// (Seldom needed, so kept out of line: inside, 4096 x 32000 bf16 with 64 entries take 88.1 us, so 86.3.)
static __device__ __noinline__ float2 entries_distance(int K, const float* ex, const float* eq, float m) {
    float2 D = make_float2(0.f, 0.f);
    for (int k = threadIdx.x & 31; k < K; k += 32)
        if (eq[k] != 0.f) sum_apart(D, two_prod(eq[k], ex[k] - m));  // (0: unused ones too)
    return warp_sum_apart(D);
}
// The same before m is known: D against X.  X is 0, or in a slice with a logit beyond 64 the largest; Q =
// sum q of a slice takes D from there to m.
struct Part {
    float X, Q;
    float2 D;
    __device__ __forceinline__ float2 distance(float m) const {
        const float up = X - m;
        return ff_add_or_far(D, fabsf(up) < INFINITY ? two_prod(Q, up) : make_float2(Q * up, 0.f));
    }
};
// And once it is, for entries in one piece: from 0 if that is near, otherwise all over again.
__device__ __forceinline__ float2 row_distance(const LmRowArgs& a, const float* ex, const float* eq, const Part& part,
                                               float2 Q, float m) {
    if (m == 0.f) return part.D;
    if (fabsf(m) <= 64.f) return ff_add_or_far(part.D, ff_mul(Q, make_float2(-m, 0.f)));
    return entries_distance(a.K, ex, eq, m);
}

// The entries' logits in columns [c0, c1) of a row at x, from what teacher_entries
// fetched: ex and their part; eid becomes -1 (and q 0) for the others.  For the tail also the
// entries' statistics.
template <int DT>
__device__ __forceinline__ void student_side(const LmRowArgs& a, int c0, int c1, const typename Elem<DT>::T* x, float* ex,
                                             float* eq, int* eid, float sc, bool slice, Part& part, MS& top) {
    const int lane = threadIdx.x & 31;
    part = Part{0.f, 0.f, make_float2(0.f, 0.f)};
    top = MS{-INFINITY, 0.f};
    async_wait();
    for (int k = lane; k < a.K; k += 32) {
        const int id = eid[k];
        if (!(id >= 0 && id >= c0 && id < c1)) {
            ex[k] = -INFINITY;
            eq[k] = 0.f;
            eid[k] = -1;
            continue;
        }
        const float v = element_of<DT>(ex[k], x + id), q = eq[k];
        ex[k] = v;
        top.m = fmaxf(top.m, v);
        if (q != 0.f) sum_apart(part.D, two_prod(q, v));
        part.Q += q;
    }
    const bool far = fabsf(top.m) < INFINITY && fabsf(top.m) > 64.f;
    part.D = warp_sum_apart(part.D);
    if (slice) {
        part.Q = warp_sum(part.Q);
        if (__any_sync(0xffffffffu, far)) {
            part.X = warp_max1(fabsf(top.m) < INFINITY ? top.m : -INFINITY);
            part.D = entries_distance(a.K, ex, eq, part.X);
        }
    }
    if (a.tail) {
        top.m = warp_max1(top.m);
        for (int k = lane; k < a.K; k += 32)
            if (eid[k] >= 0) top.s += weight_of(ex[k], top.m, sc);
        top.s = top.m == -INFINITY ? 0.f : warp_sum(top.s);
    }
}

// log sum exp((x - m) / tau) from sums against the rounded m2, which hold exp2(m sc - m2) as a factor.
__device__ __forceinline__ float2 log_sum(MS v, float sc) {
    const float m2 = __fmul_rn(v.m, sc);
    const float2 l = log_ff(v.s);
    return v.m == 0.f || is_far(m2) ? l : ff_add(l, make_float2(-fmaf(v.m, sc, -m2) * SOT_LN2, 0.f));
}

// What a row's loss depends on besides its logits.
struct RowMeta {
    int tgt;
    float w, old, ref, adv;
    bool keep;
};
// `all`: the policy's values too, which only the row's own warp needs.
template <int OP>
__device__ __forceinline__ RowMeta row_meta(const LmRowArgs& a, long long row, bool all) {
    RowMeta m;
    m.tgt = OP == LM_DISTILL ? 0 : load_index(a.target, a.target_type, row, a.V);
    m.w = OP == LM_LOGPROB ? 1.f : a.weight ? a.weight[row] : 1.f / (float)a.T;
    m.old = m.ref = m.adv = 0.f;
    if (OP == LM_POLICY && all) {
        m.old = a.old_logp[row];
        m.adv = a.adv[row];
        if (a.ref_logp) m.ref = a.ref_logp[row];
    }
    m.keep = m.tgt >= 0 && m.w != 0.f;
    return m;
}

// The row's loss and the gradient's coefficients from its joined statistics
// (one warp): r without and top with the entries of a tail, xt the target's logit.  `publish` hands
// the coefficients on before the losses, which nothing waits for, are finished; `distance` gives the
// entries' sum q (x - m) to every lane, `lead` is whether this CTA writes the row's losses.
template <int OP, class Publish, class Distance>
__device__ __forceinline__ RowCoef row_finish(const LmRowArgs& a, long long row, const RowMeta& m, MS r, MS top, float2 Q,
                                              float2 B, float xt, float sc, bool lead, Publish publish,
                                              Distance distance) {
    const bool write = lead && (threadIdx.x & 31) == 0;
    const MS all = OP == LM_DISTILL && a.tail ? ms_combine(r, top, sc) : r;
    const float m2 = __fmul_rn(all.m, sc);
    const bool far = is_far(m2);
    const float2 ln2 = make_float2(0.693147182f, -1.904654212e-9f);
    RowCoef c;
    c.M = all.m;
    const float inv = __frcp_rn(all.s);
    c.inv_S = inv * small_sum(all.m, all.s, c.k);
    c.set(all.m, sc);
    if (c.k < 0.f) c.u = c.k;
    if (OP == LM_DISTILL) {
        const float wt = m.w * a.tau;
        float qr = 0.f;
        c.fa = wt * Q.x;
        c.fb = wt;
        c.c = c.fa * c.inv_S;
        if (a.tail) {
            // no column outside the entries: no tail outcome (a NaN of the entries stays one)
            const float rest = (1.f - Q.x) - Q.y;
            qr = r.s == 0.f ? 0.f : r.s > 0.f ? (rest <= 0.f ? 0.f : rest) : r.s;
            c.fa = wt * (Q.x + qr);
            float k;
            const float two_k = small_sum(r.m, r.s, k);
            c.set(r.m, sc);
            if (k < 0.f) c.u = k;
            c.c = r.s == 0.f ? 0.f * inv * c.fa : wt * ((Q.x + qr) * rescale(r.m, c.M, sc) * inv - qr / r.s) * two_k;
        }
        publish(c);
        if (!a.loss || !lead) return c;
        const float2 E = distance(all.m);
        if (write) {
            // With y = (x - m) / tau and S = sum exp y over the row, R over what is not an entry:
            //   log p = y - log S,  log p_r = (m_r - m) / tau + log R - log S.
            // In pairs of floats: with doubles throughout, 16384 rows of 2048 take 12 us more.
            const bool tail = a.tail && !(qr <= 0.f);
            const float2 inv_tau = make_float2(a.inv_hi, a.inv_lo), logS = log_sum(all, sc);
            const float2 logR = tail ? log_sum(r, sc) : logS, logq = tail ? log_ff(qr) : logS;
            float2 sum = make_float2(0.f, 0.f);
            if (!(Q.x <= 0.f)) {  // B + Q log S - E / tau; NaN where a used entry is NaN or +inf
                const float2 d = ff_mul(E, inv_tau);
                sum = ff_add(ff_add(B, ff_mul(Q, logS)), make_float2(-d.x, -d.y));
            }
            if (tail) {  // + q_r (log q_r - log p_r)
                const float2 apart = ff_mul(two_sum(r.m, -all.m), inv_tau);
                const float2 logp = ff_add(ff_add(apart, logR), make_float2(-logS.x, -logS.y));
                sum = ff_add(sum, ff_mul(ff_add(logq, make_float2(-logp.x, -logp.y)), make_float2(qr, 0.f)));
            }
            float loss = (sum.x + sum.y) * m.w * a.tau * a.tau;
            if (!(fabsf(loss) < INFINITY)) {  // with the range of a double
                const double q = to_double(Q);
                double l = 0.0;
                if (!(q <= 0.0)) l = to_double(B) + q * to_double(logS) - to_double(E) * a.inv_tau;
                if (tail)
                    l += (double)qr * (to_double(logq) -
                                       (((double)r.m - (double)all.m) * a.inv_tau + to_double(logR) - to_double(logS)));
                loss = (float)(l * (double)m.w * (double)a.tau * (double)a.tau);
            }
            a.loss[row] = loss;
        }
        return c;
    }
    // logp = (x - m) / tau - log S, kept to more than 24 bits until it is compared.  The difference
    // is exact; through the rounded sc and m2 a logit at -65504 would be off by 1e-3.  Beyond
    // 2^24 a log-probability that was stored in 32 bits says nothing of the low part.
    const float2 logS = log_sum(all, sc), d = two_sum(xt, -all.m);
    float2 logp = ff_add(ff_mul(d, make_float2(a.inv_hi, a.inv_lo)), make_float2(-logS.x, -logS.y));
    if (!(fabsf(logp.x) < INFINITY)) logp = make_float2((float)(((double)xt - (double)all.m) * a.inv_tau) - logS.x, 0.f);
    if (fabsf(logp.x) >= 0x1p24f) logp.y = 0.f;
    float g = 0.f, loss = 0.f, kl = 0.f;
    if (OP == LM_POLICY) {
        const float2 d0 = two_sum(logp.x, -m.old);
        const float ratio = expf(fabsf(d0.x) < INFINITY ? d0.x + (d0.y + logp.y) : d0.x);
        // (a ratio beyond the range of a float times no advantage is 0)
        const float free = m.adv == 0.f && ratio == INFINITY ? 0.f : ratio * m.adv;
        const float held = fminf(fmaxf(ratio, a.clip_lo), a.clip_hi) * m.adv;
        loss = -fminf(free, held);
        g = free <= held ? -free : 0.f;
        if (free != free) loss = g = free;
        if (a.ref_logp) {
            const float2 d1 = two_sum(m.ref, -logp.x);
            const float d = fabsf(d1.x) < INFINITY ? d1.x + (d1.y - logp.y) : d1.x;
            kl = exp_minus_linear(d);
            if (a.kl_coef != 0.f) {
                loss += a.kl_coef * kl;
                g -= a.kl_coef * expm1f(d);  // (kl + d would have lost it in the rounding of a large -d)
            }
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
            // (with m2 and s as they are: what the gradient from it forms again)
            const float2 l = ff_add(ff_mul(make_float2(m2, 0.f), ln2), log_ff(all.s));
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

// ---- what NT threads (tid = 0 .. NT - 1) do with a slice.  Granules inside the
// row, [lo, hi), go in batches, so that their loads are under way together; the
// granule the row starts in and the one it ends in belong to two threads of the last
// warp, whose share is the shortest (with the first warp 6080 x 50021 fp16 take 222 us,
// so 219).  With
// CUT, byte g of `cut` names the elements of granule g that are left out.
__device__ __forceinline__ int edge_granule(const Slice& s, int tid, int NT) {
    if (tid == NT - 1 && s.ng > 0 && s.lo > 0) return 0;
    if (tid == NT - 2 && s.ng > 0 && s.hi < s.ng && (s.ng > 1 || s.lo == 0)) return s.ng - 1;
    return -1;
}
template <int DT>
__device__ __forceinline__ uint4 without(const uint4& v, unsigned out) {
    float2 f[Elem<DT>::N / 2];
    unpack<DT>(v, f);
#pragma unroll
    for (int i = 0; i < Elem<DT>::N / 2; ++i) {
        if (out >> (2 * i) & 1u) f[i].x = -INFINITY;
        if (out >> (2 * i + 1) & 1u) f[i].y = -INFINITY;
    }
    return pack<DT>(f);
}

// Behind the bytes, one for each batch of a thread names the granules of it that
// have any: one load tells a batch that it is whole (a load for each granule takes
// 318 us instead of 305 for 4096 x 50021 fp32 with 100 entries).
constexpr int BATCH = 8;  // granules of a thread
__host__ __device__ inline int cut_bytes(int G) { return (G + 3) / 4 * 4; }
__host__ __device__ inline int cut_batches(int G, int NT) { return (G + BATCH * NT - 1) / (BATCH * NT) * NT; }

template <int DT, bool CUT>
__device__ __forceinline__ void slice_stats(Running& r, const Slice& s, uint64_t policy, const unsigned char* cut, int G,
                                            int V, float sc, int tid, int NT) {
    const auto src = [&](int g) { return load16(s.src + g, policy); };
    constexpr int N = Elem<DT>::N, U = BATCH / 2;
    const unsigned char* mine = cut + cut_bytes(G) + tid;
    for (int g = s.lo + tid; g < s.hi; g += 2 * U * NT) {
        uint4 v[U], w[U];
        if (g + (2 * U - 1) * NT < s.hi) {
#pragma unroll
            for (int j = 0; j < U; ++j) v[j] = src(g + j * NT);
#pragma unroll
            for (int j = 0; j < U; ++j) w[j] = src(g + (U + j) * NT);
        } else {  // the last batch: -inf for what is not there
#pragma unroll
            for (int j = 0; j < U; ++j) v[j] = g + j * NT < s.hi ? src(g + j * NT) : nothing<DT>();
#pragma unroll
            for (int j = 0; j < U; ++j) w[j] = g + (U + j) * NT < s.hi ? src(g + (U + j) * NT) : nothing<DT>();
        }
        if (CUT) {
            const unsigned marked = *mine;
            mine += NT;
            if (marked) {
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    if (marked >> j & 1u) v[j] = without<DT>(v[j], cut[g + j * NT]);
                    if (marked >> (U + j) & 1u) w[j] = without<DT>(w[j], cut[g + (U + j) * NT]);
                }
            }
        }
        r.template add<DT>(v, sc);
        if (g + U * NT < s.hi) r.template add<DT>(w, sc);
    }
    const int e = edge_granule(s, tid, NT);
    if (e >= 0) {
        float2 f[N / 2];
        unpack<DT>(src(e), f);
        mask_cols<DT>(f, s.e0 + e * N, V, -INFINITY);
        uint4 v[1] = {pack<DT>(f)};
        if (CUT && cut[e]) v[0] = without<DT>(v[0], cut[e]);
        r.template add<DT>(v, sc);
    }
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

// grow: the gradient's row; aligned: its granules are the logits' granules.
template <int DT>
__device__ __forceinline__ void slice_grad(const Slice& s, const RowCoef& c, typename Elem<DT>::T* grow, int V, float sc,
                                           bool aligned, uint64_t policy, int tid, int NT) {
    const auto src = [&](int g) { return load16(s.src + g, policy); };
    constexpr int N = Elem<DT>::N, U = 4;
    if (aligned) {
        uint4* const dst = reinterpret_cast<uint4*>(grow + s.e0);
        for (int g = s.lo + tid; g < s.hi; g += U * NT) {
            uint4 v[U];
            if (g + (U - 1) * NT < s.hi) {
#pragma unroll
                for (int j = 0; j < U; ++j) v[j] = src(g + j * NT);
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    float2 f[N / 2];
                    unpack<DT>(v[j], f);
                    grad_of<DT>(f, c, sc);
                    store16(dst + g + j * NT, pack<DT>(f), policy);
                }
            } else {
#pragma unroll
                for (int j = 0; j < U - 1; ++j)
                    if (g + j * NT < s.hi) v[j] = src(g + j * NT);
#pragma unroll
                for (int j = 0; j < U - 1; ++j)
                    if (g + j * NT < s.hi) {
                        float2 f[N / 2];
                        unpack<DT>(v[j], f);
                        grad_of<DT>(f, c, sc);
                        store16(dst + g + j * NT, pack<DT>(f), policy);
                    }
            }
        }
        const int e = edge_granule(s, tid, NT);
        if (e >= 0) {
            float2 f[N / 2];
            unpack<DT>(src(e), f);
            grad_of<DT>(f, c, sc);
            store_cols<DT>(grow, s.e0 + e * N, V, f, false);
        }
    } else {
        for (int g = tid; g < s.ng; g += NT) {
            float2 f[N / 2];
            unpack<DT>(src(g), f);
            grad_of<DT>(f, c, sc);
            store_cols<DT>(grow, s.e0 + g * N, V, f, false);
        }
    }
}

template <int DT>
__device__ __forceinline__ void slice_zero(const Slice& s, typename Elem<DT>::T* grow, int V, bool aligned, int tid, int NT) {
    constexpr int N = Elem<DT>::N;
    float2 z[N / 2];
#pragma unroll
    for (int k = 0; k < N / 2; ++k) z[k] = make_float2(0.f, 0.f);
    for (int g = tid; g < s.ng; g += NT) store_cols<DT>(grow, s.e0 + g * N, V, z, aligned);
}

// NW streaming warps and the row's own warp.
template <int DT, int OP, int NW, bool TAIL>
__global__ void __launch_bounds__((NW + 1) * 32, NW == 4 ? (OP == LM_LOGPROB ? 8 : 7) : NW == 8 ? 4 : 2)
    lm_row_kernel(const LmRowArgs a, const LmRowLaunch L) {
    using T = typename Elem<DT>::T;
    constexpr int N = Elem<DT>::N, NT = NW * 32;
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ MS rec[NW];
    __shared__ float mail[ROW_MAX_CL][NREC];
    __shared__ RowCoef coef;
    float* const ex = reinterpret_cast<float*>(dyn);  // entries: logit, weight, column; then (tail) the slice's cut bytes
    float* const eq = ex + a.K;
    int* const eid = reinterpret_cast<int*>(eq + a.K);
    unsigned* const cut = reinterpret_cast<unsigned*>(eid + a.K);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();
    const float sc = SOT_LOG2E / a.tau;
    const long long row = blockIdx.x / L.CL;
    const RowMeta m = row_meta<OP>(a, row, warp == NW);
    const T* const x = static_cast<const T*>(a.x) + row * a.ld;
    T* const grow = OP != LM_LOGPROB && a.grad ? static_cast<T*>(a.grad) + row * a.ldg : nullptr;
    const bool aligned = same_granules<T>(x, grow);
    const Slice s = slice_at<DT>(x, a.V, L.G, rank);
    const int c0 = s.e0, c1 = s.e0 + s.ng * N;  // the slice's columns
    const uint64_t last = policy_drop(), first = grow ? policy_keep() : last;
    if (!m.keep) {  // the same for the whole cluster
        if (grow && warp < NW) slice_zero<DT>(s, grow, a.V, aligned, tid, NT);
        if (rank == 0 && tid == 0) row_outputs(a, row, 0.f);
        return;
    }
    if (L.CL > 1) cluster_arrive_started();
    if (TAIL) {
        for (int g = tid; g < (cut_bytes(L.G) + cut_batches(L.G, NT)) / 4; g += NT + 32) cut[g] = 0u;
        __syncthreads();
    }
    float2 Q = make_float2(0.f, 0.f), B = Q;
    Part part{0.f, 0.f, Q};
    float xt = 0.f;  // the target's logit, where this slice has it
    MS top{-INFINITY, 0.f};
    if (warp == NW) {
        if (OP == LM_DISTILL) {
            const float zmax = teacher_entries<DT, 8>(a, row, c0, c1, x, ex, eq, eid);
            if (TAIL) {
                for (int k = lane; k < a.K; k += 32) {
                    const int at = eid[k] - c0;
                    if (eid[k] < 0 || at < 0 || eid[k] >= c1) continue;
                    const int g = at / N, q = g - s.lo, f = q / (BATCH * NT) * NT + q % NT;
                    atomicOr(cut + g / 4, 1u << (g % 4 * 8 + at % N));
                    if (q >= 0 && g < s.hi) atomicOr(cut + cut_bytes(L.G) / 4 + f / 4, 1u << (f % 4 * 8 + q / NT % BATCH));
                }
                __syncthreads();  // the others can start
            }
            teacher_weights(a, zmax, eq, Q, B);
            student_side<DT>(a, c0, c1, x, ex, eq, eid, sc, L.CL > 1, part, top);
        } else if (m.tgt >= c0 && m.tgt < c1)
            xt = Elem<DT>::get(x[m.tgt]);
    } else {
        if (TAIL) __syncthreads();
        Running r;
        slice_stats<DT, TAIL>(r, s, first, reinterpret_cast<const unsigned char*>(cut), L.G, a.V, sc, tid, NT);
        const MS w = ms_warp(r.result(), sc);
        if (lane == 0) rec[warp] = w;
    }
    if (L.CL > 1) cluster_wait_started();  // every CTA of the cluster is there to be stored to
    __syncthreads();
    MS r{-INFINITY, 0.f};
    if (warp == NW) {
        if (lane < NW) r = rec[lane];
        r = ms_warp(r, sc);
        if (L.CL > 1 && lane < L.CL) {
            const uint32_t to = cluster_addr(smem_u32(mail[rank]), lane);
            cluster_store(to, r.m);
            cluster_store(to + 4, r.s);
            cluster_store(to + 8, top.m);
            cluster_store(to + 12, top.s);
            if (OP == LM_DISTILL) {
                cluster_store(to + 16, part.X);
                cluster_store(to + 20, part.Q);
                cluster_store(to + 24, part.D.x);
                cluster_store(to + 28, part.D.y);
            } else
                cluster_store(to + 16, xt);
        }
        __syncwarp();
    }
    if (L.CL > 1) cluster_sync();
    if (warp == NW) {
        if (L.CL > 1) {
            r = top = MS{-INFINITY, 0.f};
            part = Part{0.f, 0.f, make_float2(0.f, 0.f)};
            if (lane < L.CL) {
                const float* p = mail[lane];
                r = MS{p[0], p[1]};
                top = MS{p[2], p[3]};
                if (OP == LM_DISTILL) part = Part{p[4], p[5], make_float2(p[6], p[7])};
                else xt = p[4];
            }
            r = ms_warp(r, sc);
            if (TAIL) top = ms_warp(top, sc);
            if (OP != LM_DISTILL) xt = warp_sum(lane < L.CL ? xt : 0.f);  // the one slice that has the target gave its logit
        }
        const auto distance = [&](float M) {
            return L.CL > 1 ? ff_sum_or_far(part.distance(M)) : row_distance(a, ex, eq, part, Q, M);
        };
        const auto publish = [&](const RowCoef& k) {
            if (lane == 0) coef = k;
            if (grow) __syncthreads();  // the streaming warps go on while the losses are finished
        };
        row_finish<OP>(a, row, m, r, top, Q, B, xt, sc, rank == 0, publish, distance);
        if (!grow) return;
    } else {
        if (!grow) return;
        __syncthreads();
        slice_grad<DT>(s, coef, grow, a.V, sc, aligned, last, tid, NT);
    }
    __syncthreads();  // the corrections come after the columns they replace
    const RowCoef c = coef;
    if (OP == LM_DISTILL) {
        for (int k = tid; k < a.K; k += NT + 32)
            if (eid[k] >= 0) grow[eid[k]] = Elem<DT>::put(c.fa * c.prob(ex[k], sc) - c.fb * eq[k]);
    } else if (tid == NT && m.tgt >= c0 && m.tgt < c1)
        grow[m.tgt] = Elem<DT>::put(c.fa * c.prob(xt, sc) - c.fb);
}

// Short rows: one warp takes a row, R granules a lane, and keeps them in registers,
// so a row costs one warp's instructions and is read once.
constexpr int SHORT_NW = 8;  // rows of a CTA
constexpr int SHORT_MAX_K = 256;

template <int DT, int OP, int R, bool TAIL>
__global__ void __launch_bounds__(SHORT_NW * 32, R <= 4 ? 4 : R <= 8 ? 3 : 2) lm_short_kernel(const LmRowArgs a) {
    using T = typename Elem<DT>::T;
    constexpr int N = Elem<DT>::N, U = 4;
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ unsigned marks[TAIL ? SHORT_NW : 1][TAIL ? R * 8 : 1];  // a byte a granule
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float sc = SOT_LOG2E / a.tau;
    const long long row = (long long)blockIdx.x * SHORT_NW + warp;
    if (row >= a.T) return;
    float* const ex = reinterpret_cast<float*>(dyn) + (size_t)warp * 3 * a.K;
    float* const eq = ex + a.K;
    int* const eid = reinterpret_cast<int*>(eq + a.K);
    unsigned* const cut = marks[TAIL ? warp : 0];
    const RowMeta m = row_meta<OP>(a, row, true);
    const T* const x = static_cast<const T*>(a.x) + row * a.ld;
    T* const grow = OP != LM_LOGPROB && a.grad ? static_cast<T*>(a.grad) + row * a.ldg : nullptr;
    const bool aligned = same_granules<T>(x, grow);
    const Slice s = slice_at<DT>(x, a.V, 32 * R, 0);
    if (!m.keep) {
        if (grow) slice_zero<DT>(s, grow, a.V, aligned, lane, 32);
        if (lane == 0) row_outputs(a, row, 0.f);
        return;
    }
    const uint64_t policy = policy_drop();
    uint4 v[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int g = lane + 32 * i;
        v[i] = g < s.ng ? load16(s.src + g, policy) : nothing<DT>();
    }
    float2 Q = make_float2(0.f, 0.f), B = Q;
    Part part;
    float xt = 0.f;
    MS top{-INFINITY, 0.f};
    if (OP == LM_DISTILL) {
        teacher_weights(a, teacher_entries<DT, 4>(a, row, s.e0, s.e0 + s.ng * N, x, ex, eq, eid), eq, Q, B);
        if constexpr (TAIL) {
            for (int i = lane; i < R * 8; i += 32) cut[i] = 0u;
            __syncwarp();
            for (int k = lane; k < a.K; k += 32)
                if (eid[k] >= 0) {
                    const int at = eid[k] - s.e0;
                    atomicOr(cut + at / N / 4, 1u << (at / N % 4 * 8 + at % N));
                }
        }
        __syncwarp();
        student_side<DT>(a, s.e0, s.e0 + s.ng * N, x, ex, eq, eid, sc, false, part, top);
    } else
        xt = Elem<DT>::get(x[m.tgt]);
    Running run;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int g = lane + 32 * i;
        if (g < s.ng && (g < s.lo || g >= s.hi)) {
            float2 f[N / 2];
            unpack<DT>(v[i], f);
            mask_cols<DT>(f, s.e0 + g * N, a.V, -INFINITY);
            v[i] = pack<DT>(f);
        }
        if (TAIL && g < s.ng) {
            const unsigned out = reinterpret_cast<const unsigned char*>(cut)[g];
            if (out) v[i] = without<DT>(v[i], out);
        }
    }
#pragma unroll
    for (int i = 0; i < R; i += U)
        if (32 * i < s.ng) {
            const uint4 w[U] = {v[i], v[i + 1], v[i + 2], v[i + 3]};
            run.template add<DT>(w, sc);
        }
    const MS r = ms_warp(run.result(), sc);
    const RowCoef c = row_finish<OP>(a, row, m, r, top, Q, B, xt, sc, true, [](const RowCoef&) {},
                                      [&](float M) { return row_distance(a, ex, eq, part, Q, M); });
    if constexpr (OP != LM_LOGPROB) {
        if (!grow) return;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int g = lane + 32 * i;
            if (g < s.ng) {
                float2 f[N / 2];
                unpack<DT>(v[i], f);
                grad_of<DT>(f, c, sc);
                if (aligned && g >= s.lo && g < s.hi) store16(reinterpret_cast<uint4*>(grow + s.e0) + g, pack<DT>(f), policy);
                else store_cols<DT>(grow, s.e0 + g * N, a.V, f, false);
            }
        }
        __syncwarp();  // the corrections come after the columns they replace
        if (OP == LM_DISTILL) {
            for (int k = lane; k < a.K; k += 32)
                if (eid[k] >= 0) grow[eid[k]] = Elem<DT>::put(c.fa * c.prob(ex[k], sc) - c.fb * eq[k]);
        } else if (lane == 0)
            grow[m.tgt] = Elem<DT>::put(c.fa * c.prob(xt, sc) - c.fb);
    }
}

constexpr int MAX_SMEM = 220 * 1024;  // dynamic shared memory of a CTA
struct LmRowPlan {
    int NW;     // streaming warps of a CTA (0: the short-row kernel)
    int CL, G;  // CTAs a row, granules a slice
    size_t smem;
};

template <int DT, int OP, int NW, bool TAIL>
cudaError_t launch_row_n(const LmRowArgs& a, const LmRowPlan& p, const LmRowLaunch& L, cudaStream_t st) {
    auto kern = lm_row_kernel<DT, OP, NW, TAIL>;
    if (p.smem > 40 * 1024) {  // 48 KB with the static part need no leave
        // The leave belongs to the kernel, not to the call: always the same one, so that a call on
        // another host thread cannot lower it between here and the launch.
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_SMEM);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.T * p.CL), 1, 1);
    cfg.blockDim = dim3((NW + 1) * 32, 1, 1);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.CL;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a, L);
    return e != cudaSuccess ? e : cudaGetLastError();
}
template <int DT, int OP, int NW>
cudaError_t launch_row_k(const LmRowArgs& a, const LmRowPlan& p, const LmRowLaunch& L, cudaStream_t st) {
    if constexpr (OP == LM_DISTILL)
        if (a.tail) return launch_row_n<DT, OP, NW, true>(a, p, L, st);
    return launch_row_n<DT, OP, NW, false>(a, p, L, st);
}

template <int DT, int OP, int R>
cudaError_t launch_row_r(const LmRowArgs& a, const LmRowPlan& p, cudaStream_t st) {
    const unsigned blocks = (unsigned)((a.T + SHORT_NW - 1) / SHORT_NW);
    if constexpr (OP == LM_DISTILL) {
        if (a.tail) {
            lm_short_kernel<DT, OP, R, true><<<blocks, SHORT_NW * 32, p.smem, st>>>(a);
            return cudaGetLastError();
        }
    }
    lm_short_kernel<DT, OP, R, false><<<blocks, SHORT_NW * 32, p.smem, st>>>(a);
    return cudaGetLastError();
}

template <int DT, int OP>
cudaError_t launch_row_o(const LmRowArgs& a, const LmRowPlan& p, const LmRowLaunch& L, cudaStream_t st) {
    switch (p.NW) {
        case 0: return p.G <= 128 ? launch_row_r<DT, OP, 4>(a, p, st)
                       : p.G <= 256 ? launch_row_r<DT, OP, 8>(a, p, st)
                                    : launch_row_r<DT, OP, 16>(a, p, st);
        case 4: return launch_row_k<DT, OP, 4>(a, p, L, st);
        case 8: return launch_row_k<DT, OP, 8>(a, p, L, st);
        default: return launch_row_k<DT, OP, 16>(a, p, L, st);
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
