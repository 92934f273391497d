// topk.cuh -- scores of given tokens with entropies and the best alternatives, over rows of logits.
//
// With y = x / tau and t_v = log2(e) / tau (x_v - m) against the row's largest logit m:
//   S = sum 2^t,  A = sum 2^t t,   lse = m / tau + log S,   entropy = log S - ln 2 A / S,
// both sums of one sign, so neither loses digits to cancellation.  One pass gives them, and
// with them the largest value of every chunk (a thread's batch of granules).  At least K
// chunks have a maximum that is not below the K-th largest chunk maximum, so neither is the row's
// K-th largest logit: only chunks that reach this threshold, about K of them, are read again (from L2) for the
// K best.  The logits are read once: 4096 rows of 131072 bf16 take 156 us with K = 0 (1.02 of the measured copy
// bandwidth).  K = 64 takes 206 (2048 rows and K = 200: 144): a row's selection is a chain of shared-memory steps (threshold,
// second look, order) that ends with its CTA's registers idle, and the rows beside it do not cover all of it.
// The gradient is one pass with the stored lse: 8192 rows of 65536 bf16, a third left out, 270 us (0.97).
#pragma once
#include <cuda_runtime.h>

#include "lm.cuh"
#include "lm_row.cuh"
#include "topk.h"

namespace sot {

struct TopkLaunch {
    int CL, G;     // CTAs a row, granules a slice
    int chunks;    // places for chunk maxima in shared memory
    int cap;       // places for candidates: a power of two, at least 2 K
    int join;      // places for those of all slices, which take the whole of shared memory once they are found
    int bytes;     // of shared memory for a team
};

// Running sums of a thread against the largest logit so far, m: s = sum 2^t and a = sum 2^t t with t = (x - m) sc. The
// difference comes first, so t is good to 2^-23 of itself however far from 0 the logits lie, and the largest
// logit's weight is 1 exactly.
struct Scores {
    float m;
    float2 s, a;
    __device__ __forceinline__ Scores() : m(-INFINITY), s(make_float2(0.f, 0.f)), a(s) {}

    // m becomes the larger of itself and mx.  (Without a branch: lanes that take one go through the sums behind it apart
    // from the others, which doubles the instructions of a batch.)
    __device__ __forceinline__ void move(float mx, float sc) {
        const float M = fmaxf(m, mx), d = M == m ? 0.f : (m - M) * sc, k = ex2f(d);
        // (k = 0: what was summed so far is out of range, and d may be infinite)
        const float2 moved = fmul2(ffma2(s, make_float2(d, d), a), make_float2(k, k));
        a.x = k == 0.f ? 0.f : moved.x;
        a.y = k == 0.f ? 0.f : moved.y;
        s = fmul2(s, make_float2(k, k));
        s.x = M == INFINITY ? NAN : s.x;  // and stays
        m = M;
    }
    // Sums of a granule.  Elements of -inf make a NaN (0 times infinity) of a, which add() looks at.
    template <int DT>
    __device__ __forceinline__ void granule(const uint4& v, float sc) {
        float2 f[Elem<DT>::N / 2];
        unpack<DT>(v, f);
#pragma unroll
        for (int i = 0; i < Elem<DT>::N / 2; ++i) {
            const float2 t = fmul2(fadd2(f[i], make_float2(-m, -m)), make_float2(sc, sc));
            const float2 w = make_float2(ex2f(t.x), ex2f(t.y));
            s = fadd2(s, w);
            a = ffma2(w, t, a);
        }
    }
    __device__ __forceinline__ void one(float x, float sc) {
        if (m == -INFINITY) {  // nothing but -inf so far, and NaN
            s.x += x != x ? x : 0.f;
            return;
        }
        const float t = (x - m) * sc, w = ex2f(t);
        s.x += w;
        if (w > 0.f) a.x = fmaf(w, t, a.x);
    }
    // n granules (of at most P) whose largest element is mx.
    template <int DT, int P>
    __device__ __forceinline__ void add(const uint4 (&v)[P], int n, float mx, float sc) {
        move(mx, sc);
        const float2 s0 = s, a0 = a;
        if (m > -INFINITY) {
            if (n == P) {
#pragma unroll
                for (int j = 0; j < P; ++j) granule<DT>(v[j], sc);
            } else {
#pragma unroll
                for (int j = 0; j < P; ++j)
                    if (j < n) granule<DT>(v[j], sc);
            }
            if (fabsf(a.x + a.y) < INFINITY) return;
            s = s0;
            a = a0;
        }
#pragma unroll
        for (int j = 0; j < P; ++j)
            if (j < n) *this = with_masked<DT>(*this, v[j], sc);
    }
    // A granule that may hold -inf: element by element, 4096 rows of 131072 bf16 with half of the columns at -inf take 416 us
    // (K = 64) instead of 207; with the second half 286, with the last 72 columns 220.  (Out of line: eight copies of it
    // in the loop cost more in fetched instructions than the calls do.)
    template <int DT>
    static __device__ __noinline__ Scores with_masked(Scores r, uint4 v, float sc) {
        float2 f[Elem<DT>::N / 2];
        unpack<DT>(v, f);
#pragma unroll
        for (int i = 0; i < Elem<DT>::N / 2; ++i) {
            r.one(f[i].x, sc);
            r.one(f[i].y, sc);
        }
        return r;
    }
};

struct MSA {
    float m, s, a;
};
// Sums against stabiliser v.m taken to M >= v.m.
__device__ __forceinline__ MSA msa_to(MSA v, float M, float sc) {
    if (v.s != v.s) return MSA{M, v.s, 0.f};
    const float d = (v.m - M) * sc, k = ex2f(d);
    if (v.s == 0.f || !(k > 0.f)) return MSA{M, 0.f, 0.f};
    return MSA{M, v.s * k, fmaf(d, v.s, v.a) * k};
}
__device__ __forceinline__ MSA msa_warp(MSA v, float sc) {
    const float M = warp_max1(v.m);
    v = msa_to(v, M, sc);
    return MSA{M, warp_sum(v.s), warp_sum(v.a)};
}

// Order of the logits as whole numbers (0 and -0 alike), with the bits that a type does not have cut off.
template <int DT>
struct Key {
    static constexpr int SHIFT = DT == SOT_F32 ? 0 : DT == SOT_BF16 ? 16 : 13;
    __device__ static __forceinline__ unsigned of(float x) { return ord_encode(x + 0.f) >> SHIFT; }
    __device__ static __forceinline__ float value(unsigned k) {
        // (the bits cut off are 0 in a positive number's key, 1 in a negative one's)
        const unsigned low = k << SHIFT & 0x80000000u ? 0u : (1u << SHIFT) - 1u;
        return ord_decode(k << SHIFT | low);
    }
    static constexpr unsigned NOTHING = 0x007fffffu >> SHIFT;  // key of -inf
};
// One number for a logit and its column: larger values first, lower columns first among equal ones.
__device__ __forceinline__ unsigned long long pair_of(unsigned key, int col) {
    return (unsigned long long)key << 32 | (unsigned)~col;
}

constexpr int BIN_BITS = 8, BINS = 1 << BIN_BITS;

// What the threads of a CTA share while they select.
template <int NT>
struct SelectSmem {
    unsigned bound[2];  // the range of a threshold
    unsigned count[3];  // counters in turn
    unsigned found;     // candidates
    unsigned hits;      // chunks to look at again
    unsigned best[NT > 32 ? NT : 1];  // the threads' maxima
};

// A team of NT threads takes a row (or a cluster's slice of one): a CTA, or for short rows one of eight warps of a CTA
// (a CTA for each warp would leave an SM with seven of them at a time).
template <int NT>
constexpr int TEAMS = NT == 32 ? 8 : 1;
// Granules of a thread that are under way together; a chunk is as many, or one.  (A warp with a row of its own: four, for more
// warps on an SM: 16384 x 2048 bf16 and K = 8 take 37 us, with eight 43.)
template <int NT>
constexpr int BATCH_OF = NT == 32 ? 4 : 8;
template <int NT>
__device__ __forceinline__ int team_tid() {
    return NT == 32 ? threadIdx.x & 31 : threadIdx.x;
}
template <int NT>
__device__ __forceinline__ void team_sync() {
    if (NT == 32) __syncwarp();
    else __syncthreads();
}

// How many of the team's threads' counts there are in all; step: a running number of such sums.
template <int NT>
__device__ __forceinline__ unsigned team_count(SelectSmem<NT>& sh, unsigned mine, int& step) {
    const unsigned w = __reduce_add_sync(0xffffffffu, mine);
    if (NT == 32) return w;
    const int now = step % 3, next = (step + 1) % 3;
    ++step;
    if ((threadIdx.x & 31) == 0 && w) atomicAdd(&sh.count[now], w);
    // (the next step's: its last readers, two steps ago, have passed the barrier of the last step, and its next writers come
    // behind this one)
    if (threadIdx.x == 0) sh.count[next] = 0;
    __syncthreads();
    return sh.count[now];
}

// Sorts n2 (a power of two) numbers, largest first.
template <int NT>
__device__ __forceinline__ void sort_pairs(unsigned long long* v, int n2) {
    for (int k = 2; k <= n2; k *= 2)
        for (int j = k / 2; j > 0; j /= 2) {
            for (int i = team_tid<NT>(); i < n2 / 2; i += NT) {
                const int p = 2 * i - (i & (j - 1)), q = p + j;
                const unsigned long long x = v[p], y = v[q];
                if ((x < y) == ((p & k) == 0)) {
                    v[p] = y;
                    v[q] = x;
                }
            }
            team_sync<NT>();
        }
}
__device__ __forceinline__ unsigned long long cluster_load64(uint32_t ra) {
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(ra) : "memory");
    return v;
}
// A granule with -inf at the columns outside [0, V).
template <int DT>
__device__ __forceinline__ uint4 inside(const uint4& v, int e, int V) {
    float2 f[Elem<DT>::N / 2];
    unpack<DT>(v, f);
    mask_cols<DT>(f, e, V, -INFINITY);
    return pack<DT>(f);
}

// Calls use(logits, first column) for granule g of a slice (-inf outside the row), or use(logit, column) for its elements.
template <int DT, class Use>
__device__ __forceinline__ void each_granule(const Slice& s, int g, int V, Use use) {
    constexpr int N = Elem<DT>::N;
    uint4 v = s.src[g];
    const int e = s.e0 + g * N;
    if (g < s.lo || g >= s.hi) v = inside<DT>(v, e, V);
    float2 f[N / 2];
    unpack<DT>(v, f);
    float x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = i & 1 ? f[i / 2].y : f[i / 2].x;
    use(x, e);
}
template <int DT, class Use>
__device__ __forceinline__ void each_logit(const Slice& s, int g, int V, Use use) {
    each_granule<DT>(s, g, V, [&](const float (&x)[Elem<DT>::N], int col) {
#pragma unroll
        for (int i = 0; i < Elem<DT>::N; ++i) use(x[i], col + i);
    });
}

// The K largest of the n numbers of v in order, zeros behind them where there are fewer (a 0 among them is a place that a
// slice could not fill).  A few are placed by counting the larger ones of each.  More are first shared out over BINS bins by
// their key's distance from the largest, so that only those of a bin are counted.  (Steps of a
// sorting network were a third of the time: 4096 x 5000 bf16, K = 200 took 100 us with it, 66 like this, and 58 with the
// search in between().)  Where one bin has many, the network does it.
// bins: BINS places; to: n of them.
template <int NT>
__device__ __forceinline__ void order(SelectSmem<NT>& sh, unsigned long long* v, int n, int K, int* bins, unsigned long long* to) {
    constexpr int FEW = 64, PER = FEW > NT ? FEW / NT : 1;
    const int tid = team_tid<NT>(), lane = tid & 31;
    if (n <= FEW) {
        unsigned long long mine[PER];
        int rank[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            mine[j] = j * NT + tid < n ? v[j * NT + tid] : 0ull;
            rank[j] = 0;
        }
        if (PER > 1 || (tid & ~31) < n) {
#pragma unroll 4
            for (int i = 0; i < n; ++i) {
                const unsigned long long x = v[i];
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    if (j * NT < n) rank[j] += x > mine[j];
            }
        }
        team_sync<NT>();
        for (int i = tid; i < K; i += NT) v[i] = 0ull;
        team_sync<NT>();
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (mine[j] && rank[j] < K) v[rank[j]] = mine[j];
        team_sync<NT>();
        return;
    }
    if (tid == 0) {
        sh.bound[0] = 0xffffffffu;
        sh.bound[1] = 0;
    }
    for (int i = tid; i < BINS; i += NT) bins[i] = 0;
    unsigned lo = 0xffffffffu, hi = 0;
    for (int i = tid; i < n; i += NT) {
        const unsigned key = (unsigned)(v[i] >> 32);
        if (key) lo = min(lo, key);
        hi = max(hi, key);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    team_sync<NT>();
    if (NT > 32) {
        if (lane == 0) {
            atomicMin(&sh.bound[0], lo);
            atomicMax(&sh.bound[1], hi);
        }
        __syncthreads();
        lo = sh.bound[0];
        hi = sh.bound[1];
    }
    const int shift = max(0, 32 - __clz(hi - min(lo, hi)) - BIN_BITS);
    const auto bin = [&](unsigned long long x) { return (int)(hi - (unsigned)(x >> 32) >> shift); };
    for (int i = tid; i < n; i += NT)
        if (v[i]) atomicAdd(&bins[bin(v[i])], 1);
    team_sync<NT>();
    // where each bin starts
    if (tid < 32) {
        int count[BINS / 32], all = 0, most = 0;
#pragma unroll
        for (int j = 0; j < BINS / 32; ++j) {
            count[j] = bins[lane * (BINS / 32) + j];
            all += count[j];
            most = max(most, count[j]);
        }
        int before = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int w = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += w;
        }
        if (lane == 31) sh.found = (unsigned)before;
        before -= all;
#pragma unroll
        for (int j = 0; j < BINS / 32; ++j) {
            bins[lane * (BINS / 32) + j] = before;
            before += count[j];
        }
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) sh.hits = (unsigned)most;
    }
    team_sync<NT>();
    if (sh.hits > 64) {
        int n2 = 2;
        while (n2 < n || n2 < K) n2 *= 2;
        for (int i = n + tid; i < n2; i += NT) v[i] = 0ull;
        team_sync<NT>();
        sort_pairs<NT>(v, n2);
        return;
    }
    for (int i = tid; i < n; i += NT) {
        const unsigned long long x = v[i];
        if (x) to[atomicAdd(&bins[bin(x)], 1)] = x;
    }
    team_sync<NT>();
    const int m = (int)sh.found;
    for (int i = tid; i < m; i += NT) {
        const unsigned long long x = to[i];
        const int b = bin(x), end = bins[b];  // (where the bin after it starts, now that its own are placed)
        int r = b ? bins[b - 1] : 0;
        for (int j = r; j < end; ++j) r += to[j] > x;
        if (r < K) v[r] = x;
    }
    for (int i = m + tid; i < K; i += NT) v[i] = 0ull;
    team_sync<NT>();
}

// A key in (lo, hi], of finite values: half of the way in value, or in keys.  (Logits lie evenly in value, where a few steps
// find a threshold; taking turns, no rows need more than twice a key's bits.)
template <int DT>
__device__ __forceinline__ unsigned between(unsigned lo, unsigned hi, bool linear) {
    const float mid = 0.5f * Key<DT>::value(lo) + 0.5f * Key<DT>::value(hi);
    return linear ? min(max(Key<DT>::of(mid), lo + 1), hi) : lo + (hi - lo + 1) / 2;
}

// The largest threshold in [lo, hi] that K of the numbers of a warp reach (lo does), R of them a lane; one that not
// more than `enough` reach will do.
template <int R>
__device__ __forceinline__ unsigned warp_threshold(const unsigned (&key)[R], unsigned lo, unsigned hi, unsigned K, unsigned enough) {
    while (lo < hi) {
        const unsigned mid = lo + (hi - lo + 1) / 2;
        unsigned n = 0;
#pragma unroll
        for (int j = 0; j < R; ++j) n += key[j] >= mid;
        n = R == 1 ? __popc(__ballot_sync(0xffffffffu, n)) : __reduce_add_sync(0xffffffffu, n);
        if (n >= K) lo = mid;
        else hi = mid - 1;
        if (n >= K && n <= enough) break;
    }
    return lo;
}

// The slice's K best (fewer where it has fewer that are not -inf), sorted, in cand; the rest of cand's first
// K places 0.  ckey: the chunks' maxima, chunk c = granules (c / NT * U + j) * NT + c % NT; best: the largest of this thread's.
template <int DT, int NT, int U>
__device__ __forceinline__ void select_best(SelectSmem<NT>& sh, const unsigned* ckey, unsigned best, int C, const Slice& s, int V, int K,
                                            int cap, unsigned long long* cand, int* hit, unsigned long long* spare) {
    constexpr int N = Elem<DT>::N;
    const int tid = team_tid<NT>(), lane = tid & 31;
    const unsigned floor = Key<DT>::NOTHING + 1;
    unsigned at, top;  // a threshold that K logits reach (or all there are); the largest key
    int step = 0;
    // (of 256 threads' maxima the 128th largest would be reached by too many logits)
    constexpr int FROM_THREADS = NT == 256 ? 96 : NT / 2;
    if (K <= FROM_THREADS) {
        // K threads have a logit that reaches the K-th largest of the threads' maxima.
        constexpr int R = NT / 32;
        unsigned key[R] = {best};
        if (NT > 32) {
            sh.best[tid] = best;
            __syncthreads();
            if (tid < 32) {
#pragma unroll
                for (int j = 0; j < R; ++j) key[j] = sh.best[j * 32 + lane];
            }
        }
        if (tid < 32) {
            unsigned lo = 0xffffffffu, hi = 0, n = 0;
#pragma unroll
            for (int j = 0; j < R; ++j) {
                hi = max(hi, key[j]);
                if (key[j] >= floor) {
                    lo = min(lo, key[j]);
                    ++n;
                }
            }
            lo = __reduce_min_sync(0xffffffffu, lo);
            hi = __reduce_max_sync(0xffffffffu, hi);
            n = __reduce_add_sync(0xffffffffu, n);
            at = n < (unsigned)K ? floor : warp_threshold<R>(key, lo, hi, K, K + K / 4 + 4);
            top = max(hi, floor);
            if (lane == 0) {
                sh.bound[0] = at;
                sh.bound[1] = top;
                sh.found = sh.hits = 0;
            }
        }
        team_sync<NT>();
        at = sh.bound[0];
        top = sh.bound[1];
    } else {
        // The same with the chunks' maxima, which are more.
        unsigned lo = 0xffffffffu, hi = 0;
        for (int c = tid; c < C; c += NT) {
            const unsigned k = ckey[c];
            if (k >= floor) lo = min(lo, k);
            hi = max(hi, k);
        }
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if (NT > 32) {
            if (lane == 0) {
                atomicMin(&sh.bound[0], lo);
                atomicMax(&sh.bound[1], hi);
            }
            __syncthreads();
            lo = sh.bound[0];
            hi = sh.bound[1];
        }
        const auto reach = [&](unsigned at) {
            unsigned n = 0;
            for (int c = tid; c < C; c += NT) n += ckey[c] >= at;
            return team_count<NT>(sh, n, step);
        };
        lo = max(lo, floor);
        hi = max(hi, lo);
        top = hi;
        if (C < K || reach(lo) < (unsigned)K) lo = hi = floor;
        for (bool linear = true; lo < hi; linear = !linear) {
            const unsigned mid = between<DT>(lo, hi, linear), n = reach(mid);
            if (n >= (unsigned)K) lo = mid;
            else hi = mid - 1;
            if (n >= (unsigned)K && n <= (unsigned)(K + K / 4)) break;
        }
        at = lo;
        if (tid == 0) sh.found = sh.hits = 0;
        team_sync<NT>();
    }
    // The elements that reach `at` (more than cap of them: only counted).  Their chunks go into a list first, so that the
    // granules to read again are shared out evenly: looked at by the thread that found its chunk, with few
    // lanes of a warp at a time, 4096 rows of 131072 bf16 and K = 64 take 566 us, so 278.
    const auto gather = [&](unsigned at) {
        if (best >= at)
            for (int c = tid; c < C; c += NT)
                if (ckey[c] >= at) {
                    const unsigned i = atomicAdd(&sh.hits, 1u);
                    if (i < (unsigned)cap) hit[i] = c;
                }
        team_sync<NT>();
        const unsigned hits = sh.hits;
        if (hits > (unsigned)cap) return hits;  // each has one at least
        const float least = Key<DT>::value(at);
        for (unsigned i = tid; i < hits * U; i += NT) {
            const int c = hit[i / U], g = c / NT * U * NT + c % NT + (int)(i % U) * NT;
            if (g < s.ng)
                each_granule<DT>(s, g, V, [&](const float (&x)[N], int col) {
                    unsigned on = 0;
#pragma unroll
                    for (int j = 0; j < N; ++j) on |= x[j] >= least ? 1u << j : 0u;
                    if (on == 0) return;
                    unsigned k = atomicAdd(&sh.found, (unsigned)__popc(on));
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        if (on >> j & 1u) {
                            if (k < (unsigned)cap) cand[k] = pair_of(Key<DT>::of(x[j]), col + j);
                            ++k;
                        }
                });
        }
        team_sync<NT>();
        return sh.found;
    };
    // (Where nearly every chunk has a candidate there are more of them than places, which need not be found out.)
    unsigned n = 5ll * K > 4ll * ((s.ng + U - 1) / U) && s.ng > cap / N ? cap + 1u : gather(at);
    if (n > (unsigned)cap) {
        // Many large logits in few chunks, or many equal ones: a threshold that enough of them reach and not too many, by counting
        // over the whole slice.  Where there is none this ends at the K-th largest logit itself: those above it, and as many of
        // those equal to it as are missing, lowest columns first.
        const auto above = [&](unsigned at) {
            const float least = Key<DT>::value(at);
            unsigned n = 0;
            for (int g = tid; g < s.ng; g += NT) each_logit<DT>(s, g, V, [&](float x, int) { n += x >= least; });
            return team_count<NT>(sh, n, step);
        };
        for (bool linear = true; at < top && n > (unsigned)cap; linear = !linear) {
            const unsigned mid = between<DT>(at, top, linear), reached = above(mid);
            if (reached >= (unsigned)K) at = mid, n = reached;
            else top = mid - 1;
        }
        const bool ties = n > (unsigned)cap;
        team_sync<NT>();
        if (tid == 0) sh.found = sh.hits = 0;
        team_sync<NT>();
        n = min(gather(ties ? at + 1 : at), (unsigned)cap);  // (of ties: fewer than K)
        const float tie = Key<DT>::value(at);
        for (int g0 = 0; ties && g0 < s.ng && n < (unsigned)K; g0 += NT) {
            const int g = g0 + tid;
            unsigned mine = 0;
            if (g < s.ng) each_logit<DT>(s, g, V, [&](float x, int) { mine += x == tie; });
            unsigned before = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned w = __shfl_up_sync(0xffffffffu, before, o);
                if (lane >= o) before += w;
            }
            unsigned all = __shfl_sync(0xffffffffu, before, 31), place = n + before - mine;
            if (NT > 32) {
                __syncthreads();
                if (lane == 31) sh.best[tid >> 5] = before;
                __syncthreads();
                all = 0;
                for (int w = 0; w < NT / 32; ++w) {
                    if (w < tid >> 5) place += sh.best[w];
                    all += sh.best[w];
                }
            }
            if (mine)
                each_logit<DT>(s, g, V, [&](float x, int col) {
                    if (x == tie && place++ < (unsigned)K) cand[place - 1] = pair_of(at, col);
                });
            n = min(n + all, (unsigned)K);
        }
        team_sync<NT>();
    }
    order<NT>(sh, cand, n, K, hit, spare);
}

// A row a team, or a cluster's CTAs a slice of it each.
template <int DT, int NT, int U>
__global__ void __launch_bounds__(NT * TEAMS<NT>, NT == 32 ? 4 : 1024 / NT) topk_kernel(const TopkArgs a, const TopkLaunch L) {
    using T = typename Elem<DT>::T;
    constexpr int N = Elem<DT>::N, P = BATCH_OF<NT>, NW = NT / 32;
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ SelectSmem<NT> select[TEAMS<NT>];
    __shared__ MSA rec[NW];
    __shared__ MSA mail[ROW_MAX_CL];
    const int tid = team_tid<NT>(), lane = tid & 31, warp = tid >> 5, team = threadIdx.x / NT;
    SelectSmem<NT>& sh = select[team];
    unsigned long long* const cand = reinterpret_cast<unsigned long long*>(dyn + (NT == 32 ? team * L.bytes : 0));
    int* const hit = reinterpret_cast<int*>(cand + L.cap);
    unsigned* const ckey = reinterpret_cast<unsigned*>(hit + L.cap);
    unsigned long long* const spare = reinterpret_cast<unsigned long long*>(ckey);  // once the chunks have been looked at
    const uint32_t rank = NT == 32 ? 0 : cluster_rank();
    const float sc = SOT_LOG2E / a.tau;
    const long long row = NT == 32 ? (long long)blockIdx.x * TEAMS<NT> + team : blockIdx.x / L.CL;
    if (NT == 32 && row >= a.T) return;
    const int tgt = a.target ? load_index(a.target, a.target_type, row, a.V) : -1;
    if (a.target && tgt < 0) {  // left out: the same for the whole cluster
        if (rank) return;
        for (int k = tid; k < a.K; k += NT) {
            if (a.ids) a.ids[row * a.K + k] = -1;
            if (a.top) a.top[row * a.K + k] = 0.f;
        }
        if (tid == 0) {
            if (a.logp) a.logp[row] = 0.f;
            if (a.lse) a.lse[row] = 0.f;
            if (a.entropy) a.entropy[row] = 0.f;
        }
        return;
    }
    if (NT > 32 && L.CL > 1) cluster_arrive_started();
    const T* const x = static_cast<const T*>(a.x) + row * a.ld;
    const Slice s = slice_at<DT>(x, a.V, L.G, rank);
    const float xt = tgt >= 0 && rank == 0 && tid == 0 ? Elem<DT>::get(x[tgt]) : 0.f;
    const uint64_t policy = a.K ? policy_keep() : policy_drop();
    if (NT > 32 && tid == 0) {
        sh.bound[0] = 0xffffffffu;
        sh.bound[1] = 0;
        sh.count[0] = sh.count[1] = sh.count[2] = 0;
    }
    Scores run;
    int c = tid;  // the next chunk
    for (int g = tid; g < s.ng; g += P * NT) {
        uint4 v[P];
        const int n = min(P, (s.ng - g + NT - 1) / NT);
        if (n == P) {
#pragma unroll
            for (int j = 0; j < P; ++j) v[j] = load16(s.src + g + j * NT, policy);
        } else {
#pragma unroll
            for (int j = 0; j < P; ++j) v[j] = j < n ? load16(s.src + g + j * NT, policy) : nothing<DT>();
        }
        if (s.lo > 0 && g == 0) v[0] = inside<DT>(v[0], s.e0, a.V);
        if (s.hi < s.ng) {
#pragma unroll
            for (int j = 0; j < P; ++j)
                if (g + j * NT == s.ng - 1) v[j] = inside<DT>(v[j], s.e0 + (s.ng - 1) * N, a.V);
        }
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < P; j += U) {
            uint4 top = v[j];
#pragma unroll
            for (int i = 1; i < U; ++i) top = max2<DT>(top, v[j + i]);
            const float w = max_of<DT>(top);
            mx = fmaxf(mx, w);
            if (a.K) {
                if (j < n) ckey[c] = Key<DT>::of(w);  // (a key of -inf where all are)
                c += NT;
            }
        }
        run.template add<DT>(v, n, mx, sc);
    }
    MSA w = msa_warp(MSA{run.m, run.s.x + run.s.y, run.a.x + run.a.y}, sc);
    if (NT > 32 && lane == 0) rec[warp] = w;
    const int chunks = min((s.ng + U * NT - 1) / (U * NT) * NT, L.chunks);
    if (a.K)  // places that no chunk has taken
        for (int i = tid; i < chunks; i += NT)
            if (i / NT * U * NT + tid >= s.ng) ckey[i] = 0;
    team_sync<NT>();
    if (NT > 32) {
        w = rec[lane < NW ? lane : 0];
        if (lane >= NW) w = MSA{-INFINITY, 0.f, 0.f};
        w = msa_warp(w, sc);
    }
    // A row without a sum has no alternatives; a slice without one may still stand beside others.
    if (a.K) {
        if (w.s > 0.f) select_best<DT, NT, U>(sh, ckey, Key<DT>::of(run.m), chunks, s, a.V, a.K, L.cap, cand, hit, spare);
        else
            for (int i = tid; i < a.K; i += NT) cand[i] = 0ull;
        team_sync<NT>();
    }
    if (NT > 32 && L.CL > 1) {
        cluster_wait_started();
        if (tid == 0) {
            const uint32_t to = cluster_addr(smem_u32(&mail[rank]), 0);
            cluster_store(to, w.m);
            cluster_store(to + 4, w.s);
            cluster_store(to + 8, w.a);
        }
        cluster_sync();
        if (rank == 0) {
            w = lane < L.CL ? mail[lane] : MSA{-INFINITY, 0.f, 0.f};
            w = msa_warp(w, sc);
            if (a.K) {
                for (int i = a.K + tid; i < L.CL * a.K; i += NT) {
                    const uint32_t r = i / a.K;
                    cand[i] = cluster_load64(cluster_addr(smem_u32(cand + (i - r * a.K)), r));
                }
                __syncthreads();
                int* const bins = reinterpret_cast<int*>(cand + L.join);
                order<NT>(sh, cand, L.CL * a.K, a.K, bins, reinterpret_cast<unsigned long long*>(bins + BINS));
            }
        }
        cluster_sync();  // nobody leaves while rank 0 reads
        if (rank) return;
    }
    const float2 logS = log_ff(w.s);
    // log p of a logit: the difference to the stabiliser is exact, only what comes after it is rounded.
    const auto logp_of = [&](float v) {
        const float2 d = two_sum(v, -w.m);
        const float2 r = ff_add(ff_mul(d, make_float2(a.inv_hi, a.inv_lo)), make_float2(-logS.x, -logS.y));
        return fabsf(r.x) < INFINITY ? r.x + r.y : (float)(((double)v - (double)w.m) * a.inv_tau) - logS.x;
    };
    if (tid == 0) {
        if (a.logp) a.logp[row] = logp_of(xt);
        if (a.lse) {
            const float2 l = ff_add(ff_mul(make_float2(w.m, 0.f), make_float2(a.inv_hi, a.inv_lo)), logS);
            a.lse[row] = fabsf(l.x) < INFINITY ? l.x + l.y : (float)((double)w.m * a.inv_tau) + logS.x;
        }
        if (a.entropy) {
            const float h = logS.x + fmaf(-SOT_LN2, __fdiv_rn(w.a, w.s), logS.y);
            a.entropy[row] = w.s > 0.f ? (h < 0.f ? 0.f : h) : NAN;
        }
    }
    for (int k = tid; k < a.K; k += NT) {
        const unsigned long long p = w.s > 0.f ? cand[k] : 0ull;
        if (a.ids) a.ids[row * a.K + k] = p ? (int)~(unsigned)p : -1;
        if (a.top) a.top[row * a.K + k] = p ? logp_of(Key<DT>::value((unsigned)(p >> 32))) : w.s > 0.f ? -INFINITY : NAN;
    }
}

// Gradient from the stored lse and entropy: with G = sum of the gradients with respect to
// log-probabilities, those of the entries and of the target, and t = log2 p,
//   tau dx_v = G_v - p_v (G + gH (ln 2 t_v + H)) = G_v + p_v (c0 + c1 t_v).
// One read and one write per logit, each granule on its own.  The entries' columns are
// formed again after the rest, from logits read before anything is written.
// A CTA of NT threads takes G granules of a row.
template <int DT, int NT>
__global__ void __launch_bounds__(NT, 1536 / NT) topk_grad_kernel(const TopkGradArgs a, int G, int chunks) {
    using T = typename Elem<DT>::T;
    constexpr int N = Elem<DT>::N, U = 4;
    extern __shared__ __align__(16) float ent[];  // entries of the slice: logit
    __shared__ float red[NT / 32];
    const int tid = threadIdx.x;
    const long long row = blockIdx.x / chunks;
    const T* const x = static_cast<const T*>(a.x) + row * a.ld;
    T* const grow = static_cast<T*>(a.grad) + row * a.ldg;
    const Slice s = slice_at<DT>(x, a.V, G, blockIdx.x % chunks);
    const bool aligned = same_granules<T>(x, grow);
    // (the row's values are fetched together, whether they turn out to count or not: one wait instead of three)
    const float lse = a.lse[row], row_gl = a.g_logp ? a.g_logp[row] : 0.f, row_gh = a.g_entropy ? a.g_entropy[row] : 0.f;
    const float row_h = a.g_entropy ? a.entropy[row] : 0.f;
    const int tgt = a.target ? load_index(a.target, a.target_type, row, a.V) : -1;
    const bool keep = !a.target || tgt >= 0;
    const float inv_tau = 1.f / a.tau;
    const float gl = tgt >= 0 ? row_gl : 0.f, gh = keep ? row_gh : 0.f;
    float gt = 0.f;
    bool any = gl != 0.f || gh != 0.f;
    const int e0 = s.e0, e1 = s.e0 + s.ng * N;  // the slice's columns
    if (keep && a.g_top) {
        float mine = 0.f;
        bool some = false;
        for (int k = tid; k < a.K; k += NT) {
            const int id = a.ids[row * a.K + k];
            const float g = id >= 0 && id < a.V ? a.g_top[row * a.K + k] : 0.f;
            mine += g;
            some = some || g != 0.f;
            if (id >= e0 && id < e1 && id >= 0 && id < a.V) ent[k] = Elem<DT>::get(x[id]);
        }
        gt = block_sum<NT>(mine, red);
        any = __syncthreads_or(some) || any;
    }
    if (!any) {  // not read
        slice_zero<DT>(s, grow, a.V, aligned, tid, NT);
        return;
    }
    const float u = lse * SOT_LOG2E, sc = SOT_LOG2E / a.tau;
    const float H = gh != 0.f ? row_h : 0.f;
    // (a row without a lse has no gradient: NaN)
    const float c0 = -(gl + gt + gh * H) * inv_tau + (lse - lse), c1 = -gh * SOT_LN2 * inv_tau;
    const bool far = !(fabsf(u) < 0x1p10f);
    // p (c0 + c1 t).  Below 2^-160 p is 0, whatever t is.
    const auto near2 = [&](float2 f) {
        const float2 t = ffma2(f, make_float2(sc, sc), make_float2(-u, -u));
        const float2 b = make_float2(fmaxf(t.x, -160.f), fmaxf(t.y, -160.f));
        const float2 p = make_float2(ex2f(t.x), ex2f(t.y));
        return fmul2(p, ffma2(b, make_float2(c1, c1), make_float2(c0, c0)));
    };
    // Far from 0 the rounding of u would show: the difference comes first there.
    const auto far1 = [&](float v) {
        float d = (v - lse * a.tau) / a.tau;
        d = d > 0.f ? 0.f : d;
        const float p = expf(d);
        return p * fmaf(c1, fmaxf(d * SOT_LOG2E, -160.f), c0);
    };
    const auto value = [&](float2 f) { return far ? make_float2(far1(f.x), far1(f.y)) : near2(f); };
    const float hot = gl * inv_tau;
    const auto finish = [&](float2 (&f)[N / 2], int c) {  // columns c ..
#pragma unroll
        for (int j = 0; j < N / 2; ++j) f[j] = value(f[j]);
        if ((unsigned)(tgt - c) < (unsigned)N && tgt >= 0) {
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                f[j].x += c + 2 * j == tgt ? hot : 0.f;
                f[j].y += c + 2 * j + 1 == tgt ? hot : 0.f;
            }
        }
    };
    const uint64_t policy = policy_drop();
    if (!aligned) {
        for (int i = tid; i < s.ng; i += NT) {
            float2 f[N / 2];
            unpack<DT>(s.src[i], f);
            finish(f, s.e0 + i * N);
            store_cols<DT>(grow, s.e0 + i * N, a.V, f, false);
        }
    } else {
        uint4* const dst = reinterpret_cast<uint4*>(grow + s.e0);
        for (int i = s.lo + tid; i < s.hi; i += U * NT) {
            uint4 v[U];
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (i + j * NT < s.hi) v[j] = load16(s.src + i + j * NT, policy);
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (i + j * NT < s.hi) {
                    float2 f[N / 2];
                    unpack<DT>(v[j], f);
                    finish(f, s.e0 + (i + j * NT) * N);
                    store16(dst + i + j * NT, pack<DT>(f), policy);
                }
        }
        const int e = edge_granule(s, tid, NT);
        if (e >= 0) {
            float2 f[N / 2];
            unpack<DT>(s.src[e], f);
            finish(f, s.e0 + e * N);
            store_cols<DT>(grow, s.e0 + e * N, a.V, f, false);
        }
    }
    if (!a.g_top) return;
    __syncthreads();  // the entries come after the columns they replace
    for (int k = tid; k < a.K; k += NT) {
        const int id = a.ids[row * a.K + k];
        if (id >= e0 && id < e1 && id >= 0 && id < a.V) {
            const float g = a.g_top[row * a.K + k] + (id == tgt ? gl : 0.f);
            grow[id] = Elem<DT>::put(fmaf(g, inv_tau, value(make_float2(ent[k], ent[k])).x));
        }
    }
}

constexpr int TOPK_MAX_SMEM = 200 * 1024;

template <int DT, int NT, int U>
cudaError_t launch_topk_n(const TopkArgs& a, const TopkLaunch& L, cudaStream_t st) {
    auto kern = topk_kernel<DT, NT, U>;
    const size_t smem = (size_t)L.bytes * TEAMS<NT>;
    if (smem > 40 * 1024) {
        // (the kernel's leave, not the call's: another host thread's call cannot lower it before the launch)
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, TOPK_MAX_SMEM);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.T + TEAMS<NT> - 1) / TEAMS<NT> * L.CL), 1, 1);
    cfg.blockDim = dim3(NT * TEAMS<NT>, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = L.CL;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a, L);
    return e != cudaSuccess ? e : cudaGetLastError();
}

struct TopkPlan {
    int NT, U;
    TopkLaunch L;
};

template <int DT, int NT>
cudaError_t launch_topk_u(const TopkArgs& a, const TopkPlan& p, cudaStream_t st) {
    return p.U == 1 ? launch_topk_n<DT, NT, 1>(a, p.L, st) : launch_topk_n<DT, NT, BATCH_OF<NT>>(a, p.L, st);
}
template <int DT>
cudaError_t launch_topk_t(const TopkArgs& a, const TopkPlan& p, cudaStream_t st) {
    return p.NT == 32 ? launch_topk_u<DT, 32>(a, p, st) : p.NT == 128 ? launch_topk_u<DT, 128>(a, p, st) : launch_topk_u<DT, 256>(a, p, st);
}

template <int DT>
cudaError_t launch_topk_grad_t(const TopkGradArgs& a, int NT, int G, int chunks, cudaStream_t st) {
    const unsigned blocks = (unsigned)(a.T * chunks);
    const size_t smem = a.g_top ? a.K * sizeof(float) : 0;
    if (NT == 64) topk_grad_kernel<DT, 64><<<blocks, 64, smem, st>>>(a, G, chunks);
    else topk_grad_kernel<DT, 256><<<blocks, 256, smem, st>>>(a, G, chunks);
    return cudaGetLastError();
}

// One translation unit per type (k_topk_f32.cu, k_topk_f16.cu, k_topk_bf16.cu).
cudaError_t launch_topk_f32(const TopkArgs& a, const TopkPlan& p, cudaStream_t st);
cudaError_t launch_topk_f16(const TopkArgs& a, const TopkPlan& p, cudaStream_t st);
cudaError_t launch_topk_bf16(const TopkArgs& a, const TopkPlan& p, cudaStream_t st);
cudaError_t launch_topk_grad_f32(const TopkGradArgs& a, int NT, int G, int chunks, cudaStream_t st);
cudaError_t launch_topk_grad_f16(const TopkGradArgs& a, int NT, int G, int chunks, cudaStream_t st);
cudaError_t launch_topk_grad_bf16(const TopkGradArgs& a, int NT, int G, int chunks, cudaStream_t st);

}  // namespace sot
