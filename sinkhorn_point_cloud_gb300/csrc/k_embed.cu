// k_embed.cu -- embedding lookup with scaling, and its gradient by sorted tokens.
//
// Lookup: out[t] = scale table[id[t]], a copy of rows with one rounding: memory-bound.
//
// Gradient: grad[v] = scale sum of g[t] over the tokens t with id[t] = v, in the order of t.
//   sort     one cluster sorts the tokens by row, stably (radix passes over shared-memory
//            counts, joined through distributed shared memory), and marks the rows that tokens name; the other CTAs of
//            the launch fill the time with zeros for the table's first rows;
//   sum      a CTA takes a chunk of sorted tokens and a tile of columns, and writes
//            the rows that begin in its chunk and end there or in the next one.  A row that spans more leaves a partial sum in
//            each chunk.  Other CTAs, in between, write the zeros of the remaining rows that no token names (reads and
//            writes at the same time: writes alone reach 0.8 of the copy bandwidth);
//   join     adds up the partial sums, in a fixed order.
// No atomics on floats: repeated calls give the same bits.
//
// bf16, 4096 columns: 32768 lookups in fp32 77 us (0.80 of the measured copy bandwidth), 16384 tokens into 131072 rows 205 us
// (0.87; most of it is zeros).  65001 tokens of 1001 fp32 columns into 32003 rows 124 us (0.43; 100 us with 1000 columns,
// which need no cutting).
#include <cuda_runtime.h>

#include "embed.h"
#include "kernels.h"
#include "lm.cuh"

namespace sot {

namespace {

// Eight elements, one or two granules, as floats.
template <int DT>
__device__ __forceinline__ void floats_of(const uint4 (&v)[DT == SOT_F32 ? 2 : 1], float2 (&f)[4]) {
    if constexpr (DT == SOT_F32) {
        float2 h[2];
        unpack<DT>(v[0], h);
        f[0] = h[0];
        f[1] = h[1];
        unpack<DT>(v[1], h);
        f[2] = h[0];
        f[3] = h[1];
    } else
        unpack<DT>(v[0], f);
}
template <int DT>
__device__ __forceinline__ void store8(typename Elem<DT>::T* p, const float2 (&f)[4], uint64_t policy) {
    uint4* const q = reinterpret_cast<uint4*>(p);
    if constexpr (DT == SOT_F32) {
        const float2 h[2] = {f[0], f[1]}, g[2] = {f[2], f[3]};
        store16(q, pack<DT>(h), policy);
        store16(q + 1, pack<DT>(g), policy);
    } else
        store16(q, pack<DT>(f), policy);
}

// U indices, `step` apart from i on (the last one where i goes past n).  All loads go out before the first value is looked at: a
// branch on one of them between two loads would wait for it.
template <int U, class I>
__device__ __forceinline__ void load_some(const I* p, long long i, int step, long long n, I (&v)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = __ldg(p + min(i + (long long)u * step, n - 1));
}
template <int U>
__device__ __forceinline__ void load_indices(const void* ids, int type, long long i, int step, long long n, int V, int (&id)[U]) {
    if (type == SOT_I64) {
        long long v[U];
        load_some<U>(static_cast<const long long*>(ids), i, step, n, v);
#pragma unroll
        for (int u = 0; u < U; ++u) id[u] = v[u] >= 0 && v[u] < V ? (int)v[u] : -1;
    } else {
        int v[U];
        load_some<U>(static_cast<const int*>(ids), i, step, n, v);
#pragma unroll
        for (int u = 0; u < U; ++u) id[u] = v[u] >= 0 && v[u] < V ? v[u] : -1;
    }
}

// ---- lookup ----
constexpr int EMB_NT = 256, EMB_W = 8;
template <bool VEC>
constexpr int EMB_PIECES = VEC ? 4 : 2;

// The elements from byte `from` on of G granules in a row, G - 1 granules of them.
template <int DT, int G>
__device__ __forceinline__ void cut_out(const uint4 (&v)[G], unsigned from, uint4 (&out)[G - 1]) {
    unsigned w[4 * G];
#pragma unroll
    for (int i = 0; i < G; ++i) w[4 * i] = v[i].x, w[4 * i + 1] = v[i].y, w[4 * i + 2] = v[i].z, w[4 * i + 3] = v[i].w;
#pragma unroll
    for (int k = 2; k > 0; k /= 2) {
        const bool on = from & 4u * k;
#pragma unroll
        for (int i = 0; i + k < 4 * G; ++i) w[i] = on ? w[i + k] : w[i];
    }
    if constexpr (DT != SOT_F32) {
#pragma unroll
        for (int i = 0; i < 4 * (G - 1); ++i) w[i] = __funnelshift_r(w[i], w[i + 1], from % 4 * 8);
    }
#pragma unroll
    for (int i = 0; i < G - 1; ++i) out[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

// A thread takes U pieces of a tile of NT U pieces, eight columns each.  Where rows of table or output are not
// whole granules (VEC = false), a piece begins at a granule of the output, its columns are cut out of the table's granules
// that hold them, and a row's first and last piece are written by elements (20000 rows of 1003 bf16: 19 us, an element a
// thread 47).
template <int DT, int DO, bool VEC>
__global__ void __launch_bounds__(EMB_NT) embed_kernel(const EmbedArgs a, unsigned per_row) {
    using T = typename Elem<DT>::T;
    using O = typename Elem<DO>::T;
    constexpr int R = DT == SOT_F32 ? 2 : 1, EMB_U = EMB_PIECES<VEC>;  // granules of a piece of the table
    constexpr long long NONE = -1ll << 62;
    const long long total = a.T * per_row, tile = (long long)EMB_NT * EMB_U;
    const uint64_t keep = policy_keep(), drop = policy_drop();
    for (long long base = blockIdx.x * tile; base < total; base += gridDim.x * tile) {
        // (one division in 64 bits for a tile, the others in 32)
        const long long row0 = base / per_row;
        const unsigned first = (unsigned)(base - row0 * per_row), left = (unsigned)min(tile, total - base);
        uint4 raw[EMB_U][VEC ? R : R + 1];
        long long to[EMB_U];
        int id[EMB_U], col[EMB_U];
        {
            long long t[EMB_U];
            long long wide[EMB_U];
            int narrow[EMB_U];
#pragma unroll
            for (int j = 0; j < EMB_U; ++j) {  // (a piece past the end is the tile's first one again, and is not written)
                const unsigned i = j * EMB_NT + threadIdx.x, at = first + (i < left ? i : 0u), r = at / per_row;
                col[j] = (int)(at - r * per_row) * EMB_W;
                t[j] = row0 + r;
                const long long row = t[j] * a.ldo;
                if (!VEC) col[j] -= (int)((unsigned long long)(static_cast<O*>(a.out) + row) & 15) / (int)sizeof(O);
                to[j] = i < left && (VEC || col[j] < a.D) ? row + col[j] : NONE;
            }
            if (a.ids_type == SOT_I64) {
#pragma unroll
                for (int j = 0; j < EMB_U; ++j) wide[j] = __ldg(static_cast<const long long*>(a.ids) + t[j]);
#pragma unroll
                for (int j = 0; j < EMB_U; ++j) id[j] = wide[j] >= 0 && wide[j] < a.V ? (int)wide[j] : -1;
            } else {
#pragma unroll
                for (int j = 0; j < EMB_U; ++j) narrow[j] = __ldg(static_cast<const int*>(a.ids) + t[j]);
#pragma unroll
                for (int j = 0; j < EMB_U; ++j) id[j] = narrow[j] >= 0 && narrow[j] < a.V ? narrow[j] : -1;
            }
        }
        // (rows of frequent tokens stay in L2, what is written does not)
        const auto row_of = [&](int j) { return static_cast<const T*>(a.table) + (long long)max(id[j], 0) * a.ld; };
#pragma unroll
        for (int j = 0; j < EMB_U; ++j) {  // (a row for a token without one too: a branch would wait)
            if constexpr (VEC) {
#pragma unroll
                for (int i = 0; i < R; ++i) raw[j][i] = load16(reinterpret_cast<const uint4*>(row_of(j) + col[j]) + i, keep);
            } else {
                // the granules from the one with the piece's first column on, none that holds nothing of the row
                const T* const row = row_of(j);
                const unsigned long long lo = (unsigned long long)row & ~15ull, hi = (unsigned long long)(row + a.D - 1) & ~15ull;
                const unsigned long long at = (unsigned long long)(row + col[j]) & ~15ull;
#pragma unroll
                for (int i = 0; i <= R; ++i) raw[j][i] = load16(reinterpret_cast<const uint4*>(min(max(at + 16 * i, lo), hi)), keep);
            }
        }
#pragma unroll
        for (int j = 0; j < EMB_U; ++j)
            if (to[j] != NONE) {
                O* const out = static_cast<O*>(a.out) + to[j];
                float2 f[4];
                if constexpr (VEC) floats_of<DT>(raw[j], f);
                else {
                    uint4 v[R];
                    cut_out<DT>(raw[j], (unsigned)(unsigned long long)(row_of(j) + col[j]) & 15u, v);
                    floats_of<DT>(v, f);
                }
#pragma unroll
                for (int w = 0; w < 4; ++w) f[w] = id[j] >= 0 ? make_float2(f[w].x * a.scale, f[w].y * a.scale) : make_float2(0.f, 0.f);
                if (VEC || (col[j] >= 0 && col[j] + EMB_W <= a.D)) store8<DO>(out, f, drop);
                else {
#pragma unroll
                    for (int w = 0; w < EMB_W; ++w)
                        if (col[j] + w >= 0 && col[j] + w < a.D) out[w] = Elem<DO>::put(w & 1 ? f[w / 2].y : f[w / 2].x);
                }
            }
    }
}

// ---- gradient: sort ----
constexpr int SORT_NT = 1024, SORT_NW = SORT_NT / 32, SORT_CL = 8, SORT_MAX_BITS = 9, SORT_MAX_BINS = 1 << SORT_MAX_BITS, SORT_U = 8;

struct SortSmem {
    unsigned at[SORT_NW][SORT_MAX_BINS];  // per warp: counts, then places within the CTA's
    unsigned total[SORT_MAX_BINS];        // of this CTA
    unsigned start[SORT_MAX_BINS];        // place of a bin's first token among this CTA's
    unsigned base[SORT_MAX_BINS];         // from there to its place among all
    uint2 sums[SORT_NW];
    // a warp's batch of tokens: row, place, and rank among those of its digit in the warp
    alignas(8) unsigned key[SORT_NW][32 * SORT_U];
    unsigned pos[SORT_NW][32 * SORT_U];
    unsigned order[SORT_NW][32 * SORT_U];
};

// The lanes of a warp with the same digit, from a vote for each of its bits.  `in`: lanes that have one.
__device__ __forceinline__ unsigned same_digit(unsigned digit, bool in) {
    unsigned peers = __ballot_sync(0xffffffffu, in);
#pragma unroll
    for (int b = 0; b < SORT_MAX_BITS; ++b) {
        const unsigned set = __ballot_sync(0xffffffffu, digit >> b & 1u);
        peers &= digit >> b & 1u ? set : ~set;
    }
    return peers;
}

// The code runs once from end to end, so most of what it costs is fetching its instructions: loops stay loops, with a
// warp's batch of tokens in shared memory.
__device__ void sort_tokens(const EmbedGradArgs& a, int passes, int bits, SortSmem& sm) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();
    const int bins = 1 << bits;
    // a warp's share: contiguous, whole steps of 32
    const unsigned workers = SORT_CL * SORT_NW, T = (unsigned)a.T, steps = (T + 31) / 32, per = (steps + workers - 1) / workers * 32;
    const unsigned begin = min(T, (rank * SORT_NW + warp) * per), end = min(T, begin + per);
    unsigned *const key = sm.key[warp], *const pos = sm.pos[warp], *const at = sm.at[warp];
    unsigned* const order = sm.order[warp];
    if (a.named)
#pragma unroll 1
        for (int i = (int)rank * SORT_NT + tid; i < (a.V + 31) / 32; i += SORT_CL * SORT_NT) a.named[i] = 0u;
#pragma unroll 1
    for (int p = 0; p < passes; ++p) {
        // (the last pass writes to buffer 0)
        const bool odd = (passes - 1 - p) & 1;
        const uint2* const in = odd ? a.sorted[0] : a.sorted[1];
        uint2* const out = odd ? a.sorted[1] : a.sorted[0];
        const int shift = p * bits;
        // A batch of tokens: counts, and each token's rank among those of its digit in the warp so far.
        const auto count = [&](unsigned t0) {
            if (p == 0) {
                int id[SORT_U];
                load_indices<SORT_U>(a.ids, a.ids_type, t0 + lane, 32, T, a.V, id);
#pragma unroll
                for (int u = 0; u < SORT_U; ++u) {  // tokens without a row come last
                    key[u * 32 + lane] = id[u] < 0 ? (unsigned)a.V : (unsigned)id[u];
                    pos[u * 32 + lane] = t0 + u * 32 + lane;
                }
            } else {
                uint2 v[SORT_U];
#pragma unroll
                for (int u = 0; u < SORT_U; ++u) v[u] = __ldcg(in + min(t0 + u * 32 + lane, T - 1));
#pragma unroll
                for (int u = 0; u < SORT_U; ++u) {
                    key[u * 32 + lane] = v[u].x;
                    pos[u * 32 + lane] = v[u].y;
                }
            }
#pragma unroll 1
            for (unsigned i = lane; t0 + i - lane < end && i < 32 * SORT_U; i += 32) {
                const bool in = t0 + i < end;
                const unsigned d = key[i] >> shift & (bins - 1), peers = same_digit(d, in);
                const unsigned before = in ? at[d] : 0u;
                order[i] = before + __popc(peers & ((1u << lane) - 1u));
                __syncwarp();
                if (in && lane == __ffs(peers) - 1) at[d] = before + __popc(peers);
                __syncwarp();
            }
        };
        for (int b = lane; b < bins; b += 32) at[b] = 0;
        __syncwarp();
        // A share of one batch (65536 tokens in all) keeps its ranks; a longer one is counted here and again below.
        const bool once = per <= 32 * SORT_U;
#pragma unroll 1
        for (unsigned t0 = begin; t0 < end; t0 += 32 * SORT_U) count(t0);
        __syncthreads();
        unsigned mine = 0;  // this CTA's count of bin tid
        if (tid < bins) {
#pragma unroll 8
            for (int w = 0; w < SORT_NW; ++w) {
                const unsigned c = sm.at[w][tid];
                sm.at[w][tid] = mine;
                mine += c;
            }
            sm.total[tid] = mine;
        }
        cluster_sync();
        unsigned all = 0, before = 0;
        if (tid < bins)
#pragma unroll
            for (uint32_t r = 0; r < SORT_CL; ++r) {
                unsigned c;
                asm volatile("ld.shared::cluster.u32 %0, [%1];"
                             : "=r"(c)
                             : "r"(cluster_addr(smem_u32(&sm.total[tid]), r))
                             : "memory");
                if (r < rank) before += c;
                all += c;
            }
        unsigned scan = all, own = mine;  // inclusive over the bins: of the cluster, of this CTA
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned v = __shfl_up_sync(0xffffffffu, scan, o), w = __shfl_up_sync(0xffffffffu, own, o);
            if (lane >= o) {
                scan += v;
                own += w;
            }
        }
        if (lane == 31) sm.sums[warp] = make_uint2(scan, own);
        __syncthreads();
        const uint2 sums = lane < warp ? sm.sums[lane] : make_uint2(0u, 0u);
        const unsigned base = __reduce_add_sync(0xffffffffu, sums.x) + scan - all + before;
        const unsigned start = __reduce_add_sync(0xffffffffu, sums.y) + own - mine;
        if (tid < bins) {
            sm.base[tid] = base - start;
            sm.start[tid] = start;
        }
        __syncthreads();
        const auto write = [&](unsigned to, uint2 v) {
            out[to] = v;
            if (p == passes - 1 && a.named && v.x < (unsigned)a.V) atomicOr(a.named + v.x / 32, 1u << v.x % 32);
        };
        if (once) {
            // The CTA's tokens change places in shared memory first, so that tokens of a digit leave side by side
            // (scattered from where they were, 65001 tokens took 10 us a pass, a sector each).
            uint2 v[SORT_U];
            unsigned to[SORT_U];
            const int n = (int)(end - begin);
#pragma unroll
            for (int u = 0; u < SORT_U; ++u) {
                const int i = u * 32 + lane;
                v[u] = make_uint2(key[i], pos[i]);
                const unsigned d = v[u].x >> shift & (bins - 1);
                to[u] = sm.start[d] + order[i] + at[d];
            }
            __syncthreads();
            uint2* const local = reinterpret_cast<uint2*>(&sm.key[0][0]);  // (over keys and positions, now in registers)
#pragma unroll
            for (int u = 0; u < SORT_U; ++u)
                if (u * 32 + lane < n) local[to[u]] = v[u];
            __syncthreads();
            const int count = (int)(min(T, (rank + 1) * SORT_NW * per) - min(T, rank * SORT_NW * per));
#pragma unroll 2
            for (int i = tid; i < count; i += SORT_NT) {
                const uint2 w = local[i];
                write(sm.base[w.x >> shift & (bins - 1)] + i, w);
            }
        } else {
#pragma unroll 1
            for (unsigned t0 = begin; t0 < end; t0 += 32 * SORT_U) {
                count(t0);
#pragma unroll 2
                for (unsigned i = lane; t0 + i < end && i < 32 * SORT_U; i += 32) {
                    const unsigned d = key[i] >> shift & (bins - 1);
                    write(sm.base[d] + sm.start[d] + order[i], make_uint2(key[i], pos[i]));
                }
            }
        }
        cluster_sync();  // the other CTAs' part of the order is written, and nobody reads this CTA's totals any more
    }
}

// Zeros of the rows in [v0, v1), those in `named` (a bit for each row from `base` on; NULL: none) excepted, by NT threads.
template <int DG, int NT>
__device__ __forceinline__ void zero_rows(const EmbedGradArgs& a, long long v0, long long v1, const unsigned* named, long long base) {
    using G = typename Elem<DG>::T;
    constexpr int N = Elem<DG>::N;
    const uint64_t policy = policy_drop();
    // threads a row, rows at a time
    int width = NT;
    while (width > 1 && width / 2 * N >= a.D) width /= 2;
    const int c = threadIdx.x % width;
    for (long long v = v0 + threadIdx.x / width; v < v1; v += NT / width) {
        if (named && named[(v - base) / 32] >> ((v - base) % 32) & 1u) continue;
        G* const to = static_cast<G*>(a.grad) + v * a.ldg;
        // whole granules, and the elements before and after them one by one
        const int head = min(a.D, (int)((16 - ((unsigned long long)to & 15)) & 15) / (int)sizeof(G)), whole = (a.D - head) / N;
        const int tail = a.D - head - whole * N;
        uint4* const mid = reinterpret_cast<uint4*>(to + head);
        for (int i = c; i < whole; i += width) store16(mid + i, make_uint4(0, 0, 0, 0), policy);
        for (int i = c; i < head; i += width) to[i] = Elem<DG>::put(0.f);
        for (int i = c; i < tail; i += width) to[head + whole * N + i] = Elem<DG>::put(0.f);
    }
}

template <int DG>
__global__ void __launch_bounds__(SORT_NT) embed_sort_kernel(const EmbedGradArgs a, int passes, int bits, long long rows) {
    extern __shared__ __align__(16) unsigned char dyn[];
    if (blockIdx.x < SORT_CL) {
        if (blockIdx.x == 0 && threadIdx.x == 0) *a.spans = 0;
        sort_tokens(a, passes, bits, *reinterpret_cast<SortSmem*>(dyn));
        return;
    }
    const long long parts = gridDim.x - SORT_CL, part = blockIdx.x - SORT_CL;
    zero_rows<DG, SORT_NT>(a, rows * part / parts, rows * (part + 1) / parts, nullptr, 0);
}

// ---- gradient: sums ----
// Sorted tokens of a chunk: few, for short chains and many CTAs (8192 tokens, 32000 x 1024 bf16: 39 us, with 32 44); twice that
// for long batches, whose partial sums take T D / 2 bytes with 16.
constexpr int SUM_NT = 128, SUM_MAX_R = 32;
int chunk_tokens(long long T) { return T <= 65536 ? 16 : SUM_MAX_R; }
// Columns of a thread: as many as a granule of the incoming gradient has.
template <int DT>
constexpr int SUM_W = Elem<DT>::N;

constexpr int ZERO_BYTES = 64 << 10;  // of zeros a CTA of the sums writes

// W elements as floats, W * their size being 8, 16 or 32 bytes at an address aligned to that or to 16.
template <int DG, int W>
__device__ __forceinline__ void read_some(const typename Elem<DG>::T* p, float (&f)[W]) {
    if constexpr (W * sizeof(*p) == 8) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        float2 h[Elem<DG>::N / 2];
        unpack<DG>(make_uint4(v.x, v.y, 0u, 0u), h);
        f[0] = h[0].x, f[1] = h[0].y, f[2] = h[1].x, f[3] = h[1].y;
    } else {
#pragma unroll
        for (int i = 0; i < W; i += Elem<DG>::N) {
            float2 h[Elem<DG>::N / 2];
            unpack<DG>(*reinterpret_cast<const uint4*>(p + i), h);
#pragma unroll
            for (int j = 0; j < Elem<DG>::N / 2; ++j) f[i + 2 * j] = h[j].x, f[i + 2 * j + 1] = h[j].y;
        }
    }
}
template <int DG, int W>
__device__ __forceinline__ void write_some(typename Elem<DG>::T* p, const float (&f)[W]) {
    if constexpr (W * sizeof(*p) == 8) {
        const float2 h[Elem<DG>::N / 2] = {{f[0], f[1]}, {f[2], f[3]}};
        const uint4 v = pack<DG>(h);
        __stcs(reinterpret_cast<uint2*>(p), make_uint2(v.x, v.y));
    } else {
#pragma unroll
        for (int i = 0; i < W; i += Elem<DG>::N) {
            float2 h[Elem<DG>::N / 2];
#pragma unroll
            for (int j = 0; j < Elem<DG>::N / 2; ++j) h[j] = make_float2(f[i + 2 * j], f[i + 2 * j + 1]);
            store16(reinterpret_cast<uint4*>(p + i), pack<DG>(h), policy_drop());
        }
    }
}
// Where rows are not whole granules, a thread's W columns of row v begin this many before a multiple of W, so that they
// are aligned in the row.
template <int DG, int W>
constexpr int SUM_ALIGN = W * sizeof(typename Elem<DG>::T) < 16 ? W * sizeof(typename Elem<DG>::T) : 16;
template <int DG, int W, bool VEC>
__device__ __forceinline__ int shift_of(const EmbedGradArgs& a, unsigned v) {
    using G = typename Elem<DG>::T;
    return VEC ? 0 : (int)((unsigned long long)(static_cast<G*>(a.grad) + (long long)v * a.ldg) & (SUM_ALIGN<DG, W> - 1)) / (int)sizeof(G);
}
// Columns c .. c + W - 1 of row v (c aligned as above), those outside [0, D) excepted.
template <int DG, bool VEC, int W>
__device__ __forceinline__ void write_row(const EmbedGradArgs& a, unsigned v, int c, const float (&acc)[W]) {
    using G = typename Elem<DG>::T;
    G* const to = static_cast<G*>(a.grad) + (long long)v * a.ldg + c;
    if (c >= a.D) return;
    if constexpr (W > 1)
        if (VEC || (c >= 0 && c + W <= a.D)) {
            float f[W];
            if (a.accumulate) read_some<DG, W>(to, f);
#pragma unroll
            for (int j = 0; j < W; ++j) f[j] = a.accumulate ? fmaf(a.scale, acc[j], f[j]) : a.scale * acc[j];
            write_some<DG, W>(to, f);
            return;
        }
#pragma unroll
    for (int j = 0; j < W; ++j)
        if (c + j >= 0 && c + j < a.D) to[j] = Elem<DG>::put(a.accumulate ? fmaf(a.scale, acc[j], Elem<DG>::get(to[j])) : a.scale * acc[j]);
}
// Partial sums of rows that end beyond the chunk after the one they begin in: slot 0 of a chunk is what it has of the
// row that began before it, slot 1 of the row that goes on after it.
__device__ __forceinline__ float* part_row(const EmbedGradArgs& a, long long chunk, int slot) {
    return a.part + (chunk * 2 + slot) * a.D;
}

// A thread's columns of several rows of the incoming gradient, fetched together: as many as registers hold.  Columns that do not
// begin at a granule are cut out of two (16-bit rows of 1003: three rows at a time 58 us, four 65; fp32 of 1001: four 124,
// three 128).
template <int DT, bool VEC>
struct SumRows {
    using T = typename Elem<DT>::T;
    static constexpr int W = SUM_W<DT>, U = VEC ? 8 : DT == SOT_F32 ? 4 : 3, G = VEC ? 1 : 2;
    uint4 raw[U][G];
    unsigned from[VEC ? 1 : U];  // the first column's byte in raw[u]
    // Rows pos[i0], pos[i0 + step] ..., columns col(i0) ..; past `end` the last one again, past the row's granules its last: no branch lies
    // between two loads.
    template <class Col>
    __device__ __forceinline__ void load(const EmbedGradArgs& a, const unsigned* pos, int i0, int end, Col col, int step = 1) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = min(i0 + u * step, end - 1), c = col(i);
            const T* const src = static_cast<const T*>(a.g) + (long long)pos[i] * a.ld;
            if constexpr (VEC)
                raw[u][0] = __ldcs(reinterpret_cast<const uint4*>(src + min(c, a.D - W)));
            else {
                const unsigned long long lo = (unsigned long long)src & ~15ull, hi = (unsigned long long)(src + a.D - 1) & ~15ull;
                const unsigned long long at = (unsigned long long)(src + c);
                from[u] = (unsigned)at & 15u;
#pragma unroll
                for (int j = 0; j < G; ++j)
                    raw[u][j] = __ldg(reinterpret_cast<const uint4*>(min(max((at & ~15ull) + 16 * j, lo), hi)));
            }
        }
    }
    // (columns outside the row get anything)
    __device__ __forceinline__ void add(int u, float (&acc)[W]) const {
        uint4 v[1];
        if constexpr (VEC) v[0] = raw[u][0];
        else cut_out<DT>(raw[u], from[u], v);
        float2 f[W / 2];
        unpack<DT>(v[0], f);
#pragma unroll
        for (int j = 0; j < W / 2; ++j) {
            acc[2 * j] += f[j].x;
            acc[2 * j + 1] += f[j].y;
        }
    }
};

// Few tokens: no sort.  Every CTA reads all ids; the one of a row's first token (and a tile of columns) gathers the others of
// the row, in order.  One launch instead of three (1000 tokens into 20000 x 2048 bf16: 19 us, with three 31).  Where a row has
// many tokens, the CTAs of the first SHARES of them take a share of the columns each, and divide the tokens among
// their threads (1000 tokens of one row: 21 us, by one CTA a tile 107).
constexpr int FEW_TOKENS = 1024, MANY = 64, SHARES = 16;

template <int DT, int DG, bool VEC>
__global__ void __launch_bounds__(SUM_NT, 8) embed_few_kernel(const EmbedGradArgs a, int tiles, long long zeros, int zero_share) {
    constexpr int U = SumRows<DT, VEC>::U, W = SUM_W<DT>, PER = FEW_TOKENS / SUM_NT;
    __shared__ int ids[FEW_TOKENS];
    __shared__ unsigned mark[FEW_TOKENS > ZERO_BYTES / 32 ? FEW_TOKENS : ZERO_BYTES / 32];  // rows of this CTA; or the row's tokens
    __shared__ unsigned same;  // tokens of the row: before this CTA's in the upper half, all in the lower
    __shared__ float part[SUM_NT][W];
    const int tid = threadIdx.x, lane = tid & 31, T = (int)a.T;
    if (tid == 0) same = 0;
    int id[PER];
    if (T > 0) load_indices<PER>(a.ids, a.ids_type, tid, SUM_NT, T, a.V, id);
#pragma unroll
    for (int u = 0; u < PER; ++u) ids[u * SUM_NT + tid] = u * SUM_NT + tid < T ? id[u] : -1;
    const long long zero = blockIdx.x * zeros / gridDim.x, block = blockIdx.x - zero;
    if ((blockIdx.x + 1) * zeros / gridDim.x > zero) {
        const long long v0 = zero * zero_share, v1 = min((long long)a.V, v0 + zero_share);
        for (int i = tid; i < (zero_share + 31) / 32; i += SUM_NT) mark[i] = 0u;
        __syncthreads();
#pragma unroll
        for (int u = 0; u < PER; ++u) {
            const long long r = ids[u * SUM_NT + tid] - v0;
            if (r >= 0 && r < v1 - v0) atomicOr(&mark[r / 32], 1u << r % 32);
        }
        __syncthreads();
        zero_rows<DG, SUM_NT>(a, v0, v1, mark, v0);
        return;
    }
    const int t = (int)(block / tiles), c0 = (int)(block % tiles) * SUM_NT * W;
    __syncthreads();
    const int v = ids[t];
    if (v < 0) return;
    unsigned mine = 0;
#pragma unroll
    for (int u = 0; u < PER; ++u)
        if (ids[u * SUM_NT + tid] == v) mine += u * SUM_NT + tid < t ? 0x10001u : 1u;
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0 && mine) atomicAdd(&same, mine);
    __syncthreads();
    const int share = (int)(same >> 16), n = (int)(same & 0xffffu);
    const bool many = n >= MANY;
    if (share >= (many ? SHARES : 1)) return;
    unsigned* const pos = mark;
    if (tid < 32) {
        int k = 0;
        for (int i = many ? 0 : t / 32 * 32; i < T; i += 32) {
            const unsigned hit = __ballot_sync(0xffffffffu, ids[i + lane] == v);
            if (hit >> lane & 1u) pos[k + __popc(hit & ((1u << lane) - 1u))] = i + lane;
            k += __popc(hit);
        }
    }
    __syncthreads();
    // the thread's columns, and its tokens: every step-th one
    constexpr int LANES = SUM_NT / SHARES;
    const int step = many ? SHARES : 1, first = many ? tid / LANES : 0;
    const int col = c0 + (many ? share * LANES + tid % LANES : tid) * W - shift_of<DG, W, VEC>(a, (unsigned)v);
    float acc[W] = {};
    for (int i0 = first; i0 < n; i0 += U * step) {
        SumRows<DT, VEC> rows;
        rows.load(a, pos, i0, n, [&](int) { return col; }, step);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * step < n) rows.add(u, acc);
    }
    if (many) {
#pragma unroll
        for (int j = 0; j < W; ++j) part[tid][j] = acc[j];
        __syncthreads();
        if (tid >= LANES) return;
        for (int k = 1; k < SHARES; ++k)
#pragma unroll
            for (int j = 0; j < W; ++j) acc[j] += part[k * LANES + tid][j];
    }
    write_row<DG, VEC, W>(a, (unsigned)v, col, acc);
}

template <int DT, int DG, bool VEC>
__global__ void __launch_bounds__(SUM_NT, 8) embed_sum_kernel(const EmbedGradArgs a, int tiles, long long zeros, long long zero_from,
                                                              int zero_share) {
    constexpr int SUM_U = SumRows<DT, VEC>::U, W = SUM_W<DT>;
    __shared__ unsigned key[2 * SUM_MAX_R + 1], pos[2 * SUM_MAX_R];
    const int R = a.chunk;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // `zeros` CTAs, spread evenly over the grid, write zeros
    const long long zero = blockIdx.x * zeros / gridDim.x, block = blockIdx.x - zero;
    if ((blockIdx.x + 1) * zeros / gridDim.x > zero) {
        const long long v = zero_from + zero * zero_share;
        zero_rows<DG, SUM_NT>(a, v, min((long long)a.V, v + zero_share), a.named, 0);
        return;
    }
    const long long chunk = block / tiles;
    const int c0 = (int)(block % tiles) * SUM_NT * W, tid = threadIdx.x;
    const long long at = chunk * R;
    // The keys from the token before the chunk to the end of the next chunk; V: none.
    unsigned mine = (unsigned)a.V;
    const uint2* const sorted = a.sorted[0];
    const auto key_at = [&](long long i) { return i >= 0 && i < a.T ? __ldg(&sorted[i].x) : (unsigned)a.V; };
    if (tid < 2 * R + 1) {
        const long long i = at + tid - 1;
        const uint2 t = i >= 0 && i < a.T ? __ldg(sorted + i) : make_uint2((unsigned)a.V, 0u);
        key[tid] = mine = t.x;
        if (tid > 0) pos[tid - 1] = t.y;
    }
    const unsigned long_before = key_at(at - R - 1), long_after = key_at(at + 2 * R);
    // tokens of the chunk that have a row: they come first
    const int n = __syncthreads_count(tid >= 1 && tid <= R && mine < (unsigned)a.V);
    const auto row = [&](int i) { return i < 2 * R ? key[i + 1] : long_after; };
    if (n == 0) return;
    // The chunk before finishes a row that begins in it and ends here; this one does the same for the next.
    const bool open = key[0] == key[1];
    int from = 0, end = n;
    if (open && long_before != key[1] && row(R) != key[1])
        while (from < n && row(from) == key[1]) ++from;
    const unsigned tail = row(n - 1);
    if (n == R && row(R) == tail && !(open && key[1] == tail) && long_after != tail)
        while (end < 2 * R && row(end) == tail) ++end;
    const auto col = [&](unsigned v) { return c0 + tid * W - shift_of<DG, W, VEC>(a, v); };
    float acc[W] = {};
    for (int i0 = from; i0 < end; i0 += SUM_U) {
        SumRows<DT, VEC> rows;
        rows.load(a, pos, i0, end, [&](int i) { return col(row(i)); });
#pragma unroll
        for (int u = 0; u < SUM_U; ++u)
            if (i0 + u < end) {
                const int i = i0 + u;
                rows.add(u, acc);
                const unsigned v = row(i);
                if (i == end - 1 || row(i + 1) != v) {  // the last token of the row here
                    const bool before = open && from == 0 && key[1] == v, after = row(i + 1) == v;
                    if (before || after) {
                        float* const to = part_row(a, chunk, before ? 0 : 1);
                        const int c = col(v);
#pragma unroll
                        for (int j = 0; j < W; ++j)
                            if (c + j >= 0 && c + j < a.D) __stcg(to + c + j, acc[j]);
                        if (!before && tid == 0 && c0 == 0) a.span[atomicAdd(a.spans, 1u)] = make_uint2((unsigned)chunk, v);
                    } else
                        write_row<DG, VEC, W>(a, v, col(v), acc);
#pragma unroll
                    for (int j = 0; j < W; ++j) acc[j] = 0.f;
                }
            }
    }
}

// Rows that span chunks, from the list of the chunks where one begins (in no order: each is summed by itself).  A CTA takes
// JOIN_COLS columns of a row.  Warp w adds up the row's chunks w, w + 8, ..., the warps' sums are added in order.  Eight
// chunks' sums are fetched before it is known that they belong to the row, so that one wait finds both out.
constexpr int JOIN_NT = 256, JOIN_NW = JOIN_NT / 32, JOIN_COLS = 128, JOIN_U = 8;

template <int DG, bool VEC>
__global__ void __launch_bounds__(JOIN_NT, 4) embed_join_kernel(const EmbedGradArgs a, int tiles) {
    __shared__ float sums[JOIN_NW][JOIN_COLS];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int R = a.chunk;
    const long long spans = __ldcg(a.spans), work = spans * tiles, chunks = (a.T + R - 1) / R;
    for (long long w = blockIdx.x; w < work; w += gridDim.x) {
        const uint2 span = __ldcg(a.span + w % spans);
        const int c0 = (int)(w / spans) * JOIN_COLS;
        int col[4];
        float acc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // (columns past the end are summed as the last one, and not written)
            col[j] = min(c0 + j * 32 + lane, a.D - 1);
            acc[j] = warp == 0 ? __ldcg(part_row(a, span.x, 1) + col[j]) : 0.f;
        }
        bool on = true;
        for (long long c = span.x + 1 + warp; on; c += JOIN_U * JOIN_NW) {
            float f[JOIN_U][4];
            unsigned key[JOIN_U];
#pragma unroll
            for (int u = 0; u < JOIN_U; ++u) {  // (no branch on what is loaded before all loads are out)
                const long long at = min(c + u * JOIN_NW, chunks - 1);
                key[u] = __ldcg(&a.sorted[0][at * R].x);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[u][j] = __ldcg(part_row(a, at, 0) + col[j]);
            }
#pragma unroll
            for (int u = 0; u < JOIN_U; ++u) {
                on = on && c + u * JOIN_NW < chunks && key[u] == span.y;
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[j] += on ? f[u][j] : 0.f;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) sums[warp][j * 32 + lane] = acc[j];
        __syncthreads();
        constexpr int W = VEC ? 8 : 1;
        if (tid < JOIN_COLS / W) {
            float f[W];
#pragma unroll
            for (int j = 0; j < W; ++j) {
                f[j] = sums[0][tid * W + j];
                for (int k = 1; k < JOIN_NW; ++k) f[j] += sums[k][tid * W + j];
            }
            write_row<DG, VEC, W>(a, span.y, c0 + tid * W, f);
        }
        __syncthreads();
    }
}

// Rows of whole pieces of eight columns.  (In fp32 four would do for whole granules; 20000 rows of 1004: lookup 24.5 us, of
// 1008 24.8, gradient 67 and 61.)
bool whole_rows(const void* p, long long ld, int D, int type) {
    const long long b = type == SOT_F32 ? 4 : 2;
    return (unsigned long long)p % 16 == 0 && ld * b % 16 == 0 && D % 8 == 0;
}

template <int DT, int DO>
cudaError_t launch_embed_t(const EmbedArgs& a, int sms, cudaStream_t st) {
    const bool vec = whole_rows(a.table, a.ld, a.D, a.type) && whole_rows(a.out, a.ldo, a.D, a.out_type);
    // (columns before a row's first granule of the output count as the row's)
    const unsigned per = vec ? a.D / EMB_W : (a.D + 16 / (int)sizeof(typename Elem<DO>::T) - 1 + EMB_W - 1) / EMB_W;
    const int tile = EMB_NT * (vec ? EMB_PIECES<true> : EMB_PIECES<false>);
    const long long tiles = (a.T * per + tile - 1) / tile;
    const unsigned blocks = (unsigned)(tiles < 1ll << 30 ? tiles : 1ll << 30);
    if (vec) embed_kernel<DT, DO, true><<<blocks, EMB_NT, 0, st>>>(a, per);
    else embed_kernel<DT, DO, false><<<blocks, EMB_NT, 0, st>>>(a, per);
    return cudaGetLastError();
}

cudaError_t launch_after(const void* kern, unsigned blocks, int threads, void** args, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(blocks, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    return cudaLaunchKernelExC(&cfg, kern, args);
}

// Rows that get their zeros beside the sort: as many as that leaves time for (8192 tokens, 32000 x 1024 bf16 to fp32: 37 us,
// without any and with four times as many 43; 2000, 20000 x 2048 bf16: 28, 35 and 33; 4000, 100000 x 1024: 47, 54 and 55;
// 1500, 200000 x 512: 45, 51 and 52; 65001, 32003 x 1000 fp32: 101, 107 and 100).
constexpr long long EARLY_BYTES = 40 << 20, EARLY_BYTES_A_TOKEN = 1200;
long long early_rows(const EmbedGradArgs& a) {
    if (a.accumulate) return 0;
    const long long rows = (EARLY_BYTES + EARLY_BYTES_A_TOKEN * a.T) / ((long long)a.D * (a.grad_type == SOT_F32 ? 4 : 2));
    return rows < a.V ? rows : a.V;
}

template <int DG>
cudaError_t launch_sort(const EmbedGradArgs& a, const EmbedGradPlan& p, int sms, cudaStream_t st) {
    auto kern = embed_sort_kernel<DG>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(SortSmem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    const long long rows = early_rows(a);
    long long zero = (rows * a.D + (1 << 16) - 1) >> 16;  // 64 Ki elements a CTA
    zero = zero < sms ? zero : sms;
    zero = (zero + SORT_CL - 1) / SORT_CL * SORT_CL;
    cfg.gridDim = dim3((unsigned)(SORT_CL + zero), 1, 1);
    cfg.blockDim = dim3(SORT_NT, 1, 1);
    cfg.dynamicSmemBytes = sizeof(SortSmem);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = SORT_CL;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, kern, a, p.passes, p.bits, rows);
}

template <int DT, int DG>
cudaError_t launch_sum(const EmbedGradArgs& a, const EmbedGradPlan& p, bool vec, int sms, cudaStream_t st) {
    EmbedGradArgs b = a;
    constexpr int W = SUM_W<DT>, cols = SUM_NT * W, shift = SUM_ALIGN<DG, W> / sizeof(typename Elem<DG>::T) - 1;
    int tiles = (a.D + (vec ? 0 : shift) + cols - 1) / cols, join_tiles = (a.D + JOIN_COLS - 1) / JOIN_COLS;
    const bool few = p.passes == 0;
    long long from = few ? 0 : early_rows(a), zeros = 0;
    int share = 1;
    if (!a.accumulate) {
        const long long row = (long long)a.D * (a.grad_type == SOT_F32 ? 4 : 2), fit = ZERO_BYTES / row;
        share = (int)(fit > 1 ? fit : 1);
        zeros = (a.V - from + share - 1) / share;
    }
    const long long blocks = (few ? a.T : p.chunks) * tiles + zeros;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    if (blocks == 0) return cudaSuccess;
    if (few) {
        count_launches(1);
        if (vec) embed_few_kernel<DT, DG, true><<<(unsigned)blocks, SUM_NT, 0, st>>>(b, tiles, zeros, share);
        else embed_few_kernel<DT, DG, false><<<(unsigned)blocks, SUM_NT, 0, st>>>(b, tiles, zeros, share);
        return cudaGetLastError();
    }
    void* args[] = {&b, &tiles, &zeros, &from, &share};
    count_launches(1);
    const cudaError_t e = launch_after(vec ? (const void*)embed_sum_kernel<DT, DG, true> : (const void*)embed_sum_kernel<DT, DG, false>,
                                       (unsigned)blocks, SUM_NT, args, st);
    if (e != cudaSuccess || p.chunks < 2) return e;
    void* join_args[] = {&b, &join_tiles};
    const long long most = p.chunks * join_tiles;  // rows that span chunks are fewer than chunks
    count_launches(1);
    return launch_after(vec ? (const void*)embed_join_kernel<DG, true> : (const void*)embed_join_kernel<DG, false>,
                        (unsigned)(most < 4ll * sms ? most : 4ll * sms), JOIN_NT, join_args, st);
}

}  // namespace

cudaError_t launch_embed(const EmbedArgs& a, int sms, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    count_launches(1);
#define SOT_OUT(DT)                                                          \
    switch (a.out_type) {                                                    \
        case SOT_F32: return launch_embed_t<DT, SOT_F32>(a, sms, st);        \
        case SOT_F16: return launch_embed_t<DT, SOT_F16>(a, sms, st);        \
        default: return launch_embed_t<DT, SOT_BF16>(a, sms, st);            \
    }
    switch (a.type) {
        case SOT_F32: SOT_OUT(SOT_F32)
        case SOT_F16: SOT_OUT(SOT_F16)
        default: SOT_OUT(SOT_BF16)
    }
#undef SOT_OUT
}

EmbedGradPlan embed_grad_plan(long long T, int V, int D) {
    EmbedGradPlan p = {};
    if (T <= FEW_TOKENS) return p;  // (no sort, no scratch)
    int need = 1;
    while (need < 32 && (unsigned)V >> need) ++need;  // keys 0 .. V
    p.passes = (need + SORT_MAX_BITS - 1) / SORT_MAX_BITS;
    p.bits = (need + p.passes - 1) / p.passes;
    p.chunk = chunk_tokens(T);
    p.chunks = (T + p.chunk - 1) / p.chunk;
    const auto place = [&](size_t bytes) {
        const size_t at = p.scratch;
        p.scratch = (at + bytes + 255) & ~(size_t)255;
        return at;
    };
    for (int i = 0; i < 2; ++i) p.sorted_at[i] = place(sizeof(uint2) * T);
    p.spans_at = place(sizeof(unsigned));
    p.span_at = place(sizeof(uint2) * p.chunks);
    p.named_at = place(4 * (((size_t)V + 31) / 32));
    p.part_at = place(sizeof(float) * 2 * (size_t)p.chunks * D);
    return p;
}

cudaError_t launch_embed_grad(EmbedGradArgs a, const EmbedGradPlan& p, unsigned char* scratch, int sms, cudaStream_t st) {
    if (a.T == 0 && a.accumulate) return cudaSuccess;
    for (int i = 0; i < 2; ++i) a.sorted[i] = reinterpret_cast<uint2*>(scratch + p.sorted_at[i]);
    a.chunk = p.chunk;
    a.spans = reinterpret_cast<unsigned*>(scratch + p.spans_at);
    a.span = reinterpret_cast<uint2*>(scratch + p.span_at);
    a.named = a.accumulate ? nullptr : reinterpret_cast<unsigned*>(scratch + p.named_at);
    a.part = reinterpret_cast<float*>(scratch + p.part_at);
    const bool vec_out = whole_rows(a.grad, a.ldg, a.D, a.grad_type);
    const cudaError_t e = p.passes == 0 ? cudaSuccess
                          : a.grad_type == SOT_F32   ? launch_sort<SOT_F32>(a, p, sms, st)
                          : a.grad_type == SOT_F16 ? launch_sort<SOT_F16>(a, p, sms, st)
                                                   : launch_sort<SOT_BF16>(a, p, sms, st);
    if (e != cudaSuccess) return e;
    const bool vec = vec_out && whole_rows(a.g, a.ld, a.D, a.type);
#define SOT_OUT(DT)                                                            \
    switch (a.grad_type) {                                                     \
        case SOT_F32: return launch_sum<DT, SOT_F32>(a, p, vec, sms, st);      \
        case SOT_F16: return launch_sum<DT, SOT_F16>(a, p, vec, sms, st);      \
        default: return launch_sum<DT, SOT_BF16>(a, p, vec, sms, st);          \
    }
    switch (a.type) {
        case SOT_F32: SOT_OUT(SOT_F32)
        case SOT_F16: SOT_OUT(SOT_F16)
        default: SOT_OUT(SOT_BF16)
    }
#undef SOT_OUT
}

}  // namespace sot
