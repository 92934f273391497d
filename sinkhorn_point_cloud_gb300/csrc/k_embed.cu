// k_embed.cu -- embedding lookup with scaling, and its gradient by sorted tokens.
//
// Lookup: out[t] = scale table[id[t]], a copy of rows with one rounding: memory-bound.
//
// Gradient: grad[v] = scale sum of g[t] over the tokens t with id[t] = v, in the order of t.
//   sort     one cluster sorts the tokens by row, stably (radix passes over shared-memory
//            counts, joined through distributed shared memory), while the other CTAs of the launch
//            write the zeros of the rows that no token names;
//   sum      a CTA takes a chunk of sorted tokens and a tile of columns, and writes
//            the rows that lie inside its chunk.  A row that spans chunks leaves a partial sum in each;
//   join     adds these up, in the order of the chunks.
// No atomics on floats: repeated calls give the same bits.
#include <cuda_runtime.h>

#include "embed.h"
#include "kernels.h"
#include "lm.cuh"

namespace sot {

namespace {

// Eight elements as floats, from an address aligned to 16 bytes.
template <int DT>
__device__ __forceinline__ void load8(const typename Elem<DT>::T* p, float (&f)[8]) {
    float2 h[4];
    if constexpr (DT == SOT_F32) {
        const uint4* q = reinterpret_cast<const uint4*>(p);
        const uint4 a = __ldg(q), b = __ldg(q + 1);
        h[0] = make_float2(__uint_as_float(a.x), __uint_as_float(a.y));
        h[1] = make_float2(__uint_as_float(a.z), __uint_as_float(a.w));
        h[2] = make_float2(__uint_as_float(b.x), __uint_as_float(b.y));
        h[3] = make_float2(__uint_as_float(b.z), __uint_as_float(b.w));
    } else
        unpack<DT>(__ldg(reinterpret_cast<const uint4*>(p)), h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = h[i].x;
        f[2 * i + 1] = h[i].y;
    }
}
template <int DT>
__device__ __forceinline__ void store8(typename Elem<DT>::T* p, const float (&f)[8]) {
    if constexpr (DT == SOT_F32) {
        __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
        __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
    } else {
        const float2 h[4] = {{f[0], f[1]}, {f[2], f[3]}, {f[4], f[5]}, {f[6], f[7]}};
        __stcs(reinterpret_cast<uint4*>(p), pack<DT>(h));
    }
}

// ---- lookup ----
constexpr int EMB_NT = 256, EMB_U = 4;

// A thread takes U pieces of a tile of NT U pieces: eight columns where rows are whole granules (VEC), else one.
template <int DT, int DO, bool VEC>
__global__ void __launch_bounds__(EMB_NT) embed_kernel(const EmbedArgs a, unsigned per_row) {
    using T = typename Elem<DT>::T;
    using O = typename Elem<DO>::T;
    constexpr int W = VEC ? 8 : 1;
    const long long total = a.T * per_row, tile = (long long)EMB_NT * EMB_U;
    for (long long base = blockIdx.x * tile; base < total; base += gridDim.x * tile) {
        float f[EMB_U][W];
        O* to[EMB_U];
#pragma unroll
        for (int j = 0; j < EMB_U; ++j) {
            const long long i = base + j * EMB_NT + threadIdx.x;
            to[j] = nullptr;
            if (i < total) {
                const long long t = i / per_row;
                const int c = (int)(i - t * per_row) * W;
                const int id = load_index(a.ids, a.ids_type, t, a.V);
                to[j] = static_cast<O*>(a.out) + t * a.ldo + c;
                if (id >= 0) {
                    const T* from = static_cast<const T*>(a.table) + id * a.ld + c;
                    if constexpr (VEC) load8<DT>(from, f[j]);
                    else f[j][0] = Elem<DT>::get(*from);
#pragma unroll
                    for (int w = 0; w < W; ++w) f[j][w] *= a.scale;
                } else {
#pragma unroll
                    for (int w = 0; w < W; ++w) f[j][w] = 0.f;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < EMB_U; ++j)
            if (to[j]) {
                if constexpr (VEC) store8<DO>(to[j], f[j]);
                else *to[j] = Elem<DO>::put(f[j][0]);
            }
    }
}

// ---- gradient: sort ----
constexpr int SORT_NT = 1024, SORT_NW = SORT_NT / 32, SORT_CL = 8, SORT_MAX_BITS = 9, SORT_MAX_BINS = 1 << SORT_MAX_BITS;

struct SortSmem {
    unsigned at[SORT_NW][SORT_MAX_BINS];  // per warp: counts, then places
    unsigned total[SORT_MAX_BINS];        // of this CTA
    unsigned sums[SORT_NW];
};

// Row of token t; tokens without one come last.
__device__ __forceinline__ unsigned token_key(const EmbedGradArgs& a, long long t) {
    const int id = load_index(a.ids, a.ids_type, t, a.V);
    return id < 0 ? (unsigned)a.V : (unsigned)id;
}

__device__ void sort_tokens(const EmbedGradArgs& a, int passes, int bits, SortSmem& sm) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();
    const int bins = 1 << bits;
    // a warp's share: contiguous, whole steps of 32
    const long long workers = SORT_CL * SORT_NW, steps = (a.T + 31) / 32, per = (steps + workers - 1) / workers * 32;
    const long long begin = (rank * SORT_NW + warp) * per;
    const long long end = min(begin + per, a.T);
    for (int p = 0; p < passes; ++p) {
        // (the last pass writes to buffer 0)
        const bool odd = (passes - 1 - p) & 1;
        const unsigned *key_in = odd ? a.key[0] : a.key[1], *pos_in = odd ? a.pos[0] : a.pos[1];
        unsigned *key_out = odd ? a.key[1] : a.key[0], *pos_out = odd ? a.pos[1] : a.pos[0];
        const int shift = p * bits;
        const auto key_of = [&](long long t) { return p == 0 ? token_key(a, t) : __ldcg(key_in + t); };
        for (int b = lane; b < bins; b += 32) sm.at[warp][b] = 0;
        __syncwarp();
        for (long long t = begin + lane; t < begin + per && t - lane < end; t += 32) {
            const unsigned d = t < end ? key_of(t) >> shift & (bins - 1) : 0xffffffffu;
            const unsigned peers = __match_any_sync(0xffffffffu, d);
            if (t < end && lane == __ffs(peers) - 1) sm.at[warp][d] += __popc(peers);
            __syncwarp();
        }
        __syncthreads();
        unsigned mine = 0;  // this CTA's count of bin tid
        if (tid < bins) {
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
            for (uint32_t r = 0; r < SORT_CL; ++r) {
                unsigned c;
                asm volatile("ld.shared::cluster.u32 %0, [%1];"
                             : "=r"(c)
                             : "r"(cluster_addr(smem_u32(&sm.total[tid]), r))
                             : "memory");
                if (r < rank) before += c;
                all += c;
            }
        unsigned scan = all;  // inclusive over the bins
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned v = __shfl_up_sync(0xffffffffu, scan, o);
            if (lane >= o) scan += v;
        }
        if (lane == 31) sm.sums[warp] = scan;
        __syncthreads();
        unsigned base = scan - all + before;
        for (int w = 0; w < warp; ++w) base += sm.sums[w];
        if (tid < bins)
            for (int w = 0; w < SORT_NW; ++w) sm.at[w][tid] += base;
        __syncthreads();
        for (long long t = begin + lane; t < begin + per && t - lane < end; t += 32) {
            const unsigned key = t < end ? key_of(t) : 0u, d = t < end ? key >> shift & (bins - 1) : 0xffffffffu;
            const unsigned peers = __match_any_sync(0xffffffffu, d);
            if (t < end) {
                const unsigned to = sm.at[warp][d] + __popc(peers & ((1u << lane) - 1u));
                key_out[to] = key;
                pos_out[to] = p == 0 ? (unsigned)t : __ldcg(pos_in + t);
            }
            __syncwarp();
            if (t < end && lane == __ffs(peers) - 1) sm.at[warp][d] += __popc(peers);
            __syncwarp();
        }
        cluster_sync();  // the other CTAs' part of the order is written, and nobody reads this CTA's totals any more
    }
}

// Zeros of the rows in [v0, v1) that no token names.
template <int DG>
__device__ void zero_rows(const EmbedGradArgs& a, int v0, int v1, unsigned* named, bool vec) {
    using G = typename Elem<DG>::T;
    const int tid = threadIdx.x, n = v1 - v0;
    for (int i = tid; i < (n + 31) / 32; i += SORT_NT) named[i] = 0;
    __syncthreads();
    for (long long t = tid; t < a.T; t += SORT_NT) {
        const unsigned r = token_key(a, t) - (unsigned)v0;
        if (r < (unsigned)n) atomicOr(&named[r / 32], 1u << (r % 32));
    }
    __syncthreads();
    const int per = vec ? (a.D * (int)sizeof(G)) / 16 : a.D;
    const int width = min(SORT_NT, (per + 31) / 32 * 32), rows = SORT_NT / width;  // threads a row, rows at a time
    const int r = tid / width;
    if (r >= rows) return;
    for (int v = r; v < n; v += rows) {
        if (named[v / 32] >> (v % 32) & 1u) continue;
        G* const to = static_cast<G*>(a.grad) + (long long)(v0 + v) * a.ldg;
        if (vec)
            for (int c = tid % width; c < per; c += width) __stcs(reinterpret_cast<uint4*>(to) + c, make_uint4(0, 0, 0, 0));
        else
            for (int c = tid % width; c < per; c += width) to[c] = Elem<DG>::put(0.f);
    }
}

constexpr int ZERO_ROWS = 8192;  // of a CTA at a time, at most (a bit each)

template <int DG>
__global__ void __launch_bounds__(SORT_NT) embed_sort_kernel(const EmbedGradArgs a, int passes, int bits, bool vec) {
    extern __shared__ __align__(16) unsigned char dyn[];
    if (blockIdx.x < SORT_CL) {
        if (a.T > 0) sort_tokens(a, passes, bits, *reinterpret_cast<SortSmem*>(dyn));
        return;
    }
    const int parts = gridDim.x - SORT_CL, part = blockIdx.x - SORT_CL;
    const int share = (int)min((long long)ZERO_ROWS, ((long long)a.V + parts - 1) / parts);
    for (long long v0 = (long long)part * share; v0 < a.V; v0 += (long long)parts * share) {
        zero_rows<DG>(a, (int)v0, (int)min((long long)a.V, v0 + share), reinterpret_cast<unsigned*>(dyn), vec);
        __syncthreads();
    }
}

// ---- gradient: sums ----
constexpr int SUM_NT = 128, SUM_R = 32, SUM_U = 8, SUM_COLS = SUM_NT * 8;

// The columns of a thread: eight in a row where rows are whole granules (VEC), else SUM_NT apart.
template <bool VEC>
__device__ __forceinline__ int sum_col(int c0, int j) {
    return VEC ? c0 + threadIdx.x * 8 + j : c0 + j * SUM_NT + threadIdx.x;
}
template <int DG, bool VEC>
__device__ __forceinline__ void write_row(const EmbedGradArgs& a, unsigned v, int c0, const float (&acc)[8]) {
    using G = typename Elem<DG>::T;
    G* const to = static_cast<G*>(a.grad) + (long long)v * a.ldg;
    float f[8];
    if constexpr (VEC) {
        const int c = sum_col<VEC>(c0, 0);
        if (c >= a.D) return;
        float old[8] = {};
        if (a.accumulate) load8<DG>(to + c, old);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = a.accumulate ? fmaf(a.scale, acc[j], old[j]) : a.scale * acc[j];
        store8<DG>(to + c, f);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = sum_col<VEC>(c0, j);
            if (c < a.D)
                to[c] = Elem<DG>::put(a.accumulate ? fmaf(a.scale, acc[j], Elem<DG>::get(to[c])) : a.scale * acc[j]);
        }
    }
}
// Partial sums: slot 0 of a chunk is what it has of the row that began before it, slot 1 of the row that goes on after it.
template <bool VEC>
__device__ __forceinline__ float* part_row(const EmbedGradArgs& a, long long chunk, int slot) {
    return a.part + (chunk * 2 + slot) * a.D;
}

template <int DT, int DG, bool VEC>
__global__ void __launch_bounds__(SUM_NT) embed_sum_kernel(const EmbedGradArgs a, int tiles) {
    using T = typename Elem<DT>::T;
    __shared__ unsigned key[SUM_R + 2], pos[SUM_R];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long chunk = blockIdx.x / tiles;
    const int c0 = (int)(blockIdx.x % tiles) * SUM_COLS, tid = threadIdx.x;
    const long long at = chunk * SUM_R;
    const int n = (int)min((long long)SUM_R, a.T - at);
    if (tid < SUM_R + 2) {  // with the token before and the one after; V: none
        const long long i = at + tid - 1;
        key[tid] = i >= 0 && i < a.T ? a.key[0][i] : (unsigned)a.V;
        if (tid < n) pos[tid] = a.pos[0][at + tid];
    }
    __syncthreads();
    float acc[8] = {};
    const auto flush = [&](int i, bool first, bool ends) {  // the row of token i
        const unsigned v = key[i + 1];
        const bool before = first && key[0] == v, after = ends && key[n + 1] == v;
        if (before || after) {
            float* const to = part_row<VEC>(a, chunk, before ? 0 : 1);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = sum_col<VEC>(c0, j);
                if (c < a.D) to[c] = acc[j];
            }
        } else
            write_row<DG, VEC>(a, v, c0, acc);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    };
    bool first = true;
    for (int i0 = 0; i0 < n; i0 += SUM_U) {
        float f[SUM_U][8];
#pragma unroll
        for (int u = 0; u < SUM_U; ++u) {
            const int i = i0 + u;
            if (i >= n || key[i + 1] >= (unsigned)a.V) continue;
            const T* const from = static_cast<const T*>(a.g) + (long long)pos[i] * a.ld;
            if constexpr (VEC) {
                const int c = sum_col<VEC>(c0, 0);
                if (c < a.D) load8<DT>(from + c, f[u]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int c = sum_col<VEC>(c0, j);
                    f[u][j] = c < a.D ? Elem<DT>::get(from[c]) : 0.f;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < SUM_U; ++u) {
            const int i = i0 + u;
            if (i >= n || key[i + 1] >= (unsigned)a.V) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] += f[u][j];
            if (i == n - 1 || key[i + 2] != key[i + 1]) {
                flush(i, first, i == n - 1);
                first = false;
            }
        }
    }
}

// Rows that span chunks: the chunk where one begins adds up what the others have of it.
template <int DG, bool VEC>
__global__ void __launch_bounds__(SUM_NT) embed_join_kernel(const EmbedGradArgs a, int tiles) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long chunk = blockIdx.x / tiles;
    const int c0 = (int)(blockIdx.x % tiles) * SUM_COLS;
    const unsigned* const key = a.key[0];
    const long long end = (chunk + 1) * SUM_R;
    if (end >= a.T) return;
    const unsigned v = key[end - 1];
    if (v >= (unsigned)a.V || key[end] != v) return;                    // nothing goes on after the chunk
    if (chunk > 0 && key[end - SUM_R] == v && key[end - SUM_R - 1] == v) return;  // it began before
    float acc[8];
    const auto add = [&](const float* from, bool set) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = sum_col<VEC>(c0, j);
            const float x = c < a.D ? from[c] : 0.f;
            acc[j] = set ? x : acc[j] + x;
        }
    };
    add(part_row<VEC>(a, chunk, 1), true);
    for (long long c = chunk + 1; c * SUM_R < a.T && key[c * SUM_R] == v; ++c) add(part_row<VEC>(a, c, 0), false);
    write_row<DG, VEC>(a, v, c0, acc);
}

bool whole_rows(const void* p, long long ld, int D, int type) {
    const long long b = type == SOT_F32 ? 4 : 2;
    return (unsigned long long)p % 16 == 0 && ld * b % 16 == 0 && D % 8 == 0;
}

template <int DT, int DO>
cudaError_t launch_embed_t(const EmbedArgs& a, int sms, cudaStream_t st) {
    const bool vec = whole_rows(a.table, a.ld, a.D, a.type) && whole_rows(a.out, a.ldo, a.D, a.out_type);
    const unsigned per = vec ? a.D / 8 : a.D;
    const long long tiles = (a.T * per + EMB_NT * EMB_U - 1) / (EMB_NT * EMB_U);
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

template <int DG>
cudaError_t launch_sort(const EmbedGradArgs& a, const EmbedGradPlan& p, bool vec, int sms, cudaStream_t st) {
    auto kern = embed_sort_kernel<DG>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(SortSmem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    long long zero = 0;
    if (!a.accumulate) {
        zero = ((long long)a.V * a.D + (1 << 16) - 1) >> 16;  // 64 Ki elements a CTA, up to two CTAs an SM
        zero = zero < 2ll * sms ? zero : 2ll * sms;
        zero = (zero + SORT_CL - 1) / SORT_CL * SORT_CL;
    }
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
    return cudaLaunchKernelEx(&cfg, kern, a, p.passes, p.bits, vec);
}

template <int DT, int DG>
cudaError_t launch_sum(const EmbedGradArgs& a, const EmbedGradPlan& p, bool vec, cudaStream_t st) {
    int tiles = (a.D + SUM_COLS - 1) / SUM_COLS;
    if (p.chunks * tiles > 0x7fffffffll) return cudaErrorInvalidValue;
    const unsigned blocks = (unsigned)(p.chunks * tiles);
    EmbedGradArgs b = a;
    void* args[] = {&b, &tiles};
    count_launches(2);
    const cudaError_t e = launch_after(vec ? (const void*)embed_sum_kernel<DT, DG, true> : (const void*)embed_sum_kernel<DT, DG, false>,
                                       blocks, SUM_NT, args, st);
    if (e != cudaSuccess) return e;
    return launch_after(vec ? (const void*)embed_join_kernel<DG, true> : (const void*)embed_join_kernel<DG, false>, blocks,
                        SUM_NT, args, st);
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
    int need = 1;
    while (need < 32 && (unsigned)V >> need) ++need;  // keys 0 .. V
    p.passes = (need + SORT_MAX_BITS - 1) / SORT_MAX_BITS;
    p.bits = (need + p.passes - 1) / p.passes;
    p.chunks = (T + SUM_R - 1) / SUM_R;
    const auto place = [&](size_t bytes) {
        const size_t at = p.scratch;
        p.scratch = (at + bytes + 255) & ~(size_t)255;
        return at;
    };
    for (int i = 0; i < 2; ++i) {
        p.key_at[i] = place(sizeof(unsigned) * T);
        p.pos_at[i] = place(sizeof(unsigned) * T);
    }
    p.part_at = place(sizeof(float) * 2 * (size_t)p.chunks * D);
    return p;
}

cudaError_t launch_embed_grad(EmbedGradArgs a, const EmbedGradPlan& p, unsigned char* scratch, int sms, cudaStream_t st) {
    if (a.T == 0 && a.accumulate) return cudaSuccess;
    for (int i = 0; i < 2; ++i) {
        a.key[i] = reinterpret_cast<unsigned*>(scratch + p.key_at[i]);
        a.pos[i] = reinterpret_cast<unsigned*>(scratch + p.pos_at[i]);
    }
    a.part = reinterpret_cast<float*>(scratch + p.part_at);
    const bool vec_out = whole_rows(a.grad, a.ldg, a.D, a.grad_type);
    const cudaError_t e = a.grad_type == SOT_F32   ? launch_sort<SOT_F32>(a, p, vec_out, sms, st)
                          : a.grad_type == SOT_F16 ? launch_sort<SOT_F16>(a, p, vec_out, sms, st)
                                                   : launch_sort<SOT_BF16>(a, p, vec_out, sms, st);
    if (e != cudaSuccess || a.T == 0) return e;
    const bool vec = vec_out && whole_rows(a.g, a.ld, a.D, a.type);
#define SOT_OUT(DT)                                                            \
    switch (a.grad_type) {                                                     \
        case SOT_F32: return launch_sum<DT, SOT_F32>(a, p, vec, st);           \
        case SOT_F16: return launch_sum<DT, SOT_F16>(a, p, vec, st);           \
        default: return launch_sum<DT, SOT_BF16>(a, p, vec, st);               \
    }
    switch (a.type) {
        case SOT_F32: SOT_OUT(SOT_F32)
        case SOT_F16: SOT_OUT(SOT_F16)
        default: SOT_OUT(SOT_BF16)
    }
#undef SOT_OUT
}

}  // namespace sot
