// k_lm_balance.cu -- the router's balance loss, its per-expert counts and its
// gradient.
//
// With N kept tokens, c_e the number of their choices of expert e and
// f_e = E c_e / (K N):
//   loss[0] = coef / N sum_t sum_e f_e p_te,   loss[1] = z_coef / N sum_t lse_t^2,
//   dx_te = 1/N ( coef p_te (f_e - sum_j f_j p_tj) + 2 z_coef lse_t p_te ).
// The counts come first, then every token's row is read once, its softmax and its
// two sums formed in registers, and its gradient written from them; the sums over
// the tokens are joined in a fixed order.
//   Small batches: one cluster of CTAs does all of it in one launch, counting and
// joining through distributed shared memory.
//   Large ones: a counting kernel leaves each cluster's counts in scratch; the main
// kernel is launched along with it (programmatic dependent launch), reads its
// first rows meanwhile, adds the counts up and goes on; its last CTA to finish joins
// the sums.
//   Weights are formed against 0, which needs no maximum first, and against the
// row's maximum only where their sum leaves the middle of the range.
//   Measured on the GPU: 65536 x 256 bf16, 8 choices, a tenth left out: 19.6 us, 0.50 of
// the copy bandwidth for 66 MB, and 17.2 us where L2 holds them (with the maximum first
// 2 us more); the counting and the waits around it take 5 us of it, the rest is each
// warp's seven dependent steps of load, sums and store.  65536 x 256 fp32: 29.4 us (0.65);
// 65536 x 500 fp16: 36.7 us (0.51); 256 x 64 fp32: 5.7 us.  Loads into shared memory several steps ahead and more, lighter
// CTAs were no faster.
// A power of two of lanes takes a row, four granules of 16 bytes a lane (fewer
// for few experts, more for many), as many rows at a time as fit a warp.
#include <cuda_runtime.h>

#include "kernels.h"
#include "lm.cuh"
#include "lm.h"

namespace sot {

namespace {

constexpr int BAL_NT = 256;
constexpr int CNT_NT = 512;
constexpr int CNT_CL = 8;      // CTAs of a counting cluster
constexpr int CNT_PARTS = 16;  // counting clusters at most
constexpr int SMALL_CL = 8;    // CTAs of the small-batch kernel at most

// Adds the choices of tokens first, first + step, ... to hist; returns how many of
// these tokens are kept.
__device__ __forceinline__ int count_tokens(const LmBalanceArgs& a, long long first, long long step, int* hist) {
    int kept = 0;
    for (long long t = first; t < a.T; t += step) {
        const bool keep = !a.mask || a.mask[t];
        kept += keep;
        for (int k0 = 0; k0 < a.K; k0 += 4) {  // four loads under way
            int id[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) id[j] = k0 + j < a.K ? load_index(a.ids, a.ids_type, t * a.K + k0 + j, a.E) : -1;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (keep && id[j] >= 0) atomicAdd(&hist[id[j]], 1);
        }
    }
    return kept;
}

// A thread's sums over its tokens (compensated): the balance terms, the squares of lse.
struct Sums {
    float2 dot, z;
    __device__ __forceinline__ static void add(float2& s, float v) {
        const float2 t = two_sum(s.x, v);
        s = make_float2(t.x, s.y + t.y);
    }
    // (the compensation of an infinite sum is NaN)
    __device__ __forceinline__ static float value(float2 s) { return fabsf(s.x) < INFINITY ? s.x + s.y : s.x; }
};

__device__ __forceinline__ float group_max(float v, int lanes) {
    if (lanes == 32) return warp_max1(v);
    for (int o = lanes >> 1; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// f in shared memory: coef f_e, zeros around it; where rows may start inside a
// granule, a copy for each number of elements before them, so that a granule's
// experts are always whole aligned float4s.
constexpr int F_LEN = LM_MAX_E + 16;
template <int DT, bool SHIFT>
constexpr int f_copies = SHIFT ? Elem<DT>::N : 1;
// The float4s of a granule's experts lie F_HALF apart, so that neighbouring lanes'
// float4s are neighbours.
constexpr int F_HALF = F_LEN / 2;
template <int DT>
__device__ __forceinline__ int f_at(int e) {
    return Elem<DT>::N == 4 ? e : e / 8 * 4 + (e & 3) + (e & 4 ? F_HALF : 0);
}
template <int DT, bool SHIFT>
__device__ __forceinline__ void put_share(float* f, int e, float v) {
#pragma unroll
    for (int h = 0; h < f_copies<DT, SHIFT>; ++h) f[h * F_LEN + f_at<DT>(e + h)] = v;
}

// The rows of one warp of `warps`: `lanes` lanes a row, R granules a lane, 32 / lanes
// rows at a time, the next rows' loads under way while these are worked on.
// SHIFT: rows may start and end inside a granule.  `counted` is called once the
// first loads are under way, and gives 1/N.
template <int DT, int R, bool SHIFT, class Counted>
__device__ __forceinline__ void balance_rows(const LmBalanceArgs& a, long long warp, long long warps, const float* f,
                                             Sums& out, Counted counted) {
    using T = typename Elem<DT>::T;
    constexpr int N = Elem<DT>::N, H = R * N / 2;  // H pairs a lane
    const int lane = threadIdx.x & 31;
    const int units = (a.E + (SHIFT ? 2 * N - 2 : 0)) / N;
    int lanes = 32;
    while (lanes > 1 && lanes / 2 * R >= units) lanes >>= 1;
    const int per = 32 / lanes, sub = lane & (lanes - 1);
    const long long step = warps * per;
    out = Sums{make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    long long t = warp * per + lane / lanes;
    const auto kept = [&](long long r) { return r < a.T && (!a.mask || a.mask[r]); };
    const auto head_of = [&](const T* row) { return SHIFT ? (int)((uint32_t)(unsigned long long)row & 15u) / (int)sizeof(T) : 0; };
    const auto granules = [&](int head) { return SHIFT ? (head + a.E + N - 1) / N : units; };
    uint4 v[R];
    const auto load = [&](long long r, bool keep) {
        const T* const row = static_cast<const T*>(a.x) + r * a.ld;
        const int head = head_of(row), ng = granules(head);
        const uint4* const src = reinterpret_cast<const uint4*>(row - head);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int g = sub + i * lanes;
            v[i] = keep && g < ng ? src[g] : nothing<DT>();
        }
    };
    bool keep = kept(t), next = kept(t + step);
    load(t, keep);
    const float inv_n = counted();
    // coef f of the experts of granule i, in the order of x
    const auto shares_at = [&](int i, int head, int ng, float2 (&c)[N / 2]) {
        const int g = sub + i * lanes;
        const float4* const q = reinterpret_cast<const float4*>(f + head * F_LEN + g * 4);
#pragma unroll
        for (int k = 0; k < N / 4; ++k) {
            const float4 r = g < ng ? q[k * (F_HALF / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
            c[2 * k] = make_float2(r.x, r.y);
            c[2 * k + 1] = make_float2(r.z, r.w);
        }
    };
    // With whole granules a lane's experts are the same in every row: from 32 of them a
    // lane their shares stay in registers (65536 x 256 bf16 in L2 17.2 us, read again for every
    // row 1.1 us more); with fewer the registers pay for more warps (65536 x 64: 12.3 and 13.0).
    constexpr bool OWN = !SHIFT && H >= 16;
    float2 own[OWN ? H : 1];
    if constexpr (OWN) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float2 c[N / 2];
            shares_at(i, 0, units, c);
#pragma unroll
            for (int k = 0; k < N / 2; ++k) own[i * (N / 2) + k] = c[k];
        }
    }
    for (long long base = warp * per; base < a.T; base += step, t += step) {
        const T* const row = static_cast<const T*>(a.x) + t * a.ld;
        const int head = head_of(row), ng = granules(head);
        float2 x[H];
        const auto open = [&](const uint4 (&v)[R]) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float2 p[N / 2];
                unpack<DT>(v[i], p);
                if (SHIFT) {
                    const int g = sub + i * lanes;
                    if (g == 0 || g == ng - 1) mask_cols<DT>(p, g * N - head, a.E, -INFINITY);
                }
#pragma unroll
                for (int k = 0; k < N / 2; ++k) x[i * (N / 2) + k] = p[k];
            }
        };
        open(v);
        const bool now = keep;
        keep = next;
        if (base + step < a.T) {
            load(t + step, keep);
            next = kept(t + 2 * step);
        }
        const auto shares = [&](int i, float2 (&c)[N / 2]) {
            if constexpr (!OWN) shares_at(i, head, ng, c);
            else {
#pragma unroll
                for (int k = 0; k < N / 2; ++k) c[k] = own[i * (N / 2) + k];
            }
        };
        // The row's sums: of its weights, and of them times the shares.
        const auto add_up = [&](float& s, float& d) {
            float2 sum = make_float2(0.f, 0.f), dots = sum;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float2 c[N / 2];
                shares(i, c);
#pragma unroll
                for (int k = 0; k < N / 2; ++k) {
                    sum = fadd2(sum, x[i * (N / 2) + k]);
                    dots = ffma2(x[i * (N / 2) + k], c[k], dots);
                }
            }
            s = sum.x + sum.y;
            d = dots.x + dots.y;
            for (int o = lanes >> 1; o > 0; o >>= 1) {
                s += __shfl_xor_sync(0xffffffffu, s, o);
                d += __shfl_xor_sync(0xffffffffu, d, o);
            }
        };
        // Weights against 0; where their sum leaves the middle of the range, the row is
        // read again and its weights are formed against its maximum.  (A sum of 2^-10 loses
        // probabilities below 2^-116.)
        float m = 0.f, u = 0.f, s, d;
        bool far = false;
#pragma unroll
        for (int i = 0; i < H; ++i) x[i] = ex2_pair(x[i], 0.f, SOT_LOG2E);
        add_up(s, d);
        const bool again = now && !(s > 0x1p-10f && s < 0x1p24f);
        if (__any_sync(0xffffffffu, again)) {
            const float s0 = s, d0 = d;
            if (again) {
                const uint4* const src = reinterpret_cast<const uint4*>(row - head);
                uint4 w[R];
#pragma unroll
                for (int i = 0; i < R; ++i) w[i] = sub + i * lanes < ng ? src[sub + i * lanes] : nothing<DT>();
                open(w);
                m = -INFINITY;
#pragma unroll
                for (int i = 0; i < H; ++i) m = fmaxf(m, fmaxf(x[i].x, x[i].y));
            }
            m = group_max(m, lanes);
            if (again) {
                u = __fmul_rn(m, SOT_LOG2E);
                far = is_far(u);
                if (far) u = 0.f;
#pragma unroll
                for (int i = 0; i < H; ++i)
                    x[i] = far ? make_float2(weight_of(x[i].x, m, SOT_LOG2E), weight_of(x[i].y, m, SOT_LOG2E))
                               : ex2_pair(x[i], u, SOT_LOG2E);
            }
            add_up(s, d);
            if (!again) {
                s = s0;
                d = d0;
            }
        }
        const float inv_s = __fdividef(1.f, s), dot = d * inv_s;  // coef sum f p
        // (a row of nothing but -inf is far, and has no sum)
        const float lse = !far ? (u + __log2f(s)) * SOT_LN2 : s > 0.f ? m + __logf(s) : NAN;
        if (now && sub == 0) {
            Sums::add(out.dot, dot);
            Sums::add(out.z, lse * lse);
        }
        if (!a.grad || t >= a.T) continue;
        T* const grow = static_cast<T*>(a.grad) + t * a.ldg;
        const bool aligned = !SHIFT || same_granules<T>(row, grow);
        // (the weights of a token that is left out are 0)
        // (k first: the coefficient times lse may be out of range where their share of N tokens is not)
        const float k = now ? inv_n * inv_s : 0.f, bias = now ? fmaf(2.f * k * a.z_coef, lse, -dot * k) : 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int g = sub + i * lanes;
            float2 c[N / 2], p[N / 2];
            shares(i, c);
#pragma unroll
            for (int j = 0; j < N / 2; ++j)
                p[j] = fmul2(x[i * (N / 2) + j], ffma2(c[j], make_float2(k, k), make_float2(bias, bias)));
            if (g < ng) {
                if (SHIFT) store_cols<DT>(grow, g * N - head, a.E, p, aligned);
                else reinterpret_cast<uint4*>(grow)[g] = pack<DT>(p);
            }
        }
    }
}

// The two sums of a CTA, in every lane of warp 0 (fixed order).
template <int NT>
__device__ __forceinline__ float2 block_sums(const Sums& s, float (&red)[2][NT / 32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float d = warp_sum(Sums::value(s.dot)), z = warp_sum(Sums::value(s.z));
    if (lane == 0) {
        red[0][warp] = d;
        red[1][warp] = z;
    }
    __syncthreads();
    if (warp != 0) return make_float2(0.f, 0.f);
    return make_float2(warp_sum(lane < NT / 32 ? red[0][lane] : 0.f), warp_sum(lane < NT / 32 ? red[1][lane] : 0.f));
}
// f_e = E c_e / (K N): the factor of c_e.
__device__ __forceinline__ float share_of(const LmBalanceArgs& a, int kept) {
    return (float)a.E / ((float)a.K * (float)max(kept, 1));
}
// coef is already in the dot sums.  A z loss that is not wanted is 0 also where the squares leave the range.
__device__ __forceinline__ void write_loss(const LmBalanceArgs& a, float dot, float z, int kept) {
    a.loss[0] = kept > 0 ? dot / (float)kept : 0.f;
    a.loss[1] = kept > 0 && !(a.z_coef == 0.f && z == INFINITY) ? a.z_coef * (z / (float)kept) : 0.f;
}
// A 32-bit value of another CTA's shared memory.
__device__ __forceinline__ int cluster_load(const int* local_ptr, uint32_t rank) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(smem_u32(local_ptr), rank)) : "memory");
    return v;
}

// ---- large batches ------------------------------------------------------------
// Each cluster leaves its counts and its number of kept tokens in scratch.
__global__ void __launch_bounds__(CNT_NT) lm_count_kernel(LmBalanceArgs a) {
    __shared__ int hist[LM_MAX_E + 1];  // the last: kept tokens
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t rank = cluster_rank();
    const int part = blockIdx.x / CNT_CL;
    for (int e = threadIdx.x; e <= a.E; e += CNT_NT) hist[e] = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0u;
    __syncthreads();
    const int n = count_tokens(a, (long long)blockIdx.x * CNT_NT + threadIdx.x, (long long)gridDim.x * CNT_NT, hist);
    if (n) atomicAdd(&hist[a.E], n);
    cluster_sync();
    for (int e = rank * CNT_NT + threadIdx.x; e <= a.E; e += CNT_CL * CNT_NT) {
        int c = 0;
#pragma unroll
        for (int p = 0; p < CNT_CL; ++p) c += cluster_load(&hist[e], p);
        a.part_counts[part * (a.E + 1) + e] = c;
    }
    cluster_sync();  // no CTA leaves while a peer may still read it
}

template <int DT, int R, bool SHIFT>
__global__ void __launch_bounds__(BAL_NT, R <= 2 ? 4 : R <= 4 ? 2 : 1) lm_balance_kernel(LmBalanceArgs a) {
    __shared__ __align__(16) float f[f_copies<DT, SHIFT> * F_LEN];
    __shared__ float red[2][BAL_NT / 32];
    __shared__ bool last;
    int kept = 0;
    Sums s;
    for (int i = threadIdx.x; i < f_copies<DT, SHIFT> * F_LEN; i += BAL_NT) f[i] = 0.f;
    __syncthreads();
    balance_rows<DT, R, SHIFT>(a, (long long)blockIdx.x * (BAL_NT / 32) + (threadIdx.x >> 5),
                             (long long)gridDim.x * (BAL_NT / 32), f, s, [&]() {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        const auto total = [&](int e) {  // all loads under way at once
            int c[CNT_PARTS], sum = 0;
#pragma unroll
            for (int p = 0; p < CNT_PARTS; ++p) c[p] = p < a.parts ? a.part_counts[p * (a.E + 1) + e] : 0;
#pragma unroll
            for (int p = 0; p < CNT_PARTS; ++p) sum += c[p];
            return sum;
        };
        kept = total(a.E);
        const float k = a.coef * share_of(a, kept);
        for (int e = threadIdx.x; e < a.E; e += BAL_NT) {
            const int c = total(e);
            if (blockIdx.x == 0) a.counts[e] = c;
            put_share<DT, SHIFT>(f, e, (float)c * k);
        }
        __syncthreads();
        return kept > 0 ? 1.f / (float)kept : 0.f;
    });
    const float2 v = block_sums<BAL_NT>(s, red);
    if (threadIdx.x == 0) {
        a.part_sums[blockIdx.x] = v;
        __threadfence();
        last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (last) {
        __threadfence();
        Sums all{make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        for (int b = threadIdx.x; b < (int)gridDim.x; b += BAL_NT) {
            const float2 w = __ldcg(&a.part_sums[b]);
            Sums::add(all.dot, w.x);
            Sums::add(all.z, w.y);
        }
        const float2 w = block_sums<BAL_NT>(all, red);
        if (threadIdx.x == 0) write_loss(a, w.x, w.y, kept);
    }
}

// ---- small batches --------------------------------------------------------------
template <int DT, int R, bool SHIFT>
__global__ void __launch_bounds__(CNT_NT) lm_balance_small_kernel(LmBalanceArgs a) {
    __shared__ int hist[LM_MAX_E + 1];  // the last: kept tokens
    __shared__ __align__(16) float f[f_copies<DT, SHIFT> * F_LEN];
    __shared__ float red[2][CNT_NT / 32];
    __shared__ float sums[SMALL_CL][2];
    const uint32_t rank = cluster_rank();
    const int CL = gridDim.x;
    for (int e = threadIdx.x; e <= a.E; e += CNT_NT) hist[e] = 0;
    for (int i = threadIdx.x; i < f_copies<DT, SHIFT> * F_LEN; i += CNT_NT) f[i] = 0.f;
    __syncthreads();
    const int n = count_tokens(a, (long long)rank * CNT_NT + threadIdx.x, (long long)CL * CNT_NT, hist);
    if (n) atomicAdd(&hist[a.E], n);
    int kept = 0;
    Sums s;
    balance_rows<DT, R, SHIFT>(a, (long long)rank * (CNT_NT / 32) + (threadIdx.x >> 5), (long long)CL * (CNT_NT / 32), f, s, [&]() {
        if (CL > 1) cluster_sync();
        else __syncthreads();
        for (int p = 0; p < CL; ++p) kept += cluster_load(&hist[a.E], p);
        const float k = a.coef * share_of(a, kept);
        for (int e = threadIdx.x; e < a.E; e += CNT_NT) {
            int c = 0;
            for (int p = 0; p < CL; ++p) c += cluster_load(&hist[e], p);
            if (rank == 0) a.counts[e] = c;
            put_share<DT, SHIFT>(f, e, (float)c * k);
        }
        __syncthreads();
        return kept > 0 ? 1.f / (float)kept : 0.f;
    });
    const float2 v = block_sums<CNT_NT>(s, red);
    if (threadIdx.x == 0) {
        const uint32_t to = cluster_addr(smem_u32(sums[rank]), 0);
        cluster_store(to, v.x);
        cluster_store(to + 4, v.y);
    }
    if (CL > 1) cluster_sync();  // the sums are there, and nobody reads a CTA's counts any more
    else __syncthreads();
    if (rank == 0 && threadIdx.x == 0) {
        Sums t{make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        for (int p = 0; p < CL; ++p) {
            Sums::add(t.dot, sums[p][0]);
            Sums::add(t.z, sums[p][1]);
        }
        write_loss(a, Sums::value(t.dot), Sums::value(t.z), kept);
    }
}

template <int DT, int R, bool SHIFT>
cudaError_t launch_r(const LmBalanceArgs& a, int blocks, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(blocks, 1, 1);
    if (a.parts == 0) {
        cfg.blockDim = dim3(CNT_NT, 1, 1);
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = blocks;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        count_launches(1);
        return cudaLaunchKernelEx(&cfg, lm_balance_small_kernel<DT, R, SHIFT>, a);
    }
    count_launches(2);
    cfg.gridDim = dim3(a.parts * CNT_CL, 1, 1);
    cfg.blockDim = dim3(CNT_NT, 1, 1);
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CNT_CL;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, lm_count_kernel, a);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(blocks, 1, 1);
    cfg.blockDim = dim3(BAL_NT, 1, 1);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    return cudaLaunchKernelEx(&cfg, lm_balance_kernel<DT, R, SHIFT>, a);
}

template <int DT, bool SHIFT>
cudaError_t launch_s(const LmBalanceArgs& a, int granules, int blocks, cudaStream_t st) {
    if (granules <= 4) return launch_r<DT, 1, SHIFT>(a, blocks, st);
    if (granules <= 8) return launch_r<DT, 2, SHIFT>(a, blocks, st);
    if constexpr (DT == SOT_F32 || SHIFT) {
        if (granules > 128) {
            if constexpr (DT == SOT_F32 && SHIFT)
                if (granules > 256) return launch_r<DT, 16, SHIFT>(a, blocks, st);
            return launch_r<DT, 8, SHIFT>(a, blocks, st);
        }
    }
    return launch_r<DT, 4, SHIFT>(a, blocks, st);
}

template <int DT>
cudaError_t launch_d(const LmBalanceArgs& a, int blocks, cudaStream_t st) {
    using T = typename Elem<DT>::T;
    constexpr int N = Elem<DT>::N;
    const auto whole = [](const void* p, long long ld) {
        return (unsigned long long)p % 16 == 0 && ld * (long long)sizeof(T) % 16 == 0;
    };
    if (a.E % N == 0 && whole(a.x, a.ld) && (!a.grad || whole(a.grad, a.ldg))) return launch_s<DT, false>(a, a.E / N, blocks, st);
    return launch_s<DT, true>(a, (a.E + 2 * N - 2) / N, blocks, st);
}

}  // namespace

// Scratch of a call: none for a small batch.
LmBalancePlan lm_balance_plan(long long T, int E, int K, int dtype, int sms) {
    LmBalancePlan p = {};
    const long long bytes = T * ((long long)E * (dtype == SOT_F32 ? 4 : 2) + 4ll * K);
    // One cluster up to 512 KB of logits and choices: 900 x 256 bf16 with 8 choices takes 7.8 us
    // on the GPU against 8.1 us, and one launch without scratch instead of two launches
    // and an allocation is 5 us less on the host.
    if (bytes <= 512 * 1024) {
        const long long want = (T + CNT_NT / 32 - 1) / (CNT_NT / 32);
        p.blocks = 1;
        while (p.blocks < SMALL_CL && p.blocks < want) p.blocks *= 2;
        return p;
    }
    const long long cw = (T + CNT_CL * CNT_NT - 1) / (CNT_CL * CNT_NT), w = (T + BAL_NT / 32 - 1) / (BAL_NT / 32);
    p.parts = (int)(cw < CNT_PARTS ? cw : CNT_PARTS);
    p.blocks = (int)(w < 2ll * sms ? w : 2ll * sms);
    p.sums_at = 0;
    p.counts_at = sizeof(float2) * p.blocks;
    p.ticket_at = p.counts_at + sizeof(int) * (size_t)p.parts * (E + 1);
    p.scratch = p.ticket_at + sizeof(unsigned);
    return p;
}

cudaError_t launch_lm_balance(LmBalanceArgs a, const LmBalancePlan& p, unsigned char* scratch, cudaStream_t st) {
    a.parts = p.parts;
    if (p.parts) {
        a.part_sums = reinterpret_cast<float2*>(scratch + p.sums_at);
        a.part_counts = reinterpret_cast<int*>(scratch + p.counts_at);
        a.ticket = reinterpret_cast<unsigned*>(scratch + p.ticket_at);
    }
    switch (a.dtype) {
        case SOT_F32: return launch_d<SOT_F32>(a, p.blocks, st);
        case SOT_F16: return launch_d<SOT_F16>(a, p.blocks, st);
        default: return launch_d<SOT_BF16>(a, p.blocks, st);
    }
}

}  // namespace sot
