// k_topk.cu -- how the rows of the scores kernel (topk.cuh) and of its gradient are cut.
#include <cuda_runtime.h>

#include <algorithm>

#include "kernels.h"
#include "topk.cuh"

namespace sot {

namespace {

int pow2_from(int n) {
    int p = 2;
    while (p < n) p *= 2;
    return p;
}

void topk_plan(bool whole, const TopkArgs& a, int sms, TopkPlan* p) {
    const int N = a.dtype == SOT_F32 ? 4 : 8;
    const long long total = ((long long)a.V + (whole ? N - 1 : 2 * N - 2)) / N;  // granules of a row
    int CL = 1;
    // A warp takes a short row where there are more of them than CTAs of 128 threads find room, or little to select
    // (V = 4000 bf16, K = 64: 300 rows 15.3 us, with a CTA a row 8.6; 2400 rows 19.8 and 21.6.  V = 1000, K = 8: 1200 rows 6.9 and 9.2).
    if (total <= 512 && a.K <= 256 && (a.T > 8ll * sms || (total <= 128 && a.K <= 16))) p->NT = 32;
    else if (a.T < sms || total > 8192) p->NT = 256;
    else p->NT = 128;
    // Few rows: cut a row further, up to eight granules a thread and a CTA for each SM, as far as the
    // slices' alternatives can be joined in one place.
    if (p->NT > 32 && a.T < sms)
        while (CL < ROW_MAX_CL && a.T * CL <= sms && total > CL * 2048ll && CL * a.K <= 1024) CL *= 2;
    // (a slice's chunk maxima have to fit shared memory)
    while (CL < ROW_MAX_CL && total > CL * 262144ll) CL *= 2;
    const long long G = (total + CL - 1) / CL;
    // Chunks of a batch of granules where that leaves twice as many chunks as alternatives, otherwise single ones.
    const int batch = p->NT == 32 ? BATCH_OF<32> : BATCH_OF<256>;
    p->U = G >= 2ll * batch * a.K || G > 16384 ? batch : 1;
    p->L.CL = CL;
    p->L.G = (int)G;
    p->L.chunks = a.K ? (int)((G + p->U * p->NT - 1) / (p->U * p->NT)) * p->NT : 0;
    p->L.join = a.K ? pow2_from(CL * a.K) : 0;
    const auto place = [&](int candidates) {
        p->L.cap = a.K ? pow2_from(std::max(candidates, 256)) : 0;
        // candidates, chunks to look at again, and the chunks' maxima, where the candidates are put in order later
        const long long last = std::max<long long>(sizeof(unsigned) * p->L.chunks, sizeof(unsigned long long) * p->L.cap);
        long long bytes = (long long)(sizeof(unsigned long long) + sizeof(int)) * p->L.cap + last;
        if (CL > 1 && a.K) bytes = std::max(bytes, (long long)sizeof(unsigned long long) * 2 * p->L.join + (long long)sizeof(int) * BINS);
        p->L.bytes = (int)(bytes < TOPK_MAX_SMEM + 1 ? bytes : TOPK_MAX_SMEM + 1);
    };
    // As many candidates of a slice as all slices' alternatives together; where the chunks' maxima leave no room for them, twice
    // its own (more of them are looked for with a higher threshold).
    place(std::max(CL, 2) * a.K);
    if (p->L.bytes > TOPK_MAX_SMEM) place(2 * a.K);
}

}  // namespace

bool topk_fits(int dtype, int V, int K) {
    TopkArgs a = {};
    a.T = 1ll << 31;
    a.dtype = dtype;
    a.V = V;
    a.K = K;
    TopkPlan p;
    topk_plan(false, a, 1, &p);
    return p.L.bytes * (p.NT == 32 ? TEAMS<32> : 1) <= TOPK_MAX_SMEM;
}

cudaError_t launch_topk(const TopkArgs& a, int sms, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    TopkPlan p;
    const bool whole = (unsigned long long)a.x % 16 == 0 && a.ld % (a.dtype == SOT_F32 ? 4 : 8) == 0;
    topk_plan(whole, a, sms, &p);
    if (a.T * p.L.CL > 0x7fffffffll) return cudaErrorInvalidValue;
    count_launches(1);
    switch (a.dtype) {
        case SOT_F32: return launch_topk_f32(a, p, st);
        case SOT_F16: return launch_topk_f16(a, p, st);
        default: return launch_topk_bf16(a, p, st);
    }
}

cudaError_t launch_topk_grad(const TopkGradArgs& a, int sms, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    const int N = a.dtype == SOT_F32 ? 4 : 8;
    const long long total = ((long long)a.V + 2 * N - 2) / N;
    // Up to 512 granules 64 threads take a row (8192 x 2000 bf16: 38 us with 256).  Otherwise sixteen granules a thread, or
    // eight or four where that leaves SMs without work; more where the grid's limit asks for it.
    const int NT = total <= 512 ? 64 : 256;
    long long most = (total + 4095) / 4096 * a.T >= 24ll * sms ? 4096 : (total + 2047) / 2048 * a.T >= 2ll * sms ? 2048 : 1024;
    while ((total + most - 1) / most * a.T > 0x7fffffffll) most *= 2;
    const int chunks = (int)((total + most - 1) / most);
    const long long G = ((total + chunks - 1) / chunks + NT - 1) / NT * NT;
    count_launches(1);
    switch (a.dtype) {
        case SOT_F32: return launch_topk_grad_f32(a, NT, (int)G, chunks, st);
        case SOT_F16: return launch_topk_grad_f16(a, NT, (int)G, chunks, st);
        default: return launch_topk_grad_bf16(a, NT, (int)G, chunks, st);
    }
}

}  // namespace sot
