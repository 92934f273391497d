// topk.h -- launch interface of the scores of given tokens with entropies and the
// best alternatives, and of their gradient.
#pragma once
#include <cuda_runtime.h>

namespace sot {

constexpr int TOPK_MAX_K = 1024;  // alternatives of a row (what a distillation takes as its teacher's entries)

struct TopkArgs {
    const void* x;  // logits, row r at element r * ld
    long long T, ld;
    int V, dtype;
    float tau, inv_hi, inv_lo;  // temperature; its inverse in two floats
    double inv_tau;
    const void* target;  // NULL: every row takes part, no logp
    int target_type;
    int K;
    float *logp, *lse, *entropy;  // any may be NULL
    int* ids;                     // [T, K] or NULL
    float* top;                   // [T, K] or NULL
};

struct TopkGradArgs {
    const void* x;
    long long T, ld, ldg;
    int V, dtype;
    float tau;
    const void* target;  // NULL: every row takes part
    int target_type;
    const float *lse, *entropy;
    const float *g_logp, *g_entropy;  // NULL: 0
    const int* ids;                   // [T, K]
    const float* g_top;               // [T, K]; NULL: 0
    int K;
    void* grad;
};

// Whether the chunk maxima of a row of V logits fit shared memory.
bool topk_fits(int dtype, int V, int K);
cudaError_t launch_topk(const TopkArgs& a, int sms, cudaStream_t st);
cudaError_t launch_topk_grad(const TopkGradArgs& a, int sms, cudaStream_t st);

}  // namespace sot
