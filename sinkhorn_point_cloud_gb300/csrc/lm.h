// lm.h -- launch interface of the language-model training losses: row kernels
// over logits (token log-probabilities, distillation from a teacher's top
// entries, clipped policy loss), the paired preference loss and the router's
// balance loss.
#pragma once
#include <cuda_runtime.h>

namespace sot {

enum LmOp { LM_LOGPROB = 0, LM_POLICY = 1, LM_DISTILL = 2 };

// Largest number of teacher entries per row and of experts (registers and
// shared memory are sized by them).
constexpr int LM_MAX_K = 1024;
constexpr int LM_MAX_E = 1024;

struct LmRowArgs {
    const void* x;  // logits, row r at element r * ld
    long long T, ld, ldg;
    int V, dtype;
    void* grad;  // NULL: losses only
    float tau;
    double inv_tau;
    float inv_hi, inv_lo;  // the same in two floats
    const float* weight;  // NULL: every row weighs 1/T
    // token log-probability and policy loss
    const void* target;
    int target_type;
    float *logp, *lse;
    const float *old_logp, *ref_logp, *adv;
    float clip_lo, clip_hi, kl_coef;
    float *loss, *kl;
    // distillation
    const void* ids;
    int ids_type, K;
    const void* teacher;
    int teacher_type, tail;
};

struct LmGradArgs {
    const void* x;
    long long T, ld, ldg;
    int V, dtype;
    float tau;
    const void* target;
    int target_type;
    const float *lse, *g;
    void* grad;
};

struct LmPrefArgs {
    const float *logp, *ref_logp;
    const void* target;  // NULL: every token counts
    int target_type;
    const long long* offsets;  // [2P + 1]
    int P;
    long long T;
    float beta, smoothing, scale;
    int average;
    float *loss, *margin, *grad;
};

struct LmBalanceArgs {
    const void* x;
    long long T, ld, ldg;
    int E, dtype;
    const void* ids;
    int ids_type, K;
    const unsigned char* mask;  // NULL: every token counts
    float coef, z_coef;
    int* counts;
    float* loss;  // [2]
    void* grad;   // NULL: losses only
    // scratch of a large batch (parts = 0: a small one)
    int parts;
    float2* part_sums;
    int* part_counts;
    unsigned* ticket;
};

// Whether the tail's marks of a row of V logits fit a CTA's shared memory.
bool lm_tail_fits(int dtype, int V, int K);
cudaError_t launch_lm_row(LmOp op, const LmRowArgs& a, int sms, cudaStream_t st);
cudaError_t launch_lm_grad(const LmGradArgs& a, int sms, cudaStream_t st);
cudaError_t launch_lm_preference(const LmPrefArgs& a, cudaStream_t st);
struct LmBalancePlan {
    int blocks, parts;
    size_t sums_at, counts_at, ticket_at, scratch;
};
LmBalancePlan lm_balance_plan(long long T, int E, int K, int dtype, int sms);
cudaError_t launch_lm_balance(LmBalanceArgs a, const LmBalancePlan& p, unsigned char* scratch, cudaStream_t st);

}  // namespace sot
