// k_lm_bf16.cu -- the row kernels of the language-model losses for bf16 logits (lm_row.cuh).
#include "lm_row.cuh"

namespace sot {

cudaError_t launch_row_bf16(LmOp op, const LmRowArgs& a, const LmRowPlan& p, const LmRowLaunch& L, cudaStream_t st) {
    return launch_row_t<SOT_BF16>(op, a, p, L, st);
}

}  // namespace sot
