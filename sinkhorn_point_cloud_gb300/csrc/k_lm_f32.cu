// k_lm_f32.cu -- the row kernels of the language-model losses for f32 logits (lm_row.cuh).
#include "lm_row.cuh"

namespace sot {

cudaError_t launch_row_f32(LmOp op, const LmRowArgs& a, const LmRowPlan& p, const LmRowLaunch& L, cudaStream_t st) {
    return launch_row_t<SOT_F32>(op, a, p, L, st);
}

}  // namespace sot
