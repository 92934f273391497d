// k_topk_f32.cu -- scores, entropies and alternatives, and their gradient, for fp32 logits (topk.cuh).
#include "topk.cuh"

namespace sot {

cudaError_t launch_topk_f32(const TopkArgs& a, const TopkPlan& p, cudaStream_t st) { return launch_topk_t<SOT_F32>(a, p, st); }
cudaError_t launch_topk_grad_f32(const TopkGradArgs& a, int NT, int G, int chunks, cudaStream_t st) {
    return launch_topk_grad_t<SOT_F32>(a, NT, G, chunks, st);
}

}  // namespace sot
