// k_topk_f16.cu -- scores, entropies and alternatives, and their gradient, for fp16 logits (topk.cuh).
#include "topk.cuh"

namespace sot {

cudaError_t launch_topk_f16(const TopkArgs& a, const TopkPlan& p, cudaStream_t st) { return launch_topk_t<SOT_F16>(a, p, st); }
cudaError_t launch_topk_grad_f16(const TopkGradArgs& a, int NT, int G, int chunks, cudaStream_t st) {
    return launch_topk_grad_t<SOT_F16>(a, NT, G, chunks, st);
}

}  // namespace sot
