// k_topk_bf16.cu -- scores, entropies and alternatives, and their gradient, for bf16 logits (topk.cuh).
#include "topk.cuh"

namespace sot {

cudaError_t launch_topk_bf16(const TopkArgs& a, const TopkPlan& p, cudaStream_t st) { return launch_topk_t<SOT_BF16>(a, p, st); }
cudaError_t launch_topk_grad_bf16(const TopkGradArgs& a, int NT, int G, int chunks, cudaStream_t st) {
    return launch_topk_grad_t<SOT_BF16>(a, NT, G, chunks, st);
}

}  // namespace sot
