// routed.h -- launch interface of the routed layer for a few tokens.
#pragma once
#include <cuda_runtime.h>

namespace sot {

constexpr int ROUTED_MAX_T = 128;  // tokens of a call
constexpr int ROUTED_MAX_E = 1024;
constexpr int ROUTED_MAX_K = 32;   // experts of a token

struct RoutedArgs {
    const void* x;  // [T, H], row t at element t * ldx
    long long ldx, ldo;
    int T, H, E, F, K, dtype;
    const void* router;   // [E, H]
    const float* bias;    // [E] or NULL
    const void* gate_up;  // [E, 2 F, H]
    const void* down;     // [E, H, F]
    int renorm;
    float scale;
    void* out;       // [T, H]
    float* logits;   // [T, E]
    int* ids;        // [T, K]
    float* weights;  // [T, K]
    // scratch
    float *h, *y;    // [T K, F], [T K, H]
};

struct RoutedTcPlan {
    size_t barrier_at, up_at, down_at, h_at, scratch;
    int zeros;  // words at barrier_at that the scores' kernel writes zeros to
};
struct RoutedPlan {
    bool tc;  // the experts' products on the tensor cores
    size_t h_at, y_at, scratch;
    RoutedTcPlan on_tc;
};
RoutedPlan routed_plan(const RoutedArgs& a, int sms);
cudaError_t launch_routed(RoutedArgs a, const RoutedPlan& p, unsigned char* scratch, int sms, cudaStream_t st);

// The tensor cores' part (k_routed_tc.cu): everything after the scores.
void routed_set_test_hold(int what, unsigned long long wait_ns);  // wait_ns 0: the default
bool routed_tc_fits(const RoutedArgs& a);
RoutedTcPlan routed_tc_plan(const RoutedArgs& a, int sms);
cudaError_t launch_routed_tc(const RoutedArgs& a, const RoutedTcPlan& p, unsigned char* scratch, int sms, cudaStream_t st);

}  // namespace sot
