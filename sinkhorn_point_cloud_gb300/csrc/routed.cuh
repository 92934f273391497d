// routed.cuh -- device helpers of the routed layer: the choice of a token's experts.
#pragma once
#include "lm.cuh"
#include "routed.h"

namespace sot {

// The K best of E scores r (one warp): lane k gets the k-th expert (-1: none left) and its weight.
template <int R>
__device__ __forceinline__ void choose_of(const float* r, int E, int K, bool renorm, float scale, int& id, float& weight) {
    const int lane = threadIdx.x & 31;
    unsigned key[R];  // 0: -inf, or no expert
    float m = -INFINITY, bad = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        key[i] = 0u;
        if (i * 32 < E) {
            const int e = i * 32 + lane;
            const float v = e < E ? __ldcg(r + e) : -INFINITY;
            if (!(v < INFINITY)) bad = 1.f;
            m = fmaxf(m, v);
            if (v > -INFINITY) key[i] = ord_encode(v + 0.f);
        }
    }
    m = warp_max1(m);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (key[i]) sum += expf(ord_decode(key[i]) - m);
    sum = warp_sum(sum);
    bad = warp_max1(bad);
    float chosen = 0.f, mine = 0.f;
    id = -1;
    for (int k = 0; k < K && bad == 0.f; ++k) {
        unsigned best = 0;
#pragma unroll
        for (int i = 0; i < R; ++i) best = max(best, key[i]);
        best = __reduce_max_sync(0xffffffffu, best);
        if (best == 0) break;
        int at = 0x7fffffff;
#pragma unroll
        for (int i = R - 1; i >= 0; --i)
            if (key[i] == best) at = i * 32 + lane;
        at = __reduce_min_sync(0xffffffffu, at);
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (i * 32 + lane == at) key[i] = 0;
        const float v = expf(ord_decode(best) - m);
        chosen += v;
        if (lane == k) {
            id = at;
            mine = v;
        }
    }
    weight = bad != 0.f ? NAN : id < 0 ? 0.f : mine / (renorm ? chosen : sum) * scale;
}
// (R scores a lane)
__device__ __forceinline__ void routed_choose(const float* r, int E, int K, bool renorm, float scale, int& id, float& weight) {
    if (E <= 64) choose_of<2>(r, E, K, renorm, scale, id, weight);
    else if (E <= 256) choose_of<8>(r, E, K, renorm, scale, id, weight);
    else choose_of<ROUTED_MAX_E / 32>(r, E, K, renorm, scale, id, weight);
}

}  // namespace sot
