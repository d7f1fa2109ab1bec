// What the differential-attention kernels share: the learned weights as the
// kernels take them, and the weight of the second softmax map.
#pragma once

#include "pkv_internal.cuh"

namespace pkv {

struct DiffWeights {
    const float *lambdas;      // [4][D]
    const float *norm_weight;  // [2 D], or null: ones
    float lambda_init, out_scale, eps;  // out_scale = 1 - lambda_init
};

// lambda = exp(l0 . l1) - exp(l2 . l3) + lambda_init, by one warp (every lane
// gets it).  512 numbers at most: each warp that needs it computes it.
template <int D>
__device__ __forceinline__ float diff_lambda(const DiffWeights &w, int lane)
{
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = lane; i < D; i += 32) {
        s1 = fmaf(w.lambdas[i], w.lambdas[D + i], s1);
        s2 = fmaf(w.lambdas[2 * D + i], w.lambdas[3 * D + i], s2);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        s1 += __shfl_xor_sync(kFull, s1, o);
        s2 += __shfl_xor_sync(kFull, s2, o);
    }
    return expf(s1) - expf(s2) + w.lambda_init;
}

pkv_status check_diff_pool(const pkv_pool *pool, const char *who);
// Checks shared by the two entry points; fills *w from the caller's struct.
pkv_status check_diff_args(const pkv_pool *pool, const char *who, const pkv_diff_params *params, DiffWeights *w);

}  // namespace pkv
