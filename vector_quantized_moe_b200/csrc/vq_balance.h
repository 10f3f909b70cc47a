// Arguments of the balance-loss kernels (vq_balance.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace vq {

struct BalanceArgs {
    const float *logits;    // [T, E]
    const int32_t *ids;     // [T, k]
    const uint8_t *mask;    // [T] or NULL
    float *loss, *probs;    // [1], [E]
    int32_t *counts;        // [E + 1]
    float *part_sums;       // [parts][E]
    int32_t *part_counts;   // [parts][E + 1]
    int T, E, k;
    float coef;
};

struct BalanceBwdArgs {
    const float *logits;
    const int32_t *counts;
    const uint8_t *mask;
    const float *dloss;     // NULL: 1
    float *dlogits;
    int T, E, k;
    float coef;
};

size_t balance_workspace_bytes(int T, int E);
cudaError_t launch_balance(const BalanceArgs &a, void *ws, cudaStream_t s);
cudaError_t launch_balance_bwd(const BalanceBwdArgs &a, cudaStream_t s);

}  // namespace vq
