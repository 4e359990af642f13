// block_ops.cuh -- launchers of the operators around the layer: rows to e4m3
// (with add + RMSNorm), the linear product with its epilogue, and the router's
// balance loss.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels.cuh"
#include "moe.h"

namespace moe {

// ------------------------------------------- rows to e4m3, add + RMSNorm first

// Longest row that stays in one block's registers (1024 threads, 8 chunks of
// 8 elements each).
constexpr int kMaxRowH = 65536;

// residual, residual_out and normed may be null
cudaError_t launch_add_rmsnorm_fp8(const uint16_t *x, const uint16_t *residual, const uint16_t *w,
                                   int64_t N, int H, float eps, int gemma, uint16_t *residual_out,
                                   uint8_t *q, float *scale, uint16_t *normed, int num_sms,
                                   cudaStream_t s);
cudaError_t launch_quantize_fp8(const uint16_t *x, int64_t N, int H, uint8_t *q, float *scale,
                                int num_sms, cudaStream_t s);

// ------------------------------------------------------------------ linear

// out[n, o] = act(sum_k x[n, k] w[o, k] * x_scale[n] * w_scale[o] + bias[o])
//             + residual[n, o]; scales only for e4m3 operands, bias and
// residual nullable
struct LinearArgs {
    const void *x, *w;  // bf16, or e4m3 when fp8
    const float *x_scale, *w_scale;
    const uint16_t *bias, *residual;
    void *out;  // bf16, or fp32 when out_fp32
    int64_t N;
    int K, O;
    int act;
    int fp8, out_fp32;
    int32_t *status;  // nullable
};

// ------------------------------------------------------------ balance loss

constexpr int kBalanceCluster = 8;       // blocks that join their sums on chip
// As many clusters as fit at two blocks an SM: a cluster stays within one group
// of SMs, and 38 of them (304 blocks) took a second wave (131072 x 128: 25.8 us
// forward, 20.3 with 32).
constexpr int kBalanceMaxClusters = 32;

struct BalancePart {
    float z;      // sum of lse^2 over the cluster's tokens
    int tokens;
    int bad;      // an id >= E was seen
};

struct BalanceArgs {
    const void *logits;  // [N, E] fp32, or bf16
    int bf16;
    const int32_t *ids;      // [N, k]
    const uint8_t *mask;     // [N] or null
    int64_t N;
    int E, k;
    // forward
    int clusters;
    float *part_p;           // [clusters, E]
    int32_t *part_c;         // [clusters, E]
    BalancePart *part_s;     // [clusters]
    float *losses;           // [2]
    int32_t *counts;         // [E]
    int32_t *tokens;         // [1]; read by the backward pass
    int32_t *status;
    // backward
    const int32_t *counts_in;
    const float *grad;       // [2]
    void *dlogits;
};

int balance_clusters(int64_t N, int E);
// Whether clusters stay at the 8 blocks that every device has room for.
void balance_portable_clusters(bool only);
cudaError_t launch_balance(const BalanceArgs &a, int *launches, cudaStream_t s);
cudaError_t launch_balance_backward(const BalanceArgs &a, int num_sms, cudaStream_t s);

}  // namespace moe
