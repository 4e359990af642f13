// layernorm.cuh -- residual add + layer norm, and its backward pass.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int kMaxNormH = 65536;  // the longest rows that the operators take

struct LayerNormArgs {
    const void *x, *residual;      // residual nullable
    const void *weight, *bias;     // bias nullable
    int64_t N;
    int H;
    float eps;
    void *residual_out, *out;      // residual_out nullable
    float *mean, *rstd;            // nullable
};

struct LayerNormGradArgs {
    const void *dout, *x, *weight, *dresidual;  // dresidual nullable
    const float *mean, *rstd;
    int64_t N;
    int H;
    void *dx;                       // nullable
    float *dweight, *dbias;         // nullable
    float *part;                    // [blocks][2][H]; for dweight and dbias alone
};

// The sums over tokens of the weight's and the bias's gradients come in this
// many parts at most.
int64_t layernorm_grad_blocks(int64_t N, int H, int num_sms);
// bf16: the type of all arrays but the statistics and dweight, dbias; else fp32
cudaError_t launch_layernorm(const LayerNormArgs &a, int bf16, int num_sms, cudaStream_t s);
cudaError_t launch_layernorm_grad(const LayerNormGradArgs &a, int bf16, int num_sms, int *launches,
                                  cudaStream_t s);

}  // namespace moe
