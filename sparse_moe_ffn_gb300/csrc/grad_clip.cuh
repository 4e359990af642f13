// grad_clip.cuh -- the norm of a set of gradient tensors, and their clipping.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

// Tensors that one launch takes: their table is a kernel parameter.
constexpr int kGradTable = 512;
constexpr int kGradBlocksPerSm = 32;  // at most, see blocks_for

struct GradSet {
    const void *const *grads;
    const int64_t *sizes;
    const uint8_t *bf16;
    int64_t n;
    void *const *out;          // clipping only
    const uint8_t *out_bf16;
};

int64_t grad_norm_parts(int64_t n, int num_sms);  // doubles
cudaError_t launch_grad_norm(const GradSet &g, double *parts, float *norm, int num_sms,
                             int *launches, cudaStream_t s);
cudaError_t launch_clip_grads(const GradSet &g, const float *norm, float max_norm, int num_sms,
                              int *launches, cudaStream_t s);

}  // namespace moe
