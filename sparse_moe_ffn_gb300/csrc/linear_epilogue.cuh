// linear_epilogue.cuh -- what follows the accumulator of moe_linear: scales,
// bias, activation, residual and the one rounding of the output, all in fp32.
#pragma once

#include <cuda_bf16.h>

#include "block_ops.cuh"
#include "ptx.cuh"

namespace moe {

// 2^x and 1/x in one instruction each (off by two steps at most; what is below
// 2^-126 is 0).
__device__ __forceinline__ float ex2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// v / (1 + e^-z), with z log2(e) given.  The exponent is capped at 126, so
// that the reciprocal stays in range; beyond it the result is below 1e-36 |v|.
__device__ __forceinline__ float times_logistic(float v, float z_log2e) {
    return v * rcp_fast(1.f + ex2_fast(fminf(-z_log2e, 126.f)));
}

// act(v); gelu_tanh(v) = v / (1 + e^-2z), z = sqrt(2/pi) (v + 0.044715 v^3),
// since (1 + tanh z) / 2 = 1 / (1 + e^-2z).
template <int ACT>
__device__ __forceinline__ float linear_act(float v) {
    constexpr float kLog2e = 1.4426950408889634f;
    if (ACT == MOE_ACT_SILU) return times_logistic(v, v * kLog2e);
    if (ACT == MOE_ACT_GELU) return 0.5f * v * (1.f + erff(v * 0.70710678118654752f));
    if (ACT == MOE_ACT_GELU_TANH)
        return times_logistic(v, 1.5957691216057308f * kLog2e * v * fmaf(0.044715f * v, v, 1.f));
    if (ACT == MOE_ACT_RELU) return v < 0.f ? 0.f : v;  // a NaN stays one
    return v;
}

__device__ __forceinline__ float linear_act(int act, float v) {
    switch (act) {
        case MOE_ACT_SILU: return linear_act<MOE_ACT_SILU>(v);
        case MOE_ACT_GELU: return linear_act<MOE_ACT_GELU>(v);
        case MOE_ACT_GELU_TANH: return linear_act<MOE_ACT_GELU_TANH>(v);
        case MOE_ACT_RELU: return linear_act<MOE_ACT_RELU>(v);
        default: return v;
    }
}

}  // namespace moe
