// linear_epilogue.cuh -- what follows the accumulator of moe_linear: scales,
// bias, activation, residual and the one rounding of the output, all in fp32.
#pragma once

#include <cuda_bf16.h>

#include "block_ops.cuh"
#include "ptx.cuh"

namespace moe {

// act(v).  silu(v) = v / (1 + e^-v) and gelu_tanh(v) = v / (1 + e^-2z), z =
// sqrt(2/pi) (v + 0.044715 v^3), since (1 + tanh z) / 2 = 1 / (1 + e^-2z).
// The exponent is capped at 80: beyond it the result is below 1e-32 |v|, and
// the divisor stays in the fast division's range.
template <int ACT>
__device__ __forceinline__ float linear_act(float v) {
    if (ACT == MOE_ACT_SILU) return __fdividef(v, 1.f + __expf(fminf(-v, 80.f)));
    if (ACT == MOE_ACT_GELU) return 0.5f * v * (1.f + erff(v * 0.70710678118654752f));
    if (ACT == MOE_ACT_GELU_TANH) {
        const float z2 = 1.5957691216057308f * v * fmaf(0.044715f * v, v, 1.f);
        return __fdividef(v, 1.f + __expf(fminf(-z2, 80.f)));
    }
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
