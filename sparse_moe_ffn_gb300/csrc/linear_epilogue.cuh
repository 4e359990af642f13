// linear_epilogue.cuh -- the activations of moe_linear, in fp32: each within
// 2^-20 |v| of its formula.
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

// gelu(v) = v (1 + erf(v / sqrt 2)) / 2 = max(v, 0) - |v| Q(|v|), Q the normal
// distribution's upper tail, from Abramowitz and Stegun's rational
// approximation of erf (7.1.26, off by at most 1.5e-7):
//   2 Q(x sqrt 2) = e^(-x^2) (a1 t + a2 t^2 + ... + a5 t^5),  t = 1 / (1 + p x).
// |v| is capped where Q is 0, so that an infinite v gives no 0 * inf.  Off by
// less than 4e-7 |v|; erff took twice the instructions and, in a tile's
// epilogue, 3 us for 128 x 128 outputs a CTA.
__device__ __forceinline__ float gelu(float v) {
    const float x = fabsf(v) * 0.70710678118654752f;
    const float t = rcp_fast(fmaf(0.3275911f, x, 1.f));
    float poly = fmaf(t, 1.061405429f, -1.453152027f);
    poly = fmaf(t, poly, 1.421413741f);
    poly = fmaf(t, poly, -0.284496736f);
    poly = fmaf(t, poly, 0.254829592f);
    const float q = 0.5f * t * poly * ex2_fast(v * v * -0.72134752044448170f);  // e^(-v^2/2)
    return fmaxf(v, 0.f) - fminf(fabsf(v), 64.f) * q;
}

// act(v); gelu_tanh(v) = v / (1 + e^-2z), z = sqrt(2/pi) (v + 0.044715 v^3),
// since (1 + tanh z) / 2 = 1 / (1 + e^-2z).
template <int ACT>
__device__ __forceinline__ float linear_act(float v) {
    constexpr float kLog2e = 1.4426950408889634f;
    if (ACT == MOE_ACT_SILU) return times_logistic(v, v * kLog2e);
    if (ACT == MOE_ACT_GELU) return gelu(v);
    if (ACT == MOE_ACT_GELU_TANH)
        return times_logistic(v, 1.5957691216057308f * kLog2e * v * fmaf(0.044715f * v, v, 1.f));
    if (ACT == MOE_ACT_RELU) return v < 0.f ? 0.f : v;  // a NaN stays one
    return v;
}

// The activation of a thread's outputs, one branch for all of them.
template <int kN>
__device__ __forceinline__ void act_all(int act, float (&v)[kN]) {
    switch (act) {
#define MOE_ACT_CASE(A)                                                              \
    case A:                                                                          \
        _Pragma("unroll") for (int i = 0; i < kN; ++i) v[i] = linear_act<A>(v[i]);   \
        break;
        MOE_ACT_CASE(MOE_ACT_SILU)
        MOE_ACT_CASE(MOE_ACT_GELU)
        MOE_ACT_CASE(MOE_ACT_GELU_TANH)
        MOE_ACT_CASE(MOE_ACT_RELU)
#undef MOE_ACT_CASE
        default: break;
    }
}

}  // namespace moe
