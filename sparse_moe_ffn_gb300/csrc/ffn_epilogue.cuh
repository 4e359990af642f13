// ffn_epilogue.cuh -- what the gated feed-forward kernels share: operands that lie
// across K, and the activations with their slopes.
#pragma once

#include "linear_epilogue.cuh"
#include "linear_gemm.cuh"

namespace moe {

constexpr int kMnChunk = 64 * kSliceBytes;  // MN-major: 64 rows, 64 values of K

// Shared memory descriptor of an MN-major operand: rows of 64 values along MN
// (128 bytes, swizzled), eight values of K in 1024 bytes, 64 further rows one
// chunk on.  A step of 16 values of K is two groups of eight.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(kMnChunk >> 4) << 16;  // leading: next 64 along MN
    d |= static_cast<uint64_t>(1024 >> 4) << 32;      // stride: next 8 along K
    d |= static_cast<uint64_t>(1) << 46;              // descriptor version (sm_100 family)
    d |= static_cast<uint64_t>(2) << 61;              // 128-byte swizzle
    return d;
}
constexpr uint32_t kIdescAMn = 1u << 15, kIdescBMn = 1u << 16;
constexpr int kStepKMajor = kMmaBytes >> 4;           // 16 values of K, in 16 bytes
constexpr int kStepMnMajor = 16 * kSliceBytes >> 4;

// a = act(v) and d = act'(v).  The logistic function s is exactly 0 where 2^t
// passes the range, so that its product with a large v vanishes.
template <int ACT>
__device__ __forceinline__ void act_slope(float v, float *a, float *d) {
    constexpr float kLog2e = 1.4426950408889634f;
    if (ACT == MOE_ACT_SILU) {
        const float s = rcp_fast(1.f + ex2_fast(v * -kLog2e));
        *a = v * s;
        *d = fmaf(*a, 1.f - s, s);
    } else if (ACT == MOE_ACT_GELU) {
        // q: the normal distribution's upper tail beyond |v| (see gelu)
        const float x = fabsf(v) * 0.70710678118654752f;
        const float t = rcp_fast(fmaf(0.3275911f, x, 1.f));
        float poly = fmaf(t, 1.061405429f, -1.453152027f);
        poly = fmaf(t, poly, 1.421413741f);
        poly = fmaf(t, poly, -0.284496736f);
        poly = fmaf(t, poly, 0.254829592f);
        const float e = ex2_fast(v * v * -0.72134752044448170f);  // e^(-v^2/2)
        const float q = 0.5f * t * poly * e;
        const float c = fminf(fmaxf(v, -64.f), 64.f);
        *a = fmaxf(v, 0.f) - fabsf(c) * q;
        *d = fmaf(c * 0.39894228040143268f, e, v < 0.f ? q : 1.f - q);
    } else if (ACT == MOE_ACT_GELU_TANH) {
        constexpr float k = 1.5957691216057308f;  // 2 sqrt(2 / pi)
        const float vv = v * v;
        const float s = rcp_fast(1.f + ex2_fast(-k * kLog2e * v * fmaf(0.044715f, vv, 1.f)));
        *a = v * s;
        const float r = *a * (1.f - s);  // 0 where z' may be infinite
        *d = r == 0.f ? s : fmaf(r, k * fmaf(0.134145f, vv, 1.f), s);
    } else if (ACT == MOE_ACT_RELU) {
        *a = v < 0.f ? 0.f : v;  // a NaN stays one
        *d = v > 0.f ? 1.f : 0.f;
    } else {
        *a = v;
        *d = 1.f;
    }
}

}  // namespace moe
