// balance.cu -- the router's load statistics and balance losses, and their
// gradient with respect to the router logits.
//
//   p_n    = softmax(logits_n)        T = tokens that the mask leaves in
//   c_e    = slots (n, j) of those tokens with id e      f_e = c_e / (k T)
//   P_e    = sum_n p_ne / T           lse_n = log sum_e exp(logit_ne)
//   losses = { E sum_e f_e P_e,  sum_n lse_n^2 / T }
//   dlogit_ne = p_ne / T (g_0 E (d_e - sum_j d_j p_nj) + 2 g_1 lse_n),
//               d_e = f_e - 1/E
//
// f is a count and has no gradient.  sum_j p_nj = 1, so taking 1/E off f
// changes no gradient; it removes the cancellation in f_e - sum_j f_j p_nj,
// whose two terms agree in all but the last few percent when the load is
// nearly even.  d_e is formed in 64 bits from the counts.
// A token whose logits are all -inf has p = 0 and lse = 0 and still counts in
// T; a masked token is never read and gets gradient 0.
//
// A row is held by kLanes lanes, 8 values each (kLanes is the power of two
// that covers E); sums over tokens run in registers, then per block in shared
// memory, and the blocks' partial sums are joined in block order in 64 bits:
// no atomics on floats, the same bits every time.
#include <cuda_bf16.h>

#include "block_ops.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kVals = 8;
constexpr int kThreads = 256;
constexpr float kNegInf = -__builtin_huge_valf();

// Value v of lane t of a row is expert 4 (t + kLanes (v / 4)) + v % 4 when
// rows are read four values at a time, else t + kLanes v.
template <int kLanes, bool kVec>
__device__ __forceinline__ int expert_of(int t, int v) {
    return kVec ? 4 * (t + kLanes * (v / 4)) + v % 4 : t + kLanes * v;
}

template <bool kBf16, int kLanes, bool kVec>
__device__ __forceinline__ void load_row(const void *logits, int64_t n, int E, int t,
                                         float (&x)[kVals]) {
    if (kVec) {
#pragma unroll
        for (int c = 0; c < kVals / 4; ++c) {
            const int e = 4 * (t + kLanes * c);
            float4 f = make_float4(kNegInf, kNegInf, kNegInf, kNegInf);
            if (e < E) {
                if (kBf16) {
                    const uint2 u = __ldcg(reinterpret_cast<const uint2 *>(
                        static_cast<const uint16_t *>(logits) + n * E + e));
                    const float2 a = unpack_bf16x2(u.x), b = unpack_bf16x2(u.y);
                    f = make_float4(a.x, a.y, b.x, b.y);
                } else {
                    f = __ldcg(reinterpret_cast<const float4 *>(
                        static_cast<const float *>(logits) + n * E + e));
                }
            }
            x[4 * c] = f.x;
            x[4 * c + 1] = f.y;
            x[4 * c + 2] = f.z;
            x[4 * c + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int v = 0; v < kVals; ++v) {
            const int e = t + kLanes * v;
            x[v] = kNegInf;
            if (e < E) {
                if (kBf16)
                    x[v] = __uint_as_float(
                        static_cast<uint32_t>(
                            __ldcg(static_cast<const uint16_t *>(logits) + n * E + e))
                        << 16);
                else
                    x[v] = __ldcg(static_cast<const float *>(logits) + n * E + e);
            }
        }
    }
}

template <bool kBf16, int kLanes, bool kVec>
__device__ __forceinline__ void store_row(void *out, int64_t n, int E, int t,
                                          const float (&x)[kVals]) {
    if (kVec) {
#pragma unroll
        for (int c = 0; c < kVals / 4; ++c) {
            const int e = 4 * (t + kLanes * c);
            if (e >= E) continue;
            if (kBf16)
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(out) + n * E + e) =
                    make_uint2(pack_bf16x2(x[4 * c], x[4 * c + 1]),
                               pack_bf16x2(x[4 * c + 2], x[4 * c + 3]));
            else
                *reinterpret_cast<float4 *>(static_cast<float *>(out) + n * E + e) =
                    make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
        }
    } else {
#pragma unroll
        for (int v = 0; v < kVals; ++v) {
            const int e = t + kLanes * v;
            if (e >= E) continue;
            if (kBf16)
                static_cast<__nv_bfloat16 *>(out)[n * E + e] = __float2bfloat16_rn(x[v]);
            else
                static_cast<float *>(out)[n * E + e] = x[v];
        }
    }
}

template <int kLanes>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}

template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// x <- softmax of the row; returns its log-sum-exp.  A NaN logit reaches both
// (fmaxf drops it, the sum does not).
template <int kLanes>
__device__ __forceinline__ float softmax_row(float (&x)[kVals]) {
    float top = kNegInf;
#pragma unroll
    for (int v = 0; v < kVals; ++v) top = fmaxf(top, x[v]);
    top = row_max<kLanes>(top);
    if (top == kNegInf) top = 0.f;
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < kVals; ++v) {
        x[v] = __expf(x[v] - top);
        sum += x[v];
    }
    sum = row_sum<kLanes>(sum);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int v = 0; v < kVals; ++v) x[v] *= inv;
    return sum == 0.f ? 0.f : top + logf(sum);
}

template <bool kBf16, int kLanes, bool kVec>
__global__ void __launch_bounds__(kThreads) balance_stats_kernel(const BalanceArgs a) {
    constexpr int kPerWarp = 32 / kLanes;
    constexpr int kWarps = kThreads / 32;
    __shared__ float ps[kWarps][MOE_MAX_EXPERTS];
    __shared__ int cs[MOE_MAX_EXPERTS];
    __shared__ double zs[kWarps];
    __shared__ int ts[kWarps];
    __shared__ int bad;
    griddep_launch_dependents();
    griddep_wait();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int t = lane % kLanes, sub = lane / kLanes;
    for (int e = threadIdx.x; e < MOE_MAX_EXPERTS; e += kThreads) cs[e] = 0;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();

    // this block's tokens [first, last)
    const int64_t per = (a.N + gridDim.x - 1) / gridDim.x;
    const int64_t first = blockIdx.x * per;
    const int64_t last = first + per < a.N ? first + per : a.N;

    float p[kVals];
#pragma unroll
    for (int v = 0; v < kVals; ++v) p[v] = 0.f;
    float z = 0.f;
    int tokens = 0;
    for (int64_t base = first + warp * kPerWarp; base < last; base += kWarps * kPerWarp) {
        const int64_t n = base + sub;
        const bool in = n < last && (!a.mask || __ldcg(a.mask + n));
        float x[kVals];
        if (in) {
            load_row<kBf16, kLanes, kVec>(a.logits, n, a.E, t, x);
        } else {
#pragma unroll
            for (int v = 0; v < kVals; ++v) x[v] = kNegInf;
        }
        const float lse = softmax_row<kLanes>(x);
#pragma unroll
        for (int v = 0; v < kVals; ++v) p[v] += x[v];
        z = fmaf(lse, lse, z);
        tokens += in;
    }
    // rows of the warp, then the warps of the block, in order
#pragma unroll
    for (int d = kLanes; d < 32; d <<= 1) {
#pragma unroll
        for (int v = 0; v < kVals; ++v) p[v] += __shfl_xor_sync(0xffffffffu, p[v], d);
        z += __shfl_xor_sync(0xffffffffu, z, d);
        tokens += __shfl_xor_sync(0xffffffffu, tokens, d);
    }
    if (sub == 0) {
#pragma unroll
        for (int v = 0; v < kVals; ++v) {
            const int e = expert_of<kLanes, kVec>(t, v);
            if (e < a.E) ps[warp][e] = p[v];
        }
    }
    if (lane == 0) {
        zs[warp] = z;
        ts[warp] = tokens;
    }
    // the slots of the block's tokens, side by side
    for (int64_t i = first * a.k + threadIdx.x; i < last * a.k; i += kThreads) {
        if (a.mask && !__ldcg(a.mask + i / a.k)) continue;
        const int id = __ldcg(a.ids + i);
        if (id >= a.E) bad = 1;
        else if (id >= 0) atomicAdd(&cs[id], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += ps[w][e];
        a.part_p[static_cast<int64_t>(blockIdx.x) * a.E + e] = s;
        a.part_c[static_cast<int64_t>(blockIdx.x) * a.E + e] = cs[e];
    }
    if (threadIdx.x == 0) {
        double zz = 0.0;
        int tt = 0;
        for (int w = 0; w < kWarps; ++w) {
            zz += zs[w];
            tt += ts[w];
        }
        a.part_s[blockIdx.x] = {zz, tt, bad};
    }
}

// Joins the blocks' partial sums: kSeg threads an expert, each over every
// kSeg-th block, then in order.
constexpr int kJoinThreads = 1024;

__global__ void __launch_bounds__(kJoinThreads) balance_join_kernel(const BalanceArgs a) {
    __shared__ double ps[kJoinThreads];
    __shared__ int cs[kJoinThreads];
    __shared__ double zs[kJoinThreads / 32], ls[kJoinThreads / 32];
    __shared__ int ts[kJoinThreads / 32], bs[kJoinThreads / 32];
    griddep_launch_dependents();
    griddep_wait();
    const int seg = kJoinThreads / a.E;
    const int e = threadIdx.x % a.E, s = threadIdx.x / a.E;
    double p = 0.0;
    int c = 0;
    if (s < seg) {
#pragma unroll 8
        for (int b = s; b < a.blocks; b += seg) {
            p += __ldcg(a.part_p + static_cast<int64_t>(b) * a.E + e);
            c += __ldcg(a.part_c + static_cast<int64_t>(b) * a.E + e);
        }
    }
    ps[threadIdx.x] = p;
    cs[threadIdx.x] = c;
    double z = 0.0;
    int tokens = 0, bad = 0;
    for (int b = threadIdx.x; b < a.blocks; b += kJoinThreads) {
        z += __ldcg(&a.part_s[b].z);
        tokens += __ldcg(&a.part_s[b].tokens);
        bad |= __ldcg(&a.part_s[b].bad);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        z += __shfl_xor_sync(0xffffffffu, z, d);
        tokens += __shfl_xor_sync(0xffffffffu, tokens, d);
        bad |= __shfl_xor_sync(0xffffffffu, bad, d);
    }
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (lane == 0) {
        zs[warp] = z;
        ts[warp] = tokens;
        bs[warp] = bad;
    }
    __syncthreads();
    double loss = 0.0;
    if (threadIdx.x < a.E) {
        p = 0.0;
        c = 0;
        for (int i = 0; i < seg; ++i) {
            p += ps[i * a.E + threadIdx.x];
            c += cs[i * a.E + threadIdx.x];
        }
        a.counts[threadIdx.x] = c;
        loss = p * c;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) loss += __shfl_xor_sync(0xffffffffu, loss, d);
    if (lane == 0) ls[warp] = loss;
    __syncthreads();
    if (threadIdx.x == 0) {
        z = loss = 0.0;
        tokens = bad = 0;
        for (int w = 0; w < kJoinThreads / 32; ++w) {
            z += zs[w];
            loss += ls[w];
            tokens += ts[w];
            bad |= bs[w];
        }
        const double inv = tokens > 0 ? 1.0 / tokens : 0.0;
        a.losses[0] = static_cast<float>(a.E * loss * inv * inv / a.k);
        a.losses[1] = static_cast<float>(z * inv);
        *a.tokens = tokens;
        *a.status = bad ? MOE_ERR_DEVICE_CHECK : MOE_OK;
    }
}

template <bool kBf16, int kLanes, bool kVec>
__global__ void __launch_bounds__(kThreads) balance_grad_kernel(const BalanceArgs a) {
    constexpr int kPerWarp = 32 / kLanes;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x % 32;
    const int t = lane % kLanes, sub = lane / kLanes;
    const int T = __ldcg(a.tokens);
    const float invT = T > 0 ? 1.f / static_cast<float>(T) : 0.f;
    const float g0 = __ldcg(a.grad) * static_cast<float>(a.E) * invT;
    const float g1 = 2.f * __ldcg(a.grad + 1) * invT;
    float d[kVals];
#pragma unroll
    for (int v = 0; v < kVals; ++v) {
        const int e = expert_of<kLanes, kVec>(t, v);
        d[v] = 0.f;
        if (e < a.E && T > 0)
            d[v] = static_cast<float>(
                static_cast<double>(__ldcg(a.counts_in + e)) / (static_cast<double>(a.k) * T) -
                1.0 / a.E);
    }
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32) * kPerWarp;
    for (int64_t base = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / 32 *
                        kPerWarp;
         base < a.N; base += step) {
        const int64_t n = base + sub;
        const bool in = n < a.N && (!a.mask || __ldcg(a.mask + n));
        float x[kVals];
        if (in) {
            load_row<kBf16, kLanes, kVec>(a.logits, n, a.E, t, x);
        } else {
#pragma unroll
            for (int v = 0; v < kVals; ++v) x[v] = kNegInf;
        }
        const float lse = softmax_row<kLanes>(x);
        float mean = 0.f;
#pragma unroll
        for (int v = 0; v < kVals; ++v) mean = fmaf(d[v], x[v], mean);
        mean = row_sum<kLanes>(mean);
#pragma unroll
        for (int v = 0; v < kVals; ++v)
            x[v] = in ? x[v] * fmaf(g0, d[v] - mean, g1 * lse) : 0.f;
        if (n < a.N) store_row<kBf16, kLanes, kVec>(a.dlogits, n, a.E, t, x);
    }
}

using BalanceKernel = void (*)(BalanceArgs);

template <bool kGrad, bool kBf16, bool kVec>
BalanceKernel kernel_of(int lanes) {
#define MOE_BALANCE_KERNEL(L)                                                \
    (kGrad ? static_cast<void (*)(const BalanceArgs)>(balance_grad_kernel<kBf16, L, kVec>) \
           : static_cast<void (*)(const BalanceArgs)>(balance_stats_kernel<kBf16, L, kVec>))
    switch (lanes) {
        case 1: return MOE_BALANCE_KERNEL(1);
        case 2: return MOE_BALANCE_KERNEL(2);
        case 4: return MOE_BALANCE_KERNEL(4);
        case 8: return MOE_BALANCE_KERNEL(8);
        case 16: return MOE_BALANCE_KERNEL(16);
        default: return MOE_BALANCE_KERNEL(32);
    }
#undef MOE_BALANCE_KERNEL
}

// Rows are read four values at a time when every row starts on such a
// boundary (E a multiple of 4, the arrays aligned), else one at a time.
template <bool kGrad>
cudaError_t launch(const BalanceArgs &a, int blocks, cudaStream_t s) {
    int lanes = 1;
    while (lanes * kVals < a.E) lanes *= 2;
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.logits) |
                         (kGrad ? reinterpret_cast<uintptr_t>(a.dlogits) : 0);
    const bool vec = a.E % 4 == 0 && at % (a.bf16 ? 8 : 16) == 0;
    const BalanceKernel k =
        a.bf16 ? (vec ? kernel_of<kGrad, true, true>(lanes) : kernel_of<kGrad, true, false>(lanes))
               : (vec ? kernel_of<kGrad, false, true>(lanes)
                      : kernel_of<kGrad, false, false>(lanes));
    return launch_pdl(k, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, s, 1, a);
}

int rows_per_pass(int E) {
    int lanes = 1;
    while (lanes * kVals < E) lanes *= 2;
    return kThreads / lanes;
}

}  // namespace

int balance_blocks(int64_t N, int E) {
    const int64_t b = (N + rows_per_pass(E) - 1) / rows_per_pass(E);
    return b < 1 ? 1 : static_cast<int>(b < kBalanceMaxBlocks ? b : kBalanceMaxBlocks);
}

cudaError_t launch_balance(const BalanceArgs &a, cudaStream_t s) {
    cudaError_t e = launch<false>(a, a.blocks, s);
    if (e != cudaSuccess) return e;
    return launch_pdl(balance_join_kernel, dim3(1), dim3(kJoinThreads), 0, s, 1, a);
}

cudaError_t launch_balance_backward(const BalanceArgs &a, int num_sms, cudaStream_t s) {
    int64_t blocks = (a.N + rows_per_pass(a.E) - 1) / rows_per_pass(a.E);
    if (blocks > num_sms * 8) blocks = num_sms * 8;
    return launch<true>(a, static_cast<int>(blocks), s);
}

}  // namespace moe
