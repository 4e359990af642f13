// linear.cu -- out = act(x W^T [* sx sw] + bias) + residual.
//
// A plain tiled product on the CUDA cores: 64 x 64 outputs a block, K slices
// of 32 widened to fp32 in shared memory, one fp32 accumulator an output.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "block_ops.cuh"
#include "linear_epilogue.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kT = 64, kKs = 32;

template <bool kFp8>
__device__ __forceinline__ float element(const void *p, int64_t i) {
    if (kFp8) {
        const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t *>(p)[i],
                                                     __NV_E4M3);
        return __half2float(__half(h));
    }
    return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(p)[i]) << 16);
}

template <bool kFp8>
__global__ void __launch_bounds__(256) linear_plain_kernel(const LinearArgs a) {
    __shared__ float xs[kKs][kT + 1], ws[kKs][kT + 1];
    griddep_launch_dependents();
    griddep_wait();
    const int64_t n0 = static_cast<int64_t>(blockIdx.y) * kT;
    const int64_t o0 = static_cast<int64_t>(blockIdx.x) * kT;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < a.K; k0 += kKs) {
        for (int i = threadIdx.x; i < kT * kKs; i += 256) {
            const int r = i / kKs, k = i % kKs;
            const bool in = k0 + k < a.K;
            xs[k][r] = in && n0 + r < a.N ? element<kFp8>(a.x, (n0 + r) * a.K + k0 + k) : 0.f;
            ws[k][r] = in && o0 + r < a.O ? element<kFp8>(a.w, (o0 + r) * a.K + k0 + k) : 0.f;
        }
        __syncthreads();
#pragma unroll 8
        for (int k = 0; k < kKs; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = fmaf(xs[k][ty + 16 * i], ws[k][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + ty + 16 * i, o = o0 + tx + 16 * j;
            if (n < a.N && o < a.O) store_linear(a, n, o, acc[i][j]);
        }
}

}  // namespace

cudaError_t launch_linear(const LinearArgs &a, int num_sms, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>((a.O + kT - 1) / kT),
                    static_cast<unsigned>((a.N + kT - 1) / kT));
    return a.fp8 ? launch_pdl(linear_plain_kernel<true>, grid, dim3(256), 0, s, 1, a)
                 : launch_pdl(linear_plain_kernel<false>, grid, dim3(256), 0, s, 1, a);
}

}  // namespace moe
