// grad_clip.cu -- the norm of a set of gradient tensors of any sizes, bf16 and
// fp32 together, and the set scaled to a largest norm:
//
//   norm = sqrt(sum g^2),  out = g * (norm <= max_norm ? 1 : max_norm / norm)
//
// The tensors' table is a kernel parameter, so nothing is copied to the device
// first.  A tensor is cut into chunks of kChunk values; every block takes an
// equal run of the chunks of all tensors, and finds its first tensor by
// bisection.
//
// Squares: 32 values at most are summed in fp32 and the sum is added in 64
// bits, one addition of those for 32 values.  Where the fp32 sum is beyond its
// range, or so small that squares may have been lost, the values in hand are
// squared again in 64 bits.
#include <cuda_bf16.h>

#include "cluster.cuh"
#include "grad_clip.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 8192;  // values

template <int kMax>
struct GradTable {
    const void *src[kMax];
    void *dst[kMax];
    int64_t size[kMax];
    int first[kMax + 1];  // the chunks before each tensor
    uint8_t flags[kMax];  // see below
    int n;
};
constexpr int kSrcBf16 = 1, kDstBf16 = 2, kVector = 4;

// The tensor that chunk `c` belongs to: the last one that starts at or before it.
template <int kMax>
__device__ __forceinline__ int tensor_of(const GradTable<kMax> &t, int c) {
    int lo = 0, hi = t.n;  // first[lo] <= c < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (t.first[mid] <= c) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <int kN>
__device__ __forceinline__ double sum_squares(const float (&v)[kN]) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kN; ++i) s = fmaf(v[i], v[i], s);
    // 2^-80: what underflow takes from the sum is below 2^-60 of it
    if (s >= 8.271806125530277e-25f && s < __int_as_float(0x7f800000)) return s;
    double d = 0.0;
#pragma unroll
    for (int i = 0; i < kN; ++i)
        if (v[i] != 0.f) d = fma(static_cast<double>(v[i]), static_cast<double>(v[i]), d);
    return d;
}

__device__ __forceinline__ void unpack8(const uint4 &u, float *v) {
    const float2 a = unpack_bf16x2(u.x), b = unpack_bf16x2(u.y), c = unpack_bf16x2(u.z),
                 d = unpack_bf16x2(u.w);
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    v[4] = c.x, v[5] = c.y, v[6] = d.x, v[7] = d.y;
}

// Eight fp32 values by one access of 32 bytes, which are whole sectors: two of
// 16 a lane would ask for each sector twice.
__device__ __forceinline__ void ld_f32x8(const float *p, float *v) {
    asm volatile("ld.global.L1::no_allocate.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                   "=f"(v[6]), "=f"(v[7])
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void st_f32x8(float *p, const float *v) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]),
                 "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}

// Eight values from value i of a tensor on (32-byte aligned in fp32, else 16).
__device__ __forceinline__ void load8(const void *src, bool bf16, int64_t i, float *v) {
    if (bf16) {
        unpack8(__ldcg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(src) + i)), v);
    } else {
        ld_f32x8(static_cast<const float *>(src) + i, v);
    }
}

__device__ __forceinline__ float load1(const void *src, bool bf16, int64_t i) {
    return bf16 ? __uint_as_float(static_cast<uint32_t>(
                      __ldcg(static_cast<const uint16_t *>(src) + i))
                  << 16)
                : __ldcg(static_cast<const float *>(src) + i);
}

__device__ __forceinline__ void store8(void *dst, bool bf16, int64_t i, const float *v) {
    if (bf16) {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(dst) + i) =
            make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                       pack_bf16x2(v[6], v[7]));
    } else {
        st_f32x8(static_cast<float *>(dst) + i, v);
    }
}

__device__ __forceinline__ void store1(void *dst, bool bf16, int64_t i, float v) {
    if (bf16) static_cast<uint16_t *>(dst)[i] = static_cast<uint16_t>(pack_bf16x2(v, 0.f));
    else static_cast<float *>(dst)[i] = v;
}

// The chunks of block blockIdx.x, one by one: visit(tensor, first value, values).
// kBack: from the last one back.
template <bool kBack, int kMax, typename Visit>
__device__ __forceinline__ void for_chunks(const GradTable<kMax> &t, const Visit &visit) {
    const int64_t chunks = t.first[t.n];
    const int from = static_cast<int>(chunks * blockIdx.x / gridDim.x);
    const int to = static_cast<int>(chunks * (blockIdx.x + 1) / gridDim.x);
    if (from >= to) return;
    int k = tensor_of(t, kBack ? to - 1 : from);
    for (int i = 0; i < to - from; ++i) {
        const int c = kBack ? to - 1 - i : from + i;
        if (kBack)
            while (c < t.first[k]) --k;
        else
            while (c >= t.first[k + 1]) ++k;
        const int64_t begin = static_cast<int64_t>(c - t.first[k]) * kChunk;
        const int64_t left = t.size[k] - begin;
        visit(k, begin, left < kChunk ? static_cast<int>(left) : kChunk);
    }
}

__device__ __forceinline__ double block_sum(double v) {
    __shared__ double sums[kThreads / 32];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) v += sums[w];
    return v;
}

// parts[blockIdx.x] = the block's sum of squares; or, with `norm`, the root of
// the whole (one block).
template <int kMax>
__global__ void __launch_bounds__(kThreads)
    grad_norm_kernel(const __grid_constant__ GradTable<kMax> t, double *parts, float *norm) {
    griddep_launch_dependents();
    griddep_wait();
    double sum = 0.0;
    for_chunks<false>(t, [&](int k, int64_t begin, int n) {
        const bool bf16 = t.flags[k] & kSrcBf16;
        const void *src = t.src[k];
        int i = 0;
        if (t.flags[k] & kVector) {
            for (; i + 32 * kThreads <= n; i += 32 * kThreads) {
                float v[32];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    load8(src, bf16, begin + i + 8 * (j * kThreads + threadIdx.x), v + 8 * j);
                sum += sum_squares(v);
            }
            for (; i + 8 * threadIdx.x + 8 <= n; i += 8 * kThreads) {
                float v[8];
                load8(src, bf16, begin + i + 8 * threadIdx.x, v);
                sum += sum_squares(v);
            }
            i = n / 8 * 8;
        }
        for (i += threadIdx.x; i < n; i += kThreads) {
            const float v[1] = {load1(src, bf16, begin + i)};
            sum += sum_squares(v);
        }
    });
    sum = block_sum(sum);
    if (threadIdx.x == 0) {
        if (norm) *norm = static_cast<float>(sqrt(sum));
        else parts[blockIdx.x] = sum;
    }
}

// A small set in one launch: a cluster of eight blocks whose warps take pieces of
// 1024 values each (a piece's loads are all in flight at once), and whose sums
// are joined through shared memory, block by block in order.
constexpr int kSmallBlocks = 8;
constexpr int kSmallThreads = 1024;
constexpr int kPiece = 1024;

__global__ void __launch_bounds__(kSmallThreads)
    grad_norm_small_kernel(const __grid_constant__ GradTable<64> t, float *norm) {
    __shared__ double sums[kSmallThreads / 32];
    __shared__ double block;
    griddep_launch_dependents();
    griddep_wait();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = static_cast<int>(cluster_ctarank());
    double sum = 0.0;
    // neighbouring pieces go to different blocks
    for (int c = warp * kSmallBlocks + rank; c < t.first[t.n]; c += kSmallBlocks * kSmallThreads / 32) {
        const int k = tensor_of(t, c);
        const int64_t begin = static_cast<int64_t>(c - t.first[k]) * kPiece;
        const int64_t left = t.size[k] - begin;
        const int n = left < kPiece ? static_cast<int>(left) : kPiece;
        const bool bf16 = t.flags[k] & kSrcBf16;
        const void *src = t.src[k];
        const bool vec = t.flags[k] & kVector;
        float v[32];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = 8 * (j * 32 + lane);
            if (vec && i + 8 <= n) {
                load8(src, bf16, begin + i, v + 8 * j);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[8 * j + e] = i + e < n ? load1(src, bf16, begin + i + e) : 0.f;
            }
        }
        sum += sum_squares(v);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) sums[warp] = sum;
    __syncthreads();
    if (warp == 0) {
        sum = sums[lane];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane == 0) block = sum;
    }
    cluster_barrier();
    if (rank == 0 && warp == 0) {
        sum = 0.0;
        if (lane < kSmallBlocks) {
            const uint32_t lo = ld_cluster_u32(&block, lane);
            const uint32_t hi = ld_cluster_u32(reinterpret_cast<const uint32_t *>(&block) + 1, lane);
            sum = __hiloint2double(static_cast<int>(hi), static_cast<int>(lo));
        }
#pragma unroll
        for (int d = kSmallBlocks / 2; d > 0; d >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane == 0) *norm = static_cast<float>(sqrt(sum));
    }
    cluster_barrier();  // the blocks' sums have been read
}

__global__ void __launch_bounds__(kThreads)
    grad_norm_finish_kernel(const double *parts, int64_t n, float *norm) {
    griddep_launch_dependents();
    griddep_wait();
    double sum = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) sum += __ldcg(parts + i);
    sum = block_sum(sum);
    if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(sum));
}

template <int kMax>
__global__ void __launch_bounds__(kThreads)
    clip_grads_kernel(const __grid_constant__ GradTable<kMax> t, const float *norm,
                      float max_norm) {
    griddep_launch_dependents();
    griddep_wait();
    const float size = __ldcg(norm);
    const float factor = size <= max_norm ? 1.f : max_norm / size;
    // backwards: what the norm's kernel read last may still be in L2
    for_chunks<true>(t, [&](int k, int64_t begin, int n) {
        const bool bf16 = t.flags[k] & kSrcBf16, out_bf16 = t.flags[k] & kDstBf16;
        const void *src = t.src[k];
        void *dst = t.dst[k];
        if (factor == 1.f && src == dst) return;  // as it is
        int i = 0;
        if (t.flags[k] & kVector) {
            for (; i + 32 * kThreads <= n; i += 32 * kThreads) {
                float v[32];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    load8(src, bf16, begin + i + 8 * (j * kThreads + threadIdx.x), v + 8 * j);
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] *= factor;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    store8(dst, out_bf16, begin + i + 8 * (j * kThreads + threadIdx.x), v + 8 * j);
            }
            for (; i + 8 * threadIdx.x + 8 <= n; i += 8 * kThreads) {
                float v[8];
                load8(src, bf16, begin + i + 8 * threadIdx.x, v);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] *= factor;
                store8(dst, out_bf16, begin + i + 8 * threadIdx.x, v);
            }
            i = n / 8 * 8;
        }
        for (i += threadIdx.x; i < n; i += kThreads)
            store1(dst, out_bf16, begin + i, load1(src, bf16, begin + i) * factor);
    });
}

// ---------------------------------------------------------------- launchers

// Tensors [at, at + kMax) of the set.
template <int kMax>
GradTable<kMax> table_of(const GradSet &g, int64_t at, int chunk = kChunk) {
    GradTable<kMax> t;
    t.n = static_cast<int>(g.n - at < kMax ? g.n - at : kMax);
    t.first[0] = 0;
    for (int i = 0; i < t.n; ++i) {
        const void *src = g.grads[at + i];
        void *dst = g.out ? g.out[at + i] : nullptr;
        const int64_t size = g.sizes[at + i];
        t.src[i] = src;
        t.dst[i] = dst;
        t.size[i] = size;
        t.first[i + 1] = t.first[i] + static_cast<int>((size + chunk - 1) / chunk);
        t.flags[i] = (g.bf16[at + i] ? kSrcBf16 : 0) |
                     (g.out && g.out_bf16[at + i] ? kDstBf16 : 0) |
                     (reinterpret_cast<uintptr_t>(src) % (g.bf16[at + i] ? 16 : 32) == 0 &&
                              (!g.out || reinterpret_cast<uintptr_t>(dst) %
                                                 (g.out_bf16[at + i] ? 16 : 32) ==
                                             0)
                          ? kVector
                          : 0);
    }
    return t;
}

// Four blocks an SM are what fits at once; sets of more than 128 chunks an SM
// take 32, eight after one another, which evens out who ends last (50 M values:
// 55.4 us for norm and clipping with 4, 63.6 with 16; 604 M: 776 us with 4, 747
// with 16, 738 with 32).
int blocks_for(int chunks, int num_sms) {
    const int most = num_sms * (chunks > 128 * num_sms ? kGradBlocksPerSm : 4);
    return chunks < most ? (chunks > 0 ? chunks : 1) : most;
}

template <int kMax>
cudaError_t norm_launch(const GradSet &g, int64_t at, double *parts, float *norm, int num_sms,
                        int *blocks, cudaStream_t s) {
    const GradTable<kMax> t = table_of<kMax>(g, at);
    *blocks = blocks_for(t.first[t.n], num_sms);
    return launch_pdl(grad_norm_kernel<kMax>, dim3(static_cast<unsigned>(*blocks)), dim3(kThreads),
                      0, s, 1, t, parts, *blocks == 1 ? norm : nullptr);
}

template <int kMax>
cudaError_t clip_launch(const GradSet &g, int64_t at, const float *norm, float max_norm,
                        int num_sms, cudaStream_t s) {
    const GradTable<kMax> t = table_of<kMax>(g, at);
    if (t.first[t.n] == 0) return cudaSuccess;
    return launch_pdl(clip_grads_kernel<kMax>,
                      dim3(static_cast<unsigned>(blocks_for(t.first[t.n], num_sms))),
                      dim3(kThreads), 0, s, 1, t, norm, max_norm);
}

constexpr int kSmallTable = 64;  // a table of 1.9 KB; the large one has 15 KB
// Four pieces a warp of the cluster: one more launch costs what a dozen more do.
constexpr int kSmallPieces = 4 * kSmallBlocks * kSmallThreads / 32;

}  // namespace

int64_t grad_norm_parts(int64_t n, int num_sms) {
    return (n + kGradTable - 1) / kGradTable * num_sms * kGradBlocksPerSm;
}

cudaError_t launch_grad_norm(const GradSet &g, double *parts, float *norm, int num_sms,
                             int *launches, cudaStream_t s) {
    if (g.n <= kSmallTable) {
        int64_t pieces = 0;  // a table counts them in 32 bits
        for (int64_t i = 0; i < g.n; ++i) pieces += (g.sizes[i] + kPiece - 1) / kPiece;
        if (pieces <= kSmallPieces) {
            *launches += 1;
            return launch_pdl(grad_norm_small_kernel, dim3(kSmallBlocks), dim3(kSmallThreads), 0, s,
                              kSmallBlocks, table_of<kSmallTable>(g, 0, kPiece), norm);
        }
    }
    int64_t used = 0;
    for (int64_t at = 0; at == 0 || at < g.n; at += kGradTable) {
        float *direct = g.n <= kGradTable ? norm : nullptr;  // a single block's sum is the whole
        int blocks = 0;
        const cudaError_t err =
            g.n <= kSmallTable
                ? norm_launch<kSmallTable>(g, at, parts + used, direct, num_sms, &blocks, s)
                : norm_launch<kGradTable>(g, at, parts + used, direct, num_sms, &blocks, s);
        if (err != cudaSuccess) return err;
        *launches += 1;
        if (blocks == 1 && direct) return cudaSuccess;
        used += blocks;
    }
    *launches += 1;
    return launch_pdl(grad_norm_finish_kernel, dim3(1), dim3(kThreads), 0, s, 1,
                      static_cast<const double *>(parts), used, norm);
}

cudaError_t launch_clip_grads(const GradSet &g, const float *norm, float max_norm, int num_sms,
                              int *launches, cudaStream_t s) {
    for (int64_t at = 0; at < g.n; at += kGradTable) {
        const cudaError_t err =
            g.n <= kSmallTable ? clip_launch<kSmallTable>(g, at, norm, max_norm, num_sms, s)
                               : clip_launch<kGradTable>(g, at, norm, max_norm, num_sms, s);
        if (err != cudaSuccess) return err;
        *launches += 1;
    }
    return cudaSuccess;
}

}  // namespace moe
