// ffn_rows.cu -- the gated feed-forward block for up to four tokens: both
// steps (gate/up with their product, then down) stream their weights once,
// from memory straight into registers.
//
// A warp takes two weight rows (an output's gate and up row, or two rows of the
// down projection) and 2048 values of K: 16 loads of 16 bytes a lane, all in
// flight at once.  Rows with more values are shared by the block's warps, whose
// sums are added in a fixed order.  The tokens lie in shared memory.
//
// The down step's first weights are asked for before the kernel waits for the
// gate/up step (programmatic dependent launch): its blocks start where the
// first step's run out, so neither the launch nor the first access's latency
// leaves the memory idle.  They may be read that early because the gate/up
// kernel lets its dependents start only after its own wait: whatever wrote the
// weights has ended then.
#include "gated_ffn.cuh"
#include "linear_epilogue.cuh"
#include "linear_gemm.cuh"

namespace moe {

namespace {

constexpr int kRowsThreads = 256;
constexpr int kRowsWarps = kRowsThreads / 32;
constexpr int kLoads = 8;                    // of 16 bytes: a lane's part of a row segment
constexpr int kSegment = kLoads * 32 * 8;    // values

__device__ __forceinline__ uint4 ld_stream(const uint16_t *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

struct FfnRowsArgs {
    const uint16_t *x;          // [N, K]
    const uint16_t *w0, *w1;    // gated: gate, up [O, K]; down: w0 [O, K]
    int N, K, O;
    int act;
    const uint16_t *residual;   // down, nullable
    uint16_t *gate, *up, *out;  // gate, up nullable
    int per_row;                // warps that share a row's K: a power of two, <= kRowsWarps
    int32_t *status;
};

template <bool kGated, int kTokens>
__global__ void __launch_bounds__(kRowsThreads, 2) ffn_rows_kernel(const FfnRowsArgs a) {
    extern __shared__ uint4 xs[];  // [kTokens][K / 8]
    __shared__ float sums[kRowsWarps][2 * kTokens];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int per_block = kRowsWarps / a.per_row;  // pairs of rows
    const int mine = warp % a.per_row;             // this warp's place in the row
    const int64_t o = static_cast<int64_t>(blockIdx.x) * per_block + warp / a.per_row;
    const int64_t r0 = kGated ? o : 2 * o, r1 = kGated ? o : 2 * o + 1;
    const bool has0 = r0 < a.O, has1 = r1 < a.O;
    const uint16_t *w0 = a.w0 + (has0 ? r0 : 0) * a.K;
    const uint16_t *w1 = (kGated ? a.w1 : a.w0) + (has1 ? r1 : 0) * a.K;
    uint4 b0[kLoads], b1[kLoads];
    auto load = [&](int64_t seg) {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int64_t k = seg * kSegment + (j * 32 + lane) * 8;
            b0[j] = has0 && k < a.K ? ld_stream(w0 + k) : make_uint4(0, 0, 0, 0);
            b1[j] = has1 && k < a.K ? ld_stream(w1 + k) : make_uint4(0, 0, 0, 0);
        }
    };
    if (kGated) griddep_wait();
    griddep_launch_dependents();
    load(mine);
    if (!kGated) griddep_wait();
    if (kGated && blockIdx.x == 0 && threadIdx.x == 0) *a.status = MOE_OK;
    const int groups = a.K / 8;
    for (int i = threadIdx.x; i < a.N * groups; i += kRowsThreads)
        xs[i] = __ldcg(reinterpret_cast<const uint4 *>(a.x) + i);
    __syncthreads();
    float v[2][kTokens];
#pragma unroll
    for (int t = 0; t < kTokens; ++t) v[0][t] = v[1][t] = 0.f;
    for (int64_t seg = mine; seg * kSegment < a.K;) {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int64_t k = seg * kSegment + (j * 32 + lane) * 8;
            if (k >= a.K) break;
            const uint32_t *p0 = reinterpret_cast<const uint32_t *>(&b0[j]);
            const uint32_t *p1 = reinterpret_cast<const uint32_t *>(&b1[j]);
#pragma unroll
            for (int t = 0; t < kTokens; ++t) {
                if (t >= a.N) break;
                const uint4 u = xs[t * groups + k / 8];
                const uint32_t *px = reinterpret_cast<const uint32_t *>(&u);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = unpack_bf16x2(px[i]), g = unpack_bf16x2(p0[i]),
                                 h = unpack_bf16x2(p1[i]);
                    v[0][t] = fmaf(f.x, g.x, v[0][t]);
                    v[0][t] = fmaf(f.y, g.y, v[0][t]);
                    v[1][t] = fmaf(f.x, h.x, v[1][t]);
                    v[1][t] = fmaf(f.y, h.y, v[1][t]);
                }
            }
        }
        seg += a.per_row;
        if (seg * kSegment < a.K) load(seg);
    }
#pragma unroll
    for (int t = 0; t < kTokens; ++t)
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            v[0][t] += __shfl_xor_sync(0xffffffffu, v[0][t], d);
            v[1][t] += __shfl_xor_sync(0xffffffffu, v[1][t], d);
        }
    if (a.per_row > 1) {
        if (lane == 0)
#pragma unroll
            for (int t = 0; t < kTokens; ++t) {
                sums[warp][2 * t] = v[0][t];
                sums[warp][2 * t + 1] = v[1][t];
            }
        __syncthreads();
        if (mine != 0) return;
#pragma unroll
        for (int t = 0; t < kTokens; ++t) {
            v[0][t] = v[1][t] = 0.f;
            for (int w = warp; w < warp + a.per_row; ++w) {
                v[0][t] += sums[w][2 * t];
                v[1][t] += sums[w][2 * t + 1];
            }
        }
    }
    // lane t finishes token t
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int t = 0; t < kTokens; ++t)
        if (lane == t) s0 = v[0][t], s1 = v[1][t];
    if (lane >= a.N || !has0) return;
    const int64_t at = static_cast<int64_t>(lane) * a.O + r0;
    __nv_bfloat16 *out = reinterpret_cast<__nv_bfloat16 *>(a.out) + at;
    if (kGated) {
        float h[1] = {s0};
        act_all(a.act, h);
        *out = __float2bfloat16_rn(h[0] * s1);
        if (a.gate) {
            reinterpret_cast<__nv_bfloat16 *>(a.gate)[at] = __float2bfloat16_rn(s0);
            reinterpret_cast<__nv_bfloat16 *>(a.up)[at] = __float2bfloat16_rn(s1);
        }
    } else {
        // O is a multiple of 8: both rows exist
        if (a.residual) {
            const float2 r = unpack_bf16x2(__ldcg(reinterpret_cast<const uint32_t *>(a.residual + at)));
            s0 += r.x;
            s1 += r.y;
        }
        *reinterpret_cast<uint32_t *>(out) = pack_bf16x2(s0, s1);
    }
}

// The tokens' room in shared memory; two blocks an SM keep theirs.
constexpr int kRowsShared = 64 * 1024;

template <bool kGated, int kTokens>
cudaError_t launch_rows(FfnRowsArgs a, cudaStream_t s) {
    auto kern = ffn_rows_kernel<kGated, kTokens>;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t err = allow_shared(kern, kRowsShared, allowed);
    if (err != cudaSuccess) return err;
    const int segments = (a.K + kSegment - 1) / kSegment;
    a.per_row = 1;
    while (a.per_row < kRowsWarps && a.per_row < segments) a.per_row *= 2;
    const int per_block = kRowsWarps / a.per_row;
    const int64_t pairs = kGated ? a.O : (a.O + 1) / 2;
    return launch_pdl(kern, dim3(static_cast<unsigned>((pairs + per_block - 1) / per_block)),
                      dim3(kRowsThreads), static_cast<size_t>(a.N) * a.K * 2, s, 1, a);
}

template <bool kGated>
cudaError_t launch_tokens(const FfnRowsArgs &a, cudaStream_t s) {
    if (a.N == 1) return launch_rows<kGated, 1>(a, s);
    if (a.N == 2) return launch_rows<kGated, 2>(a, s);
    return launch_rows<kGated, 4>(a, s);
}

}  // namespace

bool ffn_rows_fit(int64_t N, int K) {
    return N <= kFfnRowsTokens && N * K * 2 <= kRowsShared;
}

cudaError_t launch_ffn_rows(FfnOp op, const FfnArgs &a, const uint16_t *x, const uint16_t *w0,
                            const uint16_t *w1, uint16_t *gate, uint16_t *up, cudaStream_t s) {
    const bool gated = op == kFfnGateUp;
    const FfnRowsArgs r = {x,     w0, w1,         static_cast<int>(a.N), gated ? a.H : a.I,
                           gated ? a.I : a.H,     a.act,
                           a.residual, gate, up, a.out[0], 1, a.status};
    return gated ? launch_tokens<true>(r, s) : launch_tokens<false>(r, s);
}

}  // namespace moe
