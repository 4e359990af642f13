// ffn_rows.cu -- the gated feed-forward block for one or two tokens: both
// steps (gate/up with their product, then down) stream their weights once,
// from memory straight into registers.
//
// A warp takes a step of K at a time: 1024 values of an output's gate and up
// row, or 2048 of a row of the down projection, 8 loads of 16 bytes a lane.  Two
// steps are in flight; a step's registers are asked for again as soon as it is
// used, across outputs too, and the blocks stay (two an SM), so that the memory
// always has more than a step of every warp.  (One step of twice the size a
// block, blocks that come and go: one token of 2048 x 8192 took 21.6 us, so
// 21.0, and 19.5 with the first weights fetched to L2 ahead.)  The warps of a
// block share long rows where there are few; their sums are added in a fixed
// order.  The tokens lie in shared memory.
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
constexpr int kLoads = 8;  // of 16 bytes: a lane's part of a step

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
    constexpr int kRows = kGated ? 2 : 1;             // weight rows of an output
    constexpr int kRowLoads = kLoads / kRows;
    constexpr int kStep = kRowLoads * 32 * 8;         // values of K
    extern __shared__ uint4 xs[];                     // [kTokens][K / 8]
    __shared__ float sums[2][kRowsWarps][kRows * kTokens];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int per_block = kRowsWarps / a.per_row;     // outputs of a group
    const int mine = warp % a.per_row;                // this warp's place in the row
    const int steps = (a.K + kStep - 1) / kStep;
    const int groups = (a.O + per_block - 1) / per_block;
    const int words = a.K / 8;

    // the next step to ask for
    int load_group = blockIdx.x, load_step = mine;
    uint4 w[2][kRows][kRowLoads];
    auto load = [&](uint4(&b)[kRows][kRowLoads]) {
        const int64_t o = static_cast<int64_t>(load_group) * per_block + warp / a.per_row;
        const bool has = load_group < groups && o < a.O;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const uint16_t *row = (r == 0 ? a.w0 : a.w1) + (has ? o : 0) * a.K;
#pragma unroll
            for (int j = 0; j < kRowLoads; ++j) {
                const int at = load_step * (kStep / 8) + j * 32 + lane;
                b[r][j] = has && at < words ? ld_stream(row + 8 * static_cast<int64_t>(at))
                                            : make_uint4(0, 0, 0, 0);
            }
        }
        load_step += a.per_row;
        if (load_step >= steps) {
            load_step = mine;
            load_group += gridDim.x;
        }
    };
    // the tokens first where they are there already: behind the weights they
    // would arrive last
    const int all = a.N * words;
    int i = threadIdx.x;
    uint4 token = make_uint4(0, 0, 0, 0);
    if (kGated) {
        // what is there already starts on its way to L2 while the kernel before
        // ends (L2 holds no stale copies, whoever writes the weights)
        if (lane < 2 * kRows) {
            const int64_t o = static_cast<int64_t>(blockIdx.x) * per_block + warp / a.per_row;
            const int k = (mine + lane / kRows * a.per_row) * kStep;
            const int n = min(kStep, a.K - k);
            if (o < a.O && n > 0)
                prefetch_l2_bulk((lane % kRows == 0 ? a.w0 : a.w1) + o * a.K + k, 2 * n);
        }
        griddep_wait();
        if (i < all) token = ld_stream(a.x + 8 * i);
    }
    griddep_launch_dependents();
    load(w[0]);
    load(w[1]);
    if (!kGated) {
        // the next two steps on their way to L2
        int g = load_group, q = load_step;
        for (int j = 0; j < 2; ++j) {
            const int64_t o = static_cast<int64_t>(g) * per_block + warp / a.per_row;
            const int n = min(kStep, a.K - q * kStep);
            if (lane == j && g < groups && o < a.O && n > 0)
                prefetch_l2_bulk(a.w0 + o * a.K + q * kStep, 2 * n);
            q += a.per_row;
            if (q >= steps) {
                q = mine;
                g += gridDim.x;
            }
        }
        griddep_wait();
        if (i < all) token = ld_stream(a.x + 8 * i);
    }
    if (kGated && blockIdx.x == 0 && threadIdx.x == 0) *a.status = MOE_OK;
    if (i < all) xs[i] = token;
    for (i += kRowsThreads; i < all; i += kRowsThreads)
        xs[i] = __ldcg(reinterpret_cast<const uint4 *>(a.x) + i);
    __syncthreads();

    float v[kRows][kTokens];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int t = 0; t < kTokens; ++t) v[r][t] = 0.f;
    int group = blockIdx.x, step = mine, turn = 0;
    // uses a step's weights; ends the output with its last one
    auto use = [&](const uint4(&b)[kRows][kRowLoads]) {
#pragma unroll
        for (int j = 0; j < kRowLoads; ++j) {
            const int at = step * (kStep / 8) + j * 32 + lane;
            if (at >= words) break;
#pragma unroll
            for (int t = 0; t < kTokens; ++t) {
                if (t >= a.N) break;
                const uint4 u = xs[t * words + at];
                const uint32_t *px = reinterpret_cast<const uint32_t *>(&u);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = unpack_bf16x2(px[i]);
#pragma unroll
                    for (int r = 0; r < kRows; ++r) {
                        const float2 g =
                            unpack_bf16x2(reinterpret_cast<const uint32_t *>(&b[r][j])[i]);
                        v[r][t] = fmaf(f.x, g.x, v[r][t]);
                        v[r][t] = fmaf(f.y, g.y, v[r][t]);
                    }
                }
            }
        }
        step += a.per_row;
        if (step < steps) return;
        float s[kRows];  // lane t: the sums of token t
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            s[r] = 0.f;
#pragma unroll
            for (int t = 0; t < kTokens; ++t) {
                float f = v[r][t];
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) f += __shfl_xor_sync(0xffffffffu, f, d);
                if (lane == t) s[r] = f;
                v[r][t] = 0.f;
            }
        }
        if (a.per_row > 1) {
            // two buffers in turn: a warp can be one output ahead, never two
            if (lane < kTokens)
#pragma unroll
                for (int r = 0; r < kRows; ++r) sums[turn][warp][r * kTokens + lane] = s[r];
            __syncthreads();
            if (mine == 0 && lane < kTokens)
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    s[r] = 0.f;
                    for (int q = warp; q < warp + a.per_row; ++q)
                        s[r] += sums[turn][q][r * kTokens + lane];
                }
            turn ^= 1;
        }
        const int64_t o = static_cast<int64_t>(group) * per_block + warp / a.per_row;
        if (mine == 0 && lane < a.N && o < a.O) {
            const int64_t at = lane * static_cast<int64_t>(a.O) + o;
            float y;
            if constexpr (kGated) {
                float h[1] = {s[0]};
                act_all(a.act, h);
                y = h[0] * s[1];
                if (a.gate) {
                    reinterpret_cast<__nv_bfloat16 *>(a.gate)[at] = __float2bfloat16_rn(s[0]);
                    reinterpret_cast<__nv_bfloat16 *>(a.up)[at] = __float2bfloat16_rn(s[1]);
                }
            } else {
                y = s[0];
                if (a.residual)
                    y += __uint_as_float(static_cast<uint32_t>(__ldcg(a.residual + at)) << 16);
            }
            reinterpret_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(y);
        }
        step = mine;
        group += gridDim.x;
    };
    while (group < groups) {
        use(w[0]);
        load(w[0]);
        if (group >= groups) break;
        use(w[1]);
        load(w[1]);
    }
}

// The tokens' room in shared memory; two blocks an SM keep theirs.
constexpr int kRowsShared = 64 * 1024;

template <bool kGated, int kTokens>
cudaError_t launch_rows(FfnRowsArgs a, int num_sms, cudaStream_t s) {
    auto kern = ffn_rows_kernel<kGated, kTokens>;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t err = allow_shared(kern, kRowsShared, allowed);
    if (err != cudaSuccess) return err;
    // warps that share a row: enough rows for all warps of two blocks an SM
    const int steps = (a.K + (kGated ? 1023 : 2047)) / (kGated ? 1024 : 2048);
    const int64_t warps = 2 * static_cast<int64_t>(num_sms) * kRowsWarps;
    a.per_row = 1;
    while (a.per_row < kRowsWarps && 2 * a.per_row <= steps &&
           2 * static_cast<int64_t>(a.O) * a.per_row <= warps)
        a.per_row *= 2;
    const int per_block = kRowsWarps / a.per_row;
    const int64_t groups = (static_cast<int64_t>(a.O) + per_block - 1) / per_block;
    const int64_t blocks = groups < 2 * num_sms ? groups : 2 * num_sms;
    return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(kRowsThreads),
                      static_cast<size_t>(a.N) * a.K * 2, s, 1, a);
}

template <bool kGated>
cudaError_t launch_tokens(const FfnRowsArgs &a, int num_sms, cudaStream_t s) {
    return a.N == 1 ? launch_rows<kGated, 1>(a, num_sms, s)
                    : launch_rows<kGated, 2>(a, num_sms, s);
}

}  // namespace

bool ffn_rows_fit(int64_t N, int K) {
    return N <= kFfnRowsTokens && N * K * 2 <= kRowsShared;
}

cudaError_t launch_ffn_rows(FfnOp op, const FfnArgs &a, const uint16_t *x, const uint16_t *w0,
                            const uint16_t *w1, uint16_t *gate, uint16_t *up, int num_sms,
                            cudaStream_t s) {
    const bool gated = op == kFfnGateUp;
    const FfnRowsArgs r = {x,     w0, w1,         static_cast<int>(a.N), gated ? a.H : a.I,
                           gated ? a.I : a.H,     a.act,
                           a.residual, gate, up, a.out[0], 1, a.status};
    return gated ? launch_tokens<true>(r, num_sms, s) : launch_tokens<false>(r, num_sms, s);
}

}  // namespace moe
