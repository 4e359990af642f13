// linear_split.cu -- moe_linear for small and middling batches: a tile of 128
// outputs x kBN tokens whose K is shared by the CTAs of a cluster.
//
// With few tokens the call streams the weights once, and there are too few
// tiles of 128 outputs to keep every SM loading; the cluster's CTAs take a
// part of K each.  The weights are on the MMA's M side (128 rows, all real
// but in the last tile), the tokens on its N side, which goes down to 16.
// Each CTA writes its partial sums straight into the shared memory of the CTA
// that owns the token (tokens are dealt out in equal runs), one cluster
// barrier later every CTA adds the parts of its own tokens in rank order and
// stores them: no workspace, no second kernel, the same bits every time.
// Going through shared memory also turns the tile: neighbouring threads then
// hold neighbouring outputs of a token.
//
//   warp 0  producer: TMA copies; up to kStages slices in flight
//   warp 1  TMEM and the MMAs
//   all     read the accumulator (warp w the TMEM lanes = outputs 32 (w % 4) ..
//           + 31), then add and store; bias, scales and residual are fetched
//           before the accumulator is waited for
//
// What bounds it, measured on a GB300: latency (launch, first TMA copy, cluster
// barrier: about 3.5 us) and then the weights' bytes, one CTA an SM (a tile's
// stages fill its shared memory).  One token of 2048 values to 8192 outputs in
// e4m3 (16.8 MB): 5.0 us, 3365 GB/s, 128 CTAs on 152 SMs; one of 8192 to 2048 in
// bf16 (33.6 MB): 9.5 us, 3500 GB/s; 64 x 2048 x 128 in bf16 to fp32: 3.8
// us; 333 x 1000 x 1111 in bf16 with gelu onto a residual, stores of
// single values: 7.5 us (1112 outputs, in vectors: 6.5).
// Every wait is bounded; a CTA that gives up records MOE_ERR_DEVICE_TIMEOUT
// and still takes part in the cluster's barriers.
#include "linear_epilogue.cuh"
#include "linear_gemm.cuh"

namespace moe {

namespace {

constexpr int kSplitThreads = 256;
constexpr int kOut = 128;  // outputs of a tile

template <int kBN>
struct SplitTile {
    static constexpr int kXBytes = kBN * kSliceBytes;
    static constexpr int kStageBytes = kRowsBytes128 + kXBytes;
    static constexpr int kStages = kBN >= 128 ? 4 : kBN >= 64 ? 6 : 8;
    static constexpr uint32_t kCols = kBN < 32 ? 32 : kBN;
    static constexpr int kPartFloats = kBN * kOut;
};

struct SplitShared {
    uint64_t full[8], empty[8], acc_full;
    uint32_t tmem_base;
    int abort_flag;
};

// kVec outputs from o on of a residual row
template <int kVec>
struct ResidualOf;
template <>
struct ResidualOf<4> {
    uint2 u;
    __device__ __forceinline__ void load(const uint16_t *p) {
        u = __ldcg(reinterpret_cast<const uint2 *>(p));
    }
    __device__ __forceinline__ void add(float (&v)[4]) const {
        const float2 a = unpack_bf16x2(u.x), b = unpack_bf16x2(u.y);
        v[0] += a.x;
        v[1] += a.y;
        v[2] += b.x;
        v[3] += b.y;
    }
};
template <>
struct ResidualOf<1> {
    uint16_t u;
    __device__ __forceinline__ void load(const uint16_t *p) { u = __ldcg(p); }
    __device__ __forceinline__ void add(float (&v)[1]) const {
        v[0] += __uint_as_float(static_cast<uint32_t>(u) << 16);
    }
};

// Adds the ranks' parts of this CTA's `mine` tokens and stores them, kVec
// outputs a thread; a thread keeps its outputs from token to token.  The
// epilogue's operands are fetched before `ready` waits for the parts.
template <bool kFp8, int kVec, int kBN, typename Ready>
__device__ __forceinline__ void store_parts(const LinearArgs &a, const float *part, int o0,
                                            int64_t first, int mine, int split, int own_log,
                                            volatile int *abort_flag, const Ready &ready) {
    constexpr int kLanes = kOut / kVec;               // threads a token
    constexpr int kStep = kSplitThreads / kLanes;     // tokens in one go
    // goes side by side: what a tile can have, as far as registers pay
    constexpr int kMost = kVec == 4 ? 4 : 8;
    constexpr int kBatch = kBN / kStep < kMost ? kBN / kStep : kMost;
    const int ch = threadIdx.x % kLanes * kVec;
    const int o = o0 + ch;
    const bool live = o < a.O;
    float ws[kVec], bias[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        ws[i] = kFp8 && live ? __ldcg(a.w_scale + o + i) : 1.f;
        bias[i] = a.bias && live
                      ? __uint_as_float(static_cast<uint32_t>(__ldcg(a.bias + o + i)) << 16)
                      : 0.f;
    }
    ResidualOf<kVec> res[kBatch] = {};
    float xs[kBatch] = {};
    const int t0 = threadIdx.x / kLanes;
    auto fetch = [&](int t) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int64_t n = first + t + b * kStep;
            if (t + b * kStep < mine && live) {
                if (a.residual) res[b].load(a.residual + n * a.O + o);
                if (kFp8) xs[b] = __ldcg(a.x_scale + n);
            }
        }
    };
    fetch(t0);
    ready();
    if (!live || *abort_flag) return;
    for (int t = t0; t < mine; t += kBatch * kStep) {
        if (t != t0) fetch(t);
        // the batch's tokens side by side: sums, epilogue, stores
        float v[kBatch][kVec];
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
#pragma unroll
            for (int i = 0; i < kVec; ++i) v[b][i] = 0.f;
        for (int r = 0; r < split; ++r) {
            const float *p = part + ((r << own_log) + t) * kOut + ch;
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (t + b * kStep >= mine) continue;
                if constexpr (kVec == 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(p + b * kStep * kOut);
                    v[b][0] += f.x;
                    v[b][1] += f.y;
                    v[b][2] += f.z;
                    v[b][3] += f.w;
                } else {
                    v[b][0] += p[b * kStep * kOut];
                }
            }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                v[b][i] = kFp8 ? fmaf(v[b][i], xs[b] * ws[i], bias[i]) : v[b][i] + bias[i];
        }
        act_all(a.act, reinterpret_cast<float(&)[kBatch * kVec]>(v));
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
            if (a.residual) res[b].add(v[b]);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (t + b * kStep >= mine) continue;
            const int64_t at = (first + t + b * kStep) * a.O + o;
            if (a.out_fp32) {
                float *out = static_cast<float *>(a.out) + at;
                if constexpr (kVec == 4)
                    *reinterpret_cast<float4 *>(out) =
                        make_float4(v[b][0], v[b][1], v[b][2], v[b][3]);
                else
                    *out = v[b][0];
            } else {
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + at;
                if constexpr (kVec == 4)
                    *reinterpret_cast<uint2 *>(out) = make_uint2(
                        pack_bf16x2(v[b][0], v[b][1]), pack_bf16x2(v[b][2], v[b][3]));
                else
                    *out = __float2bfloat16_rn(v[b][0]);
            }
        }
    }
}

template <bool kFp8, int kBN>
__global__ void __launch_bounds__(kSplitThreads, 1)
    linear_split_kernel(const __grid_constant__ CUtensorMap tm_x,
                        const __grid_constant__ CUtensorMap tm_w, const LinearArgs a,
                        const int split_log) {
    using T = SplitTile<kBN>;
    constexpr int kBNLog = kBN == 16 ? 4 : kBN == 32 ? 5 : kBN == 64 ? 6 : 7;
    const int split = 1 << split_log;
    constexpr int kStages = T::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *tiles = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    // [split ranks][tokens of this CTA][128 outputs]
    float *part = reinterpret_cast<float *>(tiles + kStages * T::kStageBytes);
    SplitShared *sm = reinterpret_cast<SplitShared *>(part + T::kPartFloats);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = static_cast<int>(cluster_ctarank());

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sm->full[s], 1);
            mbar_init(&sm->empty[s], 1);
        }
        mbar_init(&sm->acc_full, 1);
        sm->abort_flag = 0;
        fence_barrier_init();
        prefetch_tensor_map(&tm_x);
        prefetch_tensor_map(&tm_w);
    }
    if (warp == 1) {
        tmem_alloc(&sm->tmem_base, T::kCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    // the cluster's CTAs have all started before any of them is written to;
    // waited for where the partial sums leave
    cluster_arrive();
    tc_fence_after_sync();
    const uint32_t tmem = sm->tmem_base;
    volatile int *abort_flag = &sm->abort_flag;
    griddep_launch_dependents();
    griddep_wait();
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && a.status) *a.status = MOE_OK;

    const int o0 = (blockIdx.x >> split_log) * kOut;
    const int64_t n0 = static_cast<int64_t>(blockIdx.y) * kBN;
    const int per_slice = kFp8 ? kSliceBytes : kSliceBytes / 2;
    const int nk = (a.K + per_slice - 1) / per_slice;
    const int k_first = static_cast<int>(static_cast<int64_t>(nk) * rank >> split_log);
    const int k_end = static_cast<int>(static_cast<int64_t>(nk) * (rank + 1) >> split_log);
    const int slices = k_end - k_first;

    if (warp == 0) {
        const bool issues = elect_one();
        int g = 0;
        for (; g < slices; ++g) {
            const int s = g % kStages;
            const uint32_t use = g / kStages;
            if (use > 0 && !warp_wait(&sm->empty[s], (use - 1) & 1, abort_flag)) {
                if (issues) {
                    record_status(a.status, MOE_ERR_DEVICE_TIMEOUT);
                    *abort_flag = 1;
                }
                break;
            }
            if (issues) {
                uint8_t *st = tiles + s * T::kStageBytes;
                mbar_arrive_expect_tx(&sm->full[s], T::kStageBytes);
                tma_load_2d(st, &tm_w, &sm->full[s], (k_first + g) * per_slice, o0);
                tma_load_2d(st + kRowsBytes128, &tm_x, &sm->full[s], (k_first + g) * per_slice,
                            static_cast<int>(n0));
            }
        }
        // no copy may be in flight when the CTA ends
        if (issues)
            for (int i = (g > kStages ? g - kStages : 0); i < g; ++i)
                drain_wait(&sm->full[i % kStages], (i / kStages) & 1);
        __syncwarp();
    } else if (warp == 1) {
        // the whole warp runs the loop and one lane issues: descriptors and
        // barriers stay in uniform registers
        const bool issues = elect_one();
        constexpr uint32_t idesc = linear_idesc<kFp8>(kOut, kBN);
        const uint64_t desc0 = sw128_kmajor_desc(smem_addr(tiles));
        for (int g = 0; g < slices; ++g) {
            const int s = g % kStages;
            if (!warp_wait(&sm->full[s], (g / kStages) & 1, abort_flag)) {
                if (issues) {
                    record_status(a.status, MOE_ERR_DEVICE_TIMEOUT);
                    *abort_flag = 1;
                }
                break;
            }
            tc_fence_after_sync();
            if (issues) {
                const uint64_t da = desc0 + s * (T::kStageBytes >> 4);
                const uint64_t db = da + (kRowsBytes128 >> 4);
#pragma unroll
                for (int kk = 0; kk < kSliceBytes / kMmaBytes; ++kk)
                    linear_mma<kFp8>(tmem, da + 2 * kk, db + 2 * kk, idesc, (g | kk) != 0);
                mma_commit(&sm->empty[s]);
            }
        }
        if (issues) {
            mma_commit(&sm->acc_full);  // after a failure too: the MMAs issued so far
            drain_wait(&sm->acc_full, 0);
        }
        __syncwarp();
    }

    // tokens [n0, n0 + tokens) of the tile exist; this CTA stores [first, first
    // + 2^own_log) of them
    const int tokens = a.N - n0 < kBN ? static_cast<int>(a.N - n0) : kBN;
    const int own_log = kBNLog - split_log;
    const int mine = min(1 << own_log, tokens - (rank << own_log));  // may be <= 0
    const int64_t first = n0 + (rank << own_log);
    // vectors of four outputs where every row allows them
    const bool vec = a.O % 4 == 0 &&
                     reinterpret_cast<uintptr_t>(a.out) % (a.out_fp32 ? 16 : 8) == 0 &&
                     reinterpret_cast<uintptr_t>(a.residual) % 8 == 0;
    auto ready = [&] {  // the accumulator, then the parts of all ranks
        bool ok = true;
        if (lane == 0) ok = mbar_wait(&sm->acc_full, 0, abort_flag);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok && lane == 0) {
            record_status(a.status, MOE_ERR_DEVICE_TIMEOUT);
            *abort_flag = 1;
        }
        cluster_wait();
        if (ok) {
            tc_fence_after_sync();
            const int quarter = warp % 4;
            const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
            const uint32_t to = smem_addr(part) +
                                4 * ((rank << own_log) * kOut + quarter * 32 + lane);
            constexpr int kChunk = kBN < 32 ? 16 : 32;
#pragma unroll 1
            for (int c = warp / 4 * kChunk; c < tokens; c += kSplitThreads / 128 * kChunk) {
                float v[32];
                // a tile of 16 tokens has 32 columns allocated; TMEM wants whole warps
                __syncwarp();
                tmem_load32(taddr + c, v);
                tmem_load_wait();
#pragma unroll
                for (int i = 0; i < kChunk; ++i) {
                    const int t = c + i;
                    if (t < tokens)
                        st_cluster_f32(map_to_rank(to + 4 * kOut * (t & ((1 << own_log) - 1)),
                                                   t >> own_log),
                                       v[i]);
                }
            }
            tc_fence_before_sync();
        }
        cluster_barrier();
    };
    if (vec)
        store_parts<kFp8, 4, kBN>(a, part, o0, first, mine, split, own_log, abort_flag, ready);
    else
        store_parts<kFp8, 1, kBN>(a, part, o0, first, mine, split, own_log, abort_flag, ready);
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        __syncwarp();
        tmem_dealloc(tmem, T::kCols);
    }
}

template <bool kFp8, int kBN>
cudaError_t launch_one(const CUtensorMap &tm_x, const CUtensorMap &tm_w, const LinearArgs &a,
                       int split, cudaStream_t s) {
    int split_log = 0;
    while ((1 << split_log) < split) ++split_log;
    using T = SplitTile<kBN>;
    const size_t smem = 1024 + static_cast<size_t>(T::kStages) * T::kStageBytes +
                        sizeof(float) * T::kPartFloats + sizeof(SplitShared);
    auto kern = linear_split_kernel<kFp8, kBN>;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t err = allow_shared(kern, smem, allowed);
    if (err != cudaSuccess) return err;
    const dim3 grid(static_cast<unsigned>((a.O + kOut - 1) / kOut * split),
                    static_cast<unsigned>((a.N + kBN - 1) / kBN));
    return launch_pdl(kern, grid, dim3(kSplitThreads), smem, s, static_cast<unsigned>(split), tm_x,
                      tm_w, a, split_log);
}

template <bool kFp8>
cudaError_t launch_bn(const CUtensorMap &tm_x, const CUtensorMap &tm_w, const LinearArgs &a,
                      const LinearTiling &t, cudaStream_t s) {
    switch (t.bn) {
        case 16: return launch_one<kFp8, 16>(tm_x, tm_w, a, t.split, s);
        case 32: return launch_one<kFp8, 32>(tm_x, tm_w, a, t.split, s);
        case 64: return launch_one<kFp8, 64>(tm_x, tm_w, a, t.split, s);
        default: return launch_one<kFp8, 128>(tm_x, tm_w, a, t.split, s);
    }
}

}  // namespace

cudaError_t launch_linear_split(const CUtensorMap &tm_x, const CUtensorMap &tm_w,
                                const LinearArgs &a, const LinearTiling &t, cudaStream_t s) {
    return a.fp8 ? launch_bn<true>(tm_x, tm_w, a, t, s) : launch_bn<false>(tm_x, tm_w, a, t, s);
}

}  // namespace moe
