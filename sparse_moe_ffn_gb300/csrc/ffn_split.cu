// ffn_split.cu -- the gated feed-forward block and its backward pass for a decode
// batch: the weights on the MMA's M side (128 rows, in the gate/up step 64 of Wg
// and the 64 of Wu that belong to them; in dh and dx 128 columns of the weights
// as they lie, MN-major), up to 128 tokens on its N side, and K shared by the
// CTAs of a cluster (in dx the K of both products, one after the other).
//
// Each CTA writes its partial sums straight into the shared memory of the CTA
// that owns the token (tokens are dealt out in equal runs); one cluster barrier
// later every CTA adds the parts of its own tokens in rank order, and has gate
// and up of the same output next to each other.
//
//   warp 0  producer: TMA copies
//   warp 1  TMEM and the MMAs
//   all     read the accumulator, then add, finish and store
//
// A CTA takes half an SM's shared memory, so that the down step's CTAs start
// while the gate/up step's still run: their first weights are asked for before
// they wait for that step (programmatic dependent launch), and so are those of dx
// while dh or the weights' gradients are made.  The weights may be read that
// early because the block's first kernel lets its dependents start only after its
// own wait: whatever wrote them has ended then.
// Every wait is bounded; a CTA that gives up records MOE_ERR_DEVICE_TIMEOUT and
// still takes part in the cluster's barriers.
#include "ffn_epilogue.cuh"
#include "gated_ffn.cuh"

namespace moe {

namespace {

constexpr int kSplitThreads = 256;
constexpr int kM = 128;            // weight rows of a tile
constexpr int kSliceValues = 64;   // of K
constexpr int kMaxStages = 5;

struct SplitShared {
    uint64_t full[kMaxStages], empty[kMaxStages], acc_full;
    uint32_t tmem_base;
    int abort_flag;
};

template <int kBN>
struct Tile {
    static constexpr int kXBytes = kBN * kSliceBytes;
    static constexpr int kStageBytes = kRowsBytes128 + kXBytes;
    // The parts lie behind the stages; those of 128 tokens are too large for
    // that and take the stages' place, which costs a barrier between the two (64
    // tokens of 2048 x 8192: 27.1 us instead of 25.9; 128 tokens: 33.9, and 39.2
    // with the parts behind the stages and one CTA an SM).
    static constexpr bool kInPlace = kBN == 128;
    static constexpr int kStages = kBN == 16 ? 5 : kBN == 32 ? 4 : 3;
    static constexpr uint32_t kCols = kBN < 32 ? 32 : kBN;
    static constexpr int kPartBytes = 4 * kBN * kM;
    static_assert(!kInPlace || kPartBytes <= kStages * kStageBytes, "the parts fit");
    static constexpr size_t kShared = 1024 + static_cast<size_t>(kStages) * kStageBytes +
                                      (kInPlace ? 0 : kPartBytes) + sizeof(SplitShared);
};

__device__ __forceinline__ void store4(uint16_t *p, const float (&v)[4]) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

__device__ __forceinline__ void load4(const uint16_t *p, float (&v)[4]) {
    const uint2 u = __ldcg(reinterpret_cast<const uint2 *>(p));
    const float2 x = unpack_bf16x2(u.x), y = unpack_bf16x2(u.y);
    v[0] = x.x, v[1] = x.y, v[2] = y.x, v[3] = y.y;
}

template <int ACT>
__device__ __forceinline__ void gate_grads4(float (&dh)[4], const float (&g)[4],
                                            const float (&u)[4], float (&dup)[4], float (&h)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v, d;
        act_slope<ACT>(g[i], &v, &d);
        dup[i] = dh[i] * v;
        h[i] = v * u[i];
        dh[i] *= u[i] * d;
    }
}

template <FfnOp kOp, int kBN>
__global__ void __launch_bounds__(kSplitThreads, 2)
    ffn_split_kernel(const __grid_constant__ CUtensorMap tm_x0,
                     const __grid_constant__ CUtensorMap tm_x1,
                     const __grid_constant__ CUtensorMap tm_w0,
                     const __grid_constant__ CUtensorMap tm_w1, const FfnArgs a,
                     const int split_log) {
    using T = Tile<kBN>;
    constexpr bool kGated = kOp == kFfnGateUp;
    constexpr bool kAMn = kOp == kFfnDh || kOp == kFfnDx;
    constexpr bool kEarly = kOp == kFfnDown || kOp == kFfnDx;  // weights before the wait
    constexpr int kBNLog = kBN == 16 ? 4 : kBN == 32 ? 5 : kBN == 64 ? 6 : 7;
    constexpr int kStages = T::kStages;
    constexpr int kOuts = kGated ? kM / 2 : kM;  // outputs of a tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t *tiles = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *behind = tiles + kStages * T::kStageBytes;
    // [split ranks][tokens of this CTA][128 weight rows]
    float *part = reinterpret_cast<float *>(T::kInPlace ? tiles : behind);
    SplitShared *sm = reinterpret_cast<SplitShared *>(behind + (T::kInPlace ? 0 : T::kPartBytes));
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = static_cast<int>(cluster_ctarank());
    const int K = kGated || kOp == kFfnDh ? a.H : a.I;
    const int O = kGated || kOp == kFfnDh ? a.I : a.H;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sm->full[s], 1);
            mbar_init(&sm->empty[s], 1);
        }
        mbar_init(&sm->acc_full, 1);
        sm->abort_flag = 0;
        fence_barrier_init();
        prefetch_tensor_map(&tm_x0);
        prefetch_tensor_map(&tm_w0);
    }
    if (warp == 1) {
        tmem_alloc(&sm->tmem_base, T::kCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    // the cluster's CTAs have all started before any of them is written to;
    // waited for where the partial sums leave
    if (!T::kInPlace) cluster_arrive();
    tc_fence_after_sync();
    const uint32_t tmem = sm->tmem_base;
    volatile int *abort_flag = &sm->abort_flag;

    const int o0 = (blockIdx.x >> split_log) * kOuts;
    const int64_t n0 = static_cast<int64_t>(blockIdx.y) * kBN;
    const int each = (K + kSliceValues - 1) / kSliceValues;  // of a product
    const int nk = kOp == kFfnDx ? 2 * each : each;
    const int k_first = static_cast<int>(static_cast<int64_t>(nk) * rank >> split_log);
    const int k_end = static_cast<int>(static_cast<int64_t>(nk) * (rank + 1) >> split_log);
    const int slices = k_end - k_first;

    auto load_weights = [&](int g) {
        uint8_t *st = tiles + g % kStages * T::kStageBytes;
        uint64_t *bar = &sm->full[g % kStages];
        const bool second = kOp == kFfnDx && k_first + g >= each;
        const int k = (k_first + g - (second ? each : 0)) * kSliceValues;
        mbar_arrive_expect_tx(bar, T::kStageBytes);
        if (kAMn) {
            const CUtensorMap *w = second ? &tm_w1 : &tm_w0;
            tma_load_2d(st, w, bar, o0, k);
            tma_load_2d(st + kMnChunk, w, bar, o0 + 64, k);
        } else {
            tma_load_2d(st, &tm_w0, bar, k, o0);
            if (kGated) tma_load_2d(st + kRowsBytes128 / 2, &tm_w1, bar, k, o0);
        }
    };
    const int early = kEarly ? min(slices, kStages) : 0;
    if (!kEarly) griddep_wait();
    if (kEarly && warp == 0 && elect_one())
        for (int g = 0; g < early; ++g) load_weights(g);
    griddep_launch_dependents();
    if (kEarly) griddep_wait();
    if (a.reset_status && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
        *a.status = MOE_OK;

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
                if (g >= early) load_weights(g);
                const bool second = kOp == kFfnDx && k_first + g >= each;
                tma_load_2d(tiles + s * T::kStageBytes + kRowsBytes128, second ? &tm_x1 : &tm_x0,
                            &sm->full[s], (k_first + g - (second ? each : 0)) * kSliceValues,
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
        constexpr uint32_t idesc = idesc_bf16_f32(kM, kBN) | (kAMn ? kIdescAMn : 0);
        constexpr int kStepA = kAMn ? kStepMnMajor : kStepKMajor;
        const uint32_t base = smem_addr(tiles);
        const uint64_t desc_a = kAMn ? sw128_mnmajor_desc(base) : sw128_kmajor_desc(base);
        const uint64_t desc_b = sw128_kmajor_desc(base + kRowsBytes128);
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
                const uint64_t da = desc_a + s * (T::kStageBytes >> 4);
                const uint64_t db = desc_b + s * (T::kStageBytes >> 4);
#pragma unroll
                for (int kk = 0; kk < kSliceBytes / kMmaBytes; ++kk)
                    mma_f16kind(tmem, da + kStepA * kk, db + kStepKMajor * kk, idesc,
                                (g | kk) != 0);
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
    // four outputs a thread; a thread keeps its outputs from token to token
    constexpr int kLanes = kOuts / 4;                // threads a token
    constexpr int kStep = kSplitThreads / kLanes;    // tokens in one go
    const int ch = threadIdx.x % kLanes * 4;
    const int o = o0 + ch;
    const int t0 = threadIdx.x / kLanes;
    // (dh) gate and up of the first go, before the accumulator is waited for
    float gate[4] = {}, up[4] = {};
    auto fetch = [&](int t) {
        if (kOp == kFfnDh && o < O && t < mine) {
            load4(a.gate + (first + t) * O + o, gate);
            load4(a.up + (first + t) * O + o, up);
        }
    };
    fetch(t0);
    // the accumulator, then the parts of all ranks
    bool ok = true;
    if (lane == 0) ok = mbar_wait(&sm->acc_full, 0, abort_flag);
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (!ok && lane == 0) {
        record_status(a.status, MOE_ERR_DEVICE_TIMEOUT);
        *abort_flag = 1;
    }
    if (T::kInPlace) cluster_arrive();  // this CTA's MMAs have read its stages
    cluster_wait();
    if (ok) {
        tc_fence_after_sync();
        const int quarter = warp % 4;
        const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t to = smem_addr(part) + 4 * ((rank << own_log) * kM + quarter * 32 + lane);
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
                    st_cluster_f32(map_to_rank(to + 4 * kM * (t & ((1 << own_log) - 1)),
                                               t >> own_log),
                                   v[i]);
            }
        }
        tc_fence_before_sync();
    }
    cluster_barrier();

    const int split = 1 << split_log;
    if (o < O && !*abort_flag) {
        for (int t = t0; t < mine; t += kStep) {
            const int64_t at = (first + t) * O + o;
            const int64_t own = (first + t) * a.ld + o;  // in the workspace
            float res[4] = {};
            if (kOp == kFfnDown && a.residual) load4(a.residual + at, res);
            if (t != t0) fetch(t);
            float v[4] = {}, w[4] = {}, h[4];
            for (int r = 0; r < split; ++r) {
                const float *p = part + ((r << own_log) + t) * kM + ch;
                const float4 f = *reinterpret_cast<const float4 *>(p);
                v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
                if (kGated) {
                    const float4 u = *reinterpret_cast<const float4 *>(p + kM / 2);
                    w[0] += u.x, w[1] += u.y, w[2] += u.z, w[3] += u.w;
                }
            }
            if (kGated) {
                if (a.keep) {
                    store4(a.out[1] + at, v);
                    store4(a.out[2] + at, w);
                }
                act_all(a.act, v);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] *= w[i];
                store4(a.out[0] + own, v);
            } else if (kOp == kFfnDh) {
                switch (a.act) {
                    case MOE_ACT_SILU: gate_grads4<MOE_ACT_SILU>(v, gate, up, w, h); break;
                    case MOE_ACT_GELU: gate_grads4<MOE_ACT_GELU>(v, gate, up, w, h); break;
                    case MOE_ACT_GELU_TANH:
                        gate_grads4<MOE_ACT_GELU_TANH>(v, gate, up, w, h);
                        break;
                    case MOE_ACT_RELU: gate_grads4<MOE_ACT_RELU>(v, gate, up, w, h); break;
                    default: gate_grads4<MOE_ACT_NONE>(v, gate, up, w, h); break;
                }
                store4(a.out[0] + own, h);
                store4(a.out[1] + own, v);
                store4(a.out[2] + own, w);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] += res[i];
                store4(a.out[0] + at, v);
            }
        }
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        __syncwarp();
        tmem_dealloc(tmem, T::kCols);
    }
}

int split_outs(FfnOp op) { return op == kFfnGateUp ? kM / 2 : kM; }
int split_o(FfnOp op, int H, int I) { return op == kFfnGateUp || op == kFfnDh ? I : H; }

template <FfnOp kOp, int kBN>
cudaError_t launch_one(const FfnMaps &m, const FfnArgs &a, int split, cudaStream_t s) {
    int split_log = 0;
    while ((1 << split_log) < split) ++split_log;
    using T = Tile<kBN>;
    const size_t smem = T::kShared;
    auto kern = ffn_split_kernel<kOp, kBN>;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t err = allow_shared(kern, smem, allowed);
    if (err != cudaSuccess) return err;
    const int outs = split_outs(kOp), O = split_o(kOp, a.H, a.I);
    const dim3 grid(static_cast<unsigned>((O + outs - 1) / outs * split),
                    static_cast<unsigned>((a.N + kBN - 1) / kBN));
    return launch_pdl(kern, grid, dim3(kSplitThreads), smem, s, static_cast<unsigned>(split),
                      m.a[0], m.a[kOp == kFfnDx ? 1 : 0], m.b[0],
                      m.b[kOp == kFfnGateUp || kOp == kFfnDx ? 1 : 0], a, split_log);
}

template <FfnOp kOp>
cudaError_t launch_tokens(const FfnMaps &m, const FfnArgs &a, const FfnSplit &t, cudaStream_t s) {
    switch (t.bn) {
        case 16: return launch_one<kOp, 16>(m, a, t.split, s);
        case 32: return launch_one<kOp, 32>(m, a, t.split, s);
        case 64: return launch_one<kOp, 64>(m, a, t.split, s);
        default: return launch_one<kOp, 128>(m, a, t.split, s);
    }
}

}  // namespace

// The tokens' tile is the smallest that holds them all, or a smaller one where
// the weights have so few rows that clusters of 8 still fit at once: the rows
// are then read again, from L2, and twice as many CTAs do so (128 tokens of 2048
// x 8192: 34.2 us with 128 tokens a tile in the down step, 28.8 with 64).
// Beyond 128 tokens the pair kernel takes over (gate/up of 2048 x 8192, 256
// tokens: 45 us and more in all with tiles of 128, 40 with pairs), but for
//  - down and dx of up to 512 tokens whose long K four CTAs or more can share at
//    once: pairs would share it through memory and a second kernel (down of 256
//    tokens of 2048 x 8192: 33.8 us against 40.0, of 512 of 1024 x 2816 19.1
//    against 25.0; both ways, with dx, 256 of 1024 x 2816: 45.6 against 51.1.  With
//    two CTAs a tile 512 tokens of 4096 x 12288 take 112 either way, with 12
//    slices of K 512 tokens of 2048 x 768 18.6 against 15.7, dx with 256 slices
//    114 against 111.5);
//  - dh and gate/up of up to 256 tokens whose tiles are so few that two or four
//    CTAs share one (both ways, dh of 256 tokens of 2048 x 768: 40.0 against 46.2,
//    without sharing of 2048 x 8192 118 against 114).
FfnSplit ffn_split(FfnOp op, int64_t N, int H, int I, int num_sms) {
    FfnSplit t = {0, 1};
    if (N > 512) return t;
    const int n = static_cast<int>(N);
    const int outs = split_outs(op), O = split_o(op, H, I);
    const int K = op == kFfnGateUp || op == kFfnDh ? H : I;
    const int64_t rows = (O + outs - 1) / outs;
    const int nk = (K + kSliceValues - 1) / kSliceValues * (op == kFfnDx ? 2 : 1);
    const int64_t fit = 2 * static_cast<int64_t>(num_sms);
    const auto share = [&](int bn) {  // CTAs that can share a tile of bn tokens
        const int64_t tiles = rows * ((n + bn - 1) / bn);
        int split = 1;
        while (split < 8 && 2 * split <= nk && 2 * split * tiles <= fit) split *= 2;
        return split;
    };
    if (n > 128) {
        if (op == kFfnGateUp || op == kFfnDh) {
            if (n <= 256 && share(64) >= (op == kFfnDh ? 2 : 4)) return {64, share(64)};
            return t;
        }
        if (nk < 32 || (op == kFfnDx && nk > 128)) return t;
        for (const int bn : {64, 128})
            if (share(bn) >= 4) return {bn, share(bn)};
        return t;
    }
    t.bn = n <= 16 ? 16 : n <= 32 ? 32 : n <= 64 ? 64 : 128;
    while (t.bn > 16 && 8 * rows * ((n + t.bn / 2 - 1) / (t.bn / 2)) <= fit) t.bn /= 2;
    t.split = share(t.bn);
    return t;
}

cudaError_t launch_ffn_split(FfnOp op, const FfnMaps &m, const FfnArgs &a, const FfnSplit &t,
                             cudaStream_t s) {
    switch (op) {
        case kFfnGateUp: return launch_tokens<kFfnGateUp>(m, a, t, s);
        case kFfnDown: return launch_tokens<kFfnDown>(m, a, t, s);
        case kFfnDh: return launch_tokens<kFfnDh>(m, a, t, s);
        default: return launch_tokens<kFfnDx>(m, a, t, s);
    }
}

}  // namespace moe
