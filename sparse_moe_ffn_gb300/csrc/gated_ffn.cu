// gated_ffn.cu -- the products of the gated feed-forward block and of its
// backward pass (gated_ffn.cuh has the formulas), on CTA pairs: one tcgen05 MMA
// of 256 rows x 256 columns (cta_group::2) reads each operand byte for 256 rows
// of the other side, and the elementwise part runs on the accumulators.
//
// Operands come as they lie in memory.  A product's K runs along the rows of
// either operand (K-major: [rows, K]) or across them (MN-major: [K, rows], as
// the weights in dh and dx and both operands of the weights' gradients); TMA
// brings either with 128-byte swizzled rows, and the MMA's descriptors say which
// it is, so nothing is transposed in memory.
//
//   gate/up   the even CTA of a pair loads 128 rows of Wg, the odd one the same
//             rows of Wu: a pair's accumulator is 128 columns of gate next to
//             the 128 of up that belong to them
//   dx        dgate Wg + dup Wu is one product whose K is the two in a row
//   dW        the three weights' tiles are one list, and where both are of few
//             tiles dx's join them: one launch instead of two
//
//   warp 0     producer: TMA copies; the even CTA's barrier counts both CTAs'
//              bytes
//   warp 1     TMEM; in the even CTA, the MMAs
//   warps 2-9  epilogue: warp w owns TMEM lanes 32 (w % 4) .. + 31 (one row a
//              lane) and half of the columns; two accumulators alternate, so a
//              tile's epilogue runs under the next tile's MMAs
//
// Rounding: gate, up, dgate, dup and h are operands of bf16 products and are
// rounded to bf16 once each; h in the forward pass and dgate, dup in the
// backward pass are made from fp32 accumulators.
//
// Tiles run in whole waves; the slices of a partial last wave are dealt out
// evenly where K is long (FfnPlan), and ffn_join_kernel adds the partial sums
// in a fixed order.  Every wait is bounded; a CTA that gives up records
// MOE_ERR_DEVICE_TIMEOUT.
#include "ffn_epilogue.cuh"
#include "gated_ffn.cuh"
#include "linear_gemm.cuh"

namespace moe {

namespace {

constexpr int kEpiWarps = 8;
constexpr int kFfnThreads = 64 + 32 * kEpiWarps;
constexpr int kMostStages = 6;
constexpr int kSliceK = 64;            // values of K in a slice
constexpr int kBoxBytes = 32 * 128;    // 32 rows x 64 values of an output
constexpr int kMinSlices = 8;          // of a part of a tile
// Sharing the last wave has to take this much off the time that the constants below
// give, for the second epilogue and the join.  Measured, unshared and shared, where
// they say 5.9 us: down of 2048 x 2048 x 8192 115 and 132; 8.8: of 1200 x 2048 x 4096
// 55 and 60; 9.4: dx of 3000 x 1024 x 2816 58 and 66; 13.7: down of 1536 x 2048 x
// 8192 104 and 114, of 3000 x 2048 x 4096 112 and 107; 16.2: of 5000 x 1024 x 4096 91
// and 85, the weights' gradients of 4096 x 2048 x 4096 186 and 178; 20.6: of 5000 x
// 2048 x 4096 233 and 222.
constexpr double kJoinUs = 12.0;
constexpr double kLaunchUs = 2.0;

struct FfnShared {
    uint64_t full[kMostStages];   // even CTA: both CTAs' bytes of a stage landed
    uint64_t empty[kMostStages];  // both: the MMAs are done with a stage
    uint64_t acc_full[2];     // both: an accumulator is complete
    uint64_t acc_empty[2];    // even CTA: both CTAs' epilogues have read one
    uint64_t drain;           // even CTA: every MMA has completed
    uint32_t tmem_base;
    int abort_flag;
};

// kBN: accumulator columns of a tile, 256 or 128
template <FfnOp kOp, int kBN>
struct FfnTraits {
    static constexpr bool kBMn = kOp == kFfnDh || kOp == kFfnDx || kOp == kFfnDw ||
                                 kOp == kFfnGrads;
    static constexpr int kColsPerTile = kOp == kFfnGateUp ? kBN / 2 : kBN;  // of the output
    static constexpr int kBBytes = kBN / 2 * kSliceBytes;  // a CTA's share of a slice
    static constexpr int kStageBytes = kRowsBytes128 + kBBytes;
    // dh: 211 us, 216 with six; dw: room for its outputs on their way
    static constexpr int kStages = kOp == kFfnDh || kOp == kFfnDw ? 5 : kMostStages;
    static constexpr int kOutBytes = kOp == kFfnDw ? kEpiWarps * 2 * kBoxBytes : 0;
    static constexpr size_t kShared = 1024 + static_cast<size_t>(kStages) * kStageBytes +
                                      kOutBytes + sizeof(FfnShared);
    static constexpr int kPartFloats = kFfnTile * kBN;
};

// One piece of work of a pair: slices [k0, k1) of a tile; slot >= 0: its sums
// go to that partial tile.
struct FfnItem {
    int tile, k0, k1, slot;
};

// Whether a tile of kFfnGrads is one of dx.
__device__ __forceinline__ bool is_dx(const FfnPlan &p, int tile) {
    return p.dx_first ? tile < p.dx_tiles : tile >= p.tiles - p.dx_tiles;
}

// Whether a tile's M side lies MN-major.
template <FfnOp kOp>
__device__ __forceinline__ bool a_is_mn(const FfnPlan &p, int tile) {
    return kOp == kFfnDw || (kOp == kFfnGrads && !is_dx(p, tile));
}

// The pieces of pair `pair`, in order.  kFfnGrads deals its tiles out forth and
// back, the long ones first, so that a pair that got one more long one gets one
// short one less.
template <FfnOp kOp>
struct FfnWalk {
    const FfnPlan &p;
    int pair, tile, turn;
    int64_t from, to;  // of the shared slices
    __device__ __forceinline__ FfnWalk(const FfnPlan &plan, int pair_)
        : p(plan), pair(pair_), tile(pair_), turn(0), from(0), to(0) {
        if (p.parts > pair) {
            const int64_t s = static_cast<int64_t>(p.tiles - p.whole) * p.nk;
            from = s * pair / p.parts;
            to = s * (pair + 1) / p.parts;
        }
    }
    __device__ __forceinline__ bool next(FfnItem &it) {
        if (kOp == kFfnGrads) {
            const int i = turn * p.pairs + (turn % 2 ? p.pairs - 1 - pair : pair);
            if (i >= p.tiles) return false;
            it = {i, 0, is_dx(p, i) ? p.dx_nk : p.nk, -1};
            ++turn;
            return true;
        }
        if (tile < p.whole) {
            it = {tile, 0, p.nk, -1};
            tile += p.pairs;
            return true;
        }
        if (from >= to) return false;
        const int t = static_cast<int>(from / p.nk);
        const int64_t first = static_cast<int64_t>(t) * p.nk;
        const int64_t end = min(to, first + p.nk);
        it = {p.whole + t, static_cast<int>(from - first), static_cast<int>(end - first),
              2 * pair + turn};
        from = end;
        ++turn;
        return true;
    }
};

// Tiles run through bands of kBand row tiles, column tile by column tile: the
// tiles in flight share few rows of either operand.
constexpr int kBand = 16;

struct FfnTile {
    int prod, m, n;
};

template <FfnOp kOp>
__device__ __forceinline__ void ffn_dims(const FfnArgs &a, int prod, int64_t *rows, int *cols) {
    if (kOp == kFfnDw || (kOp == kFfnGrads && prod < 3)) {
        *rows = prod == 2 ? a.H : a.I;
        *cols = prod == 2 ? a.I : a.H;
    } else {
        *rows = a.N;
        *cols = kOp == kFfnGateUp || kOp == kFfnDh ? a.I : a.H;
    }
}

template <FfnOp kOp, int kBN>
__device__ __forceinline__ FfnTile ffn_tile(const FfnArgs &a, int tile) {
    FfnTile t = {0, 0, 0};
    if (kOp == kFfnGrads) {
        const FfnPlan &p = a.plan;
        if (is_dx(p, tile)) t.prod = 3;
        if (t.prod == 3 ? !p.dx_first : p.dx_first)
            tile -= t.prod == 3 ? p.tiles - p.dx_tiles : p.dx_tiles;
    }
    if (kOp == kFfnDw || (kOp == kFfnGrads && t.prod == 0)) {
        const int each = (a.I + kFfnTile - 1) / kFfnTile * ((a.H + kBN - 1) / kBN);
        t.prod = min(tile / each, 2);
        tile -= t.prod * each;
    }
    int64_t rows;
    int cols;
    ffn_dims<kOp>(a, t.prod, &rows, &cols);
    const int m_tiles = static_cast<int>((rows + kFfnTile - 1) / kFfnTile);
    constexpr int kCols = FfnTraits<kOp, kBN>::kColsPerTile;
    const int n_tiles = (cols + kCols - 1) / kCols;
    const int band = tile / (kBand * n_tiles);
    const int first = band * kBand;
    const int high = min(kBand, m_tiles - first);
    const int in = tile - band * kBand * n_tiles;
    t.m = first + in % high;
    t.n = in / high;
    return t;
}

// 32-byte load that stays out of L1 (8 words; p 32-byte aligned)
__device__ __forceinline__ void ld_global_v8(const void *p, uint32_t *v) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                   "=r"(v[6]), "=r"(v[7])
                 : "l"(p)
                 : "memory");
}

// 32 values of a bf16 row (16-byte aligned; 32-byte loads if wide), the first
// `left` of which exist (a multiple of 8).
struct Row32 {
    uint32_t w[16];
    __device__ __forceinline__ void load(const uint16_t *p, int left, bool wide) {
        if (wide && left >= 32) {
            ld_global_v8(p, &w[0]);
            ld_global_v8(p + 16, &w[8]);
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 u = 8 * i < left ? __ldcg(reinterpret_cast<const uint4 *>(p) + i)
                                         : make_uint4(0, 0, 0, 0);
            w[4 * i] = u.x;
            w[4 * i + 1] = u.y;
            w[4 * i + 2] = u.z;
            w[4 * i + 3] = u.w;
        }
    }
    __device__ __forceinline__ void add_to(float (&v)[32]) const {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 f = unpack_bf16x2(w[i]);
            v[2 * i] += f.x;
            v[2 * i + 1] += f.y;
        }
    }
};

// 32 values to a bf16 row, as Row32 reads them.  Each lane stores its own row's
// whole 32-byte sectors (but for the weights' gradients of few tokens, whose
// tiles are mostly stores: FfnArgs::boxes).  Tensor-map stores of 32 x 32 values
// would take the TMA unit's time from the operands, which keep it busy (a row of a
// box, of up to 128 bytes, costs it about two cycles): with them dh of 8192 x 2048
// x 8192 took 236 us instead of 216, and the forward pass that keeps gate and up
// 472 instead of 459.
__device__ __forceinline__ void store_row(uint16_t *p, const float (&v)[32], int left, bool wide) {
    if (wide && left >= 32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t u[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = pack_bf16x2(v[16 * h + 2 * i], v[16 * h + 2 * i + 1]);
            st_global_v8(p + 16 * h, u);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (8 * i < left)
            *reinterpret_cast<uint4 *>(p + 8 * i) =
                make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]),
                           pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                           pack_bf16x2(v[8 * i + 4], v[8 * i + 5]),
                           pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
}

// This lane's 64 values (a row of a 32 x 64 box), as a tensor-map store with
// 128-byte swizzled rows reads them.
__device__ __forceinline__ void write_box_row(uint8_t *buf, int lane, const float (&v)[32],
                                              const float (&w)[32]) {
    uint8_t *row = buf + lane * 128;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float *f = j < 4 ? v + 8 * j : w + 8 * (j - 4);
        *reinterpret_cast<uint4 *>(row + 16 * (j ^ (lane & 7))) =
            make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                       pack_bf16x2(f[6], f[7]));
    }
}

__device__ __forceinline__ void tma_store_box(const CUtensorMap *map, const void *src, int c0,
                                              int c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];"
                 ::"l"(map), "r"(smem_addr(src)), "r"(c0), "r"(c1)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// Whether the caller's arrays that the epilogue reads and writes have rows that
// start on 32 bytes (those of the workspace do: kFfnLd).
template <FfnOp kOp>
__device__ __forceinline__ bool all_wide(const FfnArgs &a, int cols) {
    uintptr_t p = reinterpret_cast<uintptr_t>(a.gate) | reinterpret_cast<uintptr_t>(a.up) |
                  reinterpret_cast<uintptr_t>(a.residual);
    if (kOp != kFfnDh)
        p |= reinterpret_cast<uintptr_t>(a.out[0]) | reinterpret_cast<uintptr_t>(a.out[1]) |
             reinterpret_cast<uintptr_t>(a.out[2]) | reinterpret_cast<uintptr_t>(a.out[3]);
    return cols % 16 == 0 && p % 32 == 0;
}

// dh -> dgate, with dup and h from the saved gate and up.
template <int ACT>
__device__ __forceinline__ void gate_grads(float (&dh)[32], const Row32 &gate, const Row32 &up,
                                           float (&dup)[32], float (&h)[32]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float2 g = unpack_bf16x2(gate.w[i]), u = unpack_bf16x2(up.w[i]);
        float a, d;
        act_slope<ACT>(g.x, &a, &d);
        dup[2 * i] = dh[2 * i] * a;
        h[2 * i] = a * u.x;
        dh[2 * i] *= u.x * d;
        act_slope<ACT>(g.y, &a, &d);
        dup[2 * i + 1] = dh[2 * i + 1] * a;
        h[2 * i + 1] = a * u.y;
        dh[2 * i + 1] *= u.y * d;
    }
}

template <FfnOp kOp, int kBN>
__global__ void __launch_bounds__(kFfnThreads, 1)
    ffn_kernel(const __grid_constant__ FfnMaps maps, const __grid_constant__ FfnArgs a) {
    using T = FfnTraits<kOp, kBN>;
    constexpr int kStageBytes = T::kStageBytes;
    constexpr int kStages = T::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *tiles = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *out_bufs = tiles + kStages * kStageBytes;
    FfnShared *sm = reinterpret_cast<FfnShared *>(out_bufs + T::kOutBytes);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = static_cast<int>(cluster_ctarank());
    const bool leader = rank == 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sm->full[s], 1);
            mbar_init(&sm->empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm->acc_full[i], 1);
            mbar_init(&sm->acc_empty[i], 2 * kEpiWarps);
        }
        mbar_init(&sm->drain, 1);
        sm->abort_flag = 0;
        fence_barrier_init();
        prefetch_tensor_map(&maps.a[0]);
        prefetch_tensor_map(&maps.b[0]);
    }
    if (warp == 1) tmem_alloc_2cta(&sm->tmem_base, 2 * kBN);
    tc_fence_before_sync();
    __syncthreads();
    cluster_barrier();  // both CTAs' barriers exist before any remote arrival
    tc_fence_after_sync();
    const uint32_t tmem = sm->tmem_base;
    volatile int *abort_flag = &sm->abort_flag;
    // in this order: what follows may read weights before its own wait
    griddep_wait();
    griddep_launch_dependents();
    if (a.reset_status && blockIdx.x == 0 && threadIdx.x == 0 && a.status) *a.status = MOE_OK;

    const int pair = blockIdx.x / 2;
    FfnWalk<kOp> walk(a.plan, pair);
    FfnItem it;

    if (warp == 0) {
        const bool issues = elect_one();
        // stages filled so far; the stage and the parity of its last release
        int64_t g = 0;
        int s = 0;
        uint32_t parity = 1;
        bool failed = false;
        while (!failed && walk.next(it)) {
            const FfnTile t = ffn_tile<kOp, kBN>(a, it.tile);
            const int row = t.m * kFfnTile + rank * 128;
            const int col = t.n * T::kColsPerTile + (kOp == kFfnGateUp ? 0 : rank * (kBN / 2));
            // dx: slices of its first product
            const bool dx = kOp == kFfnDx || (kOp == kFfnGrads && t.prod == 3);
            const int half = (kOp == kFfnGrads ? a.plan.dx_nk : a.plan.nk) / 2;
            const bool a_mn = a_is_mn<kOp>(a.plan, it.tile);
            for (int kc = it.k0; kc < it.k1; ++kc, ++g) {
                if (g >= kStages && !warp_wait(&sm->empty[s], parity, abort_flag)) {
                    if (issues) {
                        record_status(a.status, MOE_ERR_DEVICE_TIMEOUT);
                        *abort_flag = 1;
                    }
                    failed = true;
                    break;
                }
                if (issues) {
                    uint8_t *st = tiles + s * kStageBytes;
                    uint8_t *sb = st + kRowsBytes128;
                    const uint32_t bar = map_to_rank(smem_addr(&sm->full[s]), 0);
                    if (leader) mbar_arrive_expect_tx(&sm->full[s], 2 * kStageBytes);
                    const int second = dx && kc >= half ? 1 : 0;
                    const int k = (kc - second * half) * kSliceK;
                    const CUtensorMap *ma = &maps.a[t.prod + second];
                    const CUtensorMap *mb = &maps.b[kOp == kFfnGateUp ? rank : t.prod + second];
                    if (a_mn) {
                        tma_load_2d_pair(st, ma, bar, row, k);
                        tma_load_2d_pair(st + kMnChunk, ma, bar, row + 64, k);
                    } else {
                        tma_load_2d_pair(st, ma, bar, k, row);
                    }
                    if (T::kBMn) {
                        tma_load_2d_pair(sb, mb, bar, col, k);
                        if (kBN == 256) tma_load_2d_pair(sb + kMnChunk, mb, bar, col + 64, k);
                    } else {
                        tma_load_2d_pair(sb, mb, bar, k, col);
                    }
                }
                if (++s == kStages) {
                    s = 0;
                    parity ^= 1;
                }
            }
        }
        // no copy may be in flight when the pair ends
        if (leader && issues)
            for (int64_t i = (g > kStages ? g - kStages : 0); i < g; ++i)
                drain_wait(&sm->full[i % kStages], (i / kStages) & 1);
        __syncwarp();
    } else if (warp == 1) {
        if (leader) {
            // The whole warp runs the loop and one lane of it issues, so that
            // the compiler keeps descriptors and barriers in uniform registers.
            const bool issues = elect_one();
            constexpr int kStepB = T::kBMn ? kStepMnMajor : kStepKMajor;
            const uint32_t base = smem_addr(tiles);
            const uint64_t desc_b = T::kBMn ? sw128_mnmajor_desc(base + kRowsBytes128)
                                            : sw128_kmajor_desc(base + kRowsBytes128);
            int s = 0, n = 0;
            uint32_t phase = 0;
            bool failed = false;
            for (; !failed && walk.next(it); ++n) {
                const int acc = n & 1;
                const uint32_t use = n >> 1;
                if (use > 0 && !warp_wait(&sm->acc_empty[acc], (use - 1) & 1, abort_flag)) {
                    failed = true;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t d = tmem + acc * kBN;
                const bool a_mn = a_is_mn<kOp>(a.plan, it.tile);
                const uint32_t idesc = idesc_bf16_f32(kFfnTile, kBN) | (a_mn ? kIdescAMn : 0) |
                                       (T::kBMn ? kIdescBMn : 0);
                const uint64_t desc_a = a_mn ? sw128_mnmajor_desc(base) : sw128_kmajor_desc(base);
                const int step_a = a_mn ? kStepMnMajor : kStepKMajor;
                for (int kc = it.k0; kc < it.k1; ++kc) {
                    if (!warp_wait(&sm->full[s], phase, abort_flag)) {
                        failed = true;
                        break;
                    }
                    tc_fence_after_sync();
                    if (issues) {
                        const uint64_t da = desc_a + s * (kStageBytes >> 4);
                        const uint64_t db = desc_b + s * (kStageBytes >> 4);
#pragma unroll
                        for (int kk = 0; kk < kSliceK / 16; ++kk)
                            linear_mma_pair<false>(d, da + step_a * kk, db + kStepB * kk, idesc,
                                                   kk == 0 ? kc != it.k0 : 1);
                        commit_2cta(&sm->empty[s], 3);
                    }
                    if (++s == kStages) {
                        s = 0;
                        phase ^= 1;
                    }
                }
                if (!failed && issues) commit_2cta(&sm->acc_full[acc], 3);
            }
            if (failed && issues) {
                record_status(a.status, MOE_ERR_DEVICE_TIMEOUT);
                *abort_flag = 1;
            }
            if (issues) {
                commit_2cta(&sm->drain, 1);
                drain_wait(&sm->drain, 0);
            }
        }
        __syncwarp();
    } else {
        const int quarter = warp % 4, half = (warp - 2) / 4;
        constexpr int kCols = T::kColsPerTile / 2;  // a warp's
        const uint32_t empty0 = map_to_rank(smem_addr(&sm->acc_empty[0]), 0);
        const uint32_t empty1 = map_to_rank(smem_addr(&sm->acc_empty[1]), 0);
        if (kOp == kFfnDh) {
            // The first tile's gate and up start on their way to L2 now; the
            // reads below come one after the other.  (For every tile, a tile
            // ahead: 260 us instead of 236 for 8192 x 2048 x 8192.)
            const FfnTile t = ffn_tile<kOp, kBN>(a, pair);
            const int64_t r = static_cast<int64_t>(t.m) * kFfnTile + rank * 128 + quarter * 32 + lane;
            const int first = t.n * T::kColsPerTile + half * kCols;
            if (r < a.N)
                for (int c = first; c < min(first + kCols, a.I); c += 64) {
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(a.gate + r * a.I + c));
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(a.up + r * a.I + c));
                }
        }
        int n = 0, boxes = 0;
        for (; walk.next(it); ++n) {
            const FfnTile t = ffn_tile<kOp, kBN>(a, it.tile);
            int64_t rows;
            int all_cols;
            ffn_dims<kOp>(a, t.prod, &rows, &all_cols);
            const int acc = n & 1;
            const int c0 = t.n * T::kColsPerTile + half * kCols;
            const int64_t r0 = static_cast<int64_t>(t.m) * kFfnTile + rank * 128 + quarter * 32;
            const int64_t r = r0 + lane;
            // columns of this warp that exist (warp-uniform)
            const int cols = r0 < rows ? min(kCols, all_cols - c0) : 0;
            const bool wide = all_wide<kOp>(a, all_cols);
            // operands of the elementwise part, read 32 columns ahead
            Row32 e0 = {}, e1 = {};
            auto fetch = [&](int c) {
                if (c >= cols || r >= rows) return;
                const int64_t at = r * all_cols + c0 + c;
                if (kOp == kFfnDh) {
                    e0.load(a.gate + at, cols - c, wide);
                    e1.load(a.up + at, cols - c, wide);
                }
                if (kOp == kFfnDown && a.residual && it.slot < 0)
                    e0.load(a.residual + at, cols - c, wide);
            };
            fetch(0);
            __syncwarp();
            bool ok = true;
            if (lane == 0) ok = mbar_wait(&sm->acc_full[acc], (n >> 1) & 1, abort_flag);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) {
                if (lane == 0) {
                    record_status(a.status, MOE_ERR_DEVICE_TIMEOUT);
                    *abort_flag = 1;
                }
                break;
            }
            tc_fence_after_sync();
            const uint32_t taddr =
                tmem + (static_cast<uint32_t>(quarter * 32) << 16) + acc * kBN + half * kCols;
            if (kOp == kFfnDw && a.boxes && it.slot < 0) {
#pragma unroll 1
                for (int c = 0; c < cols; c += 64, ++boxes) {
                    float v[32], w[32];
                    __syncwarp();  // TMEM wants whole warps
                    tmem_load32(taddr + c, v);
                    __syncwarp();
                    tmem_load32(taddr + c + 32, w);
                    tmem_load_wait();
                    // the buffer in turn has left
                    asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                    __syncwarp();
                    uint8_t *b = out_bufs + ((warp - 2) * 2 + (boxes & 1)) * kBoxBytes;
                    write_box_row(b, lane, v, w);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0)
                        tma_store_box(&maps.out[t.prod], b, c0 + c, static_cast<int>(r0));
                }
            } else if (it.slot >= 0) {  // (kFfnDown, kFfnDx, kFfnDw)
                float *part = a.part + static_cast<int64_t>(it.slot) * T::kPartFloats +
                              ((rank * 4 + quarter) * 2 + half) * (kBN / 64) * 1024 + 4 * lane;
#pragma unroll 1
                for (int c = 0; c < cols; c += 32, part += 1024) {
                    float v[32];
                    __syncwarp();
                    tmem_load32(taddr + c, v);
                    tmem_load_wait();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        __stcg(reinterpret_cast<float4 *>(part + 128 * i),
                               make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < cols; c += 32) {
                    float v[32], w[32], x[32];
                    __syncwarp();  // TMEM wants whole warps
                    tmem_load32(taddr + c, v);
                    if (kOp == kFfnGateUp) {
                        __syncwarp();
                        tmem_load32(taddr + c + kBN / 2, w);
                    }
                    tmem_load_wait();
                    if (kOp == kFfnGateUp) {
                        // x = h = act(gate) * up
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = v[i];
                        act_all(a.act, x);
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] *= w[i];
                    }
                    if (kOp == kFfnDh) {
                        switch (a.act) {
                            case MOE_ACT_SILU: gate_grads<MOE_ACT_SILU>(v, e0, e1, w, x); break;
                            case MOE_ACT_GELU: gate_grads<MOE_ACT_GELU>(v, e0, e1, w, x); break;
                            case MOE_ACT_GELU_TANH:
                                gate_grads<MOE_ACT_GELU_TANH>(v, e0, e1, w, x);
                                break;
                            case MOE_ACT_RELU: gate_grads<MOE_ACT_RELU>(v, e0, e1, w, x); break;
                            default: gate_grads<MOE_ACT_NONE>(v, e0, e1, w, x); break;
                        }
                    }
                    if (kOp == kFfnDown && a.residual) e0.add_to(v);
                    fetch(c + 32);
                    if (r < rows) {
                        const int64_t at = r * all_cols + c0 + c;
                        const int64_t own = r * a.ld + c0 + c;  // in the workspace
                        if (kOp == kFfnGateUp) {
                            store_row(a.out[0] + own, x, cols - c, true);
                            if (a.keep) {
                                store_row(a.out[1] + at, v, cols - c, wide);
                                store_row(a.out[2] + at, w, cols - c, wide);
                            }
                        } else if (kOp == kFfnDh) {
                            store_row(a.out[0] + own, x, cols - c, true);
                            store_row(a.out[1] + own, v, cols - c, true);
                            store_row(a.out[2] + own, w, cols - c, true);
                        } else {
                            store_row(a.out[t.prod] + at, v, cols - c, wide);
                        }
                    }
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) arrive_remote_relaxed(acc ? empty1 : empty0);
        }
        if (kOp == kFfnDw) {
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // stores have landed
            __syncwarp();
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    cluster_barrier();  // both CTAs are done with TMEM and each other's barriers
    if (warp == 1) {
        tc_fence_after_sync();
        __syncwarp();
        tmem_dealloc_2cta(tmem, 2 * kBN);
    }
}

// The shared tiles: a warp adds the parts of 32 rows x 8 columns, in the order
// of their slices, and stores them.
constexpr int kJoinThreads = 256;

template <FfnOp kOp, int kBN>
__global__ void __launch_bounds__(kJoinThreads)
    ffn_join_kernel(const __grid_constant__ FfnArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x % 32;
    const int at = blockIdx.x * (kJoinThreads / 32) + threadIdx.x / 32;
    // 8 groups of 32 rows x kBN / 8 of 8 columns a tile
    constexpr int kWide = kBN / 32;
    const int local = at / (32 * kWide), chunk = at % (32 * kWide) / 4, piece = at % 4;
    const FfnPlan &p = a.plan;
    const FfnTile t = ffn_tile<kOp, kBN>(a, p.whole + local);
    int64_t rows;
    int all_cols;
    ffn_dims<kOp>(a, t.prod, &rows, &all_cols);
    const int64_t r = static_cast<int64_t>(t.m) * kFfnTile + chunk / kWide * 32 + lane;
    const int c0 = t.n * kBN + chunk % kWide * 32 + piece * 8;
    if (c0 >= all_cols || r >= rows) return;
    const int64_t to = r * all_cols + c0;
    uint4 res = make_uint4(0, 0, 0, 0);
    if (kOp == kFfnDown && a.residual)
        res = __ldcg(reinterpret_cast<const uint4 *>(a.residual + to));
    const int64_t slices = static_cast<int64_t>(p.tiles - p.whole) * p.nk;
    const int64_t from = static_cast<int64_t>(local) * p.nk, end = from + p.nk;
    // the parts [q, last) reach into the tile
    int q = static_cast<int>(from * p.parts / slices);
    while (slices * (q + 1) / p.parts <= from) ++q;
    while (q > 0 && slices * q / p.parts > from) --q;
    int last = q + 1;
    while (last < p.parts && slices * last / p.parts < end) ++last;
    const float *part = a.part + chunk * 1024 + piece * 256 + 4 * lane;
    float v[8] = {};
    // the first part's second tile, else a part's first
    int slot = 2 * q + (slices * q / p.parts < from ? 1 : 0);
    for (; q < last; q += 4) {
        float4 f[4][2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (q + j < last) {
                const float *s = part + static_cast<int64_t>(j == 0 ? slot : 2 * (q + j)) *
                                            (kFfnTile * kBN);
                f[j][0] = __ldcg(reinterpret_cast<const float4 *>(s));
                f[j][1] = __ldcg(reinterpret_cast<const float4 *>(s + 128));
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (q + j < last) {
                v[0] += f[j][0].x, v[1] += f[j][0].y, v[2] += f[j][0].z, v[3] += f[j][0].w;
                v[4] += f[j][1].x, v[5] += f[j][1].y, v[6] += f[j][1].z, v[7] += f[j][1].w;
            }
        }
        slot = 2 * (q + 4);
    }
    const uint32_t *rp = reinterpret_cast<const uint32_t *>(&res);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack_bf16x2(rp[i]);
        o[i] = kOp == kFfnDown ? pack_bf16x2(v[2 * i] + f.x, v[2 * i + 1] + f.y)
                               : pack_bf16x2(v[2 * i], v[2 * i + 1]);
    }
    *reinterpret_cast<uint4 *>(a.out[t.prod] + to) = make_uint4(o[0], o[1], o[2], o[3]);
}

template <FfnOp kOp, int kBN>
cudaError_t launch_tiles(const FfnMaps &maps, const FfnArgs &a, int *launches, cudaStream_t s) {
    const size_t smem = FfnTraits<kOp, kBN>::kShared;
    auto kern = ffn_kernel<kOp, kBN>;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t err = allow_shared(kern, smem, allowed);
    if (err != cudaSuccess) return err;
    *launches += 1;
    return launch_pdl(kern, dim3(static_cast<unsigned>(2 * a.plan.pairs)), dim3(kFfnThreads), smem,
                      s, 2, maps, a);
}

template <FfnOp kOp>
cudaError_t launch_op(const FfnMaps &maps, const FfnArgs &a, int *launches, cudaStream_t s) {
    return a.plan.bn == 128 ? launch_tiles<kOp, 128>(maps, a, launches, s)
                            : launch_tiles<kOp, 256>(maps, a, launches, s);
}

template <FfnOp kOp>
cudaError_t launch_join(const FfnArgs &a, int *launches, cudaStream_t s) {
    if (a.plan.parts == 0) return cudaSuccess;
    *launches += 1;
    const dim3 blocks(static_cast<unsigned>((a.plan.tiles - a.plan.whole) * a.plan.bn / 8));
    return a.plan.bn == 128
               ? launch_pdl(ffn_join_kernel<kOp, 128>, blocks, dim3(kJoinThreads), 0, s, 1, a)
               : launch_pdl(ffn_join_kernel<kOp, 256>, blocks, dim3(kJoinThreads), 0, s, 1, a);
}

int64_t up_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Measured times in us: a slice of a tile, and its epilogue on its own.
double slice_us(int bn) { return bn == 256 ? 0.29 : 0.21; }
double epilogue_us(FfnOp op, int bn) { return (op == kFfnDh ? 4.0 : 2.5) * bn / 256; }

// The plan for tiles of bn columns, and its time in us.
double plan_tiles(FfnOp op, int64_t N, int H, int I, int bn, int P, FfnPlan *plan) {
    FfnPlan p;
    const int64_t m = up_div(N, kFfnTile);
    int64_t tiles;
    switch (op) {
        case kFfnGateUp:
            tiles = m * up_div(I, bn / 2);
            p.nk = static_cast<int>(up_div(H, kSliceK));
            break;
        case kFfnDh:
            tiles = m * up_div(I, bn);
            p.nk = static_cast<int>(up_div(H, kSliceK));
            break;
        case kFfnDown:
            tiles = m * up_div(H, bn);
            p.nk = static_cast<int>(up_div(I, kSliceK));
            break;
        case kFfnDx:
            tiles = m * up_div(H, bn);
            p.nk = static_cast<int>(2 * up_div(I, kSliceK));
            break;
        default:
            tiles = 2 * up_div(I, kFfnTile) * up_div(H, bn) + up_div(H, kFfnTile) * up_div(I, bn);
            p.nk = static_cast<int>(up_div(N, kSliceK));
    }
    p.bn = bn;
    p.tiles = static_cast<int>(tiles);
    p.whole = p.tiles;
    p.parts = 0;
    p.pairs = p.tiles < P ? p.tiles : P;
    p.dx_tiles = p.dx_nk = p.dx_first = 0;
    const double slice = slice_us(bn), epilogue = epilogue_us(op, bn);
    const double waves = static_cast<double>(up_div(tiles, P));
    double us = waves * (p.nk * slice > epilogue ? p.nk * slice : epilogue) + epilogue;
    if (op != kFfnGateUp && op != kFfnDh) {  // theirs need whole sums
        const int rest = p.tiles % P;
        const int64_t slices = static_cast<int64_t>(rest) * p.nk;
        const int64_t most = slices / kMinSlices;
        const int parts = most < P ? static_cast<int>(most) : P;
        // the last wave's tiles one after the other, or shared and joined
        const double shared = parts > rest ? (p.nk - static_cast<double>(slices) / parts) * slice : 0;
        if (shared > kJoinUs) {
            p.whole = p.tiles - rest;
            p.parts = parts;
            p.pairs = p.whole > 0 ? P : parts;
            us += kJoinUs - shared;
        }
    }
    *plan = p;
    return us;
}

}  // namespace

namespace {

int most_pairs(int num_sms) {
    return num_sms < 4 ? 1 : num_sms / 2 < kFfnMaxPairs ? num_sms / 2 : kFfnMaxPairs;
}

// The better of the two widths' plans, and its time.
double best_plan(FfnOp op, int64_t N, int H, int I, int P, FfnPlan *plan) {
    FfnPlan narrow;
    const double a = plan_tiles(op, N, H, I, 256, P, plan);
    const double b = plan_tiles(op, N, H, I, 128, P, &narrow);
    if (b >= a || (op == kFfnDw && plan->nk <= kFfnBoxSlices)) return a;
    *plan = narrow;
    return b;
}

}  // namespace

// Tiles of 256 columns, or of 128 where those are so few that the half ones
// take less time: the constants (a slice, an epilogue, the join) are measured.
FfnPlan ffn_plan(FfnOp op, int64_t N, int H, int I, int num_sms) {
    FfnPlan p;
    best_plan(op, N, H, I, most_pairs(num_sms), &p);
    return p;
}

// A launch less, with its start, first copies, last epilogue and hand-over, takes
// kLaunchUs off; the tiles of both have to go evenly to the pairs, which they are
// dealt out to here as the kernel does it.
bool ffn_grads_plan(int64_t N, int H, int I, int num_sms, FfnPlan *plan) {
    const int P = most_pairs(num_sms);
    FfnPlan x, w;
    const double apart = best_plan(kFfnDx, N, H, I, P, &x) + best_plan(kFfnDw, N, H, I, P, &w);
    if (w.nk <= kFfnBoxSlices) return false;
    double best = apart + kLaunchUs;
    bool found = false;
    for (const int bn : {256, 128}) {
        FfnPlan px, pw;
        plan_tiles(kFfnDx, N, H, I, bn, P, &px);
        plan_tiles(kFfnDw, N, H, I, bn, P, &pw);
        if (static_cast<int64_t>(px.tiles) + pw.tiles > 8 * P) continue;
        FfnPlan p = pw;
        p.dx_tiles = px.tiles;
        p.dx_nk = px.nk;
        p.dx_first = px.nk > pw.nk ? 1 : 0;
        p.tiles = p.whole = px.tiles + pw.tiles;
        p.parts = 0;
        p.pairs = p.tiles < P ? p.tiles : P;
        int longest = 0;
        for (int pair = 0; pair < p.pairs; ++pair) {
            int slices = 0;
            for (int turn = 0;; ++turn) {
                const int i = turn * p.pairs + (turn % 2 ? p.pairs - 1 - pair : pair);
                if (i >= p.tiles) break;
                slices += (p.dx_first ? i < p.dx_tiles : i >= p.tiles - p.dx_tiles) ? p.dx_nk
                                                                                      : p.nk;
            }
            longest = slices > longest ? slices : longest;
        }
        const double us = longest * slice_us(bn) + epilogue_us(kFfnDw, bn);
        if (us < best) {
            best = us;
            *plan = p;
            found = true;
        }
    }
    return found;
}

size_t ffn_part_bytes(const FfnPlan &p) {
    return sizeof(float) * kFfnTile * p.bn * 2 * static_cast<size_t>(p.parts);
}

cudaError_t launch_ffn(FfnOp op, const FfnMaps &maps, const FfnArgs &a, int *launches,
                       cudaStream_t s) {
    switch (op) {
        case kFfnGateUp: return launch_op<kFfnGateUp>(maps, a, launches, s);
        case kFfnDown: return launch_op<kFfnDown>(maps, a, launches, s);
        case kFfnDh: return launch_op<kFfnDh>(maps, a, launches, s);
        case kFfnDx: return launch_op<kFfnDx>(maps, a, launches, s);
        case kFfnDw: return launch_op<kFfnDw>(maps, a, launches, s);
        default: return launch_op<kFfnGrads>(maps, a, launches, s);
    }
}

cudaError_t launch_ffn_join(FfnOp op, const FfnArgs &a, int *launches, cudaStream_t s) {
    switch (op) {
        case kFfnDown: return launch_join<kFfnDown>(a, launches, s);
        case kFfnDx: return launch_join<kFfnDx>(a, launches, s);
        case kFfnDw: return launch_join<kFfnDw>(a, launches, s);
        default: return cudaSuccess;
    }
}

}  // namespace moe
