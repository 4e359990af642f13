// linear_pair.cu -- moe_linear for large batches: the two CTAs of a cluster
// run one tcgen05 MMA of 256 tokens x kBN outputs (cta_group::2), so that every
// operand byte a CTA fetches serves 256 rows of the other side.
//
// Even CTA: tokens 0-127 of the tile and the first half of its weight rows;
// odd CTA: tokens 128-255 and the second half; each CTA's TMEM receives its
// own 128 tokens x kBN outputs.  Persistent clusters take tiles in an order
// that keeps the tiles in flight within a few token and output tiles (see
// tile_of), so that an operand is read from memory about once.
//
//   warp 0     producer: TMA copies of both operands' K slices; the even CTA's
//              barrier counts both CTAs' bytes
//   warp 1     TMEM; in the even CTA, the MMAs
//   warps 2-9  epilogue: warp w owns TMEM lanes 32 (w % 4) .. + 31 (one token a
//              lane) and half of the outputs; two accumulators alternate, so
//              a tile's epilogue runs under the next tile's MMAs
// In warps 0 and 1 the whole warp runs the loop and one elected lane issues:
// the compiler then keeps descriptors and barriers in uniform registers.  With
// the loop in one lane a K slice took 611 cycles, so 551 (512 is what the MMAs
// themselves need).
//
// A lane holds 32 consecutive outputs of one token.  Where rows of the output
// start on 16 bytes, a warp's 32 x 32 outputs go through shared memory into a
// tensor-map store (stored from the lanes, 32 bytes of 32 rows each, an e4m3
// call of 8192 x 2048 x 8192 took 112 us, 24 of them for the stores);
// otherwise (an odd number of outputs, an output that starts anywhere) they are
// turned there and leave with neighbouring lanes on neighbouring outputs.
//
// What bounds it, measured on a GB300: the tensor cores at the clock that the
// power limit leaves (1.3 to 1.6 GHz in a loop of calls).  8192 x 8192 x 2048 in
// bf16 onto a residual: 174 us, 1580 TFLOP/s (256 tiles are 3.4 waves of 76
// pairs and take 4); 8192 x 2048 x 8192 in e4m3 with bias and SiLU: 92 us, 3000
// TFLOP/s, of which the epilogue's shared-memory and store traffic costs the
// MMAs about 15 us.  Bare products in bf16 run at 0.92 to 0.97 of the library's
// rate, 0.85 at 2048 x 2048 x 2048.  Rows of the output that start on no 16
// bytes leave two bytes a lane and are far from any bound: 4096 x 512 x 4001 in
// e4m3 onto a residual 65 us, 10 for its bytes.  Tried and not kept: 16 epilogue warps (6% fewer cycles in e4m3, the
// same time), four or six stages, 128 outputs a tile where 256 fill the SMs.
// Every wait is bounded; a CTA that gives up records MOE_ERR_DEVICE_TIMEOUT.
#include "linear_epilogue.cuh"
#include "linear_gemm.cuh"

namespace moe {

namespace {

constexpr int kEpiWarps = 8;
constexpr int kPairThreads = 64 + 32 * kEpiWarps;
constexpr int kStages = 5;
constexpr int kTokens = 256;  // of a tile

template <int kBN>
struct PairTile {
    static constexpr int kBBytes = kBN / 2 * kSliceBytes;
    static constexpr int kStageBytes = kRowsBytes128 + kBBytes;
    static constexpr int kColsPerWarp = kBN / 2;
};

struct PairShared {
    uint64_t full[kStages];   // even CTA: both CTAs' bytes of a stage landed
    uint64_t empty[kStages];  // both: the MMAs are done with a stage
    uint64_t acc_full[2];     // both: an accumulator is complete
    uint64_t acc_empty[2];    // even CTA: both CTAs' epilogues have read one
    uint64_t drain;           // even CTA: every MMA has completed
    uint32_t tmem_base;
    int abort_flag;
    alignas(16) float scale[kEpiWarps][128];  // w_scale of a warp's columns
    alignas(16) float bias[kEpiWarps][128];
};

// Outputs on their way out: 32 tokens x 32 outputs a warp, twice in bf16.
constexpr int kOutBytes = 4096;
static_assert(32 * 32 * 4 <= kOutBytes, "a turned chunk fits");

// Tiles run through bands of kBand token tiles, output tile by output tile:
// the ~76 tiles in flight cover 8 token tiles and ~10 output tiles (bands of 4
// and 16 took the same time).
constexpr int kBand = 8;

__device__ __forceinline__ void tile_of(int tile, int m_tiles, int n_tiles, int *m, int *n) {
    const int band = tile / (kBand * n_tiles);
    const int first = band * kBand;
    const int rows = min(kBand, m_tiles - first);
    const int in = tile - band * kBand * n_tiles;
    *m = first + in % rows;
    *n = in / rows;
}

// 32-byte load that stays out of L1 (8 words; p 32-byte aligned)
__device__ __forceinline__ void ld_global_v8(const void *p, uint32_t *v) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                   "=r"(v[6]), "=r"(v[7])
                 : "l"(p)
                 : "memory");
}

// 32 bf16 values of a residual row whose start is aligned for vectors.
struct Residual32 {
    uint32_t w[16];
    // the first `left` values exist (a multiple of 8); 32-byte loads if wide
    __device__ __forceinline__ void load(const uint16_t *p, int left, bool wide) {
        if (wide && left >= 32) {
            ld_global_v8(p, &w[0]);
            ld_global_v8(p + 16, &w[8]);
        } else {
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
    }
    __device__ __forceinline__ void add(float (&v)[32]) const {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 f = unpack_bf16x2(w[i]);
            v[2 * i] += f.x;
            v[2 * i + 1] += f.y;
        }
    }
};

// This lane's row of a 32 x 32 chunk, as a tensor-map store with swizzled rows
// of 64 bytes (bf16) or 128 (fp32) reads it: neighbouring lanes' 16-byte pieces
// fall on different banks.
__device__ __forceinline__ void write_row(uint8_t *buf, int lane, bool fp32,
                                          const float (&v)[32]) {
    if (fp32) {
        uint8_t *row = buf + lane * 128;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            *reinterpret_cast<float4 *>(row + 16 * (j ^ (lane & 7))) =
                make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    } else {
        uint8_t *row = buf + lane * 64;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4 *>(row + 16 * (j ^ ((lane >> 1) & 3))) = make_uint4(
                pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
    }
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, const void *src, int c0,
                                             int c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];"
                 ::"l"(map), "r"(smem_addr(src)), "r"(c0), "r"(c1)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// The same outputs, any alignment and any part of them inside [0, O): turned in
// the buffer (columns swapped by row, so that neither side's words share a
// bank), then a lane an output, eight tokens at a time with the next eight's
// residuals on their way.
constexpr int kTurn = 8;

__device__ __forceinline__ void load_turned(const LinearArgs &a, int64_t at, int left,
                                            uint16_t (&u)[kTurn]) {
#pragma unroll
    for (int r = 0; r < kTurn; ++r)
        u[r] = r < left ? __ldcg(a.residual + at + static_cast<int64_t>(r) * a.O) : 0;
}

// `at`: the lane's output of the first token; `rows`: tokens that exist (0 for
// a lane whose output does not).
__device__ __forceinline__ void store_turned(const LinearArgs &a, float *buf, int64_t at, int rows,
                                             int lane, const float (&v)[32],
                                             uint16_t (&next)[kTurn]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) buf[lane * 32 + (i ^ lane)] = v[i];
    __syncwarp();
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += kTurn, at += static_cast<int64_t>(kTurn) * a.O) {
        float x[kTurn];
#pragma unroll
        for (int r = 0; r < kTurn; ++r) x[r] = buf[(r0 + r) * 32 + (lane ^ (r0 + r))];
        if (a.residual) {
#pragma unroll
            for (int r = 0; r < kTurn; ++r)
                x[r] += __uint_as_float(static_cast<uint32_t>(next[r]) << 16);
            load_turned(a, at + static_cast<int64_t>(kTurn) * a.O, rows - r0 - kTurn, next);
        }
#pragma unroll
        for (int r = 0; r < kTurn; ++r) {
            if (r0 + r >= rows) break;
            const int64_t i = at + static_cast<int64_t>(r) * a.O;
            if (a.out_fp32) static_cast<float *>(a.out)[i] = x[r];
            else static_cast<__nv_bfloat16 *>(a.out)[i] = __float2bfloat16_rn(x[r]);
        }
    }
    __syncwarp();
}

template <bool kFp8, int kBN>
__global__ void __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tm_x,
                       const __grid_constant__ CUtensorMap tm_w,
                       const __grid_constant__ CUtensorMap tm_out, const LinearArgs a,
                       const int vec) {
    using T = PairTile<kBN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *tiles = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *out_bufs = tiles + kStages * T::kStageBytes;
    PairShared *sm = reinterpret_cast<PairShared *>(out_bufs + kEpiWarps * kOutBytes);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_ctarank();
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
        prefetch_tensor_map(&tm_x);
        prefetch_tensor_map(&tm_w);
    }
    if (warp == 1) tmem_alloc_2cta(&sm->tmem_base, 2 * kBN);
    tc_fence_before_sync();
    __syncthreads();
    cluster_barrier();  // both CTAs' barriers exist before any remote arrival
    tc_fence_after_sync();
    const uint32_t tmem = sm->tmem_base;
    volatile int *abort_flag = &sm->abort_flag;
    griddep_launch_dependents();
    griddep_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.status) *a.status = MOE_OK;

    const int m_tiles = static_cast<int>((a.N + kTokens - 1) / kTokens);
    const int n_tiles = (a.O + kBN - 1) / kBN;
    const int total = m_tiles * n_tiles;
    const int first = blockIdx.x / 2, step = gridDim.x / 2;
    const int per_slice = kFp8 ? kSliceBytes : kSliceBytes / 2;  // values of K
    const int nk = (a.K + per_slice - 1) / per_slice;

    if (warp == 0) {
        const bool issues = elect_one();
        // stages filled so far; the stage and the parity of its last release
        int64_t g = 0;
        int s = 0;
        uint32_t parity = 1;
        bool failed = false;
        for (int tile = first; tile < total && !failed; tile += step) {
            int m, n;
            tile_of(tile, m_tiles, n_tiles, &m, &n);
            const int row = m * kTokens + static_cast<int>(rank) * 128;
            const int wrow = n * kBN + static_cast<int>(rank) * (kBN / 2);
            for (int kc = 0; kc < nk; ++kc, ++g) {
                if (g >= kStages && !warp_wait(&sm->empty[s], parity, abort_flag)) {
                    if (issues) {
                        record_status(a.status, MOE_ERR_DEVICE_TIMEOUT);
                        *abort_flag = 1;
                    }
                    failed = true;
                    break;
                }
                if (issues) {
                    uint8_t *st = tiles + s * T::kStageBytes;
                    const uint32_t bar = map_to_rank(smem_addr(&sm->full[s]), 0);
                    if (leader) mbar_arrive_expect_tx(&sm->full[s], 2 * T::kStageBytes);
                    tma_load_2d_pair(st, &tm_x, bar, kc * per_slice, row);
                    tma_load_2d_pair(st + kRowsBytes128, &tm_w, bar, kc * per_slice, wrow);
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
            constexpr uint32_t idesc = linear_idesc<kFp8>(kTokens, kBN);
            const uint64_t desc0 = sw128_kmajor_desc(smem_addr(tiles));
            int s = 0, it = 0;
            uint32_t phase = 0;
            bool failed = false;
            for (int tile = first; tile < total && !failed; tile += step, ++it) {
                const int acc = it & 1;
                const uint32_t use = it >> 1;
                if (use > 0 && !warp_wait(&sm->acc_empty[acc], (use - 1) & 1, abort_flag)) {
                    failed = true;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t d = tmem + acc * kBN;
                for (int kc = 0; kc < nk; ++kc) {
                    if (!warp_wait(&sm->full[s], phase, abort_flag)) {
                        failed = true;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint64_t da = desc0 + s * (T::kStageBytes >> 4);
                    const uint64_t db = da + (kRowsBytes128 >> 4);
                    if (issues) {
#pragma unroll
                        for (int kk = 0; kk < kSliceBytes / kMmaBytes; ++kk)
                            linear_mma_pair<kFp8>(d, da + 2 * kk, db + 2 * kk, idesc,
                                                  kk == 0 ? kc != 0 : 1);
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
        const int quarter = warp % 4, half = (warp - 2) / 4, ew = warp - 2;
        constexpr int kCols = T::kColsPerWarp;
        float *scale_s = sm->scale[ew], *bias_s = sm->bias[ew];
        const uint32_t empty0 = map_to_rank(smem_addr(&sm->acc_empty[0]), 0);
        const uint32_t empty1 = map_to_rank(smem_addr(&sm->acc_empty[1]), 0);
        uint8_t *buf = out_bufs + ew * kOutBytes;
        const bool wide_res =
            a.O % 16 == 0 && reinterpret_cast<uintptr_t>(a.residual) % 32 == 0;
        // a tile's scales and bias are read a tile ahead, in registers
        float sw_next[kCols / 32], b_next[kCols / 32], sx_next = 1.f;
        auto fetch_factors = [&](int tile) {
            if (tile >= total) return;
            int m, nt;
            tile_of(tile, m_tiles, n_tiles, &m, &nt);
            const int64_t n = static_cast<int64_t>(m) * kTokens + rank * 128 + quarter * 32 + lane;
#pragma unroll
            for (int i = 0; i < kCols / 32; ++i) {
                const int o = nt * kBN + half * kCols + 32 * i + lane;
                sw_next[i] = kFp8 && o < a.O ? __ldcg(a.w_scale + o) : 0.f;
                b_next[i] =
                    a.bias && o < a.O
                        ? __uint_as_float(static_cast<uint32_t>(__ldcg(a.bias + o)) << 16)
                        : 0.f;
            }
            if (kFp8) sx_next = n < a.N ? __ldcg(a.x_scale + n) : 0.f;
        };
        fetch_factors(first);
        int it = 0, chunk = 0;
        for (int tile = first; tile < total; tile += step, ++it) {
            int m, nt;
            tile_of(tile, m_tiles, n_tiles, &m, &nt);
            const int acc = it & 1;
            const int o0 = nt * kBN + half * kCols;
            const int64_t n0 = static_cast<int64_t>(m) * kTokens + rank * 128 + quarter * 32;
            const int64_t n = n0 + lane;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kCols / 32; ++i) {
                if (kFp8) scale_s[32 * i + lane] = sw_next[i];
                bias_s[32 * i + lane] = b_next[i];
            }
            const float sx = sx_next;
            fetch_factors(tile + step);
            // columns of this warp that exist (warp-uniform)
            const int cols = n0 < a.N ? min(kCols, a.O - o0) : 0;
            const int rows = a.N - n0 < 32 ? static_cast<int>(a.N - n0) : 32;
            // the residual is read 32 columns ahead of their use
            Residual32 res;
            auto fetch = [&](int c) {
                if (vec && a.residual && c < cols && n < a.N)
                    res.load(a.residual + n * a.O + o0 + c, cols - c, wide_res);
            };
            fetch(0);
            __syncwarp();
            bool ok = true;
            if (lane == 0) ok = mbar_wait(&sm->acc_full[acc], (it >> 1) & 1, abort_flag);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) {
                if (lane == 0) {
                    record_status(a.status, MOE_ERR_DEVICE_TIMEOUT);
                    *abort_flag = 1;
                }
                break;
            }
            tc_fence_after_sync();
            const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                                   acc * kBN + half * kCols;
#pragma unroll 1
            for (int c = 0; c < cols; c += 32, ++chunk) {
                float v[32];
                // (unaligned rows) this lane's output of the chunk
                const int64_t at = n0 * a.O + o0 + c + lane;
                const int mine = o0 + c + lane < a.O ? rows : 0;
                uint16_t turned[kTurn];
                if (!vec && a.residual) load_turned(a, at, mine, turned);
                __syncwarp();  // TMEM wants whole warps
                tmem_load32(taddr + c, v);
                tmem_load_wait();
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 b = *reinterpret_cast<const float4 *>(bias_s + c + i);
                    if (kFp8) {
                        const float4 w = *reinterpret_cast<const float4 *>(scale_s + c + i);
                        v[i] = fmaf(v[i], sx * w.x, b.x);
                        v[i + 1] = fmaf(v[i + 1], sx * w.y, b.y);
                        v[i + 2] = fmaf(v[i + 2], sx * w.z, b.z);
                        v[i + 3] = fmaf(v[i + 3], sx * w.w, b.w);
                    } else {
                        v[i] += b.x;
                        v[i + 1] += b.y;
                        v[i + 2] += b.z;
                        v[i + 3] += b.w;
                    }
                }
                act_all(a.act, v);
                if (vec) {
                    if (a.residual) res.add(v);
                    fetch(c + 32);
                    // the buffer (bf16: the half in turn) has left once at
                    // most the other half's store is in flight
                    uint8_t *b = buf;
                    if (a.out_fp32) {
                        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    } else {
                        asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                        b += (chunk & 1) * (kOutBytes / 2);
                    }
                    __syncwarp();
                    write_row(b, lane, a.out_fp32, v);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) tma_store_2d(&tm_out, b, o0 + c, static_cast<int>(n0));
                } else {
                    store_turned(a, reinterpret_cast<float *>(buf), at, mine, lane, v, turned);
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) arrive_remote_relaxed(acc ? empty1 : empty0);
        }
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // stores have landed
        __syncwarp();
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

template <bool kFp8, int kBN>
cudaError_t launch_one(const CUtensorMap &tm_x, const CUtensorMap &tm_w,
                       const CUtensorMap *tm_out, const LinearArgs &a, int num_sms,
                       cudaStream_t s) {
    const size_t smem = 1024 + static_cast<size_t>(kStages) * PairTile<kBN>::kStageBytes +
                        kEpiWarps * kOutBytes + sizeof(PairShared);
    auto kern = linear_pair_kernel<kFp8, kBN>;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t err = allow_shared(kern, smem, allowed);
    if (err != cudaSuccess) return err;
    const int64_t tiles = (a.N + kTokens - 1) / kTokens * ((a.O + kBN - 1) / kBN);
    const int64_t pairs = tiles < num_sms / 2 ? tiles : num_sms / 2;
    return launch_pdl(kern, dim3(static_cast<unsigned>(2 * pairs)), dim3(kPairThreads), smem, s, 2,
                      tm_x, tm_w, tm_out ? *tm_out : tm_x, a, tm_out ? 1 : 0);
}

}  // namespace

bool linear_out_rows_aligned(const LinearArgs &a) {
    const int64_t ld = static_cast<int64_t>(a.O) * (a.out_fp32 ? 4 : 2);
    return ld % 16 == 0 && reinterpret_cast<uintptr_t>(a.out) % 16 == 0 &&
           (!a.residual ||
            (a.O % 8 == 0 && reinterpret_cast<uintptr_t>(a.residual) % 16 == 0));
}

cudaError_t launch_linear_pair(const CUtensorMap &tm_x, const CUtensorMap &tm_w,
                               const CUtensorMap *tm_out, const LinearArgs &a,
                               const LinearTiling &t, int num_sms, cudaStream_t s) {
    if (t.bn == 256)
        return a.fp8 ? launch_one<true, 256>(tm_x, tm_w, tm_out, a, num_sms, s)
                     : launch_one<false, 256>(tm_x, tm_w, tm_out, a, num_sms, s);
    return a.fp8 ? launch_one<true, 128>(tm_x, tm_w, tm_out, a, num_sms, s)
                 : launch_one<false, 128>(tm_x, tm_w, tm_out, a, num_sms, s);
}

}  // namespace moe
