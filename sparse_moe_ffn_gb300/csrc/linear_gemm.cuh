// linear_gemm.cuh -- what the tensor-core kernels of moe_linear share: operand
// types, cluster and CTA-pair instructions, and the tile constants.
//
// A K slice is 128 bytes of every operand row (64 bf16 or 128 e4m3 values),
// one row of the 128-byte swizzle, and one MMA consumes 32 of them; so the two
// operand types differ in the MMA's kind and nowhere else.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include <atomic>

#include "block_ops.cuh"
#include "cluster.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kSliceBytes = 128;   // of an operand row
constexpr int kMmaBytes = 32;      // of an operand row, per MMA
constexpr int kRowsBytes128 = 128 * kSliceBytes;

// Instruction descriptor: K-major operands, fp32 accumulator, M x N.
template <bool kFp8>
__host__ __device__ constexpr uint32_t linear_idesc(int M, int N) {
    // kind::f8f6f4 numbers e4m3 0 in the operand fields
    return kFp8 ? (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) |
                      (static_cast<uint32_t>(M >> 4) << 24)
                : idesc_bf16_f32(M, N);
}

template <bool kFp8>
__device__ __forceinline__ void linear_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
    if (kFp8)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        mma_f16kind(d, a, b, idesc, accumulate);
}

template <bool kFp8>
__device__ __forceinline__ void linear_mma_pair(uint32_t d, uint64_t a, uint64_t b,
                                                uint32_t idesc, uint32_t accumulate) {
    if (kFp8)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
}

// One lane of the warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(e));
    return e != 0;
}

// mbar_wait by a whole warp, the same answer in every lane.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity,
                                          volatile int *abort_flag) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
}

// Waits for work already in flight, after a failure too (which mbar_wait would
// cut short): nothing may be under way when a kernel gives its memory back.
// Bounded like every wait.
__device__ __forceinline__ void drain_wait(uint64_t *bar, uint32_t parity) {
    volatile int never = 0;
    mbar_wait(bar, parity, &never);
}

// ------------------------------------------------------------------ CTA pairs

// Arrival that orders no memory accesses (the waiter only needs to know that
// this warp's TMEM reads have returned).
__device__ __forceinline__ void arrive_remote_relaxed(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
                 : "memory");
}

// Tiled load into this CTA's shared memory that completes on a barrier of the
// pair's even CTA (`bar`: a shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *map, uint32_t bar,
                                                 int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
        ".mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}

__device__ __forceinline__ void tmem_alloc_2cta(uint32_t *dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(dst_smem)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc_2cta(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr),
                 "r"(ncols)
                 : "memory");
}

// One arrival on the barrier at `bar`'s offset in the CTAs of `mask`, once the
// pair's MMAs issued so far by this thread have completed.
__device__ __forceinline__ void commit_2cta(uint64_t *bar, uint16_t mask) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(smem_addr(bar)),
        "h"(mask)
        : "memory");
}

// ---------------------------------------------------------------- launchers

// Lets `kern` have `bytes` of dynamic shared memory, once a device (`done`: one
// bit each; the call costs 0.2 us).
template <typename Kernel>
cudaError_t allow_shared(Kernel kern, size_t bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(bytes));
    if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return err;
}

// tm_x / tm_w: boxes of rows x 128 bytes over the operands (rows: see
// linear_tiling); see the kernels for how they split a tile.
struct LinearTiling {
    int pair;     // 1: the CTA-pair kernel, 0: the split-K kernel
    int bn;       // pair: outputs a tile (256 tokens); split: tokens a tile (128 outputs)
    int split;    // split: CTAs of a cluster that share a tile's K
};

LinearTiling linear_tiling(const LinearArgs &a, int num_sms);
int linear_x_box(const LinearTiling &t);
int linear_w_box(const LinearTiling &t);
// Whether the pair kernel can store through a tensor map (tm_out: boxes of 32
// rows x 32 outputs, 64-byte swizzle for bf16, 128-byte for fp32; else null).
bool linear_out_rows_aligned(const LinearArgs &a);
cudaError_t launch_linear_pair(const CUtensorMap &tm_x, const CUtensorMap &tm_w,
                               const CUtensorMap *tm_out, const LinearArgs &a,
                               const LinearTiling &t, int num_sms, cudaStream_t s);
cudaError_t launch_linear_split(const CUtensorMap &tm_x, const CUtensorMap &tm_w,
                                const LinearArgs &a, const LinearTiling &t, cudaStream_t s);

}  // namespace moe
