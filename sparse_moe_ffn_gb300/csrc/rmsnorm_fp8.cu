// rmsnorm_fp8.cu -- rows to e4m3 with one fp32 scale a row, on their own
// (weights at load, activations between two 8-bit products) or as the output
// of the residual add + RMSNorm that feeds the layer:
//
//   r        = bf16(x + residual)               (x itself without a residual)
//   y        = r / sqrt(mean(r^2) + eps) * w    or * (1 + w); without the norm y = x
//   scale    = max(amax|y| / 448, 2^-100)
//   q        = e4m3(y / scale),   normed = bf16(y)
//
// One pass over the row: with inv = 1 / sqrt(mean(r^2) + eps) the largest |y|
// is inv * amax|r w|, so the sum of squares and amax|r w| go through one
// reduction, and q = e4m3(r w * (inv / scale)) needs nothing else.  The row
// stays in registers as packed bf16 (r is bf16, so nothing is lost; with the
// norm, rows over 16384 values spill 76 bytes a thread and over 32768 464), the
// gain is read once a thread.  The reduction's maximum passes NaN on, so that a
// row with a NaN or an infinity gets a NaN scale and not a plausible one.
//
// What bounds it: memory.  9 bytes an element with residual, sum and bf16 output
// (3 without the norm): 8192 x 2048 takes 24.3 us, 6220 GB/s (a plain copy of
// as many bytes: 6200), quantising alone 9.4 us, 5340 GB/s; one row 1.8 us.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "block_ops.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kScaleMin = 7.888609052210118e-31f;  // 2^-100: an all-zero row

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

struct RowArgs {
    const uint16_t *x, *residual, *w;
    uint16_t *residual_out, *normed;
    uint8_t *q;
    float *scale;
    int64_t N;
    int H;
    float eps;
    int gemma;
};

// kRow threads a row, kChunks 8-element chunks a thread (chunk c of thread t
// is elements [8 (t + c kRow), + 8)).
template <int kRow, int kChunks, bool kNorm>
__global__ void __launch_bounds__(kRow < 256 ? 256 : kRow)
    rows_to_e4m3_kernel(const RowArgs a) {
    constexpr int kThreads = kRow < 256 ? 256 : kRow;
    constexpr int kRows = kThreads / kRow;
    constexpr int kWarps = kRow / 32;
    __shared__ float part[2][kRows][kWarps][2];
    griddep_launch_dependents();
    griddep_wait();
    const int t = threadIdx.x % kRow;
    const int sub = threadIdx.x / kRow;
    const int groups = a.H / 8;
    uint4 w[kChunks];
    if (kNorm) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
            if (t + c * kRow < groups)
                w[c] = __ldcg(reinterpret_cast<const uint4 *>(a.w) + t + c * kRow);
    }
    const float add = a.gemma ? 1.f : 0.f;
    int turn = 0;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * kRows; base < a.N;
         base += static_cast<int64_t>(gridDim.x) * kRows, turn ^= 1) {
        const int64_t n = base + sub;
        const bool row = n < a.N;
        const int64_t at = n * a.H;
        uint4 r[kChunks];
        if (row) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
                if (t + c * kRow < groups)
                    r[c] = __ldcg(reinterpret_cast<const uint4 *>(a.x + at) + t + c * kRow);
            if (kNorm && a.residual) {
                uint4 b[kChunks];
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
                    if (t + c * kRow < groups)
                        b[c] = __ldcg(reinterpret_cast<const uint4 *>(a.residual + at) + t +
                                      c * kRow);
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    uint32_t *rp = reinterpret_cast<uint32_t *>(&r[c]);
                    const uint32_t *bp = reinterpret_cast<const uint32_t *>(&b[c]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 u = unpack_bf16x2(rp[i]), v = unpack_bf16x2(bp[i]);
                        rp[i] = pack_bf16x2(u.x + v.x, u.y + v.y);
                    }
                }
            }
        }
        float ss = 0.f, amax = 0.f;
        if (row) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                if (t + c * kRow >= groups) break;
                const uint32_t *rp = reinterpret_cast<const uint32_t *>(&r[c]);
                const uint32_t *wp = reinterpret_cast<const uint32_t *>(&w[c]);
                if (kNorm && a.residual_out)
                    reinterpret_cast<uint4 *>(a.residual_out + at)[t + c * kRow] = r[c];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 u = unpack_bf16x2(rp[i]);
                    if (kNorm) {
                        const float2 g = unpack_bf16x2(wp[i]);
                        ss = fmaf(u.x, u.x, ss);
                        ss = fmaf(u.y, u.y, ss);
                        amax = max_nan(amax, fabsf(u.x * (g.x + add)));
                        amax = max_nan(amax, fabsf(u.y * (g.y + add)));
                    } else {
                        amax = max_nan(amax, max_nan(fabsf(u.x), fabsf(u.y)));
                    }
                }
            }
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            if (kNorm) ss += __shfl_xor_sync(0xffffffffu, ss, d);
            amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, d));
        }
        if (kWarps > 1) {
            // two buffers in turn: a warp can be one row ahead, never two
            float(*p)[2] = part[turn][sub];
            if (t % 32 == 0) {
                p[t / 32][0] = ss;
                p[t / 32][1] = amax;
            }
            __syncthreads();
            ss = 0.f;
            amax = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                ss += p[i][0];
                amax = max_nan(amax, p[i][1]);
            }
        }
        if (!row) continue;
        const float inv = kNorm ? 1.f / sqrtf(ss / static_cast<float>(a.H) + a.eps) : 1.f;
        const float scale = max_nan(amax * inv / kE4m3Max, kScaleMin);
        const float mul = inv / scale;
        if (t == 0) a.scale[n] = scale;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            if (t + c * kRow >= groups) break;
            const uint32_t *rp = reinterpret_cast<const uint32_t *>(&r[c]);
            const uint32_t *wp = reinterpret_cast<const uint32_t *>(&w[c]);
            float v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 u = unpack_bf16x2(rp[i]);
                const float2 g = kNorm ? unpack_bf16x2(wp[i]) : make_float2(1.f, 1.f);
                v[2 * i] = kNorm ? u.x * (g.x + add) : u.x;
                v[2 * i + 1] = kNorm ? u.y * (g.y + add) : u.y;
            }
            uint2 o;
            o.x = pack_e4m3x4(v[0] * mul, v[1] * mul, v[2] * mul, v[3] * mul);
            o.y = pack_e4m3x4(v[4] * mul, v[5] * mul, v[6] * mul, v[7] * mul);
            reinterpret_cast<uint2 *>(a.q + at)[t + c * kRow] = o;
            if (kNorm && a.normed) {
                uint4 m;
                m.x = pack_bf16x2(v[0] * inv, v[1] * inv);
                m.y = pack_bf16x2(v[2] * inv, v[3] * inv);
                m.z = pack_bf16x2(v[4] * inv, v[5] * inv);
                m.w = pack_bf16x2(v[6] * inv, v[7] * inv);
                reinterpret_cast<uint4 *>(a.normed + at)[t + c * kRow] = m;
            }
        }
    }
}

template <int kRow, int kChunks, bool kNorm>
cudaError_t launch_rows(const RowArgs &a, int num_sms, cudaStream_t s) {
    constexpr int kThreads = kRow < 256 ? 256 : kRow;
    constexpr int kRows = kThreads / kRow;
    int64_t blocks = (a.N + kRows - 1) / kRows;
    static const int resident = [] {
        int n = 0;
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, rows_to_e4m3_kernel<kRow, kChunks, kNorm>,
                                                      kThreads, 0);
        return n > 0 ? n : 1;
    }();
    // Four times what fits at once: blocks that follow one another keep the
    // memory busier than a loop does (8192 x 2048, norm 25.7 -> 24.3 us); rows
    // of up to 512 values are too short for that (65536 x 256 in one go 33.6 us
    // against 26.5).
    const int64_t limit = static_cast<int64_t>(num_sms) * resident * (a.H > 512 ? 4 : 1);
    if (blocks > limit) blocks = limit;
    return launch_pdl(rows_to_e4m3_kernel<kRow, kChunks, kNorm>,
                      dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, s, 1, a);
}

// Threads a row and chunks a thread.  Where the whole batch is in flight at one
// chunk a thread, that is the shortest path; beyond it (by about 200000 chunks
// for the norm, 100000 without it) fewer threads a row, two or four chunks each,
// keep more bytes in flight between the reductions: 8192 x 2048, norm 27.1
// -> 25.1 us and plain 11.3 -> 9.6 (in a loop, as fits at once); 64 x 2048 the
// other way, 2.1 against 2.3 and 1.5 against 1.9.  Rows over 2048 take two or
// four chunks a thread in any case, over 32768 eight.
template <bool kNorm>
cudaError_t launch_any(const RowArgs &a, int num_sms, cudaStream_t s) {
    const int groups = a.H / 8;
    const bool deep = a.N * groups >= (kNorm ? 200000 : 100000);
    if (groups <= 32) return launch_rows<32, 1, kNorm>(a, num_sms, s);
    if (groups <= 256 && deep) {
        if constexpr (kNorm) {
            if (groups <= 64) return launch_rows<32, 2, kNorm>(a, num_sms, s);
            if (groups <= 128) return launch_rows<64, 2, kNorm>(a, num_sms, s);
            return launch_rows<128, 2, kNorm>(a, num_sms, s);
        } else {
            if (groups <= 128) return launch_rows<32, 4, kNorm>(a, num_sms, s);
            return launch_rows<64, 4, kNorm>(a, num_sms, s);
        }
    }
    if (groups <= 64) return launch_rows<64, 1, kNorm>(a, num_sms, s);
    if (groups <= 128) return launch_rows<128, 1, kNorm>(a, num_sms, s);
    if (groups <= 256) return launch_rows<256, 1, kNorm>(a, num_sms, s);
    if (groups <= 512) return launch_rows<256, 2, kNorm>(a, num_sms, s);
    if (groups <= 1024) return launch_rows<256, 4, kNorm>(a, num_sms, s);
    if (groups <= 2048) return launch_rows<512, 4, kNorm>(a, num_sms, s);
    if (groups <= 4096) return launch_rows<1024, 4, kNorm>(a, num_sms, s);
    return launch_rows<1024, kMaxRowH / 8 / 1024, kNorm>(a, num_sms, s);
}

}  // namespace

cudaError_t launch_add_rmsnorm_fp8(const uint16_t *x, const uint16_t *residual, const uint16_t *w,
                                   int64_t N, int H, float eps, int gemma, uint16_t *residual_out,
                                   uint8_t *q, float *scale, uint16_t *normed, int num_sms,
                                   cudaStream_t s) {
    return launch_any<true>({x, residual, w, residual_out, normed, q, scale, N, H, eps, gemma},
                            num_sms, s);
}

cudaError_t launch_quantize_fp8(const uint16_t *x, int64_t N, int H, uint8_t *q, float *scale,
                                int num_sms, cudaStream_t s) {
    return launch_any<false>({x, nullptr, nullptr, nullptr, nullptr, q, scale, N, H, 0.f, 0},
                             num_sms, s);
}

}  // namespace moe
