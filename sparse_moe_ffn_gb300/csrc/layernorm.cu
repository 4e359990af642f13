// layernorm.cu -- residual add + layer norm over rows of bf16 or fp32, and its
// backward pass:
//
//   r    = x + residual, rounded to its type     (x itself without a residual)
//   mean = sum(r) / H,  rstd = 1 / sqrt(sum((r - mean)^2) / H + eps)
//   out  = (r - mean) rstd w + b
//
//   n = (r - mean) rstd,  t = dout w
//   dx = rstd (t - mean(t) - n mean(t n)) + dresidual
//   dw = sum over rows of dout n,  db = sum over rows of dout
//
// The variance is the sum of the squared deviations themselves, whatever the mean
// is: a row stays in registers, or, where it is too long for them, is read again
// from L2 for the deviations and for the result (the launchers say from which
// length on).  In the backward pass a thread keeps its columns' two sums over up to
// kRunRows rows in registers as well; in rows over kSumColumnsH values a kernel of
// its own makes them, from a second reading of x and dout.  The blocks' sums are
// added in 64 bits, in a fixed order, by a last kernel.
//
// Rows whose length or arrays allow 16-byte accesses take them, others go value
// by value.
#include <cuda_bf16.h>

#include <initializer_list>

#include "kernels.cuh"
#include "layernorm.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

// kVec neighbouring values of a row, as they lie in memory.
template <typename T, int kVec>
struct Piece;
template <>
struct Piece<__nv_bfloat16, 8> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        u = __ldcg(reinterpret_cast<const uint4 *>(p));
    }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const {
        *reinterpret_cast<uint4 *>(p) = u;
    }
    __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const float2 a = unpack_bf16x2(u.x), b = unpack_bf16x2(u.y), c = unpack_bf16x2(u.z),
                     d = unpack_bf16x2(u.w);
        v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
        v[4] = c.x, v[5] = c.y, v[6] = d.x, v[7] = d.y;
    }
    __device__ __forceinline__ void set(const float (&v)[8]) {
        u = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                       pack_bf16x2(v[6], v[7]));
    }
};
template <>
struct Piece<float, 4> {
    float4 f;
    __device__ __forceinline__ void load(const float *p) {
        f = __ldcg(reinterpret_cast<const float4 *>(p));
    }
    __device__ __forceinline__ void store(float *p) const { *reinterpret_cast<float4 *>(p) = f; }
    __device__ __forceinline__ void zero() { f = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&v)[4]) const {
        v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    }
    __device__ __forceinline__ void set(const float (&v)[4]) {
        f = make_float4(v[0], v[1], v[2], v[3]);
    }
};
template <>
struct Piece<__nv_bfloat16, 1> {
    uint16_t u;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        u = __ldcg(reinterpret_cast<const uint16_t *>(p));
    }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const {
        *reinterpret_cast<uint16_t *>(p) = u;
    }
    __device__ __forceinline__ void zero() { u = 0; }
    __device__ __forceinline__ void get(float (&v)[1]) const {
        v[0] = __uint_as_float(static_cast<uint32_t>(u) << 16);
    }
    __device__ __forceinline__ void set(const float (&v)[1]) {
        u = static_cast<uint16_t>(pack_bf16x2(v[0], 0.f));
    }
};
template <>
struct Piece<float, 1> {
    float f;
    __device__ __forceinline__ void load(const float *p) { f = __ldcg(p); }
    __device__ __forceinline__ void store(float *p) const { *p = f; }
    __device__ __forceinline__ void zero() { f = 0.f; }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = f; }
    __device__ __forceinline__ void set(const float (&v)[1]) { f = v[0]; }
};

// Sums of kSums values over the kRow threads of a row (all of the block's
// threads take part, each row of its own).
template <int kRow, int kRows, int kSums>
struct RowSums {
    float part[2][kRows][kRow / 32][kSums];
};

template <int kRow, int kRows, int kSums>
__device__ __forceinline__ void row_sums(RowSums<kRow, kRows, kSums> &sm, int turn, int t, int sub,
                                         float (&v)[kSums]) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
        for (int i = 0; i < kSums; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
    if (kRow == 32) return;
    // two buffers in turn: a warp can be one sum ahead, never two
    if (t % 32 == 0)
#pragma unroll
        for (int i = 0; i < kSums; ++i) sm.part[turn][sub][t / 32][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSums; ++i) v[i] = 0.f;
#pragma unroll
    for (int w = 0; w < kRow / 32; ++w)
#pragma unroll
        for (int i = 0; i < kSums; ++i) v[i] += sm.part[turn][sub][w][i];
}

template <int kRow>
__host__ __device__ constexpr int row_threads() {
    return kRow < 256 ? 256 : kRow;
}

// kRow threads a row, kChunks pieces a thread (piece c of thread t holds values
// [kVec (t + c kRow), + kVec)).
template <typename T, int kVec, int kRow, int kChunks>
__global__ void __launch_bounds__(row_threads<kRow>())
    layernorm_kernel(const LayerNormArgs a) {
    constexpr int kRows = row_threads<kRow>() / kRow;
    __shared__ RowSums<kRow, kRows, 1> sums;
    griddep_launch_dependents();
    griddep_wait();
    const int t = threadIdx.x % kRow, sub = threadIdx.x / kRow;
    const int pieces = a.H / kVec;
    const float inv_h = 1.f / static_cast<float>(a.H);
    const T *x = static_cast<const T *>(a.x), *residual = static_cast<const T *>(a.residual);
    const T *weight = static_cast<const T *>(a.weight), *bias = static_cast<const T *>(a.bias);
    // the gain and the bias are read once, the next row before this one's sums,
    // where registers are left for that
    constexpr bool kHold = kVec * kChunks <= 16 && kRow <= 512;
    constexpr bool kAhead = kHold;
    Piece<T, kVec> hw[kHold ? kChunks : 1], hb[kHold ? kChunks : 1];
    if constexpr (kHold) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            hw[c].zero();
            hb[c].zero();
            if (t + c * kRow < pieces) {
                hw[c].load(weight + kVec * (t + c * kRow));
                if (bias) hb[c].load(bias + kVec * (t + c * kRow));
            }
        }
    }
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kRows;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kRows;
    auto load = [&](int64_t n, Piece<T, kVec>(&px)[kChunks], Piece<T, kVec>(&pr)[kChunks]) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            px[c].zero();
            pr[c].zero();
            if (n < a.N && t + c * kRow < pieces) {
                const int64_t at = n * a.H + kVec * (t + c * kRow);
                px[c].load(x + at);
                if (residual) pr[c].load(residual + at);
            }
        }
    };
    Piece<T, kVec> nx[kChunks], nr[kChunks];
    if (kAhead) load(first + sub, nx, nr);
    for (int64_t base = first; base < a.N; base += stride) {
        const int64_t n = base + sub;
        const bool row = n < a.N;
        const int64_t at = n * a.H;
        if (!kAhead) load(n, nx, nr);
        Piece<T, kVec> r[kChunks];
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            r[c] = nx[c];
            if (residual) {
                float u[kVec], v[kVec];
                r[c].get(u);
                nr[c].get(v);
#pragma unroll
                for (int i = 0; i < kVec; ++i) u[i] += v[i];
                r[c].set(u);
            }
            if (a.residual_out && row && t + c * kRow < pieces)
                r[c].store(static_cast<T *>(a.residual_out) + at + kVec * (t + c * kRow));
        }
        if (kAhead) load(n + stride, nx, nr);
        float s[1] = {0.f};
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            float v[kVec];
            r[c].get(v);
#pragma unroll
            for (int i = 0; i < kVec; ++i) s[0] += v[i];
        }
        row_sums(sums, 0, t, sub, s);
        const float mean = s[0] * inv_h;
        s[0] = 0.f;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            if (t + c * kRow >= pieces) break;
            float v[kVec];
            r[c].get(v);
#pragma unroll
            for (int i = 0; i < kVec; ++i) s[0] = fmaf(v[i] - mean, v[i] - mean, s[0]);
        }
        row_sums(sums, 1, t, sub, s);
        if (!row) continue;
        const float rstd = 1.f / sqrtf(fmaf(s[0], inv_h, a.eps));
        if (t == 0) {
            if (a.mean) a.mean[n] = mean;
            if (a.rstd) a.rstd[n] = rstd;
        }
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            if (t + c * kRow >= pieces) break;
            const int h = kVec * (t + c * kRow);
            Piece<T, kVec> w, b;
            if constexpr (kHold) {
                w = hw[c];
                b = hb[c];
            } else {
                w.load(weight + h);
                b.zero();
                if (bias) b.load(bias + h);
            }
            float v[kVec], g[kVec], z[kVec];
            r[c].get(v);
            w.get(g);
            b.get(z);
#pragma unroll
            for (int i = 0; i < kVec; ++i) v[i] = fmaf((v[i] - mean) * rstd, g[i], z[i]);
            r[c].set(v);
            r[c].store(static_cast<T *>(a.out) + at + h);
        }
    }
}

// Rows too long for registers: the sum, the deviations' squares and the result
// each read them again, from L2; the blocks that fit instead hide each other's
// waits (300 x 65536 in fp32 81 us, 214 with registers that spill; 300 x 65535 in
// bf16 156 and 293).
constexpr int kLongThreads = 512;
constexpr int long_blocks(int vec) { return vec == 1 ? 4 : 2; }  // an SM

template <typename T, int kVec>
__global__ void __launch_bounds__(kLongThreads, long_blocks(kVec))
    layernorm_long_kernel(const LayerNormArgs a) {
    constexpr int kAt = 4;  // pieces on their way
    __shared__ RowSums<kLongThreads, 1, 1> sums;
    griddep_launch_dependents();
    griddep_wait();
    const int t = threadIdx.x, pieces = a.H / kVec;
    const float inv_h = 1.f / static_cast<float>(a.H);
    const T *weight = static_cast<const T *>(a.weight), *bias = static_cast<const T *>(a.bias);
    for (int64_t n = blockIdx.x; n < a.N; n += gridDim.x) {
        const int64_t at = n * a.H;
        const T *x = static_cast<const T *>(a.x) + at;
        const T *residual = a.residual ? static_cast<const T *>(a.residual) + at : nullptr;
        T *kept = a.residual_out ? static_cast<T *>(a.residual_out) + at : nullptr;
        Piece<T, kVec> r[kAt], other[kAt];
        // pieces first, first + kLongThreads, ... of r = x + residual
        auto load = [&](int first) {
#pragma unroll
            for (int j = 0; j < kAt; ++j) {
                const int i = kVec * (first + j * kLongThreads);
                r[j].zero();
                other[j].zero();
                if (i < a.H) {
                    r[j].load(x + i);
                    if (residual) other[j].load(residual + i);
                }
            }
            if (!residual) return;
#pragma unroll
            for (int j = 0; j < kAt; ++j) {
                float u[kVec], v[kVec];
                r[j].get(u);
                other[j].get(v);
#pragma unroll
                for (int i = 0; i < kVec; ++i) u[i] += v[i];
                r[j].set(u);
            }
        };
        float s[1] = {0.f};
        for (int first = t; first < pieces; first += kAt * kLongThreads) {
            load(first);
            float part = 0.f;  // sums of sums: fewer roundings in a row
#pragma unroll
            for (int j = 0; j < kAt; ++j) {
                float v[kVec];
                r[j].get(v);
#pragma unroll
                for (int i = 0; i < kVec; ++i) part += v[i];
                if (kept && first + j * kLongThreads < pieces)
                    r[j].store(kept + kVec * (first + j * kLongThreads));
            }
            s[0] += part;
        }
        if (kept) {  // x and residual may have been written over
            x = kept;
            residual = nullptr;
        }
        row_sums(sums, 0, t, 0, s);
        const float mean = s[0] * inv_h;
        s[0] = 0.f;
        for (int first = t; first < pieces; first += kAt * kLongThreads) {
            load(first);
            float part = 0.f;
#pragma unroll
            for (int j = 0; j < kAt; ++j) {
                if (first + j * kLongThreads >= pieces) break;
                float v[kVec];
                r[j].get(v);
#pragma unroll
                for (int i = 0; i < kVec; ++i) part = fmaf(v[i] - mean, v[i] - mean, part);
            }
            s[0] += part;
        }
        row_sums(sums, 1, t, 0, s);
        const float rstd = 1.f / sqrtf(fmaf(s[0], inv_h, a.eps));
        if (t == 0) {
            if (a.mean) a.mean[n] = mean;
            if (a.rstd) a.rstd[n] = rstd;
        }
        for (int first = t; first < pieces; first += kAt * kLongThreads) {
            load(first);
#pragma unroll
            for (int j = 0; j < kAt; ++j) {
                const int h = kVec * (first + j * kLongThreads);
                if (h >= a.H) break;
                Piece<T, kVec> w, b;
                w.load(weight + h);
                b.zero();
                if (bias) b.load(bias + h);
                float v[kVec], g[kVec], z[kVec];
                r[j].get(v);
                w.get(g);
                b.get(z);
#pragma unroll
                for (int i = 0; i < kVec; ++i) v[i] = fmaf((v[i] - mean) * rstd, g[i], z[i]);
                r[j].set(v);
                r[j].store(static_cast<T *>(a.out) + at + h);
            }
        }
    }
}

// kSumColumns: the block keeps its columns' sums (dweight, dbias) and stores
// them as part blockIdx.x, unless a.part is NULL (dx alone is wanted).
template <typename T, int kVec, int kRow, int kChunks, bool kSumColumns>
__global__ void __launch_bounds__(row_threads<kRow>(),
                                  kSumColumns && kRow <= 256 ? 2 : 1)
    layernorm_grad_kernel(const LayerNormGradArgs a) {
    constexpr int kThreads = row_threads<kRow>();
    constexpr int kRows = kThreads / kRow;
    constexpr int kCols = kVec * kChunks;  // a thread's
    __shared__ RowSums<kRow, kRows, 2> sums;
    griddep_launch_dependents();
    griddep_wait();
    const int t = threadIdx.x % kRow, sub = threadIdx.x / kRow;
    const int pieces = a.H / kVec;
    const float inv_h = 1.f / static_cast<float>(a.H);
    const T *dout = static_cast<const T *>(a.dout), *x = static_cast<const T *>(a.x);
    const T *dres = static_cast<const T *>(a.dresidual);
    Piece<T, kVec> w[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        w[c].zero();
        if (t + c * kRow < pieces)
            w[c].load(static_cast<const T *>(a.weight) + kVec * (t + c * kRow));
    }
    float dw[kSumColumns ? kCols : 1] = {}, db[kSumColumns ? kCols : 1] = {};
    // a row's operands: the next one's are asked for before this one's sums,
    // where registers are left for them
    constexpr bool kAhead = kSumColumns && (kCols <= 8 || (kVec == 8 && kRow > 32));
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kRows;
    Piece<T, kVec> r[kChunks], d[kChunks], e[kChunks];
    float mean = 0.f, rstd = 0.f;
    auto load = [&](int64_t n, Piece<T, kVec>(&pr)[kChunks], Piece<T, kVec>(&pd)[kChunks],
                    Piece<T, kVec>(&pe)[kChunks], float &m, float &q) {
        const bool row = n < a.N;
        const int64_t at = n * a.H;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            pr[c].zero();
            pd[c].zero();
            pe[c].zero();
            if (row && t + c * kRow < pieces) {
                pr[c].load(x + at + kVec * (t + c * kRow));
                pd[c].load(dout + at + kVec * (t + c * kRow));
                if (dres) pe[c].load(dres + at + kVec * (t + c * kRow));
            }
        }
        m = row ? __ldcg(a.mean + n) : 0.f;
        q = row ? __ldcg(a.rstd + n) : 0.f;
    };
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kRows;
    if (kAhead) load(first + sub, r, d, e, mean, rstd);
    int turn = 0;
    for (int64_t base = first; base < a.N; base += stride, turn ^= 1) {
        const int64_t n = base + sub;
        const bool row = n < a.N;
        const int64_t at = n * a.H;
        if (!kAhead) load(n, r, d, e, mean, rstd);
        Piece<T, kVec> nr[kAhead ? kChunks : 1], nd[kAhead ? kChunks : 1], ne[kAhead ? kChunks : 1];
        float nmean = 0.f, nrstd = 0.f;
        if constexpr (kAhead) load(n + stride, nr, nd, ne, nmean, nrstd);
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            if (!row || t + c * kRow >= pieces) break;
            float v[kVec], g[kVec], y[kVec];
            r[c].get(v);
            d[c].get(y);
            w[c].get(g);
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const float m = (v[i] - mean) * rstd;
                if (kSumColumns) {
                    dw[c * kVec + i] = fmaf(y[i], m, dw[c * kVec + i]);
                    db[c * kVec + i] += y[i];
                }
                const float u = y[i] * g[i];
                s[0] += u;
                s[1] = fmaf(u, m, s[1]);
            }
        }
        if (a.dx) {
            row_sums(sums, turn, t, sub, s);
            const float m1 = s[0] * inv_h, m2 = s[1] * inv_h;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                if (!row || t + c * kRow >= pieces) break;
                float v[kVec], g[kVec], y[kVec], z[kVec];
                r[c].get(v);
                d[c].get(y);
                w[c].get(g);
                e[c].get(z);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const float m = (v[i] - mean) * rstd;
                    v[i] = fmaf(rstd, fmaf(-m, m2, fmaf(y[i], g[i], -m1)), z[i]);
                }
                r[c].set(v);
                r[c].store(static_cast<T *>(a.dx) + at + kVec * (t + c * kRow));
            }
        }
        if constexpr (kAhead) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                r[c] = nr[c];
                d[c] = nd[c];
                e[c] = ne[c];
            }
            mean = nmean;
            rstd = nrstd;
        }
    }
    if (!kSumColumns || !a.part) return;
    // the rows of the block side by side, then the block's part
    float *out = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.H;
    if constexpr (kRows > 1) {
        __shared__ float side[kRows / 2][kRow * kCols];
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            float *v = which ? db : dw;
            for (int half = kRows / 2; half > 0; half /= 2) {
                __syncthreads();
                if (sub >= half && sub < 2 * half)
#pragma unroll
                    for (int i = 0; i < kCols; ++i) side[sub - half][i * kRow + t] = v[i];
                __syncthreads();
                if (sub < half)
#pragma unroll
                    for (int i = 0; i < kCols; ++i) v[i] += side[sub][i * kRow + t];
            }
        }
        if (sub > 0) return;
    }
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        if (t + c * kRow >= pieces) break;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int h = kVec * (t + c * kRow) + i;
            __stcg(out + h, dw[c * kVec + i]);
            __stcg(out + a.H + h, db[c * kVec + i]);
        }
    }
}

// dx of rows too long for registers, which are read again, from L2, for their
// second pass; the blocks that fit instead hide each other's waits.  By single
// values 4000 x 4099 in bf16 took 74 us, held in registers 117 (2000 x 16383: 131
// and 200, 300 x 65535: 128 and 350); in vectors 1024 x 16384 in fp32 59 and 70,
// 1000 x 32768 in bf16 63 and 84, but 4096 x 8192 66 and 50, which stay there.
template <typename T, int kVec>
__global__ void __launch_bounds__(kLongThreads, long_blocks(kVec))
    layernorm_grad_long_kernel(const LayerNormGradArgs a) {
    constexpr int kAt = kVec == 1 ? 4 : 2;  // pieces on their way
    __shared__ RowSums<kLongThreads, 1, 2> sums;
    griddep_launch_dependents();
    griddep_wait();
    const int t = threadIdx.x, pieces = a.H / kVec;
    const float inv_h = 1.f / static_cast<float>(a.H);
    int turn = 0;
    for (int64_t n = blockIdx.x; n < a.N; n += gridDim.x, turn ^= 1) {
        const int64_t at = n * a.H;
        const T *x = static_cast<const T *>(a.x) + at, *dout = static_cast<const T *>(a.dout) + at;
        const T *weight = static_cast<const T *>(a.weight);
        const T *dres = a.dresidual ? static_cast<const T *>(a.dresidual) + at : nullptr;
        T *dx = static_cast<T *>(a.dx) + at;
        const float mean = __ldcg(a.mean + n), rstd = __ldcg(a.rstd + n);
        Piece<T, kVec> r[kAt], d[kAt], w[kAt], e[kAt];
        auto load = [&](int first, bool all) {
#pragma unroll
            for (int j = 0; j < kAt; ++j) {
                const int i = kVec * (first + j * kLongThreads);
                e[j].zero();
                if (i < a.H) {
                    r[j].load(x + i);
                    d[j].load(dout + i);
                    w[j].load(weight + i);
                    if (all && dres) e[j].load(dres + i);
                }
            }
        };
        float s[2] = {0.f, 0.f};
        for (int first = t; first < pieces; first += kAt * kLongThreads) {
            load(first, false);
            float part[2] = {0.f, 0.f};  // sums of sums: fewer roundings in a row
#pragma unroll
            for (int j = 0; j < kAt; ++j) {
                if (first + j * kLongThreads >= pieces) break;
                float v[kVec], g[kVec], y[kVec];
                r[j].get(v);
                d[j].get(y);
                w[j].get(g);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const float u = y[i] * g[i];
                    part[0] += u;
                    part[1] = fmaf(u, (v[i] - mean) * rstd, part[1]);
                }
            }
            s[0] += part[0];
            s[1] += part[1];
        }
        row_sums(sums, turn, t, 0, s);
        const float m1 = s[0] * inv_h, m2 = s[1] * inv_h;
        for (int first = t; first < pieces; first += kAt * kLongThreads) {
            load(first, true);
#pragma unroll
            for (int j = 0; j < kAt; ++j) {
                if (first + j * kLongThreads >= pieces) break;
                float v[kVec], g[kVec], y[kVec], z[kVec];
                r[j].get(v);
                d[j].get(y);
                w[j].get(g);
                e[j].get(z);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const float m = (v[i] - mean) * rstd;
                    v[i] = fmaf(rstd, fmaf(-m, m2, fmaf(y[i], g[i], -m1)), z[i]);
                }
                r[j].set(v);
                r[j].store(dx + kVec * (first + j * kLongThreads));
            }
        }
    }
}

// Rows too long for their sums in registers: a thread kVec columns, a block a run
// of rows (part blockIdx.y).
constexpr int kColumnThreads = 256;
constexpr int kColumnRows = 4;  // at a time

// A thread adds up this many rows' dout n and dout in fp32 at most before the sum
// joins others, however many rows there are (4096 times 1 + 2^-13 - 2^-23 in one
// sum come out 6e-5 of it too small, in runs of 128 exact to 2^-24).  It costs up to
// 5% (backward, bf16: 39000 x 4096 269 us and 278, 400000 x 64 124 and 128, 3000 x
// 5000 49.0 and 51.3, 4096 x 8192 85.7 and 86.5).
constexpr int kRunRows = 128;
constexpr int64_t kMostRuns = 1 << 20;  // blocks are counted in 32 bits

template <typename T, int kVec>
__global__ void __launch_bounds__(kColumnThreads)
    layernorm_columns_kernel(const LayerNormGradArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const int h = (blockIdx.x * kColumnThreads + threadIdx.x) * kVec;
    if (h >= a.H) return;
    const int64_t first = a.N * blockIdx.y / gridDim.y, end = a.N * (blockIdx.y + 1) / gridDim.y;
    const T *x = static_cast<const T *>(a.x) + h, *dout = static_cast<const T *>(a.dout) + h;
    float dw[kVec] = {}, db[kVec] = {}, sum_w[kVec] = {}, sum_b[kVec] = {};
    for (int64_t n = first; n < end; n += kColumnRows) {
        Piece<T, kVec> r[kColumnRows], d[kColumnRows];
        float mean[kColumnRows], rstd[kColumnRows];
#pragma unroll
        for (int j = 0; j < kColumnRows; ++j) {
            r[j].zero();
            d[j].zero();
            mean[j] = rstd[j] = 0.f;
            if (n + j < end) {
                r[j].load(x + (n + j) * a.H);
                d[j].load(dout + (n + j) * a.H);
                mean[j] = __ldcg(a.mean + n + j);
                rstd[j] = __ldcg(a.rstd + n + j);
            }
        }
#pragma unroll
        for (int j = 0; j < kColumnRows; ++j) {
            if (n + j >= end) break;
            float v[kVec], y[kVec];
            r[j].get(v);
            d[j].get(y);
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                dw[i] = fmaf(y[i], (v[i] - mean[j]) * rstd[j], dw[i]);
                db[i] += y[i];
            }
        }
        if ((n - first) % kRunRows == kRunRows - kColumnRows) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                sum_w[i] += dw[i];
                sum_b[i] += db[i];
                dw[i] = db[i] = 0.f;
            }
        }
    }
    float *out = a.part + static_cast<int64_t>(blockIdx.y) * 2 * a.H + h;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        __stcg(out + i, sum_w[i] + dw[i]);
        __stcg(out + a.H + i, sum_b[i] + db[i]);
    }
}

// The parts' sum, in order: 32 columns a block, its warps taking the parts in
// turn, eight at a time.  Eight are added in fp32, those sums and the warps' in
// 64 bits, of which an SM adds (and widens to) few: with every part widened 304
// parts of 2 x 1111 columns took 9.5 us, so 6.3.
constexpr int kFinishThreads = 1024;
constexpr int kFinishAhead = 8;

__global__ void __launch_bounds__(kFinishThreads)
    layernorm_finish_kernel(const float *part, int blocks, int H, float *dweight, float *dbias) {
    constexpr int kWarps = kFinishThreads / 32;
    __shared__ double sums[kWarps][32];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + lane;  // of the 2 H sums
    const bool live = i < 2 * static_cast<int64_t>(H);
    double s = 0.0;
    for (int b = warp; live && b < blocks; b += kFinishAhead * kWarps) {
        float v[kFinishAhead];
#pragma unroll
        for (int j = 0; j < kFinishAhead; ++j)
            v[j] = b + j * kWarps < blocks
                       ? __ldcg(part + static_cast<int64_t>(b + j * kWarps) * 2 * H + i)
                       : 0.f;
        s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || !live) return;
    double f[4] = {};
#pragma unroll
    for (int w = 0; w < kWarps; w += 4)
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] += sums[w + j][lane];
    s = (f[0] + f[1]) + (f[2] + f[3]);
    float *out = i < H ? dweight : dbias;
    if (out) out[i < H ? i : i - H] = static_cast<float>(s);
}

// ---------------------------------------------------------------- launchers

// Blocks of a kernel that fit on an SM at once.
template <typename Kernel>
int resident(Kernel kern, int threads) {
    int n = 0;
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, 0);
    return n > 0 ? n : 1;
}

template <typename T, int kVec, int kRow, int kChunks>
cudaError_t launch_rows(const LayerNormArgs &a, int num_sms, cudaStream_t s) {
    constexpr int kRows = row_threads<kRow>() / kRow;
    auto kern = layernorm_kernel<T, kVec, kRow, kChunks>;
    static const int fit = resident(kern, row_threads<kRow>());
    int64_t blocks = (a.N + kRows - 1) / kRows;
    const int64_t limit = static_cast<int64_t>(fit) * num_sms * 2;
    if (blocks > limit) blocks = limit;
    return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(row_threads<kRow>()), 0, s, 1,
                      a);
}

template <typename T, int kVec>
cudaError_t launch_long(const LayerNormArgs &a, int num_sms, cudaStream_t s) {
    const int64_t fit = static_cast<int64_t>(num_sms) * long_blocks(kVec);
    return launch_pdl(layernorm_long_kernel<T, kVec>,
                      dim3(static_cast<unsigned>(a.N < fit ? a.N : fit)), dim3(kLongThreads), 0, s,
                      1, a);
}

template <typename T, int kVec>
cudaError_t launch_forward(const LayerNormArgs &a, int num_sms, cudaStream_t s) {
    const int pieces = a.H / kVec;
    if constexpr (kVec == 1) {
        // Single values: eight (sixteen) on their way a thread and row, twice with
        // the row ahead.  With two and four 100000 x 151 in bf16 took 67 us instead
        // of 39, 4000 x 4099 118 instead of 51, 1021 x 1111 in fp32 7 and 4.
        if (pieces <= 128) return launch_rows<T, 1, 32, 4>(a, num_sms, s);
        if (pieces <= 256) return launch_rows<T, 1, 32, 8>(a, num_sms, s);
        if (pieces <= 512) return launch_rows<T, 1, 64, 8>(a, num_sms, s);
        if (pieces <= 1024) return launch_rows<T, 1, 128, 8>(a, num_sms, s);
        if (pieces <= 2048) return launch_rows<T, 1, 256, 8>(a, num_sms, s);
        if (pieces <= 4096) return launch_rows<T, 1, 512, 8>(a, num_sms, s);
        if (pieces <= 8192) return launch_rows<T, 1, 512, 16>(a, num_sms, s);
        // 2000 x 16383 in fp32: 126 us from registers and 153 read again, in bf16
        // 208 and 141
        if constexpr (sizeof(T) == 4) {
            if (pieces <= 16384) return launch_rows<T, 1, 1024, 16>(a, num_sms, s);
        }
        return launch_long<T, 1>(a, num_sms, s);
    }
    if (pieces <= 32) return launch_rows<T, kVec, 32, 1>(a, num_sms, s);
    if (pieces <= 64) return launch_rows<T, kVec, 32, 2>(a, num_sms, s);
    if (pieces <= 128) return launch_rows<T, kVec, 64, 2>(a, num_sms, s);
    if (pieces <= 256) return launch_rows<T, kVec, 128, 2>(a, num_sms, s);
    if (pieces <= 512) return launch_rows<T, kVec, 256, 2>(a, num_sms, s);
    if (pieces <= 1024) return launch_rows<T, kVec, 256, 4>(a, num_sms, s);
    if (pieces <= 2048) return launch_rows<T, kVec, 512, 4>(a, num_sms, s);
    if (pieces <= 4096) return launch_rows<T, kVec, 1024, 4>(a, num_sms, s);
    // the longest rows of bf16 values are 8192 pieces
    if constexpr (kVec == 4) {
        if (pieces > 8192) return launch_long<T, kVec>(a, num_sms, s);
    }
    return launch_rows<T, kVec, 1024, 8>(a, num_sms, s);
}

// As many blocks as fit at once: two of 256 threads an SM with the sums in
// registers (as many times that as their runs of kRunRows rows need), else four
// times that, one after the other.
template <typename T, int kVec, int kRow, int kChunks, bool kSum>
cudaError_t launch_grad_rows(const LayerNormGradArgs &a, int num_sms, int *blocks,
                             cudaStream_t s) {
    constexpr int kThreads = row_threads<kRow>(), kRows = kThreads / kRow;
    const int64_t most = (a.N + kRows - 1) / kRows;
    int64_t fit = static_cast<int64_t>(num_sms) * (kSum ? (kThreads == 256 ? 2 : 1) : 4);
    if (kSum && a.part) {
        const int64_t runs = (most + fit * kRunRows - 1) / (fit * kRunRows);
        fit *= runs < kMostRuns ? runs : kMostRuns;
    }
    *blocks = static_cast<int>(most < fit ? most : fit);
    return launch_pdl(layernorm_grad_kernel<T, kVec, kRow, kChunks, kSum>,
                      dim3(static_cast<unsigned>(*blocks)), dim3(kThreads), 0, s, 1, a);
}

// 16 columns a thread in vectors of eight bf16 values (8 in rows of up to 256
// values), else 8: more leave no registers for the row ahead.
template <typename T, int kVec>
cudaError_t launch_backward(const LayerNormGradArgs &a, int num_sms, int *blocks, cudaStream_t s) {
    constexpr int kC = kVec == 8 ? 2 : 8 / kVec;  // pieces a thread
    const int threads = (a.H / kVec + kC - 1) / kC;
    if (kVec == 8 && a.H <= 256)
        return launch_grad_rows<T, kVec, 32, 8 / kVec, true>(a, num_sms, blocks, s);
    if (threads <= 32) return launch_grad_rows<T, kVec, 32, kC, true>(a, num_sms, blocks, s);
    if (threads <= 64) return launch_grad_rows<T, kVec, 64, kC, true>(a, num_sms, blocks, s);
    if (threads <= 128) return launch_grad_rows<T, kVec, 128, kC, true>(a, num_sms, blocks, s);
    if (threads <= 256) return launch_grad_rows<T, kVec, 256, kC, true>(a, num_sms, blocks, s);
    if constexpr (kVec < 8) return launch_grad_rows<T, kVec, 512, kC, true>(a, num_sms, blocks, s);
    return cudaErrorInvalidValue;
}

template <typename T, int kVec>
cudaError_t launch_columns(const LayerNormGradArgs &a, int blocks, cudaStream_t s) {
    constexpr int kColumns = kColumnThreads * kVec;
    const dim3 grid(static_cast<unsigned>((a.H + kColumns - 1) / kColumns),
                    static_cast<unsigned>(blocks));
    return launch_pdl(layernorm_columns_kernel<T, kVec>, grid, dim3(kColumnThreads), 0, s, 1, a);
}

// dx alone, of rows over kSumColumnsH.
template <typename T, int kVec>
cudaError_t launch_backward_wide(const LayerNormGradArgs &a, int num_sms, cudaStream_t s) {
    const int pieces = a.H / kVec;
    int blocks;
    if constexpr (kVec == 8) {
        if (pieces <= 1024) return launch_grad_rows<T, kVec, 256, 4, false>(a, num_sms, &blocks, s);
    }
    if constexpr (kVec > 1) {
        if (pieces <= 2048) return launch_grad_rows<T, kVec, 512, 4, false>(a, num_sms, &blocks, s);
    }
    const int64_t fit = static_cast<int64_t>(num_sms) * long_blocks(kVec);
    return launch_pdl(layernorm_grad_long_kernel<T, kVec>,
                      dim3(static_cast<unsigned>(a.N < fit ? a.N : fit)), dim3(kLongThreads), 0, s,
                      1, a);
}

// The longest rows whose sums stay in registers.  Beyond, a block would be alone
// on its SM with one row at a time: 4096 x 8192 took 98 us with 512 threads and
// 111 with 1024, with a second pass for the sums 100 (3000 x 5000: 73 and 62).
constexpr int kSumColumnsH = 4096;

bool vectors(int H, int bf16, std::initializer_list<const void *> arrays) {
    if (H % (bf16 ? 8 : 4)) return false;
    for (const void *p : arrays)
        if (reinterpret_cast<uintptr_t>(p) % 16) return false;
    return true;
}

}  // namespace

int64_t layernorm_grad_blocks(int64_t N, int H, int num_sms) {
    // of whichever kernel the arrays' types and alignment choose (a block of
    // layernorm_columns_kernel covers 2048 columns at most; fit * runs blocks of
    // launch_grad_rows are N / kRunRows + fit at most)
    const int64_t rows =
        H <= kSumColumnsH ? N / kRunRows + 2 * static_cast<int64_t>(num_sms) : 0;
    const int64_t columns = 4 * static_cast<int64_t>(num_sms) / ((H + 2047) / 2048);
    const int64_t most = rows > columns ? rows : columns;
    return N < most ? N : most > 1 ? most : 1;
}

cudaError_t launch_layernorm(const LayerNormArgs &a, int bf16, int num_sms, cudaStream_t s) {
    const bool vec = vectors(a.H, bf16, {a.x, a.residual, a.weight, a.bias, a.residual_out, a.out});
    if (bf16)
        return vec ? launch_forward<__nv_bfloat16, 8>(a, num_sms, s)
                   : launch_forward<__nv_bfloat16, 1>(a, num_sms, s);
    return vec ? launch_forward<float, 4>(a, num_sms, s) : launch_forward<float, 1>(a, num_sms, s);
}

cudaError_t launch_layernorm_grad(const LayerNormGradArgs &args, int bf16, int num_sms,
                                  int *launches, cudaStream_t s) {
    LayerNormGradArgs a = args;
    const bool vec = vectors(a.H, bf16, {a.dout, a.x, a.weight, a.dresidual, a.dx});
    const bool sums = a.dweight || a.dbias;
    // without sums there need be no workspace, or one of any size: no part is stored
    if (!sums) a.part = nullptr;
    cudaError_t err = cudaSuccess;
    int blocks = 0;
    if (a.H <= kSumColumnsH) {
        if (bf16)
            err = vec ? launch_backward<__nv_bfloat16, 8>(a, num_sms, &blocks, s)
                      : launch_backward<__nv_bfloat16, 1>(a, num_sms, &blocks, s);
        else
            err = vec ? launch_backward<float, 4>(a, num_sms, &blocks, s)
                      : launch_backward<float, 1>(a, num_sms, &blocks, s);
        *launches += 1;
    } else {
        if (sums) {  // first: dx may be one of the inputs
            // runs of 16 rows and more
            const int columns = kColumnThreads * (!vec ? 1 : bf16 ? 8 : 4);
            const int64_t fit = 4 * static_cast<int64_t>(num_sms) / ((a.H + columns - 1) / columns);
            const int64_t most = (a.N + 15) / 16 < fit ? (a.N + 15) / 16 : fit;
            blocks = static_cast<int>(most > 1 ? most : 1);
            if (bf16)
                err = vec ? launch_columns<__nv_bfloat16, 8>(a, blocks, s)
                          : launch_columns<__nv_bfloat16, 1>(a, blocks, s);
            else
                err = vec ? launch_columns<float, 4>(a, blocks, s)
                          : launch_columns<float, 1>(a, blocks, s);
            *launches += 1;
        }
        if (err == cudaSuccess && a.dx) {
            if (bf16)
                err = vec ? launch_backward_wide<__nv_bfloat16, 8>(a, num_sms, s)
                          : launch_backward_wide<__nv_bfloat16, 1>(a, num_sms, s);
            else
                err = vec ? launch_backward_wide<float, 4>(a, num_sms, s)
                          : launch_backward_wide<float, 1>(a, num_sms, s);
            *launches += 1;
        }
    }
    if (err != cudaSuccess || !sums) return err;
    *launches += 1;
    return launch_pdl(layernorm_finish_kernel, dim3((2 * a.H + 31) / 32), dim3(kFinishThreads), 0,
                      s, 1, static_cast<const float *>(a.part), blocks, a.H, a.dweight, a.dbias);
}

}  // namespace moe
