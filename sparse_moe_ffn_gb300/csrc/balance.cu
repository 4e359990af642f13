// balance.cu -- the router's load statistics and balance losses, and their
// gradient with respect to the router logits.
//
//   p_n    = softmax(logits_n)        T = tokens that the mask leaves in
//   c_e    = slots (n, j) of those tokens with id e      f_e = c_e / (k T)
//   P_e    = sum_n p_ne / T           lse_n = log sum_e exp(logit_ne)
//   losses = { E sum_e f_e P_e,  sum_n lse_n^2 / T }
//   dlogit_ne = p_ne / T (g_0 E (d_e - sum_j d_j p_nj) + 2 g_1 lse_n),
//               d_e = f_e - 1/E
//
// f is a count and has no gradient.  sum_j p_nj = 1, so taking 1/E off f
// changes no gradient; it removes the cancellation in f_e - sum_j f_j p_nj,
// whose two terms agree in all but the last few percent when the load is
// nearly even.  d_e is formed in whole numbers from the counts.
// A token whose logits are all -inf has p = 0 and lse = 0 and still counts in
// T; a masked token takes no part, whatever it holds, and gets gradient 0.
//
// A row is held by kLanes lanes, 8 values each (kLanes is the power of two
// that covers E), four rows at a time; sums over tokens run in registers, then
// per block, per cluster of blocks (distributed shared memory) and, when
// there is more than one cluster, in a second kernel: each in a fixed order,
// with no atomics on floats, so the same inputs give the same bits.  All sums
// are fp32; the joins of P and the long sums of a lane (kFoldPasses) keep what
// each addition rounds off.
//
// What bounds it: 131072 x 128 in fp32, forward 20.0 us (71 MB, 3570 GB/s), of
// which 8 us are the two kernels' starts and joins: eight times the rows take
// 109 us, 5600 GB/s for those added (rows are read one pass ahead); gradient 25.5
// us (134 MB, 5270 GB/s; a plain copy of the same bytes 21.5); 64 x 128 forward
// 4.6 us, latency.
#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

#include "block_ops.cuh"
#include "cluster.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kVals = 8;
constexpr int kThreads = 256;
constexpr int kAloneThreads = 512;  // of a block when one cluster does it all
constexpr float kNegInf = -__builtin_huge_valf();

// Value v of lane t of a row is expert 4 (t + kLanes (v / 4)) + v % 4 when
// rows are read four values at a time, else t + kLanes v.
template <int kLanes, bool kVec>
__device__ __forceinline__ int expert_of(int t, int v) {
    return kVec ? 4 * (t + kLanes * (v / 4)) + v % 4 : t + kLanes * v;
}

// The rows that a warp holds at once: kUnroll per group of kLanes lanes, so
// that many loads are in flight.  Row u of lane group `sub` is
// base + u (32 / kLanes) + sub.
constexpr int kUnroll = 4;

template <int kLanes>
constexpr int kRowsPerWarp = kUnroll * (32 / kLanes);

// Element `i` of the logits (a row's start), as the type says.
template <bool kBf16, typename P>
__device__ __forceinline__ P *at_element(P *base, int64_t i) {
    return reinterpret_cast<P *>(reinterpret_cast<uintptr_t>(base) + i * (kBf16 ? 2 : 4));
}

// This lane's values of a row as they come from memory: loading them uses none
// of them, so the loads of all rows, and of the next ones, go out together.
template <bool kBf16, bool kVec>
struct RawRow;
template <>
struct RawRow<false, true> {
    float4 c[kVals / 4];
};
template <>
struct RawRow<true, true> {
    uint2 c[kVals / 4];
};
template <>
struct RawRow<false, false> {
    float c[kVals];
};
template <>
struct RawRow<true, false> {
    uint16_t c[kVals];
};

template <bool kBf16, int kLanes, bool kVec>
__device__ __forceinline__ void load_row(const void *row, int E, int t,
                                         RawRow<kBf16, kVec> &raw) {
    constexpr int kStep = kVec ? 4 : 1;
    using Piece = typename std::remove_reference<decltype(raw.c[0])>::type;
#pragma unroll
    for (int c = 0; c < kVals / kStep; ++c) {
        const int e = kStep * (t + kLanes * c);
        if (e < E)
            raw.c[c] = __ldcg(reinterpret_cast<const Piece *>(at_element<kBf16>(row, e)));
    }
}

template <bool kBf16, int kLanes, bool kVec>
__device__ __forceinline__ void unpack_row(const RawRow<kBf16, kVec> &raw, int E, int t,
                                           float (&x)[kVals]) {
    if constexpr (kVec) {
#pragma unroll
        for (int c = 0; c < kVals / 4; ++c) {
            float4 f;
            if constexpr (kBf16) {
                const float2 a = unpack_bf16x2(raw.c[c].x), b = unpack_bf16x2(raw.c[c].y);
                f = make_float4(a.x, a.y, b.x, b.y);
            } else {
                f = raw.c[c];
            }
            const bool live = 4 * (t + kLanes * c) < E;
            x[4 * c] = live ? f.x : kNegInf;
            x[4 * c + 1] = live ? f.y : kNegInf;
            x[4 * c + 2] = live ? f.z : kNegInf;
            x[4 * c + 3] = live ? f.w : kNegInf;
        }
    } else {
#pragma unroll
        for (int v = 0; v < kVals; ++v) {
            float f;
            if constexpr (kBf16) f = __uint_as_float(static_cast<uint32_t>(raw.c[v]) << 16);
            else f = raw.c[v];
            x[v] = t + kLanes * v < E ? f : kNegInf;
        }
    }
}

// The rows of a warp that start at row `base`; past the end the last row stands
// in (it gets no weight).  `left` of them exist.
template <bool kBf16, int kLanes, bool kVec>
__device__ __forceinline__ void load_rows(const BalanceArgs &a, int64_t base, int t, int sub,
                                          RawRow<kBf16, kVec> (&raw)[kUnroll]) {
    if (base >= a.N) return;
    const int left = a.N - base < kRowsPerWarp<kLanes>
                         ? static_cast<int>(a.N - base) : kRowsPerWarp<kLanes>;
    const void *rows = at_element<kBf16>(a.logits, base * a.E);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
        load_row<kBf16, kLanes, kVec>(
            at_element<kBf16>(rows, min(u * (32 / kLanes) + sub, left - 1) * a.E), a.E, t, raw[u]);
}

template <bool kBf16, int kLanes, bool kVec>
__device__ __forceinline__ void store_row(void *row, int E, int t, const float (&x)[kVals]) {
    if (kVec) {
#pragma unroll
        for (int c = 0; c < kVals / 4; ++c) {
            const int e = 4 * (t + kLanes * c);
            if (e >= E) continue;
            if (kBf16)
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(row) + e) =
                    make_uint2(pack_bf16x2(x[4 * c], x[4 * c + 1]),
                               pack_bf16x2(x[4 * c + 2], x[4 * c + 3]));
            else
                *reinterpret_cast<float4 *>(static_cast<float *>(row) + e) =
                    make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
        }
    } else {
#pragma unroll
        for (int v = 0; v < kVals; ++v) {
            const int e = t + kLanes * v;
            if (e >= E) continue;
            if (kBf16)
                static_cast<__nv_bfloat16 *>(row)[e] = __float2bfloat16_rn(x[v]);
            else
                static_cast<float *>(row)[e] = x[v];
        }
    }
}

template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// The same over the rows that a warp holds at once, side by side: each step's
// shuffles are independent of one another.
template <int kLanes>
__device__ __forceinline__ void rows_max(float (&v)[kUnroll]) {
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1)
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            v[u] = fmaxf(v[u], __shfl_xor_sync(0xffffffffu, v[u], d));
}

template <int kLanes>
__device__ __forceinline__ void rows_sum(float (&v)[kUnroll]) {
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1)
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) v[u] += __shfl_xor_sync(0xffffffffu, v[u], d);
}

// 2^x in one instruction (off by two steps at most, and below 2^-126 it is 0);
// softmax spends its time on this, and takes 1/x and log2 x in the same way (off
// by two steps; log2 near 1 by 2^-22).
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// a, b <- (a - top) m, (b - top) m: two values an instruction.
__device__ __forceinline__ void sub_mul_pair(float &a, float &b, float top, float m) {
    asm("{\n\t.reg .b64 x, t;\n\t"
        "mov.b64 x, {%0, %1};\n\t"
        "mov.b64 t, {%2, %2};\n\t"
        "add.rn.f32x2 x, x, t;\n\t"
        "mov.b64 t, {%3, %3};\n\t"
        "mul.rn.f32x2 x, x, t;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(-top), "f"(m));
}

// x[u] <- e^(x - top) of row u; f[u]: the factor that makes them
// probabilities, lse[u]: the row's log-sum-exp.  The largest logit is taken off
// before the product with log2(e): in one fma, with top log2(e) rounded beside
// it, rows of values beyond 1e9 (experts disabled with a large finite value)
// over- or underflow.  Two values an instruction make it no slower than that
// fma (131072 x 128 forward 20.0 us either way, 20.3 one value at a time).  A
// NaN logit reaches both results (fmaxf drops it, the sum does not).
template <int kLanes>
__device__ __forceinline__ void softmax_rows(float (&x)[kUnroll][kVals], float (&f)[kUnroll],
                                             float (&lse)[kUnroll]) {
    constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
    float top[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        top[u] = x[u][0];
#pragma unroll
        for (int v = 1; v < kVals; ++v) top[u] = fmaxf(top[u], x[u][v]);
    }
    rows_max<kLanes>(top);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (top[u] == kNegInf) top[u] = 0.f;
        f[u] = 0.f;
#pragma unroll
        for (int v = 0; v < kVals; v += 2) {
            sub_mul_pair(x[u][v], x[u][v + 1], top[u], kLog2e);
            x[u][v] = exp2_fast(x[u][v]);
            x[u][v + 1] = exp2_fast(x[u][v + 1]);
            f[u] += x[u][v];
            f[u] += x[u][v + 1];
        }
    }
    rows_sum<kLanes>(f);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        lse[u] = f[u] == 0.f ? 0.f : fmaf(kLn2, __log2f(f[u]), top[u]);
        f[u] = f[u] == 0.f ? 0.f : __fdividef(1.f, f[u]);
    }
}

// A sum that keeps what each fp32 addition rounds off (two-sum), so that the
// order and number of terms cost nothing; the GPU has few 64-bit units.
struct Sum {
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(float x) {
        const float s = __fadd_rn(hi, x);
        const float b = __fsub_rn(s, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
        hi = s;
    }
    __device__ __forceinline__ float value() const { return hi + lo; }
};

// hi + low <- x, or hi + low + x.
__device__ __forceinline__ void put(float &hi, float &low, float x, bool first) {
    Sum s;
    if (!first) {
        s.hi = hi;
        s.lo = low;
    }
    s.add(x);
    hi = s.hi;
    low = s.lo;
}

__device__ __forceinline__ float of_rank(const float *p, int rank) {
    return __uint_as_float(ld_cluster_u32(p, rank));
}

__device__ __forceinline__ int of_rank(const int *p, int rank) {
    return static_cast<int>(ld_cluster_u32(p, rank));
}

struct Totals {
    float z;
    int tokens, bad;
};

// The two losses and the token count, from sum_e p_e c_e and the totals.
__device__ __forceinline__ void write_losses(const BalanceArgs &a, float pc, const Totals &t) {
    const float inv = t.tokens > 0 ? 1.f / static_cast<float>(t.tokens) : 0.f;
    a.losses[0] = static_cast<float>(a.E) / static_cast<float>(a.k) * (pc * inv) * inv;
    a.losses[1] = t.z * inv;
    *a.tokens = t.tokens;
    if (a.status) *a.status = t.bad ? MOE_ERR_DEVICE_CHECK : MOE_OK;
}

// A lane's sums over its rows are plain fp32 for this many passes (4 rows each).
// Batches of more take the kernel that then joins them to sums with the rounding
// errors kept beside (kLong), so that a sum's error does not grow with the
// tokens: 4.2 million rows that are all alike came out 2.9e-5 too far without.
// In every kernel that would cost 0.5 us (131072 x 128: 20.5 against 20.0).
constexpr int kFoldPasses = 16;

template <bool kBf16, int kLanes, bool kVec, int kBlock, int kCluster, bool kLong>
__global__ void __launch_bounds__(kBlock, 512 / kBlock) balance_stats_kernel(const BalanceArgs a) {
    constexpr int kPerWarp = 32 / kLanes;
    constexpr int kWarps = kBlock / 32;
    constexpr int kRows = kRowsPerWarp<kLanes>;
    constexpr int kLowWarps = kLong ? kWarps : 1;
    // ps_low, zs_low: what the sums in ps and zs rounded off
    __shared__ float ps[kWarps][MOE_MAX_EXPERTS], ps_low[kLowWarps][MOE_MAX_EXPERTS];
    __shared__ float p_block[MOE_MAX_EXPERTS];
    __shared__ int cs[MOE_MAX_EXPERTS];
    __shared__ float zs[kWarps], zs_low[kLowWarps], pcs[kWarps], pc_rank;
    __shared__ int ts[kWarps];
    __shared__ int bad;
    __shared__ Totals total;
    griddep_launch_dependents();
    griddep_wait();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int t = lane % kLanes, sub = lane / kLanes;
    for (int e = threadIdx.x; e < MOE_MAX_EXPERTS; e += kBlock) cs[e] = 0;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();

    float p[kVals];
#pragma unroll
    for (int v = 0; v < kVals; ++v) p[v] = 0.f;
    float z = 0.f;
    int tokens = 0;
    bool over = false;  // an id >= E was seen
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps * kRows;
    int64_t base = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kRows;
    RawRow<kBf16, kVec> raw[kUnroll];
    int id_next[kUnroll];  // slot t of each row
    auto load_next = [&](int64_t at) {
        load_rows<kBf16, kLanes, kVec>(a, at, t, sub, raw);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t n = at + u * kPerWarp + sub;
            id_next[u] = n < a.N && t < a.k ? __ldcg(a.ids + n * a.k + t) : -1;
        }
    };
    load_next(base);
    bool first = true;
    do {
        const int64_t stop =
            kLong && a.N - base > kFoldPasses * step ? base + kFoldPasses * step : a.N;
        for (; base < stop; base += step) {
            const int left = a.N - base < kRows ? static_cast<int>(a.N - base) : kRows;
            const int32_t *ids = a.ids + base * a.k;
            float x[kUnroll][kVals];
            int id[kUnroll];
            bool in[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                in[u] = u * kPerWarp + sub < left;
                id[u] = id_next[u];
                unpack_row<kBf16, kLanes, kVec>(raw[u], a.E, t, x[u]);
            }
            load_next(base + step);
            if (a.mask) {
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    in[u] = in[u] && __ldcg(a.mask + base + u * kPerWarp + sub);
#pragma unroll
                    for (int v = 0; v < kVals; ++v) x[u][v] = in[u] ? x[u][v] : kNegInf;
                }
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                over |= in[u] && id[u] >= a.E;
                if (in[u] && id[u] >= 0 && id[u] < a.E) atomicAdd(&cs[id[u]], 1);
            }
            if (a.k > kLanes) {  // more slots than lanes
                for (int u = 0; u < kUnroll; ++u)
                    for (int j = t + kLanes; in[u] && j < a.k; j += kLanes) {
                        const int more = __ldcg(ids + (u * kPerWarp + sub) * a.k + j);
                        over |= more >= a.E;
                        if (more >= 0 && more < a.E) atomicAdd(&cs[more], 1);
                    }
            }
            float f[kUnroll], lse[kUnroll];
            softmax_rows<kLanes>(x, f, lse);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const float w = in[u] ? f[u] : 0.f;
#pragma unroll
                for (int v = 0; v < kVals; ++v) p[v] = fmaf(x[u][v], w, p[v]);
                z = in[u] ? fmaf(lse[u], lse[u], z) : z;  // each lane of the row alike
                tokens += in[u];
            }
        }
        // the warp's sums so far, its rows first, to shared memory: set the first
        // time, then added with what the addition rounds off kept beside them
#pragma unroll
        for (int d = kLanes; d < 32; d <<= 1) {
#pragma unroll
            for (int v = 0; v < kVals; ++v) p[v] += __shfl_xor_sync(0xffffffffu, p[v], d);
        }
        z = row_sum<32>(t == 0 ? z : 0.f);
        if (sub == 0) {
#pragma unroll
            for (int v = 0; v < kVals; ++v) {
                const int e = expert_of<kLanes, kVec>(t, v);
                if (e >= a.E) continue;
                if constexpr (kLong) put(ps[warp][e], ps_low[warp][e], p[v], first);
                else ps[warp][e] = p[v];
            }
        }
        if (lane == 0) {
            if constexpr (kLong) put(zs[warp], zs_low[warp], z, first);
            else zs[warp] = z;
        }
#pragma unroll
        for (int v = 0; v < kVals; ++v) p[v] = 0.f;
        z = 0.f;
        first = false;
    } while (kLong && base < a.N);
    if (over) bad = 1;
    tokens = t == 0 ? tokens : 0;
    tokens = __reduce_add_sync(0xffffffffu, tokens);
    if (lane == 0) ts[warp] = tokens;
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kBlock) {
        float s = 0.f, low = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            s += ps[w][e];
            if constexpr (kLong) low += ps_low[w][e];
        }
        p_block[e] = s + low;
    }
    if (threadIdx.x == 0) {
        Totals b = {0.f, 0, bad};
        float low = 0.f;
        for (int w = 0; w < kWarps; ++w) {
            b.z += zs[w];
            if constexpr (kLong) low += zs_low[w];
            b.tokens += ts[w];
        }
        b.z += low == low ? low : 0.f;  // (a sum past fp32 leaves inf - inf there)
        total = b;
    }
    cluster_barrier();

    // the blocks of the cluster, in order: each takes a run of the experts
    const int rank = static_cast<int>(cluster_ctarank());
    const int share = (a.E + kCluster - 1) / kCluster;
    const int e = rank * share + static_cast<int>(threadIdx.x);
    const bool mine = static_cast<int>(threadIdx.x) < share && e < a.E;
    const bool alone = gridDim.x == kCluster;
    float pc = 0.f;
    if (mine) {
        Sum s;
        int c = 0;
#pragma unroll
        for (int r = 0; r < kCluster; ++r) {
            s.add(of_rank(&p_block[e], r));
            c += of_rank(&cs[e], r);
        }
        if (alone) {
            a.counts[e] = c;
            pc = s.value() * static_cast<float>(c);
        } else {
            const int64_t at = static_cast<int64_t>(blockIdx.x / kCluster) * a.E + e;
            a.part_p[at] = s.value();
            a.part_c[at] = c;
        }
    }
    Totals sum = {0.f, 0, 0};
    if (threadIdx.x == 0 && rank == 0) {
        for (int r = 0; r < kCluster; ++r) {
            sum.z += of_rank(&total.z, r);
            sum.tokens += of_rank(&total.tokens, r);
            sum.bad |= of_rank(&total.bad, r);
        }
        if (!alone) a.part_s[blockIdx.x / kCluster] = {sum.z, sum.tokens, sum.bad};
    }
    if (alone) {  // one cluster holds every token: it ends the call
        pc = row_sum<32>(pc);
        if (lane == 0) pcs[warp] = pc;
        __syncthreads();
        if (threadIdx.x == 0) {
            pc = 0.f;
            for (int w = 0; w < kWarps; ++w) pc += pcs[w];
            pc_rank = pc;
        }
        cluster_barrier();
        if (threadIdx.x == 0 && rank == 0) {
            pc = 0.f;
            for (int r = 0; r < kCluster; ++r) pc += of_rank(&pc_rank, r);
            write_losses(a, pc, sum);
        }
    }
    cluster_barrier();  // nobody leaves while its shared memory is read
}

// Joins the clusters' partial sums: `seg` threads an expert, each over every
// seg-th cluster, then in order.
constexpr int kJoinThreads = 1024;
constexpr int kJoinPer = (kBalanceMaxClusters + 3) / 4;  // at most, with E = 256

__global__ void __launch_bounds__(kJoinThreads) balance_join_kernel(const BalanceArgs a) {
    __shared__ float ps[kJoinThreads];
    __shared__ int cs[kJoinThreads];
    __shared__ float ls[kJoinThreads / 32];
    __shared__ Totals total;
    griddep_launch_dependents();
    griddep_wait();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int seg = kJoinThreads / a.E;
    const int e = threadIdx.x % a.E, s = threadIdx.x / a.E;
    Sum p;
    int c = 0;
    if (s < seg) {
#pragma unroll
        for (int i = 0; i < kJoinPer; ++i) {
            const int b = s + i * seg;
            if (b < a.clusters) {
                p.add(__ldcg(a.part_p + b * a.E + e));
                c += __ldcg(a.part_c + b * a.E + e);
            }
        }
    }
    ps[threadIdx.x] = p.value();
    cs[threadIdx.x] = c;
    if (warp == kJoinThreads / 32 - 1) {
        Totals t = {0.f, 0, 0};
        for (int b = lane; b < a.clusters; b += 32) {
            t.z += __ldcg(&a.part_s[b].z);
            t.tokens += __ldcg(&a.part_s[b].tokens);
            t.bad |= __ldcg(&a.part_s[b].bad);
        }
        t.z = row_sum<32>(t.z);
        t.tokens = __reduce_add_sync(0xffffffffu, t.tokens);
        t.bad = __reduce_or_sync(0xffffffffu, t.bad);
        if (lane == 0) total = t;
    }
    __syncthreads();
    float pc = 0.f;
    if (threadIdx.x < a.E) {
        Sum q;
        c = 0;
        const int n = seg < a.clusters ? seg : a.clusters;
        for (int i = 0; i < n; ++i) {
            q.add(ps[i * a.E + threadIdx.x]);
            c += cs[i * a.E + threadIdx.x];
        }
        a.counts[threadIdx.x] = c;
        pc = q.value() * static_cast<float>(c);
    }
    pc = row_sum<32>(pc);
    if (lane == 0) ls[warp] = pc;
    __syncthreads();
    if (threadIdx.x == 0) {
        pc = 0.f;
        for (int w = 0; w < MOE_MAX_EXPERTS / 32; ++w) pc += ls[w];
        write_losses(a, pc, total);
    }
}

template <bool kBf16, int kLanes, bool kVec>
__global__ void __launch_bounds__(kThreads, 2) balance_grad_kernel(const BalanceArgs a) {
    constexpr int kPerWarp = 32 / kLanes;
    constexpr int kRows = kRowsPerWarp<kLanes>;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x % 32;
    const int t = lane % kLanes, sub = lane / kLanes;
    int64_t base = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / 32 * kRows;
    RawRow<kBf16, kVec> raw[kUnroll];
    load_rows<kBf16, kLanes, kVec>(a, base, t, sub, raw);
    const int T = __ldcg(a.tokens);
    const float invT = T > 0 ? 1.f / static_cast<float>(T) : 0.f;
    // g0 E d_e / T with E d_e = (E c_e - k T) / (k T): the difference in whole
    // numbers
    const int64_t kT = static_cast<int64_t>(a.k) * T;
    const float g0 = T > 0 ? __ldcg(a.grad) * invT / static_cast<float>(kT) : 0.f;
    const float g1 = 2.f * __ldcg(a.grad + 1) * invT;
    float d[kVals];
#pragma unroll
    for (int v = 0; v < kVals; ++v) {
        const int e = expert_of<kLanes, kVec>(t, v);
        d[v] = e < a.E ? g0 * static_cast<float>(
                                  static_cast<int64_t>(__ldcg(a.counts_in + e)) * a.E - kT)
                       : 0.f;
    }
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32) * kRows;
    for (; base < a.N; base += step) {
        const int left = a.N - base < kRows ? static_cast<int>(a.N - base) : kRows;
        void *out = at_element<kBf16>(a.dlogits, base * a.E);
        float x[kUnroll][kVals];
        bool in[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            in[u] = u * kPerWarp + sub < left;
            unpack_row<kBf16, kLanes, kVec>(raw[u], a.E, t, x[u]);
        }
        // out may be the logits: rows of other warps are never read, and this
        // warp's next rows are not the ones stored below
        load_rows<kBf16, kLanes, kVec>(a, base + step, t, sub, raw);
        if (a.mask) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                in[u] = in[u] && __ldcg(a.mask + base + u * kPerWarp + sub);
        }
        float f[kUnroll], lse[kUnroll], mean[kUnroll];
        softmax_rows<kLanes>(x, f, lse);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            mean[u] = 0.f;
#pragma unroll
            for (int v = 0; v < kVals; ++v) mean[u] = fmaf(d[v], x[u][v], mean[u]);
        }
        rows_sum<kLanes>(mean);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const float rest = fmaf(g1, lse[u], -mean[u] * f[u]);
#pragma unroll
            for (int v = 0; v < kVals; ++v)
                x[u][v] = in[u] ? x[u][v] * f[u] * (d[v] + rest) : 0.f;
            const int r = u * kPerWarp + sub;
            if (r < left)
                store_row<kBf16, kLanes, kVec>(at_element<kBf16>(out, r * a.E), a.E, t, x[u]);
        }
    }
}

using BalanceKernel = void (*)(BalanceArgs);

enum Pass { kStats, kStatsLong, kAlone8, kAlone16, kGrad };

template <Pass kPass, bool kBf16, bool kVec, int kLanes>
BalanceKernel kernel_at() {
    if constexpr (kPass == kGrad)
        return balance_grad_kernel<kBf16, kLanes, kVec>;
    else if constexpr (kPass == kStats || kPass == kStatsLong)
        return balance_stats_kernel<kBf16, kLanes, kVec, kThreads, kBalanceCluster,
                                    kPass == kStatsLong>;
    else
        return balance_stats_kernel<kBf16, kLanes, kVec, kAloneThreads,
                                    kPass == kAlone8 ? 8 : 16, false>;
}

template <Pass kPass, bool kBf16, bool kVec>
BalanceKernel kernel_of(int lanes) {
    switch (lanes) {
        case 1: return kernel_at<kPass, kBf16, kVec, 1>();
        case 2: return kernel_at<kPass, kBf16, kVec, 2>();
        case 4: return kernel_at<kPass, kBf16, kVec, 4>();
        case 8: return kernel_at<kPass, kBf16, kVec, 8>();
        case 16: return kernel_at<kPass, kBf16, kVec, 16>();
        default: return kernel_at<kPass, kBf16, kVec, 32>();
    }
}

int lanes_of(int E) {
    int lanes = 1;
    while (lanes * kVals < E) lanes *= 2;
    return lanes;
}

std::atomic<bool> g_portable_only{false};

// Whether the device has room for a cluster of 16 blocks of this kernel, which
// no device promises (one that is partitioned may not have it); asked once a
// device, as the kernels that come here take the same threads and registers.
bool room_for_16(const void *kernel) {
    static std::atomic<uint64_t> asked{0}, room{0};
    if (g_portable_only.load(std::memory_order_relaxed)) return false;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (asked.load(std::memory_order_acquire) & bit)
        return room.load(std::memory_order_relaxed) & bit;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 16;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(16);
    cfg.blockDim = dim3(kAloneThreads);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    const bool fits = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0;
    if (!fits) cudaGetLastError();  // an answer, not an error of a later call
    if (fits) room.fetch_or(bit, std::memory_order_relaxed);
    asked.fetch_or(bit, std::memory_order_release);
    return fits;
}

// Rows are read four values at a time when every row starts on such a
// boundary (E a multiple of 4, the arrays aligned), else one at a time.
template <Pass kPass>
cudaError_t launch(const BalanceArgs &a, int blocks, cudaStream_t s) {
    const int lanes = lanes_of(a.E);
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.logits) |
                         (kPass == kGrad ? reinterpret_cast<uintptr_t>(a.dlogits) : 0);
    const bool vec = a.E % 4 == 0 && at % (a.bf16 ? 8 : 16) == 0;
    const BalanceKernel k =
        a.bf16 ? (vec ? kernel_of<kPass, true, true>(lanes) : kernel_of<kPass, true, false>(lanes))
               : (vec ? kernel_of<kPass, false, true>(lanes)
                      : kernel_of<kPass, false, false>(lanes));
    if constexpr (kPass == kAlone16) {  // clusters of more than 8 have to be asked for
        const void *f = reinterpret_cast<const void *>(k);
        cudaError_t e =
            cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        if (!room_for_16(f)) return launch<kAlone8>(a, 8, s);  // in more passes
    }
    constexpr bool kAlone = kPass == kAlone8 || kPass == kAlone16;
    constexpr unsigned kCluster = kPass == kGrad      ? 1
                                  : kPass == kAlone16 ? 16
                                  : kPass == kAlone8  ? 8
                                                      : kBalanceCluster;
    return launch_pdl(k, dim3(static_cast<unsigned>(blocks)),
                      dim3(kAlone ? kAloneThreads : kThreads), 0, s, kCluster, a);
}

int64_t rows_per_block(int E, int threads) { return threads / lanes_of(E) * kUnroll; }

}  // namespace

// One cluster does small batches on its own, of 8 blocks for one pass and of 16
// for up to three.  One pass of 16 takes less than several clusters and the
// second kernel (2048 x 128: 5.7 against 5.9 us, 3000 x 60 in bf16 5.5 against
// 5.7).  Two take up to 0.8 us more (4000 x 128: 7.1 against 6.3; 4099 x 60 6.0
// against 6.2), three 1.7 (6144 x 128: 8.6 against 6.9; 98304 x 8, the most
// tokens: 11.3 against 7.6), but a call from Python saves a launch and the
// workspace (9 us of 24 forward and backward).  A captured graph saves neither.
int balance_clusters(int64_t N, int E) {
    if (N <= 3 * 16 * rows_per_block(E, kAloneThreads)) return 1;
    const int64_t rows = kBalanceCluster * rows_per_block(E, kThreads);
    const int64_t c = (N + rows - 1) / rows;
    return static_cast<int>(c < kBalanceMaxClusters ? c : kBalanceMaxClusters);
}

void balance_portable_clusters(bool only) { g_portable_only = only; }

cudaError_t launch_balance(const BalanceArgs &a, int *launches, cudaStream_t s) {
    *launches = a.clusters > 1 ? 2 : 1;
    if (a.clusters == 1)
        return a.N <= 8 * rows_per_block(a.E, kAloneThreads) ? launch<kAlone8>(a, 8, s)
                                                             : launch<kAlone16>(a, 16, s);
    const int blocks = a.clusters * kBalanceCluster;
    const bool many = a.N > kFoldPasses * blocks * rows_per_block(a.E, kThreads);
    cudaError_t e = many ? launch<kStatsLong>(a, blocks, s) : launch<kStats>(a, blocks, s);
    if (e != cudaSuccess) return e;
    return launch_pdl(balance_join_kernel, dim3(1), dim3(kJoinThreads), 0, s, 1, a);
}

cudaError_t launch_balance_backward(const BalanceArgs &a, int num_sms, cudaStream_t s) {
    const int64_t rows = rows_per_block(a.E, kThreads);
    int64_t blocks = (a.N + rows - 1) / rows;
    if (blocks > num_sms * 2) blocks = num_sms * 2;
    return launch<kGrad>(a, static_cast<int>(blocks), s);
}

}  // namespace moe
