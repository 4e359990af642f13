// gated_ffn.cuh -- the products of the gated feed-forward block and of its
// backward pass:
//
//   gate = x Wg^T, up = x Wu^T, h = act(gate) * up     kFfnGateUp
//   out = h Wd^T (+ residual)                          kFfnDown
//   dh = dout Wd, dgate = dh * up * act'(gate),
//   dup = dh * act(gate), h again                      kFfnDh
//   dx = dgate Wg + dup Wu                             kFfnDx
//   dWg = dgate^T x, dWu = dup^T x, dWd = dout^T h     kFfnDw
//
// with x, out, dout, dx [N, H], Wg, Wu [I, H], Wd [H, I], the rest [N, I], all
// bf16.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "kernels.cuh"
#include "moe.h"

namespace moe {

enum FfnOp {
    kFfnGateUp = 0,
    kFfnDown = 1,
    kFfnDh = 2,
    kFfnDx = 3,
    kFfnDw = 4,
    kFfnGrads = 5  // kFfnDx and kFfnDw in one launch
};

// Pairs of CTAs that run at once at most; a launch's partial sums have room for
// two tiles a pair.
constexpr int kFfnMaxPairs = 76;
constexpr int kFfnTile = 256;  // rows of a tile
// The workspace's rows of h, dgate and dup start on whole lines of 128 bytes, so
// that their 32-byte stores are whole sectors.  (1021 x 1000 x 1400 with rows of I
// values and 16-byte stores: 4.6 us more of a training step; with rows on 32 bytes
// 54.0 us as with lines.)
constexpr int kFfnLd = 64;

// How a launch's tiles go to the pairs: whole waves of tiles, then, where the
// last wave is partial and K long, its tiles' K slices in `parts` equal runs,
// whose partial sums a second kernel adds.
struct FfnPlan {
    int tiles;   // output tiles
    int whole;   // tiles that one pair computes from end to end
    int parts;   // > 0: pairs that share the other tiles' slices
    int nk;      // K slices of a tile
    int bn;      // accumulator columns of a tile: 256 or 128
    int pairs;   // launched
    // kFfnGrads: dx's tiles and their slices, and whether they come before the
    // weights'; no tile is shared
    int dx_tiles, dx_nk, dx_first;
};

struct FfnArgs {
    int64_t N;
    int H, I;
    int act;
    int keep;                   // gate and up are stored
    const uint16_t *gate, *up;  // kFfnDh
    const uint16_t *residual;   // kFfnDown, nullable
    int boxes;                  // kFfnDw: the outputs leave by tensor-map stores
    int64_t ld;                 // row stride of h, dgate and dup (see kFfnLd)
    uint16_t *out[4];           // h, gate, up; h, dgate, dup; dWg, dWu, dWd (, dx); or one
    float *part;                // [2 pairs][256 x bn]
    int32_t *status;
    int reset_status;
    FfnPlan plan;
};

// The operands' tensor maps: a: the M side's, b: the N side's.  A K-major
// operand ([rows, K]) comes in boxes of 64 values of K x the rows of a CTA (128,
// or on the N side half a tile's columns), an MN-major one ([K, rows]) in boxes
// of 64 rows x 64 values of K.
struct FfnMaps {
    CUtensorMap a[5], b[5];  // kFfnGrads: kFfnDw's, then kFfnDx's
    CUtensorMap out[3];  // kFfnDw with FfnArgs::boxes: boxes of 32 rows x 64 values
};

FfnPlan ffn_plan(FfnOp op, int64_t N, int H, int I, int num_sms);
// Whether kFfnGrads takes less time than the two one after the other, and its plan.
bool ffn_grads_plan(int64_t N, int H, int I, int num_sms, FfnPlan *plan);
size_t ffn_part_bytes(const FfnPlan &p);
// The weights' gradients of up to this many slices of tokens leave by tensor-map
// stores, from tiles of 256 columns: the TMA unit has the time for them then (8
// tokens of 2048 x 8192: 25 us instead of 31, 256 tokens 33.6 and 36.7, 512 tokens
// 43.7 and 42.0, 1024 tokens 65 and 61).
constexpr int kFfnBoxSlices = 4;
cudaError_t launch_ffn(FfnOp op, const FfnMaps &maps, const FfnArgs &a, int *launches,
                       cudaStream_t s);
// Adds the partial sums, where the plan has any.
cudaError_t launch_ffn_join(FfnOp op, const FfnArgs &a, int *launches, cudaStream_t s);


// A decode batch, or a down step of some more tokens (ffn_split.cu; not the
// weights' gradients): with the tokens' operands (maps.a) in boxes of `bn` rows,
// the weights in boxes of 64 rows (gate, up), 128 (down), or, MN-major, of 64 x
// 64; bn 0: not for this batch.
struct FfnSplit {
    int bn;     // tokens of a tile
    int split;  // CTAs of a cluster that share a tile's K
};
FfnSplit ffn_split(FfnOp op, int64_t N, int H, int I, int num_sms);
cudaError_t launch_ffn_split(FfnOp op, const FfnMaps &maps, const FfnArgs &a, const FfnSplit &t,
                             cudaStream_t s);

// One or two tokens (ffn_rows.cu): kFfnGateUp (w0, w1: gate, up; their outputs
// may be null) and kFfnDown (w0), outputs in a.out[0].
constexpr int kFfnRowsTokens = 2;
bool ffn_rows_fit(int64_t N, int K);
cudaError_t launch_ffn_rows(FfnOp op, const FfnArgs &a, const uint16_t *x, const uint16_t *w0,
                            const uint16_t *w1, uint16_t *gate, uint16_t *up, int num_sms,
                            cudaStream_t s);

}  // namespace moe
