// linear.cu -- which kernel and tile moe_linear takes for its sizes.
//
// Both kernels' times follow their tile counts, so the rule estimates each
// candidate and takes the least.  The constants (microseconds) were fitted to
// measured times of every candidate on a GB300, for 19 batch sizes from 1 to
// 16384 and 8 weight shapes from 2048 x 128 to 8192 x 2048 in both operand
// types: the candidate it takes is on average 0.2% slower than the fastest one,
// 7% at worst.  What the sides are at 2048 x 2048 in bf16, pair tiles of 128
// outputs against the best split: 256 tokens 15.2 against 9.0 us, 1024 tokens
// 16.2 against 20.1; pair tiles of 256 against 128 outputs: 1024 tokens 18.5
// against 16.2, 4096 tokens 31.1 against 46.7.
#include "linear_gemm.cuh"

namespace moe {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The persistent pairs: whole waves of tiles, each the K slices' time or, when
// K is short, the epilogue's, and the last tile's epilogue on its own.
float pair_us(int64_t N, int64_t O, int nk, int bn, bool aligned, int sms) {
    const int64_t waves = ceil_div(ceil_div(N, 256) * ceil_div(O, bn), sms / 2);
    const float slices = nk * (bn == 256 ? 0.437f : 0.326f);
    const float epilogue = 3.1f * bn / 256 * (aligned ? 1.f : 8.1f);
    return 3.5f + waves * (slices > epilogue ? slices : epilogue) + 0.9f * epilogue;
}

// Clusters of `split` CTAs of one SM each: clusters of 4 fit 36 times on the
// 152 SMs and clusters of 8 15 times.
float split_us(int64_t N, int64_t O, int nk, int bn, int split, bool aligned, int sms) {
    const int fit = split <= 2 ? sms : split == 4 ? sms * 36 / 38 : sms * 15 / 19;
    const int64_t waves = ceil_div(ceil_div(N, bn) * ceil_div(O, 128) * split, fit);
    const float slice = bn == 128 ? 0.35f : bn == 64 ? 0.267f : bn == 32 ? 0.285f : 0.303f;
    const float epilogue = 0.0247f * bn / split * (aligned ? 1.f : 6.4f) + 0.0115f * bn;
    return 1.4f + waves * (1.7f + ceil_div(nk, split) * slice + epilogue);
}

}  // namespace

LinearTiling linear_tiling(const LinearArgs &a, int num_sms) {
    const int nk = static_cast<int>(ceil_div(a.K, a.fp8 ? 128 : 64));
    const bool vectors = a.O % 4 == 0;  // of the split kernel's stores
    const bool rows = linear_out_rows_aligned(a);
    LinearTiling best = {1, 256, 1};
    float least = pair_us(a.N, a.O, nk, 256, rows, num_sms);
    const auto consider = [&](float us, LinearTiling t) {
        if (us < least) {
            least = us;
            best = t;
        }
    };
    consider(pair_us(a.N, a.O, nk, 128, rows, num_sms), {1, 128, 1});
    for (int bn = 16; bn <= 128; bn *= 2) {
        if (ceil_div(a.N, bn) > 4096) continue;  // rows of its grid
        for (int split = 1; split <= 8 && split <= nk; split *= 2)
            consider(split_us(a.N, a.O, nk, bn, split, vectors, num_sms), {0, bn, split});
    }
    return best;
}

int linear_x_box(const LinearTiling &t) { return t.pair ? 128 : t.bn; }
int linear_w_box(const LinearTiling &t) { return t.pair ? t.bn / 2 : 128; }

}  // namespace moe
