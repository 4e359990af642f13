// linear.cu -- which kernel and tile moe_linear takes for its sizes.
//
// Both kernels' times follow their tile counts, so the rule estimates each
// candidate and takes the least.  The constants (microseconds) were fitted to
// measured times of every candidate on a GB300, for 19 batch sizes from 1 to
// 16384 and 11 weight shapes from 512 x 256 to 8192 x 2048 in both operand
// types: the candidate it takes is on average 0.5% slower than the fastest one,
// 16% at worst (on 7 other weight shapes 0.6%, 19% at worst).  What the sides
// are at 2048 x 2048 in bf16, pair tiles of 128 outputs against the best split:
// 256 tokens 10.6 against 7.2 us, 512 tokens 10.8 against 9.5, 1024 tokens 13.1
// against 16.0; pair tiles of 256 against 128 outputs: 1024 tokens 17.2 against
// 13.1, 4096 tokens 27.5 against 33.0.
#include <cmath>

#include "linear_gemm.cuh"

namespace moe {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Whole waves of `tiles` on `at_once`, in float: the rule is on the path of
// every call, and 64-bit divisions were a third of a microsecond of it.
float waves_of(int64_t tiles, float at_once) {
    return ceilf(static_cast<float>(tiles) / at_once - 1e-6f);
}

// The persistent pairs: whole waves of tiles, each the K slices' time or, when
// K is short, the epilogue's, and the last tile's epilogue on its own.
float pair_us(int64_t tiles, int nk, int bn, bool aligned, int sms) {
    const float slices = nk * (bn == 256 ? 0.34f : 0.237f);
    const float epilogue = 2.27f * bn / 256 * (aligned ? 1.f : 4.6f);
    return 4.2f + waves_of(tiles, static_cast<float>(sms / 2)) *
                      (slices > epilogue ? slices : epilogue) + 0.92f * epilogue;
}

}  // namespace

LinearTiling linear_tiling(const LinearArgs &a, int num_sms) {
    const int nk = static_cast<int>(ceil_div(a.K, a.fp8 ? 128 : 64));
    const int64_t m256 = (a.N + 255) >> 8, o128 = (a.O + 127) >> 7;
    const bool rows = linear_out_rows_aligned(a);
    LinearTiling best = {1, 256, 1};
    float least = pair_us(m256 * ((o128 + 1) >> 1), nk, 256, rows, num_sms);
    const auto consider = [&](float us, LinearTiling t) {
        if (us < least) {
            least = us;
            best = t;
        }
    };
    consider(pair_us(m256 * o128, nk, 128, rows, num_sms), {1, 128, 1});
    // Clusters of `split` CTAs of one SM each: clusters of 4 fit 36 times on
    // the 152 SMs and clusters of 8 15 times.
    const float fit[4] = {1.f, 1.f, 36.f / 38.f, 15.f / 19.f};
    const float slice[4] = {0.181f, 0.222f, 0.2f, 0.22f};
    const float store = a.O % 4 == 0 ? 0.0199f : 0.0653f;  // vectors or single values
    for (int b = 0; b < 4; ++b) {
        const int bn = 16 << b;
        const int64_t tiles = ((a.N + bn - 1) >> (4 + b)) * o128;
        if (a.N > static_cast<int64_t>(bn) * 4096) continue;  // rows of its grid
        for (int l = 0; l < 4 && (1 << l) <= nk; ++l) {
            const float w = waves_of(tiles << l, num_sms * fit[l]);
            const int slices = (nk + (1 << l) - 1) >> l;
            consider(0.8f + w * (1.95f + slices * slice[b] + store * bn / (1 << l) + 0.0176f * bn),
                     {0, bn, 1 << l});
        }
    }
    return best;
}

int linear_x_box(const LinearTiling &t) { return t.pair ? 128 : t.bn; }
int linear_w_box(const LinearTiling &t) { return t.pair ? t.bn / 2 : 128; }

}  // namespace moe
