// linear.cu -- which kernel and tile moe_linear takes for its sizes.
#include "linear_gemm.cuh"

namespace moe {

namespace {

// Estimated SM cycles of a call.  A CTA takes in about 64 bytes a cycle
// from L2 and its tensor core 128 x 128 outputs of a K slice in 256 cycles.
constexpr double kBytesPerCycle = 64.0;
constexpr double kCallCycles = 3000.0;

double ceil_div(double a, double b) { return static_cast<double>(static_cast<int64_t>((a + b - 1) / b)); }

double pair_cycles(double N, double O, double nk, int bn, int sms) {
    const double slice = bn * 2.0 > (16384 + bn * 64) / kBytesPerCycle
                             ? bn * 2.0 : (16384 + bn * 64) / kBytesPerCycle;
    const double waves = ceil_div(ceil_div(N, 256) * ceil_div(O, bn), sms / 2);
    return kCallCycles + waves * nk * slice + 12.0 * bn;
}

double split_cycles(double N, double O, double nk, int bn, int split, int sms) {
    const double slice = bn * 2.0 > (16384 + bn * 128) / kBytesPerCycle
                             ? bn * 2.0 : (16384 + bn * 128) / kBytesPerCycle;
    const double waves = ceil_div(ceil_div(N, bn) * ceil_div(O, 128) * split, sms);
    return kCallCycles + waves * (1500.0 + ceil_div(nk, split) * slice + 30.0 * bn);
}

}  // namespace

LinearTiling linear_tiling(const LinearArgs &a, int num_sms) {
    const double nk = ceil_div(a.K, a.fp8 ? 128 : 64);
    LinearTiling best = {1, 256, 1};
    double cost = pair_cycles(a.N, a.O, nk, 256, num_sms);
    const auto take = [&](double c, LinearTiling t) {
        if (c < cost) {
            cost = c;
            best = t;
        }
    };
    take(pair_cycles(a.N, a.O, nk, 128, num_sms), {1, 128, 1});
    for (int bn = 16; bn <= 128; bn *= 2) {
        if ((a.N + bn - 1) / bn > 4096) continue;
        for (int split = 1; split <= 8 && split <= nk; split *= 2)
            take(split_cycles(a.N, a.O, nk, bn, split, num_sms), {0, bn, split});
    }
    return best;
}

int linear_x_box(const LinearTiling &t) { return t.pair ? 128 : t.bn; }
int linear_w_box(const LinearTiling &t) { return t.pair ? t.bn / 2 : 128; }

}  // namespace moe
