// Host arithmetic: the rotary frequencies, and the alpha / gamma planner.
//
// The alpha / gamma planner: host arithmetic of "Fast Inference from
// Transformers via Speculative Decoding", section "方法细节" (期望生成 token
// 数, 墙钟加速因子, 运算量分析) and its FAQ on choosing gamma. No GPU work.

#include <algorithm>
#include <cmath>

#include "specverify.h"

namespace {

bool alpha_ok(double a) { return a >= 0.0 && a <= 1.0; }

constexpr double kPi = 3.14159265358979323846;

// The fraction of a turn that an angle of x radians leaves, in units of 2^-64.
uint64_t turns_of(double x) {
    const double t = x / (2.0 * kPi), f = t - std::floor(t);
    return f >= 1.0 ? 0 : (uint64_t)std::ldexp(f, 64);
}

}  // namespace

extern "C" {

spec_status spec_rotary_turns(int dim, double base, spec_rotary_scaling scaling, double scale, double original,
                              uint64_t* turns, float* factor) {
    if (dim < 2 || dim > SPEC_MAX_HEAD_DIM || dim % 2 != 0 || !(base > 1.0) || std::isinf(base) || !turns || !factor)
        return SPEC_EINVAL;
    const bool ranged = scaling == SPEC_ROTARY_YARN || scaling == SPEC_ROTARY_BANDS;
    if (scaling < SPEC_ROTARY_PLAIN || scaling > SPEC_ROTARY_BANDS || (scaling == SPEC_ROTARY_NTK && dim == 2)) return SPEC_EINVAL;
    if (scaling != SPEC_ROTARY_PLAIN && (!(scale >= 1.0) || std::isinf(scale))) return SPEC_EINVAL;
    if (ranged && (!(original > 0.0) || std::isinf(original))) return SPEC_EINVAL;
    if (scaling == SPEC_ROTARY_NTK) base *= std::pow(scale, dim / (dim - 2.0));
    if (std::isinf(base)) return SPEC_EINVAL;
    double low = 0.0, high = 0.0;
    if (scaling == SPEC_ROTARY_YARN) {
        // the pair that turns r times in the original length
        auto pair = [&](double r) { return dim * std::log(original / (r * 2.0 * kPi)) / (2.0 * std::log(base)); };
        low = std::max(std::floor(pair(32.0)), 0.0);
        high = std::min(std::ceil(pair(1.0)), dim - 1.0);
    }
    for (int j = 0; j < dim / 2; ++j) {
        double f = std::pow(base, -2.0 * j / dim);
        if (scaling == SPEC_ROTARY_LINEAR) f /= scale;
        if (ranged) {  // keep: how much of the pair's own frequency stays
            const double keep = scaling == SPEC_ROTARY_YARN ? 1.0 - (j - low) / std::max(high - low, 0.001)
                                                            : (original * f / (2.0 * kPi) - 1.0) / 3.0;
            const double k = std::min(std::max(keep, 0.0), 1.0);
            f = f * k + f / scale * (1.0 - k);
        }
        turns[j] = turns_of(f);
    }
    *factor = scaling == SPEC_ROTARY_YARN ? (float)(0.1 * std::log(scale) + 1.0) : 1.f;
    return SPEC_OK;
}

double spec_expected_tokens(double alpha, int gamma) {
    if (!alpha_ok(alpha) || gamma < 0) return NAN;
    if (alpha == 1.0) return gamma + 1.0;
    return (1.0 - std::pow(alpha, (double)(gamma + 1))) / (1.0 - alpha);
}

double spec_walltime_factor(double alpha, int gamma, double c) {
    if (!(c >= 0.0) || std::isinf(c)) return NAN;
    return spec_expected_tokens(alpha, gamma) / (gamma * c + 1.0);
}

double spec_ops_factor(double alpha, int gamma, double c_hat) {
    if (!(c_hat >= 0.0) || std::isinf(c_hat)) return NAN;
    return (gamma * c_hat + gamma + 1.0) / spec_expected_tokens(alpha, gamma);
}

int spec_best_gamma(double alpha, double c, int gamma_max) {
    if (!alpha_ok(alpha) || !(c >= 0.0) || std::isinf(c) || gamma_max < 1) return -1;
    double best = -1.0;
    int arg = 1;
    for (int g = 1; g <= gamma_max; ++g) {
        const double f = spec_walltime_factor(alpha, g, c);
        if (f > best) {
            best = f;
            arg = g;
        }
    }
    return arg;
}

}  // extern "C"
