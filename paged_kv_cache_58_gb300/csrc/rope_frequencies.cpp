// Rotary frequencies, plain and scaled for contexts longer than the trained one (host).
#include <cmath>
#include <cstdint>

#include "../../include/pkv.h"

extern "C" {

pkv_status pkv_rope_frequencies(double* inv_freq, float* attn_scale, int rotary_dim, double theta,
                                const pkv_rope_scaling* scaling) {
    if (!inv_freq || rotary_dim <= 0 || (rotary_dim & 1) || !(theta > 0.0) || !std::isfinite(theta))
        return PKV_ERR_INVALID;
    const int kind = scaling ? scaling->kind : PKV_ROPE_PLAIN;
    if (kind < PKV_ROPE_PLAIN || kind > PKV_ROPE_YARN_PAIRS) return PKV_ERR_UNSUPPORTED;
    const double factor = kind == PKV_ROPE_PLAIN ? 1.0 : scaling->factor;
    if (!(factor >= 1.0) || !std::isfinite(factor)) return PKV_ERR_INVALID;
    const bool yarn = kind == PKV_ROPE_YARN || kind == PKV_ROPE_YARN_PAIRS;
    const bool banded = kind == PKV_ROPE_LLAMA3 || yarn;
    const double low = banded ? scaling->low : 0.0;
    const double high = banded ? scaling->high : 1.0;
    const double trained = banded ? scaling->original_context : 1.0;
    if (!(low >= 0.0) || !(high > low) || !std::isfinite(high) || !(trained > 0.0) ||
        !std::isfinite(trained))
        return PKV_ERR_INVALID;
    if (kind == PKV_ROPE_NTK) {
        if (rotary_dim <= 2) return PKV_ERR_INVALID;
        // the base that stretches the lowest frequency by `factor` and leaves the highest
        theta *= std::pow(factor, static_cast<double>(rotary_dim) / (rotary_dim - 2));
    }
    const double two_pi = 6.283185307179586476925;
    double first = 0.0, last = 0.0;   // pair indices between which frequencies blend
    if (kind == PKV_ROPE_YARN_PAIRS) {
        if (!(theta > 1.0)) return PKV_ERR_INVALID;
        // n turns over the trained context at pair i: theta^(-2 i / rotary_dim) trained = 2 pi n
        auto pair_of = [&](double turns) {
            return rotary_dim * std::log(trained / (two_pi * turns)) / (2.0 * std::log(theta));
        };
        first = std::fmax(std::floor(pair_of(high)), 0.0);
        last = low > 0.0 ? std::fmin(std::ceil(pair_of(low)), rotary_dim - 1.0) : rotary_dim - 1.0;
        if (last <= 0.0) {   // no pair turns more than `low` times
            first = -1.0;
            last = 0.0;
        }
        if (!(last > first)) last = first + 0.001;   // a step
    }
    for (int i = 0; i < rotary_dim / 2; ++i) {
        const double f = std::pow(theta, -2.0 * i / rotary_dim);
        double g = f;
        if (kind == PKV_ROPE_LINEAR) {
            g = f / factor;
        } else if (banded) {
            // turns over the trained context: at most `low` of them stretch by `factor`,
            // at least `high` stay, between a blend linear in them or in the pair index
            const double turns = trained * f / two_pi;
            const double part = kind == PKV_ROPE_YARN_PAIRS ? (last - i) / (last - first)
                                                            : (turns - low) / (high - low);
            const double keep = std::fmin(1.0, std::fmax(0.0, part));
            g = (1.0 - keep) * f / factor + keep * f;
        }
        inv_freq[i] = g;
    }
    if (attn_scale)
        *attn_scale = yarn ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
    return PKV_OK;
}

}  // extern "C"
