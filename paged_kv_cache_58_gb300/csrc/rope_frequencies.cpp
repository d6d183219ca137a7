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
    if (kind < PKV_ROPE_PLAIN || kind > PKV_ROPE_YARN) return PKV_ERR_UNSUPPORTED;
    const double factor = kind == PKV_ROPE_PLAIN ? 1.0 : scaling->factor;
    if (!(factor >= 1.0) || !std::isfinite(factor)) return PKV_ERR_INVALID;
    const bool banded = kind == PKV_ROPE_LLAMA3 || kind == PKV_ROPE_YARN;
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
    for (int i = 0; i < rotary_dim / 2; ++i) {
        const double f = std::pow(theta, -2.0 * i / rotary_dim);
        double g = f;
        if (kind == PKV_ROPE_LINEAR) {
            g = f / factor;
        } else if (banded) {
            // turns over the trained context: at most `low` of them stretch by `factor`,
            // at least `high` stay, a linear blend between
            const double turns = trained * f / two_pi;
            const double keep = std::fmin(1.0, std::fmax(0.0, (turns - low) / (high - low)));
            g = (1.0 - keep) * f / factor + keep * f;
        }
        inv_freq[i] = g;
    }
    if (attn_scale)
        *attn_scale = kind == PKV_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
    return PKV_OK;
}

}  // extern "C"
