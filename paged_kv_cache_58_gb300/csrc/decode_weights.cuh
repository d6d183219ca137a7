// Accumulated attention weights of a decode step: what the split kernels and the finishing
// launch share.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace pkv {

// The G scores of a token, in the widest loads their alignment (4 G bytes) allows.
template <int G>
PKV_DEVINL void load_scores(const float* p, float (&s)[G]) {
    if constexpr (G == 1) {
        s[0] = *p;
    } else if constexpr (G == 2) {
        const float2 f = *reinterpret_cast<const float2*>(p);
        s[0] = f.x; s[1] = f.y;
    } else {
#pragma unroll
        for (int g = 0; g < G; g += 4) {
            const float4 f = *reinterpret_cast<const float4*>(p + g);
            s[g] = f.x; s[g + 1] = f.y; s[g + 2] = f.z; s[g + 3] = f.w;
        }
    }
}

// A token's weight in this step, sum_g 2^(s_g - M_g) / sum_g; coef[0][g] = M_g, coef[1][g] =
// 1 / sum_g.
template <int G>
PKV_DEVINL float step_weight(const float (&s)[G], const float (*coef)[G]) {
    float p = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) p = fmaf(fast_exp2(s[g] - coef[0][g]), coef[1][g], p);
    return p;
}

// The weights of one (sequence, kv head) of L tokens by the CTA that has all of its scores
// (one partition): every thread of the CTA calls, after a barrier past the last score and
// past coef.
template <int G>
PKV_DEVINL void add_own_weights(const DecodeArgs& a, int seq, int kvh, int L,
                                const float (*coef)[G]) {
    const int row = a.row_ids ? __ldg(a.row_ids + seq) : seq;
    if (row < 0) return;   // padding
    if (row >= a.num_rows || L > a.weights_stride) {
        if (threadIdx.x == 0) raise_status(a.status, PKV_ERR_OOB);
        if (row >= a.num_rows) return;
        L = static_cast<int>(a.weights_stride);
    }
    const float* sp = a.scores + (static_cast<size_t>(seq) * a.num_kv_heads + kvh) *
                                     a.score_tokens * G;
    float* wp = a.weights + (static_cast<size_t>(row) * a.num_kv_heads + kvh) *
                                static_cast<size_t>(a.weights_stride);
    for (int j = threadIdx.x; j < L; j += blockDim.x) {
        float s[G];
        load_scores<G>(sp + static_cast<size_t>(j) * G, s);
        const float p = step_weight<G>(s, coef);
        wp[j] = a.decay != 0.f ? fmaf(a.decay, wp[j], p) : p;
    }
}

}  // namespace pkv
