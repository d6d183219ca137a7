// Rows of a quantised cache: how a row of D elements becomes codes, scales and an exponent,
// and back (the format is stated in include/pkv.h, "quantised cache").
//
// A row is worked on by D / 16 neighbouring lanes, 16 elements each, so that the 16 elements
// that share an fp4 scale lie in one lane.  The row's exponent is a power of two: x 2^-e is
// exact, and the one rounding is the code's.  (A scale of amax / 448 would round twice, and
// gain nothing: e4m3 has the same relative precision over its whole normal range.)
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"

namespace pkv {

// Sizes of a format at head dimension D: bytes of a row of codes, and of what lies beside 16
// rows of one kv head (fp4: a scale per 16 elements; then 16 exponents).
template <int FMT, int D>
struct QuantRow {
    static constexpr int kCodes = FMT == PKV_FP8 ? D : D / 2;
    static constexpr int kScales = FMT == PKV_FP8 ? 0 : D;
    static constexpr int kSide = kScales + 16;
    static constexpr int kLanes = D / 16;        // lanes that share a row
    static constexpr int kLaneBytes = kCodes / kLanes;   // code bytes of a lane: 16 or 8
};

// Byte of the fp4 scale of token t (0 .. 15) and elements 16 g .. 16 g + 15 in what lies beside
// 16 rows.  K's are read a token at a time, V's four tokens of one group at a time: both as the
// decode kernel's lanes want them.
template <int D>
PKV_DEVINL int scale_at(bool is_v, int t, int g) {
    return is_v ? (t >> 2) * (D / 4) + 4 * g + (t & 3) : t * (D / 16) + g;
}

PKV_DEVINL float pow2f(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127

// Two e4m3 values (low half of x, low byte first) / two e2m1 values (byte `b` of x, low nibble
// first) as two fp16 values; every value of either is one of fp16, NaN included.
PKV_DEVINL uint32_t e4m3x2_to_f16x2(uint32_t x) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
        : "=r"(r)
        : "r"(x));
    return r;
}
PKV_DEVINL void e4m3x4_to_f16x4(uint32_t x, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
}
PKV_DEVINL void e2m1x8_to_f16x8(uint32_t x, uint32_t (&v)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
        : "r"(x));
}
PKV_DEVINL uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
PKV_DEVINL float f16lo_to_f32(uint32_t w) {
    float r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(r) : "r"(w));
    return r;
}
PKV_DEVINL float f16hi_to_f32(uint32_t w) {
    float r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, h;\n\t}" : "=f"(r) : "r"(w));
    return r;
}
// Two fp32 values to the nearest e4m3 / e2m1 (ties to even, beyond the largest to the largest).
PKV_DEVINL uint32_t to_e4m3x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %1, %2;\n\tcvt.u32.u16 %0, h;\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}
PKV_DEVINL uint32_t to_e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tcvt.u32.u8 %0, b;\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}

// 16 elements of a row: bf16 bits or fp32.
template <typename T>
struct Elems16;
template <>
struct Elems16<uint16_t> {
    uint4 w[2];
    PKV_DEVINL void load(const void* p) {
        w[0] = __ldg(static_cast<const uint4*>(p));
        w[1] = __ldg(static_cast<const uint4*>(p) + 1);
    }
    PKV_DEVINL void values(float (&x)[16]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t q[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[8 * i + 2 * k] = bf16lo_to_f32(q[k]);
                x[8 * i + 2 * k + 1] = bf16hi_to_f32(q[k]);
            }
        }
    }
    PKV_DEVINL static void store(void* p, const float (&x)[16]) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            static_cast<uint4*>(p)[i] =
                make_uint4(pack_bf16x2(x[8 * i], x[8 * i + 1]),
                           pack_bf16x2(x[8 * i + 2], x[8 * i + 3]),
                           pack_bf16x2(x[8 * i + 4], x[8 * i + 5]),
                           pack_bf16x2(x[8 * i + 6], x[8 * i + 7]));
    }
};
template <>
struct Elems16<float> {
    float4 w[4];
    PKV_DEVINL void load(const void* p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __ldg(static_cast<const float4*>(p) + i);
    }
    PKV_DEVINL void values(float (&x)[16]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[4 * i] = w[i].x;
            x[4 * i + 1] = w[i].y;
            x[4 * i + 2] = w[i].z;
            x[4 * i + 3] = w[i].w;
        }
    }
    PKV_DEVINL static void store(void* p, const float (&x)[16]) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            static_cast<float4*>(p)[i] =
                make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    }
};

// What a lane's 16 elements became: code bytes (fp4: the first two words), their scale (fp4) and
// the row's exponent, biased.
struct Quantised {
    uint32_t codes[4];
    uint32_t scale, exp;
};

// Quantises a row whose 16 elements per lane lie in x; the lanes of a row are neighbours and all
// 32 lanes of the warp call.  EXACT_DIV: x has more than bf16's digits.
//   NaN stays NaN (fp4: its 16 elements do); infinities take the largest value.
template <int FMT, int D, bool EXACT_DIV>
PKV_DEVINL Quantised quantise(const float (&x)[16]) {
    constexpr int L = QuantRow<FMT, D>::kLanes;
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));   // passes over NaN
    float top = amax;
#pragma unroll
    for (int o = 1; o < L; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // The least e with top <= 448 2^e = 1.75 2^(e + 8), or 2688 2^e = 1.3125 2^(e + 11): the
    // exponent of top less that of the largest value, one more where top's digits pass its.
    const int bits = __float_as_int(top);
    int e = FMT == PKV_FP8 ? ((bits + 0x1fffff) >> 23) - 135 : ((bits + 0x57ffff) >> 23) - 138;
    e = max(-90, min(90, e));
    const float unit = pow2f(-e);
    Quantised r;
    r.exp = static_cast<uint32_t>(e + 127);
    r.scale = 0;
    if constexpr (FMT == PKV_FP8) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r.codes[i] = to_e4m3x2(x[4 * i] * unit, x[4 * i + 1] * unit) |
                         to_e4m3x2(x[4 * i + 2] * unit, x[4 * i + 3] * unit) << 16;
    } else {
        bool nan = false;
#pragma unroll
        for (int i = 0; i < 16; ++i) nan |= x[i] != x[i];
        const float a = fminf(amax * unit, 2688.f);
        // A sixth in fp32: a product, exact where a sixth is a midpoint of e4m3 (6 m (1 / 6) is off
        // by 2^-25 of m before it is rounded, to m), so that ties stay ties.
        r.scale = to_e4m3x2(a * (1.f / 6.f), 0.f) & 0xffu;
        const float s = f16lo_to_f32(e4m3x2_to_f16x2(r.scale));
        if (nan) r.scale = 0x7fu;
        const float inv = s > 0.f ? __fdiv_rn(1.f, s) : 0.f;
        float u[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float y = x[i] * unit;
            if constexpr (EXACT_DIV) {
                // On a border only where y / s is: where y is a unit in its last place
                // off it, the quotient is off by more than half of its own.
                u[i] = s > 0.f ? __fdiv_rn(y, s) : 0.f;
            } else {
                // y and border * s have at most 8 digits: y inv is within 2 units of a border
                // where y / s is on it and 2^15 away where it is not.  Dropping four digits
                // tells the two apart.
                u[i] = __int_as_float((__float_as_int(y * inv) + 8) & ~15);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float* v = u + 8 * i;
            r.codes[i] = to_e2m1x2(v[0], v[1]) | to_e2m1x2(v[2], v[3]) << 8 |
                         to_e2m1x2(v[4], v[5]) << 16 | to_e2m1x2(v[6], v[7]) << 24;
        }
        r.codes[2] = r.codes[3] = 0;
    }
    return r;
}

// The 16 values of a lane's codes.  `scale`: the fp4 scale's byte; `exp`: the row's exponent.
template <int FMT>
PKV_DEVINL void dequantise(const uint32_t (&codes)[4], uint32_t scale, uint32_t exp,
                           float (&x)[16]) {
    const float unit = pow2f(static_cast<int>(exp) - 127);
    if constexpr (FMT == PKV_FP8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t lo, hi;
            e4m3x4_to_f16x4(codes[i], lo, hi);
            x[4 * i] = f16lo_to_f32(lo) * unit;
            x[4 * i + 1] = f16hi_to_f32(lo) * unit;
            x[4 * i + 2] = f16lo_to_f32(hi) * unit;
            x[4 * i + 3] = f16hi_to_f32(hi) * unit;
        }
    } else {
        const uint32_t s = e4m3x2_to_f16x2(scale | scale << 8);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t v[4];
            e2m1x8_to_f16x8(codes[i], v);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t w = hmul2(v[k], s);   // exact: 6 digits, of 2^-10 or more
                x[8 * i + 2 * k] = f16lo_to_f32(w) * unit;
                x[8 * i + 2 * k + 1] = f16hi_to_f32(w) * unit;
            }
        }
    }
}

}  // namespace pkv
