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
// Both halves of a times the low (high) half of b.
PKV_DEVINL uint32_t hmul2_lo(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\t.reg .b32 d;\n\tmov.b32 {l, h}, %2;\n\tmov.b32 d, {l, l};\n\t"
        "mul.rn.f16x2 %0, %1, d;\n\t}"
        : "=r"(r)
        : "r"(a), "r"(b));
    return r;
}
PKV_DEVINL uint32_t hmul2_hi(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\t.reg .b32 d;\n\tmov.b32 {l, h}, %2;\n\tmov.b32 d, {h, h};\n\t"
        "mul.rn.f16x2 %0, %1, d;\n\t}"
        : "=r"(r)
        : "r"(a), "r"(b));
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
// Two fp32 values to the nearest e4m3 (ties to even, beyond the largest to the largest).
PKV_DEVINL uint32_t to_e4m3x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %1, %2;\n\tcvt.u32.u16 %0, h;\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}
// 32 bytes at once (`wide`: p is 32-byte aligned), or 16 and 16.  A lane that moves its 32 bytes in
// two halves leaves half-written sectors to L2 (reading back 8192 tokens of 8 heads of 128 to bf16:
// 13.5 us, 11.1 in whole sectors).
PKV_DEVINL void load32(const void* p, bool wide, uint32_t* w) {
    if (wide) {
        // volatile: it stays behind the wait for the kernel before
        asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                       "=r"(w[6]), "=r"(w[7])
                     : "l"(p)
                     : "memory");
    } else {
        const uint4 u = __ldg(static_cast<const uint4*>(p));
        const uint4 v = __ldg(static_cast<const uint4*>(p) + 1);
        w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
        w[4] = v.x; w[5] = v.y; w[6] = v.z; w[7] = v.w;
    }
}
PKV_DEVINL void store32(void* p, bool wide, const uint32_t* w) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "l"(p)
                     : "memory");
    } else {
        static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// 16 elements of a row: bf16 bits or fp32.
template <typename T>
struct Elems16;
template <>
struct Elems16<uint16_t> {
    uint32_t w[8];
    PKV_DEVINL void clear() {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 0;
    }
    PKV_DEVINL void load(const void* p, bool wide) { load32(p, wide, w); }
    PKV_DEVINL void values(float (&x)[16]) const {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            x[2 * k] = bf16lo_to_f32(w[k]);
            x[2 * k + 1] = bf16hi_to_f32(w[k]);
        }
    }
    // The largest magnitude's bits as fp32: above 0x7f800000 where there is a NaN.
    PKV_DEVINL uint32_t top_bits() const {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) m = __vmaxu2(m, w[k] & 0x7fff7fffu);
        return max(m << 16, m & 0xffff0000u);
    }
    PKV_DEVINL static void store(void* p, bool wide, const float (&x)[16]) {
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = pack_bf16x2(x[2 * k], x[2 * k + 1]);
        store32(p, wide, w);
    }
};
template <>
struct Elems16<float> {
    uint32_t w[16];
    PKV_DEVINL void clear() {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = 0;
    }
    PKV_DEVINL void load(const void* p, bool wide) {
        load32(p, wide, w);
        load32(static_cast<const char*>(p) + 32, wide, w + 8);
    }
    PKV_DEVINL void values(float (&x)[16]) const {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(w[i]);
    }
    PKV_DEVINL uint32_t top_bits() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) m = max(m, w[i] & 0x7fffffffu);
        return m;
    }
    PKV_DEVINL static void store(void* p, bool wide, const float (&x)[16]) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(x[i]);
        store32(p, wide, w);
        store32(static_cast<char*>(p) + 32, wide, w + 8);
    }
};

// What a lane's 16 elements became: code bytes (fp4: the first two words), their scale (fp4) and
// the row's exponent, biased.
struct Quantised {
    uint32_t codes[4];
    uint32_t scale, exp;
};

PKV_DEVINL uint32_t to_e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\tmov.b32 %0, {l, h};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}
PKV_DEVINL uint32_t to_e2m1x8(const float* u) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(u[0]), "f"(u[1]), "f"(u[2]), "f"(u[3]), "f"(u[4]), "f"(u[5]), "f"(u[6]), "f"(u[7]));
    return r;
}

// Eight e2m1 codes with zeros' signs cleared: the ways to a code keep or lose the sign of what rounds
// to zero, and the bytes are not to depend on the way.
PKV_DEVINL uint32_t plain_zeros(uint32_t c) {
    const uint32_t m = c & 0x77777777u;                    // + 7: bit 3 set where it is not zero
    return m | (c & (m + 0x77777777u) & 0x88888888u);
}

// The least e with top <= 448 2^e = 1.75 2^(e + 8), or 2688 2^e = 1.3125 2^(e + 11), top of these
// bits: the exponent of top less that of the largest value, one more where top's digits pass its.
template <int FMT>
PKV_DEVINL int row_exponent(uint32_t top) {
    const int e = FMT == PKV_FP8 ? (static_cast<int>(top + 0x1fffffu) >> 23) - 135
                                 : (static_cast<int>(top + 0x57ffffu) >> 23) - 138;
    return max(-90, min(90, e));
}

// Quantises a row, 16 elements per lane; the lanes of a row are neighbours and all 32 lanes of the
// warp call.  NaN stays NaN (fp4: its 16 elements do); infinities take the largest value.
template <int FMT, int D, typename T>
PKV_DEVINL Quantised quantise(const Elems16<T>& in) {
    constexpr int L = QuantRow<FMT, D>::kLanes;
    float x[16];
    in.values(x);
    uint32_t own = in.top_bits();
    const bool nan = own > 0x7f800000u;
    if (__any_sync(0xffffffffu, nan)) {   // the others' largest, then
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(x[i]));
        own = __float_as_uint(m);
    }
    uint32_t top = own;
#pragma unroll
    for (int o = 1; o < L; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int e = row_exponent<FMT>(top);
    const float unit = pow2f(-e);
    Quantised r;
    r.exp = static_cast<uint32_t>(e + 127);
    r.scale = 0;
    if constexpr (FMT == PKV_FP8) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r.codes[i] = to_e4m3x4(x[4 * i] * unit, x[4 * i + 1] * unit, x[4 * i + 2] * unit,
                                   x[4 * i + 3] * unit);
    } else {
        const float a = fminf(__uint_as_float(own) * unit, 2688.f);
        // A sixth.  fp32: divided (a quotient rounds to a midpoint of e4m3 only where it is one: where a
        // is a unit off 6 m, a / 6 is off m by two thirds of a unit or more).  bf16: a product, since
        // values of eight digits on and next to 6 m are 2^-8 apart, and 6 m (1 / 6), off by 2^-25 of m
        // before it is rounded, rounds to m.
        const float sixth = sizeof(T) == 2 ? a * (1.f / 6.f) : __fdiv_rn(a, 6.f);
        r.scale = to_e4m3x2(sixth, 0.f) & 0xffu;
        const float s = f16lo_to_f32(e4m3x2_to_f16x2(r.scale));
        if (nan) r.scale = 0x7fu;
        // Multiplied by the scale's inverse and the row's unit, the border is met up to two units in
        // the last place.  In bf16 an element on a border and one next to it are 2^-8 apart, so
        // both are told apart on a grid of 2^-12 (1.5 2^11 + u), which has every border.  An fp32
        // element may lie closer: where one is within 2^-18 of the grid of the borders, 1 / 4, all
        // are divided (a quotient rounds to a border only where it is one: where y is a unit in its
        // last place off b s, y / s is off b by more than half of b's).
        const float f = s > 0.f ? unit * __fdiv_rn(1.f, s) : 0.f;
        float u[16];
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < 16; ++i) u[i] = __fadd_rn(__fmaf_rn(x[i], f, 0x1.8p11f), -0x1.8p11f);
        } else {
            float near = 1.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                u[i] = x[i] * f;
                const float grid = __fadd_rn(__fadd_rn(u[i], 0x1.8p21f), -0x1.8p21f);   // of 1 / 4
                near = fminf(near, fabsf(u[i] - grid));
            }
            if (__any_sync(0xffffffffu, near < 0x1p-18f)) {
#pragma unroll
                for (int i = 0; i < 16; ++i) u[i] = s > 0.f ? __fdiv_rn(x[i] * unit, s) : 0.f;
            }
        }
        r.codes[0] = plain_zeros(to_e2m1x8(u));
        r.codes[1] = plain_zeros(to_e2m1x8(u + 8));
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
