// Block scales and casts of the 4-bit formats (E2M1 values).
//
// As in quant_math.cuh the amax of a block is an integer maximum over BF16
// patterns.  MX scales are read off its exponent field.  An NV scale is
// E4M3((amax / 6) / t), an element's quotient x / d with d = s * t.  All of
// these quotients are a product with an (approximate) reciprocal and one
// residual step, q + (x - q d) (1/d), two fused multiply-adds, which leaves the
// error of the quotient below one FP32 rounding.  With t a power of two d has
// four significant bits and x eight, so x / d either equals a midpoint of two
// E2M1 values or is farther from it than that error, and the cast is the
// nearest value of the exact quotient; the same holds for amax / 6 and E4M3.
// (A plain multiply by 1/d breaks such ties at random.)
#pragma once
#include <cstdint>

#include "pair_math.cuh"
#include "quant_math.cuh"

namespace fp8hg {

// Eight floats -> eight E2M1 codes (nearest even, saturating), the first in
// the low four bits.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Eight codes -> their values.
__device__ __forceinline__ void e2m1x8_values(uint32_t w, float (&v)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) ptx::f16x2_to_f32(h[i], v[2 * i], v[2 * i + 1]);
}

// A scale byte's value (NaN for the byte of a non-finite block).
template <bool NV>
__device__ __forceinline__ float fp4_scale_value(uint32_t byte) {
    if constexpr (NV) {
        float lo, hi;
        ptx::f16x2_to_f32(ptx::cvt_f16x2_e4m3x2(static_cast<uint16_t>(byte)), lo, hi);
        return lo;
    } else {
        return byte == 0xFFu ? __uint_as_float(0x7FC00000u) : pow2f(static_cast<int>(byte) - 127);
    }
}

// x / d from r = 1 / d (to a few units in the last place), see above.
__device__ __forceinline__ float quotient(float x, float d, float r) {
    const float q = __fmul_rn(x, r);
    return __fmaf_rn(__fmaf_rn(-q, d, x), r, q);
}

template <bool NV>
struct Fp4Scale {
    uint32_t byte;
    float mul;       // MX: 2^-e; NV: 1 / d
    float d;         // NV: s * t
    bool nan, sat;   // a non-finite block; NV: the E4M3 scale saturated
    // NV: t the tensor's scale, rt = 1 / t (MX: not used)
    __device__ __forceinline__ Fp4Scale(uint32_t amax_bits, float t, float rt) {
        nan = amax_bits >= 0x7F80u;
        sat = false;
        d = 0.0f;
        mul = 0.0f;
        if constexpr (NV) {
            // amax / 6 / t beyond 2^96 is taken as that: it saturates, and the
            // residual stays finite
            const float sixth = quotient(__uint_as_float(amax_bits << 16), 6.0f, 1.0f / 6.0f);
            const float q = fminf(__fmul_rn(sixth, rt), 0x1p96f);
            const float s = __fmaf_rn(__fmaf_rn(-q, t, sixth), rt, q);
            sat = s > 448.0f;
            byte = nan ? 0x7Fu : ptx::cvt_e4m3x2(s, 0.0f) & 0xFFu;
            d = __fmul_rn(fp4_scale_value<true>(byte), t);
            const bool none = nan || byte == 0u;
            d = none ? 0.0f : d;
            mul = none ? 0.0f : rcp_fast(d);
        } else {
            const int ef = static_cast<int>(amax_bits >> 7);
            const int e = ef == 0 ? -127 : clamp_exp(ef - 129);
            byte = nan ? 0xFFu : static_cast<uint32_t>(e + 127);
            if (!nan) mul = pow2f(-e);
        }
    }
    // Eight values -> eight codes.  Non-finite block: 0.  NV: the residual step
    // turns -0 into 0.
    __device__ __forceinline__ uint32_t cast8(F2 (&x)[4]) const {
        float v[8];
        const F2 m2 = f2(mul), nd2 = f2(-d);
        if (NV && sat) {   // keeps the quotients finite; all such values saturate
            const float m = 8.0f * d;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = f2(fminf(fmaxf(x[i].lo(), -m), m), fminf(fmaxf(x[i].hi(), -m), m));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (NV) {
                const F2 q = mul2(x[i], m2);
                x[i] = fma2(fma2(q, nd2, x[i]), m2, q);
            } else {
                x[i] = mul2(x[i], m2);
            }
            v[2 * i] = x[i].lo();
            v[2 * i + 1] = x[i].hi();
        }
        const uint32_t c = cvt_e2m1x8(v);
        return nan ? 0u : c;
    }
    // Eight BF16 values in four words.
    __device__ __forceinline__ uint32_t cast8(const uint32_t *w) const {
        F2 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = f2_bf16(w[i]);
        return cast8(x);
    }
    // The low (H = 0) or high halves of eight words.
    template <int H>
    __device__ __forceinline__ uint32_t cast8_half(const uint32_t *w) const {
        F2 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = H ? f2(__uint_as_float(w[2 * i] & 0xFFFF0000u), __uint_as_float(w[2 * i + 1] & 0xFFFF0000u))
                     : f2(__uint_as_float(w[2 * i] << 16), __uint_as_float(w[2 * i + 1] << 16));
        return cast8(x);
    }
};

// The tensor scale's reciprocal as Fp4Scale takes it.
template <bool NV>
__device__ __forceinline__ float fp4_reciprocal(float t) {
    return NV ? __frcp_rn(t) : 0.0f;
}

// Byte offset of (row, block j) in a scale array with `tiles` tiles along k.
__device__ __forceinline__ int64_t fp4_scale_offset(uint32_t row, uint32_t j, uint32_t tiles) {
    const uint32_t r = row & 127;
    const uint64_t tile = static_cast<uint64_t>(row >> 7) * tiles + (j >> 2);
    return static_cast<int64_t>(tile * 512 + (r & 31) * 16 + (r >> 5) * 4 + (j & 3));
}

}  // namespace fp8hg
