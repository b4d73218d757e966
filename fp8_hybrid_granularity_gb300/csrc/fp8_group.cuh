// FP8 groups quantized from FP32 values in registers: sixteen neighbouring
// elements a thread, eight threads a group of 128.
#pragma once
#include <cstdint>

#include "pair_math.cuh"
#include "quant_math.cuh"

namespace fp8hg {

// Sixteen code bytes (aligned) to p, the first `left` of them.
__device__ __forceinline__ void store_bytes16(uint8_t *p, const uint32_t (&c)[4], int left) {
    if (left >= 16) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(c[0], c[1], c[2], c[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < left) p[i] = static_cast<uint8_t>(c[i >> 2] >> (8 * (i & 3)));
    }
}

// Four values -> four FP8 codes.
template <int FMT>
__device__ __forceinline__ uint32_t cvt4(float a, float b, float c, float d) {
    return FMT == FMT_E4M3 ? ptx::cvt_e4m3x4(a, b, c, d) : ptx::cvt_e5m2x4(a, b, c, d);
}

// A group's scale, the power of two at or above amax / FMAX (FMAX = 1.75 2^emax),
// without a branch.  amax is the magnitude's bit pattern with MANT mantissa
// bits below the exponent, from max3_abs or max_abs_bf16x2: adding just under a
// quarter of the exponent's unit carries exactly if the mantissa is past 1.75.
// Zero and values below the range: byte 0.  Non-finite: 0xFF and a NaN
// multiplier, which casts to 0x7F.
template <int FMT, int MANT>
struct Group {
    uint32_t byte;
    float mul;       // 2^(127 - byte)
    __device__ __forceinline__ explicit Group(float amax) { init(__float_as_uint(amax)); }
    __device__ __forceinline__ explicit Group(uint32_t amax) { init(amax); }
    __device__ __forceinline__ void init(uint32_t amax) {
        constexpr int emax = (FMT == FMT_E4M3) ? 8 : 15;
        const int e = max(static_cast<int>((amax + (1u << (MANT - 2)) - 1u) >> MANT) - emax, 0);
        const bool nan = amax >= 0xFFu << MANT;
        byte = nan ? 0xFFu : static_cast<uint32_t>(e);
        mul = __uint_as_float(nan ? 0x7FC00000u : 0x7F000000u - (static_cast<uint32_t>(e) << 23));
    }
    __device__ __forceinline__ uint32_t cast4(F2 a, F2 b) const {
        const F2 m = f2(mul);
        a = mul2(a, m);
        b = mul2(b, m);
        return cvt4<FMT>(a.lo(), a.hi(), b.lo(), b.hi());
    }
};
template <int FMT>
using GroupF32 = Group<FMT, 23>;

// Maximum over the eight lanes of a group.
__device__ __forceinline__ float group_max(float m) {
    m = max3_abs(m, m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max3_abs(m, m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    return max3_abs(m, m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
}

}  // namespace fp8hg
