// Two FP32 values in one 64-bit register pair: the packed instructions do both
// in one issue slot, rounded like the single ones.  The kernels around them
// move 5 to 9 bytes per element, for which an SM has some 40 issue slots.
#pragma once
#include <cstdint>

namespace fp8hg {

struct F2 {
    uint64_t v;
    __device__ __forceinline__ float lo() const { return __uint_as_float(static_cast<uint32_t>(v)); }
    __device__ __forceinline__ float hi() const { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ F2 f2(float both) { return f2(both, both); }
// The two BF16 values of a word.
__device__ __forceinline__ F2 f2_bf16(uint32_t w) {
    return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
// The largest of three magnitudes, a NaN if one is (one instruction, where
// maxima of bit patterns take one for each sign bit and one for each maximum).
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float max_abs(float m, F2 v) { return max3_abs(m, v.lo(), v.hi()); }
// The largest magnitude of a warp, a NaN if one is.
__device__ __forceinline__ float warp_max_abs(float m) {
    float r;
    asm volatile("redux.sync.max.abs.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(m));
    return r;
}
// The larger magnitude in each half of two BF16 pairs (a NaN if one is); the
// sign bits are left over from the operands' (one instruction, where clearing
// them first takes two).
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t m, uint32_t w) {
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(w));
    return r;
}
// Both halves' magnitudes.
__device__ __forceinline__ uint32_t magnitudes(uint32_t m) { return m & 0x7FFF7FFFu; }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
// 2^x and 1 / x of the special-function unit (two units in the last place);
// results below the normal range are 0.
__device__ __forceinline__ float ex2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

}  // namespace fp8hg
