// SwiGLU with 8-bit activation checkpoints.
//
//   h = silu(g) u,  silu(g) = g s(g),  s(g) = 1 / (1 + exp(-g))
//   dg = dh u s (1 + g (1 - s)),  du = dh g s
//
// in FP32 between the loads and the casts.  Everything is bound by HBM:
// forward 4 bytes read and 3 written per element, backward 4 read and 4 (BF16)
// or 5 (FP8, both directions and h) written.
//
// exp and the quotient are the fast forms: their relative error (about 1e-6)
// is far below the 2^-4 and 2^-9 of the casts that follow, and s stays within
// [0, 1] (exp overflowing to infinity gives 0).
//
// A thread takes 16 neighbouring elements, eight threads a group of 128.
#include <cuda_runtime.h>

#include <cstdint>

#include "lowbit.h"
#include "quant_math.cuh"

namespace fp8hg {

namespace {

template <bool VEC>
__device__ __forceinline__ void load_bf16x16(const uint16_t *p, int64_t left, uint32_t (&w)[8]) {
    if (VEC && left >= 16) {
        const uint4 a = ptx::ld_stream_v4(p), b = ptx::ld_stream_v4(p + 8);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
        w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t lo = 2 * i < left ? __ldg(p + 2 * i) : 0u;
            const uint32_t hi = 2 * i + 1 < left ? __ldg(p + 2 * i + 1) : 0u;
            w[i] = lo | (hi << 16);
        }
    }
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

// Sixteen code bytes (aligned) to p, the first `left` of them.
__device__ __forceinline__ void store_bytes16(uint8_t *p, const uint32_t (&c)[4], int64_t left) {
    if (left >= 16) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(c[0], c[1], c[2], c[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < left) p[i] = static_cast<uint8_t>(c[i >> 2] >> (8 * (i & 3)));
    }
}

__device__ __forceinline__ void load_bytes16(const uint8_t *p, int64_t left, uint32_t (&c)[4]) {
    if (left >= 16) {
        const uint4 v = ptx::ld_stream_v4(p);
        c[0] = v.x, c[1] = v.y, c[2] = v.z, c[3] = v.w;
    } else {
        c[0] = c[1] = c[2] = c[3] = 0u;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < left) c[i >> 2] |= static_cast<uint32_t>(__ldg(p + i)) << (8 * (i & 3));
    }
}

// Four FP8 codes -> floats.
template <int FMT>
__device__ __forceinline__ void fp8x4_values(uint32_t c, float (&v)[4]) {
    const uint16_t lo = static_cast<uint16_t>(c), hi = static_cast<uint16_t>(c >> 16);
    if constexpr (FMT == FMT_E4M3) {
        ptx::f16x2_to_f32(ptx::cvt_f16x2_e4m3x2(lo), v[0], v[1]);
        ptx::f16x2_to_f32(ptx::cvt_f16x2_e4m3x2(hi), v[2], v[3]);
    } else {
        ptx::f16x2_to_f32(ptx::cvt_f16x2_e5m2x2(lo), v[0], v[1]);
        ptx::f16x2_to_f32(ptx::cvt_f16x2_e5m2x2(hi), v[2], v[3]);
    }
}

// A scale byte's power of two; NaN for the byte of a non-finite group.
__device__ __forceinline__ float scale_pow2(uint32_t byte) {
    return byte == 0xFFu ? __uint_as_float(0x7FC00000u) : pow2f(static_cast<int>(byte) - 127);
}

// FP32 group scale (round-up rule); non-finite: byte 0xFF.
template <int FMT>
struct GroupF32 {
    uint32_t byte;
    float mul;
    bool nan;
    __device__ __forceinline__ explicit GroupF32(uint32_t amax_bits) {
        nan = amax_bits >= 0x7F800000u;
        const int e = ue8m0_exponent_f32<FMT>(amax_bits);
        byte = nan ? 0xFFu : static_cast<uint32_t>(e + 127);
        mul = pow2f(-e);
    }
    __device__ __forceinline__ uint32_t cast4(float a, float b, float c, float d) const {
        const uint32_t v = cvt2<FMT>(a * mul, b * mul) | (cvt2<FMT>(c * mul, d * mul) << 16);
        return nan ? kNanCodes : v;
    }
};

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Maximum over the eight lanes of a group (each half of a packed pair).
__device__ __forceinline__ uint32_t group_max_u2(uint32_t m) {
    m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    return __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
}
__device__ __forceinline__ uint32_t group_max(uint32_t m) {
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    return max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
}

template <int FMT>
__device__ __forceinline__ void cast_bf16x16(const uint32_t (&w)[8], const GroupScale<FMT, SCALE_UE8M0> &gs,
                                             uint32_t (&c)[4]) {
    uint32_t unused = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint2 v = quant8<FMT, false>(make_uint4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]),
                                           gs.mul, unused);
        c[2 * h] = gs.nan ? kNanCodes : v.x;
        c[2 * h + 1] = gs.nan ? kNanCodes : v.y;
    }
}

// ------------------------------------------------------------------- forward
template <int FH, int FC, bool CKPT, bool VEC>
__global__ void __launch_bounds__(256)
    k_swiglu_fwd(const SwigluFwdArgs a, int segs, int total_segs) {
    const int tid = threadIdx.x;
    const int seg = blockIdx.y * segs + tid % segs;
    const int rpb = blockDim.x / segs;
    const int64_t c0 = static_cast<int64_t>(seg) * 16, left = a.cols - c0;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * rpb; r0 < a.rows;
         r0 += static_cast<int64_t>(gridDim.x) * rpb) {
        const int64_t r = r0 + tid / segs;
        const bool in = tid / segs < rpb && r < a.rows && seg < total_segs;
        uint32_t g[8] = {0, 0, 0, 0, 0, 0, 0, 0}, u[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (in && left > 0) {
            load_bf16x16<VEC>(a.gate + r * a.ld_in + c0, left, g);
            load_bf16x16<VEC>(a.up + r * a.ld_in + c0, left, u);
        }
        float h[16];
        uint32_t mh = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            h[2 * i] = bf_lo(g[i]) * sigmoid(bf_lo(g[i])) * bf_lo(u[i]);
            h[2 * i + 1] = bf_hi(g[i]) * sigmoid(bf_hi(g[i])) * bf_hi(u[i]);
            mh = max(mh, max(abs_bits(h[2 * i]), abs_bits(h[2 * i + 1])));
        }
        mh = group_max(mh);
        uint32_t mgu = 0;
        if constexpr (CKPT) {
            // gate's maximum in the low half, up's in the high half
            uint32_t mg = 0, mu = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                mg = __vmaxu2(mg, g[i] & 0x7FFF7FFFu);
                mu = __vmaxu2(mu, u[i] & 0x7FFF7FFFu);
            }
            mgu = group_max_u2(max(mg & 0xFFFFu, mg >> 16) | (max(mu & 0xFFFFu, mu >> 16) << 16));
        }
        if (!in || left <= 0) continue;
        const GroupF32<FH> sh(mh);
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = sh.cast4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
        store_bytes16(a.h + r * a.ld_h + c0, c, left);
        const int64_t grp = seg >> 3;
        if ((seg & 7) == 0) a.hs[r * a.ld_hs + grp] = static_cast<uint8_t>(sh.byte);
        if constexpr (CKPT) {
            const GroupScale<FC, SCALE_UE8M0> sg(mgu & 0xFFFFu), su(mgu >> 16);
            cast_bf16x16<FC>(g, sg, c);
            store_bytes16(a.gq + r * a.ld_q + c0, c, left);
            cast_bf16x16<FC>(u, su, c);
            store_bytes16(a.uq + r * a.ld_q + c0, c, left);
            if ((seg & 7) == 0) {
                a.gs[r * a.ld_s + grp] = static_cast<uint8_t>(sg.byte);
                a.us[r * a.ld_s + grp] = static_cast<uint8_t>(su.byte);
            }
        }
    }
}

// ------------------------------------------------------------ backward, BF16
// One element's gradients from the checkpoint's values.
__device__ __forceinline__ void swiglu_grads(float g, float u, float dh, float &dg, float &du,
                                             float &h) {
    const float s = sigmoid(g), gs = g * s;
    dg = dh * u * (s + gs * (1.0f - s));
    du = dh * gs;
    h = gs * u;
}

template <int FC, bool VEC>
__global__ void __launch_bounds__(256)
    k_swiglu_bwd(const uint16_t *__restrict__ dh, int64_t ld_dh, const SwigluCkpt c,
                 uint16_t *__restrict__ dg, uint16_t *__restrict__ du, int64_t ld_d, int64_t segs) {
    for (int64_t r = blockIdx.x; r < c.rows; r += gridDim.x) {
        for (int64_t seg = blockIdx.y * static_cast<int64_t>(blockDim.x) + threadIdx.x; seg < segs;
             seg += static_cast<int64_t>(gridDim.y) * blockDim.x) {
            const int64_t c0 = seg * 16, left = c.cols - c0;
            uint32_t w[8], gc[4], uc[4];
            load_bf16x16<VEC>(dh + r * ld_dh + c0, left, w);
            load_bytes16(c.gq + r * c.ld_q + c0, left, gc);
            load_bytes16(c.uq + r * c.ld_q + c0, left, uc);
            const float sg = scale_pow2(__ldg(c.gs + r * c.ld_s + (seg >> 3)));
            const float su = scale_pow2(__ldg(c.us + r * c.ld_s + (seg >> 3)));
            uint32_t og[8], ou[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float g[4], u[4], a[4], b[4], h;
                fp8x4_values<FC>(gc[i], g);
                fp8x4_values<FC>(uc[i], u);
                const float d[4] = {bf_lo(w[2 * i]), bf_hi(w[2 * i]), bf_lo(w[2 * i + 1]),
                                    bf_hi(w[2 * i + 1])};
#pragma unroll
                for (int j = 0; j < 4; ++j) swiglu_grads(g[j] * sg, u[j] * su, d[j], a[j], b[j], h);
                og[2 * i] = ptx::cvt_bf16x2(a[0], a[1]);
                og[2 * i + 1] = ptx::cvt_bf16x2(a[2], a[3]);
                ou[2 * i] = ptx::cvt_bf16x2(b[0], b[1]);
                ou[2 * i + 1] = ptx::cvt_bf16x2(b[2], b[3]);
            }
            uint16_t *pg = dg + r * ld_d + c0, *pu = du + r * ld_d + c0;
            if (VEC && left >= 16) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    reinterpret_cast<uint4 *>(pg)[i] =
                        make_uint4(og[4 * i], og[4 * i + 1], og[4 * i + 2], og[4 * i + 3]);
                    reinterpret_cast<uint4 *>(pu)[i] =
                        make_uint4(ou[4 * i], ou[4 * i + 1], ou[4 * i + 2], ou[4 * i + 3]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (i < left) {
                        pg[i] = static_cast<uint16_t>(og[i >> 1] >> (16 * (i & 1)));
                        pu[i] = static_cast<uint16_t>(ou[i >> 1] >> (16 * (i & 1)));
                    }
            }
        }
    }
}

// ------------------------------------------------------------- backward, FP8
// A CTA takes a tile of 128 tokens x 128 columns, one group in each direction
// per row and column, and computes dg, du and h one after the other into
// shared memory.
constexpr int kT = 128, kPitch = 129;

template <int F>
__device__ __forceinline__ void emit_group16(const float (&v)[16], uint32_t m, uint8_t *q,
                                             uint8_t *s, bool first) {
    const GroupF32<F> gs(m);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = gs.cast4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    *reinterpret_cast<uint4 *>(q) = make_uint4(c[0], c[1], c[2], c[3]);
    if (first) *s = static_cast<uint8_t>(gs.byte);
}
__device__ __forceinline__ void emit_group16(int fmt, const float (&v)[16], uint32_t m, uint8_t *q,
                                             uint8_t *s, bool first) {
    if (fmt == FMT_E4M3) emit_group16<FMT_E4M3>(v, m, q, s, first);
    else emit_group16<FMT_E5M2>(v, m, q, s, first);
}

template <int FC>
__global__ void __launch_bounds__(256)
    k_swiglu_bwd_q(const uint16_t *__restrict__ dh, int64_t ld_dh, const SwigluCkpt c,
                   const SwigluGrads o) {
    extern __shared__ float tile[];
    const int tid = threadIdx.x, seg = tid & 7;
    const int64_t k0 = static_cast<int64_t>(blockIdx.x) * kT, r0 = static_cast<int64_t>(blockIdx.y) * kT;
    for (int which = 0; which < 3; ++which) {
        const int fmt_t = which == 2 ? o.fmt_h : o.fmt_t;
        for (int rr = tid >> 3; rr < kT; rr += 32) {
            const int64_t r = r0 + rr, col = k0 + seg * 16;
            uint32_t w[8], gc[4], uc[4];
            load_bf16x16<true>(dh + r * ld_dh + col, 16, w);
            load_bytes16(c.gq + r * c.ld_q + col, 16, gc);
            load_bytes16(c.uq + r * c.ld_q + col, 16, uc);
            const float sg = scale_pow2(__ldg(c.gs + r * c.ld_s + blockIdx.x));
            const float su = scale_pow2(__ldg(c.us + r * c.ld_s + blockIdx.x));
            float v[16];
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float g[4], u[4];
                fp8x4_values<FC>(gc[i], g);
                fp8x4_values<FC>(uc[i], u);
                const float d[4] = {bf_lo(w[2 * i]), bf_hi(w[2 * i]), bf_lo(w[2 * i + 1]),
                                    bf_hi(w[2 * i + 1])};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float a, b, h;
                    swiglu_grads(g[j] * sg, u[j] * su, d[j], a, b, h);
                    const float x = which == 0 ? a : which == 1 ? b : h;
                    v[4 * i + j] = x;
                    tile[rr * kPitch + seg * 16 + 4 * i + j] = x;
                    m = max(m, abs_bits(x));
                }
            }
            if (which < 2) {
                m = group_max(m);
                emit_group16(o.fmt, v, m, o.q[which] + r * o.ld_q + col,
                             o.s[which] + r * o.ld_s + blockIdx.x, seg == 0);
            }
        }
        __syncthreads();
        for (int cc = tid >> 3; cc < kT; cc += 32) {
            float v[16];
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                v[i] = tile[(seg * 16 + i) * kPitch + cc];
                m = max(m, abs_bits(v[i]));
            }
            m = group_max(m);
            emit_group16(fmt_t, v, m, o.qt[which] + (k0 + cc) * o.ld_qt + r0 + seg * 16,
                         o.st[which] + (k0 + cc) * o.ld_st + blockIdx.y, seg == 0);
        }
        __syncthreads();
    }
}

bool vec16(const void *p, int64_t ld) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0;
}

template <int FH, int FC, bool CKPT>
cudaError_t fwd(const SwigluFwdArgs &a, cudaStream_t stream) {
    // segments of 16 columns, whole groups of eight; a chunk of at most 256
    // segments per block, spread evenly
    const int64_t total = (a.cols + 127) / 128 * 8, chunks = (total + 255) / 256;
    const int segs = static_cast<int>((total / 8 + chunks - 1) / chunks * 8);
    const int rpb = 256 / segs, threads = (segs * rpb + 31) / 32 * 32;
    const int64_t rb = (a.rows + rpb - 1) / rpb;
    const dim3 grid(static_cast<unsigned>(rb < 0x7FFFFFFF ? rb : 0x7FFFFFFF),
                    static_cast<unsigned>((total + segs - 1) / segs));
    if (vec16(a.gate, a.ld_in) && vec16(a.up, a.ld_in))
        k_swiglu_fwd<FH, FC, CKPT, true><<<grid, threads, 0, stream>>>(a, segs, static_cast<int>(total));
    else
        k_swiglu_fwd<FH, FC, CKPT, false><<<grid, threads, 0, stream>>>(a, segs, static_cast<int>(total));
    return cudaGetLastError();
}

template <int FH>
cudaError_t fwd_h(const SwigluFwdArgs &a, cudaStream_t stream) {
    if (!a.gq) return fwd<FH, FMT_E4M3, false>(a, stream);
    return a.fmt == FMT_E4M3 ? fwd<FH, FMT_E4M3, true>(a, stream) : fwd<FH, FMT_E5M2, true>(a, stream);
}

}  // namespace

cudaError_t launch_swiglu_fwd(const SwigluFwdArgs &a, cudaStream_t stream) {
    return a.fmt_h == FMT_E4M3 ? fwd_h<FMT_E4M3>(a, stream) : fwd_h<FMT_E5M2>(a, stream);
}

cudaError_t launch_swiglu_bwd(const uint16_t *dh, int64_t ld_dh, const SwigluCkpt &c, uint16_t *dg,
                              uint16_t *du, int64_t ld_d, cudaStream_t stream) {
    const int64_t segs = (c.cols + 15) / 16;
    const int threads = segs < 256 ? static_cast<int>((segs + 31) / 32 * 32) : 256;
    const int64_t cb = (segs + threads - 1) / threads;
    const dim3 grid(static_cast<unsigned>(c.rows < 0x7FFFFFFF ? c.rows : 0x7FFFFFFF),
                    static_cast<unsigned>(cb < 65535 ? cb : 65535));
    const bool vec = vec16(dh, ld_dh) && vec16(dg, ld_d) && vec16(du, ld_d);
    auto go = [&](auto kern) {
        kern<<<grid, threads, 0, stream>>>(dh, ld_dh, c, dg, du, ld_d, segs);
        return cudaGetLastError();
    };
    if (c.fmt == FMT_E4M3) return vec ? go(k_swiglu_bwd<FMT_E4M3, true>) : go(k_swiglu_bwd<FMT_E4M3, false>);
    return vec ? go(k_swiglu_bwd<FMT_E5M2, true>) : go(k_swiglu_bwd<FMT_E5M2, false>);
}

cudaError_t launch_swiglu_bwd_q(const uint16_t *dh, int64_t ld_dh, const SwigluCkpt &c,
                                const SwigluGrads &g, cudaStream_t stream) {
    constexpr int smem = kT * kPitch * 4;
    const dim3 grid(static_cast<unsigned>(c.cols / kT), static_cast<unsigned>(c.rows / kT));
    auto go = [&](auto kern) {
        const cudaError_t e =
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        kern<<<grid, 256, smem, stream>>>(dh, ld_dh, c, g);
        return cudaGetLastError();
    };
    return c.fmt == FMT_E4M3 ? go(k_swiglu_bwd_q<FMT_E4M3>) : go(k_swiglu_bwd_q<FMT_E5M2>);
}

}  // namespace fp8hg
