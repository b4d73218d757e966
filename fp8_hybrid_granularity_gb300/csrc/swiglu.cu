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

#include <algorithm>
#include <cstdint>

#include "lowbit.h"
#include "pair_math.cuh"
#include "quant_math.cuh"
#include "ragged.cuh"

namespace fp8hg {

namespace {

// 1 / (1 + 2^(-g log2 e)) of two values.
__device__ __forceinline__ F2 sigmoid2(F2 g) {
    const F2 x = mul2(g, f2(-1.44269504f));
    const F2 y = add2(f2(ex2_fast(x.lo()), ex2_fast(x.hi())), f2(1.0f));
    return f2(rcp_fast(y.lo()), rcp_fast(y.hi()));
}

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

// Two FP8 codes -> their values times m.
template <int FMT>
__device__ __forceinline__ F2 fp8x2_values(uint16_t c, F2 m) {
    float lo, hi;
    ptx::f16x2_to_f32(FMT == FMT_E4M3 ? ptx::cvt_f16x2_e4m3x2(c) : ptx::cvt_f16x2_e5m2x2(c), lo, hi);
    return mul2(f2(lo, hi), m);
}

// A scale byte's power of two; NaN for the byte of a non-finite group.
__device__ __forceinline__ float scale_pow2(uint32_t byte) {
    return byte == 0xFFu ? __uint_as_float(0x7FC00000u) : pow2f(static_cast<int>(byte) - 127);
}

// FP32 group scale (round-up rule); non-finite: byte 0xFF.
template <int FMT>
struct GroupF32 {
    uint32_t byte;
    float mul;       // 2^-e; a NaN for a non-finite group, which casts to 0x7F
    __device__ __forceinline__ explicit GroupF32(float amax) {
        const uint32_t bits = __float_as_uint(amax) & 0x7FFFFFFFu;
        const bool nan = bits >= 0x7F800000u;
        const int e = ue8m0_exponent_f32<FMT>(bits);
        byte = nan ? 0xFFu : static_cast<uint32_t>(e + 127);
        mul = nan ? __uint_as_float(0x7FC00000u) : pow2f(-e);
    }
    __device__ __forceinline__ uint32_t cast4(F2 a, F2 b) const {
        const F2 m = f2(mul);
        a = mul2(a, m);
        b = mul2(b, m);
        return __byte_perm(cvt2<FMT>(a.lo(), a.hi()), cvt2<FMT>(b.lo(), b.hi()), 0x5410);
    }
};

// Maximum over the eight lanes of a group (each half of a packed pair).
__device__ __forceinline__ uint32_t group_max_u2(uint32_t m) {
    m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    return __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
}
__device__ __forceinline__ float group_max(float m) {
    m = max3_abs(m, m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max3_abs(m, m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    return max3_abs(m, m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
}

// Sixteen BF16 values of a group with this amax -> codes; the scale byte.
template <int FMT>
__device__ __forceinline__ uint32_t cast_bf16x16(const uint32_t (&w)[8], uint32_t amax_bits, uint32_t (&c)[4]) {
    const GroupScale<FMT, SCALE_UE8M0> gs(amax_bits);
    const F2 m = f2(gs.nan ? __uint_as_float(0x7FC00000u) : gs.mul);   // a NaN casts to 0x7F
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const F2 a = mul2(f2_bf16(w[2 * i]), m), b = mul2(f2_bf16(w[2 * i + 1]), m);
        c[i] = __byte_perm(cvt2<FMT>(a.lo(), a.hi()), cvt2<FMT>(b.lo(), b.hi()), 0x5410);
    }
    return gs.byte;
}

// ------------------------------------------------------------------- forward
constexpr int kFwdThreadsPerSm = 768;   // 80 registers a thread

template <int FH, int FC, bool CKPT, bool WIDE>
__global__ void __launch_bounds__(256, kFwdThreadsPerSm / 256)
    k_swiglu_fwd(const SwigluFwdArgs a, int segs, int total_segs) {
    const int tid = threadIdx.x;
    const int seg = blockIdx.y * segs + tid % segs;
    const int rpb = blockDim.x / segs;
    const int64_t c0 = static_cast<int64_t>(seg) * 16, left = a.cols - c0;
    // the next row's loads are in flight while a row is computed
    const int64_t step = static_cast<int64_t>(gridDim.x) * rpb;
    const bool mine = tid / segs < rpb && seg < total_segs;
    uint32_t ng[8] = {0, 0, 0, 0, 0, 0, 0, 0}, nu[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    auto load = [&](int64_t r) {
        if (mine && r < a.rows && left > 0) {
            ragged::load16<WIDE>(a.gate + r * a.ld_in + c0, left, ng);
            ragged::load16<WIDE>(a.up + r * a.ld_in + c0, left, nu);
        }
    };
    load(static_cast<int64_t>(blockIdx.x) * rpb + tid / segs);
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * rpb; r0 < a.rows; r0 += step) {
        const int64_t r = r0 + tid / segs;
        const bool in = mine && r < a.rows;
        uint32_t g[8], u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = ng[i], u[i] = nu[i];
        load(r + step);
        F2 h[8];
        float mh = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const F2 x = f2_bf16(g[i]);
            h[i] = mul2(mul2(x, sigmoid2(x)), f2_bf16(u[i]));
            mh = max_abs(mh, h[i]);
        }
        mh = group_max(mh);
        uint32_t mgu = 0;
        if constexpr (CKPT) {
            // gate's maximum in the low half, up's in the high half
            uint32_t mg = 0, mu = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                mg = max_abs_bf16x2(mg, g[i]);
                mu = max_abs_bf16x2(mu, u[i]);
            }
            mgu = group_max_u2(max(mg & 0xFFFFu, mg >> 16) | (max(mu & 0xFFFFu, mu >> 16) << 16));
        }
        if (!in || left <= 0) continue;
        const GroupF32<FH> sh(mh);
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = sh.cast4(h[2 * i], h[2 * i + 1]);
        store_bytes16(a.h + r * a.ld_h + c0, c, left);
        const int64_t grp = seg >> 3;
        if ((seg & 7) == 0) a.hs[r * a.ld_hs + grp] = static_cast<uint8_t>(sh.byte);
        if constexpr (CKPT) {
            const uint32_t bg = cast_bf16x16<FC>(g, mgu & 0xFFFFu, c);
            store_bytes16(a.gq + r * a.ld_q + c0, c, left);
            const uint32_t bu = cast_bf16x16<FC>(u, mgu >> 16, c);
            store_bytes16(a.uq + r * a.ld_q + c0, c, left);
            if ((seg & 7) == 0) {
                a.gs[r * a.ld_s + grp] = static_cast<uint8_t>(bg);
                a.us[r * a.ld_s + grp] = static_cast<uint8_t>(bu);
            }
        }
    }
}

// ------------------------------------------------------------ backward, BF16
// Two elements' gradients from the checkpoint's values.
__device__ __forceinline__ void swiglu_grads(F2 g, F2 u, F2 dh, F2 &dg, F2 &du, F2 &h) {
    const F2 s = sigmoid2(g), gs = mul2(g, s);
    dg = mul2(mul2(dh, u), fma2(gs, fma2(s, f2(-1.0f), f2(1.0f)), s));
    du = mul2(dh, gs);
    h = mul2(gs, u);
}

template <int FC, bool WIDE>
__global__ void __launch_bounds__(256)
    k_swiglu_bwd(const uint16_t *__restrict__ dh, int64_t ld_dh, const SwigluCkpt c,
                 uint16_t *__restrict__ dg, uint16_t *__restrict__ du, int64_t ld_d, int segs) {
    // a warp takes 32 neighbouring segments of one row, whole warps past the
    // row's end included: the stores exchange values between lanes
    const int seg = (blockIdx.y * blockDim.x + threadIdx.x);
    const int64_t c0 = static_cast<int64_t>(seg) * 16, left = c.cols - c0;
    for (int64_t r = blockIdx.x; r < c.rows; r += gridDim.x) {
        uint32_t og[8] = {0, 0, 0, 0, 0, 0, 0, 0}, ou[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (seg < segs) {
            uint32_t w[8], gc[4], uc[4];
            ragged::load16<WIDE>(dh + r * ld_dh + c0, left, w);
            load_bytes16(c.gq + r * c.ld_q + c0, left, gc);
            load_bytes16(c.uq + r * c.ld_q + c0, left, uc);
            const F2 sg = f2(scale_pow2(__ldg(c.gs + r * c.ld_s + (seg >> 3))));
            const F2 su = f2(scale_pow2(__ldg(c.us + r * c.ld_s + (seg >> 3))));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int sh = 16 * (i & 1);
                const F2 g = fp8x2_values<FC>(static_cast<uint16_t>(gc[i >> 1] >> sh), sg);
                const F2 u = fp8x2_values<FC>(static_cast<uint16_t>(uc[i >> 1] >> sh), su);
                F2 a, b, h;
                swiglu_grads(g, u, f2_bf16(w[i]), a, b, h);
                og[i] = ptx::cvt_bf16x2(a.lo(), a.hi());
                ou[i] = ptx::cvt_bf16x2(b.lo(), b.hi());
            }
        }
        ragged::store16<WIDE>(dg + r * ld_d + c0, left, og);
        ragged::store16<WIDE>(du + r * ld_d + c0, left, ou);
    }
}

// ------------------------------------------------------------- backward, FP8
// Persistent, one CTA of 1024 threads per SM, a tile of 128 tokens x 128
// columns at a time: one group in each direction per row and column.
//   rows     a thread takes 16 columns of a row (eight lanes a row), computes
//            dg, du and h, quantizes dg and du along the row at once and leaves
//            all three in shared memory in FP32 (they have to be rounded once,
//            from FP32, in each direction);
//   columns  a thread takes 16 tokens of one column of each of the three
//            (eight lanes a column: 128 bytes of codes, a whole line).
// The next tile's inputs are loaded into registers before the column pass, so
// the loads run under it.
//
// Shared memory: value (r, c) at r * 128 + (r / 16) * 4 words plus c with its
// 16-byte piece index i replaced by i ^ ((i / 8) & 3): the eight lanes of a row
// write pieces in eight different bank groups, and the 4 columns x 8 row
// sixteenths that a warp reads at a time fall into 32 banks.
constexpr int kT = 128, Q_THREADS = 1024;
constexpr int kPlane = kT * kT + 8 * 4;          // words of one of the three
constexpr int kQSmem = 3 * kPlane * 4;

template <int F>
__device__ __forceinline__ void emit_codes(const F2 *v, int n4, const GroupF32<F> &gs, uint32_t *c) {
#pragma unroll
    for (int i = 0; i < n4; ++i) c[i] = gs.cast4(v[2 * i], v[2 * i + 1]);
}

// A thread's inputs of a tile: 16 columns of a row.
struct TileIn {
    uint32_t dh[8], g[4], u[4];
    uint32_t sg, su;
};

template <bool WIDE>
__device__ __forceinline__ void load_tile(TileIn &t, const uint16_t *dh, int64_t ld_dh, const SwigluCkpt &c,
                                          int64_t r, int64_t kb, int seg) {
    const int64_t col = kb * kT + seg * 16;
    if (WIDE) {
        ragged::load16<true>(dh + r * ld_dh + col, 16, t.dh);
    } else {
        const uint4 *p = reinterpret_cast<const uint4 *>(dh + r * ld_dh + col);
        const uint4 a = __ldg(p), b = __ldg(p + 1);
        t.dh[0] = a.x, t.dh[1] = a.y, t.dh[2] = a.z, t.dh[3] = a.w;
        t.dh[4] = b.x, t.dh[5] = b.y, t.dh[6] = b.z, t.dh[7] = b.w;
    }
    load_bytes16(c.gq + r * c.ld_q + col, 16, t.g);
    load_bytes16(c.uq + r * c.ld_q + col, 16, t.u);
    t.sg = __ldg(c.gs + r * c.ld_s + kb);
    t.su = __ldg(c.us + r * c.ld_s + kb);
}

template <int FC, int FR, int FT, int FH, bool WIDE>
__global__ void __launch_bounds__(Q_THREADS, 1)
    k_swiglu_bwd_q(const uint16_t *__restrict__ dh, int64_t ld_dh, const SwigluCkpt c, const SwigluGrads o,
                   int kbs, int tiles) {
    extern __shared__ __align__(16) float plane[];
    const int tid = threadIdx.x, seg = tid & 7, row = tid >> 3;
    TileIn in;
    int tile = blockIdx.x;
    if (tile < tiles) load_tile<WIDE>(in, dh, ld_dh, c, static_cast<int64_t>(tile / kbs) * kT + row, tile % kbs, seg);
    for (; tile < tiles; tile += gridDim.x) {
        const int64_t kb = tile % kbs, rb = tile / kbs, r0 = rb * kT;
        {
            const F2 sg = f2(scale_pow2(in.sg)), su = f2(scale_pow2(in.su));
            F2 a[8], b[8];
            float ma = 0.0f, mb = 0.0f;
            float *dst = plane + row * kT + (row >> 4) * 4;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                F2 h[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const F2 g = fp8x2_values<FC>(static_cast<uint16_t>(in.g[k] >> (16 * j)), sg);
                    const F2 u = fp8x2_values<FC>(static_cast<uint16_t>(in.u[k] >> (16 * j)), su);
                    swiglu_grads(g, u, f2_bf16(in.dh[2 * k + j]), a[2 * k + j], b[2 * k + j], h[j]);
                    ma = max_abs(ma, a[2 * k + j]);
                    mb = max_abs(mb, b[2 * k + j]);
                }
                const int piece = ((4 * seg + k) ^ ((seg >> 1) & 3)) * 4;
                *reinterpret_cast<ulonglong2 *>(dst + piece) = make_ulonglong2(a[2 * k].v, a[2 * k + 1].v);
                *reinterpret_cast<ulonglong2 *>(dst + kPlane + piece) = make_ulonglong2(b[2 * k].v, b[2 * k + 1].v);
                *reinterpret_cast<ulonglong2 *>(dst + 2 * kPlane + piece) = make_ulonglong2(h[0].v, h[1].v);
            }
            const GroupF32<FR> ga(group_max(ma)), gb(group_max(mb));
            const int64_t r = r0 + row, at = r * o.ld_q + kb * kT + seg * 16;
            uint32_t q[4];
            emit_codes<FR>(a, 4, ga, q);
            *reinterpret_cast<uint4 *>(o.q[0] + at) = make_uint4(q[0], q[1], q[2], q[3]);
            emit_codes<FR>(b, 4, gb, q);
            *reinterpret_cast<uint4 *>(o.q[1] + at) = make_uint4(q[0], q[1], q[2], q[3]);
            if (seg == 0) {
                o.s[0][r * o.ld_s + kb] = static_cast<uint8_t>(ga.byte);
                o.s[1][r * o.ld_s + kb] = static_cast<uint8_t>(gb.byte);
            }
        }
        __syncthreads();
        const int next = tile + gridDim.x;
        if (next < tiles)
            load_tile<WIDE>(in, dh, ld_dh, c, static_cast<int64_t>(next / kbs) * kT + row, next % kbs, seg);
        // column cc, tokens 16 part .. + 15
        const int part = tid & 7, cc = tid >> 3;
        const int word = (((cc >> 2) ^ ((cc >> 5) & 3)) << 2) + (cc & 3);
        const float *src = plane + part * (16 * kT + 4) + word;
#pragma unroll
        for (int w = 0; w < 3; ++w) {
            F2 v[8];
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = f2(src[w * kPlane + 2 * i * kT], src[w * kPlane + (2 * i + 1) * kT]);
                m = max_abs(m, v[i]);
            }
            m = group_max(m);
            uint32_t q[4], byte;
            if (w < 2) {
                const GroupF32<FT> gs(m);
                emit_codes<FT>(v, 4, gs, q);
                byte = gs.byte;
            } else {
                const GroupF32<FH> gs(m);
                emit_codes<FH>(v, 4, gs, q);
                byte = gs.byte;
            }
            const int64_t col = kb * kT + cc;
            *reinterpret_cast<uint4 *>(o.qt[w] + col * o.ld_qt + r0 + part * 16) = make_uint4(q[0], q[1], q[2], q[3]);
            if (part == 0) o.st[w][col * o.ld_st + rb] = static_cast<uint8_t>(byte);
        }
        __syncthreads();
    }
}

int sms() {
    static int n[64] = {0};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) dev = 0;
    if (!n[dev]) {
        int v = 0;
        cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
        n[dev] = v > 0 ? v : 1;
    }
    return n[dev];
}

template <int FH, int FC, bool CKPT>
cudaError_t fwd(const SwigluFwdArgs &a, cudaStream_t stream) {
    // segments of 16 columns, whole groups of eight; a chunk of at most 256
    // segments per block, spread evenly
    const int64_t total = (a.cols + 127) / 128 * 8, chunks = (total + 255) / 256;
    const int segs = static_cast<int>((total / 8 + chunks - 1) / chunks * 8);
    const int rpb = 256 / segs, threads = (segs * rpb + 31) / 32 * 32;
    const int64_t rb = (a.rows + rpb - 1) / rpb, cb = (total + segs - 1) / segs;
    // as many CTAs as fit at once
    const int64_t resident = std::max<int64_t>(1, sms() * static_cast<int64_t>(kFwdThreadsPerSm / threads) / cb);
    const dim3 grid(static_cast<unsigned>(std::min(rb, resident)), static_cast<unsigned>(cb));
    if (ragged::wide(a.gate, a.ld_in) && ragged::wide(a.up, a.ld_in))
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
    // a row's segments in equal blocks of whole warps
    const int64_t segs = (c.cols + 15) / 16, chunks = (segs + 255) / 256;
    const int threads = static_cast<int>(((segs + chunks - 1) / chunks + 31) / 32 * 32);
    const dim3 grid(static_cast<unsigned>(c.rows), static_cast<unsigned>((segs + threads - 1) / threads));
    const bool wide = ragged::wide(dh, ld_dh) && ragged::wide(dg, ld_d) && ragged::wide(du, ld_d);
    auto go = [&](auto kern) {
        kern<<<grid, threads, 0, stream>>>(dh, ld_dh, c, dg, du, ld_d, static_cast<int>(segs));
        return cudaGetLastError();
    };
    if (c.fmt == FMT_E4M3) return wide ? go(k_swiglu_bwd<FMT_E4M3, true>) : go(k_swiglu_bwd<FMT_E4M3, false>);
    return wide ? go(k_swiglu_bwd<FMT_E5M2, true>) : go(k_swiglu_bwd<FMT_E5M2, false>);
}

namespace {

template <int FC, int FR, int FT, int FH>
cudaError_t bwd_q(const uint16_t *dh, int64_t ld_dh, const SwigluCkpt &c, const SwigluGrads &g,
                  cudaStream_t stream) {
    const int64_t kbs = c.cols / kT, tiles = kbs * (c.rows / kT);
    if (tiles > 0x7FFFFFFF) return cudaErrorInvalidValue;
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (sms < 1) sms = 1;
    const unsigned grid = static_cast<unsigned>(tiles < sms ? tiles : sms);
    auto go = [&](auto kern) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kQSmem);
        if (e != cudaSuccess) return e;
        kern<<<grid, Q_THREADS, kQSmem, stream>>>(dh, ld_dh, c, g, static_cast<int>(kbs), static_cast<int>(tiles));
        return cudaGetLastError();
    };
    return ragged::wide(dh, ld_dh) ? go(k_swiglu_bwd_q<FC, FR, FT, FH, true>)
                                   : go(k_swiglu_bwd_q<FC, FR, FT, FH, false>);
}
template <int FC, int FR, int FT>
cudaError_t bwd_q_h(const uint16_t *dh, int64_t ld_dh, const SwigluCkpt &c, const SwigluGrads &g,
                    cudaStream_t stream) {
    return g.fmt_h == FMT_E4M3 ? bwd_q<FC, FR, FT, FMT_E4M3>(dh, ld_dh, c, g, stream)
                               : bwd_q<FC, FR, FT, FMT_E5M2>(dh, ld_dh, c, g, stream);
}
template <int FC, int FR>
cudaError_t bwd_q_t(const uint16_t *dh, int64_t ld_dh, const SwigluCkpt &c, const SwigluGrads &g,
                    cudaStream_t stream) {
    return g.fmt_t == FMT_E4M3 ? bwd_q_h<FC, FR, FMT_E4M3>(dh, ld_dh, c, g, stream)
                               : bwd_q_h<FC, FR, FMT_E5M2>(dh, ld_dh, c, g, stream);
}

}  // namespace

cudaError_t launch_swiglu_bwd_q(const uint16_t *dh, int64_t ld_dh, const SwigluCkpt &c, const SwigluGrads &g,
                                cudaStream_t stream) {
    if (c.fmt == FMT_E4M3)
        return g.fmt == FMT_E4M3 ? bwd_q_t<FMT_E4M3, FMT_E4M3>(dh, ld_dh, c, g, stream)
                                 : bwd_q_t<FMT_E4M3, FMT_E5M2>(dh, ld_dh, c, g, stream);
    return g.fmt == FMT_E4M3 ? bwd_q_t<FMT_E5M2, FMT_E4M3>(dh, ld_dh, c, g, stream)
                             : bwd_q_t<FMT_E5M2, FMT_E5M2>(dh, ld_dh, c, g, stream);
}

}  // namespace fp8hg
