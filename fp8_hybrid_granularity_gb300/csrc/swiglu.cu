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
// [0, 1].  Below FP32's normal range, 2^-126 (g < -87.3), s is taken as 0.
//
// A thread takes 16 neighbouring elements, eight threads a group of 128.
// In us and of the measured copy rate:
//                          8192 x 8960    16384 x 18944
//   forward                 82 (93 %)       341 (95 %)
//   without checkpoints     56 (98 %)       234 (98 %)
//   backward, BF16          84 (104 %)      349 (106 %)
//   backward, FP8          137 (72 %)       572 (72 %)
// At 8192 x 5003, where rows begin at odd addresses, the forward reaches 73 %: a lane
// loads up to three 16-byte pieces each of gate and up for its 32 bytes and shifts
// them into place.  The BF16 backward reaches 77 %: its stores also exchange pieces
// between lanes.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fp8_group.cuh"
#include "lowbit.h"
#include "ragged.cuh"

namespace fp8hg {

namespace {

// 1 / (1 + 2^(-g log2 e)) of two values.
__device__ __forceinline__ F2 sigmoid2(F2 g) {
    const F2 x = mul2(g, f2(-1.44269504f));
    const F2 y = add2(f2(ex2_fast(x.lo()), ex2_fast(x.hi())), f2(1.0f));
    return f2(rcp_fast(y.lo()), rcp_fast(y.hi()));
}

__device__ __forceinline__ void load_bytes16(const uint8_t *p, int left, uint32_t (&c)[4]) {
    if (left >= 16) {
        const uint4 v = ptx::ld_once_v4(p);
        c[0] = v.x, c[1] = v.y, c[2] = v.z, c[3] = v.w;
    } else {
        c[0] = c[1] = c[2] = c[3] = 0u;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < left) c[i >> 2] |= ptx::ld_u8(p + i) << (8 * (i & 3));
    }
}

// Four FP8 codes -> their values times m.
template <int FMT>
__device__ __forceinline__ void fp8x4_values(uint32_t c, F2 m, F2 (&v)[2]) {
    uint32_t h[2];
    if constexpr (FMT == FMT_E4M3) ptx::cvt_f16x4_e4m3x4(c, h[0], h[1]);
    else ptx::cvt_f16x4_e5m2x4(c, h[0], h[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float lo, hi;
        ptx::f16x2_to_f32(h[i], lo, hi);
        v[i] = mul2(f2(lo, hi), m);
    }
}

// A scale byte's power of two (2^-127, a subnormal, for 0); NaN for the byte of
// a non-finite group.
__device__ __forceinline__ float scale_pow2(uint32_t byte) {
    return __uint_as_float((byte << 23) | (byte == 0u || byte == 0xFFu ? 0x400000u : 0u));
}

// Maximum over the eight lanes of a group, each half of a packed pair.
__device__ __forceinline__ uint32_t group_max_u2(uint32_t m) {
    m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    return __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
}

// Sixteen BF16 values of a group with this amax -> codes; the scale byte.
template <int FMT>
__device__ __forceinline__ uint32_t cast_bf16x16(const uint32_t (&w)[8], uint32_t amax_bits, uint32_t (&c)[4]) {
    const Group<FMT, 7> gs(amax_bits);
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = gs.cast4(f2_bf16(w[2 * i]), f2_bf16(w[2 * i + 1]));
    return gs.byte;
}

// ------------------------------------------------------------------- forward
constexpr int kFwdThreadsPerSm = 768;   // 76 registers a thread

template <int FH, int FC, bool CKPT, bool WIDE>
__global__ void __launch_bounds__(256, kFwdThreadsPerSm / 256)
    k_swiglu_fwd(const SwigluFwdArgs a, int segs, int total_segs) {
    ptx::grid_begin(static_cast<int64_t>(a.rows) * a.cols);
    const int tid = threadIdx.x;
    const int seg = column_chunk() * segs + tid % segs;
    const int rpb = blockDim.x / segs;
    const int c0 = seg * 16, left = a.cols - c0;
    // the next row's loads are in flight while a row is computed
    const uint32_t step = gridDim.x * rpb;
    const bool mine = tid / segs < rpb && seg < total_segs;
    uint32_t ng[8] = {0, 0, 0, 0, 0, 0, 0, 0}, nu[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const uint32_t rows = a.rows;
    auto load = [&](uint32_t r) {
        if (mine && r < rows && left > 0) {
            const int64_t at = row_at(r, a.ld_in) + c0;
            ragged::load16<WIDE>(a.gate + at, left, ng);
            ragged::load16<WIDE>(a.up + at, left, nu);
        }
    };
    load(blockIdx.x * rpb + tid / segs);
    for (uint32_t r0 = blockIdx.x * rpb; r0 < rows; r0 += step) {
        const uint32_t r = r0 + tid / segs;
        const bool in = mine && r < rows;
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
            mg = magnitudes(mg), mu = magnitudes(mu);
            mgu = group_max_u2(max(mg & 0xFFFFu, mg >> 16) | (max(mu & 0xFFFFu, mu >> 16) << 16));
        }
        if (!in || left <= 0) continue;
        const GroupF32<FH> sh(mh);
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = sh.cast4(h[2 * i], h[2 * i + 1]);
        store_bytes16(a.h + row_at(r, a.ld_h) + c0, c, left);
        const int grp = seg >> 3;
        if ((seg & 7) == 0) a.hs[row_at(r, a.ld_hs) + grp] = static_cast<uint8_t>(sh.byte);
        if constexpr (CKPT) {
            const int64_t at = row_at(r, a.ld_q) + c0;
            const uint32_t bg = cast_bf16x16<FC>(g, mgu & 0xFFFFu, c);
            store_bytes16(a.gq + at, c, left);
            const uint32_t bu = cast_bf16x16<FC>(u, mgu >> 16, c);
            store_bytes16(a.uq + at, c, left);
            if ((seg & 7) == 0) {
                const int64_t to = row_at(r, a.ld_s) + grp;
                a.gs[to] = static_cast<uint8_t>(bg);
                a.us[to] = static_cast<uint8_t>(bu);
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
    k_swiglu_bwd(const uint16_t *dh, uint32_t ld_dh, const SwigluCkpt c,
                 uint16_t *dg, uint16_t *du, uint32_t ld_d, int segs) {
    ptx::grid_begin(static_cast<int64_t>(c.rows) * c.cols);
    // a warp takes 32 neighbouring segments of one row, whole warps past the
    // row's end included: the stores exchange values between lanes
    const int seg = (blockIdx.x * blockDim.x + threadIdx.x);
    const int c0 = seg * 16, left = c.cols - c0;
    for (uint32_t r = blockIdx.y; r < static_cast<uint32_t>(c.rows); r += gridDim.y) {
        uint32_t og[8] = {0, 0, 0, 0, 0, 0, 0, 0}, ou[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (seg < segs) {
            uint32_t w[8], gc[4], uc[4];
            const int64_t at = row_at(r, c.ld_q) + c0, sat = row_at(r, c.ld_s) + (seg >> 3);
            ragged::load16<WIDE>(dh + row_at(r, ld_dh) + c0, left, w);
            load_bytes16(c.gq + at, left, gc);
            load_bytes16(c.uq + at, left, uc);
            const F2 sg = f2(scale_pow2(ptx::ld_u8(c.gs + sat)));
            const F2 su = f2(scale_pow2(ptx::ld_u8(c.us + sat)));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                F2 g[2], u[2];
                fp8x4_values<FC>(gc[k], sg, g);
                fp8x4_values<FC>(uc[k], su, u);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    F2 a, b, h;
                    swiglu_grads(g[j], u[j], f2_bf16(w[2 * k + j]), a, b, h);
                    og[2 * k + j] = ptx::cvt_bf16x2(a.lo(), a.hi());
                    ou[2 * k + j] = ptx::cvt_bf16x2(b.lo(), b.hi());
                }
            }
        }
        ragged::store16<WIDE>(dg + row_at(r, ld_d) + c0, left, og);
        ragged::store16<WIDE>(du + row_at(r, ld_d) + c0, left, ou);
    }
}

// ------------------------------------------------------------- backward, FP8
// Persistent, one CTA of 1024 threads per SM, a tile of 128 tokens x 128
// columns at a time: one group in each direction per row and column.
//   rows     a thread takes 16 columns of a row (eight lanes a row), computes
//            dg, du and h, quantizes dg and du along the row at once and leaves
//            all three in shared memory, a plane each, in FP32 (they are
//            rounded once, from FP32, in each direction);
//   columns  a warp takes four columns of each plane, a lane four tokens: one
//            128-bit load per token, a column's maximum in one warp reduction,
//            its 128 code bytes in one store.
// Planes are handed over one by one: a warp waits only for the plane that it is
// about to write or read (six mbarriers, every warp arrives once a tile), h
// first, which the row part has ready before the row maxima of dg and du.  So
// warps drift apart by most of a part and the arithmetic of one overlaps the
// shared-memory work of the other; with a barrier of the CTA between the parts
// 8192 x 8960 takes 162 us instead of 139.  The next tile is prefetched to L2
// while this one's rows are computed and loaded to registers under the columns
// (without the prefetch 150 us; HBM alone would take 98).  At the 64 registers that
// 1024 threads leave, 28 bytes a thread are spilled.
constexpr int kT = 128, Q_THREADS = 1024;
constexpr int kPlane = kT * kT;                  // words of one of the three
constexpr int kQSmem = 3 * kPlane * 4;

template <int F>
__device__ __forceinline__ void emit_codes(const F2 *v, int n4, const GroupF32<F> &gs, uint32_t *c) {
#pragma unroll
    for (int i = 0; i < n4; ++i) c[i] = gs.cast4(v[2 * i], v[2 * i + 1]);
}

// Where a row's piece p (columns 4 p .. + 3) stands in shared memory.  Both
// the writing lanes (pieces 4 seg + k of a row) and the reading ones (piece p
// of every fourth row) fall on eight different 16-byte banks.
__device__ __forceinline__ int plane_piece(int p, int row) { return p ^ ((p >> 3) & 3) ^ ((row >> 2) & 7); }

// Four columns' groups of 128 tokens, four tokens per lane: scales (the column
// lane & 3 in each lane), codes and the first four lanes' scale bytes.
template <int FMT>
__device__ __forceinline__ void emit_columns(const F2 (&v)[4][2], int lane, uint8_t *q, uint32_t ld, uint8_t *s) {
    float m[4];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        m[2 * c] = warp_max_abs(max3_abs(max3_abs(v[0][c].lo(), v[1][c].lo(), v[2][c].lo()), v[3][c].lo(), 0.0f));
        m[2 * c + 1] = warp_max_abs(max3_abs(max3_abs(v[0][c].hi(), v[1][c].hi(), v[2][c].hi()), v[3][c].hi(), 0.0f));
    }
    const GroupF32<FMT> gs(lane & 2 ? (lane & 1 ? m[3] : m[2]) : (lane & 1 ? m[1] : m[0]));
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const F2 mul = f2(__shfl_sync(0xFFFFFFFFu, gs.mul, 2 * c), __shfl_sync(0xFFFFFFFFu, gs.mul, 2 * c + 1));
        F2 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = mul2(v[i][c], mul);
        *reinterpret_cast<uint32_t *>(q) = cvt4<FMT>(x[0].lo(), x[1].lo(), x[2].lo(), x[3].lo());
        *reinterpret_cast<uint32_t *>(q + ld) = cvt4<FMT>(x[0].hi(), x[1].hi(), x[2].hi(), x[3].hi());
        q += 2 * static_cast<int64_t>(ld);
    }
    if (lane < 4) *s = static_cast<uint8_t>(gs.byte);
}

// A thread's inputs of a tile: 16 columns of a row.
struct TileIn {
    uint32_t dh[8], g[4], u[4];
    uint32_t sg, su;
};

template <bool WIDE>
__device__ __forceinline__ void load_tile(TileIn &t, const uint16_t *dh, uint32_t ld_dh, const SwigluCkpt &c,
                                          uint32_t r, uint32_t kb, int seg) {
    const uint32_t col = kb * kT + seg * 16;
    const uint16_t *src = dh + row_at(r, ld_dh) + col;
    if (WIDE) {
        ragged::load16<true>(src, 16, t.dh);
    } else {
        const uint4 *p = reinterpret_cast<const uint4 *>(src);
        const uint4 a = ptx::ld_v4(p), b = ptx::ld_v4(p + 1);
        t.dh[0] = a.x, t.dh[1] = a.y, t.dh[2] = a.z, t.dh[3] = a.w;
        t.dh[4] = b.x, t.dh[5] = b.y, t.dh[6] = b.z, t.dh[7] = b.w;
    }
    const int64_t at = row_at(r, c.ld_q) + col, sat = row_at(r, c.ld_s) + kb;
    load_bytes16(c.gq + at, 16, t.g);
    load_bytes16(c.uq + at, 16, t.u);
    t.sg = ptx::ld_u8(c.gs + sat);
    t.su = ptx::ld_u8(c.us + sat);
}

// The limit of one wait: 2 s.
constexpr uint32_t kWaitNs = 2000000000u;

template <int FC, int FR, int FT, int FH, bool WIDE>
__global__ void __launch_bounds__(Q_THREADS, 1)
    k_swiglu_bwd_q(const uint16_t *dh, uint32_t ld_dh, const SwigluCkpt c, const SwigluGrads o,
                   uint32_t kbs, uint32_t rbs, uint32_t step_k, uint32_t step_r, unsigned int *err) {
    extern __shared__ __align__(16) float plane[];
    __shared__ __align__(8) uint64_t bars[6];
    const uint32_t bar = ptx::smem_u32(bars);
    uint32_t phase = 0;
    auto full = [&](int p) { return bar + 8 * p; };
    auto empty = [&](int p) { return bar + 24 + 8 * p; };
    const int tid = threadIdx.x, seg = tid & 7, row = tid >> 3, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
#pragma unroll
        for (int i = 0; i < 6; ++i) ptx::mbar_init(bar + 8 * i, Q_THREADS / 32);
        ptx::fence_mbar_init();
    }
    __syncthreads();
    ptx::grid_begin(static_cast<int64_t>(c.rows) * c.cols);
    // every warp waits for and arrives at every barrier, once a tile
    auto wait = [&](uint32_t which, uint32_t parity) {
        if (ptx::mbar_wait_ns(which, parity, kWaitNs)) return true;
        atomicOr(err, 1u);
        return false;
    };
    auto arrive = [&](uint32_t which) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(which);
    };
    TileIn in;
    // tiles blockIdx.x, + gridDim.x (step_r rows of kbs and step_k), ...
    uint32_t rb = blockIdx.x / kbs, kb = blockIdx.x % kbs;
    if (rb < rbs) load_tile<WIDE>(in, dh, ld_dh, c, rb * kT + row, kb, seg);
    while (rb < rbs) {
        const uint32_t r0 = rb * kT;
        uint32_t next_r = rb + step_r, next_k = kb + step_k;
        if (next_k >= kbs) next_k -= kbs, ++next_r;
        if (warp < 24 && next_r < rbs) {
            // the next tile to L2, a line of 128 bytes per thread
            const uint32_t r = next_r * kT + (tid & 127), k0 = next_k * kT;
            const void *p = warp < 8    ? static_cast<const void *>(dh + row_at(r, ld_dh) + k0 + (tid >> 7) * 64)
                            : warp < 16 ? static_cast<const void *>((warp < 12 ? c.gq : c.uq) + row_at(r, c.ld_q) + k0)
                                        : static_cast<const void *>((warp < 20 ? c.gs : c.us) + row_at(r, c.ld_s) +
                                                                    next_k);
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
        }
        {
            const F2 sg = f2(scale_pow2(in.sg)), su = f2(scale_pow2(in.su));
            F2 a[8], b[8];
            float ma = 0.0f, mb = 0.0f;
            const uint32_t off = (row * kT + plane_piece(4 * seg, row) * 4) * 4;   // piece 4 seg + k: off ^ 16 k
            auto put = [&](int p, int k, F2 x, F2 y) {
                *reinterpret_cast<ulonglong2 *>(reinterpret_cast<char *>(plane) + (off ^ (k << 4)) + p * kPlane * 4) =
                    make_ulonglong2(x.v, y.v);
            };
            if (!wait(empty(2), phase ^ 1u)) return;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                F2 g[2], u[2], h[2];
                fp8x4_values<FC>(in.g[k], sg, g);
                fp8x4_values<FC>(in.u[k], su, u);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    swiglu_grads(g[j], u[j], f2_bf16(in.dh[2 * k + j]), a[2 * k + j], b[2 * k + j], h[j]);
                    ma = max_abs(ma, a[2 * k + j]);
                    mb = max_abs(mb, b[2 * k + j]);
                }
                put(2, k, h[0], h[1]);
            }
            arrive(full(2));
            const GroupF32<FR> ga(group_max(ma)), gb(group_max(mb));
            const int64_t at = row_at(r0 + row, o.ld_q) + kb * kT + seg * 16;
            uint32_t q[4];
            if (!wait(empty(0), phase ^ 1u)) return;
#pragma unroll
            for (int k = 0; k < 4; ++k) put(0, k, a[2 * k], a[2 * k + 1]);
            arrive(full(0));
            emit_codes<FR>(a, 4, ga, q);
            *reinterpret_cast<uint4 *>(o.q[0] + at) = make_uint4(q[0], q[1], q[2], q[3]);
            if (!wait(empty(1), phase ^ 1u)) return;
#pragma unroll
            for (int k = 0; k < 4; ++k) put(1, k, b[2 * k], b[2 * k + 1]);
            arrive(full(1));
            emit_codes<FR>(b, 4, gb, q);
            *reinterpret_cast<uint4 *>(o.q[1] + at) = make_uint4(q[0], q[1], q[2], q[3]);
            if (seg == 0) {
                const int64_t to = row_at(r0 + row, o.ld_s) + kb;
                o.s[0][to] = static_cast<uint8_t>(ga.byte);
                o.s[1][to] = static_cast<uint8_t>(gb.byte);
            }
        }
        if (next_r < rbs) load_tile<WIDE>(in, dh, ld_dh, c, next_r * kT + row, next_k, seg);
        // columns 4 warp .. + 3, tokens 4 lane .. + 3
        const float *src = plane + lane * 4 * kT + plane_piece(warp, lane * 4) * 4;
        const uint32_t col = kb * kT + warp * 4;
        const int64_t to = row_at(col, o.ld_qt) + r0 + lane * 4, sto = row_at(col + (lane & 3), o.ld_st) + rb;
#pragma unroll
        for (int i3 = 0; i3 < 3; ++i3) {
            const int w = (i3 + 2) % 3;   // h first
            if (!wait(full(w), phase)) return;
            F2 v[4][2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const ulonglong2 p = *reinterpret_cast<const ulonglong2 *>(src + w * kPlane + i * kT);
                v[i][0].v = p.x, v[i][1].v = p.y;
            }
            arrive(empty(w));
            if (w < 2) emit_columns<FT>(v, lane, o.qt[w] + to, o.ld_qt, o.st[w] + sto);
            else emit_columns<FH>(v, lane, o.qt[w] + to, o.ld_qt, o.st[w] + sto);
        }
        phase ^= 1u;
        rb = next_r, kb = next_k;
    }
}

template <int FH, int FC, bool CKPT>
cudaError_t fwd(const SwigluFwdArgs &a, cudaStream_t stream) {
    // segments of 16 columns, whole groups of eight; a chunk of at most 256
    // segments per block, spread evenly
    const int64_t total = (a.cols + 127LL) / 128 * 8, chunks = (total + 255) / 256;
    const int segs = static_cast<int>((total / 8 + chunks - 1) / chunks * 8);
    const int rpb = 256 / segs, threads = (segs * rpb + 31) / 32 * 32;
    const int64_t rb = (static_cast<int64_t>(a.rows) + rpb - 1) / rpb, cb = (total + segs - 1) / segs;
    // as many CTAs as fit at once
    const int64_t per_sm = kFwdThreadsPerSm / threads, resident = std::max<int64_t>(1, sm_count() * per_sm / cb);
    const dim3 grid = rows_first(std::min(rb, resident), cb);
    const bool wide = ragged::wide(a.gate, a.ld_in) && ragged::wide(a.up, a.ld_in);
    return launch_after(wide ? k_swiglu_fwd<FH, FC, CKPT, true> : k_swiglu_fwd<FH, FC, CKPT, false>, grid, threads, 0,
                        stream, 1, a, segs, total);
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

cudaError_t launch_swiglu_bwd(const uint16_t *dh, uint32_t ld_dh, const SwigluCkpt &c, uint16_t *dg,
                              uint16_t *du, uint32_t ld_d, cudaStream_t stream) {
    // a row's segments in equal blocks of whole warps
    const int64_t segs = (c.cols + 15LL) / 16, chunks = (segs + 255) / 256;
    const int threads = static_cast<int>(((segs + chunks - 1) / chunks + 31) / 32 * 32);
    const dim3 grid = chunks_first(c.rows, (segs + threads - 1) / threads);
    const bool wide = ragged::wide(dh, ld_dh) && ragged::wide(dg, ld_d) && ragged::wide(du, ld_d);
    auto go = [&](auto kern) {
        return launch_after(kern, grid, threads, 0, stream, 1, dh, ld_dh, c, dg, du, ld_d, segs);
    };
    if (c.fmt == FMT_E4M3) return wide ? go(k_swiglu_bwd<FMT_E4M3, true>) : go(k_swiglu_bwd<FMT_E4M3, false>);
    return wide ? go(k_swiglu_bwd<FMT_E5M2, true>) : go(k_swiglu_bwd<FMT_E5M2, false>);
}

namespace {

template <int FC, int FR, int FT, int FH>
cudaError_t bwd_q(const uint16_t *dh, uint32_t ld_dh, const SwigluCkpt &c, const SwigluGrads &g,
                  cudaStream_t stream) {
    const int64_t kbs = c.cols / kT, tiles = kbs * (c.rows / kT);
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(tiles, sm_count()));
    auto go = [&](auto kern) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kQSmem);
        if (e != cudaSuccess) return e;
        return launch_after(kern, grid, Q_THREADS, kQSmem, stream, 1, dh, ld_dh, c, g, kbs, c.rows / kT, grid % kbs,
                            grid / kbs, g.err);
    };
    return ragged::wide(dh, ld_dh) ? go(k_swiglu_bwd_q<FC, FR, FT, FH, true>)
                                   : go(k_swiglu_bwd_q<FC, FR, FT, FH, false>);
}
template <int FC, int FR, int FT>
cudaError_t bwd_q_h(const uint16_t *dh, uint32_t ld_dh, const SwigluCkpt &c, const SwigluGrads &g,
                    cudaStream_t stream) {
    return g.fmt_h == FMT_E4M3 ? bwd_q<FC, FR, FT, FMT_E4M3>(dh, ld_dh, c, g, stream)
                               : bwd_q<FC, FR, FT, FMT_E5M2>(dh, ld_dh, c, g, stream);
}
template <int FC, int FR>
cudaError_t bwd_q_t(const uint16_t *dh, uint32_t ld_dh, const SwigluCkpt &c, const SwigluGrads &g,
                    cudaStream_t stream) {
    return g.fmt_t == FMT_E4M3 ? bwd_q_h<FC, FR, FMT_E4M3>(dh, ld_dh, c, g, stream)
                               : bwd_q_h<FC, FR, FMT_E5M2>(dh, ld_dh, c, g, stream);
}

}  // namespace

cudaError_t launch_swiglu_bwd_q(const uint16_t *dh, uint32_t ld_dh, const SwigluCkpt &c, const SwigluGrads &g,
                                cudaStream_t stream) {
    if (c.fmt == FMT_E4M3)
        return g.fmt == FMT_E4M3 ? bwd_q_t<FMT_E4M3, FMT_E4M3>(dh, ld_dh, c, g, stream)
                                 : bwd_q_t<FMT_E4M3, FMT_E5M2>(dh, ld_dh, c, g, stream);
    return g.fmt == FMT_E4M3 ? bwd_q_t<FMT_E5M2, FMT_E4M3>(dh, ld_dh, c, g, stream)
                             : bwd_q_t<FMT_E5M2, FMT_E5M2>(dh, ld_dh, c, g, stream);
}

}  // namespace fp8hg
