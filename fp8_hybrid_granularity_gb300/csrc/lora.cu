// Low-rank adapters of many requests beside a shared projection.
//
//   v[t] = x[t] A_g^T,  y[t] = base[t] + s_g v[t] B_g^T     (g: the token's adapter)
//   dv[t] = s_g dy[t] B_g,  dx[t] = base[t] + dv[t] A_g
//   dA_g = sum over its tokens of dv[t]^T x[t],  dB_g = s_g sum of dy[t]^T v[t]
//
// Three kernels, each in both directions.  Tokens come in tiles of up to 128 of
// one adapter, gathered through the plan's order.
//   shrink   rows of r from rows of n or k: K split over the CTAs, partial sums
//            in FP32 that the next kernel adds in a fixed order
//   expand   rows of n or k from rows of r, added to the base's
//   outer    sums over the tokens; an adapter whose tokens several CTAs share is
//            summed by one more kernel, in a fixed order
// x, dy, A and B are BF16 and their products exact; sums are FP32.  The tensor
// cores' own sums are cut off instead of rounded, so a sum of at most 64 products
// (192 parts) stays there before it is added to registers.  v and dv, FP32 sums,
// go into the next product as two BF16 parts (16 bits, for results in BF16) or
// three (24 bits, for FP32).
//
// Ranks are small: 2 r operations per value of x, dy or y, so HBM is the bound.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "lora.cuh"

namespace fp8hg {

namespace {

using namespace lora;

constexpr int kSms = 152;

// ------------------------------------------------------------------- shrink
constexpr int kShrinkK = 64;         // of the long side per stage
constexpr int kShrinkStages = 4;

struct ShrinkArgs {
    LoraPlan plan;
    const uint16_t *x;
    uint32_t ld_x;
    const uint16_t *w;               // [adapters][r][k], or (TRANS) [adapters][k][r]
    int64_t stride_w;
    uint32_t ld_w;
    LoraWeights lw;                  // ranks
    int k, per;                      // k, and its share of a CTA (a multiple of 64)
    float *out;                      // [splits][tokens in the plan's order][RP]
};

template <int RP, bool TRANS>
__host__ __device__ constexpr int shrink_stage() {
    return kLoraTile * row_bytes(kShrinkK) + (TRANS ? kShrinkK * row_bytes(RP) : RP * row_bytes(kShrinkK));
}

template <int RP, bool TRANS, bool ALIGNED>
__global__ void __launch_bounds__(256) k_lora_shrink(const ShrinkArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int token[kLoraTile];
    constexpr int kStage = shrink_stage<RP, TRANS>(), kX = kLoraTile * row_bytes(kShrinkK);
    ptx::grid_begin(static_cast<int64_t>(a.plan.tokens) * a.k);
    if (blockIdx.x >= a.plan.words[0]) return;
    const Tile tile = tile_at(a.plan, blockIdx.x);
    if (tile.adapter < 0) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    if (tid < tile.count) token[tid] = a.plan.words[a.plan.order() + tile.first + tid];
    __syncthreads();
    const int rank = rank_of(a.lw, tile.adapter);
    const uint16_t *w = a.w + tile.adapter * a.stride_w;
    const uint32_t base = ptx::smem_u32(smem);
    const int k0 = blockIdx.y * a.per, k1 = min(a.k, k0 + a.per);
    const int steps = k1 > k0 ? (k1 - k0 + kShrinkK - 1) / kShrinkK : 0;
    const int mt = (tile.count + 15) / 16;

    auto load = [&](int step) {
        const int k = k0 + step * kShrinkK, left = k1 - k;
        const uint32_t to = base + step % kShrinkStages * kStage;
        for (int i = tid; i < mt * 16 * 8; i += 256) {
            const int row = i / 8, c = i % 8 * 8;
            const bool in = row < tile.count && c < left;
            copy8<ALIGNED>(to + row * row_bytes(kShrinkK) + 2 * c, in ? a.x + row_at(token[row], a.ld_x) + k + c : a.x, in ? left - c : 0);
        }
        if constexpr (TRANS) {
            for (int i = tid; i < kShrinkK * (RP / 8); i += 256) {
                const int row = i / (RP / 8), c = i % (RP / 8) * 8;
                const bool in = row < left && c < rank;
                copy8<ALIGNED>(to + kX + row * row_bytes(RP) + 2 * c, in ? w + row_at(k + row, a.ld_w) + c : w, in ? rank - c : 0);
            }
        } else {
            for (int i = tid; i < RP * 8; i += 256) {
                const int row = i / 8, c = i % 8 * 8;
                const bool in = row < rank && c < left;
                copy8<ALIGNED>(to + kX + row * row_bytes(kShrinkK) + 2 * c, in ? w + row_at(row, a.ld_w) + k + c : w, in ? left - c : 0);
            }
        }
    };

    // warps: 16 tokens each; with fewer tokens several share them and take every
    // second or fourth 16 of k
    const int mp = mt <= 1 ? 1 : mt <= 2 ? 2 : mt <= 4 ? 4 : 8, ways = min(4, 8 / mp);
    const int m = warp % mp, way = warp / mp;
    const bool active = m < mt && way < ways;
    float sum[RP / 8][4];
#pragma unroll
    for (int i = 0; i < RP / 8; ++i) sum[i][0] = sum[i][1] = sum[i][2] = sum[i][3] = 0.0f;
    for (int s = 0; s < kShrinkStages - 1; ++s) {
        if (s < steps) load(s);
        ptx::cp_async_commit();
    }
    for (int s = 0; s < steps; ++s) {
        ptx::cp_async_wait<kShrinkStages - 2>();
        __syncthreads();
        if (s + kShrinkStages - 1 < steps) load(s + kShrinkStages - 1);
        ptx::cp_async_commit();
        if (!active) continue;
        const uint32_t at = base + s % kShrinkStages * kStage;
        float acc[RP / 8][4];
#pragma unroll
        for (int i = 0; i < RP / 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
        for (int ks = way; ks < kShrinkK / 16; ks += ways) {
            uint32_t f[4];
            ptx::ldmatrix_x4<false>(at + (m * 16 + (lane & 15)) * row_bytes(kShrinkK) + (ks * 16 + (lane >> 4) * 8) * 2, f);
#pragma unroll
            for (int nt = 0; nt < RP / 16; ++nt) {
                uint32_t b[4];
                if constexpr (TRANS)
                    ptx::ldmatrix_x4<true>(at + kX + (ks * 16 + (lane & 15)) * row_bytes(RP) + (nt * 16 + (lane >> 4) * 8) * 2, b);
                else
                    ptx::ldmatrix_x4<false>(at + kX + (nt * 16 + (lane & 7) + (lane >> 4) * 8) * row_bytes(kShrinkK) +
                                                (ks * 16 + ((lane >> 3) & 1) * 8) * 2, b);
                ptx::mma_bf16(acc[2 * nt], f, b[0], b[1]);
                ptx::mma_bf16(acc[2 * nt + 1], f, b[2], b[3]);
            }
        }
#pragma unroll
        for (int i = 0; i < RP / 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[i][j] += acc[i][j];
    }
    ptx::cp_async_wait<0>();
    __syncthreads();
    // the ways' sums, in the stages' memory
    float *red = reinterpret_cast<float *>(smem);
    if (active) {
#pragma unroll
        for (int i = 0; i < RP / 8; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<float2 *>(red + ((way * mp + m) * 16 + (lane >> 2) + 8 * h) * (RP + 8) + i * 8 + (lane & 3) * 2) =
                    make_float2(sum[i][2 * h], sum[i][2 * h + 1]);
    }
    __syncthreads();
    float *out = a.out + (static_cast<int64_t>(blockIdx.y) * a.plan.tokens + tile.first) * RP;
    for (int i = tid; i < tile.count * (RP / 4); i += 256) {
        const int row = i / (RP / 4), c = i % (RP / 4) * 4;
        float4 t = *reinterpret_cast<const float4 *>(red + row * (RP + 8) + c);
        for (int q = 1; q < ways; ++q) {
            const float4 u = *reinterpret_cast<const float4 *>(red + (q * mp * 16 + row) * (RP + 8) + c);
            t.x += u.x, t.y += u.y, t.z += u.z, t.w += u.w;
        }
        *reinterpret_cast<float4 *>(out + row * RP + c) = t;
    }
}

// Rows of r, as the kernels after shrink read them: partial sums in the plan's
// order, or one row per token.
struct Rows {
    const float *v;
    int splits;          // 0: one row per token
    int64_t split;       // from one split to the next
    uint32_t ld;
};

// Values c .. c + 3 of the row at a position of the plan; `have` of the row's are there.
__device__ __forceinline__ float4 row_values(const Rows &s, const int *token, int64_t first, int row, int c, int have) {
    float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (s.splits > 0) {
        const float *p = s.v + (first + row) * s.ld + c;
        for (int i = 0; i < s.splits; ++i, p += s.split) {
            const uint4 q = ptx::ld_v4(p);
            t.x += __uint_as_float(q.x), t.y += __uint_as_float(q.y);
            t.z += __uint_as_float(q.z), t.w += __uint_as_float(q.w);
        }
    } else {
        const float *p = s.v + row_at(token[row], s.ld) + c;
        if (c < have) t.x = p[0];
        if (c + 1 < have) t.y = p[1];
        if (c + 2 < have) t.z = p[2];
        if (c + 3 < have) t.w = p[3];
    }
    if (c >= have) t.x = 0.0f;
    if (c + 1 >= have) t.y = 0.0f;
    if (c + 2 >= have) t.z = 0.0f;
    if (c + 3 >= have) t.w = 0.0f;
    return t;
}

// Four values times f, as PARTS planes of BF16.
template <int PARTS>
__device__ __forceinline__ void store_parts(uint8_t *at, int plane, float4 t, float f) {
    uint16_t h[4][PARTS];
    split<PARTS>(t.x * f, h[0]);
    split<PARTS>(t.y * f, h[1]);
    split<PARTS>(t.z * f, h[2]);
    split<PARTS>(t.w * f, h[3]);
#pragma unroll
    for (int p = 0; p < PARTS; ++p)
        *reinterpret_cast<uint2 *>(at + p * plane) =
            make_uint2(h[0][p] | static_cast<uint32_t>(h[1][p]) << 16, h[2][p] | static_cast<uint32_t>(h[3][p]) << 16);
}

// ------------------------------------------------------------------- expand
constexpr int kExpandN = 128;        // columns of a step

struct ExpandArgs {
    LoraPlan plan;
    Rows rows;
    const uint16_t *w;               // [adapters][n][r], or (TRANS) [adapters][r][n]
    int64_t stride_w;
    uint32_t ld_w;
    LoraWeights lw;                  // ranks, scale
    int n, per;                      // columns, and a CTA's share (a multiple of 128)
    const void *base;
    void *y;
    uint32_t ld_base, ld_y;
    float *v_out;                    // the rows of r for the backward pass, or null
    uint32_t ld_v;
};

template <bool F32>
struct Eight {
    uint32_t w[F32 ? 8 : 4];
};

// Columns c .. c + 7 of a row, of which `left` are there.
template <bool F32, bool ALIGNED>
__device__ __forceinline__ void load8(const void *base, int64_t at, int left, Eight<F32> &v) {
    if constexpr (F32) {
        const float *p = static_cast<const float *>(base) + at;
        if (ALIGNED && left >= 8) {
            const uint4 q = ptx::ld_once_v4(p), u = ptx::ld_once_v4(p + 4);
            v.w[0] = q.x, v.w[1] = q.y, v.w[2] = q.z, v.w[3] = q.w;
            v.w[4] = u.x, v.w[5] = u.y, v.w[6] = u.z, v.w[7] = u.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v.w[i] = i < left ? __float_as_uint(p[i]) : 0u;
        }
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(base) + at;
        if (ALIGNED && left >= 8) {
            const uint4 q = ptx::ld_once_v4(p);
            v.w[0] = q.x, v.w[1] = q.y, v.w[2] = q.z, v.w[3] = q.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v.w[i] = (2 * i < left ? p[2 * i] : 0u) | (2 * i + 1 < left ? static_cast<uint32_t>(p[2 * i + 1]) << 16 : 0u);
        }
    }
}
template <bool F32, bool ALIGNED>
__device__ __forceinline__ void store8(void *base, int64_t at, int left, const Eight<F32> &v) {
    if constexpr (F32) {
        float *p = static_cast<float *>(base) + at;
        if (ALIGNED && left >= 8) {
            reinterpret_cast<uint4 *>(p)[0] = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
            reinterpret_cast<uint4 *>(p)[1] = make_uint4(v.w[4], v.w[5], v.w[6], v.w[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left) p[i] = __uint_as_float(v.w[i]);
        }
    } else {
        uint16_t *p = static_cast<uint16_t *>(base) + at;
        if (ALIGNED && left >= 8) {
            *reinterpret_cast<uint4 *>(p) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left) p[i] = static_cast<uint16_t>(v.w[i >> 1] >> (16 * (i & 1)));
        }
    }
}

// Four words in each of a quad's four lanes, word j of lane i to word i of lane j.
__device__ __forceinline__ void quad_transpose(uint32_t &w0, uint32_t &w1, uint32_t &w2, uint32_t &w3) {
    const int lane = threadIdx.x & 3;
    // blocks of two, then within them
    {
        const bool hi = lane & 2;
        const uint32_t s0 = hi ? w0 : w2, s1 = hi ? w1 : w3;
        const uint32_t r0 = __shfl_xor_sync(0xFFFFFFFFu, s0, 2), r1 = __shfl_xor_sync(0xFFFFFFFFu, s1, 2);
        if (hi) w0 = r0, w1 = r1;
        else w2 = r0, w3 = r1;
    }
    {
        const bool hi = lane & 1;
        const uint32_t s0 = hi ? w0 : w1, s1 = hi ? w2 : w3;
        const uint32_t r0 = __shfl_xor_sync(0xFFFFFFFFu, s0, 1), r1 = __shfl_xor_sync(0xFFFFFFFFu, s1, 1);
        if (hi) w0 = r0, w2 = r1;
        else w1 = r0, w3 = r1;
    }
}

template <int RP, bool TRANS>
__host__ __device__ constexpr int expand_stage() {
    return TRANS ? RP * row_bytes(kExpandN) : kExpandN * row_bytes(RP);
}

// Parts of v: two for results in BF16, three for FP32.
template <int RP, bool TRANS, bool F32, bool ALIGNED>
__global__ void __launch_bounds__(256) k_lora_expand(const ExpandArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];   // two stages of weights, then v
    __shared__ int token[kLoraTile];
    constexpr int PARTS = F32 ? 3 : 2, kStage = expand_stage<RP, TRANS>(), kPlane = kLoraTile * row_bytes(RP);
    ptx::grid_begin(static_cast<int64_t>(a.plan.tokens) * a.n);
    if (blockIdx.x >= a.plan.words[0]) return;
    const Tile tile = tile_at(a.plan, blockIdx.x);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const int n0 = blockIdx.y * a.per, n1 = min(a.n, n0 + a.per);
    const bool none = tile.adapter < 0;
    if (tid < tile.count) token[tid] = a.plan.words[a.plan.order() + tile.first + tid];
    const int rank = none ? 0 : rank_of(a.lw, tile.adapter);
    const float scale = none ? 0.0f : a.lw.scale == nullptr ? 1.0f : a.lw.scale[tile.adapter];
    const uint16_t *w = a.w + (none ? 0 : tile.adapter) * a.stride_w;
    const uint32_t base = ptx::smem_u32(smem);
    const int steps = n1 > n0 ? (n1 - n0 + kExpandN - 1) / kExpandN : 0;
    const int mg = (tile.count + 31) / 32;       // groups of 32 tokens

    auto load = [&](int step) {
        const int n = n0 + step * kExpandN, left = n1 - n;
        const uint32_t to = base + (step & 1) * kStage;
        if constexpr (TRANS) {
            for (int i = tid; i < RP * (kExpandN / 8); i += 256) {
                const int row = i / (kExpandN / 8), c = i % (kExpandN / 8) * 8;
                const bool in = row < rank && c < left;
                copy8<ALIGNED>(to + row * row_bytes(kExpandN) + 2 * c, in ? w + row_at(row, a.ld_w) + n + c : a.w, in ? left - c : 0);
            }
        } else {
            for (int i = tid; i < kExpandN * (RP / 8); i += 256) {
                const int row = i / (RP / 8), c = i % (RP / 8) * 8;
                const bool in = row < left && c < rank;
                copy8<ALIGNED>(to + row * row_bytes(RP) + 2 * c, in ? w + row_at(n + row, a.ld_w) + c : a.w, in ? rank - c : 0);
            }
        }
    };
    if (steps > 0) load(0);
    ptx::cp_async_commit();
    __syncthreads();
    uint8_t *planes = smem + 2 * kStage;
    for (int i = tid; i < mg * 32 * (RP / 4); i += 256) {
        const int row = i / (RP / 4), c = i % (RP / 4) * 4;
        float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (row < tile.count) {
            if (!none) t = row_values(a.rows, token, tile.first, row, c, rank);
            if (a.v_out != nullptr && blockIdx.y == 0) {
                float *to = a.v_out + row_at(token[row], a.ld_v) + c;
                const int left = a.lw.r - c;
                if (left > 0) to[0] = t.x;
                if (left > 1) to[1] = t.y;
                if (left > 2) to[2] = t.z;
                if (left > 3) to[3] = t.w;
            }
        }
        store_parts<PARTS>(planes + row * row_bytes(RP) + 2 * c, kPlane, t, scale);
    }
    // warps: 32 tokens by a part of the step's columns
    const int mp = mg <= 1 ? 1 : mg <= 2 ? 2 : 4;
    const int subs = min(4, 8 / mp), m = warp % mp, sub = warp / mp, width = kExpandN / subs;
    const bool active = m < mg && sub < subs;
    const uint32_t vat = ptx::smem_u32(planes) + (m * 32 + (lane & 15)) * row_bytes(RP) + (lane >> 4) * 16;
    int rows[4];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = m * 32 + i * 8 + (lane >> 2);
        rows[i] = active && row < tile.count ? token[row] : -1;
    }
    for (int s = 0; s < steps; ++s) {
        if (s + 1 < steps) load(s + 1);
        ptx::cp_async_commit();
        ptx::cp_async_wait<1>();
        __syncthreads();
        const uint32_t at = base + (s & 1) * kStage;
        if (active) {
            for (int c = sub * width; c < (sub + 1) * width; c += 32) {
                const int col = n0 + s * kExpandN + c + (lane & 3) * 8, left = n1 - col;
                Eight<F32> in[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (a.base != nullptr && rows[i] >= 0 && left > 0)
                        load8<F32, ALIGNED>(a.base, row_at(rows[i], a.ld_base) + col, left, in[i]);
                    else
#pragma unroll
                        for (int j = 0; j < (F32 ? 8 : 4); ++j) in[i].w[j] = 0u;
                }
                float acc[2][4][4];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j][0] = acc[i][j][1] = acc[i][j][2] = acc[i][j][3] = 0.0f;
#pragma unroll
                for (int ks = 0; ks < RP / 16; ++ks) {
                    uint32_t b[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if constexpr (TRANS)
                            ptx::ldmatrix_x4<true>(at + (ks * 16 + (lane & 15)) * row_bytes(kExpandN) + (c + h * 16 + (lane >> 4) * 8) * 2, b[h]);
                        else
                            ptx::ldmatrix_x4<false>(at + (c + h * 16 + (lane & 7) + (lane >> 4) * 8) * row_bytes(RP) +
                                                        (ks * 16 + ((lane >> 3) & 1) * 8) * 2, b[h]);
                    }
#pragma unroll
                    for (int p = 0; p < PARTS; ++p) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t f[4];
                            ptx::ldmatrix_x4<false>(vat + p * kPlane + i * 16 * row_bytes(RP) + ks * 32, f);
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                ptx::mma_bf16(acc[i][j], f, b[j >> 1][(j & 1) * 2], b[j >> 1][(j & 1) * 2 + 1]);
                        }
                    }
                }
                // a quad's lanes hold two columns of each of four groups of eight:
                // transposed, a lane has the eight columns that it loads and stores
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t lo[4], hi[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        lo[j] = __float_as_uint(acc[i >> 1][j][(i & 1) * 2]);
                        hi[j] = __float_as_uint(acc[i >> 1][j][(i & 1) * 2 + 1]);
                    }
                    quad_transpose(lo[0], lo[1], lo[2], lo[3]);
                    quad_transpose(hi[0], hi[1], hi[2], hi[3]);
                    Eight<F32> out;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if constexpr (F32) {
                            out.w[2 * j] = __float_as_uint(__uint_as_float(in[i].w[2 * j]) + __uint_as_float(lo[j]));
                            out.w[2 * j + 1] = __float_as_uint(__uint_as_float(in[i].w[2 * j + 1]) + __uint_as_float(hi[j]));
                        } else {
                            out.w[j] = ptx::cvt_bf16x2(__uint_as_float(in[i].w[j] << 16) + __uint_as_float(lo[j]),
                                                       __uint_as_float(in[i].w[j] & 0xFFFF0000u) + __uint_as_float(hi[j]));
                        }
                    }
                    if (rows[i] >= 0 && left > 0) store8<F32, ALIGNED>(a.y, row_at(rows[i], a.ld_y) + col, left, out);
                }
            }
        }
        __syncthreads();
    }
}

// -------------------------------------------------------------------- outer
constexpr int kOuterT = 64;          // tokens of a stage

struct OuterArgs {
    LoraPlan plan;
    const uint16_t *d;               // [tokens][n]
    uint32_t ld_d;
    Rows rows;                       // of r
    LoraWeights lw;                  // ranks, scale, r
    int n, tiles;                    // columns, and tiles of a CTA
    void *out;                       // [adapters] of [n][r] or [r][n]: strides
    int64_t stride_n, stride_r, stride_g;
    float *ws;                       // [2 chunks][n][RP]
};

template <int RP>
struct OuterShape {
    static constexpr int MT = RP <= 64 ? 2 : 1;          // 16 columns each, a warp
    static constexpr int N = 8 * 16 * MT;                // columns of a CTA
    static constexpr int PARTS = 3;
    static constexpr int kD = kOuterT * row_bytes(N), kV = kOuterT * row_bytes(RP);
    static constexpr int kSmem = 2 * (kD + PARTS * kV);
};

// The tiles of a chunk of the plan; an adapter that is in several chunks leaves
// partial sums: those that begin the chunk in slot 2 c, those that end it in 2 c + 1.
template <int RP, bool F32, bool ALIGNED>
__global__ void __launch_bounds__(256) k_lora_outer(const OuterArgs a) {
    using S = OuterShape<RP>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int token[2][kOuterT];
    ptx::grid_begin(static_cast<int64_t>(a.plan.tokens) * a.n);
    const int tiles = a.plan.words[0];
    const int t0 = blockIdx.y * a.tiles, t1 = min(tiles, t0 + a.tiles);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const int n0 = blockIdx.x * S::N, n_left = a.n - n0;
    const uint32_t base = ptx::smem_u32(smem);
    float sum[S::MT][RP / 8][4];
    auto clear = [&](float (&s)[S::MT][RP / 8][4]) {
#pragma unroll
        for (int i = 0; i < S::MT; ++i)
#pragma unroll
            for (int j = 0; j < RP / 8; ++j) s[i][j][0] = s[i][j][1] = s[i][j][2] = s[i][j][3] = 0.0f;
    };
    clear(sum);
    const int *tile_first = a.plan.words + a.plan.tile_first();
    for (int t = t0; t < t1; ++t) {
        const Tile tile = tile_at(a.plan, t);
        if (tile.adapter < 0) break;             // the tokens without an adapter come last
        const int rank = rank_of(a.lw, tile.adapter);
        const float scale = a.lw.scale == nullptr ? 1.0f : a.lw.scale[tile.adapter];
        const int halves = (tile.count + kOuterT - 1) / kOuterT;
        auto load = [&](int h) {
            const int first = h * kOuterT, count = min(kOuterT, tile.count - first);
            int *tok = token[h];
            if (tid < count) tok[tid] = a.plan.words[a.plan.order() + tile.first + first + tid];
            __syncthreads();
            const uint32_t to = base + h * (S::kD + S::PARTS * S::kV);
            for (int i = tid; i < kOuterT * (S::N / 8); i += 256) {
                const int row = i / (S::N / 8), c = i % (S::N / 8) * 8;
                const bool in = row < count && c < n_left;
                copy8<ALIGNED>(to + row * row_bytes(S::N) + 2 * c, in ? a.d + row_at(tok[row], a.ld_d) + n0 + c : a.d, in ? n_left - c : 0);
            }
            ptx::cp_async_commit();
            uint8_t *v = smem + h * (S::kD + S::PARTS * S::kV) + S::kD;
            for (int i = tid; i < kOuterT * (RP / 4); i += 256) {
                const int row = i / (RP / 4), c = i % (RP / 4) * 4;
                const float4 f = row < count ? row_values(a.rows, tok, tile.first + first, row, c, rank) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                store_parts<S::PARTS>(v + row * row_bytes(RP) + 2 * c, S::kV, f, scale);
            }
        };
        load(0);
        if (halves > 1) load(1);
        for (int h = 0; h < halves; ++h) {
            if (h + 1 < halves) ptx::cp_async_wait<1>();
            else ptx::cp_async_wait<0>();
            __syncthreads();
            const uint32_t at = base + h * (S::kD + S::PARTS * S::kV);
            float acc[S::MT][RP / 8][4];
            clear(acc);
#pragma unroll
            for (int ks = 0; ks < kOuterT / 16; ++ks) {
                uint32_t f[S::MT][4];
#pragma unroll
                for (int i = 0; i < S::MT; ++i)
                    ptx::ldmatrix_x4<true>(at + (ks * 16 + (lane & 7) + (lane >> 4) * 8) * row_bytes(S::N) +
                                               ((warp * S::MT + i) * 16 + ((lane >> 3) & 1) * 8) * 2, f[i]);
#pragma unroll
                for (int p = 0; p < S::PARTS; ++p)
#pragma unroll
                    for (int nt = 0; nt < RP / 16; ++nt) {
                        uint32_t b[4];
                        ptx::ldmatrix_x4<true>(at + S::kD + p * S::kV + (ks * 16 + (lane & 15)) * row_bytes(RP) +
                                                   (nt * 16 + (lane >> 4) * 8) * 2, b);
#pragma unroll
                        for (int i = 0; i < S::MT; ++i) {
                            ptx::mma_bf16(acc[i][2 * nt], f[i], b[0], b[1]);
                            ptx::mma_bf16(acc[i][2 * nt + 1], f[i], b[2], b[3]);
                        }
                    }
            }
#pragma unroll
            for (int i = 0; i < S::MT; ++i)
#pragma unroll
                for (int j = 0; j < RP / 8; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) sum[i][j][q] += acc[i][j][q];
        }
        __syncthreads();
        const int begin = tile_first[tile.adapter], end = tile_first[tile.adapter + 1];
        if (t + 1 < t1 && t + 1 < end) continue;
        // the adapter's last tile, here or at all
        const bool whole = begin >= t0 && end <= t1;
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.y) + (begin < t0 ? 0 : 1);
#pragma unroll
        for (int i = 0; i < S::MT; ++i)
#pragma unroll
            for (int j = 0; j < RP / 8; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int c = (warp * S::MT + i) * 16 + (lane >> 2) + (q >> 1) * 8, r = j * 8 + (lane & 3) * 2 + (q & 1);
                    if (c >= n_left) continue;
                    if (!whole) {
                        a.ws[(slot * a.n + n0 + c) * RP + r] = sum[i][j][q];
                    } else if (r < a.lw.r) {
                        const int64_t at = tile.adapter * a.stride_g + (n0 + c) * a.stride_n + r * a.stride_r;
                        if constexpr (F32) static_cast<float *>(a.out)[at] = sum[i][j][q];
                        else static_cast<uint16_t *>(a.out)[at] = static_cast<uint16_t>(ptx::cvt_bf16x2(sum[i][j][q], 0.0f));
                    }
                }
        clear(sum);
    }
}

// The adapters of several chunks, and zeros for those without a token.
template <bool F32>
__global__ void __launch_bounds__(256) k_lora_outer_join(const OuterArgs a, int rp, int chunks) {
    ptx::grid_wait();
    const int *tile_first = a.plan.words + a.plan.tile_first();
    const int64_t each = static_cast<int64_t>(a.n) * a.lw.r;
    for (int g = blockIdx.y; g < a.plan.adapters; g += gridDim.y) {
        const int begin = tile_first[g], end = tile_first[g + 1];
        const int c0 = begin / a.tiles, c1 = begin < end ? (end - 1) / a.tiles : c0;
        if (begin < end && c0 == c1) continue;
        for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < each; i += static_cast<int64_t>(gridDim.x) * 256) {
            // neighbouring threads write neighbouring values
            const int64_t n = a.stride_n == 1 ? i % a.n : i / a.lw.r, r = a.stride_n == 1 ? i / a.n : i % a.lw.r;
            float s = 0.0f;
            if (begin < end) {
                s = a.ws[((2 * static_cast<int64_t>(c0) + 1) * a.n + n) * rp + r];
                for (int c = c0 + 1; c <= c1; ++c) s += a.ws[(2 * static_cast<int64_t>(c) * a.n + n) * rp + r];
            }
            const int64_t at = g * a.stride_g + n * a.stride_n + r * a.stride_r;
            if constexpr (F32) static_cast<float *>(a.out)[at] = s;
            else static_cast<uint16_t *>(a.out)[at] = static_cast<uint16_t>(ptx::cvt_bf16x2(s, 0.0f));
        }
    }
}

// ----------------------------------------------------------------- launches
int padded(int r) { return r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128; }
bool al16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <class K>
cudaError_t with_smem(K kern, size_t bytes) {
    return bytes <= 48 * 1024 ? cudaSuccess
                              : cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
}

// Parts of the long side that shrink is split into: two CTAs an SM, at least 128 of it each.
int shrink_splits(int tokens, int adapters, int k) {
    const int64_t tiles = std::max(1, tokens / kLoraTile + std::min(adapters, tokens) / 2);
    const int64_t want = (2 * kSms + tiles - 1) / tiles, most = std::max(1, k / 128);
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, most), 32)));
}

template <int RP, bool TRANS>
cudaError_t shrink(const ShrinkArgs &a, int splits, bool aligned, cudaStream_t stream) {
    auto *kern = aligned ? &k_lora_shrink<RP, TRANS, true> : &k_lora_shrink<RP, TRANS, false>;
    // the stages, or the sums of up to four ways
    const size_t smem = std::max<size_t>(kShrinkStages * shrink_stage<RP, TRANS>(), kLoraTile * (RP + 8) * sizeof(float));
    const cudaError_t e = with_smem(kern, smem);
    if (e != cudaSuccess) return e;
    return launch_after(kern, dim3(a.plan.max_tiles(), splits), 256, smem, stream, 1, a);
}
template <bool TRANS>
cudaError_t shrink_rp(const ShrinkArgs &a, int splits, bool aligned, cudaStream_t stream) {
    switch (padded(a.lw.r)) {
        case 16: return shrink<16, TRANS>(a, splits, aligned, stream);
        case 32: return shrink<32, TRANS>(a, splits, aligned, stream);
        case 64: return shrink<64, TRANS>(a, splits, aligned, stream);
        default: return shrink<128, TRANS>(a, splits, aligned, stream);
    }
}

template <int RP, bool TRANS, bool F32>
cudaError_t expand(const ExpandArgs &a, int splits, bool aligned, cudaStream_t stream) {
    auto *kern = aligned ? &k_lora_expand<RP, TRANS, F32, true> : &k_lora_expand<RP, TRANS, F32, false>;
    const size_t smem = 2 * expand_stage<RP, TRANS>() + (F32 ? 3 : 2) * kLoraTile * row_bytes(RP);
    const cudaError_t e = with_smem(kern, smem);
    if (e != cudaSuccess) return e;
    return launch_after(kern, dim3(a.plan.max_tiles(), splits), 256, smem, stream, 1, a);
}
template <bool TRANS, bool F32>
cudaError_t expand_rp(const ExpandArgs &a, int splits, bool aligned, cudaStream_t stream) {
    switch (padded(a.lw.r)) {
        case 16: return expand<16, TRANS, F32>(a, splits, aligned, stream);
        case 32: return expand<32, TRANS, F32>(a, splits, aligned, stream);
        case 64: return expand<64, TRANS, F32>(a, splits, aligned, stream);
        default: return expand<128, TRANS, F32>(a, splits, aligned, stream);
    }
}
template <bool TRANS>
cudaError_t run_expand(ExpandArgs &a, bool f32, bool aligned, cudaStream_t stream) {
    const int64_t tiles = std::max(1, a.plan.tokens / kLoraTile + std::min(a.plan.adapters, a.plan.tokens) / 2);
    const int steps = (a.n + kExpandN - 1) / kExpandN;
    const int splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min(steps, 65535), (4 * kSms + tiles - 1) / tiles)));
    a.per = (steps + splits - 1) / splits * kExpandN;
    const int e = f32 ? 4 : 8;
    aligned = aligned && al16(a.w) && a.ld_w % 8 == 0 && a.stride_w % 8 == 0 && al16(a.y) && a.ld_y % e == 0 &&
              (a.base == nullptr || (al16(a.base) && a.ld_base % e == 0));
    return f32 ? expand_rp<TRANS, true>(a, splits, aligned, stream) : expand_rp<TRANS, false>(a, splits, aligned, stream);
}

int outer_n(int rp) { return rp <= 64 ? 256 : 128; }
// Chunks of tiles that the sums over the tokens are split into: two CTAs an SM.
int outer_chunks(const LoraPlan &p, int n, int rp) {
    const int blocks = (n + outer_n(rp) - 1) / outer_n(rp);
    return std::max(1, std::min(p.max_tiles(), (2 * kSms + blocks - 1) / blocks));
}
size_t outer_ws(const LoraPlan &p, int n, int rp) {
    return 2 * static_cast<size_t>(outer_chunks(p, n, rp)) * n * rp * sizeof(float);
}

template <int RP, bool F32>
cudaError_t outer(const OuterArgs &a, int chunks, bool aligned, cudaStream_t stream) {
    auto *kern = aligned ? &k_lora_outer<RP, F32, true> : &k_lora_outer<RP, F32, false>;
    const cudaError_t e = with_smem(kern, OuterShape<RP>::kSmem);
    if (e != cudaSuccess) return e;
    return launch_after(kern, dim3((a.n + OuterShape<RP>::N - 1) / OuterShape<RP>::N, chunks), 256, OuterShape<RP>::kSmem, stream, 1, a);
}
template <bool F32>
cudaError_t run_outer(OuterArgs &a, cudaStream_t stream) {
    const int rp = padded(a.lw.r), most = outer_chunks(a.plan, a.n, rp);
    a.tiles = (a.plan.max_tiles() + most - 1) / most;
    const int chunks = (a.plan.max_tiles() + a.tiles - 1) / a.tiles;
    const bool aligned = al16(a.d) && a.ld_d % 8 == 0;
    cudaError_t e = rp == 16   ? outer<16, F32>(a, chunks, aligned, stream)
                    : rp == 32 ? outer<32, F32>(a, chunks, aligned, stream)
                    : rp == 64 ? outer<64, F32>(a, chunks, aligned, stream)
                               : outer<128, F32>(a, chunks, aligned, stream);
    if (e != cudaSuccess) return e;
    const int64_t blocks = (static_cast<int64_t>(a.n) * a.lw.r + 255) / 256;
    return launch_after(&k_lora_outer_join<F32>, dim3(static_cast<unsigned>(std::min<int64_t>(blocks, 1024)), std::min(a.plan.adapters, 256)), 256,
                        0, stream, 1, a, rp, chunks);
}

ShrinkArgs shrink_args(const LoraWeights &w, const LoraPlan &plan, bool trans, const uint16_t *x, uint32_t ld_x, float *out, int &splits) {
    ShrinkArgs s{};
    s.plan = plan;
    s.x = x;
    s.ld_x = ld_x;
    s.w = trans ? w.b : w.a;
    s.stride_w = trans ? w.stride_b : w.stride_a;
    s.ld_w = trans ? w.ld_b : w.ld_a;
    s.lw = w;
    s.k = trans ? w.n : w.k;
    s.out = out;
    splits = shrink_splits(plan.tokens, plan.adapters, s.k);
    s.per = ((s.k + splits - 1) / splits + kShrinkK - 1) / kShrinkK * kShrinkK;
    splits = (s.k + s.per - 1) / s.per;
    return s;
}
bool shrink_aligned(const ShrinkArgs &s) {
    return al16(s.x) && s.ld_x % 8 == 0 && al16(s.w) && s.ld_w % 8 == 0 && s.stride_w % 8 == 0;
}
size_t shrink_ws(int64_t tokens, int adapters, int r, int64_t k) {
    return static_cast<size_t>(shrink_splits(static_cast<int>(tokens), adapters, static_cast<int>(k))) * tokens * padded(r) * sizeof(float);
}

}  // namespace

size_t lora_ws_bytes(int64_t tokens, int adapters, int r, int64_t k) { return shrink_ws(tokens, adapters, r, k); }

size_t lora_bwd_ws_bytes(int64_t tokens, int adapters, int r, int64_t n, int64_t k) {
    const LoraPlan p{nullptr, static_cast<int>(tokens), adapters};
    const int rp = padded(r);
    return shrink_ws(tokens, adapters, r, n) + outer_ws(p, static_cast<int>(n), rp) + outer_ws(p, static_cast<int>(k), rp);
}

cudaError_t launch_lora_add(const LoraArgs &a, cudaStream_t stream) {
    int splits = 0;
    const ShrinkArgs s = shrink_args(a.w, a.plan, false, a.x, a.ld_x, a.ws, splits);
    const cudaError_t e = shrink_rp<false>(s, splits, shrink_aligned(s), stream);
    if (e != cudaSuccess) return e;
    const int rp = padded(a.w.r);
    ExpandArgs x{};
    x.plan = a.plan;
    x.rows = {a.ws, splits, static_cast<int64_t>(a.plan.tokens) * rp, static_cast<uint32_t>(rp)};
    x.w = a.w.b;
    x.stride_w = a.w.stride_b;
    x.ld_w = a.w.ld_b;
    x.lw = a.w;
    x.n = a.w.n;
    x.base = a.base;
    x.y = a.y;
    x.ld_base = a.ld_base;
    x.ld_y = a.ld_y;
    x.v_out = a.v;
    x.ld_v = a.ld_v;
    return run_expand<false>(x, a.y_f32, true, stream);
}

cudaError_t launch_lora_add_bwd(const LoraBwdArgs &a, cudaStream_t stream) {
    const int rp = padded(a.w.r);
    cudaError_t e = cudaSuccess;
    int splits = 0;
    float *ws = a.ws;
    Rows dv{};
    if (a.dx != nullptr || a.da != nullptr) {
        const ShrinkArgs s = shrink_args(a.w, a.plan, true, a.dy, a.ld_dy, ws, splits);
        e = shrink_rp<true>(s, splits, shrink_aligned(s), stream);
        if (e != cudaSuccess) return e;
        dv = {ws, splits, static_cast<int64_t>(a.plan.tokens) * rp, static_cast<uint32_t>(rp)};
    }
    ws += shrink_ws(a.plan.tokens, a.plan.adapters, a.w.r, a.w.n) / sizeof(float);
    OuterArgs o{};
    o.plan = a.plan;
    o.lw = a.w;
    if (a.db != nullptr) {
        o.d = a.dy;
        o.ld_d = a.ld_dy;
        o.rows = {a.v, 0, 0, a.ld_v};
        o.n = a.w.n;
        o.out = a.db;
        o.stride_n = a.w.r;
        o.stride_r = 1;
        o.stride_g = static_cast<int64_t>(a.w.n) * a.w.r;
        o.ws = ws;
        e = a.dw_f32 ? run_outer<true>(o, stream) : run_outer<false>(o, stream);
        if (e != cudaSuccess) return e;
    }
    ws += outer_ws(a.plan, a.w.n, rp) / sizeof(float);
    if (a.da != nullptr) {
        o.d = a.x;
        o.ld_d = a.ld_x;
        o.rows = dv;
        o.n = a.w.k;
        o.out = a.da;
        o.stride_n = 1;
        o.stride_r = a.w.k;
        o.stride_g = static_cast<int64_t>(a.w.k) * a.w.r;
        o.ws = ws;
        e = a.dw_f32 ? run_outer<true>(o, stream) : run_outer<false>(o, stream);
        if (e != cudaSuccess) return e;
    }
    if (a.dx == nullptr) return cudaSuccess;
    ExpandArgs x{};
    x.plan = a.plan;
    x.rows = dv;
    x.w = a.w.a;
    x.stride_w = a.w.stride_a;
    x.ld_w = a.w.ld_a;
    x.lw = a.w;
    x.n = a.w.k;
    x.base = a.base;
    x.y = a.dx;
    x.ld_base = a.ld_base;
    x.ld_y = a.ld_dx;
    return run_expand<true>(x, a.dx_f32, true, stream);
}

// -------------------------------------------------------------------- plan
namespace {

// A stable counting sort by one CTA: each warp counts, then places, a run of
// neighbouring tokens.  counts: [warps][adapters + 1].
__global__ void __launch_bounds__(1024) k_lora_plan(const int *ids, int tokens, int adapters, int *words) {
    extern __shared__ int counts[];
    __shared__ int warp_total[32][2];
    const LoraPlan p{words, tokens, adapters};
    ptx::grid_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, warps = blockDim.x / 32;
    const int buckets = adapters + 1;
    for (int i = tid; i < warps * buckets; i += blockDim.x) counts[i] = 0;
    __syncthreads();
    const int per = ((tokens + warps - 1) / warps + 31) / 32 * 32;
    const int64_t from = static_cast<int64_t>(warp) * per, to = min(static_cast<int64_t>(tokens), from + per);
    int *mine = counts + warp * buckets;
    auto bucket = [&](int64_t i) {
        const int g = ids[i];
        return g >= 0 && g < adapters ? g : adapters;
    };
    for (int64_t i0 = from; i0 < to; i0 += 32) {
        const int64_t i = i0 + lane;
        const int b = i < to ? bucket(i) : -1;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, b);
        if (b >= 0 && lane == __ffs(same) - 1) mine[b] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    // every thread a run of buckets: their tokens and tiles, then where they begin
    const int run = (buckets + blockDim.x - 1) / blockDim.x, b0 = min(buckets, tid * run), b1 = min(buckets, b0 + run);
    int n = 0, t = 0;
    for (int b = b0; b < b1; ++b) {
        int c = 0;
        for (int w = 0; w < warps; ++w) c += counts[w * buckets + b];
        n += c;
        t += (c + kLoraTile - 1) / kLoraTile;
    }
    int sn = n, st = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int un = __shfl_up_sync(0xFFFFFFFFu, sn, o), ut = __shfl_up_sync(0xFFFFFFFFu, st, o);
        if (lane >= o) sn += un, st += ut;
    }
    if (lane == 31) warp_total[warp][0] = sn, warp_total[warp][1] = st;
    __syncthreads();
    int bn = sn - n, bt = st - t;
    for (int w = 0; w < warp; ++w) bn += warp_total[w][0], bt += warp_total[w][1];
    for (int b = b0; b < b1; ++b) {
        words[p.starts() + b] = bn;
        words[p.tile_first() + b] = bt;
        const int first = bn;
        for (int w = 0; w < warps; ++w) {
            const int c = counts[w * buckets + b];
            counts[w * buckets + b] = bn;
            bn += c;
        }
        for (int f = first; f < bn; f += kLoraTile, ++bt) {
            words[p.tiles() + 2 * static_cast<int64_t>(bt)] = b == adapters ? -1 : b;
            words[p.tiles() + 2 * static_cast<int64_t>(bt) + 1] = f;
        }
    }
    if (b1 == buckets && b0 < b1) {
        words[p.starts() + buckets] = bn;
        words[p.tile_first() + buckets] = bt;
        words[0] = bt;
    }
    __syncthreads();
    for (int64_t i0 = from; i0 < to; i0 += 32) {
        const int64_t i = i0 + lane;
        const int b = i < to ? bucket(i) : -1;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, b);
        if (b >= 0) words[p.order() + mine[b] + __popc(same & ((1u << lane) - 1u))] = static_cast<int>(i);
        __syncwarp();
        if (b >= 0 && lane == __ffs(same) - 1) mine[b] += __popc(same);
        __syncwarp();
    }
}

}  // namespace

cudaError_t launch_lora_plan(const int *ids, const LoraPlan &p, int *words, cudaStream_t stream) {
    const int buckets = p.adapters + 1;
    const int warps = std::max(1, std::min(32, 200 * 1024 / (4 * buckets)));
    const size_t smem = static_cast<size_t>(warps) * buckets * 4;
    const cudaError_t e = with_smem(&k_lora_plan, smem);
    if (e != cudaSuccess) return e;
    return launch_after(&k_lora_plan, dim3(1), warps * 32, smem, stream, 1, ids, p.tokens, p.adapters, words);
}

}  // namespace fp8hg
