// Adapters: sums over the tokens, out_g[n][r] = sum over g's tokens of d[t][n]
// v[t][r], for dB (d = dy) and dA (d = x, v = dv) in one launch.
//
// The rows of r come first, in a kernel of their own: partial sums added, scaled,
// taken apart into BF16 parts and transposed, so that a fragment's terms, the
// tokens, are neighbours.  Of d's rows a lane takes 8 (or 4) neighbouring columns
// of eight tokens, through its own slots, and puts the pairs of tokens together
// itself.  A CTA takes 512 (or 256) columns and a chunk of the tiles; an
// adapter whose tokens are in several chunks leaves partial sums there, which one
// more kernel adds in a fixed order.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "lora.cuh"

namespace fp8hg {
namespace lora {

namespace {

constexpr int kChunk = 32;           // tokens of a lane's eight rows

// ------------------------------------------------------------ rows of r, prepared
// A tile's 16 rows of r a CTA.
template <int RP, int PARTS>
__global__ void __launch_bounds__(256) k_lora_prep(const PrepArgs a) {
    __shared__ float rows[16][kLoraTile + 4];
    ptx::grid_begin(static_cast<int64_t>(a.plan.tokens) * RP);
    const int side = blockIdx.y, tiles = adapter_tiles(a.plan);
    if ((side == 0 ? a.v : a.dv) == nullptr || static_cast<int>(blockIdx.x) >= tiles) return;
    const Tile tile = tile_at(a.plan, blockIdx.x);
    const int rank = rank_of(a.lw, tile.adapter), tid = threadIdx.x, r0 = blockIdx.z * 16;
    const float scale = a.lw.scale == nullptr ? 1.0f : a.lw.scale[tile.adapter];
    const int splits = side == 0 ? 0 : shrink_splits(tiles, a.long_side, RP);
#pragma unroll
    for (int h = 0; h < kLoraTile * 4 / 256; ++h) {
        const int m = (h * 256 + tid) / 4, c = tid % 4 * 4, r = r0 + c;
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (m < tile.count) {
            if (side == 0) {
                const float *p = a.v + row_at(a.plan.words[a.plan.order() + tile.first + m], a.ld_v) + r;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (r + e < rank) v[e] = p[e];
            } else {
                const float *p = a.dv + (tile.first + m) * static_cast<int64_t>(RP) + r;
                const int64_t step = static_cast<int64_t>(a.plan.tokens) * RP;
#pragma unroll 8
                for (int s = 0; s < splits; ++s) {
                    const uint4 q = ptx::ld_v4(p + s * step);
                    v[0] += __uint_as_float(q.x), v[1] += __uint_as_float(q.y);
                    v[2] += __uint_as_float(q.z), v[3] += __uint_as_float(q.w);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (r + e >= rank) v[e] = 0.0f;
                if (a.sum != nullptr)
                    *reinterpret_cast<float4 *>(a.sum + (tile.first + m) * static_cast<int64_t>(RP) + r) = make_float4(v[0], v[1], v[2], v[3]);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) rows[c + e][m] = v[e] * scale;
    }
    __syncthreads();
    // eight tokens of a row of r a thread
    const int r = tid / (kLoraTile / 8), m = tid % (kLoraTile / 8) * 8;
    uint32_t w[PARTS][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint32_t lo[PARTS], hi[PARTS];
        split<PARTS>(rows[r][m + 2 * e], lo);
        split<PARTS>(rows[r][m + 2 * e + 1], hi);
#pragma unroll
        for (int p = 0; p < PARTS; ++p) w[p][e] = lo[p] | hi[p] << 16;
    }
    const int64_t ld = static_cast<int64_t>(a.plan.max_tiles()) * kLoraTile;
#pragma unroll
    for (int p = 0; p < PARTS; ++p)
        *reinterpret_cast<uint4 *>(a.vt[side] + p * a.plane + (r0 + r) * ld + static_cast<int64_t>(blockIdx.x) * kLoraTile + m) =
            make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
}

// -------------------------------------------------------------------- outer
// Sixteen warps: eight times the columns, and the rows of r in two halves.
constexpr int kThreads = 512;
template <int RP, int PARTS>
struct Shape {
    static constexpr int CT = RP <= 64 ? 4 : 2;          // fragments of 16 columns, a warp
    static constexpr int CL = 2 * CT;                    // neighbouring columns of a lane
    static constexpr int COLS = 8 * 16 * CT;             // of a CTA
    static constexpr int J = RP / 16;                    // fragments of 8 rows of r, a warp
    static constexpr int V = PARTS * RP * kChunk * 2;    // of a step
    static constexpr int D = kChunk * COLS * 2;
    static constexpr int STAGES = 4;
    static constexpr int SMEM = STAGES * (V + D);
};

// CL columns from p on (`left` > 0 of them there), zeros behind: the aligned
// 16-byte pieces that hold them, moved into place.
template <int CL>
__device__ __forceinline__ void load_cols(const uint16_t *p, int left, uint32_t (&w)[CL / 2]) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    const uint32_t s = static_cast<uint32_t>(at & 15), bytes = 2u * static_cast<uint32_t>(min(CL, left));
    const uint4 *q = reinterpret_cast<const uint4 *>(at & ~static_cast<uintptr_t>(15));
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint4 u = make_uint4(0u, 0u, 0u, 0u);
        if (s + bytes > 16u * i) u = ptx::ld_v4(q + i);
        v[4 * i] = u.x, v[4 * i + 1] = u.y, v[4 * i + 2] = u.z, v[4 * i + 3] = u.w;
    }
    if (s & 8) {
#pragma unroll
        for (int i = 0; i < 6; ++i) v[i] = v[i + 2];
    }
    if (s & 4) {
#pragma unroll
        for (int i = 0; i < 7; ++i) v[i] = v[i + 1];
    }
    if (s & 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __funnelshift_r(v[i], v[i + 1], 16);
    }
#pragma unroll
    for (int i = 0; i < CL / 2; ++i) w[i] = bytes >= 4u * i + 4u ? v[i] : bytes > 4u * i ? v[i] & 0xFFFFu : 0u;
}

template <int RP, int PARTS, bool WIDE>
__global__ void __launch_bounds__(kThreads) k_lora_outer(const OuterArgs a) {
    using S = Shape<RP, PARTS>;
    extern __shared__ __align__(128) uint8_t smem[];
    ptx::grid_begin(static_cast<int64_t>(a.plan.tokens) * (static_cast<int64_t>(a.side[0].n) + a.side[1].n));
    const bool second = static_cast<int>(blockIdx.x) >= a.side[0].blocks;
    const OuterSide &o = a.side[second];
    const int n0 = (blockIdx.x - (second ? a.side[0].blocks : 0)) * S::COLS;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, g = lane >> 2, t = lane & 3;
    const int half = warp >> 3, wcol = warp & 7, col = n0 + wcol * 16 * S::CT + g * S::CL, left = o.n - col;
    const int *tile_first = a.plan.words + a.plan.tile_first(), *order = a.plan.words + a.plan.order();
    const int all = adapter_tiles(a.plan), per = a.tiles(all);
    const int t0 = blockIdx.y * per, t1 = min(all, t0 + per);
    if (t0 >= t1) return;
    const uint32_t vring = ptx::smem_u32(smem), ring = vring + S::STAGES * S::V;
    const int64_t ld_vt = static_cast<int64_t>(a.plan.max_tiles()) * kLoraTile;

    // the copies' place, some steps ahead of the products': a tile, 32 tokens of it.
    // The tile and the tokens of the next copies are asked for a step before them.
    int ahead = t0, ahead_c = 0, stage_in = 0;
    Tile from = tile_at(a.plan, t0), then = tile_at(a.plan, min(t0 + 1, t1 - 1));
    int token[4];
    auto look_up = [&]() {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int m = ahead_c * kChunk + 8 * t + 4 * half + e;
            token[e] = ahead < t1 && m < from.count && left > 0 ? order[from.first + m] : -1;
        }
    };
    look_up();
    // of a lane's eight rows the warp copies four, the warp of the other half the others
    uint32_t late[4][S::CL / 2];     // rows at odd addresses: from load to store
    auto load = [&]() {
        for (int q = tid; q < PARTS * RP * (kChunk / 8); q += kThreads) {
            const int r = q / (kChunk / 8), m = q % (kChunk / 8) * 8;     // r: part and row
            ptx::cp_async16(vring + stage_in * S::V + q * 16,
                            o.vt + (r / RP) * a.plane + (r % RP) * ld_vt + static_cast<int64_t>(ahead) * kLoraTile + ahead_c * kChunk + m, 16);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int have = token[e] >= 0 ? left : 0;
            const uint16_t *p = have > 0 ? o.d + row_at(token[e], o.ld) + col : o.d;
            if constexpr (WIDE) {
                const int n = max(0, min(S::CL, have));
                const uint32_t to = ring + (((stage_in * 8 + wcol) * 8 + 4 * half + e) * 32 + lane) * (2 * S::CL);
                if constexpr (S::CL == 8) ptx::cp_async16(to, p, 2 * n);
                else ptx::cp_async8(to, p, 2 * n);
            } else if (have > 0) {
                load_cols<S::CL>(p, have, late[e]);
            } else {
#pragma unroll
                for (int i = 0; i < S::CL / 2; ++i) late[e][i] = 0u;
            }
        }
    };
    auto store_late = [&](int stage) {
        if (WIDE) return;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t to = ring + (((stage * 8 + wcol) * 8 + 4 * half + e) * 32 + lane) * (2 * S::CL);
            if constexpr (S::CL == 8) ptx::st_shared_v4(to, late[e][0], late[e][1], late[e][2], late[e][3]);
            else ptx::st_shared_v2(to, late[e][0], late[e][1]);
        }
    };
    auto step_on = [&]() {
        stage_in = stage_in + 1 == S::STAGES ? 0 : stage_in + 1;
        if (++ahead_c * kChunk >= from.count) {
            ahead_c = 0;
            ++ahead;
            from = then;
            then = tile_at(a.plan, min(ahead + 1, t1 - 1));
        }
        look_up();
    };
    for (int s = 0; s < S::STAGES - 1; ++s) {
        if (ahead < t1) {
            load();
            store_late(stage_in);
            step_on();
        }
        ptx::cp_async_commit();
    }

    float sum[S::CT][S::J][4];
    auto clear = [&]() {
#pragma unroll
        for (int i = 0; i < S::CT; ++i)
#pragma unroll
            for (int j = 0; j < S::J; ++j) sum[i][j][0] = sum[i][j][1] = sum[i][j][2] = sum[i][j][3] = 0.0f;
    };
    clear();
    int stage = 0;
    for (int i = t0; i < t1; ++i) {
        const Tile tile = tile_at(a.plan, i);
        const int begin = tile_first[tile.adapter], end = tile_first[tile.adapter + 1];
        for (int c = 0; c * kChunk < tile.count; ++c) {
            ptx::cp_async_wait<S::STAGES - 2>();
            __syncthreads();
            const int filled = ahead < t1 ? stage_in : -1;
            if (filled >= 0) {
                load();
                step_on();
            }
            ptx::cp_async_commit();
            uint32_t d[8][S::CL / 2];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t p = ring + (((stage * 8 + wcol) * 8 + e) * 32 + lane) * (2 * S::CL);
                if constexpr (S::CL == 8) ptx::ld_shared_v4(p, d[e][0], d[e][1], d[e][2], d[e][3]);
                else ptx::ld_shared_v2(p, d[e][0], d[e][1]);
            }
            // pairs of tokens: [step of 16][fragment][its four words]
            uint32_t f[2][S::CT][4];
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int k = 0; k < S::CT; ++k) {
                    f[q][k][0] = __byte_perm(d[4 * q][k], d[4 * q + 1][k], 0x5410);
                    f[q][k][1] = __byte_perm(d[4 * q][k], d[4 * q + 1][k], 0x7632);
                    f[q][k][2] = __byte_perm(d[4 * q + 2][k], d[4 * q + 3][k], 0x5410);
                    f[q][k][3] = __byte_perm(d[4 * q + 2][k], d[4 * q + 3][k], 0x7632);
                }
            // sums of 32 tokens' products, then to registers
#pragma unroll
            for (int j = 0; j < S::J; ++j) {
                uint32_t b[PARTS][4];
#pragma unroll
                for (int p = 0; p < PARTS; ++p)
                    ptx::ld_shared_v4(vring + stage * S::V + (p * RP + (half * S::J + j) * 8 + g) * (2 * kChunk) + 16 * t, b[p][0], b[p][1], b[p][2], b[p][3]);
                float acc[S::CT][4];
#pragma unroll
                for (int k = 0; k < S::CT; ++k) acc[k][0] = acc[k][1] = acc[k][2] = acc[k][3] = 0.0f;
#pragma unroll
                for (int p = 0; p < PARTS; ++p)
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int k = 0; k < S::CT; ++k) ptx::mma_bf16(acc[k], f[q][k], b[p][2 * q], b[p][2 * q + 1]);
#pragma unroll
                for (int k = 0; k < S::CT; ++k)
#pragma unroll
                    for (int q = 0; q < 4; ++q) sum[k][j][q] += acc[k][q];
            }
            if (filled >= 0) store_late(filled);
            stage = stage + 1 == S::STAGES ? 0 : stage + 1;
        }
        if (i + 1 < t1 && i + 1 < end) continue;
        // the adapter's last tile, here or at all
        const bool whole = begin >= t0 && end <= t1;
        float *part = o.ws + (2 * static_cast<int64_t>(blockIdx.y) + (begin < t0 ? 0 : 1)) * o.n * RP;
#pragma unroll
        for (int k = 0; k < S::CT; ++k)
#pragma unroll
            for (int j = 0; j < S::J; ++j) {
                const int r = (half * S::J + j) * 8 + 2 * t;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int c = col + 2 * k + e;
                    if (c >= o.n) continue;
                    const float v0 = sum[k][j][2 * e], v1 = sum[k][j][2 * e + 1];
                    if (!whole) {
                        *reinterpret_cast<float2 *>(part + static_cast<int64_t>(c) * RP + r) = make_float2(v0, v1);
                        continue;
                    }
                    const int64_t to = tile.adapter * o.stride_g + c * o.stride_n + r * o.stride_r;
                    if (a.f32) {
                        float *p = static_cast<float *>(o.out) + to;
                        if (r < a.lw.r) p[0] = v0;
                        if (r + 1 < a.lw.r) p[o.stride_r] = v1;
                    } else {
                        uint16_t *p = static_cast<uint16_t *>(o.out) + to;
                        if (r < a.lw.r) p[0] = static_cast<uint16_t>(ptx::cvt_bf16x2(v0, 0.0f));
                        if (r + 1 < a.lw.r) p[o.stride_r] = static_cast<uint16_t>(ptx::cvt_bf16x2(v1, 0.0f));
                    }
                }
            }
        clear();
    }
    ptx::cp_async_wait<0>();
}

// The adapters of several chunks, and zeros for those without a token: 32 by 32
// values through shared memory where the result's rows run the other way.
__global__ void __launch_bounds__(256) k_lora_join(const OuterArgs a, int rp) {
    __shared__ float tile[32][33];
    ptx::grid_wait();
    const OuterSide o = a.side[blockIdx.z];
    if (o.out == nullptr) return;
    const int *tile_first = a.plan.words + a.plan.tile_first();
    const int per = a.tiles(adapter_tiles(a.plan));
    const int tx = threadIdx.x & 31, ty = threadIdx.x / 32;
    for (int g = blockIdx.y; g < a.plan.adapters; g += gridDim.y) {
        const int begin = tile_first[g], end = tile_first[g + 1];
        const int c0 = begin / per, c1 = begin < end ? (end - 1) / per : c0;
        if (begin < end && c0 == c1) continue;
        for (int64_t b = static_cast<int64_t>(blockIdx.x) * 32; b < o.n; b += static_cast<int64_t>(gridDim.x) * 32) {
            for (int r0 = 0; r0 < a.lw.r; r0 += 32) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t n = b + ty + 8 * i;
                    const int r = r0 + tx;
                    float s = 0.0f;
                    if (begin < end && n < o.n && r < a.lw.r) {
                        const float *p = o.ws + ((2 * static_cast<int64_t>(c0) + 1) * o.n + n) * rp + r;
                        s = ptx::ld_f32(p);
                        p += static_cast<int64_t>(o.n) * rp;
                        for (int c = c0 + 1; c <= c1; ++c, p += 2 * static_cast<int64_t>(o.n) * rp) s += ptx::ld_f32(p);
                    }
                    tile[ty + 8 * i][tx] = s;
                }
                __syncthreads();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool along_n = o.stride_n == 1;
                    const int u = ty + 8 * i;
                    const int64_t n = b + (along_n ? tx : u);
                    const int r = r0 + (along_n ? u : tx);
                    if (n < o.n && r < a.lw.r) {
                        const float s = along_n ? tile[tx][u] : tile[u][tx];
                        const int64_t at = g * o.stride_g + n * o.stride_n + r * o.stride_r;
                        if (a.f32) static_cast<float *>(o.out)[at] = s;
                        else static_cast<uint16_t *>(o.out)[at] = static_cast<uint16_t>(ptx::cvt_bf16x2(s, 0.0f));
                    }
                }
                __syncthreads();
            }
        }
    }
}

int cols(int rp) { return rp <= 64 ? Shape<64, 2>::COLS : Shape<128, 2>::COLS; }
int blocks_of(int n, int rp) { return (n + cols(rp) - 1) / cols(rp); }

template <int RP, int PARTS, bool WIDE>
cudaError_t run(const OuterArgs &a, cudaStream_t stream) {
    static unsigned long long done;
    using S = Shape<RP, PARTS>;
    auto *kern = &k_lora_outer<RP, PARTS, WIDE>;
    const cudaError_t e = with_smem(kern, S::SMEM, S::SMEM, done);
    if (e != cudaSuccess) return e;
    return launch_after(kern, dim3(a.side[0].blocks + a.side[1].blocks, a.chunks), kThreads, S::SMEM, stream, 1, a);
}
template <int RP>
cudaError_t pick(const OuterArgs &a, bool wide, cudaStream_t stream) {
    if (a.f32) return wide ? run<RP, 3, true>(a, stream) : run<RP, 3, false>(a, stream);
    return wide ? run<RP, 2, true>(a, stream) : run<RP, 2, false>(a, stream);
}
template <int RP>
cudaError_t prep(const PrepArgs &a, cudaStream_t stream) {
    auto *kern = a.parts == 3 ? &k_lora_prep<RP, 3> : &k_lora_prep<RP, 2>;
    return launch_after(kern, dim3(a.plan.max_tiles(), 2, RP / 16), 256, 0, stream, 1, a);
}

}  // namespace

size_t outer_vt_bytes(const LoraPlan &p, int r) {
    return static_cast<size_t>(3) * padded(r) * p.max_tiles() * kLoraTile * sizeof(uint16_t);
}
// Chunks of the tiles: one round of CTAs.
int outer_chunks(const LoraPlan &p, int n, int k, int r) {
    const int rp = padded(r), slots = kSms;
    return std::max(1, std::min(p.max_tiles(), slots / (blocks_of(n, rp) + blocks_of(k, rp))));
}

cudaError_t launch_prep(const PrepArgs &a, cudaStream_t stream) {
    switch (padded(a.lw.r)) {
        case 16: return prep<16>(a, stream);
        case 32: return prep<32>(a, stream);
        case 64: return prep<64>(a, stream);
        default: return prep<128>(a, stream);
    }
}

cudaError_t launch_outer(OuterArgs &a, cudaStream_t stream) {
    const int rp = padded(a.lw.r);
    bool wide = true;
    int64_t most = 0;
    for (OuterSide &o : a.side) {
        o.blocks = o.out != nullptr ? blocks_of(o.n, rp) : 0;
        if (o.out == nullptr) continue;
        wide = wide && aligned_to(o.d, 16) && o.ld % 8 == 0;
        most = std::max<int64_t>(most, o.n);
    }
    const cudaError_t e = rp == 16   ? pick<16>(a, wide, stream)
                          : rp == 32 ? pick<32>(a, wide, stream)
                          : rp == 64 ? pick<64>(a, wide, stream)
                                     : pick<128>(a, wide, stream);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>((most + 31) / 32, 1024)), std::min(a.plan.adapters, 64), 2);
    return launch_after(&k_lora_join, grid, 256, 0, stream, 1, a, rp);
}

}  // namespace lora
}  // namespace fp8hg
