// Adapters: rows of the long side n (or k) from rows of r, y[t] = base[t] +
// s_g v[t] W_g^T.
//
// All tiles' steps of 64 columns, dealt out evenly to one round of CTAs: a warp
// takes 16 tokens of the tile, v's fragments in registers.  base is what the
// products are added to (in BF16; an FP32 base is added after them); column 16 t + 2 j + e of a step is column 2 t + e of the
// fragment j, so that lane t of a row's four has 16 neighbouring columns to store.
#pragma once
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "lora.cuh"

namespace fp8hg {
namespace lora {

namespace {

constexpr int kThreads = kLoraTile / 16 * 32;
constexpr int kCols = 64;

template <int RP, bool TRANS, bool F32>
struct Shape {
    static constexpr int KS = RP / 16;
    static constexpr int PARTS = F32 ? 3 : 2;
    static constexpr int PIECES = F32 ? 16 : 8;              // of a row's 64 columns, 16 bytes each
    static constexpr int ROWS = 32 / PIECES;                 // of a warp's copy
    static constexpr int CTAS = F32 || RP > 64 ? 1 : RP > 16 ? 2 : 3;
    static constexpr int STAGES = CTAS == 3 ? 3 : 4;
    static constexpr int ROW = TRANS ? 2 * kCols + 16 : 2 * RP + 16;
    // 32 bytes more after every 16 rows: a fragment takes two of every sixteen
    static constexpr int W = TRANS ? RP * ROW : kCols * ROW + kCols / 16 * 32;
    static constexpr int BASE = kLoraTile * PIECES * 16;
    static constexpr int SMEM = STAGES * (W + BASE);
};

template <int RP, bool TRANS, bool F32, bool WIDE, bool WAL>
__global__ void __launch_bounds__(kThreads, Shape<RP, TRANS, F32>::CTAS) k_lora_expand(const ExpandArgs a) {
    using S = Shape<RP, TRANS, F32>;
    extern __shared__ __align__(128) uint8_t smem[];
    ptx::grid_begin(static_cast<int64_t>(a.plan.tokens) * a.n);
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, g = lane >> 2, t = lane & 3;
    const uint32_t ring = ptx::smem_u32(smem), wbase = ring + S::STAGES * S::BASE;
    const int all = (a.n + kCols - 1) / kCols;
    const int64_t total = static_cast<int64_t>(a.plan.words[0]) * all;
    const int64_t end = total * (blockIdx.x + 1) / gridDim.x;
    const int splits = a.long_side > 0 ? shrink_splits(adapter_tiles(a.plan), a.long_side, RP) : 1;

    for (int64_t at = total * blockIdx.x / gridDim.x; at < end;) {
        const Tile tile = tile_at(a.plan, static_cast<int>(at / all));
        const int first = static_cast<int>(at % all), steps = static_cast<int>(min(end - at, static_cast<int64_t>(all - first)));
        at += steps;
        const bool none = tile.adapter < 0, active = warp * 16 < tile.count;
        const int rank = none ? 0 : rank_of(a.lw, tile.adapter);
        const float scale = none ? 0.0f : a.lw.scale == nullptr ? 1.0f : a.lw.scale[tile.adapter];
        const uint16_t *w = a.w + (none ? 0 : tile.adapter) * a.stride_w;
        int token[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int m = warp * 16 + i * 8 + g;
            token[i] = m < tile.count ? a.plan.words[a.plan.order() + tile.first + m] : -1;
        }
        // the rows that the lane copies
        const uint8_t *row[16 / S::ROWS];
        if constexpr (WIDE) {
#pragma unroll
            for (int i = 0; i < 16 / S::ROWS; ++i) {
                const int m = warp * 16 + i * S::ROWS + lane / S::PIECES;
                row[i] = nullptr;
                if (m < tile.count && a.base != nullptr)
                    row[i] = static_cast<const uint8_t *>(a.base) + row_at(a.plan.words[a.plan.order() + tile.first + m], a.ld_base) * (F32 ? 4 : 2) +
                             lane % S::PIECES * 16;
            }
        }
        norm::Raw<F32> late[2];      // rows at odd addresses: from load to store
        auto load = [&](int step) {
            const int stage = step % S::STAGES, n = (first + step) * kCols, left = a.n - n;
            const uint32_t to = wbase + stage * S::W;
            if (rank > 0) {
                if constexpr (TRANS) {
                    for (int i = threadIdx.x; i < RP * (kCols / 8); i += kThreads) {
                        const int r = i / (kCols / 8), c = i % (kCols / 8) * 8;
                        const bool in = r < rank && c < left;
                        copy8<WAL>(to + r * S::ROW + 2 * c, in ? w + row_at(r, a.ld_w) + n + c : a.w, in ? left - c : 0);
                    }
                } else {
                    for (int i = threadIdx.x; i < kCols * (RP / 8); i += kThreads) {
                        const int r = i / (RP / 8), c = i % (RP / 8) * 8;
                        const bool in = r < left && c < rank;
                        copy8<WAL>(to + r * S::ROW + r / 16 * 32 + 2 * c, in ? w + row_at(n + r, a.ld_w) + c : a.w, in ? rank - c : 0);
                    }
                }
            }
            if (!active || a.base == nullptr) return;
            if constexpr (WIDE) {
                constexpr int E = F32 ? 4 : 8;     // elements of a piece
                const int c = max(0, min(E, left - lane % S::PIECES * E));
#pragma unroll
                for (int i = 0; i < 16 / S::ROWS; ++i) {
                    const bool in = row[i] != nullptr && c > 0;
                    ptx::cp_async16(slot<S::PIECES>(ring, stage, i * S::ROWS + lane / S::PIECES, lane % S::PIECES),
                                    in ? row[i] + static_cast<int64_t>(n) * (16 / E) : static_cast<const uint8_t *>(a.base), in ? c * (16 / E) : 0);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int have = token[i] < 0 ? 0 : left - 16 * t;
                    if (have > 0) late[i].template load<false>(a.base, row_at(token[i], a.ld_base) + n + 16 * t, have);
                    else late[i].zero();
                }
            }
        };
        auto store_late = [&](int step) {
            if (WIDE || !active || a.base == nullptr) return;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int p = 0; p < S::PIECES / 4; ++p) {
                    const uint32_t *v = late[i].w + 4 * p;
                    ptx::st_shared_v4(slot<S::PIECES>(ring, step % S::STAGES, i * 8 + g, t * (S::PIECES / 4) + p), v[0], v[1], v[2], v[3]);
                }
        };
        for (int s = 0; s < S::STAGES - 1; ++s) {
            if (s < steps) {
                load(s);
                store_late(s);
            }
            ptx::cp_async_commit();
        }

        uint32_t f[S::PARTS][S::KS][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int ks = 0; ks < 2 * S::KS; ++ks) {
                const int r = ks * 8 + 2 * t;
                float v[2] = {0.0f, 0.0f};
                if (token[i] >= 0 && r < rank) {
                    const float *p = a.rows + (tile.first + warp * 16 + i * 8 + g) * static_cast<int64_t>(RP) + r;
                    for (int s = 0; s < splits; ++s, p += static_cast<int64_t>(a.plan.tokens) * RP) {
                        const uint2 q = ptx::ld_v2(p);
                        v[0] += __uint_as_float(q.x), v[1] += __uint_as_float(q.y);
                    }
                    if (r + 1 >= rank) v[1] = 0.0f;
                }
                if (a.v_out != nullptr && first == 0 && token[i] >= 0) {
                    float *to = a.v_out + row_at(token[i], a.ld_v) + r;
                    if (r < a.lw.r) to[0] = v[0];
                    if (r + 1 < a.lw.r) to[1] = v[1];
                }
                uint32_t lo[S::PARTS], hi[S::PARTS];
                split<S::PARTS>(v[0] * scale, lo);
                split<S::PARTS>(v[1] * scale, hi);
#pragma unroll
                for (int p = 0; p < S::PARTS; ++p) f[p][ks >> 1][i + 2 * (ks & 1)] = lo[p] | hi[p] << 16;
            }

        for (int s = 0; s < steps; ++s) {
            ptx::cp_async_wait<S::STAGES - 2>();
            __syncthreads();
            const bool more = s + S::STAGES - 1 < steps;
            if (more) load(s + S::STAGES - 1);
            ptx::cp_async_commit();
            if (!active) continue;
            const int stage = s % S::STAGES;
            const uint32_t wat = wbase + stage * S::W;
            norm::Raw<F32> in[2];
            float acc[8][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                in[i].zero();
                if (a.base != nullptr) {
#pragma unroll
                    for (int h = 0; h < S::PIECES / 4; ++h)
                        ptx::ld_shared_v4(slot<S::PIECES>(ring, stage, i * 8 + g, t * (S::PIECES / 4) + h), in[i].w[4 * h], in[i].w[4 * h + 1],
                                          in[i].w[4 * h + 2], in[i].w[4 * h + 3]);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const F2 p = in[i].pair(j);
                    acc[j][2 * i] = F32 ? 0.0f : p.lo();
                    acc[j][2 * i + 1] = F32 ? 0.0f : p.hi();
                }
            }
            if (rank > 0) {
#pragma unroll
                for (int ks = 0; ks < S::KS; ++ks) {
                    uint32_t b[8][2];
                    if constexpr (TRANS) {
                        // rows of two neighbouring terms, 16 columns each: the lane's column of a pair
                        uint32_t u[4][8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t p = wat + (ks * 16 + 2 * t + (e & 1) + (e >> 1) * 8) * S::ROW + 32 * (g >> 1);
                            ptx::ld_shared_v4(p, u[e][0], u[e][1], u[e][2], u[e][3]);
                            ptx::ld_shared_v4(p + 16, u[e][4], u[e][5], u[e][6], u[e][7]);
                        }
                        const uint32_t sel = g & 1 ? 0x7632u : 0x5410u;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            b[j][0] = __byte_perm(u[0][j], u[1][j], sel);
                            b[j][1] = __byte_perm(u[2][j], u[3][j], sel);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; j += 2) {
                            // column i of fragment j: row 16 (i / 2) + 2 j + (i & 1)
                            const int i = lane & 7, r = 16 * (i >> 1) + 2 * (j + (lane >> 4)) + (i & 1);
                            uint32_t m[4];
                            ptx::ldmatrix_x4<false>(wat + r * S::ROW + r / 16 * 32 + (ks * 16 + ((lane >> 3) & 1) * 8) * 2, m);
                            b[j][0] = m[0], b[j][1] = m[1], b[j + 1][0] = m[2], b[j + 1][1] = m[3];
                        }
                    }
#pragma unroll
                    for (int p = 0; p < S::PARTS; ++p)
#pragma unroll
                        for (int j = 0; j < 8; ++j) ptx::mma_bf16(acc[j], f[p][ks], b[j][0], b[j][1]);
                }
            }
            const int c = (first + s) * kCols + 16 * t;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                F2 out[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    out[j] = f2(acc[j][2 * i], acc[j][2 * i + 1]);
                    if constexpr (F32) out[j] = add2(in[i].pair(j), out[j]);
                }
                norm::store_values<WIDE>(a.y, F32, token[i] >= 0 ? row_at(token[i], a.ld_y) + c : 0, token[i] >= 0 ? a.n - c : 0, out);
            }
            if (more) store_late(s + S::STAGES - 1);
        }
        ptx::cp_async_wait<0>();
        __syncthreads();      // before the next tile's copies
    }
}

template <int RP, bool TRANS, bool F32, bool WIDE, bool WAL>
cudaError_t run(const ExpandArgs &a, cudaStream_t stream) {
    using S = Shape<RP, TRANS, F32>;
    static unsigned long long done;
    auto *kern = &k_lora_expand<RP, TRANS, F32, WIDE, WAL>;
    const cudaError_t e = with_smem(kern, S::SMEM, S::SMEM, done);
    if (e != cudaSuccess) return e;
    const int64_t most = static_cast<int64_t>(a.plan.max_tiles()) * ((static_cast<int64_t>(a.n) + kCols - 1) / kCols);
    return launch_after(kern, dim3(static_cast<unsigned>(std::min<int64_t>(most, S::CTAS * kSms))), kThreads, S::SMEM, stream, 1, a);
}
template <int RP, bool TRANS, bool F32>
cudaError_t pick(const ExpandArgs &a, cudaStream_t stream) {
    const bool wide = norm::wide_rows(a.y, F32, a.ld_y) && (a.base == nullptr || norm::wide_rows(a.base, F32, a.ld_base));
    const bool wal = aligned_to(a.w, 16) && a.ld_w % 8 == 0 && a.stride_w % 8 == 0;
    if (wide) return wal ? run<RP, TRANS, F32, true, true>(a, stream) : run<RP, TRANS, F32, true, false>(a, stream);
    return wal ? run<RP, TRANS, F32, false, true>(a, stream) : run<RP, TRANS, F32, false, false>(a, stream);
}
// One direction's kernels (TRANS: the weights' rows are the rows of r).
template <bool TRANS, bool F32>
cudaError_t by_rank(const ExpandArgs &a, cudaStream_t stream) {
    switch (padded(a.lw.r)) {
        case 16: return pick<16, TRANS, F32>(a, stream);
        case 32: return pick<32, TRANS, F32>(a, stream);
        case 64: return pick<64, TRANS, F32>(a, stream);
        default: return pick<128, TRANS, F32>(a, stream);
    }
}

}  // namespace
}  // namespace lora
}  // namespace fp8hg
