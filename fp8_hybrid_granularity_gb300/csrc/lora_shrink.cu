// Adapters: rows of r from rows of the long side k (or n), out[t] = x[t] W_g^T.
//
// A CTA takes a tile of up to 128 tokens, 16 a warp, and a part of the long side
// (partial sums in FP32; the kernels behind add them in a fixed order), 64
// columns a step.  W's tile of a step is shared by the warps.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "lora.cuh"

namespace fp8hg {
namespace lora {

namespace {

constexpr int kThreads = kLoraTile / 16 * 32;
constexpr int kCols = kShrinkCols;

template <int RP, bool TRANS>
struct Shape {
    static constexpr int STAGES = RP <= 32 ? 3 : RP <= 64 ? 4 : 6;
    static constexpr int CTAS = shrink_slots(RP) / kSms;
    static constexpr int ROW = TRANS ? 2 * RP + 16 : 2 * kCols + 16;
    // 32 bytes more after every 16 rows of the transposed form: its fragments
    // take every sixteenth row
    static constexpr int W = TRANS ? kCols * ROW + kCols / 16 * 32 : RP * ROW;
    static constexpr int X = kLoraTile * kCols * 2;
    static constexpr int SMEM = STAGES * (W + X);
};

template <int RP, bool TRANS, bool WIDE, bool WAL>
__global__ void __launch_bounds__(kThreads, Shape<RP, TRANS>::CTAS) k_lora_shrink(const ShrinkArgs a) {
    using S = Shape<RP, TRANS>;
    extern __shared__ __align__(128) uint8_t smem[];
    ptx::grid_begin(static_cast<int64_t>(a.plan.tokens) * a.k);
    const Tile tile = tile_at(a.plan, blockIdx.x);      // its place is there, if it is a tile or not
    const int tiles = adapter_tiles(a.plan);
    const int splits = shrink_splits(tiles, a.k, RP);
    if (static_cast<int>(blockIdx.x) >= tiles || static_cast<int>(blockIdx.y) >= splits) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, g = lane >> 2, t = lane & 3;
    const int rank = rank_of(a.lw, tile.adapter);
    const uint16_t *w = a.w + tile.adapter * a.stride_w;
    const uint32_t ring = ptx::smem_u32(smem), base = ring + S::STAGES * S::X;
    const int all = (a.k + kCols - 1) / kCols, per = (all + splits - 1) / splits;
    const int first = blockIdx.y * per, steps = min(all - first, per);

    // the rows that the lane copies: every fourth of the warp's (those it reads, at odd addresses)
    const uint16_t *row[4];
    bool have[4];
#pragma unroll
    for (int i = 0; i < (WIDE ? 4 : 2); ++i) {
        const int m = warp * 16 + (WIDE ? i * 4 + lane / 8 : i * 8 + g);
        have[i] = m < tile.count;
        row[i] = a.x;
        if (have[i])
            row[i] += row_at(a.plan.words[a.plan.order() + tile.first + m], a.ld_x) + (WIDE ? lane % 8 * 8 : 16 * t) + first * kCols;
    }
    const bool active = warp * 16 < tile.count;
    const int64_t k0 = static_cast<int64_t>(first) * kCols;
    TileCopy<TRANS ? kCols : RP, TRANS ? RP : kCols, S::ROW, TRANS, WAL> wc(w + (TRANS ? k0 * a.ld_w : k0), a.ld_w, TRANS ? kCols : rank,
                                                                             TRANS ? rank : kCols);
    const int64_t wstep = TRANS ? static_cast<int64_t>(kCols) * a.ld_w : kCols;
    int in_stage = 0, left = a.k - first * kCols;      // of the next copies
    uint32_t late[2][8];     // rows at odd addresses: from load to store
    auto load = [&]() {
        wc.copy(base + in_stage * S::W, a.w, TRANS ? left : RP, TRANS ? RP : left, wstep);
        if (active) {
            if constexpr (WIDE) {
                const int n = max(0, min(16, 2 * (left - lane % 8 * 8)));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    ptx::cp_async16(ring + in_stage * S::X + slot<8>(i * 4 + lane / 8, lane % 8), have[i] && n > 0 ? row[i] : a.x, have[i] ? n : 0);
                    row[i] += kCols;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int n = have[i] ? left - 16 * t : 0;
                    if (n > 0) {
                        ragged::load16<false>(row[i], n, late[i]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) late[i][j] = 0u;
                    }
                    row[i] += kCols;
                }
            }
        }
        left -= kCols;
    };
    auto store_late = [&]() {
        if (!WIDE && active) {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const uint32_t(&v)[8] = late[p / 2];
                const int h = p % 2 * 4;
                ptx::st_shared_v4(ring + in_stage * S::X + slot<8>(p / 2 * 8 + g, 2 * t + p % 2), v[h], v[h + 1], v[h + 2], v[h + 3]);
            }
        }
        in_stage = in_stage + 1 == S::STAGES ? 0 : in_stage + 1;
    };
    for (int s = 0; s < S::STAGES - 1; ++s) {
        if (s < steps) {
            load();
            store_late();
        }
        ptx::cp_async_commit();
    }
    float sum[RP / 8][4];
#pragma unroll
    for (int j = 0; j < RP / 8; ++j) sum[j][0] = sum[j][1] = sum[j][2] = sum[j][3] = 0.0f;
    // the lane's places: of x; of W rows j * 8 + g, or of row 16 (i / 2) + (i & 1), and
    // 2 on: a lane's terms
    const uint32_t xat = ring + slot<8>(g, 2 * t);
    const int wi = lane & 7;
    const uint32_t wat = base + (TRANS ? (16 * (wi >> 1) + (wi & 1) + 2 * ((lane >> 3) & 1)) * S::ROW + (wi >> 1) * 32 + (lane >> 4) * 16
                                       : g * S::ROW + 32 * t);
    int stage = 0;
    for (int s = 0; s < steps; ++s) {
        ptx::cp_async_wait<S::STAGES - 2>();
        __syncthreads();
        const bool more = s + S::STAGES - 1 < steps;
        if (more) load();
        ptx::cp_async_commit();
        if (active) {
            const uint32_t at = wat + stage * S::W, xp = xat + stage * S::X;
            uint32_t f[2][8];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                ptx::ld_shared_v4(xp + i * 8 * 128, f[i][0], f[i][1], f[i][2], f[i][3]);
                ptx::ld_shared_v4((xp ^ 16) + i * 8 * 128, f[i][4], f[i][5], f[i][6], f[i][7]);
            }
            // sums of 64 products, then to registers
            auto products = [&](int j, const uint32_t (&b)[8]) {
                float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t fa[4] = {f[0][2 * q], f[1][2 * q], f[0][2 * q + 1], f[1][2 * q + 1]};
                    ptx::mma_bf16(acc, fa, b[2 * q], b[2 * q + 1]);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) sum[j][q] += acc[q];
            };
            if constexpr (TRANS) {
#pragma unroll
                for (int jj = 0; jj < RP / 16; ++jj) {
                    uint32_t b0[8], b1[8];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t m[4];
                        ptx::ldmatrix_x4<true>(at + q * 4 * S::ROW + jj * 32, m);
                        b0[2 * q] = m[0], b0[2 * q + 1] = m[1], b1[2 * q] = m[2], b1[2 * q + 1] = m[3];
                    }
                    products(2 * jj, b0);
                    products(2 * jj + 1, b1);
                }
            } else {
#pragma unroll
                for (int j = 0; j < RP / 8; ++j) {
                    uint32_t b[8];
                    ptx::ld_shared_v4(at + j * 8 * S::ROW, b[0], b[1], b[2], b[3]);
                    ptx::ld_shared_v4(at + j * 8 * S::ROW + 16, b[4], b[5], b[6], b[7]);
                    products(j, b);
                }
            }
        }
        if (more) store_late();
        stage = stage + 1 == S::STAGES ? 0 : stage + 1;
    }
    ptx::cp_async_wait<0>();
    float *out = a.out + (static_cast<int64_t>(blockIdx.y) * a.plan.tokens + tile.first) * RP;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int m = warp * 16 + h * 8 + g;
        if (m < tile.count) {
#pragma unroll
            for (int j = 0; j < RP / 8; ++j)
                *reinterpret_cast<float2 *>(out + m * RP + j * 8 + 2 * t) = make_float2(sum[j][2 * h], sum[j][2 * h + 1]);
        }
    }
}

template <int RP, bool TRANS, bool WIDE, bool WAL>
cudaError_t run(const ShrinkArgs &a, cudaStream_t stream) {
    using S = Shape<RP, TRANS>;
    static unsigned long long done;
    auto *kern = &k_lora_shrink<RP, TRANS, WIDE, WAL>;
    const cudaError_t e = with_smem(kern, S::SMEM, S::SMEM, done);
    if (e != cudaSuccess) return e;
    return launch_after(kern, dim3(a.plan.max_tiles(), most_splits(a.plan, a.k, RP)), kThreads, S::SMEM, stream, 1, a);
}
template <int RP, bool TRANS>
cudaError_t pick(const ShrinkArgs &a, cudaStream_t stream) {
    const bool wide = aligned_to(a.x, 16) && a.ld_x % 8 == 0;
    const bool wal = aligned_to(a.w, 16) && a.ld_w % 8 == 0 && a.stride_w % 8 == 0;
    if (wide) return wal ? run<RP, TRANS, true, true>(a, stream) : run<RP, TRANS, true, false>(a, stream);
    return wal ? run<RP, TRANS, false, true>(a, stream) : run<RP, TRANS, false, false>(a, stream);
}
template <bool TRANS>
cudaError_t by_rank(const ShrinkArgs &a, cudaStream_t stream) {
    switch (padded(a.lw.r)) {
        case 16: return pick<16, TRANS>(a, stream);
        case 32: return pick<32, TRANS>(a, stream);
        case 64: return pick<64, TRANS>(a, stream);
        default: return pick<128, TRANS>(a, stream);
    }
}

}  // namespace

cudaError_t launch_shrink(const ShrinkArgs &a, bool trans, cudaStream_t stream) {
    return trans ? by_rank<true>(a, stream) : by_rank<false>(a, stream);
}

}  // namespace lora
}  // namespace fp8hg
