// Adapters: rows of the long side n (or k) from rows of r, y[t] = base[t] +
// s_g v[t] W_g^T.
//
// All tiles' steps of 64 columns, dealt out evenly to one round of CTAs: a warp
// takes 16 tokens of the tile, v's fragments in registers.  base, two or three steps
// ahead in shared memory, is what the products are added to (in BF16; an FP32 base is
// added after them).  Column 16 t + 2 j + e of a step is column 2 t + e of the
// fragment j, so that lane t of a row's four has 16 neighbouring columns to store.
//
// 8192 x 18944, r 16, BF16: 105 us for 620 MB, 87 % of the copy rate (loads straight
// into registers: 186 us for the whole call, now 131).  8192 x 1536, r 64: 24.5 us for
// 50 MB: a CTA has five steps of 2.5 us there, behind a chain of reads (tile, tokens, rows
// of r) that nothing covers.  Looking the next tile up meanwhile costs registers: it
// gains 2.5 us there, but loses 2 us of 17 in a call of 500 tokens.
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

template <int RP, bool TRANS, bool F32, bool WIDE>
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
    // rows at odd addresses: the aligned 16-byte granules that hold them, one more than
    // they fill, 16 rows' last ones behind the others of a warp
    static constexpr int WARP = 16 * PIECES * 16 + (WIDE ? 0 : 16 * 16);
    static constexpr int BASE = kLoraTile / 16 * WARP;
    static constexpr int SMEM = STAGES * (W + BASE);
};

template <int RP, bool TRANS, bool F32, bool WIDE, bool WAL>
__global__ void __launch_bounds__(kThreads, Shape<RP, TRANS, F32, WIDE>::CTAS) k_lora_expand(const ExpandArgs a) {
    using S = Shape<RP, TRANS, F32, WIDE>;
    extern __shared__ __align__(128) uint8_t smem[];
    ptx::grid_begin(static_cast<int64_t>(a.plan.tokens) * a.n);
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, g = lane >> 2, t = lane & 3;
    const uint32_t ring = ptx::smem_u32(smem), wbase = ring + S::STAGES * S::BASE;
    const int all = (a.n + kCols - 1) / kCols;
    const int64_t total = static_cast<int64_t>(a.plan.words[0]) * all;
    const int64_t end = total * (blockIdx.x + 1) / gridDim.x;
    const int splits = a.long_side > 0 ? shrink_splits(a.plan, adapter_tiles(a.plan), a.long_side, RP) : 1;

    for (int64_t at = total * blockIdx.x / gridDim.x; at < end;) {
        const Tile tile = tile_at(a.plan, static_cast<int>(at / all));
        const int first = static_cast<int>(at % all), steps = static_cast<int>(min(end - at, static_cast<int64_t>(all - first)));
        at += steps;
        const bool none = tile.adapter < 0, active = warp * 16 < tile.count;
        const int rank = none ? 0 : rank_of(a.lw, tile.adapter);
        const float scale = none ? 0.0f : a.lw.scale == nullptr ? 1.0f : a.lw.scale[tile.adapter];
        const uint16_t *w = a.w + (none ? 0 : tile.adapter) * a.stride_w;
        // the rows of r, the first of their sums: asked for before the tokens are known
        const float *vp = a.rows + (tile.first + warp * 16 + g) * static_cast<int64_t>(RP) + 2 * t;
        const int64_t next = static_cast<int64_t>(a.plan.tokens) * RP;
        float v[2][2 * S::KS][2];
        bool in_v[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            in_v[i] = warp * 16 + i * 8 + g < tile.count && rank > 0;
#pragma unroll
            for (int ks = 0; ks < 2 * S::KS; ++ks) {
                uint2 q = make_uint2(0u, 0u);
                if (in_v[i]) q = ptx::ld_v2(vp + i * 8 * RP + ks * 8);
                v[i][ks][0] = __uint_as_float(q.x);
                v[i][ks][1] = __uint_as_float(q.y);
            }
        }
        int token[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int m = warp * 16 + i * 8 + g;
            token[i] = m < tile.count ? a.plan.words[a.plan.order() + tile.first + m] : -1;
        }
        // the rows that the lane copies: a granule of each, and the last one of a row
        constexpr int E = F32 ? 4 : 8, ES = 16 / E;      // elements of a granule, their size
        const int64_t n0 = static_cast<int64_t>(first) * kCols;
        constexpr int COPIES = 16 / S::ROWS + (WIDE ? 0 : 1);
        const uint8_t *row[COPIES];
        int ahead[COPIES];      // bytes from the granule to the first column
        bool in[COPIES];
        const bool with_base = active && a.base != nullptr;
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
            const bool last = i == 16 / S::ROWS;
            const int m = warp * 16 + (last ? lane & 15 : i * S::ROWS + lane / S::PIECES);
            row[i] = nullptr;
            ahead[i] = 0;
            in[i] = false;
            if (m < tile.count && with_base && (!last || lane < 16)) {
                const uintptr_t at = reinterpret_cast<uintptr_t>(a.base) +
                                     (row_at(a.plan.words[a.plan.order() + tile.first + m], a.ld_base) + n0) * ES;
                const int s = WIDE ? 0 : static_cast<int>(at & 15), p = last ? S::PIECES : lane % S::PIECES;
                row[i] = reinterpret_cast<const uint8_t *>(at - s + p * 16);
                ahead[i] = s - p * 16;
                in[i] = true;
            }
        }
        TileCopy<TRANS ? RP : kCols, TRANS ? kCols : RP, S::ROW, !TRANS, WAL> wc(w + (TRANS ? n0 : n0 * a.ld_w), a.ld_w, TRANS ? rank : kCols,
                                                                                 TRANS ? kCols : rank);
        const int64_t wstep = TRANS ? kCols : static_cast<int64_t>(kCols) * a.ld_w;
        int in_stage = 0, left = static_cast<int>(a.n - n0);      // of the next copies
        auto load = [&]() {
            if (rank > 0) wc.copy(wbase + in_stage * S::W, a.w, TRANS ? RP : left, TRANS ? left : RP, wstep);
            if (with_base) {
                const int bytes = ES * min(kCols, left);
#pragma unroll
                for (int i = 0; i < COPIES; ++i) {
                    const bool last = i == 16 / S::ROWS;
                    // a granule is read whole if a byte of it belongs to the row
                    const int have = !in[i] ? 0 : WIDE ? bytes - lane % S::PIECES * 16 : bytes + ahead[i];
                    const int n = WIDE ? max(0, min(16, have)) : have > 0 ? 16 : 0;
                    const uint32_t to = ring + in_stage * S::BASE + warp * S::WARP +
                                        (last ? 16 * S::PIECES * 16 + lane * 16
                                              : slot<S::PIECES>(i * S::ROWS + lane / S::PIECES, lane % S::PIECES));
                    if (!last || lane < 16) ptx::cp_async16(to, n > 0 ? row[i] : norm::base_granule(a.base), n);
                    row[i] += kCols * ES;
                }
            }
            left -= kCols;
            in_stage = in_stage + 1 == S::STAGES ? 0 : in_stage + 1;
        };
        for (int s = 0; s < S::STAGES - 1; ++s) {
            if (s < steps) load();
            ptx::cp_async_commit();
        }

        uint32_t f[S::PARTS][S::KS][4];
        // partial sums in their order, U splits' loads in flight
        constexpr int U = S::KS <= 4 ? 8 / S::KS : 1;
        for (int s0 = 1; s0 < splits && active && rank > 0; s0 += U) {
            uint2 q[U][2][2 * S::KS];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int ks = 0; ks < 2 * S::KS; ++ks) {
                        q[u][i][ks] = make_uint2(0u, 0u);
                        if (s0 + u < splits && in_v[i]) q[u][i][ks] = ptx::ld_v2(vp + (s0 + u) * next + i * 8 * RP + ks * 8);
                    }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int ks = 0; ks < 2 * S::KS; ++ks) {
                        v[i][ks][0] += __uint_as_float(q[u][i][ks].x);
                        v[i][ks][1] += __uint_as_float(q[u][i][ks].y);
                    }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int ks = 0; ks < 2 * S::KS; ++ks) {
                const int r = ks * 8 + 2 * t;
                const float v0 = r < rank ? v[i][ks][0] : 0.0f, v1 = r + 1 < rank ? v[i][ks][1] : 0.0f;
                if (a.v_out != nullptr && first == 0 && token[i] >= 0) {
                    float *to = a.v_out + row_at(token[i], a.ld_v) + r;
                    if (r < a.lw.r) to[0] = v0;
                    if (r + 1 < a.lw.r) to[1] = v1;
                }
                uint32_t lo[S::PARTS], hi[S::PARTS];
                lora::split<S::PARTS>(v0 * scale, lo);
                lora::split<S::PARTS>(v1 * scale, hi);
#pragma unroll
                for (int p = 0; p < S::PARTS; ++p) f[p][ks >> 1][i + 2 * (ks & 1)] = lo[p] | hi[p] << 16;
            }

        // the lane's places of the weights: rows of two neighbouring terms, 16 columns each,
        // or column i of fragment j, row 16 (i / 2) + 2 j + (i & 1)
        const int wi = lane & 7;
        const uint32_t wlane = wbase + (TRANS ? 2 * t * S::ROW + 32 * (g >> 1)
                                              : (16 * (wi >> 1) + 2 * (lane >> 4) + (wi & 1)) * S::ROW + (wi >> 1) * 32 + ((lane >> 3) & 1) * 16);
        int64_t yat[2];
        uint32_t shift[2];      // of the lane's rows of base within their granules
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            yat[i] = token[i] >= 0 ? row_at(token[i], a.ld_y) + n0 + 16 * t : 0;
            shift[i] = static_cast<uint32_t>(norm::column_address<F32>(a.base, token[i] >= 0 ? row_at(token[i], a.ld_base) : 0)) & 15u;
        }
        int stage = 0, out_left = static_cast<int>(a.n - n0) - 16 * t;
        for (int s = 0; s < steps; ++s) {
            ptx::cp_async_wait<S::STAGES - 2>();
            __syncthreads();
            const bool more = s + S::STAGES - 1 < steps;
            if (more) load();
            ptx::cp_async_commit();
            if (active) {
                const uint32_t wat = wlane + stage * S::W;
                norm::Raw<F32> old[2];
                float acc[8][4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    old[i].zero();
                    if (with_base) {
                        const uint32_t from = ring + stage * S::BASE + warp * S::WARP;
                        constexpr int N = S::PIECES / 4;
                        uint32_t u[4 * (N + 1)];
#pragma unroll
                        for (int h = 0; h < N + (WIDE ? 0 : 1); ++h) {
                            const int p = t * N + h;
                            const uint32_t at = p < S::PIECES ? slot<S::PIECES>(i * 8 + g, p) : 16 * S::PIECES * 16 + (i * 8 + g) * 16;
                            ptx::ld_shared_v4(from + at, u[4 * h], u[4 * h + 1], u[4 * h + 2], u[4 * h + 3]);
                        }
                        if constexpr (!WIDE && F32) ragged::shift_words(u, shift[i] >> 2);
                        else if constexpr (!WIDE) ragged::shift_down(u, shift[i]);
#pragma unroll
                        for (int h = 0; h < 4 * N; ++h) old[i].w[h] = u[h];
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const F2 p = old[i].pair(j);
                        acc[j][2 * i] = F32 ? 0.0f : p.lo();
                        acc[j][2 * i + 1] = F32 ? 0.0f : p.hi();
                    }
                }
                if (rank > 0) {
#pragma unroll
                    for (int ks = 0; ks < S::KS; ++ks) {
                        uint32_t b[8][2];
                        if constexpr (TRANS) {
                            uint32_t u[4][8];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t p = wat + (ks * 16 + (e & 1) + (e >> 1) * 8) * S::ROW;
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
                                uint32_t m[4];
                                ptx::ldmatrix_x4<false>(wat + 2 * j * S::ROW + ks * 32, m);
                                b[j][0] = m[0], b[j][1] = m[1], b[j + 1][0] = m[2], b[j + 1][1] = m[3];
                            }
                        }
#pragma unroll
                        for (int p = 0; p < S::PARTS; ++p)
#pragma unroll
                            for (int j = 0; j < 8; ++j) ptx::mma_bf16(acc[j], f[p][ks], b[j][0], b[j][1]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    F2 out[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        out[j] = f2(acc[j][2 * i], acc[j][2 * i + 1]);
                        if constexpr (F32) out[j] = add2(old[i].pair(j), out[j]);
                    }
                    norm::store_values<WIDE>(a.y, F32, yat[i], token[i] >= 0 ? out_left : 0, out);
                    yat[i] += kCols;
                }
                out_left -= kCols;
            }
            stage = stage + 1 == S::STAGES ? 0 : stage + 1;
        }
        ptx::cp_async_wait<0>();
        __syncthreads();      // before the next tile's copies
    }
}

template <int RP, bool TRANS, bool F32, bool WIDE, bool WAL>
cudaError_t run(const ExpandArgs &a, cudaStream_t stream) {
    using S = Shape<RP, TRANS, F32, WIDE>;
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
