// Adapters: rows of r from rows of the long side k (or n), out[t] = x[t] W_g^T.
//
// A CTA takes a tile of up to 128 tokens, the rows of a tcgen05.mma, and a part of the
// long side (partial sums in FP32; the kernels behind add them in a fixed order), 64
// columns a step; the rows of r are its columns.  W's tile is an operand with its K
// (A_g) or its rows (B_g, in the backward pass) next to one another.  Steps take
// turns at the sums in tensor memory, up to 512 columns of it, so that a sum is cut
// off only 4 times in as many steps as there are sums; they are added at the end.
// Rows past a tile's tokens, and past an adapter's rank, hold anything: they meet no
// other row's sums, and nobody reads theirs.
//
// Bound by HBM: 8192 x 8960, r 64, takes 29.5 us, 74 % of the copy rate (rows copied
// by the warps: 36; mma.sync fed through registers: 52); r 16, 8192 x 3584: 16 us.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "lora.cuh"

namespace fp8hg {
namespace lora {

namespace {

constexpr int kCols = kShrinkCols;
constexpr int kCopyWarps = 4;        // these read the sums at the end: a token a lane
constexpr int kThreads = (kCopyWarps + 1) * 32;

template <int RP, bool TRANS>
struct Shape {
    // transposed: whole rows of 128 bytes, so 64 rows of r at least
    static constexpr int N = TRANS && RP < 64 ? 64 : RP;
    static constexpr int X = kLoraTile * 128, W = TRANS ? (N / 64) * kCols * 128 : N * 128;
    static constexpr int STAGES = 216 * 1024 / (X + W) < 8 ? 216 * 1024 / (X + W) : 8;
    static constexpr int SUMS = shrink_sums(RP);
    static constexpr int TMEM = SUMS * N;      // 128, 256 or 512 columns
    static constexpr int BARS = 8 * (2 * STAGES + 1);
    static constexpr int SMEM = 1024 + STAGES * (X + W) + BARS + 16;
    // pieces of 16 bytes of W's tile, a thread
    static constexpr int P = TRANS ? RP / 8 : 8, ROWS = TRANS ? kCols : RP, PIECES = ROWS * P / (kCopyWarps * 32);
};

// WIDE, WAL: rows of x, and W, that TMA takes (16-byte multiples).  A tile whose tokens are
// neighbours is copied by it; rows that are not, by the warps.  (TMA's own gather
// takes 82 us where the warps take 36, at 8192 x 8960, r 64.)
template <int RP, bool TRANS, bool WIDE, bool WAL>
__global__ void __launch_bounds__(kThreads, 1)
    k_lora_shrink(const ShrinkArgs a, const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w) {
    using S = Shape<RP, TRANS>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    ptx::grid_begin(static_cast<int64_t>(a.plan.tokens) * a.k);
    Tile tile = tile_at(a.plan, blockIdx.x);      // its place is there, if it is a tile or not
    if (a.packed) tile.row = tile.first;
    const int tiles = adapter_tiles(a.plan), splits = shrink_splits(a.plan, tiles, a.k, RP);
    if (static_cast<int>(blockIdx.x) >= tiles || static_cast<int>(blockIdx.y) >= splits) return;
    const int all = (a.k + kCols - 1) / kCols, per = (all + splits - 1) / splits;
    const int first = blockIdx.y * per, steps = min(all - first, per);

    const uint32_t raw = ptx::smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    const uint32_t sx = base, sw = base + S::STAGES * S::X, full = sw + S::STAGES * S::W;
    const uint32_t empty = full + 8 * S::STAGES, done = empty + 8 * S::STAGES;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem_raw + (full + S::BARS - raw));
    volatile uint32_t *abort_flag = tmem_slot + 1;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::STAGES; ++i) {
            ptx::mbar_init(full + 8 * i, kCopyWarps + 1);
            ptx::mbar_init(empty + 8 * i, 1);
        }
        ptx::mbar_init(done, 1);
        *abort_flag = 0u;
        ptx::fence_mbar_init();
    }
    if (warp == kCopyWarps) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), S::TMEM);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xFFFFFFFFu, gemm_common::wait_phase(bar, parity, kWaitNs, abort_flag, a.err, 0x20u + warp));
    };

    if (warp < kCopyWarps) {
        // rows of x: eight lanes each, 32 of them a warp
        const int piece = lane % 8, m0 = warp * 32 + lane / 8;
        const int64_t k0 = static_cast<int64_t>(first) * kCols;
        const uint16_t *row[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int m = m0 + 4 * e;
            const int at = tile.first + m;
            row[e] = m < tile.count ? a.x + row_at(a.packed ? at : a.plan.words[a.plan.order() + at], a.ld_x) + k0 + piece * 8 : nullptr;
        }
        // pieces of W: rows of r, or of the long side
        const int rank = rank_of(a.lw, tile.adapter), tid = threadIdx.x, wc = tid % S::P * 8;
        const uint16_t *w = a.w + tile.adapter * a.stride_w + (TRANS ? k0 * a.ld_w : k0) + wc;
        const uint16_t *wrow[S::PIECES];
        uint32_t wto[S::PIECES];
#pragma unroll
        for (int i = 0; i < S::PIECES; ++i) {
            const int r = tid / S::P + i * (kCopyWarps * 32 / S::P);
            wrow[i] = w + row_at(r, a.ld_w);
            wto[i] = sw + (TRANS ? wc / 64 * (kCols * 128) : 0) + r * 128 + ((wc / 8 % 8) ^ (r & 7)) * 16;
        }
        constexpr int LAG = S::STAGES - 2;
        const int64_t wstep = TRANS ? static_cast<int64_t>(kCols) * a.ld_w : kCols;
        int left = a.k - first * kCols, stage = 0, lag_stage = 0, it = 0;
        uint32_t parity = 1;
        bool ok = true;
        // by TMA: x, W; a step's arrivals lag behind its copies where the warps make some
        const bool tma_x = WIDE && tile.row >= 0;
        const int lag = tma_x && WAL ? 0 : WIDE ? LAG : 0, tx = (tma_x ? S::X : 0) + (WAL ? S::W : 0);
        for (; it < steps; ++it, left -= kCols) {
            ok = wait(empty + 8 * stage, parity);
            if (!ok) break;
            if (threadIdx.x == 0) {
                const uint32_t bar = full + 8 * stage;
                const int k = (first + it) * kCols;
                ptx::mbar_arrive_expect_tx(bar, tx);
                if (tma_x) ptx::tma_load_2d(sx + stage * S::X, &map_x, bar, k, tile.row);
                if constexpr (WAL && TRANS) {
#pragma unroll
                    for (int i = 0; i < S::N / 64; ++i) ptx::tma_load_3d(sw + stage * S::W + i * (kCols * 128), &map_w, bar, i * 64, k, tile.adapter);
                } else if constexpr (WAL) {
                    ptx::tma_load_3d(sw + stage * S::W, &map_w, bar, k, 0, tile.adapter);
                }
            }
            __syncwarp();
            if constexpr (!WAL) {
#pragma unroll
                for (int i = 0; i < S::PIECES; ++i) {
                    const int r = tid / S::P + i * (kCopyWarps * 32 / S::P);
                    // of a row past the end: zeros along the long side, nothing past the rank
                    const int have = TRANS ? (r < left ? rank - wc : 0) : left - wc;
                    if (TRANS ? wc < rank : r < rank) copy8<false>(wto[i] + stage * S::W, have > 0 ? wrow[i] : a.w, have);
                    wrow[i] += wstep;
                }
            }
            if (!tma_x) {
                const uint32_t to = sx + stage * S::X + m0 * 128;
                const int n = left - piece * 8;
                if constexpr (WIDE) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (row[e] != nullptr) {
                            ptx::cp_async16(to + e * 512 + ((piece ^ (m0 + 4 * e)) & 7) * 16, n > 0 ? row[e] : a.x, max(0, min(16, 2 * n)));
                            row[e] += kCols;
                        }
                    }
                } else {
                    uint32_t v[8][4];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        v[e][0] = v[e][1] = v[e][2] = v[e][3] = 0u;
                        if (row[e] != nullptr) {
                            if (n > 0) load8(row[e], n, v[e]);
                            row[e] += kCols;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (row[e] != nullptr) ptx::st_shared_v4(to + e * 512 + ((piece ^ (m0 + 4 * e)) & 7) * 16, v[e][0], v[e][1], v[e][2], v[e][3]);
                }
            }
            ptx::cp_async_commit();
            if (it >= lag) {
                if (WIDE && !tma_x) ptx::cp_async_wait<LAG>();
                if (!(tma_x && WAL)) ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(full + 8 * lag_stage);
                lag_stage = lag_stage + 1 == S::STAGES ? 0 : lag_stage + 1;
            }
            if (++stage == S::STAGES) stage = 0, parity ^= 1;
        }
        ptx::cp_async_wait<0>();
        ptx::fence_proxy_async_smem();
        __syncwarp();
        for (int i = 0; i < min(it, lag) && ok; ++i) {
            if (lane == 0) ptx::mbar_arrive(full + 8 * lag_stage);
            lag_stage = lag_stage + 1 == S::STAGES ? 0 : lag_stage + 1;
        }
        // after a wait that ran out, the copies under way land before the CTA ends
        for (int i = max(0, it - S::STAGES); i < it && !ok && warp == 0; ++i)
            gemm_common::wait_phase(full + 8 * (i % S::STAGES), (i / S::STAGES) & 1, 2000000ull, abort_flag, a.err, 0u, false);
        ok = ok && wait(done, 0) && *abort_flag == 0u;
        if (ok) {
            ptx::tc_fence_after();
            const int m = warp * 32 + lane;
            float *out = a.out + (static_cast<int64_t>(blockIdx.y) * a.plan.tokens + tile.first + m) * RP;
            const uint32_t from = tmem + (static_cast<uint32_t>(warp * 32) << 16);
            const int sums = min(steps, S::SUMS);
#pragma unroll
            for (int c = 0; c < RP; c += 16) {
                uint32_t v[16];
                ptx::tmem_ld_32x32b_x16(from + c, v);
                ptx::tmem_wait_ld();
                float s[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) s[e] = __uint_as_float(v[e]);
                for (int i = 1; i < sums; ++i) {
                    ptx::tmem_ld_32x32b_x16(from + i * S::N + c, v);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) s[e] += __uint_as_float(v[e]);
                }
                if (m < tile.count) {
#pragma unroll
                    for (int e = 0; e < 16; e += 4) *reinterpret_cast<float4 *>(out + c + e) = make_float4(s[e], s[e + 1], s[e + 2], s[e + 3]);
                }
            }
        }
    } else {
        // sums FP32, operands BF16
        constexpr uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (TRANS ? 1u << 16 : 0u) | (static_cast<uint32_t>(S::N / 8) << 17) | (8u << 24);
        int stage = 0, sum = 0;
        uint32_t parity = 0;
        for (int it = 0; it < steps; ++it) {
            if (!wait(full + 8 * stage, parity)) break;
            ptx::tc_fence_after();
            if (lane == 0) {
                const uint64_t xd = gemm_common::desc_sw128(sx + stage * S::X);
                const uint64_t wd = TRANS ? desc_columns(sw + stage * S::W, kCols) : gemm_common::desc_sw128(sw + stage * S::W);
#pragma unroll
                for (int k = 0; k < kCols / 16; ++k)
                    ptx::tc_mma_bf16(tmem + sum * S::N, xd + 2 * k, wd + (TRANS ? k * (16 * 128 / 16) : 2 * k), idesc, it >= S::SUMS || k > 0);
                ptx::tc_commit(empty + 8 * stage);
            }
            __syncwarp();
            if (++stage == S::STAGES) stage = 0, parity ^= 1;
            if (++sum == S::SUMS) sum = 0;
        }
        if (lane == 0) ptx::tc_commit(done);
        __syncwarp();
        gemm_common::wait_phase(done, 0, kWaitNs, abort_flag, a.err, 0x20u + warp, false);
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == kCopyWarps) ptx::tmem_dealloc(tmem, S::TMEM);
}

template <int RP, bool TRANS, bool WIDE, bool WAL>
cudaError_t run(const ShrinkArgs &a, const CUtensorMap &map_x, const CUtensorMap &map_w, cudaStream_t stream) {
    using S = Shape<RP, TRANS>;
    static unsigned long long done;
    auto *kern = &k_lora_shrink<RP, TRANS, WIDE, WAL>;
    const cudaError_t e = with_smem(kern, S::SMEM, S::SMEM, done);
    if (e != cudaSuccess) return e;
    return launch_after(kern, dim3(a.plan.max_tiles(), most_splits(a.plan, a.k, RP)), kThreads, S::SMEM, stream, 1, a, map_x, map_w);
}
// W as [adapters][rows][long side], 64 values of the latter (or of a row of r) a piece.
bool weights_map(CUtensorMap *m, const ShrinkArgs &a, int rows, int cols, int box_rows) {
    const TensorMapEncodeFn enc = tensor_map_encoder();
    if (enc == nullptr) return false;
    const cuuint64_t ld = static_cast<cuuint64_t>(a.ld_w) * 2;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(a.plan.adapters)};
    // one adapter: any stride
    const cuuint64_t strides[2] = {ld, a.plan.adapters > 1 ? static_cast<cuuint64_t>(a.stride_w) * 2 : ld};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1}, es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(a.w), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
template <int RP, bool TRANS>
cudaError_t pick(const ShrinkArgs &a, cudaStream_t stream) {
    CUtensorMap map_x = {}, map_w = {};
    const bool wide = aligned_to(a.x, 16) && a.ld_x % 8 == 0 && rows_map(&map_x, a.x, a.plan.tokens, a.k, a.ld_x, kLoraTile);
    // a map's strides are not zero (one adapter for all)
    const bool wal = aligned_to(a.w, 16) && a.ld_w % 8 == 0 && a.stride_w % 8 == 0 && (a.plan.adapters == 1 || a.stride_w > 0) &&
                     weights_map(&map_w, a, TRANS ? a.k : a.lw.r, TRANS ? a.lw.r : a.k, TRANS ? kCols : RP);
    if (wide) return wal ? run<RP, TRANS, true, true>(a, map_x, map_w, stream) : run<RP, TRANS, true, false>(a, map_x, map_w, stream);
    return wal ? run<RP, TRANS, false, true>(a, map_x, map_w, stream) : run<RP, TRANS, false, false>(a, map_x, map_w, stream);
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

namespace {

// A tile's partial sums added up in place (in the first ones), 32 rows a CTA.
__global__ void __launch_bounds__(256) k_lora_sum(const SumArgs a, int rp) {
    ptx::grid_begin(static_cast<int64_t>(a.plan.tokens) * rp);
    const Tile tile = tile_at(a.plan, blockIdx.x);
    const int tiles = adapter_tiles(a.plan), splits = shrink_splits(a.plan, tiles, a.long_side, rp), quads = rp / 4;
    if (static_cast<int>(blockIdx.x) >= a.plan.words[0]) return;
    const int rank = tile.adapter < 0 ? 0 : rank_of(a.lw, tile.adapter);
    const int64_t next = static_cast<int64_t>(a.plan.tokens) * rp;
    for (int i = threadIdx.x; i < 32 * quads; i += 256) {
        const int m = blockIdx.y * 32 + i / quads, r = i % quads * 4;
        if (m >= tile.count) break;
        float *p = a.rows + (tile.first + m) * static_cast<int64_t>(rp) + r;
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (r < rank) {
#pragma unroll 8
            for (int s = 0; s < splits; ++s) {
                const uint4 q = ptx::ld_v4(p + s * next);
                v[0] += __uint_as_float(q.x), v[1] += __uint_as_float(q.y);
                v[2] += __uint_as_float(q.z), v[3] += __uint_as_float(q.w);
            }
            *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
        }
        if (a.v_out != nullptr) {
            float *to = a.v_out + row_at(a.plan.words[a.plan.order() + tile.first + m], a.ld_v) + r;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (r + e < a.lw.r) to[e] = r + e < rank ? v[e] : 0.0f;
        }
    }
}

}  // namespace

namespace {

// A warp 512 columns of a row at a time.
__global__ void __launch_bounds__(256) k_lora_pack(const PackArgs a) {
    const int side = blockIdx.y, cols = side ? a.cols[1] : a.cols[0];
    const uint16_t *from = side ? a.from[1] : a.from[0];
    uint16_t *to = side ? a.to[1] : a.to[0];
    const uint32_t ld = side ? a.ld[1] : a.ld[0], ld_to = static_cast<uint32_t>(ld_packed(cols));
    ptx::grid_begin(static_cast<int64_t>(a.plan.tokens) * cols);
    const int lane = threadIdx.x & 31, chunks = (cols + 511) / 512, rows = a.plan.words[a.plan.starts() + a.plan.adapters];
    const int64_t all = static_cast<int64_t>(rows) * chunks, step = static_cast<int64_t>(gridDim.x) * 8;
    for (int64_t i = blockIdx.x * 8 + threadIdx.x / 32; i < all; i += step) {
        const int row = static_cast<int>(i / chunks), c = static_cast<int>(i % chunks) * 512 + lane * 16;
        if (c >= cols) continue;
        uint32_t v[8];
        ragged::load16<false>(from + row_at(a.plan.words[a.plan.order() + row], ld) + c, cols - c, v);
        uint4 *p = reinterpret_cast<uint4 *>(to + row_at(row, ld_to) + c);
        p[0] = make_uint4(v[0], v[1], v[2], v[3]);
        p[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

}  // namespace

cudaError_t launch_pack(const PackArgs &a, int matrices, cudaStream_t stream) {
    const int64_t all = static_cast<int64_t>(a.plan.tokens) * ((std::max(a.cols[0], a.cols[1]) + 511) / 512);
    return launch_after(&k_lora_pack, dim3(static_cast<unsigned>(std::min<int64_t>((all + 7) / 8, 8 * kSms)), matrices), 256, 0, stream, 1, a);
}

cudaError_t launch_sum(const SumArgs &a, cudaStream_t stream) {
    return launch_after(&k_lora_sum, dim3(a.plan.max_tiles(), kLoraTile / 32), 256, 0, stream, 1, a, padded(a.lw.r));
}

}  // namespace lora
}  // namespace fp8hg
