// Adapters: sums over the tokens, out_g[n][r] = sum over g's tokens of d[t][n]
// v[t][r], for dB (d = dy) and dA (d = x, v = dv) in one launch.
//
// The rows of r come first, in a kernel of their own: partial sums added, scaled,
// taken apart into BF16 parts and transposed, a step's tokens next to one another
// as the tensor core takes them.  Then 128 columns of d are the rows of a
// tcgen05.mma, the parts of the rows of r its columns, 64 tokens a step its K: d is
// read once, in rows as they lie (its tile is an operand whose rows, not its K, are
// contiguous), and every part has sums of its own.  A CTA takes 256 (or 128)
// columns and a chunk of the tiles; an adapter whose tokens are in several chunks
// leaves partial sums there, which one more kernel adds in a fixed order.
//
// 8192 tokens, 8960 + 1536 columns, r 64 in three parts: 39 us for 172 MB, 65 % of the
// copy rate (rows copied by the warps: 58; mma.sync: 145): 41 blocks of columns by 3
// chunks keep 123 of the 152 SMs busy.  Rows of r 7, joining 8.  13 warps leave 128
// registers a thread: with r 64 and 128 the sums' warps spill 210 to 300 bytes.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "lora.cuh"

namespace fp8hg {
namespace lora {

namespace {

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
    const int splits = side == 0 ? 0 : shrink_splits(a.plan, tiles, a.long_side, RP);
    constexpr int H = kLoraTile * 4 / 256;
    const int c = tid % 4 * 4, r = r0 + c;
    float v[H][4];
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[h][e] = 0.0f;
    auto token = [&](int h) { return (h * 256 + tid) / 4; };
    if (side == 0) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
            if (token(h) >= tile.count) continue;
            const float *p = a.v + row_at(a.plan.words[a.plan.order() + tile.first + token(h)], a.ld_v) + r;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (r + e < rank) v[h][e] = p[e];
        }
    } else {
        const float *p = a.dv + tile.first * static_cast<int64_t>(RP) + r;
        const int64_t step = static_cast<int64_t>(a.plan.tokens) * RP;
#pragma unroll 8
        for (int s = 0; s < splits; ++s) {
#pragma unroll
            for (int h = 0; h < H; ++h) {
                if (token(h) >= tile.count) continue;
                const uint4 q = ptx::ld_v4(p + s * step + token(h) * RP);
                v[h][0] += __uint_as_float(q.x), v[h][1] += __uint_as_float(q.y);
                v[h][2] += __uint_as_float(q.z), v[h][3] += __uint_as_float(q.w);
            }
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (r + e >= rank) v[h][e] = 0.0f;
            if (a.sum != nullptr && token(h) < tile.count)
                *reinterpret_cast<float4 *>(a.sum + (tile.first + token(h)) * static_cast<int64_t>(RP) + r) =
                    make_float4(v[h][0], v[h][1], v[h][2], v[h][3]);
        }
    }
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) rows[c + e][token(h)] = v[h][e] * scale;
    __syncthreads();
    // eight tokens of a row of r a thread
    const int row = tid / (kLoraTile / 8), m = tid % (kLoraTile / 8) * 8;
    uint32_t w[PARTS][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint32_t lo[PARTS], hi[PARTS];
        split<PARTS>(rows[row][m + 2 * e], lo);
        split<PARTS>(rows[row][m + 2 * e + 1], hi);
#pragma unroll
        for (int p = 0; p < PARTS; ++p) w[p][e] = lo[p] | hi[p] << 16;
    }
    // as it will stand in shared memory: 64 tokens, a row of 128 bytes for each part and
    // row of r, its 16-byte pieces exchanged as the tensor core's swizzle has it
    uint8_t *to = reinterpret_cast<uint8_t *>(a.vt[side]) + (2 * static_cast<int64_t>(blockIdx.x) + m / 64) * (PARTS * RP * 128) +
                  (r0 + row) * 128 + ((m % 64 / 8) ^ (row & 7)) * 16;
#pragma unroll
    for (int p = 0; p < PARTS; ++p) *reinterpret_cast<uint4 *>(to + p * RP * 128) = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
}

// -------------------------------------------------------------------- outer
constexpr int kStep = 64;            // tokens
constexpr int kCopyWarps = 4, kSumWarps = 8;
constexpr int kThreads = (kCopyWarps + kSumWarps + 1) * 32;
// Steps whose products stay in tensor memory before they are added up in FP32: 32
// sums of 16, each cut off, are off by some 5e-7 of the result, of one sign 9e-7.
constexpr int kSteps = 8;

template <int RP, int PARTS>
struct Shape {
    static constexpr int BLOCKS = RP <= 64 ? 2 : 1;      // of 128 columns
    static constexpr int COLS = 128 * BLOCKS;            // of a CTA
    static constexpr int N = PARTS * RP;                 // of a block in tensor memory
    static constexpr int MMAS = N > 256 ? 2 : 1;
    static constexpr int A = kStep * COLS * 2, B = N * 128;
    static constexpr int STAGES = 224 * 1024 / (A + B) < 5 ? 224 * 1024 / (A + B) : 5;
    static constexpr int BARS = 8 * (2 * STAGES + 3);
    static constexpr int SMEM = 1024 + STAGES * (A + B) + BARS + 16;
    static constexpr int TMEM = BLOCKS * N <= 64 ? 64 : BLOCKS * N <= 128 ? 128 : BLOCKS * N <= 256 ? 256 : 512;
    static constexpr int SUMS = BLOCKS == 2 ? RP : RP / 2;   // rows of r of a thread
};

// Warps: four copy (a token's columns at a time; the first one the rows of r as well),
// eight add up, one issues the products.
// WIDE: rows that TMA takes (16-byte multiples); a step of 64 neighbours is copied by it.
template <int RP, int PARTS, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1)
    k_lora_outer(const OuterArgs a, const __grid_constant__ CUtensorMap map0, const __grid_constant__ CUtensorMap map1) {
    using S = Shape<RP, PARTS>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    ptx::grid_begin(static_cast<int64_t>(a.plan.tokens) * (static_cast<int64_t>(a.side[0].n) + a.side[1].n));
    const bool second = static_cast<int>(blockIdx.x) >= a.side[0].blocks;
    const OuterSide &o = a.side[second];
    const int n0 = (blockIdx.x - (second ? a.side[0].blocks : 0)) * S::COLS;
    const int *tile_first = a.plan.words + a.plan.tile_first(), *order = a.plan.words + a.plan.order();
    const int all = adapter_tiles(a.plan), per = a.tiles(all);
    const int t0 = blockIdx.y * per, t1 = min(all, t0 + per);
    if (t0 >= t1) return;

    const uint32_t raw = ptx::smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    const uint32_t sa = base, sb = base + S::STAGES * S::A, bars = sb + S::STAGES * S::B;
    const uint32_t full = bars, empty = full + 8 * S::STAGES, sum_full = empty + 8 * S::STAGES, sum_empty = sum_full + 8, drain = sum_empty + 8;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem_raw + (bars + S::BARS - raw));
    volatile uint32_t *abort_flag = tmem_slot + 1;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::STAGES; ++i) {
            ptx::mbar_init(full + 8 * i, kCopyWarps + 1);
            ptx::mbar_init(empty + 8 * i, 1);
        }
        ptx::mbar_init(sum_full, 1);
        ptx::mbar_init(sum_empty, kSumWarps);
        ptx::mbar_init(drain, 1);
        *abort_flag = 0u;
        ptx::fence_mbar_init();
    }
    if (warp == kCopyWarps + kSumWarps) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), S::TMEM);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xFFFFFFFFu, gemm_common::wait_phase(bar, parity, kWaitNs, abort_flag, a.err, 0x40u + warp));
    };

    if (warp < kCopyWarps) {
        // a token's row: 16 bytes a lane, one row (two with one block) at a time
        constexpr int ROWS = 2 / S::BLOCKS, EACH = kStep / kCopyWarps / ROWS;
        const int piece = lane % (32 / ROWS), sub = lane / (32 / ROWS), left = o.n - n0 - piece * 8;
        const int bytes = max(0, min(16, 2 * left));
        const uint32_t to0 = sa + piece / 8 * (kStep * 128);
        // this step's tokens, a lane each; the next step's are asked for meanwhile
        auto look_up = [&](const Tile &tile, int h) {
            const int m = h * kStep + warp * (kStep / kCopyWarps) + lane;
            return lane < kStep / kCopyWarps && m < tile.count ? (o.packed ? tile.first + m : order[tile.first + m]) : -1;
        };
        Tile tile = tile_at(a.plan, t0), next = tile_at(a.plan, min(t0 + 1, t1 - 1));
        int token = look_up(tile, 0), stage = 0, lag_stage = 0, it = 0, h = 0;
        uint32_t parity = 1;
        bool ok = true;
        constexpr int LAG = WIDE ? S::STAGES - 2 : 0;
        for (int t = t0; t < t1 && ok; ++it) {
            const int now = token, t_now = t, h_now = h;
            const int near = o.packed ? tile.first : tile.row;
            const int together = WIDE && near >= 0 && h * kStep + kStep <= tile.count ? near + h * kStep : -1;
            h += 1;
            if (h * kStep >= tile.count) {
                h = 0;
                ++t;
                tile = next;
                next = tile_at(a.plan, min(t + 1, t1 - 1));
            }
            token = look_up(tile, h);
            ok = wait(empty + 8 * stage, parity);
            if (!ok) break;
            if (warp == 0 && lane == 0) {
                ptx::mbar_arrive_expect_tx(full + 8 * stage, S::B + (together >= 0 ? S::A : 0));
                for (int i = 0; i < S::COLS / 64 && together >= 0; ++i)
                    ptx::tma_load_2d(sa + stage * S::A + i * (kStep * 128), second ? &map1 : &map0, full + 8 * stage, n0 + i * 64, together);
                ptx::bulk_load(sb + stage * S::B, reinterpret_cast<const uint8_t *>(o.vt) + (2 * static_cast<int64_t>(t_now) + h_now) * S::B, S::B,
                               full + 8 * stage);
            }
            const uint32_t to = to0 + stage * S::A;
            __syncwarp();
            if (together >= 0) {
            } else if constexpr (WIDE) {
#pragma unroll
                for (int e = 0; e < EACH; ++e) {
                    const int i = e * ROWS + sub, m = warp * (kStep / kCopyWarps) + i, tok = __shfl_sync(0xFFFFFFFFu, now, i);
                    const bool in = tok >= 0 && bytes > 0;
                    ptx::cp_async16(to + m * 128 + ((piece ^ m) & 7) * 16, in ? o.d + row_at(tok, o.ld) + n0 + piece * 8 : o.d, in ? bytes : 0);
                }
            } else {
                // eight rows' loads in flight
#pragma unroll
                for (int e0 = 0; e0 < EACH; e0 += 8) {
                    uint32_t w[8][4];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int tok = __shfl_sync(0xFFFFFFFFu, now, (e0 + e) * ROWS + sub);
                        w[e][0] = w[e][1] = w[e][2] = w[e][3] = 0u;
                        if (tok >= 0 && left > 0) load8(o.d + row_at(tok, o.ld) + n0 + piece * 8, left, w[e]);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int m = warp * (kStep / kCopyWarps) + (e0 + e) * ROWS + sub;
                        ptx::st_shared_v4(to + m * 128 + ((piece ^ m) & 7) * 16, w[e][0], w[e][1], w[e][2], w[e][3]);
                    }
                }
            }
            ptx::cp_async_commit();
            if (it >= LAG) {
                ptx::cp_async_wait<LAG>();
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(full + 8 * lag_stage);
                lag_stage = lag_stage + 1 == S::STAGES ? 0 : lag_stage + 1;
            }
            if (++stage == S::STAGES) stage = 0, parity ^= 1;
        }
        ptx::cp_async_wait<0>();
        ptx::fence_proxy_async_smem();
        __syncwarp();
        for (int i = 0; i < min(it, LAG) && ok; ++i) {
            if (lane == 0) ptx::mbar_arrive(full + 8 * lag_stage);
            lag_stage = lag_stage + 1 == S::STAGES ? 0 : lag_stage + 1;
        }
        // the last copies of the rows of r land before the CTA ends
        if (warp == 0) {
            for (int i = max(0, it - S::STAGES); i < it; ++i)
                gemm_common::wait_phase(full + 8 * (i % S::STAGES), (i / S::STAGES) & 1, ok ? kWaitNs : 2000000ull, abort_flag, a.err, 0x40u, false);
        }
    } else if (warp < kCopyWarps + kSumWarps) {
        const int q = warp & 3, half = (warp - kCopyWarps) >> 2;
        const int c = n0 + (S::BLOCKS == 2 ? half * 128 : 0) + q * 32 + lane, r0 = S::BLOCKS == 2 ? 0 : half * S::SUMS;
        const uint32_t from = tmem + (static_cast<uint32_t>(q * 32) << 16) + (S::BLOCKS == 2 ? half * S::N : r0);
        float sum[S::SUMS];
#pragma unroll
        for (int i = 0; i < S::SUMS; ++i) sum[i] = 0.0f;
        uint32_t parity = 0;
        bool ok = true;
        int steps = 0;
        for (int t = t0; t < t1 && ok; ++t) {
            const Tile tile = tile_at(a.plan, t);
            const int begin = tile_first[tile.adapter], end = tile_first[tile.adapter + 1];
            steps += (tile.count + kStep - 1) / kStep;
            const bool last = t + 1 == t1 || t + 1 == end;
            if (!last && steps + 2 <= kSteps) continue;
            steps = 0;
            ok = wait(sum_full, parity);
            if (!ok) break;
            parity ^= 1;
            ptx::tc_fence_after();
#pragma unroll
            for (int p = 0; p < PARTS; ++p)
#pragma unroll
                for (int i = 0; i < S::SUMS; i += 16) {
                    uint32_t v[16];
                    ptx::tmem_ld_32x32b_x16(from + p * RP + i, v);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) sum[i + e] += __uint_as_float(v[e]);
                }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(sum_empty);
            if (!last) continue;
            // the adapter's last tile, here or at all
            if (c < o.n) {
                if (begin >= t0 && end <= t1) {
                    const int64_t to = tile.adapter * o.stride_g + c * o.stride_n + r0 * o.stride_r;
                    // past the rank zeros, not products of zeros with what d holds
                    const int have = min(S::SUMS, a.lw.r - r0), used = rank_of(a.lw, tile.adapter) - r0;
                    if (a.f32) {
                        float *p = static_cast<float *>(o.out) + to;
                        for (int i = max(0, used); i < have; ++i) p[i * o.stride_r] = 0.0f;
#pragma unroll
                        for (int i = 0; i < S::SUMS; ++i, p += o.stride_r)
                            if (i < used) *p = sum[i];
                    } else {
                        uint16_t *p = static_cast<uint16_t *>(o.out) + to;
                        for (int i = max(0, used); i < have; ++i) p[i * o.stride_r] = 0;
#pragma unroll
                        for (int i = 0; i < S::SUMS; ++i, p += o.stride_r)
                            if (i < used) *p = static_cast<uint16_t>(ptx::cvt_bf16x2(sum[i], 0.0f));
                    }
                } else {
                    float *part = o.ws + ((2 * static_cast<int64_t>(blockIdx.y) + (begin < t0 ? 0 : 1)) * o.n + c) * RP + r0;
#pragma unroll
                    for (int i = 0; i < S::SUMS; i += 4)
                        *reinterpret_cast<float4 *>(part + i) = make_float4(sum[i], sum[i + 1], sum[i + 2], sum[i + 3]);
                }
            }
#pragma unroll
            for (int i = 0; i < S::SUMS; ++i) sum[i] = 0.0f;
        }
    } else if (warp == kCopyWarps + kSumWarps) {
        // sums FP32, operands BF16, d with its columns (not its tokens) next to one another
        constexpr uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (static_cast<uint32_t>(S::N / S::MMAS / 8) << 17) | (8u << 24);
        int stage = 0, steps = 0, sets = 0;
        uint32_t parity = 0;
        bool ok = true;
        for (int t = t0; t < t1 && ok; ++t) {
            const Tile tile = tile_at(a.plan, t);
            const int end = tile_first[tile.adapter + 1], mine = (tile.count + kStep - 1) / kStep;
            for (int h = 0; h < mine; ++h, ++steps) {
                if (steps == 0) {
                    ok = wait(sum_empty, (sets & 1) ^ 1);
                    if (!ok) break;
                    ptx::tc_fence_after();
                }
                ok = wait(full + 8 * stage, parity);
                if (!ok) break;
                ptx::tc_fence_after();
                if (lane == 0) {
                    const uint64_t ad = desc_columns(sa + stage * S::A, kStep), bd = gemm_common::desc_sw128(sb + stage * S::B);
#pragma unroll
                    for (int k = 0; k < kStep / 16; ++k)
#pragma unroll
                        for (int b = 0; b < S::BLOCKS; ++b)
#pragma unroll
                            for (int i = 0; i < S::MMAS; ++i)
                                ptx::tc_mma_bf16(tmem + b * S::N + i * (S::N / S::MMAS), ad + b * (2 * kStep * 128 / 16) + k * (16 * 128 / 16),
                                                 bd + i * (S::N / S::MMAS * 128 / 16) + k * 2, idesc, steps > 0 || k > 0);
                    ptx::tc_commit(empty + 8 * stage);
                }
                __syncwarp();
                if (++stage == S::STAGES) stage = 0, parity ^= 1;
            }
            if (ok && (t + 1 == t1 || t + 1 == end || steps + 2 > kSteps)) {
                if (lane == 0) ptx::tc_commit(sum_full);
                __syncwarp();
                steps = 0;
                ++sets;
            }
        }
        if (lane == 0) ptx::tc_commit(drain);
        __syncwarp();
        gemm_common::wait_phase(drain, 0, kWaitNs, abort_flag, a.err, 0x40u + warp, false);
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == kCopyWarps + kSumWarps) ptx::tmem_dealloc(tmem, S::TMEM);
}

// The adapters of several chunks, and zeros for those without a token: 32 by 32
// values a CTA, through shared memory where the result's rows run the other way.
__global__ void __launch_bounds__(256) k_lora_join(const OuterArgs a, int rp) {
    __shared__ float tile[32][33];
    ptx::grid_wait();
    const int parts = (a.lw.r + 31) / 32, r0 = blockIdx.z % parts * 32;
    const OuterSide &o = a.side[blockIdx.z / parts];
    if (o.out == nullptr) return;
    const int *tile_first = a.plan.words + a.plan.tile_first();
    const int per = a.tiles(adapter_tiles(a.plan));
    const int tx = threadIdx.x & 31, ty = threadIdx.x / 32;
    const bool along_n = o.stride_n == 1;
    for (int g = blockIdx.y; g < a.plan.adapters; g += gridDim.y) {
        const int begin = tile_first[g], end = tile_first[g + 1];
        const int c0 = begin / per, c1 = begin < end ? (end - 1) / per : c0;
        if (begin < end && c0 == c1) continue;
        const int rank = rank_of(a.lw, g);
        for (int64_t b = static_cast<int64_t>(blockIdx.x) * 32; b < o.n; b += static_cast<int64_t>(gridDim.x) * 32) {
            float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (begin < end && r0 + tx < rank) {      // zeros past the rank
                const int64_t slot = static_cast<int64_t>(o.n) * rp;
                const float *p = o.ws + (2 * static_cast<int64_t>(c0) + 1) * slot + (b + ty) * rp + r0 + tx;
                // the first chunk's, then one of each chunk after it
#pragma unroll 4
                for (int c = c0; c <= c1; ++c, p += c == c0 + 1 ? slot : 2 * slot) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (b + ty + 8 * i < o.n) s[i] += ptx::ld_f32(p + static_cast<int64_t>(8 * i) * rp);
                }
            }
            if (along_n) {
                __syncthreads();
#pragma unroll
                for (int i = 0; i < 4; ++i) tile[ty + 8 * i][tx] = s[i];
                __syncthreads();
#pragma unroll
                for (int i = 0; i < 4; ++i) s[i] = tile[tx][ty + 8 * i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t n = b + (along_n ? tx : ty + 8 * i);
                const int r = r0 + (along_n ? ty + 8 * i : tx);
                if (n < o.n && r < a.lw.r) {
                    const int64_t at = g * o.stride_g + n * o.stride_n + r * o.stride_r;
                    if (a.f32) static_cast<float *>(o.out)[at] = s[i];
                    else static_cast<uint16_t *>(o.out)[at] = static_cast<uint16_t>(ptx::cvt_bf16x2(s[i], 0.0f));
                }
            }
        }
    }
}

int cols(int rp) { return rp <= 64 ? Shape<64, 2>::COLS : Shape<128, 2>::COLS; }
int blocks_of(int n, int rp) { return (n + cols(rp) - 1) / cols(rp); }

template <int RP, int PARTS, bool WIDE>
cudaError_t run(const OuterArgs &a, const CUtensorMap (&map)[2], cudaStream_t stream) {
    static unsigned long long done;
    using S = Shape<RP, PARTS>;
    auto *kern = &k_lora_outer<RP, PARTS, WIDE>;
    const cudaError_t e = with_smem(kern, S::SMEM, S::SMEM, done);
    if (e != cudaSuccess) return e;
    return launch_after(kern, dim3(a.side[0].blocks + a.side[1].blocks, a.chunks), kThreads, S::SMEM, stream, 1, a, map[0], map[1]);
}
template <int RP>
cudaError_t pick(const OuterArgs &a, bool wide, const CUtensorMap (&map)[2], cudaStream_t stream) {
    if (a.f32) return wide ? run<RP, 3, true>(a, map, stream) : run<RP, 3, false>(a, map, stream);
    return wide ? run<RP, 2, true>(a, map, stream) : run<RP, 2, false>(a, map, stream);
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
    CUtensorMap map[2] = {};
    for (int i = 0; i < 2; ++i) {
        OuterSide &o = a.side[i];
        o.blocks = o.out != nullptr ? blocks_of(o.n, rp) : 0;
        if (o.out == nullptr) continue;
        wide = wide && aligned_to(o.d, 16) && o.ld % 8 == 0 && rows_map(&map[i], o.d, a.plan.tokens, o.n, o.ld, kStep);
        most = std::max<int64_t>(most, o.n);
    }
    const cudaError_t e = rp == 16   ? pick<16>(a, wide, map, stream)
                          : rp == 32 ? pick<32>(a, wide, map, stream)
                          : rp == 64 ? pick<64>(a, wide, map, stream)
                                     : pick<128>(a, wide, map, stream);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>((most + 31) / 32, 1024)), std::min(a.plan.adapters, 64), 2 * ((a.lw.r + 31) / 32));
    return launch_after(&k_lora_join, grid, 256, 0, stream, 1, a, rp);
}

}  // namespace lora
}  // namespace fp8hg
