// 4-bit quantizer kernels: BF16 -> E2M1 codes and block scales, the tensor
// scale, and back to values.  Their floor is HBM: 2 bytes read and about 0.53
// (MX) or 0.56 (NV) written per element and direction; beside it stand issue
// slots, 11 (NV along the rows) and 17 (NV both ways) instructions per element.
// At 8192 x 8960, in us and of the measured copy rate:
//   rows        MX 31 (88 %)   NV 32 (86 %)
//   both ways   MX 41 (82 %)   NV 48 (71 %)
//   columns     MX 31 (88 %)   NV 34 (81 %)
//   values      MX 31 (90 %)   NV 31 (91 %);   in FP32 92 (54 %)
//   tensor scale               24 to 25 (87 to 91 %), its second launch included
//
//  k_fp4_rows    along the rows: a thread takes 16 elements (an NV block, or
//                half an MX block, whose other half is in the next lane), so
//                nothing is exchanged but one shuffle for MX and the packing
//                of four scale bytes into a word.
//  k_fp4_tile    along the columns, or in both directions from one read: a
//                128 x 128 tile per CTA.
//  k_fp4_amax, k_fp4_tensor_scale   the tensor's scale.
//  k_fp4_dequant values from codes and scales.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fp4_math.cuh"
#include "lowbit.h"
#include "ragged.cuh"

namespace fp8hg {

namespace {

__device__ __forceinline__ uint32_t abs_max16(const uint32_t (&w)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_abs_bf16x2(m, w[i]);
    m = magnitudes(m);
    return max(m & 0xFFFFu, m >> 16);
}

// The low `n` bytes of eight code bytes to p (8-byte aligned).
__device__ __forceinline__ void store_codes(uint8_t *p, uint32_t lo, uint32_t hi, int n) {
    if (n >= 8) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(lo, hi);
    } else {
        const uint64_t v = (static_cast<uint64_t>(hi) << 32) | lo;
        for (int i = 0; i < n; ++i) p[i] = static_cast<uint8_t>(v >> (8 * i));
    }
}

// Four neighbouring blocks' scale bytes (one per LPB lanes) into one word, in
// the first of the 4 * LPB lanes.
template <int LPB>
__device__ __forceinline__ uint32_t gather_scales(uint32_t byte, int lane) {
    uint32_t v = byte << (8 * ((lane / LPB) & 3));
    v |= __shfl_xor_sync(0xFFFFFFFFu, v, LPB);
    v |= __shfl_xor_sync(0xFFFFFFFFu, v, 2 * LPB);
    return v;
}

// ------------------------------------------------------------- along the rows
// Block: `segs` segments of 16 elements (a multiple of 16) by some rows, a
// thread each; the segments cover k padded to 256, so that the padding's
// scale bytes are written too.
constexpr int kRowThreadsPerSm = 1280;   // 48 registers a thread

template <bool NV, bool WIDE>
__global__ void __launch_bounds__(256, kRowThreadsPerSm / 256)
    k_fp4_rows(const uint16_t *x, uint32_t rows, int cols, uint32_t ld_x,
               const float *ts, uint8_t *q, uint32_t ld_q,
               uint8_t *s, uint32_t tiles, int segs, int total_segs) {
    ptx::grid_begin(static_cast<int64_t>(rows) * cols);
    const int tid = threadIdx.x, lane = tid & 31;
    const int seg = blockIdx.x * segs + tid % segs;
    const int rpb = blockDim.x / segs;
    const float t = NV && ts ? ptx::ld_f32(ts) : 1.0f, rt = fp4_reciprocal<NV>(t);
    const int c0 = seg * 16;
    constexpr int LPB = NV ? 1 : 2;
    // The next row's load is in flight while a row is cast: a CTA per row
    // spent most of its time waiting for its one load (8192 x 3584, NV: 23.6 us).
    // Every lane of the warp stays in the loop for the shuffles.
    const uint32_t step = gridDim.y * rpb;
    const bool mine = tid / segs < rpb && seg < total_segs;
    uint32_t next[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    auto load = [&](uint32_t r) {
        if (mine && r < rows && c0 < cols) ragged::load16<WIDE>(x + row_at(r, ld_x) + c0, cols - c0, next);
    };
    load(blockIdx.y * rpb + tid / segs);
    for (uint32_t r0 = blockIdx.y * rpb; r0 < rows; r0 += step) {
        const uint32_t r = r0 + tid / segs;
        const bool in = mine && r < rows;
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = next[i];
        load(r + step);
        uint32_t m = abs_max16(w);
        if (!NV) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        const Fp4Scale<NV> sc(m, t, rt);
        const uint32_t word = gather_scales<LPB>(sc.byte, lane);
        if (!in) continue;
        if (c0 < cols) {
            const uint32_t lo = sc.cast8(w), hi = sc.cast8(w + 4);
            store_codes(q + row_at(r, ld_q) + c0 / 2, lo, hi, (cols - c0 + 1) / 2);
        }
        if (lane % (4 * LPB) == 0)
            *reinterpret_cast<uint32_t *>(s + fp4_scale_offset(r, seg / LPB, tiles)) = word;
    }
}

// ------------------------------------------- along the columns, or both ways
// A CTA takes a tile of 128 rows x 128 columns.  Each thread loads 16
// neighbouring elements of four rows, quantizes them along the row at once
// (ROWS) and leaves them in shared memory; then each thread takes two
// neighbouring columns over 32 rows (conflict-free 4-byte reads).  Codes of
// the columns go through shared memory so that a column's 64 bytes leave as
// whole sectors.  Scale tiles (128 rows x 4 blocks) are assembled in shared
// memory as well.  With 512 threads a tile, half as much for each, it takes 54 us
// instead of 48 (NV, 8192 x 8960).
constexpr int kTile = 128;

template <bool NV, bool WIDE, bool ROWS>
__global__ void __launch_bounds__(256)
    k_fp4_tile(const uint16_t *x, int rows, int cols, uint32_t ld_x,
               const float *ts, uint8_t *q, uint32_t ld_q,
               uint8_t *s, uint32_t tiles, uint8_t *qt, uint32_t ld_qt,
               uint8_t *st, uint32_t tiles_t) {
    ptx::grid_begin(static_cast<int64_t>(rows) * cols);
    constexpr int NT = NV ? 2 : 1;          // scale tiles of 4 blocks per 128 elements
    constexpr int LPB = NV ? 1 : 2;
    __shared__ __align__(16) uint8_t tile[kTile * 256];
    __shared__ __align__(16) uint8_t codes[kTile * 64];
    __shared__ __align__(16) uint8_t scales[2][NT * 512];
    const int tid = threadIdx.x, lane = tid & 31;
    const int r0 = blockIdx.y * kTile, k0 = blockIdx.x * kTile;
    const float t = NV && ts ? ptx::ld_f32(ts) : 1.0f, rt = fp4_reciprocal<NV>(t);
    {
        const int seg = tid & 7;
        const int c0 = k0 + seg * 16;
        uint32_t w[4][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + (tid >> 3) + i * 32;
#pragma unroll
            for (int j = 0; j < 8; ++j) w[i][j] = 0;
            if (r < rows && c0 < cols) ragged::load16<WIDE>(x + row_at(r, ld_x) + c0, cols - c0, w[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int rr = (tid >> 3) + i * 32;
            const int r = r0 + rr;
            // 16-byte pieces 2 seg and 2 seg + 1, swapped in the row's upper
            // half so that eight lanes' writes fall into different banks
            uint4 *row = reinterpret_cast<uint4 *>(tile + rr * 256);
            row[(2 * seg) ^ (seg >> 2)] = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
            row[(2 * seg + 1) ^ (seg >> 2)] = make_uint4(w[i][4], w[i][5], w[i][6], w[i][7]);
            if constexpr (ROWS) {
                uint32_t m = abs_max16(w[i]);
                if (!NV) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
                const Fp4Scale<NV> sc(m, t, rt);
                const uint32_t word = gather_scales<LPB>(sc.byte, lane);
                if (lane % (4 * LPB) == 0)
                    *reinterpret_cast<uint32_t *>(scales[0] + (seg / (4 * LPB)) * 512 +
                                                  (rr & 31) * 16 + (rr >> 5) * 4) = word;
                if (r < rows && c0 < cols) {
                    const uint32_t lo = sc.cast8(w[i]), hi = sc.cast8(w[i] + 4);
                    store_codes(q + row_at(r, ld_q) + c0 / 2, lo, hi, (cols - c0 + 1) / 2);
                }
            }
        }
    }
    __syncthreads();
    {
        // columns 2p, 2p + 1, rows 32 b .. 32 b + 31
        const int p = tid & 63, b = tid >> 6;
        const int piece = (p >> 2) ^ (p >> 5);   // the 16-byte piece, as swapped above
        const uint8_t *src = tile + b * 32 * 256 + piece * 16 + (p & 3) * 4;
        uint32_t v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = *reinterpret_cast<const uint32_t *>(src + i * 256);
        uint32_t m[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 32; ++i) m[i >> 4] = max_abs_bf16x2(m[i >> 4], v[i]);
        m[0] = magnitudes(m[0]), m[1] = magnitudes(m[1]);
        if (!NV) m[0] = m[1] = __vmaxu2(m[0], m[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t c[4];
            const int col = 2 * p + h;
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                const Fp4Scale<NV> sc(h ? m[part] >> 16 : m[part] & 0xFFFFu, t, rt);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint32_t *w = v + part * 16 + half * 8;
                    c[part * 2 + half] = h ? sc.template cast8_half<1>(w) : sc.template cast8_half<0>(w);
                }
                // block index along the rows within the tile
                if (NV || part == 0) {
                    const int j = NV ? 2 * b + part : b;
                    scales[1][(j >> 2) * 512 + (col & 31) * 16 + (col >> 5) * 4 + (j & 3)] =
                        static_cast<uint8_t>(sc.byte);
                }
            }
            *reinterpret_cast<uint4 *>(codes + col * 64 + ((b ^ (p & 3)) << 4)) =
                make_uint4(c[0], c[1], c[2], c[3]);
        }
    }
    __syncthreads();
    // columns' codes: four lanes write one column's 64 bytes
    {
        const int bytes = (rows + 1) / 2;   // of a whole column
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int idx = i * 256 + tid, col = idx >> 2, b = idx & 3;
            const int at = r0 / 2 + b * 16;
            if (k0 + col >= cols || at >= bytes) continue;
            const uint4 v = *reinterpret_cast<const uint4 *>(codes + col * 64 +
                                                             ((b ^ ((col >> 1) & 3)) << 4));
            uint8_t *d = qt + row_at(k0 + col, ld_qt) + at;
            if (at + 16 <= bytes) {
                *reinterpret_cast<uint4 *>(d) = v;
            } else {
                store_codes(d, v.x, v.y, bytes - at);
                if (bytes - at > 8) store_codes(d + 8, v.z, v.w, bytes - at - 8);
            }
        }
    }
    // scale tiles: 32 uint4 each; a tile of the padding along k has only zeros
    // (this kernel's tile then lies past the tensor) and is written too
    if (tid < 32 * NT) {
        if (ROWS && r0 < rows)
            reinterpret_cast<uint4 *>(s + (row_at(r0 >> 7, tiles) + (k0 >> 7) * NT) * 512)[tid] =
                reinterpret_cast<const uint4 *>(scales[0])[tid];
    } else if (tid >= 64 && tid < 64 + 32 * NT) {
        if (k0 < cols)
            reinterpret_cast<uint4 *>(st + (row_at(k0 >> 7, tiles_t) + (r0 >> 7) * NT) * 512)[tid - 64] =
                reinterpret_cast<const uint4 *>(scales[1])[tid - 64];
    }
}

// ------------------------------------------------------------- tensor scale
// Four CTAs an SM with two loads of 32 bytes in flight per thread: 8192 x 8960
// takes 24 to 25 us, with two CTAs and four loads 28.
constexpr int kAmaxBlocks = 1024;    // partial maxima at most
constexpr int kAmaxCtasPerSm = 4;

// Largest finite |x| pattern per CTA.
template <bool WIDE>
__global__ void __launch_bounds__(512, kAmaxCtasPerSm)
    k_fp4_amax(const uint16_t *x, int rows, int segs, int cols, uint32_t ld_x,
               uint32_t *part) {
    ptx::grid_begin(static_cast<int64_t>(rows) * cols);
    __shared__ uint32_t red[16];
    uint32_t m = 0;
    // segments of 16 elements, rows and segments walked together
    constexpr int U = 2;
    // a pattern plus 0x80 is negative as a signed half exactly if it is not finite
    const uint32_t step = gridDim.x * blockDim.x;
    uint32_t i = blockIdx.x * blockDim.x + threadIdx.x;
    uint32_t r = i / segs, c = i % segs;
    const uint32_t dr = step / segs, dc = step % segs;
    while (r < static_cast<uint32_t>(rows)) {
        uint32_t w[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[u][j] = 0u;
            if (r < static_cast<uint32_t>(rows))
                ragged::load16<WIDE>(x + row_at(r, ld_x) + c * 16, cols - static_cast<int>(c) * 16, w[u]);
            r += dr;
            c += dc;
            if (c >= static_cast<uint32_t>(segs)) c -= segs, ++r;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j) m = __vmaxs2(m, (w[u][j] & 0x7FFF7FFFu) + 0x00800080u);
    }
    m = __vmaxs2(m, 0x00800080u) - 0x00800080u;
    m = __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x < 32) {
        m = threadIdx.x < blockDim.x / 32 ? red[threadIdx.x] : 0u;
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if (threadIdx.x == 0) part[blockIdx.x] = m;
    }
}

__global__ void __launch_bounds__(32)
    k_fp4_tensor_scale(const uint32_t *part, int n, float *scale) {
    ptx::grid_begin(n);
    uint32_t m = 0;
#pragma unroll 8
    for (int i = threadIdx.x; i < n; i += 32) m = max(m, ptx::ld_u32(part + i));
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if (threadIdx.x == 0) {
        // 2688 = 1.3125 * 2^11, a mantissa field of 40: the power of two goes
        // up by one when the amax's mantissa is above that
        const int ef = static_cast<int>(m >> 7), mf = static_cast<int>(m & 0x7F);
        const int e = ef - 127 - 11 + (mf > 40 ? 1 : 0);
        *scale = m == 0 ? 1.0f : pow2f(max(e, -100));
    }
}

// ------------------------------------------------------------------- values
constexpr int kDequantThreadsPerSm = 1536;   // 40 registers a thread

template <bool NV, bool FP32, bool WIDE>
__global__ void __launch_bounds__(256, kDequantThreadsPerSm / 256)
    k_fp4_dequant(const uint8_t *q, const uint8_t *s,
                  const float *ts, uint32_t rows, int k, uint32_t ld, uint32_t tiles,
                  void *out, uint32_t ld_out, int segs) {
    ptx::grid_begin(static_cast<int64_t>(rows) * k);
    const float t = NV && ts ? ptx::ld_f32(ts) : 1.0f;
    const int g = blockIdx.x * blockDim.x + threadIdx.x;
    const int c0 = g * 16, left = k - c0;
    // the next row's codes and scale are in flight while a row is written
    uint2 next = make_uint2(0u, 0u);
    uint32_t next_scale = 0;
    auto load = [&](uint32_t r) {
        if (r >= rows || g >= segs) return;
        const uint8_t *src = q + row_at(r, ld) + c0 / 2;
        if (left >= 16) {
            next = ptx::ld_v2(src);
        } else {
            uint64_t v = 0;
            for (int i = 0; i < (left + 1) / 2; ++i) v |= static_cast<uint64_t>(ptx::ld_u8(src + i)) << (8 * i);
            next = make_uint2(static_cast<uint32_t>(v), static_cast<uint32_t>(v >> 32));
        }
        next_scale = ptx::ld_u8(s + fp4_scale_offset(r, NV ? g : g >> 1, tiles));
    };
    load(blockIdx.y);
    for (uint32_t r = blockIdx.y; r < rows; r += gridDim.y) {
        const uint32_t w[2] = {next.x, next.y}, byte = next_scale;
        load(r + gridDim.y);
        float v[16];
        if (g < segs) {
            const float sc = fp4_scale_value<NV>(byte);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float u[8];
                e2m1x8_values(w[h], u);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[8 * h + i] = u[i] * sc;
                    if (NV) v[8 * h + i] *= t;
                }
            }
        }
        if constexpr (FP32) {
            if (g >= segs) continue;
            float *d = static_cast<float *>(out) + row_at(r, ld_out) + c0;
            if (WIDE && left >= 16) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    reinterpret_cast<float4 *>(d)[i] =
                        make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (i < left) d[i] = v[i];
            }
        } else {
            uint32_t p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = g < segs ? ptx::cvt_bf16x2(v[2 * i], v[2 * i + 1]) : 0u;
            ragged::store16<WIDE>(static_cast<uint16_t *>(out) + row_at(r, ld_out) + c0, left, p);
        }
    }
}

template <bool NV>
cudaError_t quant_rows(const Fp4QuantArgs &a, cudaStream_t stream) {
    const int64_t total = (a.cols + 255LL) / 256 * 16;      // segments, k padded to 256
    const int64_t chunks = (total + 255) / 256;
    const int segs = static_cast<int>((total / 16 + chunks - 1) / chunks * 16);
    const int rpb = 256 / segs;
    const int threads = (segs * rpb + 31) / 32 * 32;
    const int64_t rblocks = (static_cast<int64_t>(a.rows) + rpb - 1) / rpb, cblocks = (total + segs - 1) / segs;
    // as many CTAs as fit at once
    const int64_t per_sm = kRowThreadsPerSm / threads, resident = std::max<int64_t>(1, sm_count() * per_sm / cblocks);
    const dim3 grid = chunks_first(std::min(rblocks, resident), cblocks);
    const int64_t tiles = fp4_scale_tiles(a.cols, a.kind);
    return launch_after(ragged::wide(a.x, a.ld_x) ? k_fp4_rows<NV, true> : k_fp4_rows<NV, false>, grid, threads, 0,
                        stream, 1, a.x, a.rows, a.cols, a.ld_x, a.ts, a.q, a.ld_q, a.s, tiles, segs, total);
}

template <bool NV, bool WIDE>
cudaError_t quant_tile(const Fp4QuantArgs &a, cudaStream_t stream) {
    // tiles cover both directions' padding to 256
    const dim3 grid(static_cast<unsigned>((a.cols + 255LL) / 256 * 2),
                    static_cast<unsigned>((a.rows + 255LL) / 256 * 2));
    const int64_t tiles = fp4_scale_tiles(a.cols, a.kind), tiles_t = fp4_scale_tiles(a.rows, a.kind);
    return launch_after(a.q ? k_fp4_tile<NV, WIDE, true> : k_fp4_tile<NV, WIDE, false>, grid, 256, 0, stream, 1, a.x,
                        a.rows, a.cols, a.ld_x, a.ts, a.q, a.ld_q, a.s, tiles, a.qt, a.ld_qt, a.st, tiles_t);
}

}  // namespace

size_t fp4_tensor_scale_ws_bytes() { return kAmaxBlocks * sizeof(uint32_t); }

cudaError_t launch_fp4_tensor_scale(const uint16_t *x, int rows, int cols, uint32_t ld_x,
                                    float *scale, void *ws, cudaStream_t stream) {
    const int segs = static_cast<int>((cols + 15LL) / 16);
    const int64_t n = static_cast<int64_t>(rows) * segs;
    const int64_t blocks = std::min({(n + 1023) / 1024, static_cast<int64_t>(kAmaxCtasPerSm) * sm_count(),
                                     static_cast<int64_t>(kAmaxBlocks)});
    uint32_t *part = static_cast<uint32_t *>(ws);
    if (n > 0) {
        const cudaError_t e = launch_after(ragged::wide(x, ld_x) ? k_fp4_amax<true> : k_fp4_amax<false>,
                                           static_cast<unsigned>(blocks), 512, 0, stream, 1, x, rows, segs, cols, ld_x,
                                           part);
        if (e != cudaSuccess) return e;
    }
    return launch_after(k_fp4_tensor_scale, 1, 32, 0, stream, 1, part, blocks, scale);
}

cudaError_t launch_fp4_quant(const Fp4QuantArgs &a, cudaStream_t stream) {
    const bool nv = a.kind == FP4_NV;
    if (!a.qt) return nv ? quant_rows<true>(a, stream) : quant_rows<false>(a, stream);
    if (ragged::wide(a.x, a.ld_x))
        return nv ? quant_tile<true, true>(a, stream) : quant_tile<false, true>(a, stream);
    return nv ? quant_tile<true, false>(a, stream) : quant_tile<false, false>(a, stream);
}

cudaError_t launch_fp4_dequant(const Fp4Operand &a, void *out, uint32_t ld_out, int fp32,
                               cudaStream_t stream) {
    const int64_t segs = (a.k + 15) / 16, tiles = fp4_scale_tiles(a.k, a.kind);
    // a row's segments in equal blocks of whole warps
    const int64_t chunks = (segs + 255) / 256;
    const int threads = static_cast<int>(((segs + chunks - 1) / chunks + 31) / 32 * 32);
    const int64_t cb = (segs + threads - 1) / threads;
    // as many CTAs as fit at once
    const int64_t per_sm = kDequantThreadsPerSm / threads, resident = std::max<int64_t>(1, sm_count() * per_sm / cb);
    const dim3 grid = chunks_first(std::min(a.rows, resident), cb);
    auto go = [&](auto kern) {
        return launch_after(kern, grid, threads, 0, stream, 1, a.codes, a.scale, a.ts, a.rows, a.k, a.ld, tiles, out,
                            ld_out, segs);
    };
    const bool nv = a.kind == FP4_NV;
    if (fp32) {
        if (reinterpret_cast<uintptr_t>(out) % 16 == 0 && ld_out % 4 == 0)
            return nv ? go(k_fp4_dequant<true, true, true>) : go(k_fp4_dequant<false, true, true>);
        return nv ? go(k_fp4_dequant<true, true, false>) : go(k_fp4_dequant<false, true, false>);
    }
    if (ragged::wide(out, ld_out))
        return nv ? go(k_fp4_dequant<true, false, true>) : go(k_fp4_dequant<false, false, true>);
    return nv ? go(k_fp4_dequant<true, false, false>) : go(k_fp4_dequant<false, false, false>);
}

}  // namespace fp8hg
