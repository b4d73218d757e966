// What the adapters' kernels share.
//
//   v[t] = x[t] A_g^T,  y[t] = base[t] + s_g v[t] B_g^T     (g: the token's adapter)
//   dv[t] = s_g dy[t] B_g,  dx[t] = base[t] + dv[t] A_g
//   dA_g = sum over its tokens of dv[t]^T x[t],  dB_g = s_g sum of dy[t]^T v[t]
//
//   shrink   rows of r from rows of n or k        (lora_shrink.cu)
//   expand   rows of n or k from rows of r        (lora_expand.cuh)
//   outer    sums over the tokens                 (lora_outer.cu)
//
// Tokens come in tiles of up to 128 of one adapter, gathered through the plan's
// order.  x, dy, A and B are BF16 and their products exact; sums are FP32.  The
// tensor core cuts its sums off instead of rounding them, which all lean the same
// way (measured, relative to the result, of random signs: 4.8e-7 after 32 sums of 16
// products, 7e-7 after 48, 1e-6 after 64, 2.5e-6 after 148; of one sign 9e-7 after 32,
// 1.2e-6 after 48): shrink deals its steps out to several sums, 48 of 16 each at most,
// outer takes its sums out after 32 and adds them up in registers, expand's are of
// r <= 128 products.  v and dv, FP32 sums, enter the next product as two BF16 parts (16
// bits of them, for results in BF16) or three (24 bits, for FP32).
//
// 2 r operations per value of x, dy or y and r small: HBM is the bound.  Shrink and
// outer feed tcgen05 by TMA where a tile's tokens are neighbours and by asynchronous
// copies where they are not; expand, whose result is what streams, keeps its small
// operand in registers and its products on mma.sync: a warp has 16 tokens and goes
// along their columns, so results leave the registers that base's values are added
// in (1024 multiply-adds a cycle and SM: 8192 x 18944, r 16, takes a tenth of the time
// that its bytes take).
#pragma once
#include <cstdint>

#include "adapt.h"
#include "gemm_common.cuh"
#include "norm.cuh"
#include "ptx.cuh"

namespace fp8hg {
namespace lora {

constexpr uint64_t kWaitNs = 2000000000ull;      // of a warp for another one of its CTA

// A tile of the plan.
struct Tile {
    int adapter, first, count, row;      // row: the first token's, if they are neighbours, or -1
};
__device__ __forceinline__ Tile tile_at(const LoraPlan &p, int i) {
    const int4 t = reinterpret_cast<const int4 *>(p.words + p.tiles())[i];
    return {t.x, t.y, t.z, t.w};
}
__device__ __forceinline__ int rank_of(const LoraWeights &w, int g) {
    return w.ranks == nullptr ? w.r : max(0, min(w.r, w.ranks[g]));
}

// Descriptor of an operand whose rows, not its K, lie next to one another: blocks of
// 64 rows (128 bytes, swizzled) by `ks` of K; a block's groups of eight K are 1024
// bytes apart, the blocks ks * 128.
__device__ __forceinline__ uint64_t desc_columns(uint32_t saddr, int ks) {
    const uint64_t d = gemm_common::desc_sw128(saddr) & ~(static_cast<uint64_t>(0x3FFF) << 16);
    return d | static_cast<uint64_t>(ks * 128 / 16) << 16;
}

// Eight values from p on, the first `left` of them (zeros behind), to 16 bytes
// of shared memory.  ALIGNED: p is a multiple of 16 bytes.
template <bool ALIGNED>
__device__ __forceinline__ void copy8(uint32_t dst, const uint16_t *p, int left) {
    const int n = max(0, min(8, left));
    if constexpr (ALIGNED) {
        ptx::cp_async16(dst, p, 2 * n);
    } else {
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) w[i >> 1] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
        ptx::st_shared_v4(dst, w[0], w[1], w[2], w[3]);
    }
}

// Eight values from p on, the first `left` > 0 of them (zeros behind): the aligned
// 16-byte pieces that hold them, moved into place.
__device__ __forceinline__ void load8(const uint16_t *p, int left, uint32_t (&w)[4]) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    const uint32_t s = static_cast<uint32_t>(at & 15), bytes = 2u * static_cast<uint32_t>(min(8, left));
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
    for (int i = 0; i < 4; ++i) w[i] = bytes >= 4u * i + 4u ? v[i] : bytes > 4u * i ? v[i] & 0xFFFFu : 0u;
}

// v as the sum of PARTS BF16 values: 16 bits of it with two, all 24 with three.
template <int PARTS>
__device__ __forceinline__ void split(float v, uint32_t (&h)[PARTS]) {
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
        h[i] = ptx::cvt_bf16x2(v, 0.0f) & 0xFFFFu;
        // an infinity or a NaN is in the first part alone
        v = (h[i] & 0x7F80u) == 0x7F80u ? 0.0f : v - __uint_as_float(h[i] << 16);
    }
}

__host__ __device__ constexpr int padded(int r) { return r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128; }
inline bool aligned_to(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Sixteen rows of 64 columns, a warp's part of a step: offset of 16-byte piece p of
// row r.  Copied a line (or two) of a row after the other, so that no sector is asked
// for twice; read back by the four lanes of a row, two rows at a time.
template <int PIECES>
__device__ __forceinline__ uint32_t slot(int r, int p) {
    return r * (PIECES * 16) + (p ^ (r & 7)) * 16;
}

// A thread's share of the copies of the other operand's tiles, ROWS x COLS values
// in rows of ROW bytes (and 32 more after every 16 rows if PAD): the same pieces of
// every tile, `step` elements on from one to the next.
template <int ROWS, int COLS, int ROW, bool PAD, bool ALIGNED>
struct TileCopy {
    static constexpr int P = COLS / 8, N = (ROWS * P + 255) / 256;
    const uint16_t *from[N];
    int rows, cols;          // of a whole tile that are there

    __device__ __forceinline__ TileCopy(const uint16_t *w, uint32_t ld, int rows_, int cols_) : rows(rows_), cols(cols_) {
#pragma unroll
        for (int i = 0; i < N; ++i) from[i] = w + row_at(row(i), ld) + col();
    }
    static __device__ __forceinline__ int row(int i) { return (threadIdx.x + 256 * i) / P; }
    static __device__ __forceinline__ int col() { return threadIdx.x % P * 8; }     // 256 is a multiple of P
    static __device__ __forceinline__ uint32_t at(int i) { return row(i) * ROW + (PAD ? row(i) / 16 * 32 : 0) + 2 * col(); }
    // rows_left, cols_left: of this tile
    __device__ __forceinline__ void copy(uint32_t to, const uint16_t *any, int rows_left, int cols_left, int64_t step) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (ROWS * P < 256 && row(i) >= ROWS) break;
            const bool in = row(i) < min(rows, rows_left);
            const int left = in ? min(cols, cols_left) - col() : 0;
            copy8<ALIGNED>(to + at(i), left > 0 ? from[i] : any, left);
            from[i] += step;
        }
    }
};

// The long side's splits of shrink: one round of CTAs over the plan's tiles, at least
// 128 columns each, and at most as many as keep the tensor core's sums short.  On the
// device from the plan, on the host an upper bound: as if no token were without an
// adapter, and the tiles full.
constexpr int kShrinkCols = 64;
constexpr int kMaxSplits = 16;
// Sums in tensor memory that steps take turns at, and the most steps at each: 48 sums
// of 16, each cut off, are off by some 7e-7 of the result (64: 1e-6; of one sign 1.2e-6).
__host__ __device__ constexpr int shrink_sums(int rp) { return rp <= 64 ? 8 : 4; }
constexpr int kSumSteps = 12;
__host__ __device__ inline int split_steps(int64_t steps, int ctas_a_tile, int rp) {
    int64_t n = ctas_a_tile < (steps + 1) / 2 ? ctas_a_tile : (steps + 1) / 2;
    n = n < 1 ? 1 : n > kMaxSplits ? kMaxSplits : n;
    const int64_t short_sums = (steps + shrink_sums(rp) * kSumSteps - 1) / (shrink_sums(rp) * kSumSteps);
    return static_cast<int>(n > short_sums ? n : short_sums);
}
__host__ __device__ inline int shrink_splits(const LoraPlan &p, int tiles, int k, int rp) {
    const int64_t steps = (static_cast<int64_t>(k) + kShrinkCols - 1) / kShrinkCols;
    const int full = (p.tokens + kLoraTile - 1) / kLoraTile;
    const int64_t n = split_steps(steps, kSms / (tiles > full ? tiles : full), rp), per = (steps + n - 1) / n;
    return static_cast<int>((steps + per - 1) / per);
}
inline int most_splits(const LoraPlan &p, int k, int rp) {
    return split_steps((static_cast<int64_t>(k) + kShrinkCols - 1) / kShrinkCols, kSms / ((p.tokens + kLoraTile - 1) / kLoraTile), rp);
}
__device__ __forceinline__ int adapter_tiles(const LoraPlan &p) { return p.words[p.tile_first() + p.adapters]; }

// A map of neighbouring rows, 64 BF16 values of each a piece, zeros past the last row
// and column; false if the driver does not take it.
inline bool rows_map(CUtensorMap *m, const uint16_t *p, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
    const TensorMapEncodeFn enc = tensor_map_encoder();
    if (enc == nullptr) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)}, strides[1] = {static_cast<cuuint64_t>(ld) * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)}, es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t *>(p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct ShrinkArgs {
    LoraPlan plan;
    const uint16_t *x;
    uint32_t ld_x;
    const uint16_t *w;               // [adapters][r][k], or trans: [adapters][k][r]
    int64_t stride_w;
    uint32_t ld_w;
    LoraWeights lw;                  // ranks
    int k;                           // the long side
    int packed;                      // x's rows are in the plan's order
    float *out;                      // [splits][tokens in the plan's order][padded(r)]
    unsigned int *err;               // the device's error word
};
cudaError_t launch_shrink(const ShrinkArgs &a, bool trans, cudaStream_t stream);

// Rows that TMA does not take (of a number of columns that is no multiple of 8) are
// copied once, in the plan's order, to rows of ld_packed values: read by three
// kernels, they would be put together from 16-byte pieces by every one of them
// (8192 x 8961 x 3583, r 16, backward: 857 us, with the copies 198).
__host__ __device__ constexpr int64_t ld_packed(int64_t cols) { return (cols + 63) / 64 * 64; }
inline size_t packed_bytes(int64_t tokens, int64_t cols) {
    return cols % 8 ? static_cast<size_t>(tokens) * ld_packed(cols) * sizeof(uint16_t) : 0;
}
struct PackArgs {
    LoraPlan plan;
    const uint16_t *from[2];
    uint32_t ld[2];
    int cols[2];
    uint16_t *to[2];
};
cudaError_t launch_pack(const PackArgs &a, int matrices, cudaStream_t stream);

struct SumArgs {
    LoraPlan plan;
    LoraWeights lw;                  // ranks, r
    float *rows;                     // [splits][tokens in the plan's order][padded(r)]
    int long_side;
    float *v_out;                    // the sums by token, for the backward pass, or null
    uint32_t ld_v;
};
cudaError_t launch_sum(const SumArgs &a, cudaStream_t stream);

struct ExpandArgs {
    LoraPlan plan;
    const float *rows;               // [splits][tokens in the plan's order][padded(r)]
    int long_side;                   // that they were summed over, 0: one split
    const uint16_t *w;               // [adapters][n][r], or trans: [adapters][r][n]
    int64_t stride_w;
    uint32_t ld_w;
    LoraWeights lw;                  // ranks, scale
    int n;                           // columns
    const void *base;
    void *y;
    uint32_t ld_base, ld_y;
    float *v_out;                    // the rows of r for the backward pass, or null
    uint32_t ld_v;
};
cudaError_t launch_expand(const ExpandArgs &a, bool f32, cudaStream_t stream);
cudaError_t launch_expand_t(const ExpandArgs &a, bool f32, cudaStream_t stream);     // trans

// Both products of at most so many tokens in one kernel.
constexpr int kFewTokens = 64;
struct FewArgs {
    LoraPlan plan;
    LoraWeights lw;
    const uint16_t *x;
    uint32_t ld_x;
    const void *base;
    void *y;
    uint32_t ld_base, ld_y;
    float *v_out;                    // x A^T for the backward pass, or null
    uint32_t ld_v;
};
bool few(const FewArgs &a, bool f32);      // sizes and alignments that it takes
cudaError_t launch_few(const FewArgs &a, bool f32, cudaStream_t stream);

// One of the two sums over the tokens.
struct OuterSide {
    const uint16_t *d;               // [tokens][n]
    uint32_t ld;
    int n, blocks;                   // columns, and blocks of them
    int packed;                      // d's rows are in the plan's order
    const uint16_t *vt;              // by 64 tokens: [parts][padded(r)][64], swizzled
    void *out;                       // [adapters] of n x r: strides
    int64_t stride_n, stride_r, stride_g;
    float *ws;                       // [2 chunks][n][padded(r)]
};
struct OuterArgs {
    LoraPlan plan;
    LoraWeights lw;
    OuterSide side[2];
    int chunks;                      // of the tiles
    int f32;
    unsigned int *err;               // the device's error word
    // tiles of a chunk
    __device__ __forceinline__ int tiles(int all) const { return max(1, (all + chunks - 1) / chunks); }
};
size_t outer_vt_bytes(const LoraPlan &p, int r);
int outer_chunks(const LoraPlan &p, int n, int k, int r);
struct PrepArgs {
    LoraPlan plan;
    LoraWeights lw;
    const float *v;                  // [tokens][ld_v], or null
    uint32_t ld_v;
    const float *dv;                 // [splits][tokens in the plan's order][padded(r)], or null
    int long_side;                   // that they were summed over
    float *sum;                      // dv's sum, or null
    uint16_t *vt[2];                 // of v and of dv
    int parts;
};
cudaError_t launch_prep(const PrepArgs &a, cudaStream_t stream);
cudaError_t launch_outer(OuterArgs &a, cudaStream_t stream);

}  // namespace lora
}  // namespace fp8hg
