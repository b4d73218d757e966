// Layer norm, forward.
//
//   mean = sum(x) / n,  var = sum((x - mean)^2) / n,  rstd = 1 / sqrt(var + eps)
//   y = (x - mean) rstd w + b
//
// in FP32 between the loads and the stores.  The variance is summed from the
// differences in registers, not from squares, so a row far from zero loses
// nothing.  y goes out in BF16 or FP32, and as the FP8 operand of the next
// product: quantized from FP32, one UE8M0 scale per row or per 128 columns.
//
// Bound by HBM: a row stays in registers between its load and its stores.  A
// thread takes 16 neighbouring columns, a row as many threads as that needs, in
// whole warps; CTAs step through the rows with the next row's loads in flight
// and the parameters in shared memory, where they cost no registers.  Rows of
// more than 8192 columns are read again for each sum (from the L2).
//
// 16384 x 3584, BF16 x: y in BF16 43 us (81 % of the copy rate), codes alone 49.5 (53 %;
// by groups of 128: 50), both 55; FP32 x and y, 8192 x 3584, 43 (81 %).  With codes
// neither the bytes (36 % of DRAM) nor the instructions (47 % of the SM's rate) bound
// it but the latency of three sums a row, with 14 warps an SM.  A warp for a whole row,
// without any barrier, takes 40, 49 and 55 (codes by groups of 128: 52).  The mean and the
// variance are plain divisions, by the lanes that add a row up: in every thread they
// take 2 us more of these 43 (a product with 1 / n and its correction, in every
// thread: 2 us as well).  Rows of more than 8192 columns: 4096 x 12288 164 us for 201 MB,
// the row read three times without copies ahead.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fp8_group.cuh"
#include "norm.cuh"

namespace fp8hg {

namespace {

using namespace norm;

__device__ __forceinline__ uint32_t emit_fp8(int fmt, const F2 (&v)[8], float amax, uint8_t *q, int left) {
    uint32_t c[4], byte;
    if (fmt == FMT_E4M3) {
        const GroupF32<FMT_E4M3> gs(amax);
        byte = gs.byte;
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = gs.cast4(v[2 * i], v[2 * i + 1]);
    } else {
        const GroupF32<FMT_E5M2> gs(amax);
        byte = gs.byte;
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = gs.cast4(v[2 * i], v[2 * i + 1]);
    }
    if (left > 0) store_bytes16(q, c, left);
    return byte;
}

enum { Q_NONE = 0, Q_ROW = 1, Q_GROUP = 2 };

__device__ __forceinline__ float max_of(const F2 (&y)[8]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_abs(m, y[i]);
    return m;
}

// y of sixteen columns, in every form that is asked for; amax: the row's.
template <bool WIDE>
__device__ __forceinline__ void emit(const NormArgs &a, int q_kind, uint32_t r, int c0, int left, float amax, const F2 (&y)[8]) {
    if (a.y != nullptr) store_values<WIDE>(a.y, a.y_f32, row_at(r, a.ld_y) + c0, left, y);
    if (q_kind == Q_NONE) return;
    if (q_kind == Q_GROUP) amax = group_max(max_of(y));
    const uint32_t byte = emit_fp8(a.fmt, y, amax, a.q + row_at(r, a.ld_q) + c0, left);
    if (left > 0 && (q_kind == Q_ROW ? c0 == 0 : (c0 & 127) == 0))
        a.s[row_at(r, a.ld_s) + (q_kind == Q_ROW ? 0 : c0 >> 7)] = static_cast<uint8_t>(byte);
}

// The first of a thread's sixteen columns: neighbours, or (LANES) every 32nd of its warp's.
template <bool LANES>
__device__ __forceinline__ int first_column(int t) { return LANES ? t / 32 * 512 + t % 32 : t * 16; }

// The parameters to shared memory, by the first group of threads.
template <bool LANES>
__device__ __forceinline__ void keep_both(const NormArgs &a, int group, int t, int tpr, float *w, float *b) {
    if (group == 0) {
        const int c0 = first_column<LANES>(t), left = a.cols - c0;
        F2 v[8];
        if constexpr (LANES) load_params_lanes(a.weight, a.param_f32, 1.0f, c0, left, v);
        else load_params(a.weight, a.param_f32, 1.0f, c0, left, v);
        keep_params(w, t, tpr, v);
        if constexpr (LANES) load_params_lanes(a.bias, a.param_f32, 0.0f, c0, left, v);
        else load_params(a.bias, a.param_f32, 0.0f, c0, left, v);
        keep_params(b, t, tpr, v);
    }
    __syncthreads();
}

// R rows at a time from their values in registers: the mean, the differences, rstd,
// y and where it goes.  The rows' sums share shuffles and a barrier, and their
// parameters are read from shared memory once.
template <bool WIDE, int R, bool LANES = false>
__device__ __forceinline__ void finish(const NormArgs &a, int q_kind, uint32_t r, int t, int tpr, RowReduce &row, const float *w,
                                       const float *b, F2 (&d)[R][8], float (&mean)[R], float (&rstd)[R]) {
    const int c0 = first_column<LANES>(t), cols_left = a.cols - c0;
    const uint32_t rows = a.rows;
    const float n = static_cast<float>(a.cols);
#pragma unroll
    for (int i = 0; i < R; ++i) mean[i] = total(d[i]);
    row.sum(mean, [n](float s) { return s / n; });
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const F2 m = f2(-mean[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[i][j] = add2(d[i][j], m);
        if constexpr (LANES) cut_lanes(d[i], cols_left);
        else cut(d[i], cols_left);
        F2 sq = mul2(d[i][0], d[i][0]), sp = mul2(d[i][1], d[i][1]);
#pragma unroll
        for (int j = 2; j < 8; j += 2) {
            sq = fma2(d[i][j], d[i][j], sq);
            sp = fma2(d[i][j + 1], d[i][j + 1], sp);
        }
        sq = add2(sq, sp);
        rstd[i] = sq.lo() + sq.hi();
    }
    row.sum(rstd, [n, eps = a.eps](float s) { return __frsqrt_rn(s / n + eps); });
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (a.stats != nullptr && t == 0 && r + i < rows) reinterpret_cast<float2 *>(a.stats)[r + i] = make_float2(mean[i], rstd[i]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        F2 w0, w1, b0, b1;
        kept_params(w, t, tpr, j, w0, w1);
        kept_params(b, t, tpr, j, b0, b1);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const F2 s = f2(rstd[i]);
            d[i][2 * j] = fma2(mul2(d[i][2 * j], s), w0, b0);
            d[i][2 * j + 1] = fma2(mul2(d[i][2 * j + 1], s), w1, b1);
        }
    }
    if constexpr (LANES) {      // y alone
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (a.y != nullptr) store_lanes(a.y, a.y_f32, row_at(r + i, a.ld_y) + c0, r + i < rows ? cols_left : 0, d[i]);
    } else {
        float amax[R];
#pragma unroll
        for (int i = 0; i < R; ++i) amax[i] = q_kind == Q_ROW ? max_of(d[i]) : 0.0f;
        if (q_kind == Q_ROW) row.max(amax);
#pragma unroll
        for (int i = 0; i < R; ++i) emit<WIDE>(a, q_kind, r + i, c0, r + i < rows ? cols_left : 0, amax[i], d[i]);
    }
}

template <bool XF32, bool WIDE>
__global__ void __launch_bounds__(512) k_norm(const NormArgs a, int tpr, int q_kind) {
    extern __shared__ float4 params[];    // w, b
    __shared__ float red[2][32][4];
    ptx::grid_begin(static_cast<int64_t>(a.rows) * a.cols);
    RowReduce row(red, tpr);
    const int t = threadIdx.x % tpr, group = threadIdx.x / tpr, rpb = blockDim.x / tpr;
    const int c0 = t * 16, cols_left = a.cols - c0;
    const uint32_t rows = a.rows, step = gridDim.x * rpb;
    uint32_t r = blockIdx.x * rpb + group;
    Raw<XF32> next;
    next.zero();
    if (r < rows && cols_left > 0) next.template load<WIDE>(a.x, row_at(r, a.ld_x) + c0, cols_left);
    float *w = reinterpret_cast<float *>(params), *b = w + 16 * tpr;
    keep_both<false>(a, group, t, tpr, w, b);
    for (uint32_t r0 = blockIdx.x * rpb; r0 < rows; r0 += step, r += step) {
        F2 d[1][8];
        float mean[1], rstd[1];
#pragma unroll
        for (int j = 0; j < 8; ++j) d[0][j] = next.pair(j);
        if (r + step < rows && cols_left > 0) next.template load<WIDE>(a.x, row_at(r + step, a.ld_x) + c0, cols_left);
        finish<WIDE>(a, q_kind, r, t, tpr, row, w, b, d, mean, rstd);
    }
}

// Many rows: R at a time, through shared memory, the next ones' copies in flight.
template <bool XF32, bool WIDE, int R, bool LANES>
__global__ void __launch_bounds__(512) k_norm_ring(const NormArgs a, int tpr, int q_kind) {
    constexpr int X = kSegment<XF32, WIDE>, STAGES = 2;     // bytes of a warp's columns
    extern __shared__ float4 params[];    // w, b, the rings
    __shared__ float red[2][32][4];
    ptx::grid_begin(static_cast<int64_t>(a.rows) * a.cols);
    RowReduce row(red, tpr);
    const int t = threadIdx.x % tpr, group = threadIdx.x / tpr, rpb = blockDim.x / tpr * R, warps = blockDim.x / 32;
    const int w0 = t / 32 * 512;
    const uint32_t rows = a.rows, step = gridDim.x * rpb;
    float *w = reinterpret_cast<float *>(params), *b = w + 16 * tpr;
    const uint32_t ring = ptx::smem_u32(b + 16 * tpr) + threadIdx.x / 32 * X;
    auto copy = [&](uint32_t r, int stage) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            copy_columns<XF32, WIDE, LANES>(ring + (stage * R + i) * warps * X, a.x, row_at(r + i, a.ld_x) + w0, r + i < rows ? a.cols - w0 : 0);
        ptx::cp_async_commit();
    };
    uint32_t r = blockIdx.x * rpb + group * R;
#pragma unroll
    for (int k = 0; k < STAGES; ++k) copy(r + k * step, k);
    keep_both<LANES>(a, group, t, tpr, w, b);
    int stage = 0;
    for (uint32_t r0 = blockIdx.x * rpb; r0 < rows; r0 += step, r += step) {
        ptx::cp_async_wait<STAGES - 1>();
        __syncwarp();
        F2 d[R][8];
        float mean[R], rstd[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            Raw<XF32> x;
            const uint32_t from = ring + (stage * R + i) * warps * X, shift = column_address<XF32>(a.x, row_at(r + i, a.ld_x)) & 15;
            const int left = r + i < rows ? a.cols - first_column<LANES>(t) : 0;
            if constexpr (LANES) read_lanes<XF32>(from, shift, left, x);
            else read_columns<XF32, WIDE>(from, shift, left, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) d[i][j] = x.pair(j);
        }
        __syncwarp();
        copy(r + STAGES * step, stage);
        stage ^= 1;
        finish<WIDE, R, LANES>(a, q_kind, r, t, tpr, row, w, b, d, mean, rstd);
    }
    ptx::cp_async_wait<0>();
}

// Rows of any length, a CTA each: the row is read for each of its sums, in
// pieces of 16 columns a thread.
template <bool XF32>
__global__ void __launch_bounds__(512) k_norm_long(const NormArgs a, int q_kind) {
    __shared__ float red[2][32][4];
    ptx::grid_wait();
    const int tpr = blockDim.x;
    RowReduce row(red, tpr);
    const uint32_t rows = a.rows;
    for (uint32_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const int64_t at = row_at(r, a.ld_x);
        auto piece = [&](int64_t c0, F2 (&v)[8]) {
            Raw<XF32> x;
            x.template load<false>(a.x, at + c0, static_cast<int>(a.cols - c0));
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = x.pair(i);
        };
        const int64_t first = threadIdx.x * 16, pass = tpr * 16;
        float s = 0.0f;
        for (int64_t c0 = first; c0 < a.cols; c0 += pass) {
            F2 v[8];
            piece(c0, v);
            s += total(v);
        }
        const float n = static_cast<float>(a.cols), mean = row.sum(s) / n;
        s = 0.0f;
        for (int64_t c0 = first; c0 < a.cols; c0 += pass) {
            F2 v[8];
            piece(c0, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = add2(v[i], f2(-mean));
            cut(v, static_cast<int>(a.cols - c0));
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = mul2(v[i], v[i]);
            s += total(v);
        }
        const float rstd = __frsqrt_rn(row.sum(s) / n + a.eps);
        if (a.stats != nullptr && threadIdx.x == 0) reinterpret_cast<float2 *>(a.stats)[r] = make_float2(mean, rstd);
        auto value = [&](int64_t c0, F2 (&v)[8]) {
            const int left = static_cast<int>(a.cols - c0);
            F2 w[8], b[8];
            load_params(a.weight, a.param_f32, 1.0f, static_cast<int>(c0), left, w);
            load_params(a.bias, a.param_f32, 0.0f, static_cast<int>(c0), left, b);
            if (left > 0) piece(c0, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = fma2(mul2(add2(v[i], f2(-mean)), f2(rstd)), w[i], b[i]);
            cut(v, left);
        };
        float amax = 0.0f;
        if (q_kind == Q_ROW) {
            for (int64_t c0 = first; c0 < a.cols; c0 += pass) {
                F2 v[8];
                value(c0, v);
                amax = max3_abs(amax, amax, max_of(v));
            }
            amax = row.max(amax);
        }
        // whole warps: the stores exchange values between lanes
        for (int64_t c0 = first; c0 - (threadIdx.x & 31) * 16 < a.cols; c0 += pass) {
            F2 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = f2(0.0f);
            value(c0, v);
            emit<false>(a, q_kind, r, static_cast<int>(c0), static_cast<int>(a.cols - c0), amax, v);
        }
        __syncthreads();   // a warp past its last piece is not a row ahead of the sums
    }
}

// Copies ahead pay off where every CTA, two an SM, has two sets of rows at least
// (16384 x 3584 with codes: 47 us with them, 57 without).  BF16 rows of more than 4096
// columns would leave room for one CTA an SM (8192 x 4999 with codes: 62 us instead of
// 57).  Rows at odd addresses without codes: every 32nd column a lane, one row at a time
// from 4096 columns on, three CTAs an SM where it holds them (BF16, 8192 x 4999: 52 us,
// 59 with sixteen neighbours a lane; 8192 x 7999 80 and 97; FP32 61 and 69, 109 and 125).
template <bool XF32, bool WIDE, int R, bool LANES>
cudaError_t run_ring(const NormArgs &a, const Shape &s, int q_kind, cudaStream_t stream) {
    constexpr int kWarpBytes = 2 * R * kSegment<XF32, WIDE>;
    static unsigned long long done;
    const int threads = s.tpr * s.rpb;
    const size_t smem = 2 * 16 * sizeof(float) * s.tpr + kWarpBytes * (threads / 32);
    const cudaError_t e = with_smem(&k_norm_ring<XF32, WIDE, R, LANES>, smem, 64 * 1024 + kWarpBytes * 16, done);
    if (e != cudaSuccess) return e;
    const int sets = (a.rows + s.rpb * R - 1) / (s.rpb * R);
    return launch_after(&k_norm_ring<XF32, WIDE, R, LANES>, dim3(std::min(sets, kSms * std::max(2, (LANES && R == 1 && !XF32 ? 1024 : 512) / threads))), threads, smem, stream, 1, a, s.tpr,
                        q_kind);
}
template <bool XF32, bool WIDE>
cudaError_t run(const NormArgs &a, int q_kind, cudaStream_t stream) {
    const Shape s = shape_of(a.cols);
    const int threads = s.tpr * s.rpb;
    const size_t params = 2 * 16 * sizeof(float) * s.tpr;
    constexpr int R = XF32 ? 1 : WIDE ? 4 : 2;
    if constexpr (!WIDE) {
        if (q_kind == Q_NONE && threads <= 256 && a.rows >= 4 * R * s.rpb * kSms) return run_ring<XF32, false, R, true>(a, s, q_kind, stream);
        if (q_kind == Q_NONE && threads > 256 && a.rows >= 4 * kSms) return run_ring<XF32, false, 1, true>(a, s, q_kind, stream);
    }
    if (threads <= (XF32 ? 512 : 256) && a.rows >= 4 * R * s.rpb * kSms) return run_ring<XF32, WIDE, R, false>(a, s, q_kind, stream);
    static unsigned long long done;
    const cudaError_t e = with_smem(&k_norm<XF32, WIDE>, params, 2 * 16 * sizeof(float) * 512, done);
    if (e != cudaSuccess) return e;
    const int grid = std::min((a.rows + s.rpb - 1) / s.rpb, kSms * std::max(1, 1024 / threads));
    return launch_after(&k_norm<XF32, WIDE>, dim3(grid), threads, params, stream, 1, a, s.tpr, q_kind);
}

}  // namespace

cudaError_t launch_norm(const NormArgs &a, cudaStream_t stream) {
    const int q_kind = a.q == nullptr ? Q_NONE : a.group == 0 ? Q_ROW : Q_GROUP;
    if (a.cols > kRegCols) {
        const dim3 grid(std::min(a.rows, 4 * kSms));
        return a.x_f32 ? launch_after(&k_norm_long<true>, grid, 512, 0, stream, 1, a, q_kind)
                       : launch_after(&k_norm_long<false>, grid, 512, 0, stream, 1, a, q_kind);
    }
    const bool wide = wide_rows(a.x, a.x_f32, a.ld_x) && (a.y == nullptr || wide_rows(a.y, a.y_f32, a.ld_y));
    if (a.x_f32) return wide ? run<true, true>(a, q_kind, stream) : run<true, false>(a, q_kind, stream);
    return wide ? run<false, true>(a, q_kind, stream) : run<false, false>(a, q_kind, stream);
}

}  // namespace fp8hg
