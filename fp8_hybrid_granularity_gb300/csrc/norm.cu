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

template <bool XF32, bool WIDE>
__global__ void __launch_bounds__(512) k_norm(const NormArgs a, int tpr, int q_kind) {
    extern __shared__ float4 params[];    // w, b
    __shared__ float red[2][32][4];
    ptx::grid_begin(static_cast<int64_t>(a.rows) * a.cols);
    RowReduce row(red, tpr);
    const int t = threadIdx.x % tpr, group = threadIdx.x / tpr, rpb = blockDim.x / tpr;
    const int c0 = t * 16, cols_left = a.cols - c0;
    const uint32_t rows = a.rows, step = gridDim.x * rpb;
    const float inv_n = 1.0f / static_cast<float>(a.cols);
    uint32_t r = blockIdx.x * rpb + group;
    Raw<XF32> next;
    next.zero();
    if (r < rows && cols_left > 0) next.template load<WIDE>(a.x, row_at(r, a.ld_x) + c0, cols_left);
    float *w = reinterpret_cast<float *>(params), *b = w + 16 * tpr;
    if (group == 0) {
        F2 v[8];
        load_params(a.weight, a.param_f32, 1.0f, c0, cols_left, v);
        keep_params(w, t, tpr, v);
        load_params(a.bias, a.param_f32, 0.0f, c0, cols_left, v);
        keep_params(b, t, tpr, v);
    }
    __syncthreads();
    for (uint32_t r0 = blockIdx.x * rpb; r0 < rows; r0 += step, r += step) {
        F2 d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = next.pair(i);
        if (r + step < rows && cols_left > 0) next.template load<WIDE>(a.x, row_at(r + step, a.ld_x) + c0, cols_left);
        const float mean = row.sum(total(d)) * inv_n;
        const F2 m = f2(-mean);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = add2(d[i], m);
        cut(d, cols_left);
        F2 sq = mul2(d[0], d[0]), sp = mul2(d[1], d[1]);
#pragma unroll
        for (int i = 2; i < 8; i += 2) {
            sq = fma2(d[i], d[i], sq);
            sp = fma2(d[i + 1], d[i + 1], sp);
        }
        sq = add2(sq, sp);
        const float rstd = 1.0f / sqrtf(row.sum(sq.lo() + sq.hi()) * inv_n + a.eps);
        if (a.stats != nullptr && t == 0 && r < rows)
            reinterpret_cast<float2 *>(a.stats)[r] = make_float2(mean, rstd);
        const F2 s = f2(rstd);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            F2 w0, w1, b0, b1;
            kept_params(w, t, tpr, j, w0, w1);
            kept_params(b, t, tpr, j, b0, b1);
            d[2 * j] = fma2(mul2(d[2 * j], s), w0, b0);
            d[2 * j + 1] = fma2(mul2(d[2 * j + 1], s), w1, b1);
        }
        const float amax = q_kind == Q_ROW ? row.max(max_of(d)) : 0.0f;
        emit<WIDE>(a, q_kind, r, c0, r < rows ? cols_left : 0, amax, d);
    }
}

// Rows of any length, a CTA each: the row is read for each of its sums, in
// pieces of 16 columns a thread.
template <bool XF32>
__global__ void __launch_bounds__(512) k_norm_long(const NormArgs a, int q_kind) {
    __shared__ float red[2][32][4];
    ptx::grid_wait();
    const int tpr = blockDim.x;
    RowReduce row(red, tpr);
    const float inv_n = 1.0f / static_cast<float>(a.cols);
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
        const float mean = row.sum(s) * inv_n;
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
        const float rstd = 1.0f / sqrtf(row.sum(s) * inv_n + a.eps);
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

template <bool XF32, bool WIDE>
cudaError_t run(const NormArgs &a, int q_kind, cudaStream_t stream) {
    const Shape s = shape_of(a.cols);
    const int threads = s.tpr * s.rpb;
    const int grid = std::min((a.rows + s.rpb - 1) / s.rpb, kSms * std::max(1, 1024 / threads));
    const size_t smem = 2 * 16 * sizeof(float) * s.tpr;
    auto *kern = &k_norm<XF32, WIDE>;
    static unsigned long long done;
    const cudaError_t e = with_smem(kern, smem, 2 * 16 * sizeof(float) * 512, done);
    if (e != cudaSuccess) return e;
    return launch_after(kern, dim3(grid), threads, smem, stream, 1, a, s.tpr, q_kind);
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
