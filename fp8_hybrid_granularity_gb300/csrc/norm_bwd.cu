// Layer norm, backward.
//
//   xh = (x - mean) rstd,  g = dy w
//   dx = rstd (g - sum(g) / n - xh sum(g xh) / n) [+ add]
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// in FP32 between the loads and the stores, from the statistics that the
// forward pass kept.  Bound by HBM: x, dy (and add) are read once, dx written
// once.  Laid out like the forward pass (a row in registers, 16 columns a thread);
// the sums for dw and db stay in registers over all rows of a CTA and leave as
// one row of partial sums per CTA, which a second kernel adds in a fixed order:
// results do not depend on timing.  Rows of more than 8192 columns are read twice
// for dx and once before, by columns, for dw and db.
//
// 16384 x 3584, BF16 x, dy, add and dx: 93 us in a stream of calls for 470 MB, 75 % of
// the copy rate (rows loaded into registers instead of through shared memory: 99).
// What is left are the barrier of every pair of rows and the registers of the sums,
// which leave room for 16 warps an SM.  4096 x 12288, in BF16: 230 us for 302 MB.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "norm.cuh"

namespace fp8hg {

namespace {

using namespace norm;

// Sixteen columns' sums of dw and db of one row after the other into `sums`: neighbours,
// or a warp's width apart.
template <int STEP = 1>
__device__ __forceinline__ void gather(float *sums, int cols, int c0, bool first, const F2 (&dw)[8], const F2 (&db)[8]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int c = c0 + i * STEP;
        if (c < cols) {
            const float vw = i & 1 ? dw[i / 2].hi() : dw[i / 2].lo();
            const float vb = i & 1 ? db[i / 2].hi() : db[i / 2].lo();
            sums[c] = first ? vw : sums[c] + vw;
            sums[cols + c] = first ? vb : sums[cols + c] + vb;
        }
    }
}

template <bool XF32, bool DF32, bool WIDE>
__global__ void __launch_bounds__(512) k_norm_bwd(const NormBwdArgs a, int tpr) {
    extern __shared__ float4 shared[];     // w; after the last row the sums, [2][cols], of several rows at a time
    __shared__ float red[2][32][4];
    ptx::grid_begin(static_cast<int64_t>(a.rows) * a.cols);
    RowReduce row(red, tpr);
    const int t = threadIdx.x % tpr, rpb = blockDim.x / tpr;
    const int c0 = t * 16, cols_left = a.cols - c0;
    const uint32_t rows = a.rows, step = gridDim.x * rpb;
    const float inv_n = 1.0f / static_cast<float>(a.cols);
    Raw<XF32> nx, add;
    Raw<DF32> nd;
    nx.zero();
    nd.zero();
    add.zero();
    float2 nst = make_float2(0.0f, 0.0f);
    auto load = [&](uint32_t r) {
        if (r < rows && cols_left > 0) {
            nst = reinterpret_cast<const float2 *>(a.stats)[r];
            nx.template load<WIDE>(a.x, row_at(r, a.ld_x) + c0, cols_left);
            nd.template load<WIDE>(a.dy, row_at(r, a.ld_dy) + c0, cols_left);
        }
    };
    uint32_t r = blockIdx.x * rpb + threadIdx.x / tpr;
    load(r);
    float *w = reinterpret_cast<float *>(shared);
    if (threadIdx.x < tpr) {
        F2 v[8];
        load_params(a.weight, a.param_f32, 1.0f, c0, cols_left, v);
        keep_params(w, t, tpr, v);
    }
    __syncthreads();
    F2 dw[8], db[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[i] = db[i] = f2(0.0f);
    for (uint32_t r0 = blockIdx.x * rpb; r0 < rows; r0 += step, r += step) {
        const bool in = r < rows;
        if (a.add != nullptr && in && cols_left > 0) add.template load<WIDE>(a.add, row_at(r, a.ld_add) + c0, cols_left);
        const float mean = nst.x, rstd = nst.y;
        F2 xh[8], g[8], p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            xh[i] = mul2(add2(nx.pair(i), f2(-mean)), f2(rstd));
            g[i] = nd.pair(i);
        }
        load(r + step);
        if (in) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dw[i] = fma2(g[i], xh[i], dw[i]);
                db[i] = add2(db[i], g[i]);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            F2 w0, w1;
            kept_params(w, t, tpr, j, w0, w1);
            g[2 * j] = mul2(g[2 * j], w0);
            g[2 * j + 1] = mul2(g[2 * j + 1], w1);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = mul2(g[i], xh[i]);
        const float2 s = row.both(total(g), total(p));
        const F2 mg = f2(-s.x * inv_n), mgx = f2(-s.y * inv_n);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = fma2(f2(rstd), fma2(xh[i], mgx, add2(g[i], mg)), add.pair(i));
        store_values<WIDE>(a.dx, XF32, row_at(r, a.ld_dx) + c0, in ? cols_left : 0, g);
    }
    if (a.ws == nullptr) return;
    float *part = a.ws + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
    if (rpb == 1) {
        store_values<false>(part, 1, c0, cols_left, dw);
        store_values<false>(part, 1, a.cols + c0, cols_left, db);
        return;
    }
    __syncthreads();
    for (int q = 0; q < rpb; ++q) {
        if (threadIdx.x / tpr == q) gather(w, a.cols, c0, q == 0, dw, db);
        __syncthreads();
    }
    for (int c = threadIdx.x; c < 2 * a.cols; c += blockDim.x) part[c] = w[c];
}

// The same with rows that come through shared memory, STAGES - 1 sets of R ahead (the
// sums of a set share a barrier).
template <bool XF32, bool DF32, bool WIDE, int THREADS>
struct Ring {
    static constexpr int R = XF32 || DF32 || !WIDE || THREADS > 256 ? 1 : 2;
    static constexpr int CTAS = THREADS <= 320 ? 2 : 1;
    static constexpr int STAGES = R == 1 && THREADS != 320 && (THREADS == 256 || !(XF32 || DF32)) ? 3 : 2;
    // rows at odd addresses: a lane has every 32nd of the warp's 512 columns, which need no
    // moving into place (FP32 x, 8192 x 5001: 94 us, 133 with sixteen neighbours; BF16 71
    // and 88)
    static constexpr int STEP = WIDE ? 1 : 32;
    static constexpr int X = kSegment<XF32, WIDE>, D = kSegment<DF32, WIDE>;     // bytes of a warp's columns
    static constexpr int bytes(int warps, bool add) { return STAGES * R * (X + D + (add ? X : 0)) * warps; }
};

template <bool XF32, bool DF32, bool WIDE, int THREADS>
__global__ void __launch_bounds__(THREADS, Ring<XF32, DF32, WIDE, THREADS>::CTAS) k_norm_bwd_ring(const NormBwdArgs a, int tpr) {
    using S = Ring<XF32, DF32, WIDE, THREADS>;
    constexpr int R = S::R;
    extern __shared__ float4 shared[];     // the rings, w; after the last row the sums, [2][cols], of several rows at a time
    __shared__ float red[2][32][4];
    ptx::grid_begin(static_cast<int64_t>(a.rows) * a.cols);
    RowReduce row(red, tpr);
    const int t = threadIdx.x % tpr, group = threadIdx.x / tpr, warps = blockDim.x / 32, rpb = blockDim.x / tpr * R;
    constexpr int STEP = S::STEP;
    const int w0 = t / 32 * 512, c0 = STEP == 1 ? t * 16 : w0 + threadIdx.x % 32, cols_left = a.cols - c0;
    const uint32_t rows = a.rows, step = gridDim.x * rpb;
    const float inv_n = 1.0f / static_cast<float>(a.cols);
    const bool with_add = a.add != nullptr;
    const int set = S::X + S::D + (with_add ? S::X : 0);
    const uint32_t ring = ptx::smem_u32(shared) + threadIdx.x / 32 * set;
    auto slot = [&](int stage, int i) { return ring + (stage * R + i) * warps * set; };
    float2 st[S::STAGES - 1][R];
    uint32_t r = blockIdx.x * rpb + group * R;
    auto copy = [&](uint32_t r, int stage) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int left = r + i < rows ? a.cols - w0 : 0;
            copy_columns<XF32, WIDE, !WIDE>(slot(stage, i), a.x, row_at(r + i, a.ld_x) + w0, left);
            copy_columns<DF32, WIDE, !WIDE>(slot(stage, i) + S::X, a.dy, row_at(r + i, a.ld_dy) + w0, left);
            if (with_add) copy_columns<XF32, WIDE, !WIDE>(slot(stage, i) + S::X + S::D, a.add, row_at(r + i, a.ld_add) + w0, left);
        }
        ptx::cp_async_commit();
    };
    auto stat = [&](uint32_t r) { return r < rows ? reinterpret_cast<const float2 *>(a.stats)[r] : make_float2(0.0f, 0.0f); };
#pragma unroll
    for (int k = 0; k < S::STAGES; ++k) copy(r + k * step, k);
#pragma unroll
    for (int k = 0; k < S::STAGES - 1; ++k)
#pragma unroll
        for (int i = 0; i < R; ++i) st[k][i] = stat(r + k * step + i);
    float *w = reinterpret_cast<float *>(shared) + S::STAGES * R * warps * set / 4;
    if (group == 0) {
        F2 v[8];
        if constexpr (WIDE) load_params(a.weight, a.param_f32, 1.0f, c0, cols_left, v);
        else load_params_lanes(a.weight, a.param_f32, 1.0f, c0, cols_left, v);
        keep_params(w, t, tpr, v);
    }
    __syncthreads();
    F2 dw[8], db[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[i] = db[i] = f2(0.0f);
    int stage = 0;
    for (uint32_t r0 = blockIdx.x * rpb; r0 < rows; r0 += step, r += step) {
        ptx::cp_async_wait<S::STAGES - 1>();
        __syncwarp();
        Raw<XF32> x[R];
        Raw<DF32> dy[R];
        float sums[2 * R], mean[R], rstd[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int here = r + i < rows ? cols_left : 0;
            const uint32_t shift_x = column_address<XF32>(a.x, row_at(r + i, a.ld_x)) & 15, shift_d = column_address<DF32>(a.dy, row_at(r + i, a.ld_dy)) & 15;
            if constexpr (WIDE) {
                read_columns<XF32, true>(slot(stage, i), shift_x, here, x[i]);
                read_columns<DF32, true>(slot(stage, i) + S::X, shift_d, here, dy[i]);
            } else {
                read_lanes<XF32>(slot(stage, i), shift_x, here, x[i]);
                read_lanes<DF32>(slot(stage, i) + S::X, shift_d, here, dy[i]);
            }
            mean[i] = st[0][i].x, rstd[i] = st[0][i].y;
        }
#pragma unroll
        for (int k = 0; k + 1 < S::STAGES - 1; ++k)
#pragma unroll
            for (int i = 0; i < R; ++i) st[k][i] = st[k + 1][i];
#pragma unroll
        for (int i = 0; i < R; ++i) st[S::STAGES - 2][i] = stat(r + (S::STAGES - 1) * step + i);
        // rows past the last are zeros, and so are their statistics
#pragma unroll
        for (int i = 0; i < R; ++i) {
            F2 sg = f2(0.0f), sgx = f2(0.0f);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                F2 wj[2];
                kept_params(w, t, tpr, j, wj[0], wj[1]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const F2 d = dy[i].pair(2 * j + e), xh = mul2(add2(x[i].pair(2 * j + e), f2(-mean[i])), f2(rstd[i]));
                    dw[2 * j + e] = fma2(d, xh, dw[2 * j + e]);
                    db[2 * j + e] = add2(db[2 * j + e], d);
                    const F2 g = mul2(d, wj[e]);
                    sg = add2(sg, g);
                    sgx = fma2(g, xh, sgx);
                }
            }
            sums[2 * i] = sg.lo() + sg.hi();
            sums[2 * i + 1] = sgx.lo() + sgx.hi();
        }
        row.sum(sums);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const F2 mg = f2(-sums[2 * i] * inv_n), mgx = f2(-sums[2 * i + 1] * inv_n), rs = f2(rstd[i]);
            Raw<XF32> add;
            add.zero();
            if (with_add) {
                const uint32_t shift = column_address<XF32>(a.add, row_at(r + i, a.ld_add)) & 15;
                if constexpr (WIDE) read_columns<XF32, true>(slot(stage, i) + S::X + S::D, shift, cols_left, add);
                else read_lanes<XF32>(slot(stage, i) + S::X + S::D, shift, cols_left, add);
            }
            F2 dx[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                F2 wj[2];
                kept_params(w, t, tpr, j, wj[0], wj[1]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const F2 xh = mul2(add2(x[i].pair(2 * j + e), f2(-mean[i])), rs), g = mul2(dy[i].pair(2 * j + e), wj[e]);
                    dx[2 * j + e] = fma2(rs, fma2(xh, mgx, add2(g, mg)), add.pair(2 * j + e));
                }
            }
            if constexpr (!WIDE) store_lanes(a.dx, XF32, row_at(r + i, a.ld_dx) + c0, r + i < rows ? cols_left : 0, dx);
            else store_values<WIDE>(a.dx, XF32, row_at(r + i, a.ld_dx) + c0, r + i < rows ? cols_left : 0, dx);
        }
        __syncwarp();
        copy(r + S::STAGES * step, stage);
        stage = stage + 1 == S::STAGES ? 0 : stage + 1;
    }
    ptx::cp_async_wait<0>();
    if (a.ws == nullptr) return;
    float *part = a.ws + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
    if (blockDim.x == tpr) {
        if constexpr (!WIDE) {
            store_lanes(part, 1, c0, cols_left, dw);
            store_lanes(part, 1, a.cols + c0, cols_left, db);
        } else {
            store_values<false>(part, 1, c0, cols_left, dw);
            store_values<false>(part, 1, a.cols + c0, cols_left, db);
        }
        return;
    }
    __syncthreads();
    for (int q = 0; q < static_cast<int>(blockDim.x) / tpr; ++q) {
        if (group == q) gather<STEP>(w, a.cols, c0, q == 0, dw, db);
        __syncthreads();
    }
    for (int c = threadIdx.x; c < 2 * a.cols; c += blockDim.x) part[c] = w[c];
}

// dx of rows of any length, a CTA each.
template <bool XF32, bool DF32>
__global__ void __launch_bounds__(512) k_norm_bwd_long(const NormBwdArgs a) {
    __shared__ float red[2][32][4];
    ptx::grid_wait();
    const int tpr = blockDim.x;
    RowReduce row(red, tpr);
    const float inv_n = 1.0f / static_cast<float>(a.cols);
    const uint32_t rows = a.rows;
    for (uint32_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const float2 st = reinterpret_cast<const float2 *>(a.stats)[r];
        F2 xh[8], g[8];
        auto piece = [&](int64_t c0) {
            const int left = static_cast<int>(a.cols - c0);
            Raw<XF32> x;
            Raw<DF32> dy;
            x.template load<false>(a.x, row_at(r, a.ld_x) + c0, left);
            dy.template load<false>(a.dy, row_at(r, a.ld_dy) + c0, left);
            F2 w[8];
            load_params(a.weight, a.param_f32, 1.0f, static_cast<int>(c0), left, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                xh[i] = mul2(add2(x.pair(i), f2(-st.x)), f2(st.y));
                g[i] = mul2(dy.pair(i), w[i]);
            }
        };
        const int64_t first = threadIdx.x * 16, pass = tpr * 16;
        float sg = 0.0f, sgx = 0.0f;
        for (int64_t c0 = first; c0 < a.cols; c0 += pass) {
            piece(c0);
            F2 p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = mul2(g[i], xh[i]);
            sg += total(g);
            sgx += total(p);
        }
        const float2 s = row.both(sg, sgx);
        const F2 mg = f2(-s.x * inv_n), mgx = f2(-s.y * inv_n);
        for (int64_t c0 = first; c0 - (threadIdx.x & 31) * 16 < a.cols; c0 += pass) {
            const int left = static_cast<int>(a.cols - c0);
            Raw<XF32> add;
            add.zero();
            if (left > 0) {
                piece(c0);
                if (a.add != nullptr) add.template load<false>(a.add, row_at(r, a.ld_add) + c0, left);
            }
            F2 dx[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) dx[i] = fma2(f2(st.y), fma2(xh[i], mgx, add2(g[i], mg)), add.pair(i));
            store_values<false>(a.dx, XF32, row_at(r, a.ld_dx) + c0, left, dx);
        }
        __syncthreads();   // a warp past its last piece is not a row ahead of the sums
    }
}

// Partial sums for dw and db of such rows: a warp takes 512 columns of every
// eighth row of the CTA's part.
constexpr int kColRows = 256;
template <bool XF32, bool DF32>
__global__ void __launch_bounds__(256) k_norm_columns(const NormBwdArgs a) {
    __shared__ float sums[2 * 512];
    ptx::grid_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int64_t base = static_cast<int64_t>(blockIdx.x) * 512, c0 = base + lane * 16;
    const int left = static_cast<int>(a.cols - c0);
    const uint32_t per = (static_cast<uint32_t>(a.rows) + gridDim.y - 1) / gridDim.y, from = blockIdx.y * per;
    const uint32_t to = min(static_cast<uint32_t>(a.rows), from + per);
    F2 dw[8], db[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[i] = db[i] = f2(0.0f);
    if (left > 0) {
        for (uint32_t r = from + warp; r < to; r += 8) {
            Raw<XF32> x;
            Raw<DF32> dy;
            x.template load<false>(a.x, row_at(r, a.ld_x) + c0, left);
            dy.template load<false>(a.dy, row_at(r, a.ld_dy) + c0, left);
            const float2 st = reinterpret_cast<const float2 *>(a.stats)[r];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dw[i] = fma2(dy.pair(i), mul2(add2(x.pair(i), f2(-st.x)), f2(st.y)), dw[i]);
                db[i] = add2(db[i], dy.pair(i));
            }
        }
    }
    for (int q = 0; q < 8; ++q) {
        if (warp == q) gather(sums, 512, lane * 16, q == 0, dw, db);
        __syncthreads();
    }
    float *part = a.ws + static_cast<int64_t>(blockIdx.y) * 2 * a.cols;
    for (int i = threadIdx.x; i < 512; i += 256) {
        if (base + i < a.cols) {
            part[base + i] = sums[i];
            part[a.cols + base + i] = sums[512 + i];
        }
    }
}

// Partial sums [parts][2 cols] to dw and db: 32 columns a CTA, 16 warps that
// take every 16th row each.
__global__ void __launch_bounds__(512) k_norm_sums(const float *ws, int parts, int cols, float *dweight, float *dbias) {
    __shared__ float sums[16][33];
    ptx::grid_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane, n = 2 * static_cast<int64_t>(cols);
    float s = 0.0f;
    if (c < n) {
#pragma unroll 4
        for (int p = warp; p < parts; p += 16) s += ptx::ld_f32(ws + p * n + c);
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < n) {
#pragma unroll
        for (int i = 1; i < 16; ++i) s += sums[i][lane];
        float *to = c < cols ? dweight : dbias;
        if (to != nullptr) to[c < cols ? c : c - cols] = s;
    }
}

// BF16 rows of 4097 to 5120 columns: 320 threads at 96 registers, two CTAs an SM, where
// the rows cover the second CTA's partial sums (8192 x 5008: 55 us instead of 66, 1500 x
// 4608 21 instead of 19; FP32 spills: 92 instead of 81).
bool pairs(int threads, int64_t rows, bool bf16) { return bf16 && threads > 256 && threads <= 320 && rows >= 2048; }
// Rows of partial sums for dw and db: CTAs of the kernel that makes them.
int norm_parts(int64_t rows, int64_t cols, bool bf16) {
    if (cols > kRegCols) return static_cast<int>(std::min<int64_t>((rows + kColRows - 1) / kColRows, 32));
    const Shape s = shape_of(cols);
    const int threads = s.tpr * s.rpb, ctas = pairs(threads, rows, bf16) ? 2 : std::max(1, 512 / threads);
    return static_cast<int>(std::min<int64_t>((rows + s.rpb - 1) / s.rpb, kSms * ctas));
}

constexpr size_t kMostSmem = 226 * 1024;
template <bool XF32, bool DF32, bool WIDE, int THREADS>
cudaError_t run_ring(const NormBwdArgs &a, const Shape &s, int parts, size_t smem, cudaStream_t stream) {
    static unsigned long long done;
    auto *kern = &k_norm_bwd_ring<XF32, DF32, WIDE, THREADS>;
    const cudaError_t e = with_smem(kern, smem, kMostSmem, done);
    if (e != cudaSuccess) return e;
    return launch_after(kern, dim3(parts), s.tpr * s.rpb, smem, stream, 1, a, s.tpr);
}
// Through shared memory where it holds the rows (all in FP32, with another gradient to
// add, it does not from 6000 columns on).
template <bool XF32, bool DF32, bool WIDE>
cudaError_t run_rows(const NormBwdArgs &a, const Shape &s, int parts, cudaStream_t stream) {
    const int threads = s.tpr * s.rpb, warps = threads / 32;
    const size_t rest = (s.rpb > 1 ? 2 : 1) * 16 * sizeof(float) * s.tpr;   // at most 32 KB
    if constexpr (!XF32 && !DF32) {
        if (pairs(threads, a.rows, true))
            return run_ring<false, false, WIDE, 320>(a, s, parts, rest + Ring<false, false, WIDE, 320>::bytes(warps, a.add != nullptr), stream);
    }
    const size_t rings = threads <= 256 ? Ring<XF32, DF32, WIDE, 256>::bytes(warps, a.add != nullptr)
                                        : Ring<XF32, DF32, WIDE, 512>::bytes(warps, a.add != nullptr);
    if (rest + rings > kMostSmem) return launch_after(&k_norm_bwd<XF32, DF32, WIDE>, dim3(parts), threads, rest, stream, 1, a, s.tpr);
    return threads <= 256 ? run_ring<XF32, DF32, WIDE, 256>(a, s, parts, rest + rings, stream)
                          : run_ring<XF32, DF32, WIDE, 512>(a, s, parts, rest + rings, stream);
}

template <bool XF32, bool DF32>
cudaError_t run(const NormBwdArgs &a, cudaStream_t stream) {
    const int parts = norm_parts(a.rows, a.cols, !XF32 && !DF32);
    cudaError_t e;
    if (a.cols > kRegCols) {
        // dw and db first: dx may be dy or x
        e = a.ws == nullptr ? cudaSuccess : launch_after(&k_norm_columns<XF32, DF32>, dim3((a.cols + 511) / 512, parts), 256, 0, stream, 1, a);
        if (e == cudaSuccess) e = launch_after(&k_norm_bwd_long<XF32, DF32>, dim3(std::min(a.rows, 2 * kSms)), 512, 0, stream, 1, a);
    } else {
        const Shape s = shape_of(a.cols);
        const bool wide = wide_rows(a.x, a.x_f32, a.ld_x) && wide_rows(a.dy, a.dy_f32, a.ld_dy) &&
                          wide_rows(a.dx, a.x_f32, a.ld_dx) && (a.add == nullptr || wide_rows(a.add, a.x_f32, a.ld_add));
        e = wide ? run_rows<XF32, DF32, true>(a, s, parts, stream) : run_rows<XF32, DF32, false>(a, s, parts, stream);
    }
    if (e != cudaSuccess || a.ws == nullptr) return e;
    return launch_after(&k_norm_sums, dim3(static_cast<unsigned>((2 * static_cast<int64_t>(a.cols) + 31) / 32)), 512, 0,
                        stream, 1, static_cast<const float *>(a.ws), parts, a.cols, a.dweight, a.dbias);
}

}  // namespace

size_t norm_bwd_ws_bytes(int64_t rows, int64_t cols) {
    return static_cast<size_t>(norm_parts(rows, cols, true)) * 2 * static_cast<size_t>(cols) * sizeof(float);
}

cudaError_t launch_norm_bwd(const NormBwdArgs &a, cudaStream_t stream) {
    if (a.x_f32) return a.dy_f32 ? run<true, true>(a, stream) : run<true, false>(a, stream);
    return a.dy_f32 ? run<false, true>(a, stream) : run<false, false>(a, stream);
}

}  // namespace fp8hg
