// C-ABI entry points of the layer norm and of the low-rank adapters (declared in
// include/fp8hg_adapt.h): argument validation, then the launches.  Nothing here
// allocates device memory or synchronizes.
#include <cuda_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>

#include "../../include/fp8hg_adapt.h"
#include "adapt.h"

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 30;
constexpr int64_t kMaxLd = 0x7FFFFFFF;
constexpr int64_t kMaxTokens = int64_t(1) << 24;
constexpr int64_t kMaxSide = int64_t(1) << 24;      // of a projection

inline bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline int status_from_cuda(cudaError_t e) { return e == cudaSuccess ? FP8HG_OK : FP8HG_ERR_CUDA; }
inline bool valid_kind(int k) { return k == FP8HG_OUT_BF16 || k == FP8HG_OUT_FP32; }
inline uintptr_t size_of(int kind) { return kind == FP8HG_OUT_FP32 ? 4 : 2; }
inline uint32_t u32(int64_t v) { return static_cast<uint32_t>(v); }   // a checked stride

int check_dims(int64_t a, int64_t b) {
    if (a < 0 || b < 0) return FP8HG_ERR_INVALID_ARG;
    return a > kMaxDim || b > kMaxDim ? FP8HG_ERR_SHAPE : FP8HG_OK;
}

// A matrix of `cols` columns with elements of `size` bytes that is there.
int check_matrix(const void *p, int64_t cols, int64_t ld, uintptr_t size) {
    if (!p || ld < cols) return FP8HG_ERR_INVALID_ARG;
    if (ld > kMaxLd) return FP8HG_ERR_SHAPE;
    return aligned(p, size) ? FP8HG_OK : FP8HG_ERR_ALIGNMENT;
}
int check_vector(const void *p, uintptr_t size) { return aligned(p, size) ? FP8HG_OK : FP8HG_ERR_ALIGNMENT; }

int check_plan(const void *plan, int64_t tokens, int64_t adapters) {
    if (tokens < 0 || adapters < 1) return FP8HG_ERR_INVALID_ARG;
    if (tokens > kMaxTokens || adapters > fp8hg::kLoraMaxAdapters) return FP8HG_ERR_SHAPE;
    if (!plan) return FP8HG_ERR_INVALID_ARG;
    return aligned(plan, 16) ? FP8HG_OK : FP8HG_ERR_ALIGNMENT;
}

fp8hg::LoraPlan plan_of(const void *plan, int64_t tokens, int64_t adapters) {
    return {static_cast<const int *>(plan), static_cast<int>(tokens), static_cast<int>(adapters)};
}

int check_lora(const fp8hg_lora *w) {
    if (!w) return FP8HG_ERR_INVALID_ARG;
    const int st = check_dims(w->n, w->k);
    if (st != FP8HG_OK) return st;
    if (w->n > kMaxSide || w->k > kMaxSide) return FP8HG_ERR_SHAPE;
    if (w->r < 1 || w->adapters < 1) return FP8HG_ERR_INVALID_ARG;
    if (w->r > fp8hg::kLoraMaxRank) return FP8HG_ERR_UNSUPPORTED;
    if (!w->a || !w->b || w->ld_a < w->k || w->ld_b < w->r || w->stride_a < 0 || w->stride_b < 0) return FP8HG_ERR_INVALID_ARG;
    if (w->ld_a > kMaxLd || w->ld_b > kMaxLd) return FP8HG_ERR_SHAPE;
    if (!aligned(w->a, 2) || !aligned(w->b, 2) || !aligned(w->scale, 4) || !aligned(w->ranks, 4)) return FP8HG_ERR_ALIGNMENT;
    return FP8HG_OK;
}

fp8hg::LoraWeights weights(const fp8hg_lora *w) {
    return {w->a, w->b, w->stride_a, w->stride_b, u32(w->ld_a), u32(w->ld_b), w->scale, w->ranks,
            static_cast<int>(w->r), static_cast<int>(w->n), static_cast<int>(w->k)};
}

// Sizes for which the workspace functions have an answer.
bool lora_sizes(int64_t tokens, int64_t adapters, int64_t r, int64_t n, int64_t k) {
    return tokens > 0 && tokens <= kMaxTokens && adapters > 0 && adapters <= fp8hg::kLoraMaxAdapters && r > 0 &&
           r <= fp8hg::kLoraMaxRank && n > 0 && n <= kMaxSide && k > 0 && k <= kMaxSide;
}

}  // namespace

extern "C" {

int fp8hg_layernorm(const void *x, int x_kind, int64_t rows, int64_t cols, int64_t ld_x,
                    const void *weight, const void *bias, int param_kind, float eps, void *y,
                    int y_kind, int64_t ld_y, const fp8hg_norm_codes *q, float *stats,
                    void *stream) {
    if (!valid_kind(x_kind) || !valid_kind(param_kind) || !valid_kind(y_kind)) return FP8HG_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return FP8HG_ERR_INVALID_ARG;
    int st = check_dims(rows, cols);
    if (st != FP8HG_OK) return st;
    if (q && ((q->group != 0 && q->group != 128) || (q->fmt != FP8HG_E4M3 && q->fmt != FP8HG_E5M2))) return FP8HG_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return FP8HG_OK;
    if (!y && !q && !stats) return FP8HG_ERR_INVALID_ARG;
    st = check_matrix(x, cols, ld_x, size_of(x_kind));
    if (st == FP8HG_OK && y) st = check_matrix(y, cols, ld_y, size_of(y_kind));
    if (st == FP8HG_OK) st = check_vector(weight, size_of(param_kind));
    if (st == FP8HG_OK) st = check_vector(bias, size_of(param_kind));
    if (st == FP8HG_OK) st = check_vector(stats, 8);
    if (st != FP8HG_OK) return st;
    fp8hg::NormArgs a{};
    if (q) {
        const int64_t groups = q->group ? (cols + 127) / 128 : 1;
        if (!q->codes || !q->scale) return FP8HG_ERR_INVALID_ARG;
        if (!aligned(q->codes, 16) || q->ld % 16) return FP8HG_ERR_ALIGNMENT;
        if (q->ld < cols || q->ld_scale < groups) return FP8HG_ERR_INVALID_ARG;
        if (q->ld > kMaxLd || q->ld_scale > kMaxLd) return FP8HG_ERR_SHAPE;
        a.q = q->codes;
        a.s = q->scale;
        a.ld_q = u32(q->ld);
        a.ld_s = u32(q->ld_scale);
        a.group = q->group;
        a.fmt = q->fmt;
    }
    a.x = x;
    a.x_f32 = x_kind == FP8HG_OUT_FP32;
    a.rows = static_cast<int>(rows);
    a.cols = static_cast<int>(cols);
    a.ld_x = u32(ld_x);
    a.weight = weight;
    a.bias = bias;
    a.param_f32 = param_kind == FP8HG_OUT_FP32;
    a.eps = eps;
    a.y = y;
    a.y_f32 = y_kind == FP8HG_OUT_FP32;
    a.ld_y = u32(ld_y);
    a.stats = stats;
    return status_from_cuda(fp8hg::launch_norm(a, static_cast<cudaStream_t>(stream)));
}

size_t fp8hg_layernorm_bwd_workspace(int64_t rows, int64_t cols) {
    if (rows <= 0 || cols <= 0 || rows > kMaxDim || cols > kMaxDim) return 0;
    return fp8hg::norm_bwd_ws_bytes(rows, cols);
}

int fp8hg_layernorm_bwd(const void *dy, int dy_kind, int64_t ld_dy, const void *x, int x_kind,
                        int64_t ld_x, int64_t rows, int64_t cols, const void *weight,
                        int param_kind, const float *stats, const void *add, int64_t ld_add,
                        void *dx, int64_t ld_dx, float *dweight, float *dbias, void *workspace,
                        size_t workspace_bytes, void *stream) {
    if (!valid_kind(dy_kind) || !valid_kind(x_kind) || !valid_kind(param_kind)) return FP8HG_ERR_INVALID_ARG;
    int st = check_dims(rows, cols);
    if (st == FP8HG_OK) st = check_vector(dweight, 4);
    if (st == FP8HG_OK) st = check_vector(dbias, 4);
    if (st != FP8HG_OK) return st;
    if (cols == 0) return FP8HG_OK;
    if (rows == 0) {
        const auto s = static_cast<cudaStream_t>(stream);
        cudaError_t e = cudaSuccess;
        if (dweight) e = cudaMemsetAsync(dweight, 0, sizeof(float) * cols, s);
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, sizeof(float) * cols, s);
        if (e != cudaSuccess) cudaGetLastError();   // reported here, not by the next call that asks
        return status_from_cuda(e);
    }
    st = check_matrix(dy, cols, ld_dy, size_of(dy_kind));
    if (st == FP8HG_OK) st = check_matrix(x, cols, ld_x, size_of(x_kind));
    if (st == FP8HG_OK) st = check_matrix(dx, cols, ld_dx, size_of(x_kind));
    if (st == FP8HG_OK && add) st = check_matrix(add, cols, ld_add, size_of(x_kind));
    if (st == FP8HG_OK) st = check_vector(weight, size_of(param_kind));
    if (st != FP8HG_OK) return st;
    if (!stats) return FP8HG_ERR_INVALID_ARG;
    if (!aligned(stats, 8)) return FP8HG_ERR_ALIGNMENT;
    const bool sums = dweight || dbias;
    if (sums) {
        if (!workspace || workspace_bytes < fp8hg::norm_bwd_ws_bytes(rows, cols)) return FP8HG_ERR_INVALID_ARG;
        if (!aligned(workspace, 16)) return FP8HG_ERR_ALIGNMENT;
    }
    return status_from_cuda(fp8hg::launch_norm_bwd({dy, x, add, dy_kind == FP8HG_OUT_FP32, x_kind == FP8HG_OUT_FP32,
                                                    static_cast<int>(rows), static_cast<int>(cols), u32(ld_dy), u32(ld_x),
                                                    u32(ld_add), weight, param_kind == FP8HG_OUT_FP32, stats, dx, u32(ld_dx),
                                                    dweight, dbias, sums ? static_cast<float *>(workspace) : nullptr},
                                                   static_cast<cudaStream_t>(stream)));
}

size_t fp8hg_lora_plan_bytes(int64_t tokens, int64_t adapters) {
    if (tokens < 0 || tokens > kMaxTokens || adapters < 1 || adapters > fp8hg::kLoraMaxAdapters) return 0;
    return static_cast<size_t>(plan_of(nullptr, tokens, adapters).size()) * sizeof(int32_t);
}

int fp8hg_lora_plan(const int32_t *ids, int64_t tokens, int64_t adapters, void *plan,
                    size_t plan_bytes, void *stream) {
    const int st = check_plan(plan, tokens, adapters);
    if (st != FP8HG_OK) return st;
    if (tokens > 0 && !ids) return FP8HG_ERR_INVALID_ARG;
    if (!aligned(ids, 4)) return FP8HG_ERR_ALIGNMENT;
    if (plan_bytes < fp8hg_lora_plan_bytes(tokens, adapters)) return FP8HG_ERR_INVALID_ARG;
    return status_from_cuda(fp8hg::launch_lora_plan(ids, plan_of(plan, tokens, adapters), static_cast<int *>(plan),
                                                    static_cast<cudaStream_t>(stream)));
}

size_t fp8hg_lora_workspace(int64_t tokens, int64_t adapters, int64_t r, int64_t k) {
    if (!lora_sizes(tokens, adapters, r, 1, k)) return 0;
    return fp8hg::lora_ws_bytes(tokens, static_cast<int>(adapters), static_cast<int>(r), k);
}

int fp8hg_lora_add(const fp8hg_lora *w, const void *plan, int64_t tokens, const uint16_t *x,
                   int64_t ld_x, const void *base, int64_t ld_base, void *y, int64_t ld_y,
                   int y_kind, float *v, int64_t ld_v, void *workspace, size_t workspace_bytes,
                   void *stream) {
    if (!valid_kind(y_kind)) return FP8HG_ERR_INVALID_ARG;
    int st = check_lora(w);
    if (st == FP8HG_OK) st = check_plan(plan, tokens, w->adapters);
    if (st != FP8HG_OK) return st;
    if (w->k == 0 || w->n == 0) return FP8HG_ERR_SHAPE;
    if (tokens == 0) return FP8HG_OK;
    st = check_matrix(x, w->k, ld_x, 2);
    if (st == FP8HG_OK) st = check_matrix(y, w->n, ld_y, size_of(y_kind));
    if (st == FP8HG_OK && base) st = check_matrix(base, w->n, ld_base, size_of(y_kind));
    if (st == FP8HG_OK && v) st = check_matrix(v, w->r, ld_v, 4);
    if (st != FP8HG_OK) return st;
    if (!workspace || workspace_bytes < fp8hg_lora_workspace(tokens, w->adapters, w->r, w->k)) return FP8HG_ERR_INVALID_ARG;
    if (!aligned(workspace, 16)) return FP8HG_ERR_ALIGNMENT;
    return status_from_cuda(fp8hg::launch_lora_add({weights(w), plan_of(plan, tokens, w->adapters), x, u32(ld_x), base, y,
                                                    y_kind == FP8HG_OUT_FP32, u32(ld_base), u32(ld_y), v, u32(ld_v),
                                                    static_cast<float *>(workspace)},
                                                   static_cast<cudaStream_t>(stream)));
}

size_t fp8hg_lora_bwd_workspace(int64_t tokens, int64_t adapters, int64_t r, int64_t n, int64_t k) {
    if (!lora_sizes(tokens, adapters, r, n, k)) return 0;
    return fp8hg::lora_bwd_ws_bytes(tokens, static_cast<int>(adapters), static_cast<int>(r), n, k);
}

int fp8hg_lora_add_bwd(const fp8hg_lora *w, const void *plan, int64_t tokens, const uint16_t *dy,
                       int64_t ld_dy, const uint16_t *x, int64_t ld_x, const float *v,
                       int64_t ld_v, const void *base, int64_t ld_base, void *dx, int64_t ld_dx,
                       int dx_kind, void *da, void *db, int dw_kind, void *workspace,
                       size_t workspace_bytes, void *stream) {
    if (!valid_kind(dx_kind) || !valid_kind(dw_kind)) return FP8HG_ERR_INVALID_ARG;
    int st = check_lora(w);
    if (st == FP8HG_OK) st = check_plan(plan, tokens, w->adapters);
    if (st == FP8HG_OK) st = check_vector(da, size_of(dw_kind));
    if (st == FP8HG_OK) st = check_vector(db, size_of(dw_kind));
    if (st != FP8HG_OK) return st;
    if (w->k == 0 || w->n == 0) return FP8HG_ERR_SHAPE;
    const size_t each = static_cast<size_t>(w->adapters) * w->r * size_of(dw_kind);
    if (tokens == 0) {
        const auto s = static_cast<cudaStream_t>(stream);
        cudaError_t e = cudaSuccess;
        if (da) e = cudaMemsetAsync(da, 0, each * w->k, s);
        if (e == cudaSuccess && db) e = cudaMemsetAsync(db, 0, each * w->n, s);
        if (e != cudaSuccess) cudaGetLastError();   // reported here, not by the next call that asks
        return status_from_cuda(e);
    }
    if (!dx && !da && !db) return FP8HG_OK;
    st = check_matrix(dy, w->n, ld_dy, 2);
    if (st == FP8HG_OK && da) st = check_matrix(x, w->k, ld_x, 2);
    if (st == FP8HG_OK && db) st = check_matrix(v, w->r, ld_v, 4);
    if (st == FP8HG_OK && dx) st = check_matrix(dx, w->k, ld_dx, size_of(dx_kind));
    if (st == FP8HG_OK && dx && base) st = check_matrix(base, w->k, ld_base, size_of(dx_kind));
    if (st != FP8HG_OK) return st;
    if (!workspace || workspace_bytes < fp8hg_lora_bwd_workspace(tokens, w->adapters, w->r, w->n, w->k)) return FP8HG_ERR_INVALID_ARG;
    if (!aligned(workspace, 16)) return FP8HG_ERR_ALIGNMENT;
    return status_from_cuda(fp8hg::launch_lora_add_bwd({weights(w), plan_of(plan, tokens, w->adapters), dy, x, u32(ld_dy), u32(ld_x),
                                                        v, u32(ld_v), base, dx, dx_kind == FP8HG_OUT_FP32, u32(ld_base),
                                                        u32(ld_dx), da, db, dw_kind == FP8HG_OUT_FP32,
                                                        static_cast<float *>(workspace)},
                                                       static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
