// C-ABI entry points of the 4-bit operators and of the SwiGLU with 8-bit
// checkpoints (declared in include/fp8hg_lowbit.h): argument validation, then
// the launches.  Nothing here allocates device memory or synchronizes.
#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

#include "../../include/fp8hg_lowbit.h"
#include "lowbit.h"

namespace {

inline bool aligned(const void *p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}
inline int status_from_cuda(cudaError_t e) { return e == cudaSuccess ? FP8HG_OK : FP8HG_ERR_CUDA; }
inline bool valid_fmt(int f) { return f == FP8HG_E4M3 || f == FP8HG_E5M2; }
inline bool valid_kind(int k) { return k == FP4HG_MX || k == FP4HG_NV; }

constexpr uint64_t kDefaultWaitNs = 2000000000ull;   // 2 s
// What 32-bit indices of rows, columns and tiles hold with room to spare.
constexpr int64_t kMaxDim = int64_t(1) << 30;
// Row strides (elements or bytes) of what the element-wise kernels touch.
constexpr int64_t kMaxLd = 0x7FFFFFFF;
// Rows of the quantizer along the columns: its tiles of 128, in pairs (the scales'
// padding to 256), are a grid's second dimension.
constexpr int64_t kMaxTileRows = fp8hg::kGridY / 2 * int64_t(256);

// A 4-bit operand of a call that reads it.
int check_operand(const fp4hg_operand *o) {
    if (!o || !valid_kind(o->kind) || o->reserved != 0) return FP8HG_ERR_INVALID_ARG;
    if (o->rows < 0 || o->k < 0) return FP8HG_ERR_INVALID_ARG;
    if (o->rows > kMaxDim || o->k > kMaxDim) return FP8HG_ERR_SHAPE;
    if (o->rows == 0 || o->k == 0) return FP8HG_OK;
    if (!o->codes || !o->scale) return FP8HG_ERR_INVALID_ARG;
    if (!aligned(o->codes, 16) || !aligned(o->scale, 16) || o->ld % 16) return FP8HG_ERR_ALIGNMENT;
    if (o->ld < (o->k + 1) / 2) return FP8HG_ERR_INVALID_ARG;
    if (o->tensor_scale && (o->kind == FP4HG_MX)) return FP8HG_ERR_INVALID_ARG;
    if (o->tensor_scale && !aligned(o->tensor_scale, 4)) return FP8HG_ERR_ALIGNMENT;
    return FP8HG_OK;
}

fp8hg::Fp4Operand operand(const fp4hg_operand *o) {
    return {o->codes, o->scale, o->tensor_scale, o->rows, o->k, o->ld, o->kind};
}

int check_output(const void *c, int64_t ldc, int64_t cols, int out) {
    if (!c || ldc < cols) return FP8HG_ERR_INVALID_ARG;
    return aligned(c, out == FP8HG_OUT_BF16 ? 2 : 4) ? FP8HG_OK : FP8HG_ERR_ALIGNMENT;
}

int check_opts(const fp8hg_gemm_opts *opts, int max_inject) {
    if (!opts) return FP8HG_OK;
    if (opts->inject_fault < 0 || opts->inject_fault > max_inject) return FP8HG_ERR_INVALID_ARG;
    return opts->tile == 0 ? FP8HG_OK : FP8HG_ERR_UNSUPPORTED;
}

int run_gemm(fp8hg::Fp4GemmArgs &g, const fp8hg_gemm_opts *opts, void *stream) {
    unsigned int *err = fp8hg::error_word();
    if (!err) return FP8HG_ERR_CUDA;
    g.wait_limit_ns = opts && opts->wait_limit_ns ? opts->wait_limit_ns : kDefaultWaitNs;
    g.inject_fault = opts ? opts->inject_fault : 0;
    g.err = err;
    const int rc = fp8hg::launch_fp4_gemm(g, static_cast<cudaStream_t>(stream));
    if (rc == 1) return FP8HG_ERR_UNSUPPORTED;
    return rc == 0 ? FP8HG_OK : FP8HG_ERR_CUDA;
}

// A [rows, cols] BF16 input.
int check_input(const uint16_t *x, int64_t rows, int64_t cols, int64_t ld_x) {
    if (rows < 0 || cols < 0) return FP8HG_ERR_INVALID_ARG;
    if (rows > kMaxDim || cols > kMaxDim) return FP8HG_ERR_SHAPE;
    if (rows == 0 || cols == 0) return FP8HG_OK;
    if (!x || ld_x < cols) return FP8HG_ERR_INVALID_ARG;
    if (ld_x > kMaxLd) return FP8HG_ERR_SHAPE;
    return aligned(x, 2) ? FP8HG_OK : FP8HG_ERR_ALIGNMENT;
}

// Codes and scale bytes that are written: both or neither.
int check_codes(const uint8_t *q, int64_t ld, int64_t bytes, const uint8_t *s) {
    if (!q && !s) return FP8HG_OK;
    if (!q || !s) return FP8HG_ERR_INVALID_ARG;
    if (!aligned(q, 16) || ld % 16 || !aligned(s, 16)) return FP8HG_ERR_ALIGNMENT;
    if (ld > kMaxLd) return FP8HG_ERR_SHAPE;
    return ld >= bytes ? FP8HG_OK : FP8HG_ERR_INVALID_ARG;
}

int64_t codes_ld(int64_t k) { return (k + 31) / 32 * 16; }
uint32_t u32(int64_t v) { return static_cast<uint32_t>(v); }   // a checked stride

int check_ckpt(const fp8hg_swiglu_ckpt *c) {
    if (!c || !valid_fmt(c->fmt) || c->reserved != 0) return FP8HG_ERR_INVALID_ARG;
    if (c->rows < 0 || c->cols < 0) return FP8HG_ERR_INVALID_ARG;
    if (c->rows > kMaxDim || c->cols > kMaxDim) return FP8HG_ERR_SHAPE;
    if (c->rows == 0 || c->cols == 0) return FP8HG_OK;
    if (!c->gate_q || !c->gate_s || !c->up_q || !c->up_s) return FP8HG_ERR_INVALID_ARG;
    if (!aligned(c->gate_q, 16) || !aligned(c->up_q, 16) || c->ld_q % 16) return FP8HG_ERR_ALIGNMENT;
    if (c->ld_q < c->cols || c->ld_s < (c->cols + 127) / 128) return FP8HG_ERR_INVALID_ARG;
    if (c->ld_q > kMaxLd || c->ld_s > kMaxLd) return FP8HG_ERR_SHAPE;
    return FP8HG_OK;
}

fp8hg::SwigluCkpt ckpt(const fp8hg_swiglu_ckpt *c) {
    return {c->gate_q, c->gate_s, c->up_q, c->up_s, static_cast<int>(c->rows), static_cast<int>(c->cols),
            u32(c->ld_q), u32(c->ld_s), c->fmt};
}

}  // namespace

unsigned int *fp8hg::error_word() {
    static std::atomic<unsigned int *> words[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return fp8hg::device_error_word();
    unsigned int *w = words[dev].load(std::memory_order_relaxed);
    if (!w) words[dev].store(w = fp8hg::device_error_word(), std::memory_order_relaxed);
    return w;
}

int fp8hg::sm_count() {
    static std::atomic<int> counts[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
    n = counts[dev].load(std::memory_order_relaxed);
    if (!n) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 1;
        counts[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

extern "C" {

size_t fp4_scale_bytes(int64_t rows, int64_t k, int kind) {
    if (rows <= 0 || k <= 0 || !valid_kind(kind)) return 0;
    return static_cast<size_t>(fp8hg::fp4_row_tiles(rows) * fp8hg::fp4_scale_tiles(k, kind) * 512);
}

size_t fp4_tensor_scale_workspace(void) { return fp8hg::fp4_tensor_scale_ws_bytes(); }

int fp4_tensor_scale(const uint16_t *x, int64_t rows, int64_t cols, int64_t ld_x, float *scale,
                     void *workspace, size_t workspace_bytes, void *stream) {
    const int st = check_input(x, rows, cols, ld_x);
    if (st != FP8HG_OK) return st;
    if (!scale || !workspace) return FP8HG_ERR_INVALID_ARG;
    if (!aligned(scale, 4) || !aligned(workspace, 16)) return FP8HG_ERR_ALIGNMENT;
    if (workspace_bytes < fp8hg::fp4_tensor_scale_ws_bytes()) return FP8HG_ERR_INVALID_ARG;
    return status_from_cuda(fp8hg::launch_fp4_tensor_scale(x, static_cast<int>(rows), static_cast<int>(cols),
                                                           u32(ld_x), scale, workspace,
                                                           static_cast<cudaStream_t>(stream)));
}

int fp4_quant(const uint16_t *x, int64_t rows, int64_t cols, int64_t ld_x, int kind,
              const float *tensor_scale, uint8_t *q, int64_t ld_q, uint8_t *scale, uint8_t *q_t,
              int64_t ld_qt, uint8_t *scale_t, void *stream) {
    if (!valid_kind(kind)) return FP8HG_ERR_INVALID_ARG;
    int st = check_input(x, rows, cols, ld_x);
    if (st != FP8HG_OK) return st;
    if (tensor_scale && kind == FP4HG_MX) return FP8HG_ERR_INVALID_ARG;
    if (tensor_scale && !aligned(tensor_scale, 4)) return FP8HG_ERR_ALIGNMENT;
    if (rows == 0 || cols == 0) return FP8HG_OK;
    if (!q && !q_t) return FP8HG_ERR_INVALID_ARG;
    st = check_codes(q, ld_q, (cols + 1) / 2, scale);
    if (st != FP8HG_OK) return st;
    st = check_codes(q_t, ld_qt, (rows + 1) / 2, scale_t);
    if (st != FP8HG_OK) return st;
    if (q_t && rows > kMaxTileRows) return FP8HG_ERR_SHAPE;
    return status_from_cuda(fp8hg::launch_fp4_quant({x, static_cast<int>(rows), static_cast<int>(cols), u32(ld_x),
                                                     kind, tensor_scale, q, u32(ld_q), scale, q_t, u32(ld_qt),
                                                     scale_t},
                                                    static_cast<cudaStream_t>(stream)));
}

int fp4_dequant(const fp4hg_operand *a, void *out, int64_t ld_out, int out_kind, void *stream) {
    if (out_kind != FP8HG_OUT_BF16 && out_kind != FP8HG_OUT_FP32) return FP8HG_ERR_INVALID_ARG;
    int st = check_operand(a);
    if (st != FP8HG_OK) return st;
    if (a->rows == 0 || a->k == 0) return FP8HG_OK;
    st = check_output(out, ld_out, a->k, out_kind);
    if (st != FP8HG_OK) return st;
    if (ld_out > kMaxLd || a->ld > kMaxLd) return FP8HG_ERR_SHAPE;
    return status_from_cuda(fp8hg::launch_fp4_dequant(operand(a), out, u32(ld_out),
                                                      out_kind == FP8HG_OUT_FP32,
                                                      static_cast<cudaStream_t>(stream)));
}

int fp4_gemm_scaled(const fp4hg_operand *a, const fp4hg_operand *b, void *c, int64_t ldc, int out,
                    int accumulate, const fp8hg_gemm_opts *opts, void *stream) {
    if (out != FP8HG_OUT_BF16 && out != FP8HG_OUT_FP32) return FP8HG_ERR_INVALID_ARG;
    if (accumulate != 0 && accumulate != 1) return FP8HG_ERR_INVALID_ARG;
    int st = check_operand(a);
    if (st != FP8HG_OK) return st;
    st = check_operand(b);
    if (st != FP8HG_OK) return st;
    if (a->kind != b->kind) return FP8HG_ERR_UNSUPPORTED;
    if (a->k != b->k || a->k == 0) return FP8HG_ERR_SHAPE;
    st = check_opts(opts, a->kind == FP4HG_NV ? 2 : 1);
    if (st != FP8HG_OK) return st;
    if (a->rows == 0 || b->rows == 0) return FP8HG_OK;
    st = check_output(c, ldc, b->rows, out);
    if (st != FP8HG_OK) return st;
    fp8hg::Fp4GemmArgs g{};
    g.a = operand(a);
    g.b = operand(b);
    g.c = c;
    g.ldc = ldc;
    g.out_fp32 = out == FP8HG_OUT_FP32;
    g.accumulate = accumulate;
    return run_gemm(g, opts, stream);
}

size_t fp4_linear_workspace(int64_t rows, int64_t k, int kind) {
    if (rows <= 0 || k <= 0 || !valid_kind(kind) || fp8hg::fp4_linear_quantizes(rows)) return 0;
    return static_cast<size_t>(rows * codes_ld(k)) + fp4_scale_bytes(rows, k, kind);
}

int fp4_linear(const uint16_t *x, int64_t rows, int64_t ld_x, const float *tensor_scale,
               const fp4hg_operand *w, void *y, int64_t ld_y, int out, void *workspace,
               size_t workspace_bytes, const fp8hg_gemm_opts *opts, void *stream) {
    if (out != FP8HG_OUT_BF16 && out != FP8HG_OUT_FP32) return FP8HG_ERR_INVALID_ARG;
    int st = check_operand(w);
    if (st != FP8HG_OK) return st;
    if (w->k == 0) return FP8HG_ERR_SHAPE;
    st = check_input(x, rows, w->k, ld_x);
    if (st != FP8HG_OK) return st;
    if (tensor_scale && w->kind == FP4HG_MX) return FP8HG_ERR_INVALID_ARG;
    if (tensor_scale && !aligned(tensor_scale, 4)) return FP8HG_ERR_ALIGNMENT;
    st = check_opts(opts, 1);
    if (st != FP8HG_OK) return st;
    if (rows == 0 || w->rows == 0) return FP8HG_OK;
    st = check_output(y, ld_y, w->rows, out);
    if (st != FP8HG_OK) return st;
    fp8hg::Fp4GemmArgs g{};
    g.a = {nullptr, nullptr, tensor_scale, rows, w->k, 0, w->kind};
    g.b = operand(w);
    g.c = y;
    g.ldc = ld_y;
    g.out_fp32 = out == FP8HG_OUT_FP32;
    if (fp8hg::fp4_linear_quantizes(rows)) {
        g.x = x;
        g.ld_x = ld_x;
        return run_gemm(g, opts, stream);
    }
    if (!workspace || workspace_bytes < fp4_linear_workspace(rows, w->k, w->kind))
        return FP8HG_ERR_INVALID_ARG;
    if (!aligned(workspace, 16)) return FP8HG_ERR_ALIGNMENT;
    uint8_t *codes = static_cast<uint8_t *>(workspace);
    g.a.codes = codes;
    g.a.ld = codes_ld(w->k);
    uint8_t *scale = codes + rows * g.a.ld;
    g.a.scale = scale;
    const cudaError_t e = fp8hg::launch_fp4_quant(
        {x, static_cast<int>(rows), static_cast<int>(w->k), u32(ld_x), w->kind, tensor_scale, codes, u32(g.a.ld),
         scale, nullptr, 0, nullptr},
        static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return FP8HG_ERR_CUDA;
    return run_gemm(g, opts, stream);
}

int fp8_swiglu_ckpt(const uint16_t *gate, const uint16_t *up, int64_t rows, int64_t cols,
                    int64_t ld_in, int fmt_h, uint8_t *h, int64_t ld_h, uint8_t *h_scale,
                    int64_t ld_hs, int fmt, uint8_t *gate_q, uint8_t *gate_s, uint8_t *up_q,
                    uint8_t *up_s, int64_t ld_q, int64_t ld_s, void *stream) {
    const bool keep = gate_q || gate_s || up_q || up_s;
    if (!valid_fmt(fmt_h) || (keep && !valid_fmt(fmt))) return FP8HG_ERR_INVALID_ARG;
    int st = check_input(gate, rows, cols, ld_in);
    if (st != FP8HG_OK) return st;
    st = check_input(up, rows, cols, ld_in);
    if (st != FP8HG_OK) return st;
    if (rows == 0 || cols == 0) return FP8HG_OK;
    if (!h || !h_scale) return FP8HG_ERR_INVALID_ARG;
    if (!aligned(h, 16) || ld_h % 16) return FP8HG_ERR_ALIGNMENT;
    const int64_t groups = (cols + 127) / 128;
    if (ld_h < cols || ld_hs < groups) return FP8HG_ERR_INVALID_ARG;
    if (ld_h > kMaxLd || ld_hs > kMaxLd) return FP8HG_ERR_SHAPE;
    if (keep) {
        if (!gate_q || !gate_s || !up_q || !up_s) return FP8HG_ERR_INVALID_ARG;
        if (!aligned(gate_q, 16) || !aligned(up_q, 16) || ld_q % 16) return FP8HG_ERR_ALIGNMENT;
        if (ld_q < cols || ld_s < groups) return FP8HG_ERR_INVALID_ARG;
        if (ld_q > kMaxLd || ld_s > kMaxLd) return FP8HG_ERR_SHAPE;
    }
    return status_from_cuda(fp8hg::launch_swiglu_fwd({gate, up, static_cast<int>(rows), static_cast<int>(cols),
                                                      u32(ld_in), fmt_h, fmt, h, h_scale, u32(ld_h), u32(ld_hs),
                                                      gate_q, gate_s, up_q, up_s, u32(ld_q), u32(ld_s)},
                                                     static_cast<cudaStream_t>(stream)));
}

int fp8_swiglu_ckpt_bwd(const uint16_t *dh, int64_t ld_dh, const fp8hg_swiglu_ckpt *c,
                        uint16_t *dgate, uint16_t *dup, int64_t ld_d, void *stream) {
    int st = check_ckpt(c);
    if (st != FP8HG_OK) return st;
    st = check_input(dh, c->rows, c->cols, ld_dh);
    if (st != FP8HG_OK) return st;
    if (c->rows == 0 || c->cols == 0) return FP8HG_OK;
    st = check_output(dgate, ld_d, c->cols, FP8HG_OUT_BF16);
    if (st != FP8HG_OK) return st;
    st = check_output(dup, ld_d, c->cols, FP8HG_OUT_BF16);
    if (st != FP8HG_OK) return st;
    if (ld_d > kMaxLd) return FP8HG_ERR_SHAPE;
    return status_from_cuda(fp8hg::launch_swiglu_bwd(dh, u32(ld_dh), ckpt(c), dgate, dup, u32(ld_d),
                                                     static_cast<cudaStream_t>(stream)));
}

int fp8_swiglu_ckpt_bwd_q(const uint16_t *dh, int64_t ld_dh, const fp8hg_swiglu_ckpt *c,
                          const fp8hg_swiglu_grads *g, void *stream) {
    int st = check_ckpt(c);
    if (st != FP8HG_OK) return st;
    if (!g || !valid_fmt(g->fmt) || !valid_fmt(g->fmt_t) || !valid_fmt(g->fmt_h) || g->reserved != 0)
        return FP8HG_ERR_INVALID_ARG;
    st = check_input(dh, c->rows, c->cols, ld_dh);
    if (st != FP8HG_OK) return st;
    if (c->rows == 0 || c->cols == 0) return FP8HG_OK;
    if (c->rows % 128 || c->cols % 128) return FP8HG_ERR_SHAPE;
    if (!aligned(dh, 16) || ld_dh % 8) return FP8HG_ERR_ALIGNMENT;
    fp8hg::SwigluGrads o{{g->dgate_q, g->dup_q}, {g->dgate_s, g->dup_s},
                         {g->dgate_qt, g->dup_qt, g->h_qt}, {g->dgate_st, g->dup_st, g->h_st},
                         u32(g->ld_q), u32(g->ld_s), u32(g->ld_qt), u32(g->ld_st), g->fmt, g->fmt_t, g->fmt_h,
                         nullptr};
    for (int i = 0; i < 3; ++i) {
        if ((i < 2 && (!o.q[i] || !o.s[i])) || !o.qt[i] || !o.st[i]) return FP8HG_ERR_INVALID_ARG;
        if ((i < 2 && !aligned(o.q[i], 16)) || !aligned(o.qt[i], 16)) return FP8HG_ERR_ALIGNMENT;
    }
    if (g->ld_q % 16 || g->ld_qt % 16) return FP8HG_ERR_ALIGNMENT;
    if (g->ld_q < c->cols || g->ld_s < c->cols / 128 || g->ld_qt < c->rows || g->ld_st < c->rows / 128)
        return FP8HG_ERR_INVALID_ARG;
    if (g->ld_q > kMaxLd || g->ld_s > kMaxLd || g->ld_qt > kMaxLd || g->ld_st > kMaxLd) return FP8HG_ERR_SHAPE;
    o.err = fp8hg::error_word();
    if (!o.err) return FP8HG_ERR_CUDA;
    return status_from_cuda(fp8hg::launch_swiglu_bwd_q(dh, u32(ld_dh), ckpt(c), o,
                                                       static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
