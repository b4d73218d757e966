/*
 * fp8hg_lowbit — 4-bit microscaled quantization and products, and SwiGLU with
 * 8-bit activation checkpoints, for GB300 (sm_103a).  Same library
 * (libfp8hg.so) and same conventions as fp8hg.h: device pointers, BF16 as
 * uint16_t bit patterns with row strides in elements, codes and scale bytes
 * with row strides in bytes, a caller-owned stream, no allocation and no
 * synchronization, fp8hg_status return values, argument errors before any
 * launch.  Rows and columns are at most 2^30, row strides below 2^31
 * (FP8HG_ERR_SHAPE beyond).
 *
 * 4-bit values are E2M1 (sign, two exponent bits, one mantissa bit):
 * 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives, rounded to nearest even and
 * saturating at 6.  Two codes share a byte, the element with the even index
 * in the low four bits.  Two kinds of block scales:
 *
 *   FP4HG_MX  32 elements share 2^(b - 127), with b the scale byte and
 *             b - 127 = floor(log2 amax) - 2, clamped to [-127, 127]
 *             (amax = 0: b = 0) — the rule of fp8_quant_mx32
 *   FP4HG_NV  16 elements share an E4M3 scale s, and the whole tensor one
 *             FP32 scale t: s = E4M3((amax / 6) / t), nearest even, at most
 *             448; the element's code is E2M1(x / (s t)), 0 where x = -0, a
 *             zero of x's sign where s = 0
 *
 * An element stands for code * 2^(b - 127), or code * s * t.  A block that
 * holds a NaN or an infinity gets the scale byte 0xFF (MX) or 0x7F (NV), a
 * NaN in both encodings, and codes 0: every value of it is NaN.
 *
 * Scale bytes are stored in the order the tensor cores take them: tiles of
 * 128 rows by 4 blocks, 512 bytes each, all tiles of 128 rows one after
 * another; the byte of row r and block j lies at
 *
 *   ((r / 128) * tiles + j / 4) * 512 + (r % 32) * 16 + (r % 128) / 32 * 4 + j % 4
 *
 * with `tiles` = 2 * ceil(k / 256) for MX and 4 * ceil(k / 256) for NV, that
 * is, k padded to a multiple of 256.  The quantizer writes the padding along
 * k (as zeros); the bytes of rows past the last are not used.
 */
#ifndef FP8HG_LOWBIT_H
#define FP8HG_LOWBIT_H

#include <stddef.h>
#include <stdint.h>

#include "fp8hg.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { FP4HG_MX = 0, FP4HG_NV = 1 } fp4hg_kind;

/* Bytes of the scale array of a [rows, k] tensor (0 for an empty tensor or an
 * unknown kind). */
size_t fp4_scale_bytes(int64_t rows, int64_t k, int kind);

/*
 * fp4_tensor_scale — the FP32 scale of a tensor for FP4HG_NV: the smallest
 * power of two t with amax <= 6 * 448 * t, so that no block's scale saturates;
 * 1 for a tensor of zeros.  NaNs and infinities are left out of amax (their
 * blocks are marked by the quantizer); t is at least 2^-100 and, as amax is
 * below 2^128, at most 2^117.
 *
 *   x          [rows, cols] BF16, row stride ld_x elements, 2-byte aligned
 *   scale      device pointer, one float
 *   workspace  fp4_tensor_scale_workspace() bytes of device memory, 16-byte
 *              aligned, owned by the caller; need not be cleared
 */
size_t fp4_tensor_scale_workspace(void);
int fp4_tensor_scale(const uint16_t *x, int64_t rows, int64_t cols, int64_t ld_x, float *scale,
                     void *workspace, size_t workspace_bytes, void *stream);

/*
 * fp4_quant — BF16 to 4 bits, along the rows of x, along its columns
 * (written transposed, for the operand whose product runs over the tokens),
 * or both from one read.
 *
 *   x             [rows, cols] BF16, row stride ld_x elements; any rows and
 *                 cols, 2-byte aligned (32-byte loads where x is 32-byte
 *                 aligned and ld_x a multiple of 16, shifted 16-byte pieces
 *                 elsewhere)
 *   tensor_scale  FP4HG_NV: device pointer to t, or NULL for 1; a positive
 *                 number between 2^-100 and 2^117 (what fp4_tensor_scale
 *                 gives).  FP4HG_MX: NULL
 *   q, scale      codes [rows, ceil(cols / 2)] (ld_q bytes, a multiple of 16,
 *                 16-byte aligned) and scale bytes of the [rows, cols] tensor,
 *                 or both NULL
 *   q_t, scale_t  codes [cols, ceil(rows / 2)] (ld_qt) and scale bytes of the
 *                 [cols, rows] tensor, or both NULL; rows at most 32767 * 256
 * Blocks run from the first column (row); the last one may be shorter.  The
 * unused half of a last byte is 0.  Scale arrays are 16-byte aligned.
 */
int fp4_quant(const uint16_t *x, int64_t rows, int64_t cols, int64_t ld_x, int kind,
              const float *tensor_scale, uint8_t *q, int64_t ld_q, uint8_t *scale, uint8_t *q_t,
              int64_t ld_qt, uint8_t *scale_t, void *stream);

/*
 * A 4-bit tensor of `rows` rows of `k` elements: codes 16-byte aligned, row
 * stride ld bytes (a multiple of 16, at least ceil(k / 2)); scale 16-byte
 * aligned, fp4_scale_bytes(rows, k, kind) bytes; tensor_scale as fp4_quant.
 * As fp4_quant leaves them: the unused half of a row's last byte (k odd) is 0,
 * and no scale byte of the padding along k is a NaN.
 */
typedef struct {
    const uint8_t *codes;
    const uint8_t *scale;
    const float *tensor_scale;
    int64_t rows, k, ld;
    int32_t kind, reserved;
} fp4hg_operand;

/* fp4_dequant — the values of a 4-bit tensor, [rows, k], as BF16 or FP32
 * (fp8hg_out), row stride ld_out elements. */
int fp4_dequant(const fp4hg_operand *a, void *out, int64_t ld_out, int out_kind, void *stream);

/*
 * fp4_gemm_scaled — C = A B^T, or C += A B^T, on 4-bit operands of the same
 * kind, FP32 accumulation, BF16 or FP32 output.  The forward product takes
 * X and W as they are, the data gradient dY and the transposed W, the weight
 * gradient the transposed dY and X.
 *
 *   a, b        operands, a->k = b->k > 0; any numbers of rows (0: nothing is
 *               written)
 *   c           [a->rows, b->rows], row stride ldc elements, aligned to its
 *               element size
 *   opts        NULL or fp8hg_gemm_opts (tile must be 0): bounded waits as in
 *               fp8_gemm_scaled_ex; tiles of C that a wait has run out for are
 *               not written.  inject_fault = 1: the first CTA never issues its
 *               first copy; 2 (FP4HG_NV): half of the scales of one stage of K
 *               never come, late in the first CTAs' work (FP8HG_ERR_UNSUPPORTED
 *               for shapes whose kernel has no such halves)
 * The tensors' scales meet the FP32 sums one after the other where their product
 * is no normal FP32 number: C overflows or vanishes only where its value does.
 */
int fp4_gemm_scaled(const fp4hg_operand *a, const fp4hg_operand *b, void *c, int64_t ldc, int out,
                    int accumulate, const fp8hg_gemm_opts *opts, void *stream);

/*
 * fp4_linear — y = x w^T with x quantized on the way: the result of fp4_quant
 * of x followed by fp4_gemm_scaled, in one call.  Up to 4 rows (decoding) x
 * is quantized inside the product.
 *
 *   x, ld_x        [rows, w->k] BF16, as fp4_quant
 *   tensor_scale   x's, as fp4_quant
 *   w              the weights, [n, k]
 *   y              [rows, n], row stride ld_y elements
 *   workspace      fp4_linear_workspace(rows, w->k, w->kind) bytes of device
 *                  memory (none up to 4 rows), 16-byte aligned, owned by the
 *                  caller; need not be cleared.  Calls that may overlap on the
 *                  GPU need separate ones.
 */
size_t fp4_linear_workspace(int64_t rows, int64_t k, int kind);
int fp4_linear(const uint16_t *x, int64_t rows, int64_t ld_x, const float *tensor_scale,
               const fp4hg_operand *w, void *y, int64_t ld_y, int out, void *workspace,
               size_t workspace_bytes, const fp8hg_gemm_opts *opts, void *stream);

/*
 * fp8_swiglu_ckpt — h = silu(gate) * up, silu(g) = g / (1 + exp(-g)), in FP32,
 * quantized in groups of 128 columns (UE8M0 scales rounded up, as
 * fp8_quant_token with group 128), and gate and up themselves quantized the
 * same way for the backward pass: 2 bytes per element are kept instead of 4.
 *
 *   gate, up      [rows, cols] BF16, both with row stride ld_in elements (the
 *                 two halves of one product's output, for example)
 *   fmt_h, h      codes [rows, cols] (ld_h bytes), h_scale [rows, G] (ld_hs),
 *                 G = ceil(cols / 128); the last group may be shorter
 *   fmt, gate_q, gate_s, up_q, up_s
 *                 the checkpoint: codes [rows, cols] (ld_q bytes) and scales
 *                 [rows, G] (ld_s), or all four NULL (inference)
 * Any rows and cols; h, gate_q and up_q 16-byte aligned with strides that are
 * multiples of 16; gate and up 2-byte aligned (32-byte loads where they are
 * 32-byte aligned and ld_in a multiple of 16, shifted 16-byte pieces elsewhere).
 * 1 / (1 + exp(-g)) below 2^-126 counts as 0, here and in the backward calls.
 */
int fp8_swiglu_ckpt(const uint16_t *gate, const uint16_t *up, int64_t rows, int64_t cols,
                    int64_t ld_in, int fmt_h, uint8_t *h, int64_t ld_h, uint8_t *h_scale,
                    int64_t ld_hs, int fmt, uint8_t *gate_q, uint8_t *gate_s, uint8_t *up_q,
                    uint8_t *up_s, int64_t ld_q, int64_t ld_s, void *stream);

/* A checkpoint of fp8_swiglu_ckpt as the backward calls take it. */
typedef struct {
    const uint8_t *gate_q, *gate_s, *up_q, *up_s;
    int64_t rows, cols, ld_q, ld_s;
    int32_t fmt, reserved;
} fp8hg_swiglu_ckpt;

/*
 * fp8_swiglu_ckpt_bwd — gradients of gate and up from dh and the checkpoint's
 * values g, u, with s = 1 / (1 + exp(-g)):
 *   dgate = dh * u * s * (1 + g * (1 - s)),   dup = dh * g * s
 * in FP32, rounded to BF16.
 *
 *   dh           [rows, cols] BF16 (ld_dh elements)
 *   dgate, dup   [rows, cols] BF16, both with row stride ld_d elements
 */
int fp8_swiglu_ckpt_bwd(const uint16_t *dh, int64_t ld_dh, const fp8hg_swiglu_ckpt *ckpt,
                        uint16_t *dgate, uint16_t *dup, int64_t ld_d, void *stream);

/*
 * fp8_swiglu_ckpt_bwd_q — the same gradients as the operands of the next FP8
 * products, each quantized from FP32: per 1x128 group of a row (data
 * gradient), and per 128 tokens of a column, transposed (weight gradient);
 * and h = g * s * u rebuilt from the checkpoint, per 128 tokens, transposed
 * (the down projection's weight gradient).
 *
 *   fmt, dgate_q, dup_q, dgate_s, dup_s   codes [rows, cols] (ld_q bytes),
 *                                         scales [rows, cols/128] (ld_s)
 *   fmt_t, dgate_qt, ...                  codes [cols, rows] (ld_qt), scales
 *                                         [cols, rows/128] (ld_st)
 *   fmt_h, h_qt, h_st                     the same layout and strides for h
 * Requirements: rows and cols multiples of 128, dh 16-byte aligned with ld_dh
 * % 8 == 0, codes 16-byte aligned with strides that are multiples of 16.  The
 * kernel's warps hand data to one another over waits of at most 2 s; one that ran
 * out would be FP8HG_ERR_TIMEOUT from fp8hg_get_device_error.
 */
typedef struct {
    uint8_t *dgate_q, *dup_q, *dgate_s, *dup_s;
    uint8_t *dgate_qt, *dup_qt, *dgate_st, *dup_st;
    uint8_t *h_qt, *h_st;
    int64_t ld_q, ld_s, ld_qt, ld_st;
    int32_t fmt, fmt_t, fmt_h, reserved;
} fp8hg_swiglu_grads;

int fp8_swiglu_ckpt_bwd_q(const uint16_t *dh, int64_t ld_dh, const fp8hg_swiglu_ckpt *ckpt,
                          const fp8hg_swiglu_grads *grads, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8HG_LOWBIT_H */
