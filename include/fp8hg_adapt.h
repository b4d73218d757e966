/*
 * fp8hg_adapt — what stands before a quantized projection and what is trained
 * beside a frozen one, for GB300 (sm_103a): layer norm and low-rank adapters,
 * forward and backward.  Same library (libfp8hg.so) and same conventions as
 * fp8hg.h: device pointers, BF16 as uint16_t bit patterns, row strides in
 * elements (FP8 codes and scale bytes: in bytes), a caller-owned stream, no
 * allocation and no synchronization, fp8hg_status return values, argument errors
 * before any launch.  A `kind` is FP8HG_OUT_BF16 or FP8HG_OUT_FP32.  Sizes are at
 * most 2^30, row strides below 2^31 (FP8HG_ERR_SHAPE beyond).  Pointers are
 * aligned to their element size; rows that begin at multiples of 16 or 32 bytes
 * are read and written faster.  Workspaces are device memory, 16-byte aligned,
 * owned by the caller, and need not be cleared; calls that may overlap on the GPU
 * need separate ones.  Results do not depend on timing: the same call gives the
 * same bits.
 */
#ifndef FP8HG_ADAPT_H
#define FP8HG_ADAPT_H

#include <stddef.h>
#include <stdint.h>

#include "fp8hg.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * fp8hg_layernorm — per row of n columns, in FP32:
 *   mean = sum(x) / n, var = sum((x - mean)^2) / n, rstd = 1 / sqrt(var + eps)
 *   y = (x - mean) rstd weight + bias
 * written as it is, and / or quantized from FP32 as the operand of an FP8 product.
 * (fp8_gemm_scaled itself takes rows and columns in multiples of 128.)
 *
 *   x, x_kind           [rows, cols], row stride ld_x
 *   weight, bias        [cols] of param_kind; NULL: 1, 0
 *   eps                 finite, not negative
 *   y, y_kind           [rows, cols], row stride ld_y; NULL: not written.  y may be
 *                       x where type and stride are the same
 *   q                   NULL, or where codes and scales go
 *   stats               [rows][2] floats, mean and rstd, for the backward pass;
 *                       8-byte aligned; NULL: not written
 * One of y, q and stats at least.  A group (row) with a NaN or an infinity among
 * its values has the scale byte 0xFF and codes 0x7F, like those of fp8_quant_token.
 */
typedef struct {
    uint8_t *codes;    /* [rows, cols], 16-byte aligned, ld a multiple of 16 */
    uint8_t *scale;    /* [rows, 1] (group 0) or [rows, ceil(cols / 128)] */
    int64_t ld, ld_scale;
    int32_t group;     /* 0: one scale per row, 128: per 128 columns; UE8M0, rounded up */
    int32_t fmt;       /* fp8hg_format */
} fp8hg_norm_codes;

int fp8hg_layernorm(const void *x, int x_kind, int64_t rows, int64_t cols, int64_t ld_x,
                    const void *weight, const void *bias, int param_kind, float eps, void *y,
                    int y_kind, int64_t ld_y, const fp8hg_norm_codes *q, float *stats,
                    void *stream);

/*
 * fp8hg_layernorm_bwd — from dy, x and the forward pass's stats, with
 * xh = (x - mean) rstd and g = dy weight:
 *   dx = rstd (g - sum(g) / n - xh sum(g xh) / n) + add
 *   dweight = sum over rows of dy xh,  dbias = sum over rows of dy
 *
 *   dy, dy_kind      [rows, cols], row stride ld_dy
 *   x, dx, add       [rows, cols] of x_kind; add (another branch's gradient): NULL
 *                    for none.  dx may be add, x or dy where type and
 *                    stride are the same
 *   dweight, dbias   [cols] floats; either or both NULL: not computed
 *   workspace        fp8hg_layernorm_bwd_workspace(rows, cols) bytes; not used if
 *                    both are NULL
 * rows = 0: dweight and dbias are zeros.
 */
size_t fp8hg_layernorm_bwd_workspace(int64_t rows, int64_t cols);
int fp8hg_layernorm_bwd(const void *dy, int dy_kind, int64_t ld_dy, const void *x, int x_kind,
                        int64_t ld_x, int64_t rows, int64_t cols, const void *weight,
                        int param_kind, const float *stats, const void *add, int64_t ld_add,
                        void *dx, int64_t ld_dx, float *dweight, float *dbias, void *workspace,
                        size_t workspace_bytes, void *stream);

/*
 * fp8hg_lora_plan — the tokens of a batch grouped by adapter, for all calls on
 * this batch.
 *
 *   ids        [tokens] int32: each token's adapter; one that is negative, or not
 *              below `adapters`, has none
 *   plan       fp8hg_lora_plan_bytes(tokens, adapters) bytes, 16-byte aligned; its
 *              content is the library's
 * At most 4096 adapters and 2^24 tokens (FP8HG_ERR_SHAPE beyond).
 */
size_t fp8hg_lora_plan_bytes(int64_t tokens, int64_t adapters);
int fp8hg_lora_plan(const int32_t *ids, int64_t tokens, int64_t adapters, void *plan,
                    size_t plan_bytes, void *stream);

/*
 * Adapters beside one projection [n, k]: A [adapters, r, k] and B [adapters, n, r]
 * in BF16, row strides ld_a and ld_b, stride_a and stride_b elements from one
 * adapter to the next.  1 <= r <= 128 (FP8HG_ERR_UNSUPPORTED beyond); n and k at
 * most 2^24.
 *
 *   scale   [adapters] floats; NULL: 1
 *   ranks   [adapters] int32: rows of A (columns of B) that an adapter has, 0 to
 *           r (clamped); what lies past them is not used.  NULL: r
 */
typedef struct {
    const uint16_t *a, *b;
    const float *scale;
    const int32_t *ranks;
    int64_t adapters, r, n, k;
    int64_t stride_a, ld_a, stride_b, ld_b;
} fp8hg_lora;

/*
 * fp8hg_lora_add — y[t] = base[t] + scale_g (x[t] A_g^T) B_g^T for the adapter g
 * of token t, y[t] = base[t] for a token without one.
 *
 *   plan      of `tokens` tokens and w->adapters adapters
 *   x         [tokens, k] BF16, row stride ld_x
 *   base, y   [tokens, n] of y_kind; base may be y, or NULL (zeros)
 *   v         NULL, or [tokens, r] floats (row stride ld_v), x[t] A_g^T for the
 *             backward pass; 0 past an adapter's rank and without one
 *   workspace fp8hg_lora_workspace(tokens, adapters, r, k) bytes
 * x A^T is summed in FP32 by the tensor core, which cuts off where others round: of up
 * to 48 sums of 16 products behind one another some 7e-7 of the result is lost, of
 * products of one sign 1.2e-6 (for da and db, 32 sums, 5e-7 and 9e-7).  It enters the
 * second product as two BF16 parts (y in BF16) or three (FP32).  Where an element of B
 * is infinite, y may be a NaN instead of an infinity (a part is 0); the same holds for
 * the backward pass and infinite elements of A, x and dy.
 */
size_t fp8hg_lora_workspace(int64_t tokens, int64_t adapters, int64_t r, int64_t k);
int fp8hg_lora_add(const fp8hg_lora *w, const void *plan, int64_t tokens, const uint16_t *x,
                   int64_t ld_x, const void *base, int64_t ld_base, void *y, int64_t ld_y,
                   int y_kind, float *v, int64_t ld_v, void *workspace, size_t workspace_bytes,
                   void *stream);

/*
 * fp8hg_lora_add_bwd — with dv[t] = scale_g dy[t] B_g:
 *   dx[t] = base[t] + dv[t] A_g,  da_g = sum over g's tokens of dv[t]^T x[t],
 *   db_g = scale_g sum over g's tokens of dy[t]^T v[t]
 *
 *   dy, x      [tokens, n] and [tokens, k] BF16
 *   v          [tokens, r] floats from fp8hg_lora_add (needed for db)
 *   base, dx   [tokens, k] of dx_kind: base (the projection's own data gradient)
 *              may be dx, or NULL (zeros); dx NULL: not computed
 *   da, db     [adapters, r, k] and [adapters, n, r] of dw_kind, contiguous; either
 *              may be NULL.  Zeros for adapters without tokens and past the ranks
 *   workspace  fp8hg_lora_bwd_workspace(tokens, adapters, r, n, k) bytes
 */
size_t fp8hg_lora_bwd_workspace(int64_t tokens, int64_t adapters, int64_t r, int64_t n, int64_t k);
int fp8hg_lora_add_bwd(const fp8hg_lora *w, const void *plan, int64_t tokens, const uint16_t *dy,
                       int64_t ld_dy, const uint16_t *x, int64_t ld_x, const float *v,
                       int64_t ld_v, const void *base, int64_t ld_base, void *dx, int64_t ld_dx,
                       int dx_kind, void *da, void *db, int dw_kind, void *workspace,
                       size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8HG_ADAPT_H */
