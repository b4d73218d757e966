// Launchers of the 4-bit operators and of the SwiGLU with 8-bit checkpoints,
// shared between the C-ABI layer (lowbit_api.cu) and the kernel files.
// Arguments are validated by the caller; these only configure and launch.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "internal.h"

namespace fp8hg {

enum { FP4_MX = 0, FP4_NV = 1 };

// Tiles (128 rows x 4 blocks) along k of a scale array: k padded to 256.
inline int64_t fp4_scale_tiles(int64_t k, int kind) {
    return (k + 255) / 256 * (kind == FP4_NV ? 4 : 2);
}
inline int64_t fp4_row_tiles(int64_t rows) { return (rows + 127) / 128; }

size_t fp4_tensor_scale_ws_bytes();
// Rows and columns of a tensor are below 2^31, its row strides too (elements or
// bytes): a row's offset is then one widening multiplication.
cudaError_t launch_fp4_tensor_scale(const uint16_t *x, int rows, int cols, uint32_t ld_x,
                                    float *scale, void *ws, cudaStream_t stream);

struct Fp4QuantArgs {
    const uint16_t *x;
    int rows, cols;
    uint32_t ld_x;
    int kind;
    const float *ts;
    uint8_t *q;              // along the rows, or null
    uint32_t ld_q;
    uint8_t *s;
    uint8_t *qt;             // along the columns, or null
    uint32_t ld_qt;
    uint8_t *st;
};
cudaError_t launch_fp4_quant(const Fp4QuantArgs &a, cudaStream_t stream);

struct Fp4Operand {
    const uint8_t *codes, *scale;
    const float *ts;
    int64_t rows, k, ld;
    int kind;
};
cudaError_t launch_fp4_dequant(const Fp4Operand &a, void *out, uint32_t ld_out, int fp32,
                               cudaStream_t stream);

struct Fp4GemmArgs {
    Fp4Operand a, b;
    const uint16_t *x = nullptr;   // A in BF16 instead, quantized on the way (then a: rows, k, kind, ts)
    int64_t ld_x = 0;
    void *c;
    int64_t ldc;
    int out_fp32, accumulate;
    uint64_t wait_limit_ns;
    int inject_fault;
    unsigned int *err;
};
// Whether launch_fp4_gemm takes so many rows of A in BF16.
bool fp4_linear_quantizes(int64_t rows);
// 0 on success, 1 if a tensor map could not be encoded or a fault cannot be
// injected in the kernel that the shape takes, cudaError_t + 2 on a launch failure.
int launch_fp4_gemm(const Fp4GemmArgs &g, cudaStream_t stream);

struct SwigluFwdArgs {
    const uint16_t *gate, *up;
    int rows, cols;
    uint32_t ld_in;
    int fmt_h, fmt;
    uint8_t *h, *hs;
    uint32_t ld_h, ld_hs;
    uint8_t *gq, *gs, *uq, *us;  // the checkpoint, or all null
    uint32_t ld_q, ld_s;
};
cudaError_t launch_swiglu_fwd(const SwigluFwdArgs &a, cudaStream_t stream);

struct SwigluCkpt {
    const uint8_t *gq, *gs, *uq, *us;
    int rows, cols;
    uint32_t ld_q, ld_s;
    int fmt;
};
cudaError_t launch_swiglu_bwd(const uint16_t *dh, uint32_t ld_dh, const SwigluCkpt &c, uint16_t *dg,
                              uint16_t *du, uint32_t ld_d, cudaStream_t stream);

struct SwigluGrads {
    uint8_t *q[2], *s[2];        // dgate, dup: 1x128 along the rows
    uint8_t *qt[3], *st[3];      // dgate, dup, h: 1x128 along the tokens, transposed
    uint32_t ld_q, ld_s, ld_qt, ld_st;
    int fmt, fmt_t, fmt_h;
    unsigned int *err;
};
cudaError_t launch_swiglu_bwd_q(const uint16_t *dh, uint32_t ld_dh, const SwigluCkpt &c,
                                const SwigluGrads &g, cudaStream_t stream);

// SMs of the current device (looked up once per device; any thread).
int sm_count();

// Launches a kernel that begins with ptx::grid_begin() or grid_wait(), under the
// end of the stream's last kernel where that allows it: 1 to 2 us less from one
// kernel to the next.  cluster > 1: that many CTAs in a cluster.
template <class... P, class... A>
cudaError_t launch_after(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, int cluster,
                         const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
    if (e != cudaSuccess) cudaGetLastError();   // reported here, not by the next call that asks
    return e;
}

// Grids of row blocks, which a kernel steps through, by chunks of columns, of which
// there may be more than the 65535 of a grid's second and third dimension.  Chunks
// first: the SwiGLU backward takes 63.7 us instead of 67.7 at 8192 x 5003, the values
// of 8192 x 8960 MX 30.9 instead of 32.3; the quantizer along rows 32.2 either way
// (NV).  Rows first: the SwiGLU forward takes 341 us instead of 347 at 16384 x 18944.
constexpr int kGridY = 65535;
inline dim3 chunks_first(int64_t row_blocks, int64_t chunks) {
    return dim3(static_cast<unsigned>(chunks), static_cast<unsigned>(row_blocks < kGridY ? row_blocks : kGridY));
}
inline dim3 rows_first(int64_t row_blocks, int64_t chunks) {
    const int64_t z = (chunks + kGridY - 1) / kGridY;
    return dim3(static_cast<unsigned>(row_blocks), static_cast<unsigned>((chunks + z - 1) / z), static_cast<unsigned>(z));
}
#ifdef __CUDACC__
// The chunk of a CTA in the latter; up to z - 1 are past the last.
__device__ __forceinline__ int column_chunk() { return static_cast<int>(blockIdx.z * gridDim.y + blockIdx.y); }
#endif

// Offset of a row.
__host__ __device__ inline int64_t row_at(uint32_t row, uint32_t ld) {
    return static_cast<int64_t>(static_cast<uint64_t>(row) * ld);
}

}  // namespace fp8hg
