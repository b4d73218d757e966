// Product of two 4-bit tensors, C = A B^T, with block scales.
//
// A first, plain form: 64 x 64 tiles, operands decoded to FP32 in shared
// memory, four by four outputs per thread.
#include <cuda_runtime.h>

#include <cstdint>

#include "fp4_math.cuh"
#include "lowbit.h"

namespace fp8hg {

namespace {

constexpr int kM = 64, kK = 32;

template <bool NV>
__device__ __forceinline__ void decode_tile(float (&dst)[kK][kM + 1], const Fp4Operand &o,
                                            int64_t row0, int64_t k0, int64_t tiles) {
    // a thread decodes eight elements of one row
    const int r = threadIdx.x >> 2, c = (threadIdx.x & 3) * 8;
    const int64_t row = row0 + r, k = k0 + c;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (row < o.rows && k < o.k) {
        uint32_t w = 0;
        for (int i = 0; i < 4; ++i)
            if (k + 2 * i < o.k) w |= static_cast<uint32_t>(o.codes[row * o.ld + k / 2 + i]) << (8 * i);
        e2m1x8_values(w, v);
        const float s = fp4_scale_value<NV>(o.scale[fp4_scale_offset(row, k / (NV ? 16 : 32), tiles)]);
        for (int i = 0; i < 8; ++i) v[i] = k + i < o.k ? v[i] * s : 0.0f;
    }
    for (int i = 0; i < 8; ++i) dst[c + i][r] = v[i];
}

template <bool NV>
__global__ void __launch_bounds__(256) k_gemm_fp4_plain(const Fp4GemmArgs g, int64_t tiles) {
    __shared__ float sa[kK][kM + 1], sb[kK][kM + 1];
    const int64_t m0 = static_cast<int64_t>(blockIdx.x) * kM, n0 = static_cast<int64_t>(blockIdx.y) * kM;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < g.a.k; k0 += kK) {
        decode_tile<NV>(sa, g.a, m0, k0, tiles);
        decode_tile<NV>(sb, g.b, n0, k0, tiles);
        __syncthreads();
        for (int k = 0; k < kK; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] += sa[k][ty + 16 * i] * sb[k][tx + 16 * j];
        __syncthreads();
    }
    const float t = (g.a.ts ? *g.a.ts : 1.0f) * (g.b.ts ? *g.b.ts : 1.0f);
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m >= g.a.rows || n >= g.b.rows) continue;
            float v = acc[i][j] * t;
            if (g.out_fp32) {
                float *c = static_cast<float *>(g.c) + m * g.ldc + n;
                *c = g.accumulate ? *c + v : v;
            } else {
                uint16_t *c = static_cast<uint16_t *>(g.c) + m * g.ldc + n;
                if (g.accumulate) v += __uint_as_float(static_cast<uint32_t>(*c) << 16);
                *c = static_cast<uint16_t>(ptx::cvt_bf16x2(v, 0.0f));
            }
        }
}

}  // namespace

int launch_fp4_gemm(const Fp4GemmArgs &g, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>((g.a.rows + kM - 1) / kM),
                    static_cast<unsigned>((g.b.rows + kM - 1) / kM));
    const int64_t tiles = fp4_scale_tiles(g.a.k, g.a.kind);
    if (g.a.kind == FP4_NV) k_gemm_fp4_plain<true><<<grid, 256, 0, stream>>>(g, tiles);
    else k_gemm_fp4_plain<false><<<grid, 256, 0, stream>>>(g, tiles);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? 0 : 2 + static_cast<int>(e);
}

}  // namespace fp8hg
