// Launchers of the layer norm and of the low-rank adapters, shared between the
// C-ABI layer (adapt_api.cu) and the kernel files.  Arguments are validated by
// the caller; these only configure and launch.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "lowbit.h"

namespace fp8hg {

// The SMs that work is dealt out to: a GB300's, not the device's count, because
// workspaces are functions of sizes alone, without a device, and because the host's
// grids and the device's splits of the adapters' sums have to agree.  Another number of
// SMs leaves results right and a round of CTAs less full.
constexpr int kSms = 152;

// Shared memory beyond 48 KB, a kernel's own (16 KB at most here) included, is asked for
// once per kernel and device, as much as any of its launches takes.
template <class K>
cudaError_t with_smem(K kern, size_t bytes, size_t most, unsigned long long &done) {
    if (bytes <= 32 * 1024) return cudaSuccess;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (__atomic_load_n(&done, __ATOMIC_RELAXED) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
    if (e != cudaSuccess) {
        cudaGetLastError();   // reported here, not by the next call that asks
        return e;
    }
    __atomic_fetch_or(&done, bit, __ATOMIC_RELAXED);
    return cudaSuccess;
}

// ---------------------------------------------------------------- layer norm

struct NormArgs {
    const void *x;
    int x_f32;
    int rows, cols;
    uint32_t ld_x;
    const void *weight, *bias;   // or null
    int param_f32;
    float eps;
    void *y;                     // or null
    int y_f32;
    uint32_t ld_y;
    uint8_t *q, *s;              // FP8 codes and scales, or null
    uint32_t ld_q, ld_s;
    int group, fmt;              // 0: a scale per row, 128: per 128 columns
    float *stats;                // [rows, 2], or null
};
cudaError_t launch_norm(const NormArgs &a, cudaStream_t stream);

struct NormBwdArgs {
    const void *dy, *x, *add;    // add: or null; dx = add + ...
    int dy_f32, x_f32;
    int rows, cols;
    uint32_t ld_dy, ld_x, ld_add;
    const void *weight;          // or null
    int param_f32;
    const float *stats;
    void *dx;                    // x's type
    uint32_t ld_dx;
    float *dweight, *dbias;      // either or null
    float *ws;                   // norm_bwd_ws_bytes, if dweight or dbias
};
size_t norm_bwd_ws_bytes(int64_t rows, int64_t cols);
cudaError_t launch_norm_bwd(const NormBwdArgs &a, cudaStream_t stream);

// ------------------------------------------------------------ low-rank adapters
// The tokens of a batch grouped by adapter, as int32 words in device memory:
// [0] tiles, then first position and first tile of every adapter (one more than
// adapters: the tokens without one), the tokens in that order, and the tiles
// (adapter or -1, first position, tokens, first token where they are neighbours or
// -1) of up to kLoraTile tokens of one adapter each.
constexpr int kLoraTile = 128;
constexpr int kLoraMaxAdapters = 4096;
constexpr int kLoraMaxRank = 128;
struct LoraPlan {
    const int *words;
    int tokens, adapters;
    __host__ __device__ int64_t starts() const { return 4; }
    __host__ __device__ int64_t tile_first() const { return starts() + adapters + 2; }
    __host__ __device__ int64_t order() const { return tile_first() + adapters + 2; }
    __host__ __device__ int64_t tiles() const { return (order() + tokens + 3) / 4 * 4; }
    // no more tiles than this
    __host__ __device__ int max_tiles() const {
        return tokens / kLoraTile + (adapters + 1 < tokens ? adapters + 1 : tokens);
    }
    __host__ __device__ int64_t size() const { return tiles() + 4 * static_cast<int64_t>(max_tiles()); }
};
cudaError_t launch_lora_plan(const int *ids, const LoraPlan &p, int *words, cudaStream_t stream);

struct LoraWeights {
    const uint16_t *a, *b;       // [adapters, r, k], [adapters, n, r]
    int64_t stride_a, stride_b;  // from one adapter to the next, elements
    uint32_t ld_a, ld_b;
    const float *scale;          // [adapters], or null: 1
    const int *ranks;            // [adapters], or null: r
    int r, n, k;
};

struct LoraArgs {
    LoraWeights w;
    LoraPlan plan;
    const uint16_t *x;
    uint32_t ld_x;
    const void *base;            // or null: zeros
    void *y;
    int y_f32;
    uint32_t ld_base, ld_y;
    float *v;                    // [tokens, r] x A^T, or null
    uint32_t ld_v;
    float *ws;
};
size_t lora_ws_bytes(int64_t tokens, int adapters, int r, int64_t k);
cudaError_t launch_lora_add(const LoraArgs &a, cudaStream_t stream);

struct LoraBwdArgs {
    LoraWeights w;
    LoraPlan plan;
    const uint16_t *dy, *x;
    uint32_t ld_dy, ld_x;
    const float *v;
    uint32_t ld_v;
    const void *base;            // the base projection's data gradient, or null: zeros
    void *dx;                    // or null
    int dx_f32;
    uint32_t ld_base, ld_dx;
    void *da, *db;               // [adapters, r, k], [adapters, n, r], contiguous; either or null
    int dw_f32;
    float *ws;
};
size_t lora_bwd_ws_bytes(int64_t tokens, int adapters, int r, int64_t n, int64_t k);
cudaError_t launch_lora_add_bwd(const LoraBwdArgs &a, cudaStream_t stream);

}  // namespace fp8hg
