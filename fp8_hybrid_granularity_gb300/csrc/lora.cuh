// What the adapters' kernels share: tiles of rows in shared memory, the tokens
// of a tile, FP32 values as sums of BF16 ones.
#pragma once
#include <cstdint>

#include "adapt.h"
#include "ptx.cuh"

namespace fp8hg {
namespace lora {

// Bytes of a row of `cols` 16-bit values in shared memory: 16 more than it
// needs, so that eight rows' 16-byte pieces fall on different banks.
__host__ __device__ constexpr int row_bytes(int cols) { return 2 * cols + 16; }

// A tile of the plan.
struct Tile {
    int adapter, first, count;
};
__device__ __forceinline__ Tile tile_at(const LoraPlan &p, int i) {
    const int2 t = reinterpret_cast<const int2 *>(p.words + p.tiles())[i];
    const int *starts = p.words + p.starts();
    const int end = starts[(t.x < 0 ? p.adapters : t.x) + 1];
    return {t.x, t.y, min(kLoraTile, end - t.y)};
}
__device__ __forceinline__ int rank_of(const LoraWeights &w, int g) {
    return w.ranks == nullptr ? w.r : max(0, min(w.r, w.ranks[g]));
}

// Eight values from p on, the first `left` of them (zeros behind), to 16 bytes
// of shared memory.  ALIGNED: p is a multiple of 16 bytes.
template <bool ALIGNED>
__device__ __forceinline__ void copy8(uint32_t dst, const uint16_t *p, int left) {
    const int n = max(0, min(8, left));
    if constexpr (ALIGNED) {
        ptx::cp_async16(dst, p, 2 * n);
    } else {
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) w[i >> 1] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
        ptx::st_shared_v4(dst, w[0], w[1], w[2], w[3]);
    }
}

// v as the sum of PARTS BF16 values: 16 bits of it with two, all 24 with three.
template <int PARTS>
__device__ __forceinline__ void split(float v, uint16_t (&h)[PARTS]) {
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
        h[i] = static_cast<uint16_t>(ptx::cvt_bf16x2(v, 0.0f) & 0xFFFFu);
        // an infinity or a NaN is in the first part alone
        v = (h[i] & 0x7F80u) == 0x7F80u ? 0.0f : v - __uint_as_float(static_cast<uint32_t>(h[i]) << 16);
    }
}

}  // namespace lora
}  // namespace fp8hg
