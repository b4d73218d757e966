// What the layer norm's forward and backward kernels share: rows held in
// registers, sixteen neighbouring columns a thread.
#pragma once
#include <cstdint>

#include "adapt.h"
#include "pair_math.cuh"
#include "ragged.cuh"

namespace fp8hg {
namespace norm {

// Sixteen values as loaded: BF16 pairs or FP32.
template <bool F32>
struct Raw {
    uint32_t w[F32 ? 16 : 8];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (F32 ? 16 : 8); ++i) w[i] = 0u;
    }
    template <bool WIDE>
    __device__ __forceinline__ void load(const void *base, int64_t at, int left) {
        if constexpr (F32) ragged::load16<WIDE>(static_cast<const float *>(base) + at, left, w);
        else ragged::load16<WIDE>(static_cast<const uint16_t *>(base) + at, left, w);
    }
    __device__ __forceinline__ F2 pair(int i) const {
        if constexpr (F32) return f2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        else return f2_bf16(w[i]);
    }
};

// Sixteen values to base[at ...] in BF16 or FP32 (every lane of the warp calls it).
template <bool WIDE>
__device__ __forceinline__ void store_values(void *base, int f32, int64_t at, int left, const F2 (&v)[8]) {
    if (f32) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[2 * i] = __float_as_uint(v[i].lo()), w[2 * i + 1] = __float_as_uint(v[i].hi());
        ragged::store16<WIDE>(static_cast<float *>(base) + at, left, w);
    } else {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = ptx::cvt_bf16x2(v[i].lo(), v[i].hi());
        ragged::store16<WIDE>(static_cast<uint16_t *>(base) + at, left, w);
    }
}

// Sixteen parameters from column c0 on; `none` without a tensor, 0 past the last.
__device__ __forceinline__ void load_params(const void *p, int f32, float none, int c0, int left, F2 (&v)[8]) {
    if (left <= 0 || p == nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = f2(left > 0 ? none : 0.0f);
    } else if (f32) {
        Raw<true> r;
        r.load<false>(p, c0, left);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = r.pair(i);
    } else {
        Raw<false> r;
        r.load<false>(p, c0, left);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = r.pair(i);
    }
}

// Zeros from element `left` on.
__device__ __forceinline__ void cut(F2 (&v)[8], int left) {
    if (left < 16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = f2(2 * i < left ? v[i].lo() : 0.0f, 2 * i + 1 < left ? v[i].hi() : 0.0f);
    }
}

// The same of every 32nd column.
__device__ __forceinline__ void cut_lanes(F2 (&v)[8], int left) {
    if (left <= 15 * 32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = f2(j * 64 < left ? v[j].lo() : 0.0f, j * 64 + 32 < left ? v[j].hi() : 0.0f);
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

__device__ __forceinline__ float total(const F2 (&v)[8]) {
    const F2 a = add2(add2(v[0], v[1]), add2(v[2], v[3])), b = add2(add2(v[4], v[5]), add2(v[6], v[7]));
    const F2 s = add2(a, b);
    return s.lo() + s.hi();
}

// A sum as it is.
struct Same {
    __device__ __forceinline__ float operator()(float s) const { return s; }
};

// One, two or four sums (or a maximum) over the threads of a row: `warps` whole
// warps, at most 16.  Every thread of the CTA calls them in step; two buffers in
// turn, so that one barrier for each set is enough.  `then`: what is wanted of a sum,
// taken once in the lanes that add it up, before all threads get it.
struct RowReduce {
    float (*buf)[32][4];     // [2] of a warp's four values
    int warps, first, turn;
    __device__ __forceinline__ RowReduce(float (*b)[32][4], int tpr)
        : buf(b), warps(tpr / 32), first(threadIdx.x / tpr * (tpr / 32)), turn(0) {}

    // The row's from the warps': lane l has value l / (32 / N) of warp l % W, and every
    // lane a sum that is wanted (a division by the way of zeros takes longer).
    template <int N, bool MAX, class F = Same>
    __device__ __forceinline__ void across(float (&v)[N], F then = F()) {
        constexpr int W = 32 / N < 16 ? 32 / N : 16;
        const int lane = threadIdx.x & 31, at = lane % W;
        __syncthreads();
        const float (*t)[4] = buf[turn] + first;
        turn ^= 1;
        float a = at < warps ? t[at][lane / (32 / N)] : 0.0f;
        if (W < 16 && at + W < warps) {
            const float u = t[at + W][lane / (32 / N)];
            a = MAX ? max3_abs(a, a, u) : a + u;
        }
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1) {
            const float u = __shfl_xor_sync(0xFFFFFFFFu, a, o);
            a = MAX ? max3_abs(a, a, u) : a + u;
        }
        a = then(a);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, a, i * (32 / N));
    }
    template <class F = Same>
    __device__ __forceinline__ float sum(float a, F then = F()) {
        float v[1] = {warp_sum(a)};
        if (warps > 1) {
            if ((threadIdx.x & 31) == 0) buf[turn][threadIdx.x / 32][0] = v[0];
            across<1, false>(v, then);
        } else {
            v[0] = then(v[0]);
        }
        return v[0];
    }
    __device__ __forceinline__ float max(float a) {
        float v[1] = {warp_max_abs(a)};
        if (warps > 1) {
            if ((threadIdx.x & 31) == 0) buf[turn][threadIdx.x / 32][0] = v[0];
            across<1, true>(v);
        }
        return v[0];
    }
    template <class F = Same>
    __device__ __forceinline__ void sum(float (&v)[2], F then = F()) {
        const bool up = threadIdx.x & 16;
        float a = (up ? v[1] : v[0]) + __shfl_xor_sync(0xFFFFFFFFu, up ? v[0] : v[1], 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        if (warps > 1) {
            if ((threadIdx.x & 15) == 0) buf[turn][threadIdx.x / 32][(threadIdx.x >> 4) & 1] = a;
            across<2, false>(v, then);
        } else {
            a = then(a);
            v[0] = __shfl_sync(0xFFFFFFFFu, a, 0);
            v[1] = __shfl_sync(0xFFFFFFFFu, a, 16);
        }
    }
    // four: halves, then quarters of the warp take over one value each
    template <class F = Same>
    __device__ __forceinline__ void sum(float (&v)[4], F then = F()) {
        const int lane = threadIdx.x & 31;
        const bool up = lane & 16, odd = lane & 8;
        float a = (up ? v[2] : v[0]) + __shfl_xor_sync(0xFFFFFFFFu, up ? v[0] : v[2], 16);
        float b = (up ? v[3] : v[1]) + __shfl_xor_sync(0xFFFFFFFFu, up ? v[1] : v[3], 16);
        a = (odd ? b : a) + __shfl_xor_sync(0xFFFFFFFFu, odd ? a : b, 8);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        if (warps > 1) {
            if ((lane & 7) == 0) buf[turn][threadIdx.x / 32][lane >> 3] = a;
            across<4, false>(v, then);
        } else {
            a = then(a);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, a, 8 * i);
        }
    }
    template <class F = Same>
    __device__ __forceinline__ void sum(float (&v)[1], F then = F()) {
        v[0] = sum(v[0], then);
    }
    __device__ __forceinline__ void max(float (&v)[1]) { v[0] = max(v[0]); }
    template <int N>
    __device__ __forceinline__ void max(float (&v)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = warp_max_abs(v[i]);
            if (warps > 1 && (threadIdx.x & 31) == 0) buf[turn][threadIdx.x / 32][i] = v[i];
        }
        if (warps > 1) across<N, true>(v);
    }
    __device__ __forceinline__ float2 both(float a, float b) {
        float v[2] = {a, b};
        sum(v);
        return make_float2(v[0], v[1]);
    }
};

// A thread's sixteen parameters in shared memory: pieces of four, the threads'
// pieces next to one another, so that neither access meets a bank twice.
__device__ __forceinline__ void keep_params(float *at, int t, int tpr, const F2 (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        reinterpret_cast<float4 *>(at)[j * tpr + t] =
            make_float4(v[2 * j].lo(), v[2 * j].hi(), v[2 * j + 1].lo(), v[2 * j + 1].hi());
}
__device__ __forceinline__ void kept_params(const float *at, int t, int tpr, int j, F2 &a, F2 &b) {
    const float4 q = reinterpret_cast<const float4 *>(at)[j * tpr + t];
    a = f2(q.x, q.y);
    b = f2(q.z, q.w);
}

// A warp's 512 columns of a row through shared memory: copied 16 bytes a lane next
// to one another (no sector is asked for twice), read back 16 columns a lane.  WIDE:
// rows that begin at multiples of 16 bytes; others come as the aligned 16-byte
// granules that hold them, one more than they fill, and are moved into place when
// they are read.
template <bool F32, bool WIDE>
constexpr int kSegment = (F32 ? 2048 : 1024) + (WIDE ? 0 : 16);
__device__ __forceinline__ uint32_t segment_at(int p) { return (p ^ ((p >> 3) & 3)) * 16; }
__device__ __forceinline__ const void *base_granule(const void *p) {
    return reinterpret_cast<const void *>(reinterpret_cast<uintptr_t>(p) & ~static_cast<uintptr_t>(15));
}
template <bool F32>
__device__ __forceinline__ uintptr_t column_address(const void *base, int64_t at) {
    return reinterpret_cast<uintptr_t>(base) + at * (F32 ? 4 : 2);
}

template <bool F32, bool WIDE, bool LINEAR = false>
__device__ __forceinline__ void copy_columns(uint32_t to, const void *base, int64_t at, int left) {
    constexpr int E = F32 ? 4 : 2;
    const int lane = threadIdx.x & 31, bytes = max(0, min(512, left)) * E;
    const uintptr_t a = column_address<F32>(base, at), from = a & ~static_cast<uintptr_t>(15);
    const int have = bytes > 0 ? bytes + static_cast<int>(a & 15) : 0;      // of the granules
    auto piece = [&](int p) {
        // a granule is read whole if a byte of it belongs to the row
        const int n = WIDE ? max(0, min(16, have - 16 * p)) : have > 16 * p ? 16 : 0;
        ptx::cp_async16(to + (LINEAR ? 16 * p : segment_at(p)), n > 0 ? reinterpret_cast<const void *>(from + 16 * p) : base_granule(base), n);
    };
#pragma unroll
    for (int h = 0; h < E; ++h) piece(h * 32 + lane);
    if (!WIDE && lane == 0) piece(32 * E);
}
template <bool F32, bool WIDE>
__device__ __forceinline__ void read_columns(uint32_t from, uint32_t shift, int left, Raw<F32> &v) {
    constexpr int N = F32 ? 4 : 2;
    if constexpr (WIDE) {
#pragma unroll
        for (int h = 0; h < N; ++h)
            ptx::ld_shared_v4(from + segment_at((threadIdx.x & 31) * N + h), v.w[4 * h], v.w[4 * h + 1], v.w[4 * h + 2], v.w[4 * h + 3]);
    } else {
        uint32_t w[4 * (N + 1)];
#pragma unroll
        for (int h = 0; h <= N; ++h)
            ptx::ld_shared_v4(from + segment_at((threadIdx.x & 31) * N + h), w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
        if constexpr (F32) ragged::shift_words(w, shift >> 2);
        else ragged::shift_down(w, shift);
#pragma unroll
        for (int i = 0; i < 4 * N; ++i) v.w[i] = w[i];
        // the last granule also holds what is behind the row
        if (left < 16) {
#pragma unroll
            for (int i = 0; i < 4 * N; ++i) {
                if (F32) v.w[i] = i < left ? v.w[i] : 0u;
                else v.w[i] = 2 * i + 1 < left ? v.w[i] : 2 * i < left ? v.w[i] & 0xFFFFu : 0u;
            }
        }
    }
}

// LINEAR granules read back as they lie, every 32nd column a lane: nothing to move into
// place.  left: columns from the lane's first one on.
template <bool F32>
__device__ __forceinline__ void read_lanes(uint32_t from, uint32_t shift, int left, Raw<F32> &v) {
    constexpr int E = F32 ? 4 : 2;
    from += shift + (threadIdx.x & 31) * E;
    if constexpr (F32) {
#pragma unroll
        for (int j = 0; j < 16; ++j) v.w[j] = ptx::ld_shared_u32(from + j * 32 * E);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v.w[j] = ptx::ld_shared_u16(from + 2 * j * 32 * E) | ptx::ld_shared_u16(from + (2 * j + 1) * 32 * E) << 16;
    }
    // the last granule also holds what is behind the row
    if (left <= 15 * 32) {
#pragma unroll
        for (int j = 0; j < (F32 ? 16 : 8); ++j) {
            if (F32) v.w[j] = j * 32 < left ? v.w[j] : 0u;
            else v.w[j] = (2 * j + 1) * 32 < left ? v.w[j] : 2 * j * 32 < left ? v.w[j] & 0xFFFFu : 0u;
        }
    }
}
// Every 32nd parameter from column c0 on.
__device__ __forceinline__ void load_params_lanes(const void *p, int f32, float none, int c0, int left, F2 (&v)[8]) {
    auto value = [&](int j) {
        return j * 32 >= left ? 0.0f
               : p == nullptr ? none
               : f32 ? static_cast<const float *>(p)[c0 + j * 32]
                     : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(p)[c0 + j * 32]) << 16);
    };
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = f2(value(2 * j), value(2 * j + 1));
}
// Every 32nd column of a row from at on.
__device__ __forceinline__ void store_lanes(void *base, int f32, int64_t at, int left, const F2 (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const float u = j & 1 ? v[j / 2].hi() : v[j / 2].lo();
        if (j * 32 < left) {
            if (f32) static_cast<float *>(base)[at + j * 32] = u;
            else static_cast<uint16_t *>(base)[at + j * 32] = static_cast<uint16_t>(ptx::cvt_bf16x2(u, 0.0f));
        }
    }
}

// How a row is dealt out where it fits the registers: threads a row (whole
// warps), rows a CTA.
constexpr int kRegCols = 8192;
struct Shape {
    int tpr, rpb;
};
inline Shape shape_of(int64_t cols) {
    Shape s;
    s.tpr = static_cast<int>(cols > kRegCols ? 512 : (cols + 511) / 512 * 32);
    s.rpb = s.tpr >= 256 ? 1 : 256 / s.tpr;
    return s;
}
inline bool wide_rows(const void *p, int f32, int64_t ld) { return f32 ? ragged::wide_f32(p, ld) : ragged::wide(p, ld); }

}  // namespace norm
}  // namespace fp8hg
