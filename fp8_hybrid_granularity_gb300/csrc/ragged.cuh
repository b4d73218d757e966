// Sixteen neighbouring BF16 (or FP32) values per thread, loaded from and stored
// to rows of any alignment.
//
// WIDE: the address is a multiple of 32 bytes (the row stride too): one
// 32-byte access, a whole sector per lane.  (Two 16-byte loads that bypass L1
// fetch every sector twice.)
//
// Otherwise a row may start at any even address.  A load takes the aligned
// 16-byte granules that hold the thread's 32 bytes (three at most; the granule
// shared with the neighbouring lane is an L1 hit) and shifts them into place;
// a granule is read only if a byte of it belongs to the row, so nothing
// outside the 16-byte granules of the row is touched.  A store is shifted the
// other way: each lane writes the two aligned granules that begin within its
// 32 bytes, the last bytes of the second one coming from the next lane, and
// only the ends of a row (and of a warp) are written two bytes at a time.
#pragma once
#include <cstdint>

#include "ptx.cuh"

namespace fp8hg {
namespace ragged {

// Words of a 48-byte window moved down by b bytes (b even, below 16): the
// first eight are wanted.
__device__ __forceinline__ void shift_down(uint32_t (&w)[12], uint32_t b) {
    if (b & 8) {
#pragma unroll
        for (int i = 0; i < 10; ++i) w[i] = w[i + 2];
    }
    if (b & 4) {
#pragma unroll
        for (int i = 0; i < 9; ++i) w[i] = w[i + 1];
    }
    if (b & 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
}

// Values p[0 .. 15], zeros from index `left` on (left > 0).
template <bool WIDE>
__device__ __forceinline__ void load16(const uint16_t *p, int left, uint32_t (&v)[8]) {
    if (WIDE && left >= 16) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                       "=r"(v[6]), "=r"(v[7])
                     : "l"(p)
                     : "memory");
        return;
    }
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    const uint32_t s = static_cast<uint32_t>(a & 15);
    const uint4 *g = reinterpret_cast<const uint4 *>(a & ~static_cast<uintptr_t>(15));
    const uint32_t bytes = left >= 16 ? 32u : static_cast<uint32_t>(left) * 2u;
    uint32_t w[12];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        uint4 q = make_uint4(0u, 0u, 0u, 0u);
        if (s + bytes > 16u * i) q = ptx::ld_v4(g + i);
        w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
    }
    shift_down(w, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = w[i];
        if (bytes < 4u * i + 4u) v[i] = bytes > 4u * i ? v[i] & 0xFFFFu : 0u;
    }
}

// Values to p[0 .. 15], the first `left` of them (none if left <= 0).  Every
// lane of the warp calls it; lanes without a row pass left = 0.
template <bool WIDE>
__device__ __forceinline__ void store16(uint16_t *p, int left, const uint32_t (&v)[8]) {
    if (WIDE) {
        if (left >= 16) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
                         "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                         : "memory");
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i < left) p[i] = static_cast<uint16_t>(v[i >> 1] >> (16 * (i & 1)));
        }
        return;
    }
    const int lane = threadIdx.x & 31;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    const uint32_t bytes = left >= 16 ? 32u : left > 0 ? static_cast<uint32_t>(left) * 2u : 0u;
    const uint32_t d = static_cast<uint32_t>(-static_cast<intptr_t>(a) & 15);   // to the next granule
    uint32_t w[12];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = v[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[8 + i] = __shfl_down_sync(0xFFFFFFFFu, v[i], 1);
    const uintptr_t na = __shfl_down_sync(0xFFFFFFFFu, static_cast<unsigned long long>(a), 1);
    const uint32_t nbytes = __shfl_down_sync(0xFFFFFFFFu, bytes, 1);
    // the second granule is complete with the next lane's first d bytes
    const bool joined = lane < 31 && bytes == 32u && na == a + 32 && nbytes >= d && d != 0;
    const bool head_done = __shfl_up_sync(0xFFFFFFFFu, joined ? 1 : 0, 1) && lane > 0;
    if (bytes == 0) return;
    const uint32_t from = head_done ? d : 0u;      // first byte this lane still has to write
    if (bytes == 32u) {
        // the head, and the tail where the next lane does not complete it
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (2u * i >= from && 2u * i < d) p[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
        if (!joined && d != 0) {
#pragma unroll
            for (int i = 9; i < 16; ++i)
                if (2u * i >= d + 16u) p[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
        }
        shift_down(w, d);
        uint4 *g = reinterpret_cast<uint4 *>(a + d);
        g[0] = make_uint4(w[0], w[1], w[2], w[3]);
        if (joined || d == 0) g[1] = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (2u * i >= from && 2u * i < bytes)
                p[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
    }
}

// Words of an 80-byte window moved down by s words (s below 4): the first 16 are wanted.
__device__ __forceinline__ void shift_words(uint32_t (&w)[20], uint32_t s) {
    if (s & 2) {
#pragma unroll
        for (int i = 0; i < 18; ++i) w[i] = w[i + 2];
    }
    if (s & 1) {
#pragma unroll
        for (int i = 0; i < 17; ++i) w[i] = w[i + 1];
    }
}

// Sixteen neighbouring FP32 values per thread, by the same rules: WIDE rows in
// 32-byte accesses, others (a multiple of 4 bytes) in aligned 16-byte granules.
template <bool WIDE>
__device__ __forceinline__ void load16(const float *p, int left, uint32_t (&v)[16]) {
    if (WIDE && left >= 16) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(v[8 * i]), "=r"(v[8 * i + 1]), "=r"(v[8 * i + 2]), "=r"(v[8 * i + 3]),
                           "=r"(v[8 * i + 4]), "=r"(v[8 * i + 5]), "=r"(v[8 * i + 6]), "=r"(v[8 * i + 7])
                         : "l"(p + 8 * i)
                         : "memory");
        return;
    }
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    const uint32_t s = static_cast<uint32_t>(a >> 2) & 3u;
    const uint4 *g = reinterpret_cast<const uint4 *>(a & ~static_cast<uintptr_t>(15));
    const uint32_t words = left >= 16 ? 16u : static_cast<uint32_t>(left);
    uint32_t w[20];
#pragma unroll
    for (int i = 0; i < 5; ++i) {
        uint4 q = make_uint4(0u, 0u, 0u, 0u);
        if (s + words > 4u * i) q = ptx::ld_v4(g + i);
        w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
    }
    shift_words(w, s);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = i < words ? w[i] : 0u;
}

template <bool WIDE>
__device__ __forceinline__ void store16(float *p, int left, const uint32_t (&v)[16]) {
    if (WIDE && left >= 16) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + 8 * i), "r"(v[8 * i]),
                         "r"(v[8 * i + 1]), "r"(v[8 * i + 2]), "r"(v[8 * i + 3]), "r"(v[8 * i + 4]),
                         "r"(v[8 * i + 5]), "r"(v[8 * i + 6]), "r"(v[8 * i + 7])
                         : "memory");
        return;
    }
    if (WIDE) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < left) p[i] = __uint_as_float(v[i]);
        return;
    }
    const int lane = threadIdx.x & 31;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    const int words = left >= 16 ? 16 : left > 0 ? left : 0;
    const int d = static_cast<int>(-static_cast<intptr_t>(a >> 2) & 3);   // to the next granule
    uint32_t w[20];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = v[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[16 + i] = __shfl_down_sync(0xFFFFFFFFu, v[i], 1);
    const uintptr_t na = __shfl_down_sync(0xFFFFFFFFu, static_cast<unsigned long long>(a), 1);
    const int nwords = __shfl_down_sync(0xFFFFFFFFu, words, 1);
    // the last granule is complete with the next lane's first d words
    const bool joined = lane < 31 && words == 16 && na == a + 64 && nwords >= d && d != 0;
    const bool head_done = __shfl_up_sync(0xFFFFFFFFu, joined ? 1 : 0, 1) && lane > 0;
    const int from = head_done ? d : 0;            // first word this lane still has to write
    if (words == 16) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i >= from && i < d) p[i] = __uint_as_float(w[i]);
        if (!joined && d != 0) {
#pragma unroll
            for (int i = 13; i < 16; ++i)
                if (i >= d + 12) p[i] = __uint_as_float(w[i]);
        }
        shift_words(w, d);
        uint4 *g = reinterpret_cast<uint4 *>(a + 4 * d);
#pragma unroll
        for (int i = 0; i < 3; ++i) g[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        if (joined || d == 0) g[3] = make_uint4(w[12], w[13], w[14], w[15]);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i >= from && i < words) p[i] = __uint_as_float(w[i]);
    }
}

// Whether rows from p with stride ld (elements) take the WIDE forms.
inline bool wide(const void *p, int64_t ld) {
    return reinterpret_cast<uintptr_t>(p) % 32 == 0 && ld % 16 == 0;
}
inline bool wide_f32(const void *p, int64_t ld) {
    return reinterpret_cast<uintptr_t>(p) % 32 == 0 && ld % 8 == 0;
}

}  // namespace ragged
}  // namespace fp8hg
