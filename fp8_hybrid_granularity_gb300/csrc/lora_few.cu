// Adapters: both products of few tokens (decoding) in one launch.
//
// A cluster of eight CTAs takes a run of all tiles' steps of 16 columns.  For every tile
// that it meets, its 64 warps share the long side of x A^T, 32 columns each at a time,
// and add their sums up, first in a CTA, then across the cluster's shared memory, in a
// fixed order; then they share the run's steps.  16 tokens at a time are the rows of an
// mma.sync; A's and B's rows go from memory straight into its fragments, 16 bytes a lane
// as they lie: a sum does not mind the order of its terms, so four lanes' pieces of a
// row are the K of two products, and lane t of a row of results has columns 4 t to
// 4 t + 3.
//
// Bound by latency: one token at 18944 x 3584, r 16, is 0.7 MB, and a CTA is done 4 us
// after its start: 0.9 for the plan, 0.7 for A and x, 0.8 for the cluster's barrier, 0.2
// for its sums, 0.9 for the fragments, 0.4 for the last products.  The first step's B and
// base are on their way before the barrier.  32 clusters (16 of one CTA an SM) start at
// once; of 38 the last ones wait for the first (8.5 us).  The cluster's barrier is the
// hardware's and has no time limit; every thread of a cluster, whose CTAs start together,
// comes to both of its phases, whatever the plan holds.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "lora.cuh"

namespace fp8hg {
namespace lora {

namespace {

constexpr int kCluster = 8, kThreads = 256, kWarps = kCluster * kThreads / 32;

template <int RP, bool F32>
struct Shape {
    static constexpr int KS = RP / 16, PARTS = F32 ? 3 : 2;
    static constexpr int CTAS = RP <= 64 ? 2 : 1;
    static constexpr int AHEAD = RP <= 16 ? 4 : RP <= 32 ? 2 : 1;      // pieces of the long side in flight, a warp
    // strides that meet no bank twice: of a warp's sums, stored two a lane, and of the
    // rows, read four a lane
    static constexpr int SUMS = RP + 8, ROWS = RP + 4;
    static constexpr int SMEM = (kFewTokens * (RP + ROWS) + 8 * 16 * SUMS) * 4;
};

template <int RP, bool F32>
__global__ void __launch_bounds__(kThreads, Shape<RP, F32>::CTAS) k_lora_few(const FewArgs a) {
    using S = Shape<RP, F32>;
    constexpr int KS = S::KS;
    extern __shared__ float4 few_smem[];
    __shared__ int4 tiles[kFewTokens];
    __shared__ int order[kFewTokens], ranks[kFewTokens], count;
    __shared__ float scales[kFewTokens];
    float *part = reinterpret_cast<float *>(few_smem);      // [tokens of the run's tiles][RP], of this CTA
    float *rows = part + kFewTokens * RP;                   // of the cluster, [..][ROWS]
    float *sums = rows + kFewTokens * S::ROWS;              // [8 warps][16][SUMS]
    ptx::grid_begin(static_cast<int64_t>(a.plan.tokens) * (static_cast<int64_t>(a.lw.n) + a.lw.k));
    const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int cta = static_cast<int>(ptx::cluster_ctarank()), warp = cta * 8 + tid / 32, k = a.lw.k, n = a.lw.n;
    const uint32_t clusters = gridDim.x / kCluster, cluster = blockIdx.x / kCluster, steps = (n + 15) / 16;
    // the plan, all of it at once, and what it points to
    if (tid < kFewTokens) {
        const int all = a.plan.words[0];
        const int4 tile = tid < a.plan.max_tiles() ? reinterpret_cast<const int4 *>(a.plan.words + a.plan.tiles())[tid] : make_int4(-1, 0, 0, 0);
        order[tid] = tid < a.plan.tokens ? a.plan.words[a.plan.order() + tid] : -1;
        tiles[tid] = tile;
        if (tid == 0) count = all;
    }
    __syncthreads();
    if (tid < count) {
        const int adapter = tiles[tid].x;
        ranks[tid] = adapter < 0 ? 0 : rank_of(a.lw, adapter);
        scales[tid] = adapter < 0 ? 0.0f : a.lw.scale == nullptr ? 1.0f : a.lw.scale[adapter];
    }
    // at most 64 tiles of 2^20 steps, and 32 clusters
    const uint32_t total = static_cast<uint32_t>(count) * steps;
    const uint32_t begin = total * cluster / clusters, end = total * (cluster + 1) / clusters;

    int slot = 0;
    for (uint32_t at = begin; at < end; at = (at / steps + 1) * steps) {
        const int4 tile = tiles[at / steps];      // adapter, first, count
        if (tile.x < 0) continue;
        const uint16_t *w = a.lw.a + tile.x * a.lw.stride_a;
        for (int m0 = 0; m0 < tile.z; m0 += 16) {
            const uint16_t *x[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int m = m0 + i * 8 + g;
                x[i] = m < tile.z ? a.x + row_at(order[tile.y + m], a.ld_x) : nullptr;
            }
            float acc[RP / 8][4];
#pragma unroll
            for (int j = 0; j < RP / 8; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
            for (int u0 = warp; u0 * 32 < k; u0 += kWarps * S::AHEAD) {
                uint4 xv[S::AHEAD][2], wv[S::AHEAD][RP / 8];
#pragma unroll
                for (int h = 0; h < S::AHEAD; ++h) {
                    const int c = (u0 + h * kWarps) * 32 + t * 8;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        xv[h][i] = make_uint4(0u, 0u, 0u, 0u);
                        if (c < k && x[i] != nullptr) xv[h][i] = ptx::ld_v4(x[i] + c);
                    }
#pragma unroll
                    for (int j = 0; j < RP / 8; ++j) {
                        wv[h][j] = make_uint4(0u, 0u, 0u, 0u);
                        // past the rank: nobody reads those sums
                        if (c < k && j * 8 + g < a.lw.r) wv[h][j] = ptx::ld_v4(w + row_at(j * 8 + g, a.lw.ld_a) + c);
                    }
                }
#pragma unroll
                for (int h = 0; h < S::AHEAD; ++h) {
                    const uint32_t lo[4] = {xv[h][0].x, xv[h][1].x, xv[h][0].y, xv[h][1].y};
                    const uint32_t hi[4] = {xv[h][0].z, xv[h][1].z, xv[h][0].w, xv[h][1].w};
#pragma unroll
                    for (int j = 0; j < RP / 8; ++j) ptx::mma_bf16(acc[j], lo, wv[h][j].x, wv[h][j].y);
#pragma unroll
                    for (int j = 0; j < RP / 8; ++j) ptx::mma_bf16(acc[j], hi, wv[h][j].z, wv[h][j].w);
                }
            }
            float *to = sums + (tid / 32 * 16 + g) * S::SUMS + 2 * t;
#pragma unroll
            for (int j = 0; j < RP / 8; ++j) {
                *reinterpret_cast<float2 *>(to + j * 8) = make_float2(acc[j][0], acc[j][1]);
                *reinterpret_cast<float2 *>(to + 8 * S::SUMS + j * 8) = make_float2(acc[j][2], acc[j][3]);
            }
            __syncthreads();
            for (int i = tid; i < min(16, tile.z - m0) * RP; i += kThreads) {
                float s = 0.0f;
#pragma unroll
                for (int q = 0; q < 8; ++q) s += sums[(q * 16 + i / RP) * S::SUMS + i % RP];
                part[(slot + m0) * RP + i] = s;
            }
            __syncthreads();
        }
        slot += tile.z;
    }
    // a run's part in a tile; a step's fragments of B and values of base, asked for a
    // step ahead, the first one's before the cluster's sums are there
    struct Run {
        int tile, first, last, rank, token[2];
        const uint16_t *w;
    };
    auto run_at = [&](uint32_t at, int m0) {
        Run q;
        q.tile = static_cast<int>(at / steps);
        q.first = static_cast<int>(at % steps);
        q.last = min(static_cast<int>(end - at), static_cast<int>(steps) - q.first) + q.first;
        const int4 tile = tiles[q.tile];
        q.rank = ranks[q.tile];
        q.w = q.rank == 0 ? nullptr : a.lw.b + tile.x * a.lw.stride_b;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int m = m0 + i * 8 + g;
            q.token[i] = m < tile.z ? order[tile.y + m] : -1;
        }
        return q;
    };
    // the lane's pairs of r, eight neighbours' at a time (four's with one product)
    auto pair = [&](int e) { return KS == 1 ? 4 * t + 2 * e : e / 4 * 32 + 8 * t + e % 4 * 2; };
    struct Step {
        uint32_t b[2][2 * KS];
        uint4 base[2];
    };
    auto load = [&](const Run &run, int s) {
        Step q;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int col = s * 16 + 4 * (g >> 1) + 2 * j + (g & 1);
            const uint16_t *row = run.w + row_at(col, a.lw.ld_b);
#pragma unroll
            for (int e = 0; e < 2 * KS; ++e) q.b[j][e] = 0u;
            if (s < run.last && col < n) {
                if constexpr (KS == 1) {
                    if (pair(0) < run.rank) {
                        const uint2 u = ptx::ld_v2(row + pair(0));
                        q.b[j][0] = u.x, q.b[j][1] = u.y;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 2 * KS; e += 4) {
                        if (pair(e) < run.rank) {
                            const uint4 u = ptx::ld_v4(row + pair(e));
                            q.b[j][e] = u.x, q.b[j][e + 1] = u.y, q.b[j][e + 2] = u.z, q.b[j][e + 3] = u.w;
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            q.base[i] = make_uint4(0u, 0u, 0u, 0u);
            const int c = s * 16 + 4 * t;
            if (s < run.last && c < n && run.token[i] >= 0 && a.base != nullptr) {
                const int64_t from = row_at(run.token[i], a.ld_base) + c;
                if constexpr (F32) {
                    q.base[i] = ptx::ld_v4(static_cast<const float *>(a.base) + from);
                } else {
                    const uint2 u = ptx::ld_v2(static_cast<const uint16_t *>(a.base) + from);
                    q.base[i].x = u.x, q.base[i].y = u.y;
                }
            }
        }
        return q;
    };
    __syncthreads();
    ptx::cluster_arrive();
    Step next;
    if (begin < end) {
        const Run run = run_at(begin, 0);
        next = load(run, run.first + warp);
    }
    __syncwarp();
    ptx::cluster_wait();
    for (int i = tid; i < slot * RP; i += kThreads) {
        float v[kCluster], s = 0.0f;
#pragma unroll
        for (int q = 0; q < kCluster; ++q) v[q] = ptx::ld_cluster_f32(ptx::map_shared_rank(ptx::smem_u32(part + i), q));
#pragma unroll
        for (int q = 0; q < kCluster; ++q) s += v[q];
        rows[i / RP * S::ROWS + i % RP] = s;
    }
    __syncthreads();
    ptx::cluster_arrive();      // the others' shares are read

    slot = 0;
    for (uint32_t at = begin; at < end;) {
        const int tokens = tiles[at / steps].z, adapter = tiles[at / steps].x;
        uint32_t after = at;
        for (int m0 = 0; m0 < tokens; m0 += 16) {
            const Run run = run_at(at, m0);
            const int rank = run.rank;
            const float scale = scales[run.tile];
            after = at + (run.last - run.first);
            uint32_t f[S::PARTS][KS][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float *row = rows + (slot + m0 + i * 8 + g) * S::ROWS;
                const bool in = run.token[i] >= 0 && rank > 0;
                const bool keep = run.token[i] >= 0 && a.v_out != nullptr && run.first == 0 && warp == 0;
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int e = 0; e < 2 * KS; ++e) {
                    const int r = pair(e);
                    if (e % 2 == 0 && in) v = *reinterpret_cast<const float4 *>(row + r);
                    const float v0 = r < rank ? (e % 2 ? v.z : v.x) : 0.0f, v1 = r + 1 < rank ? (e % 2 ? v.w : v.y) : 0.0f;
                    if (keep && r < a.lw.r) {
                        float *to = a.v_out + row_at(run.token[i], a.ld_v) + r;
                        to[0] = v0;
                        to[1] = v1;
                    }
                    uint32_t lo[S::PARTS], hi[S::PARTS];
                    lora::split<S::PARTS>(v0 * scale, lo);
                    lora::split<S::PARTS>(v1 * scale, hi);
#pragma unroll
                    for (int p = 0; p < S::PARTS; ++p) f[p][e >> 1][i + 2 * (e & 1)] = lo[p] | hi[p] << 16;
                }
            }
            if (m0 > 0 || at != begin) next = load(run, run.first + warp);
            for (int s = run.first + warp; s < run.last; s += kWarps) {
                Step q = next;
                next = load(run, s + kWarps);
                if (rank < RP) {      // what lies past the rank is not used
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 2 * KS; ++e) {
                            const int r = pair(e);
                            q.b[j][e] = r + 1 < rank ? q.b[j][e] : r < rank ? q.b[j][e] & 0xFFFFu : 0u;
                        }
                }
                float acc[2][4];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const F2 o = f2_bf16(j == 0 ? q.base[i].x : q.base[i].y);
                        acc[j][2 * i] = F32 ? 0.0f : o.lo();
                        acc[j][2 * i + 1] = F32 ? 0.0f : o.hi();
                    }
                if (rank > 0) {
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                        for (int p = 0; p < S::PARTS; ++p)
#pragma unroll
                            for (int j = 0; j < 2; ++j) ptx::mma_bf16(acc[j], f[p][ks], q.b[j][2 * ks], q.b[j][2 * ks + 1]);
                }
                const int c = s * 16 + 4 * t;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (run.token[i] < 0 || c >= n) continue;
                    const int64_t to = row_at(run.token[i], a.ld_y) + c;
                    if constexpr (F32) {
                        *reinterpret_cast<float4 *>(static_cast<float *>(a.y) + to) =
                            make_float4(__uint_as_float(q.base[i].x) + acc[0][2 * i], __uint_as_float(q.base[i].y) + acc[0][2 * i + 1],
                                        __uint_as_float(q.base[i].z) + acc[1][2 * i], __uint_as_float(q.base[i].w) + acc[1][2 * i + 1]);
                    } else {
                        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.y) + to) =
                            make_uint2(ptx::cvt_bf16x2(acc[0][2 * i], acc[0][2 * i + 1]), ptx::cvt_bf16x2(acc[1][2 * i], acc[1][2 * i + 1]));
                    }
                }
            }
        }
        if (adapter >= 0) slot += tokens;
        at = after;
    }
    __syncwarp();
    ptx::cluster_wait();
}

template <int RP, bool F32>
cudaError_t run(const FewArgs &a, cudaStream_t stream) {
    using S = Shape<RP, F32>;
    static unsigned long long done;
    const cudaError_t e = with_smem(&k_lora_few<RP, F32>, S::SMEM, S::SMEM, done);
    if (e != cudaSuccess) return e;
    return launch_after(&k_lora_few<RP, F32>, dim3(16 * kCluster * S::CTAS), kThreads, S::SMEM, stream, kCluster, a);
}
template <bool F32>
cudaError_t by_rank(const FewArgs &a, cudaStream_t stream) {
    switch (padded(a.lw.r)) {
        case 16: return run<16, F32>(a, stream);
        case 32: return run<32, F32>(a, stream);
        case 64: return run<64, F32>(a, stream);
        default: return run<128, F32>(a, stream);
    }
}

}  // namespace

// Up to 16 tokens (18944 x 3584, r 16, one token: 13.6 us a call, with two kernels 17.1;
// on the GPU 8.3 and 10.3 as a graph of it), or up to 64 with adapters for a quarter of
// them (8960 x 1536, r 64, 48 tokens of 24 adapters: 15.0 and 22.3; 18944 x 3584, r 16, 64
// of 64: 21 and 39): every 16 tokens of one adapter read its rows again (64 of one: 31
// and 19).  The long side is one that leaves a warp's sums short, 48 of 16.
bool few(const FewArgs &a, bool f32) {
    const uintptr_t four = f32 ? 16 : 8;
    return (a.plan.tokens <= 16 || (a.plan.tokens <= kFewTokens && a.plan.tokens <= 4 * a.plan.adapters)) && a.lw.k <= 24 * 32 * kWarps &&
           a.lw.r % 8 == 0 && a.lw.k % 8 == 0 && a.lw.n % 4 == 0 && aligned_to(a.x, 16) && a.ld_x % 8 == 0 &&
           aligned_to(a.lw.a, 16) && a.lw.ld_a % 8 == 0 && a.lw.stride_a % 8 == 0 && aligned_to(a.lw.b, 16) && a.lw.ld_b % 8 == 0 &&
           a.lw.stride_b % 8 == 0 && aligned_to(a.y, four) && a.ld_y % 4 == 0 && aligned_to(a.base, four) && a.ld_base % 4 == 0;
}

cudaError_t launch_few(const FewArgs &a, bool f32, cudaStream_t stream) { return f32 ? by_rank<true>(a, stream) : by_rank<false>(a, stream); }

}  // namespace lora
}  // namespace fp8hg
