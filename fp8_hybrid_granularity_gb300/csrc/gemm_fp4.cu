// Product of two 4-bit tensors on the 5th-generation tensor cores (tcgen05).
//
//   C[M, N] (+)= tA tB sum_k a[i, k] sa[i, k / B] b[j, k] sb[j, k / B]
//
// Every 64 elements of K are one tcgen05.mma: kind::mxf4 (UE8M0 scale per 32)
// or kind::mxf4nvf4 (E4M3 scale per 16), which multiplies the block scales in
// while it accumulates in FP32 in tensor memory.  Such an MMA takes the same
// operand bytes and the same cycles as an FP8 one of 32 elements, so the
// arithmetic runs at twice the FP8 rate and everything around it (operand
// bytes, issue, scales: two or four bytes per row and MMA) has to keep up.
//
// Operands: 128-byte rows (256 elements) by TMA, 128-byte swizzle; the scale
// bytes of 128 rows and 256 elements lie contiguous in memory in the order
// tcgen05.cp wants them (two or four tiles of 512 bytes), so a stage takes
// them with one bulk copy per 128 rows, and a scale warp moves each tile to
// tensor memory with one tcgen05.cp.  The scale warp is not the MMA's: a copy
// costs its issuing thread about as much as an MMA, and NV has two copies per
// MMA.
//
// Ragged sizes need no code in the main loop: TMA fills what lies past the
// tensor with zeros, the scale padding along K holds zeros, and rows past the
// last only reach outputs that are not stored.
//
//  k_fp4_wide   tiles of 256 x 192 (two accumulators that share each B tile),
//               persistent, one CTA per SM.
//  k_fp4_few    few rows on one side: tiles of 128 x 16 .. 128, K split over
//               the CTAs of a cluster.
//
// Every wait is bounded; when one runs out the kernel records a timeout in the
// device error word, waits (bounded) for its copies and MMAs in flight, frees
// tensor memory and returns.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>
#include <mutex>

#include "fp4_math.cuh"
#include "gemm_common.cuh"
#include "lowbit.h"

namespace fp8hg {

namespace {

using gemm_common::desc_sw128;
using gemm_common::tile_coords;
using gemm_common::wait_phase;
enum { WHO_PRODUCER = 1, WHO_MMA = 2, WHO_SCALES = 3, WHO_EPILOGUE = 4 };

constexpr int kStageBytes = 128;   // of one row: 256 elements

struct Params {
    int M, N, nk;                  // P rows (MMA's M side), Q rows (N side), K stages
    int num_mb, num_nb, num_tiles;
    const uint8_t *sa, *sb;
    int64_t scale_tiles;           // 512-byte tiles per 128 rows
    const float *ta, *tb;
    void *c;
    int64_t sm, sn;                // C's strides along P and Q, elements
    int out_fp32, accumulate, inject;
    int splits;
    uint64_t wait_limit_ns;
    unsigned int *err;
};

// Descriptor of a 32-row x 16-byte scale tile (no swizzle, 8-row core
// matrices of 128 contiguous bytes).
__device__ __forceinline__ uint64_t desc_scales(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(128 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    return d;
}

// Shared and tensor memory of a kernel with MH accumulators of 128 rows by BN
// columns, S operand stages and SLOTS scale slots in tensor memory (each freed
// by the stage that used it, so SLOTS <= S).
template <bool NV, int MH, int BN, int S, int SLOTS>
struct Layout {
    static constexpr int NG = NV ? 4 : 2;               // scale tiles per stage and 128 rows
    static constexpr uint32_t SF = NG * 512;            // their bytes
    static constexpr int NB = BN > 128 ? 2 : 1;         // 128-row scale tiles of B
    static constexpr uint32_t A = MH * 128 * kStageBytes, B = BN * kStageBytes;
    static constexpr uint32_t STAGE = A + B;
    static constexpr uint32_t OFF_SF = S * STAGE;
    static constexpr uint32_t SF_STAGE = (MH + NB) * SF;
    static constexpr uint32_t OFF_BAR = OFF_SF + S * SF_STAGE;
    // barriers: full[S], empty[S], scales[SLOTS], tfull, tempty, drain, drain2
    static constexpr uint32_t BAR_EMPTY = 8 * S, BAR_SF = 16 * S, BAR_TFULL = 16 * S + 8 * SLOTS;
    static constexpr uint32_t OFF_MISC = OFF_BAR + 256;
    static_assert(BAR_TFULL + 32 <= 256, "barriers");
    static_assert(OFF_MISC + 1040 <= 232448, "shared memory");
    static constexpr uint32_t COL_SF = MH * BN;         // first scale column
    static constexpr uint32_t COLS = (MH * 4 + NB * 4) * NG;
    static_assert(SLOTS <= S, "a slot is freed by its stage's barrier");
    static_assert(COL_SF + SLOTS * COLS <= 512, "tensor memory");
};

// The four (or fewer) MMAs per accumulator of one stage.
template <bool NV, int MH, int BN, class L>
__device__ __forceinline__ void issue_stage(uint32_t tmem, uint32_t slot_col, uint32_t b_shift,
                                            uint32_t s_a, uint32_t s_b, uint32_t idesc, bool first) {
    const uint64_t bd = desc_sw128(s_b);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int g = NV ? j : j >> 1;
        const uint32_t id = idesc | (NV ? 0u : ((j & 1) * 2u << 29) | ((j & 1) * 2u << 4));
        const uint32_t sfb = slot_col + g * (L::NB * 4) + b_shift;
#pragma unroll
        for (int h = 0; h < MH; ++h) {
            const uint64_t ad = desc_sw128(s_a + h * 128 * kStageBytes);
            const uint32_t sfa = slot_col + L::NG * L::NB * 4 + (h * L::NG + g) * 4;
            const uint32_t acc = first && j == 0 ? 0u : 1u;
            if constexpr (NV) ptx::tc_mma_nvf4(tmem + h * BN, ad + 2 * j, bd + 2 * j, id, sfa, sfb, acc);
            else ptx::tc_mma_mxf4(tmem + h * BN, ad + 2 * j, bd + 2 * j, id, sfa, sfb, acc);
        }
    }
}

// ---------------------------------------------------------------- wide tiles
constexpr int WM = 256, WN = 192, W_THREADS = 384;
constexpr uint32_t EPI_BYTES = 4096;           // staging per epilogue warp
template <bool NV>
using WideLayout = Layout<NV, 2, WN, 3, NV ? 2 : 3>;
template <bool NV>
constexpr uint32_t wide_smem = WideLayout<NV>::OFF_MISC + 16 + 8 * EPI_BYTES + 1024;

// 32 rows x 128 bytes through a warp's staging area, lane l holding row l's
// 128 bytes (16-byte pieces XOR-swizzled by row).
__device__ __forceinline__ void stage_row(uint8_t *stage, int lane, const uint32_t *w) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint4 *>(stage + lane * 128 + ((c ^ (lane & 7)) << 4)) =
            make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
}
__device__ __forceinline__ uint4 staged(const uint8_t *stage, int r, int c) {
    return *reinterpret_cast<const uint4 *>(stage + r * 128 + ((c ^ (r & 7)) << 4));
}

// The staged piece as 64 BF16 columns of C from (row0, col0).
__device__ __forceinline__ void write_bf16(const uint8_t *stage, int lane, const Params &p,
                                           int64_t row0, int64_t col0, bool vec) {
    uint16_t *c = static_cast<uint16_t *>(p.c);
    if (vec && col0 + 64 <= p.N) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int idx = i * 32 + lane, r = idx >> 3, q = idx & 7;
            if (row0 + r < p.M)
                *reinterpret_cast<uint4 *>(c + (row0 + r) * p.sm + col0 + q * 8) = staged(stage, r, q);
        }
    } else {
        // two neighbouring columns per lane, row by row
        const int64_t col = col0 + 2 * lane;
        for (int r = 0; r < 32 && row0 + r < p.M; ++r) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(
                stage + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
            uint16_t *d = c + (row0 + r) * p.sm + col;
            if (col < p.N) d[0] = static_cast<uint16_t>(w);
            if (col + 1 < p.N) d[1] = static_cast<uint16_t>(w >> 16);
        }
    }
}

// The staged piece as 32 FP32 values per row from (row0, col0): FP32 output,
// or an output that is read and added to first (one rounding).
__device__ __forceinline__ void write_f32(const uint8_t *stage, int lane, const Params &p,
                                          int64_t row0, int64_t col0, bool vec) {
    if (p.out_fp32 && vec && col0 + 32 <= p.N) {
        float *c = static_cast<float *>(p.c);
#pragma unroll 4
        for (int i = 0; i < 8; ++i) {
            const int idx = i * 32 + lane, r = idx >> 3, q = idx & 7;
            if (row0 + r >= p.M) continue;
            float4 *d = reinterpret_cast<float4 *>(c + (row0 + r) * p.sm + col0 + q * 4);
            const uint4 w = staged(stage, r, q);
            float4 v = make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z),
                                   __uint_as_float(w.w));
            if (p.accumulate) {
                const float4 o = *d;
                v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
            }
            *d = v;
        }
        return;
    }
    const int64_t col = col0 + lane;
    if (col >= p.N) return;
#pragma unroll 4
    for (int r = 0; r < 32; ++r) {
        if (row0 + r >= p.M) break;
        float v = *reinterpret_cast<const float *>(stage + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) +
                                                   (lane & 3) * 4);
        const int64_t at = (row0 + r) * p.sm + col;
        if (p.out_fp32) {
            float *c = static_cast<float *>(p.c) + at;
            *c = p.accumulate ? *c + v : v;
        } else {
            uint16_t *c = static_cast<uint16_t *>(p.c) + at;
            if (p.accumulate) v += __uint_as_float(static_cast<uint32_t>(*c) << 16);
            *c = static_cast<uint16_t>(ptx::cvt_bf16x2(v, 0.0f));
        }
    }
}

template <bool NV>
__global__ void __launch_bounds__(W_THREADS, 1)
    k_fp4_wide(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
               const Params p, const uint32_t idesc) {
    using L = WideLayout<NV>;
    constexpr int S = 3, SLOTS = NV ? 2 : 3;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    const uint32_t bar = base + L::OFF_BAR;
    const uint32_t tfull = bar + L::BAR_TFULL, tempty = tfull + 8, drain = tfull + 16, drain2 = tfull + 24;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + L::OFF_MISC);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(gbase + L::OFF_MISC + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t limit = p.wait_limit_ns, drain_limit = 2000000ull;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(bar + 8 * s, 1);                  // bytes landed
            ptx::mbar_init(bar + L::BAR_EMPTY + 8 * s, 1);   // the stage's MMAs are done
        }
        for (int i = 0; i < SLOTS; ++i) ptx::mbar_init(bar + L::BAR_SF + 8 * i, 1);
        ptx::mbar_init(tfull, 1);
        ptx::mbar_init(tempty, 256);
        ptx::mbar_init(drain, 1);
        ptx::mbar_init(drain2, 1);
        *abort_flag = 0u;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&tmap_a);
        ptx::prefetch_tmap(&tmap_b);
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ---------------------------------------------------------- producer
        uint32_t it = 0;
        bool ok = true;
        const int rta = (p.M + 127) / 128, rtb = (p.N + 127) / 128;   // row tiles of scales
        for (int tile = blockIdx.x; tile < p.num_tiles && ok; tile += gridDim.x) {
            int mb, nb;
            tile_coords(tile, p.num_mb, p.num_nb, mb, nb);
            const int ra = mb * 2, rb = nb * WN / 128;
            const int na = min(2, rta - ra), nbt = min(2, rtb - rb);
            const uint32_t bytes = L::STAGE + (na + nbt) * L::SF;
            const uint8_t *ga = p.sa + static_cast<int64_t>(ra) * p.scale_tiles * 512;
            const uint8_t *gb = p.sb + static_cast<int64_t>(rb) * p.scale_tiles * 512;
            for (int kb = 0; kb < p.nk; ++kb) {
                const uint32_t s = it % S, ph = (it / S) & 1u;
                ok = wait_phase(bar + L::BAR_EMPTY + 8 * s, ph ^ 1u, limit, abort_flag, p.err, WHO_PRODUCER);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                // inject = 1 (a test of the timeout path): the first CTA
                // never issues its first stage
                if (lane == 0 && !(p.inject == 1 && blockIdx.x == 0 && it == 0)) {
                    const uint32_t full = bar + 8 * s, sa = base + s * L::STAGE;
                    const uint32_t sf = base + L::OFF_SF + s * L::SF_STAGE;
                    ptx::mbar_arrive_expect_tx(full, bytes);
                    ptx::tma_load_2d(sa, &tmap_a, full, kb * kStageBytes, mb * WM);
                    ptx::tma_load_2d(sa + L::A, &tmap_b, full, kb * kStageBytes, nb * WN);
                    const int64_t at = static_cast<int64_t>(kb) * L::SF, rt = p.scale_tiles * 512;
                    for (int i = 0; i < na; ++i) ptx::bulk_load(sf + i * L::SF, ga + at + i * rt, L::SF, full);
                    for (int i = 0; i < nbt; ++i)
                        ptx::bulk_load(sf + (2 + i) * L::SF, gb + at + i * rt, L::SF, full);
                }
                __syncwarp();
                ++it;
            }
        }
        // the copies in flight land before the CTA ends
        const uint32_t nd = it < S ? it : S;
        for (uint32_t i = it - nd; i < it; ++i)
            wait_phase(bar + 8 * (i % S), (i / S) & 1u, drain_limit, abort_flag, p.err, WHO_PRODUCER, false);
    } else if (warp == 1) {
        // -------------------------------------------------------- MMA issuer
        uint32_t it = 0, tcount = 0;
        bool ok = true;
        for (int tile = blockIdx.x; tile < p.num_tiles && ok; tile += gridDim.x) {
            int mb, nb;
            tile_coords(tile, p.num_mb, p.num_nb, mb, nb);
            const uint32_t b_shift = (nb * WN % 128) / 32;
            ok = wait_phase(tempty, (tcount & 1u) ^ 1u, limit, abort_flag, p.err, WHO_MMA);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            ptx::tc_fence_after();
            for (int kb = 0; kb < p.nk; ++kb) {
                const uint32_t s = it % S, slot = it % SLOTS;
                ok = wait_phase(bar + 8 * s, (it / S) & 1u, limit, abort_flag, p.err, WHO_MMA) &&
                     wait_phase(bar + L::BAR_SF + 8 * slot, (it / SLOTS) & 1u, limit, abort_flag, p.err, WHO_MMA);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                ptx::tc_fence_after();
                if (lane == 0) {
                    const uint32_t sa = base + s * L::STAGE;
                    issue_stage<NV, 2, WN, L>(tmem, tmem + L::COL_SF + slot * L::COLS, b_shift, sa, sa + L::A,
                                              idesc, kb == 0);
                    ptx::tc_commit(bar + L::BAR_EMPTY + 8 * s);
                }
                __syncwarp();
                ++it;
            }
            if (!ok) break;
            if (lane == 0) ptx::tc_commit(tfull);
            __syncwarp();
            ++tcount;
        }
        if (lane == 0) ptx::tc_commit(drain);
        __syncwarp();
        wait_phase(drain, 0u, drain_limit, abort_flag, p.err, WHO_MMA, false);
    } else if (warp == 2) {
        // ------------------------------------------- scales to tensor memory
        uint32_t it = 0;
        bool ok = true;
        for (int tile = blockIdx.x; tile < p.num_tiles && ok; tile += gridDim.x) {
            for (int kb = 0; kb < p.nk; ++kb) {
                const uint32_t s = it % S, slot = it % SLOTS;
                ok = wait_phase(bar + 8 * s, (it / S) & 1u, limit, abort_flag, p.err, WHO_SCALES);
                if (ok && it >= SLOTS) {
                    // the slot is free when the MMAs of stage it - SLOTS are done
                    const uint32_t u = it - SLOTS;
                    ok = wait_phase(bar + L::BAR_EMPTY + 8 * (u % S), (u / S) & 1u, limit, abort_flag, p.err,
                                    WHO_SCALES);
                }
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                ptx::tc_fence_after();
                if (lane == 0) {
                    const uint32_t sf = base + L::OFF_SF + s * L::SF_STAGE;
                    const uint32_t col = tmem + L::COL_SF + slot * L::COLS;
#pragma unroll
                    for (int g = 0; g < L::NG; ++g) {
                        for (int i = 0; i < 2; ++i)
                            ptx::tc_cp_32x128b_warpx4(col + g * 8 + i * 4,
                                                      desc_scales(sf + (2 + i) * L::SF + g * 512));
                        for (int h = 0; h < 2; ++h)
                            ptx::tc_cp_32x128b_warpx4(col + L::NG * 8 + (h * L::NG + g) * 4,
                                                      desc_scales(sf + h * L::SF + g * 512));
                    }
                    ptx::tc_commit(bar + L::BAR_SF + 8 * slot);
                }
                __syncwarp();
                ++it;
            }
        }
        if (lane == 0) ptx::tc_commit(drain2);
        __syncwarp();
        wait_phase(drain2, 0u, drain_limit, abort_flag, p.err, WHO_SCALES, false);
    } else if (warp >= 4) {
        // ---------------------------------------------------------- epilogue
        const int q = warp & 3, half = (warp - 4) >> 2;
        uint8_t *stage = gbase + L::OFF_MISC + 16 + (warp - 4) * EPI_BYTES;
        const float alpha = (p.ta ? __ldg(p.ta) : 1.0f) * (p.tb ? __ldg(p.tb) : 1.0f);
        const bool vec = (reinterpret_cast<uintptr_t>(p.c) & 15) == 0 && p.sm % (p.out_fp32 ? 4 : 8) == 0;
        uint32_t tcount = 0;
        for (int tile = blockIdx.x; tile < p.num_tiles; tile += gridDim.x, ++tcount) {
            int mb, nb;
            tile_coords(tile, p.num_mb, p.num_nb, mb, nb);
            bool ok = wait_phase(tfull, tcount & 1u, limit, abort_flag, p.err, WHO_EPILOGUE);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            ptx::tc_fence_after();
            const int64_t row0 = static_cast<int64_t>(mb) * WM + half * 128 + q * 32;
            const int64_t col0 = static_cast<int64_t>(nb) * WN;
            const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + half * WN;
            if (p.out_fp32 || p.accumulate) {
#pragma unroll 1
                for (int chunk = 0; chunk < WN / 32; ++chunk) {
                    uint32_t r[32];
                    ptx::tmem_ld_32x32b_x32(taddr + chunk * 32, r);
                    ptx::tmem_wait_ld();
                    if (chunk == WN / 32 - 1) {
                        ptx::tc_fence_before();
                        ptx::mbar_arrive(tempty);
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
                    stage_row(stage, lane, r);
                    __syncwarp();
                    write_f32(stage, lane, p, row0, col0 + chunk * 32, vec);
                    __syncwarp();
                }
                continue;
            }
            uint32_t packed[WN / 2];
#pragma unroll
            for (int chunk = 0; chunk < WN / 32; ++chunk) {
                uint32_t r[32];
                ptx::tmem_ld_32x32b_x32(taddr + chunk * 32, r);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    packed[chunk * 16 + e] = ptx::cvt_bf16x2(__uint_as_float(r[2 * e]) * alpha,
                                                             __uint_as_float(r[2 * e + 1]) * alpha);
            }
            ptx::tc_fence_before();
            ptx::mbar_arrive(tempty);
#pragma unroll
            for (int piece = 0; piece < WN / 64; ++piece) {
                stage_row(stage, lane, packed + piece * 32);
                __syncwarp();
                write_bf16(stage, lane, p, row0, col0 + piece * 64, vec);
                __syncwarp();
            }
        }
    }

    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ few rows
// P (128 rows per CTA, the MMA's M side) times Q (BN rows): with few tokens P
// is the weights and Q the tokens, so that a token costs no row of a 128-row
// tile.  The CTAs of a cluster take consecutive parts of K; each leaves its
// FP32 partial tile in its own shared memory, and after a cluster barrier
// adds up a slice of the columns from all of them, in the order of the parts
// (the same bits every time), and stores it.
constexpr int F_THREADS = 256;
template <int BN>
constexpr int few_stages = BN <= 32 ? 8 : BN == 64 ? 6 : 5;
template <bool NV, int BN>
using FewLayout = Layout<NV, 1, BN, few_stages<BN>, 4>;
template <bool NV, int BN>
constexpr uint32_t few_smem = FewLayout<NV, BN>::OFF_MISC + 16 + 1024;

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}

template <bool NV, int BN>
__global__ void __launch_bounds__(F_THREADS, 1)
    k_fp4_few(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
              const Params p, const uint32_t idesc) {
    using L = FewLayout<NV, BN>;
    constexpr int S = few_stages<BN>, SLOTS = 4;
    constexpr uint32_t TCOLS = L::COL_SF + SLOTS * L::COLS <= 128 ? 128 : 256;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    const uint32_t bar = base + L::OFF_BAR;
    const uint32_t tfull = bar + L::BAR_TFULL, drain = tfull + 16, drain2 = tfull + 24;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + L::OFF_MISC);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(gbase + L::OFF_MISC + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t limit = p.wait_limit_ns, drain_limit = 2000000ull;
    const int splits = p.splits, part = blockIdx.x % splits, tile = blockIdx.x / splits;
    const int nb = tile % p.num_nb, mb = tile / p.num_nb;
    const int kb0 = static_cast<int>(static_cast<int64_t>(part) * p.nk / splits);
    const int kb1 = static_cast<int>(static_cast<int64_t>(part + 1) * p.nk / splits);
    const int n = kb1 - kb0;                         // at least 1: splits <= nk

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(bar + 8 * s, 1);
            ptx::mbar_init(bar + L::BAR_EMPTY + 8 * s, 1);
        }
        for (int i = 0; i < SLOTS; ++i) ptx::mbar_init(bar + L::BAR_SF + 8 * i, 1);
        ptx::mbar_init(tfull, 1);
        ptx::mbar_init(drain, 1);
        ptx::mbar_init(drain2, 1);
        *abort_flag = 0u;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), TCOLS);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    bool done = true;                                // this thread saw the accumulator complete

    if (warp == 0) {
        const uint8_t *ga = p.sa + static_cast<int64_t>(mb) * p.scale_tiles * 512;
        const uint8_t *gb = p.sb + static_cast<int64_t>(nb) * BN / 128 * p.scale_tiles * 512;
        int it = 0;
        for (; it < n; ++it) {
            const int s = it % S;
            bool ok = wait_phase(bar + L::BAR_EMPTY + 8 * s, ((it / S) & 1u) ^ 1u, limit, abort_flag, p.err,
                                 WHO_PRODUCER);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            if (lane == 0 && !(p.inject == 1 && blockIdx.x == 0 && it == 0)) {
                const uint32_t full = bar + 8 * s, sa = base + s * L::STAGE;
                const uint32_t sf = base + L::OFF_SF + s * L::SF_STAGE;
                const int kb = kb0 + it;
                const int64_t at = static_cast<int64_t>(kb) * L::SF;
                ptx::mbar_arrive_expect_tx(full, L::STAGE + 2 * L::SF);
                ptx::tma_load_2d(sa, &tmap_a, full, kb * kStageBytes, mb * 128);
                ptx::tma_load_2d(sa + L::A, &tmap_b, full, kb * kStageBytes, nb * BN);
                ptx::bulk_load(sf, ga + at, L::SF, full);
                ptx::bulk_load(sf + L::SF, gb + at, L::SF, full);
            }
            __syncwarp();
        }
        for (int i = it > S ? it - S : 0; i < it; ++i)
            wait_phase(bar + 8 * (i % S), (i / S) & 1u, drain_limit, abort_flag, p.err, WHO_PRODUCER, false);
    } else if (warp == 1) {
        const uint32_t b_shift = (nb * BN % 128) / 32;
        bool ok = true;
        for (int it = 0; it < n && ok; ++it) {
            const int s = it % S, slot = it % SLOTS;
            ok = wait_phase(bar + 8 * s, (it / S) & 1u, limit, abort_flag, p.err, WHO_MMA) &&
                 wait_phase(bar + L::BAR_SF + 8 * slot, (it / SLOTS) & 1u, limit, abort_flag, p.err, WHO_MMA);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            ptx::tc_fence_after();
            if (lane == 0) {
                const uint32_t sa = base + s * L::STAGE;
                issue_stage<NV, 1, BN, L>(tmem, tmem + L::COL_SF + slot * L::COLS, b_shift, sa, sa + L::A, idesc,
                                          it == 0);
                ptx::tc_commit(bar + L::BAR_EMPTY + 8 * s);
            }
            __syncwarp();
        }
        if (lane == 0) {
            if (ok) ptx::tc_commit(tfull);
            ptx::tc_commit(drain);
        }
        __syncwarp();
        wait_phase(drain, 0u, drain_limit, abort_flag, p.err, WHO_MMA, false);
    } else if (warp == 2) {
        bool ok = true;
        for (int it = 0; it < n && ok; ++it) {
            const int s = it % S, slot = it % SLOTS;
            ok = wait_phase(bar + 8 * s, (it / S) & 1u, limit, abort_flag, p.err, WHO_SCALES);
            if (ok && it >= SLOTS) {
                const int u = it - SLOTS;
                ok = wait_phase(bar + L::BAR_EMPTY + 8 * (u % S), (u / S) & 1u, limit, abort_flag, p.err,
                                WHO_SCALES);
            }
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            ptx::tc_fence_after();
            if (lane == 0) {
                const uint32_t sf = base + L::OFF_SF + s * L::SF_STAGE;
                const uint32_t col = tmem + L::COL_SF + slot * L::COLS;
#pragma unroll
                for (int g = 0; g < L::NG; ++g) {
                    ptx::tc_cp_32x128b_warpx4(col + g * 4, desc_scales(sf + L::SF + g * 512));
                    ptx::tc_cp_32x128b_warpx4(col + L::NG * 4 + g * 4, desc_scales(sf + g * 512));
                }
                ptx::tc_commit(bar + L::BAR_SF + 8 * slot);
            }
            __syncwarp();
        }
        if (lane == 0) ptx::tc_commit(drain2);
        __syncwarp();
        wait_phase(drain2, 0u, drain_limit, abort_flag, p.err, WHO_SCALES, false);
    } else if (warp >= 4) {
        // the partial tile, column by column of 128 rows, over the operand
        // stages (every copy and MMA is done once tfull completes)
        done = wait_phase(tfull, 0u, limit, abort_flag, p.err, WHO_EPILOGUE);
        done = __all_sync(0xFFFFFFFFu, done);
        if (done) {
            ptx::tc_fence_after();
            float *part_tile = reinterpret_cast<float *>(gbase);
            const int q = warp & 3;
#pragma unroll 1
            for (int c = 0; c < BN; c += 16) {
                uint32_t r[16];
                ptx::tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(q * 32) << 16) + c, r);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) part_tile[(c + i) * 129 + q * 32 + lane] = __uint_as_float(r[i]);
            }
            ptx::tc_fence_before();
        }
    }

    __syncthreads();
    if (splits > 1) ptx::cluster_sync();
    if (!*abort_flag) {
        const float alpha = (p.ta ? __ldg(p.ta) : 1.0f) * (p.tb ? __ldg(p.tb) : 1.0f);
        const int c0 = part * BN / splits, c1 = (part + 1) * BN / splits;
        const int64_t row0 = static_cast<int64_t>(mb) * 128, col0 = static_cast<int64_t>(nb) * BN;
        // consecutive threads along the output's contiguous direction
        const bool along_p = p.sm == 1;
        const int nc = c1 - c0;
        for (int i = threadIdx.x; i < nc * 128; i += F_THREADS) {
            const int r = along_p ? i & 127 : i / nc, c = along_p ? c0 + (i >> 7) : c0 + i % nc;
            if (row0 + r >= p.M || col0 + c >= p.N) continue;
            float v = 0.0f;
            const uint32_t off = (c * 129 + r) * 4;
            if (splits == 1) {
                v = *reinterpret_cast<const float *>(gbase + off);
            } else {
                for (int k = 0; k < splits; ++k) v += ld_cluster_f32(ptx::map_shared_rank(base + off, k));
            }
            v *= alpha;
            const int64_t at = (row0 + r) * p.sm + (col0 + c) * p.sn;
            if (p.out_fp32) {
                float *d = static_cast<float *>(p.c) + at;
                *d = p.accumulate ? *d + v : v;
            } else {
                uint16_t *d = static_cast<uint16_t *>(p.c) + at;
                if (p.accumulate) v += __uint_as_float(static_cast<uint32_t>(*d) << 16);
                *d = static_cast<uint16_t>(ptx::cvt_bf16x2(v, 0.0f));
            }
        }
    }
    // no CTA leaves while another still reads its shared memory
    __syncwarp();
    if (splits > 1) ptx::cluster_sync();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, TCOLS);
    }
}

// ------------------------------------------------------------------- launch
bool make_tmap(CUtensorMap *m, const Fp4Operand &o, uint32_t box_rows) {
    TensorMapEncodeFn enc = tensor_map_encoder();
    if (!enc) return false;
    std::memset(m, 0, sizeof(*m));
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>((o.k + 1) / 2), static_cast<cuuint64_t>(o.rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(o.ld)};
    const cuuint32_t box[2] = {kStageBytes, box_rows}, estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(o.codes), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

std::mutex g_mu;
int g_sms[64] = {0};

template <class K>
cudaError_t allow_smem(K kern, uint32_t bytes) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
}
template <bool NV>
cudaError_t set_attributes() {
    cudaError_t e = allow_smem(k_fp4_wide<NV>, wide_smem<NV>);
    if (e == cudaSuccess) e = allow_smem(k_fp4_few<NV, 16>, few_smem<NV, 16>);
    if (e == cudaSuccess) e = allow_smem(k_fp4_few<NV, 32>, few_smem<NV, 32>);
    if (e == cudaSuccess) e = allow_smem(k_fp4_few<NV, 64>, few_smem<NV, 64>);
    if (e == cudaSuccess) e = allow_smem(k_fp4_few<NV, 128>, few_smem<NV, 128>);
    return e;
}

// Instruction descriptor of the 4-bit kinds: E2M1 (1) for A and B in bits 7-9
// and 10-12, N >> 3 in bits 17-22, the scale type in bit 23 (0: E4M3, 1:
// UE8M0), M >> 4 in bits 24-28; scale-factor ids are added per MMA.
uint32_t instruction(bool nv, int n) {
    return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | ((nv ? 0u : 1u) << 23) |
           (static_cast<uint32_t>(128 >> 4) << 24);
}

template <bool NV, int BN>
cudaError_t launch_few(const CUtensorMap &ta, const CUtensorMap &tb, const Params &p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.num_tiles * p.splits));
    cfg.blockDim = dim3(F_THREADS);
    cfg.dynamicSmemBytes = few_smem<NV, BN>;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(p.splits);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_fp4_few<NV, BN>, ta, tb, p, instruction(NV, BN));
}

template <bool NV>
int launch(const Fp4GemmArgs &g, int sms, cudaStream_t stream) {
    Params p{};
    p.nk = static_cast<int>((g.a.k + 255) / 256);
    p.scale_tiles = fp4_scale_tiles(g.a.k, g.a.kind);
    p.c = g.c;
    p.out_fp32 = g.out_fp32;
    p.accumulate = g.accumulate;
    p.inject = g.inject_fault;
    p.wait_limit_ns = g.wait_limit_ns;
    p.err = g.err;
    p.splits = 1;
    CUtensorMap ta, tb;
    const int64_t wide_tiles = ((g.a.rows + WM - 1) / WM) * ((g.b.rows + WN - 1) / WN);
    if (g.a.rows > 128 && g.b.rows > 128 && 2 * wide_tiles > sms) {
        p.M = static_cast<int>(g.a.rows);
        p.N = static_cast<int>(g.b.rows);
        p.num_mb = (p.M + WM - 1) / WM;
        p.num_nb = (p.N + WN - 1) / WN;
        if (wide_tiles > 0x7FFFFFFF) return 2 + static_cast<int>(cudaErrorInvalidValue);
        p.num_tiles = static_cast<int>(wide_tiles);
        p.sa = g.a.scale;
        p.sb = g.b.scale;
        p.ta = g.a.ts;
        p.tb = g.b.ts;
        p.sm = g.ldc;
        p.sn = 1;
        if (!make_tmap(&ta, g.a, WM) || !make_tmap(&tb, g.b, WN)) return 1;
        const int grid = p.num_tiles < sms ? p.num_tiles : sms;
        k_fp4_wide<NV><<<grid, W_THREADS, wide_smem<NV>, stream>>>(ta, tb, p, instruction(NV, WN));
        const cudaError_t e = cudaGetLastError();
        return e == cudaSuccess ? 0 : 2 + static_cast<int>(e);
    }
    // few rows on one side (or few tiles): that side is Q
    const bool swap = g.a.rows <= g.b.rows;
    const Fp4Operand &P = swap ? g.b : g.a, &Q = swap ? g.a : g.b;
    p.M = static_cast<int>(P.rows);
    p.N = static_cast<int>(Q.rows);
    p.sa = P.scale;
    p.sb = Q.scale;
    p.ta = P.ts;
    p.tb = Q.ts;
    p.sm = swap ? 1 : g.ldc;
    p.sn = swap ? g.ldc : 1;
    const int bn = p.N <= 16 ? 16 : p.N <= 32 ? 32 : p.N <= 64 ? 64 : 128;
    p.num_mb = (p.M + 127) / 128;
    p.num_nb = (p.N + bn - 1) / bn;
    const int64_t tiles = static_cast<int64_t>(p.num_mb) * p.num_nb;
    if (tiles > 0x7FFFFFFF / 8) return 2 + static_cast<int>(cudaErrorInvalidValue);
    p.num_tiles = static_cast<int>(tiles);
    while (p.splits < 8 && p.splits * 2 <= p.nk && tiles * p.splits * 2 <= sms) p.splits *= 2;
    if (!make_tmap(&ta, P, 128) || !make_tmap(&tb, Q, static_cast<uint32_t>(bn))) return 1;
    cudaError_t e;
    switch (bn) {
    case 16: e = launch_few<NV, 16>(ta, tb, p, stream); break;
    case 32: e = launch_few<NV, 32>(ta, tb, p, stream); break;
    case 64: e = launch_few<NV, 64>(ta, tb, p, stream); break;
    default: e = launch_few<NV, 128>(ta, tb, p, stream); break;
    }
    return e == cudaSuccess ? 0 : 2 + static_cast<int>(e);
}

}  // namespace

int launch_fp4_gemm(const Fp4GemmArgs &g, cudaStream_t stream) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) dev = 0;
    {
        std::lock_guard<std::mutex> lock(g_mu);
        if (!g_sms[dev]) {
            cudaError_t e = set_attributes<true>();
            if (e == cudaSuccess) e = set_attributes<false>();
            if (e != cudaSuccess) return 2 + static_cast<int>(e);
            int n = 0;
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
            g_sms[dev] = n > 0 ? n : 1;
        }
    }
    return g.a.kind == FP4_NV ? launch<true>(g, g_sms[dev], stream) : launch<false>(g, g_sms[dev], stream);
}

}  // namespace fp8hg
