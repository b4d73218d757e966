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
//  k_fp4_pair   tiles of 256 x 384 per pair of CTAs, persistent.
//  k_fp4_few    few rows on one side: tiles of 128 x 16 .. 128, K split over
//               the CTAs of a cluster.
//
// Every wait is bounded; when one runs out the kernel records a timeout in the
// device error word, waits (bounded) for its copies and MMAs in flight, frees
// tensor memory and returns.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "fp4_math.cuh"
#include "gemm_common.cuh"
#include "lowbit.h"
#include "ragged.cuh"

namespace fp8hg {

namespace {

using gemm_common::desc_sw128;
using gemm_common::tile_coords;
using gemm_common::wait_phase;
enum { WHO_PRODUCER = 1, WHO_MMA = 2, WHO_SCALES = 3, WHO_EPILOGUE = 4 };

constexpr int kStageBytes = 128;   // of one row: 256 elements

struct Params {
    int M, N, nk;                  // P rows (MMA's M side), Q rows (N side), K stages
    int num_mb, num_nb, num_tiles; // pair tiles: NH parts wide, num_nb columns of them
    int half_tiles;                // and, past the last column, num_mb of one part or none
    const uint8_t *sa, *sb;
    int64_t scale_tiles;           // 512-byte tiles per 128 rows
    const float *ta, *tb;
    void *c;
    int64_t sm, sn;                // C's strides along P and Q, elements
    int out_fp32, accumulate, inject;
    int c_tma;                     // C's rows are written by TMA
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

// ---------------------------------------------------------------- pair tiles
// Tiles of 256 x 192 NH of a pair of CTAs (a cluster of two), tcgen05.mma with
// cta_group::2: per 64 elements of K one M = 256, N = 192 MMA for each of the
// NH column parts.  Each CTA holds its 128 rows of A and, of each column part,
// 96 rows of B; its tensor memory takes its 128 rows of the accumulators.
//
// NH = 2, the large products: a stage (256 elements of K) is 40 KB of operands
// per CTA for 768 cycles of MMAs.  What a 4-bit product runs short of is
// operand bytes: it takes as many per cycle as an FP8 one and reads a stage in
// half the time, and an SM gets about 60 bytes a cycle from L2 here.  Single-CTA
// tiles of 256 x 192 (two accumulators of 128 rows) need 56 KB for the same 768
// cycles.  At 16384 x 3584 x 18944: 380 us with those tiles (MX; NV 447), 296
// (327) with these: 7.5 (6.8) PFLOP/s, for which the GPU draws its power limit
// (a second of it runs at 1.7 (1.9) GHz; with zeros as operands a call takes 12
// (7) % less).
// NH = 1, where NH = 2 leaves pairs without a tile.
// A last column of at most 192 columns is computed as half tiles of an NH = 2
// launch: 8192 x 3584 x 3584 in four rounds of tiles instead of five (NV, at
// the time: 48 us instead of 55).
//
// The ring of operand stages is short (four stages, 1.6 us of MMAs), so
// what counts is how soon a stage is used and free again.  Its scales have
// barriers and a producer of their own and are in tensor memory when it lands:
// with a stage's scales coming with it and copied after it MX 16384 x 3584 x
// 18944 took 10 % longer.  NV has tensor memory for two stages of scales, so the
// second next stage's are copied while the next one's MMAs run, which is just
// too short (with two slots instead of four MX takes as long as NV); see SUB.
//
// At a tile's end the MMAs wait until an accumulator is in the epilogue's
// registers.  The epilogue's warps of both CTAs say so themselves, by a relaxed
// arrival: no memory is handed over, and a releasing one (cluster scope) first
// waits for what its SM has under way, 1300 to 2400 cycles of each tile.  So
// 16384 x 18944 x 3584 takes 357 us instead of 384 (NV), 8192 x 8960 x 1536 54
// instead of 61.
//
// Warps of each CTA: 0 operand producer, 14 scale producer, 4-11 epilogue (a
// 32-row quarter of one column part each); of the even CTA also 1 MMA issuer
// and 2, 3, 12, 13 scale copiers, for both CTAs.  Tensor memory: the
// accumulators, then the scale slots: per 128 (NV: 64) elements of K four
// columns for every 128 rows, B's first.
constexpr int PM = 256, PH = 192, P_THREADS = 512;
constexpr uint32_t EPI_BYTES = 4096;           // staging per epilogue warp
template <bool NV, int NH_>
struct PairLayout {
    static constexpr int NH = NH_, PN = PH * NH;
    static constexpr int NG = NV ? 4 : 2;      // scale tiles per stage and 128 rows
    static constexpr int NB = NH == 2 ? 3 : 2; // 128-row scale tiles that a tile's columns touch
    static constexpr int S = NH == 2 ? 4 : 6;
    static constexpr int SLOTS = NH == 2 && NV ? 2 : NH == 2 ? 4 : S;
    // Parts of a stage's scales that the MMAs wait for separately.  With two slots
    // the copies into one begin when the stage before last is done and are in the
    // way of the next MMAs: in halves 16384 x 3584 x 18944 takes 327 us instead of
    // 338, 8192 x 18944 x 3584 178 instead of 181; the second wait costs the MMA
    // thread some 75 cycles a stage, 3584 x 18944 x 1000 37 us instead of 36.
    static constexpr int SUB = SLOTS == 2 ? 2 : 1;
    static constexpr uint32_t SF = NG * 512;
    static constexpr uint32_t A = 128 * kStageBytes, BH = PH / 2 * kStageBytes;
    static constexpr uint32_t STAGE = A + NH * BH, SF_STAGE = (1 + NB) * SF;   // A's rows, then B's
    static constexpr uint32_t OFF_SF = S * STAGE, OFF_EPI = OFF_SF + S * SF_STAGE;
    static constexpr uint32_t OFF_BAR = OFF_EPI + 4 * NH * EPI_BYTES;
    // barriers: full (even CTA: both CTAs' operands, and their scales in tensor
    // memory), empty (each CTA), sfull (even CTA: both CTAs' scales), scales
    // (each CTA: copied to tensor memory), rest (even CTA: the second half of a
    // stage's scales copied),
    // tfull[2] (each CTA), tempty[2] (even CTA: both CTAs' epilogues), drain[5]
    static constexpr uint32_t EMPTY = 8 * S, SFULL = 16 * S, SCALES = 24 * S, REST = 32 * S, TFULL = 40 * S;
    static constexpr uint32_t TEMPTY = TFULL + 16, DRAIN = TEMPTY + 16;
    static constexpr uint32_t OFF_MISC = OFF_BAR + 320, SMEM = OFF_MISC + 16 + 1024;
    static constexpr uint32_t GC = 4 * (1 + NB), COLS = GC * NG;   // columns of a scale group, of a slot
    static_assert(DRAIN + 40 <= 320 && OFF_EPI % 1024 == 0 && SMEM <= 232448 && PN + SLOTS * COLS <= 512, "");
    static_assert(SLOTS <= S, "a slot is freed by its stage's barrier");
    static_assert(A % 1024 == 0 && BH % 1024 == 0, "the swizzle repeats every 1 KB");
};

// One MMA: K step j of a stage, column part h, whose scale columns begin
// `shift` columns into the slot's groups.  COLL: 1 leaves A in the collector
// for the next MMA, 2 takes it from there.
template <bool NV, class L, int COLL>
__device__ __forceinline__ void mma_pair(uint32_t tmem, uint32_t slot_col, uint64_t ad, uint64_t bd, uint32_t idesc,
                                         int h, uint32_t shift, int j, uint32_t acc) {
    const int g = NV ? j : j >> 1;
    const uint32_t id = idesc | (NV ? 0u : ((j & 1) * 2u << 29) | ((j & 1) * 2u << 4));
    const uint32_t sfb = slot_col + g * L::GC + h * (PH / 32) + shift, sfa = slot_col + g * L::GC + 4 * L::NB;
    if constexpr (NV) ptx::tc_mma_nvf4_pair<COLL>(tmem + h * PH, ad + 2 * j, bd + 2 * j, id, sfa, sfb, acc);
    else ptx::tc_mma_mxf4_pair<COLL>(tmem + h * PH, ad + 2 * j, bd + 2 * j, id, sfa, sfb, acc);
}

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

// The staged piece as 64 BF16 columns of C from (row0, col0), for a C that TMA
// cannot write: two neighbouring columns per lane, row by row.
__device__ __forceinline__ void write_bf16(const uint8_t *stage, int lane, const Params &p,
                                           int64_t row0, int64_t col0) {
    uint16_t *c = static_cast<uint16_t *>(p.c);
    const int64_t col = col0 + 2 * lane;
    for (int r = 0; r < 32 && row0 + r < p.M; ++r) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(
            stage + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
        uint16_t *d = c + (row0 + r) * p.sm + col;
        if (col < p.N) d[0] = static_cast<uint16_t>(w);
        if (col + 1 < p.N) d[1] = static_cast<uint16_t>(w >> 16);
    }
}

// The staged piece as 32 FP32 values per row from (row0, col0), for an output
// that is read and added to first (one rounding), or FP32 that TMA cannot write.
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
            const float4 o = *d;
            *d = make_float4(__uint_as_float(w.x) + o.x, __uint_as_float(w.y) + o.y, __uint_as_float(w.z) + o.z,
                             __uint_as_float(w.w) + o.w);
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

// A wait on a barrier of this CTA whose arrivals may come from the other one.
__device__ bool wait_pair(uint32_t bar, uint32_t parity, uint64_t limit, volatile uint32_t *abort_flag,
                          unsigned int *err, uint32_t who) {
    if (ptx::mbar_try_wait_cluster(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer();
    for (uint32_t n = 1;; ++n) {
        if (ptx::mbar_try_wait_cluster(bar, parity)) return true;
        if ((n & 15u) == 0) {
            if (*abort_flag) return false;
            if (ptx::globaltimer() - t0 > limit) {
                *abort_flag = 1u;
                atomicOr(err, 1u);
                atomicCAS(err + 1, 0u, who);
                return false;
            }
        }
    }
}

// The tensors' scales (NV) as two factors of a sum: 1 and their product, or, where
// that leaves FP32's normal range (each may be 2^-100 .. 2^117), the smaller and the
// larger.  A sum of products of codes and E4M3 scales is 0 or between 2^-20 and
// 2^53 in magnitude, so its product with the smaller one leaves the range only if
// the result does.
template <bool NV>
struct TensorScales {
    float first = 1.0f, second = 1.0f;
    bool split = false;
    __device__ __forceinline__ explicit TensorScales(const Params &p) {
        if constexpr (NV) {
            const float a = p.ta ? ptx::ld_f32(p.ta) : 1.0f, b = p.tb ? ptx::ld_f32(p.tb) : 1.0f;
            second = a * b;
            split = !(second >= 0x1p-126f && second < 0x1p128f);
            if (split) first = a < b ? a : b, second = a < b ? b : a;
        }
    }
};

// The tiles of a pair, in order: the wide ones dealt round, then those of one
// part, which first go to the pairs that the last deal left out, two each.
struct PairTiles {
    int pair, npairs, wide, rem;   // `wide` of them for this pair; left over from the even deals
    __device__ __forceinline__ PairTiles(const Params &p, int pair_, int npairs_)
        : pair(pair_), npairs(npairs_), wide((p.num_tiles - pair_ + npairs_ - 1) / npairs_),
          rem(p.num_tiles % npairs_) {}
    // The i-th tile's place and its column parts; 0 past the last.
    template <int NH>
    __device__ __forceinline__ int get(const Params &p, int i, int &mb, int &nb) const {
        if (i < wide) {
            tile_coords(pair + i * npairs, p.num_mb, p.num_nb, mb, nb);
            return NH;
        }
        if (NH == 1) return 0;
        const int j = i - wide, low = npairs - rem;
        const int u = pair < rem ? 2 * low + pair + j * npairs
                                 : j < 2 ? pair - rem + j * low : 2 * low + pair + (j - 2) * npairs;
        mb = u, nb = p.num_nb;
        return u < p.half_tiles ? 1 : 0;
    }
};

template <bool NV, int NH>
__global__ void __launch_bounds__(P_THREADS, 1)
    k_fp4_pair(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
               const __grid_constant__ CUtensorMap tmap_sa, const __grid_constant__ CUtensorMap tmap_sb,
               const __grid_constant__ CUtensorMap tmap_c, const Params p, const uint32_t idesc) {
    using L = PairLayout<NV, NH>;
    constexpr int S = L::S, SLOTS = L::SLOTS, SUB = L::SUB;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    const uint32_t bar = base + L::OFF_BAR;
    const uint32_t empty = bar + L::EMPTY, scales = bar + L::SCALES, sfull = bar + L::SFULL, rest = bar + L::REST,
                   tfull = bar + L::TFULL, tempty = bar + L::TEMPTY, drain = bar + L::DRAIN;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + L::OFF_MISC);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(gbase + L::OFF_MISC + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = static_cast<int>(blockIdx.x >> 1), npairs = static_cast<int>(gridDim.x >> 1);
    const PairTiles tiles(p, pair, npairs);
    const uint64_t limit = p.wait_limit_ns, drain_limit = 2000000ull;
    // the even CTA's barriers, as seen from either CTA
    const uint32_t full_l = ptx::map_shared_rank(bar, 0), sfull_l = full_l + L::SFULL, tempty_l = full_l + L::TEMPTY;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(bar + 8 * s, 2 + L::NB);      // the bytes and the scale copiers
            ptx::mbar_init(empty + 8 * s, 1);
            ptx::mbar_init(sfull + 8 * s, 1);
            ptx::mbar_init(scales + 8 * s, 1 + L::NB);
            ptx::mbar_init(rest + 8 * s, 1 + L::NB);
        }
        for (int h = 0; h < 2; ++h) {
            ptx::mbar_init(tfull + 8 * h, 1);
            ptx::mbar_init(tempty + 8 * h, 8);   // the half's four epilogue warps of each CTA
        }
        for (int i = 0; i < 5; ++i) ptx::mbar_init(drain + 8 * i, 1);
        *abort_flag = 0u;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&tmap_a);
        ptx::prefetch_tmap(&tmap_b);
        ptx::prefetch_tmap(&tmap_sa);
        ptx::prefetch_tmap(&tmap_sb);
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(ptx::smem_u32(tmem_slot), 512);
        ptx::tmem_relinquish_pair();
    }
    // The kernel after this one is not launched early: its CTAs, though they only
    // wait, slow this one down (8192 x 8960 x 1536 backward, a quantizer and two
    // products: 126 us against 116).
    ptx::grid_wait();
    ptx::tc_fence_before();
    ptx::cluster_sync();   // both CTAs' barriers and tensor memory exist
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // 512 threads are launched with 128 registers; the epilogue's two
    // warpgroups take over what the others leave (2 * 128 * (168 + 80) <= 65536)
    if (warp >= 4 && warp < 12) {
        // ---------------------------------------------------------- epilogue
        // An accumulator goes to registers, C from there in pieces of 32 rows x
        // 128 bytes through the warp's staging area: by TMA, which cuts off
        // what lies past C's edges, or (an odd C, or one that is added to) by
        // the lanes.  TMA instead of 16-byte stores of the lanes: BF16 2 to 4 %
        // of the whole product, FP32 5 to 7 %.
        ptx::setmaxnreg_inc<168>();
        const int q = warp & 3, half = (warp - 4) >> 2;
        uint8_t *stage = gbase + L::OFF_EPI + (warp - 4) * EPI_BYTES;
        const TensorScales<NV> ts(p);
        const float alpha = ts.second;
        // scales in two steps are rare: BF16 outputs then go the way of those that are
        // added to, so that the common path has nothing to ask
        const bool tma = p.c_tma && (p.out_fp32 || !ts.split);
        // a C that is added to, four values at a time (without `accumulate` such a C is TMA's)
        const bool vec = p.accumulate && (reinterpret_cast<uintptr_t>(p.c) & 15) == 0 && p.sm % 4 == 0;
        for (int i = 0, mb, nb; tiles.get<NH>(p, i, mb, nb) > half; ++i) {
            bool ok = wait_phase(tfull + 8 * half, i & 1u, limit, abort_flag, p.err, WHO_EPILOGUE);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            ptx::tc_fence_after();
            const int64_t row0 = static_cast<int64_t>(mb) * PM + rank * 128 + q * 32;
            const int64_t col0 = static_cast<int64_t>(nb) * L::PN + half * PH;
            const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + half * PH;
            auto release = [&] {
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_relaxed(tempty_l + 8 * half);
            };
            if (p.out_fp32 || p.accumulate || ts.split) {
#pragma unroll 1
                for (int part = 0; part < 3; ++part) {
                    uint32_t r[2][32];
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        ptx::tmem_ld_32x32b_x32(taddr + (part * 2 + c) * 32, r[c]);
                    ptx::tmem_wait_ld();
                    if (part == 2) release();
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int at = (part * 2 + c) * 32;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            r[c][e] = __float_as_uint(__uint_as_float(r[c][e]) * ts.first * alpha);
                        if (tma && lane == 0) ptx::bulk_wait_read();
                        __syncwarp();
                        stage_row(stage, lane, r[c]);
                        if (tma) ptx::fence_proxy_async_smem();
                        __syncwarp();
                        if (!tma) {
                            write_f32(stage, lane, p, row0, col0 + at, vec);
                        } else if (lane == 0 && row0 < p.M && col0 + at < p.N) {
                            ptx::tma_store_2d(&tmap_c, ptx::smem_u32(stage), static_cast<int>(col0) + at,
                                              static_cast<int>(row0));
                            ptx::bulk_commit();
                        }
                    }
                }
                continue;
            }
            uint32_t packed[PH / 2];
#pragma unroll
            for (int chunk = 0; chunk < PH / 64; ++chunk) {
                uint32_t r[64];
                ptx::tmem_ld_32x32b_x64(taddr + chunk * 64, r);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const F2 v = mul2(f2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])), f2(alpha));
                    packed[chunk * 32 + e] = ptx::cvt_bf16x2(v.lo(), v.hi());
                }
            }
            release();
#pragma unroll
            for (int piece = 0; piece < PH / 64; ++piece) {
                // (in this form it needs no more registers than there are)
                if (tma) {
                    if (lane == 0) ptx::bulk_wait_read();
                    __syncwarp();
                }
                stage_row(stage, lane, packed + piece * 32);
                if (tma) {
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && row0 < p.M && col0 + piece * 64 < p.N) {
                        ptx::tma_store_2d(&tmap_c, ptx::smem_u32(stage), static_cast<int>(col0) + piece * 64,
                                          static_cast<int>(row0));
                        ptx::bulk_commit();
                    }
                } else {
                    __syncwarp();
                    write_bf16(stage, lane, p, row0, col0 + piece * 64);
                    __syncwarp();
                }
            }
        }
        if (tma && lane == 0) ptx::bulk_wait();
    } else {
        ptx::setmaxnreg_dec<80>();
        // A producer's end, after `it` stages: the even CTA waits until both CTAs'
        // last copies have landed, the odd one for the arrivals that free them (the
        // cluster barrier below keeps each resident until the other is there).  A
        // CTA that stopped early cannot tell which of its last copies have been
        // counted: it gives them the drain bound to land.
        auto landed = [&](uint32_t full, uint32_t freed, uint32_t it, bool ok) {
            for (uint32_t i = it < S ? 0 : it - S; i < it; ++i)
                wait_phase((leader ? full : freed) + 8 * (i % S), (i / S) & 1u, drain_limit, abort_flag, p.err,
                           WHO_PRODUCER, false);
            if (!ok || *abort_flag) {
                const uint64_t t0 = ptx::globaltimer();
                while (ptx::globaltimer() - t0 < drain_limit) {
                }
            }
        };
        if (warp == 0) {
            // ---------------------------------------------------------- producer
            if (lane == 0) {
                uint32_t it = 0;
                bool ok = true;
                for (int i = 0, mb, nb, parts; ok && (parts = tiles.get<NH>(p, i, mb, nb)) != 0; ++i) {
                    const int arow = mb * PM + static_cast<int>(rank) * 128;
                    const int brow = nb * L::PN + static_cast<int>(rank) * (PH / 2);
                    for (int kb = 0; kb < p.nk; ++kb) {
                        const uint32_t s = it % S, full = full_l + 8 * s;
                        ok = wait_phase(empty + 8 * s, ((it / S) & 1u) ^ 1u, limit, abort_flag, p.err, WHO_PRODUCER);
                        if (!ok) break;
                        // inject = 1 (a test of the timeout path): the first
                        // CTA never issues its first stage
                        if (!(p.inject == 1 && blockIdx.x == 0 && it == 0)) {
                            const uint32_t st = base + s * L::STAGE;
                            if (leader) ptx::mbar_arrive_expect_tx(bar + 8 * s, 2 * (L::A + parts * L::BH));
                            ptx::tma_load_2d_pair(st, &tmap_a, full, kb * kStageBytes, arow);
                            ptx::tma_load_2d_pair(st + L::A, &tmap_b, full, kb * kStageBytes, brow);
                            if (parts == 2)
                                ptx::tma_load_2d_pair(st + L::A + L::BH, &tmap_b, full, kb * kStageBytes, brow + PH);
                        }
                        ++it;
                    }
                }
                landed(bar, empty, it, ok);
            }
            __syncwarp();
        } else if (warp == 14) {
            // ---------------------------------------------------- scale producer
            // On its own, because a stage of scales is free again as soon as it is
            // in tensor memory: the copies run ahead of the operands.
            if (lane == 0) {
                uint32_t it = 0;
                bool ok = true;
                for (int i = 0, mb, nb; ok && tiles.get<NH>(p, i, mb, nb) != 0; ++i) {
                    const int sarow = mb * 2 + static_cast<int>(rank), sbrow = nb * L::PN / 128;
                    for (int kb = 0; kb < p.nk; ++kb, ++it) {
                        const uint32_t s = it % S, full = sfull_l + 8 * s, sf = base + L::OFF_SF + s * L::SF_STAGE;
                        ok = wait_phase(scales + 8 * s, ((it / S) & 1u) ^ 1u, limit, abort_flag, p.err, WHO_PRODUCER);
                        if (!ok) break;
                        if (leader) ptx::mbar_arrive_expect_tx(sfull + 8 * s, 2 * L::SF_STAGE);
                        ptx::tma_load_3d_pair(sf, &tmap_sa, full, 0, kb * L::NG, sarow);
                        ptx::tma_load_3d_pair(sf + L::SF, &tmap_sb, full, 0, kb * L::NG, sbrow);
                    }
                }
                landed(sfull, scales, it, ok);
            }
            __syncwarp();
        } else if (warp == 1 && leader) {
            // -------------------------------------------------------- MMA issuer
            // The two column halves alternate, except in a tile's first and last
            // stage, where one half's four MMAs go before the other's: so the first
            // accumulator is drained under the second one's last MMAs, and the
            // second under the first one's first MMAs of the next tile.  (This one
            // thread's latency counts: with calls in its waits or another branch in
            // the inner loop the product takes 2 to 5 % longer.)
            if (lane == 0) {
                uint32_t it = 0, shift = 0;
                int parts = 0;
                bool ok = true;
                // part h of stage `it`
                auto issue = [&](int h, bool zero) {
                    const uint32_t s = it % S, st = base + s * L::STAGE, col = tmem + L::PN + it % SLOTS * L::COLS;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_pair<NV, L, 0>(tmem, col, desc_sw128(st), desc_sw128(st + L::A + h * L::BH), idesc, h,
                                           shift, j, zero && j == 0 ? 0u : 1u);
                    if (h == parts - 1) ptx::tc_commit_pair(empty + 8 * s, 0x3);
                };
                auto ready = [&] {
                    const bool r = wait_pair(bar + 8 * (it % S), (it / S) & 1u, limit, abort_flag, p.err, WHO_MMA);
                    ptx::tc_fence_after();
                    return r;
                };
                auto ready_rest = [&] {
                    if (SUB == 1) return true;
                    const bool r = wait_phase(rest + 8 * (it % S), (it / S) & 1u, limit, abort_flag, p.err, WHO_MMA);
                    ptx::tc_fence_after();
                    return r;
                };
                int mb, nb, next = tiles.get<NH>(p, 0, mb, nb);
                for (int t = 0; ok && next != 0; ++t) {
                    parts = next;
                    shift = nb * L::PN % 128 / 32;
                    ok = ready() && ready_rest();
                    for (int h = 0; h < parts && ok; ++h) {
                        ok = wait_pair(tempty + 8 * h, (t & 1u) ^ 1u, limit, abort_flag, p.err, WHO_MMA);
                        if (!ok) break;
                        ptx::tc_fence_after();
                        issue(h, true);
                        if (p.nk == 1) ptx::tc_commit_pair(tfull + 8 * h, 0x3);
                    }
                    if (!ok) break;
                    ++it;
                    next = tiles.get<NH>(p, t + 1, mb, nb);   // under the MMAs: its divisions take a while
                    for (int kb = 1; parts == 1 && kb < p.nk - 1; ++kb, ++it) {
                        ok = ready() && ready_rest();
                        if (!ok) break;
                        issue(0, false);
                    }
                    for (int kb = 1; parts == 2 && kb < p.nk - 1; ++kb, ++it) {
                        ok = ready();
                        if (!ok) break;
                        const uint32_t s = it % S;
                        const uint32_t st = base + s * L::STAGE, col = tmem + L::PN + it % SLOTS * L::COLS;
                        const uint64_t ad = desc_sw128(st), bd = desc_sw128(st + L::A);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (SUB == 2 && j == 2) {
                                ok = ready_rest();
                                if (!ok) break;
                            }
                            mma_pair<NV, L, 1>(tmem, col, ad, bd, idesc, 0, shift, j, 1u);
                            mma_pair<NV, L, 2>(tmem, col, ad, bd + (L::BH >> 4), idesc, 1, shift, j, 1u);
                        }
                        if (!ok) break;
                        ptx::tc_commit_pair(empty + 8 * s, 0x3);
                    }
                    if (p.nk == 1) continue;
                    for (int h = 0; h < parts && ok; ++h) {
                        ok = h != 0 || (ready() && ready_rest());
                        if (!ok) break;
                        issue(h, false);
                        ptx::tc_commit_pair(tfull + 8 * h, 0x3);
                    }
                    ++it;
                }
                ptx::tc_commit_pair(drain, 0x1);
                wait_phase(drain, 0u, drain_limit, abort_flag, p.err, WHO_MMA, false);
            }
            __syncwarp();
        } else if ((warp == 2 || warp == 3 || (warp >= 12 && warp < 11 + L::NB)) && leader) {
            // ------------------------------------------- scales to tensor memory
            // One of the 128-row tiles each (0: A's rows, then B's), into the slot
            // that the MMAs of stage it - SLOTS freed.  A copy costs its
            // thread about 80 cycles, so two copiers could not keep up with NV's
            // 16 copies per stage.
            if (lane == 0) {
                const int row = warp < 4 ? warp - 2 : warp - 10;
                const uint32_t dst = tmem + L::PN + (row == 0 ? 4 * L::NB : (row - 1) * 4);
                const uint64_t src = desc_scales(base + L::OFF_SF + row * L::SF);
                uint32_t it = 0;
                bool ok = true;
                for (int i = 0, mb, nb; ok && tiles.get<NH>(p, i, mb, nb) != 0; ++i) {
                    for (int kb = 0; kb < p.nk; ++kb, ++it) {
                        const uint32_t s = it % S, slot = it % SLOTS, u = it - SLOTS;
                        ok = wait_pair(sfull + 8 * s, (it / S) & 1u, limit, abort_flag, p.err, WHO_SCALES) &&
                             (it < SLOTS || wait_phase(empty + 8 * (u % S), (u / S) & 1u, limit, abort_flag, p.err,
                                                       WHO_SCALES));
                        if (!ok) break;
                        ptx::tc_fence_after();
                        const uint64_t sd = src + s * (L::SF_STAGE >> 4);
                        const uint32_t d = dst + slot * L::COLS;
#pragma unroll
                        for (int g = 0; g < L::NG; ++g) {
                            ptx::tc_cp_32x128b_warpx4_pair(d + g * L::GC, sd + g * 32);
                            if (g == L::NG / SUB - 1) ptx::tc_commit_pair(bar + 8 * s, 0x1);   // for the MMAs
                        }
                        // inject = 2 (a test of the timeout path): the second half
                        // of the first pair's second tile's second stage never comes
                        if (SUB == 2 && !(p.inject == 2 && pair == 0 && it == static_cast<uint32_t>(p.nk) + 1))
                            ptx::tc_commit_pair(rest + 8 * s, 0x1);
                        ptx::tc_commit_pair(scales + 8 * s, 0x3);   // for the scale producers
                    }
                }
                ptx::tc_commit_pair(drain + 8 * (row + 1), 0x1);
                wait_phase(drain + 8 * (row + 1), 0u, drain_limit, abort_flag, p.err, WHO_SCALES, false);
            }
            __syncwarp();
        }
    }

    // neither CTA leaves (or frees its tensor memory) while the other may still
    // read its shared memory, signal its barriers or write its tensor memory
    __syncwarp();
    ptx::tc_fence_before();
    ptx::cluster_sync();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem, 512);
    }
}

// ------------------------------------------------------------------ few rows
// P (128 rows per CTA, the MMA's M side) times Q (BN rows): with few tokens P
// is the weights and Q the tokens, so that a token costs no row of a 128-row
// tile.  The CTAs of a cluster take consecutive parts of K; each sends the
// FP32 partial sums of its tile to the CTAs that own them (a slice of P's rows
// each), which add them up in the order of the parts (the same bits every
// time) and store them.
//
// QUANT: Q comes in BF16 and the epilogue's warps, idle until the last MMA,
// quantize it into the operand stages themselves, each CTA all of its part of
// K: no quantization pass before the product, no codes in memory.
//
// What bounds a call of one token is latency: the 36 MB (MX) of 18944 x 3584
// weights take 5.4 us from memory, the call 9.1 us with x quantized on the way
// (NV 5.7 and 10.6), and 7.7 (9.4) where the call before left them in L2.
// So the first stages' copies are issued before the other warps have started.
constexpr int F_THREADS = 256;
template <bool NV, int BN>
struct FewLayout {
    static constexpr int S = BN <= 32 ? 8 : BN == 64 ? 6 : 4, SLOTS = 4, NG = NV ? 4 : 2;
    static constexpr uint32_t SF = NG * 512, A = 128 * kStageBytes, B = BN * kStageBytes;
    static constexpr uint32_t STAGE = A + B, OFF_SF = S * STAGE, SF_STAGE = 2 * SF;
    static constexpr uint32_t OFF_SUM = OFF_SF + S * SF_STAGE;          // partial sums, 128 BN floats
    // barriers: full[S], empty[S], scales[SLOTS], tfull, drain[2]
    static constexpr uint32_t OFF_BAR = OFF_SUM + BN * 512, EMPTY = 8 * S, SCALES = 16 * S;
    static constexpr uint32_t TFULL = SCALES + 8 * SLOTS, DRAIN = TFULL + 8;
    static constexpr uint32_t OFF_MISC = OFF_BAR + 256, SMEM = OFF_MISC + 16 + 1024;
    static constexpr uint32_t COL_SF = BN, COLS = 8 * NG;
    static constexpr uint32_t TCOLS = COL_SF + SLOTS * COLS <= 128 ? 128 : 256;
    // each slot is freed by its stage's barrier
    static_assert(SLOTS <= S && DRAIN + 16 <= 256 && SMEM <= 232448 && COL_SF + SLOTS * COLS <= TCOLS, "");
};

// Q in BF16, for QUANT.
struct QInput {
    const uint16_t *x;
    int64_t ld, k;
};

// The four MMAs of one stage (128 rows of A by BN of B).
template <bool NV, int BN, class L>
__device__ __forceinline__ void issue_stage(uint32_t tmem, uint32_t slot_col, uint32_t b_shift, uint32_t s_a,
                                            uint32_t s_b, uint32_t idesc, bool first) {
    const uint64_t ad = desc_sw128(s_a), bd = desc_sw128(s_b);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int g = NV ? j : j >> 1;
        const uint32_t id = idesc | (NV ? 0u : ((j & 1) * 2u << 29) | ((j & 1) * 2u << 4));
        const uint32_t sfb = slot_col + g * 4 + b_shift, sfa = slot_col + (L::NG + g) * 4;
        const uint32_t acc = first && j == 0 ? 0u : 1u;
        if constexpr (NV) ptx::tc_mma_nvf4(tmem, ad + 2 * j, bd + 2 * j, id, sfa, sfb, acc);
        else ptx::tc_mma_mxf4(tmem, ad + 2 * j, bd + 2 * j, id, sfa, sfb, acc);
    }
}

__device__ __forceinline__ void store_out(const Params &p, int64_t at, float v) {
    if (p.out_fp32) {
        float *d = static_cast<float *>(p.c) + at;
        *d = p.accumulate ? *d + v : v;
    } else {
        uint16_t *d = static_cast<uint16_t *>(p.c) + at;
        if (p.accumulate) v += __uint_as_float(static_cast<uint32_t>(*d) << 16);
        *d = static_cast<uint16_t>(ptx::cvt_bf16x2(v, 0.0f));
    }
}

// Sets the abort flag (its address in this CTA) of the cluster's CTAs.  Out of line:
// within the kernel it costs a call of one token 0.12 us of instruction fetch.
__device__ __noinline__ void abort_cluster(uint32_t flag, int ctas) {
#pragma unroll 1
    for (int i = 0; i < ctas; ++i) ptx::st_cluster_u32(ptx::map_shared_rank(flag, i), 1u);
}

template <bool NV, int BN, bool QUANT>
__global__ void __launch_bounds__(F_THREADS, 1)
    k_fp4_few(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
              const Params p, const QInput qi, const uint32_t idesc) {
    using L = FewLayout<NV, BN>;
    constexpr int S = L::S, SLOTS = L::SLOTS;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    const uint32_t bar = base + L::OFF_BAR;
    const uint32_t tfull = bar + L::TFULL, drain = bar + L::DRAIN;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + L::OFF_MISC);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(gbase + L::OFF_MISC + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t limit = p.wait_limit_ns, drain_limit = 2000000ull;
    const int splits = p.splits, part = blockIdx.x % splits, tile = blockIdx.x / splits;
    const int nb = tile % p.num_nb, mb = tile / p.num_nb;
    const int kb0 = static_cast<int>(static_cast<int64_t>(part) * p.nk / splits);
    const int kb1 = static_cast<int>(static_cast<int64_t>(part + 1) * p.nk / splits);
    const int n = kb1 - kb0;                         // at least 1: splits <= nk
    const int64_t row0 = static_cast<int64_t>(mb) * 128, col0 = static_cast<int64_t>(nb) * BN;
    const int cols = static_cast<int>(min(static_cast<int64_t>(BN), p.N - col0));
    const int rl = 7 - (31 - __clz(splits));               // this CTA's share of the sums: 2^rl rows
    const int lr = cols <= 1 ? 0 : 32 - __clz(cols - 1);   // QUANT (at most eight rows): 2^lr >= cols

    const uint8_t *ga = p.sa + static_cast<int64_t>(mb) * p.scale_tiles * 512;
    const uint8_t *gb = QUANT ? nullptr : p.sb + static_cast<int64_t>(nb) * BN / 128 * p.scale_tiles * 512;
    auto load_stage = [&](int it) {
        // inject = 1 (a test of the timeout path): the first CTA never issues
        // its first stage
        if (p.inject == 1 && blockIdx.x == 0 && it == 0) return;
        const int s = it % S, kb = kb0 + it;
        const uint32_t full = bar + 8 * s, sa = base + s * L::STAGE, sf = base + L::OFF_SF + s * L::SF_STAGE;
        const int64_t at = static_cast<int64_t>(kb) * L::SF;
        ptx::mbar_arrive_expect_tx(full, QUANT ? L::A + L::SF : L::STAGE + 2 * L::SF);
        ptx::tma_load_2d(sa, &tmap_a, full, kb * kStageBytes, mb * 128);
        ptx::bulk_load(sf, ga + at, L::SF, full);
        if (!QUANT) {
            ptx::tma_load_2d(sa + L::A, &tmap_b, full, kb * kStageBytes, nb * BN);
            ptx::bulk_load(sf + L::SF, gb + at, L::SF, full);
        }
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(bar + 8 * s, QUANT ? 1 + (16 << lr) : 1);   // the copies, the quantizing threads
            ptx::mbar_init(bar + L::EMPTY + 8 * s, 1);
        }
        for (int i = 0; i < SLOTS; ++i) ptx::mbar_init(bar + L::SCALES + 8 * i, 1);
        ptx::mbar_init(tfull, 1);
        ptx::mbar_init(drain, 1);
        ptx::mbar_init(drain + 8, 1);
        *abort_flag = 0u;
        ptx::fence_mbar_init();
    }
    ptx::grid_begin(1);   // a short one
    if (threadIdx.x == 0)
        for (int it = 0; it < 2 && it < n; ++it) load_stage(it);
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), L::TCOLS);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    // the others may write this CTA's shared memory once all have come here
    if (splits > 1) ptx::cluster_arrive();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        int it = n < 2 ? n : 2;
        for (; it < n; ++it) {
            const int s = it % S;
            bool ok = it < S || wait_phase(bar + L::EMPTY + 8 * s, ((it / S) & 1u) ^ 1u, limit, abort_flag, p.err,
                                           WHO_PRODUCER);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            if (lane == 0) load_stage(it);
            __syncwarp();
        }
        // the copies in flight land before the CTA ends.  With QUANT a stage's
        // phase also waits for the quantizing threads: where they have given
        // up, the bound passes instead, in which the copies (microseconds) land.
        for (int i = it > S ? it - S : 0; i < it; ++i)
            wait_phase(bar + 8 * (i % S), (i / S) & 1u, drain_limit, abort_flag, p.err, WHO_PRODUCER, false);
    } else if (warp == 1) {
        const uint32_t b_shift = (nb * BN % 128) / 32;
        bool ok = true;
        for (int it = 0; it < n && ok; ++it) {
            const int s = it % S, slot = it % SLOTS;
            ok = wait_phase(bar + 8 * s, (it / S) & 1u, limit, abort_flag, p.err, WHO_MMA) &&
                 wait_phase(bar + L::SCALES + 8 * slot, (it / SLOTS) & 1u, limit, abort_flag, p.err, WHO_MMA);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            ptx::tc_fence_after();
            if (lane == 0) {
                const uint32_t sa = base + s * L::STAGE;
                issue_stage<NV, BN, L>(tmem, tmem + L::COL_SF + slot * L::COLS, b_shift, sa, sa + L::A, idesc, it == 0);
                ptx::tc_commit(bar + L::EMPTY + 8 * s);
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
                ok = wait_phase(bar + L::EMPTY + 8 * (u % S), (u / S) & 1u, limit, abort_flag, p.err, WHO_SCALES);
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
                    ptx::tc_cp_32x128b_warpx4(col + (L::NG + g) * 4, desc_scales(sf + g * 512));
                }
                ptx::tc_commit(bar + L::SCALES + 8 * slot);
            }
            __syncwarp();
        }
        if (lane == 0) ptx::tc_commit(drain + 8);
        __syncwarp();
        wait_phase(drain + 8, 0u, drain_limit, abort_flag, p.err, WHO_SCALES, false);
    } else if (warp >= 4) {
        bool ok = true;
        if constexpr (QUANT) {
            // The segments of 16 elements of a stage, 2^lr rows by 16 of them,
            // go round the 128 threads, stage after stage (one token: eight
            // stages at a time), the next one's load in flight.  Rows past
            // the last are not written: they only reach outputs that are not
            // stored.  The loop is not unrolled: a decoding step runs it once
            // or twice, and the instruction fetch of an unrolled one took
            // longer than what it saved.
            const int tid = threadIdx.x - 128;
            const float t = NV && p.tb ? ptx::ld_f32(p.tb) : 1.0f, rt = fp4_reciprocal<NV>(t);
            const bool wide = (reinterpret_cast<uintptr_t>(qi.x) & 31) == 0 && (qi.ld & 15) == 0;
            auto load = [&](int idx, uint32_t (&w)[8]) {
                const int row = (idx >> 4) & ((1 << lr) - 1), it = idx >> (4 + lr);
                const int64_t c0 = static_cast<int64_t>(kb0 + it) * 256 + (idx & 15) * 16;
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = 0u;
                if (it < n && row < cols && c0 < qi.k) {
                    const uint16_t *src = qi.x + (col0 + row) * qi.ld + c0;
                    if (wide && c0 + 16 <= qi.k) ragged::load16<true>(src, 16, w);
                    else ragged::load16<false>(src, static_cast<int>(qi.k - c0), w);
                }
            };
            const int items = (n * (16 << lr) + 127) / 128;
            uint32_t w[8], next[8];
            load(tid, w);
#pragma unroll 1
            for (int a = 0; a < items; ++a) {
                const int idx = a * 128 + tid, row = (idx >> 4) & ((1 << lr) - 1), seg = idx & 15;
                const int it = idx >> (4 + lr), s = it % S;
                load(idx + 128, next);
                uint32_t m = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) m = __vmaxu2(m, w[e] & 0x7FFF7FFFu);
                m = max(m & 0xFFFFu, m >> 16);
                if (!NV) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
                ok = ok && (it >= n || wait_phase(bar + L::EMPTY + 8 * s, ((it / S) & 1u) ^ 1u, limit, abort_flag,
                                                  p.err, WHO_EPILOGUE));
                if (it < n && ok) {
                    if (row < cols) {
                        uint8_t *sq = gbase + s * L::STAGE + L::A;
                        uint8_t *sf = gbase + L::OFF_SF + s * L::SF_STAGE + L::SF;
                        const Fp4Scale<NV> sc(m, t, rt);
                        // the 128-byte swizzle of the operand tile
                        *reinterpret_cast<uint2 *>(sq + row * 128 + (((seg >> 1) ^ (row & 7)) << 4) + (seg & 1) * 8) =
                            make_uint2(sc.cast8(w), sc.cast8(w + 4));
                        const int j = NV ? seg : seg >> 1;
                        if (NV || (seg & 1) == 0)
                            sf[(j >> 2) * 512 + row * 16 + (j & 3)] = static_cast<uint8_t>(sc.byte);
                    }
                    ptx::fence_proxy_async_smem();
                    ptx::mbar_arrive(bar + 8 * s);
                }
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = next[e];
            }
        }
        ok = ok && wait_phase(tfull, 0u, limit, abort_flag, p.err, WHO_EPILOGUE);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (splits > 1) ptx::cluster_wait();
        if (ok) {
            // row r's sums go to CTA r / (128 / splits): [part][column][its rows]
            ptx::tc_fence_after();
            const int q = warp & 3, r = q * 32 + lane;
            const uint32_t off = base + L::OFF_SUM + (((part * BN) << rl) + (r & ((1 << rl) - 1))) * 4;
            const uint32_t dst = splits > 1 ? ptx::map_shared_rank(off, r >> rl) : off, step = 4u << rl;
#pragma unroll 1
            for (int c = 0; c < cols; c += 16) {
                uint32_t v[16];
                ptx::tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(q * 32) << 16) + c, v);
                ptx::tmem_wait_ld();
                const uint32_t d = dst + c * step;
                if (splits > 1) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (c + i < cols) ptx::st_cluster_u32(d + i * step, v[i]);
                } else {
                    // columns past the last have room
#pragma unroll
                    for (int i = 0; i < 16; ++i) ptx::st_shared_u32(d + i * step, v[i]);
                }
            }
            ptx::tc_fence_before();
        } else if (splits > 1 && lane == 0) {
            // the other CTAs' sums lack this part: none of the cluster stores
            abort_cluster(base + L::OFF_MISC + 4, splits);
        }
    }

    __syncwarp();
    if (splits > 1) {
        if (warp < 4) ptx::cluster_wait();
        ptx::cluster_sync();
    } else {
        __syncthreads();
    }
    if (!*abort_flag) {
        const TensorScales<NV> ts(p);
        // this CTA's rows, one to a thread group's lane; columns go round the
        // groups
        const float *sum = reinterpret_cast<const float *>(gbase + L::OFF_SUM);
        const int r = threadIdx.x & ((1 << rl) - 1);
        const int64_t row = row0 + (part << rl) + r;
        if (row < p.M) {
            const int dc = F_THREADS >> rl;
            for (int c = threadIdx.x >> rl; c < cols; c += 8 * dc) {
                // eight columns' sums before their stores: a store through a
                // generic pointer keeps later shared-memory reads behind it
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = 0.0f;
                for (int k = 0; k < splits; ++k)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (c + i * dc < cols) v[i] += sum[((k * BN + c + i * dc) << rl) + r];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c + i * dc < cols)
                        store_out(p, row * p.sm + (col0 + c + i * dc) * p.sn, v[i] * ts.first * ts.second);
            }
        }
    }
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, L::TCOLS);
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

// The scale tiles of an operand, [row tiles, tiles along K, 128 words], and a
// copy of `rows` row tiles by one stage.
bool make_scale_tmap(CUtensorMap *m, const Fp4Operand &o, int rows) {
    TensorMapEncodeFn enc = tensor_map_encoder();
    if (!enc) return false;
    std::memset(m, 0, sizeof(*m));
    const int64_t tiles = fp4_scale_tiles(o.k, o.kind);
    const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(tiles), static_cast<cuuint64_t>(fp4_row_tiles(o.rows))};
    const cuuint64_t strides[2] = {512, static_cast<cuuint64_t>(tiles) * 512};
    const cuuint32_t box[3] = {128, o.kind == FP4_NV ? 4u : 2u, static_cast<cuuint32_t>(rows)}, estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint8_t *>(o.scale), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// BF16 C, written in pieces of 32 rows x 64 columns.
bool make_out_tmap(CUtensorMap *m, const Params &p) {
    TensorMapEncodeFn enc = tensor_map_encoder();
    if (!enc) return false;
    std::memset(m, 0, sizeof(*m));
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(p.N), static_cast<cuuint64_t>(p.M)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(p.sm) * (p.out_fp32 ? 4 : 2)};
    const cuuint32_t box[2] = {p.out_fp32 ? 32u : 64u, 32}, estr[2] = {1, 1};
    return enc(m, p.out_fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.c, dims,
               strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

std::mutex g_mu;
bool g_ready[64] = {false};   // the kernels' attributes are set on a device

template <class K>
cudaError_t allow_smem(K kern, uint32_t bytes) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
}
template <bool NV>
cudaError_t set_attributes() {
    cudaError_t e = allow_smem(k_fp4_pair<NV, 2>, PairLayout<NV, 2>::SMEM);
    if (e == cudaSuccess) e = allow_smem(k_fp4_pair<NV, 1>, PairLayout<NV, 1>::SMEM);
    if (e == cudaSuccess) e = allow_smem(k_fp4_few<NV, 16, false>, FewLayout<NV, 16>::SMEM);
    if (e == cudaSuccess) e = allow_smem(k_fp4_few<NV, 16, true>, FewLayout<NV, 16>::SMEM);
    if (e == cudaSuccess) e = allow_smem(k_fp4_few<NV, 32, false>, FewLayout<NV, 32>::SMEM);
    if (e == cudaSuccess) e = allow_smem(k_fp4_few<NV, 64, false>, FewLayout<NV, 64>::SMEM);
    if (e == cudaSuccess) e = allow_smem(k_fp4_few<NV, 128, false>, FewLayout<NV, 128>::SMEM);
    return e;
}

// Instruction descriptor of the 4-bit kinds: E2M1 (1) for A and B in bits 7-9
// and 10-12, N >> 3 in bits 17-22, the scale type in bit 23 (0: E4M3, 1:
// UE8M0), M >> 4 in bits 24-28; scale-factor ids are added per MMA.
uint32_t instruction(bool nv, int m, int n) {
    return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | ((nv ? 0u : 1u) << 23) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

template <class K, class... Args>
int launch_cluster(K kern, int64_t ctas, int cluster, int threads, uint32_t smem, cudaStream_t stream,
                   const Args &...args) {
    const cudaError_t e = launch_after(kern, static_cast<unsigned>(ctas), threads, smem, stream, cluster, args...);
    return e == cudaSuccess ? 0 : 2 + static_cast<int>(e);
}

// P and Q: the operands on the MMA's M and N side; swapped: P is B.
void set_operands(Params &p, const Fp4GemmArgs &g, bool swapped, int tm, int tn) {
    const Fp4Operand &P = swapped ? g.b : g.a, &Q = swapped ? g.a : g.b;
    p.M = static_cast<int>(P.rows);
    p.N = static_cast<int>(Q.rows);
    p.num_mb = (p.M + tm - 1) / tm;
    p.num_nb = (p.N + tn - 1) / tn;
    p.sa = P.scale;
    p.sb = Q.scale;
    p.ta = P.ts;
    p.tb = Q.ts;
    p.sm = swapped ? 1 : g.ldc;
    p.sn = swapped ? g.ldc : 1;
}

// Whether the last column of 384-column tiles has at most 192 of them.
bool half_column(int64_t n) { return n % (2 * PH) != 0 && n % (2 * PH) <= PH; }

template <bool NV, int NH>
int launch_pair(const Fp4GemmArgs &g, Params &p, int sms, cudaStream_t stream) {
    using L = PairLayout<NV, NH>;
    set_operands(p, g, false, PM, L::PN);
    if (NH == 2 && half_column(p.N)) p.half_tiles = p.num_mb, --p.num_nb;
    const int64_t tiles = static_cast<int64_t>(p.num_mb) * p.num_nb + p.half_tiles;
    if (tiles > 0x7FFFFFFF) return 2 + static_cast<int>(cudaErrorInvalidValue);
    p.num_tiles = static_cast<int>(tiles) - p.half_tiles;
    CUtensorMap ta, tb, tsa, tsb, tc;
    if (!make_tmap(&ta, g.a, 128) || !make_tmap(&tb, g.b, PH / 2) || !make_scale_tmap(&tsa, g.a, 1) ||
        !make_scale_tmap(&tsb, g.b, L::NB))
        return 1;
    tc = tsb;   // not used unless c_tma
    p.c_tma = !p.accumulate && (reinterpret_cast<uintptr_t>(p.c) & 15) == 0 && p.sm % (p.out_fp32 ? 4 : 8) == 0 &&
              make_out_tmap(&tc, p);
    return launch_cluster(k_fp4_pair<NV, NH>, 2 * std::min<int64_t>(tiles, sms / 2), 2, P_THREADS, L::SMEM, stream,
                          ta, tb, tsa, tsb, tc, p, instruction(NV, PM, PH));
}

template <bool NV, int BN, bool QUANT>
int launch_few(const Fp4GemmArgs &g, Params &p, bool swapped, int splits, cudaStream_t stream) {
    set_operands(p, g, swapped, 128, BN);
    const int64_t tiles = static_cast<int64_t>(p.num_mb) * p.num_nb;
    if (tiles > 0x7FFFFFFF / 8) return 2 + static_cast<int>(cudaErrorInvalidValue);
    p.num_tiles = static_cast<int>(tiles);
    p.splits = splits;
    CUtensorMap ta, tb;
    if (!make_tmap(&ta, swapped ? g.b : g.a, 128)) return 1;
    if (QUANT) tb = ta;   // not used
    else if (!make_tmap(&tb, swapped ? g.a : g.b, BN)) return 1;
    const QInput qi{g.x, g.ld_x, g.a.k};
    return launch_cluster(k_fp4_few<NV, BN, QUANT>, tiles * splits, splits, F_THREADS, FewLayout<NV, BN>::SMEM, stream,
                          ta, tb, p, qi, instruction(NV, 128, BN));
}

// Which kernel, from its time as measured on a GB300 (microseconds; MX, NV is
// alike, 5 to 15 % slower throughout): a fixed part, then for every round of
// tiles over the machine a part per stage of K and one per tile.
//   pairs        4.5 + rounds (0.46 nk + 2.4) with 384 columns, (0.30 nk + 1.6) with 192
//   few rows     3.8 + rounds (c nk / splits + e), (c, e) by the tile's columns: 0.29, 0.4 for 16
//                ... 0.48, 2 for 128
// So 8192 x 8960 x 1536 takes 52 us with 384 columns and 55 with 192; 1024 x
// 3584 x 18944 38 and 29; 256 x 1536 x 8960 16 with pairs and 9.5 with four K
// parts of few-row tiles; 256 x 18944 x 3584 15 and 26.
struct Plan {
    int nh, bn, splits;     // nh > 0: pair tiles of 192 nh columns; else bn and K parts
    double us;
};

double rounds(int64_t tiles, int64_t slots) { return static_cast<double>((tiles + slots - 1) / slots); }

// The longest of the pairs' shares (see PairTiles) of wide and half tiles that
// take `tw` and `th`.
double wide_pairs(int64_t wide, int64_t half, int64_t pairs, double tw, double th) {
    const int64_t rem = wide % pairs, low = pairs - rem;
    const int64_t first = std::min<int64_t>(2, (half + low - 1) / low);
    const double more = half > 2 * low ? rounds(half - 2 * low, pairs) * th : 0.0;
    return static_cast<double>(wide / pairs) * tw + std::max(rem ? tw : 0.0, static_cast<double>(first) * th) + more;
}

Plan choose_few(int64_t rows, int64_t other, int nk, int sms) {
    const int widths[4] = {16, 32, 64, 128};
    const double stage[4] = {0.29, 0.31, 0.38, 0.48}, tile[4] = {0.4, 0.7, 1.6, 2.0};
    Plan best{0, 16, 1, 1e300};
    // the narrowest that holds all rows; of 64 and 128, with several tiles, the
    // faster one (a tile of 16 or 32 columns cannot begin inside a scale tile)
    for (int i = 0; i < 4; ++i) {
        if (widths[i] < rows && i < 2) continue;
        const int64_t tiles = (other + 127) / 128 * ((rows + widths[i] - 1) / widths[i]);
        for (int s = 1; s <= 8 && s <= nk; s *= 2) {
            // clusters of eight leave SMs of each GPC over
            const double us = 3.8 + rounds(tiles * s, s == 8 && sms >= 10 ? sms * 4 / 5 : sms) *
                                        (stage[i] * ((nk + s - 1) / s) + tile[i]);
            if (us < best.us) best = {0, widths[i], s, us};
        }
        if (widths[i] >= rows) break;
    }
    return best;
}

Plan choose(int64_t m, int64_t n, int nk, int sms) {
    Plan best = choose_few(std::min(m, n), std::max(m, n), nk, sms);
    if (std::min(m, n) > 32 && sms >= 2) {
        const int64_t mb = (m + PM - 1) / PM;
        const double two = 4.5 + wide_pairs(mb * ((n + PH - 1) / (2 * PH)), half_column(n) ? mb : 0, sms / 2,
                                            0.46 * nk + 2.4, 0.30 * nk + 1.6);
        const double one = 4.5 + rounds(mb * ((n + PH - 1) / PH), sms / 2) * (0.30 * nk + 1.6);
        if (one < best.us) best = {1, 0, 1, one};
        if (n > PH && two < best.us) best = {2, 0, 1, two};
    }
    return best;
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
    if (g.x) {
        const Plan plan = choose_few(g.a.rows, g.b.rows, p.nk, sms);
        return launch_few<NV, 16, true>(g, p, true, plan.splits, stream);
    }
    const bool swapped = g.a.rows <= g.b.rows;
    const Plan plan = choose(g.a.rows, g.b.rows, p.nk, sms);
    if (p.inject == 2 && plan.nh != 2) return 1;   // no stage's scales come in halves
    if (plan.nh == 2) return launch_pair<NV, 2>(g, p, sms, stream);
    if (plan.nh == 1) return launch_pair<NV, 1>(g, p, sms, stream);
    switch (plan.bn) {
    case 16: return launch_few<NV, 16, false>(g, p, swapped, plan.splits, stream);
    case 32: return launch_few<NV, 32, false>(g, p, swapped, plan.splits, stream);
    case 64: return launch_few<NV, 64, false>(g, p, swapped, plan.splits, stream);
    default: return launch_few<NV, 128, false>(g, p, swapped, plan.splits, stream);
    }
}

}  // namespace

// Quantizing inside the product, every CTA for itself, against a quantization
// pass before it (microseconds, weights from memory; MX / NV):
//   18944 x 3584   1 row 9.1 and 10.4 / 10.6 and 11.9   4 rows 9.6 and 10.4 / 11.3 and 12.0
//   1536 x 8960    1 row 5.8 and 6.9 / 6.8 and 7.6      4 rows 6.2 and 7.1 / 6.9 and 7.7
//   3584 x 18944   1 row 10.7 and 11.8 / 12.9 and 13.9  4 rows 11.4 and 12.0 / 13.2 and 13.9
// With the weights in L2 the gain is 0.3 to 0.5.  At eight rows the product's own
// quantization took 10 % longer.  The host launches once instead of twice.
bool fp4_linear_quantizes(int64_t rows) { return rows <= 4; }

int launch_fp4_gemm(const Fp4GemmArgs &g, cudaStream_t stream) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) dev = 0;
    {
        std::lock_guard<std::mutex> lock(g_mu);
        if (!g_ready[dev]) {
            cudaError_t e = set_attributes<true>();
            if (e == cudaSuccess) e = set_attributes<false>();
            if (e != cudaSuccess) return 2 + static_cast<int>(e);
            g_ready[dev] = true;
        }
    }
    return g.a.kind == FP4_NV ? launch<true>(g, sm_count(), stream) : launch<false>(g, sm_count(), stream);
}

}  // namespace fp8hg
