// Adapters: the plan of a batch, and the order of the kernels (lora.cuh).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "lora.cuh"

namespace fp8hg {

namespace {

constexpr int kPlanSmem = 200 * 1024;

// A stable counting sort by one CTA: each warp counts, then places, a run of
// neighbouring tokens.  counts: [warps][adapters + 1].
__global__ void __launch_bounds__(1024) k_lora_plan(const int *ids, int tokens, int adapters, int *words) {
    extern __shared__ int counts[];
    __shared__ int warp_total[32][2];
    const LoraPlan p{words, tokens, adapters};
    ptx::grid_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, warps = blockDim.x / 32;
    const int buckets = adapters + 1;
    for (int i = tid; i < warps * buckets; i += blockDim.x) counts[i] = 0;
    __syncthreads();
    const int per = ((tokens + warps - 1) / warps + 31) / 32 * 32;
    const int64_t from = static_cast<int64_t>(warp) * per, to = min(static_cast<int64_t>(tokens), from + per);
    int *mine = counts + warp * buckets;
    auto bucket = [&](int64_t i) {
        const int g = ids[i];
        return g >= 0 && g < adapters ? g : adapters;
    };
    for (int64_t i0 = from; i0 < to; i0 += 32) {
        const int64_t i = i0 + lane;
        const int b = i < to ? bucket(i) : -1;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, b);
        if (b >= 0 && lane == __ffs(same) - 1) mine[b] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    // every thread a run of buckets: their tokens and tiles, then where they begin
    const int run = (buckets + blockDim.x - 1) / blockDim.x, b0 = min(buckets, tid * run), b1 = min(buckets, b0 + run);
    int n = 0, t = 0;
    for (int b = b0; b < b1; ++b) {
        int c = 0;
        for (int w = 0; w < warps; ++w) c += counts[w * buckets + b];
        n += c;
        t += (c + kLoraTile - 1) / kLoraTile;
    }
    int sn = n, st = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int un = __shfl_up_sync(0xFFFFFFFFu, sn, o), ut = __shfl_up_sync(0xFFFFFFFFu, st, o);
        if (lane >= o) sn += un, st += ut;
    }
    if (lane == 31) warp_total[warp][0] = sn, warp_total[warp][1] = st;
    __syncthreads();
    int bn = sn - n, bt = st - t;
    for (int w = 0; w < warp; ++w) bn += warp_total[w][0], bt += warp_total[w][1];
    for (int b = b0; b < b1; ++b) {
        words[p.starts() + b] = bn;
        words[p.tile_first() + b] = bt;
        const int first = bn;
        for (int w = 0; w < warps; ++w) {
            const int c = counts[w * buckets + b];
            counts[w * buckets + b] = bn;
            bn += c;
        }
        for (int f = first; f < bn; f += kLoraTile, ++bt)
            reinterpret_cast<int4 *>(words + p.tiles())[bt] = make_int4(b == adapters ? -1 : b, f, min(kLoraTile, bn - f), -1);
    }
    if (b1 == buckets && b0 < b1) {
        words[p.starts() + buckets] = bn;
        words[p.tile_first() + buckets] = bt;
        words[0] = bt;
    }
    __syncthreads();
    for (int64_t i0 = from; i0 < to; i0 += 32) {
        const int64_t i = i0 + lane;
        const int b = i < to ? bucket(i) : -1;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, b);
        if (b >= 0) words[p.order() + mine[b] + __popc(same & ((1u << lane) - 1u))] = static_cast<int>(i);
        __syncwarp();
        if (b >= 0 && lane == __ffs(same) - 1) mine[b] += __popc(same);
        __syncwarp();
    }
    // an adapter's tokens are in ascending order: neighbours, if the last one says so
    __syncthreads();
    const int tiles = words[0];
    for (int b = tid; b < tiles; b += blockDim.x) {
        int4 *tile = reinterpret_cast<int4 *>(words + p.tiles()) + b;
        const int from_token = words[p.order() + tile->y];
        if (words[p.order() + tile->y + tile->z - 1] - from_token == tile->z - 1) tile->w = from_token;
    }
}

}  // namespace

cudaError_t launch_lora_plan(const int *ids, const LoraPlan &p, int *words, cudaStream_t stream) {
    static unsigned long long done;
    const int buckets = p.adapters + 1;
    const int warps = std::max(1, std::min(32, kPlanSmem / (4 * buckets)));
    const cudaError_t e = with_smem(&k_lora_plan, kPlanSmem, kPlanSmem, done);
    if (e != cudaSuccess) return e;
    return launch_after(&k_lora_plan, dim3(1), warps * 32, static_cast<size_t>(warps) * buckets * 4, stream, 1, ids, p.tokens,
                        p.adapters, words);
}

namespace {

size_t partial_bytes(int64_t tokens, int adapters, int r, int64_t k) {
    const int rp = lora::padded(r);
    return static_cast<size_t>(lora::most_splits({nullptr, static_cast<int>(tokens), adapters}, static_cast<int>(k), rp)) * tokens * rp *
           sizeof(float);
}

bool rows_aligned(const uint16_t *p, uint32_t ld) { return lora::aligned_to(p, 16) && ld % 8 == 0; }

// Rows for the kernels that TMA feeds: as they are, or copied to `to` where that is
// foreseen (odd strides of rows with a multiple of 8 columns are left to the kernels'
// own copies).  True if they are copied; p and ld are then the copy's.
bool add_rows(lora::PackArgs &c, int &matrices, const uint16_t *&p, uint32_t &ld, int cols, uint8_t *to) {
    if (rows_aligned(p, ld) || cols % 8 == 0) return false;
    c.from[matrices] = p;
    c.ld[matrices] = ld;
    c.cols[matrices] = cols;
    c.to[matrices++] = reinterpret_cast<uint16_t *>(to);
    p = reinterpret_cast<uint16_t *>(to);
    ld = static_cast<uint32_t>(lora::ld_packed(cols));
    return true;
}

}  // namespace

size_t lora_ws_bytes(int64_t tokens, int adapters, int r, int64_t k) {
    return partial_bytes(tokens, adapters, r, k) + lora::packed_bytes(tokens, k);
}

cudaError_t launch_lora_add(const LoraArgs &a, cudaStream_t stream) {
    const lora::FewArgs few{a.plan, a.w, a.x, a.ld_x, a.base, a.y, a.ld_base, a.ld_y, a.v, a.ld_v};
    if (lora::few(few, a.y_f32)) return lora::launch_few(few, a.y_f32, stream);
    lora::ShrinkArgs s{};
    s.plan = a.plan;
    s.x = a.x;
    s.ld_x = a.ld_x;
    s.w = a.w.a;
    s.stride_w = a.w.stride_a;
    s.ld_w = a.w.ld_a;
    s.lw = a.w;
    s.k = a.w.k;
    s.out = a.ws;
    s.err = error_word();
    if (s.err == nullptr) return cudaErrorUnknown;
    lora::PackArgs copies{};
    copies.plan = a.plan;
    int matrices = 0;
    s.packed = add_rows(copies, matrices, s.x, s.ld_x, a.w.k, reinterpret_cast<uint8_t *>(a.ws) + partial_bytes(a.plan.tokens, a.plan.adapters, a.w.r, a.w.k));
    cudaError_t e = matrices ? lora::launch_pack(copies, matrices, stream) : cudaSuccess;
    if (e == cudaSuccess) e = lora::launch_shrink(s, false, stream);
    if (e != cudaSuccess) return e;
    // Each CTA of a tile would add up its partial sums: left to them where there are
    // few tokens, one kernel more otherwise.
    const bool apart = a.plan.tokens > kLoraTile && (a.v != nullptr || lora::most_splits(a.plan, a.w.k, lora::padded(a.w.r)) > 1);
    if (apart) {
        e = lora::launch_sum({a.plan, a.w, a.ws, a.w.k, a.v, a.ld_v}, stream);
        if (e != cudaSuccess) return e;
    }
    lora::ExpandArgs x{};
    x.plan = a.plan;
    x.rows = a.ws;
    x.long_side = apart ? 0 : a.w.k;
    x.w = a.w.b;
    x.stride_w = a.w.stride_b;
    x.ld_w = a.w.ld_b;
    x.lw = a.w;
    x.n = a.w.n;
    x.base = a.base;
    x.y = a.y;
    x.ld_base = a.ld_base;
    x.ld_y = a.ld_y;
    x.v_out = apart ? nullptr : a.v;
    x.ld_v = a.ld_v;
    return lora::launch_expand(x, a.y_f32, stream);
}

namespace {

// The backward pass's workspace: dv's partial sums and its sum, v and dv in
// parts, the partial sums over the tokens, copies of dy and x.
struct Workspace {
    size_t partial, sum, vt, outer, dy, x, total;
    int chunks;
};
Workspace workspace_of(const LoraPlan &p, int r, int n, int k) {
    Workspace w;
    const size_t rows = static_cast<size_t>(p.tokens) * lora::padded(r) * sizeof(float);
    w.partial = partial_bytes(p.tokens, p.adapters, r, n);
    w.sum = rows;
    w.vt = lora::outer_vt_bytes(p, r);
    w.chunks = lora::outer_chunks(p, n, k, r);
    w.outer = 2 * static_cast<size_t>(w.chunks) * (static_cast<size_t>(n) + k) * lora::padded(r) * sizeof(float);
    w.dy = lora::packed_bytes(p.tokens, n);
    w.x = lora::packed_bytes(p.tokens, k);
    w.total = w.partial + w.sum + 2 * w.vt + w.outer + w.dy + w.x;
    return w;
}

}  // namespace

size_t lora_bwd_ws_bytes(int64_t tokens, int adapters, int r, int64_t n, int64_t k) {
    return workspace_of({nullptr, static_cast<int>(tokens), adapters}, r, static_cast<int>(n), static_cast<int>(k)).total;
}

cudaError_t launch_lora_add_bwd(const LoraBwdArgs &a, cudaStream_t stream) {
    const Workspace ws = workspace_of(a.plan, a.w.r, a.w.n, a.w.k);
    uint8_t *at = reinterpret_cast<uint8_t *>(a.ws);
    float *partial = reinterpret_cast<float *>(at), *sum = reinterpret_cast<float *>(at + ws.partial);
    uint16_t *vt0 = reinterpret_cast<uint16_t *>(at + ws.partial + ws.sum), *vt1 = vt0 + ws.vt / sizeof(uint16_t);
    float *parts = reinterpret_cast<float *>(vt1 + ws.vt / sizeof(uint16_t));
    uint8_t *copied = reinterpret_cast<uint8_t *>(parts) + ws.outer;
    const uint16_t *dy = a.dy, *xr = a.x;
    uint32_t ld_dy = a.ld_dy, ld_x = a.ld_x;
    lora::PackArgs copies{};
    copies.plan = a.plan;
    int matrices = 0;
    const int packed_dy = add_rows(copies, matrices, dy, ld_dy, a.w.n, copied);
    const int packed_x = a.da != nullptr && add_rows(copies, matrices, xr, ld_x, a.w.k, copied + ws.dy);
    cudaError_t e = matrices ? lora::launch_pack(copies, matrices, stream) : cudaSuccess;
    if (e != cudaSuccess) return e;
    const bool rows = a.dx != nullptr || a.da != nullptr, outer = a.da != nullptr || a.db != nullptr;
    if (rows) {
        lora::ShrinkArgs s{};
        s.plan = a.plan;
        s.x = dy;
        s.ld_x = ld_dy;
        s.packed = packed_dy;
        s.w = a.w.b;
        s.stride_w = a.w.stride_b;
        s.ld_w = a.w.ld_b;
        s.lw = a.w;
        s.k = a.w.n;
        s.out = partial;
        s.err = error_word();
        if (s.err == nullptr) return cudaErrorUnknown;
        e = lora::launch_shrink(s, true, stream);
        if (e != cudaSuccess) return e;
    }
    if (outer) {
        lora::PrepArgs p{};
        p.plan = a.plan;
        p.lw = a.w;
        p.v = a.db != nullptr ? a.v : nullptr;
        p.ld_v = a.ld_v;
        p.dv = a.da != nullptr ? partial : nullptr;
        p.long_side = a.w.n;
        p.sum = a.dx != nullptr ? sum : nullptr;
        p.vt[0] = vt0;
        p.vt[1] = vt1;
        p.parts = a.dw_f32 ? 3 : 2;
        e = lora::launch_prep(p, stream);
        if (e != cudaSuccess) return e;
        lora::OuterArgs o{};
        o.plan = a.plan;
        o.lw = a.w;
        o.f32 = a.dw_f32;
        o.err = error_word();
        if (o.err == nullptr) return cudaErrorUnknown;
        o.side[0] = {dy, ld_dy, a.w.n, 0, packed_dy, vt0, a.db, a.w.r, 1, static_cast<int64_t>(a.w.n) * a.w.r, parts};
        o.side[1] = {xr, ld_x, a.w.k, 0, packed_x, vt1, a.da, 1, a.w.k, static_cast<int64_t>(a.w.k) * a.w.r, nullptr};
        o.side[1].ws = parts + 2 * static_cast<size_t>(ws.chunks) * a.w.n * lora::padded(a.w.r);
        o.chunks = ws.chunks;
        e = lora::launch_outer(o, stream);
        if (e != cudaSuccess) return e;
    }
    if (a.dx == nullptr) return cudaSuccess;
    const bool summed = a.da != nullptr;    // by the kernel that took dv apart
    lora::ExpandArgs x{};
    x.plan = a.plan;
    x.rows = summed ? sum : partial;
    x.long_side = summed ? 0 : a.w.n;
    x.w = a.w.a;
    x.stride_w = a.w.stride_a;
    x.ld_w = a.w.ld_a;
    x.lw = a.w;
    x.n = a.w.k;
    x.base = a.base;
    x.y = a.dx;
    x.ld_base = a.ld_base;
    x.ld_y = a.ld_dx;
    return lora::launch_expand_t(x, a.dx_f32, stream);
}

}  // namespace fp8hg
