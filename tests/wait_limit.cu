// One CTA of a few warps on a barrier that nobody completes, each for limit_ns:
// out[0] counts the warps whose wait ran out, out[1] the longest of them in ns.
// Then one that has been completed.
#include "../fp8_hybrid_granularity_gb300/csrc/ptx.cuh"

using namespace fp8hg;

__global__ void k_wait(uint32_t limit_ns, unsigned long long *out) {
    __shared__ __align__(8) uint64_t bars[2];
    const uint32_t never = ptx::smem_u32(bars), done = never + 8;
    if (threadIdx.x == 0) {
        ptx::mbar_init(never, 1);
        ptx::mbar_init(done, 1);
        ptx::fence_mbar_init();
        ptx::mbar_arrive(done);
    }
    __syncthreads();
    const uint64_t t0 = ptx::globaltimer();
    const bool came = ptx::mbar_wait_ns(never, 0, limit_ns);
    const uint64_t t1 = ptx::globaltimer();
    if ((threadIdx.x & 31) == 0) {
        if (!came) atomicAdd(out, 1ull);
        atomicMax(out + 1, t1 - t0);
        if (ptx::mbar_wait_ns(done, 0, limit_ns)) atomicAdd(out + 2, 1ull);
    }
}

// out: three zeroed counters on the device.
extern "C" int wait_limit(unsigned int limit_ns, unsigned long long *out) {
    k_wait<<<1, 128>>>(limit_ns, out);
    return static_cast<int>(cudaDeviceSynchronize());
}
