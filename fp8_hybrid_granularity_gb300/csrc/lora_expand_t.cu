// Adapters: dx from dv and A (lora_expand.cuh).
#include "lora_expand.cuh"

namespace fp8hg {
namespace lora {

cudaError_t launch_expand_t(const ExpandArgs &a, bool f32, cudaStream_t stream) {
    return f32 ? by_rank<true, true>(a, stream) : by_rank<true, false>(a, stream);
}

}  // namespace lora
}  // namespace fp8hg
