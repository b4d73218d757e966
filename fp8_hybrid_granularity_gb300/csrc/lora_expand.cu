// Adapters: y from v and B (lora_expand.cuh).
#include "lora_expand.cuh"

namespace fp8hg {
namespace lora {

cudaError_t launch_expand(const ExpandArgs &a, bool f32, cudaStream_t stream) {
    return f32 ? by_rank<false, true>(a, stream) : by_rank<false, false>(a, stream);
}

}  // namespace lora
}  // namespace fp8hg
