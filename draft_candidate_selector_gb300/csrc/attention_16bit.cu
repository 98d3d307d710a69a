// attention_16bit.cu: the builds of the tensor-core attention kernel (attention.cuh) for 16-bit caches.
#include "attention.cuh"

namespace dflash {

cudaError_t launch_attention_16bit(const DeviceInfo& dev, const AttentionArgs& a,
                               const AttentionProblem& p, bool few, uint32_t* status,
                               cudaStream_t stream) {
    return launch_for_cache<false>(dev, a, p, few, status, stream);
}

}  // namespace dflash
