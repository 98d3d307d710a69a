// attention_e4m3.cu: the builds of the tensor-core attention kernel (attention.cuh) for caches of
// 8-bit floating point.
#include "attention.cuh"

namespace dflash {

cudaError_t launch_attention_e4m3(const DeviceInfo& dev, const AttentionArgs& a,
                               const AttentionProblem& p, bool few, uint32_t* status,
                               cudaStream_t stream) {
    return launch_for_cache<true>(dev, a, p, few, status, stream);
}

}  // namespace dflash
