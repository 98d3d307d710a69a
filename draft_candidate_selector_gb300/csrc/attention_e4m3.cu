// attention_e4m3.cu: the builds of the tensor-core attention kernel (attention.cuh) for caches of
// 8-bit floating point.
#include "attention.cuh"

namespace dflash {

cudaError_t launch_attention_e4m3(const DeviceInfo& dev, const AttentionArgs& a,
                                  const AttentionProblem& p, uint32_t* status,
                                  cudaStream_t stream) {
    static constexpr Launch launch[8] = {
        launch_on_tensor_cores<64, false, false, true>,  launch_on_tensor_cores<64, false, true, true>,
        launch_on_tensor_cores<64, true, false, true>,   launch_on_tensor_cores<64, true, true, true>,
        launch_on_tensor_cores<128, false, false, true>, launch_on_tensor_cores<128, false, true, true>,
        launch_on_tensor_cores<128, true, false, true>,  launch_on_tensor_cores<128, true, true, true>};
    return launch[(p.D == 128 ? 4 : 0) + (a.dtype == kFp16 ? 2 : 0) + (a.softcap > 0.f ? 1 : 0)](
        dev, a, p, status, stream);
}

}  // namespace dflash
