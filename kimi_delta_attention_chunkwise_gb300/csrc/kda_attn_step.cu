// kda_attn_step.cu -- kda_attn_step: one token of every sequence over a paged
// cache of the queries' type (the kernels: kda_attn_step.cuh).
#include "kda_attn_step.cuh"

namespace kda {

cudaError_t attn_step_workspace_bytes(const AttnStepArgs &a, size_t *bytes) {
    const int sms = device_sms();
    if (!sms) return cudaErrorUnknown;
    *bytes = with_core(a.D, a.G, a.dtype, [&](auto core) -> size_t {
        return part_bytes<decltype(core)>(a, sms);
    });
    return cudaSuccess;
}

cudaError_t launch_attn_step(const AttnStepArgs &a, cudaStream_t stream) {
    return with_core(a.D, a.G, a.dtype, [&](auto core) -> cudaError_t {
        return launch_core<decltype(core)>(a, stream);
    });
}

}  // namespace kda
