// kda_attn_step.cu -- kda_attn_step: one token of every sequence over a paged
// cache of the queries' type (the kernels: kda_attn_step.cuh).
#include "kda_attn_step.cuh"

namespace kda {

cudaError_t attn_step_workspace_bytes(const AttnStepArgs &a, size_t *bytes) {
    const int sms = device_sms();
    if (!sms) return cudaErrorUnknown;
    *bytes = with_core(a.D, a.G, a.dtype, [&](auto core) -> size_t {
        using Core = decltype(core);
        return step_direct_ctas<Core>(a, sms) ? 0 : line_bytes<Core>(sms);
    });
    return cudaSuccess;
}

cudaError_t launch_attn_step(const AttnStepArgs &a, cudaStream_t stream) {
    const int sms = device_sms();
    if (!sms) return cudaErrorUnknown;
    return with_core(a.D, a.G, a.dtype, [&](auto core) -> cudaError_t {
        using Core = decltype(core);
        if (const int ctas = step_direct_ctas<Core>(a, sms)) return launch_direct<Core>(a, ctas, stream);
        return launch_line<Core>(a, sms, stream);
    });
}

}  // namespace kda
