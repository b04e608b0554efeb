// kda_attn_step_q8.cu -- kda_attn_step_q8: one token of every sequence over a
// paged cache of 8-bit codes (the cores and the kernels for short tables:
// kda_attn_step.cuh; the kernel for others: kda_attn_flat.cuh).
//
//     z_j = scale ks_j <q, kcode_j>,  o = sum_j e^{z_j} vs_j vcode_j / sum_j e^{z_j}
//
// A token's key and value are 2 D bytes of codes and 8 of scales to a key-value
// head, half of what a bf16 cache holds.  The scales stay outside the products,
// which are products of codes that both 16-bit types hold exactly, summed in fp32
// (MmaCore says how).
#include "kda_attn_flat.cuh"

namespace kda {
namespace {

using Bf16 = __nv_bfloat16;

// The core of a problem, as a call of f(Core{}).
template <class F>
auto with_core_q8(int32_t D, int32_t G, int32_t dtype, F f) {
    if (dtype == KDA_DTYPE_BF16) {
        switch (D) {
            case 16: return with_rows<Bf16, 16, int8_t>(G, f);
            case 32: return with_rows<Bf16, 32, int8_t>(G, f);
            case 64:
                if (G <= 4) return f(MmaCore<64, 1, true, int8_t>{});
                if (G <= 8) return f(MmaCore<64, 1, false, int8_t>{});
                return f(MmaCore<64, 2, false, int8_t>{});
            default:
                if (G <= 4) return f(MmaCore<128, 1, true, int8_t>{});
                if (G <= 8) return f(MmaCore<128, 1, false, int8_t>{});
                return f(MmaCore<128, 2, false, int8_t>{});
        }
    }
    switch (D) {
        case 16: return with_rows<float, 16, int8_t>(G, f);
        case 32: return with_rows<float, 32, int8_t>(G, f);
        case 64: return with_rows<float, 64, int8_t>(G, f);
        default: return with_rows<float, 128, int8_t>(G, f);
    }
}

// Scratch: workers' parts, then owners (none for short tables).
template <class Core>
size_t q8_bytes(const AttnStepArgs &a, int sms) {
    if (step_direct_ctas<Core>(a, sms)) return 0;
    if constexpr (Core::kAhead) return flat_part_bytes<Core>(sms) + owners_bytes<Core>(a);
    else return line_bytes<Core>(sms);
}

template <class Core>
cudaError_t launch_q8(AttnStepArgs a, int sms, cudaStream_t stream) {
    const int ctas = step_direct_ctas<Core>(a, sms);
    if (a.withhold && (ctas || !Core::kAhead || a.withhold != KDA_WITHHOLD_STEP))
        return cudaErrorNotSupported;
    if (ctas) return launch_direct<Core>(a, ctas, stream);
    if constexpr (Core::kAhead) {
        float *part = static_cast<float *>(a.workspace);
        a.owners = reinterpret_cast<int2 *>(static_cast<char *>(a.workspace) +
                                            flat_part_bytes<Core>(sms));
        const cudaError_t e = launch_flat<Core, false>(a, part, sms, stream);
        return e != cudaSuccess ? e : launch_rows_join<Core, false>(a, part, sms, stream);
    } else {
        return launch_line<Core>(a, sms, stream);
    }
}

}  // namespace

cudaError_t attn_step_q8_workspace_bytes(const AttnStepArgs &a, size_t *bytes) {
    const int sms = device_sms();
    if (!sms) return cudaErrorUnknown;
    *bytes = with_core_q8(a.D, a.G, a.dtype, [&](auto core) -> size_t {
        return q8_bytes<decltype(core)>(a, sms);
    });
    return cudaSuccess;
}

cudaError_t launch_attn_step_q8(const AttnStepArgs &a, cudaStream_t stream) {
    const int sms = device_sms();
    if (!sms) return cudaErrorUnknown;
    return with_core_q8(a.D, a.G, a.dtype, [&](auto core) -> cudaError_t {
        return launch_q8<decltype(core)>(a, sms, stream);
    });
}

}  // namespace kda
