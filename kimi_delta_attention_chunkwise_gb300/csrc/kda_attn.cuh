// kda_attn.cuh -- declarations shared by the full-attention layer's translation
// units.  Not part of the public ABI (that is include/kda.h).
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "kda.h"

namespace kda {

// Arguments after validation (kda_attn_api.cu); strides in elements, never 0.
struct AttnArgs {
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const int32_t *cu_seqlens;     // device [N + 1] or nullptr (one sequence)
    float scale;
    void *out;                     // [T, HQ, D]
    float *lse;                    // [T, HQ] or nullptr
    int32_t N, T, HQ, HKV, G, D;   // G = HQ / HKV
    int32_t dtype, out_f32;
    int *status;
};
cudaError_t launch_attn_simt(const AttnArgs &a, cudaStream_t stream);
// tcgen05 engine (kda_attn_tc.cu): bf16, D = 64 or 128.
cudaError_t launch_attn_tc(const AttnArgs &a, cudaStream_t stream);

struct AppendArgs {
    const void *q, *k, *v;         // q may be nullptr
    int64_t q_stride, k_stride, v_stride;
    const int32_t *cu_seqlens;     // nullptr: see one_each
    int32_t one_each;              // no offsets: token t is sequence t (else one sequence)
    const int32_t *cache_lens;     // [N]
    const float *rope;             // [P, rot] or nullptr
    int32_t positions, rot, interleaved;
    void *q_out, *k_out;           // may be nullptr
    void *k_cache, *v_cache;
    const int32_t *block_table;
    int32_t num_pages, page_shift, max_pages;
    int32_t N, T, HQ, HKV, D, dtype;
    int *status;
};
cudaError_t launch_cache_append(const AppendArgs &a, cudaStream_t stream);

struct AttnStepArgs {
    const void *q;
    int64_t q_stride;
    const void *k_cache, *v_cache;
    const int32_t *block_table;
    int32_t num_pages, page_shift, max_pages;
    const int32_t *seq_lens;       // [N]
    float scale;
    void *out;                     // [N, HQ, D]
    float *lse;                    // [N, HQ] or nullptr
    int32_t N, HQ, HKV, G, D, dtype, out_f32;
    void *workspace;
    int *status;
};
// Scratch of the step on the current device, for these sizes and any lengths.
cudaError_t attn_step_workspace_bytes(const AttnStepArgs &a, size_t *bytes);
cudaError_t launch_attn_step(const AttnStepArgs &a, cudaStream_t stream);

// Device address of the status word on the current device (kda_api.cu).
int *device_status_word();

// SMs of the current device, asked for once per device (kda_attn_api.cu; 0:
// the query failed).
int device_sms();

// Raises a kernel's dynamic shared memory limit, once per device.
template <auto Kernel>
cudaError_t allow_smem(size_t bytes) {
    static std::atomic<uint64_t> done{0};  // one bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

}  // namespace kda
