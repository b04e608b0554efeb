// kda_attn_api.cu -- the C entry points of the full-attention layer: host
// validation, engine choice, scratch and launch.  See include/kda.h.
#include <cmath>
#include <cstdint>

#include "kda_attn.cuh"

namespace kda {
namespace {

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

kdaStatus_t cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return KDA_SUCCESS;
    (void)cudaGetLastError();
    return KDA_ERR_CUDA;
}

size_t element_size(const kdaAttnShape_t *s) { return s->dtype == KDA_DTYPE_BF16 ? 2 : 4; }

// A token stride as given, or the contiguous one for 0.
int64_t token_stride(int64_t given, int32_t heads, int32_t d) {
    return given ? given : (int64_t)heads * d;
}

bool stride_ok(int64_t stride, int32_t heads, int32_t d, size_t es) {
    if (stride == 0) return true;
    return stride >= (int64_t)heads * d && (stride * (int64_t)es) % 16 == 0 &&
           stride <= ((int64_t)1 << 36);
}

// The kernels work with scale * log2(e), a positive finite float.
bool scale_ok(float scale) { return scale > 0.f && std::isfinite(scale * 1.4426950408889634f); }

kdaStatus_t check_attn_shape(const kdaAttnShape_t *s) {
    if (!s) return KDA_ERR_INVALID_ARG;
    if (s->num_seqs < 1 || s->total_tokens < 0 || s->num_heads < 1 || s->num_kv_heads < 1 ||
        s->num_heads % s->num_kv_heads != 0 || s->head_dim < 1)
        return KDA_ERR_INVALID_ARG;
    if (s->dtype != KDA_DTYPE_BF16 && s->dtype != KDA_DTYPE_F32) return KDA_ERR_INVALID_ARG;
    if (s->out_f32 != 0 && s->out_f32 != 1) return KDA_ERR_INVALID_ARG;
    const size_t es = element_size(s);
    if (!stride_ok(s->q_stride, s->num_heads, s->head_dim, es) ||
        !stride_ok(s->k_stride, s->num_kv_heads, s->head_dim, es) ||
        !stride_ok(s->v_stride, s->num_kv_heads, s->head_dim, es))
        return KDA_ERR_INVALID_ARG;
    const int32_t d = s->head_dim;
    if (d != 16 && d != 32 && d != 64 && d != 128) return KDA_ERR_UNSUPPORTED;
    if (s->num_heads / s->num_kv_heads > 128) return KDA_ERR_UNSUPPORTED;
    if (s->num_heads > 65535) return KDA_ERR_UNSUPPORTED;  // (documented)
    // (the kernels' walks over the sequences add up to N + 1 to an index in int32)
    if (s->num_seqs > (1 << 30)) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)s->total_tokens * s->num_heads > INT32_MAX ||
        (int64_t)s->num_seqs * s->num_heads > INT32_MAX)
        return KDA_ERR_UNSUPPORTED;  // (token, head) counts travel as int32
    return KDA_SUCCESS;
}

kdaStatus_t check_cache(const kdaPagedCache_t *c, int32_t *page_shift) {
    if (!c || c->num_pages < 0 || c->max_pages < 0) return KDA_ERR_INVALID_ARG;
    switch (c->page_size) {
        case 16: *page_shift = 4; break;
        case 32: *page_shift = 5; break;
        case 64: *page_shift = 6; break;
        case 128: *page_shift = 7; break;
        case 256: *page_shift = 8; break;
        default: return c->page_size < 1 ? KDA_ERR_INVALID_ARG : KDA_ERR_UNSUPPORTED;
    }
    if ((int64_t)c->max_pages * c->page_size > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    if (c->num_pages > 0 && (!c->k || !c->v)) return KDA_ERR_INVALID_ARG;
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return KDA_ERR_INVALID_ARG;
    if (c->max_pages > 0 && !c->block_table) return KDA_ERR_INVALID_ARG;
    if (!aligned(c->block_table, 4)) return KDA_ERR_INVALID_ARG;
    return KDA_SUCCESS;
}

// A cache of 8-bit codes as one of any type, and its scales.
kdaStatus_t check_cache_q8(const kdaPagedCacheQ8_t *c, kdaPagedCache_t &same) {
    if (!c) return KDA_ERR_INVALID_ARG;
    if (c->num_pages > 0 && (!c->k_scale || !c->v_scale)) return KDA_ERR_INVALID_ARG;
    if (!aligned(c->k_scale, 16) || !aligned(c->v_scale, 16)) return KDA_ERR_INVALID_ARG;
    same = {c->k, c->v, c->block_table, c->num_pages, c->page_size, c->max_pages};
    return KDA_SUCCESS;
}

// What the step's sizes say, before its pointers.
kdaStatus_t step_sizes(const kdaPagedCache_t *cache, const kdaAttnShape_t *shape, AttnStepArgs &a) {
    kdaStatus_t st = check_attn_shape(shape);
    if (st != KDA_SUCCESS) return st;
    int32_t page_shift = 0;
    st = check_cache(cache, &page_shift);
    if (st != KDA_SUCCESS) return st;
    if (shape->total_tokens != shape->num_seqs) return KDA_ERR_INVALID_ARG;
    a.num_pages = cache->num_pages; a.page_shift = page_shift; a.max_pages = cache->max_pages;
    a.N = shape->num_seqs; a.HQ = shape->num_heads; a.HKV = shape->num_kv_heads;
    a.G = a.HQ / a.HKV; a.D = shape->head_dim; a.dtype = shape->dtype;
    a.out_f32 = shape->dtype == KDA_DTYPE_F32 ? 1 : shape->out_f32;
    a.workspace = nullptr;
    a.status = nullptr;
    a.k_scale = a.v_scale = nullptr;
    a.shared_pages = nullptr;
    a.prefix = nullptr;
    a.owners = nullptr;
    a.splits = a.prefix_rows = a.prefix_grid = a.prefix_sms = 0;
    a.wait_limit = kStepWait;
    a.withhold = KDA_WITHHOLD_NONE;
    return KDA_SUCCESS;
}

kdaStatus_t plan_attn_step(const void *q, const kdaPagedCache_t *cache, const int32_t *seq_lens,
                           float scale, void *out, float *lse, const kdaAttnShape_t *shape,
                           AttnStepArgs &a) {
    const kdaStatus_t st = step_sizes(cache, shape, a);
    if (st != KDA_SUCCESS) return st;
    if (!scale_ok(scale)) return KDA_ERR_INVALID_ARG;
    if (!q || !aligned(q, 16) || !out || !aligned(out, 16) || out == q) return KDA_ERR_INVALID_ARG;
    if (!seq_lens || !aligned(seq_lens, 4) || !aligned(lse, 4)) return KDA_ERR_INVALID_ARG;
    a.q = q;
    a.q_stride = token_stride(shape->q_stride, shape->num_heads, shape->head_dim);
    a.k_cache = cache->k; a.v_cache = cache->v; a.block_table = cache->block_table;
    a.seq_lens = seq_lens; a.scale = scale; a.out = out; a.lse = lse;
    return KDA_SUCCESS;
}

// The arguments of an append (nothing is written to `a` that a call without
// tokens would need).
kdaStatus_t plan_append(const void *q, const void *k, const void *v, const int32_t *cu_seqlens,
                        const int32_t *cache_lens, const kdaRope_t *rope, void *q_out, void *k_out,
                        const kdaPagedCache_t *cache, const kdaAttnShape_t *shape, AppendArgs &a) {
    kdaStatus_t st = check_attn_shape(shape);
    if (st != KDA_SUCCESS) return st;
    int32_t page_shift = 0;
    st = check_cache(cache, &page_shift);
    if (st != KDA_SUCCESS) return st;
    if (!cu_seqlens && shape->num_seqs != 1 && shape->num_seqs != shape->total_tokens)
        return KDA_ERR_INVALID_ARG;
    if (!cache_lens || !aligned(cache_lens, 4) || !aligned(cu_seqlens, 4))
        return KDA_ERR_INVALID_ARG;
    if (!q && q_out) return KDA_ERR_INVALID_ARG;
    if (q && !q_out) return KDA_ERR_INVALID_ARG;
    if (shape->total_tokens > 0 && (!k || !v)) return KDA_ERR_INVALID_ARG;
    const void *vec[] = {q, k, v, q_out, k_out};
    for (const void *p : vec)
        if (!aligned(p, 16)) return KDA_ERR_INVALID_ARG;
    a.q_stride = token_stride(shape->q_stride, shape->num_heads, shape->head_dim);
    a.k_stride = token_stride(shape->k_stride, shape->num_kv_heads, shape->head_dim);
    a.v_stride = token_stride(shape->v_stride, shape->num_kv_heads, shape->head_dim);
    // in place: a row's output must be the row itself
    if (q && q_out == q && a.q_stride != (int64_t)shape->num_heads * shape->head_dim)
        return KDA_ERR_INVALID_ARG;
    if (k_out && k_out == k && a.k_stride != (int64_t)shape->num_kv_heads * shape->head_dim)
        return KDA_ERR_INVALID_ARG;
    if (rope) {
        if (!rope->table || !aligned(rope->table, 16) || rope->num_positions < 0 ||
            (rope->interleaved != 0 && rope->interleaved != 1) || rope->rot_dim < 1)
            return KDA_ERR_INVALID_ARG;
        if (rope->rot_dim % 16 != 0 || rope->rot_dim > shape->head_dim) return KDA_ERR_UNSUPPORTED;
    }
    if (shape->total_tokens == 0) return KDA_SUCCESS;
    a.q = q; a.k = k; a.v = v;
    a.cu_seqlens = cu_seqlens;
    a.one_each = !cu_seqlens && shape->num_seqs == shape->total_tokens;
    a.cache_lens = cache_lens;
    a.rope = rope ? rope->table : nullptr;
    a.positions = rope ? rope->num_positions : 0;
    a.rot = rope ? rope->rot_dim : 0;
    a.interleaved = rope ? rope->interleaved : 0;
    a.q_out = q_out; a.k_out = k_out;
    a.k_cache = cache->k; a.v_cache = cache->v; a.block_table = cache->block_table;
    a.num_pages = cache->num_pages; a.page_shift = page_shift; a.max_pages = cache->max_pages;
    a.N = shape->num_seqs; a.T = shape->total_tokens;
    a.HQ = q ? shape->num_heads : 0; a.HKV = shape->num_kv_heads; a.D = shape->head_dim;
    a.dtype = shape->dtype;
    a.k_scale = a.v_scale = nullptr;
    a.k_stored = a.v_stored = nullptr;
    return KDA_SUCCESS;
}

kdaStatus_t run_append(AppendArgs &a, cudaError_t (*launch)(const AppendArgs &, cudaStream_t),
                       cudaStream_t stream) {
    a.status = device_status_word();
    if (!a.status) return cuda_status(cudaErrorUnknown);
    return cuda_status(launch(a, stream));
}

// A step's scratch and launch, by kind.
using StepBytes = cudaError_t (*)(const AttnStepArgs &, size_t *);
using StepLaunch = cudaError_t (*)(const AttnStepArgs &, cudaStream_t);

// With the caller's scratch.
kdaStatus_t run_step_ws(AttnStepArgs &a, StepBytes bytes, StepLaunch launch, void *workspace,
                        size_t workspace_bytes, cudaStream_t stream) {
    if (!aligned(workspace, 256)) return KDA_ERR_INVALID_ARG;
    size_t need = 0;
    const kdaStatus_t st = cuda_status(bytes(a, &need));
    if (st != KDA_SUCCESS) return st;
    if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_INVALID_ARG;
    a.workspace = workspace;
    a.status = device_status_word();
    if (!a.status) return cuda_status(cudaErrorUnknown);
    const cudaError_t e = launch(a, stream);
    return a.withhold && e == cudaErrorNotSupported ? KDA_ERR_UNSUPPORTED : cuda_status(e);
}

// What the diagnostic forms say besides.
kdaStatus_t diagnose(AttnStepArgs &a, int32_t withhold, int64_t wait_cycles) {
    if (withhold < KDA_WITHHOLD_NONE || withhold > KDA_WITHHOLD_SHARED) return KDA_ERR_INVALID_ARG;
    a.withhold = withhold;
    if (wait_cycles > 0) a.wait_limit = wait_cycles;
    return KDA_SUCCESS;
}

// With scratch taken on the stream.
kdaStatus_t run_step(AttnStepArgs &a, StepBytes bytes, StepLaunch launch, cudaStream_t stream) {
    size_t need = 0;
    const kdaStatus_t st = cuda_status(bytes(a, &need));
    if (st != KDA_SUCCESS) return st;
    a.status = device_status_word();
    if (!a.status) return cuda_status(cudaErrorUnknown);
    if (need == 0) return cuda_status(launch(a, stream));
    void *ws = nullptr;
    if (cudaMallocAsync(&ws, need, stream) != cudaSuccess) {
        (void)cudaGetLastError();
        return KDA_ERR_CUDA;
    }
    a.workspace = ws;
    const cudaError_t e = launch(a, stream);
    const cudaError_t f = cudaFreeAsync(ws, stream);
    return cuda_status(e != cudaSuccess ? e : f);
}

// kda_attn_step_q8's arguments
kdaStatus_t plan_step_q8(const void *q, const kdaPagedCacheQ8_t *cache, const int32_t *seq_lens,
                         float scale, void *out, float *lse, const kdaAttnShape_t *shape,
                         AttnStepArgs &a) {
    kdaPagedCache_t same;
    kdaStatus_t st = check_cache_q8(cache, same);
    if (st != KDA_SUCCESS) return st;
    st = plan_attn_step(q, &same, seq_lens, scale, out, lse, shape, a);
    if (st != KDA_SUCCESS) return st;
    a.k_scale = cache->k_scale;
    a.v_scale = cache->v_scale;
    return KDA_SUCCESS;
}

// kda_attn_step_shared's arguments
kdaStatus_t plan_step_shared(const void *q, const kdaPagedCache_t *cache, const int32_t *seq_lens,
                             const int32_t *shared_pages, float scale, void *out, float *lse,
                             const kdaAttnShape_t *shape, AttnStepArgs &a) {
    const kdaStatus_t st = plan_attn_step(q, cache, seq_lens, scale, out, lse, shape, a);
    if (st != KDA_SUCCESS) return st;
    if (!shared_pages || !aligned(shared_pages, 4)) return KDA_ERR_INVALID_ARG;
    a.shared_pages = shared_pages;
    return KDA_SUCCESS;
}

}  // namespace

int device_sms() {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
    if (dev < 64) n = known[dev].load(std::memory_order_relaxed);
    if (n) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace kda

using namespace kda;

extern "C" {

kdaStatus_t kda_attn_fwd(const void *q, const void *k, const void *v, float scale,
                         const int32_t *cu_seqlens, void *out, float *lse,
                         const kdaAttnShape_t *shape, cudaStream_t stream) {
    kdaStatus_t st = check_attn_shape(shape);
    if (st != KDA_SUCCESS) return st;
    if (shape->engine < KDA_ENGINE_AUTO || shape->engine > KDA_ENGINE_SIMT)
        return KDA_ERR_INVALID_ARG;
    if (!scale_ok(scale)) return KDA_ERR_INVALID_ARG;
    if (!cu_seqlens && shape->num_seqs != 1) return KDA_ERR_INVALID_ARG;
    if (!aligned(cu_seqlens, 4) || !aligned(lse, 4)) return KDA_ERR_INVALID_ARG;
    if (shape->total_tokens > 0) {
        const void *vec[] = {q, k, v, out};
        for (const void *p : vec)
            if (!p || !aligned(p, 16)) return KDA_ERR_INVALID_ARG;
        if (out == q || out == k || out == v) return KDA_ERR_INVALID_ARG;  // read after written
    }
    const bool tensor_ok = shape->dtype == KDA_DTYPE_BF16 &&
                           (shape->head_dim == 64 || shape->head_dim == 128);
    if (shape->engine == KDA_ENGINE_TENSOR && !tensor_ok) return KDA_ERR_UNSUPPORTED;
    // (items index a one-dimensional grid; the smallest tiles have 16 rows)
    if ((int64_t)shape->total_tokens * shape->num_heads / 16 +
            (int64_t)shape->num_seqs * shape->num_kv_heads > INT32_MAX)
        return KDA_ERR_UNSUPPORTED;
    if (shape->total_tokens == 0) return KDA_SUCCESS;
    AttnArgs a;
    a.q = q; a.k = k; a.v = v;
    a.q_stride = token_stride(shape->q_stride, shape->num_heads, shape->head_dim);
    a.k_stride = token_stride(shape->k_stride, shape->num_kv_heads, shape->head_dim);
    a.v_stride = token_stride(shape->v_stride, shape->num_kv_heads, shape->head_dim);
    a.cu_seqlens = cu_seqlens; a.scale = scale; a.out = out; a.lse = lse;
    a.N = shape->num_seqs; a.T = shape->total_tokens;
    a.HQ = shape->num_heads; a.HKV = shape->num_kv_heads; a.G = a.HQ / a.HKV;
    a.D = shape->head_dim; a.dtype = shape->dtype;
    a.out_f32 = shape->dtype == KDA_DTYPE_F32 ? 1 : shape->out_f32;
    a.status = device_status_word();
    if (!a.status) return cuda_status(cudaErrorUnknown);
    return cuda_status(tensor_ok && shape->engine != KDA_ENGINE_SIMT ? launch_attn_tc(a, stream)
                                                                     : launch_attn_simt(a, stream));
}

kdaStatus_t kda_cache_append(const void *q, const void *k, const void *v,
                             const int32_t *cu_seqlens, const int32_t *cache_lens,
                             const kdaRope_t *rope, void *q_out, void *k_out,
                             const kdaPagedCache_t *cache, const kdaAttnShape_t *shape,
                             cudaStream_t stream) {
    AppendArgs a;
    const kdaStatus_t st =
        plan_append(q, k, v, cu_seqlens, cache_lens, rope, q_out, k_out, cache, shape, a);
    if (st != KDA_SUCCESS || shape->total_tokens == 0) return st;
    return run_append(a, launch_cache_append, stream);
}

kdaStatus_t kda_cache_append_q8(const void *q, const void *k, const void *v,
                                const int32_t *cu_seqlens, const int32_t *cache_lens,
                                const kdaRope_t *rope, void *q_out, void *k_out, void *k_stored,
                                void *v_stored, const kdaPagedCacheQ8_t *cache,
                                const kdaAttnShape_t *shape, cudaStream_t stream) {
    kdaPagedCache_t same;
    kdaStatus_t st = check_cache_q8(cache, same);
    if (st != KDA_SUCCESS) return st;
    AppendArgs a;
    st = plan_append(q, k, v, cu_seqlens, cache_lens, rope, q_out, k_out, &same, shape, a);
    if (st != KDA_SUCCESS) return st;
    // what the codes stand for lies in tensors of its own
    const void *others[] = {q, k, v, q_out, k_out};
    for (const void *p : others)
        if ((k_stored && k_stored == p) || (v_stored && v_stored == p)) return KDA_ERR_INVALID_ARG;
    if ((k_stored && k_stored == v_stored) || !aligned(k_stored, 16) || !aligned(v_stored, 16))
        return KDA_ERR_INVALID_ARG;
    if (shape->total_tokens == 0) return KDA_SUCCESS;
    a.k_scale = cache->k_scale; a.v_scale = cache->v_scale;
    a.k_stored = k_stored; a.v_stored = v_stored;
    return run_append(a, launch_cache_append_q8, stream);
}

kdaStatus_t kda_attn_step_workspace_size(const kdaPagedCache_t *cache, const kdaAttnShape_t *shape,
                                         size_t *bytes) {
    if (!bytes) return KDA_ERR_INVALID_ARG;
    AttnStepArgs a;
    const kdaStatus_t st = step_sizes(cache, shape, a);
    if (st != KDA_SUCCESS) return st;
    return cuda_status(attn_step_workspace_bytes(a, bytes));
}

kdaStatus_t kda_attn_step_ws(const void *q, const kdaPagedCache_t *cache, const int32_t *seq_lens,
                             float scale, void *out, float *lse, const kdaAttnShape_t *shape,
                             void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    AttnStepArgs a;
    const kdaStatus_t st = plan_attn_step(q, cache, seq_lens, scale, out, lse, shape, a);
    if (st != KDA_SUCCESS) return st;
    return run_step_ws(a, attn_step_workspace_bytes, launch_attn_step, workspace, workspace_bytes,
                       stream);
}

kdaStatus_t kda_attn_step(const void *q, const kdaPagedCache_t *cache, const int32_t *seq_lens,
                          float scale, void *out, float *lse, const kdaAttnShape_t *shape,
                          cudaStream_t stream) {
    AttnStepArgs a;
    const kdaStatus_t st = plan_attn_step(q, cache, seq_lens, scale, out, lse, shape, a);
    if (st != KDA_SUCCESS) return st;
    return run_step(a, attn_step_workspace_bytes, launch_attn_step, stream);
}

kdaStatus_t kda_attn_step_q8_workspace_size(const kdaPagedCacheQ8_t *cache,
                                            const kdaAttnShape_t *shape, size_t *bytes) {
    if (!bytes) return KDA_ERR_INVALID_ARG;
    kdaPagedCache_t same;
    kdaStatus_t st = check_cache_q8(cache, same);
    if (st != KDA_SUCCESS) return st;
    AttnStepArgs a;
    st = step_sizes(&same, shape, a);
    if (st != KDA_SUCCESS) return st;
    return cuda_status(attn_step_q8_workspace_bytes(a, bytes));
}

kdaStatus_t kda_attn_step_q8_ws(const void *q, const kdaPagedCacheQ8_t *cache,
                                const int32_t *seq_lens, float scale, void *out, float *lse,
                                const kdaAttnShape_t *shape, void *workspace,
                                size_t workspace_bytes, cudaStream_t stream) {
    AttnStepArgs a;
    const kdaStatus_t st = plan_step_q8(q, cache, seq_lens, scale, out, lse, shape, a);
    if (st != KDA_SUCCESS) return st;
    return run_step_ws(a, attn_step_q8_workspace_bytes, launch_attn_step_q8, workspace,
                       workspace_bytes, stream);
}

kdaStatus_t kda_attn_step_q8_ws_diag(const void *q, const kdaPagedCacheQ8_t *cache,
                                     const int32_t *seq_lens, float scale, void *out, float *lse,
                                     const kdaAttnShape_t *shape, void *workspace,
                                     size_t workspace_bytes, int32_t withhold, int64_t wait_cycles,
                                     cudaStream_t stream) {
    AttnStepArgs a;
    kdaStatus_t st = plan_step_q8(q, cache, seq_lens, scale, out, lse, shape, a);
    if (st == KDA_SUCCESS) st = diagnose(a, withhold, wait_cycles);
    if (st != KDA_SUCCESS) return st;
    return run_step_ws(a, attn_step_q8_workspace_bytes, launch_attn_step_q8, workspace,
                       workspace_bytes, stream);
}

kdaStatus_t kda_attn_step_q8(const void *q, const kdaPagedCacheQ8_t *cache,
                             const int32_t *seq_lens, float scale, void *out, float *lse,
                             const kdaAttnShape_t *shape, cudaStream_t stream) {
    AttnStepArgs a;
    const kdaStatus_t st = plan_step_q8(q, cache, seq_lens, scale, out, lse, shape, a);
    if (st != KDA_SUCCESS) return st;
    return run_step(a, attn_step_q8_workspace_bytes, launch_attn_step_q8, stream);
}

kdaStatus_t kda_attn_step_shared_workspace_size(const kdaPagedCache_t *cache,
                                                const kdaAttnShape_t *shape, size_t *bytes) {
    if (!bytes) return KDA_ERR_INVALID_ARG;
    AttnStepArgs a;
    const kdaStatus_t st = step_sizes(cache, shape, a);
    if (st != KDA_SUCCESS) return st;
    return cuda_status(attn_step_shared_workspace_bytes(a, bytes));
}

kdaStatus_t kda_attn_step_shared_ws(const void *q, const kdaPagedCache_t *cache,
                                    const int32_t *seq_lens, const int32_t *shared_pages,
                                    float scale, void *out, float *lse,
                                    const kdaAttnShape_t *shape, void *workspace,
                                    size_t workspace_bytes, cudaStream_t stream) {
    AttnStepArgs a;
    const kdaStatus_t st =
        plan_step_shared(q, cache, seq_lens, shared_pages, scale, out, lse, shape, a);
    if (st != KDA_SUCCESS) return st;
    return run_step_ws(a, attn_step_shared_workspace_bytes, launch_attn_step_shared, workspace,
                       workspace_bytes, stream);
}

kdaStatus_t kda_attn_step_shared_ws_diag(const void *q, const kdaPagedCache_t *cache,
                                         const int32_t *seq_lens, const int32_t *shared_pages,
                                         float scale, void *out, float *lse,
                                         const kdaAttnShape_t *shape, void *workspace,
                                         size_t workspace_bytes, int32_t withhold,
                                         int64_t wait_cycles, cudaStream_t stream) {
    AttnStepArgs a;
    kdaStatus_t st = plan_step_shared(q, cache, seq_lens, shared_pages, scale, out, lse, shape, a);
    if (st == KDA_SUCCESS) st = diagnose(a, withhold, wait_cycles);
    if (st != KDA_SUCCESS) return st;
    return run_step_ws(a, attn_step_shared_workspace_bytes, launch_attn_step_shared, workspace,
                       workspace_bytes, stream);
}

kdaStatus_t kda_attn_step_shared(const void *q, const kdaPagedCache_t *cache,
                                 const int32_t *seq_lens, const int32_t *shared_pages, float scale,
                                 void *out, float *lse, const kdaAttnShape_t *shape,
                                 cudaStream_t stream) {
    AttnStepArgs a;
    const kdaStatus_t st =
        plan_step_shared(q, cache, seq_lens, shared_pages, scale, out, lse, shape, a);
    if (st != KDA_SUCCESS) return st;
    return run_step(a, attn_step_shared_workspace_bytes, launch_attn_step_shared, stream);
}

}  // extern "C"
