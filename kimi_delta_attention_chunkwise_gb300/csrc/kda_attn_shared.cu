// kda_attn_shared.cu -- kda_attn_step_shared: one token of every sequence over a
// paged cache whose first pages the sequences share.
//
// With S shared tokens, a row's softmax is the join of its states over the
// tokens before and from S on.  The first part is a product of all sequences'
// queries of a key-value head with the same keys: one kernel takes blocks of
// (sequence, query head) rows over them, cut among several CTAs, and leaves a
// state (maximum, sum, weighted sum) per row and cut.  The second part is the
// step of kda_attn_step.cuh, which starts at token S, runs beside the first and
// joins its states as it writes a row out.  A sequence that holds less than S
// tokens is all the step's.
#include "kda_attn_step.cuh"

namespace kda {
namespace {

constexpr int kMaxSplits = 64;

// Rows of the shared tokens' products: (sequence, query head) pairs of one
// key-value head, block by block.  CTA: item (key-value head, block), and a cut
// of the tokens.
template <class Core>
__global__ void __launch_bounds__(kThreads, Core::kCtas) attn_prefix_kernel(const AttnStepArgs a) {
    using T = typename Core::Type;
    constexpr int D = Core::kD, R = Core::kRows;
    __shared__ Joined<Core> state;
    __shared__ int32_t s_seq;
    const int tid = threadIdx.x, warp = tid >> 5;
    tc::pdl_launch_dependents();
    const int32_t shared = shared_tokens(a);
    if (blockIdx.x == 0 && tid == 0 && (*a.shared_pages < 0 || *a.shared_pages > a.max_pages))
        *a.status = KDA_ERR_INVALID_ARG;
    const int32_t all = a.N * a.G, blocks = all / R + (all % R != 0);
    const int32_t items = a.HKV * blocks;
    const int32_t item = (int32_t)(blockIdx.x % (uint32_t)items);
    const int32_t split = (int32_t)(blockIdx.x / (uint32_t)items);
    const int32_t tiles = prefix_tiles(shared), cuts = min(a.splits, tiles);
    if (split >= cuts) return;
    const int32_t s = sharing_sequence<kThreads>(a, shared, &s_seq);
    if (s >= a.N) return;
    const int32_t kvh = item / blocks, r0 = (item - kvh * blocks) * R, rows = min(R, all - r0);
    // the row's place among all rows (sequence * HQ + query head)
    auto place = [&](int r) -> int64_t {
        const int32_t n = (r0 + r) / a.G;
        return (int64_t)n * a.HQ + kvh * a.G + (r0 + r - n * a.G);
    };
    Core core;
    core.init(
        [&](int r) {
            const int32_t n = (r0 + r) / a.G;
            return static_cast<const T *>(a.q) + n * a.q_stride +
                   (int64_t)(kvh * a.G + (r0 + r - n * a.G)) * D;
        },
        rows, a.scale);
    const int32_t first = (int32_t)((int64_t)tiles * split / cuts) * kPrefixTile;
    const int32_t last = (int32_t)((int64_t)tiles * (split + 1) / cuts);
    const int32_t end = last == tiles ? shared : last * kPrefixTile;
    const bool seen = walk_tiles(a, core, s, kvh, first, end, 0, tiles_of(end - first));
    core.finish(state.acc[warp], state.m[warp], state.l[warp], seen);
    __syncthreads();
    const PrefixState p = prefix_state(a, D, split);
    for (int i = tid; i < rows * D; i += kThreads) {
        const int r = i / D, col = i % D;
        const int64_t at = place(r);
        float o, mx, sum;
        state.get(r, i, o, mx, sum);
        p.o[at * D + col] = o;
        if (col == 0) {
            p.m[at] = mx;
            p.l[at] = sum;
        }
    }
}

// What a call takes: the kernels' cores, cuts of the shared tokens and scratch.
struct Plan {
    int32_t splits;
    size_t part, prefix;  // bytes
};

// Cuts that let `items` rows' blocks fill `slots` places, no more than the
// table has room for.
int32_t cuts_for(const AttnStepArgs &a, int64_t items, int64_t slots) {
    const int64_t capacity = (int64_t)a.max_pages << a.page_shift;
    const int64_t tiles = std::max<int64_t>(1, (capacity + kPrefixTile - 1) / kPrefixTile);
    return (int32_t)std::max<int64_t>(1, std::min({slots / items, tiles, (int64_t)kMaxSplits}));
}

template <class Core>
int64_t prefix_items(const AttnStepArgs &a) {
    return (int64_t)a.HKV * (((int64_t)a.N * a.G + Core::kRows - 1) / Core::kRows);
}

cudaError_t plan_of(const AttnStepArgs &a, Plan &p) {
    const int sms = device_sms();
    if (!sms) return cudaErrorUnknown;
    p.part = with_core(a.D, a.G, a.dtype, [&](auto core) -> size_t {
        return part_bytes<decltype(core)>(a, sms);
    });
    p.part = (p.part + 255) / 256 * 256;
    p.splits = with_core(a.D, a.N * a.G, a.dtype, [&](auto core) -> int32_t {
        using Core = decltype(core);
        return cuts_for(a, prefix_items<Core>(a), (int64_t)sms * Core::kCtas);
    });
    p.prefix = (size_t)p.splits * a.N * a.HQ * (a.D + 2) * sizeof(float);
    return cudaSuccess;
}

}  // namespace

cudaError_t attn_step_shared_workspace_bytes(const AttnStepArgs &a, size_t *bytes) {
    Plan p;
    const cudaError_t e = plan_of(a, p);
    if (e == cudaSuccess) *bytes = p.part + p.prefix;
    return e;
}

cudaError_t launch_attn_step_shared(const AttnStepArgs &args, cudaStream_t stream) {
    AttnStepArgs a = args;
    Plan p;
    cudaError_t e = plan_of(a, p);
    if (e != cudaSuccess) return e;
    a.splits = p.splits;
    a.prefix = static_cast<char *>(a.workspace) + p.part;
    e = with_core(a.D, a.N * a.G, a.dtype, [&](auto core) -> cudaError_t {
        using Core = decltype(core);
        attn_prefix_kernel<Core>
            <<<(unsigned)(prefix_items<Core>(a) * a.splits), kThreads, 0, stream>>>(a);
        return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
    return with_core(a.D, a.G, a.dtype, [&](auto core) -> cudaError_t {
        return launch_core<decltype(core), true>(a, stream);
    });
}

}  // namespace kda
