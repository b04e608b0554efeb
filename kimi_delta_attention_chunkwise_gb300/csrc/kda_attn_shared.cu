// kda_attn_shared.cu -- kda_attn_step_shared: one token of every sequence over a
// paged cache whose first pages the sequences share.
//
// With S shared tokens, a row's softmax is the join of its states over the
// tokens before and from S on.  The first part is a product of all sequences'
// queries of a key-value head with the same keys: one kernel takes blocks of
// (sequence, query head) rows over them, cut among several CTAs, and leaves a
// state (maximum, sum, weighted sum) per row and piece.  The second part is a
// step from token S on, by warps for bf16 with d = 64 or 128, whose CTAs start on
// the SMs that the first leaves free; it leaves states, too, and a third kernel
// joins all of a row's.  A sequence that holds less than S tokens is all the
// step's.
//
// The plain step does it all (Plan::plain) where
//   * the table is short enough for its one launch of clusters: reading the shared
//     rows from L2 for every sequence takes less than three kernels do (192 + 50 tokens,
//     3 sequences, 8/2 heads, d = 64: 4.9 us, 11.6; 1024 + 100, 8 sequences, 32/8 heads,
//     d = 128: 10.7, 22; 1024 + 100, 32 fp32 sequences, 6/2 heads, d = 64: 10.5, 14);
//   * the CUDA-core blocks here would not be fewer than its own, as with 4, 8, ... query
//     heads to a key-value head, so that the shared keys are read as often, and it has
//     kPlainItems items or more (1-200 tokens behind 2304, 57 sequences, 16/2 heads, fp32,
//     d = 64: 40 us, 43; 32/8 heads, d = 16: 31, 37; behind 8192, 2 sequences, d = 128:
//     32/8 heads 28.9, 31.8; 16/2, 8 items, 18.9, 19.3, but at d = 64 14.4, 13.8; 8/2, 4
//     items, 15.0, 10.8).
#include "kda_attn_flat.cuh"

namespace kda {
namespace {

// Pieces to an item: more leave the step behind fewer SMs and the join more to read
// (65536 shared tokens, 64 sequences, 8/1 heads, d = 128: 64 pieces 32.1 us, one to an
// SM 37.2; 32768, 64 sequences, 8/2 heads, d = 64: 26.8, 29.5).
constexpr int kMaxSplits = 64;
// Rows to a key-value head that the step's cores take (65536 shared tokens, 32/8 heads,
// d = 128: 4 rows 55.6 us, the tensor core's tiles 62.0; 8 rows 57.7, 62.4; 16 rows
// 61.6, 62.0, but 33.7, 27.4 with 16/2 heads and 32.5, 25.2 with 8/1).
constexpr int kFewRows = 8;
constexpr int kPlainItems = 16;

// Blocks of kRows rows over the shared tokens, on the step's cores: fp32, narrow
// heads, and so few rows that the tensor core's tiles would be all but empty.
template <class Core>
__global__ void __launch_bounds__(kThreads, Core::kCtas) attn_prefix_kernel(const AttnStepArgs a) {
    using T = typename Core::Type;
    constexpr int D = Core::kD, R = Core::kRows;
    __shared__ Joined<Core> state;
    __shared__ int32_t s_seq;
    __shared__ unsigned long long s_own;
    const int tid = threadIdx.x, warp = tid >> 5;
    tc::pdl_launch_dependents();
    const int32_t shared = shared_tokens(a);
    if (blockIdx.x == 0 && tid == 0) check_shared_pages(a);
    const PrefixLine line(a, shared);
    const int32_t c = (int32_t)blockIdx.x;
    if (c >= line.grid) return;
    const int32_t s = sharing_sequence<kThreads>(a, shared, &s_seq, &s_own);
    if (s >= a.N) return;
    const int64_t u1 = share_start(line.units, c + 1, line.grid);
    Core core;
    for (int64_t u = share_start(line.units, c, line.grid); u < u1;) {
        const PrefixPiece piece(line, c, u, u1);
        const int32_t r0 = piece.block * R, rows = min(R, a.N * a.G - r0);
        core.init(
            [&](int r) {
                const int32_t n = (r0 + r) / a.G;
                return static_cast<const T *>(a.q) + n * a.q_stride +
                       (int64_t)(piece.kvh * a.G + (r0 + r - n * a.G)) * D;
            },
            rows, a.scale);
        const int32_t first = piece.tile0 * kPrefixTile;
        const int32_t end = piece.last ? shared : piece.tile1 * kPrefixTile;
        const bool seen = walk_tiles(a, core, s, piece.kvh, first, end, 0, tiles_of(end - first));
        core.finish(state.acc[warp], state.m[warp], state.l[warp], seen);
        __syncthreads();
        const PrefixState p = prefix_state(a, D, piece.index);
        for (int i = tid; i < rows * D; i += kThreads) {
            const int r = i / D, col = i % D;
            const int32_t n = (r0 + r) / a.G;
            const int64_t at = (int64_t)n * a.HQ + piece.kvh * a.G + (r0 + r - n * a.G);
            float o, mx, sum;
            state.get(r, i, o, mx, sum);
            p.o[at * D + col] = o;
            if (col == 0) {
                p.m[at] = mx;
                p.l[at] = sum;
                if (piece.last) p.pieces[at] = piece.index + 1;
            }
        }
        __syncthreads();
        u += piece.tile1 - piece.tile0;
    }
}

// The step's core behind the shared tokens.
template <class F>
auto with_rest_core(int32_t D, int32_t G, int32_t dtype, F f) {
    if (dtype == KDA_DTYPE_BF16 && D == 64) {
        if (G <= 4) return f(MmaCore<64, 1, true, __nv_bfloat16, true>{});
        if (G <= 8) return f(MmaCore<64, 1, false, __nv_bfloat16, true>{});
        return f(MmaCore<64, 2, false, __nv_bfloat16, true>{});
    }
    if (dtype == KDA_DTYPE_BF16 && D == 128) {
        if (G <= 4) return f(MmaCore<128, 1, true, __nv_bfloat16, true>{});
        if (G <= 8) return f(MmaCore<128, 1, false, __nv_bfloat16, true>{});
        return f(MmaCore<128, 2, false, __nv_bfloat16, true>{});
    }
    if (dtype == KDA_DTYPE_BF16)
        return D == 16 ? with_rows<__nv_bfloat16, 16, __nv_bfloat16>(G, f)
                       : with_rows<__nv_bfloat16, 32, __nv_bfloat16>(G, f);
    switch (D) {
        case 16: return with_rows<float, 16, float>(G, f);
        case 32: return with_rows<float, 32, float>(G, f);
        case 64: return with_rows<float, 64, float>(G, f);
        default: return with_rows<float, 128, float>(G, f);
    }
}

// Scratch of the step's parts.
template <class Core>
size_t rest_bytes(int sms) {
    if constexpr (Core::kAhead) return flat_part_bytes<Core>(sms);
    else return line_bytes<Core>(sms);
}

// The step from the shared tokens on, and the join, each a programmatic dependent
// of the kernel before.
template <class Core>
cudaError_t launch_rest(const AttnStepArgs &a, int sms, cudaStream_t stream) {
    float *part = static_cast<float *>(a.workspace);
    cudaError_t e;
    if constexpr (Core::kAhead) {
        e = launch_flat<Core, true>(a, part, sms, stream);
    } else {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr = follows_on();
        cfg.stream = stream;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        cfg.gridDim = dim3((unsigned)line_grid<Core>(a, sms));
        cfg.blockDim = dim3(kThreads);
        e = cudaLaunchKernelEx(&cfg, attn_step_kernel<Core, true>, a, part);
    }
    return e != cudaSuccess ? e : launch_rows_join<Core, true>(a, part, sms, stream);
}

// How a call's work on the shared tokens is cut, and its scratch in bytes.
struct Plan {
    bool plain;  // kda_attn_step's kernels do it all
    bool tensor;
    int32_t rows, grid, splits;
    size_t part, owners, prefix;  // in this order
};

cudaError_t plan_of(const AttnStepArgs &a, Plan &p) {
    const int sms = device_sms();
    if (!sms) return cudaErrorUnknown;
    with_rest_core(a.D, a.G, a.dtype, [&](auto core) -> int {
        using Core = decltype(core);
        p.part = (rest_bytes<Core>(sms) + 255) / 256 * 256;
        p.owners = owners_bytes<Core>(a);
        return 0;
    });
    p.tensor = a.dtype == KDA_DTYPE_BF16 && a.D >= 64 && (int64_t)a.N * a.G > kFewRows;
    int64_t slots = sms;
    if (p.tensor) {
        p.rows = prefix_tc_rows(a);
    } else {
        with_core(a.D, a.N * a.G, a.dtype, [&](auto core) -> int {
            using Core = decltype(core);
            p.rows = Core::kRows;
            slots = (int64_t)sms * Core::kCtas;
            return 0;
        });
    }
    const int64_t items = (int64_t)a.HKV * (((int64_t)a.N * a.G + p.rows - 1) / p.rows);
    p.plain = with_core(a.D, a.G, a.dtype, [&](auto core) -> bool {
        using Core = decltype(core);
        const int64_t own = step_items<Core>(a);
        return step_direct_ctas<Core>(a, sms) || (!p.tensor && own <= items && own >= kPlainItems);
    });
    if (p.plain) {
        p.owners = p.prefix = 0;
        return attn_step_workspace_bytes(a, &p.part);
    }
    // no more CTAs than the longest line has tiles, and than kMaxSplits to an item
    const int64_t capacity = (int64_t)a.max_pages << a.page_shift;
    const int64_t tiles = std::max<int64_t>(1, (capacity + kPrefixTile - 1) / kPrefixTile);
    const int64_t most = std::min<int64_t>(tiles, kMaxSplits);
    p.grid = (int32_t)std::min(slots, items * most);
    // an item's pieces: the shares that start in it (grid / items, rounded up) and
    // the one before them; and a row's own tokens' state
    p.splits = (int32_t)((p.grid + items - 1) / items + 2);
    p.prefix = prefix_bytes((int64_t)a.N * a.HQ, a.D, p.splits);
    return cudaSuccess;
}

}  // namespace

cudaError_t attn_step_shared_workspace_bytes(const AttnStepArgs &a, size_t *bytes) {
    Plan p;
    const cudaError_t e = plan_of(a, p);
    if (e == cudaSuccess) *bytes = p.part + p.owners + p.prefix;
    return e;
}

cudaError_t launch_attn_step_shared(const AttnStepArgs &args, cudaStream_t stream) {
    AttnStepArgs a = args;
    Plan p;
    cudaError_t e = plan_of(a, p);
    if (e != cudaSuccess) return e;
    // (the step behind takes its rows by copies wherever the widths are the tensor core's)
    const bool waits = a.withhold == KDA_WITHHOLD_SHARED ? p.tensor
                                                         : a.dtype == KDA_DTYPE_BF16 && a.D >= 64;
    if (a.withhold && (p.plain || !waits)) return cudaErrorNotSupported;
    if (p.plain) return launch_attn_step(a, stream);
    a.splits = p.splits;
    a.prefix_rows = p.rows;
    a.prefix_grid = p.grid;
    a.prefix_sms = p.tensor ? device_sms() : 0;
    char *ws = static_cast<char *>(a.workspace);
    a.owners = reinterpret_cast<int2 *>(ws + p.part);
    a.prefix = ws + p.part + p.owners;
    if (p.tensor) {
        e = launch_prefix_tc(a, stream);
    } else {
        e = with_core(a.D, a.N * a.G, a.dtype, [&](auto core) -> cudaError_t {
            attn_prefix_kernel<decltype(core)><<<(unsigned)a.prefix_grid, kThreads, 0, stream>>>(a);
            return cudaGetLastError();
        });
    }
    if (e != cudaSuccess) return e;
    return with_rest_core(a.D, a.G, a.dtype, [&](auto core) -> cudaError_t {
        return launch_rest<decltype(core)>(a, device_sms(), stream);
    });
}

}  // namespace kda
