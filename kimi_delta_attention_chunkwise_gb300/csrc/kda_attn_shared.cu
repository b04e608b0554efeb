// kda_attn_shared.cu -- kda_attn_step_shared: one token of every sequence over a
// paged cache whose first pages the sequences share.
//
// With S shared tokens, a row's softmax is the join of its states over the
// tokens before and from S on.  The first part is a product of all sequences'
// queries of a key-value head with the same keys: one kernel takes blocks of
// (sequence, query head) rows over them, cut among several CTAs, and leaves a
// state (maximum, sum, weighted sum) per row and piece.  The second part is the
// step of kda_attn_step.cuh from token S on, whose CTAs start as those of the
// first leave; it leaves states, too, and a third kernel joins all of a row's.  A
// sequence that holds less than S tokens is all the step's.
#include "kda_attn_step.cuh"

namespace kda {
namespace {

constexpr int kMaxSplits = 64;
constexpr int kFewRows = 16;  // rows to a key-value head that the step's cores take

// Blocks of kRows rows over the shared tokens, on the step's cores: fp32, narrow
// heads, and so few rows that the tensor core's tiles would be all but empty.
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
    const PrefixLine line(a, shared);
    const int32_t c = (int32_t)blockIdx.x;
    if (c >= line.grid) return;
    const int32_t s = sharing_sequence<kThreads>(a, shared, &s_seq);
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

// Joins the states of an item of the step (a sequence's tokens under one block of
// query heads) with those of the shared tokens.  One CTA to an item; a warp
// takes one query head and every parts-th of its states: their maxima and sums
// one to a lane, then the weighted sums, four loads in flight.
template <int D, int R>
__global__ void __launch_bounds__(kJoinThreads) attn_shared_join_kernel(const AttnStepArgs a,
                                                                        const float *part,
                                                                        int32_t step_grid) {
    constexpr int N = (D + 31) / 32;  // columns per lane
    __shared__ int64_t s_scan[kJoinWarps], s_base;
    __shared__ float s_o[kJoinWarps][D], s_m[kJoinWarps], s_l[kJoinWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int32_t blocks = (a.G + R - 1) / R, items = a.HKV * blocks;
    const int32_t s = (int32_t)blockIdx.x / items, item = (int32_t)blockIdx.x - s * items;
    Line<kJoinThreads, true> line;
    line.scan(a, s_scan);
    line.base_of(a, s, items, &s_base);
    const int64_t units = line.total * items;
    const int32_t grid = workers(units, step_grid);
    const Span span = span_of<true>(a, s);
    const int32_t tiles = tiles_of(span.len());
    // the step's CTAs on the item
    const int64_t first = s_base + (int64_t)item * tiles, end = first + tiles;
    const int32_t c0 = tiles ? first_worker(units, first, grid) : 0;
    const int32_t own = tiles ? first_worker(units, end - 1, grid) - c0 + 1 : 0;
    const bool late = tiles && share_start(units, c0, grid) != first;  // c0's second slot
    const int32_t kvh = item / blocks, h0 = (item - kvh * blocks) * R;
    const int32_t rows = min(R, a.G - h0);
    const bool shares = span.first > 0;
    // the kernels before this one have ended
    tc::pdl_wait_primaries();
    int32_t abreast = 1;  // query heads at a time, a power of two
    while (abreast < rows && abreast < kJoinWarps) abreast *= 2;
    const int32_t parts = kJoinWarps / abreast;
    for (int32_t rb = 0; rb < rows; rb += abreast) {
        const int32_t r = rb + (warp & (abreast - 1));
        const int64_t row = (int64_t)s * a.HQ + (int64_t)kvh * a.G + h0 + r;
        float mx = -INFINITY, l = 0.f, o[N];
#pragma unroll
        for (int j = 0; j < N; ++j) o[j] = 0.f;
        if (r < rows) {
            const int32_t pieces = shares ? prefix_state(a, D, 0).pieces[row] : 0;
            const int32_t all = own + pieces;
            // state i: its weighted sums, maximum and sum
            auto state_of = [&](int32_t i, const float *&so, const float *&sm, const float *&sl) {
                if (i < own && own > 1) {
                    const float *slot = part + ((int64_t)(c0 + i) * 2 + (i == 0 && late ? 1 : 0)) *
                                                   (R * (D + 2));
                    so = slot + r * D;
                    sm = slot + R * D + r;
                    sl = slot + R * D + R + r;
                } else {
                    const PrefixState p = prefix_state(a, D, i < own ? a.splits - 1 : i - own);
                    so = p.o + row * D;
                    sm = p.m + row;
                    sl = p.l + row;
                }
            };
            for (int32_t i0 = warp / abreast; i0 < all; i0 += 32 * parts) {
                const int32_t i = i0 + lane * parts;
                float m = -INFINITY, sum = 0.f;
                if (i < all) {
                    const float *so, *sm, *sl;
                    state_of(i, so, sm, sl);
                    m = *sm;
                    sum = *sl;
                }
                float top = fmaxf(mx, m);
#pragma unroll
                for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                const float ref = top == -INFINITY ? 0.f : top;
                const float f = exp2f(mx - ref), w = exp2f(m - ref);
                sum *= w;
#pragma unroll
                for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                mx = top;
                l = l * f + sum;
#pragma unroll
                for (int j = 0; j < N; ++j) o[j] *= f;
                const int32_t n = min(32, (all - i0 + parts - 1) / parts);
#pragma unroll 4
                for (int32_t k = 0; k < n; ++k) {
                    const float wk = __shfl_sync(0xffffffffu, w, k);
                    const float *so, *sm, *sl;
                    state_of(i0 + k * parts, so, sm, sl);
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        if (D >= 32 || lane < D) o[j] += so[j * 32 + lane] * wk;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (D >= 32 || lane < D) s_o[warp][j * 32 + lane] = o[j];
        if (lane == 0) {
            s_m[warp] = mx;
            s_l[warp] = l;
        }
        __syncthreads();
        for (int i = tid; i < min(abreast, rows - rb) * D; i += kJoinThreads) {
            const int w0 = i / D, col = i % D;
            float m = s_m[w0];
            for (int w = w0 + abreast; w < kJoinWarps; w += abreast) m = fmaxf(m, s_m[w]);
            const float ref = m == -INFINITY ? 0.f : m;
            float y = 0.f, sum = 0.f;
            for (int w = w0; w < kJoinWarps; w += abreast) {
                const float f = exp2f(s_m[w] - ref);
                y += s_o[w][col] * f;
                sum += s_l[w] * f;
            }
            store_row(a, (int64_t)s * a.HQ + (int64_t)kvh * a.G + h0 + rb + w0, D, col, y, m, sum);
        }
        __syncthreads();
    }
}

// The step from the shared tokens on, and the join, each a programmatic dependent
// of the kernel before.
template <class Core>
cudaError_t launch_rest(const AttnStepArgs &a, cudaStream_t stream) {
    const int sms = device_sms();
    const int64_t items = step_items<Core>(a);
    if (items > INT32_MAX) return cudaErrorInvalidValue;
    const int32_t grid = line_grid<Core>(a, sms);
    float *part = static_cast<float *>(a.workspace);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr = follows_on();
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, attn_step_kernel<Core, true>, a, part);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)items);
    cfg.blockDim = dim3(kJoinThreads);
    return cudaLaunchKernelEx(&cfg, attn_shared_join_kernel<Core::kD, Core::kRows>, a,
                              static_cast<const float *>(part), grid);
}

// How a call's work on the shared tokens is cut, and its scratch in bytes.
struct Plan {
    bool tensor;
    int32_t rows, grid, splits;
    size_t part, prefix;
};

cudaError_t plan_of(const AttnStepArgs &a, Plan &p) {
    const int sms = device_sms();
    if (!sms) return cudaErrorUnknown;
    p.part = with_core(a.D, a.G, a.dtype, [&](auto core) -> size_t {
        return line_bytes<decltype(core)>(sms);
    });
    p.part = (p.part + 255) / 256 * 256;
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
    // no more CTAs than the longest line has tiles, and than kMaxSplits to an item
    const int64_t items = (int64_t)a.HKV * (((int64_t)a.N * a.G + p.rows - 1) / p.rows);
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
    if (e == cudaSuccess) *bytes = p.part + p.prefix;
    return e;
}

cudaError_t launch_attn_step_shared(const AttnStepArgs &args, cudaStream_t stream) {
    AttnStepArgs a = args;
    Plan p;
    cudaError_t e = plan_of(a, p);
    if (e != cudaSuccess) return e;
    a.splits = p.splits;
    a.prefix_rows = p.rows;
    a.prefix_grid = p.grid;
    a.prefix = static_cast<char *>(a.workspace) + p.part;
    if (p.tensor) {
        e = launch_prefix_tc(a, stream);
    } else {
        e = with_core(a.D, a.N * a.G, a.dtype, [&](auto core) -> cudaError_t {
            attn_prefix_kernel<decltype(core)><<<(unsigned)a.prefix_grid, kThreads, 0, stream>>>(a);
            return cudaGetLastError();
        });
    }
    if (e != cudaSuccess) return e;
    return with_core(a.D, a.G, a.dtype, [&](auto core) -> cudaError_t {
        return launch_rest<decltype(core)>(a, stream);
    });
}

}  // namespace kda
