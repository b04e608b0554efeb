// kda_attn_flat.cuh -- the step's line of tiles cut among warps: kda_attn_step_q8's
// and kda_attn_step_shared's kernels for bf16 queries with D = 64 or 128, and the
// join that both end with.
//
// The units, 16 or 32 tokens of a (sequence, head) item, form one line, of which
// every warp takes an equal share.  A warp's units come to shared memory in a
// ring of its own, ahead of the one it works on and across the borders of items:
// neighbouring rows of a page, one copy of keys and one of values (and two of
// scales).  Nothing in the loop waits for another warp, and short items cost no
// start of their own.  At the end of an item the warp writes the item's results, or
// its part's state for the join.
//
// Rows come by 4-D tensor copies with a swizzle that leaves the core's reads free of
// bank conflicts (8-bit, 64 sequences of 512-8192 tokens, 32/8 heads, d = 128: 112 us,
// 5.8 TB/s of 6.8; by bulk copies of rows with conflicts 130; by kda_attn_step's
// kernel, whose CTAs share a tile of 64 tokens and hold the next one's rows in
// registers, 155).  Rows are read once, and say so to L2: without that the calls that
// follow each other take 5 us more, and one behind writes that fill L2 16.
// What the kernel takes is the bytes at the memory's rate and about 15 us: 3 for the
// line's sums and the first look-ups, 5 for the join, and the rest for SMs that get
// less of the memory than others (their last warps end 12 us after the first SMs').
// Shares that CTAs take from blocks that have not started, or blocks of their own at
// the end of the line, cost as much as they even out or 9 us more.
#pragma once

#include <cstring>

#include "kda_attn_ptx.cuh"
#include "kda_attn_step.cuh"

namespace kda {
namespace {

constexpr int kJoinGroups = kJoinThreads / 8;

// Where a warp is in the line: unit `tile` of `tiles` of sequence s under key-value
// head kvh and block `block` of its query heads.  `at`: its place in the line, where
// every item's units come behind COST places for what the item takes besides them.
template <bool SHARED, int UNIT, int COST>
struct LineCursor {
    int64_t at;
    int32_t s, kvh, block, tile, tiles, first, end;
    __device__ void enter(const AttnStepArgs &a, int32_t seq) {
        s = seq;
        const Span span = span_of<SHARED>(a, s);
        first = span.first;
        end = span.end;
        tiles = tiles_of<UNIT>(span.len());
    }
    // the first unit at place u or behind it, u being one of sequence seq's, whose
    // places start at base
    __device__ void seek(const AttnStepArgs &a, int32_t blocks, int32_t seq, int64_t base, int64_t u) {
        enter(a, seq);
        const int32_t item = (int32_t)((u - base) / (tiles + COST));
        const int32_t off = (int32_t)((u - base) - (int64_t)item * (tiles + COST));
        tile = max(off - COST, 0);
        at = u + max(COST - off, 0);
        kvh = item / blocks;
        block = item - kvh * blocks;
    }
    // the next unit, which may be behind the line
    __device__ int64_t after() const { return at + (tile + 1 < tiles ? 1 : 1 + COST); }
    // goes there (there is one)
    __device__ void next(const AttnStepArgs &a, int32_t blocks) {
        at = after();
        if (++tile < tiles) return;
        tile = 0;
        if (++block < blocks) return;
        block = 0;
        if (++kvh < a.HKV) return;
        kvh = 0;
        do enter(a, s + 1);
        while (tiles == 0);
    }
    __device__ int32_t token() const { return first + tile * UNIT; }
};

template <class Core>
struct FlatCfg {
    static constexpr uint32_t ROW = Core::kPanels * Core::kPanel;  // bytes of a key
    // what an SM's CTAs leave of its shared memory, in 16 tokens to a warp
    static constexpr uint32_t BLOCK = 2 * kWarpTokens * ROW;
    static constexpr uint32_t SCALES = Core::kScaled ? 2 * kWarpTokens * 4 : 0;
    static constexpr int ROOM = (228 * 1024 / Core::kCtas - 4096) / (int)(kWarps * (BLOCK + SCALES));
    // 32 tokens to a unit where two units of them fit: what a unit costs besides
    // its tokens is a third of the instructions
    static constexpr int SUB = ROOM >= 4 ? 2 : 1, UNIT = SUB * kWarpTokens;
    static constexpr int RING = ROOM / SUB < 4 ? ROOM / SUB : 4;  // units
    // what an item takes besides its units (queries, results), in units: behind 16384
    // shared tokens, 256 sequences of 1-600 tokens, whose shares hold a few items or
    // tens, took 12 us more without it
    static constexpr int COST = SUB == 2 ? 1 : 2;
    static constexpr uint32_t PANEL = UNIT * Core::kPanel;        // a panel of a unit's keys
    static constexpr uint32_t HALF = Core::kPanels * PANEL;       // a unit's keys, or values
    static constexpr uint32_t SMEM = kWarps * RING * SUB * (BLOCK + SCALES);
    static_assert(RING >= 2 && RING * SUB <= 32, "shared memory of an SM");
    static_assert(PANEL % 1024 == 0 && (Core::kPanels == 1 || SUB == 1), "swizzled tiles");
};

// The heads of the cache's pages as tensors.
struct FlatMaps {
    CUtensorMap k, v;
};

// The workers' shares of the line: `early` of them have 16 parts of it each, the
// others `late` (SmSplit).  No share is smaller than LEAST, unless there is one.
template <int LEAST>
struct FlatShares {
    int64_t units, parts;
    int32_t early, late, number;
    // equal shares
    __device__ FlatShares(int64_t n, int32_t most) : units(n), late(16) {
        number = early = n > 0 ? max(workers(n / LEAST, most), 1) : 0;
        parts = 16 * (int64_t)early;
    }
    __device__ FlatShares(int64_t n, int32_t most, int32_t first, int32_t weight)
        : FlatShares(n, most) {
        const int64_t all = 16 * (int64_t)first + weight * (int64_t)(most - first);
        if (first <= 0 || weight >= 16 || n < LEAST * (int64_t)first) return;
        if (weight == 0 || n * weight < LEAST * all) {
            number = early = first;
            parts = 16 * (int64_t)first;
        } else {
            early = first;
            late = weight;
            number = most;
            parts = all;
        }
    }
    __device__ int64_t start(int32_t c) const {
        const int64_t at = c <= early ? 16 * (int64_t)c : 16 * (int64_t)early + late * (int64_t)(c - early);
        return units * at / parts;
    }
    // the worker that has unit u: the last that starts at or before it
    __device__ int32_t at(int64_t u) const {
        const int64_t w = ((u + 1) * parts - 1) / units, e = 16 * (int64_t)early;
        return (int32_t)(w < e ? w / 16 : early + (w - e) / late);
    }
};

// Neighbouring channels of a row's result from its state (mx = -inf: no keys).
template <int N>
__device__ __forceinline__ void store_run(const AttnStepArgs &a, int64_t head, int D, int ch,
                                          const float (&o)[N], float mx, float sum) {
    float y[N];
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = mx == -INFINITY ? 0.f : o[i] / sum;
    if constexpr (N < 4) {
#pragma unroll
        for (int i = 0; i < N; ++i) store_out(a, head * D + ch + i, y[i]);
    } else if (a.out_f32) {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + head * D + ch + i) =
                make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + head * D + ch + i) =
                make_uint2(tc::pack_bf16x2(y[i], y[i + 1]), tc::pack_bf16x2(y[i + 2], y[i + 3]));
    }
    if (a.lse && ch == 0) a.lse[head] = mx == -INFINITY ? -INFINITY : (mx + log2f(sum)) * kLn2;
}

template <class Core, bool SHARED>
__global__ void __launch_bounds__(kThreads, Core::kCtas)
attn_flat_kernel(const AttnStepArgs a, float *part, const __grid_constant__ FlatMaps maps) {
    using T = typename Core::Type;
    using Cfg = FlatCfg<Core>;
    constexpr int D = Core::kD, R = Core::kRows, RING = Cfg::RING, SUB = Cfg::SUB;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ int64_t s_scan[2 * kWarps], s_base[kWarps];
    __shared__ int32_t s_seq[kWarps];
    __shared__ uint64_t s_full[kWarps][RING];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    tc::pdl_launch_dependents();
    if (tc::smem_u32(smem) & 1023u) {  // (the swizzle goes by addresses)
        *a.status = KDA_ERR_CUDA;
        return;
    }
    const int32_t blocks = (a.G + R - 1) / R;  // blocks of query heads
    const int32_t items = a.HKV * blocks;
    // rows of a copy, and copies to a unit
    const int32_t box = min(1 << a.page_shift, Cfg::UNIT), copies = Cfg::UNIT / box;
    if (tid == 0) {
        for (int w = 0; w < kWarps; ++w)
            for (int x = 0; x < RING; ++x)
                tc::mbar_init(&s_full[w][x], copies + (a.withhold == KDA_WITHHOLD_STEP &&
                                                       blockIdx.x == 0 && w == 0 && x == 0));
        tc::fence_mbar_init();
        tc::fence_proxy_async();
    }
    constexpr int COST = Cfg::COST;
    Line<kThreads, SHARED, Cfg::UNIT, COST> line;
    line.scan(a, s_scan);
    // (a share of more than COST places has a unit)
    using Shares = FlatShares<COST + 2>;
    Shares shares(line.total * items, (int32_t)gridDim.x * kWarps);
    if (SHARED && a.prefix_sms && (int32_t)gridDim.x == a.prefix_sms * Core::kCtas) {
        // (where no sequence holds the shared tokens, nobody works on them: 16 sequences
        // of 500-2000 tokens, 65536 said to be shared, 51 us where SMs were left for that, 25)
        const PrefixLine prefix(a, line.shares ? shared_tokens(a) : 0);
        const SmSplit split = sm_split(a, prefix, line.tokens);
        shares = Shares(line.total * items, (int32_t)gridDim.x * kWarps,
                        (a.prefix_sms - split.prefix) * Core::kCtas * kWarps, split.late);
    }
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const int32_t c = (int32_t)blockIdx.x * kWarps + w;
        if (c < shares.number) line.look(a, shares.start(c), items, &s_seq[w], &s_base[w]);
    }
    __syncthreads();
    const int32_t c = (int32_t)blockIdx.x * kWarps + warp;  // this worker
    if (c < shares.number) {
        const int64_t u0 = shares.start(c), u1 = shares.start(c + 1);
        uint8_t *ring = smem + warp * (RING * 2 * Cfg::HALF);
        float *scales = reinterpret_cast<float *>(smem + kWarps * RING * 2 * Cfg::HALF) +
                        warp * (RING * 2 * Cfg::UNIT);  // (kScaled)
        uint64_t *full = s_full[warp];
        uint32_t good = 0;   // a bit per 16 tokens in the ring: they are there
        uint32_t phase = 0;  // a bit per unit's barrier
        LineCursor<SHARED, Cfg::UNIT, COST> here, ahead;
        here.seek(a, blocks, s_seq[warp], s_base[warp], u0);
        ahead = here;
        // lane i < SUB: the i-th 16 tokens of the unit at `ahead`, and the entry of the
        // page that they lie in
        const int32_t mine = min(lane, SUB - 1) * kWarpTokens;
        auto entry_of = [&]() -> int32_t {
            const int32_t tok = ahead.token() + mine;
            return tok < ahead.end
                       ? a.block_table[(int64_t)ahead.s * a.max_pages + (tok >> a.page_shift)]
                       : 0;
        };
        bool more = true;  // there is a unit at `ahead`
        int32_t units_ahead = 0;  // copied and not worked on yet
        int32_t page = entry_of();
        // starts the copies of the unit at `ahead` to place x of the ring: whole boxes
        // (what lies behind the sequence is put out of the way in values())
        auto copy_next = [&](int32_t x) {
            if (!more) return;
            const int32_t tok = ahead.token() + mine, n = min(kWarpTokens, ahead.end - tok);
            const bool there = page >= 0 && page < a.num_pages, ok = there && n > 0;
            if (n > 0 && !there) *a.status = KDA_ERR_INVALID_ARG;
            if (lane < copies) {
                if (!ok) {
                    tc::mbar_arrive(&full[x]);
                } else {
                    const int64_t z = (int64_t)page * a.HKV + ahead.kvh;
                    const int32_t at = tok & ((1 << a.page_shift) - 1);
                    uint8_t *to = ring + x * (2 * Cfg::HALF) + mine * Core::kPanel;
                    tc::mbar_arrive_expect_tx(
                        &full[x], box * (2 * Cfg::ROW + (Core::kScaled ? 8 : 0)));
                    tma_load_4d_once(to, &maps.k, 0, at, 0, (int32_t)z, &full[x]);
                    tma_load_4d_once(to + Cfg::HALF, &maps.v, 0, at, 0, (int32_t)z, &full[x]);
                    if constexpr (Core::kScaled) {
                        const int64_t row = (z << a.page_shift) + at;
                        float *f = scales + x * (2 * Cfg::UNIT) + mine;
                        tc::bulk_g2s(f, a.k_scale + row, box * 4, &full[x]);
                        tc::bulk_g2s(f + Cfg::UNIT, a.v_scale + row, box * 4, &full[x]);
                    }
                }
            }
            constexpr uint32_t all = (1u << SUB) - 1;
            good = (good & ~(all << (x * SUB))) |
                   ((__ballot_sync(0xffffffffu, ok) & all) << (x * SUB));
            ++units_ahead;
            more = ahead.after() < u1;
            if (more) {
                ahead.next(a, blocks);
                page = entry_of();
            }
        };
        auto wait = [&](int32_t x) -> bool {
            const uint32_t p = phase >> x & 1;
            phase ^= 1u << x;
            const bool done = tc::mbar_try_wait(&full[x], p) ||
                              tc::mbar_wait_bounded(&full[x], p, a.wait_limit);
            return __all_sync(0xffffffffu, done);
        };
#pragma unroll
        for (int i = 0; i < RING; ++i) copy_next(i);
        Core core;
        core.places();
        int32_t x = 0;  // the place in the ring
        bool fresh = true, seen = false, first_item = true;
        for (bool last = false; !last;) {
            const int32_t rows = min(R, a.G - here.block * R);
            const int64_t head = (int64_t)here.kvh * a.G + here.block * R;
            if (fresh) {
                const T *qp = static_cast<const T *>(a.q) + here.s * a.q_stride + head * D;
                core.init([&](int h) { return qp + h * D; }, rows, a.scale);
                fresh = seen = false;
            }
            if (!wait(x)) {
                *a.status = KDA_ERR_TIMEOUT;
                phase ^= 1u << x;  // (its copy may land yet)
                break;
            }
            --units_ahead;
            const uint32_t blocks_good = good >> (x * SUB);
            const int32_t left = here.end - here.token();
#pragma unroll
            for (int b = 0; b < SUB; ++b) {
                const bool ok = blocks_good >> b & 1;
                const int n = min(kWarpTokens, left - b * kWarpTokens);
                if (ok) {
                    uint8_t *keys = ring + x * (2 * Cfg::HALF) + b * kWarpTokens * Core::kPanel;
                    uint8_t *values = keys + Cfg::HALF;
                    float *f = scales + x * (2 * Cfg::UNIT) + b * kWarpTokens;
                    if (n < kWarpTokens) {
                        // behind the sequence: zero values, or scales, since 0 times
                        // an infinity or a NaN would be a NaN
                        if constexpr (Core::kScaled) {
                            if ((lane & 15) >= n) f[(lane & 15) + (lane >> 4) * Cfg::UNIT] = 0.f;
                        } else {
#pragma unroll
                            for (int p = 0; p < Core::kPanels; ++p)
                                for (uint32_t i = n * Core::kPanel / 16 + lane;
                                     i < kWarpTokens * Core::kPanel / 16; i += 32)
                                    reinterpret_cast<uint4 *>(values + p * Cfg::PANEL)[i] =
                                        make_uint4(0, 0, 0, 0);
                        }
                        tc::fence_proxy_async();  // before copies to this place
                        __syncwarp();
                    }
                    core.fetch_k(keys, Cfg::PANEL, f);
                    core.scores();
                    core.fetch_v(values, Cfg::PANEL, f + Cfg::UNIT);
                }
                if (b == SUB - 1) {
                    __syncwarp();
                    copy_next(x);
                }
                if (ok) {
                    core.values(n);
                    seen = true;
                }
            }
            x = x + 1 == RING ? 0 : x + 1;
            const bool ends = here.tile + 1 == here.tiles;
            last = here.after() >= u1;
            if (ends || last) {
                const int64_t first = here.at - here.tile;  // the item's first unit
                const bool whole = ends && first >= u0;
                const int64_t row = (int64_t)here.s * a.HQ + head;
                if (whole && !SHARED) {
                    core.finish_rows(seen, rows, [&](int h, int ch, auto &y, float m, float l) {
                        store_run(a, row + h, D, ch, y, m, l);
                    });
                } else {
                    // a whole item's state, or the worker's first or last part's
                    float *to, *to_m, *to_l;
                    if (whole) {
                        const PrefixState p = prefix_state(a, D, a.splits - 1);
                        to = p.o + row * D;
                        to_m = p.m + row;
                        to_l = p.l + row;
                    } else {
                        to = part + ((int64_t)c * 2 + (first_item ? 0 : 1)) * slot_floats(R, D);
                        to_m = to + R * D;
                        to_l = to_m + R;
                    }
                    core.finish_rows(seen, rows, [&](int h, int ch, auto &y, float m, float l) {
#pragma unroll
                        for (int i = 0; i < (int)(sizeof(y) / sizeof(float)); i += 4)
                            *reinterpret_cast<float4 *>(to + h * D + ch + i) =
                                make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
                        if (ch == 0) {
                            to_m[h] = m;
                            to_l[h] = l;
                        }
                    });
                }
                if (ends && lane == 0) {
                    int2 &to = a.owners[(int64_t)here.s * items + here.kvh * blocks + here.block];
                    const int32_t c0 = whole ? c : shares.at(first);
                    to = make_int2(c0, (c - c0 + 1) * 2 + (!whole && shares.start(c0) < first - COST));
                }
                fresh = true;
                first_item = false;
            }
            if (!last) here.next(a, blocks);
        }
        // (a wait gave up: the CTA may end when its copy and those behind it have landed)
        for (; units_ahead > 0; --units_ahead) {
            (void)wait(x);
            x = x + 1 == RING ? 0 : x + 1;
        }
    }
    if (SHARED) tc::pdl_wait_primaries();
}

// N neighbouring floats, N = 2 or 4
template <int N>
__device__ __forceinline__ void load_run(const float *from, float *x) {
    if constexpr (N == 4) {
        const float4 y = *reinterpret_cast<const float4 *>(from);
        x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w;
    } else {
        const float2 y = *reinterpret_cast<const float2 *>(from);
        x[0] = y.x; x[1] = y.y;
    }
}

// Joins what workers have left of every row: parts of its item, or its item's
// state (kda_attn_step_q8's are results already), and its states over the shared
// tokens.  `parts` groups of 8 lanes to a row, each with every parts-th state, four
// at a time: what bounds the kernel is the wait for its loads, the owners, then all
// of a state together (kda_attn_step_q8, 131072 and 40007 tokens, 32/8 heads, d = 128,
// now 69 us: one state at a time costs 5 us more, as a warp to a row and a state's
// sums behind its maximum do; kda_attn_step_shared, 24 rows behind 65536 shared tokens,
// 64 us: 2.5 and 1.8 more).
template <int D, int R, bool SHARED>
__global__ void __launch_bounds__(kJoinThreads) attn_rows_join_kernel(const AttnStepArgs a,
                                                                      const float *part,
                                                                      int32_t workers,
                                                                      int32_t parts) {
    constexpr int N = D == 16 ? 2 : 4;      // neighbouring channels
    constexpr int RUNS = D / (8 * N);       // and how many such runs a lane has
    constexpr int B = 4;                    // states in flight
    __shared__ __align__(16) float s_o[kJoinGroups][D];
    __shared__ float s_m[kJoinGroups], s_l[kJoinGroups];
    const int tid = threadIdx.x, group = tid >> 3, lane = tid & 7, mine = group % parts;
    const int32_t blocks = (a.G + R - 1) / R;
    const int64_t rows = (int64_t)a.N * a.HQ;
    const int64_t row = (int64_t)blockIdx.x * (kJoinGroups / parts) + group / parts;
    const bool there = row < rows;
    const int32_t s = there ? (int32_t)(row / a.HQ) : 0;
    const int32_t hq = there ? (int32_t)(row - (int64_t)s * a.HQ) : 0;
    const int32_t kvh = hq / a.G, block = (hq - kvh * a.G) / R, r = hq - kvh * a.G - block * R;
    const Span span = span_of<SHARED>(a, s);
    const PrefixState states = prefix_state(a, D, 0);
    // the kernels before this one have ended
    tc::pdl_wait_primaries();
    const int2 who = a.owners[((int64_t)s * a.HKV + kvh) * blocks + block];
    int32_t pieces = SHARED && span.first > 0 ? states.pieces[there ? row : 0] : 0;
    // (a kernel whose wait gave up has said so and left these as they were: anything)
    int32_t own = span.len() > 0 ? who.y >> 1 : 0;
    if (own < 0 || who.x < 0 || own > workers - who.x) own = 0;
    if (SHARED) pieces = min(max(pieces, 0), a.splits - 1);
    const bool done = !there || (!SHARED && own == 1);  // written by the worker
    const int32_t all = done ? 0 : own + pieces;
    const float *slots = part + (int64_t)who.x * 2 * slot_floats(R, D);
    float mx = -INFINITY, l = 0.f, o[RUNS][N];
#pragma unroll
    for (int c = 0; c < RUNS; ++c)
#pragma unroll
        for (int j = 0; j < N; ++j) o[c][j] = 0.f;
    for (int32_t i0 = mine; i0 < all; i0 += B * parts) {
        float m[B], sum[B], x[B][RUNS][N];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int32_t i = i0 + b * parts;
            m[b] = -INFINITY;
            sum[b] = 0.f;
#pragma unroll
            for (int c = 0; c < RUNS; ++c)
#pragma unroll
                for (int j = 0; j < N; ++j) x[b][c][j] = 0.f;
            if (i >= all) continue;
            // a worker's slot, or a piece (the item's state: the last one) of arrays
            // over the rows
            const float *from, *from_m, *from_l;
            if (i < own && own > 1) {
                const float *slot =
                    slots + (i * 2 + (i == 0 ? who.y & 1 : 0)) * (int64_t)slot_floats(R, D);
                from = slot + r * D;
                from_m = slot + R * D + r;
                from_l = from_m + R;
            } else {
                const int64_t at = (int64_t)(i < own ? a.splits - 1 : i - own) * rows + row;
                from = states.o + at * D;
                from_m = states.m + at;
                from_l = states.l + at;
            }
            m[b] = *from_m;
            sum[b] = *from_l;
#pragma unroll
            for (int c = 0; c < RUNS; ++c) load_run<N>(from + (c * 8 + lane) * N, x[b][c]);
        }
        float top = mx;
#pragma unroll
        for (int b = 0; b < B; ++b) top = fmaxf(top, m[b]);
        const float ref = top == -INFINITY ? 0.f : top, f = exp2f(mx - ref);
        mx = top;
        l *= f;
#pragma unroll
        for (int c = 0; c < RUNS; ++c)
#pragma unroll
            for (int j = 0; j < N; ++j) o[c][j] *= f;
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const float w = exp2f(m[b] - ref);
            l += sum[b] * w;
#pragma unroll
            for (int c = 0; c < RUNS; ++c)
#pragma unroll
                for (int j = 0; j < N; ++j) o[c][j] += x[b][c][j] * w;
        }
    }
    if (parts == 1) {
        if (done) return;
#pragma unroll
        for (int c = 0; c < RUNS; ++c) store_run(a, row, D, (c * 8 + lane) * N, o[c], mx, l);
        return;
    }
#pragma unroll
    for (int c = 0; c < RUNS; ++c)
#pragma unroll
        for (int j = 0; j < N; ++j) s_o[group][(c * 8 + lane) * N + j] = o[c][j];
    if (lane == 0) {
        s_m[group] = mx;
        s_l[group] = l;
    }
    __syncthreads();
    if (done) return;
    // the row's groups' states, by all of its lanes
    const int first = group - mine;
    float top = -INFINITY;
    for (int p = 0; p < parts; ++p) top = fmaxf(top, s_m[first + p]);
    const float ref = top == -INFINITY ? 0.f : top;
    for (int at = mine * 8 + lane; at < D / N; at += parts * 8) {
        float y[N], sum = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) y[j] = 0.f;
        for (int p = 0; p < parts; ++p) {
            const float w = exp2f(s_m[first + p] - ref);
            float x[N];
            load_run<N>(&s_o[first + p][at * N], x);
            sum += s_l[first + p] * w;
#pragma unroll
            for (int j = 0; j < N; ++j) y[j] += x[j] * w;
        }
        store_run(a, row, D, at * N, y, top, sum);
    }
}

// Groups to a row of the join: as many as make two CTAs to an SM at most (64 rows
// behind 4096 shared tokens, 32/8 heads, 53 us: 16 groups to an SM, not 64, cost 2 us
// more, 256 3).
inline int32_t join_parts(int64_t rows, int sms) {
    int32_t parts = 1;
    while (parts < kJoinGroups && rows * parts * 2 <= (int64_t)sms * 2 * kJoinGroups) parts *= 2;
    return parts;
}

// Bytes of workers' parts, and of owners.
template <class Core>
size_t flat_part_bytes(int sms) {
    return (size_t)sms * Core::kCtas * kWarps * 2 * slot_floats(Core::kRows, Core::kD) *
           sizeof(float);
}
template <class Core>
size_t owners_bytes(const AttnStepArgs &a) {
    return ((size_t)step_items<Core>(a) * sizeof(int2) + 255) / 256 * 256;
}

// The join, a programmatic dependent of the kernel before.
template <class Core, bool SHARED>
cudaError_t launch_rows_join(const AttnStepArgs &a, const float *part, int sms,
                             cudaStream_t stream) {
    const int64_t rows = (int64_t)a.N * a.HQ;
    const int32_t parts = join_parts(rows, sms), abreast = kJoinGroups / parts;
    const int32_t workers = sms * Core::kCtas * (Core::kAhead ? kWarps : 1);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr = follows_on();
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)((rows + abreast - 1) / abreast));
    cfg.blockDim = dim3(kJoinThreads);
    return cudaLaunchKernelEx(&cfg, attn_rows_join_kernel<Core::kD, Core::kRows, SHARED>, a, part,
                              workers, parts);
}

// A cache [heads of pages, page, D] as a 4-D map {panel, page, panels, heads} whose
// box is all panels of up to 32 rows of one page, swizzled by the panels' width.
template <class Core>
bool encode_panels_map(CUtensorMap *m, const void *base, int32_t page, int32_t heads) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t es = sizeof(typename Core::Cell), row = Core::kD * es;
    const cuuint32_t panel = (cuuint32_t)(Core::kPanel / es), panels = Core::kPanels;
    const cuuint32_t rows = (cuuint32_t)std::min<int32_t>(page, FlatCfg<Core>::UNIT);
    const cuuint64_t dims[4] = {panel, (cuuint64_t)page, panels, (cuuint64_t)heads};
    const cuuint64_t strides[3] = {row, Core::kPanel, row * page};
    const cuuint32_t box[4] = {panel, rows, panels, 1u};
    const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    return enc(m, es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
               const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               Core::kPanel == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The flat kernel (SHARED: a programmatic dependent of the kernel before).
template <class Core, bool SHARED>
cudaError_t launch_flat(AttnStepArgs a, float *part, int sms, cudaStream_t stream) {
    const cudaError_t e = allow_smem<attn_flat_kernel<Core, SHARED>>(FlatCfg<Core>::SMEM);
    if (e != cudaSuccess) return e;
    // (2^31 heads of pages are terabytes; a cache of no pages: any address, of which
    // nothing is read)
    const int32_t page = 1 << a.page_shift;
    a.num_pages = std::min(a.num_pages, INT32_MAX / a.HKV);
    const int32_t heads = std::max(a.num_pages * a.HKV, 1);
    FlatMaps maps;
    memset(&maps, 0, sizeof(maps));
    if (!encode_panels_map<Core>(&maps.k, a.num_pages ? a.k_cache : a.q, page, heads) ||
        !encode_panels_map<Core>(&maps.v, a.num_pages ? a.v_cache : a.q, page, heads))
        return cudaErrorInvalidValue;
    // one wave, and no more warps than the longest possible line has units
    const int64_t capacity = (int64_t)a.max_pages << a.page_shift;
    const int64_t most =
        step_items<Core>(a) * (capacity / FlatCfg<Core>::UNIT + 1 + FlatCfg<Core>::COST);
    const int64_t grid = std::min((int64_t)sms * Core::kCtas, (most + kWarps - 1) / kWarps);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr = follows_on();
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = SHARED ? 1 : 0;
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = FlatCfg<Core>::SMEM;
    return cudaLaunchKernelEx(&cfg, attn_flat_kernel<Core, SHARED>, a, part, maps);
}

}  // namespace
}  // namespace kda
