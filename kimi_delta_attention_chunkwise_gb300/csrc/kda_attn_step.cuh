// kda_attn_step.cuh -- one token of every sequence attends to its paged cache: the
// cores and kernels behind kda_attn_step, kda_attn_step_q8 and
// kda_attn_step_shared (kda_attn_step.cu, kda_attn_step_q8.cu, kda_attn_shared.cu
// choose the core of a problem and instantiate them).
//
//     z_j = scale <q, K_j>,  o = sum_j e^{z_j} V_j / sum_j e^{z_j}    (j < len)
//
// Memory-bound: a cached row is read once for every block of a group's query
// heads: of 16 (bf16, D = 64 or 128) or 4 (fp32 and narrower heads).  Larger
// groups read the cache once a block (64 sequences of 4000 tokens, d = 128: bf16
// with 8 key-value heads and G = 16 188 us, 32 355, 64 688; fp32 with 4 and G = 4
// 165 us, 8 312, 16 607).  The work of all sequences is cut into equal shares, whatever
// their lengths: the tiles of 64 tokens of every (sequence, key-value head,
// block of query heads) form one line, and CTA c of a grid that fills the GPU
// once takes the tiles from U c / grid to U (c + 1) / grid.  A CTA holds a
// running maximum, sum and weighted sum per query head (base 2) while it stays
// within one (sequence, head) item; an item that lies in one CTA is written
// out there, and an item that several share leaves one partial result per CTA
// (at most two per CTA: its first and its last item) for a second kernel to
// join.  No atomics: the same lengths give the same bits.
//
// Within a tile each of the CTA's 4 warps takes 16 tokens (one page holds
// them) and keeps its own running state, so the main loop has no barrier; the
// warps' states are joined when the CTA leaves an item.
#pragma once

#include <algorithm>
#include <cfloat>
#include <cstdint>
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "kda_attn.cuh"
#include "kda_internal.cuh"
#include "tc_ptx.cuh"

namespace kda {
namespace {

constexpr int kTile = 64, kWarps = 4, kThreads = 32 * kWarps, kWarpTokens = 16;
// The direct kernel's longest run of tokens per CTA by the table's size, for
// items that are all resident at once and for more than that.
constexpr int kDirectTokens = 1024, kDirectMany = 256;
constexpr int kFewItems = 32;
constexpr int kJoinWarps = 8, kJoinThreads = 32 * kJoinWarps;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// ---------------------------------------------------------------------------
// the tokens that sequences share (kda_attn_step_shared)
// ---------------------------------------------------------------------------
// Tokens of the shared pages.
__device__ __forceinline__ int32_t shared_tokens(const AttnStepArgs &a) {
    return min(max(*a.shared_pages, 0), a.max_pages) << a.page_shift;
}
// What a call says that is out of range (nullptr: not kda_attn_step_shared's).
__device__ __forceinline__ void check_shared_pages(const AttnStepArgs &a) {
    if (a.shared_pages && (*a.shared_pages < 0 || *a.shared_pages > a.max_pages))
        *a.status = KDA_ERR_INVALID_ARG;
}
constexpr int kPrefixTile = 128;  // tokens

// CTA c of `grid` takes units share_start(c) .. share_start(c + 1) - 1 of a line.
__device__ __forceinline__ int64_t share_start(int64_t units, int32_t c, int32_t grid) {
    return units * c / grid;
}
// The CTAs that work: no share is empty.
__device__ __forceinline__ int32_t workers(int64_t units, int32_t grid) {
    return (int32_t)min((int64_t)grid, units);
}
// The first of the CTAs that work on a line's units from `first` on: the last
// whose share starts at or before it.
__device__ __forceinline__ int32_t first_worker(int64_t units, int64_t first, int32_t grid) {
    return (int32_t)(((first + 1) * grid - 1) / units);
}

// The workers whose shares hold an item's units from `first` on, as the last of
// them, `c`, writes them down for the join: {the first of them, their number,
// times two, and one if the first has another item before}.
__device__ __forceinline__ int2 owners_of(int64_t units, int64_t first, int32_t c, int32_t grid) {
    const int32_t c0 = first_worker(units, first, grid);
    return make_int2(c0, (c - c0 + 1) * 2 + (share_start(units, c0, grid) != first));
}

// The shared tokens' work: the tiles of every item (a key-value head and a block
// of a.prefix_rows rows, a row being sequence * G + query head of the group) form
// a line, of which every CTA takes an equal share.  An item's pieces are counted
// from the first CTA that works on it.
struct PrefixLine {
    int32_t tiles, blocks, grid;
    int64_t units;
    __device__ PrefixLine(const AttnStepArgs &a, int32_t shared) {
        const int32_t rows = a.N * a.G;
        tiles = shared / kPrefixTile + (shared % kPrefixTile != 0);
        blocks = rows / a.prefix_rows + (rows % a.prefix_rows != 0);
        units = (int64_t)tiles * a.HKV * blocks;
        grid = workers(units, a.prefix_grid);
    }
};
struct PrefixPiece {
    int32_t kvh, block;
    int32_t tile0, tile1;  // its tiles
    int32_t index;         // which of the item's pieces
    bool last;             // the item's last one
    __device__ PrefixPiece(const PrefixLine &p, int32_t c, int64_t u, int64_t u1) {
        const int32_t item = (int32_t)(u / p.tiles);
        const int64_t first = (int64_t)item * p.tiles;
        kvh = item / p.blocks;
        block = item - kvh * p.blocks;
        tile0 = (int32_t)(u - first);
        tile1 = (int32_t)min((int64_t)p.tiles, u1 - first);
        index = c - first_worker(p.units, first, p.grid);
        last = tile1 == p.tiles;
    }
};
// How the SMs are divided between the shared tokens' kernel on the tensor cores, one
// CTA to an SM, and the step behind it, whose CTAs find no room beside one: the
// former is bound by what an SM computes, the latter by what an SM takes in, until
// memory gives no more.  `prefix`: so many SMs for the former that it ends when the
// latter does.  CTAs of the step that must wait for those get shares of late / 16 of
// the others'.  Times in ns of an SM, by what was measured: 2.27 us to a unit of the
// line with two row tiles, 1.65 with one (d = 64: 1.77, 1.01), behind 5 us; 95 GB/s
// of cached rows, behind 4 us.  The starts and the rate were fitted over 18 sizes (20-500
// sequences of up to 5000 tokens behind 4096-65536, 5/1, 8/1, 8/2, 16/2, 16/4, 28/4, 32/8,
// 40/8, 64/8 heads, both widths): mean times 53.6 us, with 7 us 54.3, 11 us 56.5, with
// 85 GB/s 53.6, 75 54.1, 110 GB/s and 7 us 57.2; single sizes lie up to 7% above their best.
struct SmSplit {
    int32_t prefix, late;
};
// What a sequence's `len` own tokens count for in that, in tokens: an item's start and
// end take an SM as long as 6000 / D tokens (1000 sequences of one token of their own
// behind 512, 8/2 heads, d = 64: 317 us where tokens alone counted, since two SMs were
// left for them).
__device__ __forceinline__ int32_t own_work(const AttnStepArgs &a, int32_t len) {
    return len > 0 ? 6000 / a.D : 0;
}
__device__ __forceinline__ SmSplit sm_split(const AttnStepArgs &a, const PrefixLine &line,
                                            int64_t own_tokens) {
    const int32_t sms = a.prefix_sms;
    if (line.units == 0) return {0, 16};
    const bool two = a.prefix_rows > 128 / a.G * a.G;  // row tiles to a unit
    // (each operation rounded by itself: the same division in both kernels)
    const float unit = a.D == 64 ? (two ? 1770.f : 1010.f) : (two ? 2270.f : 1650.f);
    const float work = __fmul_rn((float)line.units, unit);
    // (rows are taken in once for every 16 query heads)
    const float rows = (float)(a.HKV * (a.G > 16 ? (a.G + 15) / 16 : 1));
    const float own = __fmul_rn(__fmul_rn((float)own_tokens, rows), a.D / 23.75f);
    auto ends = [&](int32_t p) { return __fadd_rn(5000.f, __fdiv_rn(work, (float)p)); };
    auto step_ends = [&](int32_t p) {
        return __fadd_rn(4000.f, __fdiv_rn(own, (float)(sms - p)));
    };
    // the least number of SMs that end in time
    int32_t best = sms;
    for (int32_t p = (int32_t)(threadIdx.x & 31) + 1; p < sms; p += 32)
        if (ends(p) <= step_ends(p)) {
            best = p;
            break;
        }
    best = __reduce_min_sync(0xffffffffu, best);
    if (best == sms) return {best, 16};
    const float last = step_ends(best);
    const float left = __fdiv_rn(__fmul_rn(16.f, __fsub_rn(last, ends(best))), last);
    return {best, min(max((int32_t)left, 0), 16)};
}
// One piece's states of every row (here a row is sequence * HQ + query head), and
// the number of pieces that a row has.
struct PrefixState {
    float *o, *m, *l;  // weighted sums [rows, D], maxima (base 2) and sums [rows]
    int32_t *pieces;   // [rows]
};
// (splits: the pieces a row may have, and one more for its own tokens' state
// where one CTA of the step has it whole)
__host__ __device__ inline size_t prefix_bytes(int64_t rows, int D, int32_t splits) {
    return (size_t)rows * ((size_t)splits * (D + 2) + 1) * sizeof(float);
}
__device__ __forceinline__ PrefixState prefix_state(const AttnStepArgs &a, int D, int32_t piece) {
    const int64_t rows = (int64_t)a.N * a.HQ;
    float *o = static_cast<float *>(a.prefix);
    float *m = o + rows * D * a.splits;
    float *l = m + rows * a.splits;
    return {o + rows * D * piece, m + rows * piece, l + rows * piece,
            reinterpret_cast<int32_t *>(l + rows * a.splits)};
}

// ---------------------------------------------------------------------------
// the line of tiles
// ---------------------------------------------------------------------------
__device__ __forceinline__ int32_t clamp_len(const AttnStepArgs &a, int32_t s) {
    return min(max(a.seq_lens[s], 0), a.max_pages << a.page_shift);
}

// A sequence's tokens that the step itself works on: first .. end - 1.  All of
// them, but where a prefix has been seen to (SHARED): a sequence that holds the
// whole prefix has its tokens behind it left.
struct Span {
    int32_t first, end;
    __device__ int32_t len() const { return end - first; }
};
template <bool SHARED>
__device__ __forceinline__ Span span_of(const AttnStepArgs &a, int32_t s) {
    const int32_t len = clamp_len(a, s);
    if constexpr (SHARED) {
        const int32_t first = len >= shared_tokens(a) ? shared_tokens(a) : 0;
        return {first, len};
    }
    return {0, len};
}
// (len + kTile - 1 would overflow in the last tile below 2^31)
template <int TILE = kTile>
__device__ __forceinline__ int32_t tiles_of(int32_t len) {
    return len / TILE + (len % TILE != 0);
}

// The first sequence that holds all `shared` tokens (N: none does), for the whole
// CTA, by way of `out` in shared memory, and, to *own, the tokens of all
// sequences that are not shared.  Sequences that hold fewer may have anything in
// their rows of the table.
template <int THREADS>
__device__ __forceinline__ int32_t sharing_sequence(const AttnStepArgs &a, int32_t shared,
                                                    int32_t *out, unsigned long long *own) {
    if (threadIdx.x == 0) {
        *out = a.N;
        *own = 0;
    }
    __syncthreads();
    int32_t first = a.N;
    long long mine = 0;
    for (int32_t s = (int32_t)threadIdx.x; s < a.N; s += THREADS) {
        const int32_t len = clamp_len(a, s);
        const int32_t own_len = len >= shared ? len - shared : len;
        mine += (int64_t)own_len + own_work(a, own_len);
        if (len >= shared) first = min(first, s);
    }
    first = __reduce_min_sync(0xffffffffu, first);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if ((threadIdx.x & 31) == 0) {
        atomicMin_block(out, first);
        atomicAdd_block(own, (unsigned long long)mine);
    }
    __syncthreads();
    return *out;
}

// Prefix sums of the sequences' tiles, each thread holding a run of sequences.
// COST: what an item (of at least a tile) counts for besides its tiles, in tiles.
template <int THREADS, bool SHARED, int TILE = kTile, int COST = 0>
struct Line {
    __device__ static int32_t length_of(const AttnStepArgs &a, int32_t s) {
        const int32_t tiles = tiles_of<TILE>(span_of<SHARED>(a, s).len());
        return COST && tiles ? tiles + COST : tiles;
    }
    int64_t total;   // tiles of all sequences
    int64_t before;  // tiles before this thread's run
    int64_t tokens;  // (COST) tokens of all sequences, as own_work() counts
    bool shares;     // (COST, SHARED) a sequence holds the shared tokens
    int32_t s0, s1;  // this thread's run
    __device__ void scan(const AttnStepArgs &a, int64_t *sm /* [THREADS / 32], COST: twice */) {
        const int tid = threadIdx.x, lane = tid & 31;
        const int32_t per = (a.N + THREADS - 1) / THREADS;
        s0 = min(tid * per, a.N);
        s1 = min(s0 + per, a.N);
        int64_t mine = 0, held = 0;
        int holds = 0;
        for (int32_t s = s0; s < s1; ++s) {
            mine += length_of(a, s);
            if (COST) {
                const Span span = span_of<SHARED>(a, s);
                held += (int64_t)span.len() + own_work(a, span.len());
                holds |= span.first;
            }
            if (a.seq_lens[s] > (a.max_pages << a.page_shift)) *a.status = KDA_ERR_INVALID_ARG;
        }
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        if (lane == 31) sm[tid >> 5] = incl;
        if constexpr (COST > 0) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) held += __shfl_xor_sync(0xffffffffu, held, o);
            if (lane == 0) sm[THREADS / 32 + (tid >> 5)] = held;
        }
        if constexpr (COST > 0 && SHARED) shares = __syncthreads_or(holds);
        else __syncthreads();
        before = incl - mine;
        total = tokens = 0;
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < (tid >> 5)) before += sm[w];
            total += sm[w];
            if (COST) tokens += sm[THREADS / 32 + w];
        }
    }
    // The sequence of unit u (u < total * items) and the units before it, to
    // *seq / *base in shared memory (`look`, without the barrier).
    __device__ void find(const AttnStepArgs &a, int64_t u, int32_t items, int32_t *seq,
                         int64_t *base) const {
        look(a, u, items, seq, base);
        __syncthreads();
    }
    __device__ void look(const AttnStepArgs &a, int64_t u, int32_t items, int32_t *seq,
                         int64_t *base) const {
        int64_t b = before * items;
        if (u >= b) {
            for (int32_t s = s0; s < s1; ++s) {
                const int64_t n = (int64_t)length_of(a, s) * items;
                if (u < b + n) {
                    *seq = s;
                    *base = b;
                    break;
                }
                b += n;
            }
        }
    }
    // The units before sequence `seq`, to *base in shared memory.
    __device__ void base_of(const AttnStepArgs &a, int32_t seq, int32_t items, int64_t *base) const {
        if (seq >= s0 && seq < s1) {
            int64_t b = before;
            for (int32_t s = s0; s < seq; ++s) b += length_of(a, s);
            *base = b * items;
        }
        __syncthreads();
    }
};

// Floats of a worker's partial result for the joins: weighted sums [R, D], maxima [R]
// and sums [R]; whole 16-byte vectors.
__host__ __device__ constexpr int slot_floats(int R, int D) { return (R * (D + 2) + 3) / 4 * 4; }

// A state's maximum as the joins take it.  -inf says that no key was seen; a
// state that saw keys whose scores are all -inf keeps its sum of 0 with the
// lowest finite number, so that the row comes out as the definition's 0 / 0 if
// no other state has more.
__device__ __forceinline__ float state_max(float m, bool seen) {
    return seen ? fmaxf(m, -FLT_MAX) : -INFINITY;
}

// ---------------------------------------------------------------------------
// CUDA-core core: fp32 arithmetic, 4 query heads, any supported type and width
// ---------------------------------------------------------------------------
// Eight channels of one type as they lie in memory, and as floats.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
    uint4 x, y;
    __device__ void load(const float *p) {
        x = *reinterpret_cast<const uint4 *>(p);
        y = *(reinterpret_cast<const uint4 *>(p) + 1);
    }
    __device__ void zero() { x = y = make_uint4(0, 0, 0, 0); }
    __device__ void get(float (&f)[8]) const {
        const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(w[j]);
    }
};
template <>
struct Eight<__nv_bfloat16> {
    uint4 x;
    __device__ void load(const __nv_bfloat16 *p) { x = *reinterpret_cast<const uint4 *>(p); }
    __device__ void zero() { x = make_uint4(0, 0, 0, 0); }
    __device__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = __uint_as_float(w[j] << 16);
            f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    }
};
template <>
struct Eight<int8_t> {
    uint2 x;
    __device__ void load(const int8_t *p) { x = *reinterpret_cast<const uint2 *>(p); }
    __device__ void zero() { x = make_uint2(0, 0); }
    // code + 128 as the low byte of 2^23, less 2^23 + 128: exact, and no
    // conversion instruction (a quarter of the rate)
    __device__ void get(float (&f)[8]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t w = (j < 4 ? x.x : x.y) ^ 0x80808080u;
            f[j] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7650 | (j & 3))) - 8388736.f;
        }
    }
};

// A lane owns 8 channels; D / 8 lanes make a token, 256 / D tokens a step.
// Every group of D / 8 lanes keeps its own running state over its tokens.
// T: the queries' type; C: the cache's (int8: with a scale per row, which the
// score and the weight are multiplied by).
template <typename T, int D, typename C = T, int ROWS = 4>
struct SimtCore {
    using Type = T;
    using Cell = C;
    static constexpr int kD = D, kRows = ROWS;
    // (as many as the registers of so many rows let be)
    static constexpr int kCtas = ROWS == 4 ? 3 : ROWS == 2 || D * sizeof(C) == 512 ? 4 : 5;
    static constexpr bool kAhead = false, kScaled = sizeof(C) == 1;
    static constexpr int LPT = D / 8, TPW = 32 / LPT;
    // tokens whose keys and values are in flight together: 16, or 8 where 16
    // would take 128 registers, or too many for the CTAs (8-bit codes, d = 128, G = 1:
    // 12.4 us, with 16 and 3 CTAs 18.3)
    static constexpr int NB = (sizeof(C) != 2 && D == 128) ? 4 : kWarpTokens / TPW;

    float q[kRows][8], acc[kRows][8], m[kRows], l[kRows];
    float c2;

    // query row h (of `rows`) lies at row(h)
    template <class Row>
    __device__ void init(Row row, int rows, float scale) {
        const int cl = (threadIdx.x & 31) % LPT;
        c2 = scale * kLog2e;
#pragma unroll
        for (int h = 0; h < kRows; ++h) {
            Eight<T> x;
            if (h < rows) x.load(row(h) + cl * 8);
            else x.zero();
            x.get(q[h]);
            m[h] = -INFINITY;
            l[h] = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[h][j] = 0.f;
        }
    }
    // `n` (1..16) tokens whose rows start at kp / vp, their scales at ksp / vsp
    __device__ void tile(const C *kp, const C *vp, const float *ksp, const float *vsp, int n) {
        const int lane = threadIdx.x & 31, cl = lane % LPT, sub = lane / LPT;
#pragma unroll 1
        for (int b = 0; b < kWarpTokens; b += NB * TPW) {
            if (b >= n) break;
            Eight<C> kr[NB], vr[NB];
            float kf[NB], vf[NB];  // scales
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int t = b + i * TPW + sub;
                if (t < n) {
                    kr[i].load(kp + t * D + cl * 8);
                    vr[i].load(vp + t * D + cl * 8);
                } else {
                    kr[i].zero();
                    vr[i].zero();
                }
                if constexpr (kScaled) {
                    kf[i] = t < n ? ksp[t] : 0.f;
                    vf[i] = t < n ? vsp[t] : 0.f;
                }
            }
            float s[kRows][NB];
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                float f[8];
                kr[i].get(f);
#pragma unroll
                for (int h = 0; h < kRows; ++h) {
                    float d = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) d = fmaf(q[h][j], f[j], d);
                    s[h][i] = d;
                }
            }
#pragma unroll
            for (int o = 1; o < LPT; o <<= 1)
#pragma unroll
                for (int h = 0; h < kRows; ++h)
#pragma unroll
                    for (int i = 0; i < NB; ++i)
                        s[h][i] += __shfl_xor_sync(0xffffffffu, s[h][i], o);
#pragma unroll
            for (int h = 0; h < kRows; ++h) {
                float mx = m[h];
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    if constexpr (kScaled) s[h][i] *= kf[i];
                    if (b + i * TPW + sub >= n) s[h][i] = -INFINITY;
                    mx = fmaxf(mx, s[h][i]);
                }
                const float ref = mx == -INFINITY ? 0.f : mx;
                const float corr = exp2f((m[h] - ref) * c2);
                m[h] = mx;
                l[h] *= corr;
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    s[h][i] = exp2f((s[h][i] - ref) * c2);
                    l[h] += s[h][i];
                    if constexpr (kScaled) s[h][i] *= vf[i];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[h][j] *= corr;
            }
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                float f[8];
                vr[i].get(f);
#pragma unroll
                for (int h = 0; h < kRows; ++h)
#pragma unroll
                    for (int j = 0; j < 8; ++j) acc[h][j] = fmaf(s[h][i], f[j], acc[h][j]);
            }
        }
    }
    // the warp's state: weighted sums [kRows][D], maxima (base 2) and sums [kRows]
    __device__ void finish(float *sacc, float *sm, float *sl, bool seen) {
        const int lane = threadIdx.x & 31, cl = lane % LPT, sub = lane / LPT;
#pragma unroll
        for (int h = 0; h < kRows; ++h) {
            float mx = m[h];
#pragma unroll
            for (int o = LPT; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float w = mx == -INFINITY ? 0.f : exp2f((m[h] - mx) * c2);
            float sum = l[h] * w;
#pragma unroll
            for (int o = LPT; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float x = acc[h][j] * w;
#pragma unroll
                for (int o = LPT; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                if (sub == 0) sacc[h * D + cl * 8 + j] = x;
            }
            if (lane == 0) {
                sm[h] = state_max(mx * c2, seen);
                sl[h] = sum;
            }
        }
    }
};

// ---------------------------------------------------------------------------
// tensor-core core: bf16, D = 64 or 128, 8 NT query heads (FOLD: 4)
// ---------------------------------------------------------------------------
// Scores and outputs are computed transposed, so that the 16-row side of
// mma.sync.m16n8k16 is filled by tokens (then channels) and its 8-column side
// by query heads:
//     S^T [16 tokens x 8 heads] = K Q^T,   O^T [16 channels x 8 heads] += V^T P^T
// Every operand comes straight from global memory in 16-byte vectors, without
// shared memory, because a contraction may visit its index in any order as
// long as both operands agree, and the rows of O^T may be any channels:
//   * lane (g, t) = (lane / 4, lane % 4) of the K operand holds tokens g and
//     g + 8, channels 8 (4 j + t) .. + 7 of step pair j; Q likewise;
//   * lane (g, t) of the V operand holds tokens 2t, 2t + 1, 2t + 8, 2t + 9,
//     channels 8 g .. + 7 (and 64 + 8 g .. + 7), and pairs the tokens'
//     channels with byte permutes.
// The weights P^T go from the accumulator's layout to the operand's by an 8x8
// transpose (movmatrix), as two bf16 parts that leave 2^-15 of a weight out
// (split_weights; one part alone leaves 2^-8, as much as the output's own
// rounding).  Each part takes a product, but with at most 4 query heads (FOLD)
// the 8 columns hold the heads twice, the second time for the low parts, and
// one product serves both (64 sequences of 512-8192 tokens, 32/8 heads, d =
// 128: 194.8 us, two products 205, one rounded part 197; 64 sequences of 4000
// tokens, 64/8 heads: two products 164.3 us, one part 163.9; 128/8 heads:
// 187.5, 180.8).  The reference of the
// exponentials moves only when a score passes it by more than 2^8, by a vote
// of the warp: most tiles need no shuffles and no rescaling.
// mma.sync, not tcgen05: 16 query rows at most use an eighth of its 128-row
// tile, and at HBM speed an SM gets one such instruction's operands per ~20
// cycles.
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// 16 bytes that are read once
__device__ __forceinline__ uint4 load_once(const void *p) {
    uint4 x;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                 : "l"(p));
    return x;
}

// w (>= 0) as hi + lo in bf16: hi is w cut off (by less than 2^-7 of w), lo the
// rest rounded (2^-8 of it).  lo stays positive where hi is, by 2^-20 of w and
// 2^-126 at least: 0 times an infinity among the values would be a NaN.
__device__ __forceinline__ float rest_of(float w, float hi) {
    float lo;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(lo) : "f"(w - hi), "f"(hi * 0x1p-20f), "f"(fminf(hi, 0x1p-126f)));
    return lo;
}
// (FINITE: no value is an infinity, and lo may be 0; it is multiplied by `by`)
template <bool FINITE>
__device__ __forceinline__ void split_weights(float w0, float w1, uint32_t &hi, uint32_t &lo,
                                              float by = 1.f) {
    hi = __byte_perm(__float_as_uint(w0), __float_as_uint(w1), 0x7632);
    const float h0 = __uint_as_float(hi << 16), h1 = __uint_as_float(hi & 0xFFFF0000u);
    lo = FINITE ? tc::pack_bf16x2((w0 - h0) * by, (w1 - h1) * by)
                : tc::pack_bf16x2(rest_of(w0, h0), rest_of(w1, h1));
}

//
// A cache of 8-bit codes (C = int8_t) goes the same way: a code is exact in f16 and
// in bf16, so that its products with q and with the weights are those of the
// values up to the row's scale, which multiplies the score and the weight.  A
// lane's 16-byte vectors hold twice as many channels: 16 (4 j + t) .. + 15 of
// the keys and queries, 16 g .. + 15 (D = 64: 8 g .. + 7) of the values.
//
// What a code costs decides the kernel's speed (the byte permutes and bitwise
// operations run at half the rate).  With u = code + 128 as the low byte of a
// 16-bit number:
//   * f16 (keys): 0x6400 | u is 1024 + u; less 1152.  The queries go to f16 too,
//     each row times the power of two that brings its largest to 2^14 .. 2^15:
//     exact down to 2^-31 of it, and what is smaller is off by 2^-39 of it;
//   * f16 for the values, too, with at most 4 query heads, where the weights' low
//     parts have columns of their own and go there times 2^11.  A weight times its
//     row's scale is divided by vref, which belongs to the query head: the largest such
//     product so far lies between 2^6 and 2^15.  Products down to 2^-21 keep 2^-15 as
//     two f16 parts; a tile with a smaller one (a mask's end, a weight 2^-27 of the
//     largest, a scale far above the others') takes two bf16 parts instead, whose
//     range needs no reference (64 sequences of 512-8192 tokens, 32/8 heads, d = 128:
//     112 us where no tile does, 119 where all do, 126 with scores of +-30, which move
//     references, too);
//   * bf16 for the values else (whose range needs no reference): 0x4300 | u is
//     v = 128 + u below u = 128 and 2 u from there on, so that with w = v - 256
//     the code is w below 0 and w / 2 from there on, w - max(w / 2, 0): three
//     operations that round nothing.
__device__ __forceinline__ uint32_t codes_to_f16x2(uint32_t x /* 0x64uu64uu */) {
    uint32_t y;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0xE480E480u));  // - 1152
    return y;
}
__device__ __forceinline__ uint32_t codes_to_bf16x2(uint32_t x /* 0x43uu43uu */) {
    uint32_t w, h, y;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(w) : "r"(x), "r"(0xC380C380u));  // - 256
    asm("fma.rn.relu.bf16x2 %0, %1, %2, %3;"                                // / 2 - 128, or 0
        : "=r"(h)
        : "r"(x), "r"(0x3F003F00u), "r"(0xC300C300u));
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(w), "r"(h));
    return y;
}
__device__ __forceinline__ void mma_16816_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// (the product alone)
__device__ __forceinline__ void mma_16816_f16_first(float (&c)[4], uint32_t a0, uint32_t a1,
                                                    uint32_t a2, uint32_t a3, uint32_t b0,
                                                    uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint2 load_once8(const void *p) {
    uint2 x;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
                 : "=r"(x.x), "=r"(x.y)
                 : "l"(p));
    return x;
}

// TILED: rows come by way of shared memory (kda_attn_flat.cuh), in 128-byte panels
// with the copies' swizzle; 8-bit codes always take their tokens in that order.
template <int D, int NT, bool FOLD = false, typename C = __nv_bfloat16,
          bool TILED = sizeof(C) == 1>
struct MmaCore {
    static_assert(!FOLD || NT == 1, "the heads twice in 8 columns");
    using Type = __nv_bfloat16;
    using Cell = C;
    // (8 rows with D = 128 spill 44-104 bytes of registers where rows come straight from
    // global memory, 3 CTAs to an SM)
    static constexpr int kD = D, kRows = FOLD ? 4 : 8 * NT, kCtas = NT == 1 ? 3 : 2;
    static constexpr int kParts = FOLD ? 1 : 2;  // products of the weights
    static constexpr bool kAhead = true, kScaled = sizeof(C) == 1;
    static constexpr int J = D / 32;   // 16-byte vectors of a bf16 token row per lane (K, Q)
    static constexpr int VC = D / 64;  // and of V
    static constexpr int KC = kScaled ? J / 2 : J, VV = kScaled ? 1 : VC;  // as they lie in the cache
    static constexpr int MT = D / 16;  // channel tiles of O^T
    static constexpr float kMoveBy = 8.f;
    // weights and values as f16 (kScaled), and what the low parts are multiplied by
    static constexpr bool kF16 = kScaled && FOLD;
    static constexpr float kLow = kF16 ? 0x1p11f : 1.f;
    static constexpr float kNoRef = kF16 ? -FLT_MAX : -INFINITY;
    // (kF16) the products that two f16 parts hold
    static constexpr float kLeast = 0x1p-21f, kMost = 0x1p15f;
    float vref[2], vback[2];  // (kF16) the products' references, their reciprocals

    uint4 q[NT][J], k[2][KC], v[4][VV];
    float kf[2], vf[2];  // scales of tokens g and g + 8 (kScaled)
    float qf[NT][2];     // what the queries' rows 2 t and 2 t + 1 were divided by (kScaled)
    float o[MT][NT][4], s[NT][4], ref[NT][2], sum[NT][2];
    float c2;

    // Query rows of block n from bf16 to f16, and their factors.
    __device__ void to_f16(int n) {
        uint32_t top = 0;  // the row's largest magnitude
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t x = (&q[n][j].x)[w], lo = x & 0x7FFFu, hi = x >> 16 & 0x7FFFu;
                top = max(top, max(lo, hi));
            }
#pragma unroll
        for (int x = 1; x < 4; x <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, x));
        // (an infinity or a NaN keeps the numbers beside it finite: exponent 254)
        const uint32_t e = min(max(top >> 7, 27u), 254u);
        const float f = __uint_as_float((268u - e) << 23);  // 2^(14 - (e - 127))
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t &x = (&q[n][j].x)[w];
                x = tc::pack_f16x2(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xFFFF0000u) * f);
            }
        // the factor back: rows are the accumulators' columns
        const float back = __uint_as_float((e - 14u) << 23);
#pragma unroll
        for (int x = 0; x < 2; ++x)
            qf[n][x] = __shfl_sync(0xffffffffu, back, (2 * (threadIdx.x & 3) + x) * 4);
    }
    // The token that row r of the products is.  Any order will do; for tiles it is
    // one in which rows that lanes read from shared memory together lie in
    // different banks, by the swizzle of the copies that bring them (fetch()).
    static constexpr uint32_t kPanel = D * sizeof(C) < 128 ? D * sizeof(C) : 128;  // bytes of a row
    static constexpr int kPanels = D * sizeof(C) / kPanel;
    __device__ static int token_of(int r) {
        if constexpr (!TILED) return r;
        if constexpr (kPanel == 128) return r ^ ((r & 1) << 2);
        // rows 0, 2, 4, 6: tokens 0, 1, 4, 5; the row behind each: the token's two
        // low bits turned over
        return ((r & 8) | (r & 4) | (r >> 1 & 1)) ^ ((r & 1) * 3);
    }
    // first channel of the lane's j-th vector of a query row
    __device__ static int q_channel(int j, int t) {
        return kScaled ? ((j >> 1) * 4 + t) * 16 + (j & 1) * 8 : (j * 4 + t) * 8;
    }
    // query row h (of `rows`) lies at row(h)
    template <class Row>
    __device__ void init(Row row, int rows, float scale) {
        const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
        c2 = scale * kLog2e;
        vref[0] = vref[1] = 0.f;
        vback[0] = vback[1] = 1.f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int h = FOLD ? g & 3 : n * 8 + g;
#pragma unroll
            for (int j = 0; j < J; ++j)
                q[n][j] = h < rows ? *reinterpret_cast<const uint4 *>(row(h) + q_channel(j, t))
                                   : make_uint4(0, 0, 0, 0);
            if constexpr (kScaled) to_f16(n);
            ref[n][0] = ref[n][1] = kNoRef;
            sum[n][0] = sum[n][1] = 0.f;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][n][e] = 0.f;
        }
    }
    // rows kp / vp .. of n tokens (rows from n on are not read: zeros), and
    // their scales
    __device__ void load_k(const C *kp, const float *ksp, int n) {
        const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
        constexpr int V = 16 / sizeof(C);  // channels of a vector
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
            for (int j = 0; j < KC; ++j)
                k[r][j] = token_of(g + 8 * r) < n
                              ? load_once(kp + token_of(g + 8 * r) * D + (j * 4 + t) * V)
                              : make_uint4(0, 0, 0, 0);
            if constexpr (kScaled)
                kf[r] = token_of(g + 8 * r) < n ? __ldg(ksp + token_of(g + 8 * r)) : 0.f;
        }
    }
    __device__ void load_v(const C *vp, const float *vsp, int n) {
        const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int tok = token_of(2 * t + (r & 1) + 8 * (r >> 1));
#pragma unroll
            for (int c = 0; c < VV; ++c) {
                v[r][c] = make_uint4(0, 0, 0, 0);
                if (tok >= n) continue;
                if constexpr (!kScaled) {
                    v[r][c] = load_once(vp + tok * D + c * 64 + g * 8);
                } else if constexpr (D == 128) {
                    v[r][c] = load_once(vp + tok * D + g * 16);
                } else {
                    const uint2 x = load_once8(vp + tok * D + g * 8);
                    v[r][c].x = x.x;
                    v[r][c].y = x.y;
                }
            }
        }
        if constexpr (kScaled) {
#pragma unroll
            for (int r = 0; r < 2; ++r)
                vf[r] = token_of(g + 8 * r) < n ? __ldg(vsp + token_of(g + 8 * r)) : 0.f;
        }
    }
    // 16 tokens in tiles in shared memory: panels of keys and of values, and the
    // scales of both.  16-byte chunk c of row r of a panel lies at c ^ (r & 7) (rows
    // of 64 bytes: c ^ (r >> 1 & 3)).  The lane's places: key rows g (their first
    // two vectors), value rows 2 t and 2 t + 1, scale g; rows 8 further are 8
    // tokens further.
    uint32_t at_k[2], at_v[2], at_f;
    __device__ static uint32_t chunk_at(int token, int chunk) {
        return token * kPanel + (chunk ^ (kPanel == 128 ? token & 7 : token >> 1 & 3)) * 16;
    }
    __device__ void places() {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            at_k[i] = chunk_at(token_of(g), i * 4 + t);
            at_v[i] = kPanel == 64 ? chunk_at(token_of(2 * t + i), g >> 1) + (g & 1) * 8
                                   : chunk_at(token_of(2 * t + i), g);
        }
        at_f = token_of(g);
    }
    // panels `panel` bytes apart
    __device__ void fetch_k(const uint8_t *keys, uint32_t panel, const float *scales) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int j = 0; j < KC; ++j)
                k[r][j] = *reinterpret_cast<const uint4 *>(keys + (j >> 1) * panel + at_k[j & 1] +
                                                           8 * r * kPanel);
        if constexpr (kScaled) {
#pragma unroll
            for (int r = 0; r < 2; ++r) kf[r] = scales[at_f + 8 * r];
        }
    }
    __device__ void fetch_v(const uint8_t *values, uint32_t panel, const float *scales) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < VV; ++c) {
                const uint8_t *x = values + c * panel + at_v[r & 1] + (r >> 1) * 8 * kPanel;
                if constexpr (kPanel == 64) {
                    const uint2 y = *reinterpret_cast<const uint2 *>(x);
                    v[r][c].x = y.x;
                    v[r][c].y = y.y;
                } else {
                    v[r][c] = *reinterpret_cast<const uint4 *>(x);
                }
            }
        if constexpr (kScaled) {
#pragma unroll
            for (int r = 0; r < 2; ++r) vf[r] = scales[at_f + 8 * r];
        }
    }
    __device__ void scores() {
        if constexpr (kScaled) {
            float s2[NT][4];  // (two chains of products)
#pragma unroll
            for (int j = 0; j < KC; ++j)
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t a[2][2];  // by token (g, g + 8) and channel pair
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t x = (&k[r][j].x)[w] ^ 0x80808080u;
                        a[r][0] = codes_to_f16x2(__byte_perm(x, 0x64646464u, 0x4140));
                        a[r][1] = codes_to_f16x2(__byte_perm(x, 0x64646464u, 0x4342));
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint32_t *b = &q[n][2 * j + (w >> 1)].x + 2 * (w & 1);
                        float(&to)[4] = w & 1 ? s2[n] : s[n];
                        if (j == 0 && w < 2)
                            mma_16816_f16_first(to, a[0][0], a[1][0], a[0][1], a[1][1], b[0], b[1]);
                        else
                            mma_16816_f16(to, a[0][0], a[1][0], a[0][1], a[1][1], b[0], b[1]);
                    }
                }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[n][e] = (s[n][e] + s2[n][e]) * qf[n][e & 1] * kf[e >> 1];
        } else {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
                for (int j = 0; j < KC; ++j) {
                    mma_16816(s[n], k[0][j].x, k[1][j].x, k[0][j].y, k[1][j].y, q[n][j].x,
                              q[n][j].y);
                    mma_16816(s[n], k[0][j].z, k[1][j].z, k[0][j].w, k[1][j].w, q[n][j].z,
                              q[n][j].w);
                }
            }
        }
    }
    // References (kF16) that the tile's scores s and scales vf fit, and what is held
    // brought to them.
    __device__ void move_f16() {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float r = fmaxf(fmaxf(s[0][e], s[0][e + 2]) * c2, ref[0][e]);
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, x));
            const float f = exp2f(ref[0][e] - r);
            ref[0][e] = r;
            sum[0][e] *= f;
            // the products so far are f * vref of the new weights'; theirs are y at most
            float y = 0.f;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                y = fmaxf(y, tc::exp2_approx(fmaf(s[0][2 * h + e], c2, -r)) * fabsf(vf[h]));
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, x));
            const float held = f * vref[e];
            float now = fmaxf(held, 0x1p-126f);
            if (y > now * kMost)  // the power of two that brings y to 2^6 .. 2^7
                now = __uint_as_float(min((__float_as_uint(y * 0x1p-7f) >> 23) + 1, 254u) << 23);
            const float fv = held / now;
            vref[e] = now;
            vback[e] = 1.f / now;
            if (fv != 1.f) {
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int x = e; x < 4; x += 2) o[i][0][x] *= fv;
            }
        }
    }
    // values() for kF16
    __device__ void values_f16(int n_tok) {
        const int g = (threadIdx.x & 31) >> 2;
        const bool low = threadIdx.x & 2;  // columns 4-7
        if (n_tok < kWarpTokens) {
            if (token_of(g) >= n_tok) s[0][0] = s[0][1] = -INFINITY;
            if (token_of(g + 8) >= n_tok) s[0][2] = s[0][3] = -INFINITY;
        }
        float w[4], x[4];  // weights; times the scales over vref
        auto weigh = [&]() {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = tc::exp2_approx(fmaf(s[0][i], c2, -ref[0][i & 1]));
                x[i] = w[i] * vf[i >> 1] * vback[i & 1];
            }
        };
        auto most = [&]() {
            return fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
        };
        weigh();
        // (NaN compares false: a NaN score moves nothing and shows in the sums, a
        // NaN scale in the weights)
        const bool move = fmaxf(s[0][0], s[0][2]) * c2 > ref[0][0] + kMoveBy ||
                          fmaxf(s[0][1], s[0][3]) * c2 > ref[0][1] + kMoveBy || most() > kMost;
        if (__any_sync(0xffffffffu, move)) {
            move_f16();
            weigh();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[0][i & 1] += w[i];
        const float least =
            fminf(fminf(fabsf(x[0]), fabsf(x[1])), fminf(fabsf(x[2]), fabsf(x[3])));
        uint32_t p[2];  // by half of the tokens
        // rows g and g + 8 of channel tile i are bytes i and MT + i of a lane's
        // vectors; words of four bytes at a time
        if (__any_sync(0xffffffffu, least < kLeast || most() > kMost)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t hi, lo;
                split_weights<true>(x[2 * h], x[2 * h + 1], hi, lo, kLow);
                p[h] = transpose_8x8(low ? lo : hi);
            }
#pragma unroll
            for (int w4 = 0; w4 < MT / 4; ++w4) {
                uint32_t a[4][4];
                value_words<0x43434343u>(w4, a);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    mma_16816(o[4 * w4 + c][0], codes_to_bf16x2(a[c][0]), codes_to_bf16x2(a[c][1]),
                              codes_to_bf16x2(a[c][2]), codes_to_bf16x2(a[c][3]), p[0], p[1]);
            }
            return;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const __half2 hi = __floats2half2_rn(x[2 * h], x[2 * h + 1]);
            const float2 back = __half22float2(hi);
            const __half2 lo =
                __floats2half2_rn((x[2 * h] - back.x) * kLow, (x[2 * h + 1] - back.y) * kLow);
            const __half2 mine = low ? lo : hi;
            p[h] = transpose_8x8(*reinterpret_cast<const uint32_t *>(&mine));
        }
#pragma unroll
        for (int w4 = 0; w4 < MT / 4; ++w4) {
            uint32_t a[4][4];
            value_words<0x64646464u>(w4, a);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                mma_16816_f16(o[4 * w4 + c][0], codes_to_f16x2(a[c][0]), codes_to_f16x2(a[c][1]),
                              codes_to_f16x2(a[c][2]), codes_to_f16x2(a[c][3]), p[0], p[1]);
        }
    }
    // The codes plus 128 of word w of the lane's value vectors (kScaled), below the
    // bytes of MAGIC: by byte of the word, then operand register.
    template <uint32_t MAGIC>
    __device__ void value_words(int w, uint32_t (&a)[4][4]) const {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
                const int word = w + r * (MT / 4);
                const uint32_t x = (&v[2 * hi][0].x)[word] ^ 0x80808080u,
                               y = (&v[2 * hi + 1][0].x)[word] ^ 0x80808080u;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t z = __byte_perm(x, y, h ? 0x7362 : 0x5140);
                    a[2 * h][r + 2 * hi] = __byte_perm(z, MAGIC, 0x4140);
                    a[2 * h + 1][r + 2 * hi] = __byte_perm(z, MAGIC, 0x4342);
                }
            }
    }
    // weights of the tile's n tokens and their product with V
    __device__ void values(int n_tok) {
        if constexpr (kF16) {
            values_f16(n_tok);
        } else {
            values_bf16(n_tok);
        }
    }
    __device__ void values_bf16(int n_tok) {
        const int g = (threadIdx.x & 31) >> 2;
        const bool low = FOLD && (threadIdx.x & 2);  // columns 4-7
        uint32_t p[NT][kParts][2];  // by part (high, low) and half of the tokens
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (n_tok < kWarpTokens) {
                if (token_of(g) >= n_tok) s[n][0] = s[n][1] = -INFINITY;
                if (token_of(g + 8) >= n_tok) s[n][2] = s[n][3] = -INFINITY;
            }
            float top[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) top[e] = fmaxf(s[n][e], s[n][e + 2]) * c2;
            // (NaN compares false: a NaN score moves nothing and shows in the sums)
            const bool move = top[0] > ref[n][0] + kMoveBy || top[1] > ref[n][1] + kMoveBy;
            if (__any_sync(0xffffffffu, move)) {
                float f[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float m = fmaxf(top[e], ref[n][e]);
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1)
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
                    f[e] = m == -INFINITY ? 1.f : exp2f(ref[n][e] - m);
                    ref[n][e] = m;
                    sum[n][e] *= f[e];
                }
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][n][e] *= f[e & 1];
            }
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float r = ref[n][e & 1];
                w[e] = tc::exp2_approx(fmaf(s[n][e], c2, r == -INFINITY ? 0.f : -r));
                sum[n][e & 1] += w[e];
                if constexpr (kScaled) w[e] *= vf[e >> 1];
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t hi, lo;
                split_weights<kScaled>(w[2 * e], w[2 * e + 1], hi, lo);
                p[n][0][e] = transpose_8x8(low ? lo : hi);
                if (!FOLD) p[n][kParts - 1][e] = transpose_8x8(lo);
            }
        }
        auto product = [&](int i, const uint32_t (&a)[4]) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int part = kParts - 1; part >= 0; --part)
                    mma_16816(o[i][n], a[0], a[1], a[2], a[3], p[n][part][0], p[n][part][1]);
        };
        if constexpr (kScaled) {
            // (as in values_f16)
#pragma unroll
            for (int w = 0; w < MT / 4; ++w) {
                uint32_t a[4][4];
                value_words<0x43434343u>(w, a);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) a[c][r] = codes_to_bf16x2(a[c][r]);
                    product(4 * w + c, a[c]);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                // channel i of a lane's vector: D = 128: rows g and g + 8 of the
                // tile are channels 8 g + i and 64 + 8 g + i; D = 64: 8 g + i and
                // 8 g + 4 + i
                uint32_t a[4];
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int hi = 0; hi < 2; ++hi) {
                        const uint4 &x = v[2 * hi][VV == 2 ? r : 0],
                                    &y = v[2 * hi + 1][VV == 2 ? r : 0];
                        const int ch = VV == 2 ? i : i + 4 * r;
                        const uint32_t xw = (&x.x)[ch >> 1], yw = (&y.x)[ch >> 1];
                        a[r + 2 * hi] = __byte_perm(xw, yw, (ch & 1) ? 0x7632 : 0x5410);
                    }
                product(i, a);
            }
        }
    }
    // The warp's state, MT channels of a query head at a time from the lane that
    // holds them: put(head, first channel, weighted sums, maximum (base 2), sum).
    template <class Put>
    __device__ void finish_rows(bool seen, int rows, Put put) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int h = n * 8 + 2 * t + e;
                float l = sum[n][e];
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
#pragma unroll
                for (int hi = 0; hi < 2; ++hi) {
                    float y[MT];
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        y[i] = o[i][n][e + 2 * hi];
                        if (FOLD) y[i] += __shfl_xor_sync(0xffffffffu, y[i], 2) * (1.f / kLow);
                        if (kF16) y[i] *= vref[e];
                    }
                    const int ch = !kScaled && VC == 2 ? 64 * hi + 8 * g : 2 * MT * g + MT * hi;
                    if (h < rows) put(h, ch, y, state_max(ref[n][e], seen), l);
                }
            }
    }
    __device__ void finish(float *sacc, float *sm, float *sl, bool seen) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = sum[n][e];
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
                if (g == 0 && 2 * t < kRows) {
                    sm[n * 8 + 2 * t + e] = state_max(ref[n][e], seen);
                    sl[n * 8 + 2 * t + e] = l;
                }
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int h = n * 8 + 2 * t + (e & 1);
                    const int ch = kScaled   ? 2 * MT * g + MT * (e >> 1) + i
                                   : VC == 2 ? 64 * (e >> 1) + 8 * g + i
                                             : 8 * g + 4 * (e >> 1) + i;
                    float x = o[i][n][e];
                    if (FOLD) x += __shfl_xor_sync(0xffffffffu, x, 2) * (1.f / kLow);
                    if (kF16) x *= vref[e & 1];
                    if (h < kRows) sacc[h * D + ch] = x;
                }
        }
    }
};

// ---------------------------------------------------------------------------
// the kernels
// ---------------------------------------------------------------------------
__device__ __forceinline__ void store_out(const AttnStepArgs &a, int64_t i, float y) {
    if (a.out_f32) static_cast<float *>(a.out)[i] = y;
    else static_cast<__nv_bfloat16 *>(a.out)[i] = __float2bfloat16_rn(y);
}

// Tiles tile0 .. tile1 - 1 of a sequence's tokens first .. end - 1 (first: a
// multiple of kWarpTokens) into the warp's state; false if there was no key in
// them for the warp.
template <class Core>
__device__ __forceinline__ bool walk_tiles(const AttnStepArgs &a, Core &core, int32_t s,
                                           int32_t kvh, int32_t first, int32_t end, int32_t tile0,
                                           int32_t tile1) {
    using C = typename Core::Cell;
    constexpr int D = Core::kD;
    const int warp = threadIdx.x >> 5;
    const int32_t *table = a.block_table + (int64_t)s * a.max_pages;
    // this warp's tokens of tile t: the page's table entry, and the rows
    // (tiles from tile1 on, whose tokens may pass 2^31, are not asked for)
    auto page_of = [&](int32_t t) -> int32_t {
        if (t >= tile1) return -1;
        const int32_t tok = first + t * kTile + warp * kWarpTokens;
        return tok < end ? table[tok >> a.page_shift] : -1;
    };
    auto rows_of = [&](int32_t t, int32_t page, int64_t &at) -> int {
        at = 0;
        if (t >= tile1) return 0;
        const int32_t tok = first + t * kTile + warp * kWarpTokens;
        if (tok >= end) return 0;
        if (page < 0 || page >= a.num_pages) {
            *a.status = KDA_ERR_INVALID_ARG;
            return 0;
        }
        at = (((int64_t)page * a.HKV + kvh) << a.page_shift) + (tok & ((1 << a.page_shift) - 1));
        return min(kWarpTokens, end - tok);
    };
    const C *kc = static_cast<const C *>(a.k_cache), *vc = static_cast<const C *>(a.v_cache);
    bool seen = false;
    if constexpr (Core::kAhead) {
        // the next tile's keys are on their way while this one's weights and
        // values are worked on, its values while the next scores are, and its
        // table entry a tile earlier
        int64_t at, next_at;
        int n = rows_of(tile0, page_of(tile0), at), next_n;
        int32_t next_page = page_of(tile0 + 1);
        core.load_k(kc + at * D, a.k_scale + at, n);
        core.load_v(vc + at * D, a.v_scale + at, n);
        for (int32_t t = tile0; t < tile1; ++t) {
            next_n = rows_of(t + 1, next_page, next_at);
            next_page = page_of(t + 2);
            core.scores();
            core.load_k(kc + next_at * D, a.k_scale + next_at, next_n);
            if (n > 0) core.values(n);
            seen = seen || n > 0;
            core.load_v(vc + next_at * D, a.v_scale + next_at, next_n);
            n = next_n;
        }
    } else {
        int32_t next_page = page_of(tile0);
        for (int32_t t = tile0; t < tile1; ++t) {
            int64_t at;
            const int n = rows_of(t, next_page, at);
            next_page = page_of(t + 1);
            if (n > 0) core.tile(kc + at * D, vc + at * D, a.k_scale + at, a.v_scale + at, n);
            seen = seen || n > 0;
        }
    }
    return seen;
}

// The four warps' states, joined.
template <class Core>
struct Joined {
    float acc[kWarps][Core::kRows * Core::kD], m[kWarps][Core::kRows], l[kWarps][Core::kRows];
    // element i of row r: the weighted sum, maximum (base 2) and sum
    __device__ void get(int r, int i, float &o, float &mx, float &sum) const {
        mx = m[0][r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, m[w][r]);
        const float ref = mx == -INFINITY ? 0.f : mx;
        o = sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2f(m[w][r] - ref);
            o += acc[w][i] * f;
            sum += l[w][r] * f;
        }
    }
};

// (mx = -inf: no keys)
__device__ __forceinline__ void store_row(const AttnStepArgs &a, int64_t head, int D, int col,
                                          float o, float mx, float sum) {
    store_out(a, head * D + col, mx == -INFINITY ? 0.f : o / sum);
    if (a.lse && col == 0) a.lse[head] = mx == -INFINITY ? -INFINITY : (mx + log2f(sum)) * kLn2;
}

template <class Core, bool SHARED>
__global__ void __launch_bounds__(kThreads, Core::kCtas)
attn_step_kernel(const AttnStepArgs a, float *part) {
    using T = typename Core::Type;
    constexpr int D = Core::kD, R = Core::kRows;
    __shared__ Joined<Core> state;
    __shared__ int64_t s_scan[kWarps], s_base;
    __shared__ int32_t s_seq;
    const int tid = threadIdx.x, warp = tid >> 5;
    tc::pdl_launch_dependents();
    const int32_t blocks = (a.G + R - 1) / R;  // blocks of query heads
    const int32_t items = a.HKV * blocks;
    Line<kThreads, SHARED> line;
    line.scan(a, s_scan);
    const int64_t units = line.total * items;
    const int32_t grid = workers(units, (int32_t)gridDim.x), c = (int32_t)blockIdx.x;
    if (!SHARED && tid == 0 && c == 0) check_shared_pages(a);
    // sequences without keys (SHARED: the join's)
    for (int32_t s = c; s < a.N && !SHARED; s += gridDim.x) {
        if (clamp_len(a, s) > 0) continue;
        for (int32_t i = tid; i < a.HQ * D; i += kThreads)
            store_row(a, (int64_t)s * a.HQ + i / D, D, i % D, 0.f, -INFINITY, 0.f);
    }
    // SHARED: no CTA ends before the kernel that works on the shared tokens has,
    // so that what waits for this kernel has waited for both
    if (c >= grid) {
        if (SHARED) tc::pdl_wait_primaries();
        return;
    }
    const int64_t u0 = share_start(units, c, grid), u1 = share_start(units, c + 1, grid);
    line.find(a, u0, items, &s_seq, &s_base);
    int32_t s = s_seq;
    int64_t base = s_base;
    Core core;
    for (int64_t u = u0; u < u1;) {
        const Span span = span_of<SHARED>(a, s);
        const int32_t tiles = tiles_of(span.len());
        if (u >= base + (int64_t)tiles * items) {
            base += (int64_t)tiles * items;
            ++s;
            continue;
        }
        const int32_t item = (int32_t)((u - base) / tiles);
        const int32_t tile0 = (int32_t)((u - base) - (int64_t)item * tiles);
        const int32_t tile1 = (int32_t)min((int64_t)tiles, tile0 + (u1 - u));
        const int32_t kvh = item / blocks, h0 = (item - kvh * blocks) * R;
        const int32_t rows = min(R, a.G - h0);
        const int64_t head = (int64_t)kvh * a.G + h0;
        const T *qp = static_cast<const T *>(a.q) + s * a.q_stride + head * D;
        core.init([&](int h) { return qp + h * D; }, rows, a.scale);
        const bool seen = walk_tiles(a, core, s, kvh, span.first, span.end, tile0, tile1);
        core.finish(state.acc[warp], state.m[warp], state.l[warp], seen);
        __syncthreads();
        const bool whole = tile0 == 0 && tile1 == tiles;
        float *slot = part + ((int64_t)c * 2 + (u == u0 ? 0 : 1)) * slot_floats(R, D);
        for (int i = tid; i < rows * D; i += kThreads) {
            const int r = i / D, col = i % D;
            float o, mx, sum;
            state.get(r, i, o, mx, sum);
            if (whole && SHARED) {
                const PrefixState p = prefix_state(a, D, a.splits - 1);
                const int64_t at = (int64_t)s * a.HQ + head + r;
                p.o[at * D + col] = o;
                if (col == 0) {
                    p.m[at] = mx;
                    p.l[at] = sum;
                }
            } else if (whole) {
                store_row(a, (int64_t)s * a.HQ + head + r, D, col, o, mx, sum);
            } else {
                slot[i] = o;
                if (col == 0) {
                    slot[R * D + r] = mx;
                    slot[R * D + R + r] = sum;
                }
            }
        }
        __syncthreads();
        if (SHARED && tid == 0 && tile1 == tiles)
            a.owners[(int64_t)s * items + item] =
                owners_of(units, base + (int64_t)item * tiles, c, grid);
        u += tile1 - tile0;
    }
    if (SHARED) tc::pdl_wait_primaries();
}

// Short tables: one cluster per item, its CTAs (1, 2, 4 or 8) taking equal
// runs of the item's tiles and joining their states through distributed shared
// memory.  No look-up of the line, no scratch and no second kernel, which is
// what a small step spends its time on; lengths even out less.
template <class Core>
__global__ void __launch_bounds__(kThreads, Core::kCtas)
attn_step_direct_kernel(const AttnStepArgs a) {
    using T = typename Core::Type;
    constexpr int D = Core::kD, R = Core::kRows;
    __shared__ Joined<Core> state;
    __shared__ float s_o[R * D], s_m[R], s_l[R];
    namespace cg = cooperative_groups;
    const cg::cluster_group cluster = cg::this_cluster();
    const int32_t ctas = (int32_t)cluster.num_blocks(), rank = (int32_t)cluster.block_rank();
    const int tid = threadIdx.x, warp = tid >> 5;
    const int32_t blocks = (a.G + R - 1) / R, items = a.HKV * blocks;
    const int32_t index = (int32_t)(blockIdx.x / (uint32_t)ctas);
    const int32_t s = index / items, item = index - s * items;
    const int32_t kvh = item / blocks, h0 = (item - kvh * blocks) * R;
    const int32_t rows = min(R, a.G - h0);
    const int64_t head = (int64_t)kvh * a.G + h0;
    Core core;
    const T *qp = static_cast<const T *>(a.q) + s * a.q_stride + head * D;
    core.init([&](int h) { return qp + h * D; }, rows, a.scale);
    const int32_t len = clamp_len(a, s), tiles = tiles_of(len);
    if (tid == 0 && a.seq_lens[s] > (a.max_pages << a.page_shift)) *a.status = KDA_ERR_INVALID_ARG;
    if (tid == 0 && blockIdx.x == 0) check_shared_pages(a);
    const bool seen = walk_tiles(a, core, s, kvh, 0, len,
                                 (int32_t)((int64_t)tiles * rank / ctas),
                                 (int32_t)((int64_t)tiles * (rank + 1) / ctas));
    core.finish(state.acc[warp], state.m[warp], state.l[warp], seen);
    __syncthreads();
    if (ctas == 1) {
        for (int i = tid; i < rows * D; i += kThreads) {
            float o, mx, sum;
            state.get(i / D, i, o, mx, sum);
            store_row(a, (int64_t)s * a.HQ + head + i / D, D, i % D, o, mx, sum);
        }
        return;
    }
    for (int i = tid; i < rows * D; i += kThreads) {
        float o, mx, sum;
        state.get(i / D, i, o, mx, sum);
        s_o[i] = o;
        if (i % D == 0) {
            s_m[i / D] = mx;
            s_l[i / D] = sum;
        }
    }
    cluster.sync();
    for (int i = rank * kThreads + tid; i < rows * D; i += ctas * kThreads) {
        const int r = i / D;
        float mx = -INFINITY, sum = 0.f, o = 0.f;
        for (int32_t c = 0; c < ctas; ++c) mx = fmaxf(mx, *cluster.map_shared_rank(&s_m[r], c));
        const float ref = mx == -INFINITY ? 0.f : mx;
        for (int32_t c = 0; c < ctas; ++c) {
            const float f = exp2f(*cluster.map_shared_rank(&s_m[r], c) - ref);
            o += *cluster.map_shared_rank(&s_o[i], c) * f;
            sum += *cluster.map_shared_rank(&s_l[r], c) * f;
        }
        store_row(a, (int64_t)s * a.HQ + head + r, D, i % D, o, mx, sum);
    }
    cluster.sync();  // no CTA ends while another reads its shared memory
}

// Joins the items that several CTAs of the step share, one item per CTA:
// by_item: CTA (x, y) has item x; else it has the item that CTA x + 1 of the
// step is the second to work on (whichever makes the smaller grid).  Query
// heads y * per .. of the item; a warp takes one query head and every parts-th
// of the item's CTAs.
template <int D, int R>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const AttnStepArgs a,
                                                                 const float *part,
                                                                 int32_t step_grid, int32_t per,
                                                                 int32_t by_item) {
    constexpr int N = (D + 31) / 32;  // columns per lane
    __shared__ int64_t s_scan[kJoinWarps], s_base;
    __shared__ int32_t s_seq;
    __shared__ float s_o[kJoinWarps][D], s_m[kJoinWarps], s_l[kJoinWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int32_t blocks = (a.G + R - 1) / R, items = a.HKV * blocks;
    Line<kJoinThreads, false> line;
    line.scan(a, s_scan);
    const int64_t units = line.total * items;
    const int32_t grid = workers(units, step_grid);
    const bool any = units > 0 && (by_item || (int32_t)blockIdx.x + 1 < grid);
    const int64_t start = by_item || !any ? 0 : share_start(units, (int32_t)blockIdx.x + 1, grid);
    if (by_item) {
        if (tid == 0) s_seq = (int32_t)blockIdx.x / items;
        line.base_of(a, (int32_t)blockIdx.x / items, items, &s_base);
    } else if (any) {
        line.find(a, start, items, &s_seq, &s_base);
    }
    // every CTA waits for the step to end, so that whatever follows this
    // kernel in the stream also follows the step
    tc::pdl_wait_primaries();
    if (!any) return;
    const int32_t s = s_seq;
    const int32_t tiles = tiles_of(clamp_len(a, s));
    if (tiles == 0) return;  // by_item: written by the step
    const int32_t item = by_item ? (int32_t)blockIdx.x - s * items : (int32_t)((start - s_base) / tiles);
    const int64_t first = s_base + (int64_t)item * tiles, last = first + tiles;  // the item's units
    // the first of the step's CTAs on the item
    const int32_t c0 = by_item ? first_worker(units, first, grid) : (int32_t)blockIdx.x;
    if (by_item ? share_start(units, c0 + 1, grid) >= last
                : start == first || share_start(units, c0, grid) > first)
        return;
    const int32_t kvh = item / blocks, h0 = (item - kvh * blocks) * R;
    const int32_t r0 = blockIdx.y * per, rows = min(min(per, R), a.G - h0 - r0);
    if (rows <= 0) return;
    int32_t abreast = 1;  // query heads at a time, a power of two
    while (abreast < rows && abreast < kJoinWarps) abreast *= 2;
    const int32_t parts = kJoinWarps / abreast;
    for (int32_t rb = 0; rb < rows; rb += abreast) {
        const int32_t r = rb + (warp & (abreast - 1));
        float mx = -INFINITY, l = 0.f, o[N];
#pragma unroll
        for (int j = 0; j < N; ++j) o[j] = 0.f;
        if (r < rows) {
#pragma unroll 2
            for (int32_t i = c0 + warp / abreast; i < grid; i += parts) {
                const int64_t b = share_start(units, i, grid);
                if (b >= last) break;
                const float *slot = part + ((int64_t)i * 2 + ((i == c0 && b != first) ? 1 : 0)) *
                                               slot_floats(R, D);
                const float sm = slot[R * D + r0 + r], sl = slot[R * D + R + r0 + r];
                float x[N];
#pragma unroll
                for (int j = 0; j < N; ++j)
                    x[j] = (D >= 32 || lane < D) ? slot[(r0 + r) * D + j * 32 + lane] : 0.f;
                const float nm = fmaxf(mx, sm), ref = nm == -INFINITY ? 0.f : nm;
                const float f0 = exp2f(mx - ref), f1 = exp2f(sm - ref);
                mx = nm;
                l = l * f0 + sl * f1;
#pragma unroll
                for (int j = 0; j < N; ++j) o[j] = o[j] * f0 + x[j] * f1;
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
            const int64_t head = (int64_t)s * a.HQ + (int64_t)kvh * a.G + h0 + r0 + rb + w0;
            store_row(a, head, D, col, y, m, sum);
        }
        __syncthreads();
    }
}

// CTAs of a cluster for the direct kernel, or 0: the line of tiles.
int direct_ctas(int64_t items, int64_t capacity, int64_t slots) {
    int ctas = 1;
    while (ctas < 8 && items * ctas * 2 <= slots && capacity > (int64_t)ctas * kTile) ctas *= 2;
    return capacity <= (int64_t)ctas * (items <= slots ? kDirectTokens : kDirectMany) ? ctas : 0;
}

// Launched as a programmatic dependent of the kernel before.
inline cudaLaunchAttribute follows_on() {
    cudaLaunchAttribute x = {};
    x.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    x.val.programmaticStreamSerializationAllowed = 1;
    return x;
}

template <class Core>
int64_t step_items(const AttnStepArgs &a) {
    return (int64_t)a.N * a.HKV * ((a.G + Core::kRows - 1) / Core::kRows);
}

// CTAs of the line of tiles: one wave, and no more than the longest possible line
// has tiles.
template <class Core>
int line_grid(const AttnStepArgs &a, int sms) {
    const int64_t capacity = (int64_t)a.max_pages << a.page_shift;
    return (int)std::min((int64_t)sms * Core::kCtas, step_items<Core>(a) * (capacity / kTile + 1));
}

template <class Core>
int step_direct_ctas(const AttnStepArgs &a, int sms) {
    return direct_ctas(step_items<Core>(a), (int64_t)a.max_pages << a.page_shift,
                       (int64_t)sms * Core::kCtas);
}

template <class Core>
cudaError_t launch_direct(const AttnStepArgs &a, int ctas, cudaStream_t stream) {
    const int64_t items = step_items<Core>(a);
    if (items * ctas > INT32_MAX) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.gridDim = dim3((unsigned)(items * ctas));
    cfg.blockDim = dim3(kThreads);
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_step_direct_kernel<Core>, a);
}

template <class Core>
cudaError_t launch_line(const AttnStepArgs &a, int sms, cudaStream_t stream) {
    constexpr int D = Core::kD, R = Core::kRows;
    const int64_t items = step_items<Core>(a);
    const int grid = line_grid<Core>(a, sms);
    float *part = static_cast<float *>(a.workspace);
    attn_step_kernel<Core, false><<<grid, kThreads, 0, stream>>>(a, part);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || grid == 1) return e;
    // few items: each is shared by many CTAs, and a join CTA takes one query
    // head; else all of an item's
    const int32_t most_rows = std::min<int32_t>(R, a.G), per = items < kFewItems ? 1 : most_rows;
    const bool by_item = items < grid;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr = follows_on();
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)(by_item ? items : grid - 1), (unsigned)((most_rows + per - 1) / per));
    cfg.blockDim = dim3(kJoinThreads);
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<D, R>, a, static_cast<const float *>(part),
                              (int32_t)grid, per, (int32_t)by_item);
}

// Scratch of the line of tiles.
template <class Core>
size_t line_bytes(int sms) {
    return (size_t)sms * Core::kCtas * 2 * slot_floats(Core::kRows, Core::kD) * sizeof(float);
}
// The CUDA-core core with so many rows as there are query heads to a key-value head,
// up to 4, as a call of f(Core{}): what it takes is its arithmetic's time, and fewer
// rows leave registers for more CTAs (8-bit cache, fp32 queries, 16 sequences of
// 200-2000 tokens, G = 2, d = 64: 8.4 us, with 4 rows 13.3; 64 of 200-4000, d = 128:
// 62, 97; kda_attn_step_shared, fp32, 64 of 200-4000 tokens behind 2048, d = 128, G = 1:
// 115, 123).
template <typename T, int D, typename C, class F>
auto with_rows(int32_t G, F f) {
    if (G == 1) return f(SimtCore<T, D, C, 1>{});
    if (G == 2) return f(SimtCore<T, D, C, 2>{});
    return f(SimtCore<T, D, C>{});
}
// The core of a problem whose cache has the queries' type, as a call of f(Core{}).
template <class F>
auto with_core(int32_t D, int32_t G, int32_t dtype, F f) {
    if (dtype == KDA_DTYPE_BF16) {
        switch (D) {
            case 16: return f(SimtCore<__nv_bfloat16, 16>{});
            case 32: return f(SimtCore<__nv_bfloat16, 32>{});
            case 64:
                if (G <= 4) return f(MmaCore<64, 1, true>{});
                if (G <= 8) return f(MmaCore<64, 1>{});
                return f(MmaCore<64, 2>{});
            default:
                if (G <= 4) return f(MmaCore<128, 1, true>{});
                if (G <= 8) return f(MmaCore<128, 1>{});
                return f(MmaCore<128, 2>{});
        }
    }
    switch (D) {
        case 16: return f(SimtCore<float, 16>{});
        case 32: return f(SimtCore<float, 32>{});
        case 64: return f(SimtCore<float, 64>{});
        default: return f(SimtCore<float, 128>{});
    }
}

}  // namespace
}  // namespace kda
