// kda_attn_step.cu -- one token of every sequence attends to its paged cache.
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
// the line of tiles
// ---------------------------------------------------------------------------
__device__ __forceinline__ int32_t clamp_len(const AttnStepArgs &a, int32_t s) {
    return min(max(a.seq_lens[s], 0), a.max_pages << a.page_shift);
}
// (len + kTile - 1 would overflow in the last tile below 2^31)
__device__ __forceinline__ int32_t tiles_of(int32_t len) {
    return len / kTile + (len % kTile != 0);
}

// Prefix sums of the sequences' tiles, each thread holding a run of sequences.
template <int THREADS>
struct Line {
    int64_t total;   // tiles of all sequences
    int64_t before;  // tiles before this thread's run
    int32_t s0, s1;  // this thread's run
    __device__ void scan(const AttnStepArgs &a, int64_t *sm /* [THREADS / 32] */) {
        const int tid = threadIdx.x, lane = tid & 31;
        const int32_t per = (a.N + THREADS - 1) / THREADS;
        s0 = min(tid * per, a.N);
        s1 = min(s0 + per, a.N);
        int64_t mine = 0;
        for (int32_t s = s0; s < s1; ++s) {
            mine += tiles_of(clamp_len(a, s));
            if (a.seq_lens[s] > (a.max_pages << a.page_shift)) *a.status = KDA_ERR_INVALID_ARG;
        }
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        if (lane == 31) sm[tid >> 5] = incl;
        __syncthreads();
        before = incl - mine;
        total = 0;
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < (tid >> 5)) before += sm[w];
            total += sm[w];
        }
    }
    // The sequence of unit u (u < total * items) and the units before it, to
    // *seq / *base in shared memory.
    __device__ void find(const AttnStepArgs &a, int64_t u, int32_t items, int32_t *seq,
                         int64_t *base) const {
        int64_t b = before * items;
        if (u >= b) {
            for (int32_t s = s0; s < s1; ++s) {
                const int64_t n = (int64_t)tiles_of(clamp_len(a, s)) * items;
                if (u < b + n) {
                    *seq = s;
                    *base = b;
                    break;
                }
                b += n;
            }
        }
        __syncthreads();
    }
    // The units before sequence `seq`, to *base in shared memory.
    __device__ void base_of(const AttnStepArgs &a, int32_t seq, int32_t items, int64_t *base) const {
        if (seq >= s0 && seq < s1) {
            int64_t b = before;
            for (int32_t s = s0; s < seq; ++s) b += tiles_of(clamp_len(a, s));
            *base = b * items;
        }
        __syncthreads();
    }
};

__device__ __forceinline__ int64_t share_start(int64_t units, int32_t c, int32_t grid) {
    return units * c / grid;
}
// The CTAs that work: no share is empty.
__device__ __forceinline__ int32_t workers(int64_t units, int32_t grid) {
    return (int32_t)min((int64_t)grid, units);
}

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
// A lane owns 8 channels; D / 8 lanes make a token, 256 / D tokens a step.
// Every group of D / 8 lanes keeps its own running state over its tokens.
template <typename T, int D>
struct SimtCore {
    using Type = T;
    static constexpr int kD = D, kRows = 4, kCtas = 3;
    static constexpr bool kAhead = false;
    static constexpr int LPT = D / 8, TPW = 32 / LPT;
    // tokens whose keys and values are in flight together: 16, or 8 where 16
    // would take 128 registers
    static constexpr int NB = (sizeof(T) == 4 && D == 128) ? 4 : kWarpTokens / TPW;
    static constexpr int RAW = sizeof(T) / 2;  // 16-byte vectors per lane and token

    float q[kRows][8], acc[kRows][8], m[kRows], l[kRows];
    float c2;

    __device__ static void unpack(const uint4 (&x)[RAW], float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < RAW; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(T) == 4) {
                    f[4 * i + j] = __uint_as_float(w[j]);
                } else {
                    f[2 * j] = __uint_as_float(w[j] << 16);
                    f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
                }
            }
        }
    }
    __device__ void init(const T *qp, int rows, float scale) {
        const int cl = (threadIdx.x & 31) % LPT;
        c2 = scale * kLog2e;
#pragma unroll
        for (int h = 0; h < kRows; ++h) {
            uint4 x[RAW];
#pragma unroll
            for (int i = 0; i < RAW; ++i)
                x[i] = h < rows ? *(reinterpret_cast<const uint4 *>(qp + h * D + cl * 8) + i)
                                : make_uint4(0, 0, 0, 0);
            unpack(x, q[h]);
            m[h] = -INFINITY;
            l[h] = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[h][j] = 0.f;
        }
    }
    // `n` (1..16) tokens whose rows start at kp / vp
    __device__ void tile(const T *kp, const T *vp, int n) {
        const int lane = threadIdx.x & 31, cl = lane % LPT, sub = lane / LPT;
#pragma unroll 1
        for (int b = 0; b < kWarpTokens; b += NB * TPW) {
            if (b >= n) break;
            uint4 kr[NB][RAW], vr[NB][RAW];
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int t = b + i * TPW + sub;
#pragma unroll
                for (int r = 0; r < RAW; ++r) {
                    kr[i][r] = t < n ? *(reinterpret_cast<const uint4 *>(kp + t * D + cl * 8) + r)
                                     : make_uint4(0, 0, 0, 0);
                    vr[i][r] = t < n ? *(reinterpret_cast<const uint4 *>(vp + t * D + cl * 8) + r)
                                     : make_uint4(0, 0, 0, 0);
                }
            }
            float s[kRows][NB];
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                float f[8];
                unpack(kr[i], f);
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
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[h][j] *= corr;
            }
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                float f[8];
                unpack(vr[i], f);
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
__device__ __forceinline__ void split_weights(float w0, float w1, uint32_t &hi, uint32_t &lo) {
    hi = __byte_perm(__float_as_uint(w0), __float_as_uint(w1), 0x7632);
    lo = tc::pack_bf16x2(rest_of(w0, __uint_as_float(hi << 16)),
                         rest_of(w1, __uint_as_float(hi & 0xFFFF0000u)));
}

template <int D, int NT, bool FOLD = false>
struct MmaCore {
    static_assert(!FOLD || NT == 1, "the heads twice in 8 columns");
    using Type = __nv_bfloat16;
    static constexpr int kD = D, kRows = FOLD ? 4 : 8 * NT, kCtas = NT == 1 ? 3 : 2;
    static constexpr int kParts = FOLD ? 1 : 2;  // products of the weights
    static constexpr bool kAhead = true;
    static constexpr int J = D / 32;   // 16-byte vectors of a token row per lane (K, Q)
    static constexpr int VC = D / 64;  // and of V
    static constexpr int MT = D / 16;  // channel tiles of O^T
    static constexpr float kMoveBy = 8.f;

    uint4 q[NT][J], k[2][J], v[4][VC];
    float o[MT][NT][4], s[NT][4], ref[NT][2], sum[NT][2];
    float c2;

    __device__ void init(const Type *qp, int rows, float scale) {
        const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
        c2 = scale * kLog2e;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int h = FOLD ? g & 3 : n * 8 + g;
#pragma unroll
            for (int j = 0; j < J; ++j)
                q[n][j] = h < rows ? *reinterpret_cast<const uint4 *>(qp + h * D + (j * 4 + t) * 8)
                                   : make_uint4(0, 0, 0, 0);
            ref[n][0] = ref[n][1] = -INFINITY;
            sum[n][0] = sum[n][1] = 0.f;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][n][e] = 0.f;
        }
    }
    // rows kp / vp .. of n tokens (rows from n on are not read: zeros)
    __device__ void load_k(const Type *kp, int n) {
        const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int j = 0; j < J; ++j)
                k[r][j] = g + 8 * r < n ? load_once(kp + (g + 8 * r) * D + (j * 4 + t) * 8)
                                        : make_uint4(0, 0, 0, 0);
    }
    __device__ void load_v(const Type *vp, int n) {
        const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int tok = 2 * t + (r & 1) + 8 * (r >> 1);
#pragma unroll
            for (int c = 0; c < VC; ++c)
                v[r][c] = tok < n ? load_once(vp + tok * D + c * 64 + g * 8)
                                  : make_uint4(0, 0, 0, 0);
        }
    }
    __device__ void scores() {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                mma_16816(s[n], k[0][j].x, k[1][j].x, k[0][j].y, k[1][j].y, q[n][j].x, q[n][j].y);
                mma_16816(s[n], k[0][j].z, k[1][j].z, k[0][j].w, k[1][j].w, q[n][j].z, q[n][j].w);
            }
        }
    }
    // weights of the tile's n tokens and their product with V
    __device__ void values(int n_tok) {
        const int g = (threadIdx.x & 31) >> 2;
        const bool low = FOLD && (threadIdx.x & 2);  // columns 4-7
        uint32_t p[NT][kParts][2];  // by part (high, low) and half of the tokens
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (n_tok < kWarpTokens) {
                if (g >= n_tok) s[n][0] = s[n][1] = -INFINITY;
                if (g + 8 >= n_tok) s[n][2] = s[n][3] = -INFINITY;
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
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t hi, lo;
                split_weights(w[2 * e], w[2 * e + 1], hi, lo);
                p[n][0][e] = transpose_8x8(low ? lo : hi);
                if (!FOLD) p[n][kParts - 1][e] = transpose_8x8(lo);
            }
        }
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
                    const uint4 &x = v[2 * hi][VC == 2 ? r : 0], &y = v[2 * hi + 1][VC == 2 ? r : 0];
                    const int ch = VC == 2 ? i : i + 4 * r;
                    const uint32_t xw = (&x.x)[ch >> 1], yw = (&y.x)[ch >> 1];
                    a[r + 2 * hi] = __byte_perm(xw, yw, (ch & 1) ? 0x7632 : 0x5410);
                }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int part = kParts - 1; part >= 0; --part)
                    mma_16816(o[i][n], a[0], a[1], a[2], a[3], p[n][part][0], p[n][part][1]);
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
                    const int ch = VC == 2 ? 64 * (e >> 1) + 8 * g + i : 8 * g + 4 * (e >> 1) + i;
                    float x = o[i][n][e];
                    if (FOLD) x += __shfl_xor_sync(0xffffffffu, x, 2);
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

// One item's tiles tile0 .. tile1 - 1 into the warp's state; false if there was
// no key in them for the warp.
template <class Core>
__device__ __forceinline__ bool walk_tiles(const AttnStepArgs &a, Core &core, int32_t s,
                                           int32_t kvh, int32_t len, int32_t tile0, int32_t tile1) {
    using T = typename Core::Type;
    constexpr int D = Core::kD;
    const int warp = threadIdx.x >> 5;
    const int32_t *table = a.block_table + (int64_t)s * a.max_pages;
    // this warp's tokens of tile t: the page's table entry, and the rows
    // (tiles from tile1 on, whose tokens may pass 2^31, are not asked for)
    auto page_of = [&](int32_t t) -> int32_t {
        if (t >= tile1) return -1;
        const int32_t tok = t * kTile + warp * kWarpTokens;
        return tok < len ? table[tok >> a.page_shift] : -1;
    };
    auto rows_of = [&](int32_t t, int32_t page, int64_t &at) -> int {
        at = 0;
        if (t >= tile1) return 0;
        const int32_t tok = t * kTile + warp * kWarpTokens;
        if (tok >= len) return 0;
        if (page < 0 || page >= a.num_pages) {
            *a.status = KDA_ERR_INVALID_ARG;
            return 0;
        }
        at = ((((int64_t)page * a.HKV + kvh) << a.page_shift) +
              (tok & ((1 << a.page_shift) - 1))) * D;
        return min(kWarpTokens, len - tok);
    };
    const T *kc = static_cast<const T *>(a.k_cache), *vc = static_cast<const T *>(a.v_cache);
    bool seen = false;
    if constexpr (Core::kAhead) {
        // the next tile's keys are on their way while this one's weights and
        // values are worked on, its values while the next scores are, and its
        // table entry a tile earlier
        int64_t at, next_at;
        int n = rows_of(tile0, page_of(tile0), at), next_n;
        int32_t next_page = page_of(tile0 + 1);
        core.load_k(kc + at, n);
        core.load_v(vc + at, n);
        for (int32_t t = tile0; t < tile1; ++t) {
            next_n = rows_of(t + 1, next_page, next_at);
            next_page = page_of(t + 2);
            core.scores();
            core.load_k(kc + next_at, next_n);
            if (n > 0) core.values(n);
            seen = seen || n > 0;
            core.load_v(vc + next_at, next_n);
            n = next_n;
        }
    } else {
        int32_t next_page = page_of(tile0);
        for (int32_t t = tile0; t < tile1; ++t) {
            int64_t at;
            const int n = rows_of(t, next_page, at);
            next_page = page_of(t + 1);
            if (n > 0) core.tile(kc + at, vc + at, n);
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

template <class Core>
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
    Line<kThreads> line;
    line.scan(a, s_scan);
    const int64_t units = line.total * items;
    const int32_t grid = workers(units, (int32_t)gridDim.x), c = (int32_t)blockIdx.x;
    // sequences without keys
    for (int32_t s = c; s < a.N; s += gridDim.x) {
        if (clamp_len(a, s) > 0) continue;
        for (int32_t i = tid; i < a.HQ * D; i += kThreads)
            store_row(a, (int64_t)s * a.HQ + i / D, D, i % D, 0.f, -INFINITY, 0.f);
    }
    if (c >= grid) return;
    const int64_t u0 = share_start(units, c, grid), u1 = share_start(units, c + 1, grid);
    line.find(a, u0, items, &s_seq, &s_base);
    int32_t s = s_seq;
    int64_t base = s_base;
    Core core;
    for (int64_t u = u0; u < u1;) {
        const int32_t len = clamp_len(a, s), tiles = tiles_of(len);
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
        core.init(static_cast<const T *>(a.q) + s * a.q_stride + head * D, rows, a.scale);
        const bool seen = walk_tiles(a, core, s, kvh, len, tile0, tile1);
        core.finish(state.acc[warp], state.m[warp], state.l[warp], seen);
        __syncthreads();
        const bool whole = tile0 == 0 && tile1 == tiles;
        float *slot = part + ((int64_t)c * 2 + (u == u0 ? 0 : 1)) * (R * (D + 2));
        for (int i = tid; i < rows * D; i += kThreads) {
            const int r = i / D, col = i % D;
            float o, mx, sum;
            state.get(r, i, o, mx, sum);
            if (whole) {
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
        u += tile1 - tile0;
    }
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
    core.init(static_cast<const T *>(a.q) + s * a.q_stride + head * D, rows, a.scale);
    const int32_t len = clamp_len(a, s), tiles = tiles_of(len);
    if (tid == 0 && a.seq_lens[s] > (a.max_pages << a.page_shift)) *a.status = KDA_ERR_INVALID_ARG;
    const bool seen = walk_tiles(a, core, s, kvh, len, (int32_t)((int64_t)tiles * rank / ctas),
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
    Line<kJoinThreads> line;
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
    // the first of the step's CTAs on the item: the last that starts at or before it
    const int32_t c0 = by_item ? (int32_t)(((first + 1) * grid - 1) / units) : (int32_t)blockIdx.x;
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
                                               (R * (D + 2));
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

template <class Core>
int64_t step_items(const AttnStepArgs &a) {
    return (int64_t)a.N * a.HKV * ((a.G + Core::kRows - 1) / Core::kRows);
}

template <class Core>
cudaError_t launch_core(const AttnStepArgs &a, cudaStream_t stream) {
    constexpr int D = Core::kD, R = Core::kRows;
    const int sms = device_sms();
    if (!sms) return cudaErrorUnknown;
    const int64_t capacity = (int64_t)a.max_pages << a.page_shift;
    const int64_t items = step_items<Core>(a), slots = (int64_t)sms * Core::kCtas;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.stream = stream;
    cfg.attrs = attr;
    const int ctas = direct_ctas(items, capacity, slots);
    if (ctas > 0) {
        if (items * ctas > INT32_MAX) return cudaErrorInvalidValue;
        cfg.gridDim = dim3((unsigned)(items * ctas));
        cfg.blockDim = dim3(kThreads);
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)ctas;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, attn_step_direct_kernel<Core>, a);
    }
    // no more CTAs than the longest possible line has tiles
    const int grid = (int)std::min(slots, items * (capacity / kTile + 1));
    float *part = static_cast<float *>(a.workspace);
    attn_step_kernel<Core><<<grid, kThreads, 0, stream>>>(a, part);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || grid == 1) return e;
    // few items: each is shared by many CTAs, and a join CTA takes one query
    // head; else all of an item's
    const int32_t most_rows = std::min<int32_t>(R, a.G), per = items < kFewItems ? 1 : most_rows;
    const bool by_item = items < grid;
    cfg.gridDim = dim3((unsigned)(by_item ? items : grid - 1), (unsigned)((most_rows + per - 1) / per));
    cfg.blockDim = dim3(kJoinThreads);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<D, R>, a, static_cast<const float *>(part),
                              (int32_t)grid, per, (int32_t)by_item);
}

// The core of a problem, as a call of f.template operator()<Core>().
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

cudaError_t attn_step_workspace_bytes(const AttnStepArgs &a, size_t *bytes) {
    const int sms = device_sms();
    if (!sms) return cudaErrorUnknown;
    *bytes = with_core(a.D, a.G, a.dtype, [&](auto core) -> size_t {
        using Core = decltype(core);
        const int64_t slots = (int64_t)sms * Core::kCtas;
        if (direct_ctas(step_items<Core>(a), (int64_t)a.max_pages << a.page_shift, slots)) return 0;
        return (size_t)slots * 2 * Core::kRows * (Core::kD + 2) * sizeof(float);
    });
    return cudaSuccess;
}

cudaError_t launch_attn_step(const AttnStepArgs &a, cudaStream_t stream) {
    return with_core(a.D, a.G, a.dtype, [&](auto core) -> cudaError_t {
        return launch_core<decltype(core)>(a, stream);
    });
}

}  // namespace kda
