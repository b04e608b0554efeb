// kda_attn_tc.cu -- causal attention over packed prompts on the tensor cores:
// bf16, head width D = 64 or 128.
//
//     z_ij = scale <q_i, k_j>  (j <= i),   o_i = sum_j e^{z_ij} v_j / sum_j e^{z_ij}
//
// One pass over the keys with a running reference and sum per row, in base 2.
// The rows of a tile are (token, query head) pairs of one key-value head:
// R = floor(128 / G) tokens times the G heads of a group, brought in by one
// tensor copy, so that grouped heads share every key and value tile.
//
// A CTA owns two such tiles of 128 rows (consecutive tokens) and walks the
// keys in tiles of 128, or of 64 where sequences are short (launch_attn_tc).
// Per row tile t and key tile j:
//
//     S_t = Q_t K_j^T          tcgen05, operands in shared memory, D in TMEM
//     P_t = 2^{c S_t - ref}    one thread per row; bf16, over S_t's columns
//     O_t (+)= P_t V_j         tcgen05, A = P_t from TMEM, V_j as it lies
//
// The two row tiles alternate: while the softmax of one runs, the tensor core
// works for the other.  Warps: 0-3 and 4-7 the softmax and the results of tile
// 0 and 1, 8 issues the MMAs, 9 the copies and finds the work, 10-11 make
// masked values harmless and see to it that tiles have arrived.
//
// The weights lie over the scores that they came from, in one score tile of
// TMEM.  With 128 keys and d = 128 a row tile has one of its own: the scores of
// key tile j + 1 go where the weights of tile j are, after their product: one
// thread issues both, and the tensor core runs them in order.  Otherwise there
// is room for more (64 keys: four, d = 64: six; 128 keys, d = 64: three), and
// the units (row tile, key tile) take them in turn, the scores that many units
// ahead of the products.  (Two in turn at d = 128: 4096 tokens, 16 heads, 52 us
// instead of 50, whose row tiles the compiler knows.)
//
// A CTA works on one item (two row tiles of one key-value head) after another:
// with the last copies of one it takes the grid's next block that has not
// started (clusterlaunchcontrol), so that the next item's first copies and
// scores run beside the last item's results, and long and short items even
// out.  (Taken any earlier, a CTA with a long item ahead holds a second one
// back from idle ones: 4096 tokens, 16 heads, 71 us instead of 52.)  Items are
// numbered with a sequence's last tiles first (the longest under the causal
// mask).
//
// The reference of a row moves only when the row's maximum has passed it by
// more than 2^8: until then the weights stay below 2^8, which costs fp32 sums
// nothing and bf16 weights no precision (a floating-point scale), and the
// rescaling of O_t (a read and write of 128 x D fp32) is left out.
//
// The weights are rounded to bf16 for the tensor core (relative 2^-8, the
// operand type of V); their sum is taken in fp32 before the rounding.
//
// Masked places: scores are masked by selection, so masked keys are free to
// hold anything.  A masked weight is an exact 0, but 0 times an infinity or a
// NaN in a value row is NaN: warps 10-11 look through every value tile that
// holds a masked place before the MMA reads it, set the rows behind the item's
// last token to zero and replace non-finite values by zero; if there were
// any, the rows that do see them get them added at the end (`bad`).
//
// Waits are bounded: one that gives up sets KDA_ERR_TIMEOUT in the status
// word, every role leaves its loop, and the CTA ends after its copies and
// MMAs in flight.
//
// What bounds it: d = 128: the tensor core, and the power it draws (16384 tokens,
// 32/8 heads: 1.22-1.32 ms as the clocks come down, 1.67-1.81 PFLOP/s of the
// mask's lower half, 0.87-0.94 of a library matrix product's best).  d = 64: the
// softmax (8192 tokens, 32/8 heads: 257 us, 1.07 PFLOP/s): a key tile's tensor
// work is half, its weights are not.  Short sequences: an item's chain of
// copy, scores, weights, product and store (1000 x 64 tokens, 32/8 heads: 201
// us, 6.5 TB/s).
#include <cstdint>
#include <cstring>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include "kda_attn_common.cuh"
#include "kda_attn_ptx.cuh"
#include "kda_internal.cuh"
#include "tc_ptx.cuh"

namespace kda {

namespace {

using namespace tc;

constexpr int kThreads = 384;
constexpr int kRowTile = 128;
constexpr long long kWaitLimit = 2000000000LL;  // SM clocks, about a second
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMoveBy = 8.f;  // powers of two a row's maximum may pass its reference by

template <int D, int K>
struct Cfg {
    static constexpr int PANELS = D / 64;                 // 128-byte column panels
    static constexpr uint32_t PANEL = kRowTile * 128;     // bytes
    static constexpr uint32_t Q_TILE = PANELS * PANEL;
    // Keys of a tile.  Score tiles in TMEM: one per row tile, or (RING) what the
    // outputs leave room for, taken in turn by the units.
    static constexpr int KEYS = K;
    static constexpr bool RING = !(D == 128 && K == 128);
    static constexpr int SLOTS = RING ? (512 - 2 * D) / K : 2;
    static constexpr int DEPTH = RING ? SLOTS : 1;  // score tiles that one row tile may have
    static constexpr uint32_t KV_PANEL = KEYS * 128, TILE = PANELS * KV_PANEL;  // one K or V tile
    static constexpr int STAGES = D == 128 ? 512 / K : K == 128 ? 8 : 12;  // K and V tiles in flight
    // Units that the scores run ahead of the products (RING).  Their keys are
    // at most STAGES / 2 - 1 key tiles ahead, so that at a wait for K_j the tile
    // before on its barrier is done with, with the products of the tile at hand:
    // a lone row tile goes a key tile per unit, two go one per two units (and
    // the second one's last, two at most, one by one).
    __device__ static constexpr int32_t ahead(int32_t nk1) {
        return nk1 == 0 && SLOTS > STAGES / 2 - 1 ? STAGES / 2 - 1 : SLOTS;
    }
    static_assert(!RING || (SLOTS + 2) / 2 <= STAGES / 2 - 1, "two row tiles");
    // keys whose weights are handed over first, so that the product starts
    // while the others' are taken (8192 tokens, 40/8 heads, d = 128: 32 keys
    // 458 us, 64 473, 96 482, in four parts 465; d = 64, 32/8 heads: 64 keys
    // 266 us, 32 280, 96 268).  Tiles of 64 keys go over in one
    static constexpr int EARLY = K == 128 && D == 128 ? 32 : 64;
    static constexpr uint32_t O_BASE = SLOTS * KEYS;  // TMEM columns: scores, O_0, O_1
    static constexpr uint32_t IDESC_QK = idesc_bf16_f32(128, KEYS);
    static constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, D) | (1u << 16);  // V is N-major
};

// What a CTA works on: two row tiles of one key-value head.
struct Job {
    int32_t begin, len;  // the sequence's tokens in the packed axis
    int32_t kvh;
    int32_t q0[2];       // first token of each row tile
    int32_t nt[2];       // tokens of each row tile (0: none)
    int32_t nk[2];       // key tiles of each row tile
    int32_t n;           // key tiles of the item (0: no more work)
    int32_t last;        // the item's last token
    int32_t first_mask;  // first key tile with a masked place
};

// The (row tile, key tile) pairs of an item in the order in which they are
// worked on: (0, 0), (1, 0), (0, 1), ... as far as each row tile goes.  The
// second goes at least as far as the first, or there is none.
struct Unit {
    int32_t t, j;
};
__device__ __forceinline__ Unit unit_at(int32_t u, int32_t nk0, int32_t nk1) {
    if (nk1 == 0) return {0, u};
    if (u < 2 * nk0) return {u & 1, u >> 1};
    return {1, u - nk0};
}
__device__ __forceinline__ int32_t unit_of(int t, int32_t j, int32_t nk0, int32_t nk1) {
    if (nk1 == 0) return j;
    return t == 0 ? 2 * j : j < nk0 ? 2 * j + 1 : nk0 + j;
}

constexpr int kJobs = 2;      // items known at a time
constexpr int kMasked = 8;    // masked value tiles in flight at most: the ring holds no more
constexpr int kMaxStages = 12, kMaxSlots = 6;
constexpr int kJobUsers = 11; // warps that read a job: 0-8, 10, 11

struct Shared {
    uint64_t q_full[2], q_empty[2], kv_full[kMaxStages], kv_empty[kMaxStages];
    uint64_t v_raw[kMasked], v_half[kMasked];
    uint64_t s_full[2][kMaxSlots], pv_done[2][kMaxSlots], o_free[2];  // by row tile
    uint64_t p_full[kMaxSlots], p_rest[kMaxSlots];                    // by score tile
    uint64_t job_full[kJobs], job_empty[kJobs], next_full, drained;
    uint4 next;  // the answer to the request for another block
    Job job[kJobs];
    int32_t bad[kJobs];
    uint32_t tmem;
    int32_t abort;
};

constexpr uint32_t kStage = 32 * 128;  // bytes a softmax warp's results pass through

// The tiles start at the dynamic shared memory's base, which is 1024-byte
// aligned (the kernel has no other shared memory); the results' bytes and
// Shared follow them.
template <int D, int K>
constexpr uint32_t smem_bytes() {
    using C = Cfg<D, K>;
    static_assert(C::STAGES <= kMaxStages && C::SLOTS <= kMaxSlots && C::STAGES / 2 <= kMasked,
                  "room for the barriers");
    return 2 * C::Q_TILE + C::STAGES * C::TILE + 8 * kStage + (uint32_t)sizeof(Shared);
}
static_assert(smem_bytes<128, 128>() <= 232448 && smem_bytes<128, 64>() <= 232448 &&
                  smem_bytes<64, 128>() <= 232448 && smem_bytes<64, 64>() <= 232448,
              "227 KB per CTA");

// Not 0 if one of eight bf16 has an exponent of all ones (infinity or NaN):
// its exponent field carries into the sign's place.
__device__ __forceinline__ uint32_t all_ones(const uint4 &x) {
    uint32_t y = 0;
    y |= (x.x & 0x7F807F80u) + 0x00800080u;
    y |= (x.y & 0x7F807F80u) + 0x00800080u;
    y |= (x.z & 0x7F807F80u) + 0x00800080u;
    y |= (x.w & 0x7F807F80u) + 0x00800080u;
    return y & 0x80008000u;
}
template <int D, int K>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
               const __grid_constant__ CUtensorMap map_v, const AttnArgs a) {
    using C = Cfg<D, K>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *sq = smem, *skv = smem + 2 * C::Q_TILE, *sout = skv + C::STAGES * C::TILE;
    Shared &sh = *reinterpret_cast<Shared *>(sout + 8 * kStage);
    if (smem_u32(smem) & 1023u) {  // the swizzled tiles would not match their descriptors
        *a.status = KDA_ERR_CUDA;
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int32_t R = kRowTile / a.G;  // tokens of a row tile

    if (warp == 0 && lane == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(&sh.q_full[t], 1);
            mbar_init(&sh.q_empty[t], 1);
            for (int b = 0; b < C::DEPTH; ++b) {
                mbar_init(&sh.s_full[t][b], 1);
                mbar_init(&sh.pv_done[t][b], 1);
            }
            mbar_init(&sh.o_free[t], 4);
        }
        for (int b = 0; b < C::SLOTS; ++b) {
            mbar_init(&sh.p_full[b], 5);  // four warps of weights, and K and V have arrived
            mbar_init(&sh.p_rest[b], 4);
        }
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&sh.kv_full[i], 1);
            mbar_init(&sh.kv_empty[i], 1);
        }
        for (int i = 0; i < kMasked; ++i) {
            mbar_init(&sh.v_raw[i], 1);
            mbar_init(&sh.v_half[i], 2);
        }
        for (int i = 0; i < kJobs; ++i) {
            mbar_init(&sh.job_full[i], 1);
            mbar_init(&sh.job_empty[i], kJobUsers);
        }
        mbar_init(&sh.next_full, 1);
        mbar_init(&sh.drained, 1);
        sh.abort = 0;
        fence_mbar_init();
        fence_proxy_async();
    } else if (warp == 8) {
        tmem_alloc(&sh.tmem, 512);
        tmem_relinquish();
    }
    // warp 9 looks the first item up in the meantime
    TileCursor cursor;
    SeqTile st;
    bool found = false;
    if (warp == 9) {
        if (lane < 3) {
            const CUtensorMap *m = lane == 0 ? &map_q : lane == 1 ? &map_k : &map_v;
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
        }
        __syncwarp();
        found = find_seq_tile(a.cu_seqlens, a.N, a.T, 1, 2 * R, blockIdx.x / a.HKV, cursor, st);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;

    // Waits of one thread and of a whole warp (which goes on or gives up
    // together).  `use` counts the barrier's phases.
    auto wait = [&](uint64_t *bar, uint32_t use) -> bool {
        if (mbar_try_wait(bar, use & 1)) return true;
        if (mbar_wait_bounded(bar, use & 1, kWaitLimit)) return true;
        sh.abort = 1;
        *a.status = KDA_ERR_TIMEOUT;
        return false;
    };
    auto wait_warp = [&](uint64_t *bar, uint32_t use) -> bool {
        return __all_sync(0xffffffffu, wait(bar, use));
    };
    auto arrive_warp = [&](uint64_t *bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };

    if (warp < 8) {
        // ---- softmax and results: one thread per row ---------------------
        regs_inc<208>();
        const int t = warp >> 2, row = tid & 127;
        const uint32_t lane_base = (uint32_t)(warp & 3) * 32;
        const uint32_t o_addr = tmem_addr(tmem, lane_base, C::O_BASE + t * D);
        const int tk = row / a.G;  // the row's token within the tile
        const float c2 = a.scale * kLog2e;
        uint32_t it = 0, units = 0;  // key tiles of this row tile, and units, so far
        // The scores, and the product, of the row tile's x-th key tile are done.
        // A row tile has barriers of its own for both, since it may be items
        // ahead of the other one (those without a second row tile), and as many
        // as scores run ahead: at a wait for x the phase before on its barrier
        // is done, and the next cannot be.
        auto scores_done = [&](uint32_t x) -> bool {
            if (!wait_warp(&sh.s_full[t][x % C::DEPTH], x / C::DEPTH)) return false;
            tc_fence_after();
            return true;
        };
        auto product_done = [&](uint32_t x) -> bool {
            if (!wait_warp(&sh.pv_done[t][x % C::DEPTH], x / C::DEPTH)) return false;
            tc_fence_after();
            return true;
        };
        for (uint32_t item = 0;; ++item) {
            const Job &job = sh.job[item % kJobs];
            if (!wait_warp(&sh.job_full[item % kJobs], item / kJobs) || job.n == 0) break;
            const int32_t n = job.nk[t], q0 = job.q0[t], tok = q0 + tk;
            const int32_t nk0 = job.nk[0], nk1 = job.nk[1];
            const bool mine = tk < job.nt[t];  // the row is a token's
            float ref = -INFINITY, sum = 0.f;  // the reference times c2
            bool ok = true;
            for (int32_t j = 0; j < n; ++j) {
                const uint32_t slot =
                    C::RING ? (units + unit_of(t, j, nk0, nk1)) % C::SLOTS : (uint32_t)t;
                const uint32_t s_addr = tmem_addr(tmem, lane_base, slot * C::KEYS);
                ok = scores_done(it + j);
                if (!ok) break;
                float s[C::KEYS];
#pragma unroll
                for (int i = 0; i < C::KEYS; i += 32) ld32_nowait(s_addr + i, s + i);
#pragma unroll
                for (int i = 0; i < C::KEYS; i += 32) wait_ld32(s + i);
                const int32_t seen = tok - j * C::KEYS;  // columns up to this one are seen
                if ((j + 1) * C::KEYS - 1 > q0) {
#pragma unroll
                    for (int i = 0; i < C::KEYS; ++i)
                        if (i > seen) s[i] = -INFINITY;
                }
                float m[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) m[i] = fmaxf(s[i], s[i + 4]);
#pragma unroll
                for (int i = 8; i < C::KEYS; i += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e) m[e] = max3(m[e], s[i + e], s[i + e + 4]);
                const float top = fmaxf(max3(m[0], m[1], m[2]), m[3]) * c2;
                // (also on the first tile; rows without a token of their own
                // hold anything, and would ask every time for a NaN)
                const bool move = mine && !(top - ref <= kMoveBy);
                if (__any_sync(0xffffffffu, move)) {
                    float f = 1.f;
                    if (move) {
                        const float next = fmaxf(ref, top);
                        // a row whose scores are all -inf so far keeps weights of 0
                        f = exp2_approx(ref - (next == -INFINITY ? 0.f : next));
                        sum *= f;
                        ref = next;
                    }
                    __syncwarp();
                    // rescale the row's outputs, once the last product is done
                    // (with one score tile, these scores came after it)
                    if (j > 0) {
                        ok = !C::RING || product_done(it + j - 1);
                        if (!ok) break;
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            float x[16];
                            tmem_ld16(o_addr + c, x);
                            uint32_t y[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(x[i] * f);
                            st16_nowait(o_addr + c, y);
                        }
                    }
                }
                const float neg = ref == -INFINITY ? 0.f : -ref;
                const float2 c22 = make_float2(c2, c2), neg2 = make_float2(neg, neg);
                float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
#pragma unroll
                for (int h = 0; h < C::KEYS / 32; ++h) {
                    uint32_t p[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float2 x = f2_fma(make_float2(s[h * 32 + 2 * i], s[h * 32 + 2 * i + 1]), c22,
                                          neg2);
                        x.x = exp2_approx(x.x);
                        x.y = exp2_approx(x.y);
                        if (i & 1) acc1 = f2_add(acc1, x);
                        else acc0 = f2_add(acc0, x);
                        p[i] = pack_bf16x2(x.x, x.y);
                    }
                    st16_nowait(s_addr + h * 16, p);
                    if (h == C::EARLY / 32 - 1 || h == C::KEYS / 32 - 1) {
                        tmem_wait_st();
                        tc_fence_before();
                        arrive_warp(h == C::EARLY / 32 - 1 ? &sh.p_full[slot] : &sh.p_rest[slot]);
                        __syncwarp();
                    }
                }
                acc0 = f2_add(acc0, acc1);
                sum += acc0.x + acc0.y;
            }
            if (!ok) break;
            if (n > 0) {
                if (!product_done(it + n - 1)) break;
                const float inv = 1.f / sum;
                const int64_t token = (int64_t)job.begin + tok;
                const int64_t head = (int64_t)job.kvh * a.G + (row - tk * a.G);
                const bool bad = mine && sh.bad[item % kJobs] != 0;
                if (mine && a.lse) a.lse[token * a.HQ + head] = (ref + log2f(sum)) * kLn2;
                const int64_t at = mine ? (token * a.HQ + head) * D : -1;
                // columns c .. c + N - 1 of the row, ready to be rounded
                auto columns = [&](int c, auto &x) {
                    constexpr int N = sizeof(x) / sizeof(float);
                    __syncwarp();  // the loads are the whole warp's
#pragma unroll
                    for (int i = 0; i < N; i += 32) ld32_nowait(o_addr + c + i, x + i);
#pragma unroll
                    for (int i = 0; i < N; i += 32) wait_ld32(x + i);
                    if (c + N == D) {
                        tc_fence_before();
                        arrive_warp(&sh.o_free[t]);
                    }
#pragma unroll
                    for (int i = 0; i < N; ++i) x[i] *= inv;
                    if (bad) {
                        // non-finite values of the tiles that were looked through
                        const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v) +
                                                 (int64_t)job.begin * a.v_stride +
                                                 (int64_t)job.kvh * D + c;
                        for (int32_t k = job.first_mask * C::KEYS; k <= tok; ++k)
#pragma unroll
                            for (int i = 0; i < N; ++i) {
                                const float y = __bfloat162float(v[k * a.v_stride + i]);
                                if (!isfinite(y)) x[i] += y;
                            }
                    }
                    __syncwarp();
                };
                // 128 bytes of every row, by way of shared memory (the 128-byte
                // swizzle keeps both sides free of bank conflicts): eight lanes
                // store one row's at a time, whole lines
                uint8_t *mine_out = sout + warp * kStage;
                auto store = [&](const uint4 (&v)[8], char *base, int es) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<uint4 *>(mine_out + sw128_chunk(lane, i)) = v[i];
                    __syncwarp();
#pragma unroll
                    for (int r = 0; r < 32; r += 4) {
                        const int rr = r + (lane >> 3);
                        const uint4 x =
                            *reinterpret_cast<const uint4 *>(mine_out + sw128_chunk(rr, lane & 7));
                        const int64_t o = __shfl_sync(0xffffffffu, at, rr);
                        if (o >= 0) *reinterpret_cast<uint4 *>(base + o * es + (lane & 7) * 16) = x;
                    }
                    __syncwarp();
                };
                if (a.out_f32) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        float x[32];
                        columns(c, x);
                        uint4 v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            v[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]),
                                              __float_as_uint(x[4 * i + 2]),
                                              __float_as_uint(x[4 * i + 3]));
                        store(v, reinterpret_cast<char *>(static_cast<float *>(a.out) + c), 4);
                    }
                } else {
#pragma unroll 1
                    for (int c = 0; c < D; c += 64) {
                        float x[64];
                        columns(c, x);
                        uint4 v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            v[i] = make_uint4(pack_bf16x2(x[8 * i], x[8 * i + 1]),
                                              pack_bf16x2(x[8 * i + 2], x[8 * i + 3]),
                                              pack_bf16x2(x[8 * i + 4], x[8 * i + 5]),
                                              pack_bf16x2(x[8 * i + 6], x[8 * i + 7]));
                        store(v, reinterpret_cast<char *>(static_cast<__nv_bfloat16 *>(a.out) + c), 2);
                    }
                }
                it += n;
            }
            units += nk0 + nk1;
            arrive_warp(&sh.job_empty[item % kJobs]);
            __syncwarp();
        }
    } else {
        regs_dec<88>();
        if (warp == 8) {
            // ---- MMAs ---------------------------------------------------
            if (elect_one()) {
                const uint32_t q_base = smem_u32(sq), kv_base = smem_u32(skv);
                uint32_t e0 = 0, units = 0, used0 = 0, used1 = 0, it0 = 0, it1 = 0;
                bool ok = true;
                for (uint32_t item = 0; ok; ++item) {
                    if (!wait(&sh.job_full[item % kJobs], item / kJobs)) break;
                    const Job &job = sh.job[item % kJobs];
                    const int32_t n = job.n, nk0 = job.nk[0], nk1 = job.nk[1], nu = nk0 + nk1;
                    const int32_t last0 = job.q0[0] + job.nt[0] - 1;
                    const int32_t last1 = job.q0[1] + job.nt[1] - 1;
                    if (n == 0) break;
                    // S of row tile t and key tile j; the row tile's last one
                    // frees the queries
                    auto scores = [&](int t, int32_t j, uint32_t slot) {
                        const uint64_t qd = sdesc_sw128(q_base + t * C::Q_TILE);
                        const uint64_t kd = sdesc_sw128(kv_base + (e0 + 2 * j) % C::STAGES * C::TILE);
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks)
                            mma_half(tmem + slot * C::KEYS,
                                     qd + (((ks >> 2) * C::PANEL + (ks & 3) * 32) >> 4),
                                     kd + (((ks >> 2) * C::KV_PANEL + (ks & 3) * 32) >> 4),
                                     C::IDESC_QK, ks > 0);
                        mma_commit(&sh.s_full[t][((t ? it1 : it0) + j) % C::DEPTH]);
                        if (j == (t ? nk1 : nk0) - 1) mma_commit(&sh.q_empty[t]);
                    };
                    // its queries and keys have arrived (the item's first ones)
                    auto arrived = [&](int t, int32_t j) -> bool {
                        const uint32_t e = e0 + 2 * j;
                        ok = wait(&sh.kv_full[e % C::STAGES], e / C::STAGES) &&
                             (j > 0 || wait(&sh.q_full[t], t ? used1 : used0));
                        tc_fence_after();
                        return ok;
                    };
                    // O_t (+)= P V_j, from a score tile in its use-th use
                    auto products = [&](int t, int32_t j, uint32_t slot, uint32_t use) -> bool {
                        const uint32_t sv = (e0 + 2 * j + 1) % C::STAGES;
                        const uint64_t vd = sdesc_mn(kv_base + sv * C::TILE, C::KV_PANEL);
                        auto product = [&](int ks) {
                            mma_tmem_a(tmem + C::O_BASE + t * D, tmem + slot * C::KEYS + ks * 8,
                                       vd + ks * (2048 >> 4), C::IDESC_PV,
                                       (j > 0 || ks > 0) ? 1u : 0u);
                        };
                        // steps of 16 keys that some row of the tile sees
                        const int32_t steps =
                            min(C::KEYS / 16, ((t ? last1 : last0) - j * C::KEYS) / 16 + 1);
                        // the last item's O_t has been read; V_j and the keys
                        // of the scores to come have arrived when the weights have
                        const uint32_t before = t ? used1 : used0;
                        ok = (j > 0 || before == 0 || wait(&sh.o_free[t], before - 1)) &&
                             wait(&sh.p_full[slot], use);
                        if (!ok) return false;
                        tc_fence_after();
#pragma unroll
                        for (int ks = 0; ks < C::EARLY / 16; ++ks)
                            if (ks < steps) product(ks);
                        if (C::EARLY < C::KEYS) {
                            ok = wait(&sh.p_rest[slot], use);
                            if (!ok) return false;
                            tc_fence_after();
                        }
#pragma unroll
                        for (int ks = C::EARLY / 16; ks < C::KEYS / 16; ++ks)
                            if (ks < steps) product(ks);
                        mma_commit(&sh.pv_done[t][((t ? it1 : it0) + j) % C::DEPTH]);
                        return true;
                    };
                    if constexpr (C::RING) {
                        const int32_t ahead = C::ahead(nk1);
                        auto unit_scores = [&](int32_t u) {
                            const Unit x = unit_at(u, nk0, nk1);
                            scores(x.t, x.j, (units + u) % C::SLOTS);
                            if (x.t == 1 || x.j >= nk1)
                                mma_commit(&sh.kv_empty[(e0 + 2 * x.j) % C::STAGES]);
                        };
                        for (int32_t u = 0; u < min(ahead, nu); ++u) {
                            const Unit x = unit_at(u, nk0, nk1);
                            if (!arrived(x.t, x.j)) break;
                            unit_scores(u);
                        }
                        for (int32_t u = 0; u < nu && ok; ++u) {
                            const Unit x = unit_at(u, nk0, nk1);
                            const uint32_t g = units + u;
                            if (!products(x.t, x.j, g % C::SLOTS, g / C::SLOTS)) break;
                            if (x.t == 1 || x.j >= nk1)
                                mma_commit(&sh.kv_empty[(e0 + 2 * x.j + 1) % C::STAGES]);
                            if (u + ahead < nu) unit_scores(u + ahead);
                        }
                    } else {
                        // (row tiles known to the compiler: operands of the
                        // MMAs stay in uniform registers)
                        if (!arrived(0, 0)) break;
                        scores(0, 0, 0);
                        if (nk1 > 0) {
                            if (!arrived(1, 0)) break;
                            scores(1, 0, 1);
                        }
                        mma_commit(&sh.kv_empty[e0 % C::STAGES]);
                        for (int32_t j = 0; j < n && ok; ++j) {
#pragma unroll
                            for (int t = 0; t < 2; ++t) {
                                if (j >= (t ? nk1 : nk0) || !ok) continue;
                                if (!products(t, j, t, (t ? it1 : it0) + j)) break;
                                if (j + 1 < (t ? nk1 : nk0)) scores(t, j + 1, t);
                            }
                            if (!ok) break;
                            mma_commit(&sh.kv_empty[(e0 + 2 * j + 1) % C::STAGES]);
                            if (j + 1 < n) mma_commit(&sh.kv_empty[(e0 + 2 * j + 2) % C::STAGES]);
                        }
                    }
                    if (!ok) break;
                    e0 += 2 * n;
                    units += nu;
                    used0 += 1;
                    used1 += nk1 > 0;
                    it0 += nk0;
                    it1 += nk1;
                    mbar_arrive(&sh.job_empty[item % kJobs]);
                }
            }
            __syncwarp();
        } else if (warp == 9) {
            // ---- work and copies ----------------------------------------
            const uint32_t q_bytes = (uint32_t)(R * a.G) * 128 * C::PANELS;
            uint32_t index = blockIdx.x, e0 = 0, masked = 0, used[2] = {0, 0};
            bool ok = true, asked = false;
            uint32_t item = 0, asks = 0;
            for (; ok; ++item) {
                if (item > 0)
                    found = index != kNoBlock && find_seq_tile(a.cu_seqlens, a.N, a.T, 1, 2 * R,
                                                               index / a.HKV, cursor, st);
                Job job;
                job.n = 0;
                if (found) {
                    job.begin = st.begin;
                    job.len = st.end - st.begin;
                    job.kvh = index % a.HKV;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        job.q0[t] = (st.tile * 2 + t) * R;
                        job.nt[t] = min(max(job.len - job.q0[t], 0), R);
                        job.nk[t] = job.nt[t] > 0 ? (job.q0[t] + job.nt[t] - 1) / C::KEYS + 1 : 0;
                        job.n = max(job.n, job.nk[t]);
                    }
                    job.last = min(job.q0[0] + 2 * R, job.len) - 1;
                    job.first_mask = (job.q0[0] + 1) / C::KEYS;
                }
                if (item >= kJobs) ok = wait_warp(&sh.job_empty[item % kJobs], item / kJobs - 1);
                if (!ok) break;
                if (lane == 0) {
                    sh.job[item % kJobs] = job;
                    sh.bad[item % kJobs] = 0;
                    mbar_arrive(&sh.job_full[item % kJobs]);
                }
                if (!found) {
                    // the grid's other blocks have nothing to do either: they
                    // are taken here, which is cheaper than their starting
                    while (index != kNoBlock && ok) {
                        if (lane == 0) request_block(&sh.next, &sh.next_full);
                        asked = true;
                        ok = wait_warp(&sh.next_full, asks);
                        if (!ok) break;
                        asked = false;
                        ++asks;
                        index = answered_block(&sh.next);
                        fence_proxy_async();  // the answer is read before it is overwritten
                        __syncwarp();
                    }
                    break;
                }
                if (lane == 0) {
                    auto load_q = [&](int t) {
                        if (job.nk[t] == 0 || !ok) return;
                        if (used[t] > 0) ok = wait(&sh.q_empty[t], used[t] - 1);
                        if (!ok) return;
                        mbar_arrive_expect_tx(&sh.q_full[t], q_bytes);
#pragma unroll
                        for (int p = 0; p < C::PANELS; ++p)
                            tma_load_3d(sq + t * C::Q_TILE + p * C::PANEL, &map_q, p * 64,
                                        job.kvh * a.G, job.begin + job.q0[t], &sh.q_full[t]);
                        ++used[t];
                    };
                    load_q(0);
                    for (int32_t i = 0; i < 2 * job.n && ok; ++i) {
                        const uint32_t s = e0 % C::STAGES;
                        // not before the item's last tiles: a CTA with a long
                        // item ahead would hold a second one back from others
                        if (i == 2 * job.n - 2) {
                            request_block(&sh.next, &sh.next_full);
                            asked = true;
                        }
                        if (e0 >= C::STAGES) ok = wait(&sh.kv_empty[s], e0 / C::STAGES - 1);
                        if (!ok) break;
                        // a value tile with masked places goes by way of warps 10-11
                        const int32_t j = i >> 1;
                        const bool m = (i & 1) && j >= job.first_mask;
                        uint64_t *full = m ? &sh.v_raw[masked % kMasked] : &sh.kv_full[s];
                        masked += m;
                        mbar_arrive_expect_tx(full, C::TILE);
#pragma unroll
                        for (int p = 0; p < C::PANELS; ++p)
                            tma_load_3d(skv + s * C::TILE + p * C::KV_PANEL, (i & 1) ? &map_v : &map_k,
                                        p * 64, job.kvh, job.begin + j * C::KEYS, full);
                        ++e0;
                        if (i == 0) load_q(1);
                    }
                }
                ok = __all_sync(0xffffffffu, ok) && wait_warp(&sh.next_full, asks);
                if (!ok) break;
                asked = false;
                ++asks;
                index = answered_block(&sh.next);
                fence_proxy_async();  // the answer is read before it is overwritten
                __syncwarp();
            }
            if (lane == 0) {
                // the CTA may end when every copy and answer has landed and
                // every commit that names one of its barriers has arrived
                if (asked) (void)mbar_wait_bounded(&sh.next_full, asks & 1, kWaitLimit);
                for (int t = 0; t < 2; ++t)
                    if (used[t]) {
                        (void)mbar_wait_bounded(&sh.q_full[t], (used[t] - 1) & 1, kWaitLimit);
                        if (ok && !sh.abort) ok = wait(&sh.q_empty[t], used[t] - 1);
                    }
                for (uint32_t m = masked > kMasked ? masked - kMasked : 0; m < masked; ++m)
                    (void)mbar_wait_bounded(&sh.v_raw[m % kMasked], (m / kMasked) & 1, kWaitLimit);
                for (uint32_t e = e0 > C::STAGES ? e0 - C::STAGES : 0; e < e0; ++e) {
                    if (ok && !sh.abort) ok = wait(&sh.kv_empty[e % C::STAGES], e / C::STAGES);
                    else (void)mbar_wait_bounded(&sh.kv_full[e % C::STAGES], (e / C::STAGES) & 1, kWaitLimit);
                }
            }
        } else {
            // ---- masked value tiles, and arrivals ------------------------
            const int who = tid - 10 * 32;  // 0..63
            uint32_t e0 = 0, masked = 0, units = 0, it0 = 0, it1 = 0;
            bool ok = true;
            for (uint32_t item = 0; ok; ++item) {
                if (!wait_warp(&sh.job_full[item % kJobs], item / kJobs)) break;
                const Job &job = sh.job[item % kJobs];
                const int32_t n = job.n, first_mask = job.first_mask, last = job.last;
                const int32_t nk0 = job.nk[0], nk1 = job.nk[1], nu = nk0 + nk1;
                if (n == 0) break;
                // the score tile of (t, j), and its use
                auto slot_of = [&](int t, int32_t j) -> uint32_t {
                    return C::RING ? (units + unit_of(t, j, nk0, nk1)) % C::SLOTS : (uint32_t)t;
                };
                auto use_of = [&](int t, int32_t j) -> uint32_t {
                    return C::RING ? (units + unit_of(t, j, nk0, nk1)) / C::SLOTS
                                   : (t ? it1 : it0) + j;
                };
                // from the keys that no wait of the MMAs' thread covers
                const int32_t ahead = C::ahead(nk1);
                int32_t next_k = C::RING ? unit_at(min(ahead, nu) - 1, nk0, nk1).j + 1 : 1;
                for (int32_t j = warp == 10 ? 0 : first_mask; j < n && ok; ++j) {
                    const uint32_t ev = e0 + 2 * j + 1, sv = ev % C::STAGES;
                    if (j >= first_mask) {
                        const uint32_t mi = masked % kMasked, mu = masked / kMasked;
                        ++masked;
                        ok = wait_warp(&sh.v_raw[mi], mu);
                        if (!ok) break;
                        // rows the item sees, and those the MMAs read
                        const int32_t rows = min(C::KEYS, last + 1 - j * C::KEYS);
                        const int32_t read = (rows + 15) & ~15;
                        bool found = false;
#pragma unroll 1
                        for (int p = 0; p < C::PANELS; ++p) {
                            uint4 *v = reinterpret_cast<uint4 *>(skv + sv * C::TILE + p * C::KV_PANEL);
                            for (int i = rows * 8 + who; i < read * 8; i += 64)
                                v[i] = make_uint4(0, 0, 0, 0);
#pragma unroll 1
                            for (int i0 = who; i0 < rows * 8; i0 += 64 * 8) {
                                uint4 x[8];
                                uint32_t any = 0;
#pragma unroll
                                for (int u = 0; u < 8; ++u)
                                    x[u] = i0 + u * 64 < rows * 8 ? v[i0 + u * 64]
                                                                  : make_uint4(0, 0, 0, 0);
#pragma unroll
                                for (int u = 0; u < 8; ++u) any |= all_ones(x[u]);
                                if (any == 0) continue;
                                found = true;
#pragma unroll
                                for (int u = 0; u < 8; ++u) {
                                    if (all_ones(x[u]) == 0) continue;
                                    uint32_t *w = &x[u].x;
#pragma unroll
                                    for (int b = 0; b < 4; ++b) {
                                        if ((w[b] & 0x7F80u) == 0x7F80u) w[b] &= 0xFFFF0000u;
                                        if ((w[b] & 0x7F800000u) == 0x7F800000u) w[b] &= 0x0000FFFFu;
                                    }
                                    v[i0 + u * 64] = x[u];
                                }
                            }
                        }
                        if (found) sh.bad[item % kJobs] = 1;
                        fence_proxy_async();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&sh.v_half[mi]);
                            if (warp == 10 && wait(&sh.v_half[mi], mu)) mbar_arrive(&sh.kv_full[sv]);
                        }
                        __syncwarp();
                    }
                    if (warp == 10) {
                        // V_j has arrived, and the keys of the scores that
                        // follow its products (in time for their barrier: see
                        // Cfg::ahead): one of the arrivals that let those go
                        ok = wait_warp(&sh.kv_full[sv], ev / C::STAGES);
                        int32_t to = min(j + 1, n - 1);
                        if (C::RING) {
                            const int32_t u = unit_of(nk1 > j, j, nk0, nk1) + ahead;
                            to = unit_at(min(u, nu - 1), nk0, nk1).j;
                        }
                        for (; next_k <= to && ok; ++next_k) {
                            const uint32_t ek = e0 + 2 * next_k;
                            ok = wait_warp(&sh.kv_full[ek % C::STAGES], ek / C::STAGES);
                        }
                        if (!ok) break;
                        if (lane < 2 && j < (lane ? nk1 : nk0))
                            mbar_arrive(&sh.p_full[slot_of(lane, j)]);
                        __syncwarp();
                        // not a phase ahead of the weights
                        for (int t = 0; t < 2 && ok; ++t)
                            if (j < (t ? nk1 : nk0))
                                ok = wait_warp(&sh.p_full[slot_of(t, j)], use_of(t, j));
                    }
                }
                if (!ok) break;
                e0 += 2 * n;
                units += nu;
                it0 += nk0;
                it1 += nk1;
                arrive_warp(&sh.job_empty[item % kJobs]);
                __syncwarp();
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        if (sh.abort) {
            // MMAs may still be in flight: one more commit follows them all
            if (elect_one()) {
                mma_commit(&sh.drained);
                (void)mbar_wait_bounded(&sh.drained, 0, kWaitLimit);
            }
            __syncwarp();
        }
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, int K>
cudaError_t launch_t(const AttnArgs &a, cudaStream_t stream) {
    const int32_t R = kRowTile / a.G;
    CUtensorMap mq, mk, mv;
    memset(&mq, 0, sizeof(mq));
    memset(&mk, 0, sizeof(mk));
    memset(&mv, 0, sizeof(mv));
    if (!encode_rows_map(&mq, a.q, D, a.HQ, a.T, a.q_stride, (uint32_t)a.G, (uint32_t)R) ||
        !encode_rows_map(&mk, a.k, D, a.HKV, a.T, a.k_stride, 1, K) ||
        !encode_rows_map(&mv, a.v, D, a.HKV, a.T, a.v_stride, 1, K))
        return cudaErrorInvalidValue;
    const cudaError_t e = allow_smem<attn_tc_kernel<D, K>>(smem_bytes<D, K>());
    if (e != cudaSuccess) return e;
    const int64_t tiles = (int64_t)a.T / (2 * R) + a.N;
    attn_tc_kernel<D, K>
        <<<(unsigned)(tiles * a.HKV), kThreads, smem_bytes<D, K>(), stream>>>(mq, mk, mv, a);
    return cudaGetLastError();
}

}  // namespace

// 128 keys to a tile where rows see many keys: half as many hand-overs between
// the tensor core and the softmax (16 x 4096 tokens, 32/8 heads: d = 128 1406
// us, 64 keys 1752; d = 64 1170, 1421).  64 keys, and a ring of score tiles,
// where they see few: less of a tile lies behind the diagonal, and scores are
// taken ahead while the softmax runs (1000 x 64 tokens, 32/8 heads: d = 128 201
// us, 128 keys 248; d = 64 147, 226; 300 prompts of 200 tokens on average: 308,
// 393; 266, 333; 100 of 700: 601, 615; 411, 461; with 16/16 heads 399, 385;
// 338, 343).  So the border lies between 512 and 700 tokens or above, by width
// and group; one border for all gives up as much as 12% (d = 64, 32/8 heads, a
// mean of 700).  The host knows the mean length alone, so that decides, and
// empty sequences count in it: one prompt of 16384 tokens with 63 empty ones
// takes 64-key tiles (d = 128: 1663 us, alone 1217; d = 64: 1352, 970).  A lone
// prompt has no other work to fill the hand-overs with (400 tokens, 32/8 heads:
// 12.5 us, 128 keys 11.9; 100 tokens 8.7, 9.2).
cudaError_t launch_attn_tc(const AttnArgs &a, cudaStream_t stream) {
    const bool small = a.T <= (int64_t)(a.N == 1 ? 128 : 512) * a.N;
    if (a.D == 64) return small ? launch_t<64, 64>(a, stream) : launch_t<64, 128>(a, stream);
    return small ? launch_t<128, 64>(a, stream) : launch_t<128, 128>(a, stream);
}

}  // namespace kda
