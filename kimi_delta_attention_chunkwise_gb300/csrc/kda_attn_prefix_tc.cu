// kda_attn_prefix_tc.cu -- the shared tokens of kda_attn_step_shared on the tensor
// cores: bf16, head width D = 64 or 128.
//
//     z_rj = scale <q_r, k_j>,  m_r = max_j z_rj,  l_r = sum_j e^{z_rj - m_r},
//     o_r = sum_j e^{z_rj - m_r} v_j       (j < S; a row r: sequence and query head)
//
// The rows of a 128-row tile are R = floor(128 / G) sequences times the G query
// heads of a key-value head, brought in by one tensor copy.  A piece of work is
// one or two row tiles of one key-value head over a run of key tiles of 128
// tokens (PrefixLine: equal shares for one CTA to an SM).  Per row tile t and
// key tile j, in the order (0, 0), (1, 0), (0, 1), ...:
//
//     S = Q_t K_j^T            tcgen05, operands in shared memory, D in TMEM
//     P = 2^{c S - ref}        one thread per row; two bf16 parts, over S's columns
//     O_t (+)= P V_j           tcgen05, A = P's parts from TMEM, V_j as it lies
//
// The parts leave 2^-15 of a weight out, as kda_attn_step's do: one part, 2^-8, would
// make a sequence's result depend on how many others share its pages (MmaCore's cores
// work on up to kFewRows rows).  The second product is half as much tensor work again.
//
// Two score tiles take the units in turn and the scores run two units ahead of
// the products: with two row tiles the tensor core works for one while the
// weights of the other are taken, with one on the next key tile.  Keys and
// values come a page at a time (up to 128 rows to a copy).  Nothing is masked
// but what lies behind the shared tokens, whole steps of 16 keys, which no copy
// brings and no product reads, and the tokens of pages that do not exist, which
// copies from outside of the cache leave at zero.  References move as in
// kda_attn_tc.cu: by more than 2^8 or not at all.
//
// A unit, two row tiles against 128 keys, takes 2.27 us of an SM at d = 128 (a row tile
// alone 1.65; d = 64: 1.77 and 1.01), with the second parts 25 MFLOP: 0.88 of the tensor
// cores' measured rate (with one part 1.6 us, 0.83).  A row tile alone waits for its own
// weights and they for its scores.  Few sequences are bound by the keys' and values'
// bytes, many by the units (32/8 heads, d = 128, no tokens but the shared ones, with the
// join: 32 sequences, 32768 keys 40.5 us, 3.3 TB/s; 256 sequences 142 us, 1450 TFLOP/s).
//
// Warps: 0-3 and 4-7 the weights and results of row tile 0 and 1, 8 issues the
// MMAs, 9 the copies.  Waits are bounded as there.
#include <algorithm>
#include <cstdint>
#include <cstring>

#include "kda_attn_ptx.cuh"
#include "kda_attn_step.cuh"

namespace kda {
namespace {

namespace prefix_tc {

constexpr int kThreadsTc = 384;
constexpr int kRowTile = 128, kKeys = kPrefixTile;
constexpr float kMoveBy = 8.f;
constexpr uint32_t kStage = 32 * 128;  // bytes a warp's results pass through

template <int D>
struct Cfg {
    static constexpr int PANELS = D / 64;
    static constexpr uint32_t PANEL = kRowTile * 128, TILE = PANELS * PANEL;  // bytes: Q, K and V alike
    static constexpr int STAGES = D == 128 ? 4 : 8;  // K and V tiles in flight
    // keys whose weights go to the product first (256 sequences, 32768 keys, d = 128:
    // 142 us, with 32 153)
    static constexpr int EARLY = 64;
    static constexpr uint32_t O_BASE = 2 * kKeys;     // TMEM columns: two score tiles, O_0, O_1
    static constexpr uint32_t IDESC_QK = idesc_bf16_f32(128, kKeys);
    static constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, D) | (1u << 16);  // V is N-major
};

struct Shared {
    uint64_t q_full[2], q_empty[2], kv_full[8], kv_empty[8];
    uint64_t s_full[2][2], pv_done[2][2], o_free[2];  // by row tile (and its units, in turn)
    uint64_t p_full[2], p_rest[2];                    // by score tile
    uint64_t drained;
    unsigned long long own;
    uint32_t tmem;
    int32_t abort, seq;
};

template <int D>
constexpr uint32_t smem_bytes() {
    return (2 + Cfg<D>::STAGES) * Cfg<D>::TILE + 8 * kStage + (uint32_t)sizeof(Shared);
}
static_assert(smem_bytes<128>() <= 232448 && smem_bytes<64>() <= 232448, "227 KB per CTA");

// What a piece's row tiles hold.
struct Rows {
    int32_t n0[2];  // first sequence
    int32_t n[2];   // sequences (0: no such row tile)
    __device__ Rows(const AttnStepArgs &a, int32_t R, int32_t block) {
        const int32_t per = a.prefix_rows / a.G;  // R or 2 R
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            n0[t] = block * per + t * R;
            n[t] = t * R < per ? min(max(a.N - n0[t], 0), R) : 0;
        }
    }
    __device__ bool two() const { return n[1] > 0; }
};

// 8 columns of TMEM (st16_nowait, half of it)
__device__ __forceinline__ void st8_nowait(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
        : "memory");
}
// Two weights as two bf16 parts each that leave 2^-15 out: hi is w less 2^-9 of it, cut
// off, and lo the rest, rounded.  Less 2^-9, so that lo is positive where hi is (an
// infinite value times a low part of 0 would be a NaN); for w in 1 .. 2 the rest is below
// 2^-7 + 2^-8, and half a step of it 2^-15, as of 2^-7.
__device__ __forceinline__ void split_weight_pair(float2 w, uint32_t &hi, uint32_t &lo) {
    constexpr float kLess = 1.f - 0x1p-9f;
    const float2 h = f2_mul(w, make_float2(kLess, kLess));
    const uint32_t x = __float_as_uint(h.x), y = __float_as_uint(h.y);
    hi = __byte_perm(x, y, 0x7632);
    const float2 rest = f2_add(w, make_float2(__uint_as_float((x & 0xFFFF0000u) | 0x80000000u),
                                              __uint_as_float((y & 0xFFFF0000u) | 0x80000000u)));
    lo = pack_bf16x2(rest.x, rest.y);
}

template <int D>
__global__ void __launch_bounds__(kThreadsTc, 1)
attn_prefix_tc_kernel(const __grid_constant__ CUtensorMap map_q,
                      const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v, const AttnStepArgs a,
                      const int32_t outside) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *sq = smem, *skv = smem + 2 * C::TILE, *sout = skv + C::STAGES * C::TILE;
    Shared &sh = *reinterpret_cast<Shared *>(sout + 8 * kStage);
    if (smem_u32(smem) & 1023u) {  // the swizzled tiles would not match their descriptors
        *a.status = KDA_ERR_CUDA;
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_launch_dependents();
    const int32_t shared = shared_tokens(a);
    if (blockIdx.x == 0 && tid == 0) check_shared_pages(a);
    PrefixLine line(a, shared);
    const int32_t cta = (int32_t)blockIdx.x;
    if (cta >= line.grid) return;
    const int32_t seq = sharing_sequence<kThreadsTc>(a, shared, &sh.seq, &sh.own);
    if (seq >= a.N) return;
    line.grid = min(line.grid, sm_split(a, line, (int64_t)sh.own).prefix);
    if (cta >= line.grid) return;
    const int32_t R = kRowTile / a.G;  // sequences of a row tile
    const int32_t *table = a.block_table + (int64_t)seq * a.max_pages;
    const int64_t u0 = share_start(line.units, cta, line.grid),
                  u1 = share_start(line.units, cta + 1, line.grid);

    if (warp == 0 && lane == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(&sh.q_full[t], 1);
            mbar_init(&sh.q_empty[t], 1);
            for (int b = 0; b < 2; ++b) {
                mbar_init(&sh.s_full[t][b], 1);
                mbar_init(&sh.pv_done[t][b], 1);
            }
            mbar_init(&sh.o_free[t], 4);
            mbar_init(&sh.p_full[t], 4);
            mbar_init(&sh.p_rest[t], 4);
        }
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&sh.kv_full[i],
                      1 + (a.withhold == KDA_WITHHOLD_SHARED && cta == 0 && i == 0));
            mbar_init(&sh.kv_empty[i], 1);
        }
        mbar_init(&sh.drained, 1);
        sh.abort = 0;
        fence_mbar_init();
        fence_proxy_async();
    } else if (warp == 8) {
        tmem_alloc(&sh.tmem, 512);
        tmem_relinquish();
    } else if (warp == 9 && lane < 3) {
        const CUtensorMap *m = lane == 0 ? &map_q : lane == 1 ? &map_k : &map_v;
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;

    // Waits of one thread and of a whole warp; `use` counts the barrier's phases.
    auto wait = [&](uint64_t *bar, uint32_t use) -> bool {
        if (mbar_try_wait(bar, use & 1)) return true;
        if (mbar_wait_bounded(bar, use & 1, a.wait_limit)) return true;
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
    // the page of token `tok` (a multiple of 16), -1: none
    auto page_at = [&](int32_t tok) -> int32_t {
        const int32_t page = table[tok >> a.page_shift];
        return page >= 0 && page < a.num_pages ? page : -1;
    };

    if (warp < 8) {
        // ---- weights and results: one thread per row ----------------------
        regs_inc<208>();
        const int t = warp >> 2, row = tid & 127;
        const uint32_t lane_base = (uint32_t)(warp & 3) * 32;
        const uint32_t o_addr = tmem_addr(tmem, lane_base, C::O_BASE + t * D);
        const int32_t in_tile = row / a.G, g = row - in_tile * a.G;
        const float c2 = a.scale * tc::kLog2e;
        uint32_t it = 0, units = 0;  // key tiles of this row tile, and units, so far
        bool ok = true;
        for (int64_t u = u0; u < u1 && ok;) {
            const PrefixPiece piece(line, cta, u, u1);
            const Rows rows(a, R, piece.block);
            const int32_t n = piece.tile1 - piece.tile0;
            const bool two = rows.two();
            u += n;
            if (t == 1 && !two) {
                units += n;
                continue;
            }
            const bool mine = in_tile < rows.n[t];  // the row is a sequence's
            // the steps of 16 keys that there are, a bit each
            auto entry_of = [&](int32_t j) -> bool {
                const int32_t tok = (piece.tile0 + j) * kKeys + lane * 16;
                return j < n && lane < 8 && tok < shared && page_at(tok) >= 0;
            };
            bool entry = entry_of(0);
            float ref = -INFINITY, sum = 0.f;  // the reference times c2
            bool seen = false;
            for (int32_t j = 0; j < n; ++j) {
                const uint32_t slot = (units + (two ? 2 * j + t : j)) & 1;
                const uint32_t s_addr = tmem_addr(tmem, lane_base, slot * kKeys);
                const uint32_t there = __ballot_sync(0xffffffffu, entry);
                entry = entry_of(j + 1);
                seen = seen || there != 0;
                ok = wait_warp(&sh.s_full[t][(it + j) & 1], (it + j) >> 1);
                if (!ok) break;
                tc_fence_after();
                float s[kKeys];
#pragma unroll
                for (int i = 0; i < kKeys; i += 32) ld32_nowait(s_addr + i, s + i);
#pragma unroll
                for (int i = 0; i < kKeys; i += 32) wait_ld32(s + i);
                if (there != 0xFFu) {
#pragma unroll
                    for (int i = 0; i < kKeys; ++i)
                        if (!(there >> (i / 16) & 1)) s[i] = -INFINITY;
                }
                float m[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) m[i] = fmaxf(s[i], s[i + 4]);
#pragma unroll
                for (int i = 8; i < kKeys; i += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e) m[e] = max3(m[e], s[i + e], s[i + e + 4]);
                const float top = fmaxf(max3(m[0], m[1], m[2]), m[3]) * c2;
                // (also on the first tile; rows without a sequence hold anything)
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
                    if (j > 0) {
                        ok = wait_warp(&sh.pv_done[t][(it + j - 1) & 1], (it + j - 1) >> 1);
                        if (!ok) break;
                        tc_fence_after();
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
                for (int h = 0; h < kKeys / 16; ++h) {
                    // (16 keys at a time: 32 spill 244 bytes of registers, this 52)
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float2 x = f2_fma(make_float2(s[h * 16 + 2 * i], s[h * 16 + 2 * i + 1]), c22,
                                          neg2);
                        x.x = exp2_approx(x.x);
                        x.y = exp2_approx(x.y);
                        if (i & 1) acc1 = f2_add(acc1, x);
                        else acc0 = f2_add(acc0, x);
                        split_weight_pair(x, hi[i], lo[i]);
                    }
                    st8_nowait(s_addr + h * 8, hi);
                    st8_nowait(s_addr + kKeys / 2 + h * 8, lo);
                    if (h == C::EARLY / 16 - 1 || h == kKeys / 16 - 1) {
                        tmem_wait_st();
                        tc_fence_before();
                        arrive_warp(h == C::EARLY / 16 - 1 ? &sh.p_full[slot] : &sh.p_rest[slot]);
                        __syncwarp();
                    }
                }
                acc0 = f2_add(acc0, acc1);
                sum += acc0.x + acc0.y;
            }
            if (!ok) break;
            // the states: whole lines by way of shared memory (the 128-byte
            // swizzle keeps both sides free of bank conflicts)
            ok = wait_warp(&sh.pv_done[t][(it + n - 1) & 1], (it + n - 1) >> 1);
            if (!ok) break;
            tc_fence_after();
            const PrefixState p = prefix_state(a, D, piece.index);
            const int64_t at = mine ? (int64_t)(rows.n0[t] + in_tile) * a.HQ + piece.kvh * a.G + g : -1;
            if (mine) {
                p.m[at] = state_max(ref, seen);
                p.l[at] = sum;
                if (piece.last) p.pieces[at] = piece.index + 1;
            }
            uint8_t *mine_out = sout + warp * kStage;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float x[32];
                __syncwarp();  // the loads are the whole warp's
                ld32_nowait(o_addr + c, x);
                wait_ld32(x);
                if (c + 32 == D) {
                    tc_fence_before();
                    arrive_warp(&sh.o_free[t]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<float4 *>(mine_out + sw128_chunk(lane, i)) =
                        make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                __syncwarp();
#pragma unroll
                for (int r = 0; r < 32; r += 4) {
                    const int rr = r + (lane >> 3);
                    const float4 y =
                        *reinterpret_cast<const float4 *>(mine_out + sw128_chunk(rr, lane & 7));
                    const int64_t o = __shfl_sync(0xffffffffu, at, rr);
                    if (o >= 0) *reinterpret_cast<float4 *>(p.o + o * D + c + (lane & 7) * 4) = y;
                }
            }
            it += n;
            units += two ? 2 * n : n;
        }
    } else {
        regs_dec<88>();
        if (warp == 8) {
            // ---- MMAs ---------------------------------------------------
            if (elect_one()) {
                const uint32_t q_base = smem_u32(sq), kv_base = smem_u32(skv);
                uint32_t e0 = 0, units = 0, used0 = 0, used1 = 0, it0 = 0, it1 = 0;
                bool ok = true;
                for (int64_t u = u0; u < u1 && ok;) {
                    const PrefixPiece piece(line, cta, u, u1);
                    const Rows rows(a, R, piece.block);
                    const int32_t n = piece.tile1 - piece.tile0;
                    const bool two = rows.two();
                    const int32_t nu = two ? 2 * n : n;
                    u += n;
                    auto tile_of = [&](int32_t x) -> int { return two ? x & 1 : 0; };
                    auto key_of = [&](int32_t x) -> int32_t { return two ? x >> 1 : x; };
                    // S of unit x, whose keys (and, the first time, queries) it waits
                    // for; the row tile's last one frees the queries
                    auto scores = [&](int32_t x) {
                        const int t = tile_of(x);
                        const int32_t j = key_of(x);
                        const uint32_t e = e0 + 2 * j;
                        ok = wait(&sh.kv_full[e % C::STAGES], e / C::STAGES) &&
                             (j > 0 || wait(&sh.q_full[t], t ? used1 : used0));
                        if (!ok) return;
                        tc_fence_after();
                        const uint32_t slot = (units + x) & 1;
                        const uint64_t qd = sdesc_sw128(q_base + t * C::TILE);
                        const uint64_t kd = sdesc_sw128(kv_base + e % C::STAGES * C::TILE);
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks) {
                            const uint32_t at = ((ks >> 2) * C::PANEL + (ks & 3) * 32) >> 4;
                            mma_half(tmem + slot * kKeys, qd + at, kd + at, C::IDESC_QK, ks > 0);
                        }
                        mma_commit(&sh.s_full[t][((t ? it1 : it0) + j) & 1]);
                        if (!two || t == 1) mma_commit(&sh.kv_empty[e % C::STAGES]);
                        if (j == n - 1) mma_commit(&sh.q_empty[t]);
                    };
                    // O_t (+)= P V_j of unit x
                    auto products = [&](int32_t x) {
                        const int t = tile_of(x);
                        const int32_t j = key_of(x);
                        const uint32_t e = e0 + 2 * j + 1;
                        const uint32_t slot = (units + x) & 1, use = (units + x) >> 1;
                        const uint64_t vd = sdesc_mn(kv_base + e % C::STAGES * C::TILE, C::PANEL);
                        // steps of 16 keys that there are (the last tile may hold less)
                        const int32_t steps =
                            min(kKeys / 16, (shared - (piece.tile0 + j) * kKeys) / 16);
                        // the last piece's O_t has been read
                        const uint32_t before = t ? used1 : used0;
                        ok = wait(&sh.kv_full[e % C::STAGES], e / C::STAGES) &&
                             (j > 0 || before == 0 || wait(&sh.o_free[t], before - 1)) &&
                             wait(&sh.p_full[slot], use);
                        if (!ok) return;
                        tc_fence_after();
                        auto product = [&](int ks) {
                            const uint32_t o = tmem + C::O_BASE + t * D;
                            const uint32_t p = tmem + slot * kKeys + ks * 8;
                            mma_tmem_a(o, p, vd + ks * (2048 >> 4), C::IDESC_PV,
                                       (j > 0 || ks > 0) ? 1u : 0u);
                            mma_tmem_a(o, p + kKeys / 2, vd + ks * (2048 >> 4), C::IDESC_PV, 1u);
                        };
#pragma unroll
                        for (int ks = 0; ks < C::EARLY / 16; ++ks)
                            if (ks < steps) product(ks);
                        ok = wait(&sh.p_rest[slot], use);
                        if (!ok) return;
                        tc_fence_after();
#pragma unroll
                        for (int ks = C::EARLY / 16; ks < kKeys / 16; ++ks)
                            if (ks < steps) product(ks);
                        mma_commit(&sh.pv_done[t][((t ? it1 : it0) + j) & 1]);
                        if (!two || t == 1) mma_commit(&sh.kv_empty[e % C::STAGES]);
                    };
                    scores(0);
                    if (ok && nu > 1) scores(1);
                    for (int32_t x = 0; x < nu && ok; ++x) {
                        products(x);
                        if (ok && x + 2 < nu) scores(x + 2);
                    }
                    if (!ok) break;
                    e0 += 2 * n;
                    units += nu;
                    used0 += 1;
                    it0 += n;
                    if (two) {
                        used1 += 1;
                        it1 += n;
                    }
                }
            }
            __syncwarp();
        } else if (warp == 9) {
            // ---- copies -------------------------------------------------
            const uint32_t q_bytes = (uint32_t)(R * a.G) * 128 * C::PANELS;
            const int32_t box = min(1 << a.page_shift, kKeys);     // rows of a copy
            const int32_t copies = kKeys / box;                    // to a panel
            uint32_t e0 = 0, used[2] = {0, 0};
            bool ok = true;
            for (int64_t u = u0; u < u1 && ok;) {
                const PrefixPiece piece(line, cta, u, u1);
                const Rows rows(a, R, piece.block);
                const int32_t n = piece.tile1 - piece.tile0;
                u += n;
                auto load_q = [&](int t) {
                    if (rows.n[t] == 0 || !ok) return;
                    if (used[t] > 0) ok = wait_warp(&sh.q_empty[t], used[t] - 1);
                    if (!ok) return;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&sh.q_full[t], q_bytes);
#pragma unroll
                        for (int p = 0; p < C::PANELS; ++p)
                            tma_load_3d(sq + t * C::TILE + p * C::PANEL, &map_q, p * 64,
                                        piece.kvh * a.G, rows.n0[t], &sh.q_full[t]);
                    }
                    __syncwarp();
                    ++used[t];
                };
                // lane: the copy of panel lane / copies, rows (lane % copies) * box ..
                const int32_t part = lane % copies, panel = lane / copies;
                auto z_of = [&](int32_t j) -> int32_t {  // -1: nothing there to copy
                    const int32_t tok = (piece.tile0 + j) * kKeys + part * box;
                    if (j >= n || panel >= C::PANELS || tok >= shared) return -1;
                    const int32_t page = page_at(tok);
                    if (page < 0) *a.status = KDA_ERR_INVALID_ARG;
                    const int64_t z = (int64_t)page * a.HKV + piece.kvh;
                    return page < 0 || z >= outside ? outside : (int32_t)z;
                };
                load_q(0);
                int32_t z = z_of(0);
                for (int32_t j = 0; j < n && ok; ++j) {
                    const int32_t next = z_of(j + 1);
                    const int32_t first = (piece.tile0 + j) * kKeys + part * box;
                    const uint32_t bytes =
                        (uint32_t)__popc(__ballot_sync(0xffffffffu, z >= 0)) * box * 128;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const uint32_t s = e0 % C::STAGES;
                        if (e0 >= (uint32_t)C::STAGES)
                            ok = wait_warp(&sh.kv_empty[s], e0 / C::STAGES - 1);
                        if (!ok) break;
                        if (lane == 0) mbar_arrive_expect_tx(&sh.kv_full[s], bytes);
                        __syncwarp();
                        if (z >= 0) {
                            uint8_t *to = skv + s * C::TILE + panel * C::PANEL + part * box * 128;
                            const CUtensorMap *map = kv ? &map_v : &map_k;
                            const int32_t row = first & ((1 << a.page_shift) - 1);
                            // (65536 keys, 24 rows: 60.5 us, 63.2 by the other kind)
                            if (line.blocks == 1)
                                tma_load_3d_once(to, map, panel * 64, row, z, &sh.kv_full[s]);
                            else
                                tma_load_3d(to, map, panel * 64, row, z, &sh.kv_full[s]);
                        }
                        __syncwarp();
                        ++e0;
                    }
                    if (j == 0) load_q(1);
                    z = next;
                }
            }
            // the CTA may end when every copy has landed and every commit that names
            // one of its barriers has arrived
            for (int t = 0; t < 2; ++t)
                if (used[t]) {
                    (void)mbar_wait_bounded(&sh.q_full[t], (used[t] - 1) & 1, a.wait_limit);
                    if (ok && !sh.abort) ok = wait_warp(&sh.q_empty[t], used[t] - 1);
                }
            for (uint32_t e = e0 > C::STAGES ? e0 - C::STAGES : 0; e < e0; ++e) {
                if (ok && !sh.abort) ok = wait_warp(&sh.kv_empty[e % C::STAGES], e / C::STAGES);
                else (void)mbar_wait_bounded(&sh.kv_full[e % C::STAGES], (e / C::STAGES) & 1, a.wait_limit);
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
                (void)mbar_wait_bounded(&sh.drained, 0, a.wait_limit);
            }
            __syncwarp();
        }
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// A cache of [rows of pages, page, D] bf16 as a 3-D map whose box is up to 128 rows
// of 64 channels of one page, with the 128-byte swizzle.
bool encode_cache_map(CUtensorMap *m, const void *base, int32_t d, int32_t page, int32_t heads) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)page, (cuuint64_t)heads};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)page * d * 2};
    const cuuint32_t box[3] = {64u, (cuuint32_t)std::min(page, kKeys), 1u};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_t(const AttnStepArgs &a, cudaStream_t stream) {
    const int32_t R = kRowTile / a.G, page = 1 << a.page_shift;
    // heads of pages; the copies of pages that do not exist name the one behind
    // them.  (A cache of no pages: any address, of which nothing is read)
    const int64_t heads = std::min<int64_t>((int64_t)a.num_pages * a.HKV, INT32_MAX - 1);
    const int32_t outside = (int32_t)std::max<int64_t>(heads, 1);
    CUtensorMap mq, mk, mv;
    memset(&mq, 0, sizeof(mq));
    memset(&mk, 0, sizeof(mk));
    memset(&mv, 0, sizeof(mv));
    if (!encode_rows_map(&mq, a.q, D, a.HQ, a.N, a.q_stride, (uint32_t)a.G, (uint32_t)R) ||
        !encode_cache_map(&mk, heads ? a.k_cache : a.q, D, page, outside) ||
        !encode_cache_map(&mv, heads ? a.v_cache : a.q, D, page, outside))
        return cudaErrorInvalidValue;
    const cudaError_t e = allow_smem<attn_prefix_tc_kernel<D>>(smem_bytes<D>());
    if (e != cudaSuccess) return e;
    attn_prefix_tc_kernel<D>
        <<<(unsigned)a.prefix_grid, kThreadsTc, smem_bytes<D>(), stream>>>(mq, mk, mv, a, outside);
    return cudaGetLastError();
}

}  // namespace prefix_tc
}  // namespace

int32_t prefix_tc_rows(const AttnStepArgs &a) {
    const int32_t R = prefix_tc::kRowTile / a.G;
    return (a.N > R ? 2 * R : R) * a.G;
}

cudaError_t launch_prefix_tc(const AttnStepArgs &a, cudaStream_t stream) {
    return a.D == 64 ? prefix_tc::launch_t<64>(a, stream) : prefix_tc::launch_t<128>(a, stream);
}

}  // namespace kda
