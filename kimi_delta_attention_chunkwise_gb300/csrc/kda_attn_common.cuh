// kda_attn_common.cuh -- what the prompt-attention engines share: the map from
// a block index to a tile of one sequence.
#pragma once

#include <cstdint>

#include "kda_attn.cuh"

namespace kda {

// A tile of a sequence's rows: tokens [begin, end) are the sequence's.
struct SeqTile {
    int32_t begin, end;  // the sequence's tokens in the packed axis
    int32_t tile;        // index of the tile within the sequence
};

// Where a search stands: a lane's run of neighbouring sequences from s0 (of the
// warp's 128), with the tiles before them.
struct TileCursor {
    static constexpr int PER = 4;  // sequences per lane
    int32_t s0 = -1;               // -1: nothing looked up yet
    uint32_t base = 0, incl = 0, mine = 0;  // tiles before s0, up to and in the lane's run
    int32_t begin[PER], end[PER];
    uint32_t n[PER];
};

// The `index`-th tile over all sequences, tokens(s) * rows_per_token rows of
// sequence s in tiles of tile_rows (counts that fit 32 bits).  A sequence's
// tiles come last tile first: under the causal mask the last is the longest,
// and long tiles that start early leave no long tail.  Called by one whole
// warp; false when there is no such tile.  The cursor carries the search over
// to the next: a larger index goes on where the last was found, without a
// read as long as it stays within the 128 sequences at hand.
__device__ __forceinline__ bool find_seq_tile(const int32_t *cu, int32_t N, int32_t T,
                                              uint32_t rows_per_token, uint32_t tile_rows,
                                              uint32_t index, TileCursor &at, SeqTile &out) {
    constexpr int PER = TileCursor::PER;
    const int lane = threadIdx.x & 31;
    if (at.s0 >= 0 && index < at.base) at.s0 = -1;
    bool fresh = at.s0 < 0;
    if (fresh) {
        at.s0 = 0;
        at.base = 0;
    }
    while (at.s0 < N) {
        if (fresh) {
            at.mine = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int32_t s = at.s0 + lane * PER + i;
                at.begin[i] = at.end[i] = 0;
                if (s < N) {
                    at.begin[i] = cu ? min(max(cu[s], 0), T) : 0;
                    at.end[i] = cu ? min(max(cu[s + 1], at.begin[i]), T) : T;
                }
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                at.n[i] = ((uint32_t)(at.end[i] - at.begin[i]) * rows_per_token + tile_rows - 1) /
                          tile_rows;
                at.mine += at.n[i];
            }
            at.incl = at.mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, at.incl, o);
                if (lane >= o) at.incl += x;
            }
        }
        const uint32_t here = __ballot_sync(0xffffffffu, index < at.base + at.incl);
        if (here) {
            const int src = __ffs(here) - 1;
            // the lane's sequence (of lane src: the others' is not used)
            uint32_t lo = at.base + at.incl - at.mine, before = lo, sn = at.n[0];
            int32_t sb = at.begin[0], se = at.end[0];
#pragma unroll
            for (int j = 1; j < PER; ++j) {
                lo += at.n[j - 1];
                if (index >= lo) {
                    before = lo;
                    sb = at.begin[j];
                    se = at.end[j];
                    sn = at.n[j];
                }
            }
            out.begin = __shfl_sync(0xffffffffu, sb, src);
            out.end = __shfl_sync(0xffffffffu, se, src);
            out.tile = (int32_t)__shfl_sync(0xffffffffu, sn - 1 - (index - before), src);
            return true;
        }
        at.base += __shfl_sync(0xffffffffu, at.incl, 31);
        at.s0 += 32 * PER;
        fresh = true;
    }
    return false;
}

}  // namespace kda
