// kda_attn_common.cuh -- what the prompt-attention engines share: the map from
// a block index to a tile of one sequence.
#pragma once

#include <cstdint>

#include "kda_internal.cuh"

namespace kda {

// A tile of a sequence's rows: tokens [begin, end) are the sequence's.
struct SeqTile {
    int32_t begin, end;  // the sequence's tokens in the packed axis
    int32_t tile;        // index of the tile within the sequence
};

// Where a search stands: `base` tiles lie before sequence s0.
struct TileCursor {
    int32_t s0 = 0;
    uint32_t base = 0;
};

// The `index`-th tile over all sequences, tokens(s) * rows_per_token rows of
// sequence s in tiles of tile_rows.  A sequence's tiles come last tile first:
// under the causal mask the last is the longest, and long tiles that start
// early leave no long tail.  Called by one whole warp; false when there is no
// such tile.  The cursor carries the search over to the next (a larger index
// goes on where the last was found).
__device__ __forceinline__ bool find_seq_tile(const int32_t *cu, int32_t N, int32_t T,
                                              int32_t rows_per_token, int32_t tile_rows,
                                              uint32_t index, TileCursor &at, SeqTile &out) {
    constexpr int PER = 4;  // neighbouring sequences per lane
    const int lane = threadIdx.x & 31;
    if (index < at.base) at = TileCursor();
    while (at.s0 < N) {
        int32_t b[PER], e[PER];
        uint32_t n[PER], mine = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int32_t s = at.s0 + lane * PER + i;
            b[i] = e[i] = 0;
            if (s < N) {
                b[i] = cu ? min(max(cu[s], 0), T) : 0;
                e[i] = cu ? min(max(cu[s + 1], b[i]), T) : T;
            }
            n[i] = (uint32_t)(((int64_t)(e[i] - b[i]) * rows_per_token + tile_rows - 1) / tile_rows);
            mine += n[i];
        }
        uint32_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        const uint32_t here = __ballot_sync(0xffffffffu, index < at.base + incl);
        if (here) {
            const int src = __ffs(here) - 1;
            // the lane's sequence (of lane src: the others' is not used)
            uint32_t lo = at.base + incl - mine, before = lo, sn = n[0];
            int32_t sb = b[0], se = e[0];
#pragma unroll
            for (int j = 1; j < PER; ++j) {
                lo += n[j - 1];
                if (index >= lo) {
                    before = lo;
                    sb = b[j];
                    se = e[j];
                    sn = n[j];
                }
            }
            out.begin = __shfl_sync(0xffffffffu, sb, src);
            out.end = __shfl_sync(0xffffffffu, se, src);
            out.tile = (int32_t)__shfl_sync(0xffffffffu, sn - 1 - (index - before), src);
            return true;
        }
        at.base += __shfl_sync(0xffffffffu, incl, 31);
        at.s0 += 32 * PER;
    }
    return false;
}

}  // namespace kda
