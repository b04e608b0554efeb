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

// The `index`-th tile over all sequences, sequence s having
// ceil(tokens(s) / tile_tokens * rows_per_token) tiles -- counted in rows:
// tokens(s) * rows_per_token rows in tiles of tile_rows.  A sequence's tiles
// come last tile first: under the causal mask the last is the longest, and
// long tiles that start early leave no long tail.  Called by one whole warp;
// false when there is no such tile.
__device__ __forceinline__ bool find_seq_tile(const int32_t *cu, int32_t N, int32_t T,
                                              int32_t rows_per_token, int32_t tile_rows,
                                              uint32_t index, SeqTile &out) {
    const int lane = threadIdx.x & 31;
    uint32_t base = 0;
    for (int32_t s0 = 0; s0 < N; s0 += 32) {
        const int32_t s = s0 + lane;
        int32_t b = 0, e = 0;
        if (s < N) {
            b = cu ? min(max(cu[s], 0), T) : 0;
            e = cu ? min(max(cu[s + 1], b), T) : T;
        }
        const uint32_t n = (uint32_t)(((int64_t)(e - b) * rows_per_token + tile_rows - 1) / tile_rows);
        uint32_t incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        const uint32_t here = __ballot_sync(0xffffffffu, index < base + incl);
        if (here) {
            const int src = __ffs(here) - 1;
            const uint32_t before = base + __shfl_sync(0xffffffffu, incl - n, src);
            out.begin = __shfl_sync(0xffffffffu, b, src);
            out.end = __shfl_sync(0xffffffffu, e, src);
            out.tile = (int32_t)(__shfl_sync(0xffffffffu, n, src) - 1 - (index - before));
            return true;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;
}

}  // namespace kda
