// The tiles of a packed batch of prompts, in the order in which the blocks of a
// prompt kernel take them.
#pragma once
#include "common.cuh"

namespace csa {

// Tile x of a packed batch: `tile` of sequence `s` (tiles of `per` tokens), s = -1
// behind the last one: sequences in order, the tiles of each last (longest)
// first.  Called by one warp.  (The whole batch's tiles longest first, found
// by bisection, took longer: 155 us instead of 147 on 8,139 tokens of ten
// sequences.)
__device__ __forceinline__ void find_tile(const int32_t* cu, int n_seq, int per, int x, int lane, int& s, int& tile) {
    int before = 0;
    s = -1;
    tile = 0;
    for (int base = 0; base < n_seq; base += 32) {
        const int i = base + lane;
        const int n = i < n_seq ? max(cu[i + 1] - cu[i], 0) : 0;
        int upto = (n + per - 1) / per;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        const unsigned in = __ballot_sync(0xffffffffu, x < before + upto);
        if (in) {
            const int src = __ffs(int(in)) - 1;
            s = base + src;
            tile = before + __shfl_sync(0xffffffffu, upto, src) - 1 - x;  // counted from the sequence's last tile
            return;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
}

}  // namespace csa
