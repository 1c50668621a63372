// The tiles of a packed batch of prompts, in the order in which the blocks of a
// prompt kernel take them.
#pragma once
#include "common.cuh"

namespace csa {

// First key that a query at key position t sees with a window of W keys (0: no
// window).  t may be negative (fewer keys than queries) and W anything up to
// INT32_MAX, so that t - W + 1 is formed only where it is not below 1.
__host__ __device__ __forceinline__ int first_seen(int t, int W) { return W > 0 && t >= W ? t - W + 1 : 0; }

// A tile of a packed batch and its sequence: packed rows q0 .. q0 + len_q - 1,
// keys k0 .. k0 + len_k - 1.
struct SeqTile {
    int s, tile;  // s = -1: behind the last tile
    int q0, len_q, k0, len_k;
};

// Tile x of a packed batch (tiles of `per` tokens): sequences in order, the
// tiles of each last (longest) first.  Called by one warp.  (The whole batch's
// tiles longest first, found by bisection, took longer: 155 us instead of 147
// on 8,139 tokens of ten sequences.)
__device__ __forceinline__ SeqTile find_tile(const int32_t* cu_q, const int32_t* cu_k, int n_seq, int per, int x, int lane) {
    int before = 0;
    for (int base = 0; base < n_seq; base += 32) {
        const int i = base + lane, j = min(i, n_seq - 1);
        const int q0 = cu_q[j], q1 = cu_q[j + 1], k0 = cu_k[j], k1 = cu_k[j + 1];
        const int mine = i < n_seq ? (max(q1 - q0, 0) + per - 1) / per : 0;
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        const unsigned in = __ballot_sync(0xffffffffu, x < before + upto);
        if (in) {
            const int src = __ffs(int(in)) - 1;
            SeqTile t;
            t.s = base + src;
            t.tile = before + __shfl_sync(0xffffffffu, upto, src) - 1 - x;  // counted from the sequence's last tile
            t.q0 = __shfl_sync(0xffffffffu, q0, src);
            t.len_q = __shfl_sync(0xffffffffu, q1, src) - t.q0;
            t.k0 = __shfl_sync(0xffffffffu, k0, src);
            t.len_k = __shfl_sync(0xffffffffu, k1, src) - t.k0;
            return t;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    return SeqTile{-1, 0, 0, 0, 0, 0};
}

}  // namespace csa
