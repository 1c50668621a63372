// Splitting a batch of single-token queries over the paged cache: the shares of
// the blocks, the copies of their cache rows, and the parts that are joined
// afterwards.  Shared by the kernels that attend (k_paged_decode.cu on the
// tensor cores, k_paged_decode_simt.cu on the CUDA cores).
//
// Work is dealt in steps of STEP visible tokens of one unit (sequence, head
// group): the steps of all units, and kUnitCost more for each, are laid end to
// end and cut into equal ranges, one per block (persistent, a multiple of the
// SMs), so ragged batches stay balanced whatever their lengths, which only the
// device knows.  A unit that lies in one block's range is written at once; the
// parts of others go to the workspace as (m, l, O) and a small kernel joins
// them in order.  In batch invariant mode a unit is cut at multiples of its own
// piece length instead and the blocks take whole pieces.
//
// In a block each of the four warps takes every fourth tile with its own ring
// of cp.async stages (no block barrier in the loop); the ring runs on across
// units.
#pragma once
#include "kernels.h"

namespace csa {

constexpr int kNW = 4;                 // warps of a block
constexpr int kMaxCtas = 3;            // blocks an SM, at most
constexpr int kMinSteps = 2;           // a block's share is not cut finer than this
// What a unit costs beside its steps, in steps: its query, its join, its output.
// 12 / 39 / 30 sequences, most of them short, bf16 at d = 128 / 256 / 64 (us):
//   cost 0: 30 / 43 / 58,  2: 18 / 26 / 28,  3: 17 / 27 / 25,  6: 17 / 32 / 23
// (one long row of 32 heads over 8, 1,001 tokens: 10.9 / 11.5 / 11.3 / 11.3).
// Measured with the tensor-core kernel's steps of 64 tokens; the CUDA-core kernel's
// steps of 32 use it too.
constexpr int kUnitCost = 3;
constexpr uint32_t kNoRow = 0xFFFFFFFFu;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, uint32_t n) {
    if constexpr (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(n), "n"(N) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// Shared memory for the rings, from a multiple of 128 bytes on: `extern
// __shared__` alone does not give one behind static arrays, whatever its
// declared alignment, and 16-byte copies of one 128-byte line into two shared
// lines cross from L2 twice (131,072 keys: 337 us instead of 269).
constexpr int kAlignSmem = 1024;
__device__ __forceinline__ uint8_t* aligned_smem(uint8_t* p) {
    return p + ((kAlignSmem - (smem_addr(p) & (kAlignSmem - 1))) & (kAlignSmem - 1));
}

// Place of 16-byte chunk c of row r in a tile of TOK rows of ROW bytes.  Rows are
// cut into blocks of 128 bytes (64 where those do not divide them), each block's
// rows one after another and swizzled, so that ldmatrix, and eight lanes on one
// chunk of eight rows, hit all banks.  (Swizzled tensor copies, which need no place
// computed, took longer: 276 us instead of 269 for 131,072 keys, and 274 instead
// of 190 from FP8 pages, whose tiles are half as large.)
template <int TOK, int ROW>
__device__ __forceinline__ uint32_t place(uint32_t r, uint32_t c) {
    constexpr uint32_t B = ROW % 128 == 0 ? 128 : 64, per = B / 16;
    const uint32_t x = per == 8 ? (r & 7u) : ((r >> 1) & 3u);
    return c / per * (TOK * B) + r * B + ((c % per) ^ x) * 16u;
}

// Visible tokens [lo, lo + n) of a sequence and its steps and pieces.
struct Span {
    int64_t lo;
    int n, steps;
};

// Of a token at t (any 64-bit value: t + 1 and t - W + 1 are formed where they
// cannot overflow) with places for `cap` tokens.
template <int STEP>
__host__ __device__ __forceinline__ Span span_at(int64_t t, int W, int64_t cap) {
    Span v;
    v.lo = W > 0 && t >= W ? t - W + 1 : 0;
    const int64_t hi = t < cap ? t + 1 : cap;
    v.n = hi > v.lo ? int(hi - v.lo) : 0;
    v.steps = v.n > 0 ? (v.n - 1) / STEP + 1 : 1;
    return v;
}
template <int STEP>
__device__ __forceinline__ Span span_of(const PagedDecodeArgs& a, int64_t s) {
    return span_at<STEP>(a.q_pos[s], a.W, a.max_pages * a.page_size);
}

// Batch invariant mode: steps of a piece, from the row's own length (at least
// 512 tokens, at most 64 pieces).
template <int STEP>
__host__ __device__ __forceinline__ int piece_steps(int steps) {
    const int p = (steps + 63) / 64;
    return p < 512 / STEP ? 512 / STEP : p;
}

// One block's share: units [.., x1) from position x (steps, or pieces).
struct Cursor {
    int64_t x, x1;
    int s, u;          // sequence, unit within it
    int at;            // position within the unit (steps or pieces)
    Span v;
};

struct Plan {
    int64_t x0, x1;    // this block's range
    int s, u, at;      // where x0 lies
    int n_ctas;        // blocks that have a share
    int64_t total;
};

template <int STEP>
__device__ __forceinline__ int weight(const PagedDecodeArgs& a, const Span& v) {
    if (!a.invariant) return v.steps + kUnitCost;
    const int p = piece_steps<STEP>(v.steps);
    return (v.steps + p - 1) / p;
}

// Every block derives the same plan: threads sum the weights of consecutive
// sequences, a scan gives their prefix, and the thread whose sequences hold
// x0 walks to it.
template <int STEP>
__device__ __forceinline__ void make_plan(const PagedDecodeArgs& a, int units, Plan* out) {
    __shared__ int64_t warp_sum_[kNW];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t seg = (a.batch + 32 * kNW - 1) / (32 * kNW);
    const int64_t s0 = min(tid * seg, a.batch), s1 = min(s0 + seg, a.batch);
    int64_t mine = 0;
    for (int64_t s = s0; s < s1; ++s) mine += int64_t(weight<STEP>(a, span_of<STEP>(a, s))) * units;
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    if (lane == 31) warp_sum_[warp] = upto;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kNW; ++w) {
        if (w < warp) upto += warp_sum_[w];
        total += warp_sum_[w];
    }
    const int64_t least = a.invariant ? 1 : kMinSteps;
    const int64_t n = min(int64_t(gridDim.x), (total + least - 1) / least);
    const int64_t c = blockIdx.x;
    const int64_t x0 = c < n ? c * total / n : total, x1 = c < n ? (c + 1) * total / n : total;
    if (tid == 0) { out->x0 = x0; out->x1 = x1; out->n_ctas = int(n); out->total = total; }
    int64_t x = upto - mine;  // prefix of this thread's first sequence
    if (x0 < x1 && x0 >= x && x0 < upto) {
        for (int64_t s = s0; s < s1; ++s) {
            const int w = weight<STEP>(a, span_of<STEP>(a, s));
            const int64_t e = x + int64_t(w) * units;
            if (x0 < e) {
                out->s = int(s);
                out->u = int((x0 - x) / w);
                out->at = int((x0 - x) % w);
                break;
            }
            x = e;
        }
    }
    __syncthreads();
}

// A record of the join: `n` parts, the first in slot `first`, the others in
// slots next, next + by, ...; (s, u): the row they belong to.
struct JoinRec {
    int n, first, next, by, s, u, pad0, pad1;
};

// What remains of the unit at a cursor: steps [b, e), and how far x moves.
template <int STEP>
__device__ __forceinline__ void piece_of(const PagedDecodeArgs& a, const Cursor& q, int& b, int& e, int& dx) {
    if (a.invariant) {
        const int p = piece_steps<STEP>(q.v.steps);
        b = q.at * p;
        e = min(b + p, q.v.steps);
        dx = 1;
    } else {
        // (positions from steps on are the unit's cost: nothing to do, b = e)
        dx = int(min(int64_t(q.v.steps + kUnitCost - q.at), q.x1 - q.x));
        b = min(q.at, q.v.steps);
        e = min(q.at + dx, q.v.steps);
    }
}
template <int STEP>
__device__ __forceinline__ void advance(const PagedDecodeArgs& a, int units, Cursor& q, int dx) {
    q.x += dx;
    q.at += dx;
    if (q.at >= weight<STEP>(a, q.v)) {
        q.at = 0;
        if (++q.u == units) {
            q.u = 0;
            ++q.s;
            if (q.x < q.x1) q.v = span_of<STEP>(a, q.s);
        }
    }
}

// The copying side of a warp: the tiles of its block's share in order.  C: kTok
// (tokens of a tile, 32 kNW / kTok lanes a token), kRow, kChunks, kGroups,
// kScaleBytes, kTile, kStep.  A stage is K rows, V rows, K scales, V scales.
template <class C, bool FP8>
struct Copier {
    const PagedDecodeArgs& a;
    int units, hb;
    Cursor pre;
    int pb, pe, pdx;
    uint32_t ring;
    // Of token lane % kTok of the next tile to copy: its page's entry of the block
    // table (loaded a tile ahead and first looked at when the tile is copied: its
    // latency is not waited for), place in the page, and key head; off < 0: no token.
    int32_t id;
    int off, hk;
    uint32_t* vmask;

    __device__ __forceinline__ Copier(const PagedDecodeArgs& a_, int units_, int hb_, const Cursor& c, uint32_t ring_,
                                      uint32_t* vmask_)
        : a(a_), units(units_), hb(hb_), pre(c), ring(ring_), vmask(vmask_) {
        piece_of<C::kStep>(a, pre, pb, pe, pdx);
        skip_empty();
        lookup();
    }
    __device__ __forceinline__ void skip_empty() {
        while (pb >= pe && pre.x < pre.x1) {
            advance<C::kStep>(a, units, pre, pdx);
            if (pre.x < pre.x1) piece_of<C::kStep>(a, pre, pb, pe, pdx);
        }
    }
    __device__ __forceinline__ void lookup() {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        off = -1;
        if (pre.x >= pre.x1) return;
        const int tok = pb * C::kStep + warp * C::kTok + (lane & (C::kTok - 1));
        if (tok < pre.v.n) {
            const uint32_t i = uint32_t(pre.v.lo) + uint32_t(tok);
            const uint32_t pg = a.page_size == 1 ? i : __umulhi(i, a.page_mul) >> a.page_shift;
            off = int(i - pg * uint32_t(a.page_size));
            hk = pre.u / hb;
            id = a.block_table[int64_t(pre.s) * a.max_pages + pg];
        }
    }
    __device__ __forceinline__ uint32_t resolve() {  // the token's cache row
        if (off < 0) return kNoRow;
        if (id >= 0 && id < a.n_pages)
            return (uint32_t(id) * uint32_t(a.HK) + uint32_t(hk)) * uint32_t(a.page_size) + uint32_t(off);
        flag_status(CSA_DEV_BAD_INDEX);
        return kNoRow;
    }
    __device__ __forceinline__ void issue(int stage) {  // copy the tile at `pre`, then look up the one after it
        const int lane = threadIdx.x & 31;
        if (pre.x < pre.x1) {
            const uint32_t k0 = ring + uint32_t(stage) * C::kTile, v0 = k0 + C::kTok * C::kRow;
            const uint32_t row = resolve();
            const unsigned ok = __ballot_sync(0xffffffffu, row != kNoRow) & ((1u << C::kTok) - 1u);
            if (lane == 0) vmask[stage] = ok;
            // mostly the tile's rows follow one another in a page: then their bytes do, too
            const uint32_t row0 = __shfl_sync(0xffffffffu, row, 0);
            if (__all_sync(0xffffffffu, row == row0 + uint32_t(lane & (C::kTok - 1)) && row != kNoRow)) {
                const uint64_t off0 = uint64_t(row0) * C::kRow + 16u * uint32_t(lane);
                const uint8_t *ks = (const uint8_t*)a.k_cache + off0, *vs = (const uint8_t*)a.v_cache + off0;
#pragma unroll
                for (int it = 0; it < C::kTok * C::kChunks / 32; ++it) {
                    const uint32_t i = uint32_t(it) * 32u + uint32_t(lane);
                    const uint32_t at = place<C::kTok, C::kRow>(i / C::kChunks, i % C::kChunks);
                    cp_async<16>(k0 + at, ks + 512 * it, 16u);
                    cp_async<16>(v0 + at, vs + 512 * it, 16u);
                }
            } else
#pragma unroll
            for (int it = 0; it < C::kTok * C::kChunks / 32; ++it) {
                const uint32_t i = uint32_t(it) * 32u + uint32_t(lane);
                const uint32_t r = i / C::kChunks, ch = i % C::kChunks;
                const uint32_t rr = __shfl_sync(0xffffffffu, row, int(r));
                const uint32_t n = rr == kNoRow ? 0u : 16u;
                const uint64_t off = rr == kNoRow ? 0ull : uint64_t(rr) * C::kRow + 16u * ch;
                const uint32_t at = place<C::kTok, C::kRow>(r, ch);
                cp_async<16>(k0 + at, (const uint8_t*)a.k_cache + off, n);
                cp_async<16>(v0 + at, (const uint8_t*)a.v_cache + off, n);
            }
            if constexpr (FP8) {  // lanes below 16: key scales of their token, the others: value scales
                const int t = lane & 15;
                if (t < C::kTok) {
                    const uint32_t s0 = v0 + C::kTok * C::kRow + (lane < 16 ? 0u : uint32_t(C::kScaleBytes));
                    const float* src = (lane < 16 ? a.k_scales : a.v_scales) + (row == kNoRow ? 0ull : uint64_t(row) * C::kGroups);
                    const uint32_t dst = s0 + uint32_t(t) * C::kGroups * 4;
                    const bool has = row != kNoRow;
                    if constexpr (C::kGroups == 3) {
#pragma unroll
                        for (int i = 0; i < 3; ++i) cp_async<4>(dst + 4 * i, src + i, has ? 4u : 0u);
                    } else {
                        cp_async<C::kGroups * 4>(dst, src, has ? C::kGroups * 4u : 0u);
                    }
                }
            }
            ++pb;
            skip_empty();
            lookup();
        }
        cp_commit();
    }
};

// Where the part [b, e) of the unit at `cur` goes: the slot's number, and the
// record of the join, written by the block (or piece) that holds the unit's
// beginning.  Called by all threads; slot is meant for a part only.
__device__ __forceinline__ int64_t part_slot(const PagedDecodeArgs& a, const Plan& plan, const Cursor& cur, int units,
                                             int pieces, bool begins, bool whole, JoinRec* recs) {
    int64_t slot = 0;
    JoinRec r;
    r.s = cur.s; r.u = cur.u; r.pad0 = r.pad1 = 0;
    if (a.invariant) {
        slot = cur.x;
        if (begins && recs && threadIdx.x == 0) {
            r.n = whole ? 0 : pieces; r.first = int(slot); r.next = int(slot) + 1; r.by = 1;
            recs[int64_t(cur.s) * units + cur.u] = r;
        }
    } else if (!whole) {
        slot = 2 * int64_t(blockIdx.x) + (cur.x == plan.x0 ? 0 : 1);
        if (begins && threadIdx.x == 0) {
            // the last block with a part of it: that of the unit's last step
            const int64_t xe = cur.x + cur.v.steps - 1;
            const int64_t last = ((xe + 1) * plan.n_ctas + plan.total - 1) / plan.total - 1;
            r.n = int(last - blockIdx.x) + 1; r.first = int(slot); r.next = 2 * (blockIdx.x + 1); r.by = 2;
            recs[blockIdx.x] = r;
        }
    }
    return slot;
}

// Workspace of a call: the records, then the parts' slots of heads * (D + 2)
// floats ((m, l) per head, O).  heads: of a unit; units: of a sequence.
struct DecodeLayout {
    int64_t units, recs, slots;
    size_t rec_bytes, bytes;
};
// Sets page_mul and page_shift: i / page_size for 0 <= i < 2^31 is the high word
// of i * page_mul, shifted, with page_mul = 2^(31 + s) / page_size rounded up,
// s = ceil(log2 page_size): off by less than i / 2^31 / page_size from the quotient.
void set_page_division(PagedDecodeArgs* a);
// Whether no unit can have more than 256 tokens (half a piece): the blocks then
// take whole units, as in batch invariant mode, and there is nothing to join.
// Device time split and joined / whole: 8 sequences in a window of 128 in fp32
// 9.7 / 6.4 us, one of 256 tokens in bf16 8.7 / 7.5 us, in fp32 8.5 / 8.8 us, of
// 512 9.1 / 9.9 us and 8.7 / 13.0 us.
bool one_piece(const PagedDecodeArgs& a);
DecodeLayout decode_layout(int H, int HK, int D, int64_t batch, int64_t n_ctx, bool invariant, int heads, int step);
cudaError_t launch_paged_join(const PagedDecodeArgs& a, int64_t recs_n, int hb, int heads, const JoinRec* recs,
                              const float* slots, cudaStream_t s);

}  // namespace csa
