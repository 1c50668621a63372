// Attention of one new token per sequence over the paged cache, split over the
// cache's length and joined (bf16 queries over bf16 or FP8 entries).
//
//   out = sum_i e^(l_i - M) v_i / (sum_i e^(l_i - M) + e^(sink - M)),  l_i = scale q.k_i
//
// Bound by HBM: every visible key and value row is read once, for all query
// heads that share it (G = H / HK, in groups of 8 NT heads; further groups
// read the rows again, from L2).  A byte of bf16 entries takes G multiply-adds,
// more than the CUDA cores can do beside the copy for G >= 4; mma.sync with
// the tokens as M = 16 and the heads as N = 8 wastes nothing at G = 8 and
// keeps S, P and O in registers, with no trip through TMEM for tiles this
// small:
//   S^T[token][head] = K . Q^T       A = K rows (ldmatrix), B = Q (registers)
//   O^T[dim][head]  += V^T . P^T     A = V^T (ldmatrix.trans), B = P (movmatrix of S^T's layout)
//
// Work is dealt in steps of 64 visible tokens of one (sequence, head group):
// the steps of all units are laid end to end and cut into equal ranges, one
// per CTA (persistent, a multiple of the SMs), so ragged batches stay
// balanced whatever their lengths, which only the device knows.  A unit that
// lies in one CTA's range is written at once; the parts of others go to the
// workspace as (m, l, O) and a small kernel joins them in order.  In batch
// invariant mode a unit is cut at multiples of its own piece length instead
// and the CTAs take whole pieces.
//
// In a CTA each of the four warps takes every fourth 16-token tile with its
// own ring of cp.async stages (no CTA barrier in the loop); the ring runs on
// across units.  The running maximum of a head is raised only when a tile
// exceeds it by more than 8 in log2 units (one vote a tile otherwise), sums
// stay per lane until the unit ends.
//
// FP8 entries (E4M3 codes, fp32 scale per 64 channels) are converted to f16
// exactly, one instruction per pair, and the MMAs run in f16: the query is
// scaled by a power of two per head (exact within 2^26 of the head's largest
// element), the key scales multiply S per 64 channels, and P takes the value
// scales.  So that p * scale fits f16 whatever the scales, it is kept
// relative to a power of two per (head, 64 channels) that follows its running
// maximum, and O is in those units.
#include "kernels.h"

namespace csa {

namespace {

constexpr int kNW = 4;                 // warps of a CTA
constexpr int kTok = 16;               // tokens of a warp's tile
constexpr int kStep = kNW * kTok;      // tokens of a step
constexpr int kMinSteps = 2;           // a CTA's share is not cut finer than this
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescale = 8.0f;       // log2 units
constexpr uint32_t kNoRow = 0xFFFFFFFFu;

template <int D, bool FP8, int NT>
struct Dec {
    static constexpr int kRow = FP8 ? D : 2 * D;         // bytes of a cache row
    static constexpr int kChunks = kRow / 16;
    static constexpr int kGroups = D / 64;
    static constexpr int kScaleBytes = FP8 ? kTok * kGroups * 4 : 0;
    static constexpr int kTile = 2 * (kTok * kRow + kScaleBytes);  // K and V of 16 tokens
    // Stages: about 100 KB a CTA, so that two fit an SM; one CTA of up to 192 KB for the wide heads
    static constexpr int kBudget = (D <= 128 ? 96 : 192) * 1024;
    static constexpr int kStages = kBudget / (kNW * kTile) > 8 ? 8 : kBudget / (kNW * kTile);
    static constexpr int kHeads = 8 * NT;
    static constexpr int kJoinDims = D > 64 ? D / 2 : D; // the warps' results are joined in halves of the dims
    static constexpr int kJoin = kJoinDims + 4;          // padded row of the join buffer
    static constexpr int kRing = kNW * kStages * kTile;
    static constexpr int kSmem = kRing + kNW * 8 * kJoin * 4;
    static constexpr int kCtas = 2 * (kSmem + 2048) <= 228 * 1024 ? 2 : 1;  // per SM
    static constexpr int kSlot = kHeads * (D + 2);       // floats of a partial: (m, l) per head, O
};

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
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// four E4M3 codes -> two pairs of f16 (bytes 0, 1 and bytes 2, 3), exact
__device__ __forceinline__ void f16_of_e4m3(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
        : "=r"(lo), "=r"(hi) : "r"(w));
}
// Place of 16-byte chunk c of row r: ldmatrix reads eight rows' chunks without
// bank conflicts (rows of 128 n bytes: by the row; of 64 or 192: by pairs).
template <int CHUNKS>
__device__ __forceinline__ uint32_t place(uint32_t r, uint32_t c) {
    const uint32_t x = (CHUNKS & 7) == 0 ? (r & 7u) : ((r >> 1) & 3u);
    return (r * CHUNKS + (c ^ x)) * 16u;
}

// Visible tokens [lo, lo + n) of a sequence and its steps and pieces.
struct Span {
    int64_t lo;
    int n, steps;
};

__device__ __forceinline__ Span span_of(const PagedDecodeArgs& a, int64_t s) {
    const int64_t t = a.q_pos[s], cap = a.max_pages * a.page_size;
    Span v;
    v.lo = a.W > 0 ? max(t - a.W + 1, int64_t(0)) : 0;
    const int64_t hi = min(t + 1, cap);
    v.n = int(max(hi - v.lo, int64_t(0)));
    v.steps = max((v.n + kStep - 1) / kStep, 1);
    return v;
}

// Batch invariant mode: steps of a piece, from the row's own length (at least
// 512 tokens, at most 64 pieces).
__host__ __device__ __forceinline__ int piece_steps(int steps) {
    const int p = (steps + 63) / 64;
    return p < 8 ? 8 : p;
}

}  // namespace

// One CTA's share: units [.., x1) from position x (steps, or pieces).
struct Cursor {
    int64_t x, x1;
    int s, u;          // sequence, unit within it
    int at;            // position within the unit (steps or pieces)
    Span v;
};

struct Plan {
    int64_t x0, x1;    // this CTA's range
    int s, u, at;      // where x0 lies
    int n_ctas;        // CTAs that have a share
    int64_t total;
};

__device__ __forceinline__ int weight(const PagedDecodeArgs& a, const Span& v) {
    if (!a.invariant) return v.steps;
    const int p = piece_steps(v.steps);
    return (v.steps + p - 1) / p;
}

// Every CTA derives the same plan: threads sum the weights of consecutive
// sequences, a scan gives their prefix, and the thread whose sequences hold
// x0 walks to it.
__device__ __forceinline__ void make_plan(const PagedDecodeArgs& a, int units, Plan* out) {
    __shared__ int64_t warp_sum_[kNW];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t seg = (a.batch + 32 * kNW - 1) / (32 * kNW);
    const int64_t s0 = min(tid * seg, a.batch), s1 = min(s0 + seg, a.batch);
    int64_t mine = 0;
    for (int64_t s = s0; s < s1; ++s) mine += int64_t(weight(a, span_of(a, s))) * units;
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
            const int w = weight(a, span_of(a, s));
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

template <int D, bool FP8, int NT>
__global__ void __launch_bounds__(32 * kNW, Dec<D, FP8, NT>::kCtas)
    paged_decode_kernel(const PagedDecodeArgs a, int units, int hb, JoinRec* recs, float* slots) {
    using C = Dec<D, FP8, NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Plan plan;
    __shared__ uint32_t vmask[kNW][8];
    __shared__ float2 jml[kNW][8 * NT];
    float* const jo = reinterpret_cast<float*>(smem + C::kRing);  // [kNW][8][kJoin]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c4 = lane & 3;
    pdl_launch_dependents();
    make_plan(a, units, &plan);
    if (!a.invariant && threadIdx.x == 0) recs[blockIdx.x].n = 0;
    const int64_t x0 = plan.x0, x1 = plan.x1;
    if (x0 >= x1) return;
    const int G = a.H / a.HK;
    const float sl2 = a.scale * kLog2e;

    // What remains of the unit at a cursor: steps [b, e), and how far x moves.
    auto piece = [&](const Cursor& q, int& b, int& e, int& dx) {
        if (a.invariant) {
            const int p = piece_steps(q.v.steps);
            b = q.at * p;
            e = min(b + p, q.v.steps);
            dx = 1;
        } else {
            b = q.at;
            e = int(min(int64_t(q.v.steps), q.at + (q.x1 - q.x)));
            dx = e - b;
        }
    };
    auto advance = [&](Cursor& q, int dx) {
        q.x += dx;
        q.at += dx;
        if (q.at >= weight(a, q.v)) {
            q.at = 0;
            if (++q.u == units) {
                q.u = 0;
                ++q.s;
                if (q.x < q.x1) q.v = span_of(a, q.s);
            }
        }
    };

    Cursor cur;
    cur.x = x0; cur.x1 = x1; cur.s = plan.s; cur.u = plan.u; cur.at = plan.at;
    cur.v = span_of(a, cur.s);

    // ------------------------------------------------------- the copying side
    Cursor pre = cur;
    int pb, pe, pdx;
    piece(pre, pb, pe, pdx);
    const uint32_t ring = smem_addr(smem) + uint32_t(warp) * C::kStages * C::kTile;
    uint32_t row_next = kNoRow;
    auto lookup = [&]() {  // cache row of token lane & 15 of the next tile to copy
        row_next = kNoRow;
        if (pre.x >= pre.x1) return;
        const int tok = pb * kStep + warp * kTok + (lane & 15);
        if (tok < pre.v.n) {
            const int64_t i = pre.v.lo + tok;
            const uint32_t pg = uint32_t(i) / uint32_t(a.page_size), off = uint32_t(i) % uint32_t(a.page_size);
            const int64_t id = a.block_table[int64_t(pre.s) * a.max_pages + pg];
            if (id >= 0 && id < a.n_pages)
                row_next = (uint32_t(id) * uint32_t(a.HK) + uint32_t(pre.u / hb)) * uint32_t(a.page_size) + off;
            else
                flag_status(CSA_DEV_BAD_INDEX);
        }
    };
    auto issue = [&](int stage) {  // copy the tile at `pre`, then look up the one after it
        if (pre.x < pre.x1) {
            const uint32_t k0 = ring + uint32_t(stage) * C::kTile, v0 = k0 + kTok * C::kRow;
            const uint32_t row = row_next;
            const unsigned ok = __ballot_sync(0xffffffffu, row != kNoRow) & 0xFFFFu;
            if (lane == 0) vmask[warp][stage] = ok;
#pragma unroll
            for (int it = 0; it < kTok * C::kChunks / 32; ++it) {
                const uint32_t i = uint32_t(it) * 32u + uint32_t(lane);
                const uint32_t r = i / C::kChunks, ch = i % C::kChunks;
                const uint32_t rr = __shfl_sync(0xffffffffu, row, int(r));
                const uint32_t n = rr == kNoRow ? 0u : 16u;
                const uint64_t off = rr == kNoRow ? 0ull : uint64_t(rr) * C::kRow + 16u * ch;
                const uint32_t at = place<C::kChunks>(r, ch);
                cp_async<16>(k0 + at, (const uint8_t*)a.k_cache + off, n);
                cp_async<16>(v0 + at, (const uint8_t*)a.v_cache + off, n);
            }
            if constexpr (FP8) {  // lanes 0-15: key scales of their token, 16-31: value scales
                const uint32_t s0 = v0 + kTok * C::kRow + (lane < 16 ? 0u : uint32_t(C::kScaleBytes));
                const float* src = (lane < 16 ? a.k_scales : a.v_scales) + (row == kNoRow ? 0ull : uint64_t(row) * C::kGroups);
                const uint32_t dst = s0 + uint32_t(lane & 15) * C::kGroups * 4;
                const bool has = row != kNoRow;
                if constexpr (C::kGroups == 3) {
#pragma unroll
                    for (int i = 0; i < 3; ++i) cp_async<4>(dst + 4 * i, src + i, has ? 4u : 0u);
                } else {
                    cp_async<C::kGroups * 4>(dst, src, has ? C::kGroups * 4u : 0u);
                }
            }
            if (++pb >= pe) {
                advance(pre, pdx);
                if (pre.x < pre.x1) piece(pre, pb, pe, pdx);
            }
            lookup();
        }
        cp_commit();
    };
    lookup();
#pragma unroll 1
    for (int i = 0; i < C::kStages - 1; ++i) issue(i);

    // ------------------------------------------------------ the computing side
    int stage = 0;
#pragma unroll 1
    while (cur.x < cur.x1) {
        int b, e, dx;
        piece(cur, b, e, dx);
        if (threadIdx.x == 0 && a.q_pos[cur.s] >= a.max_pages * a.page_size) flag_status(CSA_DEV_BAD_INDEX);
        const int hk = cur.u / hb, head0 = (cur.u % hb) * C::kHeads;  // within the group of G
        const int n_heads = min(C::kHeads, G - head0);
        // queries: B fragments of every 16 dims
        uint32_t qf[NT][D / 16][2];
        float sc[NT][2];  // log2-scale of the lane's two columns (heads)
        const uint16_t* qrow = (const uint16_t*)a.q + int64_t(cur.s) * a.q_ld + (int64_t(hk) * G + head0) * D;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const bool live = 8 * nt + g < n_heads;
            const uint16_t* qp = qrow + int64_t(8 * nt + g) * D;
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                qf[nt][k][0] = live ? *reinterpret_cast<const uint32_t*>(qp + 16 * k + (FP8 ? 4 : 2) * c4) : 0u;
                qf[nt][k][1] = live ? *reinterpret_cast<const uint32_t*>(qp + 16 * k + (FP8 ? 4 * c4 + 2 : 2 * c4 + 8)) : 0u;
                if constexpr (FP8) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        top = fmaxf(top, fabsf(__uint_as_float(qf[nt][k][i] << 16)));
                        top = fmaxf(top, fabsf(__uint_as_float(qf[nt][k][i] & 0xFFFF0000u)));
                    }
                }
            }
            if constexpr (FP8) {
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // 2^x with the head's largest element at 2^12..2^13 (x kept within fp32's normal range)
                const int x = min(max(12 - (int(__float_as_uint(top) >> 23) - 127), -120), 120);
                const float up = pow2f(x);
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        qf[nt][k][i] = pack_f16(__uint_as_float(qf[nt][k][i] << 16) * up,
                                                __uint_as_float(qf[nt][k][i] & 0xFFFF0000u) * up);
                const float down = sl2 * pow2f(-x);
#pragma unroll
                for (int i = 0; i < 2; ++i) sc[nt][i] = __shfl_sync(0xffffffffu, down, 4 * (2 * c4 + i));
            } else {
                sc[nt][0] = sc[nt][1] = sl2;
            }
        }
        float o[NT][D / 16][4];
        float m[NT][2], l[NT][2];
        float f[NT][FP8 ? C::kGroups : 1][2];  // FP8: the power of two that P is multiplied by
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[nt][k][i] = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[nt][i] = -INFINITY;
                l[nt][i] = 0.f;
                if constexpr (FP8)
#pragma unroll
                    for (int gr = 0; gr < C::kGroups; ++gr) f[nt][gr][i] = pow2f(100);
            }
        }

#pragma unroll 1
        for (int st = b; st < e; ++st) {
            cp_wait<C::kStages - 2>();
            __syncwarp();
            {
                const int nx = stage == 0 ? C::kStages - 1 : stage - 1;  // the stage consumed last
                issue(nx);
            }
            const uint32_t k0 = ring + uint32_t(stage) * C::kTile, v0 = k0 + kTok * C::kRow;
            const uint32_t ok = vmask[warp][stage];
            const float* ksc = reinterpret_cast<const float*>(smem + (v0 + kTok * C::kRow - smem_addr(smem)));
            const float* vsc = ksc + C::kScaleBytes / 4;
            // ---- S^T
            float s[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
            if constexpr (!FP8) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t x[4];
                    ldsm4(k0 + place<C::kChunks>(lane & 15, 2 * k + (lane >> 4)), x);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma<false>(s[nt], x, qf[nt][k][0], qf[nt][k][1]);
                }
            } else {
#pragma unroll
                for (int gr = 0; gr < C::kGroups; ++gr) {
                    float t[NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) t[nt][i] = 0.f;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // 32 dims
                        uint32_t w[4];
                        ldsm4(k0 + place<C::kChunks>(lane & 15, 4 * gr + 2 * h + (lane >> 4)), w);
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            uint32_t x[4];
                            f16_of_e4m3(w[2 * z], x[0], x[2]);
                            f16_of_e4m3(w[2 * z + 1], x[1], x[3]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma<true>(t[nt], x, qf[nt][4 * gr + 2 * h + z][0], qf[nt][4 * gr + 2 * h + z][1]);
                        }
                    }
                    const float ka = ksc[g * C::kGroups + gr], kb = ksc[(g + 8) * C::kGroups + gr];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        s[nt][0] += t[nt][0] * ka; s[nt][1] += t[nt][1] * ka;
                        s[nt][2] += t[nt][2] * kb; s[nt][3] += t[nt][3] * kb;
                    }
                }
            }
            // ---- softmax: rows g and g + 8 (tokens), columns 2 c4, 2 c4 + 1 (heads)
            const bool va = ok >> g & 1, vb = ok >> (g + 8) & 1;
            bool raise = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    s[nt][i] = va ? s[nt][i] * sc[nt][i] : -INFINITY;
                    s[nt][2 + i] = vb ? s[nt][2 + i] * sc[nt][i] : -INFINITY;
                    raise |= fmaxf(s[nt][i], s[nt][2 + i]) > m[nt][i] + kRescale;
                }
            }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float al[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float mx = fmaxf(s[nt][i], s[nt][2 + i]);
#pragma unroll
                        for (int z = 4; z < 32; z <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, z));
                        al[i] = 1.f;
                        if (mx > m[nt][i] + kRescale) {
                            al[i] = m[nt][i] == -INFINITY ? 0.f : ex2(m[nt][i] - mx);
                            m[nt][i] = mx;
                        }
                        l[nt][i] *= al[i];
                    }
#pragma unroll
                    for (int gr = 0; gr < (FP8 ? C::kGroups : 1); ++gr) {
                        float up[2] = {al[0], al[1]};
                        if constexpr (FP8) {
                            // O keeps its units: the factor of P grows by what P shrank, as far as fp32 allows
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                if (al[i] > 0.f) {
                                    const float y = fminf(1.f / al[i], pow2f(100) / f[nt][gr][i]);
                                    f[nt][gr][i] *= y;
                                    up[i] *= y;
                                } else {
                                    f[nt][gr][i] = pow2f(100);  // O is 0 and starts anew
                                }
                            }
                        }
                        constexpr int per = FP8 ? 4 : D / 16;
#pragma unroll
                        for (int k = 0; k < per; ++k)
#pragma unroll
                            for (int i = 0; i < 4; ++i) o[nt][gr * per + k][i] *= up[i & 1];
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float mm = m[nt][i] == -INFINITY ? 0.f : m[nt][i];
                    s[nt][i] = ex2(s[nt][i] - mm);
                    s[nt][2 + i] = ex2(s[nt][2 + i] - mm);
                    l[nt][i] += s[nt][i] + s[nt][2 + i];
                }
            // ---- O^T
            if constexpr (!FP8) {
                uint32_t p[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    p[nt][0] = transpose8x8(pack_bf16(s[nt][0], s[nt][1]));
                    p[nt][1] = transpose8x8(pack_bf16(s[nt][2], s[nt][3]));
                }
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t x[4];
                    ldsm4_t(v0 + place<C::kChunks>((lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)), x);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma<false>(o[nt][k], x, p[nt][0], p[nt][1]);
                }
            } else {
#pragma unroll
                for (int gr = 0; gr < C::kGroups; ++gr) {
                    const float fa = vsc[g * C::kGroups + gr], fb = vsc[(g + 8) * C::kGroups + gr];
                    float y[NT][4];
                    bool over = false;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            y[nt][i] = s[nt][i] == 0.f ? 0.f : s[nt][i] * (i < 2 ? fa : fb);
                            over |= y[nt][i] * f[nt][gr][i & 1] > 32768.f;
                        }
                    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                float top = fmaxf(y[nt][i], y[nt][2 + i]);
#pragma unroll
                                for (int z = 4; z < 32; z <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, z));
                                if (top * f[nt][gr][i] > 32768.f) {
                                    const int x = min(max(12 - (int(__float_as_uint(top) >> 23) - 127), -100), 100);
                                    const float ratio = pow2f(x) / f[nt][gr][i];
                                    f[nt][gr][i] = pow2f(x);
#pragma unroll
                                    for (int k = 0; k < 4; ++k) {
                                        o[nt][4 * gr + k][i] *= ratio;
                                        o[nt][4 * gr + k][2 + i] *= ratio;
                                    }
                                }
                            }
                    }
                    uint32_t p[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        p[nt][0] = transpose8x8(pack_f16(y[nt][0] * f[nt][gr][0], y[nt][1] * f[nt][gr][1]));
                        p[nt][1] = transpose8x8(pack_f16(y[nt][2] * f[nt][gr][0], y[nt][3] * f[nt][gr][1]));
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t w[4];
                        ldsm4_t(v0 + place<C::kChunks>(lane & 15, 4 * gr + 2 * h + (lane >> 4)), w);
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            // tokens 2 c4, 2 c4 + 1 of dims 2 g (low half) and 2 g + 1 (high half)
                            uint32_t x[4];
                            f16_of_e4m3(__byte_perm(w[2 * z], 0, 0x3120), x[0], x[1]);
                            f16_of_e4m3(__byte_perm(w[2 * z + 1], 0, 0x3120), x[2], x[3]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma<true>(o[nt][4 * gr + 2 * h + z], x, p[nt][0], p[nt][1]);
                        }
                    }
                }
            }
            __syncwarp();
            stage = stage + 1 == C::kStages ? 0 : stage + 1;
        }

        // ---- the unit (or this CTA's part of it) is done: join the warps
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int z = 4; z < 32; z <<= 1) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], z);
                if (g == 0) jml[warp][8 * nt + 2 * c4 + i] = make_float2(m[nt][i], l[nt][i]);
            }
        const bool whole = b == 0 && e == cur.v.steps;
        const bool first_unit = cur.x == x0;
        int64_t slot = 0;
        if (!whole) {
            if (a.invariant) {
                slot = cur.x;
            } else {
                slot = 2 * int64_t(blockIdx.x) + (first_unit ? 0 : 1);
                // the CTA that holds the unit's beginning says where its parts are
                if (b == 0 && threadIdx.x == 0) {
                    // the last CTA with a part of it: that of the unit's last step
                    const int64_t xe = cur.x + cur.v.steps - 1;
                    const int64_t last = ((xe + 1) * plan.n_ctas + plan.total - 1) / plan.total - 1;
                    JoinRec r;
                    r.n = int(last - blockIdx.x) + 1; r.first = int(slot); r.next = 2 * (blockIdx.x + 1); r.by = 2;
                    r.s = cur.s; r.u = cur.u; r.pad0 = r.pad1 = 0;
                    recs[blockIdx.x] = r;
                }
            }
        }
        if (a.invariant && b == 0 && threadIdx.x == 0) {
            JoinRec r;
            r.n = whole ? 0 : weight(a, cur.v); r.first = int(slot); r.next = int(slot) + 1; r.by = 1;
            r.s = cur.s; r.u = cur.u; r.pad0 = r.pad1 = 0;
            recs[int64_t(cur.s) * units + cur.u] = r;
        }
#pragma unroll
        for (int pass = 0; pass < NT * D / C::kJoinDims; ++pass) {
            const int nt = pass % NT, k0 = pass / NT * (C::kJoinDims / 16);
#pragma unroll
            for (int kk = 0; kk < C::kJoinDims / 16; ++kk)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = k0 + kk;
                    const int dim = 16 * kk + (FP8 ? 2 * g + (i >> 1) : g + 8 * (i >> 1));
                    float x = o[nt][k][i];
                    if constexpr (FP8) x = x == 0.f ? 0.f : x / f[nt][k / 4][i & 1];
                    jo[(warp * 8 + 2 * c4 + (i & 1)) * C::kJoin + dim] = x;
                }
            __syncthreads();
            for (int i = threadIdx.x; i < 8 * C::kJoinDims; i += 32 * kNW) {
                const int hh = i / C::kJoinDims, jd = i % C::kJoinDims, dim = 16 * k0 + jd, head = 8 * nt + hh;
                if (head >= n_heads) break;
                const int h = hk * G + head0 + head;
                float M = -INFINITY, L = 0.f, acc = 0.f;
#pragma unroll
                for (int w = 0; w < kNW; ++w) M = fmaxf(M, jml[w][head].x);
                const float sg = whole && a.sinks ? a.sinks[h] * kLog2e : -INFINITY;
                M = fmaxf(M, sg);
#pragma unroll
                for (int w = 0; w < kNW; ++w) {
                    const float2 v = jml[w][head];
                    const float wt = v.x == -INFINITY ? 0.f : ex2(v.x - M);
                    L += wt * v.y;  // (NaN logits leave m at -inf: they reach the result through l)
                    if (wt != 0.f) acc += wt * jo[(w * 8 + hh) * C::kJoin + jd];
                }
                if (whole) {
                    if (sg != -INFINITY) L += ex2(sg - M);
                    const float r = L == 0.f ? 0.f : acc / L;
                    ((__nv_bfloat16*)a.out)[(int64_t(cur.s) * a.H + h) * D + dim] = __float2bfloat16_rn(r);
                } else {
                    float* sp = slots + slot * C::kSlot;
                    if (dim == 0) { sp[2 * head] = M; sp[2 * head + 1] = L; }
                    sp[2 * C::kHeads + head * D + dim] = acc;
                }
            }
            __syncthreads();
        }
        advance(cur, dx);
    }
    cp_wait<0>();
}

// Join the parts of the rows that more than one CTA (or piece) worked on.
__global__ void __launch_bounds__(128)
    paged_decode_join_kernel(const PagedDecodeArgs a, int hb, int heads, const JoinRec* recs, const float* slots) {
    pdl_wait();
    const JoinRec r = recs[blockIdx.x];
    if (r.n == 0) return;
    const int D = a.D, G = a.H / a.HK, per = heads * (D + 2);
    const int hk = r.u / hb, head0 = (r.u % hb) * heads, n_heads = min(heads, G - head0);
    for (int i = threadIdx.x + 128 * blockIdx.y; i < n_heads * D; i += 128 * gridDim.y) {
        const int head = i / D, h = hk * G + head0 + head;
        const float sg = a.sinks ? a.sinks[h] * kLog2e : -INFINITY;
        float M = sg;
        for (int q = 0; q < r.n; ++q) {
            const float* sp = slots + int64_t(q == 0 ? r.first : r.next + (q - 1) * r.by) * per;
            M = fmaxf(M, sp[2 * head]);
        }
        float L = sg != -INFINITY ? ex2(sg - M) : 0.f, acc = 0.f;
#pragma unroll 4
        for (int q = 0; q < r.n; ++q) {
            const float* sp = slots + int64_t(q == 0 ? r.first : r.next + (q - 1) * r.by) * per;
            const float mq = sp[2 * head], lq = sp[2 * head + 1], x = sp[2 * heads + i];
            const float wt = mq == -INFINITY ? 0.f : ex2(mq - M);
            L += wt * lq;
            if (wt != 0.f) acc += wt * x;
        }
        ((__nv_bfloat16*)a.out)[(int64_t(r.s) * a.H + h) * D + i % D] = __float2bfloat16_rn(L == 0.f ? 0.f : acc / L);
    }
}

// Heads of a group: 8, or 16 where more share a key head and the registers hold them.
static int group_heads(int H, int HK, int D) { return H / HK > 8 && D <= 128 ? 16 : 8; }

bool paged_decode_tc_supported(int act, int cache) {
    return act == CSA_BF16 && (cache == CSA_BF16 || cache == CSA_FP8_S64);
}

struct DecodeLayout {
    int64_t units, recs;   // per sequence; records
    int64_t slots;
    size_t rec_bytes, bytes;
};

static DecodeLayout decode_layout(int H, int HK, int D, int64_t batch, int64_t n_ctx, bool invariant) {
    const int heads = group_heads(H, HK, D);
    DecodeLayout w;
    w.units = int64_t(HK) * ((H / HK + heads - 1) / heads);
    if (invariant) {
        const int64_t steps = ceil_div(n_ctx, kStep);
        w.recs = batch * w.units;
        w.slots = batch * w.units * std::min<int64_t>(64, ceil_div(steps, 8) + 1);
    } else {
        w.recs = 2 * kNumSMs;
        w.slots = 2 * w.recs;
    }
    w.rec_bytes = (size_t(w.recs) * sizeof(JoinRec) + 255) & ~size_t(255);
    w.bytes = w.rec_bytes + size_t(w.slots) * heads * (D + 2) * sizeof(float);
    return w;
}

size_t paged_decode_workspace(int H, int HK, int D, int64_t batch, int64_t n_ctx, bool invariant) {
    return decode_layout(H, HK, D, batch, n_ctx, invariant).bytes;
}

template <int D, bool FP8, int NT>
static cudaError_t launch_decode(const PagedDecodeArgs& a, void* ws, cudaStream_t s) {
    using C = Dec<D, FP8, NT>;
    static_assert(C::kStages >= 2 && C::kStages <= 8, "stages");
    const DecodeLayout w = decode_layout(a.H, a.HK, D, a.batch, a.max_pages * a.page_size, a.invariant);
    JoinRec* recs = (JoinRec*)ws;
    float* slots = (float*)((char*)ws + w.rec_bytes);
    const int hb = int(w.units / a.HK);
    cudaError_t e = ensure_smem(paged_decode_kernel<D, FP8, NT>, C::kSmem);
    if (e != cudaSuccess) return e;
    paged_decode_kernel<D, FP8, NT><<<C::kCtas * kNumSMs, 32 * kNW, C::kSmem, s>>>(a, int(w.units), hb, recs, slots);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const unsigned n = unsigned(a.invariant ? w.recs : C::kCtas * kNumSMs);
    return launch_ex(paged_decode_join_kernel, dim3(n, 2), dim3(128), 0, s, true, a, hb, int(C::kHeads),
                     (const JoinRec*)recs, (const float*)slots);
}

template <int D, bool FP8>
static cudaError_t launch_decode_d(const PagedDecodeArgs& a, void* ws, cudaStream_t s) {
    if constexpr (D <= 128)
        if (group_heads(a.H, a.HK, D) == 16) return launch_decode<D, FP8, 2>(a, ws, s);
    return launch_decode<D, FP8, 1>(a, ws, s);
}

template <bool FP8>
static cudaError_t launch_decode_fmt(const PagedDecodeArgs& a, void* ws, cudaStream_t s) {
    switch (a.D) {
        case 64: return launch_decode_d<64, FP8>(a, ws, s);
        case 128: return launch_decode_d<128, FP8>(a, ws, s);
        case 192: return launch_decode_d<192, FP8>(a, ws, s);
        default: return launch_decode_d<256, FP8>(a, ws, s);
    }
}

cudaError_t launch_paged_decode_tc(const PagedDecodeArgs& a, void* ws, cudaStream_t s) {
    return a.cache_fmt == CSA_FP8_S64 ? launch_decode_fmt<true>(a, ws, s) : launch_decode_fmt<false>(a, ws, s);
}

}  // namespace csa
