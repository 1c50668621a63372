// Causal attention over packed prompts on the 5th-generation tensor cores
// (bf16, head dims 64, 128, 192, 256).
//
//   S = Q K^T ; P = exp2(S scale log2e - m) ; O = sum P V ; out = O / sum P
//
// A q tile is 128 rows of one key / value head: floor(128 / G) tokens times
// the G query heads that share the head, so that a K / V tile serves all of
// them and short sequences fill the rows.  A CTA owns NQ q tiles of
// consecutive tokens (two at d = 128, else one) and walks the keys that
// any of its rows sees in tiles of 64, with the running maximum and sum of
// each row in the thread that owns the row; P never leaves the SM.
//
//   S[row][key]  = Q (smem) . K^T (smem)    M = 128, N = 64, K = d    -> TMEM
//   O[row][dim] += P (TMEM) . V (smem)      M = 128, N = d, K = 64    -> TMEM
//
// P (bf16) overwrites the S columns it came from.  A q tile has two S slots, so
// that S of the next key tile is there before the softmax is done with this
// one: PV of a slot, then the next QK into it.  O is rescaled in TMEM only
// when a row's maximum has grown by more than 8 (log2 units) over the one in
// use.
//
// Roles: NQ warpgroups of softmax (thread = row; they also write the output),
// an MMA warp per q tile (one lane issues; two warps, so that one feeds the
// tensor pipe under the other's waits: with one, 16,384 tokens took 12% more),
// warp TMA (one lane loads q, K and V by swizzled tensor copies; q rows of a
// tile are one box of G heads x tokens), and guard warps.  A tile that some
// row may not see completely is a guarded one: before its PV the guard warps
// clear V rows past the sequence (they belong to other sequences or are
// padding) and look for infinities and NaN in those that some row does not
// see: a probability of 0 would not keep them out of the sum.  They are
// cleared too and their rows noted, and the epilogue adds them to the rows
// that see them.
//
// At d = 128 a pair of q tiles and 64 keys is 1024 clocks of MMA, about 1280 of
// shared-memory reads for it (q is read again for every 64 keys) and, with 16
// exponentials a clock, 1024 clocks of those; the chain from S over P to the
// next S makes it about 1700.  What was tried and took longer: a quarter of the
// exponentials by a polynomial on the FMA pipes (1 to 5% longer but for short
// prompts, 2% shorter), two threads a row, key tiles of 128 with one S slot (the
// same on one long prompt, 11% longer on a packed batch of short ones), and a
// persistent CTA that loads and multiplies the next tile under the end of this
// one (1% shorter on a packed batch, 5% longer on one prompt).  16,384 tokens,
// 32 heads over 8: 2.03 to 2.12 ms on different boards in a loop of calls, 1.04 to
// 1.08 PFLOP/s, at the board's power limit (a single call from cold caches 1.82 ms).
// The d = 128 kernel spills 20 bytes at the 168 registers that 384 threads leave.
//
// Waits are bounded (sm100.cuh).  Compiled as a whole program: setmaxnreg
// moves registers from the other warps to the softmax.
#include <string.h>

#include "gqa_tiles.cuh"
#include "kernels.h"
#include "sm100.cuh"
#include "tmap.h"

namespace csa {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units

// Guarded tiles of a CTA of 256 consecutive tokens (the most: G = 1, NQ = 2) and
// 64 keys a tile: its rows end inside at most 5 tiles, and with a window begin
// inside at most 4.
constexpr int kMaxGuarded = 9;

template <int D>
struct Cfg {
    // q tiles of a CTA, CTAs of an SM: at d = 128 a K / V tile serves two q tiles
    // (one, and two CTAs an SM: 37% slower on one long prompt); at d = 64 two
    // CTAs are 3 to 8% faster, one's start and end are covered by the other.
    static constexpr int NQ = D == 128 ? 2 : 1;
    static constexpr int kCtas = D == 64 ? 2 : 1;
    static constexpr int BN = 64;                    // keys of a tile
    static constexpr int kSlots = 2;                 // S slots of a q tile
    // Stages of the V and of the K ring.  Where they are few, K has one more and is
    // loaded a tile ahead of V: S of a slot is the MMAs' next step after PV (8,192
    // tokens of d = 256, 32 heads over 8: 1.71 ms without, 1.18 ms).
    static constexpr int NS = D <= 128 ? 4 : D == 192 ? 3 : 2, kAhead = D <= 128 ? 0 : 1, NK = NS + kAhead;
    static constexpr int kThreads = NQ * 128 + 128;
    static constexpr int kTmem = 512 / kCtas;        // columns
    static constexpr int kQBytes = 128 * D * 2;
    static constexpr int kTileBytes = BN * D * 2;
};

template <int D>
struct Smem {
    using C = Cfg<D>;
    uint8_t q[C::NQ][C::kQBytes];    // [d/64][128 rows][64 bf16], 128-byte swizzle
    uint8_t k[C::NK][C::kTileBytes]; // [d/64][BN keys][64 bf16]
    uint8_t v[C::NS][C::kTileBytes];
    uint64_t q_full[C::NQ], k_full[C::NK], k_empty[C::NK], v_full[C::NS], v_empty[C::NS];
    uint64_t g_full[C::NS], v_ok[C::NS];  // guarded tiles: landed, cleared
    uint64_t s_full[2 * C::NQ], p_full[2 * C::NQ], o_done[2 * C::NQ], o_full[C::NQ], guard_done;
    uint32_t tmem_base;
    SeqTile tile;
    int bad;
    uint32_t bad_rows[kMaxGuarded][C::BN / 32];  // guarded tiles' rows with non-finite values
    int guarded_at[kMaxGuarded];                 // the guarded tiles' first keys
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
    return v;
}
__device__ __forceinline__ float lo2(uint64_t v) { return __uint_as_float(uint32_t(v)); }
__device__ __forceinline__ float hi2(uint64_t v) { return __uint_as_float(uint32_t(v >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// What a CTA works on: one sequence's tokens [tok0, tok0 + n_tok) (relative to
// the sequence) of one key / value head.
struct Work {
    int64_t q0, k0;    // packed rows of the sequence's first query and key
    int len_q, nk;     // queries; keys that exist
    int off;           // key position of query 0 (may be negative)
    int tok0, hk;
    int kb0;           // first key of the first tile
};

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, Cfg<D>::kCtas)
    prompt_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const PromptArgs a) {
    using C = Cfg<D>;
    using namespace sm100;
    constexpr int NQ = C::NQ, BN = C::BN, NS = C::NS, NK = C::NK;
    extern __shared__ uint8_t smem_raw[];
    Smem<D>& S = *reinterpret_cast<Smem<D>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kMma = NQ * 4, kTma = kMma + NQ, kGuards = 4 - NQ - 1;  // first warps, guard warps
    const int G = a.H / a.HK, tpt = 128 / G;  // tokens of a q tile
    auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_suspended<false>(bar, parity, a.status); };
    auto wait_warp = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_suspended<true>(bar, parity, a.status); };

    if (warp == kTma) {
        const SeqTile t = find_tile(a.cu_q, a.cu_k, a.n_seq, NQ * tpt, int(blockIdx.x / unsigned(a.HK)), lane);
        if (lane == 0) S.tile = t;
    }
    if (threadIdx.x == 32) {
        for (int i = 0; i < NQ; ++i) { mbar_init(&S.q_full[i], 1); mbar_init(&S.o_full[i], 1); }
        for (int i = 0; i < NK; ++i) {
            mbar_init(&S.k_full[i], 1); mbar_init(&S.k_empty[i], NQ);  // one arrival per MMA warp
        }
        for (int i = 0; i < NS; ++i) {
            mbar_init(&S.v_full[i], 1); mbar_init(&S.v_empty[i], NQ);
            mbar_init(&S.g_full[i], 1);
            mbar_init(&S.v_ok[i], kGuards);  // one arrival per guard warp
        }
        for (int i = 0; i < 2 * NQ; ++i) {
            mbar_init(&S.s_full[i], 1);
            mbar_init(&S.o_done[i], 1);
            mbar_init(&S.p_full[i], 4);  // one arrival per softmax warp of a tile
        }
        mbar_init(&S.guard_done, kGuards);
        S.bad = 0;
        for (int i = 0; i < kMaxGuarded * BN / 32; ++i) (&S.bad_rows[0][0])[i] = 0;
        fence_mbar_init();
        prefetch_tmap(&map_q);
        prefetch_tmap(&map_k);
        prefetch_tmap(&map_v);
    }
    if (warp == kMma) { tmem_alloc(&S.tmem_base, C::kTmem); tmem_relinquish(); }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // Where all 512 columns are allocated they begin at column 0: a constant, which
    // keeps the tensor instructions' addresses out of the registers.
    const uint32_t tmem = C::kTmem == 512 ? 0u : S.tmem_base;
    const uint32_t tO = tmem + NQ * 128;  // S slots at tmem + slot * BN, O of q tile i at tO + i * D

    Work w;
    int n_t[NQ];    // key tiles of each q tile
    int n_max = 0;
    const int seq = S.tile.s;
    if (seq >= 0) {
        w.hk = int(blockIdx.x % unsigned(a.HK));
        w.q0 = S.tile.q0;
        const int len_q = S.tile.len_q, len_k = S.tile.len_k;
        w.len_q = int(min(int64_t(len_q), a.n_q - w.q0));
        w.k0 = S.tile.k0;
        w.nk = int(max(min(w.k0 + len_k, a.n_k) - w.k0, int64_t(0)));
        w.off = len_k - len_q;
        w.tok0 = S.tile.tile * NQ * tpt;
        w.kb0 = first_seen(w.tok0 + w.off, a.W);
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            const int first = w.tok0 + i * tpt, last = min(first + tpt, w.len_q) - 1;
            const int hi = min(last + w.off, w.nk - 1);
            n_t[i] = (first < w.len_q && hi >= w.kb0) ? (hi - w.kb0) / BN + 1 : 0;
            n_max = max(n_max, n_t[i]);
        }
        // a tile is guarded if some row of the CTA does not see all of it
        const int t_first = min(w.tok0 + w.off, w.nk - 1), tok_last = min(w.tok0 + NQ * tpt, w.len_q) - 1;
        const int lo_last = first_seen(tok_last + w.off, a.W);
        auto guarded = [&](int j) {
            const int kb = w.kb0 + j * BN;
            return kb + BN - 1 > t_first || kb < lo_last;
        };

        if (warp == kTma) {
            if constexpr (NQ == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
            if (elect_one() && n_max > 0) {
                bool ok = true;
                int nk_issued = 0, nq_issued = 0;
                uint32_t v_par = 0, g_par = 0;  // bit st: parity of the phases begun on v_full, g_full
                auto load_q = [&](int i) {
                    mbar_arrive_expect_tx(&S.q_full[i], uint32_t(D * 2 * G * tpt));
#pragma unroll
                    for (int blk = 0; blk < D / 64; ++blk)
                        tma_load_3d(S.q[i] + blk * 16384, &map_q, 64 * blk, w.hk * G, int(w.q0) + w.tok0 + i * tpt,
                                    &S.q_full[i]);
                    nq_issued |= 1 << i;
                };
                auto load_k = [&](int j) {
                    const int st = j % NK;
                    if (j >= NK && !wait(&S.k_empty[st], uint32_t((j / NK - 1) & 1))) return false;
                    mbar_arrive_expect_tx(&S.k_full[st], C::kTileBytes);
#pragma unroll
                    for (int blk = 0; blk < D / 64; ++blk)
                        tma_load_3d(S.k[st] + blk * BN * 128, &map_k, 64 * blk, w.hk, int(w.k0) + w.kb0 + j * BN, &S.k_full[st]);
                    ++nk_issued;
                    return true;
                };
                load_q(0);
                if (C::kAhead == 1) ok = load_k(0);
                for (int j = 0; j < n_max && ok; ++j) {
                    if (j + C::kAhead < n_max) ok = load_k(j + C::kAhead);
                    if (NQ == 2 && j == 0 && n_t[NQ - 1] > 0) load_q(NQ - 1);
                    const int st = j % NS;
                    if (ok && j >= NS) ok = wait(&S.v_empty[st], uint32_t((j / NS - 1) & 1));
                    if (!ok) break;
                    uint64_t* full = guarded(j) ? &S.g_full[st] : &S.v_full[st];
                    mbar_arrive_expect_tx(full, C::kTileBytes);
#pragma unroll
                    for (int blk = 0; blk < D / 64; ++blk)
                        tma_load_3d(S.v[st] + blk * BN * 128, &map_v, 64 * blk, w.hk, int(w.k0) + w.kb0 + j * BN, full);
                    (guarded(j) ? g_par : v_par) ^= 1u << st;
                }
                // every copy has landed before the CTA ends (already so unless a consumer gave up)
                bool landed = true;
                for (int i = 0; i < NQ && landed; ++i)
                    if (nq_issued >> i & 1) landed = wait(&S.q_full[i], 0);
                for (int j = max(0, nk_issued - NK); j < nk_issued && landed; ++j)
                    landed = wait(&S.k_full[j % NK], uint32_t((j / NK) & 1));
                for (int st = 0; st < NS && landed; ++st)
                    landed = wait(&S.v_full[st], (v_par >> st & 1) ^ 1) &&
                             wait(&S.g_full[st], (g_par >> st & 1) ^ 1);
            }
        } else if (warp >= kMma && warp < kTma) {
            if constexpr (NQ == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
            if (n_max > 0) {
                // The whole warp runs the loop (uniform registers hold what the instructions need), one lane issues.
                constexpr uint32_t id_qk = instr_desc(1, 1, 0, 0, 128, BN);
                constexpr uint32_t id_pv = instr_desc(1, 1, 0, 1, 128, D);  // V: keys x dims, MN-major
                bool ok = true;
                uint32_t v_par = 0, g_par = 0;  // bit st: parity of the next phase of v_full, v_ok
                // descriptors count addresses in units of 16 bytes; offsets are added to a base
                const uint64_t d_q = smem_desc(smem_u32(S.q[0]), 16, 1024), d_k = smem_desc(smem_u32(S.k[0]), 16, 1024),
                               d_v = smem_desc(smem_u32(S.v[0]), BN * 128, 1024);
                auto commit = [&](uint64_t* bar) {
                    if (elect_one()) mma_commit(bar);
                };
                const int i = warp - kMma, n = n_t[i];
                auto qk = [&](int slot, int st) {
                    if (elect_one()) {
                        const uint64_t q0 = d_q + uint32_t(i * (C::kQBytes / 16)), kk = d_k + uint32_t(st * (C::kTileBytes / 16));
#pragma unroll
                        for (int s = 0; s < D / 16; ++s)
                            mma_f16(tmem + slot * BN, q0 + (s >> 2) * 1024 + (s & 3) * 2,
                                    kk + (s >> 2) * BN * 8 + (s & 3) * 2, id_qk, s != 0);
                        mma_commit(&S.s_full[slot]);
                    }
                };
                auto pv = [&](int slot, int st, bool first, uint64_t* done) {
                    if (elect_one()) {
                        const uint64_t vv = d_v + uint32_t(st * (C::kTileBytes / 16));
#pragma unroll
                        for (int s = 0; s < BN / 16; ++s)
                            mma_f16_ts(tO + i * D, tmem + slot * BN + 8 * s, vv + s * 128, id_pv, !first || s != 0);
                        mma_commit(done);
                    }
                };
                auto wait_v = [&](int j, int st) {
                    const bool g = guarded(j);
                    uint32_t& par = g ? g_par : v_par;
                    const uint32_t p = par >> st & 1;
                    par ^= 1u << st;
                    return wait_warp(g ? &S.v_ok[st] : &S.v_full[st], p);
                };
                // S of the first key tiles, then by tile: PV of it, S of the one that comes into its slot.
                // K and V of the next round are waited for before its P is: only that wait is in the chain.
                int st = 0, st2 = 0;       // stages of the tiles j and j + kSlots
                uint32_t k_par = 0;        // parity of k_full[st2]
                auto wait_k = [&]() { return wait_warp(&S.k_full[st2], k_par); };
                auto next_k = [&]() {
                    commit(&S.k_empty[st2]);
                    if (++st2 == NK) { st2 = 0; k_par ^= 1; }
                };
                ok = wait_warp(&S.q_full[0], 0);
                if (ok && i > 0 && n > 0) ok = wait_warp(&S.q_full[i], 0);
                for (int j = 0; j < C::kSlots && j < n_max && ok; ++j) {
                    ok = wait_k();
                    if (!ok) break;
                    if (j < n) qk(C::kSlots * i + j, st2);
                    next_k();
                }
                if (ok && C::kSlots < n_max) ok = wait_k();
                if (ok) ok = wait_v(0, 0);
                for (int j = 0; j < n_max && ok; ++j) {
                    const int slot = C::kSlots * i + j % C::kSlots;
                    if (j < n) {
                        ok = wait_warp(&S.p_full[slot], uint32_t(j / C::kSlots & 1));
                        if (!ok) break;
                        tc_fence_after();
                        pv(slot, st, j == 0, j == n - 1 ? &S.o_full[i] : &S.o_done[slot]);
                        if (j + C::kSlots < n) qk(slot, st2);
                    }
                    commit(&S.v_empty[st]);
                    if (++st == NS) st = 0;
                    if (j + C::kSlots < n_max) {
                        next_k();
                        if (j + 1 + C::kSlots < n_max) ok = wait_k();
                    }
                    if (ok && j + 1 < n_max) ok = wait_v(j + 1, st);
                }
            }
        } else if (warp > kTma) {
            if constexpr (NQ == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
            // ------------------------------------------------------- guard
            const int gt = threadIdx.x - (kTma + 1) * 32;  // 0 .. 32 kGuards - 1
            bool ok = true;
            uint32_t g_par = 0;
            int nth = 0;
            const __nv_bfloat162 zero2 = __floats2bfloat162_rn(0.f, 0.f);
            for (int j = 0; j < n_max && ok; ++j) {
                if (!guarded(j)) continue;
                const int st = j % NS, kb = w.kb0 + j * BN;
                ok = wait_warp(&S.g_full[st], g_par >> st & 1);
                if (!ok) break;
                g_par ^= 1u << st;
                const int live = min(w.nk - kb, BN);  // rows of the tile that exist
                // of those, [seen0, seen1) are seen by every row
                const int seen0 = max(lo_last - kb, 0), seen1 = t_first + 1 - kb;
                if (gt == 0) S.guarded_at[nth] = kb;
                uint4* const v = reinterpret_cast<uint4*>(S.v[st]);
                // row r's chunks are in their swizzled order, all are looked at
                for (int r = gt; r < BN; r += 32 * kGuards) {
                    if (r >= live) {
#pragma unroll
                        for (int c = 0; c < D / 8; ++c) v[(c >> 3) * BN * 8 + r * 8 + ((c ^ r) & 7)] = make_uint4(0, 0, 0, 0);
                    } else if (r < seen0 || r >= seen1) {
                        __nv_bfloat162 acc[4] = {zero2, zero2, zero2, zero2};  // NaN from any value that is not finite
#pragma unroll
                        for (int c = 0; c < D / 8; ++c) {
                            const uint4 x = v[(c >> 3) * BN * 8 + r * 8 + ((c ^ r) & 7)];
                            acc[0] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.x), zero2, acc[0]);
                            acc[1] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.y), zero2, acc[1]);
                            acc[2] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.z), zero2, acc[2]);
                            acc[3] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.w), zero2, acc[3]);
                        }
                        const __nv_bfloat162 all = __hadd2(__hadd2(acc[0], acc[1]), __hadd2(acc[2], acc[3]));
                        const float2 sum = __bfloat1622float2(all);
                        if (sum.x + sum.y != 0.f) {  // (NaN)
                            uint16_t* const e = reinterpret_cast<uint16_t*>(S.v[st]);
                            for (int i = 0; i < D; ++i) {
                                uint16_t* const p = e + (i >> 6) * BN * 64 + r * 64 + (i & 63);
                                if ((*p & 0x7F80) == 0x7F80) *p = 0;
                            }
                            atomicOr(&S.bad_rows[nth][r >> 5], 1u << (r & 31));
                            S.bad = 1;
                        }
                    }
                }
                ++nth;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.v_ok[st]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.guard_done);  // S.bad and its rows are complete
        } else {
            if constexpr (NQ == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
            // ----------------------------------------------------- softmax
            const int i = warp >> 2, r = threadIdx.x & 127;
            const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
            const int tok = w.tok0 + i * tpt + r / G, h = w.hk * G + r % G;
            const bool live = r < G * tpt && tok < w.len_q;
            const int t = live ? min(tok + w.off, w.nk - 1) : -1;       // last key that the row sees
            const int lo = first_seen(tok + w.off, a.W);  // first
            const int t_min = min(w.tok0 + i * tpt + w.off, w.nk - 1);    // of the tile's first token
            const int tl = min(w.tok0 + (i + 1) * tpt, w.len_q) - 1;
            const int lo_max = first_seen(tl + w.off, a.W);
            const float sl2 = a.scale * kLog2e;
            const uint64_t s2 = pack2(sl2, sl2);
            float m = -INFINITY, l = 0.f;
            bool ok = true;
            const int n = n_t[i];
            for (int j = 0; j < n && ok; ++j) {
                const int slot = C::kSlots * i + j % C::kSlots;
                ok = wait_warp(&S.s_full[slot], uint32_t(j / C::kSlots & 1));
                if (!ok) break;
                tc_fence_after();
                const uint32_t tS = tmem + slot * BN + lanes;
                const int kb = w.kb0 + j * BN;
                constexpr int NC = BN / 32;
                uint32_t x[NC][32];
#pragma unroll
                for (int c = 0; c < NC; ++c) tmem_ld32_start(tS + 32 * c, x[c]);
#pragma unroll
                for (int c = 0; c < NC; ++c) tmem_wait_ld32(x[c]);
                if (kb + BN - 1 > t_min || kb < lo_max) {
                    // of this row's columns [lo - kb, t - kb] are visible
#pragma unroll
                    for (int c = 0; c < BN; ++c)
                        if (c > t - kb || c < lo - kb) x[c / 32][c % 32] = 0xFF800000u;
                }
                float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < BN; c += 2)
                    mx4[c / 2 & 3] = max3(mx4[c / 2 & 3], __uint_as_float(x[c / 32][c % 32]), __uint_as_float(x[c / 32][c % 32 + 1]));
                const float mx = max3(mx4[0], mx4[1], max3(mx4[2], mx4[3], -INFINITY)) * sl2;
                if (!(mx < INFINITY)) l = __int_as_float(0x7FFFFFFF);  // NaN or +inf among the logits: the row is NaN
                float al = 1.f;
                if (mx > m + kRescaleThreshold || (m == -INFINITY && mx > -INFINITY)) {
                    al = m == -INFINITY ? 0.f : ex2(m - mx);
                    m = mx;
                }
                if (__any_sync(0xffffffffu, al != 1.f) && j > 0) {
                    // (PV of the tile before is waited for here only)
                    ok = wait_warp(&S.o_done[slot ^ (C::kSlots - 1)], uint32_t((j - 1) / C::kSlots & 1));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t ad = tO + i * D + lanes;
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32_start(ad + 32 * c, o);
                        tmem_wait_ld32(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                        tmem_st32(ad + 32 * c, o);
                    }
                }
                l *= al;
                const float neg = m == -INFINITY ? 0.f : -m;
                const uint64_t n2 = pack2(neg, neg);
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const uint64_t y = fma2(pack2(__uint_as_float(x[c][2 * e]), __uint_as_float(x[c][2 * e + 1])), s2, n2);
                        const uint64_t z = pack2(ex2(lo2(y)), ex2(hi2(y)));
                        sum[e & 1] = add2(sum[e & 1], z);
                        p[e] = bf16x2(lo2(z), hi2(z));  // P is rounded to bf16, the type that V takes it in
                    }
                    tmem_st16(tS + 16 * c, p);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.p_full[slot]);
                sum[0] = add2(sum[0], sum[1]);
                l += lo2(sum[0]) + hi2(sum[0]);
            }
            // ---------------------------------------------------- epilogue
            float f = 1.f, den = l;
            if (a.sinks && live) {
                const float sg = a.sinks[h] * kLog2e, M = fmaxf(m, sg);
                f = m == -INFINITY ? 0.f : ex2(m - M);
                den = l * f + (M == -INFINITY ? 0.f : ex2(sg - M));
            }
            f = den == 0.f ? 0.f : f / den;
            if (n > 0 && ok) ok = wait_warp(&S.o_full[i], 0) && wait_warp(&S.guard_done, 0);
            tc_fence_after();
            // The warp's rows go through its part of the q tile, which nothing reads any more (where the tile has no
            // keys q may still be under way: it is waited for), so that whole rows are written: a row a lane, 16 bytes
            // an instruction, took 4,000 clocks of a CTA.
            if (n == 0 && i == 0 && n_max > 0) wait_warp(&S.q_full[0], 0);
            uint4* const stage = reinterpret_cast<uint4*>(S.q[i] + (warp & 3) * (32 * D * 2));
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                if (n > 0 && ok) {
                    tmem_ld32_start(tO + i * D + lanes + 32 * c, o);
                    tmem_wait_ld32(o);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0;
                }
                if (S.bad) {  // the non-finite values that this row sees (they came out of the tiles as 0)
                    for (int x = 0; x < kMaxGuarded * BN; ++x) {
                        if (!(S.bad_rows[x / BN][x % BN / 32] >> (x % 32) & 1)) continue;
                        const int key = S.guarded_at[x / BN] + x % BN;
                        if (key < lo || key > t) continue;
                        const uint16_t* vp = (const uint16_t*)a.v + (w.k0 + key) * a.v_ld + int64_t(w.hk) * D + 32 * c;
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float y = bf16_bits_to_f32(vp[e]);
                            if (!(fabsf(y) < INFINITY)) o[e] = __float_as_uint(__uint_as_float(o[e]) + y);
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t y[4];
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        y[g] = bf16x2(__uint_as_float(o[8 * e + 2 * g]) * f, __uint_as_float(o[8 * e + 2 * g + 1]) * f);
                    stage[lane * (D / 8) + ((4 * c + e) ^ (lane & 7))] = make_uint4(y[0], y[1], y[2], y[3]);
                }
            }
            __syncwarp();
            const int mine = live ? int((w.q0 + tok) * a.H + h) : -1;  // row of the output
#pragma unroll 4
            for (int x = lane; x < 32 * (D / 8); x += 32) {
                const int rr = x / (D / 8), ch = x % (D / 8);
                const int to = __shfl_sync(0xffffffffu, mine, rr);
                if (to >= 0)
                    reinterpret_cast<uint4*>((__nv_bfloat16*)a.out + int64_t(to) * D)[ch] = stage[rr * (D / 8) + (ch ^ (rr & 7))];
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kMma) tmem_dealloc(tmem, C::kTmem);
}

bool prompt_tc_supported(const PromptArgs& a) {
    // a scale of 0 or below would turn the masked -inf (times scale) into NaN or +inf
    return a.act_fmt == CSA_BF16 && a.n_k > 0 && a.scale > 0.f && a.scale < INFINITY;
}

template <int D>
static cudaError_t launch_prompt_tc_d(PromptArgs a, cudaStream_t s) {
    using C = Cfg<D>;
    const int G = a.H / a.HK, tpt = 128 / G;
    CUtensorMap mq, mk, mv;
    const uint64_t dq[3] = {uint64_t(D), uint64_t(a.H), uint64_t(a.n_q)};
    const uint64_t sq[2] = {uint64_t(D) * 2, uint64_t(a.q_ld) * 2};
    const uint32_t bq[3] = {64, uint32_t(G), uint32_t(tpt)};
    const uint64_t dk[3] = {uint64_t(D), uint64_t(a.HK), uint64_t(a.n_k)};
    const uint64_t sk[2] = {uint64_t(D) * 2, uint64_t(a.k_ld) * 2};
    const uint64_t sv[2] = {uint64_t(D) * 2, uint64_t(a.v_ld) * 2};
    const uint32_t bk[3] = {64, 1, uint32_t(C::BN)};
    if (!encode_tile_map(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.q, dq, sq, bq, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tile_map(&mk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.k, dk, sk, bk, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tile_map(&mv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.v, dk, sv, bk, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    const size_t sm = sizeof(Smem<D>) + 1024;
    static_assert(sizeof(Smem<D>) + 1024 <= 227 * 1024, "shared memory");
    cudaError_t e = ensure_smem(prompt_tc_kernel<D>, sm);
    if (e == cudaSuccess) e = device_status_word(&a.status);
    if (e != cudaSuccess) return e;
    // an upper bound of the tiles: the lengths are on the device
    const int64_t tiles = a.n_q / (C::NQ * tpt) + std::min<int64_t>(a.n_seq, a.n_q);
    if (tiles * a.HK > INT32_MAX) return cudaErrorInvalidValue;
    prompt_tc_kernel<D><<<unsigned(tiles * a.HK), C::kThreads, sm, s>>>(mq, mk, mv, a);
    return cudaGetLastError();
}

cudaError_t launch_prompt_tc(const PromptArgs& a, cudaStream_t s) {
    switch (a.D) {
        case 64: return launch_prompt_tc_d<64>(a, s);
        case 128: return launch_prompt_tc_d<128>(a, s);
        case 192: return launch_prompt_tc_d<192>(a, s);
        default: return launch_prompt_tc_d<256>(a, s);
    }
}

}  // namespace csa
