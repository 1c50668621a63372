// Causal attention over packed prompts on the 5th-generation tensor cores
// (bf16, head dims 64, 128, 192, 256).
//
//   S = Q K^T ; P = exp2(S scale log2e - m) ; O = sum P V ; out = O / sum P
//
// A q tile is 128 rows of one key / value head: floor(128 / G) tokens times
// the G query heads that share the head, so that a K / V tile serves all of
// them and short sequences fill the rows.  A CTA owns NQ q tiles of
// consecutive tokens (two for d <= 128, one above) and walks the keys that
// any of its rows sees in tiles of BN, with the running maximum and sum of
// each row in the thread that owns the row; P never leaves the SM.
//
//   S[row][key]  = Q (smem) . K^T (smem)    M = 128, N = BN, K = d    -> TMEM
//   O[row][dim] += P (TMEM) . V (smem)      M = 128, N = d, K = BN    -> TMEM
//
// P (bf16) overwrites the S columns it came from.  Per q tile (NQ = 2) or per
// parity of the key tile (NQ = 1) there is one S slot, and the MMA thread
// issues the product of one slot while the softmax works on the other: PV of
// a slot, then the next QK into it (the tensor pipe runs them in order).
// O is rescaled in TMEM only when a row's maximum has grown by more than 8
// (log2 units) over the one in use.
//
// Roles: NQ warpgroups of softmax (thread = row; they also write the output),
// then warp MMA (one thread issues), warp TMA (one thread loads q, K and V by
// swizzled tensor copies; q rows of a tile are one box of G heads x tokens),
// and two guard warps.  A tile that some row may not see completely is a
// guarded one: before its PV the guard warps clear V rows past the sequence
// (they belong to other sequences or are padding) and look for infinities and
// NaN in the others, which a probability of 0 would not keep out of the sum.
// If there are any, the CTA computes its rows once more, one key at a time
// (attend_rows_slowly); that costs finite inputs only the look.
//
// Waits are bounded (sm100.cuh).
#include <string.h>

#include "kernels.h"
#include "sm100.cuh"
#include "tmap.h"

namespace csa {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units

template <int D>
struct Cfg {
    static constexpr int NQ = D <= 128 ? 2 : 1;      // q tiles of a CTA
    static constexpr int BN = D <= 128 ? 128 : 64;   // keys of a tile
    static constexpr int NS = D == 64 ? 4 : D == 192 ? 3 : 2;  // stages of the K and of the V ring
    static constexpr int kThreads = NQ * 128 + 128;
    static constexpr int kQBytes = 128 * D * 2;
    static constexpr int kTileBytes = BN * D * 2;
};

template <int D>
struct Smem {
    using C = Cfg<D>;
    uint8_t q[C::NQ][C::kQBytes];    // [d/64][128 rows][64 bf16], 128-byte swizzle
    uint8_t k[C::NS][C::kTileBytes]; // [d/64][BN keys][64 bf16]
    uint8_t v[C::NS][C::kTileBytes];
    uint64_t q_full[C::NQ], k_full[C::NS], k_empty[C::NS], v_full[C::NS], v_empty[C::NS];
    uint64_t g_full[C::NS], v_ok[C::NS];  // guarded tiles: landed, cleared
    uint64_t s_full[2], p_full[2], o_done, o_full[C::NQ];
    uint32_t tmem_base;
    int seq, tile, bad;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint64_t pack2(float x, float y) {
    return uint64_t(__float_as_uint(x)) | (uint64_t(__float_as_uint(y)) << 32);
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

// A row at a time, a key at a time, by one warp: what the tile path cannot do
// (non-finite values among the keys that some rows do not see).
template <int D>
__device__ __noinline__ void attend_rows_slowly(const PromptArgs& a, const Work& w, int tok_begin, int rows, int G,
                                                int lane) {
    constexpr int E = D / 32;
    for (int r = 0; r < rows; ++r) {
        const int tok = tok_begin + r / G, h = w.hk * G + r % G;
        if (tok >= w.len_q) break;
        const int t = min(tok + w.off, w.nk - 1), lo = a.W > 0 ? max(tok + w.off - a.W + 1, 0) : 0;
        float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            q[e] = bf16_bits_to_f32(((const uint16_t*)a.q)[(w.q0 + tok) * a.q_ld + int64_t(h) * D + lane + 32 * e]);
            o[e] = 0.f;
        }
        for (int j = lo; j <= t; ++j) {
            const uint16_t* kp = (const uint16_t*)a.k + (w.k0 + j) * a.k_ld + int64_t(w.hk) * D + lane;
            const uint16_t* vp = (const uint16_t*)a.v + (w.k0 + j) * a.v_ld + int64_t(w.hk) * D + lane;
            float x = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) x += q[e] * bf16_bits_to_f32(kp[32 * e]);
            x = warp_sum(x) * (a.scale * kLog2e);
            if (x == -INFINITY) continue;
            if (x > m) {
                const float al = m == -INFINITY ? 0.f : ex2(m - x);
                l *= al;
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = al == 0.f ? 0.f : o[e] * al;
                m = x;
            }
            const float p = ex2(x - m);
            l += p;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] += p * bf16_bits_to_f32(vp[32 * e]);
        }
        float f = 1.f, den = l;
        if (a.sinks) {
            const float sg = a.sinks[h] * kLog2e, M = fmaxf(m, sg);
            f = m == -INFINITY ? 0.f : ex2(m - M);
            den = l * f + (M == -INFINITY ? 0.f : ex2(sg - M));
        }
        f = den == 0.f ? 0.f : f / den;
        __nv_bfloat16* out = (__nv_bfloat16*)a.out + ((w.q0 + tok) * a.H + h) * int64_t(D) + lane;
#pragma unroll
        for (int e = 0; e < E; ++e) out[32 * e] = __float2bfloat16_rn(o[e] * f);
    }
}

}  // namespace

// The tile of a packed batch: sequences in order, the tiles of a sequence last
// (longest) first.  Called by one warp; s = -1 behind the last tile.
__device__ __forceinline__ void find_tile(const int32_t* cu, int n_seq, int per, int x, int lane, int& s, int& tile) {
    int before = 0;
    s = -1;
    tile = 0;
    for (int base = 0; base < n_seq; base += 32) {
        const int i = base + lane;
        const int n = i < n_seq ? max(cu[i + 1] - cu[i], 0) : 0;
        const int mine = (n + per - 1) / per;
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        const unsigned in = __ballot_sync(0xffffffffu, x < before + upto);
        if (in) {
            const int src = __ffs(int(in)) - 1;
            s = base + src;
            const int end = before + __shfl_sync(0xffffffffu, upto, src);
            tile = end - 1 - x;  // counted from the sequence's last tile
            return;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
}

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
    prompt_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const PromptArgs a) {
    using C = Cfg<D>;
    using namespace sm100;
    constexpr int NQ = C::NQ, BN = C::BN, NS = C::NS;
    extern __shared__ uint8_t smem_raw[];
    Smem<D>& S = *reinterpret_cast<Smem<D>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kMma = NQ * 4, kTma = kMma + 1;
    const int G = a.H / a.HK, tpt = 128 / G;  // tokens of a q tile

    if (warp == 0) {
        int s, tile;
        find_tile(a.cu_q, a.n_seq, NQ * tpt, int(blockIdx.x / unsigned(a.HK)), lane, s, tile);
        if (lane == 0) { S.seq = s; S.tile = tile; }
    }
    if (threadIdx.x == 32) {
        for (int i = 0; i < NQ; ++i) { mbar_init(&S.q_full[i], 1); mbar_init(&S.o_full[i], 1); }
        for (int i = 0; i < NS; ++i) {
            mbar_init(&S.k_full[i], 1); mbar_init(&S.k_empty[i], 1);
            mbar_init(&S.v_full[i], 1); mbar_init(&S.v_empty[i], 1);
            mbar_init(&S.g_full[i], 1);
            mbar_init(&S.v_ok[i], 2);  // one arrival per guard warp
        }
        for (int i = 0; i < 2; ++i) { mbar_init(&S.s_full[i], 1); mbar_init(&S.p_full[i], 4); }
        mbar_init(&S.o_done, 1);
        S.bad = 0;
        fence_mbar_init();
        prefetch_tmap(&map_q);
        prefetch_tmap(&map_k);
        prefetch_tmap(&map_v);
    }
    if (warp == kMma) { tmem_alloc(&S.tmem_base, 512); tmem_relinquish(); }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem_base;
    const uint32_t tO = tmem + 2 * BN;  // S slots at tmem + slot * BN, O of q tile i at tO + i * D

    Work w;
    int n_t[NQ];    // key tiles of each q tile
    int n_max = 0;
    const int seq = S.seq;
    if (seq >= 0) {
        w.hk = int(blockIdx.x % unsigned(a.HK));
        w.q0 = a.cu_q[seq];
        const int len_q = a.cu_q[seq + 1] - int(w.q0);
        w.len_q = int(min(int64_t(len_q), a.n_q - w.q0));
        w.k0 = a.cu_k[seq];
        const int len_k = a.cu_k[seq + 1] - int(w.k0);
        w.nk = int(max(min(w.k0 + len_k, a.n_k) - w.k0, int64_t(0)));
        w.off = len_k - len_q;
        w.tok0 = S.tile * NQ * tpt;
        w.kb0 = a.W > 0 ? max(w.tok0 + w.off - a.W + 1, 0) : 0;
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            const int first = w.tok0 + i * tpt, last = min(first + tpt, w.len_q) - 1;
            const int hi = min(last + w.off, w.nk - 1);
            n_t[i] = (first < w.len_q && hi >= w.kb0) ? (hi - w.kb0) / BN + 1 : 0;
            n_max = max(n_max, n_t[i]);
        }
        // a tile is guarded if some row of the CTA does not see all of it
        const int t_first = w.tok0 + w.off, tok_last = min(w.tok0 + NQ * tpt, w.len_q) - 1;
        const int lo_last = a.W > 0 ? max(tok_last + w.off - a.W + 1, 0) : 0;
        auto guarded = [&](int j) {
            const int kb = w.kb0 + j * BN;
            return kb + BN - 1 > t_first || kb < lo_last;
        };

        if (warp == kTma) {
            if constexpr (NQ == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
            if (lane == 0 && n_max > 0) {
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
                load_q(0);
                for (int j = 0; j < n_max && ok; ++j) {
                    const int st = j % NS;
                    const int row = int(w.k0) + w.kb0 + j * BN;
                    if (j >= NS) ok = mbar_wait(&S.k_empty[st], uint32_t((j / NS - 1) & 1));
                    if (!ok) break;
                    mbar_arrive_expect_tx(&S.k_full[st], C::kTileBytes);
#pragma unroll
                    for (int blk = 0; blk < D / 64; ++blk)
                        tma_load_3d(S.k[st] + blk * BN * 128, &map_k, 64 * blk, w.hk, row, &S.k_full[st]);
                    ++nk_issued;
                    if (NQ == 2 && j == 0 && n_t[NQ - 1] > 0) load_q(NQ - 1);
                    if (j >= NS) ok = mbar_wait(&S.v_empty[st], uint32_t((j / NS - 1) & 1));
                    if (!ok) break;
                    uint64_t* full = guarded(j) ? &S.g_full[st] : &S.v_full[st];
                    mbar_arrive_expect_tx(full, C::kTileBytes);
#pragma unroll
                    for (int blk = 0; blk < D / 64; ++blk)
                        tma_load_3d(S.v[st] + blk * BN * 128, &map_v, 64 * blk, w.hk, row, full);
                    (guarded(j) ? g_par : v_par) ^= 1u << st;
                }
                // every copy has landed before the CTA ends (already so unless a consumer gave up)
                bool landed = true;
                for (int i = 0; i < NQ && landed; ++i)
                    if (nq_issued >> i & 1) landed = mbar_wait(&S.q_full[i], 0);
                for (int j = max(0, nk_issued - NS); j < nk_issued && landed; ++j)
                    landed = mbar_wait(&S.k_full[j % NS], uint32_t((j / NS) & 1));
                for (int st = 0; st < NS && landed; ++st)
                    landed = mbar_wait(&S.v_full[st], (v_par >> st & 1) ^ 1) &&
                             mbar_wait(&S.g_full[st], (g_par >> st & 1) ^ 1);
            }
        } else if (warp == kMma) {
            if constexpr (NQ == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
            if (lane == 0 && n_max > 0) {
                const uint32_t id_qk = instr_desc(1, 1, 0, 0, 128, BN);
                const uint32_t id_pv = instr_desc(1, 1, 0, 1, 128, D);  // V: keys x dims, MN-major
                bool ok = true;
                uint32_t v_par = 0, g_par = 0;  // bit st: parity of the next phase of v_full, v_ok
                auto qk = [&](int i, int slot, int j) {
                    const uint32_t q0 = smem_u32(S.q[i]), kk = smem_u32(S.k[j % NS]);
#pragma unroll
                    for (int s = 0; s < D / 16; ++s)
                        mma_f16(tmem + slot * BN, smem_desc(q0 + (s >> 2) * 16384 + (s & 3) * 32, 16, 1024),
                                smem_desc(kk + (s >> 2) * BN * 128 + (s & 3) * 32, 16, 1024), id_qk, s != 0);
                    mma_commit(&S.s_full[slot]);
                };
                auto pv = [&](int i, int slot, int j) {
                    const uint32_t vv = smem_u32(S.v[j % NS]);
#pragma unroll
                    for (int s = 0; s < BN / 16; ++s)
                        mma_f16_ts(tO + i * D, tmem + slot * BN + 8 * s,
                                   smem_desc(vv + s * 2048, BN * 128, 1024), id_pv, (j | s) != 0);
                };
                auto wait_v = [&](int j) {
                    const int st = j % NS;
                    const bool g = guarded(j);
                    uint32_t& par = g ? g_par : v_par;
                    const uint32_t p = par >> st & 1;
                    par ^= 1u << st;
                    return mbar_wait(g ? &S.v_ok[st] : &S.v_full[st], p);
                };
                auto wait_k = [&](int j) { return mbar_wait(&S.k_full[j % NS], uint32_t((j / NS) & 1)); };
                if constexpr (NQ == 2) {
                    ok = wait_k(0);
                    for (int i = 0; i < 2 && ok; ++i)
                        if (n_t[i] > 0) {
                            ok = mbar_wait(&S.q_full[i], 0);
                            if (ok) qk(i, i, 0);
                        }
                    if (ok) mma_commit(&S.k_empty[0]);
                    for (int j = 0; j < n_max && ok; ++j) {
                        ok = wait_v(j);
                        bool have_k = false;
                        for (int i = 0; i < 2 && ok; ++i) {
                            if (j < n_t[i]) {
                                ok = mbar_wait(&S.p_full[i], uint32_t(j & 1));
                                if (!ok) break;
                                tc_fence_after();
                                pv(i, i, j);
                                if (j == n_t[i] - 1) mma_commit(&S.o_full[i]);
                            }
                            if (j + 1 < n_t[i]) {
                                if (!have_k) { ok = wait_k(j + 1); have_k = true; }
                                if (ok) qk(i, i, j + 1);
                            }
                        }
                        if (!ok) break;
                        mma_commit(&S.v_empty[j % NS]);
                        if (j + 1 < n_max) mma_commit(&S.k_empty[(j + 1) % NS]);
                    }
                } else {
                    ok = wait_k(0) && mbar_wait(&S.q_full[0], 0);
                    if (ok) { qk(0, 0, 0); mma_commit(&S.k_empty[0]); }
                    if (ok && n_max > 1) {
                        ok = wait_k(1);
                        if (ok) { qk(0, 1, 1); mma_commit(&S.k_empty[1 % NS]); }
                    }
                    for (int j = 0; j < n_max && ok; ++j) {
                        ok = wait_v(j) && mbar_wait(&S.p_full[j & 1], uint32_t((j >> 1) & 1));
                        if (!ok) break;
                        tc_fence_after();
                        pv(0, j & 1, j);
                        mma_commit(&S.v_empty[j % NS]);
                        mma_commit(&S.o_done);
                        if (j == n_max - 1) mma_commit(&S.o_full[0]);
                        if (j + 2 < n_max) {
                            ok = wait_k(j + 2);
                            if (ok) { qk(0, j & 1, j + 2); mma_commit(&S.k_empty[(j + 2) % NS]); }
                        }
                    }
                }
            }
        } else if (warp > kTma) {
            if constexpr (NQ == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
            // ------------------------------------------------------- guard
            const int gt = threadIdx.x - (kTma + 1) * 32;  // 0..63
            bool ok = true;
            uint32_t g_par = 0;
            for (int j = 0; j < n_max && ok; ++j) {
                if (!guarded(j)) continue;
                const int st = j % NS, kb = w.kb0 + j * BN;
                ok = mbar_wait(&S.g_full[st], g_par >> st & 1);
                if (!ok) break;
                g_par ^= 1u << st;
                bool bad = false;
                const int live = w.nk - kb;  // rows of the tile that exist
                for (int c = gt; c < C::kTileBytes / 16; c += 64) {
                    uint4* p = reinterpret_cast<uint4*>(S.v[st]) + c;
                    if ((c >> 3) % BN >= live) {
                        *p = make_uint4(0, 0, 0, 0);
                    } else {
                        const uint4 x = *p;
                        const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            bad |= (y[i] & 0x7F80u) == 0x7F80u || (y[i] & 0x7F800000u) == 0x7F800000u;
                    }
                }
                if (bad) S.bad = 1;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.v_ok[st]);
            }
        } else {
            if constexpr (NQ == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
            // ----------------------------------------------------- softmax
            const int i = warp >> 2, r = threadIdx.x & 127;
            const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
            const int tok = w.tok0 + i * tpt + r / G, h = w.hk * G + r % G;
            const bool live = r < G * tpt && tok < w.len_q;
            const int t = live ? min(tok + w.off, w.nk - 1) : -1;       // last key that the row sees
            const int lo = a.W > 0 ? max(tok + w.off - a.W + 1, 0) : 0;  // first
            const int t_min = w.tok0 + i * tpt + w.off;                   // of the tile's first token
            const int tl = min(w.tok0 + (i + 1) * tpt, w.len_q) - 1;
            const int lo_max = a.W > 0 ? max(tl + w.off - a.W + 1, 0) : 0;
            const float sl2 = a.scale * kLog2e;
            float m = -INFINITY, l = 0.f;
            bool ok = true;
            const int n = n_t[i];
            for (int j = 0; j < n && ok; ++j) {
                const int slot = NQ == 2 ? i : (j & 1);
                ok = mbar_wait(&S.s_full[slot], uint32_t((NQ == 2 ? j : j >> 1) & 1));
                if (!ok) break;
                tc_fence_after();
                const uint32_t tS = tmem + slot * BN + lanes;
                uint32_t x[BN / 32][32];
#pragma unroll
                for (int c = 0; c < BN / 32; ++c) tmem_ld32_start(tS + 32 * c, x[c]);
#pragma unroll
                for (int c = 0; c < BN / 32; ++c) tmem_wait_ld32(x[c]);
                const int kb = w.kb0 + j * BN;
                if (kb + BN - 1 > t_min || kb < lo_max) {
                    // columns [lo - kb, t - kb] of this row are visible
                    const int c1 = t - kb, c0 = lo - kb;
#pragma unroll
                    for (int c = 0; c < BN; ++c)
                        if (c > c1 || c < c0) x[c / 32][c % 32] = 0xFF800000u;
                }
                float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < BN; ++c) mx4[c & 3] = fmaxf(mx4[c & 3], __uint_as_float(x[c / 32][c % 32]));
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sl2;
                float al = 1.f;
                if (mx > m + kRescaleThreshold || (m == -INFINITY && mx != -INFINITY)) {
                    al = m == -INFINITY ? 0.f : ex2(m - mx);
                    m = mx;
                }
                if (__any_sync(0xffffffffu, al != 1.f) && j > 0) {
                    if (NQ == 1) {  // (NQ = 2: the S tile's commit came after the last PV's)
                        ok = mbar_wait(&S.o_done, uint32_t((j - 1) & 1));
                        if (!ok) break;
                        tc_fence_after();
                    }
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
                const uint64_t s2 = pack2(sl2, sl2), n2 = pack2(neg, neg);
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int c = 0; c < BN / 32; c += 2) {
                    uint32_t p[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const int k = 32 * c + 2 * e;
                        const uint64_t y = fma2(pack2(__uint_as_float(x[k / 32][k % 32]), __uint_as_float(x[k / 32][k % 32 + 1])), s2, n2);
                        const float p0 = ex2(lo2(y)), p1 = ex2(hi2(y));
                        sum[e & 1] = add2(sum[e & 1], pack2(p0, p1));
                        p[e] = bf16x2(p0, p1);
                    }
                    tmem_st32(tS + 16 * c, p);
                }
                sum[0] = add2(sum[0], sum[1]);
                l += lo2(sum[0]) + hi2(sum[0]);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.p_full[slot]);
            }
            // ---------------------------------------------------- epilogue
            float f = 1.f, den = l;
            if (a.sinks && live) {
                const float sg = a.sinks[h] * kLog2e, M = fmaxf(m, sg);
                f = m == -INFINITY ? 0.f : ex2(m - M);
                den = l * f + (M == -INFINITY ? 0.f : ex2(sg - M));
            }
            f = den == 0.f ? 0.f : f / den;
            if (n > 0 && ok) ok = mbar_wait(&S.o_full[i], 0);
            tc_fence_after();
            __nv_bfloat16* out = (__nv_bfloat16*)a.out + ((w.q0 + tok) * a.H + h) * int64_t(D);
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
                if (live) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t y[4];
#pragma unroll
                        for (int g = 0; g < 4; ++g)
                            y[g] = bf16x2(__uint_as_float(o[8 * e + 2 * g]) * f, __uint_as_float(o[8 * e + 2 * g + 1]) * f);
                        *reinterpret_cast<uint4*>(out + 32 * c + 8 * e) = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kMma) tmem_dealloc(tmem, 512);
    // Non-finite values in a guarded tile: each softmax warp redoes 32 rows of
    // its tile from memory (the barrier has ordered the first results' writes).
    if (seq >= 0 && S.bad && warp < kMma) {
        const int tile = warp >> 2, part = (tpt + 3) / 4;
        const int first = w.tok0 + tile * tpt + (warp & 3) * part;
        const int n = min(part, tpt - (warp & 3) * part);
        if (n > 0) attend_rows_slowly<D>(a, w, first, n * G, G, lane);
    }
}

bool prompt_tc_supported(const PromptArgs& a) {
    // a scale of 0 or below would turn the masked -inf (times scale) into NaN or +inf
    return a.act_fmt == CSA_BF16 && a.n_k > 0 && a.scale > 0.f && a.scale < INFINITY;
}

template <int D>
static cudaError_t launch_prompt_tc_d(const PromptArgs& a, cudaStream_t s) {
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
    const cudaError_t e = ensure_smem(prompt_tc_kernel<D>, sm);
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
