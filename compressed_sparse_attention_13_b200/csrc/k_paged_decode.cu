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
// The split over the blocks and the copies: paged_split.cuh.  A warp's tile is
// 16 tokens.  The running maximum of a head is raised only when a tile exceeds
// it by more than 8 in log2 units (one vote a tile otherwise), sums stay per
// lane until the unit ends.  P is rounded to the 16-bit type of the MMAs (bf16;
// f16 for FP8 entries).
//
// 32 sequences of up to 11,073 tokens, 32 heads over 8 (682 MB): 110 us, 6.2 TB/s;
// four of up to 131,072, 64 heads over 8 (1752 MB): 267 us, 6.6 TB/s; 16 of up to
// 32,768 in FP8, 32 heads over 8 (1006 MB): 163 to 183 us on different boards, 5.5 to
// 6.2 TB/s.
//
// FP8 entries (E4M3 codes, fp32 scale per 64 channels) are converted to f16
// exactly, one instruction per pair, and the MMAs run in f16: the query is
// scaled by a power of two per head (exact within 2^26 of the head's largest
// element), the key scales multiply S per 64 channels, and P takes the value
// scales.  So that p * scale fits f16 whatever the scales, it is kept in units
// per (head, 64 channels) that follow its running maximum, and O is in those
// units: a power of two when they are set, times what the row's maximum has grown
// since.  They lie between 2^-100 and 2^100, S is formed in fp32 from the codes'
// products: entries up to 2^100 in magnitude are safe.
#include "paged_split.cuh"

namespace csa {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescale = 8.0f;       // log2 units

template <int D, bool FP8, int NT>
struct Dec {
    static constexpr int kTok = 16;                      // tokens of a warp's tile
    static constexpr int kStep = kNW * kTok;             // of a step
    static constexpr int kRow = FP8 ? D : 2 * D;         // bytes of a cache row
    static constexpr int kChunks = kRow / 16;
    static constexpr int kGroups = D / 64;
    static constexpr int kScaleBytes = FP8 ? kTok * kGroups * 4 : 0;
    static constexpr int kTile = 2 * (kTok * kRow + kScaleBytes);  // K and V of 16 tokens
    // CTAs an SM, and stages of what shared memory is left for them: as many as the registers allow where the
    // warps' instructions bound the kernel (FP8; short rows), else two, one where only that leaves two stages.
    // 16 sequences of up to 32,768 tokens in FP8: d = 64, 138 us with two and 114 with three, d = 128, 178 and
    // 162 (G = 16: 236 and 252), d = 192, 352 with one and 245 with two, d = 256, 398 and 309; 32 sequences of
    // up to 11,073 in bf16: d = 64, 67 with two and 63 with three, d = 192, 172 with one and 160 with two.
    static constexpr int kCtas = D == 256 && !FP8 ? 1 : D <= 128 && (FP8 || D == 64) && NT == 1 ? 3 : 2;
    static constexpr int kBudget = (kCtas == 3 ? 60 : kCtas == 1 ? 192 : D == 256 ? 90 : 96) * 1024;
    static constexpr int kStages = kBudget / (kNW * kTile) > 8 ? 8 : kBudget / (kNW * kTile);
    static constexpr int kHeads = 8 * NT;
    static constexpr int kJoinDims = D > 64 ? D / 2 : D; // the warps' results are joined in halves of the dims
    static constexpr int kJoin = kJoinDims + 4;          // padded row of the join buffer
    static constexpr int kRing = kNW * kStages * kTile;
    static constexpr int kSmem = kRing + kNW * 8 * kJoin * 4;
    static_assert(kCtas * (kSmem + 2048 + kAlignSmem) <= 228 * 1024, "shared memory");
    static constexpr int kSlot = kHeads * (D + 2);       // floats of a partial: (m, l) per head, O
};

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
}  // namespace

template <int D, bool FP8, int NT>
__global__ void __launch_bounds__(32 * kNW, Dec<D, FP8, NT>::kCtas)
    paged_decode_kernel(const PagedDecodeArgs a, int units, int hb, JoinRec* recs, float* slots) {
    using C = Dec<D, FP8, NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = aligned_smem(smem_raw);
    __shared__ Plan plan;
    __shared__ uint32_t vmask[kNW][8];
    __shared__ float2 jml[kNW][8 * NT];
    float* const jo = reinterpret_cast<float*>(smem + C::kRing);  // [kNW][8][kJoin]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c4 = lane & 3;
    pdl_launch_dependents();
    make_plan<C::kStep>(a, units, &plan);
    if (!a.invariant && threadIdx.x == 0) recs[blockIdx.x].n = 0;
    const int64_t x0 = plan.x0, x1 = plan.x1;
    if (x0 >= x1) return;
    const int G = a.H / a.HK;
    const float sl2 = a.scale * kLog2e;

    Cursor cur;
    cur.x = x0; cur.x1 = x1; cur.s = plan.s; cur.u = plan.u; cur.at = plan.at;
    cur.v = span_of<C::kStep>(a, cur.s);

    // ------------------------------------------------------- the copying side
    constexpr int kTok = C::kTok;
    const uint32_t ring = smem_addr(smem) + uint32_t(warp) * C::kStages * C::kTile;
    Copier<C, FP8> copier(a, units, hb, cur, ring, vmask[warp]);
#pragma unroll 1
    for (int i = 0; i < C::kStages - 1; ++i) copier.issue(i);

    // ------------------------------------------------------ the computing side
    int stage = 0;
#pragma unroll 1
    while (cur.x < cur.x1) {
        int b, e, dx;
        piece_of<C::kStep>(a, cur, b, e, dx);
        if (b >= e) {
            advance<C::kStep>(a, units, cur, dx);
            continue;
        }
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
        float f[NT][FP8 ? C::kGroups : 1][2];  // FP8: what P is multiplied by
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
                copier.issue(nx);
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
                float s1[NT][4];  // a second chain of products: half the latency
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s1[nt][i] = 0.f;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t x[4];
                    ldsm4(k0 + place<kTok, C::kRow>(lane & 15, 2 * k + (lane >> 4)), x);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma<false>(k & 1 ? s1[nt] : s[nt], x, qf[nt][k][0], qf[nt][k][1]);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[nt][i] += s1[nt][i];
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
                        ldsm4(k0 + place<kTok, C::kRow>(lane & 15, 4 * gr + 2 * h + (lane >> 4)), w);
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
                    ldsm4_t(v0 + place<kTok, C::kRow>((lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)), x);
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
                        ldsm4_t(v0 + place<kTok, C::kRow>(lane & 15, 4 * gr + 2 * h + (lane >> 4)), w);
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
        if constexpr (FP8) {  // from here on what O is multiplied by (2^-100 .. 2^100); a division an element took 5 us a unit
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int gr = 0; gr < C::kGroups; ++gr)
#pragma unroll
                    for (int i = 0; i < 2; ++i) f[nt][gr][i] = __frcp_rn(f[nt][gr][i]);
        }
        const bool whole = b == 0 && e == cur.v.steps;
        const int64_t slot = part_slot(a, plan, cur, units, weight<C::kStep>(a, cur.v), b == 0, whole, recs);
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
                    if constexpr (FP8) x *= f[nt][k / 4][i & 1];
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
        advance<C::kStep>(a, units, cur, dx);
    }
    cp_wait<0>();
}

// Join the parts of the rows that more than one block (or piece) worked on.  A
// block joins a quarter of a unit's heads * D outputs: its warps first turn the
// parts' maxima and sums into weights (a warp per head), then its threads take
// four dims each and the parts in groups, added in the groups' order.
constexpr int kJoinThreads = 256, kJoinParts = kMaxCtas * kNumSMs;

__global__ void __launch_bounds__(kJoinThreads)
    paged_decode_join_kernel(const PagedDecodeArgs a, int hb, int heads, const JoinRec* recs, const float* slots) {
    __shared__ float wt[16 * kJoinParts / 4 + 2 * kJoinParts], inv[16];
    __shared__ float4 part[kJoinThreads];
    pdl_wait();
    const JoinRec r = recs[blockIdx.x];
    if (r.n == 0) return;
    const int D = a.D, G = a.H / a.HK, per = heads * (D + 2), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int hk = r.u / hb, head0 = (r.u % hb) * heads, n_heads = min(heads, G - head0);
    const int share = heads * D / 16, i0 = blockIdx.y * share;  // in groups of four dims
    const int h0 = i0 * 4 / D, h1 = min((i0 + share) * 4 / D + (share * 4 % D != 0), n_heads);  // heads of the share
    auto slot = [&](int q) { return slots + int64_t(q == 0 ? r.first : r.next + (q - 1) * r.by) * per; };
    for (int h = h0 + warp; h < h1; h += kJoinThreads / 32) {
        const float sg = a.sinks ? a.sinks[hk * G + head0 + h] * kLog2e : -INFINITY;
        float M = sg, L = 0.f;
        for (int q = lane; q < r.n; q += 32) M = fmaxf(M, slot(q)[2 * h]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        for (int q = lane; q < r.n; q += 32) {
            const float2 ml = *reinterpret_cast<const float2*>(slot(q) + 2 * h);
            const float x = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
            L += x * ml.y;  // (NaN stays NaN)
            wt[(h - h0) * r.n + q] = x;
        }
        L = warp_sum(L);
        if (sg != -INFINITY) L += ex2(sg - M);
        if (lane == 0) inv[h - h0] = L;
    }
    __syncthreads();
    const int groups = kJoinThreads / share, g = threadIdx.x / share, i = i0 + threadIdx.x % share;
    const int h = i * 4 / D;
    const bool on = g < groups && h < n_heads;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on) {
        const float* w = wt + (h - h0) * r.n;
#pragma unroll 4
        for (int q = g; q < r.n; q += groups) {
            const float2* p = reinterpret_cast<const float2*>(slot(q) + 2 * heads + 4 * i);
            const float2 x = p[0], y = p[1];
            if (w[q] != 0.f) {
                acc.x += w[q] * x.x; acc.y += w[q] * x.y;
                acc.z += w[q] * y.x; acc.w += w[q] * y.y;
            }
        }
    }
    part[threadIdx.x] = acc;
    __syncthreads();
    if (!on || g != 0) return;
    for (int k = 1; k < groups; ++k) {
        const float4 x = part[threadIdx.x + k * share];
        acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
    }
    const float L = inv[h - h0];
    const float y[4] = {acc.x / L, acc.y / L, acc.z / L, acc.w / L};
    const int64_t at = (int64_t(r.s) * a.H + hk * G + head0) * D + 4 * i;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float z = L == 0.f ? 0.f : y[k];
        if (a.act_fmt == CSA_F32) ((float*)a.out)[at + k] = z;
        else ((__nv_bfloat16*)a.out)[at + k] = __float2bfloat16_rn(z);
    }
}

// Heads of a group: 8, or 16 where more share a key head and the registers hold them.
static int group_heads(int H, int HK, int D) { return H / HK > 8 && D <= 128 ? 16 : 8; }

bool paged_decode_tc_supported(int act, int cache) {
    return act == CSA_BF16 && (cache == CSA_BF16 || cache == CSA_FP8_S64);
}

bool one_piece(const PagedDecodeArgs& a) {
    const int64_t most = a.max_pages * a.page_size;
    return (a.W > 0 ? std::min<int64_t>(a.W, most) : most) <= 256;
}

void set_page_division(PagedDecodeArgs* a) {
    int s = 0;
    while ((int64_t(1) << s) < a->page_size) ++s;
    a->page_mul = s ? uint32_t(((uint64_t(1) << (31 + s)) + a->page_size - 1) / a->page_size) : 0;
    a->page_shift = s ? s - 1 : 0;
}

DecodeLayout decode_layout(int H, int HK, int D, int64_t batch, int64_t n_ctx, bool invariant, int heads, int step) {
    DecodeLayout w;
    w.units = int64_t(HK) * ((H / HK + heads - 1) / heads);
    if (invariant) {
        const int64_t steps = ceil_div(n_ctx, step);
        w.recs = batch * w.units;
        w.slots = batch * w.units * std::min<int64_t>(64, ceil_div(steps, 512 / step) + 1);
    } else {
        w.recs = kMaxCtas * kNumSMs;
        w.slots = 2 * w.recs;
    }
    w.rec_bytes = (size_t(w.recs) * sizeof(JoinRec) + 255) & ~size_t(255);
    w.bytes = w.rec_bytes + size_t(w.slots) * heads * (D + 2) * sizeof(float);
    return w;
}

cudaError_t launch_paged_join(const PagedDecodeArgs& a, int64_t recs_n, int hb, int heads, const JoinRec* recs,
                              const float* slots, cudaStream_t s) {
    return launch_ex(paged_decode_join_kernel, dim3(unsigned(recs_n), 4), dim3(kJoinThreads), 0, s, true, a, hb, heads, recs,
                     slots);
}

constexpr int kStepTc = 64;

size_t paged_decode_workspace(int H, int HK, int D, int64_t batch, int64_t n_ctx, bool invariant) {
    return decode_layout(H, HK, D, batch, n_ctx, invariant, group_heads(H, HK, D), kStepTc).bytes;
}

template <int D, bool FP8, int NT>
static cudaError_t launch_decode(PagedDecodeArgs a, void* ws, cudaStream_t s) {
    using C = Dec<D, FP8, NT>;
    static_assert(C::kStages >= 2 && C::kStages <= 8, "stages");
    static_assert(C::kStep == kStepTc, "steps");
    const DecodeLayout w = decode_layout(a.H, a.HK, D, a.batch, a.max_pages * a.page_size, a.invariant, C::kHeads, C::kStep);
    const bool single = one_piece(a);
    if (single) a.invariant = 1;
    JoinRec* recs = single ? nullptr : (JoinRec*)ws;
    float* slots = (float*)((char*)ws + w.rec_bytes);
    const int hb = int(w.units / a.HK);
    cudaError_t e = ensure_smem(paged_decode_kernel<D, FP8, NT>, C::kSmem + kAlignSmem);
    if (e != cudaSuccess) return e;
    paged_decode_kernel<D, FP8, NT><<<C::kCtas * kNumSMs, 32 * kNW, C::kSmem + kAlignSmem, s>>>(a, int(w.units), hb, recs, slots);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (single) return cudaSuccess;
    return launch_paged_join(a, a.invariant ? w.recs : C::kCtas * kNumSMs, hb, C::kHeads, recs, slots, s);
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

cudaError_t launch_paged_decode_tc(const PagedDecodeArgs& args, void* ws, cudaStream_t s) {
    PagedDecodeArgs a = args;
    set_page_division(&a);
    return a.cache_fmt == CSA_FP8_S64 ? launch_decode_fmt<true>(a, ws, s) : launch_decode_fmt<false>(a, ws, s);
}

}  // namespace csa
